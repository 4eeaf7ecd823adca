// AdamW over many tensors at once, in place, with f32 states or with states in 8 bits.
//
//   g  = grad * grad_scale
//   m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g^2
//   p' = p - (lr wd p + lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps))
//
// The tensors' pointers travel in the kernel's arguments, kMost of them a launch, so that a
// call copies nothing and can be captured.  A block finds its tensor among the prefix sums
// of their blocks.
//
// 8-bit states: m and r = sqrt(v) as e4m3 codes, a scale for each 256 consecutive elements.
// A wave holds such a block, 4 elements a lane, so its new scale is a reduction over the
// wave's registers.  Codes are rounded up or down by chance: at beta2 = 0.999 a step changes
// r by 0.05 % and m by 10 %, half a step of e4m3 is 3 to 6 %, so the nearest code would
// keep r where it started.  r and not v is held because e4m3's 2^18 between its largest and
// smallest number would be 2^9 in r.  An r' above 0 gets the smallest code at least: the
// next update would otherwise be divided by eps alone.
#include "moe_common.hpp"
#include "moe_launch.hpp"

#include <algorithm>

namespace fp8gmm {
namespace {

constexpr int kBlock = 256;                         // elements that share a scale
constexpr int kThreads = 256;
constexpr int kMost = 48;                           // tensors a launch
constexpr int kVec = 4;                             // elements a lane at a time
constexpr int kPer = 4;                             // times
constexpr int kChunk = kThreads * kVec * kPer;      // elements a block

struct State32 {
  float* m;
  float* v;
};
struct State8 {
  uint8_t *m, *r;
  float *ms, *rs;
};
template <typename S>
struct Tensors {
  int count, first;                                 // the first one's place in the list
  uint32_t blocks[kMost];                           // before the next tensor's first block
  int64_t size[kMost];
  void* p[kMost];
  const void* g[kMost];
  S state[kMost];
};
static_assert(sizeof(Tensors<State8>) + sizeof(AdamW) <= 4096, "kernel arguments");

struct Rates {
  float b1, c1, b2, c2, eps, decay, up, root, scale;
};
__device__ __forceinline__ double power(double b, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1, b *= b) r = n & 1 ? r * b : r;
  return r;
}
// The step's coefficients.  Those of a step on the device are computed here, by every block: some 20 rounds of
// three f64 products.
__device__ __forceinline__ Rates rates(const AdamW& a, int64_t& step) {
  step = a.step_dev ? max((int64_t)1, *a.step_dev) : a.step;
  Rates r{(float)a.beta1, (float)(1.0 - a.beta1), (float)a.beta2, (float)(1.0 - a.beta2), (float)a.eps,
          (float)a.decay, (float)a.up, (float)a.root, a.grad_scale ? *a.grad_scale : 1.f};
  if (a.step_dev || a.lr_dev) {
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    r.decay = (float)(lr * a.weight_decay);
    r.up = (float)(lr / (1.0 - power(a.beta1, step)));
    r.root = 1.f / sqrtf((float)(1.0 - power(a.beta2, step)));
  }
  return r;
}

__device__ __forceinline__ v4f load4(const float* p) { return *reinterpret_cast<const v4f*>(p); }
__device__ __forceinline__ v4f load4(const uint16_t* p) {
  const v2i w = *reinterpret_cast<const v2i*>(p);
  return (v4f){bf16_lo((uint32_t)w[0]), bf16_hi((uint32_t)w[0]), bf16_lo((uint32_t)w[1]), bf16_hi((uint32_t)w[1])};
}
__device__ __forceinline__ void store4(float* p, v4f v) { *reinterpret_cast<v4f*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, v4f v) {
  *reinterpret_cast<v2i*>(p) = (v2i){(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.f); }

// Up to 4 elements at j of n; those past the end are 0 and not written.
template <typename T>
__device__ __forceinline__ v4f load_some(const T* p, int64_t j, int64_t n) {
  if (j + 4 <= n) return load4(p + j);
  v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (j + i < n) v[i] = load1(p + j + i);
  return v;
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int64_t j, int64_t n, v4f v) {
  if (j + 4 <= n) return store4(p + j, v);
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (j + i < n) store1(p + j + i, v[i]);
}
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t j, int64_t n) {
  if (j + 4 <= n) return *reinterpret_cast<const uint32_t*>(p + j);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (j + i < n) w |= (uint32_t)p[j + i] << (8 * i);
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t j, int64_t n, uint32_t w) {
  if (j + 4 <= n) {
    *reinterpret_cast<uint32_t*>(p + j) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (j + i < n) p[j + i] = (uint8_t)(w >> (8 * i));
}

// One element: p, m, v become their next values.  old_v is b2 * v.  Every product
// and sum rounds by itself: a step of another program in f32 then chooses the same codes, which would otherwise part
// by a whole step of theirs wherever a sum's last bit decides.
__device__ __forceinline__ void update(const Rates& a, float g, float old_v, float& p, float& m, float& v, float& r) {
#pragma clang fp contract(off)
  g = g * a.scale;
  m = a.b1 * m + a.c1 * g;
  v = old_v + a.c2 * g * g;
  r = sqrtf(v);
  p = p - (a.decay * p + a.up * m / (r * a.root + a.eps));
}
__device__ __forceinline__ float square(float b2, float r) {
#pragma clang fp contract(off)
  return b2 * r * r;
}

// The tensor of a block and the block's place in it.
template <typename S>
__device__ __forceinline__ int tensor_of(const Tensors<S>& all, uint32_t& block) {
  int lo = 0, hi = all.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (block < all.blocks[mid]) hi = mid;
    else lo = mid + 1;
  }
  if (lo > 0) block -= all.blocks[lo - 1];
  return lo;
}

template <typename TP, typename TG>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Tensors<State32> all, const AdamW how) {
  uint32_t block = blockIdx.x;
  const int i = tensor_of(all, block);
  const int64_t n = all.size[i];
  TP* const p = static_cast<TP*>(all.p[i]);
  const TG* const g = static_cast<const TG*>(all.g[i]);
  float *const m = all.state[i].m, *const v = all.state[i].v;
  int64_t step;
  const Rates a = rates(how, step);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t j = (int64_t)block * kChunk + (u * kThreads + (int)threadIdx.x) * kVec;
    if (j >= n) return;
    v4f pv = load_some(p, j, n), gv = load_some(g, j, n), mv = load_some(m, j, n), vv = load_some(v, j, n);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float pe = pv[c], me = mv[c], ve, re;
      update(a, gv[c], a.b2 * vv[c], pe, me, ve, re);
      pv[c] = pe;
      mv[c] = me;
      vv[c] = ve;
    }
    store_some(p, j, n, pv);
    store_some(m, j, n, mv);
    store_some(v, j, n, vv);
  }
}

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// |q| up to 448 to e4m3's grid, up or down by chance: floor(|q| / d + u) d, u = (bits + 1/2) / 2^16.  For a
// normal number the 20 mantissa bits that e4m3 lacks are |q| / d's fraction, so u is added to them and they are
// cut off.  Below 2^-6 the distance is 2^-9, which 2^-6 added to |q| makes that of the first normal numbers.
__device__ __forceinline__ float by_chance(float q, uint32_t bits) {
  const float low = q < 0x1p-6f ? 0x1p-6f : 0.f;
  const uint32_t w = (__float_as_uint(q + low) + (bits << 4 | 8)) & ~0xFFFFFu;
  return __builtin_fminf(__uint_as_float(w) - low, kE4M3Max);
}

// New codes and the scale of the wave's block of x.  bits: the element's 16 random ones.
template <bool POSITIVE>
__device__ __forceinline__ uint32_t hold(const v4f x, const uint32_t (&bits)[4], float& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) top = max(top, __float_as_uint(x[c]) & 0x7FFFFFFFu);
  top = reduce<64>(top, [](uint32_t a, uint32_t b) { return max(a, b); });
  scale = top < 0x7F800000u ? __uint_as_float(top) * (1.f / kE4M3Max) : __builtin_nanf("");
  const bool some = scale > 0.f;
  const float inverse = 1.f / scale;
  const bool normal = inverse < __builtin_inff();   // of a scale below 2^-128 it is not
  float q[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    q[c] = some ? by_chance(__builtin_fminf(normal ? __builtin_fabsf(x[c]) * inverse : __builtin_fabsf(x[c]) / scale, kE4M3Max), bits[c]) : 0.f;
    if (POSITIVE) q[c] = some && x[c] > 0.f ? __builtin_fmaxf(q[c], 0x1p-9f) : q[c];
    else q[c] = __builtin_copysignf(q[c], x[c]);
  }
  return cvt_e4m3x4(q[0], q[1], q[2], q[3]);
}

template <typename TP, typename TG>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(const Tensors<State8> all, const uint64_t seed,
                                                          const AdamW how) {
  uint32_t block = blockIdx.x;
  const int i = tensor_of(all, block);
  const int64_t n = all.size[i];
  TP* const p = static_cast<TP*>(all.p[i]);
  const TG* const g = static_cast<const TG*>(all.g[i]);
  const State8 s = all.state[i];
  int64_t step;
  const Rates a = rates(how, step);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t key = mix(mix((uint32_t)seed + mix((uint32_t)(seed >> 32) + mix((uint32_t)step))) +
                           (uint32_t)(all.first + i));
  static_assert(kBlock == 64 * kVec, "a wave holds a block");
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t b = (int64_t)block * (kChunk / kBlock) + u * (kThreads / 64) + wave, j = b * kBlock + lane * kVec;
    if (b * kBlock >= n) return;                    // the whole wave
    v4f pv = load_some(p, j, n), gv = load_some(g, j, n);
    const uint32_t mw = load_codes(s.m, j, n), rw = load_codes(s.r, j, n);
    const float ms = s.ms[b], rs = s.rs[b];
    const v2f m0 = dec_e4m3x2<false>(mw), m1 = dec_e4m3x2<true>(mw);
    const v2f r0 = dec_e4m3x2<false>(rw), r1 = dec_e4m3x2<true>(rw);
    v4f mv = {m0[0] * ms, m0[1] * ms, m1[0] * ms, m1[1] * ms};
    v4f rv = {r0[0] * rs, r0[1] * rs, r1[0] * rs, r1[1] * rs};
    const uint32_t kb = mix(key + (uint32_t)b);
    uint32_t low[4], high[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t h = mix(kb + 0x9E3779B9u * (uint32_t)(lane * kVec + c));
      low[c] = h & 0xFFFFu;
      high[c] = h >> 16;
      float pe = pv[c], me = mv[c], ve, re;
      update(a, gv[c], square(a.b2, rv[c]), pe, me, ve, re);
      pv[c] = pe;
      mv[c] = me;
      rv[c] = re;
    }
    store_some(p, j, n, pv);
    float mscale, rscale;
    store_codes(s.m, j, n, hold<false>(mv, low, mscale));
    store_codes(s.r, j, n, hold<true>(rv, high, rscale));
    if (lane == 0) {
      s.ms[b] = mscale;
      s.rs[b] = rscale;
    }
  }
}

// Launches of up to kMost tensors: state(i) is a tensor's, run(tensors, grid) launches.
template <typename S, typename F, typename R>
hipError_t in_turns(int tensors, const int64_t* sizes, void* const* params, const void* const* grads, F state, R run) {
  Tensors<S> all;
  long long blocks = 0;
  all.count = 0;
  for (int i = 0; i < tensors; ++i) {
    const long long more = (sizes[i] + kChunk - 1) / kChunk;
    if (all.count == 0) all.first = i;
    const int c = all.count++;
    blocks += more;
    all.blocks[c] = (uint32_t)blocks;
    all.size[c] = sizes[i];
    all.p[c] = params[i];
    all.g[c] = grads[i];
    all.state[c] = state(i);
    // a launch has fewer than 2^32 threads, a tensor at most 2^23 blocks
    const bool last = i + 1 == tensors;
    if (last || all.count == kMost || blocks + (sizes[i + 1] + kChunk - 1) / kChunk >= (1LL << 24)) {
      if (blocks > 0) {
        const hipError_t st = run(all, dim3((unsigned)blocks));
        if (st != hipSuccess) return st;
      }
      all.count = 0;
      blocks = 0;
    }
  }
  return hipSuccess;
}

#define BY_TYPES(RUN)                                   \
  if (param_bf16) {                                     \
    if (grad_bf16) RUN(uint16_t, uint16_t);             \
    else RUN(uint16_t, float);                          \
  } else {                                              \
    if (grad_bf16) RUN(float, uint16_t);                \
    else RUN(float, float);                             \
  }

}  // namespace

hipError_t launch_adamw(int tensors, const int64_t* sizes, void* const* params, bool param_bf16,
                        const void* const* grads, bool grad_bf16, float* const* m, float* const* v, const AdamW& how,
                        hipStream_t stream) {
  return in_turns<State32>(
      tensors, sizes, params, grads, [&](int i) { return State32{m[i], v[i]}; },
      [&](const Tensors<State32>& all, dim3 grid) {
#define RUN(P, G) hipLaunchKernelGGL((adamw_kernel<P, G>), grid, dim3(kThreads), 0, stream, all, how)
        BY_TYPES(RUN)
#undef RUN
        return hipGetLastError();
      });
}

hipError_t launch_adamw8(int tensors, const int64_t* sizes, void* const* params, bool param_bf16,
                         const void* const* grads, bool grad_bf16, uint8_t* const* m_codes, float* const* m_scales,
                         uint8_t* const* r_codes, float* const* r_scales, uint64_t seed, const AdamW& how,
                         hipStream_t stream) {
  return in_turns<State8>(
      tensors, sizes, params, grads,
      [&](int i) { return State8{m_codes[i], r_codes[i], m_scales[i], r_scales[i]}; },
      [&](const Tensors<State8>& all, dim3 grid) {
#define RUN(P, G) hipLaunchKernelGGL((adamw8_kernel<P, G>), grid, dim3(kThreads), 0, stream, all, seed, how)
        BY_TYPES(RUN)
#undef RUN
        return hipGetLastError();
      });
}

}  // namespace fp8gmm
