// AdamW over many tensors at once, in place, with f32 states or with states in 8 bits.
//
//   g  = grad * grad_scale
//   m' = b1 m + (1 - b1) g,   v' = b2 v + (1 - b2) g^2
//   p' = p - (lr wd p + lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps))
//
// The tensors' pointers travel in the kernel's arguments, kMost of them a launch, so that a
// call copies nothing and can be captured.
//
// 8-bit states: m and r = sqrt(v) as e4m3 codes, a scale for each 256 consecutive elements.
// 32 lanes hold such a block, 8 elements each, so its new scale is a reduction over their
// registers.  Codes are rounded up or down by chance: at beta2 = 0.999 a step changes
// r by 0.05 % and m by 10 %, half a step of e4m3 is 3 to 6 %, so the nearest code would
// keep r where it started.  r and not v is held because e4m3's 2^18 between its largest and
// smallest number would be 2^9 in r.  The mean of r is kept, so v = r^2 gains the rounding's
// variance at each step: with steady gradients 5 % at beta2 = 0.999.  An r' above 0 gets the
// smallest code at least: the next update would otherwise be divided by eps alone.
#include "moe_common.hpp"
#include "moe_launch.hpp"

#include <type_traits>

namespace fp8gmm {
namespace {

constexpr int kBlock = 256;                         // elements that share a scale
constexpr int kThreads = 256;
constexpr int kMost = 48;                           // tensors a launch
constexpr long long kMostBlocks = 1LL << 30;        // blocks a launch; a tensor has at most 2^25
constexpr int kVec = 4;                             // elements a lane, f32 states
constexpr int kVec8 = 8;                            // 8-bit states

struct State32 {
  float* m;
  float* v;
};
struct State8 {
  uint8_t *m, *r;
  float *ms, *rs;
};
template <typename S>
struct Tensor {
  int64_t size;
  void* p;
  const void* g;
  S state;
};
template <typename S>
struct Tensors {
  int count, first;                                 // the first one's place in the list
  uint32_t blocks[kMost];                           // before the next tensor's first block
  Tensor<S> at[kMost];
};
static_assert(sizeof(Tensors<State8>) + sizeof(AdamW) <= 4096, "kernel arguments");

struct Rates {
  float b1, c1, b2, c2, eps, decay, up, root, scale;
};
// The step's coefficients.  Those of a step or rate on the device are computed here, by every thread: they are the
// host's, in f64 and rounded once.  Beside the loads they are free where HBM has most to do (8 experts of 2048 x 1536 and
// 768 x 2048 f32 193 us with the host's, 195 with the device's); 38M bf16 elements with 8-bit states 76.5 and 81.5.
__device__ __forceinline__ Rates rates(const AdamW& a, uint32_t& step) {
  Rates r{a.b1, a.c1, a.b2, a.c2, a.eps, a.decay, a.up, a.root, a.grad_scale ? *a.grad_scale : 1.f};
  int64_t t = a.step;
  if (a.step_dev || a.lr_dev) {
    if (a.step_dev) t = max((int64_t)1, *a.step_dev);
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    r.decay = (float)(lr * a.weight_decay);
    r.up = (float)(lr / one_minus_power(a.log_beta1, t));
    r.root = (float)(1.0 / sqrt(one_minus_power(a.log_beta2, t)));
  }
  step = (uint32_t)__builtin_amdgcn_readfirstlane((int)t);
  return r;
}

// Pieces of a larger buffer begin anywhere; the widest accesses need an element's alignment only.
typedef float any4f __attribute__((ext_vector_type(4), aligned(4)));
typedef int any2i __attribute__((ext_vector_type(2), aligned(1)));

// N = 4 or 8 elements at j of n, streamed.  Without FULL those past the end are 0 and not written.
template <bool FULL, int N>
__device__ __forceinline__ void load(const float* p, int64_t j, int64_t n, float (&x)[N]) {
  if constexpr (FULL) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const any4f w = __builtin_nontemporal_load(reinterpret_cast<const any4f*>(p + j + i));
#pragma unroll
      for (int c = 0; c < 4; ++c) x[i + c] = w[c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = j + i < n ? p[j + i] : 0.f;
  }
}
template <bool FULL, int N>
__device__ __forceinline__ void load(const uint16_t* p, int64_t j, int64_t n, float (&x)[N]) {
  if constexpr (FULL) {
    typedef int vec __attribute__((ext_vector_type(N / 2), aligned(2)));
    const vec w = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p + j));
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i & 1 ? bf16_hi((uint32_t)w[i / 2]) : bf16_lo((uint32_t)w[i / 2]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = j + i < n ? __uint_as_float((uint32_t)p[j + i] << 16) : 0.f;
  }
}
template <bool FULL, int N>
__device__ __forceinline__ void store(float* p, int64_t j, int64_t n, const float (&x)[N]) {
  if constexpr (FULL) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      __builtin_nontemporal_store((any4f){x[i], x[i + 1], x[i + 2], x[i + 3]}, reinterpret_cast<any4f*>(p + j + i));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (j + i < n) p[j + i] = x[i];
  }
}
template <bool FULL, int N>
__device__ __forceinline__ void store(uint16_t* p, int64_t j, int64_t n, const float (&x)[N]) {
  if constexpr (FULL) {
    typedef int vec __attribute__((ext_vector_type(N / 2), aligned(2)));
    vec w;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = (int)pack_bf16x2(x[2 * i], x[2 * i + 1]);
    __builtin_nontemporal_store(w, reinterpret_cast<vec*>(p + j));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (j + i < n) p[j + i] = (uint16_t)pack_bf16x2(x[i], 0.f);
  }
}
// 8 codes.
template <bool FULL>
__device__ __forceinline__ v2i load_codes(const uint8_t* p, int64_t j, int64_t n) {
  if constexpr (FULL) return __builtin_nontemporal_load(reinterpret_cast<const any2i*>(p + j));
  v2i w = {0, 0};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (j + i < n) w[i / 4] |= (int)((uint32_t)p[j + i] << (8 * (i & 3)));
  return w;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t j, int64_t n, v2i w) {
  if constexpr (FULL) {
    __builtin_nontemporal_store((any2i)w, reinterpret_cast<any2i*>(p + j));
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (j + i < n) p[j + i] = (uint8_t)((uint32_t)w[i / 4] >> (8 * (i & 3)));
}

// sqrt(x), correctly rounded, for 2^-96 <= x < inf: a step of Goldschmidt's iteration, which refines the root and half its
// reciprocal together from an approximate reciprocal root, and one of Newton's with the remainder x - s^2.  From 2^-96 on
// s^2 is a multiple of 2^-144 and the remainder exact; below 2^-102 it need no longer be an f32 number.
__device__ __forceinline__ float usual_root(float x) {
  const float r = __builtin_amdgcn_rsqf(x);
  float s = x * r, h = 0.5f * r;
  const float e = __builtin_fmaf(-h, s, 0.5f);
  s = __builtin_fmaf(s, e, s);
  h = __builtin_fmaf(h, e, h);
  return __builtin_fmaf(__builtin_fmaf(-s, s, x), h, s);
}
template <int N>
__device__ __forceinline__ void roots(const float (&x)[N], float (&r)[N]) {
  constexpr uint32_t kLeast = 0x0F800000u, kPast = 0x7F800000u;   // 2^-96, inf
  uint32_t furthest = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    furthest = max(furthest, __float_as_uint(x[i]) - kLeast);
    r[i] = usual_root(x[i]);
  }
  if (furthest >= kPast - kLeast)                   // zeros, tiny ones, infinities, NaN
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = sqrtf(x[i]);
}

// N elements: p, m, v become their next values and r the roots of v; v comes as b2 times its old value.  Every product
// and sum rounds by itself: a step of another program in f32 then chooses the same codes, which would otherwise part by
// a whole step of theirs wherever a sum's last bit decides.  p's quotient alone is a product with a reciprocal (2^-23).
template <int N>
__device__ __forceinline__ void update(const Rates& a, float (&g)[N], float (&p)[N], float (&m)[N], float (&v)[N],
                                       float (&r)[N]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    g[i] = g[i] * a.scale;
    m[i] = a.b1 * m[i] + a.c1 * g[i];
    v[i] = v[i] + a.c2 * g[i] * g[i];
  }
  roots<N>(v, r);
#pragma unroll
  for (int i = 0; i < N; ++i)
    p[i] = p[i] - (a.decay * p[i] + a.up * m[i] * __builtin_amdgcn_rcpf(r[i] * a.root + a.eps));
}

// The tensor of this block and the block's place in it; -1 for a block past the last one.  Arguments come from far on
// their first use, so that a search would wait for each step: every lane looks at one tensor.
static_assert(kMost <= 64, "a lane a tensor");
template <typename S>
__device__ __forceinline__ int tensor_of(const Tensors<S>& all, uint32_t& block) {
  const int lane = threadIdx.x & 63;
  block = (uint32_t)linear_block();
  const uint32_t end = all.blocks[min(lane, kMost - 1)];
  const int i = __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane < all.count && block >= end));
  if (i == all.count) return -1;
  if (i > 0) block -= (uint32_t)__builtin_amdgcn_readlane((int)end, i - 1);
  return i;
}

// Bound by HBM: 28 bytes an element in f32, at 6 TB/s with streaming accesses (8 x 2048 x 1536 and 8 x 768 x 2048 in
// 177 us, with ordinary ones 203; four times 4 elements a thread instead of one 187).
template <typename TP, typename TG>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Tensors<State32> all, const AdamW how) {
  uint32_t block;
  const int i = tensor_of(all, block);
  if (i < 0) return;
  const int64_t n = all.at[i].size, j = ((int64_t)block * kThreads + threadIdx.x) * kVec;
  if (j >= n) return;
  const Tensor<State32> to = all.at[i];
  TP* const p = static_cast<TP*>(to.p);
  // one branch for all accesses: behind one for each, a load waits for the last one
  const auto run = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    float pv[kVec], gv[kVec], mv[kVec], vv[kVec], rv[kVec];
    load<FULL>(p, j, n, pv);
    load<FULL>(static_cast<const TG*>(to.g), j, n, gv);
    load<FULL>(to.state.m, j, n, mv);
    load<FULL>(to.state.v, j, n, vv);
    uint32_t step;
    const Rates a = rates(how, step);               // while the loads are on their way
#pragma unroll
    for (int c = 0; c < kVec; ++c) vv[c] *= a.b2;
    update<kVec>(a, gv, pv, mv, vv, rv);
    store<FULL>(p, j, n, pv);
    store<FULL>(to.state.m, j, n, mv);
    store<FULL>(to.state.v, j, n, vv);
  };
  if (j + kVec <= n) run(std::true_type{});
  else run(std::false_type{});
}

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// New codes and the scale of x's block, which 32 lanes hold.  The conversion adds the upper 20 of its random bits to the
// mantissa's 20 that e4m3 lacks (below 2^-6, to the distance's fraction) and cuts them off: floor(|q| / d + u) d.  The
// bits are 16 b + 8, so u = (b + 1/2) / 2^16 and 448, a few roundings off, does not leave its code.
template <bool POSITIVE>
__device__ __forceinline__ v2i hold(const float (&x)[kVec8], const uint32_t (&random)[kVec8], float& scale) {
  const auto larger = [](uint32_t a, uint32_t b) { return max(a, b); };
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < kVec8; ++c) top = max(top, __float_as_uint(x[c]) & 0x7FFFFFFFu);
  top = reduce<16>(top, larger);
  top = max(top, other_rows<16>(top, (threadIdx.x & 16) != 0));
  scale = top < 0x7F800000u ? __uint_as_float(top) * (1.f / kE4M3Max) : __builtin_nanf("");
  const float inverse = 1.f / scale;
  float q[kVec8];
  // a number above 0 counts as the smallest code's at least, which is then its code
#pragma unroll
  for (int c = 0; c < kVec8; ++c)
    q[c] = POSITIVE && x[c] > 0.f ? __builtin_fmaxf(x[c] * inverse, 0x1p-9f) : x[c] * inverse;
  if (!(scale > 0x1p-120f)) {                       // zeros, scales whose reciprocal is past f32, NaN
#pragma unroll
    for (int c = 0; c < kVec8; ++c) {
      q[c] = scale > 0.f ? __builtin_fmaxf(__builtin_fminf(x[c] / scale, kE4M3Max), -kE4M3Max) : 0.f;
      if (POSITIVE && q[c] > 0.f) q[c] = __builtin_fmaxf(q[c], 0x1p-9f);
    }
  }
  v2i out;
#pragma unroll
  for (int c = 0; c < kVec8; c += 4) {
    int w = __builtin_amdgcn_cvt_sr_fp8_f32(q[c], (int)random[c], 0, 0);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(q[c + 1], (int)random[c + 1], w, 1);
    w = __builtin_amdgcn_cvt_sr_fp8_f32(q[c + 2], (int)random[c + 2], w, 2);
    out[c / 4] = __builtin_amdgcn_cvt_sr_fp8_f32(q[c + 3], (int)random[c + 3], w, 3);
  }
  return out;
}

// Bound by HBM: 16 bytes an element with f32 parameters and gradients, 5.3 TB/s (8 x 7168 x 4096 and 8 x 2048 x 7168 in
// 1060 us).  With bf16 ones, 10 bytes, its 67 instructions an element count as much: 38M elements in 73 us, 5.2 TB/s.  It
// had 87 and took 80 to 85 when codes were made with integers (11 instructions a state; the conversion is one), the key's
// mixing was not scalar and the coefficients came in f64; with 4 elements a lane and divisions 104.  Ten small tensors
// 6.6 us: the wave of a tensor's end goes both ways, and its elements' loads, behind a condition each, wait for one another.
template <typename TP, typename TG>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(const Tensors<State8> all, const uint64_t seed,
                                                          const AdamW how) {
  static_assert(kBlock == 32 * kVec8, "32 lanes hold a block");
  uint32_t block;
  const int i = tensor_of(all, block);
  if (i < 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t n = all.at[i].size, b = (int64_t)block * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t j = b * kBlock + lane * kVec8;
  if (b * kBlock >= n) return;                      // all 32 lanes
  const Tensor<State8> to = all.at[i];
  const State8 s = to.state;
  TP* const p = static_cast<TP*>(to.p);
  uint32_t step = 0;
  float pv[kVec8], gv[kVec8], mv[kVec8], rv[kVec8], vv[kVec8];
  const auto begin = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    load<FULL>(p, j, n, pv);
    load<FULL>(static_cast<const TG*>(to.g), j, n, gv);
    const v2i mw = load_codes<FULL>(s.m, j, n), rw = load_codes<FULL>(s.r, j, n);
    const float ms = s.ms[b], rs = s.rs[b];
    const Rates a = rates(how, step);
#pragma unroll
    for (int c = 0; c < kVec8; c += 4) {
      const v2f m0 = dec_e4m3x2<false>(mw[c / 4]), m1 = dec_e4m3x2<true>(mw[c / 4]);
      const v2f r0 = dec_e4m3x2<false>(rw[c / 4]), r1 = dec_e4m3x2<true>(rw[c / 4]);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        mv[c + d] = (d < 2 ? m0[d & 1] : m1[d & 1]) * ms;
        const float r = (d < 2 ? r0[d & 1] : r1[d & 1]) * rs;
        vv[c + d] = a.b2 * r * r;
      }
    }
    update<kVec8>(a, gv, pv, mv, vv, rv);
    store<FULL>(p, j, n, pv);
  };
  const bool whole = j + kVec8 <= n;
  if (whole) begin(std::true_type{});
  else begin(std::false_type{});
  const uint32_t key = mix(mix((uint32_t)seed + mix((uint32_t)(seed >> 32) + mix(step))) + (uint32_t)(all.first + i));
  const uint32_t of_block = mix(key + (uint32_t)b) + 0x9E3779B9u * (uint32_t)(lane * kVec8);
  uint32_t low[kVec8], high[kVec8];
#pragma unroll
  for (int c = 0; c < kVec8; ++c) {
    const uint32_t h = mix(of_block + 0x9E3779B9u * (uint32_t)c);
    low[c] = h << 16 | 0x8000u;
    high[c] = (h & 0xFFFF0000u) | 0x8000u;
  }
  float mscale, rscale;
  const v2i mw = hold<false>(mv, low, mscale), rw = hold<true>(rv, high, rscale);
  if (whole) {
    store_codes<true>(s.m, j, n, mw);
    store_codes<true>(s.r, j, n, rw);
  } else {
    store_codes<false>(s.m, j, n, mw);
    store_codes<false>(s.r, j, n, rw);
  }
  if (lane == 0) {
    s.ms[b] = mscale;
    s.rs[b] = rscale;
  }
}

// Launches of up to kMost tensors: state(i) is a tensor's, run(tensors, grid) launches.
template <typename S, int kChunk, typename F, typename R>
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
    all.at[c] = {sizes[i], params[i], grads[i], state(i)};
    const bool last = i + 1 == tensors;
    if (last || all.count == kMost || blocks + (sizes[i + 1] + kChunk - 1) / kChunk >= kMostBlocks) {
      if (blocks > 0) {
        const hipError_t st = run(all, linear_grid(blocks));
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
  return in_turns<State32, kThreads * kVec>(
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
  return in_turns<State8, kThreads * kVec8>(
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
