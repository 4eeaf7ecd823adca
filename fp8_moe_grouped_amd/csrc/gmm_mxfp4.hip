// Grouped product on microscaled 4-bit operands, for serving.  Row r of expert g
// is token slot_of_row[r] / topk (r itself without slot_of_row); x is quantized
// to MXFP4 once a token (launch_quant_rows_mxfp4), the weights are MXFP4 already:
//
//   y[r, n]   = sum over the blocks b of 32 k of 2^(ea + ew - 254) sum_{k in b} qa[k] qw[g, n, k]
//   out[r, n] = bf16(y[r, n]),  or with SwiGLU over columns [gate | up] of N = 2I:
//   out[r, i] = bf16( silu(y[r, i]) * y[r, I + i] )
//
// The scaled matrix instruction (32x32x64) applies the blocks' powers of two and
// accumulates in f32.  A lane's operand is 32 consecutive k of one row, which is one
// block with one scale byte.  The weight is the first operand, so a lane ends with
// four consecutive columns of one row.
#include "moe_common.hpp"
#include "moe_launch.hpp"
#include "mxfp4_plan.hpp"

#include <algorithm>
#include <type_traits>

namespace fp8gmm {
namespace {

// ---------------------------------------------------------------- schedule

// The experts' rows and tiles of BM rows, 64 experts at a time, one a lane.  Every
// wave finds its own tile in registers: the LDS table of build_group_table (one
// wave's shuffles, a barrier, a binary search) took 9400 cycles from the block's
// start to its tile's first address, this takes 3900 with up to 64 experts; with more,
// locate walks the sizes again.
template <int BM>
struct TileMap {
  int start, end, first, tiles;                     // the lane's expert: rows, first tile, tiles
  int total;                                        // tiles of all experts

  __device__ __forceinline__ void scan64(const int* __restrict__ group_sizes, int G, int M, int base, int& rows,
                                         int& before, int& flags) {
    const int g = base + (int)(threadIdx.x & 63);
    const int raw = g < G ? group_sizes[g] : 0;
    if (raw < 0) flags |= kDevNegativeSize;
    const int sz = min(max(raw, 0), M);             // M < 2^24: no overflow below
    const int last = rows + wave_scan_dpp(sz);
    if (raw > M || (last > M && sz > 0)) flags |= kDevSumClamped;
    start = min(last - sz, M);
    end = min(last, M);
    tiles = (end - start + BM - 1) / BM;
    const int upto = before + wave_scan_dpp(tiles);
    first = upto - tiles;
    rows = min(__builtin_amdgcn_readlane(last, 63), M);
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  __device__ __forceinline__ void scan(const int* __restrict__ group_sizes, int G, int M, int* status) {
    int rows = 0, before = 0, flags = 0;
    for (int base = 0; base < G; base += 64) scan64(group_sizes, G, M, base, rows, before, flags);
    total = before;
    if (status != nullptr && blockIdx.x == 0 && threadIdx.x < 64 && flags) atomicOr(status, flags);
  }
  // expert and place of tile mt < total: its expert's rows and its index among the expert's tiles
  __device__ __forceinline__ void locate(const int* __restrict__ group_sizes, int G, int M, int mt, int& g, int& g0,
                                         int& g1, int& part) {
    int rows = 0, before = 0, flags = 0;
    for (int base = 0; base < G; base += 64) {
      if (G > 64) scan64(group_sizes, G, M, base, rows, before, flags);   // scan left the last 64
      const uint64_t hit = __ballot(first <= mt && mt < first + tiles);
      if (hit == 0) continue;
      const int at = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
      g = base + at;
      g0 = __builtin_amdgcn_readlane(start, at);
      g1 = __builtin_amdgcn_readlane(end, at);
      part = mt - __builtin_amdgcn_readlane(first, at);
      return;
    }
  }
};

template <int SEL>
__device__ __forceinline__ v16f mfma_mxfp4_32(const v4i& a, const v4i& b, const v16f& c, int sa, int sb) {
  const v8i a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, SEL, sa, SEL, sb);
}

// Both kernels bring 256 k (a pair of stages of 128) of a row at a time: 128 bytes, one cache line, in eight
// 16-byte chunks whose place in LDS is turned with the row, so that reads of one chunk of 16 rows hit all banks.
constexpr int kLine = 128;
__device__ __forceinline__ int swz(int row, int chunk) { return row * kLine + ((chunk ^ ((row >> 1) & 7)) << 4); }

// Results leave through LDS as rows of COLS bf16 (16 bytes past a multiple of the banks), so that a store
// instruction writes whole lines: with 32 rows x 32 bytes straight from the fragments 8190 x 768 x 2048 took 38 us
// in the large tiles, with this 35.
//
// put16: 16 columns of a row from the two halves of a wave.  Lanes l and l + 32 hold the same row, columns
// 8q + 4h + 0..3 (h = lane / 32) as two words a[q], q = 0, 1, and trade them so that each writes 16 bytes.
template <int COLS>
constexpr int kOutRow = 2 * COLS + 16;
__device__ __forceinline__ void put16(uint8_t* p, int h, const v2i& a0, const v2i& a1) {
  const auto x = __builtin_amdgcn_permlane32_swap(a0[0], a1[0], false, false);
  const auto y = __builtin_amdgcn_permlane32_swap(a0[1], a1[1], false, false);
  *reinterpret_cast<v4i*>(p + 16 * h) = (v4i){(int)x[0], (int)y[0], (int)x[1], (int)y[1]};
}
// rows x COLS (the last ones cut off at column `end`) to out, whose rows are `ld` apart
template <int COLS>
__device__ __forceinline__ void store_rows(const uint8_t* lds, uint16_t* out, size_t ld, int rows, int end) {
  constexpr int C = COLS / 8;
  const int c = threadIdx.x % C;
  if (8 * c >= end) return;
  for (int r = threadIdx.x / C; r < rows; r += 256 / C)
    *reinterpret_cast<v4i*>(out + r * ld + 8 * c) = *reinterpret_cast<const v4i*>(lds + r * kOutRow<COLS> + 16 * c);
}
__device__ __forceinline__ v2i pack4(float a, float b, float c, float d) {
  return (v2i){(int)pack_bf16x2(a, b), (int)pack_bf16x2(c, d)};
}
__device__ __forceinline__ float silu_mul(float gate, float up) {   // hardware reciprocal: rounded to bf16 right after
  return gate * __builtin_amdgcn_rcpf(1.0f + __expf(-gate)) * up;
}

// ---------------------------------------------------------------- few rows

// Bound by the weights' bytes: a block streams 128 columns of one expert (SwiGLU: 64
// gate and the matching 64 up) past up to 32 * MI of its rows.  Copies to LDS, a pair
// a row (contiguous lines, streaming policy for the weights: 7.1 TB/s alone, where
// operand loads of 16 rows x 64 bytes reach 6.1), into a ring of three slots (two
// with 128 rows, so that two blocks still share a CU).  A wave multiplies 32 columns, SwiGLU 16
// gate and their 16 up in one fragment, so that a lane ends with both.
template <int MI>
constexpr int kRing = MI <= 2 ? 3 : 2;

template <int MI, bool SWIGLU>
__global__ __launch_bounds__(256, 2) void gmm_mxfp4_stream_kernel(
    const uint8_t* __restrict__ aq, const uint8_t* __restrict__ ascale, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ wscale, const int* __restrict__ group_sizes, const int* __restrict__ slot_of_row,
    int topk, int T, int G, int M, int K, int N, uint16_t* __restrict__ out, int* status) {
  constexpr int BM = 32 * MI, BN = 128;
  constexpr int kScales = 2 * 4 * 256;              // a wave's words of its rows and of its columns
  constexpr int kSlot = (BM + BN) * kLine + kScales;
  constexpr int kLoads = MI + 6;                    // a wave's copies of a pair
  constexpr int R = kRing<MI>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  TileMap<BM> map;
  map.scan(group_sizes, G, M, status);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = map.total, half = N >> 1, n_tiles = N / BN;
  if ((int)blockIdx.x >= tiles * n_tiles) return;
  // Blocks go round the eight XCDs; each takes a run of tiles, a column tile's row tiles one after the other, so that
  // weights that several row tiles read pass through one L2.
  const int total = tiles * n_tiles, xcd = blockIdx.x % 8;
  const int at = xcd * (total / 8) + min(xcd, total % 8) + blockIdx.x / 8;
  const int mt = at % tiles, nt = at / tiles;
  int g = 0, g0 = 0, g1 = 0, tile = 0;
  map.locate(group_sizes, G, M, mt, g, g0, g1, tile);
  const int row0 = g0 + tile * BM, rows = min(BM, g1 - row0);

  const int kw = K / 128, np = (kw + 1) / 2;
  const uint32_t abytes = (uint32_t)K / 2, sbytes = (uint32_t)((kw + 3) / 4) * 16;
  const BufRsrc rb = make_rsrc(codes + (size_t)g * N * abytes, (uint32_t)N * abytes);
  const BufRsrc rsb = make_rsrc(wscale + (size_t)g * kw * N * 4, (uint32_t)kw * (uint32_t)N * 4u);
  auto column = [&](int c) {                        // column of tile column c
    if (!SWIGLU) return nt * BN + c;
    const int at = nt * 64 + (c >> 5) * 16 + (c & 15);
    return c & 16 ? half + at : at;
  };
  uint32_t vb[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = 32 * wave + 8 * j + (lane >> 3);
    vb[j] = (uint32_t)column(c) * abytes + (uint32_t)(((lane & 7) ^ ((c >> 1) & 7)) << 4);
  }
  const uint32_t vsb = ((uint32_t)(lane >> 5) * (uint32_t)N + (uint32_t)column(32 * wave + (lane & 31))) * 4u;
  auto copy_weights = [&](int p, uint8_t* slot) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, LDS_PTR(void, slot + BM * kLine + (4 * wave + j) * 1024), 16, vb[j],
                                               (uint32_t)p * kLine, 0, kCpolStream);
    dma4(rsb, slot + (BM + BN) * kLine + 1024 + wave * 256, vsb, (uint32_t)p * (uint32_t)N * 8u);
  };
  // A wave brings 8 * MI rows; rows past the tile's end repeat its last.  Loads return in order, so the slots are
  // asked for before the weights.
  const int row = row0 + min(8 * MI * wave + min(lane, 8 * MI - 1), rows - 1);
  const int slot_in = slot_of_row ? slot_of_row[row] : row;
  sched_fence();
  copy_weights(0, smem);
  sched_fence();
  int token = row;
  if (slot_of_row) token = slot_in < 0 ? T : min(slot_in / topk, T);   // row T of the quantized activations is zero
  const uint8_t* va[MI];
#pragma unroll
  for (int j = 0; j < MI; ++j) {
    const int r = 8 * (MI * wave + j) + (lane >> 3);
    va[j] = aq + (size_t)__shfl(token, 8 * j + (lane >> 3)) * abytes + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  const uint8_t* const vsa = ascale + (size_t)__shfl(token, (lane >> 1) & (8 * MI - 1)) * sbytes + 4 * (lane & 1);
  auto copy_rows = [&](int p, uint8_t* slot) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < MI; ++j) copy16(va[j] + (size_t)p * kLine, slot + (MI * wave + j) * 1024);
    copy4(vsa + 8 * p, slot + (BM + BN) * kLine + wave * 256);
  };
  copy_rows(0, smem);
  if (np > 1) {
    copy_weights(1, smem + kSlot);
    copy_rows(1, smem + kSlot);
  }

  const int h = lane >> 5, r32 = lane & 31, bcol = 32 * wave + r32;
  v16f acc[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
  int cur = 0, ahead = 2 % R;                       // slots of pair p and of pair p + 2
  // LEFT: pairs after this one, 2 standing for more.
  auto step = [&](int p, auto left_c) __attribute__((always_inline)) {
    constexpr int LEFT = decltype(left_c)::value;
    if (LEFT > 0) wait_vmem_lds<kLoads>();          // pair p is there, pair p + 1 on its way
    else wait_vmem_lds<0>();
    barrier_only();                                 // and every wave has read pair p - 1
    auto copy_ahead = [&]() __attribute__((always_inline)) {
      copy_weights(p + 2, smem + ahead * kSlot);
      copy_rows(p + 2, smem + ahead * kSlot);
    };
    if (R == 3 && LEFT > 1) copy_ahead();
    const uint8_t* const slot = smem + cur * kSlot;
    const uint8_t* const sc = slot + (BM + BN) * kLine;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (2 * p + u >= kw) break;                   // an odd K / 128 ends in half a pair
      const int xb = *reinterpret_cast<const int*>(sc + 1024 + wave * 256 + (32 * u + r32) * 4) >> (8 * h);
      v4i b[2], a[MI][2];
      int xa[MI];
#pragma unroll
      for (int s = 0; s < 2; ++s) b[s] = *reinterpret_cast<const v4i*>(slot + BM * kLine + swz(bcol, 4 * u + 2 * s + h));
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int r = 32 * i + r32;
        xa[i] = *reinterpret_cast<const int*>(sc + r / (8 * MI) * 256 + (2 * (r % (8 * MI)) + u) * 4) >> (8 * h);
#pragma unroll
        for (int s = 0; s < 2; ++s) a[i][s] = *reinterpret_cast<const v4i*>(slot + swz(r, 4 * u + 2 * s + h));
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i] = mfma_mxfp4_32<0>(b[0], a[i][0], acc[i], xb, xa[i]);
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i] = mfma_mxfp4_32<2>(b[1], a[i][1], acc[i], xb, xa[i]);
    }
    if (R == 2 && LEFT > 1) {                       // the slot that was just read
      wait_vmem_lds<63>();
      barrier_only();
      copy_ahead();
    }
    cur = cur == R - 1 ? 0 : cur + 1;
    ahead = ahead == R - 1 ? 0 : ahead + 1;
  };
  int p = 0;
  for (; p + 2 < np; ++p) step(p, std::integral_constant<int, 2>{});
  if (p + 1 < np) step(p++, std::integral_constant<int, 1>{});
  step(p, std::integral_constant<int, 0>{});

  // a lane holds row 32 i + r32, columns 8q + 4h + 0..3 of its wave's 32
  constexpr int COLS = SWIGLU ? 64 : 128;
  static_assert(BM * kOutRow<COLS> <= kSlot, "the results fit one slot");
  wait_vmem_lds<0>();
  barrier_only();                                   // every wave has read the last pair
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const v16f& c = acc[i];
    uint8_t* const o = smem + (32 * i + r32) * kOutRow<COLS>;
    if (SWIGLU) {
      v2i v[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        v[q] = pack4(silu_mul(c[4 * q], c[4 * q + 8]), silu_mul(c[4 * q + 1], c[4 * q + 9]),
                     silu_mul(c[4 * q + 2], c[4 * q + 10]), silu_mul(c[4 * q + 3], c[4 * q + 11]));
      put16(o + 32 * wave, h, v[0], v[1]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; q += 2)
        put16(o + 64 * wave + 16 * q, h, pack4(c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]),
              pack4(c[4 * q + 4], c[4 * q + 5], c[4 * q + 6], c[4 * q + 7]));
    }
  }
  __syncthreads();
  const size_t ld = SWIGLU ? half : N;
  store_rows<COLS>(smem, out + row0 * ld + nt * COLS, ld, rows, COLS);
}

// ---------------------------------------------------------------- large tiles

// Many rows: a block owns up to 256 rows x 256 columns (SwiGLU: 128 gate and the
// matching 128 up) of one expert.  Four waves, one per SIMD, 2 x 2: with 128 x 128
// a wave the operands read from LDS stay below its bandwidth (64 KB a stage of 128
// k against 1024 cycles of matrix instructions; eight waves of 64 x 128 would read
// 96 KB beside the 32 KB that arrive).  An expert's rows are cut into tiles of
// nearly equal counts of 64 rows, and a wave's instructions follow the tile's
// count (MI fragments of 32 rows): at K = 7168 a loop of 84000 cycles for 256 rows
// and 66000, the copies' time, for 64.
//
// 20000 x 7168 x 4096 over 32 skewed experts: 360 to 375 us with the quantizer, 3.1
// to 3.3 PFLOP/s.  A stage takes 1475 cycles at a clock that the power limit holds
// near 1.9 GHz; its matrix instructions alone take 1140, its copies alone 1040 when
// all lines are in L2.
//
// The contraction advances 128 k a stage; buffer loads with the LDS destination
// bring two stages (a pair: 128 bytes, one cache line, a row) at a time into one of
// two slots.  While a stage's matrix instructions issue from one register set, the
// next stage's operands are read into the other, and the copies of the pair two
// ahead go to the slot that was just read.  Scale words (four blocks of 32 k)
// arrive two pairs at a time.
constexpr int BM = 256, BN = 256;
constexpr int kSlotBytes = (BM + BN) * kLine;
constexpr int kRingBytes = 2 * kSlotBytes;
constexpr int kScaleSlot = BM * 16 + 4 * BN * 4;    // four stages' scale words, rows then columns
constexpr int kTileLds = kRingBytes + 2 * kScaleSlot;
static_assert(kTileLds <= 160 * 1024, "ring and scales fit the LDS");

template <bool SWIGLU>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1)))
void gmm_mxfp4_tile_kernel(const uint8_t* __restrict__ aq, const uint8_t* __restrict__ ascale,
                           const uint8_t* __restrict__ codes, const uint8_t* __restrict__ wscale,
                           const int* __restrict__ group_sizes, const int* __restrict__ slot_of_row, int topk, int T,
                           int G, int M, int K, int N, uint16_t* __restrict__ out, int* status) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  TileMap<BM> map;
  map.scan(group_sizes, G, M, status);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int half = N >> 1;
  const int n_tiles = SWIGLU ? half / (BN / 2) : (N + BN - 1) / BN;
  const int tiles = map.total;
  if ((int)blockIdx.x >= tiles * n_tiles) return;
  int mt, nt;
  raster_tile<4>(blockIdx.x, tiles, n_tiles, mt, nt);   // 389 us against 395 with groups of 8 and 401 with 16
  int g = 0, g0 = 0, g1 = 0, part = 0;
  map.locate(group_sizes, G, M, mt, g, g0, g1, part);
  // this tile's share of the expert's units of 64 rows
  const int parts = (g1 - g0 + BM - 1) / BM, units = (g1 - g0 + 63) / 64;
  const int u0 = first_unit(units, parts, part), u1 = first_unit(units, parts, part + 1);
  const int row0 = g0 + 64 * u0, rows = min(64 * (u1 - u0), g1 - row0);

  const int kw = K / 128, nk = kw;
  const uint32_t abytes = (uint32_t)K / 2, sbytes = (uint32_t)((kw + 3) / 4) * 16;
  const BufRsrc ra = make_rsrc(aq, (uint32_t)(T + 1) * abytes);      // below 2^32 (the launcher's rule)
  const BufRsrc rsa = make_rsrc(ascale, (uint32_t)(T + 1) * sbytes);
  const BufRsrc rb = make_rsrc(codes + (size_t)g * N * abytes, (uint32_t)N * abytes);
  const BufRsrc rsb = make_rsrc(wscale + (size_t)g * kw * N * 4, (uint32_t)kw * (uint32_t)N * 4u);
  auto slot_of = [&](int r) {                       // rows past the tile's end repeat its last
    const int row = row0 + min(r, rows - 1);
    return slot_of_row ? slot_of_row[row] : row;
  };
  auto token_of = [&](int slot) {
    return !slot_of_row ? slot : slot < 0 ? T : min(slot / topk, T);
  };
  auto column = [&](int c) {                        // column of tile column c (past N: past the buffer's end)
    return SWIGLU ? (c < BN / 2 ? nt * (BN / 2) + c : half + nt * (BN / 2) + c - BN / 2) : nt * BN + c;
  };

  auto run = [&](auto mi_c) __attribute__((always_inline)) {
    constexpr int MI = decltype(mi_c)::value;       // the tile has up to 64 * MI rows, a wave 32 * MI
    constexpr int kLoads = 2 * MI + 8;              // a wave's copies of a pair, without the scales
    uint32_t va[2 * MI], vb[8], vsa, vsb;
    // Loads return in order: the slots are asked for first, and the first columns copied while they come.
    const int slot_copy = slot_of(16 * MI * wave + min(lane, 16 * MI - 1)), slot_scale = slot_of(64 * wave + lane);
    sched_fence();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (8 * wave + j) * 8 + (lane >> 3);
      vb[j] = (uint32_t)column(c) * abytes + (uint32_t)(((lane & 7) ^ ((c >> 1) & 7)) << 4);
    }
    vsb = ((uint32_t)wave * (uint32_t)N + (uint32_t)column(4 * lane)) * 4u;
    auto copy = [&](int p, int u, int q) __attribute__((always_inline)) {    // copy q of pair p into slot u
      uint8_t* const s = smem + u * kSlotBytes;
      if (q < 2 * MI) dma16(ra, s + (2 * MI * wave + q) * 1024, va[q], (uint32_t)p * kLine);
      else dma16(rb, s + BM * kLine + (8 * wave + q - 2 * MI) * 1024, vb[q - 2 * MI], (uint32_t)p * kLine);
    };
    auto copy_scales = [&](int ks, bool rows_, bool columns) __attribute__((always_inline)) {
      uint8_t* const s = smem + kRingBytes + ((ks >> 2) & 1) * kScaleSlot;   // of stages ks .. ks + 3, ks a multiple of 4
      if (rows_) dma16(rsa, s + wave * 1024, vsa, (uint32_t)ks * 4u);
      if (columns) dma16(rsb, s + BM * 16 + wave * 1024, vsb, (uint32_t)ks * (uint32_t)N * 4u);
    };
    copy_scales(0, false, true);
#pragma unroll
    for (int q = 2 * MI; q < kLoads; ++q) copy(0, 0, q);
    sched_fence();
    const int mine = token_of(slot_copy);           // a lane has a row's token
#pragma unroll
    for (int j = 0; j < 2 * MI; ++j) {
      const int r = (2 * MI * wave + j) * 8 + (lane >> 3);
      va[j] = (uint32_t)__shfl(mine, 8 * j + (lane >> 3)) * abytes + (uint32_t)(((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
    vsa = (uint32_t)token_of(slot_scale) * sbytes;

    const int h = lane >> 5, r32 = lane & 31;
    int arow[MI], bcol[4];
#pragma unroll
    for (int i = 0; i < MI; ++i) arow[i] = wm * 32 * MI + 32 * i + r32;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      bcol[j] = (SWIGLU ? (j < 2 ? wn * 64 + 32 * j : 128 + wn * 64 + 32 * (j - 2)) : wn * 128 + 32 * j) + r32;
    v4i a[2][MI][2], b[2][4][2];
    int sa[2][MI], sb[2][4];
    // one of the kReads LDS reads of stage ks, ks % 4 = u, into register set u & 1
    constexpr int kReads = 3 * (4 + MI);
    auto read = [&](auto u_c, int ks, int q) __attribute__((always_inline)) {
      constexpr int u = decltype(u_c)::value, S = u & 1;
      const uint8_t* slot = smem + (u >> 1) * kSlotBytes;
      const uint8_t* sc = smem + kRingBytes + ((ks >> 2) & 1) * kScaleSlot;
      const int f = q / 3, s = q % 3;               // fragment, then its two halves and its scales
      if (f < 4) {
        if (s < 2) b[S][f][s] = *reinterpret_cast<const v4i*>(slot + BM * kLine + swz(bcol[f], 4 * S + 2 * s + h));
        else sb[S][f] = *reinterpret_cast<const int*>(sc + BM * 16 + (u * BN + bcol[f]) * 4);
      } else {
        if (s < 2) a[S][f - 4][s] = *reinterpret_cast<const v4i*>(slot + swz(arow[f - 4], 4 * S + 2 * s + h));
        else sa[S][f - 4] = *reinterpret_cast<const int*>(sc + arow[f - 4] * 16 + 4 * u);
      }
    };

    v16f acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    // ---- prologue: pairs 0 and 1 in flight, stage 0 in registers
    copy_scales(0, true, false);
#pragma unroll
    for (int q = 0; q < 2 * MI; ++q) copy(0, 0, q);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) copy(1, 1, q);  // K >= 1024 here: four pairs or more
    wait_vmem_lds<kLoads>();
    barrier_only();
#pragma unroll
    for (int q = 0; q < kReads; ++q) read(std::integral_constant<int, 0>{}, 0, q);

    // One stage, ks % 4 = U: its operands are in register set U & 1.  MAIN: four more stages follow.
    // The scale words are shifted to the lane's blocks (h, 2 + h) where they are used, so that
    // nothing waits for the reads of the next stage.  A SIMD has one wave, which issues in order: the
    // next stage's reads and the copies stand one by one between the matrix instructions and issue
    // while those run.
    auto step = [&](int ks, auto u_c, auto main_c) __attribute__((always_inline)) {
      constexpr int U = decltype(u_c)::value, S = U & 1;
      constexpr bool MAIN = decltype(main_c)::value;
      using Next = std::integral_constant<int, (U + 1) & 3>;
      // In a pair's second stage every wave has read that pair: its slot takes the pair two ahead,
      // and the next pair (the only copies in flight) has to be there.
      const bool more = MAIN || ks + 1 < nk, ahead = S == 1 && (MAIN || ks + 3 < nk);
      if (S == 1 && more) {
        wait_vmem_lds<0>();
        barrier_only();
      }
      int xa[MI], xb[4];
#pragma unroll
      for (int i = 0; i < MI; ++i) xa[i] = sa[S][i] >> (8 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) xb[j] = sb[S][j] >> (8 * h);
      constexpr int kSlots = 8 * MI;                // matrix instructions; the copies go out in the first three quarters
      constexpr int kOut = U == 1 ? kLoads + 2 : U == 3 ? kLoads : 0;
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        const int s = t / (4 * MI), j = t / MI % 4, i = t % MI;
        if (s == 0) acc[i][j] = mfma_mxfp4_32<0>(b[S][j][0], a[S][i][0], acc[i][j], xb[j], xa[i]);
        else acc[i][j] = mfma_mxfp4_32<2>(b[S][j][1], a[S][i][1], acc[i][j], xb[j], xa[i]);
        if (ahead) {
#pragma unroll
          for (int o = t * kOut / (6 * MI); o < min((t + 1) * kOut / (6 * MI), kOut); ++o) {
            if (o < kLoads) copy((ks + 3) >> 1, U >> 1, o);
            else if (o == kLoads) copy_scales(ks + 3, true, true);
          }
        }
        if (more) {
#pragma unroll
          for (int o = t * kReads / (kSlots - 1); o < min((t + 1) * kReads / (kSlots - 1), kReads); ++o)
            read(Next{}, ks + 1, o);
        }
        sched_fence();
      }
    };
    using U0 = std::integral_constant<int, 0>;
    using U1 = std::integral_constant<int, 1>;
    using U2 = std::integral_constant<int, 2>;
    using U3 = std::integral_constant<int, 3>;
    int ks = 0;
    for (; ks + 7 < nk; ks += 4) {
      step(ks, U0{}, std::true_type{});
      step(ks + 1, U1{}, std::true_type{});
      step(ks + 2, U2{}, std::true_type{});
      step(ks + 3, U3{}, std::true_type{});
    }
    for (; ks < nk; ks += 4) {                      // the last one to seven stages
      step(ks, U0{}, std::false_type{});
      if (ks + 1 < nk) step(ks + 1, U1{}, std::false_type{});
      if (ks + 2 < nk) step(ks + 2, U2{}, std::false_type{});
      if (ks + 3 < nk) step(ks + 3, U3{}, std::false_type{});
    }

    // ---- epilogue: a lane holds row arow[i], columns 8q + 4h + 0..3 of each fragment
    constexpr int COLS = SWIGLU ? BN / 2 : BN;
    static_assert(BM * kOutRow<COLS> <= kTileLds, "the results fit the LDS");
    wait_vmem_lds<0>();
    barrier_only();                                 // every wave has read the last stage
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int j = 0; j < (SWIGLU ? 2 : 4); ++j) {
        v2i pq[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = acc[i][j][4 * q + e];
            v[e] = SWIGLU ? silu_mul(y, acc[i][(j + 2) & 3][4 * q + e]) : y;
          }
          pq[q] = pack4(v[0], v[1], v[2], v[3]);
        }
        uint8_t* const o = smem + arow[i] * kOutRow<COLS> + COLS * wn + 64 * j;
        put16(o, h, pq[0], pq[1]);
        put16(o + 32, h, pq[2], pq[3]);
      }
    }
    __syncthreads();
    const size_t ld = SWIGLU ? half : N;
    store_rows<COLS>(smem, out + row0 * ld + nt * COLS, ld, rows, SWIGLU ? COLS : min(COLS, N - nt * BN));
  };
  if (rows > 192) run(std::integral_constant<int, 4>{});
  else if (rows > 128) run(std::integral_constant<int, 3>{});
  else if (rows > 64) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 1>{});
}

}  // namespace

template <int MI>
static hipError_t launch_stream(const uint8_t* aq, const uint8_t* ascale, const uint8_t* codes, const uint8_t* wscale,
                                const int* group_sizes, const int* slot_of_row, int topk, int T, int G, int M, int K,
                                int N, bool swiglu, uint16_t* out, int* status, hipStream_t stream) {
  const long long tiles = std::min<long long>(M, ((long long)M + 32 * MI - 1) / (32 * MI) + G);
  const dim3 grid((unsigned)(tiles * (N / 128)));
  const size_t lds = std::min(kRing<MI>, (K + 255) / 256) * ((32 * MI + 128) * kLine + 2048);   // a slot a pair at most
  if (swiglu)
    hipLaunchKernelGGL((gmm_mxfp4_stream_kernel<MI, true>), grid, dim3(256), lds, stream, aq, ascale, codes, wscale,
                       group_sizes, slot_of_row, topk, T, G, M, K, N, out, status);
  else
    hipLaunchKernelGGL((gmm_mxfp4_stream_kernel<MI, false>), grid, dim3(256), lds, stream, aq, ascale, codes, wscale,
                       group_sizes, slot_of_row, topk, T, G, M, K, N, out, status);
  return hipGetLastError();
}

hipError_t launch_gmm_mxfp4(const uint8_t* aq, const uint8_t* ascale, const uint8_t* codes, const uint8_t* wscale,
                            const int* group_sizes, const int* slot_of_row, int topk, int T, int G, int M, int K,
                            int N, bool swiglu, uint16_t* out, int* status, hipStream_t stream) {
#define STREAM(MI)                                                                                                  \
  launch_stream<MI>(aq, ascale, codes, wscale, group_sizes, slot_of_row, topk, T, G, M, K, N, swiglu, out, status, \
                    stream)
  const int rows = mxfp4_tile_rows(T, G, M, K, N);
  if (rows == 32) return STREAM(1);
  if (rows == 64) return STREAM(2);
  if (rows == 128) return STREAM(4);
#undef STREAM
  const long long tiles = std::min<long long>(M, ((long long)M + BM - 1) / BM + G);
  if (swiglu)
    hipLaunchKernelGGL(gmm_mxfp4_tile_kernel<true>, dim3((unsigned)(tiles * (N / 256))), dim3(256), kTileLds, stream, aq,
                       ascale, codes, wscale, group_sizes, slot_of_row, topk, T, G, M, K, N, out, status);
  else
    hipLaunchKernelGGL(gmm_mxfp4_tile_kernel<false>, dim3((unsigned)(tiles * ((N + 255) / 256))), dim3(256), kTileLds,
                       stream, aq, ascale, codes, wscale, group_sizes, slot_of_row, topk, T, G, M, K, N, out, status);
  return hipGetLastError();
}

}  // namespace fp8gmm
