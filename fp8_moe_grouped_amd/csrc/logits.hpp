// A token's router logits in the lanes that share it (routing and the balance losses): L = 16 lanes (four
// tokens a wave) or the wave, V logits a lane in chunks of 16 bytes.
#pragma once
#include "moe_common.hpp"

namespace fp8gmm {

__device__ __forceinline__ float load_logit(const float* x) { return *x; }
__device__ __forceinline__ float load_logit(const uint16_t* x) { return __uint_as_float((uint32_t)*x << 16); }

// Lane `at` of the L that share a token holds the experts of chunks at, at + L, ..: C logits each (16 bytes).
template <int L, int C>
__device__ __forceinline__ int expert_of(int at, int i) { return (i / C * L + at) * C + i % C; }

// A token's logits as loaded, 16 bytes a chunk: nothing waits for them before unpack().
template <int V, typename TX>
struct Chunks {
  v4i w[V * (int)sizeof(TX) / 16];
};

// MASKED ? -inf : 0 past the experts and, with `here` false, everywhere.
template <int L, int V, bool MASKED, typename TX>
__device__ __forceinline__ void load_chunks(const TX* row, int E, int at, bool here, bool wide, Chunks<V, TX>& x) {
  constexpr int C = 16 / (int)sizeof(TX);
  constexpr uint32_t kNone = !MASKED ? 0u : C == 4 ? 0xFF800000u : 0xFF80u;
  constexpr int kFill = (int)(C == 4 ? kNone : kNone << 16 | kNone);
#pragma unroll
  for (int j = 0; j < V / C; ++j) x.w[j] = (v4i){kFill, kFill, kFill, kFill};
  if (wide) {                                       // E is a multiple of C: a chunk is inside or outside
#pragma unroll
    for (int j = 0; j < V / C; ++j) {
      const int e = expert_of<L, C>(at, j * C);
      if (here && e < E) x.w[j] = *reinterpret_cast<const v4i*>(row + e);
    }
  } else if (here) {                                // one branch: behind one for each, a load waits for the last one
    uint32_t v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const TX u = row[min(expert_of<L, C>(at, i), E - 1)];
      if constexpr (C == 4) v[i] = __float_as_uint(u);
      else v[i] = u;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = expert_of<L, C>(at, i) < E ? v[i] : kNone;
#pragma unroll
    for (int j = 0; j < V / C; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x.w[j][c] = (int)(C == 4 ? v[4 * j + c] : v[8 * j % V + 2 * c] | v[8 * j % V + 2 * c + 1] << 16);
  }
}
template <int V, typename TX>
__device__ __forceinline__ void unpack(const Chunks<V, TX>& y, float (&x)[V]) {
  constexpr int C = 16 / (int)sizeof(TX);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t w = (uint32_t)y.w[i / C][C == 4 ? i % 4 : i % 8 / 2];
    x[i] = C == 4 ? __uint_as_float(w) : i & 1 ? bf16_hi(w) : bf16_lo(w);
  }
}
// The same as values at once, 0 for none.
template <int L, int V, typename TX>
__device__ __forceinline__ void load_logits(const TX* row, int E, int at, bool here, bool wide, float (&x)[V]) {
  constexpr int C = 16 / (int)sizeof(TX);
  if (wide) {                                       // E is a multiple of C: a chunk is inside or outside
#pragma unroll
    for (int i = 0; i < V; i += C) {
      const int e = expert_of<L, C>(at, i);
      const v4i w = here && e < E ? *reinterpret_cast<const v4i*>(row + e) : (v4i){0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < C; ++c)
        x[i + c] = C == 4 ? __uint_as_float((uint32_t)w[c % 4])
                          : (c & 1 ? bf16_hi((uint32_t)w[c / 2 % 4]) : bf16_lo((uint32_t)w[c / 2 % 4]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert_of<L, C>(at, i);
      x[i] = here && e < E ? load_logit(row + e) : 0.f;
    }
  }
}

// A row of the lanes' values, rounded once to the logits' type.
template <int L, int V, typename TX>
__device__ __forceinline__ void store_logits(TX* row, int E, int at, bool wide, const float (&d)[V]) {
  constexpr int C = 16 / (int)sizeof(TX);
#pragma unroll
  for (int i = 0; i < V; i += C) {
    const int e = expert_of<L, C>(at, i);
    uint32_t o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      o[c] = C == 4 ? __float_as_uint(d[i + c]) : pack_bf16x2(d[i + C / 4 * c], d[i + C / 4 * c + 1]);
    if (wide) {
      if (e < E) *reinterpret_cast<v4i*>(row + e) = (v4i){(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (e + c < E) {
          if constexpr (C == 4) row[e + c] = d[i + c];
          else row[e + c] = (TX)(o[c / 2] >> (16 * (c & 1)));
        }
    }
  }
}

}  // namespace fp8gmm
