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
