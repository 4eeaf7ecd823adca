// How the 4-bit product cuts its work: integer arithmetic that the kernels, the launcher
// and the CPU test share (constexpr functions run on both sides).
#pragma once

namespace fp8gmm {

// First unit of 64 rows of tile `part` of an expert whose `units` units make `parts` tiles, 0 <= part <= parts:
// every tile has units / parts of them, the first units % parts tiles one more.  (units * part would pass 2^31
// at 5.9 million rows.)
constexpr int first_unit(int units, int parts, int part) {
  const int more = units % parts;
  return units / parts * part + (part < more ? part : more);
}

// Rows of the kernel's tiles: 32, 64 or 128 of the stream kernel, 256 of the large tiles.  The sizes of the groups
// are not known to the launcher: about M / rows + G / 2 row tiles.  Measured in us with 32, 64, 128 and 256 rows (the
// count of large tiles in brackets):
//   7168 x 4096, 32 experts: 4 rows an expert 70 / 74 / 88 / 93, 16 rows 86 / 83 / 92 / 97, 64 rows 172 / 146 / 131 / 133
//   few tiles: 697 rows, 4 experts, 4352 x 1792 (42) 21 / 17 / 21 / 33; 1144 rows, 5 experts, 1536 x 3328 (104)
//   15 / 16 / 14 / 19; 3092 rows, 5 experts, 3840 x 1536 (90) 43 / 37 / 34 / 35; 2746 rows, 3 experts, 6528 x 2560 (120)
//   107 / 77 / 58 / 55; 7143 rows, 8 experts, 5504 x 3584 (448) 315 / 222 / 169 / 103
//   two pairs are over before a large tile's loads and stores overlap anything: 5412 rows, 7 experts, 384 x 3840 (375)
//   34 / 27 / 25 / 27
// No shape of more than 32 experts is among them.
constexpr long long mxfp4_blocks(int G, int M, int N, int rows, int columns) {
  return (long long)(M / rows + (G + 1) / 2) * ((N + columns - 1) / columns);
}
constexpr int mxfp4_tile_rows(int T, int G, int M, int K, int N) {
  const bool many = M >= 64 * (long long)G;
  // the large tiles have 32-bit offsets to the rows of the quantized tokens, of which there are T + 1
  if (many && K >= 1024 && mxfp4_blocks(G, M, N, 256, 256) >= 120 && ((long long)T + 1) * (K / 2) < (1LL << 32)) return 256;
  if (many && mxfp4_blocks(G, M, N, 128, 128) >= 200) return 128;
  return M > 24 * (long long)G && mxfp4_blocks(G, M, N, 64, 128) >= 100 ? 64 : 32;
}

}  // namespace fp8gmm
