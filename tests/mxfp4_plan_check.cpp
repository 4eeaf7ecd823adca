// Host check of csrc/mxfp4_plan.hpp.  With arguments T G M K N: prints the rows of the tiles that the launcher takes.
// Without: an expert's units of 64 rows (at most 2^24 - 1 rows) cut into tiles of
// up to 256 rows that follow each other from unit 0 to the last, each of one to four units, their
// sizes at most one unit apart.  Prints "ok", or the first count that breaks this.
#include <cstdio>
#include <cstdlib>

#include "../fp8_moe_grouped_amd/csrc/mxfp4_plan.hpp"

static bool whole(int units) {
  const int parts = (units + 3) / 4;
  int most = 0, least = 4;
  if (fp8gmm::first_unit(units, parts, 0) != 0 || fp8gmm::first_unit(units, parts, parts) != units) return false;
  for (int p = 0; p < parts; ++p) {
    const int n = fp8gmm::first_unit(units, parts, p + 1) - fp8gmm::first_unit(units, parts, p);
    most = n > most ? n : most;
    least = n < least ? n : least;
  }
  return least >= 1 && most <= 4 && most - least <= 1;
}

int main(int argc, char** argv) {
  if (argc == 6) {
    int v[5];
    for (int i = 0; i < 5; ++i) v[i] = std::atoi(argv[i + 1]);
    return std::printf("%d\n", fp8gmm::mxfp4_tile_rows(v[0], v[1], v[2], v[3], v[4])), 0;
  }
  constexpr int kMost = ((1 << 24) - 1 + 63) / 64;
  for (int units = 1; units <= kMost; units += units < 4096 ? 1 : units < 90000 ? 1237 : 4999)
    if (!whole(units)) return std::printf("units %d\n", units), 1;
  for (int units = kMost - 8; units <= kMost; ++units)
    if (!whole(units)) return std::printf("units %d\n", units), 1;
  std::printf("ok\n");
  return 0;
}
