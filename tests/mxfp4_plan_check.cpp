// Host check of csrc/mxfp4_plan.hpp: an expert's units of 64 rows (at most 2^24 - 1 rows) cut into tiles of
// up to 256 rows.  Tiles follow each other from unit 0 to the last, each of one to four units, their sizes
// at most one unit apart.  Prints "ok", or the first count that breaks this.
#include <cstdio>

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

int main() {
  constexpr int kMost = ((1 << 24) - 1 + 63) / 64;
  for (int units = 1; units <= kMost; units += units < 4096 ? 1 : units < 90000 ? 1237 : 4999)
    if (!whole(units)) return std::printf("units %d\n", units), 1;
  for (int units = kMost - 8; units <= kMost; ++units)
    if (!whole(units)) return std::printf("units %d\n", units), 1;
  std::printf("ok\n");
  return 0;
}
