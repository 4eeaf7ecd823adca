// How the 4-bit product's large tiles cut an expert's rows: integer arithmetic that
// the kernel and its CPU test share (constexpr functions run on both sides).
#pragma once

namespace fp8gmm {

// First unit of 64 rows of tile `part` of an expert whose `units` units make `parts` tiles, 0 <= part <= parts:
// every tile has units / parts of them, the first units % parts tiles one more.  (units * part would pass 2^31
// at 5.9 million rows.)
constexpr int first_unit(int units, int parts, int part) {
  const int more = units % parts;
  return units / parts * part + (part < more ? part : more);
}

}  // namespace fp8gmm
