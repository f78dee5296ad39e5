// Launch shapes of the layer operators (csrc/arx_shapes.h) for ctypes.
#include "arx_shapes.h"

extern "C" {

// out[0] the cut, out[1] splits, out[2] one split's depth, out[3] tiles.
void cut_of(uint32_t m, uint32_t n, uint32_t k, int a_rows_k, int b_rows_k, int as_is, uint64_t* out) {
  const arx::Shape s = arx::shape_of(m, n, k, a_rows_k, b_rows_k, as_is);
  const arx::CutCost& c = arx::kCost[s.cut];
  out[0] = (uint64_t)s.cut;
  out[1] = s.splits;
  out[2] = s.depth;
  out[3] = (uint64_t)arx::cdiv(m, c.tm) * arx::cdiv(n, c.tn);
}

int paired(uint32_t m, uint32_t n, uint32_t k) { return arx::worth_pairing(m, n, k); }

// out[0] lanes across, out[1] and out[2] the grid.
void columns_of(uint32_t rows, uint32_t cols, int sums, uint64_t* out) {
  const arx::ColumnShape s = arx::column_shape(rows, cols, sums);
  out[0] = (uint64_t)1 << s.lg;
  out[1] = s.x;
  out[2] = s.y;
}
}
