// arx_shapes.h — launch shapes of the layer operators: how a product is cut
// into tiles (arx_linear.hip) and a plane into columns (arx_rows.hip). Host
// arithmetic on sizes alone, without HIP, so that it can be checked without a
// GPU.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace arx {

constexpr uint32_t cdiv(uint32_t a, uint32_t b) { return a / b + (a % b != 0); }

// ---- matrix products --------------------------------------------------------

constexpr int kDepth = 64;   // of a tile's step

// How a product is cut: the kernel, and workgroups along the depth.
enum Cut { ROWS16, ROWS32, T64x64, T64x128, T128x128, T256x256, CUTS };
struct Shape {
  int cut;
  uint32_t splits;
  uint32_t depth;   // of one split, a multiple of 64
  float cost;       // microseconds
};

constexpr uint32_t kCus = 256;

// What a cut costs, in microseconds: a launch, a 64-deep step of a workgroup
// that waits for its loads, the same step where the CU is kept busy, and a
// workgroup's start and end; `resident` workgroups share a CU. A split product
// pays for its partial sums and their joining. The numbers are a least-squares
// fit to the times of 1100 cuts of 240 products (1 to 8192 rows, widths and
// depths of 256 to 8192, the three layouts) on an MI355X; the cut with the
// least cost by them is on average 1.5 % slower than the fastest one measured.
// A step of the few-rows kernel grows with the rows of A that it reads again in
// every workgroup, and beside it the tiles' cost is taken higher, as measured
// where all of B comes from memory (90 products, 1 to 32 rows).
struct CutCost {
  float launch, wait, busy, group;
  uint32_t tm, tn, resident;
};
constexpr CutCost kCost[CUTS] = {{2.3f, 0.100f, 0.105f, 0.42f, 16, 16, 2},
                                 {2.3f, 0.100f, 0.105f, 0.42f, 32, 16, 2},
                                 {3.1f, 0.264f, 0.202f, 1.0f, 64, 64, 2},
                                 {3.2f, 0.437f, 0.329f, 1.6f, 64, 128, 2},
                                 {3.4f, 0.657f, 0.498f, 2.4f, 128, 128, 2},
                                 {0.0f, 1.224f, 1.242f, 11.2f, 256, 256, 1}};
constexpr float kRowOfA[T64x64] = {0.02f, 0.033f}, kColdTiles = 1.15f;
constexpr float kJoin = 1.7f, kJoinRows = 3.0f, kJoinSplit = 0.24f, kJoinBytes = 0.25e-6f;

// as_is: the tiles can load both operands where they lie.
inline Shape shape_of(uint32_t m, uint32_t n, uint32_t k, bool a_rows_k, bool b_rows_k, bool as_is) {
  const uint32_t steps = cdiv(k ? k : 1, kDepth);
  Shape best{T64x64, 1, steps * kDepth, 0.0f};
  // Up to 32 rows of A, B can stream past once: one row, 4096 x 4096, 10.8 us
  // against 13.3 in tiles; 32 rows, 4096 x 1024, 6.6 and 8.7. The tiles catch up
  // where A or B is larger (16 rows, 32000 x 2048, 36.0 and 28.3; 32 rows,
  // 4096 x 4096, 16.8 and 13.6). Copying B for the tiles costs more than they
  // save up to 16 rows (5001 x 2001, 23.4 and 24.8), not past them.
  const bool across = !a_rows_k && !b_rows_k;
  const int rows = across && m <= 16 ? ROWS16 : across && m <= 32 && as_is ? ROWS32 : CUTS;
  for (int c = rows < CUTS ? rows : T64x64; c < (rows == ROWS16 && !as_is ? T64x64 : CUTS); ++c) {
    if (c < T64x64 && c != rows) continue;
    const CutCost& t = kCost[c];
    const float per_step = c < T64x64 ? 1.0f + kRowOfA[c] * (float)m : 1.0f;
    const uint64_t tiles = (uint64_t)cdiv(m, t.tm) * cdiv(n, t.tn);
    for (uint32_t s : {1u, 2u, 3u, 4u, 6u, 8u}) {
      // no split under 128 deep, nor where the CUs are taken as it is
      if (s > 1 && (steps < 2 * s || tiles * s > (c < T64x64 ? kCus : 4 * kCus))) break;
      const uint32_t depth = cdiv(steps, s), splits = cdiv(steps, depth);
      const float per_cu = (float)((tiles * splits + kCus - 1) / kCus);
      const float turns = (float)((uint32_t)(per_cu + t.resident - 1) / t.resident);
      const float waiting = t.wait * turns, busy = t.busy * per_cu;
      float cost = t.launch + (float)depth * per_step * (waiting > busy ? waiting : busy) + t.group * per_cu;
      if (splits > 1)
        cost += (c < T64x64 ? kJoinRows : kJoin) + kJoinSplit * splits + kJoinBytes * 4.0f * (splits + 1) * (float)m * (float)n;
      if (rows < CUTS && c >= T64x64) cost *= kColdTiles;
      if (best.cost == 0.0f || cost < best.cost) best = {c, splits, depth * kDepth, cost};
    }
  }
  return best;
}

// Whether one launch of 256 x 256 tiles takes less than two of their own.
inline bool worth_pairing(uint32_t m, uint32_t n, uint32_t k) {
  const CutCost& c = kCost[T256x256];
  const uint64_t dx = (uint64_t)cdiv(m, 256) * cdiv(k, 256), dw = (uint64_t)cdiv(n, 256) * cdiv(k, 256);
  const uint64_t dx_steps = cdiv(n, kDepth), dw_steps = cdiv(m, kDepth), longest = dx_steps > dw_steps ? dx_steps : dw_steps;
  const uint64_t shared = (dx * dx_steps + dw * dw_steps + kCus - 1) / kCus;
  const float cost = c.busy * (float)(shared > longest ? shared : longest) + c.group * (float)((dx + dw + kCus - 1) / kCus);
  return cost < shape_of(m, k, n, false, true, true).cost + shape_of(n, k, m, true, true, true).cost;
}

// ---- column walks -----------------------------------------------------------

// Columns kernel geometry: lanes over a row's groups, and how many workgroups
// share the rows.
constexpr uint32_t kFewRows = 64;   // four a thread of the 16 teams
struct ColumnShape {
  int lg;
  uint32_t x, y;   // workgroups
};
inline ColumnShape column_shape(uint32_t rows, uint32_t cols, bool sums) {
  const uint32_t groups = cols ? cdiv(cols, 8) : 1u;   // nothing is launched over no columns
  ColumnShape s;
  // As many lanes across as leave at most an eighth of them idle, at least 16
  // (256 consecutive bytes of a 16-bit row). With sums over many rows, at most
  // 64: workgroups beside each other share the rows' split, so they fill the
  // CUs at no cost in partial sums (dropout's backward pass of 16384 x 1024:
  // 25.5 us with up to 256, 20.6). With sums over few, 16: one workgroup sees
  // all the rows, and its sums are final (64 x 4096: 7.5 us in two kernels, 6.4
  // in one; 128 x 1024: 7.4 and 7.7).
  // Not past 2^23 such workgroups: a launch has fewer than 2^32 threads.
  const bool few = sums && rows <= kFewRows && groups <= 1u << 27;
  for (s.lg = few ? 4 : sums && rows > 1024u ? 6 : 8; s.lg > 4; --s.lg) {
    const uint32_t idle = cdiv(groups, 1u << s.lg) * (1u << s.lg) - groups;
    if (idle * 8u <= groups) break;
  }
  while (s.lg > 0 && (1u << (s.lg - 1)) >= groups) --s.lg;
  const uint32_t teams = 256u >> s.lg, x = cdiv(groups, 1u << s.lg);
  uint32_t y = few ? 1u : cdiv(rows, teams * 4u), most = cdiv(sums ? 2048u : 4096u, x);
  if (sums && most > 256u) most = 256u;   // the sums' own traffic stays small
  if (y > most) y = most;
  s.x = x;
  s.y = y ? y : 1u;
  return s;
}

}  // namespace arx
