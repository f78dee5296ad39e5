// arx_rows.hip — the row operators for gfx950: dropout with bias and residual,
// layer norm, and both in one pass, forward and backward.
//
//   norm_kernel          forward: a team of lanes holds one row in registers
//   norm_wide_kernel     the same for rows too wide for that, in three passes
//   norm_grad_kernel     backward: teams walk over rows, weight gradients
//                        gather in registers
//   norm_stats_kernel    the two row sums of a wide row's backward pass
//   column_kernel        one thread per column group, walking over rows:
//                        dropout forward and backward, a wide row's norm
//                        backward, an activation's slope
//   column_sum_kernel    adds the workgroups' column sums, in a fixed order
//
// All of it is bound by memory: every plane is read or written once. Sums and
// row statistics are binary32; a value is rounded once, as it is stored.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "arx_elem.h"
#include "arx_internal.h"
#include "arx_layer.h"
#include "arx_shapes.h"

namespace arx {
namespace {

__device__ __forceinline__ int valid_of(uint32_t group, uint32_t cols) {
  const uint32_t c = group * 8u;
  return c >= cols ? 0 : (cols - c < 8u ? (int)(cols - c) : 8);
}

__device__ __forceinline__ float sum8(f32x8 v) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// Sum over groups of N neighbouring lanes.
template <int N = 64>
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum over a team of L lanes: part of a wave, a wave, or (L > 64) the whole
// workgroup. `lds`: L / 64 floats of this call's own.
template <int L>
__device__ __forceinline__ float team_sum(float v, float* lds) {
  v = wave_sum<L < 64 ? L : 64>(v);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63u) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < L / 64; ++w) v += lds[w];
  }
  return v;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const Plane& p, uint32_t r) {
  return static_cast<const T*>(p.p) + (int64_t)r * p.ld;
}
template <typename T>
__device__ __forceinline__ T* row_of(const PlaneOut& p, uint32_t r) {
  return static_cast<T*>(p.p) + (int64_t)r * p.ld;
}

// What the norm works on: x, or x (+ bias) dropped (+ residual). In the join
// the norm takes h as computed, before its rounding, so y carries one rounding.
template <typename T, bool JOIN>
__device__ __forceinline__ f32x8 row_input(const RowsArgs& a, uint32_t r, uint32_t g, int valid) {
  const uint32_t c = g * 8u;
  f32x8 v = widen(load8(row_of<T>(a.x, r) + c, valid));
  if constexpr (JOIN) {
    if (a.bias) v += widen(load8(static_cast<const T*>(a.bias) + c, valid));
    if (valid > 0) v = drop8(v, (uint64_t)r * cdiv(a.cols, 8) + g, a.drop);
    if (a.residual.p) v += widen(load8(row_of<T>(a.residual, r) + c, valid));
  }
  return v;
}

template <typename W>
__device__ __forceinline__ f32x8 scale_shift(const RowsArgs& a, f32x8 v, uint32_t c, int valid) {
  if (a.weight) v *= widen(load8(static_cast<const W*>(a.weight) + c, valid));
  if (a.shift) v += widen(load8(static_cast<const W*>(a.shift) + c, valid));
  return v;
}

// Centred value with the columns past the row's end zero, for the variance.
__device__ __forceinline__ f32x8 centred(f32x8 v, float mean, int valid) {
  v -= mean;
  if (valid < 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? v[j] : 0.0f;
  }
  return v;
}

// A row in registers, V groups of eight a lane: one read, the mean, then the
// mean of the squared distances from it (no cancellation), one write. Bound by
// memory: 8192 x 8192 bf16 in 53 us (5.1 TB/s), the join of 8192 x 4096 in 58
// to 62 (4.6 to 4.3 TB/s, the generator's integer products beside it); a few rows
// take one memory latency and two reductions, 32 x 4096 in 3.8 us back to back.
template <typename T, typename W, int L, int V, bool JOIN>
__global__ __launch_bounds__(L < 256 ? 256 : L) void norm_kernel(RowsArgs a) {
  constexpr int R = L < 256 ? 256 / L : 1;
  __shared__ float lds[2][L < 64 ? 1 : L / 64];
  const uint32_t lane = threadIdx.x % L;
  // Teams of a wave or less meet no barrier; a larger team is the workgroup, whose
  // rows end together. Its two reductions alternate between two buffers.
  for (uint64_t r = (uint64_t)blockIdx.x * R + threadIdx.x / L; r < a.rows; r += (uint64_t)gridDim.x * R) {
    f32x8 v[V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t g = lane + i * L;
      v[i] = row_input<T, JOIN>(a, r, g, valid_of(g, a.cols));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (JOIN) {
        const uint32_t g = lane + i * L;
        if (a.h.p) store8<T>(row_of<T>(a.h, r) + g * 8u, narrow<T>(v[i]), valid_of(g, a.cols));
      }
      s += sum8(v[i]);
    }
    const float mean = team_sum<L>(s, lds[0]) / (float)a.cols;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = centred(v[i], mean, valid_of(lane + i * L, a.cols));
      s += sum8(v[i] * v[i]);
    }
    const float rstd = 1.0f / sqrtf(team_sum<L>(s, lds[1]) / (float)a.cols + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t g = lane + i * L;
      const int valid = valid_of(g, a.cols);
      store8<T>(row_of<T>(a.y, r) + g * 8u, narrow<T>(scale_shift<W>(a, v[i] * rstd, g * 8u, valid)), valid);
    }
    if (lane == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

// Rows of any width: three passes over the row, the later ones from the
// caches. h and y are stored in the last, so they may take an input's place.
template <typename T, typename W, bool JOIN>
__global__ __launch_bounds__(1024) void norm_wide_kernel(RowsArgs a) {
  __shared__ float lds[2][16];
  const uint32_t groups = cdiv(a.cols, 8);
  for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float s = 0.0f;
    for (uint32_t g = threadIdx.x; g < groups; g += 1024u)
      s += sum8(row_input<T, JOIN>(a, r, g, valid_of(g, a.cols)));
    const float mean = team_sum<1024>(s, lds[0]) / (float)a.cols;
    s = 0.0f;
    for (uint32_t g = threadIdx.x; g < groups; g += 1024u) {
      const int valid = valid_of(g, a.cols);
      const f32x8 d = centred(row_input<T, JOIN>(a, r, g, valid), mean, valid);
      s += sum8(d * d);
    }
    const float rstd = 1.0f / sqrtf(team_sum<1024>(s, lds[1]) / (float)a.cols + a.eps);
    for (uint32_t g = threadIdx.x; g < groups; g += 1024u) {
      const int valid = valid_of(g, a.cols);
      const f32x8 v = row_input<T, JOIN>(a, r, g, valid);
      if (JOIN && a.h.p) store8<T>(row_of<T>(a.h, r) + g * 8u, narrow<T>(v), valid);
      store8<T>(row_of<T>(a.y, r) + g * 8u, narrow<T>(scale_shift<W>(a, (v - mean) * rstd, g * 8u, valid)), valid);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

// ---- backward ---------------------------------------------------------------

// Where workgroup `wg`'s sums of kind `k` stand.
__device__ __forceinline__ float* partial_of(const RowsGradArgs& a, uint32_t wg, int sums, int k) {
  return a.partial + ((size_t)wg * sums + k) * a.cols;
}

// With xh = (x - mean) rstd and g = dy weight:
//   dv = rstd (g - mean(g) - xh mean(g xh)), join: + dh,
//   dweight = sum over rows of dy xh, dshift = sum of dy,
//   join: dresidual = dv, dx = dv dropped by the same bits, dbias = sum of dx.
// A team takes every (gridDim.x R)-th row and keeps its columns' sums in
// registers; the teams of a workgroup add theirs through shared memory. Bound
// by memory over many rows: 8192 x 8192 bf16 in 82 us with the sums' adding (4.9
// TB/s), the join of 8192 x 4096 in 71 (4.7 TB/s). One workgroup a CU keeps the
// partial sums at 4 % of the rows' bytes there; over a few hundred rows they are
// most of them (512 x 4096: 13.7 us, 2.6 at a copy's rate). Narrow rows wait for
// their many teams' sums, which the first team adds one after another (100000 x
// 64: 25.7 us, 7.8). binary32 planes in the join spill 4 to 11 registers a lane
// up to 4096 columns, at the copy's rate over many rows all the same (8192 x 4096:
// 138 us, 4.9 TB/s).
template <typename T, typename W, int L, bool JOIN>
__global__ __launch_bounds__(1024) void norm_grad_kernel(RowsGradArgs a) {
  constexpr int R = 1024 / L;
  constexpr int SUMS = JOIN ? 3 : 2;
  typedef typename Vec<T>::x8 x8;
  __shared__ float lds[2][2][16];
  __shared__ float gather[R > 1 ? 1024 * 8 : 1];
  const uint32_t lane = threadIdx.x % L, team = threadIdx.x / L, groups = cdiv(a.cols, 8), c = lane * 8u;
  const int there = valid_of(lane, a.cols);
  const float inv = 1.0f / (float)a.cols;
  f32x8 w = f32x8(1.0f), sum[SUMS];
  if (a.weight) w = widen(load8(static_cast<const W*>(a.weight) + c, there));
#pragma unroll
  for (int k = 0; k < SUMS; ++k) sum[k] = f32x8(0.0f);
  // A row's values are asked for while the row before is worked on.
  x8 in_dy, in_x, in_dh;
  float in_mean = 0.0f, in_rstd = 0.0f;
  const auto ask = [&](uint64_t row) {
    const bool live = row < a.rows;
    const uint32_t r = live ? (uint32_t)row : 0u;
    const int valid = live ? there : 0;
    in_dy = load8(row_of<T>(a.dy, r) + c, valid);
    in_x = load8(row_of<T>(a.x, r) + c, valid);
    if (JOIN) in_dh = load8(row_of<T>(a.dh, r) + c, a.dh.p ? valid : 0);
    in_mean = live ? a.mean[r] : 0.0f;
    in_rstd = live ? a.rstd[r] : 0.0f;
  };
  int turn = 0;
  const uint64_t stride = (uint64_t)gridDim.x * R;
  ask((uint64_t)blockIdx.x * R + team);
  for (uint64_t base = (uint64_t)blockIdx.x * R; base < a.rows; base += stride, turn ^= 1) {
    const bool live = base + team < a.rows;
    const uint32_t r = live ? (uint32_t)base + team : 0u;
    const int valid = live ? there : 0;
    const float mean = in_mean, rstd = in_rstd;
    const f32x8 dy = widen(in_dy), xh = centred(widen(in_x), mean, valid) * rstd;
    f32x8 dh;
    if (JOIN) dh = widen(in_dh);
    if (base + stride < a.rows) ask(base + stride + team);
    const f32x8 g = dy * w;
    float s1 = wave_sum<L < 64 ? L : 64>(sum8(g)), s2 = wave_sum<L < 64 ? L : 64>(sum8(g * xh));
    if constexpr (L > 64) {
      if ((threadIdx.x & 63u) == 0) {
        lds[turn][0][threadIdx.x >> 6] = s1;
        lds[turn][1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll
      for (int q = 0; q < L / 64; ++q) {
        s1 += lds[turn][0][team * (L / 64) + q];
        s2 += lds[turn][1][team * (L / 64) + q];
      }
    }
    s1 *= inv;
    s2 *= inv;
    f32x8 d = rstd * (dy * w - s1 - xh * s2);
    sum[0] += dy * xh;
    sum[1] += dy;
    if constexpr (JOIN) {
      if (a.dh.p) d += dh;
      if (a.dresidual.p) store8<T>(row_of<T>(a.dresidual, r) + c, narrow<T>(d), valid);
      if (valid > 0) d = drop8(d, (uint64_t)r * groups + lane, a.drop);
      if (valid > 0) sum[2] += d;
    }
    store8<T>(row_of<T>(a.dx, r) + c, narrow<T>(d), valid);
  }
#pragma unroll
  for (int k = 0; k < SUMS; ++k) {
    if ((k == 0 && !a.dweight) || (k == 1 && !a.dshift) || (k == 2 && !a.dbias)) continue;
    f32x8 s = sum[k];
    if constexpr (R > 1) {
      __syncthreads();
      *reinterpret_cast<f32x8*>(&gather[threadIdx.x * 8u]) = s;
      __syncthreads();
      if (team == 0)
        for (int t = 1; t < R; ++t) s += *reinterpret_cast<const f32x8*>(&gather[(t * L + lane) * 8u]);
    }
    if (team == 0) store8<float>(partial_of(a, blockIdx.x, SUMS, k) + c, s, there);
  }
}

// A wide row's mean(g) and mean(g xh).
template <typename T, typename W>
__global__ __launch_bounds__(1024) void norm_stats_kernel(RowsGradArgs a) {
  __shared__ float lds[2][16];
  const uint32_t groups = cdiv(a.cols, 8);
  for (uint64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (uint32_t g = threadIdx.x; g < groups; g += 1024u) {
      const int valid = valid_of(g, a.cols);
      f32x8 d = widen(load8(row_of<T>(a.dy, r) + g * 8u, valid));
      if (a.weight) d *= widen(load8(static_cast<const W*>(a.weight) + g * 8u, valid));
      s1 += sum8(d);
      s2 += sum8(d * centred(widen(load8(row_of<T>(a.x, r) + g * 8u, valid)), mean, valid) * rstd);
    }
    s1 = team_sum<1024>(s1, lds[0]);
    s2 = team_sum<1024>(s2, lds[1]);
    if (threadIdx.x == 0) {
      a.stats[2u * (size_t)r] = s1 / (float)a.cols;
      a.stats[2u * (size_t)r + 1u] = s2 / (float)a.cols;
    }
  }
}

// Where finished column sums go.
struct SumsOut {
  void* out[3];   // [cols] each, or null
  int dtype[3];
  __device__ __forceinline__ void put(int k, uint32_t c, float s) const {
    if (dtype[k] == ARX_BF16) static_cast<__bf16*>(out[k])[c] = (__bf16)s;
    else if (dtype[k] == ARX_F16) static_cast<_Float16*>(out[k])[c] = (_Float16)s;
    else static_cast<float*>(out[k])[c] = s;
  }
};

// ---- one thread per column group --------------------------------------------

// 256 threads as 2^lg lanes over column groups by 256 >> lg rows; blockIdx.x
// over the columns, blockIdx.y over the rows, UNROLL rows of a thread in
// flight. Bound by memory: dropout with bias and residual of 8192 x 4096 bf16
// in 40 us (5.0 TB/s). op.begin(group, valid) reads what a column keeps, op.row(r) works
// on one row's group, and sums of kind k are op.sum[k].
template <typename OP>
__global__ __launch_bounds__(256) void column_kernel(OP op, uint32_t rows, uint32_t cols, int lg, float* partial,
                                                     SumsOut sums) {
  __shared__ float gather[OP::SUMS > 0 ? 256 * 8 : 1];
  const uint32_t lanes = 1u << lg, lane = threadIdx.x & (lanes - 1u), team = threadIdx.x >> lg, teams = 256u >> lg;
  const uint32_t g = blockIdx.x * lanes + lane;
  const int valid = valid_of(g, cols);
  op.begin(g, valid);
  const uint64_t step = (uint64_t)gridDim.y * teams;
  uint64_t r = (uint64_t)blockIdx.y * teams + team;
  if (valid > 0) {
    for (; r + (OP::UNROLL - 1) * step < rows; r += OP::UNROLL * step) {
      typename OP::In in[OP::UNROLL];
#pragma unroll
      for (int u = 0; u < OP::UNROLL; ++u) in[u] = op.load((uint32_t)(r + u * step), g, valid);
#pragma unroll
      for (int u = 0; u < OP::UNROLL; ++u) op.row(in[u], (uint32_t)(r + u * step), g, valid);
    }
    for (; r < rows; r += step) op.row(op.load((uint32_t)r, g, valid), (uint32_t)r, g, valid);
  }
  if constexpr (OP::SUMS > 0) {
#pragma unroll
    for (int k = 0; k < OP::SUMS; ++k) {
      f32x8 s = op.sum[k];
      if (teams > 1) {
        __syncthreads();
        *reinterpret_cast<f32x8*>(&gather[threadIdx.x * 8u]) = s;
        __syncthreads();
        if (team == 0)
          for (uint32_t t = 1; t < teams; ++t)
            s += *reinterpret_cast<const f32x8*>(&gather[(t * lanes + lane) * 8u]);
      }
      if (team != 0) continue;
      if (gridDim.y > 1) {
        store8<float>(partial + ((size_t)blockIdx.y * OP::SUMS + k) * cols + g * 8u, s, valid);
      } else if (sums.out[k]) {   // all the rows: these are the sums
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < valid) sums.put(k, g * 8u + j, s[j]);
      }
    }
  }
}

template <typename T>
struct DropoutAdd {
  static constexpr int SUMS = 0, UNROLL = 4;
  struct In {
    typename Vec<T>::x8 x, residual;
  };
  RowsArgs a;
  f32x8 bias;
  __device__ void begin(uint32_t g, int valid) {
    bias = a.bias ? widen(load8(static_cast<const T*>(a.bias) + g * 8u, valid)) : f32x8(0.0f);
  }
  __device__ In load(uint32_t r, uint32_t g, int valid) const {
    In in;
    in.x = load8(row_of<T>(a.x, r) + g * 8u, valid);
    if (a.residual.p) in.residual = load8(row_of<T>(a.residual, r) + g * 8u, valid);
    return in;
  }
  __device__ void row(const In& in, uint32_t r, uint32_t g, int valid) {
    f32x8 v = widen(in.x);
    if (a.bias) v += bias;
    v = drop8(v, (uint64_t)r * cdiv(a.cols, 8) + g, a.drop);
    if (a.residual.p) v += widen(in.residual);
    store8<T>(row_of<T>(a.h, r) + g * 8u, narrow<T>(v), valid);
  }
};

template <typename T, bool BIAS>
struct DropoutGrad {
  static constexpr int SUMS = BIAS ? 1 : 0, UNROLL = 4;
  using In = typename Vec<T>::x8;
  RowsGradArgs a;
  f32x8 sum[1];
  __device__ void begin(uint32_t, int) { sum[0] = f32x8(0.0f); }
  __device__ In load(uint32_t r, uint32_t g, int valid) const { return load8(row_of<T>(a.dh, r) + g * 8u, valid); }
  __device__ void row(const In& in, uint32_t r, uint32_t g, int valid) {
    const f32x8 d = drop8(widen(in), (uint64_t)r * cdiv(a.cols, 8) + g, a.drop);
    sum[0] += d;
    if (a.dx.p) store8<T>(row_of<T>(a.dx, r) + g * 8u, narrow<T>(d), valid);
  }
};

// A wide row's backward pass, its row sums known (norm_stats_kernel).
template <typename T, typename W, bool JOIN>
struct NormGradWide {
  static constexpr int SUMS = JOIN ? 3 : 2, UNROLL = 2;
  struct In {
    typename Vec<T>::x8 dy, x, dh;
    float mean, rstd, s1, s2;
  };
  RowsGradArgs a;
  f32x8 w, sum[3];
  __device__ void begin(uint32_t g, int valid) {
    w = a.weight ? widen(load8(static_cast<const W*>(a.weight) + g * 8u, valid)) : f32x8(1.0f);
    sum[0] = sum[1] = sum[2] = f32x8(0.0f);
  }
  __device__ In load(uint32_t r, uint32_t g, int valid) const {
    In in;
    in.dy = load8(row_of<T>(a.dy, r) + g * 8u, valid);
    in.x = load8(row_of<T>(a.x, r) + g * 8u, valid);
    if (JOIN && a.dh.p) in.dh = load8(row_of<T>(a.dh, r) + g * 8u, valid);
    in.mean = a.mean[r];
    in.rstd = a.rstd[r];
    in.s1 = a.stats[2u * (size_t)r];
    in.s2 = a.stats[2u * (size_t)r + 1u];
    return in;
  }
  __device__ void row(const In& in, uint32_t r, uint32_t g, int valid) {
    const f32x8 dy = widen(in.dy), xh = (widen(in.x) - in.mean) * in.rstd;
    f32x8 d = in.rstd * (dy * w - in.s1 - xh * in.s2);
    sum[0] += dy * xh;
    sum[1] += dy;
    if constexpr (JOIN) {
      if (a.dh.p) d += widen(in.dh);
      if (a.dresidual.p) store8<T>(row_of<T>(a.dresidual, r) + g * 8u, narrow<T>(d), valid);
      d = drop8(d, (uint64_t)r * cdiv(a.cols, 8) + g, a.drop);
      sum[2] += d;
    }
    store8<T>(row_of<T>(a.dx, r) + g * 8u, narrow<T>(d), valid);
  }
};

// The gradient in front of an activation, and its column sums from before
// the rounding. It is rounded to the operands' type because the matrix cores
// take no wider one beside them: dx and dw are 2.3e-3 from the 64-bit result in
// bf16 where a gradient in 32 bits would leave 1.7e-3, their own rounding; two
// terms of the type would hold it, at twice the products' time (220 to 240 us of
// 8192 x 4096 x 2048).
template <typename T, int ACT, bool BIAS>
struct ActGrad {
  static constexpr int SUMS = BIAS ? 1 : 0, UNROLL = 4;
  struct In {
    typename Vec<T>::x8 dy, z;
  };
  ActGradArgs a;
  f32x8 sum[1];
  __device__ void begin(uint32_t, int) { sum[0] = f32x8(0.0f); }
  __device__ In load(uint32_t r, uint32_t g, int valid) const {
    In in;
    in.dy = load8(row_of<T>(a.dy, r) + g * 8u, valid);
    if constexpr (ACT != ARX_ACT_NONE) in.z = load8(row_of<T>(a.z, r) + g * 8u, valid);
    return in;
  }
  __device__ void row(const In& in, uint32_t r, uint32_t g, int valid) {
    f32x8 d = widen(in.dy);
    if constexpr (ACT != ARX_ACT_NONE) {
      const f32x8 z = widen(in.z);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] *= act_slope<ACT>(z[j]);
    }
    sum[0] += d;
    if (a.g) store8<T>(static_cast<T*>(a.g) + (size_t)r * (cdiv(a.n, 8) * 8u) + g * 8u, narrow<T>(d), 8);
  }
};

// ---- the workgroups' column sums --------------------------------------------

struct ColumnSumArgs {
  const float* partial;  // [groups][sums][cols]
  SumsOut to;
  uint32_t groups, cols;
  int sums;
};

// 64 columns by 16 slices of the workgroups; always the same order. A latency or
// two: 256 workgroups' sums of 8192 columns in 4.6 us.
__global__ __launch_bounds__(1024) void column_sum_kernel(ColumnSumArgs a) {
  __shared__ float lds[16][64];
  const int k = blockIdx.y;
  if (!a.to.out[k]) return;
  const uint32_t lane = threadIdx.x & 63u, slice = threadIdx.x >> 6, c = blockIdx.x * 64u + lane;
  float s = 0.0f;
  if (c < a.cols) {
#pragma unroll 8
    for (uint32_t g = slice; g < a.groups; g += 16u) s += a.partial[((size_t)g * a.sums + k) * a.cols + c];
  }
  lds[slice][lane] = s;
  __syncthreads();
  if (slice != 0 || c >= a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int q = 0; q < 16; ++q) s += lds[q][lane];
  a.to.put(k, c, s);
}

// ---- launches ---------------------------------------------------------------

// A launch has fewer than 2^32 threads; past that many rows, teams loop.
constexpr uint32_t kMaxGroups = 1u << 20;
uint32_t row_groups(uint32_t teams) { return teams < kMaxGroups ? teams : kMaxGroups; }

// Workgroups of the backward norm kernel: one a CU.
constexpr uint32_t kGradGroups = 256;
// Widest row whose sums stay in registers, one group a lane. Two groups spill:
// 2048 x 16384 bf16 took 243 us, and takes 71 in two kernels, which read dy and x
// twice (41 at a copy's rate).
constexpr uint32_t kGradCols = 8192;

hipError_t launch_column_sum(const ColumnSumArgs& a, hipStream_t stream) {
  bool any = false;
  for (int k = 0; k < a.sums; ++k) any = any || a.to.out[k];
  if (!any || a.cols == 0) return hipSuccess;
  column_sum_kernel<<<dim3(cdiv(a.cols, 64), a.sums), 1024, 0, stream>>>(a);
  return hipGetLastError();
}

// The column kernel, and its sums' adding where several workgroups have parts.
template <typename OP>
hipError_t launch_column(const OP& op, uint32_t rows, uint32_t cols, float* partial, const SumsOut& to,
                         hipStream_t stream) {
  if (cols == 0) return hipSuccess;
  const ColumnShape s = column_shape(rows, cols, OP::SUMS > 0);
  column_kernel<OP><<<dim3(s.x, s.y), 256, 0, stream>>>(op, rows, cols, s.lg, partial, to);
  const hipError_t rc = hipGetLastError();
  if (rc != hipSuccess || OP::SUMS == 0 || s.y == 1) return rc;
  return launch_column_sum({partial, to, s.y, cols, OP::SUMS}, stream);
}

template <typename T, typename W, bool JOIN>
hipError_t norm_typed(const RowsArgs& a, hipStream_t stream) {
  const uint32_t groups = cdiv(a.cols, 8);
#define ARX_NORM(L, V)                                                                                      \
  if (groups <= L * V) {                                                                                    \
    constexpr uint32_t R = L < 256 ? 256 / L : 1;                                                           \
    norm_kernel<T, W, L, V, JOIN><<<row_groups(cdiv(a.rows, R)), L < 256 ? 256 : L, 0, stream>>>(a);        \
    return hipGetLastError();                                                                               \
  }
  ARX_NORM(8, 1)
  ARX_NORM(32, 1)
  ARX_NORM(64, 1)
  ARX_NORM(64, 2)
  ARX_NORM(256, 1)
  if constexpr (JOIN) {
    // Few rows: one group a lane, so that a row's generator and sums take the
    // least time (32 x 4096 bf16: 5.2 us against 6.5); many: fewer waves to
    // meet (8192 x 8192: 143 us against 172).
    if (a.rows <= 1024u) {
      ARX_NORM(512, 1)
      ARX_NORM(1024, 1)
    }
  }
  ARX_NORM(256, 2)
  ARX_NORM(256, 4)
  ARX_NORM(1024, 2)
  ARX_NORM(1024, 4)
#undef ARX_NORM
  norm_wide_kernel<T, W, JOIN><<<row_groups(a.rows), 1024, 0, stream>>>(a);
  return hipGetLastError();
}

// Floats of a wide backward pass's column sums, in front of its row sums.
size_t wide_sums(uint32_t rows, uint32_t cols, int sums) {
  return ((size_t)column_shape(rows, cols, true).y * sums * cols + 3) & ~(size_t)3;
}

template <typename T>
constexpr int code_of() {
  return sizeof(T) == 4 ? ARX_F32 : (std::is_same<T, __bf16>::value ? ARX_BF16 : ARX_F16);
}

template <typename T, typename W, bool JOIN>
hipError_t norm_grad_typed(const RowsGradArgs& a, hipStream_t stream) {
  const uint32_t groups = cdiv(a.cols, 8);
  constexpr int SUMS = JOIN ? 3 : 2;
  const SumsOut to = {{a.dweight, a.dshift, JOIN ? a.dbias : nullptr}, {code_of<W>(), code_of<W>(), code_of<T>()}};
  hipError_t rc;
  if (a.cols <= kGradCols) {
#define ARX_NORM_GRAD(L)                                                                      \
  if (groups <= L) {                                                                          \
    constexpr uint32_t R = 1024 / L;                                                          \
    const uint32_t need = cdiv(a.rows, R);                                                    \
    const uint32_t wgs = need < kGradGroups ? (need ? need : 1u) : kGradGroups;               \
    norm_grad_kernel<T, W, L, JOIN><<<wgs, 1024, 0, stream>>>(a);                             \
    if ((rc = hipGetLastError()) != hipSuccess) return rc;                                    \
    return launch_column_sum({a.partial, to, wgs, a.cols, SUMS}, stream);                     \
  }
    ARX_NORM_GRAD(8)
    ARX_NORM_GRAD(32)
    ARX_NORM_GRAD(64)
    ARX_NORM_GRAD(128)
    ARX_NORM_GRAD(256)
    ARX_NORM_GRAD(512)
    ARX_NORM_GRAD(1024)
#undef ARX_NORM_GRAD
  }
  NormGradWide<T, W, JOIN> op;
  op.a = a;
  op.a.stats = a.partial + wide_sums(a.rows, a.cols, SUMS);
  if (a.rows > 0) {
    norm_stats_kernel<T, W><<<row_groups(a.rows), 1024, 0, stream>>>(op.a);
    if ((rc = hipGetLastError()) != hipSuccess) return rc;
  }
  return launch_column(op, a.rows, a.cols, a.partial, to, stream);
}

template <typename F>
hipError_t by_types(int dtype, int wdtype, F f) {
  if (dtype == ARX_BF16) return wdtype == ARX_F32 ? f((__bf16)0, 0.0f) : f((__bf16)0, (__bf16)0);
  if (dtype == ARX_F16) return wdtype == ARX_F32 ? f((_Float16)0, 0.0f) : f((_Float16)0, (_Float16)0);
  return f(0.0f, 0.0f);
}

}  // namespace

hipError_t launch_norm(const RowsArgs& a, bool join, int dtype, int wdtype, hipStream_t stream) {
  return by_types(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    return join ? norm_typed<T, W, true>(a, stream) : norm_typed<T, W, false>(a, stream);
  });
}

hipError_t launch_norm_backward(const RowsGradArgs& a, bool join, int dtype, int wdtype, hipStream_t stream) {
  return by_types(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    return join ? norm_grad_typed<T, W, true>(a, stream) : norm_grad_typed<T, W, false>(a, stream);
  });
}

hipError_t launch_dropout_add(const RowsArgs& a, int dtype, hipStream_t stream) {
  return by_types(dtype, dtype, [&](auto t, auto) {
    DropoutAdd<decltype(t)> op;
    op.a = a;
    return launch_column(op, a.rows, a.cols, nullptr, SumsOut{}, stream);
  });
}

hipError_t launch_dropout_add_backward(const RowsGradArgs& a, int dtype, hipStream_t stream) {
  return by_types(dtype, dtype, [&](auto t, auto) {
    using T = decltype(t);
    if (!a.dbias) {
      DropoutGrad<T, false> op;
      op.a = a;
      return launch_column(op, a.rows, a.cols, nullptr, SumsOut{}, stream);
    }
    DropoutGrad<T, true> op;
    op.a = a;
    return launch_column(op, a.rows, a.cols, a.partial, SumsOut{{a.dbias}, {dtype}}, stream);
  });
}

size_t rows_workspace(size_t rows, size_t cols, int sums) {
  const size_t columns = wide_sums((uint32_t)rows, (uint32_t)cols, sums) * 4;
  if (cols > kGradCols) return columns + rows * 8;
  const size_t teams = (size_t)kGradGroups * sums * cols * 4;
  return columns > teams ? columns : teams;
}

template <typename T, int ACT>
static hipError_t act_grad_typed(const ActGradArgs& a, int dtype, hipStream_t stream) {
  if (!a.dbias) {
    ActGrad<T, ACT, false> op;
    op.a = a;
    return launch_column(op, a.m, a.n, nullptr, SumsOut{}, stream);
  }
  ActGrad<T, ACT, true> op;
  op.a = a;
  return launch_column(op, a.m, a.n, a.partial, SumsOut{{a.dbias}, {dtype}}, stream);
}

hipError_t launch_act_grad(const ActGradArgs& a, int act, int dtype, hipStream_t stream) {
  return by_types(dtype, dtype, [&](auto t, auto) {
    using T = decltype(t);
    switch (act) {
      case ARX_ACT_RELU: return act_grad_typed<T, ARX_ACT_RELU>(a, dtype, stream);
      case ARX_ACT_GELU: return act_grad_typed<T, ARX_ACT_GELU>(a, dtype, stream);
      case ARX_ACT_GELU_TANH: return act_grad_typed<T, ARX_ACT_GELU_TANH>(a, dtype, stream);
      case ARX_ACT_SILU: return act_grad_typed<T, ARX_ACT_SILU>(a, dtype, stream);
      default: return act_grad_typed<T, ARX_ACT_NONE>(a, dtype, stream);
    }
  });
}

size_t act_grad_workspace(size_t m, size_t n) {
  return ((column_shape((uint32_t)m, (uint32_t)n, true).y * n + 3) & ~(size_t)3) * 4;
}

}  // namespace arx
