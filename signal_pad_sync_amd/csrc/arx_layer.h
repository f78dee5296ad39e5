// arx_layer.h — arguments and launchers of the layer operators: the row
// kernels (arx_rows.hip) and the matrix products (arx_linear.hip). Host code
// in arx_layer.cpp checks the arguments first.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "arx.h"

namespace arx {

// Dropout: an element stays if its 16 bits reach `threshold`.
struct Drop {
  uint32_t threshold;  // 65536 p, rounded; 0 keeps everything
  float scale;         // 65536 / (65536 - threshold)
  uint64_t seed, offset;
};

// A plane of rows: element (r, c) at p[r * ld + c].
struct Plane {
  const void* p;
  int64_t ld;
};
struct PlaneOut {
  void* p;  // null: not wanted
  int64_t ld;
};

// Forward: v = x (+ bias), dropped (+ residual) -> h; layer norm of v -> y.
struct RowsArgs {
  Plane x, residual;
  const void* bias;
  const void *weight, *shift;  // of the norm, or null
  PlaneOut h, y;
  float *mean, *rstd;          // [rows], or null
  uint32_t rows, cols;
  float eps;
  Drop drop;
};

// Backward: gradients of the same. Column sums go to `partial`
// [groups][sums][cols] f32 first.
struct RowsGradArgs {
  Plane dy, dh, x;
  const float *mean, *rstd;
  const void* weight;
  PlaneOut dx, dresidual;
  void *dweight, *dshift, *dbias;  // [cols], or null
  uint32_t rows, cols;
  Drop drop;
  float* partial;
  float* stats;                    // [rows][2] for rows too wide for registers
};

hipError_t launch_dropout_add(const RowsArgs& a, int dtype, hipStream_t stream);
hipError_t launch_dropout_add_backward(const RowsGradArgs& a, int dtype, hipStream_t stream);
// join: with dropout, bias, residual and h in front of the norm.
hipError_t launch_norm(const RowsArgs& a, bool join, int dtype, int wdtype, hipStream_t stream);
hipError_t launch_norm_backward(const RowsGradArgs& a, bool join, int dtype, int wdtype, hipStream_t stream);
// Bytes of workspace the backward launchers need for `sums` column sums.
size_t rows_workspace(size_t rows, size_t cols, int sums);

// g = dy * act'(z) into `g` ([m][n] rounded up to a multiple of eight columns,
// the last ones zero) and its column sums into dbias; either may be null. act
// none: dbias alone.
struct ActGradArgs {
  Plane dy, z;
  void* g;
  void* dbias;
  uint32_t m, n;
  float* partial;
};
hipError_t launch_act_grad(const ActGradArgs& a, int act, int dtype, hipStream_t stream);
size_t act_grad_workspace(size_t m, size_t n);

// An operand as lines of contiguous elements. whole: its lines go on to a
// multiple of eight elements, in zeros.
struct Lines {
  const void* p;
  int64_t ld;
  uint32_t lines, cols;
  bool whole;
};
// Whether the tiles can load it as it stands: 16-byte chunks all the way, and
// a tile's offsets within 32 bits.
bool lines_as_is(const Lines& l);
size_t padded_bytes(uint32_t lines, uint32_t cols);
// Copies those of up to three that cannot be (nulls are let pass) to `space`,
// padded_bytes() each, and points them there.
hipError_t launch_pad(Lines* l, int count, int dtype, void* space, hipStream_t stream);

// C[i][j] = sum over k of A(i, k) B(j, k), then the epilogue
// z = C + bias[j] -> z; y = act(z) + residual -> y.
// A(i, k) = a[i * lda + k], or a[k * lda + i] with a_rows_k; B the same.
struct GemmArgs {
  const void *a, *b;
  int64_t lda, ldb;
  bool a_rows_k, b_rows_k;
  bool a_whole, b_whole;  // as in Lines
  uint32_t m, n, k;
  const void* bias;
  Plane residual;
  PlaneOut y, z;
  int act;
  void* workspace;
};
hipError_t launch_gemm(const GemmArgs& a, int dtype, hipStream_t stream);
// The products of a backward pass, operands as the tiles take them: one launch
// or two. Their workspaces may be the same.
hipError_t launch_gemm_pair(const GemmArgs& dx, const GemmArgs& dw, int dtype, hipStream_t stream);
// Bytes for the forward product (aligned: both operands start on 16-byte
// boundaries and their ld is a multiple of 8 below 2^22), and for the partial
// sums of any product alone.
size_t gemm_workspace(uint32_t m, uint32_t n, uint32_t k, bool aligned);
size_t gemm_splits_workspace(uint32_t m, uint32_t n, uint32_t k, bool a_rows_k, bool b_rows_k);

}  // namespace arx
