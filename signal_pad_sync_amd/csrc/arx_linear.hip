// arx_linear.hip — matrix products for gfx950 with bias, activation and
// residual in the epilogue.
//
//   gemm_kernel   C = A B^T on the matrix cores, 128 x 128 tiles
//
// Sums are binary32 in the matrix cores' accumulators; z and y are each
// rounded once, from the same binary32 value.
#include <hip/hip_runtime.h>

#include "arx_elem.h"
#include "arx_layer.h"

namespace arx {
namespace {

__host__ __device__ constexpr uint32_t cdiv(uint32_t a, uint32_t b) { return a / b + (a % b != 0); }

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float act_any(int kind, float z) {
  switch (kind) {
    case ARX_ACT_RELU: return act<ARX_ACT_RELU>(z);
    case ARX_ACT_GELU: return act<ARX_ACT_GELU>(z);
    case ARX_ACT_GELU_TANH: return act<ARX_ACT_GELU_TANH>(z);
    case ARX_ACT_SILU: return act<ARX_ACT_SILU>(z);
    default: return z;
  }
}

template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p, int valid) {
  typename Vec<T>::x4 v;
  if (valid >= 4) {
    __builtin_memcpy(&v, p, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < valid ? p[j] : (T)0.0f;
  }
  return __builtin_convertvector(v, f32x4);
}
template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 f, int valid) {
  const typename Vec<T>::x4 v = __builtin_convertvector(f, typename Vec<T>::x4);
  if (valid >= 4) {
    __builtin_memcpy(p, &v, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < valid) p[j] = v[j];
  }
}

// Four sums of row i, columns j.. : bias, z, activation, residual, y.
template <typename T>
__device__ __forceinline__ void epilogue4(const GemmArgs& g, uint32_t i, uint32_t j, f32x4 c) {
  if (i >= g.m || j >= g.n) return;
  const int valid = g.n - j < 4u ? (int)(g.n - j) : 4;
  if (g.bias) c += load4(static_cast<const T*>(g.bias) + j, valid);
  if (g.z.p) store4<T>(static_cast<T*>(g.z.p) + (int64_t)i * g.z.ld + j, c, valid);
  if (g.act != ARX_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = act_any(g.act, c[e]);
  }
  if (g.residual.p) c += load4(static_cast<const T*>(g.residual.p) + (int64_t)i * g.residual.ld + j, valid);
  store4<T>(static_cast<T*>(g.y.p) + (int64_t)i * g.y.ld + j, c, valid);
}

// One operand's 128 x 32 tile: rows [r0, r0 + 128) of `rows`, k [k0, k0 + 32)
// of `k`, elements past either end zero. ROWS_K: the row index is the
// contiguous one, and the tile is turned on its way into shared memory.
constexpr int kTile = 128, kDepth = 32, kPitch = kDepth + 8;

template <typename T, bool ROWS_K>
__device__ __forceinline__ void stage(T* lds, const T* p, int64_t ld, uint32_t r0, uint32_t rows, uint32_t k0,
                                      uint32_t k) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = threadIdx.x + i * 256u;
    if constexpr (!ROWS_K) {
      const uint32_t r = t / 4u, c = (t % 4u) * 8u;
      const int valid = r0 + r < rows && k0 + c < k ? (int)min(8u, k - k0 - c) : 0;
      *reinterpret_cast<typename Vec<T>::x8*>(lds + r * kPitch + c) =
          load8(p + (int64_t)(r0 + r) * ld + (k0 + c), valid);
    } else {
      const uint32_t c = t / 16u, r = (t % 16u) * 8u;
      const int valid = k0 + c < k && r0 + r < rows ? (int)min(8u, rows - r0 - r) : 0;
      const typename Vec<T>::x8 v = load8(p + (int64_t)(k0 + c) * ld + (r0 + r), valid);
#pragma unroll
      for (int j = 0; j < 8; ++j) lds[(r + j) * kPitch + c] = v[j];
    }
  }
}

// Four waves, each 64 x 64 of the tile. The second operand of the tile takes
// the matrix instruction's rows, so a lane ends with four neighbouring
// columns of one row of C: lane l holds row l % 16, columns 4 (l / 16) + 0..3.
template <typename T, bool A_ROWS_K, bool B_ROWS_K>
__global__ __launch_bounds__(256) void gemm_kernel(GemmArgs g) {
  __shared__ __align__(16) T as[kTile * kPitch], bs[kTile * kPitch];
  const uint32_t tn = cdiv(g.n, kTile), i0 = blockIdx.x / tn * kTile, j0 = blockIdx.x % tn * kTile;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, wi = (wave >> 1) * 64u, wj = (wave & 1u) * 64u;
  f32x4 c[4][4];
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) c[x][y] = f32x4(0.0f);
  for (uint32_t k0 = 0; k0 < g.k; k0 += kDepth) {
    __syncthreads();
    stage<T, A_ROWS_K>(as, static_cast<const T*>(g.a), g.lda, i0, g.m, k0, g.k);
    stage<T, B_ROWS_K>(bs, static_cast<const T*>(g.b), g.ldb, j0, g.n, k0, g.k);
    __syncthreads();
    typename Vec<T>::x8 fa[4], fb[4];
    const uint32_t at = (lane & 15u) * kPitch + (lane >> 4) * 8u;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      fa[x] = *reinterpret_cast<const typename Vec<T>::x8*>(as + (wi + x * 16u) * kPitch + at);
      fb[x] = *reinterpret_cast<const typename Vec<T>::x8*>(bs + (wj + x * 16u) * kPitch + at);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) c[x][y] = mfma16(fb[y], fa[x], c[x][y]);
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      epilogue4<T>(g, i0 + wi + x * 16u + (lane & 15u), j0 + wj + y * 16u + (lane >> 4) * 4u, c[x][y]);
}

template <typename T>
hipError_t gemm_typed(const GemmArgs& g, hipStream_t stream) {
  const uint32_t tiles = cdiv(g.m, kTile) * cdiv(g.n, kTile);
  if (!g.a_rows_k && !g.b_rows_k) gemm_kernel<T, false, false><<<tiles, 256, 0, stream>>>(g);
  else if (!g.a_rows_k) gemm_kernel<T, false, true><<<tiles, 256, 0, stream>>>(g);
  else if (g.b_rows_k) gemm_kernel<T, true, true><<<tiles, 256, 0, stream>>>(g);
  else gemm_kernel<T, true, false><<<tiles, 256, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(const GemmArgs& g, int dtype, hipStream_t stream) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  return dtype == ARX_BF16 ? gemm_typed<__bf16>(g, stream) : gemm_typed<_Float16>(g, stream);
}

size_t gemm_workspace(uint32_t, uint32_t, uint32_t, bool, bool) { return 0; }

}  // namespace arx
