// arx_linear.hip — matrix products for gfx950 with bias, activation and
// residual in the epilogue.
//
//   tile_kernel   C = A B^T on the matrix cores, tile by tile
//   rows_kernel   the same for a few rows of A: B streams past once
//   join_kernel   adds the splits of a long depth, in order
//   pad_kernel    rows that start off 16-byte boundaries, copied onto them
//
// Sums are binary32 in the matrix cores' accumulators; z and y are each
// rounded once, from the same binary32 value.
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "arx_elem.h"
#include "arx_layer.h"
#include "arx_shapes.h"

namespace arx {
namespace {

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

template <int ACT>
__device__ __forceinline__ void act_each(f32x8& v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = act<ACT>(v[e]);
}

__device__ __forceinline__ void act8(int kind, f32x8& v) {
  switch (kind) {
    case ARX_ACT_RELU: return act_each<ARX_ACT_RELU>(v);
    case ARX_ACT_GELU: return act_each<ARX_ACT_GELU>(v);
    case ARX_ACT_GELU_TANH: return act_each<ARX_ACT_GELU_TANH>(v);
    case ARX_ACT_SILU: return act_each<ARX_ACT_SILU>(v);
    default: return;
  }
}

// f(0), ..., f(N - 1) with constants, so that what they index stays in registers.
template <typename F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each_of(std::make_integer_sequence<int, N>{}, f);
}

// Eight sums of row i, columns j.. : bias, z, activation, residual, y. The
// residual comes as an argument, so that it can be asked for ahead of time.
template <typename T>
__device__ __forceinline__ typename Vec<T>::x8 residual8(const GemmArgs& g, uint32_t i, uint32_t j) {
  const int valid = i < g.m && j < g.n ? (int)min(8u, g.n - j) : 0;
  return load8(static_cast<const T*>(g.residual.p) + (int64_t)i * g.residual.ld + j, g.residual.p ? valid : 0);
}
template <typename T>
__device__ __forceinline__ void epilogue8(const GemmArgs& g, uint32_t i, uint32_t j, f32x8 c,
                                          typename Vec<T>::x8 residual) {
  if (i >= g.m || j >= g.n) return;
  const int valid = g.n - j < 8u ? (int)(g.n - j) : 8;
  if (g.bias) c += widen(load8(static_cast<const T*>(g.bias) + j, valid));
  if (g.z.p) store8<T>(static_cast<T*>(g.z.p) + (int64_t)i * g.z.ld + j, narrow<T>(c), valid);
  act8(g.act, c);
  if (g.residual.p) c += widen(residual);
  store8<T>(static_cast<T*>(g.y.p) + (int64_t)i * g.y.ld + j, narrow<T>(c), valid);
}

// ---- tiles ------------------------------------------------------------------

// Operand tiles are kDepth = 64 deep and come to shared memory without passing
// through registers, 16 bytes a lane. Two layouts, each with its 16-byte
// chunks permuted so that the fragment reads meet no bank twice:
//   depth-contiguous operand (row r, k contiguous): row r is 128 bytes, chunk
//   c of it at place c ^ (r & 7);
//   row-contiguous operand (ROWS_K): depth k is a line of TILE rows, 32-byte
//   piece p of it at place p ^ (k & 3), read with the transposing LDS load.
// Sixteen zero bytes that lanes past the end of the depth read instead.
__device__ const uint4 kZeros = {0, 0, 0, 0};

// One lane's 16 bytes to its place in the wave's 1 KiB block at LDS address
// `block`, from base + off or from p. The builtin for this makes the compiler
// wait for every LDS read under way at the next use of any; the instruction
// itself has no result register, and the waits for it are written out
// (wait_and_meet). It stays between the statements that it stands between.
// m0 holds a load's LDS address and is written right before it; the compiler
// keeps nothing of its own there across a statement, and the clobber tells it
// not to. It warns at every use that m0 is a register that it reserves.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds(const char* base, uint32_t off, uint32_t block) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(block), "v"(off), "s"(base) : "m0");
}
__device__ __forceinline__ void to_lds(const void* p, uint32_t block) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(block), "v"(p) : "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// What one of NW waves loads of one operand's tile: block q * NW + wave of 1 KiB.
template <typename T, int TILE, bool ROWS_K, int NW>
struct Loader {
  static constexpr int BLOCKS = TILE / 8 / NW;   // per wave
  static constexpr int LINES = ROWS_K ? 512 / TILE : 8;   // lines of a block: depths or rows
  uint32_t off[ROWS_K ? 1 : BLOCKS];         // byte offset of this lane's chunk
  uint32_t line;                             // first depth (ROWS_K) or first chunk of this lane
  const char* base;                          // tile's corner, at depth 0
  int64_t step;                              // bytes between depths (ROWS_K)

  __device__ __forceinline__ void init(const void* p, int64_t ld, uint32_t r0, uint32_t rows, uint32_t wave) {
    const uint32_t lane = threadIdx.x & 63u;
    if constexpr (ROWS_K) {
      constexpr uint32_t CHUNKS = TILE / 8;
      line = wave * LINES + lane / CHUNKS;
      uint32_t c = (lane % CHUNKS) ^ (2u * (line & 3u));
      const uint32_t last = (rows - r0 - 1u) / 8u;    // a line holds its last chunk whole
      if (c > last) c = last;                         // past it: a chunk again, for rows that nothing stores
      off[0] = (uint32_t)(line * ld * sizeof(T)) + c * 16u;
      base = reinterpret_cast<const char*>(static_cast<const T*>(p) + r0);
      step = ld * sizeof(T);
    } else {
      line = (lane & 7u) ^ (lane >> 3);
#pragma unroll
      for (int q = 0; q < BLOCKS; ++q) {
        uint32_t r = (q * NW + wave) * 8u + (lane >> 3);
        if (r >= rows - r0) r = rows - r0 - 1u;
        off[q] = (uint32_t)(r * ld * sizeof(T)) + line * 16u;
      }
      base = reinterpret_cast<const char*>(static_cast<const T*>(p) + (int64_t)r0 * ld);
      step = sizeof(T);
    }
  }

  // Block q of the depths [k0, k0 + 64), all there, into the tile at `lds`.
  __device__ __forceinline__ void load(uint32_t lds, uint32_t k0, int q, uint32_t wave) const {
    const char* const at = base + (int64_t)k0 * step;
    if constexpr (ROWS_K) to_lds(at + (int64_t)(q * NW * LINES) * step, off[0], lds + (q * NW + wave) * 1024u);
    else to_lds(at, off[q], lds + (q * NW + wave) * 1024u);
  }

  // All blocks of the depths [k0, k0 + 64), those from k on zero.
  __device__ __forceinline__ void load_end(uint32_t lds, uint32_t k0, uint32_t k, uint32_t wave) const {
    const char* const at = base + (int64_t)k0 * step;
#pragma unroll
    for (int q = 0; q < BLOCKS; ++q) {
      const char* src;
      if constexpr (ROWS_K) src = k0 + q * NW * LINES + line < k ? at + (int64_t)(q * NW * LINES) * step + off[0] : nullptr;
      else src = k0 + line * 8u < k ? at + off[q] : nullptr;
      to_lds(src ? src : reinterpret_cast<const char*>(&kZeros), lds + (q * NW + wave) * 1024u);
    }
  }
};

// A fragment for the 16 x 16 x 32 matrix instruction: lane l holds row l % 16,
// depths 8 (l / 16) + 0..7 of the kk-th thirty-two.
template <typename T, int TILE, bool ROWS_K>
struct Fragments {
  typedef typename Vec<T>::x8 x8;
  uint32_t at[ROWS_K ? 4 : 2];
  // r0: the wave's first row, a multiple of 32, and of 64 where it has more than 32.
  __device__ __forceinline__ void init(uint32_t r0) {
    const uint32_t l = threadIdx.x & 63u;
    if constexpr (ROWS_K) {
      // A group of 16 lanes reads four depths of one 32-byte piece, 8 bytes a
      // lane, and gets each row's four depths.
      const uint32_t j = l & 15u, depth = (l >> 4) * 8u + (j >> 2);
#pragma unroll
      for (uint32_t p = 0; p < 4; ++p)
        at[p] = depth * (TILE * 2u) + r0 / 64u * 128u + (((r0 / 16u + p) & 3u) ^ (j >> 2)) * 32u + (j & 3u) * 8u;
    } else {
#pragma unroll
      for (uint32_t kk = 0; kk < 2; ++kk) at[kk] = (r0 + (l & 15u)) * 128u + (((kk * 4u + (l >> 4)) ^ (l & 7u)) << 4);
    }
  }
  // The wave's rows [16 x, 16 x + 16), the kk-th thirty-two depths.
  __device__ __forceinline__ x8 read(const char* lds, int x, int kk) const {
    if constexpr (ROWS_K) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4* P;
      const char* const p = lds + at[x & 3] + (x >> 2) * 128 + kk * (32 * TILE * 2);
      union {
        s16x4 half[2];
        x8 all;
      } u;
      u.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
      u.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * TILE * 2));
      return u.all;
    } else {
      return *reinterpret_cast<const x8*>(lds + at[kk] + x * 2048);
    }
  }
};

// Waits until at most N of the wave's loads are outstanding and its LDS reads
// are done, then meets the workgroup.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(N % 16 + N / 16 * 0x4000 + 0x0070);   // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

struct TileArgs {
  GemmArgs g;
  uint32_t tiles_n, tiles;  // tiles across, in all
  uint32_t depth;           // k of one split, a multiple of kDepth
  float* partial;           // [splits][m][n], or null: one split, with the epilogue
};

// Workgroup -> tile. Workgroups go round the 8 XCDs, each with an L2 of its
// own: an XCD takes consecutive tiles, and tiles run down 8 rows before the
// next column, so that what an XCD works on at a time shares operands.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles, uint32_t tiles_n, uint32_t* ti, uint32_t* tj) {
  const uint32_t xcd = id & 7u, each = tiles >> 3, more = tiles & 7u;
  const uint32_t t = xcd * each + (xcd < more ? xcd : more) + (id >> 3);
  const uint32_t band = 8u * tiles_n, first = t / band * 8u, tiles_m = tiles / tiles_n;
  const uint32_t high = tiles_m - first < 8u ? tiles_m - first : 8u, in = t % band;
  *ti = first + in % high;
  *tj = in / high;
}

// C's TM x TN tile on WM x WN waves, each in 16 x 16 blocks. The depth runs
// through NS buffers: while the matrix cores work on one, the loads of the
// next NS - 1 are under way. B's fragments take the matrix instruction's rows,
// so a lane's sums are neighbours in a row of C. The 16 x 16 x 32 instruction
// moves a fifth less through the registers for a product than 32 x 32 x 16,
// and where power bounds the clock that is time: 8192^3 in 750 to 810 us
// by card (1467 to 1353 TFLOP/s) plain, 831 to 893 with gelu, bias, residual and
// z; the matrix cores are busy in 72 to 77 % and 70 to 72 % of the cycles, at the
// clock that the power leaves. A few hundred rows fill the chip once or less,
// and then a step waits for its loads: 1024 x 4096 x 4096 in 128 x 128 tiles, two
// buffers, takes 61 us with the matrix cores busy in 25 % of the cycles. Eight waves of
// 128 x 64 read 192 KiB of LDS a step, as long as its products take; four of
// 128 x 128 would read 128 and have no registers left.
template <int TM, int TN, int NS>
constexpr int kTileBytes = NS * (TM + TN) * 128;

template <typename T, int TM, int TN, int WM, int WN, int NS, bool A_ROWS_K, bool B_ROWS_K>
__device__ __forceinline__ void tile_body(const TileArgs& t, uint32_t id, char* lds) {
  constexpr int NW = WM * WN, MI = TM / WM / 16, NI = TN / WN / 16, BYTES = (TM + TN) * 128;
  constexpr int LA = TM / 8 / NW, LOADS = LA + TN / 8 / NW;
  constexpr int PITCH = TN / WN + 4;
  static_assert(NW * 32 * PITCH * 4 <= NS * BYTES, "the epilogue's blocks fit the buffers");
  static_assert((NS - 1) * LOADS < 64, "the wait count fits its field");
  const GemmArgs& g = t.g;
  uint32_t ti, tj;
  tile_of(id, t.tiles, t.tiles_n, &ti, &tj);
  const uint32_t i0 = ti * TM, j0 = tj * TN, lane = threadIdx.x & 63u;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wi = wave / WN * (TM / WM),
                 wj = wave % WN * (TN / WN);
  const uint32_t k_first = blockIdx.y * t.depth, k_last = min(g.k, k_first + t.depth);
  const uint32_t steps = k_last > k_first ? (k_last - k_first + kDepth - 1) / kDepth : 0u;
  Loader<T, TM, A_ROWS_K, NW> la;
  Loader<T, TN, B_ROWS_K, NW> lb;
  la.init(g.a, g.lda, i0, g.m, wave);
  lb.init(g.b, g.ldb, j0, g.n, wave);
  Fragments<T, TM, A_ROWS_K> ra;
  Fragments<T, TN, B_ROWS_K> rb;
  ra.init(wi);
  rb.init(wj);
  f32x4 c[MI][NI];
#pragma unroll
  for (int x = 0; x < MI; ++x)
#pragma unroll
    for (int y = 0; y < NI; ++y) c[x][y] = f32x4(0.0f);
  typename Vec<T>::x8 fa[2][MI], fb[2][NI];
  const uint32_t lds_at = lds_address(lds);

  // Depth of step s. Rows a power of two apart put one depth of all of them on
  // few memory channels, so the XCDs start at different depths and go round.
  const uint32_t whole = (k_last - k_first) / kDepth, start = whole / 8u * (blockIdx.x & 7u);
  const auto depth_of = [&](uint32_t s) {
    const uint32_t turned = s + start < whole ? s + start : s + start - whole;
    return k_first + (s < whole ? turned : s) * kDepth;
  };
  const auto load_end = [&](uint32_t s) {
    const uint32_t buf = lds_at + (s % NS) * BYTES, k0 = depth_of(s);
    la.load_end(buf, k0, k_last, wave);
    lb.load_end(buf + TM * 128, k0, k_last, wave);
  };
  // Half a step, in the order that stands here: the products of the fragments
  // in `from`; between them, over three quarters of the time, the reads of the
  // kk-th half of step `at` into the other set, and evenly the loads of step
  // `ahead`. A product waits only for its own fragments, which come in the
  // order of their use.
  const auto phase = [&](auto from_, uint32_t at, auto kk_, auto loads_, uint32_t ahead) {
    constexpr int from = from_, kk = kk_, loads = loads_, M = MI * NI, F = MI + NI, SPAN = M * 3 / 4;
    const char* const buf = lds + (at % NS) * BYTES;
    const uint32_t to = lds_at + (ahead % NS) * BYTES, k0 = depth_of(ahead);
    each<M>([&](auto i_) {
      constexpr int i = i_, x = i / NI, y = i % NI;
      constexpr int f0 = i >= SPAN ? F : i * F / SPAN, f1 = i + 1 >= SPAN ? F : (i + 1) * F / SPAN;
      constexpr int l0 = i * loads / M, l1 = (i + 1) * loads / M;
      c[x][y] = mfma(fb[from][y], fa[from][x], c[x][y]);
      each<f1 - f0>([&](auto f_) {
        constexpr int f = f0 + f_;
        if constexpr (f >= 1 && f <= NI) fb[from ^ 1][f - 1] = rb.read(buf + TM * 128, f - 1, kk);
        else fa[from ^ 1][f ? f - NI : 0] = ra.read(buf, f ? f - NI : 0, kk);
      });
      each<l1 - l0>([&](auto l_) {
        constexpr int l = l0 + l_;
        if constexpr (l < LA) la.load(to, k0, l, wave);
        else lb.load(to + TM * 128, k0, l - LA, wave);
      });
      if constexpr (f1 > f0 || l1 > l0) __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_sched_barrier(0);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

  if (steps > 0) {
#pragma unroll
    for (uint32_t s = 0; s < NS; ++s)
      if (s < steps) load_end(s);
    if (steps >= NS) wait_and_meet<(NS - 1) * LOADS>();
    else wait_and_meet<0>();
    fa[0][0] = ra.read(lds, 0, 0);
#pragma unroll
    for (int y = 0; y < NI; ++y) fb[0][y] = rb.read(lds + TM * 128, y, 0);
#pragma unroll
    for (int x = 1; x < MI; ++x) fa[0][x] = ra.read(lds, x, 0);
    // Where a step behaves as most do: more than the buffers hold ahead of
    // it, and the tiles that it loads are whole.
    uint32_t s = 0;
    for (; s + NS < whole; ++s) {
      phase(I0{}, s, I1{}, I0{}, s);
      // The next step's tiles are here, and no wave needs this one's again.
      wait_and_meet<(NS - 2) * LOADS>();
      phase(I1{}, s + 1, I0{}, std::integral_constant<int, LOADS>{}, s + NS);
    }
    for (; s < steps; ++s) {
      phase(I0{}, s, I1{}, I0{}, s);
      wait_and_meet<0>();
      if (s + NS < steps) load_end(s + NS);
      phase(I1{}, s + 1 < steps ? s + 1 : s, I0{}, I0{}, s);   // the last step's reads are of no use, and in bounds
    }
  }
  wait_and_meet<0>();   // no wave reads the buffers any more

  // A wave turns its blocks through shared memory of its own, 32 rows at a
  // time, so that C's rows are read and written in whole lines.
  float* const turn = reinterpret_cast<float*>(lds) + wave * (32 * PITCH);
  float* const partial = t.partial ? t.partial + (size_t)blockIdx.y * g.m * g.n : nullptr;
  constexpr int ACROSS = TN / WN / 8;   // lanes across the wave's columns, eight each
  constexpr int EACH = 32 * ACROSS / 64, DOWN = 64 / ACROSS;   // rows of a lane, rows of a wave at a time
  const uint32_t row = lane / ACROSS, col = lane % ACROSS * 8u, j = j0 + wj + col;
  each<MI / 2>([&](auto at) {
    constexpr int x = at;
    const uint32_t first = i0 + wi + x * 32u + row;
    typename Vec<T>::x8 residual[EACH];
    if (!partial) {
#pragma unroll
      for (int e = 0; e < EACH; ++e) residual[e] = residual8<T>(g, first + e * DOWN, j);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int y = 0; y < NI; ++y)
        *reinterpret_cast<f32x4*>(turn + (h * 16 + (lane & 15u)) * PITCH + y * 16 + (lane >> 4) * 4u) = c[2 * x + h][y];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const uint32_t i = first + e * DOWN;
      f32x8 v;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(turn + (row + e * DOWN) * PITCH + col);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(turn + (row + e * DOWN) * PITCH + col + 4);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        v[n] = lo[n];
        v[n + 4] = hi[n];
      }
      if (!partial) epilogue8<T>(g, i, j, v, residual[e]);
      else if (i < g.m && j < g.n)
        store8<float>(partial + (size_t)i * g.n + j, v, g.n - j < 8u ? (int)(g.n - j) : 8);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  });
}

template <typename T, int TM, int TN, int WM, int WN, int NS, bool A_ROWS_K, bool B_ROWS_K>
__global__ __launch_bounds__(WM * WN * 64) void tile_kernel(TileArgs t) {
  __shared__ __align__(1024) char lds[kTileBytes<TM, TN, NS>];
  tile_body<T, TM, TN, WM, WN, NS, A_ROWS_K, B_ROWS_K>(t, blockIdx.x, lds);
}

// The two products of a backward pass in one launch, dw's tiles (both operands
// with their rows contiguous) and dx's: neither leaves CUs idle at its end, and
// where one has few long tiles the other's short ones fill in beside them.
template <typename T, bool DW_FIRST>
__global__ __launch_bounds__(512) void pair_kernel(TileArgs dw, TileArgs dx) {
  __shared__ __align__(1024) char lds[kTileBytes<256, 256, 2>];
  const uint32_t first = DW_FIRST ? dw.tiles : dx.tiles;
  if ((blockIdx.x < first) == DW_FIRST)
    tile_body<T, 256, 256, 2, 4, 2, true, true>(dw, DW_FIRST ? blockIdx.x : blockIdx.x - first, lds);
  else
    tile_body<T, 256, 256, 2, 4, 2, false, true>(dx, DW_FIRST ? blockIdx.x - first : blockIdx.x, lds);
}

// ---- a few rows -------------------------------------------------------------

// Up to 16 R rows of A against 16 rows of B a workgroup, both with the depth
// contiguous and at any alignment. Bound by reading B once: it goes straight
// to registers, and the eight waves take the depth's 64-deep chunks in turn,
// so that a workgroup has all of a depth of 2048 under way at once; their sums
// meet in shared memory. Two workgroups share a CU, so one's loads run beside
// the other's sums (sixteen waves: 8192 from 2048 12.2 us instead of 10.2,
// 2048 from 4096 the same). Four lanes read 64 consecutive bytes of a row. One
// token of 4096 to 2048: 8.6 us, of which a workgroup's two bursts, the launch
// and the sums' meeting take 6.4 (4096 to 256, memory idle); to 4096 from 2048, one
// burst, 7.0. Every workgroup reads all of x: 32 tokens of 2048 to 4096 take 10.2.
// 32 tokens, 1024 to 1024: 5.9 us (7.9 in tiles, split and joined).
template <typename T, int R>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4, 4))) void rows_kernel(TileArgs t) {
  const GemmArgs& g = t.g;
  constexpr int WAVES = 8, PITCH = 20;
  typedef typename Vec<T>::x8 x8;
  __shared__ __align__(16) float lds[WAVES][16 * R][PITCH];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, r = lane & 15u, k_lane = (lane >> 4) * 8u;
  const uint32_t j0 = blockIdx.x * 16u;
  const uint32_t k_first = blockIdx.y * t.depth, k_end = min(g.k, k_first + t.depth);
  const T* a[R];
#pragma unroll
  for (int q = 0; q < R; ++q) a[q] = static_cast<const T*>(g.a) + (int64_t)min(r + 16u * q, g.m - 1u) * g.lda + k_lane;
  const T* const b = static_cast<const T*>(g.b) + (int64_t)min(j0 + r, g.n - 1u) * g.ldb + k_lane;
  f32x4 c[R];
#pragma unroll
  for (int q = 0; q < R; ++q) c[q] = f32x4(0.0f);
  uint32_t s = k_first / 64u + wave;
  // U chunks at once while the wave has as many whole ones
  const auto bursts = [&](auto unroll) {
    constexpr int U = decltype(unroll)::value;
    for (; s + (U - 1) * WAVES < k_end / 64u; s += U * WAVES) {
      x8 fb[U][2], fa[U][R][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) fb[u][h] = load8(b + (s + u * WAVES) * 64u + h * 32, 8);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) fa[u][q][h] = load8(a[q] + (s + u * WAVES) * 64u + h * 32, 8);
      __builtin_amdgcn_sched_barrier(0);   // every load is under way before the first product waits
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) c[q] = mfma(fb[u][h], fa[u][q][h], c[q]);
    }
  };
  bursts(std::integral_constant<int, 4>{});
  bursts(std::integral_constant<int, 2>{});
  for (; s * 64u < k_end; s += WAVES) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = s * 64u + h * 32u + k_lane;
      const int valid = k < k_end ? (int)min(8u, k_end - k) : 0;
      const x8 fb = load8(b + s * 64u + h * 32, valid);
#pragma unroll
      for (int q = 0; q < R; ++q) c[q] = mfma(fb, load8(a[q] + s * 64u + h * 32, valid), c[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < R; ++q) *reinterpret_cast<f32x4*>(&lds[wave][r + 16 * q][(lane >> 4) * 4u]) = c[q];
  __syncthreads();
  const uint32_t i = threadIdx.x / 2u, j = threadIdx.x % 2u * 8u;
  if (i >= 16u * R) return;
  f32x8 v = f32x8(0.0f);
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const f32x4 lo = *reinterpret_cast<const f32x4*>(&lds[w][i][j]), hi = *reinterpret_cast<const f32x4*>(&lds[w][i][j + 4]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] += lo[e];
      v[e + 4] += hi[e];
    }
  }
  if (!t.partial) epilogue8<T>(g, i, j0 + j, v, residual8<T>(g, i, j0 + j));
  else if (i < g.m && j0 + j < g.n)
    store8<float>(t.partial + ((size_t)blockIdx.y * g.m + i) * g.n + j0 + j, v,
                  g.n - j0 - j < 8u ? (int)(g.n - j0 - j) : 8);
}

// The splits' sums in order, then the epilogue. A latency: 3.0 us for four
// splits of 32 x 4096.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs g, const float* partial, int splits) {
  const uint32_t across = cdiv(g.n, 8);
  const uint64_t all = (uint64_t)g.m * across, step = (uint64_t)gridDim.x * 256u;
  for (uint64_t e = (uint64_t)blockIdx.x * 256u + threadIdx.x; e < all; e += step) {
    const uint32_t i = (uint32_t)(e / across), j = (uint32_t)(e % across) * 8u;
    const int valid = g.n - j < 8u ? (int)(g.n - j) : 8;
    f32x8 c = load8(partial + (size_t)i * g.n + j, valid);
#pragma unroll 4
    for (int s = 1; s < splits; ++s) c += load8(partial + ((size_t)s * g.m + i) * g.n + j, valid);
    epilogue8<T>(g, i, j, c, residual8<T>(g, i, j));
  }
}

// Lines copied to a distance that is a multiple of eight, zero past their end:
// up to three operands in one launch, since the tiles' loads take whole 16-byte
// chunks. 333 x 1001 and 777 x 1001: 3.7 us, and a product of 12.8 that takes 8.6
// from 1000 on 16-byte boundaries.
struct PadArgs {
  const void* p[3];
  int64_t ld[3];
  void* out[3];
  uint32_t cols[3];
  uint64_t end[3];   // items (groups of eight) up to each one's last
};
template <typename T>
__global__ __launch_bounds__(256) void pad_kernel(PadArgs a) {
  const uint64_t step = (uint64_t)gridDim.x * 256u;
  for (uint64_t e = (uint64_t)blockIdx.x * 256u + threadIdx.x; e < a.end[2]; e += step) {
    const int w = e < a.end[0] ? 0 : (e < a.end[1] ? 1 : 2);
    const uint64_t item = w ? e - a.end[w - 1] : e;
    const uint32_t cols = a.cols[w], across = cdiv(cols, 8), j = (uint32_t)(item % across) * 8u;
    const T* const from = static_cast<const T*>(a.p[w]) + (int64_t)(item / across) * a.ld[w] + j;
    store8<T>(static_cast<T*>(a.out[w]) + item * 8u, load8(from, cols - j < 8u ? (int)(cols - j) : 8), 8);
  }
}

// ---- launches ---------------------------------------------------------------

uint32_t grid_of(uint64_t items) {
  const uint64_t groups = (items + 255) / 256;
  return (uint32_t)(groups < 8192 ? (groups ? groups : 1) : 8192);
}

template <typename T, int TM, int TN, int WM, int WN, int NS>
hipError_t launch_tiles(TileArgs t, uint32_t splits, hipStream_t stream) {
  const GemmArgs& g = t.g;
  t.tiles_n = cdiv(g.n, TN);
  t.tiles = cdiv(g.m, TM) * t.tiles_n;
  const dim3 grid(t.tiles, splits);
  if (!g.a_rows_k && !g.b_rows_k) tile_kernel<T, TM, TN, WM, WN, NS, false, false><<<grid, WM * WN * 64, 0, stream>>>(t);
  else if (!g.a_rows_k) tile_kernel<T, TM, TN, WM, WN, NS, false, true><<<grid, WM * WN * 64, 0, stream>>>(t);
  else tile_kernel<T, TM, TN, WM, WN, NS, true, true><<<grid, WM * WN * 64, 0, stream>>>(t);
  return hipGetLastError();
}

template <typename T, int R>
hipError_t launch_rows(const TileArgs& t, uint32_t splits, hipStream_t stream) {
  rows_kernel<T, R><<<dim3(cdiv(t.g.n, 16), splits), 512, 0, stream>>>(t);
  return hipGetLastError();
}

// Copies the operands that the tiles cannot load as they stand to `space`,
// which moves on, and points them there.
template <typename T>
hipError_t pad_lines(Lines* l, int count, char** space, hipStream_t stream) {
  PadArgs pad{};
  uint64_t items = 0;
  for (int i = 0; i < 3; ++i) {
    if (i < count && l[i].p && !lines_as_is(l[i])) {
      const uint32_t across = cdiv(l[i].cols, 8);
      pad.p[i] = l[i].p;
      pad.ld[i] = l[i].ld;
      pad.out[i] = *space;
      pad.cols[i] = l[i].cols;
      items += (uint64_t)l[i].lines * across;
      l[i].p = *space;
      l[i].ld = (int64_t)across * 8;
      l[i].whole = true;
      *space += padded_bytes(l[i].lines, l[i].cols);
    }
    pad.end[i] = items;
  }
  if (items == 0) return hipSuccess;
  pad_kernel<T><<<grid_of(items), 256, 0, stream>>>(pad);
  return hipGetLastError();
}

template <typename T>
hipError_t gemm_typed(const GemmArgs& given, hipStream_t stream) {
  TileArgs t{};
  t.g = given;
  GemmArgs& g = t.g;
  Lines l[2] = {{g.a, g.lda, g.a_rows_k ? g.k : g.m, g.a_rows_k ? g.m : g.k, g.a_whole},
                {g.b, g.ldb, g.b_rows_k ? g.k : g.n, g.b_rows_k ? g.n : g.k, g.b_whole}};
  const Shape s = shape_of(g.m, g.n, g.k, g.a_rows_k, g.b_rows_k, lines_as_is(l[0]) && lines_as_is(l[1]));
  hipError_t rc = hipSuccess;
  char* space = static_cast<char*>(g.workspace);
  if (s.cut >= T64x64 && g.k > 0) {   // the tiles' loads go by whole chunks
    if ((rc = pad_lines<T>(l, 2, &space, stream)) != hipSuccess) return rc;
    g.a = l[0].p;
    g.lda = l[0].ld;
    g.b = l[1].p;
    g.ldb = l[1].ld;
  }
  t.depth = s.depth;
  t.partial = s.splits > 1 ? reinterpret_cast<float*>(space) : nullptr;
  switch (s.cut) {
    case ROWS16: rc = launch_rows<T, 1>(t, s.splits, stream); break;
    case ROWS32: rc = launch_rows<T, 2>(t, s.splits, stream); break;
    case T64x64: rc = launch_tiles<T, 64, 64, 2, 2, 4>(t, s.splits, stream); break;
    case T64x128: rc = launch_tiles<T, 64, 128, 2, 2, 3>(t, s.splits, stream); break;
    case T128x128: rc = launch_tiles<T, 128, 128, 2, 2, 2>(t, s.splits, stream); break;
    default: rc = launch_tiles<T, 256, 256, 2, 4, 2>(t, s.splits, stream); break;
  }
  if (rc != hipSuccess || s.splits == 1) return rc;
  join_kernel<T><<<grid_of((uint64_t)g.m * cdiv(g.n, 8)), 256, 0, stream>>>(g, t.partial, (int)s.splits);
  return hipGetLastError();
}

TileArgs whole_tiles(const GemmArgs& g) {
  TileArgs t{};
  t.g = g;
  t.tiles_n = cdiv(g.n, 256);
  t.tiles = cdiv(g.m, 256) * t.tiles_n;
  t.depth = cdiv(g.k ? g.k : 1, kDepth) * kDepth;
  return t;
}

template <typename T>
hipError_t pair_typed(const GemmArgs& dx, const GemmArgs& dw, hipStream_t stream) {
  const TileArgs tx = whole_tiles(dx), tw = whole_tiles(dw);
  if (dw.k >= dx.k) pair_kernel<T, true><<<tx.tiles + tw.tiles, 512, 0, stream>>>(tw, tx);   // long tiles first
  else pair_kernel<T, false><<<tx.tiles + tw.tiles, 512, 0, stream>>>(tw, tx);
  return hipGetLastError();
}

}  // namespace

bool lines_as_is(const Lines& l) {
  return ((uintptr_t)l.p & 15u) == 0 && l.ld % 8 == 0 && (l.whole || l.cols % 8 == 0) && l.ld < (1 << 22);
}
size_t padded_bytes(uint32_t lines, uint32_t cols) {
  return ((size_t)lines * (cdiv(cols, 8) * 8u) * 2u + 255) & ~(size_t)255;
}

hipError_t launch_pad(Lines* l, int count, int dtype, void* space, hipStream_t stream) {
  char* at = static_cast<char*>(space);
  return dtype == ARX_BF16 ? pad_lines<__bf16>(l, count, &at, stream) : pad_lines<_Float16>(l, count, &at, stream);
}

hipError_t launch_gemm(const GemmArgs& g, int dtype, hipStream_t stream) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  return dtype == ARX_BF16 ? gemm_typed<__bf16>(g, stream) : gemm_typed<_Float16>(g, stream);
}

hipError_t launch_gemm_pair(const GemmArgs& dx, const GemmArgs& dw, int dtype, hipStream_t stream) {
  // dx: [m][k] over n; dw: [n][k] over m
  if (dx.m > 0 && dx.n > 0 && dw.m > 0 && worth_pairing(dx.m, dw.m, dx.n))
    return dtype == ARX_BF16 ? pair_typed<__bf16>(dx, dw, stream) : pair_typed<_Float16>(dx, dw, stream);
  const hipError_t rc = launch_gemm(dx, dtype, stream);
  return rc == hipSuccess ? launch_gemm(dw, dtype, stream) : rc;
}

static size_t sums_of(const Shape& s, uint32_t m, uint32_t n) { return s.splits > 1 ? (size_t)s.splits * m * n * 4u : 0; }

size_t gemm_splits_workspace(uint32_t m, uint32_t n, uint32_t k, bool a_rows_k, bool b_rows_k) {
  return sums_of(shape_of(m, n, k, a_rows_k, b_rows_k, true), m, n);
}

size_t gemm_workspace(uint32_t m, uint32_t n, uint32_t k, bool aligned) {
  const Shape s = shape_of(m, n, k, false, false, true);
  size_t bytes = sums_of(s, m, n);
  if (aligned && k % 8 == 0) return bytes;
  // enough as well where they are aligned after all
  const Shape o = shape_of(m, n, k, false, false, false);
  const size_t sums = sums_of(o, m, n) + (o.cut >= T64x64 ? padded_bytes(m, k) + padded_bytes(n, k) : 0);
  return sums > bytes ? sums : bytes;
}

}  // namespace arx
