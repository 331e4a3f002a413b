// Tensor-core GEMM for the six contractions of the MLP block (sm_103a).
//
//   C[m, n] = Σ_segments Σ_k A(m, k)·B(n, k)   (float32 accumulation in TMEM)
//
// covering: fc1 column-parallel forward (U_i = X·A_i, GeLU/SwiGLU epilogue),
// fc2 row-parallel forward (P_i = Y_i·B_i as float32 partials, or the shard sum
// folded into one accumulator), fc2 input gradient with the activation
// derivative fused (dU_i = act'(U_i) ⊙ dZ·B_iᵀ), both weight gradients
// (dB_i = Y_iᵀ·dZ, dA_i = Xᵀ·dU_i) and fc1's input gradient (Σ_i dU_i·A_iᵀ)
// ("Tensor Parallelism（TP）与 Sequence Parallelism（SP）", §2–§5;
// "tensor-parallelism-matrix-split", §Backward：为什么有些梯度需要求和).
//
// Two kernels: gemm_pair_kernel (every GEMM with M > 128) computes 256×256
// tiles on CTA pairs (clusters of 2) with tcgen05.mma cta_group::2 and a
// 6-stage ring, each CTA loading its own operand halves with plain TMA
// (described at its definition); gemm_kernel (M ≤ 128) is the single-CTA form
// below.
//
// Design (one CTA per SM, persistent over output tiles):
//   warp 0      TMA producer: 128-byte-swizzled 128×64 A and 256×64 B tiles
//               into a 4-stage shared-memory ring (mbarrier full/empty pairs);
//   warp 1      MMA issuer: tcgen05.mma cta_group::1 M=128 N=256 K=16 from
//               shared-memory descriptors into one of two TMEM accumulators;
//   warp 2      TMEM allocator (512 columns = two 128×256 fp32 accumulators);
//   warps 4-7   epilogue: tcgen05.ld of the finished accumulator (each warp its
//               32-lane quarter), activation math, outputs staged through a
//               per-warp shared-memory buffer and stored as whole 128-byte
//               lines, so the epilogue of tile t overlaps the MMAs of tile t+1.
// K-major and MN-major operands are both read straight from their row-major
// storage: for MN-major operands TMA loads 64(MN)×64(K) boxes and the UMMA
// descriptor walks them with LBO = 8 KB (next 64-wide MN block) and SBO = 1 KB
// (next 8 K-rows).  Ragged M, N and K are covered by TMA's zero fill and
// predicated stores.  Every mbarrier wait is bounded (device status word).
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "checkpoint.cuh"
#include "internal.h"

namespace tpmlp {
namespace tc {

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 64;  // 64 16-bit elements = one 128-byte swizzle row
constexpr int UMMA_K = 16;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK * 2;  // 16 KB
constexpr int B_BYTES = BN * BK * 2;  // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int TMEM_COLS = 2 * BN;
constexpr int MAX_MAPS = 32;
constexpr int MAX_SEGS = 16;
constexpr int MAX_PARTS = 16;
constexpr int GROUP_M = 16;
constexpr int NARROW_TN = 128;  // of the pair kernel
constexpr int NUM_BARS = 2 * STAGES + 5;
// Epilogue staging: two 32-row × 128-byte buffers for each of the 4 epilogue
// warps, after the 256-byte barrier block.
constexpr int EPI_STAGE_BYTES = 32 * 128;
constexpr int EPI_WARP_BYTES = 2 * EPI_STAGE_BYTES;
constexpr int EPI_SMEM_BYTES = 4 * EPI_WARP_BYTES;
constexpr size_t SMEM_BYTES = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + 256 + EPI_SMEM_BYTES;

// MN-major box: 64 elements along M/N (128 bytes) × 64 K-rows = 8 KB.
constexpr uint32_t MN_BOX_BYTES = 64 * BK * 2;

struct Seg {
  int32_t map_a, map_b, k_len, pad;
};

struct Params {
  CUtensorMap maps[MAX_MAPS];
  Seg segs[MAX_SEGS];
  int32_t seg_begin[MAX_PARTS + 1];
  int32_t M, N;           // logical output extent (N = F for SwiGLU fc1)
  int32_t mt, nt;         // tile counts along M and N
  int32_t nparts;         // output partials handled by this launch
  int32_t part_base;      // index of this launch's first partial
  int32_t swiglu_up_row;  // > 0: SwiGLU fc1, B rows of the up half start here
  // > 0: a K-major A operand is split along M into chunks of this many rows,
  // chunk j read through maps[seg.map_a + j] (the SP all-gather fused into the
  // loads: every 128-row block lies inside one chunk).
  int32_t a_chunk_rows;
  int32_t a_nchunks;
  int32_t pad1;
  unsigned* status;
  uint64_t timeout_ns;
  EpiParams epi;
};

// Tile t of an mt × nt grid per partial, in groups of GROUP_M rows.
__device__ __forceinline__ void decode_tile_grid(int t, int mt, int nt, int& part, int& mb, int& nb) {
  const int per_part = mt * nt;
  part = t / per_part;
  const int r = t - part * per_part;
  const int span = GROUP_M * nt;
  const int g = r / span;
  const int first_m = g * GROUP_M;
  const int gsz = min(mt - first_m, GROUP_M);
  const int rr = r - g * span;
  mb = first_m + rr % gsz;
  nb = rr / gsz;
}
__device__ __forceinline__ void decode_tile(int t, const Params& p, int& part, int& mb, int& nb) {
  decode_tile_grid(t, p.mt, p.nt, part, mb, nb);
}

// ---------------------------------------------------------------- epilogues
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
               : "memory");
  return v;
}

// Output staging.  After tcgen05.ld a lane holds one row, so storing straight
// from registers makes every warp store touch 32 rows × 16 bytes (32 lines).
// Instead lane r puts its row's 16-byte units u of a 128-byte line segment into
// slot u ^ (r & 7) of row r of a 32 × 128-byte buffer (conflict-free: the 8
// lanes of a quarter-warp hit 8 different slots), and the flush reads it back
// with 8 consecutive lanes on one row, so each warp store writes 4 whole lines.
__device__ __forceinline__ void stage_put(uint32_t buf, int lane, int unit, uint4 v) {
  sts128(buf + static_cast<uint32_t>(lane) * 128u + (static_cast<uint32_t>(unit ^ (lane & 7)) << 4), v);
}
// Writes the staged line segments of rows m0 .. m0 + 31: row m's segment starts
// at byte address line(m); rows at or past M and units at or past `units` are
// skipped.
template <typename LineFn>
__device__ __forceinline__ void stage_flush(uint32_t buf, int lane, int64_t m0, int64_t M, int units, LineFn line) {
  __syncwarp();
  const int u = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    const uint4 v = lds128(buf + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(u ^ (r & 7)) << 4));
    const int64_t m = m0 + r;
    if (m < M && u < units) *reinterpret_cast<uint4*>(line(m) + u * 16) = v;
  }
  __syncwarp();
}
// The read counterpart: loads the 128-byte line segments of rows m0 .. m0 + 31
// (row m's at byte address line(m), 8 lanes per row, rows at or past M and
// units at or past `units` read as zero) into the buffer in the same layout,
// for stage_get to hand each lane its own row's units.
// COHERENT: L2-coherent loads, for data this kernel writes back (main_grad);
// otherwise the read-only path.
template <bool COHERENT = false, typename LineFn>
__device__ __forceinline__ void stage_fill(uint32_t buf, int lane, int64_t m0, int64_t M, int units, LineFn line) {
  const int u = lane & 7;
  uint4 t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = m0 + i * 4 + (lane >> 3);
    if (m < M && u < units) {
      const char* a = line(m) + u * 16;
      t[i] = COHERENT ? __ldcg(reinterpret_cast<const uint4*>(a)) : ldg_nc_v4(a);
    } else {
      t[i] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    sts128(buf + static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(u ^ (r & 7)) << 4), t[i]);
  }
  __syncwarp();
}
__device__ __forceinline__ uint4 stage_get(uint32_t buf, int lane, int unit) {
  return lds128(buf + static_cast<uint32_t>(lane) * 128u + (static_cast<uint32_t>(unit ^ (lane & 7)) << 4));
}
// 16-byte units of a line segment starting at column n that lie (start) before N
__device__ __forceinline__ int units_before(int64_t N, int64_t n, int cols_per_unit) {
  const int64_t left = N - n;
  if (left <= 0) return 0;
  const int64_t u = (left + cols_per_unit - 1) / cols_per_unit;
  return u >= 8 ? 8 : static_cast<int>(u);
}

// fc2 input gradient epilogue for 8 columns: dU = act'(U) ⊙ dY.  SwiGLU:
// dG = dY·Up·silu'(G) and dUp = dY·silu(G), written to dU's gate and up halves.
// (packed into *gate, and for SwiGLU the up half into *up)
template <int DT>
__device__ __forceinline__ void epi_dact8(const EpiParams& e, const float* dy, uint4 u_raw, uint4 up_raw,
                                          uint4* gate, uint4* upo) {
  float u[8], r[8];
  unpack8<DT>(u_raw, u);
  if (e.act == ACT_SWIGLU) {
    float up[8], r2[8];
    unpack8<DT>(up_raw, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sg = sigmoid_f<false>(u[i]);
      r[i] = dy[i] * up[i] * (sg * (1.0f + u[i] * (1.0f - sg)));
      r2[i] = dy[i] * (u[i] * sg);
    }
    *gate = pack8<DT>(r);
    *upo = pack8<DT>(r2);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = dy[i] * act_grad<false>(e.act, u[i]);
  *gate = pack8<DT>(r);
}

// L2 prefetch of the saved U row segment a fc2-input-gradient tile will read,
// issued before the epilogue waits for the accumulator.
template <int TN, int EP>
__device__ __forceinline__ void epi_prefetch_aux(const Params& p, int64_t m, int nb, int elem_bytes, int w) {
  const EpiParams& e = p.epi;
  if (m >= p.M) return;
  if (e.kind == EPI_ACC_F32) {  // the float32 main_grad rows this tile will update
    const char* row = static_cast<const char*>(e.out) + (m * e.ldo + static_cast<int64_t>(nb) * TN) * 4;
    const int64_t left = (p.N - static_cast<int64_t>(nb) * TN) * 4;
#pragma unroll
    for (int b = 0; b < TN * 4 / 128; ++b)
      if (b * 128 < left) prefetch_l2(row + b * 128);
    return;
  }
  if constexpr (EP == EPI_DACT_CKPT) {  // the codes of the warp's half: TN/2 bytes a row
    static_assert(TN == 256, "a half is one line");
    const int64_t n0 = static_cast<int64_t>(nb) * TN + (w >> 2) * (TN / 2);
    if (n0 < p.N) {
      prefetch_l2(e.codes + m * e.ldc + n0);
      if (e.act == ACT_SWIGLU) prefetch_l2(e.codes + m * e.ldc + e.swiglu_F + n0);
    }
    return;
  }
  if (e.kind != EPI_DACT) return;
  const char* row = static_cast<const char*>(e.aux) + (m * e.ldaux + static_cast<int64_t>(nb) * TN) * elem_bytes;
  const int64_t left = (p.N - static_cast<int64_t>(nb) * TN) * elem_bytes;
#pragma unroll
  for (int b = 0; b < TN * 2 / 128; ++b) {
    if (b * 128 < left) {
      prefetch_l2(row + b * 128);
      if (e.act == ACT_SWIGLU) prefetch_l2(row + e.swiglu_F * elem_bytes + b * 128);
    }
  }
}

// Drains one 128-row × BN-column accumulator (this warp's 32 lanes = rows)
// from tensor memory and runs the epilogue.  All 32 lanes execute the
// tcgen05.ld instructions; rows past M only skip their stores.  `stage` is this
// warp's pair of staging buffers.
// HELD (GemmDesc::held) is a constant of the kernels, so that a block without a checkpoint
// has none of its code: asked for at run time it cost small blocks 2.5 to 5% (a step of 64
// tokens, h 256, f 1024: 65.6 µs against 62.4; 2048 tokens, h 1024, f 4096 with partial sums:
// 165.4 against 161.3), and the blocks with one 3 to 6% (GELU, 2048 tokens: 129.5 against 125.2).
template <int DT, int TN, bool HELD>
__device__ __forceinline__ void epilogue_tile(const Params& p, uint32_t trow, int64_t m, int nb, int part,
                                              uint32_t stage) {
  static_assert(TN % 64 == 0, "16-bit outputs are staged in 64-column line segments");
  const EpiParams& e = p.epi;
  if constexpr (HELD) {  // fc1's forward and fc2's input gradient have epilogues of their own then
    __builtin_assume(p.swiglu_up_row <= 0);
    __builtin_assume(e.kind != EPI_ACT && e.kind != EPI_DACT);
  }
  const int lane = static_cast<int>(m & 31);  // rows of a warp start at a multiple of 32
  const int64_t m0 = m - lane;
  const uint32_t buf0 = stage, buf1 = stage + EPI_STAGE_BYTES;
  if (p.swiglu_up_row > 0) {
    // SwiGLU fc1, per 64-column segment of the gate half (two 32-column chunks):
    // the gate and up halves of U go out through the two staging buffers, then
    // Y = silu(gate) · up through the first.
    static_assert(TN % 128 == 0, "SwiGLU tiles hold whole 64-column gate and up segments");
    using T = typename Storage<DT>::T;
    constexpr int64_t ES = static_cast<int64_t>(sizeof(T));
    char* ubase = static_cast<char*>(e.out);
    char* ybase = static_cast<char*>(e.out2);
#pragma unroll 1
    for (int sg = 0; sg < TN / 128; ++sg) {
      const int64_t nl = static_cast<int64_t>(nb) * (TN / 2) + sg * 64;
      const int units = units_before(p.N, nl, 8);
      uint4 yk[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float g[32], up[32];
        tmem_ld32(trow + (2 * sg + half) * 32, g);
        tmem_ld32(trow + TN / 2 + (2 * sg + half) * 32, up);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          stage_put(buf0, lane, half * 4 + j, pack8<DT>(g + 8 * j));
          stage_put(buf1, lane, half * 4 + j, pack8<DT>(up + 8 * j));
          float a[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = g[8 * j + i];
            a[i] = x * sigmoid_f<false>(x) * up[8 * j + i];
          }
          yk[half * 4 + j] = pack8<DT>(a);
        }
      }
      stage_flush(buf0, lane, m0, p.M, units, [&](int64_t mm) { return ubase + (mm * e.ldo + nl) * ES; });
      stage_flush(buf1, lane, m0, p.M, units,
                  [&](int64_t mm) { return ubase + (mm * e.ldo + e.swiglu_F + nl) * ES; });
#pragma unroll
      for (int j = 0; j < 8; ++j) stage_put(buf0, lane, j, yk[j]);
      stage_flush(buf0, lane, m0, p.M, units, [&](int64_t mm) { return ybase + (mm * e.ldo2 + nl) * ES; });
    }
    return;
  }
  if (e.kind == EPI_DACT) {
    // Per 64-column segment: the saved U (and for SwiGLU the up half) is read as
    // whole lines through the staging buffers, each lane takes its row's units,
    // and the buffers are then reused to stage dU.
    using T = typename Storage<DT>::T;
    const bool swi = e.act == ACT_SWIGLU;
    const int64_t nbase = static_cast<int64_t>(nb) * TN;
    const char* ubase = static_cast<const char*>(e.aux);
    char* obase = static_cast<char*>(e.out);
    constexpr int64_t ES = static_cast<int64_t>(sizeof(T));
#pragma unroll 1
    for (int sg = 0; sg < TN / 64; ++sg) {
      const int64_t nl = nbase + sg * 64;
      const int units = units_before(p.N, nl, 8);
      stage_fill(buf0, lane, m0, p.M, units, [&](int64_t mm) { return ubase + (mm * e.ldaux + nl) * ES; });
      if (swi)
        stage_fill(buf1, lane, m0, p.M, units,
                   [&](int64_t mm) { return ubase + (mm * e.ldaux + e.swiglu_F + nl) * ES; });
      uint4 ug[8], uu[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ug[j] = stage_get(buf0, lane, j);
        uu[j] = swi ? stage_get(buf1, lane, j) : make_uint4(0, 0, 0, 0);
      }
      __syncwarp();  // every lane has its units before the buffers take dU
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[32];
        tmem_ld32(trow + (2 * sg + half) * 32, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 g, u2;
          epi_dact8<DT>(e, v + 8 * j, ug[half * 4 + j], uu[half * 4 + j], &g, &u2);
          stage_put(buf0, lane, half * 4 + j, g);
          if (swi) stage_put(buf1, lane, half * 4 + j, u2);
        }
      }
      stage_flush(buf0, lane, m0, p.M, units, [&](int64_t mm) { return obase + (mm * e.ldo + nl) * ES; });
      if (swi)
        stage_flush(buf1, lane, m0, p.M, units,
                    [&](int64_t mm) { return obase + (mm * e.ldo + e.swiglu_F + nl) * ES; });
    }
    return;
  }
  if (e.kind == EPI_ACC_F32) {
    // main_grad += C, one 32-column (128-byte) line segment at a time: the
    // segment is read as whole lines with L2-coherent loads (this kernel writes
    // it back), each lane adds its row's accumulator values in place, and the
    // segment is written back as whole lines.
    char* base = static_cast<char*>(e.out);
    const int64_t nbase = static_cast<int64_t>(nb) * TN;
#pragma unroll 1
    for (int c = 0; c < TN / 32; ++c) {
      const int64_t nl = nbase + c * 32;
      const int units = units_before(p.N, nl, 4);
      auto line = [&](int64_t mm) { return base + (mm * e.ldo + nl) * 4; };
      stage_fill<true>(buf0, lane, m0, p.M, units, line);
      float v[32];
      tmem_ld32(trow + c * 32, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4 o = stage_get(buf0, lane, j);
        o.x = __float_as_uint(__uint_as_float(o.x) + v[4 * j]);
        o.y = __float_as_uint(__uint_as_float(o.y) + v[4 * j + 1]);
        o.z = __float_as_uint(__uint_as_float(o.z) + v[4 * j + 2]);
        o.w = __float_as_uint(__uint_as_float(o.w) + v[4 * j + 3]);
        stage_put(buf0, lane, j, o);
      }
      stage_flush(buf0, lane, m0, p.M, units, line);
    }
    return;
  }
  const int64_t nbase = static_cast<int64_t>(nb) * TN;
  if (e.kind == EPI_F32) {
    // float32 partials: a 32-column chunk is one 128-byte line segment
    char* base = static_cast<char*>(e.out) + static_cast<int64_t>(p.part_base + part) * e.part_stride * 4;
#pragma unroll 1
    for (int c = 0; c < TN / 32; ++c) {
      float v[32];
      tmem_ld32(trow + c * 32, v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        stage_put(buf0, lane, j,
                  make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                             __float_as_uint(v[4 * j + 3])));
      const int64_t nl = nbase + c * 32;
      stage_flush(buf0, lane, m0, p.M, units_before(p.N, nl, 4),
                  [&](int64_t mm) { return base + (mm * e.ldo + nl) * 4; });
    }
    return;
  }
  if (e.kind == EPI_STORE || e.kind == EPI_ACT) {
    using T = typename Storage<DT>::T;
    const bool act = e.kind == EPI_ACT;
    // HELD: the shard of the warp's first row, and that shard's first row, by one division a
    // tile (2048 tokens, h 1024, f 4096, SwiGLU: 184 -> 182 µs); without, one a row
    const int64_t shard0 = HELD && e.scatter ? m0 / e.rows_per_shard : 0;
    const int64_t row0 = shard0 * e.rows_per_shard;
#pragma unroll 1
    for (int c = 0; c < TN / 32; ++c) {
      float v[32];
      tmem_ld32(trow + c * 32, v);
      const int half = c & 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        stage_put(buf0, lane, half * 4 + j, pack8<DT>(v + 8 * j));
        if (act) {
          float a[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = act_fwd<false>(e.act, v[8 * j + i]);
          stage_put(buf1, lane, half * 4 + j, pack8<DT>(a));
        }
      }
      if (half) {
        const int64_t nl = nbase + (c - 1) * 32;
        const int units = units_before(p.N, nl, 8);
        if (e.kind == EPI_STORE && e.scatter) {
          stage_flush(buf0, lane, m0, p.M, units, [&](int64_t mm) {
            int64_t sh = shard0, r = mm - row0;
            if constexpr (HELD) {
              for (; r >= e.rows_per_shard; r -= e.rows_per_shard) ++sh;
            } else {
              sh = mm / e.rows_per_shard;
              r = mm - sh * e.rows_per_shard;
            }
            return static_cast<char*>(e.shard[sh]) + (r * e.ldo + nl) * static_cast<int64_t>(sizeof(T));
          });
        } else {
          char* base = static_cast<char*>(e.out);
          stage_flush(buf0, lane, m0, p.M, units,
                      [&](int64_t mm) { return base + (mm * e.ldo + nl) * static_cast<int64_t>(sizeof(T)); });
        }
        if (act) {
          char* base2 = static_cast<char*>(e.out2);
          stage_flush(buf1, lane, m0, p.M, units,
                      [&](int64_t mm) { return base2 + (mm * e.ldo2 + nl) * static_cast<int64_t>(sizeof(T)); });
        }
      }
    }
    return;
  }
}

// ---------------------------------------------------------------- checkpoint epilogues
// The block that keeps U in 8 bits (checkpoint.cuh).  A lane holds a row's 32
// consecutive accumulators after one tcgen05.ld: a group of the checkpoint, so its
// scale needs no exchange.  64 codes of a row are staged like the 16-bit outputs, as
// eight 8-byte units at a row pitch of 72 bytes: 16 lanes on one unit, or 8 lanes on
// each of two rows, meet 32 different banks.  8-byte units keep any f (a multiple of
// 8) aligned.
constexpr uint32_t CODE_PITCH = 72;

__device__ __forceinline__ void sts64(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
template <typename LineFn>
__device__ __forceinline__ void code_flush(uint32_t buf, int lane, int64_t m0, int64_t M, int units, LineFn line) {
  __syncwarp();
  const int u = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    const uint2 v = lds64(buf + static_cast<uint32_t>(r) * CODE_PITCH + static_cast<uint32_t>(u) * 8u);
    if (m0 + r < M && u < units) *reinterpret_cast<uint2*>(line(m0 + r) + u * 8) = v;
  }
  __syncwarp();
}
__device__ __forceinline__ void code_row_put(uint32_t buf, int lane, int half, const uint32_t* codes) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    sts64(buf + static_cast<uint32_t>(lane) * CODE_PITCH + static_cast<uint32_t>(half * 4 + j) * 8u,
          make_uint2(codes[2 * j], codes[2 * j + 1]));
}

// 32 float32 values of a row to 8 words of codes; returns the scale byte.  Columns at
// or past `left` hold another matrix's values or nothing: they count as zero.
// The float maximum passes over NaN and shows an infinity; only a group with one, or one
// that is cut off, is gone over bit by bit as checkpoint.cuh has it.
__device__ __forceinline__ uint32_t encode_group(const float* v, int64_t left, uint32_t* codes) {
  float tops[4] = {};  // four chains of dependent maxima instead of one
#pragma unroll
  for (int i = 0; i < 32; ++i) tops[i & 3] = fmaxf(tops[i & 3], fabsf(v[i]));
  uint32_t top = __float_as_uint(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
  if (left >= 32 && top < 0x7f800000u) {
    const uint32_t byte = ckpt_byte(top);
    const float inv = ckpt_inverse(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) codes[j] = ckpt_encode4<true>(v + 4 * j, inv);
    return byte;
  }
  const int have = static_cast<int>(left < 32 ? left : 32);
  top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, i < have ? ckpt_abs(v[i]) : 0u);
  const uint32_t byte = ckpt_byte(top);
  const float inv = ckpt_inverse(byte);
#pragma unroll
  for (int j = 0; j < 8; ++j) codes[j] = ckpt_encode4(v + 4 * j, inv);
  return byte;
}

// A row's G scale bytes from `first` on, `have` of them in the matrix, in one access where
// the pitch keeps them aligned.
template <int G>
__device__ __forceinline__ void put_scales(uint8_t* row, int64_t first, int64_t have, bool whole, uint32_t bytes) {
  if (whole && have >= G) {
    if constexpr (G == 4)
      *reinterpret_cast<uint32_t*>(row + first) = bytes;
    else
      *reinterpret_cast<uint16_t*>(row + first) = static_cast<uint16_t>(bytes);
    return;
  }
#pragma unroll
  for (int i = 0; i < G; ++i)
    if (i < have) row[first + i] = static_cast<uint8_t>(bytes >> (8 * i));
}
__device__ __forceinline__ uint32_t get_scales4(const uint8_t* row, int64_t first, int64_t have, bool whole) {
  if (whole && have >= 4) return *reinterpret_cast<const uint32_t*>(row + first);
  uint32_t bytes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < have) bytes |= static_cast<uint32_t>(row[first + i]) << (8 * i);
  return bytes;
}

// 1/(1 + e^-x) in four instructions (a product, 2^t, a sum, the approximate reciprocal),
// where Y and dU are rounded to 8 or 11 bits.  The product's rounding and log2 e's are in the
// exponent: far below zero, where the result is e^x, it is off by up to |x|·2^-23 of itself
// beside a few steps of float32 (2^-17 at x = −64), and it is 0 from x = −88 down, where e^x is
// below 2^-126.  2^t may flush to zero, since 1 is added to it.  The exact divide has a
// branch for every element, which keeps the epilogue's elements one behind the other.
__device__ __forceinline__ float sigmoid_short(float x) {
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return r;
}

// fn with the activation of one input as a constant: a test of it for every element would
// keep the elements one behind the other (GELU step of 2048 tokens, h 1024, f 4096: 157 µs,
// so 136; ReLU, 1024 tokens, h 1024, f 8192: 166, 149).
template <typename Fn>
__device__ __forceinline__ void by_activation(int act, Fn fn) {
  if (act == ACT_GELU)
    fn(std::integral_constant<int, ACT_GELU>{});
  else if (act == ACT_RELU)
    fn(std::integral_constant<int, ACT_RELU>{});
  else
    fn(std::integral_constant<int, ACT_IDENTITY>{});
}

// fc1 forward: the checkpoint of C, rounded once from the accumulator, and Y = act(C).
// A warp takes half of the tile's columns (`part`) of its 32 rows, 64 at a time through
// its one staging buffer.
template <int DT, int TN, typename Release>
__device__ __forceinline__ void epilogue_act_ckpt(const Params& p, uint32_t trow, int64_t m, int nb, int part,
                                                  uint32_t buf, Release release) {
  const EpiParams& e = p.epi;
  const int lane = static_cast<int>(m & 31);
  const int64_t m0 = m - lane;
  constexpr int64_t ES = static_cast<int64_t>(sizeof(typename Storage<DT>::T));
  char* ybase = static_cast<char*>(e.out2);
  const int64_t groups = (static_cast<int64_t>(p.N) + CKPT_GROUP - 1) / CKPT_GROUP;
  if (p.swiglu_up_row > 0) {
    // the tile is TN/2 gate columns and their up columns: Y, then both halves' codes
    static_assert(TN == 256, "a warp's half is 64 gate columns");
    const int64_t nl = static_cast<int64_t>(nb) * (TN / 2) + part * 64;
    const int units = units_before(p.N, nl, 8);
    uint32_t gc[16], uc[16], gs = 0, us = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float g[32], up[32];
      tmem_ld32(trow + (2 * part + half) * 32, g);
      tmem_ld32(trow + TN / 2 + (2 * part + half) * 32, up);
      if (half == 1) release();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = g[8 * j + i];
          a[i] = x * sigmoid_short(x) * up[8 * j + i];
        }
        stage_put(buf, lane, half * 4 + j, pack8<DT>(a));
      }
      const int64_t left = p.N - nl - half * 32;
      gs |= encode_group(g, left, gc + 8 * half) << (8 * half);
      us |= encode_group(up, left, uc + 8 * half) << (8 * half);
    }
    stage_flush(buf, lane, m0, p.M, units, [&](int64_t mm) { return ybase + (mm * e.ldo2 + nl) * ES; });
#pragma unroll
    for (int half = 0; half < 2; ++half) code_row_put(buf, lane, half, gc + 8 * half);
    code_flush(buf, lane, m0, p.M, units, [&](int64_t mm) { return e.codes + mm * e.ldc + nl; });
#pragma unroll
    for (int half = 0; half < 2; ++half) code_row_put(buf, lane, half, uc + 8 * half);
    code_flush(buf, lane, m0, p.M, units, [&](int64_t mm) { return e.codes + mm * e.ldc + e.swiglu_F + nl; });
    if (m < p.M) {
      uint8_t* row = e.scales + m * e.lds;
      const int64_t first = nl / CKPT_GROUP;
      put_scales<2>(row, first, groups - first, true, gs);
      put_scales<2>(row + groups, first, groups - first, groups % 2 == 0, us);
    }
    return;
  }
  uint32_t bytes = 0;
  const int64_t n0 = static_cast<int64_t>(nb) * TN + part * (TN / 2);
#pragma unroll 1
  for (int sg = 0; sg < TN / 128; ++sg) {
    const int64_t nl = n0 + sg * 64;
    const int units = units_before(p.N, nl, 8);
    uint32_t codes[16];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float v[32];
      tmem_ld32(trow + part * (TN / 2) + (2 * sg + half) * 32, v);
      if (half == 1 && sg + 1 == TN / 128) release();
      by_activation(e.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float a[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = act_fwd<false>(ACT, v[8 * j + i]);
          stage_put(buf, lane, half * 4 + j, pack8<DT>(a));
        }
      });
      bytes |= encode_group(v, p.N - nl - half * 32, codes + 8 * half) << (8 * (2 * sg + half));
    }
    stage_flush(buf, lane, m0, p.M, units, [&](int64_t mm) { return ybase + (mm * e.ldo2 + nl) * ES; });
#pragma unroll
    for (int half = 0; half < 2; ++half) code_row_put(buf, lane, half, codes + 8 * half);
    code_flush(buf, lane, m0, p.M, units, [&](int64_t mm) { return e.codes + mm * e.ldc + nl; });
  }
  if (m < p.M) {
    const int64_t first = n0 / CKPT_GROUP;
    put_scales<4>(e.scales + m * e.lds, first, groups - first, e.lds % 4 == 0, bytes);
  }
}

// fc2 input gradient: with U the checkpoint's values, dU = act'(U) ⊙ C, and Y = act(U),
// which fc2's weight gradient needs.  The warps share the tile as above, and take one
// group of 32 columns after the other by the same instructions: the first pass over
// straight-line code for all of them waits longer for its instructions than it computes,
// and 64 columns at a time leave no registers for the next codes (a step of 2048 tokens, h
// 1024, f 4096, SwiGLU: 204 µs, groups: 189).  Codes and scale bytes do not wait for the
// product: the first group's are loaded before the accumulator is waited for, the next
// group's before this one's arithmetic (186 -> 184).
//
// A group's 32 codes of a row are four 8-byte units: lane l loads unit l & 3 of row
// l / 4 + 8i, and hands them to the rows' lanes through shared memory (1 KB, unit u of row
// r in slot u ^ (r / 4 & 3): 16 lanes meet 32 banks either way).
struct CodesAhead {
  uint2 g[4], u[4];
  uint32_t gs = 0, us = 0;
};
template <typename LineFn>
__device__ __forceinline__ void code_load(uint2* t, int lane, int64_t m0, int64_t M, int units, LineFn line) {
  const int u = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + i * 8 + (lane >> 2);
    t[i] = m < M && u < units ? *reinterpret_cast<const uint2*>(line(m) + u * 8) : make_uint2(0, 0);
  }
}
__device__ __forceinline__ uint32_t code_slot(uint32_t buf, int r, int u) {
  return buf + static_cast<uint32_t>(r) * 32u + (static_cast<uint32_t>(u ^ (r >> 2 & 3)) << 3);
}
__device__ __forceinline__ void code_put(const uint2* t, uint32_t buf, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sts64(code_slot(buf, i * 8 + (lane >> 2), lane & 3), t[i]);
}
__device__ __forceinline__ void code_get(uint2* t, uint32_t buf, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) t[j] = lds64(code_slot(buf, lane, j));
}
__device__ __forceinline__ void codes_ahead(const Params& p, int64_t m, int64_t nl, CodesAhead& a) {
  const EpiParams& e = p.epi;
  const int lane = static_cast<int>(m & 31);
  const int units = units_before(p.N, nl, 8);
  code_load(a.g, lane, m - lane, p.M, units, [&](int64_t mm) { return e.codes + mm * e.ldc + nl; });
  if (e.act == ACT_SWIGLU)
    code_load(a.u, lane, m - lane, p.M, units, [&](int64_t mm) { return e.codes + mm * e.ldc + e.swiglu_F + nl; });
}
template <int TN>
__device__ __forceinline__ void codes_first(const Params& p, int64_t m, int nb, int part, CodesAhead& a) {
  const EpiParams& e = p.epi;
  const int64_t n0 = static_cast<int64_t>(nb) * TN + part * (TN / 2);
  codes_ahead(p, m, n0, a);
  if (m >= p.M) return;
  const int64_t groups = (static_cast<int64_t>(p.N) + CKPT_GROUP - 1) / CKPT_GROUP;
  const uint8_t* row = e.scales + m * e.lds;
  const int64_t first = n0 / CKPT_GROUP;
  a.gs = get_scales4(row, first, groups - first, e.lds % 4 == 0);
  if (e.act == ACT_SWIGLU) a.us = get_scales4(row + groups, first, groups - first, groups % 4 == 0);
}
// A row's 32 16-bit outputs: four 16-byte units at a pitch of 64 bytes, unit u in slot
// u ^ (r / 2 & 3), stored by 4 lanes a row.
__device__ __forceinline__ uint32_t group_slot(uint32_t buf, int r, int u) {
  return buf + static_cast<uint32_t>(r) * 64u + (static_cast<uint32_t>(u ^ (r >> 1 & 3)) << 4);
}
template <typename LineFn>
__device__ __forceinline__ void group_flush(uint32_t buf, int lane, int64_t m0, int64_t M, int units, LineFn line) {
  const int u = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    const uint4 v = lds128(group_slot(buf, r, u));
    if (m0 + r < M && u < units) *reinterpret_cast<uint4*>(line(m0 + r) + u * 16) = v;
  }
}
template <int DT, int TN, typename Release>
__device__ __forceinline__ void epilogue_dact_ckpt(const Params& p, uint32_t trow, int64_t m, int nb, int part,
                                                   uint32_t buf, CodesAhead& held, Release release) {
  const EpiParams& e = p.epi;
  const int lane = static_cast<int>(m & 31);
  const int64_t m0 = m - lane;
  constexpr int64_t ES = static_cast<int64_t>(sizeof(typename Storage<DT>::T));
  constexpr int GROUPS = TN / 2 / CKPT_GROUP;
  const bool swi = e.act == ACT_SWIGLU;
  char* obase = static_cast<char*>(e.out);
  char* ybase = static_cast<char*>(e.out2);
  const uint32_t buf2 = buf + 32u * 64u;
  int64_t nl = static_cast<int64_t>(nb) * TN + part * (TN / 2);
  uint32_t gs = held.gs, us = held.us;
#pragma unroll 1
  for (int c = 0; c < GROUPS; ++c, nl += CKPT_GROUP, gs >>= 8, us >>= 8) {
    const int units = units_before(p.N, nl, 8);
    code_put(held.g, buf, lane);
    if (swi) code_put(held.u, buf2, lane);
    __syncwarp();
    uint2 cg[4], cu[4];
    code_get(cg, buf, lane);
    if (swi) code_get(cu, buf2, lane);
    if (c + 1 < GROUPS) codes_ahead(p, m, nl + CKPT_GROUP, held);
    __syncwarp();  // every lane has its codes before the buffers take outputs
    float dy[32];
    tmem_ld32(trow + part * (TN / 2) + c * CKPT_GROUP, dy);
    if (c + 1 == GROUPS) release();
    const float gscale = ckpt_scale(gs & 255u), uscale = ckpt_scale(us & 255u);
    // (asked once for the warp's rows: hardly a group ends at the type's largest values)
    const bool near_end = __any_sync(0xffffffffu, ckpt_near_end<DT>(gs & 255u) || ckpt_near_end<DT>(us & 255u));
    uint4 yk[4];
    auto group = [&](auto act) {
      constexpr int ACT = decltype(act)::value;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float u[8], d[8], y[8];
        ckpt_decode4(cg[j].x, gscale, u);
        ckpt_decode4(cg[j].y, gscale, u + 4);
        if (near_end) {
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = ckpt_back_in_range<DT>(u[i]);
        }
        if constexpr (ACT == ACT_SWIGLU) {
          float up[8], d2[8];
          ckpt_decode4(cu[j].x, uscale, up);
          ckpt_decode4(cu[j].y, uscale, up + 4);
          if (near_end) {
#pragma unroll
            for (int i = 0; i < 8; ++i) up[i] = ckpt_back_in_range<DT>(up[i]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float s = sigmoid_short(u[i]), silu = u[i] * s;
            d[i] = dy[8 * j + i] * up[i] * (s + silu * (1.0f - s));
            d2[i] = dy[8 * j + i] * silu;
            y[i] = silu * up[i];
          }
          sts128(group_slot(buf2, lane, j), pack8<DT>(d2));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            d[i] = dy[8 * j + i] * held_act_grad<false>(ACT, u[i]);
            y[i] = held_act_fwd<false>(ACT, u[i]);
          }
          sts128(group_slot(buf2, lane, j), pack8<DT>(y));
        }
        sts128(group_slot(buf, lane, j), pack8<DT>(d));
        yk[j] = pack8<DT>(y);
      }
    };
    if (swi)
      group(std::integral_constant<int, ACT_SWIGLU>{});
    else
      by_activation(e.act, group);
    __syncwarp();
    group_flush(buf, lane, m0, p.M, units, [&](int64_t mm) { return obase + (mm * e.ldo + nl) * ES; });
    if (swi) {
      group_flush(buf2, lane, m0, p.M, units, [&](int64_t mm) { return obase + (mm * e.ldo + e.swiglu_F + nl) * ES; });
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) sts128(group_slot(buf2, lane, j), yk[j]);
      __syncwarp();
    }
    group_flush(buf2, lane, m0, p.M, units, [&](int64_t mm) { return ybase + (mm * e.ldo2 + nl) * ES; });
    __syncwarp();
  }
}

// The epilogue that a kernel is built with: EPI_STORE stands for all but the checkpoint
// kinds.  Those have twice the warps, each with one staging buffer and half of a tile's
// columns: the four of the others are one a scheduler, and at a short K (h = 1024) their
// dependent arithmetic, not the tensor cores, sets the pace (SwiGLU block of 2048 tokens, h
// 1024, f 4096: a step 299 µs with four, 239 with eight; 16 for the input gradient, with a
// stage less in the ring: 183 -> 189, GELU 158 -> 152).
template <int EP>
struct EpiWarps {
  static constexpr int N = EP == EPI_STORE ? 4 : 8;
  static constexpr int THREADS = 128 + 32 * N;
  static constexpr uint32_t BYTES = EPI_SMEM_BYTES / N;
};
// w: the warp among the epilogue's (its rows are the quarter w & 3 of the tile's)
// release: hands the accumulator back, once its last columns have been read.  (It waits
// for the warp's stores so far, so it comes before the last flushes, and not at all where
// no tile follows.)
template <int DT, int TN, int EP, bool HELD, typename Release>
__device__ __forceinline__ void run_epilogue(const Params& p, uint32_t trow, int64_t m, int nb, int part, int w,
                                             uint32_t staging, CodesAhead& held, Release release) {
  const uint32_t stage = staging + static_cast<uint32_t>(w) * EpiWarps<EP>::BYTES;
  if constexpr (EP == EPI_ACT_CKPT) {
    epilogue_act_ckpt<DT, TN>(p, trow, m, nb, w >> 2, stage, release);
  } else if constexpr (EP == EPI_DACT_CKPT) {
    epilogue_dact_ckpt<DT, TN>(p, trow, m, nb, w >> 2, stage, held, release);
  } else {
    epilogue_tile<DT, TN, HELD>(p, trow, m, nb, part, stage);
    release();
  }
}

// The dry run.  An epilogue's first pass in a launch waits for its instructions from L2:
// 8 to 16 thousand cycles more than the next pass takes.  In a block that keeps a checkpoint
// the epilogue's warps therefore run once on rows behind the matrix, where nothing is loaded
// or stored, while the predecessor ends and the first product runs.  They read the second
// accumulator, which the issuer takes after their release only.  (SwiGLU step of 2048 tokens,
// h 1024, f 4096: 208 -> 204 µs, GELU 165 -> 157.)
__device__ __forceinline__ int64_t no_row(const Params& p) { return (static_cast<int64_t>(p.M) + 31) / 32 * 32; }

// ---------------------------------------------------------------- kernel
template <int DT, bool A_MN, bool B_MN, int EP, bool HELD>
__global__ void __launch_bounds__(EpiWarps<EP>::THREADS, 1) gemm_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte alignment of the tile ring (128-byte swizzle atoms are 1 KB).
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* smem_a = smem;
  uint8_t* smem_b = smem + STAGES * A_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + STAGES);
  const uint32_t tfull0 = smem_u32(bars + 2 * STAGES);
  const uint32_t tempty0 = smem_u32(bars + 2 * STAGES + 2);
  const uint32_t drain_bar = smem_u32(bars + 2 * STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8u * a, 1);
      mbar_init(tempty0 + 8u * a, 32 * EpiWarps<EP>::N);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int num_tiles = p.mt * p.nt * p.nparts;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      for (int s = p.seg_begin[0]; s < p.seg_begin[p.nparts]; ++s) {
        tma_prefetch_map(&p.maps[p.segs[s].map_a]);
        tma_prefetch_map(&p.maps[p.segs[s].map_b]);
      }
      if constexpr (HELD) pdl_enter();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0, issued_phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        int part, mb, nb;
        decode_tile(t, p, part, mb, nb);
        for (int si = p.seg_begin[part]; ok && si < p.seg_begin[part + 1]; ++si) {
          const Seg sg = p.segs[si];
          const CUtensorMap* ma = &p.maps[sg.map_a];
          const CUtensorMap* mbp = &p.maps[sg.map_b];
          const int nkb = (sg.k_len + BK - 1) / BK;
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait_bounded(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.status, p.timeout_ns)) {
              ok = false;
              break;
            }
            const uint32_t fb = full0 + 8u * stage;
            mbar_arrive_expect_tx(fb, STAGE_BYTES);
            const uint32_t sa = smem_u32(smem_a + stage * A_BYTES);
            const uint32_t sb = smem_u32(smem_b + stage * B_BYTES);
            const int k0 = kb * BK;
            if constexpr (!A_MN) {
              if (p.a_chunk_rows > 0) {
                // rows past M (last tile) read the last chunk out of range: zero fill
                const int m_off = mb * BM;
                const int j = min(m_off / p.a_chunk_rows, p.a_nchunks - 1);
                tma_load_2d(sa, ma + j, fb, k0, m_off - j * p.a_chunk_rows);
              } else {
                tma_load_2d(sa, ma, fb, k0, mb * BM);
              }
            } else {
              tma_load_2d(sa, ma, fb, mb * BM, k0);
              tma_load_2d(sa + MN_BOX_BYTES, ma, fb, mb * BM + 64, k0);
            }
            if constexpr (!B_MN) {
              if (p.swiglu_up_row > 0) {
                tma_load_2d(sb, mbp, fb, k0, nb * (BN / 2));
                tma_load_2d(sb + B_BYTES / 2, mbp, fb, k0, p.swiglu_up_row + nb * (BN / 2));
              } else {
                tma_load_2d(sb, mbp, fb, k0, nb * BN);
              }
            } else {
#pragma unroll
              for (int j = 0; j < BN / 64; ++j) tma_load_2d(sb + j * MN_BOX_BYTES, mbp, fb, nb * BN + j * 64, k0);
            }
            issued_mask |= 1u << stage;
            issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      if (!ok) {
        // Let the copies already in flight land before the CTA exits.
        for (int s = 0; s < STAGES; ++s)
          if ((issued_mask >> s) & 1u)
            (void)mbar_wait_bounded(full0 + 8u * s, (issued_phase >> s) & 1u, nullptr, nullptr, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc_f16(DT == DT_BF16, A_MN, B_MN, BM, BN);
      if constexpr (HELD) pdl_enter();
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x, ++it) {
        int part, mb, nb;
        decode_tile(t, p, part, mb, nb);
        const int acc = it & 1;
        const uint32_t acc_phase = static_cast<uint32_t>(it >> 1) & 1u;
        // free at first; after a dry run the second accumulator once that has ended
        const uint32_t before = HELD && acc ? acc_phase : acc_phase ^ 1u;
        if (!mbar_wait_bounded(tempty0 + 8u * acc, before, abort_flag, p.status, p.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        uint32_t accumulate = 0;
        for (int si = p.seg_begin[part]; ok && si < p.seg_begin[part + 1]; ++si) {
          const int nkb = (p.segs[si].k_len + BK - 1) / BK;
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait_bounded(full0 + 8u * stage, phase, abort_flag, p.status, p.timeout_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem_a + stage * A_BYTES);
            const uint32_t sb = smem_u32(smem_b + stage * B_BYTES);
#pragma unroll
            for (int ks = 0; ks < BK / UMMA_K; ++ks) {
              // K-major: the next 16 K-elements are 32 bytes further along each
              // swizzled 128-byte row.  MN-major: 16 K-rows = two 1 KB atoms.
              const uint64_t ad = A_MN ? make_sdesc_sw128(sa + ks * 2048u, MN_BOX_BYTES, 1024u)
                                       : make_sdesc_sw128(sa + ks * 32u, 16u, 1024u);
              const uint64_t bd = B_MN ? make_sdesc_sw128(sb + ks * 2048u, MN_BOX_BYTES, 1024u)
                                       : make_sdesc_sw128(sb + ks * 32u, 16u, 1024u);
              tc_mma_f16(d_tmem, ad, bd, idesc, accumulate);
              accumulate = 1u;
            }
            tc_commit(empty0 + 8u * stage);  // frees the stage once these MMAs finish
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) break;
        tc_commit(tfull0 + 8u * acc);  // accumulator ready for the epilogue
      }
      if (!ok) {
        tc_commit(drain_bar);
        (void)mbar_wait_bounded(drain_bar, 0u, nullptr, nullptr, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lane quarter accessible to this warp
    const int first = blockIdx.x, step = gridDim.x;
    int it = HELD ? -1 : 0;  // -1: dry
    for (int t = HELD ? first - step : first; t < num_tiles; t += step, ++it) {
      const bool dry = HELD && it < 0;
      int part, mb, nb;
      decode_tile(dry ? first : t, p, part, mb, nb);
      const int acc = it & 1;
      const uint32_t acc_phase = static_cast<uint32_t>(it >> 1) & 1u;
      const int64_t m = (dry ? no_row(p) : static_cast<int64_t>(mb) * BM + q * 32) + lane;
      epi_prefetch_aux<BN, EP>(p, m, nb, DT == DT_F32 ? 4 : 2, warp - 4);
      CodesAhead held;
      if constexpr (EP == EPI_DACT_CKPT) codes_first<BN>(p, m, nb, (warp - 4) >> 2, held);
      if (!dry) {
        const bool ok = mbar_wait_bounded(tfull0 + 8u * acc, acc_phase, abort_flag, p.status, p.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      tc_fence_after();
      const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
      run_epilogue<DT, BN, EP, HELD>(p, trow, m, nb, part, warp - 4, smem_u32(smem + STAGES * STAGE_BYTES + 256), held, [&] {
        if (HELD && t + 2 * step >= num_tiles) return;  // nobody takes this accumulator again
        tc_fence_before();
        mbar_arrive(tempty0 + 8u * acc);
      });
      if (dry) pdl_enter();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- 2-SM kernel
// A CTA pair (cluster of 2) computes one 256×256 tile with tcgen05.mma
// .cta_group::2 (M = 256, N = 256, K = 16), issued by the even CTA.  Each CTA
// loads only its half of A (128 rows) and its half of B (128 rows of the
// 256-wide N tile) — half the L2→SM traffic per FLOP of the 1-SM kernel — into
// a 6-stage ring of 32 KB stages; both CTAs' TMA copies complete on the even
// CTA's "full" barrier, and the MMA commits are multicast to both CTAs' "empty"
// and "accumulator full" barriers.  Each CTA's tensor memory holds its 128 rows
// of both 256-column accumulators; both epilogues release an accumulator by
// arriving on the even CTA's "accumulator empty" barrier.
constexpr int PAIR_STAGES = 6;
constexpr int HALF_M = BM;      // rows of A per CTA
constexpr int PA_BYTES = HALF_M * BK * 2;  // 16 KB
constexpr int PB_BYTES = 128 * BK * 2;     // 16 KB: room for up to 128 B rows per CTA
constexpr int PSTAGE_BYTES = PA_BYTES + PB_BYTES;
constexpr int PAIR_NUM_BARS = 2 * PAIR_STAGES + 5;
constexpr size_t PAIR_SMEM_BYTES = 1024 + static_cast<size_t>(PAIR_STAGES) * PSTAGE_BYTES + 256 + EPI_SMEM_BYTES;

// TN: N extent of the pair's tile; each CTA holds TN/2 rows of B.
// Pair slot q (the q-th cluster of 2) computes the tiles t = q, q + S, q + 2S, …
// (S slots).  Every CTA loads its own 128 A rows and TN/2 B rows: no operand
// is shared between clusters, so every copy stays inside its own pair.
template <int DT, bool A_MN, bool B_MN, int TN, int EP, bool HELD>
__global__ void __launch_bounds__(EpiWarps<EP>::THREADS, 1) gemm_pair_kernel(const __grid_constant__ Params p) {
  constexpr int HALF_N = TN / 2;
  // bytes of one stage (both CTAs): A halves + B halves; an MN-major B half is
  // 64-column boxes, two even when TN/2 = 96
  constexpr uint32_t B_BOXES = HALF_N > 64 ? 2 : 1;
  constexpr uint32_t CTA_STAGE_TX = PA_BYTES + (B_MN ? B_BOXES * MN_BOX_BYTES : HALF_N * BK * 2);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* smem_a = smem;
  uint8_t* smem_b = smem + PAIR_STAGES * PA_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + PAIR_STAGES * PSTAGE_BYTES);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = smem_u32(bars + PAIR_STAGES);
  const uint32_t tfull0 = smem_u32(bars + 2 * PAIR_STAGES);
  const uint32_t tempty0 = smem_u32(bars + 2 * PAIR_STAGES + 2);
  const uint32_t drain_bar = smem_u32(bars + 2 * PAIR_STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + PAIR_NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // within the pair; 0 issues the pair's MMAs
  constexpr uint32_t lead = 0u;              // cluster rank of the pair's even CTA
  const bool leader = rank == 0;
  constexpr uint16_t pair_mask = 0x3u;       // both CTAs of the pair
  auto decode = [&](int t, int& part, int& mb, int& nb) { decode_tile(t, p, part, mb, nb); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < PAIR_STAGES; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);  // the pair's MMA commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8u * a, 1);
      mbar_init(tempty0 + 8u * a, 2 * EpiWarps<EP>::N);  // the epilogue warps of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int slot = static_cast<int>(cluster_id_x());
  const int nslots = static_cast<int>(gridDim.x >> 1);
  const int num_tiles = p.mt * p.nt * p.nparts;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      for (int s = p.seg_begin[0]; s < p.seg_begin[p.nparts]; ++s) {
        tma_prefetch_map(&p.maps[p.segs[s].map_a]);
        tma_prefetch_map(&p.maps[p.segs[s].map_b]);
      }
      if constexpr (HELD) pdl_enter();
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued_mask = 0, issued_phase = 0;
      bool ok = true;
      for (int t = slot; ok && t < num_tiles; t += nslots) {
        int part, mb, nb;
        decode(t, part, mb, nb);
        const int m_off = mb * (2 * HALF_M) + static_cast<int>(rank) * HALF_M;
        int n_row;  // first B row (K-major) / column (MN-major) this CTA loads
        if (p.swiglu_up_row > 0)
          n_row = (leader ? 0 : p.swiglu_up_row) + nb * HALF_N;  // gate half / up half
        else
          n_row = nb * TN + static_cast<int>(rank) * HALF_N;
        for (int si = p.seg_begin[part]; ok && si < p.seg_begin[part + 1]; ++si) {
          const Seg sg = p.segs[si];
          const CUtensorMap* ma = &p.maps[sg.map_a];
          const CUtensorMap* mbp = &p.maps[sg.map_b];
          const int nkb = (sg.k_len + BK - 1) / BK;
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait_bounded(empty0 + 8u * stage, phase ^ 1u, abort_flag, p.status, p.timeout_ns)) {
              ok = false;
              break;
            }
            const uint32_t fb_local = full0 + 8u * stage;
            const uint32_t fb = mapa_shared(fb_local, lead);  // the pair's even-CTA barrier
            if (leader) mbar_arrive_expect_tx(fb_local, 2 * CTA_STAGE_TX);
            const uint32_t sa = smem_u32(smem_a + stage * PA_BYTES);
            const uint32_t sb = smem_u32(smem_b + stage * PB_BYTES);
            const int k0 = kb * BK;
            if constexpr (!A_MN) {
              if (p.a_chunk_rows > 0) {
                // rows past M (last tile) read the last chunk out of range: zero fill
                const int j = min(m_off / p.a_chunk_rows, p.a_nchunks - 1);
                tma_load_2d_pair(sa, ma + j, fb, k0, m_off - j * p.a_chunk_rows);
              } else
                tma_load_2d_pair(sa, ma, fb, k0, m_off);
            } else {
              tma_load_2d_pair(sa, ma, fb, m_off, k0);
              tma_load_2d_pair(sa + MN_BOX_BYTES, ma, fb, m_off + 64, k0);
            }
            if constexpr (!B_MN) {
              tma_load_2d_pair(sb, mbp, fb, k0, n_row);
            } else {
              tma_load_2d_pair(sb, mbp, fb, n_row, k0);
              if constexpr (B_BOXES > 1) tma_load_2d_pair(sb + MN_BOX_BYTES, mbp, fb, n_row + 64, k0);
            }
            issued_mask |= 1u << stage;
            issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == PAIR_STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      if (!ok) {
        // Let copies in flight land before the CTA exits.  The even CTA can watch
        // its full barriers; the odd CTA's copies complete there too, so it waits
        // a fixed time instead.
        if (leader) {
          for (int s = 0; s < PAIR_STAGES; ++s)
            if ((issued_mask >> s) & 1u)
              (void)mbar_wait_bounded(full0 + 8u * s, (issued_phase >> s) & 1u, nullptr, nullptr, p.timeout_ns);
        } else {
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = make_idesc_f16(DT == DT_BF16, A_MN, B_MN, 2 * HALF_M, TN);
      if constexpr (HELD) pdl_enter();
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;
      bool ok = true;
      for (int t = slot; ok && t < num_tiles; t += nslots, ++it) {
        int part, mb, nb;
        decode(t, part, mb, nb);
        const int acc = it & 1;
        const uint32_t acc_phase = static_cast<uint32_t>(it >> 1) & 1u;
        // free at first; after a dry run the second accumulator once that has ended
        const uint32_t before = HELD && acc ? acc_phase : acc_phase ^ 1u;
        if (!mbar_wait_bounded(tempty0 + 8u * acc, before, abort_flag, p.status, p.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        uint32_t accumulate = 0;
        for (int si = p.seg_begin[part]; ok && si < p.seg_begin[part + 1]; ++si) {
          const int nkb = (p.segs[si].k_len + BK - 1) / BK;
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait_bounded(full0 + 8u * stage, phase, abort_flag, p.status, p.timeout_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem_a + stage * PA_BYTES);
            const uint32_t sb = smem_u32(smem_b + stage * PB_BYTES);
#pragma unroll
            for (int ks = 0; ks < BK / UMMA_K; ++ks) {
              const uint64_t ad = A_MN ? make_sdesc_sw128(sa + ks * 2048u, MN_BOX_BYTES, 1024u)
                                       : make_sdesc_sw128(sa + ks * 32u, 16u, 1024u);
              const uint64_t bd = B_MN ? make_sdesc_sw128(sb + ks * 2048u, MN_BOX_BYTES, 1024u)
                                       : make_sdesc_sw128(sb + ks * 32u, 16u, 1024u);
              tc_mma_f16_pair(d_tmem, ad, bd, idesc, accumulate);
              accumulate = 1u;
            }
            tc_commit_pair_mc(empty0 + 8u * stage, pair_mask);  // frees the stage in both CTAs
            if (++stage == PAIR_STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) break;
        tc_commit_pair_mc(tfull0 + 8u * acc, pair_mask);  // both CTAs' accumulator halves ready
      }
      if (!ok) {
        tc_commit_pair_mc(drain_bar, static_cast<uint16_t>(1u << lead));
        (void)mbar_wait_bounded(drain_bar, 0u, nullptr, nullptr, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;
    const uint32_t tempty_leader = mapa_shared(tempty0, lead);
    int it = HELD ? -1 : 0;  // -1: dry
    for (int t = HELD ? slot - nslots : slot; t < num_tiles; t += nslots, ++it) {
      const bool dry = HELD && it < 0;
      int part, mb, nb;
      decode(dry ? slot : t, part, mb, nb);
      const int acc = it & 1;
      const uint32_t acc_phase = static_cast<uint32_t>(it >> 1) & 1u;
      const int64_t row = static_cast<int64_t>(mb) * (2 * HALF_M) + static_cast<int64_t>(rank) * HALF_M + q * 32;
      const int64_t m = (dry ? no_row(p) : row) + lane;
      epi_prefetch_aux<TN, EP>(p, m, nb, DT == DT_F32 ? 4 : 2, warp - 4);
      CodesAhead held;
      if constexpr (EP == EPI_DACT_CKPT) codes_first<TN>(p, m, nb, (warp - 4) >> 2, held);
      if (!dry) {
        const bool ok = mbar_wait_bounded(tfull0 + 8u * acc, acc_phase, abort_flag, p.status, p.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      tc_fence_after();
      const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
      run_epilogue<DT, TN, EP, HELD>(p, trow, m, nb, part, warp - 4, smem_u32(smem + PAIR_STAGES * PSTAGE_BYTES + 256), held, [&] {
        if (HELD && t + 2 * nslots >= num_tiles) return;  // nobody takes this accumulator again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_leader + 8u * acc);
      });
      if (dry) pdl_enter();
    }
  }

  tc_fence_before();
  cluster_sync_all();  // the pair's MMAs and cross-CTA arrivals are all done
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

static EncodeFn get_encode() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  return fn;
}

// 2-D map over a row-major [outer, inner] matrix with row pitch ld (elements).
static int make_map(CUtensorMap* m, int dtype, const void* base, int64_t inner, int64_t outer,
                    int64_t ld, uint32_t box_inner, uint32_t box_outer) {
  EncodeFn enc = get_encode();
  if (!enc) return set_error(TPMLP_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t es[2] = {1, 1};
  const CUresult r = enc(m, dtype == DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                         2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(TPMLP_ERR_CUDA, "cuTensorMapEncodeTiled failed (code " + std::to_string(static_cast<int>(r)) + ")");
  return TPMLP_OK;
}

// mode 0: one CTA per tile; 1: CTA pairs (clusters of 2).
template <int DT, bool A_MN, bool B_MN, int TN, int EP, bool HELD>
static int launch_one(const Params& p, int64_t tiles, int mode, cudaStream_t st, const DeviceInfo& dev) {
  static std::mutex mu;
  static uint64_t attr_gen[64][2] = {};  // the device context the attributes were set in
  static int max_clusters[64][2] = {};
  auto* k1 = gemm_kernel<DT, A_MN, B_MN, EP, HELD>;
  auto* kp = gemm_pair_kernel<DT, A_MN, B_MN, TN, EP, HELD>;
  const unsigned csize = 2u;
  constexpr unsigned threads = EpiWarps<EP>::THREADS;
  int clusters = 0;
  {
    std::lock_guard<std::mutex> lk(mu);
    const int d = (dev.device >= 0 && dev.device < 64) ? dev.device : 0;
    if (attr_gen[d][mode] != dev.generation) {
      const cudaError_t e =
          mode ? cudaFuncSetAttribute(kp, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(PAIR_SMEM_BYTES))
               : cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES));
      if (e != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
      if (mode) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = csize;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(csize * static_cast<unsigned>(std::max(1, dev.num_sms / static_cast<int>(csize))));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = PAIR_SMEM_BYTES;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        const cudaError_t e2 = cudaOccupancyMaxActiveClusters(&n, kp, &cfg);
        if (e2 != cudaSuccess || n <= 0)
          return set_error(TPMLP_ERR_CUDA, std::string("cudaOccupancyMaxActiveClusters: ") + cudaGetErrorString(e2));
        max_clusters[d][mode] = n;
      }
      attr_gen[d][mode] = dev.generation;
    }
    clusters = max_clusters[d][mode];
  }
  // mode 0: a CTA an SM; 1: pair slots, at most the resident clusters of 2
  const int64_t slots = std::min<int64_t>(tiles, mode ? clusters : dev.num_sms);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3((mode ? csize : 1u) * static_cast<unsigned>(slots));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = mode ? PAIR_SMEM_BYTES : SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  if (mode) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = csize;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (HELD) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  const cudaError_t le = mode ? cudaLaunchKernelEx(&cfg, kp, p) : cudaLaunchKernelEx(&cfg, k1, p);
  if (le != cudaSuccess)
    return set_error(TPMLP_ERR_CUDA,
                     std::string(mode ? "2-SM GEMM launch: " : "tensor-core GEMM launch: ") + cudaGetErrorString(le));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string("tensor-core GEMM launch: ") + cudaGetErrorString(e));
  return TPMLP_OK;
}

template <int DT, int TN, bool HELD>
static int dispatch_layout(const Params& p, int64_t tiles, int mode, cudaStream_t st, const DeviceInfo& dev, bool a_mn,
                           bool b_mn) {
  if (!a_mn && !b_mn) return launch_one<DT, false, false, TN, EPI_STORE, HELD>(p, tiles, mode, st, dev);
  if (!a_mn && b_mn) return launch_one<DT, false, true, TN, EPI_STORE, HELD>(p, tiles, mode, st, dev);
  if (a_mn && b_mn) return launch_one<DT, true, true, TN, EPI_STORE, HELD>(p, tiles, mode, st, dev);
  return set_error(TPMLP_ERR_UNSUPPORTED, "MN-major A with K-major B is not instantiated");
}

template <int DT>
static int dispatch(const Params& p, int64_t tiles, int mode, int tn, bool held, cudaStream_t st, const DeviceInfo& dev,
                    bool a_mn, bool b_mn) {
  if (p.epi.kind == EPI_ACT_CKPT) return launch_one<DT, false, false, BN, EPI_ACT_CKPT, true>(p, tiles, mode, st, dev);
  if (p.epi.kind == EPI_DACT_CKPT) return launch_one<DT, false, true, BN, EPI_DACT_CKPT, true>(p, tiles, mode, st, dev);
  if (!held) return dispatch_layout<DT, BN, false>(p, tiles, mode, st, dev, a_mn, b_mn);
  if (tn == NARROW_TN) return dispatch_layout<DT, NARROW_TN, true>(p, tiles, mode, st, dev, a_mn, b_mn);
  return dispatch_layout<DT, BN, true>(p, tiles, mode, st, dev, a_mn, b_mn);
}

}  // namespace tc

int launch_gemm_tc(const GemmDesc& g, cudaStream_t st) {
  using namespace tc;
  DeviceInfo* dev = nullptr;
  int rc = current_device(&dev);
  if (rc != TPMLP_OK) return rc;
  if (g.M <= 0 || g.N <= 0) return TPMLP_OK;
  if (g.M >= (1ll << 31) || g.N >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "GEMM extent >= 2^31");
  const bool swiglu = g.swiglu_up_row > 0;
  if (swiglu && (g.a_mn || g.b_mn)) return set_error(TPMLP_ERR_UNSUPPORTED, "SwiGLU pairing needs K-major operands");
  const bool chunked = g.a_chunk_rows > 0;
  if (chunked && (g.a_mn || g.a_chunk_rows % BM != 0 || g.a_chunks.empty() ||
                  static_cast<int64_t>(g.a_chunks.size()) * g.a_chunk_rows != g.M))
    return set_error(TPMLP_ERR_UNSUPPORTED, "chunked A needs K-major chunks of a multiple of 128 rows covering M");

  // CTA pairs (256-row tiles) whenever there is more than one 128-row block.
  const bool pair = g.M > BM;
  // N tile of the pair kernel.  (A 192-wide variant that trims the last wave of
  // N = h GEMMs measured slower per tile than it saved, so one width is used.)
  // A block with a checkpoint gets half the width where that fills pairs which would
  // otherwise stand idle: the order of each element's sum stays the same.  (The two N = h
  // GEMMs of the SwiGLU block of 2048 tokens, h 1024, f 4096: 32 tiles on 76 pairs, a step
  // 230 µs; 64 tiles, 227: the halves read more operands from L2.)
  const int64_t wide_tiles = (g.M + 2 * BM - 1) / (2 * BM) * ((g.N + BN - 1) / BN) * g.nparts;
  const bool halves = g.held && !g.beside && g.epi.kind != EPI_ACT_CKPT && g.epi.kind != EPI_DACT_CKPT;
  const int tn = pair && halves && !swiglu && wide_tiles * 4 <= dev->num_sms ? NARROW_TN : BN;
  Params p;
  memset(&p, 0, sizeof(p));
  p.M = static_cast<int32_t>(g.M);
  p.N = static_cast<int32_t>(g.N);
  p.mt = static_cast<int32_t>((g.M + (pair ? 2 * BM : BM) - 1) / (pair ? 2 * BM : BM));
  const int tile_n = swiglu ? tn / 2 : tn;
  p.nt = static_cast<int32_t>((g.N + tile_n - 1) / tile_n);
  const int mode = pair ? 1 : 0;
  const uint32_t a_box_rows = static_cast<uint32_t>(BM);  // K-major A: one 128-row box per CTA
  const uint32_t b_box_rows = static_cast<uint32_t>(pair ? tn / 2 : (swiglu ? BN / 2 : BN));
  p.swiglu_up_row = static_cast<int32_t>(g.swiglu_up_row);
  p.a_chunk_rows = chunked ? static_cast<int32_t>(g.a_chunk_rows) : 0;
  p.a_nchunks = chunked ? static_cast<int32_t>(g.a_chunks.size()) : 0;
  p.status = dev->status;
  p.timeout_ns = wait_timeout_ns();
  p.epi = g.epi;

  // Launch batches: consecutive partials whose segments fit the parameter block.
  int seg_i = 0;
  const int nseg = static_cast<int>(g.segs.size());
  int part = 0;
  while (part < g.nparts) {
    int nparts = 0, nsegs = 0, nmaps = 0;
    p.part_base = part;
    p.seg_begin[0] = 0;
    while (part < g.nparts && nparts < MAX_PARTS) {
      int cnt = 0;
      while (seg_i + nsegs + cnt < nseg && g.segs[seg_i + nsegs + cnt].part == part) ++cnt;
      if (cnt == 0) return set_error(TPMLP_ERR_INVALID_ARG, "a GEMM partial has no K segment");
      if (nsegs + cnt > MAX_SEGS) {
        if (nparts == 0) return set_error(TPMLP_ERR_UNSUPPORTED, "too many K segments in one partial");
        break;
      }
      const int chunks = chunked ? static_cast<int>(g.a_chunks.size()) : 1;
      if (nmaps + cnt * (chunks + 1) > MAX_MAPS) {
        if (nparts == 0) return set_error(TPMLP_ERR_UNSUPPORTED, "too many tensor maps in one partial");
        break;
      }
      for (int c = 0; c < cnt; ++c) {
        const GemmSeg& s = g.segs[seg_i + nsegs + c];
        if (s.k <= 0 || s.k >= (1ll << 31)) return set_error(TPMLP_ERR_INVALID_ARG, "bad K segment");
        const int idx = nsegs + c;
        Seg& d = p.segs[idx];
        d.k_len = static_cast<int32_t>(s.k);
        d.map_a = nmaps;
        if (chunked) {
          for (int j = 0; j < chunks; ++j) {
            rc = make_map(&p.maps[nmaps++], g.dtype, g.a_chunks[j], s.k, g.a_chunk_rows, g.lda, BK, a_box_rows);
            if (rc != TPMLP_OK) return rc;
          }
        } else if (!g.a_mn) {
          rc = make_map(&p.maps[nmaps++], g.dtype, s.a, s.k, g.M, g.lda, BK, a_box_rows);
        } else {
          rc = make_map(&p.maps[nmaps++], g.dtype, s.a, g.M, s.k, g.lda, 64, BK);
        }
        if (rc != TPMLP_OK) return rc;
        d.map_b = nmaps;
        if (!g.b_mn)
          rc = make_map(&p.maps[nmaps++], g.dtype, s.b, s.k, g.b_rows, g.ldb, BK, b_box_rows);
        else
          rc = make_map(&p.maps[nmaps++], g.dtype, s.b, g.N, s.k, g.ldb, 64, BK);
        if (rc != TPMLP_OK) return rc;
      }
      nsegs += cnt;
      ++nparts;
      p.seg_begin[nparts] = nsegs;
      ++part;
    }
    p.nparts = nparts;
    const int64_t tiles = static_cast<int64_t>(p.mt) * p.nt * nparts;
    if (tiles >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "too many tiles");
    double ksum = 0.0;
    for (int c = 0; c < nsegs; ++c) ksum += static_cast<double>(p.segs[c].k_len);
    const double work = 2.0 * static_cast<double>(g.M) * static_cast<double>(swiglu ? 2 * g.N : g.N) * ksum;
    const int ph = prof_begin(PROF_GEMM_TC, st);
    if (g.dtype == DT_BF16)
      rc = dispatch<DT_BF16>(p, tiles, mode, tn, g.held, st, *dev, g.a_mn, g.b_mn);
    else
      rc = dispatch<DT_F16>(p, tiles, mode, tn, g.held, st, *dev, g.a_mn, g.b_mn);
    prof_end(ph, work, st);
    if (rc != TPMLP_OK) return rc;
    seg_i += nsegs;
  }
  return TPMLP_OK;
}

}  // namespace tpmlp
