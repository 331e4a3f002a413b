// Attention of one new token per sequence over a paged key/value cache: the
// serving form of the attention core (attn.cu), for the same heads and groups.
//
//   o = Σ_u softmax_u(q·k_u·scale)·v_u over the sequence's first `length` keys,
//   lse = log2 Σ_u 2^(q·k_u·scale·log2 e)
//
// Bound by HBM: a key and a value of a group are read once for its r query
// heads, 4·r·d FLOPs for 4·d bytes; 5.7 … 6.1 TB/s measured (one sequence of
// 131001 keys, 64/8 heads of 128: 94 µs; 64 sequences of 17 … 8192: 192–204 µs).  What
// follows from that:
//
// * A CTA takes one group (key/value head) and its four warps split the keys; with
//   rows that whole 128-byte lines do not divide (d = 96) it takes two neighbouring
//   heads side by side, which share lines (16 sequences of 1200 … 2900 keys, 64
//   heads of 96: 137 µs; with rounded probabilities 140, and 158 one at a time).
// * The work, counted in steps of a CTA (16 keys a warp) over all (sequence, group)
//   units, is cut into equal shares, one a CTA, whatever the sequences' lengths: a
//   share may hold the end of one unit, whole units and the beginning of another.
//   A unit counts LEAD steps more for its fixed cost (256 sequences of 17 … 700
//   keys: 113 µs without, 78 µs with).  Parts of units leave (maximum, sum,
//   unnormalised o) in the workspace and decode_join_kernel joins them in order;
//   whole units are written at once.  No atomics: the same bits on every call.
// * The copies run ahead from one unit into the next, so the pipeline drains only
//   at the share's end.
// * Each warp streams its own 16 keys of a step through a private ring of
//   cp.async stages, so no warp waits for another before the unit's end.  Rows
//   behind the length (and on pages that do not exist) are filled with zeros by
//   the copy itself, and their scores are masked: what the cache holds there,
//   NaN included, is never used.
// * Scores are computed transposed, Sᵀ = K·Qᵀ and Oᵀ += Vᵀ·Pᵀ with
//   mma.m16n8k16: 16 keys (or head columns) are the rows and 8 query heads the
//   columns, so a group of up to 8 heads wastes no rows on padding, and the
//   probabilities become the second product's operand by one 8×8 transposition
//   in registers.  (One token has too few rows for the 128-row tcgen05 tiles; at
//   8 FLOPs a byte the tensor pipe is far from a limit.)
// * Softmax statistics, o and the partials are float32.  The probabilities enter
//   the second product in two parts of the storage type (Prob), so o is as exact as
//   with float32 probabilities: 0.00166 of its size off the 64-bit result in bf16,
//   which is the rounding of o itself (0.00215 with rounded probabilities; fp16
//   0.00021 and 0.00027).  The second part's products cost 93.6 against 93.2 µs for
//   the long sequence and 78.2 against 76.9 for many short ones (heads of 96 two at a
//   time: 137.1 against 139.7).
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "internal.h"

namespace tpmlp {
namespace decode {

constexpr int WARPS = 4;
constexpr int SUB = 16;            // keys of a warp's step
constexpr int STAGES = 3;
constexpr int CTAS = 2;            // per SM
constexpr int MAX_SEQS = 1024;     // sequences of one launch (prefix sums in shared memory)
constexpr unsigned LEAD = 3;       // a unit's fixed cost (its queries, the join of the warps), in steps
constexpr int JOIN_ROW = 36;       // floats of a row of o in the join of the warps
constexpr int MAX_CTAS = 512;
constexpr int JOIN_SLICES = 8;
constexpr int JOIN_THREADS = JOIN_SLICES * 32;

struct Params {
  const void* q;
  int64_t ldq;
  const void* k;
  const void* v;
  int64_t page_stride, token_stride, head_stride;
  int64_t pages;
  unsigned page_size, width;  // width: entries of a block-table row
  unsigned page_magic, page_shift;  // key / page_size = key·magic >> shift for keys below 2³¹
  int one_page;  // 16 keys from a multiple of 16 lie on one page, and their offsets fit 32 bits
  const int32_t* table;
  int64_t ldt;
  const int32_t* lengths;
  void* o;
  int64_t ldo;
  float* lse;  // or NULL
  int n, heads, kv_heads, r;
  int blocks;  // blocks of query heads per group (1 unless r > 16)
  int set;     // units (group and block of query heads) that a CTA takes side by side: 1 or 2
  float scale_log2;
  int4* info;      // [CTAs] (sequence, set of units, last CTA, —), sequence −1: nothing to join
  float2* part_ml; // [CTAs][2][units of a set][heads of a block] (maximum, sum)
  float* part_o;   // the same, [d] each
  unsigned* status;
};

// `real` false: zeros, nothing is read.  LINES: L2 fetches whole 128-byte lines,
// else half lines.
template <bool LINES>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;
  if constexpr (LINES)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <int DT>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (DT == DT_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  using S = Storage<DT>;
  typename S::T t[2] = {S::from(lo), S::from(hi)};
  uint32_t r;
  memcpy(&r, t, 4);
  return r;
}
// Probabilities in two parts of the storage type: one a step below the value, and
// what that leaves.  Both are above zero, so that an infinity among the values meets
// no zero and no sign but the probability's (two parts around the nearest value would
// make NaN of it); together they are off by 3·(eps/2)² (a remainder of up to 3 half
// steps, rounded).  fp16 takes probabilities times 2^15: its subnormals, where this
// ends, begin at 2^-29 of the largest.
template <int DT>
struct Prob {
  static constexpr float BELOW = DT == DT_BF16 ? 1.0f - 1.0f / 128.0f : 1.0f - 1.0f / 1024.0f;
  static constexpr float LOG2_SCALE = DT == DT_BF16 ? 0.0f : 15.0f;
  static constexpr float UNSCALE = DT == DT_BF16 ? 1.0f : 1.0f / 32768.0f;
  static __device__ __forceinline__ uint32_t main(float lo, float hi) { return pack2<DT>(lo * BELOW, hi * BELOW); }
  static __device__ __forceinline__ uint32_t rest(float lo, float hi, uint32_t part) {
    if constexpr (DT == DT_BF16) {
      return pack2<DT>(lo - __uint_as_float(part << 16), hi - __uint_as_float(part & 0xffff0000u));
    } else {
      __half2 h;
      memcpy(&h, &part, 4);
      const float2 f = __half22float2(h);
      return pack2<DT>(lo - f.x, hi - f.y);
    }
  }
  // The base-2 log-sum-exp of scores with maximum m and probabilities' sum l.
  static __device__ __forceinline__ float lse(float m, float l) { return l == 0.0f ? -INFINITY : m + log2f(l * UNSCALE); }
};
__device__ __forceinline__ float exp2_hw(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Max, sum and weights where nothing was visible: −∞ minus −∞ must not appear.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

// The keys of sequence i, no more than its block-table row holds.
__device__ __forceinline__ unsigned length_of(const Params& p, int i) {
  const int len = p.lengths[i];
  if (len <= 0) return 0;
  const uint64_t room = static_cast<uint64_t>(p.width) * p.page_size;
  if (static_cast<uint64_t>(len) > room) {
    atomicCAS(p.status, 0u, STATUS_BAD_INDEX);
    return static_cast<unsigned>(room);
  }
  return static_cast<unsigned>(len);
}

// Per head width: bytes of a staged row (an odd number of 16-byte units, so
// ldmatrix meets no bank conflict), of a stage, and of the rings.
template <int HDIM>
struct Dim {
  static constexpr int ROW = HDIM * 2 + 16;
  static constexpr int STAGE = 2 * SUB * ROW;
  static constexpr size_t SMEM = static_cast<size_t>(WARPS) * STAGES * STAGE;
};

// A CTA's part of a set of units: steps [t0, t1) of the nb steps of a sequence.
struct Part {
  int seq, set;
  unsigned nb, t0, t1, len;
};

template <int DT, int HDIM, int NT, int SET>
__global__ void __launch_bounds__(WARPS * 32, CTAS) paged_decode_kernel(const __grid_constant__ Params p) {
  using T = typename Storage<DT>::T;
  constexpr int HB = 8 * NT;  // query heads of a block
  constexpr int KS = HDIM / 16;
  constexpr int WAYS = WARPS / SET;        // warps that share a unit's keys
  constexpr unsigned TILE = WAYS * SUB;    // keys of a step
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ unsigned prefix[MAX_SEQS + 1];  // steps (and leads) before each sequence, per set of units
  __shared__ unsigned wsum[WARPS];
  __shared__ float sm_m[WARPS][HB], sm_l[WARPS][HB];
  __shared__ unsigned sm_mask[WARPS][STAGES];
  __shared__ __align__(16) float so[WARPS][8][JOIN_ROW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mine = warp / WAYS, turn = warp % WAYS;  // this warp's unit of the set, and its place among its warps
  pdl_go();
  pdl_wait();

  // Steps of every sequence, with LEAD for the fixed cost, and their sums.
  unsigned run = 0;
  for (int i0 = 0; i0 < p.n; i0 += WARPS * 32) {
    const int i = i0 + tid;
    const unsigned steps = i < p.n ? (length_of(p, i) + TILE - 1) / TILE : 0u;
    const unsigned c = steps > 0 ? steps + LEAD : 0u;
    unsigned inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    unsigned before = run;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += wsum[w];
      run += wsum[w];
    }
    if (i < p.n) prefix[i] = before + inc - c;
  }
  if (tid == 0) prefix[p.n] = run;
  __syncthreads();
  const int64_t ups = static_cast<int64_t>(p.kv_heads) * p.blocks / SET;  // sets of a sequence
  const int64_t total = static_cast<int64_t>(run) * ups;
  const int64_t c = blockIdx.x;
  const int64_t G = min(static_cast<int64_t>(gridDim.x), max(total, static_cast<int64_t>(1)));  // no empty share between others
  const int64_t x0 = c < G ? total * c / G : total, x1 = c < G ? total * (c + 1) / G : total;
  if (tid == 0) p.info[c] = make_int4(-1, 0, 0, 0);

  // Sequences without a key.
  for (int i = static_cast<int>(c); i < p.n; i += static_cast<int>(gridDim.x)) {
    if (prefix[i + 1] != prefix[i]) continue;
    T* o = static_cast<T*>(p.o) + i * p.ldo;
    for (int e = tid; e < p.heads * HDIM; e += WARPS * 32) o[e] = Storage<DT>::from(0.0f);
    if (p.lse != nullptr)
      for (int e = tid; e < p.heads; e += WARPS * 32) p.lse[static_cast<int64_t>(i) * p.heads + e] = -INFINITY;
  }
  if (x0 >= x1) return;

  const uint32_t ring = smem_u32(smem) + warp * STAGES * Dim<HDIM>::STAGE;
  const int g8 = lane >> 2, t4 = lane & 3;
  // Where the lane's i-th 16-byte copy of a step goes to and, with all its keys on
  // one page, comes from.
  constexpr int COPIES = SUB * (HDIM / 8) / 32;
  uint32_t lane_dst[COPIES];
  int lane_src[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    const int id = i * 32 + lane, row = id / (HDIM / 8), col = id - row * (HDIM / 8);
    lane_dst[i] = row * Dim<HDIM>::ROW + col * 16;
    lane_src[i] = row * static_cast<int>(p.token_stride) + col * 8;
  }

  // The first part with steps at or behind x, in a sequence at or behind `from`; x
  // is moved to its end.  False at the share's end.
  auto next_part = [&](int64_t& x, int from, Part* part) {
    Part s;
    s.seq = from;
    while (x < x1) {
      while (prefix[s.seq + 1] == prefix[s.seq] || x >= static_cast<int64_t>(prefix[s.seq + 1]) * ups) ++s.seq;
      const unsigned n = prefix[s.seq + 1] - prefix[s.seq];  // LEAD, then the steps
      const int64_t in_seq = x - static_cast<int64_t>(prefix[s.seq]) * ups;
      s.set = static_cast<int>(in_seq >> 32 ? in_seq / n : static_cast<unsigned>(in_seq) / n);
      const unsigned v0 = static_cast<unsigned>(in_seq - static_cast<int64_t>(s.set) * n);
      const unsigned v1 = static_cast<unsigned>(min(static_cast<int64_t>(n), v0 + (x1 - x)));
      x += v1 - v0;
      if (v1 <= LEAD) continue;
      s.nb = n - LEAD;
      s.t0 = v0 > LEAD ? v0 - LEAD : 0;
      s.t1 = v1 - LEAD;
      s.len = length_of(p, s.seq);
      *part = s;
      return true;
    }
    return false;
  };
  auto page_index = [&](unsigned key) {
    return static_cast<unsigned>((static_cast<uint64_t>(key) * p.page_magic) >> p.page_shift);
  };

  // The copies run STAGES − 1 steps ahead of the arithmetic, from one part into the
  // next.  A step of this warp: keys [step·TILE + turn·SUB, + SUB); the page of key
  // `lane` of a step is looked up one step ahead of its copies.
  int lo = 0;
  for (int hi = p.n - 1; lo < hi;) {  // the last sequence with prefix·ups <= x0
    const int mid = (lo + hi + 1) / 2;
    if (static_cast<int64_t>(prefix[mid]) * ups <= x0) lo = mid;
    else hi = mid - 1;
  }
  Part s;
  int64_t x = x0;  // the end of part s; fx: of part f
  if (!next_part(x, lo, &s)) return;
  Part f = s;
  int64_t fx = x;
  bool more = true;  // steps to copy
  unsigned fstep = f.t0;
  int64_t fgroup = ((f.set * SET + mine) / p.blocks) * p.head_stride;
  int fill = 0, use = 0;
  auto look_up = [&]() -> int {
    const unsigned key = fstep * TILE + turn * SUB + (lane & 15);
    return more && key < f.len ? p.table[f.seq * p.ldt + page_index(key)] : -1;
  };
  int page = look_up();
  auto fetch = [&]() {
    if (more) {
      const unsigned key0 = fstep * TILE + turn * SUB, key = key0 + (lane & 15);
      const bool seen = key < f.len, good = seen && page >= 0 && page < p.pages;
      if (seen && !good) atomicCAS(p.status, 0u, STATUS_BAD_INDEX);
      const unsigned mask = __ballot_sync(0xffffffffu, good) & 0xffffu;
      if (lane == 0) sm_mask[warp][fill] = mask;
      const uint32_t dst = ring + fill * Dim<HDIM>::STAGE;
      const T* kb = static_cast<const T*>(p.k) + fgroup;
      const T* vb = static_cast<const T*>(p.v) + fgroup;
      const int64_t at = good ? page * p.page_stride + (key - page_index(key) * p.page_size) * p.token_stride : 0;
      if (mask == 0xffffu && p.one_page) {
        // 16 keys of one page: the lane's rows are a fixed distance apart
        const int64_t at0 = at - (lane & 15) * p.token_stride;
        kb += at0;
        vb += at0;
        // with one unit a CTA, the rest of a line is another head's, read at another time
        constexpr bool LINES = HDIM % 64 == 0 || SET > 1;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          cp_async16<LINES>(dst + lane_dst[i], kb + lane_src[i], true);
          cp_async16<LINES>(dst + SUB * Dim<HDIM>::ROW + lane_dst[i], vb + lane_src[i], true);
        }
      } else if (mask != 0) {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int id = i * 32 + lane, row = id / (HDIM / 8), col = id - row * (HDIM / 8);
          const int64_t src = __shfl_sync(0xffffffffu, at, row) + col * 8;
          const bool real = (mask >> row) & 1u;
          cp_async16<HDIM % 64 == 0>(dst + lane_dst[i], kb + src, real);
          cp_async16<HDIM % 64 == 0>(dst + SUB * Dim<HDIM>::ROW + lane_dst[i], vb + src, real);
        }
      }
      fill = fill + 1 < STAGES ? fill + 1 : 0;
      if (++fstep == f.t1) {
        more = next_part(fx, f.seq, &f);
        if (more) {
          fstep = f.t0;
          fgroup = ((f.set * SET + mine) / p.blocks) * p.head_stride;
        }
      }
      page = look_up();
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch();

  // Qᵀ of a part as the first product's B operand: pairs along d, query heads as
  // columns.  A part's are loaded before the last one's parts are joined.
  uint32_t qf[NT][KS][2];
  auto load_q = [&](const Part& part) {
    const int unit = part.set * SET + mine, group = unit / p.blocks, block = unit - group * p.blocks;
    const int head0 = group * p.r + block * HB, nheads = min(HB, p.r - block * HB);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int hq = nt * 8 + g8;
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) + part.seq * p.ldq +
                                                             static_cast<int64_t>(head0 + hq) * HDIM);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[nt][ks][0] = hq < nheads ? qp[ks * 8 + t4] : 0u;
        qf[nt][ks][1] = hq < nheads ? qp[ks * 8 + 4 + t4] : 0u;
      }
    }
  };
  load_q(s);
  while (true) {
    float acc[NT][KS][4];
    float mx[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mx[nt][0] = mx[nt][1] = -INFINITY;
      sum[nt][0] = sum[nt][1] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[nt][mt][j] = 0.0f;
    }

    for (unsigned step = s.t0; step < s.t1; ++step) {
      fetch();
      cp_wait<STAGES - 1>();
      __syncwarp();
      const unsigned mask = sm_mask[warp][use];
      if (mask != 0) {
        const uint32_t sk = ring + use * Dim<HDIM>::STAGE, sv = sk + SUB * Dim<HDIM>::ROW;
        float e2[NT][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) e2[nt][0][j] = e2[nt][1][j] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t a[4];
          ldsm4(sk + (lane & 15) * Dim<HDIM>::ROW + ks * 32 + (lane >> 4) * 16, a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<DT>(e2[nt][ks & 1], a, qf[nt][ks][0], qf[nt][ks][1]);
        }
        const bool low = (mask >> g8) & 1u, high = (mask >> (g8 + 8)) & 1u;
        uint32_t pf[NT][2], pr[NT][2];  // the probabilities' two parts
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = (e2[nt][0][j] + e2[nt][1][j]) * p.scale_log2;
          if (!low) e[0] = e[1] = -INFINITY;
          if (!high) e[2] = e[3] = -INFINITY;
          float top[2] = {fmaxf(e[0], e[2]), fmaxf(e[1], e[3])};
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
            top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
          }
          const float m0 = fmaxf(mx[nt][0], top[0]), m1 = fmaxf(mx[nt][1], top[1]);
          if (__any_sync(0xffffffffu, m0 != mx[nt][0] || m1 != mx[nt][1])) {
            const float f0 = exp2_hw(mx[nt][0] - finite_max(m0)), f1 = exp2_hw(mx[nt][1] - finite_max(m1));
            sum[nt][0] *= f0;
            sum[nt][1] *= f1;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              acc[nt][mt][0] *= f0;
              acc[nt][mt][1] *= f1;
              acc[nt][mt][2] *= f0;
              acc[nt][mt][3] *= f1;
            }
            mx[nt][0] = m0;
            mx[nt][1] = m1;
          }
          const float b0 = finite_max(m0) - Prob<DT>::LOG2_SCALE, b1 = finite_max(m1) - Prob<DT>::LOG2_SCALE;
          e[0] = exp2_hw(e[0] - b0);
          e[1] = exp2_hw(e[1] - b1);
          e[2] = exp2_hw(e[2] - b0);
          e[3] = exp2_hw(e[3] - b1);
          sum[nt][0] += e[0] + e[2];
          sum[nt][1] += e[1] + e[3];
          const uint32_t p0 = Prob<DT>::main(e[0], e[1]), p1 = Prob<DT>::main(e[2], e[3]);
          pf[nt][0] = transpose8x8(p0);
          pf[nt][1] = transpose8x8(p1);
          pr[nt][0] = transpose8x8(Prob<DT>::rest(e[0], e[1], p0));
          pr[nt][1] = transpose8x8(Prob<DT>::rest(e[2], e[3], p1));
        }
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          uint32_t a[4];
          ldsm4_trans(sv + ((lane & 7) + ((lane >> 4) & 1) * 8) * Dim<HDIM>::ROW + mt * 32 + ((lane >> 3) & 1) * 16, a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<DT>(acc[nt][mt], a, pf[nt][0], pf[nt][1]);
            mma16816<DT>(acc[nt][mt], a, pr[nt][0], pr[nt][1]);
          }
        }
      }
      use = use + 1 < STAGES ? use + 1 : 0;
      __syncwarp();  // the stage is read before its next copies are issued
    }

    Part ahead;
    const int64_t end_x = x;
    const bool again = next_part(x, s.seq, &ahead);
    if (again) load_q(ahead);

    // The warps' parts of their units, joined in warp order, 32 columns of eight
    // query heads at a time.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        sum[nt][0] += __shfl_xor_sync(0xffffffffu, sum[nt][0], o);
        sum[nt][1] += __shfl_xor_sync(0xffffffffu, sum[nt][1], o);
      }
      if (g8 == 0) {
        const int h0 = nt * 8 + 2 * t4;
        sm_m[warp][h0] = mx[nt][0];
        sm_m[warp][h0 + 1] = mx[nt][1];
        sm_l[warp][h0] = sum[nt][0];
        sm_l[warp][h0 + 1] = sum[nt][1];
      }
    }
    const bool begins = s.t0 == 0, ends = s.t1 == s.nb, whole = begins && ends;
    const int64_t slot = c * 2 + (begins ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int quarter = 0; quarter < HDIM / 32; ++quarter) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* a = acc[nt][quarter * 2 + h];
          float* w = &so[warp][2 * t4][h * 16 + g8];
          w[0] = a[0];
          w[JOIN_ROW] = a[1];
          w[8] = a[2];
          w[JOIN_ROW + 8] = a[3];
        }
        __syncthreads();
        for (int e = tid; e < SET * 64; e += WARPS * 32) {  // a unit's 8 heads × 8 float4
          const int us = e / 64, hq = (e >> 3) & 7, col = (e & 7) * 4, h = nt * 8 + hq;
          const int un = s.set * SET + us, gr = un / p.blocks, bl = un - gr * p.blocks;
          if (h >= p.r - bl * HB) continue;
          const int head = gr * p.r + bl * HB + h, dcol = quarter * 32 + col;
          float m = -INFINITY;
#pragma unroll
          for (int w = 0; w < WAYS; ++w) m = fmaxf(m, sm_m[us * WAYS + w][h]);
          const float base = finite_max(m);
          float l = 0.0f;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < WAYS; ++w) {
            const float f0 = exp2_hw(sm_m[us * WAYS + w][h] - base);
            l = fmaf(f0, sm_l[us * WAYS + w][h], l);
            const float4 a = *reinterpret_cast<const float4*>(&so[us * WAYS + w][hq][col]);
            v.x = fmaf(f0, a.x, v.x), v.y = fmaf(f0, a.y, v.y), v.z = fmaf(f0, a.z, v.z), v.w = fmaf(f0, a.w, v.w);
          }
          if (whole) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint2 u;
            u.x = pack2<DT>(v.x * inv, v.y * inv);
            u.y = pack2<DT>(v.z * inv, v.w * inv);
            *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + s.seq * p.ldo + static_cast<int64_t>(head) * HDIM + dcol) = u;
            if (p.lse != nullptr && dcol == 0)
              p.lse[static_cast<int64_t>(s.seq) * p.heads + head] = Prob<DT>::lse(m, l);
          } else {
            const int64_t at = (slot * SET + us) * HB + h;
            __stcg(reinterpret_cast<float4*>(p.part_o + at * HDIM + dcol), v);
            if (dcol == 0) __stcg(p.part_ml + at, make_float2(m, l));
          }
        }
        __syncthreads();
      }
    }
    if (begins && !ends && tid == 0) {
      // the CTA whose share holds the set's last step
      const int64_t last_x = end_x + (s.nb - s.t1) - 1;
      p.info[c] = make_int4(s.seq, s.set, static_cast<int>(((last_x + 1) * G - 1) / total), 0);
    }
    if (!again) break;
    s = ahead;
  }
  cp_wait<0>();
}

// One CTA per share and query head of a set: the share whose last set goes on in
// other shares joins their parts, in order.
template <int DT, int HDIM, int HB>
__global__ void __launch_bounds__(JOIN_THREADS) decode_join_kernel(const __grid_constant__ Params p) {
  using T = typename Storage<DT>::T;
  pdl_go();
  pdl_wait();
  const int per = min(p.r, HB);  // heads of a unit, at most
  const int c = blockIdx.x, us = blockIdx.y / per, hq = blockIdx.y - us * per;
  const int4 info = __ldcg(p.info + c);
  if (info.x < 0) return;
  const int unit = info.y * p.set + us, group = unit / p.blocks, block = unit - group * p.blocks;
  if (hq >= p.r - block * HB) return;
  const int head = group * p.r + block * HB + hq;
  auto slot_of = [&](int i) { return ((static_cast<int64_t>(c + i) * 2 + (i == 0 ? 1 : 0)) * p.set + us) * HB + hq; };
  const int count = info.z - c + 1;
  // JOIN_SLICES slices of the parts side by side, four columns a lane, then the
  // slices in order.
  __shared__ float4 so[JOIN_SLICES][32];
  __shared__ float sl[JOIN_SLICES];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const bool on = lane * 4 < HDIM;
  float m = -INFINITY;
  for (int i = lane; i < count; i += 32) m = fmaxf(m, __ldcg(p.part_ml + slot_of(i)).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = finite_max(m);
  float l = 0.0f;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = slice; i < count; i += JOIN_SLICES) {
    const int64_t s = slot_of(i);
    const float2 ml = __ldcg(p.part_ml + s);
    const float4 a = on ? __ldcg(reinterpret_cast<const float4*>(p.part_o + s * HDIM) + lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float f = exp2_hw(ml.x - base);
    l = fmaf(f, ml.y, l);
    v.x = fmaf(f, a.x, v.x), v.y = fmaf(f, a.y, v.y), v.z = fmaf(f, a.z, v.z), v.w = fmaf(f, a.w, v.w);
  }
  so[slice][lane] = v;
  if (lane == 0) sl[slice] = l;
  __syncthreads();
  if (slice != 0) return;
#pragma unroll
  for (int k = 1; k < JOIN_SLICES; ++k) {
    const float4 a = so[k][lane];
    v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    l += sl[k];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (on) {
    uint2 u;
    u.x = pack2<DT>(v.x * inv, v.y * inv);
    u.y = pack2<DT>(v.z * inv, v.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + info.x * p.ldo + static_cast<int64_t>(head) * HDIM + lane * 4) = u;
  }
  if (p.lse != nullptr && lane == 0)
    p.lse[static_cast<int64_t>(info.x) * p.heads + head] = Prob<DT>::lse(m, l);
}

// ---------------------------------------------------------------- host
namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int check_shape(int64_t n, int heads, int kv_heads, int d, int dtype) {
  if (n < 0) return set_error(TPMLP_ERR_INVALID_ARG, "n must be >= 0");
  if (heads < 1 || kv_heads < 1 || kv_heads > heads)
    return set_error(TPMLP_ERR_INVALID_ARG, "heads >= 1 and kv_heads in [1, heads] required");
  if (heads % kv_heads != 0)
    return set_error(TPMLP_ERR_NOT_DIVISIBLE, "the number of heads must be divisible by the number of kv heads");
  if (dtype != DT_F16 && dtype != DT_BF16)
    return set_error(TPMLP_ERR_UNSUPPORTED, "the paged attention runs in float16 or bfloat16 storage");
  if (d != 64 && d != 96 && d != 128) return set_error(TPMLP_ERR_UNSUPPORTED, "head width must be 64, 96 or 128");
  if (heads > 65535 || n >= (1ll << 24)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  return TPMLP_OK;
}

int check_ptr(const void* p, size_t align, const char* name) {
  if (p == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return set_error(align >= 16 ? TPMLP_ERR_UNSUPPORTED : TPMLP_ERR_INVALID_ARG,
                     std::string(name) + " is not " + std::to_string(align) + "-byte aligned");
  return TPMLP_OK;
}

// Query heads of a block: one or two columns of 8.
int heads_of_block(int r) { return r <= 8 ? 8 : 16; }

// Units that the warps of a CTA can take side by side.
int units_of_set(int heads, int kv_heads, int d) {
  if (d * 2 % 128 == 0) return 1;
  const int r = heads / kv_heads, hb = heads_of_block(r), units = kv_heads * ((r + hb - 1) / hb);
  return units % 2 == 0 ? 2 : 1;
}

struct Layout {
  size_t info, ml, o, total;
};
Layout layout(int heads, int kv_heads, int d) {
  Layout L{};
  const size_t parts = static_cast<size_t>(MAX_CTAS) * 2 * units_of_set(heads, kv_heads, d) * heads_of_block(heads / kv_heads);
  L.info = 0;
  L.ml = align256(MAX_CTAS * sizeof(int4));
  L.o = L.ml + align256(parts * sizeof(float2));
  L.total = L.o + align256(parts * d * sizeof(float));
  return L;
}

template <int DT, int HDIM, int NT, int SET>
cudaError_t launch(const Params& p, const DeviceInfo* dev, cudaStream_t st) {
  constexpr int HB = 8 * NT;
  auto* fn = paged_decode_kernel<DT, HDIM, NT, SET>;
  static SmemDone done;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), Dim<HDIM>::SMEM, *dev, &done);
  if (e != cudaSuccess) return e;
  const unsigned ctas = static_cast<unsigned>(std::min(CTAS * dev->num_sms, MAX_CTAS));
  if ((e = launch_pdl(fn, dim3(ctas), WARPS * 32, Dim<HDIM>::SMEM, st, 1, p)) != cudaSuccess) return e;
  const unsigned heads = static_cast<unsigned>(SET * std::min(p.r, HB));
  return launch_pdl(decode_join_kernel<DT, HDIM, HB>, dim3(ctas, heads), JOIN_THREADS, 0, st, 1, p);
}

template <int DT>
cudaError_t launch_dt(const Params& p, int d, const DeviceInfo* dev, cudaStream_t st) {
  const bool one = heads_of_block(p.r) == 8;
  if (d == 128) return one ? launch<DT, 128, 1, 1>(p, dev, st) : launch<DT, 128, 2, 1>(p, dev, st);
  if (d == 64) return one ? launch<DT, 64, 1, 1>(p, dev, st) : launch<DT, 64, 2, 1>(p, dev, st);
  if (p.set == 2) return one ? launch<DT, 96, 1, 2>(p, dev, st) : launch<DT, 96, 2, 2>(p, dev, st);
  return one ? launch<DT, 96, 1, 1>(p, dev, st) : launch<DT, 96, 2, 1>(p, dev, st);
}

}  // namespace
}  // namespace decode

// The rules of a paged cache for `kv_heads` heads of d elements.
int check_kv_cache(const tpmlp_kv_cache* c, int kv_heads, int d, int dtype) {
  using decode::check_ptr;
  if (c == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, "cache is NULL");
  const size_t e = dtype == DT_F32 ? 4 : 2;
  if (const int rc = check_ptr(c->k, 16, "cache k")) return rc;
  if (const int rc = check_ptr(c->v, 16, "cache v")) return rc;
  if (c->pages < 1 || c->page_size < 1) return set_error(TPMLP_ERR_INVALID_ARG, "pages and page_size must be >= 1");
  if (c->pages >= (1ll << 31) || c->page_size >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  const int64_t strides[3] = {c->page_stride, c->token_stride, c->head_stride};
  const int64_t extents[3] = {c->pages, c->page_size, kv_heads};
  for (int i = 0; i < 3; ++i) {
    if (extents[i] > 1 && strides[i] < d)
      return set_error(TPMLP_ERR_INVALID_ARG, "cache strides must be at least the head width");
    if (extents[i] > 1 && strides[i] * e % 16 != 0)
      return set_error(TPMLP_ERR_UNSUPPORTED, "cache strides must be multiples of 16 bytes");
  }
  return TPMLP_OK;
}

namespace decode {

int check_call(const void* q, int64_t ld_q, const tpmlp_kv_cache* cache, const int32_t* block_table, int64_t ld_table,
               int64_t table_width, const int32_t* lengths, float scale, const void* o, int64_t ld_o, const float* lse,
               int64_t n, int heads, int kv_heads, int d, int dtype, const void* ws, size_t ws_bytes) {
  int rc = check_shape(n, heads, kv_heads, d, dtype);
  if (rc) return rc;
  const int64_t W = static_cast<int64_t>(heads) * d;
  if ((rc = check_kv_cache(cache, kv_heads, d, dtype))) return rc;
  if (n > 0 && ((rc = check_ptr(q, 16, "q")) || (rc = check_ptr(o, 16, "o")) ||
                (rc = check_ptr(block_table, 4, "block_table")) || (rc = check_ptr(lengths, 4, "lengths")) ||
                (lse != nullptr && (rc = check_ptr(lse, 4, "lse")))))
    return rc;
  if (ld_q < W || ld_o < W) return set_error(TPMLP_ERR_INVALID_ARG, "ld_q and ld_o must be at least heads*d");
  if (ld_q % 8 != 0 || ld_o % 8 != 0) return set_error(TPMLP_ERR_UNSUPPORTED, "q and o rows must be 16-byte aligned");
  if (table_width < 1 || ld_table < table_width)
    return set_error(TPMLP_ERR_INVALID_ARG, "table_width must be in [1, ld_table]");
  if (table_width >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  if (!std::isfinite(scale)) return set_error(TPMLP_ERR_INVALID_ARG, "scale must be finite");
  const Layout L = layout(heads, kv_heads, d);
  if (ws == nullptr || ws_bytes < L.total)
    return set_error(TPMLP_ERR_WORKSPACE, "paged attention workspace needs " + std::to_string(L.total) + " bytes");
  return check_ptr(ws, 256, "ws");
}

}  // namespace decode
}  // namespace tpmlp

using namespace tpmlp;
using namespace tpmlp::decode;

extern "C" {

size_t tpmlp_paged_attn_workspace_size(int64_t n, int heads, int kv_heads, int d) {
  if (check_shape(n, heads, kv_heads, d, DT_BF16) != TPMLP_OK) return 0;
  return layout(heads, kv_heads, d).total;
}

int tpmlp_paged_attn_decode(const void* q, int64_t ld_q, const tpmlp_kv_cache* cache, const int32_t* block_table,
                            int64_t ld_table, int64_t table_width, const int32_t* lengths, float scale, void* o,
                            int64_t ld_o, float* lse, int64_t n, int heads, int kv_heads, int d, int dtype, void* ws,
                            size_t ws_bytes, void* stream) {
  int rc = check_call(q, ld_q, cache, block_table, ld_table, table_width, lengths, scale, o, ld_o, lse, n, heads, kv_heads, d,
                      dtype, ws, ws_bytes);
  if (rc || n == 0) return rc;
  const int64_t W = static_cast<int64_t>(heads) * d;
  const Layout L = layout(heads, kv_heads, d);
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(ws);
  Params p{};
  p.ldq = ld_q;
  p.k = cache->k;
  p.v = cache->v;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  p.pages = cache->pages;
  p.page_size = static_cast<unsigned>(cache->page_size);
  int log2 = 0;
  while ((1ll << log2) < cache->page_size) ++log2;
  p.page_shift = 31 + log2;
  p.page_magic = static_cast<unsigned>(((1ull << p.page_shift) + p.page_size - 1) / p.page_size);
  p.one_page = p.page_size % SUB == 0 && cache->token_stride < (1 << 26);
  p.width = static_cast<unsigned>(table_width);
  p.ldt = ld_table;
  p.ldo = ld_o;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.r = heads / kv_heads;
  const int hb = heads_of_block(p.r);
  p.blocks = (p.r + hb - 1) / hb;
  // Rows that whole 128-byte lines do not divide share lines with the next head's:
  // where heads are neighbours, neighbours are read together.
  p.set = d * 2 % 128 != 0 && cache->head_stride == d ? units_of_set(heads, kv_heads, d) : 1;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.info = reinterpret_cast<int4*>(w + L.info);
  p.part_ml = reinterpret_cast<float2*>(w + L.ml);
  p.part_o = reinterpret_cast<float*>(w + L.o);
  p.status = dev->status;
  // Larger batches run as several launches of up to MAX_SEQS sequences (fewer where
  // the steps of the longest possible ones, of 32 keys at least, pass 32 bits).
  const uint64_t longest = std::min<uint64_t>(static_cast<uint64_t>(table_width) * cache->page_size, 1ull << 31);
  const int64_t most = std::min<int64_t>(MAX_SEQS, static_cast<int64_t>((1ull << 32) / (longest / 32 + LEAD + 2)));
  for (int64_t i = 0; i < n; i += most) {
    p.n = static_cast<int>(std::min<int64_t>(most, n - i));
    p.q = static_cast<const uint8_t*>(q) + i * ld_q * 2;
    p.o = static_cast<uint8_t*>(o) + i * ld_o * 2;
    p.lse = lse != nullptr ? lse + i * heads : nullptr;
    p.table = block_table + i * ld_table;
    p.lengths = lengths + i;
    const int ph = prof_begin(PROF_SP_REGION, st);
    const cudaError_t e = dtype == DT_F16 ? launch_dt<DT_F16>(p, d, dev, st) : launch_dt<DT_BF16>(p, d, dev, st);
    // the lengths are on the device: queries and outputs only
    prof_end(ph, static_cast<double>(p.n) * W * 4, st, 2);
    if (e != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string("paged attention: ") + cudaGetErrorString(e));
  }
  return TPMLP_OK;
}

}  // extern "C"
