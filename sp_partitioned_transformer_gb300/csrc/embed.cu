// Token embedding at the entry of the trunk: lookup with a scale into the
// sequence chunks, and the table's gradient by sorted tokens ("Tensor
// Parallelism（TP）与 Sequence Parallelism（SP）", §1 (the [b, s] batch becomes
// [s, b, h] behind the embedding) and §5 table, the vocab-parallel embedding
// row: a token outside the table gives a zero row).
//
//   forward   x[m] = scale·E[tok_m]                 (one multiply, one rounding)
//   gradient  dE[v] = scale·Σ_{m : tok_m = v} dX[m] (float32 sum, fixed order)
//
// The gradient runs as two launches.  Its sums are taken in a fixed order, so it is
// the same bits on every call:
//   embed_sort_kernel    a stable radix sort of (token, m) by one cluster of
//                        CTAs (counts exchanged through distributed shared
//                        memory).  When the whole table is written, the other
//                        clusters of the launch fill its first rows with zeros
//                        meanwhile, and the sort marks the rows that have a token;
//                        when sums are added to a float32 gradient, they bring
//                        its rows into L2;
//   embed_grad_kernel    pieces of consecutive sorted rows × column tiles:
//                        every piece costs the same however the tokens are
//                        distributed.  A run of one token inside a piece is
//                        summed in registers and written; a run that crosses a
//                        piece's border leaves a float32 partial row in every
//                        piece, and the last CTA to leave one adds up the run's
//                        rows in order (a counter decides who, never the order).
//                        Between these CTAs, others fill the rest of the table's
//                        rows without a token (writes beside the pieces' reads).
#include <algorithm>
#include <string>

#include "internal.h"

namespace tpmlp {
namespace embed {

struct Tokens {
  const void* p;
  int64_t st, sb;  // strides of the sequence and the batch dimension, in elements
  unsigned b;
  int wide;  // int64 (else int32)
};

struct Chunks {
  void* p[TPMLP_MAX_TP];
  unsigned rpc;  // rows per chunk
};

// The row's token, or `none` where it is outside [0, vocab).
__device__ __forceinline__ unsigned token_of(const Tokens& t, unsigned m, unsigned vocab, unsigned none) {
  const unsigned ti = m / t.b;
  const int64_t at = static_cast<int64_t>(ti) * t.st + static_cast<int64_t>(m - ti * t.b) * t.sb;
  const int64_t v = t.wide ? static_cast<const int64_t*>(t.p)[at] : static_cast<const int32_t*>(t.p)[at];
  return (v < 0 || v >= static_cast<int64_t>(vocab)) ? none : static_cast<unsigned>(v);
}

// A unit of a row: 16 bytes (VEC), or one element when the row length or an
// address rules 16-byte accesses out.
template <int DT, bool VEC>
struct Unit {
  using T = typename Storage<DT>::T;
  static constexpr int N = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  static __device__ __forceinline__ Raw load(const T* p) {
    if constexpr (VEC) return ld_stream_v4(p);
    else return *p;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float* v) {
    if constexpr (!VEC) {
      v[0] = Storage<DT>::to_f32(r);
    } else if constexpr (DT == DT_F32) {
      v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
    } else {
      unpack8<DT>(r, v);
    }
  }
  template <bool STREAM = false>
  static __device__ __forceinline__ void store(T* p, const float* v) {
    if constexpr (!VEC) {
      *p = Storage<DT>::from(v[0]);
    } else {
      uint4 r;
      if constexpr (DT == DT_F32) memcpy(&r, v, 16);
      else r = pack8<DT>(v);
      if constexpr (STREAM) __stcs(reinterpret_cast<uint4*>(p), r);
      else *reinterpret_cast<uint4*>(p) = r;
    }
  }
};

// ---------------------------------------------------------------- forward
// One warp per 128 units of a row, four loads in flight a lane.  Bound by HBM:
// the table's rows once, the output once.  STREAM: an output that L2 (129 MB) cannot
// keep for its reader beside the table's rows is written through it with evict-first
// stores.  They make every large lookup faster by itself, but the reader pays for
// what it then has to fetch: the rule begins where lookup and reader together gain
// (lookup and the LayerNorm behind it, rows of 8192 in bf16: 64 MB 41.7 µs kept
// against 44.9 through, 96 MB 63.0 against 64.5, 112 MB 74.8 against 74.5, 128 MB
// 85.2 against 83.9, 512 MB 307 against 299; the lookup alone 19.7 against 18.5 at
// 64 MB, 135 against 119 at 512; rows of 1024 in fp16 and 4096 in float32 cross
// between 96 and 128 MB too).
constexpr int FWD_WARPS = 8;
constexpr int FWD_U = 4;
constexpr int64_t FWD_STREAM = 112 << 20;  // bytes of output from which on it passes through L2

template <int DT, bool VEC, bool STREAM>
__global__ void __launch_bounds__(FWD_WARPS * 32) embed_forward_kernel(Tokens tok, const void* table,
                                                                       const __grid_constant__ Chunks out, float scale,
                                                                       unsigned M, int64_t h, unsigned vocab,
                                                                       unsigned segs) {
  using U = Unit<DT, VEC>;
  using T = typename U::T;
  const unsigned lane = threadIdx.x & 31;
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * FWD_WARPS + (threadIdx.x >> 5);
  const uint64_t row = segs == 1 ? w : w / segs;
  pdl_go();
  pdl_wait();
  if (row >= M) return;
  const unsigned m = static_cast<unsigned>(row);
  const int64_t units = h / U::N;
  const int64_t u0 = static_cast<int64_t>(w - row * segs) * (32 * FWD_U) + lane;
  const unsigned v = token_of(tok, m, vocab, vocab);
  const unsigned c = m / out.rpc;
  T* dst = static_cast<T*>(out.p[c]) + static_cast<int64_t>(m - c * out.rpc) * h;
  const T* src = static_cast<const T*>(table) + static_cast<int64_t>(v) * h;
  typename U::Raw r[FWD_U];
  if (v < vocab) {
#pragma unroll
    for (int i = 0; i < FWD_U; ++i)
      if (u0 + i * 32 < units) r[i] = U::load(src + (u0 + i * 32) * U::N);
  }
#pragma unroll
  for (int i = 0; i < FWD_U; ++i) {
    if (u0 + i * 32 >= units) break;
    float x[U::N];
    if (v < vocab) {
      U::unpack(r[i], x);
#pragma unroll
      for (int j = 0; j < U::N; ++j) x[j] *= scale;
    } else {
#pragma unroll
      for (int j = 0; j < U::N; ++j) x[j] = 0.0f;
    }
    U::template store<STREAM>(dst + (u0 + i * 32) * U::N, x);
  }
}

// ---------------------------------------------------------------- sort
// Least-significant-digit radix sort, 9 bits a pass (two passes up to 262143
// table rows).  CTA c of the cluster owns a contiguous share of the items and
// warp w of it a contiguous share of that, so ranks that follow (digit, CTA,
// warp, item) order are stable.  Per pass: per-warp digit counts in shared
// memory; the CTA's totals read by the other CTAs; a scan over the digits;
// then each warp places its items 32 at a time.  Latency-bound.
constexpr int SORT_BITS = 9;
constexpr int SORT_BINS = 1 << SORT_BITS;
constexpr int SORT_ROUNDS = 4;  // loads in flight a lane
constexpr int SORT_CLUSTER = 8;
constexpr int64_t SORT_ALONE = 512;  // tokens that one CTA sorts
constexpr uint64_t SORT_FILL = 48ull << 20;  // bytes of the table filled beside the sort, about its time's worth
// Bytes of the float32 gradient's rows brought into L2 beside the sort, for the first
// tokens: half of the cache (129 MB).  4096 rows of 8192 48.6 µs without, 43.4 with
// 64 MB, 42.8 with 96, 44.3 with 128; where 300 tokens share the rows, so that most
// of it is done in vain, 26.1, 27.0, 29.3, 31.4.  (64 MB of dX instead: 45.2 and 26.3.)
constexpr uint64_t SORT_WARM = 64ull << 20;
constexpr size_t sort_smem(int warps) { return static_cast<size_t>(warps * SORT_BINS + 2 * SORT_BINS + 32) * sizeof(unsigned); }

struct SortArgs {
  Tokens tok;
  unsigned M, vocab;
  int passes;
  uint2* pair[2];    // (key, row)
  unsigned* left;    // counters of the sums, to set to zero
  unsigned left_n;
  uint8_t* present;  // [vocab] marks of the rows with a token, or NULL
  uint8_t* fill;     // the table's first bytes, to fill with zeros
  uint64_t fill_bytes;
  const uint8_t* warm;  // the float32 gradient, or NULL
  unsigned warm_rows;   // tokens whose rows of it are brought into L2
  uint64_t warm_bytes;  // of a row
};

// Zeros to [p0, p0 + bytes) by threads me, me + n, …: 16-byte stores between the
// aligned borders, bytes outside.
__device__ __forceinline__ void fill_zero(uint8_t* p, uint64_t bytes, uint64_t me, uint64_t n) {
  const uintptr_t p0 = reinterpret_cast<uintptr_t>(p), p1 = p0 + bytes;
  const uintptr_t q0 = min((p0 + 15) & ~static_cast<uintptr_t>(15), p1), q1 = max(p1 & ~static_cast<uintptr_t>(15), q0);
  for (uint64_t i = me; i < (q1 - q0) / 16; i += n) __stcs(reinterpret_cast<uint4*>(q0) + i, make_uint4(0, 0, 0, 0));
  if (me < q0 - p0) p[me] = 0;
  if (me < p1 - q1) reinterpret_cast<uint8_t*>(q1)[me] = 0;
}

__device__ __forceinline__ unsigned ld_remote(uint32_t cluster_addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

template <int WARPS, int C>
__global__ void __launch_bounds__(WARPS * 32) embed_sort_kernel(const __grid_constant__ SortArgs a) {
  constexpr unsigned T = WARPS * 32;
  constexpr int PER = SORT_BINS > static_cast<int>(T) ? SORT_BINS / static_cast<int>(T) : 1;  // bins of a thread
  extern __shared__ unsigned sm[];
  const unsigned tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = C > 1 ? cluster_ctarank() : 0;
  auto sync_cluster = [] {
    if constexpr (C > 1) cluster_sync_all();
    else __syncthreads();
  };
  pdl_go();
  pdl_wait();
  if (blockIdx.x >= C) {
    if (a.warm != nullptr) {
      const unsigned lines = static_cast<unsigned>(a.warm_bytes / 128);
      const uint64_t all = static_cast<uint64_t>(a.warm_rows) * lines, step = static_cast<uint64_t>(gridDim.x - C) * T;
      for (uint64_t i = static_cast<uint64_t>(blockIdx.x - C) * T + tid; i < all; i += step) {
        const unsigned m = static_cast<unsigned>(i / lines), k = token_of(a.tok, m, a.vocab, a.vocab);
        if (k != a.vocab) prefetch_l2(a.warm + k * a.warm_bytes + (i - static_cast<uint64_t>(m) * lines) * 128);
      }
      return;
    }
    fill_zero(a.fill, a.fill_bytes, static_cast<uint64_t>(blockIdx.x - C) * T + tid, static_cast<uint64_t>(gridDim.x - C) * T);
    return;
  }
  for (unsigned i = rank * T + tid; i < a.left_n; i += C * T) a.left[i] = 0;
  if (a.present != nullptr) {
    fill_zero(a.present, a.vocab, rank * T + tid, C * T);
    sync_cluster();
  }
  unsigned* cnt = sm;                          // [warp][bin]: counts, then places behind the bin's first
  unsigned* tot = sm + WARPS * SORT_BINS;      // [bin]: this CTA's totals
  unsigned* place = tot + SORT_BINS;           // [bin]: the place of this CTA's first item
  unsigned* wsum = place + SORT_BINS;          // block scan
  const unsigned share = ((a.M + C - 1) / C + WARPS - 1) / WARPS;  // items of a warp
  const uint64_t first = static_cast<uint64_t>(rank * WARPS + warp) * share;
  const unsigned begin = static_cast<unsigned>(min(first, static_cast<uint64_t>(a.M)));
  const unsigned end = static_cast<unsigned>(min(first + share, static_cast<uint64_t>(a.M)));
  const unsigned none = a.vocab;  // the key of a token outside the table: sorted last
  unsigned* mine = cnt + warp * SORT_BINS;
  const unsigned bin0 = tid * PER;
  const bool scans = bin0 < SORT_BINS;

  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * SORT_BITS;
    const uint2* src = a.pair[(pass + 1) & 1];
    uint2* dst = a.pair[pass & 1];
    for (unsigned i = lane; i < SORT_BINS; i += 32) mine[i] = 0;
    __syncwarp();
    auto load = [&](unsigned i) { return pass == 0 ? make_uint2(token_of(a.tok, i, a.vocab, none), i) : __ldcg(src + i); };
    uint2 k[SORT_ROUNDS];
    for (unsigned i0 = begin; i0 < end; i0 += 32 * SORT_ROUNDS) {
#pragma unroll
      for (int r = 0; r < SORT_ROUNDS; ++r) {
        const unsigned i = i0 + r * 32 + lane;
        k[r] = i < end ? load(i) : make_uint2(0, 0);
      }
#pragma unroll
      for (int r = 0; r < SORT_ROUNDS; ++r)
        if (i0 + r * 32 + lane < end) {
          atomicAdd(mine + ((k[r].x >> shift) & (SORT_BINS - 1)), 1u);
          if (pass == 0 && a.present != nullptr && k[r].x < a.vocab) a.present[k[r].x] = 1;
        }
    }
    __syncthreads();
    // Per digit: exclusive counts over the warps, and the CTA's total.
    if (scans) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        unsigned sum = 0;
#pragma unroll 8
        for (int w = 0; w < WARPS; ++w) {
          const unsigned c = cnt[w * SORT_BINS + bin0 + j];
          cnt[w * SORT_BINS + bin0 + j] = sum;
          sum += c;
        }
        tot[bin0 + j] = sum;
      }
    }
    sync_cluster();
    unsigned before[PER], all[PER], own = 0;
    if (scans) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        before[j] = 0;
        all[j] = 0;
        if constexpr (C > 1) {
          unsigned v[C];
#pragma unroll
          for (int c = 0; c < C; ++c) v[c] = ld_remote(mapa_shared(smem_u32(tot + bin0 + j), c));
#pragma unroll
          for (int c = 0; c < C; ++c) {
            before[j] += static_cast<unsigned>(c) < rank ? v[c] : 0u;
            all[j] += v[c];
          }
        } else {
          all[j] = tot[bin0 + j];
        }
        own += all[j];
      }
    }
    // Exclusive scan of the digits' totals.
    unsigned inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= static_cast<unsigned>(o)) inc += n;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    if (scans) {
      unsigned base = inc - own;
#pragma unroll
      for (int w = 0; w < SORT_BINS / PER / 32; ++w) base += static_cast<unsigned>(w) < warp ? wsum[w] : 0u;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        place[bin0 + j] = base + before[j];
        base += all[j];
      }
    }
    __syncthreads();
    for (unsigned i0 = begin; i0 < end; i0 += 32 * SORT_ROUNDS) {
      if (end - begin > 32 * SORT_ROUNDS) {  // else they are still in registers
#pragma unroll
        for (int r = 0; r < SORT_ROUNDS; ++r) {
          const unsigned i = i0 + r * 32 + lane;
          k[r] = i < end ? load(i) : make_uint2(0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < SORT_ROUNDS; ++r) {
        if (i0 + r * 32 >= end) break;
        const bool in = i0 + r * 32 + lane < end;
        const unsigned dig = in ? (k[r].x >> shift) & (SORT_BINS - 1) : SORT_BINS;
        const unsigned peers = __match_any_sync(0xffffffffu, dig);
        const unsigned below = __popc(peers & ((1u << lane) - 1u));
        unsigned at = 0;
        if (in) at = mine[dig];
        __syncwarp();
        if (in && below == 0) mine[dig] = at + __popc(peers);
        __syncwarp();
        if (in) __stcg(dst + place[dig] + at + below, k[r]);
      }
    }
    // The next pass reads what the whole cluster wrote; and no CTA leaves or
    // reuses its totals while another still reads them.
    sync_cluster();
  }
}

// ---------------------------------------------------------------- gradient
constexpr int MAX_PIECE = 64;      // sorted rows of a piece: see piece_rows()
constexpr int GRAD_THREADS = 128;  // one unit of columns a thread
// Rows in flight a thread.  When a row's sum is added to the float32 gradient, half
// as many, and two of the gradient's rows: what a piece waits for is the latency of
// those reads one after the other (4096 rows of 8192: 51.9 µs with the reads at each
// run's end behind a prefetch into L2, 48.6 in twos), but more of them in registers
// leave fewer than the seven CTAs an SM that 72 registers do (four CTAs: 54 µs).
template <bool VEC, bool ACC>
struct InFlight {
  static constexpr int ROWS = VEC && ACC ? 4 : 8, SUMS = VEC ? 2 : 8;
};

struct GradArgs {
  const uint2* pair;  // (token, row) in the order of the tokens
  unsigned M, vocab, pieces, piece;  // piece: sorted rows of a piece
  int64_t h;
  unsigned tiles;  // column tiles
  float scale;
  void* grad;   // [vocab, h]: storage type, or float32 to add to
  float* part;     // [pieces][2][h]
  unsigned* left;  // [pieces][tiles] partial rows left of the run that begins in the piece; zeros at the start
  // Whole gradient: of every `every` CTAs the first sums a piece's tile, the others
  // fill fill_rows rows each of the table from row0 on.
  const uint8_t* present;
  unsigned row0, fill_rows, every, sums;  // sums: pieces·tiles
};
constexpr unsigned FILL_BYTES = 64 * 1024;  // of a filling CTA, about,
constexpr unsigned FILL_ROWS = 32;          // and at most (a warp takes a row at a time)

__device__ __forceinline__ unsigned key_at(const GradArgs& a, int64_t i) { return __ldcg(&a.pair[i].x); }

// A unit of the float32 gradient.
template <int N>
__device__ __forceinline__ void load_sum(const float* p, float* v) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + j);
      v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
    }
  } else {
    v[0] = *p;
  }
}

// A finished row unit: scale, then round once, or add to the float32 gradient's
// unit `g`.
template <int DT, bool VEC, bool ACC>
__device__ __forceinline__ void write_row(const GradArgs& a, unsigned v, int64_t col, const float* acc, const float* g) {
  using U = Unit<DT, VEC>;
  float x[U::N];
#pragma unroll
  for (int j = 0; j < U::N; ++j) x[j] = ACC ? fmaf(acc[j], a.scale, g[j]) : acc[j] * a.scale;
  if constexpr (ACC) {
    float* p = static_cast<float*>(a.grad) + static_cast<int64_t>(v) * a.h + col;
    if constexpr (U::N >= 4) {
#pragma unroll
      for (int j = 0; j < U::N; j += 4) *reinterpret_cast<float4*>(p + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    } else {
      *p = x[0];
    }
  } else {
    U::store(static_cast<typename U::T*>(a.grad) + static_cast<int64_t>(v) * a.h + col, x);
  }
}

template <int N>
__device__ __forceinline__ void store_partial(float* p, const float* acc) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int j = 0; j < N; j += 4) __stcg(reinterpret_cast<float4*>(p + j), make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
  } else {
    __stcg(p, acc[0]);
  }
}

template <int N>
__device__ __forceinline__ void load_partial(const float* p, float* v) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(p + j));
      v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
    }
  } else {
    v[0] = __ldcg(p);
  }
}

// The piece in which the run of token k that reaches into `piece` begins, and the
// one in which the run that goes on behind `piece` ends; 32 pieces a step, one a
// lane.
__device__ __forceinline__ unsigned run_start(const GradArgs& a, unsigned k, unsigned piece) {
  for (int64_t i = static_cast<int64_t>(piece) - 1 - (threadIdx.x & 31);; i -= 32) {
    const bool begins = i <= 0 || key_at(a, i * a.piece) != k || key_at(a, i * a.piece - 1) != k;
    const unsigned hit = __ballot_sync(0xffffffffu, begins);
    if (hit != 0) return static_cast<unsigned>(i + (threadIdx.x & 31) - (__ffs(hit) - 1));
  }
}
__device__ __forceinline__ unsigned run_end(const GradArgs& a, unsigned k, unsigned piece) {
  for (uint64_t i = static_cast<uint64_t>(piece) + 1 + (threadIdx.x & 31);; i += 32) {
    const uint64_t m = (i + 1) * a.piece;
    const bool ends = m >= a.M || key_at(a, m - 1) != k || key_at(a, m) != k;
    const unsigned hit = __ballot_sync(0xffffffffu, ends);
    if (hit != 0) return static_cast<unsigned>(i - (threadIdx.x & 31) + __ffs(hit) - 1);
  }
}

template <int DT, bool VEC, bool ACC>
__global__ void __launch_bounds__(GRAD_THREADS) embed_grad_kernel(const __grid_constant__ GradArgs a,
                                                                  const __grid_constant__ Chunks dx) {
  using U = Unit<DT, VEC>;
  using T = typename U::T;
  __shared__ unsigned key[MAX_PIECE + 2];  // with the neighbours' border keys
  __shared__ const T* row[MAX_PIECE];
  __shared__ bool go;
  pdl_go();
  pdl_wait();
  unsigned id = blockIdx.x;
  if constexpr (!ACC) {
    const unsigned turn = id / a.every, in = id - turn * a.every;
    if (in > 0) {
      const uint64_t first = a.row0 + static_cast<uint64_t>(turn * (a.every - 1) + in - 1) * a.fill_rows;
      const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      const uint64_t row_bytes = static_cast<uint64_t>(a.h) * sizeof(T);
      for (uint64_t v = first + warp; v < first + a.fill_rows && v < a.vocab; v += GRAD_THREADS / 32)
        if (!__ldcg(a.present + v)) fill_zero(static_cast<uint8_t*>(a.grad) + v * row_bytes, row_bytes, lane, 32);
      return;
    }
    id = turn;
    if (id >= a.sums) return;
  }
  const unsigned piece = id / a.tiles, tile = id - piece * a.tiles;
  const unsigned m0 = piece * a.piece, n = min(a.piece, a.M - m0);
  constexpr unsigned END = 0xffffffffu;  // no token: vocab < 2^31
  for (unsigned i = threadIdx.x; i < n + 2; i += GRAD_THREADS)
    key[i] = (i == 0 && m0 == 0) || m0 + i - 1 >= a.M ? END : key_at(a, m0 + i - 1);
  for (unsigned i = threadIdx.x; i < n; i += GRAD_THREADS) {
    const unsigned m = __ldcg(&a.pair[m0 + i].y), c = m / dx.rpc;
    row[i] = static_cast<const T*>(dx.p[c]) + static_cast<int64_t>(m - c * dx.rpc) * a.h;
  }
  __syncthreads();
  const int64_t col = (static_cast<int64_t>(tile) * GRAD_THREADS + threadIdx.x) * U::N;
  const bool in = col < a.h;
  constexpr int ROWS = InFlight<VEC, ACC>::ROWS, SUMS = InFlight<VEC, ACC>::SUMS;
  float acc[U::N];
#pragma unroll
  for (int j = 0; j < U::N; ++j) acc[j] = 0.0f;
  bool starts = key[0] != key[1];  // the running sum's run begins in this piece
  bool left[2] = {false, false};   // partial rows of this piece: of a run from before, of one that begins here
  for (unsigned i0 = 0; i0 < n && key[i0 + 1] != a.vocab; i0 += ROWS) {
    typename U::Raw r[ROWS];
    float g[SUMS][U::N];  // the gradient's rows that the next runs' sums are added to
#pragma unroll
    for (int u = 0; u < ROWS; ++u)
      if (in && i0 + u < n) r[u] = U::load(row[i0 + u] + col);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const unsigned i = i0 + u;
      if (i >= n) break;
      if constexpr (ACC) {
        if (u % SUMS == 0) {
#pragma unroll
          for (int w = 0; w < SUMS; ++w) {
            if (!in || i + w >= n) continue;
            const unsigned k = key[i + w + 1];  // written here: its run ends here and begins in this piece
            if (k != key[i + w + 2] && k != key[0] && k != a.vocab)
              load_sum<U::N>(static_cast<const float*>(a.grad) + static_cast<int64_t>(k) * a.h + col, g[w]);
          }
        }
      }
      const unsigned k = key[i + 1];
      if (k == a.vocab) break;  // tokens outside the table come last
      float x[U::N];
      U::unpack(r[u], x);
#pragma unroll
      for (int j = 0; j < U::N; ++j) acc[j] += x[j];
      const bool last = k != key[i + 2];
      if (last || i + 1 == n) {
        if (last && starts) {
          if (in) write_row<DT, VEC, ACC>(a, k, col, acc, g[u % SUMS]);
        } else {
          if (in) store_partial<U::N>(a.part + (static_cast<int64_t>(piece) * 2 + (starts ? 1 : 0)) * a.h + col, acc);
          left[0] = left[0] || !starts;
          left[1] = left[1] || starts;
        }
        starts = true;
#pragma unroll
        for (int j = 0; j < U::N; ++j) acc[j] = 0.0f;
      }
    }
  }
  if (!left[0] && !left[1]) return;
  // The runs that cross this piece's borders: the last of a run's CTAs (of this
  // tile) adds their partial rows, first the one of the piece where it begins.
  __threadfence();
  __syncthreads();
#pragma unroll
  for (int slot = 0; slot < 2; ++slot) {
    if (!left[slot]) continue;
    const unsigned k = slot == 0 ? key[1] : key[n];
    const unsigned first = slot == 1 ? piece : run_start(a, k, piece);
    const unsigned end = slot == 0 && (key[n] != k || key[n + 1] != k) ? piece : run_end(a, k, piece);
    if (threadIdx.x == 0) go = atomicAdd(a.left + static_cast<int64_t>(first) * a.tiles + tile, 1u) == end - first;
    __syncthreads();
    if (go && in) {
      __threadfence();
      load_partial<U::N>(a.part + (static_cast<int64_t>(first) * 2 + 1) * a.h + col, acc);
#pragma unroll 8
      for (unsigned i = first + 1; i <= end; ++i) {
        float x[U::N];
        load_partial<U::N>(a.part + static_cast<int64_t>(i) * 2 * a.h + col, x);
#pragma unroll
        for (int j = 0; j < U::N; ++j) acc[j] += x[j];
      }
      float g[U::N];
      if constexpr (ACC) load_sum<U::N>(static_cast<const float*>(a.grad) + static_cast<int64_t>(k) * a.h + col, g);
      write_row<DT, VEC, ACC>(a, k, col, acc, g);
    }
    __syncthreads();  // `go` is read before the other run sets it
  }
}

// ---------------------------------------------------------------- host
namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
size_t esize(int dtype) { return dtype == DT_F32 ? 4 : 2; }

int check(int64_t s, int64_t b, int64_t h, int64_t vocab, int tp, int dtype, int tok_type) {
  if (s < 0 || b < 0 || h <= 0) return set_error(TPMLP_ERR_INVALID_ARG, "s, b >= 0 and h >= 1 required");
  if (vocab < 1) return set_error(TPMLP_ERR_INVALID_ARG, "vocab must be >= 1");
  if (tp < 1 || tp > TPMLP_MAX_TP) return set_error(TPMLP_ERR_INVALID_ARG, "tp must be in [1, 64]");
  if (dtype < DT_F32 || dtype > DT_BF16) return set_error(TPMLP_ERR_INVALID_ARG, "unknown dtype");
  if (tok_type != TPMLP_I32 && tok_type != TPMLP_I64) return set_error(TPMLP_ERR_INVALID_ARG, "unknown index type");
  if (s > (1ll << 31) || b > (1ll << 31) || s * b >= (1ll << 31) || h >= (1ll << 31) || vocab >= (1ll << 31))
    return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  if (s % tp != 0)
    return set_error(TPMLP_ERR_NOT_DIVISIBLE, "First dimension of the tensor should be divisible by tensor parallel size");
  return TPMLP_OK;
}

int check_ptr(const void* p, size_t align, const char* name) {
  if (p == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " is misaligned");
  return TPMLP_OK;
}

int check_chunks(const void* const* a, int n, size_t align, const char* name) {
  if (a == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " array is NULL");
  for (int i = 0; i < n; ++i)
    if (const int rc = check_ptr(a[i], align, name)) return rc;
  return TPMLP_OK;
}

// 16-byte units: rows of whole units at 16-byte addresses.
bool vector_rows(const void* const* chunks, int tp, const void* other, int64_t h, size_t e) {
  uintptr_t bits = reinterpret_cast<uintptr_t>(other) | static_cast<uintptr_t>(h * e);
  for (int i = 0; i < tp; ++i) bits |= reinterpret_cast<uintptr_t>(chunks[i]);
  return bits % 16 == 0;
}

// Sorted rows of a piece: as many as leave six CTAs for each of 152 SMs (a piece of
// 16-bit rows has a CTA for every 1024 columns), from 8 to 64.  Longer pieces have
// fewer borders to cross, shorter ones balance: added to the gradient, 4096 rows of
// 8192 took 53.4 µs with pieces of 64, 48.6 with 32 and 49.3 with 16 (26.1 with 32
// and 32.7 with 16 when 300 tokens share the rows); 16384 of 512 29.6 with 16 and
// 35.6 with 8; the whole gradient from 8192 rows of 6144 126.0 with 64, 123.5 with 32.
unsigned piece_rows(int64_t M, int64_t h) {
  const int64_t tiles = (h + 1023) / 1024;
  unsigned rows = MAX_PIECE;
  while (rows > 8 && (M + rows - 1) / rows * tiles < 6 * 152) rows /= 2;
  return rows;
}

struct Layout {
  unsigned piece;
  size_t pair[2], present, left, part, total;
  unsigned pieces;
};
Layout layout(int64_t M, int64_t h, int64_t vocab) {
  Layout L{};
  const size_t one = align256(static_cast<size_t>(M) * sizeof(uint2));
  L.pair[0] = 0;
  L.pair[1] = one;
  L.present = 2 * one;
  L.left = L.present + (M > 0 ? align256(static_cast<size_t>(vocab)) : 0);
  L.piece = piece_rows(M, h);
  L.pieces = static_cast<unsigned>((M + L.piece - 1) / L.piece);
  // (counters for the tiles of single elements, the most that a row can have)
  L.part = L.left + (L.pieces > 1 ? align256(static_cast<size_t>(L.pieces) * ((h + GRAD_THREADS - 1) / GRAD_THREADS) * 4) : 0);
  // a single piece has no border that a run could cross
  L.total = L.part + (L.pieces > 1 ? align256(static_cast<size_t>(L.pieces) * 2 * h * sizeof(float)) : 0);
  return L;
}

int check_launch(const char* what, cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  return TPMLP_OK;
}

template <int WARPS, int C>
cudaError_t launch_sort(unsigned grid, const DeviceInfo& dev, cudaStream_t st, const SortArgs& a) {
  auto* fn = embed_sort_kernel<WARPS, C>;
  constexpr size_t smem = sort_smem(WARPS);
  if (smem > 48 * 1024) {
    static SmemDone done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem, dev, &done);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(fn, dim3(grid), WARPS * 32, smem, st, C, a);
}

template <int DT, bool VEC, bool ACC>
cudaError_t launch_sums(GradArgs g, const Chunks& dx, cudaStream_t st, int* kernels) {
  g.sums = g.pieces * g.tiles;
  uint64_t grid = g.sums;
  if (!ACC) {
    // filling CTAs between the summing ones, at least one behind each
    const uint64_t fills = (g.vocab - g.row0 + g.fill_rows - 1) / g.fill_rows;
    const uint64_t beside = std::max<uint64_t>(1, (fills + g.sums - 1) / g.sums);
    g.every = static_cast<unsigned>(beside) + 1;
    grid = static_cast<uint64_t>(g.sums) * g.every;
  }
  cudaError_t e = launch_pdl(embed_grad_kernel<DT, VEC, ACC>, dim3(static_cast<unsigned>(grid)), GRAD_THREADS, 0, st, 1, g, dx);
  *kernels += 1;
  return e;
}

int backward(const void* tokens, int tok_type, int64_t stride_s, int64_t stride_b, const void* const* dx, void* grad,
             bool acc, float scale, void* ws, size_t ws_bytes, int64_t s, int64_t b, int64_t h, int64_t vocab, int tp,
             int dtype, cudaStream_t st) {
  int rc = check(s, b, h, vocab, tp, dtype, tok_type);
  if (rc) return rc;
  const size_t e = esize(dtype);
  const int64_t M = s * b;
  if ((M > 0 && ((rc = check_ptr(tokens, tok_type == TPMLP_I64 ? 8 : 4, "tokens")) || (rc = check_chunks(dx, tp, e, "dx")))) ||
      (rc = check_ptr(grad, acc ? 4 : e, acc ? "main_grad" : "dtable")))
    return rc;
  const Layout L = layout(M, h, vocab);
  if (L.total > 0) {
    if (ws == nullptr || ws_bytes < L.total)
      return set_error(TPMLP_ERR_WORKSPACE, "embedding backward workspace needs " + std::to_string(L.total) + " bytes");
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
      return set_error(TPMLP_ERR_UNSUPPORTED, "ws is not 256-byte aligned");
  }
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  const uint64_t table_bytes = static_cast<uint64_t>(vocab) * h * e;
  if (M == 0) {
    if (acc) return TPMLP_OK;
    return check_launch("embedding backward", cudaMemsetAsync(grad, 0, table_bytes, st));
  }
  const bool vec = vector_rows(dx, tp, grad, h, e);
  const int64_t per = vec ? 16 / static_cast<int64_t>(e) : 1;
  const int64_t tiles = (h / per + GRAD_THREADS - 1) / GRAD_THREADS;
  // (the grid: twice the summing CTAs at most, and a filling CTA for each row of the table at most)
  if (static_cast<int64_t>(L.pieces) * tiles + vocab >= (1ll << 30))
    return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  uint8_t* w = static_cast<uint8_t*>(ws);
  SortArgs sa{};
  sa.tok = Tokens{tokens, stride_s, stride_b, static_cast<unsigned>(b), tok_type == TPMLP_I64};
  sa.M = static_cast<unsigned>(M);
  sa.vocab = static_cast<unsigned>(vocab);
  int bits = 1;  // of the keys 0 … vocab
  while (bits < 32 && (static_cast<uint64_t>(vocab) >> bits) != 0) ++bits;
  sa.passes = (bits + SORT_BITS - 1) / SORT_BITS;
  for (int i = 0; i < 2; ++i) sa.pair[i] = reinterpret_cast<uint2*>(w + L.pair[i]);
  const int ph = prof_begin(PROF_SP_REGION, st);
  cudaError_t er;
  const unsigned cluster = M > SORT_ALONE ? SORT_CLUSTER : 1, threads = cluster > 1 ? 1024 : 256;
  unsigned grid = cluster;
  sa.left = reinterpret_cast<unsigned*>(w + L.left);
  sa.left_n = L.pieces > 1 ? L.pieces * static_cast<unsigned>(tiles) : 0;
  const uint64_t row_bytes = static_cast<uint64_t>(h) * e;
  const uint64_t early = std::min<uint64_t>(vocab, SORT_FILL / row_bytes);  // rows filled beside the sort
  uint64_t want;  // threads beside the sort
  if (acc) {
    sa.warm = static_cast<const uint8_t*>(grad);
    sa.warm_bytes = static_cast<uint64_t>(h) * sizeof(float);
    sa.warm_rows = static_cast<unsigned>(std::min<uint64_t>(M, SORT_WARM / sa.warm_bytes));
    want = sa.warm_rows * (sa.warm_bytes / 128);
  } else {
    sa.present = w + L.present;
    sa.fill = static_cast<uint8_t*>(grad);
    sa.fill_bytes = early * row_bytes;
    want = sa.fill_bytes / 16;
  }
  const uint64_t most = 2048ull / threads * dev->num_sms;
  grid += static_cast<unsigned>((std::min((want + threads - 1) / threads, most) + cluster - 1) / cluster) * cluster;
  if (cluster == 1) er = launch_sort<8, 1>(grid, *dev, st, sa);
  else er = launch_sort<32, SORT_CLUSTER>(grid, *dev, st, sa);
  if (er != cudaSuccess) return check_launch("embedding sort", er);
  GradArgs g{};
  g.pair = sa.pair[(sa.passes - 1) & 1];
  g.M = sa.M;
  g.vocab = sa.vocab;
  g.pieces = L.pieces;
  g.piece = L.piece;
  g.h = h;
  g.scale = scale;
  g.grad = grad;
  g.part = reinterpret_cast<float*>(w + L.part);
  g.present = w + L.present;
  g.left = sa.left;
  g.tiles = static_cast<unsigned>(tiles);
  g.row0 = static_cast<unsigned>(early);
  g.fill_rows = static_cast<unsigned>(std::max<uint64_t>(1, std::min<uint64_t>(FILL_BYTES / row_bytes, FILL_ROWS)));
  Chunks c{};
  for (int i = 0; i < tp; ++i) c.p[i] = const_cast<void*>(dx[i]);
  c.rpc = static_cast<unsigned>(M / tp);
  int kernels = 1;
#define SUMS(D)                                                                                              \
  (vec ? (acc ? launch_sums<D, true, true>(g, c, st, &kernels) : launch_sums<D, true, false>(g, c, st, &kernels)) \
       : (acc ? launch_sums<D, false, true>(g, c, st, &kernels) : launch_sums<D, false, false>(g, c, st, &kernels)))
  er = dtype == DT_F32 ? SUMS(DT_F32) : dtype == DT_F16 ? SUMS(DT_F16) : SUMS(DT_BF16);
#undef SUMS
  prof_end(ph, static_cast<double>(M) * h * e + (acc ? 0.0 : static_cast<double>(table_bytes)), st, kernels);
  return check_launch("embedding backward", er);
}

}  // namespace
}  // namespace embed
}  // namespace tpmlp

using namespace tpmlp;
using namespace tpmlp::embed;

extern "C" {

int tpmlp_embed_forward(const void* tokens, int tok_type, int64_t stride_s, int64_t stride_b, const void* table,
                        float scale, void* const* out, int64_t s, int64_t b, int64_t h, int64_t vocab, int tp, int dtype,
                        void* stream) {
  int rc = check(s, b, h, vocab, tp, dtype, tok_type);
  if (rc) return rc;
  const size_t e = esize(dtype);
  if ((rc = check_ptr(table, e, "table"))) return rc;
  const int64_t M = s * b;
  if (M == 0) return TPMLP_OK;
  if ((rc = check_ptr(tokens, tok_type == TPMLP_I64 ? 8 : 4, "tokens")) ||
      (rc = check_chunks(const_cast<const void* const*>(out), tp, e, "out")))
    return rc;
  const bool vec = vector_rows(const_cast<const void* const*>(out), tp, table, h, e);
  const int64_t units = vec ? h * static_cast<int64_t>(e) / 16 : h;
  const int64_t segs = (units + 32 * FWD_U - 1) / (32 * FWD_U);
  const int64_t blocks = (M * segs + FWD_WARPS - 1) / FWD_WARPS;
  if (blocks >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  const Tokens t{tokens, stride_s, stride_b, static_cast<unsigned>(b), tok_type == TPMLP_I64};
  Chunks c{};
  for (int i = 0; i < tp; ++i) c.p[i] = out[i];
  c.rpc = static_cast<unsigned>(M / tp);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int ph = prof_begin(PROF_SP_REGION, st);
  const bool stream_out = vec && M * h * static_cast<int64_t>(e) >= FWD_STREAM;
  cudaError_t er;
#define FWD(D, V, S)                                                                                             \
  er = launch_pdl(embed_forward_kernel<D, V, S>, dim3(static_cast<unsigned>(blocks)), FWD_WARPS * 32, 0, st, 1, t, \
                  table, c, scale, static_cast<unsigned>(M), h, static_cast<unsigned>(vocab),                    \
                  static_cast<unsigned>(segs))
#define FWD_DT(D)                                                      \
  do {                                                                 \
    if (!vec) FWD(D, false, false);                                    \
    else if (stream_out) FWD(D, true, true);                           \
    else FWD(D, true, false);                                          \
  } while (0)
  if (dtype == DT_F32) FWD_DT(DT_F32); else if (dtype == DT_F16) FWD_DT(DT_F16); else FWD_DT(DT_BF16);
#undef FWD_DT
#undef FWD
  prof_end(ph, 2.0 * static_cast<double>(M) * h * e, st);
  return check_launch("embedding forward", er);
}

size_t tpmlp_embed_backward_workspace(int64_t s, int64_t b, int64_t h, int64_t vocab) {
  if (check(s, b, h, vocab, 1, DT_F32, TPMLP_I32) != TPMLP_OK) return 0;
  return layout(s * b, h, vocab).total;
}

int tpmlp_embed_backward(const void* tokens, int tok_type, int64_t stride_s, int64_t stride_b, const void* const* dx,
                         void* dtable, float scale, void* ws, size_t ws_bytes, int64_t s, int64_t b, int64_t h,
                         int64_t vocab, int tp, int dtype, void* stream) {
  return backward(tokens, tok_type, stride_s, stride_b, dx, dtable, false, scale, ws, ws_bytes, s, b, h, vocab, tp,
                  dtype, static_cast<cudaStream_t>(stream));
}

int tpmlp_embed_backward_main_grad(const void* tokens, int tok_type, int64_t stride_s, int64_t stride_b,
                                   const void* const* dx, float* main_grad, float scale, void* ws, size_t ws_bytes,
                                   int64_t s, int64_t b, int64_t h, int64_t vocab, int tp, int dtype, void* stream) {
  return backward(tokens, tok_type, stride_s, stride_b, dx, main_grad, true, scale, ws, ws_bytes, s, b, h, vocab, tp,
                  dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
