// Norms of queries and keys per head with the position rotation, in one pass
// over the fused QKV projection's output (the group layout of attn.cu), its
// backward, and the serving form that writes keys and values into a paged cache.
//
//   x̂ = x/√(mean_d(x²) + eps),  n = x̂·γ            (γ_q or γ_k; optional)
//   (y_a, y_b) = (n_a·c − n_b·s, n_b·c + n_a·s)      over pairs (a, b) of the
//                head's first `rot` columns: (i, i + rot/2), or (2i, 2i + 1)
//   backward: dn = Rᵀ·dy, t = dn·γ, dx = (t − x̂·mean_d(t·x̂))/√(mean_d(x²) + eps),
//             dγ = Σ dn·x̂ over tokens and the heads that share γ
//
// All of it is bound by HBM (each element read once and written once; nothing
// but the 2·d sums of dγ crosses a head), so the layout serves wide accesses and
// few instructions:
// * a head is d/16 lanes, each holding the two 8-element vectors whose elements
//   are paired by the rotation, so that the rotation needs no exchange and the
//   row sum is a shuffle over 4, 6, 8 or 16 lanes;
// * a warp steps over a contiguous range of items (kind of head, row, batch of
//   heads); its lanes copy their own vectors of the items ahead into shared
//   memory with cp.async, so that loads stay in flight behind the arithmetic and
//   no lane waits for another; the angles are fetched one item ahead;
// * γ and the angles of an item are combined once and serve all its heads, and
//   the arithmetic runs on float32 pairs.
#include <algorithm>
#include <string>

#include "internal.h"

namespace tpmlp {
namespace qkrope {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int STAGES = 4;    // items in flight or in work, of every warp
constexpr int FWD_U = 2;     // heads a lane group takes of an item
constexpr int BWD_U = 2;
constexpr int FWD_CTAS = 4;  // per SM
constexpr int BWD_CTAS = 3;

// What a warp does with its heads: the kinds take different warps, so that a
// warp's γ and angles can be combined once for all its heads.
enum Kind { QUERY = 0, KEY = 1, VALUE = 2 };

struct Params {
  const void* x;   // [rows, ldx]
  void* y;         // [rows, ldy]: the rotated QKV, or (append) q only
  int64_t ldx, ldy;
  const void* gq;
  const void* gk;
  const float* cos;
  const float* sin;
  int64_t max_pos;
  const void* pos;  // NULL: row / b
  int pos64;
  unsigned b, rows;
  unsigned r, r_magic;  // query heads of a group; ⌊2³²/r⌋ + 1: j / r of a query head j is the product's upper half
  int heads, kv_heads;
  int d, rot, interleaved, norm;
  float eps, inv_d;
  unsigned batches[3];  // items per row of queries, keys and values (0 values: in place, v stays)
  uint64_t qk_items, v_items;
  unsigned* status;
  // append
  void* kc;
  void* vc;
  const int64_t* slots;
  int64_t pages, page_size;
  int64_t page_stride, token_stride, head_stride;
  // backward
  const void* dy;
  int64_t lddy;
  float* part;  // [blocks][2][d]
};

// Float32 pairs: one instruction for both halves (the kernels' arithmetic is a
// third of their time otherwise).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float2 swap2(float2 v) { return make_float2(v.y, v.x); }

// `real` false: nothing is read and zeros are written.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight elements of storage type DT, and in float32 as four pairs.
template <int DT>
struct Vec8 {
  static constexpr int N = DT == DT_F32 ? 2 : 1;  // 16-byte units
  uint4 r[N];
  static constexpr int E = DT == DT_F32 ? 4 : 2;  // bytes of an element
  __device__ __forceinline__ void load(const void* base, int elem) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + elem * E);
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = __ldg(p + i);
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p)[i] = r[i];
  }
  // To and from this lane's place in the ring (a shared address): units THREADS apart.
  static __device__ __forceinline__ void fetch(uint32_t ring, const uint8_t* p, bool real) {
#pragma unroll
    for (int i = 0; i < N; ++i) cp_async16(ring + i * THREADS * 16, p + i * 16, real);
  }
  __device__ __forceinline__ void take(uint32_t ring) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r[i].x), "=r"(r[i].y), "=r"(r[i].z), "=r"(r[i].w)
                   : "r"(ring + i * THREADS * 16)
                   : "memory");
  }
  __device__ __forceinline__ void get(float2* v) const {
    if constexpr (DT == DT_F32) {
      memcpy(v, r, 32);
    } else {
      float t[8];
      unpack8<DT>(r[0], t);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = make_float2(t[2 * i], t[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void set(const float2* v) {
    if constexpr (DT == DT_F32) {
      memcpy(r, v, 32);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DT_BF16) {
          const __nv_bfloat162 h = __float22bfloat162_rn(v[i]);
          memcpy(&w[i], &h, 4);
        } else {
          const __half2 h = __float22half2_rn(v[i]);
          memcpy(&w[i], &h, 4);
        }
      }
      r[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// What a lane holds of every head: two vectors, and how the rotation pairs them.
struct LanePlan {
  bool live;    // the lane has columns (d/16 lanes of the group do)
  int ca, cb;   // first column of the two vectors
  bool ra, rb;  // each is rotated (split halves: both or none)
};

__device__ __forceinline__ LanePlan lane_plan(const Params& p, int l) {
  LanePlan q;
  const int n = p.d / 16;
  q.live = l < n;
  if (p.interleaved) {
    q.ca = l * 8;
    q.cb = (l + n) * 8;
    q.ra = q.live && q.ca < p.rot;
    q.rb = q.live && q.cb < p.rot;
  } else {
    const int half = p.rot / 16;
    const bool r = l < half;
    q.ca = r ? l * 8 : p.rot + (l - half) * 16;
    q.cb = r ? l * 8 + p.rot / 2 : q.ca + 8;
    q.ra = q.rb = q.live && r;
  }
  return q;
}

__device__ __forceinline__ int64_t position_of(const Params& p, unsigned row) {
  int64_t at;
  if (p.pos == nullptr) at = row / p.b;
  else at = p.pos64 ? static_cast<const int64_t*>(p.pos)[row] : static_cast<const int32_t*>(p.pos)[row];
  if (at < 0 || at >= p.max_pos) {
    // outside the tables: reported, and the nearest angle taken instead of a bad read
    atomicCAS(p.status, 0u, STATUS_BAD_INDEX);
    at = at < 0 ? 0 : p.max_pos - 1;
  }
  return at;
}

// cos and sin of the lane's eight pairs.  Split halves: pair i is element i of
// the two vectors.  Interleaved: pairs 0–3 lie in the first vector, 4–7 in the
// second.  Lanes whose columns are not rotated load nothing.
struct Angles {
  float4 c[2], s[2];
  __device__ __forceinline__ void load(const Params& p, const LanePlan& q, int64_t pos) {
    const int64_t at = pos * (p.rot / 2);
    const int64_t a = at + (p.interleaved ? q.ca / 2 : q.ca), b = at + (p.interleaved ? q.cb / 2 : q.ca + 4);
    if (q.ra) {
      c[0] = __ldg(reinterpret_cast<const float4*>(p.cos + a));
      s[0] = __ldg(reinterpret_cast<const float4*>(p.sin + a));
    }
    if (q.rb) {
      c[1] = __ldg(reinterpret_cast<const float4*>(p.cos + b));
      s[1] = __ldg(reinterpret_cast<const float4*>(p.sin + b));
    }
  }
  __device__ __forceinline__ float cosine(int i) const { return reinterpret_cast<const float*>(c)[i]; }
  __device__ __forceinline__ float sine(int i) const { return reinterpret_cast<const float*>(s)[i]; }
};

// Lanes of a head's group: a power of two that holds d/16 lanes, or exactly six
// for d = 96 (five heads a warp instead of four).
template <int GL>
__device__ __forceinline__ float group_sum(float v, int lane) {
  if constexpr (GL == 6) {
    const int l = lane % 6, first = lane - l;
    // opposite lanes, then the three pairs; lanes 30 and 31 form no group
    v += __shfl_sync(0xffffffffu, v, first + (l < 3 ? l + 3 : l - 3));
    const float a = __shfl_sync(0xffffffffu, v, first + (l < 5 ? l + 1 : 0));
    const float b = __shfl_sync(0xffffffffu, v, first + (l < 4 ? l + 2 : l - 4));
    // the same order of the three on every lane
    const int k = l % 3;
    const float p0 = k == 0 ? v : k == 1 ? b : a, p1 = k == 0 ? a : k == 1 ? v : b, p2 = k == 0 ? b : k == 1 ? a : v;
    v = p0 + p1 + p2;
  } else {
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// Sum of squares of the lane's 16 elements.
__device__ __forceinline__ float squares(const float2* a, const float2* b) {
  float2 s = mul2(a[0], a[0]), t = mul2(b[0], b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s = fma2(a[i], a[i], s);
    t = fma2(b[i], b[i], t);
  }
  return (s.x + t.x) + (s.y + t.y);
}

// The place of a warp in its items: a kind, a row and a batch of PER heads of that
// kind in the row.  A warp has a contiguous range of the query and key items
// (queries of all rows, then keys), then one of the value items: the sums of dγ
// are then the same whether values move or not.
template <int PER>
struct Cursor {
  int kind;
  unsigned row, batch;
  unsigned left;  // query and key items still to come
  uint64_t v0;    // first value item
  // Places the cursor and returns the number of items.
  __device__ __forceinline__ unsigned begin(const Params& p, uint64_t w, uint64_t warps) {
    const uint64_t q0 = p.qk_items * w / warps, q1 = p.qk_items * (w + 1) / warps;
    v0 = p.v_items * w / warps;
    const uint64_t v1 = p.v_items * (w + 1) / warps;
    left = static_cast<unsigned>(q1 - q0);
    if (left > 0) seek(p, q0);
    else values(p);
    return left + static_cast<unsigned>(v1 - v0);
  }
  __device__ __forceinline__ void seek(const Params& p, uint64_t at) {
    const uint64_t queries = static_cast<uint64_t>(p.rows) * p.batches[QUERY];
    kind = at < queries ? QUERY : KEY;
    if (kind == KEY) at -= queries;
    place(p, at);
  }
  __device__ __forceinline__ void values(const Params& p) {
    kind = VALUE;
    row = batch = 0;
    if (p.v_items > 0) place(p, v0);
  }
  __device__ __forceinline__ void place(const Params& p, uint64_t at) {
    row = static_cast<unsigned>(at / p.batches[kind]);
    batch = static_cast<unsigned>(at - static_cast<uint64_t>(row) * p.batches[kind]);
  }
  __device__ __forceinline__ void next(const Params& p) {
    if (left > 0 && --left == 0) return values(p);
    if (++batch < p.batches[kind]) return;
    batch = 0;
    if (++row < p.rows) return;
    row = 0;
    if (kind == QUERY) kind = KEY;
  }
  __device__ __forceinline__ int count(const Params& p) const { return kind == QUERY ? p.heads : p.kv_heads; }
};

// First column of head j of a kind in the fused projection's row.
__device__ __forceinline__ int column_of(const Params& p, int kind, int j) {
  if (kind == QUERY) return (j + 2 * static_cast<int>(p.r == 1 ? j : __umulhi(j, p.r_magic))) * p.d;
  return (j * static_cast<int>(p.r + 2) + static_cast<int>(p.r) + kind - 1) * p.d;
}

// ---------------------------------------------------------------- forward, append
// γ and the angles of a row and kind, combined: y = r·(u·x + v·partner(x)).
// Split halves: the partner of one vector is the other; interleaved: the pair's
// other element.  Not rotated: u = γ alone.
struct Combined {
  float2 u[8], v[8];
  template <int DT>
  __device__ __forceinline__ void make(const Params& p, const LanePlan& q, int kind, const Angles& t) {
    float2 g[8];
    if (p.norm && q.live) {
      Vec8<DT> w;
      w.load(kind == QUERY ? p.gq : p.gk, q.ca);
      w.get(g);
      w.load(kind == QUERY ? p.gq : p.gk, q.cb);
      w.get(g + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = both(1.0f);
    }
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool on = i < 4 ? q.ra : q.rb;
        u[i] = on ? mul2(g[i], both(t.cosine(i))) : g[i];
        v[i] = on ? make_float2(-g[i].y * t.sine(i), g[i].x * t.sine(i)) : both(0.0f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = make_float2(t.cosine(2 * i), t.cosine(2 * i + 1));
        const float2 s = make_float2(t.sine(2 * i), t.sine(2 * i + 1));
        u[i] = q.ra ? mul2(g[i], c) : g[i];
        u[4 + i] = q.ra ? mul2(g[4 + i], c) : g[4 + i];
        v[i] = neg2(mul2(g[4 + i], s));
        v[4 + i] = mul2(g[i], s);
      }
    }
  }
};

// The slot's row of the cache, −1 for a token that is not cached.
__device__ __forceinline__ int64_t cache_row_of(const Params& p, unsigned row) {
  const int64_t slot = p.slots[row];
  if (slot < 0) return -1;
  const int64_t page = slot / p.page_size;
  if (page < p.pages) return page * p.page_stride + (slot - page * p.page_size) * p.token_stride;
  atomicCAS(p.status, 0u, STATUS_BAD_INDEX);  // behind the cache: reported, nothing written
  return -1;
}

// APPEND: q goes to y, k and v to the cache.
template <int DT, int GL, int U, bool APPEND>
__global__ void __launch_bounds__(THREADS, FWD_CTAS) qk_forward_kernel(const __grid_constant__ Params p) {
  using V = Vec8<DT>;
  constexpr int G = 32 / GL, E = V::E, VEC = V::N * THREADS * 16, STAGE = U * 2 * VEC;
  extern __shared__ uint4 smem[];
  const int lane = threadIdx.x & 31;
  const LanePlan q = lane_plan(p, lane < G * GL ? lane % GL : 32);
  const int grp = lane / GL, ca = q.ca * E, cb = q.cb * E;
  const uint32_t ring = smem_u32(smem) + threadIdx.x * 16;
  Cursor<G * U> at, ahead;
  const unsigned n = at.begin(p, static_cast<uint64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5),
                              static_cast<uint64_t>(gridDim.x) * WARPS);
  if (n == 0) return;
  ahead = at;
  auto fetch = [&](unsigned i) {
    if (i < n) {
      const uint32_t st = ring + (i % STAGES) * STAGE;
      const int count = ahead.count(p), j0 = static_cast<int>(ahead.batch) * G * U + grp;
      const uint8_t* x = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(ahead.row) * p.ldx * E;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int j = j0 + k * G;
        const bool on = j < count && q.live;
        const uint8_t* c = x + (on ? column_of(p, ahead.kind, j) * E : 0);
        V::fetch(st + k * 2 * VEC, c + (on ? ca : 0), on);
        V::fetch(st + k * 2 * VEC + VEC, c + (on ? cb : 0), on);
      }
      ahead.next(p);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  Angles t;
  if (p.rot > 0 && at.kind != VALUE) t.load(p, q, position_of(p, at.row));
  Combined c;
  bool fresh = true;  // t holds a row's angles that c does not have yet
  for (unsigned i = 0; i < n; ++i) {
    fetch(i + STAGES - 1);
    if (fresh && at.kind != VALUE) c.make<DT>(p, q, at.kind, t);
    Cursor<G * U> next = at;
    next.next(p);
    fresh = next.row != at.row || next.kind != at.kind;
    if (p.rot > 0 && fresh && i + 1 < n && next.kind != VALUE) t.load(p, q, position_of(p, next.row));
    uint8_t* y = static_cast<uint8_t*>(p.y) + static_cast<int64_t>(at.row) * p.ldy * E;
    bool cached = true;
    if constexpr (APPEND) {
      if (at.kind != QUERY) {
        const int64_t row = cache_row_of(p, at.row);
        cached = row >= 0;
        y = static_cast<uint8_t*>(at.kind == KEY ? p.kc : p.vc) + row * E;
      }
    }
    cp_wait<STAGES - 1>();
    const uint32_t st = ring + (i % STAGES) * STAGE;
    const int count = at.count(p), j0 = static_cast<int>(at.batch) * G * U + grp;
    V va[U], vb[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      va[k].take(st + k * 2 * VEC);
      vb[k].take(st + k * 2 * VEC + VEC);
    }
    if (at.kind != VALUE) {
      float2 x[U][8];
      float r[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        va[k].get(x[k]);
        vb[k].get(x[k] + 4);
        r[k] = 1.0f;
      }
      if (p.norm) {
#pragma unroll
        for (int k = 0; k < U; ++k) r[k] = squares(x[k], x[k] + 4);
#pragma unroll
        for (int k = 0; k < U; ++k) r[k] = rsqrtf(fmaf(group_sum<GL>(r[k], lane), p.inv_d, p.eps));
      }
      if (p.interleaved) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 s = swap2(x[k][e]);
            x[k][e] = mul2(x[k][e], c.u[e]);
            if (e < 4 ? q.ra : q.rb) x[k][e] = fma2(s, c.v[e], x[k][e]);
            x[k][e] = mul2(x[k][e], both(r[k]));
          }
      } else if (q.ra) {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = x[k][e], b = x[k][4 + e];
            x[k][e] = mul2(fma2(b, c.v[e], mul2(a, c.u[e])), both(r[k]));
            x[k][4 + e] = mul2(fma2(a, c.v[4 + e], mul2(b, c.u[4 + e])), both(r[k]));
          }
      } else {
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = mul2(mul2(x[k][e], c.u[e]), both(r[k]));
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        va[k].set(x[k]);
        vb[k].set(x[k] + 4);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int j = j0 + k * G;
      if (j < count && q.live && cached) {
        uint8_t* d;
        if constexpr (APPEND) d = y + (at.kind == QUERY ? static_cast<int64_t>(j) * p.d : j * p.head_stride) * E;
        else d = y + column_of(p, at.kind, j) * E;
        va[k].store(d + ca);
        vb[k].store(d + cb);
      }
    }
    at = next;
  }
}

// ---------------------------------------------------------------- backward
// A lane keeps the dγ sums of its 16 columns, stored when the warp passes from
// queries to keys and at the end, added over the block and over the blocks, in
// block order, by qk_gamma_kernel.
template <int DT, int GL, int U>
__global__ void __launch_bounds__(THREADS, BWD_CTAS) qk_backward_kernel(const __grid_constant__ Params p) {
  using V = Vec8<DT>;
  constexpr int G = 32 / GL, E = V::E, VEC = V::N * THREADS * 16, PLACE = 4 * VEC, STAGE = U * PLACE;
  extern __shared__ uint4 smem[];
  __shared__ float sums[WARPS][2][GL * 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const LanePlan q = lane_plan(p, lane < G * GL ? lane % GL : 32);
  const int grp = lane / GL, ca = q.ca * E, cb = q.cb * E;
  const uint32_t ring = smem_u32(smem) + threadIdx.x * 16;
  if (p.norm) {
    for (int i = lane; i < 2 * GL * 16; i += 32) (&sums[warp][0][0])[i] = 0.0f;
    __syncwarp();
  }
  float2 sum[8], g[8];  // dγ, γ of the lane's columns (γ = 0 on a lane without)
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = both(0.0f);
  int kind = -1;        // whose
  auto store_sums = [&]() {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // over the warp's lane groups, in their order
      float2 v = sum[k];
#pragma unroll
      for (int o = 1; o < G; ++o) {
        const int from = min(lane + o * GL, 31);
        v.x += __shfl_sync(0xffffffffu, sum[k].x, from);
        v.y += __shfl_sync(0xffffffffu, sum[k].y, from);
      }
      if (lane < GL && q.live) *reinterpret_cast<float2*>(&sums[warp][kind][k < 4 ? q.ca + 2 * k : q.cb + 2 * (k - 4)]) = v;
    }
  };
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * WARPS + warp;
  const uint64_t warps = static_cast<uint64_t>(gridDim.x) * WARPS;
  Cursor<G * U> at, ahead;
  const unsigned n = at.begin(p, w, warps);
  ahead = at;
  auto fetch = [&](unsigned i) {
    if (i < n) {
      const uint32_t st = ring + (i % STAGES) * STAGE;
      const int count = ahead.count(p), j0 = static_cast<int>(ahead.batch) * G * U + grp;
      const uint8_t* dy = static_cast<const uint8_t*>(p.dy) + static_cast<int64_t>(ahead.row) * p.lddy * E;
      const uint8_t* x = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(ahead.row) * p.ldx * E;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int j = j0 + k * G;
        const bool on = j < count && q.live;
        const int col = on ? column_of(p, ahead.kind, j) * E : 0, a = on ? ca : 0, b = on ? cb : 0;
        V::fetch(st + k * PLACE, dy + col + a, on);
        V::fetch(st + k * PLACE + VEC, dy + col + b, on);
        if (p.norm && ahead.kind != VALUE) {
          V::fetch(st + k * PLACE + 2 * VEC, x + col + a, on);
          V::fetch(st + k * PLACE + 3 * VEC, x + col + b, on);
        }
      }
      ahead.next(p);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  Angles soon, t;
  if (p.rot > 0 && n > 0 && at.kind != VALUE) soon.load(p, q, position_of(p, at.row));
  bool fresh = true;  // `soon` holds the angles of the row to come
  for (unsigned i = 0; i < n; ++i) {
    fetch(i + STAGES - 1);
    if (fresh) t = soon;
    Cursor<G * U> next = at;
    next.next(p);
    fresh = next.row != at.row || next.kind != at.kind;
    if (p.rot > 0 && fresh && i + 1 < n && next.kind != VALUE) soon.load(p, q, position_of(p, next.row));
    if (p.norm && at.kind != VALUE && at.kind != kind) {
      if (kind >= 0) store_sums();
      kind = at.kind;
      if (q.live) {
        Vec8<DT> v;
        v.load(kind == QUERY ? p.gq : p.gk, q.ca);
        v.get(g);
        v.load(kind == QUERY ? p.gq : p.gk, q.cb);
        v.get(g + 4);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = both(0.0f);
    }
    cp_wait<STAGES - 1>();
    const uint32_t st = ring + (i % STAGES) * STAGE;
    const int count = at.count(p), j0 = static_cast<int>(at.batch) * G * U + grp;
    uint8_t* y = static_cast<uint8_t*>(p.y) + static_cast<int64_t>(at.row) * p.ldy * E;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const bool on = j0 + k * G < count && q.live;
      V va, vb;
      va.take(st + k * PLACE);
      vb.take(st + k * PLACE + VEC);
      if (at.kind != VALUE) {
        float2 a[8];  // dy, then dn = Rᵀ·dy, then dx
        va.get(a);
        vb.get(a + 4);
        if (p.rot > 0) {
          if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < 4 ? q.ra : q.rb)
                a[e] = fma2(swap2(a[e]), make_float2(t.sine(e), -t.sine(e)), mul2(a[e], both(t.cosine(e))));
          } else if (q.ra) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 x = a[e], y = a[4 + e];
              const float2 c = make_float2(t.cosine(2 * e), t.cosine(2 * e + 1));
              const float2 s = make_float2(t.sine(2 * e), t.sine(2 * e + 1));
              a[e] = fma2(y, s, mul2(x, c));
              a[4 + e] = fma2(neg2(x), s, mul2(y, c));
            }
          }
        }
        if (p.norm) {
          float2 x[8];
          va.take(st + k * PLACE + 2 * VEC);
          vb.take(st + k * PLACE + 3 * VEC);
          va.get(x);
          vb.get(x + 4);
          float ss = squares(x, x + 4);
          float2 v = both(0.0f), prod[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            prod[e] = mul2(a[e], x[e]);
            a[e] = mul2(a[e], g[e]);
            v = fma2(a[e], x[e], v);
          }
          ss = group_sum<GL>(ss, lane);
          const float ts = group_sum<GL>(v.x + v.y, lane);
          const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
          const float2 rr = both(r), m = both(-ts * r * p.inv_d * r);  // −mean(t·x̂)·r: x̂ = r·x
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sum[e] = fma2(prod[e], rr, sum[e]);
            a[e] = mul2(fma2(x[e], m, a[e]), rr);
          }
        }
        va.set(a);
        vb.set(a + 4);
      }
      if (on) {
        uint8_t* e = y + column_of(p, at.kind, j0 + k * G) * E;
        va.store(e + ca);
        vb.store(e + cb);
      }
    }
    at = next;
  }
  if (!p.norm) return;
  if (kind >= 0) store_sums();
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.d; i += THREADS) {
    const int s = i / p.d, c = i - s * p.d;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += sums[k][s][c];
    p.part[static_cast<int64_t>(blockIdx.x) * 2 * p.d + i] = v;
  }
}

// dγ = Σ over the blocks' partial rows, 32 columns a CTA, 32 slices of the
// blocks side by side and the slices in order.
__global__ void __launch_bounds__(1024) qk_gamma_kernel(const float* __restrict__ part, int blocks, int d, float* dgq,
                                                        float* dgk) {
  __shared__ float s[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.0f;
  if (col < 2 * d)
    for (int i = slice; i < blocks; i += 32) v += __ldcg(part + static_cast<int64_t>(i) * 2 * d + col);
  s[slice][threadIdx.x & 31] = v;
  __syncthreads();
  if (slice == 0 && col < 2 * d) {
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s[k][threadIdx.x];
    if (col < d) dgq[col] = v;
    else dgk[col - d] = v;
  }
}

// ---------------------------------------------------------------- host
namespace {

size_t esize(int dtype) { return dtype == DT_F32 ? 4 : 2; }
int group_lanes(int d) { return d == 96 ? 6 : d <= 64 ? 4 : d <= 128 ? 8 : 16; }
constexpr int BWD_MAX_BLOCKS = 1024;

int check_shape(int64_t rows, int64_t b, int heads, int kv_heads, int d, int dtype) {
  if (rows < 0 || b < 1) return set_error(TPMLP_ERR_INVALID_ARG, "rows >= 0 and b >= 1 required");
  if (dtype < DT_F32 || dtype > DT_BF16) return set_error(TPMLP_ERR_INVALID_ARG, "unknown dtype");
  if (heads < 1 || kv_heads < 1 || kv_heads > heads)
    return set_error(TPMLP_ERR_INVALID_ARG, "heads >= 1 and kv_heads in [1, heads] required");
  if (heads % kv_heads != 0)
    return set_error(TPMLP_ERR_NOT_DIVISIBLE, "the number of heads must be divisible by the number of kv heads");
  if (d < 16 || d > 256 || d % 16 != 0)
    return set_error(TPMLP_ERR_UNSUPPORTED, "head width must be a multiple of 16 in [16, 256]");
  if (heads > 16384 || rows >= (1ll << 31) || b >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  return TPMLP_OK;
}

int check_ptr(const void* p, size_t align, const char* name) {
  if (p == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align != 0)
    return set_error(align >= 16 ? TPMLP_ERR_UNSUPPORTED : TPMLP_ERR_INVALID_ARG,
                     std::string(name) + " is not " + std::to_string(align) + "-byte aligned");
  return TPMLP_OK;
}

int check_ld(int64_t ld, int64_t w, size_t e, const char* name) {
  if (ld < w) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " is smaller than the row");
  if (ld * e % 16 != 0) return set_error(TPMLP_ERR_UNSUPPORTED, std::string(name) + " rows must be 16-byte aligned");
  return TPMLP_OK;
}

// The rope's own rules, and positions: `last` is the largest position that rows
// without a position array reach (−1: an array is required).
int check_rope(const tpmlp_qk_rope* r, int d, const void* positions, int pos_type, int64_t last, size_t e) {
  if (r == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, "rope is NULL");
  int rc;
  if ((r->q_gamma == nullptr) != (r->k_gamma == nullptr))
    return set_error(TPMLP_ERR_INVALID_ARG, "q_gamma and k_gamma must both be given or both be NULL");
  (void)e;
  if (r->q_gamma != nullptr) {
    if ((rc = check_ptr(r->q_gamma, 16, "q_gamma")) || (rc = check_ptr(r->k_gamma, 16, "k_gamma"))) return rc;
    if (!(r->eps >= 0.0f)) return set_error(TPMLP_ERR_INVALID_ARG, "eps must be >= 0");
  }
  if (r->interleaved != 0 && r->interleaved != 1) return set_error(TPMLP_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (r->rot < 0 || r->rot > d) return set_error(TPMLP_ERR_INVALID_ARG, "rot must be in [0, d]");
  if (r->rot % 16 != 0) return set_error(TPMLP_ERR_UNSUPPORTED, "rot must be a multiple of 16");
  if (pos_type != TPMLP_I32 && pos_type != TPMLP_I64) return set_error(TPMLP_ERR_INVALID_ARG, "unknown index type");
  if (r->rot > 0) {
    if ((rc = check_ptr(r->cos, 16, "cos")) || (rc = check_ptr(r->sin, 16, "sin"))) return rc;
    if (r->max_pos < 1) return set_error(TPMLP_ERR_INVALID_ARG, "max_pos must be >= 1");
    if (positions == nullptr) {
      if (last < 0) return set_error(TPMLP_ERR_INVALID_ARG, "positions is NULL");
      if (last >= r->max_pos) return set_error(TPMLP_ERR_INVALID_ARG, "the rotation tables are shorter than the sequence");
    }
  }
  if (positions != nullptr) return check_ptr(positions, pos_type == TPMLP_I64 ? 8 : 4, "positions");
  return TPMLP_OK;
}

Params base(const tpmlp_qk_rope* r, const void* positions, int pos_type, int64_t rows, int64_t b, int heads,
            int kv_heads, int d, const DeviceInfo* dev) {
  Params p{};
  p.gq = r->q_gamma;
  p.gk = r->k_gamma;
  p.norm = r->q_gamma != nullptr;
  p.eps = r->eps;
  p.inv_d = 1.0f / static_cast<float>(d);
  p.cos = r->cos;
  p.sin = r->sin;
  p.max_pos = r->max_pos;
  p.rot = r->rot;
  p.interleaved = r->interleaved;
  p.pos = positions;
  p.pos64 = pos_type == TPMLP_I64;
  p.rows = static_cast<unsigned>(rows);
  p.b = static_cast<unsigned>(b);
  p.r = static_cast<unsigned>(heads / kv_heads);
  p.r_magic = static_cast<unsigned>((1ull << 32) / p.r + 1);  // unused for r = 1
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.d = d;
  p.status = dev->status;
  return p;
}

int check_launch(const char* what, cudaError_t e = cudaSuccess) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  return TPMLP_OK;
}

// Items of `per` heads of each kind per row; values only where they move.
void set_items(Params& p, int per, bool values) {
  p.batches[QUERY] = static_cast<unsigned>((p.heads + per - 1) / per);
  p.batches[KEY] = static_cast<unsigned>((p.kv_heads + per - 1) / per);
  p.batches[VALUE] = values ? p.batches[KEY] : 0;
  p.qk_items = static_cast<uint64_t>(p.rows) * (p.batches[QUERY] + p.batches[KEY]);
  p.v_items = static_cast<uint64_t>(p.rows) * p.batches[VALUE];
}
// As many CTAs as there are warps with a query or key item, at most `most`.
unsigned grid_of(const Params& p, int most) {
  return static_cast<unsigned>(std::min<uint64_t>((p.qk_items + WARPS - 1) / WARPS, static_cast<uint64_t>(most)));
}

template <int DT, int GL, int U, bool APPEND>
cudaError_t launch_one(const Params& p, const DeviceInfo* dev, cudaStream_t st) {
  constexpr int smem = STAGES * U * 2 * Vec8<DT>::N * THREADS * 16;
  auto* fn = qk_forward_kernel<DT, GL, U, APPEND>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  fn<<<grid_of(p, FWD_CTAS * dev->num_sms), THREADS, smem, st>>>(p);
  return cudaGetLastError();
}

template <int DT, int GL, bool APPEND>
cudaError_t launch_forward(Params& p, bool values, const DeviceInfo* dev, cudaStream_t st) {
  constexpr int G = 32 / GL;
  // FWD_U heads a lane group amortise the angles; where that leaves warps without
  // an item, one head each spreads the work over the SMs instead.
  set_items(p, FWD_U * G, values);
  if (p.qk_items >= static_cast<uint64_t>(FWD_CTAS) * WARPS * dev->num_sms)
    return launch_one<DT, GL, FWD_U, APPEND>(p, dev, st);
  set_items(p, G, values);
  return launch_one<DT, GL, 1, APPEND>(p, dev, st);
}

template <int DT, bool APPEND>
cudaError_t launch_forward_dt(Params& p, bool values, const DeviceInfo* dev, cudaStream_t st) {
  const int gl = group_lanes(p.d);
  return gl == 4   ? launch_forward<DT, 4, APPEND>(p, values, dev, st)
         : gl == 6 ? launch_forward<DT, 6, APPEND>(p, values, dev, st)
         : gl == 8 ? launch_forward<DT, 8, APPEND>(p, values, dev, st)
                   : launch_forward<DT, 16, APPEND>(p, values, dev, st);
}

template <bool APPEND>
int forward(Params& p, bool values, int dtype, const DeviceInfo* dev, cudaStream_t st, const char* what) {
  const int ph = prof_begin(PROF_SP_REGION, st);
  const cudaError_t e = dtype == DT_F32   ? launch_forward_dt<DT_F32, APPEND>(p, values, dev, st)
                        : dtype == DT_F16 ? launch_forward_dt<DT_F16, APPEND>(p, values, dev, st)
                                          : launch_forward_dt<DT_BF16, APPEND>(p, values, dev, st);
  const int cols = (p.heads + (values ? 2 : 1) * p.kv_heads) * p.d;
  prof_end(ph, 2.0 * p.rows * cols * esize(dtype), st);
  return check_launch(what, e);
}

template <int DT, int GL>
cudaError_t launch_backward(const Params& p, unsigned grid, cudaStream_t st) {
  constexpr int smem = STAGES * BWD_U * 4 * Vec8<DT>::N * THREADS * 16;
  auto* fn = qk_backward_kernel<DT, GL, BWD_U>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  fn<<<grid, THREADS, smem, st>>>(p);
  return cudaGetLastError();
}
template <int DT>
cudaError_t launch_backward_dt(const Params& p, unsigned grid, cudaStream_t st) {
  const int gl = group_lanes(p.d);
  return gl == 4   ? launch_backward<DT, 4>(p, grid, st)
         : gl == 6 ? launch_backward<DT, 6>(p, grid, st)
         : gl == 8 ? launch_backward<DT, 8>(p, grid, st)
                   : launch_backward<DT, 16>(p, grid, st);
}

}  // namespace

// The forward and backward inside the attention block (attn.cu): row m of
// [s·b, W] at position m / b.
int check_block_rope(const tpmlp_qk_rope* rope, int64_t s, int64_t b, int heads, int kv_heads, int d, int dtype) {
  if (const int rc = check_shape(s * b, b, heads, kv_heads, d, dtype)) return rc;
  return check_rope(rope, d, nullptr, TPMLP_I32, s > 0 ? s - 1 : 0, esize(dtype));
}

}  // namespace qkrope
}  // namespace tpmlp

using namespace tpmlp;
using namespace tpmlp::qkrope;

extern "C" {

int tpmlp_qk_norm_rope_forward(const void* qkv, int64_t ld_qkv, void* out, int64_t ld_out, const tpmlp_qk_rope* rope,
                               const void* positions, int pos_type, int64_t rows, int64_t b, int heads, int kv_heads,
                               int d, int dtype, void* stream) {
  int rc = check_shape(rows, b, heads, kv_heads, d, dtype);
  if (rc) return rc;
  const size_t e = esize(dtype);
  const int64_t W = static_cast<int64_t>(heads + 2 * kv_heads) * d;
  if ((rc = check_ptr(qkv, 16, "qkv")) || (rc = check_ptr(out, 16, "out")) || (rc = check_ld(ld_qkv, W, e, "ld_qkv")) ||
      (rc = check_ld(ld_out, W, e, "ld_out")) ||
      (rc = check_rope(rope, d, positions, pos_type, rows > 0 ? (rows - 1) / b : 0, e)))
    return rc;
  if (qkv == out && ld_qkv != ld_out)
    return set_error(TPMLP_ERR_INVALID_ARG, "in place, ld_qkv and ld_out must be equal");
  if (rows == 0) return TPMLP_OK;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  Params p = base(rope, positions, pos_type, rows, b, heads, kv_heads, d, dev);
  p.x = qkv;
  p.y = out;
  p.ldx = ld_qkv;
  p.ldy = ld_out;
  return forward<false>(p, /*values=*/qkv != out, dtype, dev, static_cast<cudaStream_t>(stream), "QK norm and rotation");
}

int tpmlp_qk_norm_rope_append(const void* qkv, int64_t ld_qkv, void* q, int64_t ld_q, const tpmlp_kv_cache* cache,
                              const int64_t* slots, const tpmlp_qk_rope* rope, const void* positions, int pos_type,
                              int64_t rows, int heads, int kv_heads, int d, int dtype, void* stream) {
  int rc = check_shape(rows, 1, heads, kv_heads, d, dtype);
  if (rc) return rc;
  const size_t e = esize(dtype);
  const int64_t W = static_cast<int64_t>(heads + 2 * kv_heads) * d;
  if ((rc = check_ptr(qkv, 16, "qkv")) || (rc = check_ptr(q, 16, "q")) || (rc = check_ld(ld_qkv, W, e, "ld_qkv")) ||
      (rc = check_ld(ld_q, static_cast<int64_t>(heads) * d, e, "ld_q")) || (rc = check_ptr(slots, 8, "slots")) ||
      (rc = check_rope(rope, d, positions, pos_type, -1, e)) || (rc = check_kv_cache(cache, kv_heads, d, dtype)))
    return rc;
  if (rows == 0) return TPMLP_OK;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  Params p = base(rope, positions, pos_type, rows, 1, heads, kv_heads, d, dev);
  p.x = qkv;
  p.y = q;
  p.ldx = ld_qkv;
  p.ldy = ld_q;
  p.kc = cache->k;
  p.vc = cache->v;
  p.slots = slots;
  p.pages = cache->pages;
  p.page_size = cache->page_size;
  p.page_stride = cache->page_stride;
  p.token_stride = cache->token_stride;
  p.head_stride = cache->head_stride;
  return forward<true>(p, /*values=*/true, dtype, dev, static_cast<cudaStream_t>(stream), "QK norm, rotation and cache append");
}

size_t tpmlp_qk_norm_rope_backward_workspace(int64_t rows, int heads, int kv_heads, int d) {
  if (check_shape(rows, 1, heads, kv_heads, d, DT_BF16) != TPMLP_OK || rows == 0) return 0;
  return static_cast<size_t>(BWD_MAX_BLOCKS) * 2 * d * sizeof(float);
}

int tpmlp_qk_norm_rope_backward(const void* qkv, int64_t ld_qkv, const void* dout, int64_t ld_dout, void* dqkv,
                                int64_t ld_dqkv, float* dq_gamma, float* dk_gamma, const tpmlp_qk_rope* rope,
                                const void* positions, int pos_type, int64_t rows, int64_t b, int heads, int kv_heads,
                                int d, int dtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_shape(rows, b, heads, kv_heads, d, dtype);
  if (rc) return rc;
  const size_t e = esize(dtype);
  const int64_t W = static_cast<int64_t>(heads + 2 * kv_heads) * d;
  if ((rc = check_rope(rope, d, positions, pos_type, rows > 0 ? (rows - 1) / b : 0, e)) ||
      (rc = check_ptr(dout, 16, "dout")) || (rc = check_ptr(dqkv, 16, "dqkv")) ||
      (rc = check_ld(ld_dout, W, e, "ld_dout")) || (rc = check_ld(ld_dqkv, W, e, "ld_dqkv")))
    return rc;
  const bool norm = rope->q_gamma != nullptr;
  const size_t need = norm ? tpmlp_qk_norm_rope_backward_workspace(rows, heads, kv_heads, d) : 0;
  if (norm) {
    if ((rc = check_ptr(qkv, 16, "qkv")) || (rc = check_ld(ld_qkv, W, e, "ld_qkv")) ||
        (rc = check_ptr(dq_gamma, 4, "dq_gamma")) || (rc = check_ptr(dk_gamma, 4, "dk_gamma")))
      return rc;
    if (need > 0) {
      if (ws == nullptr || ws_bytes < need)
        return set_error(TPMLP_ERR_WORKSPACE, "QK norm backward workspace needs " + std::to_string(need) + " bytes");
      if ((rc = check_ptr(ws, 16, "ws"))) return rc;
    }
  }
  if (dout == dqkv && ld_dout != ld_dqkv)
    return set_error(TPMLP_ERR_INVALID_ARG, "in place, ld_dout and ld_dqkv must be equal");
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (!norm) return TPMLP_OK;
    cudaError_t er = cudaMemsetAsync(dq_gamma, 0, d * sizeof(float), st);
    if (er == cudaSuccess) er = cudaMemsetAsync(dk_gamma, 0, d * sizeof(float), st);
    return check_launch("QK norm backward", er);
  }
  Params p = base(rope, positions, pos_type, rows, b, heads, kv_heads, d, dev);
  p.x = qkv;
  p.ldx = ld_qkv;
  p.dy = dout;
  p.lddy = ld_dout;
  p.y = dqkv;
  p.ldy = ld_dqkv;
  p.part = static_cast<float*>(ws);
  const bool values = dout != dqkv;
  const int gl = group_lanes(d);
  set_items(p, 32 / gl * BWD_U, values);
  const unsigned blocks = grid_of(p, std::min(BWD_CTAS * dev->num_sms, BWD_MAX_BLOCKS));
  const int ph = prof_begin(PROF_SP_REGION, st);
  cudaError_t er = dtype == DT_F32   ? launch_backward_dt<DT_F32>(p, blocks, st)
                   : dtype == DT_F16 ? launch_backward_dt<DT_F16>(p, blocks, st)
                                     : launch_backward_dt<DT_BF16>(p, blocks, st);
  if (er == cudaSuccess && norm) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((2 * d + 31) / 32), 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    er = cudaLaunchKernelEx(&cfg, qk_gamma_kernel, static_cast<const float*>(p.part), static_cast<int>(blocks), d, dq_gamma, dk_gamma);
  }
  const int qk = (heads + kv_heads) * d, cols = qk + (values ? kv_heads * d : 0);
  prof_end(ph, static_cast<double>(rows) * (2.0 * cols + (norm ? qk : 0)) * e, st, norm ? 2 : 1);
  return check_launch("QK norm and rotation backward", er);
}

}  // extern "C"
