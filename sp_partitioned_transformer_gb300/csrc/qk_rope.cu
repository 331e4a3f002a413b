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
//   no lane waits for another; the forward reads a row's angles when it comes to the
//   row (64 heads of 96: 55.3 µs, 56.1 with the angles fetched an item ahead: the
//   registers cost more than the wait);
// * γ and the angles of an item are combined once and serve all its heads, and
//   the arithmetic runs on float32 pairs.
#include <algorithm>
#include <string>

#include "internal.h"

namespace tpmlp {
namespace qkrope {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int FWD_STAGES = 4;  // items in flight or in work, of every warp
constexpr int BWD_STAGES = 3;
constexpr int FWD_U = 2;     // heads a lane group takes of an item
constexpr int BWD_U = 2;
constexpr int FWD_CTAS = 3;  // per SM
constexpr int BWD_CTAS = 3;

// The heads of an item are all of one kind, so that γ and the angles are
// combined once for all of them.
enum Kind { QUERY = 0, KEY = 1, VALUE = 2 };

struct Params {
  const void* x;   // [rows, ldx]
  void* y;         // [rows, ldy]: the rotated QKV, or (append) q only
  unsigned ldx, ldy;  // row strides in bytes
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
  unsigned batches[2];  // items per row of queries, and of keys and of values
  int values;           // v moves (not in place)
  unsigned* status;
  // append
  void* kc;
  void* vc;
  const int64_t* slots;
  int64_t pages, page_size;
  int64_t page_stride, token_stride, head_stride;
  // backward
  const void* dy;
  unsigned lddy;
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

// `real` false: nothing is read and zeros are written.  HALF: L2 fetches half lines,
// for heads of 96, whose rows whole 128-byte lines do not divide (the rest of a
// line is another kind of head, read at another time: 61.4 against 63.9 µs at 64
// heads of 96).
template <bool HALF>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;
  if constexpr (HALF) asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
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
    for (int i = 0; i < N; ++i) r[i] = p[i];
  }
  // To and from this lane's place in the ring (a shared address): units THREADS apart.
  template <bool HALF>
  static __device__ __forceinline__ void fetch(uint32_t ring, const uint8_t* p, bool real) {
#pragma unroll
    for (int i = 0; i < N; ++i) cp_async16<HALF>(ring + i * THREADS * 16, p + i * 16, real);
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
      const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DT_BF16) {
          v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
          __half2 h;
          memcpy(&h, &w[i], 4);
          v[i] = __half22float2(h);
        }
      }
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
    q.ca = r ? l * 8 : p.rot + (l - half) * 8;
    q.cb = q.ca + (r ? p.rot : p.d - p.rot) / 2;  // neighbouring lanes hold neighbouring vectors
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
      c[0] = *reinterpret_cast<const float4*>(p.cos + a);
      s[0] = *reinterpret_cast<const float4*>(p.sin + a);
    }
    if (q.rb) {
      c[1] = *reinterpret_cast<const float4*>(p.cos + b);
      s[1] = *reinterpret_cast<const float4*>(p.sin + b);
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

// The place of a warp in its items: a row, a kind and a batch of PER heads of that
// kind in the row, in this order of significance (queries, keys and values of a
// row lie side by side in memory: taking them at different times costs DRAM
// efficiency).  Head j of a kind begins at unit a·j + 2·⌊j·m / 2³²⌋ + c of the
// row, in heads: a query head has two more heads (its group's key and value)
// behind every r of its kind.
template <int PER>
struct Cursor {
  int kind, count;
  unsigned row, batch, batches;
  int a, c;
  unsigned m;
  // Places the cursor at the warp's first item; the number of its items.
  __device__ __forceinline__ unsigned begin(const Params& p, uint64_t w, uint64_t warps) {
    const unsigned per_row = p.batches[QUERY] + 2 * p.batches[KEY];
    const uint64_t items = static_cast<uint64_t>(p.rows) * per_row, at = items * w / warps;
    const unsigned n = static_cast<unsigned>(items * (w + 1) / warps - at);
    row = static_cast<unsigned>(at / per_row);
    batch = static_cast<unsigned>(at - static_cast<uint64_t>(row) * per_row);
    set(p, QUERY);
    if (batch >= batches) {
      batch -= batches;
      set(p, KEY);
      if (batch >= batches) {
        batch -= batches;
        set(p, VALUE);
      }
    }
    return n;
  }
  __device__ __forceinline__ void set(const Params& p, int k) {
    const int r = static_cast<int>(p.r);
    const bool query = k == QUERY;
    kind = k;
    count = query ? p.heads : p.kv_heads;
    batches = query ? p.batches[QUERY] : p.batches[KEY];
    a = query ? (r == 1 ? 3 : 1) : r + 2;
    m = query && r > 1 ? p.r_magic : 0u;
    c = query ? 0 : r + k - 1;
  }
  __device__ __forceinline__ void next(const Params& p) {
    if (++batch < batches) return;
    batch = 0;
    row += kind == VALUE;
    set(p, kind == VALUE ? QUERY : kind + 1);
  }
  __device__ __forceinline__ int unit(int j) const { return a * j + 2 * static_cast<int>(__umulhi(j, m)) + c; }
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

// 16 bytes to global memory where `on`.
__device__ __forceinline__ void store16(uint8_t* p, const uint4& v, bool on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q st.global.v4.u32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(p), "r"(v.x),
      "r"(v.y), "r"(v.z), "r"(v.w), "r"(static_cast<unsigned>(on))
      : "memory");
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

// APPEND: q goes to y, k and v to the cache.
template <int DT, int GL, int U, bool APPEND>
__global__ void __launch_bounds__(THREADS, FWD_CTAS) qk_forward_kernel(const __grid_constant__ Params p) {
  using V = Vec8<DT>;
  constexpr int G = 32 / GL, E = V::E, VEC = V::N * THREADS * 16, STAGE = U * 2 * VEC, STAGES = FWD_STAGES;
  extern __shared__ uint4 smem[];
  pdl_go();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const LanePlan q = lane_plan(p, lane < G * GL ? lane % GL : 32);
  const int grp = q.live ? lane / GL : 1 << 20;  // no head for a lane without columns
  const int ca = q.ca * E, ba = (q.cb - q.ca) * E, head_bytes = p.d * E;
  const uint32_t ring = smem_u32(smem) + threadIdx.x * 16;
  Cursor<G * U> at, ahead;
  const unsigned n = at.begin(p, static_cast<uint64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5),
                              static_cast<uint64_t>(gridDim.x) * WARPS);
  ahead = at;
  uint32_t fill = 0, use = 0;  // stages that the next copies go to, and the item in work lies in
  const uint8_t* const src = static_cast<const uint8_t*>(p.x) + ca;
  auto fetch = [&](unsigned i) {
    if (i < n) {
      const bool moves = ahead.kind != VALUE || p.values;
      const uint8_t* x = src + static_cast<uint64_t>(ahead.row) * p.ldx;
      int j = static_cast<int>(ahead.batch) * G * U + grp;
#pragma unroll
      for (int k = 0; k < U; ++k, j += G) {
        const bool on = j < ahead.count && moves;
        const uint8_t* c = x + ahead.unit(j) * head_bytes;
        V::template fetch<GL == 6>(ring + fill + k * 2 * VEC, c, on);
        V::template fetch<GL == 6>(ring + fill + k * 2 * VEC + VEC, c + ba, on);
      }
      ahead.next(p);
      fill = fill < (STAGES - 1) * STAGE ? fill + STAGE : 0;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  Combined c;
  bool fresh = true;  // c is not yet this row's and kind's
  for (unsigned i = 0; i < n; ++i) {
    fetch(i + STAGES - 1);
    const int kind = at.kind;
    if (fresh && kind != VALUE) {
      Angles t;
      if (p.rot > 0) t.load(p, q, position_of(p, at.row));
      c.make<DT>(p, q, kind, t);
    }
    uint8_t* y = static_cast<uint8_t*>(p.y) + static_cast<uint64_t>(at.row) * p.ldy + ca;
    int j = static_cast<int>(at.batch) * G * U + grp;
    bool on[U];
    uint8_t* d[U];
#pragma unroll
    for (int k = 0; k < U; ++k, j += G) {
      on[k] = j < at.count && (kind != VALUE || p.values);
      if constexpr (!APPEND) d[k] = y + at.unit(j) * head_bytes;
      else d[k] = y + j * head_bytes;
    }
    if constexpr (APPEND) {
      if (kind != QUERY) {
        const int64_t row = cache_row_of(p, at.row);
        uint8_t* b = static_cast<uint8_t*>(kind == KEY ? p.kc : p.vc) + row * E + ca;
        j = static_cast<int>(at.batch) * G * U + grp;
#pragma unroll
        for (int k = 0; k < U; ++k, j += G) {
          on[k] = on[k] && row >= 0;
          d[k] = b + j * p.head_stride * E;
        }
      }
    }
    at.next(p);
    fresh = at.kind != kind || at.batch == 0;
    cp_wait<STAGES - 1>();
    V va[U], vb[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      va[k].take(ring + use + k * 2 * VEC);
      vb[k].take(ring + use + k * 2 * VEC + VEC);
    }
    use = use < (STAGES - 1) * STAGE ? use + STAGE : 0;
    if (kind == VALUE) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          store16(d[k] + e * 16, va[k].r[e], on[k]);
          store16(d[k] + ba + e * 16, vb[k].r[e], on[k]);
        }
      }
      continue;
    }
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
    } else {
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = x[k][e], b = x[k][4 + e];
          float2 s = mul2(a, c.u[e]), t = mul2(b, c.u[4 + e]);
          if (q.ra) {
            s = fma2(b, c.v[e], s);
            t = fma2(a, c.v[4 + e], t);
          }
          x[k][e] = mul2(s, both(r[k]));
          x[k][4 + e] = mul2(t, both(r[k]));
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      va[k].set(x[k]);
      vb[k].set(x[k] + 4);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        store16(d[k] + e * 16, va[k].r[e], on[k]);
        store16(d[k] + ba + e * 16, vb[k].r[e], on[k]);
      }
    }
  }
}

// ---------------------------------------------------------------- backward
// A lane sums dγ of its 16 columns in registers, and adds that to a place of its
// own in shared memory when the warp passes to another kind of head; the lanes'
// sums are added over the block at the end, and over the blocks, in block order,
// by qk_gamma_kernel.
template <int DT, int GL, int U>
__global__ void __launch_bounds__(THREADS, BWD_CTAS) qk_backward_kernel(const __grid_constant__ Params p) {
  using V = Vec8<DT>;
  constexpr int G = 32 / GL, E = V::E, VEC = V::N * THREADS * 16, PLACE = 4 * VEC, STAGE = U * PLACE, STAGES = BWD_STAGES;
  extern __shared__ uint4 smem[];
  __shared__ float2 sums[2][8][THREADS];  // [queries, keys][pair of columns]
  pdl_go();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const LanePlan q = lane_plan(p, lane < G * GL ? lane % GL : 32);
  const int grp = q.live ? lane / GL : 1 << 20;  // no head for a lane without columns
  const int ca = q.ca * E, ba = (q.cb - q.ca) * E, head_bytes = p.d * E;
  const uint32_t ring = smem_u32(smem) + threadIdx.x * 16;
  float2 sum[8], g[8];  // dγ, γ of the lane's columns (γ = 0 on a lane without)
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    g[k] = sum[k] = both(0.0f);
    sums[0][k][threadIdx.x] = sums[1][k][threadIdx.x] = sum[k];
  }
  int kind = -1;  // whose
  auto store_sums = [&]() {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float2& s = sums[kind][k][threadIdx.x];
      s = make_float2(s.x + sum[k].x, s.y + sum[k].y);
      sum[k] = both(0.0f);
    }
  };
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * WARPS + warp;
  const uint64_t warps = static_cast<uint64_t>(gridDim.x) * WARPS;
  Cursor<G * U> at, ahead;
  const unsigned n = at.begin(p, w, warps);
  ahead = at;
  uint32_t fill = 0, use = 0;  // stages that the next copies go to, and the item in work lies in
  auto fetch = [&](unsigned i) {
    if (i < n) {
      const uint8_t* dy = static_cast<const uint8_t*>(p.dy) + static_cast<uint64_t>(ahead.row) * p.lddy + ca;
      const uint8_t* x = static_cast<const uint8_t*>(p.x) + static_cast<uint64_t>(ahead.row) * p.ldx + ca;
      const bool moves = ahead.kind != VALUE || p.values;
      int j = static_cast<int>(ahead.batch) * G * U + grp;
#pragma unroll
      for (int k = 0; k < U; ++k, j += G) {
        const bool on = j < ahead.count && moves;
        const int col = ahead.unit(j) * head_bytes;
        V::template fetch<GL == 6>(ring + fill + k * PLACE, dy + col, on);
        V::template fetch<GL == 6>(ring + fill + k * PLACE + VEC, dy + col + ba, on);
        if (p.norm && ahead.kind != VALUE) {
          V::template fetch<GL == 6>(ring + fill + k * PLACE + 2 * VEC, x + col, on);
          V::template fetch<GL == 6>(ring + fill + k * PLACE + 3 * VEC, x + col + ba, on);
        }
      }
      ahead.next(p);
      fill = fill < (STAGES - 1) * STAGE ? fill + STAGE : 0;
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
    uint8_t* y = static_cast<uint8_t*>(p.y) + static_cast<uint64_t>(at.row) * p.ldy + ca;
    int j = static_cast<int>(at.batch) * G * U + grp;
    bool on[U];
    uint8_t* dst[U];
#pragma unroll
    for (int k = 0; k < U; ++k, j += G) {
      on[k] = j < at.count && (at.kind != VALUE || p.values);
      dst[k] = y + at.unit(j) * head_bytes;
    }
    const int now = at.kind;
    if (p.norm && now != VALUE && now != kind) {
      if (kind >= 0) store_sums();
      kind = now;
      if (q.live) {
        V v;
        v.load(kind == QUERY ? p.gq : p.gk, q.ca);
        v.get(g);
        v.load(kind == QUERY ? p.gq : p.gk, q.cb);
        v.get(g + 4);
      }
    }
    at.next(p);
    fresh = at.kind == QUERY && at.batch == 0;
    if (p.rot > 0 && fresh && i + 1 < n) soon.load(p, q, position_of(p, at.row));
    cp_wait<STAGES - 1>();
#pragma unroll
    for (int k = 0; k < U; ++k) {
      V va, vb;
      const uint32_t st = ring + use + k * PLACE;
      va.take(st);
      vb.take(st + VEC);
      if (now == VALUE) {
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          store16(dst[k] + e * 16, va.r[e], on[k]);
          store16(dst[k] + ba + e * 16, vb.r[e], on[k]);
        }
        continue;
      }
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
            const float2 x = a[e], y2 = a[4 + e];
            const float2 c = make_float2(t.cosine(2 * e), t.cosine(2 * e + 1));
            const float2 s = make_float2(t.sine(2 * e), t.sine(2 * e + 1));
            a[e] = fma2(y2, s, mul2(x, c));
            a[4 + e] = fma2(x, neg2(s), mul2(y2, c));
          }
        }
      }
      if (p.norm) {
        float2 x[8], prod[8];
        va.take(st + 2 * VEC);
        vb.take(st + 3 * VEC);
        va.get(x);
        vb.get(x + 4);
        float2 v = both(0.0f), v2 = both(0.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          prod[e] = mul2(a[e], x[e]);
          a[e] = mul2(a[e], g[e]);
          if (e < 4) v = fma2(a[e], x[e], v);
          else v2 = fma2(a[e], x[e], v2);
        }
        const float ss = group_sum<GL>(squares(x, x + 4), lane);
        const float ts = group_sum<GL>((v.x + v2.x) + (v.y + v2.y), lane);
        // a place without a head holds zeros: with eps = 0 its root would make NaN of its nothing in dγ
        const float r = on[k] ? rsqrtf(fmaf(ss, p.inv_d, p.eps)) : 0.0f;
        const float2 rr = both(r), m = both(-ts * r * p.inv_d * r);  // −mean(t·x̂)·r: x̂ = r·x
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum[e] = fma2(prod[e], rr, sum[e]);
          a[e] = mul2(fma2(x[e], m, a[e]), rr);
        }
      }
      va.set(a);
      vb.set(a + 4);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        store16(dst[k] + e * 16, va.r[e], on[k]);
        store16(dst[k] + ba + e * 16, vb.r[e], on[k]);
      }
    }
    use = use < (STAGES - 1) * STAGE ? use + STAGE : 0;
  }
  if (!p.norm) return;
  if (kind >= 0) store_sums();
  __syncthreads();
  // Column c of γ_q or γ_k: the pair k of the lane that holds it, over the lane
  // groups of every warp.
  for (int i = threadIdx.x; i < 2 * p.d; i += THREADS) {
    const int s = i / p.d, col = i - s * p.d;
    int l = 0, k = 0;
    for (int o = 0; o < p.d / 16; ++o) {
      const LanePlan w = lane_plan(p, o);
      if (col >= w.ca && col < w.ca + 8) l = o, k = col - w.ca;
      if (col >= w.cb && col < w.cb + 8) l = o, k = 8 + col - w.cb;
    }
    float v = 0.0f;
    for (int t = 0; t < WARPS; ++t)
      for (int o = 0; o < G; ++o) v += reinterpret_cast<const float*>(&sums[s][k / 2][t * 32 + o * GL + l])[k & 1];
    p.part[static_cast<int64_t>(blockIdx.x) * 2 * p.d + i] = v;
  }
}

// dγ = Σ over the blocks' partial rows, 32 columns a CTA, 32 slices of the
// blocks side by side and the slices in order.
__global__ void __launch_bounds__(1024) qk_gamma_kernel(const float* part, int blocks, int d, float* dgq,
                                                        float* dgk) {
  __shared__ float s[32][33];
  pdl_go();
  pdl_wait();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.0f;
  if (col < 2 * d) {
    for (int i0 = slice; i0 < blocks; i0 += 32 * 16) {  // 16 loads in flight
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k)
        x[k] = i0 + 32 * k < blocks ? __ldcg(part + static_cast<int64_t>(i0 + 32 * k) * 2 * d + col) : 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) v += x[k];
    }
  }
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
  if (ld >= (1ll << 29)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  if (ld * e % 16 != 0) return set_error(TPMLP_ERR_UNSUPPORTED, std::string(name) + " rows must be 16-byte aligned");
  return TPMLP_OK;
}

// The rope's own rules, and positions: `last` is the largest position that rows
// without a position array reach (−1: an array is required).
int check_rope(const tpmlp_qk_rope* r, int d, const void* positions, int pos_type, int64_t last) {
  if (r == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, "rope is NULL");
  int rc;
  if ((r->q_gamma == nullptr) != (r->k_gamma == nullptr))
    return set_error(TPMLP_ERR_INVALID_ARG, "q_gamma and k_gamma must both be given or both be NULL");
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

// Whether rows of wa bytes, lda apart from a on, and rows of wb bytes, ldb apart from
// b on, share a byte.  Row i of a and row j of b do when −wb < x < wa for their
// distance x = b + j·ldb − (a + i·lda).
bool rows_overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int64_t rows) {
  const int64_t x0 = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  if (x0 >= (rows - 1) * lda + wa || x0 <= -((rows - 1) * ldb + wb)) return false;
  // the first j >= from with x + j·ldb > −wb
  auto first = [&](int64_t x, int64_t from) {
    const int64_t t = -wb - x;
    return std::max(from, t >= 0 ? t / ldb + 1 : -((-t + ldb - 1) / ldb) + 1);
  };
  if (lda == ldb) {  // j − i alone decides
    const int64_t k = first(x0, 1 - rows);
    return k < rows && x0 + k * ldb < wa;
  }
  for (int64_t i = 0; i < rows; ++i) {
    const int64_t x = x0 - i * lda, j = first(x, 0);
    if (j < rows && x + j * ldb < wa) return true;
  }
  return false;
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

// Items of `per` heads of each kind per row; how many in all.
uint64_t set_items(Params& p, int per) {
  p.batches[QUERY] = static_cast<unsigned>((p.heads + per - 1) / per);
  p.batches[KEY] = static_cast<unsigned>((p.kv_heads + per - 1) / per);
  return static_cast<uint64_t>(p.rows) * (p.batches[QUERY] + 2 * p.batches[KEY]);
}
// As many CTAs as there are warps with an item, at most `most`.
unsigned grid_of(uint64_t items, int most) {
  return static_cast<unsigned>(std::min<uint64_t>((items + WARPS - 1) / WARPS, static_cast<uint64_t>(most)));
}

template <int DT, int GL, int U, bool APPEND>
cudaError_t launch_one(const Params& p, uint64_t items, const DeviceInfo* dev, cudaStream_t st) {
  constexpr int smem = FWD_STAGES * U * 2 * Vec8<DT>::N * THREADS * 16;
  auto* fn = qk_forward_kernel<DT, GL, U, APPEND>;
  if (smem > 48 * 1024) {
    static SmemDone done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem, *dev, &done);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(fn, dim3(grid_of(items, FWD_CTAS * dev->num_sms)), THREADS, smem, st, 1, p);
}

template <int DT, int GL, bool APPEND>
cudaError_t launch_forward(Params& p, const DeviceInfo* dev, cudaStream_t st) {
  constexpr int G = 32 / GL;
  // FWD_U heads a lane group amortise the angles; where that leaves warps without
  // an item, one head each spreads the work over the SMs instead.
  uint64_t items = set_items(p, FWD_U * G);
  if (items >= static_cast<uint64_t>(FWD_CTAS) * WARPS * dev->num_sms)
    return launch_one<DT, GL, FWD_U, APPEND>(p, items, dev, st);
  items = set_items(p, G);
  return launch_one<DT, GL, 1, APPEND>(p, items, dev, st);
}

template <int DT, bool APPEND>
cudaError_t launch_forward_dt(Params& p, const DeviceInfo* dev, cudaStream_t st) {
  const int gl = group_lanes(p.d);
  return gl == 4   ? launch_forward<DT, 4, APPEND>(p, dev, st)
         : gl == 6 ? launch_forward<DT, 6, APPEND>(p, dev, st)
         : gl == 8 ? launch_forward<DT, 8, APPEND>(p, dev, st)
                   : launch_forward<DT, 16, APPEND>(p, dev, st);
}

template <bool APPEND>
int forward(Params& p, bool values, int dtype, const DeviceInfo* dev, cudaStream_t st, const char* what) {
  p.values = values;
  const int ph = prof_begin(PROF_SP_REGION, st);
  const cudaError_t e = dtype == DT_F32   ? launch_forward_dt<DT_F32, APPEND>(p, dev, st)
                        : dtype == DT_F16 ? launch_forward_dt<DT_F16, APPEND>(p, dev, st)
                                          : launch_forward_dt<DT_BF16, APPEND>(p, dev, st);
  const int cols = (p.heads + (values ? 2 : 1) * p.kv_heads) * p.d;
  prof_end(ph, 2.0 * p.rows * cols * esize(dtype), st);
  return check_launch(what, e);
}

template <int DT, int GL>
cudaError_t launch_backward(const Params& p, unsigned grid, const DeviceInfo* dev, cudaStream_t st) {
  constexpr int smem = BWD_STAGES * BWD_U * 4 * Vec8<DT>::N * THREADS * 16;
  auto* fn = qk_backward_kernel<DT, GL, BWD_U>;
  static SmemDone done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem, *dev, &done);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, dim3(grid), THREADS, smem, st, 1, p);
}
template <int DT>
cudaError_t launch_backward_dt(const Params& p, unsigned grid, const DeviceInfo* dev, cudaStream_t st) {
  const int gl = group_lanes(p.d);
  return gl == 4   ? launch_backward<DT, 4>(p, grid, dev, st)
         : gl == 6 ? launch_backward<DT, 6>(p, grid, dev, st)
         : gl == 8 ? launch_backward<DT, 8>(p, grid, dev, st)
                   : launch_backward<DT, 16>(p, grid, dev, st);
}

}  // namespace

// Refuses an output whose rows share memory with an input's (row strides and
// widths in elements).
int check_apart(const void* in, int64_t ld_in, int64_t w_in, const void* out, int64_t ld_out, int64_t w_out, int64_t rows,
                int dtype, const char* what) {
  const int64_t e = static_cast<int64_t>(esize(dtype));
  if (rows > 0 && rows_overlap(in, ld_in * e, w_in * e, out, ld_out * e, w_out * e, rows))
    return set_error(TPMLP_ERR_INVALID_ARG, std::string(what) + " must not overlap");
  return TPMLP_OK;
}

// The forward and backward inside the attention block (attn.cu): row m of
// [s·b, W] at position m / b.
int check_block_rope(const tpmlp_qk_rope* rope, int64_t s, int64_t b, int heads, int kv_heads, int d, int dtype) {
  if (const int rc = check_shape(s * b, b, heads, kv_heads, d, dtype)) return rc;
  return check_rope(rope, d, nullptr, TPMLP_I32, s > 0 ? s - 1 : 0);
}

int check_append(const void* qkv, int64_t ld_qkv, const void* q, int64_t ld_q, const tpmlp_kv_cache* cache,
                 const int64_t* slots, const tpmlp_qk_rope* rope, const void* positions, int pos_type, int64_t rows,
                 int heads, int kv_heads, int d, int dtype) {
  int rc = check_shape(rows, 1, heads, kv_heads, d, dtype);
  if (rc) return rc;
  const size_t e = esize(dtype);
  const int64_t W = static_cast<int64_t>(heads + 2 * kv_heads) * d;
  if (rows > 0 && ((rc = check_ptr(qkv, 16, "qkv")) || (rc = check_ptr(q, 16, "q")) || (rc = check_ptr(slots, 8, "slots"))))
    return rc;
  if ((rc = check_ld(ld_qkv, W, e, "ld_qkv")) || (rc = check_ld(ld_q, static_cast<int64_t>(heads) * d, e, "ld_q")) ||
      (rc = check_rope(rope, d, positions, pos_type, rows > 0 ? -1 : 0)))
    return rc;
  if ((rc = check_kv_cache(cache, kv_heads, d, dtype))) return rc;
  return check_apart(qkv, ld_qkv, W, q, ld_q, static_cast<int64_t>(heads) * d, rows, dtype, "qkv and q");
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
  if ((rc = check_ld(ld_qkv, W, e, "ld_qkv")) || (rc = check_ld(ld_out, W, e, "ld_out")) ||
      (rc = check_rope(rope, d, positions, pos_type, rows > 0 ? (rows - 1) / b : 0)))
    return rc;
  if (rows == 0) return TPMLP_OK;
  if ((rc = check_ptr(qkv, 16, "qkv")) || (rc = check_ptr(out, 16, "out"))) return rc;
  if (qkv == out && ld_qkv != ld_out)
    return set_error(TPMLP_ERR_INVALID_ARG, "in place, ld_qkv and ld_out must be equal");
  if (qkv != out && (rc = check_apart(qkv, ld_qkv, W, out, ld_out, W, rows, dtype, "qkv and out"))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  Params p = base(rope, positions, pos_type, rows, b, heads, kv_heads, d, dev);
  p.x = qkv;
  p.y = out;
  p.ldx = static_cast<unsigned>(ld_qkv * e);
  p.ldy = static_cast<unsigned>(ld_out * e);
  return forward<false>(p, /*values=*/qkv != out, dtype, dev, static_cast<cudaStream_t>(stream), "QK norm and rotation");
}

int tpmlp_qk_norm_rope_append(const void* qkv, int64_t ld_qkv, void* q, int64_t ld_q, const tpmlp_kv_cache* cache,
                              const int64_t* slots, const tpmlp_qk_rope* rope, const void* positions, int pos_type,
                              int64_t rows, int heads, int kv_heads, int d, int dtype, void* stream) {
  int rc = check_append(qkv, ld_qkv, q, ld_q, cache, slots, rope, positions, pos_type, rows, heads, kv_heads, d, dtype);
  if (rc || rows == 0) return rc;
  const size_t e = esize(dtype);
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  Params p = base(rope, positions, pos_type, rows, 1, heads, kv_heads, d, dev);
  p.x = qkv;
  p.y = q;
  p.ldx = static_cast<unsigned>(ld_qkv * e);
  p.ldy = static_cast<unsigned>(ld_q * e);
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
  if ((rc = check_rope(rope, d, positions, pos_type, rows > 0 ? (rows - 1) / b : 0)) ||
      (rows > 0 && ((rc = check_ptr(dout, 16, "dout")) || (rc = check_ptr(dqkv, 16, "dqkv")))) ||
      (rc = check_ld(ld_dout, W, e, "ld_dout")) || (rc = check_ld(ld_dqkv, W, e, "ld_dqkv")))
    return rc;
  const bool norm = rope->q_gamma != nullptr;
  const size_t need = norm ? tpmlp_qk_norm_rope_backward_workspace(rows, heads, kv_heads, d) : 0;
  if (norm) {
    if ((rows > 0 && (rc = check_ptr(qkv, 16, "qkv"))) || (rc = check_ld(ld_qkv, W, e, "ld_qkv")) ||
        (rc = check_ptr(dq_gamma, 4, "dq_gamma")) || (rc = check_ptr(dk_gamma, 4, "dk_gamma")))
      return rc;
    if (need > 0) {
      if (ws == nullptr || ws_bytes < need)
        return set_error(TPMLP_ERR_WORKSPACE, "QK norm backward workspace needs " + std::to_string(need) + " bytes");
      if ((rc = check_ptr(ws, 16, "ws"))) return rc;
    }
  }
  if (rows > 0 && dout == dqkv && ld_dout != ld_dqkv)
    return set_error(TPMLP_ERR_INVALID_ARG, "in place, ld_dout and ld_dqkv must be equal");
  if (dout != dqkv && (rc = check_apart(dout, ld_dout, W, dqkv, ld_dqkv, W, rows, dtype, "dout and dqkv"))) return rc;
  if (norm && (qkv != dqkv || ld_qkv != ld_dqkv) &&
      (rc = check_apart(qkv, ld_qkv, W, dqkv, ld_dqkv, W, rows, dtype, "qkv and dqkv")))
    return rc;
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
  p.ldx = norm ? static_cast<unsigned>(ld_qkv * e) : 0;
  p.dy = dout;
  p.lddy = static_cast<unsigned>(ld_dout * e);
  p.y = dqkv;
  p.ldy = static_cast<unsigned>(ld_dqkv * e);
  p.part = static_cast<float*>(ws);
  const bool values = dout != dqkv;
  p.values = values;
  const uint64_t items = set_items(p, 32 / group_lanes(d) * BWD_U);
  const unsigned blocks = grid_of(items, std::min(BWD_CTAS * dev->num_sms, BWD_MAX_BLOCKS));
  const int ph = prof_begin(PROF_SP_REGION, st);
  cudaError_t er = dtype == DT_F32   ? launch_backward_dt<DT_F32>(p, blocks, dev, st)
                   : dtype == DT_F16 ? launch_backward_dt<DT_F16>(p, blocks, dev, st)
                                     : launch_backward_dt<DT_BF16>(p, blocks, dev, st);
  if (er == cudaSuccess && norm) {
    er = launch_pdl(qk_gamma_kernel, dim3(static_cast<unsigned>((2 * d + 31) / 32)), 1024, 0, st, 1,
                    static_cast<const float*>(p.part), static_cast<int>(blocks), d, dq_gamma, dk_gamma);
  }
  const int qk = (heads + kv_heads) * d, cols = qk + (values ? kv_heads * d : 0);
  prof_end(ph, static_cast<double>(rows) * (2.0 * cols + (norm ? qk : 0)) * e, st, norm ? 2 : 1);
  return check_launch("QK norm and rotation backward", er);
}

}  // extern "C"
