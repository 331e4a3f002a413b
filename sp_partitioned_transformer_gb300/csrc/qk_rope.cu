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
// but the 2·d sums of dγ crosses a head), so the layout serves wide accesses: a
// head is d/16 lanes, each holding the two 8-element vectors whose elements are
// paired by the rotation, so that the rotation needs no exchange and the row sum
// is a shuffle over 4, 8 or 16 lanes.  A warp takes one token and a batch of its
// heads in the order in which they lie in memory, all loads first; the angles'
// cos and sin are read once a batch.
#include <algorithm>
#include <string>

#include "internal.h"

namespace tpmlp {
namespace qkrope {

constexpr int WARPS = 8;

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
  int per_group;  // query heads of a group + 2
  int total;      // heads + 2·kv_heads
  int kv_heads;
  int d, rot, interleaved, norm;
  float eps, inv_d;
  int skip_v;     // in place: v stays where it is
  unsigned batches;  // warps per token
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

// Eight elements of storage type DT, in float32.
template <int DT>
struct Vec8 {
  uint4 r[DT == DT_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + elem * (DT == DT_F32 ? 4 : 2);
    r[0] = *reinterpret_cast<const uint4*>(p);
    if constexpr (DT == DT_F32) r[1] = *reinterpret_cast<const uint4*>(p + 16);
  }
  __device__ __forceinline__ void get(float* v) const {
    if constexpr (DT == DT_F32) {
      memcpy(v, r, 32);
    } else {
      unpack8<DT>(r[0], v);
    }
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (DT == DT_F32) {
      memcpy(r, v, 32);
    } else {
      r[0] = pack8<DT>(v);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t elem) const {
    uint8_t* p = static_cast<uint8_t*>(base) + elem * (DT == DT_F32 ? 4 : 2);
    *reinterpret_cast<uint4*>(p) = r[0];
    if constexpr (DT == DT_F32) *reinterpret_cast<uint4*>(p + 16) = r[1];
  }
};

// What a lane holds of every head: two vectors, and how the rotation pairs them.
struct LanePlan {
  bool live;    // the lane has columns (d/16 lanes of the group do)
  int ca, cb;   // first column of the two vectors
  bool ra, rb;  // each is rotated (split halves: both or none)
};

template <int GL>
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
  if (p.rot > 0 && (at < 0 || at >= p.max_pos)) {
    // outside the tables: reported, and the nearest angle taken instead of a bad read
    atomicCAS(p.status, 0u, STATUS_BAD_INDEX);
    at = at < 0 ? 0 : p.max_pos - 1;
  }
  return at;
}

// cos and sin of the lane's pairs: split halves, pair i is element i of the two
// vectors; interleaved, pairs 0–3 are in the first vector and 4–7 in the second.
struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void load(const Params& p, const LanePlan& q, int64_t pos) {
    const int64_t at = pos * (p.rot / 2);
    if (p.interleaved) {
      if (q.ra) four(p, at + q.ca / 2, 0);
      if (q.rb) four(p, at + q.cb / 2, 4);
    } else if (q.ra) {
      four(p, at + q.ca, 0);
      four(p, at + q.ca + 4, 4);
    }
  }
  __device__ __forceinline__ void four(const Params& p, int64_t at, int i) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.cos + at));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p.sin + at));
    c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
    s[i] = b.x, s[i + 1] = b.y, s[i + 2] = b.z, s[i + 3] = b.w;
  }
};

// dir = 1 rotates, −1 rotates back.  Columns that are not rotated are not
// touched (an infinity there must not meet a zero sine).
__device__ __forceinline__ void rotate(const Params& p, const LanePlan& q, const Angles& t, float dir, float* a, float* b) {
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (q.ra) {
        const float u = a[2 * i], v = a[2 * i + 1], s = dir * t.s[i];
        a[2 * i] = u * t.c[i] - v * s;
        a[2 * i + 1] = v * t.c[i] + u * s;
      }
      if (q.rb) {
        const float u = b[2 * i], v = b[2 * i + 1], s = dir * t.s[4 + i];
        b[2 * i] = u * t.c[4 + i] - v * s;
        b[2 * i + 1] = v * t.c[4 + i] + u * s;
      }
    }
  } else if (q.ra) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = a[i], v = b[i], s = dir * t.s[i];
      a[i] = u * t.c[i] - v * s;
      b[i] = v * t.c[i] + u * s;
    }
  }
}

template <int GL>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- forward, append
// One warp: one token, 32/GL·U heads.  APPEND: q goes to y, k and v to the cache.
template <int DT, int GL, int U, bool APPEND>
__global__ void __launch_bounds__(WARPS * 32) qk_forward_kernel(const __grid_constant__ Params p) {
  constexpr int G = 32 / GL;
  const unsigned lane = threadIdx.x & 31;
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  const uint64_t row64 = w / p.batches;
  if (row64 >= p.rows) return;
  const unsigned row = static_cast<unsigned>(row64);
  const int batch = static_cast<int>(w - row64 * p.batches);
  const int l = lane % GL, grp = lane / GL;
  const LanePlan q = lane_plan<GL>(p, l);
  const int64_t xr = static_cast<int64_t>(row) * p.ldx;
  const int u0 = batch * (G * U) + grp;
  Vec8<DT> va[U], vb[U];
  int kind[U];  // 0 query, 1 key, 2 value, −1 nothing to do
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = u0 + i * G;
    const int j = u % p.per_group;
    kind[i] = u >= p.total ? -1 : j < p.per_group - 2 ? 0 : j - p.per_group + 3;
    if (!APPEND && kind[i] == 2 && p.skip_v) kind[i] = -1;
    if (kind[i] >= 0 && q.live) {
      va[i].load(p.x, xr + static_cast<int64_t>(u) * p.d + q.ca);
      vb[i].load(p.x, xr + static_cast<int64_t>(u) * p.d + q.cb);
    }
  }
  Angles t;
  if (p.rot > 0) t.load(p, q, position_of(p, row));
  int64_t cache_row = -1;
  if constexpr (APPEND) {
    const int64_t slot = p.slots[row];
    if (slot >= 0) {
      const int64_t page = slot / p.page_size;
      if (page < p.pages) cache_row = page * p.page_stride + (slot - page * p.page_size) * p.token_stride;
      else atomicCAS(p.status, 0u, STATUS_BAD_INDEX);  // behind the cache: reported, nothing written
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = u0 + i * G;
    float a[8], b[8];
    const bool turn = kind[i] == 0 || kind[i] == 1;
    if (turn && q.live) {
      va[i].get(a);
      vb[i].get(b);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = b[j] = 0.0f;
    }
    if (p.norm) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
      const float r = rsqrtf(fmaf(group_sum<GL>(ss), p.inv_d, p.eps));
      if (turn && q.live) {
        const void* gm = kind[i] == 0 ? p.gq : p.gk;
        Vec8<DT> ga, gb;
        float g[8];
        ga.load(gm, q.ca);
        gb.load(gm, q.cb);
        ga.get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = a[j] * r * g[j];
        gb.get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = b[j] * r * g[j];
      }
    }
    if (kind[i] < 0 || !q.live) continue;
    if (turn) {
      if (p.rot > 0) rotate(p, q, t, 1.0f, a, b);
      va[i].set(a);
      vb[i].set(b);
    }
    if constexpr (APPEND) {
      const int g = u / p.per_group;
      if (kind[i] == 0) {
        const int64_t at = static_cast<int64_t>(row) * p.ldy + static_cast<int64_t>(u - 2 * g) * p.d;
        va[i].store(p.y, at + q.ca);
        vb[i].store(p.y, at + q.cb);
      } else if (cache_row >= 0) {
        void* dst = kind[i] == 1 ? p.kc : p.vc;
        const int64_t at = cache_row + g * p.head_stride;
        va[i].store(dst, at + q.ca);
        vb[i].store(dst, at + q.cb);
      }
    } else {
      const int64_t at = static_cast<int64_t>(row) * p.ldy + static_cast<int64_t>(u) * p.d;
      va[i].store(p.y, at + q.ca);
      vb[i].store(p.y, at + q.cb);
    }
  }
}

// ---------------------------------------------------------------- backward
// Warps step over (token, batch of heads); every lane keeps the dγ sums of its
// 16 columns, one set for γ_q and one for γ_k, added over the block at the end
// and over the blocks, in block order, by qk_gamma_kernel.
template <int DT, int GL, int U>
__global__ void __launch_bounds__(WARPS * 32) qk_backward_kernel(const __grid_constant__ Params p) {
  constexpr int G = 32 / GL;
  __shared__ float sums[WARPS][2][GL * 16];
  const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % GL, grp = lane / GL;
  const LanePlan q = lane_plan<GL>(p, l);
  float sq[16], sk[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) sq[j] = sk[j] = 0.0f;
  const uint64_t items = static_cast<uint64_t>(p.rows) * p.batches;
  for (uint64_t w = static_cast<uint64_t>(blockIdx.x) * WARPS + warp; w < items;
       w += static_cast<uint64_t>(gridDim.x) * WARPS) {
    const unsigned row = static_cast<unsigned>(w / p.batches);
    const int batch = static_cast<int>(w - static_cast<uint64_t>(row) * p.batches);
    const int u0 = batch * (G * U) + grp;
    Vec8<DT> xa[U], xb[U], da[U], db[U];
    int kind[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = u0 + i * G;
      const int j = u % p.per_group;
      kind[i] = u >= p.total ? -1 : j < p.per_group - 2 ? 0 : j - p.per_group + 3;
      if (kind[i] == 2 && p.skip_v) kind[i] = -1;
      if (kind[i] >= 0 && q.live) {
        const int64_t dat = static_cast<int64_t>(row) * p.lddy + static_cast<int64_t>(u) * p.d;
        da[i].load(p.dy, dat + q.ca);
        db[i].load(p.dy, dat + q.cb);
        if (p.norm && kind[i] < 2) {
          const int64_t xat = static_cast<int64_t>(row) * p.ldx + static_cast<int64_t>(u) * p.d;
          xa[i].load(p.x, xat + q.ca);
          xb[i].load(p.x, xat + q.cb);
        }
      }
    }
    Angles t;
    if (p.rot > 0) t.load(p, q, position_of(p, row));
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = u0 + i * G;
      const bool turn = (kind[i] == 0 || kind[i] == 1) && q.live;
      float a[8], b[8];
      if (turn) {
        da[i].get(a);
        db[i].get(b);
        if (p.rot > 0) rotate(p, q, t, -1.0f, a, b);
      }
      if (p.norm) {
        float x[16], ga[8], gb[8];
        float ss = 0.0f, ts = 0.0f;
        if (turn) {
          xa[i].get(x);
          xb[i].get(x + 8);
          const void* gm = kind[i] == 0 ? p.gq : p.gk;
          Vec8<DT> g;
          g.load(gm, q.ca);
          g.get(ga);
          g.load(gm, q.cb);
          g.get(gb);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            ss = fmaf(x[j], x[j], fmaf(x[8 + j], x[8 + j], ss));
            ts = fmaf(a[j] * ga[j], x[j], fmaf(b[j] * gb[j], x[8 + j], ts));
          }
        }
        ss = group_sum<GL>(ss);
        ts = group_sum<GL>(ts);
        if (turn) {
          const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
          const float m = ts * r * p.inv_d;  // mean of t·x̂
          const float fq = kind[i] == 0 ? 1.0f : 0.0f;
          (void)fq;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float na = x[j] * r, nb = x[8 + j] * r;
            if (kind[i] == 0) {
              sq[j] = fmaf(a[j], na, sq[j]);
              sq[8 + j] = fmaf(b[j], nb, sq[8 + j]);
            } else {
              sk[j] = fmaf(a[j], na, sk[j]);
              sk[8 + j] = fmaf(b[j], nb, sk[8 + j]);
            }
            a[j] = r * (a[j] * ga[j] - na * m);
            b[j] = r * (b[j] * gb[j] - nb * m);
          }
        }
      }
      if (kind[i] < 0 || !q.live) continue;
      if (turn) {
        da[i].set(a);
        db[i].set(b);
      }
      const int64_t at = static_cast<int64_t>(row) * p.ldy + static_cast<int64_t>(u) * p.d;
      da[i].store(p.y, at + q.ca);
      db[i].store(p.y, at + q.cb);
    }
  }
  if (!p.norm) return;
  // Over the lane groups of the warp, then over the block's warps.
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int o = GL; o < 32; o <<= 1) {
      sq[j] += __shfl_xor_sync(0xffffffffu, sq[j], o);
      sk[j] += __shfl_xor_sync(0xffffffffu, sk[j], o);
    }
  }
  if (grp == 0 && q.live) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sums[warp][0][q.ca + j] = sq[j];
      sums[warp][0][q.cb + j] = sq[8 + j];
      sums[warp][1][q.ca + j] = sk[j];
      sums[warp][1][q.cb + j] = sk[8 + j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.d; i += WARPS * 32) {
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
int group_lanes(int d) { return d <= 64 ? 4 : d <= 128 ? 8 : 16; }
constexpr int BWD_U = 2;
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
  if (heads > 65535 || rows >= (1ll << 31) || b >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
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
  p.per_group = heads / kv_heads + 2;
  p.total = heads + 2 * kv_heads;
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

template <int DT, int GL, bool APPEND>
int launch_forward(Params& p, const DeviceInfo* dev, cudaStream_t st) {
  constexpr int G = 32 / GL;
  // Four heads a lane group amortise the angles; with few rows one head each
  // spreads the work over the SMs instead.
  const bool few = static_cast<int64_t>(p.rows) * ((p.total + 4 * G - 1) / (4 * G)) < 16ll * dev->num_sms;
  const int per = few ? G : 4 * G;
  p.batches = static_cast<unsigned>((p.total + per - 1) / per);
  const int64_t blocks = (static_cast<int64_t>(p.rows) * p.batches + WARPS - 1) / WARPS;
  if (blocks >= (1ll << 31)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  if (few) qk_forward_kernel<DT, GL, 1, APPEND><<<static_cast<unsigned>(blocks), WARPS * 32, 0, st>>>(p);
  else qk_forward_kernel<DT, GL, 4, APPEND><<<static_cast<unsigned>(blocks), WARPS * 32, 0, st>>>(p);
  return TPMLP_OK;
}

template <bool APPEND>
int forward(Params& p, int dtype, const DeviceInfo* dev, cudaStream_t st, const char* what) {
  const int ph = prof_begin(PROF_SP_REGION, st);
  int rc = TPMLP_OK;
#define FWD(D)                                                                \
  do {                                                                        \
    const int gl = group_lanes(p.d);                                          \
    if (gl == 4) rc = launch_forward<D, 4, APPEND>(p, dev, st);               \
    else if (gl == 8) rc = launch_forward<D, 8, APPEND>(p, dev, st);          \
    else rc = launch_forward<D, 16, APPEND>(p, dev, st);                      \
  } while (0)
  if (dtype == DT_F32) FWD(DT_F32); else if (dtype == DT_F16) FWD(DT_F16); else FWD(DT_BF16);
#undef FWD
  const int cols = (p.skip_v ? p.total - p.kv_heads : p.total) * p.d;
  prof_end(ph, 2.0 * p.rows * cols * esize(dtype), st);
  return rc ? rc : check_launch(what);
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
  p.skip_v = qkv == out;
  return forward<false>(p, dtype, dev, static_cast<cudaStream_t>(stream), "QK norm and rotation");
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
  return forward<true>(p, dtype, dev, static_cast<cudaStream_t>(stream), "QK norm, rotation and cache append");
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
  p.skip_v = dout == dqkv;
  p.part = static_cast<float*>(ws);
  const int gl = group_lanes(d), G = 32 / gl;
  p.batches = static_cast<unsigned>((p.total + G * BWD_U - 1) / (G * BWD_U));
  const int64_t want = (rows * p.batches + WARPS - 1) / WARPS;
  const int blocks = static_cast<int>(std::min<int64_t>(want, std::min(2 * dev->num_sms, BWD_MAX_BLOCKS)));
  const int ph = prof_begin(PROF_SP_REGION, st);
#define BWD(D)                                                                                   \
  do {                                                                                           \
    if (gl == 4) qk_backward_kernel<D, 4, BWD_U><<<blocks, WARPS * 32, 0, st>>>(p);              \
    else if (gl == 8) qk_backward_kernel<D, 8, BWD_U><<<blocks, WARPS * 32, 0, st>>>(p);         \
    else qk_backward_kernel<D, 16, BWD_U><<<blocks, WARPS * 32, 0, st>>>(p);                     \
  } while (0)
  if (dtype == DT_F32) BWD(DT_F32); else if (dtype == DT_F16) BWD(DT_F16); else BWD(DT_BF16);
#undef BWD
  cudaError_t er = cudaGetLastError();
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
    er = cudaLaunchKernelEx(&cfg, qk_gamma_kernel, static_cast<const float*>(p.part), blocks, d, dq_gamma, dk_gamma);
  }
  const int cols = (p.skip_v ? p.total - p.kv_heads : p.total) * p.d;
  prof_end(ph, static_cast<double>(rows) * (2.0 * cols + (norm ? (p.total - p.kv_heads) * p.d : 0)) * e, st, norm ? 2 : 1);
  return check_launch("QK norm and rotation backward", er);
}

}  // extern "C"
