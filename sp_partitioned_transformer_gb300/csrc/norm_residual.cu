// The residual path of a layer in the sequence-parallel region: the RMS norm behind
// a block with its gate and residual scale, and the norm in front of the next block,
// on the [s/tp, b, h] sequence chunks (the region of sp_region.cu).
//
//   n = z·ρ_z·γ₁,  ρ_z = 1/√(mean z² + eps)        (n = z without γ₁)
//   x = r + α·g⊙n, rounded to the storage type
//   y = x·ρ_x·γ₂,  ρ_x = 1/√(mean x² + eps)
// backward, from dx (of x, past the next block) and dy (of y):
//   t  = dy·γ₂, x̂ = x·ρ_x:   dr = dx + ρ_x·(t − x̂·mean(t·x̂))
//   t' = α·g·γ₁·dr, ẑ = z·ρ_z: dz = ρ_z·(t' − ẑ·mean(t'·ẑ))
//   dγ₂ = Σ dy·x̂, and with S = Σ dr·ẑ over the rows that share a gate:
//   dγ₁ = α·Σ g·S over the gates, dgate = α·γ₁·S
// so that one sum per column and gate serves both.
//
// Everything is bound by HBM: forward r, z in and x, y out, backward dx, dy, x, z in
// and dr, dz out, each element once.  Rows are dealt out in units: unit (gi, k) has
// the rows m = (k + K·i)·gate_rows + gi, so that a CTA meets one gate only and sums
// its rows' column sums for itself.
#include <algorithm>
#include <atomic>
#include <string>

#include "checkpoint.cuh"
#include "internal.h"

namespace tpmlp {
namespace normres {

// Units of a backward at most (one a gate where there are more gates): 4 or 8 for each of
// 152 SMs, as far as narrow rows leave room for.
constexpr int max_units(int64_t h) { return h < 4096 ? 1216 : 608; }

// The chunks' pointers stand together, behind the scalars: with few chunks all that a
// kernel reads of its parameters is a few neighbouring lines.
struct Fwd {
  const void* post;  // γ₁
  const void* pre;   // γ₂
  const void* gate;  // [gate_rows, h]
  uint8_t* codes;    // checkpoint of z
  uint8_t* scales;
  float* rstd_z;
  float* rstd_x;
  float scale, eps;
  int h, rpc, rows, gate_rows, K;  // rows = s·b, rpc rows a chunk
  int has_z;
  int stages;
  struct {
    const void* r;
    const void* z;
    void* x;
    void* y;
  } chunk[TPMLP_MAX_TP];
};

struct Bwd {
  const void* post;
  const void* pre;
  const void* gate;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* rstd_z;
  const float* rstd_x;
  float* part1;  // [units, pitch] of S
  float* part2;  // [units, pitch] of dγ₂
  int64_t pitch;  // h rounded up to 4
  float scale;
  int h, rpc, rows, gate_rows, K;
  int has_dx, has_dz, has_z;  // has_z: z (or its checkpoint) is read
  int stages;
  struct {
    const void* dx;
    const void* dy;
    const void* x;
    const void* z;
    void* dr;
    void* dz;
  } chunk[TPMLP_MAX_TP];
};

// Chunk and row within it of m = m0 + i·step, stepped without divisions.
struct Pos {
  int j, r, qs, rs, rpc;
  __device__ __forceinline__ Pos(int m0, int step, int rpc_)
      : j(m0 / rpc_), r(m0 - m0 / rpc_ * rpc_), qs(step / rpc_), rs(step - step / rpc_ * rpc_), rpc(rpc_) {}
  __device__ __forceinline__ void next() {
    j += qs;
    if (r >= rpc - rs) {  // (r + rs may pass 2³¹)
      r -= rpc - rs;
      ++j;
    } else {
      r += rs;
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The CTA's sum, in a fixed order.  red: one of two arrays of 32, used in turn, so
// that the one barrier also frees the other.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.0f);
}

template <int DT>
__device__ __forceinline__ float at(const void* p, int64_t i) {
  return Storage<DT>::to_f32(static_cast<const typename Storage<DT>::T*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  static_cast<typename Storage<DT>::T*>(p)[i] = Storage<DT>::from(v);
}

// ------------------------------------------------------------------ rows of whole vectors
// A CTA of G threads takes a row at a time; thread t owns the 8-element vectors
// t, t + G, … < h/8 (V of them at most), copies its own vectors of the rows ahead into a
// ring of shared memory with cp.async, and reads only what it copied itself, so that no
// barrier stands between a load and its use and HBM reads run ahead of the two sums
// that a row has to wait for.  Four neighbouring threads hold a group of a checkpoint.
constexpr int MAX_STAGES = 5;
// An SM's loads ahead of the rows in work.  More cost: backward at 4096 rows of 8192 with one
// row ahead (64 KB) 71.0 µs, two 77.2; forward 49.6 and 50.3.
constexpr size_t AHEAD_BYTES = 64 << 10;

template <int DT>
struct Vec {  // 8 elements as stored
  static constexpr int N = DT == DT_F32 ? 2 : 1;  // 16-byte units
  uint4 u[N];
};

template <int DT>
__device__ __forceinline__ void values(const Vec<DT>& r, float2* f) {
  if constexpr (DT == DT_F32) {
    memcpy(f, r.u, 32);
  } else {
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == DT_BF16)
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      else
        f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    }
  }
}

template <int DT>
__device__ __forceinline__ Vec<DT> rounded(const float2* f) {
  Vec<DT> r;
  if constexpr (DT == DT_F32) {
    memcpy(r.u, f, 32);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == DT_BF16) {
        const __nv_bfloat162 b = __float22bfloat162_rn(f[i]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        const __half2 b = __float22half2_rn(f[i]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

// 8 elements from element i on, 16-byte aligned.
template <int DT>
__device__ __forceinline__ Vec<DT> load_vec(const void* p, int64_t i) {
  Vec<DT> r;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const typename Storage<DT>::T*>(p) + i);
#pragma unroll
  for (int k = 0; k < Vec<DT>::N; ++k) r.u[k] = q[k];
  return r;
}
// 8 elements to p, aligned to all of them.
template <int DT>
__device__ __forceinline__ void store_vec(void* p, const Vec<DT>& r) {
  if constexpr (DT == DT_F32)
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r.u[0].x), "r"(r.u[0].y), "r"(r.u[0].z),
                 "r"(r.u[0].w), "r"(r.u[1].x), "r"(r.u[1].y), "r"(r.u[1].z), "r"(r.u[1].w), "l"(p)
                 : "memory");
  else
    *static_cast<uint4*>(p) = r.u[0];
}

// A thread's vectors in the ring: vector v of input `in` lies at in·in_bytes + v·v_bytes
// from the stage's address, a float32 vector's halves G units apart.
template <int DT, int V>
struct Ring {
  uint32_t first, v_bytes, in_bytes, stage_bytes;
  __device__ __forceinline__ Ring(uint32_t smem, int nin)
      : first(smem + threadIdx.x * 16u),
        v_bytes(blockDim.x * 16u * Vec<DT>::N),
        in_bytes(v_bytes * V),
        stage_bytes(in_bytes * nin) {}
  // 8 elements at p to shared address a
  __device__ __forceinline__ void fetch(uint32_t a, const char* p) const {
    if constexpr (DT == DT_F32) {  // the halves share a 32-byte sector: through L1, which fetches it once
#pragma unroll
      for (int k = 0; k < 2; ++k)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(a + k * blockDim.x * 16u), "l"(p + 16 * k) : "memory");
    } else {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(a), "l"(p) : "memory");
    }
  }
  __device__ __forceinline__ void fetch_codes(uint32_t a, const uint8_t* p) const {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(a), "l"(p) : "memory");
  }
  __device__ __forceinline__ void fetch_word(uint32_t a, const uint8_t* p) const {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(a), "l"(p) : "memory");
  }
  __device__ __forceinline__ Vec<DT> get(uint32_t a) const {
    Vec<DT> r;
#pragma unroll
    for (int k = 0; k < Vec<DT>::N; ++k)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.u[k].x), "=r"(r.u[k].y), "=r"(r.u[k].z), "=r"(r.u[k].w)
                   : "r"(a + k * blockDim.x * 16u)
                   : "memory");
    return r;
  }
  __device__ __forceinline__ uint2 get_codes(uint32_t a) const {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
    return r;
  }
  __device__ __forceinline__ uint32_t get_word(uint32_t a) const {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
    return r;
  }
  __device__ __forceinline__ uint32_t get_byte(uint32_t a) const {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
    return r;
  }
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `left` of this thread's newest groups are in flight.
__device__ __forceinline__ void cp_wait(int left) {
  if (left >= 4)
    asm volatile("cp.async.wait_group 4;" ::: "memory");
  else if (left == 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (left == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (left == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The CTA's sum, in a fixed order: a shuffle tree in the warp, then every thread adds
// the warps' sums itself (reads that all lanes share).  red: one of two arrays of 16, the
// entries behind the last warp zero, used in turn: the one barrier frees the other.
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const float4* r4 = reinterpret_cast<const float4*>(red);
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = r4[i];
    s = __fadd2_rn(s, __fadd2_rn(make_float2(a.x, a.y), make_float2(a.z, a.w)));
  }
  return s.x + s.y;
}

// A row on a cluster of CL CTAs: each has a share of whole groups of 4 vectors, and the
// CTAs' sums meet in every CTA's `other` (one of two arrays, used in turn).
template <int CL>
struct Share {
  int rank, first, nv;  // first vector, vectors
  __device__ __forceinline__ explicit Share(int all) {
    rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int each = CL > 1 ? ((all + CL - 1) / CL + 3) & ~3 : all;
    first = rank * each;
    nv = min(each, all - first);
  }
};
template <int CL>
__device__ __forceinline__ void all_sync() {
  if constexpr (CL > 1)
    cluster_sync_all();
  else
    __syncthreads();
}
template <int CL>
__device__ __forceinline__ float row_sum_all(float v, float* red, float* other, int rank) {
  const float s = row_sum(v, red);
  if constexpr (CL == 1) return s;
  if (threadIdx.x < CL) {
    const uint32_t at = mapa_shared(smem_u32(other + rank), threadIdx.x);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(s) : "memory");
  }
  cluster_sync_all();
  float all = 0.0f;
#pragma unroll
  for (int i = 0; i < CL; ++i) all += other[i];
  return all;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// scale·g·γ₁ of a vector.
template <int DT>
__device__ __forceinline__ void branch_weight(const void* gate, const void* post, float scale, int64_t goff, int col,
                                              float2* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = both(scale);
  float2 f[4];
  if (gate) {
    values<DT>(load_vec<DT>(gate, goff + col), f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mul2(w[i], f[i]);
  }
  if (post) {
    values<DT>(load_vec<DT>(post, col), f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mul2(w[i], f[i]);
  }
}

// A checkpoint's vector to b; returns what b is still to be multiplied by for ẑ: ρ and the
// group's power of two, but for groups at the end of the type's range, whose values are
// brought into it first.
template <int DT>
__device__ __forceinline__ float held_vector(uint2 codes, uint32_t byte, float rho, float2* b) {
  ckpt_numbers4(codes.x, b);
  ckpt_numbers4(codes.y, b + 2);
  const float scale = ckpt_scale(byte);
  if (!ckpt_near_end<DT>(byte)) return scale * rho;
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = make_float2(ckpt_in_range<DT>(b[k].x * scale), ckpt_in_range<DT>(b[k].y * scale));
  return rho;
}

// All vectors of a thread but its last lie in the row: (V − 1)·G ≤ nv.
template <int V>
__device__ __forceinline__ bool inside(int v, int vi, int nv) {
  return v < V - 1 || vi < nv;
}

// FULL: z and both norms, known to the compiler.  CL: CTAs of a row.
template <int DT, int V, bool FULL, int CL = 1>
__global__ void __launch_bounds__(512, 1) vec_fwd_kernel(const __grid_constant__ Fwd p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][16];
  __shared__ float other[2][CL];
  constexpr int E = DT == DT_F32 ? 4 : 2;
  pdl_enter();
  const int G = blockDim.x, t = threadIdx.x, S = p.stages;
  const bool has_z = FULL || p.has_z, post = FULL || p.post != nullptr, pre = FULL || p.pre != nullptr;
  const int h = p.h, groups = (h + 31) >> 5;
  const Share<CL> share(h >> 3);
  const int nv = share.nv;
  const float inv_h = 1.0f / static_cast<float>(h);
  if (t < 32) red[t >> 4][t & 15] = 0.0f;
  all_sync<CL>();  // (the peers' shared memory is there from here on)
  const int unit = blockIdx.x / CL, gi = unit % p.gate_rows;
  const int64_t first = static_cast<int64_t>(unit / p.gate_rows) * p.gate_rows + gi;
  const int step = p.K * p.gate_rows;
  const int n = static_cast<int>((p.rows - 1 - first) / step) + 1;  // rows of the unit
  const Ring<DT, V> ring(smem_u32(smem), 1 + has_z);
  const uint32_t g_bytes = G * 8 * E;  // from a thread's vector to its next

  Pos ahead(static_cast<int>(first), step, p.rpc), pos = ahead;
  auto fetch = [&](uint32_t a) {
    const int64_t off = (static_cast<int64_t>(ahead.r) * h + (share.first + t) * 8) * E;
    const char* r = static_cast<const char*>(p.chunk[ahead.j].r) + off;
    const char* z = static_cast<const char*>(p.chunk[ahead.j].z) + off;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (inside<V>(v, v * G + t, nv)) {
        if (has_z) ring.fetch(a + ring.in_bytes + v * ring.v_bytes, z + v * g_bytes);
        ring.fetch(a + v * ring.v_bytes, r + v * g_bytes);
      }
    }
  };
  uint32_t a_ahead = ring.first, a = ring.first;
  const uint32_t a_end = ring.first + S * ring.stage_bytes;
  for (int i = 0; i < S - 1; ++i) {
    if (i < n) {
      fetch(a_ahead);
      ahead.next();
    }
    cp_commit();
    a_ahead += ring.stage_bytes;
  }
  float2 w[V][4];
  Vec<DT> g2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = (share.first + v * G + t) * 8;
    if (inside<V>(v, v * G + t, nv)) {
      branch_weight<DT>(p.gate, p.post, p.scale, static_cast<int64_t>(gi) * h, col, w[v]);
      if (pre) g2[v] = load_vec<DT>(p.pre, col);
    }
  }

  int64_t m = first;
  for (int i = 0; i < n; ++i, m += step, pos.next()) {
    if (i + S - 1 < n) {
      fetch(a_ahead);
      ahead.next();
    }
    cp_commit();
    if ((a_ahead += ring.stage_bytes) == a_end) a_ahead = ring.first;
    cp_wait(S - 1);
    const int64_t off = (static_cast<int64_t>(pos.r) * h + (share.first + t) * 8) * E;
    float rz = 1.0f;
    if (post) {
      float2 q = both(0.0f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (inside<V>(v, v * G + t, nv)) {
          float2 z[4];
          values<DT>(ring.get(a + ring.in_bytes + v * ring.v_bytes), z);
#pragma unroll
          for (int k = 0; k < 4; ++k) q = __ffma2_rn(z[k], z[k], q);
        }
      }
      rz = 1.0f / sqrtf(row_sum_all<CL>(q.x + q.y, red[0], other[0], share.rank) * inv_h + p.eps);
      if (t == 0 && share.rank == 0) p.rstd_z[m] = rz;
    }
    float2 q = both(0.0f);
    Vec<DT> x[V];
    char* xo = static_cast<char*>(p.chunk[pos.j].x) + off;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int vi = v * G + t;
      const bool in = inside<V>(v, vi, nv);
      float2 z[4] = {};
      if (in) {
        x[v] = ring.get(a + v * ring.v_bytes);
        float2 f[4];
        values<DT>(x[v], f);
        if (has_z) {
          values<DT>(ring.get(a + ring.in_bytes + v * ring.v_bytes), z);
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = __ffma2_rn(w[v][k], mul2(z[k], both(rz)), f[k]);
          x[v] = rounded<DT>(f);
          store_vec<DT>(xo + v * g_bytes, x[v]);
          values<DT>(x[v], f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) q = __ffma2_rn(f[k], f[k], q);
      }
      if (p.codes) {  // (with z only) four lanes are a group; lanes behind the row's end bring nothing
        const float* zf = &z[0].x;
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, ckpt_abs(zf[k]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t byte = ckpt_byte(top);
        const float inv = ckpt_inverse(byte);
        if (in) {
          *reinterpret_cast<uint2*>(p.codes + m * h + (share.first + vi) * 8) = make_uint2(ckpt_encode4(zf, inv), ckpt_encode4(zf + 4, inv));
          if ((t & 3) == 0) p.scales[m * groups + ((share.first + vi) >> 2)] = static_cast<uint8_t>(byte);
        }
      }
    }
    if (pre) {
      const float rx = 1.0f / sqrtf(row_sum_all<CL>(q.x + q.y, red[1], other[1], share.rank) * inv_h + p.eps);
      if (t == 0 && share.rank == 0) p.rstd_x[m] = rx;
      char* yo = static_cast<char*>(p.chunk[pos.j].y) + off;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (inside<V>(v, v * G + t, nv)) {
          float2 f[4], g[4];
          values<DT>(x[v], f);
          values<DT>(g2[v], g);
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = mul2(mul2(f[k], both(rx)), g[k]);
          store_vec<DT>(yo + v * g_bytes, rounded<DT>(f));
        }
      }
    }
    if (!post || !pre) all_sync<CL>();  // one sum a row: nothing else frees its array
    if ((a += ring.stage_bytes) == a_end) a = ring.first;
  }
}

// The backward's inputs in a stage: dx, dy, x, z, those that there are.  A row's vectors are
// unpacked once: t and x̂ stay in registers from the first sum to dr, t' and ẑ (in their
// place) from there to dz.
// HELD: all of them, z as a checkpoint, known to the compiler, which takes a third off the
// instructions; without, they are asked for row by row.  (4096 rows of 6144, float16, z
// held: 67.6 -> 58.3 µs.  With z in 16 bits HBM is the bound and the tighter bursts of
// loads cost more than the instructions: 69.7 -> 71.0 µs at 4096 rows of 8192.)

// CL: CTAs of a row.
template <int DT, int V, bool HELD, int CL = 1>
__global__ void __launch_bounds__(512, 1) vec_bwd_kernel(const __grid_constant__ Bwd p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][16];
  __shared__ float other[2][CL];
  constexpr int E = DT == DT_F32 ? 4 : 2;
  pdl_enter();
  const int G = blockDim.x, t = threadIdx.x, S = p.stages;
  const int h = p.h, groups = (h + 31) >> 5;
  const Share<CL> share(h >> 3);
  const int nv = share.nv;
  const float inv_h = 1.0f / static_cast<float>(h);
  if (t < 32) red[t >> 4][t & 15] = 0.0f;
  all_sync<CL>();
  const int unit = blockIdx.x / CL, gi = unit % p.gate_rows;
  const int64_t first = static_cast<int64_t>(unit / p.gate_rows) * p.gate_rows + gi;
  const int step = p.K * p.gate_rows;
  const int n = static_cast<int>((p.rows - 1 - first) / step) + 1;  // rows of the unit
  const bool pre = HELD || p.pre != nullptr, post = HELD || p.post != nullptr, held = HELD || p.codes != nullptr;
  const bool has_dx = HELD || p.has_dx, has_dz = HELD || p.has_dz, has_z = HELD || p.has_z;
  // whether a row's scale bytes are whole aligned words, which come through the ring
  const bool words = groups % 4 == 0 && reinterpret_cast<uintptr_t>(p.scales) % 4 == 0;
  const Ring<DT, V> ring(smem_u32(smem), has_dx + 2 * pre + has_z);
  const uint32_t o_dy = has_dx * ring.in_bytes, o_x = o_dy + pre * ring.in_bytes, o_z = o_x + pre * ring.in_bytes;
  const uint32_t g_bytes = G * 8 * E;  // from a thread's vector to its next

  Pos ahead(static_cast<int>(first), step, p.rpc), pos = ahead;
  int64_t m_ahead = first;
  auto fetch = [&](uint32_t a) {
    const int64_t off = (static_cast<int64_t>(ahead.r) * h + (share.first + t) * 8) * E;
    const char* dx = static_cast<const char*>(p.chunk[ahead.j].dx) + off;
    const char* dy = static_cast<const char*>(p.chunk[ahead.j].dy) + off;
    const char* x = static_cast<const char*>(p.chunk[ahead.j].x) + off;
    const char* z = static_cast<const char*>(p.chunk[ahead.j].z) + off;
    const uint8_t* c = p.codes + m_ahead * h + (share.first + t) * 8;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (inside<V>(v, v * G + t, nv)) {
        const uint32_t av = a + v * ring.v_bytes;
        if (pre) {
          ring.fetch(av + o_dy, dy + v * g_bytes);
          ring.fetch(av + o_x, x + v * g_bytes);
        }
        if (has_dx) ring.fetch(av, dx + v * g_bytes);
        if (held) {
          ring.fetch_codes(av + o_z, c + v * G * 8);
          if (words) ring.fetch_word(av + o_z + 8, p.scales + m_ahead * groups + ((share.first + v * G + t) >> 4) * 4);  // beside them
        } else if (has_z)
          ring.fetch(av + o_z, z + v * g_bytes);
      }
    }
  };
  uint32_t a_ahead = ring.first, a = ring.first;
  const uint32_t a_end = ring.first + S * ring.stage_bytes;
  for (int i = 0; i < S - 1; ++i) {
    if (i < n) {
      fetch(a_ahead);
      ahead.next();
      m_ahead += step;
    }
    cp_commit();
    a_ahead += ring.stage_bytes;
  }
  float2 w[V][4], sum1[V][4], sum2[V][4];
  Vec<DT> g2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = (share.first + v * G + t) * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k) sum1[v][k] = sum2[v][k] = both(0.0f);
    if (inside<V>(v, v * G + t, nv)) {
      branch_weight<DT>(p.gate, p.post, p.scale, static_cast<int64_t>(gi) * h, col, w[v]);
      if (pre) g2[v] = load_vec<DT>(p.pre, col);
    }
  }

  float rx_lane = 0.0f, rz_lane = 1.0f;
  int64_t m = first;
  for (int i = 0; i < n; ++i, m += step, pos.next()) {
    if (i + S - 1 < n) {
      fetch(a_ahead);
      ahead.next();
      m_ahead += step;
    }
    cp_commit();
    if ((a_ahead += ring.stage_bytes) == a_end) a_ahead = ring.first;
    if ((i & 31) == 0 && i + (t & 31) < n) {  // ρ of the next 32 rows, a row a lane
      const int64_t ml = m + static_cast<int64_t>(t & 31) * step;
      if (pre) rx_lane = p.rstd_x[ml];
      if (post) rz_lane = p.rstd_z[ml];
    }
    const float rx = __shfl_sync(0xffffffffu, rx_lane, i & 31), rz = __shfl_sync(0xffffffffu, rz_lane, i & 31);
    cp_wait(S - 1);
    const int64_t off = (static_cast<int64_t>(pos.r) * h + (share.first + t) * 8) * E;
    float2 b1[V][4], b2[V][4];  // t, then dr, then t'; x̂, then ẑ
    float c1 = 0.0f;
    if (pre) {
      float2 q = both(0.0f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (inside<V>(v, v * G + t, nv)) {
          float2 d[4], g[4];
          values<DT>(ring.get(a + o_dy + v * ring.v_bytes), d);
          values<DT>(ring.get(a + o_x + v * ring.v_bytes), b2[v]);
          values<DT>(g2[v], g);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            b2[v][k] = mul2(b2[v][k], both(rx));
            b1[v][k] = mul2(d[k], g[k]);
            sum2[v][k] = __ffma2_rn(d[k], b2[v][k], sum2[v][k]);
            q = __ffma2_rn(b1[v][k], b2[v][k], q);
          }
        }
      }
      c1 = row_sum_all<CL>(q.x + q.y, red[0], other[0], share.rank) * inv_h;
    }
    float2 q = both(0.0f);
    char* dro = static_cast<char*>(p.chunk[pos.j].dr) + off;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (inside<V>(v, v * G + t, nv)) {
        const uint32_t av = a + v * ring.v_bytes;
        float2 d[4] = {};
        if (has_dx) values<DT>(ring.get(av), d);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // ρ·(t − x̂·mean(t·x̂))
          b1[v][k] = pre ? __ffma2_rn(__ffma2_rn(b2[v][k], both(-c1), b1[v][k]), both(rx), d[k]) : d[k];
        store_vec<DT>(dro + v * g_bytes, rounded<DT>(b1[v]));
        if (has_z) {
          float rho = rz;
          if (held) {
            const uint2 c = ring.get_codes(av + o_z);
            const int group = (share.first + v * G + t) >> 2;
            const uint32_t byte = words ? ring.get_word(av + o_z + 8) >> (8 * (group & 3)) & 255u : p.scales[m * groups + group];
            rho = held_vector<DT>(c, byte, rz, b2[v]);
          } else {
            values<DT>(ring.get(av + o_z), b2[v]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            b2[v][k] = mul2(b2[v][k], both(rho));
            sum1[v][k] = __ffma2_rn(b1[v][k], b2[v][k], sum1[v][k]);
            b1[v][k] = mul2(w[v][k], b1[v][k]);
            q = __ffma2_rn(b1[v][k], b2[v][k], q);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) b1[v][k] = mul2(w[v][k], b1[v][k]);
        }
      }
    }
    if (has_dz) {
      float c2 = 0.0f;
      if (post) c2 = row_sum_all<CL>(q.x + q.y, red[1], other[1], share.rank) * inv_h;
      char* dzo = static_cast<char*>(p.chunk[pos.j].dz) + off;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (inside<V>(v, v * G + t, nv)) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (post) b1[v][k] = mul2(__ffma2_rn(b2[v][k], both(-c2), b1[v][k]), both(rz));
          store_vec<DT>(dzo + v * g_bytes, rounded<DT>(b1[v]));
        }
      }
    }
    if (!pre || !post) all_sync<CL>();  // one sum a row: nothing else frees its array (post is with dz only)
    if ((a += ring.stage_bytes) == a_end) a = ring.first;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int vi = v * G + t;
    if (inside<V>(v, vi, nv)) {
      const int64_t e = static_cast<int64_t>(unit) * p.pitch + (share.first + vi) * 8;
      if (has_z) {
        reinterpret_cast<float4*>(p.part1 + e)[0] = make_float4(sum1[v][0].x, sum1[v][0].y, sum1[v][1].x, sum1[v][1].y);
        reinterpret_cast<float4*>(p.part1 + e)[1] = make_float4(sum1[v][2].x, sum1[v][2].y, sum1[v][3].x, sum1[v][3].y);
      }
      if (pre) {
        reinterpret_cast<float4*>(p.part2 + e)[0] = make_float4(sum2[v][0].x, sum2[v][0].y, sum2[v][1].x, sum2[v][1].y);
        reinterpret_cast<float4*>(p.part2 + e)[1] = make_float4(sum2[v][2].x, sum2[v][2].y, sum2[v][3].x, sum2[v][3].y);
      }
    }
  }
}

// The sums of two values, as row_sum.  red: one of two arrays of 16, used in turn.
__device__ __forceinline__ float2 row_sum2(float2 v, float2* red) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const float4* r4 = reinterpret_cast<const float4*>(red);
  float2 s = make_float2(0.0f, 0.0f), u = s;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float4 a = r4[i], b = r4[i + 1];
    s = __fadd2_rn(s, __fadd2_rn(make_float2(a.x, a.y), make_float2(a.z, a.w)));
    u = __fadd2_rn(u, __fadd2_rn(make_float2(b.x, b.y), make_float2(b.z, b.w)));
  }
  return __fadd2_rn(s, u);
}

// The same backward for a layer with all its parts and rows of 257 to 384 threads, whose
// registers leave room for a second row: the next row's first sum is taken beside this
// row's second, so that a row has one barrier, and two rows' arithmetic to put between
// loads and their use where only 9 to 12 warps an SM share the work.
template <int DT, bool HELD>
__global__ void __launch_bounds__(384, 1) vec_bwd_pair_kernel(const __grid_constant__ Bwd p) {
  constexpr int V = 2;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float2 red[2][16];
  constexpr int E = DT == DT_F32 ? 4 : 2;
  pdl_enter();
  const int G = blockDim.x, t = threadIdx.x, S = p.stages;
  const int h = p.h, nv = h >> 3, groups = (h + 31) >> 5;
  const float inv_h = 1.0f / static_cast<float>(h);
  if (t < 32) red[t >> 4][t & 15] = make_float2(0.0f, 0.0f);
  __syncthreads();
  const int gi = blockIdx.x % p.gate_rows;
  const int64_t first = static_cast<int64_t>(blockIdx.x / p.gate_rows) * p.gate_rows + gi;
  const int step = p.K * p.gate_rows;
  const int n = static_cast<int>((p.rows - 1 - first) / step) + 1;  // rows of the unit
  // A checkpoint's row lies in its part of a stage as in memory, codes and behind them
  // scale bytes: the barrier between a row's arrival and its use here lets a thread copy
  // what another reads, 16 codes or 4 bytes at once where the addresses allow it.
  const bool wide = h % 16 == 0 && reinterpret_cast<uintptr_t>(p.codes) % 16 == 0;
  const bool words = groups % 4 == 0 && reinterpret_cast<uintptr_t>(p.scales) % 4 == 0;
  const Ring<DT, V> ring(smem_u32(smem), 4);
  const uint32_t o_dy = ring.in_bytes, o_x = 2 * ring.in_bytes, o_z = 3 * ring.in_bytes;
  // from this thread's place in a stage: its first vector's 8 codes, its word of bytes, and its group's byte
  const uint32_t o_codes = o_z - t * 8, o_bytes = o_z + V * G * 8 - t * 12, o_byte = o_z + V * G * 8 - t * 16 + (t >> 2);
  const uint32_t g_bytes = G * 8 * E;

  Pos ahead(static_cast<int>(first), step, p.rpc), pos = ahead;
  int64_t m_ahead = first;
  auto fetch = [&](uint32_t a) {
    const int64_t off = (static_cast<int64_t>(ahead.r) * h + t * 8) * E;
    const char* dx = static_cast<const char*>(p.chunk[ahead.j].dx) + off;
    const char* dy = static_cast<const char*>(p.chunk[ahead.j].dy) + off;
    const char* x = static_cast<const char*>(p.chunk[ahead.j].x) + off;
    const char* z = static_cast<const char*>(p.chunk[ahead.j].z) + off;
    const uint8_t* c = p.codes + m_ahead * h + t * 8;
    if (HELD && wide && 2 * t < nv) ring.fetch(a + o_z, reinterpret_cast<const char*>(c) + t * 8);
    if (HELD && words && 4 * t < groups) ring.fetch_word(a + o_bytes, p.scales + m_ahead * groups + t * 4);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (inside<V>(v, v * G + t, nv)) {
        const uint32_t av = a + v * ring.v_bytes;
        ring.fetch(av + o_dy, dy + v * g_bytes);
        ring.fetch(av + o_x, x + v * g_bytes);
        ring.fetch(av, dx + v * g_bytes);
        if (!HELD)
          ring.fetch(av + o_z, z + v * g_bytes);
        else if (!wide)
          ring.fetch_codes(a + o_codes + v * G * 8, c + v * G * 8);
      }
    }
  };
  const uint32_t a_end = ring.first + S * ring.stage_bytes;
  uint32_t a_ahead = ring.first, a = ring.first;
  for (int i = 0; i < S - 1; ++i) {
    if (i < n) {
      fetch(a_ahead);
      ahead.next();
      m_ahead += step;
    }
    cp_commit();
    a_ahead += ring.stage_bytes;
  }
  float2 w[V][4], sum1[V][4], sum2[V][4];
  Vec<DT> g2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = (v * G + t) * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k) sum1[v][k] = sum2[v][k] = both(0.0f);
    if (col < h) {
      branch_weight<DT>(p.gate, p.post, p.scale, static_cast<int64_t>(gi) * h, col, w[v]);
      g2[v] = load_vec<DT>(p.pre, col);
    }
  }
  float rx_lane = 0.0f, rz_lane = 0.0f;
  // ρ of row i of the unit
  auto scalars = [&](int i, int64_t m, float& rx, float& rz) {
    if ((i & 31) == 0 && i + (t & 31) < n) {
      const int64_t ml = m + static_cast<int64_t>(t & 31) * step;
      rx_lane = p.rstd_x[ml];
      rz_lane = p.rstd_z[ml];
    }
    rx = __shfl_sync(0xffffffffu, rx_lane, i & 31);
    rz = __shfl_sync(0xffffffffu, rz_lane, i & 31);
  };
  // t and x̂ of the row at `at` to u1, u2; returns the sum of their products
  auto open = [&](uint32_t at, float rx, float2 (&u1)[V][4], float2 (&u2)[V][4]) {
    float2 q = both(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (inside<V>(v, v * G + t, nv)) {
        float2 d[4], g[4];
        values<DT>(ring.get(at + o_dy + v * ring.v_bytes), d);
        values<DT>(ring.get(at + o_x + v * ring.v_bytes), u2[v]);
        values<DT>(g2[v], g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u2[v][k] = mul2(u2[v][k], both(rx));
          u1[v][k] = mul2(d[k], g[k]);
          sum2[v][k] = __ffma2_rn(d[k], u2[v][k], sum2[v][k]);
          q = __ffma2_rn(u1[v][k], u2[v][k], q);
        }
      }
    }
    return q.x + q.y;
  };

  float2 b1[V][4], b2[V][4];  // of this row: t, then dr, then t'; x̂, then ẑ
  float rx, rz;
  scalars(0, first, rx, rz);
  cp_wait(S - 2);
  float c1 = row_sum2(make_float2(open(a, rx, b1, b2), 0.0f), red[1]).x * inv_h;
  int64_t m = first;
  for (int i = 0; i < n; ++i, m += step, pos.next()) {
    if (i + S - 1 < n) {
      fetch(a_ahead);
      ahead.next();
      m_ahead += step;
    }
    cp_commit();
    if ((a_ahead += ring.stage_bytes) == a_end) a_ahead = ring.first;
    uint32_t a_next = a + ring.stage_bytes;
    if (a_next == a_end) a_next = ring.first;
    cp_wait(S - 2);
    const int64_t off = (static_cast<int64_t>(pos.r) * h + t * 8) * E;
    float2 q = both(0.0f);
    char* dro = static_cast<char*>(p.chunk[pos.j].dr) + off;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (inside<V>(v, v * G + t, nv)) {
        const uint32_t av = a + v * ring.v_bytes;
        float2 d[4];
        values<DT>(ring.get(av), d);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // ρ·(t − x̂·mean(t·x̂))
          b1[v][k] = __ffma2_rn(__ffma2_rn(b2[v][k], both(-c1), b1[v][k]), both(rx), d[k]);
        store_vec<DT>(dro + v * g_bytes, rounded<DT>(b1[v]));
        float rho = rz;  // with a checkpoint, times the group's power of two
        if (HELD) {
          const uint2 c = ring.get_codes(a + o_codes + v * G * 8);
          const uint32_t byte = words ? ring.get_byte(a + o_byte + v * (G >> 2)) : p.scales[m * groups + ((v * G + t) >> 2)];
          rho = held_vector<DT>(c, byte, rz, b2[v]);
        } else {
          values<DT>(ring.get(av + o_z), b2[v]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          b2[v][k] = mul2(b2[v][k], both(rho));
          sum1[v][k] = __ffma2_rn(b1[v][k], b2[v][k], sum1[v][k]);
          b1[v][k] = mul2(w[v][k], b1[v][k]);
          q = __ffma2_rn(b1[v][k], b2[v][k], q);
        }
      }
    }
    float2 n1[V][4], n2[V][4];  // t and x̂ of the next row
    float rx_next = 0.0f, rz_next = 0.0f, q1 = 0.0f;
    if (i + 1 < n) {
      scalars(i + 1, m + step, rx_next, rz_next);
      q1 = open(a_next, rx_next, n1, n2);
    }
    const float2 c = row_sum2(make_float2(q1, q.x + q.y), red[i & 1]);
    char* dzo = static_cast<char*>(p.chunk[pos.j].dz) + off;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (inside<V>(v, v * G + t, nv)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) b1[v][k] = mul2(__ffma2_rn(b2[v][k], both(-c.y * inv_h), b1[v][k]), both(rz));
        store_vec<DT>(dzo + v * g_bytes, rounded<DT>(b1[v]));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        b1[v][k] = n1[v][k];
        b2[v][k] = n2[v][k];
      }
    }
    c1 = c.x * inv_h;
    rx = rx_next;
    rz = rz_next;
    a = a_next;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int vi = v * G + t;
    if (inside<V>(v, vi, nv)) {
      const int64_t e = static_cast<int64_t>(blockIdx.x) * p.pitch + vi * 8;
      float4* p1 = reinterpret_cast<float4*>(p.part1 + e);
      float4* p2 = reinterpret_cast<float4*>(p.part2 + e);
      p1[0] = make_float4(sum1[v][0].x, sum1[v][0].y, sum1[v][1].x, sum1[v][1].y);
      p1[1] = make_float4(sum1[v][2].x, sum1[v][2].y, sum1[v][3].x, sum1[v][3].y);
      p2[0] = make_float4(sum2[v][0].x, sum2[v][0].y, sum2[v][1].x, sum2[v][1].y);
      p2[1] = make_float4(sum2[v][2].x, sum2[v][2].y, sum2[v][3].x, sum2[v][3].y);
    }
  }
}

// ------------------------------------------------------------------ rows of other widths
// Rows that are not whole 16-byte units take loads of W elements (1, 2 or 4: what their
// addresses allow), neighbouring lanes on neighbouring pieces, N pieces a thread straight
// into registers, and the next row's loads before this row's arithmetic where the registers
// allow (N·W = 8).  32/W lanes are a group of a checkpoint.
template <int DT, int W>
struct Piece {
  static constexpr int BYTES = W * (DT == DT_F32 ? 4 : 2);
  static constexpr int WORDS = (BYTES + 3) / 4;
  uint32_t w[WORDS];
};
template <int DT, int W>
__device__ __forceinline__ Piece<DT, W> load_piece(const void* p, int64_t i) {
  Piece<DT, W> r;
  const char* q = static_cast<const char*>(p) + i * static_cast<int64_t>(sizeof(typename Storage<DT>::T));
  if constexpr (Piece<DT, W>::BYTES == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(q);
  } else if constexpr (Piece<DT, W>::BYTES == 4) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(q);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(q);
    r.w[0] = v.x;
    r.w[1] = v.y;
  }
  return r;
}
template <int DT, int W>
__device__ __forceinline__ void store_piece(void* p, int64_t i, const float* f) {
  typename Storage<DT>::T t[W];
#pragma unroll
  for (int k = 0; k < W; ++k) t[k] = Storage<DT>::from(f[k]);
  char* q = static_cast<char*>(p) + i * static_cast<int64_t>(sizeof(typename Storage<DT>::T));
  if constexpr (Piece<DT, W>::BYTES == 2) {
    *reinterpret_cast<typename Storage<DT>::T*>(q) = t[0];
  } else if constexpr (Piece<DT, W>::BYTES == 4) {
    uint32_t v;
    memcpy(&v, t, 4);
    *reinterpret_cast<uint32_t*>(q) = v;
  } else {
    uint2 v;
    memcpy(&v, t, 8);
    *reinterpret_cast<uint2*>(q) = v;
  }
}
template <int DT, int W>
__device__ __forceinline__ void piece_values(const Piece<DT, W>& r, float* f) {
  typename Storage<DT>::T t[W];
  memcpy(t, r.w, Piece<DT, W>::BYTES);
#pragma unroll
  for (int k = 0; k < W; ++k) f[k] = Storage<DT>::to_f32(t[k]);
}
template <int DT, int W>
__device__ __forceinline__ void load_values(const void* p, int64_t i, float* f) {
  piece_values<DT, W>(load_piece<DT, W>(p, i), f);
}
// scale·g·γ₁ of a piece.
template <int DT, int W>
__device__ __forceinline__ void piece_weight(const void* gate, const void* post, float scale, int64_t goff, int col, float* w) {
  float f[W];
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = scale;
  if (gate) {
    load_values<DT, W>(gate, goff + col, f);
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] *= f[k];
  }
  if (post) {
    load_values<DT, W>(post, col, f);
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] *= f[k];
  }
}

template <int DT, int W, int N>
__global__ void __launch_bounds__(512, 1) piece_fwd_kernel(const __grid_constant__ Fwd p) {
  __shared__ __align__(16) float red[2][16];
  constexpr bool AHEAD = N * W <= 8;
  pdl_enter();
  const int G = blockDim.x, t = threadIdx.x;
  const int h = p.h, groups = (h + 31) >> 5;
  const float inv_h = 1.0f / static_cast<float>(h);
  if (t < 32) red[t >> 4][t & 15] = 0.0f;
  __syncthreads();
  const int gi = blockIdx.x % p.gate_rows;
  const int64_t first = static_cast<int64_t>(blockIdx.x / p.gate_rows) * p.gate_rows + gi;
  const int step = p.K * p.gate_rows;
  Pos pos(static_cast<int>(first), step, p.rpc), next = pos;
  // a piece behind the row's end loads the row's first instead, and counts as zero: no load
  // waits for a branch
  auto inner = [&](int i) {
    const int col = (i * G + t) * W;
    return col < h ? col : 0;
  };
  Piece<DT, W> rn[N] = {}, zn[N] = {};
  auto fetch = [&](const Pos& at) {
    const int64_t off = static_cast<int64_t>(at.r) * h;
#pragma unroll
    for (int i = 0; i < N; ++i) rn[i] = load_piece<DT, W>(p.chunk[at.j].r, off + inner(i));
    if (p.has_z) {
#pragma unroll
      for (int i = 0; i < N; ++i) zn[i] = load_piece<DT, W>(p.chunk[at.j].z, off + inner(i));
    }
  };
  if (AHEAD) fetch(next);
  float w[N][W], g2[N][W];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int col = (i * G + t) * W;
#pragma unroll
    for (int k = 0; k < W; ++k) w[i][k] = g2[i][k] = 0.0f;
    if (col < h) {
      piece_weight<DT, W>(p.gate, p.post, p.scale, static_cast<int64_t>(gi) * h, col, w[i]);
      if (p.pre) load_values<DT, W>(p.pre, col, g2[i]);
    }
  }
  for (int64_t m = first; m < p.rows; m += step, pos.next()) {
    if (!AHEAD) fetch(pos);
    float x[N][W], z[N][W];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      piece_values<DT, W>(rn[i], x[i]);
      piece_values<DT, W>(zn[i], z[i]);
      if ((i * G + t) * W >= h) {
#pragma unroll
        for (int k = 0; k < W; ++k) x[i][k] = z[i][k] = 0.0f;
      }
    }
    next.next();
    if (AHEAD && m + step < p.rows) fetch(next);
    const int64_t off = static_cast<int64_t>(pos.r) * h;
    float rz = 1.0f;
    if (p.post) {
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) q = fmaf(z[i][k], z[i][k], q);
      rz = 1.0f / sqrtf(row_sum(q, red[0]) * inv_h + p.eps);
      if (t == 0) p.rstd_z[m] = rz;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int col = (i * G + t) * W;
      if (p.has_z) {
#pragma unroll
        for (int k = 0; k < W; ++k)
          x[i][k] = Storage<DT>::to_f32(Storage<DT>::from(fmaf(w[i][k], z[i][k] * rz, x[i][k])));
        if (col < h) store_piece<DT, W>(p.chunk[pos.j].x, off + col, x[i]);
      }
      if (col < h) {  // (behind the row's end an infinite ρ would leave NaN)
#pragma unroll
        for (int k = 0; k < W; ++k) q = fmaf(x[i][k], x[i][k], q);
      }
      if (p.codes) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < W; ++k) top = max(top, ckpt_abs(z[i][k]));
#pragma unroll
        for (int o = 1; o < 32 / W; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t byte = ckpt_byte(top);
        if (col < h) {
          float four[4] = {};
#pragma unroll
          for (int k = 0; k < W; ++k) four[k] = z[i][k];
          const uint32_t c = ckpt_encode4(four, ckpt_inverse(byte));
          uint8_t* q8 = p.codes + m * h + col;
          if constexpr (W == 4)
            *reinterpret_cast<uint32_t*>(q8) = c;
          else if constexpr (W == 2)
            *reinterpret_cast<uint16_t*>(q8) = static_cast<uint16_t>(c);
          else
            *q8 = static_cast<uint8_t>(c);
          if ((col & 31) == 0) p.scales[m * groups + (col >> 5)] = static_cast<uint8_t>(byte);
        }
      }
    }
    if (p.pre) {
      const float rx = 1.0f / sqrtf(row_sum(q, red[1]) * inv_h + p.eps);
      if (t == 0) p.rstd_x[m] = rx;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int col = (i * G + t) * W;
#pragma unroll
        for (int k = 0; k < W; ++k) x[i][k] = x[i][k] * rx * g2[i][k];
        if (col < h) store_piece<DT, W>(p.chunk[pos.j].y, off + col, x[i]);
      }
    }
    if (!p.post || !p.pre) __syncthreads();  // one sum a row: nothing else frees its array
  }
}

// The column sums and weights of 16 elements a thread are more than its registers hold:
// they are in shared memory then, each thread's own.
template <int DT, int W, int N>
__global__ void __launch_bounds__(512, 1) piece_bwd_kernel(const __grid_constant__ Bwd p) {
  extern __shared__ __align__(16) float own_smem[];
  __shared__ __align__(16) float red[2][16];
  constexpr bool OWN = N * W > 8;
  constexpr bool AHEAD = N * W <= 8;
  pdl_enter();
  const int G = blockDim.x, t = threadIdx.x;
  const int h = p.h, groups = (h + 31) >> 5;
  const float inv_h = 1.0f / static_cast<float>(h);
  if (t < 32) red[t >> 4][t & 15] = 0.0f;
  __syncthreads();
  const int gi = blockIdx.x % p.gate_rows;
  const int64_t first = static_cast<int64_t>(blockIdx.x / p.gate_rows) * p.gate_rows + gi;
  const int step = p.K * p.gate_rows;
  const bool pre = p.pre != nullptr, post = p.post != nullptr;
  Pos pos(static_cast<int>(first), step, p.rpc), next = pos;
  auto inner = [&](int i) {  // as in the forward
    const int col = (i * G + t) * W;
    return col < h ? col : 0;
  };
  Piece<DT, W> dxn[N] = {}, dyn[N] = {}, xn[N] = {}, zn[N] = {};
  uint32_t cn[N] = {}, bn[N] = {};
  float rxn = 0.0f, rzn = 1.0f;
  auto fetch = [&](const Pos& at, int64_t m) {
    const int64_t off = static_cast<int64_t>(at.r) * h;
    if (pre) rxn = p.rstd_x[m];
    if (post) rzn = p.rstd_z[m];
    if (p.has_dx) {
#pragma unroll
      for (int i = 0; i < N; ++i) dxn[i] = load_piece<DT, W>(p.chunk[at.j].dx, off + inner(i));
    }
    if (pre) {
#pragma unroll
      for (int i = 0; i < N; ++i) dyn[i] = load_piece<DT, W>(p.chunk[at.j].dy, off + inner(i));
#pragma unroll
      for (int i = 0; i < N; ++i) xn[i] = load_piece<DT, W>(p.chunk[at.j].x, off + inner(i));
    }
    if (p.codes) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint8_t* q8 = p.codes + m * h + inner(i);
        if constexpr (W == 4)
          cn[i] = *reinterpret_cast<const uint32_t*>(q8);
        else if constexpr (W == 2)
          cn[i] = *reinterpret_cast<const uint16_t*>(q8);
        else
          cn[i] = *q8;
        bn[i] = p.scales[m * groups + (inner(i) >> 5)];
      }
    } else if (p.has_z) {
#pragma unroll
      for (int i = 0; i < N; ++i) zn[i] = load_piece<DT, W>(p.chunk[at.j].z, off + inner(i));
    }
  };
  if (AHEAD) fetch(next, first);
  float kept[4][OWN ? 1 : N][W];
  enum { WEIGHT, GAMMA2, SUM1, SUM2 };
  auto get = [&](int a, int i, int k) {
    if constexpr (OWN) return own_smem[((a * N + i) * W + k) * G + t];
    else return kept[a][i][k];
  };
  auto set = [&](int a, int i, int k, float v) {
    if constexpr (OWN) own_smem[((a * N + i) * W + k) * G + t] = v;
    else kept[a][i][k] = v;
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int col = (i * G + t) * W;
    float wi[W] = {}, gi2[W] = {};
    if (col < h) {
      piece_weight<DT, W>(p.gate, p.post, p.scale, static_cast<int64_t>(gi) * h, col, wi);
      if (pre) load_values<DT, W>(p.pre, col, gi2);
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
      set(WEIGHT, i, k, wi[k]);
      set(GAMMA2, i, k, gi2[k]);
      set(SUM1, i, k, 0.0f);
      set(SUM2, i, k, 0.0f);
    }
  }
  for (int64_t m = first; m < p.rows; m += step, pos.next()) {
    if (!AHEAD) fetch(pos, m);
    const float rx = rxn, rz = rzn;
    float d[N][W], b1[N][W], b2[N][W], z[N][W];  // dx; t, then dr and t'; x̂; ẑ
    float c1 = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float y[W];
      piece_values<DT, W>(dxn[i], d[i]);
      piece_values<DT, W>(dyn[i], y);
      piece_values<DT, W>(xn[i], b2[i]);
      if (p.codes) {
        float four[4];
        ckpt_decode4(cn[i], ckpt_scale(bn[i]), four);
#pragma unroll
        for (int k = 0; k < W; ++k) z[i][k] = ckpt_in_range<DT>(four[k]);
      } else {
        piece_values<DT, W>(zn[i], z[i]);
      }
      if ((i * G + t) * W >= h) {
#pragma unroll
        for (int k = 0; k < W; ++k) d[i][k] = y[k] = b2[i][k] = z[i][k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < W; ++k) {
        b2[i][k] *= rx;
        b1[i][k] = y[k] * get(GAMMA2, i, k);
        set(SUM2, i, k, fmaf(y[k], b2[i][k], get(SUM2, i, k)));
        q = fmaf(b1[i][k], b2[i][k], q);
      }
    }
    next.next();
    if (AHEAD && m + step < p.rows) fetch(next, m + step);
    if (pre) c1 = row_sum(q, red[0]) * inv_h;
    const int64_t off = static_cast<int64_t>(pos.r) * h;
    q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int col = (i * G + t) * W;
#pragma unroll
      for (int k = 0; k < W; ++k) b1[i][k] = pre ? fmaf(fmaf(b2[i][k], -c1, b1[i][k]), rx, d[i][k]) : d[i][k];
      if (col < h) {
        store_piece<DT, W>(p.chunk[pos.j].dr, off + col, b1[i]);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          z[i][k] *= rz;
          set(SUM1, i, k, fmaf(b1[i][k], z[i][k], get(SUM1, i, k)));
          b1[i][k] *= get(WEIGHT, i, k);
          q = fmaf(b1[i][k], z[i][k], q);
        }
      }
    }
    if (p.has_dz) {
      float c2 = 0.0f;
      if (post) c2 = row_sum(q, red[1]) * inv_h;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int col = (i * G + t) * W;
        if (col < h) {
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (post) b1[i][k] = fmaf(z[i][k], -c2, b1[i][k]) * rz;
          store_piece<DT, W>(p.chunk[pos.j].dz, off + col, b1[i]);
        }
      }
    }
    if (!pre || !post) __syncthreads();  // one sum a row: nothing else frees its array (post is with dz only)
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int col = (i * G + t) * W;
    if (col < h) {
      const int64_t e = static_cast<int64_t>(blockIdx.x) * p.pitch + col;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        if (p.has_z) p.part1[e + k] = get(SUM1, i, k);
        if (pre) p.part2[e + k] = get(SUM2, i, k);
      }
    }
  }
}

// ------------------------------------------------------------------ any row
// One row of the unit at a time on the whole CTA, an element a thread and step: any h
// and alignment.  A warp's 32 columns are a group of the checkpoint.
constexpr int ANY_THREADS = 256;

template <int DT>
__global__ void __launch_bounds__(ANY_THREADS) any_fwd_kernel(const __grid_constant__ Fwd p) {
  __shared__ float red[2][32];
  pdl_enter();
  const int h = p.h, h32 = (h + 31) & ~31, groups = h32 >> 5;
  const float inv_h = 1.0f / static_cast<float>(h);
  const int gi = blockIdx.x % p.gate_rows, k = blockIdx.x / p.gate_rows;
  const int64_t goff = static_cast<int64_t>(gi) * h;
  const int64_t first = static_cast<int64_t>(k) * p.gate_rows + gi;  // every unit has a row: K ≤ rows/gate_rows
  const int step = p.K * p.gate_rows;
  Pos pos(static_cast<int>(first), step, p.rpc);
  for (int64_t m = first; m < p.rows; m += step, pos.next()) {
    const int64_t off = static_cast<int64_t>(pos.r) * h;
    const void* r = p.chunk[pos.j].r;
    const void* z = p.chunk[pos.j].z;
    float rz = 1.0f;
    if (p.post) {
      float q = 0.0f;
      for (int c = threadIdx.x; c < h; c += ANY_THREADS) {
        const float v = at<DT>(z, off + c);
        q = fmaf(v, v, q);
      }
      rz = 1.0f / sqrtf(block_sum(q, red[0]) * inv_h + p.eps);
      if (threadIdx.x == 0) p.rstd_z[m] = rz;
    }
    float q = 0.0f;
    for (int c = threadIdx.x; c < h32; c += ANY_THREADS) {
      const bool in = c < h;
      float xv = in ? at<DT>(r, off + c) : 0.0f;
      if (p.has_z) {
        const float zv = in ? at<DT>(z, off + c) : 0.0f;
        if (in) {
          float cg = p.scale;
          if (p.gate) cg *= at<DT>(p.gate, goff + c);
          if (p.post) cg *= at<DT>(p.post, c);
          xv = Storage<DT>::to_f32(Storage<DT>::from(fmaf(cg, zv * rz, xv)));
          put<DT>(p.chunk[pos.j].x, off + c, xv);
        }
        if (p.codes) {
          const uint32_t byte = ckpt_byte(__reduce_max_sync(0xffffffffu, ckpt_abs(zv)));
          const float one[4] = {zv, 0.0f, 0.0f, 0.0f};
          if (in) p.codes[m * h + c] = static_cast<uint8_t>(ckpt_encode4(one, ckpt_inverse(byte)));
          if ((c & 31) == 0) p.scales[m * groups + (c >> 5)] = static_cast<uint8_t>(byte);
        }
      }
      q = fmaf(xv, xv, q);
    }
    if (p.pre) {
      const float rx = 1.0f / sqrtf(block_sum(q, red[1]) * inv_h + p.eps);
      if (threadIdx.x == 0) p.rstd_x[m] = rx;
      const void* x = p.has_z ? p.chunk[pos.j].x : r;  // this thread's own elements again
      for (int c = threadIdx.x; c < h; c += ANY_THREADS)
        put<DT>(p.chunk[pos.j].y, off + c, at<DT>(x, off + c) * rx * at<DT>(p.pre, c));
    }
    if (!p.post || !p.pre) __syncthreads();  // one sum a row: nothing else frees its array
  }
}

template <int DT>
__global__ void __launch_bounds__(ANY_THREADS) any_bwd_kernel(const __grid_constant__ Bwd p) {
  __shared__ float red[2][32];
  pdl_enter();
  const int h = p.h, groups = (h + 31) >> 5;
  const float inv_h = 1.0f / static_cast<float>(h);
  const int gi = blockIdx.x % p.gate_rows, k = blockIdx.x / p.gate_rows;
  const int64_t goff = static_cast<int64_t>(gi) * h;
  float* part1 = p.part1 + static_cast<int64_t>(blockIdx.x) * p.pitch;
  float* part2 = p.part2 + static_cast<int64_t>(blockIdx.x) * p.pitch;
  const int64_t first = static_cast<int64_t>(k) * p.gate_rows + gi;
  const int step = p.K * p.gate_rows;
  Pos pos(static_cast<int>(first), step, p.rpc);
  for (int64_t m = first; m < p.rows; m += step, pos.next()) {
    const int64_t off = static_cast<int64_t>(pos.r) * h;
    const int j = pos.j;
    const float rx = p.pre ? p.rstd_x[m] : 0.0f, rz = p.post ? p.rstd_z[m] : 1.0f;
    float c1 = 0.0f;
    if (p.pre) {
      float q = 0.0f;
      for (int c = threadIdx.x; c < h; c += ANY_THREADS)
        q = fmaf(at<DT>(p.chunk[j].dy, off + c) * at<DT>(p.pre, c), at<DT>(p.chunk[j].x, off + c) * rx, q);
      c1 = block_sum(q, red[0]) * inv_h;
    }
    auto z_at = [&](int c) {
      if (p.codes == nullptr) return at<DT>(p.chunk[j].z, off + c);
      float v[4];
      ckpt_decode4(p.codes[m * h + c], ckpt_scale(p.scales[m * groups + (c >> 5)]), v);
      return ckpt_in_range<DT>(v[0]);
    };
    auto dr_at = [&](int c) {
      float d = p.has_dx ? at<DT>(p.chunk[j].dx, off + c) : 0.0f;
      if (p.pre)
        d += rx * (at<DT>(p.chunk[j].dy, off + c) * at<DT>(p.pre, c) - at<DT>(p.chunk[j].x, off + c) * rx * c1);
      return d;
    };
    auto cg_at = [&](int c) {
      float g = p.scale;
      if (p.gate) g *= at<DT>(p.gate, goff + c);
      if (p.post) g *= at<DT>(p.post, c);
      return g;
    };
    float q = 0.0f;
    for (int c = threadIdx.x; c < h; c += ANY_THREADS) {
      const float old1 = m == first ? 0.0f : part1[c], old2 = m == first ? 0.0f : part2[c];
      float s1 = 0.0f, s2 = 0.0f;
      if (p.has_z) {
        const float d = dr_at(c), zh = z_at(c) * rz;
        s1 = d * zh;
        q = fmaf(cg_at(c) * d, zh, q);
      }
      if (p.pre) s2 = at<DT>(p.chunk[j].dy, off + c) * (at<DT>(p.chunk[j].x, off + c) * rx);
      part1[c] = old1 + s1;
      part2[c] = old2 + s2;
    }
    const float c2 = p.post && p.has_dz ? block_sum(q, red[1]) * inv_h : 0.0f;
    for (int c = threadIdx.x; c < h; c += ANY_THREADS) {
      const float d = dr_at(c);  // before dr, which may be dx, is written
      if (p.has_dz) {
        float t = cg_at(c) * d;
        if (p.post) t = rz * (t - z_at(c) * rz * c2);
        put<DT>(p.chunk[j].dz, off + c, t);
      }
      put<DT>(p.chunk[j].dr, off + c, d);
    }
    if (!p.pre || !p.post || !p.has_dz) __syncthreads();  // one sum a row: nothing else frees its array
  }
}

// ------------------------------------------------------------------ column sums
// dγ₂[c] = Σ_u part2[u][c]; S[gi][c] = Σ_k part1[k·gate_rows + gi][c], dgate = α·γ₁·S and
// dγ₁[c] = α·Σ_gi g·S.  A CTA takes 32 columns of one of the two arrays (blockIdx.y): 8
// lanes of 4 columns on a unit, 4 units a warp at once, and four gates together, so that
// the few hundred units of a backward are a handful of independent loads a thread.  The
// sums are then added across the warp, and in warp order across the CTA: the same
// association on every call.
constexpr int COL_WARPS = 16;  // at most
constexpr int COL_GATES = 4;

template <int DT>
__global__ void __launch_bounds__(32 * COL_WARPS) columns_kernel(const __grid_constant__ Bwd p, float* dpost, float* dpre,
                                                                 float* dgate) {
  __shared__ __align__(16) float red[COL_GATES][COL_WARPS][32];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t h = p.h;
  const int c0 = blockIdx.x * 32 + (lane & 7) * 4, c = blockIdx.x * 32 + lane;
  const bool pre = blockIdx.y == 0;
  if (pre ? dpre == nullptr : dpost == nullptr && dgate == nullptr) return;
  // dγ₂ is the sum of all units: as of one gate
  const int gates = pre ? 1 : p.gate_rows, n = pre ? p.K * p.gate_rows : p.K;
  const float* part = (pre ? p.part2 : p.part1) + c0;
  const int64_t pitch = gates * p.pitch;
  const float gamma = !pre && p.post && c < p.h ? at<DT>(p.post, c) : 1.0f;
  float post = 0.0f;  // of the gates that this warp finishes: gi ≡ warp (mod COL_GATES)
  for (int g0 = 0; g0 < gates; g0 += COL_GATES) {
    const int count = min(gates - g0, COL_GATES);
    float4 a[COL_GATES] = {};
    if (c0 < p.pitch) {
#pragma unroll 2
      for (int k = warp * 4 + (lane >> 3); k < n; k += warps * 4) {
#pragma unroll
        for (int g = 0; g < COL_GATES; ++g) {
          if (g < count) {
            const float4 v = *reinterpret_cast<const float4*>(part + k * pitch + (g0 + g) * p.pitch);
            a[g].x += v.x;
            a[g].y += v.y;
            a[g].z += v.z;
            a[g].w += v.w;
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < COL_GATES; ++g) {
      if (g < count) {
#pragma unroll
        for (int o = 8; o < 32; o *= 2) {
          a[g].x += __shfl_xor_sync(0xffffffffu, a[g].x, o);
          a[g].y += __shfl_xor_sync(0xffffffffu, a[g].y, o);
          a[g].z += __shfl_xor_sync(0xffffffffu, a[g].z, o);
          a[g].w += __shfl_xor_sync(0xffffffffu, a[g].w, o);
        }
        if (lane < 8) *reinterpret_cast<float4*>(&red[g][warp][lane * 4]) = a[g];
      }
    }
    __syncthreads();
    if (warp < count && c < p.h) {
      float s = 0.0f;
      for (int i = 0; i < warps; ++i) s += red[warp][i][lane];
      const int64_t gi = g0 + warp;
      if (pre)
        dpre[c] = s;
      else if (dgate)
        dgate[gi * h + c] = p.scale * gamma * s;
      if (!pre) post = fmaf(p.gate ? at<DT>(p.gate, gi * h + c) : 1.0f, s, post);
    }
  }
  if (pre || dpost == nullptr) return;
  __syncthreads();
  if (warp < COL_GATES) red[0][warp][lane] = post;
  __syncthreads();
  if (warp == 0 && c < p.h) {
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < COL_GATES; ++g) s += red[0][g][lane];
    dpost[c] = p.scale * s;
  }
}

size_t esize(int dtype) { return dtype == DT_F32 ? 4 : 2; }

int64_t pitch_of(int64_t h) { return (h + 3) / 4 * 4; }

// Units of a gate: see max_units; never more than the gate's rows.
int64_t units_of_a_gate(int64_t rows, int64_t gate_rows, int64_t h) {
  if (rows == 0 || gate_rows == 0) return 0;
  return std::max<int64_t>(1, std::min(rows / gate_rows, max_units(h) / gate_rows));
}

int check_sizes(int64_t s, int64_t b, int64_t h, int tp, int dtype) {
  if (s < 0 || b < 0 || h <= 0) return set_error(TPMLP_ERR_INVALID_ARG, "s, b >= 0 and h >= 1 required");
  if (tp < 1 || tp > TPMLP_MAX_TP) return set_error(TPMLP_ERR_INVALID_ARG, "tp must be in [1, 64]");
  if (dtype < DT_F32 || dtype > DT_BF16) return set_error(TPMLP_ERR_INVALID_ARG, "unknown dtype");
  if (s > (1ll << 31) || b > (1ll << 31) || s * b >= (1ll << 31) - 65536 || h >= (1ll << 28))
    return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  if (s % tp != 0)
    return set_error(TPMLP_ERR_NOT_DIVISIBLE, "First dimension of the tensor should be divisible by tensor parallel size");
  return TPMLP_OK;
}

int check_one(const void* p, size_t align, const char* name) {
  if (p == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align != 0) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " is misaligned");
  return TPMLP_OK;
}

int check_arr(const void* const* a, int n, size_t align, const char* name) {
  if (a == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, std::string(name) + " array is NULL");
  for (int i = 0; i < n; ++i) {
    const int rc = check_one(a[i], align, name);
    if (rc != TPMLP_OK) return rc;
  }
  return TPMLP_OK;
}

int check_norms(const tpmlp_rms_residual* n, int64_t b, int dtype) {
  if (n == nullptr) return set_error(TPMLP_ERR_INVALID_ARG, "norms is NULL");
  const size_t e = esize(dtype);
  int rc;
  if (n->post_gamma && (rc = check_one(n->post_gamma, e, "post_gamma"))) return rc;
  if (n->pre_gamma && (rc = check_one(n->pre_gamma, e, "pre_gamma"))) return rc;
  if (n->gate && (rc = check_one(n->gate, e, "gate"))) return rc;
  if (!(n->eps >= 0.0f)) return set_error(TPMLP_ERR_INVALID_ARG, "eps must be >= 0");
  if (n->gate && n->gate_rows != 1 && n->gate_rows != b)
    return set_error(TPMLP_ERR_INVALID_ARG, "gate_rows must be 1 or b");
  return TPMLP_OK;
}

// The chunks' addresses or'ed: what all of them are aligned to.
uintptr_t address_bits(const void* const* a, int n) {
  uintptr_t bits = 0;
  for (int j = 0; j < n; ++j) bits |= reinterpret_cast<uintptr_t>(a[j]);
  return bits;
}
uintptr_t address_bits(const tpmlp_rms_residual* n) {
  return reinterpret_cast<uintptr_t>(n->post_gamma) | reinterpret_cast<uintptr_t>(n->pre_gamma) |
         reinterpret_cast<uintptr_t>(n->gate);
}

// A row of nv vectors on G threads of V each, and the stages that shared memory holds.
struct RowShape {
  int V = 0, G = 0, stages = 0, ctas = 0;  // ctas: resident on the device
  size_t smem = 0;
};

// nv vectors, V a thread.
RowShape shape_of(int64_t nv, int V) {
  RowShape r;
  r.V = V;
  r.G = static_cast<int>(((nv + V - 1) / V + 31) / 32 * 32);
  return r;
}

// CTAs of G threads that an SM's registers hold: each of its four parts has 512 a lane.  A
// persistent grid of more than are resident would leave the rest for a second wave.
int ctas_by_registers(int regs, int G) {
  const int warps = 4 * (512 / ((regs + 7) / 8 * 8));
  return std::max(1, std::min({warps / (G / 32), 2048 / G, 24}));
}

// Stages and resident CTAs: `regs` registers a thread, `nin` inputs of `unit` bytes a vector.
// As many CTAs as registers and threads allow while each could keep three stages, then
// the stages that have AHEAD_BYTES in flight; fewer than two (and `beside`): no shape.
bool fill_shape(const DeviceInfo& dev, int regs, int nin, int unit, int beside, RowShape* r) {
  const size_t stage = static_cast<size_t>(nin) * r->V * r->G * unit;
  const size_t room = dev.smem_per_sm, cta_max = dev.max_smem_optin;
  const size_t fixed = 1024 + 256;  // the system's share of a CTA and the sums' arrays
  int ctas = ctas_by_registers(regs, r->G);
  while (ctas > 1 && ctas * (3 * stage + fixed) > room) --ctas;
  const size_t fit = (std::min(room / ctas, cta_max + 1024) - fixed) / stage;
  if (fit < static_cast<size_t>(2 + beside)) return false;
  const size_t want = 1 + beside + (AHEAD_BYTES + ctas * stage - 1) / (ctas * stage);
  const int stages = static_cast<int>(std::min({fit, want, static_cast<size_t>(MAX_STAGES)}));
  r->stages = stages;
  r->smem = stages * stage;
  r->ctas = ctas * dev.num_sms;
  return true;
}

// A kernel's registers, asked for once.
template <auto Kernel>
int kernel_regs() {
  static std::atomic<int> known{0};
  int n = known.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, Kernel) != cudaSuccess) return 128;
    n = a.numRegs;
    known.store(n, std::memory_order_relaxed);
  }
  return n;
}

// The units of a launch: at most `most` (as many as are resident; backward: max_units),
// over the gates.
template <typename P>
unsigned deal_units(P* p, int most) {
  if (std::is_same<P, Bwd>::value) most = std::min(most, max_units(p->h));
  p->K = std::max(1, std::min(p->rows / p->gate_rows, most / p->gate_rows));
  return static_cast<unsigned>(p->K * p->gate_rows);
}

// beside: rows in work beside the one whose stage is freed next; cluster: CTAs of a row.
template <auto Kernel, typename P>
cudaError_t launch_rows(P& p, RowShape r, int nin, int unit, const DeviceInfo& dev, cudaStream_t st, bool* done,
                        int beside = 0, int cluster = 1) {
  *done = fill_shape(dev, kernel_regs<Kernel>(), nin, unit, beside, &r);
  if (!*done) return cudaSuccess;
  static SmemDone smem_done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(Kernel), dev.max_smem_optin - 256, dev, &smem_done);
  if (e != cudaSuccess) return e;
  p.stages = r.stages;
  // (clusters of four do not fill every group of SMs to the last)
  const unsigned units = deal_units(&p, std::max(1, r.ctas / cluster - (cluster > 2 ? 2 : 0)));
  return launch_pdl(Kernel, dim3(units * cluster), static_cast<unsigned>(r.G), r.smem, st, cluster, p);
}

// The shape of one CTA's share of a row.
RowShape share_of(int64_t nv, int cluster, int V) { return shape_of(((nv + cluster - 1) / cluster + 3) / 4 * 4, V); }

// Whether V vectors a thread leave at most a quarter of the lanes idle, all in their last vector.
bool fills(int64_t nv, int V) {
  const int64_t G = shape_of(nv, V).G;
  return 3 * G * V <= 4 * nv && (V - 1) * G <= nv;
}

// Vectors a thread: two (float32: one); four on half the threads cost more (2048 columns
// 50.8 µs against 46.0, 4096: 50.2 against 44.3, 8192: 49.3 against 45.4, 134 and 268 MB
// each).  Three from 4104 to 6144 columns, where two leave an SM one CTA of 9 to 12 warps
// (6144: 39.7 µs against 37.4), four where two would be more than 512 threads, and one
// for rows that two would not fill.
int forward_vectors(int64_t nv, bool f32) {
  if (f32) return nv <= 512 ? 1 : 2;
  if (nv > 512) return nv <= 768 ? 3 : nv <= 1024 ? 2 : 4;
  return nv > 256 || fills(nv, 2) ? 2 : 1;
}

template <int DT>
cudaError_t forward_rows(Fwd& p, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  const int64_t nv = p.h / 8;
  const int nin = 1 + p.has_z, unit = 16 * Vec<DT>::N;
  *done = false;
  // rows that a CTA's 512 threads cannot hold go to a cluster of two or four
  constexpr int WIDE = DT == DT_F32 ? 2 : 4;
  if (share_of(nv, 1, WIDE).G > 512) {
    const RowShape two = share_of(nv, 2, WIDE), four = share_of(nv, 4, WIDE);
    if (two.G <= 512) return launch_rows<vec_fwd_kernel<DT, WIDE, false, 2>>(p, two, nin, unit, dev, st, done, 0, 2);
    if (four.G <= 512) return launch_rows<vec_fwd_kernel<DT, WIDE, false, 4>>(p, four, nin, unit, dev, st, done, 0, 4);
    return cudaSuccess;
  }
  const int V = forward_vectors(nv, DT == DT_F32);
  const RowShape r = shape_of(nv, V);
  if constexpr (DT != DT_F32) {
    // alone on its SM a CTA gains from fewer instructions (8192 columns 45.3 -> 43.1 µs, with a checkpoint 55.2 -> 51.9);
    // with neighbours to fill its waits it is 5% either way
    if (V == 2 && r.G > 384 && p.has_z && p.post && p.pre)
      return launch_rows<vec_fwd_kernel<DT, 2, true>>(p, r, nin, unit, dev, st, done);
    if (V == 4) return launch_rows<vec_fwd_kernel<DT, 4, false>>(p, r, nin, unit, dev, st, done);
    if (V == 3) return launch_rows<vec_fwd_kernel<DT, 3, false>>(p, r, nin, unit, dev, st, done);
  }
  if (V == 2) return launch_rows<vec_fwd_kernel<DT, 2, false>>(p, r, nin, unit, dev, st, done);
  return launch_rows<vec_fwd_kernel<DT, 1, false>>(p, r, nin, unit, dev, st, done);
}

template <int DT>
cudaError_t backward_rows(Bwd& p, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  const int64_t nv = p.h / 8;
  const int nin = p.has_dx + 2 * (p.pre != nullptr) + p.has_z, unit = 16 * Vec<DT>::N;
  const bool held = nin == 4 && p.post && p.codes;  // (a norm behind the block comes with dz)
  *done = false;
  // wider rows: a cluster of two or four CTAs (float32: so many that a share's rows fit a ring)
  constexpr int WIDE = DT == DT_F32 ? 1 : 2;
  const RowShape one = share_of(nv, 1, DT == DT_F32 ? 2 : WIDE), two = share_of(nv, 2, WIDE), four = share_of(nv, 4, WIDE);
  if (one.G > (DT == DT_F32 ? 384 : 512)) {
    if (two.G <= 512)
      return held ? launch_rows<vec_bwd_kernel<DT, WIDE, true, 2>>(p, two, nin, unit, dev, st, done, 0, 2)
                  : launch_rows<vec_bwd_kernel<DT, WIDE, false, 2>>(p, two, nin, unit, dev, st, done, 0, 2);
    if (four.G <= 512)
      return held ? launch_rows<vec_bwd_kernel<DT, WIDE, true, 4>>(p, four, nin, unit, dev, st, done, 0, 4)
                  : launch_rows<vec_bwd_kernel<DT, WIDE, false, 4>>(p, four, nin, unit, dev, st, done, 0, 4);
    return cudaSuccess;
  }
  const int V = DT == DT_F32 ? (nv <= 512 ? 1 : 2) : fills(nv, 2) || nv > 256 ? 2 : 1;
  const RowShape r = shape_of(nv, V);
  if constexpr (DT != DT_F32)  // (its third and fourth row would not fit)
    if (nin == 4 && p.post && V == 2 && r.G > 256 && r.G <= 384)
      return held ? launch_rows<vec_bwd_pair_kernel<DT, true>>(p, r, nin, unit, dev, st, done, 1)
                  : launch_rows<vec_bwd_pair_kernel<DT, false>>(p, r, nin, unit, dev, st, done, 1);
  if (V == 1)
    return held ? launch_rows<vec_bwd_kernel<DT, 1, true>>(p, r, nin, unit, dev, st, done)
                : launch_rows<vec_bwd_kernel<DT, 1, false>>(p, r, nin, unit, dev, st, done);
  return held ? launch_rows<vec_bwd_kernel<DT, 2, true>>(p, r, nin, unit, dev, st, done)
              : launch_rows<vec_bwd_kernel<DT, 2, false>>(p, r, nin, unit, dev, st, done);
}

// The arrays of a call, outputs first: an output may share memory with nothing but, where
// it is allowed, the same chunk of one input.
class Apart {
 public:
  // n chunks of `bytes`; may_be: the index of the array (in the order of adding) that this input's chunks may equal; −1: none
  void add(const void* const* a, int n, int64_t bytes, bool output, int may_be = -1) {
    for (int j = 0; j < n; ++j)
      one_[count_++] = {reinterpret_cast<uintptr_t>(a[j]), reinterpret_cast<uintptr_t>(a[j]) + static_cast<uintptr_t>(bytes),
                        arrays_, j, output, may_be};
    ++arrays_;
  }
  // An array that may be NULL: not there.
  void add(const void* a, int64_t bytes, bool output) {
    if (a != nullptr) add(&a, 1, bytes, output);
  }
  int check(const char* what) const {
    for (int i = 0; i < count_ && one_[i].output; ++i) {
      for (int j = 0; j < count_; ++j) {
        const One &o = one_[i], &c = one_[j];
        if (i == j || o.at >= c.end || c.at >= o.end) continue;
        if (c.at == o.at && c.index == o.index && c.may_be == o.array) continue;
        return set_error(TPMLP_ERR_INVALID_ARG, std::string(what) + ": an output must not overlap another array");
      }
    }
    return TPMLP_OK;
  }

 private:
  struct One {
    uintptr_t at, end;
    int array, index;
    bool output;
    int may_be;
  };
  One one_[6 * TPMLP_MAX_TP + 16];
  int count_ = 0, arrays_ = 0;
};

int report(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return TPMLP_OK;
  return set_error(TPMLP_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}


// Elements of a piece: what the width and the addresses allow (`bits`: all of them or'ed).
int piece_width(int64_t h, uintptr_t bits, uintptr_t code_bits, size_t e) {
  for (int w = e == 4 ? 2 : 4; w > 1; w /= 2)
    if (h % w == 0 && bits % (w * e) == 0 && code_bits % w == 0) return w;
  return 1;
}

template <auto Kernel, typename P>
cudaError_t launch_pieces(P& p, int per_thread, const DeviceInfo& dev, cudaStream_t st) {
  const int G = (p.h + per_thread * 32 - 1) / (per_thread * 32) * 32;
  int ctas = ctas_by_registers(kernel_regs<Kernel>(), G);
  size_t smem = 0;
  if (std::is_same<P, Bwd>::value && per_thread > 8) {
    smem = static_cast<size_t>(4 * per_thread * G) * sizeof(float);
    static SmemDone done;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(Kernel), dev.max_smem_optin - 256, dev, &done);
    if (e != cudaSuccess) return e;
    ctas = std::min<int>(ctas, std::max<int>(1, static_cast<int>(dev.smem_per_sm / (smem + 1280))));
  }
  const unsigned grid = deal_units(&p, ctas * dev.num_sms);
  return launch_pdl(Kernel, dim3(grid), static_cast<unsigned>(G), smem, st, 1, p);
}

// Rows of up to 16 elements a thread on 512 threads; false: wider.
template <int DT, int W>
bool forward_pieces(Fwd& p, const DeviceInfo& dev, cudaStream_t st, cudaError_t* err) {
  if (p.h <= 8 * 512)
    *err = launch_pieces<piece_fwd_kernel<DT, W, 8 / W>>(p, 8, dev, st);
  else if (p.h <= 16 * 512)
    *err = launch_pieces<piece_fwd_kernel<DT, W, 16 / W>>(p, 16, dev, st);
  else
    return false;
  return true;
}
template <int DT, int W>
bool backward_pieces(Bwd& p, const DeviceInfo& dev, cudaStream_t st, cudaError_t* err) {
  if (p.h <= 8 * 512)
    *err = launch_pieces<piece_bwd_kernel<DT, W, 8 / W>>(p, 8, dev, st);
  else if (p.h <= 16 * 512)
    *err = launch_pieces<piece_bwd_kernel<DT, W, 16 / W>>(p, 16, dev, st);
  else
    return false;
  return true;
}
template <int DT>
cudaError_t forward_pieces(Fwd& p, int w, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  cudaError_t err = cudaSuccess;
  if constexpr (DT != DT_F32)
    if (w == 4) return *done = forward_pieces<DT, 4>(p, dev, st, &err), err;
  if (w == 2) return *done = forward_pieces<DT, 2>(p, dev, st, &err), err;
  return *done = forward_pieces<DT, 1>(p, dev, st, &err), err;
}
template <int DT>
cudaError_t backward_pieces(Bwd& p, int w, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  cudaError_t err = cudaSuccess;
  if constexpr (DT != DT_F32)
    if (w == 4) return *done = backward_pieces<DT, 4>(p, dev, st, &err), err;
  if (w == 2) return *done = backward_pieces<DT, 2>(p, dev, st, &err), err;
  return *done = backward_pieces<DT, 1>(p, dev, st, &err), err;
}

}  // namespace normres
}  // namespace tpmlp

using namespace tpmlp;

#define BY_TYPE(dtype, CALL)                                      \
  ((dtype) == DT_F32 ? CALL(DT_F32) : (dtype) == DT_F16 ? CALL(DT_F16) : CALL(DT_BF16))

extern "C" {

int tpmlp_sp_rms_residual_forward(const void* const* r, const void* const* z, const tpmlp_rms_residual* norms, void* const* x,
                                  void* const* y, uint8_t* codes, uint8_t* scales, float* rstd_z, float* rstd_x, int64_t s,
                                  int64_t b, int64_t h, int tp, int dtype, void* stream) {
  using namespace normres;
  int rc = check_sizes(s, b, h, tp, dtype);
  if (rc || (rc = check_norms(norms, b, dtype))) return rc;
  const bool has_z = z != nullptr;
  if (!has_z && (norms->post_gamma || norms->gate || codes))
    return set_error(TPMLP_ERR_INVALID_ARG, "a norm behind the block, a gate or a checkpoint without z");
  if (!has_z && !norms->pre_gamma) return set_error(TPMLP_ERR_INVALID_ARG, "neither z nor pre_gamma is given");
  if ((codes == nullptr) != (scales == nullptr)) return set_error(TPMLP_ERR_INVALID_ARG, "codes without scales");
  if (s * b == 0) return TPMLP_OK;
  const size_t e = esize(dtype);
  if ((rc = check_arr(r, tp, e, "r")) || (has_z && (rc = check_arr(z, tp, e, "z"))) ||
      (has_z && (rc = check_arr(const_cast<const void* const*>(x), tp, e, "x"))) ||
      (norms->pre_gamma && (rc = check_arr(const_cast<const void* const*>(y), tp, e, "y"))) ||
      (norms->post_gamma && (rc = check_one(rstd_z, 4, "rstd_z"))) ||
      (norms->pre_gamma && (rc = check_one(rstd_x, 4, "rstd_x"))))
    return rc;
  const int64_t chunk = s / tp * b * h * static_cast<int64_t>(e), weights = h * static_cast<int64_t>(e);
  Apart apart;
  if (has_z) apart.add(const_cast<const void* const*>(x), tp, chunk, true);
  if (norms->pre_gamma) apart.add(const_cast<const void* const*>(y), tp, chunk, true);
  apart.add(codes, s * b * h, true);
  apart.add(scales, s * b * ((h + 31) / 32), true);
  if (norms->post_gamma) apart.add(rstd_z, s * b * 4, true);
  if (norms->pre_gamma) apart.add(rstd_x, s * b * 4, true);
  apart.add(r, tp, chunk, false, has_z ? 0 : -1);
  if (has_z) apart.add(z, tp, chunk, false);
  apart.add(norms->post_gamma, weights, false);
  apart.add(norms->pre_gamma, weights, false);
  if (norms->gate) apart.add(norms->gate, norms->gate_rows * weights, false);
  if ((rc = apart.check("x (but for r itself), y, the checkpoint and 1/rms"))) return rc;
  Fwd p;
  memset(&p, 0, sizeof(p));
  for (int j = 0; j < tp; ++j) {
    p.chunk[j].r = r[j];
    if (has_z) p.chunk[j].z = z[j], p.chunk[j].x = x[j];
    if (norms->pre_gamma) p.chunk[j].y = y[j];
  }
  p.post = norms->post_gamma;
  p.pre = norms->pre_gamma;
  p.gate = norms->gate;
  p.codes = codes;
  p.scales = scales;
  p.rstd_z = rstd_z;
  p.rstd_x = rstd_x;
  p.scale = norms->scale;
  p.eps = norms->eps;
  p.h = static_cast<int>(h);
  p.rpc = static_cast<int>(s / tp * b);
  p.rows = static_cast<int>(s * b);
  p.gate_rows = norms->gate ? static_cast<int>(norms->gate_rows) : 1;
  p.has_z = has_z;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  const int ph = prof_begin(PROF_SP_REGION, st);
  uintptr_t bits = address_bits(norms) | address_bits(r, tp);
  if (has_z) bits |= address_bits(z, tp) | address_bits(const_cast<const void* const*>(x), tp);
  if (p.pre) bits |= address_bits(const_cast<const void* const*>(y), tp);
  const uintptr_t code_bits = reinterpret_cast<uintptr_t>(codes);
  const bool vec = h % 8 == 0 && bits % (8 * e) == 0 && code_bits % 8 == 0;
  bool done = false;
  cudaError_t err = cudaSuccess;
  if (vec) {
#define CALL(D) forward_rows<D>(p, *dev, st, &done)
    err = BY_TYPE(dtype, CALL);
#undef CALL
  }
  if (!done && err == cudaSuccess) {
    const int w = piece_width(h, bits, code_bits, e);
#define CALL(D) forward_pieces<D>(p, w, *dev, st, &done)
    err = BY_TYPE(dtype, CALL);
#undef CALL
  }
  if (!done && err == cudaSuccess) {
    const unsigned grid = deal_units(&p, max_units(h));
#define CALL(D) launch_pdl(any_fwd_kernel<D>, dim3(grid), ANY_THREADS, 0, st, 1, p)
    err = BY_TYPE(dtype, CALL);
#undef CALL
  }
  const double per = e * (1.0 + (has_z ? 2 : 0) + (p.pre ? 1 : 0)) + (codes ? 1.03125 : 0.0);
  prof_end(ph, static_cast<double>(s * b) * h * per, st);
  return report(err, "RMS norm and residual");
}

size_t tpmlp_sp_rms_residual_backward_workspace(int64_t s, int64_t b, int64_t h, int64_t gate_rows) {
  if (s < 0 || b < 0 || h <= 0 || gate_rows < 1 || s > (1ll << 31) || b > (1ll << 31) || s * b >= (1ll << 31) ||
      h >= (1ll << 28) || gate_rows > std::max<int64_t>(b, 1))
    return 0;
  return static_cast<size_t>(2 * normres::units_of_a_gate(s * b, gate_rows, h) * gate_rows * normres::pitch_of(h)) *
         sizeof(float);
}

int tpmlp_sp_rms_residual_backward(const void* const* dx, const void* const* dy, const void* const* x, const void* const* z,
                                   const uint8_t* codes, const uint8_t* scales, const tpmlp_rms_residual* norms,
                                   const float* rstd_z, const float* rstd_x, void* const* dr, void* const* dz,
                                   float* dpost_gamma, float* dpre_gamma, float* dgate, void* ws, size_t ws_bytes, int64_t s,
                                   int64_t b, int64_t h, int tp, int dtype, void* stream) {
  using namespace normres;
  int rc = check_sizes(s, b, h, tp, dtype);
  if (rc || (rc = check_norms(norms, b, dtype))) return rc;
  const bool has_dz = dz != nullptr;
  if (!has_dz && (norms->post_gamma || norms->gate))
    return set_error(TPMLP_ERR_INVALID_ARG, "a norm behind the block or a gate without dz");
  if (dx == nullptr && norms->pre_gamma == nullptr)
    return set_error(TPMLP_ERR_INVALID_ARG, "neither dx nor pre_gamma is given");
  if ((codes == nullptr) != (scales == nullptr)) return set_error(TPMLP_ERR_INVALID_ARG, "codes without scales");
  const bool has_z = norms->post_gamma || norms->gate;  // dz = α·dr needs no z
  const int64_t gate_rows = norms->gate ? norms->gate_rows : 1;
  const size_t e = esize(dtype);
  if ((norms->post_gamma && (rc = check_one(dpost_gamma, 4, "dpost_gamma"))) ||
      (norms->pre_gamma && (rc = check_one(dpre_gamma, 4, "dpre_gamma"))) ||
      (norms->gate && (rc = check_one(dgate, 4, "dgate"))))
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s * b == 0) {  // empty sums
    cudaError_t err = cudaSuccess;
    if (norms->post_gamma) err = cudaMemsetAsync(dpost_gamma, 0, h * 4, st);
    if (err == cudaSuccess && norms->pre_gamma) err = cudaMemsetAsync(dpre_gamma, 0, h * 4, st);
    if (err == cudaSuccess && norms->gate) err = cudaMemsetAsync(dgate, 0, gate_rows * h * 4, st);
    return report(err, "cudaMemsetAsync");
  }
  if ((dx && (rc = check_arr(dx, tp, e, "dx"))) || (norms->pre_gamma && (rc = check_arr(dy, tp, e, "dy"))) ||
      (norms->pre_gamma && (rc = check_arr(x, tp, e, "x"))) || (has_z && !codes && (rc = check_arr(z, tp, e, "z"))) ||
      (norms->post_gamma && (rc = check_one(rstd_z, 4, "rstd_z"))) ||
      (norms->pre_gamma && (rc = check_one(rstd_x, 4, "rstd_x"))) ||
      (rc = check_arr(const_cast<const void* const*>(dr), tp, e, "dr")) ||
      (has_dz && (rc = check_arr(const_cast<const void* const*>(dz), tp, e, "dz"))))
    return rc;
  const size_t need = tpmlp_sp_rms_residual_backward_workspace(s, b, h, gate_rows);
  if (ws == nullptr || ws_bytes < need)
    return set_error(TPMLP_ERR_WORKSPACE, "RMS norm backward workspace needs " + std::to_string(need) + " bytes");
  if ((rc = check_one(ws, 256, "ws"))) return rc;
  const int64_t chunk = s / tp * b * h * static_cast<int64_t>(e), weights = h * static_cast<int64_t>(e);
  Apart apart;
  apart.add(const_cast<const void* const*>(dr), tp, chunk, true);
  if (has_dz) apart.add(const_cast<const void* const*>(dz), tp, chunk, true);
  if (norms->post_gamma) apart.add(dpost_gamma, h * 4, true);
  if (norms->pre_gamma) apart.add(dpre_gamma, h * 4, true);
  if (norms->gate) apart.add(dgate, gate_rows * h * 4, true);
  apart.add(ws, static_cast<int64_t>(need), true);
  if (dx) apart.add(dx, tp, chunk, false, 0);
  if (norms->pre_gamma) apart.add(dy, tp, chunk, false);
  if (norms->pre_gamma) apart.add(x, tp, chunk, false);
  if (has_z && codes) {
    apart.add(codes, s * b * h, false);
    apart.add(scales, s * b * ((h + 31) / 32), false);
  } else if (has_z) {
    apart.add(z, tp, chunk, false);
  }
  if (norms->post_gamma) apart.add(rstd_z, s * b * 4, false);
  if (norms->pre_gamma) apart.add(rstd_x, s * b * 4, false);
  apart.add(norms->post_gamma, weights, false);
  apart.add(norms->pre_gamma, weights, false);
  if (norms->gate) apart.add(norms->gate, gate_rows * weights, false);
  if ((rc = apart.check("dr (but for dx itself), dz, the parameters' gradients and ws"))) return rc;
  Bwd p;
  memset(&p, 0, sizeof(p));
  for (int j = 0; j < tp; ++j) {
    if (dx) p.chunk[j].dx = dx[j];
    if (norms->pre_gamma) p.chunk[j].dy = dy[j], p.chunk[j].x = x[j];
    if (has_z && !codes) p.chunk[j].z = z[j];
    p.chunk[j].dr = dr[j];
    if (has_dz) p.chunk[j].dz = dz[j];
  }
  p.post = norms->post_gamma;
  p.pre = norms->pre_gamma;
  p.gate = norms->gate;
  p.codes = has_z ? codes : nullptr;
  p.scales = scales;
  p.rstd_z = rstd_z;
  p.rstd_x = rstd_x;
  p.scale = norms->scale;
  p.h = static_cast<int>(h);
  p.rpc = static_cast<int>(s / tp * b);
  p.rows = static_cast<int>(s * b);
  p.gate_rows = static_cast<int>(gate_rows);
  p.has_dx = dx != nullptr;
  p.has_dz = has_dz;
  p.has_z = has_z;
  p.part1 = static_cast<float*>(ws);
  p.pitch = pitch_of(h);
  p.part2 = p.part1 + units_of_a_gate(s * b, gate_rows, h) * gate_rows * p.pitch;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  uintptr_t bits = address_bits(norms) | address_bits(const_cast<const void* const*>(dr), tp);
  if (dx) bits |= address_bits(dx, tp);
  if (p.pre) bits |= address_bits(dy, tp) | address_bits(x, tp);
  if (has_z && !codes) bits |= address_bits(z, tp);
  if (has_dz) bits |= address_bits(const_cast<const void* const*>(dz), tp);
  const uintptr_t code_bits = reinterpret_cast<uintptr_t>(p.codes);
  const bool vec = h % 8 == 0 && bits % (8 * e) == 0 && code_bits % 8 == 0;
  const int ph = prof_begin(PROF_SP_REGION, st);
  bool done = false;
  cudaError_t err = cudaSuccess;
  if (vec) {
#define CALL(D) backward_rows<D>(p, *dev, st, &done)
    err = BY_TYPE(dtype, CALL);
#undef CALL
  }
  if (!done && err == cudaSuccess) {
    const int w = piece_width(h, bits, code_bits, e);
#define CALL(D) backward_pieces<D>(p, w, *dev, st, &done)
    err = BY_TYPE(dtype, CALL);
#undef CALL
  }
  if (!done && err == cudaSuccess) {
    const unsigned grid = deal_units(&p, max_units(h));
#define CALL(D) launch_pdl(any_bwd_kernel<D>, dim3(grid), ANY_THREADS, 0, st, 1, p)
    err = BY_TYPE(dtype, CALL);
#undef CALL
  }
  const bool sums = norms->post_gamma || norms->pre_gamma || norms->gate;
  if (err == cudaSuccess && sums) {
    const dim3 grid(static_cast<unsigned>((h + 31) / 32), 2);
    float* dpost = norms->post_gamma ? dpost_gamma : nullptr;
    float* dpre = norms->pre_gamma ? dpre_gamma : nullptr;
    float* dg = norms->gate ? dgate : nullptr;
    // beside the row kernel's last CTAs smaller ones find room sooner; narrow rows have fewer of them (8192 columns
    // 1.0 µs less with 8 warps, 1024 columns 3.7 µs less with 16)
    const unsigned threads = 32 * (h < 4096 ? COL_WARPS : COL_WARPS / 2);
#define CALL(D) launch_pdl(columns_kernel<D>, grid, threads, 0, st, 1, p, dpost, dpre, dg)
    err = BY_TYPE(dtype, CALL);
#undef CALL
  }
  const double per = e * (1.0 + (dx ? 1 : 0) + (p.pre ? 2 : 0) + (has_dz ? 1 : 0)) + (has_z ? (codes ? 1.03125 : e) : 0.0);
  prof_end(ph, static_cast<double>(s * b) * h * per, st, sums ? 2 : 1);
  return report(err, "RMS norm and residual backward");
}

}  // extern "C"
