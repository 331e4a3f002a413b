// Checkpoints of activations in 8 bits (checkpoint.cuh has the format): packing and
// restoring.  The MLP block's own checkpoint is written and read in its GEMMs'
// epilogues (gemm_tc.cu); its float32 path uses the kernels here.
//
// Both are bound by HBM: packing reads 2 (or 4) bytes of an element and writes
// 1 + 1/32, restoring the reverse.  A lane takes 16 neighbouring elements, whose 16-bit
// values are one 32-byte access and whose codes one of 16, so that a group is two lanes and
// its largest value one shuffle (4096 × 24576 bf16: 47.0 µs, 0.96 of a plain copy's rate;
// 52.6 µs with 8 elements and 16-byte accesses, 49.2 µs with the five CTAs an SM that 46
// registers leave instead of six; restoring 2048 × 28672 27.5 and 29.4 µs).  Where the rows
// of either side are not whole units of such accesses, lanes take the largest power of
// two of elements that they are, and more rows each.
#include <algorithm>
#include <string>

#include "checkpoint.cuh"
#include "internal.h"

namespace tpmlp {
namespace ckpt {

constexpr int THREADS = 256;

// A slot is what a lane takes at once: EL = 16, 8, 4, 2 or 1 elements.  A CTA covers a
// tile of `by·R` rows × `bx` slots, bx a power of two, a thread's R slots `by` rows apart
// and their loads in flight together; tiles are numbered along the columns first.  (One
// contiguous piece of a dense tensor a CTA measured the same.)
struct Shape {
  int64_t rows, cols, ld;  // ld: row stride of the 16- or 32-bit tensor
  int64_t groups;          // of a row
  int bx_log2;
  unsigned col_tiles;
};

template <int EL>
struct RowsOf {
  static constexpr int N = EL == 16 ? 2 : EL == 8 ? 4 : EL == 4 ? 8 : 16;
};

// This thread's slot and first row.
template <int R>
__device__ __forceinline__ void place(const Shape& s, int64_t& slot, int64_t& row0, int& by) {
  const unsigned rt = blockIdx.x / s.col_tiles, ct = blockIdx.x - rt * s.col_tiles;
  by = THREADS >> s.bx_log2;
  slot = (static_cast<int64_t>(ct) << s.bx_log2) + (threadIdx.x & ((1 << s.bx_log2) - 1));
  row0 = static_cast<int64_t>(rt) * (by * R) + (threadIdx.x >> s.bx_log2);
}

// EL elements as stored, in 4-byte words.
template <int DT, int EL>
struct Raw {
  static constexpr int BYTES = EL * (DT == DT_F32 ? 4 : 2);
  static constexpr int W = (BYTES + 3) / 4;
  uint32_t w[W];
};

// BYTES bytes at q (aligned to them, to 32 at most) to or from words.
template <int BYTES>
__device__ __forceinline__ void load_bytes(const void* q, uint32_t* w) {
  if constexpr (BYTES >= 32) {
#pragma unroll
    for (int k = 0; k < BYTES / 4; k += 8)
      asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[k]), "=r"(w[k + 1]), "=r"(w[k + 2]), "=r"(w[k + 3]), "=r"(w[k + 4]), "=r"(w[k + 5]),
                     "=r"(w[k + 6]), "=r"(w[k + 7])
                   : "l"(static_cast<const char*>(q) + 4 * k)
                   : "memory");
  } else if constexpr (BYTES == 16) {
    const uint4 v = ld_stream_v4(q);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = *static_cast<const uint2*>(q);
    w[0] = v.x;
    w[1] = v.y;
  } else if constexpr (BYTES == 4) {
    w[0] = *static_cast<const uint32_t*>(q);
  } else if constexpr (BYTES == 2) {
    w[0] = *static_cast<const uint16_t*>(q);
  } else {
    w[0] = *static_cast<const uint8_t*>(q);
  }
}
template <int BYTES>
__device__ __forceinline__ void store_bytes(void* q, const uint32_t* w) {
  if constexpr (BYTES >= 32) {
#pragma unroll
    for (int k = 0; k < BYTES / 4; k += 8)
      asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[k]), "r"(w[k + 1]), "r"(w[k + 2]),
                   "r"(w[k + 3]), "r"(w[k + 4]), "r"(w[k + 5]), "r"(w[k + 6]), "r"(w[k + 7]),
                   "l"(static_cast<char*>(q) + 4 * k)
                   : "memory");
  } else if constexpr (BYTES == 16) {
    *static_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (BYTES == 8) {
    *static_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  } else if constexpr (BYTES == 4) {
    *static_cast<uint32_t*>(q) = w[0];
  } else if constexpr (BYTES == 2) {
    *static_cast<uint16_t*>(q) = static_cast<uint16_t>(w[0]);
  } else {
    *static_cast<uint8_t*>(q) = static_cast<uint8_t>(w[0]);
  }
}

template <int DT, int EL>
__device__ __forceinline__ void* element(const void* p, int64_t i) {
  return const_cast<char*>(static_cast<const char*>(p)) + i * static_cast<int64_t>(sizeof(typename Storage<DT>::T));
}

template <int DT, int EL>
__device__ __forceinline__ void values(const Raw<DT, EL>& r, float* v) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int i = 0; i < EL; ++i) v[i] = __uint_as_float(r.w[i]);
  } else {
    typename Storage<DT>::T t[EL];
    memcpy(t, r.w, Raw<DT, EL>::BYTES);
#pragma unroll
    for (int i = 0; i < EL; ++i) v[i] = Storage<DT>::to_f32(t[i]);
  }
}

template <int DT, int EL>
__global__ void __launch_bounds__(THREADS, DT == DT_F32 ? 4 : 6) pack_kernel(const void* x, uint8_t* codes,
                                                                             uint8_t* scales, Shape s) {
  constexpr int R = RowsOf<EL>::N, LANES = CKPT_GROUP / EL;  // of a group
  pdl_enter();
  int64_t slot, row0;
  int by;
  place<R>(s, slot, row0, by);
  const int64_t col = slot * EL;
  const bool in = col < s.cols;
  Raw<DT, EL> raw[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t row = row0 + k * by;
    raw[k] = Raw<DT, EL>{};
    if (in && row < s.rows) load_bytes<Raw<DT, EL>::BYTES>(element<DT, EL>(x, row * s.ld + col), raw[k].w);
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t row = row0 + k * by;
    float v[EL < 4 ? 4 : EL] = {};
    values<DT, EL>(raw[k], v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < EL; ++i) top = max(top, ckpt_abs(v[i]));
#pragma unroll
    for (int o = 1; o < LANES; o *= 2)  // (EL ≤ 2: a tile is no wider than its row, which may be part of a group)
      if (EL > 2 || o < 1 << s.bx_log2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = ckpt_byte(top);
    const float inv = ckpt_inverse(byte);
    if (in && row < s.rows) {
      uint32_t c[(EL + 3) / 4];
#pragma unroll
      for (int i = 0; i < EL; i += 4) c[i / 4] = ckpt_encode4(v + i, inv);
      store_bytes<EL>(codes + row * s.cols + col, c);
      if (slot % LANES == 0) scales[row * s.groups + slot / LANES] = static_cast<uint8_t>(byte);
    }
  }
}

template <int DT, int EL>
__global__ void __launch_bounds__(THREADS) unpack_kernel(const uint8_t* codes, const uint8_t* scales, void* x, Shape s) {
  constexpr int R = RowsOf<EL>::N, LANES = CKPT_GROUP / EL;
  pdl_enter();
  int64_t slot, row0;
  int by;
  place<R>(s, slot, row0, by);
  const int64_t col = slot * EL;
  if (col >= s.cols) return;
  uint32_t c[R][(EL + 3) / 4], byte[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t row = row0 + k * by;
    if (row < s.rows) {
      load_bytes<EL>(codes + row * s.cols + col, c[k]);
      byte[k] = scales[row * s.groups + slot / LANES];
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t row = row0 + k * by;
    if (row >= s.rows) break;
    float v[EL < 4 ? 4 : EL];
    const float scale = ckpt_scale(byte[k]);
#pragma unroll
    for (int i = 0; i < EL; i += 4) ckpt_decode4(c[k][i / 4], scale, v + i);
    Raw<DT, EL> r;
    typename Storage<DT>::T t[EL];
#pragma unroll
    for (int i = 0; i < EL; ++i) t[i] = Storage<DT>::from(ckpt_in_range<DT>(v[i]));
    memcpy(r.w, t, sizeof(t));
    store_bytes<Raw<DT, EL>::BYTES>(element<DT, EL>(x, row * s.ld + col), r.w);
  }
}

// A dense tensor whose rows are whole units of no more than two elements:
// a CTA takes a piece of it — whole rows, or 4096 columns of one — copies the piece to
// shared memory in the 16-byte units that lie in it whatever row they begin in, works on
// it there, 4 columns a lane, and copies the result out in the same way.  (48000 × 1025
// bf16: packing 73 µs, restoring 59; 121 and 116 with lanes of one element.)
constexpr int PIECE = 4096;  // elements at most

// n bytes at g to shared memory, byte i to s + (g mod 16) + i; s is 16-byte aligned.
// E: elements have E bytes and g is aligned to them.
template <int E>
__device__ __forceinline__ void bytes_in(uint8_t* s, const uint8_t* g, int n) {
  const int first = static_cast<int>(reinterpret_cast<uintptr_t>(g) & 15), end = first + n;
  const uint8_t* base = g - first;  // only its units from `first` on, and up to `end`, are touched
  const int lo = (first + 15) >> 4, hi = end >> 4;
  for (int u = lo + static_cast<int>(threadIdx.x); u < hi; u += THREADS)
    *reinterpret_cast<uint4*>(s + 16 * u) = ld_stream_v4(base + 16 * static_cast<int64_t>(u));
  // what lies before the first whole unit and behind the last, an element a thread
  const int head = min(16 * lo, end), tail = max(16 * hi, head), at = static_cast<int>(threadIdx.x) * E;
  const int i = at < 16 ? first + at : tail + at - 16;
  if (at < 16 ? i < head : at < 32 && i < end) {
    if constexpr (E == 4)
      *reinterpret_cast<uint32_t*>(s + i) = *reinterpret_cast<const uint32_t*>(base + i);
    else if constexpr (E == 2)
      *reinterpret_cast<uint16_t*>(s + i) = *reinterpret_cast<const uint16_t*>(base + i);
    else
      s[i] = base[i];
  }
}
template <int E>
__device__ __forceinline__ void bytes_out(uint8_t* g, const uint8_t* s, int n) {
  const int first = static_cast<int>(reinterpret_cast<uintptr_t>(g) & 15), end = first + n;
  uint8_t* base = g - first;
  const int lo = (first + 15) >> 4, hi = end >> 4;
  for (int u = lo + static_cast<int>(threadIdx.x); u < hi; u += THREADS)
    *reinterpret_cast<uint4*>(base + 16 * static_cast<int64_t>(u)) = *reinterpret_cast<const uint4*>(s + 16 * u);
  const int head = min(16 * lo, end), tail = max(16 * hi, head), at = static_cast<int>(threadIdx.x) * E;
  const int i = at < 16 ? first + at : tail + at - 16;
  if (at < 16 ? i < head : at < 32 && i < end) {
    if constexpr (E == 4)
      *reinterpret_cast<uint32_t*>(base + i) = *reinterpret_cast<const uint32_t*>(s + i);
    else if constexpr (E == 2)
      *reinterpret_cast<uint16_t*>(base + i) = *reinterpret_cast<const uint16_t*>(s + i);
    else
      base[i] = s[i];
  }
}

struct Pieces {
  int64_t rows, cols, groups;
  int R;           // rows of a piece, 0: a piece is part of a row
  int per_row;     // pieces of a row then
  int lanes_log2;  // of a group: 8, or fewer for rows of up to 16 columns
};

// This CTA's piece: `rows` rows of `cols` columns from element `e0`, scale byte `g0` on,
// with `groups` groups a row.
struct Piece {
  int64_t e0, g0;
  int rows, cols, groups;
  __device__ __forceinline__ explicit Piece(const Pieces& p) {
    if (p.R > 0) {
      const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.R;
      rows = static_cast<int>(min(static_cast<int64_t>(p.R), p.rows - r0));
      cols = static_cast<int>(p.cols);
      e0 = r0 * p.cols;
      g0 = r0 * p.groups;
    } else {
      const unsigned row = blockIdx.x / static_cast<unsigned>(p.per_row);
      const int64_t c0 = static_cast<int64_t>(blockIdx.x - row * static_cast<unsigned>(p.per_row)) * PIECE;
      rows = 1;
      cols = static_cast<int>(min(static_cast<int64_t>(PIECE), p.cols - c0));
      e0 = row * p.cols + c0;
      g0 = row * p.groups + c0 / CKPT_GROUP;
    }
    groups = (cols + CKPT_GROUP - 1) / CKPT_GROUP;
  }
};

template <int DT>
__global__ void __launch_bounds__(THREADS) pack_piece_kernel(const void* x, uint8_t* codes, uint8_t* scales, Pieces all) {
  using T = typename Storage<DT>::T;
  constexpr int E = sizeof(T);
  __shared__ __align__(16) uint8_t in[PIECE * E + 16];
  __shared__ __align__(16) uint8_t out[PIECE + 16];
  pdl_enter();
  const Piece p(all);
  const uint8_t* xg = static_cast<const uint8_t*>(x) + p.e0 * E;
  bytes_in<E>(in, xg, p.rows * p.cols * E);
  __syncthreads();
  const T* v_in = reinterpret_cast<const T*>(in + (reinterpret_cast<uintptr_t>(xg) & 15));
  uint8_t* c_out = out + (reinterpret_cast<uintptr_t>(codes + p.e0) & 15);
  const int l2 = all.lanes_log2, lane = threadIdx.x & ((1 << l2) - 1);
  const int total = p.rows * p.groups, step = THREADS >> l2, first = static_cast<int>(threadIdx.x) >> l2;
  const int step_rows = step / p.groups, step_groups = step - step_rows * p.groups;
  int row = first / p.groups, in_row = first - row * p.groups;
  for (int g = first; g - first < total; g += step) {  // whole warps: a group's lanes meet
    const int col = in_row * CKPT_GROUP + lane * 4;
    const int have = g < total ? min(4, p.cols - col) : 0, at = row * p.cols + col;
    float v[4] = {};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < have) v[i] = Storage<DT>::to_f32(v_in[at + i]);
      top = max(top, ckpt_abs(v[i]));
    }
#pragma unroll
    for (int o = 1; o < 8; o *= 2)
      if (o < 1 << l2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t byte = ckpt_byte(top), c = ckpt_encode4(v, ckpt_inverse(byte));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) c_out[at + i] = static_cast<uint8_t>(c >> (8 * i));
    if (g < total && lane == 0) scales[p.g0 + g] = static_cast<uint8_t>(byte);
    row += step_rows;
    if ((in_row += step_groups) >= p.groups) {
      in_row -= p.groups;
      ++row;
    }
  }
  __syncthreads();
  bytes_out<1>(codes + p.e0, out, p.rows * p.cols);
}

template <int DT>
__global__ void __launch_bounds__(THREADS) unpack_piece_kernel(const uint8_t* codes, const uint8_t* scales, void* x,
                                                               Pieces all) {
  using T = typename Storage<DT>::T;
  constexpr int E = sizeof(T);
  __shared__ __align__(16) uint8_t in[PIECE + 16];
  __shared__ __align__(16) uint8_t out[PIECE * E + 16];
  pdl_enter();
  const Piece p(all);
  uint8_t* xg = static_cast<uint8_t*>(x) + p.e0 * E;
  bytes_in<1>(in, codes + p.e0, p.rows * p.cols);
  __syncthreads();
  const uint8_t* c_in = in + (reinterpret_cast<uintptr_t>(codes + p.e0) & 15);
  T* v_out = reinterpret_cast<T*>(out + (reinterpret_cast<uintptr_t>(xg) & 15));
  const int l2 = all.lanes_log2, lane = threadIdx.x & ((1 << l2) - 1);
  const int total = p.rows * p.groups, step = THREADS >> l2, first = static_cast<int>(threadIdx.x) >> l2;
  const int step_rows = step / p.groups, step_groups = step - step_rows * p.groups;
  int row = first / p.groups, in_row = first - row * p.groups;
  for (int g = first; g < total; g += step) {
    const int col = in_row * CKPT_GROUP + lane * 4;
    const int have = min(4, p.cols - col), at = row * p.cols + col;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) c |= static_cast<uint32_t>(c_in[at + i]) << (8 * i);
    float v[4];
    ckpt_decode4(c, ckpt_scale(scales[p.g0 + g]), v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) v_out[at + i] = Storage<DT>::from(ckpt_in_range<DT>(v[i]));
    row += step_rows;
    if ((in_row += step_groups) >= p.groups) {
      in_row -= p.groups;
      ++row;
    }
  }
  __syncthreads();
  bytes_out<E>(xg, out, p.rows * p.cols * E);
}

// u and y = act(u) of the float32 block's checkpoint: codes [M, n1], each half of a
// SwiGLU row with its own groups.  One element of y a thread: the CUDA-core GEMMs around
// it take far longer.
__global__ void __launch_bounds__(THREADS) act_kernel(const uint8_t* codes, const uint8_t* scales, float* u, float* y,
                                                      int64_t M, int64_t f, int act) {
  const int64_t groups = (f + CKPT_GROUP - 1) / CKPT_GROUP;
  const int halves = act == ACT_SWIGLU ? 2 : 1;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; i < M * f;
       i += static_cast<int64_t>(gridDim.x) * THREADS) {
    const int64_t m = i / f, c = i - m * f;
    float w[2] = {0.0f, 0.0f};
    for (int k = 0; k < halves; ++k) {
      const int64_t row = m * halves + k;
      float v[4];
      ckpt_decode4(codes[row * f + c], ckpt_scale(scales[row * groups + (c >> 5)]), v);
      w[k] = ckpt_in_range<DT_F32>(v[0]);
      u[row * f + c] = w[k];
    }
    y[i] = halves == 2 ? w[0] * sigmoid_f<true>(w[0]) * w[1] : held_act_fwd<true>(act, w[0]);
  }
}

size_t esize(int dtype) { return dtype == DT_F32 ? 4 : 2; }

// Slots along a row: as many of the CTA's threads as leave at most a tenth of the
// lanes behind the row's end, whole warps where the row has them.
int pick_bx(int64_t slots, int least) {
  int best = least;
  double best_eff = 0.0;
  for (int l = 8; l >= least; --l) {
    const int64_t bx = 1ll << l;
    const double eff = static_cast<double>(slots) / static_cast<double>((slots + bx - 1) / bx * bx);
    if (eff >= 0.9) return l;
    if (eff > best_eff) {
      best_eff = eff;
      best = l;
    }
  }
  return best;
}

int check_args(bool pack, const void* x, int64_t ld, const void* codes, const void* scales, int64_t rows, int64_t cols,
               int dtype) {
  if (rows < 0 || cols < 1) return set_error(TPMLP_ERR_INVALID_ARG, "rows >= 0 and cols >= 1 required");
  if (dtype < DT_F32 || dtype > DT_BF16) return set_error(TPMLP_ERR_INVALID_ARG, "unknown dtype");
  if (rows >= (1ll << 40) || cols >= (1ll << 31) || (rows > 0 && cols > (1ll << 40) / rows)) return set_error(TPMLP_ERR_UNSUPPORTED, "extent too large");
  if (rows == 0) return TPMLP_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr)
    return set_error(TPMLP_ERR_INVALID_ARG, "x, codes or scales is NULL");
  if (ld < cols && rows > 1) return set_error(TPMLP_ERR_INVALID_ARG, "the row stride is smaller than a row");
  if (reinterpret_cast<uintptr_t>(x) % esize(dtype) != 0) return set_error(TPMLP_ERR_INVALID_ARG, "x is misaligned");
  const uintptr_t at = reinterpret_cast<uintptr_t>(x);
  const uintptr_t end = at + static_cast<uintptr_t>((rows > 1 ? (rows - 1) * ld : 0) + cols) * esize(dtype);
  const int64_t groups = (cols + CKPT_GROUP - 1) / CKPT_GROUP;
  const auto meets = [&](const void* p, int64_t n) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(p);
    return q < end && at < q + static_cast<uintptr_t>(n);
  };
  if (meets(codes, rows * cols) || meets(scales, rows * groups))
    return set_error(TPMLP_ERR_INVALID_ARG, "x and the checkpoint must not overlap");
  return pack ? check_checkpoint_apart(codes, scales, rows, cols) : TPMLP_OK;
}

template <int DT>
int launch(bool pack, void* x, int64_t ld, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols, cudaStream_t st) {
  const size_t e = sizeof(typename Storage<DT>::T);
  Shape s{};
  s.rows = rows;
  s.cols = cols;
  s.ld = rows > 1 ? ld : cols;
  s.groups = (cols + CKPT_GROUP - 1) / CKPT_GROUP;
  // elements of a lane: what the addresses of both sides allow
  const uintptr_t at = reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(rows > 1 ? s.ld * e : 0);
  const uintptr_t held = reinterpret_cast<uintptr_t>(codes) | static_cast<uintptr_t>(cols);
  int el = 16;
  while (el > 1 && (at % std::min<size_t>(el * e, 32) != 0 || held % el != 0)) el /= 2;
  if (el <= 2 && s.ld == cols) {
    Pieces p{rows, cols, s.groups, 0, 0, 3};
    while (p.lanes_log2 > 0 && cols <= 4 << (p.lanes_log2 - 1)) --p.lanes_log2;
    if (cols <= PIECE)
      p.R = static_cast<int>(PIECE / cols);
    else
      p.per_row = static_cast<int>((cols + PIECE - 1) / PIECE);
    const int64_t pieces = p.R ? (rows + p.R - 1) / p.R : rows * p.per_row;  // below 2^31: of 2^11 elements, out of 2^40
    const int ph = prof_begin(PROF_SP_REGION, st);
    const dim3 grid(static_cast<unsigned>(pieces));
    const void* xc = x;
    const uint8_t *cc = codes, *sc = scales;
    const cudaError_t err = pack ? launch_pdl(pack_piece_kernel<DT>, grid, THREADS, 0, st, 1, xc, codes, scales, p)
                                 : launch_pdl(unpack_piece_kernel<DT>, grid, THREADS, 0, st, 1, cc, sc, x, p);
    prof_end(ph, static_cast<double>(rows) * (static_cast<double>(cols) * (e + 1) + s.groups), st);
    if (err != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string("checkpoint: ") + cudaGetErrorString(err));
    return TPMLP_OK;
  }
  const int64_t slots = (cols + el - 1) / el;
  int least = 0;  // a tile is no wider than the row needs, but of whole groups
  while ((1ll << least) < std::max<int64_t>(std::min<int64_t>(slots, 32), el > 2 ? CKPT_GROUP / el : 1)) ++least;
  s.bx_log2 = slots > 32 ? pick_bx(slots, 5) : least;
  const int each = el == 16 ? RowsOf<16>::N : el == 8 ? RowsOf<8>::N : el == 4 ? RowsOf<4>::N : RowsOf<1>::N;
  const int64_t bx = 1ll << s.bx_log2, tile_rows = THREADS / bx * each;
  s.col_tiles = static_cast<unsigned>((slots + bx - 1) / bx);
  // the grid's x extent is below 2^31: launches of as many rows as it holds
  const int64_t most = ((1ll << 31) - 1) / s.col_tiles * tile_rows;
  const int ph = prof_begin(PROF_SP_REGION, st);
  cudaError_t err = cudaSuccess;
  int kernels = 0;
  for (int64_t r0 = 0; r0 < s.rows && err == cudaSuccess; r0 += most, ++kernels) {
    Shape t = s;
    t.rows = std::min(most, s.rows - r0);
    const dim3 grid(static_cast<unsigned>((t.rows + tile_rows - 1) / tile_rows * s.col_tiles));
    void* xr = static_cast<char*>(x) + r0 * s.ld * static_cast<int64_t>(e);
    uint8_t* cr = codes + r0 * s.cols;
    uint8_t* sr = scales + r0 * s.groups;
    const void* xc = xr;
    const uint8_t *cc = cr, *sc = sr;
#define PACK(EL) launch_pdl(pack_kernel<DT, EL>, grid, THREADS, 0, st, 1, xc, cr, sr, t)
#define UNPACK(EL) launch_pdl(unpack_kernel<DT, EL>, grid, THREADS, 0, st, 1, cc, sc, xr, t)
#define BY_EL(F) (el == 16 ? F(16) : el == 8 ? F(8) : el == 4 ? F(4) : el == 2 ? F(2) : F(1))
    err = pack ? BY_EL(PACK) : BY_EL(UNPACK);
#undef BY_EL
#undef UNPACK
#undef PACK
  }
  prof_end(ph, static_cast<double>(rows) * (static_cast<double>(cols) * (e + 1) + s.groups), st, kernels);
  if (err != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string("checkpoint: ") + cudaGetErrorString(err));
  return TPMLP_OK;
}

int call(bool pack, void* x, int64_t ld, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols, int dtype,
         cudaStream_t st) {
  const int rc = check_args(pack, x, ld, codes, scales, rows, cols, dtype);
  if (rc != TPMLP_OK || rows == 0) return rc;
  if (dtype == DT_F32) return launch<DT_F32>(pack, x, ld, codes, scales, rows, cols, st);
  if (dtype == DT_F16) return launch<DT_F16>(pack, x, ld, codes, scales, rows, cols, st);
  return launch<DT_BF16>(pack, x, ld, codes, scales, rows, cols, st);
}

}  // namespace ckpt

int check_checkpoint_apart(const void* codes, const void* scales, int64_t rows, int64_t cols) {
  const uintptr_t c = reinterpret_cast<uintptr_t>(codes), s = reinterpret_cast<uintptr_t>(scales);
  const int64_t groups = (cols + CKPT_GROUP - 1) / CKPT_GROUP;
  if (c < s + static_cast<uintptr_t>(rows * groups) && s < c + static_cast<uintptr_t>(rows * cols))
    return set_error(TPMLP_ERR_INVALID_ARG, "codes and scales must not overlap");
  return TPMLP_OK;
}

int launch_checkpoint_act(const uint8_t* codes, const uint8_t* scales, float* u, float* y, int64_t M, int64_t f, int act,
                          cudaStream_t st) {
  const int ph = prof_begin(PROF_SP_REGION, st);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((M * f + ckpt::THREADS - 1) / ckpt::THREADS, 65536));
  ckpt::act_kernel<<<grid, ckpt::THREADS, 0, st>>>(codes, scales, u, y, M, f, act);
  prof_end(ph, static_cast<double>(M) * f * (act == ACT_SWIGLU ? 14 : 9), st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(TPMLP_ERR_CUDA, std::string("checkpoint activation: ") + cudaGetErrorString(e));
  return TPMLP_OK;
}

}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

int tpmlp_checkpoint_pack(const void* x, int64_t ld_x, uint8_t* codes, uint8_t* scales, int64_t rows, int64_t cols,
                          int dtype, void* stream) {
  return ckpt::call(true, const_cast<void*>(x), ld_x, codes, scales, rows, cols, dtype, static_cast<cudaStream_t>(stream));
}

int tpmlp_checkpoint_unpack(const uint8_t* codes, const uint8_t* scales, void* x, int64_t ld_x, int64_t rows, int64_t cols,
                            int dtype, void* stream) {
  return ckpt::call(false, x, ld_x, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), rows, cols, dtype,
                    static_cast<cudaStream_t>(stream));
}

}  // extern "C"
