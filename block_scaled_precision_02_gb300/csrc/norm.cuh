// What the layer-norm kernels share: arguments, statistics, the row kernel
// (one row per warp or CTA, in registers) and the slots that whole rows are
// copied to.
//
// Statistics are float32 and come from data on the chip: partial means and
// sums of squared deviations merge as
//   M2(A+B) = M2(A) + M2(B) + n_A (mean_A - mean)^2 + n_B (mean_B - mean)^2,
// which does not cancel when the mean is large against the spread.
#pragma once

#include <algorithm>
#include <type_traits>

#include "rowops.cuh"

namespace mxq {

// What a row kernel writes: bf16 or float32 rows, or MX codes of a format.
constexpr int OUT_BF16 = -2, OUT_F32 = -1;

struct NormArgs {
  const void* x;
  int64_t ld;
  int rows, cols;
  const void* w;          // [cols] or NULL (1)
  const void* b;          // [cols] or NULL (0)
  int w_f32, b_f32;
  float eps;
  void* y;                // row outputs; NULL: statistics only
  float* mean;
  float* rstd;
  uint8_t *q_row, *s_row, *q_col, *s_col;
  int ceil_mode, mma;
  int pack_row, pack_col;         // the scales of four blocks may go as one word
  int wide_col;                   // q_col is 32-byte aligned
};

// 1 / sqrt(v): the hardware's estimate and one Newton step, within 2 ulp; at
// v = 0 or an infinity the estimate is the result.  v r is normal for every
// v, v / 2 is not.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return v > 0.f && v < INFINITY ? r * fmaf(v * r, -0.5f * r, 1.5f) : r;
}

__device__ __forceinline__ float norm_value(float x, float mean, float rstd, float w, float b) {
  return __fmaf_rn(__fmul_rn(__fsub_rn(x, mean), rstd), w, b);
}

template <int VE>
__device__ __forceinline__ void load_affine(const NormArgs& a, int at, float (&w)[VE], float (&b)[VE]) {
  if (a.w) load_param<VE>(a.w, a.w_f32, at, w);
  else
#pragma unroll
    for (int j = 0; j < VE; ++j) w[j] = 1.f;
  if (a.b) load_param<VE>(a.b, a.b_f32, at, b);
  else
#pragma unroll
    for (int j = 0; j < VE; ++j) b[j] = 0.f;
}

// Where a thread's vectors lie in a row: warp w of a group holds 32 * NV
// vectors in a row, lane l those at first + 32 k (fixed distances from one
// address, so loads and stores need no arithmetic of their own).
template <int NV>
__device__ __forceinline__ int first_vec(int w, int lane) { return w * 32 * NV + lane; }

// Elements of a row of `cols` that warp w holds.
template <int VE, int NV>
__device__ __forceinline__ int warp_count(int cols, int w) { return max(0, min(32 * NV * VE, cols - w * 32 * NV * VE)); }

// Sum of squared deviations of a thread's valid vectors from m.
template <int VE, int NV>
__device__ __forceinline__ float sq_dev(const float (&v)[NV][VE], float m, int first, int nvec) {
  float s[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float d[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) d[j] = (v[k][j] - m) * (v[k][j] - m);
    s[k] = first + 32 * k < nvec ? tree_sum(d) : 0.f;
  }
  return tree_sum(s);
}

// Sum of VE elements, and of their squared distances from m.
template <int VE>
__device__ __forceinline__ float vec_sum(const float (&v)[VE]) {
  if constexpr (VE == 1) return v[0];
  else {
    float2 p = pair(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < VE; j += 2) p = add2(p, pair(v[j], v[j + 1]));
    float x, y;
    halves(p, x, y);
    return x + y;
  }
}
template <int VE>
__device__ __forceinline__ float vec_sq_dev(const float (&v)[VE], float m) {
  if constexpr (VE == 1) return (v[0] - m) * (v[0] - m);
  else {
    const float2 mm = splat(m);
    float2 d = sub2(pair(v[0], v[1]), mm), p = mul2(d, d);
#pragma unroll
    for (int j = 2; j < VE; j += 2) {
      d = sub2(pair(v[j], v[j + 1]), mm);
      p = fma2(d, d, p);
    }
    float x, y;
    halves(p, x, y);
    return x + y;
  }
}

// One row per warp (WARP: eight rows per CTA, no barrier) or per CTA (one
// barrier); the row stays in registers, VE * NV elements per thread, so x is
// read once and y written once: HBM bounds it.
template <typename TX, int OUT, int VE, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) norm_row_kernel(const NormArgs a) {
  __shared__ float2 part[32];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = first_vec<NV>(WARP ? 0 : warp, lane);
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  if (WARP && row >= a.rows) return;
  const int nvec = a.cols / VE;
  const TX* x = static_cast<const TX*>(a.x) + row * a.ld;

  float v[NV][VE];
  {
    Vec<TX, VE> raw[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      raw[k].fill(0);
      if (first + 32 * k < nvec) raw[k].load(x + (first + 32 * k) * VE);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < VE; ++j) v[k][j] = raw[k].get(j);
  }

  float s[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) s[k] = tree_sum(v[k]);
  float sum = warp_sum(tree_sum(s));
  const float inv_c = 1.f / static_cast<float>(a.cols);
  float mean, m2;
  if constexpr (WARP) {
    mean = sum * inv_c;
    m2 = warp_sum(sq_dev<VE, NV>(v, mean, first, nvec));
  } else {
    const int n = warp_count<VE, NV>(a.cols, warp);
    m2 = warp_sum(sq_dev<VE, NV>(v, n ? sum / static_cast<float>(n) : 0.f, first, nvec));
    if (lane == 0) part[warp] = make_float2(sum, m2);
    __syncthreads();
    const bool have = lane < static_cast<int>(blockDim.x >> 5);
    const float2 pw = have ? part[lane] : make_float2(0.f, 0.f);
    const int nw = have ? warp_count<VE, NV>(a.cols, lane) : 0;
    mean = warp_sum(pw.x) * inv_c;
    const float d = nw ? pw.x / static_cast<float>(nw) - mean : 0.f;
    m2 = warp_sum(pw.y + static_cast<float>(nw) * d * d);
  }
  const float rstd = 1.f / sqrtf(m2 * inv_c + a.eps);
  if (first == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }

  if constexpr (OUT < 0) {
    using TY = typename std::conditional<OUT == OUT_F32, float, __nv_bfloat16>::type;
    if (!a.y) return;
    TY* y = static_cast<TY*>(a.y) + row * a.cols;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int at = (first + 32 * k) * VE;
      if (at >= nvec * VE) continue;
      float w[VE], b[VE], o[VE];
      load_affine<VE>(a, at, w, b);
#pragma unroll
      for (int j = 0; j < VE; ++j) o[j] = norm_value(v[k][j], mean, rstd, w[j], b[j]);
      store_vec<TY, VE>(y + at, o);
    }
  } else {
    // 32 / VE neighbouring lanes hold a block; its amax by shuffles
    constexpr int LPB = 32 / VE;
    constexpr int QW = code_words<OUT, VE>();
    const int kb = a.cols / 32;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int at = (first + 32 * k) * VE;
      const bool valid = at < a.cols;
      float o[VE];
      float m = 0.f;
      if (valid) {
        float w[VE], b[VE];
        load_affine<VE>(a, at, w, b);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          o[j] = norm_value(v[k][j], mean, rstd, w[j], b[j]);
          m = fmax3_nan(m, fabsf(o[j]), 0.f);
        }
      }
#pragma unroll
      for (int i = 1; i < LPB; i <<= 1) m = fmax3_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, i), 0.f);
      const uint32_t ab = __float_as_uint(m) & 0x7FFFFFFFu;
      float mult;
      const uint32_t code = mx_scale<OUT>(ab, a.ceil_mode, mult);
      if (valid) {
        uint32_t q[QW];
        mx_codes<OUT, VE>(o, mult, code == 0xFFu, q);
        uint8_t* dst = a.q_row + (OUT == MXQ_E2M1 ? (row * a.cols + at) / 2 : row * a.cols + at);
        if constexpr (OUT == MXQ_E2M1 && VE == 4) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(q[0]);
        else if constexpr (QW == 1) *reinterpret_cast<uint32_t*>(dst) = q[0];
        else *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
      }
      if (a.pack_row) {     // the scales of four neighbouring blocks as one word
        uint32_t word = code << (8 * ((lane / LPB) & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, LPB);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * LPB);
        if (valid && lane % (4 * LPB) == 0)
          *reinterpret_cast<uint32_t*>(a.s_row + scale_at(row, at / 32, kb, a.mma)) = word;
      } else if (valid && lane % LPB == 0) {
        a.s_row[scale_at(row, at / 32, kb, a.mma)] = static_cast<uint8_t>(code);
      }
    }
  }
}

// ---------------------------------------------------------------- rows in slots
constexpr int MAX_GROUPS = 32, MAX_STAGES = 8;
constexpr int MAX_BARRIERS = 15;           // named barriers 1..15; a group of one warp needs none
constexpr int kRingBytes = 216 * 1024;

__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(threads) : "memory");
}

// After a wait has given up: no exit while copies may be in flight.  `slot`
// and `phase` are the next slot to be used and its parity.
__device__ __forceinline__ void await_ring(const uint64_t* full, int stages, int slot, int phase, int* status) {
  for (int i = 0; i < stages; ++i) mbar_wait(smem_u32(full + i), i >= slot ? phase : phase ^ 1, status);
}

// A matrix whose rows go through slots.  Bulk copies move whole 16-byte words,
// so a row that starts or ends inside one is copied with its neighbours'
// bytes in those words; only where such a word would leave the matrix (its
// first and last row) nothing is copied and the row is read in place.
template <typename T>
struct RowSource {
  const T* base;
  int64_t ld;
  int cols, rows;

  __device__ __forceinline__ const T* row(int64_t r) const { return base + r * ld; }
  __device__ __forceinline__ int head(int64_t r) const { return static_cast<int>(reinterpret_cast<uintptr_t>(row(r)) & 15); }
  __device__ __forceinline__ uint32_t bytes(int64_t r) const {
    return static_cast<uint32_t>((head(r) + cols * static_cast<int>(sizeof(T)) + 15) & ~15);
  }
  __device__ __forceinline__ bool copied(int64_t r) const {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(row(r)) - head(r);
    return lo >= reinterpret_cast<uintptr_t>(base) && lo + bytes(r) <= reinterpret_cast<uintptr_t>(row(rows - 1) + cols);
  }
  __device__ __forceinline__ void issue(uint8_t* slot, uint32_t bar, int64_t r) const {
    bulk_load_1d(smem_u32(slot), reinterpret_cast<const uint8_t*>(row(r)) - head(r), bytes(r), bar);
  }
};

// Bytes of a slot for rows of `row_bytes`.
__host__ __device__ constexpr int slot_bytes(int row_bytes, bool whole) { return (row_bytes + 15) / 16 * 16 + (whole ? 0 : 16); }

// Block-wide sum over 1024 threads (all threads get it); `red` holds 32 floats.
__device__ __forceinline__ float block_sum_1024(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(red[threadIdx.x & 31]);
}

// ---------------------------------------------------------------- host
using namespace mxq_host;

constexpr int kMaxRowElems = 32768;       // forward: one CTA's registers

inline int round_up(int v, int m) { return (v + m - 1) / m * m; }

template <typename TX, int OUT, int VE, int NV>
int launch_row(const NormArgs& a, bool warp, int threads, cudaStream_t st) {
  if (warp)
    return launch_pdl(norm_row_kernel<TX, OUT, VE, NV, true>, dim3((a.rows + 7) / 8), dim3(256), 0, st, a);
  return launch_pdl(norm_row_kernel<TX, OUT, VE, NV, false>, dim3(a.rows), dim3(threads), 0, st, a);
}

// One row per warp while a lane holds at most 32 elements (8 without vectors),
// else one per CTA of just enough warps that a thread does.  Single elements
// go eight to a thread while 1024 threads hold the row: with 32 the loads
// spill (1531 x 2049 float32: 16.3 us, 8.4 with eight).
template <typename TX, int OUT, int VE>
int dispatch_row(const NormArgs& a, cudaStream_t st) {
  const int nvec = a.cols / VE;
  if constexpr (VE == 1) {
    const int nv = nvec <= 8 * 1024 ? 8 : 32;
    const bool warp = nvec <= 32 * 8;
    const int threads = round_up((nvec + nv - 1) / nv, 32);
    return nv == 8 ? launch_row<TX, OUT, 1, 8>(a, warp, threads, st) : launch_row<TX, OUT, 1, 32>(a, false, threads, st);
  } else {
    constexpr int MAXV = 32 / VE;
    const bool warp = nvec <= 32 * MAXV;
    const int threads = warp ? 32 : round_up((nvec + MAXV - 1) / MAXV, 32);
    const int nv = (nvec + threads - 1) / threads;
    if (nv <= 1) return launch_row<TX, OUT, VE, 1>(a, warp, threads, st);
    if (nv <= 2) return launch_row<TX, OUT, VE, 2>(a, warp, threads, st);
    if constexpr (MAXV >= 8)
      if (nv <= MAXV / 2) return launch_row<TX, OUT, VE, MAXV / 2>(a, warp, threads, st);
    return launch_row<TX, OUT, VE, MAXV>(a, warp, threads, st);
  }
}

// Groups of G threads in a CTA: more than one warp takes a named barrier each.
inline int ring_groups(int threads, int G) { return std::min(G > 32 ? MAX_BARRIERS : MAX_GROUPS, threads / G); }

inline int check_norm(const void* x, int64_t rows, int64_t cols, int64_t ld, int x_type, const void* w, int w_type,
               const void* b, int b_type, const float* mean, const float* rstd) {
  if (!valid_type(x_type) || (w && !valid_type(w_type)) || (b && !valid_type(b_type))) return MXQ_ERR_BAD_ARG;
  if (rows < 0 || cols < 1 || ld < cols) return MXQ_ERR_BAD_SHAPE;
  if (rows > 0x7FFFFFF0ll || cols > kMaxCols) return MXQ_ERR_BAD_SHAPE;
  if (rows && (!x || !mean || !rstd)) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(x, type_size(x_type)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4)) return MXQ_ERR_MISALIGNED;
  if ((w && !aligned_to(w, type_size(w_type))) || (b && !aligned_to(b, type_size(b_type)))) return MXQ_ERR_MISALIGNED;
  return MXQ_OK;
}

inline NormArgs norm_args(const void* x, int64_t rows, int64_t cols, int64_t ld, const void* w, int w_type, const void* b,
                   int b_type, float eps, float* mean, float* rstd) {
  NormArgs a{};
  a.x = x, a.ld = ld, a.rows = static_cast<int>(rows), a.cols = static_cast<int>(cols);
  a.w = w, a.b = b, a.w_f32 = w_type == MXQ_F32, a.b_f32 = b_type == MXQ_F32;
  a.eps = eps, a.mean = mean, a.rstd = rstd;
  return a;
}

// Statistics only (mean and rstd of every row), for 16-byte aligned rows.
int norm_stats(const NormArgs& a, int x_type, cudaStream_t st);

}  // namespace mxq
