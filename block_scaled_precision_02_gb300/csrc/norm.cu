// Layer norm over the rows of a matrix: y = (x - mean) * rstd * w + b, as
// bf16 / float32 or straight to MX codes and scales, and its backward pass
// with the reduction of the weight's and bias's gradients.
//
// Statistics are float32 and come from the data held in registers: partial
// means and sums of squared deviations merge as
//   M2(A+B) = M2(A) + M2(B) + n_A (mean_A - mean)^2 + n_B (mean_B - mean)^2,
// which does not cancel when the mean is large against the spread.
#include <algorithm>
#include <atomic>

#include "rowops.cuh"

namespace mxq {
namespace {

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

// 1 / sqrt(v): the hardware's estimate and one Newton step, within 2 ulp.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return r * fmaf(-0.5f * v * r, r, 1.5f);
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

// Elements of a row of `cols` that warp w of a group of G threads holds, when
// thread t holds the vectors k*G + t.
template <int VE, int NV>
__device__ __forceinline__ int warp_count(int cols, int G, int w) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) n += max(0, min(32 * VE, cols - (k * G + 32 * w) * VE));
  return n;
}

// Sum of squared deviations of a thread's valid vectors from m.
template <int VE, int NV>
__device__ __forceinline__ float sq_dev(const float (&v)[NV][VE], float m, int t, int G, int nvec) {
  float s[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float d[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) d[j] = (v[k][j] - m) * (v[k][j] - m);
    s[k] = k * G + t < nvec ? tree_sum(d) : 0.f;
  }
  return tree_sum(s);
}

// One row per warp (WARP: eight rows per CTA, no barrier) or per CTA (one
// barrier); the row stays in registers, VE * NV elements per thread, so x is
// read once and y written once: HBM bounds it.
template <typename TX, int OUT, int VE, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) norm_row_kernel(const NormArgs a) {
  __shared__ float2 part[32];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = WARP ? 32 : blockDim.x, t = WARP ? lane : threadIdx.x;
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
      if (k * G + t < nvec) raw[k].load(x + (k * G + t) * VE);
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
    m2 = warp_sum(sq_dev<VE, NV>(v, mean, t, G, nvec));
  } else {
    const int n = warp_count<VE, NV>(a.cols, G, warp);
    m2 = warp_sum(sq_dev<VE, NV>(v, n ? sum / static_cast<float>(n) : 0.f, t, G, nvec));
    if (lane == 0) part[warp] = make_float2(sum, m2);
    __syncthreads();
    const bool have = lane < (G >> 5);
    const float2 pw = have ? part[lane] : make_float2(0.f, 0.f);
    const int nw = have ? warp_count<VE, NV>(a.cols, G, lane) : 0;
    mean = warp_sum(pw.x) * inv_c;
    const float d = nw ? pw.x / static_cast<float>(nw) - mean : 0.f;
    m2 = warp_sum(pw.y + static_cast<float>(nw) * d * d);
  }
  const float rstd = 1.f / sqrtf(m2 * inv_c + a.eps);
  if (t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }

  if constexpr (OUT < 0) {
    using TY = typename std::conditional<OUT == OUT_F32, float, __nv_bfloat16>::type;
    if (!a.y) return;
    TY* y = static_cast<TY*>(a.y) + row * a.cols;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int at = (k * G + t) * VE;
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
      const int at = (k * G + t) * VE;
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

// ---------------------------------------------------------------- many rows
// Groups of threads in a persistent CTA, each with a ring of whole rows in
// shared memory that one of its threads fills by bulk copies ahead of use.
// A row moves from its slot to registers; the barrier of the group's
// reduction says that all have read it, and the slot takes a later row of the
// group.  Loads stay in flight through reductions and stores, which registers
// alone do not allow (the row kernel's CTAs load, reduce and store in turn).
// The elements' arithmetic runs on packed pairs.
constexpr int MAX_GROUPS = 32, MAX_STAGES = 8;
constexpr int MAX_BARRIERS = 15;           // named barriers 1..15; a group of one warp needs none
constexpr int FWD_THREADS = 640, BWD_THREADS = 512;
constexpr int BWD_KEEP = 16;               // elements of a thread whose x and dy stay in registers
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

// Weight and bias as float32 in shared memory.  Vectors of four or eight
// elements read them as 16-byte words without bank conflicts: the second
// halves of eight-element vectors have a plane of their own.  Single elements
// read (w, b) pairs.
template <int VE>
__device__ __forceinline__ int plane_at(int e, int cols) {
  if constexpr (VE == 8) return ((e >> 2) & 1) * (cols / 2) + (e >> 3) * 4 + (e & 3);
  return e;
}
template <int VE>
__device__ __forceinline__ void stage_affine(const NormArgs& a, float* ws) {
  for (int i = threadIdx.x; i < a.cols / VE; i += blockDim.x) {
    float w[VE], b[VE];
    load_affine<VE>(a, i * VE, w, b);
    if constexpr (VE == 1) {
      *reinterpret_cast<float2*>(ws + 2 * i) = make_float2(w[0], b[0]);
    } else {
#pragma unroll
      for (int j = 0; j < VE; j += 4) {
        const int at = plane_at<VE>(i * VE + j, a.cols);
        *reinterpret_cast<float4*>(ws + at) = make_float4(w[j], w[j + 1], w[j + 2], w[j + 3]);
        *reinterpret_cast<float4*>(ws + a.cols + at) = make_float4(b[j], b[j + 1], b[j + 2], b[j + 3]);
      }
    }
  }
}
template <int VE>
__device__ __forceinline__ void staged(const float* ws, int at, int cols, float (&w)[VE]) {
#pragma unroll
  for (int i = 0; i < VE; i += 4) {
    const float4 t = *reinterpret_cast<const float4*>(ws + plane_at<VE>(at + i, cols));
    w[i] = t.x, w[i + 1] = t.y, w[i + 2] = t.z, w[i + 3] = t.w;
  }
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

template <typename TX, typename TY, int VE, int NV, bool FULL>
__global__ void __launch_bounds__(FWD_THREADS, 1) norm_ring_kernel(const NormArgs a, int G, int stages, int* status) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 part[2][FWD_THREADS / 32];
  __shared__ __align__(8) uint64_t full[MAX_GROUPS][MAX_STAGES];
  const int lane = threadIdx.x & 31;
  const int P = blockDim.x / G, g = threadIdx.x / G, t = threadIdx.x - g * G;
  const int gw = t >> 5, wpg = G >> 5;
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[g][i]), 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  grid_dep_launch();
  float* ws = reinterpret_cast<float*>(ring);
  const RowSource<TX> src{static_cast<const TX*>(a.x), a.ld, a.cols, a.rows};
  const int nvec = a.cols / VE;
  const int sb = slot_bytes(a.cols * static_cast<int>(sizeof(TX)), VE > 1);
  uint8_t* slots = ring + slot_bytes(8 * a.cols, true) + static_cast<size_t>(g) * stages * sb;
  const int64_t gi = static_cast<int64_t>(blockIdx.x) * P + g, step = static_cast<int64_t>(gridDim.x) * P;
  const float inv_c = 1.f / static_cast<float>(a.cols);
  const int n_mine = warp_count<VE, NV>(a.cols, G, gw), n_lane = lane < wpg ? warp_count<VE, NV>(a.cols, G, lane) : 0;
  const float inv_mine = n_mine ? 1.f / static_cast<float>(n_mine) : 0.f;
  const float inv_lane = n_lane ? 1.f / static_cast<float>(n_lane) : 0.f;
  bool alive = true;
  const auto issue = [&](int slot, int64_t row) {
    const uint32_t bar = smem_u32(&full[g][slot]);
    const bool copy = VE > 1 || src.copied(row);
    mbar_arrive_expect_tx(bar, copy ? src.bytes(row) : 0u);
    if (copy) src.issue(slots + slot * sb, bar, row);
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i)
      if (gi + i * step < a.rows) issue(i, gi + i * step);
  stage_affine<VE>(a, ws);
  __syncthreads();

  int slot = 0, phase = 0, buf = 0;
  for (int64_t row = gi; row < a.rows; row += step) {
    if (alive) alive = mbar_wait(smem_u32(&full[g][slot]), phase, status);
    Vec<TX, VE> v[NV];                                   // as loaded: widened anew at each use
    float s[NV];
    const auto take = [&](const TX* from) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!FULL) v[k].fill(0);
        if (FULL || k * G + t < nvec) v[k].load(from + (k * G + t) * VE);
      }
    };
    const auto wide = [&](int k, float (&f)[VE]) {
#pragma unroll
      for (int j = 0; j < VE; ++j) f[j] = v[k].get(j);
    };
    if (VE > 1 || src.copied(row)) take(reinterpret_cast<const TX*>(slots + slot * sb + (VE > 1 ? 0 : src.head(row))));
    else take(src.row(row));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float f[VE];
      wide(k, f);
      s[k] = vec_sum(f);
    }
    float sum = warp_sum(tree_sum(s));
    const float near = wpg == 1 ? sum * inv_c : sum * inv_mine;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float f[VE];
      wide(k, f);
      s[k] = FULL || k * G + t < nvec ? vec_sq_dev(f, near) : 0.f;
    }
    float mean = near, m2 = warp_sum(tree_sum(s));
    if (wpg > 1) {
      if (lane == 0) part[buf][g * wpg + gw] = make_float2(sum, m2);
      group_barrier(g, G);
    } else {
      __syncwarp();
    }
    if (t == 0 && row + stages * step < a.rows) issue(slot, row + stages * step);     // all have read the slot
    if (++slot == stages) slot = 0, phase ^= 1;
    if (wpg > 1) {
      const float2 pw = lane < wpg ? part[buf][g * wpg + lane] : make_float2(0.f, 0.f);
      buf ^= 1;
      mean = warp_sum(pw.x) * inv_c;
      const float d = n_lane ? pw.x * inv_lane - mean : 0.f;
      m2 = warp_sum(pw.y + static_cast<float>(n_lane) * d * d);
    }
    const float rstd = inv_sqrt(m2 * inv_c + a.eps);
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    TY* y = static_cast<TY*>(a.y) + row * a.cols;
    const float2 mm = splat(mean), rr = splat(rstd);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int at = (k * G + t) * VE;
      if (!FULL && at >= a.cols) continue;
      float f[VE], o[VE];
      wide(k, f);
      if constexpr (VE == 1) {
        const float2 wb = *reinterpret_cast<const float2*>(ws + 2 * at);
        o[0] = norm_value(f[0], mean, rstd, wb.x, wb.y);
      } else {
        float w[VE], b[VE];
        staged<VE>(ws, at, a.cols, w);
        staged<VE>(ws + a.cols, at, a.cols, b);
#pragma unroll
        for (int j = 0; j < VE; j += 2)
          halves(fma2(mul2(sub2(pair(f[j], f[j + 1]), mm), rr), pair(w[j], w[j + 1]),
                                 pair(b[j], b[j + 1])),
                       o[j], o[j + 1]);
      }
      store_vec<TY, VE>(y + at, o);
    }
  }
  if (!alive && t == 0) await_ring(full[g], stages, slot, phase, status);
}

// Block-wide sum over 1024 threads (all threads get it); `red` holds 32 floats.
__device__ __forceinline__ float block_sum_1024(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(red[threadIdx.x & 31]);
}

// Rows too long for the registers of one CTA (more than 32768 elements): one
// CTA per row and three passes over it (sum, deviations, output), the later
// two from L2.
template <typename TX, int OUT>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  __shared__ float red[32];
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + row * a.ld;
  const float inv_c = 1.f / static_cast<float>(a.cols);
  Vec<TX, 1> e;
  float s = 0.f;
  for (int i = threadIdx.x; i < a.cols; i += 1024) {
    e.load(x + i);
    s += e.get(0);
  }
  const float mean = block_sum_1024(s, red) * inv_c;
  s = 0.f;
  for (int i = threadIdx.x; i < a.cols; i += 1024) {
    e.load(x + i);
    s += (e.get(0) - mean) * (e.get(0) - mean);
  }
  const float rstd = 1.f / sqrtf(block_sum_1024(s, red) * inv_c + a.eps);
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  if (!a.y) return;
  using TY = typename std::conditional<OUT == OUT_F32, float, __nv_bfloat16>::type;
  TY* y = static_cast<TY*>(a.y) + row * a.cols;
  for (int i = threadIdx.x; i < a.cols; i += 1024) {
    float w[1], b[1], o[1];
    load_affine<1>(a, i, w, b);
    e.load(x + i);
    o[0] = norm_value(e.get(0), mean, rstd, w[0], b[0]);
    store_vec<TY, 1>(y + i, o);
  }
}

// Quantizing norm with column blocks.  A CTA walks over tiles of 32 rows and
// up to S columns.  A warp holds its rows' words in registers, 16 consecutive
// columns to a lane: it takes their statistics, then computes y once, encodes
// the row blocks (two lanes each), and leaves y as float32 in shared memory,
// where a thread then finds whole column blocks.  x is read from HBM once for
// both copies.  CLUSTER: the CTAs of a cluster hold the slabs of the same
// rows; each warp sends its rows' (sum, M2) of the slab to every CTA by
// counted asynchronous stores and merges what arrives.  Otherwise the
// statistics are given.
//
// y lies in four planes of S / 4: column 16 i + 4 p + q at p S/4 + 4 i + q,
// so that a lane's sixteen values go out as four 16-byte stores without bank
// conflicts.
__device__ __forceinline__ void store32(uint8_t* p, const uint32_t (&q)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(q[0]), "r"(q[1]), "r"(q[2]),
               "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7])
               : "memory");
}

constexpr int TILE_SLABS = 8;                            // CTAs of a cluster (the portable limit)

template <typename TX, int FMT, int ORIENT, bool CLUSTER, int S, int T>
__global__ void __launch_bounds__(T, T == 256 ? 2 : 1) norm_tile_kernel(const NormArgs a, int slabs, int* status) {
  constexpr int RW = 32 / (T / 32);                      // rows of a warp
  constexpr int GS = 32 / RW;                            // lanes that end up with a row's sums
  constexpr int NV = S / 512;                            // runs of 16 columns of a lane
  constexpr int WV = 16 / static_cast<int>(sizeof(TX));  // elements of a 16-byte word
  constexpr int NW = 16 / WV;                            // words of a run
  extern __shared__ __align__(16) float wtile[];         // weight [S], bias [S], y [32][S], in planes
  float* const btile = wtile + S;
  float* const ytile = wtile + 2 * S;
  __shared__ float2 parts[2][TILE_SLABS][32];            // [buffer][rank][row] (sum, M2)
  __shared__ __align__(8) uint64_t bar[2];
  if constexpr (CLUSTER) {
    if (threadIdx.x == 0) {
      mbar_init(smem_u32(&bar[0]), 1);
      mbar_init(smem_u32(&bar[1]), 1);
      fence_mbar_init();
    }
    cluster_sync();
  }
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % slabs;
  const int tiles = a.rows / 32;
  const int team = blockIdx.x / slabs, teams = gridDim.x / slabs;
  // a contiguous range of tiles: four in a row share a word of column scales
  const int first = static_cast<int>(static_cast<int64_t>(tiles) * team / teams);
  const int last = static_cast<int>(static_cast<int64_t>(tiles) * (team + 1) / teams);
  const int c0 = rank * S;
  const int nc = min(S, a.cols - c0);                    // columns of this slab (a multiple of 32)
  const float inv_nc = 1.f / static_cast<float>(nc), inv_c = 1.f / static_cast<float>(a.cols);
  const int lr = lane / GS, lk = lane % GS;              // this lane's row and slab in the merge
  const float n_k = static_cast<float>(lk < slabs ? min(S, a.cols - lk * S) : 0);
  bool alive = true;

  Vec<TX, WV> raw[RW][NV][NW];
  const auto load = [&](int tile) {
    const TX* x = static_cast<const TX*>(a.x) + (static_cast<int64_t>(tile) * 32 + warp * RW) * a.ld + c0 + lane * 16;
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          raw[r][v][i].fill(0);
          if (v * 512 + lane * 16 < nc) raw[r][v][i].load(x + r * a.ld + v * 512 + i * WV);
        }
  };
  const auto run = [&](int r, int v, float (&f)[16]) {
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int j = 0; j < WV; ++j) f[i * WV + j] = raw[r][v][i].get(j);
  };
  // one value per row, added over the warp: the lanes of group r end with row r's
  const auto rows_sum = [&](const float (&s)[RW]) {
    float b;
    if constexpr (RW == 4) {
      const bool hi = lane & 16;
      const float a0 = (hi ? s[2] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? s[0] : s[2], 16);
      const float a1 = (hi ? s[3] : s[1]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? s[1] : s[3], 16);
      const bool up = lane & 8;
      b = (up ? a1 : a0) + __shfl_xor_sync(0xFFFFFFFFu, up ? a0 : a1, 8);
    } else {
      const bool hi = lane & 16;
      b = (hi ? s[1] : s[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? s[0] : s[1], 16);
    }
#pragma unroll
    for (int o = GS / 2; o; o >>= 1) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    return b;
  };
  const auto group_sum = [&](float b) {
#pragma unroll
    for (int o = GS / 2; o; o >>= 1) b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    return b;
  };

  uint32_t col_scales[S / T];                            // this thread's columns, a byte per tile
  if (first < last) load(first);
  for (int c = threadIdx.x * 4; c < nc; c += T * 4) {
    float w[4], b[4];
    load_affine<4>(a, c0 + c, w, b);
    const int at = (c & 15) / 4 * (S / 4) + c / 16 * 4;
    *reinterpret_cast<float4*>(wtile + at) = make_float4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<float4*>(btile + at) = make_float4(b[0], b[1], b[2], b[3]);
  }
  __syncthreads();
  for (int tile = first; tile < last; ++tile) {
    const int64_t row0 = static_cast<int64_t>(tile) * 32;
    float mean, rstd;                                    // of row lr of this warp
    if constexpr (CLUSTER) {
      const int buf = (tile - first) & 1;
      if (threadIdx.x == 0) mbar_arrive_expect_tx(smem_u32(&bar[buf]), 256 * slabs);
      float s[RW];
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        s[r] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float f[16];
          run(r, v, f);
          s[r] += vec_sum(f);
        }
      }
      const float sum = rows_sum(s);
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const float near = __shfl_sync(0xFFFFFFFFu, sum, r * GS) * inv_nc;
        s[r] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float f[16];
          run(r, v, f);
          if (v * 512 + lane * 16 < nc) s[r] += vec_sq_dev(f, near);
        }
      }
      const float m2 = rows_sum(s);
      if (lk < slabs)
        st_async_f2(smem_u32(&parts[buf][rank][warp * RW + lr]), smem_u32(&bar[buf]), lk, sum, m2);
      if (alive) alive = mbar_wait_sleep(smem_u32(&bar[buf]), ((tile - first) >> 1) & 1, status);
      const float2 p = lk < slabs ? parts[buf][lk][warp * RW + lr] : make_float2(0.f, 0.f);
      mean = group_sum(p.x) * inv_c;
      const float d = lk < slabs ? p.x / n_k - mean : 0.f;
      rstd = inv_sqrt(group_sum(p.y + n_k * d * d) * inv_c + a.eps);
      if (rank == 0 && lk == 0) {
        a.mean[row0 + warp * RW + lr] = mean;
        a.rstd[row0 + warp * RW + lr] = rstd;
      }
    } else {
      mean = a.mean[row0 + warp * RW + lr];
      rstd = a.rstd[row0 + warp * RW + lr];
    }

#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = v * 512 + lane * 16;
      const bool valid = at < nc;
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const int64_t row = row0 + warp * RW + r;
        const float2 mm = splat(__shfl_sync(0xFFFFFFFFu, mean, r * GS));
        const float2 rr = splat(__shfl_sync(0xFFFFFFFFu, rstd, r * GS));
        float y[16];
        float m = 0.f;
        if (valid) {
          run(r, v, y);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int po = p * (S / 4) + at / 4;
            const float4 w = *reinterpret_cast<const float4*>(wtile + po), b = *reinterpret_cast<const float4*>(btile + po);
            const float2 u0 = fma2(mul2(sub2(pair(y[4 * p], y[4 * p + 1]), mm), rr), pair(w.x, w.y), pair(b.x, b.y));
            const float2 u1 = fma2(mul2(sub2(pair(y[4 * p + 2], y[4 * p + 3]), mm), rr), pair(w.z, w.w), pair(b.z, b.w));
            y[4 * p] = u0.x, y[4 * p + 1] = u0.y, y[4 * p + 2] = u1.x, y[4 * p + 3] = u1.y;
            m = fmax3_nan(m, fabsf(u0.x), fabsf(u0.y));
            m = fmax3_nan(m, fabsf(u1.x), fabsf(u1.y));
            if constexpr (ORIENT & MXQ_COL)
              *reinterpret_cast<float4*>(ytile + (warp * RW + r) * S + po) = make_float4(u0.x, u0.y, u1.x, u1.y);
          }
        }
        if constexpr (ORIENT & MXQ_ROW) {
          m = fmax3_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1), 0.f);
          float mult;
          const uint32_t code = mx_scale<FMT>(__float_as_uint(m) & 0x7FFFFFFFu, a.ceil_mode, mult);
          if (valid) {
            uint32_t q[code_words<FMT, 16>()];
            mx_codes<FMT, 16>(y, mult, code == 0xFFu, q);
            const int64_t el = row * a.cols + c0 + at;
            uint8_t* dst = a.q_row + (FMT == MXQ_E2M1 ? el / 2 : el);
            if constexpr (FMT == MXQ_E2M1) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
            else *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
          }
          const int kb = a.cols / 32, k = (c0 + at) / 32;
          if (a.pack_row) {                              // the scales of four neighbouring blocks as one word
            uint32_t word = code << (8 * ((lane >> 1) & 3));
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
            if (valid && lane % 8 == 0) *reinterpret_cast<uint32_t*>(a.s_row + scale_at(row, k, kb, a.mma)) = word;
          } else if (valid && lane % 2 == 0) {
            a.s_row[scale_at(row, k, kb, a.mma)] = static_cast<uint8_t>(code);
          }
        }
      }
    }
    if (tile + 1 < last) load(tile + 1);                 // in flight through the column pass

    if constexpr (ORIENT & MXQ_COL) {
      __syncthreads();
      const int kb = a.rows / 32;
      // the word of scales is complete when its four tiles are all this CTA's
      const bool flush = (tile & 3) == 3 || tile + 1 == last;
      const bool word = a.pack_col && (tile & 3) == 3 && tile - 3 >= first;
#pragma unroll
      for (int u = 0; u < S / T; ++u) {
        const int pos = threadIdx.x + u * T;             // a column of a plane
        const int c = (pos % (S / 4)) / 4 * 16 + pos / (S / 4) * 4 + pos % 4;
        if (c >= nc) continue;
        float y[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) y[r] = ytile[r * S + pos];
        float mult;
        const uint32_t code = mx_scale<FMT>(amax32_tree([&](int j) { return fabsf(y[j]); }), a.ceil_mode, mult);
        uint32_t q[code_words<FMT, 32>()];
        mx_codes<FMT, 32>(y, mult, code == 0xFFu, q);
        const int64_t el = static_cast<int64_t>(c0 + c) * a.rows + row0;
        uint8_t* dst = a.q_col + (FMT == MXQ_E2M1 ? el / 2 : el);
        if constexpr (FMT == MXQ_E2M1) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
        } else if (a.wide_col) {
          store32(dst, q);
        } else {
          *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
          *reinterpret_cast<uint4*>(dst + 16) = make_uint4(q[4], q[5], q[6], q[7]);
        }
        uint32_t& acc = col_scales[u];
        acc = ((tile & 3) == 0 || tile == first ? 0u : acc) | code << (8 * (tile & 3));
        if (word) {
          *reinterpret_cast<uint32_t*>(a.s_col + scale_at(c0 + c, tile - 3, kb, a.mma)) = acc;
        } else if (flush) {
          for (int k = max(first, tile & ~3); k <= tile; ++k)
            a.s_col[scale_at(c0 + c, k, kb, a.mma)] = static_cast<uint8_t>(acc >> (8 * (k & 3)));
        }
      }
      __syncthreads();
    }
  }
  // peers may still be sending: they wait for this CTA's sums, it for theirs,
  // so nothing is on its way once every tile is merged -- unless a wait gave up
  if constexpr (CLUSTER) cluster_sync();
}

// ---------------------------------------------------------------- backward
struct BwdArgs {
  const void* dy;
  int64_t ld_dy;
  const void* x;
  int64_t ld_x;
  int rows, cols;
  const float* mean;
  const float* rstd;
  const void* w;
  int w_f32;
  void* dx;               // [rows][cols], the type of x
  float* part;            // [parts][2][cols] sums of dy*h and dy over a CTA's rows; NULL: not wanted
  float* coef;            // [rows][2] (long rows only)
};

// A thread owns VE * NV columns and keeps their two column sums in registers
// while its CTA walks over rows, RB per step (their loads are in flight
// together and share one barrier); a group of G threads has a row.  x and dy
// are read once and dx written once, so HBM bounds it; the column sums of a
// CTA go out once at the end and a second kernel adds them up in a fixed
// order.
template <typename TX, typename TD, int VE, int NV, int RB>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const BwdArgs a, int G) {
  __shared__ float2 red[2][RB][32];
  extern __shared__ __align__(16) float comb[];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = blockDim.x / G, g = threadIdx.x / G, t = threadIdx.x - g * G;
  const int wpg = G >> 5;
  const int nvec = a.cols / VE;
  const float inv_c = 1.f / static_cast<float>(a.cols);

  float w[NV][VE], aw[NV][VE], ab[NV][VE];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      w[k][j] = 1.f;
      aw[k][j] = ab[k][j] = 0.f;
    }
    if (a.w && k * G + t < nvec) load_param<VE>(a.w, a.w_f32, (k * G + t) * VE, w[k]);
  }

  int buf = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * P * RB;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * P * RB; base < a.rows; base += step) {
    const int64_t row = base + g * RB;
    Vec<TX, VE> xr[RB][NV];
    Vec<TD, VE> dr[RB][NV];
    float mean[RB], rstd[RB], c1[RB], c2[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const bool in = row + r < a.rows;
      mean[r] = in ? a.mean[row + r] : 0.f;
      rstd[r] = in ? a.rstd[row + r] : 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        xr[r][k].fill(0);
        dr[r][k].fill(0);
        if (in && k * G + t < nvec) {
          xr[r][k].load(static_cast<const TX*>(a.x) + (row + r) * a.ld_x + (k * G + t) * VE);
          dr[r][k].load(static_cast<const TD*>(a.dy) + (row + r) * a.ld_dy + (k * G + t) * VE);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float s1[NV], s2[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float u[VE], v[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float h = (xr[r][k].get(j) - mean[r]) * rstd[r];
          const float d = dr[r][k].get(j);
          u[j] = d * w[k][j];
          v[j] = u[j] * h;
          aw[k][j] = fmaf(d, h, aw[k][j]);
          ab[k][j] += d;
        }
        s1[k] = tree_sum(u);
        s2[k] = tree_sum(v);
      }
      c1[r] = warp_sum(tree_sum(s1));
      c2[r] = warp_sum(tree_sum(s2));
    }
    if (wpg > 1) {
      if (lane == 0)
#pragma unroll
        for (int r = 0; r < RB; ++r) red[buf][r][warp] = make_float2(c1[r], c2[r]);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        c1[r] = c2[r] = 0.f;
        for (int i = 0; i < wpg; ++i) {
          const float2 v = red[buf][r][g * wpg + i];
          c1[r] += v.x;
          c2[r] += v.y;
        }
      }
      buf ^= 1;
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      if (row + r >= a.rows) continue;
      const float m1 = c1[r] * inv_c, m2 = c2[r] * inv_c;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (k * G + t >= nvec) continue;
        float o[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float h = (xr[r][k].get(j) - mean[r]) * rstd[r];
          o[j] = (fmaf(dr[r][k].get(j), w[k][j], -m1) - h * m2) * rstd[r];
        }
        store_vec<TX, VE>(static_cast<TX*>(a.dx) + (row + r) * a.cols + (k * G + t) * VE, o);
      }
    }
  }
  if (!a.part) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  if (P > 1) {                      // the groups of the CTA first, in their order
    for (int i = 1; i < P; ++i) {
      __syncthreads();
      if (g == i)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            comb[(2 * (k * VE + j)) * G + t] = aw[k][j];
            comb[(2 * (k * VE + j) + 1) * G + t] = ab[k][j];
          }
      __syncthreads();
      if (g == 0)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            aw[k][j] += comb[(2 * (k * VE + j)) * G + t];
            ab[k][j] += comb[(2 * (k * VE + j) + 1) * G + t];
          }
    }
    if (g) return;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (k * G + t >= nvec) continue;
    if constexpr (VE == 1) {
      out[k * G + t] = aw[k][0];
      out[a.cols + k * G + t] = ab[k][0];
    } else {
      store_vec<float, VE>(out + (k * G + t) * VE, aw[k]);
      store_vec<float, VE>(out + a.cols + (k * G + t) * VE, ab[k]);
    }
  }
}

// The same for many rows, through rings of rows (x and dy side by side in a
// slot).  Up to 16 elements a thread: x and dy stay in registers from the sums
// to dx.  More (KEEP false): the slot is read again for dx and given
// back after the next row's barrier, and the weights are read from shared
// memory, because the column sums fill the registers.
template <typename TX, typename TD, int VE, int NV, bool FULL>
__global__ void __launch_bounds__(BWD_THREADS, 1) norm_bwd_ring_kernel(const BwdArgs a, int G, int stages, int* status) {
  constexpr bool KEEP = VE * NV <= BWD_KEEP;
  constexpr int KV = KEEP ? NV : 1;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][2][BWD_THREADS / 32];     // [buffer][sum][warp of the CTA]
  __shared__ __align__(8) uint64_t full[MAX_GROUPS][MAX_STAGES];
  const int lane = threadIdx.x & 31;
  const int P = blockDim.x / G, g = threadIdx.x / G, t = threadIdx.x - g * G;
  const int gw = t >> 5, wpg = G >> 5;
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[g][i]), 1);
    fence_mbar_init();
  }
  const int nvec = a.cols / VE;
  const RowSource<TX> sx{static_cast<const TX*>(a.x), a.ld_x, a.cols, a.rows};
  const RowSource<TD> sd{static_cast<const TD*>(a.dy), a.ld_dy, a.cols, a.rows};
  const int xb = slot_bytes(a.cols * static_cast<int>(sizeof(TX)), VE > 1);
  const int sb = xb + slot_bytes(a.cols * static_cast<int>(sizeof(TD)), VE > 1);
  const int wsize = a.w_f32 ? 4 : 2;
  uint8_t* ws = ring;                                // !KEEP: the weights, as they are
  uint8_t* slots = ring + (KEEP ? 0 : slot_bytes(wsize * a.cols, true)) + static_cast<size_t>(g) * stages * sb;
  grid_dep_wait();
  grid_dep_launch();
  const float inv_c = 1.f / static_cast<float>(a.cols);
  const int64_t gi = static_cast<int64_t>(blockIdx.x) * P + g, step = static_cast<int64_t>(gridDim.x) * P;
  bool alive = true;
  const auto copied = [&](int64_t row) { return VE > 1 || (sx.copied(row) && sd.copied(row)); };
  const auto issue = [&](int slot, int64_t row) {
    const uint32_t bar = smem_u32(&full[g][slot]);
    const bool copy = copied(row);
    mbar_arrive_expect_tx(bar, copy ? sx.bytes(row) + sd.bytes(row) : 0u);
    if (copy) {
      sx.issue(slots + slot * sb, bar, row);
      sd.issue(slots + slot * sb + xb, bar, row);
    }
  };
  // a vector of x and dy of the row in `slot`
  const auto take = [&](int slot, int64_t row, bool in_ring, int k, Vec<TX, VE>& xv, Vec<TD, VE>& dv) {
    if (!FULL) {
      xv.fill(0);
      dv.fill(0);
      if (k * G + t >= nvec) return;
    }
    if (in_ring) {
      const uint8_t* p = slots + slot * sb;
      xv.load(reinterpret_cast<const TX*>(p + (VE > 1 ? 0 : sx.head(row))) + (k * G + t) * VE);
      dv.load(reinterpret_cast<const TD*>(p + xb + (VE > 1 ? 0 : sd.head(row))) + (k * G + t) * VE);
    } else {
      xv.load(sx.row(row) + (k * G + t) * VE);
      dv.load(sd.row(row) + (k * G + t) * VE);
    }
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i)
      if (gi + i * step < a.rows) issue(i, gi + i * step);
  float w[KV][VE], aw[NV][VE], ab[NV][VE];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = 0; j < VE; ++j) aw[k][j] = ab[k][j] = 0.f;
#pragma unroll
  for (int k = 0; k < KV; ++k) {
#pragma unroll
    for (int j = 0; j < VE; ++j) w[k][j] = 1.f;
    if (KEEP && a.w && k * G + t < nvec) load_param<VE>(a.w, a.w_f32, (k * G + t) * VE, w[k]);
  }
  if (!KEEP && a.w)
    for (int i = threadIdx.x; i < a.cols; i += blockDim.x) {
      if (a.w_f32) reinterpret_cast<float*>(ws)[i] = static_cast<const float*>(a.w)[i];
      else reinterpret_cast<uint16_t*>(ws)[i] = static_cast<const uint16_t*>(a.w)[i];
    }
  __syncthreads();

  int slot = 0, phase = 0, buf = 0;
  float mean_n = gi < a.rows ? a.mean[gi] : 0.f, rstd_n = gi < a.rows ? a.rstd[gi] : 0.f;
  for (int64_t row = gi; row < a.rows; row += step) {
    const float mean = mean_n, rstd = rstd_n;
    if (row + step < a.rows) mean_n = a.mean[row + step], rstd_n = a.rstd[row + step];
    const float2 mm = splat(mean), rr = splat(rstd);
    const bool in_ring = copied(row);
    if (alive) alive = mbar_wait(smem_u32(&full[g][slot]), phase, status);
    Vec<TX, VE> xs[KV];
    Vec<TD, VE> ds[KV];
    if (KEEP)
#pragma unroll
      for (int k = 0; k < NV; ++k) take(slot, row, in_ring, k, xs[KEEP ? k : 0], ds[KEEP ? k : 0]);
    float s1[NV], s2[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Vec<TX, VE>& xv = xs[KEEP ? k : 0];
      Vec<TD, VE>& dv = ds[KEEP ? k : 0];
      if (!KEEP) take(slot, row, in_ring, k, xv, dv);
      float hk[VE], uk[VE], wk[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) wk[j] = KEEP ? w[KEEP ? k : 0][j] : 1.f;
      if (!KEEP && a.w && (FULL || k * G + t < nvec)) load_param<VE>(ws, a.w_f32, (k * G + t) * VE, wk);
      if constexpr (VE == 1) {
        const float d = dv.get(0);
        hk[0] = (xv.get(0) - mean) * rstd;
        uk[0] = d * wk[0];
        aw[k][0] = fmaf(d, hk[0], aw[k][0]);
        ab[k][0] += d;
        s1[k] = uk[0];
        s2[k] = uk[0] * hk[0];
      } else {
        float2 p1, p2;
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
          const float2 hh = mul2(sub2(pair(xv.get(j), xv.get(j + 1)), mm), rr);
          const float2 dd = pair(dv.get(j), dv.get(j + 1));
          const float2 uu = mul2(dd, pair(wk[j], wk[j + 1]));
          halves(fma2(dd, hh, pair(aw[k][j], aw[k][j + 1])), aw[k][j], aw[k][j + 1]);
          halves(add2(dd, pair(ab[k][j], ab[k][j + 1])), ab[k][j], ab[k][j + 1]);
          p1 = j ? add2(p1, uu) : uu;
          p2 = j ? fma2(uu, hh, p2) : mul2(uu, hh);
          halves(hh, hk[j], hk[j + 1]);
          halves(uu, uk[j], uk[j + 1]);
        }
        float x, y;
        halves(p1, x, y);
        s1[k] = x + y;
        halves(p2, x, y);
        s2[k] = x + y;
      }
    }
    // both sums in one butterfly: the lower half of the warp takes the first,
    // the upper half the second
    const float c1 = tree_sum(s1), c2 = tree_sum(s2);
    const bool up = lane & 16;
    float v = (up ? c2 : c1) + __shfl_xor_sync(0xFFFFFFFFu, up ? c1 : c2, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (wpg > 1) {
      if ((lane & 15) == 0) red[buf][lane >> 4][g * wpg + gw] = v;
      group_barrier(g, G);
    } else {
      __syncwarp();
    }
    if (t == 0) {
      if constexpr (KEEP) {                  // all have read this slot
        if (row + stages * step < a.rows) issue(slot, row + stages * step);
      } else {                               // all are done with the last one
        const int64_t next = row + (stages - 1) * step;
        if (row != gi && next < a.rows) issue(slot ? slot - 1 : stages - 1, next);
      }
    }
    if (wpg > 1) {
      const float* half = red[buf][lane >> 4] + g * wpg + (lane & 15);
      v = (lane & 15) < wpg ? half[0] : 0.f;
      if (wpg > 16) v += (lane & 15) + 16 < wpg ? half[16] : 0.f;
#pragma unroll
      for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      buf ^= 1;
    }
    const float m1 = __shfl_sync(0xFFFFFFFFu, v, 0) * inv_c, m2 = __shfl_sync(0xFFFFFFFFu, v, 16) * inv_c;
    TX* dx = static_cast<TX*>(a.dx) + row * a.cols;
    const float2 c1c1 = splat(m1), c2c2 = splat(-m2);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!FULL && k * G + t >= nvec) continue;
      float hk[VE], uk[VE], o[VE];
      Vec<TX, VE>& xv = xs[KEEP ? k : 0];
      Vec<TD, VE>& dv = ds[KEEP ? k : 0];
      if (!KEEP) take(slot, row, in_ring, k, xv, dv);
      float wk[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) wk[j] = KEEP ? w[KEEP ? k : 0][j] : 1.f;
      if (!KEEP && a.w) load_param<VE>(ws, a.w_f32, (k * G + t) * VE, wk);
      if constexpr (VE == 1) {
        hk[0] = (xv.get(0) - mean) * rstd;
        uk[0] = dv.get(0) * wk[0];
      } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
          halves(mul2(sub2(pair(xv.get(j), xv.get(j + 1)), mm), rr), hk[j], hk[j + 1]);
          halves(mul2(pair(dv.get(j), dv.get(j + 1)), pair(wk[j], wk[j + 1])), uk[j], uk[j + 1]);
        }
      }
      if constexpr (VE == 1) {
        o[0] = fmaf(hk[0], -m2, uk[0] - m1) * rstd;
      } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2)
          halves(mul2(fma2(pair(hk[j], hk[j + 1]), c2c2,
                                           sub2(pair(uk[j], uk[j + 1]), c1c1)),
                                 rr),
                       o[j], o[j + 1]);
      }
      store_vec<TX, VE>(dx + (k * G + t) * VE, o);
    }
    if (++slot == stages) slot = 0, phase ^= 1;
  }
  if (!alive && t == 0) await_ring(full[g], stages, slot, phase, status);
  if (!a.part) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  float* comb = reinterpret_cast<float*>(ring);
  for (int i = 1; i < P; ++i) {              // the groups of the CTA, in their order
    __syncthreads();                         // (every copy has been waited for: the ring is free)
    if (g == i)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          comb[(2 * (k * VE + j)) * G + t] = aw[k][j];
          comb[(2 * (k * VE + j) + 1) * G + t] = ab[k][j];
        }
    __syncthreads();
    if (g == 0)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          aw[k][j] += comb[(2 * (k * VE + j)) * G + t];
          ab[k][j] += comb[(2 * (k * VE + j) + 1) * G + t];
        }
  }
  if (g) return;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (k * G + t >= nvec) continue;
    store_vec<float, VE>(out + (k * G + t) * VE, aw[k]);
    store_vec<float, VE>(out + a.cols + (k * G + t) * VE, ab[k]);
  }
}

// Rows too long for the registers: their two sums first ...
template <typename TX, typename TD>
__global__ void __launch_bounds__(1024) norm_bwd_long_rows_kernel(const BwdArgs a) {
  __shared__ float red[32];
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + row * a.ld_x;
  const TD* dy = static_cast<const TD*>(a.dy) + row * a.ld_dy;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float c1 = 0.f, c2 = 0.f;
  for (int i = threadIdx.x; i < a.cols; i += 1024) {
    Vec<TX, 1> xe;
    Vec<TD, 1> de;
    xe.load(x + i);
    de.load(dy + i);
    float w[1] = {1.f};
    if (a.w) load_param<1>(a.w, a.w_f32, i, w);
    const float u = de.get(0) * w[0];
    c1 += u;
    c2 += u * ((xe.get(0) - mean) * rstd);
  }
  c1 = block_sum_1024(c1, red);
  c2 = block_sum_1024(c2, red);
  if (threadIdx.x == 0) {
    a.coef[2 * row] = c1 / static_cast<float>(a.cols);
    a.coef[2 * row + 1] = c2 / static_cast<float>(a.cols);
  }
}

// ... then a column per thread over a range of rows (blockIdx.y).
template <typename TX, typename TD>
__global__ void __launch_bounds__(256) norm_bwd_long_cols_kernel(const BwdArgs a) {
  grid_dep_wait();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float w[1] = {1.f};
  if (a.w) load_param<1>(a.w, a.w_f32, c, w);
  float aw = 0.f, ab = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    Vec<TX, 1> xe;
    Vec<TD, 1> de;
    xe.load(static_cast<const TX*>(a.x) + row * a.ld_x + c);
    de.load(static_cast<const TD*>(a.dy) + row * a.ld_dy + c);
    const float rstd = a.rstd[row], h = (xe.get(0) - a.mean[row]) * rstd, d = de.get(0);
    aw = fmaf(d, h, aw);
    ab += d;
    float o[1] = {(fmaf(d, w[0], -a.coef[2 * row]) - h * a.coef[2 * row + 1]) * rstd};
    store_vec<TX, 1>(static_cast<TX*>(a.dx) + row * a.cols + c, o);
  }
  if (a.part) {
    a.part[static_cast<int64_t>(blockIdx.y) * 2 * a.cols + c] = aw;
    a.part[static_cast<int64_t>(blockIdx.y) * 2 * a.cols + a.cols + c] = ab;
  }
}

// dw[c], db[c] = sums over the parts, in their order: 32 columns per CTA,
// eight threads per column.
__global__ void __launch_bounds__(256) norm_bwd_sum_kernel(const float* part, int parts, int cols, float* dw, float* db) {
  __shared__ float red[8][33];
  grid_dep_wait();
  const int cx = threadIdx.x & 31, sy = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + cx;      // over both sums
  float s = 0.f;
  if (c < 2ll * cols) {
    const float* p = part + c;
#pragma unroll 8
    for (int i = sy; i < parts; i += 8) s += p[static_cast<int64_t>(i) * 2 * cols];
  }
  red[sy][cx] = s;
  __syncthreads();
  if (sy == 0 && c < 2ll * cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][cx];
    if (c < cols) {
      if (dw) dw[c] = s;
    } else if (db) {
      db[c - cols] = s;
    }
  }
}

// ---------------------------------------------------------------- host
using namespace mxq_host;

constexpr int kMaxRowElems = 32768;       // forward: one CTA's registers
constexpr int kMaxBwdElems = 16384;       // backward: data and two column sums

bool valid_type(int t) { return t == MXQ_BF16 || t == MXQ_F32; }
int type_size(int t) { return t == MXQ_F32 ? 4 : 2; }
bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int round_up(int v, int m) { return (v + m - 1) / m * m; }

template <typename TX, int OUT, int VE, int NV>
int launch_row(const NormArgs& a, bool warp, int threads, cudaStream_t st) {
  if (warp)
    return launch_pdl(norm_row_kernel<TX, OUT, VE, NV, true>, dim3((a.rows + 7) / 8), dim3(256), 0, st, a);
  return launch_pdl(norm_row_kernel<TX, OUT, VE, NV, false>, dim3(a.rows), dim3(threads), 0, st, a);
}

// One row per warp while a lane holds at most 32 elements (8 without vectors),
// else one per CTA of just enough warps that a thread does.  Single elements
// go eight to a thread while 1024 threads hold the row: with 32 the loads
// spill (1531 x 2049 float32: PLACEHOLDER).
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
int ring_groups(int threads, int G) { return std::min(G > 32 ? MAX_BARRIERS : MAX_GROUPS, threads / G); }

// Rings for rows of 512 bytes and more (up to what two slots hold) when every
// group gets four or more.  False: not taken.
template <typename TX, typename TY, int VE>
bool try_norm_ring(const NormArgs& a, int* rc, cudaStream_t st) {
  constexpr int NV = VE > 1 ? 64 / (VE * static_cast<int>(sizeof(TX))) : 16;     // 64 bytes of a row
  const int nvec = a.cols / VE;
  if (!a.y || a.cols * sizeof(TX) < 512 || nvec > FWD_THREADS * NV) return false;
  if (VE > 1 && (a.cols * sizeof(TX) % 16 || a.ld * sizeof(TX) % 16)) return false;
  const int G = round_up((nvec + NV - 1) / NV, 32), P = ring_groups(FWD_THREADS, G);
  const int slot = slot_bytes(a.cols * static_cast<int>(sizeof(TX)), VE > 1), fixed = slot_bytes(8 * a.cols, true);
  const int stages = std::min(MAX_STAGES, (kRingBytes - fixed) / (P * slot));
  if (fixed > kRingBytes || stages < 2 || a.rows < 4ll * P * sm_count()) return false;
  int* status = status_ptr();
  auto kern = norm_ring_kernel<TX, TY, VE, NV, false>;
  if constexpr (VE > 1)
    if (nvec == G * NV) kern = norm_ring_kernel<TX, TY, VE, NV, true>;
  if (!status || cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
    *rc = MXQ_ERR_CUDA;
  else
    *rc = launch_pdl(kern, dim3(sm_count()), dim3(P * G), fixed + P * stages * slot, st, a, G, stages, status);
  return true;
}

template <typename TX, int OUT>
int norm_rows(const NormArgs& a, bool vec, cudaStream_t st) {
  constexpr int VE = sizeof(TX) == 2 && OUT != OUT_F32 ? 8 : 4;
  if constexpr (OUT < 0) {
    if (a.cols > kMaxRowElems) return launch_pdl(norm_long_kernel<TX, OUT>, dim3(a.rows), dim3(1024), 0, st, a);
    using TY = typename std::conditional<OUT == OUT_F32, float, __nv_bfloat16>::type;
    int rc;
    if (vec ? try_norm_ring<TX, TY, VE>(a, &rc, st) : try_norm_ring<TX, TY, 1>(a, &rc, st)) return rc;
    if (!vec) return dispatch_row<TX, OUT, 1>(a, st);
  }
  return dispatch_row<TX, OUT, VE>(a, st);
}

// CTAs (clusters of `slabs`) of a tile kernel that run at once, asked once per
// device and size.
template <typename K>
int resident(K kern, int slabs, int threads, int smem, std::atomic<int>& known) {
  int n = known.load(std::memory_order_relaxed);
  if (n) return n;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(slabs * 4 * sm_count());
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = slabs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) return 0;
  known.store(n, std::memory_order_relaxed);
  return n;
}

template <typename TX, int FMT, int ORIENT, bool CLUSTER, int S, int T>
int launch_tile(const NormArgs& a, cudaStream_t st) {
  static std::atomic<int> known[64][TILE_SLABS + 1];
  const int slabs = (a.cols + S - 1) / S, cluster = CLUSTER ? slabs : 1;
  const int smem = ((ORIENT & MXQ_COL) ? 34 : 2) * S * 4;
  auto kern = norm_tile_kernel<TX, FMT, ORIENT, CLUSTER, S, T>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
  const int n = resident(kern, cluster, T, smem, known[dev][cluster]);
  int* status = status_ptr();
  if (!n || !status) return MXQ_ERR_CUDA;
  const int64_t teams = std::min<int64_t>(a.rows / 32, CLUSTER ? n : std::max(1, n / slabs));
  if (CLUSTER)
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(teams * slabs)), dim3(T), smem, st, slabs, a, slabs, status);
  return launch_pdl(kern, dim3(static_cast<unsigned>(teams * slabs)), dim3(T), smem, st, a, slabs, status);
}

// Rows only: the row kernel.  With column blocks: a portable cluster (8 CTAs)
// holds 32 rows of up to 4096 columns in slabs of 512, or 8192 in slabs of
// 1024; longer rows get their statistics first, then slab by slab (x is read
// twice).
template <typename TX, int FMT, int ORIENT>
int norm_mx_tiles(const NormArgs& a, cudaStream_t st) {
  if constexpr (ORIENT != MXQ_ROW) {
    if (a.cols <= TILE_SLABS * 512) return launch_tile<TX, FMT, ORIENT, true, 512, 256>(a, st);
    if (a.cols <= TILE_SLABS * 1024) return launch_tile<TX, FMT, ORIENT, true, 1024, 512>(a, st);
  }
  NormArgs s = a;
  s.y = nullptr;
  if (const int rc = norm_rows<TX, OUT_BF16>(s, true, st)) return rc;
  return launch_tile<TX, FMT, ORIENT, false, 512, 256>(a, st);
}

template <typename TX, int FMT>
int norm_mx(const NormArgs& a, int orient, cudaStream_t st) {
  if (orient == MXQ_ROW) return a.cols <= kMaxRowElems ? norm_rows<TX, FMT>(a, true, st) : norm_mx_tiles<TX, FMT, MXQ_ROW>(a, st);
  return orient == MXQ_DUAL ? norm_mx_tiles<TX, FMT, MXQ_DUAL>(a, st) : norm_mx_tiles<TX, FMT, MXQ_COL>(a, st);
}

template <typename TX>
int norm_mx_fmt(const NormArgs& a, int fmt, int orient, cudaStream_t st) {
  if (fmt == MXQ_E4M3) return norm_mx<TX, MXQ_E4M3>(a, orient, st);
  if (fmt == MXQ_E5M2) return norm_mx<TX, MXQ_E5M2>(a, orient, st);
  return norm_mx<TX, MXQ_E2M1>(a, orient, st);
}

int check_norm(const void* x, int64_t rows, int64_t cols, int64_t ld, int x_type, const void* w, int w_type,
               const void* b, int b_type, const float* mean, const float* rstd) {
  if (!valid_type(x_type) || (w && !valid_type(w_type)) || (b && !valid_type(b_type))) return MXQ_ERR_BAD_ARG;
  if (rows < 0 || cols < 1 || ld < cols) return MXQ_ERR_BAD_SHAPE;
  if (rows > 0x7FFFFFF0ll || cols > 0x7FFFFFF0ll) return MXQ_ERR_BAD_SHAPE;
  if (rows && (!x || !mean || !rstd)) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(x, type_size(x_type)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4)) return MXQ_ERR_MISALIGNED;
  if ((w && !aligned_to(w, type_size(w_type))) || (b && !aligned_to(b, type_size(b_type)))) return MXQ_ERR_MISALIGNED;
  return MXQ_OK;
}

NormArgs norm_args(const void* x, int64_t rows, int64_t cols, int64_t ld, const void* w, int w_type, const void* b,
                   int b_type, float eps, float* mean, float* rstd) {
  NormArgs a{};
  a.x = x, a.ld = ld, a.rows = static_cast<int>(rows), a.cols = static_cast<int>(cols);
  a.w = w, a.b = b, a.w_f32 = w_type == MXQ_F32, a.b_f32 = b_type == MXQ_F32;
  a.eps = eps, a.mean = mean, a.rstd = rstd;
  return a;
}

// Backward: CTAs (parts of the column sums) that a launch may use.
int bwd_parts() { return 4 * sm_count(); }

template <typename TX, typename TD, int VE, int NV>
int launch_bwd(const BwdArgs& a, int G, int& parts, cudaStream_t st) {
  const int P = std::max(1, 512 / G);
  const int threads = P * G;
  const size_t smem = P > 1 ? static_cast<size_t>(2) * VE * NV * G * sizeof(float) : 0;
  const int64_t groups = (a.rows + P - 1) / P;
  const int most = std::min(bwd_parts(), std::max(1, 2048 / threads) * sm_count());
  parts = static_cast<int>(std::min<int64_t>(most, groups));
  return launch_pdl(norm_bwd_kernel<TX, TD, VE, NV, 1>, dim3(parts), dim3(threads), smem, st, a, G);
}

// Rings while a group's slots fit and every group gets two rows or more.
template <typename TX, typename TD, int VE, int NV>
bool launch_bwd_ring(const BwdArgs& a, int G, int P, int* rc, int& parts, cudaStream_t st) {
  const int slot = slot_bytes(a.cols * static_cast<int>(sizeof(TX)), VE > 1) +
                   slot_bytes(a.cols * static_cast<int>(sizeof(TD)), VE > 1);
  const int fixed = VE * NV <= BWD_KEEP ? 0 : slot_bytes((a.w_f32 ? 4 : 2) * a.cols, true);
  const int stages = std::min(MAX_STAGES, (kRingBytes - fixed) / (P * slot));
  if (stages < 2) return false;
  int* status = status_ptr();
  auto kern = norm_bwd_ring_kernel<TX, TD, VE, NV, false>;
  if constexpr (VE > 1)
    if (a.cols / VE == G * NV) kern = norm_bwd_ring_kernel<TX, TD, VE, NV, true>;
  const int smem = std::max(fixed + P * stages * slot, P > 1 ? 2 * VE * NV * G * 4 : 0);
  parts = sm_count();
  if (!status || cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
    *rc = MXQ_ERR_CUDA;
  else
    *rc = launch_pdl(kern, dim3(parts), dim3(P * G), smem, st, a, G, stages, status);
  return true;
}

template <typename TX, typename TD, int VE>
bool try_bwd_ring(const BwdArgs& a, int* rc, int& parts, cudaStream_t st) {
  constexpr int N1 = BWD_KEEP / VE, N2 = 2 * BWD_KEEP / VE;
  const int nvec = a.cols / VE;
  if (VE > 1 && (a.cols * sizeof(TX) % 16 || a.cols * sizeof(TD) % 16 || a.ld_x * sizeof(TX) % 16 ||
                 a.ld_dy * sizeof(TD) % 16))
    return false;
  const int nv = nvec <= BWD_THREADS * N1 ? N1 : N2;
  if (nvec > BWD_THREADS * N2) return false;
  const int G = round_up((nvec + nv - 1) / nv, 32), P = ring_groups(BWD_THREADS, G);
  if (a.rows < 2ll * P * sm_count()) return false;
  return nv == N1 ? launch_bwd_ring<TX, TD, VE, N1>(a, G, P, rc, parts, st)
                  : launch_bwd_ring<TX, TD, VE, N2>(a, G, P, rc, parts, st);
}

template <typename TX, typename TD, int VE>
int dispatch_bwd(const BwdArgs& a, int& parts, cudaStream_t st) {
  const int nvec = a.cols / VE;
  constexpr int N1 = VE == 1 ? 4 : 1;
  constexpr int N2 = 16 / VE;
  if (nvec <= N1 * 1024) return launch_bwd<TX, TD, VE, N1>(a, round_up((nvec + N1 - 1) / N1, 32), parts, st);
  return launch_bwd<TX, TD, VE, N2>(a, round_up((nvec + N2 - 1) / N2, 32), parts, st);
}

template <typename TX, typename TD>
int norm_bwd(const BwdArgs& a, bool vec, int& parts, cudaStream_t st) {
  if (a.cols <= kMaxBwdElems) {
    constexpr int VE = sizeof(TX) == 2 && sizeof(TD) == 2 ? 8 : 4;
    int rc;
    if (vec ? try_bwd_ring<TX, TD, VE>(a, &rc, parts, st) : try_bwd_ring<TX, TD, 1>(a, &rc, parts, st)) return rc;
    return vec ? dispatch_bwd<TX, TD, VE>(a, parts, st) : dispatch_bwd<TX, TD, 1>(a, parts, st);
  }
  const int rc = launch_pdl(norm_bwd_long_rows_kernel<TX, TD>, dim3(a.rows), dim3(1024), 0, st, a);
  if (rc) return rc;
  const int strips = (a.cols + 255) / 256;
  parts = std::max(1, std::min(std::min(a.rows, bwd_parts()), 8 * sm_count() / strips));
  return launch_pdl(norm_bwd_long_cols_kernel<TX, TD>, dim3(strips, parts), dim3(256), 0, st, a);
}

}  // namespace
}  // namespace mxq

using namespace mxq;
using namespace mxq_host;

extern "C" int mxq_layer_norm(const void* x, int64_t rows, int64_t cols, int64_t ld, int x_type, const void* w,
                              int w_type, const void* b, int b_type, float eps, int y_type, void* y, float* mean,
                              float* rstd, void* stream) {
  if (!valid_type(y_type)) return MXQ_ERR_BAD_ARG;
  const int rc = check_norm(x, rows, cols, ld, x_type, w, w_type, b, b_type, mean, rstd);
  if (rc) return rc;
  if (rows && !y) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(y, type_size(y_type))) return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  if (!rows) return MXQ_OK;
  NormArgs a = norm_args(x, rows, cols, ld, w, w_type, b, b_type, eps, mean, rstd);
  a.y = y;
  const int ve = x_type == MXQ_BF16 && y_type == MXQ_BF16 ? 8 : 4;
  const bool vec = cols % ve == 0 && ld % ve == 0 && aligned16(x) && aligned16(y) && aligned16(w) && aligned16(b);
  const auto st = static_cast<cudaStream_t>(stream);
  if (x_type == MXQ_BF16)
    return y_type == MXQ_BF16 ? norm_rows<__nv_bfloat16, OUT_BF16>(a, vec, st) : norm_rows<__nv_bfloat16, OUT_F32>(a, vec, st);
  return y_type == MXQ_BF16 ? norm_rows<float, OUT_BF16>(a, vec, st) : norm_rows<float, OUT_F32>(a, vec, st);
}

extern "C" int mxq_layer_norm_mx(const void* x, int64_t rows, int64_t cols, int64_t ld, int x_type, const void* w,
                                 int w_type, const void* b, int b_type, float eps, int fmt, int orient,
                                 int scale_mode, int sf_layout, void* q_row, uint8_t* s_row, void* q_col,
                                 uint8_t* s_col, float* mean, float* rstd, void* stream) {
  if (fmt != MXQ_E4M3 && fmt != MXQ_E5M2 && fmt != MXQ_E2M1) return MXQ_ERR_BAD_ARG;
  if (orient != MXQ_ROW && orient != MXQ_COL && orient != MXQ_DUAL) return MXQ_ERR_BAD_ARG;
  if (scale_mode != MXQ_SCALE_FLOOR_OCP && scale_mode != MXQ_SCALE_CEIL) return MXQ_ERR_BAD_ARG;
  if (sf_layout != MXQ_SF_CANONICAL && sf_layout != MXQ_SF_MMA) return MXQ_ERR_BAD_ARG;
  if ((orient & MXQ_ROW) && (!q_row || !s_row)) return MXQ_ERR_BAD_ARG;
  if ((orient & MXQ_COL) && (!q_col || !s_col)) return MXQ_ERR_BAD_ARG;
  const int rc = check_norm(x, rows, cols, ld, x_type, w, w_type, b, b_type, mean, rstd);
  if (rc) return rc;
  const int unit = sf_layout == MXQ_SF_MMA ? 128 : 32;
  if (rows < 1 || rows % unit || cols % unit) return MXQ_ERR_BAD_SHAPE;
  if (!aligned16(x) || ld % (16 / type_size(x_type)) || !aligned16(w) || !aligned16(b)) return MXQ_ERR_MISALIGNED;
  if ((orient & MXQ_ROW) && !aligned16(q_row)) return MXQ_ERR_MISALIGNED;
  if ((orient & MXQ_COL) && !aligned16(q_col)) return MXQ_ERR_MISALIGNED;
  if (sf_layout == MXQ_SF_MMA && (((orient & MXQ_ROW) && !aligned16(s_row)) || ((orient & MXQ_COL) && !aligned16(s_col))))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  NormArgs a = norm_args(x, rows, cols, ld, w, w_type, b, b_type, eps, mean, rstd);
  a.q_row = static_cast<uint8_t*>(q_row), a.s_row = s_row;
  a.q_col = static_cast<uint8_t*>(q_col), a.s_col = s_col;
  a.ceil_mode = scale_mode == MXQ_SCALE_CEIL;
  a.mma = sf_layout == MXQ_SF_MMA;
  a.pack_row = cols % 128 == 0 && aligned_to(s_row, 4);
  a.pack_col = rows % 128 == 0 && aligned_to(s_col, 4);
  a.wide_col = aligned_to(q_col, 32);
  const auto st = static_cast<cudaStream_t>(stream);
  return x_type == MXQ_BF16 ? norm_mx_fmt<__nv_bfloat16>(a, fmt, orient, st) : norm_mx_fmt<float>(a, fmt, orient, st);
}

extern "C" int mxq_layer_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return MXQ_ERR_BAD_ARG;
  if (rows < 0 || cols < 1) return MXQ_ERR_BAD_SHAPE;
  const size_t parts = static_cast<size_t>(std::min<int64_t>(rows, bwd_parts()));
  *bytes = parts * 2 * static_cast<size_t>(cols) * sizeof(float) +
           (cols > kMaxBwdElems ? static_cast<size_t>(rows) * 2 * sizeof(float) : 0);
  return MXQ_OK;
}

extern "C" int mxq_layer_norm_backward(const void* dy, int64_t ld_dy, int dy_type, const void* x, int64_t ld_x,
                                       int x_type, int64_t rows, int64_t cols, const float* mean, const float* rstd,
                                       const void* w, int w_type, void* dx, float* dw, float* db, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (!valid_type(dy_type)) return MXQ_ERR_BAD_ARG;
  const int rc = check_norm(x, rows, cols, ld_x, x_type, w, w_type, nullptr, 0, mean, rstd);
  if (rc) return rc;
  if (ld_dy < cols) return MXQ_ERR_BAD_SHAPE;
  if (rows && (!dy || !dx)) return MXQ_ERR_BAD_ARG;
  const bool sums = dw || db;
  size_t need = 0;
  mxq_layer_norm_backward_workspace_size(rows, cols, &need);
  if (rows && (sums || cols > kMaxBwdElems) && (!workspace || workspace_bytes < need)) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(dy, type_size(dy_type)) || !aligned_to(dx, type_size(x_type)) || !aligned16(workspace) ||
      !aligned_to(dw, 4) || !aligned_to(db, 4))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  const auto st = static_cast<cudaStream_t>(stream);
  if (!rows) {
    if (dw && cudaMemsetAsync(dw, 0, cols * sizeof(float), st) != cudaSuccess) return MXQ_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, cols * sizeof(float), st) != cudaSuccess) return MXQ_ERR_CUDA;
    return MXQ_OK;
  }
  BwdArgs a{};
  a.dy = dy, a.ld_dy = ld_dy, a.x = x, a.ld_x = ld_x;
  a.rows = static_cast<int>(rows), a.cols = static_cast<int>(cols);
  a.mean = mean, a.rstd = rstd, a.w = w, a.w_f32 = w_type == MXQ_F32, a.dx = dx;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.coef = static_cast<float*>(workspace) + std::min<int64_t>(rows, bwd_parts()) * 2 * cols;
  const int ve = x_type == MXQ_BF16 && dy_type == MXQ_BF16 ? 8 : 4;
  const bool vec = cols % ve == 0 && ld_x % ve == 0 && ld_dy % ve == 0 && aligned16(x) && aligned16(dy) &&
                   aligned16(dx) && aligned16(w);
  int parts = 0, rc2;
  if (x_type == MXQ_BF16)
    rc2 = dy_type == MXQ_BF16 ? norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, vec, parts, st)
                              : norm_bwd<__nv_bfloat16, float>(a, vec, parts, st);
  else
    rc2 = dy_type == MXQ_BF16 ? norm_bwd<float, __nv_bfloat16>(a, vec, parts, st) : norm_bwd<float, float>(a, vec, parts, st);
  if (rc2 || !sums) return rc2;
  const int grid = static_cast<int>((2 * cols + 31) / 32);
  return launch_pdl(norm_bwd_sum_kernel, dim3(grid), dim3(256), 0, st, static_cast<const float*>(workspace), parts,
                    a.cols, dw, db);
}
