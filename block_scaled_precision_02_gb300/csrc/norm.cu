// Layer norm over the rows of a matrix, y = (x - mean) * rstd * w + b.
#include "norm.cuh"

namespace mxq {
namespace {

constexpr int FWD_THREADS = 640;

// ---------------------------------------------------------------- many rows
// Groups of threads in a persistent CTA, each with a ring of whole rows in
// shared memory that one of its threads fills by bulk copies ahead of use.
// A row moves from its slot to registers; the barrier of the group's
// reduction says that all have read it, and the slot takes a later row of the
// group.  Loads stay in flight through reductions and stores, which registers
// alone do not allow (the row kernel's CTAs load, reduce and store in turn).
// The elements' arithmetic runs on packed pairs.
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

// W16: bf16 weight and bias stay bf16 in shared memory, which halves their
// reads: as float32 those weigh more than the row's own traffic (4096 x 14336
// bf16: 48.2 us against 45.4; 4096 x 20000: 91 against 54, because a float32
// copy leaves no room for two slots).
template <typename TX, typename TY, int VE, int NV, bool FULL, bool W16>
__global__ void __launch_bounds__(FWD_THREADS, 1) norm_ring_kernel(const NormArgs a, int G, int stages, int* status) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 part[2][FWD_THREADS / 32];
  __shared__ __align__(8) uint64_t full[MAX_GROUPS][MAX_STAGES];
  const int lane = threadIdx.x & 31;
  const int P = blockDim.x / G, g = threadIdx.x / G, t = threadIdx.x - g * G;
  const int gw = t >> 5, wpg = G >> 5, first = first_vec<NV>(gw, lane);
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
  uint8_t* slots = ring + slot_bytes((W16 ? 4 : 8) * a.cols, true) + static_cast<size_t>(g) * stages * sb;
  const int64_t gi = static_cast<int64_t>(blockIdx.x) * P + g, step = static_cast<int64_t>(gridDim.x) * P;
  const float inv_c = 1.f / static_cast<float>(a.cols);
  const int n_mine = warp_count<VE, NV>(a.cols, gw), n_lane = lane < wpg ? warp_count<VE, NV>(a.cols, lane) : 0;
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
  uint32_t* const w16 = reinterpret_cast<uint32_t*>(ring);     // W16: weight [cols], bias [cols]
  if constexpr (W16) {
    for (int i = threadIdx.x; i < a.cols / 2; i += blockDim.x) {
      w16[i] = a.w ? static_cast<const uint32_t*>(a.w)[i] : 0x3F803F80u;      // ones
      w16[a.cols / 2 + i] = a.b ? static_cast<const uint32_t*>(a.b)[i] : 0u;
    }
  } else {
    stage_affine<VE>(a, ws);
  }
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
        if (FULL || first + 32 * k < nvec) v[k].load(from + (first + 32 * k) * VE);
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
      s[k] = FULL || first + 32 * k < nvec ? vec_sq_dev(f, near) : 0.f;
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
      const int at = (first + 32 * k) * VE;
      if (!FULL && at >= a.cols) continue;
      float f[VE], o[VE];
      wide(k, f);
      if constexpr (VE == 1) {
        const float2 wb = *reinterpret_cast<const float2*>(ws + 2 * at);
        o[0] = norm_value(f[0], mean, rstd, wb.x, wb.y);
      } else {
        float w[VE], b[VE];
        if constexpr (W16) {
          Vec<__nv_bfloat16, VE> wv, bv;
          wv.load(reinterpret_cast<const __nv_bfloat16*>(w16) + at);
          bv.load(reinterpret_cast<const __nv_bfloat16*>(w16) + a.cols + at);
#pragma unroll
          for (int j = 0; j < VE; ++j) w[j] = wv.get(j), b[j] = bv.get(j);
        } else {
          staged<VE>(ws, at, a.cols, w);
          staged<VE>(ws + a.cols, at, a.cols, b);
        }
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

// ---------------------------------------------------------------- host
// Rings for rows of 512 bytes and more (up to what two slots hold) when every
// group gets four or more: below that a ring has nothing to run ahead on, and
// the row kernel's shorter prologue wins.  A thread holds 64 bytes of a row,
// 640 threads a CTA: with 1024 the registers (64) force the loads into turns
// (4096 x 14336 bf16: 57 us, 45 with 640, 46 with 512).  False: not taken.
template <typename TX, typename TY, int VE>
bool try_norm_ring(const NormArgs& a, int* rc, cudaStream_t st) {
  constexpr int NV = VE > 1 ? 64 / (VE * static_cast<int>(sizeof(TX))) : 16;     // 64 bytes of a row
  const int nvec = a.cols / VE;
  if (!a.y || a.cols * sizeof(TX) < 512 || nvec > FWD_THREADS * NV) return false;
  if (VE > 1 && (a.cols * sizeof(TX) % 16 || a.ld * sizeof(TX) % 16)) return false;
  const int G = round_up((nvec + NV - 1) / NV, 32), P = ring_groups(FWD_THREADS, G);
  const bool w16 = VE == 8 && !(a.w && a.w_f32) && !(a.b && a.b_f32);
  const int slot = slot_bytes(a.cols * static_cast<int>(sizeof(TX)), VE > 1);
  const int fixed = slot_bytes((w16 ? 4 : 8) * a.cols, true);
  const int stages = std::min(MAX_STAGES, (kRingBytes - fixed) / (P * slot));
  if (fixed > kRingBytes || stages < 2 || a.rows < 4ll * P * sm_count()) return false;
  int* status = status_ptr();
  auto kern = norm_ring_kernel<TX, TY, VE, NV, false, false>;
  if constexpr (VE > 1)
    if (nvec == G * NV) kern = norm_ring_kernel<TX, TY, VE, NV, true, false>;
  if constexpr (VE == 8)
    if (w16) kern = nvec == G * NV ? norm_ring_kernel<TX, TY, VE, NV, true, true> : norm_ring_kernel<TX, TY, VE, NV, false, true>;
  if (!status || cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
    *rc = MXQ_ERR_CUDA;
  else
    *rc = launch_pdl(kern, dim3(sm_count()), dim3(P * G), fixed + P * stages * slot, st, a, G, stages, status);
  return true;
}

template <typename TX, int OUT>
int norm_rows(const NormArgs& a, bool vec, cudaStream_t st) {
  constexpr int VE = sizeof(TX) == 2 && OUT != OUT_F32 ? 8 : 4;
  if (a.cols > kMaxRowElems) return launch_pdl(norm_long_kernel<TX, OUT>, dim3(a.rows), dim3(1024), 0, st, a);
  using TY = typename std::conditional<OUT == OUT_F32, float, __nv_bfloat16>::type;
  int rc;
  if (vec ? try_norm_ring<TX, TY, VE>(a, &rc, st) : try_norm_ring<TX, TY, 1>(a, &rc, st)) return rc;
  return vec ? dispatch_row<TX, OUT, VE>(a, st) : dispatch_row<TX, OUT, 1>(a, st);
}

}  // namespace

int norm_stats(const NormArgs& a, int x_type, cudaStream_t st) {
  NormArgs s = a;
  s.y = nullptr;
  return x_type == MXQ_BF16 ? norm_rows<__nv_bfloat16, OUT_BF16>(s, true, st) : norm_rows<float, OUT_BF16>(s, true, st);
}

}  // namespace mxq

using namespace mxq;

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

