// Device helpers of the row-wise training-step kernels (norm.cu, loss.cu,
// gradnorm.cu): vectors of a few consecutive bf16 or float32 elements, warp
// sums, the merge of partial means and squared deviations, and the MX
// encoding of a 32-block of float32 values.
#pragma once

#include "common.cuh"

namespace mxq {

// The longest row.  Kernels count a row's elements in int and step past its
// end, by 4096 at most, before they compare.
constexpr int64_t kMaxCols = 0x7FFF0000;

// VE consecutive elements of T in registers, as loaded (VE * sizeof(T) is 2,
// 4, 8 or 16 bytes and the address is aligned to it); get() widens one.
template <typename T, int VE>
struct Vec {
  static constexpr int BYTES = VE * static_cast<int>(sizeof(T));
  static constexpr int W = BYTES >= 4 ? BYTES / 4 : 1;
  uint32_t w[W];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (BYTES == 16) {
      const uint4 t = *reinterpret_cast<const uint4*>(p);
      w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
    } else if constexpr (BYTES == 8) {
      const uint2 t = *reinterpret_cast<const uint2*>(p);
      w[0] = t.x, w[1] = t.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void fill(uint32_t word) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = word;
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else return (j & 1) ? bf16hi(w[j >> 1]) : bf16lo(w[j >> 1]);
  }
};

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Store VE consecutive elements, rounded to T (nearest even); the address is
// aligned to VE * sizeof(T) bytes (32 bytes go as two 16-byte stores).
template <typename T, int VE>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VE]) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (VE == 1) *p = v[0];
    else {
#pragma unroll
      for (int i = 0; i < VE; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  } else {
    if constexpr (VE == 1) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(bf16x2_rn(v[0], 0.f));
    else if constexpr (VE == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]));
    else
      *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]),
                                                bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
  }
}

// VE consecutive weights (bf16 or float32 by a uniform run-time flag).
template <int VE>
__device__ __forceinline__ void load_param(const void* base, int is_f32, int64_t at, float (&out)[VE]) {
  if (is_f32) {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (VE == 1) out[0] = *p;
    else {
#pragma unroll
      for (int i = 0; i < VE; i += 4) {
        const float4 t = *reinterpret_cast<const float4*>(p + i);
        out[i] = t.x, out[i + 1] = t.y, out[i + 2] = t.z, out[i + 3] = t.w;
      }
    }
  } else {
    Vec<__nv_bfloat16, VE> t;
    t.load(static_cast<const __nv_bfloat16*>(base) + at);
#pragma unroll
    for (int i = 0; i < VE; ++i) out[i] = t.get(i);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum of N registers as a balanced tree (the rounding error grows with log N).
template <int N>
__device__ __forceinline__ float tree_sum(const float (&v)[N]) {
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = v[i];
#pragma unroll
  for (int n = N; n > 1; n = (n + 1) / 2)
#pragma unroll
    for (int i = 0; i < n / 2; ++i) t[i] = t[i] + t[n - 1 - i];
  return t[0];
}

// Pairs of float32 and the packed operations on them: each half rounds to
// nearest exactly as the scalar operation would.
__device__ __forceinline__ float2 pair(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ float2 splat(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __fadd2_rn(a, make_float2(-b.x, -b.y)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ void halves(float2 p, float& x, float& y) { x = p.x, y = p.y; }

// One cluster barrier, in two halves: what a thread did before the arrive is
// visible to every thread of the cluster after the wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Write two floats into the shared memory of the cluster's CTA `rank`, at the
// place of this CTA's address `addr`.
__device__ __forceinline__ void st_cluster_f2(uint32_t addr, uint32_t rank, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_map(addr, rank)), "f"(a), "f"(b) : "memory");
}

// The same as an asynchronous store that counts its 8 bytes on the target
// CTA's mbarrier at `bar`: no fence, so the sender's earlier global stores
// need not have landed.
__device__ __forceinline__ void st_async_f2(uint32_t addr, uint32_t bar, uint32_t rank, float a, float b) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                   cluster_map(addr, rank)),
               "f"(a), "f"(b), "r"(cluster_map(bar, rank))
               : "memory");
}

// Bounded wait for phases that take microseconds: the thread sleeps in the
// barrier unit instead of polling.  PEERS: other CTAs of the cluster complete
// the phase by stores of theirs, so the acquire is at cluster scope.
template <bool PEERS = false>
__device__ __forceinline__ bool mbar_wait_sleep(uint32_t bar, uint32_t parity, int* status) {
  const auto done = [&](uint32_t hint_ns) {
    return PEERS ? mbar_try_wait_cl_sleep(bar, parity, hint_ns) : mbar_try_wait_sleep(bar, parity, hint_ns);
  };
  if (done(2000u)) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (!done(20000u))
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_timeout(status);
      return false;
    }
  return true;
}

// After a wait for peers' stores has given up, and the cluster's last barrier:
// what was sent to this CTA's shared memory lands within microseconds, and
// the CTA stays for a hundred.
__device__ __forceinline__ void linger() {
  const unsigned long long t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 100000ull) __nanosleep(1000);
}

// Scale byte of an MX block whose largest magnitude has the bits `ab`, and the
// multiplier 2^-e of its elements; a block that holds NaN or an infinity gets
// 0xFF (and zero codes: `bad` of mx_codes).
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t ab, int ceil_mode, float& mult) {
  const bool bad = ab >= 0x7F800000u;
  const int e = scale_exp<FMT>(bad ? 0u : ab, ceil_mode);
  mult = exp2_neg(e);
  return bad ? 0xFFu : static_cast<uint32_t>(e + 127);
}

// N values of a block to N FP8 bytes or N/2 E2M1 bytes, in element order.
template <int FMT, int N>
constexpr int code_words() { return FMT == MXQ_E2M1 ? (N + 7) / 8 : N / 4; }

template <int FMT, int N>
__device__ __forceinline__ void mx_codes(const float (&y)[N], float mult, bool bad,
                                         uint32_t (&out)[code_words<FMT, N>()]) {
  const float2 mm = splat(mult);
  float v[N];
#pragma unroll
  for (int i = 0; i < N; i += 2) halves(mul2(pair(y[i], y[i + 1]), mm), v[i], v[i + 1]);
  if constexpr (FMT == MXQ_E2M1) {
#pragma unroll
    for (int k = 0; k < code_words<FMT, N>(); ++k) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 8 * k; i < N && i < 8 * k + 8; i += 2) w |= cvt_e2m1x2(v[i], v[i + 1]) << (4 * (i - 8 * k));
      out[k] = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      out[i / 4] = cvt_fp8x4<FMT>(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
  if (bad) {                                 // rare: a branch costs less than a select per word
#pragma unroll
    for (int k = 0; k < code_words<FMT, N>(); ++k) out[k] = 0u;
  }
}

// Byte of the scale of (row, k-block) in either layout (kb blocks per row).
__device__ __forceinline__ int64_t scale_at(int64_t row, int64_t k, int64_t kb, int mma) {
  if (!mma) return row * kb + k;
  return ((row >> 7) * (kb >> 2) + (k >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (k & 3);
}

// ---------------------------------------------------------------- host: checks of arguments
inline bool valid_type(int t) { return t == MXQ_BF16 || t == MXQ_F32; }
inline int type_size(int t) { return t == MXQ_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace mxq
