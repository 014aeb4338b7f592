// Dropout from a counter-based generator, with the residual stream's sum:
//   y_i = residual_i + [u_i >= t] x_i / (1 - p),   t = round(p 2^32)
// where u_i is word i & 3 of Philox-4x32-10(key = seed, counter = offset + (i >> 2)),
// i = r cols + c.  The mask is a function of i, so the backward pass computes
// it again: the same call on dy.
//
// One generator call serves four elements, 20 wide products and 20 three-input
// exclusive ors: between HBM (4 to 12 bytes an element) and the integer units.
// 8192 x 14336 bf16: with residual 108 us (97 % of the copy rate), without 95 (74 %).
#include <algorithm>
#include <cmath>

#include "rowops.cuh"

namespace mxq {
namespace {

constexpr int TPB = 256;

struct DropArgs {
  const void* x;
  const void* res;
  void* y;
  int64_t rows, cols, ld, ld_res;
  uint64_t offset;
  const int64_t* offset_dev;              // or nullptr
  uint32_t below;                         // draws below it drop the element
  float scale;
  uint32_t key[10][2];                    // the rounds' keys
};

// Philox-4x32-10 of (counter, 0, 0): the products as one wide multiplication
// each, the keys from the kernel's parameters.
__device__ __forceinline__ u32x4 draw(const DropArgs& a, uint64_t counter) {
  uint32_t x = static_cast<uint32_t>(counter), y = static_cast<uint32_t>(counter >> 32), z = 0u, w = 0u;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * x, q = static_cast<uint64_t>(0xCD9E8D57u) * z;
    x = static_cast<uint32_t>(q >> 32) ^ y ^ a.key[r][0];
    z = static_cast<uint32_t>(p >> 32) ^ w ^ a.key[r][1];
    y = static_cast<uint32_t>(q);
    w = static_cast<uint32_t>(p);
  }
  return u32x4{x, y, z, w};
}

// A matrix without gaps: a thread takes V vectors of 8 elements, TPB vectors
// apart.  What does not fill a vector at the end goes singly.
template <typename T, bool RES, int V>
__global__ void __launch_bounds__(TPB) dropout_kernel(const __grid_constant__ DropArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const uint64_t base = a.offset + (a.offset_dev ? static_cast<uint64_t>(*a.offset_dev) : 0u);
  const int64_t n = a.rows * a.cols;
  const T* const x = static_cast<const T*>(a.x);
  const T* const res = static_cast<const T*>(a.res);
  T* const y = static_cast<T*>(a.y);
  constexpr int N = 16 / static_cast<int>(sizeof(T)), W = 8 / N;         // elements of a word, words of a vector
  const int64_t step = static_cast<int64_t>(gridDim.x) * TPB * 8 * V;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * TPB * V + threadIdx.x) * 8; i0 < n; i0 += step) {
    Vec<T, N> v[V][W], r[V][W];
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int h = 0; h < W; ++h)
        if (i0 + k * TPB * 8 + 8 <= n) {
          v[k][h].load(x + i0 + k * TPB * 8 + h * N);
          if constexpr (RES) r[k][h].load(res + i0 + k * TPB * 8 + h * N);
        }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t i = i0 + k * TPB * 8;
      if (i + 8 <= n) {
        float o[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 u = draw(a, base + static_cast<uint64_t>(i >> 2) + h);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = 4 * h + e;
            const float kept = v[k][at / N].get(at % N) * a.scale;
            o[at] = w[e] >= a.below ? kept : 0.f;
            if constexpr (RES) o[at] += r[k][at / N].get(at % N);
          }
        }
        store_vec<T, 8>(y + i, o);
      } else {
        for (int64_t j = i; j < n; j += 4) {
          const u32x4 u = draw(a, base + static_cast<uint64_t>(j >> 2));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < n) {
              float o[1], q[1];
              load_elems<T, 1>(x + j + e, o);
              o[0] = w[e] >= a.below ? o[0] * a.scale : 0.f;
              if constexpr (RES) {
                load_elems<T, 1>(res + j + e, q);
                o[0] += q[0];
              }
              store_vec<T, 1>(y + j + e, o);
            }
        }
      }
    }
  }
}

// Any strides and sizes: thread i takes the 4 elements of one counter.
template <typename T, bool RES>
__global__ void __launch_bounds__(TPB) dropout_any_kernel(const __grid_constant__ DropArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const uint64_t base = a.offset + (a.offset_dev ? static_cast<uint64_t>(*a.offset_dev) : 0u);
  const int64_t n = a.rows * a.cols;
  const T* const x = static_cast<const T*>(a.x);
  const T* const res = static_cast<const T*>(a.res);
  T* const y = static_cast<T*>(a.y);
  const int64_t step = static_cast<int64_t>(gridDim.x) * TPB * 4;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * TPB + threadIdx.x) * 4; i < n; i += step) {
    const u32x4 u = draw(a, base + static_cast<uint64_t>(i >> 2));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    int64_t row = i / a.cols, col = i - row * a.cols;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < n) {
        float v[1];
        load_elems<T, 1>(x + row * a.ld + col, v);
        v[0] = w[k] >= a.below ? v[0] * a.scale : 0.f;
        if constexpr (RES) {
          float r[1];
          load_elems<T, 1>(res + row * a.ld_res + col, r);
          v[0] += r[0];
        }
        store_vec<T, 1>(y + i + k, v);
      }
      if (++col == a.cols) col = 0, ++row;
    }
  }
}

template <typename T, bool RES, int V>
int run_flat(const DropArgs& a, int64_t n, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((n + 8 * V * TPB - 1) / (8 * V * TPB), 0x7FFFFFFF)));
  return mxq_host::launch_pdl(dropout_kernel<T, RES, V>, grid, dim3(TPB), 0, st, a);
}

// bf16 tensors that fill the GPU several times take four vectors to a thread
// (8192 x 14336 with residual: 118 us with one, 108 with four; without 109 and
// 95); with fewer elements (1531 x 2049: 4.3 and 5.1 us) or float32 (8192 x
// 7167: 66 and 69) one is better.
constexpr int64_t LONG_ELEMS = 1 << 24;

template <typename T, bool RES>
int run(const DropArgs& a, cudaStream_t st) {
  const int64_t n = a.rows * a.cols;
  const bool flat = (a.rows == 1 || (a.ld == a.cols && (!RES || a.ld_res == a.cols))) && mxq_host::aligned16(a.x) &&
                    mxq_host::aligned16(a.res) && mxq_host::aligned16(a.y);
  if (!flat) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((n + 4 * TPB - 1) / (4 * TPB), 0x7FFFFFFF)));
    return mxq_host::launch_pdl(dropout_any_kernel<T, RES>, grid, dim3(TPB), 0, st, a);
  }
  if constexpr (sizeof(T) == 2)
    if (n >= LONG_ELEMS) return run_flat<T, RES, 4>(a, n, st);
  return run_flat<T, RES, 1>(a, n, st);
}

}  // namespace
}  // namespace mxq

using namespace mxq;
using namespace mxq_host;

extern "C" int mxq_dropout(const void* x, int64_t rows, int64_t cols, int64_t ld, int type, const void* residual,
                           int64_t ld_residual, double p, uint64_t seed, uint64_t offset, const int64_t* offset_dev,
                           void* y, void* stream) {
  if (!valid_type(type) || !(p >= 0.0 && p < 1.0)) return MXQ_ERR_BAD_ARG;
  if (rows < 0 || rows > kMaxCols || cols < 1 || cols > kMaxCols || ld < cols || (residual && ld_residual < cols))
    return MXQ_ERR_BAD_SHAPE;
  if (!rows) return MXQ_OK;
  if (!x || !y) return MXQ_ERR_BAD_ARG;
  const int s = type_size(type);
  if (!aligned_to(x, s) || !aligned_to(residual, s) || !aligned_to(y, s) || !aligned_to(offset_dev, 8)) return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  // p < 1 can round to 2^32: the last draw is then still kept
  const double t = std::nearbyint(p * 4294967296.0);
  DropArgs a{x, residual, y, rows, cols, ld, ld_residual, offset, offset_dev,
             t >= 4294967295.0 ? 0xFFFFFFFFu : static_cast<uint32_t>(t), static_cast<float>(1.0 / (1.0 - p)), {}};
  for (uint32_t r = 0; r < 10; ++r) {
    a.key[r][0] = static_cast<uint32_t>(seed) + r * 0x9E3779B9u;
    a.key[r][1] = static_cast<uint32_t>(seed >> 32) + r * 0xBB67AE85u;
  }
  const auto st = static_cast<cudaStream_t>(stream);
  if (type == MXQ_F32) return residual ? run<float, true>(a, st) : run<float, false>(a, st);
  return residual ? run<__nv_bfloat16, true>(a, st) : run<__nv_bfloat16, false>(a, st);
}
