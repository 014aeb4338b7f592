// Dropout from a counter-based generator, with the residual stream's sum:
//   y_i = residual_i + [u_i >= t] x_i / (1 - p),   t = round(p 2^32)
// where u_i is word i & 3 of Philox-4x32-10(key = seed, counter = offset + (i >> 2)),
// i = r cols + c.  The mask is a function of i, so the backward pass computes
// it again: the same call on dy.
//
// One generator call serves four elements, 20 wide products and 20 three-input
// exclusive ors: between HBM (4 to 12 bytes an element) and the integer units.
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
  uint64_t seed, offset;
  const int64_t* offset_dev;              // or nullptr
  uint32_t below;                         // draws below it drop the element
  float scale;
};

__device__ __forceinline__ u32x4 draw(const DropArgs& a, uint64_t counter) {
  return philox4x32_10(u32x4{static_cast<uint32_t>(counter), static_cast<uint32_t>(counter >> 32), 0u, 0u},
                       static_cast<uint32_t>(a.seed), static_cast<uint32_t>(a.seed >> 32));
}

// Whole vectors of a matrix without gaps: thread i takes the 8 elements from 8 i.
template <typename T, bool RES>
__global__ void __launch_bounds__(TPB) dropout_kernel(const DropArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const uint64_t base = a.offset + (a.offset_dev ? static_cast<uint64_t>(*a.offset_dev) : 0u);
  const int64_t n = a.rows * a.cols;
  const T* const x = static_cast<const T*>(a.x);
  const T* const res = static_cast<const T*>(a.res);
  T* const y = static_cast<T*>(a.y);
  const int64_t step = static_cast<int64_t>(gridDim.x) * TPB * 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * TPB + threadIdx.x) * 8; i < n; i += step) {
    float v[8], r[8];
    load_elems<T, 8>(x + i, v);
    if constexpr (RES) load_elems<T, 8>(res + i, r);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 u = draw(a, base + static_cast<uint64_t>(i >> 2) + h);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float kept = v[4 * h + k] * a.scale;
        float o = w[k] >= a.below ? kept : 0.f;
        if constexpr (RES) o += r[4 * h + k];
        v[4 * h + k] = o;
      }
    }
    store_vec<T, 8>(y + i, v);
  }
}

// Any strides and sizes: thread i takes the 4 elements of one counter.
template <typename T, bool RES>
__global__ void __launch_bounds__(TPB) dropout_any_kernel(const DropArgs a) {
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

template <typename T, bool RES>
int run(const DropArgs& a, cudaStream_t st) {
  const int64_t n = a.rows * a.cols;
  const bool flat = (a.rows == 1 || (a.ld == a.cols && (!RES || a.ld_res == a.cols))) && n % 8 == 0 && mxq_host::aligned16(a.x) &&
                    mxq_host::aligned16(a.res) && mxq_host::aligned16(a.y);
  const int64_t per = flat ? 8 * TPB : 4 * TPB, want = (n + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(want, 0x7FFFFFFF)));
  return flat ? mxq_host::launch_pdl(dropout_kernel<T, RES>, grid, dim3(TPB), 0, st, a)
              : mxq_host::launch_pdl(dropout_any_kernel<T, RES>, grid, dim3(TPB), 0, st, a);
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
  DropArgs a{x, residual, y, rows, cols, ld, ld_residual, seed, offset, offset_dev,
             t >= 4294967295.0 ? 0xFFFFFFFFu : static_cast<uint32_t>(t), static_cast<float>(1.0 / (1.0 - p))};
  const auto st = static_cast<cudaStream_t>(stream);
  if (type == MXQ_F32) return residual ? run<float, true>(a, st) : run<float, false>(a, st);
  return residual ? run<__nv_bfloat16, true>(a, st) : run<__nv_bfloat16, false>(a, st);
}
