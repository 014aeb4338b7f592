// Tokens sorted by expert and back, with weights and gradients:
//   sort      e[s] -> a row for every slot s (a token's j-th choice), the rows
//             of an expert in one stretch, in the slots' order
//   gather    rows[r] = x[slot(r) / top], 0 in padding
//   combine   y[t] = sum_j w[t][j] rows[row(t, j)]
//   backward  drows[row(t, j)] = w[t][j] dy[t], 0 in padding
//             dw[t][j] = sum_c dy[t][c] rows[row(t, j)][c]
//
// The sort is a counting sort of small integers: latency and launches bound
// it.  The others move rows and are bound by HBM.
#include <algorithm>

#include "rowops.cuh"

namespace mxq {
namespace {

using namespace mxq_host;

constexpr int kMaxExperts = 1024;

// ---------------------------------------------------------------- sort
constexpr int SORT_WARPS = 16, SORT_T = 32 * SORT_WARPS;
constexpr int SORT_SLOTS = 2048;          // slots of a CTA, until there are SORT_CTAS of them
constexpr int SORT_CTAS = 128;

struct SortArgs {
  const void* experts;
  int64_t slots, per;                     // per: slots of a CTA
  int64_t rows;
  int e64, E, align;
  int32_t *offsets, *counts, *slot_row, *row_slot, *block_expert;
  int32_t* part;                          // [CTAs][E] counts, where there are several CTAs
};

// The expert of a slot, or -1 where the slot is dropped.
__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t s) {
  if (a.e64) {
    const int64_t e = static_cast<const int64_t*>(a.experts)[s];
    return e >= 0 && e < a.E ? static_cast<int>(e) : -1;
  }
  const int e = static_cast<const int32_t*>(a.experts)[s];
  return e >= 0 && e < a.E ? e : -1;
}

__global__ void __launch_bounds__(SORT_T) expert_count_kernel(const SortArgs a) {
  extern __shared__ int hist[];
  grid_dep_launch();
  for (int e = threadIdx.x; e < a.E; e += SORT_T) hist[e] = 0;
  __syncthreads();
  grid_dep_wait();
  const int64_t lo = blockIdx.x * a.per, hi = min(a.slots, lo + a.per);
  for (int64_t s = lo + threadIdx.x; s < hi; s += SORT_T) {
    const int e = expert_of(a, s);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += SORT_T) a.part[static_cast<int64_t>(blockIdx.x) * a.E + e] = hist[e];
}

// Exclusive prefix sum over the CTA's threads; `total` gets the sum.
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int p = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int q = __shfl_up_sync(0xFFFFFFFFu, p, o);
    if (lane >= o) p += q;
  }
  if (lane == 31) warp_sums[warp] = p;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < SORT_WARPS; ++w) {
    const int s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
  __syncthreads();
  return before + p - v;
}

// Every CTA takes `per` slots, every warp of it an even stretch of them.  A
// slot's row is the start of its expert's stretch, the slots of that expert in
// earlier CTAs, in earlier warps of its CTA, and earlier in its warp: an order
// that depends on nothing but the slots.
__global__ void __launch_bounds__(SORT_T) expert_place_kernel(const SortArgs a) {
  extern __shared__ int sm[];
  int* const off = sm;                            // [E + 1] starts of the experts' stretches
  int* const cnt = off + a.E + 1;                 // [E] slots of each expert
  int* const wcnt = cnt + a.E;                    // [SORT_WARPS][E]
  __shared__ int warp_sums[SORT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < SORT_WARPS * a.E; i += SORT_T) wcnt[i] = 0;
  __syncthreads();
  grid_dep_wait();

  const int64_t lo = blockIdx.x * a.per, hi = min(a.slots, lo + a.per);
  const int64_t each = (a.per + SORT_WARPS * 32 - 1) / (SORT_WARPS * 32) * 32;
  const int64_t wlo = min(hi, lo + warp * each), whi = min(hi, wlo + each);
  int* const mine = wcnt + warp * a.E;
  for (int64_t s = wlo + lane; s < whi; s += 32) {
    const int e = expert_of(a, s);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();

  // this CTA's counts by warp become the counts of earlier CTAs and warps
  for (int e = threadIdx.x; e < a.E; e += SORT_T) {
    int before = 0, all = 0;
    if (gridDim.x > 1) {
#pragma unroll 8
      for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
        const int n = __ldcg(a.part + static_cast<int64_t>(b) * a.E + e);
        if (b < static_cast<int>(blockIdx.x)) before += n;
        all += n;
      }
    }
    int run = before;
#pragma unroll
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int n = wcnt[w * a.E + e];
      wcnt[w * a.E + e] = run;
      run += n;
    }
    cnt[e] = gridDim.x > 1 ? all : run;
  }
  __syncthreads();
  int base = 0;
  for (int e0 = 0; e0 < a.E; e0 += SORT_T) {
    const int e = e0 + threadIdx.x;
    const int v = e < a.E ? (cnt[e] + a.align - 1) / a.align * a.align : 0;
    int total;
    const int p = block_prefix(v, warp_sums, total);
    if (e < a.E) off[e] = base + p;
    base += total;
  }
  if (threadIdx.x == 0) off[a.E] = base;
  __syncthreads();

  for (int64_t s0 = wlo; s0 < whi; s0 += 32) {
    const int64_t s = s0 + lane;
    const int e = s < whi ? expert_of(a, s) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int first = 0;
    if (e >= 0) first = mine[e];
    __syncwarp();
    if (e >= 0 && rank == 0) mine[e] = first + __popc(same);
    __syncwarp();
    if (s < whi) {
      const int row = e >= 0 ? off[e] + first + rank : -1;
      a.slot_row[s] = row;
      if (row >= 0 && row < a.rows) a.row_slot[row] = static_cast<int32_t>(s);
    }
  }

  // what no slot fills: the padding of every expert, the rows behind the last
  for (int e = blockIdx.x * SORT_WARPS + warp; e < a.E; e += gridDim.x * SORT_WARPS)
    for (int r = off[e] + cnt[e] + lane; r < off[e + 1]; r += 32) a.row_slot[r] = -1;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * SORT_T, at = static_cast<int64_t>(blockIdx.x) * SORT_T + threadIdx.x;
  for (int64_t r = off[a.E] + at; r < a.rows; r += stride) a.row_slot[r] = -1;
  for (int64_t b = at; b < a.rows / a.align; b += stride) {
    const int r = static_cast<int>(b * a.align);
    int e = -1;
    if (r < off[a.E]) {                           // the last expert that starts at or before r (empty ones start where the next does)
      int l = 0, h = a.E;
      while (h - l > 1) {
        const int m = (l + h) / 2;
        if (off[m] <= r) l = m;
        else h = m;
      }
      e = l;
    }
    a.block_expert[b] = e;
  }
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e <= a.E; e += SORT_T) a.offsets[e] = off[e];
    for (int e = threadIdx.x; e < a.E; e += SORT_T) a.counts[e] = cnt[e];
  }
}

// ---------------------------------------------------------------- rows
constexpr int ROW_T = 256, ROW_WARPS = ROW_T / 32;
constexpr int U = 4;                      // vectors of a lane in flight per row

struct RowArgs {
  const void* src;                        // gather: x; combine: rows; backward: rows
  const void* dy;                         // backward
  void* out;                              // rows; y; drows
  float* dw;
  const int32_t *slot_row, *row_slot;
  const void* w;                          // or nullptr: 1
  int w_f32;
  int64_t tokens, rows, cols, ld, ld_dy;
  int top;
  int64_t pieces;                         // stretches of 32 * U vectors to a row
};

__device__ __forceinline__ float weight_of(const RowArgs& a, int64_t slot) {
  if (!a.w) return 1.f;
  return a.w_f32 ? static_cast<const float*>(a.w)[slot] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[slot]);
}

// One warp takes one stretch of a token: it is read once and written to the
// row of each of the token's slots.  Padding rows are warps of their own.
template <typename T, int VE>
__global__ void __launch_bounds__(ROW_T) gather_kernel(const RowArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * static_cast<int64_t>(ROW_WARPS) + (threadIdx.x >> 5);
  const int64_t row = item / a.pieces, c0 = (item - row * a.pieces) * (32 * U * VE) + lane * VE;
  T* const out = static_cast<T*>(a.out);
  Vec<T, VE> v[U];
  if (row >= a.tokens) {
    const int64_t r = row - a.tokens;
    if (r >= a.rows || a.row_slot[r] >= 0) return;
    v[0].fill(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 32 * VE;
      if (c < a.cols) v[0].store(out + r * a.cols + c);
    }
    return;
  }
  const T* const x = static_cast<const T*>(a.src) + row * a.ld;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + u * 32 * VE;
    if (c < a.cols) v[u].load(x + c);
  }
  for (int j = 0; j < a.top; ++j) {
    const int64_t r = a.slot_row[row * a.top + j];
    if (r < 0 || r >= a.rows) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 32 * VE;
      if (c < a.cols) v[u].store(out + r * a.cols + c);
    }
  }
}

template <typename T, typename TY, int VE>
__global__ void __launch_bounds__(ROW_T) combine_kernel(const RowArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * static_cast<int64_t>(ROW_WARPS) + (threadIdx.x >> 5);
  const int64_t t = item / a.pieces, c0 = (item - t * a.pieces) * (32 * U * VE) + lane * VE;
  if (t >= a.tokens) return;
  float acc[U][VE];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[u][i] = 0.f;
#pragma unroll 2
  for (int j = 0; j < a.top; ++j) {
    const int64_t slot = t * a.top + j, r = a.slot_row[slot];
    if (r < 0 || r >= a.rows) continue;
    const float w = weight_of(a, slot);
    const T* const src = static_cast<const T*>(a.src) + r * a.ld;
    Vec<T, VE> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 32 * VE;
      v[u].fill(0);
      if (c < a.cols) v[u].load(src + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < VE; ++i) acc[u][i] = fmaf(w, v[u].get(i), acc[u][i]);
  }
  TY* const y = static_cast<TY*>(a.out) + t * a.cols;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + u * 32 * VE;
    if (c < a.cols) store_vec<TY, VE>(y + c, acc[u]);
  }
}

// A CTA takes a token: dy's stretches stay in registers while the rows of its
// slots pass (rows of more than a stretch per warp go round again).
template <typename T, typename TY, int VE>
__global__ void __launch_bounds__(ROW_T) combine_bwd_kernel(const RowArgs a) {
  __shared__ float red[ROW_WARPS];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T* const out = static_cast<T*>(a.out);
  if (blockIdx.x >= a.tokens) {
    // ROW_WARPS rows, a warp each: padding gets zeros
    const int64_t r = (blockIdx.x - a.tokens) * static_cast<int64_t>(ROW_WARPS) + warp;
    if (r >= a.rows || a.row_slot[r] >= 0) return;
    Vec<T, VE> z;
    z.fill(0);
    for (int64_t c = lane * VE; c < a.cols; c += 32 * VE) z.store(out + r * a.cols + c);
    return;
  }
  const int64_t t = blockIdx.x;
  const TY* const dy = static_cast<const TY*>(a.dy) + t * a.ld_dy;
  for (int j = 0; j < a.top; ++j) {
    const int64_t slot = t * a.top + j, r = a.slot_row[slot];
    const bool live = r >= 0 && r < a.rows;
    float dot = 0.f;
    if (live) {
      const float w = weight_of(a, slot);
      const T* const src = static_cast<const T*>(a.src) + r * a.ld;
      for (int64_t c0 = threadIdx.x * VE; c0 < a.cols; c0 += ROW_T * VE * 2) {
        Vec<T, VE> v[2];
        float g[2][VE];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t c = c0 + u * ROW_T * VE;
          if (c < a.cols) {
            v[u].load(src + c);
            load_elems<TY, VE>(dy + c, g[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t c = c0 + u * ROW_T * VE;
          if (c < a.cols) {
            float q[VE], d[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              q[i] = g[u][i] * v[u].get(i);
              d[i] = g[u][i] * w;
            }
            dot += tree_sum(q);
            store_vec<T, VE>(out + r * a.cols + c, d);
          }
        }
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) red[warp] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < ROW_WARPS; ++k) s += red[k];
      a.dw[slot] = live ? s : 0.f;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host
bool plan_sizes(int64_t tokens, int64_t top, int64_t rows) {
  return tokens >= 0 && top >= 1 && rows >= 0 && top <= kMaxCols && tokens <= kMaxCols / top && rows <= kMaxCols;
}

bool wide(const void* p, int64_t ld, int type, int64_t cols) {
  const int s = type_size(type);
  return aligned16(p) && (ld * s) % 16 == 0 && (cols * s) % 16 == 0;
}

int ctas(int64_t items, unsigned* grid) {
  const int64_t n = (items + ROW_WARPS - 1) / ROW_WARPS;
  if (n > 0x7FFFFFFF) return MXQ_ERR_BAD_SHAPE;
  *grid = static_cast<unsigned>(n);
  return MXQ_OK;
}

template <typename T, int VE>
int run_gather(RowArgs a, cudaStream_t st) {
  a.pieces = (a.cols + 32 * U * VE - 1) / (32 * U * VE);
  unsigned grid = 0;
  if (const int rc = ctas((a.tokens + a.rows) * a.pieces, &grid)) return rc;
  return grid ? launch_pdl(gather_kernel<T, VE>, dim3(grid), dim3(ROW_T), 0, st, a) : MXQ_OK;
}

template <typename T, typename TY, int VE>
int run_combine(RowArgs a, cudaStream_t st) {
  a.pieces = (a.cols + 32 * U * VE - 1) / (32 * U * VE);
  unsigned grid = 0;
  if (const int rc = ctas(a.tokens * a.pieces, &grid)) return rc;
  return grid ? launch_pdl(combine_kernel<T, TY, VE>, dim3(grid), dim3(ROW_T), 0, st, a) : MXQ_OK;
}

template <typename T, typename TY, int VE>
int run_backward(const RowArgs& a, cudaStream_t st) {
  const int64_t grid = a.tokens + (a.rows + ROW_WARPS - 1) / ROW_WARPS;
  if (grid > 0x7FFFFFFF) return MXQ_ERR_BAD_SHAPE;
  return grid ? launch_pdl(combine_bwd_kernel<T, TY, VE>, dim3(static_cast<unsigned>(grid)), dim3(ROW_T), 0, st, a) : MXQ_OK;
}

int64_t sort_ctas(int64_t slots) { return std::max<int64_t>(1, std::min<int64_t>(SORT_CTAS, (slots + SORT_SLOTS - 1) / SORT_SLOTS)); }

}  // namespace
}  // namespace mxq

using namespace mxq;
using namespace mxq_host;

extern "C" int mxq_expert_rows(int64_t slots, int experts, int align, int64_t* rows) {
  if (!rows) return MXQ_ERR_BAD_ARG;
  if (slots < 0 || slots > kMaxCols || experts < 1 || experts > kMaxExperts) return MXQ_ERR_BAD_SHAPE;
  if (align != 128 && align != 256) return MXQ_ERR_BAD_ARG;
  const int64_t r = (slots + std::min<int64_t>(experts, slots) * (align - 1)) / align * align;
  if (r > kMaxCols) return MXQ_ERR_BAD_SHAPE;
  *rows = r;
  return MXQ_OK;
}

extern "C" int mxq_expert_sort_workspace_size(int64_t slots, int experts, size_t* bytes) {
  if (!bytes) return MXQ_ERR_BAD_ARG;
  if (slots < 0 || slots > kMaxCols || experts < 1 || experts > kMaxExperts) return MXQ_ERR_BAD_SHAPE;
  *bytes = static_cast<size_t>(sort_ctas(slots)) * experts * sizeof(int32_t);
  return MXQ_OK;
}

extern "C" int mxq_expert_sort(const void* experts, int experts_64, int64_t slots, int num_experts, int align,
                               int64_t rows, int32_t* offsets, int32_t* counts, int32_t* slot_row, int32_t* row_slot,
                               int32_t* block_expert, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t need_rows = 0;
  size_t need = 0;
  if (const int rc = mxq_expert_rows(slots, num_experts, align, &need_rows)) return rc;
  mxq_expert_sort_workspace_size(slots, num_experts, &need);
  if (experts_64 != 0 && experts_64 != 1) return MXQ_ERR_BAD_ARG;
  if (rows != need_rows) return MXQ_ERR_BAD_SHAPE;
  if (!offsets || !counts || (slots && (!experts || !slot_row || !row_slot || !block_expert))) return MXQ_ERR_BAD_ARG;
  if (!workspace || workspace_bytes < need) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(experts, experts_64 ? 8 : 4) || !aligned_to(offsets, 4) || !aligned_to(counts, 4) ||
      !aligned_to(slot_row, 4) || !aligned_to(row_slot, 4) || !aligned_to(block_expert, 4) || !aligned16(workspace))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  const int64_t n = sort_ctas(slots);
  SortArgs a{experts, slots, (slots + n - 1) / n, rows, experts_64, num_experts, align, offsets, counts, slot_row,
             row_slot, block_expert, static_cast<int32_t*>(workspace)};
  const auto st = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(n));
  if (n > 1)
    if (const int rc = launch_pdl(expert_count_kernel, grid, dim3(SORT_T), num_experts * sizeof(int), st, a)) return rc;
  const size_t smem = ((2 + SORT_WARPS) * num_experts + 1) * sizeof(int);
  static bool set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MXQ_ERR_CUDA;
  if (!set[dev & 63]) {
    if (cudaFuncSetAttribute(expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ((2 + SORT_WARPS) * kMaxExperts + 1) * sizeof(int)) != cudaSuccess)
      return MXQ_ERR_CUDA;
    set[dev & 63] = true;
  }
  return launch_pdl(expert_place_kernel, grid, dim3(SORT_T), smem, st, a);
}

extern "C" int mxq_expert_gather(const void* x, int64_t tokens, int64_t cols, int64_t ld, int x_type,
                                 const int32_t* slot_row, int64_t top, const int32_t* row_slot, int64_t rows, void* out,
                                 void* stream) {
  if (!valid_type(x_type)) return MXQ_ERR_BAD_ARG;
  if (!plan_sizes(tokens, top, rows) || cols < 1 || cols > kMaxCols || ld < cols) return MXQ_ERR_BAD_SHAPE;
  if ((tokens && (!x || !slot_row)) || (rows && (!row_slot || !out))) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(x, type_size(x_type)) || !aligned_to(out, type_size(x_type)) || !aligned_to(slot_row, 4) ||
      !aligned_to(row_slot, 4))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  RowArgs a{};
  a.src = x, a.out = out, a.slot_row = slot_row, a.row_slot = row_slot;
  a.tokens = tokens, a.rows = rows, a.cols = cols, a.ld = ld, a.top = static_cast<int>(top);
  const auto st = static_cast<cudaStream_t>(stream);
  const bool v = wide(x, ld, x_type, cols) && aligned16(out);
  if (x_type == MXQ_F32) return v ? run_gather<float, 4>(a, st) : run_gather<float, 1>(a, st);
  return v ? run_gather<__nv_bfloat16, 8>(a, st) : run_gather<__nv_bfloat16, 1>(a, st);
}

extern "C" int mxq_expert_combine(const void* rows_in, int64_t rows, int64_t cols, int64_t ld, int type,
                                  const int32_t* slot_row, int64_t tokens, int64_t top, const void* weights, int w_type,
                                  void* y, int y_type, void* stream) {
  if (!valid_type(type) || !valid_type(y_type) || (weights && !valid_type(w_type))) return MXQ_ERR_BAD_ARG;
  if (!plan_sizes(tokens, top, rows) || cols < 1 || cols > kMaxCols || ld < cols) return MXQ_ERR_BAD_SHAPE;
  if ((rows && !rows_in) || (tokens && (!slot_row || !y))) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(rows_in, type_size(type)) || !aligned_to(y, type_size(y_type)) || !aligned_to(slot_row, 4) ||
      (weights && !aligned_to(weights, type_size(w_type))))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  RowArgs a{};
  a.src = rows_in, a.out = y, a.slot_row = slot_row, a.w = weights, a.w_f32 = w_type == MXQ_F32;
  a.tokens = tokens, a.rows = rows, a.cols = cols, a.ld = ld, a.top = static_cast<int>(top);
  const auto st = static_cast<cudaStream_t>(stream);
  const bool v = wide(rows_in, ld, type, cols) && aligned16(y);
  using bf = __nv_bfloat16;
  if (type == MXQ_F32) {
    if (y_type == MXQ_F32) return v ? run_combine<float, float, 4>(a, st) : run_combine<float, float, 1>(a, st);
    return v ? run_combine<float, bf, 4>(a, st) : run_combine<float, bf, 1>(a, st);
  }
  if (y_type == MXQ_F32) return v ? run_combine<bf, float, 8>(a, st) : run_combine<bf, float, 1>(a, st);
  return v ? run_combine<bf, bf, 8>(a, st) : run_combine<bf, bf, 1>(a, st);
}

extern "C" int mxq_expert_combine_backward(const void* dy, int64_t ld_dy, int dy_type, const void* rows_in, int64_t ld,
                                           int type, int64_t rows, int64_t cols, const int32_t* slot_row,
                                           const int32_t* row_slot, int64_t tokens, int64_t top, const void* weights,
                                           int w_type, void* drows, float* dweights, void* stream) {
  if (!valid_type(type) || !valid_type(dy_type) || !valid_type(w_type)) return MXQ_ERR_BAD_ARG;
  if (!plan_sizes(tokens, top, rows) || cols < 1 || cols > kMaxCols || ld < cols || ld_dy < cols) return MXQ_ERR_BAD_SHAPE;
  if ((rows && (!rows_in || !row_slot || !drows)) || (tokens && (!dy || !slot_row || !weights || !dweights)))
    return MXQ_ERR_BAD_ARG;
  if (!aligned_to(rows_in, type_size(type)) || !aligned_to(dy, type_size(dy_type)) || !aligned_to(drows, type_size(type)) ||
      !aligned_to(slot_row, 4) || !aligned_to(row_slot, 4) || !aligned_to(weights, type_size(w_type)) ||
      !aligned_to(dweights, 4))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  RowArgs a{};
  a.src = rows_in, a.dy = dy, a.out = drows, a.dw = dweights, a.slot_row = slot_row, a.row_slot = row_slot;
  a.w = weights, a.w_f32 = w_type == MXQ_F32;
  a.tokens = tokens, a.rows = rows, a.cols = cols, a.ld = ld, a.ld_dy = ld_dy, a.top = static_cast<int>(top);
  const auto st = static_cast<cudaStream_t>(stream);
  // a vector is 16 bytes of the rows; dy's side of it is 8, 16 or 32
  const bool v = wide(rows_in, ld, type, cols) && aligned16(drows) && wide(dy, ld_dy, dy_type, cols);
  using bf = __nv_bfloat16;
  if (type == MXQ_F32) {
    if (dy_type == MXQ_F32) return v ? run_backward<float, float, 4>(a, st) : run_backward<float, float, 1>(a, st);
    return v ? run_backward<float, bf, 4>(a, st) : run_backward<float, bf, 1>(a, st);
  }
  if (dy_type == MXQ_F32) return v ? run_backward<bf, float, 8>(a, st) : run_backward<bf, float, 1>(a, st);
  return v ? run_backward<bf, bf, 8>(a, st) : run_backward<bf, bf, 1>(a, st);
}
