// Tokens gathered into rows by expert, straight to MX operands:
//   rows[r] = x[slot(r) / top], 0 in padding, quantized as mxq_quantize does
// (row blocks of 1 x 32, column blocks of 32 x 1 stored transposed), without
// the bf16 rows ever being in memory.
#include <algorithm>
#include <atomic>

#include "rowops.cuh"

namespace mxq {
namespace {

constexpr int T = 256;
constexpr int TILE = 128;                 // rows and columns of a tile: one 512-byte chunk of scales each way
constexpr int PITCH = TILE * 2 + 16;      // bytes from row to row: 16-byte reads down a column of rows and 4-byte
                                          // reads along a row both pass without bank conflicts
constexpr int BUF = TILE * PITCH;

struct GatherMx {
  const __nv_bfloat16* x;
  const int32_t* row_slot;
  int64_t tokens, rows, ld;
  int cols, top;
  int tiles_r, tiles_c;
  uint8_t *q_row, *s_row, *q_col, *s_col;
  int ceil_mode, mma;
  int wide;                               // codes start at 32-byte boundaries
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Codes of a block (32 bytes of FP8, 16 of packed E2M1).
template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&q)[code_words<FMT, 32>()], int wide) {
  if constexpr (FMT == MXQ_E2M1) {
    *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
  } else if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(q[0]), "r"(q[1]), "r"(q[2]),
                 "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
    *reinterpret_cast<uint4*>(p + 16) = make_uint4(q[4], q[5], q[6], q[7]);
  }
}

// One block of 32 values: codes to `dst`, scale byte returned.
template <int FMT>
__device__ __forceinline__ uint32_t encode(const float (&v)[32], int ceil_mode, uint8_t* dst, int wide) {
  float mult;
  const uint32_t code = mx_scale<FMT>(amax32_tree([&](int j) { return fabsf(v[j]); }), ceil_mode, mult);
  uint32_t q[code_words<FMT, 32>()];
  mx_codes<FMT, 32>(v, mult, code == 0xFFu, q);
  store_codes<FMT>(dst, q, wide);
  return code;
}

template <int FMT, int ORIENT>
__global__ void __launch_bounds__(T) gather_mx_kernel(const GatherMx a) {
  extern __shared__ __align__(16) uint8_t buf[];
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x;
  const int ntiles = a.tiles_r * a.tiles_c;

  // a row's 16 chunks of 16 bytes go to 16 neighbouring threads
  const auto load = [&](int tile, int b) {
    const int64_t r0 = static_cast<int64_t>(tile / a.tiles_c) * TILE;
    const int c = (tile % a.tiles_c) * TILE + (tid & 15) * 8;
#pragma unroll
    for (int i = 0; i < TILE / 16; ++i) {
      const int r = i * 16 + (tid >> 4);
      const int slot = a.row_slot[r0 + r];
      const int64_t token = slot / a.top;
      const bool live = slot >= 0 && token < a.tokens && c < a.cols;
      cp_async16(smem_u32(buf + b * BUF + r * PITCH + (tid & 15) * 16), live ? a.x + token * a.ld + c : a.x, live);
    }
    cp_async_commit();
  };

  int b = 0;
  if (static_cast<int>(blockIdx.x) < ntiles) load(blockIdx.x, 0);
  for (int tile = blockIdx.x; tile < ntiles; tile += gridDim.x, b ^= 1) {
    const bool more = tile + static_cast<int>(gridDim.x) < ntiles;
    if (more) {
      load(tile + gridDim.x, b ^ 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    const uint8_t* const t = buf + b * BUF;
    const int64_t r0 = static_cast<int64_t>(tile / a.tiles_c) * TILE;
    const int c0 = (tile % a.tiles_c) * TILE;
    if constexpr (ORIENT & MXQ_ROW) {
      // a thread takes two neighbouring blocks of a row
      const int r = tid >> 1, h = (tid & 1) * 2;
      const int64_t row = r0 + r;
      const int kb = a.cols / 32;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = c0 + (h + k) * 32;
        if (c < a.cols) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(t + r * PITCH + (h + k) * 64 + i * 16);
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[8 * i + 2 * j] = bf16lo(q[j]), v[8 * i + 2 * j + 1] = bf16hi(q[j]);
          }
          const int64_t el = row * a.cols + c;
          const uint32_t s = encode<FMT>(v, a.ceil_mode, a.q_row + (FMT == MXQ_E2M1 ? el / 2 : el), a.wide);
          a.s_row[scale_at(row, c / 32, kb, a.mma)] = static_cast<uint8_t>(s);
        }
      }
    }
    if constexpr (ORIENT & MXQ_COL) {
      // a thread takes 32 rows of two neighbouring columns
      const int cp = tid & 63, rb = tid >> 6;
      const int c = c0 + 2 * cp;
      if (c < a.cols) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = *reinterpret_cast<const uint32_t*>(t + (rb * 32 + i) * PITCH + cp * 4);
        const int64_t row = r0 + rb * 32;
        const int64_t kb = a.rows / 32;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = k ? bf16hi(w[i]) : bf16lo(w[i]);
          const int64_t el = (c + k) * a.rows + row;
          const uint32_t s = encode<FMT>(v, a.ceil_mode, a.q_col + (FMT == MXQ_E2M1 ? el / 2 : el), a.wide);
          a.s_col[scale_at(c + k, row / 32, kb, a.mma)] = static_cast<uint8_t>(s);
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host
template <int FMT, int ORIENT>
int run(const GatherMx& a, cudaStream_t st) {
  static std::atomic<int> known[64];
  auto kern = gather_mx_kernel<FMT, ORIENT>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
  int n = known[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * BUF) != cudaSuccess) return MXQ_ERR_CUDA;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, T, 2 * BUF) != cudaSuccess || n < 1) return MXQ_ERR_CUDA;
    known[dev].store(n, std::memory_order_relaxed);
  }
  const int grid = std::min(a.tiles_r * a.tiles_c, n * mxq_host::sm_count());
  return mxq_host::launch_pdl(kern, dim3(grid), dim3(T), 2 * BUF, st, a);
}

template <int FMT>
int choose(const GatherMx& a, int orient, cudaStream_t st) {
  if (orient == MXQ_ROW) return run<FMT, MXQ_ROW>(a, st);
  return orient == MXQ_COL ? run<FMT, MXQ_COL>(a, st) : run<FMT, MXQ_DUAL>(a, st);
}

}  // namespace
}  // namespace mxq

using namespace mxq;
using namespace mxq_host;

extern "C" int mxq_expert_gather_mx(const void* x, int64_t tokens, int64_t cols, int64_t ld, const int32_t* row_slot,
                                    int64_t rows, int64_t top, int fmt, int orient, int scale_mode, int sf_layout,
                                    void* q_row, uint8_t* s_row, void* q_col, uint8_t* s_col, void* stream) {
  if (fmt != MXQ_E4M3 && fmt != MXQ_E5M2 && fmt != MXQ_E2M1) return MXQ_ERR_BAD_ARG;
  if (orient != MXQ_ROW && orient != MXQ_COL && orient != MXQ_DUAL) return MXQ_ERR_BAD_ARG;
  if (scale_mode != MXQ_SCALE_FLOOR_OCP && scale_mode != MXQ_SCALE_CEIL) return MXQ_ERR_BAD_ARG;
  if (sf_layout != MXQ_SF_CANONICAL && sf_layout != MXQ_SF_MMA) return MXQ_ERR_BAD_ARG;
  if (tokens < 0 || tokens > kMaxCols || top < 1 || top > kMaxCols || rows < 0 || rows > kMaxCols || rows % TILE || cols < 1 ||
      cols > kMaxCols || cols % (sf_layout == MXQ_SF_MMA ? 128 : 32) || ld < cols)
    return MXQ_ERR_BAD_SHAPE;
  const int64_t tiles_r = rows / TILE, tiles_c = (cols + TILE - 1) / TILE;
  if (tiles_r * tiles_c > 0x7FFF0000) return MXQ_ERR_BAD_SHAPE;
  if (!rows) return MXQ_OK;
  if (!x || !row_slot) return MXQ_ERR_BAD_ARG;
  if ((orient & MXQ_ROW) && (!q_row || !s_row)) return MXQ_ERR_BAD_ARG;
  if ((orient & MXQ_COL) && (!q_col || !s_col)) return MXQ_ERR_BAD_ARG;
  if (!aligned16(x) || ld % 8 || !aligned_to(row_slot, 4)) return MXQ_ERR_MISALIGNED;
  if (((orient & MXQ_ROW) && !aligned16(q_row)) || ((orient & MXQ_COL) && !aligned16(q_col))) return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  GatherMx a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.row_slot = row_slot;
  a.tokens = tokens, a.rows = rows, a.ld = ld;
  a.cols = static_cast<int>(cols), a.top = static_cast<int>(top);
  a.tiles_r = static_cast<int>(tiles_r), a.tiles_c = static_cast<int>(tiles_c);
  a.q_row = static_cast<uint8_t*>(q_row), a.s_row = s_row;
  a.q_col = static_cast<uint8_t*>(q_col), a.s_col = s_col;
  a.ceil_mode = scale_mode == MXQ_SCALE_CEIL;
  a.mma = sf_layout == MXQ_SF_MMA;
  a.wide = (!(orient & MXQ_ROW) || aligned_to(q_row, 32)) && (!(orient & MXQ_COL) || aligned_to(q_col, 32));
  const auto st = static_cast<cudaStream_t>(stream);
  if (fmt == MXQ_E4M3) return choose<MXQ_E4M3>(a, orient, st);
  return fmt == MXQ_E5M2 ? choose<MXQ_E5M2>(a, orient, st) : choose<MXQ_E2M1>(a, orient, st);
}
