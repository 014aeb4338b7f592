// Tokens gathered into rows by expert, straight to MX operands:
//   rows[r] = x[slot(r) / top], 0 in padding, quantized as mxq_quantize does
// (row blocks of 1 x 32, column blocks of 32 x 1 stored transposed), without
// the bf16 rows ever being in memory.
//
// A tile's rows come by asynchronous copies (zeros for padding) while the tile
// before is encoded; a thread encodes whole blocks, from 16 words of a row or
// from 32 of two columns.  8192 x 4096, 2 of 16 experts, rows and columns: 54 us for
// 20224 rows (35.5 of bytes at the copy rate); rows alone 35, columns alone 38 (22.8).
// No unit is full (issue ports 57 %, ALU 49 %, memory 55 %): the registers allow 24
// warps an SM, and each waits in turn for its own results, for a port, for the tile's
// two barriers and for shared memory (1.4, 1.4, 1.3 and 1.0 of 9 cycles an
// instruction).  Three CTAs an SM against two: 54 and 62 us.
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

// The larger magnitudes of two pairs of bf16, half by half (a NaN gives NaN);
// the signs of the halves mean nothing.
__device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int N>
__device__ __forceinline__ uint32_t amax_words(const uint32_t (&w)[N]) {
  uint32_t t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = w[i];
#pragma unroll
  for (int n = N / 2; n; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = amax2(t[i], t[i + n]);
  return t[0];
}
// The halves' magnitudes as float32 bits.
__device__ __forceinline__ uint32_t mag_lo(uint32_t m) { return (m << 16) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t mag_hi(uint32_t m) { return m & 0x7FFF0000u; }

// Codes of a block (32 bytes of FP8, 16 of packed E2M1).
template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* p, uint32_t (&q)[code_words<FMT, 32>()], bool bad, int wide) {
  if (bad) {                                 // rare
#pragma unroll
    for (int i = 0; i < code_words<FMT, 32>(); ++i) q[i] = 0u;
  }
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

// A block of 32 neighbours in 16 words: codes to `dst`, scale byte returned.
template <int FMT>
__device__ __forceinline__ uint32_t encode_row(const uint32_t (&w)[16], int ceil_mode, uint8_t* dst, int wide) {
  const uint32_t m = amax_words(w);
  float mult;
  const uint32_t code = mx_scale<FMT>(max(mag_lo(m), mag_hi(m)), ceil_mode, mult);
  uint32_t q[code_words<FMT, 32>()];
  if constexpr (FMT == MXQ_E2M1) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[2 * i] = bf16lo(w[i]), v[2 * i + 1] = bf16hi(w[i]);
    mx_codes<FMT, 32>(v, mult, false, q);
  } else {
    const uint64_t mm = f32x2_splat(mult);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fp8x4_rows<FMT>(w[2 * i], w[2 * i + 1], mm);
  }
  store_codes<FMT>(dst, q, code == 0xFFu, wide);
  return code;
}

// One of two neighbouring columns (the low or high halves of 32 words), of the
// largest magnitude `ab`.
template <int FMT, int HALF>
__device__ __forceinline__ uint32_t encode_col(const uint32_t (&w)[32], uint32_t ab, int ceil_mode, uint8_t* dst, int wide) {
  float mult;
  const uint32_t code = mx_scale<FMT>(ab, ceil_mode, mult);
  uint32_t q[code_words<FMT, 32>()];
  if constexpr (FMT == MXQ_E2M1) {
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = HALF ? bf16hi(w[i]) : bf16lo(w[i]);
    mx_codes<FMT, 32>(v, mult, false, q);
  } else {
    const uint64_t mm = f32x2_splat(mult);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fp8x4_col<FMT, HALF>(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3], mm);
  }
  store_codes<FMT>(dst, q, code == 0xFFu, wide);
  return code;
}

// A tile of padding: codes and scales of zeros are zeros.
template <int FMT, int ORIENT>
__device__ __forceinline__ void zero_tile(const GatherMx& a, int64_t r0, int c0) {
  constexpr int SH = FMT == MXQ_E2M1 ? 1 : 0;            // E2M1: half a byte to a code
  const int cols = min(TILE, a.cols - c0);
  const uint4 z = make_uint4(0, 0, 0, 0);
  if constexpr (ORIENT & MXQ_ROW) {
    const int words = cols >> (4 + SH);                  // of a row
    for (int i = threadIdx.x; i < TILE * words; i += T)
      *reinterpret_cast<uint4*>(a.q_row + (((r0 + i / words) * a.cols + c0) >> SH) + i % words * 16) = z;
    const int kb = a.cols / 32;
    for (int i = threadIdx.x; i < TILE * (cols / 32); i += T)
      a.s_row[scale_at(r0 + i % TILE, c0 / 32 + i / TILE, kb, a.mma)] = 0;
  }
  if constexpr (ORIENT & MXQ_COL) {
    constexpr int WORDS = TILE >> (4 + SH);
    for (int i = threadIdx.x; i < cols * WORDS; i += T)
      *reinterpret_cast<uint4*>(a.q_col + (((c0 + i / WORDS) * a.rows + r0) >> SH) + i % WORDS * 16) = z;
    for (int c = threadIdx.x; c < cols; c += T)
      *reinterpret_cast<uint32_t*>(a.s_col + scale_at(c0 + c, r0 / 32, a.rows / 32, a.mma)) = 0u;
  }
}

template <int FMT, int ORIENT>
__global__ void __launch_bounds__(T, 3) gather_mx_kernel(const GatherMx a) {
  extern __shared__ __align__(16) uint8_t buf[];
  __shared__ int token[2][TILE];                         // token of each row of a tile, -1: none
  __shared__ uint32_t col_scales[TILE];
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x;
  const int ntiles = a.tiles_r * a.tiles_c, step = gridDim.x;
  const int lc = (tid & 15) * 8, lr = tid >> 4;          // this thread's chunk of 16 bytes of rows lr, lr + 16, ...

  const auto slot_of = [&](int tile) {
    return tid < TILE && tile < ntiles ? a.row_slot[static_cast<int64_t>(tile / a.tiles_c) * TILE + tid] : -1;
  };
  // tokens of a tile's rows to place b; returns (after the barrier) whether it has any
  const auto keep = [&](int slot, int b) {
    const int t = slot < 0 ? -1 : slot / a.top;
    if (tid < TILE) token[b][tid] = t < a.tokens ? t : -1;
    return __syncthreads_or(t >= 0);
  };
  const auto load = [&](int tile, int b) {
    const int c = (tile % a.tiles_c) * TILE + lc;
    const uint32_t dst = smem_u32(buf) + b * BUF + lr * PITCH + lc * 2;
#pragma unroll
    for (int i = 0; i < TILE / 16; ++i) {
      const int t = token[b][i * 16 + lr];
      const bool live = t >= 0 && c < a.cols;
      cp_async16(dst + i * 16 * PITCH, live ? a.x + t * a.ld + c : a.x, live);
    }
    cp_async_commit();
  };

  int tile = blockIdx.x, b = 0;
  bool live = keep(slot_of(tile), 0), live_next = keep(slot_of(tile + step), 1);
  if (live) load(tile, 0);
  else cp_async_commit();
  for (; tile < ntiles; tile += step, b ^= 1) {
    const int ahead = slot_of(tile + 2 * step);
    if (live_next) load(tile + step, b ^ 1);
    else cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const uint8_t* const t = buf + b * BUF;
    const int64_t r0 = static_cast<int64_t>(tile / a.tiles_c) * TILE;
    const int c0 = (tile % a.tiles_c) * TILE;
    if (!live) {
      zero_tile<FMT, ORIENT>(a, r0, c0);
      live = live_next, live_next = keep(ahead, b);
      continue;
    }
    if constexpr (ORIENT & MXQ_ROW) {
      // a thread takes every other block of a row
      const int r = tid >> 1, h = tid & 1;
      const int64_t row = r0 + r;
      const int kb = a.cols / 32;
      uint32_t scales = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = c0 + (h + 2 * k) * 32;
        if (c < a.cols) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 q = *reinterpret_cast<const uint4*>(t + r * PITCH + (h + 2 * k) * 64 + i * 16);
            w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
          }
          const int64_t el = row * a.cols + c;
          const uint32_t s = encode_row<FMT>(w, a.ceil_mode, a.q_row + (FMT == MXQ_E2M1 ? el / 2 : el), a.wide);
          if (!a.mma) a.s_row[row * kb + c / 32] = static_cast<uint8_t>(s);
          scales |= s << (8 * (h + 2 * k));
        }
      }
      if (a.mma) {                                       // whole tiles: the four scales of a row as one word
        scales |= __shfl_xor_sync(0xFFFFFFFFu, scales, 1);
        if (!h) *reinterpret_cast<uint32_t*>(a.s_row + scale_at(row, c0 / 32, kb, 1)) = scales;
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
        const uint32_t m = amax_words(w);
        const int64_t el = c * a.rows + r0 + rb * 32;
        uint8_t* const dst = a.q_col + (FMT == MXQ_E2M1 ? el / 2 : el);
        const int64_t next = FMT == MXQ_E2M1 ? a.rows / 2 : a.rows;
        const uint32_t s0 = encode_col<FMT, 0>(w, mag_lo(m), a.ceil_mode, dst, a.wide);
        const uint32_t s1 = encode_col<FMT, 1>(w, mag_hi(m), a.ceil_mode, dst + next, a.wide);
        uint8_t* const sc = reinterpret_cast<uint8_t*>(col_scales + 2 * cp) + rb;
        sc[0] = static_cast<uint8_t>(s0);
        sc[4] = static_cast<uint8_t>(s1);
      }
    }
    live = live_next, live_next = keep(ahead, b);
    if constexpr (ORIENT & MXQ_COL) {
      // a column's four scales side by side, in either layout (rows are whole tiles)
      const int c = c0 + tid;
      if (tid < TILE && c < a.cols)
        *reinterpret_cast<uint32_t*>(a.s_col + scale_at(c, r0 / 32, a.rows / 32, a.mma)) = col_scales[tid];
    }
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
  if (((orient & MXQ_ROW) && sf_layout == MXQ_SF_MMA && !aligned16(s_row)) || ((orient & MXQ_COL) && !aligned16(s_col)))
    return MXQ_ERR_MISALIGNED;
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
