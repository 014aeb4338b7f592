// Layer norm straight to MX codes and scales: the float32 y is quantized by
// the rules of the MX quantizer, in row blocks, column blocks or both.
#include <atomic>

#include "norm.cuh"

namespace mxq {
namespace {

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

template <typename TX, int FMT, int ORIENT, bool CLUSTER, int S, int T, bool FULL>
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
  const int nc = FULL ? S : min(S, a.cols - c0);         // columns of this slab (a multiple of 32)
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
          if (!FULL) raw[r][v][i].fill(0);
          if (FULL || v * 512 + lane * 16 < nc) raw[r][v][i].load(x + r * a.ld + v * 512 + i * WV);
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

  // the slab's part of the statistics of the rows in registers, to every CTA
  const auto send_stats = [&](int tile) {
    const int buf = (tile - first) & 1;
    // (once a wait has given up, its phase may still be open: no second arrival)
    if (threadIdx.x == 0 && alive) mbar_arrive_expect_tx(smem_u32(&bar[buf]), 256 * slabs);
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
        if (FULL || v * 512 + lane * 16 < nc) s[r] += vec_sq_dev(f, near);
      }
    }
    const float m2 = rows_sum(s);
    if (lk < slabs)
      st_async_f2(smem_u32(&parts[buf][rank][warp * RW + lr]), smem_u32(&bar[buf]), lk, sum, m2);
  };

  // scale addresses: a part of the thread's own, and one of the tile
  const int kbr = a.cols / 32, kbc = a.rows / 32;        // scales of a row of the row and the column copy
  const int k0 = (c0 + lane * 16) / 32;
  const int64_t row_step = a.mma ? 16 : kbr;
  uint8_t* const my_rows = a.s_row + scale_at(0, k0, kbr, a.mma) + warp * RW * row_step;
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
  if (CLUSTER && first < last) send_stats(first);
  for (int tile = first; tile < last; ++tile) {
    const int64_t row0 = static_cast<int64_t>(tile) * 32;
    float mean, rstd;                                    // of row lr of this warp
    if constexpr (CLUSTER) {
      const int buf = (tile - first) & 1;
      if (alive) alive = mbar_wait_sleep<true>(smem_u32(&bar[buf]), ((tile - first) >> 1) & 1, status);
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
      const bool valid = FULL || at < nc;
      float y[RW][16], m[RW];
      float2 mm[RW], rr[RW];
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        mm[r] = splat(__shfl_sync(0xFFFFFFFFu, mean, r * GS));
        rr[r] = splat(__shfl_sync(0xFFFFFFFFu, rstd, r * GS));
        m[r] = 0.f;
        run(r, v, y[r]);
      }
      if (valid) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int po = p * (S / 4) + at / 4;
          const float4 w = *reinterpret_cast<const float4*>(wtile + po), b = *reinterpret_cast<const float4*>(btile + po);
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            float(&o)[16] = y[r];
            const float2 u0 = fma2(mul2(sub2(pair(o[4 * p], o[4 * p + 1]), mm[r]), rr[r]), pair(w.x, w.y), pair(b.x, b.y));
            const float2 u1 = fma2(mul2(sub2(pair(o[4 * p + 2], o[4 * p + 3]), mm[r]), rr[r]), pair(w.z, w.w), pair(b.z, b.w));
            o[4 * p] = u0.x, o[4 * p + 1] = u0.y, o[4 * p + 2] = u1.x, o[4 * p + 3] = u1.y;
            m[r] = fmax3_nan(m[r], fabsf(u0.x), fabsf(u0.y));
            m[r] = fmax3_nan(m[r], fabsf(u1.x), fabsf(u1.y));
            if constexpr (ORIENT & MXQ_COL)
              *reinterpret_cast<float4*>(ytile + (warp * RW + r) * S + po) = make_float4(u0.x, u0.y, u1.x, u1.y);
          }
        }
      }
      if constexpr (ORIENT & MXQ_ROW) {
        const int64_t el = (row0 + warp * RW) * a.cols + c0 + at;
        uint8_t* const codes = a.q_row + (FMT == MXQ_E2M1 ? el / 2 : el);
        uint8_t* const scales = my_rows + v * (a.mma ? 4 * 512 : 16) +
                                (a.mma ? static_cast<int64_t>(tile >> 2) * (kbr >> 2) * 512 + (tile & 3) * 4 : row0 * kbr);
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const float top = fmax3_nan(m[r], __shfl_xor_sync(0xFFFFFFFFu, m[r], 1), 0.f);
          float mult;
          const uint32_t code = mx_scale<FMT>(__float_as_uint(top) & 0x7FFFFFFFu, a.ceil_mode, mult);
          if (valid) {
            uint32_t q[code_words<FMT, 16>()];
            mx_codes<FMT, 16>(y[r], mult, code == 0xFFu, q);
            uint8_t* dst = codes + (FMT == MXQ_E2M1 ? static_cast<int64_t>(r) * a.cols / 2 : static_cast<int64_t>(r) * a.cols);
            if constexpr (FMT == MXQ_E2M1) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
            else *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
          }
          if (a.pack_row) {                              // the scales of four neighbouring blocks as one word
            uint32_t word = code << (8 * ((lane >> 1) & 3));
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
            if (valid && lane % 8 == 0) *reinterpret_cast<uint32_t*>(scales + r * row_step) = word;
          } else if (valid && lane % 2 == 0) {
            scales[r * row_step] = static_cast<uint8_t>(code);
          }
        }
      }
    }
    if (tile + 1 < last) load(tile + 1);           // in flight through the column pass

    if constexpr (ORIENT & MXQ_COL) {
      __syncthreads();
      // the word of scales is complete when its four tiles are all this CTA's
      const bool flush = (tile & 3) == 3 || tile + 1 == last;
      const bool word = a.pack_col && (tile & 3) == 3 && tile - 3 >= first;
#pragma unroll
      for (int u = 0; u < S / T; ++u) {
        // between the columns: the next tile has arrived, and its statistics
        // travel while the remaining columns are encoded
        if (CLUSTER && u == S / T - 1 && tile + 1 < last) send_stats(tile + 1);
        const int pos = threadIdx.x + u * T;             // a column of a plane
        const int c = (pos % (S / 4)) / 4 * 16 + pos / (S / 4) * 4 + pos % 4;
        if (!FULL && c >= nc) continue;                  // (the last turn: no exchange is skipped)
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
        if (flush) {
          uint8_t* const scales = a.s_col + scale_at(c0 + c, tile & ~3, kbc, a.mma);     // four tiles, side by side
          if (word) *reinterpret_cast<uint32_t*>(scales) = acc;
          else
            for (int k = max(first, tile & ~3); k <= tile; ++k) scales[k & 3] = static_cast<uint8_t>(acc >> (8 * (k & 3)));
        }
      }
      __syncthreads();
    }
  }
  // peers may still be sending: they wait for this CTA's sums, it for theirs,
  // so nothing is on its way once every tile is merged -- unless a wait gave up
  if constexpr (CLUSTER) {
    cluster_sync();
    if (!alive) linger();
  }
}

// ---------------------------------------------------------------- host
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

template <typename TX, int FMT, int ORIENT, bool CLUSTER, int S, int T, bool FULL>
int launch_tile(const NormArgs& a, cudaStream_t st) {
  static std::atomic<int> known[64][TILE_SLABS + 1];
  const int slabs = (a.cols + S - 1) / S, cluster = CLUSTER ? slabs : 1;
  const int smem = ((ORIENT & MXQ_COL) ? 34 : 2) * S * 4;
  auto kern = norm_tile_kernel<TX, FMT, ORIENT, CLUSTER, S, T, FULL>;
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

template <typename TX, int FMT, int ORIENT, bool CLUSTER, int S, int T>
int choose_tile(const NormArgs& a, cudaStream_t st) {
  return a.cols % S == 0 ? launch_tile<TX, FMT, ORIENT, CLUSTER, S, T, true>(a, st)
                         : launch_tile<TX, FMT, ORIENT, CLUSTER, S, T, false>(a, st);
}

// Rows only: the row kernel.  With column blocks: a portable cluster (8 CTAs)
// holds 32 rows of up to 4096 columns in slabs of 512, or 8192 in slabs of
// 1024; longer rows get their statistics first, then slab by slab (x is read
// twice).
template <typename TX, int FMT, int ORIENT>
int norm_mx_tiles(const NormArgs& a, cudaStream_t st) {
  if constexpr (ORIENT != MXQ_ROW) {
    if (a.cols <= TILE_SLABS * 512) return choose_tile<TX, FMT, ORIENT, true, 512, sizeof(TX) == 2 ? 256 : 512>(a, st);
    if (a.cols <= TILE_SLABS * 1024) return choose_tile<TX, FMT, ORIENT, true, 1024, 512>(a, st);
  }
  if (const int rc = norm_stats(a, sizeof(TX) == 2 ? MXQ_BF16 : MXQ_F32, st)) return rc;
  return choose_tile<TX, FMT, ORIENT, false, 512, sizeof(TX) == 2 ? 256 : 512>(a, st);
}

template <typename TX, int FMT>
int norm_mx(const NormArgs& a, int orient, cudaStream_t st) {
  if (orient == MXQ_ROW) return a.cols <= kMaxRowElems ? dispatch_row<TX, FMT, 16 / static_cast<int>(sizeof(TX))>(a, st) : norm_mx_tiles<TX, FMT, MXQ_ROW>(a, st);
  return orient == MXQ_DUAL ? norm_mx_tiles<TX, FMT, MXQ_DUAL>(a, st) : norm_mx_tiles<TX, FMT, MXQ_COL>(a, st);
}

template <typename TX>
int norm_mx_fmt(const NormArgs& a, int fmt, int orient, cudaStream_t st) {
  if (fmt == MXQ_E4M3) return norm_mx<TX, MXQ_E4M3>(a, orient, st);
  if (fmt == MXQ_E5M2) return norm_mx<TX, MXQ_E5M2>(a, orient, st);
  return norm_mx<TX, MXQ_E2M1>(a, orient, st);
}

}  // namespace
}  // namespace mxq

using namespace mxq;

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

