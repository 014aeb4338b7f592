// Block-scaled products of all experts in one launch:
//   products  C[r][n] = sum_k A[r][k] B[e(r)][n][k], rows in stretches by expert
//   gradient  C[e][n][k] = sum over e's rows r of A[n][r] B[k][r]
// (A and B dequantized, accumulated in float32 on the tensor cores).  The
// stretches' bounds are read from the plan in device memory: no size of one
// reaches the host.
//
// A tile is 128 CTAS x BN of C.  CTAS == 2: a pair of CTAs on two SMs computes
// 256 x 256 with tcgen05.mma.cta_group::2, each holding its 128 rows of A and
// half of B.  CTAS == 1: 128 x 256, or 128 x 128 with two accumulators in tensor
// memory, one of which drains while the other fills.
// Roles (one CTA per SM, persistent over tiles), as in the plain products:
// warp 0 loads A and its scales by TMA into a ring of stages, the last warp B and
// its; warp 6 copies the stages' scales to tensor memory, warp 1 issues the MMAs;
// warps 2-5, and 7-10 where two groups share 256 columns, store.
// Measured: 8192 tokens, 2 of 8 experts, 14336 x 4096 E4M3 590 us at full clocks (3.26
// PFLOP/s, the tensor pipe active 81 % of the time; a plain product of 16384 such rows
// 617), 650 to 690 among others under the power cap; the gradient of 4096 x 4096 188 us.
// Short contractions are bound by tile ends (4096 x 1024, 16 experts: 72 us, half the
// rate).  Few tokens: the weights' bytes (64 tokens, 16 experts of 4096 x 4096: 51 us, 86 %
// of the copy rate), fewer still a tile's own steps, 0.25 us each even from L2 (one tile,
// K = 14336: 31.1 us; 31.0 with a quarter of A's or B's rows loaded or without copies of
// scales, 24.8 with one MMA of four).
// Columns are a multiple of 128: the last of wider tiles can reach beyond C.  Its
// loads then bring the next expert's weights or zeros, and what they give is not
// stored.
// Order of tiles: expert by expert, down the rows first, so that an expert's
// weights stream through once while its rows stay in L2.
#include <algorithm>
#include <atomic>

#include "gemm.cuh"

namespace mxq {
namespace egemm {

using namespace gemm;

constexpr int PRODUCT = 0, WGRAD = 1;

struct Params {
  const int32_t* offsets;         // [E + 1] first rows of the experts' stretches
  const int32_t* block_expert;    // PRODUCT: expert of each `align` rows
  int experts, align, rows;
  int tiles_m, tiles_n, ntiles;   // of all of C (PRODUCT) or of one expert's C; ntiles in all
  int kblocks;                    // PRODUCT: steps of BKB bytes
  int kstep;                      // WGRAD: rows of a step
  int b_rows, b_steps;            // PRODUCT: rows and steps of B from expert to expert (one of them 0)
  int m_rows;                     // WGRAD: rows of C from expert to expert
  int kb4a, kb4b;                 // scale chunks per 128 rows of A and of B
  int out_fp32;
  int64_t ldc;
  void* c;
  uint32_t a_type, b_type;
  uint32_t tx_bytes;              // of a stage (all CTAs of a pair)
  int stall;                      // failure-detection test hook: 1 where CTA 0 never loads B of its first step
  int* status;
};

template <int KIND, int CTAS, int BN_>
struct Cfg {
  static constexpr bool FP4 = KIND == KIND_MXF4;
  static constexpr int TM = 128 * CTAS;
  static constexpr int BN = BN_;
  static constexpr int NACC = BN == 128 ? 2 : 1;
  static constexpr bool EDGE = BN > 128;                 // the last tile can reach beyond C
  // of four storing warps; FP4's pair has room for one staging buffer beside
  // six stages (117 us against 125 with five and two groups)
  static constexpr int GROUPS = BN == 128 || (CTAS == 2 && FP4) ? 1 : 2;
  static constexpr int COLS = BN / GROUPS;               // of a group
  static constexpr int STORE_WARPS = 4 * GROUPS;
  static constexpr int THREADS = 32 * (4 + STORE_WARPS);
  // stages of the ring: what fits beside the staging
  static constexpr int STAGES = CTAS == 1 && BN == 256 ? 4 : 6;
  static constexpr int NBUF = BN == 128 ? 2 : 1;         // staging buffers of a group
  static constexpr int OUT = GROUPS * NBUF * STG_BYTES;
  static constexpr int B_ROWS = BN / CTAS;               // of this CTA
  static constexpr int A_BYTES = BM * BKB;
  static constexpr int B_BYTES = B_ROWS * BKB;
  static constexpr int CHUNKS = FP4 ? 2 : 1;             // 512-byte scale chunks per 128 rows and step
  static constexpr int SFA_BYTES = 512 * CHUNKS;
  static constexpr int SFB_BYTES = BN / 128 * SFA_BYTES;
  static constexpr int TX_CTA = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int SFA_COLS = 4 * CHUNKS;
  static constexpr int SF_COLS = SFA_COLS * (1 + BN / 128);
  static constexpr int TMEM_COLS = 512;
  static_assert(NACC * BN + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");
  static constexpr int SMEM = STAGES * TX_CTA + OUT + 256 + 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Work of one tile: `steps` stages from step ak of A (rows m0 ..) and bk of B
// (rows br ..), into rows cm .. and columns n0 .. of C.  No steps: zeros.
struct Item {
  int m0, br, ak, bk, steps, cm, n0;
};

template <int MODE, int TM, int BN>
struct Items {
  const Params& p;
  int live = 0;                   // PRODUCT: tiles of rows that belong to an expert
  __device__ __forceinline__ explicit Items(const Params& p_) : p(p_) {
    if (MODE == PRODUCT) live = min(max(p.offsets[p.experts] / TM, 0), p.tiles_m) * p.tiles_n;
  }
  // Whatever the plan holds, a tile lies within the operands and C.
  __device__ __forceinline__ Item at(int tile) const {
    if constexpr (MODE == PRODUCT) {
      const int b = tile / p.tiles_n;
      if (tile >= live) return Item{0, 0, 0, 0, 0, b * TM, (tile - b * p.tiles_n) * BN};
      const int e = min(max(p.block_expert[static_cast<int64_t>(b) * TM / p.align], 0), p.experts - 1);
      const int first = min(max(p.offsets[e] / TM, 0), p.tiles_m - 1);
      const int blocks = min(max(p.offsets[e + 1] / TM - first, 1), p.tiles_m - first);
      const int local = max(tile - first * p.tiles_n, 0);
      const int n = min(local / blocks, p.tiles_n - 1), m = first + local % blocks;
      return Item{m * TM, e * p.b_rows + n * BN, 0, e * p.b_steps, p.kblocks, m * TM, n * BN};
    } else {
      const int per = p.tiles_m * p.tiles_n;
      const int e = tile / per, r = tile - e * per;
      const int n = r / p.tiles_m, m = r - n * p.tiles_m;
      const int end = p.rows / p.kstep;
      const int k0 = min(max(p.offsets[e] / p.kstep, 0), end), k1 = min(max(p.offsets[e + 1] / p.kstep, k0), end);
      return Item{m * TM, n * BN, k0, k0, k1 - k0, e * p.m_rows + m * TM, n * BN};
    }
  }
};

// ---------------------------------------------------------------- forms for one CTA and for a pair
template <int CTAS>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  if constexpr (CTAS == 2) tma_load_2d_pair(dst, map, bar, x, y);
  else tma_load_2d(dst, map, bar, x, y);
}
template <int CTAS>
__device__ __forceinline__ void commit_all(uint32_t bar) {
  if constexpr (CTAS == 2) tc_commit_pair_both(bar);
  else tc_commit(bar);
}
template <int CTAS>
__device__ __forceinline__ void commit_self(uint32_t bar) {
  if constexpr (CTAS == 2) tc_commit_pair_self(bar);
  else tc_commit(bar);
}
template <int CTAS>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t sdesc) {
  if constexpr (CTAS == 2) tc_cp_sf_pair(taddr, sdesc);
  else tc_cp_sf(taddr, sdesc);
}
template <int CTAS>
__device__ __forceinline__ void sync_all() {
  if constexpr (CTAS == 2) cluster_sync();
  else __syncthreads();
}

// 128 rows and COLS columns to C (rows cm .., columns n0 ..), by the four warps of
// barrier `bar`, through NBUF swizzled staging buffers and TMA stores.  read(c, v)
// gives this thread's row's columns 32 c .. 32 c + 63; release() follows the last
// read, before the stores.
template <int COLS, int NBUF, bool EDGE, typename Read, typename Release>
__device__ __forceinline__ void store_acc(int out_fp32, int row, bool leader, int bar, int& buf, uint8_t* sOut,
                                          const CUtensorMap* map_c, int cm, int n0, int cols, Read read,
                                          Release release) {
  const auto put = [&](const uint32_t* w, int at) {      // 64 bytes of every row, from column n0 + at on
    if (leader) bulk_wait_read_staging<NBUF>();
    named_bar(bar, 128);
    uint8_t* stg = sOut + buf * STG_BYTES;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int phys = j ^ ((row >> 1) & 3);             // 64-byte swizzle
      *reinterpret_cast<uint4*>(stg + row * 64 + phys * 16) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
    fence_proxy_async_smem();
    named_bar(bar, 128);
    if (leader && (!EDGE || n0 + at < cols)) {
      tma_store_2d(map_c, smem_u32(stg), n0 + at, cm);
      bulk_commit();
    }
    buf ^= NBUF - 1;
  };
  if (!out_fp32) {
    uint32_t pk[COLS / 2];
#pragma unroll
    for (int c = 0; c < COLS / 32; c += 2) {
      uint32_t v[64];
      read(c, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
        pk[c * 16 + j] = *reinterpret_cast<const uint32_t*>(&b2);
      }
    }
    release();
#pragma unroll
    for (int c = 0; c < COLS / 32; ++c) put(pk + c * 16, c * 32);
  } else if constexpr (COLS <= 128) {
    // all columns in registers first, too
    uint32_t v[COLS];
#pragma unroll
    for (int c = 0; c < COLS / 32; c += 2) read(c, v + c * 32);
    release();
#pragma unroll
    for (int c = 0; c < COLS / 16; ++c) put(v + c * 16, c * 16);
  } else {
    for (int c = 0; c < COLS / 32; c += 2) {
      uint32_t v[64];
      read(c, v);
      if (c + 2 == COLS / 32) release();
#pragma unroll
      for (int h = 0; h < 4; ++h) put(v + h * 16, c * 32 + h * 16);
    }
  }
}

// Columns 32 c .. 32 c + 63 of this thread's accumulator row.
__device__ __forceinline__ void read_acc(uint32_t lane_addr, int c, uint32_t* v) {
  tmem_ld32(lane_addr + c * 32, v);
  tmem_ld32(lane_addr + c * 32 + 32, v + 32);
  tmem_ld_wait();
}

// Zeros to this warp's 32 rows and COLS columns, row by row.
template <int COLS>
__device__ __forceinline__ void store_zeros(const Params& p, int q, int lane, int cm, int n0) {
  const int size = p.out_fp32 ? 4 : 2;
  uint8_t* row = static_cast<uint8_t*>(p.c) + (static_cast<int64_t>(cm + q * 32) * p.ldc + n0) * size;
  for (int r = 0; r < 32; ++r, row += p.ldc * size)
    for (int b = lane * 16; b < COLS * size; b += 512) *reinterpret_cast<uint4*>(row + b) = make_uint4(0, 0, 0, 0);
}

template <int KIND, int CTAS, int BN, int MODE>
__global__ void __launch_bounds__(Cfg<KIND, CTAS, BN>::THREADS, 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_sfa, const __grid_constant__ CUtensorMap map_sfb,
                   const __grid_constant__ CUtensorMap map_c, const Params p) {
  using C = Cfg<KIND, CTAS, BN>;
  using It = Items<MODE, C::TM, C::BN>;
  constexpr int STAGES = C::STAGES;
  constexpr int WARP_B = C::THREADS / 32 - 1;                      // the second producer
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * C::A_BYTES;
  uint8_t* sSFA = sB + STAGES * C::B_BYTES;
  uint8_t* sSFB = sSFA + STAGES * C::SFA_BYTES;
  uint8_t* sOut = sSFB + STAGES * C::SFB_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + C::OUT);     // used in rank 0
  uint64_t* empty = full + STAGES;
  uint64_t* sf_full = empty + STAGES;                              // rank 0: a slot's scales are in tensor memory
  uint64_t* acc_full = sf_full + STAGES;                           // [NACC]
  uint64_t* acc_empty = acc_full + 2;                              // [NACC], used in rank 0
  uint64_t* drain = acc_empty + 2;
  uint64_t* sf_drain = drain + 1;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sf_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sf_drain + 1) + 1;
  volatile int* epi_fail = reinterpret_cast<volatile int*>(sf_drain + 1) + 2;     // [2], of the groups

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0u;
  const int team = static_cast<int>(blockIdx.x) / CTAS, teams = static_cast<int>(gridDim.x) / CTAS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&sf_full[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&acc_full[b]), 1);
      mbar_init(smem_u32(&acc_empty[b]), 4 * C::GROUPS * CTAS);    // the storing warps of all CTAs
    }
    mbar_init(smem_u32(drain), 1);
    mbar_init(smem_u32(sf_drain), 1);
    *abort_flag = 0;
    epi_fail[0] = epi_fail[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    prefetch_tensormap(&map_sfa);
    prefetch_tensormap(&map_sfb);
    prefetch_tensormap(&map_c);
  }
  if (warp == 1) {
    if constexpr (CTAS == 2) tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
    else tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), C::TMEM_COLS);
  }
  tc_fence_before();
  sync_all<CTAS>();                // barriers initialised, tensor memory allocated
  tc_fence_after();
  grid_dep_launch();
  grid_dep_wait();                 // before any global-memory access
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_sf = tmem + C::NACC * C::BN;

  if (warp == 0 || warp == WARP_B) {
    // ------------------------------------------------------------ producers (all CTAs)
    // one thread for A and its scales, one for B and its: issuing is what a
    // step's loads cost
    if (lane == 0) {
      const bool a_side = warp == 0;
      const It items(p);
      // stage use counter; the test hook passes over a first step, whose phase never completes
      int u = !a_side && blockIdx.x == 0 ? p.stall : 0;
      int k0 = u;
      for (int tile = team; tile < p.ntiles && !*abort_flag; tile += teams) {
        const Item it = items.at(tile);
        const int ar = it.m0 + static_cast<int>(rank) * 128, br = it.br + static_cast<int>(rank) * C::B_ROWS;
        for (int k = k0; k < it.steps; ++k, ++u) {
          const int s = u % STAGES;
          if (!mbar_wait_suspend(smem_u32(&empty[s]), ((u / STAGES) & 1) ^ 1, p.status)) { *abort_flag = 1; break; }
          const uint32_t fb = CTAS == 2 ? cluster_map(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
          // scale maps: one 512-byte chunk per row
          if (a_side) {
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[s]), p.tx_bytes);
            load_tile<CTAS>(smem_u32(sA + s * C::A_BYTES), &map_a, fb, (it.ak + k) * BKB, ar);
            load_tile<CTAS>(smem_u32(sSFA + s * C::SFA_BYTES), &map_sfa, fb, 0, (ar / 128) * p.kb4a + (it.ak + k) * C::CHUNKS);
          } else {
            load_tile<CTAS>(smem_u32(sB + s * C::B_BYTES), &map_b, fb, (it.bk + k) * BKB, br);
#pragma unroll
            for (int h = 0; h < BN / 128; ++h)
              load_tile<CTAS>(smem_u32(sSFB + s * C::SFB_BYTES + h * C::SFA_BYTES), &map_sfb, fb, 0,
                              (it.br / 128 + h) * p.kb4b + (it.bk + k) * C::CHUNKS);
          }
        }
        if (it.steps) k0 = 0;
      }
      // no copy of any CTA is still landing when the kernel ends (the other
      // CTA of a pair is held at the final cluster barrier)
      if (rank == 0)
        for (int s = 0; s < STAGES && s < u; ++s) {
          const int last = u - 1 - (u - 1 - s) % STAGES;       // most recent use of stage s
          (void)mbar_wait_suspend(smem_u32(&full[s]), (last / STAGES) & 1, p.status);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (rank 0)
    if (lane == 0 && rank == 0) {
      const uint64_t a_desc0 = operand_desc(smem_u32(sA), 0), b_desc0 = operand_desc(smem_u32(sB), 0);
      uint32_t idesc[4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) idesc[kk] = instr_desc(p.a_type, p.b_type, C::BN, C::TM, C::FP4 ? (kk & 1) * 2 : kk);
      const It items(p);
      bool ok = true;
      int s = 0, ph = 0, t = 0;
      for (int tile = team; ok && tile < p.ntiles && !*abort_flag; tile += teams) {
        const Item it = items.at(tile);
        if (!it.steps) continue;
        const int ab = C::NACC == 2 ? (t & 1) : 0;            // accumulator and its use's parity
        const uint32_t aph = C::NACC == 2 ? ((t >> 1) & 1) : (t & 1);
        const uint32_t acc = tmem + ab * C::BN;
        ++t;
        if (!mbar_wait_suspend(smem_u32(&acc_empty[ab]), aph ^ 1, p.status)) { ok = false; break; }
        tc_fence_after();
        for (int k = 0; k < it.steps; ++k) {
          if (!mbar_wait_suspend(smem_u32(&sf_full[s]), ph, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sfa_t = tmem_sf + s * C::SF_COLS, sfb_t = sfa_t + C::SFA_COLS;
          const uint64_t ad = a_desc0 + ((s * C::A_BYTES) >> 4), bd = b_desc0 + ((s * C::B_BYTES) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t sfa = C::FP4 ? sfa_t + 4 * (kk >> 1) : sfa_t;
            const uint32_t sfb = C::FP4 ? sfb_t + 4 * (BN / 128) * (kk >> 1) : sfb_t;
            if constexpr (CTAS == 2) tc_mma_pair<KIND>(acc, ad + 2 * kk, bd + 2 * kk, idesc[kk], sfa, sfb, (k | kk) != 0);
            else tc_mma<KIND>(acc, ad + 2 * kk, bd + 2 * kk, idesc[kk], sfa, sfb, (k | kk) != 0);
          }
          commit_all<CTAS>(smem_u32(&empty[s]));               // stage free in all CTAs
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
        if (!ok) break;
        commit_all<CTAS>(smem_u32(&acc_full[ab]));
      }
      if (!ok) *abort_flag = 1;
      commit_self<CTAS>(smem_u32(drain));
      (void)mbar_wait_suspend(smem_u32(drain), 0, p.status);
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------ scale copies (rank 0)
    if (lane == 0 && rank == 0) {
      const uint64_t sfa_desc0 = smem_desc(smem_u32(sSFA), 0, 128, 0);
      const uint64_t sfb_desc0 = smem_desc(smem_u32(sSFB), 0, 128, 0);
      const It items(p);
      bool ok = true;
      int s = 0, ph = 0;
      for (int tile = team; ok && tile < p.ntiles && !*abort_flag; tile += teams) {
        const int steps = items.at(tile).steps;
        for (int k = 0; k < steps; ++k) {
          if (!mbar_wait_suspend(smem_u32(&full[s]), ph, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sfa_t = tmem_sf + s * C::SF_COLS;
#pragma unroll
          for (int c = 0; c < C::CHUNKS; ++c)
            cp_scales<CTAS>(sfa_t + 4 * c, sfa_desc0 + ((s * C::SFA_BYTES + c * 512) >> 4));
#pragma unroll
          for (int h = 0; h < BN / 128; ++h)
#pragma unroll
            for (int c = 0; c < C::CHUNKS; ++c)
              cp_scales<CTAS>(sfa_t + C::SFA_COLS + 4 * (BN / 128) * c + 4 * h,
                              sfb_desc0 + ((s * C::SFB_BYTES + h * C::SFA_BYTES + c * 512) >> 4));
          commit_self<CTAS>(smem_u32(&sf_full[s]));
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
      }
      if (!ok) *abort_flag = 1;
      commit_self<CTAS>(smem_u32(sf_drain));                   // no copy in flight at exit
      (void)mbar_wait_suspend(smem_u32(sf_drain), 0, p.status);
    }
  } else {
    // ------------------------------------------------------------ stores (all CTAs)
    const int q = warp & 3;                                    // lane quarter of tensor memory
    const int grp = warp >= 7 ? 1 : 0;                         // columns COLS grp ..
    const bool leader = (warp == 2 || warp == 7) && lane == 0;
    const int row = q * 32 + lane;
    uint8_t* const staging = sOut + grp * C::NBUF * STG_BYTES;
    const It items(p);
    int t = 0, buf = 0;
    for (int tile = team; tile < p.ntiles; tile += teams) {
      const Item it = items.at(tile);
      const int cm = it.cm + static_cast<int>(rank) * 128, n0 = it.n0 + grp * C::COLS;
      if (!it.steps) {
        // C ends at a multiple of 128 columns (a bound per lane instead: 8 tokens 39.9 us
        // against 35.4, 8192 tokens of 4096 x 1024 76.2 against 72.1)
        if (!C::EDGE || n0 + C::COLS <= p.ldc) store_zeros<C::COLS>(p, q, lane, cm, n0);
        else if (C::COLS > 128 && n0 < p.ldc) store_zeros<128>(p, q, lane, cm, n0);
        continue;
      }
      const int ab = C::NACC == 2 ? (t & 1) : 0;
      const uint32_t aph = C::NACC == 2 ? ((t >> 1) & 1) : (t & 1);
      const uint32_t lane_addr = tmem + ab * C::BN + grp * C::COLS + (static_cast<uint32_t>(q * 32) << 16);
      const auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(smem_u32(&acc_empty[ab]));
          else mbar_arrive_remote(cluster_map(smem_u32(&acc_empty[ab]), 0));
        }
      };
      // a group's warps decide together, so none is left alone at a named barrier
      if (!mbar_wait_suspend(smem_u32(&acc_full[ab]), aph, p.status)) epi_fail[grp] = 1;
      ++t;
      named_bar(1 + grp, 128);
      if (epi_fail[grp]) { *abort_flag = 1; break; }
      tc_fence_after();
      store_acc<C::COLS, C::NBUF, C::EDGE>(p.out_fp32, row, leader, 1 + grp, buf, staging, &map_c, cm, n0, static_cast<int>(p.ldc),
                                  [&](int c, uint32_t* v) { read_acc(lane_addr, c, v); }, release);
    }
    if (leader) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  sync_all<CTAS>();                // the tensor cores' work on either CTA's memory has finished
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CTAS == 2) tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace egemm
}  // namespace mxq

// ==================================================================== host
using namespace mxq_host;

namespace {

using mxq::egemm::Params;
using mxq::egemm::PRODUCT;
using mxq::egemm::WGRAD;

// One call: operands [a_rows][ka] and [b_rows][kb], C [c_rows][c_cols].
struct Args {
  const void* a_q;
  const uint8_t* a_s;
  const void* b_q;
  const uint8_t* b_s;
  int a_fmt, b_fmt;
  int64_t a_rows, ka, b_rows, kb, c_rows, c_cols;
  Params p;
  void* c;
};

// Teams of CTAS CTAs that run at once (cached per device); 0 on an error.
template <int CTAS, typename K>
int resident(K kern, int smem, int threads, std::atomic<int>& known) {
  int n = known.load(std::memory_order_relaxed);
  if (n) return n;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
  n = sm_count();
  if (CTAS == 2) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sm_count() / 2));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      return 0;
    }
  }
  known.store(n, std::memory_order_relaxed);
  return n;
}

template <int KIND, int CTAS, int BN, int MODE>
int launch(Args& g, cudaStream_t st) {
  using namespace mxq::gemm;
  using Cf = mxq::egemm::Cfg<KIND, CTAS, BN>;
  static std::atomic<int> known[64];
  auto kern = mxq::egemm::expert_gemm_kernel<KIND, CTAS, BN, MODE>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
  const int teams = resident<CTAS>(kern, Cf::SMEM, Cf::THREADS, known[dev]);
  if (!teams) return MXQ_ERR_CUDA;
  const int per = Cf::FP4 ? 2 : 1;                       // codes of a byte
  const bool a_u4 = !Cf::FP4 && g.a_fmt == MXQ_E2M1, b_u4 = !Cf::FP4 && g.b_fmt == MXQ_E2M1;
  CUtensorMap ma, mb, msa, msb, mc;
  const auto scales = [&](CUtensorMap* m, const uint8_t* s, int64_t rows, int64_t k) {
    return encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, s, 128, (rows / 128) * (k / 128), 512, 128, Cf::CHUNKS,
                     CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  const bool f32 = g.p.out_fp32;
  if (!encode_operand(&ma, g.a_q, a_u4, g.ka, g.ka / per, g.a_rows, 128) ||
      !encode_operand(&mb, g.b_q, b_u4, g.kb, g.kb / per, g.b_rows, Cf::B_ROWS) || !scales(&msa, g.a_s, g.a_rows, g.ka) ||
      !scales(&msb, g.b_s, g.b_rows, g.kb) ||
      !encode_2d(&mc, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.c, g.c_cols, g.c_rows,
                 g.c_cols * (f32 ? 4 : 2), f32 ? 16 : 32, BM, CU_TENSOR_MAP_SWIZZLE_64B))
    return MXQ_ERR_CUDA;
  Params& p = g.p;
  const int64_t m_rows = MODE == PRODUCT ? g.c_rows : p.m_rows;
  p.tiles_m = static_cast<int>(m_rows / Cf::TM);
  p.tiles_n = static_cast<int>((g.c_cols + Cf::BN - 1) / Cf::BN);
  const int64_t ntiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * (MODE == WGRAD ? p.experts : 1);
  if (ntiles > 0x7FFF0000) return MXQ_ERR_BAD_SHAPE;
  p.ntiles = static_cast<int>(ntiles);
  p.kstep = 128 * per;
  p.kblocks = static_cast<int>(g.ka / p.kstep);
  if (MODE == PRODUCT && p.b_steps) p.b_steps = p.kblocks;
  p.kb4a = static_cast<int>(g.ka / 128);
  p.kb4b = static_cast<int>(g.kb / 128);
  p.ldc = g.c_cols;
  p.c = g.c;
  p.a_type = mma_type(g.a_fmt, Cf::FP4);
  p.b_type = mma_type(g.b_fmt, Cf::FP4);
  p.tx_bytes = CTAS * (tx_bytes(Cf::A_BYTES, a_u4) + tx_bytes(Cf::B_BYTES, b_u4) + Cf::SFA_BYTES + Cf::SFB_BYTES);
  p.status = status_ptr();
  if (!p.status) return MXQ_ERR_CUDA;
  p.stall = take_test_stall(3);
  const dim3 grid(CTAS * std::min(p.ntiles, teams));
  if constexpr (CTAS == 2)
    return launch_pdl_cluster(kern, grid, dim3(Cf::THREADS), Cf::SMEM, st, 2, ma, mb, msa, msb, mc, p);
  else
    return launch_pdl(kern, grid, dim3(Cf::THREADS), Cf::SMEM, st, ma, mb, msa, msb, mc, p);
}

// Which tile.  Measured on 4096 x 4096 E4M3 weights of 16 experts unless said:
//  * pairs, where both sides allow it and at least every second SM gets a tile
//    (8192 tokens of 2, align 256: 196 us, 221 on 128 x 256 tiles; one token: 16
//    and 13 on 128 x 128), and for the weights' gradient from 1536 rows an expert
//    on (2048 rows, 8 experts: 194 and 212; 256 rows of 2048 x 2048: 72 and 55);
//  * 128 x 256, from two tiles an SM on (8192 tokens of 2, align 128: 210 us, 266
//    on 128 x 128; 512 tokens over 8 experts of 1024 x 1024: 7.6 and 6.0);
//  * both for an odd multiple of 128 columns only where the half of a last tile that
//    is wasted, and the longer tile ends, are small against the contraction (a step:
//    128 bytes of it; float32 outputs, whose tile ends take twice as long, count half:
//    K = 1024, 640 columns 19.3 us on pairs, 16.1 on 128 x 128).  6127 tokens of 2, 5
//    experts, K x columns, bf16, against 128 x 128:
//      pairs from 12 steps and 640 columns on (1536 x 640: 17.7 us and 18.9; 1024 x 640
//      14.3 and 14.0), from 8 and 1152 (1024 x 1920: 29.0 and 30.1; 512 x 1920 24.7
//      and 22.3); E2M1, with one storing group, from 16 and 640 (4096 x 640: 22.1 and
//      23.3; 2048 x 640 16.6 and 14.2), from 8 and 2048 (2048 x 4224: 58.5 and 62.7;
//      1024 x 4224 54.5 and 43.9);
//      128 x 256 from 8 steps and 896 columns on (1024 x 1920: 27.5 and 29.4; 512 x 1920
//      22.9 and 21.5), from 2048 whatever the steps (512 x 4224: 40.5 and 42.5);
//    gradients: pairs from 640 on (8192 tokens of 2, 8 experts, 2048 x 896: 33.2 and
//    37.3; of small ones the rounds of tiles decide, 1024 x 640 22.8 and 20.3), 128 x 256 from
//    2048 on (4224 x 3200: 25.1 and 26.2; 1024 x 1152: 26.7 and 23.1).
template <int KIND, int MODE>
int choose(Args& g, bool pair, cudaStream_t st) {
  const int64_t sms = sm_count(), rows = MODE == PRODUCT ? g.c_rows : g.p.m_rows * static_cast<int64_t>(g.p.experts);
  const int64_t wide = (g.c_cols + 255) / 256;                    // columns of 256-wide tiles
  const bool even = g.c_cols % 256 == 0;
  // columns from which odd multiples of 128 take pairs, and 128 x 256
  int64_t odd_pair = 640, odd_wide = 2048;
  if (MODE == PRODUCT) {
    constexpr bool FP4 = KIND == mxq::gemm::KIND_MXF4;
    const int64_t steps = g.ka / (FP4 ? 256 : 128) / (g.p.out_fp32 ? 2 : 1);
    odd_pair = steps >= (FP4 ? 16 : 12) ? 640 : steps < 8 ? INT64_MAX : FP4 ? 2048 : 1152;
    odd_wide = steps >= 8 ? 896 : 2048;
  }
  if (pair && (even || g.c_cols >= odd_pair) && 2 * (rows / 256 * wide) >= sms && (MODE == PRODUCT || g.p.rows >= 1536ll * g.p.experts))
    return launch<KIND, 2, 256, MODE>(g, st);
  if ((even || g.c_cols >= odd_wide) && rows / 128 * wide >= 2 * sms) return launch<KIND, 1, 256, MODE>(g, st);
  return launch<KIND, 1, 128, MODE>(g, st);
}

template <int MODE>
int run(Args& g, bool pair, void* stream) {
  using namespace mxq::gemm;
  const auto st = static_cast<cudaStream_t>(stream);
  if (g.a_fmt == MXQ_E2M1 && g.b_fmt == MXQ_E2M1) return choose<KIND_MXF4, MODE>(g, pair, st);
  return choose<KIND_MXF8, MODE>(g, pair, st);
}

// Checks that both calls share.
int check(const void* a_q, const uint8_t* a_s, int a_fmt, const void* b_q, const uint8_t* b_s, int b_fmt, int64_t rows,
          int64_t N, int64_t K, int experts, int align, const int32_t* offsets, const void* c, int out_fp32) {
  if (!valid_fmt(a_fmt) || !valid_fmt(b_fmt) || (out_fp32 != 0 && out_fp32 != 1)) return MXQ_ERR_BAD_ARG;
  if (align != 128 && align != 256) return MXQ_ERR_BAD_ARG;
  if (rows < 0 || rows % align || rows > 0x7FFF0000 || experts < 1 || experts > 1024 || N < 128 || N % 128 || K < 128 || K % 128)
    return MXQ_ERR_BAD_SHAPE;
  // coordinates of rows, columns and scale chunks are 32 bits
  if (N > 0x7FFF0000 / experts || K > 0x7FFF0000 / experts) return MXQ_ERR_BAD_SHAPE;
  if (N / 128 * experts * (K / 128) > 0x7FFF0000 || rows / 128 * (std::max(N, K) / 128) > 0x7FFF0000) return MXQ_ERR_BAD_SHAPE;
  if (!offsets || (rows && (!a_q || !a_s || !b_q || !b_s))) return MXQ_ERR_BAD_ARG;
  if (!aligned16(a_q) || !aligned16(a_s) || !aligned16(b_q) || !aligned16(b_s) || !aligned16(c) ||
      (reinterpret_cast<uintptr_t>(offsets) & 3u))
    return MXQ_ERR_MISALIGNED;
  const bool fp4 = a_fmt == MXQ_E2M1 && b_fmt == MXQ_E2M1;
  if (!fp4 && ((a_fmt == MXQ_E2M1 && !aligned32(a_q)) || (b_fmt == MXQ_E2M1 && !aligned32(b_q)))) return MXQ_ERR_MISALIGNED;
  return MXQ_OK;
}

}  // namespace

extern "C" int mxq_expert_gemm(const void* a_q, const uint8_t* a_s, int a_fmt, const void* b_q, const uint8_t* b_s,
                               int b_fmt, int64_t rows, int64_t N, int64_t K, int experts, int align,
                               const int32_t* offsets, const int32_t* block_expert, int b_along_k, void* c,
                               int out_fp32, void* stream) {
  if (const int rc = check(a_q, a_s, a_fmt, b_q, b_s, b_fmt, rows, N, K, experts, align, offsets, c, out_fp32)) return rc;
  if (b_along_k != 0 && b_along_k != 1) return MXQ_ERR_BAD_ARG;
  const bool fp4 = a_fmt == MXQ_E2M1 && b_fmt == MXQ_E2M1;
  if (fp4 && K % 256) return MXQ_ERR_BAD_SHAPE;
  if (rows && (!block_expert || !c)) return MXQ_ERR_BAD_ARG;
  if (reinterpret_cast<uintptr_t>(block_expert) & 3u) return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  if (!rows) return MXQ_OK;
  Args g{};
  g.a_q = a_q, g.a_s = a_s, g.b_q = b_q, g.b_s = b_s, g.a_fmt = a_fmt, g.b_fmt = b_fmt;
  g.a_rows = rows, g.ka = K;
  g.b_rows = b_along_k ? N : experts * N, g.kb = b_along_k ? experts * K : K;
  g.c = c, g.c_rows = rows, g.c_cols = N;
  g.p.offsets = offsets, g.p.block_expert = block_expert;
  g.p.experts = experts, g.p.align = align, g.p.rows = static_cast<int>(rows);
  g.p.b_rows = b_along_k ? 0 : static_cast<int>(N);
  g.p.b_steps = b_along_k;
  g.p.out_fp32 = out_fp32;
  return run<PRODUCT>(g, align == 256, stream);
}

extern "C" int mxq_expert_wgrad(const void* a_q, const uint8_t* a_s, int a_fmt, const void* b_q, const uint8_t* b_s,
                                int b_fmt, int64_t rows, int64_t N, int64_t K, int experts, int align,
                                const int32_t* offsets, void* c, int out_fp32, void* stream) {
  if (const int rc = check(a_q, a_s, a_fmt, b_q, b_s, b_fmt, rows, N, K, experts, align, offsets, c, out_fp32)) return rc;
  const bool fp4 = a_fmt == MXQ_E2M1 && b_fmt == MXQ_E2M1;
  if (fp4 && align != 256) return MXQ_ERR_BAD_SHAPE;
  if (!c) return MXQ_ERR_BAD_ARG;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  if (!rows)
    return cudaMemsetAsync(c, 0, static_cast<size_t>(experts) * N * K * (out_fp32 ? 4 : 2), static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
  Args g{};
  g.a_q = a_q, g.a_s = a_s, g.b_q = b_q, g.b_s = b_s, g.a_fmt = a_fmt, g.b_fmt = b_fmt;
  g.a_rows = N, g.ka = rows, g.b_rows = K, g.kb = rows;
  g.c = c, g.c_rows = experts * N, g.c_cols = K;
  g.p.offsets = offsets;
  g.p.experts = experts, g.p.align = align, g.p.rows = static_cast<int>(rows);
  g.p.m_rows = static_cast<int>(N);
  g.p.out_fp32 = out_fp32;
  return run<WGRAD>(g, N % 256 == 0, stream);
}
