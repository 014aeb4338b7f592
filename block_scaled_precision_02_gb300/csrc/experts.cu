// Tokens sorted by expert and back, with weights and gradients:
//   sort      e[s] -> a row for every slot s (a token's j-th choice), the rows
//             of an expert in one stretch, in the slots' order
//   gather    rows[r] = x[slot(r) / top], 0 in padding
//   combine   y[t] = sum_j w[t][j] rows[row(t, j)]
//   backward  drows[row(t, j)] = w[t][j] dy[t], 0 in padding
//             dw[t][j] = sum_c dy[t][c] rows[row(t, j)][c]
//
// The sort is a counting sort of small integers: latency and launches bound
// it (3.3 us for one token, 6.7 for 8192 of 2).  The others move rows and are
// bound by HBM; of 8192 x 4096 bf16 with 2 of 16 experts, against the bytes that
// each must move once at the measured copy rate: gather 37 us (87 % of it with its
// padding), combine 32 (94 %), its backward pass 64 (85 %; one expert a token 96 %).
// Rows without a common alignment wait for loads: a gather of 8192 x 4095 takes 48 us
// (67 %), its schedulers issuing in 34 % of the cycles, 70 % of the warps' time a wait for
// global memory; the backward pass of 3648 x 1021, 4 slots, 17 us (61 %) with 61 % and 52 %.
#include <algorithm>
#include <atomic>

#include "rowops.cuh"

namespace mxq {
namespace {

using namespace mxq_host;

constexpr int kMaxExperts = 1024;

// ---------------------------------------------------------------- sort
constexpr int SORT_WARPS = 16, SORT_T = 32 * SORT_WARPS;
constexpr int SORT_SLOTS = 2048;          // slots of a CTA, until there are SORT_CLUSTER or SORT_CTAS of them
// Up to 32768 slots one cluster of CTAs sorts, which read each other's counts
// from shared memory: a launch less, 8 us of the host's path (8192 tokens, 2 of
// 16 experts: 6.1 us on the device either way).  Beyond, SORT_CTAS count first
// and place in a second launch (8192 tokens, 8 of 64: 7.8 us against 15.8).
constexpr int SORT_CLUSTER = 8, SORT_CTAS = 128;
constexpr int64_t CLUSTER_SLOTS = 32768;

struct SortArgs {
  const void* experts;
  int64_t slots, per;                     // per: slots of a CTA
  int64_t rows;
  int e64, E, align;
  int32_t *offsets, *counts, *slot_row, *row_slot, *block_expert;
  int32_t* part;                          // [CTAs][E] counts, where they come from a launch of their own
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
// that depends on nothing but the slots.  CLUSTER: the grid is one cluster.
template <bool CLUSTER>
__global__ void __launch_bounds__(SORT_T) expert_place_kernel(const SortArgs a) {
  extern __shared__ int sm[];
  int* const off = sm;                            // [E + 1] starts of the experts' stretches
  int* const cnt = off + a.E + 1;                 // [E] slots of each expert
  int* const own = cnt + a.E;                     // [E] this CTA's
  int* const wcnt = own + a.E;                    // [SORT_WARPS][E]
  __shared__ int warp_sums[SORT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < SORT_WARPS * a.E; i += SORT_T) wcnt[i] = 0;
  __syncthreads();
  grid_dep_wait();

  const int64_t lo = blockIdx.x * a.per, hi = min(a.slots, lo + a.per);
  const int64_t each = (a.per + SORT_WARPS * 32 - 1) / (SORT_WARPS * 32) * 32;
  const int64_t wlo = min(hi, lo + warp * each), whi = min(hi, wlo + each);
  int* const mine = wcnt + warp * a.E;
#pragma unroll 8
  for (int64_t s = wlo + lane; s < whi; s += 32) {
    const int e = expert_of(a, s);
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();

  if constexpr (CLUSTER) {
    for (int e = threadIdx.x; e < a.E; e += SORT_T) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < SORT_WARPS; ++w) n += wcnt[w * a.E + e];
      own[e] = n;
    }
    cluster_sync();
  }
  // this CTA's counts by warp become the counts of earlier CTAs and warps
  for (int e = threadIdx.x; e < a.E; e += SORT_T) {
    int before = 0, all = 0;
    if (gridDim.x > 1) {
#pragma unroll 8
      for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
        int n;
        if constexpr (CLUSTER)
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(cluster_map(smem_u32(own + e), b)) : "memory");
        else
          n = __ldcg(a.part + static_cast<int64_t>(b) * a.E + e);
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
  if constexpr (CLUSTER) cluster_arrive();        // this CTA has read its peers' counts
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

  int next = wlo + lane < whi ? expert_of(a, wlo + lane) : -1;
  for (int64_t s0 = wlo; s0 < whi; s0 += 32) {
    const int64_t s = s0 + lane;
    const int e = next;
    next = s + 32 < whi ? expert_of(a, s + 32) : -1;     // on its way while this one is placed
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
  if constexpr (CLUSTER) cluster_wait();          // its own counts stay until every peer has read them
}

// ---------------------------------------------------------------- rows
// The kernels below stay on the GPU and walk over tokens (and, for zeros, over
// blocks of rows); the plan's entries of the next step are read while the
// current step's rows are on their way, so that one latency is seen per step
// instead of two.
//
// A row is taken in vectors of VE elements, the width of 16 bytes of its type.
// ANY: rows may start anywhere.  The vectors then lie on what is written: its
// first elements up to a 16-byte boundary (`head`) and its last ones go
// singly, and what is read is put together from the two aligned words that
// hold it.
constexpr int ROW_T = 256, ROW_WARPS = ROW_T / 32;
constexpr int U = 4;                      // vectors of a lane in flight per row

struct RowArgs {
  const void* src;                        // gather: x; combine: rows; backward: rows
  const void* dy;                         // backward
  void* out;                              // rows; y; drows
  float* dw;
  const int32_t *slot_row, *offsets, *counts;
  const void* w;                          // or nullptr: 1
  int w_f32;
  int64_t tokens, rows, cols, ld, ld_dy;
  int top, experts;
  int shared;                             // "tokens" that share a row of x or dy: top where slots go apart, else 1
  int lanes;                              // of a warp to a row: 4 .. 32
  int pieces;                             // stretches of lanes * U vectors to a row
};

__device__ __forceinline__ float weight_of(const RowArgs& a, int64_t slot) {
  if (!a.w) return 1.f;
  return a.w_f32 ? static_cast<const float*>(a.w)[slot] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.w)[slot]);
}

// Row of a slot, or -1 where it has none.
__device__ __forceinline__ int row_of(const RowArgs& a, int64_t slot) {
  const int r = a.slot_row[slot];
  return r < a.rows ? r : -1;
}

// VE elements from anywhere: the aligned 16-byte words that hold the first and
// the last of them, shifted together.  Both words hold elements of the vector,
// so they lie where the row does.
template <typename T, int VE>
__device__ __forceinline__ void load_any(Vec<T, VE>& v, const T* p) {
  static_assert(Vec<T, VE>::BYTES == 16 || Vec<T, VE>::BYTES == 8, "a vector of one or half a word");
  constexpr int W = Vec<T, VE>::W;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const int shift = static_cast<int>(at & 15);
  const uint4* const q = reinterpret_cast<const uint4*>(at - shift);
  const uint4 lo = q[0], hi = q[shift + 4 * W > 16 ? 1 : 0];
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const int bits = 8 * (shift & 3);
#pragma unroll
  for (int i = 0; i < W; ++i) v.w[i] = __funnelshift_r(w[i], w[i + 1], bits);
}

template <bool ANY, typename T, int VE>
__device__ __forceinline__ void load_vec(Vec<T, VE>& v, const T* p) {
  if constexpr (ANY) load_any<T, VE>(v, p);
  else v.load(p);
}

// Elements before the first boundary of a vector of VE elements of T.
template <typename T, int VE>
__device__ __forceinline__ int head_of(const T* p, int64_t cols) {
  constexpr int B = VE * static_cast<int>(sizeof(T)) > 16 ? 16 : VE * static_cast<int>(sizeof(T));
  const int h = static_cast<int>((0 - reinterpret_cast<uintptr_t>(p)) & (B - 1)) / static_cast<int>(sizeof(T));
  return static_cast<int>(min(static_cast<int64_t>(h), cols));
}

// Walks of a grid's warps over the tokens' stretches: a warp's lanes fall into
// groups of a.lanes, each of which takes a stretch of a token of its own.  A
// place is advanced without a division.
struct Walk {
  int64_t rounds;                         // steps of this warp
  int64_t row0;                           // its first token (that of its first group)
  int piece0, group, lane, per;           // per: groups of a warp
  int64_t row_step;
  int piece_step, pieces;
  __device__ __forceinline__ Walk(const RowArgs& a) {
    const int l = threadIdx.x & 31;
    per = 32 / a.lanes;
    group = l / a.lanes;
    lane = l - group * a.lanes;
    pieces = a.pieces;
    const int64_t step = blockIdx.x * static_cast<int64_t>(ROW_WARPS) + (threadIdx.x >> 5);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * ROW_WARPS, steps = (a.tokens + per - 1) / per * pieces;
    rounds = step < steps ? (steps - step + stride - 1) / stride : 0;
    row0 = step / pieces * per;
    piece0 = static_cast<int>(step % pieces);
    row_step = stride / pieces * per;
    piece_step = static_cast<int>(stride % pieces);
  }
};

struct Place {
  int64_t row;                            // of the warp's first group
  int piece;
  __device__ __forceinline__ explicit Place(const Walk& w) : row(w.row0), piece(w.piece0) {}
  __device__ __forceinline__ void next(const Walk& w) {
    row += w.row_step;
    piece += w.piece_step;
    if (piece >= w.pieces) piece -= w.pieces, row += w.per;
  }
};

// Zeros to `n` rows from row r0 on, by CTA `part` of `parts`: one stretch of memory.
template <typename T, int VE, bool ANY, int THREADS = ROW_T>
__device__ __forceinline__ void zero_rows(const RowArgs& a, int64_t r0, int64_t n, int64_t part, int64_t parts) {
  if (n <= 0) return;
  T* const p = static_cast<T*>(a.out) + r0 * a.cols;
  const int64_t len = n * a.cols;
  const int head = ANY ? head_of<T, VE>(p, len) : 0;
  const int64_t nv = (len - head) / VE;
  Vec<T, VE> z;
  z.fill(0);
  for (int64_t i = part * THREADS + threadIdx.x; i < nv; i += parts * THREADS) z.store(p + head + i * VE);
  if (ANY && part == 0) {
    Vec<T, 1> o;
    o.fill(0);
    if (static_cast<int>(threadIdx.x) < head) o.store(p + threadIdx.x);
    const int64_t c = head + nv * VE + threadIdx.x;
    if (c < len) o.store(p + c);
  }
}

// Zeros to the rows that hold no slot: what is left of every expert's stretch
// (the experts dealt out over the CTAs, several CTAs to one where there are
// enough), and the rows behind the last.
template <typename T, int VE, bool ANY, int THREADS = ROW_T>
__device__ __forceinline__ void zero_padding(const RowArgs& a) {
  const int teams = min(a.experts, static_cast<int>(gridDim.x)), parts = gridDim.x / teams;
  const int team = blockIdx.x % teams, part = blockIdx.x / teams;
  if (part < parts)
    for (int e = team; e < a.experts; e += teams) {
      const int64_t end = min(static_cast<int64_t>(max(a.offsets[e + 1], 0)), a.rows);
      const int64_t from = min(max(static_cast<int64_t>(a.offsets[e]) + a.counts[e], int64_t(0)), end);
      zero_rows<T, VE, ANY, THREADS>(a, from, end - from, part, parts);
    }
  const int64_t last = min(static_cast<int64_t>(max(a.offsets[a.experts], 0)), a.rows);
  zero_rows<T, VE, ANY, THREADS>(a, last, a.rows - last, blockIdx.x, gridDim.x);
}

// Aligned rows: a token's stretch is read once and written to the row of each of its
// slots (read once a row instead, many tokens of several experts would come twice from
// HBM).  Where slots go apart, and in rows without a common alignment, whose vectors
// lie on what is written, every slot reads its token again.
template <typename T, int VE, bool ANY>
__global__ void __launch_bounds__(ROW_T) gather_kernel(const RowArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  zero_padding<T, VE, ANY>(a);                           // nothing waits for these stores
  const Walk w(a);
  T* const out = static_cast<T*>(a.out);
  Place at(w);
  for (int64_t n = 0; n < w.rounds; ++n, at.next(w)) {
    const int64_t t = at.row + w.group, v0 = static_cast<int64_t>(at.piece) * a.lanes * U + w.lane;
    if (t >= a.tokens) continue;
    const T* const x = static_cast<const T*>(a.src) + (a.shared > 1 ? t / a.shared : t) * a.ld;
    if constexpr (!ANY) {
      Vec<T, VE> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t c = (v0 + u * a.lanes) * VE;
        if (c < a.cols) v[u].load(x + c);
      }
      for (int j = 0; j < a.top; ++j) {
        const int64_t r = row_of(a, t * a.top + j);
        if (r < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t c = (v0 + u * a.lanes) * VE;
          if (c < a.cols) v[u].store(out + r * a.cols + c);
        }
      }
    } else {
      for (int j = 0; j < a.top; ++j) {
        const int64_t r = row_of(a, t * a.top + j);
        if (r < 0) continue;
        T* const o = out + r * a.cols;
        const int head = head_of<T, VE>(o, a.cols);
        const int64_t nv = (a.cols - head) / VE;
        Vec<T, VE> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * a.lanes < nv) load_any<T, VE>(v[u], x + head + (v0 + u * a.lanes) * VE);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * a.lanes < nv) v[u].store(o + head + (v0 + u * a.lanes) * VE);
        if (v0 < a.lanes)                                // the row's first stretch: its single elements
          for (int64_t i = w.lane; i < a.cols - nv * VE; i += a.lanes) {
            const int64_t c = i < head ? i : i + nv * VE;
            o[c] = x[c];
          }
      }
    }
  }
}

// ---------------------------------------------------------------- combine
// Few tokens, or rows that have no vectors: a warp takes a stretch of a token
// and reads its slots' rows straight into registers, two slots at a time where they
// are vectors (one token of 8 slots, 4096 bf16 columns: 4.3 us, one at a time 6.8), one
// where they are elements (515 x 2049 of 3 slots 3.5 us, two at a time 3.8; 2000 x
// 1021 of 8 9.1 and 9.9).
template <typename T, typename TY, int VE>
__global__ void __launch_bounds__(ROW_T) combine_direct_kernel(const RowArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  const int64_t t = item / static_cast<uint32_t>(a.pieces);
  const int64_t c0 = static_cast<int64_t>(item % static_cast<uint32_t>(a.pieces)) * (32 * U * VE) + lane * VE;
  if (t >= a.tokens) return;
  float acc[U][VE];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[u][i] = 0.f;
#pragma unroll (VE == 1 ? 1 : 2)
  for (int j = 0; j < a.top; ++j) {
    const int64_t slot = t * a.top + j, r = row_of(a, slot);
    if (r < 0) continue;
    const float g = weight_of(a, slot);
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
      for (int i = 0; i < VE; ++i) acc[u][i] = fmaf(g, v[u].get(i), acc[u][i]);
  }
  TY* const y = static_cast<TY*>(a.out) + t * a.cols;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t c = c0 + u * 32 * VE;
    if (c < a.cols) store_vec<TY, VE>(y + c, acc[u]);
  }
}

// Many tokens: a warp's work is one sequence of units: a stretch of the row of one slot, the
// slots of a token in their order.  Every lane copies its own vectors of a unit
// to shared memory S units ahead (asynchronously: registers would hold less
// than half of what has to be in flight), and the unit's row number and weight
// S units before that.  S = 4 and two CTAs: 128 KiB of rows in flight an SM, 32 us
// for 8192 x 4096; three CTAs of S = 3 spill (51), S = 6 is 38.
constexpr int S = 4;

constexpr int combine_words(bool any) { return 32 * U + (any ? 1 : 0); }    // of a warp's unit
constexpr int combine_smem(bool any) { return S * ROW_WARPS * combine_words(any) * 16 + 2 * S * ROW_T * 8; }

template <typename T, typename TY, int VE, bool ANY>
__global__ void __launch_bounds__(ROW_T, 2) combine_kernel(const RowArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int WORDS = combine_words(ANY);
  uint2* const plan = reinterpret_cast<uint2*>(ring + S * ROW_WARPS * WORDS * 16) + threadIdx.x;    // [2 S][ROW_T]
  const Walk w(a);
  const int lane = threadIdx.x & 31;
  uint8_t* const mine = ring + (threadIdx.x >> 5) * (WORDS * 16) + (ANY ? 0 : lane * 16);
  const uint32_t to = smem_u32(mine) + (ANY ? lane * 16 : 0), plan_to = smem_u32(plan);
  const T* const src = static_cast<const T*>(a.src);
  const int vecs = a.lanes * U, cols = static_cast<int>(a.cols);
  grid_dep_launch();
  grid_dep_wait();
  // a token's row of y: elements before its vectors, and how many vectors
  const auto head_at = [&](int64_t t) { return ANY ? head_of<TY, VE>(static_cast<TY*>(a.out) + t * cols, cols) : 0; };

  float acc[U][VE];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VE; ++i) acc[u][i] = 0.f;
  Place use(w), copy(w), look(w);
  int use_j = 0, copy_j = 0, look_j = 0;
  int64_t use_n = w.rounds, copy_n = w.rounds, look_n = w.rounds;     // steps left
  int slot = 0, at = 0;                                  // of the ring (S), of the plan (2 S)
  for (int n = -2 * S; use_n > 0; n += n < 0) {
    cp_async_wait<S - 1>();
    if constexpr (ANY) __syncwarp();                     // lanes read each other's words
    int r = -1;
    float g = 1.f;
    Vec<T, VE> x[U];
    if (n >= 0 && use.row + w.group < a.tokens) {
      const uint2 q = plan[at * ROW_T];
      r = static_cast<int>(q.x) < a.rows ? static_cast<int>(q.x) : -1;
      if (a.w) {
        const bool high = !a.w_f32 && (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.w) >> 1) +
                                       static_cast<uint32_t>((use.row + w.group) * a.top + use_j)) & 1;
        g = a.w_f32 ? __uint_as_float(q.y) : high ? bf16hi(q.y) : bf16lo(q.y);
      }
      if (r >= 0) {
        uint8_t* const from = mine + slot * (ROW_WARPS * WORDS * 16);
        if constexpr (!ANY) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint4 p = *reinterpret_cast<const uint4*>(from + u * 512);
            x[u].w[0] = p.x, x[u].w[1] = p.y, x[u].w[2] = p.z, x[u].w[3] = p.w;
          }
        } else {
          const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(src + r * a.ld + head_at(use.row)) & 15);
#pragma unroll
          for (int u = 0; u < U; ++u) load_any<T, VE>(x[u], reinterpret_cast<const T*>(from + (u * 32 + lane) * 16 + shift));
        }
      }
    }
    if constexpr (ANY) __syncwarp();
    if (n >= -S && copy_n > 0) {
      const int64_t t = copy.row + w.group;
      if (t < a.tokens) {
        const int cr = static_cast<int>(plan[(at >= S ? at - S : at + S) * ROW_T].x);
        if (cr >= 0 && cr < a.rows) {
          const uint32_t dst = to + slot * (ROW_WARPS * WORDS * 16);
          const T* const row = src + cr * a.ld;
          if constexpr (!ANY) {
            const int c = (copy.piece * vecs + w.lane) * VE, step = a.lanes * VE;
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (c + u * step < cols) cp_async16(dst + u * 512, row + c + u * step);
          } else {
            // the aligned words that hold any of the stretch's elements
            const int head = head_at(t);
            const uintptr_t p = (reinterpret_cast<uintptr_t>(row + head + copy.piece * (32 * U * VE)) & ~uintptr_t(15)) + lane * 16;
            const uintptr_t end = reinterpret_cast<uintptr_t>(row + head + (cols - head) / VE * VE);
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (p + u * 512 < end) cp_async16(dst + u * 512, reinterpret_cast<const void*>(p + u * 512));
            if (lane == 0 && p + U * 512 < end) cp_async16(dst + U * 512, reinterpret_cast<const void*>(p + U * 512));
          }
        }
      }
      if (++copy_j == a.top) copy_j = 0, --copy_n, copy.next(w);
    }
    if (look_n > 0) {
      const int64_t t = look.row + w.group;
      if (t < a.tokens) {
        const int64_t id = t * a.top + look_j;
        cp_async4(plan_to + at * (ROW_T * 8), a.slot_row + id);
        // a bf16 weight comes with its neighbour
        if (a.w)
          cp_async4(plan_to + at * (ROW_T * 8) + 4,
                    reinterpret_cast<const void*>((reinterpret_cast<uintptr_t>(a.w) + (a.w_f32 ? 4 : 2) * id) & ~uintptr_t(3)));
      }
      if (++look_j == a.top) look_j = 0, --look_n, look.next(w);
    }
    cp_async_commit();
    if (n >= -S) slot = slot + 1 == S ? 0 : slot + 1;
    at = at + 1 == 2 * S ? 0 : at + 1;
    if (n < 0) continue;
    if (r >= 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[u][i] = fmaf(g, x[u].get(i), acc[u][i]);
    }
    if (++use_j < a.top) continue;
    const int64_t t = use.row + w.group;
    if (t < a.tokens) {
      const int head = head_at(t), nv = (cols - head) / VE;
      const int v = use.piece * vecs + w.lane;
      TY* const y = static_cast<TY*>(a.out) + t * cols + head + static_cast<int64_t>(v) * VE;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v + u * a.lanes < nv) store_vec<TY, VE>(y + u * a.lanes * VE, acc[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < VE; ++i) acc[u][i] = 0.f;
    use_j = 0, --use_n;
    use.next(w);
  }
  cp_async_wait<0>();

  if constexpr (ANY) {
    // the single elements before and behind a row's vectors, 16 lanes to a token
    const int64_t team = (blockIdx.x * static_cast<int64_t>(ROW_T) + threadIdx.x) >> 4, teams = static_cast<int64_t>(gridDim.x) * (ROW_T / 16);
    const int l = threadIdx.x & 15;
    for (int64_t t = team; t < a.tokens; t += teams) {
      const int head = head_at(t), nv = (cols - head) / VE;
      const int c = l < head ? l : l + nv * VE;
      if (c >= cols) continue;
      float sum[1] = {0.f};
#pragma unroll 4
      for (int j = 0; j < a.top; ++j) {
        const int r = row_of(a, t * a.top + j);
        if (r >= 0) {
          float e[1];
          load_elems<T, 1>(static_cast<const T*>(a.src) + r * a.ld + c, e);
          sum[0] = fmaf(weight_of(a, t * a.top + j), e[0], sum[0]);
        }
      }
      store_vec<TY, 1>(static_cast<TY*>(a.out) + t * cols + c, sum);
    }
  }
}

constexpr int BWD_T = 256, BWD_WARPS = BWD_T / 32;

// Few tokens, rows without a common alignment, longer ones than the ring takes, dy
// of another type: G of a CTA's BWD_WARPS warps take a token; dy's NV vectors of a
// lane stay in registers while the rows of its slots pass, two at a time.  Longer
// rows, and those without alignment, go round in stretches, whose parts of the sums
// are added up.  Four CTAs an SM, although some forms then spill: what counts is rows
// in flight (8192 x 4096 float32 rows of 2 slots, bf16 dy: 109 us, at three CTAs 120, at
// two 146; 8192 x 14336 bf16 204, 222, 264; but bf16 rows with float32 dy, 8192 x 4096: 88,
// 77, 87, and 8192 x 1024 22, 25, 32).  Without
// alignment and G = 8 six (3047 x 14335, 4 slots: 152 us, at four 173), else four
// (1021 bf16 columns: 18.4 us, at five 20.1).
template <typename T, typename TY, int VE, int G, int NV, bool ANY>
__global__ void __launch_bounds__(BWD_T, ANY && G == 8 ? 6 : 4) combine_bwd_kernel(const RowArgs a) {
  constexpr int TEAMS = BWD_WARPS / G;
  __shared__ float red[2][TEAMS][2][G];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / G, part = warp % G;
  const int idx = part * 32 + lane;                      // thread of the team
  T* const out = static_cast<T*>(a.out);
  int buf = 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * TEAMS;
  int r[2];
  float g[2];
  const auto fetch = [&](int64_t t, int j) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      r[k] = -1, g[k] = 0.f;
      if (t < a.tokens && j + k < a.top) {
        r[k] = row_of(a, t * a.top + j + k);
        if (r[k] >= 0) g[k] = weight_of(a, t * a.top + j + k);
      }
    }
  };
  int64_t t = blockIdx.x * static_cast<int64_t>(TEAMS) + team;
  fetch(t, 0);
  for (; t < a.tokens; t += stride) {
    const TY* const dy = static_cast<const TY*>(a.dy) + (a.shared > 1 ? t / a.shared : t) * a.ld_dy;
    float d[NV][VE];
    const bool whole = !ANY && a.cols <= G * 32 * NV * VE;       // dy is read once
    if (whole) {
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int64_t c = (static_cast<int64_t>(n) * G * 32 + idx) * VE;
        if (c < a.cols) load_elems<TY, VE>(dy + c, d[n]);
      }
    }
    for (int j = 0; j < a.top; j += 2) {
      const int rr[2] = {r[0], r[1]};
      const float gg[2] = {g[0], g[1]};
      if (j + 2 < a.top) fetch(t, j + 2);
      else fetch(t + stride, 0);
      float dot[2] = {0.f, 0.f};
      if (whole) {
        Vec<T, VE> x[2][NV];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int64_t c = (static_cast<int64_t>(n) * G * 32 + idx) * VE;
            if (rr[k] >= 0 && c < a.cols) x[k][n].load(static_cast<const T*>(a.src) + rr[k] * a.ld + c);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (rr[k] < 0) continue;
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int64_t c = (static_cast<int64_t>(n) * G * 32 + idx) * VE;
            if (c < a.cols) {
              float q[VE], o[VE];
#pragma unroll
              for (int i = 0; i < VE; ++i) q[i] = d[n][i] * x[k][n].get(i), o[i] = d[n][i] * gg[k];
              dot[k] += tree_sum(q);
              store_vec<T, VE>(out + rr[k] * a.cols + c, o);
            }
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (rr[k] < 0) continue;
          const T* const x = static_cast<const T*>(a.src) + rr[k] * a.ld;
          T* const o = out + rr[k] * a.cols;
          const int head = ANY ? head_of<T, VE>(o, a.cols) : 0;
          const int64_t nv = (a.cols - head) / VE;
          for (int64_t v0 = idx; v0 < nv; v0 += G * 32 * NV) {
            Vec<T, VE> xv[NV];
            Vec<TY, (VE * sizeof(TY) > 16 ? VE / 2 : VE)> dv[NV][VE * sizeof(TY) > 16 ? 2 : 1];
            constexpr int H = VE * sizeof(TY) > 16 ? VE / 2 : VE, P = VE / H;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
              const int64_t v = v0 + n * G * 32, c = head + v * VE;
              if (v < nv) {
                load_vec<ANY>(xv[n], x + c);
#pragma unroll
                for (int h = 0; h < P; ++h) load_vec<ANY>(dv[n][h], dy + c + h * H);
              }
            }
#pragma unroll
            for (int n = 0; n < NV; ++n) {
              const int64_t v = v0 + n * G * 32, c = head + v * VE;
              if (v < nv) {
                float q[VE], p[VE];
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                  const float dd = dv[n][i / H].get(i % H);
                  q[i] = dd * xv[n].get(i), p[i] = dd * gg[k];
                }
                dot[k] += tree_sum(q);
                store_vec<T, VE>(o + c, p);
              }
            }
          }
          if constexpr (ANY) {
            for (int64_t i = idx; i < a.cols - nv * VE; i += G * 32) {
              const int64_t c = i < head ? i : i + nv * VE;
              float e[1], f[1];
              load_elems<T, 1>(x + c, e);
              load_elems<TY, 1>(dy + c, f);
              dot[k] = fmaf(e[0], f[0], dot[k]);
              f[0] *= gg[k];
              store_vec<T, 1>(o + c, f);
            }
          }
        }
      }
      dot[0] = warp_sum(dot[0]);
      dot[1] = warp_sum(dot[1]);
      if constexpr (G == 1) {
        if (lane < 2 && j + lane < a.top) a.dw[t * a.top + j + lane] = lane ? dot[1] : dot[0];
      } else {
        if (lane == 0) red[buf][team][0][part] = dot[0], red[buf][team][1][part] = dot[1];
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(G * 32) : "memory");
        if (idx < 2 && j + idx < a.top) {
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < G; ++k) sum += red[buf][team][idx][k];
          a.dw[t * a.top + j + idx] = sum;
        }
        buf ^= 1;                                        // the next sums go elsewhere: one barrier a round is enough
      }
    }
  }
  zero_padding<T, VE, ANY, BWD_T>(a);
}

// Many tokens of aligned rows, dy of the rows' type: the ring of combine.  G warps
// take a token, whose units are dy and then the rows of its slots; dy's vectors
// stay in registers.  Sums of up to DOTS slots meet in shared memory.
constexpr int DOTS = 8;
constexpr int bwd_ring_smem() { return S * ROW_T * U * 16 + 2 * S * ROW_T * 8; }

template <typename T, int VE, int G>
__global__ void __launch_bounds__(ROW_T, 2) combine_bwd_ring_kernel(const RowArgs a) {
  constexpr int TEAMS = ROW_WARPS / G;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][TEAMS][DOTS][G];
  uint8_t* const mine = ring + (threadIdx.x >> 5) * (U * 512) + (threadIdx.x & 31) * 16;
  uint2* const plan = reinterpret_cast<uint2*>(ring + S * ROW_T * U * 16) + threadIdx.x;          // [2 S][ROW_T]
  const uint32_t to = smem_u32(mine), plan_to = smem_u32(plan);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / G, part = warp % G;
  const int idx = part * 32 + lane, cols = static_cast<int>(a.cols);
  const int c0 = idx * VE;
  constexpr int STEP = G * 32 * VE;
  const T* const src = static_cast<const T*>(a.src);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * TEAMS;
  grid_dep_launch();
  grid_dep_wait();

  // units of a token: -1 is dy, then its slots
  int64_t use_t = blockIdx.x * static_cast<int64_t>(TEAMS) + team, copy_t = use_t, look_t = use_t;
  int use_j = -1, copy_j = -1, look_j = -1;
  int slot = 0, at = 0, buf = 0;
  Vec<T, VE> d[U];
#pragma unroll
  for (int u = 0; u < U; ++u) d[u].fill(0);
  for (int n = -2 * S; use_t < a.tokens; n += n < 0) {
    cp_async_wait<S - 1>();
    int r = -1;
    float g = 0.f;
    Vec<T, VE> x[U];
    if (n >= 0) {
      const uint8_t* const from = mine + slot * (ROW_T * U * 16);
      if (use_j < 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) d[u].load(reinterpret_cast<const T*>(from + u * 512));
      } else {
        const uint2 q = plan[at * ROW_T];
        r = static_cast<int>(q.x) < a.rows ? static_cast<int>(q.x) : -1;
        const bool high = (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.w) >> 1) + static_cast<uint32_t>(use_t * a.top + use_j)) & 1;
        g = a.w_f32 ? __uint_as_float(q.y) : high ? bf16hi(q.y) : bf16lo(q.y);
#pragma unroll
        for (int u = 0; u < U; ++u) x[u].load(reinterpret_cast<const T*>(from + u * 512));
      }
    }
    if (n >= -S && copy_t < a.tokens) {
      const uint32_t dst = to + slot * (ROW_T * U * 16);
      const int cr = copy_j < 0 ? -1 : static_cast<int>(plan[(at >= S ? at - S : at + S) * ROW_T].x);
      if (copy_j < 0 || (cr >= 0 && cr < a.rows)) {
        const T* const row = copy_j < 0 ? static_cast<const T*>(a.dy) + copy_t * a.ld_dy : src + cr * a.ld;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c0 + u * STEP < cols) cp_async16(dst + u * 512, row + c0 + u * STEP);
      }
      if (++copy_j == a.top) copy_j = -1, copy_t += stride;
    }
    if (look_t < a.tokens) {
      if (look_j >= 0) {
        const int64_t id = look_t * a.top + look_j;
        cp_async4(plan_to + at * (ROW_T * 8), a.slot_row + id);
        cp_async4(plan_to + at * (ROW_T * 8) + 4,
                  reinterpret_cast<const void*>((reinterpret_cast<uintptr_t>(a.w) + (a.w_f32 ? 4 : 2) * id) & ~uintptr_t(3)));
      }
      if (++look_j == a.top) look_j = -1, look_t += stride;
    }
    cp_async_commit();
    if (n >= -S) slot = slot + 1 == S ? 0 : slot + 1;
    at = at + 1 == 2 * S ? 0 : at + 1;
    if (n < 0) continue;
    if (use_j >= 0) {
      float dot = 0.f;
      if (r >= 0) {
        T* const o = static_cast<T*>(a.out) + static_cast<int64_t>(r) * cols + c0;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (c0 + u * STEP < cols) {
            float q[VE], w[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) q[i] = d[u].get(i) * x[u].get(i), w[i] = d[u].get(i) * g;
            dot += tree_sum(q);
            store_vec<T, VE>(o + u * STEP, w);
          }
      }
      dot = warp_sum(dot);
      const int64_t id = use_t * a.top + use_j;
      if constexpr (G == 1) {
        if (lane == 0) a.dw[id] = dot;
      } else {
        const int k = use_j & (DOTS - 1);
        if (lane == 0) red[buf][team][k][part] = dot;
        if (k == DOTS - 1 || use_j == a.top - 1) {
          asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(G * 32) : "memory");
          if (idx <= k) {
            float sum = 0.f;
#pragma unroll
            for (int p = 0; p < G; ++p) sum += red[buf][team][idx][p];
            a.dw[id - k + idx] = sum;
          }
          buf ^= 1;
        }
      }
    }
    if (++use_j == a.top) use_j = -1, use_t += stride;
  }
  cp_async_wait<0>();
  zero_padding<T, VE, false>(a);
}

// ---------------------------------------------------------------- host
bool plan_sizes(int64_t tokens, int64_t top, int64_t rows) {
  return tokens >= 0 && top >= 1 && rows >= 0 && top <= kMaxCols && tokens <= kMaxCols / top && rows <= kMaxCols;
}

// Rows that start at 16-byte boundaries and hold whole words.
bool wide(const void* p, int64_t ld, int type, int64_t cols) {
  const int s = type_size(type);
  return aligned16(p) && (ld * s) % 16 == 0 && (cols * s) % 16 == 0;
}

// CTAs that stay on the GPU: as many as fit, or as there is work for.
template <typename K>
int stay(K kern, int64_t want, std::atomic<int>* known, unsigned* grid, int smem = 0, int threads = ROW_T) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
  int n = known[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (smem && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return MXQ_ERR_CUDA;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess || n < 1) return MXQ_ERR_CUDA;
    n *= sm_count();
    known[dev].store(n, std::memory_order_relaxed);
  }
  *grid = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(want, n)));
  return MXQ_OK;
}

// Lanes of a row: the power of two that its vectors fill with U each, 4 .. 32.
void set_lanes(RowArgs& a, int ve) {
  a.lanes = 4;
  while (a.lanes < 32 && a.lanes * U * ve < a.cols) a.lanes *= 2;
  a.pieces = static_cast<int>((a.cols + a.lanes * U * ve - 1) / (a.lanes * U * ve));
}

int64_t walk_ctas(const RowArgs& a) {
  const int per = 32 / a.lanes;
  return ((a.tokens + per - 1) / per * a.pieces + ROW_WARPS - 1) / ROW_WARPS;
}

// Warps of tokens per SM up to which a warp takes slots instead of tokens, each of
// which reads its token again: a token's rows are then written by as many warps, not
// one after another.  1024 bf16 columns, 4 slots: 1216 tokens (8 warps) 4.5 us against
// 6.0, 2432 6.0 and 7.2, 4864 8.8 and 8.2.  1021 columns, which are read again for
// every row either way, but in more instructions: 1216 tokens 6.9 and 8.4, 2432 9.3
// and 8.9, 9728 40 and 24.
constexpr int gather_apart(bool any) { return any ? 12 : 24; }

template <typename T, int VE, bool ANY>
int run_gather(RowArgs a, cudaStream_t st) {
  static std::atomic<int> known[64];
  set_lanes(a, VE);
  unsigned grid = 0;
  a.shared = 1;
  if (a.top > 1 && walk_ctas(a) * ROW_WARPS < gather_apart(ANY) * static_cast<int64_t>(sm_count()))
    a.shared = a.top, a.tokens *= a.top, a.top = 1;
  const int64_t want = std::max<int64_t>(walk_ctas(a), (a.rows * a.cols + ROW_T * VE - 1) / (ROW_T * VE));
  if (const int rc = stay(gather_kernel<T, VE, ANY>, want, known, &grid)) return rc;
  return launch_pdl(gather_kernel<T, VE, ANY>, dim3(grid), dim3(ROW_T), 0, st, a);
}

template <typename T, typename TY, int VE, bool ANY>
int run_combine_ring(RowArgs a, cudaStream_t st) {
  static std::atomic<int> known[64];
  set_lanes(a, VE);
  if (ANY) a.lanes = 32, a.pieces = static_cast<int>((a.cols + 32 * U * VE - 1) / (32 * U * VE));      // a warp's words lie side by side
  unsigned grid = 0;
  constexpr int smem = combine_smem(ANY);
  if (const int rc = stay(combine_kernel<T, TY, VE, ANY>, walk_ctas(a), known, &grid, smem)) return rc;
  return launch_pdl(combine_kernel<T, TY, VE, ANY>, dim3(grid), dim3(ROW_T), smem, st, a);
}

template <typename T, typename TY, int VE>
int run_combine_direct(RowArgs a, cudaStream_t st) {
  a.pieces = static_cast<int>((a.cols + 32 * U * VE - 1) / (32 * U * VE));
  const int64_t grid = (a.tokens * a.pieces + ROW_WARPS - 1) / ROW_WARPS;
  if (grid > 0x0FFFFFFF) return MXQ_ERR_BAD_SHAPE;       // 2^31 warps, a terabyte of y
  return launch_pdl(combine_direct_kernel<T, TY, VE>, dim3(static_cast<unsigned>(grid)), dim3(ROW_T), 0, st, a);
}

// The ring pays from about 2^21 elements of y on (8192 x 4096 bf16: 32 us, read
// directly 47; 515 x 2049 float32: 8.9 and 3.5).  Rows without a common alignment
// take it as bf16 of DIRECT_COLS columns or more (8192 x 4095, one slot: 27 us, element by
// element 49), as their single elements go round apart (16384 x 77, 4 slots: 40
// and 6); float32 ones are read element by element as fast (5238 x 1023, 5
// slots: 23 us, 31 in the ring).
constexpr int64_t RING_ELEMS = 1 << 21, DIRECT_COLS = 512;

template <typename T, typename TY, int VE>
int run_combine(const RowArgs& a, bool vectors, cudaStream_t st) {
  const bool many = a.tokens * a.cols >= RING_ELEMS;
  if (vectors) return many ? run_combine_ring<T, TY, VE, false>(a, st) : run_combine_direct<T, TY, VE>(a, st);
  if constexpr (sizeof(T) == 2)
    if (many && a.cols >= DIRECT_COLS) return run_combine_ring<T, TY, VE, true>(a, st);
  return run_combine_direct<T, TY, 1>(a, st);
}

// Warps of tokens per SM up to which each slot is a team's own work, which reads its
// token's dy again: so few tokens leave part of the GPU idle and a token's slots wait
// for one another.  Aligned rows, 4096 bf16 columns: 250 tokens of 2 slots 4.7 us and
// 5.2 with a team to a token, of 8 slots 11.1 and 10.3; 325 of 2: 5.8 and 5.4.  Others
// cost more instructions, and win until 32 warps fill an SM: 1021 bf16 columns, 4
// slots, 1216 tokens 6.2 and 14.7, 3648 (24 warps) 16.7 and 19.2, 4864 21.7 and 20.5;
// 2049 float32, 456 tokens 10.0 and 12.0, 608 13.4 and 13.9.
constexpr int apart(bool any) { return any ? 28 : 12; }

template <typename T, typename TY, int VE, int G, int NV, bool ANY>
int launch_backward(RowArgs a, cudaStream_t st) {
  static std::atomic<int> known[64];
  unsigned grid = 0;
  a.shared = 1;
  if (a.top > 1 && a.tokens * G < apart(ANY) * sm_count()) a.shared = a.top, a.tokens *= a.top, a.top = 1;
  const int64_t want = std::max<int64_t>((a.tokens * G + BWD_WARPS - 1) / BWD_WARPS,
                                         (a.rows * a.cols + BWD_T * VE - 1) / (BWD_T * VE));
  if (const int rc = stay(combine_bwd_kernel<T, TY, VE, G, NV, ANY>, want, known, &grid, 0, BWD_T)) return rc;
  return launch_pdl(combine_bwd_kernel<T, TY, VE, G, NV, ANY>, dim3(grid), dim3(BWD_T), 0, st, a);
}

// Elements of dy from which the ring pays (16384 x 1024 bf16, 4 slots: 51 us, 63
// read directly; 8192 x 4096, one slot: 33 and 48; 600 x 4096: 7.6 and 6.5).
constexpr int64_t BWD_RING = 1 << 22;

template <typename T, int VE, int G>
int launch_backward_ring(const RowArgs& a, cudaStream_t st) {
  static std::atomic<int> known[64];
  unsigned grid = 0;
  if (const int rc = stay(combine_bwd_ring_kernel<T, VE, G>, (a.tokens * G + ROW_WARPS - 1) / ROW_WARPS, known, &grid, bwd_ring_smem()))
    return rc;
  return launch_pdl(combine_bwd_ring_kernel<T, VE, G>, dim3(grid), dim3(ROW_T), bwd_ring_smem(), st, a);
}

// As many warps to a token as its vectors fill, eight at most.  Rows without
// alignment pay for every vector in instructions and take fewer warps, one vector a
// lane: 3047 tokens of 4 slots, 501 float32 columns (125 vectors) 17.0 us with one
// warp, 18.6 with two; 695 (174) 24.8 with two, 27.6 with four; 1021 (255) 29.7 with four,
// 32.8 with two, 36.4 with eight; 2049 (512) 47.9 with eight, 52.7 with four.
template <typename T, typename TY, int VE>
int run_backward(const RowArgs& a, bool vectors, cudaStream_t st) {
  if (!vectors) {
    if (a.cols <= 128 * VE) return launch_backward<T, TY, VE, 1, 1, true>(a, st);
    if (a.cols <= 192 * VE) return launch_backward<T, TY, VE, 2, 1, true>(a, st);
    if (a.cols <= 384 * VE) return launch_backward<T, TY, VE, 4, 1, true>(a, st);
    return launch_backward<T, TY, VE, 8, 1, true>(a, st);
  }
  if constexpr (sizeof(T) == sizeof(TY))
    if (a.tokens * a.cols >= BWD_RING && a.cols > 64 * VE && a.cols <= 1024 * VE) {
      if (a.cols <= 128 * VE) return launch_backward_ring<T, VE, 1>(a, st);
      if (a.cols <= 256 * VE) return launch_backward_ring<T, VE, 2>(a, st);
      if (a.cols <= 512 * VE) return launch_backward_ring<T, VE, 4>(a, st);
      return launch_backward_ring<T, VE, 8>(a, st);
    }
  if (a.cols <= 32 * VE) return launch_backward<T, TY, VE, 1, 1, false>(a, st);
  if (a.cols <= 64 * VE) return launch_backward<T, TY, VE, 2, 1, false>(a, st);
  if (a.cols <= 128 * VE) return launch_backward<T, TY, VE, 4, 1, false>(a, st);
  if (a.cols <= 256 * VE) return launch_backward<T, TY, VE, 8, 1, false>(a, st);
  return launch_backward<T, TY, VE, 8, 2, false>(a, st);
}

int64_t sort_ctas(int64_t slots) {
  const int most = slots <= CLUSTER_SLOTS ? SORT_CLUSTER : SORT_CTAS;
  return std::max<int64_t>(1, std::min<int64_t>(most, (slots + SORT_SLOTS - 1) / SORT_SLOTS));
}

constexpr int sort_smem(int experts) { return ((3 + SORT_WARPS) * experts + 1) * static_cast<int>(sizeof(int)); }

template <bool CLUSTER>
int run_place(const SortArgs& a, int64_t n, cudaStream_t st) {
  static std::atomic<bool> set[64];
  auto kern = expert_place_kernel<CLUSTER>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
  if (!set[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, sort_smem(kMaxExperts)) != cudaSuccess)
      return MXQ_ERR_CUDA;
    set[dev].store(true, std::memory_order_relaxed);
  }
  const dim3 grid(static_cast<unsigned>(n));
  if (CLUSTER) return launch_pdl_cluster(kern, grid, dim3(SORT_T), sort_smem(a.E), st, static_cast<int>(n), a);
  return launch_pdl(kern, grid, dim3(SORT_T), sort_smem(a.E), st, a);
}

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
  *bytes = slots <= CLUSTER_SLOTS ? 16 : static_cast<size_t>(sort_ctas(slots)) * experts * sizeof(int32_t);
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
  if (n == 1) return run_place<false>(a, n, st);
  if (slots <= CLUSTER_SLOTS) return run_place<true>(a, n, st);
  if (const int rc = launch_pdl(expert_count_kernel, dim3(static_cast<unsigned>(n)), dim3(SORT_T), num_experts * sizeof(int), st, a))
    return rc;
  return run_place<false>(a, n, st);
}

extern "C" int mxq_expert_gather(const void* x, int64_t tokens, int64_t cols, int64_t ld, int x_type,
                                 const int32_t* slot_row, int64_t top, const int32_t* offsets, const int32_t* counts,
                                 int experts, int64_t rows, void* out, void* stream) {
  if (!valid_type(x_type)) return MXQ_ERR_BAD_ARG;
  if (!plan_sizes(tokens, top, rows) || cols < 1 || cols > kMaxCols || ld < cols) return MXQ_ERR_BAD_SHAPE;
  if (experts < 1 || experts > kMaxExperts) return MXQ_ERR_BAD_SHAPE;
  if ((tokens && (!x || !slot_row)) || (rows && (!offsets || !counts || !out))) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(x, type_size(x_type)) || !aligned_to(out, type_size(x_type)) || !aligned_to(slot_row, 4) ||
      !aligned_to(offsets, 4) || !aligned_to(counts, 4))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  RowArgs a{};
  a.src = x, a.out = out, a.slot_row = slot_row, a.offsets = offsets, a.counts = counts, a.experts = experts;
  a.tokens = tokens, a.rows = rows, a.cols = cols, a.ld = ld, a.top = static_cast<int>(top);
  const auto st = static_cast<cudaStream_t>(stream);
  const bool v = wide(x, ld, x_type, cols) && aligned16(out);
  if (!rows) return MXQ_OK;
  if (x_type == MXQ_F32) return v ? run_gather<float, 4, false>(a, st) : run_gather<float, 4, true>(a, st);
  return v ? run_gather<__nv_bfloat16, 8, false>(a, st) : run_gather<__nv_bfloat16, 8, true>(a, st);
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
  if (!tokens) return MXQ_OK;
  using bf = __nv_bfloat16;
  if (type == MXQ_F32) {
    if (y_type == MXQ_F32) return run_combine<float, float, 4>(a, v, st);
    return run_combine<float, bf, 4>(a, v, st);
  }
  if (y_type == MXQ_F32) return run_combine<bf, float, 8>(a, v, st);
  return run_combine<bf, bf, 8>(a, v, st);
}

extern "C" int mxq_expert_combine_backward(const void* dy, int64_t ld_dy, int dy_type, const void* rows_in, int64_t ld,
                                           int type, int64_t rows, int64_t cols, const int32_t* slot_row,
                                           int64_t tokens, int64_t top, const int32_t* offsets, const int32_t* counts,
                                           int experts, const void* weights, int w_type, void* drows, float* dweights,
                                           void* stream) {
  if (!valid_type(type) || !valid_type(dy_type) || !valid_type(w_type)) return MXQ_ERR_BAD_ARG;
  if (!plan_sizes(tokens, top, rows) || cols < 1 || cols > kMaxCols || ld < cols || ld_dy < cols) return MXQ_ERR_BAD_SHAPE;
  if (experts < 1 || experts > kMaxExperts) return MXQ_ERR_BAD_SHAPE;
  if ((rows && (!rows_in || !drows)) || (tokens && (!dy || !slot_row || !weights || !dweights))) return MXQ_ERR_BAD_ARG;
  if ((rows || tokens) && (!offsets || !counts)) return MXQ_ERR_BAD_ARG;     // every launch reads the stretches' ends
  if (!aligned_to(rows_in, type_size(type)) || !aligned_to(dy, type_size(dy_type)) || !aligned_to(drows, type_size(type)) ||
      !aligned_to(slot_row, 4) || !aligned_to(offsets, 4) || !aligned_to(counts, 4) || !aligned_to(weights, type_size(w_type)) ||
      !aligned_to(dweights, 4))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  RowArgs a{};
  a.src = rows_in, a.dy = dy, a.out = drows, a.dw = dweights, a.slot_row = slot_row;
  a.offsets = offsets, a.counts = counts, a.experts = experts;
  a.w = weights, a.w_f32 = w_type == MXQ_F32;
  a.tokens = tokens, a.rows = rows, a.cols = cols, a.ld = ld, a.ld_dy = ld_dy, a.top = static_cast<int>(top);
  const auto st = static_cast<cudaStream_t>(stream);
  // a vector is 16 bytes of the rows; dy's side of it is 8, 16 or 32
  const bool v = wide(rows_in, ld, type, cols) && aligned16(drows) && wide(dy, ld_dy, dy_type, cols);
  if (!tokens && !rows) return MXQ_OK;
  using bf = __nv_bfloat16;
  if (type == MXQ_F32) {
    if (dy_type == MXQ_F32) return run_backward<float, float, 4>(a, v, st);
    return run_backward<float, bf, 4>(a, v, st);
  }
  if (dy_type == MXQ_F32) return run_backward<bf, float, 8>(a, v, st);
  return run_backward<bf, bf, 8>(a, v, st);
}
