// Clipped policy loss with a KL term, from logits: the loss, the tokens'
// log-probabilities and the gradient of the logits in one pass over them.
//
//   lp = z_a - lse(z),  r = exp(lp - old),  u = min(r A, clip(r, 1-lo, 1+hi) A)
//   k3 = exp(ref - lp) - (ref - lp) - 1,    l = -u + beta k3,  loss = sum w l
//   dl/dlp = -A r [r A <= clip(r) A] + beta (1 - exp(ref - lp))
//   dz_v = scale w dl/dlp ([v == a] - exp(z_v - lse))
//
// A row's exponentials stay in the registers of one CTA, or of a cluster of
// up to eight CTAs, so the logits are read once and the gradient is written
// once: HBM bounds it (one exponential per element).  A warp takes its own
// maximum m_w and keeps e_v = exp(z_v - m_w); the pairs (m_w, sum e_v) of all
// warps go to every CTA of the cluster, and p_v = e_v exp(m_w - lse) needs no
// second exponential.
#include <algorithm>
#include <atomic>

#include "rowops.cuh"

namespace mxq {
namespace {

constexpr int MAX_SLABS = 8;             // CTAs of a cluster (the portable limit)
constexpr int MAX_E = 32;                // elements of a thread (register kernel)
constexpr float kLog2e = 1.4426950408889634f;

struct LossArgs {
  const void* z;
  int64_t ld_z;
  void* g;                               // NULL: no gradient
  int64_t ld_g;
  const void* targets;
  int targets64;
  const float *old_lp, *adv, *weights, *ref_lp;
  float lo, hi, beta, scale;
  int tokens, vocab;
  float* logp;
  float* terms;                          // [tokens] w * l
  float* loss;
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// exp(v - m) for m a maximum: the difference first, so that its rounding is
// relative to the distance from the maximum and not to the logits' size.
__device__ __forceinline__ float exp_rel(float v, float m) { return ex2((v - m) * kLog2e); }

// exp(v - m) of a pair, m and log2(e) splat.
__device__ __forceinline__ void exp_pair(float a, float b, float2 mm, float2 l2e, float& x, float& y) {
  float p, q;
  halves(mul2(sub2(pair(a, b), mm), l2e), p, q);
  x = ex2(p);
  y = ex2(q);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Elements [e0, e0 + VE) of a row of V, where only those in [0, V) exist; the
// others are -inf.  Whole vectors go as one aligned load.
template <typename T, int VE>
__device__ __forceinline__ void load_edge(const T* row, int e0, int V, float (&v)[VE]) {
  if (e0 >= 0 && e0 + VE <= V) {
    Vec<T, VE> r;
    r.load(row + e0);
#pragma unroll
    for (int j = 0; j < VE; ++j) v[j] = r.get(j);
  } else {
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      v[j] = -INFINITY;
      if (e0 + j >= 0 && e0 + j < V) {
        Vec<T, 1> r;
        r.load(row + e0 + j);
        v[j] = r.get(0);
      }
    }
  }
}

template <typename T, int VE>
__device__ __forceinline__ void store_edge(T* row, int e0, int V, const float (&v)[VE]) {
  if (e0 >= 0 && e0 + VE <= V) store_vec<T, VE>(row + e0, v);
  else
#pragma unroll
    for (int j = 0; j < VE; ++j)
      if (e0 + j >= 0 && e0 + j < V) {
        const float one[1] = {v[j]};
        store_vec<T, 1>(row + e0 + j, one);
      }
}

// The 16-byte words of a row, less a ragged last one, into L2.
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* row, int V) {
  const uintptr_t begin = reinterpret_cast<uintptr_t>(row) & ~uintptr_t(15);
  const uintptr_t end = reinterpret_cast<uintptr_t>(row + V) & ~uintptr_t(15);
  if (end > begin)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(begin), "r"(static_cast<unsigned>(end - begin)) : "memory");
}

// What a token brings besides its logits: loaded together, and ahead of use,
// because each is a trip to memory of its own.
struct TokenIn {
  float w, adv, old_lp, ref_lp;
  int64_t target;
};

__device__ __forceinline__ TokenIn token_in(const LossArgs& a, int64_t row) {
  TokenIn t{0.f, 0.f, 0.f, 0.f, -1};
  if (row < a.tokens) {
    t.w = a.weights[row];
    t.adv = a.adv[row];
    t.old_lp = a.old_lp[row];
    if (a.beta != 0.f) t.ref_lp = a.ref_lp[row];
    t.target = a.targets64 ? static_cast<const int64_t*>(a.targets)[row]
                           : static_cast<int64_t>(static_cast<const int*>(a.targets)[row]);
  }
  return t;
}

// Loss term and its slope dl/dlp of one token.
__device__ __forceinline__ void token_loss(const LossArgs& a, const TokenIn& t, float lp, float& l, float& slope) {
  const float x = lp - t.old_lp;
  // no advantage, no term: also where the ratio is finite but beyond float32
  const float r = t.adv == 0.f && x < INFINITY ? 0.f : expf(x);
  const float ra = r * t.adv, ca = fminf(fmaxf(r, 1.f - a.lo), 1.f + a.hi) * t.adv;
  const float nan = __int_as_float(0x7FFFFFFF);
  l = ra <= ca ? -ra : (ca < ra ? -ca : nan);
  slope = ra <= ca ? -ra : (ca < ra ? 0.f : nan);
  if (a.beta != 0.f) {
    const float d = t.ref_lp - lp;
    const float e = expm1f(d);
    l += a.beta * (e - d);
    slope -= a.beta * e;
  }
}

// The loss: the tokens' terms, added by one CTA that follows the rows'
// kernels.  It starts early and waits for them: 5 x 32001 takes 4.9 us in a
// graph, 6.4 with the sum in the last row's CTA and 10.2 with a fill of that
// CTA's ticket before each call (a ticket kept at zero would have to outlive
// the call).  A thread adds its own terms in their order as an unevaluated pair
// (the rounding error of each float32 addition is exactly (a - (s - v)) +
// (b - v) with s = a + b, v = s - a, and is kept apart), the threads' sums go
// up a fixed tree in float64.  All-float64 additions at two lanes a cycle took
// longer than the loads.
__global__ void __launch_bounds__(1024) loss_sum_kernel(const LossArgs a) {
  __shared__ double sums[32];
  grid_dep_wait();
  grid_dep_launch();
  float hi = 0.f, lo = 0.f;
#pragma unroll 8
  for (int i = threadIdx.x; i < a.tokens; i += blockDim.x) {
    const float t = __ldcg(a.terms + i);
    const float sum = __fadd_rn(hi, t), v = __fsub_rn(sum, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(sum, v)), __fsub_rn(t, v)));
    hi = sum;
  }
  // an infinite or NaN sum has no error term
  double s = fabsf(hi) < INFINITY ? static_cast<double>(hi) + static_cast<double>(lo) : static_cast<double>(hi);
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  s = threadIdx.x < (blockDim.x >> 5) ? sums[threadIdx.x] : 0.0;
  s = warp_sum(s);
  if (threadIdx.x == 0) a.loss[0] = static_cast<float>(s);
}

// CTAs of the register kernels that an SM holds, by registers: 42 a thread for
// 16 elements or fewer, 56 or 64 for 32 (64 where single elements move).
template <int VE, int NV, int TPB>
constexpr int policy_ctas() {
  return TPB == 32 ? 4 : (VE * NV <= 16 ? 1536 : VE > 1 && TPB % 3 == 0 ? 1152 : 1024) / TPB;
}

// `slabs` CTAs (one cluster) per token; a thread holds NV vectors of VE
// elements.  Vectors start at the row's first 16-byte boundary at or before
// its first element, `h` elements ahead of it, so rows of odd length still
// move in whole words; only the first and the last vector are ragged.
// LONG: rows beyond the registers of a cluster; two passes, the second from
// L2.
// TPB threads have a row (32: eight rows to a CTA, no barrier); CLUSTER: as
// many CTAs as `slabs` says do, else one.
// Without clusters a row's threads also bring the row `ahead` of it into L2:
// a CTA loads, reduces and stores in turn, and the few that fit an SM do not
// cover one another's trip to memory (16384 x 8192 bf16: 158 us without, 125
// with; 16384 x 1000: 30 and 25.5).
template <typename TZ, typename TG, int VE, int NV, bool LONG, int TPB, bool CLUSTER>
__global__ void __launch_bounds__(TPB == 32 ? 256 : TPB, policy_ctas<VE, NV, TPB>())
    policy_kernel(const LossArgs a, int slabs, int64_t ahead) {
  constexpr int WPB = TPB / 32;
  __shared__ float2 pairs[(CLUSTER ? MAX_SLABS : 1) * WPB];
  if (CLUSTER) cluster_arrive();
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = TPB == 32 ? 0 : threadIdx.x >> 5;
  const int t = TPB == 32 ? lane : threadIdx.x;
  if (!CLUSTER) slabs = 1;
  const int rank = CLUSTER ? blockIdx.x % slabs : 0;
  const int64_t row = TPB == 32 ? static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x / slabs;
  if (TPB == 32 && row >= a.tokens) return;
  const TZ* z = static_cast<const TZ*>(a.z) + row * a.ld_z;
  TG* g = a.g ? static_cast<TG*>(a.g) + row * a.ld_g : nullptr;
  const int V = a.vocab;
  const int h = static_cast<int>((reinterpret_cast<uintptr_t>(z) / sizeof(TZ)) % VE);
  const int nvec = (V + h + VE - 1) / VE;
  const TokenIn tok = token_in(a, row);
  const float ahead_w = !CLUSTER && ahead && row + ahead < a.tokens ? a.weights[row + ahead] : 0.f;

  if (ahead_w != 0.f && t == 0) prefetch_row(z + ahead * a.ld_z, V);
  if (tok.w == 0.f) {                    // nothing of the row is read
    const float zero[VE] = {};
    if (g)
      for (int i = rank * TPB + t; i < nvec; i += slabs * TPB) store_edge<TG, VE>(g, i * VE - h, V, zero);
    if (rank == 0 && t == 0) {
      a.logp[row] = 0.f;
      a.terms[row] = 0.f;
    }
    if (CLUSTER) cluster_wait();
  } else {
    const bool inside = tok.target >= 0 && tok.target < V;
    float za = __int_as_float(0x7FFFFFFF);
    if (inside) {
      Vec<TZ, 1> one;
      one.load(z + tok.target);
      za = one.get(0);
    }
    const int first = LONG ? rank * TPB + t : rank * TPB * NV + t;
    float e[NV][VE];
    float m = -INFINITY, s = 0.f;
    if constexpr (LONG) {
      for (int i = first; i < nvec; i += slabs * TPB) {
        float v[VE];
        load_edge<TZ, VE>(z, i * VE - h, V, v);
        float top = m;
#pragma unroll
        for (int j = 0; j < VE; ++j) top = fmaxf(top, v[j]);
        const float ms = top == -INFINITY ? 0.f : top;
        s *= exp_rel(m, ms);
        m = top;
#pragma unroll
        for (int j = 0; j < VE; ++j) s += exp_rel(v[j], ms);
      }
      const float top = warp_max(m);
      s = warp_sum(s * exp_rel(m, top == -INFINITY ? 0.f : top));
      m = top;
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (first + k * TPB < nvec) load_edge<TZ, VE>(z, (first + k * TPB) * VE - h, V, e[k]);
        else
#pragma unroll
          for (int j = 0; j < VE; ++j) e[k][j] = -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < VE; ++j) m = fmaxf(m, e[k][j]);
      m = warp_max(m);
      const float ms = m == -INFINITY ? 0.f : m;
      const float2 mm = splat(ms), l2e = splat(kLog2e);
      float part[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if constexpr (VE == 1) e[k][0] = exp_rel(e[k][0], ms);
        else
#pragma unroll
          for (int j = 0; j < VE; j += 2) exp_pair(e[k][j], e[k][j + 1], mm, l2e, e[k][j], e[k][j + 1]);
        part[k] = tree_sum(e[k]);
      }
      s = warp_sum(tree_sum(part));
    }
    float top = m, total = m == -INFINITY ? __int_as_float(0x7FFFFFFF) : s;
    if constexpr (TPB > 32) {
      if constexpr (CLUSTER) {
        cluster_wait();                  // every CTA of the cluster has started
        if (lane < slabs) st_cluster_f2(smem_u32(&pairs[rank * WPB + warp]), lane, m, s);
        cluster_sync();
      } else {
        if (lane == 0) pairs[warp] = make_float2(m, s);
        __syncthreads();
      }
      top = -INFINITY;
      for (int i = lane; i < slabs * WPB; i += 32) top = fmaxf(top, pairs[i].x);
      top = warp_max(top);
      total = 0.f;
      for (int i = lane; i < slabs * WPB; i += 32) total += pairs[i].y * exp_rel(pairs[i].x, top);
      total = warp_sum(total);
    }
    const float lp = (za - top) - logf(total);
    float l, slope;
    token_loss(a, tok, lp, l, slope);
    if (rank == 0 && t == 0) {
      a.logp[row] = lp;
      a.terms[row] = tok.w * l;
    }
    if (g) {
      const float k = a.scale * tok.w * slope;
      const int at = inside ? static_cast<int>(tok.target) : -VE;
      if constexpr (LONG) {
        const float f = -k / total;
        for (int i = first; i < nvec; i += slabs * TPB) {
          const int e0 = i * VE - h;
          float v[VE];
          load_edge<TZ, VE>(z, e0, V, v);
#pragma unroll
          for (int j = 0; j < VE; ++j) v[j] = fmaf(exp_rel(v[j], top), f, e0 + j == at ? k : 0.f);
          store_edge<TG, VE>(g, e0, V, v);
        }
      } else {
        // this warp's exponentials are relative to m
        const float f = -k * (exp_rel(m, top) / total);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          if (first + q * TPB >= nvec) continue;
          const int e0 = (first + q * TPB) * VE - h;
          float o[VE];
#pragma unroll
          for (int j = 0; j < VE; ++j) o[j] = e[q][j] * f;
          if (static_cast<unsigned>(at - e0) < static_cast<unsigned>(VE)) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
              if (e0 + j == at) o[j] += k;
          }
          store_edge<TG, VE>(g, e0, V, o);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- long rows of many tokens
// A persistent CTA (or cluster of `slabs`) takes token after token.  Its part
// of a row streams through a ring of 16 KiB chunks in shared memory: one warp
// issues the bulk copies, the others take the running maximum and sum as
// chunks arrive (first pass), exchange them over the cluster, and read the
// same chunks again to write the gradient (second pass), which frees them.
// The ring holds a whole part and a share of the next token's, so loads run
// ahead through the exchange and the stores, and two CTAs share an SM, so one
// computes while the other waits.  Two exponentials per element instead of
// one, but no data held in registers.  Eight warps to a CTA: with sixteen the
// waits and branches of each chunk weigh twice as much (2048 x 131072 bf16, no
// token masked: 229 us against 189 when that was chosen; 181 us since, 88 % of
// the measured copy rate).
constexpr int RING_CHUNK = 16384, RING_SLOTS = 6, RING_AHEAD = 2;
constexpr int RING_TPB = 256, RING_WARPS = RING_TPB / 32;
constexpr float kLowest = -3.402823466e38f;

// A thread's running maximum and sum over VE more elements.
template <int VE>
__device__ __forceinline__ void take_in(const float (&v)[VE], float& m, float& s) {
  float top = m;
#pragma unroll
  for (int j = 0; j < VE; j += 2) top = fmax3_nan(top, v[j], v[j + 1]);
  s *= ex2((m - top) * kLog2e);
  m = top;
  const float2 mm = splat(m), l2e = splat(kLog2e);
  float e[VE];
#pragma unroll
  for (int j = 0; j < VE; j += 2) exp_pair(v[j], v[j + 1], mm, l2e, e[j], e[j + 1]);
  s += tree_sum(e);
}

// The gradient's VE elements in place of the logits: exp(v - top) * f, and k
// more at the target.
template <int VE>
__device__ __forceinline__ void to_gradient(float (&v)[VE], float2 top, float f, int target, float k) {
  const float2 l2e = splat(kLog2e);
#pragma unroll
  for (int j = 0; j < VE; j += 2) {
    float x, y;
    exp_pair(v[j], v[j + 1], top, l2e, x, y);
    v[j] = x * f;
    v[j + 1] = y * f;
  }
  if (static_cast<unsigned>(target) < static_cast<unsigned>(VE)) {
#pragma unroll
    for (int j = 0; j < VE; ++j)
      if (j == target) v[j] += k;
  }
}

template <typename TZ, typename TG>
__global__ void __launch_bounds__(RING_TPB + 32, 2) policy_ring_kernel(const LossArgs a, int slabs, int part, int* status) {
  constexpr int VE = 16 / static_cast<int>(sizeof(TZ));      // elements of a 16-byte word of logits
  constexpr int CV = RING_CHUNK / 16;                        // words of a chunk
  constexpr int U = CV / RING_TPB;                           // words of a thread in it
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 pairs[2][MAX_SLABS * RING_WARPS];
  __shared__ __align__(8) uint64_t full[RING_SLOTS], empty[RING_SLOTS], xbar[2];
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING_SLOTS; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), RING_WARPS);
    }
    mbar_init(smem_u32(&xbar[0]), 1);
    mbar_init(smem_u32(&xbar[1]), 1);
    fence_mbar_init();
  }
  cluster_sync();
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % slabs;
  const int64_t row0 = blockIdx.x / slabs, step = gridDim.x / slabs;
  const int V = a.vocab;
  const int w0 = rank * part;                                // first word of this CTA's part
  bool alive = true;                                         // false once a wait has given up

  // elements between a row's first word boundary and its first element; words
  // [lo, hi) are whole, a ragged first or last one is read by its thread alone
  const auto shift = [&](int64_t row) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(a.z) / sizeof(TZ) + row * a.ld_z) % VE);
  };

  int slot = 0, phase = 0;                                   // the next chunk's slot and its parity
  if (warp == RING_WARPS) {
    if (lane == 0) {
      int n = 0;                                           // chunks issued
      float next = row0 < a.tokens ? a.weights[row0] : 0.f;
      for (int64_t row = row0; row < a.tokens && alive; row += step) {
        const float wt = next;
        if (row + step < a.tokens) next = a.weights[row + step];
        if (wt == 0.f) continue;
        const int h = shift(row);
        const uint8_t* base = static_cast<const uint8_t*>(a.z) + (row * a.ld_z - h) * static_cast<int64_t>(sizeof(TZ));
        const int lo = h ? 1 : 0, hi = (V + h) / VE, end = min(w0 + part, (V + h + VE - 1) / VE);
        for (int w = w0; w < end; w += CV) {
          if (n >= RING_SLOTS) {
            alive = mbar_wait_sleep(smem_u32(&empty[slot]), phase ^ 1, status);
            if (!alive) break;
          }
          const int b = max(w, lo), e = min(min(w + CV, end), hi);
          const uint32_t bytes = e > b ? static_cast<uint32_t>(e - b) * 16u : 0u;
          mbar_arrive_expect_tx(smem_u32(&full[slot]), bytes);
          if (bytes)
            bulk_load_1d(smem_u32(ring + slot * RING_CHUNK + (b - w) * 16), base + static_cast<int64_t>(b) * 16, bytes,
                         smem_u32(&full[slot]));
          ++n;
          if (++slot == RING_SLOTS) slot = 0, phase ^= 1;
        }
      }
      // no exit with copies in flight
      for (int i = max(0, n - RING_SLOTS); i < n; ++i)
        mbar_wait(smem_u32(&full[i % RING_SLOTS]), (i / RING_SLOTS) & 1, status);
    }
    __syncwarp();
  } else {
    const int t = threadIdx.x;
    int live = 0;                                          // tokens taken
    TokenIn next = token_in(a, row0);
    for (int64_t row = row0; row < a.tokens; row += step) {
      const TokenIn tok = next;
      next = token_in(a, row + step);
      const TZ* z = static_cast<const TZ*>(a.z) + row * a.ld_z;
      TG* g = a.g ? static_cast<TG*>(a.g) + row * a.ld_g : nullptr;
      const int h = shift(row);
      const int lo = h ? 1 : 0, hi = (V + h) / VE, end = min(w0 + part, (V + h + VE - 1) / VE);
      if (tok.w == 0.f) {                                  // nothing of the row is read
        const float zero[VE] = {};
        if (g)
          for (int w = w0 + t; w < end; w += RING_TPB) store_edge<TG, VE>(g, w * VE - h, V, zero);
        if (rank == 0 && t == 0) {
          a.logp[row] = 0.f;
          a.terms[row] = 0.f;
        }
        continue;
      }
      const bool inside = tok.target >= 0 && tok.target < V;
      float za = __int_as_float(0x7FFFFFFF);
      if (inside) {
        Vec<TZ, 1> one;
        one.load(z + tok.target);
        za = one.get(0);
      }
      const int whole_lo = max(w0, lo), whole_hi = min(end, hi);   // this part's whole words

      const auto whole = [&](const uint8_t* chunk, int at, float (&v)[VE]) {
        const uint4 q = *reinterpret_cast<const uint4*>(chunk + at * 16);
        Vec<TZ, VE> r;
        r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
#pragma unroll
        for (int j = 0; j < VE; ++j) v[j] = r.get(j);
      };
      // the ragged words, where this part has them: the first is thread 0's,
      // the last thread 32's, straight from memory
      const int edge = t == 0 && lo && w0 == 0 ? 0 : t == 32 && hi >= w0 && hi < end ? hi : -1;

      // first pass: running maximum and sum; the lowest float32 stands for
      // "none yet", so no difference is inf - inf
      float m = kLowest, s = 0.f;
      const int slot0 = slot;
      for (int w = w0; w < end; w += CV) {
        if (alive) alive = mbar_wait_sleep(smem_u32(&full[slot]), phase, status);
        const uint8_t* chunk = ring + slot * RING_CHUNK;
        if (w >= whole_lo && w + CV <= whole_hi) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[VE];
            whole(chunk, t + u * RING_TPB, v);
            take_in(v, m, s);
          }
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[VE];
            const int word = w + t + u * RING_TPB;
            if (word >= whole_lo && word < whole_hi) {
              whole(chunk, t + u * RING_TPB, v);
              take_in(v, m, s);
            }
          }
        }
        if (++slot == RING_SLOTS) slot = 0, phase ^= 1;
      }
      if (edge >= 0) {
        float v[VE];
        load_edge<TZ, VE>(z, edge * VE - h, V, v);
        take_in(v, m, s);
      }
      const float wm = warp_max(m);
      s = warp_sum(s * ex2((m - wm) * kLog2e));
      const int par = live & 1;
      // (once a wait has given up, its phase may still be open: no second arrival)
      if (t == 0 && alive) mbar_arrive_expect_tx(smem_u32(&xbar[par]), slabs * RING_WARPS * 8);
      if (lane < slabs)
        st_async_f2(smem_u32(&pairs[par][rank * RING_WARPS + warp]), smem_u32(&xbar[par]), lane, wm, s);
      if (alive) alive = mbar_wait_sleep<true>(smem_u32(&xbar[par]), (live >> 1) & 1, status);
      ++live;
      float top = kLowest;
      for (int i = lane; i < slabs * RING_WARPS; i += 32) top = fmaxf(top, pairs[par][i].x);
      top = warp_max(top);
      float total = 0.f;
      for (int i = lane; i < slabs * RING_WARPS; i += 32) total += pairs[par][i].y * ex2((pairs[par][i].x - top) * kLog2e);
      total = warp_sum(total);
      const float lp = (za - top) - logf(total);
      float l, slope;
      token_loss(a, tok, lp, l, slope);
      if (rank == 0 && t == 0) {
        a.logp[row] = lp;
        a.terms[row] = tok.w * l;
      }

      // second pass: the gradient, and the chunks are free
      const float k = a.scale * tok.w * slope;
      const int at = inside ? static_cast<int>(tok.target) : -VE;
      const float2 tt = splat(top);
      const float f = -k / total;
      int sl = slot0;
      for (int w = w0; w < end; w += CV) {
        const uint8_t* chunk = ring + sl * RING_CHUNK;
        if (g && w >= whole_lo && w + CV <= whole_hi) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[VE];
            const int e0 = (w + t + u * RING_TPB) * VE - h;
            whole(chunk, t + u * RING_TPB, v);
            to_gradient(v, tt, f, at - e0, k);
            store_vec<TG, VE>(g + e0, v);
          }
        } else if (g) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[VE];
            const int word = w + t + u * RING_TPB, e0 = word * VE - h;
            if (word >= whole_lo && word < whole_hi) {
              whole(chunk, t + u * RING_TPB, v);
              to_gradient(v, tt, f, at - e0, k);
              store_vec<TG, VE>(g + e0, v);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty[sl]));
        if (++sl == RING_SLOTS) sl = 0;
      }
      if (g && edge >= 0) {
        float v[VE];
        const int e0 = edge * VE - h;
        load_edge<TZ, VE>(z, e0, V, v);
        to_gradient(v, tt, f, at - e0, k);
        store_edge<TG, VE>(g, e0, V, v);
      }
    }
  }
  cluster_sync();                                            // no peer writes here any more,
  if (!alive) linger();                                      // unless a wait gave up
}

using namespace mxq_host;

template <typename TZ, typename TG, int VE, int NV, bool LONG, int TPB, bool CLUSTER>
int launch_policy(const LossArgs& a, int slabs, cudaStream_t st) {
  const int64_t grid = TPB == 32 ? (static_cast<int64_t>(a.tokens) + 7) / 8 : static_cast<int64_t>(a.tokens) * slabs;
  if (grid > 0x7FFFFFFF) return MXQ_ERR_BAD_SHAPE;
  auto kern = policy_kernel<TZ, TG, VE, NV, LONG, TPB, CLUSTER>;
  const dim3 g(static_cast<unsigned>(grid)), b(TPB == 32 ? 256 : TPB);
  // The rows that run at once; a quarter of them start within the next row's
  // trip to memory (half or all of them ahead, 16384 x 8192: 126 and 131 us,
  // a quarter 125).  Nothing is ahead while most rows start together.
  const int64_t live = static_cast<int64_t>(sm_count()) * policy_ctas<VE, NV, TPB>() * (TPB == 32 ? 8 : 1);
  const int64_t ahead = a.tokens >= 2 * live ? live / 4 : 0;
  return CLUSTER ? launch_pdl_cluster(kern, g, b, 0, st, slabs, a, slabs, int64_t{0})
                 : launch_pdl(kern, g, b, 0, st, a, 1, ahead);
}

// Clusters of `slabs` CTAs that run at once (asked once per device and size).
template <typename TZ, typename TG>
int ring_clusters(int slabs) {
  static std::atomic<int> known[64][MAX_SLABS + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][slabs].load(std::memory_order_relaxed);
  if (n) return n;
  auto kern = policy_ring_kernel<TZ, TG>;
  const int smem = RING_CHUNK * RING_SLOTS;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(slabs * 4 * sm_count());
  cfg.blockDim = dim3(RING_TPB + 32);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = slabs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) return 0;
  known[dev][slabs].store(n, std::memory_order_relaxed);
  return n;
}

// Words of a row of logits, whatever its shift.
template <typename TZ>
int64_t row_words(const LossArgs& a) {
  constexpr int VE = 16 / static_cast<int>(sizeof(TZ));
  const bool flush = a.ld_z % VE == 0 && reinterpret_cast<uintptr_t>(a.z) % 16 == 0;
  return (static_cast<int64_t>(a.vocab) + (flush ? 0 : VE - 1) + VE - 1) / VE;
}

// The ring kernel takes rows beyond the register kernels' (float32), or their
// last step of 12288 to 16384 elements and on (bf16), when every CTA gets two
// tokens or more, in the smallest cluster whose CTAs keep RING_AHEAD chunks of
// the ring for the next token.  Here against in registers, no token masked, us:
// bf16 16384 x 12000 205 and 178, 8192 x 12296 110 and 120, 8192 x 16384 115 and
// 131; float32 8192 x 12001 144 and 122 (bf16 gradient 132 and 101), 4096 x 16384
// 100 and 87, 4096 x 16392 108 and 168.  0: not for it.
template <typename TZ>
int ring_slabs(const LossArgs& a) {
  if (a.vocab <= (sizeof(TZ) == 2 ? 12288 : 16384)) return 0;
  for (int slabs = 1; slabs <= MAX_SLABS; slabs *= 2)
    if ((row_words<TZ>(a) + slabs - 1) / slabs <= (RING_SLOTS - RING_AHEAD) * (RING_CHUNK / 16))
      return static_cast<int64_t>(a.tokens) * slabs >= 4 * sm_count() ? slabs : 0;
  return 0;
}

template <typename TZ, typename TG>
int launch_ring(const LossArgs& a, int slabs, cudaStream_t st) {
  const int part = static_cast<int>((row_words<TZ>(a) + slabs - 1) / slabs);
  const int clusters = std::min(a.tokens, ring_clusters<TZ, TG>(slabs));
  int* status = status_ptr();
  if (!clusters || !status) return MXQ_ERR_CUDA;
  return launch_pdl_cluster(policy_ring_kernel<TZ, TG>, dim3(clusters * slabs), dim3(RING_TPB + 32),
                            RING_CHUNK * RING_SLOTS, st, slabs, a, slabs, part, status);
}

// With enough tokens to fill the GPU, a row goes to the fewest threads that
// hold it, 32 elements each: a warp, or a CTA of 4, 6, 8, 12 or 16 (half as many
// elements to twice the threads: 16384 x 1000 bf16 30 -> 38 us, 8192 columns
// 154 -> 161; without the CTAs of 6 and 12: 6000 columns 93 -> 114 us, 12000
// columns 177 -> 228).  Longer rows, and rows of few tokens, to clusters: the
// fewest CTAs of 16 warps that hold a row, and more with few tokens, until there
// are two for every SM or eight to a row.
template <typename TZ, typename TG, int VE>
int dispatch_policy(const LossArgs& a, cudaStream_t st) {
  constexpr int NMAX = MAX_E / VE;
  // the words of a row, whatever its shift
  const bool flush = a.ld_z % VE == 0 && reinterpret_cast<uintptr_t>(a.z) / sizeof(TZ) % VE == 0;
  const int64_t nvec = (static_cast<int64_t>(a.vocab) + (flush ? 0 : VE - 1) + VE - 1) / VE;
  if (a.tokens >= sm_count() && nvec <= 512 * NMAX) {
    if (nvec <= 32 * NMAX)
      return nvec <= 32 * NMAX / 4 ? launch_policy<TZ, TG, VE, NMAX / 4, false, 32, false>(a, 1, st)
                                   : launch_policy<TZ, TG, VE, NMAX, false, 32, false>(a, 1, st);
    if (nvec <= 128 * NMAX)
      return nvec <= 64 * NMAX ? launch_policy<TZ, TG, VE, NMAX / 2, false, 128, false>(a, 1, st)
                               : launch_policy<TZ, TG, VE, NMAX, false, 128, false>(a, 1, st);
    if (nvec <= 192 * NMAX) return launch_policy<TZ, TG, VE, NMAX, false, 192, false>(a, 1, st);
    if (nvec <= 256 * NMAX) return launch_policy<TZ, TG, VE, NMAX, false, 256, false>(a, 1, st);
    if (nvec <= 384 * NMAX) return launch_policy<TZ, TG, VE, NMAX, false, 384, false>(a, 1, st);
    return launch_policy<TZ, TG, VE, NMAX, false, 512, false>(a, 1, st);
  }
  constexpr int TPB = 512;
  int slabs = static_cast<int>(std::min<int64_t>((nvec + TPB * NMAX - 1) / (TPB * NMAX), MAX_SLABS + 1));
  if (slabs > MAX_SLABS) return launch_policy<TZ, TG, VE, 1, true, TPB, true>(a, MAX_SLABS, st);
  while (slabs < MAX_SLABS && static_cast<int64_t>(a.tokens) * slabs < 2 * sm_count() && nvec > TPB * slabs)
    slabs = std::min(MAX_SLABS, 2 * slabs);
  const int64_t nv = (nvec + static_cast<int64_t>(TPB) * slabs - 1) / (static_cast<int64_t>(TPB) * slabs);
  if (nv <= NMAX / 4) return launch_policy<TZ, TG, VE, NMAX / 4, false, TPB, true>(a, slabs, st);
  if (nv <= NMAX / 2) return launch_policy<TZ, TG, VE, NMAX / 2, false, TPB, true>(a, slabs, st);
  return launch_policy<TZ, TG, VE, NMAX, false, TPB, true>(a, slabs, st);
}

template <typename TZ, typename TG>
int policy_rows(const LossArgs& a, cudaStream_t st) {
  constexpr int VE = sizeof(TZ) == 2 && sizeof(TG) == 2 ? 8 : 4;
  constexpr int RVE = 16 / static_cast<int>(sizeof(TZ));
  // whole words on both sides: every row of the gradient starts at the same
  // element of its word as the row of logits
  const auto same = [&](int ve) {
    return !a.g || ((a.ld_z - a.ld_g) % ve == 0 && (reinterpret_cast<uintptr_t>(a.z) / sizeof(TZ)) % ve ==
                                                       (reinterpret_cast<uintptr_t>(a.g) / sizeof(TG)) % ve);
  };
  if (same(RVE))
    if (const int slabs = ring_slabs<TZ>(a)) return launch_ring<TZ, TG>(a, slabs, st);
  return same(VE) ? dispatch_policy<TZ, TG, VE>(a, st) : dispatch_policy<TZ, TG, 1>(a, st);
}

template <typename TZ, typename TG>
int policy(const LossArgs& a, cudaStream_t st) {
  const int rc = policy_rows<TZ, TG>(a, st);
  return rc ? rc : launch_pdl(loss_sum_kernel, dim3(1), dim3(std::min(1024, (a.tokens + 31) / 32 * 32)), 0, st, a);
}

}  // namespace
}  // namespace mxq

using namespace mxq;
using namespace mxq_host;

extern "C" int mxq_policy_loss_workspace_size(int64_t tokens, size_t* bytes) {
  if (!bytes) return MXQ_ERR_BAD_ARG;
  if (tokens < 0) return MXQ_ERR_BAD_SHAPE;
  *bytes = 256 + static_cast<size_t>(tokens) * sizeof(float);
  return MXQ_OK;
}

extern "C" int mxq_policy_loss(const void* logits, int64_t tokens, int64_t vocab, int64_t ld, int logits_type,
                               const void* targets, int targets_64, const float* old_logp, const float* advantages,
                               const float* weights, const float* ref_logp, float clip_low, float clip_high,
                               float beta, float grad_scale, float* loss, float* logp, void* grad, int64_t ld_grad,
                               int grad_type, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_type(logits_type) || (grad && !valid_type(grad_type))) return MXQ_ERR_BAD_ARG;
  if ((targets_64 != 0 && targets_64 != 1) || !loss) return MXQ_ERR_BAD_ARG;
  if (tokens < 0 || vocab < 1 || ld < vocab || (grad && ld_grad < vocab)) return MXQ_ERR_BAD_SHAPE;
  if (tokens > 0x7FFFFFFFll / MAX_SLABS || vocab > kMaxCols) return MXQ_ERR_BAD_SHAPE;
  if (tokens && (!logits || !targets || !old_logp || !advantages || !weights || !logp)) return MXQ_ERR_BAD_ARG;
  if (tokens && beta != 0.f && !ref_logp) return MXQ_ERR_BAD_ARG;
  if (!(clip_low >= 0.f) || !(clip_high >= 0.f)) return MXQ_ERR_BAD_ARG;
  size_t need = 0;
  mxq_policy_loss_workspace_size(tokens, &need);
  if (!workspace || workspace_bytes < need) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(logits, type_size(logits_type)) || !aligned_to(targets, targets_64 ? 8 : 4) ||
      !aligned_to(old_logp, 4) || !aligned_to(advantages, 4) || !aligned_to(weights, 4) || !aligned_to(ref_logp, 4) ||
      !aligned_to(loss, 4) || !aligned_to(logp, 4) || (grad && !aligned_to(grad, type_size(grad_type))) ||
      !aligned16(workspace))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  const auto st = static_cast<cudaStream_t>(stream);
  if (!tokens) return cudaMemsetAsync(loss, 0, sizeof(float), st) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
  LossArgs a{};
  a.z = logits, a.ld_z = ld, a.g = grad, a.ld_g = ld_grad;
  a.targets = targets, a.targets64 = targets_64;
  a.old_lp = old_logp, a.adv = advantages, a.weights = weights, a.ref_lp = ref_logp;
  a.lo = clip_low, a.hi = clip_high, a.beta = beta, a.scale = grad_scale;
  a.tokens = static_cast<int>(tokens), a.vocab = static_cast<int>(vocab);
  a.logp = logp, a.loss = loss;
  a.terms = static_cast<float*>(workspace);
  using bf16 = __nv_bfloat16;
  if (logits_type == MXQ_BF16)
    return grad && grad_type == MXQ_F32 ? policy<bf16, float>(a, st) : policy<bf16, bf16>(a, st);
  return grad && grad_type == MXQ_BF16 ? policy<float, bf16>(a, st) : policy<float, float>(a, st);
}
