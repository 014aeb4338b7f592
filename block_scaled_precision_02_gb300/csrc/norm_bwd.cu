// Backward pass of layer norm: the input's gradient and the reductions of the
// weight's and the bias's.
#include "norm.cuh"

namespace mxq {
namespace {

constexpr int BWD_THREADS = 512;
constexpr int BWD_KEEP = 16;               // elements of a thread whose x and dy stay in registers
constexpr int kMaxBwdElems = 16384;        // a row and its two column sums in one CTA

struct BwdArgs {
  const void* dy;
  int64_t ld_dy;
  const void* x;
  int64_t ld_x;
  int rows, cols;
  const float* mean;
  const float* rstd;
  const void* w;
  int w_f32;
  void* dx;               // [rows][cols], the type of x
  float* part;            // [parts][2][cols] sums of dy*h and dy over a CTA's rows; NULL: not wanted
  float* coef;            // [rows][2] (long rows only)
};

// A thread owns VE * NV columns and keeps their two column sums in registers
// while its CTA walks over rows; a group of G threads has a row.  x and dy are
// read once and dx written once; the column sums of a CTA go out once at the
// end and a second kernel adds them up in a fixed order.  For few rows, and
// for rows that the rings below do not take: bound by the latency of a row's
// load, reduction and store.
template <typename TX, typename TD, int VE, int NV>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(const BwdArgs a, int G) {
  __shared__ float2 red[2][32];
  extern __shared__ __align__(16) float comb[];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = blockDim.x / G, g = threadIdx.x / G, t = threadIdx.x - g * G;
  const int wpg = G >> 5, first = first_vec<NV>(t >> 5, lane);
  const int nvec = a.cols / VE;
  const float inv_c = 1.f / static_cast<float>(a.cols);

  float w[NV][VE], aw[NV][VE], ab[NV][VE];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      w[k][j] = 1.f;
      aw[k][j] = ab[k][j] = 0.f;
    }
    if (a.w && first + 32 * k < nvec) load_param<VE>(a.w, a.w_f32, (first + 32 * k) * VE, w[k]);
  }

  int buf = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * P;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * P; base < a.rows; base += step) {
    const int64_t row = base + g;
    const bool in = row < a.rows;            // a CTA's groups stay together for the barrier
    const float mean = in ? a.mean[row] : 0.f, rstd = in ? a.rstd[row] : 0.f;
    Vec<TX, VE> xr[NV];
    Vec<TD, VE> dr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      xr[k].fill(0);
      dr[k].fill(0);
      if (in && first + 32 * k < nvec) {
        xr[k].load(static_cast<const TX*>(a.x) + row * a.ld_x + (first + 32 * k) * VE);
        dr[k].load(static_cast<const TD*>(a.dy) + row * a.ld_dy + (first + 32 * k) * VE);
      }
    }
    float s1[NV], s2[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float u[VE], v[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float h = (xr[k].get(j) - mean) * rstd;
        const float d = dr[k].get(j);
        u[j] = d * w[k][j];
        v[j] = u[j] * h;
        aw[k][j] = fmaf(d, h, aw[k][j]);
        ab[k][j] += d;
      }
      s1[k] = tree_sum(u);
      s2[k] = tree_sum(v);
    }
    float c1 = warp_sum(tree_sum(s1)), c2 = warp_sum(tree_sum(s2));
    if (wpg > 1) {
      if (lane == 0) red[buf][warp] = make_float2(c1, c2);
      __syncthreads();
      c1 = c2 = 0.f;
      for (int i = 0; i < wpg; ++i) {
        const float2 v = red[buf][g * wpg + i];
        c1 += v.x;
        c2 += v.y;
      }
      buf ^= 1;
    }
    if (!in) continue;
    const float m1 = c1 * inv_c, m2 = c2 * inv_c;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (first + 32 * k >= nvec) continue;
      float o[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float h = (xr[k].get(j) - mean) * rstd;
        o[j] = (fmaf(dr[k].get(j), w[k][j], -m1) - h * m2) * rstd;
      }
      store_vec<TX, VE>(static_cast<TX*>(a.dx) + row * a.cols + (first + 32 * k) * VE, o);
    }
  }
  if (!a.part) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  if (P > 1) {                      // the groups of the CTA first, in their order
    for (int i = 1; i < P; ++i) {
      __syncthreads();
      if (g == i)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            comb[(2 * (k * VE + j)) * G + t] = aw[k][j];
            comb[(2 * (k * VE + j) + 1) * G + t] = ab[k][j];
          }
      __syncthreads();
      if (g == 0)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            aw[k][j] += comb[(2 * (k * VE + j)) * G + t];
            ab[k][j] += comb[(2 * (k * VE + j) + 1) * G + t];
          }
    }
    if (g) return;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (first + 32 * k >= nvec) continue;
    if constexpr (VE == 1) {
      out[first + 32 * k] = aw[k][0];
      out[a.cols + first + 32 * k] = ab[k][0];
    } else {
      store_vec<float, VE>(out + (first + 32 * k) * VE, aw[k]);
      store_vec<float, VE>(out + a.cols + (first + 32 * k) * VE, ab[k]);
    }
  }
}

// The same for many rows, through rings of rows (x and dy side by side in a
// slot).  Up to 16 elements a thread: x and dy stay in registers from the sums
// to dx.  More (KEEP false): the slot is read again for dx and given
// back after the next row's barrier, and the weights are read from shared
// memory, because the column sums fill the registers.
static_assert(BWD_THREADS <= 512, "half a warp adds the warps' sums of a row");
template <typename TX, typename TD, int VE, int NV, bool FULL>
__global__ void __launch_bounds__(BWD_THREADS, 1) norm_bwd_ring_kernel(const BwdArgs a, int G, int stages, int* status) {
  constexpr bool KEEP = VE * NV <= BWD_KEEP;
  constexpr int KV = KEEP ? NV : 1;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][2][BWD_THREADS / 32];     // [buffer][sum][warp of the CTA]
  __shared__ __align__(8) uint64_t full[MAX_GROUPS][MAX_STAGES];
  const int lane = threadIdx.x & 31;
  const int P = blockDim.x / G, g = threadIdx.x / G, t = threadIdx.x - g * G;
  const int gw = t >> 5, wpg = G >> 5, first = first_vec<NV>(gw, lane);
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(smem_u32(&full[g][i]), 1);
    fence_mbar_init();
  }
  const int nvec = a.cols / VE;
  const RowSource<TX> sx{static_cast<const TX*>(a.x), a.ld_x, a.cols, a.rows};
  const RowSource<TD> sd{static_cast<const TD*>(a.dy), a.ld_dy, a.cols, a.rows};
  const int xb = slot_bytes(a.cols * static_cast<int>(sizeof(TX)), VE > 1);
  const int sb = xb + slot_bytes(a.cols * static_cast<int>(sizeof(TD)), VE > 1);
  const int wsize = a.w_f32 ? 4 : 2;
  uint8_t* ws = ring;                                // !KEEP: the weights, as they are
  uint8_t* slots = ring + (KEEP ? 0 : slot_bytes(wsize * a.cols, true)) + static_cast<size_t>(g) * stages * sb;
  grid_dep_wait();
  grid_dep_launch();
  const float inv_c = 1.f / static_cast<float>(a.cols);
  const int64_t gi = static_cast<int64_t>(blockIdx.x) * P + g, step = static_cast<int64_t>(gridDim.x) * P;
  bool alive = true;
  const auto copied = [&](int64_t row) { return VE > 1 || (sx.copied(row) && sd.copied(row)); };
  const auto issue = [&](int slot, int64_t row) {
    const uint32_t bar = smem_u32(&full[g][slot]);
    const bool copy = copied(row);
    mbar_arrive_expect_tx(bar, copy ? sx.bytes(row) + sd.bytes(row) : 0u);
    if (copy) {
      sx.issue(slots + slot * sb, bar, row);
      sd.issue(slots + slot * sb + xb, bar, row);
    }
  };
  // a vector of x and dy of the row in `slot`
  const auto take = [&](int slot, int64_t row, bool in_ring, int k, Vec<TX, VE>& xv, Vec<TD, VE>& dv) {
    if (!FULL) {
      xv.fill(0);
      dv.fill(0);
      if (first + 32 * k >= nvec) return;
    }
    if (in_ring) {
      const uint8_t* p = slots + slot * sb;
      xv.load(reinterpret_cast<const TX*>(p + (VE > 1 ? 0 : sx.head(row))) + (first + 32 * k) * VE);
      dv.load(reinterpret_cast<const TD*>(p + xb + (VE > 1 ? 0 : sd.head(row))) + (first + 32 * k) * VE);
    } else {
      xv.load(sx.row(row) + (first + 32 * k) * VE);
      dv.load(sd.row(row) + (first + 32 * k) * VE);
    }
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i)
      if (gi + i * step < a.rows) issue(i, gi + i * step);
  float w[KV][VE], aw[NV][VE], ab[NV][VE];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = 0; j < VE; ++j) aw[k][j] = ab[k][j] = 0.f;
#pragma unroll
  for (int k = 0; k < KV; ++k) {
#pragma unroll
    for (int j = 0; j < VE; ++j) w[k][j] = 1.f;
    if (KEEP && a.w && first + 32 * k < nvec) load_param<VE>(a.w, a.w_f32, (first + 32 * k) * VE, w[k]);
  }
  if (!KEEP && a.w)
    for (int i = threadIdx.x; i < a.cols; i += blockDim.x) {
      if (a.w_f32) reinterpret_cast<float*>(ws)[i] = static_cast<const float*>(a.w)[i];
      else reinterpret_cast<uint16_t*>(ws)[i] = static_cast<const uint16_t*>(a.w)[i];
    }
  __syncthreads();

  int slot = 0, phase = 0, buf = 0;
  float mean_n = gi < a.rows ? a.mean[gi] : 0.f, rstd_n = gi < a.rows ? a.rstd[gi] : 0.f;
  for (int64_t row = gi; row < a.rows; row += step) {
    const float mean = mean_n, rstd = rstd_n;
    if (row + step < a.rows) mean_n = a.mean[row + step], rstd_n = a.rstd[row + step];
    const float2 mm = splat(mean), rr = splat(rstd);
    const bool in_ring = copied(row);
    if (alive) alive = mbar_wait(smem_u32(&full[g][slot]), phase, status);
    Vec<TX, VE> xs[KV];
    Vec<TD, VE> ds[KV];
    if (KEEP)
#pragma unroll
      for (int k = 0; k < NV; ++k) take(slot, row, in_ring, k, xs[KEEP ? k : 0], ds[KEEP ? k : 0]);
    float s1[NV], s2[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Vec<TX, VE>& xv = xs[KEEP ? k : 0];
      Vec<TD, VE>& dv = ds[KEEP ? k : 0];
      if (!KEEP) take(slot, row, in_ring, k, xv, dv);
      float hk[VE], uk[VE], wk[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) wk[j] = KEEP ? w[KEEP ? k : 0][j] : 1.f;
      if (!KEEP && a.w && (FULL || first + 32 * k < nvec)) load_param<VE>(ws, a.w_f32, (first + 32 * k) * VE, wk);
      if constexpr (VE == 1) {
        const float d = dv.get(0);
        hk[0] = (xv.get(0) - mean) * rstd;
        uk[0] = d * wk[0];
        aw[k][0] = fmaf(d, hk[0], aw[k][0]);
        ab[k][0] += d;
        s1[k] = uk[0];
        s2[k] = uk[0] * hk[0];
      } else {
        float2 p1, p2;
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
          const float2 hh = mul2(sub2(pair(xv.get(j), xv.get(j + 1)), mm), rr);
          const float2 dd = pair(dv.get(j), dv.get(j + 1));
          const float2 uu = mul2(dd, pair(wk[j], wk[j + 1]));
          halves(fma2(dd, hh, pair(aw[k][j], aw[k][j + 1])), aw[k][j], aw[k][j + 1]);
          halves(add2(dd, pair(ab[k][j], ab[k][j + 1])), ab[k][j], ab[k][j + 1]);
          p1 = j ? add2(p1, uu) : uu;
          p2 = j ? fma2(uu, hh, p2) : mul2(uu, hh);
          halves(hh, hk[j], hk[j + 1]);
          halves(uu, uk[j], uk[j + 1]);
        }
        float x, y;
        halves(p1, x, y);
        s1[k] = x + y;
        halves(p2, x, y);
        s2[k] = x + y;
      }
    }
    // both sums in one butterfly: the lower half of the warp takes the first,
    // the upper half the second
    const float c1 = tree_sum(s1), c2 = tree_sum(s2);
    const bool up = lane & 16;
    float v = (up ? c2 : c1) + __shfl_xor_sync(0xFFFFFFFFu, up ? c1 : c2, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (wpg > 1) {
      if ((lane & 15) == 0) red[buf][lane >> 4][g * wpg + gw] = v;
      group_barrier(g, G);
    } else {
      __syncwarp();
    }
    if (t == 0) {
      if constexpr (KEEP) {                  // all have read this slot
        if (row + stages * step < a.rows) issue(slot, row + stages * step);
      } else {                               // all are done with the last one
        const int64_t next = row + (stages - 1) * step;
        if (row != gi && next < a.rows) issue(slot ? slot - 1 : stages - 1, next);
      }
    }
    if (wpg > 1) {
      v = (lane & 15) < wpg ? red[buf][lane >> 4][g * wpg + (lane & 15)] : 0.f;
#pragma unroll
      for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      buf ^= 1;
    }
    const float m1 = __shfl_sync(0xFFFFFFFFu, v, 0) * inv_c, m2 = __shfl_sync(0xFFFFFFFFu, v, 16) * inv_c;
    TX* dx = static_cast<TX*>(a.dx) + row * a.cols;
    const float2 c1c1 = splat(m1), c2c2 = splat(-m2);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!FULL && first + 32 * k >= nvec) continue;
      float hk[VE], uk[VE], o[VE];
      Vec<TX, VE>& xv = xs[KEEP ? k : 0];
      Vec<TD, VE>& dv = ds[KEEP ? k : 0];
      if (!KEEP) take(slot, row, in_ring, k, xv, dv);
      float wk[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) wk[j] = KEEP ? w[KEEP ? k : 0][j] : 1.f;
      if (!KEEP && a.w) load_param<VE>(ws, a.w_f32, (first + 32 * k) * VE, wk);
      if constexpr (VE == 1) {
        hk[0] = (xv.get(0) - mean) * rstd;
        uk[0] = dv.get(0) * wk[0];
      } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2) {
          halves(mul2(sub2(pair(xv.get(j), xv.get(j + 1)), mm), rr), hk[j], hk[j + 1]);
          halves(mul2(pair(dv.get(j), dv.get(j + 1)), pair(wk[j], wk[j + 1])), uk[j], uk[j + 1]);
        }
      }
      if constexpr (VE == 1) {
        o[0] = fmaf(hk[0], -m2, uk[0] - m1) * rstd;
      } else {
#pragma unroll
        for (int j = 0; j < VE; j += 2)
          halves(mul2(fma2(pair(hk[j], hk[j + 1]), c2c2,
                                           sub2(pair(uk[j], uk[j + 1]), c1c1)),
                                 rr),
                       o[j], o[j + 1]);
      }
      store_vec<TX, VE>(dx + (first + 32 * k) * VE, o);
    }
    if (++slot == stages) slot = 0, phase ^= 1;
  }
  if (!alive && t == 0) await_ring(full[g], stages, slot, phase, status);
  if (!a.part) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
  float* comb = reinterpret_cast<float*>(ring);
  for (int i = 1; i < P; ++i) {              // the groups of the CTA, in their order
    __syncthreads();                         // (every copy has been waited for: the ring is free)
    if (g == i)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          comb[(2 * (k * VE + j)) * G + t] = aw[k][j];
          comb[(2 * (k * VE + j) + 1) * G + t] = ab[k][j];
        }
    __syncthreads();
    if (g == 0)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          aw[k][j] += comb[(2 * (k * VE + j)) * G + t];
          ab[k][j] += comb[(2 * (k * VE + j) + 1) * G + t];
        }
  }
  if (g) return;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (first + 32 * k >= nvec) continue;
    store_vec<float, VE>(out + (first + 32 * k) * VE, aw[k]);
    store_vec<float, VE>(out + a.cols + (first + 32 * k) * VE, ab[k]);
  }
}

// Rows too long for the registers: their two sums first ...
template <typename TX, typename TD>
__global__ void __launch_bounds__(1024) norm_bwd_long_rows_kernel(const BwdArgs a) {
  __shared__ float red[32];
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + row * a.ld_x;
  const TD* dy = static_cast<const TD*>(a.dy) + row * a.ld_dy;
  const float mean = a.mean[row], rstd = a.rstd[row];
  float c1 = 0.f, c2 = 0.f;
  for (int i = threadIdx.x; i < a.cols; i += 1024) {
    Vec<TX, 1> xe;
    Vec<TD, 1> de;
    xe.load(x + i);
    de.load(dy + i);
    float w[1] = {1.f};
    if (a.w) load_param<1>(a.w, a.w_f32, i, w);
    const float u = de.get(0) * w[0];
    c1 += u;
    c2 += u * ((xe.get(0) - mean) * rstd);
  }
  c1 = block_sum_1024(c1, red);
  c2 = block_sum_1024(c2, red);
  if (threadIdx.x == 0) {
    a.coef[2 * row] = c1 / static_cast<float>(a.cols);
    a.coef[2 * row + 1] = c2 / static_cast<float>(a.cols);
  }
}

// ... then a column per thread over a range of rows (blockIdx.y).
template <typename TX, typename TD>
__global__ void __launch_bounds__(256) norm_bwd_long_cols_kernel(const BwdArgs a) {
  grid_dep_wait();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float w[1] = {1.f};
  if (a.w) load_param<1>(a.w, a.w_f32, c, w);
  float aw = 0.f, ab = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    Vec<TX, 1> xe;
    Vec<TD, 1> de;
    xe.load(static_cast<const TX*>(a.x) + row * a.ld_x + c);
    de.load(static_cast<const TD*>(a.dy) + row * a.ld_dy + c);
    const float rstd = a.rstd[row], h = (xe.get(0) - a.mean[row]) * rstd, d = de.get(0);
    aw = fmaf(d, h, aw);
    ab += d;
    float o[1] = {(fmaf(d, w[0], -a.coef[2 * row]) - h * a.coef[2 * row + 1]) * rstd};
    store_vec<TX, 1>(static_cast<TX*>(a.dx) + row * a.cols + c, o);
  }
  if (a.part) {
    a.part[static_cast<int64_t>(blockIdx.y) * 2 * a.cols + c] = aw;
    a.part[static_cast<int64_t>(blockIdx.y) * 2 * a.cols + a.cols + c] = ab;
  }
}

// dw[c], db[c] = sums over the parts, in a fixed order: 32 columns per CTA and
// 32 threads per column, so that all of a thread's few loads are in flight at
// once (the kernel is bound by their latency).
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float* part, int parts, int cols, float* dw, float* db) {
  __shared__ float red[32][33];
  grid_dep_wait();
  const int cx = threadIdx.x & 31, sy = threadIdx.x >> 5;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 32;          // over both sums
  float s = 0.f;
  if (c0 + cx < 2ll * cols) {
    const float* p = part + c0 + cx;
#pragma unroll 5
    for (int i = sy; i < parts; i += 32) s += p[static_cast<int64_t>(i) * 2 * cols];
  }
  red[sy][cx] = s;
  __syncthreads();
  s = warp_sum(red[cx][sy]);                                         // warp sy: column c0 + sy
  const int64_t c = c0 + sy;
  if (cx == 0 && c < 2ll * cols) {
    if (c < cols) {
      if (dw) dw[c] = s;
    } else if (db) {
      db[c - cols] = s;
    }
  }
}

// ---------------------------------------------------------------- host
// Backward: CTAs (parts of the column sums) that a launch may use.
int bwd_parts() { return 4 * sm_count(); }

template <typename TX, typename TD, int VE, int NV>
int launch_bwd(const BwdArgs& a, int G, int& parts, cudaStream_t st) {
  const int P = std::max(1, 512 / G);
  const int threads = P * G;
  const size_t smem = P > 1 ? static_cast<size_t>(2) * VE * NV * G * sizeof(float) : 0;
  const int64_t groups = (a.rows + P - 1) / P;
  const int most = std::min(bwd_parts(), std::max(1, 2048 / threads) * sm_count());
  parts = static_cast<int>(std::min<int64_t>(most, groups));
  return launch_pdl(norm_bwd_kernel<TX, TD, VE, NV>, dim3(parts), dim3(threads), smem, st, a, G);
}

// Rings while a group's slots fit and every group gets two rows or more.
template <typename TX, typename TD, int VE, int NV>
bool launch_bwd_ring(const BwdArgs& a, int G, int P, int* rc, int& parts, cudaStream_t st) {
  const int slot = slot_bytes(a.cols * static_cast<int>(sizeof(TX)), VE > 1) +
                   slot_bytes(a.cols * static_cast<int>(sizeof(TD)), VE > 1);
  const int fixed = VE * NV <= BWD_KEEP ? 0 : slot_bytes((a.w_f32 ? 4 : 2) * a.cols, true);
  const int stages = std::min(MAX_STAGES, (kRingBytes - fixed) / (P * slot));
  if (stages < 2) return false;
  int* status = status_ptr();
  auto kern = norm_bwd_ring_kernel<TX, TD, VE, NV, false>;
  if constexpr (VE > 1)
    if (a.cols / VE == G * NV) kern = norm_bwd_ring_kernel<TX, TD, VE, NV, true>;
  const int smem = std::max(fixed + P * stages * slot, P > 1 ? 2 * VE * NV * G * 4 : 0);
  parts = sm_count();
  if (!status || cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
    *rc = MXQ_ERR_CUDA;
  else
    *rc = launch_pdl(kern, dim3(parts), dim3(P * G), smem, st, a, G, stages, status);
  return true;
}

template <typename TX, typename TD, int VE>
bool try_bwd_ring(const BwdArgs& a, int* rc, int& parts, cudaStream_t st) {
  constexpr int N1 = BWD_KEEP / VE, N2 = 2 * BWD_KEEP / VE;
  const int nvec = a.cols / VE;
  if (VE > 1 && (a.cols * sizeof(TX) % 16 || a.cols * sizeof(TD) % 16 || a.ld_x * sizeof(TX) % 16 ||
                 a.ld_dy * sizeof(TD) % 16))
    return false;
  const int nv = nvec <= BWD_THREADS * N1 ? N1 : N2;
  if (nvec > BWD_THREADS * N2) return false;
  const int G = round_up((nvec + nv - 1) / nv, 32), P = ring_groups(BWD_THREADS, G);
  if (a.rows < 2ll * P * sm_count()) return false;
  return nv == N1 ? launch_bwd_ring<TX, TD, VE, N1>(a, G, P, rc, parts, st)
                  : launch_bwd_ring<TX, TD, VE, N2>(a, G, P, rc, parts, st);
}

template <typename TX, typename TD, int VE>
int dispatch_bwd(const BwdArgs& a, int& parts, cudaStream_t st) {
  const int nvec = a.cols / VE;
  constexpr int N1 = VE == 1 ? 4 : 1;
  constexpr int N2 = 16 / VE;
  if (nvec <= N1 * 1024) return launch_bwd<TX, TD, VE, N1>(a, round_up((nvec + N1 - 1) / N1, 32), parts, st);
  return launch_bwd<TX, TD, VE, N2>(a, round_up((nvec + N2 - 1) / N2, 32), parts, st);
}

template <typename TX, typename TD>
int norm_bwd(const BwdArgs& a, bool vec, int& parts, cudaStream_t st) {
  if (a.cols <= kMaxBwdElems) {
    constexpr int VE = sizeof(TX) == 2 && sizeof(TD) == 2 ? 8 : 4;
    int rc;
    if (vec ? try_bwd_ring<TX, TD, VE>(a, &rc, parts, st) : try_bwd_ring<TX, TD, 1>(a, &rc, parts, st)) return rc;
    return vec ? dispatch_bwd<TX, TD, VE>(a, parts, st) : dispatch_bwd<TX, TD, 1>(a, parts, st);
  }
  const int rc = launch_pdl(norm_bwd_long_rows_kernel<TX, TD>, dim3(a.rows), dim3(1024), 0, st, a);
  if (rc) return rc;
  const int strips = (a.cols + 255) / 256;
  parts = std::max(1, std::min(std::min(a.rows, bwd_parts()), 8 * sm_count() / strips));
  return launch_pdl(norm_bwd_long_cols_kernel<TX, TD>, dim3(strips, parts), dim3(256), 0, st, a);
}

}  // namespace
}  // namespace mxq

using namespace mxq;

extern "C" int mxq_layer_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return MXQ_ERR_BAD_ARG;
  if (rows < 0 || cols < 1) return MXQ_ERR_BAD_SHAPE;
  const size_t parts = static_cast<size_t>(std::min<int64_t>(rows, bwd_parts()));
  *bytes = parts * 2 * static_cast<size_t>(cols) * sizeof(float) +
           (cols > kMaxBwdElems ? static_cast<size_t>(rows) * 2 * sizeof(float) : 0);
  return MXQ_OK;
}

extern "C" int mxq_layer_norm_backward(const void* dy, int64_t ld_dy, int dy_type, const void* x, int64_t ld_x,
                                       int x_type, int64_t rows, int64_t cols, const float* mean, const float* rstd,
                                       const void* w, int w_type, void* dx, float* dw, float* db, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (!valid_type(dy_type)) return MXQ_ERR_BAD_ARG;
  const int rc = check_norm(x, rows, cols, ld_x, x_type, w, w_type, nullptr, 0, mean, rstd);
  if (rc) return rc;
  if (ld_dy < cols) return MXQ_ERR_BAD_SHAPE;
  if (rows && (!dy || !dx)) return MXQ_ERR_BAD_ARG;
  const bool sums = dw || db;
  size_t need = 0;
  mxq_layer_norm_backward_workspace_size(rows, cols, &need);
  if (rows && (sums || cols > kMaxBwdElems) && (!workspace || workspace_bytes < need)) return MXQ_ERR_BAD_ARG;
  if (!aligned_to(dy, type_size(dy_type)) || !aligned_to(dx, type_size(x_type)) || !aligned16(workspace) ||
      !aligned_to(dw, 4) || !aligned_to(db, 4))
    return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  const auto st = static_cast<cudaStream_t>(stream);
  if (!rows) {
    if (dw && cudaMemsetAsync(dw, 0, cols * sizeof(float), st) != cudaSuccess) return MXQ_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, cols * sizeof(float), st) != cudaSuccess) return MXQ_ERR_CUDA;
    return MXQ_OK;
  }
  BwdArgs a{};
  a.dy = dy, a.ld_dy = ld_dy, a.x = x, a.ld_x = ld_x;
  a.rows = static_cast<int>(rows), a.cols = static_cast<int>(cols);
  a.mean = mean, a.rstd = rstd, a.w = w, a.w_f32 = w_type == MXQ_F32, a.dx = dx;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.coef = static_cast<float*>(workspace) + std::min<int64_t>(rows, bwd_parts()) * 2 * cols;
  const int ve = x_type == MXQ_BF16 && dy_type == MXQ_BF16 ? 8 : 4;
  const bool vec = cols % ve == 0 && ld_x % ve == 0 && ld_dy % ve == 0 && aligned16(x) && aligned16(dy) &&
                   aligned16(dx) && aligned16(w);
  int parts = 0, rc2;
  if (x_type == MXQ_BF16)
    rc2 = dy_type == MXQ_BF16 ? norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, vec, parts, st)
                              : norm_bwd<__nv_bfloat16, float>(a, vec, parts, st);
  else
    rc2 = dy_type == MXQ_BF16 ? norm_bwd<float, __nv_bfloat16>(a, vec, parts, st) : norm_bwd<float, float>(a, vec, parts, st);
  if (rc2 || !sums) return rc2;
  const int grid = static_cast<int>((2 * cols + 31) / 32);
  return launch_pdl(norm_bwd_sum_kernel, dim3(grid), dim3(1024), 0, st, static_cast<const float*>(workspace), parts,
                    a.cols, dw, db);
}
