// Global 2-norm over a list of tensors, and clipping by it:
//   n = sqrt(sum g^2),  c = min(1, max_norm / (n + 1e-6)),  out = c g.
//
// The tensors are cut into chunks that a persistent grid walks through; the
// list travels in the kernel's parameters, so nothing is copied to the device
// and nothing is kept between calls.  Both kernels are bound by HBM: the norm
// reads every element once, the scaling reads and writes it once.
#include <algorithm>

#include "rowops.cuh"

namespace mxq {
namespace {

constexpr int TPB = 256;
constexpr int DIRECT_CHUNK = 4096;                   // elements of a CTA that has one chunk
constexpr int TABLE_SMALL = 64, TABLE_LARGE = 512;   // tensors of one launch (2 KiB, 16 KiB of parameters)

struct Entry {
  const void* g;
  void* out;
  int64_t n;
  uint32_t first;          // its first chunk in the launch
  int16_t g_f32, out_f32;
};

template <int N>
struct Table {
  Entry e[N];
  uint16_t from[N / 4 + 1];  // the entry of chunk i << shift: where a search starts
  int shift;
  int count;
  uint32_t chunks;
  int chunk;                 // elements (a multiple of 8)
};

// The last entry with first <= c: its bucket's first entry, then onwards.
template <int N>
__device__ __forceinline__ int entry_of(const Table<N>& t, uint32_t c) {
  int i = t.from[c >> t.shift];
  while (i + 1 < t.count && t.e[i + 1].first <= c) ++i;
  return i;
}

// A thread's sum of squares.  Squares of ordinary values add up in float32
// over a batch and in float64 across batches; a batch whose largest value
// lies outside 2^-50 .. 2^50 (its square could overflow or vanish in float32)
// or is not finite is squared in float64.
template <int N>
__device__ __forceinline__ void add_squares(const float (&v)[N], double& acc) {
  float m = 0.f, q[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m = fmax3_nan(m, fabsf(v[i]), 0.f);
    q[i] = v[i] * v[i];
  }
  if ((m >= 0x1p-50f && m <= 0x1p50f) || m == 0.f) {
    acc += static_cast<double>(tree_sum(q));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) acc += static_cast<double>(v[i]) * static_cast<double>(v[i]);
  }
}

template <typename T>
__device__ __forceinline__ void squares_of(const T* p, int len, double& acc) {
  constexpr int VE = 16 / static_cast<int>(sizeof(T));
  constexpr int U = sizeof(T) == 2 ? 4 : 8;          // vectors in flight: 32 elements
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const int nvec = len / VE;
    for (int i = threadIdx.x; i < nvec; i += TPB * U) {
      Vec<T, VE> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        r[u].fill(0);
        if (i + u * TPB < nvec) r[u].load(p + (i + u * TPB) * VE);
      }
      float v[U * VE];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VE; ++j) v[u * VE + j] = r[u].get(j);
      add_squares(v, acc);
    }
    done = nvec * VE;
  }
  for (int i = done + threadIdx.x; i < len; i += TPB) {
    Vec<T, 1> r;
    r.load(p + i);
    const float v[1] = {r.get(0)};
    add_squares(v, acc);
  }
}

// Sum over the CTA, in thread 0.  Float64 runs at two lanes a cycle on an SM,
// so one warp finishes.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[TPB / 32];
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  v = threadIdx.x < TPB / 32 ? red[threadIdx.x] : 0.0;
#pragma unroll
  for (int o = TPB / 64; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <int N>
__global__ void __launch_bounds__(TPB) square_sum_kernel(const __grid_constant__ Table<N> t, double* part) {
  grid_dep_wait();
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = t.e[entry_of(t, c)];
    const int64_t off = static_cast<int64_t>(c - e.first) * t.chunk;
    const int len = static_cast<int>(min(static_cast<int64_t>(t.chunk), e.n - off));
    if (e.g_f32) squares_of(static_cast<const float*>(e.g) + off, len, acc);
    else squares_of(static_cast<const __nv_bfloat16*>(e.g) + off, len, acc);
  }
  const double s = block_sum(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// Root of the sum of all parts, added in a fixed order, the same in every CTA.
// The float32 root of a sum within float32's range is within an ulp of the
// float64 one and takes a fraction of its time.
__device__ __forceinline__ float norm_of(const double* part, int parts) {
  __shared__ float norm;
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += TPB) s += part[i];
  s = block_sum(s);
  if (threadIdx.x == 0) norm = s > 1e-30 && s < 1e30 ? sqrtf(static_cast<float>(s)) : static_cast<float>(sqrt(s));
  __syncthreads();
  return norm;
}

__global__ void __launch_bounds__(TPB) norm_kernel(const double* part, int parts, float* norm) {
  grid_dep_wait();
  const float n = norm_of(part, parts);
  if (threadIdx.x == 0) norm[0] = n;
}

template <typename TI, typename TO>
__device__ __forceinline__ void scale_of(const TI* p, TO* o, int len, float c) {
  constexpr int VE = sizeof(TI) == 2 && sizeof(TO) == 2 ? 8 : 4;
  constexpr int U = 4;
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(p) & (VE * sizeof(TI) - 1)) == 0 &&
      (reinterpret_cast<uintptr_t>(o) & 15 & (VE * sizeof(TO) - 1)) == 0) {
    const int nvec = len / VE;
    // rounds of U vectors at fixed distances from one address, then the rest
    int i = threadIdx.x;
#pragma unroll 1
    for (; i + (U - 1) * TPB < nvec; i += TPB * U) {
      const TI* q = p + i * VE;
      TO* d = o + i * VE;
      Vec<TI, VE> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u].load(q + u * TPB * VE);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) v[j] = r[u].get(j) * c;
        store_vec<TO, VE>(d + u * TPB * VE, v);
      }
    }
#pragma unroll 1
    for (; i < nvec; i += TPB) {
      Vec<TI, VE> r;
      r.load(p + i * VE);
      float v[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) v[j] = r.get(j) * c;
      store_vec<TO, VE>(o + i * VE, v);
    }
    done = nvec * VE;
  }
#pragma unroll 1
  for (int i = done + threadIdx.x; i < len; i += TPB) {
    Vec<TI, 1> r;
    r.load(p + i);
    const float v[1] = {r.get(0) * c};
    store_vec<TO, 1>(o + i, v);
  }
}

// Scales its chunks, last first: the chunks that the norm kernel read last are
// still in L2.  SUM: a few CTAs, each of which derives the norm from the parts
// (a short list is one launch shorter); otherwise one CTA per chunk with the
// norm given: launched in order, the chunks in flight stay close together in
// memory, which HBM rewards (402.9 M bf16 to float32: 455 us with 608 CTAs
// striding over 16384-element chunks, 355 us with one per 4096: the two passes
// move 3.22 GB in 477 us, the measured copy rate).
template <int N, bool SUM>
__global__ void __launch_bounds__(TPB, 6) scale_kernel(const __grid_constant__ Table<N> t, const double* part, int parts,
                                                    float max_norm, float* norm) {
  grid_dep_wait();
  float n;
  if constexpr (SUM) {
    n = norm_of(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = n;
  } else {
    n = norm[0];
  }
  float c = max_norm / (n + 1e-6f);
  if (c > 1.f) c = 1.f;                              // a NaN norm stays NaN
  for (uint32_t k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const uint32_t ch = t.chunks - 1 - k;
    const Entry& e = t.e[entry_of(t, ch)];
    if (e.g == e.out && c == 1.f) continue;          // in place and nothing to change
    const int64_t off = static_cast<int64_t>(ch - e.first) * t.chunk;
    const int len = static_cast<int>(min(static_cast<int64_t>(t.chunk), e.n - off));
    const float* gf = static_cast<const float*>(e.g) + off;
    const __nv_bfloat16* gb = static_cast<const __nv_bfloat16*>(e.g) + off;
    float* of = static_cast<float*>(e.out) + off;
    __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(e.out) + off;
    if (e.g_f32) {
      if (e.out_f32) scale_of(gf, of, len, c);
      else scale_of(gf, ob, len, c);
    } else {
      if (e.out_f32) scale_of(gb, of, len, c);
      else scale_of(gb, ob, len, c);
    }
  }
}

using namespace mxq_host;

int grid_limit() { return 4 * sm_count(); }

int check_grads(const mxq_grad* g, int n, bool clip) {
  if (n < 0 || (n && !g)) return MXQ_ERR_BAD_ARG;
  for (int i = 0; i < n; ++i) {
    if (g[i].n < 0 || g[i].n > (1ll << 42)) return MXQ_ERR_BAD_SHAPE;
    if (g[i].g_type != MXQ_BF16 && g[i].g_type != MXQ_F32) return MXQ_ERR_BAD_ARG;
    if (clip && g[i].out_type != MXQ_BF16 && g[i].out_type != MXQ_F32) return MXQ_ERR_BAD_ARG;
    if (!g[i].n) continue;
    if (!g[i].g || (clip && !g[i].out)) return MXQ_ERR_BAD_ARG;
    if (clip && g[i].g == g[i].out && g[i].g_type != g[i].out_type) return MXQ_ERR_BAD_ARG;
    if (reinterpret_cast<uintptr_t>(g[i].g) & (g[i].g_type == MXQ_F32 ? 3 : 1)) return MXQ_ERR_MISALIGNED;
    if (clip && (reinterpret_cast<uintptr_t>(g[i].out) & (g[i].out_type == MXQ_F32 ? 3 : 1))) return MXQ_ERR_MISALIGNED;
  }
  return MXQ_OK;
}

// Elements of a chunk: enough chunks for every CTA to have several, 2048 (one
// round of a CTA's loads) to 16384.
int chunk_size(int64_t total) {
  const int64_t want = total / (4ll * grid_limit());
  return want >= 16384 ? 16384 : want >= 8192 ? 8192 : want >= 4096 ? 4096 : 2048;
}

// Fills t with entries from *i on, as many as fit; false when none is left.
template <int N>
bool next_table(const mxq_grad* g, int n, int chunk, int* i, Table<N>& t) {
  t.count = 0;
  t.chunks = 0;
  t.chunk = chunk;
  for (; *i < n && t.count < N; ++*i) {
    const mxq_grad& s = g[*i];
    if (!s.n) continue;
    const int64_t c = (s.n + chunk - 1) / chunk;
    if (t.chunks + c > 0x7FFFFFFF) break;
    t.e[t.count++] = Entry{s.g, s.out, s.n, t.chunks, static_cast<int16_t>(s.g_type == MXQ_F32),
                           static_cast<int16_t>(s.out_type == MXQ_F32)};
    t.chunks += static_cast<uint32_t>(c);
  }
  t.shift = 0;
  while ((t.chunks >> t.shift) > N / 4) ++t.shift;
  for (uint32_t b = 0, k = 0; t.count && b <= (t.chunks - 1) >> t.shift; ++b) {
    while (k + 1 < static_cast<uint32_t>(t.count) && t.e[k + 1].first <= b << t.shift) ++k;
    t.from[b] = static_cast<uint16_t>(k);
  }
  return t.count > 0;
}

template <int N>
int run(const mxq_grad* g, int n, int64_t total, bool clip, float max_norm, float* norm, double* part, cudaStream_t st) {
  const int chunk = chunk_size(total);
  Table<N> t;
  int parts = 0;
  for (int i = 0; next_table(g, n, chunk, &i, t);) {
    const int grid = static_cast<int>(std::min<int64_t>(t.chunks, grid_limit()));
    const int rc = launch_pdl(square_sum_kernel<N>, dim3(grid), dim3(TPB), 0, st, t, part + parts);
    if (rc) return rc;
    parts += grid;
  }
  const bool direct = total > 16ll * grid_limit() * 2048;       // every CTA of the norm kernel had 16 rounds or more
  if (!clip || !parts || direct) {
    const int rc = launch_pdl(norm_kernel, dim3(1), dim3(TPB), 0, st, static_cast<const double*>(part), parts, norm);
    if (rc || !clip || !parts) return rc;
  }
  for (int i = 0; next_table(g, n, direct ? DIRECT_CHUNK : chunk, &i, t);) {
    const double* p = part;
    const int rc = direct ? launch_pdl(scale_kernel<N, false>, dim3(t.chunks), dim3(TPB), 0, st, t, p, parts, max_norm, norm)
                          : launch_pdl(scale_kernel<N, true>, dim3(std::min<int64_t>(t.chunks, grid_limit())), dim3(TPB), 0,
                                       st, t, p, parts, max_norm, norm);
    if (rc) return rc;
  }
  return MXQ_OK;
}

int grad_call(const mxq_grad* g, int n, bool clip, float max_norm, float* norm, void* ws, size_t bytes, void* stream) {
  if (!norm) return MXQ_ERR_BAD_ARG;
  const int rc = check_grads(g, n, clip);
  if (rc) return rc;
  if (clip && !(max_norm >= 0.f)) return MXQ_ERR_BAD_ARG;
  size_t need = 0;
  mxq_grad_norm_workspace_size(n, &need);
  if (!ws || bytes < need) return MXQ_ERR_BAD_ARG;
  if ((reinterpret_cast<uintptr_t>(norm) & 3) || !aligned16(ws)) return MXQ_ERR_MISALIGNED;
  if (!device_ok()) return MXQ_ERR_UNSUPPORTED;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += g[i].n;
  const auto st = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  return n <= TABLE_SMALL ? run<TABLE_SMALL>(g, n, total, clip, max_norm, norm, part, st)
                          : run<TABLE_LARGE>(g, n, total, clip, max_norm, norm, part, st);
}

}  // namespace
}  // namespace mxq

extern "C" int mxq_grad_norm_workspace_size(int ntensors, size_t* bytes) {
  if (!bytes || ntensors < 0) return MXQ_ERR_BAD_ARG;
  // every launch fills its table up, short of a list of more than 2^31 chunks
  const size_t launches = static_cast<size_t>(ntensors) / mxq::TABLE_LARGE + 2;
  *bytes = launches * mxq::grid_limit() * sizeof(double);
  return MXQ_OK;
}

extern "C" int mxq_grad_norm(const mxq_grad* grads, int ntensors, float* norm, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return mxq::grad_call(grads, ntensors, false, 0.f, norm, workspace, workspace_bytes, stream);
}

extern "C" int mxq_clip_grad_norm(const mxq_grad* grads, int ntensors, float max_norm, float* norm, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return mxq::grad_call(grads, ntensors, true, max_norm, norm, workspace, workspace_bytes, stream);
}
