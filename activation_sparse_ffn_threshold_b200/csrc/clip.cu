// clip.cu -- the norm of all gradients together, and their clipping.
//
//     n = scale * sqrt(sum over all tensors of g^2),   out = g * scale * min(1, max_norm / (n + eps))
//
// Two kernels: k_grad_squares adds up squares, a partial sum per CTA; every CTA of k_grad_scale
// adds the partial sums up again in the same order (no atomics: the result depends on the tensors'
// sizes, types and alignments alone) and multiplies its share of the values.  The tensors' table travels in the kernels'
// parameters, so nothing is copied to the device and a captured call holds its own table.
//
// Bound by bytes: each value is read twice and written once.  Measured: 1.08 GB in 20 bf16
// tensors, into others, 515 us (the bytes 496), 270 MB 126; the squares alone 169 for 1.08 GB (6.4 TB/s).
#include <algorithm>
#include <cmath>
#include <new>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                               // 16-byte vectors a thread requests at a time
constexpr int kRounds = 2;                             // such requests to a chunk, one ahead of its use
constexpr int kChunkBytes = kThreads * kVecs * 16 * kRounds;  // a CTA's piece of work

template <int CAP>
struct ClipTable {
  const void *in[CAP];
  void *out[CAP];
  int64_t numel[CAP];
  uint32_t first[CAP + 1];  // its first chunk
  uint8_t type[CAP];        // sfnn_dtype
  int count;
};
struct ClipArgs {
  double *partial;
  int partials;       // of all tables
  float max_norm, scale, eps;
  float *norm;        // written by the launch that has it
};

// A chunk's values lie in [lo, hi) of tensor `t`.
struct Chunk {
  int t;
  int64_t lo, hi;
};
__host__ __device__ constexpr int elem_bytes(int type) { return type == SFNN_F32 ? 4 : 2; }
// `t`: a tensor near by (the chunk before's).
template <int CAP>
__device__ __forceinline__ Chunk chunk_at(const ClipTable<CAP> &tab, uint32_t c, int t) {
  while (tab.first[t + 1] <= c) ++t;
  while (tab.first[t] > c) --t;
  const int per = kChunkBytes / elem_bytes(tab.type[t]);
  Chunk k;
  k.t = t;
  k.lo = (int64_t)(c - tab.first[t]) * per;
  k.hi = min(k.lo + per, tab.numel[t]);
  return k;
}
// The tensor of chunk c, from nothing.
template <int CAP>
__device__ __forceinline__ int tensor_at(const ClipTable<CAP> &tab, uint32_t c) {
  int lo = 0, hi = tab.count;  // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int TYPE>
__device__ __forceinline__ void widen(const uint4 &w, float *v) {
  if (TYPE == SFNN_F32) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16(u[i], TYPE == SFNN_BF16);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <int TYPE>
__device__ __forceinline__ float load_one(const void *p, int64_t i) {
  return TYPE == SFNN_F32 ? static_cast<const float *>(p)[i] : load16(p, i, TYPE == SFNN_BF16);
}

// The squares of up to 8 values: in 32 bits where their sum can be neither near overflow nor
// made of numbers that squaring loses (16-bit and fp32 gradients in earnest), else in 64.
template <int N>
__device__ __forceinline__ double squares(const float *v) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(v[i], v[i], s);
  if (s > 0x1p-60f && s < 0x1p120f) return s;
  double q = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) q = fma((double)v[i], (double)v[i], q);
  return q;
}

// Values before the first 16-byte boundary at or after `p` (elements of E bytes).
template <int E>
__device__ __forceinline__ int head_of(const void *p) {
  return (int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / E;
}

// What L2 should do with a line that is read: let it go first, or keep it, as the last kKeep chunks (40
// MB), which the scaling reads first.  (270 MB of bf16, both kernels: 4 % less time than with all
// lines let go first; 100 MB kept: none.)
constexpr uint32_t kKeep = 40u * 1024 * 1024 / kChunkBytes;
__device__ __forceinline__ uint64_t policy_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_last() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 ld_hint(const void *p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}

template <int TYPE>
__device__ __forceinline__ double chunk_squares(const void *base, int64_t lo, int64_t hi, uint64_t policy) {
  constexpr int E = TYPE == SFNN_F32 ? 4 : 2, N = 16 / E;
  const char *p = static_cast<const char *>(base) + lo * E;
  const int n = (int)(hi - lo);
  const int head = min(head_of<E>(p), n), vecs = (n - head) / N;
  const uint4 *v = reinterpret_cast<const uint4 *>(p + head * E);
  double sum = 0.0;
  uint4 w[2][kVecs];
  auto request = [&](int round) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int k = threadIdx.x + (round * kVecs + i) * kThreads;
      w[round & 1][i] = k < vecs ? ld_hint(v + k, policy) : make_uint4(0, 0, 0, 0);
    }
  };
  request(0);
#pragma unroll
  for (int round = 0; round < kRounds; ++round) {
    if (round + 1 < kRounds) request(round + 1);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float f[N];
      widen<TYPE>(w[round & 1][i], f);
      if (threadIdx.x + (round * kVecs + i) * kThreads < vecs) sum += squares<N>(f);
    }
  }
  const int rest = n - vecs * N;  // the head's, then the tail's
  if ((int)threadIdx.x < rest) {
    const int i = (int)threadIdx.x < head ? threadIdx.x : threadIdx.x + vecs * N;
    const float f = load_one<TYPE>(p, i);
    sum += squares<1>(&f);
  }
  return sum;
}

__device__ __forceinline__ double block_sum(double v) {  // the whole CTA; every thread gets it
  __shared__ double s[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) v += s[i];
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) k_grad_squares(const __grid_constant__ ClipTable<CAP> tab,
                                                           double *__restrict__ partial) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  const uint32_t chunks = tab.first[tab.count];
  int t = blockIdx.x < chunks ? tensor_at(tab, blockIdx.x) : 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = chunk_at(tab, c, t);
    t = k.t;
    const int type = tab.type[k.t];
    const void *in = tab.in[k.t];
    const uint64_t policy = c + kKeep < chunks ? policy_first() : policy_last();
    sum += type == SFNN_F32    ? chunk_squares<SFNN_F32>(in, k.lo, k.hi, policy)
           : type == SFNN_BF16 ? chunk_squares<SFNN_BF16>(in, k.lo, k.hi, policy)
                               : chunk_squares<SFNN_F16>(in, k.lo, k.hi, policy);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <int TYPE>
__device__ __forceinline__ void store_one(void *p, int64_t i, float v) {
  if (TYPE == SFNN_F32)
    static_cast<float *>(p)[i] = v;
  else
    static_cast<uint16_t *>(p)[i] = (uint16_t)pack16(v, 0.f, TYPE == SFNN_BF16);
}
template <int TYPE>
__device__ __forceinline__ uint4 scaled(const uint4 &w, float k) {
  constexpr int N = TYPE == SFNN_F32 ? 4 : 8;
  float f[N];
  widen<TYPE>(w, f);
  if (TYPE == SFNN_F32)
    return make_uint4(__float_as_uint(f[0] * k), __float_as_uint(f[1] * k), __float_as_uint(f[2] * k),
                      __float_as_uint(f[3] * k));
  constexpr bool b = TYPE == SFNN_BF16;
  return make_uint4(pack16(f[0] * k, f[1] * k, b), pack16(f[2] * k, f[3] * k, b), pack16(f[N - 4] * k, f[N - 3] * k, b),
                    pack16(f[N - 2] * k, f[N - 1] * k, b));
}
template <int TYPE>
__device__ __forceinline__ void chunk_scale(const void *base, void *to, int64_t lo, int64_t hi, float k) {
  constexpr int E = TYPE == SFNN_F32 ? 4 : 2, N = 16 / E;
  const char *p = static_cast<const char *>(base) + lo * E;
  char *q = static_cast<char *>(to) + lo * E;
  const int n = (int)(hi - lo);
  // vectors where both sides reach a 16-byte boundary together
  const bool together = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
  if (!together) {
    for (int i = threadIdx.x; i < n; i += kThreads) store_one<TYPE>(q, i, load_one<TYPE>(p, i) * k);
    return;
  }
  const int head = min(head_of<E>(p), n), vecs = (n - head) / N;
  const uint4 *v = reinterpret_cast<const uint4 *>(p + head * E);
  uint4 *o = reinterpret_cast<uint4 *>(q + head * E);
#pragma unroll 1
  for (int at = threadIdx.x; at < kVecs * kRounds * kThreads; at += kVecs * kThreads) {
    uint4 w[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (at + i * kThreads < vecs) w[i] = v[at + i * kThreads];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (at + i * kThreads < vecs) __stcs(o + at + i * kThreads, scaled<TYPE>(w[i], k));
  }
  const int rest = n - vecs * N;
  if ((int)threadIdx.x < rest) {
    const int i = (int)threadIdx.x < head ? threadIdx.x : threadIdx.x + vecs * N;
    store_one<TYPE>(q, i, load_one<TYPE>(p, i) * k);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) k_grad_scale(const __grid_constant__ ClipTable<CAP> tab,
                                                         const __grid_constant__ ClipArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  for (int i = threadIdx.x; i < a.partials; i += kThreads) sum += __ldcg(a.partial + i);
  const float n = (float)((double)a.scale * sqrt(block_sum(sum)));
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = n;
  const float q = a.max_norm / (n + a.eps);
  const float k = a.scale * (q >= 1.f ? 1.f : q);  // (a NaN stays one)
  // the values read last by the sums are read first here: L2 holds some of them
  const int64_t chunks = tab.first[tab.count], step = gridDim.x;
  if ((int64_t)blockIdx.x >= chunks) return;
  int64_t c = blockIdx.x + (chunks - 1 - blockIdx.x) / step * step;
  for (int t = tensor_at(tab, (uint32_t)c); c >= 0; c -= step) {
    const Chunk w = chunk_at(tab, (uint32_t)c, t);
    t = w.t;
    const void *in = tab.in[w.t];
    void *out = tab.out[w.t];
    if (in == out && k == 1.f) continue;
    const int type = tab.type[w.t];
    if (type == SFNN_F32)
      chunk_scale<SFNN_F32>(in, out, w.lo, w.hi, k);
    else if (type == SFNN_BF16)
      chunk_scale<SFNN_BF16>(in, out, w.lo, w.hi, k);
    else
      chunk_scale<SFNN_F16>(in, out, w.lo, w.hi, k);
  }
}

// A table's tensors; wide tables cost a launch more to carry (their bytes are copied with it).
constexpr int kSmall = 64, kLarge = 960;
constexpr int kCtasPerSm = 8;

template <int CAP>
void fill(ClipTable<CAP> &tab, const sfnn_grad *g, int count) {
  uint32_t chunks = 0;
  tab.count = count;
  for (int i = 0; i < count; ++i) {
    tab.in[i] = g[i].in;
    tab.out[i] = g[i].out;
    tab.numel[i] = g[i].numel;
    tab.type[i] = (uint8_t)g[i].dtype;
    tab.first[i] = chunks;
    const int64_t per = kChunkBytes / elem_bytes((int)g[i].dtype);
    chunks += (uint32_t)((g[i].numel + per - 1) / per);
  }
  tab.first[count] = chunks;
}
template <int CAP>
cudaError_t launch_squares(const sfnn_grad *g, int count, int grid, double *partial, cudaStream_t s) {
  ClipTable<CAP> tab;
  fill(tab, g, count);
  return launch_pdl(k_grad_squares<CAP>, dim3(grid), dim3(kThreads), 0, s, tab, partial);
}
template <int CAP>
cudaError_t launch_scale(const sfnn_grad *g, int count, int grid, const ClipArgs &a, cudaStream_t s) {
  ClipTable<CAP> tab;
  fill(tab, g, count);
  return launch_pdl(k_grad_scale<CAP>, dim3(grid), dim3(kThreads), 0, s, tab, a);
}

int64_t chunks_of(const sfnn_grad *g, int count) {
  int64_t n = 0;
  for (int i = 0; i < count; ++i) n += (g[i].numel * elem_bytes((int)g[i].dtype) + kChunkBytes - 1) / kChunkBytes;
  return n;
}
int grid_of(const sfnn_grad *g, int count, int sms) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks_of(g, count), (int64_t)sms * kCtasPerSm));
}

// Whether something that is written, the norm and the workspace among it, overlaps something else that is
// written or read.
struct Span {
  uintptr_t lo, hi;
  bool written;
};
sfnn_status overlaps(const sfnn_grad *g, int count, const float *norm, const void *ws, int64_t ws_bytes) {
  Span *s = new (std::nothrow) Span[2 * (size_t)count + 2];
  if (!s) return SFNN_ERR_OOM;
  size_t n = 0;
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm), work = reinterpret_cast<uintptr_t>(ws);
  s[n++] = {at, at + 4, true};
  s[n++] = {work, work + (uintptr_t)ws_bytes, true};
  for (int i = 0; i < count; ++i) {
    if (!g[i].numel) continue;
    const uintptr_t bytes = (uintptr_t)g[i].numel * elem_bytes((int)g[i].dtype);
    const uintptr_t in = reinterpret_cast<uintptr_t>(g[i].in), out = reinterpret_cast<uintptr_t>(g[i].out);
    if (in != out) s[n++] = {in, in + bytes, false};
    s[n++] = {out, out + bytes, true};
  }
  std::sort(s, s + n, [](const Span &a, const Span &b) { return a.lo < b.lo; });
  uintptr_t end = 0, written_end = 0;
  bool bad = false;
  for (size_t i = 0; i < n; ++i) {
    bad = bad || s[i].lo < (s[i].written ? end : written_end);
    end = std::max(end, s[i].hi);
    if (s[i].written) written_end = std::max(written_end, s[i].hi);
  }
  delete[] s;
  return bad ? SFNN_ERR_INVALID_ARG : SFNN_OK;
}

}  // namespace
}  // namespace sfnn

using namespace sfnn;

extern "C" {

int64_t sfnn_clip_workspace(int32_t count) {
  if (count < 0) return -1;
  return std::max<int64_t>(1, (count + kLarge - 1) / kLarge) * std::max(device_sms(), 1) * kCtasPerSm * 8;
}

sfnn_status sfnn_clip_grad_norm(const sfnn_grad *grads, int32_t count, float max_norm, float scale, float eps, float *norm,
                                void *ws, int64_t ws_bytes, sfnn_stream_t stream) {
  if (count < 0 || (count && !grads) || !(max_norm >= 0.f) || !std::isfinite(scale) || scale < 0.f || !(eps >= 0.f))
    return SFNN_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const sfnn_grad &g = grads[i];
    if (g.dtype != SFNN_F32 && g.dtype != SFNN_F16 && g.dtype != SFNN_BF16) return SFNN_ERR_INVALID_ARG;
    if (g.numel < 0) return SFNN_ERR_INVALID_ARG;
    if (g.numel > (1ll << 40)) return SFNN_ERR_UNSUPPORTED;
    const uintptr_t odd = (uintptr_t)elem_bytes((int)g.dtype) - 1;
    if (g.numel && (!g.in || !g.out || (reinterpret_cast<uintptr_t>(g.in) & odd) || (reinterpret_cast<uintptr_t>(g.out) & odd)))
      return SFNN_ERR_INVALID_ARG;
  }
  if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u) || !ws || (reinterpret_cast<uintptr_t>(ws) & 7u) ||
      ws_bytes < sfnn_clip_workspace(count))
    return SFNN_ERR_INVALID_ARG;
  if (chunks_of(grads, count) > 0x7fffffffll) return SFNN_ERR_UNSUPPORTED;
  const sfnn_status st = overlaps(grads, count, norm, ws, sfnn_clip_workspace(count));
  if (st != SFNN_OK) return st;
  const int sms = device_sms();
  if (sms < 1) return SFNN_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ClipArgs a{};
  a.partial = static_cast<double *>(ws);
  a.max_norm = max_norm;
  a.scale = scale;
  a.eps = eps;
  const int tables = std::max(1, (count + kLarge - 1) / kLarge);
  auto part = [&](int t, const sfnn_grad *&g, int &n) {
    g = grads + (size_t)t * kLarge;
    n = std::min(kLarge, count - t * kLarge);
    return grid_of(g, n, sms);
  };
  const sfnn_grad *g;
  int n;
  for (int t = 0; t < tables; ++t) {
    const int grid = part(t, g, n);
    const cudaError_t e = n <= kSmall ? launch_squares<kSmall>(g, n, grid, a.partial + a.partials, s)
                                      : launch_squares<kLarge>(g, n, grid, a.partial + a.partials, s);
    if (e != cudaSuccess) return SFNN_ERR_CUDA;
    a.partials += grid;
  }
  for (int t = tables; t-- > 0;) {
    const int grid = part(t, g, n);
    a.norm = t == 0 ? norm : nullptr;
    const cudaError_t e = n <= kSmall ? launch_scale<kSmall>(g, n, grid, a, s) : launch_scale<kLarge>(g, n, grid, a, s);
    if (e != cudaSuccess) return SFNN_ERR_CUDA;
  }
  return SFNN_OK;
}

}  // extern "C"
