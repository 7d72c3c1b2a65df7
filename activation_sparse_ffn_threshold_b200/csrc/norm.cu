// norm.cu -- the norms around a block, with its gate and residual scale, forward and backward.
//
//     R = a X + c gate * post(Z),   H = pre(R)
//     pre, post:  v^ = v rsqrt(mean v^2 + eps)  or  (v - mean v) rsqrt(var v + eps),  v^ * w + b
//
// Backward, a row at a time, from dR, dH and the forward pass's means and reciprocal deviations:
//
//     u = dH w,   D = dR + s (u - [layer] mean u - R^ mean(u R^)),   dX = a D
//     q = c D,    dgate = q post(Z),   p = q gate,   v = p w_post
//     dZ = s_z (v - [layer] mean v - Z^ mean(v Z^))
//     dw = sum dH R^,  db = sum dH,  dw_post = sum p Z^,  db_post = sum p   (over the rows)
//
// R is formed again from X and Z (which the backward pass reads anyway) and not read back: R
// rounded to its type would add its rounding to dw.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"
#include "norm.cuh"

namespace sfnn {
namespace {

// ---------------------------------------------------------------- a thread's values
// Rows that start on 16 bytes and whose length is a multiple of 8 are read by vectors of 8
// values; others value by value.  A thread's `V` values from vector (or value) `k` on.
// (X may be written where it was read: no read-only loads.)
__device__ __forceinline__ uint4 ld_row(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// WIDE: values of a row (16 or 32 bits), else 16-bit weights or gates.
template <bool WIDE, int V>
__device__ __forceinline__ void load_values(const void *p, int64_t at, int type32, bool bf16, float *v) {
  if (V == 8) {
    if (WIDE && type32) {
      const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + at);
      const uint4 a = ld_row(q), b = ld_row(q + 1);
      v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    } else {
      const uint16_t *q = static_cast<const uint16_t *>(p) + at;
      const uint4 a = WIDE ? ld_row(q) : ld_keep(q);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16(u[i], bf16);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      }
    }
  } else {
    v[0] = WIDE && type32 ? static_cast<const float *>(p)[at] : load16(p, at, bf16);
  }
}
template <bool WIDE, int V>
__device__ __forceinline__ void store_values(void *p, int64_t at, int type32, bool bf16, const float *v) {
  if (V == 8) {
    if (WIDE && type32) {
      float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) =
          make_uint4(pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16), pack16(v[4], v[5], bf16), pack16(v[6], v[7], bf16));
    }
  } else if (WIDE && type32) {
    static_cast<float *>(p)[at] = v[0];
  } else {
    static_cast<uint16_t *>(p)[at] = (uint16_t)pack16(v[0], 0.f, bf16);
  }
}

// ---------------------------------------------------------------- sums over a row
constexpr int kMaxCluster = 8;  // CTAs that share a row (the portable size)
constexpr int kMaxWarps = 16;  // of a CTA

// A row belongs to `warps` warps of the CTA, all rows of a CTA in step, or (CLUSTER) to all warps of
// `ctas` CTAs, which then write their warps' sums into each other's shared memory.  The sums of N
// values; the buffers alternate, so one barrier a sum is enough: who writes a buffer again has passed
// the barrier of the sum between, which every reader of it reached after reading.
template <bool CLUSTER>
struct RowSum {
  static constexpr int kSlots = CLUSTER ? kMaxCluster * kMaxWarps : kMaxWarps;
  float2 *slots;  // [2][kSlots]
  int warps, ctas, rank, turn;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N == 1 || N == 2, "a slot holds two");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    spread<N, 16>(v);
    if (!CLUSTER && warps == 1) return;
    float2 *s = slots + turn * kSlots;
    turn ^= 1;
    const float2 own = make_float2(v[0], v[N - 1]);
    if (CLUSTER) {
      if (lane < ctas)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_addr(s + rank * warps + warp, lane)),
                     "f"(own.x), "f"(own.y)
                     : "memory");
      __syncwarp();
      cluster_sync_all();
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = 0.f;
      for (int i = lane; i < warps * ctas; i += 32) {
        v[0] += s[i].x;
        if (N == 2) v[N - 1] += s[i].y;
      }
      spread<N, 16>(v);
    } else {
      if (lane == 0) s[warp] = own;
      __syncthreads();
      // every lane takes a warp's sum (16 of them, twice over), and they are added up again
      const int i = lane & 15;
      const float2 part = i < warps ? s[warp / warps * warps + i] : make_float2(0.f, 0.f);
      v[0] = part.x;
      if (N == 2) v[N - 1] = part.y;
      spread<N, 8>(v);
    }
  }

 private:
  template <int N, int FROM>
  __device__ __forceinline__ void spread(float (&v)[N]) {
#pragma unroll
    for (int o = FROM; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  }
};

// Where a thread stands: its place in the row's threads, and the row.
template <bool CLUSTER>
struct Place {
  int lane, groups, mine, ctas, rank;  // groups of threads in the CTA, each with its row
  int64_t unit, units;                 // CTAs, or clusters
  __device__ __forceinline__ explicit Place(int threads) {
    ctas = CLUSTER ? threads / (int)blockDim.x : 1;
    rank = CLUSTER ? (int)cluster_rank() : 0;
    lane = CLUSTER ? rank * (int)blockDim.x + (int)threadIdx.x : (int)threadIdx.x % threads;
    groups = CLUSTER ? 1 : (int)blockDim.x / threads;
    mine = CLUSTER ? 0 : (int)threadIdx.x / threads;
    unit = CLUSTER ? blockIdx.x / ctas : blockIdx.x;
    units = CLUSTER ? gridDim.x / ctas : gridDim.x;
  }
  __device__ __forceinline__ RowSum<CLUSTER> sums(float2 *slots, int threads) const {
    return {slots, CLUSTER ? (int)blockDim.x / 32 : threads / 32, ctas, rank, 0};
  }
};

// ---------------------------------------------------------------- forward
// NV vectors of V values a thread, a row to `threads` threads of a CTA (CLUSTER: of all the cluster's).
// Bound by latency at the few rows it serves: loads, then a chain of sums.  1 x 4096 fp32, RMS: 4 us in a
// row of launches, 5.6 with the call.
template <bool bf16, int V, int NV, bool CLUSTER>
__global__ void __launch_bounds__(256, 2) k_norm_forward(const __grid_constant__ NormParams P, int threads) {
  __shared__ float2 slots[2 * RowSum<CLUSTER>::kSlots];
  pdl_wait();
  pdl_launch_dependents();
  const Place<CLUSTER> at(threads);
  const int lane = at.lane;
  const int64_t row = at.unit * at.groups + at.mine;
  const bool live = row < P.T;
  RowSum<CLUSTER> sum = at.sums(slots, threads);
  if (CLUSTER) cluster_sync_all();  // the others have started before a sum is written to them
  float x[NV * V], z[NV * V];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (lane + k * threads) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) x[k * V + i] = z[k * V + i] = 0.f;
    if (live && c < P.d) {
      load_values<true, V>(P.x, row * P.ldx + c, P.x32, bf16, x + k * V);
      if (P.z) load_values<true, V>(P.z, row * P.ldz + c, P.z32, bf16, z + k * V);
    }
  }
  // the row's mean and reciprocal deviation; columns past d hold zeros
  auto stats = [&](const float *v, int kind) {
    float m = 0.f, q = 0.f;
    if (kind == SFNN_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < NV * V; ++i) m += v[i];
      float t[1] = {m};
      sum(t);
      m = t[0] * P.inv_d;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((lane + k * threads) * V < P.d)
#pragma unroll
        for (int i = 0; i < V; ++i) q = fmaf(v[k * V + i] - m, v[k * V + i] - m, q);
    float t[1] = {q};
    sum(t);
    return make_float2(m, rsqrtf(t[0] * P.inv_d + P.eps));
  };
  float2 of_z = make_float2(0.f, 1.f), of_r = make_float2(0.f, 1.f);
  if (P.z) {
    if (P.post != SFNN_NORM_NONE) of_z = stats(z, P.post);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * threads) * V;
      if (!live || c >= P.d) continue;
      float g[V], w[V], b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = w[i] = 1.f, b[i] = 0.f;
      if (P.gate) load_values<false, V>(P.gate, row * P.ldg + c, 0, bf16, g);
      if (P.wp) load_values<false, V>(P.wp, c, 0, bf16, w);
      if (P.bp) load_values<false, V>(P.bp, c, 0, bf16, b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float p = fmaf((z[k * V + i] - of_z.x) * of_z.y, w[i], b[i]);
        x[k * V + i] = fmaf(P.c * g[i], p, P.a * x[k * V + i]);
      }
      store_values<true, V>(P.r, row * P.ldr + c, P.x32, bf16, x + k * V);
    }
  }
  if (P.pre != SFNN_NORM_NONE) {
    of_r = stats(x, P.pre);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * threads) * V;
      if (!live || c >= P.d) continue;
      float w[V], b[V];
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = 1.f, b[i] = 0.f;
      if (P.w) load_values<false, V>(P.w, c, 0, bf16, w);
      if (P.b) load_values<false, V>(P.b, c, 0, bf16, b);
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = fmaf((x[k * V + i] - of_r.x) * of_r.y, w[i], b[i]);
      store_values<false, V>(P.h, row * P.ldh + c, 0, bf16, w);
    }
  }
  if (P.stats && live && lane == 0)
    *reinterpret_cast<float4 *>(P.stats + row * 4) = make_float4(of_r.x, of_r.y, of_z.x, of_z.y);
}

// ---------------------------------------------------------------- backward
// Rows too long for the way through shared memory, which takes up to 8192 values whatever the types (512 threads
// of 16): 8 values a thread, a row to the threads of a cluster, rows dealt to the clusters in turn, their
// columns' sums in registers.  FULL: all four, else dw and S1 alone.  Bound by latency, as nothing is on its way
// while a row's sums go round: 4000 x 8200 bf16 both norms RMS 397 us, LayerNorm and RMS 1000 (8192 wide through shared
// memory 88 and 138, and with an fp32 stream, of which one row fits at a time, 148 and 199).
template <bool bf16, int V, bool FULL>
__global__ void __launch_bounds__(512, FULL ? 1 : 2) k_norm_backward(const __grid_constant__ NormBackParams P, int threads) {
  constexpr int NV = 8 / V;
  __shared__ float2 slots[2 * RowSum<true>::kSlots];
  pdl_wait();
  pdl_launch_dependents();
  const NormParams &F = P.f;
  const Place<true> at(threads);
  const int lane = at.lane;
  RowSum<true> sum = at.sums(slots, threads);
  cluster_sync_all();  // the others have started before a sum is written to them
  float sw[8], sb[FULL ? 8 : 1], sum1[8], sum0[FULL ? 8 : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sw[i] = sum1[i] = 0.f;
    if (FULL) sb[i] = sum0[i] = 0.f;
  }
  for (int64_t row = at.unit; row < F.T; row += at.units) {
    float x[8], z[8], dr[8], dh[8];
    const float4 st = __ldg(reinterpret_cast<const float4 *>(F.stats) + row);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * threads) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) x[k * V + i] = z[k * V + i] = dr[k * V + i] = dh[k * V + i] = 0.f;
      if (c >= F.d) continue;
      load_values<true, V>(F.x, row * F.ldx + c, F.x32, bf16, x + k * V);
      if (F.z) load_values<true, V>(F.z, row * F.ldz + c, F.z32, bf16, z + k * V);
      if (P.dr) load_values<true, V>(P.dr, row * P.lddr + c, F.x32, bf16, dr + k * V);
      if (P.dh) load_values<false, V>(P.dh, row * P.lddh + c, 0, bf16, dh + k * V);
    }
    // z becomes Z^, x R^
    if (F.z) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (lane + k * threads) * V;
        if (c >= F.d) continue;
        float g[V], w[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = w[i] = 1.f, b[i] = 0.f;
        if (F.gate) load_values<false, V>(F.gate, row * F.ldg + c, 0, bf16, g);
        if (F.wp) load_values<false, V>(F.wp, c, 0, bf16, w);
        if (F.bp) load_values<false, V>(F.bp, c, 0, bf16, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          z[k * V + i] = (z[k * V + i] - st.z) * st.w;
          x[k * V + i] = fmaf(F.c * g[i], fmaf(z[k * V + i], w[i], b[i]), F.a * x[k * V + i]);
        }
      }
    }
    if (P.dh) {
      float u[8], s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (lane + k * threads) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) u[k * V + i] = 0.f;
        if (c >= F.d) continue;
        float w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = 1.f;
        if (F.w) load_values<false, V>(F.w, c, 0, bf16, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int j = k * V + i;
          x[j] = (x[j] - st.x) * st.y;
          u[j] = dh[j] * w[i];
          s1 += u[j];
          s2 = fmaf(u[j], x[j], s2);
          sw[j] = fmaf(dh[j], x[j], sw[j]);
          if (FULL) sb[j] += dh[j];
        }
      }
      float s[2] = {s1, s2};
      sum(s);
      const float m1 = F.pre == SFNN_NORM_LAYER ? s[0] * F.inv_d : 0.f, m2 = s[1] * F.inv_d;
#pragma unroll
      for (int j = 0; j < 8; ++j) dr[j] = fmaf(st.y, u[j] - fmaf(x[j], m2, m1), dr[j]);
    }
    if (P.dx)
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = (lane + k * threads) * V;
        if (c >= F.d) continue;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = F.a * dr[k * V + i];
        store_values<true, V>(P.dx, row * F.d + c, F.x32, bf16, v);
      }
    if (!F.z) continue;
    float n1 = 0.f, n2 = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * threads) * V;
      if (c >= F.d) {
#pragma unroll
        for (int i = 0; i < V; ++i) dr[k * V + i] = 0.f;
        continue;
      }
      float g[V], w[V], b[V], dg[V];
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = w[i] = 1.f, b[i] = 0.f;
      if (F.gate) load_values<false, V>(F.gate, row * F.ldg + c, 0, bf16, g);
      if (F.wp) load_values<false, V>(F.wp, c, 0, bf16, w);
      if (F.bp) load_values<false, V>(F.bp, c, 0, bf16, b);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = k * V + i;
        const float q = F.c * dr[j];
        dg[i] = q * fmaf(z[j], w[i], b[i]);
        const float p = F.ldg ? dr[j] * g[i] : dr[j];
        if (FULL) sum0[j] += p;
        sum1[j] = fmaf(p, z[j], sum1[j]);
        dr[j] = q * g[i] * w[i];
        n1 += dr[j];
        n2 = fmaf(dr[j], z[j], n2);
      }
      if (P.dgate) store_values<false, V>(P.dgate, row * F.d + c, 0, bf16, dg);
    }
    if (!P.dz) continue;
    if (F.post != SFNN_NORM_NONE) {
      float s[2] = {n1, n2};
      sum(s);
      n1 = F.post == SFNN_NORM_LAYER ? s[0] * F.inv_d : 0.f;
      n2 = s[1] * F.inv_d;
    } else {
      n1 = n2 = 0.f;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * threads) * V;
      if (c >= F.d) continue;
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = st.w * (dr[k * V + i] - fmaf(z[k * V + i], n2, n1));
      store_values<true, V>(P.dz, row * F.d + c, F.z32, bf16, v);
    }
  }
  if (!P.part) return;
  float *part = P.part + at.unit * P.sums * F.d;
  auto put = [&](int at, const float *v) {
    if (at < 0) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * threads) * V;
      if (c < F.d) store_values<true, V>(part, (int64_t)at * F.d + c, 1, bf16, v + k * V);
    }
  };
  put(P.at[kSumW], sw);
  put(P.at[kSum1], sum1);
  if (FULL) {
    put(P.at[kSumB], sb);
    put(P.at[kSum0], sum0);
  }
}

// The gradients of the channels' weights from the groups' sums: 32 columns a CTA, a share of the
// groups a warp, added up in their order.
struct NormSums {
  const float *part;
  int groups, sums, d;
  int at[kSums];
  float c;
  const void *gate, *wp, *bp;  // one gate row, or null
  void *dw, *db, *dgate, *dwp, *dbp;
};
constexpr int kSumWarps = 16, kSumAhead = 10;  // a CTA's sums of every SM in one request
template <bool bf16>
__global__ void __launch_bounds__(kSumWarps * 32) k_norm_sums(const __grid_constant__ NormSums P) {
  __shared__ float s[kSums][kSumWarps][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int64_t group = (int64_t)P.sums * P.d;
  float v[kSums] = {};
  if (c < P.d)
    for (int g = warp; g < P.groups; g += kSumWarps * kSumAhead) {
#pragma unroll
      for (int k = 0; k < kSums; ++k) {
        if (P.at[k] < 0) continue;
        const float *p = P.part + (int64_t)P.at[k] * P.d + c;
        float f[kSumAhead];
#pragma unroll
        for (int i = 0; i < kSumAhead; ++i) f[i] = g + i * kSumWarps < P.groups ? __ldg(p + (g + i * kSumWarps) * group) : 0.f;
#pragma unroll
        for (int i = 0; i < kSumAhead; ++i) v[k] += f[i];
      }
    }
#pragma unroll
  for (int k = 0; k < kSums; ++k) s[k][warp][lane] = v[k];
  __syncthreads();
  if (warp || c >= P.d) return;
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    v[k] = 0.f;
    if (P.at[k] >= 0)
#pragma unroll
      for (int i = 0; i < kSumWarps; ++i) v[k] += s[k][i][lane];
  }
  auto put = [&](void *p, float f) {
    if (p) static_cast<uint16_t *>(p)[c] = (uint16_t)pack16(f, 0.f, bf16);
  };
  const float g = P.c * (P.gate ? load16(P.gate, c, bf16) : 1.f);
  put(P.dw, v[kSumW]);
  put(P.db, v[kSumB]);
  put(P.dwp, g * v[kSum1]);
  put(P.dbp, g * v[kSum0]);
  if (P.dgate)
    put(P.dgate, P.c * fmaf(P.wp ? load16(P.wp, c, bf16) : 1.f, v[kSum1], P.bp ? load16(P.bp, c, bf16) * v[kSum0] : 0.f));
}

// ---------------------------------------------------------------- host
constexpr int kMaxWidth = 32768;
constexpr int kRingRows = 4;  // rows an SM from which the way through shared memory is worth its start

bool rows_ok(const void *p, int64_t ld, int d, bool wide) { return p && on(p, wide ? 4 : 2) && ld >= d && ld <= (1ll << 36); }
bool vectors(const void *p, int64_t ld) { return !p || (on(p, 16) && ld % 8 == 0); }

sfnn_status check(const sfnn_norm_desc *q) {
  if (!q || q->T < 0 || q->d < 1) return SFNN_ERR_INVALID_ARG;
  if (q->dtype != SFNN_F16 && q->dtype != SFNN_BF16) return SFNN_ERR_INVALID_ARG;
  if (q->x_dtype != q->dtype && q->x_dtype != SFNN_F32) return SFNN_ERR_INVALID_ARG;
  if (q->z_dtype != q->dtype && q->z_dtype != SFNN_F32) return SFNN_ERR_INVALID_ARG;
  for (int kind : {q->pre, q->post})
    if (kind != SFNN_NORM_NONE && kind != SFNN_NORM_RMS && kind != SFNN_NORM_LAYER) return SFNN_ERR_INVALID_ARG;
  if (!(q->eps >= 0.f)) return SFNN_ERR_INVALID_ARG;
  if (q->d > kMaxWidth || q->T > (1 << 28)) return SFNN_ERR_UNSUPPORTED;
  if (q->T && !q->z && (q->post != SFNN_NORM_NONE || q->gate || q->pre == SFNN_NORM_NONE || q->residual_scale != 1.f))
    return SFNN_ERR_INVALID_ARG;
  if ((q->pre == SFNN_NORM_NONE && (q->w || q->b)) || (q->post == SFNN_NORM_NONE && (q->post_w || q->post_b)))
    return SFNN_ERR_INVALID_ARG;
  for (const void *p : {q->w, q->b, q->post_w, q->post_b, q->gate})
    if (!on(p, 2)) return SFNN_ERR_INVALID_ARG;
  if (q->T == 0) return SFNN_OK;
  if (!rows_ok(q->x, q->ldx, q->d, q->x_dtype == SFNN_F32)) return SFNN_ERR_INVALID_ARG;
  if (q->z && !rows_ok(q->z, q->ldz, q->d, q->z_dtype == SFNN_F32)) return SFNN_ERR_INVALID_ARG;
  if (q->gate && q->ldg != 0 && !rows_ok(q->gate, q->ldg, q->d, false)) return SFNN_ERR_INVALID_ARG;
  return SFNN_OK;
}

NormParams params(const sfnn_norm_desc *q) {
  NormParams P{};
  P.x = q->x, P.z = q->z, P.gate = q->gate, P.w = q->w, P.b = q->b, P.wp = q->post_w, P.bp = q->post_b;
  P.ldx = q->ldx, P.ldz = q->ldz, P.ldg = q->ldg;
  P.T = q->T, P.d = q->d;
  P.x32 = q->x_dtype == SFNN_F32, P.z32 = q->z_dtype == SFNN_F32;
  P.pre = q->pre, P.post = q->post;
  P.eps = q->eps, P.a = q->residual_scale, P.c = q->branch_scale;
  P.inv_d = 1.f / (float)q->d;
  return P;
}
bool vectors(const NormParams &P) {
  return P.d % 8 == 0 && vectors(P.x, P.ldx) && vectors(P.z, P.ldz) && vectors(P.gate, P.ldg) && vectors(P.w, 0) &&
         vectors(P.b, 0) && vectors(P.wp, 0) && vectors(P.bp, 0);
}

// `threads` threads share a row: of one CTA, or of `ctas` CTAs of `block` threads.
template <class Kernel, class Params>
cudaError_t launch_rows(Kernel kernel, int grid, int block, int ctas, int threads, const Params &P, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = (unsigned)ctas;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P, threads);
}

template <bool bf16>
cudaError_t run_forward(const NormParams &P, bool vec, cudaStream_t s) {
  // A thread holds 8, 16 or 32 values: as many as leave a row a warp, at most 32.
  const int per = P.d <= 256 ? 8 : P.d <= 512 ? 16 : 32;
  int ctas = vec ? 1 : 2;
  while (P.d > per * 256 * ctas) ctas *= 2;
  int block = (int)up((P.d + per * ctas - 1) / (per * ctas), 32);
  const int threads = block * ctas, rows = ctas > 1 ? 1 : std::max(1, 128 / block);
  block *= rows;
  const int64_t units = (P.T + (int64_t)rows - 1) / rows;  // (T is at most 2^28, a row's CTAs at most 4)
  auto run = [&](auto kernel) { return launch_rows(kernel, (int)(units * ctas), block, ctas, threads, P, s); };
  // (shorter rows without vectors all go through shared memory)
  if (!vec) return run(k_norm_forward<bf16, 1, 32, true>);
  if (ctas > 1) return run(k_norm_forward<bf16, 8, 4, true>);
  return per == 8    ? run(k_norm_forward<bf16, 8, 1, false>)
         : per == 16 ? run(k_norm_forward<bf16, 8, 2, false>)
                     : run(k_norm_forward<bf16, 8, 4, false>);
}

// The shape of the backward kernel for long rows: a row's threads, and the clusters that rows are dealt to.
struct BackShape {
  int threads, ctas, block, grid;
  int64_t groups() const { return grid / ctas; }
};
BackShape back_shape(int64_t T, int d, bool full, int sms) {
  BackShape b;
  b.ctas = 2;
  while (d > 4096 * b.ctas) b.ctas *= 2;  // 8 values a thread, 512 threads a CTA
  b.block = (int)up((d + 8 * b.ctas - 1) / (8 * b.ctas), 32);
  b.threads = b.block * b.ctas;
  b.grid = (int)std::min<int64_t>(T, std::max(1, sms * (full ? 1 : 2) / b.ctas)) * b.ctas;
  return b;
}
int64_t back_workspace(int64_t T, int d, int sums, int sms) {  // (the larger of the two kernels')
  T = std::max<int64_t>(T, 1);
  return up(std::max(back_shape(T, d, false, sms).groups(), std::min<int64_t>(T, sms)) * sums * d * 4, 256);
}

template <bool bf16>
cudaError_t run_backward(const NormBackParams &P, bool vec, bool full, const BackShape &b, cudaStream_t s) {
  auto run = [&](auto kernel) { return launch_rows(kernel, b.grid, b.block, b.ctas, b.threads, P, s); };
  if (vec) return full ? run(k_norm_backward<bf16, 8, true>) : run(k_norm_backward<bf16, 8, false>);
  return full ? run(k_norm_backward<bf16, 1, true>) : run(k_norm_backward<bf16, 1, false>);
}

}  // namespace
}  // namespace sfnn

using namespace sfnn;

extern "C" {

int64_t sfnn_norm_workspace(int32_t T, int32_t d) {
  if (T < 0 || d < 1 || d > kMaxWidth) return -1;
  return back_workspace(T, d, kSums, std::max(1, device_sms()));
}

sfnn_status sfnn_norm_forward(const sfnn_norm_desc *q, void *r, int64_t ldr, void *h, int64_t ldh, float *stats,
                              int32_t *err, sfnn_stream_t stream) {
  const sfnn_status st = check(q);
  if (st != SFNN_OK) return st;
  if (q->T == 0) return SFNN_OK;
  NormParams P = params(q);
  if ((q->z && !rows_ok(r, ldr, q->d, P.x32)) || (q->pre != SFNN_NORM_NONE && !rows_ok(h, ldh, q->d, false)) || !on(stats, 16) || !err ||
      !on(err, 4))
    return SFNN_ERR_INVALID_ARG;
  P.r = q->z ? r : nullptr;
  P.h = q->pre != SFNN_NORM_NONE ? h : nullptr;
  P.ldr = ldr;
  P.ldh = ldh;
  P.stats = stats;
  const bool vec = vectors(P) && vectors(P.r, ldr) && vectors(P.h, ldh);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = q->dtype == SFNN_BF16;
  const int sms = device_sms();
  if (sms < 1) return SFNN_ERR_CUDA;
  // Rows that do not start on 16 bytes, and many rows, go through shared memory, where they fit.  (Few rows
  // of vectors: 300 x 4096 host-bound either way, 4000 x 8192 52 us through shared memory, 99 in registers.)
  RingPlan plan{};
  cudaError_t e = cudaSuccess;
  if (!vec || P.T >= kRingRows * sms) e = norm_forward_ring(P, err, bf16, vec, sms, s, plan);
  if (!plan.fits) e = bf16 ? run_forward<true>(P, vec, s) : run_forward<false>(P, vec, s);
  return e == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
}

sfnn_status sfnn_norm_backward(const sfnn_norm_desc *q, const float *stats, const void *dr, int64_t lddr, const void *dh,
                               int64_t lddh, void *dx, void *dz, void *dgate, void *dw, void *db, void *dpost_w,
                               void *dpost_b, void *ws, int64_t ws_bytes, int32_t *err, sfnn_stream_t stream) {
  const sfnn_status st = check(q);
  if (st != SFNN_OK) return st;
  const bool bf16 = q->dtype == SFNN_BF16;
  if ((dh && q->pre == SFNN_NORM_NONE) || ((dw || db) && q->pre == SFNN_NORM_NONE) || (dgate && !q->gate) ||
      ((dpost_w || dpost_b) && q->post == SFNN_NORM_NONE) || (dz && !q->z))
    return SFNN_ERR_INVALID_ARG;
  for (void *p : {dgate, dw, db, dpost_w, dpost_b})
    if (!on(p, 2)) return SFNN_ERR_INVALID_ARG;
  if (!on(dx, q->x_dtype == SFNN_F32 ? 4 : 2) || !on(dz, q->z_dtype == SFNN_F32 ? 4 : 2)) return SFNN_ERR_INVALID_ARG;
  const bool one_gate = q->gate && q->ldg == 0;
  NormSums S{};
  S.dw = dw, S.db = db, S.dwp = dpost_w, S.dbp = dpost_b, S.dgate = one_gate ? dgate : nullptr;
  const bool asked[kSums] = {dw != nullptr, db != nullptr, dpost_w || S.dgate, dpost_b || (S.dgate && q->post_b)};
  for (int i = 0; i < kSums; ++i) S.at[i] = asked[i] ? S.sums++ : -1;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (q->T == 0) {  // sums over no tokens
    for (void *p : {S.dw, S.db, S.dwp, S.dbp, S.dgate})
      if (p && cudaMemsetAsync(p, 0, (size_t)q->d * 2, s) != cudaSuccess) return SFNN_ERR_CUDA;
    return SFNN_OK;
  }
  const bool x32 = q->x_dtype == SFNN_F32;
  if ((dr && !rows_ok(dr, lddr, q->d, x32)) || (dh && !rows_ok(dh, lddh, q->d, false)) || !stats || !on(stats, 16) ||
      !err || !on(err, 4))
    return SFNN_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (sms < 1) return SFNN_ERR_CUDA;
  if (S.sums && (!ws || !on(ws, 16) || ws_bytes < back_workspace(q->T, q->d, S.sums, sms))) return SFNN_ERR_INVALID_ARG;
  NormBackParams P{};
  P.f = params(q);
  P.f.stats = const_cast<float *>(stats);
  P.dr = dr, P.lddr = lddr;
  P.dh = dh, P.lddh = lddh;
  P.dx = dx, P.dz = dz;
  P.dgate = one_gate ? nullptr : dgate;
  P.part = S.sums ? static_cast<float *>(ws) : nullptr;
  P.err = err;
  P.sums = S.sums;
  std::copy(S.at, S.at + kSums, P.at);
  const bool vec = vectors(P.f) && vectors(dr, lddr) && vectors(dh, lddh) && vectors(dx, 0) && vectors(dz, 0) &&
                   vectors(P.dgate, 0);
  RingPlan plan{};
  const bool all = asked[kSumB] || asked[kSum0];
  cudaError_t e = norm_backward_ring(P, all, bf16, vec, sms, s, plan);
  if (!plan.fits) {
    const BackShape b = back_shape(q->T, q->d, all, sms);
    plan.groups = (int)b.groups();
    e = bf16 ? run_backward<true>(P, vec, all, b, s) : run_backward<false>(P, vec, all, b, s);
  }
  if (e != cudaSuccess) return SFNN_ERR_CUDA;
  if (S.sums) {
    S.part = P.part;
    S.groups = plan.groups;
    S.d = q->d;
    S.c = P.f.c;
    S.gate = one_gate ? q->gate : nullptr;
    S.wp = q->post_w, S.bp = q->post_b;
    const dim3 grid((unsigned)((q->d + 31) / 32)), block(kSumWarps * 32);
    if ((bf16 ? launch_pdl(k_norm_sums<true>, grid, block, 0, s, S) : launch_pdl(k_norm_sums<false>, grid, block, 0, s, S)) !=
        cudaSuccess)
      return SFNN_ERR_CUDA;
  }
  return SFNN_OK;
}

}  // extern "C"
