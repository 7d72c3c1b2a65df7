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
#include <atomic>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

struct NormParams {
  const void *x, *z, *gate, *w, *b, *wp, *bp;
  int64_t ldx, ldz, ldg;  // ldg 0: one gate row
  void *r, *h;
  int64_t ldr, ldh;
  float *stats;  // [T][4]: mean and reciprocal deviation of R, of Z; or null
  int T, d, x32, z32;
  int pre, post;  // sfnn_norm
  float eps, a, c, inv_d;
};

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
// What is summed over the rows.  Behind the post norm two sums serve five gradients, since a gate row,
// w_post and b_post are the same for every row (with p = D, or D gate where each token has its gate):
//
//     S1 = sum p Z^,  S0 = sum p:   dw_post = c gate S1,  db_post = c gate S0,  dgate = c (w_post S1 + b_post S0)
enum { kSumW, kSumB, kSum1, kSum0, kSums };
struct NormBackParams {
  NormParams f;
  const void *dr, *dh;
  int64_t lddr, lddh;
  void *dx, *dz, *dgate;  // contiguous; dgate: of a gate of every token
  float *part;            // [groups][sums][d], or null
  int32_t *err;
  int sums;       // that are asked for
  int at[kSums];  // their places in part, or -1
};

// 8 values of a row a thread, a row to `threads` threads of a CTA (CLUSTER: of all the cluster's CTAs),
// rows dealt to these groups in turn; a group keeps its columns' sums in registers.  FULL: all four,
// else dw and S1 alone.
template <bool bf16, int V, bool FULL, bool CLUSTER>
__global__ void __launch_bounds__(512, FULL ? 1 : 2) k_norm_backward(const __grid_constant__ NormBackParams P, int threads) {
  constexpr int NV = 8 / V;
  __shared__ float2 slots[2 * RowSum<CLUSTER>::kSlots];
  pdl_wait();
  pdl_launch_dependents();
  const NormParams &F = P.f;
  const Place<CLUSTER> at(threads);
  const int lane = at.lane, groups = at.groups, mine = at.mine;
  const int64_t unit = at.unit, units = at.units;
  RowSum<CLUSTER> sum = at.sums(slots, threads);
  if (CLUSTER) cluster_sync_all();
  float sw[8], sb[FULL ? 8 : 1], sum1[8], sum0[FULL ? 8 : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sw[i] = sum1[i] = 0.f;
    if (FULL) sb[i] = sum0[i] = 0.f;
  }
  // every group makes the same number of turns
  for (int64_t first = unit * groups; first < F.T; first += units * groups) {
    const int64_t row = first + mine;
    const bool live = row < F.T;
    float x[8], z[8], dr[8], dh[8];
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) st = __ldg(reinterpret_cast<const float4 *>(F.stats) + row);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + k * threads) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) x[k * V + i] = z[k * V + i] = dr[k * V + i] = dh[k * V + i] = 0.f;
      if (!live || c >= F.d) continue;
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
        if (!live || c >= F.d) continue;
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
        if (!live || c >= F.d) continue;
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
        if (!live || c >= F.d) continue;
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
      if (!live || c >= F.d) {
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
      if (!live || c >= F.d) continue;
      float v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = st.w * (dr[k * V + i] - fmaf(z[k * V + i], n2, n1));
      store_values<true, V>(P.dz, row * F.d + c, F.z32, bf16, v);
    }
  }
  if (!P.part) return;
  float *part = P.part + (unit * groups + mine) * P.sums * F.d;
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

// ---------------------------------------------------------------- rows through shared memory
// The kernels above hold a row's values in registers, and while a row's sums go round nothing is
// on its way from memory.  These keep the next rows coming: a CTA an SM, its threads in groups that
// each take a row at a time, with stages of their own that bulk copies fill while the rows before are
// worked on; a group waits for nothing but its own rows and sums.  The values stay in shared memory
// until each is needed, beside them the channels' weights.  A thread has 16 values (two vectors of 8).
constexpr int kMaxStages = 4;
constexpr int kMaxGroups = 16;  // 15 named barriers; 16 groups are warps, which need none
constexpr int kRingValues = 16;
enum { kOfX, kOfZ, kOfDr, kOfDh, kOfGate, kOfRows };

struct RingParams {
  const void *p[kOfRows];  // arrays whose rows pass through the ring (null: none)
  int64_t ld[kOfRows];     // bytes
  int bytes[kOfRows];      // of a row
  int at[kOfRows];         // in a stage
  int stage, stages;       // bytes of a stage (a row of every array)
  int groups, threads;     // of a CTA, of a group
  int held[4];             // where the channels' weights lie behind the stages (-1: all the same, see weight())
};
// The channels' weights as the kernels use them, in 32 bits: c gate w_post (without the gate where every
// token has its own), w, and for FULL c gate b_post and b.
enum { kPostW, kPreW, kPostB, kPreB, kWeights };

// Pairs of fp32 values in a 64-bit register, one instruction for both.  (Kept as such from the load to
// the store: taken apart in between, every instruction is joined by moves.)
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ float2 apart(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ float within(Pair p) {
  const float2 v = apart(p);
  return v.x + v.y;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void lds_pairs(uint32_t a, Pair &x, Pair &y) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a) : "memory");
}
__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

struct RingSmem {  // beside the stages and the weights
  uint64_t full[kMaxGroups * kMaxStages];
  float slots[2][2][64];  // [turn][value][a group's warps, rounded up to 4]
};

// WIDE: X or Z is fp32.  FULL: means and biases.  EXACT: what is usual -- both vectors of every thread are
// there (a width of whole 512s), X, Z, the pre norm and, backward, all gradients, no gate for each
// token -- whose tests cost as much as the arithmetic (backward, 4096 wide: 727 instructions a warp and
// row with them).
template <bool bf16, bool WIDE, bool FULL, bool EXACT>
struct Ring {
  const RingParams &R;
  const NormParams &F;
  RingSmem &S;
  int32_t *err;
  int mine, lane;        // the group, the thread's place in it
  int row, step;         // the row at hand; from one to the next
  int slot, phase, turn;
  bool dead;             // a wait has run out
  uint32_t cur, stage0;  // the stage at hand, the group's first
  uint32_t weights, slots;

  __device__ __forceinline__ Ring(const RingParams &R_, const NormParams &F_, unsigned char *smem, RingSmem &S_, int32_t *err_)
      : R(R_), F(F_), S(S_), err(err_), slot(0), phase(0), turn(0), dead(false) {
    mine = threadIdx.x / R.threads;
    lane = threadIdx.x - mine * R.threads;
    slots = smem_u32(S.slots) + (uint32_t)(mine * ((R.threads / 32 + 3) & ~3) * 4);
    row = blockIdx.x * R.groups + mine;
    step = gridDim.x * R.groups;
    cur = stage0 = smem_u32(smem) + (uint32_t)(mine * R.stages * R.stage);
    weights = smem_u32(smem) + (uint32_t)(R.groups * R.stages * R.stage);
    for (int i = threadIdx.x; i < 4 * 64; i += blockDim.x) S.slots[i >> 7][(i >> 6) & 1][i & 63] = 0.f;
    if (threadIdx.x == 0) {
      for (int i = 0; i < R.groups * R.stages; ++i) bar_init(&S.full[i], 1);
      bar_init_fence();
      fence_async_shared();
    }
    __syncthreads();
    if (lane < 32)
      for (int i = 0; i < R.stages; ++i) request(row + i * step, i);
#pragma unroll 1
    for (int k = 0; k < kWeights; ++k) {
      const int at = k == 0 ? R.held[0] : k == 1 ? R.held[1] : k == 2 ? R.held[2] : R.held[3];
      if (at < 0) continue;
      ulonglong2 *to = reinterpret_cast<ulonglong2 *>(smem + (size_t)R.groups * R.stages * R.stage + at);
      const void *p = k == kPostW ? F.wp : k == kPreW ? F.w : k == kPostB ? F.bp : F.b;
      for (int c = threadIdx.x * 8; c < F.d; c += blockDim.x * 8) {
        Pair v[4], g[4];
        if (p)
          widen8(ld_keep(static_cast<const uint16_t *>(p) + c), v);
        else
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = both(1.f);
        if (k == kPostW || k == kPostB) {
          if (F.gate && !F.ldg)
            widen8(ld_keep(static_cast<const uint16_t *>(F.gate) + c), g);
          else
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = both(1.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = mul2(mul2(g[j], both(F.c)), v[j]);
        }
        to[c / 4] = make_ulonglong2(v[0], v[1]);
        to[c / 4 + 1] = make_ulonglong2(v[2], v[3]);
      }
    }
    __syncthreads();
  }
  __device__ __forceinline__ void request(int r, int s) const {  // the group's first warp, an array a lane
    if (r >= F.T) return;
    uint64_t *bar = &S.full[mine * R.stages + s];
    if (lane == 0) bar_expect_tx(bar, (uint32_t)R.stage);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kOfRows; ++k)
      if (lane == k && R.p[k])
        bulk_load(stage0 + (uint32_t)(s * R.stage + R.at[k]), static_cast<const unsigned char *>(R.p[k]) + r * R.ld[k],
                  (uint32_t)R.bytes[k], bar);
    __syncwarp();
  }
  // The row at hand is there.  A wait that runs out is latched, and the kernel goes on with what it
  // has: only its last waits, for the copies that must have landed before it ends, then take their time.
  __device__ __forceinline__ void wait() {
    uint64_t *bar = &S.full[mine * R.stages + slot];
    const bool ok = dead && row + R.stages * step < F.T ? bar_try(bar, (uint32_t)phase) : bar_wait(bar, (uint32_t)phase);
    if (!ok) {
      if (!dead) latch_error(err, kErrTimeout);
      dead = true;
    }
  }
  __device__ __forceinline__ void barrier() const {  // the group's threads
    if (R.threads == 32)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(mine + 1), "r"(R.threads) : "memory");
  }
  // The group is done with the row's stage (a barrier lies behind its last use): on to the next.
  __device__ __forceinline__ void release() const {
    if (lane < 32) request(row + R.stages * step, slot);
  }
  __device__ __forceinline__ void next() {
    row += step;
    cur += (uint32_t)R.stage;
    if (++slot == R.stages) slot = 0, phase ^= 1, cur = stage0;
  }
  // Sums over the row; buffers alternate, so one barrier a sum is enough.
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if (R.threads == 32) return;
    const uint32_t at = slots + (uint32_t)turn * 512u;
    turn ^= 1;
    if ((lane & 31) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + n * 256u + (uint32_t)(lane >> 5) * 4u), "f"(v[n]) : "memory");
    barrier();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float4 t = lds_f4(at + n * 256u);
      v[n] = (t.x + t.y) + (t.z + t.w);
      for (int i = 4; i * 32 < R.threads; i += 4) {
        t = lds_f4(at + n * 256u + i * 4);
        v[n] += (t.x + t.y) + (t.z + t.w);
      }
    }
  }

  // 8 values of the row at hand, of an array, from column c on
  __device__ __forceinline__ void value8(int k, int c, bool wide, Pair v[4]) const {
    if (WIDE && wide) {
      const uint32_t p = cur + (uint32_t)(R.at[k] + c * 4);
      lds_pairs(p, v[0], v[1]);
      lds_pairs(p + 16, v[2], v[3]);
    } else {
      widen8(lds_u4(cur + (uint32_t)(R.at[k] + c * 2)), v);
    }
  }
  // 8 weights, as the enumeration above says
  __device__ __forceinline__ void weight(int k, int c, Pair v[4]) const {
    if (!(EXACT && (k == kPostW || k == kPreW)) && R.held[k] < 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = both(k == kPostW ? F.c : k == kPreW ? 1.f : 0.f);
      return;
    }
    const uint32_t p = weights + (uint32_t)(R.held[k] + c * 4);
    lds_pairs(p, v[0], v[1]);
    lds_pairs(p + 16, v[2], v[3]);
  }
  static __device__ __forceinline__ void widen8(const uint4 &w, Pair v[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16 ? make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u)) : unpack16(u[i], false);
      v[i] = pair(f.x, f.y);
    }
  }
  static __device__ __forceinline__ void store(void *p, int64_t at, bool wide, const Pair v[4]) {
    if (WIDE && wide) {
      ulonglong2 *q = reinterpret_cast<ulonglong2 *>(static_cast<float *>(p) + at);
      q[0] = make_ulonglong2(v[0], v[1]);
      q[1] = make_ulonglong2(v[2], v[3]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = apart(v[i]);
        u[i] = pack16(f.x, f.y, bf16);
      }
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  __device__ __forceinline__ bool gated() const { return !EXACT && R.p[kOfGate]; }  // a gate for each token
  // (Z - mean) and post(Z) gate c of 8 columns.
  __device__ __forceinline__ void branch(int c, float mz, float sz, Pair z[4], Pair v[4]) const {
    value8(kOfZ, c, F.z32, z);
    weight(kPostW, c, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (FULL) z[i] = add2(z[i], both(-mz));
      v[i] = mul2(z[i], v[i]);
    }
    if (!FULL && !gated()) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(sz));
      return;
    }
    Pair b[4];
    if (FULL)
      weight(kPostB, c, b);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = both(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fma2(v[i], both(sz), b[i]);
    if (!gated()) return;
    value8(kOfGate, c, false, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], b[i]);
  }
};

constexpr int kForwardThreads = 1024, kBackwardThreads = 512;

template <bool bf16, bool WIDE, bool FULL, bool EXACT>
__global__ void __launch_bounds__(kForwardThreads, 1) k_norm_forward_ring(const __grid_constant__ NormParams P,
                                                                          const __grid_constant__ RingParams R, int32_t *err) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ RingSmem more;
  pdl_wait();
  pdl_launch_dependents();
  Ring<bf16, WIDE, FULL, EXACT> ring(R, P, ring_smem, more, err);
  const int c0 = ring.lane * 8, c1 = c0 + R.threads * 8;
  const bool in[2] = {EXACT || c0 < P.d, EXACT || c1 < P.d}, has_z = EXACT || P.z, has_pre = EXACT || P.pre != SFNN_NORM_NONE;
  auto mean_of = [&](Pair v) {
    float t[1] = {within(v)};
    ring.sum(t);
    return t[0] * P.inv_d;
  };
  for (; ring.row < P.T; ring.next()) {
    ring.wait();
    float mz = 0.f, sz = 1.f, mr = 0.f, sr = 1.f;
    if (P.post != SFNN_NORM_NONE) {
#pragma unroll
      for (int pass = FULL ? 0 : 1; pass < 2; ++pass) {  // mean, then deviation
        if (FULL && pass == 0 && P.post != SFNN_NORM_LAYER) continue;
        Pair q = both(0.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!in[k]) continue;
          Pair z[4];
          ring.value8(kOfZ, k ? c1 : c0, P.z32, z);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (FULL && pass) z[i] = add2(z[i], both(-mz));
            q = FULL && !pass ? add2(q, z[i]) : fma2(z[i], z[i], q);
          }
        }
        const float m = mean_of(q);
        if (pass)
          sz = rsqrtf(m + P.eps);
        else
          mz = m;
      }
    }
    Pair r[8], q = both(0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = k ? c1 : c0;
      Pair *rk = r + 4 * k, z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rk[i] = both(0.f);
      if (!in[k]) continue;
      ring.value8(kOfX, c, P.x32, rk);
      if (has_z) {
        Pair v[4];
        ring.branch(c, mz, sz, z, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) rk[i] = fma2(rk[i], both(P.a), v[i]);
      }
      if (has_z) ring.store(P.r, (int64_t)ring.row * P.ldr + c, P.x32, rk);
      if (!FULL)
#pragma unroll
        for (int i = 0; i < 4; ++i) q = fma2(rk[i], rk[i], q);
    }
    if (!has_pre || R.threads == 32) ring.barrier();
    if (has_pre) {
      if (FULL) {
        if (P.pre == SFNN_NORM_LAYER) {
#pragma unroll
          for (int i = 0; i < 8; ++i) q = add2(q, r[i]);
          mr = mean_of(q);
        }
        q = both(0.f);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (in[k])
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              r[4 * k + i] = add2(r[4 * k + i], both(-mr));
              q = fma2(r[4 * k + i], r[4 * k + i], q);
            }
      }
      sr = rsqrtf(mean_of(q) + P.eps);
    }
    ring.release();
    if (has_pre) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = k ? c1 : c0;
        if (!in[k]) continue;
        Pair w[4], b[4];
        ring.weight(kPreW, c, w);
        if (FULL) ring.weight(kPreB, c, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair hat = mul2(r[4 * k + i], both(sr));
          w[i] = FULL ? fma2(hat, w[i], b[i]) : mul2(hat, w[i]);
        }
        ring.store(P.h, (int64_t)ring.row * P.ldh + c, false, w);
      }
    }
    if (P.stats && ring.lane == 0) *reinterpret_cast<float4 *>(P.stats + (int64_t)ring.row * 4) = make_float4(mr, sr, mz, sz);
  }
}

template <bool bf16, bool WIDE, bool FULL, bool EXACT>  // FULL: the sums of dH and D as well
__global__ void __launch_bounds__(kBackwardThreads, 1) k_norm_backward_ring(const __grid_constant__ NormBackParams P,
                                                                            const __grid_constant__ RingParams R) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ RingSmem more;
  pdl_wait();
  pdl_launch_dependents();
  const NormParams &F = P.f;
  Ring<bf16, WIDE, FULL, EXACT> ring(R, F, ring_smem, more, P.err);
  const int c0 = ring.lane * 8, c1 = c0 + R.threads * 8;
  const bool in[2] = {EXACT || c0 < F.d, EXACT || c1 < F.d};
  const bool has_z = EXACT || F.z, has_dh = EXACT || P.dh, has_dr = EXACT || P.dr, has_dx = EXACT || P.dx;
  Pair sw[8], sum1[8], sb[FULL ? 8 : 1], sum0[FULL ? 8 : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sw[i] = sum1[i] = both(0.f);
    if (FULL) sb[i] = sum0[i] = both(0.f);
  }
  const bool has_dz = EXACT || P.dz, two_sums = has_dz && F.post != SFNN_NORM_NONE;
  // (of columns past d these stay zero)
  Pair D[8], hat[8], z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) D[i] = hat[i] = z[i] = both(0.f);
  for (; ring.row < F.T; ring.next()) {
    const float4 st = __ldg(reinterpret_cast<const float4 *>(F.stats) + ring.row);  // of R, of Z: mean, 1 / deviation
    ring.wait();
    Pair s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = k ? c1 : c0;
      Pair *Dk = D + 4 * k, *hk = hat + 4 * k, *zk = z + 4 * k;
      if (!in[k]) continue;
      if (has_dh) {
        ring.value8(kOfX, c, F.x32, hk);
        if (has_z) {  // R^ = a s X + s (c gate post(Z) - mean)
          Pair v[4];
          ring.branch(c, st.z, st.w * (FULL || ring.gated() ? 1.f : st.y), zk, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (FULL) v[i] = add2(v[i], both(-st.x));
            if (FULL || ring.gated()) v[i] = mul2(v[i], both(st.y));
            hk[i] = fma2(hk[i], both(F.a * st.y), v[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) hk[i] = mul2(FULL ? add2(hk[i], both(-st.x)) : hk[i], both(st.y));
        }
        Pair dh[4];
        ring.value8(kOfDh, c, false, dh);
        ring.weight(kPreW, c, Dk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          Dk[i] = mul2(dh[i], Dk[i]);
          if (FULL) s1 = add2(s1, Dk[i]), sb[4 * k + i] = add2(sb[4 * k + i], dh[i]);
          s2 = fma2(Dk[i], hk[i], s2);
          sw[4 * k + i] = fma2(dh[i], hk[i], sw[4 * k + i]);
        }
      } else if (has_z) {
        ring.value8(kOfZ, c, F.z32, zk);
        if (FULL)
#pragma unroll
          for (int i = 0; i < 4; ++i) zk[i] = add2(zk[i], both(-st.z));
      }
    }
    float k1 = 0.f, k2 = 0.f;  // D = dR + s u - s mean u - s mean(u R^) R^
    if (has_dh) {
      if (FULL) {
        float t[2] = {within(s1), within(s2)};
        ring.sum(t);
        k1 = F.pre == SFNN_NORM_LAYER ? -st.y * t[0] * F.inv_d : 0.f;
        k2 = -st.y * t[1] * F.inv_d;
      } else {
        float t[1] = {within(s2)};
        ring.sum(t);
        k2 = -st.y * t[0] * F.inv_d;
      }
    }
    Pair n1 = both(0.f), n2 = both(0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = k ? c1 : c0;
      Pair *Dk = D + 4 * k, *hk = hat + 4 * k, *zk = z + 4 * k;
      if (!in[k]) continue;
      Pair v[4];
      if (has_dr)
        ring.value8(kOfDr, c, F.x32, v);
      else
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = both(0.f);
      if (has_dh) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (FULL) v[i] = add2(v[i], both(k1));
          Dk[i] = fma2(Dk[i], both(st.y), fma2(hk[i], both(k2), v[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) Dk[i] = v[i];
      }
      if (has_dx) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(both(F.a), Dk[i]);
        ring.store(P.dx, (int64_t)ring.row * F.d + c, F.x32, v);
      }
      if (!has_z) continue;
      Pair w[4];
      ring.weight(kPostW, c, w);
      if (ring.gated()) {
        Pair g[4];
        ring.value8(kOfGate, c, false, g);
        if (P.dgate) {
          if (FULL) ring.weight(kPostB, c, v);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = mul2(Dk[i], fma2(mul2(zk[i], both(st.w)), w[i], FULL ? v[i] : both(0.f)));
          ring.store(P.dgate, (int64_t)ring.row * F.d + c, false, v);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) Dk[i] = mul2(Dk[i], g[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // D becomes s_z v
        if (FULL) sum0[4 * k + i] = add2(sum0[4 * k + i], Dk[i]);
        Dk[i] = mul2(Dk[i], both(st.w));
        sum1[4 * k + i] = fma2(Dk[i], zk[i], sum1[4 * k + i]);
        Dk[i] = mul2(Dk[i], w[i]);
        if (FULL) n1 = add2(n1, Dk[i]);
        n2 = fma2(Dk[i], zk[i], n2);
      }
    }
    if (!two_sums || R.threads == 32) ring.barrier();
    float m1 = 0.f, m2 = 0.f;  // dZ = s_z (v - mean v - Z^ mean(v Z^))
    if (two_sums) {
      float t[FULL ? 2 : 1];
      t[0] = within(n2);
      if (FULL) t[FULL ? 1 : 0] = within(n1);
      ring.sum(t);
      m2 = -st.w * st.w * t[0] * F.inv_d;
      if (FULL && F.post == SFNN_NORM_LAYER) m1 = -t[FULL ? 1 : 0] * F.inv_d;
    }
    ring.release();
    if (!has_dz) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = k ? c1 : c0;
      if (!in[k]) continue;
      Pair v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = fma2(z[4 * k + i], both(m2), D[4 * k + i]);
        if (FULL) v[i] = add2(v[i], both(m1));
      }
      ring.store(P.dz, (int64_t)ring.row * F.d + c, F.z32, v);
    }
  }
  if (!P.part) return;
  float *part = P.part + ((int64_t)blockIdx.x * R.groups + ring.mine) * P.sums * F.d;
  auto put = [&](int at, const Pair *v) {
    if (at < 0) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!in[k]) continue;
      ulonglong2 *q = reinterpret_cast<ulonglong2 *>(part + (int64_t)at * F.d + (k ? c1 : c0));
      q[0] = make_ulonglong2(v[4 * k], v[4 * k + 1]);
      q[1] = make_ulonglong2(v[4 * k + 2], v[4 * k + 3]);
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
constexpr int kSumWarps = 16;
template <bool bf16>
__global__ void __launch_bounds__(kSumWarps * 32) k_norm_sums(const __grid_constant__ NormSums P) {
  __shared__ float s[kSums][kSumWarps][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const int64_t group = (int64_t)P.sums * P.d;
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    if (P.at[k] < 0) continue;
    const float *p = P.part + (int64_t)P.at[k] * P.d + c;
    float v = 0.f;
    if (c < P.d)
#pragma unroll 8
      for (int g = warp; g < P.groups; g += kSumWarps) v += __ldg(p + g * group);
    s[k][warp][lane] = v;
  }
  __syncthreads();
  if (warp || c >= P.d) return;
  float v[kSums];
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
  int ctas = 1;
  while (P.d > per * 256 * ctas) ctas *= 2;
  int block = (int)up((P.d + per * ctas - 1) / (per * ctas), 32);
  const int threads = block * ctas, rows = ctas > 1 ? 1 : std::max(1, 128 / block);
  block *= rows;
  const int64_t units = (P.T + (int64_t)rows - 1) / rows;  // (T is at most 2^28, a row's CTAs at most 4)
  auto run = [&](auto kernel) { return launch_rows(kernel, (int)(units * ctas), block, ctas, threads, P, s); };
  if (ctas > 1) return vec ? run(k_norm_forward<bf16, 8, 4, true>) : run(k_norm_forward<bf16, 1, 32, true>);
  if (per == 8) return vec ? run(k_norm_forward<bf16, 8, 1, false>) : run(k_norm_forward<bf16, 1, 8, false>);
  if (per == 16) return vec ? run(k_norm_forward<bf16, 8, 2, false>) : run(k_norm_forward<bf16, 1, 16, false>);
  return vec ? run(k_norm_forward<bf16, 8, 4, false>) : run(k_norm_forward<bf16, 1, 32, false>);
}

// The backward kernel's shape: a row's threads, and the groups that rows are dealt to.
struct BackShape {
  int threads, ctas, block, per_cta, grid;
  int64_t groups() const { return (int64_t)grid / ctas * per_cta; }
};
BackShape back_shape(int64_t T, int d, bool full, int sms) {
  BackShape b;
  b.ctas = 1;
  while (d > 4096 * b.ctas) b.ctas *= 2;  // 8 values a thread, 512 threads a CTA
  b.block = (int)up((d + 8 * b.ctas - 1) / (8 * b.ctas), 32);
  b.threads = b.block * b.ctas;
  b.per_cta = b.ctas > 1 ? 1 : std::max(1, 512 / b.threads);
  b.block *= b.per_cta;
  const int64_t units = (T + b.per_cta - 1) / b.per_cta, most = std::max(1, sms * (full ? 1 : 2) / b.ctas);
  b.grid = (int)std::min(units, most) * b.ctas;
  return b;
}
int ring_threads(int d) { return (int)up((d + kRingValues - 1) / kRingValues, 32); }
int64_t ring_groups(int64_t T, int d, int sms) {  // at most
  const int groups = std::max(1, std::min(kMaxGroups, kBackwardThreads / ring_threads(d)));
  return std::min((T + groups - 1) / groups, (int64_t)sms) * groups;
}
int64_t back_workspace(int64_t T, int d, int sums, int sms) {  // (the larger of the two kernels')
  T = std::max<int64_t>(T, 1);
  return up(std::max(back_shape(T, d, false, sms).groups(), ring_groups(T, d, sms)) * sums * d * 4, 256);
}

template <bool bf16, int V, bool FULL>
cudaError_t run_backward(const NormBackParams &P, const BackShape &b, cudaStream_t s) {
  return b.ctas == 1 ? launch_rows(k_norm_backward<bf16, V, FULL, false>, b.grid, b.block, 1, b.threads, P, s)
                     : launch_rows(k_norm_backward<bf16, V, FULL, true>, b.grid, b.block, b.ctas, b.threads, P, s);
}
// The rows' way through shared memory.
constexpr int kRingSmem = 225 * 1024;
struct RingShape {
  int block, grid, smem;
  int64_t groups;
  bool fits;  // (else the rows are too long for shared memory)
};
RingShape ring_shape(RingParams &R, const NormParams &F, bool exact, bool backward, const void *dr, int64_t lddr, const void *dh, int64_t lddh,
                     int most_threads, int sms) {
  const int d = F.d;
  R.threads = ring_threads(d);
  auto row = [&](int k, const void *p, int64_t ld, bool wide) {
    R.p[k] = p;
    R.ld[k] = ld * (wide ? 4 : 2);
    R.bytes[k] = d * (wide ? 4 : 2);
    R.at[k] = R.stage;
    if (p) R.stage += R.bytes[k];
  };
  row(kOfX, F.x, F.ldx, F.x32);
  row(kOfZ, F.z, F.ldz, F.z32);
  row(kOfDr, dr, lddr, F.x32);
  row(kOfDh, dh, lddh, false);
  row(kOfGate, F.ldg ? F.gate : nullptr, F.ldg, false);
  int held = 0;
  const bool gate = F.gate && !F.ldg;
  const bool needed[kWeights] = {exact || (F.z && (gate || F.wp)), exact || F.w, F.bp != nullptr, F.b && !backward};
  for (int k = 0; k < kWeights; ++k) {
    R.held[k] = needed[k] ? held : -1;
    held += needed[k] ? d * 4 : 0;
  }
  // As many groups as threads allow, fewer where that leaves them two stages each.
  const int budget = kRingSmem - held;
  R.groups = std::max(1, std::min(R.threads == 32 ? kMaxGroups : kMaxGroups - 1, most_threads / R.threads));
  while (R.groups > 1 && R.groups * 2 * R.stage > budget) --R.groups;
  R.stages = std::min(kMaxStages, budget / (R.groups * R.stage));
  RingShape s;
  s.block = R.threads * R.groups;
  s.smem = R.groups * R.stages * R.stage + held;
  s.grid = (int)std::min<int64_t>(((int64_t)F.T + R.groups - 1) / R.groups, sms);
  s.groups = (int64_t)s.grid * R.groups;
  s.fits = R.threads <= most_threads && R.stages > 0;
  return s;
}
constexpr int kRingRows = 4;  // rows an SM from which the ring is worth its start
template <class Kernel, class... Args>
cudaError_t launch_ring(Kernel kernel, const RingShape &s, std::atomic<uint64_t> &ready, cudaStream_t stream, const Args &...args) {
  const cudaError_t e = allow_smem(kernel, kRingSmem, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)s.grid), dim3((unsigned)s.block), (size_t)s.smem, stream, args...);
}
template <bool bf16, bool WIDE, bool FULL, bool EXACT>
cudaError_t run_ring(const RingShape &s, const NormParams &P, const RingParams &R, int32_t *err, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  return launch_ring(k_norm_forward_ring<bf16, WIDE, FULL, EXACT>, s, ready, stream, P, R, err);
}
template <bool bf16, bool WIDE, bool FULL, bool EXACT>
cudaError_t run_ring(const RingShape &s, const NormBackParams &P, const RingParams &R, int32_t *, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  return launch_ring(k_norm_backward_ring<bf16, WIDE, FULL, EXACT>, s, ready, stream, P, R);
}
template <bool bf16, bool WIDE, class Params>
cudaError_t run_ring(bool full, bool exact, const RingShape &s, const Params &P, const RingParams &R, int32_t *err,
                     cudaStream_t stream) {
  if (full) return exact ? run_ring<bf16, WIDE, true, true>(s, P, R, err, stream) : run_ring<bf16, WIDE, true, false>(s, P, R, err, stream);
  return exact ? run_ring<bf16, WIDE, false, true>(s, P, R, err, stream) : run_ring<bf16, WIDE, false, false>(s, P, R, err, stream);
}
template <class Params>
cudaError_t run_ring(bool bf16, bool wide, bool full, bool exact, const RingShape &s, const Params &P, const RingParams &R,
                     int32_t *err, cudaStream_t stream) {
  if (bf16)
    return wide ? run_ring<true, true>(full, exact, s, P, R, err, stream) : run_ring<true, false>(full, exact, s, P, R, err, stream);
  return wide ? run_ring<false, true>(full, exact, s, P, R, err, stream) : run_ring<false, false>(full, exact, s, P, R, err, stream);
}
bool exact_rows(const NormParams &P) { return P.d % (32 * kRingValues) == 0 && P.z && P.pre != SFNN_NORM_NONE && !P.ldg; }

template <bool bf16>
cudaError_t run_backward(const NormBackParams &P, bool vec, bool full, const BackShape &b, cudaStream_t s) {
  if (vec)  // rows too long for the ring (at least 4096 values), and so for one CTA
    return full ? launch_rows(k_norm_backward<bf16, 8, true, true>, b.grid, b.block, b.ctas, b.threads, P, s)
                : launch_rows(k_norm_backward<bf16, 8, false, true>, b.grid, b.block, b.ctas, b.threads, P, s);
  return full ? run_backward<bf16, 1, true>(P, b, s) : run_backward<bf16, 1, false>(P, b, s);
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
  cudaError_t e;
  RingParams R{};
  const bool full = P.pre == SFNN_NORM_LAYER || P.post == SFNN_NORM_LAYER || P.b || P.bp;
  const bool exact = exact_rows(P);
  const RingShape shape = ring_shape(R, P, exact, false, nullptr, 0, nullptr, 0, kForwardThreads, sms);
  if (vec && shape.fits && P.T >= kRingRows * sms)
    e = run_ring(bf16, P.x32 || P.z32, full, exact, shape, P, R, err, s);
  else
    e = bf16 ? run_forward<true>(P, vec, s) : run_forward<false>(P, vec, s);
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
  int64_t groups;
  cudaError_t e;
  RingParams R{};
  bool full = P.f.pre == SFNN_NORM_LAYER || P.f.post == SFNN_NORM_LAYER || P.f.bp || asked[kSumB] || asked[kSum0];
  const bool exact = exact_rows(P.f) && dr && dh && dx && dz;
  const RingShape shape = ring_shape(R, P.f, exact, true, dr, lddr, dh, lddh, kBackwardThreads, sms);
  if (vec && shape.fits) {
    groups = shape.groups;
    e = run_ring(bf16, P.f.x32 || P.f.z32, full, exact, shape, P, R, err, s);
  } else {
    full = asked[kSumB] || asked[kSum0];
    const BackShape b = back_shape(q->T, q->d, full, sms);
    groups = b.groups();
    e = bf16 ? run_backward<true>(P, vec, full, b, s) : run_backward<false>(P, vec, full, b, s);
  }
  if (e != cudaSuccess) return SFNN_ERR_CUDA;
  if (S.sums) {
    S.part = P.part;
    S.groups = (int)groups;
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
