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
constexpr int kMaxWarps = 32;

// A row belongs to `warps` warps of the CTA, all rows of a CTA in step, or (CLUSTER) to all warps of
// `ctas` CTAs, which then write their warps' sums into each other's shared memory.  The sums of two
// values; the buffers alternate, so one barrier a sum is enough: who writes a buffer again has passed
// the barrier of the sum between, which every reader of it reached after reading.
template <bool CLUSTER>
struct RowSum {
  static constexpr int kSlots = CLUSTER ? kMaxCluster * 16 : kMaxWarps;
  float2 *slots;  // [2][kSlots]
  int warps, ctas, rank, turn;
  __device__ __forceinline__ float2 operator()(float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (!CLUSTER && warps == 1) return v;
    float2 *s = slots + turn * kSlots;
    turn ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (CLUSTER) {
      if (lane < ctas)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_addr(s + rank * warps + warp, lane)),
                     "f"(v.x), "f"(v.y)
                     : "memory");
      __syncwarp();
      cluster_sync_all();
    } else {
      if (lane == 0) s[warp] = v;
      __syncthreads();
      s += warp / warps * warps;
    }
    v = make_float2(0.f, 0.f);
    const int n = CLUSTER ? warps * ctas : warps;
    for (int i = 0; i < n; ++i) v.x += s[i].x, v.y += s[i].y;
    return v;
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
__global__ void __launch_bounds__(512) k_norm_forward(const __grid_constant__ NormParams P, int threads) {
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
      m = sum(make_float2(m, 0.f)).x * P.inv_d;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((lane + k * threads) * V < P.d)
#pragma unroll
        for (int i = 0; i < V; ++i) q = fmaf(v[k * V + i] - m, v[k * V + i] - m, q);
    return make_float2(m, rsqrtf(sum(make_float2(q, 0.f)).x * P.inv_d + P.eps));
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
struct NormBackParams {
  NormParams f;
  const void *dr, *dh;
  int64_t lddr, lddh;
  void *dx, *dz, *dgate;  // contiguous; dgate: of a gate of every token
  float *part;            // [groups][sums][d], or null
  int sums;               // vectors that are summed over the rows
  int at_w, at_b, at_gate, at_wp, at_bp;  // their places in part, -1: not asked for
};

// 8 values of a row a thread, a row to `threads` threads of a CTA (CLUSTER: of all the cluster's CTAs),
// rows dealt to these groups in turn; a group keeps its columns' sums in registers.  FULL: every sum,
// else dw and dw_post alone.
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
  float sw[8], sb[FULL ? 8 : 1], sg[FULL ? 8 : 1], swp[8], sbp[FULL ? 8 : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sw[i] = swp[i] = 0.f;
    if (FULL) sb[i] = sg[i] = sbp[i] = 0.f;
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
      const float2 s = sum(make_float2(s1, s2));
      const float m1 = F.pre == SFNN_NORM_LAYER ? s.x * F.inv_d : 0.f, m2 = s.y * F.inv_d;
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
        const float p = q * g[i];
        if (FULL) sg[j] += dg[i], sbp[j] += p;
        swp[j] = fmaf(p, z[j], swp[j]);
        dr[j] = p * w[i];
        n1 += dr[j];
        n2 = fmaf(dr[j], z[j], n2);
      }
      if (P.dgate) store_values<false, V>(P.dgate, row * F.d + c, 0, bf16, dg);
    }
    if (!P.dz) continue;
    if (F.post != SFNN_NORM_NONE) {
      const float2 s = sum(make_float2(n1, n2));
      n1 = F.post == SFNN_NORM_LAYER ? s.x * F.inv_d : 0.f;
      n2 = s.y * F.inv_d;
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
  put(P.at_w, sw);
  put(P.at_wp, swp);
  if (FULL) {
    put(P.at_b, sb);
    put(P.at_gate, sg);
    put(P.at_bp, sbp);
  }
}

// out[s][c] = sum over the groups of part[group][s][c], in their order: 32 columns a CTA, a share of
// the groups a warp.
struct NormSums {
  const float *part;
  int groups, sums, d;
  void *out[5];
};
template <bool bf16>
__global__ void __launch_bounds__(256) k_norm_sums(const __grid_constant__ NormSums P) {
  __shared__ float s[8][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cols = (int64_t)P.sums * P.d, c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < cols)
#pragma unroll 4
    for (int g = warp; g < P.groups; g += 8) v += __ldg(P.part + g * cols + c);
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][lane];
    const int which = (int)(c / P.d);
    static_cast<uint16_t *>(P.out[which])[c - (int64_t)which * P.d] = (uint16_t)pack16(v, 0.f, bf16);
  }
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
  const int per = P.d <= 256 ? 8 : 16;  // values a thread
  int ctas = 1;
  while (P.d > per * 512 * ctas) ctas *= 2;
  int block = (int)up((P.d + per * ctas - 1) / (per * ctas), 32);
  const int threads = block * ctas, rows = ctas > 1 ? 1 : std::max(1, 128 / block);
  block *= rows;
  const int64_t units = (P.T + (int64_t)rows - 1) / rows;  // (T is at most 2^28, a row's CTAs at most 4)
  auto run = [&](auto kernel) { return launch_rows(kernel, (int)(units * ctas), block, ctas, threads, P, s); };
  if (ctas > 1) return vec ? run(k_norm_forward<bf16, 8, 2, true>) : run(k_norm_forward<bf16, 1, 16, true>);
  if (per == 8) return vec ? run(k_norm_forward<bf16, 8, 1, false>) : run(k_norm_forward<bf16, 1, 8, false>);
  return vec ? run(k_norm_forward<bf16, 8, 2, false>) : run(k_norm_forward<bf16, 1, 16, false>);
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
int64_t back_workspace(int64_t T, int d, int sums, int sms) {  // (the larger grid)
  return up(back_shape(std::max<int64_t>(T, 1), d, false, sms).groups() * sums * d * 4, 256);
}

template <bool bf16, int V, bool FULL>
cudaError_t run_backward(const NormBackParams &P, const BackShape &b, cudaStream_t s) {
  return b.ctas == 1 ? launch_rows(k_norm_backward<bf16, V, FULL, false>, b.grid, b.block, 1, b.threads, P, s)
                     : launch_rows(k_norm_backward<bf16, V, FULL, true>, b.grid, b.block, b.ctas, b.threads, P, s);
}
template <bool bf16>
cudaError_t run_backward(const NormBackParams &P, bool vec, bool full, const BackShape &b, cudaStream_t s) {
  if (vec) return full ? run_backward<bf16, 8, true>(P, b, s) : run_backward<bf16, 8, false>(P, b, s);
  return full ? run_backward<bf16, 1, true>(P, b, s) : run_backward<bf16, 1, false>(P, b, s);
}

}  // namespace
}  // namespace sfnn

using namespace sfnn;

extern "C" {

int64_t sfnn_norm_workspace(int32_t T, int32_t d) {
  if (T < 0 || d < 1 || d > kMaxWidth) return -1;
  return back_workspace(T, d, 5, std::max(1, device_sms()));
}

sfnn_status sfnn_norm_forward(const sfnn_norm_desc *q, void *r, int64_t ldr, void *h, int64_t ldh, float *stats,
                              sfnn_stream_t stream) {
  const sfnn_status st = check(q);
  if (st != SFNN_OK) return st;
  if (q->T == 0) return SFNN_OK;
  NormParams P = params(q);
  if ((q->z && !rows_ok(r, ldr, q->d, P.x32)) || (q->pre != SFNN_NORM_NONE && !rows_ok(h, ldh, q->d, false)) || !on(stats, 16))
    return SFNN_ERR_INVALID_ARG;
  P.r = q->z ? r : nullptr;
  P.h = q->pre != SFNN_NORM_NONE ? h : nullptr;
  P.ldr = ldr;
  P.ldh = ldh;
  P.stats = stats;
  const bool vec = vectors(P) && vectors(P.r, ldr) && vectors(P.h, ldh);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = q->dtype == SFNN_BF16 ? run_forward<true>(P, vec, s) : run_forward<false>(P, vec, s);
  return e == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
}

sfnn_status sfnn_norm_backward(const sfnn_norm_desc *q, const float *stats, const void *dr, int64_t lddr, const void *dh,
                               int64_t lddh, void *dx, void *dz, void *dgate, void *dw, void *db, void *dpost_w,
                               void *dpost_b, void *ws, int64_t ws_bytes, sfnn_stream_t stream) {
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
  NormBackParams P{};
  auto asked = [&](void *out) {
    if (!out) return -1;
    S.out[S.sums] = out;
    return S.sums++;
  };
  P.at_w = asked(dw);
  P.at_wp = asked(dpost_w);
  const int plain = S.sums;
  P.at_b = asked(db);
  P.at_gate = asked(one_gate ? dgate : nullptr);
  P.at_bp = asked(dpost_b);
  const bool full = S.sums > plain;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (q->T == 0) {  // sums over no tokens
    for (int i = 0; i < S.sums; ++i)
      if (cudaMemsetAsync(S.out[i], 0, (size_t)q->d * 2, s) != cudaSuccess) return SFNN_ERR_CUDA;
    return SFNN_OK;
  }
  const bool x32 = q->x_dtype == SFNN_F32;
  if ((dr && !rows_ok(dr, lddr, q->d, x32)) || (dh && !rows_ok(dh, lddh, q->d, false)) || !stats || !on(stats, 16))
    return SFNN_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (sms < 1) return SFNN_ERR_CUDA;
  if (S.sums && (!ws || !on(ws, 16) || ws_bytes < back_workspace(q->T, q->d, S.sums, sms))) return SFNN_ERR_INVALID_ARG;
  P.f = params(q);
  P.f.stats = const_cast<float *>(stats);
  P.dr = dr, P.lddr = lddr;
  P.dh = dh, P.lddh = lddh;
  P.dx = dx, P.dz = dz;
  P.dgate = one_gate ? nullptr : dgate;
  P.part = S.sums ? static_cast<float *>(ws) : nullptr;
  P.sums = S.sums;
  const bool vec = vectors(P.f) && vectors(dr, lddr) && vectors(dh, lddh) && vectors(dx, 0) && vectors(dz, 0) &&
                   vectors(P.dgate, 0);
  const BackShape b = back_shape(q->T, q->d, full, sms);
  const cudaError_t e = bf16 ? run_backward<true>(P, vec, full, b, s) : run_backward<false>(P, vec, full, b, s);
  if (e != cudaSuccess) return SFNN_ERR_CUDA;
  if (S.sums) {
    S.part = P.part;
    S.groups = (int)b.groups();
    S.d = q->d;
    const dim3 grid((unsigned)(((int64_t)S.sums * q->d + 31) / 32));
    if ((bf16 ? launch_pdl(k_norm_sums<true>, grid, dim3(256), 0, s, S)
              : launch_pdl(k_norm_sums<false>, grid, dim3(256), 0, s, S)) != cudaSuccess)
      return SFNN_ERR_CUDA;
  }
  return SFNN_OK;
}

}  // extern "C"
