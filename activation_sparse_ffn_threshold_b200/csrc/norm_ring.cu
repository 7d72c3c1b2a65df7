// norm_ring.cu -- the norms' kernels whose rows pass through shared memory (formulas in norm.cu).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.cuh"
#include "norm.cuh"

namespace sfnn {
namespace {

// With a row's values held in registers nothing is on its way from memory while the row's sums go
// round.  These kernels keep the next rows coming: a CTA an SM, its threads in groups that
// each take a row at a time, with stages of their own that bulk copies fill while the rows before are
// worked on; a group waits for nothing but its own rows and sums.  The values stay in shared memory
// until each is needed, beside them the channels' weights.  A thread has 16 values: two vectors of 8, or,
// where rows do not start on 16 bytes (ODD), 16 single columns, neighbouring lanes' side by side.  Such a
// row is copied with what the 16-byte blocks at its ends hold besides.
//
// Bound by bytes.  Measured, bf16, both norms and one gate row (us; bytes over the time in TB/s):
//     8192 x 4096   forward 52 (5.2)   backward 82 and 5 for the sums (4.9)
//     4000 x 8192   forward 51 (5.1)   backward 88 (4.5)
// Backward from 4097 values on there is one group (8192 x 5120: 133 us, 3.8 TB/s), and of an fp32 stream near 8192
// one stage, so that nothing is on its way while a row is worked on (4000 x 8192: 148 us, 4.0 TB/s).
// Forward the longest rows are 8856 values of an fp32 stream with everything that may be there, 16384 at most.
// Rows held in registers instead took 99 for 4000 x 8192 and 244 for 8192 x 4096 backward.
constexpr int kMaxStages = 4;
constexpr int kMaxGroups = 16;  // 15 named barriers; 16 groups are warps, which need none
constexpr int kRingValues = 16;
enum { kOfX, kOfZ, kOfDr, kOfDh, kOfGate, kOfRows };

struct RingParams {
  const void *p[kOfRows];  // arrays whose rows pass through the ring (null: none)
  int64_t ld[kOfRows];     // bytes
  int bytes[kOfRows];      // of a row
  int at[kOfRows];         // its place in a stage
  int stage, stages;       // bytes of a stage (a row of every array)
  int groups, threads;     // of a CTA, of a group
  int held[4];             // where the channels' weights lie behind the stages (-1: all the same, see weight())
};
// The channels' weights as the kernels use them, in 32 bits: c gate w_post (without the gate where every
// token has its own), w, and for FULL c gate b_post and b.
enum { kPostW, kPreW, kPostB, kPreB, kWeights };

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
  alignas(16) float slots[2][2][64];  // [turn][value][a group's warps, rounded up to 4], read four at a time
};

// WIDE: X or Z is fp32.  FULL: means and biases.  EXACT: what is usual -- both vectors of every thread are
// there (a width of whole 512s), X, Z, the pre norm and, backward, all gradients, no gate for each
// token -- whose tests cost as much as the arithmetic (backward, 4096 wide: 727 instructions a warp and
// row with them).
template <bool bf16, bool WIDE, bool FULL, bool EXACT, bool ODD>
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
  int have;              // ODD: columns of this thread

  __device__ __forceinline__ Ring(const RingParams &R_, const NormParams &F_, unsigned char *smem, RingSmem &S_, int32_t *err_)
      : R(R_), F(F_), S(S_), err(err_), slot(0), phase(0), turn(0), dead(false) {
    mine = threadIdx.x / R.threads;
    lane = threadIdx.x - mine * R.threads;
    have = lane < F.d ? (F.d - lane + R.threads - 1) / R.threads : 0;
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
    // The weights, all requested together (one after the other: 0.5 to 1 us more a launch).
    float *const to = reinterpret_cast<float *>(smem + (size_t)R.groups * R.stages * R.stage);
    const uint16_t *const from[kWeights] = {
        static_cast<const uint16_t *>(F.wp), static_cast<const uint16_t *>(F.w), static_cast<const uint16_t *>(F.bp),
        static_cast<const uint16_t *>(F.b)};
    const uint16_t *const gate = F.ldg ? nullptr : static_cast<const uint16_t *>(F.gate);
    if (!ODD) {
#pragma unroll 1
      for (int c = threadIdx.x * 8; c < F.d; c += blockDim.x * 8) {
        uint4 raw[kWeights], rg;
#pragma unroll
        for (int k = 0; k < kWeights; ++k)
          if (R.held[k] >= 0 && from[k]) raw[k] = ld_keep(from[k] + c);
        if (gate) rg = ld_keep(gate + c);
#pragma unroll
        for (int k = 0; k < kWeights; ++k) {
          if (R.held[k] < 0) continue;
          Pair v[4], g[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = g[i] = both(1.f);
          if (from[k]) widen8(raw[k], v);
          if (gate) widen8(rg, g);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k == kPostW || k == kPostB) v[i] = mul2(mul2(g[i], both(F.c)), v[i]);
          ulonglong2 *q = reinterpret_cast<ulonglong2 *>(to + R.held[k] / 4 + c);
          q[0] = make_ulonglong2(v[0], v[1]);
          q[1] = make_ulonglong2(v[2], v[3]);
        }
      }
    } else {
#pragma unroll 1
      for (int c0 = threadIdx.x; c0 < F.d; c0 += 8 * blockDim.x) {
        float v[kWeights][8], g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = c0 + i * (int)blockDim.x;
#pragma unroll
          for (int k = 0; k < kWeights; ++k) v[k][i] = R.held[k] >= 0 && from[k] && c < F.d ? load16(from[k], c, bf16) : 1.f;
          g[i] = gate && c < F.d ? load16(gate, c, bf16) : 1.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = c0 + i * (int)blockDim.x;
#pragma unroll
          for (int k = 0; k < kWeights; ++k)
            if (R.held[k] >= 0 && c < F.d) to[R.held[k] / 4 + c] = k == kPostW || k == kPostB ? g[i] * F.c * v[k][i] : v[k][i];
        }
      }
    }
    __syncthreads();
  }
  // Bytes of row r of an array that lie before it in its first 16-byte block.
  __device__ __forceinline__ uint32_t before(int k, int r) const {
    return ODD ? ((uint32_t)reinterpret_cast<uintptr_t>(R.p[k]) + (uint32_t)r * (uint32_t)R.ld[k]) & 15u : 0u;
  }
  __device__ __forceinline__ void request(int r, int s) const {  // the group's first warp, an array a lane
    if (r >= F.T) return;
    uint64_t *bar = &S.full[mine * R.stages + s];
    uint32_t total = (uint32_t)R.stage;
    if (ODD) {
      total = 0;
#pragma unroll
      for (int k = 0; k < kOfRows; ++k)
        if (R.p[k]) total += (before(k, r) + (uint32_t)R.bytes[k] + 15u) & ~15u;
    }
    if (lane == 0) bar_expect_tx(bar, total);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kOfRows; ++k)
      if (lane == k && R.p[k]) {
        const uint32_t skip = before(k, r);
        bulk_load(stage0 + (uint32_t)(s * R.stage + R.at[k]),
                  static_cast<const unsigned char *>(R.p[k]) + (int64_t)r * R.ld[k] - skip,
                  ODD ? (skip + (uint32_t)R.bytes[k] + 15u) & ~15u : (uint32_t)R.bytes[k], bar);
      }
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

  // Columns of half k (0 or 1) of this thread's values: 8 from here on, or (ODD) the i-th of them.
  __device__ __forceinline__ int column(int k) const { return lane * 8 + k * R.threads * 8; }
  __device__ __forceinline__ int column(int k, int i) const { return lane + (8 * k + i) * R.threads; }
  __device__ __forceinline__ bool in(int k) const { return EXACT || ODD || column(k) < F.d; }
  __device__ __forceinline__ bool in(int k, int i) const { return 8 * k + i < have; }

  // Half k of the row at hand, of an array; zeros past the row (ODD).
  __device__ __forceinline__ void value8(int a, int k, bool wide, Pair v[4]) const {
    if (ODD) {
      const uint32_t p = cur + (uint32_t)R.at[a] + before(a, row);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = 0.f;
        if (!in(k, i)) continue;
        if (WIDE && wide) {
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[i]) : "r"(p + (uint32_t)column(k, i) * 4u) : "memory");
        } else {
          uint16_t h;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(p + (uint32_t)column(k, i) * 2u) : "memory");
          f[i] = bf16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
    } else if (WIDE && wide) {
      const uint32_t p = cur + (uint32_t)(R.at[a] + column(k) * 4);
      lds_pairs(p, v[0], v[1]);
      lds_pairs(p + 16, v[2], v[3]);
    } else {
      widen8(lds_u4(cur + (uint32_t)(R.at[a] + column(k) * 2)), v);
    }
  }
  // Weights of half k, as the enumeration above says; zeros past the row (ODD).
  __device__ __forceinline__ void weight(int a, int k, Pair v[4]) const {
    const bool held = (EXACT && (a == kPostW || a == kPreW)) || R.held[a] >= 0;
    const float fill = a == kPostW ? F.c : a == kPreW ? 1.f : 0.f;
    if (ODD) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = in(k, i) ? fill : 0.f;
        if (held && in(k, i))
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[i]) : "r"(weights + (uint32_t)(R.held[a] + column(k, i) * 4)) : "memory");
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
    } else if (held) {
      const uint32_t p = weights + (uint32_t)(R.held[a] + column(k) * 4);
      lds_pairs(p, v[0], v[1]);
      lds_pairs(p + 16, v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = both(fill);
    }
  }
  // What a mean was taken from: zeros again past the row.
  __device__ __forceinline__ void cut(int k, Pair v[4]) const {
    if (!ODD) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = apart(v[i]);
      v[i] = pair(in(k, 2 * i) ? f.x : 0.f, in(k, 2 * i + 1) ? f.y : 0.f);
    }
  }
  static __device__ __forceinline__ void widen8(const uint4 &w, Pair v[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16 ? make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u)) : unpack16(u[i], false);
      v[i] = pair(f.x, f.y);
    }
  }
  // Half k to the row that starts `at` elements behind p.
  __device__ __forceinline__ void store(void *p, int64_t at, int k, bool wide, const Pair v[4]) const {
    if (ODD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = apart(v[i / 2]);
        const float one = i % 2 ? f.y : f.x;
        if (!in(k, i)) continue;
        if (WIDE && wide)
          static_cast<float *>(p)[at + column(k, i)] = one;
        else
          static_cast<uint16_t *>(p)[at + column(k, i)] = (uint16_t)pack16(one, 0.f, bf16);
      }
    } else if (WIDE && wide) {
      ulonglong2 *q = reinterpret_cast<ulonglong2 *>(static_cast<float *>(p) + at + column(k));
      q[0] = make_ulonglong2(v[0], v[1]);
      q[1] = make_ulonglong2(v[2], v[3]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = apart(v[i]);
        u[i] = pack16(f.x, f.y, bf16);
      }
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at + column(k)) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  __device__ __forceinline__ bool gated() const { return !EXACT && R.p[kOfGate]; }  // a gate for each token
  // (Z - mean) and post(Z) gate c of half k.
  __device__ __forceinline__ void branch(int k, float mz, float sz, Pair z[4], Pair v[4]) const {
    value8(kOfZ, k, F.z32, z);
    weight(kPostW, k, v);
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
      weight(kPostB, k, b);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = both(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fma2(v[i], both(sz), b[i]);
    if (!gated()) return;
    value8(kOfGate, k, false, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], b[i]);
  }
};

constexpr int kForwardThreads = 1024, kBackwardThreads = 512;

template <bool bf16, bool WIDE, bool FULL, bool EXACT, bool ODD>
__global__ void __launch_bounds__(kForwardThreads, 1) k_norm_forward_ring(const __grid_constant__ NormParams P,
                                                                          const __grid_constant__ RingParams R, int32_t *err) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ RingSmem more;
  pdl_wait();
  pdl_launch_dependents();
  Ring<bf16, WIDE, FULL, EXACT, ODD> ring(R, P, ring_smem, more, err);
  const bool has_z = EXACT || P.z, has_pre = EXACT || P.pre != SFNN_NORM_NONE;
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
          if (!ring.in(k)) continue;
          Pair z[4];
          ring.value8(kOfZ, k, P.z32, z);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (FULL && pass) z[i] = add2(z[i], both(-mz));
          if (FULL && pass) ring.cut(k, z);
#pragma unroll
          for (int i = 0; i < 4; ++i) q = FULL && !pass ? add2(q, z[i]) : fma2(z[i], z[i], q);
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
      Pair *rk = r + 4 * k, z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rk[i] = both(0.f);
      if (!ring.in(k)) continue;
      ring.value8(kOfX, k, P.x32, rk);
      if (has_z) {
        Pair v[4];
        ring.branch(k, mz, sz, z, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) rk[i] = fma2(rk[i], both(P.a), v[i]);
      }
      if (has_z) ring.store(P.r, (int64_t)ring.row * P.ldr, k, P.x32, rk);
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
          if (ring.in(k)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r[4 * k + i] = add2(r[4 * k + i], both(-mr));
            ring.cut(k, r + 4 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) q = fma2(r[4 * k + i], r[4 * k + i], q);
          }
      }
      sr = rsqrtf(mean_of(q) + P.eps);
    }
    ring.release();
    if (has_pre) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
          if (!ring.in(k)) continue;
        Pair w[4], b[4];
        ring.weight(kPreW, k, w);
        if (FULL) ring.weight(kPreB, k, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair hat = mul2(r[4 * k + i], both(sr));
          w[i] = FULL ? fma2(hat, w[i], b[i]) : mul2(hat, w[i]);
        }
        ring.store(P.h, (int64_t)ring.row * P.ldh, k, false, w);
      }
    }
    if (P.stats && ring.lane == 0) *reinterpret_cast<float4 *>(P.stats + (int64_t)ring.row * 4) = make_float4(mr, sr, mz, sz);
  }
}

// FULL: the sums of dH and D as well.  PLAIN: neither a post norm nor a gate (a block whose norm comes
// first): dZ is D scaled, Z's own sums and their registers go (8192 x 4096 bf16,
// LayerNorm 119 -> 80 us, RMS 79 -> 72).
template <bool bf16, bool WIDE, bool FULL, bool EXACT, bool ODD, bool PLAIN>
__global__ void __launch_bounds__(kBackwardThreads, 1) k_norm_backward_ring(const __grid_constant__ NormBackParams P,
                                                                            const __grid_constant__ RingParams R) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ RingSmem more;
  pdl_wait();
  pdl_launch_dependents();
  const NormParams &F = P.f;
  Ring<bf16, WIDE, FULL, EXACT, ODD> ring(R, F, ring_smem, more, P.err);
  const bool has_z = EXACT || F.z, has_dh = EXACT || P.dh, has_dr = EXACT || P.dr, has_dx = EXACT || P.dx;
  constexpr int kOwn = PLAIN ? 1 : 8;  // what belongs to Z's own norm and gate
  Pair sw[8], sb[FULL ? 8 : 1], sum1[kOwn], sum0[FULL ? kOwn : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sw[i] = both(0.f);
    if (FULL) sb[i] = both(0.f);
    if (!PLAIN) sum1[i] = both(0.f);
    if (!PLAIN && FULL) sum0[i] = both(0.f);
  }
  const bool has_dz = EXACT || P.dz, two_sums = !PLAIN && has_dz && F.post != SFNN_NORM_NONE;
  // (of columns past d these stay zero)
  Pair D[8], hat[8], z[kOwn];
#pragma unroll
  for (int i = 0; i < 8; ++i) D[i] = hat[i] = both(0.f);
#pragma unroll
  for (int i = 0; i < kOwn; ++i) z[i] = both(0.f);
  for (; ring.row < F.T; ring.next()) {
    const float4 st = __ldg(reinterpret_cast<const float4 *>(F.stats) + ring.row);  // of R, of Z: mean, 1 / deviation
    ring.wait();
    Pair s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Pair *Dk = D + 4 * k, *hk = hat + 4 * k, *zk = PLAIN ? z : z + 4 * k;
      if (!ring.in(k)) continue;
      if (has_dh) {
        ring.value8(kOfX, k, F.x32, hk);
        if (PLAIN && has_z) {  // R^ = a s X + c s Z - s mean
          Pair v[4];
          ring.value8(kOfZ, k, F.z32, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = FULL ? fma2(v[i], both(F.c * st.y), both(-st.x * st.y)) : mul2(v[i], both(F.c * st.y));
            hk[i] = fma2(hk[i], both(F.a * st.y), v[i]);
          }
        } else if (has_z) {  // R^ = a s X + s (c gate post(Z) - mean)
          Pair v[4];
          ring.branch(k, st.z, st.w * (FULL || ring.gated() ? 1.f : st.y), zk, v);
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
        ring.value8(kOfDh, k, false, dh);
        ring.weight(kPreW, k, Dk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          Dk[i] = mul2(dh[i], Dk[i]);
          if (FULL) s1 = add2(s1, Dk[i]), sb[4 * k + i] = add2(sb[4 * k + i], dh[i]);
          s2 = fma2(Dk[i], hk[i], s2);
          sw[4 * k + i] = fma2(dh[i], hk[i], sw[4 * k + i]);
        }
      } else if (!PLAIN && has_z) {
        ring.value8(kOfZ, k, F.z32, zk);
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
      Pair *Dk = D + 4 * k, *hk = hat + 4 * k, *zk = PLAIN ? z : z + 4 * k;
      if (!ring.in(k)) continue;
      Pair v[4];
      if (has_dr)
        ring.value8(kOfDr, k, F.x32, v);
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
        ring.store(P.dx, (int64_t)ring.row * F.d, k, F.x32, v);
      }
      if (PLAIN && has_dz) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul2(both(F.c), Dk[i]);
        ring.store(P.dz, (int64_t)ring.row * F.d, k, F.z32, v);
      }
      if (PLAIN || !has_z) continue;
      Pair w[4];
      ring.weight(kPostW, k, w);
      if (ring.gated()) {
        Pair g[4];
        ring.value8(kOfGate, k, false, g);
        if (P.dgate) {
          if (FULL) ring.weight(kPostB, k, v);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = mul2(Dk[i], fma2(mul2(zk[i], both(st.w)), w[i], FULL ? v[i] : both(0.f)));
          ring.store(P.dgate, (int64_t)ring.row * F.d, k, false, v);
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
    if (PLAIN || !has_dz) continue;
#pragma unroll
    for (int k = 0; k < (PLAIN ? 0 : 2); ++k) {
      if (!ring.in(k)) continue;
      Pair v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = fma2(z[4 * k + i], both(m2), D[4 * k + i]);
        if (FULL) v[i] = add2(v[i], both(m1));
      }
      ring.store(P.dz, (int64_t)ring.row * F.d, k, F.z32, v);
    }
  }
  if (!P.part) return;
  // The groups' sums, by way of shared memory (no copy is on its way any more), as one of the CTA's.
  const int width = P.sums * F.d;
  float *part = P.part + (int64_t)blockIdx.x * width;
  float *own = reinterpret_cast<float *>(ring_smem) + (size_t)ring.mine * width;
  __syncthreads();
  auto put = [&](int at, const Pair *v) {
    if (at < 0) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!ring.in(k)) continue;
      float *to = own + (size_t)at * F.d;
      if (ODD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = apart(v[4 * k + i / 2]);
          if (ring.in(k, i)) to[ring.column(k, i)] = i % 2 ? f.y : f.x;
        }
      } else {
        ulonglong2 *q = reinterpret_cast<ulonglong2 *>(to + ring.column(k));
        q[0] = make_ulonglong2(v[4 * k], v[4 * k + 1]);
        q[1] = make_ulonglong2(v[4 * k + 2], v[4 * k + 3]);
      }
    }
  };
  put(P.at[kSumW], sw);
  if (FULL) put(P.at[kSumB], sb);
  if (!PLAIN) put(P.at[kSum1], sum1);
  if (!PLAIN && FULL) put(P.at[kSum0], sum0);
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    const float *from = reinterpret_cast<const float *>(ring_smem) + i;
    float v = 0.f;
    for (int g = 0; g < R.groups; ++g) v += from[(size_t)g * width];
    part[i] = v;
  }
}

// The rows' way through shared memory.
constexpr int kRingSmem = 225 * 1024;
// Where the backward kernel has more values than registers (Z's own sums with means or biases) it takes no
// more than this for stages beyond the second: what is left of the SM's 256 KB serves the loads of what it
// spilled (8192 x 4096 bf16, LayerNorm and RMS: three stages 133 us, two 121; 16384 x 2048 124 and 115).
constexpr int kLeftSmem = 194 * 1024;
struct RingShape {
  int block, grid, smem;
  bool fits;
};
bool plain_branch(const NormParams &F) { return F.post == SFNN_NORM_NONE && !F.gate; }
int ring_threads(int d) { return (int)up((d + kRingValues - 1) / kRingValues, 32); }
RingShape ring_shape(RingParams &R, const NormParams &F, bool odd, bool exact, bool backward, const void *dr, int64_t lddr,
                     const void *dh, int64_t lddh, int sums, int most_threads, int most, int sms) {
  const int d = F.d;
  R.threads = ring_threads(d);
  auto row = [&](int k, const void *p, int64_t ld, bool wide) {
    R.p[k] = p;
    R.ld[k] = ld * (wide ? 4 : 2);
    R.bytes[k] = d * (wide ? 4 : 2);
    R.at[k] = R.stage;
    if (p) R.stage += odd ? (int)up(R.bytes[k] + 15, 16) : R.bytes[k];
  };
  row(kOfX, F.x, F.ldx, F.x32);
  row(kOfZ, F.z, F.ldz, F.z32);
  row(kOfDr, dr, lddr, F.x32);
  row(kOfDh, dh, lddh, false);
  row(kOfGate, F.ldg ? F.gate : nullptr, F.ldg, false);
  int held = 0;
  const bool gate = F.gate && !F.ldg;
  const bool needed[kWeights] = {(exact && !(backward && plain_branch(F))) || (F.z && (gate || F.wp)), exact || F.w, F.bp != nullptr, F.b && !backward};
  for (int k = 0; k < kWeights; ++k) {
    R.held[k] = needed[k] ? held : -1;
    held += needed[k] ? (int)up(d * 4, 16) : 0;
  }
  // As many groups as threads allow, fewer where that leaves them two stages each, or where few rows
  // then reach all SMs.
  const int budget = kRingSmem - held;
  R.groups = std::max(1, std::min(R.threads == 32 ? kMaxGroups : kMaxGroups - 1, most_threads / R.threads));
  R.groups = std::min(R.groups, std::max(1, (F.T + sms - 1) / sms));
  while (R.groups > 1 && (R.groups * 2 * R.stage > budget || R.groups * sums * d * 4 > kRingSmem)) --R.groups;
  R.stages = std::max(0, std::min(kMaxStages, budget / (R.groups * R.stage)));
  R.stages = std::min(R.stages, std::max(2, (most - held) / (R.groups * R.stage)));
  RingShape s;
  s.block = R.threads * R.groups;
  s.smem = std::max(R.groups * R.stages * R.stage + held, R.groups * sums * d * 4);
  s.grid = (int)std::min<int64_t>(((int64_t)F.T + R.groups - 1) / R.groups, sms);
  s.fits = R.threads <= most_threads && R.stages > 0 && s.smem <= kRingSmem;
  return s;
}

bool exact_rows(const NormParams &P, bool vec) {
  return vec && P.d % (32 * kRingValues) == 0 && P.z && P.pre != SFNN_NORM_NONE && !P.ldg;
}

template <class Kernel, class... Args>
cudaError_t launch_ring(Kernel kernel, const RingShape &s, std::atomic<uint64_t> &ready, cudaStream_t stream, const Args &...args) {
  const cudaError_t e = allow_smem(kernel, kRingSmem, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)s.grid), dim3((unsigned)s.block), (size_t)s.smem, stream, args...);
}
template <bool bf16, bool WIDE, bool FULL, bool EXACT, bool ODD>
cudaError_t run_ring(const RingShape &s, const NormParams &P, const RingParams &R, int32_t *err, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  return launch_ring(k_norm_forward_ring<bf16, WIDE, FULL, EXACT, ODD>, s, ready, stream, P, R, err);
}
template <bool bf16, bool WIDE, bool FULL, bool EXACT, bool ODD>
cudaError_t run_ring(const RingShape &s, const NormBackParams &P, const RingParams &R, int32_t *, cudaStream_t stream) {
  static std::atomic<uint64_t> ready[2];
  return plain_branch(P.f) ? launch_ring(k_norm_backward_ring<bf16, WIDE, FULL, EXACT, ODD, true>, s, ready[1], stream, P, R)
                           : launch_ring(k_norm_backward_ring<bf16, WIDE, FULL, EXACT, ODD, false>, s, ready[0], stream, P, R);
}
template <bool bf16, bool WIDE, bool FULL, class Params>
cudaError_t run_ring(bool exact, bool odd, const RingShape &s, const Params &P, const RingParams &R, int32_t *err, cudaStream_t stream) {
  return odd     ? run_ring<bf16, WIDE, FULL, false, true>(s, P, R, err, stream)
         : exact ? run_ring<bf16, WIDE, FULL, true, false>(s, P, R, err, stream)
                 : run_ring<bf16, WIDE, FULL, false, false>(s, P, R, err, stream);
}
template <bool bf16, class Params>
cudaError_t run_ring(bool wide, bool full, bool exact, bool odd, const RingShape &s, const Params &P, const RingParams &R,
                     int32_t *err, cudaStream_t stream) {
  if (wide)
    return full ? run_ring<bf16, true, true>(exact, odd, s, P, R, err, stream) : run_ring<bf16, true, false>(exact, odd, s, P, R, err, stream);
  return full ? run_ring<bf16, false, true>(exact, odd, s, P, R, err, stream) : run_ring<bf16, false, false>(exact, odd, s, P, R, err, stream);
}

}  // namespace

cudaError_t norm_forward_ring(const NormParams &P, int32_t *err, bool bf16, bool vec, int sms, cudaStream_t s, RingPlan &plan) {
  const bool full = P.pre == SFNN_NORM_LAYER || P.post == SFNN_NORM_LAYER || P.b || P.bp, exact = exact_rows(P, vec);
  RingParams R{};
  const RingShape shape = ring_shape(R, P, !vec, exact, false, nullptr, 0, nullptr, 0, 0, kForwardThreads, kRingSmem, sms);
  plan = {shape.fits, shape.grid};
  if (!shape.fits) return cudaSuccess;
  return bf16 ? run_ring<true>(P.x32 || P.z32, full, exact, !vec, shape, P, R, err, s)
              : run_ring<false>(P.x32 || P.z32, full, exact, !vec, shape, P, R, err, s);
}
cudaError_t norm_backward_ring(const NormBackParams &P, bool sums_all, bool bf16, bool vec, int sms, cudaStream_t s, RingPlan &plan) {
  const NormParams &F = P.f;
  const bool full = F.pre == SFNN_NORM_LAYER || F.post == SFNN_NORM_LAYER || F.bp || sums_all;
  const bool exact = exact_rows(F, vec) && P.dr && P.dh && P.dx && P.dz;
  RingParams R{};
  const RingShape shape = ring_shape(R, F, !vec, exact, true, P.dr, P.lddr, P.dh, P.lddh, P.sums, kBackwardThreads,
                                     full && !plain_branch(F) ? kLeftSmem : kRingSmem, sms);
  plan = {shape.fits, shape.grid};
  if (!shape.fits) return cudaSuccess;
  return bf16 ? run_ring<true>(F.x32 || F.z32, full, exact, !vec, shape, P, R, P.err, s)
              : run_ring<false>(F.x32 || F.z32, full, exact, !vec, shape, P, R, P.err, s);
}

}  // namespace sfnn
