// dense.cu -- the dense product of the gated FFN on the tensor cores (tcgen05, CTA pairs).
//
// Forward:   G = X Wg^T + b, U = X Wu^T, H = relu(G) * U in one kernel; Y = H Wd^T.
// Backward:  dH = dY Wd (epilogue: dU = dH * relu(G), dG = dH * U * [G > 0], H again),
//            dX = dG Wg + dU Wu (one accumulation over both), dWg = dG^T X, dWu = dU^T X,
//            dWd = dY^T H.
// Every one of them is C = A . B^T with K contiguous ("K-major") or M / N contiguous
// ("MN-major") operands, so one kernel serves all: no operand is transposed in memory.
//
// A persistent kernel, one pair of CTAs per pair of SMs, tiles of 256 x 256: each CTA holds
// 128 rows of A and 128 rows of B per 64-deep K chunk (32 KB a stage), the pair's MMA
// (M = 256, N = 256) reads both CTAs' shared memory, so an operand byte loaded feeds twice
// the products of a single CTA's tile -- what bounds a 16-bit product on this part is the
// tensor pipe only as long as L2 -> shared memory traffic stays under it.  Warp 0 loads
// (TMA, 128-byte swizzle), warp 1 of the pair's first CTA issues the MMAs, warps 2-9 run
// the epilogue of the tile before out of the other half of tensor memory (2 x 256 columns).
//
// Every wait is bounded (about a second); one that runs out latches SFNN_ERR_TIMEOUT and the
// kernel leaves in order: its loads have landed by then, tensor memory is freed.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kThreads = 320;
constexpr int kStages = 6;
constexpr uint32_t kStageBytes = 32768;  // per CTA: 128 x 64 of A, 128 x 64 of B
constexpr int kTile = 256;
constexpr int kTmem = 512;

struct TilePos {
  int m, n;
};
// Tiles are walked in bands of 8 rows of tiles, down a band's columns: the ~74 tiles in
// flight then span about 8 x 9 tiles, whose A and B rows L2 holds.
__device__ __forceinline__ TilePos tile_pos(int t, int tiles_m, int tiles_n) {
  constexpr int kBand = 8;
  const int per = kBand * tiles_n;
  const int band = t / per, r = t - band * per;
  const int rows = min(kBand, tiles_m - band * kBand);
  return {band * kBand + r % rows, r / rows};
}

// The unit of work that pair `i` takes in its `n`-th turn (-1: none left).
struct Walk {
  int pair, pairs, first, rest, extra, mine, light;
  __device__ __forceinline__ Walk(const DenseParams &P, int pair_, int pairs_)
      : pair(pair_), pairs(pairs_), first(P.first), rest(P.rest) {
    const int over = first % pairs;  // pairs below `over` take one long unit more
    mine = first / pairs + (pair < over);
    light = over && pair >= over ? pair - over : -1;
    extra = over ? P.extra : 0;
    gap = over ? pairs - over : 0;
  }
  int gap;  // pairs with one long unit less
  __device__ __forceinline__ int unit(int n) const {
    if (n < mine) return pair + n * pairs;
    int k = n - mine;
    if (light >= 0) {
      if (k < extra) {
        const int u = light + gap * k;
        return u < rest ? first + u : -1;
      }
      k -= extra;
    }
    const int u = gap * extra + pair + pairs * k;
    return u < rest ? first + u : -1;
  }
};
struct Unit {
  const DenseProblem *p;  // for its tensor maps; what loops read is copied (it lies in the
  TilePos pos;            // kernel's parameters, and an indexed read of those is slow)
  int part, k_lo, k_hi;
  int M, N, nk0, a_mn, b_mn, out32, relu, split;
  void *out;
  int64_t ldo;
  float *parts;
};
__device__ __forceinline__ Unit unit_at(const DenseParams &P, int u) {
  int i = 0, units = P.p[0].tiles_m * P.p[0].tiles_n * P.p[0].split;
  while (u >= units) {
    u -= units;
    ++i;
    units = P.p[i].tiles_m * P.p[i].tiles_n * P.p[i].split;
  }
  Unit r;
  r.p = &P.p[i];
  r.part = 0;
  r.k_lo = 0;
  r.k_hi = r.p->nk;
  int tile = u;
  if (r.p->split > 1) {  // (at most 16 parts of K: 32 bits hold the products)
    tile = u / r.p->split;
    r.part = u - tile * r.p->split;
    r.k_lo = (int)((uint32_t)r.part * (uint32_t)r.p->nk / (uint32_t)r.p->split);
    r.k_hi = (int)((uint32_t)(r.part + 1) * (uint32_t)r.p->nk / (uint32_t)r.p->split);
  }
  r.pos = tile_pos(tile, r.p->tiles_m, r.p->tiles_n);
  r.M = r.p->M;
  r.N = r.p->N;
  r.nk0 = r.p->nk0;
  r.a_mn = r.p->a_mn;
  r.b_mn = r.p->b_mn;
  r.out32 = r.p->out32;
  r.relu = r.p->relu;
  r.split = r.p->split;
  r.out = r.p->out;
  r.ldo = r.p->ldo;
  r.parts = r.p->part;
  return r;
}

// 32 values as 16-bit elements to p (16-byte aligned); `cols` of them exist (multiple of 8).
__device__ __forceinline__ void store32(void *p, const float v[32], int cols, bool bf16) {
  uint4 *q = reinterpret_cast<uint4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 8 < cols) {
      uint4 w;
      w.x = pack16(v[8 * i], v[8 * i + 1], bf16);
      w.y = pack16(v[8 * i + 2], v[8 * i + 3], bf16);
      w.z = pack16(v[8 * i + 4], v[8 * i + 5], bf16);
      w.w = pack16(v[8 * i + 6], v[8 * i + 7], bf16);
      q[i] = w;
    }
}
// relu(G) as 16-bit elements: a positive value that rounds to zero keeps the type's
// smallest positive value, so that the stored value's sign is the ReLU's mask.
__device__ __forceinline__ uint32_t pack16_relu(float a, float b, bool bf16) {
  uint32_t w = pack16(a, b, bf16);
  if (a > 0.f && (w & 0xffffu) == 0) w |= 1u;
  if (b > 0.f && (w >> 16) == 0) w |= 0x10000u;
  return w;
}
__device__ __forceinline__ void store32_relu(void *p, const float v[32], int cols, bool bf16) {
  uint4 *q = reinterpret_cast<uint4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 8 < cols) {
      uint4 w;
      w.x = pack16_relu(v[8 * i], v[8 * i + 1], bf16);
      w.y = pack16_relu(v[8 * i + 2], v[8 * i + 3], bf16);
      w.z = pack16_relu(v[8 * i + 4], v[8 * i + 5], bf16);
      w.w = pack16_relu(v[8 * i + 6], v[8 * i + 7], bf16);
      q[i] = w;
    }
}
__device__ __forceinline__ void load32(const void *p, float v[32], int cols, bool bf16) {
  const uint4 *q = reinterpret_cast<const uint4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (i * 8 < cols) w = __ldg(q + i);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16(a[j], bf16);
      v[8 * i + 2 * j] = f.x;
      v[8 * i + 2 * j + 1] = f.y;
    }
  }
}

// ---------------------------------------------------------------- epilogues
// Each thread owns one row of the tile (its tensor-memory lane) and a half of the tile's
// columns.  `row` < M on entry.

__device__ __forceinline__ void epi_store(const DenseParams &P, const Unit &Q, uint32_t taddr, int64_t row, bool live,
                                          int n0) {
  const bool bf16 = P.bf16, parts = Q.split > 1;
  const int64_t ld = parts ? Q.N : Q.ldo;
  float *f32 = parts ? Q.parts + ((int64_t)Q.part * Q.M + row) * ld : static_cast<float *>(Q.out) + row * ld;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    uint32_t raw[32];
    __syncwarp();
    tm_ld32(taddr + c, raw);
    tm_wait_ld();
    // relu: the hidden layer, whose rows are padded to 8 columns
    const int cols = (Q.relu ? (Q.N + 7) / 8 * 8 : Q.N) - (n0 + c);
    if (!live || cols <= 0) continue;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i] = __uint_as_float(raw[i]);
      if (Q.relu) {
        if (P.bias && n0 + c + i < Q.N) v[i] += load16(P.bias, n0 + c + i, bf16);
        v[i] = v[i] < 0.f ? 0.f : v[i];
      }
    }
    if (Q.out32 || parts) {
      float *o = f32 + n0 + c;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * 4 < cols) reinterpret_cast<float4 *>(o)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
      store32(static_cast<uint16_t *>(Q.out) + row * ld + n0 + c, v, cols, bf16);
    }
  }
}

// The pair's tile holds 128 neurons: gate columns 0..127, up columns 128..255.  This
// thread takes 64 of them from n0 on (one act8 block).
__device__ __forceinline__ void epi_gated(const DenseParams &P, const Unit &Q, uint32_t tgate, int64_t row,
                                          bool live, int n0) {
  const bool bf16 = P.bf16;
  const int cols64 = (int)min((int64_t)64, Q.ldo - n0);  // writable columns of H (a multiple of 8)
  float r[64], u[64];
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    uint32_t a[32], b[32];
    tm_ld32(tgate + c, a);
    tm_ld32(tgate + 128 + c, b);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float g = __uint_as_float(a[i]);
      if (P.bias) {
        const int col = n0 + c + i;
        g += col < Q.N ? load16(P.bias, col, bf16) : 0.f;
      }
      r[c + i] = g < 0.f ? 0.f : g;  // NaN stays NaN
      u[c + i] = __uint_as_float(b[i]);
    }
  }
  if (!live || cols64 <= 0) return;
  if (P.save == SFNN_SAVE_FULL) {
    uint16_t *rp = static_cast<uint16_t *>(P.r) + row * P.ldr + n0, *up = static_cast<uint16_t *>(P.u) + row * P.ldr + n0;
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
      store32_relu(rp + c, r + c, cols64 - c, bf16);
      store32(up + c, u + c, cols64 - c, bf16);
    }
  } else if (P.save == SFNN_SAVE_ACT8) {
    uint32_t rt = 0, ut = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      rt = max(rt, __float_as_uint(r[i]) & 0x7fffffffu);
      ut = max(ut, __float_as_uint(u[i]) & 0x7fffffffu);
    }
    const Act8Scale sr = act8_scale(rt, 255.f), su = act8_scale(ut, 127.f);
    P.rs[row * P.lds + (n0 >> 6)] = sr.scale;
    P.us[row * P.lds + (n0 >> 6)] = su.scale;
    uint4 *rp = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(P.r) + row * P.ldr + n0);
    uint4 *up = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(P.u) + row * P.ldr + n0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // whole blocks: code rows are padded to 64 columns
      uint32_t wr[4], wu[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float *a = r + 16 * i + 4 * j, *c = u + 16 * i + 4 * j;
        uint32_t pos = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) pos |= a[k] > 0.f ? 1u << (8 * k) : 0u;
        wr[j] = act8_lift(act8_codes(a[0], a[1], a[2], a[3], sr.inv), pos);
        wu[j] = act8_codes(c[0], c[1], c[2], c[3], su.inv);
      }
      rp[i] = make_uint4(wr[0], wr[1], wr[2], wr[3]);
      up[i] = make_uint4(wu[0], wu[1], wu[2], wu[3]);
    }
  }
  uint16_t *hp = static_cast<uint16_t *>(Q.out) + row * Q.ldo + n0;
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) r[c + i] *= u[c + i];
    store32(hp + c, r + c, cols64 - c, bf16);
  }
}

// Sums of 32 columns over a warp's 32 rows: lane i gets column i's.
__device__ __forceinline__ float column_sums(float v[32], int lane) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const bool hi = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = hi ? v[i] : v[i + o], keep = hi ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

// 128 columns of dH from n0 on; reads the saved relu(G) and U of this row, writes dG, dU, H.
__device__ __forceinline__ void epi_dgated(const DenseParams &P, const Unit &Q, uint32_t taddr, int64_t row,
                                           bool live, int n0) {
  const bool bf16 = P.bf16;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    uint32_t raw[32];
    const int cols = Q.N - (n0 + c);
    const bool on = live && cols > 0;
    float r[32], u[32];
    if (on) {
      if (P.save == SFNN_SAVE_FULL) {
        load32(static_cast<const uint16_t *>(P.r) + row * P.ldr + n0 + c, r, cols, bf16);
        load32(static_cast<const uint16_t *>(P.u) + row * P.ldr + n0 + c, u, cols, bf16);
      } else {
        const float sr = __ldg(P.rs + row * P.lds + ((n0 + c) >> 6)), su = __ldg(P.us + row * P.lds + ((n0 + c) >> 6));
        const uint4 *rp = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(P.r) + row * P.ldr + n0 + c);
        const uint4 *up = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(P.u) + row * P.ldr + n0 + c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 wr = __ldg(rp + i), wu = __ldg(up + i);
          const uint32_t ar[4] = {wr.x, wr.y, wr.z, wr.w}, au[4] = {wu.x, wu.y, wu.z, wu.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t code = (ar[j] >> (8 * k)) & 0xffu;
              // a code above zero keeps its neuron on even where its scale is zero
              const float v = (float)code * sr;
              r[16 * i + 4 * j + k] = code && v == 0.f ? __uint_as_float(1u) : v;
              u[16 * i + 4 * j + k] = (float)(int8_t)((au[j] >> (8 * k)) & 0xffu) * su;
            }
        }
      }
    }
    __syncwarp();
    tm_ld32(taddr + c, raw);
    tm_wait_ld();
    float dg[32], du[32];
    if (on) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float dh = __uint_as_float(raw[i]);
        du[i] = dh * r[i];
        dg[i] = r[i] > 0.f ? dh * u[i] : 0.f;
        r[i] *= u[i];
      }
      const int64_t at = row * Q.ldo + n0 + c;
      store32(static_cast<uint16_t *>(P.dg) + at, dg, cols, bf16);
      store32(static_cast<uint16_t *>(P.du) + at, du, cols, bf16);
      store32(static_cast<uint16_t *>(Q.out) + at, r, cols, bf16);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) dg[i] = 0.f;
    }
    if (P.colpart) {
      __syncwarp();
      const float sum = column_sums(dg, lane);
      const int64_t block = (row - lane) >> 5;
      if (block * 32 < Q.M && lane < cols) P.colpart[block * Q.N + n0 + c + lane] = sum;
    }
  }
}

// ---------------------------------------------------------------- the kernel
template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_dense(const __grid_constant__ DenseParams P) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  const uint32_t stage0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const Walk walk(P, pair, pairs);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&acc_full[i], 1);
      bar_init(&acc_empty[i], 16);  // 8 epilogue warps of each CTA
    }
    bar_init_fence();
  }
  if (warp == 1) tm_alloc<2>(&tmem_slot, kTmem);
  tm_fence_before();
  __syncthreads();
  cluster_sync_all();
  tm_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      int id = walk.unit(0);
      Unit w{}, next = unit_at(P, max(id, 0));
      for (int n = 0; ok && id >= 0; ++n) {
        w = next;
        const CUtensorMap *a0 = &w.p->a0, *b0 = &w.p->b0, *a1 = &w.p->a1, *b1 = &w.p->b1;
        const int m0 = w.pos.m * kTile + (int)rank * 128;
        // gated: the first CTA loads 128 gate rows, the second the same 128 up rows
        const int n0 = EPI == kEpiGated ? w.pos.n * 128 : w.pos.n * kTile + (int)rank * 128;
        for (int kc = w.k_lo; kc < w.k_hi; ++kc, ++it) {
          if (kc == w.k_lo + 1 || w.k_hi == w.k_lo + 1) {  // the next unit, while this one's loads are under way
            id = walk.unit(n + 1);
            next = unit_at(P, max(id, 0));
          }
          const int s = it % kStages;
          if (!bar_wait(&empty[s], (uint32_t)((it / kStages) & 1) ^ 1u)) {
            ok = false;
            break;
          }
          if (rank == 0) bar_expect_tx(&full[s], 2 * kStageBytes);
          const uint32_t bar = cluster_addr(&full[s], 0);
          const uint32_t sa = stage0 + (uint32_t)s * kStageBytes, sb = sa + 16384u;
          const bool second = kc >= w.nk0;
          const int k0 = (second ? kc - w.nk0 : kc) * 64;
          const CUtensorMap *ma = second ? a1 : a0;
          const CUtensorMap *mb = (EPI == kEpiGated ? rank != 0 : second) ? b1 : b0;
          if (EPI == kEpiStore && w.a_mn) {
            tma_load_2d_pair(sa, ma, m0, k0, bar);
            tma_load_2d_pair(sa + 8192u, ma, m0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(sa, ma, k0, m0, bar);
          }
          if (EPI == kEpiDGated || (EPI == kEpiStore && w.b_mn)) {
            tma_load_2d_pair(sb, mb, n0, k0, bar);
            tma_load_2d_pair(sb + 8192u, mb, n0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(sb, mb, k0, n0, bar);
          }
        }
      }
      if (!ok) latch_error(P.err, kErrTimeout);
      // the last stages' release signals arrive in this CTA's shared memory: wait for them
      for (int s = 0; s < kStages && ok; ++s) {
        const int j = it - kStages + s;
        if (j >= 0 && !bar_wait(&empty[j % kStages], (uint32_t)((j / kStages) & 1))) {
          ok = false;
          latch_error(P.err, kErrTimeout);
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      int it = 0;
      bool ok = true;
      int id = walk.unit(0);
      Unit w{}, next = unit_at(P, max(id, 0));
      for (int n = 0; ok && id >= 0; ++n) {
        w = next;
        const int a_mn = EPI == kEpiStore ? w.a_mn : 0, b_mn = EPI == kEpiStore ? w.b_mn : EPI == kEpiDGated;
        const uint32_t idesc = mma_desc_16(256, 256, P.bf16, a_mn, b_mn);
        // a 16-deep step of an operand: 2 KB of an MN-major tile, 32 bytes of a K-major one
        const uint32_t step_a = a_mn ? 2048u : 32u, step_b = b_mn ? 2048u : 32u;
        const uint32_t lbo_a = a_mn ? 8192u : 16u, lbo_b = b_mn ? 8192u : 16u;
        const int buf = n & 1;
        if (!bar_wait(&acc_empty[buf], (uint32_t)((n >> 1) & 1) ^ 1u)) {
          ok = false;
          break;
        }
        tm_fence_after();
        const uint32_t d = tmem + (uint32_t)buf * 256u;
        for (int kc = w.k_lo; kc < w.k_hi; ++kc, ++it) {
          if (kc == w.k_lo + 1 || w.k_hi == w.k_lo + 1) {  // the next unit, while this one's MMAs run
            id = walk.unit(n + 1);
            next = unit_at(P, max(id, 0));
          }
          const int s = it % kStages;
          if (!bar_wait(&full[s], (uint32_t)((it / kStages) & 1))) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t sa = stage0 + (uint32_t)s * kStageBytes, sb = sa + 16384u;
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            mma_16<2>(d, mat_desc(sa + k * step_a, lbo_a, 1024), mat_desc(sb + k * step_b, lbo_b, 1024), idesc,
                      (kc > w.k_lo || k > 0) ? 1u : 0u);
          mma_commit_pair(&empty[s]);
        }
        if (ok) mma_commit_pair(&acc_full[buf]);
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    if (EPI == kEpiStore && P.colsum) {  // while the first tile is multiplied: db from its 32-row sums
      for (int c = blockIdx.x * 256 + threadIdx.x - 64; c < P.cols; c += gridDim.x * 256) {
        float sum = 0.f;
#pragma unroll 8
        for (int b = 0; b < P.col_blocks; ++b) sum += __ldg(P.colpart + (int64_t)b * P.cols + c);
        P.colsum[c] = (uint16_t)pack16(sum, 0.f, P.bf16);
      }
    }
    __syncwarp();
    for (int n = 0, id; (id = walk.unit(n)) >= 0; ++n) {
      const Unit w = unit_at(P, id);
      const int buf = n & 1;
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full[buf], (uint32_t)((n >> 1) & 1)))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        break;
      }
      __syncwarp();
      tm_fence_after();
      const int64_t row = (int64_t)w.pos.m * kTile + rank * 128 + quad * 32 + lane;
      const bool live = row < w.M;
      const uint32_t acc = tmem + lanes + (uint32_t)buf * 256u;
      if (EPI == kEpiGated)
        epi_gated(P, w, acc + half * 64, row, live, w.pos.n * 128 + half * 64);
      else if (EPI == kEpiDGated)
        epi_dgated(P, w, acc + half * 128, row, live, w.pos.n * kTile + half * 128);
      else
        epi_store(P, w, acc + half * 128, row, live, w.pos.n * kTile + half * 128);
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(cluster_addr(&acc_empty[buf], 0));
    }
  }
  __syncwarp();
  tm_fence_before();
  __syncthreads();
  cluster_sync_all();
  tm_fence_after();
  if (warp == 1) tm_dealloc<2>(tmem, kTmem);
}

constexpr size_t kSmem = (size_t)kStages * kStageBytes + 1024;

template <int EPI>
cudaError_t run(const DenseParams &P, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose kernel attribute is set
  const cudaError_t attr = allow_smem(k_dense<EPI>, kSmem, ready);
  if (attr != cudaSuccess) return attr;
  const int grid = 2 * std::min(num_sms / 2, P.first + P.rest);
  return launch_pdl(k_dense<EPI>, dim3(grid), dim3(kThreads), kSmem, s, P);
}

}  // namespace

cudaError_t launch_dense(DenseParams &P, int epi, int num_sms, cudaStream_t s) {
  auto units = [&](int i) { return P.p[i].tiles_m * P.p[i].tiles_n * P.p[i].split; };
  P.first = units(0);
  P.rest = 0;
  int len = 1;
  for (int i = 1; i < P.count; ++i) {
    P.rest += units(i);
    len = std::max(len, P.p[i].nk / P.p[i].split);
  }
  P.extra = P.count > 1 ? (P.p[0].nk / P.p[0].split + len / 2) / len : 0;
  if (epi == kEpiGated) return run<kEpiGated>(P, num_sms, s);
  if (epi == kEpiDGated) return run<kEpiDGated>(P, num_sms, s);
  return run<kEpiStore>(P, num_sms, s);
}

}  // namespace sfnn
