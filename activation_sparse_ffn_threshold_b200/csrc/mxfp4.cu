// mxfp4.cu -- microscaled 4-bit values: quantisation, restoring, and the product.
//
// Format.  32 values along K share a power of two 2^e, e = floor(log2 max|v|) - 2 clamped to
// [-127, 127] (so the largest value lies in [4, 8) units), held as a byte e + 127; 255 stands
// for a NaN block (one that holds a NaN or an infinity).  A value is one of 0, .5, 1, 1.5, 2,
// 3, 4, 6 units with a sign, rounded to nearest even and saturating at 6; two a byte, element
// 2k in the low nibble, rows of K / 2 bytes.
//
// The scale bytes are stored as the tensor core's scale memory wants them: 512-byte tiles of
// 128 rows x 4 blocks, byte (r % 32) * 16 + (r / 32) * 4 + block, so a tile goes from global
// memory to shared memory to tensor memory as it lies.  Rows are padded to 256 and K to 256
// with zero bytes (a finite scale, times zero-filled codes).
//
// Product: Y = (Xq 2^ex) . (Wq 2^ew)^T with tcgen05's block-scaled MMA (kind::mxf4, K = 64 an
// instruction, four times the 16-bit rate), fp32 accumulators.  At that rate a 256 x 256 x 256
// step of a CTA pair takes 512 cycles; the six copies of its scales into tensor memory take
// their turn in the same pipe and add about 300 (4096 x 28672 x 8192: 470 us, 337 with the copies
// left out; issuing them a step ahead 499, writing the scales from registers by four warps of
// their own 760, all timed in turn.  511 to 529 us, 3.7 PFLOP/s, for seconds on several cards).
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kBlock = 32;

__host__ __device__ inline int64_t mx_ktiles(int64_t K) { return (K + 255) / 256 * 2; }  // 4-block tiles of a row, even
__host__ __device__ inline int64_t mx_rtiles(int64_t R) { return (R + 255) / 256 * 2; }  // 128-row tiles, even
__device__ __forceinline__ int64_t mx_scale_at(int64_t row, int kb, int64_t kt) {
  return ((row >> 7) * kt + (kb >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (kb & 3);
}
__device__ __forceinline__ float mx_scale_value(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fffffffu : (e == 0u ? 0x00400000u : e << 23));
}
// The scale byte of a block whose largest magnitude has the fp32 pattern `top`.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  return (uint32_t)max((int)(top >> 23) - 2, 0);
}
// v / 2^e for the scale byte (exact: a power of two; in two steps where 2^-e overflows)
__device__ __forceinline__ float mx_unscale(float v, uint32_t byte) {
  if (byte == 255u) return 0.f;
  const int k = 127 - (int)byte;  // v * 2^k, |k| <= 127
  const int a = k >> 1, b = k - a;
  return v * __uint_as_float((uint32_t)(a + 127) << 23) * __uint_as_float((uint32_t)(b + 127) << 23);
}
// Two values (in units) as e2m1 codes: lo in the low nibble.
__device__ __forceinline__ uint32_t mx_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.u32.u8 %0, t;\n}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float mx_value(uint32_t code) {  // a 4-bit code in units
  const uint32_t m = code & 7u;
  const float v = m < 5u ? 0.5f * (float)m : (m == 5u ? 3.f : (m == 6u ? 4.f : 6.f));
  return code & 8u ? -v : v;
}

constexpr int kWarps = 8;
constexpr int kVecs = 8;
constexpr int kChunk = 32 * kVecs * 8;  // columns per warp

// A warp takes 2048 columns of one (padded) row: 8 values a lane at a time, all its loads
// requested first; four lanes hold a block.  Bound by instructions: 11008 x 4096 takes 35 us with 0.77
// of the issue slots in use, its bytes (2 read, 0.53 written a value) 17.5 at the copy rate.
__global__ void __launch_bounds__(kWarps * 32)
    k_mx_quantize(const uint16_t *__restrict__ x, int64_t ldx, int64_t R, int K, int bf16, int vec,
                  uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t kt = mx_ktiles(K);
  if (row >= mx_rtiles(R) * 128) return;
  const int c0 = blockIdx.y * kChunk + lane * 8;
  uint4 w[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = c0 + i * 256;
    w[i] = make_uint4(0, 0, 0, 0);
    if (row < R && c < K) {  // K is a multiple of 32: whole vectors
      const uint16_t *p = x + row * ldx + c;
      if (vec) {
        w[i] = ld_stream(p);
      } else {
        uint32_t a[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j >> 1] |= (uint32_t)__ldg(p + j) << (16 * (j & 1));
        w[i] = make_uint4(a[0], a[1], a[2], a[3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = c0 + i * 256;
    const uint32_t a[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16(a[j], bf16);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (c >= kt * 128) continue;  // past the padded row
    const uint32_t e = mx_scale_byte(top);
    if (row < R && c < K) {
      uint32_t q = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) q |= mx_pair(mx_unscale(v[2 * j], e), mx_unscale(v[2 * j + 1], e)) << (8 * j);
      *reinterpret_cast<uint32_t *>(codes + (row * K + c) / 2) = q;
    }
    if ((lane & 3) == 0) scales[mx_scale_at(row, c >> 5, kt)] = (uint8_t)e;  // padding: top = 0 -> 0
  }
}

__global__ void __launch_bounds__(kWarps * 32)
    k_mx_restore(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t R, int K, int bf16,
                 int vec, uint16_t *__restrict__ out, int64_t ldo) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= R) return;
  const int64_t kt = mx_ktiles(K);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = blockIdx.y * kChunk + lane * 8 + i * 256;
    if (c >= K) continue;
    const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(codes + (row * K + c) / 2));
    const float s = mx_scale_value(__ldg(scales + mx_scale_at(row, c >> 5, kt)));
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pack16(mx_value((q >> (8 * j)) & 15u) * s, mx_value((q >> (8 * j + 4)) & 15u) * s, bf16);
    uint16_t *p = out + row * ldo + c;
    if (vec) {
      *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// ---------------------------------------------------------------- the product
constexpr int kThreads = 320;
constexpr int kMaxStages = 6;
constexpr int kTmem = 512;
constexpr int kAcc = 0, kSf = 256;      // tensor-memory columns: accumulators, scale slots
constexpr int kSfSlot = 32;             // of a stage: A 2 x 4 columns, B 2 x 8 from column 8 on
constexpr uint32_t kPairStage = 16384 + 16384 + 1024 + 2048;  // A, B, their scales (a multiple of 1024)

struct alignas(64) MxParams {
  CUtensorMap a, b, sa, sb;
  int M, N, nk;          // nk: 256-deep steps
  int tiles_m, tiles_n;
  int out_dtype, vec;    // vec: rows of C are 16-byte aligned
  void *out;
  int64_t ldo;
  int32_t *err;
};

// kind::mxf4: e2m1 operands (K-major), ue8m0 scales of 32 values; sf_id picks the two scale
// bytes of a 32-bit word that an instruction's 64 values use.
__device__ __forceinline__ uint32_t mx_idesc(int M, int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
         (sf_id << 29);
}
template <int CG>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t accumulate) {
  if (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// A 512-byte scale tile to 4 tensor-memory columns (32 lanes x 16 bytes, repeated for the four
// lane quarters), in both CTAs of a pair from their own shared memory.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(16u >> 4) << 16) |
                        ((uint64_t)(128u >> 4) << 32) | (1ull << 46);  // no swizzle, 8-row groups 128 bytes apart
  if (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

struct TilePos {
  int m, n;
};
__device__ __forceinline__ TilePos tile_pos(int t, int tiles_m, int tiles_n) {  // bands of 8 tile rows
  constexpr int kBand = 8;
  const int per = kBand * tiles_n;
  const int band = t / per, r = t - band * per;
  const int rows = min(kBand, tiles_m - band * kBand);
  return {band * kBand + r % rows, r / rows};
}

// 64 bytes (of E-byte values) of each of a warp's rows: a lane holds its row's (w), the warp
// stores them through a 2 KB panel of shared memory with 4 lanes of 16 bytes to a row, or,
// where rows do not start on 16 bytes, value by value along the row (a lane storing its own
// row touches 32 lines an instruction: 2508 x 9175 x 480 took 241 us, now 32).  `left`:
// columns that exist from the first on.
constexpr uint32_t kPanel = 2048;
template <int E>
__device__ __forceinline__ void panel_store(uint32_t panel, const uint32_t w[16], unsigned char *base, int64_t ld, int rows,
                                            int left, int vec) {
  const int lane = threadIdx.x & 31;
  constexpr int COLS = 64 / E;
  if (left <= 0) return;  // (the whole warp)
  auto at = [&](int row, int piece) { return panel + (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4)); };
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at(lane, j)), "r"(w[4 * j]), "r"(w[4 * j + 1]),
                 "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                 : "memory");
  __syncwarp();
  if (vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 8 + (lane >> 2), piece = lane & 3;
      uint4 q;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                   : "r"(at(row, piece))
                   : "memory");
      if (row >= rows) continue;
      unsigned char *o = base + row * ld + piece * 16;
      const int have = left - piece * (16 / E);
      if (have >= 16 / E) {
        *reinterpret_cast<uint4 *>(o) = q;
      } else {
        const uint32_t a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 16 / E; ++j)
          if (j < have) {
            if (E == 4)
              reinterpret_cast<uint32_t *>(o)[j] = a[j & 3];
            else
              reinterpret_cast<uint16_t *>(o)[j] = (uint16_t)(a[(j >> 1) & 3] >> (16 * (j & 1)));
          }
      }
    }
  } else {
    // 32 lanes: one row's 32 values, or two rows' 16
    const int c = lane % COLS, cols = min(COLS, left);
#pragma unroll 8
    for (int r = 0; r < 32; r += 32 / COLS) {
      const int row = r + lane / COLS;
      const uint32_t p = at(row, c * E >> 4) + (uint32_t)(c * E & 15);
      unsigned char *o = base + row * ld;
      if (E == 4) {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
        if (row < rows && c < cols) reinterpret_cast<uint32_t *>(o)[c] = v;
      } else {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p) : "memory");
        if (row < rows && c < cols) reinterpret_cast<uint16_t *>(o)[c] = v;
      }
    }
  }
}

// 256 x 256 tiles by CTA pairs, 128 rows of X and of W in each CTA (more tokens: few_serves).
//
// The accumulators are single (256 columns; the scales need the rest of tensor memory): the
// epilogue warps copy a finished tile to registers, hand the columns back, and store while
// the next tile's MMAs run.  Scale slots go by stage: a slot is written again only after the
// stage's MMAs have completed.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_mx(const __grid_constant__ MxParams P) {
  extern __shared__ unsigned char smem_raw[];
  // stages, panels, barriers: all of the SM's shared memory, so none is spent on alignment --
  // dynamic shared memory alone starts on 1024 bytes (checked: the swizzle needs it)
  const uint32_t stage0 = smem_u32(smem_raw);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw + kMaxStages * kPairStage + 8 * kPanel);
  uint64_t *full = bars, *empty = bars + kMaxStages;
  uint64_t &acc_full = bars[2 * kMaxStages], &acc_empty = bars[2 * kMaxStages + 1];
  uint32_t &tmem_slot = *reinterpret_cast<uint32_t *>(&bars[2 * kMaxStages + 2]);
  if (stage0 & 1023u) {
    if (threadIdx.x == 0) latch_error(P.err, SFNN_ERR_UNSUPPORTED);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  const int ntiles = P.tiles_m * P.tiles_n;
  constexpr uint32_t b_bytes = 16384u, stage_bytes = kPairStage;
  constexpr int stages = kMaxStages, nsf = 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    bar_init(&acc_full, 1);
    bar_init(&acc_empty, 16);
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
      for (int t = unit; t < ntiles && ok; t += units) {
        const TilePos pos = tile_pos(t, P.tiles_m, P.tiles_n);
        const int m0 = pos.m * 256 + (int)rank * 128;
        const int n0 = pos.n * 256, nb0 = n0 + (int)rank * 128;  // the tile's columns, this CTA's rows of W
        const int rb = n0 >> 7;                                  // first scale tile row of W
        for (int kc = 0; kc < P.nk; ++kc, ++it) {
          const int s = it % stages;
          if (!bar_wait(&empty[s], (uint32_t)((it / stages) & 1) ^ 1u)) {
            ok = false;
            break;
          }
          constexpr uint32_t bytes = 16384u + b_bytes + 1024u + nsf * 1024u;
          if (rank == 0) bar_expect_tx(&full[s], 2 * bytes);
          const uint32_t a = stage0 + (uint32_t)s * stage_bytes, b = a + 16384u, sa = b + b_bytes, sb = sa + 1024u;
          const uint32_t bar = cluster_addr(&full[s], 0);
          tma_load_2d_pair(a, &P.a, kc * 128, m0, bar);
          tma_load_2d_pair(b, &P.b, kc * 128, nb0, bar);
          tma_load_2d_pair(sa, &P.sa, 0, (m0 >> 7) * P.nk + kc, bar);
          for (int r = 0; r < nsf; ++r) tma_load_2d_pair(sb + r * 1024u, &P.sb, 0, (rb + r) * P.nk + kc, bar);
        }
      }
      if (!ok) latch_error(P.err, kErrTimeout);
      for (int s = 0; s < stages && ok; ++s) {  // the last releases arrive here: wait for them
        const int j = it - stages + s;
        if (j >= 0 && !bar_wait(&empty[j % stages], (uint32_t)((j / stages) & 1))) {
          ok = false;
          latch_error(P.err, kErrTimeout);
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      int it = 0, i = 0;
      bool ok = true;
      const uint32_t id0 = mx_idesc(256, 256, 0), id2 = mx_idesc(256, 256, 2);
      for (int t = unit; t < ntiles && ok; t += units, ++i) {
        if (!bar_wait(&acc_empty, (uint32_t)(i & 1) ^ 1u)) {
          ok = false;
          break;
        }
        tm_fence_after();
        for (int kc = 0; kc < P.nk; ++kc, ++it) {
          const int s = it % stages;
          if (!bar_wait(&full[s], (uint32_t)((it / stages) & 1))) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t a = stage0 + (uint32_t)s * stage_bytes, b = a + 16384u, sa = b + b_bytes, sb = sa + 1024u;
          const uint32_t ta = tmem + kSf + (uint32_t)(s * kSfSlot), tb = ta + 8u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the step's two 128-deep scale tiles
            copy_scales<2>(ta + h * 4, sa + h * 512);
            for (int r = 0; r < nsf; ++r) copy_scales<2>(tb + h * 8 + r * 4, sb + r * 1024 + h * 512);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_mx<2>(tmem + kAcc, mat_desc(a + k * 32, 16, 1024), mat_desc(b + k * 32, 16, 1024), (k & 1) ? id2 : id0,
                      ta + (k >> 1) * 4, tb + (k >> 1) * 8, (kc > 0 || k > 0) ? 1u : 0u);
          mma_commit_pair(&empty[s]);
        }
        if (ok) mma_commit_pair(&acc_full);
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t panel = stage0 + stages * stage_bytes + (uint32_t)(warp - 2) * kPanel;
    int i = 0;
    for (int t = unit; t < ntiles; t += units, ++i) {
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full, (uint32_t)(i & 1)))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        break;
      }
      __syncwarp();
      tm_fence_after();
      const TilePos pos = tile_pos(t, P.tiles_m, P.tiles_n);
      const int64_t row = (int64_t)pos.m * 256 + rank * 128 + quad * 32 + lane;
      const int64_t row0 = row - lane;
      const int n0 = pos.n * 256 + half * 128;
      uint32_t v[4][32];  // this warp's 128 columns
#pragma unroll
      for (int u = 0; u < 4; ++u)
        tm_ld32(tmem + ((uint32_t)(quad * 32) << 16) + kAcc + half * 128 + u * 32, v[u]);
      tm_wait_ld();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty, 0));
      const int rows = (int)min((int64_t)32, P.M - row0);
      if (rows <= 0 || n0 >= P.N) continue;  // (the whole warp)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = n0 + u * 32;
        if (P.out_dtype == SFNN_F32) {
          unsigned char *o = static_cast<unsigned char *>(P.out) + (row0 * P.ldo + c) * 4;
          panel_store<4>(panel, v[u], o, P.ldo * 4, rows, P.N - c, P.vec);
          panel_store<4>(panel, v[u] + 16, o + 64, P.ldo * 4, rows, P.N - c - 16, P.vec);
        } else {
          const bool bf16 = P.out_dtype == SFNN_BF16;
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) p[j] = pack16(__uint_as_float(v[u][2 * j]), __uint_as_float(v[u][2 * j + 1]), bf16);
          panel_store<2>(panel, p, static_cast<unsigned char *>(P.out) + (row0 * P.ldo + c) * 2, P.ldo * 2, rows, P.N - c,
                         P.vec);
        }
      }
    }
  }
  __syncwarp();
  tm_fence_before();
  __syncthreads();
  cluster_sync_all();
  tm_fence_after();
  if (warp == 1) tm_dealloc<2>(tmem, kTmem);
}

// ---------------------------------------------------------------- one to four tokens
// Y = Xq . Wq^T on CUDA cores with the tokens quantised by every CTA itself: one launch, no
// workspace.  Bound by the weights' bytes (half a byte a value); the products run on bytes,
// exactly: a code is turned into twice its value (0, 1, 2, 3, 4, 6, 8, 12) by byte permutes,
// four products an instruction (dp4a), 32 of them an int32 that the two block scales then
// multiply.  A negative weight's byte is its one's complement; the sum of x over the negative
// weights, which that takes too much, is added back by a second dp4a on the sign bytes.
//
// Measured: 1 token, 11008 x 4096: 10.1 to 10.5 us, 0.63 of the issue slots (the bytes alone: 3.7).
//
// A CTA owns a contiguous share of the rows, a warp takes one row at a time: a lane holds 32
// values (16 bytes) of every 1024, a row's loads go out while the row before is multiplied.
constexpr int kRowThreads = 512;
constexpr int kRowLoads = 4;  // 16-byte loads of a lane in flight for a row: 4096 values

__device__ __forceinline__ uint32_t mx_magnitudes(uint32_t sel) { return __byte_perm(0x03020100u, 0x0c080604u, sel); }
__device__ __forceinline__ uint32_t mx_signs(uint32_t sel) { return __byte_perm(0x0000ff00u, 0u, sel); }

template <int TT>
__global__ void __launch_bounds__(kRowThreads)
    k_mx_rows(const uint16_t *__restrict__ x, int64_t ldx, int T, int vec, int bf16, const uint4 *__restrict__ codes,
              const uint8_t *__restrict__ scales, int N, int K, void *__restrict__ out, int64_t ldo, int out_dtype) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int nb = K / kBlock;
  // bytes of token t: two planes of 16 bytes a block (a warp's 16-byte reads then have no bank
  // conflicts), then its scales
  uint4 *xq = reinterpret_cast<uint4 *>(smem);
  // as two factors, at most 1 and at least 1: with the weights' scale between them no product
  // leaves fp32's range that comes back to it
  float2 *xs = reinterpret_cast<float2 *>(smem + (size_t)TT * K);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = (int)((int64_t)blockIdx.x * N / gridDim.x), r1 = (int)((int64_t)(blockIdx.x + 1) * N / gridDim.x);
  const int64_t kt = mx_ktiles(K);
  pdl_wait();
  pdl_launch_dependents();

  // a lane's block of iteration `it` is it * 32 + lane: its codes lie 512 bytes and its scale
  // byte 8 tiles (4096 bytes) from those of the iteration before
  const int iters = (nb + 31) / 32;
  const uint4 *codes_at = codes + lane;
  const uint8_t *scales_at = scales + (lane >> 2) * 512 + (lane & 3);
  uint4 w[kRowLoads];
  uint32_t sb[kRowLoads];
  auto request = [&](int row, int it) {
    const uint4 *c = codes_at + (int64_t)row * nb + it * 32;
    const uint8_t *e = scales_at + ((int64_t)(row >> 7) * kt + it * 8) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
    const int left = row < r1 ? nb - it * 32 - lane : 0;
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i) {
      w[i] = make_uint4(0, 0, 0, 0);
      sb[i] = 0;
      if (i * 32 < left) {
        w[i] = ld_stream(c + i * 32);
        sb[i] = __ldg(e + i * 4096);
      }
    }
  };
  request(r0 + warp, 0);

  for (int g0 = 0; g0 < TT * nb * 4; g0 += kRowThreads) {  // 8 values a thread; 4 neighbouring lanes a block
    const int g = g0 + threadIdx.x, t = g / (nb * 4), c = (g - t * nb * 4) * 8;
    uint32_t a[4] = {0, 0, 0, 0};
    if (t < T) {
      const uint16_t *p = x + t * ldx + c;
      if (vec) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
        a[0] = q.x, a[1] = q.y, a[2] = q.z, a[3] = q.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j >> 1] |= (uint32_t)__ldg(p + j) << (16 * (j & 1));
      }
    }
    uint32_t top = 0;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16(a[j], bf16);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
      top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (t >= TT) continue;
    const uint32_t e = mx_scale_byte(top);
    uint32_t q = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) q |= mx_pair(mx_unscale(v[2 * j], e), mx_unscale(v[2 * j + 1], e)) << (8 * j);
    const uint32_t sel = q & 0x77777777u, neg = (q >> 3) & 0x11111111u;
    const uint32_t s0 = mx_signs(neg), s1 = mx_signs(neg >> 16);
    const uint32_t lo = __vsub4(mx_magnitudes(sel) ^ s0, s0), hi = __vsub4(mx_magnitudes(sel >> 16) ^ s1, s1);
    const int b = c >> 5, part = (c >> 3) & 3;  // 8 values: half a plane's 16 bytes
    reinterpret_cast<uint2 *>(xq + ((size_t)t * 2 + (part >> 1)) * nb + b)[part & 1] = make_uint2(lo, hi);
    if (part == 0) {
      const float v = 0.25f * mx_scale_value(e);  // the products are of doubled values
      xs[t * nb + b] = make_float2(v > 1.f ? 1.f : v, v > 1.f ? v : 1.f);
    }
  }
  __syncthreads();

  for (int row = r0 + warp; row < r1; row += kRowThreads / 32) {
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.f;
    for (int it = 0; it < iters; it += kRowLoads) {
      uint4 cw[kRowLoads];
      uint32_t cs[kRowLoads];
#pragma unroll
      for (int i = 0; i < kRowLoads; ++i) {
        cw[i] = w[i];
        cs[i] = sb[i];
      }
      const bool more = it + kRowLoads < iters;
      request(more ? row : row + kRowThreads / 32, more ? it + kRowLoads : 0);
#pragma unroll
      for (int i = 0; i < kRowLoads; ++i) {
        if (it + i >= iters) break;  // (the whole warp)
        const int b = (it + i) * 32 + lane;
        if (b >= nb) continue;
        const uint32_t word[4] = {cw[i].x, cw[i].y, cw[i].z, cw[i].w};
        uint32_t val[8], sgn[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t sel = word[j] & 0x77777777u, neg = (word[j] >> 3) & 0x11111111u;
          sgn[2 * j] = mx_signs(neg);
          sgn[2 * j + 1] = mx_signs(neg >> 16);
          val[2 * j] = mx_magnitudes(sel) ^ sgn[2 * j];
          val[2 * j + 1] = mx_magnitudes(sel >> 16) ^ sgn[2 * j + 1];
        }
        const float ws = mx_scale_value(cs[i]);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint4 p0 = xq[t * 2 * nb + b], p1 = xq[t * 2 * nb + nb + b];
          const uint32_t xv[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
          int dot = 0, over = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dot = __dp4a((int)xv[j], (int)val[j], dot);
            over = __dp4a((int)xv[j], (int)sgn[j], over);
          }
          const float2 sx = xs[t * nb + b];
          acc[t] = fmaf((float)(dot - over) * sx.x * ws, sx.y, acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float s = warp_sum(acc[t]);
      if (lane == 0 && t < T) {
        if (out_dtype == SFNN_F32)
          static_cast<float *>(out)[t * ldo + row] = s;
        else
          static_cast<uint16_t *>(out)[t * ldo + row] = (uint16_t)pack16(s, 0.f, out_dtype == SFNN_BF16);
      }
    }
  }
}

bool rows_serve(int T, int K) { return T <= 4 && (int64_t)T * K <= 65536; }

template <int TT>
cudaError_t launch_rows(const void *x, int64_t ldx, int T, int vec, int bf16, const void *wc, const void *wsc, int N, int K,
                        void *y, int64_t ldy, int y_dtype, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t attr = allow_smem(k_mx_rows<TT>, (size_t)(TT == 4 ? 65536 / 3 * 4 : 65536) * 5 / 4 + 256, ready);
  if (attr != cudaSuccess) return attr;
  return launch_pdl(k_mx_rows<TT>, dim3(std::min(sms, (N + 15) / 16)), dim3(kRowThreads), (size_t)TT * K * 5 / 4, s,
                    static_cast<const uint16_t *>(x), ldx, T, vec, bf16, static_cast<const uint4 *>(wc),
                    static_cast<const uint8_t *>(wsc), N, K, y, ldy, y_dtype);
}

// ---------------------------------------------------------------- few tokens
// The weights on the MMA's M side (128-row tiles, as their scales lie), up to 128 tokens on its
// N side (blockIdx.y: which 128).  Bound by the weights' bytes and, in small layers, by latency: a cluster of 2 or 4
// CTAs splits a tile's K so that the SMs are filled, each CTA then adds up a share of the
// tokens: its own accumulators and, in rank order, those the other CTAs put into its shared
// memory.
constexpr int kFewThreads = 192;  // warp 0 loads, warp 1 issues the MMAs, warps 2-5 take 32 weight rows each
constexpr int kFewTokens = 128;  // of a CTA: the rows that a tile of their scales holds
constexpr int kFewStages = 8;
constexpr int kFewSf = 16;  // scale columns of a stage: A 2 x 4, B 2 x 4 (128 tokens)

struct alignas(64) FewParams {
  CUtensorMap w, x, sw, sx;
  int T, N, nk;   // nk: 256-deep steps
  int tiles;
  int t8, t16;    // T rounded up to 8 (rows loaded), to 16 (MMA N)
  int stages, split, share;  // share: tokens that a CTA of a cluster adds up
  int apart;                 // the parts land behind the stages (else in them)
  int acc_cols, tmem_cols;   // columns of the accumulators (then the scales), of all
  int out_dtype;
  void *out;
  int64_t ldo;
  int32_t *err;
};

__global__ void __launch_bounds__(kFewThreads) k_mx_few(const __grid_constant__ FewParams P) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kFewStages], empty[kFewStages], acc_full, acc_empty, parts_in;
  __shared__ uint32_t tmem_slot;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t stage0 = (raw + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = P.split, part = split > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / split, units = gridDim.x / split;
  const int group = blockIdx.y, T = min(P.T - group * kFewTokens, kFewTokens);  // this CTA's tokens
  const uint32_t x_bytes = (uint32_t)P.t8 * 128u;
  // w (16 KB), its scales, x, its scales; an MMA may read 1 KB past x's rows, into the scales
  const uint32_t stage_bytes = 16384u + 1024u + x_bytes + 1024u;
  const int stages = P.stages;
  const int k_lo = (int)((int64_t)part * P.nk / split), steps = (int)((int64_t)(part + 1) * P.nk / split) - k_lo;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    bar_init(&acc_full, 1);
    bar_init(&acc_empty, 4);
    bar_init(&parts_in, 4u * (uint32_t)(split > 1 ? split - 1 : 1));
    bar_init_fence();
  }
  if (split > 1) cluster_sync_all();  // every CTA's barrier is there before a part arrives
  if (warp == 1) tm_alloc<1>(&tmem_slot, (uint32_t)P.tmem_cols);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      pdl_wait();
      pdl_launch_dependents();
      const uint32_t bytes = 16384u + 1024u + x_bytes + 1024u;
      int it = 0;
      bool ok = true;
      for (int t = unit; t < P.tiles && ok; t += units) {
        for (int i = 0; i < steps; ++i, ++it) {
          const int s = it % stages, k = k_lo + i;
          if (!bar_wait(&empty[s], (uint32_t)((it / stages) & 1) ^ 1u)) {
            ok = false;
            break;
          }
          bar_expect_tx(&full[s], bytes);
          const uint32_t w = stage0 + (uint32_t)s * stage_bytes, x = w + 16384u, sw = x + x_bytes, sx = sw + 1024u;
          tma_load_2d(w, &P.w, k * 128, t * 128, &full[s]);
          tma_load_2d(sw, &P.sw, 0, t * P.nk + k, &full[s]);
          tma_load_2d(x, &P.x, k * 128, group * kFewTokens, &full[s]);
          tma_load_2d(sx, &P.sx, 0, group * P.nk + k, &full[s]);
        }
      }
      for (int s = 0; s < stages && ok; ++s) {  // every load has been consumed before the CTA ends
        const int j = it - stages + s;
        if (j >= 0 && !bar_wait(&empty[j % stages], (uint32_t)((j / stages) & 1))) ok = false;
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id0 = mx_idesc(128, P.t16, 0), id2 = mx_idesc(128, P.t16, 2);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = unit; t < P.tiles && ok; t += units, ++n) {
        if (!bar_wait(&acc_empty, (uint32_t)(n & 1) ^ 1u)) {
          ok = false;
          break;
        }
        tm_fence_after();
        for (int i = 0; i < steps; ++i, ++it) {
          const int s = it % stages;
          if (!bar_wait(&full[s], (uint32_t)((it / stages) & 1))) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t w = stage0 + (uint32_t)s * stage_bytes, x = w + 16384u, sw = x + x_bytes, sx = sw + 1024u;
          const uint32_t ta = tmem + (uint32_t)(P.acc_cols + s * kFewSf), tb = ta + 8u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            copy_scales<1>(ta + h * 4, sw + h * 512);
            copy_scales<1>(tb + h * 4, sx + h * 512);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_mx<1>(tmem, mat_desc(w + k * 32, 16, 1024), mat_desc(x + k * 32, 16, 1024), (k & 1) ? id2 : id0,
                      ta + (k >> 1) * 4, tb + (k >> 1) * 4, (i > 0 || k > 0) ? 1u : 0u);
          mma_commit(&empty[s]);
        }
        if (ok) mma_commit(&acc_full);
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  }
  const int quad = warp & 3, row = quad * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  const bool worker = warp >= 2;
  // this thread's weight row for tokens [t0, t1): out[t][col], with the other CTAs' parts
  // (four tokens of a row side by side, then the next row: 16-byte accesses without conflicts)
  auto finish = [&](int tile, int t0, int t1, const unsigned char *sums) {
    const int col = tile * 128 + row;
    for (int c = t0; c < t1; c += 16) {
      uint32_t g[16];
      float v[16];
      __syncwarp();
      tm_ld16(lanes + c, g);
      tm_wait_ld();
      if (col >= P.N) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = sums && part > 0 ? 0.f : __uint_as_float(g[i]);
      if (sums)
        for (int p = part > 0 ? 0 : 1; p < split; ++p) {  // rank order, this CTA's own in its place
          if (p == part) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(g[i]);
          } else {
            const unsigned char *a = sums + ((size_t)(p < part ? p : p - 1) * P.share + (c - t0)) * 512 + row * 16;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + 4 * i < t1) {
                const float4 q = *reinterpret_cast<const float4 *>(a + i * 2048);
                v[4 * i] += q.x, v[4 * i + 1] += q.y, v[4 * i + 2] += q.z, v[4 * i + 3] += q.w;
              }
          }
        }
      if (P.out_dtype == SFNN_F32) {
        float *o = static_cast<float *>(P.out) + (group * kFewTokens + c) * P.ldo + col;
#pragma unroll
        for (int i = 0; i < 16; ++i, o += P.ldo)
          if (c + i < t1) *o = v[i];
      } else {
        const bool bf16 = P.out_dtype == SFNN_BF16;
        uint16_t *o = static_cast<uint16_t *>(P.out) + (group * kFewTokens + c) * P.ldo + col;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const uint32_t w = pack16(v[i], v[i + 1], bf16);
          if (c + i < t1) *o = (uint16_t)w;
          o += P.ldo;
          if (c + i + 1 < t1) *o = (uint16_t)(w >> 16);
          o += P.ldo;
        }
      }
    }
  };
  bool good = true;
  if (worker) {
    pdl_wait();
    int n = 0;
    for (int t = unit; t < P.tiles; t += units, ++n) {
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full, (uint32_t)(n & 1)))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        good = false;
        break;
      }
      __syncwarp();
      tm_fence_after();
      if (split > 1) break;  // one tile per cluster
      finish(t, 0, T, nullptr);
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty, 0));
    }
  }
  __syncwarp();
  if (split > 1) {
    const uint32_t sums = stage0 - raw + (P.apart ? (uint32_t)stages * stage_bytes : 0u);  // the same offset in every CTA
    if (!P.apart) cluster_sync_all();  // no load or MMA touches a stage any more
    tm_fence_after();
    if (worker) {
      for (int k = 1; k < split; ++k) {
        const int q = (part + k) % split;  // each CTA begins with another
        const int t0 = min(T, q * P.share), t1 = min(T, t0 + P.share);
        const uint32_t dst0 = cluster_addr(smem_raw, (uint32_t)q) + sums +
                              (uint32_t)((part < q ? part : part - 1) * P.share * 512 + row * 16);
        for (int c = t0; c < t1; c += 16) {
          uint32_t g[16];
          __syncwarp();
          tm_ld16(lanes + c, g);
          tm_wait_ld();
          const uint32_t dst = dst0 + (uint32_t)(c - t0) * 512u;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + 4 * i < t1)
              asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (uint32_t)i * 2048u), "r"(g[4 * i]),
                           "r"(g[4 * i + 1]), "r"(g[4 * i + 2]), "r"(g[4 * i + 3])
                           : "memory");
        }
        __syncwarp();  // the arrival releases the whole warp's stores
        if (lane == 0) bar_arrive_cluster(cluster_addr(&parts_in, (uint32_t)q));
      }
    }
    __syncwarp();
    cluster_arrive();  // this CTA writes to no other any more
    if (worker) {
      if (!__all_sync(0xffffffffu, bar_wait(&parts_in, 0))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
      } else if (good && unit < P.tiles) {
        __syncwarp();
        const int t0 = min(T, part * P.share);
        finish(unit, t0, min(T, t0 + P.share), smem_raw + sums);
      }
    }
    __syncwarp();
    cluster_wait();  // nor does another write to this one
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == 1) tm_dealloc<1>(tmem, (uint32_t)P.tmem_cols);
}

cudaError_t launch_pair(const MxParams &P, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const size_t smem = (size_t)kMaxStages * kPairStage + 8 * kPanel + (2 * kMaxStages + 3) * 8;
  const cudaError_t attr = allow_smem(k_mx, smem, ready);
  if (attr != cudaSuccess) return attr;
  return launch_pdl(k_mx, dim3(2 * std::min(num_sms / 2, P.tiles_m * P.tiles_n)), dim3(kThreads), smem, s, P);
}

cudaError_t launch_few(FewParams &P, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t attr = allow_smem(k_mx_few, 224 * 1024, ready);
  if (attr != cudaSuccess) return attr;
  const int tokens = std::min(P.T, kFewTokens), groups = (P.T + kFewTokens - 1) / kFewTokens;
  P.t8 = (tokens + 7) / 8 * 8;
  P.t16 = (tokens + 15) / 16 * 16;
  P.tiles = (P.N + 127) / 128;
  P.split = 1;
  // more CTAs to a tile while they fit two to an SM and each keeps two steps
  while (P.split < 4 && P.tiles * groups * P.split * 2 <= 2 * num_sms && P.nk >= 4 * P.split) P.split *= 2;
  P.share = ((tokens + P.split - 1) / P.split + 3) / 4 * 4;
  const int stage = 16384 + 1024 + P.t8 * 128 + 1024;
  const int parts = P.split > 1 ? (P.split - 1) * P.share * 512 : 0;
  P.apart = parts <= 16 * 1024;
  const int steps = (P.nk + P.split - 1) / P.split;
  P.stages = std::min({kFewStages, steps, (108 * 1024 - (P.apart ? parts : 0)) / stage});
  const int stage_mem = P.stages * stage;
  P.acc_cols = (P.t16 + 31) / 32 * 32 + 32;  // read 32 columns at a time, from any token on
  P.tmem_cols = 32;
  while (P.tmem_cols < P.acc_cols + P.stages * kFewSf) P.tmem_cols *= 2;
  // The SM's share of shared memory that goes with the share of tensor memory (456 bytes a
  // column, less what the launch adds): CTAs that could not all allocate never share an SM,
  // or one would wait for columns held by a cluster that waits for it.
  const size_t smem = std::max<size_t>(1024 + (P.apart ? stage_mem + parts : std::max(stage_mem, parts)),
                                       P.tmem_cols * 456 - 2048);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.split > 1 ? P.tiles * P.split : std::min(P.tiles, std::max(1, 2 * num_sms / groups)), groups);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = (unsigned)P.split;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = P.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_mx_few, P);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sfnn_status mx_check(int64_t R, int32_t K, const void *codes, const void *scales) {
  if (R < 0 || K < 1) return SFNN_ERR_INVALID_ARG;
  if (K % kBlock || K > (1 << 20) || R > (1 << 24)) return SFNN_ERR_UNSUPPORTED;
  if (R > 0 && (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16))) return SFNN_ERR_INVALID_ARG;
  return SFNN_OK;
}
sfnn_status value_check(const void *p, int64_t ld, int64_t R, int64_t cols, int32_t dtype, bool f32_too) {
  if (dtype != SFNN_F16 && dtype != SFNN_BF16 && !(f32_too && dtype == SFNN_F32)) return SFNN_ERR_INVALID_ARG;
  if (ld < cols) return SFNN_ERR_INVALID_ARG;
  if (R > 0 && (!p || !aligned(p, dtype == SFNN_F32 ? 4 : 2))) return SFNN_ERR_INVALID_ARG;
  return SFNN_OK;
}
bool rows16(const void *p, int64_t ld, int esize) { return aligned(p, 16) && ld * esize % 16 == 0; }

cudaError_t quantize(const void *x, int64_t ldx, int64_t R, int K, int32_t dtype, void *codes, void *scales,
                     cudaStream_t s) {
  const dim3 grid((unsigned)(mx_rtiles(R) * 128 / kWarps), (unsigned)((mx_ktiles(K) * 128 + kChunk - 1) / kChunk));
  return launch_pdl(k_mx_quantize, grid, dim3(kWarps * 32), 0, s, static_cast<const uint16_t *>(x), ldx, R, K,
                    (int)(dtype == SFNN_BF16), (int)rows16(x, ldx, 2), static_cast<uint8_t *>(codes),
                    static_cast<uint8_t *>(scales));
}

// More than 128 tokens go to k_mx_few in groups of 128 where k_mx's 256 x 256 tiles leave SMs
// idle that parts of a long K can fill (256 tokens, 4096 x 11008: 17.5 us against 27.6; 512
// tokens, 1024 x 14336: 15.8 and 34.1; but 512 tokens, 2048 x 2048, 8 steps: 12.3 and 9.9), or
// where they take a second round and 128 x 128 tiles only one (384 tokens, 11008 x 4096: 14.5
// and 23.4; with more tiles than two to an SM, 512 tokens: 25.5 and 23.5).
bool few_serves(int T, int N, int nk, int sms) {
  if (T <= kFewTokens) return true;
  const int64_t units = (int64_t)((T + 127) / 128) * ((N + 127) / 128);
  const int64_t tiles = (int64_t)((T + 255) / 256) * ((N + 255) / 256);
  return (units <= sms && nk >= 16) || (units <= 2 * sms && tiles > sms / 2);
}

sfnn_status product(const void *xc, const void *xs, int T, const void *wc, const void *wsc, int N, int K, void *out,
                    int64_t ldo, int32_t out_dtype, int32_t *err, cudaStream_t s) {
  const int sms = device_sms();
  if (sms < 2) return SFNN_ERR_CUDA;
  const int nk = (K + 255) / 256;
  const int64_t rows_x = mx_rtiles(T) * nk, rows_w = mx_rtiles(N) * nk;
  if (few_serves(T, N, nk, sms)) {
    FewParams P{};
    P.T = T;
    P.N = N;
    P.nk = nk;
    P.out = out;
    P.ldo = ldo;
    P.out_dtype = out_dtype;
    P.err = err;
    if (!make_tensor_map(&P.x, xc, 1, T, K / 2, K / 2, std::min((T + 7) / 8 * 8, kFewTokens), 128, true) ||
        !make_tensor_map(&P.w, wc, 1, N, K / 2, K / 2, 128, 128, true) ||
        !make_tensor_map(&P.sx, xs, 4, rows_x, 256, 256, 1, 256, false) ||
        !make_tensor_map(&P.sw, wsc, 4, rows_w, 256, 256, 1, 256, false))
      return SFNN_ERR_CUDA;
    return launch_few(P, sms, s) == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
  }
  MxParams P{};
  P.M = T;
  P.N = N;
  P.nk = nk;
  P.out = out;
  P.ldo = ldo;
  P.out_dtype = out_dtype;
  P.vec = rows16(out, ldo, out_dtype == SFNN_F32 ? 4 : 2);
  P.err = err;
  P.tiles_m = (T + 255) / 256;
  P.tiles_n = (N + 255) / 256;
  if (!make_tensor_map(&P.a, xc, 1, T, K / 2, K / 2, 128, 128, true) ||
      !make_tensor_map(&P.b, wc, 1, N, K / 2, K / 2, 128, 128, true) ||
      !make_tensor_map(&P.sa, xs, 4, rows_x, 256, 256, 1, 256, false) ||
      !make_tensor_map(&P.sb, wsc, 4, rows_w, 256, 256, 1, 256, false))
    return SFNN_ERR_CUDA;
  return launch_pair(P, sms, s) == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
}

}  // namespace
}  // namespace sfnn

using namespace sfnn;

extern "C" {

int64_t sfnn_mxfp4_scale_bytes(int64_t rows, int32_t K) {
  if (rows < 0 || K < 1) return -1;
  return mx_rtiles(rows) * mx_ktiles(K) * 512;
}

sfnn_status sfnn_mxfp4_quantize(const void *x, int64_t ldx, int32_t rows, int32_t K, int32_t dtype, void *codes,
                                void *scales, sfnn_stream_t stream) {
  sfnn_status st = mx_check(rows, K, codes, scales);
  if (st == SFNN_OK) st = value_check(x, ldx, rows, K, dtype, false);
  if (st != SFNN_OK || rows == 0) return st;
  return quantize(x, ldx, rows, K, dtype, codes, scales, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SFNN_OK
             : SFNN_ERR_CUDA;
}

sfnn_status sfnn_mxfp4_restore(const void *codes, const void *scales, int32_t rows, int32_t K, int32_t dtype, void *out,
                               int64_t ldo, sfnn_stream_t stream) {
  sfnn_status st = mx_check(rows, K, codes, scales);
  if (st == SFNN_OK) st = value_check(out, ldo, rows, K, dtype, false);
  if (st != SFNN_OK || rows == 0) return st;
  const dim3 grid((unsigned)(((int64_t)rows + kWarps - 1) / kWarps), (unsigned)((K + kChunk - 1) / kChunk));
  return launch_pdl(k_mx_restore, grid, dim3(kWarps * 32), 0, reinterpret_cast<cudaStream_t>(stream),
                    static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), (int64_t)rows, K,
                    (int)(dtype == SFNN_BF16), (int)rows16(out, ldo, 2), static_cast<uint16_t *>(out),
                    ldo) == cudaSuccess
             ? SFNN_OK
             : SFNN_ERR_CUDA;
}

sfnn_status sfnn_mxfp4_product(const void *x_codes, const void *x_scales, int32_t T, const void *w_codes,
                               const void *w_scales, int32_t N, int32_t K, void *y, int64_t ldy, int32_t y_dtype,
                               int32_t *err, sfnn_stream_t stream) {
  sfnn_status st = mx_check(T, K, x_codes, x_scales);
  if (st == SFNN_OK) st = N < 1 ? SFNN_ERR_INVALID_ARG : mx_check(N, K, w_codes, w_scales);
  if (st == SFNN_OK) st = value_check(y, ldy, T, N, y_dtype, true);
  if (st != SFNN_OK || T == 0) return st;
  if (!err || !aligned(err, 4)) return SFNN_ERR_INVALID_ARG;
  return product(x_codes, x_scales, T, w_codes, w_scales, N, K, y, ldy, y_dtype, err,
                 reinterpret_cast<cudaStream_t>(stream));
}

int64_t sfnn_mxfp4_linear_workspace(int32_t T, int32_t K) {
  if (T < 0 || K < 1) return -1;
  if (rows_serve(T, K)) return 0;
  return ((int64_t)T * K / 2 + 255) / 256 * 256 + sfnn_mxfp4_scale_bytes(T, K);
}

sfnn_status sfnn_mxfp4_linear(const void *x, int64_t ldx, int32_t T, int32_t dtype, const void *w_codes,
                              const void *w_scales, int32_t N, int32_t K, void *y, int64_t ldy, int32_t y_dtype, void *ws,
                              int64_t ws_bytes, int32_t *err, sfnn_stream_t stream) {
  sfnn_status st = mx_check(T, K, w_codes, w_scales);
  if (st == SFNN_OK) st = N < 1 ? SFNN_ERR_INVALID_ARG : mx_check(N, K, w_codes, w_scales);
  if (st == SFNN_OK) st = value_check(x, ldx, T, K, dtype, false);
  if (st == SFNN_OK) st = value_check(y, ldy, T, N, y_dtype, true);
  if (st != SFNN_OK || T == 0) return st;
  if (!err || !aligned(err, 4)) return SFNN_ERR_INVALID_ARG;
  const int64_t need = sfnn_mxfp4_linear_workspace(T, K);
  if (need > 0 && (!ws || !aligned(ws, 16) || ws_bytes < need)) return SFNN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows_serve(T, K)) {
    const int vec = rows16(x, ldx, 2), bf16 = dtype == SFNN_BF16, sms = device_sms();
    if (sms < 1) return SFNN_ERR_CUDA;
    const cudaError_t e = T == 1   ? launch_rows<1>(x, ldx, T, vec, bf16, w_codes, w_scales, N, K, y, ldy, y_dtype, sms, s)
                          : T == 2 ? launch_rows<2>(x, ldx, T, vec, bf16, w_codes, w_scales, N, K, y, ldy, y_dtype, sms, s)
                                   : launch_rows<4>(x, ldx, T, vec, bf16, w_codes, w_scales, N, K, y, ldy, y_dtype, sms, s);
    return e == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
  }
  void *scales = static_cast<unsigned char *>(ws) + ((int64_t)T * K / 2 + 255) / 256 * 256;
  if (quantize(x, ldx, T, K, dtype, ws, scales, s) != cudaSuccess) return SFNN_ERR_CUDA;
  return product(ws, scales, T, w_codes, w_scales, N, K, y, ldy, y_dtype, err, s);
}

}  // extern "C"
