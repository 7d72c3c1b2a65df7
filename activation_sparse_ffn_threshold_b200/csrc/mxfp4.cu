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
// step of a CTA pair takes about 512 cycles and moves 35 KB per SM from L2: what bounds it is
// the L2 -> shared memory path as much as the tensor pipe.
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
// requested first; four lanes hold a block.  Bound by bytes (2 read, 0.53 written a value).
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
constexpr int kSfSlot = 32;             // A: 2 x 4 columns; B: 2 x 12 from column 8 on

struct alignas(64) MxParams {
  CUtensorMap a, b, sa, sb;
  int M, N, nk;          // nk: 256-deep steps
  int tiles_m, tiles_n;
  int nt;                // columns of C per tile (CG = 2: 256)
  int stages;
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

// CG = 2: 256 x 256 tiles by CTA pairs, 128 rows of X and of W in each CTA.  CG = 1: 128
// tokens x nt columns (nt a multiple of 32) by single CTAs, for few tokens: nt is chosen so
// that the tiles fill the SMs.
//
// The accumulators are single (256 columns; the scales need the rest of tensor memory): the
// epilogue warps copy a finished tile to registers, hand the columns back, and store while
// the next tile's MMAs run.  Scale slots go by stage: a slot is written again only after the
// stage's MMAs have completed.
template <int CG>
__global__ void __launch_bounds__(kThreads, 1) k_mx(const __grid_constant__ MxParams P) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty;
  __shared__ uint32_t tmem_slot;
  const uint32_t stage0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int unit = CG == 2 ? blockIdx.x >> 1 : blockIdx.x, units = CG == 2 ? gridDim.x >> 1 : gridDim.x;
  const int ntiles = P.tiles_m * P.tiles_n;
  const uint32_t b_bytes = CG == 2 ? 16384u : (uint32_t)P.nt * 128u;
  const uint32_t stage_bytes = 16384u + b_bytes + 4096u;
  const int stages = P.stages;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    bar_init(&acc_full, 1);
    bar_init(&acc_empty, 8 * CG);
    bar_init_fence();
  }
  if (warp == 1) tm_alloc<CG>(&tmem_slot, kTmem);
  tm_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
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
        const int m0 = (CG == 2 ? pos.m * 256 : pos.m * 128) + (int)rank * 128;
        const int n0 = pos.n * P.nt;                                   // the tile's columns
        const int nb0 = CG == 2 ? n0 + (int)rank * 128 : n0;           // this CTA's rows of W
        const int rb = n0 >> 7;                                        // first scale tile row of W
        const int nsf = CG == 2 ? 2 : ((n0 & 127) + P.nt + 127) >> 7;  // and how many
        for (int kc = 0; kc < P.nk; ++kc, ++it) {
          const int s = it % stages;
          if (!bar_wait(&empty[s], (uint32_t)((it / stages) & 1) ^ 1u)) {
            ok = false;
            break;
          }
          const uint32_t bytes = 16384u + b_bytes + 1024u + (uint32_t)nsf * 1024u;
          if (rank == 0) bar_expect_tx(&full[s], CG * bytes);
          const uint32_t a = stage0 + (uint32_t)s * stage_bytes, b = a + 16384u, sa = b + b_bytes, sb = sa + 1024u;
          if (CG == 2) {
            const uint32_t bar = cluster_addr(&full[s], 0);
            tma_load_2d_pair(a, &P.a, kc * 128, m0, bar);
            tma_load_2d_pair(b, &P.b, kc * 128, nb0, bar);
            tma_load_2d_pair(sa, &P.sa, 0, (m0 >> 7) * P.nk + kc, bar);
            for (int r = 0; r < nsf; ++r) tma_load_2d_pair(sb + r * 1024u, &P.sb, 0, (rb + r) * P.nk + kc, bar);
          } else {
            tma_load_2d(a, &P.a, kc * 128, m0, &full[s]);
            tma_load_2d(b, &P.b, kc * 128, nb0, &full[s]);
            tma_load_2d(sa, &P.sa, 0, (m0 >> 7) * P.nk + kc, &full[s]);
            for (int r = 0; r < nsf; ++r) tma_load_2d(sb + r * 1024u, &P.sb, 0, (rb + r) * P.nk + kc, &full[s]);
          }
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
    if (rank == 0) {
      int it = 0, i = 0;
      bool ok = true;
      const uint32_t id0 = mx_idesc(128 * CG, P.nt, 0), id2 = mx_idesc(128 * CG, P.nt, 2);
      for (int t = unit; t < ntiles && ok; t += units, ++i) {
        const TilePos pos = tile_pos(t, P.tiles_m, P.tiles_n);
        const int n0 = pos.n * P.nt;
        const int nsf = CG == 2 ? 2 : ((n0 & 127) + P.nt + 127) >> 7;
        const int shift = CG == 2 ? 0 : (n0 & 127) >> 5;  // 32-row groups of the first scale tile before the tile
        if (!__all_sync(0xffffffffu, bar_wait(&acc_empty, (uint32_t)(i & 1) ^ 1u))) {
          ok = false;
          break;
        }
        tm_fence_after();
        for (int kc = 0; kc < P.nk; ++kc, ++it) {
          const int s = it % stages;
          if (!__all_sync(0xffffffffu, bar_wait(&full[s], (uint32_t)((it / stages) & 1)))) {
            ok = false;
            break;
          }
          const uint32_t a = stage0 + (uint32_t)s * stage_bytes, b = a + 16384u, sa = b + b_bytes, sb = sa + 1024u;
          if (CG == 1 && shift) {
            // the MMA wants the tile's first column's scales in an aligned tensor-memory column:
            // move the 32-row groups (a 4-byte word of each lane's 16) down to the tile's start
            for (int h = 0; h < 2; ++h)
              for (int c = 0; c < P.nt >> 5; ++c) {
                const int f = c + shift;
                const uint32_t at = sb + (uint32_t)(h * 512 + lane * 16);
                uint32_t w;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at + (uint32_t)((f >> 2) * 1024 + (f & 3) * 4)));
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + (uint32_t)((c >> 2) * 1024 + (c & 3) * 4)), "r"(w)
                             : "memory");
              }
            fence_async_shared();
            __syncwarp();
          }
          if (lane == 0) {
            tm_fence_after();
            const uint32_t ta = tmem + kSf + (uint32_t)(s * kSfSlot), tb = ta + 8u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // the step's two 128-deep scale tiles
              copy_scales<CG>(ta + h * 4, sa + h * 512);
              for (int r = 0; r < nsf; ++r) copy_scales<CG>(tb + h * 12 + r * 4, sb + r * 1024 + h * 512);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_mx<CG>(tmem + kAcc, mat_desc(a + k * 32, 16, 1024), mat_desc(b + k * 32, 16, 1024), (k & 1) ? id2 : id0,
                         ta + (k >> 1) * 4, tb + (k >> 1) * 12, (kc > 0 || k > 0) ? 1u : 0u);
            if (CG == 2)
              mma_commit_pair(&empty[s]);
            else
              mma_commit(&empty[s]);
          }
          __syncwarp();
        }
        if (ok && lane == 0) {
          if (CG == 2)
            mma_commit_pair(&acc_full);
          else
            mma_commit(&acc_full);
        }
      }
      if (!ok && lane == 0) latch_error(P.err, kErrTimeout);
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    int i = 0;
    for (int t = unit; t < ntiles; t += units, ++i) {
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full, (uint32_t)(i & 1)))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        break;
      }
      __syncwarp();
      tm_fence_after();
      const TilePos pos = tile_pos(t, P.tiles_m, P.tiles_n);
      const int64_t row = (int64_t)pos.m * (128 * CG) + rank * 128 + quad * 32 + lane;
      const int n0 = pos.n * P.nt;
      // 32-column units half, half + 2, ...: at most four
      uint32_t v[4][32];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if ((half + 2 * u) * 32 < P.nt) tm_ld32(tmem + ((uint32_t)(quad * 32) << 16) + kAcc + (half + 2 * u) * 32, v[u]);
      tm_wait_ld();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(cluster_addr(&acc_empty, 0));
      if (row >= P.M) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = n0 + (half + 2 * u) * 32;
        const int cols = min(32, min(P.N, n0 + P.nt) - col);
        if ((half + 2 * u) * 32 >= P.nt || cols <= 0) continue;
        if (P.out_dtype == SFNN_F32) {
          float *o = static_cast<float *>(P.out) + row * P.ldo + col;
          if (P.vec && cols == 32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              reinterpret_cast<uint4 *>(o)[j] = make_uint4(v[u][4 * j], v[u][4 * j + 1], v[u][4 * j + 2], v[u][4 * j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < cols) o[j] = __uint_as_float(v[u][j]);
          }
        } else {
          const bool bf16 = P.out_dtype == SFNN_BF16;
          uint16_t *o = static_cast<uint16_t *>(P.out) + row * P.ldo + col;
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            p[j] = pack16(__uint_as_float(v[u][2 * j]), __uint_as_float(v[u][2 * j + 1]), bf16);
          if (P.vec && cols == 32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              reinterpret_cast<uint4 *>(o)[j] = make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < cols) o[j] = (uint16_t)(p[j >> 1] >> (16 * (j & 1)));
          }
        }
      }
    }
  }
  __syncwarp();
  tm_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tm_fence_after();
  if (warp == 1) tm_dealloc<CG>(tmem, kTmem);
}

size_t mx_smem(int stages, uint32_t b_bytes) { return (size_t)stages * (16384 + b_bytes + 4096) + 1024; }

cudaError_t launch_mx(const MxParams &P, bool pair, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready1{0}, ready2{0};
  const size_t limit = 220 * 1024;
  const cudaError_t attr = pair ? allow_smem(k_mx<2>, limit, ready2) : allow_smem(k_mx<1>, limit, ready1);
  if (attr != cudaSuccess) return attr;
  cudaLaunchConfig_t cfg = {};
  const int tiles = P.tiles_m * P.tiles_n;
  cfg.gridDim = dim3(pair ? 2 * std::min(num_sms / 2, tiles) : std::min(num_sms, tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = mx_smem(P.stages, pair ? 16384u : (uint32_t)P.nt * 128u);
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  if (pair) {
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 2;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return pair ? cudaLaunchKernelEx(&cfg, k_mx<2>, P) : cudaLaunchKernelEx(&cfg, k_mx<1>, P);
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

sfnn_status product(const void *xc, const void *xs, int T, const void *wc, const void *wsc, int N, int K, void *out,
                    int64_t ldo, int32_t out_dtype, int32_t *err, cudaStream_t s) {
  const int sms = device_sms();
  if (sms < 2) return SFNN_ERR_CUDA;
  MxParams P{};
  P.M = T;
  P.N = N;
  P.nk = (K + 255) / 256;
  P.out = out;
  P.ldo = ldo;
  P.out_dtype = out_dtype;
  P.vec = rows16(out, ldo, out_dtype == SFNN_F32 ? 4 : 2);
  P.err = err;
  const bool pair = T > 128;
  if (pair) {
    P.nt = 256;
    P.tiles_m = (T + 255) / 256;
    P.stages = kMaxStages;
  } else {
    // the narrowest tile (a multiple of 32) that still needs the fewest rounds over the SMs
    P.tiles_m = 1;
    const int units = (N + 31) / 32;
    const int rounds = (units + 8 * sms - 1) / (8 * sms);
    P.nt = 32 * std::min(8, (units + rounds * sms - 1) / (rounds * sms));
    P.stages = std::min<int>(kMaxStages, (int)((219 * 1024) / (16384 + P.nt * 128 + 4096)));
  }
  P.tiles_n = (N + P.nt - 1) / P.nt;
  const int64_t rows_a = mx_rtiles(T) * P.nk, rows_b = mx_rtiles(N) * P.nk;
  if (!make_tensor_map(&P.a, xc, 1, T, K / 2, K / 2, 128, 128, true) ||
      !make_tensor_map(&P.b, wc, 1, N, K / 2, K / 2, pair ? 128 : P.nt, 128, true) ||
      !make_tensor_map(&P.sa, xs, 4, rows_a, 256, 256, 1, 256, false) ||
      !make_tensor_map(&P.sb, wsc, 4, rows_b, 256, 256, 1, 256, false))
    return SFNN_ERR_CUDA;
  return launch_mx(P, pair, sms, s) == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
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
  if (!err) return SFNN_ERR_INVALID_ARG;
  return product(x_codes, x_scales, T, w_codes, w_scales, N, K, y, ldy, y_dtype, err,
                 reinterpret_cast<cudaStream_t>(stream));
}

int64_t sfnn_mxfp4_linear_workspace(int32_t T, int32_t K) {
  if (T < 0 || K < 1) return -1;
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
  if (!err || !ws || !aligned(ws, 16) || ws_bytes < sfnn_mxfp4_linear_workspace(T, K)) return SFNN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void *scales = static_cast<unsigned char *>(ws) + ((int64_t)T * K / 2 + 255) / 256 * 256;
  if (quantize(x, ldx, T, K, dtype, ws, scales, s) != cudaSuccess) return SFNN_ERR_CUDA;
  return product(ws, scales, T, w_codes, w_scales, N, K, y, ldy, y_dtype, err, s);
}

}  // extern "C"
