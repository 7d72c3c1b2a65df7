// slim.cu -- the dense products for few tokens (T <= 128): bound by the weights' bytes.
//
// The tokens lie on the MMA's M side (128 lanes, T of them real; the rest of the A tile is
// whatever shared memory holds, and only reaches accumulator lanes nobody reads), the
// weights on its N side, so a CTA can own ANY number of weight rows: the rows are dealt out
// evenly over the SMs (75 or 76 neurons each of 11008 over 148), every CTA streams its own
// rows over all of K once, and nothing is split or joined.  A stage holds one or more
// 64-deep chunks of every row (TMA, 128-byte swizzle), as many stages as about 100 KB hold,
// so that two CTAs of consecutive kernels fit one SM: the down projection's CTA starts
// while the gate/up kernel drains, and requests its first weights before it waits for H.
//
// Down projection with more than 32 tokens: a CTA's share of the weight rows (28 of 4096)
// no longer outweighs the H rows it reads with them, so a cluster of CTAs splits K over wider
// tiles and adds its parts through distributed shared memory in rank order.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kThreads = 192;  // warp 0 loads, warp 1 issues the MMAs, warps 2-5 take 32 tokens each
constexpr int kMaxStages = 8;

struct alignas(64) SlimParams {
  CUtensorMap a, b0, b1;
  int T, N, nk;         // nk: 64-deep chunks of K
  int nb, nb8, n16;     // weight rows of a tile; rounded up to 8 (bytes), to 16 (MMA N)
  int tiles;
  int tb8;              // T rounded up to 8
  int kps, stages;      // chunks per stage
  int split;            // CTAs of a cluster that share a tile's K
  int early;            // weights may be read before the kernel before has finished
  int tmem_cols;
  int bf16, out32, relu;
  const void *bias;
  void *out;
  int64_t ldo;
  int32_t *err;
};

// `cols` values of one token to p (4-byte aligned when 16-bit: tiles start on even columns).
__device__ __forceinline__ void store_cols(const SlimParams &P, int64_t row, int col, const float v[32], int cols) {
  if (P.out32) {
    float *o = static_cast<float *>(P.out) + row * P.ldo + col;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < cols) o[i] = v[i];
  } else {
    uint16_t *o = static_cast<uint16_t *>(P.out) + row * P.ldo + col;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const uint32_t w = pack16(v[i], v[i + 1], P.bf16);
      if (i + 1 < cols)
        *reinterpret_cast<uint32_t *>(o + i) = w;
      else if (i < cols)
        o[i] = (uint16_t)w;
    }
  }
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads) k_slim(const __grid_constant__ SlimParams P) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty;
  __shared__ uint32_t tmem_slot;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t stage0 = (raw + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = GATED ? 1 : P.split;
  const int part = split > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / split, units = gridDim.x / split;
  const uint32_t a_bytes = (uint32_t)P.tb8 * 128u, b_bytes = (uint32_t)P.nb8 * 128u;
  const uint32_t chunk_bytes = a_bytes + (GATED ? 2u : 1u) * b_bytes;
  const uint32_t stage_bytes = chunk_bytes * (uint32_t)P.kps;
  const int stages = P.stages;
  const int k_lo = (int)((int64_t)part * P.nk / split), k_hi = (int)((int64_t)(part + 1) * P.nk / split);
  const int steps = (k_hi - k_lo + P.kps - 1) / P.kps;
  const uint32_t up_col = (uint32_t)P.n16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    bar_init(&acc_full, 1);
    bar_init(&acc_empty, 4);
    bar_init_fence();
  }
  if (warp == 1) tm_alloc<1>(&tmem_slot, (uint32_t)P.tmem_cols);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // the box rows are tb8 and nb: a tile's rows past N and T read as zeros and still count
      auto load_b = [&](int s, int t, int k0, int kn) {
        const uint32_t st = stage0 + (uint32_t)s * stage_bytes;
        for (int c = 0; c < kn; ++c) {
          const uint32_t at = st + (uint32_t)c * chunk_bytes + a_bytes;
          tma_load_2d(at, &P.b0, (k0 + c) * 64, t * P.nb, &full[s]);
          if (GATED) tma_load_2d(at + b_bytes, &P.b1, (k0 + c) * 64, t * P.nb, &full[s]);
        }
      };
      auto load_a = [&](int s, int k0, int kn) {
        const uint32_t st = stage0 + (uint32_t)s * stage_bytes;
        for (int c = 0; c < kn; ++c) tma_load_2d(st + (uint32_t)c * chunk_bytes, &P.a, (k0 + c) * 64, 0, &full[s]);
      };
      const uint32_t chunk_tx = a_bytes + (GATED ? 2u : 1u) * (uint32_t)P.nb * 128u;
      const int pre = P.early ? min(stages, steps) : 0;
      if (unit < P.tiles)
        for (int i = 0; i < pre; ++i) {
          const int k0 = k_lo + i * P.kps, kn = min(P.kps, k_hi - k0);
          bar_expect_tx(&full[i], chunk_tx * (uint32_t)kn);
          load_b(i, unit, k0, kn);
        }
      pdl_wait();
      pdl_launch_dependents();
      int it = 0;
      bool ok = true;
      for (int t = unit; t < P.tiles && ok; t += units) {
        for (int i = 0; i < steps; ++i, ++it) {
          const int s = it % stages, k0 = k_lo + i * P.kps, kn = min(P.kps, k_hi - k0);
          if (it >= pre) {
            if (!bar_wait(&empty[s], (uint32_t)((it / stages) & 1) ^ 1u)) {
              ok = false;
              break;
            }
            bar_expect_tx(&full[s], chunk_tx * (uint32_t)kn);
            load_b(s, t, k0, kn);
          }
          load_a(s, k0, kn);
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
      const uint32_t idesc = mma_desc_16(128, P.n16, P.bf16, 0, 0);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = unit; t < P.tiles && ok; t += units, ++n) {
        if (!bar_wait(&acc_empty, (uint32_t)(n & 1) ^ 1u)) {
          ok = false;
          break;
        }
        tm_fence_after();
        for (int i = 0; i < steps; ++i, ++it) {
          const int s = it % stages, kn = min(P.kps, k_hi - (k_lo + i * P.kps));
          if (!bar_wait(&full[s], (uint32_t)((it / stages) & 1))) {
            ok = false;
            break;
          }
          tm_fence_after();
          for (int c = 0; c < kn; ++c) {
            const uint32_t a = stage0 + (uint32_t)s * stage_bytes + (uint32_t)c * chunk_bytes, b = a + a_bytes;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t acc = (i > 0 || c > 0 || k > 0) ? 1u : 0u;
              const uint64_t da = mat_desc(a + k * 32, 16, 1024);
              mma_16<1>(tmem, da, mat_desc(b + k * 32, 16, 1024), idesc, acc);
              if (GATED) mma_16<1>(tmem + up_col, da, mat_desc(b + b_bytes + k * 32, 16, 1024), idesc, acc);
            }
          }
          mma_commit(&empty[s]);
        }
        if (ok) mma_commit(&acc_full);
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  } else {
    const int quad = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int row = quad * 32 + lane;
    const bool busy = quad * 32 < P.T;
    pdl_wait();  // nothing is written before the kernel before has finished
    int n = 0;
    for (int t = unit; t < P.tiles; t += units, ++n) {
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full, (uint32_t)(n & 1)))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        break;
      }
      __syncwarp();
      tm_fence_after();
      const int n0 = t * P.nb, rows = min(P.nb, P.N - n0);
      if (split > 1) break;  // one tile per cluster, joined below
      if (busy)
        for (int c = 0; c < rows; c += 32) {
          uint32_t g[32];
          float v[32];
          __syncwarp();
          tm_ld32(lanes + c, g);
          if (GATED) {
            uint32_t u[32];
            tm_ld32(lanes + up_col + c, u);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x = __uint_as_float(g[i]);
              if (P.bias && c + i < rows) x += load16(P.bias, n0 + c + i, P.bf16);
              v[i] = (x < 0.f ? 0.f : x) * __uint_as_float(u[i]);
            }
          } else {
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[i] = __uint_as_float(g[i]);
              if (P.relu) {
                if (P.bias && c + i < rows) v[i] += load16(P.bias, n0 + c + i, P.bf16);
                v[i] = v[i] < 0.f ? 0.f : v[i];
              }
            }
          }
          if (row < P.T) store_cols(P, row, n0 + c, v, rows - c);
        }
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster(cluster_addr(&acc_empty, 0));
    }
  }
  __syncwarp();
  if (split > 1) {
    // Every CTA of the cluster has its accumulators: the others put theirs into rank 0's
    // stage memory (no load or MMA touches it any more), rank 0 adds them in rank order.
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const bool busy = warp >= 2 && quad * 32 < P.T;
    const int n0 = unit * P.nb, rows = min(P.nb, P.N - n0);
    const uint32_t sums = stage0 - raw;  // the same offset in every CTA
    cluster_sync_all();
    tm_fence_after();
    if (busy && part > 0) {
      const uint32_t dst0 = cluster_addr(smem_raw, 0) + sums;
      for (int c = 0; c < rows; c += 32) {
        uint32_t g[32];
        __syncwarp();
        tm_ld32(lanes + c, g);
        tm_wait_ld();
        const uint32_t dst = dst0 + (uint32_t)(((part - 1) * P.n16 + c) * 128 + row) * 4u;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < rows)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + (uint32_t)i * 512u), "r"(g[i]) : "memory");
      }
    }
    __syncwarp();
    cluster_sync_all();
    if (busy && part == 0)
      for (int c = 0; c < rows; c += 32) {
        uint32_t g[32];
        float v[32];
        __syncwarp();
        tm_ld32(lanes + c, g);
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(g[i]);
        for (int p = 1; p < split; ++p) {
          const float *src = reinterpret_cast<const float *>(smem_raw + sums) + ((p - 1) * P.n16 + c) * 128 + row;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < rows) v[i] += src[i * 128];
        }
        if (row < P.T) store_cols(P, row, n0 + c, v, rows - c);
      }
    __syncwarp();
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == 1) tm_dealloc<1>(tmem, (uint32_t)P.tmem_cols);
}

int up_to(int v, int to) { return (v + to - 1) / to * to; }

template <bool GATED>
cudaError_t launch(SlimParams &P, int grid, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t attr = allow_smem(k_slim<GATED>, 224 * 1024, ready);
  if (attr != cudaSuccess) return attr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = (unsigned)(GATED ? 1 : P.split);
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_slim<GATED>, P);
}

}  // namespace

bool slim_serves(int T) { return T <= 128; }

sfnn_status launch_slim(const SlimArgs &q, int sms, cudaStream_t s) {
  const bool gated = q.w1 != nullptr;
  SlimParams P{};
  P.T = q.T;
  P.N = q.N;
  P.nk = (int)((q.K + 63) / 64);
  P.tb8 = up_to(q.T, 8);
  P.split = 1;
  // weight rows of a CTA: an even share (an even number, so that 16-bit results go out in
  // 4-byte words), at most 128, at least 16
  const int rounds = (q.N + sms * 128 - 1) / (sms * 128);
  P.nb = std::max(16, up_to((q.N + sms * rounds - 1) / (sms * rounds), 2));
  if (!gated && q.T > 32 && P.nb < q.T) {
    // a cluster splits K: tiles of about 128 rows, so that H's rows are read by fewer CTAs
    int split = 2;
    while (split < 4 && split * 2 * P.nb <= 128 && P.nk >= split * 16) split *= 2;
    if (rounds == 1 && P.nk >= split * 8) {
      P.split = split;
      P.nb = std::min(128, std::max(16, up_to((int)(((int64_t)q.N * split + sms - 1) / sms), 2)));
    }
  }
  P.nb8 = up_to(P.nb, 8);
  P.n16 = up_to(P.nb, 16);
  P.tiles = (q.N + P.nb - 1) / P.nb;
  P.tmem_cols = 32;
  while (P.tmem_cols < (gated ? 2 : 1) * P.n16 || P.tmem_cols < up_to(P.n16, 32) + (gated ? P.n16 : 0)) P.tmem_cols *= 2;
  const int chunk = P.tb8 * 128 + (gated ? 2 : 1) * P.nb8 * 128;
  // two CTAs on an SM (besides the A tile's overhang), where that leaves enough in flight
  const int budget = (q.T > 64 || chunk > 24 * 1024 ? 200 : 92) * 1024;
  P.kps = std::max(1, std::min({4, 20 * 1024 / chunk, (P.nk + P.split - 1) / P.split}));
  P.stages = std::max(2, std::min(kMaxStages, budget / (P.kps * chunk)));
  // (a cluster's parts are joined in rank 0's stage memory: T lanes x nb columns of 3 parts)
  size_t smem = (size_t)P.stages * P.kps * chunk + 16384 + 1024;
  if (P.split > 1) smem = std::max(smem, (size_t)(P.split - 1) * P.n16 * 512 + 1024);
  P.early = q.early;
  P.bf16 = q.bf16;
  P.out32 = q.out32;
  P.relu = q.relu;
  P.bias = q.bias;
  P.out = q.out;
  P.ldo = q.ldo;
  P.err = q.err;
  if (!make_tensor_map(&P.a, q.x, 2, q.T, q.K, q.ldx, P.tb8, 64, true) ||
      !make_tensor_map(&P.b0, q.w0, 2, q.N, q.K, q.ldw0, P.nb, 64, true) ||
      (gated && !make_tensor_map(&P.b1, q.w1, 2, q.N, q.K, q.ldw1, P.nb, 64, true)))
    return SFNN_ERR_CUDA;
  const int grid = P.split > 1 ? P.tiles * P.split : std::min(P.tiles, sms);
  const cudaError_t e = gated ? launch<true>(P, grid, smem, s) : launch<false>(P, grid, smem, s);
  return e == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
}

}  // namespace sfnn
