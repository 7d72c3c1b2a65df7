// slim.cu -- the dense products for few tokens (T <= 128) whose time is the weights' bytes (the
// rule is slim_serves in gated.cu).
//
// The weights lie on the MMA's M side (128 lanes), the tokens on its N side.  A tile need not
// fill the 128 lanes: the rest of the A tile is whatever shared memory holds, and only
// reaches accumulator lanes nobody reads.  So a tile is any number of weight rows, the rows
// are dealt out evenly over the SMs (75 neurons each of 11008 over 148), and every byte of
// them is read once.  An even share under 64 rows would be a thin tile (28 of 4096 rows of
// the down projection), slow in small copies: a cluster of 2 or 4 CTAs takes a wider tile,
// splits its K, and adds the parts through distributed shared memory in rank order (1 token,
// 4096 x 11008, both kernels: 61 us against 76 with thin tiles).
//
// A stage holds at least two 64-deep chunks of every row: 256 contiguous bytes of it (TMA,
// 128-byte swizzle).
//
// Measured: 37 tokens, 8192 x 28672 bf16, both kernels 243 to 267 us on several cards (5.3 to 5.8
// TB/s of weights); 1 token, 4096 x 11008 fp16, 53.9 us: 6.4 and 7.1 TB/s while they stream, 12 us
// of ends and beginnings.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kThreads = 192;  // warp 0 loads, warp 1 issues the MMAs, warps 2-5 take 32 weight rows each
constexpr int kMaxStages = 8;

struct alignas(64) SlimParams {
  CUtensorMap x, w0, w1;
  int T, N, nk;         // nk: 64-deep chunks of K
  int nb, nb8;          // weight rows of a tile; rounded up to 8 (its place in a stage)
  int tiles;
  int t8, t16;          // T rounded up to 8 (rows loaded), to 16 (MMA N)
  int kps, stages;      // chunks per stage
  int split;            // CTAs of a cluster that share a tile's K
  int apart;            // the parts are joined in memory of their own behind the stages (else in the stages)
  int m64;              // 64-lane MMAs (a row's accumulators: lane r % 16 of quarter r / 16)
  int early;            // weights may be read before the kernel before has finished
  int tmem_cols, up_col;
  int bf16, out32;
  const void *bias;
  void *out;
  int64_t ldo;
  int32_t *err;
};

// This thread's weight row: its accumulators of tokens [t0, t0 + 8) -> out[t][col].  (The
// epilogues go by eight tokens in a loop: unrolled further, a single token's few instructions
// lie far apart, and each first fetch of them is a microsecond at the kernel's end.)
__device__ __forceinline__ void store_tokens(const SlimParams &P, int col, int t0, const float v[8]) {
  if (P.out32) {
    float *o = static_cast<float *>(P.out) + t0 * P.ldo + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t0 + i < P.T) o[i * P.ldo] = v[i];
  } else {
    uint16_t *o = static_cast<uint16_t *>(P.out) + t0 * P.ldo + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t0 + i < P.T) o[i * P.ldo] = (uint16_t)pack16(v[i], 0.f, P.bf16);
  }
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads) k_slim(const __grid_constant__ SlimParams P) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty, parts_in;
  __shared__ uint32_t tmem_slot;
  constexpr int NP = GATED ? 2 : 1;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t stage0 = (raw + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = P.split;
  const int part = split > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / split, units = gridDim.x / split;
  // a chunk: the tokens' rows, then the weight tiles (an MMA reads past a tile's rows into
  // what follows, at the end into the overhang behind the last stage)
  const uint32_t x_bytes = (uint32_t)P.t8 * 128u, w_bytes = (uint32_t)P.nb8 * 128u;
  const uint32_t chunk_bytes = x_bytes + NP * w_bytes;
  const uint32_t stage_bytes = chunk_bytes * (uint32_t)P.kps;
  const int stages = P.stages;
  const int k_lo = (int)((int64_t)part * P.nk / split), k_hi = (int)((int64_t)(part + 1) * P.nk / split);
  const int steps = (k_hi - k_lo + P.kps - 1) / P.kps;

  const int pre = P.early && unit < P.tiles ? min(stages, steps) : 0;  // stages of weights requested ahead
  auto load_w = [&](int s, int t, int k0, int kn) {
    const uint32_t at = stage0 + (uint32_t)s * stage_bytes + x_bytes;
    for (int c = 0; c < kn; ++c) tma_load_2d(at + (uint32_t)c * chunk_bytes, &P.w0, (k0 + c) * 64, t * P.nb, &full[s]);
    if (GATED)
      for (int c = 0; c < kn; ++c)
        tma_load_2d(at + w_bytes + (uint32_t)c * chunk_bytes, &P.w1, (k0 + c) * 64, t * P.nb, &full[s]);
  };
  // rows of a box past T or N read as zeros and count like the others
  const uint32_t chunk_tx = x_bytes + NP * (uint32_t)P.nb * 128u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    bar_init(&acc_full, 1);
    bar_init(&acc_empty, 4);
    bar_init(&parts_in, 4u * (uint32_t)(split > 1 ? split - 1 : 1));
    bar_init_fence();
    fence_async_shared();
    // the first weights, before the rest of the CTA is set up
    for (int i = 0; i < pre; ++i) {
      const int k0 = k_lo + i * P.kps, kn = min(P.kps, k_hi - k0);
      bar_expect_tx(&full[i], chunk_tx * (uint32_t)kn);
      load_w(i, unit, k0, kn);
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();  // rank 0's barrier is there before a part arrives
  if (warp == 1) tm_alloc<1>(&tmem_slot, (uint32_t)P.tmem_cols);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      auto load_x = [&](int s, int k0, int kn) {
        const uint32_t st = stage0 + (uint32_t)s * stage_bytes;
        for (int c = 0; c < kn; ++c) tma_load_2d(st + (uint32_t)c * chunk_bytes, &P.x, (k0 + c) * 64, 0, &full[s]);
      };
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
            load_w(s, t, k0, kn);
          }
          load_x(s, k0, kn);
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
      const uint32_t idesc = mma_desc_16(P.m64 ? 64 : 128, P.t16, P.bf16, 0, 0);
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
            const uint32_t x = stage0 + (uint32_t)s * stage_bytes + (uint32_t)c * chunk_bytes, w = x + x_bytes;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t acc = (i > 0 || c > 0 || k > 0) ? 1u : 0u;
              const uint64_t dx = mat_desc(x + k * 32, 16, 1024);
              mma_16<1>(tmem, mat_desc(w + k * 32, 16, 1024), dx, idesc, acc);
              if (GATED) mma_16<1>(tmem + (uint32_t)P.up_col, mat_desc(w + w_bytes + k * 32, 16, 1024), dx, idesc, acc);
            }
          }
          mma_commit(&empty[s]);
        }
        if (ok) mma_commit(&acc_full);
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  }
  const int quad = warp & 3;
  const int row = P.m64 ? (lane < 16 ? quad * 16 + lane : 128) : quad * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  const bool worker = warp >= 2;
  const bool busy = worker && quad * (P.m64 ? 16 : 32) < P.nb;
  auto load_bias = [&](int t) {
    const int col = t * P.nb + row;
    return GATED && P.bias && row < P.nb && col < P.N ? load16(P.bias, col, P.bf16) : 0.f;
  };
  // the epilogue of this thread's weight row, with the other parts of a split tile at `sums`
  auto epilogue = [&](int t, float bias, const float *sums) {
    const int col = t * P.nb + row;
    const bool live = row < P.nb && col < P.N;
#pragma unroll 1
    for (int c = 0; c < P.T; c += 8) {
      uint32_t g[8], u[8];
      float v[8];
      __syncwarp();
      tm_ld8(lanes + c, g);
      if (GATED) tm_ld8(lanes + (uint32_t)P.up_col + c, u);
      tm_wait_ld();
      if (!live) continue;
      if (sums)
#pragma unroll 1
        for (int p = 0; p < split - 1; ++p) {
          const float *a = sums + ((size_t)(p * NP) * P.T + c) * 128 + row;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < P.T) {
              g[i] = __float_as_uint(__uint_as_float(g[i]) + a[i * 128]);
              if (GATED) u[i] = __float_as_uint(__uint_as_float(u[i]) + a[(P.T + i) * 128]);
            }
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = __uint_as_float(g[i]);
        if (GATED) {
          v[i] += bias;
          v[i] = v[i] < 0.f ? 0.f : v[i];
          v[i] *= __uint_as_float(u[i]);
        }
      }
      store_tokens(P, col, c, v);
    }
  };
  if (worker) {
    pdl_wait();  // nothing is written before the kernel before has finished
    int n = 0;
    for (int t = unit; t < P.tiles; t += units, ++n) {
      const float bias = load_bias(t);
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full, (uint32_t)(n & 1)))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        break;
      }
      __syncwarp();
      tm_fence_after();
      if (split > 1) break;  // one tile per cluster, joined below
      if (busy) epilogue(t, bias, nullptr);
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty, 0));
    }
  }
  __syncwarp();
  if (split > 1) {
    // The other ranks put their accumulators into rank 0's shared memory, which adds them in
    // rank order: behind the stages where they fit, else into the stages, once every CTA of
    // the cluster has its accumulators (no load or MMA touches the stages any more).
    const uint32_t sums = stage0 - raw + (P.apart ? (uint32_t)stages * stage_bytes : 0u);  // the same offset in every CTA
    if (!P.apart) cluster_sync_all();
    tm_fence_after();
    if (worker && part > 0) {
      const uint32_t dst0 = cluster_addr(smem_raw, 0) + sums + (uint32_t)((part - 1) * NP * P.T * 128 + row) * 4u;
      if (busy)
#pragma unroll 1
        for (int p = 0; p < NP; ++p)
#pragma unroll 1
          for (int c = 0; c < P.T; c += 8) {
            uint32_t g[8];
            __syncwarp();
            tm_ld8(lanes + (uint32_t)(p * P.up_col + c), g);
            tm_wait_ld();
            const uint32_t dst = dst0 + (uint32_t)(p * P.T + c) * 512u;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c + i < P.T)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + (uint32_t)i * 512u), "r"(g[i]) : "memory");
          }
      __syncwarp();  // the arrival releases the whole warp's stores
      if (lane == 0) bar_arrive_cluster(cluster_addr(&parts_in, 0));
    }
    __syncwarp();
    cluster_arrive();  // this CTA writes to no other any more
    if (worker && part == 0) {
      const float bias = load_bias(unit);
      if (!__all_sync(0xffffffffu, bar_wait(&parts_in, 0))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
      } else {
        __syncwarp();
        if (busy) epilogue(unit, bias, reinterpret_cast<const float *>(smem_raw + sums));
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
  attrs[1].val.clusterDim.x = (unsigned)P.split;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = P.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_slim<GATED>, P);
}

// Clusters of `split` CTAs, one CTA to an SM, that the device runs at a time (a cluster lies
// within one GPC, so fours leave some SMs over).  0: the query failed.
int active_clusters(int split) {
  static std::atomic<int> known[64][2];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int> &slot = known[dev][split == 4];
  int n = slot.load(std::memory_order_relaxed);
  if (n) return n;
  static std::atomic<uint64_t> ready{0};
  if (allow_smem(k_slim<false>, 224 * 1024, ready) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split * 64);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 190 * 1024;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, k_slim<false>, &cfg) != cudaSuccess) return 0;
  slot.store(n, std::memory_order_relaxed);
  return n;
}

struct SlimPlan {
  int nb, split, rounds;
};
// Weight rows of a tile: an even share, at most 128.  A share under 64 rows is widened by
// splitting K over a cluster (while a part keeps 8 chunks and the parts fit rank 0's memory).
SlimPlan plan(int T, int N, int64_t K, int np, int sms) {
  const int nk = (int)((K + 63) / 64);
  SlimPlan p;
  p.rounds = (N + sms * 128 - 1) / (sms * 128);
  p.split = 1;
  p.nb = (N + sms * p.rounds - 1) / (sms * p.rounds);
  while (p.rounds == 1 && p.split < 4 && p.nb < 64 && nk >= 16 * p.split && (2 * p.split - 1) * np * T <= 384) {
    // no more tiles than clusters run at a time: another wave would double the time
    const int clusters = active_clusters(2 * p.split);
    if (clusters < 1 || (N + clusters - 1) / clusters > 128) break;
    p.split *= 2;
    p.nb = (N + clusters - 1) / clusters;
  }
  p.nb = std::max(p.nb, 8);
  return p;
}

}  // namespace

// Time of the kernel in units of 128 bytes read by one SM (2.9 ns at its share of the copy
// rate): the weight rows and tokens of its tiles times their chunks, and the epilogue, about
// 15 units a token for each product and part of K (fitted to 330 products of 4 to 128 tokens).
int64_t slim_cost(int T, int N, int64_t K, bool gated, int sms) {
  const int np = gated ? 2 : 1;
  const SlimPlan p = plan(T, N, K, np, sms);
  return p.rounds * (int64_t)(np * p.nb + T) * ((K + 63) / 64) / p.split + 15 * np * p.split * T;
}

sfnn_status launch_slim(const SlimArgs &q, int sms, cudaStream_t s) {
  const bool gated = q.w1 != nullptr;
  const int np = gated ? 2 : 1;
  SlimParams P{};
  P.T = q.T;
  P.N = q.N;
  P.nk = (int)((q.K + 63) / 64);
  P.t8 = up_to(q.T, 8);
  P.t16 = up_to(q.T, 16);
  const SlimPlan shape = plan(q.T, q.N, q.K, np, sms);
  P.nb = shape.nb;
  P.split = shape.split;
  P.nb8 = up_to(P.nb, 8);
  P.m64 = P.split == 1 && P.nb <= 64;
  P.tiles = (q.N + P.nb - 1) / P.nb;
  P.up_col = gated ? up_to(P.t16, 32) : 0;  // tensor memory is read 32 columns at a time
  P.tmem_cols = 32;
  while (P.tmem_cols < P.up_col + up_to(P.t16, 32)) P.tmem_cols *= 2;
  const int chunk = (P.t8 + np * P.nb8) * 128;
  const int over = std::max(0, (P.m64 ? 8192 : 16384) - P.nb8 * 128);  // an MMA reads all its lanes' rows
  // All of shared memory in flight (timed in turn: 1 token, 4096 x 11008, 54.6 us; with 131 and 83
  // KB, so that the gate/up and the down kernel share an SM, 59.0; 37 tokens, 8192 x 28672, 0.89 of
  // the time).
  const int budget = 190 * 1024;
  const int parts = (P.split - 1) * np * P.T * 512;  // bytes of the other ranks' accumulators
  P.apart = parts <= 16 * 1024;
  P.kps = std::max(2, std::min(8, 24 * 1024 / chunk));
  P.stages = std::max(2, std::min(kMaxStages, (budget - (P.apart ? parts : 0)) / (P.kps * chunk)));
  const int stage_mem = P.stages * P.kps * chunk;
  const size_t smem = 1024 + std::max(stage_mem + over, P.apart ? stage_mem + parts : parts);
  P.early = q.early;
  P.bf16 = q.bf16;
  P.out32 = q.out32;
  P.bias = q.bias;
  P.out = q.out;
  P.ldo = q.ldo;
  P.err = q.err;
  if (!make_tensor_map(&P.x, q.x, 2, q.T, q.K, q.ldx, P.t8, 64, true) ||
      !make_tensor_map(&P.w0, q.w0, 2, q.N, q.K, q.ldw0, P.nb, 64, true) ||
      (gated && !make_tensor_map(&P.w1, q.w1, 2, q.N, q.K, q.ldw1, P.nb, 64, true)))
    return SFNN_ERR_CUDA;
  const int grid = P.split > 1 ? P.tiles * P.split : std::min(P.tiles, sms);
  const cudaError_t e = gated ? launch<true>(P, grid, smem, s) : launch<false>(P, grid, smem, s);
  return e == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
}

}  // namespace sfnn
