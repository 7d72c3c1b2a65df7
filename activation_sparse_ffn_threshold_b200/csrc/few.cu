// few.cu -- the linear layer for few tokens (up to 256; the rule is few_plan's cost against the square
// tiles of dense.cu, in linear.cu).
//
// What bounds it is the weights' bytes, and after them the tokens', which every CTA reads beside its
// weights.  So the weights lie on the MMA's M side, up to 256 rows a CTA (two M = 128 products that share
// the tokens' chunk in shared memory), the tokens on its N side, and K is split over the CTAs of a cluster
// so that few wide tiles still fill the SMs.  The ranks then exchange their sums through distributed
// shared memory, each taking a share of the tokens, adds them in rank order and stores it -- the work at
// the end is split too.  A tile need not fill the 128 lanes: the rest of the A tile is whatever shared
// memory holds, and only reaches accumulator lanes nobody reads.
//
// Sums that leave as fp32 are dealt to several accumulators (see kSegment in dense.cu).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kThreads = 320;  // warp 0 loads, warp 1 issues the MMAs, warps 2-9 end: two for each 32 lanes
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;
constexpr int kRows = 256;     // weight rows of a tile, at most
constexpr int kBudget = 200 * 1024;
constexpr int kApart = 40 * 1024;      // up to this, the exchange has memory of its own
constexpr int kExchange = 224 * 1024;  // and this is the most it may have

struct alignas(64) FewParams {
  CUtensorMap x, w;
  int T, N, nk;        // nk: 64-deep chunks of K
  int nb, nb8, tiles;  // weight rows of a tile; rounded up to 8
  int halves;          // of 128 rows
  int t8, t16;         // T rounded up to 8 (rows loaded), to 16 (MMA N)
  int kps, stages;     // chunks a stage
  int split, share;    // CTAs of a cluster that share a tile's K; tokens that each of them ends
  int apart;           // the exchange's memory lies behind the stages (else in them)
  int accs, acc_cols;  // accumulators of a half, chunks dealt to them in turn; their columns
  int tmem_cols;
  int bf16, out32;
  void *out;
  int64_t ldo;
  LinearEnd end;
  int32_t *err;
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_few(const __grid_constant__ FewParams P) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty;
  __shared__ uint32_t tmem_slot;
  const uint32_t raw = smem_u32(smem_raw), stage0 = (raw + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, split = P.split;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / split, units = gridDim.x / split;
  const uint32_t x_bytes = (uint32_t)P.t8 * 128u, chunk_bytes = x_bytes + (uint32_t)P.nb8 * 128u;
  const uint32_t stage_bytes = chunk_bytes * (uint32_t)P.kps;
  const int k_lo = rank * P.nk / split, k_hi = (rank + 1) * P.nk / split;
  const int steps = (k_hi - k_lo + P.kps - 1) / P.kps;
  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      bar_init(&full[s], 1);
      bar_init(&empty[s], 1);
    }
    bar_init(&acc_full, 1);
    bar_init(&acc_empty, 8);
    bar_init_fence();
    fence_async_shared();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.x)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&P.w)) : "memory");
  }
  if (warp == 1) tm_alloc<1>(&tmem_slot, (uint32_t)P.tmem_cols);
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      pdl_wait();
      pdl_launch_dependents();
      int it = 0;
      bool ok = true;
      for (int t = unit; t < P.tiles && ok; t += units)
        for (int i = 0; i < steps; ++i, ++it) {
          const int s = it % P.stages, k0 = k_lo + i * P.kps, kn = min(P.kps, k_hi - k0);
          if (!bar_wait(&empty[s], (uint32_t)((it / P.stages) & 1) ^ 1u)) {
            ok = false;
            break;
          }
          bar_expect_tx(&full[s], (x_bytes + (uint32_t)P.nb * 128u) * (uint32_t)kn);
          const uint32_t at = stage0 + (uint32_t)s * stage_bytes;
          for (int c = 0; c < kn; ++c)
            tma_load_2d(at + (uint32_t)c * chunk_bytes + x_bytes, &P.w, (k0 + c) * 64, t * P.nb, &full[s]);
          for (int c = 0; c < kn; ++c) tma_load_2d(at + (uint32_t)c * chunk_bytes, &P.x, (k0 + c) * 64, 0, &full[s]);
        }
      for (int s = 0; s < P.stages && ok; ++s) {  // every load has been consumed before the CTA ends
        const int j = it - P.stages + s;
        if (j >= 0 && !bar_wait(&empty[j % P.stages], (uint32_t)((j / P.stages) & 1))) ok = false;
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = mma_desc_16(128, P.t16, BF16, 0, 0);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = unit; t < P.tiles && ok; t += units, ++n) {
        if (!bar_wait(&acc_empty, (uint32_t)(n & 1) ^ 1u)) {
          ok = false;
          break;
        }
        tm_fence_after();
        int acc = 0, round = 0;  // the chunk's accumulator; whether it holds sums already
        for (int i = 0; i < steps; ++i, ++it) {
          const int s = it % P.stages, kn = min(P.kps, k_hi - (k_lo + i * P.kps));
          if (!bar_wait(&full[s], (uint32_t)((it / P.stages) & 1))) {
            ok = false;
            break;
          }
          tm_fence_after();
          for (int c = 0; c < kn; ++c) {
            const uint32_t x = stage0 + (uint32_t)s * stage_bytes + (uint32_t)c * chunk_bytes, w = x + x_bytes;
            for (int h = 0; h < P.halves; ++h) {
              const uint32_t d = tmem + (uint32_t)((h * P.accs + acc) * P.acc_cols);
#pragma unroll
              for (uint32_t k = 0; k < 4; ++k)
                mma_16<1>(d, mat_desc(w + (uint32_t)h * 16384u + k * 32, 16, 1024), mat_desc(x + k * 32, 16, 1024), idesc,
                          round > 0 || k > 0);
            }
            if (++acc == P.accs) acc = 0, round = 1;
          }
          mma_commit(&empty[s]);
        }
        if (ok) mma_commit(&acc_full);
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  }
  __syncwarp();
  const bool worker = warp >= 2;
  const int quad = warp & 3, set = (warp - 2) >> 2;
  const int half = P.halves > 1 ? set : 0;            // this warp's rows ...
  const int row = half * 128 + quad * 32 + lane;
  const int turn = P.halves > 1 ? 8 : 16, first = P.halves > 1 ? 0 : set * 8;  // ... and its eights of tokens
  const bool busy = worker && half * 128 + quad * 32 < P.nb;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * P.accs * P.acc_cols);
  // eight tokens' sums of this thread's weight row
  auto sums8 = [&](int t, uint32_t g[8]) {
    __syncwarp();
    tm_ld8(lanes + (uint32_t)t, g);
#pragma unroll 1
    for (int a = 1; a < P.accs; ++a) {
      uint32_t h[8];
      tm_ld8(lanes + (uint32_t)(a * P.acc_cols + t), h);
      tm_wait_ld();
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = __float_as_uint(__uint_as_float(g[i]) + __uint_as_float(h[i]));
    }
    tm_wait_ld();
  };
  const int row_slots = P.halves * 128;
  // The tokens [lo, hi) of tile t; `parts`: the other ranks' sums of them.  (With each choice made value
  // by value this was 67 instructions a value, and 40 us of 48 at 256 tokens, 200 x 20000.)
  auto finish = [&](int t, int lo, int hi, const float *parts) {
    const int col = t * P.nb + row;
    const bool live = row < P.nb && col < P.N;
    const LinearEnd &E = P.end;
    const float bias = E.bias && live ? load16(E.bias, col, BF16) : 0.f;
    const int act = E.act;
    const bool res = E.res && live;
#pragma unroll 1
    for (int c = lo + first; c < hi; c += turn) {
      const int n = min(8, hi - c);
      float v[8], r[8];
      if (res) {  // on its way while the accumulators are read
        const int64_t at = (int64_t)c * E.ldres + col;
        if (P.out32) {
          const float *q = static_cast<const float *>(E.res) + at;
#pragma unroll
          for (int i = 0; i < 8; ++i, q += E.ldres) r[i] = i < n ? *q : 0.f;
        } else {
          const uint16_t *q = static_cast<const uint16_t *>(E.res) + at;
#pragma unroll
          for (int i = 0; i < 8; ++i, q += E.ldres) r[i] = i < n ? load16(q, 0, BF16) : 0.f;
        }
      }
      uint32_t g[8];
      sums8(c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(g[i]);
      if (parts) {
        float own[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) own[i] = v[i], v[i] = 0.f;
        const float *from = parts + (size_t)(c - lo) * row_slots + row;
#pragma unroll 1
        for (int p = 0; p < split; ++p) {
          if (p == rank) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += own[i];
            continue;
          }
          const float *q = from;
#pragma unroll
          for (int i = 0; i < 8; ++i, q += row_slots) v[i] += *q;  // (tokens past the last: whatever is there)
          from += (size_t)P.share * row_slots;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += bias;
      if (act == SFNN_LINEAR_RELU) {
        if (E.slopes) {  // nb is a multiple of 32 then: a warp's columns are a word
          unsigned char *s = static_cast<unsigned char *>(E.slopes) + c * slope_row_bytes(P.N, act) + (col >> 5) * 4;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t word = __ballot_sync(0xffffffffu, live && !(v[i] <= 0.f));
            if (lane == 0 && live && i < n) *reinterpret_cast<uint32_t *>(s + i * slope_row_bytes(P.N, act)) = word;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = max_nan(v[i], 0.f);
      } else if (act != SFNN_LINEAR_NONE) {
        uint32_t code[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act_value(v[i], act, E.slopes != nullptr, code[i]);
        if (E.slopes && live) {
          unsigned char *s = static_cast<unsigned char *>(E.slopes) + c * slope_row_bytes(P.N, act) + (int64_t)col * 2;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < n) *reinterpret_cast<uint16_t *>(s + i * slope_row_bytes(P.N, act)) = (uint16_t)code[i];
        }
      }
      if (res)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      if (!live) continue;
      const int64_t at = (int64_t)c * P.ldo + col;
      if (P.out32) {
        float *o = static_cast<float *>(P.out) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, o += P.ldo)
          if (i < n) *o = v[i];
      } else {
        uint16_t *o = static_cast<uint16_t *>(P.out) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, o += P.ldo)
          if (i < n) *o = (uint16_t)pack16(v[i], 0.f, BF16);
      }
    }
  };
  bool ok = true;
  if (worker) {
    pdl_wait();  // nothing is written, nor the residual read, before the kernel before has finished
    int n = 0;
    for (int t = unit; t < P.tiles; t += units, ++n) {
      ok = __all_sync(0xffffffffu, bar_wait(&acc_full, (uint32_t)(n & 1)));
      if (!ok) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        break;
      }
      __syncwarp();
      tm_fence_after();
      if (split > 1) break;  // one tile per cluster, joined below
      if (busy) finish(t, 0, P.T, nullptr);
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty, 0));
    }
  }
  __syncwarp();
  if (split > 1) {
    // the same place in every CTA's shared memory
    const uint32_t place = stage0 - raw + (P.apart ? (uint32_t)P.stages * stage_bytes : 0u);
    if (!P.apart) cluster_sync_all();  // no load or MMA touches the stages any more, in any CTA
    if (worker && busy && ok) {
#pragma unroll 1
      for (int j = 1; j < split; ++j) {
        const int q = (rank + j) % split, lo = q * P.share, hi = min(P.T, lo + P.share);
        const uint32_t dst = cluster_addr(smem_raw, (uint32_t)q) + place +
                             (uint32_t)(((rank < q ? rank : rank - 1) * P.share * row_slots + row) * 4);
#pragma unroll 1
        for (int c = lo + first; c < hi; c += turn) {
          uint32_t g[8];
          sums8(c, g);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < hi)
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + (uint32_t)((c + i - lo) * row_slots * 4)), "r"(g[i])
                           : "memory");
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // (also: no CTA ends while another still writes to it)
    if (worker && busy && ok && unit < P.tiles) {
      const int lo = rank * P.share, hi = min(P.T, lo + P.share);
      finish(unit, lo, hi, reinterpret_cast<const float *>(smem_raw + place));
    }
  }
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  if (warp == 1) tm_dealloc<1>(tmem, (uint32_t)P.tmem_cols);
}

int up_to(int v, int to) { return (v + to - 1) / to * to; }
// Tokens that a rank ends: whole eights, as tensor memory is read.
int share_of(int T, int split) { return up_to((T + split - 1) / split, 8); }

// Clusters of `split` CTAs, one CTA to an SM, that the device runs at a time (a cluster lies within one
// GPC).  0: the query failed.
int active_clusters(int split, int sms) {
  if (split == 1) return sms;
  static std::atomic<int> known[64][kMaxSplit + 1];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int> &slot = known[dev][split];
  int n = slot.load(std::memory_order_relaxed);
  if (n) return n;
  static std::atomic<uint64_t> ready{0};
  if (allow_smem(k_few<false>, 224 * 1024, ready) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split * 64);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kBudget;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, k_few<false>, &cfg) != cudaSuccess) return 0;
  slot.store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

// The shape with the least time (ns) of 1, 2, 4 and 8 CTAs to a cluster.  The time is a fit to 110 random
// products of 1 to 256 tokens, 64 to 28672 wide either way, each with every split: a chunk of K costs its
// weight rows, its tokens and its MMAs, whose times add up more than they overlap while the chunks in
// flight bound the rate; then the exchange, and the end by tokens.  It is off by 6 % on average, and the
// choice, dense.cu's tiles among its options (linear.cu), takes 1.2 % longer than the best.
FewPlan few_plan(int T, int N, int64_t K, bool words, int sms) {
  FewPlan best{};
  best.cost = INT64_MAX;
  if (T > 256) return best;
  const int nk = (int)((K + 63) / 64), t16 = up_to(T, 16);
  for (int split = 1; split <= kMaxSplit; split *= 2) {
    if (split > 1 && nk < 2 * split) break;
    const int clusters = active_clusters(split, sms);
    if (clusters < 1) continue;
    const int64_t rounds = ((int64_t)N + clusters * kRows - 1) / (clusters * kRows);
    if (rounds > 1 && split > 1) continue;
    FewPlan p;
    p.split = split;
    p.nb = std::max(16, up_to((int)((N + clusters * rounds - 1) / (clusters * rounds)), words ? 32 : 8));
    if (p.nb > kRows) continue;
    const int64_t chunks = (nk + split - 1) / split, share = share_of(T, split), wide = p.nb > 128 ? 2 : 1;
    if ((split - 1) * share * wide * 512 > kExchange) continue;
    p.cost = 3250 + rounds * chunks * (202000 + 2185 * p.nb + 315 * T + 538 * wide * t16) / 1000 + rounds * share * 20 * wide +
             (split > 1 ? 625 + 182 * split + 12 * T * wide : 0);
    if (p.cost < best.cost) best = p;
  }
  return best;
}

sfnn_status launch_few(const FewArgs &q, const FewPlan &plan, int sms, cudaStream_t s) {
  FewParams P{};
  P.T = q.T;
  P.N = q.N;
  P.nk = (int)((q.K + 63) / 64);
  P.nb = plan.nb;
  P.nb8 = up_to(P.nb, 8);
  P.tiles = (q.N + P.nb - 1) / P.nb;
  P.halves = P.nb > 128 ? 2 : 1;
  P.t8 = up_to(q.T, 8);
  P.t16 = up_to(q.T, 16);
  P.split = plan.split;
  P.share = share_of(q.T, P.split);
  P.acc_cols = up_to(P.t16, 32);
  P.accs = 1;
  // an fp32 result: no more than 64 sums of the tensor cores in one accumulator, as far as tensor memory goes
  const int nk = P.nk / P.split;
  if (q.out32) P.accs = std::max(1, std::min({nk, (nk + 15) / 16, 512 / (P.acc_cols * P.halves)}));
  P.tmem_cols = 32;
  while (P.tmem_cols < P.halves * P.accs * P.acc_cols) P.tmem_cols *= 2;
  const int chunk = (P.t8 + P.nb8) * 128;
  const int over = P.halves * 16384 - P.nb8 * 128;  // an MMA reads all its lanes' rows
  const int parts = (P.split - 1) * P.share * P.halves * 512;
  P.apart = parts <= kApart;
  // four chunks of every row at a time, 512 contiguous bytes of it, or as many as leave three stages
  // (28672 x 7168, one token: 120 us a chunk at a time, 82 with two, 69 with four)
  const int room = kBudget - over - (P.apart ? parts : 0);
  P.kps = 4;
  while (P.kps > 1 && (P.kps > 2 ? 3 : 2) * P.kps * chunk > room) --P.kps;
  P.stages = std::max(2, std::min(kMaxStages, room / (P.kps * chunk)));
  const int stage_mem = P.stages * P.kps * chunk;
  const size_t smem = 1024 + std::max(stage_mem + std::max(over, P.apart ? parts : 0), parts);
  P.bf16 = q.bf16;
  P.out32 = q.out32;
  P.out = q.out;
  P.ldo = q.ldo;
  P.end = *q.end;
  P.err = q.err;
  if (!make_tensor_map(&P.x, q.x, 2, q.T, q.K, q.ldx, P.t8, 64, true) ||
      !make_tensor_map(&P.w, q.w, 2, q.N, q.K, q.ldw, P.nb, 64, true))
    return SFNN_ERR_CUDA;
  static std::atomic<uint64_t> ready[2];
  auto kernel = P.bf16 ? k_few<true> : k_few<false>;
  if (smem > 226 * 1024 || allow_smem(kernel, 226 * 1024, ready[P.bf16]) != cudaSuccess) return SFNN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.split > 1 ? P.tiles * P.split : std::min(P.tiles, sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = (unsigned)P.split;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = P.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
}

}  // namespace sfnn
