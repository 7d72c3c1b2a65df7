// few.cu -- the linear layer for few tokens (up to 1024; the rule is few_plan's cost against the square
// tiles of dense.cu, in linear.cu).
//
// What bounds it is the weights' bytes, and after them the tokens', which every CTA reads beside its
// weights.  So the weights lie on the MMA's M side, up to 256 rows a CTA (two M = 128 products that share
// the tokens' chunk in shared memory), the tokens on its N side, whose width goes by 16, and K is split over
// the CTAs of a cluster so that few wide tiles still fill the SMs.  The ranks then exchange their sums
// through distributed shared memory, each taking a share of the tokens, adds them in rank order and stores
// it -- the work at the end is split too.  A tile need not fill the 128 lanes: the rest of the A tile is
// whatever shared memory holds, and only reaches accumulator lanes nobody reads.  More tokens than 256 are
// tiles of their own, which read the same weights beside one another, through the L2.
//
// Measured (fp16, bias; the weights from memory): 4096 x 16384 1 token 26 us and 64 tokens 30 (the weights'
// bytes alone 20.5), 28672 x 7168 50 tokens onto fp32 82 (63), 4096 x 4096 1 token 12, 128 tokens 14 and
// 512 tokens 28 (a library's product 14, 10 and 15: its tiles share loads across SMs, these read the L2 at 11.7
// bytes a ns and exchange sums at the 15 bytes a clock of an SM's way to its cluster), 1024 x 1024 256 tokens 7.
//
// Sums that leave as fp32 are dealt to several accumulators (see kSegment in dense.cu), kMostDealt chunks to
// one at most: 128 steps of 16 products, each of which costs up to 2^-24 of the sum (measured, K = 28672: rms
// 2.2e-6 of the result at 50 tokens, whose accumulators take 28 chunks, 1.3e-6 with 16; without the limit 4.3e-6
// at 128 tokens, 8.5e-6 at 200 and 3.4e-5 at 1024).  Shapes that would need more are left to the square tiles,
// which add up 16 chunks at a time.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kThreads = 320;  // warp 0 loads, warp 1 issues the MMAs, warps 2-9 end: two for each 32 lanes
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;
constexpr int kRows = 256;     // weight rows of a tile, at most
constexpr int kTokens = 256;   // and tokens
constexpr int kMostTokens = 1024;
constexpr int kBudget = 200 * 1024;
constexpr int kApart = 40 * 1024;      // up to this, the exchange has memory of its own
constexpr int kExchange = 224 * 1024;  // and this is the most it may have
constexpr int kMostSmem = 226 * 1024;
constexpr int kDealt = 16;      // chunks of K that an accumulator of an fp32 result should hold ...
constexpr int kMostDealt = 32;  // ... and may

struct alignas(64) FewParams {
  CUtensorMap x, w;
  int T, N, nk;        // nk: 64-deep chunks of K
  int nb, nb8;         // weight rows of a tile; rounded up to 8
  int halves;          // of 128 rows
  int t8, t16;         // tokens of a tile, eights (rows loaded); rounded up to 16 (MMA N)
  int tt, tiles;       // tiles of tokens, which lie side by side for each tile of weight rows; tiles in all
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
  if (split > 1 && P.apart) cluster_arrive();  // this CTA has started: the others may write to it (waited for below)

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
            tma_load_2d(at + (uint32_t)c * chunk_bytes + x_bytes, &P.w, (k0 + c) * 64, t / P.tt * P.nb, &full[s]);
          for (int c = 0; c < kn; ++c) tma_load_2d(at + (uint32_t)c * chunk_bytes, &P.x, (k0 + c) * 64, t % P.tt * P.t8, &full[s]);
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
  const int turn = P.halves > 1 ? 16 : 32, first = P.halves > 1 ? 0 : set * 16;  // ... and its sixteens of tokens
  const bool busy = worker && half * 128 + quad * 32 < P.nb;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * P.accs * P.acc_cols);
  const int row_slots = P.halves * 128;
  // sums of this thread's weight row: tokens [t, t + 8) of its tile and, if `more`, the next eight
  auto sums = [&](int t, bool more, uint32_t g[16]) {
    __syncwarp();
    tm_ld8(lanes + (uint32_t)t, g);
    if (more) tm_ld8(lanes + (uint32_t)t + 8, g + 8);
#pragma unroll 1
    for (int a = 1; a < P.accs; ++a) {
      uint32_t h[16];
      tm_ld8(lanes + (uint32_t)(a * P.acc_cols + t), h);
      if (more) tm_ld8(lanes + (uint32_t)(a * P.acc_cols + t) + 8, h + 8);
      tm_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < 8 || more) g[i] = __float_as_uint(__uint_as_float(g[i]) + __uint_as_float(h[i]));
    }
    tm_wait_ld();
  };
  // The tokens [lo, hi) of tile t; `parts`: the other ranks' sums of them, [4 tokens][row][4].
  // (With each choice made value by value this was 67 instructions a value, and 40 us of 48 at 256 tokens,
  // 200 x 20000; eight tokens at a time 600 clocks for 140 instructions, most of it waiting.)
  auto finish_by = [&](auto by, int t, int lo, int hi, const float *parts) {
    constexpr int G = decltype(by)::value;
    const int col = t / P.tt * P.nb + row, t0 = t % P.tt * P.t8;
    const bool live = row < P.nb && col < P.N;
    const LinearEnd &E = P.end;
    const float bias = E.bias && live ? load16(E.bias, col, BF16) : 0.f;
    const int act = E.act;
    const bool res = E.res && live;
#pragma unroll 1
    for (int c = lo + first; c < hi; c += turn) {
      const int n = min(G, hi - c);
      float v[G], r[G];
      if (res) {  // on its way while the accumulators are read
        const int64_t at = (int64_t)(t0 + c) * E.ldres + col;
        if (P.out32) {
          const float *q = static_cast<const float *>(E.res) + at;
#pragma unroll
          for (int i = 0; i < G; ++i, q += E.ldres) r[i] = i < n ? *q : 0.f;
        } else {
          const uint16_t *q = static_cast<const uint16_t *>(E.res) + at;
#pragma unroll
          for (int i = 0; i < G; ++i, q += E.ldres) r[i] = i < n ? load16(q, 0, BF16) : 0.f;
        }
      }
      uint32_t g[16];
      sums(c, n > 8, g);
#pragma unroll
      for (int i = 0; i < G; ++i) v[i] = i < 8 || n > 8 ? __uint_as_float(g[i]) : 0.f;
      if (parts) {
        float own[G];
#pragma unroll
        for (int i = 0; i < G; ++i) own[i] = v[i], v[i] = 0.f;
        const float4 *from = reinterpret_cast<const float4 *>(parts) + (size_t)((c - lo) >> 2) * row_slots + row;
#pragma unroll 1
        for (int p = 0; p < split; ++p) {
          if (p == rank) {
#pragma unroll
            for (int i = 0; i < G; ++i) v[i] += own[i];
            continue;
          }
#pragma unroll
          for (int i = 0; i < G / 4; ++i)
            if (i < 2 || n > 8) {  // (tokens past the last of an eight: whatever is there)
              const float4 f = from[i * row_slots];
              v[4 * i] += f.x, v[4 * i + 1] += f.y, v[4 * i + 2] += f.z, v[4 * i + 3] += f.w;
            }
          from += (size_t)(P.share >> 2) * row_slots;
        }
      }
#pragma unroll
      for (int i = 0; i < G; ++i) v[i] += bias;
      if (act == SFNN_LINEAR_RELU) {
        if (E.slopes) {  // nb is a multiple of 32 then: a warp's columns are a word
          unsigned char *s = static_cast<unsigned char *>(E.slopes) + (t0 + c) * slope_row_bytes(P.N, act) + (col >> 5) * 4;
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const uint32_t word = __ballot_sync(0xffffffffu, live && !(v[i] <= 0.f));
            if (lane == 0 && live && i < n) *reinterpret_cast<uint32_t *>(s + i * slope_row_bytes(P.N, act)) = word;
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) v[i] = max_nan(v[i], 0.f);
      } else if (act != SFNN_LINEAR_NONE) {
        uint32_t code[G];
        act_values<G>(v, act, E.slopes != nullptr, code);
        if (E.slopes && live) {
          unsigned char *s = static_cast<unsigned char *>(E.slopes) + (t0 + c) * slope_row_bytes(P.N, act) + (int64_t)col * 2;
#pragma unroll
          for (int i = 0; i < G; ++i)
            if (i < n) *reinterpret_cast<uint16_t *>(s + i * slope_row_bytes(P.N, act)) = (uint16_t)code[i];
        }
      }
      if (res)
#pragma unroll
        for (int i = 0; i < G; ++i) v[i] += r[i];
      if (!live) continue;
      const int64_t at = (int64_t)(t0 + c) * P.ldo + col;
      if (P.out32) {
        float *o = static_cast<float *>(P.out) + at;
#pragma unroll
        for (int i = 0; i < G; ++i, o += P.ldo)
          if (i < n) *o = v[i];
      } else {
        uint16_t *o = static_cast<uint16_t *>(P.out) + at;
#pragma unroll
        for (int i = 0; i < G; i += 2, o += 2 * P.ldo) {
          const uint32_t two = pack16(v[i], v[i + 1], BF16);
          if (i < n) *o = (uint16_t)two;
          if (i + 1 < n) o[P.ldo] = (uint16_t)(two >> 16);
        }
      }
    }
  };
  auto finish = [&](int t, int lo, int hi, const float *parts) {
    // (eight at a time for one token: gelu 27.8 us with sixteens, 27.0 so, of 4096 x 16384)
    if (P.t8 > 8) finish_by(std::integral_constant<int, 16>{}, t, lo, hi, parts);
    else finish_by(std::integral_constant<int, 8>{}, t, lo, hi, parts);
  };
  auto tokens = [&](int t) { return min(P.t8, P.T - t % P.tt * P.t8); };
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
      if (busy) finish(t, 0, tokens(t), nullptr);
      tm_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty, 0));
    }
  }
  __syncwarp();
  if (split > 1) {
    // the same place in every CTA's shared memory
    const uint32_t place = stage0 - raw + (P.apart ? (uint32_t)P.stages * stage_bytes : 0u);
    // Every CTA has started before a sum is written to it, and where that goes into the stages, no load or MMA
    // touches those any more.  (The first is known long before it is asked for.)
    if (P.apart)
      cluster_wait();
    else
      cluster_sync_all();
    if (worker && busy && ok) {
      const int count = tokens(unit);
#pragma unroll 1
      for (int j = 1; j < split; ++j) {
        const int q = (rank + j) % split, lo = q * P.share, hi = min(count, lo + P.share);
        const uint32_t dst = cluster_addr(smem_raw, (uint32_t)q) + place +
                             (uint32_t)((rank < q ? rank : rank - 1) * (P.share >> 2) * row_slots + row) * 16u;
#pragma unroll 1
        for (int c = lo + first; c < hi; c += turn) {
          const bool more = hi - c > 8;
          uint32_t g[16];
          sums(c, more, g);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < 2 || more)
              asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               dst + (uint32_t)((((c - lo) >> 2) + i) * row_slots) * 16u),
                           "r"(g[4 * i]), "r"(g[4 * i + 1]), "r"(g[4 * i + 2]), "r"(g[4 * i + 3])
                           : "memory");
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // (also: no CTA ends while another still writes to it)
    if (worker && busy && ok && unit < P.tiles) {
      const int lo = rank * P.share, hi = min(tokens(unit), lo + P.share);
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

// Accumulators of an fp32 result, as far as tensor memory goes; `chunks`: the fewest of a rank, which every
// accumulator must get one of.
int accumulators(int chunks, int tokens, int halves) {
  return std::max(1, std::min({chunks, (chunks + kDealt - 1) / kDealt, 512 / (up_to(tokens, 32) * halves)}));
}

// One limit for every launch: set again, a lower one would take back the higher.
template <bool BF16>
cudaError_t allow() {
  static std::atomic<uint64_t> ready{0};
  return allow_smem(k_few<BF16>, kMostSmem, ready);
}

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
  if (allow<false>() != cudaSuccess) return 0;
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

// The shape with the least time (ns) of 1, 2, 4 and 8 CTAs to a cluster and a few widths of the tiles of
// tokens.  The time is a fit to 255 products of 1 to 1024 tokens, 64 to 28672 wide either way, each in every
// shape (off by 5 % on average; the shape it takes is 0.8 % slower than the best of them, the square tiles
// among them, at most 15 %).  The products of the fit have a bias and no activation; neither this cost nor that of
// the square tiles knows the epilogue.  A chunk of K costs the longest of one CTA's pace, the weights' bytes from memory
// and all bytes through the L2 (5.5 and 11.7 bytes a ns of all CTAs); then come the end by tokens and the
// exchange.  No one shape does for all: 4096 x 4096, 8 tokens, takes 21, 14 and 12 us with 1, 2 and 4 CTAs,
// 4096 x 16384 27 us with 1 and none wider than 2 fits; 256 tokens of 2048 x 8192 take 19 us as two tiles,
// 257 of 4096 x 12288 43 as three.  Against the square tiles: 257 tokens of 2048 x 2048 12 us to 15, of 4096
// x 12288 43 to 54, 400 of 4096 x 16384 60 to 58.  More than 1024 tokens are not looked at: there the square
// tiles, which read each byte for more products, lose by little at most (1000 of 1024 x 1024: 10 us to 14).
FewPlan few_plan(int T, int N, int64_t K, bool words, bool out32, int sms) {
  FewPlan best{};
  best.cost = 1e30;
  if (T > kMostTokens) return best;
  const int nk = (int)((K + 63) / 64), least = (T + kTokens - 1) / kTokens;
  for (int split = 1; split <= kMaxSplit; split *= 2) {
    if (split > 1 && nk < 2 * split) break;
    const int clusters = active_clusters(split, sms);
    if (clusters < 1) continue;
    for (int want = least; want <= 2 * least + 2; ++want) {
      FewPlan p;
      p.split = split;
      p.tn = up_to((T + want - 1) / want, 8);
      const int tt = (T + p.tn - 1) / p.tn;
      if (tt < want) break;
      const int64_t rounds = ((int64_t)tt * ((N + kRows - 1) / kRows) + clusters - 1) / clusters;
      if (rounds > 1 && split > 1) continue;
      const int64_t wide_tiles = std::max<int64_t>(1, clusters * rounds / tt);
      p.nb = std::max(16, up_to((int)((N + wide_tiles - 1) / wide_tiles), words ? 32 : 8));
      if (p.nb > kRows) continue;
      const int share = share_of(p.tn, split), halves = p.nb > 128 ? 2 : 1;
      if ((split - 1) * share * halves * 512 > kExchange) continue;
      const int rank_chunks = (nk + split - 1) / split;
      if (out32 && rank_chunks > kMostDealt * accumulators(nk / split, p.tn, halves)) continue;
      const double tiles = (double)((N + p.nb - 1) / p.nb) * tt, ctas = std::min<double>(tiles * split, sms);
      const double weights = std::max(1., ctas / tt / split) * split * p.nb;  // rows of a chunk that differ
      const double chunk = std::max({232 + 0.869 * p.nb + 0.718 * halves * up_to(p.tn, 16), weights * 128 / 5480,
                                     ctas * (p.nb + p.tn) * 128 / 11700});
      p.cost = 3640 + rounds * (rank_chunks * chunk + 15.2 * share * halves) +
               (split > 1 ? 432 + 284 * split + 13.6 * p.tn * halves : 0);
      if (p.cost < best.cost) best = p;
    }
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
  P.halves = P.nb > 128 ? 2 : 1;
  P.t8 = plan.tn;
  P.t16 = up_to(P.t8, 16);
  P.tt = (q.T + P.t8 - 1) / P.t8;
  P.tiles = (q.N + P.nb - 1) / P.nb * P.tt;
  P.split = plan.split;
  P.share = share_of(P.t8, P.split);
  P.acc_cols = up_to(P.t16, 32);
  P.accs = q.out32 ? accumulators(P.nk / P.split, P.t8, P.halves) : 1;
  P.tmem_cols = 32;
  while (P.tmem_cols < P.halves * P.accs * P.acc_cols) P.tmem_cols *= 2;
  const int chunk = (P.t8 + P.nb8) * 128;
  const int over = P.halves * 16384 - P.nb8 * 128;  // an MMA reads all its lanes' rows
  const int parts = (P.split - 1) * P.share * P.halves * 512;
  P.apart = parts <= kApart;
  // four chunks of every row at a time, 512 contiguous bytes of it, or as many as leave three stages
  // (28672 x 7168, one token: 120 us a chunk at a time, 82 with two, 69 with four; two where the work has
  // no second stage of four: no faster, 1024 x 1024 5.7 -> 6.1)
  const int room = kBudget - over - (P.apart ? parts : 0);
  P.kps = 4;
  while (P.kps > 1 && (P.kps > 2 ? 3 : 2) * P.kps * chunk > room) --P.kps;
  // No more stages than the work fills: what is left is the next launch's, whose CTAs then get ready beside
  // these (in a row of launches, 1 token: 2048 x 2048 7.4 -> 6.9 us, 512 x 2048 5.9 -> 5.3).
  const int rounds = P.split > 1 ? 1 : (P.tiles + sms - 1) / sms;
  const int loads = rounds * ((P.nk + P.split * P.kps - 1) / (P.split * P.kps));
  P.stages = std::max(1, std::min({kMaxStages, room / (P.kps * chunk), loads}));
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
  if (smem > kMostSmem || (P.bf16 ? allow<true>() : allow<false>()) != cudaSuccess) return SFNN_ERR_CUDA;
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
  return cudaLaunchKernelEx(&cfg, P.bf16 ? k_few<true> : k_few<false>, P) == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
}

}  // namespace sfnn
