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
// (TMA, 128-byte swizzle), warp 1 of the pair's first CTA issues the MMAs, the others (8, or
// 16 for fp32 results) run the epilogue of the tile before out of the other half of tensor memory (2 x 256 columns).
// Plain stores also have tiles of 512 x 256 (TALL, at the kernel).
//
// Measured (4096 x 11008 bf16, 4096 tokens): forward and backward 2.2 ms in a graph, 2.36 before the
// tall tiles (1.5 PFLOP/s; a library product holds 1.39 for long under the power cap).  The tensor
// pipe is busy 57 to 77 % of a kernel's cycles alone with square tiles.  What it waits for there: the
// last round of tiles, and L2.
//
// Every wait is bounded (about a second); one that runs out latches SFNN_ERR_TIMEOUT and the
// kernel leaves in order: its loads have landed by then, tensor memory is freed.
#include <algorithm>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

// Epilogue warps: 16 for fp32 results, which read and write most and add up segments besides (8192 tokens, 64 ->
// 8192 onto an fp32 residual 226 us with 8, 191 with 16; 4096, 4096 -> 16384 477 and 457).  8 for the others,
// whose epilogue hides behind a ring of 6 chunks (16-bit residual 107 and 114 us, none 46 and 50).
// 16 warps leave 96 registers a thread, and tiles of 256 columns, with 64 sums in each, spill: 1.5 KB of stores and
// as much of loads a thread, in the epilogue.
template <int EPI>
constexpr int kEpiWarps = EPI == kEpiLinear32 ? 16 : 8;
template <int EPI>
constexpr int kThreads = 64 + 32 * kEpiWarps<EPI>;
// K chunks in flight; the backward epilogue's saved values take one's place (below), as do 16 warps' panels
template <int EPI>
constexpr int kStagesOf = EPI == kEpiDGated || EPI == kEpiDGated8 || kEpiWarps<EPI> == 16 ? 5 : 6;
constexpr int kMaxStages = 6;
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

// ---------------------------------------------------------------- staging
// An accumulator lane is a row, so a thread's values lie along a row, and 32 threads writing
// 16 bytes each would touch 32 lines an instruction (measured: 9 to 17 us for one tile's
// epilogue).  A warp's values pass through shared memory instead, 64 bytes of each of its 32
// rows at a time: written by row, read (and stored) with 4 lanes to a row.  The 16-byte
// pieces of row r are rotated by (r / 2) % 4, so neither side has bank conflicts.
constexpr uint32_t kPanel = 2048;      // 32 rows x 64 bytes
template <int EPI>  // a warp's panels: two, and two more for the saved values that come in
constexpr uint32_t kWarpPanels = EPI == kEpiDGated || EPI == kEpiDGated8 ? 4 * kPanel : 2 * kPanel;
__device__ __forceinline__ uint32_t panel_at(uint32_t panel, int row, int piece) {
  return panel + (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4 &v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// 64 bytes of this lane's row, to `base` (the warp's first row) + row * ld bytes for the rows
// and 16-byte pieces that exist.  The whole warp; the panel is free again afterwards.
__device__ __forceinline__ void panel_out(uint32_t panel, const uint4 w[4], unsigned char *base, int64_t ld, int rows,
                                          int pieces) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) sts16(panel_at(panel, lane, j), w[j]);
  __syncwarp();
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = lds16(panel_at(panel, i * 8 + (lane >> 2), lane & 3));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 8 + (lane >> 2), piece = lane & 3;
    if (row < rows && piece < pieces) *reinterpret_cast<uint4 *>(base + row * ld + piece * 16) = v[i];
  }
}
// Two of them at a time, through two panels: half the waits.
__device__ __forceinline__ void panels_out(uint32_t panel, const uint32_t a[16], unsigned char *pa, const uint32_t b[16],
                                           unsigned char *pb, int64_t ld, int rows, int pieces) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sts16(panel_at(panel, lane, j), make_uint4(a[4 * j], a[4 * j + 1], a[4 * j + 2], a[4 * j + 3]));
    sts16(panel_at(panel + kPanel, lane, j), make_uint4(b[4 * j], b[4 * j + 1], b[4 * j + 2], b[4 * j + 3]));
  }
  __syncwarp();
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = panel_at(panel, i * 8 + (lane >> 2), lane & 3);
    v[i] = lds16(at);
    v[4 + i] = lds16(at + kPanel);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 8 + (lane >> 2), piece = lane & 3;
    if (row < rows && piece < pieces) {
      *reinterpret_cast<uint4 *>(pa + row * ld + piece * 16) = v[i];
      *reinterpret_cast<uint4 *>(pb + row * ld + piece * 16) = v[4 + i];
    }
  }
}
// The way in: request 64 bytes of each of the warp's rows (zeros where none exist) into a
// panel, without waiting (cp.async) ...
__device__ __forceinline__ void panel_request(uint32_t panel, const unsigned char *base, int64_t ld, int rows, int pieces) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i * 8 + (lane >> 2), piece = lane & 3;
    const bool there = row < rows && piece < pieces;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(panel_at(panel, row, piece)),
                 "l"(there ? base + row * ld + piece * 16 : base), "r"(there ? 16 : 0)
                 : "memory");
  }
}
// ... and, once it is there, N 16-byte pieces of this lane's row from piece j on.
template <int N>
__device__ __forceinline__ void panel_row(uint32_t panel, int j, uint32_t w[4 * N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint4 v = lds16(panel_at(panel, threadIdx.x & 31, j + i));
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
}

__device__ __forceinline__ void words_to(uint4 w[4], const uint32_t a[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
}
// 32 values as 16-bit elements.
__device__ __forceinline__ void pack32(uint4 w[4], const float v[32], bool bf16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i].x = pack16(v[8 * i], v[8 * i + 1], bf16);
    w[i].y = pack16(v[8 * i + 2], v[8 * i + 3], bf16);
    w[i].z = pack16(v[8 * i + 4], v[8 * i + 5], bf16);
    w[i].w = pack16(v[8 * i + 6], v[8 * i + 7], bf16);
  }
}
// ---------------------------------------------------------------- epilogues
// Each thread owns one row of the tile (its tensor-memory lane) and a half of the tile's
// columns; a warp owns 32 rows from `row0` on and stores them through its `panel`s.

template <bool bf16, int width>
__device__ __forceinline__ void epi_store(const DenseParams &P, const Unit &Q, uint32_t taddr, int64_t row0, int n0,
                                          uint32_t panel) {
  const bool parts = Q.split > 1;
  const int rows = (int)min((int64_t)32, Q.M - row0);
  // relu: the hidden layer, whose rows are padded to 8 columns
  const int end = Q.relu ? (Q.N + 7) / 8 * 8 : Q.N;
  const bool wide = Q.out32 || parts;
  const int64_t ld = (parts ? (int64_t)Q.N : Q.ldo) * (wide ? 4 : 2);
  unsigned char *base = parts ? reinterpret_cast<unsigned char *>(Q.parts) + ((int64_t)Q.part * Q.M + row0) * ld
                              : static_cast<unsigned char *>(Q.out) + row0 * ld;
#pragma unroll 1
  for (int c = 0; c < width; c += 32) {
    const int cols = end - (n0 + c);
    if (rows <= 0 || cols <= 0) break;  // (the whole warp)
    uint32_t raw[32];
    float v[32];
    __syncwarp();
    tm_ld32(taddr + c, raw);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
    if (Q.relu) {
      const int col = n0 + c + (int)(threadIdx.x & 31);
      const float own = P.bias && col < Q.N ? load16(P.bias, col, bf16) : 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[i] += __shfl_sync(0xffffffffu, own, i);
        v[i] = v[i] < 0.f ? 0.f : v[i];
      }
    }
    if (wide) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = make_uint4(__float_as_uint(v[16 * h + 4 * j]), __float_as_uint(v[16 * h + 4 * j + 1]),
                            __float_as_uint(v[16 * h + 4 * j + 2]), __float_as_uint(v[16 * h + 4 * j + 3]));
        panel_out(panel + h * kPanel, w, base + (n0 + c + 16 * h) * 4, ld, rows, (cols - 16 * h + 3) / 4);
      }
    } else {
      uint4 w[4];
      pack32(w, v, bf16);
      panel_out(panel + ((c >> 5) & 1) * kPanel, w, base + (n0 + c) * 2, ld, rows, (cols + 7) / 8);
    }
  }
}

__device__ __forceinline__ void words32_out(uint32_t panel, const float *v, unsigned char *base, int64_t ld, int rows,
                                            int cols) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = make_uint4(__float_as_uint(v[16 * h + 4 * j]), __float_as_uint(v[16 * h + 4 * j + 1]),
                        __float_as_uint(v[16 * h + 4 * j + 2]), __float_as_uint(v[16 * h + 4 * j + 3]));
    panel_out(panel + h * kPanel, w, base + 64 * h, ld, rows, (cols - 16 * h + 3) / 4);
  }
}

// The same of a tall tile, whose sums are in registers (neither parts of K nor a hidden layer's ReLU).
template <bool bf16, int width>
__device__ __forceinline__ void epi_store_sums(const Unit &Q, int64_t row0, int n0, uint32_t panel, float (&sum)[width]) {
  const int rows = (int)min((int64_t)32, Q.M - row0);
  const int64_t ld = Q.ldo * (Q.out32 ? 4 : 2);
  unsigned char *base = static_cast<unsigned char *>(Q.out) + row0 * ld;
#pragma unroll
  for (int c = 0; c < width; c += 32) {
    const int cols = Q.N - (n0 + c);
    if (rows <= 0 || cols <= 0) break;  // (the whole warp)
    if (Q.out32) {
      words32_out(panel, sum + c, base + (int64_t)(n0 + c) * 4, ld, rows, cols);
    } else {
      uint4 w[4];
      pack32(w, sum + c, bf16);
      panel_out(panel + ((c >> 5) & 1) * kPanel, w, base + (int64_t)(n0 + c) * 2, ld, rows, (cols + 7) / 8);
    }
  }
}

// The pair's tile holds 128 neurons: gate columns 0..127, up columns 128..255.  This
// warp takes 64 of them from n0 on (one act8 block); its first panel holds their biases.
template <bool bf16, class Done>
__device__ __forceinline__ void epi_gated(const DenseParams &P, const Unit &Q, uint32_t tgate, int64_t row0, int n0,
                                          uint32_t panel, Done done) {
  const int lane = threadIdx.x & 31;
  const int rows = (int)min((int64_t)32, Q.M - row0);
  const int cols = (int)min((int64_t)64, Q.ldo - n0);  // writable columns of H (a multiple of 8)
  float r[64], u[64];
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    uint32_t a[32], b[32];
    __syncwarp();
    tm_ld32(tgate + c, a);
    tm_ld32(tgate + 128 + c, b);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const uint4 q = lds16(panel + (uint32_t)(c + i) * 4u);  // biases (zeros without one)
      const uint32_t bias[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float g = __uint_as_float(a[i + j]) + __uint_as_float(bias[j]);
        r[c + i + j] = g < 0.f ? 0.f : g;  // NaN stays NaN
        u[c + i + j] = __uint_as_float(b[i + j]);
      }
    }
  }
  done();  // the accumulators are free
  if (rows <= 0 || cols <= 0) return;  // (the whole warp)
  uint4 w[4];
  if (P.save != SFNN_SAVE_NONE) {  // whole blocks: code rows are padded to 64 columns
    const bool full = P.save == SFNN_SAVE_FULL;
    uint32_t rt = 0, ut = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      rt = max(rt, __float_as_uint(r[i]) & 0x7fffffffu);
      ut = max(ut, __float_as_uint(u[i]) & 0x7fffffffu);
    }
    auto scales = [&](float sr, float su) {
      if (lane < rows) {
        P.rs[(row0 + lane) * P.lds + (n0 >> 6)] = sr;
        P.us[(row0 + lane) * P.lds + (n0 >> 6)] = su;
      }
    };
    if (full) {
      const Code16Scale sr = code16_scale(rt, kHalfR), su = code16_scale(ut, kHalfU);
      scales(sr.scale, su.scale);
      unsigned char *rp = static_cast<unsigned char *>(P.r) + (row0 * P.ldr + n0) * 2;
      unsigned char *up = static_cast<unsigned char *>(P.u) + (row0 * P.ldr + n0) * 2;
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t q[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = code16_pair_relu(r[c + 2 * i], r[c + 2 * i + 1], sr.to);
        words_to(w, q);
        panel_out(panel, w, rp + c * 2, P.ldr * 2, rows, 4);
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = code16_pair(u[c + 2 * i], u[c + 2 * i + 1], su.to);
        words_to(w, q);
        panel_out(panel + kPanel, w, up + c * 2, P.ldr * 2, rows, 4);
      }
    } else {
      const Act8Scale sr = act8_scale(rt, 255.f), su = act8_scale(ut, 127.f);
      scales(sr.scale, su.scale);
      auto codes = [&](const float *v, float inv, bool relu) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float *a = v + 16 * i + 4 * j;
            q[j] = relu ? act8_codes<true>(a[0], a[1], a[2], a[3], inv) : act8_codes<false>(a[0], a[1], a[2], a[3], inv);
            if (relu) {
              uint32_t pos = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) pos |= a[k] > 0.f ? 1u << (8 * k) : 0u;
              q[j] = act8_lift(q[j], pos);
            }
          }
          w[i] = make_uint4(q[0], q[1], q[2], q[3]);
        }
      };
      codes(r, sr.inv, true);
      panel_out(panel, w, static_cast<unsigned char *>(P.r) + row0 * P.ldr + n0, P.ldr, rows, 4);
      codes(u, su.inv, false);
      panel_out(panel + kPanel, w, static_cast<unsigned char *>(P.u) + row0 * P.ldr + n0, P.ldr, rows, 4);
    }
  }
  unsigned char *hp = static_cast<unsigned char *>(Q.out) + (row0 * Q.ldo + n0) * 2;
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) r[c + i] *= u[c + i];
    pack32(w, r + c, bf16);
    panel_out(panel + (c >> 5) * kPanel, w, hp + c * 2, Q.ldo * 2, rows, (cols - c) / 8);
  }
}

// Sums over the warp's 32 rows of 32 columns of fp32 values, of which a lane holds its row's:
// lane c gets column c's.  The values pass through the two panels (columns 0..15, 16..31), whose
// rows the lower and the upper lanes read in another order, so that they meet in no bank.
__device__ __forceinline__ float column_sums(uint32_t panel, const uint32_t v[32]) {
  const int lane = threadIdx.x & 31, c = lane & 15, up = lane >> 4;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    sts16(panel_at(panel + (j >> 2) * kPanel, lane, j & 3), make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
  __syncwarp();
  float sum = 0.f;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];"
                 : "=f"(f)
                 : "r"(panel_at(panel + up * kPanel, i ^ up, c >> 2) + (uint32_t)((c & 3) * 4)));
    sum += f;
  }
  return sum;
}

// Request the saved relu(G) and U of a warp's rows into the panels `in` and `in` + 1: 64 bytes
// a row of each, 32 codes of 16 bits or 64 of 8; a lane keeps its row's two scales.
template <bool CODES8>
__device__ __forceinline__ void saved_request(const DenseParams &P, const Unit &Q, int64_t row0, int n0, uint32_t in,
                                              float2 &scales) {
  const int rows = (int)min((int64_t)32, Q.M - row0), lane = threadIdx.x & 31;
  constexpr int E = CODES8 ? 1 : 2;
  const int pieces = n0 < Q.N ? 4 : 0;  // code rows are padded to 64 columns
  const int64_t at = pieces > 0 && rows > 0 ? (row0 * P.ldr + n0) * E : 0;
  panel_request(in, static_cast<const unsigned char *>(P.r) + at, P.ldr * E, rows, pieces);
  panel_request(in + kPanel, static_cast<const unsigned char *>(P.u) + at, P.ldr * E, rows, pieces);
  cp_async_commit();
  scales = make_float2(0.f, 0.f);
  if (pieces && lane < rows)
    scales = make_float2(__ldg(P.rs + (row0 + lane) * P.lds + (n0 >> 6)), __ldg(P.us + (row0 + lane) * P.lds + (n0 >> 6)));
}

// relu(G) and U of 32 columns of a row, as they were saved: 8 words of four codes or 16 of
// two, and the scales.  They are widened where they are used and not before: held as floats
// they cost the kernel its registers, and a spill here misses L1 (shared memory leaves it
// next to nothing; measured: 13 to 20 us a tile instead of 3 to 5).
template <bool CODES8>
struct SavedWords {
  uint32_t r[CODES8 ? 8 : 16], u[CODES8 ? 8 : 16];
  float rs, r0, us;
  __device__ __forceinline__ void set_scales(float sr, float su) {
    if (CODES8) {
      rs = sr == 0.f ? __uint_as_float(1u) : sr;  // a lifted code of a block whose scale is zero keeps its neuron on
      r0 = -8388608.f * rs;
      us = su;
    } else {
      rs = code16_from(sr);
      us = code16_from(su);
    }
  }
  // columns 2 i and 2 i + 1
  __device__ __forceinline__ void get(int i, float2 &rv, float2 &uv) const {
    if (CODES8) {
      // a code as a float: its bits under the exponent of 2^23, less 2^23 (and half the range if signed)
      const uint32_t a = r[i >> 1], b = u[i >> 1] ^ 0x80808080u, lo = 0x7440u + 2u * (i & 1), hi = lo + 1;
      constexpr float kZero = 8388608.f + 128.f;
      rv.x = fmaf(__uint_as_float(__byte_perm(a, 0x4b000000u, lo)), rs, r0);
      rv.y = fmaf(__uint_as_float(__byte_perm(a, 0x4b000000u, hi)), rs, r0);
      uv.x = (__uint_as_float(__byte_perm(b, 0x4b000000u, lo)) - kZero) * us;
      uv.y = (__uint_as_float(__byte_perm(b, 0x4b000000u, hi)) - kZero) * us;
    } else {
      rv = code16_values_relu(r[i], rs);
      uv = code16_values(u[i], us);
    }
  }
};

// 32 columns of dH: H, dU and dG.
template <bool CODES8, bool bf16>
__device__ __forceinline__ void dgated32(const DenseParams &P, const Unit &Q, uint32_t taddr, int64_t row0, int n0,
                                         SavedWords<CODES8> &v, uint32_t panel) {
  const int lane = threadIdx.x & 31, rows = (int)min((int64_t)32, Q.M - row0), pieces = (Q.N - n0) / 8;
  if (rows <= 0 || pieces <= 0) return;  // (the whole warp)
  const int64_t at = (row0 * Q.ldo + n0) * 2, ld = Q.ldo * 2;
  uint32_t h[16], du[16], dg[32];
  {
    __syncwarp();
    tm_ld32(taddr, dg);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float2 r, u;
      v.get(i, r, u);
      const float x = __uint_as_float(dg[2 * i]), y = __uint_as_float(dg[2 * i + 1]);
      h[i] = pack16(r.x * u.x, r.y * u.y, bf16);
      du[i] = pack16(x * r.x, y * r.y, bf16);
      // r is 0 where the gate is off (and in rows past M), NaN in a block that is not finite
      dg[2 * i] = __float_as_uint(r.x > 0.f ? x * u.x : r.x);
      dg[2 * i + 1] = __float_as_uint(r.y > 0.f ? y * u.y : r.y);
    }
  }
  panels_out(panel, h, static_cast<unsigned char *>(Q.out) + at, du, static_cast<unsigned char *>(P.du) + at, ld, rows,
             pieces);
  if (P.colpart) {  // of dG before it is rounded
    const float sum = column_sums(panel, dg);
    if (n0 + lane < Q.N) P.colpart[(row0 >> 5) * Q.N + n0 + lane] = sum;
  }
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = pack16(__uint_as_float(dg[8 * i + 2 * j]), __uint_as_float(dg[8 * i + 2 * j + 1]), bf16);
    w[i] = make_uint4(q[0], q[1], q[2], q[3]);
  }
  panel_out(panel, w, static_cast<unsigned char *>(P.dg) + at, ld, rows, pieces);
}

// `width` columns of dH from n0 on; the first saved piece has been requested.
template <bool CODES8, bool bf16, int width>
__device__ __forceinline__ void epi_dgated(const DenseParams &P, const Unit &Q, uint32_t taddr, int64_t row0, int n0,
                                           float2 scales, uint32_t panel) {
  const uint32_t in = panel + 2 * kPanel;
#pragma unroll 1
  for (int c = 0; c < width; c += 32) {
    const bool first = !CODES8 || (c & 32) == 0, last = !CODES8 || (c & 32);  // of a saved piece
    SavedWords<CODES8> v;
    v.set_scales(scales.x, scales.y);
    if (first) {
      cp_async_wait<0>();
      __syncwarp();
    }
    const int piece = CODES8 && (c & 32) ? 2 : 0;
    panel_row<CODES8 ? 2 : 4>(in, piece, v.r);
    panel_row<CODES8 ? 2 : 4>(in + kPanel, piece, v.u);
    if (last && c + 32 < width) {
      __syncwarp();  // every lane has its row
      saved_request<CODES8>(P, Q, row0, n0 + c + 32, in, scales);
    }
    dgated32<CODES8, bf16>(P, Q, taddr + c, row0, n0 + c, v, panel);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- the linear layer's epilogue
// The residual: 32 columns of a warp's rows come in as panels go out (a row's 64 bytes by 4 lanes), or,
// where rows do not consist of 16-byte pieces, a column a lane.  16-bit values wait in registers,
// requested a piece ahead; an fp32 result has its sums there.
template <bool WIDE>
struct ResPiece {
  uint4 w[WIDE ? 1 : 4];
};
__device__ __forceinline__ uint32_t res_half(const LinearEnd &E, const Unit &Q, int64_t row0, int col, int rows, int r) {
  const int lane = threadIdx.x & 31;
  if (r >= rows || col + lane >= Q.N) return 0u;
  return static_cast<const uint16_t *>(E.res)[(row0 + r) * E.ldres + col + lane];
}
template <int ESIZE>
__device__ __forceinline__ uint4 res_word(const LinearEnd &E, const Unit &Q, int64_t row0, int col, int rows, int i) {
  const int lane = threadIdx.x & 31, row = (i & 3) * 8 + (lane >> 2), c = col + ((i >> 2) * 4 + (lane & 3)) * (16 / ESIZE);
  const unsigned char *base = static_cast<const unsigned char *>(E.res) + row0 * E.ldres * ESIZE;
  if (row < rows && c < Q.N) return *reinterpret_cast<const uint4 *>(base + (row * E.ldres + c) * ESIZE);
  return make_uint4(0, 0, 0, 0);
}
template <bool WIDE>
__device__ __forceinline__ void res_request(const LinearEnd &E, const Unit &Q, int64_t row0, int col, int rows,
                                            ResPiece<WIDE> &p) {
  if (WIDE || !E.res) return;
  if (E.vec_res) {
#pragma unroll
    for (int i = 0; i < (WIDE ? 0 : 4); ++i) p.w[i] = res_word<2>(E, Q, row0, col, rows, i);
  } else {
#pragma unroll
    for (int i = 0; i < (WIDE ? 0 : 4); ++i) {
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = res_half(E, Q, row0, col, rows, 8 * i + j);
      p.w[i] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
  }
}
// Added to this lane's row of 32 columns.
template <bool bf16, bool WIDE>
__device__ __forceinline__ void res_add(const LinearEnd &E, const Unit &Q, int64_t row0, int col, int rows,
                                        const ResPiece<WIDE> &p, uint32_t panel, float *v) {
  if (!E.res) return;
  const int lane = threadIdx.x & 31;
  __syncwarp();
  if (!WIDE && !E.vec_res) {  // a column, staged as 32 bits
#pragma unroll
    for (int i = 0; i < (WIDE ? 0 : 4); ++i) {
      const uint32_t u[4] = {p.w[i].x, p.w[i].y, p.w[i].z, p.w[i].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = unpack16(u[j / 2], bf16);
        const uint32_t at = panel_at(panel + (lane >> 4) * kPanel, 8 * i + j, (lane & 15) >> 2) + (lane & 3) * 4;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(j % 2 ? f.y : f.x) : "memory");
      }
    }
  } else if (!E.vec_res) {  // the same, 16 rows requested together
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 16) {
      float f[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        f[r] = 0.f;
        if (r0 + r < rows && col + lane < Q.N) {
          const int64_t i = (row0 + r0 + r) * E.ldres + col + lane;
          f[r] = static_cast<const float *>(E.res)[i];
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t at = panel_at(panel + (lane >> 4) * kPanel, r0 + r, (lane & 15) >> 2) + (lane & 3) * 4;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(f[r]) : "memory");
      }
    }
  } else if (WIDE) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = res_word<4>(E, Q, row0, col, rows, 4 * h + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) sts16(panel_at(panel + h * kPanel, i * 8 + (lane >> 2), lane & 3), w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < (WIDE ? 0 : 4); ++i) sts16(panel_at(panel, i * 8 + (lane >> 2), lane & 3), p.w[i]);
  }
  __syncwarp();
  if (WIDE || !E.vec_res) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint4 w = lds16(panel_at(panel + (j >> 2) * kPanel, lane, j & 3));
      v[4 * j] += __uint_as_float(w.x), v[4 * j + 1] += __uint_as_float(w.y);
      v[4 * j + 2] += __uint_as_float(w.z), v[4 * j + 3] += __uint_as_float(w.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 w = lds16(panel_at(panel, lane, j));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16(u[i], bf16);
        v[8 * j + 2 * i] += f.x, v[8 * j + 2 * i + 1] += f.y;
      }
    }
  }
}
// 32 columns of this lane's row, value by value: rows that do not consist of 16-byte pieces.
template <bool bf16, bool WIDE>
__device__ __forceinline__ void ragged_out(const Unit &Q, int64_t row0, int col, int rows, uint32_t panel, const float *v) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    sts16(panel_at(panel + (j >> 2) * kPanel, lane, j & 3),
          make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                     __float_as_uint(v[4 * j + 3])));
  __syncwarp();
  if (col + lane >= Q.N) return;
#pragma unroll 8
  for (int r = 0; r < rows; ++r) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];"
                 : "=f"(f)
                 : "r"(panel_at(panel + (lane >> 4) * kPanel, r, (lane & 15) >> 2) + (uint32_t)((lane & 3) * 4)));
    const int64_t i = (row0 + r) * Q.ldo + col + lane;
    if (WIDE)
      static_cast<float *>(Q.out)[i] = f;
    else
      static_cast<uint16_t *>(Q.out)[i] = (uint16_t)pack16(f, 0.f, bf16);
  }
}
// Two columns' biases to each of a piece's first 16 lanes (zeros past the last), requested a piece ahead and
// handed round.  (A column's own to each lane is twice the shuffles: 1.5 us of a tile's 5; all of them read
// by every lane 2.7.)
__device__ __forceinline__ uint32_t bias_request(const LinearEnd &E, int col, int N) {
  if (!E.bias) return 0u;
  const uint16_t *p = static_cast<const uint16_t *>(E.bias);
  const int c = col + 2 * ((int)threadIdx.x & 15);
  return (c < N ? __ldg(p + c) : 0u) | (c + 1 < N ? (uint32_t)__ldg(p + c + 1) << 16 : 0u);
}

// One 32-column piece of the tile, whose sums are in v; `bits` of a ReLU's slopes for the caller to keep.
template <bool bf16, int width, bool WIDE>
__device__ __forceinline__ void linear32(const DenseParams &P, const Unit &Q, int64_t row0, int n0, int c, int rows,
                                         uint32_t panel, ResPiece<WIDE> &piece, uint32_t &bias, float *v, uint32_t &word) {
  const LinearEnd &E = P.end;
  const int lane = threadIdx.x & 31, col = n0 + c, cols = Q.N - col;
  if (Q.split > 1) {  // sums of a part of K, rows of N rounded up to 4
    const int64_t ld = (Q.N + 3) / 4 * 16;
    words32_out(panel, v, reinterpret_cast<unsigned char *>(Q.parts) + ((int64_t)Q.part * Q.M + row0) * ld + (int64_t)col * 4,
                ld, rows, cols);
    return;
  }
  if (E.bias) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 f = unpack16(__shfl_sync(0xffffffffu, bias, i), bf16);
      v[2 * i] += f.x, v[2 * i + 1] += f.y;
    }
    if (c + 32 < width) bias = bias_request(E, col + 32, Q.N);
  }
  if (E.act == SFNN_LINEAR_RELU) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      word |= v[i] <= 0.f ? 0u : 1u << i;
      v[i] = max_nan(v[i], 0.f);
    }
  } else if (E.act != SFNN_LINEAR_NONE) {
    uint32_t q[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t code[16];
      act_values<16>(v + 16 * h, E.act, E.slopes != nullptr, code);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[8 * h + i] = __byte_perm(code[2 * i], code[2 * i + 1], 0x5410);
    }
    if (E.slopes) {
      uint4 w[4];
      words_to(w, q);
      const int64_t ld = slope_row_bytes(Q.N, E.act);
      panel_out(panel, w, static_cast<unsigned char *>(E.slopes) + row0 * ld + (int64_t)col * 2, ld, rows, 4);
    }
  }
  res_add<bf16, WIDE>(E, Q, row0, col, rows, piece, panel, v);
  if (c + 32 < width) res_request<WIDE>(E, Q, row0, col + 32, rows, piece);
  if (!E.vec_out) {
    ragged_out<bf16, WIDE>(Q, row0, col, rows, panel, v);
  } else if (WIDE) {
    words32_out(panel, v, static_cast<unsigned char *>(Q.out) + (row0 * Q.ldo + col) * 4, Q.ldo * 4, rows, cols);
  } else {
    uint4 w[4];
    pack32(w, v, bf16);
    panel_out(panel, w, static_cast<unsigned char *>(Q.out) + (row0 * Q.ldo + col) * 2, Q.ldo * 2, rows, (cols + 7) / 8);
  }
}

template <bool bf16, int width>
__device__ __forceinline__ void keep_bits(const DenseParams &P, const Unit &Q, int64_t row0, int n0, int rows,
                                          const uint32_t *bits) {
  const LinearEnd &E = P.end;
  const int lane = threadIdx.x & 31;
  if (!E.slopes || E.act != SFNN_LINEAR_RELU || Q.split > 1 || lane >= rows) return;
  uint32_t *p = static_cast<uint32_t *>(E.slopes) + (row0 + lane) * (slope_row_bytes(Q.N, E.act) / 4) + n0 / 32;
  if constexpr (width == 128)
    *reinterpret_cast<uint4 *>(p) = make_uint4(bits[0], bits[1], bits[width / 32 - 2], bits[width / 32 - 1]);
  else if constexpr (width == 64)
    *reinterpret_cast<uint2 *>(p) = make_uint2(bits[0], bits[width / 32 - 1]);
  else
    *p = bits[0];
}

// The whole tile where neither a residual, a ragged output nor a part of K stands in the way: without those
// branches between them a value takes 9 instructions instead of 12 with a bias, 22 instead of 33 with GELU
// (8192 tokens, 512 -> 8192: bias 78 -> 70 us, ReLU 89 -> 72, GELU 148 -> 101; 1999 tokens, 4096 -> 16384,
// GELU, for seconds under the power cap 237 -> 232).
template <int ACT>
using Act = std::integral_constant<int, ACT>;
template <bool bf16, int width, int ACT, bool KEEP>
__device__ __forceinline__ void linear_plain(const DenseParams &P, const Unit &Q, uint32_t taddr, int64_t row0, int n0,
                                             int rows, uint32_t panel, uint32_t bias, uint32_t *bits) {
  const LinearEnd &E = P.end;
#pragma unroll 1
  for (int c = 0; c < width && n0 + c < Q.N; c += 32) {
    const int col = n0 + c;
    uint32_t raw[32], word = 0, code[32];
    float v[32];
    __syncwarp();
    tm_ld32(taddr + c, raw);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 f = unpack16(__shfl_sync(0xffffffffu, bias, i), bf16);
      v[2 * i] = __uint_as_float(raw[2 * i]) + f.x;
      v[2 * i + 1] = __uint_as_float(raw[2 * i + 1]) + f.y;
    }
    if (c + 32 < width) bias = bias_request(E, col + 32, Q.N);
    if (ACT == SFNN_LINEAR_RELU) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (KEEP) word |= v[i] <= 0.f ? 0u : 1u << i;
        v[i] = max_nan(v[i], 0.f);
      }
    } else if (ACT != SFNN_LINEAR_NONE) {
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        smooth_values<ACT == SFNN_LINEAR_GELU, KEEP>(v[i], v[i + 1], code[i], code[i + 1]);
    }
    uint4 w[4];
    if (KEEP && ACT > SFNN_LINEAR_RELU) {
      uint32_t q[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = __byte_perm(code[2 * i], code[2 * i + 1], 0x5410);
      words_to(w, q);
      const int64_t ld = slope_row_bytes(Q.N, ACT);
      panel_out(panel + kPanel, w, static_cast<unsigned char *>(E.slopes) + row0 * ld + (int64_t)col * 2, ld, rows, 4);
    }
    pack32(w, v, bf16);
    panel_out(panel, w, static_cast<unsigned char *>(Q.out) + (row0 * Q.ldo + col) * 2, Q.ldo * 2, rows, (Q.N - col + 7) / 8);
    if (KEEP && ACT == SFNN_LINEAR_RELU)
#pragma unroll
      for (int i = 0; i < width / 32; ++i)
        if (c == 32 * i) bits[i] = word;
  }
}

template <bool bf16, int width>
__device__ __forceinline__ void epi_linear(const DenseParams &P, const Unit &Q, uint32_t taddr, int64_t row0, int n0,
                                           uint32_t panel, ResPiece<false> &piece, uint32_t &bias) {
  const int rows = (int)min((int64_t)32, Q.M - row0);
  if (rows <= 0 || n0 >= Q.N) return;  // (the whole warp)
  uint32_t bits[width / 32] = {};
  const LinearEnd &E = P.end;
  if (Q.split == 1 && !E.res && E.vec_out) {
    const bool keep = E.slopes != nullptr;
    auto plain = [&](auto act, auto kept) {
      linear_plain<bf16, width, decltype(act)::value, decltype(kept)::value>(P, Q, taddr, row0, n0, rows, panel, bias, bits);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    if (E.act == SFNN_LINEAR_NONE)
      plain(Act<SFNN_LINEAR_NONE>{}, No{});
    else if (E.act == SFNN_LINEAR_RELU)
      keep ? plain(Act<SFNN_LINEAR_RELU>{}, Yes{}) : plain(Act<SFNN_LINEAR_RELU>{}, No{});
    else if (E.act == SFNN_LINEAR_GELU)
      keep ? plain(Act<SFNN_LINEAR_GELU>{}, Yes{}) : plain(Act<SFNN_LINEAR_GELU>{}, No{});
    else
      keep ? plain(Act<SFNN_LINEAR_SILU>{}, Yes{}) : plain(Act<SFNN_LINEAR_SILU>{}, No{});
    keep_bits<bf16, width>(P, Q, row0, n0, rows, bits);
    return;
  }
#pragma unroll 1
  for (int c = 0; c < width && n0 + c < Q.N; c += 32) {
    uint32_t raw[32], word = 0;
    float v[32];
    __syncwarp();
    tm_ld32(taddr + c, raw);
    tm_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
    linear32<bf16, width, false>(P, Q, row0, n0, c, rows, panel, piece, bias, v, word);
#pragma unroll
    for (int i = 0; i < width / 32; ++i)
      if (c == 32 * i) bits[i] = word;
  }
  keep_bits<bf16, width>(P, Q, row0, n0, rows, bits);
}

// An fp32 result shows what the tensor cores' accumulators lose: they cut each sum off instead of
// rounding it, about 2^-25 of it a 16-deep step towards zero (K = 28672: 1.1e-5 of the result with a
// quarter of K in one sum).  So K is summed up in segments of kSegment chunks, each from zero, which
// the epilogue's threads add up in registers while the next segment is multiplied.
constexpr int kSegment = 16;
template <bool bf16, int width>
__device__ __forceinline__ void epi_linear32(const DenseParams &P, const Unit &Q, int64_t row0, int n0, uint32_t panel,
                                             ResPiece<true> &piece, uint32_t &bias, float (&sum)[width]) {
  const int rows = (int)min((int64_t)32, Q.M - row0);
  if (rows <= 0 || n0 >= Q.N) return;  // (the whole warp)
  uint32_t bits[width / 32] = {};
#pragma unroll
  for (int c = 0; c < width; c += 32)
    if (n0 + c < Q.N) linear32<bf16, width, true>(P, Q, row0, n0, c, rows, panel, piece, bias, sum + c, bits[c / 32]);
  keep_bits<bf16, width>(P, Q, row0, n0, rows, bits);
}

// ---------------------------------------------------------------- the kernel
// TN: columns of a tile.  TALL: two 256-row halves to a tile of 512, whose chunks share the B operand's: a
// quarter less comes through the L2, which bounds the main loop of the others (4096 x 4096 -> 16384: 4.3 GB,
// 11.1 TB/s).  Both halves' sums fill tensor memory, so the epilogue takes a half into registers, gives its
// columns back, and works while the other half, or the next tile's first chunks, are multiplied: the first
// half is a ring of chunks ahead of the second at a tile's start and end.  Plain stores only: the linear
// layer's epilogue takes 5 us a half (GELU 10), more than that hides (4096 x 4096 -> 16384 GELU, with 384
// threads and 216 registers for its warps: 551 us against 410).
template <int EPI, bool BF16, int TN, bool TALL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads<EPI>, 1)
    k_dense(const __grid_constant__ DenseParams P) {
  constexpr bool kDGated = EPI == kEpiDGated || EPI == kEpiDGated8, kSegments = EPI == kEpiLinear32;
  constexpr int kStages = TALL ? 4 : kStagesOf<EPI>, kRows = TALL ? 512 : kTile;
  constexpr uint32_t kStageBytes = TALL ? 49152 : sfnn::kStageBytes;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
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
      bar_init(&acc_empty[i], 2 * kEpiWarps<EPI>);  // both CTAs' epilogue warps
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
        const int m0 = w.pos.m * kRows + (int)rank * 128;
        // gated: the first CTA loads 128 gate rows, the second the same 128 up rows
        const int n0 = EPI == kEpiGated ? w.pos.n * 128 : w.pos.n * TN + (int)rank * (TN / 2);
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
          if (rank == 0) bar_expect_tx(&full[s], (TALL ? 4 : 2) * 16384u + (uint32_t)TN * 128u);
          const uint32_t bar = cluster_addr(&full[s], 0);
          const uint32_t sa = stage0 + (uint32_t)s * kStageBytes, sb = sa + kStageBytes - 16384u;
          const bool second = kc >= w.nk0;
          const int k0 = (second ? kc - w.nk0 : kc) * 64;
          const CUtensorMap *ma = second ? a1 : a0;
          const CUtensorMap *mb = (EPI == kEpiGated ? rank != 0 : second) ? b1 : b0;
          if (EPI == kEpiStore && w.a_mn) {
            tma_load_2d_pair(sa, ma, m0, k0, bar);
            tma_load_2d_pair(sa + 8192u, ma, m0 + 64, k0, bar);
            if (TALL) {
              tma_load_2d_pair(sa + 16384u, ma, m0 + 256, k0, bar);
              tma_load_2d_pair(sa + 24576u, ma, m0 + 320, k0, bar);
            }
          } else {
            tma_load_2d_pair(sa, ma, k0, m0, bar);
            if (TALL) tma_load_2d_pair(sa + 16384u, ma, k0, m0 + 256, bar);
          }
          if (kDGated || (EPI == kEpiStore && w.b_mn)) {
            tma_load_2d_pair(sb, mb, n0, k0, bar);
            if (TN == 256) tma_load_2d_pair(sb + 8192u, mb, n0 + 64, k0, bar);
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
      int it = 0, turn = 0;
      bool ok = true;
      int id = walk.unit(0);
      Unit w{}, next = unit_at(P, max(id, 0));
      for (int n = 0; ok && id >= 0; ++n) {
        w = next;
        const int a_mn = EPI == kEpiStore ? w.a_mn : 0, b_mn = EPI == kEpiStore ? w.b_mn : kDGated;
        const uint32_t idesc = mma_desc_16(256, TN, BF16, a_mn, b_mn);
        // a 16-deep step of an operand: 2 KB of an MN-major tile, 32 bytes of a K-major one
        const uint32_t step_a = a_mn ? 2048u : 32u, step_b = b_mn ? 2048u : 32u;
        const uint32_t lbo_a = a_mn ? 8192u : 16u, lbo_b = b_mn ? 8192u : 16u;
        if constexpr (TALL) {
          // a chunk's MMAs into one half's sums
          auto multiply = [&](int i, int h) {
            const uint32_t sa = stage0 + (uint32_t)((it + i) % kStages) * kStageBytes, sb = sa + kStageBytes - 16384u;
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              mma_16<2>(tmem + (uint32_t)h * 256u, mat_desc(sa + (uint32_t)h * 16384u + k * step_a, lbo_a, 1024),
                        mat_desc(sb + k * step_b, lbo_b, 1024), idesc, (i > 0 || k > 0) ? 1u : 0u);
          };
          const int nk = w.k_hi - w.k_lo, head = min(kStages, nk), tail = min(kStages, nk - head), base = it;
          auto there = [&](int i) {
            const int j = base + i;
            const bool got = bar_wait(&full[j % kStages], (uint32_t)((j / kStages) & 1));
            tm_fence_after();
            return got;
          };
          const uint32_t parity = (uint32_t)(n & 1) ^ 1u;
          ok = bar_wait(&acc_empty[0], parity);
          tm_fence_after();
          for (int i = 0; ok && i < head; ++i) {
            ok = there(i);
            if (ok) multiply(i, 0);
          }
          id = walk.unit(n + 1);  // the next unit, while this one's MMAs run
          next = unit_at(P, max(id, 0));
          ok = ok && bar_wait(&acc_empty[1], parity);
          tm_fence_after();
          for (int i = 0; ok && i < nk - tail; ++i) {
            if (i >= head) {
              ok = there(i);
              if (!ok) break;
              multiply(i, 0);
            }
            multiply(i, 1);
            mma_commit_pair(&empty[(base + i) % kStages]);
          }
          for (int i = nk - tail; ok && i < nk; ++i) {
            ok = there(i);
            if (ok) multiply(i, 0);
          }
          if (ok) {
            mma_commit_pair(&acc_full[0]);
            for (int i = nk - tail; i < nk; ++i) {
              multiply(i, 1);
              mma_commit_pair(&empty[(base + i) % kStages]);
            }
            mma_commit_pair(&acc_full[1]);
          }
          it += nk;
          continue;
        }
        for (int k_lo = w.k_lo, k_hi; ok && k_lo < w.k_hi; k_lo = k_hi, ++turn) {
          k_hi = kSegments ? min(k_lo + kSegment, w.k_hi) : w.k_hi;
          const int buf = turn & 1;
          if (!bar_wait(&acc_empty[buf], (uint32_t)((turn >> 1) & 1) ^ 1u)) {
            ok = false;
            break;
          }
          tm_fence_after();
          const uint32_t d = tmem + (uint32_t)buf * 256u;
          for (int kc = k_lo; kc < k_hi; ++kc, ++it) {
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
                        (kc > k_lo || k > 0) ? 1u : 0u);
            mma_commit_pair(&empty[s]);
          }
          if (ok) mma_commit_pair(&acc_full[buf]);
        }
      }
      if (!ok) latch_error(P.err, kErrTimeout);
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t panel = stage0 + kStages * kStageBytes + (uint32_t)(warp - 2) * kWarpPanels<EPI>;
    if (EPI == kEpiStore && P.colsum) {  // while the first tile is multiplied: db from its 32-row sums
      for (int c = blockIdx.x * 256 + threadIdx.x - 64; c < P.cols; c += gridDim.x * 256) {
        float sum = 0.f;
#pragma unroll 8
        for (int b = 0; b < P.col_blocks; ++b) sum += __ldg(P.colpart + (int64_t)b * P.cols + c);
        P.colsum[c] = (uint16_t)pack16(sum, 0.f, BF16);
      }
    }
    __syncwarp();
    int turn = 0;
    for (int n = 0, id; (id = walk.unit(n)) >= 0; ++n) {
      const Unit w = unit_at(P, id);
      const int buf = n & 1;
      int64_t row0 = (int64_t)w.pos.m * kRows + rank * 128 + quad * 32;
      constexpr int kWide = TN / (kEpiWarps<EPI> / 4);  // columns of this warp
      const int n0 = EPI == kEpiGated ? w.pos.n * 128 + half * 64 : w.pos.n * TN + half * kWide;
      // what the epilogue reads besides the accumulators, requested before they are there
      float2 scales;
      if (EPI == kEpiGated) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          const float b = P.bias && n0 + c + lane < w.N ? load16(P.bias, n0 + c + lane, BF16) : 0.f;
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(panel + (uint32_t)(c + lane) * 4u), "f"(b) : "memory");
        }
      }
      if (kDGated) saved_request<EPI == kEpiDGated8>(P, w, row0, n0, panel + 2 * kPanel, scales);
      ResPiece<kSegments> piece;
      uint32_t bias = 0;
      if ((EPI == kEpiLinear || kSegments) && w.split == 1) {
        res_request<kSegments>(P.end, w, row0, n0, (int)max((int64_t)0, min((int64_t)32, w.M - row0)), piece);
        bias = bias_request(P.end, n0, w.N);
      }
      if constexpr (TALL) {
        bool there = true;
        for (int h = 0; h < 2; ++h, row0 += 256) {
          there = __all_sync(0xffffffffu, bar_wait(&acc_full[h], (uint32_t)(n & 1)));
          if (!there) break;
          __syncwarp();
          tm_fence_after();
          float sum[kWide];
#pragma unroll
          for (int c = 0; c < kWide; c += 32) {
            uint32_t raw[32];
            tm_ld32(tmem + lanes + (uint32_t)(h * 256 + half * kWide + c), raw);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c + i] = __uint_as_float(raw[i]);
          }
          tm_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty[h], 0));
          epi_store_sums<BF16, kWide>(w, row0, n0, panel, sum);
        }
        if (!there) {
          if (lane == 0) latch_error(P.err, kErrTimeout);
          break;
        }
        continue;
      }
      if constexpr (kSegments) {
        float sum[kWide];
#pragma unroll
        for (int i = 0; i < kWide; ++i) sum[i] = 0.f;
        bool there = true;
        for (int k = w.k_lo; k < w.k_hi; k += kSegment, ++turn) {
          const int buf = turn & 1;
          there = __all_sync(0xffffffffu, bar_wait(&acc_full[buf], (uint32_t)((turn >> 1) & 1)));
          if (!there) break;
          __syncwarp();
          tm_fence_after();
#pragma unroll
          for (int c = 0; c < kWide; c += 16) {  // (more at a time do not fit the registers)
            uint32_t raw[16];
            tm_ld16(tmem + lanes + (uint32_t)(buf * 256 + half * kWide + c), raw);
            tm_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(raw[i]);
          }
          tm_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty[buf], 0));
        }
        if (!there) {
          if (lane == 0) latch_error(P.err, kErrTimeout);
          break;
        }
        epi_linear32<BF16, kWide>(P, w, row0, n0, panel, piece, bias, sum);
        continue;
      }
      if (!__all_sync(0xffffffffu, bar_wait(&acc_full[buf], (uint32_t)((n >> 1) & 1)))) {
        if (lane == 0) latch_error(P.err, kErrTimeout);
        break;
      }
      __syncwarp();
      tm_fence_after();
      const uint32_t acc = tmem + lanes + (uint32_t)buf * 256u;
      auto done = [&] {
        tm_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive_cluster_relaxed(cluster_addr(&acc_empty[buf], 0));
      };
      if (EPI == kEpiGated) {
        epi_gated<BF16>(P, w, acc + half * 64, row0, n0, panel, done);
      } else {
        if (kDGated)
          epi_dgated<EPI == kEpiDGated8, BF16, kWide>(P, w, acc + half * kWide, row0, n0, scales, panel);
        else if constexpr (EPI == kEpiLinear)
          epi_linear<BF16, kWide>(P, w, acc + half * kWide, row0, n0, panel, piece, bias);
        else
          epi_store<BF16, kWide>(P, w, acc + half * kWide, row0, n0, panel);
        done();
      }
    }
    if (kDGated) cp_async_wait<0>();
  }
  __syncwarp();
  tm_fence_before();
  __syncthreads();
  cluster_sync_all();
  tm_fence_after();
  if (warp == 1) tm_dealloc<2>(tmem, kTmem);
}

template <int EPI>
constexpr size_t kSmem = (size_t)kStagesOf<EPI> * kStageBytes + kEpiWarps<EPI> * kWarpPanels<EPI> + 1024;

template <int EPI, bool BF16, int TN, bool TALL = false>
cudaError_t run_as(const DenseParams &P, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // devices whose kernel attribute is set
  const cudaError_t attr = allow_smem(k_dense<EPI, BF16, TN, TALL>, kSmem<EPI>, ready);
  if (attr != cudaSuccess) return attr;
  const int grid = 2 * std::min(num_sms / 2, P.first + P.rest);
  return launch_pdl(k_dense<EPI, BF16, TN, TALL>, dim3(grid), dim3(kThreads<EPI>), kSmem<EPI>, s, P);
}
template <int EPI>
cudaError_t run(const DenseParams &P, int num_sms, cudaStream_t s) {
  if (EPI != kEpiGated && P.p[0].tn == 128) {
    constexpr int kNarrow = EPI != kEpiGated ? 128 : 256;
    return P.bf16 ? run_as<EPI, true, kNarrow>(P, num_sms, s) : run_as<EPI, false, kNarrow>(P, num_sms, s);
  }
  if constexpr (EPI == kEpiStore)
    if (P.tall) return P.bf16 ? run_as<EPI, true, 256, true>(P, num_sms, s) : run_as<EPI, false, 256, true>(P, num_sms, s);
  return P.bf16 ? run_as<EPI, true, 256>(P, num_sms, s) : run_as<EPI, false, 256>(P, num_sms, s);
}

}  // namespace

namespace {
// About when the last pair is done, in ns: `chunk` for a chunk of a tile of `rows` rows, units of one length
// after the other's.
int64_t done_at(const DenseParams &P, int rows, int chunk, int pairs) {
  int64_t units = 0, work = 0, longest = 0, shortest = INT64_MAX;
  for (int i = 0; i < P.count; ++i) {
    const int64_t n = (int64_t)((P.p[i].M + rows - 1) / rows) * P.p[i].tiles_n, len = (int64_t)P.p[i].nk * chunk;
    units += n;
    work += n * len;
    longest = std::max(longest, len);
    shortest = std::min(shortest, len);
  }
  if (units <= 2 * pairs) return units <= pairs ? longest : std::max(longest, 2 * shortest);
  return std::max(longest, work / pairs + shortest / 2);
}
// Tiles of 512 rows: where they are done first.  (Gradients of T x K x N, bf16, us with 256 rows and with 512:
// 4096 x 4096 x 16384 785 and 714, 3000 x 8192 x 8192 584 and 524, 8192 x 1024 x 4096 120 and 112, but 1500 x
// 2048 x 8192 83 and 97, whose 24 long units leave most pairs idle at the end.)
bool tall_tiles(const DenseParams &P, int epi, int num_sms) {
  if (epi != kEpiStore) return false;
  for (int i = 0; i < P.count; ++i)
    if (P.p[i].relu || P.p[i].tn != 256 || P.p[i].split > 1) return false;
  return done_at(P, 512, 770, num_sms / 2) < done_at(P, 256, 430, num_sms / 2);
}
}  // namespace

cudaError_t launch_dense(DenseParams &P, int epi, int num_sms, cudaStream_t s) {
  P.tall = tall_tiles(P, epi, num_sms);
  if (P.tall)
    for (int i = 0; i < P.count; ++i) P.p[i].tiles_m = (P.p[i].M + 511) / 512;
  auto units = [&](int i) { return P.p[i].tiles_m * P.p[i].tiles_n * P.p[i].split; };
  // a unit's length in K chunks: a tile's epilogue (about 2.5 us) takes as long as nine
  constexpr int kEpilogue = 9;
  P.first = units(0);
  P.rest = 0;
  int len = kEpilogue;
  for (int i = 1; i < P.count; ++i) {
    P.rest += units(i);
    len = std::max(len, P.p[i].nk / P.p[i].split);
  }
  // (a part of a split K goes out in fp32, about half an epilogue more)
  const int lead = std::max(kEpilogue, P.p[0].nk / P.p[0].split) + (P.p[0].split > 1 ? kEpilogue / 2 : 0);
  P.extra = P.count > 1 ? (lead + len / 2 + 1) / len : 0;
  if (epi == kEpiGated) return run<kEpiGated>(P, num_sms, s);
  if (epi == kEpiDGated) return P.save == SFNN_SAVE_ACT8 ? run<kEpiDGated8>(P, num_sms, s) : run<kEpiDGated>(P, num_sms, s);
  if (epi == kEpiLinear) return P.p[0].out32 ? run<kEpiLinear32>(P, num_sms, s) : run<kEpiLinear>(P, num_sms, s);
  return run<kEpiStore>(P, num_sms, s);
}

}  // namespace sfnn
