// product.cu -- the host side that the dense operators share: shapes of their tensor-core products,
// the choice between the two kernels, and the joining of what a split product leaves.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {

int device_sms() {
  static std::atomic<int> known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 64) {
    const int k = known[dev].load(std::memory_order_relaxed);
    if (k) return k;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

// out[i] = sum over the parts of a split product, in their order.  Bound by the parts' bytes.
__global__ void __launch_bounds__(256) k_join(const float *__restrict__ part, int parts, int M, int N, int bf16, int out32,
                                              void *__restrict__ out, int64_t ldo) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t total = (int64_t)M * N / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(part) + p * total + i);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const int64_t row = i * 4 / N, col = i * 4 - row * N;
    if (out32)
      *reinterpret_cast<float4 *>(static_cast<float *>(out) + row * ldo + col) = s;
    else
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + row * ldo + col) =
          make_uint2(pack16(s.x, s.y, bf16), pack16(s.z, s.w, bf16));
  }
}
// db[i] = the sum of its 32-row sums (where no product follows that adds them up on the way).
__global__ void __launch_bounds__(256) k_colsum(const float *__restrict__ part, int blocks, int n, int bf16,
                                                uint16_t *__restrict__ out) {
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < blocks; ++k) s += part[(int64_t)k * n + c];
  out[c] = (uint16_t)(pack16(s, 0.f, bf16) & 0xffffu);
}

}  // namespace

cudaError_t launch_colsum(const float *part, int blocks, int n, int bf16, void *out, cudaStream_t s) {
  return launch_pdl(k_colsum, dim3((n + 255) / 256), dim3(256), 0, s, part, blocks, n, bf16, static_cast<uint16_t *>(out));
}

bool mat_ok(const void *p, int64_t ld, int64_t cols) {
  return p && a16(p) && ld >= cols && ld % 8 == 0 && ld <= (1ll << 36);
}

// C [M x N] = A . B^T: tensor maps and tile counts.  a_mn: A is stored [K x M]; b_mn: B is [K x N].
bool set_pair(DenseProblem &P, int which, const Operand &a, const Operand &b, int M, int N, int64_t K) {
  CUtensorMap *ma = which ? &P.a1 : &P.a0, *mb = which ? &P.b1 : &P.b0;
  return (a.mn ? make_tensor_map(ma, a.p, 2, K, M, a.ld, 64, 64, true)
               : make_tensor_map(ma, a.p, 2, M, K, a.ld, 128, 64, true)) &&
         (b.mn ? make_tensor_map(mb, b.p, 2, K, N, b.ld, 64, 64, true)
               : make_tensor_map(mb, b.p, 2, N, K, b.ld, P.tn / 2, 64, true));
}
// Parts of K of an M x N product of nk chunks: where its 256 x 256 tiles leave most SMs idle
// and K is long, as many as fill the SMs, of at least 8 chunks each.
int parts_of(int64_t M, int64_t N, int nk, int sms) {
  const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256), pairs = sms / 2;
  if (tiles < 1 || tiles * 2 > pairs) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>({pairs / tiles, nk / 8, 16}));
}
int64_t parts_bytes(int64_t M, int64_t N, int nk, int sms) {
  const int p = parts_of(M, N, nk, sms);
  return p > 1 ? up(p * M * up(N, 4) * 4, 256) : 0;
}

// Columns of a tile: 128 where that many tiles still fit one round of CTA pairs (a tile's
// latency counts: step of 257 tokens, 512 x 2048, 46.7 us against 51.8 with 256, timed in turn; 52
// to 57 with 128 on other cards and hosts).  Beyond, 256, even where halves would fill the last
// round better: they read each operand byte for half the products (4096 tokens, 4096 x 11008,
// with halves in the down product: 1.09 times as long).
int tile_columns(int M, int N, int split, int sms) {
  return (int64_t)((M + 255) / 256) * ((N + 127) / 128) * split <= sms / 2 ? 128 : 256;
}

// Up to 128 tokens, two kernels can form weights [N x K] . x: the slim one, whose tiles have
// all tokens and an even share of the weight rows, and the square tiles of the dense one.  The
// dense one's time in the units of slim_cost: rounds of tiles, each SM of a pair reading half of
// the tile's weight rows and tokens, and 1000 (3 us) for its longer way in and out.  Measured
// at 33 pairs of sizes from 280 x 2048 to 8192 x 14000 and 4 to 128 tokens, forward passes are
// 1.5 % on average above the best of the four pairings (both products slim: 17 %, both dense:
// 15 %).  Both slim / both dense, us, at 64 tokens: 512 x 2048 22.2 / 16.9, 280 x 25376 56.5 /
// 32.8, 2048 x 8192 43.1 / 36.0, 8192 x 14000 129 / 153; at 4: 12.7 / 16.2, 34.2 / 34.4, 31.7 /
// 35.5, 115 / 174.
bool slim_serves(int T, int N, int64_t K, bool gated, int sms) {
  if (T > 128 || sms < 2) return false;
  const int split = gated ? 1 : parts_of(T, N, chunks(K), sms);
  const int rows = gated ? 256 : tile_columns(T, N, split, sms), outs = gated ? 128 : rows;
  const int64_t units = (int64_t)((N + outs - 1) / outs) * split, pairs = sms / 2;
  const int64_t dense = (units + pairs - 1) / pairs * (rows + T) / 2 * chunks(K) / split + 1000;
  return slim_cost(T, N, K, gated, sms) < dense;
}

bool set_problem(DenseProblem &P, const Operand &a, const Operand &b, int M, int N, int64_t K, void *out, int64_t ldo, int split,
                 int tn) {
  P.M = M;
  P.N = N;
  P.nk0 = P.nk = chunks(K);
  P.tn = tn;
  P.tiles_m = (M + 255) / 256;
  P.tiles_n = (N + tn - 1) / tn;
  P.split = split;
  P.a_mn = a.mn;
  P.b_mn = b.mn;
  P.out = out;
  P.ldo = ldo;
  return set_pair(P, 0, a, b, M, N, K);
}
cudaError_t join(const DenseProblem &P, int bf16, int sms, cudaStream_t s) {
  if (P.split == 1) return cudaSuccess;
  const int64_t blocks = ((int64_t)P.M * P.N / 4 + 255) / 256;
  return launch_pdl(k_join, dim3((unsigned)std::min<int64_t>(blocks, 8 * sms)), dim3(256), 0, s, P.part, P.split, P.M, P.N,
                    bf16, P.out32, P.out, P.ldo);
}

}  // namespace sfnn
