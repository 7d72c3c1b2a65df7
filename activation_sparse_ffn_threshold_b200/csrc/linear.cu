// linear.cu -- the linear layer with its epilogue: Y = act(X W^T + b) + residual, and its gradients
//
//     dZ = dY act'(Z),   dX = dZ W,   dW = dZ^T X,   db = sum over tokens of dZ,   dresidual = dY
//
// Forward: one product (dense.cu, or few.cu for few tokens) whose epilogue does the rest; a K split
// over CTA pairs is joined by k_linear_join, which then does it.  Backward: k_linear_slopes makes dZ
// in the tensor cores' type and its columns' sums over 32 rows, from its values before that rounding;
// then dX and dW in one launch, which adds the sums up on its way.  Without an activation dY is dZ.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "async.cuh"
#include "common.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

// Rows of a split product's parts are `ld` floats (N rounded up to 4) apart.
__host__ __device__ constexpr int64_t part_ld(int64_t N) { return (N + 3) / 4 * 4; }

// A warp takes 128 columns of a row, a lane 4 of them.
__global__ void __launch_bounds__(256) k_linear_join(const float *__restrict__ part, int parts, int M, int N, int bf16,
                                                     int out32, void *out, int64_t ldo,
                                                     const __grid_constant__ LinearEnd E) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, blocks = (N + 127) / 128;
  const int64_t ld = part_ld(N), work = (int64_t)M * blocks, slope_ld = slope_row_bytes(N, E.act);
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < work; i += (int64_t)gridDim.x * 8) {
    const int64_t row = i / blocks;
    const int col = (int)(i - row * blocks) * 128 + lane * 4;
    const int cols = min(4, N - col);  // (may be negative)
    float v[4] = {};
    if (cols > 0) {
#pragma unroll 4
      for (int p = 0; p < parts; ++p) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(part + ((int64_t)p * M + row) * ld + col));
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
    }
    uint32_t bits = 0, code[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < cols && E.bias) v[j] += load16(E.bias, col + j, bf16);
      bits |= v[j] <= 0.f || j >= cols ? 0u : 1u << (4 * (lane & 7) + j);
    }
    act_values<4>(v, E.act, E.slopes != nullptr, code);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < cols && E.res) {
        const int64_t at = row * E.ldres + col + j;
        v[j] += out32 ? static_cast<const float *>(E.res)[at] : load16(E.res, at, bf16);
      }
      if (j < cols) {
        const int64_t at = row * ldo + col + j;
        if (out32)
          static_cast<float *>(out)[at] = v[j];
        else
          static_cast<uint16_t *>(out)[at] = (uint16_t)pack16(v[j], 0.f, bf16);
      }
    }
    if (!E.slopes) continue;
    unsigned char *s = static_cast<unsigned char *>(E.slopes) + row * slope_ld;
    if (E.act == SFNN_LINEAR_RELU) {
#pragma unroll
      for (int o = 1; o < 8; o *= 2) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
      if ((lane & 7) == 0) reinterpret_cast<uint32_t *>(s)[col / 32] = bits;
    } else if (col < (N + 31) / 32 * 32) {
      *reinterpret_cast<uint2 *>(s + (int64_t)col * 2) = make_uint2(__byte_perm(code[0], code[1], 0x5410), __byte_perm(code[2], code[3], 0x5410));
    }
  }
}

// dZ from dY, and its columns' sums over blocks of rows before it is rounded.  A CTA has a block of 8
// `per` rows and 256 columns, a warp `per` rows of it, a lane 8 neighbouring columns.  VEC: dY's rows start
// on 16 bytes (those of act' and dZ always do); a lane's pieces of the next kAhead rows are then on their
// way into shared memory, where nobody else reads them.  Else four rows are read at a time.
// Bound by bytes.  (Rows in flight in registers instead: 4096 x 16384 bf16 with a ReLU's slopes 98 us.
// Value by value, unrolled, 333 x 2047 took 9 us, most of it first fetches of its instructions.)
struct SlopeParams {
  const void *dy;
  int64_t lddy;
  int act, M, N, per;
  const void *slopes;
  void *dz;  // or null: dY is dZ.  Rows of N rounded up to 8
  int64_t lddz;
  float *colpart;  // or null
};
constexpr int kAhead = 6;
constexpr int slope_piece(bool dy32) { return dy32 ? 48 : 32; }  // bytes of a lane's row: dY, act'
constexpr size_t slope_smem(bool dy32, bool vec) { return vec ? (size_t)kAhead * 256 * slope_piece(dy32) : 0; }

template <bool bf16, bool DY32, bool VEC>
__global__ void __launch_bounds__(256) k_linear_slopes(const __grid_constant__ SlopeParams P) {
  extern __shared__ __align__(16) unsigned char ahead[];
  __shared__ float sums[8][256];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * 256, col = c0 + lane * 8;
  const int64_t slope_ld = slope_row_bytes(P.N, P.act), rows = 8 * P.per;
  constexpr int E = DY32 ? 4 : 2;
  constexpr uint32_t kPlane = kAhead * 256 * 16;  // a 16-byte column of the pieces
  const uint32_t own = smem_u32(ahead) + threadIdx.x * 16u;
  const bool relu = P.act == SFNN_LINEAR_RELU, smooth = !relu && P.act != SFNN_LINEAR_NONE;
  for (int64_t block = blockIdx.y; block * rows < P.M; block += gridDim.y) {
    float sum[8] = {};
    const int64_t row0 = block * rows + (int64_t)warp * P.per;
    const int live = col < P.N ? (int)max((int64_t)0, min((int64_t)P.per, P.M - row0)) : 0;
    const unsigned char *dy = static_cast<const unsigned char *>(P.dy) + (row0 * P.lddy + col) * E;
    const unsigned char *slopes = static_cast<const unsigned char *>(P.slopes) + row0 * slope_ld + (relu ? col >> 5 << 2 : col * 2);
    uint16_t *dz = static_cast<uint16_t *>(P.dz) + row0 * P.lddz + col;
    auto request = [&](int r) {
      if (VEC && r < live) {
        const uint32_t to = own + (uint32_t)(r % kAhead) * (256u * 16u);
        const unsigned char *d = dy + r * P.lddy * E, *s = slopes + r * slope_ld;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(d) : "memory");
        if (DY32) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + kPlane), "l"(d + 16) : "memory");
        if (relu) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + (DY32 ? 2 : 1) * kPlane), "l"(s) : "memory");
        if (smooth) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (DY32 ? 2 : 1) * kPlane), "l"(s) : "memory");
      }
      cp_async_commit();
    };
    if (VEC)
#pragma unroll 1
      for (int r = 0; r < kAhead - 1; ++r) request(r);
#pragma unroll(VEC ? 1 : 4)
    for (int r = 0; r < live; ++r) {
      float v[8];
      uint4 code = make_uint4(0, 0, 0, 0);
      if (VEC) {
        request(r + kAhead - 1);
        cp_async_wait<kAhead - 1>();
        const uint32_t at = own + (uint32_t)(r % kAhead) * (256u * 16u);
        uint4 a, b = code;
        auto lds = [](uint32_t p) {
          uint4 w;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(p) : "memory");
          return w;
        };
        a = lds(at);
        if (DY32) b = lds(at + kPlane);
        if (relu || smooth) code = lds(at + (DY32 ? 2 : 1) * kPlane);
        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (DY32) {
            v[i] = __uint_as_float(u[i]), v[4 + i] = __uint_as_float(u[4 + i]);
          } else {
            const float2 f = unpack16(u[i], bf16);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
          }
        }
      } else {
        const unsigned char *d = dy + r * P.lddy * E, *s = slopes + r * slope_ld;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = col + j >= P.N ? 0.f : DY32 ? reinterpret_cast<const float *>(d)[j] : load16(d, j, bf16);
        if (relu) code.x = __ldg(reinterpret_cast<const uint32_t *>(s));
        if (smooth) code = ld_stream(s);
      }
      if (relu) {
        const uint32_t on = code.x >> (col & 31);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = on >> j & 1u ? v[j] : 0.f;
      } else if (smooth) {
        const uint32_t u[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] *= slope_value(u[j] & 0xffffu);
          v[2 * j + 1] *= slope_value(u[j] >> 16);
        }
        if (!VEC)  // (codes past the row are anything)
#pragma unroll
          for (int j = 1; j < 8; ++j) v[j] = col + j < P.N ? v[j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
      if (P.dz)
        *reinterpret_cast<uint4 *>(dz + r * P.lddz) =
            make_uint4(pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16), pack16(v[4], v[5], bf16), pack16(v[6], v[7], bf16));
    }
    if (VEC) cp_async_wait<0>();
    if (!P.colpart) continue;
    __syncthreads();  // the block before has been added up
    float4 *mine = reinterpret_cast<float4 *>(&sums[warp][lane * 8]);
    mine[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    mine[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    __syncthreads();
    const int c = c0 + threadIdx.x;
    if (c >= P.N) continue;
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) total += sums[w][threadIdx.x];
    P.colpart[block * P.N + c] = total;
  }
}
template <bool bf16, bool DY32, bool VEC>
cudaError_t launch_slopes(const SlopeParams &P, dim3 grid, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  constexpr size_t smem = slope_smem(DY32, VEC);
  const cudaError_t e = smem ? allow_smem(k_linear_slopes<bf16, DY32, VEC>, smem, ready) : cudaSuccess;
  return e != cudaSuccess ? e : launch_pdl(k_linear_slopes<bf16, DY32, VEC>, grid, dim3(256), smem, s, P);
}

// ---------------------------------------------------------------- host
constexpr int kMaxWidth = 1 << 20;
int64_t row_blocks(int64_t T) { return (T + 31) / 32; }  // at most
// Rows of a warp in k_linear_slopes: 4, or 16 where blocks of 128 rows still fill the SMs.
int slope_rows(int64_t T, int64_t N, int sms) { return (T + 127) / 128 * ((N + 255) / 256) >= 4 * sms ? 16 : 4; }

sfnn_status check(const sfnn_linear_desc *q) {
  if (!q || q->T < 0 || q->K < 1 || q->N < 1) return SFNN_ERR_INVALID_ARG;
  if (q->dtype != SFNN_F16 && q->dtype != SFNN_BF16) return q->dtype == SFNN_F32 ? SFNN_ERR_UNSUPPORTED : SFNN_ERR_INVALID_ARG;
  if (q->y_dtype != q->dtype && q->y_dtype != SFNN_F32) return SFNN_ERR_INVALID_ARG;
  if (q->act < SFNN_LINEAR_NONE || q->act > SFNN_LINEAR_SILU) return SFNN_ERR_INVALID_ARG;
  if (q->K % 8 || q->K > kMaxWidth || q->N > kMaxWidth || q->T > (1 << 24)) return SFNN_ERR_UNSUPPORTED;
  if (!mat_ok(q->w, q->ldw, q->K) || (q->T > 0 && !mat_ok(q->x, q->ldx, q->K)) || !on(q->b, 2)) return SFNN_ERR_INVALID_ARG;
  return SFNN_OK;
}
// Rows of values of the output's type: any alignment of it, any row stride of at least N.
bool values_ok(const void *p, int64_t ld, const sfnn_linear_desc *q) {
  return p && on(p, q->y_dtype == SFNN_F32 ? 4 : 2) && ld >= q->N && ld <= (1ll << 36);
}
bool pieces(const void *p, int64_t ld, const sfnn_linear_desc *q) {
  const int per = q->y_dtype == SFNN_F32 ? 4 : 8;
  return a16(p) && ld % per == 0 && q->N % per == 0;
}
bool slopes_ok(const void *p) { return p && a16(p); }

// The square tiles' time in ns, fitted to the products that few_plan's is fitted to (off by 6 % on average).
double dense_cost(int T, int N, int64_t K, int sms) {
  const int split = parts_of(T, N, chunks(K), sms), rows = tile_columns(T, N, split, sms);
  const int64_t units = (int64_t)((N + rows - 1) / rows) * ((T + 255) / 256) * split, pairs = sms / 2;
  const int64_t rounds = (units + pairs - 1) / pairs;
  return 2820 + rounds * (chunks(K) / split * (245 + 0.528 * rows) + 32.3 * (rows / 2 + 30)) +
         (split > 1 ? 2130 + 1.28e-3 * split * T * N : 0);
}

int64_t dz_bytes(int64_t T, int64_t N) { return up(T * up(N, 8) * 2, 256); }
int64_t workspace(int64_t T, int64_t K, int64_t N, bool backward, int sms) {
  if (!backward) return parts_bytes(T, N, chunks(K), sms);
  return dz_bytes(T, N) + up(row_blocks(T) * N * 4, 256) + parts_bytes(T, K, chunks(N), sms) +
         parts_bytes(N, K, chunks(T), sms);
}

}  // namespace
}  // namespace sfnn

using namespace sfnn;

extern "C" {

int64_t sfnn_linear_workspace(int32_t T, int32_t K, int32_t N, int32_t backward) {
  if (T < 0 || K < 1 || N < 1) return -1;
  return workspace(T, K, N, backward != 0, std::max(1, device_sms()));
}
int64_t sfnn_linear_slope_bytes(int32_t T, int32_t N, int32_t act) {
  if (T < 0 || N < 1 || act < SFNN_LINEAR_NONE || act > SFNN_LINEAR_SILU) return -1;
  return T * slope_row_bytes(N, act);
}

sfnn_status sfnn_linear_forward(const sfnn_linear_desc *q, const void *residual, int64_t ldr, void *y, int64_t ldy,
                                void *slopes, void *ws, int64_t ws_bytes, int32_t *err, sfnn_stream_t stream) {
  const sfnn_status st = check(q);
  if (st != SFNN_OK) return st;
  if (slopes && (!a16(slopes) || q->act == SFNN_LINEAR_NONE)) return SFNN_ERR_INVALID_ARG;
  if (q->T == 0) return SFNN_OK;
  if (!values_ok(y, ldy, q) || (residual && !values_ok(residual, ldr, q)) || !err || !on(err, 4)) return SFNN_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (sms < 2) return SFNN_ERR_CUDA;
  const int64_t need = workspace(q->T, q->K, q->N, false, sms);
  if (need && (!ws || !a16(ws) || ws_bytes < need)) return SFNN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int T = q->T, N = q->N, bf16 = q->dtype == SFNN_BF16, out32 = q->y_dtype == SFNN_F32;
  LinearEnd end{};
  end.bias = q->b;
  end.res = residual;
  end.ldres = ldr;
  end.act = q->act;
  end.slopes = slopes;
  end.vec_out = pieces(y, ldy, q);
  end.vec_res = residual && pieces(residual, ldr, q);
  const FewPlan few = few_plan(T, N, q->K, slopes && q->act == SFNN_LINEAR_RELU, out32, sms);
  if (few.cost < dense_cost(T, N, q->K, sms)) {
    FewArgs a{};
    a.x = q->x;
    a.ldx = q->ldx;
    a.w = q->w;
    a.ldw = q->ldw;
    a.T = T;
    a.N = N;
    a.K = q->K;
    a.out = y;
    a.ldo = ldy;
    a.bf16 = bf16;
    a.out32 = out32;
    a.end = &end;
    a.err = err;
    return launch_few(a, few, sms, s);
  }
  DenseParams P{};
  P.count = 1;
  const int split = parts_of(T, N, chunks(q->K), sms);
  if (!set_problem(P.p[0], Operand{q->x, q->ldx, false}, Operand{q->w, q->ldw, false}, T, N, q->K, y, ldy, split,
                   tile_columns(T, N, split, sms)))
    return SFNN_ERR_CUDA;
  P.p[0].out32 = out32;
  P.p[0].part = static_cast<float *>(ws);
  P.bf16 = bf16;
  P.end = end;
  P.err = err;
  if (launch_dense(P, kEpiLinear, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
  if (split > 1) {
    const int64_t warps = (int64_t)T * ((N + 127) / 128);
    if (launch_pdl(k_linear_join, dim3((unsigned)std::min<int64_t>((warps + 7) / 8, 8 * sms)), dim3(256), 0, s, P.p[0].part,
                   split, T, N, bf16, out32, y, ldy, end) != cudaSuccess)
      return SFNN_ERR_CUDA;
  }
  return SFNN_OK;
}

sfnn_status sfnn_linear_backward(const sfnn_linear_desc *q, const void *slopes, const void *dy, int64_t lddy, void *dx,
                                 void *dw, void *db, void *ws, int64_t ws_bytes, int32_t *err, sfnn_stream_t stream) {
  const sfnn_status st = check(q);
  if (st != SFNN_OK) return st;
  if (!a16(dx) || !a16(dw) || !on(db, 2)) return SFNN_ERR_INVALID_ARG;
  const int T = q->T, K = q->K, N = q->N, bf16 = q->dtype == SFNN_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // sums over no tokens
    if ((dw && cudaMemsetAsync(dw, 0, (size_t)N * K * 2, s) != cudaSuccess) ||
        (db && cudaMemsetAsync(db, 0, (size_t)N * 2, s) != cudaSuccess))
      return SFNN_ERR_CUDA;
    return SFNN_OK;
  }
  if (!values_ok(dy, lddy, q) || (q->act != SFNN_LINEAR_NONE && !slopes_ok(slopes)) || !err || !on(err, 4))
    return SFNN_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (sms < 2) return SFNN_ERR_CUDA;
  if (!ws || !a16(ws) || ws_bytes < workspace(T, K, N, true, sms)) return SFNN_ERR_INVALID_ARG;
  unsigned char *w = static_cast<unsigned char *>(ws);
  float *colpart = reinterpret_cast<float *>(w + dz_bytes(T, N));
  float *parts_x = colpart + up(row_blocks(T) * N * 4, 256) / 4;
  float *parts_w = parts_x + parts_bytes(T, K, chunks(N), sms) / 4;

  // dY itself where it is what the tensor cores read
  const bool as_is = q->act == SFNN_LINEAR_NONE && q->y_dtype == q->dtype && mat_ok(dy, lddy, N);
  Operand dz{dy, lddy, false};
  if (!as_is) dz = Operand{w, up(N, 8), false};
  int blocks = 0;
  if (db || (!as_is && (dx || dw))) {
    SlopeParams P{};
    P.dy = dy;
    P.lddy = lddy;
    P.act = q->act;
    P.M = T;
    P.N = N;
    P.slopes = slopes;
    P.dz = as_is || (!dx && !dw) ? nullptr : w;
    P.lddz = up(N, 8);
    P.colpart = db ? colpart : nullptr;
    const bool vec = N % 8 == 0 && a16(dy) && lddy % 8 == 0;
    P.per = slope_rows(T, N, sms);
    blocks = (T + 8 * P.per - 1) / (8 * P.per);
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)std::min(blocks, 65535));
    const bool wide = q->y_dtype == SFNN_F32;
    auto of_type = [&](auto b16) {
      constexpr bool B = decltype(b16)::value;
      if (vec) return wide ? launch_slopes<B, true, true>(P, grid, s) : launch_slopes<B, false, true>(P, grid, s);
      return wide ? launch_slopes<B, true, false>(P, grid, s) : launch_slopes<B, false, false>(P, grid, s);
    };
    if ((bf16 ? of_type(std::true_type{}) : of_type(std::false_type{})) != cudaSuccess)
      return SFNN_ERR_CUDA;
  }
  // dX and dW in one launch, the one with the longer tiles first
  DenseParams P{};
  auto add_x = [&] {
    DenseProblem &D = P.p[P.count++];
    const int split = parts_of(T, K, chunks(N), sms);
    D.part = parts_x;
    return set_problem(D, dz, Operand{q->w, q->ldw, true}, T, K, N, dx, K, split);
  };
  auto add_w = [&] {
    DenseProblem &D = P.p[P.count++];
    const int split = parts_of(N, K, chunks(T), sms);
    D.part = parts_w;
    return set_problem(D, Operand{dz.p, dz.ld, true}, Operand{q->x, q->ldx, true}, N, K, T, dw, K, split);
  };
  const bool x_first = chunks(N) / parts_of(T, K, chunks(N), sms) >= chunks(T) / parts_of(N, K, chunks(T), sms);
  if ((dx && x_first && !add_x()) || (dw && !add_w()) || (dx && !x_first && !add_x())) return SFNN_ERR_CUDA;
  if (!P.count) return !db || launch_colsum(colpart, blocks, N, bf16, db, s) == cudaSuccess ? SFNN_OK : SFNN_ERR_CUDA;
  P.bf16 = bf16;
  P.err = err;
  P.colpart = colpart;
  P.colsum = static_cast<uint16_t *>(db);
  P.col_blocks = blocks;
  P.cols = N;
  if (launch_dense(P, kEpiStore, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
  for (int i = 0; i < P.count; ++i)
    if (join(P.p[i], bf16, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
  return SFNN_OK;
}

}  // extern "C"
