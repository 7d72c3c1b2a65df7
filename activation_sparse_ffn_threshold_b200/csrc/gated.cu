// gated.cu -- the gated FFN over all neurons: forward, backward, and the entry points.
#include <algorithm>

#include "common.cuh"
#include "context.cuh"
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

int64_t row_blocks(int64_t T) { return (T + 31) / 32; }

int64_t hidden_bytes(int64_t T, int64_t n) { return up(T * up(n, 8) * 2, 256); }

sfnn_status check(const sfnn_gated_desc *q) {
  if (!q || q->T < 0 || q->d < 1 || q->n < 1) return SFNN_ERR_INVALID_ARG;
  if (q->dtype != SFNN_F16 && q->dtype != SFNN_BF16)
    return q->dtype == SFNN_F32 ? SFNN_ERR_UNSUPPORTED : SFNN_ERR_INVALID_ARG;
  if (q->d % 8) return SFNN_ERR_UNSUPPORTED;
  if (q->down_layout != SFNN_DOWN_WIDTH_MAJOR && q->down_layout != SFNN_DOWN_NEURON_MAJOR) return SFNN_ERR_INVALID_ARG;
  if (q->down_layout == SFNN_DOWN_WIDTH_MAJOR && q->n % 8) return SFNN_ERR_UNSUPPORTED;
  if (q->d > (1 << 20) || q->n > (1 << 20) || q->T > (1 << 24)) return SFNN_ERR_UNSUPPORTED;
  if (!mat_ok(q->w_gate, q->ld_gate, q->d) || !mat_ok(q->w_up, q->ld_up, q->d) ||
      !mat_ok(q->w_down, q->ld_down, q->down_layout == SFNN_DOWN_WIDTH_MAJOR ? q->n : q->d))
    return SFNN_ERR_INVALID_ARG;
  if ((q->T > 0 && !mat_ok(q->x, q->ldx, q->d)) || !on(q->b, 2)) return SFNN_ERR_INVALID_ARG;
  return SFNN_OK;
}

sfnn_status check_saved(const sfnn_gated_desc *q, const sfnn_gated_saved *sv) {
  if (sv->kind != SFNN_SAVE_FULL && sv->kind != SFNN_SAVE_ACT8) return SFNN_ERR_INVALID_ARG;
  if (q->n % 8) return SFNN_ERR_UNSUPPORTED;
  const bool eight = sv->kind == SFNN_SAVE_ACT8;
  const int64_t nb = up(q->n, kAct8Block) / kAct8Block, db = up(q->d, kAct8Block) / kAct8Block;
  if (sv->ld < nb * kAct8Block || sv->ld % 16 || sv->lds < nb) return SFNN_ERR_INVALID_ARG;
  if (eight && (sv->ld_x < db * kAct8Block || sv->ld_x % 16 || sv->lds_x < db)) return SFNN_ERR_INVALID_ARG;
  if (q->T == 0) return SFNN_OK;
  if (!sv->r || !sv->u || !a16(sv->r) || !a16(sv->u)) return SFNN_ERR_INVALID_ARG;
  if (!sv->r_scales || !sv->u_scales || !on(sv->r_scales, 4) || !on(sv->u_scales, 4)) return SFNN_ERR_INVALID_ARG;
  if (eight && (!sv->x || !sv->x_scales || !a16(sv->x) || !on(sv->x_scales, 4))) return SFNN_ERR_INVALID_ARG;
  return SFNN_OK;
}

// (`kernels` counts the launches.)
sfnn_status product(const Operand &a, const Operand &b, int M, int N, int64_t K, void *out, int64_t ldo, int out32, int bf16,
                    float *parts, int32_t *err, cudaStream_t s, int &kernels, const void *relu_bias = nullptr) {
  const int sms = device_sms();
  DenseParams P{};
  P.count = 1;
  const int split = parts ? parts_of(M, N, chunks(K), sms) : 1;
  if (!set_problem(P.p[0], a, b, M, N, K, out, ldo, split, tile_columns(M, N, split, sms))) return SFNN_ERR_CUDA;
  P.p[0].out32 = out32;
  P.p[0].relu = relu_bias != nullptr;
  P.p[0].part = parts;
  P.bias = relu_bias;
  P.bf16 = bf16;
  P.err = err;
  if (launch_dense(P, kEpiStore, sms, s) != cudaSuccess || join(P.p[0], bf16, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
  kernels += split > 1 ? 2 : 1;
  return SFNN_OK;
}

int64_t workspace(int32_t T, int32_t d, int32_t n, int32_t backward) {
  if (T < 0 || d < 1 || n < 1) return -1;
  const int sms = device_sms();
  if (!backward) return hidden_bytes(T, n) + parts_bytes(T, d, chunks(n), sms);
  return 3 * hidden_bytes(T, n) + hidden_bytes(T, d) + up(row_blocks(T) * n * 4, 256) +
         parts_bytes(T, d, 2 * chunks(n), sms);
}

sfnn_status forward(const sfnn_gated_desc *q, void *y, int64_t ldy, int32_t y_dtype, sfnn_gated_saved *sv, void *ws,
                    int64_t ws_bytes, int32_t *err, sfnn_stream_t stream, int &kernels) {
  sfnn_status st = check(q);
  if (st != SFNN_OK) return st;
  const int kind = sv ? sv->kind : SFNN_SAVE_NONE;
  if (kind != SFNN_SAVE_NONE && (st = check_saved(q, sv)) != SFNN_OK) return st;
  if (y_dtype != q->dtype && y_dtype != SFNN_F32) return SFNN_ERR_INVALID_ARG;
  if (q->T == 0) return SFNN_OK;
  if (!mat_ok(y, y_dtype == SFNN_F32 ? ldy * 2 : ldy, q->d) || ldy < q->d || !err || !on(err, 4) || !ws || !a16(ws) ||
      ws_bytes < workspace(q->T, q->d, q->n, 0))
    return SFNN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int bf16 = q->dtype == SFNN_BF16;
  const int64_t ldh = up(q->n, 8);
  if (kind == SFNN_SAVE_ACT8 &&
      launch_act8_quantize(q->x, q->ldx, q->T, q->d, bf16, false, static_cast<uint8_t *>(sv->x), sv->ld_x,
                           sv->x_scales, sv->lds_x, s) != cudaSuccess)
    return SFNN_ERR_CUDA;
  kernels += kind == SFNN_SAVE_ACT8;
  const int sms = device_sms();
  const bool slim_up = kind == SFNN_SAVE_NONE && slim_serves(q->T, q->n, q->d, true, sms);
  const bool slim_down =
      q->down_layout == SFNN_DOWN_WIDTH_MAJOR && slim_serves(q->T, q->d, q->n, false, sms);
  float *parts = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + hidden_bytes(q->T, q->n));
  const Operand h{ws, ldh, false}, wd{q->w_down, q->ld_down, q->down_layout == SFNN_DOWN_NEURON_MAJOR};
  auto down = [&](int early) -> sfnn_status {
    if (!slim_down) return product(h, wd, q->T, q->d, q->n, y, ldy, y_dtype == SFNN_F32, bf16, parts, err, s, kernels);
    SlimArgs a{};
    a.x = ws;
    a.ldx = ldh;
    a.w0 = q->w_down;
    a.ldw0 = q->ld_down;
    a.T = q->T;
    a.N = q->d;
    a.K = q->n;
    a.out = y;
    a.ldo = ldy;
    a.bf16 = bf16;
    a.out32 = y_dtype == SFNN_F32;
    a.early = early;
    a.err = err;
    ++kernels;
    return launch_slim(a, sms, s);
  };
  if (slim_up) {
    SlimArgs a{};
    a.x = q->x;
    a.ldx = q->ldx;
    a.w0 = q->w_gate;
    a.ldw0 = q->ld_gate;
    a.w1 = q->w_up;
    a.ldw1 = q->ld_up;
    a.bias = q->b;
    a.T = q->T;
    a.N = q->n;
    a.K = q->d;
    a.out = ws;
    a.ldo = ldh;
    a.bf16 = bf16;
    a.err = err;
    if ((st = launch_slim(a, sms, s)) != SFNN_OK) return st;
    ++kernels;
    return down(1);
  }
  DenseParams P{};
  DenseProblem &Q = P.p[0];
  P.count = 1;
  Q.M = q->T;
  Q.N = q->n;
  Q.nk0 = Q.nk = chunks(q->d);
  Q.split = 1;
  Q.tn = 256;  // 128 neurons, gate and up
  Q.tiles_m = (q->T + 255) / 256;
  Q.tiles_n = (q->n + 127) / 128;
  Q.out = ws;
  Q.ldo = ldh;
  if (!make_tensor_map(&Q.a0, q->x, 2, q->T, q->d, q->ldx, 128, 64, true) ||
      !make_tensor_map(&Q.b0, q->w_gate, 2, q->n, q->d, q->ld_gate, 128, 64, true) ||
      !make_tensor_map(&Q.b1, q->w_up, 2, q->n, q->d, q->ld_up, 128, 64, true))
    return SFNN_ERR_CUDA;
  P.bf16 = bf16;
  P.bias = q->b;
  P.save = kind;
  if (kind != SFNN_SAVE_NONE) {
    P.r = sv->r;
    P.u = sv->u;
    P.ldr = sv->ld;
    P.rs = sv->r_scales;
    P.us = sv->u_scales;
    P.lds = sv->lds;
  }
  P.err = err;
  if (launch_dense(P, kEpiGated, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
  ++kernels;
  return down(0);
}

}  // namespace
}  // namespace sfnn

using namespace sfnn;

extern "C" {

int64_t sfnn_gated_workspace(int32_t T, int32_t d, int32_t n, int32_t backward) { return workspace(T, d, n, backward); }

sfnn_status sfnn_gated_forward(const sfnn_gated_desc *q, void *y, int64_t ldy, int32_t y_dtype, sfnn_gated_saved *sv,
                               void *ws, int64_t ws_bytes, int32_t *err, sfnn_stream_t stream) {
  int kernels = 0;
  return forward(q, y, ldy, y_dtype, sv, ws, ws_bytes, err, stream, kernels);
}

sfnn_status sfnn_gated_backward(const sfnn_gated_desc *q, const void *dy, int64_t lddy, const sfnn_gated_saved *sv,
                                void *dx, void *dw_gate, void *dw_up, void *dw_down, void *db, void *ws,
                                int64_t ws_bytes, int32_t *err, sfnn_stream_t stream) {
  if (!q || !sv) return SFNN_ERR_INVALID_ARG;
  sfnn_gated_desc qq = *q;  // act8: x is not read, its blocks are
  if (sv->kind == SFNN_SAVE_ACT8) {
    qq.x = q->w_gate;
    qq.ldx = q->ld_gate;
  }
  sfnn_status st = check(&qq);
  if (st != SFNN_OK) return st;
  if (q->down_layout != SFNN_DOWN_WIDTH_MAJOR) return SFNN_ERR_UNSUPPORTED;
  if ((st = check_saved(q, sv)) != SFNN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int T = q->T, d = q->d, n = q->n, bf16 = q->dtype == SFNN_BF16;
  if ((dx && !a16(dx)) || (dw_gate && !a16(dw_gate)) || (dw_up && !a16(dw_up)) || (dw_down && !a16(dw_down)) ||
      !on(db, 2))
    return SFNN_ERR_INVALID_ARG;
  if (T == 0) {  // sums over no tokens
    if ((dw_gate && cudaMemsetAsync(dw_gate, 0, (size_t)n * d * 2, s) != cudaSuccess) ||
        (dw_up && cudaMemsetAsync(dw_up, 0, (size_t)n * d * 2, s) != cudaSuccess) ||
        (dw_down && cudaMemsetAsync(dw_down, 0, (size_t)n * d * 2, s) != cudaSuccess) ||
        (db && cudaMemsetAsync(db, 0, (size_t)n * 2, s) != cudaSuccess))
      return SFNN_ERR_CUDA;
    return SFNN_OK;
  }
  if (!mat_ok(dy, lddy, d) || !err || !on(err, 4) || !ws || !a16(ws) || ws_bytes < sfnn_gated_workspace(T, d, n, 1))
    return SFNN_ERR_INVALID_ARG;
  const int64_t hb = hidden_bytes(T, n), ldh = up(n, 8);
  unsigned char *w = static_cast<unsigned char *>(ws);
  void *h = w, *dg = w + hb, *du = w + 2 * hb, *xr = w + 3 * hb;
  float *colpart = reinterpret_cast<float *>(w + 3 * hb + hidden_bytes(T, d));
  float *parts = colpart + up(row_blocks(T) * n * 4, 256) / 4;
  const int sms = device_sms();

  Operand x{q->x, q->ldx, true};
  if (sv->kind == SFNN_SAVE_ACT8 && (dw_gate || dw_up)) {
    if (launch_act8_restore(static_cast<const uint8_t *>(sv->x), sv->ld_x, sv->x_scales, sv->lds_x, T, d, false, bf16, xr,
                            up(d, 8), s) != cudaSuccess)
      return SFNN_ERR_CUDA;
    x = Operand{xr, up(d, 8), true};
  }
  {
    DenseParams P{};
    P.count = 1;
    if (!set_problem(P.p[0], Operand{dy, lddy, false}, Operand{q->w_down, q->ld_down, true}, T, n, d, h, ldh, 1,
                     tile_columns(T, n, 1, sms)))
      return SFNN_ERR_CUDA;
    P.bf16 = bf16;
    P.dg = dg;
    P.du = du;
    P.colpart = db ? colpart : nullptr;
    P.save = sv->kind;
    P.r = sv->r;
    P.u = sv->u;
    P.ldr = sv->ld;
    P.rs = sv->r_scales;
    P.us = sv->u_scales;
    P.lds = sv->lds;
    P.err = err;
    if (launch_dense(P, kEpiDGated, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
  }
  // dX, dWg, dWu and dWd in one launch (they all wait for dG, dU and H only), dX's long tiles
  // first; db is added up by its epilogue warps while they wait for the first tile
  DenseParams P{};
  const DenseProblem *split = nullptr;
  if (dx) {
    DenseProblem &Q = P.p[P.count++];
    const Operand ag{dg, ldh, false}, au{du, ldh, false}, bg{q->w_gate, q->ld_gate, true}, bu{q->w_up, q->ld_up, true};
    if (!set_problem(Q, ag, bg, T, d, n, dx, d) || !set_pair(Q, 1, au, bu, T, d, n)) return SFNN_ERR_CUDA;
    Q.nk += chunks(n);
    Q.split = parts_of(T, d, Q.nk, sms);
    Q.part = parts;
    split = &Q;
  }
  const Operand tg{dg, ldh, true}, tu{du, ldh, true}, th{h, ldh, true}, ty{dy, lddy, true};
  if (dw_gate && !set_problem(P.p[P.count++], tg, x, n, d, T, dw_gate, d)) return SFNN_ERR_CUDA;
  if (dw_up && !set_problem(P.p[P.count++], tu, x, n, d, T, dw_up, d)) return SFNN_ERR_CUDA;
  if (dw_down && !set_problem(P.p[P.count++], ty, th, d, n, T, dw_down, n)) return SFNN_ERR_CUDA;
  const int blocks = (int)row_blocks(T);
  if (P.count) {
    P.bf16 = bf16;
    P.err = err;
    P.colpart = colpart;
    P.colsum = static_cast<uint16_t *>(db);
    P.col_blocks = blocks;
    P.cols = n;
    if (launch_dense(P, kEpiStore, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
    if (split && join(*split, bf16, sms, s) != cudaSuccess) return SFNN_ERR_CUDA;
  } else if (db && launch_colsum(colpart, blocks, n, bf16, db, s) != cudaSuccess) {
    return SFNN_ERR_CUDA;
  }
  return SFNN_OK;
}

sfnn_status sfnn_forward_prompt(sfnn_handle h, const void *X, int32_t T, float *Y, void *ws, int64_t ws_bytes,
                                sfnn_stream_t stream) {
  if (!h || T < 0) return SFNN_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != h->device) return SFNN_ERR_INVALID_ARG;
  const Layout &L = h->L;
  if (L.dt != SFNN_F16 || L.rows_q) return SFNN_ERR_UNSUPPORTED;
  if (T == 0) return SFNN_OK;
  const uint16_t *rows = static_cast<const uint16_t *>(h->rows);
  const int64_t ld = (int64_t)L.nproj * L.d;
  if (L.act == SFNN_REGLU) {
    sfnn_gated_desc q{};
    q.T = T;
    q.d = L.d;
    q.n = L.n;
    q.dtype = SFNN_F16;
    q.down_layout = SFNN_DOWN_NEURON_MAJOR;
    q.x = X;
    q.ldx = L.d;
    q.w_gate = rows;
    q.w_up = rows + L.d;
    q.w_down = rows + 2 * (int64_t)L.d;
    q.ld_gate = q.ld_up = q.ld_down = ld;
    q.b = h->bias;
    int kernels = 0;
    const sfnn_status st = forward(&q, Y, L.d, SFNN_F32, nullptr, ws, ws_bytes, h->err, stream, kernels);
    h->launches += kernels;
    return st;
  }
  if (!mat_ok(X, L.d, L.d) || !Y || !a16(Y) || !ws || !a16(ws) || ws_bytes < sfnn_gated_workspace(T, L.d, L.n, 0))
    return SFNN_ERR_INVALID_ARG;
  if (T > (1 << 24)) return SFNN_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float *parts = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + hidden_bytes(T, L.n));
  const Operand x{X, L.d, false}, wu{rows, ld, false}, hh{ws, up(L.n, 8), false}, wd{rows + L.d, ld, true};
  int kernels = 0;
  sfnn_status st = product(x, wu, T, L.n, L.d, ws, up(L.n, 8), 0, 0, nullptr, h->err, s, kernels, h->bias);
  if (st == SFNN_OK) st = product(hh, wd, T, L.d, L.n, Y, L.d, 1, 0, parts, h->err, s, kernels);
  h->launches += kernels;
  return st;
}

}  // extern "C"
