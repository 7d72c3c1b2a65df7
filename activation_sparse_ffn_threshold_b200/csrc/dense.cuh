// dense.cuh -- the dense tensor-core product shared by the gated FFN's forward and
// backward: its parameters and host launcher, and the 8-bit block format its epilogues
// write and read.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "sfnn.h"
#include "umma.cuh"

namespace sfnn {

// ---------------------------------------------------------------- 16-bit elements
__device__ __forceinline__ uint32_t pack16(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 unpack16(uint32_t w, bool bf16) {
  if (bf16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float load16(const void *p, int64_t i, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : __half2float(static_cast<const __half *>(p)[i]);
}

// ---------------------------------------------------------------- act8
// 64 values of a row share an fp32 scale: max|v| / 127 with codes -127..127, or for
// relu(v) max / 255 with codes 0..255.  A code is the integer nearest to v / scale, the even one
// where two are equally near (or within 2^-16 of it).  A
// positive relu'd value keeps a code of at least 1: code > 0 is exactly the ReLU's mask,
// which the backward pass needs.  A block with a NaN or an infinity gets a NaN scale (and so
// restores as NaN); a block whose largest magnitude is below 2^-112 gets scale 0.
constexpr int kAct8Block = 64;

struct Act8Scale {
  float scale, inv;
};
// `top`: the largest fp32 bit pattern of the block's magnitudes (NaN > inf > finite); below
// 2^-112 the reciprocal could overflow.  inv = qmax / top to half an ulp: an approximate
// reciprocal and a Newton step, whose residual is exact.
__device__ __forceinline__ Act8Scale act8_scale(uint32_t top, float qmax) {
  Act8Scale s;
  float r;
  s.scale = __uint_as_float(top) * (1.f / qmax);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s.scale));
  s.inv = fmaf(fmaf(-__uint_as_float(top), r, qmax), r * (1.f / qmax), r);
  if (top < 0x07800000u) s.scale = s.inv = 0.f;
  if (top >= 0x7f800000u) s.scale = __uint_as_float(0x7fffffffu);
  return s;
}

// Codes of four values as bytes.  16-bit values and their block's largest often meet where
// v / scale lies exactly between two codes, and v * inv, off by up to 2^-24 of itself, would fall to
// either side (2.3e-4 of normal fp16 values' codes).  v * inv + 384 (256 where no value is
// negative) is one fused multiply-add whose sum has a step of 2^-15, so that such a quotient is
// exact again; adding 1.5 * 2^23 less that then leaves the nearest integer, ties to even, in the
// low byte.  |v * inv| <= qmax (1 + 2^-23), so no code leaves its range; in a NaN block the codes
// mean nothing.
template <bool RELU>
__device__ __forceinline__ uint32_t act8_codes(float a, float b, float c, float d, float inv) {
  constexpr float kGrid = RELU ? 256.f : 384.f, kMagic = 12582912.f - kGrid;
  const uint32_t x = __float_as_uint(fmaf(a, inv, kGrid) + kMagic), y = __float_as_uint(fmaf(b, inv, kGrid) + kMagic);
  const uint32_t z = __float_as_uint(fmaf(c, inv, kGrid) + kMagic), w = __float_as_uint(fmaf(d, inv, kGrid) + kMagic);
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}
// ... and of four relu'd values: a positive one whose code is 0 gets code 1 (`positive`: bit 0
// of each byte whose value is positive).
__device__ __forceinline__ uint32_t act8_lift(uint32_t codes, uint32_t positive) {
  const uint32_t some = ((codes & 0x7f7f7f7fu) + 0x7f7f7f7fu) | codes;  // bit 7 of each byte that is not zero
  return codes | (positive & ~(some >> 7));
}

// ---------------------------------------------------------------- the saved hidden layer in 16 bits
// What the forward pass keeps at full precision: blocks of 64 that share a power of two P, the
// one at or below the block's largest magnitude (at least 2^-101), and 16 bits a value, a float
// with more mantissa where most values lie: U a sign and 12 bits of mantissa in the three octaves
// from P / 4 up, 11 in the nine below them, and equal steps from 2^-11 P on down; relu(G), never
// negative, one bit more.  So U is off by at most 2^-13 of itself, 2^-12 below P / 4, and 2^-23 P
// below 2^-11 P, relu(G) by half of that: a neuron keeps its precision beside one thousands of
// times as large, and loses less than fp16 would round it by (2^-11) down to 2^-12 P.  Of a
// gradient's error, what is left is the rounding of dG, dU or H to the tensor cores' type, and its
// own.  A positive relu(G) keeps a code of at least 1: code > 0 is exactly the ReLU's mask.
// (Fixed point holds values of like size better, to 2^-17 of the largest, but one 2^-12 of it to
// four bits.  Gradients of an fp16 step of 257 tokens are 0.00030 off 64 bits with either, most of
// it the roundings to fp16; with 11 bits of mantissa throughout 0.00031.)
//
// The codes come from an fp32 number's bits, scaled so that P has the exponent field 12 and
// fp32's own subnormal numbers are the small values' equal steps: its bits from the 11th
// mantissa bit up count the lower octaves' codes, those from the 12th up the upper octaves', less
// what puts both at one code where they meet; the larger of the two is the code.
// The scaling takes two multiplications, as one power of two would leave fp32's range.
constexpr float kCodeDown = 1.1754943508222875e-38f;  // 2^-126
constexpr float kCodeUp = 8.507059173023462e37f;      // 2^126
constexpr uint32_t kCodeLow = 26;                     // the smallest block exponent (biased): 2^-101
constexpr uint32_t kMeet = 10u << 11;                 // the code where the octaves meet (twice that for relu(G))
struct Code16Scale {
  float scale, to;  // P; what a value is multiplied by, before kCodeDown
};
// `half`: half a step of the upper octaves in a mantissa's bits (a largest value that rounds up to a
// power of two takes that one as P).
__device__ __forceinline__ Code16Scale code16_scale(uint32_t top, uint32_t half) {
  const uint32_t e = max((top + half) >> 23, kCodeLow);
  Code16Scale s;
  s.scale = __uint_as_float(e >= 255u ? 0x7fffffffu : e << 23);
  s.to = __uint_as_float((265u - e) << 23);  // 2^(138 - e); of a block that is not finite the codes mean nothing
  return s;
}
constexpr uint32_t kHalfU = 0x400u, kHalfR = 0x200u;
__device__ __forceinline__ float code16_from(float scale) { return scale * 0x1p-11f; }  // 2^(e - 138)
__device__ __forceinline__ uint32_t code16_pair(float a, float b, float to) {  // signed
  auto code = [&](float v) {
    const uint32_t x = __float_as_uint(fabsf(v) * to * kCodeDown);
    return (uint32_t)max((int)(x + 0x800u) >> 12, ((int)(x + kHalfU) >> 11) - (int)kMeet);
  };
  const uint32_t sign = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632) & 0x80008000u;
  return __byte_perm(code(a), code(b), 0x5410) | sign;
}
__device__ __forceinline__ uint32_t code16_pair_relu(float a, float b, float to) {
  auto code = [&](float v) {
    const uint32_t x = __float_as_uint(v * to * kCodeDown);
    const int c = max((int)(x + 0x400u) >> 11, ((int)(x + kHalfR) >> 10) - (int)(2u * kMeet));
    return (uint32_t)max(c, v > 0.f ? 1 : 0);
  };
  return __byte_perm(code(a), code(b), 0x5410);
}
// The values of a word of two codes (`from`: code16_from of the block's scale).
__device__ __forceinline__ float2 code16_values(uint32_t w, float from) {
  auto value = [&](uint32_t half) {  // the code in the upper half of a word
    const uint32_t c = (half >> 5) & 0x03fff800u;
    return __uint_as_float(min(2u * c, c + (kMeet << 11)) | (half & 0x80000000u)) * kCodeUp * from;
  };
  return make_float2(value(w << 16), value(w));
}
__device__ __forceinline__ float2 code16_values_relu(uint32_t w, float from) {
  auto value = [&](uint32_t half) {
    const uint32_t c = (half >> 6) & 0x03fffc00u;
    return __uint_as_float(min(2u * c, c + (kMeet << 11))) * kCodeUp * from;
  };
  return make_float2(value(w << 16), value(w));
}

// ---------------------------------------------------------------- the product
// C = sum over up to two (A, B) pairs of A . B^T, tiles of 256 x 256 by CTA pairs.
enum DenseEpi : int {
  kEpiStore = 0,  // C as 16-bit or fp32 values
  kEpiGated = 1,  // B0 = gate rows, B1 = up rows (128 each per tile): H = relu(G + b) * U
  kEpiDGated = 2,  // C = dH: dU = dH * R, dG = dH * U * [R > 0], H = R * U
  kEpiDGated8 = 3,  // the same with R and U held as 8-bit blocks
  kEpiLinear = 4,  // act(C + bias) + residual, 16-bit
  kEpiLinear32 = 5  // the same as fp32, K summed up in segments
};

// The end of a linear layer: Y = act(Z + bias) + residual, and what the backward pass needs of act'.
struct LinearEnd {
  const void *bias;  // [N] or null
  const void *res;   // [M x N] of the output's type, or null
  int64_t ldres;
  int act;           // sfnn_linear_act
  void *slopes;      // or null: act'(Z) as it is kept (below)
  int vec_out, vec_res;  // rows of whole 16-byte pieces
};

// What is kept of act': of a ReLU a bit per value (a value above zero, or a NaN), 32 columns a word,
// rows of whole 128 columns; of the others 16-bit fixed point, code = 2^15 act' + 2^14, which holds
// act' (-0.13 to 1.13) to 2^-16, where the type would round it as often as the result itself; 0xffff
// is a NaN.  Rows of whole 32 columns.
__host__ __device__ inline int64_t slope_row_bytes(int64_t N, int act) {
  return act == SFNN_LINEAR_NONE ? 0 : act == SFNN_LINEAR_RELU ? (N + 127) / 128 * 16 : (N + 31) / 32 * 64;
}
// Pairs of fp32 values in a 64-bit register, one instruction for both.  (Kept as such from the load to
// the store: taken apart in between, every instruction is joined by moves.)
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ float2 apart(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ float within(Pair p) {
  const float2 v = apart(p);
  return v.x + v.y;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// act(z) and, where `keep`, the code of act'(z) of the smooth ones in a word's lower half; the limits
// at the infinities, NaN for a NaN.
//
// gelu: z Phi(z), Phi the normal distribution's integral.  Phi(-a) e^(a^2 / 2) is smooth from 1/2 at
// a = 0 to 0; it is taken as a polynomial of degree 8 in t = 1 / (1 + 0.295 a), fitted to its smallest
// relative error over a in [0, 14] (3.7e-8; with the roundings 1e-6 down to z = -5, 5e-6 of 1e-38 at
// -13), and times the e^(-z^2 / 2) that Phi' takes too: two special functions and a dozen
// multiply-adds, most of them two values to an instruction
// (1999 tokens, 4096 x 16384: 399 us with CUDA's normcdff, 230 without an activation).
// silu: z / (1 + e^-z).
__device__ __forceinline__ float max_nan(float a, float b) {
  float v;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float v;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float exp2_approx(float v) {
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v));
  return v;
}
__device__ __forceinline__ float rcp_approx(float v) {
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(v));
  return v;
}
template <bool GELU, bool KEEP>
__device__ __forceinline__ void smooth_values(float &z0, float &z1, uint32_t &code0, uint32_t &code1) {
  // (both results are 0 from there on: e^88 is beyond 2^126, its reciprocal flushed; silu is off by 88 2^-126 at most)
  const float low0 = max_nan(z0, -88.f), low1 = max_nan(z1, -88.f);
  // (with a slope both are finite: 0 or 1 beyond)
  const float b0 = KEEP ? min_nan(low0, 80.f) : low0, b1 = KEEP ? min_nan(low1, 80.f) : low1;
  const Pair b = pair(b0, b1);
  float p0, p1, s0, s1;
  if (GELU) {
    const float2 x = apart(mul2(mul2(b, b), pair(-0.7213475204f, -0.7213475204f)));
    const Pair e = pair(exp2_approx(x.x), exp2_approx(x.y));
    const Pair t = pair(rcp_approx(fmaf(0.295f, fabsf(b0), 1.f)), rcp_approx(fmaf(0.295f, fabsf(b1), 1.f)));
    Pair q = fma2(pair(0.0394212678f, 0.0394212678f), t, pair(-0.183406666f, -0.183406666f));
    q = fma2(q, t, pair(0.271017522f, 0.271017522f));
    q = fma2(q, t, pair(-0.117072001f, -0.117072001f));
    q = fma2(q, t, pair(0.166289508f, 0.166289508f));
    q = fma2(q, t, pair(0.0847446173f, 0.0847446173f));
    q = fma2(q, t, pair(0.12169943f, 0.12169943f));
    q = fma2(q, t, pair(0.117289335f, 0.117289335f));
    q = mul2(fma2(q, t, pair(1.7007178e-05f, 1.7007178e-05f)), e);
    const float2 r = apart(q);
    p0 = b0 > 0.f ? 1.f - r.x : r.x;
    p1 = b1 > 0.f ? 1.f - r.y : r.y;
    if (KEEP) {
      const float2 s = apart(fma2(mul2(b, pair(0.3989422804f, 0.3989422804f)), e, pair(p0, p1)));
      s0 = s.x, s1 = s.y;
    }
  } else {
    const float2 x = apart(mul2(b, pair(-1.4426950409f, -1.4426950409f)));
    p0 = rcp_approx(1.f + exp2_approx(x.x));
    p1 = rcp_approx(1.f + exp2_approx(x.y));
    if (KEEP) {
      s0 = p0 * fmaf(b0, 1.f - p0, 1.f);
      s1 = p1 * fmaf(b1, 1.f - p1, 1.f);
    }
  }
  if (KEEP) {  // the sum's last bit is worth 1; a NaN's lower half is 0xffff
    code0 = __float_as_uint(fmaf(s0, 32768.f, 8388608.f + 16384.f));
    code1 = __float_as_uint(fmaf(s1, 32768.f, 8388608.f + 16384.f));
  }
  z0 = low0 * p0;
  z1 = low1 * p1;
}
// The same for N values.  The choice stands outside: made value by value it kept their chains of
// multiply-adds from running beside one another (8192 tokens, 512 -> 8192, GELU: 208 us, 148 so).
template <int N>
__device__ __forceinline__ void act_values(float *v, int act, bool keep, uint32_t *code) {
  auto all = [&](auto gelu, auto kept) {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      smooth_values<decltype(gelu)::value, decltype(kept)::value>(v[i], v[i + 1], code[i], code[i + 1]);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (act == SFNN_LINEAR_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = max_nan(v[i], 0.f);
  } else if (act == SFNN_LINEAR_GELU) {
    keep ? all(Yes{}, Yes{}) : all(Yes{}, No{});
  } else if (act == SFNN_LINEAR_SILU) {
    keep ? all(No{}, Yes{}) : all(No{}, No{});
  }
}
__device__ __forceinline__ float slope_value(uint32_t code) {
  return code == 0xffffu ? __uint_as_float(0x7fffffffu) : (float)((int)code - 16384) * 0x1p-15f;
}

struct alignas(64) DenseProblem {
  CUtensorMap a0, b0, a1, b1;
  int M, N;       // rows and columns of C (gated: neurons)
  int nk0, nk;    // K chunks of 64 of the first pair, of both
  int tn;         // columns of a tile: 256, or 128 (never gated); one launch's problems have the same
  int tiles_m, tiles_n;
  int split;      // parts of K, each a unit of work of its own (kEpiStore)
  int a_mn, b_mn; // the operands' majors
  int out32;      // fp32 C
  int relu;       // C = relu(C + bias)
  void *out;      // C, or H
  int64_t ldo;
  float *part;    // split > 1: [split][M][N] fp32 sums instead of C
};
constexpr int kMaxProblems = 4;

struct DenseParams {
  DenseProblem p[kMaxProblems];
  int count;
  // Work of pair `i` of `pairs`: units i, i + pairs, ... of the first problem (its units take
  // longest), then of the others' units, where a pair with one long unit less first takes
  // `extra` more (the host sets it to the two lengths' ratio).
  int first, rest, extra;
  int tall;           // tiles of 512 rows (launch_dense sets it)
  int bf16;
  const void *bias;   // kEpiGated, relu: [N] or null
  int save;           // sfnn_save of r and u
  void *r, *u;        // kEpiGated: written; kEpiDGated: read
  float *rs, *us;
  int64_t ldr, lds;   // their row strides (elements), their scales' row strides
  void *dg, *du;      // kEpiDGated: written, row stride ldo as out (H)
  float *colpart;     // kEpiDGated: [rows / 32][N] sums of dG over 32 rows, or null;
                      // kEpiStore: such sums to add up over `col_blocks` blocks into
  uint16_t *colsum;   // this, of `cols` columns (null: none)
  int col_blocks, cols;
  // kEpiLinear (and bias above): what joins the product on its way out
  LinearEnd end;
  int32_t *err;
};

// The kernel's dynamic shared memory limit on the current device (once per device).
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &ready) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---------------------------------------------------------------- host (product.cu)
int device_sms();  // SMs of the current device (0: no device)

inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
inline int chunks(int64_t K) { return (int)((K + 63) / 64); }
inline bool on(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline bool a16(const void *p) { return on(p, 16); }
bool mat_ok(const void *p, int64_t ld, int64_t cols);  // an operand: aligned rows of 16-bit values

struct Operand {
  const void *p;
  int64_t ld;
  bool mn;  // M or N contiguous, not K
};
bool set_pair(DenseProblem &P, int which, const Operand &a, const Operand &b, int M, int N, int64_t K);
bool set_problem(DenseProblem &P, const Operand &a, const Operand &b, int M, int N, int64_t K, void *out, int64_t ldo,
                 int split = 1, int tn = 256);
int parts_of(int64_t M, int64_t N, int nk, int sms);
int64_t parts_bytes(int64_t M, int64_t N, int nk, int sms);
int tile_columns(int M, int N, int split, int sms);
bool slim_serves(int T, int N, int64_t K, bool gated, int sms);
// What a split product leaves, added up (nothing to do where K was not split).
cudaError_t join(const DenseProblem &P, int bf16, int sms, cudaStream_t s);
// out[c] = sum over the blocks of part[block][c]
cudaError_t launch_colsum(const float *part, int blocks, int n, int bf16, void *out, cudaStream_t s);

// Fills first, rest and extra from the problems.
cudaError_t launch_dense(DenseParams &P, int epi, int num_sms, cudaStream_t s);

// The products of few tokens (slim.cu): out = x . w0^T, or with w1 the gated hidden layer
// relu(x . w0^T + bias) * (x . w1^T).  K-major weights; `early`: w0 may be read while the
// kernel launched before still runs (it waited for everything before it).
struct SlimArgs {
  const void *x, *w0, *w1, *bias;
  int64_t ldx, ldw0, ldw1;
  int T, N;
  int64_t K;
  void *out;
  int64_t ldo;
  int bf16, out32, early;
  int32_t *err;
};
int64_t slim_cost(int T, int N, int64_t K, bool gated, int num_sms);
sfnn_status launch_slim(const SlimArgs &q, int num_sms, cudaStream_t s);

// The linear layer for few tokens (few.cu): weight rows and tokens of a tile, CTAs to a cluster, and the time it
// should take in ns (1e30: it does not take the product).  `words`: a ReLU's slopes are kept; `out32`: an fp32 result.
struct FewPlan {
  int nb, tn, split;
  double cost;
};
FewPlan few_plan(int T, int N, int64_t K, bool words, bool out32, int sms);
struct FewArgs {
  const void *x, *w;
  int64_t ldx, ldw;
  int T, N;
  int64_t K;
  void *out;
  int64_t ldo;
  int bf16, out32;
  const LinearEnd *end;
  int32_t *err;
};
sfnn_status launch_few(const FewArgs &q, const FewPlan &plan, int sms, cudaStream_t s);

// Rows of 16-bit values to act8 blocks and back (act8.cu).  Code rows are ldq bytes apart
// (a multiple of 16, at least T's columns rounded up to 64), scale rows lds floats.
cudaError_t launch_act8_quantize(const void *x, int64_t ldx, int T, int cols, int bf16, bool relu, uint8_t *codes,
                                 int64_t ldq, float *scales, int64_t lds, cudaStream_t s);
cudaError_t launch_act8_restore(const uint8_t *codes, int64_t ldq, const float *scales, int64_t lds, int T, int cols,
                                bool relu, int bf16, void *out, int64_t ldo, cudaStream_t s);

}  // namespace sfnn
