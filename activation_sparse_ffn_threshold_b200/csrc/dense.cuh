// dense.cuh -- the dense tensor-core product shared by the gated FFN's forward and
// backward: its parameters and host launcher, and the 8-bit block format its epilogues
// write and read.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

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
  kEpiDGated8 = 3  // the same with R and U held as 8-bit blocks
};

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

int device_sms();  // SMs of the current device (0: no device)

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

// Rows of 16-bit values to act8 blocks and back (act8.cu).  Code rows are ldq bytes apart
// (a multiple of 16, at least T's columns rounded up to 64), scale rows lds floats.
cudaError_t launch_act8_quantize(const void *x, int64_t ldx, int T, int cols, int bf16, bool relu, uint8_t *codes,
                                 int64_t ldq, float *scales, int64_t lds, cudaStream_t s);
cudaError_t launch_act8_restore(const uint8_t *codes, int64_t ldq, const float *scales, int64_t lds, int T, int cols,
                                bool relu, int bf16, void *out, int64_t ldo, cudaStream_t s);

}  // namespace sfnn
