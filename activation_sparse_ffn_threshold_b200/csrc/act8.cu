// act8.cu -- 16-bit rows to 8-bit blocks and back (the format is in dense.cuh).
//
// Bound by bytes: 2 read + 1.0625 written per value (and back).  A warp takes 2048 columns
// of one row: every lane requests up to eight 16-byte vectors before it uses the first, so
// a row's bytes are in flight together; eight neighbouring lanes hold one 64-value block
// and find its largest magnitude with three shuffles, so a value is read once.
//
// Measured, relu, 8192 x 11008 bf16: 61 us to quantise (of 42 at the copy rate: 0.74 of the
// issue slots go to codes), 44 to restore, 106 there and back.
#include "dense.cuh"
#include "launch.cuh"

namespace sfnn {
namespace {

constexpr int kWarps = 8;
constexpr int kVecs = 8;               // 8-value vectors per lane
constexpr int kChunk = 32 * kVecs * 8;  // columns per warp

// Rows that do not start on 16 bytes are read and written by aligned 16-byte vectors all the
// same: a lane's 8 values lie across its vector and the next lane's.  A read touches only
// vectors that hold a value of the row; a write leaves the row's ragged ends to single stores.

// 8 halves from half `k` (0..7) on of the 16 in s: s[0..3] is the result.
__device__ __forceinline__ void shift_halves(uint32_t s[8], int k) {
  if (k & 4)
#pragma unroll
    for (int j = 0; j < 6; ++j) s[j] = s[j + 2];
  if (k & 2)
#pragma unroll
    for (int j = 0; j < 5; ++j) s[j] = s[j + 1];
  if (k & 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = __funnelshift_r(s[j], s[j + 1], 16);
}
__device__ __forceinline__ uint4 ld16_stream(const void *p) {
  uint4 w;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
  return w;
}
// The aligned vector at p if it holds a byte of [lo, hi).
__device__ __forceinline__ uint4 ld16_within(uintptr_t p, uintptr_t lo, uintptr_t hi) {
  return p < hi && p + 16 > lo ? ld16_stream(reinterpret_cast<const void *>(p)) : make_uint4(0, 0, 0, 0);
}

// relu of two 16-bit values (NaNs stay)
template <bool bf16>
__device__ __forceinline__ uint32_t relu16(uint32_t w) {
  if (bf16) {
    const __nv_bfloat162 v = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&w), __floats2bfloat162_rn(0.f, 0.f));
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __hmax2_nan(*reinterpret_cast<const __half2 *>(&w), __floats2half2_rn(0.f, 0.f));
  return *reinterpret_cast<const uint32_t *>(&v);
}

// ALIGNED: every row starts on 16 bytes
template <bool RELU, bool bf16, bool ALIGNED>
__global__ void __launch_bounds__(kWarps * 32)
    k_act8_quantize(const uint16_t *__restrict__ x, int64_t ldx, int T, int cols,
                    uint8_t *__restrict__ codes, int64_t ldq, float *__restrict__ scales, int64_t lds) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= T) return;
  const int c0 = blockIdx.y * kChunk + lane * 8;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(x + row * ldx), hi = lo + (uintptr_t)cols * 2;
  const int k = ALIGNED ? 0 : (int)(lo & 15u) >> 1;  // the row's first value within its vector
  const uintptr_t at = lo - 2 * k + (uintptr_t)c0 * 2;
  uint4 w[kVecs], last[ALIGNED ? 1 : kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (ALIGNED) {
      w[i] = make_uint4(0, 0, 0, 0);
      if (c0 + i * 256 < cols) w[i] = ld16_stream(reinterpret_cast<const void *>(at + i * 512));
    } else {
      w[i] = ld16_within(at + i * 512, lo, hi);
    }
    if (!ALIGNED) {
      last[ALIGNED ? 0 : i] = make_uint4(0, 0, 0, 0);
      if (k && lane == 31) last[ALIGNED ? 0 : i] = ld16_within(at + i * 512 + 16, lo, hi);
    }
  }
  const int end = (cols + kAct8Block - 1) / kAct8Block * kAct8Block;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = c0 + i * 256;
    uint32_t a[8] = {w[i].x, w[i].y, w[i].z, w[i].w, 0, 0, 0, 0};
    if (!ALIGNED && k) {  // (the whole warp: a row)
      const uint4 l = last[ALIGNED ? 0 : i];
      const uint32_t e[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[4 + j] = __shfl_down_sync(0xffffffffu, a[j], 1);
        if (lane == 31) a[4 + j] = e[j];
      }
      shift_halves(a, k);
    }
    if ((!ALIGNED || (cols & 7)) && cols - c < 8)  // the next row's values, or none
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c + 2 * j >= cols) a[j] = 0;
        if (c + 2 * j + 1 >= cols) a[j] &= 0xffffu;
      }
    // relu and the block's largest magnitude on pairs of 16-bit values (their bit patterns order
    // like their magnitudes, NaNs above infinities)
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (RELU) a[j] = relu16<bf16>(a[j]);
      m = __vmaxu2(m, a[j] & 0x7fff7fffu);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (c >= end) continue;
    const uint32_t top = max(m & 0xffffu, m >> 16);
    const Act8Scale s = act8_scale(__float_as_uint(unpack16(top, bf16).x), RELU ? 255.f : 127.f);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16(a[j], bf16);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
    uint32_t q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      q[j] = act8_codes<RELU>(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], s.inv);
      if (RELU)  // a relu'd value is positive where its bits are not zero
        q[j] = act8_lift(q[j], __byte_perm(__vminu2(a[2 * j], 0x00010001u), __vminu2(a[2 * j + 1], 0x00010001u), 0x6420));
    }
    *reinterpret_cast<uint2 *>(codes + row * ldq + c) = make_uint2(q[0], q[1]);
    if ((lane & 7) == 0) scales[row * lds + (c >> 6)] = s.scale;
  }
}

// Values [from, to) of 8 halves to p.
__device__ __forceinline__ void store_halves(uint16_t *p, const uint32_t o[4], int from, int to) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j >= from && j < to) p[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
}

template <bool RELU, bool bf16, bool ALIGNED>
__global__ void __launch_bounds__(kWarps * 32)
    k_act8_restore(const uint8_t *__restrict__ codes, int64_t ldq, const float *__restrict__ scales, int64_t lds, int T,
                   int cols, uint16_t *__restrict__ out, int64_t ldo) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= T) return;
  const int c0 = blockIdx.y * kChunk + lane * 8;
  uint2 w[kVecs];
  float s[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = c0 + i * 256;
    if (!ALIGNED) {
      w[i] = make_uint2(0, 0);
      s[i] = 0.f;
    }
    if (c < cols) {
      w[i] = __ldg(reinterpret_cast<const uint2 *>(codes + row * ldq + c));
      s[i] = __ldg(scales + row * lds + (c >> 6));
    }
  }
  const int m = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(out + row * ldo) & 15u) >> 1;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = c0 + i * 256;
    if (ALIGNED ? c >= cols : c - lane * 8 >= cols) break;  // (unaligned: the whole warp)
    const uint32_t a[2] = {w[i].x, w[i].y};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = (a[j >> 1] >> (16 * (j & 1))) & 0xffu, hi = (a[j >> 1] >> (16 * (j & 1) + 8)) & 0xffu;
      o[j] = RELU ? pack16((float)lo * s[i], (float)hi * s[i], bf16)
                  : pack16((float)(int8_t)lo * s[i], (float)(int8_t)hi * s[i], bf16);
    }
    // this lane's 8 values begin at half m of an aligned vector: that vector holds the last m
    // of the lane before and the first 8 - m of this one
    const int valid = min(8, cols - c);
    uint16_t *p = out + row * ldo + c;
    if (ALIGNED || m == 0) {
      if (valid == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
      else
        store_halves(p, o, 0, valid);
    } else {
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = __shfl_up_sync(0xffffffffu, o[j], 1);
        v[4 + j] = o[j];
      }
      shift_halves(v, 8 - m);
      if (valid > 0) {
        if (lane > 0 && valid >= 8 - m)
          *reinterpret_cast<uint4 *>(p - m) = make_uint4(v[0], v[1], v[2], v[3]);
        else if (lane > 0) {  // the row ends within the vector
          uint32_t b[4] = {v[0], v[1], v[2], v[3]};
          store_halves(p - m, b, 0, m + valid);
        } else {
          store_halves(p, o, 0, min(valid, 8 - m));
        }
        // the values behind this lane's vector, where no next lane takes them
        if (lane == 31 || valid < 8 || cols - c == 8) store_halves(p, o, 8 - m, valid);
      }
    }
  }
}

bool aligned16(const void *p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }
dim3 grid_of(int64_t T, int64_t cols) {  // (either may be near 2^31)
  return dim3((unsigned)((T + kWarps - 1) / kWarps), (unsigned)((cols + kChunk - 1) / kChunk));
}

}  // namespace

cudaError_t launch_act8_quantize(const void *x, int64_t ldx, int T, int cols, int bf16, bool relu, uint8_t *codes,
                                 int64_t ldq, float *scales, int64_t lds, cudaStream_t s) {
  auto run = [&](auto *k) {
    return launch_pdl(k, grid_of(T, cols), dim3(kWarps * 32), 0, s, static_cast<const uint16_t *>(x), ldx, T, cols, codes,
                      ldq, scales, lds);
  };
  if (aligned16(x, ldx))
    return relu ? (bf16 ? run(k_act8_quantize<true, true, true>) : run(k_act8_quantize<true, false, true>))
                : (bf16 ? run(k_act8_quantize<false, true, true>) : run(k_act8_quantize<false, false, true>));
  return relu ? (bf16 ? run(k_act8_quantize<true, true, false>) : run(k_act8_quantize<true, false, false>))
              : (bf16 ? run(k_act8_quantize<false, true, false>) : run(k_act8_quantize<false, false, false>));
}

cudaError_t launch_act8_restore(const uint8_t *codes, int64_t ldq, const float *scales, int64_t lds, int T, int cols,
                                bool relu, int bf16, void *out, int64_t ldo, cudaStream_t s) {
  auto run = [&](auto *k) {
    return launch_pdl(k, grid_of(T, cols), dim3(kWarps * 32), 0, s, codes, ldq, scales, lds, T, cols,
                      static_cast<uint16_t *>(out), ldo);
  };
  if (aligned16(out, ldo))
    return relu ? (bf16 ? run(k_act8_restore<true, true, true>) : run(k_act8_restore<true, false, true>))
                : (bf16 ? run(k_act8_restore<false, true, true>) : run(k_act8_restore<false, false, true>));
  return relu ? (bf16 ? run(k_act8_restore<true, true, false>) : run(k_act8_restore<true, false, false>))
              : (bf16 ? run(k_act8_restore<false, true, false>) : run(k_act8_restore<false, false, false>));
}

}  // namespace sfnn

extern "C" {

static sfnn_status act8_check(const void *x, int64_t ldx, int32_t T, int32_t cols, int32_t dtype, const void *codes,
                              int64_t ldq, const void *scales, int64_t lds) {
  if (T < 0 || cols < 1 || (dtype != SFNN_F16 && dtype != SFNN_BF16)) return SFNN_ERR_INVALID_ARG;
  const int64_t blocks = ((int64_t)cols + SFNN_ACT8_BLOCK - 1) / SFNN_ACT8_BLOCK;
  if (ldx < cols || ldq < blocks * SFNN_ACT8_BLOCK || ldq % 16 || lds < blocks) return SFNN_ERR_INVALID_ARG;
  if (T == 0) return SFNN_OK;
  if (!x || !codes || !scales) return SFNN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(codes) & 15u) || (reinterpret_cast<uintptr_t>(scales) & 3u) ||
      (reinterpret_cast<uintptr_t>(x) & 1u))
    return SFNN_ERR_INVALID_ARG;
  if (((int64_t)cols + sfnn::kChunk - 1) / sfnn::kChunk > 65535) return SFNN_ERR_UNSUPPORTED;
  return SFNN_OK;
}

sfnn_status sfnn_act8_quantize(const void *x, int64_t ldx, int32_t T, int32_t cols, int32_t dtype, int32_t relu,
                               void *codes, int64_t ldq, float *scales, int64_t lds, sfnn_stream_t stream) {
  const sfnn_status st = act8_check(x, ldx, T, cols, dtype, codes, ldq, scales, lds);
  if (st != SFNN_OK || T == 0) return st;
  return sfnn::launch_act8_quantize(x, ldx, T, cols, dtype == SFNN_BF16, relu != 0, static_cast<uint8_t *>(codes), ldq,
                                    scales, lds, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SFNN_OK
             : SFNN_ERR_CUDA;
}

sfnn_status sfnn_act8_restore(const void *codes, int64_t ldq, const float *scales, int64_t lds, int32_t T, int32_t cols,
                              int32_t relu, int32_t dtype, void *out, int64_t ldo, sfnn_stream_t stream) {
  const sfnn_status st = act8_check(out, ldo, T, cols, dtype, codes, ldq, scales, lds);
  if (st != SFNN_OK || T == 0) return st;
  return sfnn::launch_act8_restore(static_cast<const uint8_t *>(codes), ldq, scales, lds, T, cols, relu != 0,
                                   dtype == SFNN_BF16, out, ldo, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SFNN_OK
             : SFNN_ERR_CUDA;
}

}  // extern "C"
