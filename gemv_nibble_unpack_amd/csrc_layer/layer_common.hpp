// Shared helpers of the decoder-layer operators (residual norm, cache append,
// attention over the 8-bit cache): loads widened to float32, 8-bit codes.
#pragma once

#include "common.hpp"
#include "gemv_nibble_unpack_layer.h"

namespace w4 {

typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f2v __attribute__((ext_vector_type(2)));

constexpr uint32_t F32_INF = 0x7F800000u;
// float bits of |x|: as unsigned integers these order like the magnitudes,
// with infinity above every finite value and NaN above infinity, so an integer
// max over them finds the largest magnitude and cannot lose a NaN
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}
// wave-wide unsigned max and float sum: the 16-lane rows on DPP, the four rows
// through scalars. Every lane of the wave must be active.
__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
  v = max(v, dpp_u<0xB1>(v));
  v = max(v, dpp_u<0x4E>(v));
  v = max(v, dpp_u<0x141>(v));
  v = max(v, dpp_u<0x140>(v));
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)v, 0),
                         (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)v, 32),
                         (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
  return max(a, b);
}
__device__ __forceinline__ float lane_f(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ float wave_sum_f(float v) {
  v = row_sum16(v);
  return (lane_f(v, 0) + lane_f(v, 16)) + (lane_f(v, 32) + lane_f(v, 48));
}

// eight / four consecutive elements widened to float32 (fp16 is uint16_t)
__device__ __forceinline__ void load8f(const uint16_t* p, float (&x)[8]) {
  const h8 h = __builtin_bit_cast(h8, *reinterpret_cast<const u4*>(p));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)h[i];
}
__device__ __forceinline__ void load8f(const float* p, float (&x)[8]) {
  const f4 a = *reinterpret_cast<const f4*>(p), b = *reinterpret_cast<const f4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = a[i];
    x[4 + i] = b[i];
  }
}
__device__ __forceinline__ void store8f(uint16_t* p, const float (&x)[8]) {
  h8 h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (_Float16)x[i];
  *reinterpret_cast<u4*>(p) = __builtin_bit_cast(u4, h);
}
__device__ __forceinline__ void store8f(float* p, const float (&x)[8]) {
  *reinterpret_cast<f4*>(p) = f4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f4*>(p + 4) = f4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ f4 load4f(const uint16_t* p) {
  const h4 h = __builtin_bit_cast(h4, *reinterpret_cast<const u2*>(p));
  return f4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
}
__device__ __forceinline__ f4 load4f(const float* p) { return *reinterpret_cast<const f4*>(p); }
__device__ __forceinline__ f2v load2f(const uint16_t* p) {
  const h2 h = *reinterpret_cast<const h2*>(p);
  return f2v{(float)h[0], (float)h[1]};
}
__device__ __forceinline__ f2v load2f(const float* p) { return *reinterpret_cast<const f2v*>(p); }

// Four 8-bit codes of y (already divided by the scale), packed little-endian.
// y is clamped to the code range first: it can exceed it by a rounding, and by
// more where the scale itself was a subnormal.
//   INT8: half-to-even by adding 1.5 * 2^23, where the floats are the
//   integers; the low byte of the sum's bits is the code in two's complement.
//   E4M3: the hardware conversion (round to nearest even).
template <int Q>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
#pragma clang fp contract(off)
  if constexpr (Q == W4_Q_I8) {
    constexpr float R = 12582912.0f;
    const uint32_t ua = __float_as_uint(__builtin_amdgcn_fmed3f(a, -127.f, 127.f) + R),
                   ub = __float_as_uint(__builtin_amdgcn_fmed3f(b, -127.f, 127.f) + R),
                   uc = __float_as_uint(__builtin_amdgcn_fmed3f(c, -127.f, 127.f) + R),
                   ud = __float_as_uint(__builtin_amdgcn_fmed3f(d, -127.f, 127.f) + R);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(ud, uc, 0x0c0c0400u),
                                 __builtin_amdgcn_perm(ub, ua, 0x0c0c0400u), 0x05040100u);
  } else {
    a = __builtin_amdgcn_fmed3f(a, -448.f, 448.f);
    b = __builtin_amdgcn_fmed3f(b, -448.f, 448.f);
    c = __builtin_amdgcn_fmed3f(c, -448.f, 448.f);
    d = __builtin_amdgcn_fmed3f(d, -448.f, 448.f);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  }
}

// the values of four codes, in units of the scale
template <int Q>
__device__ __forceinline__ f4 decode4(uint32_t w) {
  if constexpr (Q == W4_Q_I8) {
    return f4{(float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16),
              (float)(int8_t)(w >> 24)};
  } else {
    const f2v lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f2v hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return f4{lo[0], lo[1], hi[0], hi[1]};
  }
}

// Grids of more blocks than one dimension launches (fewer than 2^32 threads along
// x): rows of GRID_X blocks, read with block_number(). The last row may have blocks past the end, which
// the kernels must leave without work.
constexpr int GRID_X = 1 << 21;
constexpr int64_t MAX_BLOCKS = 0x7fffffff;
inline dim3 grid_of(int64_t blocks) {
  if (blocks <= GRID_X) return dim3((unsigned)blocks);
  return dim3(GRID_X, (unsigned)((blocks + GRID_X - 1) / GRID_X));
}
__device__ __forceinline__ int block_number() { return blockIdx.y * GRID_X + blockIdx.x; }

inline bool kv8_page_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

}  // namespace w4
