// Shared pieces of the MXFP4 operators (E2M1 codes, one E8M0 scale for each 32
// elements): the packed weights' layout, the scales, the codes' conversions.
#pragma once

#include "../csrc_layer/layer_common.hpp"
#include "gemv_nibble_unpack_mx.h"

namespace w4 {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef u4 u4_any __attribute__((aligned(1)));       // 16 bytes at any address

// Packed weights: tiles of 16 rows x 128 k, strip (16 rows) by strip. Lane l = 16 g + r
// of a tile holds row r's codes 32 g .. 32 g + 31, 16 bytes as the caller's rows
// have them: one block, so one scale a lane. That is the operand of
// v_mfma_scale_f32_16x16x128_f8f6f4 as it lies; v_mfma_scale_f32_32x32x64 takes
// two strips' tiles, blocks 2 s and 2 s + 1 in its step s. The scales follow, a
// 4-byte word for each lane and four tiles along k (byte kt % 4), then a byte
// for each row: the largest scale of its blocks that are not all zeros, which
// the fp16 products count the scales from.
struct MxGeometry {
  int NT, KT, KQ;
  int64_t s_off, e_off, total;
};
__host__ __device__ inline MxGeometry mx_geometry(int64_t N, int K) {
  MxGeometry g;
  g.NT = (int)((N + 15) / 16);
  g.KT = (K + 127) / 128;
  g.KQ = (g.KT + 3) / 4;
  g.s_off = (int64_t)g.NT * g.KT * TILE_BYTES;
  g.e_off = g.s_off + (int64_t)g.NT * g.KQ * 256;
  g.total = g.e_off + (int64_t)g.NT * 16;
  return g;
}

// Loads from global memory, said to the compiler: of a pointer chosen between a
// tensor and a constant it makes flat loads, which also pass through the LDS side.
#define W4_GLOBAL __attribute__((address_space(1)))
template <typename T>
__device__ __forceinline__ T g_load(const void* p) {
  return *(const W4_GLOBAL T*)p;
}
// base the same for the wave: a scalar base and 32 bits a lane
template <typename T>
__device__ __forceinline__ T g_load(const void* base, uint32_t offset) {
  return *(const W4_GLOBAL T*)((const W4_GLOBAL uint8_t*)base + offset);
}

// 2^(byte - 127), NaN for 255; byte 0 is the subnormal 2^-127
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// the eight codes of a word as float32 / as fp16 times `scale` (a power of two)
__device__ __forceinline__ void fp4_f32(uint32_t w, float (&x)[8]) {
  const f2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const f2v b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const f2v c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const f2v d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1];
  x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
}
__device__ __forceinline__ h8 fp4_h8(uint32_t w, float scale) {
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 0);
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 1);
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 2);
  const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, 3);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The fp16 products take a weight as code * 2^(byte - rowmax + H_UP), at most 6 *
// 2^12 in fp16, and multiply the row's sum by 2^(rowmax - 127 - H_UP): exact
// for blocks down to 2^-35 of the row's largest scale, below that rounded to
// 2^-36 of it (fp16's least subnormal). Blocks of zeros, whose scales rowmax leaves
// out, may lie above it: held at 2^H_UP, since an exponent of 255 would make them NaN.
constexpr int H_UP = 12;
__device__ __forceinline__ float h_scale(uint32_t byte, uint32_t rowmax) {
  const int e = (int)byte - (int)rowmax + 127 + H_UP;
  return byte == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)min(max(e, 1), 127 + H_UP) << 23);
}

}  // namespace w4
