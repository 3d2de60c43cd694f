// MXFP4 coding and decoding, and the weights' packed layout.
//
// A block of 32 has e = floor(log2 max|x|) - 2, so that the largest element lies in
// [4, 8) times 2^e and codes as 4 or 6. x / 2^e is exact in float32 (a
// multiplication by a power of two), so a code is one rounding of the input:
// nearest, ties to the even code, 6 above 5. The block's largest magnitude is an
// integer maximum over the float bits, which also finds infinities and NaN.
// K is a multiple of 32, so a tensor of rows is a string of blocks: thread for
// thread 8 elements, four threads a block.
//
// Bound: bytes. 11008 x 4096 float32 are coded in 45 us and decoded in 32 (204 MB each,
// 4.5 and 6.4 TB/s; a large copy 4.85); one row of 4096 in 1.6 and 1.4.
#include "mx_common.hpp"

namespace w4 {

__device__ __forceinline__ uint32_t quad_max_u(uint32_t v) {
  v = max(v, dpp_u<0xB1>(v));
  return max(v, dpp_u<0x4E>(v));
}

template <typename T>
__global__ __launch_bounds__(256) void k_quantize_mx4(const T* __restrict__ X, int64_t groups,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)block_number() * 256 + threadIdx.x;     // groups of 8
  const bool live = i < groups;
  float x[8];
  load8f(X + 8 * (live ? i : groups - 1), x);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, abs_bits(x[e]));
  m = quad_max_u(m);
  const bool bad = m >= F32_INF;
  const uint32_t byte = bad ? 255u : (uint32_t)max((int)(m >> 23) - 2, 0);
  const float inv = __uint_as_float(bad ? 0u : (254u - byte) << 23);
  uint32_t w = 0;
  if (!bad) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0] * inv, x[1] * inv, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * inv, x[3] * inv, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4] * inv, x[5] * inv, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6] * inv, x[7] * inv, 1.0f, 3);
  }
  if (!live) return;
  *reinterpret_cast<uint32_t*>(codes + 4 * i) = w;
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

template <typename T>
__global__ __launch_bounds__(256) void k_dequantize_mx4(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales,
                                                        int64_t groups, T* __restrict__ Y) {
  const int64_t i = (int64_t)block_number() * 256 + threadIdx.x;
  if (i >= groups) return;
  const float s = e8m0(scales[i >> 2]);
  float x[8];
  fp4_f32(*reinterpret_cast<const uint32_t*>(codes + 4 * i), x);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= s;
  store8f(Y + 8 * i, x);
}

// one wave a tile
__global__ __launch_bounds__(256) void k_prepack_mx4(const uint8_t* __restrict__ codes, int64_t N,
                                                     int K, uint8_t* __restrict__ Wp,
                                                     int64_t tiles) {
  const MxGeometry geo = mx_geometry(N, K);
  const int64_t tile = (int64_t)block_number() * 4 + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t t = tile / geo.KT;
  const int kt = (int)(tile - t * geo.KT);
  const int64_t n = 16 * t + r;
  const int k = 128 * kt + 32 * g;
  u4 w = {0u, 0u, 0u, 0u};
  if (n < N && k < K) w = *reinterpret_cast<const u4*>(codes + n * (K / 2) + k / 2);
  *reinterpret_cast<u4*>(Wp + tile * TILE_BYTES + 16 * lane) = w;
}

__global__ __launch_bounds__(64) void k_unprepack_mx4(const uint8_t* __restrict__ Wp, int64_t N, int K,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, int64_t strips) {
  const MxGeometry geo = mx_geometry(N, K);
  const int64_t t = block_number();
  if (t >= strips) return;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const int64_t n = 16 * t + r;
  if (n >= N) return;
  for (int kt = 0; kt < geo.KT; ++kt) {
    const int k = 128 * kt + 32 * g;
    if (k >= K) return;
    *reinterpret_cast<u4*>(codes + n * (K / 2) + k / 2) =
        *reinterpret_cast<const u4*>(Wp + (t * geo.KT + kt) * TILE_BYTES + 16 * lane);
    scales[n * (K / 32) + k / 32] =
        Wp[geo.s_off + ((t * geo.KQ + (kt >> 2)) * 64 + lane) * 4 + (kt & 3)];
  }
}

// scales and rows' largest ones: one wave a strip
__global__ __launch_bounds__(64) void k_prepack_mx4_scales(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales,
                                                           int64_t N, int K, uint8_t* __restrict__ Wp,
                                                           int64_t strips) {
  const MxGeometry geo = mx_geometry(N, K);
  const int64_t t = block_number();
  if (t >= strips) return;
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  const int64_t n = 16 * t + r;
  uint32_t most = 0;
  for (int q = 0; q < geo.KQ; ++q) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = 4 * (4 * q + j) + g;
      if (n < N && b < K / 32) {
        const uint32_t s = scales[n * (K / 32) + b];
        word |= s << (8 * j);
        const u4 w = *reinterpret_cast<const u4*>(codes + n * (K / 2) + 16 * (int64_t)b);
        if (s != 255 && ((w[0] | w[1] | w[2] | w[3]) & 0x77777777u)) most = max(most, s);
      }
    }
    *reinterpret_cast<uint32_t*>(Wp + geo.s_off + ((t * geo.KQ + q) * 64 + lane) * 4) = word;
  }
  most = max(most, (uint32_t)__shfl_xor((int)most, 16, 64));
  most = max(most, (uint32_t)__shfl_xor((int)most, 32, 64));
  if (g == 0) Wp[geo.e_off + n] = (uint8_t)most;
}

static bool mx_sizes_ok(int64_t rows, int K) {
  return rows >= 0 && rows <= 0x7fffffff && K >= 32 && K % 32 == 0 && K <= W4_MAX_K;
}

}  // namespace w4

using namespace w4;

extern "C" int quantize_mx4(const void* X, int in_dtype, int rows, int K, uint8_t* codes,
                            uint8_t* scales, hipStream_t stream) {
  if (in_dtype != W4_IN_F16 && in_dtype != W4_IN_F32) return W4_ERR_ARG;
  if (!mx_sizes_ok(rows, K)) return W4_ERR_SHAPE;
  if (rows == 0) return W4_OK;
  if (!X || !codes || !scales) return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(codes, 16)) return W4_ERR_ALIGN;
  const int64_t groups = (int64_t)rows * K / 8, blocks = (groups + 255) / 256;
  if (blocks > MAX_BLOCKS) return W4_ERR_SHAPE;
  if (in_dtype == W4_IN_F16)
    hipLaunchKernelGGL((k_quantize_mx4<uint16_t>), grid_of(blocks), dim3(256), 0, stream,
                       (const uint16_t*)X, groups, codes, scales);
  else
    hipLaunchKernelGGL((k_quantize_mx4<float>), grid_of(blocks), dim3(256), 0, stream,
                       (const float*)X, groups, codes, scales);
  return launch_status();
}

extern "C" int dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int rows, int K,
                              int out_dtype, void* Y, hipStream_t stream) {
  if (out_dtype != W4_OUT_F16 && out_dtype != W4_OUT_F32) return W4_ERR_ARG;
  if (!mx_sizes_ok(rows, K)) return W4_ERR_SHAPE;
  if (rows == 0) return W4_OK;
  if (!Y || !codes || !scales) return W4_ERR_NULL;
  if (!aligned(Y, 16) || !aligned(codes, 16)) return W4_ERR_ALIGN;
  const int64_t groups = (int64_t)rows * K / 8, blocks = (groups + 255) / 256;
  if (blocks > MAX_BLOCKS) return W4_ERR_SHAPE;
  if (out_dtype == W4_OUT_F16)
    hipLaunchKernelGGL((k_dequantize_mx4<uint16_t>), grid_of(blocks), dim3(256), 0, stream, codes,
                       scales, groups, (uint16_t*)Y);
  else
    hipLaunchKernelGGL((k_dequantize_mx4<float>), grid_of(blocks), dim3(256), 0, stream, codes,
                       scales, groups, (float*)Y);
  return launch_status();
}

extern "C" size_t prepack_mx4_bytes(int N, int K) {
  if (N < 1 || N > (1 << 30) || !mx_sizes_ok(N, K)) return 0;
  return (size_t)mx_geometry(N, K).total;
}

extern "C" int prepack_mx4(const uint8_t* codes, const uint8_t* scales, int N, int K, uint8_t* Wp,
                           hipStream_t stream) {
  if (prepack_mx4_bytes(N, K) == 0) return W4_ERR_SHAPE;
  if (!codes || !scales || !Wp) return W4_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(Wp, 16)) return W4_ERR_ALIGN;
  const MxGeometry g = mx_geometry(N, K);
  const int64_t tiles = (int64_t)g.NT * g.KT, blocks = (tiles + 3) / 4;
  if (blocks > MAX_BLOCKS) return W4_ERR_SHAPE;
  hipLaunchKernelGGL(k_prepack_mx4, grid_of(blocks), dim3(256), 0, stream, codes, (int64_t)N, K, Wp,
                     tiles);
  hipLaunchKernelGGL(k_prepack_mx4_scales, grid_of(g.NT), dim3(64), 0, stream, codes, scales,
                     (int64_t)N, K, Wp, (int64_t)g.NT);
  return launch_status();
}

extern "C" int unprepack_mx4(const uint8_t* Wp, int N, int K, uint8_t* codes, uint8_t* scales,
                             hipStream_t stream) {
  if (prepack_mx4_bytes(N, K) == 0) return W4_ERR_SHAPE;
  if (!codes || !scales || !Wp) return W4_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(Wp, 16)) return W4_ERR_ALIGN;
  const MxGeometry g = mx_geometry(N, K);
  hipLaunchKernelGGL(k_unprepack_mx4, grid_of(g.NT), dim3(64), 0, stream, Wp, (int64_t)N, K, codes,
                     scales, (int64_t)g.NT);
  return launch_status();
}
