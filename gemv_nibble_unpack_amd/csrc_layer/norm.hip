// Residual addition + root-mean-square norm + per-row 8-bit codes.
//
// One pass: with h = x + residual, g = h * weight, the row needs
// S = sum h^2 and G = max |g|. The normalised row is y = g * r, r =
// 1/sqrt(S/K + eps), its scale max|y|/L = G * r / L (L = 127 or 448), and the
// codes y / scale = g * (L / G): the root cancels, so both reductions are
// taken together and the row is coded from the registers it was loaded into.
// Bound: bytes (fp16 with residual: 4 read, 3 written per element). 2048 rows of
// 4096 in fp16 with residual take 11.0 us, 5.3 TB/s (a large copy reaches 4.8);
// 333 float32 rows of 8640 take 5.0 us, 2.9 TB/s, one row of 4096 2.1 us, both
// of them launch and latency. A row's chunks are all loaded before any is used:
// one round trip to memory, one barrier.

#include "layer_common.hpp"

namespace w4 {

// One row per group of WAVES waves; CPT > 0: CPT chunks of 8 elements per lane
// held in registers (K <= 512 * WAVES * CPT), loads of every chunk issued
// before any is used. CPT == 0: rows too long for that are read twice (the
// second time from L2), the residual sum being written then.
// A block of 256 threads holds 4 / WAVES rows; longer rows take one block.
template <typename T, int Q, int WAVES, int CPT>
__global__ __launch_bounds__(WAVES < 4 ? 256 : 64 * WAVES) void k_add_rmsnorm(
    const T* X, const T* R, const T* __restrict__ Wt, int M, int K, float eps, T* H,
    uint8_t* __restrict__ Yq, float* __restrict__ scale) {
  constexpr int ROWS = WAVES < 4 ? 4 / WAVES : 1;
  constexpr int LANES = 64 * WAVES;
  __shared__ float shs[WAVES < 4 ? 4 : WAVES];
  __shared__ uint32_t shm[WAVES < 4 ? 4 : WAVES];
  const int tid = threadIdx.x % LANES;
  const int sub = threadIdx.x / LANES;
  // rows past the end repeat the last row up to its barriers and store nothing
  const int mrow = blockIdx.x * ROWS + sub;
  const bool live = mrow < M;
  const int m = live ? mrow : M - 1;
  const size_t base = (size_t)m * K;
  const T* x = X + base;
  const T* r = R ? R + base : nullptr;
  const int nch = K / 8;

  float ss = 0.f;
  uint32_t mx = 0;
  float h[CPT > 0 ? CPT : 1][8], g[CPT > 0 ? CPT : 1][8];
  if constexpr (CPT > 0) {
    // chunks past the row re-read its last chunk and count as zero, so that
    // no load waits inside a branch
#pragma unroll
    for (int i = 0; i < CPT; ++i) load8f(x + 8 * min(tid + i * LANES, nch - 1), h[i]);
    float b[CPT][8];
    if (R) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) load8f(r + 8 * min(tid + i * LANES, nch - 1), b[i]);
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) load8f(Wt + 8 * min(tid + i * LANES, nch - 1), g[i]);
    if (R) {
#pragma unroll
      for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += b[i][e];
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const bool in = tid + i * LANES < nch;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[i][e] = in ? g[i][e] * h[i][e] : 0.f;
        ss += in ? h[i][e] * h[i][e] : 0.f;
        mx = max(mx, abs_bits(g[i][e]));
      }
    }
  } else {
    for (int c = tid; c < nch; c += LANES) {
      float a[8], w[8];
      load8f(x + 8 * c, a);
      load8f(Wt + 8 * c, w);
      if (R) {
        float b[8];
        load8f(r + 8 * c, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += b[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss += a[e] * a[e];
        mx = max(mx, abs_bits(a[e] * w[e]));
      }
    }
  }
  mx = wave_max_u(mx);
  // the row's sum over its waves; `first` also takes the maximum across
  auto across = [&](bool first) {
    ss = wave_sum_f(ss);
    if constexpr (WAVES > 1) {
      const int wv = threadIdx.x >> 6;
      if (!first) __syncthreads();               // shs is read out
      if ((threadIdx.x & 63) == 0) {
        shs[wv] = ss;
        if (first) shm[wv] = mx;
      }
      __syncthreads();
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) ss += shs[sub * WAVES + i];
      if (first) {
        mx = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) mx = max(mx, shm[sub * WAVES + i]);
      }
    }
  };
  across(true);
  constexpr float L = Q == W4_Q_I8 ? 127.f : 448.f;
  const float gm = __uint_as_float(mx);
  const bool bad = mx >= F32_INF;
  // a row whose largest product is below 2^-64 is coded after a multiplication
  // by 2^64, so that L / G stays finite
  const float up = gm < 0x1p-64f ? 0x1p64f : 1.0f;
  const float inv = bad || mx == 0 ? 0.f : L / (gm * up);
  // the row's scale: the codes do not need the root
  auto settle = [&] {
    float mean = ss / (float)K + eps;
    // Float32 rows whose squares leave float32 (fp16 ones cannot): the squares are
    // summed again with h taken times 2^100 or 2^-80, as the mean is small or
    // infinite. The same for all threads of a row, and a row with barriers has
    // its block to itself.
    float f = 1.f;
    if constexpr (sizeof(T) == 4) {
      static_assert(WAVES == 1 || WAVES >= 4, "a row with barriers has its block to itself");
      if (__builtin_expect(!(mean >= 0x1p-100f && mean < __builtin_inff()) && !bad && mx != 0, 0)) {
        f = mean < 1.f ? 0x1p100f : 0x1p-80f;
        ss = 0.f;
        if constexpr (CPT > 0) {
#pragma unroll
          for (int i = 0; i < CPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float a = tid + i * LANES < nch ? h[i][e] * f : 0.f;
              ss += a * a;
            }
        } else {
          for (int c = tid; c < nch; c += LANES) {
            float a[8], b[8];
            load8f(x + 8 * c, a);
            if (r) load8f(r + 8 * c, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              a[e] = (r ? a[e] + b[e] : a[e]) * f;
              ss += a[e] * a[e];
            }
          }
        }
        across(false);
        mean = ss / (float)K + eps * f * f;
      }
    }
    const float root = 1.0f / sqrtf(mean);         // of the mean in units of f^-2
    // gm * (root * f) / L, the factor taken where it brings the product towards 1
    // (products that are all zero have scale 0 also where eps = 0 makes the root infinite)
    if (live && tid == 0) {
      const bool early = (gm < 1.f) == (f > 1.f);
      scale[m] = bad ? __uint_as_float(0x7FC00000u)
                     : mx == 0 ? 0.f : gm * (early ? f : 1.f) * root / L * (early ? 1.f : f);
    }
  };
  // Rows that are read again settle before H replaces them. Of the others, those of
  // several waves code first (one float32 row of 4096, replayed, 2.75 us, 2.83 the
  // other way round), those of one wave settle first (4096 rows of 512 3.87 us, 4.01).
  constexpr bool late = CPT > 0 && WAVES > 1;
  if constexpr (!late) settle();
  uint8_t* out = Yq + base;
  auto emit = [&](int c, const float (&v)[8]) {
    u2 w = {0u, 0u};
    if (!bad) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = v[e] * up * inv;
      w = u2{code4<Q>(y[0], y[1], y[2], y[3]), code4<Q>(y[4], y[5], y[6], y[7])};
    }
    *reinterpret_cast<u2*>(out + 8 * c) = w;
  };
  if constexpr (CPT > 0) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = tid + i * LANES;
      if (live && c < nch) {
        if (H) store8f(H + base + 8 * c, h[i]);
        emit(c, g[i]);
      }
    }
    if constexpr (late) settle();
  } else {
    for (int c = tid; c < nch; c += LANES) {
      float a[8], w[8];
      load8f(x + 8 * c, a);
      load8f(Wt + 8 * c, w);
      if (R) {
        float b[8];
        load8f(r + 8 * c, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += b[e];
      }
      if (!live) continue;
      if (H) store8f(H + base + 8 * c, a);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] *= w[e];
      emit(c, a);
    }
  }
}

template <typename T, int Q>
int launch_norm(const void* X, const void* R, const void* Wt, int M, int K, float eps, void* H,
                void* Yq, float* scale, hipStream_t stream) {
#define W4_NORM(WV, C)                                                                           \
  hipLaunchKernelGGL((k_add_rmsnorm<T, Q, WV, C>), dim3(ceil_div(M, WV < 4 ? 4 / WV : 1)),       \
                     dim3(WV < 4 ? 256 : 64 * WV), 0, stream, (const T*)X, (const T*)R,          \
                     (const T*)Wt, M, K, eps, (T*)H, (uint8_t*)Yq, scale)
  // waves by the row: 4096 rows of 512 4.8 us on one wave each, 6.6 on four; 2048
  // rows of 4096 11.3 us on four, 11.7 on eight (one row 4.7 and 4.5)
  if (K <= 1024) W4_NORM(1, 2);
  else if (K <= 4096) W4_NORM(4, 2);
  else if (K <= 8192) W4_NORM(8, 2);
  // (one shape measured, in the first form of these kernels: 333 float32 rows of 8640 4.9
  // us, 16 waves x 2 6.0, 4 x 5 5.3)
  else if (K <= 12288) W4_NORM(8, 3);
  else if (K <= 16384) W4_NORM(16, 2);
  else W4_NORM(16, 0);
#undef W4_NORM
  return launch_status();
}

}  // namespace w4

using namespace w4;

extern "C" int add_rmsnorm_q8(const void* X, const void* residual, const void* weight, int in_dtype,
                              int M, int K, float eps, int q_dtype, void* residual_out, void* Yq,
                              float* y_scale, hipStream_t stream) {
  if (in_dtype != W4_IN_F16 && in_dtype != W4_IN_F32) return W4_ERR_ARG;
  if (q_dtype != W4_Q_I8 && q_dtype != W4_Q_F8) return W4_ERR_ARG;
  if (!(eps >= 0.f) || eps > 3.0e38f) return W4_ERR_ARG;
  if (M < 0 || K < 8 || K % 8 || K > W4_MAX_K) return W4_ERR_SHAPE;
  if (M == 0) return W4_OK;
  if (!X || !weight || !Yq || !y_scale) return W4_ERR_NULL;
  if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
      !aligned(residual_out, 16) || !aligned(Yq, 16) || !aligned(y_scale, 4))
    return W4_ERR_ALIGN;
  auto go = [&](auto launch) {
    return launch(X, residual, weight, M, K, eps, residual_out, Yq, y_scale, stream);
  };
  if (in_dtype == W4_IN_F16)
    return q_dtype == W4_Q_I8 ? go(launch_norm<uint16_t, W4_Q_I8>)
                              : go(launch_norm<uint16_t, W4_Q_F8>);
  return q_dtype == W4_Q_I8 ? go(launch_norm<float, W4_Q_I8>) : go(launch_norm<float, W4_Q_F8>);
}
