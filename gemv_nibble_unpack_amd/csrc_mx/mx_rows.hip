// Products of up to 64 rows with MXFP4 weights: the weights are streamed once.
//
// A block owns SP strips of 16 weight rows, its waves share out the k tiles; a
// lane's 16 bytes are the operand as they lie (mx_common.hpp). Rows of A come from
// the caches, 16 a column operand. D = W A^T: a lane ends with four
// neighbouring columns of C for one row. The waves' sums meet in LDS.
//
// Bound: round trips to memory, a few one after another in each wave (waits are 47 to 72%
// of the waves' lives, the matrix cores 2 to 9% busy), and with many rows what each block reads
// of them. us: 1 x 4096 x 4096 fp16 4.6 (9 MB; 1.8 at the copy rate), 27 x 11008 x 4096 fp16 13.7
// (24 MB, 5.1; a block reads 221 KB of rows beside 104 of weights), 45 x 3200 x 8640 8-bit rows
// 13.0 (15 MB, 3.1; 389 KB beside 73, 200 blocks on 256 CUs), 8 x 4096 x 11008 4-bit rows
// 7.5 (24 MB, 5.0).
#include "mx_gemm.hpp"

namespace w4 {

// operands of one k tile: SP strips of weights, QT column operands of rows
template <int ACT, int QT, int SP>
struct RowTile {
  u4 w[SP];
  uint32_t s[SP];                          // the weights' scale
  u4 a[QT][ACT == W4_MX_A16 ? 4 : mx_row8(ACT) ? 2 : 1];
  uint32_t as[QT];                         // A4: the rows' scales
};

constexpr int ROW_WAVES = 8;

template <int ACT, int QT, int SP>
__global__ __launch_bounds__(64 * ROW_WAVES) void k_mx_rows(const MxParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using T = RowTile<ACT, QT, SP>;
  constexpr int WAVES = ROW_WAVES;
  const MxGeometry geo = mx_geometry(p.N, p.K);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int t0 = block_number() * SP;
  if (t0 >= geo.NT) return;

  const uint8_t *wt[SP], *ws[SP];
  uint32_t rowmax[SP];
#pragma unroll
  for (int i = 0; i < SP; ++i) {
    const int64_t t = min(t0 + i, geo.NT - 1);
    wt[i] = p.Wp + t * geo.KT * TILE_BYTES;
    ws[i] = p.Wp + geo.s_off + t * geo.KQ * 256;
    rowmax[i] = mx_half(ACT) ? p.Wp[geo.e_off + 16 * t + c] : 0;
  }
  const uint8_t* row[QT];
  const uint8_t* srow[QT];
#pragma unroll
  for (int u = 0; u < QT; ++u) {
    const int64_t m = min(16 * u + c, p.M - 1);
    row[u] = p.A + m * act_bytes<ACT>(p.K);
    srow[u] = ACT == W4_MX_A4 ? p.a_scales + m * (p.K / 32) : nullptr;
  }

  f4 acc[SP][QT];
#pragma unroll
  for (int i = 0; i < SP; ++i)
#pragma unroll
    for (int u = 0; u < QT; ++u) acc[i][u] = f4{0.f, 0.f, 0.f, 0.f};

  auto chunk = [&](const uint8_t* r, int k) {          // 16 bytes of a row at element k
    return g_load<u4>(k < p.K ? r + act_bytes<ACT>(k) : mx_zeros);
  };
  auto load = [&](int kt, T& f) {
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      f.w[i] = g_load<u4>(wt[i] + (int64_t)kt * TILE_BYTES, 16 * lane);
      f.s[i] = g_load<uint8_t>(ws[i] + (kt >> 2) * 256 + (kt & 3), 4 * lane);
    }
    const int k = 128 * kt;
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      if constexpr (ACT == W4_MX_A16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f.a[u][j] = chunk(row[u], k + 32 * g + 8 * j);
      } else if constexpr (ACT == MX_A8_EXACT) {
        f.a[u][0] = chunk(row[u], k + 32 * g), f.a[u][1] = chunk(row[u], k + 32 * g + 16);
      } else if constexpr (ACT == W4_MX_A8) {            // k 16 g .. and 64 + 16 g ..
        f.a[u][0] = chunk(row[u], k + 16 * g), f.a[u][1] = chunk(row[u], k + 64 + 16 * g);
      } else {
        f.a[u][0] = chunk(row[u], k + 32 * g);
        f.as[u] = g_load<uint8_t>(k + 32 * g < p.K ? srow[u] + 4 * kt + g : mx_zeros);
      }
    }
  };
  auto multiply = [&](const T& f) {
    if constexpr (mx_half(ACT)) {
      h8 a[QT][4];
#pragma unroll
      for (int u = 0; u < QT; ++u) {
        if constexpr (ACT == W4_MX_A16) {
#pragma unroll
          for (int x = 0; x < 4; ++x) a[u][x] = __builtin_bit_cast(h8, f.a[u][x]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) a[u][x] = fp8_h8(f.a[u][x / 2][2 * (x & 1)], f.a[u][x / 2][2 * (x & 1) + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        const float up = h_scale(f.s[i], rowmax[i]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const h8 b = fp4_h8(f.w[i][x], up);
#pragma unroll
          for (int u = 0; u < QT; ++u)
            acc[i][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a[u][x], acc[i][u], 0, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        const v8i b = {(int)f.w[i][0], (int)f.w[i][1], (int)f.w[i][2], (int)f.w[i][3]};
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          const u4 x = f.a[u][0];
          if constexpr (ACT == W4_MX_A8) {
            const u4 y = f.a[u][1];
            const v8i a = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
            acc[i][u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc[i][u], 4, 0, 0, f.s[i], 0, 127);
          } else {
            const v8i a = {(int)x[0], (int)x[1], (int)x[2], (int)x[3]};
            acc[i][u] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc[i][u], 4, 4, 0, f.s[i], 0, f.as[u]);
          }
        }
      }
    }
  };

  // U tiles' loads together (a second set in flight meanwhile takes registers, so
  // resident waves: one fp16 row, N = 11008, K = 4096 8.0 -> 11.9 us)
  constexpr int U = SP >= 3 ? 1 : SP == 2 ? 2 : 4;
  const int end = geo.KT * (wave + 1) / WAVES;
  for (int kt = geo.KT * wave / WAVES; kt < end; kt += U) {
    T f[U];
#pragma unroll
    for (int j = 0; j < U; ++j) load(min(kt + j, end - 1), f[j]);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (kt + j < end) multiply(f[j]);
  }

  // ---- the waves' sums ------------------------------------------------------
  f4* sums = reinterpret_cast<f4*>(smem);                // [WAVES][SP * QT][64]
#pragma unroll
  for (int i = 0; i < SP; ++i)
#pragma unroll
    for (int u = 0; u < QT; ++u) sums[(wave * SP * QT + i * QT + u) * 64 + lane] = acc[i][u];
  __syncthreads();
  for (int x = threadIdx.x; x < SP * QT * 64; x += 64 * WAVES) {
    f4 v = sums[x];
    for (int z = 1; z < WAVES; ++z) {
      const f4 y = sums[z * SP * QT * 64 + x];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += y[e];
    }
    const int l = x & 63, u = (x >> 6) % QT, i = (x >> 6) / QT;
    const int m = 16 * u + (l & 15), n = 16 * (t0 + i) + 4 * (l >> 4);
    if (m >= p.M || t0 + i >= geo.NT) continue;
    const float as = mx_row8(ACT) ? p.a_scale[m] : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (mx_half(ACT)) v[e] = ldexpf(v[e], (int)p.Wp[geo.e_off + n + e] - 127 - H_UP);
      if constexpr (mx_row8(ACT)) v[e] *= as;
      if (n + e < p.N) {
        const int64_t at = (int64_t)m * p.N + n + e;
        if (p.out == W4_OUT_F16)
          reinterpret_cast<uint16_t*>(p.C)[at] = f2h(v[e] + (p.bias ? h2f(p.bias[n + e]) : 0.f));
        else
          reinterpret_cast<float*>(p.C)[at] = v[e];
      }
    }
  }
}

template <int ACT, int QT, int SP>
int launch_rows_sp(const MxParams& p, hipStream_t stream) {
  constexpr int lds = ROW_WAVES * SP * QT * 1024;
  allow_smem((const void*)&k_mx_rows<ACT, QT, SP>, lds);
  hipLaunchKernelGGL((k_mx_rows<ACT, QT, SP>), grid_of(((int64_t)p.N + 16 * SP - 1) / (16 * SP)),
                     dim3(64 * ROW_WAVES), lds, stream, p);
  return launch_status();
}

// Strips a block: rounds of blocks over the 256 CUs times what a block reads for a k
// tile, SP KiB of weights and the rows. N = 11008, K = 4096, us for 1, 2, 3, 4 strips:
// 27 fp16 rows 26.3, 20.9, 14.6, 17.3, 64 8-bit rows 28.3, 20.8, 13.9, 15.3, one 4-bit row 6.5, 8.1,
// 6.8, 7.5; N = 4096: 16 8-bit rows 5.6, 7.4, 7.8, 9.1. Where one round of three strips and two
// of two are near each other it can be off: one fp16 row, N = 11008, 10.2, 8.8, 9.6, 11.8.
template <int ACT, int QT>
int launch_rows(const MxParams& p, hipStream_t stream) {
  const int strips = ceil_div(p.N, 16);
  const double rows = p.M * act_bytes<ACT>(128) / 1024.0;
  int best = 1;
  double least = 1e30;
  for (int sp = 1; sp <= 4; ++sp) {
    const double cost = ceil_div(ceil_div(strips, sp), 256) * (sp + rows);
    if (cost < least) least = cost, best = sp;
  }
  switch (best) {
    case 1: return launch_rows_sp<ACT, QT, 1>(p, stream);
    case 2: return launch_rows_sp<ACT, QT, 2>(p, stream);
    case 3: return launch_rows_sp<ACT, QT, 3>(p, stream);
    default: return launch_rows_sp<ACT, QT, 4>(p, stream);
  }
}

template <int ACT>
int launch_rows_act(const MxParams& p, hipStream_t stream) {
  if (p.M <= 16) return launch_rows<ACT, 1>(p, stream);
  if (p.M <= 32) return launch_rows<ACT, 2>(p, stream);
  if (p.M <= 48) return launch_rows<ACT, 3>(p, stream);
  return launch_rows<ACT, 4>(p, stream);
}

int launch_mx_rows(int act, const MxParams& p, hipStream_t stream) {
  return act == W4_MX_A16 ? launch_rows_act<W4_MX_A16>(p, stream)
         : act == W4_MX_A8 ? p.out == W4_OUT_F32 ? launch_rows_act<MX_A8_EXACT>(p, stream)
                                                 : launch_rows_act<W4_MX_A8>(p, stream)
                           : launch_rows_act<W4_MX_A4>(p, stream);
}

}  // namespace w4
