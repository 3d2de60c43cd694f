// Products of up to 64 rows with MXFP4 weights: the weights are streamed once.
//
// A block owns SP strips of 16 weight rows, its waves share out the k tiles; a
// lane's 16 bytes are the operand as they lie (mx_common.hpp). Rows of A come from
// the caches, 16 a column operand. D = W A^T: a lane ends with four
// neighbouring columns of C for one row. The waves' sums meet in LDS.
#include "mx_gemm.hpp"

namespace w4 {

template <int ACT>
struct RowFrag {
  h8 h[mx_half(ACT) ? 4 : 1];
  v8i q;
  uint32_t s;
};

template <int ACT, int QT, int SP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx_rows(const MxParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
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
    wt[i] = p.Wp + t * geo.KT * TILE_BYTES + 16 * lane;
    ws[i] = p.Wp + geo.s_off + t * geo.KQ * 256 + 4 * lane;
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
    return *reinterpret_cast<const u4*>(k < p.K ? r + act_bytes<ACT>(k) : mx_zeros);
  };
  auto load_a = [&](int u, int kt, RowFrag<ACT>& f) {
    if constexpr (ACT == W4_MX_A16) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f.h[j] = __builtin_bit_cast(h8, chunk(row[u], 128 * kt + 32 * g + 8 * j));
    } else if constexpr (ACT == MX_A8_EXACT) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u4 a = chunk(row[u], 128 * kt + 32 * g + 16 * j);
        f.h[2 * j] = fp8_h8(a[0], a[1]);
        f.h[2 * j + 1] = fp8_h8(a[2], a[3]);
      }
    } else if constexpr (ACT == W4_MX_A8) {            // k 16 g .. and 64 + 16 g ..
      const u4 a = chunk(row[u], 128 * kt + 16 * g), b = chunk(row[u], 128 * kt + 64 + 16 * g);
      f.q = v8i{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
    } else {
      const u4 a = chunk(row[u], 128 * kt + 32 * g);
      f.q = v8i{(int)a[0], (int)a[1], (int)a[2], (int)a[3]};
      f.s = *(128 * kt + 32 * g < p.K ? srow[u] + 4 * kt + g : mx_zeros);
    }
  };
  auto product = [&](const u4 w, uint32_t s, uint32_t top, const RowFrag<ACT>& f, f4 d) {
    if constexpr (mx_half(ACT)) {
      const float up = h_scale(s, top);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(fp4_h8(w[j], up), f.h[j], d, 0, 0, 0);
      return d;
    } else {
      const v8i a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
      if constexpr (ACT == W4_MX_A8)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, f.q, d, 4, 0, 0, s, 0, 127);
      else
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, f.q, d, 4, 4, 0, s, 0, f.s);
    }
  };

  constexpr int U = 4 / SP;
  int kt = geo.KT * wave / WAVES;
  const int end = geo.KT * (wave + 1) / WAVES;
  for (; kt < end; kt += U) {
    u4 w[U][SP];
    uint32_t s[U][SP];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < SP; ++i) {
        const int x = min(kt + j, end - 1);
        w[j][i] = *reinterpret_cast<const u4*>(wt[i] + (int64_t)x * TILE_BYTES);
        s[j][i] = ws[i][(x >> 2) * 256 + (x & 3)];
      }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (kt + j >= end) break;
#pragma unroll
      for (int u = 0; u < QT; ++u) {
        RowFrag<ACT> f;
        load_a(u, kt + j, f);
#pragma unroll
        for (int i = 0; i < SP; ++i) acc[i][u] = product(w[j][i], s[j][i], rowmax[i], f, acc[i][u]);
      }
    }
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
int launch_rows(const MxParams& p, hipStream_t stream) {
  constexpr int WAVES = 8, lds = WAVES * SP * QT * 1024;
  allow_smem((const void*)&k_mx_rows<ACT, QT, SP, WAVES>, lds);
  hipLaunchKernelGGL((k_mx_rows<ACT, QT, SP, WAVES>), grid_of(((int64_t)p.N + 16 * SP - 1) / (16 * SP)),
                     dim3(64 * WAVES), lds, stream, p);
  return launch_status();
}

template <int ACT>
int launch_rows_act(const MxParams& p, hipStream_t stream) {
  if (p.M <= 16) return launch_rows<ACT, 1, 1>(p, stream);
  if (p.M <= 32) return launch_rows<ACT, 2, 1>(p, stream);
  return launch_rows<ACT, 4, 1>(p, stream);
}

int launch_mx_rows(int act, const MxParams& p, hipStream_t stream) {
  return act == W4_MX_A16 ? launch_rows_act<W4_MX_A16>(p, stream)
         : act == W4_MX_A8 ? p.out == W4_OUT_F32 ? launch_rows_act<MX_A8_EXACT>(p, stream)
                                                 : launch_rows_act<W4_MX_A8>(p, stream)
                           : launch_rows_act<W4_MX_A4>(p, stream);
}

}  // namespace w4
