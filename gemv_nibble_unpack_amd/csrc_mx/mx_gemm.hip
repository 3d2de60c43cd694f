// Tiled product of many rows with MXFP4 weights.
//
// Four waves (2 along m, 2 along n) own a tile of 64 TM x 64 TN outputs, each 32 TM x
// 32 TN of them on 32 x 32 matrix instructions: v_mfma_scale_f32_32x32x64_f8f6f4
// for 4-bit and 8-bit rows (the one shape that multiplies 4-bit codes at twice
// the rate of 8-bit ones), v_mfma_f32_32x32x16_f16 for fp16 rows, whose weights
// widen in registers. Weights are the row operand, so a lane ends with runs of
// four columns of C. Rows and weights come to LDS by direct loads, a ring of
// NS stages.
#include "mx_gemm.hpp"

namespace w4 {

template <int ACT, int TM, int TN, int NS_>
struct MxTile {
  static constexpr int NS = NS_;
  static constexpr int BM = 64 * TM, BN = 64 * TN, STRIPS = BN / 16;
  static constexpr int TK = ACT == W4_MX_A16 ? 64 : 128;          // k of a stage
  static constexpr int STEPS = TK / 64;
  static constexpr int RB = act_bytes<ACT>(TK);                   // bytes of a staged row
  static constexpr int CH = RB / 16;                              // and its 16-byte chunks
  static constexpr int WB = 8 * TK;                               // bytes of a staged strip
  static constexpr int A_BYTES = BM * RB, W_BYTES = STRIPS * WB;
  static constexpr int STAGE = A_BYTES + W_BYTES;
  static constexpr int A_LOADS = A_BYTES / 4096, W_LOADS = W_BYTES / 4096;   // a wave's, of 1 KiB
  static constexpr int LOADS = A_LOADS + W_LOADS;
  static constexpr int LDS = NS * STAGE;
  static_assert(A_BYTES % 4096 == 0 && W_BYTES % 4096 == 0, "whole loads for each wave");
  static_assert(LDS <= 160 * 1024, "LDS exceeds the CU");
};

// where chunk c of a staged row lies: rows of a fragment spread over the banks
template <int CH>
__device__ __forceinline__ int mx_chunk(int row, int c) {
  return CH == 4 ? c ^ ((row >> 2) & 3) : c ^ ((row >> 1) & 7);
}

// (a device function, so that the kernel's host stub holds no device assembly)
template <int ACT, int TM, int TN, int NS_>
__device__ __forceinline__ void mx_gemm_tile(const MxParams& p, int mblocks, int nblocks, int per_xcd) {
  using S = MxTile<ACT, TM, TN, NS_>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int id = blockIdx.x, local = id >> 3;
  const int tix = (id & 7) * per_xcd + local;            // an XCD's tiles share their columns
  if (local >= per_xcd || tix >= mblocks * nblocks) return;
  const int nb = tix / mblocks, mb = tix - nb * mblocks;

  const MxGeometry geo = mx_geometry(p.N, p.K);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int l31 = lane & 31, half = lane >> 5;
  const int m0 = mb * S::BM, t0 = nb * S::STRIPS;
  const int nst = (p.K + S::TK - 1) / S::TK;

  auto issue = [&](int st, int slot) {
    uint8_t* sa = smem + slot * S::STAGE;
#pragma unroll
    for (int q = 0; q < S::A_LOADS; ++q) {
      constexpr int RPL = 64 / S::CH;                    // rows of a load
      const int row = (wave * S::A_LOADS + q) * RPL + lane / S::CH;
      const int c = mx_chunk<S::CH>(row, lane % S::CH);
      const int k = st * S::TK + c * (S::TK / S::CH);
      const uint8_t* src = p.A + (int64_t)min(m0 + row, p.M - 1) * act_bytes<ACT>(p.K) + act_bytes<ACT>(k);
      __builtin_amdgcn_global_load_lds(k < p.K ? src : mx_zeros, sa + (wave * S::A_LOADS + q) * 1024,
                                       16, 0, 0);
    }
    uint8_t* sw = sa + S::A_BYTES;
#pragma unroll
    for (int q = 0; q < S::W_LOADS; ++q) {
      constexpr int LPS = S::WB / 16;                    // lanes of a strip: 64 or 32
      const int strip = (wave * S::W_LOADS + q) * (64 / LPS) + lane / LPS;
      const int t = min(t0 + strip, geo.NT - 1);
      const uint8_t* src = p.Wp + (int64_t)t * geo.KT * TILE_BYTES + (int64_t)st * S::WB + (lane % LPS) * 16;
      __builtin_amdgcn_global_load_lds(src, sw + (wave * S::W_LOADS + q) * 1024, 16, 0, 0);
    }
  };

  // ---- scales: four k tiles' worth at a time, one quad ahead ------------------
  const int r = lane & 15, hi = (lane >> 4) & 1;         // this lane's weight row: strip 2 j + hi, row r
  const uint8_t* wscale[TN];
  uint32_t top[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t t = min(t0 + 2 * (wn * TN + j) + hi, geo.NT - 1);
    wscale[j] = p.Wp + geo.s_off + t * geo.KQ * 256 + (half * 16 + r) * 4;
    top[j] = mx_half(ACT) ? p.Wp[geo.e_off + 16 * t + r] : 0;
  }
  const uint8_t* ascale[TM];
  const int KB = p.K / 32;
#pragma unroll
  for (int i = 0; i < TM; ++i)
    ascale[i] = ACT == W4_MX_A4
                    ? p.a_scales + (int64_t)min(m0 + 32 * (wm * TM + i) + l31, p.M - 1) * KB
                    : nullptr;
  constexpr bool AS = ACT == W4_MX_A4;
  uint32_t sw[TN][2], sw_next[TN][2];                    // [column tile][step]: a byte a k tile
  u4 sa[AS ? TM : 1], sa_next[AS ? TM : 1];              // [row tile]: a word a k tile, a byte a block
  auto load_scales = [&](int q) {
    q = min(q, geo.KQ - 1);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        sw_next[j][s] = *reinterpret_cast<const uint32_t*>(wscale[j] + (int64_t)q * 256 + s * 128);
    if constexpr (AS) {
      if (16 * q + 16 <= KB) {
#pragma unroll
        for (int i = 0; i < TM; ++i) sa_next[i] = *reinterpret_cast<const u4_any*>(ascale[i] + 16 * q);
      } else {                                           // the row ends inside
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t w = 0;
            for (int y = 0; y < 4; ++y) {
              const int b = 16 * q + 4 * x + y;
              w |= (uint32_t)*(b < KB ? ascale[i] + b : mx_zeros) << (8 * y);
            }
            sa_next[i][x] = w;
          }
      }
    }
  };

  f16v acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  auto compute = [&](int st, int slot) {
    const uint8_t* a = smem + slot * S::STAGE;
    const uint8_t* w = a + S::A_BYTES + (2 * wn * TN + hi) * S::WB + (half * 16 + r) * 16;
#pragma unroll
    for (int s = 0; s < S::STEPS; ++s) {
      u4 wf[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) wf[j] = *reinterpret_cast<const u4*>(w + 2 * j * S::WB + s * 512);
      if constexpr (mx_half(ACT)) {
        h8 af[TM][4];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int row = 32 * (wm * TM + i) + l31;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if constexpr (ACT == W4_MX_A16) {
              af[i][x] = *reinterpret_cast<const h8*>(a + row * S::RB + 16 * mx_chunk<8>(row, 4 * half + x));
            } else if (x % 2 == 0) {
              const u4 y = *reinterpret_cast<const u4*>(
                  a + row * S::RB + 16 * mx_chunk<8>(row, 4 * s + 2 * half + x / 2));
              af[i][x] = fp8_h8(y[0], y[1]);
              af[i][x + 1] = fp8_h8(y[2], y[3]);
            }
          }
        }
        const int kt = ACT == W4_MX_A16 ? st >> 1 : st, step = ACT == W4_MX_A16 ? st & 1 : s;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const uint32_t byte = ((step ? sw[j][1] : sw[j][0]) >> (8 * (kt & 3))) & 255u;
          const float up = h_scale(byte, top[j]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const h8 b = fp4_h8(wf[j][x], up);
#pragma unroll
            for (int i = 0; i < TM; ++i)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, af[i][x], acc[i][j], 0, 0, 0);
          }
        }
      } else {
        v8i af[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int row = 32 * (wm * TM + i) + l31;
          if constexpr (ACT == W4_MX_A8) {
            const u4 x = *reinterpret_cast<const u4*>(a + row * S::RB + 16 * mx_chunk<8>(row, 4 * s + half));
            const u4 y = *reinterpret_cast<const u4*>(a + row * S::RB + 16 * mx_chunk<8>(row, 4 * s + 2 + half));
            af[i] = v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
          } else {
            const u4 x = *reinterpret_cast<const u4*>(a + row * S::RB + 16 * mx_chunk<4>(row, 2 * s + half));
            af[i] = v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3]};
          }
        }
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const v8i b = {(int)wf[j][0], (int)wf[j][1], (int)wf[j][2], (int)wf[j][3]};
          const uint32_t sb = sw[j][s] >> (8 * (st & 3));
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            if constexpr (ACT == W4_MX_A8) {
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, af[i], acc[i][j], 4, 0, 0, sb, 0, 127);
            } else {
              const uint32_t sx = sa[i][0] >> (8 * (2 * s + half));
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, af[i], acc[i][j], 4, 4, 0, sb, 0, sx);
            }
          }
        }
      }
    }
    if constexpr (AS) {                                  // the next k tile's words to the front
#pragma unroll
      for (int i = 0; i < TM; ++i) sa[i] = u4{sa[i][1], sa[i][2], sa[i][3], 0u};
    }
  };

  constexpr int QS = 512 / S::TK;                        // stages of a quad
#pragma unroll
  for (int q = 0; q < S::NS - 1; ++q) issue(min(q, nst - 1), q);
  load_scales(0);
  int slot = 0;
  for (int st = 0; st < nst; ++st) {
    // every stage issues the same loads (the last ones again past the end), so
    // that a fixed count waits for this stage's alone
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S::NS - 2) * S::LOADS) : "memory");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    issue(min(st + S::NS - 1, nst - 1), slot == 0 ? S::NS - 1 : slot - 1);
    if (st % QS == 0) {
#pragma unroll
      for (int j = 0; j < TN; ++j) sw[j][0] = sw_next[j][0], sw[j][1] = sw_next[j][1];
#pragma unroll
      for (int i = 0; i < (AS ? TM : 1); ++i) sa[i] = sa_next[i];
      load_scales(st / QS + 1);
    }
    compute(st, slot);
    slot = slot + 1 == S::NS ? 0 : slot + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // ---- epilogue: lane holds row 32 .. + l31, columns 8 (e >> 2) + 4 half + (e & 3) --
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = m0 + 32 * (wm * TM + i) + l31;
    const float as = mx_row8(ACT) ? p.a_scale[min(m, p.M - 1)] : 1.f;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int n = 16 * t0 + 32 * (wn * TN + j) + 8 * (e >> 2) + 4 * half + (e & 3);
        if (m < p.M && n < p.N) {
          float v = acc[i][j][e];
          if constexpr (mx_half(ACT)) v = ldexpf(v, (int)p.Wp[geo.e_off + n] - 127 - H_UP);
          if constexpr (mx_row8(ACT)) v *= as;
          const int64_t at = (int64_t)m * p.N + n;
          if (p.out == W4_OUT_F16)
            reinterpret_cast<uint16_t*>(p.C)[at] = f2h(v + (p.bias ? h2f(p.bias[n]) : 0.f));
          else
            reinterpret_cast<float*>(p.C)[at] = v;
        }
      }
  }
}

template <int ACT, int TM, int TN, int NS>
__global__ __launch_bounds__(256, 1) void k_mx_gemm(const MxParams p, int mblocks, int nblocks,
                                                    int per_xcd) {
  mx_gemm_tile<ACT, TM, TN, NS>(p, mblocks, nblocks, per_xcd);
}

template <int ACT, int TM, int TN, int NS>
int launch_tile(const MxParams& p, hipStream_t stream) {
  using S = MxTile<ACT, TM, TN, NS>;
  const int mblocks = ceil_div(p.M, S::BM), nblocks = ceil_div(p.N, S::BN);
  const int64_t tiles = (int64_t)mblocks * nblocks;
  if (tiles > (1 << 23)) return W4_ERR_SHAPE;
  const int per_xcd = (int)((tiles + 7) / 8);
  allow_smem((const void*)&k_mx_gemm<ACT, TM, TN, NS>, S::LDS);
  hipLaunchKernelGGL((k_mx_gemm<ACT, TM, TN, NS>), dim3(per_xcd * 8), dim3(256), S::LDS, stream, p,
                     mblocks, nblocks, per_xcd);
  return launch_status();
}

int launch_mx_gemm(int act, const MxParams& p, hipStream_t stream) {
  const bool big = (int64_t)p.M * p.N >= 128LL * 256 * 256;
  if (act == W4_MX_A16)
    return big ? launch_tile<W4_MX_A16, 4, 4, 3>(p, stream) : launch_tile<W4_MX_A16, 2, 2, 4>(p, stream);
  if (act == W4_MX_A8 && p.out == W4_OUT_F32)
    return big ? launch_tile<MX_A8_EXACT, 4, 4, 3>(p, stream) : launch_tile<MX_A8_EXACT, 2, 2, 4>(p, stream);
  if (act == W4_MX_A8)
    return big ? launch_tile<W4_MX_A8, 4, 4, 3>(p, stream) : launch_tile<W4_MX_A8, 2, 2, 4>(p, stream);
  return big ? launch_tile<W4_MX_A4, 4, 4, 4>(p, stream) : launch_tile<W4_MX_A4, 2, 2, 4>(p, stream);
}

}  // namespace w4

using namespace w4;

static constexpr int ROWS_MOST = 64;

static bool mx_gemm_sizes_ok(int M, int N, int K) {
  return M >= 0 && M <= (1 << 30) && prepack_mx4_bytes(N, K) != 0;
}

extern "C" size_t mx4_workspace_bytes(int op, int M, int N, int K) {
  if (op < W4_MX_A16 || op > W4_MX_A4 || !mx_gemm_sizes_ok(M, N, K) || M == 0) return 0;
  return 0;
}

static int mx_gemm(int act, MxParams p, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (p.out != W4_OUT_F16 && p.out != W4_OUT_F32) return W4_ERR_ARG;
  if (!mx_gemm_sizes_ok(p.M, p.N, p.K)) return W4_ERR_SHAPE;
  if (p.M == 0) return W4_OK;
  if (!p.A || !p.Wp || !p.C || (act == W4_MX_A8 && !p.a_scale) || (act == W4_MX_A4 && !p.a_scales))
    return W4_ERR_NULL;
  if (!aligned(p.A, 16) || !aligned(p.Wp, 16) || !aligned(p.C, 16) || !aligned(p.bias, 2) ||
      !aligned(p.a_scale, 4) || !aligned(workspace, 256))
    return W4_ERR_ALIGN;
  const size_t need = mx4_workspace_bytes(act, p.M, p.N, p.K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return W4_ERR_WORKSPACE;
  p.counters = (uint32_t*)workspace;
  p.part = workspace ? (float*)((uint8_t*)workspace + WS_COUNTERS) : nullptr;
  return p.M <= ROWS_MOST ? launch_mx_rows(act, p, stream) : launch_mx_gemm(act, p, stream);
}

extern "C" int mx4a16_gemm(const uint16_t* A, const uint8_t* Wp, const uint16_t* bias, void* C,
                           int out_dtype, int M, int N, int K, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  MxParams p{};
  p.A = (const uint8_t*)A, p.Wp = Wp, p.bias = bias, p.C = C;
  p.M = M, p.N = N, p.K = K, p.out = out_dtype;
  return mx_gemm(W4_MX_A16, p, workspace, workspace_bytes, stream);
}

extern "C" int mx4a8_gemm(const uint8_t* Aq, const float* a_scale, const uint8_t* Wp,
                          const uint16_t* bias, void* C, int out_dtype, int M, int N, int K,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  MxParams p{};
  p.A = Aq, p.a_scale = a_scale, p.Wp = Wp, p.bias = bias, p.C = C;
  p.M = M, p.N = N, p.K = K, p.out = out_dtype;
  return mx_gemm(W4_MX_A8, p, workspace, workspace_bytes, stream);
}

extern "C" int mx4a4_gemm(const uint8_t* Aq, const uint8_t* a_scales, const uint8_t* Wp,
                          const uint16_t* bias, void* C, int out_dtype, int M, int N, int K,
                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  MxParams p{};
  p.A = Aq, p.a_scales = a_scales, p.Wp = Wp, p.bias = bias, p.C = C;
  p.M = M, p.N = N, p.K = K, p.out = out_dtype;
  return mx_gemm(W4_MX_A4, p, workspace, workspace_bytes, stream);
}
