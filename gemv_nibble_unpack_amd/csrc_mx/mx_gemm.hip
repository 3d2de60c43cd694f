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

// How a block takes the scales of MXFP4 rows: not at all, as words (rows a
// multiple of 4 scales long, aligned), or as pairs of aligned words shifted.
enum { ROW_SCALES_NONE, ROW_SCALES_WORDS, ROW_SCALES_SHIFTED };

template <int ACT, int TM, int TN, int NS_, int RS>
struct MxTile {
  static constexpr int NS = NS_;
  static constexpr int BM = 64 * TM, BN = 64 * TN, STRIPS = BN / 16;
  static constexpr int TK = ACT == W4_MX_A16 ? 64 : 128;          // k of a stage
  static constexpr int QS = 512 / TK;                             // stages of a quad of k tiles
  static constexpr int RB = act_bytes<ACT>(TK);                   // bytes of a staged row
  static constexpr int CH = RB / 16;                              // and its 16-byte chunks
  static constexpr int WB = 8 * TK;                               // bytes of a staged strip
  static constexpr int A_BYTES = BM * RB, W_BYTES = STRIPS * WB;
  static constexpr int AS_BYTES = RS * BM * 4;                    // rows' scales
  static constexpr int STAGE = A_BYTES + W_BYTES + AS_BYTES;
  static constexpr int A_LOADS = A_BYTES / 4096, W_LOADS = W_BYTES / 4096;   // a wave's, of 1 KiB
  static constexpr int AS_LOADS = (RS * BM + 255) / 256;          // of 256 bytes
  static constexpr int LOADS = A_LOADS + W_LOADS + AS_LOADS + 1;  // and one of weights' scales
  static constexpr int WS_BYTES = STRIPS * 256;                   // weights' scales of a quad
  static constexpr int LDS = NS * STAGE + 2 * WS_BYTES;
  static_assert(A_BYTES % 4096 == 0 && W_BYTES % 4096 == 0, "whole loads for each wave");
  static_assert(STRIPS <= 4 * QS && NS <= QS, "a quad's scales come during the quad before");
  static_assert(LDS <= 160 * 1024, "LDS exceeds the CU");
};

// where chunk c of a staged row lies: rows of a fragment spread over the banks
template <int CH>
__device__ __forceinline__ int mx_chunk(int row, int c) {
  return CH == 4 ? c ^ ((row >> 2) & 3) : c ^ ((row >> 1) & 7);
}

// operands of 64 k for a wave's row and column tiles
template <int ACT, int TM, int TN>
struct MxFrags {
  u4 w[TN];
  u4 a[TM][ACT == W4_MX_A16 ? 4 : ACT == W4_MX_A4 ? 1 : 2];
};

// (a device function, so that the kernel's host stub holds no device assembly)
template <int ACT, int TM, int TN, int NS_, int RS>
__device__ __forceinline__ void mx_gemm_tile(const MxParams& p, int mblocks, int nblocks, int per_xcd) {
  using S = MxTile<ACT, TM, TN, NS_, RS>;
  using F = MxFrags<ACT, TM, TN>;
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
  const int r = lane & 15, hi = (lane >> 4) & 1;         // this lane's weight row: strip 2 j + hi, row r
  const int m0 = mb * S::BM, t0 = nb * S::STRIPS;
  const int KB = p.K / 32;
  const int nst = geo.KT * (128 / S::TK);
  uint8_t* const wscales = smem + S::NS * S::STAGE;      // [2 quads][strip][64 lanes] words

  // ---- direct loads to LDS -------------------------------------------------------
  // a sixteenth or more of quad q's weight scales: strips 4 piece .. (twice where there are fewer)
  auto issue_scales = [&](int q, int piece) {
    const int strip = (4 * piece + wave) % S::STRIPS;
    const int t = min(t0 + strip, geo.NT - 1);
    __builtin_amdgcn_global_load_lds(
        p.Wp + geo.s_off + ((int64_t)t * geo.KQ + min(q, geo.KQ - 1)) * 256 + lane * 4,
        wscales + (q & 1) * S::WS_BYTES + strip * 256, 4, 0, 0);
  };
  // load q of a stage: rows, weights, rows' scales
  auto issue = [&](int st, int slot, int q) {
    st = min(st, nst - 1);                               // past the end: again the last
    uint8_t* dst = smem + slot * S::STAGE;
    if (q < S::A_LOADS) {
      constexpr int RPL = 64 / S::CH;                    // rows of a load
      const int row = (wave * S::A_LOADS + q) * RPL + lane / S::CH;
      const int c = mx_chunk<S::CH>(row, lane % S::CH);
      const int k = st * S::TK + c * (S::TK / S::CH);
      const uint8_t* src = p.A + (int64_t)min(m0 + row, p.M - 1) * act_bytes<ACT>(p.K) + act_bytes<ACT>(k);
      __builtin_amdgcn_global_load_lds(k < p.K ? src : mx_zeros, dst + (wave * S::A_LOADS + q) * 1024,
                                       16, 0, 0);
    } else if (q < S::A_LOADS + S::W_LOADS) {
      q -= S::A_LOADS;
      constexpr int LPS = S::WB / 16;                    // lanes of a strip: 64 or 32
      const int strip = (wave * S::W_LOADS + q) * (64 / LPS) + lane / LPS;
      const int t = min(t0 + strip, geo.NT - 1);
      const uint8_t* src = p.Wp + (int64_t)t * geo.KT * TILE_BYTES + (int64_t)st * S::WB + (lane % LPS) * 16;
      __builtin_amdgcn_global_load_lds(src, dst + S::A_BYTES + (wave * S::W_LOADS + q) * 1024, 16, 0, 0);
    } else if constexpr (RS != ROW_SCALES_NONE) {
      q -= S::A_LOADS + S::W_LOADS;
      // words [part][row]; shifted: the aligned words that a row's four scales lie in
      const int item = ((q * 4 + wave) * 64 + lane) % (RS * S::BM);
      const int row = min(m0 + item % S::BM, p.M - 1), part = item / S::BM;
      uintptr_t src = (uintptr_t)(p.a_scales + (int64_t)row * KB + 4 * st);
      if constexpr (RS == ROW_SCALES_SHIFTED) {
        const uintptr_t last = (uintptr_t)(p.a_scales + (int64_t)p.M * KB - 1) & ~(uintptr_t)3;
        src = (src & ~(uintptr_t)3) + 4 * part;
        src = src < last ? src : last;
      }
      __builtin_amdgcn_global_load_lds((const void*)src,
                                       dst + S::A_BYTES + S::W_BYTES + ((q * 4 + wave) * 256) % S::AS_BYTES,
                                       4, 0, 0);
    }
  };

  f16v acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  uint32_t sw[TN][2];                                    // [column tile][block pair]: a byte a k tile
  uint32_t sa[RS == ROW_SCALES_NONE ? 1 : TM];           // [row tile]: bytes of blocks half, half + 2
  uint32_t top[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j)
    top[j] = mx_half(ACT) ? p.Wp[geo.e_off + 16 * (int64_t)min(t0 + 2 * (wn * TN + j) + hi, geo.NT - 1) + r] : 0;
  uint32_t shift[RS == ROW_SCALES_SHIFTED ? TM : 1];     // of a row's scales in their words, in bytes
  if constexpr (RS == ROW_SCALES_SHIFTED) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
      shift[i] = (uint32_t)((uintptr_t)(p.a_scales + (int64_t)min(m0 + 32 * (wm * TM + i) + l31, p.M - 1) * KB) & 3);
  }

  auto quad_scales = [&](int q) {
    const uint8_t* w = wscales + (q & 1) * S::WS_BYTES + (2 * wn * TN + hi) * 256 + (half * 16 + r) * 4;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s) sw[j][s] = *reinterpret_cast<const uint32_t*>(w + j * 512 + s * 128);
  };
  uint32_t raw[RS == ROW_SCALES_NONE ? 1 : TM][RS == ROW_SCALES_SHIFTED ? 2 : 1];
  auto read_row_scales = [&](int slot, int i) {
    if constexpr (RS != ROW_SCALES_NONE) {
      const uint8_t* w = smem + slot * S::STAGE + S::A_BYTES + S::W_BYTES + 4 * (32 * (wm * TM + i) + l31);
#pragma unroll
      for (int x = 0; x < RS; ++x) raw[i][x] = *reinterpret_cast<const uint32_t*>(w + 4 * S::BM * x);
    }
  };
  auto row_scales = [&](int kt) {
    if constexpr (RS != ROW_SCALES_NONE) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        uint32_t v = raw[i][0];
        if constexpr (RS == ROW_SCALES_SHIFTED) {
          v = __builtin_amdgcn_alignbyte(raw[i][1], v, shift[i]);
          // scales past the row's end may be NaN
          const int left = KB - 4 * kt;
          if (left < 4) v &= (1u << (8 * max(left, 0))) - 1u;
        }
        sa[i] = v >> (8 * half);
      }
    }
  };
  // operand q of step s (64 k) of a stage
  constexpr int AF = sizeof(F::a) / 16 / TM, FETCHES = TN + TM * AF;
  auto fetch = [&](F& f, int slot, int s, int q) {
    const uint8_t* a = smem + slot * S::STAGE;
    if (q < TN) {
      const uint8_t* w = a + S::A_BYTES + (2 * wn * TN + hi) * S::WB + (half * 16 + r) * 16 + s * 512;
      f.w[q] = *reinterpret_cast<const u4*>(w + 2 * q * S::WB);
    } else {
      const int i = (q - TN) / AF, x = (q - TN) % AF;
      const int row = 32 * (wm * TM + i) + l31;
      const int c = ACT == W4_MX_A16    ? 4 * half + x
                    : ACT == W4_MX_A8   ? 4 * s + 2 * x + half          // k 16 half .. and 32 + 16 half ..
                    : ACT == MX_A8_EXACT ? 4 * s + 2 * half + x
                                         : 2 * s + half;
      f.a[i][x] = *reinterpret_cast<const u4*>(a + row * S::RB + 16 * mx_chunk<S::CH>(row, c));
    }
  };
  auto v8 = [](const u4 x, const u4 y) {
    return v8i{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
  };
  // step s of k tile kt; between the products, `between(h)` for h < GAPS: what is
  // not a matrix instruction costs its own time only where none is running
  constexpr int GAPS = mx_half(ACT) ? 4 * TN : TM * TN;
  auto multiply = [&](const F& f, int kt, int s, auto between) {
    if constexpr (mx_half(ACT)) {
      h8 af[TM][4];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if constexpr (ACT == W4_MX_A16) af[i][x] = __builtin_bit_cast(h8, f.a[i][x]);
          else af[i][x] = fp8_h8(f.a[i][x / 2][2 * (x & 1)], f.a[i][x / 2][2 * (x & 1) + 1]);
        }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const float up = h_scale((sw[j][s] >> (8 * (kt & 3))) & 255u, top[j]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const h8 b = fp4_h8(f.w[j][x], up);
#pragma unroll
          for (int i = 0; i < TM; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, af[i][x], acc[i][j], 0, 0, 0);
          between(4 * j + x);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const v8i b = {(int)f.w[j][0], (int)f.w[j][1], (int)f.w[j][2], (int)f.w[j][3]};
        const uint32_t sb = sw[j][s] >> (8 * (kt & 3));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          if constexpr (ACT == W4_MX_A8)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, v8(f.a[i][0], f.a[i][1]), acc[i][j],
                                                                        4, 0, 0, sb, 0, 127);
          else if (s == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                b, v8i{(int)f.a[i][0][0], (int)f.a[i][0][1], (int)f.a[i][0][2], (int)f.a[i][0][3]},
                acc[i][j], 4, 4, 0, sb, 0, sa[i]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                b, v8i{(int)f.a[i][0][0], (int)f.a[i][0][1], (int)f.a[i][0][2], (int)f.a[i][0][3]},
                acc[i][j], 4, 4, 0, sb, 2, sa[i]);
          between(TM * j + i);
        }
      }
    }
  };

  // Ring of NS stages. Every stage issues the same loads, so a fixed count waits
  // for the next stage's alone; the barrier publishes it and frees the stage that
  // every wave has read out.
  auto turn = [&] {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S::NS - 2) * S::LOADS) : "memory");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  auto next = [](int slot) { return slot + 1 == S::NS ? 0 : slot + 1; };
  auto issue_item = [&](int st, int slot, int q) {
    if (q < S::LOADS - 1) issue(st, slot, q);
    else issue_scales(st / S::QS + 1, st % S::QS);
  };
#pragma unroll
  for (int q = 0; q < S::QS; ++q) issue_scales(0, q);
#pragma unroll
  for (int q = 0; q < S::NS; ++q)
#pragma unroll
    for (int x = 0; x < S::LOADS; ++x) issue_item(q, q, x);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S::NS - 1) * S::LOADS) : "memory");
  asm volatile("s_barrier" ::: "memory");

  // The operands of a step are read from LDS while the one before is multiplied.
  // `share` spreads n pieces of work evenly over the first `gaps` gaps.
  F f0, f1;
  int slot = 0, st = 0;
#pragma unroll
  for (int q = 0; q < FETCHES; ++q) fetch(f0, 0, 0, q);
#pragma unroll
  for (int i = 0; i < TM; ++i) read_row_scales(0, i);
  auto share = [](int h, int gaps, int n, auto piece) {
#pragma unroll
    for (int q = 0; q < n; ++q)
      if (h == (2 * q + 1) * gaps / (2 * n)) piece(q);
  };
  // within the last step of stage st: the turn, then stage st + NS into its place
  // and the next stage's first operands into `f`
  auto advance = [&](int h, F& f) {
    if (h == 0) {
      __builtin_amdgcn_sched_barrier(0);
      turn();
    }
    const int old = slot, now = next(slot);
    constexpr int R = RS == ROW_SCALES_NONE ? 0 : TM;
    share(h, GAPS - GAPS / 8, FETCHES + R, [&](int q) {
      if (q < FETCHES) fetch(f, now, 0, q);
      else read_row_scales(now, q - FETCHES);
    });
    share(h, GAPS, S::LOADS, [&](int q) { issue_item(st + S::NS, old, q); });
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int kt = 0; kt < geo.KT; ++kt) {
    if ((kt & 3) == 0) quad_scales(kt >> 2);
    row_scales(kt);
    if constexpr (S::TK == 64) {                         // two stages a k tile
      multiply(f0, kt, 0, [&](int h) { advance(h, f1); });
      slot = next(slot);
      ++st;
    } else {
      multiply(f0, kt, 0, [&](int h) {
        share(h, GAPS - GAPS / 8, FETCHES, [&](int q) { fetch(f1, slot, 1, q); });
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    multiply(f1, kt, 1, [&](int h) { advance(h, f0); });
    slot = next(slot);
    ++st;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // ---- epilogue: lane holds row 32 (..) + l31, columns 8 (e >> 2) + 4 half + (e & 3) of
  // a tile. 32 rows at a time go through LDS, so that a row's columns are stored together.
  constexpr int WC = 32 * TN;                            // the wave's columns
  constexpr int PITCH = WC * 4 + 16;
  static_assert(4 * 32 * PITCH <= S::NS * S::STAGE, "the staged rows lie in the ring");
  uint8_t* cw = smem + wave * 32 * PITCH;
  const int n0 = 16 * t0 + wn * WC;
  auto store = [&](auto half_out) {
    constexpr bool HO = decltype(half_out)::value;
    constexpr int EB = HO ? 2 : 4, PER = WC * EB / 16, WIDE = 16 / EB;   // 16-byte pieces of a row
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      __builtin_amdgcn_sched_barrier(0);                 // one tile's values in registers at a time
      const int mi = m0 + 32 * (wm * TM + i);
      const float as = mx_row8(ACT) ? p.a_scale[min(mi + l31, p.M - 1)] : 1.f;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 32 * j + 8 * q + 4 * half, n = n0 + c;
          f4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
          if constexpr (mx_half(ACT)) {
            const uint32_t tops = *reinterpret_cast<const uint32_t*>(p.Wp + geo.e_off + min(n, 16 * geo.NT - 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = ldexpf(v[e], (int)(tops >> (8 * e) & 255u) - 127 - H_UP);
          }
          if constexpr (mx_row8(ACT)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] *= as;
          }
          if constexpr (HO) {
            if (p.bias) {
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += h2f(p.bias[min(n + e, p.N - 1)]);
            }
            h4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = (_Float16)v[e];
            *reinterpret_cast<u2*>(cw + l31 * PITCH + 2 * c) = __builtin_bit_cast(u2, h);
          } else {
            *reinterpret_cast<f4*>(cw + l31 * PITCH + 4 * c) = v;
          }
        }
      uint8_t* C = reinterpret_cast<uint8_t*>(p.C);
      if (p.N % WIDE == 0) {
        constexpr int PIECES = 32 * PER / 64;
        u4 v[PIECES];
#pragma unroll
        for (int x = 0; x < PIECES; ++x)
          v[x] = *reinterpret_cast<const u4*>(cw + (64 * x + lane) / PER * PITCH + (64 * x + lane) % PER * 16);
#pragma unroll
        for (int x = 0; x < PIECES; ++x) {
          const int row = (64 * x + lane) / PER, c = (64 * x + lane) % PER * WIDE;
          if (mi + row < p.M && n0 + c < p.N)
            *reinterpret_cast<u4*>(C + ((int64_t)(mi + row) * p.N + n0 + c) * EB) = v[x];
        }
      } else {
        typedef typename std::conditional<HO, uint16_t, uint32_t>::type E;
        for (int x = lane; x < 32 * WC; x += 64) {
          const int row = x / WC, c = x % WC;
          if (mi + row < p.M && n0 + c < p.N)
            *reinterpret_cast<E*>(C + ((int64_t)(mi + row) * p.N + n0 + c) * EB) =
                *reinterpret_cast<const E*>(cw + row * PITCH + EB * c);
        }
      }
    }
  };
  if (p.out == W4_OUT_F16) store(std::true_type{});
  else store(std::false_type{});
}

template <int ACT, int TM, int TN, int NS, int RS>
__global__ __launch_bounds__(256, 1) void k_mx_gemm(const MxParams p, int mblocks, int nblocks,
                                                    int per_xcd) {
  mx_gemm_tile<ACT, TM, TN, NS, RS>(p, mblocks, nblocks, per_xcd);
}

template <int ACT, int TM, int TN, int NS, int RS>
int launch_tile(const MxParams& p, hipStream_t stream) {
  using S = MxTile<ACT, TM, TN, NS, RS>;
  const int mblocks = ceil_div(p.M, S::BM), nblocks = ceil_div(p.N, S::BN);
  const int64_t tiles = (int64_t)mblocks * nblocks;
  if (tiles > (1 << 23)) return W4_ERR_SHAPE;
  const int per_xcd = (int)((tiles + 7) / 8);
  allow_smem((const void*)&k_mx_gemm<ACT, TM, TN, NS, RS>, S::LDS);
  hipLaunchKernelGGL((k_mx_gemm<ACT, TM, TN, NS, RS>), dim3(per_xcd * 8), dim3(256), S::LDS, stream, p,
                     mblocks, nblocks, per_xcd);
  return launch_status();
}

// The tile by the most that a CU gets of it, in units of a 256 x 256 tile's time (100):
// a 128 x 256 one costs 60 of it (4-bit rows 65), a 128 x 128 one 34 (46), a 64 x 128
// one 22 (32). 2048 rows (8-bit, us): N = 8192, K = 4096 67, 74, 81 for the first
// three; N = 4096, K = 11008 108, 73, 88; 777 rows, N = K = 4096 44, 28, 21.
template <int ACT, int RS>
int launch_gemm(const MxParams& p, hipStream_t stream) {
  constexpr bool A4 = ACT == W4_MX_A4;
  auto cost = [&](int bm, int bn, int each) {
    const int64_t tiles = (int64_t)ceil_div(p.M, bm) * ceil_div(p.N, bn);
    return (tiles + 255) / 256 * each;
  };
  const int64_t c[4] = {cost(256, 256, 100), cost(128, 256, A4 ? 65 : 60), cost(128, 128, A4 ? 46 : 34),
                        cost(64, 128, A4 ? 32 : 22)};
  const int64_t least = min(min(c[0], c[1]), min(c[2], c[3]));
  if (least == c[0]) return launch_tile<ACT, 4, 4, A4 ? 4 : 3, RS>(p, stream);
  if (least == c[1]) return launch_tile<ACT, 2, 4, A4 ? 4 : 3, RS>(p, stream);
  if (least == c[2]) return launch_tile<ACT, 2, 2, A4 ? 4 : 3, RS>(p, stream);
  return launch_tile<ACT, 1, 2, 4, RS>(p, stream);
}

int launch_mx_gemm(int act, const MxParams& p, hipStream_t stream) {
  if (act == W4_MX_A16) return launch_gemm<W4_MX_A16, ROW_SCALES_NONE>(p, stream);
  if (act == W4_MX_A8)
    return p.out == W4_OUT_F32 ? launch_gemm<MX_A8_EXACT, ROW_SCALES_NONE>(p, stream)
                               : launch_gemm<W4_MX_A8, ROW_SCALES_NONE>(p, stream);
  return p.K % 128 == 0 && aligned(p.a_scales, 4) ? launch_gemm<W4_MX_A4, ROW_SCALES_WORDS>(p, stream)
                                                  : launch_gemm<W4_MX_A4, ROW_SCALES_SHIFTED>(p, stream);
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
