// Tiled product of many rows with MXFP4 weights.
//
// WM waves along m and WN along n own a tile of 32 TM WM x 32 TN WN
// outputs, each 32 TM x 32 TN of them on 32 x 32 matrix instructions:
// v_mfma_scale_f32_32x32x64_f8f6f4 for 4-bit and 8-bit rows (the one shape that
// multiplies 4-bit codes at twice the rate of 8-bit ones), v_mfma_f32_32x32x16_f16
// for fp16 rows, whose weights widen in registers. Weights are the row operand,
// so a lane ends with runs of four columns of C. Rows, weights and scales come to
// LDS by direct loads, a ring of NS stages of 128 k.
//
// Instructions alone, on random data, reach 4.2 PFLOP/s (4-bit weights, 8-bit rows), 6.8 (4-bit
// rows) and 1.7 (fp16); zeros a third more. A call of 2048 x 4096 x 11008, 8-bit rows, takes 75 us
// (2.5 PFLOP/s), 2048 x 11008 x 4096 72 on 4-bit rows (2.6) and 185 on fp16 rows (1.0), 777 x
// 4096 x 4096 on fp16 rows 35.
//
// Bound: the loop's matrix instructions, then its loads, then what is outside it. A stage of 128 k in
// us, whole, with all loads on one stage that the caches hold, without loads, without loads and LDS
// reads, instructions at the rates above: 8-bit rows, 128 x 256 tile, 0.78, 0.68, 0.62, 0.59, 0.51; 4-bit rows, 256 x
// 256, 1.06, 1.00, 0.79, 0.71, 0.63; fp16 rows, 128 x 256, 1.82, 1.71, 1.53, 1.41, 1.26. So a stage's loads
// cost their issue and their way into LDS, and with 8-bit rows more what comes from behind the
// caches (221 MB for 46 of operands). Launch, first loads and the result are 11 us (8-bit rows,
// 2048 x 4096 of them) and 15 (4-bit rows, 2048 x 8192).
#include "mx_gemm.hpp"

namespace w4 {

// How a block takes the scales of MXFP4 rows: not at all, as words (rows a
// multiple of 4 scales long, aligned), or as pairs of aligned words shifted.
enum { ROW_SCALES_NONE, ROW_SCALES_WORDS, ROW_SCALES_SHIFTED };

template <int ACT, int WM_, int WN_, int TM_, int TN_, int NS_, int RS_>
struct MxTile {
  static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, NS = NS_, RS = RS_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, STRIPS = BN / 16;
  static constexpr int RB = act_bytes<ACT>(128);                  // bytes of a staged row
  static constexpr int CH = RB / 16;                              // and its 16-byte chunks
  static constexpr int A_BYTES = BM * RB, W_BYTES = STRIPS * TILE_BYTES;
  static constexpr int AS_BYTES = RS * BM * 4;                    // rows' scales
  static constexpr int STAGE = A_BYTES + W_BYTES + AS_BYTES;
  // a wave's loads: rows and weights 1 KiB each, scales a word a lane
  static constexpr int A_LOADS = A_BYTES / 1024 / WAVES, W_LOADS = W_BYTES / 1024 / WAVES;
  static constexpr int AS_LOADS = (RS * BM + 64 * WAVES - 1) / (64 * WAVES);
  static constexpr int LOADS = A_LOADS + W_LOADS + AS_LOADS + 1;
  static constexpr int WS_BYTES = STRIPS * 256;                   // weights' scales of a quad of k tiles
  static constexpr int LDS = NS * STAGE + 2 * WS_BYTES;
  static constexpr bool SPLIT = BM == 64;                     // may be split along k
  static_assert(W_BYTES % (1024 * WAVES) == 0 && A_BYTES % (1024 * WAVES) == 0, "whole loads for each wave");
  static_assert(STRIPS <= 4 * WAVES && NS <= 4, "a quad's scales come during the quad before");
  static_assert(LDS <= 160 * 1024, "LDS exceeds the CU");
};

// where chunk c of a staged row lies: rows of a fragment spread over the banks
template <int CH>
__device__ __forceinline__ int mx_chunk(int row, int c) {
  return CH == 4 ? c ^ ((row >> 2) & 3) : CH == 8 ? c ^ ((row >> 1) & 7) : c ^ (row & 15);
}

// operands of 64 k for a wave's row and column tiles
template <int ACT, int TM, int TN>
struct MxFrags {
  u4 w[TN];
  u4 a[TM][ACT == W4_MX_A16 ? 4 : ACT == W4_MX_A4 ? 1 : 2];
};

// (a device function, so that the kernel's host stub holds no device assembly)
template <int ACT, typename S>
__device__ __forceinline__ void mx_gemm_tile(const MxParams& p, int mblocks, int nblocks, int per_xcd,
                                             int splits) {
  constexpr int TM = S::TM, TN = S::TN, RS = S::RS;
  using F = MxFrags<ACT, TM, TN>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int id = blockIdx.x, local = id >> 3;
  const int tix = (id & 7) * per_xcd + local;            // an XCD's tiles share their columns
  if (local >= per_xcd || tix >= mblocks * nblocks * splits) return;
  const int split = tix / (mblocks * nblocks), tile = tix - split * (mblocks * nblocks);
  const int nb = tile / mblocks, mb = tile - nb * mblocks;

  const MxGeometry geo = mx_geometry(p.N, p.K);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % S::WM, wn = wave / S::WM;
  const int l31 = lane & 31, half = lane >> 5;
  const int r = lane & 15, hi = (lane >> 4) & 1;         // this lane's weight row: strip 2 j + hi, row r
  const int m0 = mb * S::BM, t0 = p.strip0 + nb * S::STRIPS;
  const int KB = p.K / 32;
  // this block's k tiles: whole quads
  const int kt0 = 4 * (int)((int64_t)geo.KQ * split / splits);
  const int kt1 = min(geo.KT, 4 * (int)((int64_t)geo.KQ * (split + 1) / splits));
  uint8_t* const wscales = smem + S::NS * S::STAGE;      // [2 quads][strip][64 lanes] words

  // ---- direct loads to LDS -------------------------------------------------------
  // a quarter of quad q's weight scales (all of them more than once where strips are few)
  auto issue_scales = [&](int q, int piece) {
    const int strip = (piece * S::WAVES + wave) % S::STRIPS, t = min(t0 + strip, geo.NT - 1);
    __builtin_amdgcn_global_load_lds(
        p.Wp + geo.s_off + ((int64_t)t * geo.KQ + min(q, geo.KQ - 1)) * 256 + lane * 4,
        wscales + (q & 1) * S::WS_BYTES + strip * 256, 4, 0, 0);
  };
  // load q of k tile kt: rows, weights, rows' scales
  auto issue = [&](int kt, int slot, int q) {
    kt = min(kt, kt1 - 1);                               // past the end: again the last
    uint8_t* dst = smem + slot * S::STAGE;
    if (q < S::A_LOADS) {
      const int first = (wave * S::A_LOADS + q) * 1024;
      const int row = first / S::RB + lane / S::CH;
      const int c = mx_chunk<S::CH>(row, lane % S::CH);
      const int k = 128 * kt + c * (128 / S::CH);
      const uint8_t* src = p.A + (int64_t)min(m0 + row, p.M - 1) * act_bytes<ACT>(p.K) + act_bytes<ACT>(k);
      __builtin_amdgcn_global_load_lds(k < p.K ? src : mx_zeros, dst + first, 16, 0, 0);
    } else if (q < S::A_LOADS + S::W_LOADS) {
      const int strip = wave * S::W_LOADS + q - S::A_LOADS, t = min(t0 + strip, geo.NT - 1);
      __builtin_amdgcn_global_load_lds(p.Wp + ((int64_t)t * geo.KT + kt) * TILE_BYTES + lane * 16,
                                       dst + S::A_BYTES + strip * TILE_BYTES, 16, 0, 0);
    } else if constexpr (RS != ROW_SCALES_NONE) {
      // words [part][row]; shifted: the aligned words that a row's four scales lie in
      const int base = ((q - S::A_LOADS - S::W_LOADS) * S::WAVES + wave) * 64 % (RS * S::BM), item = base + lane;
      const int row = min(m0 + item % S::BM, p.M - 1), part = item / S::BM;
      uintptr_t src = (uintptr_t)(p.a_scales + (int64_t)row * KB + 4 * kt);
      if constexpr (RS == ROW_SCALES_SHIFTED) {
        const uintptr_t last = (uintptr_t)(p.a_scales + (int64_t)p.M * KB - 1) & ~(uintptr_t)3;
        src = (src & ~(uintptr_t)3) + 4 * part;
        src = src < last ? src : last;
      }
      __builtin_amdgcn_global_load_lds((const void*)src, dst + S::A_BYTES + S::W_BYTES + base * 4, 4, 0, 0);
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
      const uint8_t* w = a + S::A_BYTES + (2 * wn * TN + hi) * TILE_BYTES + (half * 16 + r) * 16 + s * 512;
      f.w[q] = *reinterpret_cast<const u4*>(w + 2 * q * TILE_BYTES);
    } else {
      const int i = (q - TN) / AF, x = (q - TN) % AF;
      const int row = 32 * (wm * TM + i) + l31;
      const int c = ACT == W4_MX_A16    ? 8 * s + 4 * half + x
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
  // every wave has read out. Weights' scales come a quarter with each stage of the
  // quad before, into the half of their place that was read at its start.
  auto turn = [&] {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S::NS - 2) * S::LOADS) : "memory");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  auto next = [](int slot) { return slot + 1 == S::NS ? 0 : slot + 1; };
  auto issue_item = [&](int kt, int slot, int q) {
    if (q < S::LOADS - 1) issue(kt, slot, q);
    else issue_scales((kt >> 2) + 1, kt & 3);
  };
#pragma unroll
  for (int q = 0; q < 4; ++q) issue_scales(kt0 >> 2, q);
#pragma unroll
  for (int q = 0; q < S::NS; ++q)
#pragma unroll
    for (int x = 0; x < S::LOADS; ++x) issue_item(kt0 + q, q, x);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S::NS - 1) * S::LOADS) : "memory");
  asm volatile("s_barrier" ::: "memory");

  // The operands of a step are read from LDS while the one before is multiplied.
  // `share` spreads n pieces of work evenly over the first `gaps` gaps.
  F f0, f1;
  int slot = 0;
#pragma unroll
  for (int q = 0; q < FETCHES; ++q) fetch(f0, 0, 0, q);
#pragma unroll
  for (int i = 0; i < TM; ++i) read_row_scales(0, i);
  auto share = [](int h, int gaps, int n, auto piece) {
#pragma unroll
    for (int q = 0; q < n; ++q)
      if (h == (2 * q + 1) * gaps / (2 * n)) piece(q);
  };
  constexpr int R = RS == ROW_SCALES_NONE ? 0 : TM;
  for (int kt = kt0; kt < kt1; ++kt) {
    if ((kt & 3) == 0) quad_scales(kt >> 2);
    row_scales(kt);
    multiply(f0, kt, 0, [&](int h) {
      share(h, GAPS - GAPS / 8, FETCHES, [&](int q) { fetch(f1, slot, 1, q); });
      __builtin_amdgcn_sched_barrier(0);
    });
    // the turn, then k tile kt + NS into the place of this one and the next one's
    // first operands
    const int now = next(slot);
    multiply(f1, kt, 1, [&](int h) {
      if (h == 0) {
        __builtin_amdgcn_sched_barrier(0);
        turn();
      }
      share(h, GAPS - GAPS / 8, FETCHES + R, [&](int q) {
        if (q < FETCHES) fetch(f0, now, 0, q);
        else read_row_scales(now, q - FETCHES);
      });
      share(h, GAPS, S::LOADS, [&](int q) { issue_item(kt + S::NS, slot, q); });
      __builtin_amdgcn_sched_barrier(0);
    });
    slot = now;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // ---- split along k: the tile's last block adds the parts, in their order -----------
  if constexpr (S::SPLIT) {
    if (splits > 1) {
      constexpr int PAIRS = TM * TN * 8, PT = PAIRS * 2 * S::THREADS;      // a thread's values in pairs; a part
      uint32_t* part = reinterpret_cast<uint32_t*>(p.part) + (int64_t)tile * splits * PT + 2 * tid;
      auto at = [&](int z, int x) { return part + (int64_t)z * PT + x * 2 * S::THREADS; };
#pragma unroll
      for (int x = 0; x < PAIRS; ++x) {
        const f16v& a = acc[x / 8 / TN][x / 8 % TN];
        dev_store2(at(split, x), __float_as_uint(a[x % 8 * 2]), __float_as_uint(a[x % 8 * 2 + 1]));
      }
      stores_done();
      __syncthreads();
      unsigned* flag = reinterpret_cast<unsigned*>(smem);
      if (tid == 0) *flag = dev_arrive(p.counters + tile) == (unsigned)(splits - 1);
      __syncthreads();
      const bool last = *flag != 0;
      __syncthreads();
      if (!last) return;
      if (tid == 0) dev_store(p.counters + tile, 0u);
      // four parts' loads go out together: each is a round trip to the level that all XCDs share
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
      for (int z0 = 0; z0 < splits; z0 += 4) {
        uint64_t v[4][PAIRS];
#pragma unroll
        for (int z = 0; z < 4; ++z)
#pragma unroll
          for (int x = 0; x < PAIRS; ++x) v[z][x] = dev_load2(at(min(z0 + z, splits - 1), x));
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          if (z0 + z >= splits) break;
#pragma unroll
          for (int x = 0; x < PAIRS; ++x) {
            f16v& a = acc[x / 8 / TN][x / 8 % TN];
            a[x % 8 * 2] += __uint_as_float((uint32_t)v[z][x]);
            a[x % 8 * 2 + 1] += __uint_as_float((uint32_t)(v[z][x] >> 32));
          }
        }
      }
    }
  }

  // ---- epilogue: lane holds row 32 (..) + l31, columns 8 (e >> 2) + 4 half + (e & 3) of
  // a tile. 32 rows at a time go through LDS, so that a row's columns are stored together.
  constexpr int WC = 32 * TN;                            // the wave's columns
  constexpr int PITCH = WC * 4 + 16;
  static_assert(S::WAVES * 32 * PITCH <= S::NS * S::STAGE, "the staged rows lie in the ring");
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

template <int ACT, typename S>
__global__ __launch_bounds__(S::THREADS, S::WAVES == 4 ? 1 : S::LDS > 80 * 1024 ? 2 : 4) void k_mx_gemm(const MxParams p, int mblocks,
                                                                                  int nblocks, int per_xcd,
                                                                                  int splits) {
  mx_gemm_tile<ACT, S>(p, mblocks, nblocks, per_xcd, splits);
}

// The tile and the split along k, from the sizes (and not from the result's type,
// which mx4_workspace_bytes does not know).
struct MxPlan {
  int bm, bn, splits;
  int64_t tiles;
  size_t ws;
  int first;                             // columns of a first launch of 256 x 256 tiles
};
static MxPlan mx_plan(int act, int M, int N, int K) {
  // The tile by the most that a CU gets of it, in units of a 256 x 256 tile's time
  // (100). us, 256 x 256, 128 x 256, 128 x 128, 64 x 128, of 8-bit rows; of 4-bit rows; of fp16
  // rows, which have no 256 x 256 tile, since its stages would not fit:
  //   2048 x 8192 x 4096   60, 71, 74, 115;   48, 55, 74, 95;    133, 174, 194
  //   2048 x 4096 x 11008  118, 79, 88, 126;  86, 63, 84, 103;   170, 195, 238
  //   777 x 4096 x 4096    47, 29, 22, 22;    36, 24, 19, 21;    56, 37, 42
  //   200 x 4096 x 4096    44, 26, 19, 14.5;  33, 22, 17, 13;    47, 29, 23
  // The units choose the least of each (777 8-bit rows: 22.0, where the last takes 21.7).
  const int bms[4] = {256, 128, 128, 64}, bns[4] = {256, 256, 128, 128}, each[4] = {100, 60, 34, 22};
  MxPlan best{};
  int64_t least = INT64_MAX;
  auto consider = [&](int first, int64_t before) {       // of the columns from `first` on
    for (int x = act == W4_MX_A16; x < 4; ++x) {
      const int64_t tiles = (int64_t)ceil_div(M, bms[x]) * ceil_div(N - first, bns[x]);
      const int64_t cost = before + (tiles + 255) / 256 * each[x];
      if (cost < least) least = cost, best = MxPlan{bms[x], bns[x], 1, tiles, 0, first};
    }
  };
  consider(0, 0);
  // Whole rounds of 256 x 256 tiles, then the other columns in the tile that is best
  // for them, a second launch (4): 2048 x 11008 x 4096 97 -> 91 us on 8-bit rows and 80 -> 76
  // on 4-bit ones, 2048 x 12288 x 4096 99 -> 94 and 82 -> 78. No such split of fp16 rows'
  // largest tile gains by this count.
  const int64_t rows = ceil_div(M, 256), rounds = rows * ceil_div(N, 256) / 256;
  if (act != W4_MX_A16 && rounds > 0) {
    const int64_t columns = 256 * (rounds * 256 / rows);
    if (columns > 0 && columns < N) consider((int)columns, rounds * each[0] + 4);
  }
  // The smallest tile where it leaves CUs without work: splits along k, of whole quads
  // of k tiles. A k tile takes 0.55, 0.3 or 0.26 us (fp16, 8-bit, 4-bit rows), the
  // exchange about 3 us and 0.017 for each block: 45 x 3200 x 8640, 8-bit rows, 26 us
  // whole, 14.7 in 4, 15.3 in 8; 200 x 4096 x 4096, fp16, 30 whole, 25 in 2 or 4.
  if (best.bm == 64 && best.tiles < 256 && best.first == 0) {
    const int KT = (K + 127) / 128, KQ = (KT + 3) / 4;
    const double t = act == W4_MX_A16 ? 0.55 : act == W4_MX_A8 ? 0.3 : 0.26;
    double least_us = t * KT;
    for (int s = 2; s <= min(KQ, 8); ++s) {
      const double us = t * 4 * ((KQ + s - 1) / s) + 3 + 0.017 * best.tiles * s;
      if (us < least_us) least_us = us, best.splits = s;
    }
  }
  if (best.splits > 1) best.ws = WS_COUNTERS + (size_t)(best.tiles * best.splits * best.bm * best.bn * 4);
  return best;
}

template <int ACT, typename S>
int launch_tile(const MxParams& p, const MxPlan& plan, hipStream_t stream) {
  // (the columns from p.strip0 on)
  const int64_t blocks = plan.tiles * plan.splits;
  if (blocks > (1 << 22)) return W4_ERR_SHAPE;
  const int per_xcd = (int)((blocks + 7) / 8);
  allow_smem((const void*)&k_mx_gemm<ACT, S>, S::LDS);
  hipLaunchKernelGGL((k_mx_gemm<ACT, S>), dim3(per_xcd * 8), dim3(S::THREADS), S::LDS, stream, p,
                     ceil_div(p.M, S::BM), (int)(plan.tiles / ceil_div(p.M, S::BM)), per_xcd, plan.splits);
  return launch_status();
}

// Stages: what the CU's LDS holds, two blocks of it for the smaller tiles. fp16 rows
// take eight waves (2048 x 11008 x 4096 185 us, 205 on four; 777 x 4096 x 4096 36,
// 42), which hide the widening of the weights, 8-bit and 4-bit rows four (2048 x
// 8192 x 4096 67 and 50 us, 93 and 52 on eight).
template <int ACT, int RS>
int launch_gemm(MxParams p, hipStream_t stream) {
  const MxPlan plan = mx_plan(ACT == MX_A8_EXACT ? W4_MX_A8 : ACT, p.M, p.N, p.K);
  if constexpr (ACT == W4_MX_A16) {
    if (plan.bn == 256) return launch_tile<ACT, MxTile<ACT, 2, 4, 2, 2, 3, RS>>(p, plan, stream);
    if (plan.bm == 128) return launch_tile<ACT, MxTile<ACT, 2, 4, 2, 1, 3, RS>>(p, plan, stream);
    return launch_tile<ACT, MxTile<ACT, 2, 4, 1, 1, 3, RS>>(p, plan, stream);
  } else {
    constexpr int NS = ACT == W4_MX_A4 ? 4 : 3;
    if (plan.first > 0) {
      const MxPlan whole{256, 256, 1, (int64_t)ceil_div(p.M, 256) * (plan.first / 256), 0, 0};
      if (const int st = launch_tile<ACT, MxTile<ACT, 2, 2, 4, 4, NS, RS>>(p, whole, stream)) return st;
      p.strip0 = plan.first / 16;
    }
    if (plan.bm == 256) return launch_tile<ACT, MxTile<ACT, 2, 2, 4, 4, NS, RS>>(p, plan, stream);
    if (plan.bn == 256) return launch_tile<ACT, MxTile<ACT, 2, 2, 2, 4, 4, RS>>(p, plan, stream);
    if (plan.bm == 128) return launch_tile<ACT, MxTile<ACT, 2, 2, 2, 2, NS, RS>>(p, plan, stream);
    return launch_tile<ACT, MxTile<ACT, 2, 2, 1, 2, 4, RS>>(p, plan, stream);
  }
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

// Few rows stream the weights. 33 to 64 rows: up to 768 strips (N = 12288), three a CU:
// 64 x 11008 x 4096 rows 24.6, 13.0, 13.5 us (fp16, 8-bit, 4-bit), tiles 22.6, 14.6,
// 13.7; 64 x 4096 x 4096 18.8, 10.5, 10.3 and 17, 12, 12; 64 x 22016 x 4096 45, 25, 27
// and 24, 15, 14.
static bool few_rows(int M, int N) { return M <= 32 || (M <= 64 && N <= 768 * 16); }

static bool mx_gemm_sizes_ok(int M, int N, int K) {
  return M >= 0 && M <= (1 << 30) && prepack_mx4_bytes(N, K) != 0;
}

extern "C" size_t mx4_workspace_bytes(int op, int M, int N, int K) {
  if (op < W4_MX_A16 || op > W4_MX_A4 || !mx_gemm_sizes_ok(M, N, K) || M == 0) return 0;
  return few_rows(M, N) ? 0 : mx_plan(op, M, N, K).ws;
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
  return few_rows(p.M, p.N) ? launch_mx_rows(act, p, stream) : launch_mx_gemm(act, p, stream);
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
