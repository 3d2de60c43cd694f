// Attention of many new tokens (prompts, chunks of prompts) over the paged
// 8-bit cache.
//
// A block takes two tiles of 128 query rows of a (sequence, kv head), 32 for
// each of its eight waves: the k-th tile from the end of the sequence's rows
// (A, waves 0-3) and the k-th from the start (B, waves 4-7). It walks the cached
// tokens in turns of two steps of 64. While both tiles see the turn's tokens,
// every wave takes both steps; once tile B is done, waves 4-7 store it and turn
// to tile A, of which each group then takes one step a turn, joined at the
// end. So every SIMD has two busy waves throughout, all blocks of a prompt
// have the same number of turns, and a turn's codes are fetched and widened
// (exactly, to fp16) once for all. They are laid in LDS in the order in which
// the matrix instructions read them; the next turn's codes are in flight
// meanwhile (registers, then the other of two LDS stages). Head dims above 128
// need the registers of two waves for one: there a block is four waves, one
// tile, one step a turn. Per wave and step, with v_mfma_f32_32x32x16_f16:
//
//   S^T = K q^T    64 tokens x 32 rows
//   w   = 2^(S a - m) * v_scale / r    one fma and one exponential an element
//   O^T += V^T w^T
//
// Token order: row i = 8 x + 4 g + y of a K operand is token 16 g + 4 x + y of its
// 32, so that lane (column c, half g) of the product holds the 16 consecutive
// tokens 16 g .. 16 g + 15 of one page (one key and one value scale a lane), which
// are, 8 at a time, the k slots that the same lane feeds to the second product:
// the weights never leave their registers.
//
// The running maximum is raised (and O, the sum rescaled) only when a row's
// new maximum exceeds it by more than 8 in log2 units, or a value scale
// arrives that is more than twice r, the largest one at the last such turn;
// until then weights in units of r stay below 2^9, which P_UP_MANY = 2^6 keeps
// inside fp16 (below 2^15).
//
// Bound: in the long run instruction issue. A wave's step is 32 matrix instructions
// (1024 clocks of the matrix core) and about 340 vector ones beside 32 exponentials;
// vector instructions issue only in about half of a matrix instruction's clocks,
// and a turn adds the widening. 2048 tokens of 32 heads of 128 take 64 us for every
// 2048 cached tokens before them (measured to 8192; 4.0 us a turn, 1.07 PFLOP/s, where a
// large fp16 library product reaches 1165 TFLOP/s). Over themselves they take 52
// to 61 us over boxes, 560 to 660 TFLOP/s, the matrix cores busy 24% of the time,
// where that rate would take 32: the rest, not measured apart, are a block's start
// and end, the masked part of the diagonal, and the second phase, whose turns fetch
// and widen as much for half the products. 256 rows over 8192 tokens of 256 heads
// 310 us, 890 TFLOP/s. Measured beside it: one tile of 128 rows a block, two blocks a
// CU 74 us; both tiles in a block, but the long one's waves alone at the end 65;
// the next step's first product under this step's exponentials 65 to 83
// (registers).

#include "attn.hpp"

namespace w4 {

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr float P_UP_MANY = 64.0f, LOG2_P_UP_MANY = 6.0f;
constexpr float M_SLACK = 8.0f, R_SLACK = 2.0f;
constexpr float REF_MIN_MANY = 0x1p-100f;
constexpr float RATIO_MIN = 0x1p-40f;     // of r; weights times this round to zero

// max over the two halves of a wave, left in every lane
__device__ __forceinline__ float halves_max(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <int DP>
struct AttnMany {
  static constexpr int STEP = 64, ROWS = MANY_ROWS, PAIR = many_pair(DP) ? 2 : 1;
  static constexpr int THREADS = 256 * PAIR;
  static constexpr int KS = DP / 16;                 // k steps of the first product
  static constexpr int DT = DP / 32;                 // dim tiles of the second
  static constexpr int NS = PAIR, TURN = STEP * NS;  // steps, tokens of a turn
  static constexpr int CH = 4 * DP;                  // 16-code chunks of K (and of V) a step
  static constexpr int PER = (CH + THREADS - 1) / THREADS;   // chunks per thread and step
  // a fragment: 64 lanes x 16 bytes in lane order, with gaps after each half
  // and each fragment that put the eight 16-byte pieces which eight lanes
  // store at a time (eight fragments of a token, or two dims x four groups of
  // tokens) into different banks
  static constexpr int HALF = 512 + 32, FRAG = 2 * HALF + 32;
  static constexpr int K_FRAGS = 2 * KS, V_FRAGS = 4 * DT;
  static constexpr int STAGE = (K_FRAGS + V_FRAGS) * FRAG;
  static constexpr int LDS = 2 * NS * STAGE + 16;
  // joining tile A's two halves: per row DP floats (4 of padding) and m, l, r
  static constexpr int OROW = DP + 4;
  static_assert(ROWS * (OROW + 3) * 4 <= 2 * NS * STAGE, "the join fits the stages");
};

// The sequence that takes the rank-th place by cached length, longest first
// (equal ones by number): blocks start in the order of their ids, and what
// starts last should be short. 4, 8, 16 and 32 sequences of 20 to 900 new tokens
// over 950 to 4800, in any order, 32 and 8 heads of 128: 154, 212, 416 and 851
// us; in the caller's order, pairs slowest, 285, 395, 602 and 1067. Batches above
// a wave's lanes have blocks for many rounds and keep their order. (In the
// kernel of few rows the lookup costs more than the order gives: 64 single
// tokens over 2 to 4096 67 to 62 us, but 32 over 1500 24.6 to 26.9.)
__device__ __forceinline__ int by_length(const AttnParams& p, int rank) {
  if (p.batch == 1 || p.batch > 64) return rank;
  const int lane = threadIdx.x & 63;
  const int mine = lane < p.batch ? p.kv_len[lane] : 0;
  int before = 0;
  for (int j = 0; j < p.batch; ++j) {
    const int other = __builtin_amdgcn_readlane(mine, j);
    before += other > mine || (other == mine && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < p.batch && before == rank));
}

template <int DP, int Q>
__global__ __launch_bounds__(AttnMany<DP>::THREADS) void k_attn_many(const AttnParams p) {
  using C = AttnMany<DP>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  unsigned* slast = reinterpret_cast<unsigned*>(smem + C::LDS - 16);

  // heads fastest (a head's blocks share an XCD's L2 when kv_heads is a
  // multiple of 8), then the pairs of row tiles of a sequence, which read the same
  // codes, then sequences from the longest, parts slowest
  int t = block_number();          // past the grid's end: split >= parts below
  const int h = t % p.kv_heads;
  t /= p.kv_heads;
  const int pair = t % p.tiles;
  t /= p.tiles;
  const int b = by_length(p, t % p.batch);
  const int split = t / p.batch;

  int row0, n, len;
  bool fits;
  if (!attn_span(p, b, row0, n, len, fits)) return;
  const int rows = min(n, p.max_q) * p.group;
  // tile A is the pair-th from the end of this sequence's tiles, tile B the
  // pair-th from its start (absent where the two meet)
  const int tiles = (rows + C::ROWS - 1) / C::ROWS;
  const int ta = tiles - 1 - pair, tb = C::PAIR == 2 && pair < ta ? pair : -1;
  if (ta < (C::PAIR == 2 ? pair : 0)) return;
  const int first = len - n;
  const int seen = fits ? max(0, first + (min((ta + 1) * C::ROWS, rows) - 1) / p.group + 1) : 0;
  const int parts = max(1, (seen + p.chunk - 1) / p.chunk);
  if (split >= parts) return;

  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, g = lane >> 5;
  const int P = 1 << p.page_shift;
  const uint32_t page_bytes = (uint32_t)p.kv_heads * DP << p.page_shift;
  const uint8_t* khead = p.kc + ((int64_t)h * DP << p.page_shift);
  const uint8_t* vhead = p.vc + ((int64_t)h * DP << p.page_shift);
  const int32_t* tab = p.table + (size_t)b * p.cols;
  const int c0 = split * p.chunk, c1 = min(seen, c0 + p.chunk);
  const int last16 = (max(seen, 1) - 1) & ~15;

  // ---- this lane's query row of a tile ---------------------------------------
  const int group = C::PAIR == 2 ? wave >> 2 : 0;    // waves 0-3 / 4-7
  int wr, lim, lim_all, lim_any;
  h8 qf[C::KS];
  // row c of the wave: token of the sequence, query head
  auto row_of = [&](int& tok, int& hh) {
    const int r = min(wr + c, rows - 1);
    tok = r / p.group, hh = h * p.group + (r - tok * p.group);
    return wr + c < rows;
  };
  auto take_rows = [&](int tile) {                   // tile < 0: no rows
    wr = tile >= 0 ? tile * C::ROWS + 32 * (wave & 3) : rows;
    int tok, hh;
    const bool in = row_of(tok, hh);
    lim = in && fits ? first + tok + 1 : 0;
    // tokens that every / some row of the wave sees
    lim_all = wr + 31 < rows && fits ? first + wr / p.group + 1 : 0;
    lim_any = wr < rows && fits ? first + min(wr + 31, rows - 1) / p.group + 1 : 0;
    const uint16_t* q = p.q + (int64_t)(row0 + tok) * p.q_stride + (int64_t)hh * p.dim;
    auto quad = [&](int d) {
      return d < p.dim ? *reinterpret_cast<const u2*>(q + d) : u2{0u, 0u};
    };
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
      const u2 x = quad(16 * s + 8 * g), y = quad(16 * s + 8 * g + 4);
      qf[s] = __builtin_bit_cast(h8, u4{x[0] ^ p.q_sign, x[1] ^ p.q_sign, y[0] ^ p.q_sign,
                                        y[1] ^ p.q_sign});
    }
  };
  take_rows(group == 0 ? ta : tb);
  // the two waves of a SIMD run the same code from the same barrier; without a
  // preference waves 4-7 lagged by 1500 cycles a turn, which 0-3 then waited for
  if (group == 1) __builtin_amdgcn_s_setprio(2);

  // ---- one turn's codes: registers, then LDS ------------------------------
  // Lane i of a wave holds group i % (4 NS) (16 tokens) of a turn: its page
  // number (fetched a turn before its codes) and its scales. Groups past the
  // last visible token repeat the last one.
  u4 kraw[C::NS][C::PER], vraw[C::NS][C::PER];
  float ksl, vsl;
  uint32_t bad;
  int idl;
  auto at16 = [&](int t0, int gi) { return min(t0 + 16 * gi, last16); };
  auto load_ids = [&](int t0) { idl = tab[at16(t0, lane & (4 * C::NS - 1)) >> p.page_shift]; };
  auto load_codes = [&](int t0, int s, int id) {
    const int ts = t0 + C::STEP * s, gv = tid & 3;
    // values: a thread's chunks belong to group tid & 3 (lanes 4 apart hold
    // the turn's two steps)
    const uint32_t iv = C::NS == 1 ? id : s == 0 ? __builtin_amdgcn_ds_swizzle(id, 0x001B)
                                                 : __builtin_amdgcn_ds_swizzle(id, 0x009B);
    const uint8_t* vp = vhead + (uint64_t)iv * page_bytes + (at16(ts, gv) & (P - 1));
#pragma unroll
    for (int i = 0; i < C::PER; ++i) {
      const int idx = tid + C::THREADS * i;
      const int tk = idx / (DP / 16), j = idx % (DP / 16);
      // keys: 16 tokens are DP chunks, whole waves of them at these dims
      constexpr bool whole = DP % 64 == 0 && DP != 192;
      const int gk = whole ? __builtin_amdgcn_readfirstlane(min(tk >> 4, 3)) : min(tk >> 4, 3);
      const uint32_t ik = whole ? __builtin_amdgcn_readlane(id, 4 * s + gk) : __shfl(id, 4 * s + gk, 64);
      if (C::CH % C::THREADS == 0 || idx < C::CH) {
        kraw[s][i] = *reinterpret_cast<const u4*>(
            khead + (uint64_t)ik * page_bytes + (at16(ts, gk) & (P - 1)) * DP + (tk & 15) * DP +
            16 * j);
        vraw[s][i] = *reinterpret_cast<const u4*>(vp + ((idx >> 2) << p.page_shift));
      }
    }
  };
  auto load = [&](int t0) {
    const bool ok = idl >= 0 && idl < p.pages;
    const int id = ok ? idl : 0;
    bad = ok ? 0u : 0x7FC00000u;                     // a page outside the pool: its key scale is NaN
    load_ids(t0 + C::TURN);
#pragma unroll
    for (int s = 0; s < C::NS; ++s) load_codes(t0, s, id);
    const uint64_t at = (uint64_t)(uint32_t)id * (uint32_t)p.kv_heads + h;
    ksl = p.ks[at];
    vsl = p.vs[at];
  };
  auto stage = [&](int t0, uint8_t* base) {
#pragma unroll
    for (int s = 0; s < C::NS; ++s) {
#pragma unroll
      for (int i = 0; i < C::PER; ++i) {
        const int idx = tid + C::THREADS * i;
        if (C::CH % C::THREADS != 0 && idx >= C::CH) continue;
        uint8_t* st = base + s * C::STAGE;
        {
          const int tk = idx / (DP / 16), j = idx % (DP / 16);
          const int y = tk & 15;
          const int row = 8 * (y >> 2) + 4 * ((tk >> 4) & 1) + (y & 3);
          uint8_t* o = st + ((tk >> 5) * C::KS + j) * C::FRAG + row * 16;
          *reinterpret_cast<h8*>(o) = widen8<Q>(kraw[s][i][0], kraw[s][i][1]);
          *reinterpret_cast<h8*>(o + C::HALF) = widen8<Q>(kraw[s][i][2], kraw[s][i][3]);
        }
        const int vg = idx & 3, d = idx >> 2;
        u4 v = vraw[s][i];
        // codes past the length may be E4M3 NaNs: 0 * NaN would reach the sums
        if (Q == W4_Q_F8 && t0 + C::TURN > seen) {
          const int left = min(max(seen - t0 - C::STEP * s - 16 * vg, 0), 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = min(max(left - 4 * e, 0), 4);
            v[e] &= k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1u;
          }
        }
        uint8_t* o = st + (C::K_FRAGS + (d >> 5) * 4 + (vg >> 1) * 2) * C::FRAG + (d & 31) * 16 +
                     (vg & 1) * C::HALF;
        *reinterpret_cast<h8*>(o) = widen8<Q>(v[0], v[1]);
        *reinterpret_cast<h8*>(o + C::FRAG) = widen8<Q>(v[2], v[3]);
      }
    }
  };

  f16v o[C::DT];
  float m, l, ref, inv_ref;
  auto clear = [&] {
    m = -__builtin_inff(), l = 0.f, ref = REF_MIN_MANY, inv_ref = 1.0f / REF_MIN_MANY;
#pragma unroll
    for (int d = 0; d < C::DT; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  };
  clear();

  auto step = [&](int t0, const uint8_t* s, const float (&sk)[2], const float (&sv)[2]) {
    const uint8_t* fr = s + c * 16 + g * C::HALF;
    auto frag = [&](int i) { return *reinterpret_cast<const h8*>(fr + i * C::FRAG); };
    // Operand fragments come from LDS one group ahead of the products that
    // take them; the scheduling barriers keep the compiler from sinking a
    // group's reads down to their use, where each would be waited for alone.
    f16v x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[i][e] = 0.f;
    {
      h8 f[2][2];
      auto read = [&](int q) {
#pragma unroll
        for (int i = 0; i < 2; ++i) f[q & 1][i] = frag(i * C::KS + q);
      };
      read(0);
#pragma unroll
      for (int q = 0; q < C::KS; ++q) {
        if (q + 1 < C::KS) read(q + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          x[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[q & 1][i], qf[q], x[i], 0, 0, 0);
      }
    }
    const int left0 = lim - t0 - 16 * g;             // of tile 0's 16 tokens, and 32 less of tile 1's
    if (t0 + C::STEP > lim_all) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) x[i][e] = e < left0 - 32 * i ? x[i][e] : -__builtin_inff();
    }
    // The factors a are not negative (a negative softmax scale has gone into
    // q's sign), so a tile's largest product gives its largest score. A zero
    // factor becomes 2^-126, which keeps a masked -inf what it is; a NaN scale
    // stays NaN through the difference.
    float a[2], mx = -__builtin_inff(), rmax = ref;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = fmaxf(sk[i] * p.scale_log2, 0x1p-126f) + (sk[i] - sk[i]);
      // (the median with infinity is the maximum, without the quieting of
      // each operand that fmaxf asks for)
      float tm = x[i][0];
#pragma unroll
      for (int e = 1; e < 16; ++e)
        tm = __builtin_amdgcn_fmed3f(tm, x[i][e], __builtin_inff());
      mx = fmaxf(mx, tm * a[i]);
      rmax = fmaxf(rmax, left0 - 32 * i > 0 ? sv[i] : 0.f);
    }
    mx = halves_max(mx);
    if (__any(mx > m + M_SLACK || rmax > R_SLACK * ref)) {
      const float nm = fmaxf(m, mx);
      const float base = nm == -__builtin_inff() ? 0.f : nm;
      const float alpha = __builtin_amdgcn_exp2f(m - base);
      // r is one value for the wave
      float nr2 = rmax;
#pragma unroll
      for (int w = 32; w; w >>= 1) nr2 = fmaxf(nr2, __shfl_xor(nr2, w, 64));
      const float f = alpha * (ref / nr2);
      m = nm;
      ref = nr2;
      inv_ref = 1.0f / nr2;
      l *= alpha;
#pragma unroll
      for (int d = 0; d < C::DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= f;
    }
    const float base = m == -__builtin_inff() ? 0.f : m;
    h8 w[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // weight in units of r; a page that the row does not see may have any scale
      float ratio = sv[i] * inv_ref;
      ratio = ratio < RATIO_MIN ? RATIO_MIN : ratio;
      ratio = left0 - 32 * i > 0 ? ratio : 1.f;
      const float ai = left0 - 32 * i > 0 ? a[i] : 1.f;
      const float shift = __builtin_amdgcn_logf(ratio) + LOG2_P_UP_MANY - base;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i][e], ai, shift));
        sum += y;
        w[i][e >> 3][e & 7] = (_Float16)y;
      }
      l += sum * __builtin_amdgcn_rcpf(ratio);
    }
    // product z of the second: k slots z / DT, dims z % DT
    h8 vf[2][2];
    auto readv = [&](int gv) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        vf[gv & 1][j] =
            frag(C::K_FRAGS + 4 * ((2 * gv + j) % C::DT) + (2 * gv + j) / C::DT);
    };
    readv(0);
#pragma unroll
    for (int gv = 0; gv < 2 * C::DT; ++gv) {
      if (gv + 1 < 2 * C::DT) readv(gv + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int d = (2 * gv + j) % C::DT, iu = (2 * gv + j) / C::DT;
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[gv & 1][j], w[iu >> 1][iu & 1], o[d], 0, 0,
                                                      0);
      }
    }
  };

  // ---- results: lane (c, g) holds dims 32 d + 8 x + 4 g + y of row r ---------
  auto put = [&](float M, float L, float up) {       // up: o's units over L's
    int tok, hh;
    if (!row_of(tok, hh)) return;
    const size_t at = (size_t)(row0 + tok) * p.q_heads + hh;
    const float nan = __uint_as_float(0x7FC00000u);
    const float inv = !fits ? nan : L == 0.f ? 0.f : up / L;
#pragma unroll
    for (int d = 0; d < C::DT; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int dim = 32 * d + 8 * q + 4 * g;
        const h4 y = {(_Float16)(o[d][4 * q] * inv), (_Float16)(o[d][4 * q + 1] * inv),
                      (_Float16)(o[d][4 * q + 2] * inv), (_Float16)(o[d][4 * q + 3] * inv)};
        if (dim < p.dim)
          *reinterpret_cast<u2*>(p.out + at * p.dim + dim) = __builtin_bit_cast(u2, y);
      }
    if (p.lse && g == 0)
      p.lse[at] = !fits ? nan : L == 0.f ? -__builtin_inff()
                                         : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
  };
  // A part of a split sequence is the block's registers in lane order (waves
  // 0-3 tile A, 4-7 tile B), O in absolute units, then (M, L).
  const size_t unit = ((size_t)b * p.kv_heads + h) * p.tiles + pair;
  const size_t slot =
      part_slot(p.by_row, b, h, pair, row0, p.group, C::ROWS * C::PAIR, p.tiles, p.kv_heads);
  constexpr size_t PART = (size_t)C::THREADS * (C::DT * 16 + 2), NEXT = 2 * C::THREADS;
  uint32_t* po = reinterpret_cast<uint32_t*>(p.part) + slot * p.splits * PART + 2 * tid;
  // what the wave has of its rows: the output, or its part
  auto finish = [&] {
    const float L = (l + __shfl_xor(l, 32, 64)) * (1.0f / P_UP_MANY);
    const float up = ref * (1.0f / P_UP_MANY);
    if (parts == 1) {
      put(m, L, up);
      return;
    }
    uint32_t* q = po + split * PART;
#pragma unroll
    for (int d = 0; d < C::DT; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 2)
        dev_store2(q + (d * 8 + e / 2) * NEXT, __float_as_uint(o[d][e] * up),
                   __float_as_uint(o[d][e + 1] * up));
    dev_store2(q + C::DT * 8 * NEXT, __float_as_uint(m), __float_as_uint(L));
  };

  // tokens that tile B sees; past them waves 4-7 work on tile A
  const int seen_b = C::PAIR == 2 && tb >= 0 && fits
                         ? first + (min((tb + 1) * C::ROWS, rows) - 1) / p.group + 1 : 0;
  // first turn of the second phase, in which waves 4-7 help with tile A
  const int turn_b = min(c1, c0 + max(0, (seen_b - c0 + C::TURN - 1) / C::TURN * C::TURN));
  const bool helps = C::PAIR == 2 && turn_b < c1;
  {
    load_ids(c0);
    load(c0);
    stage(c0, smem);
    float ks = __uint_as_float(__float_as_uint(ksl) | bad), vs = vsl;
    __syncthreads();
    int buf = 0, t0 = c0;
    // turns up to tend, steps s0 .. s1 - 1 of each
    auto turns = [&](int tend, int s0, int s1) {
      for (; t0 < tend; t0 += C::TURN) {
        const bool more = t0 + C::TURN < c1;
        if (more) load(t0 + C::TURN);
#pragma clang loop unroll(disable)
        for (int s = s0; s < s1; ++s) {
          const int ts = t0 + C::STEP * s;
          if (ts >= lim_any || ts >= c1) break;
          float sk[2], sv[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float k0 = lane_f(ks, 4 * s + 2 * i), k1 = lane_f(ks, 4 * s + 2 * i + 1);
            const float v0 = lane_f(vs, 4 * s + 2 * i), v1 = lane_f(vs, 4 * s + 2 * i + 1);
            sk[i] = g ? k1 : k0;
            sv[i] = g ? v1 : v0;
          }
          step(ts, smem + (C::NS * buf + s) * C::STAGE, sk, sv);
        }
        if (more) {
          stage(t0 + C::TURN, smem + C::NS * (buf ^ 1) * C::STAGE);
          ks = __uint_as_float(__float_as_uint(ksl) | bad);
          vs = vsl;
        }
        __syncthreads();
        buf ^= 1;
      }
    };
    if constexpr (C::PAIR == 2) {
      turns(turn_b, 0, 2);
      if (helps && group == 1) {
        if (tb >= 0) finish();
        take_rows(ta);
        clear();
      }
    }
    turns(c1, group, group + 1);
  }
  if constexpr (C::PAIR == 2) {
    if (helps) {                                     // uniform over the block
      // waves 4-7 hand their half of tile A to waves 0-3
      float* so = reinterpret_cast<float*>(smem);
      const int row = 32 * (wave & 3) + c;
      float* sm = so + C::ROWS * C::OROW + 3 * row;
      if (group == 1) {
#pragma unroll
        for (int d = 0; d < C::DT; ++d)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f4*>(so + row * C::OROW + 32 * d + 8 * q + 4 * g) =
                f4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
        const float lt = l + __shfl_xor(l, 32, 64);
        if (g == 0) sm[0] = m, sm[1] = lt, sm[2] = ref;
      }
      __syncthreads();
      if (group == 0) {
        const float m1 = sm[0], l1 = sm[1], ref1 = sm[2];
        const float nm = fmaxf(m, m1), nref = fmaxf(ref, ref1);
        const float base = nm == -__builtin_inff() ? 0.f : nm;
        const float e0 = __builtin_amdgcn_exp2f(m - base), e1 = __builtin_amdgcn_exp2f(m1 - base);
        const float f0 = e0 * (ref / nref), f1 = e1 * (ref1 / nref);
#pragma unroll
        for (int d = 0; d < C::DT; ++d)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f4 y = *reinterpret_cast<const f4*>(so + row * C::OROW + 32 * d + 8 * q + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][4 * q + e] = o[d][4 * q + e] * f0 + y[e] * f1;
          }
        l = l * e0 + 0.5f * l1 * e1;                 // each half of the wave adds one half
        m = nm, ref = nref;
      }
    }
  }
  // tile A; tile B too if it lasted to the end
  if (group == 0 || (!helps && tb >= 0)) finish();
  if (parts == 1) return;

  // ---- chunks joined by the block that arrives last (as in attn.hip)
  stores_done();
  __syncthreads();
  if (tid == 0) *slast = dev_arrive(p.counters + unit) == (unsigned)(parts - 1);
  __syncthreads();
  if (!*slast) return;
  if (tid == 0) dev_store(p.counters + unit, 0u);
  if (group == 1) {
    if (tb < 0) return;
    take_rows(tb);
  }
  // parts that hold something of this wave's tile
  const int mine = group == 0 ? parts : max(1, (seen_b + p.chunk - 1) / p.chunk);
  float M = -__builtin_inff(), L = 0.f;
#pragma unroll
  for (int d = 0; d < C::DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  // a part's loads are issued together: each is a round trip to the level
  // that all XCDs share
  constexpr int HALVES = DP > 128 ? 2 : 1, DH = C::DT / HALVES;
  for (int z = 0; z < mine; ++z) {
    const uint64_t ml = dev_load2(po + z * PART + C::DT * 8 * NEXT);
    float fo = 0.f, fn = 0.f;
#pragma unroll
    for (int y = 0; y < HALVES; ++y) {
      uint64_t v[DH * 8];
#pragma unroll
      for (int e = 0; e < DH * 8; ++e) v[e] = dev_load2(po + z * PART + (y * DH * 8 + e) * NEXT);
      if (y == 0) {
        const float Mz = __uint_as_float((uint32_t)ml), Lz = __uint_as_float((uint32_t)(ml >> 32));
        const float nm = fmaxf(M, Mz);
        const float base = nm == -__builtin_inff() ? 0.f : nm;
        fo = __builtin_amdgcn_exp2f(M - base);
        fn = __builtin_amdgcn_exp2f(Mz - base);
        M = nm;
        L = L * fo + Lz * fn;
      }
#pragma unroll
      for (int e = 0; e < DH * 8; ++e) {
        const int d = y * DH + e / 8, q = 2 * (e & 7);
        o[d][q] = o[d][q] * fo + __uint_as_float((uint32_t)v[e]) * fn;
        o[d][q + 1] = o[d][q + 1] * fo + __uint_as_float((uint32_t)(v[e] >> 32)) * fn;
      }
    }
  }
  put(M, L, 1.0f);
}

template <int DP, int Q>
static int launch(const AttnParams& p, int64_t blocks, hipStream_t stream) {
  constexpr int lds = AttnMany<DP>::LDS;
  allow_smem((const void*)k_attn_many<DP, Q>, lds);
  hipLaunchKernelGGL((k_attn_many<DP, Q>), grid_of(blocks), dim3(AttnMany<DP>::THREADS),
                     lds, stream, p);
  return launch_status();
}

int launch_attn_many(const AttnParams& p, int dp, int kind, int64_t blocks, hipStream_t stream) {
#define W4_DP(D)                                                       \
  case D:                                                              \
    return kind == W4_Q_I8 ? launch<D, W4_Q_I8>(p, blocks, stream)     \
                           : launch<D, W4_Q_F8>(p, blocks, stream)
  switch (dp) {
    W4_DP(64);
    W4_DP(96);
    W4_DP(128);
    W4_DP(192);
    default:
      return kind == W4_Q_I8 ? launch<256, W4_Q_I8>(p, blocks, stream)
                             : launch<256, W4_Q_F8>(p, blocks, stream);
  }
#undef W4_DP
}

}  // namespace w4
