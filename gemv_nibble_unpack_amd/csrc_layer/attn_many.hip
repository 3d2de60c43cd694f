// Attention of many new tokens (prompts, chunks of prompts) over the paged
// 8-bit cache.
//
// A block takes two tiles of 128 query rows of a (sequence, kv head), 32 for
// each of its eight waves, and walks the cached tokens that its last row sees
// in steps of 64. The tiles are the k-th from the end and the k-th from the
// start of the sequence's rows: each SIMD holds a wave of either, all blocks of
// a prompt have the same number of wave steps, and a step's codes are fetched
// and widened once for both. Head dims above 128 need the registers of two
// waves for one: there a block is four waves and one tile. The step's codes are read once per block, widened to fp16 (exact) and
// laid in LDS in the order in which the matrix instructions read them; the
// next step's codes are in flight meanwhile (registers, then the other of two
// LDS stages). Per wave and step, with v_mfma_f32_32x32x16_f16:
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
// new maximum exceeds it by more than 8 in log2 units, or a larger value
// scale arrives; until then weights stay below 2^8, which P_UP_MANY = 2^7
// keeps inside fp16 with room to spare. r is the largest value scale met.

#include "attn.hpp"

namespace w4 {

typedef float f16v __attribute__((ext_vector_type(16)));

constexpr float P_UP_MANY = 128.0f, LOG2_P_UP_MANY = 7.0f;
constexpr float M_SLACK = 8.0f;
constexpr float REF_MIN_MANY = 0x1p-100f;
constexpr float RATIO_MIN = 0x1p-40f;     // smaller value scales count as this times r

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
  static constexpr int CH = 4 * DP;                  // 16-code chunks of K (and of V) a step
  static constexpr int PER = (CH + THREADS - 1) / THREADS;   // chunks per thread
  static constexpr int DEPTH = PAIR == 2 ? 2 : 1;    // steps of codes on their way
  // a fragment: 64 lanes x 16 bytes in lane order, with gaps after each half
  // and each fragment that put the eight 16-byte pieces which eight lanes
  // store at a time (eight fragments of a token, or two dims x four groups of
  // tokens) into different banks
  static constexpr int HALF = 512 + 32, FRAG = 2 * HALF + 32;
  static constexpr int K_FRAGS = 2 * KS, V_FRAGS = 4 * DT;
  static constexpr int STAGE = (K_FRAGS + V_FRAGS) * FRAG;
  static constexpr int LDS = 2 * STAGE + 16;
};

template <int DP, int Q>
__global__ __launch_bounds__(AttnMany<DP>::THREADS) void k_attn_many(const AttnParams p) {
  using C = AttnMany<DP>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  unsigned* slast = reinterpret_cast<unsigned*>(smem + 2 * C::STAGE);

  // heads fastest (a head's blocks share an XCD's L2 when kv_heads is a
  // multiple of 8), then splits and sequences, pairs of row tiles slowest
  int t = blockIdx.x;
  const int h = t % p.kv_heads;
  t /= p.kv_heads;
  const int split = t % p.splits;
  t /= p.splits;
  const int b = t % p.batch;
  const int pair = t / p.batch;

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

  // ---- this lane's query row ---------------------------------------------
  // the wave's first row (past the end for a wave without a tile)
  const int wr = wave < 4 ? ta * C::ROWS + 32 * wave
                          : tb >= 0 ? tb * C::ROWS + 32 * (wave - 4) : rows;
  const int r = wr + c;
  const int rc = r < rows ? r : rows - 1;
  const int tok = rc / p.group, hh = h * p.group + (rc - tok * p.group);
  const int lim = r < rows && fits ? first + tok + 1 : 0;
  // tokens that every / some row of the wave sees
  const int lim_all = wr + 31 < rows && fits ? first + wr / p.group + 1 : 0;
  const int lim_any = wr < rows && fits ? first + (min(wr + 31, rows - 1)) / p.group + 1 : 0;
  h8 qf[C::KS];
  {
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
  }

  // ---- one step's codes: registers, then LDS ------------------------------
  // Lane i of a wave holds group i & 3 (16 tokens) of a step: its page number
  // and its scales. Groups past the last visible token repeat the last one.
  // Codes are fetched DEPTH steps ahead, page numbers one step before them.
  u4 kraw[C::DEPTH][C::PER], vraw[C::DEPTH][C::PER];
  float ksl[C::DEPTH], vsl[C::DEPTH];
  uint32_t bad[C::DEPTH];
  int idl;
  auto at16 = [&](int t0, int gi) { return min(t0 + 16 * gi, last16); };
  auto load_ids = [&](int t0) { idl = tab[at16(t0, lane & 3) >> p.page_shift]; };
  // the step at t0 into registers x, then the page numbers of the step at t1
  auto load = [&](int t0, int t1, int x) {
    const bool ok = idl >= 0 && idl < p.pages;
    const int id = ok ? idl : 0;
    const uint32_t i0 = __builtin_amdgcn_readlane(id, 0), i1 = __builtin_amdgcn_readlane(id, 1);
    const uint32_t i2 = __builtin_amdgcn_readlane(id, 2), i3 = __builtin_amdgcn_readlane(id, 3);
    load_ids(t1);
    auto pick = [&](int gi) {
      const uint32_t lo = gi & 1 ? i1 : i0, hi = gi & 1 ? i3 : i2;
      return gi & 2 ? hi : lo;
    };
    const uint8_t* vp = vhead + (uint64_t)pick(tid & 3) * page_bytes + (at16(t0, tid & 3) & (P - 1));
#pragma unroll
    for (int i = 0; i < C::PER; ++i) {
      const int idx = tid + C::THREADS * i;
      if (C::CH % C::THREADS == 0 || idx < C::CH) {
        const int tk = idx / (DP / 16), j = idx % (DP / 16);
        kraw[x][i] = *reinterpret_cast<const u4*>(
            khead + (uint64_t)pick(tk >> 4) * page_bytes +
            ((at16(t0, tk >> 4) & (P - 1)) + (tk & 15)) * DP + 16 * j);
        vraw[x][i] = *reinterpret_cast<const u4*>(vp + ((idx >> 2) << p.page_shift));
      }
    }
    const uint64_t at = (uint64_t)(uint32_t)id * (uint32_t)p.kv_heads + h;
    ksl[x] = p.ks[at];
    vsl[x] = p.vs[at];
    bad[x] = ok ? 0u : 0x7FC00000u;                  // a page outside the pool: its key scale is NaN
  };
  auto stage = [&](int t0, uint8_t* s, int x) {
#pragma unroll
    for (int i = 0; i < C::PER; ++i) {
      const int idx = tid + C::THREADS * i;
      if (C::CH % C::THREADS == 0 || idx < C::CH) {
        {
          const int tk = idx / (DP / 16), j = idx % (DP / 16);
          const int y = tk & 15;
          const int row = 8 * (y >> 2) + 4 * ((tk >> 4) & 1) + (y & 3);
          uint8_t* o = s + ((tk >> 5) * C::KS + j) * C::FRAG + row * 16;
          *reinterpret_cast<h8*>(o) = widen8<Q>(kraw[x][i][0], kraw[x][i][1]);
          *reinterpret_cast<h8*>(o + C::HALF) = widen8<Q>(kraw[x][i][2], kraw[x][i][3]);
        }
        const int vg = idx & 3, d = idx >> 2;
        u4 v = vraw[x][i];
        // codes past the length may be E4M3 NaNs: 0 * NaN would reach the sums
        if (Q == W4_Q_F8 && t0 + C::STEP > seen) {
          const int left = min(max(seen - t0 - 16 * vg, 0), 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = min(max(left - 4 * e, 0), 4);
            v[e] &= k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1u;
          }
        }
        uint8_t* o = s + (C::K_FRAGS + (d >> 5) * 4 + (vg >> 1) * 2) * C::FRAG + (d & 31) * 16 +
                     (vg & 1) * C::HALF;
        *reinterpret_cast<h8*>(o) = widen8<Q>(v[0], v[1]);
        *reinterpret_cast<h8*>(o + C::FRAG) = widen8<Q>(v[2], v[3]);
      }
    }
  };

  f16v o[C::DT];
  float m = -__builtin_inff(), l = 0.f, ref = REF_MIN_MANY, inv_ref = 1.0f / REF_MIN_MANY;
#pragma unroll
  for (int d = 0; d < C::DT; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;

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
      h8 f[2][4];
      auto read = [&](int gq) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i) f[gq & 1][2 * q + i] = frag(i * C::KS + 2 * gq + q);
      };
      read(0);
#pragma unroll
      for (int gq = 0; gq < C::KS / 2; ++gq) {
        if (gq + 1 < C::KS / 2) read(gq + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            x[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[gq & 1][2 * q + i], qf[2 * gq + q], x[i],
                                                          0, 0, 0);
      }
    }
    h8 vf[2][C::DT];
    auto readv = [&](int iu) {
#pragma unroll
      for (int d = 0; d < C::DT; ++d) vf[iu & 1][d] = frag(C::K_FRAGS + 4 * d + iu);
    };
    readv(0);
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
    if (__any(mx > m + M_SLACK || rmax > ref)) {
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
#pragma unroll
    for (int iu = 0; iu < 4; ++iu) {
      if (iu < 3) readv(iu + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < C::DT; ++d)
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[iu & 1][d], w[iu >> 1][iu & 1], o[d], 0, 0,
                                                      0);
    }
  };

  if (c0 < c1) {
    // One turn: step t0 is in LDS stage `cur`, the next ones are in registers
    // or on their way there (steps past the chunk repeat its last tokens).
    float sk[2], sv[2];
    auto scales = [&](int x) {
      const float ks = __uint_as_float(__float_as_uint(ksl[x]) | bad[x]), vs = vsl[x];
      const float k0 = lane_f(ks, 0), k1 = lane_f(ks, 1), k2 = lane_f(ks, 2), k3 = lane_f(ks, 3);
      const float v0 = lane_f(vs, 0), v1 = lane_f(vs, 1), v2 = lane_f(vs, 2), v3 = lane_f(vs, 3);
      sk[0] = g ? k1 : k0, sk[1] = g ? k3 : k2;
      sv[0] = g ? v1 : v0, sv[1] = g ? v3 : v2;
    };
    auto turn = [&](int t0, int cur) {
      constexpr int D = C::DEPTH;
      load(t0 + D * C::STEP, t0 + (D + 1) * C::STEP, D == 2 ? cur : 0);
      if (t0 < lim_any) step(t0, smem + cur * C::STAGE, sk, sv);
      if (t0 + C::STEP < c1) {
        stage(t0 + C::STEP, smem + (cur ^ 1) * C::STAGE, D == 2 ? cur ^ 1 : 0);
        scales(D == 2 ? cur ^ 1 : 0);
      }
      __syncthreads();
    };
    load_ids(c0);
    load(c0, c0 + C::STEP, 0);
    if constexpr (C::DEPTH == 2) load(c0 + C::STEP, c0 + 2 * C::STEP, 1);
    stage(c0, smem, 0);
    scales(0);
    __syncthreads();
    for (int t0 = c0; t0 < c1; t0 += 2 * C::STEP) {
      turn(t0, 0);
      if (t0 + C::STEP < c1) turn(t0 + C::STEP, 1);
    }
  }
  l = (l + __shfl_xor(l, 32, 64)) * (1.0f / P_UP_MANY);

  // ---- results: lane (c, g) holds dims 32 d + 8 x + 4 g + y of row r ---------
  auto put = [&](float M, float L, float up) {       // up: o's units over L's
    if (r >= rows) return;
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
  if (parts == 1) {
    put(m, l, ref * (1.0f / P_UP_MANY));
    return;
  }

  // ---- chunks joined by the block that arrives last (as in attn.hip); a part
  // is the block's registers in lane order, O in absolute units, then (M, L)
  const size_t unit = ((size_t)b * p.kv_heads + h) * p.tiles + pair;
  constexpr size_t PART = (size_t)C::THREADS * (C::DT * 16 + 2), NEXT = 2 * C::THREADS;
  uint32_t* po = reinterpret_cast<uint32_t*>(p.part) + unit * p.splits * PART + 2 * tid;
  {
    uint32_t* q = po + split * PART;
    const float up = ref * (1.0f / P_UP_MANY);
#pragma unroll
    for (int d = 0; d < C::DT; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 2)
        dev_store2(q + (d * 8 + e / 2) * NEXT, __float_as_uint(o[d][e] * up),
                   __float_as_uint(o[d][e + 1] * up));
    dev_store2(q + C::DT * 8 * NEXT, __float_as_uint(m), __float_as_uint(l));
  }
  stores_done();
  __syncthreads();
  if (tid == 0) *slast = dev_arrive(p.counters + unit) == (unsigned)(parts - 1);
  __syncthreads();
  if (!*slast) return;
  if (tid == 0) dev_store(p.counters + unit, 0u);
  float M = -__builtin_inff(), L = 0.f;
  for (int z = 0; z < parts; ++z) {
    const uint64_t ml = dev_load2(po + z * PART + C::DT * 8 * NEXT);
    const float Mz = __uint_as_float((uint32_t)ml), Lz = __uint_as_float((uint32_t)(ml >> 32));
    const float nm = fmaxf(M, Mz);
    const float base = nm == -__builtin_inff() ? 0.f : nm;
    const float fo = z ? __builtin_amdgcn_exp2f(M - base) : 0.f;
    const float fn = __builtin_amdgcn_exp2f(Mz - base);
    M = nm;
    L = L * fo + Lz * fn;
#pragma unroll
    for (int d = 0; d < C::DT; ++d) {
      uint64_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = dev_load2(po + z * PART + (d * 8 + e) * NEXT);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = __uint_as_float((uint32_t)v[e]), y = __uint_as_float((uint32_t)(v[e] >> 32));
        o[d][2 * e] = z ? o[d][2 * e] * fo + x * fn : x * fn;
        o[d][2 * e + 1] = z ? o[d][2 * e + 1] * fo + y * fn : y * fn;
      }
    }
  }
  put(M, L, 1.0f);
}

template <int DP, int Q>
static int launch(const AttnParams& p, int64_t blocks, hipStream_t stream) {
  constexpr int lds = AttnMany<DP>::LDS;
  allow_smem((const void*)k_attn_many<DP, Q>, lds);
  hipLaunchKernelGGL((k_attn_many<DP, Q>), dim3((unsigned)blocks), dim3(AttnMany<DP>::THREADS),
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
