// Attention of one or a few new tokens over the paged 8-bit cache.
//
// The query rows of a (sequence, kv head) are its new tokens times the query
// heads that share the kv head, token-major; a block takes 16 * QT of them and
// one chunk of the cached tokens. Each of its four waves takes every fourth
// step of 64 tokens, with a running maximum, sum and output of its own:
//
//   S^T = K q^T    v_mfma_f32_16x16x32_f16, rows = tokens, columns = query rows
//   w   = 2^(S a - m)           float32; a = k_scale * sm_scale * log2 e
//   O^T += V^T w^T              the same instruction, rows = dims
//
// Token order inside a step is chosen so that nothing moves between lanes: the
// wave's four 16-lane rows g own the tokens 16g .. 16g+15. Row i of the K
// operand of tile t is token 16 (i >> 2) + 4 t + (i & 3); the product leaves
// lane (column c, row g) with tokens 16 g + 4 t + 0..3, which over two tiles are
// the 8 consecutive tokens that the second product's k slots of that lane
// take, and the V operand reads them as 8 consecutive bytes of the transposed
// value page. 16 tokens lie in one page, so a lane needs one key scale and one
// value scale per step. The codes are widened to fp16 in registers (exact).
//
// Value scales: with r the largest value scale met so far, w is multiplied by
// v_scale / r <= 1 before its rounding to fp16 and O is kept in units of r
// (rescaled together with the running maximum), so weights keep fp16's
// relative precision at any magnitude of the values. The factor 2^10 on w
// moves small weights out of fp16's subnormals.
//
// Chunks: a sequence's chunks are joined by the block that arrives last
// (agent-scope stores and loads, one arrival counter per row tile, left zero).
//
// Bound: the bytes of the codes (2 per cached token, head and dim). One token
// over 131072 cached ones of 8 heads of 128 takes 56 us (4.8 TB/s; a plain read
// of as many bytes 42), 32 sequences of 1 to 4096 tokens 34 us (4.0 TB/s, the
// blocks of the longest last), one token over 517 cached 7.8 us (a chain of
// dependent reads: length, page number, codes, parts). Widening in registers
// costs about 51 codes a clock and CU, 4 times what memory delivers, so nothing
// is staged through LDS. Keeping two steps' codes in registers at once measured
// slower (68 us on the long one, for the registers it takes) than fetching
// into the registers that the last step freed.
#include "attn.hpp"

namespace w4 {

constexpr float P_UP = 1024.0f;
constexpr float REF_MIN = 0x1p-100f;

template <int DP, int Q, int QT>
struct AttnFew {
  static constexpr int ROWS = 16 * QT;
  static constexpr int KH = DP / 64;                // 64-dim halves of a K row
  static constexpr bool KR = DP % 64 != 0;          // and a rest of 32 dims
  static constexpr int KS = DP / 32;                // k steps of the first product
  static constexpr int DT = DP / 16;                // 16-dim tiles of the second
  static constexpr int OROW = DP + 4;               // staged floats per row
  static constexpr int LDS = 4 * ROWS * OROW * 4 + 4 * ROWS * 2 * 4 + 16 + 16;
};

template <int DP>
struct KVRegs {
  u4 k[4][DP / 64 ? DP / 64 : 1];
  u2 kr[4];
  u4 v[DP / 16];
  float ks, vs;
  uint32_t bad;
};

// two blocks a CU where their registers allow it (<256, INT8, 2> spills 3)
template <int DP, int Q, int QT>
__global__ __launch_bounds__(256, DP < 256 && DP * QT <= 256 ? 2 : 1) void k_attn_few(const AttnParams p) {
  using C = AttnFew<DP, Q, QT>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  float* so = reinterpret_cast<float*>(smem);                       // [4][ROWS][OROW]
  float* sml = so + 4 * C::ROWS * C::OROW;                          // [4][ROWS][2]
  float* sref = sml + 4 * C::ROWS * 2;                              // [4]
  unsigned* slast = reinterpret_cast<unsigned*>(sref + 4);

  int t = block_number();          // past the grid's end: split >= parts below
  const int h = t % p.kv_heads;
  t /= p.kv_heads;
  const int tile = t % p.tiles;
  t /= p.tiles;
  const int b = t % p.batch;
  const int split = t / p.batch;
  int row0, n, len;
  bool fits;
  if (!attn_span(p, b, row0, n, len, fits)) return;
  const int rows = min(n, p.max_q) * p.group;
  const int r0 = tile * C::ROWS;
  if (r0 >= rows) return;
  const int nr = min(rows - r0, C::ROWS);           // rows of this tile
  const int first = len - n;                        // position of new token 0
  // cached tokens that the tile's last row sees
  const int seen = fits ? max(0, first + (r0 + nr - 1) / p.group + 1) : 0;
  const int parts = max(1, (seen + p.chunk - 1) / p.chunk);
  if (split >= parts) return;

  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int P = 1 << p.page_shift;

  // ---- this lane's query rows (columns c of QT operands) -------------------
  h8 qf[QT][C::KS];
  int lim[QT];                                      // tokens that the row sees
#pragma unroll
  for (int u = 0; u < QT; ++u) {
    const int r = r0 + 16 * u + c;
    const bool in = r < rows;
    const int rc = in ? r : r0;
    const int tok = rc / p.group, hh = h * p.group + (rc - tok * p.group);
    lim[u] = in && fits ? first + tok + 1 : 0;
    const uint16_t* q = p.q + (int64_t)(row0 + tok) * p.q_stride + (int64_t)hh * p.dim;
    auto quad = [&](int d) {                         // dims past the head are zero
      const u2 x = d < p.dim ? *reinterpret_cast<const u2*>(q + d) : u2{0u, 0u};
      return u2{x[0] ^ p.q_sign, x[1] ^ p.q_sign};
    };
    auto oct = [&](int d) {
      const u2 a = quad(d), b2 = quad(d + 4);
      return __builtin_bit_cast(h8, u4{a[0], a[1], b2[0], b2[1]});
    };
#pragma unroll
    for (int s = 0; s < C::KH; ++s) {
      qf[u][2 * s] = oct(64 * s + 16 * g);
      qf[u][2 * s + 1] = oct(64 * s + 16 * g + 8);
    }
    if constexpr (C::KR) qf[u][C::KS - 1] = oct(64 * C::KH + 8 * g);
  }

  const int32_t* tab = p.table + (size_t)b * p.cols;
  const int c0 = split * p.chunk;
  const int c1 = min(seen, c0 + p.chunk);
  const int last16 = (max(seen, 1) - 1) & ~15;      // start of the last group with a token
  const uint32_t page_bytes = (uint32_t)p.kv_heads * DP << p.page_shift;
  const uint8_t* khead = p.kc + ((int64_t)h * DP << p.page_shift);
  const uint8_t* vhead = p.vc + ((int64_t)h * DP << p.page_shift);

  // A step's codes into registers: K operand row c takes tokens of group c >> 2,
  // this lane's own tokens are group g. The next step's keys are fetched as
  // soon as the first product has taken this one's, the values after the
  // second, so the same registers serve; page numbers are fetched one step
  // before. All loads go out before the work that follows in the program.
  KVRegs<DP> r;
  int ikn, ivn;                                     // page numbers of the next loads
  auto load_ids = [&](int t0) {
    ikn = tab[min(t0 + 16 * (c >> 2), last16) >> p.page_shift];
    ivn = tab[min(t0 + 16 * g, last16) >> p.page_shift];
  };
  auto load_k = [&](int t0) {
    const int tk = min(t0 + 16 * (c >> 2), last16);
    const uint32_t ik = ikn >= 0 && ikn < p.pages ? ikn : 0;
    const uint8_t* kp = khead + (uint64_t)ik * page_bytes + ((tk & (P - 1)) + (c & 3)) * DP + 16 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int s = 0; s < C::KH; ++s)
        r.k[i][s] = *reinterpret_cast<const u4*>(kp + 4 * i * DP + 64 * s);
      if constexpr (C::KR)
        r.kr[i] = *reinterpret_cast<const u2*>(kp + 4 * i * DP + 64 * C::KH - 8 * g);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load_v = [&](int t0) {
    const int tv = min(t0 + 16 * g, last16);
    const bool ok = ivn >= 0 && ivn < p.pages;
    const uint32_t iv = ok ? ivn : 0;
    load_ids(t0 + 256);
    r.bad = ok ? 0u : 0x7FC00000u;                   // a page outside the pool: its key scale is NaN
    const uint64_t at = (uint64_t)iv * (uint32_t)p.kv_heads + h;
    r.ks = p.ks[at];
    r.vs = p.vs[at];
    const uint8_t* vp = vhead + (uint64_t)iv * page_bytes + (c << p.page_shift) + (tv & (P - 1));
#pragma unroll
    for (int d = 0; d < C::DT; ++d)
      r.v[d] = *reinterpret_cast<const u4*>(vp + ((16 * d) << p.page_shift));
    __builtin_amdgcn_sched_barrier(0);
  };

  f4 o[QT][C::DT];
  float m[QT], l[QT];
  float ref = REF_MIN;
#pragma unroll
  for (int u = 0; u < QT; ++u) {
    m[u] = -__builtin_inff();
    l[u] = 0.f;
#pragma unroll
    for (int d = 0; d < C::DT; ++d) o[u][d] = f4{0.f, 0.f, 0.f, 0.f};
  }

  auto step = [&](int t0, bool more) {
    f4 s[QT][4];
#pragma unroll
    for (int u = 0; u < QT; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u][i] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int x = 0; x < C::KH; ++x) {
        const h8 a0 = widen8<Q>(r.k[i][x][0], r.k[i][x][1]);
        const h8 a1 = widen8<Q>(r.k[i][x][2], r.k[i][x][3]);
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          s[u][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, qf[u][2 * x], s[u][i], 0, 0, 0);
          s[u][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, qf[u][2 * x + 1], s[u][i], 0, 0, 0);
        }
      }
      if constexpr (C::KR) {
        const h8 a = widen8<Q>(r.kr[i][0], r.kr[i][1]);
#pragma unroll
        for (int u = 0; u < QT; ++u)
          s[u][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qf[u][C::KS - 1], s[u][i], 0, 0, 0);
      }
    }
    if (more) load_k(t0 + 256);
    const int tg = t0 + 16 * g;                     // this lane's 16 tokens
    const float a = __uint_as_float(__float_as_uint(r.ks) | r.bad) * p.scale_log2;
    // a lane without a token in reach may hold any scale: it counts as none
    const float vs = tg < c1 ? r.vs : 0.f;
    const float nref = fmaxf(ref, rows_max(vs));
    const float shrink = ref / nref;
    const float pv = vs / nref * P_UP;
    ref = nref;
    h8 w[QT][2];
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      const int left = min(lim[u], c1) - tg;        // of the 16, the first `left` count
      // a page that the row does not see may have any scale, NaN among them
      const float pvu = left > 0 ? pv : 0.f;
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = s[u][i][e] * a;
          s[u][i][e] = 4 * i + e < left ? x : -__builtin_inff();
          mx = fmaxf(mx, s[u][i][e]);
        }
      const float nm = fmaxf(m[u], rows_max(mx));
      const float base = nm == -__builtin_inff() ? 0.f : nm;
      const float alpha = __builtin_amdgcn_exp2f(m[u] - base);
      m[u] = nm;
      float sum = 0.f;
      h8 hw[2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f(s[u][i][e] - base);
          sum += x;
          hw[i >> 1][4 * (i & 1) + e] = (_Float16)(x * pvu);
        }
      l[u] = l[u] * alpha + sum;
      w[u][0] = hw[0];
      w[u][1] = hw[1];
      const float f = alpha * shrink;
#pragma unroll
      for (int d = 0; d < C::DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[u][d][e] *= f;
    }
    // codes past the length may be E4M3 NaNs: 0 * NaN would reach the sums
    if (Q == W4_Q_F8 && t0 + 64 > c1) {
      const int left = min(max(c1 - tg, 0), 16);
#pragma unroll
      for (int d = 0; d < C::DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = min(max(left - 4 * e, 0), 4);
          r.v[d][e] &= k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1u;
        }
    }
#pragma unroll
    for (int d = 0; d < C::DT; ++d) {
      const h8 v0 = widen8<Q>(r.v[d][0], r.v[d][1]);
      const h8 v1 = widen8<Q>(r.v[d][2], r.v[d][3]);
#pragma unroll
      for (int u = 0; u < QT; ++u) {
        o[u][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w[u][0], o[u][d], 0, 0, 0);
        o[u][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w[u][1], o[u][d], 0, 0, 0);
      }
    }
    if (more) load_v(t0 + 256);
  };

  if (c0 + 64 * wave < c1) {
    int t0 = c0 + 64 * wave;
    load_ids(t0);
    load_k(t0);
    load_v(t0);
    for (; t0 < c1; t0 += 256) step(t0, t0 + 256 < c1);
  }

  // ---- the four waves' results to LDS ---------------------------------------
#pragma unroll
  for (int u = 0; u < QT; ++u) {
    const float lt = rows_sum(l[u]);
    const int r = 16 * u + c;
    if (g == 0) {
      sml[(wave * C::ROWS + r) * 2] = m[u];
      sml[(wave * C::ROWS + r) * 2 + 1] = lt;
    }
#pragma unroll
    for (int d = 0; d < C::DT; ++d)
      *reinterpret_cast<f4*>(so + (wave * C::ROWS + r) * C::OROW + 16 * d + 4 * g) = o[u][d];
  }
  if (lane == 0) sref[wave] = ref;
  __syncthreads();

  // Row r's result over the four waves: M, L and, for 4 dims, O in absolute
  // units (sum of 2^(s - M) v)
  auto waves_ml = [&](int r, float (&f)[4], float& M, float& L) {
    M = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < 4; ++i) M = fmaxf(M, sml[(i * C::ROWS + r) * 2]);
    const float base = M == -__builtin_inff() ? 0.f : M;
    L = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = __builtin_amdgcn_exp2f(sml[(i * C::ROWS + r) * 2] - base);
      L += e * sml[(i * C::ROWS + r) * 2 + 1];
      f[i] = e * sref[i] * (1.0f / P_UP);
    }
  };
  auto waves_o = [&](int r, int d, const float (&f)[4]) {
    f4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f4 x = *reinterpret_cast<const f4*>(so + (i * C::ROWS + r) * C::OROW + d);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += f[i] * x[e];
    }
    return s;
  };
  auto finish = [&](int r, int d, float M, float L, f4 s) {
    const int rr = r0 + r, tok = rr / p.group, hh = h * p.group + (rr - tok * p.group);
    const size_t at = (size_t)(row0 + tok) * p.q_heads + hh;
    const float nan = __uint_as_float(0x7FC00000u);
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    h4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (_Float16)(fits ? s[e] * inv : nan);
    if (d < p.dim) *reinterpret_cast<u2*>(p.out + at * p.dim + d) = __builtin_bit_cast(u2, y);
    if (p.lse && d == 0) {
      const float v = M + __builtin_amdgcn_logf(L);          // log2 units
      p.lse[at] = !fits ? nan : L == 0.f ? -__builtin_inff() : v * 0.69314718055994531f;
    }
  };
  constexpr int NV = DP / 4;
  if (parts == 1) {
    for (int i = tid; i < nr * NV; i += 256) {
      const int r = i / NV, d = 4 * (i % NV);
      float f[4], M, L;
      waves_ml(r, f, M, L);
      finish(r, d, M, L, waves_o(r, d, f));
    }
    return;
  }

  // ---- split over chunks: store the part, the last block joins --------------
  const size_t unit = ((size_t)b * p.kv_heads + h) * p.tiles + tile;
  uint32_t* po = reinterpret_cast<uint32_t*>(p.part) +
                 unit * p.splits * (size_t)(C::ROWS * (DP + 2));
  const size_t pstride = (size_t)C::ROWS * (DP + 2);          // one part: O rows, then (M, L)
  for (int i = tid; i < nr * NV; i += 256) {
    const int r = i / NV, d = 4 * (i % NV);
    float f[4], M, L;
    waves_ml(r, f, M, L);
    const f4 s = waves_o(r, d, f);
    uint32_t* q = po + split * pstride;
    dev_store2(q + r * DP + d, __float_as_uint(s[0]), __float_as_uint(s[1]));
    dev_store2(q + r * DP + d + 2, __float_as_uint(s[2]), __float_as_uint(s[3]));
    if (d == 0) dev_store2(q + C::ROWS * DP + 2 * r, __float_as_uint(M), __float_as_uint(L));
  }
  stores_done();
  __syncthreads();
  if (tid == 0) *slast = dev_arrive(p.counters + unit) == (unsigned)(parts - 1);
  __syncthreads();
  if (!*slast) return;
  if (tid == 0) dev_store(p.counters + unit, 0u);
  // Items are (row, 4 dims); where they leave threads idle, 2, 4 or 8 threads
  // share an item's parts. Eight parts' loads are issued together: each is a
  // round trip to the level that all XCDs share, and one after another they
  // took longer than the block's own share of the tokens.
  const int items = nr * NV;
  const int share = items <= 32 ? 8 : items <= 64 ? 4 : items <= 128 ? 2 : 1;
  float* sj = so;                                   // [share][items][6]
  for (int i0 = 0; i0 < items; i0 += 256 / share) {
    const int lane_item = tid & (256 / share - 1), pg = tid / (256 / share);
    const int i = min(i0 + lane_item, items - 1);
    const int rr = i / NV, d = 4 * (i % NV);
    float M = -__builtin_inff(), L = 0.f;
    f4 s = {0.f, 0.f, 0.f, 0.f};
    for (int z = pg; z < parts; z += 8 * share) {
      uint64_t ml[8], x[8], y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t* q = po + min(z + k * share, parts - 1) * pstride;
        ml[k] = dev_load2(q + C::ROWS * DP + 2 * rr);
        x[k] = dev_load2(q + rr * DP + d);
        y[k] = dev_load2(q + rr * DP + d + 2);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (z + k * share >= parts) break;
        const float Mk = __uint_as_float((uint32_t)ml[k]), Lk = __uint_as_float(ml[k] >> 32);
        const float nm = fmaxf(M, Mk);
        const float base = nm == -__builtin_inff() ? 0.f : nm;
        const float fo = __builtin_amdgcn_exp2f(M - base), fn = __builtin_amdgcn_exp2f(Mk - base);
        M = nm;
        L = L * fo + Lk * fn;
        s[0] = s[0] * fo + __uint_as_float((uint32_t)x[k]) * fn;
        s[1] = s[1] * fo + __uint_as_float((uint32_t)(x[k] >> 32)) * fn;
        s[2] = s[2] * fo + __uint_as_float((uint32_t)y[k]) * fn;
        s[3] = s[3] * fo + __uint_as_float((uint32_t)(y[k] >> 32)) * fn;
      }
    }
    if (share > 1) {                                // uniform; one pass over the items then
      float* q = sj + (pg * items + i) * 6;
      if (lane_item < items) {
        q[0] = M, q[1] = L;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[2 + e] = s[e];
      }
      __syncthreads();
      if (pg != 0 || lane_item >= items) return;
      for (int g2 = 1; g2 < share; ++g2) {
        const float* w = sj + (g2 * items + i) * 6;
        const float nm = fmaxf(M, w[0]);
        const float base = nm == -__builtin_inff() ? 0.f : nm;
        const float fo = __builtin_amdgcn_exp2f(M - base), fn = __builtin_amdgcn_exp2f(w[0] - base);
        M = nm;
        L = L * fo + w[1] * fn;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = s[e] * fo + w[2 + e] * fn;
      }
    }
    if (i0 + lane_item < items) finish(rr, d, M, L, s);
  }
}

// The launch for these sizes: rows per tile, tiles, chunk and splits, and the
// workspace they need.
struct AttnPlan {
  bool many;                       // k_attn_many
  bool by_row;                     // parts numbered by row (part_slot)
  int qt, tile, tiles, chunk, splits;
  int64_t units;
  size_t ws;
};

inline AttnPlan attn_plan(int batch, int tokens, int max_q, int max_kv, int group, int kv_heads,
                          int dp) {
  AttnPlan a{};
  max_kv = max(max_kv, 1);         // nothing cached: one block writes the empty rows
  const int64_t rows = (int64_t)max_q * group;
  // Rows by sequence and kv head. Up to 16 fill one operand of k_attn_few, up to
  // 64 are two or four tiles of its 32-row form. 4 sequences of 3000 to 4000
  // cached tokens, 8 kv heads of 128: 20 rows 21 us against k_attn_many's 31,
  // 64 rows 24 against 31, 96 rows 27 against 33; 32 sequences of 500 to 1000: 64
  // rows 23.5 against 26.8, 96 rows 31.6 against 28.5.
  a.many = rows > 64;
  a.qt = rows > 16 ? 2 : 1;
  const int tile = a.tile = a.many ? MANY_ROWS * (many_pair(dp) ? 2 : 1) : 16 * a.qt;
  a.tiles = (int)((rows + tile - 1) / tile);
  a.units = (int64_t)batch * kv_heads * a.tiles;
  constexpr int least = 256;
  int64_t splits = 1, slots = a.units;
  if (a.units <= WS_COUNTER_SLOTS) {
    if (a.many) {
      // blocks with work, at most: a ragged batch has fewer than its longest
      // sequence's tiles times its size. Parts are numbered by the smaller count.
      const int64_t by_row = ((int64_t)tokens * group / tile + batch) * kv_heads;
      a.by_row = by_row < a.units;
      slots = min(a.units, by_row);
      const int64_t room = (W4_ATTN_WORKSPACE_MAX - WS_COUNTERS) / ((int64_t)tile * (dp + 4) * 4);
      // One block a CU at a time. The number of chunks with the shortest run
      // of whole rounds over the 256 CUs, a part's store and load costing as
      // much as 45 tokens: 256 tokens of 32 heads over 16384 cached ones take
      // 463 us unsplit, 99 us in 9 chunks; 2048 tokens over themselves (256
      // blocks already) 55 us unsplit, 56 in 2. 119 tokens of 16 heads over 9424:
      // dims of 128, 192, 256 44.9, 62.3, 78.8 us; at 65 tokens (fewer parts)
      // 44.0, 63.4, 80.5, at 130 with dims above 128 74 and 92.
      const int64_t most = min((int64_t)((max_kv + 511) / 512), room / slots);
      double best = 1e30;
      for (int64_t s = 1; s <= max(most, (int64_t)1) && s <= 256; ++s) {
        const double cost = (double)((slots * s + 255) / 256) / s + (s > 1 ? 45.0 * s / max_kv : 0.0);
        if (cost < best) best = cost, splits = s;
      }
    } else {
      // About one round of the 512 resident blocks: one token of 8 kv heads
      // over 131072 cached ones takes 56 us in 64 chunks, 60 in 96, 63 in
      // 128. A batch's lengths are mostly below their bound and leave blocks
      // without work: 32 sequences of 1 to 4096 tokens take 34 us in 3 chunks,
      // 38 in 2 (the one batch that the 640 rests on). Chunks of 256 tokens (one
      // step a wave) or more.
      const int64_t target = batch > 1 ? 640 : 512;
      splits = max((int64_t)1, min((int64_t)(max_kv + least - 1) / least,
                                   (target + a.units / 2) / a.units));
    }
  }
  // whole steps of a block's four waves, whole turns of k_attn_many (in steps of
  // 256 the case above takes 84 us where it takes 80)
  const int unit = a.many ? 128 : least;
  a.chunk = (int)(((max_kv + splits - 1) / splits + unit - 1) / unit * unit);
  a.splits = max(1, (max_kv + a.chunk - 1) / a.chunk);
  a.ws = a.splits == 1 ? 0 : WS_COUNTERS + (size_t)(slots * part_bytes(a.many, tile, dp, a.splits));
  return a;
}

template <int DP, int Q>
int launch_attn(const AttnParams& p, const AttnPlan& a, hipStream_t stream) {
  const int64_t blocks = a.units * a.splits;
  if (blocks > MAX_BLOCKS) return W4_ERR_SHAPE;
#define W4_AT(QT)                                                                       \
  do {                                                                                  \
    constexpr int lds = AttnFew<DP, Q, QT>::LDS;                                        \
    allow_smem((const void*)k_attn_few<DP, Q, QT>, lds);                                \
    hipLaunchKernelGGL((k_attn_few<DP, Q, QT>), grid_of(blocks), dim3(256), lds,        \
                       stream, p);                                                      \
  } while (0)
  if (a.qt == 1) W4_AT(1);
  else W4_AT(2);
#undef W4_AT
  return launch_status();
}

}  // namespace w4

using namespace w4;

static bool attn_sizes_ok(int batch, int tokens, int max_q, int max_kv, int q_heads, int kv_heads,
                          int head_dim) {
  return batch >= 0 && tokens >= 0 && max_q >= 0 && max_kv >= 0 && max_kv <= (1 << 30) &&
         kv_heads >= 1 && kv_heads < 65536 && q_heads >= 1 && q_heads % kv_heads == 0 &&
         kv8_padded_dim(head_dim) != 0 &&
         (int64_t)min(max_q, tokens) * (q_heads / kv_heads) <= 0x7fffffff / 2;
}

extern "C" size_t paged_attn_kv8_workspace_bytes(int batch, int tokens, int max_q, int max_kv,
                                                 int q_heads, int kv_heads, int head_dim) {
  if (!attn_sizes_ok(batch, tokens, max_q, max_kv, q_heads, kv_heads, head_dim)) return 0;
  if (batch == 0 || tokens == 0 || max_q == 0) return 0;
  return attn_plan(batch, tokens, min(max_q, tokens), max_kv, q_heads / kv_heads, kv_heads,
                   kv8_padded_dim(head_dim)).ws;
}

// For the tests, not in the header: the slots of a call's parts (-1 without
// a block) in slots[batch * kv_heads * tiles], q_indptr being host memory, and
// the bytes of a slot; returns their count, 0 if the call is not split.
extern "C" int64_t w4_attn_part_slots(int batch, int tokens, int max_q, int max_kv, int q_heads,
                                      int kv_heads, int head_dim, const int32_t* q_indptr,
                                      int64_t* slots, int64_t capacity, int64_t* bytes) {
  if (paged_attn_kv8_workspace_bytes(batch, tokens, max_q, max_kv, q_heads, kv_heads, head_dim) == 0)
    return 0;
  const int group = q_heads / kv_heads, dp = kv8_padded_dim(head_dim);
  max_q = min(max_q, tokens);
  const AttnPlan a = attn_plan(batch, tokens, max_q, max_kv, group, kv_heads, dp);
  *bytes = part_bytes(a.many, a.tile, dp, a.splits);
  if (a.units > capacity) return a.units;
  for (int b = 0; b < batch; ++b) {
    const int row0 = q_indptr ? q_indptr[b] : b, end = q_indptr ? q_indptr[b + 1] : b + 1;
    const bool live = row0 >= 0 && end > row0 && end <= tokens;
    const int64_t rows = live ? (int64_t)min(end - row0, max_q) * group : 0;
    for (int h = 0; h < kv_heads; ++h)
      for (int t = 0; t < a.tiles; ++t)
        slots[((int64_t)b * kv_heads + h) * a.tiles + t] =
            (int64_t)t * a.tile < rows
                ? part_slot(a.by_row, b, h, t, row0, group, a.tile, a.tiles, kv_heads)
                : -1;
  }
  return a.units;
}

extern "C" int paged_attn_kv8(const uint16_t* q, int64_t q_stride, const void* k_codes,
                              const void* v_codes, const float* k_scale, const float* v_scale,
                              const int32_t* q_indptr, const int32_t* kv_len,
                              const int32_t* page_table, int batch, int tokens, int max_q,
                              int max_kv, int table_cols, int q_heads, int kv_heads, int head_dim,
                              int page_size, int num_pages, int q_dtype, float sm_scale,
                              uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  if (q_dtype != W4_Q_I8 && q_dtype != W4_Q_F8) return W4_ERR_ARG;
  if (!(sm_scale > -3.0e38f && sm_scale < 3.0e38f)) return W4_ERR_ARG;
  if (!attn_sizes_ok(batch, tokens, max_q, max_kv, q_heads, kv_heads, head_dim) ||
      table_cols < 1 || !kv8_page_ok(page_size) || num_pages < 1 ||
      q_stride < (int64_t)q_heads * head_dim || q_stride % 4 || (!q_indptr && tokens != batch))
    return W4_ERR_SHAPE;
  if (batch == 0 || tokens == 0 || max_q == 0) return W4_OK;
  if (!q || !k_codes || !v_codes || !k_scale || !v_scale || !kv_len || !page_table || !out)
    return W4_ERR_NULL;
  if (!aligned(q, 8) || !aligned(out, 8) || !aligned(k_codes, 16) || !aligned(v_codes, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(kv_len, 4) ||
      !aligned(page_table, 4) || !aligned(q_indptr, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 256))
    return W4_ERR_ALIGN;
  AttnParams p{};
  p.max_q = min(max_q, tokens);
  const int dp = kv8_padded_dim(head_dim);
  const AttnPlan a = attn_plan(batch, tokens, p.max_q, max_kv, q_heads / kv_heads, kv_heads, dp);
  if (a.ws > 0 && (!workspace || workspace_bytes < a.ws)) return W4_ERR_WORKSPACE;
  p.q = q, p.q_stride = q_stride;
  p.kc = (const uint8_t*)k_codes, p.vc = (const uint8_t*)v_codes, p.ks = k_scale, p.vs = v_scale;
  p.indptr = q_indptr, p.kv_len = kv_len, p.table = page_table;
  p.out = out, p.lse = lse;
  p.counters = (uint32_t*)workspace;
  p.part = workspace ? (float*)((uint8_t*)workspace + WS_COUNTERS) : nullptr;
  p.scale_log2 = fabsf(sm_scale) * 1.4426950408889634f;
  p.q_sign = sm_scale < 0.f ? 0x80008000u : 0u;
  p.batch = batch, p.tokens = tokens, p.max_kv = max_kv, p.cols = table_cols;
  p.q_heads = q_heads, p.kv_heads = kv_heads, p.group = q_heads / kv_heads, p.dim = head_dim;
  p.page_shift = __builtin_ctz(page_size), p.pages = num_pages;
  p.tiles = a.tiles, p.chunk = a.chunk, p.splits = a.splits, p.by_row = a.by_row;
  if (a.many) {
    if (a.units * a.splits > MAX_BLOCKS) return W4_ERR_SHAPE;
    return launch_attn_many(p, dp, q_dtype, a.units * a.splits, stream);
  }
#define W4_DP(D)                                                  \
  case D:                                                         \
    return q_dtype == W4_Q_I8 ? launch_attn<D, W4_Q_I8>(p, a, stream) \
                              : launch_attn<D, W4_Q_F8>(p, a, stream)
  switch (dp) {
    W4_DP(64);
    W4_DP(96);
    W4_DP(128);
    W4_DP(192);
    default:
      return q_dtype == W4_Q_I8 ? launch_attn<256, W4_Q_I8>(p, a, stream)
                                : launch_attn<256, W4_Q_F8>(p, a, stream);
  }
#undef W4_DP
}
