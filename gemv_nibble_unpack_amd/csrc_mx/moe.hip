// A mixture-of-experts layer on MXFP4 weights for a few tokens.
//
// A (token, choice) is a pair. Two kernels: the first finds each token's experts
// and writes h = act(gate) * up of every pair, the second multiplies by the
// down projections and sums a token's pairs. Up to ROUTE_IN tokens every block of the
// first kernel takes the choices itself, above that a kernel before it does.
//
// Bound: the bytes of the experts in use.
#include "mx_gemm.hpp"

namespace w4 {

constexpr int MOE_PAIRS = W4_MOE_MAX_TOKENS * W4_MOE_MAX_TOP;
constexpr int ROUTE_IN = 8;
constexpr int MOE_THREADS = 512, MOE_WAVES = 8;
constexpr int DOWN_SP = 4;               // strips of a block that takes one expert

// which experts are in use and by whom
struct MoeRoute {
  int active;                            // experts in use
  int bad[W4_MOE_MAX_TOKENS];            // the token's logits hold a NaN or +infinity
  int expert[W4_MOE_MAX_EXPERTS];        // in ascending order
  int first[W4_MOE_MAX_EXPERTS + 1];     // of its pairs in `list`
  int list[MOE_PAIRS];                   // pairs token * top + choice, by expert
  float weight[MOE_PAIRS];               // of pair; -1: a choice that is none
};

struct MoeParams {
  const uint16_t* x;
  const void* logits;
  const uint8_t *w1, *w2;
  uint16_t* out;
  uint32_t* counters;
  MoeRoute* route;
  float *h, *y;                          // [pairs][I], [pairs][H]
  int T, H, I, E, top, act, renorm, half_logits;
};

struct MoeChoice {                       // in LDS while the choices are taken
  int id[MOE_PAIRS];                     // expert, -1 for none
  int waves[MOE_WAVES];
};

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);           // -0 as +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One wave: the `top` largest logits of token t, ties to the lowest expert, and
// their softmax weights.
__device__ void route_token(const MoeParams& p, int t, MoeRoute& r, MoeChoice& ch) {
  constexpr int R = W4_MOE_MAX_EXPERTS / 64;
  const int lane = threadIdx.x & 63;
  const float ninf = -__builtin_inff();
  float v[R];
  uint32_t key[R];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = 64 * i + lane;
    v[i] = ninf;
    if (e < p.E)
      v[i] = p.half_logits ? h2f(reinterpret_cast<const uint16_t*>(p.logits)[(int64_t)t * p.E + e])
                           : reinterpret_cast<const float*>(p.logits)[(int64_t)t * p.E + e];
    bad |= !(v[i] < __builtin_inff());
    key[i] = e < p.E ? order_key(v[i]) : 0u;
  }
  bad = __ballot(bad) != 0;
  float most = 0.f, sum = 0.f;
  for (int j = 0; j < p.top; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) m = max(m, key[i]);
    m = wave_max_u(m);
    int id = -1;
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      const uint64_t b = __ballot(key[i] == m);
      if (b) id = 64 * i + __builtin_ctzll(b);
    }
    const float l = __uint_as_float(m & 0x80000000u ? m & 0x7FFFFFFFu : ~m);
    const bool none = bad || m == 0 || l == ninf;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (id == 64 * i + lane) key[i] = 0;
    if (j == 0) {
      most = l;
      if (!p.renorm && !none) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) s += expf(v[i] - most);        // of -infinity: 0
        sum = wave_sum_f(s);
      }
    }
    const float w = none ? 0.f : expf(l - most);
    if (p.renorm) sum += w;
    if (lane == 0) {
      ch.id[t * p.top + j] = none ? -1 : id;
      r.weight[t * p.top + j] = none ? -1.f : w;
    }
  }
  if (lane == 0) {
    r.bad[t] = bad;
    for (int j = 0; j < p.top; ++j)
      if (ch.id[t * p.top + j] >= 0) r.weight[t * p.top + j] /= sum;
  }
}

// The whole block: experts in use and their pairs, from the choices.
__device__ void route_lists(const MoeParams& p, MoeRoute& r, MoeChoice& ch) {
  const int pairs = p.T * p.top, e = threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int n = 0, before = 0;
  if (e < p.E)
    for (int i = 0; i < pairs; ++i) {
      const int id = ch.id[i];
      n += id == e;
      before += id >= 0 && id < e;                       // their pairs come first
    }
  const uint64_t used = __ballot(n > 0);
  if (lane == 0) ch.waves[wave] = __builtin_popcountll(used);
  __syncthreads();
  int a = __builtin_popcountll(used & ((1ull << lane) - 1)), all = 0;
  for (int i = 0; i < MOE_WAVES; ++i) {
    if (i < wave) a += ch.waves[i];
    all += ch.waves[i];
  }
  if (n > 0) {
    r.expert[a] = e;
    r.first[a] = before;
    int at = before;
    for (int i = 0; i < pairs; ++i)
      if (ch.id[i] == e) r.list[at++] = i;
    if (a == all - 1) r.first[all] = at;
  }
  if (threadIdx.x == 0) r.active = all;
  __syncthreads();
}

__global__ __launch_bounds__(MOE_THREADS) void k_moe_route(const MoeParams p) {
  __shared__ MoeChoice ch;
  for (int t = threadIdx.x >> 6; t < p.T; t += MOE_WAVES) route_token(p, t, *p.route, ch);
  __syncthreads();
  route_lists(p, *p.route, ch);
}

__device__ __forceinline__ float moe_act(float g, int act) {
  if (act == W4_ACT_RELU2) {
    g = fmaxf(g, 0.f);
    return g * g;
  }
  const float z = act == W4_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.f + expf(-z));           // tanh(z) = 2 / (1 + exp(-2 z)) - 1
}

// h of one strip of 16 inner rows (gate and up) for one expert's pairs
template <int QT, bool ROUTE>
__global__ __launch_bounds__(MOE_THREADS) void k_moe_up(const MoeParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];     // sums
  __shared__ typename std::conditional<ROUTE, MoeRoute, int>::type own;
  __shared__ typename std::conditional<ROUTE, MoeChoice, int>::type ch;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int strips = p.I / 16;
  const int a = block_number() / strips, s = block_number() - a * strips;
  const MoeRoute* r = p.route;
  if constexpr (ROUTE) {
    if (wave < p.T) route_token(p, wave, own, ch);
    __syncthreads();
    route_lists(p, own, ch);
    if (block_number() == 0)                             // for the second kernel
      for (int i = threadIdx.x; i < (int)(sizeof(MoeRoute) / 4); i += MOE_THREADS)
        reinterpret_cast<int*>(p.route)[i] = reinterpret_cast<const int*>(&own)[i];
    r = &own;
  }
  if (a >= r->active) return;
  const int e = r->expert[a], first = r->first[a], n = r->first[a + 1] - first;
  const MxGeometry geo = mx_geometry((int64_t)p.E * 2 * p.I, p.H);

  const uint8_t *wt[2], *ws[2];
  uint32_t rowmax[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = (int64_t)e * 2 * strips + i * strips + s;
    wt[i] = p.w1 + t * geo.KT * TILE_BYTES + 16 * lane;
    ws[i] = p.w1 + geo.s_off + t * geo.KQ * 256 + 4 * lane;
    rowmax[i] = p.w1[geo.e_off + 16 * t + c];
  }
  const uint16_t* row[QT];
#pragma unroll
  for (int u = 0; u < QT; ++u)
    row[u] = p.x + (int64_t)(r->list[first + min(16 * u + c, n - 1)] / p.top) * p.H;
  f4 acc[2][QT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int u = 0; u < QT; ++u) acc[i][u] = f4{0.f, 0.f, 0.f, 0.f};

  constexpr int U = 2;
  const int end = geo.KT * (wave + 1) / MOE_WAVES;
  for (int kt = geo.KT * wave / MOE_WAVES; kt < end; kt += U) {
    u4 w[U][2];
    uint32_t sc[U][2];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = min(kt + j, end - 1);
        w[j][i] = *reinterpret_cast<const u4*>(wt[i] + (int64_t)x * TILE_BYTES);
        sc[j][i] = ws[i][(x >> 2) * 256 + (x & 3)];
      }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (kt + j >= end) break;
      const int k = 128 * (kt + j) + 32 * g;
      float up[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) up[i] = h_scale(sc[j][i], rowmax[i]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const h8 b0 = fp4_h8(w[j][0][x], up[0]), b1 = fp4_h8(w[j][1][x], up[1]);
#pragma unroll
        for (int u = 0; u < QT; ++u) {
          if (16 * u >= n) break;
          const h8 f = *reinterpret_cast<const h8*>(k < p.H ? (const uint8_t*)(row[u] + k + 8 * x) : mx_zeros);
          acc[0][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b0, f, acc[0][u], 0, 0, 0);
          acc[1][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b1, f, acc[1][u], 0, 0, 0);
        }
      }
    }
  }

  f4* sums = reinterpret_cast<f4*>(smem);                // [wave][gate, up][QT][64]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int u = 0; u < QT; ++u) sums[((wave * 2 + i) * QT + u) * 64 + lane] = acc[i][u];
  __syncthreads();
  for (int x = threadIdx.x; x < QT * 64; x += MOE_THREADS) {
    const int l = x & 63, u = x >> 6, col = 16 * u + (l & 15), i = 16 * s + 4 * (l >> 4);
    if (col >= n) continue;
    f4 gv = {0.f, 0.f, 0.f, 0.f}, uv = gv;
    for (int z = 0; z < MOE_WAVES; ++z) {
      const f4 ga = sums[(z * 2 * QT + u) * 64 + l], ua = sums[((z * 2 + 1) * QT + u) * 64 + l];
#pragma unroll
      for (int y = 0; y < 4; ++y) gv[y] += ga[y], uv[y] += ua[y];
    }
    const uint8_t* top0 = p.w1 + geo.e_off + ((int64_t)e * 2 * strips + s) * 16 + 4 * (l >> 4);
    f4 h;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const float gate = ldexpf(gv[y], (int)top0[y] - 127 - H_UP);
      h[y] = moe_act(gate, p.act) * ldexpf(uv[y], (int)top0[16 * strips + y] - 127 - H_UP);
    }
    *reinterpret_cast<f4*>(p.h + (int64_t)r->list[first + col] * p.I + i) = h;
  }
}

// The largest power of two that brings values of magnitude m into fp16's range, as a
// factor, and its reciprocal
__device__ __forceinline__ void h_factor(float m, float& up, float& down) {
  const int e = min(max((int)(__float_as_uint(m) >> 23), 20), 230);  // also of infinity
  up = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
  down = __uint_as_float((uint32_t)(e - 14) << 23);
}

// TOKENS: a block takes every expert in use for its strip, columns are the tokens
// (up to 16), and the sums over a token's experts stay in its registers.
// Otherwise: SP strips of one expert for its pairs, joined by the last block of a
// strip group.
template <int QT, int SP, bool TOKENS>
__global__ __launch_bounds__(MOE_THREADS) void k_moe_down(const MoeParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ unsigned slast;
  static_assert(!TOKENS || QT == 1, "tokens are the columns of one operand");
  const MoeRoute& r = *p.route;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int strips = p.H / 16, groups = (strips + SP - 1) / SP;
  const int a = TOKENS ? 0 : block_number() / groups;
  const int grp = block_number() - a * groups;
  if (grp >= groups || (!TOKENS && a > 0 && a >= r.active)) return;
  const bool empty = !TOKENS && r.active == 0;           // no token chose: the rows are 0
  const int experts = TOKENS ? r.active : empty ? 0 : 1;
  const int first = TOKENS || empty ? 0 : r.first[a], n = TOKENS ? p.T : empty ? 0 : r.first[a + 1] - first;
  const MxGeometry geo = mx_geometry((int64_t)p.E * p.H, p.I);

  f4 acc[SP][QT];
#pragma unroll
  for (int i = 0; i < SP; ++i)
#pragma unroll
    for (int u = 0; u < QT; ++u) acc[i][u] = f4{0.f, 0.f, 0.f, 0.f};

  const int units = experts * geo.KT;
  const int end = (int)((int64_t)units * (wave + 1) / MOE_WAVES);
  int unit = (int)((int64_t)units * wave / MOE_WAVES);
  int ex = unit / geo.KT, kt = unit - ex * geo.KT;       // a unit: expert, k tile
  int pair[QT];
  auto enter = [&] {                                     // this lane's pairs of expert ex, -1 for none
    if constexpr (TOKENS) {
      pair[0] = -1;
      const int f = r.first[ex], l = r.first[ex + 1];
      for (int i = f; i < l; ++i)
        if (r.list[i] / p.top == c) pair[0] = r.list[i];
    } else {
#pragma unroll
      for (int u = 0; u < QT; ++u) pair[u] = 16 * u + c < n ? r.list[first + 16 * u + c] : -1;
    }
  };
  if (unit < end) enter();
  for (; unit < end; ++unit) {
    const int64_t t = (int64_t)r.expert[a + ex] * strips + grp * SP;
    u4 w[SP];
    float up[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      const int64_t ti = t + min(i, strips - 1 - grp * SP);
      w[i] = *reinterpret_cast<const u4*>(p.w2 + (ti * geo.KT + kt) * TILE_BYTES + 16 * lane);
      const uint32_t byte = p.w2[geo.s_off + (ti * geo.KQ + (kt >> 2)) * 256 + 4 * lane + (kt & 3)];
      up[i] = h_scale(byte, p.w2[geo.e_off + 16 * ti + c]);
    }
    h8 hf[QT][4];
    float down[QT];
    const int k = 128 * kt + 32 * g;
#pragma unroll
    for (int u = 0; u < QT; ++u) {
      float v[32];
      const bool in = pair[u] >= 0 && k < p.I;
      const float* hp = p.h + (int64_t)max(pair[u], 0) * p.I + min(k, p.I - 32);
      const float weight = TOKENS && in ? r.weight[pair[u]] : 1.f;
      float m = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const f4 x = *reinterpret_cast<const f4*>(hp + 4 * q);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          v[4 * q + y] = in ? x[y] * weight : 0.f;
          m = fmaxf(m, fabsf(v[4 * q + y]));
        }
      }
      m = fmaxf(m, __shfl_xor(m, 16, 64));
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      float f;
      h_factor(m, f, down[u]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int y = 0; y < 8; ++y) hf[u][q][y] = (_Float16)(v[8 * q + y] * f);
    }
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      f4 d[QT];
#pragma unroll
      for (int u = 0; u < QT; ++u) d[u] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const h8 b = fp4_h8(w[i][x], up[i]);
#pragma unroll
        for (int u = 0; u < QT; ++u) d[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, hf[u][x], d[u], 0, 0, 0);
      }
      // rows 4 g .. of the strip, each counted from its largest scale
      const int64_t ti = t + min(i, strips - 1 - grp * SP);
      const uint32_t tops = *reinterpret_cast<const uint32_t*>(p.w2 + geo.e_off + 16 * ti + 4 * g);
#pragma unroll
      for (int u = 0; u < QT; ++u)
#pragma unroll
        for (int y = 0; y < 4; ++y)
          // a token that did not choose the expert takes nothing, NaN weights neither
          if (!TOKENS || pair[u] >= 0)
            acc[i][u][y] += ldexpf(d[u][y] * down[u], (int)(tops >> (8 * y) & 255u) - 127 - H_UP);
    }
    if (++kt == geo.KT) {
      kt = 0;
      ++ex;
      if (unit + 1 < end) enter();
    }
  }

  f4* sums = reinterpret_cast<f4*>(smem);                // [wave][SP][QT][64]
#pragma unroll
  for (int i = 0; i < SP; ++i)
#pragma unroll
    for (int u = 0; u < QT; ++u) sums[((wave * SP + i) * QT + u) * 64 + lane] = acc[i][u];
  __syncthreads();
  const float nan = __uint_as_float(0x7FC00000u);
  for (int x = threadIdx.x; x < SP * QT * 64; x += MOE_THREADS) {
    const int l = x & 63, u = (x >> 6) % QT, i = (x >> 6) / QT;
    const int col = 16 * u + (l & 15), strip = grp * SP + i;
    if (col >= n || strip >= strips) continue;
    f4 v = {0.f, 0.f, 0.f, 0.f};
    for (int z = 0; z < MOE_WAVES; ++z) {
      const f4 q = sums[((z * SP + i) * QT + u) * 64 + l];
#pragma unroll
      for (int y = 0; y < 4; ++y) v[y] += q[y];
    }
    const int at = 16 * strip + 4 * (l >> 4);
    if constexpr (TOKENS) {
      h4 o;
#pragma unroll
      for (int y = 0; y < 4; ++y) o[y] = (_Float16)(r.bad[col] ? nan : v[y]);
      *reinterpret_cast<u2*>(p.out + (int64_t)col * p.H + at) = __builtin_bit_cast(u2, o);
    } else {
      const int pr = r.list[first + col];
      const float wgt = r.weight[pr];
      uint32_t* y = reinterpret_cast<uint32_t*>(p.y) + (int64_t)pr * p.H + at;
      dev_store2(y, __float_as_uint(v[0] * wgt), __float_as_uint(v[1] * wgt));
      dev_store2(y + 2, __float_as_uint(v[2] * wgt), __float_as_uint(v[3] * wgt));
    }
  }
  if constexpr (TOKENS) return;
  if (!empty) {
    stores_done();
    __syncthreads();
    if (threadIdx.x == 0) slast = dev_arrive(p.counters + grp) == (unsigned)(r.active - 1);
    __syncthreads();
    if (!slast) return;
    if (threadIdx.x == 0) dev_store(p.counters + grp, 0u);
  }
  // the last block of these columns: each token's pairs in the order of its choices
  for (int x = threadIdx.x; x < p.T * SP * 4; x += MOE_THREADS) {
    const int tok = x / (SP * 4), col = 16 * SP * grp + 4 * (x % (SP * 4));
    if (col >= p.H) continue;
    f4 v = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.top; ++j) {
      const int pr = tok * p.top + j;
      if (empty || r.weight[pr] < 0.f) continue;
      const uint32_t* y = reinterpret_cast<const uint32_t*>(p.y) + (int64_t)pr * p.H + col;
      const uint64_t lo = dev_load2(y), hi = dev_load2(y + 2);
      v[0] += __uint_as_float((uint32_t)lo), v[1] += __uint_as_float((uint32_t)(lo >> 32));
      v[2] += __uint_as_float((uint32_t)hi), v[3] += __uint_as_float((uint32_t)(hi >> 32));
    }
    h4 o;
#pragma unroll
    for (int y = 0; y < 4; ++y) o[y] = (_Float16)(r.bad[tok] ? nan : v[y]);
    *reinterpret_cast<u2*>(p.out + (int64_t)tok * p.H + col) = __builtin_bit_cast(u2, o);
  }
}

static bool moe_sizes_ok(int T, int H, int I, int E, int top) {
  return T >= 0 && T <= W4_MOE_MAX_TOKENS && E >= 1 && E <= W4_MOE_MAX_EXPERTS && top >= 1 &&
         top <= W4_MOE_MAX_TOP && top <= E && H >= 32 && H % 32 == 0 && H <= W4_MAX_K && I >= 32 &&
         I % 32 == 0 && I <= W4_MAX_K;
}
static bool moe_tokens(int T) { return T <= 16; }        // tokens as columns, nothing to join

struct MoeSpace {
  int64_t h, y, total;
};
static MoeSpace moe_space(int T, int H, int I, int top) {
  MoeSpace s;
  s.h = WS_COUNTERS + (int64_t)((sizeof(MoeRoute) + 255) / 256 * 256);
  s.y = s.h + (int64_t)T * top * I * 4;
  s.total = s.y + (moe_tokens(T) ? 0 : (int64_t)T * top * H * 4);
  return s;
}

template <int QT>
int launch_up(const MoeParams& p, bool route, int64_t blocks, hipStream_t stream) {
  constexpr int lds = MOE_WAVES * 2 * QT * 1024;
  if (route) {
    if constexpr (QT == 1)
      hipLaunchKernelGGL((k_moe_up<1, true>), grid_of(blocks), dim3(MOE_THREADS), lds, stream, p);
  } else {
    hipLaunchKernelGGL((k_moe_up<QT, false>), grid_of(blocks), dim3(MOE_THREADS), lds, stream, p);
  }
  return launch_status();
}
template <int QT>
int launch_down(const MoeParams& p, int64_t blocks, hipStream_t stream) {
  constexpr int lds = MOE_WAVES * DOWN_SP * QT * 1024;
  allow_smem((const void*)&k_moe_down<QT, DOWN_SP, false>, lds);
  hipLaunchKernelGGL((k_moe_down<QT, DOWN_SP, false>), grid_of(blocks), dim3(MOE_THREADS), lds, stream, p);
  return launch_status();
}

}  // namespace w4

using namespace w4;

extern "C" size_t moe_mx4_workspace_bytes(int tokens, int hidden, int inner, int experts, int top_k) {
  if (!moe_sizes_ok(tokens, hidden, inner, experts, top_k) || tokens == 0) return 0;
  return (size_t)moe_space(tokens, hidden, inner, top_k).total;
}

extern "C" int moe_mx4(const uint16_t* x, const void* logits, int logits_dtype, int tokens, int hidden,
                       int inner, int experts, int top_k, int renormalize, int act,
                       const uint8_t* w_gate_up, const uint8_t* w_down, uint16_t* out,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (logits_dtype != W4_IN_F16 && logits_dtype != W4_IN_F32) return W4_ERR_ARG;
  if (act < W4_ACT_SILU || act > W4_ACT_RELU2) return W4_ERR_ARG;
  if (!moe_sizes_ok(tokens, hidden, inner, experts, top_k)) return W4_ERR_SHAPE;
  if (tokens == 0) return W4_OK;
  if (!x || !logits || !w_gate_up || !w_down || !out) return W4_ERR_NULL;
  if (!aligned(x, 16) || !aligned(logits, logits_dtype == W4_IN_F16 ? 2 : 4) ||
      !aligned(w_gate_up, 16) || !aligned(w_down, 16) || !aligned(out, 8) || !aligned(workspace, 256))
    return W4_ERR_ALIGN;
  const MoeSpace s = moe_space(tokens, hidden, inner, top_k);
  if (!workspace || workspace_bytes < (size_t)s.total) return W4_ERR_WORKSPACE;
  uint8_t* ws = (uint8_t*)workspace;
  MoeParams p{};
  p.x = x, p.logits = logits, p.w1 = w_gate_up, p.w2 = w_down, p.out = out;
  p.counters = (uint32_t*)ws, p.route = (MoeRoute*)(ws + WS_COUNTERS);
  p.h = (float*)(ws + s.h), p.y = (float*)(ws + s.y);
  p.T = tokens, p.H = hidden, p.I = inner, p.E = experts, p.top = top_k, p.act = act;
  p.renorm = renormalize != 0, p.half_logits = logits_dtype == W4_IN_F16;

  const bool route = tokens <= ROUTE_IN;
  if (!route) {
    hipLaunchKernelGGL(k_moe_route, dim3(1), dim3(MOE_THREADS), 0, stream, p);
    if (const int st = launch_status()) return st;
  }
  const int64_t most = min(experts, tokens * top_k);     // experts in use, at most
  const int64_t up = most * (inner / 16);
  const int st = tokens <= 16   ? launch_up<1>(p, route, up, stream)
                 : tokens <= 32 ? launch_up<2>(p, route, up, stream)
                                : launch_up<4>(p, route, up, stream);
  if (st) return st;
  if (moe_tokens(tokens)) {
    hipLaunchKernelGGL((k_moe_down<1, 1, true>), grid_of(hidden / 16), dim3(MOE_THREADS),
                       MOE_WAVES * 1024, stream, p);
    return launch_status();
  }
  const int64_t down = most * ((hidden / 16 + DOWN_SP - 1) / DOWN_SP);
  return tokens <= 32 ? launch_down<2>(p, down, stream) : launch_down<4>(p, down, stream);
}
