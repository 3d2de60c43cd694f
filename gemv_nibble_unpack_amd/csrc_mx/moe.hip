// A mixture-of-experts layer on MXFP4 weights for a few tokens.
//
// A (token, choice) is a pair. Two kernels: the first finds each token's experts
// and writes h = w * act(gate) * up of every pair, the second multiplies by the
// down projections and sums a token's pairs. One token's choices every wave of the
// first kernel takes itself, more tokens' a kernel before it (which took longer in
// every block already for two: 33.4 us against 31.0 at 64 experts of 1536).
//
// fp16 x meets the weights widened to fp16 (mx_common.hpp). h, a product of two
// sums, has float32's range: it is kept as two bfloat16 numbers, hi + lo (16 bits
// of it, relative error 2^-17), each multiplied by the weights, which are exact in
// bfloat16, with float32 sums.
//
// Bound: the bytes of the experts in use. One token on 4 of 64 experts (hidden 4096,
// inner 1536, 40 MB) takes 10.1 + 7.7 us: choices, one round trip to memory, the weights;
// 16 tokens on about 41 of them 5 + 57 + 39 us (4.3 TB/s over the two products),
// 61 tokens on 16 experts (hidden 3200, inner 4320, 352 MB) 7.5 + 54 + 44 us.
#include "mx_gemm.hpp"

namespace w4 {

typedef __bf16 b2v __attribute__((ext_vector_type(2)));
typedef __bf16 b4v __attribute__((ext_vector_type(4)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));

constexpr int MOE_PAIRS = W4_MOE_MAX_TOKENS * W4_MOE_MAX_TOP;
constexpr int MOE_COLS = 16;             // tokens that the second kernel takes as columns
constexpr int MOE_THREADS = 512, MOE_WAVES = 8, ROUTE_THREADS = 1024;
constexpr int DOWN_SP = 4, DOWN_WAVES = 4;       // strips and waves of a block that takes one expert

// which experts are in use and by whom
struct MoeRoute {
  int active;                            // experts in use
  int bad[W4_MOE_MAX_TOKENS];            // the token's logits hold a NaN or +infinity
  int expert[W4_MOE_MAX_EXPERTS];        // in ascending order
  int first[W4_MOE_MAX_EXPERTS + 1];     // of its pairs in `list`
  int list[MOE_PAIRS];                   // pairs token * top + choice, by expert
  float weight[MOE_PAIRS];               // of pair; -1: a choice that is none
  int16_t column[MOE_COLS * W4_MOE_MAX_TOP][MOE_COLS];   // of expert in use and token: its pair, or -1
};

struct MoeParams {
  const uint16_t* x;
  const void* logits;
  const uint8_t *w1, *w2;
  uint16_t* out;
  uint32_t* counters;
  MoeRoute* route;
  __bf16* h;                             // [pairs][I], hi, then lo; grouped: see h_at
  float* y;                              // [pairs][H]
  int T, H, I, E, top, act, renorm, half_logits, grouped;
};

// Grouped h: 16 places in `list` by 128 k, in the order in which the second product's
// lanes take them: hi and lo, four steps of k, then 16 bytes a lane, so that a wave
// reads whole lines (61 tokens on 16 experts of 4320: 45 us, 53 on rows of h, whose
// lanes lie a row apart).
constexpr int H_GROUP = 2 * 16 * 128;
__host__ __device__ inline int64_t h_group(int place, int kt, int I) {
  return ((int64_t)(place >> 4) * ((I + 127) / 128) + kt) * H_GROUP;
}

struct MoeChoice {                       // in LDS while the choices are taken
  int id[MOE_PAIRS];                     // expert, -1 for none
  int place[MOE_PAIRS];                  // among the expert's pairs
  int count[W4_MOE_MAX_EXPERTS], before[W4_MOE_MAX_EXPERTS];
  int waves[2][ROUTE_THREADS / 64];
};

__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);           // -0 as +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One wave: the `top` largest logits of token t (of up to 64 R experts), ties to the
// lowest expert, and their softmax weights, choice j in lane j (-1 for none).
template <int R>
__device__ __forceinline__ void route_token(const MoeParams& p, int t, int& id, float& weight, bool& bad) {
  const int lane = threadIdx.x & 63;
  const float ninf = -__builtin_inff();
  float v[R];
  uint32_t key[R];
  bad = false;
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
  id = -1;
  float l = ninf, most = 0.f;
  for (int j = 0; j < p.top; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) m = max(m, key[i]);
    m = wave_max_u(m);
    int e = 0;
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      const uint64_t b = __ballot(key[i] == m);
      if (b) e = 64 * i + __builtin_ctzll(b);
    }
    const float lj = __uint_as_float(m & 0x80000000u ? m & 0x7FFFFFFFu : ~m);
    if (bad || m == 0 || lj == ninf) break;              // the same for the wave
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (e == 64 * i + lane) key[i] = 0;
    if (j == 0) most = lj;
    if (lane == j) id = e, l = lj;
  }
  const float w = id >= 0 ? expf(l - most) : 0.f;
  float s = w;
  if (!p.renorm && !bad) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) s += v[i] == ninf ? 0.f : expf(v[i] - most);
  }
  s = wave_sum_f(s);
  weight = id >= 0 ? w / s : -1.f;
}

// The whole block: experts in use and their pairs, from the choices. An expert's
// pairs come in any order: they are columns of its products, none meets another.
__device__ __forceinline__ void route_lists(const MoeParams& p, MoeRoute& r, MoeChoice& ch) {
  const int pairs = p.T * p.top, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < pairs; i += ROUTE_THREADS)
    if (ch.id[i] >= 0) ch.place[i] = atomicAdd(&ch.count[ch.id[i]], 1);
  __syncthreads();
  const int n = tid < p.E ? ch.count[tid] : 0;
  const uint64_t used = __ballot(n > 0);
  int upto = n;                                          // pairs of this expert and those before
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int q = __shfl_up(upto, o, 64);
    if (lane >= o) upto += q;
  }
  if (lane == 63) {
    ch.waves[0][wave] = __builtin_popcountll(used);
    ch.waves[1][wave] = upto;
  }
  __syncthreads();
  int a = __builtin_popcountll(used & ((1ull << lane) - 1)), all = 0, sum = 0;
  upto -= n;
  for (int i = 0; i < ROUTE_THREADS / 64; ++i) {
    if (i < wave) a += ch.waves[0][i], upto += ch.waves[1][i];
    all += ch.waves[0][i], sum += ch.waves[1][i];
  }
  if (n > 0) {
    r.expert[a] = tid;
    r.first[a] = upto;
    ch.before[tid] = upto;
    ch.count[tid] = a;
  }
  if (tid == 0) r.active = all, r.first[all] = sum;
  const bool columns = p.T <= MOE_COLS;
  if (columns)
    for (int i = tid; i < all * MOE_COLS / 2; i += ROUTE_THREADS) reinterpret_cast<uint32_t*>(r.column)[i] = 0xFFFFFFFFu;
  __syncthreads();
  for (int i = tid; i < pairs; i += ROUTE_THREADS)
    if (ch.id[i] >= 0) {
      r.list[ch.before[ch.id[i]] + ch.place[i]] = i;
      if (columns) r.column[ch.count[ch.id[i]]][i / p.top] = (int16_t)i;
    }
}

template <int R>
__global__ __launch_bounds__(ROUTE_THREADS) void k_moe_route(const MoeParams p) {
  __shared__ MoeChoice ch;
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < W4_MOE_MAX_EXPERTS) ch.count[threadIdx.x] = 0;
  for (int t = threadIdx.x >> 6; t < p.T; t += ROUTE_THREADS / 64) {
    int id;
    float weight;
    bool bad;
    route_token<R>(p, t, id, weight, bad);
    if (lane < p.top) ch.id[t * p.top + lane] = id, p.route->weight[t * p.top + lane] = weight;
    if (lane == 0) p.route->bad[t] = bad;
  }
  __syncthreads();
  route_lists(p, *p.route, ch);
}

__device__ __forceinline__ float moe_act(float g, int act) {
  if (act == W4_ACT_RELU2) {
    g = g < 0.f ? 0.f : g;               // (a maximum would lose a NaN)
    return g * g;
  }
  const float z = act == W4_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.f + expf(-z));           // tanh(z) = 2 / (1 + exp(-2 z)) - 1
}

// h of P strips of 16 inner rows (gate and up) for one expert's pairs, 16 QT of them at
// a time. R: one token, whose choices (of up to 64 R experts) the waves take themselves;
// 0: they are there.
template <int P, int QT, int R, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_moe_up(const MoeParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];     // sums
  constexpr int SP = 2 * P;              // strips: gate, up, gate, up ..
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int strips = p.I / 16, groups = (strips + P - 1) / P;
  const int a = block_number() / groups, s0 = (block_number() - a * groups) * P;
  f4* sums = reinterpret_cast<f4*>(smem);                // [wave][SP][QT][64]
  uint8_t* const xs = smem + WAVES * SP * QT * 1024;     // the one token's x, 16 bytes of zeros behind it
  const MoeRoute* r = p.route;
  int e, n = 1, first = 0, own = 0;
  float own_weight = 0.f;
  // (what the weights' addresses come from in scalar registers)
  if constexpr (R != 0) {                                // every wave for itself
    for (int i = threadIdx.x; i < p.H / 8; i += 64 * WAVES)
      reinterpret_cast<u4*>(xs)[i] = reinterpret_cast<const u4*>(p.x)[i];
    if (threadIdx.x == 0) reinterpret_cast<u4*>(xs)[p.H / 8] = u4{0u, 0u, 0u, 0u};
    int id;
    float weight;
    bool bad;
    route_token<R>(p, 0, id, weight, bad);
    const uint64_t chosen = __ballot(id >= 0);
    const int active = __builtin_popcountll(chosen);
    int rank = 0;                                        // among the chosen, by expert
    for (int j = 0; j < active; ++j) rank += __builtin_amdgcn_readlane(id, j) < id;
    if (block_number() == 0 && wave == 0) {              // for the second kernel
      MoeRoute& w = *p.route;
      if (lane < p.top) w.weight[lane] = weight;
      if (lane < active) w.expert[rank] = id, w.first[rank] = rank, w.list[rank] = lane;
      if (lane == 0) w.active = active, w.first[active] = active, w.bad[0] = bad;
      if (lane < active)
        for (int i = 0; i < MOE_COLS; ++i) w.column[rank][i] = (int16_t)(i == 0 ? lane : -1);
    }
    if (a >= active) return;
    own = __builtin_ctzll(__ballot(id >= 0 && rank == a));
    e = __builtin_amdgcn_readlane(id, own);
    own_weight = lane_f(weight, own);
    __syncthreads();
  } else {
    const int active = r->active;
    e = __builtin_amdgcn_readfirstlane(r->expert[min(a, W4_MOE_MAX_EXPERTS - 1)]);
    first = __builtin_amdgcn_readfirstlane(r->first[min(a, W4_MOE_MAX_EXPERTS - 1)]);
    n = __builtin_amdgcn_readfirstlane(r->first[min(a + 1, W4_MOE_MAX_EXPERTS)]) - first;
    if (a >= active) return;
  }
  const MxGeometry geo = mx_geometry((int64_t)p.E * 2 * p.I, p.H);

  const uint8_t *wt[SP], *ws[SP];
  uint32_t rowmax[SP];
#pragma unroll
  for (int i = 0; i < SP; ++i) {
    const int64_t t = (int64_t)e * 2 * strips + (i & 1) * strips + min(s0 + i / 2, strips - 1);
    wt[i] = p.w1 + t * geo.KT * TILE_BYTES;
    ws[i] = p.w1 + geo.s_off + t * geo.KQ * 256;
    rowmax[i] = p.w1[geo.e_off + 16 * t + c];
  }
  const int end = geo.KT * (wave + 1) / WAVES;
  for (int n0 = 0; n0 < n; n0 += 16 * QT) {
    int64_t row[QT];                                     // of x
#pragma unroll
    for (int u = 0; u < QT; ++u)
      row[u] = R != 0 ? 0 : (int64_t)(r->list[first + min(n0 + 16 * u + c, n - 1)] / p.top) * p.H;
    f4 acc[SP][QT];
#pragma unroll
    for (int i = 0; i < SP; ++i)
#pragma unroll
      for (int u = 0; u < QT; ++u) acc[i][u] = f4{0.f, 0.f, 0.f, 0.f};

    constexpr int U = R != 0 ? 4 / P : P == 1 ? 2 : 1;
    for (int kt = geo.KT * wave / WAVES; kt < end; kt += U) {
      u4 w[U][SP];
      uint32_t sc[U][SP];
      h8 f[R != 0 ? 1 : U][QT][4];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int x = min(kt + j, end - 1), k = 128 * x + 32 * g;
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          w[j][i] = g_load<u4>(wt[i] + (int64_t)x * TILE_BYTES, 16 * lane);
          sc[j][i] = g_load<uint8_t>(ws[i] + (x >> 2) * 256 + (x & 3), 4 * lane);
        }
        if constexpr (R == 0) {
#pragma unroll
          for (int u = 0; u < QT; ++u)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              f[j][u][y] = g_load<h8>(k < p.H ? (const uint8_t*)(p.x + row[u] + k + 8 * y) : mx_zeros);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (kt + j >= end) break;
        constexpr bool LOCAL = R != 0;
        if constexpr (LOCAL) {
          const int k = 128 * (kt + j) + 32 * g;
#pragma unroll
          for (int u = 0; u < QT; ++u)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              f[0][u][y] = *reinterpret_cast<const h8*>(xs + 2 * (k < p.H ? k + 8 * y : p.H));
        }
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          const float up = h_scale(sc[j][i], rowmax[i]);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const h8 b = fp4_h8(w[j][i][y], up);
#pragma unroll
            for (int u = 0; u < QT; ++u)
              acc[i][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, f[LOCAL ? 0 : j][u][y], acc[i][u], 0, 0, 0);
          }
        }
      }
    }

    if (n0 > 0) __syncthreads();                         // the sums before are read out
#pragma unroll
    for (int i = 0; i < SP; ++i)
#pragma unroll
      for (int u = 0; u < QT; ++u) sums[((wave * SP + i) * QT + u) * 64 + lane] = acc[i][u];
    __syncthreads();
    for (int x = threadIdx.x; x < P * QT * 64; x += 64 * WAVES) {
      const int l = x & 63, u = (x >> 6) % QT, i = (x >> 6) / QT;
      const int col = n0 + 16 * u + (l & 15), s = s0 + i;
      if (col >= n || s >= strips) continue;
      f4 gv = {0.f, 0.f, 0.f, 0.f}, uv = gv;
#pragma unroll
      for (int z = 0; z < WAVES; ++z) {
        const f4 ga = sums[((z * SP + 2 * i) * QT + u) * 64 + l], ua = sums[((z * SP + 2 * i + 1) * QT + u) * 64 + l];
#pragma unroll
        for (int y = 0; y < 4; ++y) gv[y] += ga[y], uv[y] += ua[y];
      }
      const uint8_t* top0 = p.w1 + geo.e_off + ((int64_t)e * 2 * strips + s) * 16 + 4 * (l >> 4);
      const int pair = R != 0 ? own : r->list[first + col];
      const float weight = R != 0 ? own_weight : r->weight[pair];
      b4v hi, lo;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float gate = ldexpf(gv[y], (int)top0[y] - 127 - H_UP);
        const float h = weight * (moe_act(gate, p.act) * ldexpf(uv[y], (int)top0[16 * strips + y] - 127 - H_UP));
        hi[y] = (__bf16)h;
        const float rest = h - (float)hi[y];
        lo[y] = (__bf16)(abs_bits((float)hi[y]) >= F32_INF ? 0.f : rest);
      }
      const int k = 16 * s + 4 * (l >> 4), place = R != 0 ? a : first + col;
      int64_t at = (int64_t)pair * p.I + k, rest_at = (int64_t)p.T * p.top * p.I;
      if (p.grouped) {
        at = h_group(place, k >> 7, p.I) + (k >> 3 & 3) * 512 + ((k >> 5 & 3) * 16 + (place & 15)) * 8 + (k & 4);
        rest_at = H_GROUP / 2;
      }
      *reinterpret_cast<u2*>(p.h + at) = __builtin_bit_cast(u2, hi);
      *reinterpret_cast<u2*>(p.h + at + rest_at) = __builtin_bit_cast(u2, lo);
    }
  }
}

// eight weights as bfloat16 (exact: two bits of mantissa, any power of two)
__device__ __forceinline__ b8v fp4_b8(uint32_t w, float scale) {
  const b2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const b2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const b2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const b2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return b8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// a lane's 32 elements of h, hi and lo, in a k tile
struct HFrag {
  b8v hi[4], lo[4];
};
__device__ __forceinline__ f4 down_product(const u4 w, uint32_t byte, const HFrag& f, f4 d) {
  const float s = e8m0(byte);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const b8v b = fp4_b8(w[x], s);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, f.hi[x], d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, f.lo[x], d, 0, 0, 0);
  }
  return d;
}

// A few tokens whose h fits in LDS: the tokens are the columns, a block takes every
// expert in use for its strip and a token's sum over them stays in its registers.
__global__ __launch_bounds__(MOE_THREADS) void k_moe_down_tokens(const MoeParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];     // h, then 16 bytes of zeros
  __shared__ f4 sums[MOE_WAVES][64];
  __shared__ int16_t column[MOE_COLS * W4_MOE_MAX_TOP][MOE_COLS];
  const MoeRoute& r = *p.route;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int strips = p.H / 16, strip = block_number();
  if (strip >= strips) return;
  const MxGeometry geo = mx_geometry((int64_t)p.E * p.H, p.I);
  // a unit: expert in use, k tile
  const int active = __builtin_amdgcn_readfirstlane(r.active), units = active * geo.KT;
  const int end = (int)((int64_t)units * (wave + 1) / MOE_WAVES);
  int unit = (int)((int64_t)units * wave / MOE_WAVES);
  constexpr int U = 8;
  u4 w[U];
  uint32_t s[U];
  auto weights = [&] {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (unit + j >= end) break;
      const int ex = (unit + j) / geo.KT, kt = unit + j - ex * geo.KT;
      const int64_t t = (int64_t)__builtin_amdgcn_readfirstlane(r.expert[ex]) * strips + strip;
      w[j] = g_load<u4>(p.w2 + (t * geo.KT + kt) * TILE_BYTES, 16 * lane);
      s[j] = g_load<uint8_t>(p.w2 + geo.s_off + (t * geo.KQ + (kt >> 2)) * 256 + (kt & 3), 4 * lane);
    }
  };
  weights();                                             // on their way while h comes to LDS
  const int plane = p.T * p.top * p.I * 2;               // bytes
  for (int i = threadIdx.x; i < plane / 8; i += MOE_THREADS)
    reinterpret_cast<u4*>(smem)[i] = reinterpret_cast<const u4*>(p.h)[i];
  if (threadIdx.x == 0) *reinterpret_cast<u4*>(smem + 2 * plane) = u4{0u, 0u, 0u, 0u};
  for (int i = threadIdx.x; i < active * MOE_COLS / 2; i += MOE_THREADS)
    reinterpret_cast<uint32_t*>(column)[i] = reinterpret_cast<const uint32_t*>(r.column)[i];
  __syncthreads();
  f4 acc = {0.f, 0.f, 0.f, 0.f};
  while (unit < end) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (unit + j >= end) break;
      const int ex = (unit + j) / geo.KT, k = 128 * (unit + j - ex * geo.KT) + 32 * g;
      const int pair = column[ex][c];
      const bool in = pair >= 0 && k < p.I;
      const int at = (pair * p.I + k) * 2;
      HFrag f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        f.hi[x] = *reinterpret_cast<const b8v*>(smem + (in ? at + 16 * x : 2 * plane));
        f.lo[x] = *reinterpret_cast<const b8v*>(smem + (in ? at + plane + 16 * x : 2 * plane));
      }
      const f4 d = down_product(w[j], s[j], f, acc);
      // a token that did not choose the expert takes nothing, NaN weights neither
#pragma unroll
      for (int y = 0; y < 4; ++y) acc[y] = pair >= 0 ? d[y] : acc[y];
    }
    unit += U;
    weights();
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave > 0 || c >= p.T) return;
  const float nan = __uint_as_float(0x7FC00000u);
  f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int z = 0; z < MOE_WAVES; ++z)
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] += sums[z][lane][y];
  h4 o;
#pragma unroll
  for (int y = 0; y < 4; ++y) o[y] = (_Float16)(r.bad[c] ? nan : v[y]);
  *reinterpret_cast<u2*>(p.out + (int64_t)c * p.H + 16 * strip + 4 * g) = __builtin_bit_cast(u2, o);
}

// SP strips of one expert for its pairs, 16 of them at a time; the last block of a
// group of strips sums each token's pairs, in the order of its choices.
// Four blocks of four waves a CU (128 registers), a k tile's weights on their way while the one
// before is multiplied. us at 16 tokens on 64 experts of 1536 and 61 on 16 of 4320, with rows
// of h: 37.3 and 52, eight waves 45.7 and 49; two strips a block 46 and 60; now 38 and 44.
__global__ __launch_bounds__(64 * DOWN_WAVES, 4) void k_moe_down_pairs(const MoeParams p) {
  constexpr int SP = DOWN_SP, WAVES = DOWN_WAVES;
  __shared__ f4 sums[WAVES][SP][64];
  __shared__ unsigned slast;
  const MoeRoute& r = *p.route;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int strips = p.H / 16, groups = (strips + SP - 1) / SP;
  const int a = block_number() / groups, grp = block_number() - a * groups;
  const int active = r.active;
  if (a > 0 && a >= active) return;
  const bool empty = active == 0;                        // no token chose: the rows are 0
  if (!empty) {
    const int first = __builtin_amdgcn_readfirstlane(r.first[a]);
    const int n = __builtin_amdgcn_readfirstlane(r.first[a + 1]) - first;
    const MxGeometry geo = mx_geometry((int64_t)p.E * p.H, p.I);
    const int64_t t = (int64_t)__builtin_amdgcn_readfirstlane(r.expert[a]) * strips + grp * SP;
    const uint8_t *wt[SP], *ws[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      const int64_t ti = t + min(i, strips - 1 - grp * SP);
      wt[i] = p.w2 + ti * geo.KT * TILE_BYTES;
      ws[i] = p.w2 + geo.s_off + ti * geo.KQ * 256;
    }
    const int end = geo.KT * (wave + 1) / WAVES;
    const int kt_step = p.grouped ? H_GROUP : 128, x_step = p.grouped ? 512 : 8;
    const int lo_step = p.grouped ? H_GROUP / 2 : p.T * p.top * p.I;
    for (int n0 = 0; n0 < n; n0 += 16) {
      // this lane's h: columns past n take the last one's again, nobody takes theirs
      const int place = first + min(n0 + c, n - 1);
      const uint32_t own = p.grouped ? 2 * (uint32_t)(h_group(place, 0, p.I) + (16 * g + (place & 15)) * 8)
                                     : 2 * (uint32_t)(r.list[place] * p.I + 32 * g);
      f4 acc[SP];
#pragma unroll
      for (int i = 0; i < SP; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
      u4 w[SP];
      uint32_t s[SP];
      auto weights = [&](int kt) {
#pragma unroll
        for (int i = 0; i < SP; ++i) {
          w[i] = g_load<u4>(wt[i] + (int64_t)kt * TILE_BYTES, 16 * lane);
          s[i] = g_load<uint8_t>(ws[i] + (kt >> 2) * 256 + (kt & 3), 4 * lane);
        }
      };
      int kt = geo.KT * wave / WAVES;
      if (kt < end) weights(kt);
      for (; kt < end; ++kt) {
        HFrag f;
        const int k = 128 * kt + 32 * g;
        const bool in = k < p.I;
        const uint32_t at = in ? own : 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          f.hi[x] = g_load<b8v>(p.h + (kt * kt_step + x * x_step), at);
          f.lo[x] = g_load<b8v>(p.h + (kt * kt_step + x * x_step + lo_step), at);
        }
        if (128 * kt + 128 > p.I) {                      // the weights there are zeros, h may be a NaN
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            f.hi[x] = in ? f.hi[x] : b8v{};
            f.lo[x] = in ? f.lo[x] : b8v{};
          }
        }
        u4 v[SP];
        uint32_t sv[SP];
#pragma unroll
        for (int i = 0; i < SP; ++i) v[i] = w[i], sv[i] = s[i];
        if (kt + 1 < end) weights(kt + 1);
#pragma unroll
        for (int i = 0; i < SP; ++i) acc[i] = down_product(v[i], sv[i], f, acc[i]);
      }
      if (n0 > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < SP; ++i) sums[wave][i][lane] = acc[i];
      __syncthreads();
      for (int x = threadIdx.x; x < SP * 64; x += 64 * WAVES) {
        const int l = x & 63, i = x >> 6, col = n0 + (l & 15), strip = grp * SP + i;
        if (col >= n || strip >= strips) continue;
        f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int z = 0; z < WAVES; ++z)
#pragma unroll
          for (int y = 0; y < 4; ++y) v[y] += sums[z][i][l][y];
        uint32_t* y = reinterpret_cast<uint32_t*>(p.y) + (int64_t)r.list[first + col] * p.H + 16 * strip + 4 * (l >> 4);
        dev_store2(y, __float_as_uint(v[0]), __float_as_uint(v[1]));
        dev_store2(y + 2, __float_as_uint(v[2]), __float_as_uint(v[3]));
      }
    }
    stores_done();
    __syncthreads();
    if (threadIdx.x == 0) slast = dev_arrive(p.counters + grp) == (unsigned)(active - 1);
    __syncthreads();
    if (!slast) return;
    if (threadIdx.x == 0) dev_store(p.counters + grp, 0u);
  }
  const float nan = __uint_as_float(0x7FC00000u);
  // Four pieces of four choices' loads together: each is a round trip to the level that
  // all XCDs share.
  constexpr int PIECES = 4, STEP = 64 * WAVES;
  const int pieces = p.T * SP * 4;
  for (int x0 = threadIdx.x; x0 < pieces; x0 += PIECES * STEP) {
    f4 v[PIECES];
#pragma unroll
    for (int q = 0; q < PIECES; ++q) v[q] = f4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < (empty ? 0 : p.top); j0 += 4) {
      uint64_t lo[PIECES][4], hi[PIECES][4];
      float weight[PIECES][4];
#pragma unroll
      for (int q = 0; q < PIECES; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int x = x0 + q * STEP, tok = x / (SP * 4), col = 16 * SP * grp + 4 * (x % (SP * 4));
          weight[q][j] = -1.f;
          if (x >= pieces || j0 + j >= p.top || col >= p.H) continue;
          const uint32_t* y = reinterpret_cast<const uint32_t*>(p.y) + (int64_t)(tok * p.top + j0 + j) * p.H + col;
          weight[q][j] = r.weight[tok * p.top + j0 + j];
          lo[q][j] = dev_load2(y), hi[q][j] = dev_load2(y + 2);
        }
#pragma unroll
      for (int q = 0; q < PIECES; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (weight[q][j] >= 0.f) {
            v[q][0] += __uint_as_float((uint32_t)lo[q][j]), v[q][1] += __uint_as_float((uint32_t)(lo[q][j] >> 32));
            v[q][2] += __uint_as_float((uint32_t)hi[q][j]), v[q][3] += __uint_as_float((uint32_t)(hi[q][j] >> 32));
          }
    }
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int x = x0 + q * STEP, tok = x / (SP * 4), col = 16 * SP * grp + 4 * (x % (SP * 4));
      if (x >= pieces || col >= p.H) continue;
      h4 o;
#pragma unroll
      for (int y = 0; y < 4; ++y) o[y] = (_Float16)(r.bad[tok] ? nan : v[q][y]);
      *reinterpret_cast<u2*>(p.out + (int64_t)tok * p.H + col) = __builtin_bit_cast(u2, o);
    }
  }
}

static bool moe_sizes_ok(int T, int H, int I, int E, int top) {
  return T >= 0 && T <= W4_MOE_MAX_TOKENS && E >= 1 && E <= W4_MOE_MAX_EXPERTS && top >= 1 &&
         top <= W4_MOE_MAX_TOP && top <= E && H >= 32 && H % 32 == 0 && H <= W4_MAX_K && I >= 32 &&
         I % 32 == 0 && I <= W4_MAX_K;
}
// tokens as columns, nothing to join: where a strip a block gives the CUs work and h
// (4 bytes an element) fits in LDS
constexpr int MOE_H_LDS = 64 * 1024, MOE_X_LDS = 32 * 1024;
static bool moe_columns(int T, int H, int I, int top) {
  return T <= MOE_COLS && H >= 128 * 16 && (int64_t)T * top * I * 4 <= MOE_H_LDS;
}

// h grouped: where an expert has more than 4 pairs in the mean (16 tokens on 64 experts of
// 1536, one pair each: 37 us in rows, 40 grouped; 61 on 16 of 4320: 53 and 45)
static bool moe_grouped(int T, int H, int I, int E, int top) {
  return !moe_columns(T, H, I, top) && T * top > 4 * E;
}

struct MoeSpace {
  int64_t h, y, total;
};
static MoeSpace moe_space(int T, int H, int I, int E, int top) {
  MoeSpace s;
  s.h = WS_COUNTERS + (int64_t)((sizeof(MoeRoute) + 255) / 256 * 256);
  s.y = s.h + (moe_grouped(T, H, I, E, top) ? h_group(T * top + 15, 0, I) * 2 : (int64_t)T * top * I * 4);
  s.total = s.y + (moe_columns(T, H, I, top) ? 0 : (int64_t)T * top * H * 4);
  return s;
}

template <int P, int QT, int R, int WAVES>
int launch_up_r(const MoeParams& p, int64_t experts, hipStream_t stream) {
  const int lds = WAVES * 2 * P * QT * 1024 + (R != 0 ? p.H * 2 + 16 : 0);
  allow_smem((const void*)&k_moe_up<P, QT, R, WAVES>, R != 0 ? 80 * 1024 : lds);
  hipLaunchKernelGGL((k_moe_up<P, QT, R, WAVES>), grid_of(experts * ((p.I / 16 + P - 1) / P)), dim3(64 * WAVES),
                     lds, stream, p);
  return launch_status();
}
template <int P>
int launch_up(const MoeParams& p, bool in, int64_t experts, hipStream_t stream) {
  if (in)
    return p.E <= 64    ? launch_up_r<P, 1, 1, 8>(p, experts, stream)
           : p.E <= 128 ? launch_up_r<P, 1, 2, 8>(p, experts, stream)
                        : launch_up_r<P, 1, 8, 8>(p, experts, stream);
  // four waves a block (16 tokens on 64 experts of 1536, hidden 4096: 57 us, 66 on eight);
  // two column operands where an expert has more than 12 pairs in the mean
  return p.T * p.top > 12 * p.E ? launch_up_r<P, 2, 0, 4>(p, experts, stream)
                                : launch_up_r<P, 1, 0, 4>(p, experts, stream);
}

}  // namespace w4

using namespace w4;

extern "C" size_t moe_mx4_workspace_bytes(int tokens, int hidden, int inner, int experts, int top_k) {
  if (!moe_sizes_ok(tokens, hidden, inner, experts, top_k) || tokens == 0) return 0;
  return (size_t)moe_space(tokens, hidden, inner, experts, top_k).total;
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
  const MoeSpace s = moe_space(tokens, hidden, inner, experts, top_k);
  if (!workspace || workspace_bytes < (size_t)s.total) return W4_ERR_WORKSPACE;
  uint8_t* ws = (uint8_t*)workspace;
  MoeParams p{};
  p.x = x, p.logits = logits, p.w1 = w_gate_up, p.w2 = w_down, p.out = out;
  p.counters = (uint32_t*)ws, p.route = (MoeRoute*)(ws + WS_COUNTERS);
  p.h = (__bf16*)(ws + s.h), p.y = (float*)(ws + s.y);
  p.T = tokens, p.H = hidden, p.I = inner, p.E = experts, p.top = top_k, p.act = act;
  p.grouped = moe_grouped(tokens, hidden, inner, experts, top_k);
  p.renorm = renormalize != 0, p.half_logits = logits_dtype == W4_IN_F16;

  const bool in = tokens == 1 && hidden * 2 <= MOE_X_LDS;
  if (!in) {
    if (experts <= 64) hipLaunchKernelGGL(k_moe_route<1>, dim3(1), dim3(ROUTE_THREADS), 0, stream, p);
    else if (experts <= 128) hipLaunchKernelGGL(k_moe_route<2>, dim3(1), dim3(ROUTE_THREADS), 0, stream, p);
    else hipLaunchKernelGGL(k_moe_route<8>, dim3(1), dim3(ROUTE_THREADS), 0, stream, p);
    if (const int st = launch_status()) return st;
  }
  const int64_t most = min(experts, tokens * top_k);     // experts in use, at most
  // pairs of strips a block where that leaves the CUs enough blocks (that case 57 us, 60
  // with one; one token on 4 experts 11.5 with one, 13 with two, before its choices were
  // taken without barriers)
  const int st = most * (inner / 16) > 1024 ? launch_up<2>(p, in, most, stream) : launch_up<1>(p, in, most, stream);
  if (st) return st;
  if (moe_columns(tokens, hidden, inner, top_k)) {
    const int lds = tokens * top_k * inner * 4 + 16;
    allow_smem((const void*)&k_moe_down_tokens, MOE_H_LDS + 16);
    hipLaunchKernelGGL(k_moe_down_tokens, grid_of(hidden / 16), dim3(MOE_THREADS), lds, stream, p);
  } else {
    hipLaunchKernelGGL(k_moe_down_pairs, grid_of(most * ((hidden / 16 + DOWN_SP - 1) / DOWN_SP)), dim3(64 * DOWN_WAVES), 0,
                       stream, p);
  }
  return launch_status();
}
