// Append of new keys and values to the paged 8-bit cache, with the position
// rotation of queries and keys on the way.
//
// The scale of a page and head covers all its tokens, so a block takes the new
// tokens of one (sequence, page, kv head): it reads the keys and values into
// registers, finds the largest magnitudes, settles the page's two scales,
// re-codes the page's earlier tokens only where a scale grew, and writes the
// codes. Other blocks turn the queries of the same tokens (the heads that
// share the kv head). Bound: bytes (2 per element read, 1 written; queries 2
// and 2); what costs beside them is a block's chain of dependent reads (lengths,
// page number, scale), so the tokens are fetched beside that chain. Measured: a
// 2048-token prompt of 32 and 8 heads of 128 14.0 us (47 MB, 3.4 TB/s), ragged
// chunks of 3168 tokens with 32 and 32 heads of 100 in pages of 16 39.2 us (102
// MB, 2.6 TB/s: 8000 blocks with work of about 12 KB, as many without; half of
// the time the vector units are busy; 32.6 us repeated on the same tensors), one
// token of 16 sequences 5.4 us (latency; 6.9 with plain divisions of the block
// number). Keys and values in blocks
// apart, each read twice, took 20, 78 and 6.6 us; two or four heads a block 51
// and 56 us on the ragged chunks where one took 51.
//
// Rotation: a' = a cos - b sin, b' = b cos + a sin with every product and sum
// rounded (no contraction), so the codes do not depend on how a compiler
// fuses them.

#include "layer_common.hpp"

namespace w4 {

struct AppendParams {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float* rope;
  const int32_t *indptr, *kv_len, *table;
  uint8_t *kc, *vc;
  float *ks, *vs;
  uint16_t* q_out;
  int rope_rows, rot, style;
  int batch, tokens, max_q, cols;
  int q_heads, kv_heads, dim, dp, page, pages;
  int columns;        // pages a sequence's new tokens can touch
  int q_span;         // kv heads whose queries one block turns
  int q_blocks;       // blocks of queries per page (0 without queries)
  uint32_t per_page_inv;   // floor_inv of blocks per page
};

// sequences of a launch, the y of its grid
constexpr int BATCH_Y = 65535;

// n / d for n below 2^32 with inv = floor(2^32 / d) (2^32 - 1 for d = 1): the high
// word of n * inv is the quotient or one less.
inline uint32_t floor_inv(uint32_t d) {
  return d == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / d);
}
__device__ __forceinline__ uint32_t div_inv(uint32_t n, uint32_t d, uint32_t inv) {
  const uint32_t q = __umulhi(n, inv);
  return q + (n - q * d >= d ? 1u : 0u);
}

// The new tokens of sequence b: first row, count, first position. False if
// there are none or the lengths do not fit (see the header).
__device__ __forceinline__ bool append_span(const AppendParams& p, int b, int& row, int& n,
                                            int& start) {
  const int len = p.kv_len[b];                  // read beside q_indptr
  row = b;
  n = 1;
  if (p.indptr) {
    row = p.indptr[b];
    n = p.indptr[b + 1] - row;
  }
  start = len - n;
  return row >= 0 && n > 0 && n <= p.tokens - row && n <= p.max_q && len >= n &&
         len <= (int64_t)p.cols * p.page && (p.rot == 0 || len <= p.rope_rows);
}

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&o)[VEC]) {
  if constexpr (VEC == 4) {
    const f4 t = load4f(p);
    o[0] = t[0], o[1] = t[1], o[2] = t[2], o[3] = t[3];
  } else {
    const f2v t = load2f(p);
    o[0] = t[0], o[1] = t[1];
  }
}

// A head's elements as units of two vectors: in the half layout a vector of
// the first half with its partner in the second, then the dims that do not
// turn, in pairs; in the interleaved layout all vectors, in pairs. An odd
// vector at the end stands alone (d1 < 0).
__host__ __device__ inline int rope_units(int dim, int rot, int style, int vec) {
  const int turned = style == W4_ROPE_HALF ? rot / 2 / vec : 0;
  return turned + ((dim - 2 * turned * vec) / vec + 1) / 2;
}
template <int VEC>
__device__ __forceinline__ void unit_dims(int u, int dim, int rot, int style, int& d0, int& d1) {
  const int half = style == W4_ROPE_HALF ? rot / 2 : 0;
  d0 = u * VEC;
  if (d0 < half) {
    d1 = d0 + half;
    return;
  }
  d0 += half;                                        // past the turned pairs
  d1 = d0 + ((dim - 2 * half) / VEC + 1) / 2 * VEC;
  if (d1 >= dim) d1 = -1;
}
template <int VEC>
struct Unit {
  float y0[VEC], y1[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Unit<VEC> load_unit(const T* x, int d0, int d1) {
  Unit<VEC> y;
  load_vec<T, VEC>(x + d0, y.y0);
  load_vec<T, VEC>(x + (d1 >= 0 ? d1 : d0), y.y1);   // alone: the same vector twice
  return y;
}
// the table's cosines and sines of a unit (row cs): of both vectors in the
// interleaved layout, of the pair in the half layout; 1 and 0 for dims that do
// not turn
template <int VEC>
struct Angle {
  float c[VEC], s[VEC];
};
template <int VEC>
__device__ __forceinline__ Angle<VEC> load_angle(const float* cs, int d0, int d1, int rot,
                                                 int style) {
  Angle<VEC> a;
  const int half = rot / 2;
  if (style == W4_ROPE_HALF) {
    const bool in = d0 < half;
    const float* t = cs + (in ? d0 : 0);
    if (rot) {
      load_vec<float, VEC>(t, a.c);
      load_vec<float, VEC>(t + half, a.s);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      a.c[e] = in ? a.c[e] : 1.f;
      a.s[e] = in ? a.s[e] : 0.f;
    }
    return a;
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {                 // pairs of y0, then pairs of y1
    // a vector turns as a whole or not at all (rot is a multiple of 4)
    const int d = v == 0 || d1 < 0 ? d0 : d1;
    const bool in = d < rot;
    const float* t = cs + (in ? d / 2 : 0);
    float c[VEC / 2], z[VEC / 2];
    if (rot) {
      if constexpr (VEC == 4) {
        load_vec<float, 2>(t, c);
        load_vec<float, 2>(t + half, z);
      } else {
        c[0] = t[0], z[0] = t[half];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      a.c[v * (VEC / 2) + e] = in ? c[e] : 1.f;
      a.s[v * (VEC / 2) + e] = in ? z[e] : 0.f;
    }
  }
  return a;
}
template <int VEC>
__device__ __forceinline__ void turn_unit(Unit<VEC>& y, const Angle<VEC>& t, bool half, int d0,
                                          int d1, int rot) {
#pragma clang fp contract(off)
  if (half) {
    if (d0 >= rot / 2) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float a = y.y0[e], b = y.y1[e];
      y.y0[e] = a * t.c[e] - b * t.s[e];
      y.y1[e] = b * t.c[e] + a * t.s[e];
    }
    return;
  }
  auto one = [&](float (&v)[VEC], int d, int from) {
    if (d >= rot) return;
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float c = t.c[from + e / 2], s = t.s[from + e / 2];
      const float a = v[e], b = v[e + 1];
      v[e] = a * c - b * s;
      v[e + 1] = b * c + a * s;
    }
  };
  one(y.y0, d0, 0);
  one(y.y1, d1 >= 0 ? d1 : d0, VEC / 2);
}

// the scale for a largest magnitude m (bits), see the header
template <int Q>
__device__ __forceinline__ float scale_for(uint32_t m) {
  if (m >= F32_INF) return __uint_as_float(0x7FC00000u);
  if (m == 0) return 0.f;
  if constexpr (Q == W4_Q_I8) {
    return __uint_as_float(m) / 127.0f;
  } else {
    // smallest power of two not below m / 448, at least 2^-126
    const uint32_t f = __float_as_uint(__uint_as_float(m) / 448.0f);
    const uint32_t e = max((f + 0x7FFFFFu) & 0x7F800000u, 0x00800000u);
    return __uint_as_float(e);
  }
}

// The codes of VEC elements, packed (0 where s is 0 or NaN). E4M3: r is the exact
// reciprocal of s, by which the product is the quotient bit for bit (ragged
// chunks 43.8 us divided, 40.9 so); 0, only where U > 2: there is none.
template <int Q, int U, int VEC>
__device__ __forceinline__ uint32_t codes_of(const float (&y)[VEC], float s, float r) {
  if (!(s > 0.f)) return 0u;
  if (Q == W4_Q_F8 && (U <= 2 || __builtin_expect(r != 0.f, 1))) {
    if constexpr (VEC == 4) return code4<Q>(y[0] * r, y[1] * r, y[2] * r, y[3] * r);
    else return code4<Q>(y[0] * r, y[1] * r, 0.f, 0.f);
  }
  if constexpr (VEC == 4) return code4<Q>(y[0] / s, y[1] / s, y[2] / s, y[3] / s);
  else return code4<Q>(y[0] / s, y[1] / s, 0.f, 0.f);
}
// The r of codes_of for a thread's E4M3 elements y. This kernel's own scales are
// powers of two from 2^-126 to 2^120, whose reciprocals are exact; a page that
// was filled elsewhere may have any. Threads of one or two units then divide them
// here, and go on with r = 1 (a branch at every codes_of: the ragged chunks, replayed,
// 35 us, this 31); more units cannot be held twice, r = 0 lets codes_of divide
// (the same chunks in pages of 128 61 us, 71 divided here).
template <int U, typename Units>
__device__ __forceinline__ float exact_reciprocal(Units& y, float s) {
  const uint32_t b = __builtin_amdgcn_readfirstlane(__float_as_uint(s));   // one value in a block
  if (__builtin_expect((b & 0x007FFFFFu) == 0 && b >= 0x00800000u && b < 0x7F000000u, 1))
    return __uint_as_float(0x7F000000u - b);           // 2^-e for 2^e
  if (U > 2) return 0.f;
  if (s > 0.f) {
#pragma unroll
    for (int z = 0; z < U; ++z) {
      for (float& e : y[z].y0) e /= s;
      for (float& e : y[z].y1) e /= s;
    }
  }
  return 1.f;
}
template <int VEC>
__device__ __forceinline__ void put_codes(uint8_t* p, uint32_t w) {
  if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = w;
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w;
}
template <int Q>
__device__ __forceinline__ uint32_t recoded(uint32_t w, float ratio) {
#pragma clang fp contract(off)
  const f4 f = decode4<Q>(w);
  return code4<Q>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// U: units a thread holds of a head's keys and of its values (a page's new
// tokens are at most U * NT units). img_row: bytes of one dim's staged values.
template <typename T, int Q, int VEC, int NT, int U>
__global__ __launch_bounds__(NT) void k_rope_append(const AppendParams p, int img_row) {
  extern __shared__ __attribute__((aligned(16))) uint8_t img[];
  __shared__ uint32_t shm[2][NT / 64];
  // along one page: a block for each kv head, then blocks of q_span kv heads'
  // queries
  const int per_page = p.kv_heads + p.q_blocks;
  const int j = div_inv(blockIdx.x, per_page, p.per_page_inv);
  const int which = blockIdx.x - j * per_page;
  const int b = blockIdx.y;
  int row, n, start;
  if (!append_span(p, b, row, n, start)) return;
  const int P = p.page, D = p.dim, DP = p.dp;
  const int col = (start >> __builtin_ctz(P)) + j;
  const int lo = max(start, col * P), hi = min(start + n, (col + 1) * P);   // new positions
  if (lo >= hi) return;
  const int cnt = hi - lo;
  row += lo - start;                            // token row of position lo
  const int tid = threadIdx.x;
  const float* cs = p.rot ? p.rope + (size_t)lo * p.rot : nullptr;
  const int nu = rope_units(D, p.rot, p.style, VEC);

  const bool half = p.style == W4_ROPE_HALF;
  if (which >= p.kv_heads) {                    // queries
    const int group = p.q_heads / p.kv_heads;
    const int first = (which - p.kv_heads) * p.q_span * group;
    const int per = min(p.q_span * group, p.q_heads - first) * nu;   // units of one token
    const int all = cnt * per;
    const bool few = all < (1 << 20);           // small_div's range
    for (int i0 = tid; i0 < all; i0 += 2 * NT) {      // two at a time, read before either is stored
      Unit<VEC> y[2];
      int d0[2], d1[2];
      size_t at[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int i = min(i0 + z * NT, all - 1);
        const int tok = few ? small_div(i, per) : i / per;
        const int rem = i - tok * per, g = few ? small_div(rem, nu) : rem / nu;
        unit_dims<VEC>(rem - g * nu, D, p.rot, p.style, d0[z], d1[z]);
        y[z] = load_unit<T, VEC>((const T*)p.q + (row + tok) * p.q_stride + (int64_t)(first + g) * D,
                                 d0[z], d1[z]);
        const Angle<VEC> a = load_angle<VEC>(cs + (size_t)tok * p.rot, d0[z], d1[z], p.rot, p.style);
        turn_unit<VEC>(y[z], a, half, d0[z], d1[z], p.rot);
        at[z] = ((size_t)(row + tok) * p.q_heads + first + g) * D;
      }
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if (i0 + z * NT >= all) break;
        auto put = [&](int d, const float (&v)[VEC]) {
          uint16_t* o = p.q_out + at[z] + d;
          if constexpr (VEC == 4)
            *reinterpret_cast<u2*>(o) = __builtin_bit_cast(
                u2, h4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]});
          else
            *reinterpret_cast<h2*>(o) = h2{(_Float16)v[0], (_Float16)v[1]};
        };
        put(d0[z], y[z].y0);
        if (d1[z] >= 0) put(d1[z], y[z].y1);
      }
    }
    return;
  }

  const int h = which;
  // ---- the new keys and values ------------------------------------------------
  const int nv = rope_units(D, 0, W4_ROPE_INTERLEAVED, VEC);
  Unit<VEC> ky[U], vy[U];
  Angle<VEC> ang[U];
  // unit i = tid + z * NT of a head's keys: token, dims (threads past the end
  // repeat the last unit and store nothing)
  auto kunit = [&](int z, int& tok, int& d0, int& d1) {
    const int i = min(tid + z * NT, cnt * nu - 1);
    tok = small_div(i, nu);
    unit_dims<VEC>(i - tok * nu, D, p.rot, p.style, d0, d1);
    return tid + z * NT < cnt * nu;
  };
  auto vunit = [&](int z, int& tok, int& d0, int& d1) {
    const int i = min(tid + z * NT, cnt * nv - 1);
    tok = small_div(i, nv);
    unit_dims<VEC>(i - tok * nv, D, 0, W4_ROPE_INTERLEAVED, d0, d1);
    return tid + z * NT < cnt * nv;
  };
#pragma unroll
  for (int z = 0; z < U; ++z) {
    int kt, k0, k1, vt, v0, v1;
    kunit(z, kt, k0, k1);
    vunit(z, vt, v0, v1);
    ang[z] = load_angle<VEC>(cs + (size_t)kt * p.rot, k0, k1, p.rot, p.style);
    ky[z] = load_unit<T, VEC>((const T*)p.k + (row + kt) * p.k_stride + (int64_t)h * D, k0, k1);
    vy[z] = load_unit<T, VEC>((const T*)p.v + (row + vt) * p.v_stride + (int64_t)h * D, v0, v1);
  }
  // a page outside the pool: the block goes on without storing
  const int idt = p.table[(size_t)b * p.cols + col];
  const bool store = idt >= 0 && idt < p.pages;
  const int id = store ? idt : 0;
  const int lead = lo - col * P;                // earlier tokens of the page
  const size_t ph = (size_t)id * p.kv_heads + h;
  float kold = p.ks[ph], vold = p.vs[ph];

  // ---- the page's scales --------------------------------------------------------
  uint32_t km = 0, vm = 0;
#pragma unroll
  for (int z = 0; z < U; ++z) {
    int tok, d0, d1;
    kunit(z, tok, d0, d1);
    turn_unit<VEC>(ky[z], ang[z], half, d0, d1, p.rot);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      km = max(km, max(abs_bits(ky[z].y0[e]), abs_bits(ky[z].y1[e])));
      vm = max(vm, max(abs_bits(vy[z].y0[e]), abs_bits(vy[z].y1[e])));
    }
  }
  km = wave_max_u(km);
  vm = wave_max_u(vm);
  if constexpr (NT > 64) {
    if ((tid & 63) == 0) {
      shm[0][tid >> 6] = km;
      shm[1][tid >> 6] = vm;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      km = max(km, shm[0][i]);
      vm = max(vm, shm[1][i]);
    }
  }
  if (lead == 0) kold = vold = 0.f;
  // max of magnitudes by their bits: a NaN of either side wins
  const float ks = __uint_as_float(max(__float_as_uint(scale_for<Q>(km)), abs_bits(kold)));
  const float vs = __uint_as_float(max(__float_as_uint(scale_for<Q>(vm)), abs_bits(vold)));
  if (!store) return;
  if (tid == 0) {
    p.ks[ph] = ks;
    p.vs[ph] = vs;
  }

  const float kr = Q == W4_Q_F8 ? exact_reciprocal<U>(ky, ks) : 0.f;
  const float vr = Q == W4_Q_F8 ? exact_reciprocal<U>(vy, vs) : 0.f;

  // ---- keys: earlier slots, the new ones, their padding, a begun page's rest -----
  const int pad = (DP - D) / 4;
  {
    uint8_t* kc = p.kc + ph * P * DP;
    if (lead > 0 && kold < ks) {              // grown (false for NaN)
      const float ratio = kold / ks;
      uint32_t* w = reinterpret_cast<uint32_t*>(kc);
      for (int i = tid; i < lead * (DP / 4); i += NT) w[i] = recoded<Q>(w[i], ratio);
    }
    uint8_t* dst = kc + (size_t)lead * DP;
#pragma unroll
    for (int z = 0; z < U; ++z) {
      int tok, d0, d1;
      if (kunit(z, tok, d0, d1)) {
        put_codes<VEC>(dst + tok * DP + d0, codes_of<Q, U>(ky[z].y0, ks, kr));
        if (d1 >= 0) put_codes<VEC>(dst + tok * DP + d1, codes_of<Q, U>(ky[z].y1, ks, kr));
      }
      if (vunit(z, tok, d0, d1)) {                  // values, staged as [dim][new token]
        const uint32_t w0 = codes_of<Q, U>(vy[z].y0, vs, vr);
        const uint32_t w1 = codes_of<Q, U>(vy[z].y1, vs, vr);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          img[(d0 + e) * img_row + tok] = (uint8_t)(w0 >> (8 * e));
          if (d1 >= 0) img[(d1 + e) * img_row + tok] = (uint8_t)(w1 >> (8 * e));
        }
      }
    }
    for (int i = tid; i < cnt * pad; i += NT) {
      const int tok = small_div(i, pad);
      *reinterpret_cast<uint32_t*>(dst + tok * DP + D + 4 * (i - tok * pad)) = 0u;
    }
    if (lead == 0) {
      uint32_t* w = reinterpret_cast<uint32_t*>(kc + (size_t)cnt * DP);
      for (int i = tid; i < (P - cnt) * (DP / 4); i += NT) w[i] = 0u;
    }
  }
  __syncthreads();
  // ---- values: rows of slots --------------------------------------------------------
  {
    uint8_t* vc = p.vc + ph * P * DP;
    if (lead == 0) {
      // the whole page, 16 slots at a time; staged rows are words
      const int sh = __builtin_ctz(P) - 4;
      for (int i = tid; i < DP << sh; i += NT) {
        const int d = i >> sh, slot = 16 * (i - (d << sh));
        const uint32_t* src = reinterpret_cast<const uint32_t*>(img + d * img_row + slot);
        u4 w;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int left = min(max(cnt - slot - 4 * x, 0), 4);   // new tokens of the word
          w[x] = d >= D || left == 0 ? 0u
                                     : src[x] & (left == 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u);
        }
        *reinterpret_cast<u4*>(vc + (size_t)d * P + slot) = w;
      }
      return;
    }
    // words of four slots that change: those of the new tokens, from the first
    // one if the scale grew
    const bool grown = vold < vs;
    const float ratio = grown ? vold / vs : 1.f;
    const int w0 = grown ? 0 : lead / 4;
    const int nw = (lead + cnt + 3) / 4 - w0;
    for (int i = tid; i < DP * nw; i += NT) {
      const int d = small_div(i, nw), slot = 4 * (w0 + i - d * nw);
      uint32_t* at = reinterpret_cast<uint32_t*>(vc + (size_t)d * P + slot);
      uint32_t w = *at;
      if (grown) {
        const uint32_t r = recoded<Q>(w, ratio);
        // slots from `lead` on are not earlier tokens: left as they are
        const int before = min(max(lead - slot, 0), 4);
        const uint32_t m = before == 4 ? 0xFFFFFFFFu : (1u << (8 * before)) - 1u;
        w = (r & m) | (w & ~m);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = slot + e - lead;
        if (tok >= 0 && tok < cnt) {
          const uint32_t c = d < D ? img[d * img_row + tok] : 0u;
          w = (w & ~(0xFFu << (8 * e))) | (c << (8 * e));
        }
      }
      *at = w;
    }
  }
}

template <typename T, int Q>
int launch_append(AppendParams& p, hipStream_t stream) {
  // vectors of four lie on one side of every pair: half layout rot/2 a
  // multiple of 4 (rot is a multiple of 4 in either layout)
  const bool v4 = p.style == W4_ROPE_INTERLEAVED || p.rot % 8 == 0;
  const int slots = min(p.page, p.max_q);
  // bytes of a staged row: words, one more than the slots need, which keeps the
  // rows of neighbouring dims off one bank
  const int img_row = (slots + 3) / 4 * 4 + 4;
  const int vec = v4 ? 4 : 2;
  const int units = slots * max(rope_units(p.dim, p.rot, p.style, vec),
                                rope_units(p.dim, 0, W4_ROPE_INTERLEAVED, vec));
  const int64_t per_head = (int64_t)slots * (p.q_heads / p.kv_heads) *
                           rope_units(p.dim, p.rot, p.style, vec);
  // threads by the units of a page and head. 1024 units (64 slots of 128 dims):
  // 512 threads x 2 13.9 us on the 2048-token prompt, 256 x 4 16.0, 1024 x 1 17.7.
  // The 1024-thread forms (pages of 128, or of 64 with dims above 128) have 128 registers a
  // thread: fp16 in vectors of four fits, fp16 in pairs spills 25, float32 16
  // to 18, in pairs 53 to 58.
#define W4_AP(VEC, NT, U)                                                                       \
  do {                                                                                          \
    /* queries of as many kv heads as give each thread four units */                            \
    p.q_span = (int)max((int64_t)1, min((int64_t)p.kv_heads, 4 * NT / per_head));               \
    p.q_blocks = p.q ? (p.kv_heads + p.q_span - 1) / p.q_span : 0;                              \
    p.per_page_inv = floor_inv(p.kv_heads + p.q_blocks);                                        \
    const int64_t blocks = (int64_t)p.columns * (p.kv_heads + p.q_blocks);   /* a sequence */   \
    if (blocks * NT > 0x7fffffff) return W4_ERR_SHAPE;                                          \
    const dim3 grid((unsigned)blocks, p.batch);                                                 \
    hipLaunchKernelGGL((k_rope_append<T, Q, VEC, NT, U>), grid, dim3(NT),                       \
                       (size_t)p.dp * img_row + 16, stream, p, img_row);                        \
  } while (0)
  if (v4) {
    if (units <= 64) W4_AP(4, 64, 1);
    else if (units <= 256) W4_AP(4, 256, 1);
    else if (units <= 1024) W4_AP(4, 512, 2);
    else W4_AP(4, 1024, 4);
  } else {
    if (units <= 128) W4_AP(2, 64, 2);
    else if (units <= 512) W4_AP(2, 256, 2);
    else if (units <= 2048) W4_AP(2, 512, 4);
    else W4_AP(2, 1024, 8);
  }
#undef W4_AP
  return launch_status();
}

}  // namespace w4

using namespace w4;

extern "C" int kv8_padded_dim(int d) {
  if (d < 4 || d % 4 || d > W4_MAX_HEAD_DIM) return 0;
  return d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : d <= 192 ? 192 : 256;
}

extern "C" int rope_append_kv8(const void* q, const void* k, const void* v, int in_dtype,
                               int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               const float* rope, int rope_rows, int rot_dim, int rope_style,
                               const int32_t* q_indptr, const int32_t* kv_len,
                               const int32_t* page_table, int batch, int tokens, int max_q,
                               int table_cols, int q_heads, int kv_heads, int head_dim,
                               int page_size, int num_pages, int q_dtype, void* k_codes,
                               void* v_codes, float* k_scale, float* v_scale, uint16_t* q_out,
                               hipStream_t stream) {
  if (in_dtype != W4_IN_F16 && in_dtype != W4_IN_F32) return W4_ERR_ARG;
  if (q_dtype != W4_Q_I8 && q_dtype != W4_Q_F8) return W4_ERR_ARG;
  if (rope_style != W4_ROPE_HALF && rope_style != W4_ROPE_INTERLEAVED) return W4_ERR_ARG;
  const int dp = kv8_padded_dim(head_dim);
  if (batch < 0 || tokens < 0 || max_q < 0 || table_cols < 1 || kv_heads < 1 || q_heads < 1 ||
      q_heads % kv_heads || dp == 0 || !kv8_page_ok(page_size) || num_pages < 1 || rot_dim < 0 ||
      rot_dim % 4 || rot_dim > head_dim || (rot_dim > 0 && rope_rows < 1))
    return W4_ERR_SHAPE;
  if (k_stride < (int64_t)kv_heads * head_dim || v_stride < (int64_t)kv_heads * head_dim ||
      k_stride % 4 || v_stride % 4 ||
      (q && (q_stride < (int64_t)q_heads * head_dim || q_stride % 4)))
    return W4_ERR_SHAPE;
  if (!q_indptr && tokens != batch) return W4_ERR_SHAPE;
  if (batch == 0 || tokens == 0 || max_q == 0) return W4_OK;
  if (!k || !v || !kv_len || !page_table || !k_codes || !v_codes || !k_scale || !v_scale ||
      (q && !q_out) || (rot_dim && !rope))
    return W4_ERR_NULL;
  const size_t a = in_dtype == W4_IN_F16 ? 8 : 16;
  if (!aligned(q, a) || !aligned(k, a) || !aligned(v, a) || !aligned(q_out, 8) ||
      !aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(rope, 16) ||
      !aligned(q_indptr, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return W4_ERR_ALIGN;
  AppendParams p{};
  p.q = q, p.k = k, p.v = v;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
  p.rope = rope, p.rope_rows = rope_rows, p.rot = rot_dim, p.style = rope_style;
  p.indptr = q_indptr, p.kv_len = kv_len, p.table = page_table;
  p.kc = (uint8_t*)k_codes, p.vc = (uint8_t*)v_codes, p.ks = k_scale, p.vs = v_scale;
  p.q_out = q_out;
  p.batch = batch, p.tokens = tokens, p.max_q = min(max_q, tokens), p.cols = table_cols;
  p.q_heads = q_heads, p.kv_heads = kv_heads, p.dim = head_dim, p.dp = dp;
  p.page = page_size, p.pages = num_pages;
  p.columns = (int)(((int64_t)p.max_q + page_size - 2) / page_size + 1);
  const size_t e = in_dtype == W4_IN_F16 ? 2 : 4;
  for (int64_t b0 = 0; b0 < batch; b0 += BATCH_Y) {  // one launch, save for huge batches
    p.batch = (int)min(batch - b0, (int64_t)BATCH_Y);
    const int st = in_dtype == W4_IN_F16
                       ? (q_dtype == W4_Q_I8 ? launch_append<uint16_t, W4_Q_I8>(p, stream)
                                             : launch_append<uint16_t, W4_Q_F8>(p, stream))
                       : (q_dtype == W4_Q_I8 ? launch_append<float, W4_Q_I8>(p, stream)
                                             : launch_append<float, W4_Q_F8>(p, stream));
    if (st != W4_OK) return st;
    p.kv_len += p.batch;
    p.table += (int64_t)p.batch * p.cols;
    if (p.indptr) {
      p.indptr += p.batch;
      continue;
    }
    auto rows = [&](const void* x, int64_t stride) {
      return x ? (const uint8_t*)x + p.batch * stride * e : nullptr;
    };
    p.q = rows(p.q, q_stride), p.k = rows(p.k, k_stride), p.v = rows(p.v, v_stride);
    if (p.q_out) p.q_out += (int64_t)p.batch * q_heads * head_dim;
    p.tokens -= p.batch;
  }
  return W4_OK;
}
