// Append of new keys and values to the paged 8-bit cache, with the position
// rotation of queries and keys on the way.
//
// The scale of a page and head covers all its tokens, so the unit of work is
// one (sequence, page, kv head) and one of three roles: the page's keys, its
// values, or the queries of the same tokens (the heads that share the kv
// head). A block finds the largest new magnitude, settles the page's scale,
// re-codes the page's earlier tokens only if the scale grew, and codes the new
// ones. The inputs are read twice (the second time from cache) instead of
// being held, which keeps every page size and head dim in one kernel.
// Bound: bytes (2 per element read, 1 written; queries 2 and 2).
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
  int roles;          // 3, or 2 without queries
};

// The new tokens of sequence b: first row, count, first position. False if
// there are none or the lengths do not fit (see the header).
__device__ __forceinline__ bool append_span(const AppendParams& p, int b, int& row, int& n,
                                            int& start) {
  row = b;
  n = 1;
  if (p.indptr) {
    row = p.indptr[b];
    const int end = p.indptr[b + 1];
    if (row < 0 || end <= row || end > p.tokens) return false;
    n = end - row;
  }
  const int len = p.kv_len[b];
  start = len - n;
  return n <= p.max_q && start >= 0 && len <= (int64_t)p.cols * p.page &&
         (p.rot == 0 || len <= p.rope_rows);
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

// A head's elements as units of work: in the half layout the rot/2 / VEC
// vectors of the first half, each with its partner in the second, then the
// vectors that do not turn; in the interleaved layout every vector by itself.
__device__ __forceinline__ int rope_units(int dim, int rot, int style, int vec) {
  return (dim - (style == W4_ROPE_HALF ? rot / 2 : 0)) / vec;
}

// Unit u of the head at x, turned by the table row cs: y0 at dim d0 and, if
// d1 >= 0, y1 at dim d1.
template <typename T, int VEC>
__device__ __forceinline__ void rotated(const T* x, const float* cs, int u, int rot, int style,
                                        float (&y0)[VEC], int& d0, float (&y1)[VEC], int& d1) {
#pragma clang fp contract(off)
  const int half = rot / 2;
  d0 = u * VEC;
  d1 = -1;
  if (style == W4_ROPE_HALF) {
    if (d0 < half) {
      d1 = d0 + half;
      float a[VEC], b[VEC], c[VEC], s[VEC];
      load_vec<T, VEC>(x + d0, a);
      load_vec<T, VEC>(x + d1, b);
      load_vec<float, VEC>(cs + d0, c);
      load_vec<float, VEC>(cs + half + d0, s);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        y0[e] = a[e] * c[e] - b[e] * s[e];
        y1[e] = b[e] * c[e] + a[e] * s[e];
      }
      return;
    }
    d0 += half;
    load_vec<T, VEC>(x + d0, y0);
    return;
  }
  load_vec<T, VEC>(x + d0, y0);
  if (d0 < rot) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float c = cs[(d0 + e) / 2], s = cs[half + (d0 + e) / 2];
      const float a = y0[e], b = y0[e + 1];
      y0[e] = a * c - b * s;
      y0[e + 1] = b * c + a * s;
    }
  }
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

// the codes of VEC elements, packed (0 where s is 0 or NaN)
template <int Q, int VEC>
__device__ __forceinline__ uint32_t codes_of(const float (&y)[VEC], float s) {
  if (!(s > 0.f)) return 0u;
  if constexpr (VEC == 4) return code4<Q>(y[0] / s, y[1] / s, y[2] / s, y[3] / s);
  else return code4<Q>(y[0] / s, y[1] / s, 0.f, 0.f);
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

// img_row: bytes of one dim's staged values (at least the new tokens of a page)
template <typename T, int Q, int VEC, int NT>
__global__ __launch_bounds__(NT) void k_rope_append(const AppendParams p, int img_row) {
  extern __shared__ __attribute__((aligned(16))) uint8_t img[];
  __shared__ uint32_t shm[NT / 64];
  int t = blockIdx.x;
  const int h = t % p.kv_heads;
  t /= p.kv_heads;
  const int role = t % p.roles;
  t /= p.roles;
  const int b = t / p.columns;
  const int j = t - b * p.columns;
  int row, n, start;
  if (!append_span(p, b, row, n, start)) return;
  const int P = p.page, D = p.dim, DP = p.dp;
  const int col = start / P + j;
  const int lo = max(start, col * P), hi = min(start + n, (col + 1) * P);   // new positions
  if (lo >= hi) return;
  const int cnt = hi - lo;
  row += lo - start;                            // token row of position lo
  const int tid = threadIdx.x;
  const float* cs = p.rot ? p.rope + (size_t)lo * p.rot : nullptr;

  if (role == 2) {                              // the queries of the heads on kv head h
    const int G = p.q_heads / p.kv_heads;
    const int nu = rope_units(D, p.rot, p.style, VEC);
    const int per = G * nu;                     // units of one token
    for (int i = tid; i < cnt * per; i += NT) {
      const int tok = i / per, rem = i - tok * per;
      const int g = rem / nu, u = rem - g * nu;
      const int hh = h * G + g;
      float y0[VEC], y1[VEC];
      int d0, d1;
      rotated<T, VEC>((const T*)p.q + (row + tok) * p.q_stride + (int64_t)hh * D,
                      cs + (size_t)tok * p.rot, u, p.rot, p.style, y0, d0, y1, d1);
      uint16_t* o = p.q_out + ((size_t)(row + tok) * p.q_heads + hh) * D;
      auto put = [&](int d, const float (&y)[VEC]) {
        if constexpr (VEC == 4)
          *reinterpret_cast<u2*>(o + d) = __builtin_bit_cast(
              u2, h4{(_Float16)y[0], (_Float16)y[1], (_Float16)y[2], (_Float16)y[3]});
        else
          *reinterpret_cast<h2*>(o + d) = h2{(_Float16)y[0], (_Float16)y[1]};
      };
      put(d0, y0);
      if (d1 >= 0) put(d1, y1);
    }
    return;
  }

  const int id = p.table[(size_t)b * p.cols + col];
  if (id < 0 || id >= p.pages) return;
  const bool keys = role == 0;
  const size_t ph = (size_t)id * p.kv_heads + h;
  float* sc = (keys ? p.ks : p.vs) + ph;
  uint8_t* codes = (keys ? p.kc : p.vc) + ph * P * DP;
  const T* src = keys ? (const T*)p.k + row * p.k_stride + (int64_t)h * D
                      : (const T*)p.v + row * p.v_stride + (int64_t)h * D;
  const int64_t stride = keys ? p.k_stride : p.v_stride;
  const int rot = keys ? p.rot : 0;
  const int nu = rope_units(D, rot, p.style, VEC);
  const int lead = lo - col * P;                // earlier tokens of the page
  const float old = lead > 0 ? *sc : 0.f;

  // ---- the page's scale -----------------------------------------------------
  uint32_t mx = 0;
  for (int i = tid; i < cnt * nu; i += NT) {
    const int tok = i / nu;
    float y0[VEC], y1[VEC];
    int d0, d1;
    rotated<T, VEC>(src + tok * stride, cs + (size_t)tok * p.rot, i - tok * nu, rot, p.style, y0,
                    d0, y1, d1);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      mx = max(mx, abs_bits(y0[e]));
      if (d1 >= 0) mx = max(mx, abs_bits(y1[e]));
    }
  }
  mx = wave_max_u(mx);
  if constexpr (NT > 64) {
    if ((tid & 63) == 0) shm[tid >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) mx = max(mx, shm[i]);
  }
  // max of magnitudes by their bits: a NaN of either side wins
  const float s = __uint_as_float(max(__float_as_uint(scale_for<Q>(mx)), abs_bits(old)));
  if (tid == 0) *sc = s;
  const bool grown = lead > 0 && old < s;       // false if either is NaN
  const float ratio = grown ? old / s : 1.f;

  if (keys) {
    // earlier slots, the new ones, their padding, and a begun page's rest
    if (grown) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int i = tid; i < lead * (DP / 4); i += NT) w[i] = recoded<Q>(w[i], ratio);
    }
    uint8_t* dst = codes + (size_t)lead * DP;
    for (int i = tid; i < cnt * nu; i += NT) {
      const int tok = i / nu;
      float y0[VEC], y1[VEC];
      int d0, d1;
      rotated<T, VEC>(src + tok * stride, cs + (size_t)tok * p.rot, i - tok * nu, rot, p.style, y0,
                      d0, y1, d1);
      put_codes<VEC>(dst + tok * DP + d0, codes_of<Q, VEC>(y0, s));
      if (d1 >= 0) put_codes<VEC>(dst + tok * DP + d1, codes_of<Q, VEC>(y1, s));
    }
    const int pad = (DP - D) / 4;
    for (int i = tid; i < cnt * pad; i += NT) {
      const int tok = i / pad;
      *reinterpret_cast<uint32_t*>(dst + tok * DP + D + 4 * (i - tok * pad)) = 0u;
    }
    if (lead == 0) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes + (size_t)cnt * DP);
      for (int i = tid; i < (P - cnt) * (DP / 4); i += NT) w[i] = 0u;
    }
    return;
  }

  // ---- values: codes staged as [dim][new token], written as rows of slots -----
  for (int i = tid; i < cnt * nu; i += NT) {
    const int tok = i / nu, d = (i - tok * nu) * VEC;
    float y[VEC];
    load_vec<T, VEC>(src + tok * stride + d, y);
    const uint32_t w = codes_of<Q, VEC>(y, s);
#pragma unroll
    for (int e = 0; e < VEC; ++e) img[(d + e) * img_row + tok] = (uint8_t)(w >> (8 * e));
  }
  __syncthreads();
  // words of four slots that change: every word of a begun page, otherwise
  // those up to the last new token, from the first one if the scale grew
  const int w0 = lead == 0 || grown ? 0 : lead / 4;
  const int w1 = lead == 0 ? P / 4 : (lead + cnt + 3) / 4;
  const int nw = w1 - w0;
  for (int i = tid; i < DP * nw; i += NT) {
    const int d = i / nw, slot = 4 * (w0 + i - d * nw);
    uint32_t* dst = reinterpret_cast<uint32_t*>(codes + (size_t)d * P + slot);
    uint32_t w = 0;
    if (lead > 0) {
      w = *dst;
      if (grown) {
        const uint32_t r = recoded<Q>(w, ratio);
        // slots from `lead` on are not earlier tokens: left as they are
        const int before = min(max(lead - slot, 0), 4);
        const uint32_t m = before == 4 ? 0xFFFFFFFFu : (1u << (8 * before)) - 1u;
        w = (r & m) | (w & ~m);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = slot + e - lead;
      if (tok >= 0 && tok < cnt) {
        const uint32_t c = d < D ? img[d * img_row + tok] : 0u;
        w = (w & ~(0xFFu << (8 * e))) | (c << (8 * e));
      }
    }
    *dst = w;
  }
}

template <typename T, int Q>
int launch_append(const AppendParams& p, hipStream_t stream) {
  const int64_t blocks = (int64_t)p.batch * p.columns * p.roles * p.kv_heads;
  if (blocks > 0x7fffff) return W4_ERR_SHAPE;    // 2^31 threads
  // vectors of four lie on one side of every pair: half layout rot/2 a
  // multiple of 4 (rot is a multiple of 4 in either layout)
  const bool v4 = p.style == W4_ROPE_INTERLEAVED || p.rot % 8 == 0;
  const int img_row = (min(p.page, p.max_q) + 3) / 4 * 4 + 4;
  const size_t lds = (size_t)p.dp * img_row;
  const bool one = p.max_q == 1;
#define W4_AP(VEC, NT)                                                                             \
  hipLaunchKernelGGL((k_rope_append<T, Q, VEC, NT>), dim3((unsigned)blocks), dim3(NT), lds, stream, \
                     p, img_row)
  if (one) {
    if (v4) W4_AP(4, 64);
    else W4_AP(2, 64);
  } else {
    if (v4) W4_AP(4, 256);
    else W4_AP(2, 256);
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
  p.columns = (p.max_q + page_size - 2) / page_size + 1;
  p.roles = q ? 3 : 2;
  if (in_dtype == W4_IN_F16)
    return q_dtype == W4_Q_I8 ? launch_append<uint16_t, W4_Q_I8>(p, stream)
                              : launch_append<uint16_t, W4_Q_F8>(p, stream);
  return q_dtype == W4_Q_I8 ? launch_append<float, W4_Q_I8>(p, stream)
                            : launch_append<float, W4_Q_F8>(p, stream);
}
