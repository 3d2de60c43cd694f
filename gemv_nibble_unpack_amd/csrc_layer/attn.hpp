// Attention over the paged 8-bit cache: parameters and the pieces that the
// kernels share.
#pragma once

#include "layer_common.hpp"

namespace w4 {

struct AttnParams {
  const uint16_t* q;
  int64_t q_stride;
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  const int32_t *indptr, *kv_len, *table;
  uint16_t* out;
  float* lse;
  uint32_t* counters;       // split launches: arrivals per (sequence, head, row tile)
  float* part;              // split launches: partial results
  float scale_log2;         // |softmax scale| * log2(e)
  uint32_t q_sign;          // 0x80008000 if the softmax scale is negative: flips a pair of q's
  int batch, tokens, max_q, max_kv, cols;
  int q_heads, kv_heads, group, dim;
  int page_shift, pages;
  int tiles;                // row tiles (k_attn_many: blocks' worth of them) of max_q * group rows
  int chunk, splits;        // cached tokens per block (a multiple of 64), blocks along them
  int by_row;               // k_attn_many: how its parts are numbered (see part_slot)
};

constexpr int MANY_ROWS = 128;    // query rows of a tile of k_attn_many
constexpr bool many_pair(int dp) { return dp <= 128; }   // two tiles a block

// The place of the parts of (sequence b, kv head h, row tile or pair of tiles),
// counted in sets of `splits` parts. Numbered by unit there are batch * tiles *
// kv_heads of them. A ragged batch has far more tiles than work; numbered by
// row (`by_row`), a sequence's places start where its first row falls among
// all rows, cut into `tile` rows: it has at most ceil(n * group / tile) tiles, so
// with row0 + n <= tokens every place is below (tokens * group / tile + batch) *
// kv_heads, and sequences that follow each other do not meet. The plan takes
// the smaller of the two and the kernels number as it says.
__host__ __device__ __forceinline__ int64_t part_slot(bool by_row, int b, int h, int t, int row0,
                                                      int group, int tile, int tiles,
                                                      int kv_heads) {
  return by_row ? ((int64_t)row0 * group / tile + b + t) * kv_heads + h
                : ((int64_t)b * kv_heads + h) * tiles + t;
}
// workspace bytes of a set of parts: rows' outputs and the statistics (M, L), which
// k_attn_many keeps for every lane
constexpr int64_t part_bytes(bool many, int tile, int dp, int splits) {
  return (int64_t)splits * tile * (dp + (many ? 4 : 2)) * 4;
}

int launch_attn_many(const AttnParams& p, int dp, int kind, int64_t blocks, hipStream_t stream);

// Sequence b's query rows and cached length. False: no new tokens, or ones
// outside the inputs. `fits` false: the lengths contradict each other or the
// bounds; the rows get NaN.
__device__ __forceinline__ bool attn_span(const AttnParams& p, int b, int& row, int& n, int& len,
                                          bool& fits) {
  row = b;
  n = 1;
  if (p.indptr) {
    row = p.indptr[b];
    const int end = p.indptr[b + 1];
    if (row < 0 || end <= row || end > p.tokens) return false;
    n = end - row;
  }
  len = p.kv_len[b];
  fits = n <= p.max_q && len >= 0 && len <= p.max_kv &&
         len <= ((int64_t)p.cols << p.page_shift);
  return true;
}

// Four 8-bit codes as exact fp16 values.
//   INT8: code + 128 as the low byte of the fp16 number 1024 + u, minus 1152.
//   E4M3: the hardware conversion.
template <int Q>
__device__ __forceinline__ void widen4(uint32_t w, h2& lo, h2& hi) {
  if constexpr (Q == W4_Q_I8) {
    const uint32_t u = w ^ 0x80808080u;
    const h2 k = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    lo = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + k;
    hi = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + k;
  } else {
    lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
  }
}
template <int Q>
__device__ __forceinline__ h8 widen8(uint32_t w0, uint32_t w1) {
  h2 a, b, c, d;
  widen4<Q>(w0, a, b);
  widen4<Q>(w1, c, d);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// max / sum over the four 16-lane rows of a wave, left in every lane
__device__ __forceinline__ float rows_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float rows_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

}  // namespace w4
