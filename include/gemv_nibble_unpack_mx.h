/*
 * gemv_nibble_unpack_mx.h -- C ABI of the microscaled 4-bit floating point
 * operators (MI355X, gfx950): coding rows to MXFP4, products with MXFP4
 * weights, and a mixture-of-experts layer on them. Same library, status codes
 * and conventions as gemv_nibble_unpack.h (device pointers, caller-owned
 * buffers, asynchronous on `stream`, nothing allocated, nothing synchronised,
 * every argument checked before a launch); what differs is said here. M and N are
 * at most 2^30.
 *
 * The format (OCP microscaling, MXFP4)
 * ------------------------------------
 * A row of K elements (K a multiple of 32) is K/32 blocks. A block is 32 E2M1
 * codes (sign, two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6)
 * and one E8M0 scale byte s; an element is code * 2^(s - 127), and s = 255 makes
 * the block NaN.
 *   codes  uint8 [rows, K/2], element 2j in the low four bits of byte j
 *   scales uint8 [rows, K/32]
 * Any codes and scales may be given, not only those of quantize_mx4.
 */
#ifndef GEMV_NIBBLE_UNPACK_MX_H
#define GEMV_NIBBLE_UNPACK_MX_H

#include "gemv_nibble_unpack.h"

#ifdef __cplusplus
extern "C" {
#endif

/* the products, for mx4_workspace_bytes */
#define W4_MX_A16 0   /* mx4a16_gemm */
#define W4_MX_A8  1   /* mx4a8_gemm  */
#define W4_MX_A4  2   /* mx4a4_gemm  */

/* activations of moe_mx4 */
#define W4_ACT_SILU  0   /* g / (1 + exp(-g))                                          */
#define W4_ACT_GELU  1   /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2             */
#define W4_ACT_RELU2 2   /* max(g, 0)^2                                                */

#define W4_MOE_MAX_TOKENS  64
#define W4_MOE_MAX_EXPERTS 512
#define W4_MOE_MAX_TOP     16

/*
 * quantize_mx4 -- rows to MXFP4. For each block of 32:
 *   e = floor(log2 max|x|) - 2, at least -127; s = e + 127 (0 for a block of zeros);
 *   code = E2M1(x / 2^e): nearest, ties to the even code, magnitudes above 5 to 6,
 *   the sign kept (also of zeros). A block that holds a NaN or an infinity gets s = 255 and
 *   codes 0. x / 2^e is exact, so the codes do not depend on the arithmetic.
 *   X fp16 or float32 [rows,K] per in_dtype (W4_IN_F16, W4_IN_F32), 16-byte
 *   aligned; codes 16-byte aligned. rows = 0 returns W4_OK without a launch.
 * Serves both operands: weights (then prepack_mx4) and the rows of mx4a4_gemm.
 * Errors: W4_ERR_ARG (in_dtype), W4_ERR_SHAPE (K not a multiple of 32 in [32,
 * W4_MAX_K], rows negative), W4_ERR_NULL, W4_ERR_ALIGN, W4_ERR_HIP.
 */
int quantize_mx4(const void* X, int in_dtype, int rows, int K, uint8_t* codes, uint8_t* scales,
                 hipStream_t stream);

/*
 * dequantize_mx4 -- MXFP4 rows to fp16 (W4_OUT_F16; rounded once) or float32
 * (W4_OUT_F32; exact) [rows,K], 16-byte aligned; infinite past the type's range.
 * Errors as quantize_mx4.
 */
int dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int rows, int K, int out_dtype,
                   void* Y, hipStream_t stream);

/*
 * prepack_mx4 -- weights [N,K] (codes and scales as above) to the buffer Wp of
 * prepack_mx4_bytes(N, K) bytes that the products read: the codes in the order
 * in which the matrix cores take them, padded with zeros to 16 rows x 128 k,
 * then the scales in that order. Opaque, laid out once. A matrix of several
 * experts, [experts * N, K] with N a multiple of 16, is packed as one.
 * prepack_mx4_bytes gives 0 for sizes that are not served.
 * unprepack_mx4 is the inverse.
 */
size_t prepack_mx4_bytes(int N, int K);
int prepack_mx4(const uint8_t* codes, const uint8_t* scales, int N, int K, uint8_t* Wp,
                hipStream_t stream);
int unprepack_mx4(const uint8_t* Wp, int N, int K, uint8_t* codes, uint8_t* scales,
                  hipStream_t stream);

/*
 * mx4a16_gemm, mx4a8_gemm, mx4a4_gemm -- C[M,N] = A[M,K] x W[N,K]^T with MXFP4
 * weights (Wp from prepack_mx4) and float32 sums:
 *   mx4a16_gemm: A fp16 [M,K];
 *   mx4a8_gemm:  Aq E4M3 codes [M,K], a_scale float32 [M]: an element is code *
 *                a_scale (what add_rmsnorm_q8 with W4_Q_F8 and quantize_f8 write); the
 *                sum of code * W is a float32 number, which a_scale multiplies;
 *   mx4a4_gemm:  Aq, a_scales MXFP4 rows, uint8 [M,K/2] and [M,K/32].
 *   W4_OUT_F16: C = fp16(sum + bias[n]), bias fp16 [N] or NULL; W4_OUT_F32: C = sum
 *   (bias ignored). Other out_dtypes are refused.
 * 4-bit rows meet the weights in the matrix cores' own scaled products (exact
 * terms, float32 sums), and so do 8-bit rows for an fp16 result: there, the bits
 * of terms below 2^-13 of the largest of eight neighbours along k are dropped (8e-6 of the
 * result's norm on normal data, at worst 2^-10 of the sum of magnitudes; where that is
 * too much, W4_OUT_F32 keeps them). For a float32 result 8-bit rows, and fp16 rows
 * always, meet weights that are widened to fp16, counted from row n's largest scale: exact for blocks whose scale is at least 2^-35 of the
 * largest in their row of W, rounded to 2^-36 of the largest below that.
 * A block with scale 255 makes every sum that meets it NaN, as a NaN of A does for
 * its row, which an infinity makes infinite or NaN.
 * Every M is served (M = 0 returns W4_OK without a launch): few rows by a
 * kernel that streams the weights, more by a tiled product (of at most 2^22 tiles;
 * W4_ERR_SHAPE past that). A, Wp and C are 16-byte aligned, a_scale to 4 bytes, bias to
 * 2, a_scales lies at any address. The outputs overlap no input. Workspace: mx4_workspace_bytes(op, M, N, K) bytes (0 if
 * none is needed or an argument is invalid), the rules of w4_workspace_bytes.
 * Errors: W4_ERR_ARG (out_dtype), W4_ERR_SHAPE, W4_ERR_NULL, W4_ERR_ALIGN,
 * W4_ERR_WORKSPACE, W4_ERR_HIP.
 */
size_t mx4_workspace_bytes(int op, int M, int N, int K);
int mx4a16_gemm(const uint16_t* A, const uint8_t* Wp, const uint16_t* bias, void* C, int out_dtype,
                int M, int N, int K, void* workspace, size_t workspace_bytes, hipStream_t stream);
int mx4a8_gemm(const uint8_t* Aq, const float* a_scale, const uint8_t* Wp, const uint16_t* bias,
               void* C, int out_dtype, int M, int N, int K, void* workspace,
               size_t workspace_bytes, hipStream_t stream);
int mx4a4_gemm(const uint8_t* Aq, const uint8_t* a_scales, const uint8_t* Wp, const uint16_t* bias,
               void* C, int out_dtype, int M, int N, int K, void* workspace,
               size_t workspace_bytes, hipStream_t stream);

/*
 * moe_mx4 -- a mixture-of-experts layer for a few tokens, from the router's
 * logits to the sum over the chosen experts. For token t:
 *   the top_k largest of its logits are chosen, ties to the lowest expert;
 *   w_j = exp(l_j - max) / sum of these over the chosen (renormalize) or over
 *   all experts (renormalize 0);
 *   h_j = act(Wg x) * (Wu x) of expert j, out = sum_j w_j (Wd h_j), fp16.
 *   x fp16 [tokens, hidden]; logits float32 or fp16 [tokens, experts] per
 *   logits_dtype (W4_IN_F32, W4_IN_F16);
 *   w_gate_up: prepack_mx4 of [experts * 2 * inner, hidden], an expert's gate
 *   rows, then its up rows; w_down: of [experts * hidden, inner].
 *   act: W4_ACT_*.
 * Sums are float32 in an order that does not change from call to call. x meets
 * the weights as in mx4a16_gemm; w_j h_j is formed in float32 and kept as the sum of two
 * bfloat16 numbers for the second product (relative 2^-17), whose weights are
 * bfloat16 numbers, exact within that type's range.
 * An expert with logit -infinity is never chosen; a token whose logits are all
 * -infinity gets zeros, one that has a NaN or +infinity among them NaN. A NaN in
 * a token's x or in an expert's weights reaches the tokens that meet it.
 *   tokens 0 .. W4_MOE_MAX_TOKENS (0 returns W4_OK without a launch), experts to
 *   W4_MOE_MAX_EXPERTS, top_k to W4_MOE_MAX_TOP and at most experts, hidden and
 *   inner multiples of 32 up to W4_MAX_K. x and weights are 16-byte aligned, out 8;
 *   out may be x.
 *   Workspace: moe_mx4_workspace_bytes(...) bytes (0 for arguments that are not
 *   served), the rules of w4_workspace_bytes.
 * Errors: W4_ERR_ARG (logits_dtype, act), W4_ERR_SHAPE, W4_ERR_NULL,
 * W4_ERR_ALIGN, W4_ERR_WORKSPACE, W4_ERR_HIP.
 */
size_t moe_mx4_workspace_bytes(int tokens, int hidden, int inner, int experts, int top_k);
int moe_mx4(const uint16_t* x, const void* logits, int logits_dtype, int tokens, int hidden,
            int inner, int experts, int top_k, int renormalize, int act, const uint8_t* w_gate_up,
            const uint8_t* w_down, uint16_t* out, void* workspace, size_t workspace_bytes,
            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_NIBBLE_UNPACK_MX_H */
