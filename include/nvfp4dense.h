/*
 * nvfp4dense.h -- C ABI of the dense feed-forward operators for NVIDIA B200
 * (sm_100a), library libnvfp4dense.so: MXFP4 quantisation, products with MXFP4
 * weights (W4A16 and W4A4), and the gated feed-forward block with its backward
 * pass.  They serve, quantise and train the MLP that a layer runs next to its
 * routed experts (nvfp4moe.h).
 *
 * MXFP4 (OCP Microscaling Formats, "MXFP4"): E2M1 codes, one E8M0 scale per 32
 * consecutive elements along K,
 *   codes   u8 [R, 16 ceil(K/32)]  element 2j in the low nibble of byte j;
 *                                  codes past K are zero
 *   scales  u8 [R, ceil(K/32)]     value 2^(byte - 127); 255 = NaN
 * and the value of an element is E2M1(code) * 2^(byte - 127).
 *
 * Conventions: those of nvfp4moe.h.  Status codes are its nvfp4_status.
 * Pointers are device pointers, 16-byte aligned (workspaces 256-byte), owned
 * by the caller; calls are asynchronous on `stream`; arguments are validated
 * on the host and an invalid call enqueues nothing; calls that share a
 * workspace must not overlap on the GPU.  Sizes of zero tokens or rows are
 * valid: nothing is read, and only outputs that do not depend on tokens are
 * written (weight gradients: zeros).  Row strides (ldx) are in elements: at
 * least the row length and, except in mxfp4_quantize, a multiple of 8.
 * A row's results do not depend on the values of other rows of the call, and two
 * equal calls give equal bits.
 */
#ifndef NVFP4DENSE_H
#define NVFP4DENSE_H

#include "nvfp4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4DENSE_ABI_VERSION 1

#if defined(__GNUC__)
#define NVFP4DENSE_API __attribute__((visibility("default")))
#else
#define NVFP4DENSE_API
#endif

/* element types */
#define NVFP4DENSE_BF16 0
#define NVFP4DENSE_F16 1
#define NVFP4DENSE_F32 2

/* activations: none, GELU in its tanh form, SiLU */
#define NVFP4DENSE_ACT_NONE 0
#define NVFP4DENSE_ACT_GELU_TANH 1
#define NVFP4DENSE_ACT_SILU 2

/* ---------------------------------------------------------------------------
 * mxfp4_quantize: x [rows, K] (bf16, f16 or f32; row stride ldx, any) -> codes,
 * scales.  Per block of 32: a = max|x|, X = clamp(floor(log2 a) - 2, -127, 127)
 * (a = 0: -127), scale byte X + 127, code = the E2M1 value nearest to x 2^-X,
 * ties to the even code, saturating at 6.  A block that holds a NaN or an
 * infinity gets scale 255 and codes 0, so that it reads as NaN.
 * x may be of any alignment its type has; rows off the 16-byte grid are read by the
 * aligned 16-byte pieces that hold their elements, so up to 14 bytes before and behind
 * a row too, whatever these hold.  rows <= 2^31 - 1, K < 2^24, rows * K < 2^40.
 * ------------------------------------------------------------------------- */
NVFP4DENSE_API nvfp4_status mxfp4_quantize(const void* x_dev, int32_t dtype, int64_t rows, int64_t K, int64_t ldx,
                                           uint8_t* codes_dev, uint8_t* scales_dev, void* stream);

/* mxfp4_dequantize: codes, scales -> out [rows, K] (f32 or bf16), exact except
 * that magnitudes of 2^128 and above are infinite. */
NVFP4DENSE_API nvfp4_status mxfp4_dequantize(const uint8_t* codes_dev, const uint8_t* scales_dev, int64_t rows,
                                             int64_t K, void* out_dev, int32_t dtype, void* stream);

/* An MXFP4 weight matrix [N, K]; K a multiple of 32, N of 8 (gated: of 16). */
typedef struct {
  const uint8_t* codes;   /* [N, K/2] */
  const uint8_t* scales;  /* [N, K/32] */
  int32_t N;              /* 8 <= N <= 2^18 */
  int32_t K;              /* 32 <= K <= 2^18 */
} mxfp4_weight;

/* ---------------------------------------------------------------------------
 * mxfp4_linear (W4A16): y = x W^T, bf16 x [T, K] and y, products of the exact
 * weight values (magnitudes of 2^128 and above, which mxfp4_quantize does not
 * write, are infinite) with fp32 accumulation, one rounding.  With an activation W
 * stacks N/2 gate rows over N/2 up rows and y [T, N/2] = act(x Wg^T) * (x Wu^T).
 * dtype: BF16.  T <= 2^20.
 * mxfp4_linear_a4 (W4A4): x (bf16 or f16, y alike) is first quantised as by
 * mxfp4_quantize; the E2M1 products are exact and summed in fp32.
 * The workspace queries return 0 for arguments the call would refuse; at 256
 * bytes the call uses no workspace and takes NULL.
 * ------------------------------------------------------------------------- */
NVFP4DENSE_API size_t mxfp4_linear_workspace_bytes(int32_t T, const mxfp4_weight* w, int32_t act);
NVFP4DENSE_API nvfp4_status mxfp4_linear(const void* x_dev, int32_t dtype, int64_t ldx, int32_t T,
                                         const mxfp4_weight* w, int32_t act, void* y_dev, void* ws_dev,
                                         size_t ws_bytes, void* stream);
NVFP4DENSE_API size_t mxfp4_linear_a4_workspace_bytes(int32_t T, const mxfp4_weight* w, int32_t act);
NVFP4DENSE_API nvfp4_status mxfp4_linear_a4(const void* x_dev, int32_t dtype, int64_t ldx, int32_t T,
                                            const mxfp4_weight* w, int32_t act, void* y_dev, void* ws_dev,
                                            size_t ws_bytes, void* stream);

/* The weights of a gated feed-forward block, bf16 or f16:
 * gate, up [I, H], down [H, I]; H and I multiples of 8, up to 2^18. */
typedef struct {
  const void* gate;
  const void* up;
  const void* down;
  int32_t H, I;
  int32_t act;    /* GELU_TANH or SILU */
  int32_t dtype;  /* BF16 or F16, of the weights and of every tensor below */
} gated_ffn_weights;

/* ---------------------------------------------------------------------------
 * gated_ffn_forward: g = x gate^T, u = x up^T, h = act(g) u, y = h down^T.
 *   x [T, H] (row stride ldx), y [T, H]
 *   saved gated_ffn_saved_bytes bytes, 256-byte aligned, for
 *         gated_ffn_backward (h in 16 bits, act(g) and u act'(g) in 24: 8 bytes
 *         per token and hidden unit, and padding: rows of 64, blocks of 32 x 16
 *         tokens x hidden units), or NULL
 * fp32 accumulation; h is rounded to the 16-bit type (without `saved`, at up to 4
 * tokens, or 16 with I <= 512 and T H I <= 140e6: kept as two of them).  T <= 2^20.
 * With `saved` the workspace is not used.
 * ------------------------------------------------------------------------- */
NVFP4DENSE_API size_t gated_ffn_saved_bytes(int32_t T, const gated_ffn_weights* f);
NVFP4DENSE_API size_t gated_ffn_forward_workspace_bytes(int32_t T, const gated_ffn_weights* f);
NVFP4DENSE_API nvfp4_status gated_ffn_forward(const void* x_dev, int64_t ldx, int32_t T, const gated_ffn_weights* f,
                                              void* y_dev, void* saved_dev, void* ws_dev, size_t ws_bytes,
                                              void* stream);

/* ---------------------------------------------------------------------------
 * gated_ffn_backward: the gradients of gated_ffn_forward for dy [T, H],
 *   dh = dy down, dg = dh u act'(g), du = dh act(g) (dg, du rounded to the
 *   16-bit type), dx = dg gate + du up, dgate = dg^T x, dup = du^T x,
 *   ddown = dy^T h,
 * with x and `saved` of that forward.  Any of dx [T, H], dgate, dup [I, H],
 * ddown [H, I] may be NULL (not computed); each is overwritten.
 * dy and x have row strides lddy, ldx.
 * ------------------------------------------------------------------------- */
NVFP4DENSE_API size_t gated_ffn_backward_workspace_bytes(int32_t T, const gated_ffn_weights* f);
NVFP4DENSE_API nvfp4_status gated_ffn_backward(const void* dy_dev, int64_t lddy, const void* x_dev, int64_t ldx,
                                               const void* saved_dev, int32_t T, const gated_ffn_weights* f,
                                               void* dx_dev, void* dgate_dev, void* dup_dev, void* ddown_dev,
                                               void* ws_dev, size_t ws_bytes, void* stream);

/* As their namesakes in nvfp4moe.h, for this library. */
NVFP4DENSE_API nvfp4_status nvfp4dense_get_device_status(void* stream);
NVFP4DENSE_API const char* nvfp4dense_last_cuda_error(void);
NVFP4DENSE_API int nvfp4dense_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4DENSE_H */
