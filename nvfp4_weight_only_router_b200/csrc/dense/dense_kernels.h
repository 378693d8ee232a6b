// Internal launch interface between the dense C ABI (api_dense.cu) and its
// kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../kernels.h"

namespace nvfp4moe {

// element types and activations, as in nvfp4dense.h
constexpr int kBf16 = 0, kF16 = 1, kF32 = 2;
constexpr int kActNone = 0, kActGelu = 1, kActSilu = 2;

constexpr int kMxBlock = 32;    // elements per E8M0 scale
constexpr int kSfChunkB = 512;  // block scales of 128 rows x 4 blocks in the tensor core's order

inline int64_t mx_blocks(int64_t K) { return (K + kMxBlock - 1) / kMxBlock; }
inline int64_t mx_pitch(int64_t K) { return mx_blocks(K) * (kMxBlock / 2); }
// 512-byte scale chunks along K: whole stages of 256 elements
inline int mx_sf_chunks(int K) { return (K + 255) / 256 * 2; }

// ------------------------------------------------------------ mxfp4_quant.cu
cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st);
cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* out,
                                    int dtype, cudaStream_t st);
// x [T, K] -> codes [T, K/2] and scale chunks; and the weight's row-major
// scales -> the chunks of each bn-row tile of the product (one launch)
struct MxPrepArgs {
  const void* x;
  int dtype;
  int T, K;
  int64_t ldx;
  uint8_t* xq;           // [T, K/2]
  uint8_t* xsf;          // [ceil(T/128)][chunks][512]
  const uint8_t* wscales;  // [N (gated: 2 N), K/32]
  int N;                 // output columns
  bool gated;            // a tile: bn/2 gate rows, then their bn/2 up rows
  int bn;
  uint8_t* wsf;          // [mx_wsf_blocks][chunks][512]
};
// 128-row scale blocks of the weight: ceil(bn/128) for each tile
inline int64_t mx_wsf_blocks(int N, bool gated, int bn) {
  const int tn = gated ? bn / 2 : bn;
  return (int64_t)((N + tn - 1) / tn) * ((bn + 127) / 128);
}
cudaError_t launch_mxfp4_prep_a4(const MxPrepArgs& a, cudaStream_t st);

// SMs of the current device, asked for once per device (148 where there is none:
// workspace queries answer without a GPU)
int sms();

// ---------------------------------------------------------------- skinny.cu
// whether launch_skinny is the faster kernel for an MXFP4 product (N: output
// columns), or for both products of a gated block
bool skinny_fits_mx(int T, int N, int K, bool gated, bool quant_x);
bool skinny_fits_ffn(int T, int H, int I);
bool skinny_splits_hidden(int T, int H, int I);
struct SkinnyArgs {
  const void* x;      // [T, K]
  int64_t ldx;        // elements
  const void* w0;     // 16-bit: [N, K] (gate); MXFP4: codes
  const void* w1;     // 16-bit gated: up [N, K]
  const uint8_t* scales;  // MXFP4
  void* y;            // [T, N]
  int T, N, K;        // N: output columns
  int act;            // kActNone: plain; else gated
  int dtype;          // of x and y
  bool mx;            // MXFP4 weights
  bool quant_x;       // x through MXFP4 first
  bool after_producer;  // x, and no weight, is written by the kernel launched just before on the stream
  // 16-bit weights: values kept as two, each rounded to 16 bits, the second of what
  // the first leaves.  T counts tokens; the second follows in a row of its own.
  bool split_x, split_y;  // plain: of x; gated: of y
};
cudaError_t launch_skinny(const SkinnyArgs& a, cudaStream_t st);

// ------------------------------------------------------------- pair_gemm.cu
// A stage of the operands of one product: A [M, K] and B [N, K] by pointer and
// row pitch in elements; *_mn: stored with K outermost ([K, M], [K, N]).
struct PairOperand {
  const void* p;
  int64_t ld;
  bool mn;
};
struct PairSegment {
  PairOperand a, b;
  int K;
};
struct PairGemm {
  PairSegment seg[2];
  int nseg;
  int M, N;       // output rows and columns
  void* out;      // [M, N], 16-bit, pitch N
};
constexpr int kPairMaxProblems = 4;
// plain products, one launch for all (at most kPairMaxProblems); out = sum over segments A B^T
cudaError_t launch_pair_gemm(const PairGemm* g, int n, int dtype, int* status, cudaStream_t st);
// Row pitch of the 16-bit tensors that one kernel hands to the next (h, dg, du):
// whole 128-byte lines.  A TMA box row off them is two requests, and the copies
// of a 1001 x 2008 x 1000 step, not the products, then set its time.
inline int64_t pair_pitch(int64_t I) { return (I + 63) / 64 * 64; }
// What the forward pass keeps for the backward one: h [T, pair_pitch(I)], and p = u act'(g)
// and a = act(g) in 24 bits, in blocks of 32 rows x 16 hidden units (row blocks
// outermost, edges padded) as an epilogue warp holds them, a row per lane:
// 32 x 32 bytes of p's upper 16 bits, as many of a's, 32 x 16 bytes of p's
// lower 8 bits and of a's.
constexpr int kKeptBlockB = 32 * 16 * 6;
struct PairKept {
  uint8_t *h, *blocks;
  size_t bytes;
};
inline PairKept pair_kept(void* base, int64_t T, int64_t I) {
  const size_t hb = ((size_t)(T * pair_pitch(I)) * 2 + 255) / 256 * 256;
  uint8_t* b = static_cast<uint8_t*>(base);
  return PairKept{b, b + hb, hb + (size_t)((T + 31) / 32 * ((I + 15) / 16)) * kKeptBlockB};
}
// h = act(x gate^T) * (x up^T)
struct PairGated {
  const void *x, *gate, *up;
  int64_t ldx;
  int64_t ldw;
  int T, I, K;
  int act, dtype;
  void* h;         // [T, I]
  int64_t ldh;
  bool keep;       // kept.h == h
  PairKept kept;
};
cudaError_t launch_pair_gated(const PairGated& a, int* status, cudaStream_t st);
// dh = dy down with dg = dh p, du = dh a written in its place
struct PairGatedBwd {
  const void* dy;         // [T, H]
  int64_t lddy;
  const void* down;       // [H, I]
  int T, H, I;
  int dtype;
  PairKept kept;
  void *dg, *du;          // [T, pair_pitch(I)]
};
cudaError_t launch_pair_gated_bwd(const PairGatedBwd& a, int* status, cudaStream_t st);
// bf16 x MXFP4 weights, decoded on the way into the products.  Every tile of rows
// decodes them again, in tiles of at most 128 columns; above two tiles of rows
// decoding once into bf16 for 256-column tiles is faster for most weights (us, that /
// here: 2816 x 2112 T = 256 12.8 / 10.9, T = 512 14.1 / 13.5, T = 1024 19.5 / 22.5; 4224
// x 2816 gated 16.2 / 13.7, 18.6 / 17.1, 26.1 / 28.4; 8192 x 2816 19.7 / 16.6, 27.5 /
// 28.1, 41.2 / 51.3; 32768 x 1024 32.3 / 24.0, 50.0 / 38.3, 61.8 / 69.6; rows as long as
// 8192 with 2816 columns 27.7 / 30.6, 32.8 / 37.1, 50.2 / 69.2)
constexpr int kPairW4MaxTokens = 512;
struct PairW4 {
  const void* x;
  int64_t ldx;
  const uint8_t *codes, *scales;  // [N (gated: 2 N), K]
  int T, N, K;
  int act;
  void* y;
};
cudaError_t launch_pair_w4(const PairW4& a, int* status, cudaStream_t st);
// MXFP4 x MXFP4 -> 16-bit, plain (act none) or gated (N = output columns)
struct PairMx {
  const uint8_t *xq, *xsf, *wq, *wsf;
  int T, N, K;
  int act, dtype, bn;  // bn: pair_mx_tile of the same product
  void* y;
};
int pair_mx_tile(int T, int N, int K, int act);
cudaError_t launch_pair_mx(const PairMx& a, int* status, cudaStream_t st);

}  // namespace nvfp4moe
