// MXFP4 quantisation and dequantisation (OCP microscaling: E2M1 elements, one
// E8M0 scale per 32 consecutive elements of a row).
//
//   a = max|x| over the block, X = clamp(floor(log2 a) - 2, -127, 127),
//   code = E2M1 nearest to x 2^-X (ties to the even code, saturating at 6),
//   value = E2M1 2^X.  A block with a NaN or an infinity gets scale 255 (NaN)
//   and codes 0; a ragged last block is filled up with zeros.
//
// Bound by memory: K (2 + 1/2 + 1/32) bytes per bf16 row.  A thread holds one
// block: 64 bytes of a 16-bit row by two 32-byte loads, its maximum by packed
// integer comparisons, its codes by one 16-byte store, so that a block costs
// no shuffles and neighbouring threads write neighbouring codes and scales.
// Rows off the 16-byte grid (and ragged last blocks) read the aligned 16-byte
// pieces that hold the block and shift them into place in registers; only
// pieces that hold an element of the block are read.
#include <type_traits>

#include "mxfp4_codec.cuh"

namespace nvfp4moe {

namespace {

constexpr int kQT = 256;  // threads

struct QuantArgs {
  const void* x;
  int64_t rows, K, ldx;
  uint8_t* codes;
  uint8_t* scales;
  int64_t nb;      // blocks per row
  int64_t walked;  // blocks walked per row: nb, or up to whole chunks
  int sf_chunks;   // MMA order: 512-byte chunks per row block
  int align;       // bytes that divide every row's address: 32, 16, or less (0)
};

// The bits of one block.
template <typename T>
struct Blk {
  static constexpr int W = 32 * sizeof(T) / 4;
  uint32_t w[W];
};

// Valid elements c..min(c + 32, K) of a row whose first element is row0
// elements past x, zeros behind them.
template <typename T>
__device__ __forceinline__ Blk<T> load_block_any(const void* x, int64_t row0, int64_t c, int64_t K) {
  constexpr int W = Blk<T>::W;
  Blk<T> r;
  const int valid = (int)(K - c < 32 ? (K - c > 0 ? K - c : 0) : 32);
  const uintptr_t a = reinterpret_cast<uintptr_t>(x) + (uintptr_t)(row0 + c) * sizeof(T);
  const int o = (int)(a & 15);                           // bytes before the block in its first piece
  const int bytes = valid * (int)sizeof(T);
  const uint4* src = reinterpret_cast<const uint4*>(a - o);
  uint32_t v[W + 4];
#pragma unroll
  for (int i = 0; i < W / 4 + 1; ++i) {
    const uint4 q = 16 * i < o + bytes && valid > 0 ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
    v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
  }
  if (o & 8) {
#pragma unroll
    for (int i = 0; i < W + 2; ++i) v[i] = v[i + 2];
  }
  if (o & 4) {
#pragma unroll
    for (int i = 0; i < W + 1; ++i) v[i] = v[i + 1];
  }
  const bool odd = o & 2;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t w = v[i];
    if (sizeof(T) == 2 && odd) w = __byte_perm(v[i], v[i + 1], 0x5432);
    const int left = bytes - 4 * i;                      // valid bytes of this word
    r.w[i] = left >= 4 ? w : (left > 0 ? w & 0xFFFFu : 0u);
  }
  return r;
}

template <typename T, int ALIGN>
__device__ __forceinline__ Blk<T> load_block(const void* x, int64_t row0, int64_t c, int64_t K) {
  constexpr int W = Blk<T>::W;
  if (ALIGN < 16 || c + 32 > K) return load_block_any<T>(x, row0, c, K);
  Blk<T> r;
  const char* p = static_cast<const char*>(x) + (row0 + c) * (int64_t)sizeof(T);
  if (ALIGN == 32) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      uint32_t q[8];
      ld_nc_v8(p + 32 * i, q);
#pragma unroll
      for (int k = 0; k < 8; ++k) r.w[8 * i + k] = q[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 q = ldg_nc_v4(p + 16 * i);
      r.w[4 * i] = q.x; r.w[4 * i + 1] = q.y; r.w[4 * i + 2] = q.z; r.w[4 * i + 3] = q.w;
    }
  }
  return r;
}

// The block's scale byte and its 32 codes.
template <typename T>
__device__ __forceinline__ uint4 encode_block(const Blk<T>& r, uint32_t& byte) {
  constexpr bool F16 = std::is_same<T, __half>::value;
  uint32_t a = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 32; ++i) a = max(a, r.w[i] & 0x7FFFFFFFu);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) a = __vmaxu2(a, r.w[i] & 0x7FFF7FFFu);
    float lo, hi;
    unpack16x2(a, F16, lo, hi);
    a = max(abs_bits(lo), abs_bits(hi));
  }
  byte = mx_scale_byte(a);
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r.w[8 * q + k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) unpack16x2(r.w[4 * q + k], F16, v[2 * k], v[2 * k + 1]);
    }
    c[q] = mx_encode8(v, byte);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// One block of the flattened (row, block) order per thread and step, U steps
// of kQT blocks per CTA with their loads issued together.
template <typename T, int ALIGN, bool MMA, int U>
__device__ __forceinline__ void quant_cta(const QuantArgs& p, int64_t cta) {
  const int64_t first = cta * (kQT * U);
  const int64_t r0 = first / p.walked;
  const uint32_t b0 = (uint32_t)(first - r0 * p.walked), per = (uint32_t)p.walked;
  Blk<T> blk[U];
  int64_t row[U];
  uint32_t b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = b0 + u * kQT + threadIdx.x, dr = i / per;
    row[u] = r0 + dr;
    b[u] = i - dr * per;
    // past the last row: nothing is read
    blk[u] = load_block<T, ALIGN>(p.x, row[u] * p.ldx, (int64_t)b[u] * 32, row[u] < p.rows ? p.K : 0);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] >= p.rows) continue;
    uint32_t byte;
    const uint4 c = encode_block<T>(blk[u], byte);
    if (!MMA || b[u] < p.nb) reinterpret_cast<uint4*>(p.codes)[row[u] * p.nb + b[u]] = c;
    if (MMA) {
      // blocks past K: scale 2^-127 on zero codes
      const int64_t chunk = (row[u] >> 7) * p.sf_chunks + (b[u] >> 2);
      const int r = (int)(row[u] & 127);
      p.scales[chunk * kSfChunkB + 16 * (r & 31) + 4 * (r >> 5) + (b[u] & 3)] = (uint8_t)byte;
    } else {
      p.scales[row[u] * p.nb + b[u]] = (uint8_t)byte;
    }
  }
}
constexpr int kSmallBlocks = 4 * 148 * kQT;
constexpr int kPrepU = 2;  // steps of the kernel that prepares a product

template <typename T, int ALIGN, int U>
__global__ void __launch_bounds__(kQT) mxfp4_quantize_kernel(QuantArgs p) {
  quant_cta<T, ALIGN, false, U>(p, blockIdx.x);
}

struct TileScales {
  const uint8_t* ws;
  uint8_t* wsf;
  int64_t words;
  int N, bn;
  bool gated;
};

// Blocks below qblocks quantise activations into the tensor core's operand
// form; the others lay the weight's scales out (one 4-byte word a thread: the
// scales of 4 blocks of one row).
template <typename T, int ALIGN>
__global__ void __launch_bounds__(kQT) mxfp4_prep_kernel(QuantArgs p, int64_t qblocks, TileScales t) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the product sets up meanwhile
  if ((int64_t)blockIdx.x < qblocks) {
    quant_cta<T, ALIGN, true, kPrepU>(p, blockIdx.x);
    return;
  }
  const int64_t w = ((int64_t)blockIdx.x - qblocks) * kQT + threadIdx.x;
  if (w >= t.words) return;
  const int wi = (int)(w & 127);
  const int64_t ch = w >> 7;
  const int c = (int)(ch % p.sf_chunks);
  const int64_t rb = ch / p.sf_chunks;
  const int bpt = (t.bn + 127) / 128;  // scale blocks per tile
  const int tile = (int)(rb / bpt), l = (int)(rb % bpt) * 128 + (wi >> 2) + 32 * (wi & 3);  // row of the tile
  const int half = t.bn / 2;
  const int r = t.gated ? tile * half + l % half : tile * t.bn + l;
  uint32_t v = 0;
  if (l < t.bn && r < t.N) {
    const uint8_t* src = t.ws + ((int64_t)(t.gated && l >= half ? t.N : 0) + r) * p.nb;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * c + i < p.nb) v |= (uint32_t)src[4 * c + i] << (8 * i);
  }
  reinterpret_cast<uint32_t*>(t.wsf)[w] = v;
}

// The value of element c of a row.
__device__ __forceinline__ float mx_value(const uint8_t* codes, const uint8_t* scales, int64_t row, uint32_t c, int64_t nb) {
  const uint32_t code = ((uint32_t)__ldg(codes + row * (16 * nb) + (c >> 1)) >> (4 * (c & 1))) & 15u;
  uint32_t h[4];
  e2m1x8_to_f16x2(code, h);
  float lo, hi;
  unpack16x2(h[0], true, lo, hi);
  return lo * mx_scale(__ldg(scales + row * nb + (c >> 5)));
}

// 32 bytes of output per thread (G = 8 values of f32, 16 of bf16), contiguous
// over a warp, from one load of codes and one scale; four such groups with their
// loads issued together.  Rows of whole groups, 32-byte aligned output.
constexpr int kDU = 4, kDGroups = kQT * kDU;
constexpr int kAU = 2, kAGroups = kQT * kAU;  // any length

template <typename T>
__global__ void __launch_bounds__(kQT) mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t rows,
                                                               int64_t K, T* __restrict__ out) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // a product may set up meanwhile
  constexpr int G = 32 / sizeof(T);
  const int64_t nb = (K + 31) / 32, first = (int64_t)blockIdx.x * kDGroups;
  const uint32_t gpr = (uint32_t)(K / G);
  const int64_t r0 = first / gpr;
  const uint32_t g0 = (uint32_t)(first - r0 * gpr);
  uint32_t w[kDU][G / 8], sc[kDU];
#pragma unroll
  for (int u = 0; u < kDU; ++u) {
    const uint32_t i = g0 + u * kQT + threadIdx.x, dr = i / gpr, g = i - dr * gpr;
    const int64_t row = r0 + dr;
    sc[u] = 0;
#pragma unroll
    for (int k = 0; k < G / 8; ++k) w[u][k] = 0;
    if (row < rows) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes) + row * (4 * nb) + g * (G / 8);
      if constexpr (G == 16) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(src));
        w[u][0] = q.x;
        w[u][1] = q.y;
      } else {
        w[u][0] = __ldg(src);
      }
      sc[u] = __ldg(scales + row * nb + g / (32 / G));
    }
  }
#pragma unroll
  for (int u = 0; u < kDU; ++u) {
    const int64_t at = (first + u * kQT + threadIdx.x) * G;  // rows are whole groups: out is flat
    if (at >= rows * K) continue;
    const float s = mx_scale(sc[u]);
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < G / 8; ++q) {
      uint32_t h[4];
      e2m1x8_to_f16x2(w[u][q], h);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        unpack16x2(h[k], true, lo, hi);
        lo *= s;
        hi *= s;
        if constexpr (G == 16) {
          o[4 * q + k] = pack16x2(lo, hi, false);
        } else {
          o[2 * k] = __float_as_uint(lo);
          o[2 * k + 1] = __float_as_uint(hi);
        }
      }
    }
    st_v8(out + at, o);
  }
}

// Any K and alignment: a thread writes 8 consecutive values of the flat output,
// which is 16-byte aligned.  Their codes lie in two words of the row and their
// scales in two bytes; a group that runs over the end of its row goes value by
// value.  Two groups a thread: one or four take 11% and 22% longer at 30000 x
// 2817 f32 (76.1 us); a value per thread and store took 8.0 us at 1000 x 2100
// f32 (5.6), this form for whole groups 83 us at 32768 x 2816 (63.5 above).
template <typename T>
__global__ void __launch_bounds__(kQT) mxfp4_dequantize_any_kernel(const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales, int64_t rows,
                                                                   int64_t K, T* __restrict__ out) {
  const int64_t nb = (K + 31) / 32, first = (int64_t)blockIdx.x * (kAGroups * 8), n = rows * K;
  const uint32_t k = (uint32_t)K, words = (uint32_t)(4 * nb);
  const int64_t r0 = first / K;
  const uint32_t c0 = (uint32_t)(first - r0 * K);
  uint32_t w[kAU], s0[kAU], s1[kAU], c[kAU];
  int64_t row[kAU];
#pragma unroll
  for (int u = 0; u < kAU; ++u) {
    const uint32_t i = c0 + (u * kQT + threadIdx.x) * 8, dr = i / k;
    row[u] = r0 + dr;
    c[u] = i - dr * k;
    w[u] = s0[u] = s1[u] = 0;
    if (row[u] < rows && c[u] + 8 <= k) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes) + row[u] * words;
      const uint32_t at = c[u] >> 3, sh = (c[u] & 7) * 4;
      const uint32_t lo = __ldg(src + at);
      w[u] = sh ? __funnelshift_r(lo, __ldg(src + at + 1), sh) : lo;
      s0[u] = __ldg(scales + row[u] * nb + (c[u] >> 5));
      s1[u] = __ldg(scales + row[u] * nb + ((c[u] + 7) >> 5));
    }
  }
#pragma unroll
  for (int u = 0; u < kAU; ++u) {
    const int64_t at = first + (int64_t)(u * kQT + threadIdx.x) * 8;
    if (row[u] >= rows) continue;
    float v[8];
    if (c[u] + 8 <= k) {
      uint32_t h[4];
      e2m1x8_to_f16x2(w[u], h);
      const float a = mx_scale(s0[u]), b = mx_scale(s1[u]);
      const uint32_t left = 32 - (c[u] & 31);  // values under the first scale
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack16x2(h[i], true, v[2 * i], v[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= i < left ? a : b;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t j = c[u] + i, dr = j / k;  // K may be less than 8
        v[i] = row[u] + dr < rows ? mx_value(codes, scales, row[u] + dr, j - dr * k, nb) : 0.f;
      }
    }
    if (at + 8 > n) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < n) out[at + i] = (T)v[i];
    } else if constexpr (sizeof(T) == 4) {
      float4* o = reinterpret_cast<float4*>(out + at);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(out + at) = make_uint4(pack16x2(v[0], v[1], false), pack16x2(v[2], v[3], false),
                                                       pack16x2(v[4], v[5], false), pack16x2(v[6], v[7], false));
    }
  }
}

unsigned blocks_for(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

int row_align(const void* p, int64_t ld, int elsize) {
  for (int a = 32; a >= 16; a /= 2)
    if (reinterpret_cast<uintptr_t>(p) % a == 0 && (ld * elsize) % a == 0) return a;
  return 0;
}

template <typename T, int U>
void quantize_u(const QuantArgs& p, cudaStream_t st) {
  const unsigned grid = blocks_for(p.rows * p.walked, U * kQT);
  if (p.align == 32) mxfp4_quantize_kernel<T, 32, U><<<grid, kQT, 0, st>>>(p);
  else if (p.align == 16) mxfp4_quantize_kernel<T, 16, U><<<grid, kQT, 0, st>>>(p);
  else mxfp4_quantize_kernel<T, 0, U><<<grid, kQT, 0, st>>>(p);
}

// Two blocks a thread keep more bytes in flight; up to about four CTAs an SM
// twice the threads do that better (bf16, us, two / one: 1 x 2816 2.5 / 2.1,
// 1000 x 2816 3.4 / 3.1; 1000 x 2100 f32 5.4 / 5.2).
template <typename T>
void quantize_t(const QuantArgs& p, cudaStream_t st) {
  if (p.rows * p.walked <= (int64_t)kSmallBlocks) quantize_u<T, 1>(p, st);
  else quantize_u<T, 2>(p, st);
}

template <typename T>
void dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, T* out, cudaStream_t st) {
  constexpr int G = 32 / sizeof(T);
  if (K % G == 0 && reinterpret_cast<uintptr_t>(out) % 32 == 0)
    mxfp4_dequantize_kernel<T><<<blocks_for(rows * (K / G), kDGroups), kQT, 0, st>>>(codes, scales, rows, K, out);
  else
    mxfp4_dequantize_any_kernel<T><<<blocks_for(rows * K, kAGroups * 8), kQT, 0, st>>>(codes, scales, rows, K, out);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st) {
  QuantArgs p{};
  p.x = x;
  p.rows = rows;
  p.K = K;
  p.ldx = ldx;
  p.codes = codes;
  p.scales = scales;
  p.nb = p.walked = mx_blocks(K);
  p.align = row_align(x, ldx, dtype == kF32 ? 4 : 2);
  if (dtype == kF32) quantize_t<float>(p, st);
  else if (dtype == kF16) quantize_t<__half>(p, st);
  else quantize_t<__nv_bfloat16>(p, st);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* out,
                                    int dtype, cudaStream_t st) {
  if (dtype == kF32) dequantize_t(codes, scales, rows, K, static_cast<float*>(out), st);
  else dequantize_t(codes, scales, rows, K, static_cast<__nv_bfloat16*>(out), st);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_prep_a4(const MxPrepArgs& a, cudaStream_t st) {
  QuantArgs p{};
  p.x = a.x;
  p.rows = a.T;
  p.K = a.K;
  p.ldx = a.ldx;
  p.codes = a.xq;
  p.scales = a.xsf;
  p.nb = mx_blocks(a.K);
  p.sf_chunks = mx_sf_chunks(a.K);
  p.walked = (int64_t)p.sf_chunks * 4;
  const int64_t qb = blocks_for(p.rows * p.walked, kPrepU * kQT);
  const TileScales t{a.wscales, a.wsf, mx_wsf_blocks(a.N, a.gated, a.bn) * p.sf_chunks * 128, a.N, a.bn, a.gated};
  const unsigned grid = (unsigned)qb + blocks_for(t.words, kQT);
  // x's rows are 16-byte aligned (checked by the entry point)
  if (row_align(a.x, a.ldx, 2) == 32) {
    if (a.dtype == kF16) mxfp4_prep_kernel<__half, 32><<<grid, kQT, 0, st>>>(p, qb, t);
    else mxfp4_prep_kernel<__nv_bfloat16, 32><<<grid, kQT, 0, st>>>(p, qb, t);
  } else {
    if (a.dtype == kF16) mxfp4_prep_kernel<__half, 16><<<grid, kQT, 0, st>>>(p, qb, t);
    else mxfp4_prep_kernel<__nv_bfloat16, 16><<<grid, kQT, 0, st>>>(p, qb, t);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4moe
