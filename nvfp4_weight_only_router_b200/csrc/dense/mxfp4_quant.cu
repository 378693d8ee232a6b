// MXFP4 quantisation and dequantisation (OCP microscaling: E2M1 elements, one
// E8M0 scale per 32 consecutive elements of a row).
//
//   a = max|x| over the block, X = clamp(floor(log2 a) - 2, -127, 127),
//   code = E2M1 nearest to x 2^-X (ties to the even code, saturating at 6),
//   value = E2M1 2^X.  A block with a NaN or an infinity gets scale 255 (NaN)
//   and codes 0; a ragged last block is filled up with zeros.
//
// Bound by memory: K (2 + 1/2 + 1/32) bytes per bf16 row.  Two forms:
//   16-bit types: a thread holds one block, 64 bytes by two 32-byte loads, its
//   maximum by packed integer comparisons, its codes by one 16-byte store,
//   without shuffles (32768 x 2816 bf16: 36 us, 6.5 TB/s);
//   f32: a thread holds 8 elements, four neighbouring lanes a block, whose
//   maximum takes two shuffles: with a whole block a thread, every lane of a
//   load touches a line of its own (32768 x 2820: 69 us, 113 that way; 16-bit
//   rows off the grid the other way round, 32768 x 2813 bf16 47 and 75).
// Rows off the 16-byte grid (and ragged last blocks) read the aligned 16-byte
// pieces that hold their elements and shift them into place in registers; only
// pieces that hold an element of the row are read.
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

// The bits of N elements.
template <typename T, int N>
struct Bits {
  static constexpr int W = N * sizeof(T) / 4;
  uint32_t w[W];
};

// Elements c..c + N - 1 of a row whose first element is row0 elements past x,
// zeros past K; only aligned pieces that hold an element of the row are read.
template <typename T, int N>
__device__ __forceinline__ Bits<T, N> load_any(const void* x, int64_t row0, int64_t c, int64_t K) {
  constexpr int W = Bits<T, N>::W;
  Bits<T, N> r;
  const int valid = (int)(K - c < N ? (K - c > 0 ? K - c : 0) : N);
  const uintptr_t a = reinterpret_cast<uintptr_t>(x) + (uintptr_t)(row0 + c) * sizeof(T);
  const int o = (int)(a & 15);  // bytes before the elements in their first piece
  const int bytes = valid * (int)sizeof(T);
  const uint4* src = reinterpret_cast<const uint4*>(a - o);
  uint32_t v[W + 4];
#pragma unroll
  for (int i = 0; i < W / 4 + 1; ++i) {
    const uint4 q = 16 * i < o + bytes && valid > 0 ? ld_v4(src + i) : make_uint4(0u, 0u, 0u, 0u);
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
    const int left = bytes - 4 * i;  // valid bytes of this word
    r.w[i] = left >= 4 ? w : (left > 0 ? w & 0xFFFFu : 0u);
  }
  return r;
}

// The same for rows whose addresses ALIGN (32, 16 or 0) divides.
template <typename T, int N, int ALIGN>
__device__ __forceinline__ Bits<T, N> load_bits(const void* x, int64_t row0, int64_t c, int64_t K) {
  constexpr int W = Bits<T, N>::W;
  if (ALIGN < 16 || c + N > K) return load_any<T, N>(x, row0, c, K);
  Bits<T, N> r;
  const char* p = static_cast<const char*>(x) + (row0 + c) * (int64_t)sizeof(T);
  if (ALIGN == 32 && W % 8 == 0) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      uint32_t q[8];
      ld_v8_stream(p + 32 * i, q);
#pragma unroll
      for (int k = 0; k < 8; ++k) r.w[8 * i + k] = q[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 q = ld_v4_stream(p + 16 * i);
      r.w[4 * i] = q.x; r.w[4 * i + 1] = q.y; r.w[4 * i + 2] = q.z; r.w[4 * i + 3] = q.w;
    }
  }
  return r;
}

// Bits of the largest magnitude, as fp32.
template <typename T, int N>
__device__ __forceinline__ uint32_t max_bits(const Bits<T, N>& r) {
  uint32_t a = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) a = max(a, r.w[i] & 0x7FFFFFFFu);
    return a;
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) a = __vmaxu2(a, r.w[i] & 0x7FFF7FFFu);
    float lo, hi;
    unpack16x2(a, std::is_same<T, __half>::value, lo, hi);
    return max(abs_bits(lo), abs_bits(hi));
  }
}

// Codes of elements 8 q..8 q + 7.
template <typename T, int N>
__device__ __forceinline__ uint32_t codes8(const Bits<T, N>& r, int q, uint32_t byte) {
  float v[8];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r.w[8 * q + k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack16x2(r.w[4 * q + k], std::is_same<T, __half>::value, v[2 * k], v[2 * k + 1]);
  }
  return mx_encode8(v, byte);
}

// One block of the flattened (row, block) order per thread and step, U steps
// of kQT blocks per CTA with their loads issued together.
template <typename T, int ALIGN, bool MMA, int U>
__device__ __forceinline__ void quant_cta(const QuantArgs& p, int64_t cta) {
  const int64_t first = cta * (kQT * U);
  const int64_t r0 = first / p.walked;
  const uint32_t b0 = (uint32_t)(first - r0 * p.walked), per = (uint32_t)p.walked;
  Bits<T, 32> blk[U];
  int64_t row[U];
  uint32_t b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = b0 + u * kQT + threadIdx.x, dr = i / per;
    row[u] = r0 + dr;
    b[u] = i - dr * per;
    // past the last row: nothing is read
    blk[u] = load_bits<T, 32, ALIGN>(p.x, row[u] * p.ldx, (int64_t)b[u] * 32, row[u] < p.rows ? p.K : 0);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] >= p.rows) continue;
    const uint32_t byte = mx_scale_byte(max_bits(blk[u]));
    const uint4 c = make_uint4(codes8(blk[u], 0, byte), codes8(blk[u], 1, byte), codes8(blk[u], 2, byte),
                               codes8(blk[u], 3, byte));
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
  after_previous();
  let_next();
  quant_cta<T, ALIGN, false, U>(p, blockIdx.x);
}

// 8 elements per thread and step of the flattened (row, group of 8) order, U
// steps with their loads issued together; a quad of lanes is in one block.
template <typename T, int ALIGN, int U>
__global__ void __launch_bounds__(kQT) mxfp4_quantize_quad_kernel(QuantArgs p) {
  after_previous();
  let_next();
  const uint32_t per = (uint32_t)(4 * p.nb);
  const int64_t first = (int64_t)blockIdx.x * (kQT * U);
  const int64_t r0 = first / per;
  const uint32_t g0 = (uint32_t)(first - r0 * per);
  Bits<T, 8> grp[U];
  int64_t row[U];
  uint32_t g[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = g0 + u * kQT + threadIdx.x, dr = i / per;
    row[u] = r0 + dr;
    g[u] = i - dr * per;
    // past the last row: nothing is read
    grp[u] = load_bits<T, 8, ALIGN>(p.x, row[u] * p.ldx, (int64_t)g[u] * 8, row[u] < p.rows ? p.K : 0);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t a = max_bits(grp[u]);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const uint32_t byte = mx_scale_byte(a), c = codes8(grp[u], 0, byte);
    if (row[u] >= p.rows) continue;
    reinterpret_cast<uint32_t*>(p.codes)[row[u] * per + g[u]] = c;
    if ((threadIdx.x & 3) == 0) p.scales[row[u] * p.nb + (g[u] >> 2)] = (uint8_t)byte;
  }
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
  after_previous();
  let_next();
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
  const uint32_t code = (ld_u8(codes + row * (16 * nb) + (c >> 1)) >> (4 * (c & 1))) & 15u;
  uint32_t h[4];
  e2m1x8_to_f16x2(code, h);
  float lo, hi;
  unpack16x2(h[0], true, lo, hi);
  return lo * mx_scale(ld_u8(scales + row * nb + (c >> 5)));
}

// 32 bytes of output per thread (G = 8 values of f32, 16 of bf16), contiguous
// over a warp, from one load of codes and one scale; four such groups with their
// loads issued together.  Rows of whole groups, 32-byte aligned output.
constexpr int kDU = 4, kDGroups = kQT * kDU;
constexpr int kAU = 2, kAGroups = kQT * kAU;  // any length

template <typename T>
__global__ void __launch_bounds__(kQT) mxfp4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
                                                               int64_t rows, int64_t K, T* out) {
  after_previous();
  let_next();
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
        const uint2 q = ld_v2(src);
        w[u][0] = q.x;
        w[u][1] = q.y;
      } else {
        w[u][0] = ld_u32(src);
      }
      sc[u] = ld_u8(scales + row * nb + g / (32 / G));
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
// which is 16-byte aligned.  Their codes lie in two words of the row, or end one
// row and begin the next, and their scales in two bytes or three (K < 8: value
// by value).  Two groups a thread: one or four take 11% and 22% longer at 30000
// x 2817 f32 (75 us); a value per thread and store took 8.0 us at 1000 x 2100
// f32 (5.1), this form for whole groups 83 us at 32768 x 2816 (63.5 above).
template <typename T>
__global__ void __launch_bounds__(kQT) mxfp4_dequantize_any_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                   int64_t rows, int64_t K, T* out) {
  after_previous();
  let_next();
  const int64_t nb = (K + 31) / 32, first = (int64_t)blockIdx.x * (kAGroups * 8), n = rows * K;
  const uint32_t k = (uint32_t)K, words = (uint32_t)(4 * nb);
  const int64_t r0 = first / K;
  const uint32_t c0 = (uint32_t)(first - r0 * K);
  uint32_t w[kAU], s0[kAU], s1[kAU], s2[kAU], c[kAU];
  int64_t row[kAU];
#pragma unroll
  for (int u = 0; u < kAU; ++u) {
    const uint32_t i = c0 + (u * kQT + threadIdx.x) * 8, dr = i / k;
    row[u] = r0 + dr;
    c[u] = i - dr * k;
    w[u] = s0[u] = s1[u] = s2[u] = 0;
    if (row[u] < rows && k >= 8) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes) + row[u] * words;
      const uint8_t* sc = scales + row[u] * nb;
      const uint32_t at = c[u] >> 3, sh = (c[u] & 7) * 4, valid = min(8u, k - c[u]);
      const uint32_t lo = ld_u32(src + at);
      w[u] = sh ? __funnelshift_r(lo, at + 1 < words ? ld_u32(src + at + 1) : 0u, sh) : lo;
      s0[u] = ld_u8(sc + (c[u] >> 5));
      s1[u] = ld_u8(sc + ((c[u] + valid - 1) >> 5));
      if (valid < 8) {
        w[u] &= (1u << (4 * valid)) - 1u;
        if (row[u] + 1 < rows) {
          w[u] |= ld_u32(src + words) << (4 * valid);
          s2[u] = ld_u8(sc + nb);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kAU; ++u) {
    const int64_t at = first + (int64_t)(u * kQT + threadIdx.x) * 8;
    if (row[u] >= rows) continue;
    float v[8];
    if (k >= 8) {
      uint32_t h[4];
      e2m1x8_to_f16x2(w[u], h);
      const float a = mx_scale(s0[u]), b = mx_scale(s1[u]), d = mx_scale(s2[u]);
      const uint32_t left = 32 - (c[u] & 31), valid = k - c[u];  // values under the first scale, of this row
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack16x2(h[i], true, v[2 * i], v[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= i >= valid ? d : i < left ? a : b;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t j = c[u] + i, dr = j / k;
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
cudaError_t quantize_u(const QuantArgs& p, cudaStream_t st) {
  if constexpr (sizeof(T) == 4) {
    const unsigned grid = blocks_for(p.rows * p.nb * 4, U * kQT);
    auto fn = p.align == 32   ? mxfp4_quantize_quad_kernel<T, 32, U>
              : p.align == 16 ? mxfp4_quantize_quad_kernel<T, 16, U>
                              : mxfp4_quantize_quad_kernel<T, 0, U>;
    return launch_overlapped(fn, grid, 1, kQT, 0, st, p);
  } else {
    const unsigned grid = blocks_for(p.rows * p.nb, U * kQT);
    auto fn = p.align == 32   ? mxfp4_quantize_kernel<T, 32, U>
              : p.align == 16 ? mxfp4_quantize_kernel<T, 16, U>
                              : mxfp4_quantize_kernel<T, 0, U>;
    return launch_overlapped(fn, grid, 1, kQT, 0, st, p);
  }
}

// Two steps a thread keep more bytes in flight; up to four CTAs an SM more
// threads do that better (us, two / one: 1000 x 2816 bf16 3.4 / 2.9, 1000 x 2100
// f32 4.8 / 3.7, 8192 x 2816 bf16 8.4 / 8.7).
template <typename T>
cudaError_t quantize_t(const QuantArgs& p, cudaStream_t st) {
  return p.rows * p.nb <= (int64_t)kSmallBlocks ? quantize_u<T, 1>(p, st) : quantize_u<T, 2>(p, st);
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, T* out, cudaStream_t st) {
  constexpr int G = 32 / sizeof(T);
  if (K % G == 0 && reinterpret_cast<uintptr_t>(out) % 32 == 0)
    return launch_overlapped(mxfp4_dequantize_kernel<T>, blocks_for(rows * (K / G), kDGroups), 1, kQT, 0, st, codes,
                             scales, rows, K, out);
  return launch_overlapped(mxfp4_dequantize_any_kernel<T>, blocks_for(rows * K, kAGroups * 8), 1, kQT, 0, st, codes,
                           scales, rows, K, out);
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
  if (dtype == kF32) return quantize_t<float>(p, st);
  return dtype == kF16 ? quantize_t<__half>(p, st) : quantize_t<__nv_bfloat16>(p, st);
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* out,
                                    int dtype, cudaStream_t st) {
  return dtype == kF32 ? dequantize_t(codes, scales, rows, K, static_cast<float*>(out), st)
                       : dequantize_t(codes, scales, rows, K, static_cast<__nv_bfloat16*>(out), st);
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
  const bool wide = row_align(a.x, a.ldx, 2) == 32;
  auto fn = a.dtype == kF16 ? (wide ? mxfp4_prep_kernel<__half, 32> : mxfp4_prep_kernel<__half, 16>)
                            : (wide ? mxfp4_prep_kernel<__nv_bfloat16, 32> : mxfp4_prep_kernel<__nv_bfloat16, 16>);
  return launch_overlapped(fn, grid, 1, kQT, 0, st, p, qb, t);
}

}  // namespace nvfp4moe
