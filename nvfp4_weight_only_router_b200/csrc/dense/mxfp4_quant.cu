// MXFP4 quantisation and dequantisation (OCP microscaling: E2M1 elements, one
// E8M0 scale per 32 consecutive elements of a row).
//
//   a = max|x| over the block, X = clamp(floor(log2 a) - 2, -127, 127),
//   code = E2M1 nearest to x 2^-X (ties to the even code, saturating at 6),
//   value = E2M1 2^X.  A block with a NaN or an infinity gets scale 255 (NaN)
//   and codes 0; a ragged last block is filled up with zeros.
//
// Bound by memory: K (2 + 1/2 + 1/32) bytes per bf16 row.  A thread holds 8
// consecutive elements (one or two 16-byte loads, one 4-byte store of codes),
// four neighbouring lanes form a block and share its maximum through two
// shuffles, so loads and stores of a warp are contiguous.  Four groups per
// thread keep four loads in flight.
#include <type_traits>

#include "mxfp4_codec.cuh"

namespace nvfp4moe {

namespace {

constexpr int kQT = 256;  // threads
constexpr int kQU = 4;    // groups of 8 elements per thread
constexpr int kQGroups = kQT * kQU;

// The bits of 8 elements; loaded first for all of a thread's groups.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) == 4 ? 2 : 1];
};

template <typename T>
__device__ __forceinline__ void raw_to_f32(const Raw<T>& r, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack16x2(w[k], std::is_same<T, __half>::value, v[2 * k], v[2 * k + 1]);
  }
}

// One group of 8 elements from column c of a row (the row's first element at
// x): vector loads where the group lies inside the row and vec holds.
template <typename T>
__device__ __forceinline__ Raw<T> load_group(const void* x, int64_t row0, int64_t c, int64_t K, bool vec) {
  Raw<T> r;
  if (vec && c + 8 <= K) {
    const char* p = static_cast<const char*>(x) + (row0 + c) * (int64_t)sizeof(T);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = ldg_nc_v4(p + 16 * i);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[k] = 0u;
      if (c + k < K) {
        if constexpr (sizeof(T) == 4) w[k] = static_cast<const uint32_t*>(x)[row0 + c + k];
        else w[k] = static_cast<const uint16_t*>(x)[row0 + c + k];
      }
    }
    if constexpr (sizeof(T) == 4) {
      r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
      r.v[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      r.v[0] = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
    }
  }
  return r;
}

struct QuantArgs {
  const void* x;
  int64_t rows, K, ldx;
  uint8_t* codes;
  uint8_t* scales;
  int64_t nb;        // blocks per row
  int64_t groups;    // groups of 8 walked per row: 4 nb, or up to whole chunks
  int sf_chunks;     // MMA order: 512-byte chunks per row block
  bool vec;
};

// Codes of one group and its block's scale byte (valid in every lane of the quad).
template <typename T>
__device__ __forceinline__ uint32_t encode_group(const Raw<T>& raw, uint32_t& byte) {
  float v[8];
  raw_to_f32<T>(raw, v);
  uint32_t a = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) a = max(a, abs_bits(v[k]));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  byte = mx_scale_byte(a);
  return mx_encode8(v, byte);
}

// Walks the groups [blk * kQGroups, + kQGroups) of the flattened (row, group)
// order; all lanes of a quad are in the same block of the same row.
template <typename T, bool MMA>
__device__ __forceinline__ void quant_block(const QuantArgs& p, int64_t blk) {
  const int64_t first = blk * kQGroups;
  const int64_t r0 = first / p.groups;
  const uint32_t g0 = (uint32_t)(first - r0 * p.groups), gpr = (uint32_t)p.groups;
  Raw<T> raw[kQU];
  int64_t row[kQU];
  uint32_t grp[kQU];
#pragma unroll
  for (int u = 0; u < kQU; ++u) {
    const uint32_t g = g0 + u * kQT + threadIdx.x, dr = g / gpr;
    row[u] = r0 + dr;
    grp[u] = g - dr * gpr;
    if (row[u] < p.rows) raw[u] = load_group<T>(p.x, row[u] * p.ldx, (int64_t)grp[u] * 8, p.K, p.vec);
    else raw[u] = Raw<T>{};
  }
#pragma unroll
  for (int u = 0; u < kQU; ++u) {
    uint32_t byte;
    const uint32_t c = encode_group<T>(raw[u], byte);
    if (row[u] >= p.rows) continue;
    const int64_t b = grp[u] >> 2;
    if (!MMA || b < p.nb) reinterpret_cast<uint32_t*>(p.codes)[row[u] * (4 * p.nb) + grp[u]] = c;
    if ((threadIdx.x & 3) == 0) {
      if (MMA) {
        // blocks past K: scale 2^-127 on zero codes
        const int64_t chunk = (row[u] >> 7) * p.sf_chunks + (b >> 2);
        const int r = (int)(row[u] & 127);
        p.scales[chunk * kSfChunkB + 16 * (r & 31) + 4 * (r >> 5) + (b & 3)] = (uint8_t)byte;
      } else {
        p.scales[row[u] * p.nb + b] = (uint8_t)byte;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kQT) mxfp4_quantize_kernel(QuantArgs p) {
  quant_block<T, false>(p, blockIdx.x);
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
template <typename T>
__global__ void __launch_bounds__(kQT) mxfp4_prep_kernel(QuantArgs p, int64_t qblocks, TileScales t) {
  if ((int64_t)blockIdx.x < qblocks) {
    quant_block<T, true>(p, blockIdx.x);
    return;
  }
  const int64_t w = ((int64_t)blockIdx.x - qblocks) * kQT + threadIdx.x;
  if (w >= t.words) return;
  const int wi = (int)(w & 127);
  const int64_t ch = w >> 7;
  const int c = (int)(ch % p.sf_chunks);
  const int64_t rb = ch / p.sf_chunks;
  const int bpt = t.bn >= 256 ? 2 : 1;  // scale blocks per tile
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

// 8 codes per thread; a row's values are K apart in `out`.
template <typename T>
__global__ void __launch_bounds__(kQT) mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t rows,
                                                               int64_t K, T* __restrict__ out, bool vec) {
  const int64_t nb = (K + 31) / 32;
  const int64_t first = (int64_t)blockIdx.x * kQGroups;
  const uint32_t gpr = (uint32_t)(4 * nb);
  const int64_t r0 = first / gpr;
  const uint32_t g0 = (uint32_t)(first - r0 * gpr);
  uint32_t w[kQU], sc[kQU];
#pragma unroll
  for (int u = 0; u < kQU; ++u) {
    const uint32_t g = g0 + u * kQT + threadIdx.x, dr = g / gpr;
    const int64_t row = r0 + dr;
    w[u] = sc[u] = 0;
    if (row < rows) {
      w[u] = __ldcs(reinterpret_cast<const uint32_t*>(codes) + row * gpr + (g - dr * gpr));
      sc[u] = __ldg(scales + row * nb + ((g - dr * gpr) >> 2));
    }
  }
#pragma unroll
  for (int u = 0; u < kQU; ++u) {
    const uint32_t g = g0 + u * kQT + threadIdx.x, dr = g / gpr;
    const int64_t row = r0 + dr, c = (int64_t)(g - dr * gpr) * 8;
    if (row >= rows || c >= K) continue;
    uint32_t h[4];
    e2m1x8_to_f16x2(w[u], h);
    const float s = mx_scale(sc[u]);
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      unpack16x2(h[k], true, v[2 * k], v[2 * k + 1]);
      v[2 * k] *= s;
      v[2 * k + 1] *= s;
    }
    T* dst = out + row * K + c;
    if (vec && c + 8 <= K) {
      if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4*>(dst), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack16x2(v[0], v[1], false), pack16x2(v[2], v[3], false),
                                                    pack16x2(v[4], v[5], false), pack16x2(v[6], v[7], false));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < K) {
          if constexpr (sizeof(T) == 4) dst[k] = v[k];
          else dst[k] = __float2bfloat16_rn(v[k]);
        }
    }
  }
}

int64_t blocks_for(int64_t groups) { return (groups + kQGroups - 1) / kQGroups; }

bool vector_rows(const void* p, int64_t ld, int elsize) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * elsize) % 16 == 0;
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
  p.nb = mx_blocks(K);
  p.groups = 4 * p.nb;
  p.vec = vector_rows(x, ldx, dtype == kF32 ? 4 : 2);
  const unsigned grid = (unsigned)blocks_for(rows * p.groups);
  if (dtype == kF32) mxfp4_quantize_kernel<float><<<grid, kQT, 0, st>>>(p);
  else if (dtype == kF16) mxfp4_quantize_kernel<__half><<<grid, kQT, 0, st>>>(p);
  else mxfp4_quantize_kernel<__nv_bfloat16><<<grid, kQT, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* out,
                                    int dtype, cudaStream_t st) {
  const unsigned grid = (unsigned)blocks_for(rows * 4 * mx_blocks(K));
  const bool vec = vector_rows(out, K, dtype == kF32 ? 4 : 2);
  if (dtype == kF32)
    mxfp4_dequantize_kernel<float><<<grid, kQT, 0, st>>>(codes, scales, rows, K, static_cast<float*>(out), vec);
  else
    mxfp4_dequantize_kernel<__nv_bfloat16>
        <<<grid, kQT, 0, st>>>(codes, scales, rows, K, static_cast<__nv_bfloat16*>(out), vec);
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
  p.groups = (int64_t)p.sf_chunks * 16;
  p.vec = vector_rows(a.x, a.ldx, 2);
  const int64_t qb = blocks_for(p.rows * p.groups);
  const TileScales t{a.wscales, a.wsf, mx_wsf_blocks(a.N, a.gated, a.bn) * p.sf_chunks * 128, a.N, a.bn, a.gated};
  const unsigned grid = (unsigned)(qb + (t.words + kQT - 1) / kQT);
  if (a.dtype == kF16) mxfp4_prep_kernel<__half><<<grid, kQT, 0, st>>>(p, qb, t);
  else mxfp4_prep_kernel<__nv_bfloat16><<<grid, kQT, 0, st>>>(p, qb, t);
  return cudaGetLastError();
}

}  // namespace nvfp4moe
