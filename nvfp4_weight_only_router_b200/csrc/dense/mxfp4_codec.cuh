// MXFP4 (E2M1 codes, one power-of-two scale byte per 32 elements): block
// encoding and decoding shared by the quantiser, the products' operand
// loads and the dequantiser.
#pragma once

#include "../common.cuh"
#include "../nvfp4_encode.cuh"
#include "dense_kernels.h"

namespace nvfp4moe {

// Launches.  Every kernel of this library may start while the kernel before it
// on the stream still runs (programmatic dependent launch): its launch and set-up
// then overlap that kernel's tail.  It touches global memory only behind
// after_previous(), which returns when that kernel is complete, and lets the next
// one start (let_next) only then, so that a kernel which waits for its
// predecessor knows everything before that one complete as well.  (The second
// kernel of a call may therefore load weights ahead of its own wait: they are not
// what the first one writes.)  Few-token calls in a row take 0.8 us less each.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Loads of what the kernel before may have written.  Not the read-only path
// (__ldg): its loads need data that does not change while the kernel runs, and the
// compiler may move them ahead of after_previous().  _stream: read once.
__device__ __forceinline__ uint32_t ld_u8(const void* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_u32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_v4_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void ld_v8_stream(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}

template <typename P, typename... Args>
cudaError_t launch_overlapped(void (*fn)(P, Args...), unsigned gx, unsigned gy, int threads, int smem, cudaStream_t st,
                              const P& p, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p, args...);
}

// Scale byte X + 127 of a block whose largest magnitude is amax >= 0, with
// X = floor(log2 amax) - 2 clamped to [-127, 127] (2 is the exponent of the
// largest E2M1 value, 6 = 1.5 * 2^2).  The exponent field of a normal fp32 is
// floor(log2) + 127; every subnormal amax and zero clamp to X = -127, and the
// largest finite amax gives X = 125.  255 (NaN) for an infinity or a NaN,
// which the caller leaves in amax's exponent field.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

// 2^-X as fp32 for a scale byte 0..252 (X = -127 gives 2^127, X = 125 gives 2^-125).
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^X as fp32: subnormal at byte 0, NaN at byte 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte == 0u ? 0x00400000u : byte << 23));
}

// Bits of the largest |v| with NaN above infinity above every finite value.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight E2M1 codes of v * inv (element i in nibble i).  The product is exact
// unless it is subnormal, far below the grid's first threshold.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8], uint32_t byte) {
  if (byte == 255u) return 0u;
  const float inv = mx_inv_scale(byte);
  float s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = v[k] * inv;
  return e2m1x8_rne(s);
}

// The two factors that turn a code's bits placed at a bf16's sign, two low
// exponent bits and top mantissa bit (v 2^-126, subnormal codes included)
// into v 2^X: 2^(126 + X) for X <= 1, and 2^127 followed by 2^(X - 1) above.
struct MxFactor {
  uint32_t f0, f1;  // bf16x2; f1 applies where big
  bool big;
};
__device__ __forceinline__ bool mx_big(uint32_t byte) { return byte > 128u && byte != 255u; }
__device__ __forceinline__ MxFactor mx_factor(uint32_t byte) {
  MxFactor m;
  const uint32_t h = byte == 255u ? 0x7FFFu : (min(byte, 128u) + 126u) << 7;
  m.f0 = h | (h << 16);
  m.big = mx_big(byte);
  const uint32_t b = (byte - 1u) << 7;
  m.f1 = b | (b << 16);
  return m;
}

__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t o;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
  return o;
}

// Eight codes (a 32-bit word) -> four bf16x2 of elements (j, j + 4), j = 0..3,
// times the first factor.
__device__ __forceinline__ void mx_place8(uint32_t w, const MxFactor& m, uint32_t (&o)[4]) {
  constexpr uint32_t M = 0x01C001C0u, S = 0x80008000u;
  o[0] = ((w << 6) & M) | ((w << 12) & S);
  o[1] = ((w << 2) & M) | ((w << 8) & S);
  o[2] = ((w >> 2) & M) | ((w << 4) & S);
  o[3] = ((w >> 6) & M) | (w & S);
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = bmul2(o[j], m.f0);
}
// The values (exact: E2M1 times a power of two is a bf16 unless it overflows or
// lies below 2^-133).
__device__ __forceinline__ void mx_decode8(uint32_t w, const MxFactor& m, uint32_t (&o)[4]) {
  mx_place8(w, m, o);
  if (m.big) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = bmul2(o[j], m.f1);
  }
}

// ------------------------------------------------------------ 16-bit elements
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi, bool f16) {
  uint32_t o;
  if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi), "f"(lo));
  return o;
}
__device__ __forceinline__ void unpack16x2(uint32_t v, bool f16, float& lo, float& hi) {
  if (f16) {
    lo = __half2float(__ushort_as_half((unsigned short)(v & 0xFFFFu)));
    hi = __half2float(__ushort_as_half((unsigned short)(v >> 16)));
  } else {
    lo = __uint_as_float(v << 16);
    hi = __uint_as_float(v & 0xFFFF0000u);
  }
}

// ---------------------------------------------------------------- activations
// gelu_tanh and silu with their derivatives, in fp32.  With s = 1 / (1 + exp(-z)),
// silu: z = g, gelu_tanh: z = 2 sqrt(2/pi) (g + 0.044715 g^3) (0.5 (1 + tanh(z / 2)) = s):
// act = g s, act' = s + g s (1 - s) dz/dg.  The fast exponential and division run
// once per hidden unit in epilogues that must not outlast the products.  In units of
// 2^-23, the exponential is off by 2 + 1.173 |z| relative, z's own roundings move it by up
// to 3.3 |z|, the sum, division and product add 4: s and act are within 2^-20 (1 + 0.6 |z|)
// relative (z < 0; above, the exponential is a small part of the sum and 2^-20 holds),
// which 16 bits do not show.  Where exp exceeds 2^126 the division gives the limit s = 0.
constexpr float kGeluK0 = 1.5957691216057308f, kGeluK1 = 0.044715f;  // 2 sqrt(2 / pi)
__device__ __forceinline__ float act_fwd(float g, int act) {
  const float z = act == kActSilu ? g : kGeluK0 * (g + kGeluK1 * g * g * g);
  return __fdividef(g, 1.0f + __expf(-z));
}
__device__ __forceinline__ void act_fwd_grad(float g, int act, float& a, float& da) {
  // s (1 - s) is 0 in fp32 well before |g| = 128 for both; the clamp keeps
  // dz finite beyond and lets a NaN through
  const float c = fabsf(g) > 128.0f ? copysignf(128.0f, g) : g;
  const float z = act == kActSilu ? c : kGeluK0 * (c + kGeluK1 * c * c * c);
  const float dz = act == kActSilu ? 1.0f : kGeluK0 * (1.0f + 3.0f * kGeluK1 * c * c);
  const float s = __fdividef(1.0f, 1.0f + __expf(-z));
  a = g * s;
  da = s + c * s * (1.0f - s) * dz;
}

// ------------------------------------------------ 24-bit kept values, wide access
// What the forward pass keeps for the backward one (act(g) and u act'(g)) is
// stored as the top 24 bits of its fp32: 16 bits in one plane and 8 in
// another.  Rounded to 16 bits they would add an error as large as the
// gradients' own rounding; 24 bits (2^-15) add none that shows, and 8 bytes
// per hidden unit with h in 16 bits is what four 16-bit tensors would take.
__device__ __forceinline__ uint32_t keep_hi2(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ uint32_t keep_lo4(float a, float b, float c, float d) {
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0051),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0051), 0x5410);
}
// value i (0..3) of two hi words (values 0, 1 and 2, 3) and one lo word
__device__ __forceinline__ float kept(uint32_t hi01, uint32_t hi23, uint32_t lo, int i) {
  const uint32_t hi = (i & 2) ? hi23 : hi01;
  const uint32_t h = (i & 1) ? (hi & 0xFFFF0000u) : (hi << 16);
  return __uint_as_float(h | (__byte_perm(lo, 0u, 0x4440 + i) << 8));
}

__device__ __forceinline__ void st_v8(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

}  // namespace nvfp4moe
