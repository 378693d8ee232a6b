// Products of few tokens (up to 32 a CTA) with a weight matrix: y[t, n] = sum_k x[t, k]
// w[n, k], optionally gated (y[t, i] = act(gate_i) up_i), with 16-bit or MXFP4
// weights.
//
// Bound by the weight stream (T = 1, MXFP4 4224 x 2816: 6.3 MB) and, at these
// sizes, by the latency of a few dependent loads, so the kernel is one wave of
// small CTAs that put their whole share of the weights in flight at once: a
// CTA owns 16 rows (gated: 8 gate rows and their 8 up rows), its 8 warps take
// interleaved steps of K, and the 8 partial tiles meet in shared memory.  The
// products run on the warp-level tensor instruction m16n8k16 (the memory pipe
// is the limit, not the tensor pipe).  Its K order is free as long as both
// operands agree, so each lane loads 16 consecutive bytes of its two rows and
// the matching elements of x:
//   16-bit:  8 elements, two instructions;
//   MXFP4:   32 codes = one block with one scale, eight instructions; the
//            codes become bf16 in registers (exact), pairing elements j and
//            j + 4 of every 8.
// Gated tiles put gate row i and up row i into rows r and r + 8 of the tile,
// which one lane holds both of.  With quant_x a lane holds a whole 32-element
// block of x per token: it quantises it to MXFP4 and back in registers (the
// values are bf16 exactly), so the W4A4 product of few tokens is this kernel too.
//
// after_producer: weights are loaded while the kernel before on the stream still
// runs, x once its results are visible.
#include <algorithm>

#include "mxfp4_codec.cuh"

namespace nvfp4moe {

namespace {

constexpr int kSkThreads = 256, kSkWarps = 8;

template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  const uint32_t a[4] = {a0, a1, a2, a3};
  if (F16) mma_f16_16816(d, a, b0, b1);
  else mma_bf16_16816(d, a, b0, b1);
}

struct SkinnyParams {
  const uint8_t *x, *w0, *w1, *s0, *s1;
  uint16_t* y;
  int64_t ldx_bytes;
  int T, N, units;   // units: 16-byte pieces of a weight row
  int act;
  bool f16;          // type of y (and of x)
  bool after;        // x is written by the kernel before
  bool split;        // plain: rows 2t, 2t + 1 of x are a token; gated: of y
};

// Steps of K in flight per warp: for one group of tokens the whole K of the
// layer's sizes, for more what the registers allow.
template <int CODEC, int NT8, bool XS>
struct SkCfg {
  static constexpr int U = CODEC == 1 ? 3 : (NT8 == 1 ? 11 : 6);
  static constexpr int XW = CODEC == 1 ? 4 : 1;  // 16-byte pieces of x per step and token
  static constexpr int XPASS = kSkWarps * U * 4 * XW * 16, XPITCH = XPASS + 32;  // bytes of a token
  static constexpr int RED = kSkWarps * NT8 * 32 * 16;                           // the partial tiles
  static int smem(int T) { return XS ? std::max(RED, std::min(T, NT8 * 8) * XPITCH) : RED; }
};

// 8 elements of x in shared memory -> the bf16 values that MXFP4 keeps of them
// (exact).  A quad of lanes has a block; the whole warp takes part.
__device__ __forceinline__ void quantize_in_place(uint8_t* at, bool valid, bool f16) {
  uint4* const p = reinterpret_cast<uint4*>(at);
  const uint4 x = valid ? *p : make_uint4(0u, 0u, 0u, 0u);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
  float lo, hi;
  unpack16x2(m2, f16, lo, hi);
  uint32_t m = max(abs_bits(lo), abs_bits(hi));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t byte = mx_scale_byte(m);
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) unpack16x2(w[k], f16, v[2 * k], v[2 * k + 1]);
  uint32_t o[4];
  mx_decode8(mx_encode8(v, byte), mx_factor(byte), o);
  if (valid)
    *p = make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                    __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
}

// The product with a value's first part, with that of the rest (which is 0 where the
// first is infinite: times an infinite weight it would make a NaN of an infinity).
__device__ __forceinline__ float with_rest(float head, float rest) { return isfinite(head) ? head + rest : head; }

// CODEC 0: 16-bit weights (bf16, or f16 with OPT); 1: MXFP4 (bf16 products; OPT
// quantises x, of either 16-bit type).
// XS: a pass's part of x is copied to shared memory at once, behind the loads of
// the weights, instead of one dependent load a step.  For 16-bit weights and up
// to 8 tokens: a load in each of 11 steps took 2 us more (a block of 2816 x 2112
// at T = 1: 10.4 and 8.2 us).  With MXFP4 weights there are 3 steps, and the copy
// takes 0.4 us more than it saves, unless x is to be quantised for one token,
// which the CTA's threads then share (4224 x 2816 gated: T = 1 7.0 and 6.1 us,
// T = 4 7.2 and 8.3).
template <int CODEC, int NT8, bool GATED, bool OPT, bool XS>
__global__ void __launch_bounds__(kSkThreads, 2) skinny_kernel(SkinnyParams p) {
  constexpr bool F16 = CODEC == 0 && OPT, QX = CODEC == 1 && OPT;
  using C = SkCfg<CODEC, NT8, XS>;
  constexpr int U = C::U, XW = C::XW;
  extern __shared__ __align__(16) uint8_t xs[];
  auto red = reinterpret_cast<float4(*)[NT8][32]>(xs);  // behind the last pass
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  if (!p.after) {
    after_previous();
    let_next();
  }

  // this CTA's tokens
  const uint8_t* px = p.x + (size_t)blockIdx.y * (NT8 * 8) * p.ldx_bytes;
  uint16_t* py = p.y + (size_t)blockIdx.y * (NT8 * 8) * p.N;  // split: only one block of tokens
  const int T = p.T - (int)blockIdx.y * (NT8 * 8);

  const int row_a = GATED ? blockIdx.x * 8 + r : blockIdx.x * 16 + r;
  const int row_b = GATED ? row_a : row_a + 8;
  const bool ok_a = row_a < p.N, ok_b = row_b < p.N;
  const size_t pitch = (size_t)p.units * 16;
  const uint8_t* wa = p.w0 + (ok_a ? row_a : 0) * pitch;
  const uint8_t* wb = (GATED ? p.w1 : p.w0) + (ok_b ? row_b : 0) * pitch;
  const uint8_t* sa = CODEC == 1 ? p.s0 + (size_t)(ok_a ? row_a : 0) * p.units : nullptr;
  const uint8_t* sb = CODEC == 1 ? (GATED ? p.s1 : p.s0) + (size_t)(ok_b ? row_b : 0) * p.units : nullptr;

  float acc[NT8][4];
#pragma unroll
  for (int j = 0; j < NT8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

  const int steps = (p.units + 3) / 4;
  bool first = true;
  for (int base = 0; base < steps; base += kSkWarps * U) {
    const int s0 = base + warp;
    // pieces of a token in this pass
    const int u0 = 4 * base, n = min((p.units - u0) * XW, C::XPASS / 16), nt = min(T, NT8 * 8);
    auto copy_x = [&]() {
      for (int i = threadIdx.x; i < nt * n; i += kSkThreads) {
        const int t = i / n, k = i - t * n;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(xs + t * C::XPITCH + k * 16)),
                     "l"(px + (size_t)t * p.ldx_bytes + ((size_t)u0 * XW + k) * 16)
                     : "memory");
      }
    };
    if (XS && !first) __syncthreads();  // the pass before has read its part
    if (XS && (!first || !p.after)) copy_x();
    uint4 va[U], vb[U];
    uint32_t ca[U], cb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = 4 * (s0 + u * kSkWarps) + c;
      va[u] = vb[u] = make_uint4(0u, 0u, 0u, 0u);
      ca[u] = cb[u] = 0u;
      if (unit < p.units) {
        va[u] = ld_v4_stream(wa + (size_t)unit * 16);
        vb[u] = ld_v4_stream(wb + (size_t)unit * 16);
        if (CODEC == 1) {
          ca[u] = ld_u8(sa + unit);
          cb[u] = ld_u8(sb + unit);
        }
      }
    }
    if (first && p.after) {
      after_previous();
      let_next();
    }
    if constexpr (XS) {
      if (first && p.after) copy_x();
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
      if constexpr (QX) {
        for (int i0 = 0; i0 < nt * n; i0 += kSkThreads) {
          const int i = i0 + threadIdx.x, t = i / n, k = i - t * n;
          quantize_in_place(xs + t * C::XPITCH + k * 16, i < nt * n, p.f16);
        }
        __syncthreads();
      }
    }
    first = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = 4 * (s0 + u * kSkWarps) + c;
      if (4 * (s0 + u * kSkWarps) >= p.units) break;  // the same for the whole warp
      uint4 xv[NT8][XW];
#pragma unroll
      for (int j = 0; j < NT8; ++j) {
        const int t = j * 8 + r;
#pragma unroll
        for (int i = 0; i < XW; ++i) {
          xv[j][i] = make_uint4(0u, 0u, 0u, 0u);
          // plain loads: x may have been written by the kernel before
          if (XS && t < T && unit < p.units)
            xv[j][i] = *reinterpret_cast<const uint4*>(xs + t * C::XPITCH + ((unit - u0) * XW + i) * 16);
          if (!XS && t < T && unit < p.units)
            xv[j][i] = *reinterpret_cast<const uint4*>(px + (size_t)t * p.ldx_bytes + ((size_t)unit * XW + i) * 16);
        }
      }
      if constexpr (CODEC == 0) {
#pragma unroll
        for (int j = 0; j < NT8; ++j) {
          mma16<F16>(acc[j], va[u].x, vb[u].x, va[u].y, vb[u].y, xv[j][0].x, xv[j][0].y);
          mma16<F16>(acc[j], va[u].z, vb[u].z, va[u].w, vb[u].w, xv[j][0].z, xv[j][0].w);
        }
      } else {
        const MxFactor fa = mx_factor(ca[u]), fb = mx_factor(cb[u]);
        MxFactor fx[NT8];
        uint32_t xq[NT8][4];
        if constexpr (QX && !XS) {
#pragma unroll
          for (int j = 0; j < NT8; ++j) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&xv[j][0]);
            uint32_t m2 = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) m2 = __vmaxu2(m2, w[i] & 0x7FFF7FFFu);
            float lo, hi;
            unpack16x2(m2, p.f16, lo, hi);
            const uint32_t byte = mx_scale_byte(max(abs_bits(lo), abs_bits(hi)));
            fx[j] = mx_factor(byte);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) unpack16x2(w[4 * q + k], p.f16, v[2 * k], v[2 * k + 1]);
              xq[j][q] = mx_encode8(v, byte);
            }
          }
        }
        const uint32_t wav[4] = {va[u].x, va[u].y, va[u].z, va[u].w}, wbv[4] = {vb[u].x, vb[u].y, vb[u].z, vb[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t a[4], b[4];
          mx_decode8(wav[q], fa, a);
          mx_decode8(wbv[q], fb, b);
#pragma unroll
          for (int j = 0; j < NT8; ++j) {
            uint32_t o[4];
            if constexpr (QX && !XS) {
              mx_decode8(xq[j][q], fx[j], o);
            } else {
              const uint4 xw = xv[j][q];
              o[0] = __byte_perm(xw.x, xw.z, 0x5410);
              o[1] = __byte_perm(xw.x, xw.z, 0x7632);
              o[2] = __byte_perm(xw.y, xw.w, 0x5410);
              o[3] = __byte_perm(xw.y, xw.w, 0x7632);
            }
            mma16<false>(acc[j], a[0], b[0], a[1], b[1], o[0], o[1]);
            mma16<false>(acc[j], a[2], b[2], a[3], b[3], o[2], o[3]);
          }
        }
      }
    }
  }
  if (XS) __syncthreads();
#pragma unroll
  for (int j = 0; j < NT8; ++j) red[warp][j][lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
  __syncthreads();
  if (threadIdx.x < 32 * NT8) {
    const int j = threadIdx.x >> 5;
    float4 d = red[0][j][lane];
#pragma unroll
    for (int w = 1; w < kSkWarps; ++w) {
      const float4 e = red[w][j][lane];
      d.x += e.x; d.y += e.y; d.z += e.z; d.w += e.w;
    }
    const int t0 = j * 8 + 2 * c;
    if (CODEC == 0 && !GATED && p.split) {  // one token's two parts
      if (t0 < T) {
        uint16_t* y = py + (size_t)(t0 >> 1) * p.N;
        const uint32_t v = pack16x2(with_rest(d.x, d.y), with_rest(d.z, d.w), p.f16);
        if (ok_a) y[row_a] = (uint16_t)v;
        if (ok_b) y[row_b] = (uint16_t)(v >> 16);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + i;
      if (t >= T) break;
      const float v0 = i ? d.y : d.x, v1 = i ? d.w : d.z;
      uint16_t* y = py + (size_t)t * p.N;
      if (GATED) {
        const float h = act_fwd(v0, p.act) * v1;
        const uint32_t v = pack16x2(h, 0.f, p.f16);
        if (CODEC == 0 && p.split) {
          float head, zero;
          unpack16x2(v, p.f16, head, zero);
          y += (size_t)t * p.N;
          if (ok_a) y[p.N + row_a] = (uint16_t)pack16x2(isfinite(head) ? h - head : 0.f, 0.f, p.f16);
        }
        if (ok_a) y[row_a] = (uint16_t)v;
      } else {
        const uint32_t v = pack16x2(v0, v1, p.f16);
        if (ok_a) y[row_a] = (uint16_t)v;
        if (ok_b) y[row_b] = (uint16_t)(v >> 16);
      }
    }
  }
}

template <int CODEC, int NT8, bool GATED, bool OPT, bool XS>
cudaError_t launch_one(const SkinnyParams& p, cudaStream_t st) {
  auto fn = skinny_kernel<CODEC, NT8, GATED, OPT, XS>;
  using C = SkCfg<CODEC, NT8, XS>;
  cudaError_t err = configure_kernel_once((const void*)fn, C::smem(NT8 * 8));
  if (err != cudaSuccess) return err;
  const int rows = GATED ? 8 : 16;
  return launch_overlapped(fn, (unsigned)((p.N + rows - 1) / rows), (unsigned)((p.T + 31) / 32), kSkThreads,
                           C::smem(p.T), st, p);
}

template <int CODEC, bool GATED, bool OPT>
cudaError_t launch_nt(const SkinnyParams& p, cudaStream_t st) {
  constexpr bool QX = CODEC == 1 && OPT;
  if constexpr (QX) {
    if (p.T == 1) return launch_one<CODEC, 1, GATED, OPT, true>(p, st);
  }
  if (p.T <= 8) return launch_one<CODEC, 1, GATED, OPT, CODEC == 0>(p, st);
  if (p.T <= 16) return launch_one<CODEC, 2, GATED, OPT, false>(p, st);
  if constexpr (QX) return cudaErrorInvalidValue;  // skinny_fits_mx: at most 16 tokens
  else return launch_one<CODEC, 4, GATED, OPT, false>(p, st);
}

}  // namespace

// Measured against the tensor-core kernels (whole calls in a graph, us, few-token
// kernel / the other, N x K, `silu` gated).  With MXFP4 weights the crossing lies
// where the CTAs no longer fit the SMs at once (2 on each; up to 16 tokens not even
// there, the weights then being most of the time), or, with x quantised in every
// CTA, where there is more than one on an SM or K is long.
//   W4A16  T = 16:  2816 x 8192 14.0 / 24.4, 16384 x 2816 18.2 / 23.8 (four waves),
//                   8192 x 8192 27.1 / 35.3, 32768 x 1024 16.5 / 20.6
//          T = 24:  8192 x 2816 14.6 / 13.9 (two waves), 2816 x 8192 18.7 / 24.5
//          T = 32:  8192 x 2816 17.0 / 13.9, 2816 x 2112 7.9 / 9.1, 2816 x 8192 22.8 / 24.5
//          T = 64:  2816 x 2112 14.1 / 9.3 (two waves), 1024 x 1024 3.4 / 6.2
//          T = 128: 512 x 2816 silu 5.9 / 10.9 (one wave)
//   W4A4   T = 1:   2816 x 8192 12.0 / 12.2
//          T = 8:   4224 x 2816 silu 7.1 / 8.1, 8192 x 2816 11.9 / 8.8 (two waves),
//                   2816 x 8192 15.1 / 12.2 (long)
//          T = 16:  1024 x 1024 3.5 / 5.7 (a CTA an SM), 2816 x 2112 8.3 / 6.9 (two)
bool skinny_fits_mx(int T, int N, int K, bool gated, bool quant_x) {
  if (T > 128) return false;
  const int n = sms(), rows = gated ? 8 : 16;
  const int64_t ctas = (int64_t)((N + rows - 1) / rows) * ((T + 31) / 32);
  if (quant_x) return T <= 16 && ctas <= (T <= 8 ? 2 * n : n) && (T == 1 || K <= 4096);
  return T <= 16 || ctas <= 2 * n;
}

// The gated block, both products by one kernel or both by the other (a mixture
// is slower than either: the second then waits for the first).  T H I at the
// crossing, in millions, for I x H (weights not in L2): 1024 x 8192 270, 2112 x 2816
// 200, 2816 x 2112 70, 4096 x 1024 120, 4096 x 2816 130, 5632 x 2816 160; the limit is
// off by at most 3% of the time for these.  At T = 16: 2112 x 2816 15.1 / 18.9, 2816 x
// 2112 20.0 / 19.7, 1024 x 8192 25.4 / 29.9, 5632 x 2816 39.3 / 36.5.  At T = 8 the
// few-token kernel always (8192 x 2816 42.9 / 44.9), above 64 never (1024 x 1024
// at 96: 10.9 / 10.8).
bool skinny_fits_ffn(int T, int H, int I) {
  return T <= 8 || (T <= 64 && (int64_t)T * H * I <= 140000000);
}

// Whether the block, where it is this kernel's, keeps h in two 16-bit parts, so that y is off by its own
// rounding alone.  Rounded once to 16 bits, h leaves y 1.4 times that far from the
// exact one, and where few hidden units make up its sums up to 1.8 times.  Up to four
// tokens the second parts are columns that the tensor instruction has anyway (us, one
// part / two, weights not in L2, H x I: 2816 x 2112 T = 1 10.9 / 11.0, T = 4 11.6 / 12.0,
// 1024 x 4096 T = 4 12.8 / 14.0); for more the second product takes twice the tokens
// (T = 8: 2816 x 512 7.3 / 7.3, 1024 x 512 4.7 / 4.9, 2816 x 2112 12.6 / 14.9; T = 16:
// 2816 x 512 8.3 / 8.8).
bool skinny_splits_hidden(int T, int H, int I) {
  return skinny_fits_ffn(T, H, I) && (T <= 4 || (T <= 16 && I <= 512));
}

cudaError_t launch_skinny(const SkinnyArgs& a, cudaStream_t st) {
  if (a.split_x && a.split_y) return cudaErrorInvalidValue;
  const bool gated = a.act != kActNone;
  SkinnyParams p{};
  p.x = static_cast<const uint8_t*>(a.x);
  p.w0 = static_cast<const uint8_t*>(a.w0);
  p.w1 = static_cast<const uint8_t*>(a.w1);
  p.units = a.mx ? a.K / 32 : a.K / 8;
  p.s0 = a.scales;
  if (a.mx && gated) {
    p.w1 = p.w0 + (size_t)a.N * p.units * 16;
    p.s1 = p.s0 + (size_t)a.N * p.units;
  }
  p.y = static_cast<uint16_t*>(a.y);
  p.ldx_bytes = a.ldx * 2;
  p.T = a.T;
  p.N = a.N;
  p.act = a.act;
  p.f16 = a.dtype == kF16;
  p.after = a.after_producer;
  p.split = a.split_x || a.split_y;
  if (a.split_x) p.T = 2 * a.T;
  const bool opt = a.mx ? a.quant_x : p.f16;
  if (a.mx) {
    if (gated) return opt ? launch_nt<1, true, true>(p, st) : launch_nt<1, true, false>(p, st);
    return opt ? launch_nt<1, false, true>(p, st) : launch_nt<1, false, false>(p, st);
  }
  if (gated) return opt ? launch_nt<0, true, true>(p, st) : launch_nt<0, true, false>(p, st);
  return opt ? launch_nt<0, false, true>(p, st) : launch_nt<0, false, false>(p, st);
}

}  // namespace nvfp4moe
