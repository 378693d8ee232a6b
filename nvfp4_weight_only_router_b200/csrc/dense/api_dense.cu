// C ABI of the dense feed-forward operators: argument validation, workspace
// layout and launch sequencing on the caller's stream.  See
// include/nvfp4dense.h.
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <mutex>

#include "../../../include/nvfp4dense.h"
#include "dense_kernels.h"

using namespace nvfp4moe;

namespace {

// Per-device status word (see nvfp4dense_get_device_status).
__device__ int g_dense_status;

constexpr int kMaxDevices = 64;
int* g_status_ptr[kMaxDevices] = {};
std::mutex g_status_mu;

thread_local cudaError_t t_last_cuda_error = cudaSuccess;

nvfp4_status cuda_fail(cudaError_t e) {
  t_last_cuda_error = e != cudaSuccess ? e : cudaErrorUnknown;
  return NVFP4_ERR_CUDA;
}
nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : cuda_fail(e); }

}  // namespace

int* nvfp4moe::device_status_ptr() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_status_mu);
  if (!g_status_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_dense_status) != cudaSuccess) return nullptr;
    g_status_ptr[dev] = static_cast<int*>(p);
  }
  return g_status_ptr[dev];
}

int nvfp4moe::sms() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  n = known[dev].load(std::memory_order_relaxed);
  if (n) return n;
  if (sm_count(&n) != cudaSuccess) return 148;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

constexpr int32_t kMaxTokens = 1 << 20, kMaxDim = 1 << 18;

bool row_stride_ok(int64_t ld, int64_t row, int32_t T) { return T <= 1 || (ld >= row && ld <= (int64_t(1) << 32)); }

// ---------------------------------------------------------------- products
struct LinearLayout {
  size_t xq = 0, xsf = 0, wsf = 0, total = 256;
  int bn = 0;
};

nvfp4_status check_linear(int32_t T, const mxfp4_weight* w, int32_t act) {
  if (!w || !w->codes || !w->scales || T < 0 || act < kActNone || act > kActSilu) return NVFP4_ERR_INVALID_ARG;
  if (w->N < 1 || w->K < 1) return NVFP4_ERR_INVALID_ARG;
  if (T > kMaxTokens || w->N > kMaxDim || w->K > kMaxDim || w->K % 32 != 0 || w->N % (act ? 16 : 8) != 0)
    return NVFP4_ERR_UNSUPPORTED;
  if (!aligned(w->codes, 16) || !aligned(w->scales, 16)) return NVFP4_ERR_ALIGNMENT;
  return NVFP4_OK;
}

bool few_tokens(int32_t T, const mxfp4_weight* w, int32_t act, bool a4) {
  return skinny_fits_mx(T, act ? w->N / 2 : w->N, w->K, act != kActNone, a4);
}

// W4A16 of many tokens: the weight as bf16
size_t linear_bytes(int32_t T, const mxfp4_weight* w) {
  return T <= kPairW4MaxTokens ? 256 : round_up((size_t)w->N * w->K * 2, 256);
}

LinearLayout a4_layout(int32_t T, const mxfp4_weight* w, int32_t act) {
  LinearLayout L;
  if (few_tokens(T, w, act, true)) return L;
  const int n = act ? w->N / 2 : w->N;
  L.bn = pair_mx_tile(T, n, w->K, act);
  const size_t chunks = (size_t)mx_sf_chunks(w->K) * kSfChunkB;
  L.xsf = round_up((size_t)T * mx_pitch(w->K), 256);
  L.wsf = L.xsf + (size_t)((T + 127) / 128) * chunks;
  L.total = L.wsf + (size_t)mx_wsf_blocks(n, act != kActNone, L.bn) * chunks;
  return L;
}

nvfp4_status linear_checks(const void* x, int32_t dtype, int64_t ldx, int32_t T, const mxfp4_weight* w,
                           const void* y, const void* ws, size_t ws_bytes, size_t need, bool a4) {
  if (T > 0 && (!x || !y)) return NVFP4_ERR_INVALID_ARG;
  if (dtype < kBf16 || dtype > kF32) return NVFP4_ERR_INVALID_ARG;
  if (dtype == kF32 || (!a4 && dtype != kBf16)) return NVFP4_ERR_UNSUPPORTED;
  if (!row_stride_ok(ldx, w->K, T)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || (T > 1 && ldx % 8 != 0)) return NVFP4_ERR_ALIGNMENT;
  if (need > 256 && (!ws || ws_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return NVFP4_ERR_ALIGNMENT;
  return NVFP4_OK;
}

SkinnyArgs skinny_mx(const void* x, int64_t ldx, int32_t T, const mxfp4_weight* w, int32_t act, int32_t dtype, void* y,
                     bool quant_x) {
  SkinnyArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.w0 = w->codes;
  a.scales = w->scales;
  a.y = y;
  a.T = T;
  a.N = act ? w->N / 2 : w->N;
  a.K = w->K;
  a.act = act;
  a.dtype = dtype;
  a.mx = true;
  a.quant_x = quant_x;
  return a;
}

// -------------------------------------------------------------- feed-forward
nvfp4_status check_ffn(int32_t T, const gated_ffn_weights* f) {
  if (!f || !f->gate || !f->up || !f->down || T < 0 || f->H < 1 || f->I < 1) return NVFP4_ERR_INVALID_ARG;
  if (f->act < kActNone || f->act > kActSilu || f->dtype < kBf16 || f->dtype > kF32) return NVFP4_ERR_INVALID_ARG;
  if (f->act == kActNone || f->dtype == kF32) return NVFP4_ERR_UNSUPPORTED;
  if (T > kMaxTokens || f->H > kMaxDim || f->I > kMaxDim || f->H % 8 != 0 || f->I % 8 != 0)
    return NVFP4_ERR_UNSUPPORTED;
  if (!aligned(f->gate, 16) || !aligned(f->up, 16) || !aligned(f->down, 16)) return NVFP4_ERR_ALIGNMENT;
  return NVFP4_OK;
}

PairOperand rows_of(const void* p, int64_t ld) { return PairOperand{p, ld, false}; }
PairOperand cols_of(const void* p, int64_t ld) { return PairOperand{p, ld, true}; }

}  // namespace

int nvfp4moe::fail_cuda(cudaError_t e) { return cuda_fail(e); }

extern "C" {

int nvfp4dense_abi_version(void) { return NVFP4DENSE_ABI_VERSION; }

const char* nvfp4dense_last_cuda_error(void) { return cudaGetErrorString(t_last_cuda_error); }

nvfp4_status nvfp4dense_get_device_status(void* stream) {
  int* p = device_status_ptr();
  if (!p) return cuda_fail(cudaGetLastError());
  int v = 0;
  if (cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) return cuda_fail(cudaGetLastError());
  if (cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return cuda_fail(cudaGetLastError());
  if (v != 0 && cudaMemset(p, 0, sizeof(int)) != cudaSuccess) return cuda_fail(cudaGetLastError());
  return static_cast<nvfp4_status>(v);
}

// ---------------------------------------------------------------- quantise
static nvfp4_status check_mx_dims(int64_t rows, int64_t K) {
  if (rows < 0 || K < 1) return NVFP4_ERR_INVALID_ARG;
  if (rows > 0x7FFFFFFF || K >= (int64_t(1) << 24) || rows * K >= (int64_t(1) << 40))
    return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

nvfp4_status mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                            uint8_t* scales, void* stream) {
  NvtxRange nv("mxfp4_quantize");
  nvfp4_status st = check_mx_dims(rows, K);
  if (st != NVFP4_OK) return st;
  if (dtype < kBf16 || dtype > kF32) return NVFP4_ERR_INVALID_ARG;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !scales || (rows > 1 && (ldx < K || ldx > (int64_t(1) << 32)))) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(x, dtype == kF32 ? 4 : 2) || !aligned(codes, 16) || !aligned(scales, 16)) return NVFP4_ERR_ALIGNMENT;
  return cuda_status(launch_mxfp4_quantize(x, dtype, rows, K, rows > 1 ? ldx : round_up(K, 8), codes, scales,
                                           as_stream(stream)));
}

nvfp4_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* out,
                              int32_t dtype, void* stream) {
  NvtxRange nv("mxfp4_dequantize");
  nvfp4_status st = check_mx_dims(rows, K);
  if (st != NVFP4_OK) return st;
  if (dtype < kBf16 || dtype > kF32) return NVFP4_ERR_INVALID_ARG;
  if (dtype == kF16) return NVFP4_ERR_UNSUPPORTED;  // f16 does not hold the format's range
  if (rows == 0) return NVFP4_OK;
  if (!codes || !scales || !out) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16)) return NVFP4_ERR_ALIGNMENT;
  return cuda_status(launch_mxfp4_dequantize(codes, scales, rows, K, out, dtype, as_stream(stream)));
}

// ---------------------------------------------------------------- products
size_t mxfp4_linear_workspace_bytes(int32_t T, const mxfp4_weight* w, int32_t act) {
  return check_linear(T, w, act) == NVFP4_OK ? linear_bytes(T, w) : 0;
}

nvfp4_status mxfp4_linear(const void* x, int32_t dtype, int64_t ldx, int32_t T, const mxfp4_weight* w, int32_t act,
                          void* y, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nv("mxfp4_linear");
  nvfp4_status st = check_linear(T, w, act);
  if (st != NVFP4_OK) return st;
  st = linear_checks(x, dtype, ldx, T, w, y, ws, ws_bytes, linear_bytes(T, w), false);
  if (st != NVFP4_OK || T == 0) return st;
  if (T == 1) ldx = w->K;
  cudaStream_t s = as_stream(stream);
  if (few_tokens(T, w, act, false)) return cuda_status(launch_skinny(skinny_mx(x, ldx, T, w, act, dtype, y, false), s));
  if (T <= kPairW4MaxTokens) {
    const PairW4 a{x, ldx, w->codes, w->scales, T, act ? w->N / 2 : w->N, w->K, act, y};
    return cuda_status(launch_pair_w4(a, device_status_ptr(), s));
  }
  cudaError_t e = launch_mxfp4_dequantize(w->codes, w->scales, w->N, w->K, ws, kBf16, s);
  if (e != cudaSuccess) return cuda_fail(e);
  if (act) {
    PairGated a{};
    a.x = x;
    a.ldx = ldx;
    a.gate = ws;
    a.up = static_cast<const uint16_t*>(ws) + (size_t)(w->N / 2) * w->K;
    a.ldw = w->K;
    a.T = T;
    a.I = w->N / 2;
    a.K = w->K;
    a.act = act;
    a.dtype = kBf16;
    a.h = y;
    a.ldh = a.I;
    return cuda_status(launch_pair_gated(a, device_status_ptr(), s));
  }
  PairGemm g{};
  g.seg[0] = PairSegment{rows_of(x, ldx), rows_of(ws, w->K), w->K};
  g.nseg = 1;
  g.M = T;
  g.N = w->N;
  g.out = y;
  return cuda_status(launch_pair_gemm(&g, 1, kBf16, device_status_ptr(), s));
}

size_t mxfp4_linear_a4_workspace_bytes(int32_t T, const mxfp4_weight* w, int32_t act) {
  return check_linear(T, w, act) == NVFP4_OK ? a4_layout(T, w, act).total : 0;
}

nvfp4_status mxfp4_linear_a4(const void* x, int32_t dtype, int64_t ldx, int32_t T, const mxfp4_weight* w, int32_t act,
                             void* y, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nv("mxfp4_linear_a4");
  nvfp4_status st = check_linear(T, w, act);
  if (st != NVFP4_OK) return st;
  const LinearLayout L = a4_layout(T, w, act);
  st = linear_checks(x, dtype, ldx, T, w, y, ws, ws_bytes, L.total, true);
  if (st != NVFP4_OK || T == 0) return st;
  if (T == 1) ldx = w->K;
  cudaStream_t s = as_stream(stream);
  if (few_tokens(T, w, act, true)) return cuda_status(launch_skinny(skinny_mx(x, ldx, T, w, act, dtype, y, true), s));
  uint8_t* base = static_cast<uint8_t*>(ws);
  MxPrepArgs pa{};
  pa.x = x;
  pa.dtype = dtype;
  pa.T = T;
  pa.K = w->K;
  pa.ldx = ldx;
  pa.xq = base + L.xq;
  pa.xsf = base + L.xsf;
  pa.wscales = w->scales;
  pa.N = act ? w->N / 2 : w->N;
  pa.gated = act != kActNone;
  pa.bn = L.bn;
  pa.wsf = base + L.wsf;
  cudaError_t e = launch_mxfp4_prep_a4(pa, s);
  if (e != cudaSuccess) return cuda_fail(e);
  PairMx m{};
  m.xq = pa.xq;
  m.xsf = pa.xsf;
  m.wq = w->codes;
  m.wsf = pa.wsf;
  m.T = T;
  m.N = pa.N;
  m.K = w->K;
  m.act = act;
  m.dtype = dtype;
  m.bn = L.bn;
  m.y = y;
  return cuda_status(launch_pair_mx(m, device_status_ptr(), s));
}

// -------------------------------------------------------------- feed-forward
size_t gated_ffn_saved_bytes(int32_t T, const gated_ffn_weights* f) {
  if (check_ffn(T, f) != NVFP4_OK) return 0;
  return T == 0 ? 256 : pair_kept(nullptr, T, f->I).bytes;
}

size_t gated_ffn_forward_workspace_bytes(int32_t T, const gated_ffn_weights* f) {
  // h, in two parts for few tokens
  return check_ffn(T, f) == NVFP4_OK
             ? round_up((size_t)T * pair_pitch(f->I) * (skinny_splits_hidden(T, f->H, f->I) ? 4 : 2) + 1, 256) : 0;
}

nvfp4_status gated_ffn_forward(const void* x, int64_t ldx, int32_t T, const gated_ffn_weights* f, void* y, void* saved,
                               void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nv("gated_ffn_forward");
  nvfp4_status st = check_ffn(T, f);
  if (st != NVFP4_OK) return st;
  if ((T > 0 && (!x || !y)) || !row_stride_ok(ldx, f->H, T)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(saved, 256) || (T > 1 && ldx % 8 != 0)) return NVFP4_ERR_ALIGNMENT;
  if (!saved) {
    if (!ws || ws_bytes < gated_ffn_forward_workspace_bytes(T, f)) return NVFP4_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return NVFP4_ERR_ALIGNMENT;
  }
  if (T == 0) return NVFP4_OK;
  if (T == 1) ldx = f->H;
  cudaStream_t s = as_stream(stream);
  int* status = device_status_ptr();
  void* const h = saved ? saved : ws;
  const bool fits = skinny_fits_ffn(T, f->H, f->I), few = fits && !saved;  // what is kept: only by the other kernel
  const bool split = few && skinny_splits_hidden(T, f->H, f->I);
  const int64_t ldh = few ? f->I : pair_pitch(f->I);
  cudaError_t e;
  if (few) {
    SkinnyArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.w0 = f->gate;
    a.w1 = f->up;
    a.y = h;
    a.T = T;
    a.N = f->I;
    a.K = f->H;
    a.act = f->act;
    a.dtype = f->dtype;
    a.split_y = split;
    e = launch_skinny(a, s);
  } else {
    PairGated a{};
    a.x = x;
    a.ldx = ldx;
    a.gate = f->gate;
    a.up = f->up;
    a.ldw = f->H;
    a.T = T;
    a.I = f->I;
    a.K = f->H;
    a.act = f->act;
    a.dtype = f->dtype;
    a.h = h;
    a.ldh = ldh;
    a.keep = saved != nullptr;
    a.kept = pair_kept(saved, T, f->I);
    e = launch_pair_gated(a, status, s);
  }
  if (e != cudaSuccess) return cuda_fail(e);
  if (fits) {
    SkinnyArgs a{};
    a.x = h;
    a.ldx = ldh;
    a.w0 = f->down;
    a.y = y;
    a.T = T;
    a.N = f->H;
    a.K = f->I;
    a.act = kActNone;
    a.dtype = f->dtype;
    a.after_producer = true;
    a.split_x = split;
    return cuda_status(launch_skinny(a, s));
  }
  PairGemm g{};
  g.seg[0] = PairSegment{rows_of(h, ldh), rows_of(f->down, f->I), f->I};
  g.nseg = 1;
  g.M = T;
  g.N = f->H;
  g.out = y;
  return cuda_status(launch_pair_gemm(&g, 1, f->dtype, status, s));
}

size_t gated_ffn_backward_workspace_bytes(int32_t T, const gated_ffn_weights* f) {
  return check_ffn(T, f) == NVFP4_OK ? round_up(2 * round_up((size_t)T * pair_pitch(f->I) * 2, 256) + 1, 256) : 0;
}

nvfp4_status gated_ffn_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* saved, int32_t T,
                                const gated_ffn_weights* f, void* dx, void* dgate, void* dup, void* ddown, void* ws,
                                size_t ws_bytes, void* stream) {
  NvtxRange nv("gated_ffn_backward");
  nvfp4_status st = check_ffn(T, f);
  if (st != NVFP4_OK) return st;
  if (T > 0 && (!dy || !x || !saved)) return NVFP4_ERR_INVALID_ARG;
  if (!row_stride_ok(lddy, f->H, T) || !row_stride_ok(ldx, f->H, T)) return NVFP4_ERR_INVALID_ARG;
  const void* ps[] = {dy, x, dx, dgate, dup, ddown};
  for (const void* p : ps)
    if (!aligned(p, 16)) return NVFP4_ERR_ALIGNMENT;
  if (!aligned(saved, 256)) return NVFP4_ERR_ALIGNMENT;
  if (T > 1 && (ldx % 8 != 0 || lddy % 8 != 0)) return NVFP4_ERR_ALIGNMENT;
  if (!ws || ws_bytes < gated_ffn_backward_workspace_bytes(T, f)) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return NVFP4_ERR_ALIGNMENT;
  cudaStream_t s = as_stream(stream);
  const int H = f->H, I = f->I;
  if (T == 0) {  // empty sums
    for (void* p : {dgate, dup, ddown})
      if (p) {
        const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)H * I * 2, s);
        if (e != cudaSuccess) return cuda_fail(e);
      }
    return NVFP4_OK;
  }
  if (T == 1) ldx = lddy = H;
  const int64_t ldi = pair_pitch(I);
  const PairKept kept = pair_kept(const_cast<void*>(saved), T, I);
  uint16_t* dg = static_cast<uint16_t*>(ws);
  uint16_t* du = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + round_up((size_t)T * ldi * 2, 256));
  int* status = device_status_ptr();
  if (dx || dgate || dup) {
    PairGatedBwd a{};
    a.dy = dy;
    a.lddy = lddy;
    a.down = f->down;
    a.T = T;
    a.H = H;
    a.I = I;
    a.dtype = f->dtype;
    a.kept = kept;
    a.dg = dg;
    a.du = du;
    const cudaError_t e = launch_pair_gated_bwd(a, status, s);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  PairGemm q[4];
  int n = 0;
  if (dx) {
    PairGemm& p = q[n++];
    p.seg[0] = PairSegment{rows_of(dg, ldi), cols_of(f->gate, H), I};
    p.seg[1] = PairSegment{rows_of(du, ldi), cols_of(f->up, H), I};
    p.nseg = 2;
    p.M = T;
    p.N = H;
    p.out = dx;
  }
  auto weight_grad = [&](const void* a, int64_t lda, const void* b, int64_t ldb, int M, int N, void* out) {
    PairGemm& p = q[n++];
    p.seg[0] = PairSegment{cols_of(a, lda), cols_of(b, ldb), T};
    p.nseg = 1;
    p.M = M;
    p.N = N;
    p.out = out;
  };
  if (dgate) weight_grad(dg, ldi, x, ldx, I, H, dgate);
  if (dup) weight_grad(du, ldi, x, ldx, I, H, dup);
  if (ddown) weight_grad(dy, lddy, kept.h, ldi, H, I, ddown);
  if (n == 0) return NVFP4_OK;
  return cuda_status(launch_pair_gemm(q, n, f->dtype, status, s));
}

}  // extern "C"
