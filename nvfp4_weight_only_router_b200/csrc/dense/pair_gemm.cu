// Dense products on the 5th-generation tensor cores, two SMs per tile
// (cta_group::2): D[256 rows, BN columns] += A[256, k] B[BN, k]^T with fp32
// accumulators in tensor memory.  16-bit operands (kind::f16, 64 elements of K
// per sub-stage), 16-bit by MXFP4 weights decoded into the stages (the same
// products), or MXFP4 operands (kind::mxf4, E2M1 with an E8M0 scale per 32, 256
// elements per sub-stage).
//
// Bound by the tensor pipe at 256 columns (512 cycles per 64 of K; 4096 x 4224 x
// 2816 in 58.7 us, 1.66 PFLOP/s), at fewer by what issues a stage and by the
// copies: a pair of SMs shares one B tile (each loads half of it), so that every
// byte of A and B feeds 256 rows or BN columns, and a copy takes about 1.3
// cycles per line and SM.  MXFP4 at 192 columns takes 480 to 530 cycles per 256
// of K: 384 for the products and about 24 for each of the six copies of scales,
// which share the tensor pipe (a warp of their own for the scales' loads, or one
// for each side's copies, changed nothing).
//
// Forms:
//   plain   out = sum over K segments A B^T, 16-bit; several products in one
//           launch (their tiles in one list, so that the last wave of one is
//           filled by the next).  An operand may be stored with K outermost
//           (the transposes of a backward pass); TMA then brings 64 x 64
//           boxes and the descriptors say M- or N-major.
//   gated   B's halves are gate rows and up rows of the same hidden units (SM 0
//           loads the gate half, SM 1 the up half); each accumulator row then
//           holds both, and the epilogue writes h = act(g) u and, if kept for
//           the backward pass, p = u act'(g) and a = act(g).
//   gated backward   the accumulators are dh; the epilogue reads p and a and
//           writes dg = dh p and du = dh a, so dh never leaves the chip.
//
// Warps: 0 and 2 TMA producers of A and B (in both SMs), 1 MMA issuer (in SM 0
// of the pair), 3 MXFP4 scales into tensor memory (likewise, ahead of the
// products, whose issue they would delay), 4-11 epilogue: a warp per
// tensor-memory lane quarter and column half, 12-19 (MXFP4 weights by 16-bit
// rows) converters of B, whose producer then shares A's work.  Two accumulators, so that a
// tile's epilogue overlaps the next tile's products (MXFP4 tiles have at most
// 192 columns: scales need tensor memory too).  Every wait is bounded in wall
// time; one that gives up records a timeout and the pair tears down.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "../tc_common.cuh"
#include "mxfp4_codec.cuh"

namespace nvfp4moe {

namespace {

constexpr int kPProdA = 0, kPMma = 1, kPProdB = 2, kPScale = 3, kPEpi0 = 4, kPEpiWarps = 8;
constexpr int kPConv0 = 12, kPConvWarps = 8, kPConvPer = 2;  // W4: warps, and warps of a stage
constexpr int kPTmem = 512;
constexpr int kPOutB = 4096;  // output buffer of an epilogue warp: 32 rows x 64 columns
constexpr int kKind16 = 0, kKindMx = 1, kKindW4 = 2;
constexpr int kEpiPlain = 0, kEpiGated = 1, kEpiGatedBwd = 2;

template <int KIND, int BN>
struct PCfg {
  static constexpr int THREADS = 32 * (KIND == kKindW4 ? kPConv0 + kPConvWarps : kPConv0);
  // sub-stages of 128 bytes of K per stage: a stage's waits and commits take
  // about 320 cycles, more than the products of 64 x up to 128 columns
  static constexpr int KS = BN <= 128 ? 2 : 1;
  static constexpr int A_SUB = 128 * 128, B_SUB = BN / 2 * 128;
  static constexpr int SFB_BLK = (BN + 127) / 128;                  // 128-row scale blocks of B
  static constexpr int SFA_SUB = KIND == kKindMx ? 2 * kSfChunkB : 0;
  static constexpr int SFB_SUB = KIND == kKindMx ? SFB_BLK * 2 * kSfChunkB : 0;
  static constexpr int STAGE = KS * (A_SUB + B_SUB + SFA_SUB + SFB_SUB);
  static constexpr int SF_COL0 = 2 * BN;                            // behind the two accumulators
  static constexpr int SF_COLS = KIND == kKindMx ? 8 + 8 * SFB_BLK : 0;  // per sub-stage
  static constexpr int NS_SMEM = (225 * 1024 - kPEpiWarps * kPOutB) / STAGE;
  static constexpr int NS_TMEM = KIND == kKindMx ? (kPTmem - SF_COL0) / (KS * SF_COLS) : 8;
  static constexpr int NS = NS_SMEM < NS_TMEM ? NS_SMEM : NS_TMEM;
  static_assert(NS >= 3 && SF_COL0 + NS * KS * SF_COLS <= kPTmem, "tensor memory");
};

template <int KIND, int BN>
struct alignas(1024) PSmem {
  using C = PCfg<KIND, BN>;
  uint8_t a[C::NS][C::KS][C::A_SUB];
  uint8_t b[C::NS][C::KS][C::B_SUB];
  uint8_t out[kPEpiWarps][kPOutB];     // output on its way to global memory
  uint8_t sfa[KIND == kKindMx ? C::NS : 1][KIND == kKindMx ? C::KS * C::SFA_SUB : 16];
  uint8_t sfb[KIND == kKindMx ? C::NS : 1][KIND == kKindMx ? C::KS * C::SFB_SUB : 16];
  uint64_t full[C::NS], empty[C::NS];  // full: SM 0's barrier counts both SMs' bytes
  uint64_t scaled[C::NS];              // MXFP4: the stage's scales are in tensor memory
  uint64_t d_full[2], d_empty[2];      // d_empty: SM 0's, arrivals of both SMs' epilogues
  uint64_t fin, fin_sf;
  uint32_t taddr;
  int abort_flag;
  int issued[2];                       // stages behind the producers
};

struct alignas(64) PProb {
  CUtensorMap a[2], b[2];  // by K segment; gated: b[0] gate rows, b[1] up rows
  CUtensorMap o[2];        // output; gated backward: dg, du
  int M, N;                // output rows and columns
  int kc0, kc;             // K stages of segment 0 and in all
  int tm, t0;              // tiles along M; first tile in the list
  int a_mn, b_mn;
  const uint8_t *wq, *ws;  // W4: codes and scales of B's rows (gated: gate, then up)
  int K;                   // W4
  int tx;                  // bytes of a stage that complete on the barrier, of both SMs
};

struct PEpi {
  uint8_t* kept;           // PairKept's blocks (null: not kept)
  int act, f16;
  int ksteps;              // MXFP4: MMA steps of 64 along K
};

template <int NP>
struct alignas(64) PParams {
  PProb p[NP];
  CUtensorMap sfa, sfb;    // MXFP4 scale chunks
  PEpi e;
  int np, n_tiles;
  int* status;
};

// ------------------------------------------------------------------ PTX forms
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Execution order only: barrier initialisation has its own fence, and at the
// end each SM has waited for every arrival that the other, or a commit, sends to
// its barriers (the releasing form takes 1000 cycles, and would not order the
// commits' arrivals).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// A pair that gave up has not: this one orders what its threads did before.
__device__ __forceinline__ void cluster_sync_ordered() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// shared::cluster address of `p` in SM 0 of the pair
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t n) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(n)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t n) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(n) : "memory");
}
// One lane of a converged warp.  Copies, products and commits are issued by
// the branch that it selects, from a loop that the whole warp runs: a loop in
// one lane (or an election for each instruction) took 470 to 680 cycles a
// stage where the products take 512 (256 columns) or less.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}
// into this SM's shared memory, completing on SM 0's barrier
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t* bar) {  // arrives in both SMs
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_here(uint64_t* bar) {  // arrives in this SM
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// On a barrier of either SM, of an epilogue that has read its accumulator: what is
// ordered is tensor memory alone, by the tcgen05 fences on both sides; a release
// at cluster scope would order all memory, about 1000 cycles each time.
__device__ __forceinline__ void arrive_read(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same of a converter that has written shared memory for products which a
// thread of the other SM issues: a release that this thread observes.
__device__ __forceinline__ void arrive_written(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void mma16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc), "r"(sfa), "r"(sfb)
      : "memory");
}
// a 512-byte scale chunk of each SM's shared memory into its tensor memory
__device__ __forceinline__ void cp_sf_pair(uint32_t taddr, uint32_t smem_addr) {
  uint64_t d = (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)1u << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// Descriptor of an operand stored with K outermost: boxes of 64 (M or N) x 64
// (K), 128-byte swizzled rows.  8-row atoms 1024 bytes apart along K (stride
// offset), boxes 8192 bytes apart along M or N (leading offset).
__device__ __forceinline__ uint64_t make_mn_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(8192u >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

template <int KIND, int BN>
__device__ __forceinline__ bool pwait(PSmem<KIND, BN>& sm, uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_wait_bounded(bar, parity)) return true;
  atomicExch(&sm.abort_flag, 1);
  record_status(status, kStatusTimeout);
  return false;
}

struct PTile {
  int prob, m, n;
};
// A stage's barrier (completed by copies and tcgen05.commit, whose data only
// the asynchronous engines touch), waited for by a whole warp.
template <int KIND, int BN>
__device__ __forceinline__ bool swait(PSmem<KIND, BN>& sm, uint64_t* bar, uint32_t parity, int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, pwait(sm, bar, parity, status));
}
// The same for a stage that converters of both SMs have written: the phase has
// completed, so that the acquiring test succeeds at once.
template <int KIND, int BN>
__device__ __forceinline__ bool swait_written(PSmem<KIND, BN>& sm, uint64_t* bar, uint32_t parity, int* status) {
  if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
  return swait(sm, bar, parity, status) && __all_sync(0xffffffffu, try_wait_cluster(bar, parity));
}

template <int NP>
__device__ __forceinline__ PTile ptile(const PParams<NP>& p, int t) {
  PTile r;
  r.prob = 0;
#pragma unroll
  for (int i = 1; i < NP; ++i)
    if (i < p.np && t >= p.p[i].t0) r.prob = i;
  const int l = t - p.p[r.prob].t0, tm = p.p[r.prob].tm;
  r.m = l % tm;
  r.n = l / tm;
  return r;
}

// ---- output.  A lane holds columns of one row; 32-byte stores of 32 rows are
// 32 lines an instruction (6500 cycles for a 256 x 256 tile, exposed behind the
// last one), so a warp lays CW columns of its rows out in shared memory, in the
// swizzle that keeps both sides free of conflicts, and a TMA store writes them
// as whole lines and leaves what lies past the edges alone.
template <int CW>
struct POut {
  static constexpr int BYTES = 32 * CW * 2, BUFS = kPOutB / BYTES;
  static constexpr CUtensorMapSwizzle SW = CW == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                           : CW == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_32B;
  // 16 columns (group g of CW / 16) of row `lane`
  static __device__ __forceinline__ void put(uint8_t* buf, int lane, int g, const uint32_t (&w)[8]) {
    const int x = CW == 64 ? lane & 7 : CW == 32 ? (lane >> 1) & 3 : (lane >> 2) & 1;
    uint8_t* r = buf + lane * (CW * 2);
    *reinterpret_cast<uint4*>(r + ((2 * g) ^ x) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(r + ((2 * g + 1) ^ x) * 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
};
// at most `left` of the warp's earlier stores still read their buffers
template <int LEFT>
__device__ __forceinline__ void out_reuse(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
  __syncwarp();
}
__device__ __forceinline__ void out_ready() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const uint8_t* buf, int n, int row) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(n), "r"(row), "r"(smem_u32(buf))
               : "memory");
}
__device__ __forceinline__ void out_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// p and a of 16 hidden units of one row
struct Kept16 {
  uint32_t ph[8], ah[8], pl[4], al[4];
};
// the lane's part of a kept block
__device__ __forceinline__ void kept_load(const uint8_t* blk, int lane, Kept16& k) {
  ld_v8_stream(blk + lane * 32, k.ph);
  ld_v8_stream(blk + 1024 + lane * 32, k.ah);
  const uint4 a = ld_v4_stream(blk + 2048 + lane * 16), b = ld_v4_stream(blk + 2560 + lane * 16);
  k.pl[0] = a.x; k.pl[1] = a.y; k.pl[2] = a.z; k.pl[3] = a.w;
  k.al[0] = b.x; k.al[1] = b.y; k.al[2] = b.z; k.al[3] = b.w;
}
__device__ __forceinline__ void kept_store(uint8_t* blk, int lane, const Kept16& k) {
  st_v8(blk + lane * 32, k.ph);
  st_v8(blk + 1024 + lane * 32, k.ah);
  *reinterpret_cast<uint4*>(blk + 2048 + lane * 16) = make_uint4(k.pl[0], k.pl[1], k.pl[2], k.pl[3]);
  *reinterpret_cast<uint4*>(blk + 2560 + lane * 16) = make_uint4(k.al[0], k.al[1], k.al[2], k.al[3]);
}

__device__ __forceinline__ void pack16(const float* v, bool f16, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack16x2(v[2 * i], v[2 * i + 1], f16);
}

// Epilogue of 16 hidden units of a row: h packed into w, and p and a written
// where kept (blk, null where the warp's rows or the units lie outside).
template <bool KEEP>  // whether e.kept may be given
__device__ __forceinline__ void gate16(const PEpi& e, uint8_t* blk, int lane, const float* g, const float* u, bool f16,
                                       uint32_t (&w)[8]) {
  float v[16];
  if (!KEEP || !e.kept) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = act_fwd(g[i], e.act) * u[i];
  } else {
    float p[16];
    Kept16 k;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float da;
      act_fwd_grad(g[i], e.act, v[i], da);
      p[i] = u[i] * da;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      k.ph[i] = keep_hi2(p[2 * i], p[2 * i + 1]);
      k.ah[i] = keep_hi2(v[2 * i], v[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k.pl[i] = keep_lo4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
      k.al[i] = keep_lo4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    if (blk) kept_store(blk, lane, k);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= u[i];
  }
  pack16(v, f16, w);
}

template <int KIND, int BN, int EPI, int NP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PCfg<KIND, BN>::THREADS, 1)
    pair_gemm_kernel(const __grid_constant__ PParams<NP> p) {
  using C = PCfg<KIND, BN>;
  using Smem = PSmem<KIND, BN>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

  // The first tile's description and descriptors are fetched while the pair
  // sets up: cold, they took 3300 cycles behind it.
  PTile tile = ptile<NP>(p, cluster);
  if (warp == kPProdA || warp == kPProdB) {
    const PProb& q = p.p[tile.prob];
    if (elect_one()) {
      prefetch_map(warp == kPProdA || KIND == kKindW4 ? &q.a[0] : &q.b[EPI == kEpiGated ? rank : 0]);
      if (KIND == kKindMx) prefetch_map(warp == kPProdA ? &p.sfa : &p.sfb);
    }
    __syncwarp();
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      // W4: SM 0's producer and the converters of each SM
      mbar_init(&sm.full[s], KIND == kKindW4 ? 1 + 2 * kPConvPer : 1);
      mbar_init(&sm.empty[s], 1);
      mbar_init(&sm.scaled[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.d_full[b], 1);
      mbar_init(&sm.d_empty[b], 2 * kPEpiWarps);
    }
    mbar_init(&sm.fin, 1);
    mbar_init(&sm.fin_sf, 1);
    sm.abort_flag = 0;
    sm.issued[0] = sm.issued[1] = 0;
    fence_mbar_init();
  }
  if (warp == kPMma) {
    tmem_alloc2(&sm.taddr, kPTmem);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t taddr = sm.taddr;
  after_previous();
  let_next();

  if (warp == kPProdA || warp == kPProdB) {
    // ------------------------------------------- TMA producers of A and of B
    // W4: both of A, a stage each in turn.  A warp takes 550 cycles for a stage's
    // wait, arrival and two copies, whatever their size, nearly as long as the
    // converters (64 columns: about 600 cycles a stage, the release of SM 1's part
    // 1000 of the 2400 that a stage's four are shared by).
    const bool is_a = warp == kPProdA || KIND == kKindW4;
    const int turn = warp == kPProdB;
    const uint32_t full0 = leader_addr(&sm.full[0]), op0 = smem_u32(is_a ? sm.a[0][0] : sm.b[0][0]);
    const uint32_t sf0 = smem_u32(is_a ? sm.sfa[0] : sm.sfb[0]);
    uint32_t s = 0, parity = 1;  // the first pass finds every stage free
    int issued = 0;
    bool ok = true;
    for (int t = cluster; t < p.n_tiles && ok; t += clusters) {
      if (t != cluster) tile = ptile<NP>(p, t);
      const PTile d = tile;
      const PProb& q = p.p[d.prob];
      const int kc_all = q.kc, kc0 = q.kc0, tx = q.tx;
      // SM 1 has no rows of A where M ends in SM 0: what its shared memory holds
      // in their place only reaches accumulator rows that are not stored
      const bool has = !is_a || rank == 0 || q.M > 128;
      // first row (M or N) of this SM's part, and of its scales
      const int row = is_a ? d.m * 256 + (int)rank * 128
                           : EPI == kEpiGated ? d.n * (BN / 2) : d.n * BN + (int)rank * (BN / 2);
      const int sf_row = is_a ? row >> 7 : d.n * C::SFB_BLK;
      const bool mn = KIND != kKindMx && (is_a ? q.a_mn : BN >= 128 && q.b_mn);
      const int boxes = is_a ? 2 : BN / 128;  // 64-row boxes of an operand with K outermost
      const CUtensorMap* map = is_a ? &q.a[0] : &q.b[EPI == kEpiGated ? rank : 0];
      for (int kc = 0, kk = 0; kc < kc_all; ++kc, kk += C::KS) {
        if (kc == kc0) {  // the second segment
          map = is_a ? &q.a[1] : &q.b[1];
          kk = 0;
        }
        const bool mine = KIND != kKindW4 || (issued & 1) == turn;
        if (mine) ok = swait(sm, &sm.empty[s], parity, p.status);
        if (!ok) break;
        const uint32_t bar = full0 + 8 * s;
        if (mine && elect_one()) {
          if (is_a && rank == 0) mbar_arrive_expect_tx(&sm.full[s], tx);
#pragma unroll
          for (int u = 0; u < C::KS; ++u) {
            if (!has) break;
            const uint32_t dst = op0 + (s * C::KS + u) * (is_a ? C::A_SUB : C::B_SUB);
            if constexpr (KIND != kKindMx) {
              if (mn) {
                tma_load_pair(dst, map, row, (kk + u) * 64, bar);
                if (boxes > 1) tma_load_pair(dst + 8192, map, row + 64, (kk + u) * 64, bar);
              } else {
                tma_load_pair(dst, map, (kk + u) * 64, row, bar);
              }
            } else {
              tma_load_pair(dst, map, (kk + u) * 128, row, bar);
              tma_load_pair(sf0 + (s * C::KS + u) * (is_a ? C::SFA_SUB : C::SFB_SUB), is_a ? &p.sfa : &p.sfb,
                            (kk + u) * 256, sf_row, bar);
            }
          }
        }
        __syncwarp();
        ++issued;
        if (++s == C::NS) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    if (lane == 0) sm.issued[turn] = issued;
    // The last products' commits arrive on the stages' barriers of both SMs: an SM
    // leaves behind them (a stage that was never used is free at once).
    for (int i = 0; i < C::NS && ok; ++i) {
      ok = swait(sm, &sm.empty[s], parity, p.status);
      if (++s == C::NS) {
        s = 0;
        parity ^= 1;
      }
    }
  } else if (warp == kPMma) {
    // ---------------------------------------------------------- MMA issuer
    if (rank == 0) {
      const uint32_t a0 = smem_u32(sm.a[0][0]), b0 = smem_u32(sm.b[0][0]);
      uint32_t s = 0, parity = 0, titer = 0;
      bool ok = true;
      const uint32_t sf0 = taddr + (uint32_t)C::SF_COL0;
      for (int t = cluster; t < p.n_tiles && ok; t += clusters, ++titer) {
        if (t != cluster) tile = ptile<NP>(p, t);
        const PProb& q = p.p[tile.prob];
        const int db = titer & 1, duse = titer >> 1;
        if (duse > 0) ok = __all_sync(0xffffffffu, pwait(sm, &sm.d_empty[db], (duse - 1) & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t dcol = taddr + (uint32_t)(db * BN);
        const bool a_mn = KIND != kKindMx && q.a_mn, b_mn = KIND != kKindMx && q.b_mn;
        const int kc_all = q.kc;
        // D fp32 (kind::f16), M = 256, N = BN
        uint32_t idesc = ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
        if (KIND != kKindMx) {
          idesc |= 1u << 4;
          if (!p.e.f16) idesc |= (1u << 7) | (1u << 10);
          idesc |= (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16;
        } else {
          idesc |= (1u << 7) | (1u << 10) | (1u << 23);  // E2M1 x E2M1, E8M0 scales
        }
        const uint32_t astep = a_mn ? 2048u >> 4 : 2u, bstep = b_mn ? 2048u >> 4 : 2u;
        // a stage's descriptor is its first stage's with the address advanced
        const uint64_t ad0 = a_mn ? make_mn_desc(a0) : make_sw128_desc(a0);
        const uint64_t bd0 = b_mn ? make_mn_desc(b0) : make_sw128_desc(b0);
        for (int kc = 0; kc < kc_all; ++kc) {
          // MXFP4: the warp that copies the scales has waited for the stage
          if constexpr (KIND == kKindW4) ok = swait_written(sm, &sm.full[s], parity, p.status);
          else ok = swait(sm, KIND == kKindMx ? &sm.scaled[s] : &sm.full[s], parity, p.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int u = 0; u < C::KS; ++u) {
              const uint64_t ad = ad0 + (uint64_t)((s * C::KS + u) * (C::A_SUB >> 4));
              const uint64_t bd = bd0 + (uint64_t)((s * C::KS + u) * (C::B_SUB >> 4));
              if constexpr (KIND != kKindMx) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma16_pair(dcol, ad + (uint64_t)(k * astep), bd + (uint64_t)(k * bstep), idesc,
                             kc > 0 || u > 0 || k > 0);
              } else {
                const uint32_t ta = sf0 + (s * C::KS + u) * C::SF_COLS, tb = ta + 8;
                const uint32_t id1 = idesc | 2u << 4 | 2u << 29;  // scale bytes 2-3 of a chunk
                const int nks = p.e.ksteps - 4 * (kc * C::KS + u);
                if (nks >= 4) {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    mma_mx_pair(dcol, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), k & 1 ? id1 : idesc,
                                ta + 4 * (k >> 1), tb + 4 * C::SFB_BLK * (k >> 1), kc > 0 || u > 0 || k > 0);
                } else {  // K ends inside the sub-stage
                  for (int k = 0; k < nks; ++k)
                    mma_mx_pair(dcol, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), k & 1 ? id1 : idesc,
                                ta + 4 * (k >> 1), tb + 4 * C::SFB_BLK * (k >> 1), kc > 0 || u > 0 || k > 0);
                }
              }
            }
            commit_pair(&sm.empty[s]);
            if (kc == kc_all - 1) commit_pair(&sm.d_full[db]);
          }
          __syncwarp();
          if (++s == C::NS) {
            s = 0;
            parity ^= 1;
          }
        }
        if (!ok) break;
      }
      // every MMA issued has completed before the tear-down
      if (elect_one()) commit_pair(&sm.fin);
      __syncwarp();
      // as have the arrivals of both SMs' epilogues, of each accumulator's last tile
      for (uint32_t db = 0; db < 2 && ok; ++db)
        if (titer > db) ok = __all_sync(0xffffffffu, pwait(sm, &sm.d_empty[db], ((titer - 1 - db) >> 1) & 1, p.status));
    }
    mbar_wait_bounded(&sm.fin, 0);
    __syncwarp();
  } else if (KIND == kKindMx && warp == kPScale) {
    // ------------------------- scales into tensor memory, ahead of the products
    if (rank == 0) {
      const uint32_t sf0 = taddr + (uint32_t)C::SF_COL0, sfa0 = smem_u32(sm.sfa[0]), sfb0 = smem_u32(sm.sfb[0]);
      uint32_t s = 0, parity = 0;
      bool ok = true;
      int left = cluster < p.n_tiles ? ((p.n_tiles - cluster - 1) / clusters + 1) * p.p[0].kc : 0;
      for (; left > 0; --left) {
        ok = swait(sm, &sm.full[s], parity, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int u = 0; u < C::KS; ++u) {
            const uint32_t ta = sf0 + (s * C::KS + u) * C::SF_COLS, tb = ta + 8;
            const uint32_t fa = sfa0 + (s * C::KS + u) * C::SFA_SUB, fb = sfb0 + (s * C::KS + u) * C::SFB_SUB;
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
              cp_sf_pair(ta + 4 * ch, fa + ch * kSfChunkB);
#pragma unroll
              for (int bb = 0; bb < C::SFB_BLK; ++bb)
                cp_sf_pair(tb + 4 * (ch * C::SFB_BLK + bb), fb + (bb * 2 + ch) * kSfChunkB);
            }
          }
          commit_here(&sm.scaled[s]);
        }
        __syncwarp();
        if (++s == C::NS) {
          s = 0;
          parity ^= 1;
        }
      }
      // the copies issued have completed before the tear-down
      if (elect_one()) commit_here(&sm.fin_sf);
      __syncwarp();
      mbar_wait_bounded(&sm.fin_sf, 0);
      __syncwarp();
    }
  } else if (KIND == kKindW4 && warp >= kPConv0) {
    // ------------------------- MXFP4 weights into the stages' B tiles as bf16
    // Two warps convert every fourth stage: what a stage costs besides its
    // arithmetic (the wait, the fence, the arrival) then overlaps among the
    // pairs.  A warp reads its next stage while it converts one.
    constexpr int ROWS = BN / 2, BPR = 2 * C::KS;        // rows of this SM, blocks of 32 per row and stage
    constexpr int NB = ROWS * BPR / (32 * kPConvPer), DR = 32 / BPR;  // blocks per lane, rows between them
    constexpr int GROUPS = kPConvWarps / kPConvPer;
    const int cw = warp - kPConv0, group = cw / kPConvPer;
    const int r0 = (cw % kPConvPer) * (NB * DR) + lane / BPR, kb = lane % BPR;
    const uint32_t full0 = leader_addr(&sm.full[0]);
    const PProb& q = p.p[0];
    const int K = q.K, kc_all = q.kc, N = q.N, units = K / 32;
    const uint8_t* const wq = q.wq + (EPI == kEpiGated && rank ? (size_t)N * units * 16 : 0);
    const uint8_t* const ws = q.ws + (EPI == kEpiGated && rank ? (size_t)N * units : 0);
    const int total = cluster < p.n_tiles ? ((p.n_tiles - cluster - 1) / clusters + 1) * kc_all : 0;
    struct Stage {
      uint4 code[NB];
      uint32_t scale[NB];
    };
    // the next stage to read
    int lt = cluster, lk = group, lrow = 0;
    auto settle = [&]() {  // into the tile that holds it
      while (lk >= kc_all) {
        lk -= kc_all;
        lt += clusters;
      }
      if (lt < p.n_tiles) {
        const int n = ptile<NP>(p, lt).n;
        lrow = (EPI == kEpiGated ? n * (BN / 2) : n * BN + (int)rank * (BN / 2)) + r0;
      }
    };
    settle();
    auto read = [&](Stage& b) {
      const int unit = lk * BPR + kb;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int row = lrow + i * DR;
        b.code[i] = make_uint4(0u, 0u, 0u, 0u);
        b.scale[i] = 0u;
        if (lt < p.n_tiles && row < N && unit < units) {
          b.code[i] = ld_v4_stream(wq + ((size_t)row * units + unit) * 16);
          b.scale[i] = ld_u8(ws + (size_t)row * units + unit);
        }
      }
      lk += GROUPS;
      if (lk >= kc_all) settle();
    };
    auto convert = [&](const Stage& b, int it) {
      const int s = it % C::NS;
      if (!swait(sm, &sm.empty[s], ((it / C::NS) & 1) ^ 1, p.status)) return false;
      uint8_t* const dst = sm.b[s][kb >> 1];
      // a warp without scales above 2 leaves the second factor out: as a branch
      // for every word it keeps the compiler from interleaving them
      auto decode = [&](auto has_big) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int r = r0 + i * DR;
          const MxFactor f = mx_factor(b.scale[i]);
          const uint32_t w[4] = {b.code[i].x, b.code[i].y, b.code[i].z, b.code[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t o[4];
            mx_place8(w[q], f, o);
            if constexpr (decltype(has_big)::value) {
              const uint32_t f1 = f.big ? f.f1 : 0x3F803F80u;
#pragma unroll
              for (int j = 0; j < 4; ++j) o[j] = bmul2(o[j], f1);
            }
            // 128-byte rows, 16-byte pieces exchanged by row as TMA does
            *reinterpret_cast<uint4*>(dst + r * 128 + (((kb & 1) * 4 + q) ^ (r & 7)) * 16) =
                make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                           __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
          }
        }
      };
      bool big = false;
#pragma unroll
      for (int i = 0; i < NB; ++i) big |= mx_big(b.scale[i]);
      if (__any_sync(0xffffffffu, big)) decode(std::true_type{});
      else decode(std::false_type{});
      out_ready();  // visible to the products
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&sm.full[s]);
        else arrive_written(full0 + 8 * s);
      }
      return true;
    };
    Stage even, odd;
    read(even);
    for (int it = group; it < total; it += 2 * GROUPS) {
      read(odd);
      if (!convert(even, it) || it + GROUPS >= total) break;
      read(even);
      if (!convert(odd, it + GROUPS)) break;
    }
  } else if (warp >= kPEpi0) {
    // ------------------------------------------------------------ epilogue
    constexpr int HC = EPI == kEpiGated ? BN / 4 : BN / 2;  // output columns of this warp
    constexpr int CW = EPI == kEpiGatedBwd ? 32 : HC % 64 == 0 ? 64 : HC % 32 == 0 ? 32 : 16;
    using Out = POut<CW>;
    // backward: dg and du side by side
    constexpr int BUFS = EPI == kEpiGatedBwd ? Out::BUFS / 2 : Out::BUFS;
    const int ew = warp - kPEpi0, quarter = warp & 3, half = ew >> 2;
    const bool f16 = p.e.f16;
    uint32_t titer = 0, chunk = 0;
    for (int t = cluster; t < p.n_tiles; t += clusters, ++titer) {
      if (t != cluster) tile = ptile<NP>(p, t);
      const PTile d = tile;
      const PProb& q = p.p[d.prob];
      const int M = q.M, N = q.N;
      const int db = titer & 1, duse = titer >> 1;
      const int row0 = d.m * 256 + (int)rank * 128 + quarter * 32;
      const int col0 = half * HC, n0 = d.n * (EPI == kEpiGated ? BN / 2 : BN) + col0;
      const uint32_t tcol = taddr + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(db * BN + col0);
      // the kept block of this warp's rows and hidden units n..n + 15, null outside
      const int blks = (N + 15) >> 4;
      auto kept_blk = [&](int n) {
        return row0 < M && n < N ? p.e.kept + ((size_t)(row0 >> 5) * blks + (n >> 4)) * kKeptBlockB : nullptr;
      };
      constexpr int AHEAD = 2;
      Kept16 kept16[EPI == kEpiGatedBwd ? AHEAD + 1 : 1];
      auto fetch = [&](int c) {
        const uint8_t* blk = kept_blk(n0 + c);
        if (blk) kept_load(blk, lane, kept16[(c / 16) % (AHEAD + 1)]);  // else: unused
      };
      // backward: p and a of the first columns are on their way while the
      // products run, and those of the next 32 while 16 are computed
      if constexpr (EPI == kEpiGatedBwd) {
#pragma unroll
        for (int c = 0; c < 16 * AHEAD; c += 16) fetch(c);
      }
      if (!pwait(sm, &sm.d_full[db], duse & 1, p.status)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < HC; c += CW) {
        uint8_t* buf = sm.out[ew] + (chunk++ % BUFS) * (kPOutB / BUFS);
        out_reuse<BUFS - 1>(lane);
        float v32[32];  // plain: of two groups
#pragma unroll
        for (int k = 0; k < CW; k += 16) {
          uint32_t w[8];
          if constexpr (EPI == kEpiGated) {
            float g[16], u[16];
            tmem_ld16(tcol + c + k, g);
            tmem_ld16(tcol + BN / 2 + c + k, u);
            gate16<KIND == kKind16>(p.e, KIND == kKind16 && p.e.kept ? kept_blk(n0 + c + k) : nullptr, lane, g, u, f16, w);
          } else if constexpr (EPI == kEpiPlain) {
            if (k % 32 == 0) tmem_ld32(tcol + c + k, v32);
            pack16(v32 + k % 32, f16, w);
          } else {
            if (c + k + 16 * AHEAD < HC) fetch(c + k + 16 * AHEAD);
            const Kept16& r = kept16[((c + k) / 16) % (AHEAD + 1)];
            float v[16], o[16];
            tmem_ld16(tcol + c + k, v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = v[i] * kept(r.ah[(i / 4) * 2], r.ah[(i / 4) * 2 + 1], r.al[i / 4], i & 3);
            pack16(o, f16, w);
            Out::put(buf + Out::BYTES, lane, k / 16, w);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = v[i] * kept(r.ph[(i / 4) * 2], r.ph[(i / 4) * 2 + 1], r.pl[i / 4], i & 3);
            pack16(o, f16, w);
          }
          Out::put(buf, lane, k / 16, w);
        }
        if (c + CW == HC) {  // all read: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_read(leader_addr(&sm.d_empty[db]));
        }
        out_ready();
        if (lane == 0) {
          if (row0 < M && n0 + c < N) {
            tma_store(&q.o[0], buf, n0 + c, row0);
            if (EPI == kEpiGatedBwd) tma_store(&q.o[1], buf + Out::BYTES, n0 + c, row0);
          }
          out_commit();
        }
      }
    }
    out_reuse<0>(lane);  // the buffers outlive the stores' reads
  }

  // ------------------------------------------------------------- tear-down
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort_flag) {
    // copies in flight land before the pair leaves (SM 1's complete on SM 0's barriers)
    const int issued = max(sm.issued[0], sm.issued[1]);
    for (int it = max(0, issued - C::NS); it < issued; ++it)
      mbar_wait_bounded(&sm.full[it % C::NS], (it / C::NS) & 1, kAbortDrainNs);
  }
  __syncthreads();
  if (sm.abort_flag) cluster_sync_ordered();
  else cluster_sync();
  if (warp == kPMma) {
    tc_fence_after();
    tmem_dealloc2(taddr, kPTmem);
  }
}

// ---------------------------------------------------------------------- host
// rows of a box of A: a box's time goes by its rows, those past M included
int a_box(int M) { return M >= 128 ? 128 : (M + 7) / 8 * 8; }

template <int EPI, int BN>
constexpr int out_cols() {  // columns of an output box, as in the kernel
  return EPI == kEpiGatedBwd ? 32 : (EPI == kEpiGated ? BN / 4 : BN / 2) % 64 == 0 ? 64
                                : (EPI == kEpiGated ? BN / 4 : BN / 2) % 32 == 0   ? 32 : 16;
}
// [M, N] 16-bit output, boxes of 32 rows
template <int EPI, int BN>
bool map_out(CUtensorMap* m, void* out, int M, int N, int64_t ld) {
  constexpr int CW = out_cols<EPI, BN>();
  return encode_tma_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, out, N, M, (uint64_t)ld * 2, CW, 32, POut<CW>::SW);
}

// ldo: the outputs' row pitch in elements, 0 for N.
template <int KIND, int BN, int EPI, int NP>
cudaError_t launch_pair(PParams<NP>& p, void* const (&out)[NP], void* out1, int64_t ldo, cudaStream_t st) {
  using C = PCfg<KIND, BN>;
  for (int i = 0; i < p.np; ++i) {
    PProb& q = p.p[i];
    const int64_t ld = ldo ? ldo : q.N;
    if (!map_out<EPI, BN>(&q.o[0], out[i], q.M, q.N, ld) ||
        (EPI == kEpiGatedBwd && !map_out<EPI, BN>(&q.o[1], out1, q.M, q.N, ld)))
      return cudaErrorInvalidValue;
    const int a = q.a_mn ? C::A_SUB : a_box(q.M) * 128, b = KIND == kKindW4 ? 0 : C::B_SUB + C::SFB_SUB;
    q.tx = C::KS * ((q.M > 128 ? 2 : 1) * (a + C::SFA_SUB) + 2 * b);
  }
  constexpr int smem = (int)sizeof(PSmem<KIND, BN>) + 1024;
  static_assert(smem <= 232448, "shared memory budget");
  auto fn = pair_gemm_kernel<KIND, BN, EPI, NP>;
  cudaError_t err = configure_kernel_once((const void*)fn, smem);
  if (err != cudaSuccess) return err;
  const int clusters = std::max(1, std::min(p.n_tiles, sms() / 2));
  return launch_overlapped(fn, 2 * clusters, 1, C::THREADS, smem, st, p);
}

bool map16(CUtensorMap* m, const PairOperand& o, int rows, int K, int dtype, int box_rows) {
  const CUtensorMapDataType dt = dtype == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (o.mn) return encode_tma_2d(m, dt, o.p, rows, K, o.ld * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  return encode_tma_2d(m, dt, o.p, K, rows, o.ld * 2, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile width of a list of problems: the one whose busiest cluster is done
// first.  Clusters take every `clusters`-th tile; a sub-stage (128 bytes of K)
// takes `cycles`, and behind the last tile comes its epilogue.
struct Width {
  int bn, cycles, tail;
};
constexpr Width kWidths16[] = {{256, 512, 3000}, {128, 290, 2000}, {64, 200, 1500}};
constexpr Width kWidths16Mn[] = {{256, 540, 3000}, {128, 430, 2000}};  // an MN-major box is 64 columns of each SM's half
constexpr Width kWidthsW4[] = {{128, 400, 2000}, {64, 310, 1500}};  // 256 was measured at T = 512 to 4096: never faster
constexpr Width kWidthsMx[] = {{192, 560, 3000}, {128, 480, 2000}, {64, 400, 1500}};
struct Tiles {
  int64_t m, cols, subs;  // tiles along M, columns, sub-stages along K
};
template <int NW>
int pick_bn(const Width (&widths)[NW], const Tiles* g, int n, int clusters) {
  int best = 0;
  int64_t least = INT64_MAX;
  for (const Width& w : widths) {
    // a cluster's load changes with c only at the problems' first tiles
    int64_t worst = 0, first = 0;
    for (int k = 0; k < n; ++k) {
      const int64_t c = first % clusters;
      first += g[k].m * cdiv(g[k].cols, w.bn);
      int64_t t0 = 0, cycles = 0;
      for (int i = 0; i < n; ++i) {
        const int64_t t1 = t0 + g[i].m * cdiv(g[i].cols, w.bn);
        // multiples of `clusters` plus c in [t0, t1)
        const int64_t tiles = (t1 + clusters - 1 - c) / clusters - (t0 + clusters - 1 - c) / clusters;
        const int64_t subs = w.bn <= 128 ? cdiv(g[i].subs, 2) * 2 : g[i].subs;
        cycles += tiles * subs * w.cycles;
        t0 = t1;
      }
      worst = std::max(worst, cycles);
    }
    if (worst + w.tail < least) {
      least = worst + w.tail;
      best = w.bn;
    }
  }
  return best;
}

// stages of a K of `subs` sub-stages
int stages(int64_t subs, int bn) { return (int)(bn <= 128 ? cdiv(subs, 2) : subs); }

}  // namespace

cudaError_t launch_pair_gemm(const PairGemm* g, int n, int dtype, int* status, cudaStream_t st) {
  if (n < 1 || n > kPairMaxProblems) return cudaErrorInvalidValue;
  bool mn = false;
  for (int i = 0; i < n; ++i)
    for (int s = 0; s < g[i].nseg; ++s) mn |= g[i].seg[s].b.mn;
  Tiles tiles[kPairMaxProblems];
  for (int i = 0; i < n; ++i) {
    tiles[i] = Tiles{cdiv(g[i].M, 256), g[i].N, 0};
    for (int s = 0; s < g[i].nseg; ++s) tiles[i].subs += cdiv(g[i].seg[s].K, 64);
  }
  const int bn = mn ? pick_bn(kWidths16Mn, tiles, n, sms() / 2) : pick_bn(kWidths16, tiles, n, sms() / 2);
  PParams<kPairMaxProblems> p;
  std::memset(&p, 0, sizeof(p));
  void* out[kPairMaxProblems] = {};
  int t0 = 0;
  for (int i = 0; i < n; ++i) {
    PProb& q = p.p[i];
    for (int s = 0; s < 2; ++s) {
      const PairSegment& sg = g[i].seg[s < g[i].nseg ? s : 0];
      if (!map16(&q.a[s], sg.a, g[i].M, sg.K, dtype, a_box(g[i].M)) || !map16(&q.b[s], sg.b, g[i].N, sg.K, dtype, bn / 2))
        return cudaErrorInvalidValue;
    }
    out[i] = g[i].out;
    q.M = g[i].M;
    q.N = g[i].N;
    q.kc0 = stages(cdiv(g[i].seg[0].K, 64), bn);
    q.kc = q.kc0 + (g[i].nseg > 1 ? stages(cdiv(g[i].seg[1].K, 64), bn) : 0);
    q.tm = (int)cdiv(q.M, 256);
    q.t0 = t0;
    q.a_mn = g[i].seg[0].a.mn;
    q.b_mn = g[i].seg[0].b.mn;
    t0 += q.tm * (int)cdiv(q.N, bn);
  }
  p.e.f16 = dtype == kF16;
  p.np = n;
  p.n_tiles = t0;
  p.status = status;
  if (bn == 64) return launch_pair<kKind16, 64, kEpiPlain, kPairMaxProblems>(p, out, nullptr, 0, st);
  if (bn == 128) return launch_pair<kKind16, 128, kEpiPlain, kPairMaxProblems>(p, out, nullptr, 0, st);
  return launch_pair<kKind16, 256, kEpiPlain, kPairMaxProblems>(p, out, nullptr, 0, st);
}

cudaError_t launch_pair_gated(const PairGated& a, int* status, cudaStream_t st) {
  const int64_t tm = cdiv(a.T, 256);
  const Tiles tiles{tm, 2 * (int64_t)a.I, cdiv(a.K, 64)};
  const int bn = pick_bn(kWidths16, &tiles, 1, sms() / 2);
  PParams<1> p;
  std::memset(&p, 0, sizeof(p));
  PProb& q = p.p[0];
  const PairOperand x{a.x, a.ldx, false}, wg{a.gate, a.ldw, false}, wu{a.up, a.ldw, false};
  if (!map16(&q.a[0], x, a.T, a.K, a.dtype, a_box(a.T)) || !map16(&q.b[0], wg, a.I, a.K, a.dtype, bn / 2) ||
      !map16(&q.b[1], wu, a.I, a.K, a.dtype, bn / 2))
    return cudaErrorInvalidValue;
  q.M = a.T;
  q.N = a.I;
  q.kc0 = q.kc = stages(cdiv(a.K, 64), bn);
  q.tm = (int)tm;
  if (a.keep) p.e.kept = a.kept.blocks;
  p.e.act = a.act;
  p.e.f16 = a.dtype == kF16;
  p.np = 1;
  p.n_tiles = (int)(tm * cdiv(a.I, bn / 2));
  p.status = status;
  if (bn == 64) return launch_pair<kKind16, 64, kEpiGated, 1>(p, {a.h}, nullptr, a.ldh, st);
  if (bn == 128) return launch_pair<kKind16, 128, kEpiGated, 1>(p, {a.h}, nullptr, a.ldh, st);
  return launch_pair<kKind16, 256, kEpiGated, 1>(p, {a.h}, nullptr, a.ldh, st);
}

cudaError_t launch_pair_gated_bwd(const PairGatedBwd& a, int* status, cudaStream_t st) {
  const int64_t tm = cdiv(a.T, 256);
  const Tiles tiles{tm, a.I, cdiv(a.H, 64)};
  const int bn = pick_bn(kWidths16Mn, &tiles, 1, sms() / 2);
  PParams<1> p;
  std::memset(&p, 0, sizeof(p));
  PProb& q = p.p[0];
  const PairOperand dy{a.dy, a.lddy, false}, wd{a.down, a.I, true};
  if (!map16(&q.a[0], dy, a.T, a.H, a.dtype, a_box(a.T)) || !map16(&q.b[0], wd, a.I, a.H, a.dtype, bn / 2))
    return cudaErrorInvalidValue;
  q.M = a.T;
  q.N = a.I;
  q.kc0 = q.kc = stages(cdiv(a.H, 64), bn);
  q.tm = (int)tm;
  q.b_mn = 1;
  p.e.kept = a.kept.blocks;
  p.e.f16 = a.dtype == kF16;
  p.np = 1;
  p.n_tiles = (int)(tm * cdiv(a.I, bn));
  p.status = status;
  if (bn == 128) return launch_pair<kKind16, 128, kEpiGatedBwd, 1>(p, {a.dg}, a.du, pair_pitch(a.I), st);
  return launch_pair<kKind16, 256, kEpiGatedBwd, 1>(p, {a.dg}, a.du, pair_pitch(a.I), st);
}

cudaError_t launch_pair_w4(const PairW4& a, int* status, cudaStream_t st) {
  const bool gated = a.act != kActNone;
  const int64_t tm = cdiv(a.T, 256);
  const Tiles tiles{tm, gated ? 2 * (int64_t)a.N : a.N, cdiv(a.K, 64)};
  const int bn = pick_bn(kWidthsW4, &tiles, 1, sms() / 2);
  PParams<1> p;
  std::memset(&p, 0, sizeof(p));
  PProb& q = p.p[0];
  const PairOperand x{a.x, a.ldx, false};
  if (!map16(&q.a[0], x, a.T, a.K, kBf16, a_box(a.T))) return cudaErrorInvalidValue;
  q.wq = a.codes;
  q.ws = a.scales;
  q.K = a.K;
  q.M = a.T;
  q.N = a.N;
  q.kc0 = q.kc = stages(cdiv(a.K, 64), bn);
  q.tm = (int)tm;
  p.e.act = a.act;
  p.np = 1;
  p.n_tiles = (int)(tm * cdiv(a.N, gated ? bn / 2 : bn));
  p.status = status;
  if (gated) {
    if (bn == 64) return launch_pair<kKindW4, 64, kEpiGated, 1>(p, {a.y}, nullptr, 0, st);
    return launch_pair<kKindW4, 128, kEpiGated, 1>(p, {a.y}, nullptr, 0, st);
  }
  if (bn == 64) return launch_pair<kKindW4, 64, kEpiPlain, 1>(p, {a.y}, nullptr, 0, st);
  return launch_pair<kKindW4, 128, kEpiPlain, 1>(p, {a.y}, nullptr, 0, st);
}

int pair_mx_tile(int T, int N, int K, int act) {
  const Tiles tiles{cdiv(T, 256), act != kActNone ? 2 * (int64_t)N : N, cdiv(K, 256)};
  return pick_bn(kWidthsMx, &tiles, 1, sms() / 2);
}

cudaError_t launch_pair_mx(const PairMx& a, int* status, cudaStream_t st) {
  const bool gated = a.act != kActNone;
  const int bn = a.bn, tn = gated ? bn / 2 : bn;  // output columns per tile
  const int64_t pitch = mx_pitch(a.K), tm = cdiv(a.T, 256), tiles_n = cdiv(a.N, tn);
  const int chunks = mx_sf_chunks(a.K), blks = (bn + 127) / 128;
  PParams<1> p;
  std::memset(&p, 0, sizeof(p));
  PProb& q = p.p[0];
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B, ns = CU_TENSOR_MAP_SWIZZLE_NONE;
  if (!encode_tma_2d(&q.a[0], u8, a.xq, a.K / 2, a.T, pitch, 128, a_box(a.T), sw) ||
      !encode_tma_2d(&q.b[0], u8, a.wq, a.K / 2, a.N, pitch, 128, bn / 2, sw) ||
      !encode_tma_2d(&q.b[1], u8, a.wq + (gated ? a.N * pitch : 0), a.K / 2, a.N, pitch, 128, bn / 2, sw) ||
      !encode_tma_2d(&p.sfa, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.xsf, (uint64_t)chunks * 128, cdiv(a.T, 128),
                     (uint64_t)chunks * kSfChunkB, 256, 1, ns) ||
      !encode_tma_2d(&p.sfb, CU_TENSOR_MAP_DATA_TYPE_UINT32, a.wsf, (uint64_t)chunks * 128, tiles_n * blks,
                     (uint64_t)chunks * kSfChunkB, 256, blks, ns))
    return cudaErrorInvalidValue;
  q.M = a.T;
  q.N = a.N;
  q.kc0 = q.kc = stages(cdiv(a.K, 256), bn);
  q.tm = (int)tm;
  p.e.act = a.act;
  p.e.f16 = a.dtype == kF16;
  p.e.ksteps = (int)cdiv(a.K, 64);
  p.np = 1;
  p.n_tiles = (int)(tm * tiles_n);
  p.status = status;
  if (gated) {
    if (bn == 64) return launch_pair<kKindMx, 64, kEpiGated, 1>(p, {a.y}, nullptr, 0, st);
    if (bn == 128) return launch_pair<kKindMx, 128, kEpiGated, 1>(p, {a.y}, nullptr, 0, st);
    return launch_pair<kKindMx, 192, kEpiGated, 1>(p, {a.y}, nullptr, 0, st);
  }
  if (bn == 64) return launch_pair<kKindMx, 64, kEpiPlain, 1>(p, {a.y}, nullptr, 0, st);
  if (bn == 128) return launch_pair<kKindMx, 128, kEpiPlain, 1>(p, {a.y}, nullptr, 0, st);
  return launch_pair<kKindMx, 192, kEpiPlain, 1>(p, {a.y}, nullptr, 0, st);
}

}  // namespace nvfp4moe
