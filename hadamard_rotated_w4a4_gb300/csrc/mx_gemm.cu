// The MXFP4 product Y[m][n] = sum_b 2^(Ew + Ea - 254) sum_j w_j a_j on the tensor
// cores' block-scaled path (tcgen05.mma kind::mxf4, one scale byte per 32 elements
// of each operand): the tensor core applies the scales itself, so nothing is folded
// on the CUDA cores.
//
// The weights are the MMA's M operand and the tokens its N operand: one token costs
// no more tensor work than 16, a warp's lanes hold consecutive outputs n, and every
// store of Y is contiguous.  Stages of 256 elements of K (128 bytes a row, 128-byte
// swizzle) and their scale tiles come by TMA; the scale tiles go on to TMEM
// (tcgen05.cp) in front of the MMAs that use them.
//
// Two kernels:
//   small (few tiles): a CTA multiplies 128 weight rows by up to 128 tokens; a cluster of
//     S CTAs may share a tile, each with a contiguous share of K, so that few tiles still
//     stream the weights through every SM.  The S partial tiles meet in distributed
//     shared memory and are summed in rank order: no workspace, no dependence on
//     timing.
//   pair: persistent CTA pairs (cta_group::2) multiply 256 weight rows by up
//     to 256 tokens.  Each CTA stages half of both operands, which is what lets shared
//     memory (written once, read once per MMA, 128 bytes a cycle) keep up with the
//     tensor core.  The accumulators leave TMEM for registers at once, and their stores
//     (32 bytes a cycle and SM at most) overlap the next tile's MMAs.  With a workspace
//     the last waves' K work is cut evenly over the pairs (stream-K).
//
// Bounds and measurements (GB300, CUDA graphs).  Pair: a stage of a 256 x 256 tile takes 574
// cycles and is 530 of shared memory by its bytes; about 1,800 pass between two tiles.  The
// MMAs alone were not timed (at the nominal 13.5 PFLOP/s a stage is 391 cycles).  M4096
// K5120 N17408 bf16 101 us in a burst on one set of operands (7.2 PFLOP/s), 107 on three in
// turn, 111 sustained, under the power cap; M1024 K17408 N5120 31 us (5.8).  Small: bound by
// the weights' stream where K x N is large (K69632 N5120, one token: 6.1 TB/s), else by
// set-up and round trips.  K5120 N5120, weights from memory: one token 5.0 us, 64 tokens
// 7.8, 256 tokens 8.6; weights in L2: one token 4.1.
//
// The epilogue, act(sum + bias) + residual, on the fp32 sums before their one rounding, as
// instances of their own: the plain product's are as they were.  Bound: the residual's bytes and
// the epilogue warps' instructions beside the next tile's MMAs.  Against the plain bf16 product
// (us): M1024 N5120 K17408 (fp32 out) 35.0, bias 35.3, fp32 residual 44.7, SiLU 36.4, GELU 37.5; M4096
// N17408 K5120 102, 103, 124 (285 MB more to read), 104, 107; M333 N4600 K1184 5.0, 5.6, 6.4, 6.3, 6.5;
// M64 N5120 K5120 6.7, 7.4, 7.8, 7.5, 7.8.
#include <cuda_bf16.h>

#include "tc_ptx.cuh"
#include "w4a4_kernels.cuh"

namespace w4a4 {

namespace {

constexpr int kTW = 128;      // weight rows per CTA
constexpr int kStageK = 256;  // elements of K per stage
// Bound of every wait in SM cycles: 1.04 s at 2.07 GHz, the top clock, longer below it.
constexpr int64_t kWaitCycles = int64_t(1) << 31;
constexpr int kWBytes = kTW * 128;
constexpr int kSfTile = 1024;  // a stage's scales of 128 rows: two 512-byte tiles

struct MxArgs {
  void* y;
  int64_t ldy;
  int64_t M, N;
  int K, stages;
  int box;      // token rows of one load
  int ring;     // small kernel: stages in shared memory
  int apart;    // small kernel: where the partial tiles lie, 0 = over the stages
  // pair kernel
  int mt, wt;   // token tiles (the last one narrower), weight tiles
  int whole;    // tiles 0 .. whole - 1 go to the pairs whole, in turn; the rest by stages
  int64_t units;     // stages of the rest (0: none)
  uint32_t* flags;   // [pairs][2 CTAs][8 warps], zero between calls
  float4* parts;     // [pairs][2][8][32][32]: a warp's 128 accumulators of 32 lanes
  int* err;
  int64_t wait, delay;  // cycles: the pipeline waits' bound; a test's hold on the first copy
  MxEpilogue ep;
};

struct Bars {
  uint64_t full[12], empty[12], acc_full, acc_empty;
  uint32_t tmem;
  volatile int abort;
};

// Bounded wait; on giving up, every other wait of the CTA gives up too.
__device__ __forceinline__ bool wait_bar(Bars& S, uint64_t* b, uint32_t parity, const MxArgs& p) {
  if (mbar_try(b, parity)) return true;
  const int64_t t0 = clock64();
  while (!mbar_try(b, parity)) {
    if (S.abort) return false;
    if (clock64() - t0 > p.wait) {
      S.abort = 1;
      if (p.err) atomicOr(p.err, 32);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void hold(const MxArgs& p) {
  if (p.delay > 0) {
    const int64_t t0 = clock64();
    while (clock64() - t0 < p.delay) {
    }
  }
}
// As above without the shared give-up, for copies and MMAs in flight.
__device__ __forceinline__ void drain_bar(uint64_t* b, uint32_t parity) {
  const int64_t t0 = clock64();
  while (!mbar_try(b, parity) && clock64() - t0 < kWaitCycles) {
  }
}

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// One lane of the converged warp; the compiler knows that a single thread runs what
// it guards.  The copy and MMA loops are run by their whole warps and elect a lane for
// the instructions alone, so that addresses, descriptors and columns stay in uniform
// registers: a lane test around the loop costs about 100 cycles per copy or MMA, an
// election around it 33 (M1024 K17408 N5120 35.7 us, against 31.6 with the loop uniform).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same in two halves, for what needs no data of the others.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t map_rank(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}

// ---------------------------------------------------------------- tcgen05, both group sizes
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(dst)), "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(dst)), "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}
// 512-byte scale tile (32 rows x 16 bytes, no swizzle) to 4 TMEM columns of all four
// lane quarters; in a pair, each CTA's own tile to its own TMEM.
template <int CG>
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint32_t smem) {
  const uint64_t d = static_cast<uint64_t>((smem >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
                     (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
// kind::mxf4 instruction descriptor: A and B e2m1 (code 1), K-major, ue8m0 scales,
// K = 64, 128 rows of A per CTA; mx_sf(2) picks the second byte pair of the scale words.
__device__ __forceinline__ uint32_t mx_idesc(int cg, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(cg * kTW >> 4) << 24);
}
constexpr uint32_t kSfHigh = (2u << 4) | (2u << 29);
template <int CG>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t acc) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}
// Arrival, when every MMA issued so far is done, on a barrier of this CTA, or on the
// same barrier of both CTAs of the pair.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 1)
    mma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            su32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// One stage's MMAs: `steps` of K = 64 (four but for the end of K), behind the scale
// tiles they use.  sfw: TMEM column of the weights' scales, the tokens' follow; a scale
// operand has to start on a scale tile's first column, so token tiles start at multiples
// of 128 rows.  kAtoms: token scale tiles per 128 of K.
template <int CG, int kAtoms>
__device__ __forceinline__ void stage_mmas(uint32_t d, uint32_t wsm, uint32_t asm_, uint32_t sfsm, uint32_t sfw,
                                           uint32_t idesc, int steps, uint32_t acc) {
  const uint32_t sfa = sfw + 8;
  const uint64_t base = (static_cast<uint64_t>(1) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
                        (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);  // as kmajor_desc_sw128
  const uint64_t wd = base | ((wsm >> 4) & 0x3FFFu), ad = base | ((asm_ >> 4) & 0x3FFFu);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < steps) {
      // the scales of 128 elements in front of their two MMAs, not of a whole stage in
      // front of four: a copy runs beside the MMA before it (M2048 K20480 N9728: 105.5 -> 100 us)
      if (!(k & 1)) {
        const int j = k >> 1;
        sf_copy<CG>(sfw + 4 * j, sfsm + 512 * j);
#pragma unroll
        for (int t = 0; t < kAtoms; ++t)
          sf_copy<CG>(sfa + 4 * (j * kAtoms + t), sfsm + kSfTile + t * kSfTile + 512 * j);
      }
      mma_mx<CG>(d, wd + 2 * k, ad + 2 * k, (k & 1) ? idesc | kSfHigh : idesc, sfw + 4 * (k >> 1),
                 sfa + 4 * (k >> 1) * kAtoms, k > 0 ? 1u : acc);
    }
  }
}

// TMA load of a tile, its bytes counted on `bar`: this CTA's, or (pair) the leader's.
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// ---------------------------------------------------------------- bias, activation, residual
// act(r + bias) + residual on tokens m0 .. m0 + lim - 1 of this lane's weight row n, in place
// in the accumulators (r[i] = token i), two tokens an instruction.
//   SiLU and the tanh form of GELU: x / (1 + exp(-z)), z = x or 2 sqrt(2/pi) (x + 0.044715 x^3), since
//     (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)).
//   GELU: max(x, 0) - |x| q / 2, q = erfc(|x| / sqrt 2) by Abramowitz and Stegun, "Handbook of Mathematical
//     Functions", 7.1.26 (off by 1.5e-7 at most): no branches, a quarter of erff's instructions (M333 N4600 K1184
//     11.9 us with that).
// The residual is all that is read: 32 tokens' loads of a warp's 32 neighbours go out together (one after the other,
// each behind the sum before it, M4096 K5120 N17408 took 293 us), the first before the sums are there, the next
// before these are stored; and its lines are asked into L2 while the products run.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 pair_of(float a) { return make_float2(a, a); }
template <int ACT>
__device__ __forceinline__ float2 activate(float2 x) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (ACT == kActRelu) {
    return make_float2(x.x <= 0.0f ? 0.0f : x.x, x.y <= 0.0f ? 0.0f : x.y);
  } else if constexpr (ACT == kActGelu) {
    const float2 a = make_float2(fminf(fabsf(x.x), 0x1p100f), fminf(fabsf(x.y), 0x1p100f));  // q is 0 there: inf stays inf
    const float2 d = __ffma2_rn(a, pair_of(0.3275911f * 0.70710678118654752f), pair_of(1.0f));
    const float2 t = make_float2(rcp(d.x), rcp(d.y));
    float2 q = __ffma2_rn(t, pair_of(0.5f * 1.061405429f), pair_of(0.5f * -1.453152027f));
    q = __ffma2_rn(q, t, pair_of(0.5f * 1.421413741f));
    q = __ffma2_rn(q, t, pair_of(0.5f * -0.284496736f));
    q = __ffma2_rn(q, t, pair_of(0.5f * 0.254829592f));
    q = __fmul2_rn(q, t);
    const float2 u = __fmul2_rn(__fmul2_rn(x, x), pair_of(-0.5f * kLog2e));
    q = __fmul2_rn(q, make_float2(ex2(u.x), ex2(u.y)));
    return __ffma2_rn(make_float2(-a.x, -a.y), q, make_float2(x.x > 0.0f ? x.x : 0.0f, x.y > 0.0f ? x.y : 0.0f));
  } else {
    float2 u = pair_of(-kLog2e);
    if constexpr (ACT == kActGeluTanh) u = __ffma2_rn(__fmul2_rn(x, x), pair_of(-kLog2e * 0.07135481282553567f), pair_of(-kLog2e * 1.5957691216057308f));
    u = __fmul2_rn(u, x);
    const float2 d = __fadd2_rn(make_float2(ex2(u.x), ex2(u.y)), pair_of(1.0f));
    return __fmul2_rn(x, make_float2(rcp(d.x), rcp(d.y)));
  }
}
template <int ACT, int NC>
__device__ __forceinline__ void activate_all(uint32_t (&r)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; i += 2) {
    const float2 y = activate<ACT>(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])));
    r[i] = __float_as_uint(y.x);
    r[i + 1] = __float_as_uint(y.y);
  }
}
// What a kernel's instance does with its sums: stores them; bias and activation alone; an fp32 or a bf16 residual as well.
// (With both types in one instance M4096 N17408 K5120 took 129 us with fp32 and 142 with bf16, for 125 and 115.)  That
// the residual is there is asked again in front of its loads: without the branch they were compiled among the sums'
// arithmetic instead of together, 182 us.
enum Epi : int { kPlain, kEpi, kEpiF32, kEpiBf16 };
// Lines of the residual that this warp's epilogue will read, tokens m0 .. m0 + lim - 1 of weight rows n0 .. n0 + 31.
template <int EPI>
__device__ __forceinline__ void ask_residual(const MxEpilogue& e, int64_t n0, int64_t N, int64_t m0, int lim) {
  if (EPI < kEpiF32 || !e.residual || n0 >= N) return;
  for (int i = threadIdx.x & 31; i < lim; i += 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(e.residual) + ((m0 + i) * e.ldr + n0) * (EPI == kEpiBf16 ? 2 : 4)));
}
// Residual of tokens m0 .. m0 + NC - 1 of weight row n, as it lies there: bf16 is widened where it is added, which waits
// for it (here every load would be waited for by itself).  Lanes and tokens past the last read the last.
template <int EPI, int NC>
__device__ __forceinline__ void load_residual(uint32_t (&v)[NC], const MxEpilogue& e, int64_t n, int64_t N, int64_t m0, int lim) {
  if (EPI < kEpiF32 || !e.residual || lim <= 0) return;
  const int64_t at = m0 * e.ldr + min(n, N - 1);
  if constexpr (EPI == kEpiBf16) {
    const uint16_t* const p = static_cast<const uint16_t*>(e.residual) + at;
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] = p[min(i, lim - 1) * e.ldr];
  } else {
    const uint32_t* const p = static_cast<const uint32_t*>(e.residual) + at;
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] = p[min(i, lim - 1) * e.ldr];
  }
}
template <int EPI, int NC>
__device__ __forceinline__ void add_residual(uint32_t (&r)[NC], const uint32_t (&v)[NC], const MxEpilogue& e) {
  if (EPI < kEpiF32 || !e.residual) return;
#pragma unroll
  for (int i = 0; i < NC; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(EPI == kEpiBf16 ? v[i] << 16 : v[i]));
}
template <int NC>
__device__ __forceinline__ void bias_act(uint32_t (&r)[NC], const MxEpilogue& e, int64_t n, int64_t N) {
  if (e.bias) {
    const float2 b = pair_of(e.bias[min(n, N - 1)]);
#pragma unroll
    for (int i = 0; i < NC; i += 2) {
      const float2 y = __fadd2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), b);
      r[i] = __float_as_uint(y.x);
      r[i + 1] = __float_as_uint(y.y);
    }
  }
  if (e.act == kActRelu) activate_all<kActRelu>(r);
  else if (e.act == kActSilu) activate_all<kActSilu>(r);
  else if (e.act == kActGelu) activate_all<kActGelu>(r);
  else if (e.act == kActGeluTanh) activate_all<kActGeluTanh>(r);
}

// ---------------------------------------------------------------- stores of Y
// Tokens 0 .. lim - 1 of this lane's weight row n from NC accumulators (r[i] = token
// i); y points at token 0.  bf16: neighbouring lanes trade so that the even lane
// stores the pair (n, n + 1) of token i and the odd lane that of token i + 1, 4 bytes
// each; with an odd N, row stride or address, 2 bytes each.
template <bool BF16, int NC, bool FULL>
__device__ __forceinline__ void store_cols_t(const uint32_t (&r)[NC], void* y, int64_t ldy, int64_t n, int64_t N, int lim) {
  if constexpr (!BF16) {
    float* p = static_cast<float*>(y) + n;
    if (n < N)
#pragma unroll
      for (int i = 0; i < NC; ++i, p += ldy)
        if (FULL || i < lim) *p = __uint_as_float(r[i]);
  } else {
    __nv_bfloat16* base = static_cast<__nv_bfloat16*>(y);
    if (((N | ldy) & 1) == 0 && (reinterpret_cast<uintptr_t>(y) & 3) == 0) {
      const int odd = static_cast<int>(n & 1);
      __nv_bfloat16* p = base + odd * ldy + n - odd;
#pragma unroll
      for (int i = 0; i < NC; i += 2, p += 2 * ldy) {
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? r[i] : r[i + 1], 1);
        const float lo = __uint_as_float(odd ? got : r[i]), hi = __uint_as_float(odd ? r[i + 1] : got);
        if (n < N && (FULL || i + odd < lim)) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(lo, hi);
      }
    } else if (n < N) {
      __nv_bfloat16* p = base + n;
#pragma unroll
      for (int i = 0; i < NC; ++i, p += ldy)
        if (FULL || i < lim) *p = __float2bfloat16_rn(__uint_as_float(r[i]));
    }
  }
}
template <bool BF16, int NC>
__device__ __forceinline__ void store_cols(const uint32_t (&r)[NC], void* y, int64_t ldy, int64_t n, int64_t N, int lim) {
  if (lim >= NC) store_cols_t<BF16, NC, true>(r, y, ldy, n, N, lim);
  else store_cols_t<BF16, NC, false>(r, y, ldy, n, N, lim);
}

// ---------------------------------------------------------------- small
template <int NT>
struct Small {
  static constexpr int kStageBytes = kWBytes + NT * 128 + 2 * kSfTile;
  // stages in flight with two CTAs an SM, and with one
  static constexpr int kRing2 = NT <= 32 ? 5 : NT == 64 ? 4 : 3;
  static constexpr int kRing1 = NT == 16 ? 11 : NT == 32 ? 10 : NT == 64 ? 8 : 6;
  static constexpr int kSfCols = 16, kCols = 256;  // TMEM columns of a stage's scales, of the CTA
  static constexpr int kPartBytes = NT * 512;  // the partial tiles that the CTAs of a split exchange
  static constexpr int kMost1 = 226 * 1024, kMost2 = 113 * 1024;  // shared memory with one CTA an SM, with two
  // Partial tiles behind the stages if that fits, else in their place; and enough that
  // neither a third CTA nor one of the int4 and int8 products (over 148 KB, all of
  // the TMEM) fits beside it on an SM, whose TMEM holds two: one that waited for TMEM
  // while its cluster waits for it could wait for ever.
  static constexpr int kLeast = 80 * 1024;
  static constexpr bool apart(int ring, int most) { return 1024 + ring * kStageBytes + kPartBytes <= most; }
  static constexpr int smem(int ring, int most) {
    const int stages = ring * kStageBytes;
    const int need = 1024 + (apart(ring, most) ? stages + kPartBytes : stages > kPartBytes ? stages : kPartBytes);
    return need > kLeast ? need : kLeast;
  }
  static_assert(kRing1 <= 12 && NT + kRing1 * kSfCols <= kCols && smem(kRing1, kMost1) <= kMost1 && smem(kRing2, kMost2) <= kMost2);
};
constexpr int kSmallThreads = 192;  // 4 epilogue warps, a copy warp, an MMA warp

// grid (S, weight tiles, token tiles), cluster (S, 1, 1).
template <int NT, bool BF16, int EPI>
__global__ void __launch_bounds__(kSmallThreads, 2) mx_small_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                    const __grid_constant__ CUtensorMap amap,
                                                                    const __grid_constant__ CUtensorMap wsmap,
                                                                    const __grid_constant__ CUtensorMap asmap,
                                                                    const MxArgs p) {
  using C = Small<NT>;
  extern __shared__ uint8_t raw[];
  const uint32_t smem = (su32(raw) + 1023u) & ~1023u;
  __shared__ Bars S;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTW, m0 = static_cast<int64_t>(blockIdx.z) * NT;
  const int s0 = static_cast<int>(static_cast<int64_t>(p.stages) * rank / split);
  const int s1 = static_cast<int>(static_cast<int64_t>(p.stages) * (rank + 1) / split);
  constexpr uint32_t kTx = C::kStageBytes;
  auto load = [&](int s, int st) {
    const uint32_t base = smem + st * C::kStageBytes, bar = su32(&S.full[st]);
    mbar_expect_tx(&S.full[st], kTx);
    load_2d<1>(base, &wmap, s * 128, static_cast<int32_t>(n0), bar);
    load_2d<1>(base + kWBytes + NT * 128, &wsmap, s * 256, static_cast<int32_t>(blockIdx.y), bar);
    load_2d<1>(base + kWBytes, &amap, s * 128, static_cast<int32_t>(m0), bar);
    load_2d<1>(base + kWBytes + NT * 128 + kSfTile, &asmap, s * 256, static_cast<int32_t>(m0 >> 7), bar);
  };

  const int first = min(p.ring, s1 - s0);  // stages that need no free slot
  if (warp == 4 && elect_one()) {  // the copies start before the rest of the set-up
    prefetch_map(&wmap);
    prefetch_map(&wsmap);
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.acc_full, 1);
    S.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    grid_dep_wait();
    if (p.delay == 0)
      for (int i = 0; i < first; ++i) load(s0 + i, i);
  }
  if (warp == 5) {
    tmem_alloc<1>(&S.tmem, C::kCols);
    tc_fence_before();
  }
  __syncthreads();
  grid_dep_launch();  // behind the allocation: the next kernel must not take the TMEM this one waits for
  if (split > 1) cluster_arrive_relaxed();
  tc_fence_after();
  const uint32_t tmem = S.tmem;

  if (warp == 4) {
    bool filled = true;
    if (p.delay > 0) {  // a test holds the first copies back, and issues none once a wait gave up
      hold(p);
      filled = !__any_sync(0xFFFFFFFFu, S.abort);
      if (filled && elect_one())
        for (int i = 0; i < first; ++i) load(s0 + i, i);
      __syncwarp();
    }
    int st = 0, round = 0;  // stage s0 + ring + ... reuses slot st after `round` uses
    for (int s = s0 + p.ring; filled && s < s1; ++s) {
      if (!__all_sync(0xFFFFFFFFu, wait_bar(S, &S.empty[st], round & 1, p))) break;
      if (elect_one()) load(s, st);
      __syncwarp();
      if (++st == p.ring) st = 0, ++round;
    }
    if (S.abort && filled)  // copies still in flight must land before the CTA leaves
      for (int i = 0; i < first; ++i) drain_bar(&S.full[i], (i < st ? round + 1 : round) & 1);
  } else if (warp == 5) {
    const uint32_t idesc = mx_idesc(1, NT);
    int st = 0, round = 0;
    for (int s = s0; s < s1; ++s) {
      if (!__all_sync(0xFFFFFFFFu, wait_bar(S, &S.full[st], round & 1, p))) break;
      tc_fence_after();
      const uint32_t base = smem + st * C::kStageBytes;
      if (elect_one()) {
        stage_mmas<1, 1>(tmem, base, base + kWBytes, base + kWBytes + NT * 128, tmem + NT + st * C::kSfCols, idesc,
                         (min(kStageK, p.K - s * kStageK) + 63) / 64, s > s0);
        commit<1>(&S.empty[st]);
      }
      __syncwarp();
      if (++st == p.ring) st = 0, ++round;
    }
    if (elect_one()) commit<1>(&S.acc_full);
    if (S.abort) drain_bar(&S.acc_full, 0);
  }

  __syncwarp();
  if (EPI && warp < 4) {
    grid_dep_wait();  // the residual and the bias may be what the kernel in front of this one writes
    ask_residual<EPI>(p.ep, n0 + 32 * warp, p.N, m0, static_cast<int>(min(static_cast<int64_t>(NT), p.M - m0)));
  }
  const int64_t n = n0 + 32 * (warp & 3) + lane;
  const int tok = static_cast<int>(min(static_cast<int64_t>(NT), p.M - m0));
  constexpr int NC = NT < 32 ? NT : 32;  // columns per pass
  uint32_t res[NC];
  if (EPI && warp < 4 && split == 1) load_residual<EPI>(res, p.ep, n, p.N, m0, tok);
  const bool whole = warp < 4 && __all_sync(0xFFFFFFFFu, wait_bar(S, &S.acc_full, 0, p) && !S.abort);
  tc_fence_after();
  const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  constexpr int kEsz = BF16 ? 2 : 4;
  uint8_t* const y = static_cast<uint8_t*>(p.y) + m0 * p.ldy * kEsz;
  if (split == 1) {
    constexpr int kUnroll = EPI ? 1 : NT / NC;  // the epilogue's code once: its first fetch is a part of such a call's time
    if (whole)
#pragma unroll kUnroll
      for (int c = 0; c < NT; c += NC) {
        uint32_t r[NC];
#pragma unroll
        for (int i = 0; i < NC; i += 16) tmem_ld16(lanes + c + i, *reinterpret_cast<uint32_t(*)[16]>(r + i));
#pragma unroll
        for (int i = 0; i < NC; i += 16) tmem_wait(*reinterpret_cast<uint32_t(*)[16]>(r + i));
        if constexpr (EPI) {
          bias_act(r, p.ep, n, p.N);
          add_residual<EPI>(r, res, p.ep);
          if (c + NC < NT) load_residual<EPI>(res, p.ep, n, p.N, m0 + c + NC, tok - c - NC);
        }
        store_cols<BF16>(r, y + c * p.ldy * kEsz, p.ldy, n, p.N, tok - c);
      }
  } else {
    // rank r sums and writes tokens r * share ..; share is a power of two, 4 at least.
    // Partials: [rank][share / 4][128 rows][4 tokens], 16 bytes a lane.
    const int share = NT / split, log = 31 - __clz(share);
    const uint32_t mine = smem + p.apart + 16u * (rank * (share / 4) * kTW + 32 * (warp & 3) + lane);
    cluster_wait();  // every CTA of the cluster runs
    if (p.apart == 0) {
      cluster_arrive_relaxed();
      cluster_wait();  // and has no MMA that reads its stages
    }
    if (whole)
#pragma unroll
      for (int c = 0; c < NT; c += NC) {
        uint32_t r[NC];
#pragma unroll
        for (int i = 0; i < NC; i += 16) tmem_ld16(lanes + c + i, *reinterpret_cast<uint32_t(*)[16]>(r + i));
#pragma unroll
        for (int i = 0; i < NC; i += 16) tmem_wait(*reinterpret_cast<uint32_t(*)[16]>(r + i));
#pragma unroll
        for (int i = 0; i < NC; i += 4)
          if (c + i < tok)
            asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             map_rank(mine + 16u * ((((c + i) & (share - 1)) >> 2) * kTW), (c + i) >> log)),
                         "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
                         : "memory");
      }
    cluster_sync();
    if (whole) {
      const uint8_t* part = raw + (smem - su32(raw)) + p.apart + 16 * (32 * warp + lane);
      for (int i = 0; i < share && rank * share + i < tok; i += 4) {
        float4 v = *reinterpret_cast<const float4*>(part + 16 * ((i >> 2) * kTW));
        for (int q = 1; q < split; ++q) {
          const float4 o = *reinterpret_cast<const float4*>(part + 16 * ((q * (share >> 2) + (i >> 2)) * kTW));
          v = make_float4(__fadd_rn(v.x, o.x), __fadd_rn(v.y, o.y), __fadd_rn(v.z, o.z), __fadd_rn(v.w, o.w));
        }
        uint32_t r[4] = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
        const int64_t m = static_cast<int64_t>(rank) * share + i;
        if constexpr (EPI) {
          uint32_t v4[4];
          load_residual<EPI>(v4, p.ep, n, p.N, m0 + m, static_cast<int>(tok - m));
          bias_act(r, p.ep, n, p.N);
          add_residual<EPI>(r, v4, p.ep);
        }
        store_cols<BF16>(r, y + m * p.ldy * kEsz, p.ldy, n, p.N, static_cast<int>(tok - m));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_free<1>(tmem, C::kCols);
}

// ---------------------------------------------------------------- pair
constexpr int kMaxTok = 256;
constexpr int kPairStages = 6;
constexpr int kPairAtoms = kMaxTok / 128;
constexpr int kPairSf = kWBytes + (kMaxTok / 2) * 128;
constexpr int kPairStageBytes = kPairSf + (1 + kPairAtoms) * kSfTile;
constexpr int kPairSfCols = 8 + 8 * kPairAtoms;
constexpr int kPairSmem = 1024 + kPairStages * kPairStageBytes;
constexpr int kPairThreads = 320;  // 8 epilogue warps, a copy warp, an MMA warp
static_assert(kMaxTok + kPairStages * kPairSfCols <= 512, "TMEM columns");

// Weight and token tile of tile t.  Whole tiles: tokens first, so that the pairs at work
// share few weight tiles.  With every tile's stages cut, weights first: pairs a token
// tile apart then read the same weights at the same time.
__device__ __forceinline__ int tile_w(const MxArgs& p, int t) { return p.whole == 0 ? t % p.wt : t / p.mt; }
__device__ __forceinline__ int tile_m(const MxArgs& p, int t) { return p.whole == 0 ? t / p.wt : t % p.mt; }

// Tokens of the tile at m0 that the MMA computes: a multiple of 32, whose halves are
// whole 8-row swizzle atoms.
__device__ __forceinline__ int tile_tok(const MxArgs& p, int m0) {
  return static_cast<int>(min(static_cast<int64_t>(kMaxTok), (p.M - m0 + 31) & ~int64_t(31)));
}

// The work of a pair, in order: whole tiles `pair`, pair + pairs, ... below p.whole,
// then the range [lo, hi) of the remaining tiles' stages.  A range is at least a tile
// long, so a tile is cut between two pairs at most: the one whose range ends in it
// holds the first stages (head), the one whose range begins in it the last (tail).
struct Work {
  int tile, s0, s1;  // the segment: stages [s0, s1) of a tile
  int step;
  int cut_tile, cut_s0;  // where the range goes on
  int64_t left;          // its stages still to come
  __device__ __forceinline__ Work(const MxArgs& p, int pair, int pairs) : tile(pair - pairs), s0(0), s1(0), step(pairs) {
    // a pair that waits for a tail waits for one that started before it: ranges in
    // descending order of the pair's number
    const int64_t at = pairs - 1 - pair, lo = p.units * at / pairs;
    left = p.units * (at + 1) / pairs - lo;
    cut_tile = p.whole + static_cast<int>(lo / p.stages);
    cut_s0 = static_cast<int>(lo % p.stages);
  }
  __device__ __forceinline__ bool next(const MxArgs& p) {
    if (tile + step < p.whole) {
      tile += step;
      s1 = p.stages;
      return true;
    }
    if (left <= 0) return false;
    step = p.whole;  // no whole tile follows
    tile = cut_tile++;
    s0 = cut_s0;
    cut_s0 = 0;
    s1 = static_cast<int>(min(static_cast<int64_t>(p.stages), s0 + left));
    left -= s1 - s0;
    return true;
  }
};

// Persistent.  CTA `rank` of the pair holds weight rows 128 rank .. of the tile, one
// half of its tokens as its part of the N operand, and every token's scales.
template <bool BF16, int EPI>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap asmap, const MxArgs p) {
  extern __shared__ uint8_t raw[];
  const uint32_t smem = (su32(raw) + 1023u) & ~1023u;
  __shared__ Bars S;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.acc_empty, 16);  // the epilogue warps of both CTAs
    S.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    tmem_alloc<2>(&S.tmem, 512);
    tc_fence_before();
  }
  if (warp == 8 && elect_one()) {
    prefetch_map(&wmap);
    prefetch_map(&amap);
    prefetch_map(&wsmap);
    prefetch_map(&asmap);
  }
  Work work(p, pair, pairs);
  bool more = work.next(p);
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised
  grid_dep_launch();  // behind the allocation: the next kernel must not take the TMEM this one waits for
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  grid_dep_wait();

  if (warp == 8) {
    const uint32_t tx = 2u * (kWBytes + static_cast<uint32_t>(p.box) * 128u + (1 + kPairAtoms) * kSfTile);
    const uint32_t full0 = map_rank(su32(&S.full[0]), 0);  // the leader's barriers count both CTAs' copies
    int st = 0, round = 0;
    hold(p);
    for (; !S.abort && more; more = work.next(p)) {
      const int32_t w0 = tile_w(p, work.tile) * 256 + static_cast<int32_t>(rank) * kTW;
      const int32_t m0 = tile_m(p, work.tile) * kMaxTok;
      const int32_t half = tile_tok(p, m0) / 2 * static_cast<int32_t>(rank);
      for (int s = work.s0; s < work.s1; ++s) {
        if (round > 0 && !__all_sync(0xFFFFFFFFu, wait_bar(S, &S.empty[st], (round - 1) & 1, p))) break;
        const uint32_t base = smem + st * kPairStageBytes, bar = full0 + st * 8;
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(&S.full[st], tx);
          load_2d<2>(base, &wmap, s * 128, w0, bar);
          load_2d<2>(base + kWBytes, &amap, s * 128, m0 + half, bar);
          load_2d<2>(base + kPairSf, &wsmap, s * 256, w0 >> 7, bar);
#pragma unroll
          for (int a = 0; a < kPairAtoms; ++a)
            load_2d<2>(base + kPairSf + (1 + a) * kSfTile, &asmap, s * 256, (m0 >> 7) + a, bar);
        }
        __syncwarp();
        if (++st == kPairStages) st = 0, ++round;
      }
    }
    if (S.abort && rank == 0)  // copies in flight must land before the CTAs leave
      for (int i = 0; i < kPairStages; ++i)
        if (round > 0 || i < st) drain_bar(&S.full[i], (i < st ? round : round - 1) & 1);
    __syncwarp();
  } else if (warp == 9) {
    if (rank == 0) {  // the whole warp runs the loop, so that what an MMA takes stays in uniform registers
      int st = 0, round = 0, seg = 0;
      for (; !S.abort && more; more = work.next(p)) {
        const uint32_t idesc = mx_idesc(2, tile_tok(p, tile_m(p, work.tile) * kMaxTok));
        if (seg > 0 && !__all_sync(0xFFFFFFFFu, wait_bar(S, &S.acc_empty, static_cast<uint32_t>(seg - 1) & 1, p))) break;
        ++seg;
        tc_fence_after();
        for (int s = work.s0; s < work.s1; ++s) {
          if (!__all_sync(0xFFFFFFFFu, wait_bar(S, &S.full[st], round & 1, p))) break;
          tc_fence_after();
          const uint32_t base = smem + st * kPairStageBytes;
          if (elect_one()) {
            stage_mmas<2, kPairAtoms>(tmem, base, base + kWBytes, base + kPairSf, tmem + kMaxTok + st * kPairSfCols, idesc,
                                      (min(kStageK, p.K - s * kStageK) + 63) / 64, s > work.s0);
            commit<2>(&S.empty[st]);
          }
          __syncwarp();
          if (++st == kPairStages) st = 0, ++round;
        }
        if (elect_one()) commit<2>(&S.acc_full);
        __syncwarp();
      }
      if (S.abort) {  // MMAs in flight: the parity of a further commit is not known, so wait out the bound
        const int64_t t0 = clock64();
        while (clock64() - t0 < kWaitCycles) {
        }
      }
    }
    __syncwarp();
  } else {
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 128 * (warp >> 2);
    const uint32_t empty = map_rank(su32(&S.acc_empty), 0);
    uint32_t seg = 0;
    bool live = true;  // cleared when a wait gave up; the barrier below still counts this warp
    for (; more; more = work.next(p)) {
      if (EPI && work.s0 == 0) {
        const int64_t m0 = static_cast<int64_t>(tile_m(p, work.tile)) * kMaxTok + 128 * (warp >> 2);
        ask_residual<EPI>(p.ep, static_cast<int64_t>(tile_w(p, work.tile)) * 256 + rank * kTW + 32 * (warp & 3), p.N, m0,
                     static_cast<int>(min(static_cast<int64_t>(128), p.M - m0)));
      }
      live = live && __all_sync(0xFFFFFFFFu, wait_bar(S, &S.acc_full, seg & 1, p));
      ++seg;
      uint32_t r[128];
      if (live) {
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32(lanes + c, *reinterpret_cast<uint32_t(*)[32]>(r + c));
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_wait32(*reinterpret_cast<uint32_t(*)[32]>(r + c));
        tc_fence_before();
        __syncwarp();
        if (elect_one())
          // relaxed: the loads from TMEM are complete, and a release would wait for the
          // last tile's stores (over 1000 cycles)
          asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(empty) : "memory");
      }
      // no warp's stores may queue in front of another warp's arrival: the MMAs wait for it
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (!live) continue;
      if (work.s0 > 0) {  // tail: deposit for the pair that holds the head, the next one up
        const int64_t at = (static_cast<int64_t>(pair) * 2 + rank) * 8 + warp;
        float4* part = p.parts + at * 1024 + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          __stcg(part + i * 32, make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                            __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])));
        __threadfence();
        __syncwarp();
        if (lane == 0) asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.flags + at), "r"(1u) : "memory");
        continue;
      }
      if (work.s1 < p.stages) {  // head: add the tail, deposited by the pair before this one
        const int64_t at = (static_cast<int64_t>(pair - 1) * 2 + rank) * 8 + warp;
        const int64_t t0 = clock64();
        uint32_t there = 0;
        while (true) {
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(there) : "l"(p.flags + at) : "memory");
          if (__all_sync(0xFFFFFFFFu, there != 0) || __any_sync(0xFFFFFFFFu, S.abort || clock64() - t0 > p.wait)) break;
        }
        if (!__all_sync(0xFFFFFFFFu, there != 0)) {
          S.abort = 1;
          if (p.err && lane == 0) atomicOr(p.err, 32);
          live = false;
          continue;
        }
        const float4* part = p.parts + at * 1024 + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float4 v = __ldcg(part + i * 32);
          r[4 * i] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i]), v.x));
          r[4 * i + 1] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i + 1]), v.y));
          r[4 * i + 2] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i + 2]), v.z));
          r[4 * i + 3] = __float_as_uint(__fadd_rn(__uint_as_float(r[4 * i + 3]), v.w));
        }
        if (lane == 0) p.flags[at] = 0u;
      }
      const int64_t n = static_cast<int64_t>(tile_w(p, work.tile)) * 256 + rank * kTW + 32 * (warp & 3) + lane;
      const int64_t m0 = static_cast<int64_t>(tile_m(p, work.tile)) * kMaxTok + 128 * (warp >> 2);
      const int lim = static_cast<int>(min(static_cast<int64_t>(128), p.M - m0));
      uint8_t* const y = static_cast<uint8_t*>(p.y) + m0 * p.ldy * (BF16 ? 2 : 4);
      if constexpr (EPI) {
        // 16 tokens at a time: beside the 128 accumulators no more fit the 168 registers that ten warps leave
        uint32_t res[16];
        load_residual<EPI>(res, p.ep, n, p.N, m0, lim);
        bias_act(r, p.ep, n, p.N);
#pragma unroll
        for (int c = 0; c < 128; c += 16) {
          uint32_t (&part)[16] = *reinterpret_cast<uint32_t(*)[16]>(r + c);
          add_residual<EPI>(part, res, p.ep);
          if (c < 112) load_residual<EPI>(res, p.ep, n, p.N, m0 + c + 16, lim - c - 16);
          store_cols<BF16>(part, y + c * p.ldy * (BF16 ? 2 : 4), p.ldy, n, p.N, lim - c);
        }
      } else {
        store_cols<BF16>(r, y, p.ldy, n, p.N, lim);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's MMAs and arrivals no longer touch this CTA
  if (warp == 9) tmem_free<2>(tmem, 512);
}

// ---------------------------------------------------------------- launches
template <class Kernel>
cudaError_t launch(Kernel kernel, bool (&configured)[64], dim3 grid, int threads, int smem, int cluster,
                   const CUtensorMap (&m)[4], const MxArgs& a, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], a);
}

// CTAs that share a tile's K: the power of two up to 8 (a quarter of the tokens at
// most, no CTA without a stage, all CTAs resident) with the least of its stages and its
// exchange.  In units of 10 ns, measured on a GB300: 25 a stage; the exchange of the
// partial tiles 30, 80, 200, 330 for 16, 32, 64, 128 tokens, half as much again with two
// CTAs on an SM.  K17408 N256, one tile of 128 tokens: 19.8 us alone, 8.2 over 8 CTAs;
// K2048 N2560: 4.6 us alone, 7.4 over 2.
int small_split(int nt, int64_t tiles, int stages) {
  const int exchange = nt == 16 ? 30 : nt == 32 ? 80 : nt == 64 ? 200 : 330;
  int best = 1, least = stages * 25;
  for (int split = 2; split <= 8 && split <= nt / 4 && split <= stages && tiles * split <= 2 * num_sms(); split *= 2) {
    const int cost = (stages + split - 1) / split * 25 + (tiles * split > num_sms() ? exchange * 3 / 2 : exchange);
    if (cost < least) best = split, least = cost;
  }
  return best;
}

template <int NT, int EPI>
cudaError_t launch_small(const CUtensorMap (&m)[4], const MxArgs& a, int y_bf16, cudaStream_t st) {
  using C = Small<NT>;
  static bool configured[2][64] = {};
  const int64_t wt = (a.N + kTW - 1) / kTW, mt = (a.M + NT - 1) / NT, tiles = wt * mt;
  const int split = small_split(NT, tiles, a.stages);
  const dim3 grid(split, static_cast<unsigned>(wt), static_cast<unsigned>(mt));
  MxArgs b = a;
  const bool alone = tiles * split <= num_sms();
  const int most = alone ? C::kMost1 : C::kMost2;
  b.ring = alone ? C::kRing1 : C::kRing2;
  if (b.ring > (a.stages + split - 1) / split) b.ring = (a.stages + split - 1) / split;
  b.apart = split > 1 && C::apart(b.ring, most) ? b.ring * C::kStageBytes : 0;
  const int smem = C::smem(b.ring, most);
  return y_bf16 ? launch(mx_small_kernel<NT, true, EPI>, configured[1], grid, kSmallThreads, smem, split, m, b, st)
                : launch(mx_small_kernel<NT, false, EPI>, configured[0], grid, kSmallThreads, smem, split, m, b, st);
}

// The small kernel serves up to 128 tokens, and more while its tiles (128 x 128) have an
// SM each: no pair of SMs to bring together, and K is split.  M512 K17408 N640: 14.0 us,
// the pair kernel 22.0; M256 K5120 N5120 8.1 and 9.6; M512 K5120 N5120 (160 tiles on 152
// SMs) 10.1 and 10.3, at K17408 26.3 and 23.1.
bool use_small(int64_t M, int64_t N) { return M <= 128 || (M + 127) / 128 * ((N + 127) / 128) <= num_sms(); }

// The first MiB of a workspace holds counters that every product leaves at zero (the
// int4 products keep theirs there too, and may be given the same workspace): the flags
// lie in it, the partial tiles behind it.
constexpr size_t kWsCounters = size_t(1) << 20;

// The pair kernel's schedule.
struct PairPlan {
  int mt, tiles, whole, pairs;
  int64_t units;
  size_t ws_bytes;
};
PairPlan plan_pair(int64_t M, int64_t N, int64_t K) {
  PairPlan q{};
  const int64_t pairs = num_sms() / 2, wt = (N + 255) / 256;
  const int stages = static_cast<int>((K + kStageK - 1) / kStageK);
  q.mt = static_cast<int>((M + kMaxTok - 1) / kMaxTok);
  q.tiles = static_cast<int>(wt * q.mt);
  q.whole = q.tiles;
  // Whole tiles leave the pairs idle for the unused part of the last wave.  Cutting the
  // last wave and what is left by stages instead costs a deposit and a pick-up, about
  // kCutStages of MMAs.
  constexpr int kCutStages = 28;
  const int64_t waves = (q.tiles + pairs - 1) / pairs;
  if (q.tiles > pairs && (waves * pairs - q.tiles) * stages > kCutStages * pairs) {
    q.whole = static_cast<int>((waves - 2) * pairs);
    q.units = static_cast<int64_t>(q.tiles - q.whole) * stages;
    q.ws_bytes = kWsCounters + static_cast<size_t>(pairs) * 16 * 1024 * sizeof(float4);
  }
  q.pairs = static_cast<int>(q.tiles < pairs ? q.tiles : pairs);
  return q;
}

}  // namespace

size_t mx_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) { return use_small(M, N) ? 0 : plan_pair(M, N, K).ws_bytes; }

static int64_t g_wait = kWaitCycles, g_delay = 0;
void mx_set_wait_limit(uint64_t wait_ns, uint64_t producer_delay_ns) {
  const auto cycles = [](uint64_t ns) { return static_cast<int64_t>(ns / 100 * 207 + ns % 100 * 207 / 100); };  // 2.07 GHz
  g_wait = wait_ns ? cycles(wait_ns) : kWaitCycles;
  g_delay = cycles(producer_delay_ns);
}

template <int EPI>
static cudaError_t launch_mx(const CUtensorMap (&m)[4], const MxArgs& a, bool small, int pairs, int y_bf16, cudaStream_t stream) {
  if (!small) {
    static bool configured[2][64] = {};
    const dim3 grid(static_cast<unsigned>(2 * pairs));
    return y_bf16 ? launch(mx_pair_kernel<true, EPI>, configured[1], grid, kPairThreads, kPairSmem, 0, m, a, stream)
                  : launch(mx_pair_kernel<false, EPI>, configured[0], grid, kPairThreads, kPairSmem, 0, m, a, stream);
  }
  switch (a.box) {
    case 16: return launch_small<16, EPI>(m, a, y_bf16, stream);
    case 32: return launch_small<32, EPI>(m, a, y_bf16, stream);
    case 64: return launch_small<64, EPI>(m, a, y_bf16, stream);
    default: return launch_small<128, EPI>(m, a, y_bf16, stream);
  }
}

cudaError_t launch_mx_gemm(const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, const uint8_t* a_codes,
                           const uint8_t* a_scales, int64_t M, int64_t K, void* y, int y_bf16, int64_t ldy, void* ws,
                           const MxEpilogue* ep, cudaStream_t stream) {
  MxArgs a{};
  a.y = y; a.ldy = ldy; a.M = M; a.N = N;
  a.K = static_cast<int>(K);
  a.stages = static_cast<int>((K + kStageK - 1) / kStageK);
  a.err = device_error_word();
  a.wait = g_wait;
  a.delay = g_delay;
  if (ep) a.ep = *ep;
  PairPlan q{};
  const bool small = use_small(M, N);
  if (small) {
    a.box = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  } else {
    q = plan_pair(M, N, K);
    a.mt = q.mt; a.wt = static_cast<int>((N + 255) / 256); a.whole = q.tiles;
    if (ws && q.units > 0) {
      a.whole = q.whole;
      a.units = q.units;
      a.flags = static_cast<uint32_t*>(ws);
      a.parts = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + kWsCounters);
    }
    a.box = a.mt > 1 ? kMaxTok / 2 : static_cast<int>((M + 31) / 32 * 16);
  }
  const uint64_t kt = static_cast<uint64_t>((K + 127) / 128) * 128, row = static_cast<uint64_t>(K / 2);
  CUtensorMap m[4];
  cudaError_t e = encode_2d_map(&m[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, row, static_cast<uint64_t>(N), row, 128,
                                kTW, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess)
    e = encode_2d_map(&m[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, row, static_cast<uint64_t>(M), row, 128, static_cast<uint32_t>(a.box),
                      CU_TENSOR_MAP_SWIZZLE_128B);
  // scale tiles as rows of 4-byte words: what lies past the last tile reads as zero
  if (e == cudaSuccess)
    e = encode_2d_map(&m[2], CU_TENSOR_MAP_DATA_TYPE_UINT32, w_scales, kt, static_cast<uint64_t>((N + 127) / 128), kt * 4,
                      256, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e == cudaSuccess)
    e = encode_2d_map(&m[3], CU_TENSOR_MAP_DATA_TYPE_UINT32, a_scales, kt, static_cast<uint64_t>((M + 127) / 128), kt * 4,
                      256, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (e != cudaSuccess) return e;
  if (!ep) return launch_mx<kPlain>(m, a, small, q.pairs, y_bf16, stream);
  if (!ep->residual) return launch_mx<kEpi>(m, a, small, q.pairs, y_bf16, stream);
  return ep->r_bf16 ? launch_mx<kEpiBf16>(m, a, small, q.pairs, y_bf16, stream) : launch_mx<kEpiF32>(m, a, small, q.pairs, y_bf16, stream);
}

}  // namespace w4a4
