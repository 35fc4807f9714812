// The MXFP4 product Y[m][n] = sum_b 2^(Ew + Ea - 254) sum_j w_j a_j on the tensor
// cores' block-scaled path (tcgen05.mma kind::mxf4, one scale byte per 32 elements
// of each operand): the tensor core applies the scales itself, so nothing is folded
// on the CUDA cores.
//
// The weights are the MMA's M operand (128 rows a tile) and the tokens its N operand
// (NT a tile): one token costs no more tensor work than 16, a warp's lanes hold
// consecutive outputs n, and every store of Y is contiguous.  Stages of 256 elements
// of K (128 bytes a row, 128-byte swizzle) and their scale tiles come by TMA; the
// scale tiles go on to TMEM (tcgen05.cp) in front of the MMAs that use them.
//
// A cluster of S CTAs may share one tile, each with a contiguous share of K: the S
// partial tiles are exchanged through distributed shared memory and summed in rank
// order, so the result does not depend on timing and no workspace is needed.
#include <cuda_bf16.h>

#include "tc_ptx.cuh"
#include "w4a4_kernels.cuh"

namespace w4a4 {

namespace {

constexpr int kTW = 128;       // weight rows per tile
constexpr int kStageK = 256;   // elements of K per stage
constexpr int kThreads = 192;  // 4 epilogue warps, a copy warp, an MMA warp
constexpr uint64_t kWaitNs = 1000000000ull;

struct MxArgs {
  const uint8_t* w_scales;
  const uint8_t* a_scales;
  void* y;
  int64_t ldy;
  int64_t M, N;
  int K, ktiles, stages, y_bf16;
  int* err;
};

template <int NT>
struct Cfg {
  static constexpr int kAtoms = NT > 128 ? 2 : 1;  // 128-row scale tiles a token tile touches
  static constexpr int kWBytes = kTW * 128, kABytes = NT * 128;
  static constexpr int kSfW = 1024, kSfA = kAtoms * 1024;
  static constexpr int kStageBytes = kWBytes + kABytes + kSfW + kSfA;
  static constexpr int kStages = NT == 256 ? 4 : NT == 128 ? 6 : 8;
  static constexpr int kSfCols = 8 + 8 * kAtoms;  // TMEM columns of one stage's scales
  static constexpr int kCols = NT + kSfCols * kStages <= 128 ? 128 : NT + kSfCols * kStages <= 256 ? 256 : 512;
  static constexpr int kSmem = 1024 + kStages * kStageBytes;
};

struct Bars {
  uint64_t full[8], empty[8], done;
  uint32_t tmem;
  volatile int abort;
};

// Bounded wait; on giving up, every other wait of the CTA gives up too.
__device__ __forceinline__ bool wait_bar(Bars& S, uint64_t* b, uint32_t parity, int* err) {
  if (mbar_try(b, parity)) return true;
  const uint64_t t0 = gtime();
  while (!mbar_try(b, parity)) {
    if (S.abort) return false;
    if (gtime() - t0 > kWaitNs) {
      S.abort = 1;
      if (err) atomicOr(err, 32);
      return false;
    }
  }
  return true;
}
// As above without the shared give-up, for copies and MMAs in flight.
__device__ __forceinline__ void drain_bar(uint64_t* b, uint32_t parity) {
  const uint64_t t0 = gtime();
  while (!mbar_try(b, parity) && gtime() - t0 < kWaitNs) {
  }
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(su32(dst)),
               "l"(src), "r"(bytes), "r"(su32(bar))
               : "memory");
}

// 512-byte scale tile (32 rows x 16 bytes, no swizzle) to 4 TMEM columns of all four
// lane quarters.
__device__ __forceinline__ void sf_copy(uint32_t taddr, const void* smem) {
  const uint64_t d = static_cast<uint64_t>((su32(smem) >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
                     (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// kind::mxf4 instruction descriptor: A and B e2m1 (code 1), K-major, ue8m0 scales,
// K = 64; sf picks the byte pair of the scale words.
__device__ __forceinline__ uint32_t mx_idesc(int n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(kTW >> 4) << 24) | (sf << 29);
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                       uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t local, uint32_t rank, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

__device__ __forceinline__ void put(const MxArgs& p, int64_t m, int64_t n, float v) {
  if (p.y_bf16)
    static_cast<__nv_bfloat16*>(p.y)[m * p.ldy + n] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.y)[m * p.ldy + n] = v;
}

// grid (S, weight tiles, token tiles), cluster (S, 1, 1).
template <int NT>
__global__ void __launch_bounds__(kThreads, 1) mx_gemm_kernel(const __grid_constant__ CUtensorMap wmap,
                                                              const __grid_constant__ CUtensorMap amap, const MxArgs p) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (su32(raw) & 1023)) & 1023);
  __shared__ Bars S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTW, m0 = static_cast<int64_t>(blockIdx.z) * NT;
  const int s0 = static_cast<int>(static_cast<int64_t>(p.stages) * rank / split);
  const int s1 = static_cast<int>(static_cast<int64_t>(p.stages) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.done, 1);
    S.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&S.tmem)), "n"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;

  if (warp == 4 && lane == 0) {
    const int64_t wt = n0 >> 7, at = m0 >> 7, atiles = (p.M + 127) >> 7;
    int it = 0;
    for (int s = s0; s < s1; ++s, ++it) {
      const int st = it % C::kStages;
      if (it >= C::kStages && !wait_bar(S, &S.empty[st], (it / C::kStages - 1) & 1, p.err)) break;
      uint8_t* base = smem + st * C::kStageBytes;
      const uint32_t sf = 512u * min(2, p.ktiles - 2 * s);
      uint32_t bytes = C::kWBytes + C::kABytes + sf;
      for (int t = 0; t < C::kAtoms; ++t) bytes += at + t < atiles ? sf : 0u;
      mbar_expect_tx(&S.full[st], bytes);
      tma_2d(base, &wmap, s * 128, static_cast<int32_t>(n0), &S.full[st]);
      tma_2d(base + C::kWBytes, &amap, s * 128, static_cast<int32_t>(m0), &S.full[st]);
      uint8_t* sfp = base + C::kWBytes + C::kABytes;
      bulk_load(sfp, p.w_scales + (wt * p.ktiles + 2 * s) * 512, sf, &S.full[st]);
      for (int t = 0; t < C::kAtoms; ++t)
        if (at + t < atiles)
          bulk_load(sfp + C::kSfW + t * 1024, p.a_scales + ((at + t) * p.ktiles + 2 * s) * 512, sf, &S.full[st]);
    }
    if (S.abort)  // copies still in flight must land before the CTA leaves
      for (int i = it > C::kStages ? it - C::kStages : 0; i < it; ++i) drain_bar(&S.full[i % C::kStages], (i / C::kStages) & 1);
  } else if (warp == 5 && lane == 0) {
    // a token tile narrower than a scale tile starts inside it: 32 rows are a column
    const uint32_t sub = NT < 128 ? static_cast<uint32_t>(m0 & 127) >> 5 : 0u;
    int it = 0;
    uint32_t acc = 0;
    for (int s = s0; s < s1; ++s, ++it) {
      const int st = it % C::kStages;
      if (!wait_bar(S, &S.full[st], (it / C::kStages) & 1, p.err)) break;
      tc_fence_after();
      uint8_t* base = smem + st * C::kStageBytes;
      uint8_t* sfp = base + C::kWBytes + C::kABytes;
      const uint32_t sfw = tmem + NT + st * C::kSfCols, sfa = sfw + 8;
      const int steps = (min(kStageK, p.K - s * kStageK) + 63) / 64;  // MMAs of K = 64
      for (int j = 0; 2 * j < steps; ++j) {
        sf_copy(sfw + 4 * j, sfp + 512 * j);
        for (int t = 0; t < C::kAtoms; ++t) sf_copy(sfa + 4 * (j * C::kAtoms + t), sfp + C::kSfW + t * 1024 + 512 * j);
      }
      for (int k = 0; k < steps; ++k) {
        mma_mx(tmem, kmajor_desc_sw128(base) + 2 * k, kmajor_desc_sw128(base + C::kWBytes) + 2 * k,
               mx_idesc(NT, (k & 1) * 2), sfw + 4 * (k >> 1), sfa + 4 * (k >> 1) * C::kAtoms + sub, acc);
        acc = 1;
      }
      mma_commit(&S.empty[st]);
    }
    mma_commit(&S.done);
    if (S.abort) drain_bar(&S.done, 0);
  }

  __syncwarp();
  const bool whole = warp < 4 && __all_sync(0xFFFFFFFFu, wait_bar(S, &S.done, 0, p.err) && !S.abort);
  tc_fence_after();
  const int64_t n = n0 + 32 * (warp & 3) + lane;
  const int tok = static_cast<int>(min(static_cast<int64_t>(NT), p.M - m0));
  if (split == 1) {
    if (whole) {
      for (int c = 0; c < tok; c += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + c, r);
        tmem_wait(r);
        if (n < p.N)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < tok) put(p, m0 + c + i, n, __uint_as_float(r[i]));
      }
    }
  } else {
    // tokens r * share .. of the tile are summed and written by rank r
    const int share = (tok + split - 1) / split;
    cluster_sync();  // every CTA's operand stages are free
    if (whole) {
      for (int c = 0; c < tok; c += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + c, r);
        tmem_wait(r);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c + i < tok) {
            const int to = (c + i) / share, slot = (c + i) % share;
            st_cluster(su32(smem) + 4u * ((rank * share + slot) * kTW + 32 * warp + lane), to, __uint_as_float(r[i]));
          }
      }
    }
    cluster_sync();
    if (whole && n < p.N) {
      const float* part = reinterpret_cast<const float*>(smem) + 32 * warp + lane;
      for (int i = 0; i < share && rank * share + i < tok; ++i) {
        float v = part[i * kTW];
        for (int r = 1; r < split; ++r) v = __fadd_rn(v, part[(r * share + i) * kTW]);
        put(p, m0 + rank * share + i, n, v);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kCols));
}

template <int NT>
cudaError_t launch_tile(const CUtensorMap& wmap, const CUtensorMap& amap, const MxArgs& a, int split, cudaStream_t st) {
  using C = Cfg<NT>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(mx_gemm_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(split, static_cast<unsigned>((a.N + kTW - 1) / kTW), static_cast<unsigned>((a.M + NT - 1) / NT));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<NT>, wmap, amap, a);
}

}  // namespace

cudaError_t launch_mx_gemm(const uint8_t* w_codes, const uint8_t* w_scales, int64_t N, const uint8_t* a_codes,
                           const uint8_t* a_scales, int64_t M, int64_t K, void* y, int y_bf16, int64_t ldy,
                           cudaStream_t stream) {
  MxArgs a{};
  a.w_scales = w_scales; a.a_scales = a_scales; a.y = y; a.ldy = ldy; a.M = M; a.N = N;
  a.K = static_cast<int>(K);
  a.ktiles = static_cast<int>((K + 127) / 128);
  a.stages = static_cast<int>((K + kStageK - 1) / kStageK);
  a.y_bf16 = y_bf16;
  a.err = device_error_word();
  const int nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  const int64_t tiles = ((N + kTW - 1) / kTW) * ((M + nt - 1) / nt);
  // K shared by as many CTAs (a power of two up to 8) as still have two stages each
  // while the tiles leave SMs idle
  int split = 1;
  while (split < 8 && tiles * split * 2 <= num_sms() && a.stages >= split * 4) split *= 2;
  CUtensorMap wmap, amap;
  cudaError_t e = encode_2d_map(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, static_cast<uint64_t>(K / 2),
                                static_cast<uint64_t>(N), static_cast<uint64_t>(K / 2), 128, kTW,
                                CU_TENSOR_MAP_SWIZZLE_128B);
  if (e == cudaSuccess)
    e = encode_2d_map(&amap, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, static_cast<uint64_t>(K / 2),
                      static_cast<uint64_t>(M), static_cast<uint64_t>(K / 2), 128, static_cast<uint32_t>(nt),
                      CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  switch (nt) {
    case 16: return launch_tile<16>(wmap, amap, a, split, stream);
    case 32: return launch_tile<32>(wmap, amap, a, split, stream);
    case 64: return launch_tile<64>(wmap, amap, a, split, stream);
    case 128: return launch_tile<128>(wmap, amap, a, split, stream);
    default: return launch_tile<256>(wmap, amap, a, split, stream);
  }
}

}  // namespace w4a4
