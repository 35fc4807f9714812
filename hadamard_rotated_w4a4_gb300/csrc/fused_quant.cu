// Quantisers fused with what stands in front of them: plain rows to MXFP4, SwiGLU
// and residual addition + RMS norm to int4, int8 or MXFP4, all with the optional
// per-block H32 rotation; and the reading back of the three formats.
//
// All of them stream: one read of each input, one write of each output.  Four lanes
// share a 32-element block (quad_block.cuh), so loads and stores of a warp are
// contiguous and no value passes through shared memory.
//
// Bounds and measurements (GB300, CUDA graphs, inputs larger than L2 in rotation; a plain
// copy reaches 6.8 TB/s).  Between the memory and the issue of instructions (rotation and
// rounding; ncu: 60-76% of issue slots).  M1024 K17408, fp32 inputs near the memory: rows to
// MXFP4 14.0 us (5.8 TB/s), SwiGLU to int8 25.2 (6.5), MXFP4 read back as fp32 13.9 (5.8);
// bf16 inputs, twice the instructions a byte, by their issue: rows to MXFP4 11.9 (3.8),
// SwiGLU to int8 17.9 (5.1), MXFP4 read back as bf16 9.8 (4.6).  Norm of bf16 to int8:
// M16384 K5120 115 us (5.2), M4096 K2048 13.7 (4.4), M16384 K768 19.5 (4.6), one row 2.2;
// M1024 K17408 72 (1.8: see rmsnorm_quantize_kernel).  Two chunks a thread: one loses 13% on
// bf16 rows, four lose 7% on fp32.
#include <cuda_fp16.h>
#include <type_traits>

#include "quad_block.cuh"

namespace w4a4 {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // chunks per thread: their loads are in flight together

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Division of n < 2^31 by a fixed d >= 1: q = (hi32(n * mul) + n) >> shift with shift =
// ceil(log2 d) and mul = floor(2^32 (2^shift - d) / d) + 1 (round-up multiplier).
struct FastDiv {
  uint32_t d, mul, shift;
  explicit FastDiv(int64_t by) : d(static_cast<uint32_t>(by)), shift(0) {
    while ((uint64_t(1) << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// Row and column (in chunks) of flat chunk c.  I = uint32_t where every index of the
// call fits it (fits32), else int64_t with a plain division.
template <typename I>
__device__ __forceinline__ void chunk_at(I c, const FastDiv& f, I& row, I& col) {
  if constexpr (sizeof(I) == 4) row = f.div(c);
  else row = c / f.d;
  col = c - row * static_cast<I>(f.d);
}
// chunks below 2^31 and element offsets below 2^32
bool fits32(int64_t M, int64_t ld, int64_t ld2 = 0) {
  const int64_t top = int64_t(1) << 32;
  return M < top / 8 && M * (ld > ld2 ? ld : ld2) < top;
}

// v = silu(v) * u, silu(g) = g / (1 + 2^(-g log2 e)).  The approximate exponential and
// reciprocal (about 2 units in the last place each, and |g| / 2 more from rounding the
// exponent) stay far below the step of the 8-bit codes that follow.
__device__ __forceinline__ void swiglu8(float (&v)[8], const float (&u)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 g = make_float2(v[i], v[i + 1]);
    const float2 t = __fmul2_rn(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    const float2 y = __fmul2_rn(__fmul2_rn(g, r), make_float2(u[i], u[i + 1]));
    v[i] = y.x;
    v[i + 1] = y.y;
  }
}

// ---------------------------------------------------------------- rows and SwiGLU
// kPair: the rows are silu(x) * x2, else x.
template <int FMT, typename T, bool kPair, typename I>
__global__ void __launch_bounds__(kThreads) rows_quantize_kernel(const T* __restrict__ x, const T* __restrict__ x2,
                                                                 I chunks, FastDiv cpr, I ldx, I ldx2, int rotate,
                                                                 bool wide, QuantOut o) {
  grid_dep_launch();
  grid_dep_wait();
  const int q = threadIdx.x & 3;
  const I first = static_cast<I>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  I row[kUnroll], col[kUnroll];
  bool ok[kUnroll];
  Chunk<T> a[kUnroll] = {}, b[kPair ? kUnroll : 1] = {};
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const I c = first + j * kThreads;
    ok[j] = c < chunks;  // chunks is a multiple of 4: a block's lanes agree
    row[j] = col[j] = 0;
    if (ok[j]) {
      chunk_at<I>(c, cpr, row[j], col[j]);
      a[j].template load<true>(x + row[j] * ldx + col[j] * 8, wide);
      if constexpr (kPair) b[j].template load<true>(x2 + row[j] * ldx2 + col[j] * 8, wide);
    }
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    float v[8];
    a[j].get(v);
    if constexpr (kPair) {
      float u[8];
      b[j].get(u);
      swiglu8(v, u);
    }
    if (rotate) quad_rotate(v, q);
    quad_quantize<FMT, I>(v, q, ok[j], first + j * kThreads, row[j], col[j] >> 2, static_cast<I>(cpr.d >> 2), o);
  }
}

// ---------------------------------------------------------------- residual + RMS norm
struct NoResidual {};

// T threads share a row (T a power of two up to 32, several rows a CTA; or a multiple
// of 32, one row a CTA) and hold C chunks each from the load to the store: h = x + r is
// summed in fp32, squared and summed over the row in a fixed order, and y = h *
// rsqrt(mean + eps) * g goes on to the rotation and the codes.
// Up to four chunks stay in registers, but for 16-48 bytes of some MXFP4 instances.  Eight,
// 64 of the 64 registers that 1024 threads leave each, do not: 0.4-1.5 KB a thread goes
// through local memory, on rows of K above 16384 where there are more rows than SMs, and
// on all of K above 32768 (M1024 bf16 to int8: K16384 33 us, K17408 72 us).
template <int FMT, typename TX, typename TR, int C>
__global__ void __launch_bounds__(1024) rmsnorm_quantize_kernel(const TX* __restrict__ x, const TR* r, TR* r_out,
                                                                const void* __restrict__ g, int g_bf16, int64_t M, int cpr,
                                                                int64_t ldx, int64_t ldr, int64_t ldr_out, float eps, int T,
                                                                int rotate, bool wide, QuantOut o) {
  constexpr bool kRes = !std::is_same<TR, NoResidual>::value;
  __shared__ float part[32];
  grid_dep_launch();
  grid_dep_wait();
  const int t = T > 32 ? threadIdx.x : threadIdx.x & (T - 1);
  const int64_t row = T > 32 ? static_cast<int64_t>(blockIdx.x)
                             : static_cast<int64_t>(blockIdx.x) * (blockDim.x / T) + threadIdx.x / T;
  const int q = threadIdx.x & 3;
  const bool in = row < M;
  x += row * ldx;
  if constexpr (kRes) {
    r += row * ldr;
    r_out += row * ldr_out;
  }
  // Residual chunks are loaded beside x's while the registers allow it (a load behind
  // the first store of r_out, which may be r, waits for both loads in front of it).
  constexpr bool kAhead = kRes && C * (sizeof(std::conditional_t<kRes, TR, float>) == 2 ? 4 : 8) <= 16;
  using RChunk = Chunk<std::conditional_t<kRes, TR, float>>;
  float v[C][8];
  RChunk ra[kAhead ? C : 1];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int col = t + j * T;
    if (in && col < cpr) {
      Chunk<TX> a;
      a.load(x + col * 8, wide);
      if constexpr (kAhead) ra[j].load(r + col * 8, wide);
      a.get(v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    }
  }
  if constexpr (kRes) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = t + j * T;
      if (in && col < cpr) {
        float u[8];
        if constexpr (kAhead) {
          ra[j].get(u);
        } else {
          ra[0].load(r + col * 8, wide);
          ra[0].get(u);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 h = __fadd2_rn(make_float2(v[j][i], v[j][i + 1]), make_float2(u[i], u[i + 1]));
          v[j][i] = h.x;
          v[j][i + 1] = h.y;
        }
        store8(r_out + col * 8, v[j], wide);
      }
    }
  }
  float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 h = make_float2(v[j][i], v[j][i + 1]);
      s2 = __ffma2_rn(h, h, s2);
    }
  float s = __fadd_rn(s2.x, s2.y);
  for (int d = 1; d < min(T, 32); d <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  if (T > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    s = lane < T / 32 ? part[lane] : 0.0f;
    for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  }
  const float inv = rsqrtf(__fadd_rn(__fdiv_rn(s, static_cast<float>(cpr * 8)), eps));
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int col = t + j * T;
    const bool ok = in && col < cpr;
    if (ok) {
      float w[8];
      if (g == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
      } else if (g_bf16) {
        Chunk<__nv_bfloat16> a;
        a.load(static_cast<const __nv_bfloat16*>(g) + col * 8, false);
        a.get(w);
      } else {
        Chunk<float> a;
        a.load(static_cast<const float*>(g) + col * 8, wide);
        a.get(w);
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 y = __fmul2_rn(__fmul2_rn(make_float2(v[j][i], v[j][i + 1]), make_float2(inv, inv)),
                                    make_float2(w[i], w[i + 1]));
        v[j][i] = y.x;
        v[j][i + 1] = y.y;
      }
    }
    if (rotate) quad_rotate(v[j], q);
    quad_quantize<FMT, int64_t>(v[j], q, ok, row * cpr + col, row, col >> 2, cpr >> 2, o);
  }
}

// ---------------------------------------------------------------- reading back
template <int FMT, typename TY, typename I>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const void* __restrict__ scales, I chunks, FastDiv cpr,
                                                              I ktiles, TY* __restrict__ y, I ldy, bool wide) {
  grid_dep_launch();
  grid_dep_wait();
  const I first = static_cast<I>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint2 w[kUnroll];
  float d[kUnroll];
  I row[kUnroll], col[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const I c = first + j * kThreads;
    if (c >= chunks) continue;
    chunk_at<I>(c, cpr, row[j], col[j]);
    if constexpr (FMT == kMx) {
      w[j].x = __ldg(reinterpret_cast<const uint32_t*>(codes) + c);
      const uint32_t e = __ldg(static_cast<const uint8_t*>(scales) + mx_scale_at<I>(row[j], col[j] >> 2, ktiles));
      // 2^(e - 127): byte 0 is the subnormal 2^-127, byte 255 is NaN
      d[j] = __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
    } else if constexpr (FMT == kInt8) {
      w[j] = __ldg(reinterpret_cast<const uint2*>(codes) + c);
      d[j] = __ldg(static_cast<const float*>(scales) + (c >> 2));
    } else {  // elements 0..15 in the low nibbles of the block's 16 bytes, 16..31 in the high ones
      w[j] = __ldg(reinterpret_cast<const uint2*>(codes) + (c >> 2) * 2 + (c & 1));
      d[j] = __ldg(static_cast<const float*>(scales) + (c >> 2));
    }
  }
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const I c = first + j * kThreads;
    if (c >= chunks) continue;
    float v[8];
    if constexpr (FMT == kMx) {
      uint32_t h[4];  // pairs of f16, exact
      asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
          "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
          "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
          : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
          : "r"(w[j].x));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __half2 p;
        memcpy(&p, &h[i], 4);
        const float2 f = __fmul2_rn(__half22float2(p), make_float2(d[j], d[j]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    } else {
      const int up = FMT == kInt4 && (c & 2) == 0 ? 4 : 0;  // an int4 code to the top of its byte
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t word = (i < 4 ? w[j].x : w[j].y) << up;
        const int code = static_cast<int>(word << (24 - 8 * (i & 3))) >> (FMT == kInt8 ? 24 : 28);
        v[i] = __fmul_rn(static_cast<float>(code), d[j]);
      }
    }
    store8(y + row[j] * ldy + col[j] * 8, v, wide);
  }
}

// ---------------------------------------------------------------- MXFP4 import
template <typename I>
__global__ void __launch_bounds__(kThreads) import_mx_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, I nblk, FastDiv bpr,
                                                             I ktiles, uint8_t* __restrict__ out,
                                                             uint8_t* __restrict__ out_scales) {
  grid_dep_launch();
  grid_dep_wait();
  const I i = static_cast<I>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= nblk) return;
  I row, blk;
  chunk_at<I>(i, bpr, row, blk);
  reinterpret_cast<uint4*>(out)[i] = __ldg(reinterpret_cast<const uint4*>(codes) + i);
  uint8_t* s = out_scales + mx_scale_at<I>(row, blk, ktiles);
  *s = __ldg(scales + i);
  if (blk == bpr.d - 1)
    for (int p = 1; p < 4 - static_cast<int>(blk & 3); ++p) s[p] = 0;
}

// Launch that may begin before the kernel in front of it ends; each kernel here waits
// for that one's results itself.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int threads, cudaStream_t st, A... args) {
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int64_t grid_for(int64_t items, int per_thread) { return (items + kThreads * per_thread - 1) / (kThreads * per_thread); }

template <int FMT, typename T, bool kPair>
cudaError_t launch_rows(const void* x, const void* x2, int64_t M, int64_t K, int64_t ldx, int64_t ldx2, int rotate,
                        const QuantOut& o, cudaStream_t st) {
  const int64_t chunks = M * (K / 8), grid = grid_for(chunks, kUnroll);
  const T *a = static_cast<const T*>(x), *b = static_cast<const T*>(x2);
  const FastDiv cpr(K / 8);
  const bool wide = wide_rows(a, ldx) && (!b || wide_rows(b, ldx2));
  return fits32(M, ldx, ldx2)
             ? launch(rows_quantize_kernel<FMT, T, kPair, uint32_t>, grid, kThreads, st, a, b, chunks, cpr, ldx, ldx2, rotate, wide, o)
             : launch(rows_quantize_kernel<FMT, T, kPair, int64_t>, grid, kThreads, st, a, b, chunks, cpr, ldx, ldx2, rotate, wide, o);
}

template <int FMT, typename TX, typename TR, int C>
cudaError_t launch_norm_c(const NormArgs& n, const QuantOut& o, int64_t grid, int threads, int T, cudaStream_t st) {
  const TX* x = static_cast<const TX*>(n.x);
  const TR* r = static_cast<const TR*>(n.r);
  TR* ro = static_cast<TR*>(n.r_out);
  // 32-byte accesses for every fp32 operand, or for none
  bool wide = (reinterpret_cast<uintptr_t>(n.g) & 31) == 0 && (n.x_bf16 || wide_rows(reinterpret_cast<const float*>(x), n.ldx));
  if (r && !n.r_bf16)
    wide = wide && wide_rows(reinterpret_cast<const float*>(r), n.ldr) && wide_rows(reinterpret_cast<const float*>(ro), n.ldr_out);
  return launch(rmsnorm_quantize_kernel<FMT, TX, TR, C>, grid, threads, st, x, r, ro, n.g, n.g_bf16, n.M,
                static_cast<int>(n.K / 8), n.ldx, n.ldr, n.ldr_out, n.eps, T, n.rotate, wide, o);
}

template <int FMT, typename TX, typename TR>
cudaError_t launch_norm(const NormArgs& n, const QuantOut& o, cudaStream_t st) {
  const int64_t cpr = n.K / 8;
  int T, C = 1, threads;
  if (cpr <= 32) {  // several rows a CTA
    T = 4;
    while (T < cpr) T *= 2;
    threads = 128;
  } else {
    // few rows: as many threads a row as there are, for the shortest chain; many rows:
    // up to 512 threads, for more than one row on an SM (M16384 K5120 bf16: 117 us, with
    // up to 256 threads 128, up to 1024 124)
    const int64_t most = n.M <= num_sms() ? 1024 : 512;
    while (C < 8 && (cpr + C - 1) / C > most) C *= 2;
    threads = T = static_cast<int>(((cpr + C - 1) / C + 31) / 32 * 32);
  }
  const int64_t grid = (n.M + threads / T - 1) / (threads / T);
  if (C == 1) return launch_norm_c<FMT, TX, TR, 1>(n, o, grid, threads, T, st);
  if (C == 2) return launch_norm_c<FMT, TX, TR, 2>(n, o, grid, threads, T, st);
  if (C == 4) return launch_norm_c<FMT, TX, TR, 4>(n, o, grid, threads, T, st);
  return launch_norm_c<FMT, TX, TR, 8>(n, o, grid, threads, T, st);
}

template <int FMT, typename TX>
cudaError_t launch_norm_r(const NormArgs& n, const QuantOut& o, cudaStream_t st) {
  if (!n.r) return launch_norm<FMT, TX, NoResidual>(n, o, st);
  return n.r_bf16 ? launch_norm<FMT, TX, __nv_bfloat16>(n, o, st) : launch_norm<FMT, TX, float>(n, o, st);
}

template <int FMT>
cudaError_t launch_norm_x(const NormArgs& n, const QuantOut& o, cudaStream_t st) {
  return n.x_bf16 ? launch_norm_r<FMT, __nv_bfloat16>(n, o, st) : launch_norm_r<FMT, float>(n, o, st);
}

template <int FMT, typename TY>
cudaError_t launch_back(const uint8_t* codes, const void* scales, int64_t M, int64_t K, void* y, int64_t ldy,
                        cudaStream_t st) {
  const int64_t chunks = M * (K / 8), kt = (K + 127) / 128, grid = grid_for(chunks, kUnroll);
  const FastDiv cpr(K / 8);
  TY* out = static_cast<TY*>(y);
  const bool wide = wide_rows(out, ldy);
  return fits32(M, ldy)
             ? launch(dequantize_kernel<FMT, TY, uint32_t>, grid, kThreads, st, codes, scales, chunks, cpr, kt, out, ldy, wide)
             : launch(dequantize_kernel<FMT, TY, int64_t>, grid, kThreads, st, codes, scales, chunks, cpr, kt, out, ldy, wide);
}

}  // namespace

cudaError_t launch_rows_quantize(int fmt, const void* x, const void* x2, int bf16, int64_t M, int64_t K, int64_t ldx,
                                 int64_t ldx2, int rotate, uint8_t* codes, void* scales, uint8_t* expanded,
                                 cudaStream_t st) {
  const QuantOut o{codes, scales, expanded, (K + 127) / 128};
  auto go = [&](auto f32, auto b16) { return (bf16 ? b16 : f32)(x, x2, M, K, ldx, ldx2, rotate, o, st); };
  if (!x2) return go(launch_rows<kMx, float, false>, launch_rows<kMx, __nv_bfloat16, false>);
  if (fmt == kInt4) return go(launch_rows<kInt4, float, true>, launch_rows<kInt4, __nv_bfloat16, true>);
  if (fmt == kInt8) return go(launch_rows<kInt8, float, true>, launch_rows<kInt8, __nv_bfloat16, true>);
  return go(launch_rows<kMx, float, true>, launch_rows<kMx, __nv_bfloat16, true>);
}

cudaError_t launch_rmsnorm_quantize(int fmt, const NormArgs& n, uint8_t* codes, void* scales, uint8_t* expanded,
                                    cudaStream_t st) {
  const QuantOut o{codes, scales, expanded, (n.K + 127) / 128};
  if (fmt == kInt4) return launch_norm_x<kInt4>(n, o, st);
  if (fmt == kInt8) return launch_norm_x<kInt8>(n, o, st);
  return launch_norm_x<kMx>(n, o, st);
}

cudaError_t launch_dequantize(int fmt, const uint8_t* codes, const void* scales, int64_t M, int64_t K, void* y,
                              int y_bf16, int64_t ldy, cudaStream_t st) {
  auto go = [&](auto f32, auto b16) { return (y_bf16 ? b16 : f32)(codes, scales, M, K, y, ldy, st); };
  if (fmt == kInt4) return go(launch_back<kInt4, float>, launch_back<kInt4, __nv_bfloat16>);
  if (fmt == kInt8) return go(launch_back<kInt8, float>, launch_back<kInt8, __nv_bfloat16>);
  return go(launch_back<kMx, float>, launch_back<kMx, __nv_bfloat16>);
}

cudaError_t launch_import_mx(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, uint8_t* out,
                             uint8_t* out_scales, cudaStream_t st) {
  const int64_t B = K / 32, kt = (K + 127) / 128, grid = grid_for(rows * B, 1);
  const FastDiv bpr(B);
  return fits32(rows, K)
             ? launch(import_mx_kernel<uint32_t>, grid, kThreads, st, codes, scales, rows * B, bpr, kt, out, out_scales)
             : launch(import_mx_kernel<int64_t>, grid, kThreads, st, codes, scales, rows * B, bpr, kt, out, out_scales);
}

}  // namespace w4a4
