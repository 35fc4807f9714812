// Quantisers fused with what stands in front of them: plain rows to MXFP4, SwiGLU
// and residual addition + RMS norm to int4, int8 or MXFP4, all with the optional
// per-block H32 rotation; and the reading back of the three formats.
//
// All of them stream: one read of each input, one write of each output.  Four lanes
// share a 32-element block (quad_block.cuh), so loads and stores of a warp are
// contiguous and no value passes through shared memory.
#include "quad_block.cuh"

namespace w4a4 {

namespace {

constexpr int kThreads = 256;

// Row and column (in chunks) of flat chunk c; the 32-bit division serves all but
// inputs of 2^32 chunks and more.
__device__ __forceinline__ void chunk_at(int64_t c, int64_t cpr, int64_t& row, int64_t& col) {
  if ((c >> 32) == 0) {
    const uint32_t r = static_cast<uint32_t>(c) / static_cast<uint32_t>(cpr);
    row = r;
    col = static_cast<uint32_t>(c) - r * static_cast<uint32_t>(cpr);
  } else {
    row = c / cpr;
    col = c - row * cpr;
  }
}

// silu(g) * u.  The fast exponential and quotient are good to a few units in the last
// place, far below the step of the 8-bit codes that follow.
__device__ __forceinline__ float swiglu(float g, float u) {
  return __fmul_rn(__fdividef(g, __fadd_rn(1.0f, __expf(-g))), u);
}

// ---------------------------------------------------------------- rows and SwiGLU
// kPair: the rows are silu(x) * x2, else x.
template <int FMT, typename T, bool kPair>
__global__ void __launch_bounds__(kThreads) rows_quantize_kernel(const T* __restrict__ x, const T* __restrict__ x2,
                                                                 int64_t chunks, int64_t cpr, int64_t ldx, int64_t ldx2,
                                                                 int rotate, QuantOut o) {
  const int q = threadIdx.x & 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  // whole warps iterate (the shuffles need all lanes); chunks is a multiple of 4
  for (int64_t c = first; c - (threadIdx.x & 31) < chunks; c += step) {
    const bool ok = c < chunks;
    int64_t row = 0, col = 0;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (ok) {
      chunk_at(c, cpr, row, col);
      load8(x + row * ldx + col * 8, v);
      if constexpr (kPair) {
        float u[8];
        load8(x2 + row * ldx2 + col * 8, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = swiglu(v[i], u[i]);
      }
    }
    if (rotate) quad_rotate(v, q);
    quad_quantize<FMT>(v, q, ok, c, row, col >> 2, cpr >> 2, o);
  }
}

// ---------------------------------------------------------------- residual + RMS norm
struct NoResidual {};

template <typename TR>
__device__ __forceinline__ void add_residual(float (&v)[8], const TR* r) {
  float u[8];
  load8(r, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(v[i], u[i]);
}

// T threads share a row (T a power of two up to 32, several rows a CTA; or a multiple
// of 32, one row a CTA) and hold C chunks each, in registers from the load to the
// store: h = x + r is summed in fp32, squared and summed over the row in a fixed
// order, and y = h * rsqrt(mean + eps) * g goes on to the rotation and the codes.
template <int FMT, typename TX, typename TR, int C>
__global__ void __launch_bounds__(1024) rmsnorm_quantize_kernel(const TX* __restrict__ x, const TR* r, TR* r_out,
                                                                const void* __restrict__ g, int g_bf16, int64_t M,
                                                                int64_t cpr, int64_t ldx, int64_t ldr, int64_t ldr_out,
                                                                float eps, int T, int rotate, QuantOut o) {
  constexpr bool kRes = !std::is_same<TR, NoResidual>::value;
  __shared__ float part[32];
  const int t = threadIdx.x % T;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / T) + threadIdx.x / T;
  const int q = threadIdx.x & 3;
  const bool in = row < M;
  float v[C][8];
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int64_t col = t + static_cast<int64_t>(j) * T;
    if (in && col < cpr) {
      load8(x + row * ldx + col * 8, v[j]);
      if constexpr (kRes) {
        add_residual(v[j], r + row * ldr + col * 8);
        store8(r_out + row * ldr_out + col * 8, v[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __fmaf_rn(v[j][i], v[j][i], s);
  }
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
    const int64_t col = t + static_cast<int64_t>(j) * T;
    const bool ok = in && col < cpr;
    if (ok) {
      float w[8];
      if (g == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
      } else if (g_bf16) {
        load8(static_cast<const __nv_bfloat16*>(g) + col * 8, w);
      } else {
        load8(static_cast<const float*>(g) + col * 8, w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = __fmul_rn(__fmul_rn(v[j][i], inv), w[i]);
    }
    if (rotate) quad_rotate(v[j], q);
    quad_quantize<FMT>(v[j], q, ok, row * cpr + col, row, col >> 2, cpr >> 2, o);
  }
}

// ---------------------------------------------------------------- reading back
template <int FMT, typename TY>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const void* __restrict__ scales, int64_t chunks,
                                                              int64_t cpr, int64_t ktiles, TY* __restrict__ y,
                                                              int64_t ldy) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; c < chunks; c += step) {
    int64_t row, col;
    chunk_at(c, cpr, row, col);
    float v[8];
    if constexpr (FMT == kMx) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + c);
      const uint32_t e = __ldg(static_cast<const uint8_t*>(scales) + mx_scale_at(row, col >> 2, ktiles));
      // 2^(e - 127): byte 0 is the subnormal 2^-127, byte 255 is NaN
      const float d = e == 0 ? __uint_as_float(0x00400000u)
                             : e == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(e << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t n = (w >> (4 * i)) & 15u, p = (n >> 1) & 3u, f = n & 1u;
        // exponent p and mantissa bit f: p = 0 is f / 2, else (1 + f / 2) 2^(p - 1)
        const uint32_t mag = p == 0 ? (f ? 0x3F000000u : 0u) : ((p + 126u) << 23) | (f << 22);
        v[i] = __fmul_rn(__uint_as_float(mag | ((n >> 3) << 31)), d);
      }
    } else {
      const float d = __ldg(static_cast<const float*>(scales) + (c >> 2));
      uint2 w;
      int shift;
      if constexpr (FMT == kInt8) {
        w = __ldg(reinterpret_cast<const uint2*>(codes) + c);
        shift = 24;
      } else {  // elements 0..15 in the low nibbles of the block's 16 bytes, 16..31 in the high ones
        const int q = static_cast<int>(c & 3);
        w = __ldg(reinterpret_cast<const uint2*>(codes + (c >> 2) * 16 + (q & 1) * 8));
        shift = q < 2 ? 28 : 24;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t word = i < 4 ? w.x : w.y;
        int code = static_cast<int>(word << (24 - 8 * (i & 3)));  // byte to the top
        if constexpr (FMT == kInt8) code >>= 24;
        else code = (shift == 28 ? code << 4 : code) >> 28;
        v[i] = __fmul_rn(static_cast<float>(code), d);
      }
    }
    store8(y + row * ldy + col * 8, v);
  }
}

// ---------------------------------------------------------------- MXFP4 import
__global__ void __launch_bounds__(kThreads) import_mx_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t nblk, int64_t B,
                                                             int64_t ktiles, uint8_t* __restrict__ out,
                                                             uint8_t* __restrict__ out_scales) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < nblk; i += step) {
    int64_t row, blk;
    chunk_at(i, B, row, blk);
    reinterpret_cast<uint4*>(out)[i] = __ldg(reinterpret_cast<const uint4*>(codes) + i);
    uint8_t* s = out_scales + mx_scale_at(row, blk, ktiles);
    *s = __ldg(scales + i);
    if (blk == B - 1)
      for (int64_t p = 1; p < 4 - (blk & 3); ++p) s[p] = 0;
  }
}

unsigned grid_for(int64_t items) {
  const int64_t want = (items + kThreads - 1) / kThreads, cap = static_cast<int64_t>(num_sms()) * 8;
  return static_cast<unsigned>(want < cap ? want : cap);
}

template <int FMT, typename T>
void launch_rows(const void* x, const void* x2, int64_t M, int64_t K, int64_t ldx, int64_t ldx2, int rotate,
                 const QuantOut& o, cudaStream_t st) {
  const int64_t chunks = M * (K / 8);
  const T* a = static_cast<const T*>(x);
  const T* b = static_cast<const T*>(x2);
  if (b)
    rows_quantize_kernel<FMT, T, true><<<grid_for(chunks), kThreads, 0, st>>>(a, b, chunks, K / 8, ldx, ldx2, rotate, o);
  else if constexpr (FMT == kMx)
    rows_quantize_kernel<FMT, T, false><<<grid_for(chunks), kThreads, 0, st>>>(a, b, chunks, K / 8, ldx, ldx2, rotate, o);
}

template <int FMT, typename TX, typename TR>
void launch_norm(const NormArgs& n, const QuantOut& o, cudaStream_t st) {
  const int64_t cpr = n.K / 8;
  int T, C = 1, threads;
  if (cpr <= 32) {  // several rows a CTA
    T = 4;
    while (T < cpr) T *= 2;
    threads = 128;
  } else {
    // few rows: as many threads a row as there are, for the shortest chain; many rows:
    // up to 512 threads, for more than one row on an SM
    const int64_t most = n.M <= num_sms() ? 1024 : 512;
    while (C < 8 && (cpr + C - 1) / C > most) C *= 2;
    threads = T = static_cast<int>(((cpr + C - 1) / C + 31) / 32 * 32);
  }
  const unsigned grid = static_cast<unsigned>((n.M + threads / T - 1) / (threads / T));
  const TX* x = static_cast<const TX*>(n.x);
  const TR* r = static_cast<const TR*>(n.r);
  TR* ro = static_cast<TR*>(n.r_out);
  auto go = [&](auto kernel) {
    kernel<<<grid, threads, 0, st>>>(x, r, ro, n.g, n.g_bf16, n.M, cpr, n.ldx, n.ldr, n.ldr_out, n.eps, T, n.rotate, o);
  };
  if (C == 1) go(rmsnorm_quantize_kernel<FMT, TX, TR, 1>);
  else if (C == 2) go(rmsnorm_quantize_kernel<FMT, TX, TR, 2>);
  else if (C == 4) go(rmsnorm_quantize_kernel<FMT, TX, TR, 4>);
  else go(rmsnorm_quantize_kernel<FMT, TX, TR, 8>);
}

template <int FMT, typename TX>
void launch_norm_r(const NormArgs& n, const QuantOut& o, cudaStream_t st) {
  if (!n.r) launch_norm<FMT, TX, NoResidual>(n, o, st);
  else if (n.r_bf16) launch_norm<FMT, TX, __nv_bfloat16>(n, o, st);
  else launch_norm<FMT, TX, float>(n, o, st);
}

template <int FMT>
void launch_norm_x(const NormArgs& n, const QuantOut& o, cudaStream_t st) {
  if (n.x_bf16) launch_norm_r<FMT, __nv_bfloat16>(n, o, st);
  else launch_norm_r<FMT, float>(n, o, st);
}

template <int FMT>
void launch_back(const uint8_t* codes, const void* scales, int64_t M, int64_t K, void* y, int y_bf16, int64_t ldy,
                 cudaStream_t st) {
  const int64_t chunks = M * (K / 8), kt = (K + 127) / 128;
  if (y_bf16)
    dequantize_kernel<FMT, __nv_bfloat16><<<grid_for(chunks), kThreads, 0, st>>>(
        codes, scales, chunks, K / 8, kt, static_cast<__nv_bfloat16*>(y), ldy);
  else
    dequantize_kernel<FMT, float><<<grid_for(chunks), kThreads, 0, st>>>(codes, scales, chunks, K / 8, kt,
                                                                         static_cast<float*>(y), ldy);
}

}  // namespace

cudaError_t launch_rows_quantize(int fmt, const void* x, const void* x2, int bf16, int64_t M, int64_t K, int64_t ldx,
                                 int64_t ldx2, int rotate, uint8_t* codes, void* scales, uint8_t* expanded,
                                 cudaStream_t st) {
  const QuantOut o{codes, scales, expanded, (K + 127) / 128};
  auto go = [&](auto f32, auto b16) { bf16 ? b16(x, x2, M, K, ldx, ldx2, rotate, o, st) : f32(x, x2, M, K, ldx, ldx2, rotate, o, st); };
  if (fmt == kInt4) go(launch_rows<kInt4, float>, launch_rows<kInt4, __nv_bfloat16>);
  else if (fmt == kInt8) go(launch_rows<kInt8, float>, launch_rows<kInt8, __nv_bfloat16>);
  else go(launch_rows<kMx, float>, launch_rows<kMx, __nv_bfloat16>);
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm_quantize(int fmt, const NormArgs& n, uint8_t* codes, void* scales, uint8_t* expanded,
                                    cudaStream_t st) {
  const QuantOut o{codes, scales, expanded, (n.K + 127) / 128};
  if (fmt == kInt4) launch_norm_x<kInt4>(n, o, st);
  else if (fmt == kInt8) launch_norm_x<kInt8>(n, o, st);
  else launch_norm_x<kMx>(n, o, st);
  return cudaGetLastError();
}

cudaError_t launch_dequantize(int fmt, const uint8_t* codes, const void* scales, int64_t M, int64_t K, void* y,
                              int y_bf16, int64_t ldy, cudaStream_t st) {
  if (fmt == kInt4) launch_back<kInt4>(codes, scales, M, K, y, y_bf16, ldy, st);
  else if (fmt == kInt8) launch_back<kInt8>(codes, scales, M, K, y, y_bf16, ldy, st);
  else launch_back<kMx>(codes, scales, M, K, y, y_bf16, ldy, st);
  return cudaGetLastError();
}

cudaError_t launch_import_mx(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, uint8_t* out,
                             uint8_t* out_scales, cudaStream_t st) {
  const int64_t B = K / 32;
  import_mx_kernel<<<grid_for(rows * B), kThreads, 0, st>>>(codes, scales, rows * B, B, (K + 127) / 128, out, out_scales);
  return cudaGetLastError();
}

}  // namespace w4a4
