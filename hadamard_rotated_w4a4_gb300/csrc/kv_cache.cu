// Appending to the 8-bit paged key/value cache, and reading it back.
//
// Append: x1, x2 -> x1 cos - x2 sin, x2 cos + x1 sin at the token's position (q and k),
// then H32 per 32 elements (k and v), then int8.  The 16 tokens of a block share one
// power-of-two scale per head, for K and for V: 2^E, E the least with amax <= 127 * 2^E.
// A block is filled by several calls.  When a later token needs a larger E, the codes
// before it are rounded to it: a shift, so that k such steps leave an error of less than
// (1/2 + 1/4 + ...) of the last step, one step at most whatever the order of the tokens.
// (Scales amax / 127 would add half a step each time.)
//
// A warp quantises one (block, head, K or V): its 16 x D values stay in registers between
// the maximum and the rounding, so everything is read once.  Angles are taken in 64 bits
// as turns and reduced there, for 16 tokens once per CTA, and the CTA's heads share them.
#include <cuda_bf16.h>

#include "kv_cache.cuh"
#include "quad_block.cuh"

namespace w4a4 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Blocks of 16 tokens that the last n of len tokens touch, and the first of them.
__device__ __forceinline__ int touched(const Seq& q, int& first) {
  const int start = max(q.len - q.n, 0);
  first = start / kKvTokens;
  return q.n == 0 || q.len == 0 ? 0 : (q.len + kKvTokens - 1) / kKvTokens - first;
}

// The x-th touched block of a call: sequence, block, or b = -1.
struct Found {
  int b, block;
  Seq q;
};
__device__ __forceinline__ Found find_block(const KvSeqs& s, int page, int x, int* err) {  // by a whole warp
  const int lane = threadIdx.x & 31;
  Found f{-1, 0, {}};
  if (!s.cu) {
    const int most = (s.each + kKvTokens - 2) / kKvTokens + 1;  // that each tokens can touch
    const int b = x / most;
    if (b >= s.batch) return f;
    f.q = kv_seq(s, b, page, err);
    int first;
    const int n = touched(f.q, first);
    if (x % most < n) f.b = b, f.block = first + x % most;
    return f;
  }
  for (int b0 = 0; b0 < s.batch; b0 += 32) {
    const int b = b0 + lane;
    Seq q{};
    int first = 0;
    if (b < s.batch) q = kv_seq(s, b, page, err);
    const int n = b < s.batch ? touched(q, first) : 0;
    int at = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, at, d);
      if (lane >= d) at += o;
    }
    const unsigned past = __ballot_sync(0xFFFFFFFFu, x < at);
    if (past) {
      const int src = __ffs(past) - 1;
      f.b = b0 + src;
      f.block = __shfl_sync(0xFFFFFFFFu, first + x - (at - n), src);
      f.q.first = __shfl_sync(0xFFFFFFFFu, q.first, src);
      f.q.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
      f.q.len = __shfl_sync(0xFFFFFFFFu, q.len, src);
      return f;
    }
    x -= __shfl_sync(0xFFFFFFFFu, at, 31);
  }
  return f;
}

// A row of D values over D / 8 lanes, 8 each: 32 / (D / 8) rows a warp at a time.
template <int D>
struct Lanes {
  static constexpr int kPerRow = D / 8, kRows = 32 / kPerRow, kSteps = kKvTokens / kRows;
};

// The rotation by position of this lane's eight values (elements 8 cc ..), angles of nf pairs.
template <int D>
__device__ __forceinline__ void rope(float (&v)[8], const float2* trig, int cc, int nf, int interleaved) {
  if (interleaved) {  // pairs (2i, 2i + 1)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * cc + i < nf) {
        const float2 t = trig[4 * cc + i];
        const float a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = a * t.x - b * t.y;
        v[2 * i + 1] = b * t.x + a * t.y;
      }
    return;
  }
  // pairs (i, i + nf), nf a multiple of 8: eight of them between two lanes of the row
  const int nl = nf >> 3, lane = threadIdx.x & 31;
  const bool lo = cc < nl, in = cc < 2 * nl;
  const int src = lane + (!in ? 0 : lo ? nl : -nl);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = __shfl_sync(0xFFFFFFFFu, v[i], src);
    if (in) {
      const float2 t = trig[8 * (lo ? cc : cc - nl) + i];
      v[i] = lo ? v[i] * t.x - o * t.y : v[i] * t.x + o * t.y;
    }
  }
}

// grid (touched blocks at most, shares of the heads): a warp takes (head, K or V), then heads of q.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const KvCache c, const KvSeqs s, const KvNew a, int* err) {
  using L = Lanes<D>;
  __shared__ float2 trig[kKvTokens][D / 2];
  __shared__ int at[6];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 0) {
    const Found f = find_block(s, c.page, static_cast<int>(blockIdx.x), err);
    if (lane == 0) {
      at[0] = f.b;
      if (f.b >= 0) {
        const int p0 = f.block * kKvTokens, start = f.q.len - f.q.n;  // start < 0: its first tokens have no place
        if (start < 0) kv_flag(err);
        at[1] = max(max(start, 0) - p0, 0);             // the block's new rows: first, end
        at[2] = min(f.q.len - p0, kKvTokens);
        at[3] = p0;
        at[4] = f.q.first + p0 - start;                 // token of the block's row 0
        at[5] = kv_page(s, c, f.b, p0, err);
      }
    }
  }
  __syncthreads();
  if (at[0] < 0) return;
  const int lo = at[1], hi = at[2], p0 = at[3], tok0 = at[4], page = at[5];
  if (a.nf > 0) {
    for (int i = threadIdx.x; i < (hi - lo) * a.nf; i += kThreads) {
      const int r = lo + i / a.nf, j = i % a.nf;
      const double turn = static_cast<double>(p0 + r) * (a.freqs[j] * 0.15915494309189533577);  // 1 / (2 pi)
      const float x = static_cast<float>(turn - rint(turn));
      float2 t;
      sincospif(2.0f * x, &t.y, &t.x);
      trig[r][j] = t;
    }
    __syncthreads();
  }
  const int rr = lane / L::kPerRow, cc = lane % L::kPerRow;
  const int kv_tasks = page >= 0 ? 2 * c.heads : 0, tasks = kv_tasks + a.q_heads;
  for (int task = blockIdx.y * kWarps + warp; task < tasks; task += gridDim.y * kWarps) {
    const bool is_q = task >= kv_tasks;
    const int h = is_q ? task - kv_tasks : task >> 1, is_v = is_q ? 0 : task & 1;
    const T* x = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) + h * (is_q ? a.ldqh : is_v ? a.ldvh : a.ldkh) + 8 * cc;
    const int64_t ld = is_q ? a.ldq : is_v ? a.ldv : a.ldk;
    Chunk<T> raw[L::kSteps];
#pragma unroll
    for (int i = 0; i < L::kSteps; ++i) {
      const int r = i * L::kRows + rr;
      if (r >= lo && r < hi) raw[i].load(x + (tok0 + r) * ld, false);
      else raw[i] = Chunk<T>{};
    }
    if (is_q) {
#pragma unroll
      for (int i = 0; i < L::kSteps; ++i) {
        const int r = i * L::kRows + rr;
        if (i * L::kRows >= hi || (i + 1) * L::kRows <= lo) continue;
        float v[8];
        raw[i].get(v);
        if (a.nf > 0) rope<D>(v, trig[r], cc, a.nf, a.interleaved);
        if (r >= lo && r < hi) {
          const int64_t o = (tok0 + r) * a.ldo + h * a.ldoh + 8 * cc;
          if (a.o_bf16) store8(static_cast<__nv_bfloat16*>(a.q_out) + o, v, false);
          else store8(static_cast<float*>(a.q_out) + o, v, false);
        }
      }
      continue;
    }
    float v[L::kSteps][8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < L::kSteps; ++i) {
      raw[i].get(v[i]);
      if (i * L::kRows >= hi || (i + 1) * L::kRows <= lo) continue;  // no new row: zeros
      if (!is_v && a.nf > 0) {
        const int r = i * L::kRows + rr;
        rope<D>(v[i], trig[r], cc, a.nf, a.interleaved);
        if (r < lo || r >= hi)  // it has no angles, and whatever stands in their place may be a NaN
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      }
      if (c.rotated) quad_rotate(v[i], lane & 3);
      amax = max3_abs(amax, lane_amax(v[i]), 0.0f);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) amax = max3_abs(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d), 0.0f);
    bool bad = !(amax <= 3.402823466e38f);
    // 127 = 1.984375 * 2^6
    const uint32_t bits = __float_as_uint(amax);
    int E = static_cast<int>(bits >> 23) - 127 - 6 + ((bits & 0x7FFFFFu) > 0x7E0000u);
    E = min(max(E, kKvLow), kKvHigh);
    uint8_t* const scale = c.scales + kv_scale_at(c, page, h, is_v) + p0 % c.page / kKvTokens;
    int8_t* const codes = c.codes + kv_at(c, page, h, is_v) + static_cast<int64_t>(p0 % c.page) * D + 8 * cc;
    if (lo > 0) {
      const int was = *scale;
      bad = bad || was == 255;
      const int old = min(max(was - 127, kKvLow), kKvHigh);
      if (!bad && E > old) {  // the rows before: their codes, at the larger scale
        const float f = pow2i(old - E);
        for (int r = rr; r < lo; r += L::kRows) {
          uint2* const p = reinterpret_cast<uint2*>(codes + r * D);
          const uint2 w = *p;
          uint32_t o[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int q = static_cast<int8_t>((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
            o[i >> 2] |= (static_cast<uint32_t>(__float2int_rn(static_cast<float>(q) * f)) & 0xFFu) << (8 * (i & 3));
          }
          *p = make_uint2(o[0], o[1]);
        }
      }
      E = max(E, old);
    }
    const float inv = bad ? 0.0f : pow2i(-E);
#pragma unroll
    for (int i = 0; i < L::kSteps; ++i) {
      const int r = i * L::kRows + rr;
      if (r < lo || r >= hi) continue;
      uint32_t o[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = bad ? 0 : min(max(__float2int_rn(v[i][j] * inv), -127), 127);
        o[j >> 2] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (j & 3));
      }
      *reinterpret_cast<uint2*>(codes + r * D) = make_uint2(o[0], o[1]);
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = static_cast<uint8_t>(bad ? 255 : E + 127);
  }
}

// A warp per token: K, then V of its heads.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(const KvCache c, const KvSeqs s, T* k, T* v, int64_t ldk,
                                                            int64_t ldkh, int64_t ldv, int64_t ldvh, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t wide = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (wide >= s.tokens) return;
  const int t = static_cast<int>(wide);
  int b;
  if (s.cu) {  // the last sequence that starts at t or before
    int lo = 0, hi = s.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
  } else {
    b = t / s.each;
  }
  const Seq q = kv_seq(s, b, c.page, err);
  if (t < q.first || t >= q.first + q.n) return;  // behind the last sequence
  const int pos = q.len - q.n + (t - q.first);
  int page = -1;
  if (pos >= 0) page = kv_page(s, c, b, pos, err);
  else kv_flag(err);
  const int per = c.dim >> 3, row = pos >= 0 ? pos % c.page : 0, blk = row / kKvTokens;
  const int n = 2 * c.heads * per;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) {
    const int hv = i / per, cc = i % per, h = hv >> 1;
    float o[8] = {};
    if (page >= 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(c.codes + kv_at(c, page, h, hv & 1) + static_cast<int64_t>(row) * c.dim + 8 * cc);
      const float f = kv_scale(c.scales[kv_scale_at(c, page, h, hv & 1) + blk]);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? w.x : w.y) >> (8 * (j & 3)))) * f;
    }
    if (hv & 1) store8(v + t * ldv + h * ldvh + 8 * cc, o, false);
    else store8(k + t * ldk + h * ldkh + 8 * cc, o, false);
  }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace

cudaError_t launch_kv8_append(const KvCache& c, const KvSeqs& s, const KvNew& a, cudaStream_t st) {
  // touched blocks: of n tokens, (n + 14) / 16 + 1 at most
  const int64_t few = s.batch < s.tokens ? s.batch : s.tokens;
  const int64_t blocks = s.cu ? s.tokens / kKvTokens + 2 * few : static_cast<int64_t>(s.batch) * ((s.each + kKvTokens - 2) / kKvTokens + 1);
  const int64_t shares = (2 * c.heads + a.q_heads + kWarps - 1) / kWarps;
  // heads over several CTAs while there are fewer than four CTAs an SM
  int64_t y = (4 * static_cast<int64_t>(num_sms()) + blocks - 1) / blocks;
  y = y < shares ? y : shares;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(y));
  int* err = device_error_word();
  switch (c.dim * 2 + a.x_bf16) {
    case 128: return launch(kv8_append_kernel<64, float>, grid, st, c, s, a, err);
    case 129: return launch(kv8_append_kernel<64, __nv_bfloat16>, grid, st, c, s, a, err);
    case 256: return launch(kv8_append_kernel<128, float>, grid, st, c, s, a, err);
    case 257: return launch(kv8_append_kernel<128, __nv_bfloat16>, grid, st, c, s, a, err);
    case 512: return launch(kv8_append_kernel<256, float>, grid, st, c, s, a, err);
    default: return launch(kv8_append_kernel<256, __nv_bfloat16>, grid, st, c, s, a, err);
  }
}

cudaError_t launch_kv8_read(const KvCache& c, const KvSeqs& s, void* k, void* v, int bf16, int64_t ldk, int64_t ldkh,
                            int64_t ldv, int64_t ldvh, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((s.tokens + kWarps - 1) / kWarps));
  int* err = device_error_word();
  if (bf16)
    return launch(kv8_read_kernel<__nv_bfloat16>, grid, st, c, s, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v),
                  ldk, ldkh, ldv, ldvh, err);
  return launch(kv8_read_kernel<float>, grid, st, c, s, static_cast<float*>(k), static_cast<float*>(v), ldk, ldkh, ldv, ldvh, err);
}

}  // namespace w4a4
