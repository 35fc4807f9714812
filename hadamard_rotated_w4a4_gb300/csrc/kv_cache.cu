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
// the maximum and the rounding, so everything is read once.  Angles are whole
// numbers of 2^-64 turns, reduced by themselves, for 16 tokens once per CTA, and the CTA's heads
// share them.
//
// Bound: waves of CTAs and the latency of their loads for long prompts, latency else.  8192 tokens of
// 40 + 16 heads of 128 in bf16: 47.6 us, 4.6 TB/s of q, k, v and codes (0.68 of a plain copy's; first
// form 98 us; 55 with angles reduced in fp64).  Its 513 CTAs have 304 places, two an SM: 303 CTAs
// take 27.8 us (4.65 TB/s), 455 take 45.9, 607 take 51.3 (5.0 TB/s); issue is active 39% of the time.
// 64 sequences' next token, 20 + 8 heads of 256 in fp32, 5.4 us; one token 3.6 us.  Reading 8192 tokens back
// to bf16, codes from L2: 13.0 us, 3.9 TB/s, latency: loads of 8 bytes behind the look-up of a page and a
// scale, in 1.1 waves of CTAs.
//
// Sine and cosine are fp32's, 1.3 units of 2^-24 off at most (0.31 root mean square; 0.26 of 64 bits rounded).
// 64 bits for 8192 tokens would cost more than that gives: of 8.4 million codes of k 11 and 10 differ from
// those of 64 bits (two inputs), 11 and 9 with cosines of 64 bits.
#include <cuda_bf16.h>

#include "kv_cache.cuh"
#include "quad_block.cuh"

namespace w4a4 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Blocks of 16 tokens that the last n of len tokens touch, and the first of them.  More new tokens than there are: the
// first of them have no place.
__device__ __forceinline__ int touched(const Seq& q, int& first, int* err) {
  if (q.n > q.len) kv_flag(err);
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
    const int n = touched(f.q, first, err);
    if (x % most < n) f.b = b, f.block = first + x % most;
    return f;
  }
  for (int b0 = 0; b0 < s.batch; b0 += 32) {
    const int b = b0 + lane;
    Seq q{};
    int first = 0;
    if (b < s.batch) q = kv_seq(s, b, page, err);
    const int n = b < s.batch ? touched(q, first, err) : 0;
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

// A row of D values over D / 16 lanes, lane k of them with the chunks of 8 elements k and k + D / 16: the pairs
// (i, i + D / 2) of a full rotary rotation lie in one lane, and the 32-blocks in four neighbours either way.
template <int D>
struct Lanes {
  static constexpr int kPerRow = D / 16, kRows = 32 / kPerRow, kSteps = kKvTokens / kRows;
};

// How the pairs lie: none, (2i, 2i + 1), (i, i + D / 2), (i, i + nf).
enum Pairs : int { kNoPairs, kNeighbours, kHalves, kApart };

__device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}

// The rotation by position of a lane's two chunks of a row, cs and sn the cosines and sines of the row's angles.
template <int D>
__device__ __forceinline__ void rope(float (&v)[2][8], const float* cs, const float* sn, int k, int nf, Pairs pairs) {
  constexpr int kPerRow = Lanes<D>::kPerRow;
  if (pairs == kHalves) {
    float c[8], s[8];
    load8(cs + 8 * k, c);
    load8(sn + 8 * k, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[0][i], b = v[1][i];
      v[0][i] = a * c[i] - b * s[i];
      v[1][i] = b * c[i] + a * s[i];
    }
  } else if (pairs == kNeighbours) {  // what lies past the pairs as it is: an infinity times a sine of zero would be a NaN
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c4 = *reinterpret_cast<const float4*>(cs + 4 * (k + h * kPerRow)), s4 = *reinterpret_cast<const float4*>(sn + 4 * (k + h * kPerRow));
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
      const int here = nf - 4 * (k + h * kPerRow);  // pairs of the chunk
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[h][2 * i], b = v[h][2 * i + 1];
        const float x = a * c[i] - b * s[i], y = b * c[i] + a * s[i];
        if (i < here) v[h][2 * i] = x, v[h][2 * i + 1] = y;
      }
    }
  } else {  // nf a multiple of 8: eight pairs between two chunks, of whichever lanes
    const int nl = nf >> 3, base = (threadIdx.x & 31) - k;
    float old[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) old[0][i] = v[0][i], old[1][i] = v[1][i];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ch = k + h * kPerRow;
      const bool lo = ch < nl, in = ch < 2 * nl;
      const int other = !in ? ch : lo ? ch + nl : ch - nl;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = __shfl_sync(0xFFFFFFFFu, old[0][i], base + other % kPerRow), y = __shfl_sync(0xFFFFFFFFu, old[1][i], base + other % kPerRow);
        const float o = other < kPerRow ? x : y;
        if (in) {
          const float c = cs[8 * (lo ? ch : other) + i], s = sn[8 * (lo ? ch : other) + i];
          v[h][i] = lo ? old[h][i] * c - o * s : old[h][i] * c + o * s;
        }
      }
    }
  }
}

// grid (touched blocks at most, shares of the heads): a warp takes (head, K or V), then heads of q.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const KvCache c, const KvSeqs s, const KvNew a, int* err) {
  using L = Lanes<D>;
  __shared__ __align__(16) float cs[kKvTokens][D / 2], sn[kKvTokens][D / 2];
  __shared__ int at[6];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 0) {
    const Found f = find_block(s, c.page, static_cast<int>(blockIdx.x), err);
    if (lane == 0) {
      at[0] = f.b;
      if (f.b >= 0) {
        const int p0 = f.block * kKvTokens, start = f.q.len - f.q.n;  // start < 0: its first tokens are skipped
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
  const Pairs pairs = a.nf == 0 ? kNoPairs : a.interleaved ? kNeighbours : 2 * a.nf == D ? kHalves : kApart;
  if (pairs != kNoPairs) {
    // angle j of every row by the same threads, so that its share of a turn is taken once
    for (int j = threadIdx.x % (D / 2); j < a.nf; j += D / 2) {
      // a position's share of a turn in units of 2^-64, so that a position times it is exact but for whole turns
      const double turns = a.freqs[j] * 0.15915494309189533577;  // 1 / (2 pi)
      const uint64_t share = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
      const float bad = static_cast<float>(turns - turns);  // 0, or NaN
      for (int r = lo + threadIdx.x / (D / 2); r < hi; r += kThreads / (D / 2)) {
        const int half = static_cast<int>((share * static_cast<uint32_t>(p0 + r)) >> 32);  // in units of 2^-31 pi
        const float x = __int2float_rn(half);
        const float rest = fmaf(__int2float_rn(half - __float2int_rn(x)), 3.14159265f * 0x1p-31f, bad);  // what its rounding left
        float sine, cosine;
        sincospif(x * 0x1p-31f, &sine, &cosine);
        cs[r][j] = fmaf(-sine, rest, cosine);
        sn[r][j] = fmaf(cosine, rest, sine);
      }
    }
    __syncthreads();
  }
  const int rr = lane / L::kPerRow, k = lane % L::kPerRow;
  const int kv_tasks = page >= 0 ? 2 * c.heads : 0, tasks = kv_tasks + a.q_heads;
  for (int task = blockIdx.y * kWarps + warp; task < tasks; task += gridDim.y * kWarps) {
    const bool is_q = task >= kv_tasks;
    const int h = is_q ? task - kv_tasks : task >> 1, is_v = is_q ? 0 : task & 1;
    const int64_t ld = is_q ? a.ldq : is_v ? a.ldv : a.ldk;
    const T* x = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) + h * (is_q ? a.ldqh : is_v ? a.ldvh : a.ldkh) + (tok0 + rr) * ld + 8 * k;
    Chunk<T> raw[L::kSteps][2];
#pragma unroll
    for (int i = 0; i < L::kSteps; ++i) {
      const int r = i * L::kRows + rr;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        raw[i][g] = Chunk<T>{};
        if (r >= lo && r < hi) raw[i][g].load(x + i * L::kRows * ld + g * (D / 2), false);
      }
    }
    const bool turn = pairs != kNoPairs && !is_v;
    if (is_q) {
      const int64_t o = (tok0 + rr) * a.ldo + h * a.ldoh + 8 * k;
#pragma unroll
      for (int i = 0; i < L::kSteps; ++i) {
        const int r = i * L::kRows + rr;
        if (i * L::kRows >= hi || (i + 1) * L::kRows <= lo) continue;
        float v[2][8];
        raw[i][0].get(v[0]);
        raw[i][1].get(v[1]);
        if (turn) rope<D>(v, cs[r], sn[r], k, a.nf, pairs);
        if (r >= lo && r < hi)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int64_t to = o + i * L::kRows * a.ldo + g * (D / 2);
            if (a.o_bf16) store8(static_cast<__nv_bfloat16*>(a.q_out) + to, v[g], false);
            else store8(static_cast<float*>(a.q_out) + to, v[g], false);
          }
      }
      continue;
    }
    float v[L::kSteps][2][8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < L::kSteps; ++i) {
      raw[i][0].get(v[i][0]);
      raw[i][1].get(v[i][1]);
      if (i * L::kRows >= hi || (i + 1) * L::kRows <= lo) continue;  // no new row: zeros
      const int r = i * L::kRows + rr;
      if (turn) {
        rope<D>(v[i], cs[r], sn[r], k, a.nf, pairs);
        if (r < lo || r >= hi)  // it has no angles, and whatever stands in their place may be a NaN
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][0][j] = v[i][1][j] = 0.0f;
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (c.rotated) quad_rotate(v[i][g], lane & 3);
        amax = max3_abs(amax, lane_amax(v[i][g]), 0.0f);
      }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) amax = max3_abs(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d), 0.0f);
    bool bad = !(amax <= 3.402823466e38f);
    // 127 = 1.984375 * 2^6
    const uint32_t bits = __float_as_uint(amax);
    int E = static_cast<int>(bits >> 23) - 127 - 6 + ((bits & 0x7FFFFFu) > 0x7E0000u);
    E = max(E, kKvLow);
    const bool clip = E > kKvHigh;  // past the largest scale: the codes saturate
    E = min(E, kKvHigh);
    const int in_page = p0 & (c.page - 1);
    uint8_t* const scale = c.scales + kv_scale_at(c, page, h, is_v) + in_page / kKvTokens;
    int8_t* const codes = c.codes + kv_at(c, page, h, is_v) + static_cast<int64_t>(in_page) * D + 8 * k;
    if (lo > 0) {
      const int was = *scale;
      bad = bad || was == 255;
      const int old = min(max(was - 127, kKvLow), kKvHigh);
      if (!bad && E > old) {  // the rows before: their codes, at the larger scale
        const float f = pow2i(old - E);
        for (int r = rr; r < lo; r += L::kRows)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint2* const p = reinterpret_cast<uint2*>(codes + r * D + g * (D / 2));
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
    if (bad || clip)
#pragma unroll
      for (int i = 0; i < L::kSteps; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int g = 0; g < 2; ++g) v[i][g][j] = bad ? 0.0f : fminf(fmaxf(v[i][g][j], -127.0f * pow2i(kKvHigh)), 127.0f * pow2i(kKvHigh));
    // |v| / 2^E is at most 127: plus 1.5 * 2^23 it is that and the nearest integer (ties to even), whose low byte is
    // the code in two's complement
    constexpr float kMagic = 12582912.0f;
#pragma unroll
    for (int i = 0; i < L::kSteps; ++i) {
      const int r = i * L::kRows + rr;
      if (r < lo || r >= hi) continue;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t t[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 y = __ffma2_rn(make_float2(v[i][g][j], v[i][g][j + 1]), make_float2(inv, inv), make_float2(kMagic, kMagic));
          t[j] = __float_as_uint(y.x);
          t[j + 1] = __float_as_uint(y.y);
        }
        *reinterpret_cast<uint2*>(codes + r * D + g * (D / 2)) =
            make_uint2(prmt(prmt(t[0], t[1], 0x0040u), prmt(t[2], t[3], 0x0040u), 0x5410u),
                       prmt(prmt(t[4], t[5], 0x0040u), prmt(t[6], t[7], 0x0040u), 0x5410u));
      }
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
  // heads over several CTAs, each with the angles for itself, up to about a CTA an SM (64 blocks of 28 heads in fp32:
  // 64 CTAs 7.0 us, 128 5.4, 256 6.4; 513 blocks of 56 heads: 513 CTAs 47.8 us, 1026 49.4)
  int64_t y = (num_sms() + blocks / 2) / blocks;
  y = y < 1 ? 1 : y < shares ? y : shares;
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
