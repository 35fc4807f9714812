// Attention of few query rows over the 8-bit paged cache: single tokens and verification
// batches, the stream of the cache's codes.
//
// A tile is a sequence's head of K and V with up to 16 query rows (tokens x the heads that
// share it).  Its keys are cut in units of 64 and the units of all tiles dealt evenly to two
// CTAs per SM, so that sequences of any lengths fill the GPU; a tile cut between CTAs is
// joined by the last of them to arrive, its parts added in the order of their CTAs: equal
// inputs give equal bits.
//
// In a CTA each warp takes blocks of 16 keys by itself, with its own running maximum and sum
// and its own ring of copies (cp.async): no barrier until the tile's end.  No transposition
// either, because the order of a contraction is free: for Q K^T, lane (r, c) = (lane / 4,
// lane % 4) takes 16 consecutive elements 64 j + 16 c of key r, and Q is read in the same
// order; for P V, it takes elements 16 r .. of the four keys whose weights its accumulators
// hold.  Eight neighbouring lanes copy 128 bytes on end (copies of what each lane itself reads
// moved every sector twice: 131072 keys, 4 sequences 245 us), and the pieces of a row trade
// places by its number so that the reads meet no bank twice.
//
// Bound: the codes' stream, 2 D + 1/8 bytes a key and head.  8 heads of 128: 131072 keys of 4
// sequences 189-193 us, 5.6 TB/s (0.83 of a plain copy's); 64 sequences of 515 to 8192 keys 90 us,
// 4.5 TB/s, the rest what a tile costs beside its keys; one token over 1000 keys 9.8 us, one
// latency behind another (lengths, pages, codes, the join).
#include <cuda_bf16.h>

#include "kv_attention.cuh"

namespace w4a4 {

namespace {

constexpr int kRows = 16;          // query rows of a tile
constexpr size_t kWsCounters = size_t(1) << 20;  // as in the other workspaces: zero between calls

template <int D>
struct Shape {
  // Two CTAs of four warps an SM (registers hold no more: the accumulators alone are D / 2 a lane): one's lookups,
  // joins and stores run beside the other's stream.
  static constexpr int kWarps = 4, kThreads = 32 * kWarps;
  static constexpr int kUnit = kWarps;   // blocks of 16 keys in a unit
  // What a tile costs beside its keys (lookups, q, the join), in units: without it the CTAs that got many short
  // sequences finished last.
  static constexpr int kOnce = 8;
  static constexpr int kLeast = 2;  // units of a CTA at least, for fewer parts to join
  static constexpr int kStage = 32 * D;  // bytes of 16 keys and values
  static constexpr int kRing = D == 256 ? 3 : D == 128 ? 5 : 8;
  static constexpr int kRingBytes = kWarps * kRing * kStage;
  static constexpr int kMergeBytes = kWarps * kRows * D * 4;
  static constexpr int kQLd = 2 * D + 8;  // bytes of a row of q: two lanes' 8-byte reads share no bank
  static constexpr int kMain = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
  static constexpr int kQ = kMain, kPrefix = kQ + kRows * kQLd;
  static constexpr int smem(int batch) { return kPrefix + 8 * (batch + 1); }
  static constexpr int kPart = kRows * (D + 2);  // floats of a cut tile's part
};

struct DecodeArgs {
  KvCache c;
  KvSeqs s;
  KvAttn a;
  int group;       // query heads per head of K and V
  int most_rows;   // sequences with more query rows (tokens x group) are another kernel's
  uint32_t* tickets;  // [grid], zero between calls; null: tiles are not cut
  float* parts;       // [grid][2][kPart]
  int* err;
};

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Where 16-byte piece ch of a block's row lies: piece ch ^ place of that row.  A read of K by eight lanes takes four
// neighbouring pieces of two rows, one of V two pieces of every second row of eight.
template <int D>
__device__ __forceinline__ int k_place(int row) { return D == 64 ? 0 : (row & 1) << 2; }
template <int D>
__device__ __forceinline__ int v_place(int row) { return D == 64 ? (row >> 1) & 3 : row & 6; }
// Where the four floats from element d of a row lie in the warps' sums: by the lane that wrote them and the row, so that
// neither the writes (four lanes 128 bytes apart, of two rows) nor the reads meet a bank more than twice.
template <int D>
__device__ __forceinline__ int merge_place(int row, int d) {
  return ((d >> 2) ^ ((D == 64 ? d >> 4 : d >> 5) & 3) ^ ((row & 1) << 2)) << 2;
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A sequence's tiles, and the units of each.
struct Plan {
  int tiles;        // row tiles x heads
  int units;        // of a tile: kOnce and those of its keys
  int step0, step1;  // blocks of 16 keys that some query of the sequence sees
};
template <int D>
__device__ __forceinline__ Plan plan_of(const DecodeArgs& p, const Seq& q) {
  constexpr int kUnit = Shape<D>::kUnit;
  Plan o{0, 1, 0, 0};
  const int64_t rows = static_cast<int64_t>(q.n) * p.group;
  if (q.n == 0 || rows > p.most_rows) return o;
  o.tiles = static_cast<int>((rows + kRows - 1) / kRows) * p.c.heads;
  int lo, hi;
  seen(p.a, q.len - q.n, q.len, lo, hi);
  o.step0 = min(lo, q.len) / kKvTokens;
  o.step1 = (q.len + kKvTokens - 1) / kKvTokens;
  if (p.tickets) o.units = Shape<D>::kOnce + max(1, (o.step1 - o.step0 + kUnit - 1) / kUnit);
  return o;
}

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, 2) kv8_decode_kernel(const DecodeArgs p) {
  using C = Shape<D>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads, kUnit = C::kUnit;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows], sm_f[kRows];
  __shared__ int sm_lo[kRows], sm_hi[kRows];
  __shared__ float2 sm_scale[kWarps][C::kRing];
  __shared__ int64_t sm_carry[kWarps];
  __shared__ int sm_last;
  int64_t* const prefix = reinterpret_cast<int64_t*>(smem + C::kPrefix);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  grid_dep_wait();
  grid_dep_launch();

  // units before each sequence: of up to 32 in the lanes of every warp, else in shared memory
  const bool small = p.s.batch <= 32;
  int64_t total = 0, mine = 0, before = 0;
  Seq seq{};
  if (small) {
    if (lane < p.s.batch) {
      seq = kv_seq(p.s, lane, p.c.page, p.err);
      const Plan o = plan_of<D>(p, seq);
      mine = static_cast<int64_t>(o.tiles) * o.units;
    }
    int64_t at = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xFFFFFFFFu, at, d);
      if (lane >= d) at += o;
    }
    before = at - mine;
    total = __shfl_sync(0xFFFFFFFFu, at, 31);
  } else {
    for (int b0 = 0; b0 < p.s.batch; b0 += kThreads) {
      const int b = b0 + tid;
      mine = 0;
      if (b < p.s.batch) {
        const Plan o = plan_of<D>(p, kv_seq(p.s, b, p.c.page, p.err));
        mine = static_cast<int64_t>(o.tiles) * o.units;
      }
      int64_t at = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, at, d);
        if (lane >= d) at += o;
      }
      if (lane == 31) sm_carry[warp] = at;
      __syncthreads();
      before = total;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm_carry[w];
        total += sm_carry[w];
      }
      if (b < p.s.batch) prefix[b] = before + at - mine;
      __syncthreads();
    }
  }
  const int64_t G = total == 0 ? 0 : max(int64_t(1), min(static_cast<int64_t>(gridDim.x), total / C::kLeast));  // CTAs at work
  if (static_cast<int64_t>(blockIdx.x) >= G) return;
  const auto range = [&](int64_t cta) { return total * cta / G; };
  const int64_t u_end = range(blockIdx.x + 1);

  for (int64_t u = range(blockIdx.x); u < u_end;) {
    // the tile of unit u
    int b;
    Seq q;
    int64_t in;
    if (small) {
      b = 31 - __clz(__ballot_sync(0xFFFFFFFFu, lane < p.s.batch && before <= u));
      q.first = __shfl_sync(0xFFFFFFFFu, seq.first, b);
      q.n = __shfl_sync(0xFFFFFFFFu, seq.n, b);
      q.len = __shfl_sync(0xFFFFFFFFu, seq.len, b);
      in = u - __shfl_sync(0xFFFFFFFFu, before, b);
    } else {
      b = 0;
      for (int hi = p.s.batch; hi - b > 1;) {
        const int mid = (b + hi) >> 1;
        if (prefix[mid] <= u) b = mid;
        else hi = mid;
      }
      q = kv_seq(p.s, b, p.c.page, nullptr);
      in = u - prefix[b];
    }
    const Plan plan = plan_of<D>(p, q);
    const int tile = static_cast<int>(in / plan.units), u0 = static_cast<int>(in % plan.units);
    const int64_t tile_u = u - u0;  // the tile's first unit
    const int u1 = static_cast<int>(min(static_cast<int64_t>(plan.units), u0 + (u_end - u)));
    const int once = p.tickets ? C::kOnce : 0;
    if (u1 <= once) break;  // no key of this tile, the CTA's last
    const int head = tile % p.c.heads, row0 = tile / p.c.heads * kRows;
    const int rows = min(kRows, q.n * p.group - row0);
    int first, last, ignore;  // keys of the tile's first and last query
    seen(p.a, q.len - q.n + row0 / p.group, q.len, first, ignore);
    seen(p.a, q.len - q.n + (row0 + rows - 1) / p.group, q.len, ignore, last);
    int s0 = max(plan.step0, min(first, q.len) / kKvTokens), s1 = min(plan.step1, (max(last, 0) + kKvTokens - 1) / kKvTokens);
    if (p.tickets) {
      s0 = max(s0, plan.step0 + max(u0 - once, 0) * kUnit);
      s1 = min(s1, plan.step0 + (u1 - once) * kUnit);
    }

    const int steps = s1 - s0 > warp ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * C::kRing * C::kStage;
    const uint8_t* const ring_p = smem + warp * C::kRing * C::kStage;
    // q's loads go out first: 8 elements a pass
    constexpr int kPasses = kRows * D / 8 / kThreads;
    Chunk<float> q_raw[kPasses];
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int ch = pass * kThreads + tid, row = ch / (D / 8), g = row0 + row;
      if (row < rows) {
        const int64_t at = static_cast<int64_t>(q.first + g / p.group) * p.a.ldq + (head * p.group + g % p.group) * p.a.ldqh + 8 * (ch % (D / 8));
        if (p.a.q_bf16) reinterpret_cast<Chunk<__nv_bfloat16>&>(q_raw[pass]).load(static_cast<const __nv_bfloat16*>(p.a.q) + at, false);
        else q_raw[pass].load(static_cast<const float*>(p.a.q) + at, false);
      }
    }
    // lane i looks up the page and the scales of this warp's i-th block of 32
    int64_t look_at = -1;  // its first K code
    int look_s = 0;        // scale bytes of K and V
    const auto look = [&](int i0) {
      const int i = i0 + lane;
      look_at = -1;
      look_s = 0x7F7F;
      if (i < steps) {
        const int t = (s0 + warp + kWarps * i) * kKvTokens;
        const int page = kv_page(p.s, p.c, b, t, p.err);
        if (page >= 0) {
          const int in_page = t % p.c.page;
          const int64_t sc = kv_scale_at(p.c, page, head, 0) + in_page / kKvTokens;
          look_at = kv_at(p.c, page, head, 0) + static_cast<int64_t>(in_page) * D;
          look_s = p.c.scales[sc] | p.c.scales[sc + p.c.page / kKvTokens] << 8;
        }
      }
    };
    const auto issue = [&](int i) {
      if (i < steps) {
        if ((i & 31) == 0) look(i);
        const int64_t at = __shfl_sync(0xFFFFFFFFu, look_at, i & 31);
        const int st = i % C::kRing;
        const bool there = at >= 0;  // nothing is read where there is no page
        const int8_t* const k = p.c.codes + (there ? at : 0) + 16 * lane;
        const int8_t* const v = k + static_cast<int64_t>(p.c.page) * D;
        const uint32_t dst = ring + st * C::kStage;
#pragma unroll
        for (int m = 0; m < D / 32; ++m) {
          const int piece = 32 * m + lane, row = piece / (D / 16), ch = piece % (D / 16);
          cp_async16(dst + row * D + ((ch ^ k_place<D>(row)) << 4), k + 512 * m, there);
          cp_async16(dst + 16 * D + row * D + ((ch ^ v_place<D>(row)) << 4), v + 512 * m, there);
        }
        const int sc = __shfl_sync(0xFFFFFFFFu, look_s, i & 31);
        if (lane == 0)  // a block without a page: codes of zero, whose weights are taken out below
          sm_scale[warp][st] = make_float2(there ? kv_scale(sc & 255) : 0.0f, kv_exponent(sc >> 8));
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kRing - 1; ++i) issue(i);
    // q: rotated as the keys are, scaled by a power of two per row
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int ch = pass * kThreads + tid, row = ch / (D / 8), cc = ch % (D / 8);
      float v[8] = {};
      if (row < rows) {
        if (p.a.q_bf16) {
          reinterpret_cast<const Chunk<__nv_bfloat16>&>(q_raw[pass]).get(v);
        } else {
          q_raw[pass].get(v);
        }
      }
      if (p.c.rotated) quad_rotate(v, lane & 3);
      float amax = lane_amax(v);
#pragma unroll
      for (int d = 1; d < D / 8; d <<= 1) amax = max3_abs(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d), 0.0f);
      const int e = row_exponent(amax);
      const float f = pow2i(-e);
      uint32_t* const o = reinterpret_cast<uint32_t*>(smem + C::kQ + row * C::kQLd + 16 * cc);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack_half(v[2 * i] * f, v[2 * i + 1] * f);
      if (cc == 0) {
        sm_f[row] = p.a.scale * 1.4426950408889634f * pow2i(e);
        int lo, hi;  // rows past the last: as the last, so that they ask for no mask
        seen(p.a, q.len - q.n + (row0 + min(row, rows - 1)) / p.group, q.len, lo, hi);
        sm_lo[row] = lo;
        sm_hi[row] = hi;
      }
    }
    __syncthreads();
    const float f0 = sm_f[r], f1 = sm_f[r + 8];
    const int lo0 = sm_lo[r], lo1 = sm_lo[r + 8], hi0 = sm_hi[r], hi1 = sm_hi[r + 8];
    // a block with all its keys in lo_all .. hi_all needs no mask
    int lo_all = max(lo0, lo1), hi_all = min(hi0, hi1);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      lo_all = max(lo_all, __shfl_xor_sync(0xFFFFFFFFu, lo_all, d));
      hi_all = min(hi_all, __shfl_xor_sync(0xFFFFFFFFu, hi_all, d));
    }
    constexpr bool kQRegs = D <= 128;  // q's fragments in registers, or read again for every block
    uint32_t qa[kQRegs ? D / 16 : 1][4];
    const uint8_t* const q_lo = smem + C::kQ + r * C::kQLd + 32 * c;
    const auto q_frag = [&](int k, uint32_t (&f)[4]) {  // k = 4 j + w: elements 64 j + 16 c + 4 w ..
      const uint2 x = *reinterpret_cast<const uint2*>(q_lo + 128 * (k >> 2) + 8 * (k & 3));
      const uint2 y = *reinterpret_cast<const uint2*>(q_lo + 8 * C::kQLd + 128 * (k >> 2) + 8 * (k & 3));
      f[0] = x.x; f[1] = y.x; f[2] = x.y; f[3] = y.y;
    };
    if constexpr (kQRegs)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) q_frag(k, qa[k]);

    float o[D / 8][4] = {};
    float m0 = kNegInf, m1 = kNegInf, l0 = 0.0f, l1 = 0.0f;
    for (int i = 0; i < steps; ++i) {
      issue(i + C::kRing - 1);
      cp_wait<C::kRing - 1>();
      __syncwarp();
      const int st = i % C::kRing;
      const float2 sc = sm_scale[warp][st];
      const uint8_t* const src = ring_p + st * C::kStage;
      float s[2][4] = {};
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const uint8_t* const at = src + r * D + (((4 * j + c) ^ k_place<D>(r)) << 4);
        const uint4 u = *reinterpret_cast<const uint4*>(at), v = *reinterpret_cast<const uint4*>(at + 8 * D);
        const uint32_t w[2][4] = {{u.x, u.y, u.z, u.w}, {v.x, v.y, v.z, v.w}};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t f[4];
          if constexpr (kQRegs) {
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) f[i2] = qa[4 * j + k][i2];
          } else {
            q_frag(4 * j + k, f);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t x = w[n][k] ^ 0x80808080u;
            mma16816(s[n], f[0], f[1], f[2], f[3], codes_half2(x, 0x4140u), codes_half2(x, 0x4342u));
          }
        }
      }
      const float g0 = f0 * sc.x, g1 = f1 * sc.x, ev = sc.y;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = fmaf(s[n][0], g0, ev);
        s[n][1] = fmaf(s[n][1], g0, ev);
        s[n][2] = fmaf(s[n][2], g1, ev);
        s[n][3] = fmaf(s[n][3], g1, ev);
      }
      const int key0 = (s0 + warp + kWarps * i) * kKvTokens;
      if (key0 < lo_all || key0 + kKvTokens > hi_all || sc.x == 0.0f) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + 8 * n + 2 * c + e;
            if (key < lo0 || key >= hi0 || sc.x == 0.0f) s[n][e] = kNegInf;
            if (key < lo1 || key >= hi1 || sc.x == 0.0f) s[n][2 + e] = kNegInf;
          }
      }
      float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      if (__any_sync(0xFFFFFFFFu, t0 > m0 + (kShift + kLag) || t1 > m1 + (kShift + kLag))) {
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, d));
          t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, d));
        }
        const float n0 = fmaxf(m0, t0 - kShift), n1 = fmaxf(m1, t1 - kShift);
        const float c0 = n0 == m0 ? 1.0f : ex2(m0 - n0), c1 = n1 == m1 ? 1.0f : ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= c0;
        l1 *= c1;
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
          o[t][0] *= c0;
          o[t][1] *= c0;
          o[t][2] *= c1;
          o[t][3] *= c1;
        }
      }
      const float z0 = m0 == kNegInf ? 0.0f : m0, z1 = m1 == kNegInf ? 0.0f : m1;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = ex2(s[n][0] - z0);
        s[n][1] = ex2(s[n][1] - z0);
        s[n][2] = ex2(s[n][2] - z1);
        s[n][3] = ex2(s[n][3] - z1);
      }
      const float w0 = (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]), w1 = (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
      const float back = ex2(-ev);  // a NaN scale in a row that sees none of the block counts for nothing
      l0 += w0 == 0.0f ? 0.0f : w0 * back;
      l1 += w1 == 0.0f ? 0.0f : w1 * back;
      const uint32_t a0 = pack_half(s[0][0], s[0][1]), a1 = pack_half(s[0][2], s[0][3]);
      const uint32_t a2 = pack_half(s[1][0], s[1][1]), a3 = pack_half(s[1][2], s[1][3]);
      constexpr int kWords = D == 64 ? 2 : 4;
#pragma unroll
      for (int h = 0; h < (D == 64 ? 1 : D / 128); ++h) {
        uint32_t w[4][kWords];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int key = (kk >> 1) * 8 + 2 * c + (kk & 1);
          const uint8_t* const at = src + 16 * D + key * D;
          if constexpr (D == 64) {
            const uint2 x = *reinterpret_cast<const uint2*>(at + (((r >> 1) ^ v_place<D>(key)) << 4) + 8 * (r & 1));
            w[kk][0] = x.x ^ 0x80808080u;
            w[kk][1] = x.y ^ 0x80808080u;
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(at + (((8 * h + r) ^ v_place<D>(key)) << 4));
            w[kk][0] = x.x ^ 0x80808080u;
            w[kk][1] = x.y ^ 0x80808080u;
            w[kk][2 % kWords] = x.z ^ 0x80808080u;
            w[kk][3 % kWords] = x.w ^ 0x80808080u;
          }
        }
#pragma unroll
        for (int q4 = 0; q4 < kWords; ++q4)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const uint32_t sel = e == 0 ? 0x5140u : 0x7362u;  // bytes e, e + 1 of the two keys
            const uint32_t x = prmt(w[0][q4], w[1][q4], sel), y = prmt(w[2][q4], w[3][q4], sel);
            const int t = 16 * h + 4 * q4 + e;
            mma16816(o[t], a0, a1, a2, a3, codes_half2(x, 0x4140u), codes_half2(y, 0x4140u));
            mma16816(o[t + 1], a0, a1, a2, a3, codes_half2(x, 0x4342u), codes_half2(y, 0x4342u));
          }
      }
    }
    cp_wait<0>();

    // the warps' sums together: a common maximum, then the sum over the warps in their order
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, d);
      l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, d);
    }
    if (c == 0) {
      sm_m[warp][r] = m0;
      sm_m[warp][r + 8] = m1;
      sm_l[warp][r] = l0;
      sm_l[warp][r + 8] = l1;
    }
    __syncthreads();  // every warp's copies and reads of its ring are done as well
    float top0 = kNegInf, top1 = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      top0 = fmaxf(top0, sm_m[w][r]);
      top1 = fmaxf(top1, sm_m[w][r + 8]);
    }
    const float c0 = m0 == kNegInf ? (l0 == l0 ? 0.0f : 1.0f) : ex2(m0 - top0), c1 = m1 == kNegInf ? (l1 == l1 ? 0.0f : 1.0f) : ex2(m1 - top1);
    float* const merge = reinterpret_cast<float*>(smem) + warp * kRows * D;
#pragma unroll
    for (int t = 0; t < D / 8; t += 4)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = D == 64 ? 8 * (2 * c + e) + t : 128 * (t >> 4) + 16 * (2 * c + e) + (t & 15);
        *reinterpret_cast<float4*>(merge + r * D + merge_place<D>(r, d)) = make_float4(o[t][e] * c0, o[t + 1][e] * c0, o[t + 2][e] * c0, o[t + 3][e] * c0);
        *reinterpret_cast<float4*>(merge + (r + 8) * D + merge_place<D>(r, d)) =
            make_float4(o[t][2 + e] * c1, o[t + 1][2 + e] * c1, o[t + 2][2 + e] * c1, o[t + 3][2 + e] * c1);
      }
    __syncthreads();
    const bool whole = u0 <= once && u1 == plan.units;
    const int64_t c_first = whole ? 0 : ((tile_u + once + 1) * G - 1) / total;  // the CTA of the tile's first keys
    const int parts = whole ? 1 : static_cast<int>(((tile_u + plan.units) * G - 1) / total - c_first) + 1;
    float* const mine = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (range(blockIdx.x) < tile_u)) * C::kPart;
    const auto write = [&](int row, int cc, float (&v)[8], float l) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = l == 0.0f ? 0.0f : v[i] / l;
      if (p.c.rotated) quad_rotate(v, lane & 3);
      if (row < rows) {
        const int g = row0 + row;
        const int64_t at = static_cast<int64_t>(q.first + g / p.group) * p.a.ldo + (head * p.group + g % p.group) * p.a.ldoh + 8 * cc;
        if (p.a.o_bf16) store8(static_cast<__nv_bfloat16*>(p.a.out) + at, v, false);
        else store8(static_cast<float*>(p.a.out) + at, v, false);
      }
    };
    constexpr int kTogether = D < 256 ? 256 / D : 1;  // rows of a warp's pass over 8-element pieces
    const int pieces = (rows + kTogether - 1) / kTogether * kTogether * (D / 8);
    for (int ch = tid; ch < pieces; ch += kThreads) {
      const int row = ch / (D / 8), cc = ch % (D / 8);
      float top = kNegInf, l = 0.0f, v[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w][row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float m = sm_m[w][row], x = sm_l[w][row];
        l += m == kNegInf ? (x == x ? 0.0f : x) : x * ex2(m - top);
        const float* const s = reinterpret_cast<const float*>(smem) + (w * kRows + row) * D;
        const float4 y = *reinterpret_cast<const float4*>(s + merge_place<D>(row, 8 * cc));
        const float4 z = *reinterpret_cast<const float4*>(s + merge_place<D>(row, 8 * cc + 4));
        v[0] += y.x; v[1] += y.y; v[2] += y.z; v[3] += y.w;
        v[4] += z.x; v[5] += z.y; v[6] += z.z; v[7] += z.w;
      }
      if (whole) {
        write(row, cc, v, l);
      } else {
        float* const d = mine + row * D + 8 * cc;
        __stcg(reinterpret_cast<float4*>(d), make_float4(v[0], v[1], v[2], v[3]));
        __stcg(reinterpret_cast<float4*>(d) + 1, make_float4(v[4], v[5], v[6], v[7]));
        if (cc == 0) {
          __stcg(mine + kRows * D + row, top);
          __stcg(mine + kRows * (D + 1) + row, l);
        }
      }
    }
    if (!whole) {
      __syncthreads();
      if (tid == 0) {
        uint32_t* const ticket = p.tickets + c_first;  // a CTA is the first of one cut tile at most
        __threadfence();  // the CTA's parts, which the barrier has put before this
        const uint32_t got = atomicAdd(ticket, 1u);
        sm_last = got == static_cast<uint32_t>(parts - 1);
        if (sm_last) *ticket = 0u;
        __threadfence();
      }
      __syncthreads();
      if (sm_last) {
        // part i is CTA c_first + i's; its first tile's unless the tile begins inside its range
        const int64_t part0 = 2 * c_first + (range(c_first) < tile_u);
        const auto part = [&](int i) { return p.parts + (i == 0 ? part0 : 2 * (c_first + i)) * C::kPart; };
        for (int ch = tid; ch < pieces; ch += kThreads) {
          const int row = ch / (D / 8), cc = ch % (D / 8);
          float top = kNegInf, l = 0.0f, v[8] = {};
#pragma unroll 8
          for (int i = 0; i < parts; ++i) top = fmaxf(top, __ldcg(part(i) + kRows * D + row));
#pragma unroll 8
          for (int i = 0; i < parts; ++i) {
            const float* const s = part(i);
            const float m = __ldcg(s + kRows * D + row), x = __ldcg(s + kRows * (D + 1) + row);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(s + row * D + 8 * cc));
            const float4 z = __ldcg(reinterpret_cast<const float4*>(s + row * D + 8 * cc) + 1);
            const float f = m == kNegInf ? (x == x ? 0.0f : 1.0f) : ex2(m - top);
            l += x * f;
            v[0] += y.x * f; v[1] += y.y * f; v[2] += y.z * f; v[3] += y.w * f;
            v[4] += z.x * f; v[5] += z.y * f; v[6] += z.z * f; v[7] += z.w * f;
          }
          write(row, cc, v, l);
        }
      }
    }
    __syncthreads();  // shared memory is free for the next tile
    u += u1 - u0;
  }
}

template <int D>
cudaError_t launch_decode(const DecodeArgs& p, cudaStream_t st) {
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(kv8_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::smem(kKvMaxBatch));
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(Shape<D>::kThreads);
  cfg.dynamicSmemBytes = Shape<D>::smem(p.s.batch);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_decode_kernel<D>, p);
}

}  // namespace

size_t kv8_attention_workspace_bytes(int dim) {
  const size_t mine = kWsCounters + static_cast<size_t>(2 * num_sms()) * 2 * kRows * (dim + 2) * sizeof(float);
  const size_t other = kv8_prompt_workspace_bytes(dim);
  return mine > other ? mine : other;
}

// Few query rows (tokens x query heads per head of K and V) are this kernel's work, more the other's (kv_prompt.cu).  Up
// to 32, two tiles that read the keys twice: 24 rows over 4000 keys of 64 sequences, heads of 128, 111 us here and 149
// there (of 64: 76 and 138); 64 rows 208 and 146.  Heads of 256 have 16 rows at most here (24 rows over 6000 keys of 8
// sequences 71 and 56).  And all rows of a call whose tiles have few keys, by the tables' width, each as many as 512
// keys for itself: 64 tokens of a prompt, 32 heads of 128 over 4: 7.3 and 14.7 us; 512 tokens 28 and 28.
// A call with offsets may hold both kinds: each kernel takes its own.
cudaError_t launch_kv8_attention(const KvCache& c, const KvSeqs& s, const KvAttn& a, void* ws, cudaStream_t st) {
  DecodeArgs p{};
  p.c = c;
  p.s = s;
  p.a = a;
  p.group = a.q_heads / c.heads;
  const int64_t tiles = c.heads * (s.cu ? static_cast<int64_t>(s.tokens) * p.group / kRows + s.batch
                                        : s.batch * ((static_cast<int64_t>(s.each) * p.group + kRows - 1) / kRows));
  const bool small = c.dim <= 128 && tiles * (static_cast<int64_t>(s.width) * c.page + 512) <= (int64_t(1) << 18);
  const int most = small ? 0x7FFFFFFF : c.dim <= 128 ? 2 * kRows : kRows;
  p.most_rows = most;
  p.tickets = static_cast<uint32_t*>(ws);
  p.parts = ws ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsCounters) : nullptr;
  p.err = device_error_word();
  const bool few = s.cu ? p.group <= most : static_cast<int64_t>(s.each) * p.group <= most;
  const bool many = static_cast<int64_t>(s.cu ? s.tokens : s.each) * p.group > most;
  cudaError_t e = cudaSuccess;
  if (few) e = c.dim == 64 ? launch_decode<64>(p, st) : c.dim == 128 ? launch_decode<128>(p, st) : launch_decode<256>(p, st);
  if (e == cudaSuccess && many) e = launch_kv8_prompt(c, s, a, most + 1, ws, st);
  return e;
}

}  // namespace w4a4
