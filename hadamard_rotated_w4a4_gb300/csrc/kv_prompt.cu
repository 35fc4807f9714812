// Attention of many query rows over the 8-bit paged cache: prompts and pieces of them.
//
// A CTA takes up to 256 query rows (128 with heads of 256) of one head of K and V, rows being
// tokens x the heads that share it, and goes over the keys in tiles of 128 with the running
// maximum and sum of a softmax.  S = Q K^T and O += P V run on the tensor cores
// (tcgen05.mma kind::f16), accumulators in TMEM; P overwrites its S there and is the second
// product's A operand.  Bounds: the two products, 4 D operations a row and key; the exponential,
// one a row and key; and the way from codes to fp16.
//
// Warps: 0-3 and 4-7 the softmax of 128 rows each, a row a thread, so that no maximum crosses
// lanes; 8 issues the MMAs; 9 looks up pages and scales and copies blocks of 16 keys' codes and
// values' codes (cp.async.bulk) to their rings; 10-15 take these blocks in turn and write them as the
// products' B operands: keys are rows of 128 bytes in the 128-byte swizzle either way, K read along
// d (K-major), V along the keys (MN-major).  The two row tiles take turns: while one's weights are
// computed the other's products run.  With heads of 256 TMEM has room for one row tile with two S,
// and the next tile's S runs beside the softmax.
//
// The running maximum is looked for, and O rescaled, only where a weight might not fit fp16.
//
// Measured: 4096 tokens behind 12288, 40 heads of 128 over 8: 1277 us, 940 TFLOP/s (0.50 of a
// bf16 product's burst).  A key tile takes 3800 cycles, two row tiles of 1900.  By themselves their products
// would take 2080, and shared memory 2500 at 128 bytes a cycle (Q K^T reads 128 KB, P V 64, the conversion
// reads and writes 128).  Neither fills it: a row tile's softmax, P V and next Q K^T stand behind one another,
// with one S each.  Without the conversion's writes 1100 us, without the exponentials 1090, without both
// 1002.  Kept out: products of
// 64 keys with two S a row tile (1399 us: Q read twice as often), two threads a row (1277), codes
// by plain loads into registers (1484 at best).  8 drafted tokens of 8 sequences of up to 6000 keys,
// heads of 256: 36 us; prompts of 7 sequences, heads of 64, window 500: 33 us; both are set-up,
// one tile's chain and the join more than products.
#include <cuda_bf16.h>

#include "kv_attention.cuh"
#include "tc_ptx.cuh"

namespace w4a4 {

namespace {

constexpr int kThreads = 512;
constexpr int kBK = 128;                         // keys of a tile
constexpr int kBlocks = kBK / kKvTokens;         // blocks of 16 keys, each with its scales
constexpr int64_t kWaitCycles = int64_t(1) << 31;  // 1.04 s at the top clock, longer below it
constexpr size_t kWsCounters = size_t(1) << 20;
constexpr int kConvertWarps = 6;
constexpr float kMost = 32768.0f;  // of 16 weights together, below fp16's largest

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int D>
struct Shape {
  static constexpr int kTiles = D == 256 ? 1 : 2;   // row tiles of 128
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kBufs = D == 256 ? 1 : 2;    // converted tiles of K, and of V
  static constexpr int kTile = kBK * D * 2;         // bytes of one
  static constexpr int kPanel = 128 * 128;          // bytes of 64 elements of 128 rows
  static constexpr int kQ = 0, kK = kQ + kRows * D * 2, kV = kK + kBufs * kTile, kRaw = kV + kBufs * kTile;
  static constexpr int kBlock = kKvTokens * D;      // bytes of a block's codes
  static constexpr int kDepth = D == 256 ? 1 : 2, kSlots = kConvertWarps * kDepth;  // of them in a warp's ring, in all rings
  static constexpr int kPieces = D / 32;              // 16-code pieces of a lane in a block of 16 keys
  static constexpr int kPrefix = kK;  // find_work's sums, before the first tile of K
  static constexpr int kSmem = 1024 + kRaw + kSlots * kBlock;
  // registers a thread: warps 0-3, 4-7 (which heads of 256 leave idle), 8-11 and 12-15;
  // together no more than the launch's 4 x 128
  static constexpr int kRegs0 = 176, kRegs1 = D == 256 ? 24 : 176, kRegs2 = D == 256 ? 128 : 80;
  static_assert(kRegs0 + kRegs1 + 2 * kRegs2 <= 4 * 128);
  static constexpr int kS = 0, kO = 256;            // TMEM columns
  static constexpr int kPart = kRows * (D + 2);     // floats of a cut tile's part
  static_assert(kSmem <= 227 * 1024 - 2 * 1024 && kO + kTiles * D <= 512 && 4 * kKvMaxBatch <= kBufs * kTile);
};

struct PromptArgs {
  KvCache c;
  KvSeqs s;
  KvAttn a;
  int group;
  int least_rows;  // sequences with fewer query rows are another kernel's
  int sms;
  float* parts;    // [sms][kPart]: with few tiles, their keys cut over the SMs; null: not cut
  int* err;
  int64_t wait, delay;
};

struct Bars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], sc_full[4], sc_empty[4];
  uint64_t p_ready[2][2];  // [S][half of the keys]
  uint64_t pv_done[2][2];  // [row tile][half]
  uint64_t o_done[2];      // once, at the end
  uint64_t q_full;         // once
  uint64_t raw_full[12], raw_empty[12];  // [warp][its ring]
  int raw_none[12];        // no page: nothing was copied
  uint32_t tmem;
  volatile int abort;
};

// Bounded wait; on giving up, every other wait of the CTA gives up too.  The clock is read every 64 tries: the CTA's
// sixteen warps wait about half of the time, and what they do meanwhile takes issue slots from the others.
__device__ __forceinline__ bool wait_bar(Bars& S, uint64_t* b, uint32_t parity, const PromptArgs& p) {
  if (mbar_try(b, parity)) return true;
  const int64_t t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try(b, parity)) return true;
    if (S.abort) return false;
    if (clock64() - t0 > p.wait) {
      S.abort = 1;
      if (p.err) atomicOr(p.err, 64);
      return false;
    }
  }
}
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// Operand descriptors in the 128-byte swizzle (layout type 2): K-major, 8-row groups 1024 bytes
// apart; MN-major, groups of 8 keys 1024 bytes apart and 64-element panels `panel` bytes apart.
__device__ __forceinline__ uint64_t desc_k(uint32_t smem) {
  return static_cast<uint64_t>((smem >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t smem, uint32_t panel) {
  return static_cast<uint64_t>((smem >> 4) & 0x3FFFu) | (static_cast<uint64_t>(panel >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// kind::f16, fp16 operands, fp32 sums, 128 rows; bit 16: B is MN-major.
__device__ __forceinline__ constexpr uint32_t idesc_f16(int n, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
// A from TMEM: row = lane, two fp16 of K a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// H32 of 32 values of one thread, the butterfly of quad_rotate.
__device__ __forceinline__ void rotate32(float (&v)[32]) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(i & h)) {
        const float a = v[i], b = v[i + h];
        v[i] = __fadd_rn(a, b);
        v[i + h] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] *= c_h32();
}

// Keys that the rows row0 .. row0 + rows - 1 see, from a block's start on, and the tiles of them.
__device__ __forceinline__ int key_tiles(const PromptArgs& p, const Seq& q, int row0, int rows, int& key0) {
  int lo, hi, ignore;
  seen(p.a, q.len - q.n + row0 / p.group, q.len, lo, ignore);
  seen(p.a, q.len - q.n + (row0 + rows - 1) / p.group, q.len, ignore, hi);
  key0 = min(lo, q.len) / kKvTokens * kKvTokens;
  return max(1, (max(hi, 0) - key0 + kBK - 1) / kBK);
}

// A sequence's row tiles, all heads, and the key tiles of its last.
struct Plan {
  int tiles, keys;
};
template <int D>
__device__ __forceinline__ Plan plan_of(const PromptArgs& p, const Seq& q) {
  const int64_t rows = static_cast<int64_t>(q.n) * p.group;
  if (q.n == 0 || rows < p.least_rows) return {0, 0};
  const int n = static_cast<int>((rows + Shape<D>::kRows - 1) / Shape<D>::kRows), row0 = (n - 1) * Shape<D>::kRows;
  int key0;
  return {n * p.c.heads, key_tiles(p, q, row0, static_cast<int>(rows) - row0, key0)};
}

// What a CTA does: rows row0 .. row0 + rows - 1 of (sequence, head), key tiles t0 .. t1 - 1 of
// those that start at key0, as part `part` of `parts`; part i of a tile is kept at slot0 + i.
struct Work {
  int b, head, row0, rows;
  Seq q;
  int key0, t0, t1, part, parts, slot0;
};
// Sum of v over the CTA's threads, and before this one's.  carry: shared, of 32.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* carry, int threads, int64_t& before) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t at = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, at, d);
    if (lane >= d) at += o;
  }
  __syncthreads();
  if (lane == 31) carry[warp] = at;
  __syncthreads();
  int64_t total = 0;
  before = at - v;
  for (int i = 0; i < threads / 32; ++i) {
    if (i < warp) before += carry[i];
    total += carry[i];
  }
  return total;
}
// By whole CTAs; prefix: shared, of batch entries, not used for up to 32 sequences: then each warp finds it by itself,
// without a barrier.  join: of the join's CTAs, one a cut tile: its work is that of the tile's first part.  False:
// nothing to do.
// With fewer row tiles than SMs and a workspace, a sequence's tiles have their keys cut into parts, each of as
// many key tiles at most as let all parts have an SM; two at least, since a part costs its q, its first copies
// and its write of O.  Tiles in descending order: with a causal mask a sequence's later rows see more keys.
template <int D>
__device__ __forceinline__ bool find_work(const PromptArgs& p, int* prefix, int64_t* carry, int threads, int cta, bool join, Work& w) {
  const int tid = threadIdx.x, lane = tid & 31;
  const bool small = p.s.batch <= 32;
  int64_t tiles = 0, keys = 0, total = 0, before = 0;
  Plan o{0, 0};
  Seq seq{};
  if (small) {
    if (lane < p.s.batch) {
      seq = kv_seq(p.s, lane, p.c.page, p.err);
      o = plan_of<D>(p, seq);
    }
    tiles = o.tiles;
    keys = static_cast<int64_t>(o.tiles) * o.keys;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, d);
      keys += __shfl_xor_sync(0xFFFFFFFFu, keys, d);
    }
  } else {
    for (int b0 = 0; b0 < p.s.batch; b0 += threads) {
      o = Plan{0, 0};
      if (b0 + tid < p.s.batch) o = plan_of<D>(p, kv_seq(p.s, b0 + tid, p.c.page, p.err));
      tiles += block_scan(o.tiles, carry, threads, before);
      keys += block_scan(static_cast<int64_t>(o.tiles) * o.keys, carry, threads, before);
    }
  }
  if (tiles == 0) return false;
  // ceil(n / most) a tile, at most n / most + 1: keys / most + tiles parts
  int most = 0;
  if (p.parts && 2 * tiles <= p.sms) most = static_cast<int>(max(int64_t(2), (keys + p.sms - tiles - 1) / (p.sms - tiles)));
  if (join && !most) return false;
  const auto parts_of = [&](const Plan& o) { return most ? (o.keys + most - 1) / most : 1; };
  // The CTA's tile is `in` of sequence b, whose parts begin at slot `first` of all.  The join counts tiles, and the
  // slots before them beside.
  const auto count = [&](const Plan& o) { return static_cast<int64_t>(o.tiles) * (join ? 1 : parts_of(o)); };
  int at, b = 0, in, first;
  if (small) {
    const int64_t sum = count(o), slots = static_cast<int64_t>(o.tiles) * parts_of(o);
    before = sum;
    int64_t slots_before = slots;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, before, d), y = __shfl_up_sync(0xFFFFFFFFu, slots_before, d);
      if (lane >= d) before += x, slots_before += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, before, 31);
    before -= sum;
    slots_before -= slots;
    if (cta >= total) return false;
    at = static_cast<int>(total) - 1 - cta;
    b = 31 - __clz(__ballot_sync(0xFFFFFFFFu, lane < p.s.batch && before <= at));
    w.q.first = __shfl_sync(0xFFFFFFFFu, seq.first, b);
    w.q.n = __shfl_sync(0xFFFFFFFFu, seq.n, b);
    w.q.len = __shfl_sync(0xFFFFFFFFu, seq.len, b);
    in = at - static_cast<int>(__shfl_sync(0xFFFFFFFFu, before, b));
    first = static_cast<int>(__shfl_sync(0xFFFFFFFFu, slots_before, b));
  } else {
    int64_t slots = 0;
    first = 0;
    for (int b0 = 0; b0 < p.s.batch; b0 += threads) {
      o = Plan{0, 0};
      if (b0 + tid < p.s.batch) o = plan_of<D>(p, kv_seq(p.s, b0 + tid, p.c.page, nullptr));
      const int64_t sum = block_scan(count(o), carry, threads, before);
      if (b0 + tid < p.s.batch) prefix[b0 + tid] = static_cast<int>(total + before);
      total += sum;
      if (join) {
        int64_t mine;
        const int64_t all = block_scan(static_cast<int64_t>(o.tiles) * parts_of(o), carry, threads, mine);
        if (b0 + tid < p.s.batch) prefix[p.s.batch + b0 + tid] = static_cast<int>(slots + mine);
        slots += all;
      }
    }
    __syncthreads();
    if (cta >= total) return false;
    at = static_cast<int>(total) - 1 - cta;
    for (int hi = p.s.batch; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (prefix[mid] <= at) b = mid;
      else hi = mid;
    }
    w.q = kv_seq(p.s, b, p.c.page, nullptr);
    in = at - prefix[b];
    first = join ? prefix[p.s.batch + b] : prefix[b];
  }
  w.b = b;
  const int parts = most ? parts_of(plan_of<D>(p, w.q)) : 1;
  w.part = join ? 0 : in % parts;
  if (!join) in /= parts;
  w.slot0 = first + in * parts;
  w.head = in % p.c.heads;
  w.row0 = in / p.c.heads * Shape<D>::kRows;
  w.rows = min(Shape<D>::kRows, w.q.n * p.group - w.row0);
  const int n = key_tiles(p, w.q, w.row0, w.rows, w.key0);
  w.parts = min(parts, (n + 1) / 2);  // an earlier row tile may see fewer keys than the last
  w.t0 = static_cast<int>(static_cast<int64_t>(n) * w.part / w.parts);
  w.t1 = static_cast<int>(static_cast<int64_t>(n) * (w.part + 1) / w.parts);
  return w.part < w.parts;
}

// Blocks of 16 keys of tiles 0 .. n - 1 in the order of the tiles, K's eight and then V's: their codes to the rings
// of the warps that take them, by one warp, and each tile's scales.
template <int D>
__device__ __forceinline__ void copy_codes(const PromptArgs& p, const Work& w, int key0, int n, uint8_t* smem, Bars& S, float (&sc)[4][3][kBlocks]) {
  using C = Shape<D>;
  const int lane = threadIdx.x & 31, v = (lane >> 3) & 1, b = lane & 7;  // lanes 0-15: the tile's blocks
  const auto page_of = [&](int j) {  // of tile j's block, -1: none
    const int t = key0 + j * kBK + b * kKvTokens;
    return lane < 16 && j < n && t < w.q.len ? kv_page(p.s, p.c, w.b, t, p.err) : -1;
  };
  int next = page_of(0);
  for (int j = 0; j < n; ++j) {
    const int page = next, t = key0 + j * kBK + b * kKvTokens, in_page = t & (p.c.page - 1);
    next = page_of(j + 1);
    bool ok = true;
    // as many lanes at a time as there are places: a later one may wait for an earlier one's block to be taken
#pragma unroll 1
    for (int from = 0; from < 16; from += C::kSlots, __syncwarp()) {
      if (lane < from || lane >= min(16, from + C::kSlots)) continue;
      const int u = 16 * j + lane, turn = u / kConvertWarps, slot = u % kConvertWarps * C::kDepth + turn % C::kDepth, round = turn / C::kDepth;
      if (round > 0) ok = wait_bar(S, &S.raw_empty[slot], (round - 1) & 1, p);
      if (ok) {
        S.raw_none[slot] = page < 0;
        if (page < 0) {
          mbar_arrive(&S.raw_full[slot]);
        } else {
          mbar_expect_tx(&S.raw_full[slot], C::kBlock);
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           su32(smem + C::kRaw + slot * C::kBlock)),
                       "l"(p.c.codes + kv_at(p.c, page, w.head, v) + static_cast<int64_t>(in_page) * D), "r"(C::kBlock), "r"(su32(&S.raw_full[slot]))
                       : "memory");
        }
      }
    }
    // a block without a page, or past the sequence: no weight (its codes are zeros)
    const int byte = page < 0 ? -1 : p.c.scales[kv_scale_at(p.c, page, w.head, v) + in_page / kKvTokens];
    // not k_empty: this tile's own products may be done by now, and a parity does not tell two phases on
    if (j >= 4) ok = ok && wait_bar(S, &S.sc_empty[j & 3], (j / 4 - 1) & 1, p);
    if (!__all_sync(0xFFFFFFFFu, ok)) return;
    const float f = kv_scale(byte);
    if (lane < 8) {
      sc[j & 3][0][b] = byte < 0 ? 0.0f : f;
    } else if (lane < 16) {
      sc[j & 3][1][b] = byte < 0 ? kNegInf : kv_exponent(byte);
      sc[j & 3][2][b] = byte < 0 ? 0.0f : ex2(-kv_exponent(byte));
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.sc_full[j & 3]);
  }
}

// The ring's blocks, of which warp `first` of kConvertWarps takes every kConvertWarps-th: to fp16 in the swizzled rows
// of the tile's buffer.  A lane takes 16 codes of rows lane / 4 and lane / 4 + 8 in every panel of 64: eight
// neighbours write on different banks, and find the swizzle's share of an address in a register.  (With the codes
// loaded to registers, the fence before the MMAs waited for the next block's loads as well: 1000 cycles a block.)
template <int D>
__device__ __forceinline__ void convert(const PromptArgs& p, int n, int first, uint8_t* smem, Bars& S) {
  using C = Shape<D>;
  const int lane = threadIdx.x & 31, units = n * 2 * kBlocks;
  const uint32_t k0 = su32(smem + C::kK) + (lane >> 2) * 128;
  const uint32_t lo = k0 + (((2 * (lane & 3)) ^ (lane >> 2)) << 4), hi = k0 + (((2 * (lane & 3) + 1) ^ (lane >> 2)) << 4);
  // The ring is the warp's own: whoever waits for a round of a place has seen the one before, so that a phase's parity
  // says which of the two it is.
  for (int u = first, turn = 0; u < units; u += kConvertWarps, ++turn) {
    const int slot = first * C::kDepth + turn % C::kDepth, round = turn / C::kDepth;
    const int j = u >> 4, v = (u >> 3) & 1, b = u & 7, buf = j % C::kBufs;
    if (!__all_sync(0xFFFFFFFFu, wait_bar(S, &S.raw_full[slot], round & 1, p))) return;
    const bool none = S.raw_none[slot] != 0;
    const uint8_t* const raw = smem + C::kRaw + slot * C::kBlock + (lane >> 2) * D + 16 * (lane & 3);
    uint4 x[C::kPieces];
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i)
      x[i] = none ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(raw + (i & 1) * 8 * D + (i >> 1) * 64);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.raw_empty[slot]);
    if (j >= C::kBufs && !__all_sync(0xFFFFFFFFu, wait_bar(S, v ? &S.v_empty[buf] : &S.k_empty[buf], (j / C::kBufs - 1) & 1, p))) return;
    const uint32_t at = (v ? C::kV - C::kK : 0) + buf * C::kTile + b * kKvTokens * 128;
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) {
      const uint32_t a = x[i].x ^ 0x80808080u, b4 = x[i].y ^ 0x80808080u, c = x[i].z ^ 0x80808080u, d = x[i].w ^ 0x80808080u;
      const uint32_t to = at + (i & 1) * 1024 + (i >> 1) * C::kPanel;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(lo + to), "r"(codes_half2(a, 0x4140u)), "r"(codes_half2(a, 0x4342u)),
                   "r"(codes_half2(b4, 0x4140u)), "r"(codes_half2(b4, 0x4342u))
                   : "memory");
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(hi + to), "r"(codes_half2(c, 0x4140u)), "r"(codes_half2(c, 0x4342u)),
                   "r"(codes_half2(d, 0x4140u)), "r"(codes_half2(d, 0x4342u))
                   : "memory");
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(v ? &S.v_full[buf] : &S.k_full[buf]);
  }
}

// q to shared memory by warps 0-7: rotated as the keys are, scaled by a power of two per row, in the swizzle; four
// pieces' loads are out at a time, in a loop of one piece (eight unrolled: 1 us more where a CTA has few key tiles).  Rows
// past the last are zeros (a NaN there would have its warp look for maxima).
template <int D>
__device__ __forceinline__ void load_q(const PromptArgs& p, const Work& w, int qtiles, uint8_t* smem, float* row_factor) {
  using C = Shape<D>;
  const float sign = p.a.scale < 0.0f ? -1.0f : 1.0f;
  constexpr int kOnce = 4, kTogether = D < 256 ? 256 / D : 1;  // pieces a thread has out; rows of a warp's pass
  constexpr int kStep = 256 / (D / 8);                         // rows of all threads' pass
  const int rows = (w.rows + kTogether - 1) / kTogether * kTogether, cc = threadIdx.x % (D / 8), row0 = threadIdx.x / (D / 8);
  const auto place = [&](int row, int cc) {
    return reinterpret_cast<uint4*>(smem + C::kQ + (row >> 7) * 128 * D * 2 + (cc >> 3) * C::kPanel + (row & 127) * 128 + (((cc & 7) ^ (row & 7)) << 4));
  };
  for (int ch = rows * (D / 8) + threadIdx.x; ch < qtiles * 128 * (D / 8); ch += 256) *place(ch / (D / 8), ch % (D / 8)) = make_uint4(0, 0, 0, 0);
  for (int row = rows + threadIdx.x; row < qtiles * 128; row += 256) row_factor[row] = 0.0f;
  // row row0 is head `h` of the group at token `t`; kStep rows on without another division
  int t = (w.row0 + row0) / p.group, h = w.row0 + row0 - t * p.group;
  const int dt = kStep / p.group, dh = kStep - dt * p.group;
  Chunk<float> raw[kOnce];
  int ahead = row0;  // the next row to ask for
  const auto ask = [&](Chunk<float>& x) {
    if (ahead < w.rows) {
      const int64_t at = static_cast<int64_t>(w.q.first + t) * p.a.ldq + (w.head * p.group + h) * p.a.ldqh + 8 * cc;
      if (p.a.q_bf16) reinterpret_cast<Chunk<__nv_bfloat16>&>(x).load(static_cast<const __nv_bfloat16*>(p.a.q) + at, false);
      else x.load(static_cast<const float*>(p.a.q) + at, false);
    }
    ahead += kStep;
    t += dt;
    h += dh;
    if (h >= p.group) h -= p.group, ++t;
  };
#pragma unroll
  for (int i = 0; i < kOnce; ++i) ask(raw[i]);
#pragma unroll 1
  for (int row = row0; row < rows; row += kStep) {  // the same trips for a warp: its pieces fill whole rows
    float v[8] = {};
    if (row < w.rows) {
      if (p.a.q_bf16) reinterpret_cast<const Chunk<__nv_bfloat16>&>(raw[0]).get(v);
      else raw[0].get(v);
    }
#pragma unroll
    for (int i = 0; i + 1 < kOnce; ++i) raw[i] = raw[i + 1];
    ask(raw[kOnce - 1]);
    if (p.c.rotated) quad_rotate(v, threadIdx.x & 3);
    float amax = lane_amax(v);
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) amax = max3_abs(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d), 0.0f);
    const int e = row_exponent(amax);
    const float f = sign * pow2i(-e);  // the scale's sign goes to q: the scores' factors are positive
    *place(row, cc) = make_uint4(pack_half(v[0] * f, v[1] * f), pack_half(v[2] * f, v[3] * f), pack_half(v[4] * f, v[5] * f), pack_half(v[6] * f, v[7] * f));
    if (cc == 0) row_factor[row] = fabsf(p.a.scale) * 1.4426950408889634f * pow2i(e);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv8_prompt_kernel(const __grid_constant__ PromptArgs p) {
  using C = Shape<D>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Bars S;
  __shared__ float sm_f[C::kRows];
  // per tile of keys: K scales, V exponents, 2^-exponent
  __shared__ __align__(16) float sm_sc[4][3][kBlocks];
  __shared__ int64_t sm_carry[32];
  __shared__ Work sm_work;
  uint8_t* const smem = raw_smem + ((1024u - (su32(raw_smem) & 1023u)) & 1023u);
  const uint32_t sbase = su32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], kBlocks);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], kBlocks);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_ready[i][0], 4);
      mbar_init(&S.p_ready[i][1], 4);
      mbar_init(&S.pv_done[i][0], 1);
      mbar_init(&S.pv_done[i][1], 1);
      mbar_init(&S.o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&S.sc_full[i], 1);
    mbar_init(&S.q_full, 8);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&S.raw_full[i], 1);
      mbar_init(&S.raw_empty[i], 1);
    }

    S.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&S.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  grid_dep_launch();  // behind the allocation
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  grid_dep_wait();
  // Of up to 32 sequences warp 0 finds the CTA's work; all warps read it from shared memory, from where the compiler
  // takes it for the same in every lane (straight from the shuffles the loops cost 11% more).
  if (p.s.batch > 32 || warp == 0) {
    Work w;
    const bool some = find_work<D>(p, reinterpret_cast<int*>(smem + C::kPrefix), sm_carry, kThreads, static_cast<int>(blockIdx.x), false, w);
    if (tid == 0) {
      if (!some) w.rows = 0;
      sm_work = w;
      for (int i = 0; i < 4; ++i) mbar_init(&S.sc_empty[i], C::kTiles == 2 && w.rows > 128 ? 8 : 4);  // the softmax's warps
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  }
  __syncthreads();
  const Work w = sm_work;
  if (w.rows == 0) {
    __syncthreads();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    return;
  }
  const int n = w.t1 - w.t0;
  const int key0 = w.key0 + w.t0 * kBK;
  const int qtiles = C::kTiles == 2 && w.rows > 128 ? 2 : 1;

  if (warp >= 8) {
    if constexpr (C::kRegs2 < 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegs2));
    if (p.delay > 0 && warp == 9) {
      const int64_t t0 = clock64();
      while (clock64() - t0 < p.delay) {
      }
    }
    if (warp > 9) {
      convert<D>(p, n, warp - 10, smem, S);
    } else if (warp == 9) {
      copy_codes<D>(p, w, key0, n, smem, S, sm_sc);
    } else if (__all_sync(0xFFFFFFFFu, wait_bar(S, &S.q_full, 0, p))) {
      const auto qk = [&](int t, int s, int j) {  // row tile t, into S number s
        const uint32_t q = sbase + C::kQ + t * 128 * D * 2, k = sbase + C::kK + (j % C::kBufs) * C::kTile;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_f16(tmem + C::kS + s * 128, desc_k(q + (i >> 2) * C::kPanel + (i & 3) * 32), desc_k(k + (i >> 2) * C::kPanel + (i & 3) * 32),
                    idesc_f16(kBK, false), i > 0);
          mma_commit(&S.s_full[s]);
        }
        __syncwarp();
      };
      // half h of the tile's keys
      const auto pv = [&](int t, int s, int j, int h, bool last) {
        const uint32_t v = sbase + C::kV + (j % C::kBufs) * C::kTile;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kBK / 32; ++i)
            mma_ts(tmem + C::kO + t * D, tmem + C::kS + s * 128 + 32 * h + 8 * i, desc_mn(v + 8192 * h + i * 2048, C::kPanel), idesc_f16(D, true),
                   j > 0 || h > 0 || i > 0);
          if (last) mma_commit(&S.v_empty[j % C::kBufs]);
          mma_commit(&S.pv_done[t][h]);
          if (j == n - 1 && h == 1) mma_commit(&S.o_done[t]);
        }
        __syncwarp();
      };
      const auto ready = [&](uint64_t* b, int phase) {
        const bool ok = __all_sync(0xFFFFFFFFu, wait_bar(S, b, phase & 1, p));
        tc_fence_after();
        return ok;
      };
      const auto free_k = [&](int j) {
        if (elect_one()) mma_commit(&S.k_empty[j % C::kBufs]);
        __syncwarp();
      };
      bool live = true;
      if constexpr (C::kTiles == 2) {
        for (int j = 0; live && j <= n; ++j) {
          if (j < n && !(live = ready(&S.k_full[j % C::kBufs], j / C::kBufs))) break;
          for (int t = 0; t < qtiles; ++t) {
            if (j > 0) {
              if (t == 0 && !(live = ready(&S.v_full[(j - 1) % C::kBufs], (j - 1) / C::kBufs))) break;
              if (!(live = ready(&S.p_ready[t][0], j - 1))) break;
              pv(t, t, j - 1, 0, false);
              if (!(live = ready(&S.p_ready[t][1], j - 1))) break;
              pv(t, t, j - 1, 1, t == qtiles - 1);
            }
            if (j < n) qk(t, t, j);
          }
          if (live && j < n) free_k(j);
        }
      } else {
        if ((live = ready(&S.k_full[0], 0))) {
          qk(0, 0, 0);
          free_k(0);
        }
        for (int j = 0; live && j < n; ++j) {
          if (j + 1 < n) {
            if (!(live = ready(&S.k_full[(j + 1) % C::kBufs], (j + 1) / C::kBufs))) break;
            qk(0, (j + 1) & 1, j + 1);
            free_k(j + 1);
          }
          if (!(live = ready(&S.v_full[j % C::kBufs], j / C::kBufs))) break;
          for (int h = 0; h < 2; ++h) {
            if (!(live = ready(&S.p_ready[j & 1][h], j >> 1))) break;
            pv(0, j & 1, j, h, h == 1);
          }
        }
      }
    }
  } else {
    load_q<D>(p, w, qtiles, smem, sm_f);
    fence_async_smem();
    asm volatile("bar.sync 1, 256;" ::: "memory");  // the rows' factors
    if (lane == 0) mbar_arrive(&S.q_full);
  }
  if (warp >= 8) {
  } else if ((warp >> 2) < qtiles) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegs0));
    const int t = warp >> 2, row = tid & (C::kRows - 1);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16), o_at = lanes + C::kO + t * D;
    const float f = sm_f[row];
    int lo, hi;
    seen(p.a, w.q.len - w.q.n + (w.row0 + min(row, w.rows - 1)) / p.group, w.q.len, lo, hi);
    int lo_all = lo, hi_all = hi;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      lo_all = max(lo_all, __shfl_xor_sync(0xFFFFFFFFu, lo_all, d));
      hi_all = min(hi_all, __shfl_xor_sync(0xFFFFFFFFu, hi_all, d));
    }
    constexpr int kHalf = kBK / 2, kHB = kBlocks / 2;
    // scores to the exponents of their weights, -infinity where the row does not see the key
    const auto mask = [&](float (&x)[kHalf], const float (&kscale)[kHB], const float (&vexp)[kHB], int key) {
#pragma unroll
      for (int c = 0; c < kHalf; ++c) {
        const float y = fmaf(x[c], kscale[c >> 4] * f, vexp[c >> 4]);
        x[c] = key + c >= lo && key + c < hi ? y : kNegInf;
      }
    };
    // 16 weights 2^(x g + c), as fp16, and their sum
    const auto weights = [&](const float* x, float g, float c, uint32_t* o) {
      float2 all = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float2 a = __ffma2_rn(make_float2(x[i], x[i + 1]), make_float2(g, g), make_float2(c, c));
        const float2 e = make_float2(ex2(a.x), ex2(a.y));
        all = i == 0 ? e : __fadd2_rn(all, e);
        o[i / 2] = pack_half(e.x, e.y);
      }
      return all.x + all.y;
    };
    float m = kNegInf, l = 0.0f;
    bool live = true;
    for (int j = 0; live && j < n; ++j) {
      const int s = C::kTiles == 2 ? t : j & 1, phase = C::kTiles == 2 ? j : j >> 1;
      live = __all_sync(0xFFFFFFFFu, wait_bar(S, &S.s_full[s], phase & 1, p) && wait_bar(S, &S.sc_full[j & 3], (j >> 2) & 1, p));
      if (!live) break;
      tc_fence_after();
      const uint32_t s_at = lanes + C::kS + s * 128;
      const int k0 = key0 + j * kBK;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t r[kHalf];
        tmem_ld32(s_at + h * kHalf, *reinterpret_cast<uint32_t(*)[32]>(r));
        tmem_ld32(s_at + h * kHalf + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) tie16(r + c);
        const bool masked = k0 + h * kHalf < lo_all || k0 + (h + 1) * kHalf > hi_all;
        // Weights against the maximum so far.  None is negative, so that sums of 16 of at most kMost say that each fits
        // fp16: the maximum itself is looked for, and O and the sums rescaled, only where a sum does not.
        float (&x)[kHalf] = *reinterpret_cast<float(*)[kHalf]>(&r);
        const float* const at = &sm_sc[j & 3][0][h * kHB];
        const float4 g4 = *reinterpret_cast<const float4*>(at), e4 = *reinterpret_cast<const float4*>(at + kBlocks), b4 = *reinterpret_cast<const float4*>(at + 2 * kBlocks);
        const float kscale[4] = {g4.x, g4.y, g4.z, g4.w}, vexp[4] = {e4.x, e4.y, e4.z, e4.w}, vback[4] = {b4.x, b4.y, b4.z, b4.w};
        if (masked) mask(x, kscale, vexp, k0 + h * kHalf);
        bool sure = j + h == 0;  // no reference yet
        while (true) {
          if (sure) {
            float top = kNegInf;
#pragma unroll
            for (int b = 0; b < kHB; ++b) {
              float y = fmaxf(x[16 * b], x[16 * b + 1]);
#pragma unroll
              for (int c = 2; c < 16; c += 2) y = fmaxf(fmaxf(y, x[16 * b + c]), x[16 * b + c + 1]);
              top = fmaxf(top, masked ? y : fmaf(y, kscale[b] * f, vexp[b]));
            }
            const float next = fmaxf(m, top - kShift), c = next == m ? 1.0f : ex2(m - next);
            m = next;
            l *= c;
            if (j + h > 0) {
              // O so far: the product before this one has to be done.  The product of the tile before that one is (this
              // tile's S came behind it), so that a phase's parity tells which of the two is meant.
              live = (j == 0 || __all_sync(0xFFFFFFFFu, wait_bar(S, &S.pv_done[t][1], (j - 1) & 1, p))) &&
                     (h == 0 || __all_sync(0xFFFFFFFFu, wait_bar(S, &S.pv_done[t][0], j & 1, p)));
              if (!live) break;
              tc_fence_after();
#pragma unroll 1
              for (int d = 0; d < D; d += 32) {
                uint32_t o[32];
                tmem_ld32(o_at + d, o);
                tmem_wait32(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * c);
                tmem_st32(o_at + d, o);
              }
            }
          }
          const float z = m == kNegInf ? 0.0f : m;
          float sum = 0.0f, most = 0.0f;
          uint32_t w2[kHalf / 2];
          if (!masked) {
#pragma unroll
            for (int b = 0; b < kHB; ++b) {
              const float all = weights(x + 16 * b, kscale[b] * f, vexp[b] - z, w2 + 8 * b);
              most = max_nan(most, all);
              sum = fmaf(all, vback[b], sum);
            }
          } else {
#pragma unroll
            for (int b = 0; b < kHB; ++b) {
              const float all = weights(x + 16 * b, 1.0f, -z, w2 + 8 * b);
              most = max_nan(most, all);
              if (all != 0.0f) sum = fmaf(all, vback[b], sum);  // a NaN scale that the row does not see counts for nothing
            }
          }
          if (sure || !__any_sync(0xFFFFFFFFu, !(most <= kMost) || m == kNegInf)) {
            l += sum;
            tmem_st32(s_at + h * (kHalf / 2), w2);
            break;
          }
          sure = true;
        }
        if (!live) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_ready[s][h]);
      }
      if (lane == 0) mbar_arrive(&S.sc_empty[j & 3]);
    }
    if (live && __all_sync(0xFFFFFFFFu, wait_bar(S, &S.o_done[t], 0, p))) {
      tc_fence_after();
      const int g = w.row0 + row;
      const int64_t at = static_cast<int64_t>(w.q.first + g / p.group) * p.a.ldo + (w.head * p.group + g % p.group) * p.a.ldoh;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint8_t* const stage = smem + C::kQ + (t * 4 + (warp & 3)) * 32 * D * 2;  // 4 KB at least
      float* const part = w.parts > 1 ? p.parts + static_cast<int64_t>(w.slot0 + w.part) * C::kPart : nullptr;
      if (part) {
        part[C::kRows * D + row] = m;
        part[C::kRows * (D + 1) + row] = l;
      }
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        tmem_ld32(o_at + d, o);
        tmem_wait32(o);
        float (&v)[32] = *reinterpret_cast<float(*)[32]>(&o);
        if (part) {
          // four elements of every row together: a warp's rows side by side
          float4* const to = reinterpret_cast<float4*>(part) + (d >> 2) * C::kRows + row;
          if (row < w.rows)
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i * C::kRows] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          continue;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = l == 0.0f ? 0.0f : v[i] * inv;
        if (p.c.rotated) rotate32(v);
        // by way of shared memory, whose Q is done with: pieces of a row side by side
        if (p.a.o_bf16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __floats2bfloat162_rn(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
            memcpy(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), y, 16);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int from = 8 * i + (lane >> 2), cc = lane & 3;
            const int64_t to = __shfl_sync(0xFFFFFFFFu, at, from);
            if (row - lane + from < w.rows)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + to + d + 8 * cc) =
                  *reinterpret_cast<const uint4*>(stage + from * 64 + ((cc ^ ((from >> 1) & 3)) << 4));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int from = 4 * i + (lane >> 3), cc = lane & 7;
            const int64_t to = __shfl_sync(0xFFFFFFFFu, at, from);
            if (row - lane + from < w.rows)
              *reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + to + d + 4 * cc) =
                  *reinterpret_cast<const float4*>(stage + from * 128 + ((cc ^ (from & 7)) << 4));
          }
        }
        __syncwarp();
      }
    }
  } else {
    if constexpr (C::kRegs1 < 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegs1));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegs1));
  }
  tc_fence_before();
  __syncthreads();
  if (S.abort) {  // MMAs in flight read shared memory and write TMEM: wait out the bound
    const int64_t t0 = clock64();
    while (clock64() - t0 < kWaitCycles) {
    }
  }
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// The parts of cut tiles together, in a fixed order.  grid (cut tiles at most, 32 rows x 32 elements of a tile): a
// thread takes four elements of a row, a warp 32 rows side by side as the parts hold them, and the warps of a group
// every groups-th part; the groups meet in shared memory, where a row's 32 elements meet for H32.  (One group, its
// warps over rows 8 KB apart: 24 parts 20 us, 76 parts 49.)
constexpr int kJoinGroup = 256, kJoinMost = 4, kAtOnce = 8;
// What sums of weights 2^(. - m), l of them together, count for against `top`: nothing without a key seen, unless NaN.
__device__ __forceinline__ float join_factor(float m, float l, float top) {
  return m == kNegInf ? (l == l ? 0.0f : 1.0f) : ex2(m - top);
}
template <int D>
__global__ void __launch_bounds__(kJoinGroup* kJoinMost) kv8_join_kernel(const __grid_constant__ PromptArgs p) {
  using C = Shape<D>;
  __shared__ int prefix[2 * kKvMaxBatch];
  __shared__ int64_t carry[32];
  __shared__ __align__(16) float sm_v[kJoinMost][32][36];
  __shared__ float sm_m[kJoinMost][32], sm_l[kJoinMost][32];
  grid_dep_launch();
  grid_dep_wait();
  __shared__ Work sm_work;
  const int tid = threadIdx.x, groups = blockDim.x / kJoinGroup, group = tid / kJoinGroup;
  const int row0 = blockIdx.y / (D / 32) * 32, chunk = blockIdx.y % (D / 32);
  if (p.s.batch > 32 || tid < 32) {  // of up to 32 sequences one warp finds the tile
    Work found;
    if (!find_work<D>(p, prefix, carry, blockDim.x, static_cast<int>(blockIdx.x), true, found)) found.rows = 0;
    if (tid == 0) sm_work = found;
  }
  __syncthreads();
  const Work w = sm_work;
  if (row0 >= w.rows || w.parts == 1) return;
  const int in = tid & 31, row = row0 + in, quad = tid / 32 % 8;
  float top = kNegInf, l = 0.0f;
  float4 v = make_float4(0, 0, 0, 0);
  // eight parts' loads out together; what is summed so far moves to the new maximum
  for (int i0 = group; i0 < w.parts && row < w.rows; i0 += kAtOnce * groups) {
    float m[kAtOnce], x[kAtOnce];
    float4 y[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      m[i] = kNegInf;
      x[i] = 0.0f;
      y[i] = make_float4(0, 0, 0, 0);
      if (i0 + i * groups < w.parts) {
        const float* const at = p.parts + static_cast<int64_t>(w.slot0 + i0 + i * groups) * C::kPart;
        m[i] = __ldcg(at + C::kRows * D + row);
        x[i] = __ldcg(at + C::kRows * (D + 1) + row);
        y[i] = __ldcg(reinterpret_cast<const float4*>(at) + (8 * chunk + quad) * C::kRows + row);
      }
    }
    float next = top;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) next = fmaxf(next, m[i]);
    const float c = next == top ? 1.0f : ex2(top - next);
    top = next;
    l *= c;
    v.x *= c; v.y *= c; v.z *= c; v.w *= c;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float f = join_factor(m[i], x[i], top);
      l += x[i] * f;
      v.x += y[i].x * f; v.y += y[i].y * f; v.z += y[i].z * f; v.w += y[i].w * f;
    }
  }
  *reinterpret_cast<float4*>(&sm_v[group][in][4 * quad]) = v;
  if (quad == 0) {
    sm_m[group][in] = top;
    sm_l[group][in] = l;
  }
  __syncthreads();
  if (tid < 128) {
    const int r = tid >> 2, e = 8 * (tid & 3);
    float m = kNegInf, sum = 0.0f, o[8] = {};
    for (int g = 0; g < groups; ++g) m = fmaxf(m, sm_m[g][r]);
    for (int g = 0; g < groups; ++g) {
      const float f = join_factor(sm_m[g][r], sm_l[g][r], m);
      sum += sm_l[g][r] * f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += sm_v[g][r][e + i] * f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = sum == 0.0f ? 0.0f : o[i] / sum;
    if (p.c.rotated) quad_rotate(o, tid & 3);
    if (row0 + r < w.rows) {
      const int g = w.row0 + row0 + r;
      const int64_t at = static_cast<int64_t>(w.q.first + g / p.group) * p.a.ldo + (w.head * p.group + g % p.group) * p.a.ldoh + 32 * chunk + e;
      if (p.a.o_bf16) store8(static_cast<__nv_bfloat16*>(p.a.out) + at, o, false);
      else store8(static_cast<float*>(p.a.out) + at, o, false);
    }
  }
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, int threads, int smem, const PromptArgs& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Row tiles: most_tiles at most; all_tiles at least if every token belongs to a sequence, which only the device knows: a
// buffer's offsets may name a few of its rows.  Whether tiles may be cut is decided here alone, by the call's sizes: the
// kernel gets parts to cut into only where the join follows.  So a short batch is not cut in a buffer whose rows would not
// be if all were named: 100 rows of 512 behind 15900 keys, 40 heads of 128 over 8, take 269 us.  A join behind every call
// with offsets would make that 58 us and cost all others its launch: ragged prompts of heads of 64 33.1 -> 36.1 us, 4096
// tokens of 8 sequences of 4000 keys 379 -> 382.
template <int D>
cudaError_t launch_prompt(PromptArgs p, int64_t all_tiles, int64_t most_tiles, cudaStream_t st) {
  using C = Shape<D>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(kv8_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  // tiles are cut while there are two SMs each and three key tiles
  if (2 * all_tiles > p.sms || static_cast<int64_t>(p.s.width) * p.c.page <= 2 * kBK) p.parts = nullptr;
  const int64_t grid = most_tiles > p.sms ? most_tiles : p.sms;
  e = launch(kv8_prompt_kernel<D>, dim3(static_cast<unsigned>(p.parts ? grid : most_tiles)), kThreads, C::kSmem, p, st);
  if (e != cudaSuccess || !p.parts) return e;
  const int64_t cut = most_tiles < p.sms / 2 ? most_tiles : p.sms / 2, parts = p.sms / cut;
  const int groups = parts >= 4 * kAtOnce ? 4 : parts >= 2 * kAtOnce ? 2 : 1;  // about eight parts each
  const int64_t rows = (p.s.cu ? static_cast<int64_t>(p.s.tokens) : p.s.each) * p.group;  // of a sequence at most
  const int64_t y = ((rows < C::kRows ? rows : C::kRows) + 31) / 32 * (D / 32);
  return launch(kv8_join_kernel<D>, dim3(static_cast<unsigned>(cut), static_cast<unsigned>(y)), groups * kJoinGroup, 0, p, st);
}

int64_t g_wait = kWaitCycles, g_delay = 0;

}  // namespace

void kv8_set_wait_limit(uint64_t wait_ns, uint64_t producer_delay_ns) {
  const auto cycles = [](uint64_t ns) { return static_cast<int64_t>(ns / 100 * 207 + ns % 100 * 207 / 100); };  // 2.07 GHz
  g_wait = wait_ns ? cycles(wait_ns) : kWaitCycles;
  g_delay = cycles(producer_delay_ns);
}

size_t kv8_prompt_workspace_bytes(int dim) {
  const size_t part = dim == 64 ? Shape<64>::kPart : dim == 128 ? Shape<128>::kPart : Shape<256>::kPart;
  return kWsCounters + static_cast<size_t>(num_sms()) * part * sizeof(float);
}

cudaError_t launch_kv8_prompt(const KvCache& c, const KvSeqs& s, const KvAttn& a, int least_rows, void* ws, cudaStream_t st) {
  PromptArgs p{};
  p.c = c;
  p.s = s;
  p.a = a;
  p.group = a.q_heads / c.heads;
  p.least_rows = least_rows;
  p.sms = num_sms();
  p.parts = ws ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsCounters) : nullptr;
  p.err = device_error_word();
  p.wait = g_wait;
  p.delay = g_delay;
  // row tiles at most: each sequence's last may be short
  const int64_t rows = c.dim == 256 ? Shape<256>::kRows : Shape<128>::kRows;
  const int64_t few = s.batch < s.tokens ? s.batch : s.tokens;
  const int64_t most = c.heads * (s.cu ? static_cast<int64_t>(s.tokens) * p.group / rows + few
                                       : s.batch * ((static_cast<int64_t>(s.each) * p.group + rows - 1) / rows));
  // and if all tokens belong to one, at least: with all the rows that may be the other kernel's taken off
  const int64_t mine = static_cast<int64_t>(s.tokens) * p.group - static_cast<int64_t>(least_rows - 1) * s.batch;
  const int64_t all = s.cu ? c.heads * (mine > 0 ? (mine + rows - 1) / rows : 0) : most;
  switch (c.dim) {
    case 64: return launch_prompt<64>(p, all, most, st);
    case 128: return launch_prompt<128>(p, all, most, st);
    default: return launch_prompt<256>(p, all, most, st);
  }
}

}  // namespace w4a4
