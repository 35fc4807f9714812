// The 8-bit paged key/value cache as the kernels see it: pages of `page` tokens, a scale
// byte (2^(s - 127), 255 = NaN) for each 16 tokens and head, and the sequences of a call.
#pragma once

#include "w4a4_device.cuh"
#include "w4a4_kernels.cuh"

namespace w4a4 {

constexpr int kKvTokens = 16;               // tokens that share a scale
constexpr int kKvLow = -40, kKvHigh = 40;   // exponents that a scale may have

__device__ __forceinline__ void kv_flag(int* err) {
  if (err) atomicOr(err, kErrPage);
}

// Sequence b of a call: tokens first .. first + n - 1 are its last n, len tokens in all
// (what the table holds at most).  Offsets and lengths are the caller's data: whatever
// they say, the tokens lie in 0 .. tokens - 1 and the length in the table's pages.
struct Seq {
  int first, n, len;
};
__device__ __forceinline__ Seq kv_seq(const KvSeqs& s, int b, int page, int* err) {
  Seq q;
  if (s.cu) {
    const int a = s.cu[b], e = s.cu[b + 1];
    q.first = min(max(a, 0), s.tokens);
    q.n = min(max(e, q.first), s.tokens) - q.first;
    if (a != q.first || e != q.first + q.n) kv_flag(err);
  } else {
    q.first = b * s.each;
    q.n = s.each;
  }
  const int len = s.lens[b], cap = s.width * page;
  q.len = min(max(len, 0), cap);
  if (len != q.len) kv_flag(err);
  return q;
}

// Page that holds token t of sequence b, or -1 where the table's entry is not one.
__device__ __forceinline__ int kv_page(const KvSeqs& s, const KvCache& c, int b, int t, int* err) {
  const int p = s.table[static_cast<int64_t>(b) * s.ldt + (t >> c.page_log)];
  if (static_cast<unsigned>(p) < static_cast<unsigned>(c.pages)) return p;
  kv_flag(err);
  return -1;
}

// First code of (page, head, K or V), and the first of its scales.
__device__ __forceinline__ int64_t kv_at(const KvCache& c, int page, int head, int v) {
  return ((static_cast<int64_t>(page) * c.heads + head) * 2 + v) * c.page * c.dim;
}
__device__ __forceinline__ int64_t kv_scale_at(const KvCache& c, int page, int head, int v) {
  return ((static_cast<int64_t>(page) * c.heads + head) * 2 + v) * (c.page / kKvTokens);
}

// 2^e of -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The exponent that byte s stands for, as a float: NaN for 255; a byte that no append wrote (of a page of zeros, for
// instance) counts as the nearest that one would.
__device__ __forceinline__ float kv_exponent(int s) {
  return s == 255 ? __uint_as_float(0x7FC00000u) : static_cast<float>(min(max(s - 127, kKvLow), kKvHigh));
}
__device__ __forceinline__ float kv_scale(int s) {
  return s == 255 ? __uint_as_float(0x7FC00000u) : pow2i(min(max(s - 127, kKvLow), kKvHigh));
}

}  // namespace w4a4
