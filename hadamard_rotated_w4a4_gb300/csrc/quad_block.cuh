// A 32-element block held by four neighbouring lanes, eight consecutive elements
// each (lane q = lane & 3 holds elements 8q .. 8q + 7): the H32 rotation, the
// block maximum and the three code formats.  Chunk c = 8 elements is the unit the
// fused quantisers index by; it is 16 bytes of bf16 or 32 of fp32, so a warp's
// loads and stores of consecutive chunks are contiguous without a transposition.
#pragma once

#include <cuda_bf16.h>

#include "w4a4_device.cuh"
#include "w4a4_kernels.cuh"

namespace w4a4 {

// ---------------------------------------------------------------- loads and stores of a chunk
// A chunk as it is loaded: 8 fp32, or 8 bf16 in 4 registers.  fp32 chunks move as one
// 32-byte access where the address allows it (`wide`, the same for a whole call): two of
// 16 bytes each fill half of every 32-byte sector they touch.
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  float v[8];
  // kLast: this kernel does not read the values again, and L2 may drop them before its
  // codes.  Another reader of the same rows then finds fewer of them there.
  template <bool kLast = false>
  __device__ __forceinline__ void load(const float* p, bool wide) {
    if (wide && kLast) {
      asm volatile("ld.global.L2::evict_first.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                   : "l"(p)
                   : "memory");
    } else if (wide) {
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                   : "l"(p)
                   : "memory");
    } else {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i];
  }
};
template <>
struct Chunk<__nv_bfloat16> {
  uint4 a;
  template <bool kLast = false>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    a = kLast ? __ldcs(q) : *q;
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bf16 is the high half of the fp32 of the same value
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
__device__ __forceinline__ void store8(float* p, const float (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8], bool) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // round to nearest even
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    memcpy(&w[i], &h, 4);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// Whether rows of T at p, ld elements apart, can move 32 bytes at a time.
template <typename T>
bool wide_rows(const T* p, int64_t ld) {
  return sizeof(T) == 4 && ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * 4)) & 31) == 0;
}

// a - b on register pairs (a fused multiply by -1 rounds like the subtraction).
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.0f, -1.0f), a); }

// ---------------------------------------------------------------- rotation
// The normalised 32-point Walsh-Hadamard transform, stages h = 1, 2, 4 inside the
// lane, 8 and 16 across lanes: each pair becomes (a + b, a - b) with the fp32 adds
// of the one-lane form (a fused multiply by +-1 rounds like the add), then one
// multiply by fl32(1/sqrt 32).  Stages past the first run on register pairs, the same
// operations two to an instruction.  All 32 lanes must call it.
__device__ __forceinline__ void quad_rotate(float (&v)[8], int q) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float a = v[i], b = v[i + 1];
    v[i] = __fadd_rn(a, b);
    v[i + 1] = __fsub_rn(a, b);
  }
  float2 (&w)[4] = *reinterpret_cast<float2 (*)[4]>(&v);
#pragma unroll
  for (int h = 1; h < 4; h <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & h)) {
        const float2 a = w[i], b = w[i + h];
        w[i] = __fadd2_rn(a, b);
        w[i + h] = sub2(a, b);
      }
#pragma unroll
  for (int h = 1; h < 4; h <<= 1) {
    const float s = (q & h) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __ffma2_rn(w[i], make_float2(s, s),
                        make_float2(__shfl_xor_sync(0xFFFFFFFFu, w[i].x, h), __shfl_xor_sync(0xFFFFFFFFu, w[i].y, h)));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __fmul2_rn(w[i], make_float2(c_h32(), c_h32()));
}

// max |v| over this lane's eight values, then over the block's four lanes; NaN if any
// element is NaN.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float lane_amax(const float (&v)[8]) {
  return max3_abs(max3_abs(max3_abs(v[0], v[1], v[2]), v[3], v[4]), max3_abs(v[5], v[6], v[7]), 0.0f);
}
__device__ __forceinline__ float quad_amax(const float (&v)[8]) {
  float a = lane_amax(v);
  a = max3_abs(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1), 0.0f);
  return max3_abs(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2), 0.0f);
}

// ---------------------------------------------------------------- code formats
enum Fmt : int { kInt4 = 4, kInt8 = 8, kMx = 32 };

// Where a fused quantiser writes its codes.
struct QuantOut {
  uint8_t* codes;
  void* scales;       // fp32 [rows][K/32] (int4, int8) or scale tiles of bytes (MXFP4)
  uint8_t* expanded;  // int4 only, may be null: the offset codes a + 8 as bytes
  int64_t ktiles;     // MXFP4: scale tiles along K, ceil(K / 128)
};

// Byte of the scale of (row, block) in the MXFP4 scale tiles: 512-byte tiles of 128
// rows x 4 blocks, in the order the tensor core's scale copy reads them (row r of
// the tile at 16 * (r % 32) + 4 * (r / 32), its four blocks in a row).  I: uint32_t
// where the tiles' bytes fit it, else int64_t.
template <typename I>
__device__ __forceinline__ I mx_scale_at(I row, I blk, I ktiles) {
  return ((row >> 7) * ktiles + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// Two values to a byte of e2m1 codes (lo in the low nibble): round to nearest, ties
// to even, saturating at +-6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// a / top, correctly rounded, top a small integer: a multiply by the reciprocal and one
// correction of the exact remainder (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990).  The remainder of a tiny or huge a may
// leave the range in which it is exact: the division itself then.
__device__ __forceinline__ float div_by(float a, float top) {
  if (!(a > 1e-30f && a < 1e30f)) return __fdiv_rn(a, top);
  const float r = top == 7.0f ? 1.0f / 7.0f : 1.0f / 127.0f;
  const float q = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-top, q, a), r, q);
}

// Quantise this lane's eight values of a block and store them if ok.
//   kInt4: d = amax / 7, codes round-half-away(v * fl(1/d)) clamped to -8..7, nibbles
//          in the Q4_0 order (element i low, i + 16 high);
//   kInt8: d = amax / 127, codes clamped to -127..127, element order;
//   kMx:   scale 2^E, E = clamp(floor(log2 amax) - 2, -127, 127) stored as E + 127,
//          codes e2m1(v * 2^-E), element 2i in the low nibble of byte i.
// A block with an infinity or a NaN gets a NaN scale and zero codes, so it reads
// back, and multiplies, as NaN.  c is the chunk's flat index row * K / 8 + col.
template <int FMT, typename I>
__device__ __forceinline__ void quad_quantize(float (&v)[8], int q, bool ok, I c, I row, I blk, I nblk_row,
                                              const QuantOut& o) {
  const float a = quad_amax(v);
  const bool bad = !(a <= 3.402823466e38f);
  float2 (&v2)[4] = *reinterpret_cast<float2 (*)[4]>(&v);
  if constexpr (FMT == kMx) {
    // floor(log2 a) from the exponent field; a subnormal a ends at the clamp
    const int e = max(static_cast<int>(__float_as_uint(a) >> 23) - 127 - 2, -127);
    // 2^-E, e in -127 .. 125: its exponent field is 127 - e, in 2 .. 254
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) v2[i] = __fmul2_rn(v2[i], make_float2(inv, inv));
    const uint32_t w = e2m1x8(v);
    if (ok) {
      reinterpret_cast<uint32_t*>(o.codes)[c] = bad ? 0u : w;
      if (q == 0) {
        uint8_t* s = static_cast<uint8_t*>(o.scales) + mx_scale_at<I>(row, blk, static_cast<I>(o.ktiles));
        *s = bad ? 255 : static_cast<uint8_t>(e + 127);
        if (blk == nblk_row - 1)  // the tile's unused blocks multiply zero codes: any finite scale
          for (int p = 1; p < 4 - static_cast<int>(blk & 3); ++p) s[p] = 0;
      }
    }
  } else {
    constexpr float kTop = FMT == kInt4 ? 7.0f : 127.0f;
    constexpr float kLow = FMT == kInt4 ? -8.0f : -127.0f;
    const float d = bad ? __uint_as_float(0x7FC00000u) : div_by(a, kTop);
    // a scale without a finite reciprocal (2^-128 at most, or NaN): codes of 0
    const float rcp = __frcp_rn(d);
    const float inv = rcp <= 3.402823466e38f ? rcp : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v2[i] = __fmul2_rn(v2[i], make_float2(inv, inv));
    // Where the scale is finite, |v| is at most kTop and a part in 2^21 of it (a few ulp, and
    // the rounding of a subnormal d):
    // v + 1.5 * 2^23 is 1.5 * 2^23 plus the nearest integer (ties to even), whose low
    // byte is that integer in two's complement.  It is the rounding half away from zero
    // unless some v lies halfway (or is NaN); then the general path rounds.
    constexpr float kMagic = 12582912.0f;
    uint32_t t[8], w[2];
    float x[8];  // v - nearest
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 s = __fadd2_rn(v2[i], make_float2(kMagic, kMagic));
      const float2 r = __fadd2_rn(s, make_float2(-kMagic, -kMagic));
      const float2 dx = sub2(v2[i], r);
      x[2 * i] = dx.x;
      x[2 * i + 1] = dx.y;
      t[2 * i] = __float_as_uint(s.x);
      t[2 * i + 1] = __float_as_uint(s.y);
    }
    if (lane_amax(x) < 0.5f) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[h] = prmt(prmt(t[4 * h], t[4 * h + 1], 0x0040u), prmt(t[4 * h + 2], t[4 * h + 3], 0x0040u), 0x5410u);
    } else {
      w[0] = w[1] = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float r = fminf(fmaxf(round_half_away(v[i]), kLow), kTop);
        w[i >> 2] |= (bad ? 0u : static_cast<uint32_t>(static_cast<int>(r)) & 0xFFu) << (8 * (i & 3));
      }
    }
    if (ok && q == 0) static_cast<float*>(o.scales)[c >> 2] = d;
    if constexpr (FMT == kInt8) {
      if (ok) reinterpret_cast<uint2*>(o.codes)[c] = make_uint2(w[0], w[1]);
    } else {
      w[0] &= 0x0F0F0F0Fu;
      w[1] &= 0x0F0F0F0Fu;
      // lane q pairs with lane q + 2, which holds the elements 16 further on
      const uint32_t h0 = __shfl_down_sync(0xFFFFFFFFu, w[0], 2), h1 = __shfl_down_sync(0xFFFFFFFFu, w[1], 2);
      if (ok) {
        if (q < 2) {
          uint2* p = reinterpret_cast<uint2*>(o.codes) + (c >> 2) * 2 + q;
          *p = make_uint2(w[0] | (h0 << 4), w[1] | (h1 << 4));
        }
        if (o.expanded)  // a + 8 = nibble ^ 8
          reinterpret_cast<uint2*>(o.expanded)[c] = make_uint2(w[0] ^ 0x08080808u, w[1] ^ 0x08080808u);
      }
    }
  }
}

}  // namespace w4a4
