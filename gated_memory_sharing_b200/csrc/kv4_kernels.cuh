// The KV cache held in 4 bits: rows quantised as they are written, read back,
// and the cross-attention decode that reads them ("Decoder-Hybrid-Decoder
// Architecture for Efficient Reasoning with Long Generation", Paper-Notes
// page, 方法详解 > 整体框架: one KV cache, written once by the self-decoder's
// full-attention layer and read by every cross-attention layer; 研究背景与动机:
// a cross-attention layer moves O(d_kv N) memory per decoded token).
//
// Per token and KV head a row of D values is kept in D / 16 blocks of 16:
//
//   x ~ 2^e * s * c,   s = e4m3(min(448, max|x| 2^-e / 6)),   c = e2m1(|x| 2^-e / s)
//
// with e a whole number per KV head and both roundings to nearest even.  c is
// one of 0, .5, 1, 1.5, 2, 3, 4, 6 (and a sign); s * c has at most 6
// significant bits and is a multiple of 2^-10, so it is exact in f16, bf16 and
// f32.  A border between two values of c (or s) is a product of a few bits, so
// comparing |x| (or the maximum) with it is exact in f32 and both roundings
// are the definition's, bit for bit.  A block that holds a NaN or an infinity
// gets the scale NaN and reads back as NaN.  4.5 bits an element.
//
// Layout.  A page holds P tokens (a power of two from 16) of all KV heads:
// [page][head][P / 16] groups of 16 tokens, each 18 D bytes and laid out as
// the m16n8k16 A fragments that the attention feeds to the tensor cores, lane
// (g = lane / 4, t = lane % 4), so that a lane's fragments of 64 values a
// token are one 16-byte load:
//   K codes, 8 D bytes: per 64 values (blocks 4c .. 4c+3) 32 lanes x 16 bytes;
//     lane (g, t): token g (8 bytes), token g + 8 (8 bytes), each 2 bytes per
//     block b: values 16 b + 4 t .. + 3 (the lower nibble first)
//   V codes, 8 D bytes: per 64 values 32 lanes x 16 bytes; lane (g, t): four
//     words of one byte per block b: value 16 b + 2 g of tokens 2t (lower
//     nibble), 2t + 1; value 16 b + 2 g + 1 of these; and both of tokens 2t + 8,
//     2t + 9
//   K scales, D bytes: [g][token g, token g + 8][block]
//   V scales, D bytes: [t][block][tokens 2t, 2t + 1, 2t + 8, 2t + 9]
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace sambay {
namespace kv4 {

constexpr int kGroup = 16;                    // tokens of a group
constexpr int kStatusBadIndex = 1;            // == SAMBAY_ERR_INVALID_ARG
constexpr int kMaxExp = 64;                   // |e| of a head

template <int D>
struct Block {
  static constexpr int kK = 0;                // K codes
  static constexpr int kV = 8 * D;            // V codes
  static constexpr int kKs = 16 * D;          // K scales
  static constexpr int kVs = 17 * D;          // V scales
  static constexpr int kBytes = 18 * D;
};

// Which pages a call works on.
struct Pages {
  uint8_t* cache;          // [num_pages][Hkv][P / 16][18 D]
  const int32_t* table;    // [B, table_pages]
  const int32_t* k_exp;    // [Hkv] or null (0)
  const int32_t* v_exp;    // [Hkv] or null (0)
  int B, Hkv, page_log2, num_pages, table_pages;   // P = 2^page_log2 tokens
};

// One of the small index arrays' values.  EARLY: by a kernel that has not yet
// waited for the one in front of it; through L2, past what an SM may have kept.
template <bool EARLY>
__device__ __forceinline__ int index_at(const int32_t* p, int i) { return EARLY ? __ldcg(p + i) : p[i]; }

template <bool EARLY = false>
__device__ __forceinline__ int head_exp(const int32_t* e, int h) {
  return e ? max(-kMaxExp, min(kMaxExp, index_at<EARLY>(e, h))) : 0;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// The group of token `pos` of sequence b for head h; null where the position
// or its page is outside the table or the pool.
template <int D>
__device__ __forceinline__ uint8_t* group_of(const Pages& pg, int b, int h, int pos) {
  if (pos < 0 || (pos >> pg.page_log2) >= pg.table_pages) return nullptr;
  const int page = pg.table[static_cast<long long>(b) * pg.table_pages + (pos >> pg.page_log2)];
  if (page < 0 || page >= pg.num_pages) return nullptr;
  const int in = (pos & ((1 << pg.page_log2) - 1)) / kGroup;
  return pg.cache +
         (((static_cast<long long>(page) * pg.Hkv + h) << (pg.page_log2 - 4)) + in) * Block<D>::kBytes;
}

// ---------------------------------------------------------------- rows in and out

// Two 4-bit values of each byte of a word, as f16 (the lower nibble in the lower half).
__device__ __forceinline__ void e2m1x8_f16x2(uint32_t w, uint32_t (&d)[4]) {
  asm("{\n\t.reg .b8 p, q, r, s;\n\tmov.b32 {p, q, r, s}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\tcvt.rn.f16x2.e2m1x2 %1, q;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, r;\n\tcvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}
// Four e4m3 scales as f16 pairs (exact; NaN stays NaN).
__device__ __forceinline__ void e4m3x4_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, p;\n\tcvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// Both halves of `a` times the lower or the upper half of `b` (an operand
// selection of the multiply, no instruction of its own).
__device__ __forceinline__ uint32_t mul_f16x2_half(uint32_t a, uint32_t b, int upper) {
  uint32_t d;
  if (upper)
    asm("{\n\t.reg .f16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {h, h};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(d) : "r"(a), "r"(b));
  else
    asm("{\n\t.reg .f16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {l, l};\n\tmul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 8 x 8 of 16 bits, rows over g and columns 2t, 2t + 1, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {          // without its sign; not of NaN
  uint32_t two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(two)));
}
__device__ __forceinline__ uint32_t e4m3_code(float x) {              // nearest even, at most 448
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(x));
  return two & 0x7Fu;
}
// Eight codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1_codes(float2 a, float2 b, float2 c, float2 d) {
  uint32_t w;
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
      "mov.b32 %0, {p, q, r, s};\n\t}"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return w;
}

// Pairs of f32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Four consecutive values of a row, and of them the largest |x|'s bits (those
// of a NaN or an infinity are the largest), for each io type.
//
// Both roundings (amax / 6 to e4m3, x / s to e2m1) are made by the conversion
// instructions from a product with a rounded reciprocal, at most 2^-21 off.
// That decides rightly except where the exact quotient lies on a border
// between two values (or, for f32, within the error of one).
//   bf16: x and the border times the divisor have at most 8 significant bits,
//     so a quotient that is not on a border is at least 2^-9 of it away.  Adding
//     and taking away kRound leaves multiples of 2^-13 below 2^9: a quotient
//     of e2m1 that is on a border becomes it (all are multiples of 1/4), the
//     others stay on their side.  For the scale, a factor of 1 + 2^-20 puts
//     every quotient above its exact value, and cutting it to 16 bits does the same.
//   f32: the same rounding finds the quotients within 2^-14 of a number of 4
//     bits (every border is one); comparing x with that number times the
//     divisor, exact in f32, settles them.
constexpr float kRound = 1536.0f;            // 1.5 x 2^10

__device__ __forceinline__ float2 rounded(float2 x, float fac) {
  return add2(fma2(x, make_float2(fac, fac), make_float2(kRound, kRound)), make_float2(-kRound, -kRound));
}

template <typename T> struct Four;
template <> struct Four<bf16> {
  uint2 v;
  static constexpr uint32_t kInf = 0x7F80u;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
  // two maxima side by side, until top_of()
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m;
    asm("{\n\t.reg .b32 a, b;\n\tabs.bf16x2 a, %1;\n\tabs.bf16x2 b, %2;\n\tmax.NaN.bf16x2 %0, a, b;\n\t}" : "=r"(m) : "r"(v.x), "r"(v.y));
    return m;
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
  static __device__ __forceinline__ uint32_t top_of(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
  static __device__ __forceinline__ float top_value(uint32_t bits) { return __uint_as_float(bits << 16); }
  // e4m3 code of amax / 6 * two; two: a power of two
  static __device__ __forceinline__ uint32_t scale_code(float amax, float two) {
    const float y = amax * two * (0.16666667f * 1.00000095f);
    return e4m3_code(fminf(__uint_as_float(__float_as_uint(y) & 0xFFFFFF80u), 448.0f));
  }
  __device__ __forceinline__ void values(float (&x)[4]) const {
    x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  // the largest |x| that is a number
  __device__ __forceinline__ float top_abs() const {
    float x[4];
    values(x);
    return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
  }
  // the four over the scale (fac: 2^-e over it), rounded as said
  __device__ __forceinline__ void quotients(float fac, float, float, float2& a, float2& b) const {
    a = rounded(make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u)), fac);
    b = rounded(make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u)), fac);
  }
};
template <> struct Four<float> {
  float4 v;
  static constexpr uint32_t kInf = 0x7F800000u;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
  __device__ __forceinline__ uint32_t top() const {
    return max(max(abs_bits(v.x), abs_bits(v.y)), max(abs_bits(v.z), abs_bits(v.w)));
  }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t top_of(uint32_t m) { return m; }
  static __device__ __forceinline__ float top_value(uint32_t bits) { return __uint_as_float(bits); }
  static __device__ __forceinline__ uint32_t scale_code(float amax, float two) {
    const float a = amax * two;
    const uint32_t c = e4m3_code(fminf(a * 0.16666667f, 448.0f));
    // off by one code at most: 6 times the border on either side
    const float w = e4m3_value(c);
    const float up = c < 126 ? 3.0f * (w + e4m3_value(c + 1)) : INFINITY;
    const float down = c > 0 ? 3.0f * (w + e4m3_value(c - 1)) : -1.0f;
    const bool odd = c & 1u;
    if (a > up || (a == up && odd && c < 126)) return c + 1;
    return a < down || (a == down && odd) ? c - 1 : c;
  }
  __device__ __forceinline__ void values(float (&x)[4]) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
  __device__ __forceinline__ float top_abs() const {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
  }
  // x over s * 2^e, on the right side of a border that it is near
  static __device__ __forceinline__ float settled(float x, float y, float s, float two) {
    const uint32_t b = __float_as_uint(y);
    if ((b & 0xFFFFFu) != 0 || y == 0.0f) return y;
    const float ax = fabsf(x * two), t = fabsf(y) * s;
    return __uint_as_float(ax > t ? b + 1u : ax < t ? b - 1u : b);
  }
  __device__ __forceinline__ void quotients(float fac, float s, float two, float2& a, float2& b) const {
    a = rounded(make_float2(v.x, v.y), fac);
    b = rounded(make_float2(v.z, v.w), fac);
    a = make_float2(settled(v.x, a.x, s, two), settled(v.y, a.y, s, two));
    b = make_float2(settled(v.z, b.x, s, two), settled(v.w, b.y, s, two));
  }
};

__device__ __forceinline__ void store4(float* p, float2 a, float2 b) {
  *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(bf16* p, float2 a, float2 b) {
  Pack16 u;
  u.h2[0] = __floats2bfloat162_rn(a.x, a.y);
  u.h2[1] = __floats2bfloat162_rn(b.x, b.y);
  *reinterpret_cast<uint2*>(p) = make_uint2(u.u.x, u.u.y);
}

constexpr int kRowWarps = 4;     // of a CTA (4 x 32768 bf16 tokens written: 151 us, with 8 warps 156 us)

template <typename T>
struct RowParams {
  Pages pg;
  const T* K;              // write: rows, [B, T] tokens at k_stride elements
  const T* V;
  T* Ko;                   // read: rows [B, T, Hkv, D]
  T* Vo;
  const int32_t* pos;      // [B] cached tokens before the call's
  const int32_t* count;    // [B] rows of each sequence, or null (T)
  int T_, groups;          // groups: of 16 tokens that T rows may touch, (T + 30) / 16
  int heads_log2;          // of a CTA's warps, 2^heads_log2 side by side over the row, the others over the groups
  unsigned head_ctas;      // CTAs over a row
  long long k_stride, v_stride;
};

// Rows of sequence b: min(count, T) of them; a count outside 0 .. T is recorded.
template <bool EARLY = false>
__device__ __forceinline__ int rows_of(const int32_t* count, int b, int T, bool tell) {
  if (!count) return T;
  const int n = index_at<EARLY>(count, b);
  if ((n < 0 || n > T) && tell) record_status(kStatusBadIndex);
  return max(0, min(T, n));
}

// A warp's work in both directions: the 16 tokens of a group, 64 values of one
// head.  Lane (g, t) has values 16 b + 4 t .. + 3 of blocks b = 0 .. 3 of
// tokens g and g + 8 (half 0 and 1).
template <int D>
struct Unit {
  int b, col;              // col: first value of the row's Hkv * D
  int c;                   // 64-value part of the head
  int row[2];              // the lane's two rows of the call, -1 where they are none
  bool all;                // all 16 tokens are rows of the call
  uint8_t* grp;            // null: nothing to do

  template <typename T>
  __device__ __forceinline__ explicit Unit(const RowParams<T>& p) {
    constexpr int C = D / 64;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // CTAs over the row first: those that run together work on whole rows
    const unsigned deep = blockIdx.x / p.head_ctas, along = blockIdx.x - deep * p.head_ctas;
    const int hc = (along << p.heads_log2) + (warp & ((1 << p.heads_log2) - 1));
    const int gi = deep * (kRowWarps >> p.heads_log2) + (warp >> p.heads_log2);
    b = blockIdx.y;
    col = hc * 64;
    c = hc % C;
    grp = nullptr;
    row[0] = row[1] = -1;
    all = false;
    if (hc >= p.pg.Hkv * C || gi >= p.groups) return;
    const int n = rows_of(p.count, b, p.T_, hc == 0 && gi == 0);
    const int pos = p.pos[b];
    // the group's place in the sequence, and its first token's row of the call (from -15 on)
    const int at16 = (pos >> 4) + gi;
    const long long r0 = static_cast<long long>(at16) * kGroup - pos;
    if (n == 0 || r0 >= n) return;
    // what no table reaches stays outside it
    grp = group_of<D>(p.pg, b, hc / C, at16 < 0 ? -1 : min(at16, 1 << 26) * kGroup);
    if (!grp) {
      if (lane == 0) record_status(kStatusBadIndex);
      return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long r = r0 + (lane >> 2) + 8 * i;
      row[i] = r >= 0 && r < n ? static_cast<int>(r) : -1;
    }
    all = r0 >= 0 && r0 + kGroup <= n;
  }
};

// What a warp keeps of one side (K or V): per half the codes (two words, 16
// bits a block) and, in lane t = half (0 or 1), the word of the four scales.
template <typename T>
__device__ __forceinline__ void quantise(const Four<T> (&x)[2][4], float two, uint32_t (&codes)[2][2], uint32_t& scales) {
  const int lane = threadIdx.x & 31, t = lane & 3;
  // the blocks' maxima over the four lanes; lane t ends with those of half t & 1, blocks 2 (t >> 1), + 1
  uint32_t m[4], w[2];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t m0 = x[0][b].top(), m1 = x[1][b].top();
    m[b] = Four<T>::most(t & 1 ? m1 : m0, __shfl_xor_sync(0xFFFFFFFFu, t & 1 ? m0 : m1, 1));
  }
#pragma unroll
  for (int b = 0; b < 2; ++b)
    w[b] = Four<T>::top_of(
        Four<T>::most(t & 2 ? m[2 + b] : m[b], __shfl_xor_sync(0xFFFFFFFFu, t & 2 ? m[b] : m[2 + b], 2)));
  uint32_t code = 0;
  float s[2], fac[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const bool bad = w[b] >= Four<T>::kInf;
    const uint32_t c = bad ? 0x7Fu : Four<T>::scale_code(Four<T>::top_value(w[b]), two);
    s[b] = bad ? 0.0f : e4m3_value(c);
    fac[b] = s[b] > 0.0f ? __fdividef(two, s[b]) : 0.0f;           // 0: codes of 0
    code |= c << (8 * b);
  }
  scales = code | __shfl_xor_sync(0xFFFFFFFFu, code, 2) << 16;     // as it should be in lanes t = 0, 1
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float2 y[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int src = (lane & ~3) | i | (b >> 1) << 1;
      const float f = __shfl_sync(0xFFFFFFFFu, fac[b & 1], src);
      const float sb = sizeof(T) == 4 ? __shfl_sync(0xFFFFFFFFu, s[b & 1], src) : 0.0f;
      x[i][b].quotients(f, sb, two, y[2 * b], y[2 * b + 1]);
    }
    codes[i][0] = e2m1_codes(y[0], y[1], y[2], y[3]);
    codes[i][1] = e2m1_codes(y[4], y[5], y[6], y[7]);
  }
}

// Codes of tokens g, g + 8 (K's order) to V's order and back: bytes of two
// blocks move as 16 bits, 8 tokens by 8 pairs of values at a time.
__device__ __forceinline__ void to_v_order(const uint32_t (&k)[2][2], uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t r01 = movmatrix_trans(__byte_perm(k[i][0], 0, 0x3120));
    const uint32_t r23 = movmatrix_trans(__byte_perm(k[i][1], 0, 0x3120));
    const uint32_t w0 = __byte_perm(r01, r23, 0x5410), w1 = __byte_perm(r01, r23, 0x7632);   // tokens 2t, 2t + 1
    v[2 * i] = (w0 & 0x0F0F0F0Fu) | (w1 << 4 & 0xF0F0F0F0u);
    v[2 * i + 1] = (w0 >> 4 & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u);
  }
}
__device__ __forceinline__ void from_v_order(const uint32_t (&v)[4], uint32_t (&k)[2][2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t e = v[2 * i], o = v[2 * i + 1];
    const uint32_t w0 = (e & 0x0F0F0F0Fu) | (o << 4 & 0xF0F0F0F0u), w1 = (e >> 4 & 0x0F0F0F0Fu) | (o & 0xF0F0F0F0u);
    k[i][0] = __byte_perm(movmatrix_trans(__byte_perm(w0, w1, 0x5410)), 0, 0x3120);
    k[i][1] = __byte_perm(movmatrix_trans(__byte_perm(w0, w1, 0x7632)), 0, 0x3120);
  }
}

template <typename T>
__device__ __forceinline__ void load_rows(const T* p, long long stride, const int (&row)[2], Four<T> (&x)[2][4]) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (row[i] >= 0)
        x[i][b].load(p + row[i] * stride + 16 * b + 4 * t);
      else
        x[i][b].zero();
}

// Bound by the rows' bytes (bf16: 2 in and 0.56 out an element) and by ALU
// instructions (about 330 of 730 for a unit's 2048 elements).  4 x 32768 bf16
// tokens of 20 heads of 64: 151 us, 5.7 TB/s, 0.87 of the copy bandwidth.
// Warp: one unit.  Bytes of the group that belong to other tokens keep their
// values: K's codes and both scales are stored per token; of V's codes, where
// two tokens share a byte, a group that is not all the call's is read first.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRowWarps, sizeof(T) == 4 ? 4 : 10) kv4_write_kernel(const RowParams<T> p) {
  const Pages& pg = p.pg;
  pdl_wait();
  const Unit<D> un(p);
  if (!un.grp) return;                 // the whole warp's
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int KS = D / 16;
  Four<T> kx[2][4], vx[2][4];
  load_rows(p.K + un.b * (p.T_ * p.k_stride) + un.col, p.k_stride, un.row, kx);
  load_rows(p.V + un.b * (p.T_ * p.v_stride) + un.col, p.v_stride, un.row, vx);
  uint32_t codes[2][2], scales;
  quantise(kx, pow2i(-head_exp(pg.k_exp, un.col / D)), codes, scales);
  {
    uint8_t* dst = un.grp + Block<D>::kK + un.c * 512 + lane * 16;
    if (un.all) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(codes[0][0], codes[0][1], codes[1][0], codes[1][1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (un.row[i] >= 0) *reinterpret_cast<uint2*>(dst + 8 * i) = make_uint2(codes[i][0], codes[i][1]);
    }
    if (t < 2 && (t ? un.row[1] : un.row[0]) >= 0)
      *reinterpret_cast<uint32_t*>(un.grp + Block<D>::kKs + g * (2 * KS) + t * KS + 4 * un.c) = scales;
  }
  quantise(vx, pow2i(-head_exp(pg.v_exp, un.col / D)), codes, scales);
  uint32_t v[4];
  to_v_order(codes, v);
  // scales: rows over tokens, columns (blocks 0 1, 2 3) of half 0 and of half 1
  const uint32_t st = movmatrix_trans(t < 2 ? scales : 0u);
  const uint32_t other = __shfl_down_sync(0xFFFFFFFFu, st, 8);              // half 1's
  uint2 sv = make_uint2(__byte_perm(st, other, 0x6420), __byte_perm(st, other, 0x7531));
  uint4* vdst = reinterpret_cast<uint4*>(un.grp + Block<D>::kV + un.c * 512 + lane * 16);
  uint2* sdst = reinterpret_cast<uint2*>(un.grp + Block<D>::kVs + t * (4 * KS) + 16 * un.c + 8 * (g & 1));
  if (!un.all) {
    // whether tokens 2t, 2t + 1, 2t + 8, 2t + 9 are rows (bit 4 g of the ballots: token g's)
    const uint32_t lo = __ballot_sync(0xFFFFFFFFu, un.row[0] >= 0), hi = __ballot_sync(0xFFFFFFFFu, un.row[1] >= 0);
    const bool l0 = lo >> (8 * t) & 1, l1 = lo >> (8 * t + 4) & 1, h0 = hi >> (8 * t) & 1, h1 = hi >> (8 * t + 4) & 1;
    const uint32_t ml = (l0 ? 0x0F0F0F0Fu : 0u) | (l1 ? 0xF0F0F0F0u : 0u), mh = (h0 ? 0x0F0F0F0Fu : 0u) | (h1 ? 0xF0F0F0F0u : 0u);
    const uint4 old = *vdst;
    v[0] = (v[0] & ml) | (old.x & ~ml);
    v[1] = (v[1] & ml) | (old.y & ~ml);
    v[2] = (v[2] & mh) | (old.z & ~mh);
    v[3] = (v[3] & mh) | (old.w & ~mh);
    if (g < 2) {
      const uint32_t ms = (l0 ? 0xFFu : 0u) | (l1 ? 0xFF00u : 0u) | (h0 ? 0xFF0000u : 0u) | (h1 ? 0xFF000000u : 0u);
      const uint2 was = *sdst;
      sv.x = (sv.x & ms) | (was.x & ~ms);
      sv.y = (sv.y & ms) | (was.y & ~ms);
    }
  }
  *vdst = make_uint4(v[0], v[1], v[2], v[3]);
  if (g < 2) *sdst = sv;
}

// The values of one side into its rows: codes and scales as quantise() gives them.
template <typename T>
__device__ __forceinline__ void store_rows(T* p, long long stride, const int (&row)[2], const uint32_t (&codes)[2][2],
                                           uint32_t scales, float two) {
  const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t sl[2];
    e4m3x4_f16x2(__shfl_sync(0xFFFFFFFFu, scales, (lane & ~3) | i), sl[0], sl[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t x[4];
      e2m1x8_f16x2(codes[i][k], x);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 a = f16x2_f32(mul_f16x2_half(x[2 * e], sl[k], e)), b = f16x2_f32(mul_f16x2_half(x[2 * e + 1], sl[k], e));
        a.x *= two; a.y *= two; b.x *= two; b.y *= two;
        if (row[i] >= 0) store4(p + row[i] * stride + 16 * (2 * k + e) + 4 * t, a, b);
      }
    }
  }
}

// Bound by bytes: 4 x 32768 bf16 tokens back in 140 us, 6.1 TB/s, 0.94 of the copy bandwidth.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kRowWarps) kv4_read_kernel(const RowParams<T> p) {
  const Pages& pg = p.pg;
  pdl_wait();
  const Unit<D> un(p);
  if (!un.grp) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int KS = D / 16;
  const uint4 kc = *reinterpret_cast<const uint4*>(un.grp + Block<D>::kK + un.c * 512 + lane * 16);
  const uint4 vc = *reinterpret_cast<const uint4*>(un.grp + Block<D>::kV + un.c * 512 + lane * 16);
  const uint32_t ks = *reinterpret_cast<const uint32_t*>(un.grp + Block<D>::kKs + g * (2 * KS) + (t & 1) * KS + 4 * un.c);
  const uint2 sv = *reinterpret_cast<const uint2*>(un.grp + Block<D>::kVs + t * (4 * KS) + 16 * un.c + 8 * (g & 1));
  const long long stride = static_cast<long long>(pg.Hkv) * D, base = un.b * (p.T_ * stride) + un.col;
  uint32_t codes[2][2] = {{kc.x, kc.y}, {kc.z, kc.w}};
  store_rows(p.Ko + base, stride, un.row, codes, ks, pow2i(head_exp(pg.k_exp, un.col / D)));
  const uint32_t v[4] = {vc.x, vc.y, vc.z, vc.w};
  from_v_order(v, codes);
  // rows (blocks 0 1, 2 3) of half 0, of half 1; columns over tokens
  const uint32_t vs = movmatrix_trans(g & 2 ? __byte_perm(sv.x, sv.y, 0x7362) : __byte_perm(sv.x, sv.y, 0x5140));
  store_rows(p.Vo + base, stride, un.row, codes, vs, pow2i(head_exp(pg.v_exp, un.col / D)));
}

// ---------------------------------------------------------------- attention

// The tokens of all (sequence, KV head, row tile) pairs are cut into tiles of
// 4096 / D tokens (4608 bytes of cache) and laid end to end; every warp of the
// grid takes the same share of that line, whatever the lengths are, and goes
// through it on its own: no CTA-wide synchronisation, and a warp that changes
// from one pair to the next does not hold up the others.  Pairs that lie in
// one warp's share are finished there; of the others every warp leaves (m, l,
// O) for the combine kernel, which adds them in the line's order.
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 2;                       // of a warp's ring,
constexpr int kStageTiles = 2;                   // two tiles each
constexpr int kTileBytes = 4608;
constexpr int kScaleBytes = 512;                 // a tile's scales of K, then of V, as f16
constexpr int kWarpSmem = kStages * kStageTiles * kTileBytes + kScaleBytes;
constexpr int kAttnSmem = kWarps * (kWarpSmem + kStages * 8);      // three times this fit an SM
constexpr long long kWaitCycles = 1LL << 31;     // a copy that has not come after about a second
// Probabilities are kept times 2^15 (the largest of a row is 2^15): as f16 they
// then have 11 bits down to 2^-29 of the largest instead of 2^-14, which shows
// where the likeliest tokens' values are zero.  Numerator and denominator carry
// the same factor.  The largest score is taken away before the scale is
// multiplied in, so that the largest exponent is 15 however large the logits
// are: with 15 - scale * largest rounded to f32 it was off by half a step of
// that, past f16's end at 2^16 from logits of 2^24 on.
constexpr float kPShift = 15.0f;
constexpr float kNone = 3e38f;                   // less the largest score of a row that has seen nothing

// Resident CTAs an SM.  The kernel is bound by what the warp schedulers can
// dispatch, not by latency (12, 16 and 20 warps an SM measured the same), so a
// variant gets the registers that it needs: 168 a thread for 8 columns, 255 for
// 16 (168 spill: 64 x 2048 tokens at 16 query heads a KV head 82 us, 255 67 us).
__host__ __device__ constexpr int attn_ctas(int nt) { return nt == 1 ? 3 : 2; }

struct AttnParams {
  Pages pg;
  const void* q;           // [B, T, Hq, D] io
  void* out;               // [B, T, Hq, D] io
  const int32_t* lens;     // [B] cached tokens, the T new ones among them
  const int32_t* count;    // [B] query tokens of each sequence, or null (T)
  float* o_part;           // [warp][first or last pair][cols, D]  partial outputs
  float* ml_part;          // [warp][first or last pair][cols, 4]  their (largest score, l, factor of the scores, -)
  int T_, Hq, G;
  int group_inv;           // ceil(2^16 / G): r * group_inv >> 16 is r / G (r < 256, G <= 16)
  int row_tiles, cols;     // cols: min(8 NT, G T) columns of a row tile
  int page_bytes;
  uint32_t piece_mask, piece_low;      // groups of a page that a stage may hold: a bit each; their number less 1
  int warps;               // of the grid: at most one share of the line each
  float scale_log2;        // scale * log2(e)
};

__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T> __device__ __forceinline__ void load2(const T* p, float* x);
template <> __device__ __forceinline__ void load2<float>(const float* p, float* x) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  x[0] = v.x;
  x[1] = v.y;
}
template <> __device__ __forceinline__ void load2<bf16>(const bf16* p, float* x) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  x[0] = __uint_as_float(v << 16);
  x[1] = __uint_as_float(v & 0xFFFF0000u);
}
__device__ __forceinline__ void store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(bf16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
// The same with a zero accumulator in.
__device__ __forceinline__ void mma16816_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// A warp's ring: bulk copies that complete on one mbarrier a stage.
__device__ __forceinline__ void bar_init(uint32_t bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred q;\n\tmbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  if (bar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!bar_try(bar, parity))
    if (clock64() - t0 > kWaitCycles) return false;
  return true;
}
// Untiled copy of whole 16 bytes to this CTA's shared memory (no multicast).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Cached tokens of sequence b, inside the table; `tell` records a length outside it.
template <bool EARLY = false>
__device__ __forceinline__ int len_of(const AttnParams& p, int b, bool tell) {
  const int len = index_at<EARLY>(p.lens, b), cap = p.pg.table_pages << p.pg.page_log2;
  if (tell && (len < 0 || len > cap)) record_status(kStatusBadIndex);
  return max(0, min(cap, len));
}
// Tiles of a pair of a sequence: an empty one has one, which writes its zeros.
template <int D>
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + 4096 / D - 1) / (4096 / D)); }

// The line is measured in units, one a tile and, where shares are long, kSwitch
// more in front of each pair's first: what changing to a pair costs a warp, so
// that a run of empty and short sequences is not one warp's (37 sequences of 0 ..
// 5000 tokens: 33.4 us, without it 37.0 us; 1 and 4 units: 34.3 and 33.9 us).
// The line's length (below 2^31, the host sees to it) is cut into shares, none
// without a tile: share w has `base` units, or one more (the first `rem`).
constexpr int kSwitch = 2;
struct Line {
  int shares, base, rem;
  int gap;                 // units in front of a pair
  __device__ __forceinline__ int begin(int w) const { return w * base + min(w, rem); }
  // the share that holds unit x
  __device__ __forceinline__ int share_of(int x) const {
    const int cut = rem * (base + 1);
    return x < cut ? x / (base + 1) : rem + (x - cut) / base;
  }
};

// tiles: of one pair of every sequence
__device__ __forceinline__ Line make_line(const AttnParams& p, int tiles) {
  const int pairs = p.pg.Hkv * p.row_tiles;
  Line line;
  line.gap = tiles * pairs >= 4 * p.warps ? kSwitch : 0;
  const int units = (tiles + line.gap * p.pg.B) * pairs;
  line.shares = min(units, p.warps);
  line.base = static_cast<unsigned>(units) / static_cast<unsigned>(line.shares);
  line.rem = units - line.base * line.shares;
  return line;
}

// The line of a call, and the unit in it at which sequence b begins (one warp of
// the combine kernel).
template <int D>
__device__ __forceinline__ Line line_of(const AttnParams& p, int b, int* before) {
  int s = 0, sb = 0;
  for (int i = threadIdx.x & 31; i < p.pg.B; i += 32) {
    const int n = tiles_of<D>(len_of<true>(p, i, false));
    s += n;
    if (i < b) sb += n;
  }
  const Line line = make_line(p, __reduce_add_sync(0xFFFFFFFFu, s));
  *before = (static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, sb)) + line.gap * b) * p.pg.Hkv * p.row_tiles;
  return line;
}

// A place in the line.
struct Cursor {
  int b, h, rt, tile;      // sequence, KV head, row tile, tile
  int len, tiles;          // of sequence b
};

// n tiles on (no further than the pair's end); true if that is another pair.
// len: the length of a sequence that is reached.
template <int D, typename Len>
__device__ __forceinline__ bool advance(const AttnParams& p, Cursor& c, int n, Len len) {
  if ((c.tile += n) < c.tiles) return false;
  c.tile = 0;
  if (++c.rt == p.row_tiles) {
    c.rt = 0;
    if (++c.h == p.pg.Hkv) {
      c.h = 0;
      if (++c.b < p.pg.B) {
        c.len = len(c.b);
        c.tiles = tiles_of<D>(c.len);
      }
    }
  }
  return true;
}

// Units left of `left` after n tiles; 0 behind the last sequence.
__device__ __forceinline__ int pair_left(const AttnParams& p, const Cursor& c, int left, int n) {
  return c.b < p.pg.B ? left - n : 0;
}

// Inclusive sums over the warp's lanes.
__device__ __forceinline__ int scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The place in the line where share gw begins, and the units from there to its
// end: 0 where the share is none (one warp).  A lane sums the tiles of B / 32
// sequences; then the sequences of the lane that holds the place are looked
// through.  *gap: the line's.  (Lengths must not change while a call runs; if
// they do, what is computed is undefined, but stays inside the arrays: here, in
// pair_left() and in the combine kernel; and every copy is waited for, since the
// cursor that works takes the lengths that the one that loads has read.)
template <int D>
__device__ __forceinline__ int begin_of(const AttnParams& p, int gw, Cursor& c, int* gap) {
  const int lane = threadIdx.x & 31;
  const int pairs = p.pg.Hkv * p.row_tiles, per = (p.pg.B + 31) >> 5;
  int mine = 0, len = 0;
  for (int i = lane * per; i < min(p.pg.B, lane * per + per); ++i) {
    len = len_of(p, i, gw == 0);
    mine += tiles_of<D>(len);
  }
  int upto = scan(mine);                             // tiles of one pair of these sequences and those before
  const Line line = make_line(p, __shfl_sync(0xFFFFFFFFu, upto, 31));
  *gap = line.gap;
  if (gw >= line.shares) return 0;
  int x = line.begin(gw);
  int left = line.begin(gw + 1) - x;
  int before = upto - mine + line.gap * min(p.pg.B, lane * per);
  upto += line.gap * min(p.pg.B, lane * per + per);
  int k = __ffs(__ballot_sync(0xFFFFFFFFu, upto * pairs > x)) - 1;
  x -= __shfl_sync(0xFFFFFFFFu, before, k) * pairs;
  c.b = k;
  if (per > 1) {
    bool found = false;
    for (int b0 = k * per; b0 < p.pg.B && !found; b0 += 32) {
      const int i = b0 + lane;
      len = i < p.pg.B ? len_of(p, i, false) : 0;
      mine = i < p.pg.B ? tiles_of<D>(len) + line.gap : 0;
      const int sum = scan(mine);
      const unsigned past = __ballot_sync(0xFFFFFFFFu, sum * pairs > x);
      if (past) {
        k = __ffs(past) - 1;
        x -= __shfl_sync(0xFFFFFFFFu, sum - mine, k) * pairs;
        c.b = b0 + k;
        found = true;
      } else {
        x -= __shfl_sync(0xFFFFFFFFu, sum, 31) * pairs;
      }
    }
    if (!found) return 0;                            // lengths that changed meanwhile
  }
  c.len = __shfl_sync(0xFFFFFFFFu, len, k);
  c.tiles = tiles_of<D>(c.len);
  const int units = c.tiles + line.gap;
  const int pair = static_cast<unsigned>(x) / static_cast<unsigned>(units);
  if (pair >= pairs) return 0;                       // as above
  x -= pair * units + line.gap;
  c.tile = max(0, x);
  left += min(0, x);                                 // a share that begins in a pair's gap
  c.h = p.row_tiles == 1 ? pair : pair / p.row_tiles;
  c.rt = pair - c.h * p.row_tiles;
  return left;
}

// This thread's 128 bytes of an array, to L2.
__device__ __forceinline__ void prefetch_part(const void* p, long long bytes) {
  const long long at = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) * 128;
  if (at < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(p) + at));
}

// Bound by the cache's bytes (4.5 bits an element) and nearly as much by what
// unpacking them costs: a scheduler dispatches, for 16
// tokens of 64 values, 32 conversions of codes (2 clocks each), 32 multiplies by
// scales (1.4), 8 MMAs (3.4) and the softmax, about 190 clocks of the 198 that
// the bytes take at 6.56 TB/s.  Measured (a captured pass, the combine kernel in
// it): 16 sequences x 34816 tokens 141 us, 5.7 TB/s, 0.87 of the copy bandwidth
// (without its loads 133 us, without its arithmetic 125 us); 64 x 2048 44 us,
// 4.3 TB/s, of which about 13 us are starting (lengths, table, first tiles one
// after the other), the last parts and the combine kernel.
//
// Query row r of a (sequence, KV head): token r / G, head r % G of the group.
// The MMAs compute S^T = K Q^T and O^T = V^T P^T: tokens (values) are the 16
// rows of A, straight from the cache's layout, and 8 query rows the columns.
// q is scaled per row by a power of two into f16's range (bf16 fits f16's 11
// bits; with SPLIT (f32 io) it is a pair of f16, 22 bits, and so is P).
template <typename T, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, attn_ctas(NT)) kv4_attn_kernel(const AttnParams p) {
  constexpr int KS = D / 16;
  constexpr int NQ = SPLIT ? 2 : 1;
  constexpr int TILE = 4096 / D, GP = TILE / kGroup, WIN = 32 / GP;     // WIN: tiles of 32 groups
  constexpr int SG = kStageTiles * GP;                                  // groups of a stage
  constexpr int S = kStages, kStageBytes = kStageTiles * kTileBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  const Pages& pg = p.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // the first warps of all CTAs, then their second ones: few shares spread over the GPU
  const int gw = warp * gridDim.x + blockIdx.x;
  uint8_t* ring = smem + warp * kWarpSmem;
  uint8_t* scales = ring + S * kStageBytes;
  const uint32_t ring_addr = shared_addr(ring);
  const uint32_t bars = shared_addr(smem + kWarps * kWarpSmem) + warp * (S * 8);

  // The lengths say which pages and queries a warp needs; meanwhile (and while
  // the kernel in front finishes) they, the table and the queries come to L2, as
  // far as the grid's threads reach.
  prefetch_part(p.lens, 4LL * pg.B);
  prefetch_part(pg.table, 4LL * pg.B * pg.table_pages);
  prefetch_part(p.q, static_cast<long long>(pg.B) * p.T_ * p.Hq * D * sizeof(T));
  pdl_wait();
  pdl_launch_dependents();             // the combine kernel's CTAs come as this one's leave
  Cursor c{};                          // the tile being worked on
  int gap;
  int left = begin_of<D>(p, gw, c, &gap);      // units of the share that are still to be worked on
  if (left <= 0) return;
  if (lane < S) bar_init(bars + 8 * lane);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();

  Cursor in = c;                       // the next tile to load

  // Pages of the 32 groups of the loading cursor's window, one a lane.
  int page = -1;
  bool window = true;                  // to be loaded
  uint32_t have = 0;                   // SG bits a stage: which groups were loaded
  int to_load = left;                  // ... to be asked for
  int next_len = 0;                    // of the sequence that was loaded from last
  // The tiles that a stage takes at a place: two of one pair, from an even one on.
  auto step_of = [&](const Cursor& x, int units) {
    return (x.tile & 1) ? 1 : min(min(kStageTiles, units), x.tiles - x.tile);
  };
  auto issue = [&](int st) {
    const int n = step_of(in, to_load);
    next_len = in.len;
    const int tok = in.tile * TILE + lane * kGroup;
    if (window || in.tile % WIN == 0) {
      window = false;
      const int first = tok - in.tile % WIN * TILE;
      page = -1;
      if (first < in.len) {
        page = pg.table[static_cast<long long>(in.b) * pg.table_pages + (first >> pg.page_log2)];
        if (page < 0 || page >= pg.num_pages) {
          page = -1;
          record_status(kStatusBadIndex);
        }
      }
    }
    // lane q: group q of the stage
    const int pid = __shfl_sync(0xFFFFFFFFu, page, in.tile % WIN * GP + lane);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, lane < n * GP && pid >= 0);
    const int at = (in.h << (pg.page_log2 - 4)) + ((tok & ((1 << pg.page_log2) - 1)) / kGroup);   // group of the page
    const uint8_t* src = pg.cache + static_cast<long long>(pid) * p.page_bytes + at * Block<D>::kBytes;
    const uint32_t bar = bars + 8 * st;
    if (lane == 0) bar_expect(bar, __popc(mask) * Block<D>::kBytes);
    // what lies in one page is one piece (its groups below the sequence's end)
    const uint32_t piece = (mask >> lane) & p.piece_mask;
    if (piece && (lane & p.piece_low) == 0)
      bulk_load(ring_addr + st * kStageBytes + lane * Block<D>::kBytes, src, __popc(piece) * Block<D>::kBytes, bar);
    have = (have & ~(((1u << SG) - 1) << (SG * st))) | mask << (SG * st);
    window = advance<D>(p, in, n, [&](int b) { return len_of(p, b, false); });
    to_load = window ? pair_left(p, in, to_load, n + gap) : to_load - n;
  };
  // The queries of a pair, as they lie there: column g's values 16 b + 4 t .. + 3.
  Four<T> raw[NT][KS];
  int nq = 0, kexp = 0, vexp = 0;      // query tokens of the sequence; the head's exponents
  auto fetch = [&]() {
    const int row0 = c.rt * (8 * NT);
    nq = rows_of(p.count, c.b, p.T_, c.h == 0 && row0 == 0);
    kexp = head_exp(pg.k_exp, c.h);
    vexp = head_exp(pg.v_exp, c.h);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + 8 * n + g, tok = r * p.group_inv >> 16;
      const T* qr = static_cast<const T*>(p.q) +
                    ((static_cast<long long>(c.b) * p.T_ + tok) * p.Hq + c.h * p.G + r - tok * p.G) * D + 4 * t;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        if (tok < p.T_)                // rows from nq G on are not written, whatever they are
          raw[n][ks].load(qr + 16 * ks);
        else
          raw[n][ks].zero();
    }
  };
  uint32_t qb[NQ][NT][KS][2];
  float f[NT][2];
  int lim[NT][2];
  float low[NT][2], l[NT][2], o[NT][KS][4];    // low: less the largest score
  // where registers allow, the first queries are on their way while the first pages are looked up
  constexpr bool kEarly = !SPLIT;
  if (kEarly) fetch();
  issue(0);
  bool fresh = true;
  int st = 0, lim_min = 0;
  uint32_t parity = 0;

  for (int i = 0; left > 0;) {         // i: tiles done
    const int n = step_of(c, left);
    if (to_load > 0) issue(st ^ 1);
    if (fresh) {
      // B fragments of Q (column g of n-tile n), and per accumulator column its factor and its last token
      if (!kEarly || i > 0) fetch();
      fresh = false;
      lim_min = c.len;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = c.rt * (8 * NT) + 8 * n + g;
        float am = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) am = fmaxf(am, raw[n][ks].top_abs());
        am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        // the row's largest value to 2^14 .. 2^15; zeros, infinities as they are
        const int xe = static_cast<int>(__float_as_uint(am) >> 23);
        const int ex = xe == 0 || xe == 255 ? 0 : xe - 127 - 14;       // -140 .. 113
        const int exa = max(-100, min(100, -ex));
        const float down0 = pow2i(exa), down1 = pow2i(-ex - exa);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          float x[4];
          raw[n][ks].values(x);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float u = x[2 * e] * down0 * down1, v = x[2 * e + 1] * down0 * down1;
            qb[0][n][ks][e] = pack_f16(u, v);
            if (SPLIT) {
              const float2 hi = f16x2_f32(qb[0][n][ks][e]);
              qb[NQ - 1][n][ks][e] = pack_f16(u - hi.x, v - hi.y);
            }
          }
        }
        // scale * log2(e) * 2^(row + head), in two steps so that each stays finite
        const int e2 = ex + kexp;                                      // -204 .. 177
        const int e2a = max(-100, min(100, e2));
        // kept normal and finite: a masked -infinity times it stays one
        const float fac = fminf(fmaxf(p.scale_log2 * pow2i(e2a) * pow2i(e2 - e2a), 1.2e-38f), 3e38f);
        // columns that are none see all, and are not written
        const int limit = r < nq * p.G ? c.len - (nq - 1 - (r * p.group_inv >> 16)) : 0x7FFFFFFF;
        lim_min = min(lim_min, limit);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[n][e] = __shfl_sync(0xFFFFFFFFu, fac, (2 * t + e) * 4);
          lim[n][e] = min(c.len, __shfl_sync(0xFFFFFFFFu, limit, (2 * t + e) * 4));
          low[n][e] = kNone;
          l[n][e] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.0f;
      }
      lim_min = __reduce_min_sync(0xFFFFFFFFu, lim_min);
    }
    if (!bar_wait(bars + 8 * st, parity >> st & 1)) {
      // lost: tell, and leave when the copies in flight have come (or again do not)
      record_status(kStatusTimeout);
      bar_wait(bars + 8 * st, parity >> st & 1);
      if (to_load < left - n - (c.tile + n == c.tiles ? gap : 0)) bar_wait(bars + 8 * (st ^ 1), parity >> (st ^ 1) & 1);
      return;
    }
    parity ^= 1u << st;

    const uint32_t mask = have >> (SG * st) & ((1u << SG) - 1);
    const uint8_t* stage = ring + st * kStageBytes;
    // The parts of a tile's work.  S^T of a group (entries 0, 1: token g, columns
    // 2t, 2t + 1; entries 2, 3: token g + 8); sl: the scales of tokens g and
    // g + 8, two blocks each.
    auto scores = [&](float (&s)[NT][4], const uint8_t* grp, const uint32_t (&sl)[2][KS / 2]) {
      float part[NT][4];
#pragma unroll
      for (int k = 0; k < KS / 4; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(grp + Block<D>::kK + k * 512 + lane * 16);
        const uint32_t kc[2][2] = {{v.x, v.z}, {v.y, v.w}};      // [two blocks][token g, g + 8]
#pragma unroll
        for (int bp = 0; bp < 2; ++bp) {               // blocks 4k + 2 bp, + 1
          uint32_t x0[4], x1[4];
          e2m1x8_f16x2(kc[bp][0], x0);
          e2m1x8_f16x2(kc[bp][1], x1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int kb = 4 * k + 2 * bp + e;
            const uint32_t s0 = sl[0][2 * k + bp], s1 = sl[1][2 * k + bp];
            const uint32_t a0 = mul_f16x2_half(x0[2 * e], s0, e), a1 = mul_f16x2_half(x1[2 * e], s1, e);
            const uint32_t a2 = mul_f16x2_half(x0[2 * e + 1], s0, e), a3 = mul_f16x2_half(x1[2 * e + 1], s1, e);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (SPLIT) {
                // two blocks' products, then added in f32: the tensor cores' own sums
                // cut what f32 rounds, and over many tokens that shows
                float (&d)[4] = part[n];
                if (kb % 2 == 0)
                  mma16816_f16_zero(d, a0, a1, a2, a3, qb[NQ - 1][n][kb][0], qb[NQ - 1][n][kb][1]);
                else
                  mma16816_f16(d, a0, a1, a2, a3, qb[NQ - 1][n][kb][0], qb[NQ - 1][n][kb][1]);
                mma16816_f16(d, a0, a1, a2, a3, qb[0][n][kb][0], qb[0][n][kb][1]);
                if (kb == 1) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) s[n][i] = d[i];
                } else if (kb % 2 == 1) {
                  const float2 u = add2(make_float2(s[n][0], s[n][1]), make_float2(d[0], d[1]));
                  const float2 v = add2(make_float2(s[n][2], s[n][3]), make_float2(d[2], d[3]));
                  s[n][0] = u.x; s[n][1] = u.y; s[n][2] = v.x; s[n][3] = v.y;
                }
              } else if (kb == 0) {
                mma16816_f16_zero(s[n], a0, a1, a2, a3, qb[0][n][kb][0], qb[0][n][kb][1]);
              } else {
                mma16816_f16(s[n], a0, a1, a2, a3, qb[0][n][kb][0], qb[0][n][kb][1]);
              }
            }
          }
        }
      }
    };
    // Online softmax per column: p = 2^(f (s + low) + kPShift), f > 0, low = less the
    // largest s so far; mx: a lane's largest s.  Most tiles hold no larger one.
    auto raise = [&](const float (&mx)[NT][2]) {
      bool grown = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) grown |= mx[n][e] > -low[n][e];
      if (!__any_sync(0xFFFFFFFFu, grown)) return;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float corr[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = mx[n][e];
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
          const float to = fminf(low[n][e], -x);
          corr[e] = ex2_approx((to - low[n][e]) * f[n][e]);        // from kNone: of zeros
          low[n][e] = to;
          l[n][e] *= corr[e];
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const float2 u = mul2(make_float2(o[n][k][0], o[n][k][1]), make_float2(corr[0], corr[1]));
          const float2 v = mul2(make_float2(o[n][k][2], o[n][k][3]), make_float2(corr[0], corr[1]));
          o[n][k][0] = u.x; o[n][k][1] = u.y; o[n][k][2] = v.x; o[n][k][3] = v.y;
        }
      }
    };
    // P of a group as B fragments, and into the rows' sums.
    auto probabilities = [&](const float (&s)[NT][4], uint32_t (&pb)[NQ][NT][2]) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 fn = make_float2(f[n][0], f[n][1]), low2 = make_float2(low[n][0], low[n][1]);
        const float2 shift = make_float2(kPShift, kPShift);
        const float2 u = fma2(add2(make_float2(s[n][0], s[n][1]), low2), fn, shift);
        const float2 v = fma2(add2(make_float2(s[n][2], s[n][3]), low2), fn, shift);
        const float2 pu = make_float2(ex2_approx(u.x), ex2_approx(u.y)), pv = make_float2(ex2_approx(v.x), ex2_approx(v.y));
        const float2 ln = add2(make_float2(l[n][0], l[n][1]), add2(pu, pv));
        l[n][0] = ln.x;
        l[n][1] = ln.y;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 pe = e ? pv : pu;
          const uint32_t hi = pack_f16(pe.x, pe.y);
          pb[0][n][e] = movmatrix_trans(hi);
          if (SPLIT) {
            const float2 h2 = f16x2_f32(hi);
            pb[NQ - 1][n][e] = movmatrix_trans(pack_f16(pe.x - h2.x, pe.y - h2.y));
          }
        }
      }
    };
    // O^T += V^T P^T of blocks 4k .. 4k + 3 of a group; lo, hi: the scales of its
    // tokens 2t, 2t + 1 and 2t + 8, 2t + 9.
    auto outputs = [&](int k, const uint8_t* grp, const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                       const uint32_t (&pb)[NQ][NT][2]) {
      const uint4 v = *reinterpret_cast<const uint4*>(grp + Block<D>::kV + k * 512 + lane * 16);
      uint32_t x0[4], x1[4], x2[4], x3[4];
      e2m1x8_f16x2(v.x, x0);           // values 2g, tokens 2t, 2t + 1
      e2m1x8_f16x2(v.y, x1);           // values 2g + 1
      e2m1x8_f16x2(v.z, x2);           // values 2g, tokens 2t + 8, 2t + 9
      e2m1x8_f16x2(v.w, x3);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a0 = mul_f16x2(x0[e], lo[e]), a1 = mul_f16x2(x1[e], lo[e]);
        const uint32_t a2 = mul_f16x2(x2[e], hi[e]), a3 = mul_f16x2(x3[e], hi[e]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float (&acc)[4] = o[n][4 * k + e];
          if (SPLIT) {
            float d[4];
            mma16816_f16_zero(d, a0, a1, a2, a3, pb[NQ - 1][n][0], pb[NQ - 1][n][1]);
            mma16816_f16(d, a0, a1, a2, a3, pb[0][n][0], pb[0][n][1]);
            const float2 u = add2(make_float2(acc[0], acc[1]), make_float2(d[0], d[1]));
            const float2 v = add2(make_float2(acc[2], acc[3]), make_float2(d[2], d[3]));
            acc[0] = u.x; acc[1] = u.y; acc[2] = v.x; acc[3] = v.y;
          } else {
            mma16816_f16(acc, a0, a1, a2, a3, pb[0][n][0], pb[0][n][1]);
          }
        }
      }
    };
    // A tile that every column sees all of.  (f32 at head size 128 would spill
    // here, and takes all tiles by groups: 16 x 4096 tokens, 128 heads on 8, 50 us, 64 us so.)
    constexpr bool kWhole = !(SPLIT && D == 128);
    auto whole_tile = [&](const uint8_t* base) {
      // Its scales, 8 of K or V (`first`) converted a lane: every lane needs 1/4
      // (K) or 1/8 (V) of them, which they would convert 8 and 4 times over.
      auto stage_scales = [&](int first) {
        const uint2 v = *reinterpret_cast<const uint2*>(base + lane * 8 / D * Block<D>::kBytes + first + lane * 8 % D);
        uint4 h;
        e4m3x4_f16x2(v.x, h.x, h.y);
        e4m3x4_f16x2(v.y, h.z, h.w);
        __syncwarp();
        *reinterpret_cast<uint4*>(scales + lane * 16) = h;
        __syncwarp();
      };
      stage_scales(Block<D>::kKs);
      float s[GP][NT][4], mx[NT][2];
#pragma unroll
      for (int q = 0; q < GP; ++q) {
        uint32_t sl[2][KS / 2];
#pragma unroll
        for (int k = 0; k < KS / 4; ++k) {
          const uint4 u = *reinterpret_cast<const uint4*>(scales + (q * D + g * (2 * KS)) * 2 + k * 16);
          if (KS == 4) {
            sl[0][0] = u.x; sl[0][1] = u.y; sl[1][0] = u.z; sl[1][1] = u.w;
          } else {
            sl[k][0] = u.x; sl[k][1] = u.y; sl[k][KS / 2 - 2] = u.z; sl[k][KS / 2 - 1] = u.w;
          }
        }
        scores(s[q], base + q * Block<D>::kBytes, sl);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[n][e] = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
          for (int q = 1; q < GP; ++q) mx[n][e] = fmaxf(mx[n][e], fmaxf(s[q][n][e], s[q][n][e + 2]));
        }
      raise(mx);
      stage_scales(Block<D>::kVs);
#pragma unroll
      for (int q = 0; q < GP; ++q) {
        uint32_t pb[NQ][NT][2];
        probabilities(s[q], pb);
#pragma unroll
        for (int k = 0; k < KS / 4; ++k) {
          const uint4* sv = reinterpret_cast<const uint4*>(scales + (q * D + t * (4 * KS) + k * 16) * 2);
          const uint4 u = sv[0], v = sv[1];
          const uint32_t lo[4] = {u.x, u.z, v.x, v.z}, hi[4] = {u.y, u.w, v.y, v.w};
          outputs(k, base + q * Block<D>::kBytes, lo, hi, pb);
        }
      }
    };
    // A group of a tile that columns see different parts of, or that is not all
    // there.  Few tiles are: short code, a group at a time, counts for more than
    // its speed (twice the code here cost calls of 12 to 33 us 3.5 us each).
    auto edge_group = [&](int tok, const uint8_t* grp) {
      uint32_t sl[2][KS / 2];
      if (KS == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(grp + Block<D>::kKs + g * 8);
        e4m3x4_f16x2(u.x, sl[0][0], sl[0][1]);
        e4m3x4_f16x2(u.y, sl[1][0], sl[1][1]);
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(grp + Block<D>::kKs + g * 16);
        e4m3x4_f16x2(u.x, sl[0][0], sl[0][1]);
        e4m3x4_f16x2(u.y, sl[0][KS / 2 - 2], sl[0][KS / 2 - 1]);
        e4m3x4_f16x2(u.z, sl[1][0], sl[1][1]);
        e4m3x4_f16x2(u.w, sl[1][KS / 2 - 2], sl[1][KS / 2 - 1]);
      }
      float s[NT][4], mx[NT][2];
      scores(s, grp, sl);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (tok + g >= lim[n][e]) s[n][e] = -INFINITY;
          if (tok + g + 8 >= lim[n][e]) s[n][e + 2] = -INFINITY;
          mx[n][e] = fmaxf(s[n][e], s[n][e + 2]);
        }
      raise(mx);
      uint32_t pb[NQ][NT][2];
      probabilities(s, pb);
      // The scales of tokens that are not the sequence's are blanked, whose P is 0
      // (0 x NaN is not).  A block of NaN reaches only the columns that see its
      // token: its scale is blanked too, and these columns are set to NaN after.
      uint32_t keep = 0, w[KS], nan = 0, bad[KS / 4];    // bad: per block the first such token of the group, a byte each
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (tok + 2 * t + (e & 1) + 8 * (e >> 1) < c.len) keep |= 0xFFu << (8 * e);
#pragma unroll
      for (int k = 0; k < KS / 4; ++k) {
        const uint4 u = *reinterpret_cast<const uint4*>(grp + Block<D>::kVs + t * (4 * KS) + 16 * k);
        w[4 * k] = u.x & keep; w[4 * k + 1] = u.y & keep; w[4 * k + 2] = u.z & keep; w[4 * k + 3] = u.w & keep;
#pragma unroll
        for (int e = 0; e < 4; ++e) nan |= __vcmpeq4(w[4 * k + e], 0x7F7F7F7Fu);
      }
      const bool any_nan = __any_sync(0xFFFFFFFFu, nan != 0);
      if (any_nan) {
#pragma unroll
        for (int k = 0; k < KS / 4; ++k) {
          bad[k] = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t is = __vcmpeq4(w[4 * k + e], 0x7F7F7F7Fu);
            w[4 * k + e] &= ~is;
            const int first = is & 0xFFu ? 2 * t : is & 0xFF00u ? 2 * t + 1 : is & 0xFF0000u ? 2 * t + 8 : is ? 2 * t + 9 : 0xFF;
            bad[k] |= static_cast<uint32_t>(first) << (8 * e);
          }
          bad[k] = __vminu4(bad[k], __shfl_xor_sync(0xFFFFFFFFu, bad[k], 1));
          bad[k] = __vminu4(bad[k], __shfl_xor_sync(0xFFFFFFFFu, bad[k], 2));
        }
      }
#pragma unroll
      for (int k = 0; k < KS / 4; ++k) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) e4m3x4_f16x2(w[4 * k + e], lo[e], hi[e]);
        outputs(k, grp, lo, hi, pb);
      }
      if (any_nan) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int first = bad[k / 4] >> (8 * (k % 4)) & 0xFF;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (first < 16 && tok + first < lim[n][e & 1]) o[n][k][e] = __int_as_float(0x7FC00000);
        }
      }
    };
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      const int tok0 = (c.tile + k) * TILE;
      const uint32_t here = mask >> (GP * k) & ((1u << GP) - 1);
      if (kWhole && here == (1u << GP) - 1 && tok0 + TILE <= lim_min) {
        whole_tile(stage + k * kTileBytes);
      } else {
#pragma unroll 1
        for (int q = 0; q < GP; ++q)
          if (here >> q & 1) edge_group(tok0 + q * kGroup, stage + k * kTileBytes + q * Block<D>::kBytes);
      }
    }
    __syncwarp();                      // the stage is read; the next iteration's copies may refill it
    st ^= 1;

    if (c.tile + n == c.tiles || left == n) {
      // the pair, or this warp's share of it, is done
      const int h = c.h, row0 = c.rt * (8 * NT);
      const float ve = pow2i(vexp);
      const bool from_start = i >= c.tile;                     // the pair's first tile is in this share
      const bool done = from_start && c.tile + n == c.tiles;
      // the share's first pair leaves its part in slot 0, its last one in slot 1
      const long long slot = static_cast<long long>(gw) * 2 + (i == c.tile || !from_start ? 0 : 1);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float ls = l[n][e];
          ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 4);
          ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 8);
          ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 16);
          const int col = 8 * n + 2 * t + e, r = row0 + col;
          if (r < nq * p.G) {
            if (done) {
              const float inv = ls == 0.0f ? 0.0f : ve / ls;
              const int tok = r * p.group_inv >> 16;
              T* dst = static_cast<T*>(p.out) +
                       ((static_cast<long long>(c.b) * p.T_ + tok) * p.Hq + h * p.G + r - tok * p.G) * D;
#pragma unroll
              for (int k = 0; k < KS; ++k) store2(dst + 16 * k + 2 * g, o[n][k][e] * inv, o[n][k][e + 2] * inv);
            } else {
              float* dst = p.o_part + (slot * p.cols + col) * D;
#pragma unroll
              for (int k = 0; k < KS; ++k) store2(dst + 16 * k + 2 * g, o[n][k][e], o[n][k][e + 2]);
              if (g == 0)
                *reinterpret_cast<float4*>(p.ml_part + (slot * p.cols + col) * 4) = make_float4(-low[n][e], ls, f[n][e], 0.0f);
            }
          }
        }
      fresh = true;
    }
    left = advance<D>(p, c, n, [&](int) { return next_len; }) ? pair_left(p, c, left, n + gap) : left - n;
    i += n;
  }
}

// A running sum of parts of one row: values relative to 2^(f m), f the row's
// factor, and what they are to be divided by.
template <int V>
struct RowSum {
  float m = -kNone, den = 0.0f, num[V] = {};
  __device__ __forceinline__ void add(float f, float m2, float den2, const float (&x)[V]) {
    const float d = (m2 - m) * f, c = ex2_approx(fminf(-d, 0.0f)), c2 = ex2_approx(fminf(d, 0.0f));
    m = fmaxf(m, m2);
    den = den * c + den2 * c2;
#pragma unroll
    for (int v = 0; v < V; ++v) num[v] = num[v] * c + x[v] * c2;
  }
};

// Rows whose pair was shared by several warps, from their parts in the line's
// order.  Grid y: sequences.  A few us, nearly all of it latency (its launch
// overlaps the attention's end, its lengths are read before that), for batches of
// up to some hundreds: every warp sums the lengths of all sequences, which grows
// with the batch squared (100 tokens of one head, with the attention: 256
// sequences 9.4 us, 1024 28 us, 4096 110 us, 65535 15 ms).
//   COLS > 0: WARPS warps (each every WARPS-th part) for COLS columns of a pair,
//   D / 32 values a lane.
//   COLS = 0: a CTA for 32 values of a row; 8 lanes take 4 values each, 32 of
//   them every 32nd part, and then their sums are added in order.
template <typename T, int D, int NT, int COLS, int WARPS = 1>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const AttnParams p) {
  constexpr bool MANY = COLS == 0;
  constexpr int kCols = MANY ? 1 : COLS;
  constexpr int V = MANY ? 4 : D / 32, SLICES = D / 32;
  const Pages& pg = p.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  // the pair, its first column here, and the lane's first value
  const unsigned u = MANY ? blockIdx.x / SLICES : blockIdx.x * (8 / WARPS) + warp / WARPS;
  const unsigned per = (p.cols + kCols - 1) / kCols;
  const int pair = u / per, col0 = (u - pair * per) * kCols;
  const int at = MANY ? blockIdx.x % SLICES * 32 + (threadIdx.x & 7) * 4 : lane * V;
  const int h = p.row_tiles == 1 ? pair : pair / p.row_tiles, rt = pair - h * p.row_tiles;
  const bool in = h < pg.Hkv;
  int before;
  const Line line = line_of<D>(p, b, &before);
  const int tiles = tiles_of<D>(len_of<true>(p, b, false));
  const int a = before + (in ? pair : 0) * (tiles + line.gap);
  const int w0 = min(line.shares - 1, line.share_of(a + line.gap));
  const int w1 = min(line.shares - 1, line.share_of(a + line.gap + tiles - 1));
  const int first = line.begin(w0) >= a ? 0 : 1;       // whether the share begins with this pair
  const int rows = rows_of<true>(p.count, b, p.T_, false) * p.G;       // real ones of a KV head
  const float ve = pow2i(head_exp<true>(pg.v_exp, in ? h : 0));
  // what was read so far no kernel of this call writes; every thread waits, so
  // that this kernel does not end before the one whose parts it reads
  pdl_wait();
  if (!in || w0 == w1) return;         // w0 == w1: finished by that warp
  // row r of the KV head: where it goes
  auto store = [&](const RowSum<V>& sum, int r) {
    const float inv = sum.den == 0.0f ? 0.0f : ve / sum.den;
    const int tok = r * p.group_inv >> 16;
    T* dst = static_cast<T*>(p.out) + ((static_cast<long long>(b) * p.T_ + tok) * p.Hq + h * p.G + r - tok * p.G) * D + at;
#pragma unroll
    for (int v = 0; v < V; v += 2) store2(dst + v, sum.num[v] * inv, sum.num[v + 1] * inv);
  };
  const int r0 = rt * (8 * NT) + col0;
  auto part_of = [&](long long k) { return *reinterpret_cast<const float2*>(p.ml_part + k * 4); };
  auto factor_of = [&](long long k) { return p.ml_part[k * 4 + 2]; };
  if (!MANY) {
    RowSum<V> sum[kCols];
    float f[kCols] = {};
#pragma unroll kCols == 1 ? 4 : 2
    for (int w = w0 + warp % WARPS; w <= w1; w += WARPS) {
      const long long k = (static_cast<long long>(w) * 2 + (w == w0 ? first : 0)) * p.cols + col0;
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        if (r0 + c < rows && col0 + c < p.cols) {
          const float2 ml = part_of(k + c);
          f[c] = factor_of(k + c);
          float x[V];
#pragma unroll
          for (int v = 0; v < V; v += 2) load2(p.o_part + (k + c) * D + at + v, x + v);
          sum[c].add(f[c], ml.x, ml.y, x);
        }
    }
    if constexpr (WARPS > 1) {
      static_assert(WARPS == 1 || COLS == 1, "several warps take one row");
      __shared__ float part[8][32][V + 2];
      float* mine = part[warp][lane];
      mine[V] = sum[0].m;
      mine[V + 1] = sum[0].den;
#pragma unroll
      for (int v = 0; v < V; ++v) mine[v] = sum[0].num[v];
      // the row's warps, which left or stayed together
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / WARPS), "n"(WARPS * 32) : "memory");
      if (warp % WARPS != 0) return;
#pragma unroll
      for (int k = 1; k < WARPS; ++k) {
        const float* other = part[warp + k][lane];
        float x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = other[v];
        sum[0].add(f[0], other[V], other[V + 1], x);
      }
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      if (r0 + c < rows && col0 + c < p.cols) store(sum[c], r0 + c);
    return;
  }
  if (r0 >= rows) return;              // the whole CTA's
  RowSum<V> sum;
  const float f = factor_of((static_cast<long long>(w0) * 2 + first) * p.cols + col0);
#pragma unroll 4
  for (int w = w0 + (threadIdx.x >> 3); w <= w1; w += 32) {
    const long long k = (static_cast<long long>(w) * 2 + (w == w0 ? first : 0)) * p.cols + col0;
    const float2 ml = part_of(k);
    float x[V];
#pragma unroll
    for (int v = 0; v < V; v += 2) load2(p.o_part + k * D + at + v, x + v);
    sum.add(f, ml.x, ml.y, x);
  }
  // the four of a warp, then the warps
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = __shfl_xor_sync(0xFFFFFFFFu, sum.num[v], o);
    sum.add(f, __shfl_xor_sync(0xFFFFFFFFu, sum.m, o), __shfl_xor_sync(0xFFFFFFFFu, sum.den, o), x);
  }
  __shared__ float sh[8][8][V + 2];
  if (lane < 8) {
    float* mine = sh[warp][lane];
    mine[V] = sum.m;
    mine[V + 1] = sum.den;
#pragma unroll
    for (int v = 0; v < V; ++v) mine[v] = sum.num[v];
  }
  __syncthreads();
  if (threadIdx.x >= 8) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    const float* other = sh[k][lane];
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = other[v];
    sum.add(f, other[V], other[V + 1], x);
  }
  store(sum, r0);
}

}  // namespace kv4
}  // namespace sambay
