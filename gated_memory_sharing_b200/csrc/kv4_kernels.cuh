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
//   V codes, 8 D bytes: per 64 values 32 lanes x 16 bytes; lane (g, t): tokens
//     2t, 2t + 1, 2t + 8, 2t + 9 (4 bytes each), one byte per block b: values
//     16 b + 2 g, + 1
//   K scales, D bytes: [g][token g, token g + 8][block]
//   V scales, D bytes: [t][block][tokens 2t, 2t + 1, 2t + 8, 2t + 9]
#pragma once

#include <cuda_fp16.h>

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

__device__ __forceinline__ int head_exp(const int32_t* e, int h) {
  return e ? max(-kMaxExp, min(kMaxExp, e[h])) : 0;
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

// ---------------------------------------------------------------- quantising

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const uint32_t m = code & 7u, e = code >> 3;                 // no sign
  return e == 0 ? static_cast<float>(m) * 0.001953125f : __uint_as_float(((e + 120u) << 23) | (m << 20));
}

// e4m3 code of amax / 6, to nearest even, at most 448 (code 126).  The
// conversion of the rounded quotient is off by one code at most; comparing
// amax with 6 times the border on either side, exact in f32, settles it.
__device__ __forceinline__ uint32_t block_scale(float amax) {
  const float y = fminf(amax * 0.16666667f, 448.0f);
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(y));
  uint32_t c = two & 0x7Fu;
  const float v = e4m3_value(c);
  const float up = 3.0f * (v + e4m3_value(c + 1)), down = c > 0 ? 3.0f * (v + e4m3_value(c - 1)) : -1.0f;
  if (c < 126 && (amax > up || (amax == up && (c & 1u)))) return c + 1;
  if (amax < down || (amax == down && (c & 1u))) return c - 1;
  return c;
}

// e2m1 code of x / s, to nearest even, saturating: the borders that |x|
// passes, each exact in f32 (at most 7 bits).
__device__ __forceinline__ uint32_t e2m1_code(float x, float s) {
  const float a = fabsf(x);
  uint32_t c = 0;
  c += a > 0.25f * s;
  c += a >= 0.75f * s;
  c += a > 1.25f * s;
  c += a >= 1.75f * s;
  c += a > 2.5f * s;
  c += a >= 3.5f * s;
  c += a > 5.0f * s;
  return s > 0.0f ? c | (x < 0.0f ? 8u : 0u) : 0u;             // also 0 where s is NaN
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale's code for a block whose largest |x| has the bits `m` (of a NaN or
// an infinity if it holds one); *s receives the scale.
__device__ __forceinline__ uint32_t scale_of(uint32_t m, float inv, float* s) {
  if (m >= 0x7F800000u) {
    *s = __int_as_float(0x7FC00000);
    return 0x7Fu;
  }
  const uint32_t c = block_scale(__uint_as_float(m) * inv);
  *s = e4m3_value(c);
  return c;
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

template <typename T>
struct RowParams {
  Pages pg;
  const T* K;              // write: rows, [B, T] tokens at k_stride elements
  const T* V;
  T* Ko;                   // read: rows [B, T, Hkv, D]
  T* Vo;
  const int32_t* pos;      // [B] cached tokens before the call's
  const int32_t* count;    // [B] rows of each sequence, or null (T)
  int T_;
  long long k_stride, v_stride;
};

// Rows of sequence b: min(count, T) of them; a count outside 0 .. T is recorded.
__device__ __forceinline__ int rows_of(const int32_t* count, int b, int T, bool tell) {
  if (!count) return T;
  const int n = count[b];
  if ((n < 0 || n > T) && tell) record_status(kStatusBadIndex);
  return max(0, min(T, n));
}

// One row of one head per 8 threads.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_write_kernel(const RowParams<T> p) {
  const Pages& pg = p.pg;
  const long long unit = (blockIdx.x * 256LL + threadIdx.x) >> 3;
  const int j = threadIdx.x & 7;
  const long long units = static_cast<long long>(pg.B) * p.T_ * pg.Hkv;
  const bool in = unit < units;
  const int h = in ? static_cast<int>(unit % pg.Hkv) : 0;
  const long long row = in ? unit / pg.Hkv : 0;
  const int b = static_cast<int>(row / p.T_), tok = static_cast<int>(row % p.T_);
  const bool live = in && tok < rows_of(p.count, b, p.T_, h == 0 && tok == 0 && j == 0);
  const int pos = static_cast<int>(static_cast<unsigned>(p.pos[b]) + tok);   // a wrapped sum is refused below
  uint8_t* grp = live ? group_of<D>(pg, b, h, pos) : nullptr;
  if (live && !grp && j == 0) record_status(kStatusBadIndex);
  const int r = pos & 15, g = r & 7;
  const T* kr = p.K + row * p.k_stride + h * D;
  const T* vr = p.V + row * p.v_stride + h * D;
  // every lane takes part in the shuffles; only lanes with a group load and store
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    // K: thread (t = j % 4, half of the blocks): blocks 4c + 2 (j / 4), + 1
    const float kinv = pow2i(-head_exp(pg.k_exp, h));
    const int t = j & 3, b0 = 4 * c + 2 * (j >> 2);
    uint32_t word = 0, sc = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (grp) {
        load2(kr + 16 * (b0 + i) + 4 * t, x);
        load2(kr + 16 * (b0 + i) + 4 * t + 2, x + 2);
      }
      uint32_t m = max(max(abs_bits(x[0]), abs_bits(x[1])), max(abs_bits(x[2]), abs_bits(x[3])));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      float s;
      sc |= scale_of(m, kinv, &s) << (8 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) word |= e2m1_code(x[e] * kinv, s) << (16 * i + 4 * e);
    }
    if (grp) {
      *reinterpret_cast<uint32_t*>(grp + Block<D>::kK + c * 512 + (g * 4 + t) * 16 + (r >> 3) * 8 + (j >> 2) * 4) = word;
      if (t == 0)
        *reinterpret_cast<uint16_t*>(grp + Block<D>::kKs + g * (D / 8) + (r >> 3) * (D / 16) + b0) =
            static_cast<uint16_t>(sc);
    }
    // V: thread j holds values 16 b + 2 j, + 1 of blocks b = 4c .. 4c + 3
    const float vinv = pow2i(-head_exp(pg.v_exp, h));
    const int tv = g >> 1, w = (r & 1) + 2 * (r >> 3);
    word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[2] = {0.f, 0.f};
      if (grp) load2(vr + 16 * (4 * c + i) + 2 * j, x);
      uint32_t m = max(abs_bits(x[0]), abs_bits(x[1]));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
      float s;
      const uint32_t code = scale_of(m, vinv, &s);
      word |= (e2m1_code(x[0] * vinv, s) | e2m1_code(x[1] * vinv, s) << 4) << (8 * i);
      if (grp && j == i) grp[Block<D>::kVs + tv * (D / 4) + (4 * c + i) * 4 + w] = static_cast<uint8_t>(code);
    }
    if (grp) *reinterpret_cast<uint32_t*>(grp + Block<D>::kV + c * 512 + (j * 4 + tv) * 16 + w * 4) = word;
  }
}

// ---------------------------------------------------------------- reading back

// Two 4-bit values of a byte (the lower nibble in the lower half).
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t byte) {
  uint32_t d;
  asm("{\n\t.reg .b8 p;\n\tcvt.u8.u32 p, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, p;\n\t}" : "=r"(d) : "r"(byte));
  return d;
}
// The four bytes of a word.
__device__ __forceinline__ void e2m1x8_f16x2(uint32_t w, uint32_t (&d)[4]) {
  asm("{\n\t.reg .b8 p, q, r, s;\n\tmov.b32 {p, q, r, s}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\tcvt.rn.f16x2.e2m1x2 %1, q;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, r;\n\tcvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w));
}
// Four e4m3 scales as f16 pairs (exact).
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
__device__ __forceinline__ float e4m3_or_nan(uint32_t code) {
  return (code & 0x7Fu) == 0x7Fu ? __int_as_float(0x7FC00000) : e4m3_value(code & 0x7Fu);
}

// One row of one head per 8 threads, as kv4_write_kernel lays them out.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const RowParams<T> p) {
  const Pages& pg = p.pg;
  const long long unit = (blockIdx.x * 256LL + threadIdx.x) >> 3;
  const int j = threadIdx.x & 7;
  if (unit >= static_cast<long long>(pg.B) * p.T_ * pg.Hkv) return;
  const int h = static_cast<int>(unit % pg.Hkv);
  const long long row = unit / pg.Hkv;
  const int b = static_cast<int>(row / p.T_), tok = static_cast<int>(row % p.T_);
  if (tok >= rows_of(p.count, b, p.T_, h == 0 && tok == 0 && j == 0)) return;
  const int pos = static_cast<int>(static_cast<unsigned>(p.pos[b]) + tok);   // a wrapped sum is refused below
  const uint8_t* grp = group_of<D>(pg, b, h, pos);
  if (!grp) {
    if (j == 0) record_status(kStatusBadIndex);
    return;
  }
  const int r = pos & 15, g = r & 7;
  T* kr = p.Ko + unit * D;
  T* vr = p.Vo + unit * D;
  const float ke = pow2i(head_exp(pg.k_exp, h)), ve = pow2i(head_exp(pg.v_exp, h));
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const int t = j & 3, b0 = 4 * c + 2 * (j >> 2);
    uint32_t v[4];
    e2m1x8_f16x2(*reinterpret_cast<const uint32_t*>(grp + Block<D>::kK + c * 512 + (g * 4 + t) * 16 + (r >> 3) * 8 +
                                                    (j >> 2) * 4), v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s = e4m3_or_nan(grp[Block<D>::kKs + g * (D / 8) + (r >> 3) * (D / 16) + b0 + i]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 x = f16x2_f32(v[2 * i + e]);
        store2(kr + 16 * (b0 + i) + 4 * t + 2 * e, x.x * s * ke, x.y * s * ke);
      }
    }
    const int tv = g >> 1, w = (r & 1) + 2 * (r >> 3);
    e2m1x8_f16x2(*reinterpret_cast<const uint32_t*>(grp + Block<D>::kV + c * 512 + (j * 4 + tv) * 16 + w * 4), v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = e4m3_or_nan(grp[Block<D>::kVs + tv * (D / 4) + (4 * c + i) * 4 + w]);
      const float2 x = f16x2_f32(v[i]);
      store2(vr + 16 * (4 * c + i) + 2 * j, x.x * s * ve, x.y * s * ve);
    }
  }
}

// ---------------------------------------------------------------- attention

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;            // tokens of a warp's tile
constexpr int kTileGroups = kTile / kGroup;
// Probabilities are kept times 2^15 (the largest of a row is 2^15): as f16 they
// then have 11 bits down to 2^-29 of the largest instead of 2^-14, which shows
// where the likeliest tokens' values are zero.  Numerator and denominator carry
// the same factor.
constexpr float kPShift = 15.0f;

struct AttnParams {
  Pages pg;
  const void* q;           // [B, T, Hq, D] io
  void* out;               // [B, T, Hq, D] io
  const int32_t* lens;     // [B] cached tokens, the T new ones among them
  const int32_t* count;    // [B] query tokens of each sequence, or null (T)
  float* o_part;           // [B, Hkv, row tiles, splits, 8 NT, D]  partial outputs (splits > 1)
  float* ml_part;          // [B, Hkv, row tiles, splits, 8 NT, 2]  their (m, l), m in base 2
  int T_, Hq, G;
  int splits, row_tiles;
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
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t dup_lo(uint32_t v) { return __byte_perm(v, v, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t v) { return __byte_perm(v, v, 0x3232); }

// Query row r of a (sequence, KV head): token r / G, head r % G of the group.
// The MMAs compute S^T = K Q^T and O^T = V^T P^T: tokens (values) are the 16
// rows of A, straight from the cache's layout, and 8 query rows the columns.
// q is scaled per row by a power of two into f16's range (bf16 fits f16's 11
// bits; with SPLIT (f32 io) it is a pair of f16, 22 bits, and so is P).
template <typename T, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kThreads) kv4_attn_kernel(const AttnParams p) {
  constexpr int KS = D / 16;
  constexpr int NQ = SPLIT ? 2 : 1;
  const Pages& pg = p.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % p.splits, rt = blockIdx.x / p.splits, h = blockIdx.y, b = blockIdx.z;
  const int nq = rows_of(p.count, b, p.T_, threadIdx.x == 0 && h == 0 && blockIdx.x == 0);
  int len = p.lens[b];
  const int cap = pg.table_pages << pg.page_log2;
  if ((len < 0 || len > cap) && threadIdx.x == 0 && h == 0 && blockIdx.x == 0) record_status(kStatusBadIndex);
  len = max(0, min(cap, len));
  const int row0 = rt * 8 * NT;
  // this split's tiles
  const int tiles = (len + kTile - 1) / kTile;
  const int per = (tiles + p.splits - 1) / p.splits;
  const int tile0 = split * per, tile1 = min(tiles, tile0 + per);

  // B fragments of Q (column g of n-tile n), and per accumulator column its factor and its last token
  uint32_t qb[NQ][NT][KS][2];
  float f[NT][2];
  int lim[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = row0 + 8 * n + g;
    const bool real = r < nq * p.G;
    float x[KS][4];
    float am = 0.0f;
    const T* qr = static_cast<const T*>(p.q) +
                  ((static_cast<long long>(b) * p.T_ + r / p.G) * p.Hq + h * p.G + r % p.G) * D;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      x[ks][0] = x[ks][1] = x[ks][2] = x[ks][3] = 0.0f;
      if (real) {
        load2(qr + 16 * ks + 4 * t, x[ks]);
        load2(qr + 16 * ks + 4 * t + 2, x[ks] + 2);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) am = fmaxf(am, fabsf(x[ks][e]));
    }
    am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
    // the row's largest value to 2^14 .. 2^15; zeros, infinities as they are
    const int xe = static_cast<int>(__float_as_uint(am) >> 23);
    const int ex = xe == 0 || xe == 255 ? 0 : xe - 127 - 14;       // -140 .. 113
    const float down0 = pow2i(max(-100, min(100, -ex)) ), down1 = pow2i(-ex - max(-100, min(100, -ex)));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = x[ks][2 * i] * down0 * down1, c = x[ks][2 * i + 1] * down0 * down1;
        qb[0][n][ks][i] = pack_f16(a, c);
        if (SPLIT) {
          const float2 hi = f16x2_f32(qb[0][n][ks][i]);
          qb[NQ - 1][n][ks][i] = pack_f16(a - hi.x, c - hi.y);
        }
      }
    // scale * log2(e) * 2^(row + head), in two steps so that each stays finite
    const int e2 = ex + head_exp(pg.k_exp, h);                     // -204 .. 177
    const int e2a = max(-100, min(100, e2));
    const float fac = p.scale_log2 * pow2i(e2a) * pow2i(e2 - e2a);
    const int limit = real ? len - (nq - 1 - r / p.G) : 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f[n][e] = __shfl_sync(0xFFFFFFFFu, fac, (2 * t + e) * 4);
      lim[n][e] = __shfl_sync(0xFFFFFFFFu, limit, (2 * t + e) * 4);
    }
  }

  float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.0f;
  }

  for (int tile = tile0 + warp; tile < tile1; tile += kWarps) {
    const int tok0 = tile * kTile;
    const uint8_t* grp[kTileGroups];
    float s[NT][kTileGroups][4];
#pragma unroll
    for (int q = 0; q < kTileGroups; ++q) {
      const int tok = tok0 + q * kGroup;
      grp[q] = tok < len ? group_of<D>(pg, b, h, tok) : nullptr;
      if (tok < len && !grp[q] && lane == 0) record_status(kStatusBadIndex);
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][q][0] = s[n][q][1] = s[n][q][2] = s[n][q][3] = 0.0f;
      if (grp[q]) {
        uint32_t kc[KS], ks_[2][(KS + 3) / 4];
#pragma unroll
        for (int c = 0; c < KS / 4; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(grp[q] + Block<D>::kK + c * 512 + lane * 16);
          kc[4 * c] = v.x; kc[4 * c + 1] = v.y; kc[4 * c + 2] = v.z; kc[4 * c + 3] = v.w;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            ks_[i][c] = *reinterpret_cast<const uint32_t*>(grp[q] + Block<D>::kKs + g * (D / 8) + i * (D / 16) + 4 * c);
        }
#pragma unroll
        for (int c = 0; c < KS / 4; ++c) {
          uint32_t sl[2][2];
          e4m3x4_f16x2(ks_[0][c], sl[0][0], sl[0][1]);
          e4m3x4_f16x2(ks_[1][c], sl[1][0], sl[1][1]);
#pragma unroll
          for (int bp = 0; bp < 2; ++bp) {           // blocks 4c + 2 bp, + 1
            uint32_t x0[4], x1[4];                   // tokens g and g + 8
            e2m1x8_f16x2(kc[4 * c + bp], x0);
            e2m1x8_f16x2(kc[4 * c + 2 + bp], x1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t s0 = i ? dup_hi(sl[0][bp]) : dup_lo(sl[0][bp]);
              const uint32_t s1 = i ? dup_hi(sl[1][bp]) : dup_lo(sl[1][bp]);
              const uint32_t a0 = mul_f16x2(x0[2 * i], s0), a1 = mul_f16x2(x1[2 * i], s1);
              const uint32_t a2 = mul_f16x2(x0[2 * i + 1], s0), a3 = mul_f16x2(x1[2 * i + 1], s1);
              const int kb = 4 * c + 2 * bp + i;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816_f16(s[n][q], a0, a1, a2, a3, qb[0][n][kb][0], qb[0][n][kb][1]);
                if (SPLIT) mma16816_f16(s[n][q], a0, a1, a2, a3, qb[NQ - 1][n][kb][0], qb[NQ - 1][n][kb][1]);
              }
            }
          }
        }
      }
      // entries 0, 1: token g, columns 2t, 2t + 1; entries 2, 3: token g + 8
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[n][q][e] = grp[q] && tok + g + 8 * (e >> 1) < lim[n][e & 1] ? s[n][q][e] * f[n][e & 1] : -INFINITY;
    }
    // online softmax per column
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < kTileGroups; ++q) mx = fmaxf(mx, fmaxf(s[n][q][e], s[n][q][e + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        const float mn = fmaxf(m[n][e], mx);
        const float ref = mn == -INFINITY ? 0.0f : mn - kPShift;        // a column that sees none of these tokens
        const float corr = mn == -INFINITY ? 0.0f : ex2_approx(m[n][e] - mn);
        m[n][e] = mn;
        l[n][e] *= corr;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          o[n][k][e] *= corr;
          o[n][k][e + 2] *= corr;
        }
#pragma unroll
        for (int q = 0; q < kTileGroups; ++q) {
          s[n][q][e] = ex2_approx(s[n][q][e] - ref);
          s[n][q][e + 2] = ex2_approx(s[n][q][e + 2] - ref);
          l[n][e] += s[n][q][e] + s[n][q][e + 2];
        }
      }
    // O^T += V^T P^T
#pragma unroll
    for (int q = 0; q < kTileGroups; ++q) {
      if (!grp[q]) continue;
      uint32_t pb[NQ][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t hi = pack_f16(s[n][q][2 * i], s[n][q][2 * i + 1]);
          pb[0][n][i] = movmatrix_trans(hi);
          if (SPLIT) {
            const float2 h2 = f16x2_f32(hi);
            pb[NQ - 1][n][i] = movmatrix_trans(pack_f16(s[n][q][2 * i] - h2.x, s[n][q][2 * i + 1] - h2.y));
          }
        }
      // scales of tokens past the sequence's end are not its own: 0 (their P is 0, and 0 x NaN is not)
      const int left = len - (tok0 + q * kGroup);
      uint32_t keep = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * t + (i & 1) + 8 * (i >> 1) < left) keep |= 0xFFu << (8 * i);
#pragma unroll
      for (int c = 0; c < KS / 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(grp[q] + Block<D>::kV + c * 512 + lane * 16);
        const uint4 sv = *reinterpret_cast<const uint4*>(grp[q] + Block<D>::kVs + t * (D / 4) + c * 16);
        const uint32_t scw[4] = {sv.x & keep, sv.y & keep, sv.z & keep, sv.w & keep};
        uint32_t x0[4], x1[4], x2[4], x3[4];
        e2m1x8_f16x2((v.x & 0x0F0F0F0Fu) | ((v.y << 4) & 0xF0F0F0F0u), x0);     // values 2g, tokens 2t, 2t + 1
        e2m1x8_f16x2(((v.x >> 4) & 0x0F0F0F0Fu) | (v.y & 0xF0F0F0F0u), x1);     // values 2g + 1
        e2m1x8_f16x2((v.z & 0x0F0F0F0Fu) | ((v.w << 4) & 0xF0F0F0F0u), x2);     // values 2g, tokens 2t + 8, 2t + 9
        e2m1x8_f16x2(((v.z >> 4) & 0x0F0F0F0Fu) | (v.w & 0xF0F0F0F0u), x3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t slo, shi;
          e4m3x4_f16x2(scw[i], slo, shi);
          const uint32_t a0 = mul_f16x2(x0[i], slo), a1 = mul_f16x2(x1[i], slo);
          const uint32_t a2 = mul_f16x2(x2[i], shi), a3 = mul_f16x2(x3[i], shi);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816_f16(o[n][4 * c + i], a0, a1, a2, a3, pb[0][n][0], pb[0][n][1]);
            if (SPLIT) mma16816_f16(o[n][4 * c + i], a0, a1, a2, a3, pb[NQ - 1][n][0], pb[NQ - 1][n][1]);
          }
        }
      }
    }
  }

  // the warps' (m, l, O) in shared memory: [warp][column][D + 2]
  __shared__ float sh[kWarps][8 * NT][D + 2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float ls = l[n][e];
      ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 4);
      ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 8);
      ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 16);
      float* d = sh[warp][8 * n + 2 * t + e];
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        d[16 * k + 2 * g] = o[n][k][e];
        d[16 * k + 2 * g + 1] = o[n][k][e + 2];
      }
      if (g == 0) {
        d[D] = m[n][e];
        d[D + 1] = ls;
      }
    }
  __syncthreads();
  const float ve = pow2i(head_exp(pg.v_exp, h));
  const int cols = min(8 * NT, nq * p.G - row0);
  const long long slot = ((static_cast<long long>(b) * pg.Hkv + h) * p.row_tiles + rt) * p.splits + split;
  for (int i = threadIdx.x; i < cols * D; i += kThreads) {
    const int c = i / D, d = i % D;
    float ms = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ms = fmaxf(ms, sh[w][c][D]);
    const float ref = ms == -INFINITY ? 0.0f : ms;
    float num = 0.0f, den = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float fw = ex2_approx(sh[w][c][D] - ref);
      num += fw * sh[w][c][d];
      den += fw * sh[w][c][D + 1];
    }
    if (p.splits == 1) {
      const int r = row0 + c;
      static_cast<T*>(p.out)[((static_cast<long long>(b) * p.T_ + r / p.G) * p.Hq + h * p.G + r % p.G) * D + d] =
          from_f32<T>(den == 0.0f ? 0.0f : num / den * ve);
    } else {
      p.o_part[(slot * 8 * NT + c) * D + d] = num;
      if (d == 0) {
        p.ml_part[(slot * 8 * NT + c) * 2] = ms;
        p.ml_part[(slot * 8 * NT + c) * 2 + 1] = den;
      }
    }
  }
}

// out from the splits' partials, in split order.  Thread: one output element.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const AttnParams p) {
  pdl_wait();
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  const Pages& pg = p.pg;
  if (i >= static_cast<long long>(pg.B) * p.T_ * p.Hq * D) return;
  const int d = static_cast<int>(i % D);
  const long long qh = i / D;
  const int hq = static_cast<int>(qh % p.Hq);
  const int tok = static_cast<int>(qh / p.Hq % p.T_), b = static_cast<int>(qh / p.Hq / p.T_);
  if (tok >= rows_of(p.count, b, p.T_, false)) return;
  const int h = hq / p.G, r = tok * p.G + hq % p.G;
  const int rt = r / (8 * NT), c = r % (8 * NT);
  const long long slot = ((static_cast<long long>(b) * pg.Hkv + h) * p.row_tiles + rt) * p.splits;
  float ms = -INFINITY;
  for (int s = 0; s < p.splits; ++s) ms = fmaxf(ms, p.ml_part[((slot + s) * 8 * NT + c) * 2]);
  const float ref = ms == -INFINITY ? 0.0f : ms;
  float num = 0.0f, den = 0.0f;
  for (int s = 0; s < p.splits; ++s) {
    const long long k = (slot + s) * 8 * NT + c;
    const float fw = ex2_approx(p.ml_part[k * 2] - ref);
    num += fw * p.o_part[k * D + d];
    den += fw * p.ml_part[k * 2 + 1];
  }
  static_cast<T*>(p.out)[i] = from_f32<T>(den == 0.0f ? 0.0f : num / den * pow2i(head_exp(pg.v_exp, h)));
}

}  // namespace kv4
}  // namespace sambay
