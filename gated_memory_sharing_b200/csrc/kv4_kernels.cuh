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

// The tokens of all (sequence, KV head, row tile) pairs are cut into tiles of
// 4096 / D tokens (4608 bytes of cache) and laid end to end; every warp of the
// grid takes the same share of that line, whatever the lengths are, and goes
// through it on its own: no CTA-wide synchronisation, and a warp that changes
// from one pair to the next does not hold up the others.  Pairs that lie in
// one warp's share are finished there; of the others every warp leaves (m, l,
// O) for the combine kernel, which adds them in the line's order.
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 3;
constexpr int kStageBytes = 4608;
// Probabilities are kept times 2^15 (the largest of a row is 2^15): as f16 they
// then have 11 bits down to 2^-29 of the largest instead of 2^-14, which shows
// where the likeliest tokens' values are zero.  Numerator and denominator carry
// the same factor.
constexpr float kPShift = 15.0f;

// Resident CTAs an SM: what the registers of a variant allow (128 registers a
// thread for 4, 168 for 3, 255 for 2).
constexpr int attn_ctas(int d, int nt, bool split) {
  const int size = d * nt * (split ? 2 : 1);
  return size <= 128 && nt == 1 ? 4 : size <= 256 ? 3 : 2;
}

struct AttnParams {
  Pages pg;
  const void* q;           // [B, T, Hq, D] io
  void* out;               // [B, T, Hq, D] io
  const int32_t* lens;     // [B] cached tokens, the T new ones among them
  const int32_t* count;    // [B] query tokens of each sequence, or null (T)
  float* o_part;           // [warp][first or last pair][cols, D]  partial outputs
  float* ml_part;          // [warp][first or last pair][cols, 2]  their (m, l), m in base 2
  int T_, Hq, G;
  int row_tiles, cols;     // cols: min(8 NT, G T) columns of a row tile
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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Cached tokens of sequence b, inside the table; `tell` records a length outside it.
__device__ __forceinline__ int len_of(const AttnParams& p, int b, bool tell) {
  const int len = p.lens[b], cap = p.pg.table_pages << p.pg.page_log2;
  if (tell && (len < 0 || len > cap)) record_status(kStatusBadIndex);
  return max(0, min(cap, len));
}
// Tiles of a pair of a sequence: an empty one has one, which writes its zeros.
template <int D>
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + 4096 / D - 1) / (4096 / D)); }

// The line: its length in tiles, the warps that share it (none of them without
// a tile), and where share w begins.
struct Line {
  long long tiles;
  int shares;
  __device__ __forceinline__ long long begin(long long w) const { return tiles * w / shares; }
  // the share that holds tile x
  __device__ __forceinline__ int share_of(long long x) const {
    return static_cast<int>(((x + 1) * shares - 1) / tiles);
  }
};

// The line of a call, and the tile in it at which sequence b begins (one warp).
template <int D>
__device__ __forceinline__ Line line_of(const AttnParams& p, int b, bool tell, long long* before) {
  long long s = 0, sb = 0;
  for (int i = threadIdx.x & 31; i < p.pg.B; i += 32) {
    const int n = tiles_of<D>(len_of(p, i, tell));
    s += n;
    if (i < b) sb += n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    sb += __shfl_xor_sync(0xFFFFFFFFu, sb, o);
  }
  *before = sb * p.pg.Hkv * p.row_tiles;
  Line line;
  line.tiles = s * p.pg.Hkv * p.row_tiles;
  line.shares = static_cast<int>(min(line.tiles, static_cast<long long>(p.warps)));
  return line;
}

// A place in the line.
struct Cursor {
  int b, pair, tile;       // pair: KV head * row tiles + row tile
  int len, tiles;          // of sequence b
};

template <int D>
__device__ __forceinline__ void advance(const AttnParams& p, Cursor& c) {
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.pair < p.pg.Hkv * p.row_tiles) return;
  c.pair = 0;
  if (++c.b < p.pg.B) {
    c.len = len_of(p, c.b, false);
    c.tiles = tiles_of<D>(c.len);
  }
}

// Tile x of the line.
template <int D>
__device__ __forceinline__ Cursor find(const AttnParams& p, long long x) {
  const int lane = threadIdx.x & 31;
  const int pairs = p.pg.Hkv * p.row_tiles;
  Cursor c{};
  for (int b0 = 0; b0 < p.pg.B; b0 += 32) {
    const int len = b0 + lane < p.pg.B ? len_of(p, b0 + lane, false) : 0;
    const int n = b0 + lane < p.pg.B ? tiles_of<D>(len) : 0;
    long long upto = static_cast<long long>(n) * pairs;            // of this and the sequences before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned past = __ballot_sync(0xFFFFFFFFu, upto > x);
    if (past) {
      const int k = __ffs(past) - 1;
      c.b = b0 + k;
      c.len = __shfl_sync(0xFFFFFFFFu, len, k);
      c.tiles = __shfl_sync(0xFFFFFFFFu, n, k);
      const long long in = x - (__shfl_sync(0xFFFFFFFFu, upto, k) - static_cast<long long>(c.tiles) * pairs);
      c.pair = static_cast<int>(in / c.tiles);
      c.tile = static_cast<int>(in % c.tiles);
      return c;
    }
    x -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  return c;                                                        // not reached: x is in the line
}

// Query row r of a (sequence, KV head): token r / G, head r % G of the group.
// The MMAs compute S^T = K Q^T and O^T = V^T P^T: tokens (values) are the 16
// rows of A, straight from the cache's layout, and 8 query rows the columns.
// q is scaled per row by a power of two into f16's range (bf16 fits f16's 11
// bits; with SPLIT (f32 io) it is a pair of f16, 22 bits, and so is P).
template <typename T, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, attn_ctas(D, NT, SPLIT)) kv4_attn_kernel(const AttnParams p) {
  constexpr int KS = D / 16;
  constexpr int NQ = SPLIT ? 2 : 1;
  constexpr int TILE = 4096 / D, GP = TILE / kGroup;
  constexpr int kChunks = Block<D>::kBytes / 16;      // 16-byte pieces of a group
  extern __shared__ __align__(128) uint8_t smem[];
  const Pages& pg = p.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // the first warps of all CTAs, then their second ones: few shares spread over the GPU
  const int gw = warp * gridDim.x + blockIdx.x;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  const uint32_t ring_addr = shared_addr(ring);

  long long none;
  const Line line = line_of<D>(p, 0, gw == 0, &none);
  if (gw >= line.shares) return;
  const long long begin = line.begin(gw);
  const int share = static_cast<int>(line.begin(gw + 1) - begin);

  Cursor in = find<D>(p, begin);       // the next tile to load
  Cursor c = in;                       // the tile being worked on

  // Pages of the 32 groups of the loading cursor's window (512 tokens), one a lane.
  int win_b = -1, win = -1, page = -1;
  uint32_t have = 0;                   // GP bits a stage: which groups were loaded
  auto issue = [&](int i, int st) {
    if (i < share) {
      const int tok0 = in.tile * TILE;
      if (in.b != win_b || (tok0 >> 9) != win) {
        win_b = in.b;
        win = tok0 >> 9;
        const int tok = win * 512 + lane * kGroup;
        page = -1;
        if (tok < in.len) {
          page = pg.table[static_cast<long long>(in.b) * pg.table_pages + (tok >> pg.page_log2)];
          if (page < 0 || page >= pg.num_pages) {
            page = -1;
            record_status(kStatusBadIndex);
          }
        }
      }
      const int h = in.pair / p.row_tiles;
      uint32_t mask = 0;
#pragma unroll
      for (int q = 0; q < GP; ++q) {
        const int tok = tok0 + q * kGroup;
        const int pid = __shfl_sync(0xFFFFFFFFu, page, (tok >> 4) & 31);
        if (pid >= 0) {
          mask |= 1u << q;
          const int at = (tok & ((1 << pg.page_log2) - 1)) / kGroup;
          const uint8_t* src =
              pg.cache + (((static_cast<long long>(pid) * pg.Hkv + h) << (pg.page_log2 - 4)) + at) * Block<D>::kBytes;
          const uint32_t dst = ring_addr + st * kStageBytes + q * Block<D>::kBytes;
#pragma unroll
          for (int k = 0; k < (kChunks + 31) / 32; ++k) {
            const int x = lane + 32 * k;
            if (x < kChunks) cp_async16(dst + x * 16, src + x * 16);
          }
        }
      }
      have = (have & ~(((1u << GP) - 1) << (GP * st))) | mask << (GP * st);
      advance<D>(p, in);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i, i);

  uint32_t qb[NQ][NT][KS][2];
  float f[NT][2];
  int lim[NT][2];
  float m[NT][2], l[NT][2], o[NT][KS][4];
  bool fresh = true;
  int st = 0, lim_min = 0;

  for (int i = 0; i < share; ++i) {
    issue(i + kStages - 1, st == 0 ? kStages - 1 : st - 1);
    if (fresh) {
      // B fragments of Q (column g of n-tile n), and per accumulator column its factor and its last token
      fresh = false;
      const int h = c.pair / p.row_tiles, row0 = c.pair % p.row_tiles * (8 * NT);
      const int nq = rows_of(p.count, c.b, p.T_, c.pair == 0);
      lim_min = c.len;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = row0 + 8 * n + g;
        const bool real = r < nq * p.G;
        const int tok = r / p.G;
        float x[KS][4];
        float am = 0.0f;
        const T* qr =
            static_cast<const T*>(p.q) + ((static_cast<long long>(c.b) * p.T_ + tok) * p.Hq + h * p.G + r % p.G) * D;
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
        const int exa = max(-100, min(100, -ex));
        const float down0 = pow2i(exa), down1 = pow2i(-ex - exa);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float u = x[ks][2 * e] * down0 * down1, v = x[ks][2 * e + 1] * down0 * down1;
            qb[0][n][ks][e] = pack_f16(u, v);
            if (SPLIT) {
              const float2 hi = f16x2_f32(qb[0][n][ks][e]);
              qb[NQ - 1][n][ks][e] = pack_f16(u - hi.x, v - hi.y);
            }
          }
        // scale * log2(e) * 2^(row + head), in two steps so that each stays finite
        const int e2 = ex + head_exp(pg.k_exp, h);                     // -204 .. 177
        const int e2a = max(-100, min(100, e2));
        // kept normal and finite: a masked -infinity times it stays one
        const float fac = fminf(fmaxf(p.scale_log2 * pow2i(e2a) * pow2i(e2 - e2a), 1.2e-38f), 3e38f);
        const int limit = real ? c.len - (nq - 1 - tok) : 0x7FFFFFFF;  // columns that are none see all, and are not written
        lim_min = min(lim_min, limit);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[n][e] = __shfl_sync(0xFFFFFFFFu, fac, (2 * t + e) * 4);
          lim[n][e] = min(c.len, __shfl_sync(0xFFFFFFFFu, limit, (2 * t + e) * 4));
          m[n][e] = -INFINITY;
          l[n][e] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.0f;
      }
      lim_min = __reduce_min_sync(0xFFFFFFFFu, lim_min);
    }
    cp_async_wait<kStages - 1>();
    __syncwarp();

    const int tok0 = c.tile * TILE;
    const uint32_t mask = have >> (GP * st) & ((1u << GP) - 1);
    const uint8_t* stage = ring + st * kStageBytes;
    float s[NT][GP][4];
    // S^T of group q: entries 0, 1: token g, columns 2t, 2t + 1; entries 2, 3: token g + 8
    auto scores = [&](int q) {
      const uint8_t* grp = stage + q * Block<D>::kBytes;
      uint32_t kc[KS], sc[2][KS / 4];
#pragma unroll
      for (int k = 0; k < KS / 4; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(grp + Block<D>::kK + k * 512 + lane * 16);
        kc[4 * k] = v.x; kc[4 * k + 1] = v.y; kc[4 * k + 2] = v.z; kc[4 * k + 3] = v.w;
      }
      if (KS == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(grp + Block<D>::kKs + g * 8);
        sc[0][0] = v.x; sc[1][0] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(grp + Block<D>::kKs + g * 16);
        sc[0][0] = v.x; sc[0][KS / 4 - 1] = v.y; sc[1][0] = v.z; sc[1][KS / 4 - 1] = v.w;
      }
#pragma unroll
      for (int k = 0; k < KS / 4; ++k) {
        uint32_t sl[2][2];
        e4m3x4_f16x2(sc[0][k], sl[0][0], sl[0][1]);
        e4m3x4_f16x2(sc[1][k], sl[1][0], sl[1][1]);
#pragma unroll
        for (int bp = 0; bp < 2; ++bp) {             // blocks 4k + 2 bp, + 1
          uint32_t x0[4], x1[4];                     // tokens g and g + 8
          e2m1x8_f16x2(kc[4 * k + bp], x0);
          e2m1x8_f16x2(kc[4 * k + 2 + bp], x1);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t s0 = e ? dup_hi(sl[0][bp]) : dup_lo(sl[0][bp]);
            const uint32_t s1 = e ? dup_hi(sl[1][bp]) : dup_lo(sl[1][bp]);
            const uint32_t a0 = mul_f16x2(x0[2 * e], s0), a1 = mul_f16x2(x1[2 * e], s1);
            const uint32_t a2 = mul_f16x2(x0[2 * e + 1], s0), a3 = mul_f16x2(x1[2 * e + 1], s1);
            const int kb = 4 * k + 2 * bp + e;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816_f16(s[n][q], a0, a1, a2, a3, qb[0][n][kb][0], qb[0][n][kb][1]);
              if (SPLIT) mma16816_f16(s[n][q], a0, a1, a2, a3, qb[NQ - 1][n][kb][0], qb[NQ - 1][n][kb][1]);
            }
          }
        }
      }
    };
    // O^T += V^T P^T of group q.  Where not all see all (EDGE): the bytes of
    // `keep` that are 0 blank the scales of tokens that are not the sequence's,
    // whose P is 0 (0 x NaN is not), and a block of NaN reaches only the columns
    // that see its token: its scale is blanked too, and the columns set to NaN.
    auto outputs = [&](int q, uint32_t keep, auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
      const uint8_t* grp = stage + q * Block<D>::kBytes;
      uint32_t pb[NQ][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t hi = pack_f16(s[n][q][2 * e], s[n][q][2 * e + 1]);
          pb[0][n][e] = movmatrix_trans(hi);
          if (SPLIT) {
            const float2 h2 = f16x2_f32(hi);
            pb[NQ - 1][n][e] = movmatrix_trans(pack_f16(s[n][q][2 * e] - h2.x, s[n][q][2 * e + 1] - h2.y));
          }
        }
#pragma unroll
      for (int k = 0; k < KS / 4; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(grp + Block<D>::kV + k * 512 + lane * 16);
        const uint4 sv = *reinterpret_cast<const uint4*>(grp + Block<D>::kVs + t * (D / 4) + k * 16);
        uint32_t scw[4] = {sv.x & keep, sv.y & keep, sv.z & keep, sv.w & keep};
        uint32_t x0[4], x1[4], x2[4], x3[4];
        e2m1x8_f16x2((v.x & 0x0F0F0F0Fu) | ((v.y << 4) & 0xF0F0F0F0u), x0);     // values 2g, tokens 2t, 2t + 1
        e2m1x8_f16x2(((v.x >> 4) & 0x0F0F0F0Fu) | (v.y & 0xF0F0F0F0u), x1);     // values 2g + 1
        e2m1x8_f16x2((v.z & 0x0F0F0F0Fu) | ((v.w << 4) & 0xF0F0F0F0u), x2);     // values 2g, tokens 2t + 8, 2t + 9
        e2m1x8_f16x2(((v.z >> 4) & 0x0F0F0F0Fu) | (v.w & 0xF0F0F0F0u), x3);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int bad = 0x7FFFFFFF;                       // first token of the group whose block is NaN
          if (EDGE) {
            const uint32_t nan = __vcmpeq4(scw[e], 0x7F7F7F7Fu);
            if (__any_sync(0xFFFFFFFFu, nan != 0)) {
              scw[e] &= ~nan;
              if (nan) bad = tok0 + q * kGroup + 2 * t + (nan & 0xFFu ? 0 : nan & 0xFF00u ? 1 : nan & 0xFF0000u ? 8 : 9);
              bad = min(bad, __shfl_xor_sync(0xFFFFFFFFu, bad, 1));
              bad = min(bad, __shfl_xor_sync(0xFFFFFFFFu, bad, 2));
            }
          }
          uint32_t slo, shi;
          e4m3x4_f16x2(scw[e], slo, shi);
          const uint32_t a0 = mul_f16x2(x0[e], slo), a1 = mul_f16x2(x1[e], slo);
          const uint32_t a2 = mul_f16x2(x2[e], shi), a3 = mul_f16x2(x3[e], shi);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816_f16(o[n][4 * k + e], a0, a1, a2, a3, pb[0][n][0], pb[0][n][1]);
            if (SPLIT) mma16816_f16(o[n][4 * k + e], a0, a1, a2, a3, pb[NQ - 1][n][0], pb[NQ - 1][n][1]);
            if (EDGE) {
#pragma unroll
              for (int i2 = 0; i2 < 4; ++i2)
                if (bad < lim[n][i2 & 1]) o[n][4 * k + e][i2] = __int_as_float(0x7FC00000);
            }
          }
        }
      }
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < GP; ++q) s[n][q][0] = s[n][q][1] = s[n][q][2] = s[n][q][3] = 0.0f;
    const bool whole = mask == (1u << GP) - 1 && tok0 + TILE <= lim_min;   // every column sees every token
    if (whole) {
#pragma unroll
      for (int q = 0; q < GP; ++q) scores(q);
    } else {
#pragma unroll
      for (int q = 0; q < GP; ++q) {
        if (mask >> q & 1) scores(q);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(mask >> q & 1) || tok0 + q * kGroup + g + 8 * (e >> 1) >= lim[n][e & 1]) s[n][q][e] = -INFINITY;
      }
    }
    // online softmax per column: the factor f > 0, so the largest s is the largest logit
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < GP; ++q) mx = fmaxf(mx, fmaxf(s[n][q][e], s[n][q][e + 2]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        const float mn = fmaxf(m[n][e], mx * f[n][e]);
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
        for (int q = 0; q < GP; ++q) {
          s[n][q][e] = ex2_approx(fmaf(s[n][q][e], f[n][e], -ref));
          s[n][q][e + 2] = ex2_approx(fmaf(s[n][q][e + 2], f[n][e], -ref));
          l[n][e] += s[n][q][e] + s[n][q][e + 2];
        }
      }
    if (whole) {
#pragma unroll
      for (int q = 0; q < GP; ++q) outputs(q, 0xFFFFFFFFu, std::false_type());
    } else {
#pragma unroll
      for (int q = 0; q < GP; ++q) {
        const int left = c.len - (tok0 + q * kGroup);
        uint32_t keep = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (2 * t + (e & 1) + 8 * (e >> 1) < left) keep |= 0xFFu << (8 * e);
        if (mask >> q & 1) outputs(q, keep, std::true_type());
      }
    }
    __syncwarp();                      // the stage is read; the next iteration's copies may refill it
    st = st == kStages - 1 ? 0 : st + 1;

    if (c.tile + 1 == c.tiles || i + 1 == share) {
      // the pair, or this warp's share of it, is done
      const int h = c.pair / p.row_tiles, row0 = c.pair % p.row_tiles * (8 * NT);
      const int nq = rows_of(p.count, c.b, p.T_, false);
      const float ve = pow2i(head_exp(pg.v_exp, h));
      const bool from_start = i >= c.tile;                     // the pair's first tile is in this share
      const bool done = from_start && c.tile + 1 == c.tiles;
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
              T* dst = static_cast<T*>(p.out) +
                       ((static_cast<long long>(c.b) * p.T_ + r / p.G) * p.Hq + h * p.G + r % p.G) * D;
#pragma unroll
              for (int k = 0; k < KS; ++k) store2(dst + 16 * k + 2 * g, o[n][k][e] * inv, o[n][k][e + 2] * inv);
            } else {
              float* dst = p.o_part + (slot * p.cols + col) * D;
#pragma unroll
              for (int k = 0; k < KS; ++k) store2(dst + 16 * k + 2 * g, o[n][k][e], o[n][k][e + 2]);
              if (g == 0) store2(p.ml_part + (slot * p.cols + col) * 2, m[n][e], ls);
            }
          }
        }
      fresh = true;
    }
    advance<D>(p, c);
  }
}

// Rows whose pair was shared by several warps, from their parts in the line's
// order.  WARPS warps a row (8 where a pair has many parts, else 1).
template <typename T, int D, int NT, int WARPS>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const AttnParams p) {
  constexpr int V = D / 32;            // values a lane
  pdl_wait();
  const Pages& pg = p.pg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = WARPS == 1 ? blockIdx.x * 8LL + warp : blockIdx.x;
  if (row >= static_cast<long long>(pg.B) * p.T_ * p.Hq) return;
  const int hq = static_cast<int>(row % p.Hq);
  const int tok = static_cast<int>(row / p.Hq % p.T_), b = static_cast<int>(row / p.Hq / p.T_);
  if (tok >= rows_of(p.count, b, p.T_, false)) return;
  const int h = hq / p.G, r = tok * p.G + hq % p.G;
  const int pair = h * p.row_tiles + r / (8 * NT), col = r % (8 * NT);
  long long before;
  const Line line = line_of<D>(p, b, false, &before);
  const int tiles = tiles_of<D>(len_of(p, b, false));
  const long long a = before + static_cast<long long>(pair) * tiles;
  const int w0 = line.share_of(a), w1 = line.share_of(a + tiles - 1);
  if (w0 == w1) return;                // finished by that warp
  const int first = line.begin(w0) == a ? 0 : 1;
  auto slot = [&](int w) { return (static_cast<long long>(w) * 2 + (w == w0 ? first : 0)) * p.cols + col; };
  float ms = -INFINITY;
  for (int w = w0 + lane; w <= w1; w += 32) ms = fmaxf(ms, p.ml_part[slot(w) * 2]);
#pragma unroll
  for (int o = 16; o; o >>= 1) ms = fmaxf(ms, __shfl_xor_sync(0xFFFFFFFFu, ms, o));
  const float ref = ms == -INFINITY ? 0.0f : ms;
  float num[V], den = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) num[v] = 0.0f;
  // this warp's run of the parts
  const int n = w1 - w0 + 1, per = (n + WARPS - 1) / WARPS;
  const int lo = w0 + (WARPS == 1 ? 0 : warp * per), hi = min(w1 + 1, lo + per);
#pragma unroll 4
  for (int w = lo; w < hi; ++w) {
    const long long k = slot(w);
    const float2 ml = *reinterpret_cast<const float2*>(p.ml_part + k * 2);
    const float fw = ex2_approx(ml.x - ref);
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      float x[2];
      load2(p.o_part + k * D + lane * V + v, x);
      num[v] = fmaf(fw, x[0], num[v]);
      num[v + 1] = fmaf(fw, x[1], num[v + 1]);
    }
    den = fmaf(fw, ml.y, den);
  }
  if (WARPS > 1) {
    __shared__ float sh[WARPS][D + 1];
#pragma unroll
    for (int v = 0; v < V; ++v) sh[warp][lane * V + v] = num[v];
    if (lane == 0) sh[warp][D] = den;
    __syncthreads();
    if (warp != 0) return;
    den = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) num[v] = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
#pragma unroll
      for (int v = 0; v < V; ++v) num[v] += sh[w][lane * V + v];
      den += sh[w][D];
    }
  }
  const float inv = den == 0.0f ? 0.0f : pow2i(head_exp(pg.v_exp, h)) / den;
  T* dst = static_cast<T*>(p.out) + row * D + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) store2(dst + v, num[v] * inv, num[v + 1] * inv);
}

}  // namespace kv4
}  // namespace sambay
