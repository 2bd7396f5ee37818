// What the 8-bit cache's kernels share: a call's arguments, which sequence, page and place a
// token has, scale bytes and codes.
#pragma once

#include "common.cuh"
#include "ops_host.h"
#include "types.cuh"

namespace moe {

// Tokens begin .. end - 1 of sequence b (clamped to the call's tokens; descending: empty).
__device__ __forceinline__ void kv8_range(const Kv8Args& a, int b, int& begin, int& end) {
  if (a.offsets) {
    begin = min(max(a.offsets[b], 0), a.N);
    end = max(min(max(a.offsets[b + 1], 0), a.N), begin);
  } else {
    begin = b * a.seq_len;
    end = begin + a.seq_len;
  }
}
// Position of the sequence's first token of the call. Clamped: what lies outside stays outside (2^28 tokens at most), and
// neither sums with tokens nor differences from a window leave 32 bits.
__device__ __forceinline__ int kv8_past(const Kv8Args& a, int b) {
  return a.past ? min(max(a.past[b], -(1 << 28)), 1 << 30) : 0;
}
// How many positions a row of sequence b sees, its own the last, with positions clamped as above: less by what was taken
// from them (0 and fewer: none that can be held). No window: more than there are positions.
__device__ __forceinline__ int kv8_window(const Kv8Args& a, int b) {
  constexpr int all = (1 << 30) + (1 << 28) + 1;
  if (!a.window) return all;
  const int over = a.past ? max(a.past[b], 1 << 30) - (1 << 30) : 0;
  return min(max(a.window - over, -(1 << 28)), all);
}
// The sequence that a row is a token of, or -1, by bisection of the ascending offsets.
__device__ __forceinline__ int kv8_seq_of(const Kv8Args& a, int row, int& begin, int& end) {
  int b = 0;
  if (!a.offsets) {
    b = row / a.seq_len;
  } else {
    int hi = a.B;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (a.offsets[mid] <= row) b = mid;
      else hi = mid;
    }
  }
  kv8_range(a, b, begin, end);
  return row >= begin && row < end ? b : -1;
}
// The page that holds a position of sequence b, or -1.
__device__ __forceinline__ int kv8_page(const Kv8Args& a, int b, int pos) {
  if (pos < 0 || pos >= a.capacity) return -1;
  const int id = a.pages[(int64_t)b * a.max_pages + (pos >> a.page_log)];
  return id >= 0 && id < a.n_pages ? id : -1;
}
// Codes of the place `at` of a page for head h (which 0: K, 1: V), and the byte of its scale.
__device__ __forceinline__ int64_t kv8_codes(const Kv8Args& a, int page, int h, int which, int at) {
  return page * a.page_bytes + (((h * 2 + which) << a.page_log) + at) * (int64_t)a.D;
}
__device__ __forceinline__ int64_t kv8_scale(const Kv8Args& a, int page, int h, int which, int at) {
  return page * a.page_bytes + a.scales_at + ((h * 2 + which) << (a.page_log - a.block_log)) + (at >> a.block_log);
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float kv8_power(int byte) {
  return __uint_as_float(byte == 255 ? 0x7fc00000u : byte == 0 ? 0x00400000u : (uint32_t)byte << 23);
}
// Four codes as f32.
template <int CODE>
__device__ __forceinline__ float4 kv8_values(uint32_t w) {
  if constexpr (CODE == MOE_I8) {
    w ^= 0x80808080u;  // code + 128 in the low mantissa byte of 2^23
    constexpr float off = MAGIC_2P23 + 128.f;
    return make_float4(magic_byte(w, 0) - off, magic_byte(w, 1) - off, magic_byte(w, 2) - off, magic_byte(w, 3) - off);
  } else {
    uint32_t lo, hi;
    asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(x.x, x.y, y.x, y.y);
  }
}
// Four values of at most the code's largest magnitude, each rounded to the nearest code (even on ties).
template <int CODE>
__device__ __forceinline__ uint32_t kv8_encode(float x0, float x1, float x2, float x3) {
  if constexpr (CODE == MOE_I8) {
    constexpr float round = 12582912.f;  // 1.5 * 2^23: the sum's low byte is the rounded value
    const uint32_t a = __byte_perm(__float_as_uint(x0 + round), __float_as_uint(x1 + round), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(x2 + round), __float_as_uint(x3 + round), 0x0040);
    return __byte_perm(a, b, 0x5410);
  } else {
    uint32_t r;
    asm("{.reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
        " mov.b32 %0, {a, b};}" : "=r"(r) : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return r;
  }
}

// Codes 2 hi, 2 hi + 1 of a word as a pair of 16-bit numbers.
template <int CODE, bool BF16>
__device__ __forceinline__ uint32_t pair_of(uint32_t w, bool hi) {
  if constexpr (CODE == MOE_I8 && !BF16) {  // w has code + 128: 1024 + 128 + code in f16, less 1152
    const uint32_t u = __byte_perm(w, 0x64646464u, hi ? 0x4342 : 0x4140), off = 0x64806480u;
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&off));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else if constexpr (CODE == MOE_I8) {
    // 0x43 above a byte u is 128 + u in bf16, but 2 u where u's first bit falls into the exponent. With u = code + 128
    // that is 256 + code below 0 and 256 + 2 code from there on: one integer and three bf16 operations
    // (by masks it is three and one, and the integer pipe has half the rate)
    const uint32_t u = __byte_perm(w, 0x43434343u, hi ? 0x4342 : 0x4140), one = 0x3f803f80u, off = 0xc380c380u, half = 0xbf00bf00u;
    auto v = [](const uint32_t& x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
    const __nv_bfloat162 twice = __hfma2_relu(v(u), v(one), v(off)), h = __hfma2(twice, v(half), __hadd2(v(u), v(off)));
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    uint32_t h;
    asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(h) : "r"(hi ? w >> 16 : w));
    if constexpr (BF16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(f.y), "f"(f.x));
    }
    return h;
  }
}
// What pair_of wants of a word of codes.
template <int CODE>
__device__ __forceinline__ uint32_t code_word(uint32_t w) {
  return CODE == MOE_I8 ? w ^ 0x80808080u : w;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
}  // namespace moe
