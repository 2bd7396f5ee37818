// What the attention kernels over the 8-bit cache share: the line of work that their CTAs cut, and the sums of parts.
#pragma once

#include "kv8.cuh"
#include "kv8_rows.h"

namespace moe {

// A row's sums over some of its tokens: o in units of 2^(m + E), l of 2^m.
struct alignas(16) Kv8Stats {
  float m, E, l, pad;
};

namespace {

using Stats = Kv8Stats;
constexpr float LOWEST = -3e38f;  // the reference of a row that has seen nothing

// ---- the line of work ------------------------------------------------------------------
// A sequence's rows (of one key/value head) are cut into tiles of `rows`; each has the groups of GROUP tokens that
// any of the sequence's rows sees, one at least, and behind them PAD places that stand for what a piece of the line costs
// whatever its length (a cut among them counts as one behind them). Order: sequences, tiles (from both ends in turn, as
// later ones see more), heads, groups.
struct Seq {
  int begin, n, past, window;  // first row, tokens, position of the first, positions that a row sees
  int base, end;       // tokens that any of its rows sees, from a multiple of GROUP on
  int tiles, groups;   // row tiles, groups of tokens
};
template <int GROUP>
constexpr int pad_of() { return GROUP >= 128 ? 2 : 256 / GROUP; }
// a * b / c, by 32-bit division where that does.
__device__ __forceinline__ long long scaled(long long a, int b, long long c) {
  if (a < 1 << 22 && c < 1ll << 32) return (uint32_t)a * (uint32_t)b / (uint32_t)c;  // (b: CTAs, at most 1,023)
  return a * b / c;
}
template <int GROUP>
__device__ __forceinline__ Seq seq_of(const Kv8Args& a, int b, int rows) {
  Seq s;
  int end;
  kv8_range(a, b, s.begin, end);
  s.n = end - s.begin;
  s.past = kv8_past(a, b);
  s.end = min(s.past + s.n, a.capacity);
  s.window = kv8_window(a, b);
  s.base = max(s.past - s.window + 1, 0) & ~(GROUP - 1);
  s.end = max(s.end, s.base);
  const bool many = a.few_rows >= 0 && s.n * a.rep > a.few_rows;  // sequences of many rows have a kernel of their own
  s.tiles = many == (GROUP >= 128) ? kv8_tiles(s.n * a.rep, rows) : 0;
  s.groups = max(1, (s.end - s.base + GROUP - 1) / GROUP);
  return s;
}
template <int WARPS>
struct Scratch {
  long long sums[WARPS];
  long long at;
  int found, last;
};
// The groups of all sequences (a whole CTA).
template <int GROUP, int WARPS>
__device__ __forceinline__ long long line_length(const Kv8Args& a, int rows, Scratch<WARPS>* x) {
  long long total = 0;
  if (a.B == 1) {
    const Seq s = seq_of<GROUP>(a, 0, rows);
    return (long long)s.tiles * (s.groups + pad_of<GROUP>()) * a.G;
  }
  for (int b = threadIdx.x; b < a.B; b += 32 * WARPS) {
    const Seq s = seq_of<GROUP>(a, b, rows);
    total += (long long)s.tiles * (s.groups + pad_of<GROUP>());
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if ((threadIdx.x & 31) == 0) x->sums[threadIdx.x >> 5] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) total += x->sums[w];
  return total * a.G;
}
// The sequence that place `at` of the line is in; `at` becomes the place in it.
template <int GROUP, int WARPS>
__device__ __forceinline__ int find_place(const Kv8Args& a, int rows, long long& at, Scratch<WARPS>* x) {
  if (a.B == 1) return 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32 * WARPS) {
    const int b = b0 + threadIdx.x;
    long long mine = 0;
    if (b < a.B) {
      const Seq s = seq_of<GROUP>(a, b, rows);
      mine = (long long)s.tiles * (s.groups + pad_of<GROUP>()) * a.G;
    }
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    __syncthreads();  // the last round's sums have been read
    if (lane == 31) x->sums[warp] = sum;
    __syncthreads();
    long long from = before + sum - mine;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) from += x->sums[w];
      before += x->sums[w];
    }
    if (at >= from && at < from + mine) {
      x->found = b;
      x->at = at - from;
    }
    if (at < before) break;
  }
  __syncthreads();
  at = x->at;
  return x->found;
}
// The place at which CTA c's piece begins, and the CTA whose piece has place `at`.
__device__ __forceinline__ long long begin_of(int c, long long total, int ctas) { return scaled(total, c, ctas); }
__device__ __forceinline__ int owner_of(long long at, long long total, int ctas) {
  if (at + 1 < 1 << 22 && total < 1ll << 32) return (int)(((uint32_t)(at + 1) * (uint32_t)ctas - 1) / (uint32_t)total);
  return (int)(((at + 1) * ctas - 1) / total);
}
// Counts to `n` with field i of the tickets, three fields a word; true for the last one, which leaves it at 0.
__device__ __forceinline__ bool ticket(uint32_t* words, int i, int n) {
  uint32_t* w = words + i / 3;
  const int shift = i % 3 * 10;
  const bool last = (atomicAdd(w, 1u << shift) >> shift & 1023u) == (uint32_t)n - 1;
  if (last) atomicSub(w, (uint32_t)n << shift);
  return last;
}

// ---- sums and results ------------------------------------------------------------------
// What turns a row's sums over all tokens into its outputs: three factors, as the powers of two may be far from 1.
struct RowScale {
  float inv, p1, p2;
};
__device__ __forceinline__ RowScale row_scale(const Kv8Args& a, int h, const Stats& s) {
  float keep = 1.f, l = s.l;
  if (a.sinks) {
    const float sink = a.sinks[h] * 1.44269504f, top = fmaxf(s.m, sink);
    keep = ex2(s.m - top);
    l = l * keep + (sink == top ? 1.f : ex2(sink - top));
  }
  if (s.l == 0.f) return RowScale{0.f, 1.f, 1.f};  // has seen nothing
  const int E = (int)s.E, e1 = E / 2, e2 = E - e1;
  return RowScale{keep / l, __uint_as_float((uint32_t)(127 + e1) << 23), __uint_as_float((uint32_t)(127 + e2) << 23)};
}
template <typename T>
__device__ __forceinline__ void store4(T* out, const RowScale& r, const float4& x) {
  alignas(16) T y[4] = {from_f32<T>(x.x * r.inv * r.p1 * r.p2), from_f32<T>(x.y * r.inv * r.p1 * r.p2),
                        from_f32<T>(x.z * r.inv * r.p1 * r.p2), from_f32<T>(x.w * r.inv * r.p1 * r.p2)};
  if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(y);
  else *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(y);
}
// Where row r of the tile from row0 on of the sequence's tokens begin .. begin + n - 1 goes, or null.
template <typename T>
__device__ __forceinline__ T* out_row(const Kv8Args& a, int begin, int n, int g, int row0, int r, int& h) {
  if (r >= n * a.rep - row0) return nullptr;
  const int row = row0 + r, i = row / a.rep;
  h = g * a.rep + row - i * a.rep;
  return static_cast<T*>(a.o) + (int64_t)(begin + i) * a.os + h * a.D;
}
// Adds up the sums of `n` parts of a tile and head, part p in slot(p), in order: into slot `to` or, where
// they are all (to < 0), into the outputs.
template <typename T, typename F>
__device__ __forceinline__ void join(const Kv8Args& a, const Kv8Parts& f, int threads, int begin, int tokens, int row0,
                                     int g, int n, int to, F slot) {
  constexpr int AHEAD = 4;  // parts in flight (eight take registers that the many-rows kernel's loop then lacks: 390 -> 417 us)
  const int per = f.rows * a.D / 4;
  for (int i0 = 0; i0 < per; i0 += threads) {
    const int i = min(i0 + (int)threadIdx.x, per - 1), r = i * 4 / a.D, d = i * 4 - r * a.D;
    float m = LOWEST, E = 0.f, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < n; p0 += AHEAD) {
      float4 x[AHEAD], y[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int64_t at = (int64_t)slot(min(p0 + j, n - 1)) * f.rows + r;
        x[j] = __ldcg(reinterpret_cast<const float4*>(f.stats + at));
        y[j] = __ldcg(reinterpret_cast<const float4*>(f.parts + at * a.D + d));
      }
      float m1 = m;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) m1 = fmaxf(m1, x[j].x);
      float top = m - m1 + E;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) top = fmaxf(top, x[j].x - m1 + x[j].y);
      const float E1 = m1 == LOWEST ? 0.f : ceilf(top), keep = ex2((m - m1) + (E - E1));
      l *= ex2(m - m1);
      o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
      m = m1;
      E = E1;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (p0 + j >= n) break;
        if (x[j].x == LOWEST && x[j].z == 0.f) continue;  // saw nothing: has no sums
        const float w = ex2((x[j].x - m) + (x[j].y - E));
        l = fmaf(x[j].z, ex2(x[j].x - m), l);
        o.x = fmaf(y[j].x, w, o.x);
        o.y = fmaf(y[j].y, w, o.y);
        o.z = fmaf(y[j].z, w, o.z);
        o.w = fmaf(y[j].w, w, o.w);
      }
    }
    const Stats st{m, E, l, 0.f};
    if (i0 + (int)threadIdx.x >= per) break;
    if (to >= 0) {
      const int64_t at = (int64_t)to * f.rows + r;
      __stcg(reinterpret_cast<float4*>(f.parts + at * a.D + d), o);
      if (d == 0) __stcg(reinterpret_cast<float4*>(f.stats + at), make_float4(m, E, l, 0.f));
      continue;
    }
    int h = 0;
    T* out = out_row<T>(a, begin, tokens, g, row0, r, h);
    if (!out) continue;
    store4(out + d, row_scale(a, h, st), o);
  }
}

// Whether this CTA is the last of n to come to field i of the tickets; what they wrote is visible to it then.
template <typename Sync>
__device__ __forceinline__ bool last_of(const Kv8Parts& f, int i, int n, int* shared, Sync sync) {
  __threadfence();
  sync();
  if (threadIdx.x == 0) *shared = ticket(f.tickets, i, n);
  sync();
  const bool last = *shared != 0;
  if (last) __threadfence();
  return last;
}
// Joins a stretch of the line (a tile and head, which CTAs c0 .. c1 have parts of) once the last of them has written its
// part: parts of up to 24 CTAs at once, more of them by sixteens first. A CTA has two parts at most, of the
// stretch it begins with and of the one that goes on behind it.
// The slot of CTA c's part of the stretch whose first CTA is c0.
__device__ __forceinline__ int part_slot(int c, int c0, long long line0, long long total, int ctas) {
  return 2 * c + (c == c0 && line0 >= begin_of(c, total, ctas));
}
template <typename T, int CTAS, typename Sync>
__device__ __forceinline__ void join_stretch(const Kv8Args& a, const Kv8Parts& f, int threads, int begin, int tokens,
                                             int row0, int g, int c0, int c1, int slot0, int* shared, Sync sync) {
  const int cta = blockIdx.x;
  auto slot = [&](int c) { return c == c0 ? slot0 : 2 * c; };
  auto add = [&](int n, int to, auto from_slot) { join<T>(a, f, threads, begin, tokens, row0, g, n, to, from_slot); };
  if (c1 - c0 < 24) {
    if (last_of(f, c0, c1 - c0 + 1, shared, sync)) add(c1 - c0 + 1, -1, [&](int p) { return slot(c0 + p); });
    return;
  }
  const int sixteen = cta >> 4, lo = max(c0, sixteen * 16), hi = min(c1, sixteen * 16 + 15);
  auto field = [&](int x) { return 2 * x + (c0 >= x * 16); };  // two stretches can meet in a sixteen
  if (!last_of(f, CTAS + field(sixteen), hi - lo + 1, shared, sync)) return;
  add(hi - lo + 1, 2 * CTAS + field(sixteen), [&](int p) { return slot(lo + p); });
  const int n = (c1 >> 4) - (c0 >> 4) + 1;
  if (last_of(f, c0, n, shared, sync)) add(n, -1, [&](int p) { return 2 * CTAS + field((c0 >> 4) + p); });
}

}  // namespace
}  // namespace moe
