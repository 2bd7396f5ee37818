// Attention over the 8-bit cache for few rows a key/value head: single tokens, short parts of prompts, of which every code is
// read once for eight or sixteen rows and the cache's bytes are the bound. f32 prompts and those with heads of more than 128
// or more than 128 heads a key/value head come here as well; they are bound by the products, and by codes that are
// converted again for each tile (16,384 tokens x 16 heads of 256, bf16: 21.9 ms; 1,524 tokens x 16 heads of 128, f32: 175 us).
//
// A warp takes 16 tokens at a time, with the rows (query tokens x the heads that share a key/value head) along the
// short side of the m16n8k16 products:
//   S^T [16 tokens][8 rows] = K Q^T        O^T [dim][8 rows] += V^T P^T
// K's and V's lanes are chosen so that a lane's operands are 16 neighbouring bytes of a token: any order of the
// dimensions does as long as Q's lanes, and the outputs', follow it. S^T's accumulators become P^T's operands by one
// 8 x 8 transposition in registers.
//
// Softmax without a reduction per step: a row keeps a reference m of its scores s (in powers of two) and
// an integer E, such that s <= m + 8 and s + v <= m + E + 8 for all s so far, v the exponent of the
// token's V scale. Weights are 2^(s - m) in the sum and 2^(s - m + v - E) as operands of V's codes, so
// neither a token of weight with tiny values nor one of large values without weight takes the
// others' bits. Only a score beyond its bound makes the warp look for new references.
//
// Operands: codes are exact in f16 and bf16. f16 rows are operands as they are; bf16 rows are f16 times a power
// of two a row (as they are down to 2^-32 of the row's largest); f32 ones are three bf16 parts, which are the
// value. Weights are bf16 parts, whose bits go by each weight's own size: two for bf16 outputs (16 bits), three for the
// others (24). (f16 parts, one or two, on V's codes in f16, which take two instructions a pair where bf16 takes four, lost
// bits below 2^-20 of the row's largest product of weight and V scale and all below 2^-30: 64 sequences 211 us where this
// takes 217, but 3,000 tokens behind a first one of 2^27 times each one's weight and no value were 1.5% off, of 2^45 lost.)
//
// The call's groups of tokens, of all sequences, row tiles and heads, are one line that the CTAs cut into
// equal pieces, two CTAs an SM. A tile and head that a cut goes through is joined by the CTA that is done with its part last,
// in the order of the line.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "kv8_line.cuh"
#include "tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

// ---- operands --------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// An 8 x 8 matrix of 16-bit values, a row on four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two f32 values as n parts each, packed in pairs (low half first).
template <int n, bool BF16>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t (&out)[n]) {
#pragma unroll
  for (int p = 0; p < n; ++p) {
    uint32_t h;
    if constexpr (!BF16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    else if (n == 3 && p == 0) h = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);  // cut off: no rounding to infinity
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    out[p] = h;
    if (p + 1 < n) {
      if constexpr (BF16) {
        x0 -= __uint_as_float(h << 16);
        x1 -= __uint_as_float(h & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x0 -= f.x;
        x1 -= f.y;
      }
    }
  }
}
// Rows of 128 bytes of the cache, from row `y` on, to shared memory.
__device__ __forceinline__ void copy_rows(void* dst, const CUtensorMap* map, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(smem_addr(dst)), "l"(map), "r"(smem_addr(bar)), "r"(0), "r"(y) : "memory");
}

// Warps that work, beside the one that fetches, and tokens of a group: what two CTAs an SM have registers for, and
// shared memory for two groups a warp. Two sixteens a group where the registers suffice: one's products run beside the
// other's arithmetic.
template <typename T, int DP, int NT>
struct FewPlan {
  static constexpr int WARPS = sizeof(T) == 4 || DP * NT == 256 ? 3 : NT == 2 ? 5 : 6;
  static constexpr int U = sizeof(T) == 2 && DP <= 128 && NT == 1 ? 2 : 1, GROUP = 16 * U;
  static constexpr int TILE = DP * 16;  // 16 tokens' K or V
  static constexpr int STAGE = 2 * U * TILE;
  static constexpr int Q = 8 * NT * DP * sizeof(T);
  // places for the warps' sums of eight rows, as far as there is room (with two of them where U is 2 for heads of 128, one
  // CTA an SM fits: 64 sequences 218 -> 300 us)
  static constexpr int SUMS = DP == 64 ? WARPS : U == 2 ? 1 : 2;
  static constexpr int AT_SUM = WARPS * 2 * STAGE, AT_Q = AT_SUM + SUMS * 8 * DP * 4, BYTES = AT_Q + 2 * Q + 1024;  // (alignment)
};
// A CTA's part of a tile and head, as the fetching warp tells the others.
struct Piece {
  int groups;                  // of the whole stretch of the line; 0: no more pieces
  int c0, c1, slot0;           // the CTAs that have parts of it, where the first of them keeps its own
  int b, begin, n, past, window;  // sequence, its first row, tokens, position, positions that a row sees
  int row0, g;                 // the tile's first row, head
  int from, to, first, final;  // tokens that count here, positions of the tile's first and last row
};
template <int WARPS, int GROUP>
struct FewShared {
  Scratch<WARPS + 1> scratch;
  Piece piece[2];
  uint64_t piece_full[2], piece_free[2], full[WARPS][2], free[WARPS][2];
  float k_factor[WARPS][2][GROUP], v_exponent[WARPS][2][GROUP];  // of each token's scales
  int held[WARPS][2];  // which sixteens of the group a page holds
};
// DP: dimensions that the registers have room for (64, 128, 256), FULL: head_dim is DP, NT: eights of rows.
template <typename T, int CODE, int DP, bool FULL, int NT>
__global__ void __launch_bounds__(32 * (FewPlan<T, DP, NT>::WARPS + 1), 2)
kv8_few(Kv8Args a, Kv8Parts f, const __grid_constant__ CUtensorMap map) {
  using P = FewPlan<T, DP, NT>;
  constexpr bool F32 = std::is_same<T, float>::value, BF = std::is_same<T, __nv_bfloat16>::value;
  constexpr int WARPS = P::WARPS, THREADS = 32 * WARPS, U = P::U, GROUP = P::GROUP;
  constexpr int QP = F32 ? 3 : 1, PP = BF ? 2 : 3;  // parts of q and of the weights
  constexpr int KJ = DP / 64, VJ = DP == 256 ? 2 : 1, MT = DP / 16;
  constexpr float MOST = 256.f;  // weights up to 2^8
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ FewShared<WARPS, GROUP> sh;
  __shared__ Stats stats[WARPS][8 * NT];
  static_assert(2 * (P::BYTES + sizeof(sh) + sizeof(stats) + 16 + 1024) <= 228 * 1024, "two CTAs an SM");
  const int D = FULL ? DP : a.D;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, qr = lane >> 2, qt = lane & 3;
  if (threadIdx.x < 2) {
    mbar_init(&sh.piece_full[threadIdx.x], 2);
    mbar_init(&sh.piece_free[threadIdx.x], WARPS);
  }
  if (threadIdx.x < 2 * WARPS) {
    mbar_init(&sh.full[0][0] + threadIdx.x, 2);
    mbar_init(&sh.free[0][0] + threadIdx.x, 1);
  }
  fence_mbar_init();
  __syncthreads();
  pdl_wait_prior_grids();
  const long long total = line_length<GROUP>(a, f.rows, &sh.scratch);
  // every warp 32 tokens at least: a call with few tokens is joined by few
  constexpr int LEAST = WARPS * 32 / GROUP;
  const int ctas = (int)min((long long)gridDim.x, (total + LEAST - 1) / LEAST), cta = blockIdx.x;
  if (cta >= ctas) return;
  const long long begin_line = begin_of(cta, total, ctas);
  long long in_seq = begin_line;
  const int b0 = find_place<GROUP>(a, f.rows, in_seq, &sh.scratch);
  bool ok = true;  // no wait of the warp has run out of time
  uint32_t round = 0;  // groups that the warp has had: its stage and the parity of the barriers

  if (warp == WARPS) {
    // ---- the warp that fetches: pieces, their rows of q, and a group for every warp in turn -------------
    const int page_mask = (1 << a.page_log) - 1, nb = 1 << (a.page_log - a.block_log);
    const int page_rows = (int)(a.page_bytes >> 7), head_rows = a.D << a.page_log >> 7;  // of 128 bytes
    const uint64_t policy = policy_evict_first();
    int b = b0;
    Seq s = seq_of<GROUP>(a, b, f.rows);
    constexpr int PAD = pad_of<GROUP>();
    const int start = (int)scaled(in_seq, 1, s.groups + PAD);
    int g = start % a.G, turn = start / a.G, j0 = (int)(in_seq - (long long)start * (s.groups + PAD));
    long long line = begin_line, left = begin_of(cta + 1, total, ctas) - begin_line;
    if (j0 >= s.groups) {  // (behind a stretch's groups: with the next one)
      const long long skip = min((long long)s.groups + PAD - j0, left);
      line += skip, left -= skip, j0 = 0;
      if (++g == a.G) g = 0, ++turn;
    }
    for (int k = 0; ok; ++k) {
      while (left > 0 && turn >= s.tiles) {  // the next sequence with rows
        s = seq_of<GROUP>(a, ++b, f.rows);
        turn = 0;
      }
      Piece x{};
      if (left > 0) {
        const int j1 = (int)min((long long)s.groups, j0 + left);  // groups j0 .. j1 - 1 of the stretch
        const long long line0 = line - j0;
        x.groups = s.groups;
        x.c0 = j0 == 0 ? cta : owner_of(line0, total, ctas);
        x.c1 = j1 == s.groups ? cta : owner_of(line0 + s.groups - 1, total, ctas);
        x.slot0 = part_slot(x.c0, x.c0, line0, total, ctas);
        x.b = b;
        x.begin = s.begin;
        x.n = s.n;
        x.past = s.past;
        x.window = s.window;
        x.row0 = (turn & 1 ? s.tiles - 1 - turn / 2 : turn / 2) * 8 * NT;
        x.g = g;
        x.first = s.past + x.row0 / a.rep;
        x.final = s.past + (x.row0 + (kv8_rows_left(s.n * a.rep, x.row0, 8 * NT) - 1)) / a.rep;
        x.from = max(max(x.first - s.window + 1, 0), s.base + j0 * GROUP);
        x.to = min(min(x.final + 1, s.end), s.base + j1 * GROUP);
        const long long gone = min((long long)s.groups + PAD - j0, left);
        line += gone;
        left -= gone;
        j0 = 0;
        if (++g == a.G) g = 0, ++turn;
      }
      const int ps = k & 1;
      if (k > 1) ok = __all_sync(0xffffffffu, mbar_wait(&sh.piece_free[ps], (k >> 1) - 1 & 1));
      if (!ok) break;
      const int rows = kv8_rows_left(x.n * a.rep, x.row0, 8 * NT);
      if (lane == 0) {
        sh.piece[ps] = x;
        mbar_arrive_expect_tx(&sh.piece_full[ps], x.groups ? rows * D * (int)sizeof(T) : 0);
        mbar_arrive(&sh.piece_full[ps]);
      }
      if (x.groups == 0) break;
      __syncwarp();
      if (lane < rows) {
        const int row = x.row0 + lane, i = row / a.rep;
        bulk_g2s(ring + P::AT_Q + ps * P::Q + lane * D * (int)sizeof(T),
                 static_cast<const T*>(a.q) + (int64_t)(x.begin + i) * a.qs + (x.g * a.rep + row - i * a.rep) * (int64_t)D,
                 D * (int)sizeof(T), &sh.piece_full[ps], policy);
      }
      // A lane looks up the page of one warp's sixteen, and the scales of one token (K's and V's; of groups of one sixteen,
      // K's on lanes 0 .. 15 and V's on the others) of each warp's group.
      const int32_t* table = a.pages + (int64_t)x.b * a.max_pages;
      const int g0 = x.from / GROUP, g1 = x.from < x.to ? (x.to + GROUP - 1) / GROUP : g0;
      auto page_of = [&](int grp) {
        const int t = (grp + lane / U) * GROUP + lane % U * 16;
        int id = -1;
        if (lane < WARPS * U && t < x.to) id = table[t >> a.page_log];
        return id < a.n_pages ? id : -1;
      };
      auto scales_of = [&](int pages, int grp, int(&v)[WARPS][U]) {
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const int page = __shfl_sync(0xffffffffu, pages, w * U + (U == 1 ? 0 : lane >> 4));
          const int at = ((grp + w) * GROUP + (U == 1 ? lane & 15 : lane)) & page_mask;
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int which = U == 1 ? lane >> 4 : i;
            v[w][i] = 0;
            if (page >= 0) v[w][i] = a.cache[page * a.page_bytes + a.scales_at + (2 * x.g + which) * nb + (at >> a.block_log)];
          }
        }
      };
      int pages = page_of(g0), ahead = page_of(g0 + WARPS), sc[WARPS][U];
      scales_of(pages, g0, sc);
      for (int grp = g0; grp < g1 && ok; grp += WARPS, ++round) {
        const int st = round & 1;
        const int next = ahead;
        ahead = page_of(grp + 2 * WARPS);
        bool in_time = true;
        if (round > 1 && lane < WARPS) in_time = mbar_wait(&sh.free[lane][st], (round >> 1) - 1 & 1);
        ok = __all_sync(0xffffffffu, in_time);
        // lane w tells warp w's barrier what comes; lane w U + u copies K of its sixteen u, lane 16 + w U + u V
        const uint32_t held = __ballot_sync(0xffffffffu, pages >= 0);
        if (lane < WARPS && ok) {
          const int mine = held >> lane * U & ((1 << U) - 1);
          sh.held[lane][st] = mine;
          mbar_arrive_expect_tx(&sh.full[lane][st], __popc(mine) * 32 * D);
        }
        const int page = __shfl_sync(0xffffffffu, pages, lane & 15);
        if ((lane & 15) < WARPS * U && page >= 0 && ok) {
          const int w = (lane & 15) / U, u = (lane & 15) % U, v = lane >> 4;
          const int at = ((grp + w) * GROUP + 16 * u) & page_mask;
          copy_rows(ring + (w * 2 + st) * P::STAGE + (v * U + u) * P::TILE, &map,
                    page * page_rows + (2 * x.g + v) * head_rows + (at * D >> 7), &sh.full[w][st]);
        }
        if (!ok) break;
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          // factors of the scores (kv8_power, in the fewest operations: all warps wait for this one), exponents of the values
          auto k_of = [&](int x) { return x == 255 ? nan : __uint_as_float(max((uint32_t)x << 23, 0x400000u)); };
          auto v_of = [&](int x) { return x == 255 ? nan : (float)(x - 127); };
          if constexpr (U == 1) {
            if (lane < 16) sh.k_factor[w][st][lane] = k_of(sc[w][0]);
            else sh.v_exponent[w][st][lane - 16] = v_of(sc[w][0]);
          } else {
            sh.k_factor[w][st][lane] = k_of(sc[w][0]);
            sh.v_exponent[w][st][lane] = v_of(sc[w][U - 1]);
          }
        }
        __syncwarp();
        if (lane < WARPS) mbar_arrive(&sh.full[lane][st]);
        pages = next;
        if (grp + WARPS < g1) scales_of(pages, grp + WARPS, sc);
      }
    }
    if (!ok && lane == 0) atomicOr(f.ctrl + CTRL_STATUS, DEV_ERR_MBAR_TIMEOUT);
    return;
  }

  // ---- the warps that work ---------------------------------------------------------------------------
  // Where the lane's operands are in a tile, rows of 128 bytes whose 16-byte pieces are exchanged by the row's number (the
  // 128-byte swizzle), so that no two lanes of a read meet in a bank: of K, 16 dimensions times KJ from dimension 16 KJ qt
  // on of tokens qr and qr + 8; of V, 16 dimensions (8 of narrow heads) of every 128, of tokens 2 qt, 2 qt + 1 and the
  // same + 8. Dimensions that the head does not have are some that it has: their q is 0, their outputs go nowhere.
  auto place = [&](int token, int at) {  // of byte `at` of a token
    const int x = token * D + at;
    return x ^ ((x >> 7 & 7) << 4);
  };
  int k_at[2][KJ], v_at[4][VJ];
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int j = 0; j < KJ; ++j) k_at[e][j] = place(qr + 8 * e, FULL ? (qt * KJ + j) * 16 : min((qt * KJ + j) * 16, D - 16));
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int j = 0; j < VJ; ++j) {
      const int at = DP == 64 ? qr * 8 : j * 128 + qr * 16;
      v_at[e][j] = place(2 * qt + (e & 1) + (e >> 1) * 8, FULL ? at : min(at, DP == 64 ? D - 8 : D - 16));
    }
  auto workers_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); };
  float* const sum = reinterpret_cast<float*>(ring + P::AT_SUM);  // [SUMS][8][DP]

  for (int k = 0;; ++k) {
    const int ps = k & 1;
    ok = ok && mbar_wait(&sh.piece_full[ps], k >> 1 & 1);
    {
      uint32_t all_ok;
      asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
                   : "=r"(all_ok) : "r"((uint32_t)ok), "n"(THREADS) : "memory");
      if (!all_ok) break;
    }
    const Piece& pc = sh.piece[ps];
    if (pc.groups == 0) break;
    const int row0 = pc.row0, rows = pc.n * a.rep - pc.row0, from = pc.from, to = pc.to, first = pc.first, final = pc.final;

    // ---- q ----
    uint32_t qf[QP][NT][KJ * 4][2];
    // A score is its sum times a factor of the row, K's scale and another factor of the row: no product of three of them
    // leaves f32 on its way to a score that does not.
    float rf[NT][2], rf2[NT][2];
    int pos[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const T* q = reinterpret_cast<const T*>(ring + P::AT_Q + ps * P::Q) + (8 * n + qr) * D;
      float x[KJ][16];
      float top = 0.f;
      bool finite = true;
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int at = (qt * KJ + j) * 16;
          const bool in = 8 * n + qr < rows && (FULL || at < D);
          const float4 v = in ? load4(q + at + 4 * w) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[j][4 * w] = v.x, x[j][4 * w + 1] = v.y, x[j][4 * w + 2] = v.z, x[j][4 * w + 3] = v.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            finite = finite && fabsf(x[j][4 * w + e]) <= 3.402823466e38f;
            top = fmaxf(top, fabsf(x[j][4 * w + e]));
          }
        }
      float mul = 1.f, inv = 1.f;
      if constexpr (BF || F32) {  // the row's largest to 2^14 .. 2^15
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(__float_as_uint(top) >> 23), 16), 254);
        mul = __uint_as_float((uint32_t)(268 - e) << 23);
        inv = __uint_as_float((uint32_t)(e - 14) << 23);
      }
      const uint32_t good = __ballot_sync(0xffffffffu, finite);
      if ((good >> (qr * 4) & 15u) != 15u) inv = __uint_as_float(0x7fc00000u);  // the row's scores are NaN
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          uint32_t p[QP];
          split_pair<QP, F32>(x[j][2 * w] * mul, x[j][2 * w + 1] * mul, p);
#pragma unroll
          for (int k = 0; k < QP; ++k) qf[k][n][j * 4 + w / 2][w & 1] = p[k];
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float factor = __shfl_sync(0xffffffffu, inv, (2 * qt + c) * 4);
        rf[n][c] = factor > 1.f ? 1.f : factor;
        rf2[n][c] = fminf(fmaxf(fmaxf(factor, 1.f) * a.scale * 1.44269504f, -3e38f), 3e38f);
        pos[n][c] = pc.past + (row0 + min(8 * n + 2 * qt + c, rows - 1)) / a.rep;
      }
    }

    // ---- tokens ----
    float m[NT][2], E[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = LOWEST;
      E[n][0] = E[n][1] = l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
    // groups that every row sees whole
    const int window = pc.window, whole0 = max((from + GROUP - 1) / GROUP, ((final - window) >> (U + 3)) + 1);
    const int whole1 = min((first + 1) / GROUP, to / GROUP);
    auto work = [&](int st, int held, int grp) {
      const uint8_t* src = ring + (warp * 2 + st) * P::STAGE;
      const bool whole = grp >= whole0 && grp < whole1 && held == (1 << U) - 1;
      float sc[U][NT][4], ev[U][2];  // scores of token qr + 8 (e >> 1), row 2 qt + (e & 1); exponents of V's scales
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // several accumulators: a chain of products waits for each one's latency
        constexpr int SN = QP == 1 && NT * U == 1 ? 4 : 2;
        float S[SN][NT][4];
#pragma unroll
        for (int x = 0; x < SN; ++x)
#pragma unroll
          for (int n = 0; n < NT; ++n) S[x][n][0] = S[x][n][1] = S[x][n][2] = S[x][n][3] = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          const uint4 u0 = *reinterpret_cast<const uint4*>(src + u * P::TILE + k_at[0][j]);
          const uint4 u1 = *reinterpret_cast<const uint4*>(src + u * P::TILE + k_at[1][j]);
          const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t x = code_word<CODE>(w0[w]), y = code_word<CODE>(w1[w]);
            const uint32_t A[4] = {pair_of<CODE, F32>(x, false), pair_of<CODE, F32>(y, false), pair_of<CODE, F32>(x, true),
                                   pair_of<CODE, F32>(y, true)};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < QP; ++p) mma<F32>(S[QP == 1 ? w % SN : p != 0][n], A, qf[p][n][j * 4 + w]);
          }
        }
        float kf[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          kf[e] = sh.k_factor[warp][st][16 * u + qr + 8 * e];
          ev[u][e] = sh.v_exponent[warp][st][16 * u + qr + 8 * e];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = S[0][n][e] + S[1][n][e];
            if constexpr (SN == 4) x += S[2][n][e] + S[3][n][e];
            sc[u][n][e] = x * rf[n][e & 1] * kf[e >> 1] * rf2[n][e & 1];
          }
      }
      if (!whole) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = grp * GROUP + 16 * u + qr + 8 * (e >> 1), p = pos[n][e & 1];
              if (!(held >> u & 1) || t < from || t >= to || t > p || t <= p - window) sc[u][n][e] = -INFINITY;
            }
      }
      float w1[U][NT][4], wv[U][NT][4];  // weights in the sum, and as V's operands
      auto weigh = [&]() {
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float d = sc[u][n][e] - m[n][e & 1];
              w1[u][n][e] = ex2(d);
              wv[u][n][e] = ex2(d + (ev[u][e >> 1] - E[n][e & 1]));
              top = fmaxf(top, fmaxf(w1[u][n][e], wv[u][n][e]));
            }
        return top > MOST;
      };
      if (__any_sync(0xffffffffu, weigh())) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
            float top = -INFINITY, vtop = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) top = fmaxf(top, fmaxf(sc[u][n][c2], sc[u][n][2 + c2]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float m1 = fmaxf(m[n][c2], top);
            // exponents beside the distance to m1: a large score has steps beyond them
#pragma unroll
            for (int u = 0; u < U; ++u)
              vtop = fmaxf(vtop, fmaxf(sc[u][n][c2] - m1 + ev[u][0], sc[u][n][2 + c2] - m1 + ev[u][1]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, x));
            if (m1 > LOWEST) {
              const float dm = m[n][c2] - m1, E1 = ceilf(fmaxf(dm + E[n][c2], vtop));
              const float keep = ex2(dm + (E[n][c2] - E1));
              l[n][c2] *= ex2(dm);
              m[n][c2] = m1;
              E[n][c2] = E1;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[i][n][c2] *= keep;
                o[i][n][2 + c2] *= keep;
              }
            }
          }
        weigh();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t pf[PP][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {  // tokens qr + 8 e
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
              l[n][c2] += w1[u][n][2 * e + c2];
              if (!whole && sc[u][n][2 * e + c2] == -INFINITY) wv[u][n][2 * e + c2] = 0.f;  // (a NaN scale behind the mask)
            }
            uint32_t h[PP];
            split_pair<PP, true>(wv[u][n][2 * e], wv[u][n][2 * e + 1], h);
#pragma unroll
            for (int k = 0; k < PP; ++k) pf[k][n][e] = transpose8(h[k]);
          }
        auto value_tile = [&](int i, uint32_t lo, uint32_t hi) {  // words of tokens (2 qt, + 1) and (2 qt + 8, + 9)
          const uint32_t A[4] = {pair_of<CODE, true>(lo, false), pair_of<CODE, true>(lo, true), pair_of<CODE, true>(hi, false),
                                 pair_of<CODE, true>(hi, true)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            // The products' accumulator cuts bits off, always towards 0: f32 rows' sums go through it for one sixteen at a
            // time only (1,524 tokens, 16 heads of 128: 175 us -> 188, outputs 4.8e-7 -> 1.9e-7 off, long ones 3.2e-6 -> 5.6e-7)
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            float(&sum)[4] = F32 ? t : o[i][n];
#pragma unroll
            for (int k = PP - 1; k >= 0; --k) mma<true>(sum, A, pf[k][n]);
            if constexpr (F32) {
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][n][e] += t[e];
            }
          }
        };
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
          uint32_t w[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint8_t* p = src + (U + u) * P::TILE + v_at[e][j];
            if constexpr (DP == 64) {
              const uint2 x = *reinterpret_cast<const uint2*>(p);
              w[e][0] = x.x, w[e][1] = x.y, w[e][2] = 0, w[e][3] = 0;
            } else {
              const uint4 x = *reinterpret_cast<const uint4*>(p);
              w[e][0] = x.x, w[e][1] = x.y, w[e][2] = x.z, w[e][3] = x.w;
            }
            if (CODE == MOE_E4M3 && !whole) {  // what lies behind the tokens may be no number, and would not go with a weight of 0
              const int t = grp * GROUP + 16 * u + 2 * qt + (e & 1) + (e >> 1) * 8;
              if (!(held >> u & 1) || t < from || t >= to) w[e][0] = w[e][1] = w[e][2] = w[e][3] = 0;
            }
          }
#pragma unroll
          for (int x = 0; x < (DP == 64 ? 2 : 4); ++x) {
            // [a0 b0 a1 b1], [a2 b2 a3 b3] of the two tokens
            const uint32_t lo = __byte_perm(w[0][x], w[1][x], 0x5140), lo2 = __byte_perm(w[0][x], w[1][x], 0x7362);
            const uint32_t hi = __byte_perm(w[2][x], w[3][x], 0x5140), hi2 = __byte_perm(w[2][x], w[3][x], 0x7362);
            value_tile(j * 8 + 2 * x, code_word<CODE>(lo), code_word<CODE>(hi));
            value_tile(j * 8 + 2 * x + 1, code_word<CODE>(lo2), code_word<CODE>(hi2));
          }
        }
      }
    };
    const int g0 = from / GROUP, g1 = from < to ? (to + GROUP - 1) / GROUP : g0;
    for (int grp = g0; grp < g1; grp += WARPS, ++round) {  // (all warps as often)
      const int st = round & 1;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sh.full[warp][st], round >> 1 & 1));
      if (ok) {
        const int held = sh.held[warp][st];
        if (held) work(st, held, grp + warp);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.free[warp][st]);
    }

    // ---- the warps' sums ----
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][c2] += __shfl_xor_sync(0xffffffffu, l[n][c2], x);
        if (qr == 0) stats[warp][8 * n + 2 * qt + c2] = Stats{m[n][c2], E[n][c2], l[n][c2], 0.f};
      }
    workers_sync();
    Stats all[NT][2];
    float keep[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        float M = LOWEST, top = LOWEST, L = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const Stats& x = stats[w][8 * n + 2 * qt + c2];
          M = fmaxf(M, x.m);
        }
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const Stats& x = stats[w][8 * n + 2 * qt + c2];
          L = fmaf(x.l, ex2(x.m - M), L);
          top = fmaxf(top, x.m - M + x.E);
        }
        const float E1 = M == LOWEST ? 0.f : ceilf(top);
        keep[n][c2] = ex2((m[n][c2] - M) + (E[n][c2] - E1));
        all[n][c2] = Stats{M, E1, L, 0.f};
      }
    const bool own = pc.c0 == pc.c1;
    const int64_t part = (int64_t)(cta == pc.c0 ? pc.slot0 : 2 * cta) * f.rows;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int w0 = 0; w0 < WARPS; w0 += P::SUMS) {  // always in the same order
        workers_sync();
        if (warp < w0 || warp >= w0 + P::SUMS) continue;
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const int d = (DP == 64 ? qr * 8 : i / 8 * 128 + qr * 16) + 2 * (i % 8);
            float2* p = reinterpret_cast<float2*>(sum + (warp - w0) * 8 * DP + (2 * qt + c2) * DP + d);
            const float x = o[i][n][c2] * keep[n][c2], y = o[i][n][2 + c2] * keep[n][c2];
            *p = w0 == 0 ? make_float2(x, y) : make_float2(p->x + x, p->y + y);
          }
        if (warp == 0 && qr == 0) {
          stats[0][8 * n + 2 * qt] = all[n][0];
          stats[0][8 * n + 2 * qt + 1] = all[n][1];
        }
      }
      workers_sync();
      for (int i = threadIdx.x; i < 8 * D / 4; i += THREADS) {
        const int r8 = i * 4 / D, d = i * 4 - r8 * D, r = 8 * n + r8;
        float4 x = *reinterpret_cast<const float4*>(sum + r8 * DP + d);
#pragma unroll
        for (int w = 1; w < min(P::SUMS, WARPS); ++w) {
          const float4 y = *reinterpret_cast<const float4*>(sum + (w * 8 + r8) * DP + d);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const Stats st = stats[0][r];
        if (!own) {
          __stcg(reinterpret_cast<float4*>(f.parts + (part + r) * D + d), x);
          if (d == 0) __stcg(reinterpret_cast<float4*>(f.stats + part + r), make_float4(st.m, st.E, st.l, 0.f));
          continue;
        }
        int h = 0;
        T* out = out_row<T>(a, pc.begin, pc.n, pc.g, row0, r, h);
        if (!out) continue;
        store4(out + d, row_scale(a, h, st), x);
      }
    }
    if (!own)
      join_stretch<T, KV8_CTAS>(a, f, THREADS, pc.begin, pc.n, row0, pc.g, pc.c0, pc.c1, pc.slot0, &sh.scratch.last,
                                workers_sync);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.piece_free[ps]);
    workers_sync();  // sum and stats may be used again
  }
  if (!ok) {  // a copy did not come in time: none may be in flight when the CTA ends
    if (lane == 0) atomicOr(f.ctrl + CTRL_STATUS, DEV_ERR_MBAR_TIMEOUT);
    for (int st = 0; st < 2; ++st) {
      mbar_wait(&sh.full[warp][st], round + st >> 1 & 1);
      mbar_wait(&sh.piece_full[st], 0);
    }
  }
  pdl_launch_dependents();
}

// The cache as rows of 128 bytes, in boxes of 16 tokens' K or V (records and heads are whole rows), swizzled. A pool
// without pages has none to copy.
inline cudaError_t cache_map(CUtensorMap* m, const Kv8Args& a) {
  *m = CUtensorMap{};
  if (a.n_pages == 0) return cudaSuccess;
  const auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {128, (cuuint64_t)(a.page_bytes / 128 * a.n_pages)}, strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)a.D / 8}, es[2] = {1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.cache, dims, strides, box, es,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
template <typename T, int CODE, int DP, bool FULL, int NT>
cudaError_t few_launch(const Kv8Args& a, const Kv8Parts& f, bool pdl, cudaStream_t st) {
  using P = FewPlan<T, DP, NT>;
  CUtensorMap map;
  const cudaError_t me = cache_map(&map, a);
  if (me != cudaSuccess) return me;
  const auto kern = kv8_few<T, CODE, DP, FULL, NT>;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), P::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(KV8_CTAS);
  cfg.blockDim = dim3(32 * (P::WARPS + 1));
  cfg.dynamicSmemBytes = P::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, f, map);
}
template <typename T, int CODE, int DP, bool FULL>
cudaError_t few_rows(const Kv8Args& a, const Kv8Parts& f, bool pdl, cudaStream_t st) {
  if constexpr (DP < 256)
    if (f.rows == 16) return few_launch<T, CODE, DP, FULL, 2>(a, f, pdl, st);
  return few_launch<T, CODE, DP, FULL, 1>(a, f, pdl, st);
}
template <typename T, int CODE>
cudaError_t few_dims(const Kv8Args& a, const Kv8Parts& f, bool pdl, cudaStream_t st) {
  // f32, whose time goes into its parts' products, has the one form for any width
  if constexpr (sizeof(T) == 2) {
    if (a.D == 64) return few_rows<T, CODE, 64, true>(a, f, pdl, st);
    if (a.D == 128) return few_rows<T, CODE, 128, true>(a, f, pdl, st);
    if (a.D == 256) return few_rows<T, CODE, 256, true>(a, f, pdl, st);
  }
  if (a.D <= 64) return few_rows<T, CODE, 64, false>(a, f, pdl, st);
  if (a.D <= 128) return few_rows<T, CODE, 128, false>(a, f, pdl, st);
  return few_rows<T, CODE, 256, false>(a, f, pdl, st);
}

}  // namespace

// For each type, both codes (one source each, so that they compile beside each other).
template <typename T>
cudaError_t kv8_few_launch(const Kv8Args& a, const Kv8Parts& f, bool pdl, cudaStream_t st) {
  return a.code == MOE_I8 ? few_dims<T, MOE_I8>(a, f, pdl, st) : few_dims<T, MOE_E4M3>(a, f, pdl, st);
}

}  // namespace moe
