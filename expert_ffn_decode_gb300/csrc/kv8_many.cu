// Attention over the 8-bit cache for many rows a key/value head: prompts. Bound by the tensor cores and by what
// feeds them: every code becomes a 16-bit operand once for 256 rows.
//
// A CTA works on two tiles of up to 128 rows (tokens x the heads that share a key/value head) of one head, 128
// tokens of the cache at a time, on
//   S [rows][tokens] = Q K^T      O [rows][dim] += P V
// with S, the weights P (over S, packed) and O in tensor memory, a row a lane. Its warps:
//   0 .. 7, 8 .. 15    softmax of tile 0 and of tile 1, two threads a row: one tile's arithmetic beside the other's products
//   16 .. 19, 20 .. 23  K's codes to f16 operands, V's to bf16 ones, in the 128-byte swizzle
//   24, 25             the warp that copies (codes, q), the one that issues products
// K and V alternate through three places for codes and three for operands. Scales are powers of two and go into the
// operands: K times 2^5 over the largest K scale of the 128 tokens as f16, exact for scales down to 2^-29 of that (of e4m3's
// smallest codes to 2^-20; where one is smaller, no scale of the group goes in, and scores get theirs one by one), V as bf16
// in units that depend on the largest V scale the CTA has seen for the tiles: exact, whatever the others, while that one is at
// most 2^49, and for scales down to 2^-170 of a larger one. (Scales beside the operands, read from shared memory for each
// score, took 505 us where this took 395 with weights of one part: 512 tokens x 32 heads behind 32,768.) bf16 rows of q
// become f16 ones in place, times a power of two a row.
// Softmax keeps a reference m of a row's scores that is only raised when a score exceeds it by 16 (powers of two); then,
// and when V's unit rises, the row of O is scaled in tensor memory. A group's scores are read twice: for the largest, which
// says whether the reference does, and for the weights, which are made over them.
// As operands weights are two bf16 parts: 16 bits of each, however small it is beside the row's largest. Half of them
// (32 of each thread's 64 tokens) are handed over at a time, so that their products, twice as many, run beside the others'
// arithmetic. (One f16 part takes 2.74 ms for a 16,384-token prompt where this takes 3.12, but has 11 bits down to 2^-17 of
// the largest weight, fewer below and none from 2^-28 on, which is where the tokens behind a first one are that has nearly all
// weight and next to no value, as in trained models. Handed over all at once, 3.31.)
//
// No unit is full (counters of 512 tokens x 32 heads behind 32,768 tokens, 367 us: issue slots 58%, tensor pipe 47%, shared
// memory 34%): a tile's chain of products, weights and products is what a group's 6,300 cycles go into. Whole prompts wait
// for their busiest CTA besides, as a tile's place on the line has the groups that any row of the sequence sees: 1,032
// groups for 16,384 tokens where the mean is 869, twice the mean for 2,048 to 8,192 (145, 387 and 1,447 us).
// With weights of one f16 part S in halves of 64 tokens with two places a tile, products beside weights, took 3.1 ms for
// 16,384 tokens where one place took 2.73 (N = 64 reads q twice as often); all eight converting warps on K, then V, 2.92.
//
// The CTAs cut one line of all sequences' tiles, heads and groups of tokens into equal pieces, as in kv8_few.cuh.
#include <cuda.h>

#include <cstddef>
#include <type_traits>

#include "kv8_line.cuh"
#include "tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int TOK = 128;  // tokens of a group
constexpr int SOFTMAX = 512, THREADS = SOFTMAX + 384;
constexpr uint32_t HALF = 16384;  // 128 rows of 128 bytes: 64 dimensions of an operand of 128 rows
constexpr float SLACK = 16.f;  // weights of up to 2^16: more would take from the powers below that parts and sinks are added by
// V's operands are in units of 2^(unit - 127), unit a multiple of 16 that the largest scale byte is at most HEAD above: sums
// of 2^30 weights of 2^SLACK times codes of 2^9 stay f32 numbers.
constexpr int HEAD = 64;
constexpr int FAR = 1 << 20;
constexpr uint32_t T_S = 0, T_O = 256;  // tensor memory: 128 columns a tile each

template <int DP>
struct Plan {
  static constexpr uint32_t HALVES = DP / 64, OPERAND = HALVES * HALF;
  static constexpr uint32_t Q = 0, OPS = 2 * OPERAND, RAW = OPS + 3 * OPERAND, RAW_SIZE = TOK * DP;
  static constexpr uint32_t BYTES = RAW + 3 * RAW_SIZE + 1024;  // (alignment)
};
// A CTA's part of a tile pair and head, as the copying warp tells the others.
struct Piece {
  int groups;                  // of the whole stretch of the line; 0: no more pieces
  int c0, c1, slot0;           // the CTAs that have parts of it, where the first of them keeps its own
  int b, begin, n, past, window;  // sequence, its first row, tokens, position, positions that a row sees
  int row0, g;                 // the first of the rows, head
  int from, to;                // tokens that count here
  int g0, g1;                  // groups with some
};
struct alignas(16) Shared {
  Scratch<THREADS / 32> scratch;
  Piece piece[2];
  uint64_t piece_full[2], piece_free[2], q_full, q_ready, q_free, raw_full[3], raw_free[3], op_full[3], op_free[3], s_full[2],
      p_ready[2][2], o_full[2];
  uint32_t tmem;
  int top[2][2][4], low[2][4];     // largest scale byte of a warp's tokens, K and V, smallest of K
  int E[2];                        // of V for a group: what O is in units of
  int s_exp[2];                    // its scores are sums times 2^s_exp; where K's scales are too far apart for that, FAR
  alignas(4) uint8_t k_byte[2][TOK];  // and each token's times its own scale
  alignas(16) uint32_t valid[2][2][4];  // tokens that count, as K's and V's warps found
  alignas(16) uint32_t nan[2][2][4];    // those of them with a NaN scale
  uint32_t scale[2][2][TOK];       // what a token's codes are multiplied with, as a pair of operands: K's f16, V's bf16
  float row[2][2][128];            // a row's two threads: their largest scores, their sums
};

static_assert(offsetof(Shared, valid) % 16 == 0 && offsetof(Shared, nan) % 16 == 0, "read sixteen bytes at a time");

__device__ __forceinline__ uint32_t idesc(int n, bool bf16, bool b_mn) {  // operands f16 or bf16, both of them
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 | 8u << 24;
}
__device__ __forceinline__ uint64_t desc_sw128(const uint8_t* p, uint32_t lbo) {
  return (smem_desc(p, lbo, 1024) & ~((uint64_t)7 << 61)) | (uint64_t)2 << 61;
}
// Products with operands in shared memory, and with A in tensor memory: descriptors by their low words, as one thread
// issues all of a CTA's products and has few instructions for each.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t tmem_a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.u32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d),
      "r"(tmem_a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n)); }
template <int n>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n)); }
__device__ __forceinline__ void copy_bytes(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void copy_q(void* dst, const CUtensorMap* map, int x, int head, int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(head), "r"(token)
      : "memory");
}
// Pairs of f32: a b + c, a + b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Codes 2 hi, 2 hi + 1 of a word times a power of two (as a pair), in f16 or bf16.
template <int CODE, bool BF16>
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, bool hi, uint32_t f) {
  if constexpr (BF16) {
    if constexpr (CODE == MOE_I8) {  // as pair_of, times f: f (u - 256) - f / 2 max(u - 256, 0)
      auto v = [](const uint32_t& x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
      const uint32_t u = __byte_perm(w, 0x43434343u, hi ? 0x4342 : 0x4140), one = 0x3f803f80u, off = 0xc380c380u, half = 0xbf00bf00u;
      const __nv_bfloat162 twice = __hfma2_relu(v(u), v(one), v(off));
      const __nv_bfloat162 z = __hfma2(twice, __hmul2(v(f), v(half)), __hfma2(v(u), v(f), __hmul2(v(f), v(off))));
      return *reinterpret_cast<const uint32_t*>(&z);
    }
    const uint32_t x = pair_of<CODE, true>(w, hi);
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&f));
    return *reinterpret_cast<const uint32_t*>(&y);
  }
  const __half2 s = *reinterpret_cast<const __half2*>(&f);
  __half2 y;
  if constexpr (CODE == MOE_I8) {  // 1024 + 128 + code, less 1152, in one operation
    const uint32_t u = __byte_perm(w, 0x64646464u, hi ? 0x4342 : 0x4140);
    y = __hfma2(*reinterpret_cast<const __half2*>(&u), s, __hmul2(s, __float2half2_rn(-1152.f)));
  } else {
    const uint32_t x = pair_of<CODE, false>(w, hi);
    y = __hmul2(*reinterpret_cast<const __half2*>(&x), s);
  }
  return *reinterpret_cast<const uint32_t*>(&y);
}
// Two weights as two bf16 parts each.
__device__ __forceinline__ void two_parts(float2 w, uint32_t& big, uint32_t& small) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(big) : "f"(w.y), "f"(w.x));
  const float2 rest = fma2(make_float2(__uint_as_float(big << 16), __uint_as_float(big & 0xffff0000u)), make_float2(-1.f, -1.f), w);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(small) : "f"(rest.y), "f"(rest.x));
}
// 2^n for n up to 127, 0 below 2^-149.
__device__ __forceinline__ float power_of(int n) {
  return __uint_as_float(n >= -126 ? (uint32_t)(n + 127) << 23 : n >= -149 ? 1u << (n + 149) : 0u);
}
// scale * 2^n, the exponents of q and K added up first: neither's power alone need be an f32 number. (Sums below 2^35 make
// scores of no more than 2^-90 with what is 0 here; from 2^120 on scores are not told apart.)
__device__ __forceinline__ float score_factor(float scale, int n) {
  n = max(min(n, 120), -250);
  return __uint_as_float((uint32_t)((n >> 1) + 127) << 23) * scale * __uint_as_float((uint32_t)(n - (n >> 1) + 127) << 23);
}
template <int threads>
__device__ __forceinline__ bool all_of(int barrier, bool x) {  // whether x holds for all of some warps' threads
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(r) : "r"((uint32_t)x), "r"(barrier), "n"(threads) : "memory");
  return r != 0;
}

// half_tokens: tokens of a tile of 128 rows.
template <typename T, int CODE, int DP>
__global__ void __launch_bounds__(THREADS, 1)
kv8_many(Kv8Args a, Kv8Parts f, int half_tokens, const __grid_constant__ CUtensorMap q_map) {
  using P = Plan<DP>;
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int D = a.D, half_rows = half_tokens * a.rep;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.piece_full[i], 1);
      mbar_init(&sh.piece_free[i], SOFTMAX + 256 + 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i][0], SOFTMAX / 2);
      mbar_init(&sh.p_ready[i][1], SOFTMAX / 2);
      mbar_init(&sh.o_full[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_free[i], 128);
      mbar_init(&sh.op_full[i], 128);
      mbar_init(&sh.op_free[i], 1);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_ready, SOFTMAX);
    mbar_init(&sh.q_free, SOFTMAX + 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait_prior_grids();
  const long long total = line_length<TOK>(a, f.rows, &sh.scratch);
  const int ctas = (int)min((long long)gridDim.x, total), cta = blockIdx.x;
  if (cta >= ctas) return;
  const long long begin_line = begin_of(cta, total, ctas);
  long long in_seq = begin_line;
  const int b0 = find_place<TOK>(a, f.rows, in_seq, &sh.scratch);
  if (warp == 25) tmem_alloc(&sh.tmem, 512);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = sh.tmem;
  bool ok = true;  // no wait of the thread has run out of time

  if (warp < SOFTMAX / 32) {
    // ---- softmax: half of a row's tokens a thread -------------------------------------------------------------
    more_registers<96>();
    const int h = warp >> 3, part = warp >> 2 & 1, r = tid & 127;  // tile, half of the tokens, row of the tile
    const uint32_t lanes = tm + ((uint32_t)(warp & 3) * 32u << 16);
    const uint32_t t_s = lanes + T_S + h * 128 + part * 64, t_o = lanes + T_O + h * 128;  // weights: over the first half of t_s
    const float scale2 = fabsf(a.scale) * 1.44269504f;
    uint32_t group = 0, filled = 0;          // groups and pieces with some so far
    auto rows_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(SOFTMAX) : "memory"); };
    const int pair = 4 + h * 4 + (warp & 3);  // the barrier of the two warps that share rows
    auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory"); };
    for (int k = 0;; ++k) {
      ok = all_of<SOFTMAX>(1, ok && mbar_wait(&sh.piece_full[k & 1], k >> 1 & 1));
      if (!ok) break;
      const Piece& pc = sh.piece[k & 1];
      if (pc.groups == 0) break;
      const int first = pc.past + pc.row0 / a.rep + h * half_tokens;  // position of the tile's first row
      const int pos = first + r / a.rep, from = max(pos - pc.window + 1, 0);  // of the tokens that the row sees
      const int t_last = first + half_tokens - 1;  // of the tile's last row
      const int left = pc.n * a.rep - pc.row0 - h * half_rows;  // rows from the tile's first on
      const bool real = r < half_rows && r < left, tile_real = left > 0;
      float m = 0.f, l = 0.f;
      int q_exp = 0;  // rows of q are their operands times 2^q_exp
      bool fresh = true;  // has seen no token
      int E = 0;
      const int n_groups = pc.g1 - pc.g0;
      if (n_groups > 0) {
        ok = ok && mbar_wait(&sh.q_full, filled & 1);
        // A row of q that is not finite gives a row that is not. bf16 rows become f16 ones, times a power of two that
        // takes their largest to 2^14 .. 2^15: as they are down to 2^-29 of it, and less than 2^-39 of it off below.
        uint8_t* q = sm + P::Q + h * P::OPERAND + r * 128;
        auto piece = [&](int c) { return reinterpret_cast<uint4*>(q + (c >> 3) * HALF + ((c ^ r) & 7) * 16); };
        uint32_t most = 0;
        if (real && ok) {
#pragma unroll 1
          for (int c = part; c < DP / 8; c += 2) {
            const uint4 u = *piece(c);
            most = __vmaxu2(__vmaxu2(most, __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu)),
                            __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
          }
          most = max(most & 0xffffu, most >> 16);
          if (most >= (BF ? 0x7f80u : 0x7c00u)) l = __uint_as_float(0x7fc00000u);
        }
        if constexpr (BF) {
          sh.row[h][part][r] = __uint_as_float(most);
          pair_sync();
          const int e = min(max((int)(max(most, __float_as_uint(sh.row[h][part ^ 1][r])) >> 7), 16), 254);
          const float mul = __uint_as_float((uint32_t)(268 - e) << 23);
          q_exp = e - 141;
          if (real && ok) {
#pragma unroll 1
            for (int c = part; c < DP / 8; c += 2) {
              uint4 u = *piece(c);
              auto half_of = [&](uint32_t x) {
                uint32_t y;
                asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(__uint_as_float(x & 0xffff0000u) * mul), "f"(__uint_as_float(x << 16) * mul));
                return y;
              };
              *piece(c) = make_uint4(half_of(u.x), half_of(u.y), half_of(u.z), half_of(u.w));
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&sh.q_ready);
        }
        mbar_arrive(&sh.q_free);
      }
      for (int j = 0; j < n_groups; ++j, ++group) {
        const int t0 = (pc.g0 + j) * TOK, par = group & 1;
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&sh.s_full[h], group & 1));
        tc_fence_after_sync();
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&sh.op_full[(2 * group + 1) % 3], (2 * group + 1) / 3 & 1));  // E is there
        const uint4 valid = *reinterpret_cast<const uint4*>(sh.valid[0][par]);
        const uint4 nk = *reinterpret_cast<const uint4*>(sh.nan[0][par]), nv = *reinterpret_cast<const uint4*>(sh.nan[1][par]);
        const bool whole = (valid.x & valid.y & valid.z & valid.w) == ~0u && t0 + TOK - 1 <= first && t0 > t_last - pc.window &&
                           sh.s_exp[par] != FAR && (nk.x | nk.y | nk.z | nk.w | nv.x | nv.y | nv.z | nv.w) == 0;
        if (!tile_real || t0 > t_last || t0 + TOK - 1 <= first - pc.window) {  // the mask leaves the tile's rows nothing here
          uint32_t z[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = 0;
#pragma unroll
          for (int c = 0; c < 64; c += 16) tmem_st16(t_s + c, z);
          tmem_st_wait();
          tc_fence_before_sync();
          mbar_arrive(&sh.p_ready[h][0]);
        } else {
          // which of 32 tokens from t0 + 64 part + 32 c on the row sees
          auto seen_of = [&](int c) {
            const int tc = t0 + part * 64 + c * 32;
            const int lo = min(max(from - tc, 0), 32), hi = min(max(pos + 1 - tc, 0), 32);
            return sh.valid[0][par][part * 2 + c] & (uint32_t)((1ull << hi) - (1ull << min(lo, hi)));
          };
          const bool far = sh.s_exp[par] == FAR;  // (for all tokens of the group)
          const float factor = far ? 1.f : score_factor(scale2, sh.s_exp[par] + q_exp);
          auto factors = [&](int c, float* x) {  // scores of 32 tokens from sums that their scales are not in yet
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const uint32_t bytes = *reinterpret_cast<const uint32_t*>(&sh.k_byte[par][part * 64 + c * 32 + i]);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int n = max(min((int)(bytes >> 8 * y & 255) - 127 + q_exp, 120), -250);
                x[i + y] *= __uint_as_float((uint32_t)((n >> 1) + 127) << 23);
                x[i + y] *= scale2 * __uint_as_float((uint32_t)(n - (n >> 1) + 127) << 23);
              }
            }
          };
          const int E1 = sh.E[par];
          bool stays;
          // ---- the scores by the row's reference as it is: weights if it does ----
          float top[2] = {-INFINITY, -INFINITY};
          {
            auto scores = [&](int c, float (&x)[32]) {  // of 32 tokens, by the row's reference
              tmem_ld32(t_s + c * 32, x);
              tmem_ld_wait();
              float2 f2 = make_float2(factor, factor), ref = make_float2(-m, -m);
              if (!whole) {
                if (far) factors(c, x);
                const uint32_t seen = seen_of(c), bad = sh.nan[0][par][part * 2 + c] | sh.nan[1][par][part * 2 + c];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  x[i] = seen >> i & 1 ? fmaf(x[i], factor, -m) : -INFINITY;
                  if (seen & bad & 1u << i) x[i] = __uint_as_float(0x7fc00000u);
                }
                f2 = make_float2(1.f, 1.f), ref = make_float2(0.f, 0.f);
              }
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 d = fma2(make_float2(x[i], x[i + 1]), f2, ref);
                x[i] = d.x, x[i + 1] = d.y;
              }
            };
            if (whole) {  // (factors are not negative)
              float x[32], y[32];
              tmem_ld32(t_s, x);
              tmem_ld32(t_s + 32, y);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                top[0] = max3(top[0], x[i], x[i + 1]);
                top[1] = max3(top[1], y[i], y[i + 1]);
              }
              top[0] = fmaf(fmaxf(top[0], top[1]), factor, -m);
            } else {
#pragma unroll 1
              for (int c = 1; c >= 0; --c) {
                float x[32];
                scores(c, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  top[0] = max3(top[0], x[i], x[i + 1]);
                  top[1] = max3(top[1], x[i + 2], x[i + 3]);
                }
              }
              top[0] = fmaxf(top[0], top[1]);
            }
            const bool need = real && (fresh ? top[0] > -INFINITY : top[0] > SLACK);
            stays = all_of<64>(pair, !need && E1 == E);
            if (stays) {
              float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
              for (int c = 0; c < 2; ++c) {
                float x[32];
                scores(c, x);
#pragma unroll
                for (int y = 0; y < 32; y += 16) {
                  uint32_t big[8], small[8];
#pragma unroll
                  for (int i = 0; i < 16; i += 4) {
                    const float2 w0 = make_float2(ex2(x[y + i]), ex2(x[y + i + 1])), w1 = make_float2(ex2(x[y + i + 2]), ex2(x[y + i + 3]));
                    sum[0] = add2(sum[0], w0);
                    sum[1] = add2(sum[1], w1);
                    two_parts(w0, big[i / 2], small[i / 2]);
                    two_parts(w1, big[i / 2 + 1], small[i / 2 + 1]);
                  }
                  tmem_st8(t_s + c * 32 + y / 2, big);
                  tmem_st8(t_s + c * 32 + 16 + y / 2, small);
                }
                if (c == 0) {
                  tmem_st_wait();
                  tc_fence_before_sync();
                  mbar_arrive(&sh.p_ready[h][0]);
                }
              }
              const float2 both = add2(sum[0], sum[1]);
              l += both.x + both.y;
            }
          }
          if (!stays) {
            // ---- a reference moves: both threads of a row; the scores are still there ----
            sh.row[h][part][r] = top[0];
            pair_sync();
            const float mx = fmaxf(top[0], sh.row[h][part ^ 1][r]);
            const bool move = real && (fresh ? mx > -INFINITY : mx > SLACK);
            // rounded down, as far as a large score's steps are: its weight is not lost below the operands' bits
            const float dm = move ? fmaf(fabsf(mx), -0x1p-22f, mx) : 0.f, keep = move && !fresh ? ex2(-dm) : 1.f;
            m = __fadd_rd(m, dm);
            l *= keep;
            fresh = fresh && !move;
            if (j > 0) {
              const float f = keep * (E - E1 > -127 ? __uint_as_float((uint32_t)(127 + E - E1) << 23) : 0.f);
#pragma unroll 1
              for (int c = part * 16; c < D; c += 32) {
                uint32_t x[16];
                tmem_ld16(t_o + c, x);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                tmem_st16(t_o + c, x);
              }
            }
            E = E1;
            float more = 0.f;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              const uint32_t seen = seen_of(c), bad = sh.nan[0][par][part * 2 + c] | sh.nan[1][par][part * 2 + c];
              float x[32];
              uint32_t big[16], small[16];
              tmem_ld32(t_s + c * 32, x);
              tmem_ld_wait();
              if (far) factors(c, x);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                // (scores of 2^27 and more have steps beyond the slack: their references are not exact)
                x[i] = seen >> i & 1 ? ex2(fminf(fmaf(x[i], factor, -m), SLACK)) : 0.f;
                if (seen & bad & 1u << i) x[i] = __uint_as_float(0x7fc00000u);
                more += x[i];
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) two_parts(make_float2(x[2 * i], x[2 * i + 1]), big[i], small[i]);
              tmem_st16(t_s + c * 32, big);  // (over scores that have been read)
              tmem_st16(t_s + c * 32 + 16, small);
            }
            l += more;
            tmem_st_wait();
            tc_fence_before_sync();
            mbar_arrive(&sh.p_ready[h][0]);
          }
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&sh.p_ready[h][1]);
      }
      // ---- the piece's rows: sums in units of 2^m, o of 2^E times that ----
      if (n_groups > 0) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&sh.o_full[h], filled & 1));
        tc_fence_after_sync();
        ++filled;
      }
      sh.row[h][part][r] = l;
      pair_sync();
      l += sh.row[h][part ^ 1][r];
      const bool nothing = fresh && l == 0.f;
      const bool own = pc.c0 == pc.c1;
      const int64_t at = (int64_t)(cta == pc.c0 ? pc.slot0 : 2 * cta) * f.rows + h * half_rows + r;
      int hd = 0;
      T* out = real ? out_row<T>(a, pc.begin, pc.n, pc.g, pc.row0, h * half_rows + r, hd) : nullptr;
      RowScale rs{0.f, 1.f, 1.f};
      if (own) {
        if (!nothing && real) rs = row_scale(a, hd, Stats{m, (float)E, l, 0.f});
      } else if (part == 0 && r < half_rows) {
        __stcg(reinterpret_cast<float4*>(f.stats + at),
               nothing || !real ? make_float4(LOWEST, 0.f, 0.f, 0.f) : make_float4(m, (float)E, l, 0.f));
      }
#pragma unroll 1
      for (int c = part * 16; c < D; c += 32) {
        uint32_t x[16];
        if (n_groups > 0) {
          tmem_ld16(t_o + c, x);
          tmem_ld_wait();
        }
        if (own) {
          alignas(16) T y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = from_f32<T>(nothing ? 0.f : __uint_as_float(x[i]) * rs.inv * rs.p1 * rs.p2);
          if (out) {
            reinterpret_cast<uint4*>(out + c)[0] = reinterpret_cast<const uint4*>(y)[0];
            reinterpret_cast<uint4*>(out + c)[1] = reinterpret_cast<const uint4*>(y)[1];
          }
        } else if (real && !nothing) {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            __stcg(reinterpret_cast<float4*>(f.parts + at * D + c + i),
                   make_float4(__uint_as_float(x[i]), __uint_as_float(x[i + 1]), __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])));
        }
      }
      if (!own)
        join_stretch<T, KV8_MANY_CTAS>(a, f, SOFTMAX, pc.begin, pc.n, pc.row0, pc.g, pc.c0, pc.c1, pc.slot0, &sh.scratch.last,
                                       rows_sync);
      tc_fence_before_sync();  // (the next products over O are behind the next weights)
      mbar_arrive(&sh.piece_free[k & 1]);
    }
  } else if (warp < SOFTMAX / 32 + 8) {
    // ---- codes to operands: K's warps, which see to the scales as well, and V's --------------------------------
    fewer_registers<40>();
    const int which = warp >= SOFTMAX / 32 + 4, ct = tid & 127;
    const int nb = 1 << (a.page_log - a.block_log), page_mask = (1 << a.page_log) - 1;
    uint32_t group = 0;
    for (int k = 0;; ++k) {
      ok = all_of<128>(2 + which, ok && mbar_wait(&sh.piece_full[k & 1], k >> 1 & 1));
      if (!ok) break;
      const Piece& pc = sh.piece[k & 1];
      if (pc.groups == 0) break;
      const int32_t* table = a.pages + (int64_t)pc.b * a.max_pages;
      const uint8_t* scales = a.cache + a.scales_at + (2 * pc.g + which) * nb;
      const int from = pc.from, to = pc.to, g1 = pc.g1;
      auto page_of = [&](int grp) {  // of the thread's token
        const int t = grp * TOK + ct;
        int id = -1;
        if (t >= from && t < to) id = table[t >> a.page_log];
        return id < a.n_pages ? id : -1;
      };
      auto scale_of = [&](int page, int grp) {
        return page < 0 ? 0 : (int)scales[page * a.page_bytes + (((grp * TOK + ct) & page_mask) >> a.block_log)];
      };
      int top = 0;  // largest scale byte: of V, so far in the piece, of K in the group
      int page = page_of(pc.g0), page1 = page_of(pc.g0 + 1), byte = scale_of(page, pc.g0);
      for (int grp = pc.g0; grp < g1; ++grp, ++group) {
        const uint32_t unit = 2 * group + which, slot = unit % 3;
        const int par = group & 1;
        const int page2 = page_of(grp + 2), byte1 = scale_of(page1, grp + 1);
        if (unit >= 3) ok = ok && mbar_wait(&sh.op_free[slot], unit / 3 - 1 & 1);
        const uint32_t valid = __ballot_sync(0xffffffffu, page >= 0), nan = __ballot_sync(0xffffffffu, page >= 0 && byte == 255);
        const int most = __reduce_max_sync(0xffffffffu, page >= 0 && byte < 255 ? byte : 0);
        if (which == 0) {
          const int least = __reduce_min_sync(0xffffffffu, page >= 0 && byte < 255 ? byte : 255);
          if (lane == 0) sh.low[par][warp & 3] = least;
          sh.k_byte[par][ct] = (uint8_t)byte;
        }
        if (lane == 0) {
          sh.valid[which][par][warp & 3] = valid;
          sh.nan[which][par][warp & 3] = nan;
          sh.top[which][par][warp & 3] = most;
        }
        ok = ok && mbar_wait(&sh.raw_full[slot], unit / 3 & 1);
        ok = all_of<128>(2 + which, ok);
        if (!ok) break;
        if (which == 0) top = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = max(top, sh.top[which][par][w]);
        {
          const bool live = page >= 0 && byte < 255;
          const int unit = max(0, (top - HEAD + 15) & ~15);
          // K's codes as f16 have their bits down to 2^-24: scales that differ by more do not go into one operand
          bool far = false;
          if (!which) {
            int low = 255;
#pragma unroll
            for (int w = 0; w < 4; ++w) low = min(low, sh.low[par][w]);
            far = top - low > (CODE == MOE_I8 ? 29 : 20);
          }
          uint32_t scale;  // K: 2^(byte - top + 5); V: 2^(byte - unit)
          if (which) asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(scale) : "f"(power_of(byte - unit)));
          else asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(scale) : "f"(far ? 1.f : __uint_as_float((uint32_t)max(132 + byte - top, 1) << 23)));
          if (!which && a.scale < 0.f) scale ^= 0x80008000u;  // (so that the scores' factors are not negative)
          sh.scale[which][par][ct] = live ? scale : 0u;
          if (ct == 0) {
            if (which) sh.E[par] = unit - 127;
            else sh.s_exp[par] = far ? FAR : top - 127 - 5;
          }
        }
        all_of<128>(2 + which, true);  // the scales are there
        // 16 codes a turn; eight neighbouring lanes take four pieces of two tokens, which the swizzle (16-byte pieces
        // exchanged by the row's number) puts into different banks
        constexpr int C = DP / 16, TURN = 128 / C;
        const int c = DP == 128 ? (ct & 3) | (ct >> 3 & 1) << 2 : ct & 3, t1 = DP == 128 ? (ct >> 2 & 1) | ct >> 4 << 1 : ct >> 2;
        const uint8_t* src = sm + P::RAW + slot * P::RAW_SIZE + t1 * D + c * 16;
        uint8_t* dst = sm + P::OPS + slot * P::OPERAND + (c / 4) * HALF + t1 * 128;
        if (c * 16 < D) {
          const uint32_t* sc = sh.scale[which][par] + t1;
          auto convert = [&](auto bf16) {
#pragma unroll
            for (int i = 0; i < TOK / TURN; ++i) {
              const int t = t1 + i * TURN;
              const uint4 u = *reinterpret_cast<const uint4*>(src + i * TURN * D);
              const uint32_t f = sc[i * TURN];
              const uint32_t w[4] = {code_word<CODE>(u.x), code_word<CODE>(u.y), code_word<CODE>(u.z), code_word<CODE>(u.w)};
              uint32_t x[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) x[y] = scaled_pair<CODE, decltype(bf16)::value>(w[y / 2], y & 1, f);
              uint8_t* row = dst + i * TURN * 128;
              const int at = ((2 * c) & 7) ^ (t & 7);
              *reinterpret_cast<uint4*>(row + (at << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<uint4*>(row + ((at ^ 1) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
            }
          };
          if (which) convert(std::true_type{});
          else convert(std::false_type{});
          if (CODE == MOE_E4M3 && which) {  // what does not count may be no numbers, and would not go with weights of 0
            const uint4 v = *reinterpret_cast<const uint4*>(sh.valid[1][par]);
            if ((v.x & v.y & v.z & v.w) != ~0u)
#pragma unroll 1
              for (int t = t1; t < TOK; t += TURN)
                if (!(sh.valid[1][par][t >> 5] >> (t & 31) & 1)) {
                  uint8_t* row = dst + (t - t1) * 128;
                  const int at = ((2 * c) & 7) ^ (t & 7);
                  *reinterpret_cast<uint4*>(row + (at << 4)) = *reinterpret_cast<uint4*>(row + ((at ^ 1) << 4)) = make_uint4(0, 0, 0, 0);
                }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&sh.op_full[slot]);
        mbar_arrive(&sh.raw_free[slot]);
        page = page1;
        page1 = page2;
        byte = byte1;
      }
      mbar_arrive(&sh.piece_free[k & 1]);
    }
  } else {
    fewer_registers<40>();
    if (warp == 24) {
      // ---- pieces, q and codes on their way ---------------------------------------------------------------
      int b = b0;
      Seq s = seq_of<TOK>(a, b, f.rows);
      constexpr int PAD = pad_of<TOK>();
      const int start = (int)scaled(in_seq, 1, s.groups + PAD);
      int g = start % a.G, turn = start / a.G, j0 = (int)(in_seq - (long long)start * (s.groups + PAD));
      long long line = begin_line, left = begin_of(cta + 1, total, ctas) - begin_line;
      if (j0 >= s.groups) {  // (behind a stretch's groups: with the next one)
        const long long skip = min((long long)s.groups + PAD - j0, left);
        line += skip, left -= skip, j0 = 0;
        if (++g == a.G) g = 0, ++turn;
      }
      uint32_t unit = 0, filled = 0;
      const int part = min(1 << a.page_log, TOK), parts = TOK / part;  // tokens of a copy, copies of a group
      for (int k = 0; ok; ++k) {
        while (left > 0 && turn >= s.tiles) {  // the next sequence with rows
          s = seq_of<TOK>(a, ++b, f.rows);
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
          x.row0 = (turn & 1 ? s.tiles - 1 - turn / 2 : turn / 2) * f.rows;
          x.g = g;
          const int t = x.row0 / a.rep, first = s.past + t, final = s.past + min(t + 2 * half_tokens, s.n) - 1;
          x.from = max(max(first - s.window + 1, 0), s.base + j0 * TOK);
          x.to = min(min(final + 1, s.end), s.base + j1 * TOK);
          x.g0 = x.from / TOK;
          x.g1 = x.from < x.to ? (x.to + TOK - 1) / TOK : x.g0;
          const long long gone = min((long long)s.groups + PAD - j0, left);
          line += gone;
          left -= gone;
          j0 = 0;
          if (++g == a.G) g = 0, ++turn;
        }
        if (k > 1) ok = __all_sync(0xffffffffu, mbar_wait(&sh.piece_free[k & 1], (k >> 1) - 1 & 1));
        if (!ok) break;
        if (lane == 0) {
          sh.piece[k & 1] = x;
          mbar_arrive(&sh.piece_full[k & 1]);
        }
        if (x.groups == 0) break;
        if (x.g0 == x.g1) continue;
        if (filled > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sh.q_free, filled - 1 & 1));
        if (!ok) break;
        ++filled;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, 2 * (DP / 64) * half_rows * 128);
          for (int h = 0; h < 2; ++h)
            for (int y = 0; y < DP / 64; ++y)
              copy_q(sm + P::Q + h * P::OPERAND + y * HALF, &q_map, y * 64, x.g * a.rep, x.begin + x.row0 / a.rep + h * half_tokens,
                     &sh.q_full);
        }
        const int32_t* table = a.pages + (int64_t)x.b * a.max_pages;
        auto page_of = [&](int grp) {
          const int t = grp * TOK + lane * part;
          int id = -1;
          if (lane < parts && t < x.to && t + part > x.from) id = table[t >> a.page_log];
          return id < a.n_pages ? id : -1;
        };
        int page = page_of(x.g0), page1 = page_of(x.g0 + 1);
        for (int grp = x.g0; grp < x.g1 && ok; ++grp) {
          const int page2 = page_of(grp + 2);
          const uint32_t held = __ballot_sync(0xffffffffu, page >= 0);
          for (int which = 0; which < 2; ++which, ++unit) {
            const int slot = unit % 3;
            if (unit >= 3) ok = ok && __all_sync(0xffffffffu, mbar_wait(&sh.raw_free[slot], unit / 3 - 1 & 1));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[slot], __popc(held) * part * D);
            __syncwarp();
            if (page >= 0)
              copy_bytes(sm + P::RAW + slot * P::RAW_SIZE + lane * part * D,
                         a.cache + kv8_codes(a, page, x.g, which, (grp * TOK + lane * part) & ((1 << a.page_log) - 1)), part * D,
                         &sh.raw_full[slot]);
          }
          page = page1;
          page1 = page2;
        }
      }
      if (!ok) {  // a wait ran out: no copy may be in flight when the CTA ends
        for (int i = 0; i < 3; ++i) mbar_wait(&sh.raw_full[i], unit / 3 & 1);
        mbar_wait(&sh.q_full, filled + 1 & 1);
      }
    } else if (warp == 25) {
      // ---- products -----------------------------------------------------------------------------------------
      if (elect_one()) {
        const int steps = D / 16;
        const uint32_t s_desc = idesc(TOK, false, false), o_desc = idesc(D, true, true);
        uint32_t unit = 0, group = 0, filled = 0;
        auto op_ready = [&](uint32_t u) { ok = ok && mbar_wait(&sh.op_full[u % 3], u / 3 & 1); };
        const uint64_t q_desc = desc_sw128(sm + P::Q, 16), k_desc = desc_sw128(sm + P::OPS, 16), v_desc = desc_sw128(sm + P::OPS, HALF);
        const uint32_t hi = (uint32_t)(q_desc >> 32);  // (of all)
        auto scores = [&](int h, uint32_t u) {
          const uint32_t q = (uint32_t)q_desc + h * (P::OPERAND >> 4), kk = (uint32_t)k_desc + u % 3 * (P::OPERAND >> 4);
#pragma unroll 2
          for (int s = 0; s < steps; ++s)
              mma_ss(tm + T_S + h * 128, q + ((s / 4) * HALF + (s % 4) * 32 >> 4), kk + ((s / 4) * HALF + (s % 4) * 32 >> 4), hi, s_desc, s > 0);
          mma_commit(&sh.s_full[h]);
        };
        auto values = [&](int h, uint32_t u, bool first, int c) {  // tokens 32 c .. 32 c + 31 of both halves
          const uint32_t v = (uint32_t)v_desc + u % 3 * (P::OPERAND >> 4);
#pragma unroll 2
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int p = 1; p >= 0; --p)
              mma_ts(tm + T_O + h * 128, tm + T_S + h * 128 + s / 2 * 64 + c * 32 + p * 16 + s % 2 * 8,
                     v + ((s / 2 * 4 + c * 2 + s % 2) * 2048 >> 4), hi, o_desc, !first || c > 0 || s > 0 || p == 0);
        };
        for (int k = 0; ok; ++k) {
          ok = mbar_wait(&sh.piece_full[k & 1], k >> 1 & 1);
          if (!ok || sh.piece[k & 1].groups == 0) break;
          const int n = sh.piece[k & 1].g1 - sh.piece[k & 1].g0;
          mbar_arrive(&sh.piece_free[k & 1]);
          if (n == 0) continue;
          ok = mbar_wait(BF ? &sh.q_ready : &sh.q_full, filled++ & 1);
          op_ready(unit);
          if (!ok) break;
          tc_fence_after_sync();
          scores(0, unit);
          scores(1, unit);
          mma_commit(&sh.op_free[unit % 3]);
          if (n == 1) mma_commit(&sh.q_free);
          for (int j = 0; j < n; ++j, unit += 2, ++group) {
            const bool more = j + 1 < n;
            op_ready(unit + 1);
            ok = ok && mbar_wait(&sh.p_ready[0][0], group & 1);
            if (!ok) break;
            tc_fence_after_sync();
            values(0, unit + 1, j == 0, 0);
            ok = ok && mbar_wait(&sh.p_ready[0][1], group & 1);
            if (more) op_ready(unit + 2);
            if (!ok) break;
            tc_fence_after_sync();
            values(0, unit + 1, j == 0, 1);
            if (more) scores(0, unit + 2);
            else mma_commit(&sh.o_full[0]);
            ok = mbar_wait(&sh.p_ready[1][0], group & 1);
            if (!ok) break;
            tc_fence_after_sync();
            values(1, unit + 1, j == 0, 0);
            ok = mbar_wait(&sh.p_ready[1][1], group & 1);
            if (!ok) break;
            tc_fence_after_sync();
            values(1, unit + 1, j == 0, 1);
            mma_commit(&sh.op_free[(unit + 1) % 3]);
            if (more) {
              scores(1, unit + 2);
              mma_commit(&sh.op_free[(unit + 2) % 3]);
              if (j + 2 == n) mma_commit(&sh.q_free);
            } else {
              mma_commit(&sh.o_full[1]);
            }
          }
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before_sync();
  const bool failed = __syncthreads_or(!ok);
  tc_fence_after_sync();
  if (failed && tid == 0) atomicOr(f.ctrl + CTRL_STATUS, DEV_ERR_MBAR_TIMEOUT);
  if (warp == 25) tmem_dealloc(tm, 512);
  pdl_launch_dependents();
}

// q [tokens][heads][dim] in boxes of the tokens and heads of a tile's rows and 64 dimensions, swizzled.
cudaError_t query_map(CUtensorMap* m, const Kv8Args& a, int half_tokens) {
  const auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.H, (cuuint64_t)a.N};
  const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)a.qs * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.rep, (cuuint32_t)half_tokens}, es[3] = {1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, es,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
template <typename T, int CODE, int DP>
cudaError_t launch(const Kv8Args& a, const Kv8Parts& f, int half_tokens, bool pdl, cudaStream_t st) {
  CUtensorMap map;
  cudaError_t e = query_map(&map, a, half_tokens);
  if (e != cudaSuccess) return e;
  const auto kern = kv8_many<T, CODE, DP>;
  e = ensure_smem(reinterpret_cast<const void*>(kern), Plan<DP>::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(KV8_MANY_CTAS);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Plan<DP>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, f, half_tokens, map);
}
template <typename T>
cudaError_t by_code(const Kv8Args& a, const Kv8Parts& f, int half_tokens, bool pdl, cudaStream_t st) {
  if (a.code == MOE_I8)
    return a.D <= 64 ? launch<T, MOE_I8, 64>(a, f, half_tokens, pdl, st) : launch<T, MOE_I8, 128>(a, f, half_tokens, pdl, st);
  return a.D <= 64 ? launch<T, MOE_E4M3, 64>(a, f, half_tokens, pdl, st) : launch<T, MOE_E4M3, 128>(a, f, half_tokens, pdl, st);
}

}  // namespace

cudaError_t kv8_many_launch(const Kv8Args& a, Kv8Parts f, bool pdl, cudaStream_t st) {
  const int half_tokens = 128 / a.rep;
  f.rows = 2 * half_tokens * a.rep;
  return a.type == MOE_F16 ? by_code<__half>(a, f, half_tokens, pdl, st) : by_code<__nv_bfloat16>(a, f, half_tokens, pdl, st);
}

}  // namespace moe
