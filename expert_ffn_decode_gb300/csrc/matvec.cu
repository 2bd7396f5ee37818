// Matrix-vector products with 4-bit weights and group scales: y_t = W x_t (+ bias) (+ y_t).
//
// A row's block of 32 values with scale d and offset m contributes
//   d * sum_i q_i x_i + m * sum_i x_i
// (Q4_0 and planes without offsets: m = -8 d; Q4_K: d and m are the sub-block's d sc and
// -dmin mn), so a nibble is used as the integer it is and never rounded. The inner sum runs on
// the tensor cores by mma.m16n8k16, whose operands are registers: at one vector there is a
// matrix row of work for one accumulator column, far too little for a tcgen05 tile. Bytes are the
// floor: 128,000 x 2048 Q4_0 and one vector take 33.8 us (65% of HBM's rate; one warp a row
// with f32 products 888 us). Nothing is full: 2.9 instructions a weight issue in 62% of the slots,
// ALU 40%, DRAM 50%. What is left over the floor is the latency of each warp's chain from shared
// memory through nibbles, products and scales with 16 warps an SM (124 registers a thread). A pair of nibbles becomes an f16 operand by one AND (the
// bits of a nibble in the low bits of an f16 are the subnormal q 2^-24, or 16 q 2^-24 for the
// high one) and one multiplication by a power of two to q 2^-10. The multiplication is
// needed for the sums, not for the values: a subnormal operand counts in the accumulator's
// alignment with the exponent of the smallest normal number, and up to ten bits of every
// product are lost (1.2 times outside the rounding bound beside a value 10^6 times its
// neighbours).
//
// x is held as f16 pieces: within a block of 32 values it is scaled by a power of two that
// puts the largest magnitude at 2^13 .. 2^14, then split into two parts (22 bits of each value
// down to 2^-15 of the block's largest, fewer below; 16-bit types in calls of several vectors take
// one, which holds them). A block's sums of q x and of x and their products with d and m stay in that
// scale, in f32, and only then is the scale taken back: near f32's largest number a sum of x may
// lie outside f32 where y does not. (A 24-bit fixed point of the block was 1.3 times outside
// the bound in the same place.)
//
// Columns of one mma are (vector, part) pairs. A single vector has two of eight: the other six
// take three more blocks. Lane t of a quad of lanes then holds a whole block's nibbles of its
// row, and x is zero outside the columns of the lane's own block, so the accumulator's
// column pair t is block t's sum and each lane applies one block's scale. Rows of an even number
// of Q4_0 blocks (36 bytes a pair) need no shifts to bring the 18-byte blocks to whole words.
#include "common.cuh"
#include "ops_host.h"
#include "types.cuh"

namespace moe {
namespace {

constexpr int MV_PITCH = 176;    // bytes of a staged row: 256 values of the widest type and 16 of misalignment;
                                 // 48 mod 128 spreads four 20-byte blocks of 8 rows over all banks
constexpr int MV_SPITCH = 32;    // planes: staged bytes of a row's scales (and of its offsets)

// Types of weight rows, as template values (Q4_0_PAIRS: one vector, an even number of blocks a row).
enum { ROW_Q4_0, ROW_Q4_0_PAIRS, ROW_Q4_1, ROW_Q4_K, ROW_PLANES };
constexpr bool is_q4_0(int rt) { return rt == ROW_Q4_0 || rt == ROW_Q4_0_PAIRS; }

// How a call's vectors sit in the mma columns.
//   MULTI false: one vector, four blocks an mma.
//   MULTI true: NT tiles of 8 columns of PARTS parts, one block an mma.
template <bool MULTI_, int NT_, int PARTS_, int WARPS_>
struct Cols {
  static constexpr bool MULTI = MULTI_;
  static constexpr int NT = NT_, PARTS = PARTS_;
  static constexpr int VECS = MULTI ? 8 * NT / PARTS : 1;
  static constexpr int JOIN = MULTI ? VECS : 2;  // tiles of 16 sums a warp puts up at a time
  static constexpr int XBYTES = MULTI ? 16 * NT : 4;  // bytes of x pieces for each of a row's values
  // Warps of a CTA and stages of a warp's ring. Several vectors' x pieces
  // leave room for one CTA an SM, which then has sixteen warps to share them (8192 x 2560, eight
  // vectors: 10.8 us, 12.5 with eight), or eight where longer rows leave no more room.
  static constexpr int WARPS = WARPS_, DEPTH = MULTI ? 2 : 4;
};

struct MvArgs {
  MatvecArgs a;
  int64_t row_bytes, total;    // of the weights (planes: of the nibble plane)
  int64_t srow, stotal;        // planes: of the scales and of the offsets
  int nb;                      // blocks of a row
  int nu;                      // runs of 256 values, 8 blocks, of a row (the last may be partial)
  int ks;                      // warps that share a tile of 16 rows
  int tiles;
  int pdl;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The nibbles of word w (rows g) and u (rows g + 8) against x pieces: low nibbles are values
// 4 j .. 4 j + 3 of a half block in the order 0, 2 | 1, 3, high ones of the other half.
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t low_h2(uint32_t w) { return mul_h2(w & 0x000f000fu, 0x74007400u); }   // 2^14
__device__ __forceinline__ uint32_t high_h2(uint32_t w) { return mul_h2(w & 0x00f000f0u, 0x64006400u); }  // 2^10
template <bool first>
__device__ __forceinline__ void mma_low(float (&c)[4], uint32_t w, uint32_t u, uint32_t b0, uint32_t b1) {
  if (first) mma16816_zero(c, low_h2(w), low_h2(u), low_h2(w >> 8), low_h2(u >> 8), b0, b1);
  else mma16816(c, low_h2(w), low_h2(u), low_h2(w >> 8), low_h2(u >> 8), b0, b1);
}
template <bool first>
__device__ __forceinline__ void mma_high(float (&c)[4], uint32_t w, uint32_t u, uint32_t b0, uint32_t b1) {
  if (first) mma16816_zero(c, high_h2(w), high_h2(u), high_h2(w >> 8), high_h2(u >> 8), b0, b1);
  else mma16816(c, high_h2(w), high_h2(u), high_h2(w >> 8), high_h2(u >> 8), b0, b1);
}
// Single vector, where the integer pipe is what bounds: the odd bytes' high nibbles are the bytes
// less their low nibbles, an exact f16 sum instead of a mask. High nibbles come out as
// q 2^-6 and have an accumulator of their own, h.
struct Nibbles {
  uint32_t low[2], high[2];  // even, odd bytes
};
__device__ __forceinline__ Nibbles nibbles(uint32_t w) {
  Nibbles n;
  const uint32_t odd = __byte_perm(w, 0, 0x4341);
  n.low[0] = low_h2(w);
  n.low[1] = low_h2(odd);
  n.high[0] = mul_h2(w & 0x00f000f0u, 0x74007400u);
  asm("{ .reg .b32 m; neg.f16x2 m, %2; fma.rn.f16x2 %0, %1, %3, m; }"
      : "=r"(n.high[1]) : "r"(odd), "r"(n.low[1]), "r"(0x74007400u));
  return n;
}
template <bool first>
__device__ __forceinline__ void mma_word(float (&c)[4], float (&h)[4], uint32_t w, uint32_t u, uint32_t l0, uint32_t l1,
                                         uint32_t h0, uint32_t h1) {
  const Nibbles a = nibbles(w), b = nibbles(u);
  if (first) {
    mma16816_zero(c, a.low[0], b.low[0], a.low[1], b.low[1], l0, l1);
    mma16816_zero(h, a.high[0], b.high[0], a.high[1], b.high[1], h0, h1);
  } else {
    mma16816(c, a.low[0], b.low[0], a.low[1], b.low[1], l0, l1);
    mma16816(h, a.high[0], b.high[0], a.high[1], b.high[1], h0, h1);
  }
}
__device__ __forceinline__ float half_bits(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)u)); }
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The scale of a block of x, a power of two that brings its largest magnitude mx to 2^13 .. 2^14
// (the smallest normal number comes to 2, and 0 stays), and 2^10 / scale; both normal.
__device__ __forceinline__ float2 block_scale(float mx) {
  const uint32_t e = min(max(__float_as_uint(mx) >> 23, 13u), 254u);
  return make_float2(__uint_as_float((267 - e) << 23), __uint_as_float((e - 3) << 23));
}
// Scaled x in f16 pieces, and for each block and vector {2^10 / scale, 2^-10 sum of scaled x}. A thread
// takes four values of a vector; the eight threads of a block are neighbours. Values past the row's
// end are not written: they belong to blocks whose sums are dropped.
template <int RT, class C>
__device__ __forceinline__ void put_x(float4 v, float back, float sum, int vec, int at, uint8_t* xf, float2* info) {
  const int b = at / 32, r = at % 32;
  const float f[4] = {v.x, v.y, v.z, v.w};
  uint2 parts[2];
  parts[0] = make_uint2(pack_h2(f[0], f[2]), pack_h2(f[1], f[3]));
  if (C::PARTS == 2) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&parts[0].x));
    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&parts[0].y));
    parts[1] = make_uint2(pack_h2(f[0] - a.x, f[2] - a.y), pack_h2(f[1] - c.x, f[3] - c.y));
  }
  if constexpr (!C::MULTI) {
    int quad = b / 4, t = b & 3, nib = r / 16;
    if (RT == ROW_Q4_K) {  // lane t: 16 bytes, half t % 2 of a run of 64; nibble: which sub-block of it
      t = (b >> 1 & 1) * 2 + r / 16;
      nib = b & 1;
    } else if (is_q4_0(RT)) {  // every second block: 36 bytes apart, the quad's lanes meet four banks
      quad = b / 8 * 2 + b % 2;
      t = b / 2 & 3;
    }
    const int j = r % 16 / 4;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<uint2*>(xf + quad * 512 + (nib * 2 + j / 2) * 128 + (2 * t + q) * 16 + j % 2 * 8) = parts[q];
  } else {
#pragma unroll
    for (int q = 0; q < C::PARTS; ++q) {
      const int col = vec * C::PARTS + q, lane = col % 8 * 4 + r % 16 / 4;
      *reinterpret_cast<uint2*>(xf + ((b * C::NT + col / 8) * 32 + lane) * 16 + r / 16 * 8) = parts[q];
    }
  }
  if ((threadIdx.x & 7) == 0) info[b * C::VECS + vec] = make_float2(back, sum * 0.0009765625f);
}
template <int RT, class C, typename TX>
__device__ __forceinline__ void stage_x(const MvArgs& p, int t0, int nv, uint8_t* xf, float2* info) {
  const TX* x = static_cast<const TX*>(p.a.x) + t0 * p.a.xs;
  constexpr int AHEAD = 4, STEP = C::WARPS * 32 * 4;  // pieces of a turn; values between a thread's pieces
  const int cols = p.a.cols;
  // The thread's pieces run through the vectors end to end; the next turn's are loaded before
  // this one's are converted.
  int vec = 0, at = threadIdx.x * 4;
  while (at >= cols) at -= cols, ++vec;
  int lv[AHEAD], la[AHEAD];
  float4 ld[AHEAD];
  auto fetch = [&]() {
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      lv[n] = vec;
      la[n] = at;
      ld[n] = vec < nv ? load4(x + vec * p.a.xs + at) : make_float4(0.f, 0.f, 0.f, 0.f);
      at += STEP;
      while (at >= cols) at -= cols, ++vec;
    }
  };
  fetch();
  const int turns = (cols * nv + STEP * AHEAD - 1) / (STEP * AHEAD);
  for (int turn = 0; turn < turns; ++turn) {
    float4 v[AHEAD];
    int vv[AHEAD], va[AHEAD];
    float mx[AHEAD], sum[AHEAD], back[AHEAD];
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      v[n] = ld[n];
      vv[n] = lv[n];
      va[n] = la[n];
      mx[n] = fmaxf(fmaxf(fabsf(v[n].x), fabsf(v[n].y)), fmaxf(fabsf(v[n].z), fabsf(v[n].w)));
    }
    if (turn + 1 < turns) fetch();
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {  // over the 8 threads of a block
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xffffffffu, mx[n], o));
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      const float2 s = block_scale(mx[n]);
      v[n] = make_float4(v[n].x * s.x, v[n].y * s.x, v[n].z * s.x, v[n].w * s.x);
      sum[n] = (v[n].x + v[n].y) + (v[n].z + v[n].w);
      back[n] = s.y;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], o);
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (RT == ROW_Q4_0_PAIRS) {  // an even block's bytes are used from the third on, its first two last
        const int next = (threadIdx.x & 28) | ((threadIdx.x + 1) & 3);
        const float a = __shfl_sync(0xffffffffu, v[n].x, next), b = __shfl_sync(0xffffffffu, v[n].y, next);
        if (va[n] % 64 < 32) v[n] = make_float4(v[n].z, v[n].w, a, b);
      }
      if (vv[n] < nv) put_x<RT, C>(v[n], back[n], sum[n], vv[n], va[n], xf, info);
    }
  }
}

// The scale and offset of Q4_K sub-block j from its super-block's 16 header bytes.
__device__ __forceinline__ void q4k_scale(uint4 h, int j, float& d, float& m) {
  const uint32_t s = j & 3, sh = s * 8;
  uint32_t sc, mn;
  if (j < 4) {
    sc = h.y >> sh & 63;
    mn = h.z >> sh & 63;
  } else {
    const uint32_t b = h.w >> sh;
    sc = (b & 15) | (h.y >> sh >> 6 & 3) << 4;
    mn = (b >> 4 & 15) | (h.z >> sh >> 6 & 3) << 4;
  }
  d = half_bits(h.x & 0xffffu) * (float)sc;
  m = -half_bits(h.x >> 16) * (float)mn;
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// A warp's steps: the tiles of its group in turn, and in each its range of runs. Each step's rows are
// copied to the warp's own ring, so a warp never waits for another one but to join the partial sums
// of a tile. A step's products come before the copy into the stage that the step before it left: with
// DEPTH stages DEPTH - 2 copies are in flight beside the products, two for one vector and none for
// several, where the other warps' products are what hides them.
template <int RT, class C>
__global__ void __launch_bounds__(C::WARPS * 32, C::MULTI ? 1 : 2) matvec_kernel(const __grid_constant__ MvArgs p) {
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int WARPS = C::WARPS, DEPTH = C::DEPTH;
  constexpr int STAGE = 16 * (MV_PITCH + (RT == ROW_PLANES ? 2 * MV_SPITCH : 0));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  uint8_t* ring = sm + warp * DEPTH * STAGE;
  uint8_t* xf = sm + WARPS * DEPTH * STAGE;
  float2* info = reinterpret_cast<float2*>(xf + (size_t)(p.nu * 256) * C::XBYTES);
  float* red = reinterpret_cast<float*>(info + p.nu * 8 * C::VECS);  // [2][warps][16 * VECS]
  float4* zero = reinterpret_cast<float4*>(red + 2 * WARPS * 16 * C::JOIN);
  const int groups = WARPS / p.ks, group = warp / p.ks, part = warp % p.ks;
  const int stride = gridDim.x * groups, first = blockIdx.x * groups + group;
  const int ua = p.nu * part / p.ks, ub = p.nu * (part + 1) / p.ks, per_tile = ub - ua;
  const int my_tiles = first < p.tiles ? (p.tiles - first + stride - 1) / stride : 0;
  const int steps = my_tiles * per_tile;
  // bytes of a row's full run
  constexpr int RUN = is_q4_0(RT) ? 144 : RT == ROW_Q4_1 ? 160 : RT == ROW_Q4_K ? 144 : 128;
  constexpr int BLOCK = RUN / 8;

  if (p.pdl) pdl_launch_dependents();
  // ---- weights: the copies of one step -----------------------------------------------
  // The 16 rows' windows in 16-byte pieces, consecutive pieces on consecutive lanes: an
  // instruction then touches few lines (four lanes a row, eight rows at once, are fewer
  // instructions and slower: 33.6 -> 36.9 us for the 128,000 x 2048 head). Tiles and full runs
  // start at multiples of 16 bytes, so where a lane's pieces are within them never changes.
  constexpr int PIECES = RT == ROW_Q4_K || RT == ROW_PLANES ? RUN / 16 : RUN / 16 + 1;
  constexpr int TURNS = (16 * PIECES + 31) / 32;
  int from[TURNS], to[TURNS];  // a piece's place in the tile's bytes (run 0) and in the stage
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int at = i * 32 + lane, r = at / PIECES, c = at % PIECES * 16, b = r * (int)p.row_bytes;
    to[i] = r * MV_PITCH + c;
    from[i] = r < 16 && (b & ~15) + c < b + RUN ? (b & ~15) + c : -1;
  }
  int c_tile = first, c_u = ua, c_left = steps;  // the next step to copy
  uint32_t c_at = smem_addr(ring);               // its stage
  const uint8_t* c_src = p.a.w + (int64_t)first * 16 * p.row_bytes + ua * RUN;
  const int64_t next_tile = (int64_t)stride * 16 * p.row_bytes - (int64_t)(per_tile - 1) * RUN;
  const uint32_t ring_end = c_at + (DEPTH - 1) * STAGE;
  auto copy_step = [&]() {
    if (c_left > 0) {
      if (c_tile + 1 < p.tiles && c_u * 8 + 8 <= p.nb) {
#pragma unroll
        for (int i = 0; i < TURNS; ++i)
          if (from[i] >= 0) copy16(c_at + to[i], c_src + from[i]);
      } else {  // fewer rows, a partial run, and a last row that may end inside a piece
        const int rows = min(16, p.a.rows - c_tile * 16), bytes = min(8, p.nb - c_u * 8) * BLOCK;
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
          const int r = (i * 32 + lane) / PIECES;
          if (from[i] >= 0 && r < rows && from[i] < r * (int)p.row_bytes + bytes)
            copy16(c_at + to[i], c_src + from[i], (int)min((int64_t)16, p.a.w + p.total - (c_src + from[i])));
        }
      }
      if constexpr (RT == ROW_PLANES) {
        const int r = lane >> 1, at = (lane & 1) * 16;
        const int64_t sl = ((((int64_t)c_tile * 16 + r) * p.srow + c_u * 256 / p.a.group * 2) & ~(int64_t)15) + at;
        const int left = (int)min((int64_t)16, p.stotal - sl);
        if (c_tile * 16 + r < p.a.rows && left > 0) {
          copy16(c_at + 16 * MV_PITCH + r * MV_SPITCH + at, p.a.scales + sl, left);
          if (p.a.mins) copy16(c_at + 16 * (MV_PITCH + MV_SPITCH) + r * MV_SPITCH + at, p.a.mins + sl, left);
        }
      }
      --c_left;
      c_at = c_at == ring_end ? ring_end - (DEPTH - 1) * STAGE : c_at + STAGE;
      if (++c_u == ub) {
        c_u = ua;
        c_tile += stride;
        c_src += next_tile;
      } else {
        c_src += RUN;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) copy_step();

  // ---- x ------------------------------------------------------------------------------
  pdl_wait_prior_grids();
  const int t0 = blockIdx.y * C::VECS, nv = min(C::VECS, p.a.T - t0);
  if (p.a.x_type == MOE_F32) stage_x<RT, C, float>(p, t0, nv, xf, info);
  else if (p.a.x_type == MOE_F16) stage_x<RT, C, __half>(p, t0, nv, xf, info);
  else stage_x<RT, C, __nv_bfloat16>(p, t0, nv, xf, info);
  if (tid == 0) *zero = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();

  // single vector: where this lane's x pieces are, or a zero (column n = lane / 4 is part n & 1
  // of the block, or sub-block, n / 2 of the run)
  const uint8_t* xl[2];
  int xstep[2];
#pragma unroll
  for (int nib = 0; nib < 2; ++nib) {
    const int slot = RT == ROW_Q4_K ? (t & 2) + nib : t;
    const bool mine = g >> 1 == slot;
    xl[nib] = mine ? xf + nib * 256 + (2 * t + (g & 1)) * 16 : reinterpret_cast<const uint8_t*>(zero);
    xstep[nib] = mine;
  }

  constexpr int AV = C::MULTI ? 2 / C::PARTS : 1;  // vectors of a lane in a tile of columns
  float acc[C::NT][AV][2];                         // [column tile][vector][row g, g + 8]
#pragma unroll
  for (int n = 0; n < C::NT; ++n)
#pragma unroll
    for (int v = 0; v < AV; ++v) acc[n][v][0] = acc[n][v][1] = 0.f;

  // where the two rows' windows start in a stage, and their scales'
  int row_at[2];
#pragma unroll
  for (int r = 0; r < 2; ++r)
    row_at[r] = (g + 8 * r) * MV_PITCH + (((g + 8 * r) * (int)p.row_bytes) & 15);
  // Q4_0, single vector: a block starts on 2 bytes, so its words are funnelled from aligned ones;
  // where they are and by how much is the lane's own, whatever the tile
  int word_at[2][2];
  uint32_t word_shift[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = row_at[i / 2] + (2 * t + i % 2) * 18;
    word_at[i / 2][i % 2] = at & ~3;
    word_shift[i / 2][i % 2] = at & 2 ? 32 : 16;
  }
  uint4 x[2][4];  // single vector: the pieces of a run, kept from tile to tile if there is one run
  float2 xin[2];
  int stage = 0;
  const bool add = (p.a.flags & MOE_ACCUMULATE) != 0;
  auto get = [&](int64_t at) {
    return p.a.y_type == MOE_F32   ? static_cast<const float*>(p.a.y)[at]
           : p.a.y_type == MOE_F16 ? __half2float(static_cast<const __half*>(p.a.y)[at])
                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(p.a.y)[at]);
  };
  auto put = [&](int64_t at, float v) {
    if (p.a.y_type == MOE_F32) static_cast<float*>(p.a.y)[at] = v;
    else if (p.a.y_type == MOE_F16) static_cast<__half*>(p.a.y)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p.a.y)[at] = __float2bfloat16_rn(v);
  };
  float old = 0.f, first_sums[2] = {0.f, 0.f};
  for (int k = 0, tile = first; k < my_tiles; ++k, tile += stride) {
    // single vector: the pair's join is this warp's; what its sums will be added to is loaded while
    // they are made
    const bool join = !C::MULTI && (k >> 1 & (p.ks - 1)) == part;
    const int64_t my_row = ((int64_t)(k & 1 ? tile - stride : tile) + (lane >> 4) * stride) * 16 + (lane & 15);
    if (join && !(k & 1)) {
      old = 0.f;
      if (add && my_row < p.a.rows) old = get(t0 * p.a.ys + my_row);
      if (p.a.bias && my_row < p.a.rows) old += p.a.bias[my_row];
    }
    for (int u0 = ua; u0 < ub; ++u0) {
      if constexpr (!C::MULTI) {
        if (k == 0 || per_tile > 1) {
#pragma unroll
          for (int qq = 0; qq < 2; ++qq) {
            xin[qq] = info[u0 * 8 + (is_q4_0(RT) ? 2 * t + qq : qq * 4 + t)];
            if (is_q4_0(RT)) xin[qq].y *= -8.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i / 4][i % 4] = *reinterpret_cast<const uint4*>(
                xl[i / 2 % 2] + (xstep[i / 2 % 2] ? (u0 * 2 + i / 4) * 512 + (i & 1) * 128 : 0));
        }
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
      __syncwarp();
      const uint8_t* st = ring + stage;
      stage = stage == (DEPTH - 1) * STAGE ? 0 : stage + STAGE;
      const uint8_t* base[2];
      const uint8_t* sbase[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        base[r] = st + row_at[r];
        sbase[r] = st + 16 * MV_PITCH + (g + 8 * r) * MV_SPITCH;
        if (RT == ROW_PLANES)
          sbase[r] += ((g + 8 * r) * (int)p.srow + u0 * 256 / p.a.group * 2) & 15;
      }
      // word i of block b (of the step) of row r, and the block's scale and offset
      auto scale_of = [&](int r, int b, float& d, float& m) {
        if constexpr (RT == ROW_Q4_1) {
          const uint32_t h = *reinterpret_cast<const uint32_t*>(base[r] + b * 20);
          d = half_bits(h & 0xffffu);
          m = half_bits(h >> 16);
        } else if constexpr (is_q4_0(RT)) {
          d = half_bits(*reinterpret_cast<const uint16_t*>(base[r] + b * 18));
          m = -8.f * d;
        } else if constexpr (RT == ROW_Q4_K) {
          q4k_scale(*reinterpret_cast<const uint4*>(base[r]), b, d, m);
        } else {
          const int at = b * 32 / p.a.group * 2;
          d = half_bits(*reinterpret_cast<const uint16_t*>(sbase[r] + at));
          m = p.a.mins ? half_bits(*reinterpret_cast<const uint16_t*>(sbase[r] + 16 * MV_SPITCH + at)) : -8.f * d;
        }
      };
#pragma unroll
      for (int qq = 0; qq < 2; ++qq) {
        if constexpr (!C::MULTI) {
          const int b = is_q4_0(RT) ? 2 * t + qq : qq * 4 + t;  // this lane's block of the run
          float dd[2], mm[2];
          uint32_t w[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if constexpr (RT == ROW_Q4_0_PAIRS) {
              const uint32_t* u = reinterpret_cast<const uint32_t*>(base[r] + t * 36);
              if (qq == 0) {
#pragma unroll
                for (int i = 0; i < 3; ++i) w[r][i] = u[i + 1];
                w[r][3] = __byte_perm(u[4], u[0], 0x7610);
                dd[r] = half_bits(u[0] & 0xffffu);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[r][i] = u[i + 5];
                dd[r] = half_bits(u[4] >> 16);
              }
            } else if constexpr (RT == ROW_Q4_0) {
              const uint32_t* u = reinterpret_cast<const uint32_t*>(st + word_at[r][qq]);
              uint32_t v[5];
#pragma unroll
              for (int i = 0; i < 5; ++i) v[i] = u[i];
#pragma unroll
              for (int i = 0; i < 4; ++i) w[r][i] = __funnelshift_rc(v[i], v[i + 1], word_shift[r][qq]);
              dd[r] = half_bits((v[0] >> (word_shift[r][qq] & 16 ^ 16)) & 0xffffu);
            } else if constexpr (RT == ROW_Q4_1) {
              const uint32_t* u = reinterpret_cast<const uint32_t*>(base[r] + b * 20);
#pragma unroll
              for (int i = 0; i < 4; ++i) w[r][i] = u[i + 1];
              dd[r] = half_bits(u[0] & 0xffffu);
              mm[r] = half_bits(u[0] >> 16);
            } else {
              const uint4 u = *reinterpret_cast<const uint4*>(base[r] + (RT == ROW_Q4_K ? 16 : 0) + b * 16);
              w[r][0] = u.x;
              w[r][1] = u.y;
              w[r][2] = u.z;
              w[r][3] = u.w;
              scale_of(r, b, dd[r], mm[r]);
            }
          }
          float c[4], h[4];
          mma_word<true>(c, h, w[0][0], w[1][0], x[qq][0].x, x[qq][0].y, x[qq][2].x, x[qq][2].y);
          mma_word<false>(c, h, w[0][1], w[1][1], x[qq][0].z, x[qq][0].w, x[qq][2].z, x[qq][2].w);
          mma_word<false>(c, h, w[0][2], w[1][2], x[qq][1].x, x[qq][1].y, x[qq][3].x, x[qq][3].y);
          mma_word<false>(c, h, w[0][3], w[1][3], x[qq][1].z, x[qq][1].w, x[qq][3].z, x[qq][3].w);
          if (u0 * 8 + b < p.nb) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float s = fmaf(h[2 * r] + h[2 * r + 1], 0.0625f, c[2 * r] + c[2 * r + 1]);
              // (Q4_0: d (sum q x - 8 sum x))
              const float u = is_q4_0(RT) ? dd[r] * (s + xin[qq].y) : fmaf(dd[r], s, mm[r] * xin[qq].y);
              acc[0][0][r] = fmaf(xin[qq].x, u, acc[0][0][r]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int b = qq * 4 + i, blk = u0 * 8 + b;
            if (blk >= p.nb) break;
            uint32_t w0[2], w1[2];  // the words of the first and the second 16 values
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (RT == ROW_Q4_0) {
                const uint8_t* s = base[r] + b * 18 + 2 + t * 4;
                w0[r] = *reinterpret_cast<const uint16_t*>(s) | (uint32_t)*reinterpret_cast<const uint16_t*>(s + 2) << 16;
              } else if constexpr (RT == ROW_Q4_1) {
                w0[r] = *reinterpret_cast<const uint32_t*>(base[r] + b * 20 + 4 + t * 4);
              } else if constexpr (RT == ROW_PLANES) {
                w0[r] = *reinterpret_cast<const uint32_t*>(base[r] + b * 16 + t * 4);
              } else {  // sub-block b: a nibble of the run's 32 bytes
                w0[r] = *reinterpret_cast<const uint32_t*>(base[r] + 16 + b / 2 * 32 + t * 4);
                w1[r] = *reinterpret_cast<const uint32_t*>(base[r] + 16 + b / 2 * 32 + 16 + t * 4);
              }
            }
            float d[2], m[2];
            scale_of(0, b, d[0], m[0]);
            scale_of(1, b, d[1], m[1]);
#pragma unroll
            for (int n = 0; n < C::NT; ++n) {
              const uint4 x = *reinterpret_cast<const uint4*>(xf + ((blk * C::NT + n) * 32 + lane) * 16);
              float c[4];
              if constexpr (RT == ROW_Q4_K) {
                if (i & 1) {
                  mma_high<true>(c, w0[0], w0[1], x.x, x.y);
                  mma_high<false>(c, w1[0], w1[1], x.z, x.w);
                } else {
                  mma_low<true>(c, w0[0], w0[1], x.x, x.y);
                  mma_low<false>(c, w1[0], w1[1], x.z, x.w);
                }
              } else {
                mma_low<true>(c, w0[0], w0[1], x.x, x.y);
                mma_high<false>(c, w0[0], w0[1], x.z, x.w);
              }
#pragma unroll
              for (int v = 0; v < AV; ++v) {
                const float2 in = info[blk * C::VECS + (n * 4 + t) * AV + v];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const float s = C::PARTS == 2 ? c[2 * r] + c[2 * r + 1] : c[2 * r + v];
                  acc[n][v][r] = fmaf(in.x, fmaf(d[r], s, m[r] * in.y), acc[n][v][r]);
                }
              }
            }
          }
        }
      }
      __syncwarp();
      copy_step();
    }
    // ---- join the partial sums, in order --------------------------------------------------
    if constexpr (!C::MULTI) {  // of two tiles at once
      if (!(k & 1) && k + 1 < my_tiles) {
        first_sums[0] = acc[0][0][0];
        first_sums[1] = acc[0][0][1];
        acc[0][0][0] = acc[0][0][1] = 0.f;
        continue;
      }
      // four sums a lane, each over the quad's lanes: lane t keeps sum t (row g + 8 (t & 1) of tile t / 2)
      float v[4] = {k & 1 ? first_sums[0] : acc[0][0][0], k & 1 ? first_sums[1] : acc[0][0][1], acc[0][0][0], acc[0][0][1]};
      acc[0][0][0] = acc[0][0][1] = 0.f;
      const float a = (t & 2 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, t & 2 ? v[0] : v[2], 2);
      const float b = (t & 2 ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, t & 2 ? v[1] : v[3], 2);
      const float s = (t & 1 ? b : a) + __shfl_xor_sync(0xffffffffu, t & 1 ? a : b, 1);
      float* sums = red + ((k >> 1 & 1) * WARPS + group * p.ks) * 32;
      sums[part * 32 + (t >> 1) * 16 + (t & 1) * 8 + g] = s;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(p.ks * 32) : "memory");
      if (join && my_row < p.a.rows) {
        float sum = 0.f;
        for (int w = 0; w < p.ks; ++w) sum += sums[w * 32 + lane];
        put(t0 * p.a.ys + my_row, sum + old);
      }
    } else {
      float* mine = red + ((k & 1) * WARPS + warp) * 16 * C::VECS;
#pragma unroll
      for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int v = 0; v < AV; ++v)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            mine[((n * 4 + t) * AV + v) * 16 + g + 8 * r] = acc[n][v][r];
            acc[n][v][r] = 0.f;
          }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(p.ks * 32) : "memory");
      for (int i = part * 32 + lane; i < 16 * nv; i += p.ks * 32) {
        const int64_t row = (int64_t)tile * 16 + i % 16;
        if (row >= p.a.rows) continue;
        const float* from = red + ((k & 1) * WARPS + group * p.ks) * 16 * C::VECS + i;
        float s = 0.f;
        for (int w = 0; w < p.ks; ++w) s += from[w * 16 * C::VECS];
        if (p.a.bias) s += p.a.bias[row];
        const int64_t at = (t0 + i / 16) * p.a.ys + row;
        put(at, s + (add ? get(at) : 0.f));
      }
    }
  }
}

constexpr int MV_CTAS = 304;            // two on each of 152 SMs
constexpr int MV_SMEM = 227 * 1024;     // shared memory of a CTA at most

// Shared memory: the rings, the x pieces and block sums, two sets of partial sums, a zero.
template <int RT, class C>
int smem_bytes(const MvArgs& p) {
  const int stage = 16 * (MV_PITCH + (RT == ROW_PLANES ? 2 * MV_SPITCH : 0));
  return C::WARPS * C::DEPTH * stage + p.nu * 256 * C::XBYTES + p.nu * 8 * C::VECS * 8 +
         2 * C::WARPS * 16 * C::JOIN * 4 + 16;
}

template <int RT, class C>
cudaError_t launch(MvArgs& p, cudaStream_t st) {
  const int smem = smem_bytes<RT, C>(p);
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(matvec_kernel<RT, C>), smem);
  if (e != cudaSuccess) return e;
  const int ctas = !C::MULTI && smem <= 113 * 1024 ? MV_CTAS : MV_CTAS / 2;
  // Warps that share a tile: the count whose slowest warp has the fewest runs to walk, and the
  // larger one when two tie (fewer rows wait for a warp).
  int64_t best = -1;
  for (int ks = C::WARPS; ks >= C::WARPS / 8; ks /= 2) {  // (at most 8 groups have a barrier of their own)
    const int per = C::WARPS / ks;
    const int64_t rounds = (p.tiles + (int64_t)ctas * per - 1) / ((int64_t)ctas * per);
    const int64_t cost = rounds * ((p.nu + ks - 1) / ks * 8 + (ks > 1 ? 1 : 0));
    if (best < 0 || cost < best) {
      best = cost;
      p.ks = ks;
    }
  }
  const int per = C::WARPS / p.ks;
  const int want = (p.tiles + per - 1) / per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < ctas ? want : ctas), (unsigned)((p.a.T + C::VECS - 1) / C::VECS));
  cfg.blockDim = dim3(C::WARPS * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = p.pdl ? attr : nullptr;
  cfg.numAttrs = p.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, matvec_kernel<RT, C>, p);
}

// Launches the form if its shared memory fits.
template <int RT, class C>
bool try_launch(MvArgs& p, cudaStream_t st, cudaError_t* e) {
  if (smem_bytes<RT, C>(p) > MV_SMEM) return false;
  *e = launch<RT, C>(p, st);
  return true;
}
// The column form of a call. A pass of several vectors reads the weights once for all of
// them, up to sixteen, but keeps x pieces for each: 16 bytes a value for four f32 vectors or
// eight of 16 bits. Rows too long for that (about 2,000 values for sixteen f32 vectors, 5,000
// for eight, 10,000 for four; twice that in 16 bits) take fewer vectors a pass, in the end one.
// (8192 x 2048: sixteen f32 vectors 15.4 us in one pass of eight warps, 16.6 in two of sixteen;
// sixteen bf16 ones 11.3 and 14.9.) There is no form for more vectors than that: every further
// sixteen read and unpack the matrix again (8192 x 2560 Q4_1, bf16: 16 vectors 14.8 us, 64 56, 512 380).
template <int RT>
cudaError_t launch_cols(MvArgs& p, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.a.T > 8 && (p.a.x_type == MOE_F32 ? try_launch<RT, Cols<true, 4, 2, 8>>(p, st, &e)
                                          : try_launch<RT, Cols<true, 2, 1, 16>>(p, st, &e)))
    return e;
  if (p.a.T > 1 && p.a.x_type != MOE_F32) {
    if (try_launch<RT, Cols<true, 1, 1, 16>>(p, st, &e) || try_launch<RT, Cols<true, 1, 1, 8>>(p, st, &e)) return e;
  } else if (p.a.T > 1) {
    if (p.a.T > 4 &&
        (try_launch<RT, Cols<true, 2, 2, 16>>(p, st, &e) || try_launch<RT, Cols<true, 2, 2, 8>>(p, st, &e)))
      return e;
    if (try_launch<RT, Cols<true, 1, 2, 16>>(p, st, &e) || try_launch<RT, Cols<true, 1, 2, 8>>(p, st, &e)) return e;
  }
  if constexpr (RT == ROW_Q4_0)
    if (p.nb % 2 == 0) return launch<ROW_Q4_0_PAIRS, Cols<false, 1, 2, 8>>(p, st);
  return launch<RT, Cols<false, 1, 2, 8>>(p, st);
}

}  // namespace

cudaError_t matvec_launch(const MatvecArgs& a, cudaStream_t st) {
  MvArgs p{};
  p.a = a;
  p.nb = a.cols / 32;
  p.nu = (p.nb + 7) / 8;
  p.tiles = (int)(((int64_t)a.rows + 15) / 16);
  p.pdl = (a.flags & MOE_NO_PDL) == 0;
  p.row_bytes = a.qtype == MOE_Q4_0 ? p.nb * 18 : a.qtype == MOE_Q4_1 ? p.nb * 20 : a.qtype == MOE_Q4_K ? p.nb * 18 : p.nb * 16;
  p.total = p.row_bytes * a.rows;
  if (a.qtype == MOE_Q4_PLANES) {
    p.srow = a.cols / a.group * 2;
    p.stotal = p.srow * a.rows;
  }
  switch (a.qtype) {
    case MOE_Q4_0: return launch_cols<ROW_Q4_0>(p, st);
    case MOE_Q4_1: return launch_cols<ROW_Q4_1>(p, st);
    case MOE_Q4_K: return launch_cols<ROW_Q4_K>(p, st);
    default: return launch_cols<ROW_PLANES>(p, st);
  }
}

}  // namespace moe
