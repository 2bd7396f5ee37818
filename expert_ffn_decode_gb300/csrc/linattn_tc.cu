// Linear attention over prompts, 64 tokens at a time on the tensor cores.
//
// With G_t the sum of g from the chunk's start to token t and S the state before the chunk,
//   o_t = scale [ exp(G_t) S^T q_t + sum_{s <= t} exp(G_t - G_s) (q_t . k_s) v_s ]
//   S'  = exp(G_63) S + sum_s exp(G_63 - G_s) k_s v_s^T
// which is four products a chunk, with everything that depends on the decays applied to
// f32 accumulators or to operands that are split again afterwards:
//   P   [t][s]   = Q K^T                      scores, then masked and decayed
//   O2^T[dv][t]  = S^T Q^T                    what the state before the chunk gives
//   O1^T[dv][t]  = V^T P^T                    what the chunk's own tokens give
//   A^T [dv][dk] = V^T (exp(G_63 - G_s) K)    what the chunk adds to the state
// The outputs and the state are held transposed, dv on the tensor memory's lanes: then V^T
// is one operand for two products, S^T comes from tensor memory without a pass through
// shared memory, and a thread owns a piece of a row of S^T in f32 registers.
//
// Rounding: the tensor cores take 16-bit parts. A bf16 or f16 q, k, v is an operand as it is; f32
// ones, and their scores, decayed keys and states as operands, are three bf16 parts, which are the
// f32 value whatever its neighbours are. (Two f16 parts of the value times a power of two for the
// tile are half the products, 2 x 1024 tokens x 16 heads 64 us against 68, but values far below the
// tile's largest lose their bits: a document before a reset took those of the one behind it.) For 16-bit types
// scores and the state as an operand keep two parts (16 bits in bf16, 22 in f16). The decayed keys
// are summed into the f32 state, so they keep more bits for bf16 too: three bf16 parts or
// two f16 ones. f16 parts need their values in f16's range: scores and states are scaled by a
// power of two for each row, decayed keys for each chunk, and keep their 22 bits down to 2^-15 of the
// largest there, fewer below. Products of parts below the last kept
// bit are left out. Sums, statistics and the state are f32.
#include <cuda.h>

#include <type_traits>

#include "linattn.cuh"
#include "tc.cuh"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int CH = 64;                  // tokens of a chunk
constexpr int D = 128;                  // key and value width of the tiles (narrower ones are zero-filled)
constexpr uint32_t TILE = CH * D * 2;   // one part of a [64][128] operand
// One part of the scores, without what the mask leaves empty: the 16 columns s = 16 i .. of
// step i of the product over s are kept for the rows t >= 16 i.
constexpr uint32_t PTILE = 5120;
__host__ __device__ constexpr uint32_t p_base(int i) { return 32u * (64 * i - 8 * i * (i - 1)); }
__host__ __device__ constexpr uint32_t p_pitch(int i) { return 16u * (64 - 16 * i); }  // from 8 columns to the next 8

template <int NP>
struct Plan {
  static constexpr int NPP = NP == 1 ? 2 : 3;  // parts of scores and state operands
  static constexpr uint32_t Q = 0, K = NP * TILE, V = 2 * NP * TILE, KT = 3 * NP * TILE;
  static constexpr uint32_t P = KT + 3 * TILE;
  static constexpr uint32_t MISC = P + NPP * PTILE;
  // NP 1: 114,560 bytes and 1,024 of slack, two CTAs an SM
  static constexpr uint32_t BYTES = MISC + (NP == 1 ? 6016 : 7296);
  // Tensor memory columns: scores then O1, O2, and the state's parts, [warpgroup][part]; where there
  // are two of them A takes their place once O2 is done (a thread's columns of A are its columns of
  // the parts).
  static constexpr uint32_t T_O1 = 0, T_O2 = 64, T_S = 128, T_A = NP == 1 ? 128 : 320, T_COLS = NP == 1 ? 256 : 512;
};

struct Decays {
  float4 g[CH];      // G_t in powers of two: sum's high and low part, resets so far, exp(g_t)
  float w[CH];       // exp(G_63 - G_s)
  float eg[CH];      // scale * exp(G_t)
  float ieg[CH];     // exp(-G_t), where `mild`
  float lam;         // exp(G_63)
  float ghi, glo;    // sum over the chunk without resets
  int reset;         // whether the chunk forgets
  int mild;          // no resets, and every exp(G_t) within 2^-80 .. 2^20
  int pad[3];
};
template <int NWG>  // warpgroups
struct Misc {
  Decays d[2];       // of this chunk and the next
  uint64_t full_q, full_k, full_v;  // a tile has landed
  uint64_t qk, qs, end;             // products are done
  uint32_t tmem;
  int scratch[UNIT_SCRATCH];
  // f16: largest magnitudes on the way to the scales, and the scores' inverse scales
  alignas(16) float pinv[CH];
  float kmax[8], smax[NWG][128], pmax[NWG][64];
};

// bf16 (or f16) operands, K-major (0) or MN-major (1), f32 accumulator, shape M x N.
template <bool F16>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int ta, int tb) {
  return 1u << 4 | (F16 ? 0u : 1u << 7 | 1u << 10) | (uint32_t)ta << 15 | (uint32_t)tb << 16 | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(M >> 4) << 24;
}
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of a converged warp, the same one every time. Branching on it (and on a warp index
// the compiler knows to be uniform) keeps the operands of what follows in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Operand descriptors of a [64][128] tile, for step s of 16 along K. A tile of one part
// comes by TMA as two halves of 64 columns, rows of 128 bytes in the 128-byte swizzle; tiles of
// several parts and the decayed keys are written by threads as core matrices without one.
__device__ __forceinline__ uint64_t desc_sw128(const uint8_t* p, uint32_t lbo) {
  return (smem_desc(p, lbo, 1024) & ~((uint64_t)7 << 61)) | (uint64_t)2 << 61;
}
template <int NP>
__device__ __forceinline__ uint64_t desc_k(const uint8_t* tile, int s) {  // columns along K
  if constexpr (NP == 1) return desc_sw128(tile + (s / 4) * (TILE / 2) + (s % 4) * 32, 16);
  return smem_desc(tile + s * 2048, 1024, 128);
}
template <int NP>
__device__ __forceinline__ uint64_t desc_mn(const uint8_t* tile, int s) {  // rows along K
  if constexpr (NP == 1) return desc_sw128(tile + s * 2048, TILE / 2);
  return smem_desc(tile + s * 256, 128, 1024);
}
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// 64 tokens of one head (zeros past the tensor's end, and for columns past the head's width).
// Columns 64 .. 127 only for heads that have some.
__device__ __forceinline__ void tma_load_tile(uint8_t* dst, const CUtensorMap* map, int dim, int head, int t0,
                                              uint64_t* bar) {
  mbar_arrive_expect_tx(bar, dim > 64 ? TILE : TILE / 2);
  tma_load(dst, map, 0, head, t0, bar);
  if (dim > 64) tma_load(dst + TILE / 2, map, 64, head, t0, bar);
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
               "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A pair of 16-bit values (low half first) as f32.
template <bool F16>
__device__ __forceinline__ float2 unpack(uint32_t u) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two f32 values as n parts each, packed in pairs; the parts sum to the value to 8 n (f16: 11 n) bits. The
// first of three bf16 parts is cut off: they then are the value, and the largest numbers do not round
// to an infinity.
template <int n, bool F16 = false>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t* out) {
#pragma unroll
  for (int p = 0; p < n; ++p) {
    uint32_t h;
    if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    else if (n == 3 && p == 0) h = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    out[p] = h;
    if (p + 1 < n) {
      const float2 f = unpack<F16>(h);
      x0 -= f.x;
      x1 -= f.y;
    }
  }
}
// The power of two that brings a magnitude up to mx (0 and what is not finite included) to
// 2^14 .. 2^15, inside f16, and its inverse; both normal.
__device__ __forceinline__ float2 f16_scale(float mx) {
  const int e = min(max((int)(__float_as_uint(mx) >> 23), 16), 254);
  return make_float2(__uint_as_float((uint32_t)(268 - e) << 23), __uint_as_float((uint32_t)(e - 14) << 23));
}
// Tiles written by threads are kept as [column / 8][row][8 columns]: 8 rows x 16 bytes are one core matrix, so the
// same bytes serve as a K-major operand (columns along K: core matrices 1024 bytes apart
// along K, 128 along rows) and as an MN-major one (rows along K: 128 along K, 1024 along columns).
__device__ __forceinline__ uint32_t piece(int kc, int row) { return (uint32_t)(kc * CH + row) * 16u; }

// Tiles are shared out by turns of a warp: 8 rows x 32 columns, 8 columns a lane. A warp's turns
// are `pieces` neighbours in the rows of its number modulo 8 (two warps share them when
// there are sixteen).
__device__ __forceinline__ int piece_row() { return (threadIdx.x >> 5 & 7) * 8 + (threadIdx.x & 7); }
template <int pieces>
__device__ __forceinline__ int piece_col(int i) { return ((threadIdx.x >> 8) * pieces + i) * 4; }

// A thread's share of rows t0 .. t0 + n - 1 (zeros up to 64) of a [tokens][dim] f32 matrix:
// 8-column pieces of one row, fetched early and put into the tile as bf16 parts when that
// is free. A warp's 32 pieces of one i fill four whole 128-byte lines.
template <int NP, int PIECES>
struct Loader {
  float r[NP == 1 ? 1 : PIECES][8];
  __device__ __forceinline__ void fetch(const float* src, int64_t stride, int t0, int n, int dim) {
    const int lane = threadIdx.x & 31, row = piece_row(), kc0 = piece_col<PIECES>(0) + (lane >> 3);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int kc = kc0 + i * 4;
      const bool in = row < n && kc * 8 < dim;
      const float* p = in ? src + (t0 + row) * stride + kc * 8 : src;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 u = in ? reinterpret_cast<const float4*>(p)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
        r[i][4 * j] = u.x;
        r[i][4 * j + 1] = u.y;
        r[i][4 * j + 2] = u.z;
        r[i][4 * j + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void put(uint8_t* dst) const {
    const int lane = threadIdx.x & 31, row = piece_row(), kc0 = piece_col<PIECES>(0) + (lane >> 3);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      uint32_t u[4][NP];
#pragma unroll
      for (int j = 0; j < 4; ++j) split_pair<NP>(r[i][2 * j], r[i][2 * j + 1], u[j]);
      uint8_t* d = dst + piece(kc0 + i * 4, row);
#pragma unroll
      for (int q = 0; q < NP; ++q)
        *reinterpret_cast<uint4*>(d + q * TILE) = make_uint4(u[0][q], u[1][q], u[2][q], u[3][q]);
    }
  }
};
// Where piece kc (8 columns) of a row of a loaded tile is.
template <int NP>
__device__ __forceinline__ uint32_t tile_piece(int kc, int row) {
  if constexpr (NP == 1) return (uint32_t)((kc >> 3) * (TILE / 2) + row * 128 + (((kc & 7) ^ (row & 7)) << 4));
  return piece(kc, row);
}
// Eight values of a piece, the parts added up (exact: they do not overlap).
template <int NP, bool F16>
__device__ __forceinline__ void read_piece(const uint8_t* p, float (&x)[8]) {
#pragma unroll
  for (int q = NP - 1; q >= 0; --q) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + q * TILE);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack<F16>(w[j]);
      x[2 * j] = f.x + (q == NP - 1 ? 0.f : x[2 * j]);
      x[2 * j + 1] = f.y + (q == NP - 1 ? 0.f : x[2 * j + 1]);
    }
  }
}
// The products of parts i < NA of one operand and j < NB of the other with i + j <= LIM, each
// in the first `ks` of KS steps of 16 along K: the smallest first, because the tensor core's accumulator
// loses up to a last bit with every step, of what it holds by then.
template <int NA, int NB, int LIM, int KS, typename F>
__device__ __forceinline__ void each_product(int ks, F f) {
  bool first = true;
#pragma unroll
  for (int sum = LIM; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (i + j == sum)
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            if (s < ks) f(i, j, s, first);
            first = false;
          }
}

// The chunk's decays, by one warp (lane: tokens 2 lane, 2 lane + 1). Sums are carried as an
// f32 value and its rounding error, in powers of two, so that G_t - G_s keeps f32 accuracy
// however far down the chunk has decayed. A g below -104 (exp(g) < 2^-150, 0 in f32) is a
// reset: it is counted instead of added, and tokens on two sides of one do not meet.
__device__ __forceinline__ void chunk_decays(const LinattnArgs& a, int h, int t0, int n, Decays* m) {
  const int lane = threadIdx.x & 31;
  float raw[2], hi[2], lo[2];
  int r[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = 2 * lane + j;
    float g = t < n ? a.g[a.token_decay ? (int64_t)(t0 + t) * a.H + h : h] : 0.f;
    raw[j] = g;
    r[j] = g < -104.f;
    if (r[j]) g = 0.f;
    hi[j] = g * 1.44269504f;
    lo[j] = fmaf(g, 1.44269504f, -hi[j]) + g * 1.92596299e-8f;
  }
  auto add = [](float& h0, float& l0, float h1, float l1) {  // (h0, l0) + (h1, l1)
    const float s = h0 + h1, bb = s - h0;
    l0 = (h0 - (s - bb)) + (h1 - bb) + l0 + l1;
    h0 = s;
  };
  float ch = hi[0], cl = lo[0];
  add(ch, cl, hi[1], lo[1]);
  int cr = r[0] + r[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float xh = __shfl_up_sync(0xffffffffu, ch, o), xl = __shfl_up_sync(0xffffffffu, cl, o);
    const int xr = __shfl_up_sync(0xffffffffu, cr, o);
    if (lane >= o) {
      float sh = xh, sl = xl;
      add(sh, sl, ch, cl);
      ch = sh;
      cl = sl;
      cr += xr;
    }
  }
  const float eh = __shfl_sync(0xffffffffu, ch, 31), el = __shfl_sync(0xffffffffu, cl, 31);
  const int er = __shfl_sync(0xffffffffu, cr, 31);
  // sum up to the first of the lane's two tokens: the sum before the lane, plus it
  float ph = __shfl_up_sync(0xffffffffu, ch, 1), pl = __shfl_up_sync(0xffffffffu, cl, 1);
  int pr = __shfl_up_sync(0xffffffffu, cr, 1);
  if (lane == 0) ph = 0.f, pl = 0.f, pr = 0;
  add(ph, pl, hi[0], lo[0]);
  pr += r[0];
  const bool ok = fminf(ph, ch) > -80.f && fmaxf(ph, ch) < 20.f && ph == ph && ch == ch;
  const bool mild = __all_sync(0xffffffffu, ok) && er == 0;
  const float gh[2] = {ph, ch}, gl[2] = {pl, cl};
  const int gr[2] = {pr, cr};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = 2 * lane + j;
    m->g[t] = make_float4(gh[j], gl[j], (float)gr[j], expf(raw[j]));
    m->w[t] = gr[j] == er ? ex2((eh - gh[j]) + (el - gl[j])) : 0.f;
    m->eg[t] = gr[j] == 0 ? ex2(gh[j] + gl[j]) * a.scale : 0.f;
    m->ieg[t] = ex2(-(gh[j] + gl[j]));
  }
  if (lane == 0) {
    m->lam = er == 0 ? ex2(eh + el) : 0.f;
    m->ghi = eh;
    m->glo = el;
    m->reset = er != 0;
    m->mild = mild;
  }
}

// f32 takes one CTA an SM, of sixteen warps.
constexpr int chunk_threads(int np) { return np == 1 ? 256 : 512; }
struct Maps {
  CUtensorMap q, k, v, o;  // 16-bit types only
};

// MODE 0: the state that a unit's tokens alone leave, and its decay, into the workspace.
// MODE 1: the outputs, from the state before the unit; the sequence's last unit stores it.
// `wd`: decays [states][H], `wst`: states [states][H][dk][dv]. WIDE: keys
// of more than 112 values, whose eight steps along K are then fixed (237 against 259 us for
// 16,384 tokens x 32 heads of 128).
//
// Eight warps; one lane of warp 3, which has no scores to mask, also issues the products and
// the TMA copies, each as soon as its inputs are ready and its target is free:
//   QS, KV while the scores are masked | PV | the next chunk's QK while the state is updated;
//   the next k after QK, q after QS, v after the outputs, which are turned in v's place, have
//   left it.
// Two CTAs share an SM for 16-bit types, so one's products run beside the other's arithmetic;
// f32 has one of sixteen warps, and its products of a chunk start when its tiles are written.
template <typename T, int NP, int MODE, bool WIDE>
__global__ void __launch_bounds__(chunk_threads(NP), NP == 1 ? 2 : 1)
lin_chunk(LinattnArgs a, const __grid_constant__ Maps maps, LinattnCut cut, int n_ws, int behind_join, float* wd, float* wst,
          uint32_t* ctrl) {
  using L = Plan<NP>;
  static_assert(sizeof(Misc<chunk_threads(NP) / 128>) <= L::BYTES - L::MISC, "misc");
  constexpr bool F16 = std::is_same<T, __half>::value;  // the type of the parts
  constexpr bool F32 = std::is_same<T, float>::value;
  constexpr int NPP = L::NPP, LIM = NPP - 1;  // products of parts i, j with i + j <= LIM
  constexpr int KP = F16 ? 2 : 3;       // parts of the decayed keys
  constexpr int NT = chunk_threads(NP), NWG = NT / 128;  // threads; warpgroups, which share rows
  constexpr int CPT = D / NWG, TPT = CH / NWG, SPT = 4 / NWG;  // a thread's columns of S, tokens, mask steps
  constexpr int PIECES = 8 / NWG;                              // a warp's turns through a tile
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = sm_raw + ((1024u - (smem_addr(sm_raw) & 1023u)) & 1023u);
  auto* m = reinterpret_cast<Misc<NWG>*>(sm + L::MISC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2, quarter = warp & 3;
  const bool iwarp = __shfl_sync(0xffffffffu, warp, 0) == 3;  // whose elected lane issues
  // The heads of a unit are neighbours. Whole units come first and the sequences' last ones,
  // of any length, fill what is left (143 -> 120 us for a ragged batch of 9 f16 prompts); the state
  // pass has no last units.
  const int h = blockIdx.x % a.H, row = quarter * 32 + lane;  // row: this thread's lane of tensor memory
  const int at = blockIdx.x / a.H, u = MODE == 0 || at < cut.rest ? a.B + at : at - cut.rest;
  // Behind the join everything but the states is older than the state pass, which has ended: this
  // grid then sets up and loads its first chunk beside the join and waits for the states alone.
  if (!behind_join) pdl_wait_prior_grids();
  const Unit un = find_unit(a, cut, n_ws, u, m->scratch);
  if (!un.found) {
    if (behind_join) pdl_wait_prior_grids();  // no grid ends before the one it stands behind
    if (MODE == 1 && u < a.B && h == 0 && tid == 0) atomicOr(ctrl + CTRL_STATUS, DEV_ERR_OFFSETS);
    return;
  }
  int begin, end;
  seq_range(a, un.b, begin, end);
  const int last = end;
  begin += un.i * un.seg;
  end = min(begin + un.seg, end);
  const int slot = seq_slot(a, un.b);
  T* o = static_cast<T*>(a.o) + (int64_t)h * a.dv;
  if (slot < 0) {
    if (behind_join) pdl_wait_prior_grids();
    if (MODE == 1)
      for (int i = tid; i < (end - begin) * a.dv; i += NT)
        o[(begin + i / a.dv) * a.os + i % a.dv] = from_f32<T>(0.f);
    return;
  }
  if (warp == 0) tmem_alloc(&m->tmem, L::T_COLS);
  if (tid == 0) {
    mbar_init(&m->full_q, 1);
    mbar_init(&m->full_k, 1);
    mbar_init(&m->full_v, 1);
    mbar_init(&m->qk, 1);
    mbar_init(&m->qs, 1);
    mbar_init(&m->end, 1);
    fence_mbar_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = __shfl_sync(0xffffffffu, m->tmem, 0), tlane = tm + ((uint32_t)quarter * 32u << 16);
  const int hq = h / a.rep, ks = WIDE ? D / 16 : (a.dk + 15) / 16;  // steps of 16 along the keys' width
  const bool cols = WIDE || wg * CPT < a.dk;                // whether this thread's part of S^T has columns
  const T* q = static_cast<const T*>(a.q) + (int64_t)hq * a.dk;
  const T* k = static_cast<const T*>(a.k) + (int64_t)hq * a.dk;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv;
  const int64_t sz = (int64_t)a.dk * a.dv;
  float* pool = a.state + ((int64_t)slot * a.H + h) * sz;
  float* mine = wst + ((int64_t)(un.slot0 + un.i) * a.H + h) * sz;  // sequences of several units

  if (NP == 1 && begin < end && iwarp && elect_one()) {
    tma_load_tile(sm + L::K, &maps.k, a.dk, hq, begin, &m->full_k);
    if (MODE == 1) tma_load_tile(sm + L::Q, &maps.q, a.dk, hq, begin, &m->full_q);
    tma_load_tile(sm + L::V, &maps.v, a.dv, h, begin, &m->full_v);
  }
  // f32: a chunk's q, k and v on their way
  Loader<NP, PIECES> lq, lk, lv;
  auto fetch = [&](int t0) {
    if constexpr (F32) {
      const int n = min(CH, end - t0);
      if (MODE == 1) lq.fetch(q, a.qs, t0, n, a.dk);
      lk.fetch(k, a.ks, t0, n, a.dk);
      lv.fetch(v, a.vs, t0, n, a.dv);
    }
  };
  auto put_qk = [&]() {
    if constexpr (F32) {
      if (MODE == 1) lq.put(sm + L::Q);
      lk.put(sm + L::K);
    }
  };
  if (F32 && begin < end) {
    fetch(begin);
    put_qk();
  }
  if (warp == 7) chunk_decays(a, h, begin, min(CH, end - begin), &m->d[0]);

  if (behind_join) pdl_wait_prior_grids();
  // S^T: this thread's row, CPT key columns from CPT wg on
  float S[CPT];
  {
    const float* from = un.n > 1 ? mine : pool;
    const bool zero = MODE == 0 || (un.n == 1 && a.fresh);
#pragma unroll
    for (int j = 0; j < CPT; ++j)
      S[j] = !zero && row < a.dv && wg * CPT + j < a.dk ? from[(wg * CPT + j) * a.dv + row] : 0.f;
  }
  float sinv = 1.f;  // f16: inverse scale of this row of the operand
  auto put_state = [&]() {  // the state's parts as an operand in tensor memory
    float sc = 1.f;
    if constexpr (F16) {
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < CPT; ++j) mx = fmaxf(mx, fabsf(S[j]));
      m->smax[wg][row] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 1; i < NWG; ++i) mx = fmaxf(mx, m->smax[(wg + i) % NWG][row]);
      const float2 f = f16_scale(mx);
      sc = f.x;
      sinv = f.y;
    }
    if (cols) {
#pragma unroll
      for (int c = 0; c < CPT / 32; ++c) {
        uint32_t u[NPP][16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          uint32_t s[NPP];
          split_pair<NPP, F16>(S[c * 32 + 2 * j] * sc, S[c * 32 + 2 * j + 1] * sc, s);
#pragma unroll
          for (int p = 0; p < NPP; ++p) u[p][j] = s[p];
        }
#pragma unroll
        for (int p = 0; p < NPP; ++p) tmem_st16(tlane + L::T_S + (wg * NPP + p) * (CPT / 2) + c * 16, u[p]);
      }
      tmem_st_wait();
    }
  };
  auto add_state = [&](float lam, float ainv) {  // S = lam S + A
    if (cols) {
#pragma unroll
      for (int c = 0; c < CPT / 16; ++c) {
        if (wg * (CPT / 16) + c >= ks) break;  // columns that A does not have
        uint32_t r[16];
        tmem_ld16(tlane + L::T_A + wg * CPT + c * 16, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = __uint_as_float(r[j]);
          S[c * 16 + j] = fmaf(lam, S[c * 16 + j], F16 ? x * ainv : x);
        }
      }
    }
  };
  // A masked product with an infinity or a NaN is a NaN, which would reach the chunk's earlier
  // tokens: a chunk with such an output goes token by token, from global memory and the state
  // before it.
  auto token_by_token = [&](int t0, int n, const Decays* d) {
    float* part = reinterpret_cast<float*>(sm + L::V);
    for (int t = 0; t < n; ++t) {
      const float vv = row < a.dv ? to_f32(v[(t0 + t) * a.vs + row]) : 0.f;
      const float lam = d->g[t].w;
      float acc = 0.f;
#pragma unroll
      for (int c = 0; c < CPT / 4; ++c) {
        const int at = wg * CPT + c * 4;
        if (at < a.dk) {
          const float4 kk = load4(k + (t0 + t) * a.ks + at), qq = load4(q + (t0 + t) * a.qs + at);
          const float k4[4] = {kk.x, kk.y, kk.z, kk.w}, q4[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            S[c * 4 + j] = fmaf(lam, S[c * 4 + j], k4[j] * vv);
            acc = fmaf(q4[j], S[c * 4 + j], acc);
          }
        }
      }
      if (wg > 0) part[wg * 128 + row] = acc;
      __syncthreads();
      if (wg == 0 && row < a.dv) {
#pragma unroll
        for (int i = 1; i < NWG; ++i) acc += part[i * 128 + row];
        o[(t0 + t) * a.os + row] = from_f32<T>(acc * a.scale);
      }
      __syncthreads();
    }
    fence_proxy_async_smem();
    __syncthreads();
  };
  if (MODE == 1) put_state();

  uint32_t ph = 0;  // parity of this chunk's phases
  bool ok = true;
  auto issue_scores = [&](uint32_t p) {
    if (MODE == 1 && iwarp && elect_one()) {
      if (NP == 1) ok = mbar_wait(&m->full_q, p) && mbar_wait(&m->full_k, p) && ok;
      tc_fence_after_sync();
      each_product<NP, NP, LIM, D / 16>(ks, [&](int i, int j, int s, bool first) {
        mma_f16(tm + L::T_O1, desc_k<NP>(sm + L::Q + i * TILE, s), desc_k<NP>(sm + L::K + j * TILE, s),
                idesc<F16>(128, CH, 0, 0), !first);
      });
      mma_commit(&m->qk);
    }
    __syncwarp();
  };
  float sum_hi = 0.f, sum_lo = 0.f;
  int resets = 0;
  for (int t0 = begin; t0 < end; t0 += CH, ph ^= 1) {
    const int n = min(CH, end - t0);
    const Decays* d = &m->d[ph];
    const bool more = t0 + CH < end;
    // the state pass has no q: v alternates between the two places
    uint8_t* tv = sm + (NP == 1 && MODE == 0 && ph ? L::Q : L::V);
    if constexpr (F32) {
      fence_proxy_async_smem();
      __syncthreads();  // q and k are there; the last chunk's outputs have left v's place
      lv.put(tv);
    }
    if (F32 || t0 == begin) issue_scores(ph);
    // ---- the decayed keys ---------------------------------------------------------------
    if (NP == 1) ok = mbar_wait(&m->full_k, ph) && ok;
    if (NP == 1 && t0 == begin) __syncthreads();  // the first decays (f32: above)
    float2 kscale = make_float2(1.f, 1.f);
    if constexpr (F16) {
      // The largest finite magnitude of what a token's key is after its decay: of the lane's row of k, as
      // packed f16 bits, of which the unsigned order is that of magnitudes, times the row's own decay
      // (a key that a reset or a strong decay leaves nothing of must not take the others' bits).
      const int r = piece_row();
      auto largest = [&](auto keep) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const int kc = piece_col<PIECES>(i) + (lane >> 3);
          if (r < n && kc < 2 * ks) {
            const uint4 u = *reinterpret_cast<const uint4*>(sm + L::K + tile_piece<NP>(kc, r));
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(keep(u.x & 0x7fff7fffu), keep(u.y & 0x7fff7fffu)),
                                       __vmaxu2(keep(u.z & 0x7fff7fffu), keep(u.w & 0x7fff7fffu))));
          }
        }
        return max(mx & 0xffffu, mx >> 16);
      };
      uint32_t mx = largest([](uint32_t u) { return u; });
      if (__any_sync(0xffffffffu, mx >= 0x7c00u)) mx = largest([](uint32_t u) { return u & __vcmpltu2(u, 0x7c007c00u); });
      const float decayed = __half2float(__ushort_as_half((unsigned short)mx)) * d->w[r];
      const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(decayed));  // of non-negative numbers
      if (lane == 0) m->kmax[warp] = __uint_as_float(most);
      __syncthreads();
      float km = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) km = fmaxf(km, m->kmax[i]);
      kscale = f16_scale(km);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int r = piece_row(), kc = piece_col<PIECES>(i) + (lane >> 3);
      if (piece_col<PIECES>(i) >= 2 * ks) break;
      const float w = d->w[r] * kscale.x;
      float x[8];
      read_piece<NP, F16>(sm + L::K + tile_piece<NP>(kc, r), x);
      if (n < CH && r >= n) {  // rows past the chunk's tokens are other sequences' or none
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
      }
      uint32_t u[4][KP];
#pragma unroll
      for (int j = 0; j < 4; ++j) split_pair<KP, F16>(x[2 * j] * w, x[2 * j + 1] * w, u[j]);
#pragma unroll
      for (int p = 0; p < KP; ++p)
        *reinterpret_cast<uint4*>(sm + L::KT + p * TILE + piece(kc, r)) = make_uint4(u[0][p], u[1][p], u[2][p], u[3][p]);
    }
    if (NP == 1 && n < CH) {
      ok = mbar_wait(&m->full_v, ph) && ok;
      for (int i = n * 16 + tid; i < CH * 16; i += NT)
        *reinterpret_cast<uint4*>(tv + tile_piece<1>(i & 15, i >> 4)) = make_uint4(0, 0, 0, 0);
    }
    sum_lo += d->glo;
    {
      const float s = sum_hi + d->ghi, bb = s - sum_hi;
      sum_lo += (sum_hi - (s - bb)) + (d->ghi - bb);
      sum_hi = s;
    }
    resets |= d->reset;
    fence_proxy_async_smem();
    tc_fence_before_sync();
    if (__syncthreads_or(!ok)) {  // k has been read, the state's parts and the decayed keys are there
      ok = false;
      break;
    }
    tc_fence_after_sync();
    if (more) fetch(t0 + CH);
    if (warp == 7 && more) chunk_decays(a, h, t0 + CH, min(CH, end - t0 - CH), &m->d[ph ^ 1]);
    // ---- the state's share, and what the chunk adds to the state -------------------------
    if (iwarp && elect_one()) {
      if (MODE == 1) {
        each_product<NPP, NP, LIM, D / 16>(ks, [&](int i, int j, int s, bool first) {
          mma_ts(tm + L::T_O2, tm + L::T_S + (s * 16 / CPT * NPP + i) * (CPT / 2) + s * 16 % CPT / 2,
                 desc_k<NP>(sm + L::Q + j * TILE, s), idesc<F16>(128, CH, 0, 0), !first);
        });
        mma_commit(&m->qs);
        ok = mbar_wait(&m->qk, ph) && ok;
      }
      if (NP == 1 && more) tma_load_tile(sm + L::K, &maps.k, a.dk, hq, t0 + CH, &m->full_k);
      if (MODE == 1) ok = mbar_wait(&m->qs, ph) && ok;
      if (NP == 1 && MODE == 1 && more) tma_load_tile(sm + L::Q, &maps.q, a.dk, hq, t0 + CH, &m->full_q);
      if (NP == 1) ok = mbar_wait(&m->full_v, ph) && ok;
      // (this chunk's v has landed, so its barrier is free for the next one's)
      if (NP == 1 && MODE == 0 && more) tma_load_tile(sm + (ph ? L::V : L::Q), &maps.v, a.dv, h, t0 + CH, &m->full_v);
      tc_fence_after_sync();
      each_product<NP, KP, KP - 1, CH / 16>(CH / 16, [&](int i, int j, int s, bool first) {
        mma_f16(tm + L::T_A, desc_mn<NP>(tv + i * TILE, s), smem_desc(sm + L::KT + j * TILE + s * 256, 128, 1024),
                idesc<F16>(128, 16 * ks, 1, 1), !first);
      });
      if (MODE == 0) mma_commit(&m->end);
    }
    __syncwarp();
    // ---- masked scores and the chunk's own share -----------------------------------------
    if (MODE == 1 && quarter < 2 && wg * SPT < 2 * (quarter + 1)) {
      // Lanes 0 .. 63 hold the tokens' rows of scores; a thread takes SPT steps of 16 columns. The
      // mask leaves rows below 32 none of the last two steps.
      ok = mbar_wait(&m->qk, ph) && ok;
      tc_fence_after_sync();
      const float4 gt = d->g[row];
      const float et = d->eg[row];
      uint32_t sc[SPT][16];
      float mx = 0.f;
#pragma unroll
      for (int c = 0; c < SPT; ++c) {
        const int step = wg * SPT + c;  // of the product over s
        uint32_t (&s)[16] = sc[c];
        tmem_ld16(tlane + L::T_O1 + step * 16, s);
        tmem_ld_wait();
        // exp(G_t - G_s): where the chunk's decays are mild, as a product of two factors (16-bit
        // types; a score that overflows on the way ends in the token-by-token form)
        if (!F32 && d->mild) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 f = *reinterpret_cast<const float4*>(&d->ieg[step * 16 + 4 * j]);
            s[4 * j] = __float_as_uint(__uint_as_float(s[4 * j]) * f.x * et);
            s[4 * j + 1] = __float_as_uint(__uint_as_float(s[4 * j + 1]) * f.y * et);
            s[4 * j + 2] = __float_as_uint(__uint_as_float(s[4 * j + 2]) * f.z * et);
            s[4 * j + 3] = __float_as_uint(__uint_as_float(s[4 * j + 3]) * f.w * et);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float4 gs = d->g[step * 16 + j];
            const float x = ex2((gt.x - gs.x) + (gt.y - gs.y));
            s[j] = gt.z == gs.z ? __float_as_uint(__uint_as_float(s[j]) * x * a.scale) : 0u;
          }
        }
        if (step >= 2 * quarter) {  // (rows 32 .. 63 see all of the first 32 columns)
#pragma unroll
          for (int j = 0; j < 16; ++j) s[j] = step * 16 + j <= row ? s[j] : 0u;
        }
        if (F16) {
#pragma unroll
          for (int j = 0; j < 16; ++j) mx = fmaxf(mx, fabsf(__uint_as_float(s[j])));
        }
      }
      float rs = 1.f;
      if constexpr (F16) {  // a row's threads are in (quarter + 1) NWG / 2 warps
        if (NWG == 4 || quarter == 1) {
          m->pmax[wg][row] = mx;
          asm volatile("bar.sync %0, %1;" ::"r"(2 + quarter), "r"((quarter + 1) * NWG * 16) : "memory");
          for (int i = 0; i < (quarter + 1) * NWG / 2; ++i) mx = fmaxf(mx, m->pmax[i][row]);
        }
        const float2 f = f16_scale(mx);
        rs = f.x;
        if (wg == 0) m->pinv[row] = f.y;
      }
#pragma unroll
      for (int c = 0; c < SPT; ++c) {
        const int step = wg * SPT + c;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t u[4][NPP];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c0 = e * 8 + 2 * j;
            const float p0 = __uint_as_float(sc[c][c0]), p1 = __uint_as_float(sc[c][c0 + 1]);
            split_pair<NPP, F16>(F16 ? p0 * rs : p0, F16 ? p1 * rs : p1, u[j]);
          }
          if (row >= step * 16) {
#pragma unroll
            for (int x = 0; x < NPP; ++x)
              *reinterpret_cast<uint4*>(sm + L::P + x * PTILE + p_base(step) + e * p_pitch(step) +
                                        (row - step * 16) * 16) = make_uint4(u[0][x], u[1][x], u[2][x], u[3][x]);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      asm volatile("bar.arrive 1, %0;" ::"n"(NWG * 48 + 32) : "memory");  // the warps of scores and the issuer's
    }
    if (MODE == 1 && iwarp) {
      asm volatile("bar.sync 1, %0;" ::"n"(NWG * 48 + 32) : "memory");
      tc_fence_after_sync();
      if (elect_one()) {
        each_product<NP, NPP, LIM, CH / 16>(CH / 16, [&](int i, int j, int s, bool first) {
          mma_f16(tm + L::T_O1 + s * 16, desc_mn<NP>(tv + i * TILE, s),
                  smem_desc(sm + L::P + j * PTILE + p_base(s), p_pitch(s), 128), idesc<F16>(128, CH - 16 * s, 1, 0),
                  !first);
        });
        mma_commit(&m->end);
      }
      __syncwarp();
    }
    ok = mbar_wait(&m->end, ph) && ok;
    tc_fence_after_sync();
    if (MODE == 0) {
      add_state(d->lam, kscale.y);
      if (more) put_qk();
      __syncthreads();  // the next decays are there
      continue;
    }
    // ---- outputs ----------------------------------------------------------------------
    // A thread's row is one value channel: turned in v's place into rows of tokens, whole
    // ones for 32-bit types, two halves of 64 channels otherwise.
    T* stage = reinterpret_cast<T*>(sm + L::V);
    constexpr int SW = sizeof(T) == 4 ? D : 64;  // channels of a staged row
    float bad = 0.f;
#pragma unroll
    for (int c = 0; c < TPT / 16; ++c) {
      uint32_t o1[16], o2[16];
      tmem_ld16(tlane + L::T_O1 + wg * TPT + c * 16, o1);
      tmem_ld16(tlane + L::T_O2 + wg * TPT + c * 16, o2);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const int t = wg * TPT + c * 16 + j;
        const float4 e = *reinterpret_cast<const float4*>(&d->eg[t]);
        const float ev[4] = {e.x, e.y, e.z, e.w};
        float pv[4] = {1.f, 1.f, 1.f, 1.f};
        if (F16) {
          const float4 p = *reinterpret_cast<const float4*>(&m->pinv[t]);
          pv[0] = p.x, pv[1] = p.y, pv[2] = p.z, pv[3] = p.w;
        }
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const float y1 = __uint_as_float(o1[j + f]), y2 = __uint_as_float(o2[j + f]);
          const float x = F16 ? fmaf(ev[f], y2 * sinv, y1 * pv[f]) : fmaf(ev[f], y2, y1);
          bad = fmaf(x, 0.f, bad);
          stage[(row / SW) * CH * SW + (t + f) * SW + row % SW] = from_f32<T>(x);
        }
      }
    }
    fence_proxy_async_smem();
    tc_fence_before_sync();
    // a sum of zeros unless a value is not finite (one of the rows past the chunk's tokens, then,
    // costs time and nothing else)
    const bool redo = __syncthreads_or(bad != 0.f && row < a.dv);
    tc_fence_after_sync();
    // the next chunk's scores may take O1's place: its q and k have come meanwhile
    if (!F32 && more) issue_scores(ph ^ 1);
    if (more) put_qk();
    if (redo) {
      token_by_token(t0, n, d);
    } else {
      if (NP == 1 && n == CH) {
        if (iwarp && elect_one()) {
          tma_store(&maps.o, stage, 0, h, t0);
          if (a.dv > 64) tma_store(&maps.o, stage + CH * SW, 64, h, t0);
          store_commit();
        }
      } else {
        constexpr int PC = SW * (int)sizeof(T) / 16;  // 16-byte pieces of a staged row
        for (int i = tid; i < CH * (D / SW) * PC; i += NT) {
          const int t = i / PC % CH, c = i / PC / CH * SW + i % PC * (16 / (int)sizeof(T));
          if (t < n && c < a.dv)
            *reinterpret_cast<uint4*>(o + (t0 + t) * a.os + c) =
                *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(stage) + i * 16);
        }
      }
      add_state(d->lam, kscale.y);
    }
    put_state();
    if (NP == 1 && iwarp && elect_one()) {
      store_wait_read();
      if (more) tma_load_tile(sm + L::V, &maps.v, a.dv, h, t0 + CH, &m->full_v);
    }
    __syncwarp();
  }
  if (NP == 1 && begin < end && iwarp && elect_one()) {  // no copy is left in flight, whatever ended the loop
    const uint32_t p = ok ? ph ^ 1 : ph;
    ok = mbar_wait(&m->full_k, p) && ok;
    if (MODE == 1) ok = mbar_wait(&m->full_q, p) && ok;
    ok = mbar_wait(&m->full_v, p) && ok;
  }
  ok = !__syncthreads_or(!ok);
  if (!ok && tid == 0) atomicOr(ctrl + CTRL_STATUS, DEV_ERR_MBAR_TIMEOUT);
  float* to = MODE == 0 ? mine + (int64_t)a.H * sz : pool;  // what a unit leaves is the next one's start
  if (ok && (MODE == 0 || end == last)) {
#pragma unroll
    for (int j = 0; j < CPT; ++j)
      if (row < a.dv && wg * CPT + j < a.dk) to[(wg * CPT + j) * a.dv + row] = S[j];
  }
  if (MODE == 0 && tid == 0) wd[(int64_t)(un.slot0 + un.i) * a.H + h] = resets ? 0.f : ex2(sum_hi + sum_lo);
  if (NP == 1 && MODE == 1 && iwarp && elect_one()) store_wait_all();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tm, L::T_COLS);
}

// The states before the units of each sequence of several: unit 0's is the sequence's own, and
// each next one adds what the unit between leaves, in order. A thread keeps eight units of
// 2 x 4 values in flight. `by_seq`: a CTA for each sequence, else for each unit, of which the
// first does the work (many sequences, few of them long).
__global__ void __launch_bounds__(256) lin_join(LinattnArgs a, LinattnCut cut, int n_ws, int by_seq, const float* wd,
                                                float* wst) {
  __shared__ int scratch[UNIT_SCRATCH];
  pdl_wait_prior_grids();
  pdl_launch_dependents();  // the output pass may set up
  const Unit un = find_unit(a, cut, n_ws, by_seq ? blockIdx.x : a.B + blockIdx.x, scratch, false);
  if (!un.found || un.n == 1 || (!by_seq && un.i != 0)) return;
  const int slot = seq_slot(a, un.b);
  if (slot < 0) return;
  const int64_t sz = (int64_t)a.dk * a.dv, step = a.H * sz;
  const int h = blockIdx.y, at = (blockIdx.z * 512 + threadIdx.x) * 4;
  const float* pool = a.state + ((int64_t)slot * a.H + h) * sz;
  float* w = wst + ((int64_t)un.slot0 * a.H + h) * sz;
  float4 s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = at + k * 1024;
    if (i >= sz) continue;
    s[k] = a.fresh ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(pool + i);
    *reinterpret_cast<float4*>(w + i) = s[k];
  }
  constexpr int AHEAD = 8;
  for (int u0 = 1; u0 < un.n; u0 += AHEAD) {
    float4 x[AHEAD][2];
    float lam[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int u = min(u0 + j, un.n - 1);
      lam[j] = wd[(int64_t)(un.slot0 + u - 1) * a.H + h];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (at + k * 1024 < sz) x[j][k] = *reinterpret_cast<const float4*>(w + u * step + at + k * 1024);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (u0 + j >= un.n) break;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = at + k * 1024;
        if (i >= sz) continue;
        s[k] = make_float4(fmaf(lam[j], s[k].x, x[j][k].x), fmaf(lam[j], s[k].y, x[j][k].y),
                           fmaf(lam[j], s[k].z, x[j][k].z), fmaf(lam[j], s[k].w, x[j][k].w));
        *reinterpret_cast<float4*>(w + (u0 + j) * step + i) = s[k];
      }
    }
  }
}

template <typename K, typename... Args>
cudaError_t launch(K kern, dim3 grid, int threads, int smem, bool pdl, cudaStream_t st, Args... args) {
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// A [tokens][heads][dim] tensor of 16-bit values in boxes of 64 tokens x 64 columns of one head, rows of
// 128 bytes, in the 128-byte swizzle for operands and as they are for outputs.
cudaError_t make_map(CUtensorMap* m, const void* base, int dim, int heads, int tokens, int64_t stride, bool swizzle) {
  const auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, 64}, es[3] = {1, 1, 1};
  const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int NP, bool WIDE>
cudaError_t chunk_launch(const LinattnArgs& a, int type, uint8_t* ws, bool pdl, cudaStream_t st) {
  LinattnSplit sp = linattn_split(a.N, a.offsets ? a.N : a.seq_len, a.B, a.H, type);
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(ws);
  float* wd = reinterpret_cast<float*>(ws + sp.decays);
  float* wst = reinterpret_cast<float*>(ws + sp.states);
  Maps maps{};
  cudaError_t e = cudaSuccess;
  if (NP == 1 && a.N > 0) {
    const int G = a.H / a.rep;
    if ((e = make_map(&maps.q, a.q, a.dk, G, a.N, a.qs, true)) != cudaSuccess) return e;
    if ((e = make_map(&maps.k, a.k, a.dk, G, a.N, a.ks, true)) != cudaSuccess) return e;
    if ((e = make_map(&maps.v, a.v, a.dv, a.H, a.N, a.vs, true)) != cudaSuccess) return e;
    if ((e = make_map(&maps.o, a.o, a.dv, a.H, a.N, a.os, false)) != cudaSuccess) return e;
  }
  const int smem = Plan<NP>::BYTES + 1024;  // 1,024-byte alignment
  const int rest = sp.cut.rest = a.offsets ? sp.units - a.B : (a.seq_len - 1) / sp.cut.seg * a.B;
  if (rest > 0) {
    e = launch(lin_chunk<T, NP, 0, WIDE>, dim3((unsigned)rest * a.H), chunk_threads(NP), smem, pdl, st, a, maps, sp.cut, sp.n_ws, 0, wd,
               wst, ctrl);
    if (e != cudaSuccess) return e;
    const int by_seq = a.B <= rest;
    const dim3 jgrid((unsigned)(by_seq ? a.B : rest), (unsigned)a.H, (unsigned)((a.dk * a.dv + 2047) / 2048));
    e = launch(lin_join, jgrid, 256, 0, pdl, st, a, sp.cut, sp.n_ws, by_seq, (const float*)wd, wst);
    if (e != cudaSuccess) return e;
  }
  return launch(lin_chunk<T, NP, 1, WIDE>, dim3((unsigned)(rest + a.B) * a.H), chunk_threads(NP), smem, pdl, st, a, maps, sp.cut, sp.n_ws,
                rest > 0 ? 1 : 0, wd, wst, ctrl);
}

}  // namespace

cudaError_t linattn_chunk_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool wide = a.dk > 112;
  if (type == MOE_F32)
    return wide ? chunk_launch<float, 3, true>(a, type, w, pdl, st) : chunk_launch<float, 3, false>(a, type, w, pdl, st);
  if (type == MOE_F16)
    return wide ? chunk_launch<__half, 1, true>(a, type, w, pdl, st) : chunk_launch<__half, 1, false>(a, type, w, pdl, st);
  return wide ? chunk_launch<__nv_bfloat16, 1, true>(a, type, w, pdl, st)
              : chunk_launch<__nv_bfloat16, 1, false>(a, type, w, pdl, st);
}

}  // namespace moe
