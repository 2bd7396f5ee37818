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
// shared memory, and a thread owns half a row of S^T in f32 registers.
//
// Rounding: the tensor cores take bf16 parts. A bf16 q, k, v is one part; an f16 one splits
// into two exactly and an f32 one into three (8 bits each, 24 in all). Scores and the state
// as an operand keep two parts (16 bits) for 16-bit outputs and three for f32; the decayed
// keys keep three always, because they are summed into the f32 state. Products of parts
// below the last kept bit are left out. Sums, statistics and the state itself are f32.
#include "linattn.cuh"
#include "tc.cuh"

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
  static constexpr int NPP = NP == 3 ? 3 : 2;  // parts of scores and state operands
  static constexpr uint32_t Q = 0, K = NP * TILE, V = 2 * NP * TILE, KT = 3 * NP * TILE;
  static constexpr uint32_t P = KT + 3 * TILE;
  static constexpr uint32_t MISC = P + NPP * PTILE;
  static constexpr uint32_t BYTES = MISC + 3584;  // bf16: 112,128 bytes, two CTAs an SM
  // tensor memory columns: scores then O1, O2, and the state's parts, whose place A takes
  // once O2 is done
  static constexpr uint32_t T_O1 = 0, T_O2 = 64, T_S = 128, T_A = 128;
  static constexpr uint32_t T_COLS = NP == 3 ? 512 : 256;
};

struct Decays {
  float4 g[CH];      // G_t in powers of two: sum's high and low part, resets so far, exp(g_t)
  float w[CH];       // exp(G_63 - G_s)
  float eg[CH];      // exp(G_t)
  float lam;         // exp(G_63)
  float ghi, glo;    // sum over the chunk without resets
  int reset;         // whether the chunk forgets
};
struct Misc {
  Decays d[2];       // of this chunk and the next
  uint64_t bar;
  uint32_t tmem;
  int scratch[4 + 16];
};
static_assert(sizeof(Misc) <= 3584, "misc");

// bf16 K-major (bit 0) or MN-major (1) operands, f32 accumulator, shape M x N.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int ta, int tb) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)ta << 15 | (uint32_t)tb << 16 | (uint32_t)(N >> 3) << 17 |
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two f32 values as n bf16 parts each, packed in pairs (low half: x0); the parts sum to the
// value to 8 n bits.
template <int n>
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t* out) {
#pragma unroll
  for (int p = 0; p < n; ++p) {
    uint32_t h;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    out[p] = h;
    if (p + 1 < n) {
      x0 -= __uint_as_float(h << 16);
      x1 -= __uint_as_float(h & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// Whether a pair of bf16 holds an infinity or a NaN (an exponent of all ones).
__device__ __forceinline__ uint32_t non_finite(uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Tiles are kept as [column / 8][row][8 columns]: 8 rows x 16 bytes are one core matrix, so the
// same bytes serve as a K-major operand (columns along K: core matrices 1024 bytes apart
// along K, 128 along rows) and as an MN-major one (rows along K: 128 along K, 1024 along columns).
__device__ __forceinline__ uint32_t piece(int kc, int row) { return (uint32_t)(kc * CH + row) * 16u; }

// A thread's share of rows t0 .. t0 + n - 1 (zeros up to 64) of a [tokens][dim] matrix: four
// 8-column pieces of one row. A warp's 32 pieces of one i are 64 contiguous bytes (16-bit
// types) of 8 rows and fill four whole 128-byte lines of shared memory. One bf16 part goes
// to shared memory as it is, asynchronously; other types pass through registers (fetch early,
// put when the tile is free).
template <typename T, int NP>
struct Loader {
  static constexpr int W = NP == 1 ? 1 : sizeof(T) * 2;  // 32-bit words of a piece held here
  uint32_t r[D / 32][W];
  __device__ __forceinline__ void fetch(uint8_t* dst, const T* src, int64_t stride, int t0, int n, int dim) {
    const int lane = threadIdx.x & 31, row = (threadIdx.x >> 5) * 8 + (lane & 7);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int kc = i * 4 + (lane >> 3);
      const bool in = row < n && kc * 8 < dim;
      const T* p = in ? src + (t0 + row) * stride + kc * 8 : src;
      if constexpr (NP == 1) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst + piece(kc, row))), "l"(p),
                     "r"(in ? 16 : 0)
                     : "memory");
      } else {
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
          const uint4 u = in ? reinterpret_cast<const uint4*>(p)[j] : make_uint4(0, 0, 0, 0);
          r[i][4 * j] = u.x;
          r[i][4 * j + 1] = u.y;
          r[i][4 * j + 2] = u.z;
          r[i][4 * j + 3] = u.w;
        }
      }
    }
  }
  __device__ __forceinline__ void put(uint8_t* dst) const {
    if constexpr (NP > 1) {
      const int lane = threadIdx.x & 31, row = (threadIdx.x >> 5) * 8 + (lane & 7);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t u[4][NP];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 x;
          if constexpr (sizeof(T) == 4) x = make_float2(__uint_as_float(r[i][2 * j]), __uint_as_float(r[i][2 * j + 1]));
          else x = __half22float2(*reinterpret_cast<const __half2*>(&r[i][j]));
          split_pair<NP>(x.x, x.y, u[j]);
        }
        uint8_t* d = dst + piece(i * 4 + (lane >> 3), row);
#pragma unroll
        for (int q = 0; q < NP; ++q)
          *reinterpret_cast<uint4*>(d + q * TILE) = make_uint4(u[0][q], u[1][q], u[2][q], u[3][q]);
      }
    }
  }
};
template <int pending>
__device__ __forceinline__ void copies_wait() {  // all but the last `pending` groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(pending) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Eight values of a piece, the parts added up (exact: they do not overlap).
template <int NP>
__device__ __forceinline__ void read_piece(const uint8_t* p, float (&x)[8]) {
#pragma unroll
  for (int q = NP - 1; q >= 0; --q) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + q * TILE);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = lo_f32(w[j]) + (q == NP - 1 ? 0.f : x[2 * j]);
      x[2 * j + 1] = hi_f32(w[j]) + (q == NP - 1 ? 0.f : x[2 * j + 1]);
    }
  }
}

// The products of parts i < NA of one operand and j < NB of the other with i + j <= LIM, each
// in KS steps of 16 along K: the smallest first, because the tensor core's accumulator
// loses up to a last bit with every step, of what it holds by then.
template <int NA, int NB, int LIM, int KS, typename F>
__device__ __forceinline__ void each_product(F f) {
  bool first = true;
#pragma unroll
  for (int sum = LIM; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (i + j == sum)
#pragma unroll
          for (int s = 0; s < KS; ++s, first = false) f(i, j, s, first);
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
  const float gh[2] = {ph, ch}, gl[2] = {pl, cl};
  const int gr[2] = {pr, cr};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = 2 * lane + j;
    m->g[t] = make_float4(gh[j], gl[j], (float)gr[j], expf(raw[j]));
    m->w[t] = gr[j] == er ? ex2((eh - gh[j]) + (el - gl[j])) : 0.f;
    m->eg[t] = gr[j] == 0 ? ex2(gh[j] + gl[j]) : 0.f;
  }
  if (lane == 0) {
    m->lam = er == 0 ? ex2(eh + el) : 0.f;
    m->ghi = eh;
    m->glo = el;
    m->reset = er != 0;
  }
}

// MODE 0: the state that a unit's tokens alone leave, and its decay, into the workspace.
// MODE 1: the outputs, from the state before the unit; the sequence's last unit stores it.
// `wd`: decays [states][H], `wst`: states [states][H][dk][dv]; seg: tokens of a unit.
template <typename T, int NP, int MODE>
__global__ void __launch_bounds__(256, NP == 1 ? 2 : 1)
lin_chunk(LinattnArgs a, int seg, int n_ws, float* wd, float* wst, uint32_t* ctrl) {
  using L = Plan<NP>;
  constexpr int NPP = L::NPP, LIM = NP == 3 ? 2 : 1;  // products of parts i, j with i + j <= LIM
  extern __shared__ __align__(1024) uint8_t sm[];
  Misc* m = reinterpret_cast<Misc*>(sm + L::MISC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2, quarter = warp & 3;
  const int h = blockIdx.y, row = quarter * 32 + lane;  // row: this thread's lane of tensor memory
  pdl_wait_prior_grids();
  const Unit un = find_unit(a, seg, n_ws, blockIdx.x, m->scratch);
  if (!un.found || (MODE == 0 && un.i == un.n - 1)) return;
  int begin, end;
  seq_range(a, un.b, begin, end);
  const int last = end;
  begin += un.i * seg;
  end = min(begin + seg, end);
  const int slot = seq_slot(a, un.b);
  T* o = static_cast<T*>(a.o) + (int64_t)h * a.dv;
  if (slot < 0) {
    if (MODE == 1)
      for (int i = tid; i < (end - begin) * a.dv; i += 256)
        o[(begin + i / a.dv) * a.os + i % a.dv] = from_f32<T>(0.f);
    return;
  }
  if (warp == 0) tmem_alloc(&m->tmem, L::T_COLS);
  if (tid == 0) {
    mbar_init(&m->bar, 1);
    fence_mbar_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = m->tmem, tlane = tm + ((uint32_t)quarter * 32u << 16);
  const T* q = static_cast<const T*>(a.q) + (int64_t)(h / a.rep) * a.dk;
  const T* k = static_cast<const T*>(a.k) + (int64_t)(h / a.rep) * a.dk;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv;
  const int64_t sz = (int64_t)a.dk * a.dv;
  float* pool = a.state + ((int64_t)slot * a.H + h) * sz;
  float* mine = wst + ((int64_t)(un.slot0 + un.i) * a.H + h) * sz;  // sequences of several units

  // S^T: this thread's row, key columns 64 wg .. 64 wg + 63
  float S[64];
  {
    const float* from = un.n > 1 ? mine : pool;
    const bool zero = MODE == 0 || (un.n == 1 && a.fresh);
#pragma unroll
    for (int j = 0; j < 64; ++j)
      S[j] = !zero && row < a.dv && wg * 64 + j < a.dk ? from[(wg * 64 + j) * a.dv + row] : 0.f;
  }
  auto put_state = [&]() {  // the state's parts as an operand in tensor memory
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t u[NPP][16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        uint32_t s[NPP];
        split_pair<NPP>(S[c * 32 + 2 * j], S[c * 32 + 2 * j + 1], s);
#pragma unroll
        for (int p = 0; p < NPP; ++p) u[p][j] = s[p];
      }
#pragma unroll
      for (int p = 0; p < NPP; ++p) tmem_st16(tlane + L::T_S + p * 64 + wg * 32 + c * 16, u[p]);
    }
    tmem_st_wait();
    tc_fence_before_sync();
  };
  if (MODE == 1) put_state();

  uint32_t phase = 0;
  bool ok = true;
  float sum_hi = 0.f, sum_lo = 0.f;
  int resets = 0;
  Loader<T, NP> lq, lk, lv;
  auto fetch_qk = [&](int t0) {
    const int n = min(CH, end - t0);
    if (t0 < end) {
      if (MODE == 1) lq.fetch(sm + L::Q, q, a.qs, t0, n, a.dk);
      lk.fetch(sm + L::K, k, a.ks, t0, n, a.dk);
    }
    copies_commit();
  };
  auto put_qk = [&]() {
    if (MODE == 1) lq.put(sm + L::Q);
    lk.put(sm + L::K);
  };
  // the state before the products that read it, and the state after the chunk's share
  auto add_state = [&](float lam) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t r[16];
      tmem_ld16(tlane + L::T_A + wg * 64 + c * 16, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) S[c * 16 + j] = fmaf(lam, S[c * 16 + j], __uint_as_float(r[j]));
    }
  };
  // A masked product with an infinity or a NaN is a NaN, which would reach the chunk's earlier
  // tokens: a chunk whose v holds one goes token by token, from global memory.
  auto token_by_token = [&](int t0, int n, const Decays* d) {
    float* part = reinterpret_cast<float*>(sm + L::V);
    for (int t = 0; t < n; ++t) {
      const float vv = row < a.dv ? to_f32(v[(t0 + t) * a.vs + row]) : 0.f;
      const float lam = d->g[t].w;
      float acc = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const int at = wg * 64 + c * 4;
        if (at < a.dk) {
          const float4 kk = load4(k + (t0 + t) * a.ks + at);
          const float4 qq = MODE == 1 ? load4(q + (t0 + t) * a.qs + at) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float k4[4] = {kk.x, kk.y, kk.z, kk.w}, q4[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            S[c * 4 + j] = fmaf(lam, S[c * 4 + j], k4[j] * vv);
            acc = fmaf(q4[j], S[c * 4 + j], acc);
          }
        }
      }
      if (MODE == 1) {
        if (wg == 1) part[row] = acc;
        __syncthreads();
        if (wg == 0 && row < a.dv) o[(t0 + t) * a.os + row] = from_f32<T>((acc + part[row]) * a.scale);
        __syncthreads();
      }
    }
  };
  auto v_non_finite = [&](const uint8_t* tile) {  // among this thread's own pieces
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(tile + piece(i * 4 + (lane >> 3), warp * 8 + (lane & 7)));
      bad |= non_finite(u.x) | non_finite(u.y) | non_finite(u.z) | non_finite(u.w);
    }
    return bad != 0;
  };

  if (warp == 7) chunk_decays(a, h, begin, min(CH, end - begin), &m->d[0]);
  fetch_qk(begin);
  put_qk();
  int buf = 0;
  for (int t0 = begin; t0 < end && ok; t0 += CH, buf ^= 1) {
    const int n = min(CH, end - t0);
    const Decays* d = &m->d[buf];
    copies_wait<0>();
    fence_proxy_async_smem();
    __syncthreads();  // q and k are there; the last chunk's outputs have left v's place
    tc_fence_after_sync();
    lv.fetch(sm + L::V, v, a.vs, t0, n, a.dv);
    copies_commit();
    sum_lo += d->glo;
    {
      const float s = sum_hi + d->ghi, bb = s - sum_hi;
      sum_lo += (sum_hi - (s - bb)) + (d->ghi - bb);
      sum_hi = s;
    }
    resets |= d->reset;
    // ---- scores and the state's share ----------------------------------------------
    if (MODE == 1 && tid == 0) {
      each_product<NP, NP, LIM, D / 16>([&](int i, int j, int s, bool first) {
        mma_f16(tm + L::T_O1, smem_desc(sm + L::Q + i * TILE + s * 2048, 1024, 128),
                smem_desc(sm + L::K + j * TILE + s * 2048, 1024, 128), idesc_bf16(128, CH, 0, 0), !first);
      });
      each_product<NPP, NP, LIM, D / 16>([&](int i, int j, int s, bool first) {
        mma_ts(tm + L::T_O2, tm + L::T_S + i * 64 + s * 8, smem_desc(sm + L::Q + j * TILE + s * 2048, 1024, 128),
               idesc_bf16(128, CH, 0, 0), !first);
      });
      mma_commit(&m->bar);
    }
    // the decayed keys, three parts
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int r = warp * 8 + (lane & 7);
      const uint32_t at = piece(i * 4 + (lane >> 3), r);
      const float w = d->w[r];
      float x[8];
      read_piece<NP>(sm + L::K + at, x);
      uint32_t u[4][3];
#pragma unroll
      for (int j = 0; j < 4; ++j) split_pair<3>(x[2 * j] * w, x[2 * j + 1] * w, u[j]);
#pragma unroll
      for (int p = 0; p < 3; ++p)
        *reinterpret_cast<uint4*>(sm + L::KT + p * TILE + at) = make_uint4(u[0][p], u[1][p], u[2][p], u[3][p]);
    }
    if (MODE == 1) {
      ok = mbar_wait(&m->bar, phase);
      phase ^= 1;
      tc_fence_after_sync();
    }
    __syncthreads();  // q and k have been read: the next chunk's may come
    fetch_qk(t0 + CH);
    if (warp == 7 && t0 + CH < end) chunk_decays(a, h, t0 + CH, min(CH, end - t0 - CH), &m->d[buf ^ 1]);
    if (MODE == 1 && quarter < 2 && wg <= quarter) {
      // Lanes 0 .. 63 hold the tokens' rows of scores; columns 32 wg .. 32 wg + 31 here, of
      // which the mask leaves none for rows below 32 and wg 1.
      const float4 gt = d->g[row];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int step = wg * 2 + c;  // of the product over s
        uint32_t s[16];
        tmem_ld16(tlane + L::T_O1 + step * 16, s);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t u[4][NPP];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float p[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int col = step * 16 + e * 8 + 2 * j + f;
              const float4 gs = d->g[col];
              const float x = ex2((gt.x - gs.x) + (gt.y - gs.y));
              p[f] = col <= row && gt.z == gs.z ? __uint_as_float(s[e * 8 + 2 * j + f]) * x : 0.f;
            }
            split_pair<NPP>(p[0], p[1], u[j]);
          }
          if (row >= step * 16) {
#pragma unroll
            for (int x = 0; x < NPP; ++x)
              *reinterpret_cast<uint4*>(sm + L::P + x * PTILE + p_base(step) + e * p_pitch(step) +
                                        (row - step * 16) * 16) = make_uint4(u[0][x], u[1][x], u[2][x], u[3][x]);
          }
        }
      }
    }
    lv.put(sm + L::V);
    copies_wait<1>();
    fence_proxy_async_smem();
    tc_fence_before_sync();
    if (__syncthreads_or(v_non_finite(sm + L::V))) {
      token_by_token(t0, n, d);
      put_qk();
      if (MODE == 1) put_state();
      ok = !__syncthreads_or(!ok);
      continue;
    }
    tc_fence_after_sync();
    // ---- the chunk's own share, and what it adds to the state ------------------------------
    if (tid == 0) {
      if (MODE == 1)
        each_product<NP, NPP, LIM, CH / 16>([&](int i, int j, int s, bool first) {
          mma_f16(tm + L::T_O1 + s * 16, smem_desc(sm + L::V + i * TILE + s * 256, 128, 1024),
                  smem_desc(sm + L::P + j * PTILE + p_base(s), p_pitch(s), 128), idesc_bf16(128, CH - 16 * s, 1, 0),
                  !first);
        });
      each_product<NP, 3, 2, CH / 16>([&](int i, int j, int s, bool first) {
        mma_f16(tm + L::T_A, smem_desc(sm + L::V + i * TILE + s * 256, 128, 1024),
                smem_desc(sm + L::KT + j * TILE + s * 256, 128, 1024), idesc_bf16(128, D, 1, 1), !first);
      });
      mma_commit(&m->bar);
    }
    ok = mbar_wait(&m->bar, phase) && ok;
    phase ^= 1;
    tc_fence_after_sync();
    add_state(d->lam);
    if (MODE == 1) {
      // outputs, a thread's row is one value channel: turned in v's place into rows of tokens
      T* stage = reinterpret_cast<T*>(sm + L::V);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t o1[16], o2[16];
        tmem_ld16(tlane + L::T_O1 + wg * 32 + c * 16, o1);
        tmem_ld16(tlane + L::T_O2 + wg * 32 + c * 16, o2);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int t = wg * 32 + c * 16 + j;
          const float x = fmaf(d->eg[t], __uint_as_float(o2[j]), __uint_as_float(o1[j]));
          stage[t * D + row] = from_f32<T>(x * a.scale);
        }
      }
    }
    put_qk();
    tc_fence_before_sync();
    ok = !__syncthreads_or(!ok);
    tc_fence_after_sync();
    if (MODE == 1) {
      put_state();
      constexpr int PC = D * (int)sizeof(T) / 16;  // 16-byte pieces of a token's row
#pragma unroll
      for (int i = 0; i < CH * PC / 256; ++i) {
        const int t = (i * 256 + tid) / PC, c = (i * 256 + tid) % PC;
        if (t < n && c * (16 / (int)sizeof(T)) < a.dv)
          *reinterpret_cast<uint4*>(o + (t0 + t) * a.os + c * (16 / sizeof(T))) =
              *reinterpret_cast<const uint4*>(sm + L::V + (i * 256 + tid) * 16);
      }
    }
  }
  copies_wait<0>();
  if (!ok && tid == 0) atomicOr(ctrl + CTRL_STATUS, DEV_ERR_MBAR_TIMEOUT);
  float* to = MODE == 0 ? mine + (int64_t)a.H * sz : pool;  // what a unit leaves is the next one's start
  if (ok && (MODE == 0 || end == last)) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (row < a.dv && wg * 64 + j < a.dk) to[(wg * 64 + j) * a.dv + row] = S[j];
  }
  if (MODE == 0 && tid == 0) wd[(int64_t)(un.slot0 + un.i) * a.H + h] = resets ? 0.f : ex2(sum_hi + sum_lo);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tm, L::T_COLS);
}

// The states before the units of each sequence of several: unit 0's is the sequence's own, and
// each next one adds what the unit between leaves, in order.
__global__ void __launch_bounds__(256) lin_join(LinattnArgs a, int seg, int n_ws, const float* wd, float* wst) {
  __shared__ int scratch[4 + 16];
  pdl_wait_prior_grids();
  const Unit un = find_unit(a, seg, n_ws, blockIdx.x, scratch);
  if (!un.found || un.i != 0 || un.n == 1) return;
  const int slot = seq_slot(a, un.b);
  if (slot < 0) return;
  const int64_t sz = (int64_t)a.dk * a.dv, step = a.H * sz;
  const int i = (blockIdx.z * 256 + threadIdx.x) * 4, h = blockIdx.y;
  if (i >= sz) return;
  float* w = wst + ((int64_t)un.slot0 * a.H + h) * sz + i;
  float4 s = a.fresh ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : *reinterpret_cast<const float4*>(a.state + ((int64_t)slot * a.H + h) * sz + i);
  *reinterpret_cast<float4*>(w) = s;
  for (int u = 1; u < un.n; ++u) {
    w += step;
    const float lam = wd[(int64_t)(un.slot0 + u - 1) * a.H + h];
    const float4 x = *reinterpret_cast<const float4*>(w);
    s = make_float4(fmaf(lam, s.x, x.x), fmaf(lam, s.y, x.y), fmaf(lam, s.z, x.z), fmaf(lam, s.w, x.w));
    *reinterpret_cast<float4*>(w) = s;
  }
}

template <typename K, typename... Args>
cudaError_t launch(K kern, dim3 grid, int smem, bool pdl, cudaStream_t st, Args... args) {
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, int NP>
cudaError_t chunk_launch(const LinattnArgs& a, uint8_t* ws, bool pdl, cudaStream_t st) {
  const LinattnSplit sp = linattn_split(a.N, a.B, a.H, a.dk, a.dv);
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(ws);
  float* wd = reinterpret_cast<float*>(ws + sp.decays);
  float* wst = reinterpret_cast<float*>(ws + sp.states);
  const dim3 grid((unsigned)sp.units, (unsigned)a.H);
  const bool several = a.offsets ? sp.units > a.B : a.seq_len > sp.seg;
  cudaError_t e = cudaSuccess;
  if (several) {
    e = launch(lin_chunk<T, NP, 0>, grid, Plan<NP>::BYTES, pdl, st, a, sp.seg, sp.n_ws, wd, wst, ctrl);
    if (e != cudaSuccess) return e;
    const dim3 jgrid((unsigned)sp.units, (unsigned)a.H, (unsigned)((a.dk * a.dv + 1023) / 1024));
    e = launch(lin_join, jgrid, 0, pdl, st, a, sp.seg, sp.n_ws, (const float*)wd, wst);
    if (e != cudaSuccess) return e;
  }
  return launch(lin_chunk<T, NP, 1>, grid, Plan<NP>::BYTES, pdl, st, a, sp.seg, sp.n_ws, wd, wst, ctrl);
}

}  // namespace

cudaError_t linattn_chunk_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (type == MOE_F32) return chunk_launch<float, 3>(a, w, pdl, st);
  if (type == MOE_F16) return chunk_launch<__half, 2>(a, w, pdl, st);
  return chunk_launch<__nv_bfloat16, 1>(a, w, pdl, st);
}

}  // namespace moe
