// Linear attention with a decay for each head: per sequence and head, with the state S
// [key_dim][value_dim] in f32,
//   S = exp(g_t) S + k_t v_t^T,   o_t = scale * S^T q_t.
//
// lin_step takes one token of every sequence; lin_scan walks the tokens of short prompts with
// the state in registers; longer prompts go by chunks on the tensor cores (linattn_tc.cu).
#include "linattn.cuh"

namespace moe {
namespace {

// One token: the state is read and written once and everything else is small, so the kernel
// is a stream of the states (128 KB a head) and bound by it. 256 threads take COLS * 4 value
// columns of one head: a thread owns 4 neighbouring columns of every GROUPS-th run of rows, so
// a warp's load is whole lines, all of a thread's loads are in flight together, and the
// outputs are joined over the row groups in order. COLS 32 or 16 is a whole head; calls with
// few heads take 8 (up to four CTAs a head), so that one sequence already spreads over the GPU.
template <typename T, int COLS>
__global__ void __launch_bounds__(256) lin_step(LinattnArgs a) {
  constexpr int GROUPS = 256 / COLS, ROWS = 128 / GROUPS;
  __shared__ float qs[128], ks[128];
  __shared__ float4 part[GROUPS][COLS];
  const int tid = threadIdx.x, c = tid % COLS, grp = tid / COLS;
  const int h = blockIdx.y, b = blockIdx.z, col = (blockIdx.x * COLS + c) * 4;
  pdl_wait_prior_grids();
  const int slot = seq_slot(a, b);
  const bool live = col < a.dv;
  T* o = static_cast<T*>(a.o) + b * a.os + (int64_t)h * a.dv;
  if (slot < 0) {
    if (live && grp == 0)
      for (int j = 0; j < 4; ++j) o[col + j] = from_f32<T>(0.f);
    return;
  }
  float* st = a.state + ((int64_t)slot * a.H + h) * a.dk * a.dv + col;
  float4 S[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int d = grp * ROWS + i;
    S[i] = live && d < a.dk && !a.fresh ? *reinterpret_cast<const float4*>(st + d * a.dv)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int hq = h / a.rep;
  if (tid < 128) {
    const T* k = static_cast<const T*>(a.k) + b * a.ks + (int64_t)hq * a.dk;
    ks[tid] = tid < a.dk ? to_f32(k[tid]) : 0.f;
  } else {
    const T* q = static_cast<const T*>(a.q) + b * a.qs + (int64_t)hq * a.dk;
    qs[tid - 128] = tid - 128 < a.dk ? to_f32(q[tid - 128]) : 0.f;
  }
  const float4 v = live ? load4(static_cast<const T*>(a.v) + b * a.vs + (int64_t)h * a.dv + col)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  const float lam = expf(a.g[a.token_decay ? (int64_t)b * a.H + h : h]);
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int d = grp * ROWS + i;
    const float k = ks[d], q = qs[d];
    S[i].x = fmaf(lam, S[i].x, k * v.x);
    S[i].y = fmaf(lam, S[i].y, k * v.y);
    S[i].z = fmaf(lam, S[i].z, k * v.z);
    S[i].w = fmaf(lam, S[i].w, k * v.w);
    acc.x = fmaf(q, S[i].x, acc.x);
    acc.y = fmaf(q, S[i].y, acc.y);
    acc.z = fmaf(q, S[i].z, acc.z);
    acc.w = fmaf(q, S[i].w, acc.w);
    if (live && d < a.dk) *reinterpret_cast<float4*>(st + d * a.dv) = S[i];
  }
  part[grp][c] = acc;
  __syncthreads();
  if (tid < COLS * 4) {
    const int at = blockIdx.x * COLS * 4 + tid;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < GROUPS; ++r) s += reinterpret_cast<const float*>(&part[r][0])[tid];
    if (at < a.dv) o[at] = from_f32<T>(s * a.scale);
  }
}

// A warp holds 8 columns of the state, or a quarter of their rows (KQ 4); lane = 8 * part +
// column, and the part owns the key values 16 j + 4 part + (0 .. 3) of the warp's, so a warp's
// share of o_t is two shuffles away. A CTA takes 32 columns of one head of one sequence in four
// warps, or 16 in eight, whose shares are joined when the staged tokens have been walked. DKP:
// key_dim rounded up to 64 or 128. What bounds a short prompt is each token's chain of shared
// memory reads, products and shuffles: 16 heads take 2.5 us and 0.1 us a token. The next tokens
// are on their way while these are walked.
template <typename T, int DKP, int KQ>
__global__ void __launch_bounds__(KQ == 1 ? 128 : 256) lin_scan(LinattnArgs a) {
  constexpr int COLS = KQ == 1 ? 32 : 16, NT = COLS * 4 * KQ, TOK = KQ == 1 ? 16 : 32;  // TOK: tokens staged at a time
  __shared__ __align__(16) float qs[TOK][DKP], ks[TOK][DKP], vs[TOK][COLS], ls[TOK];
  __shared__ float shares[KQ == 1 ? 1 : TOK][KQ][COLS];
  const int tid = threadIdx.x, lane = tid & 31, kq = tid / 32 % KQ;
  const int h = blockIdx.y, b = blockIdx.z;
  const int col0 = blockIdx.x * COLS, lc = tid / (32 * KQ) * 8 + (lane & 7), col = col0 + lc, part = lane >> 3;
  pdl_wait_prior_grids();
  const bool live = col < a.dv;
  int begin, end;
  seq_range(a, b, begin, end);
  const int slot = seq_slot(a, b);
  T* o = static_cast<T*>(a.o) + (int64_t)h * a.dv;
  if (slot < 0) {
    for (int t = begin + kq * 4 + part; t < end; t += 4 * KQ)
      if (live) o[t * a.os + col] = from_f32<T>(0.f);
    return;
  }
  const T* q = static_cast<const T*>(a.q) + (int64_t)(h / a.rep) * a.dk;
  const T* k = static_cast<const T*>(a.k) + (int64_t)(h / a.rep) * a.dk;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv;
  constexpr int QN = TOK * DKP / 4 / NT;  // four-value pieces of a thread
  float4 nq[QN], nk[QN], nv;
  float ng = 0.f;
  auto fetch = [&](int t0) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int at = i * NT + tid, t = t0 + at / (DKP / 4), d = at % (DKP / 4) * 4;
      const bool in = t < end && d < a.dk;
      nq[i] = in ? load4(q + t * a.qs + d) : z;
      nk[i] = in ? load4(k + t * a.ks + d) : z;
    }
    const int t = t0 + tid / (COLS / 4), d = col0 + tid % (COLS / 4) * 4;
    nv = tid < TOK * COLS / 4 && t < end && d < a.dv ? load4(v + t * a.vs + d) : z;
    if (tid < TOK && t0 + tid < end) ng = a.g[a.token_decay ? (int64_t)(t0 + tid) * a.H + h : h];
  };
  fetch(begin);
  float* st = a.state + ((int64_t)slot * a.H + h) * a.dk * a.dv;
  constexpr int ROWS = DKP / 4 / KQ;
  float S[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int d = kq * (DKP / KQ) + i / 4 * 16 + part * 4 + i % 4;
    S[i] = live && d < a.dk && !a.fresh ? st[d * a.dv + col] : 0.f;
  }
  for (int t0 = begin; t0 < end; t0 += TOK) {
    const int n = min(TOK, end - t0);
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int at = i * NT + tid;
      *reinterpret_cast<float4*>(&qs[at / (DKP / 4)][at % (DKP / 4) * 4]) = nq[i];
      *reinterpret_cast<float4*>(&ks[at / (DKP / 4)][at % (DKP / 4) * 4]) = nk[i];
    }
    if (tid < TOK * COLS / 4) *reinterpret_cast<float4*>(&vs[tid / (COLS / 4)][tid % (COLS / 4) * 4]) = nv;
    if (tid < n) ls[tid] = expf(ng);
    __syncthreads();
    if (t0 + TOK < end) fetch(t0 + TOK);
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      const float lam = ls[t], vv = vs[t][lc];
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) {
        const int d = kq * (DKP / KQ) + i * 16 + part * 4;
        const float4 kk = *reinterpret_cast<const float4*>(&ks[t][d]);
        const float4 qq = *reinterpret_cast<const float4*>(&qs[t][d]);
        const float k4[4] = {kk.x, kk.y, kk.z, kk.w}, q4[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          S[i * 4 + j] = fmaf(lam, S[i * 4 + j], k4[j] * vv);
          acc[j] = fmaf(q4[j], S[i * 4 + j], acc[j]);
        }
      }
      float s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (KQ > 1) {
        if (part == 0) shares[t][kq][lc] = s;
      } else if (live && part == 0) {
        o[(t0 + t) * a.os + col] = from_f32<T>(s * a.scale);
      }
    }
    __syncthreads();
    if (KQ > 1) {
      for (int i = tid; i < n * COLS; i += NT) {
        const int t = i / COLS, c = i % COLS;
        if (col0 + c >= a.dv) continue;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < KQ; ++w) s += shares[t][w][c];
        o[(t0 + t) * a.os + col0 + c] = from_f32<T>(s * a.scale);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int d = kq * (DKP / KQ) + i / 4 * 16 + part * 4 + i % 4;
    if (live && d < a.dk) st[d * a.dv + col] = S[i];
  }
}

template <typename K>
cudaError_t launch(K kern, dim3 grid, int threads, bool pdl, cudaStream_t st, const LinattnArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, int KQ>
cudaError_t scan_launch(const LinattnArgs& a, bool pdl, cudaStream_t st) {
  constexpr int COLS = KQ == 1 ? 32 : 16;
  const dim3 grid((unsigned)((a.dv + COLS - 1) / COLS), (unsigned)a.H, (unsigned)a.B);
  return a.dk <= 64 ? launch(lin_scan<T, 64, KQ>, grid, COLS * 4 * KQ, pdl, st, a)
                    : launch(lin_scan<T, 128, KQ>, grid, COLS * 4 * KQ, pdl, st, a);
}

template <typename T>
cudaError_t step_launch(const LinattnArgs& a, bool pdl, cudaStream_t st) {
  // As many CTAs as two an SM: a whole head each (96 sequences x 32 heads 61.7 us, 63.0 in quarters);
  // narrow heads in narrow CTAs (37 sequences x 10 heads of 72 x 40 3.0 us, 3.3 in parts of 32
  // columns, 4.2 with 128).
  if ((int64_t)a.B * a.H >= 304) {
    const dim3 grid(1, (unsigned)a.H, (unsigned)a.B);
    if (a.dv > 64) return launch(lin_step<T, 32>, grid, 256, pdl, st, a);
    if (a.dv > 32) return launch(lin_step<T, 16>, grid, 256, pdl, st, a);
  }
  return launch(lin_step<T, 8>, dim3((unsigned)((a.dv + 31) / 32), (unsigned)a.H, (unsigned)a.B), 256, pdl, st, a);
}

// Whether a walk takes CTAs of 16 columns: if they are one an SM at most (64 tokens: 16 heads 9.0 us,
// 12.8 with 32 columns; 32 heads 12.4 and 12.9; 64 heads 23.4 and 17.8).
bool scan_few(const LinattnArgs& a) { return (int64_t)a.B * a.H * ((a.dv + 15) / 16) <= 152; }

// Whether walking the tokens is quicker than chunks, by what each takes in ns at widths of 128
// (heads: of all sequences). The walk: launch, the states both ways, each token of the longest
// sequence and, where heads fill the SMs, each token of each head. Chunks: a chain of them for
// a sequence, or waves of heads. Measured with keys and values of 128 (other widths follow the same
// lines: narrower values walk in fewer CTAs, narrower keys are not in the estimate), us, walk / bf16
// chunks (f32 chunks):
//   tokens x heads    32 x 16: 5.2 / 10.1 (13.7)   64 x 16: 8.9 / 9.8 (15.5)   128 x 16: 16.1 / 13.0 (25.6)
//                     32 x 64: 10.0 / 10.7 (13.9)  32 x 256: 27 / 14.5 (27)   4 x 2048: 53 / 92 (178)
//                     16 x 2048: 116 / 95 (186)
// With offsets only the total is known here: one sequence may have all of it. Beyond 256 tokens
// chunks are cut into units that run side by side.
bool scan_is_quicker(const LinattnArgs& a, int type, bool few) {
  const double heads = (double)a.B * a.H, longest = a.offsets ? a.N : a.seq_len, work = (double)a.N * a.H;
  if (longest > 256) return false;
  const double cols = ((a.dv + 31) / 32) / 4.0, chunks = ((int)longest + 63) / 64;
  const double crowd = work - 32 * longest;
  const double scan = 2300 + 20 * heads * cols + (few ? 108 : 165) * longest + (crowd > 0 ? 2.6 * crowd * cols : 0);
  double chain, wave;
  if (type == MOE_F32) {
    chain = 5200 + 10250 * chunks;
    wave = heads * (52 + 63 * chunks);
  } else if (type == MOE_F16) {
    chain = 7000 + 4000 * chunks;
    wave = heads * (38 + 17 * chunks);
  } else {
    chain = 7000 + 3000 * chunks;
    wave = heads * (36 + 14 * chunks);
  }
  return scan < (chain > wave ? chain : wave);
}

}  // namespace

cudaError_t linattn_prefill_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st) {
  const bool few = scan_few(a);
  if (!scan_is_quicker(a, type, few)) return linattn_chunk_launch(a, type, ws, pdl, st);
  if (type == MOE_F32) return few ? scan_launch<float, 4>(a, pdl, st) : scan_launch<float, 1>(a, pdl, st);
  if (type == MOE_F16) return few ? scan_launch<__half, 4>(a, pdl, st) : scan_launch<__half, 1>(a, pdl, st);
  return few ? scan_launch<__nv_bfloat16, 4>(a, pdl, st) : scan_launch<__nv_bfloat16, 1>(a, pdl, st);
}

cudaError_t linattn_step_launch(const LinattnArgs& a, int type, bool pdl, cudaStream_t st) {
  if (type == MOE_F32) return step_launch<float>(a, pdl, st);
  if (type == MOE_F16) return step_launch<__half>(a, pdl, st);
  return step_launch<__nv_bfloat16>(a, pdl, st);
}

}  // namespace moe
