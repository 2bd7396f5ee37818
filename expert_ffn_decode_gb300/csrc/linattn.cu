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

constexpr int SCAN_TOK = 16;  // tokens staged at a time

// A warp holds the state's columns for 8 values of v; lane = 8 * part + column, and the part
// owns the key values 16 j + 4 part + (0 .. 3), so o_t is two shuffles away from its sum.
// A CTA of 4 warps takes 32 columns of one head of one sequence. DKP: key_dim rounded up to
// 64 or 128. The next tokens are on their way while these are walked.
template <typename T, int DKP>
__global__ void __launch_bounds__(128) lin_scan(LinattnArgs a) {
  __shared__ __align__(16) float qs[SCAN_TOK][DKP], ks[SCAN_TOK][DKP], vs[SCAN_TOK][32], ls[SCAN_TOK];
  const int tid = threadIdx.x, lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int col0 = blockIdx.x * 32, lc = (tid >> 5) * 8 + (lane & 7), col = col0 + lc, part = lane >> 3;
  pdl_wait_prior_grids();
  const bool live = col < a.dv;
  int begin, end;
  seq_range(a, b, begin, end);
  const int slot = seq_slot(a, b);
  T* o = static_cast<T*>(a.o) + (int64_t)h * a.dv;
  if (slot < 0) {
    for (int t = begin + part; t < end; t += 4)
      if (live) o[t * a.os + col] = from_f32<T>(0.f);
    return;
  }
  const T* q = static_cast<const T*>(a.q) + (int64_t)(h / a.rep) * a.dk;
  const T* k = static_cast<const T*>(a.k) + (int64_t)(h / a.rep) * a.dk;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv;
  constexpr int QN = SCAN_TOK * DKP / 4 / 128;  // four-value pieces of a thread
  float4 nq[QN], nk[QN], nv;
  float ng = 0.f;
  auto fetch = [&](int t0) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int at = i * 128 + tid, t = t0 + at / (DKP / 4), d = at % (DKP / 4) * 4;
      const bool in = t < end && d < a.dk;
      nq[i] = in ? load4(q + t * a.qs + d) : z;
      nk[i] = in ? load4(k + t * a.ks + d) : z;
    }
    const int t = t0 + tid / 8, d = col0 + tid % 8 * 4;
    nv = t < end && d < a.dv ? load4(v + t * a.vs + d) : z;
    if (tid < SCAN_TOK && t0 + tid < end) ng = a.g[a.token_decay ? (int64_t)(t0 + tid) * a.H + h : h];
  };
  fetch(begin);
  float* st = a.state + ((int64_t)slot * a.H + h) * a.dk * a.dv;
  float S[DKP / 4];
#pragma unroll
  for (int i = 0; i < DKP / 4; ++i) {
    const int d = i / 4 * 16 + part * 4 + i % 4;
    S[i] = live && d < a.dk && !a.fresh ? st[d * a.dv + col] : 0.f;
  }
  for (int t0 = begin; t0 < end; t0 += SCAN_TOK) {
    const int n = min(SCAN_TOK, end - t0);
#pragma unroll
    for (int i = 0; i < QN; ++i) {
      const int at = i * 128 + tid;
      *reinterpret_cast<float4*>(&qs[at / (DKP / 4)][at % (DKP / 4) * 4]) = nq[i];
      *reinterpret_cast<float4*>(&ks[at / (DKP / 4)][at % (DKP / 4) * 4]) = nk[i];
    }
    *reinterpret_cast<float4*>(&vs[tid / 8][tid % 8 * 4]) = nv;
    if (tid < n) ls[tid] = expf(ng);
    __syncthreads();
    if (t0 + SCAN_TOK < end) fetch(t0 + SCAN_TOK);
    for (int t = 0; t < n; ++t) {
      const float lam = ls[t], vv = vs[t][lc];
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < DKP / 16; ++i) {
        const float4 kk = *reinterpret_cast<const float4*>(&ks[t][i * 16 + part * 4]);
        const float4 qq = *reinterpret_cast<const float4*>(&qs[t][i * 16 + part * 4]);
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
      if (live && part == 0) o[(t0 + t) * a.os + col] = from_f32<T>(s * a.scale);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < DKP / 4; ++i) {
    const int d = i / 4 * 16 + part * 4 + i % 4;
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

template <typename T>
cudaError_t scan_launch(const LinattnArgs& a, bool pdl, cudaStream_t st) {
  const dim3 grid((unsigned)((a.dv + 31) / 32), (unsigned)a.H, (unsigned)a.B);
  return a.dk <= 64 ? launch(lin_scan<T, 64>, grid, 128, pdl, st, a) : launch(lin_scan<T, 128>, grid, 128, pdl, st, a);
}

template <typename T>
cudaError_t step_launch(const LinattnArgs& a, bool pdl, cudaStream_t st) {
  if ((int64_t)a.B * a.H >= 304) {  // as many CTAs as two an SM: a whole head each
    const dim3 grid(1, (unsigned)a.H, (unsigned)a.B);
    if (a.dv > 64) return launch(lin_step<T, 32>, grid, 256, pdl, st, a);
    if (a.dv > 32) return launch(lin_step<T, 16>, grid, 256, pdl, st, a);
  }
  return launch(lin_step<T, 8>, dim3((unsigned)((a.dv + 31) / 32), (unsigned)a.H, (unsigned)a.B), 256, pdl, st, a);
}

}  // namespace

cudaError_t linattn_prefill_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st) {
  // Prompts that are walked token by token: as long as that is quicker than one chunk (one
  // sequence, 16 heads of 128: the walk takes 2.3 us and 0.2 us a token, a chunk 8.9 us in bf16,
  // 11 in f16, 16 in f32). With offsets only the total is known here.
  const int most = type == MOE_F32 ? 64 : 36;
  if ((a.offsets ? a.N : a.seq_len) > most) return linattn_chunk_launch(a, type, ws, pdl, st);
  if (type == MOE_F32) return scan_launch<float>(a, pdl, st);
  if (type == MOE_F16) return scan_launch<__half>(a, pdl, st);
  return scan_launch<__nv_bfloat16>(a, pdl, st);
}

cudaError_t linattn_step_launch(const LinattnArgs& a, int type, bool pdl, cudaStream_t st) {
  if (type == MOE_F32) return step_launch<float>(a, pdl, st);
  if (type == MOE_F16) return step_launch<__half>(a, pdl, st);
  return step_launch<__nv_bfloat16>(a, pdl, st);
}

}  // namespace moe
