// Linear attention with a decay for each head: per sequence and head, with the state S
// [key_dim][value_dim] in f32,
//   S = exp(g_t) S + k_t v_t^T,   o_t = scale * S^T q_t.
//
// lin_scan walks a sequence's tokens in turn with the state in registers.
#include "linattn.cuh"

namespace moe {
namespace {

constexpr int SCAN_TOK = 16;  // tokens staged at a time

// A warp holds the state's columns for 8 values of v; lane = 8 * part + column, and the part
// owns the key values 16 j + 4 part + (0 .. 3), so o_t is two shuffles away from its sum.
// A CTA of 4 warps takes 32 columns of one head of one sequence. DKP: key_dim rounded up to
// 64 or 128.
template <typename T, int DKP>
__global__ void __launch_bounds__(128) lin_scan(LinattnArgs a) {
  __shared__ float qs[SCAN_TOK][DKP], ks[SCAN_TOK][DKP], vs[SCAN_TOK][32], ls[SCAN_TOK];
  const int tid = threadIdx.x, lane = tid & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int col0 = blockIdx.x * 32, lc = tid >> 5 << 3 | (lane & 7), col = col0 + lc, part = lane >> 3;
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
  float* st = a.state + ((int64_t)slot * a.H + h) * a.dk * a.dv;
  float S[DKP / 4];
#pragma unroll
  for (int i = 0; i < DKP / 4; ++i) {
    const int d = i / 4 * 16 + part * 4 + i % 4;
    S[i] = live && d < a.dk && !a.fresh ? st[d * a.dv + col] : 0.f;
  }
  const T* q = static_cast<const T*>(a.q) + (int64_t)(h / a.rep) * a.dk;
  const T* k = static_cast<const T*>(a.k) + (int64_t)(h / a.rep) * a.dk;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv;
  for (int t0 = begin; t0 < end; t0 += SCAN_TOK) {
    const int n = min(SCAN_TOK, end - t0);
    for (int i = tid; i < n * DKP; i += 128) {
      const int t = i / DKP, d = i % DKP;
      qs[t][d] = d < a.dk ? to_f32(q[(t0 + t) * a.qs + d]) : 0.f;
      ks[t][d] = d < a.dk ? to_f32(k[(t0 + t) * a.ks + d]) : 0.f;
    }
    for (int i = tid; i < n * 32; i += 128)
      vs[i / 32][i % 32] = col0 + i % 32 < a.dv ? to_f32(v[(t0 + i / 32) * a.vs + col0 + i % 32]) : 0.f;
    if (tid < n) ls[tid] = expf(a.g[a.token_decay ? (int64_t)(t0 + tid) * a.H + h : h]);
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float lam = ls[t], vv = vs[t][lc];
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < DKP / 4; ++i) {
        const int d = i / 4 * 16 + part * 4 + i % 4;
        S[i] = fmaf(lam, S[i], ks[t][d] * vv);
        acc = fmaf(qs[t][d], S[i], acc);
      }
      acc += __shfl_xor_sync(0xffffffffu, acc, 8);
      acc += __shfl_xor_sync(0xffffffffu, acc, 16);
      if (live && part == 0) o[(t0 + t) * a.os + col] = from_f32<T>(acc * a.scale);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < DKP / 4; ++i) {
    const int d = i / 4 * 16 + part * 4 + i % 4;
    if (live && d < a.dk) st[d * a.dv + col] = S[i];
  }
}

template <typename T>
cudaError_t scan_launch(const LinattnArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.dv + 31) / 32), (unsigned)a.H, (unsigned)a.B);
  if (a.dk <= 64) lin_scan<T, 64><<<grid, 128, 0, st>>>(a);
  else lin_scan<T, 128><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t linattn_prefill_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st) {
  if (a.N > 48) return linattn_chunk_launch(a, type, ws, pdl, st);
  return linattn_step_launch(a, type, pdl, st);
}

cudaError_t linattn_step_launch(const LinattnArgs& a, int type, bool pdl, cudaStream_t st) {
  if (type == MOE_F32) return scan_launch<float>(a, st);
  if (type == MOE_F16) return scan_launch<__half>(a, st);
  return scan_launch<__nv_bfloat16>(a, st);
}

}  // namespace moe
