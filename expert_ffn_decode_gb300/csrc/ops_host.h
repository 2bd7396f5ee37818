// Host side of the operators next to the step (4-bit matrix-vector product, linear
// attention): the argument blocks their kernels take, their launchers and the error text
// shared with api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/moeffn.h"

namespace moe {

// ---- error text (api.cu) --------------------------------------------------------------
int set_error(int code, const char* fmt, ...);
int set_cuda_error(cudaError_t e, const char* what);
void clear_error();

// ---- 4-bit matrix-vector product (matvec.cu) -------------------------------------------
struct MatvecArgs {
  const void* x;
  const uint8_t* w;
  const uint8_t* scales;  // planes: f16 [rows][groups]
  const uint8_t* mins;    // planes: f16 [rows][groups] or null
  const float* bias;
  void* y;
  int64_t xs, ys;         // values from one vector to the next
  int rows, cols, T;
  int qtype, group, x_type, y_type;
  uint32_t flags;
};
cudaError_t matvec_launch(const MatvecArgs& a, cudaStream_t st);

// ---- linear attention (linattn.cu) ----------------------------------------------------
struct LinattnArgs {
  const void *q, *k, *v;
  const float* g;
  const int32_t* offsets;  // null: equal sequences of `seq_len` tokens
  const int32_t* slots;    // null: sequence b in state b
  float* state;
  void* o;
  int64_t qs, ks, vs, os;  // values from one token to the next
  int B, N, seq_len, H, rep, dk, dv, n_states;  // rep: heads that share a q/k head
  float scale;
  int fresh, token_decay;
};
// How a prompt call is cut: sequences into units of `seg` tokens (a multiple of 64), so that
// units x heads fill the GPU's CTA places about once (152 SMs, two CTAs each; one for f32). A cut
// costs a second pass over k and v, a state's round trip and two launches: one sequence with
// 16 heads of 128 in bf16 takes 21 us whole and 24 cut at 320 tokens, 30 and 25 at 512, 56 and
// 27 at 1024; units of 128 tokens against 256 take 25 and 35 us at 512, 52 and 50 at 4096.
// `units` bounds their number from what the host knows, `n_ws` the states that sequences of
// several units keep in the workspace; the rest are byte offsets in it.
constexpr int LINATTN_MIN_SEG = 128;
struct LinattnSplit {
  int seg, units, n_ws;
  size_t decays, states, total;
};
inline LinattnSplit linattn_split(int N, int B, int H, int dk, int dv, int type) {
  LinattnSplit s{};
  const int places = type == MOE_F32 ? 152 : 304;
  const int want = places / H > 1 ? places / H : 1;
  int64_t seg = ((int64_t)N + want - 1) / want;
  seg = (seg + 63) / 64 * 64;
  if (seg < LINATTN_MIN_SEG) seg = LINATTN_MIN_SEG;
  const int whole = type == MOE_F32 ? 256 : 384;  // f32: 47 us whole and 47 cut at 256 tokens, 57 and 46 at 320
  if (N <= whole) seg = whole;
  s.seg = seg > 1 << 30 ? 1 << 30 : (int)seg;
  s.units = N / s.seg + B;       // sum of ceil(n_b / seg), an empty sequence counting one
  s.n_ws = 2 * (N / s.seg);      // a sequence longer than seg has at most 2 n_b / seg units
  size_t o = 512;
  s.decays = o;
  o = (o + (size_t)s.n_ws * H * 4 + 255) / 256 * 256;
  s.states = o;
  o = (o + (size_t)s.n_ws * H * dk * dv * 4 + 255) / 256 * 256;
  s.total = o;
  return s;
}
cudaError_t linattn_prefill_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st);
cudaError_t linattn_step_launch(const LinattnArgs& a, int type, bool pdl, cudaStream_t st);

}  // namespace moe
