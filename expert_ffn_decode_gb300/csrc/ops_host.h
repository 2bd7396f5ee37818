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
// costs a second pass over k and v, a state's round trip and two launches, so a call stays whole
// if its longest sequence has no more than `whole` tokens, which then take no longer in one
// piece than two passes over `seg`. One sequence with 16 heads of 128 in bf16 takes 21 us whole
// and 24 cut at 320 tokens, 30 and 25 at 512, 56 and 27 at 1024 (f16 on the same line, which it
// crosses earlier: 26 and 28 at 320, 30 and 28 at 384; f32 46 and 44 at 256, 57 and 43 at 320);
// 8 sequences of 512 tokens 35 and 51, 16 of 448 43 and 92; units of 128 tokens against
// 256 take 25 and 35 us at 512, 52 and 50 at 4096. All measured with 16 heads of 128.
// `longest` bounds a sequence's tokens: with offsets the host knows the total alone, and where
// that leaves it open the kernels look (`ask`).
// `units` bounds the units' number, `n_ws` the states that sequences of several units keep in the
// workspace; the rest are byte offsets in it.
constexpr int LINATTN_MIN_SEG = 128;
struct LinattnCut {
  int seg, whole;
  int ask;   // whether to stay whole is up to the offsets
  int rest;  // units but the sequences' last ones that are launched
};
struct LinattnSplit {
  LinattnCut cut;
  int units, n_ws;
  size_t decays, states;
};
inline int linattn_units_wanted(int H, int type) {
  const int places = type == MOE_F32 ? 152 : 304;
  return places / H > 1 ? places / H : 1;
}
inline int64_t linattn_whole(int64_t seg, int type) {
  return (type == MOE_F32 ? 48 + seg * 33 / 20 : 144 + seg * 9 / 4) / 64 * 64;
}
inline LinattnSplit linattn_split(int N, int longest, int B, int H, int type) {
  LinattnSplit s{};
  const int want = linattn_units_wanted(H, type);
  int64_t seg = ((int64_t)N + want - 1) / want;
  seg = (seg + 63) / 64 * 64;
  if (seg < LINATTN_MIN_SEG) seg = LINATTN_MIN_SEG;
  if (seg > 1 << 28) seg = 1 << 28;
  const int64_t whole = linattn_whole(seg, type);
  if (longest <= whole) seg = whole;
  s.cut = {(int)seg, (int)whole, longest > whole && (longest + B - 1) / B <= whole, 0};
  const int cuts = longest <= whole ? 0 : N / s.cut.seg;
  s.units = cuts + B;         // sum of ceil(n_b / seg), an empty sequence counting one
  s.n_ws = 2 * cuts;          // a sequence longer than seg has at most 2 n_b / seg units
  s.decays = 512;
  s.states = (s.decays + (size_t)s.n_ws * H * 4 + 255) / 256 * 256;
  return s;
}
// Bytes that do for N tokens or fewer, however they are shared out: `n_ws` is at most twice the
// units wanted, of MIN_SEG tokens or more.
inline size_t linattn_workspace(int N, int H, int dk, int dv, int type) {
  if (N <= linattn_whole(LINATTN_MIN_SEG, type)) return 512;
  const int want = linattn_units_wanted(H, type), most = N / LINATTN_MIN_SEG;
  const size_t n = 2 * (size_t)(want < most ? want : most);
  const size_t states = (512 + n * H * 4 + 255) / 256 * 256;
  return (states + n * H * dk * dv * 4 + 255) / 256 * 256;
}
cudaError_t linattn_prefill_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st);
cudaError_t linattn_step_launch(const LinattnArgs& a, int type, bool pdl, cudaStream_t st);

}  // namespace moe
