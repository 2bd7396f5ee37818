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
cudaError_t linattn_prefill_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st);
cudaError_t linattn_step_launch(const LinattnArgs& a, int type, bool pdl, cudaStream_t st);

}  // namespace moe
