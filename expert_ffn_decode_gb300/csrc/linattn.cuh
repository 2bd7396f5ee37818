// What the linear attention kernels share: the bounds and the state of a sequence, and the
// split of long sequences into units of `seg` tokens.
#pragma once

#include "common.cuh"
#include "ops_host.h"
#include "types.cuh"

namespace moe {

// Tokens begin .. end - 1 of sequence b (clamped to the call's tokens; descending: empty).
__device__ __forceinline__ void seq_range(const LinattnArgs& a, int b, int& begin, int& end) {
  if (a.offsets) {
    begin = min(max(a.offsets[b], 0), a.N);
    end = max(min(max(a.offsets[b + 1], 0), a.N), begin);
  } else {
    begin = b * a.seq_len;
    end = begin + a.seq_len;
  }
}
// The state of sequence b, or -1 when the sequence is inactive.
__device__ __forceinline__ int seq_slot(const LinattnArgs& a, int b) {
  const int s = a.slots ? a.slots[b] : b;
  return s >= 0 && s < a.n_states ? s : -1;
}
// Units of a sequence of n tokens: an empty one has one too (its state may start fresh).
__host__ __device__ __forceinline__ int seq_units(int n, int seg) { return n > seg ? (n + seg - 1) / seg : 1; }

struct Unit {
  int b;      // sequence
  int i, n;   // unit i of n
  int slot0;  // workspace state of the sequence's unit 0 (sequences of several units)
  bool found;
};
// Unit u of the call, in sequence order: a whole CTA adds up the units of the sequences
// before it. `n_ws`: states in the workspace; a sequence whose units would not fit (offsets
// that descend can make sequences share tokens) is not found. `scratch`: 4 + 2 * (threads / 32)
// ints of shared memory.
__device__ __forceinline__ Unit find_unit(const LinattnArgs& a, int seg, int n_ws, int u, int* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  int base_u = 0, base_s = 0;
  if (tid == 0) scratch[0] = -1;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + tid;
    int nu = 0;
    if (b < a.B) {
      int begin, end;
      seq_range(a, b, begin, end);
      nu = seq_units(end - begin, seg);
    }
    const int ns = nu > 1 ? nu : 0;
    int cu = nu, cs = ns;  // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, cu, o), y = __shfl_up_sync(0xffffffffu, cs, o);
      if (lane >= o) {
        cu += x;
        cs += y;
      }
    }
    __syncthreads();  // the last round's sums have been read
    if (lane == 31) {
      scratch[4 + 2 * warp] = cu;
      scratch[5 + 2 * warp] = cs;
    }
    __syncthreads();
    int pu = base_u, ps = base_s;
    for (int w = 0; w < nw; ++w) {
      const int x = scratch[4 + 2 * w], y = scratch[5 + 2 * w];
      if (w < warp) {
        pu += x;
        ps += y;
      }
      base_u += x;
      base_s += y;
    }
    pu += cu - nu;
    ps += cs - ns;
    if (u >= pu && u < pu + nu) {
      scratch[0] = b;
      scratch[1] = u - pu;
      scratch[2] = nu;
      scratch[3] = ps;
    }
    if (u < base_u) break;
  }
  __syncthreads();
  Unit r;
  r.b = scratch[0];
  r.i = scratch[1];
  r.n = scratch[2];
  r.slot0 = scratch[3];
  r.found = r.b >= 0 && (r.n == 1 || r.slot0 + r.n <= n_ws);
  __syncthreads();  // scratch may be reused
  return r;
}

// Prompts by chunks on the tensor cores (linattn_tc.cu).
cudaError_t linattn_chunk_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st);

}  // namespace moe
