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
  int b;      // sequence, or -1: the call has no such unit
  int i, n;   // unit i of n
  int seg;    // tokens of a unit
  int slot0;  // workspace state of the sequence's unit 0 (sequences of several units)
  bool found;
};
constexpr int UNIT_SCRATCH = 4 + 3 * 8;  // ints of shared memory that find_unit takes (8 warps)
// Unit u of the call: u < B are the last (or only) units of the sequences, u >= B counts the
// others, each of seg tokens, in sequence order. Of up to 256 sequences the last units of more
// than half of seg come first (`by_rank`), so that a grid in this order ends with its shortest
// pieces. A whole CTA (256 threads of it) settles whether the call stays whole, where that is
// open, and adds up what the sequences before u's have. `n_ws`: states in the workspace. Offsets that
// go back and rise again make sequences share tokens and have more units than the call's tokens: a
// sequence whose states do not fit, or whose units are not all launched, is not found (b stays).
__device__ __forceinline__ Unit find_unit(const LinattnArgs& a, LinattnCut cut, int n_ws, int u, int* scratch,
                                          bool by_rank = true) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool ranked = by_rank && a.B <= 256;
  int seg = cut.seg, begin_u = 0, end_u = 0;
  const bool own = u < a.B && (a.B == 1 || !ranked);  // the last unit of sequence u
  if (own) {
    seq_range(a, u, begin_u, end_u);
    // whole by its own length: nothing of the other sequences matters, however many there are
    if (end_u - begin_u <= seg) return Unit{u, 0, 1, seg, 0, true};
  }
  int first = 0, past = 0;  // of sequence tid
  if (tid < min(256, a.B)) seq_range(a, tid, first, past);
  if (cut.ask) {
    int longest = past - first;
    for (int b = 256 + tid; tid < 256 && b < a.B; b += 256) {
      int begin, end;
      seq_range(a, b, begin, end);
      longest = max(longest, end - begin);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0 && warp < 8) scratch[4 + warp] = longest;
    __syncthreads();
    for (int w = 0; w < 8; ++w) longest = max(longest, scratch[4 + w]);
    if (longest <= cut.whole) seg = cut.whole;
  }
  Unit r{0, 0, 1, seg, 0, true};
  if (own) {
    r.b = u;
    r.n = seq_units(end_u - begin_u, seg);
    r.i = r.n - 1;
    if (r.n == 1) return r;
  }
  int base_u = 0, base_s = 0;
  if (tid == 0) scratch[0] = -1;
  for (int b0 = 0; b0 < a.B; b0 += 256) {
    const int b = tid < 256 ? b0 + tid : a.B;
    int ns = 0, tail = 0;
    if (b < a.B) {
      int begin = first, end = past;
      if (b0 > 0) seq_range(a, b, begin, end);
      ns = seq_units(end - begin, seg);
      tail = end - begin - (ns - 1) * seg;
    }
    const int nu = max(ns - 1, 0);                // units but the last
    const int nl = tail > seg / 2;                // whether the last one is long
    if (ns == 1) ns = 0;                          // states
    int cu = nu, cs = ns, cl = nl;                // inclusive sums over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, cu, o), y = __shfl_up_sync(0xffffffffu, cs, o);
      const int z = __shfl_up_sync(0xffffffffu, cl, o);
      if (lane >= o) {
        cu += x;
        cs += y;
        cl += z;
      }
    }
    __syncthreads();  // the last round's sums have been read
    if (lane == 31 && warp < 8) {
      scratch[4 + 3 * warp] = cu;
      scratch[5 + 3 * warp] = cs;
      scratch[6 + 3 * warp] = cl;
    }
    __syncthreads();
    int pu = base_u + cu - nu, ps = base_s + cs - ns, pl = cl - nl, longs = 0;
    for (int w = 0; w < 8; ++w) {
      const int x = scratch[4 + 3 * w], y = scratch[5 + 3 * w], z = scratch[6 + 3 * w];
      if (w < warp) {
        pu += x;
        ps += y;
        pl += z;
      }
      base_u += x;
      base_s += y;
      longs += z;
    }
    const int rank = !ranked ? b : nl ? pl : longs + b - pl;
    if (b < a.B && (u < a.B ? rank == u : u - a.B >= pu && u - a.B < pu + nu)) {
      scratch[0] = b;
      scratch[1] = u < a.B ? nu : u - a.B - pu;
      scratch[2] = nu + 1;
      scratch[3] = ps + nu + 1 <= n_ws && pu + nu <= cut.rest ? ps : -1;
    }
    if (u < a.B ? u < b0 + 256 : u - a.B < base_u) break;
  }
  __syncthreads();
  r.b = scratch[0];
  r.i = scratch[1];
  r.n = scratch[2];
  r.slot0 = scratch[3];
  r.found = r.b >= 0 && (r.n == 1 || r.slot0 >= 0);
  __syncthreads();  // scratch may be reused
  return r;
}

// Prompts by chunks on the tensor cores (linattn_tc.cu).
cudaError_t linattn_chunk_launch(const LinattnArgs& a, int type, void* ws, bool pdl, cudaStream_t st);

}  // namespace moe
