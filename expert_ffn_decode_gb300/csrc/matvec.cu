// Matrix-vector products with 4-bit weights and group scales: y_t = W x_t (+ bias) (+ y_t).
//
// A row's block of 32 values with scale d and offset m contributes
//   d * sum_i q_i x_i + m * sum_i x_i
// (Q4_0 and planes without offsets: m = -8 d; Q4_K: d and m are the sub-block's d sc and
// -dmin mn), so a nibble is used as the integer it is and never rounded.
#include "common.cuh"
#include "ops_host.h"
#include "types.cuh"

namespace moe {
namespace {

// One warp a row, a lane every 32nd block.
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) matvec_kernel(MatvecArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int nb = a.cols / 32;
  if (row >= a.rows) return;
  for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
    const TX* x = static_cast<const TX*>(a.x) + t * a.xs;
    float acc = 0.f;
    for (int b = lane; b < nb; b += 32) {
      const uint8_t* nib;
      int nib_shift = -1;  // Q4_K: a sub-block is one nibble of 32 bytes
      float d, m;
      if (a.qtype == MOE_Q4_K) {
        const uint8_t* s = a.w + (row * (nb / 8) + b / 8) * 144;
        const int j = b % 8;
        const uint8_t* p = s + 4;
        const int sc = j < 4 ? p[j] & 63 : (p[j + 4] & 15) | (p[j - 4] >> 6) << 4;
        const int mn = j < 4 ? p[j + 4] & 63 : (p[j + 4] >> 4) | (p[j] >> 6) << 4;
        d = __half2float(*reinterpret_cast<const __half*>(s)) * sc;
        m = -__half2float(*reinterpret_cast<const __half*>(s + 2)) * mn;
        nib = s + 16 + j / 2 * 32;
        nib_shift = j % 2 * 4;
      } else if (a.qtype == MOE_Q4_PLANES) {
        nib = a.w + (row * nb + b) * 16;
        const int64_t g = row * (a.cols / a.group) + b * 32 / a.group;
        d = __half2float(reinterpret_cast<const __half*>(a.scales)[g]);
        m = a.mins ? __half2float(reinterpret_cast<const __half*>(a.mins)[g]) : -8.f * d;
      } else {
        const bool q1 = a.qtype == MOE_Q4_1;
        const uint8_t* s = a.w + (row * nb + b) * (q1 ? 20 : 18);
        d = __half2float(*reinterpret_cast<const __half*>(s));
        m = q1 ? __half2float(*reinterpret_cast<const __half*>(s + 2)) : -8.f * d;
        nib = s + (q1 ? 4 : 2);
      }
      float s = 0.f, sx = 0.f;
      for (int i = 0; i < 32; ++i) {
        const float xv = to_f32(x[b * 32 + i]);
        const int q = nib_shift >= 0 ? nib[i] >> nib_shift & 15 : nib[i % 16] >> i / 16 * 4 & 15;
        s = fmaf((float)q, xv, s);
        sx += xv;
      }
      acc = fmaf(d, s, acc);
      acc = fmaf(m, sx, acc);
    }
    acc = warp_sum(acc);
    if (lane == 0) {
      if (a.bias) acc += a.bias[row];
      TY* y = static_cast<TY*>(a.y) + t * a.ys + row;
      if (a.flags & MOE_ACCUMULATE) acc += to_f32(*y);
      *y = from_f32<TY>(acc);
    }
  }
}

template <typename TX>
cudaError_t launch_y(const MatvecArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.rows + 7) / 8), (unsigned)(a.T < 64 ? a.T : 64));
  if (a.y_type == MOE_F32) matvec_kernel<TX, float><<<grid, 256, 0, st>>>(a);
  else if (a.y_type == MOE_F16) matvec_kernel<TX, __half><<<grid, 256, 0, st>>>(a);
  else matvec_kernel<TX, __nv_bfloat16><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t matvec_launch(const MatvecArgs& a, cudaStream_t st) {
  if (a.x_type == MOE_F32) return launch_y<float>(a, st);
  if (a.x_type == MOE_F16) return launch_y<__half>(a, st);
  return launch_y<__nv_bfloat16>(a, st);
}

}  // namespace moe
