// Grouped expert products with 4-bit weights: one wave per (weight row,
// grouped row), fp32 multiply-adds.
#include "grouped.h"

namespace moe {
namespace {

__device__ __forceinline__ float e2m1(unsigned q) {
  const int ex = (q >> 1) & 3, m = q & 1;
  const float v = ex ? (float)(2 + m) * (float)(1 << ex) * 0.25f : 0.5f * m;
  return (q & 8) ? -v : v;
}

template <int FMT, bool F32>
__global__ __launch_bounds__(256) void grouped_stream_kernel(GroupedArgs a) {
  const int lane = threadIdx.x & 63, n = blockIdx.y * 4 + (threadIdx.x >> 6), i = blockIdx.x;
  int e = 0, lo = 0, hi = 0;
  for (e = 0; e < a.E; ++e) {
    group_range(a.offsets, e, a.R, &lo, &hi);
    if (i >= lo && i < hi) break;
  }
  if (e == a.E || n >= a.N) return;
  const int m = row_of(a.in, i), mo = row_of(a.out, i);
  if (mo < 0) return;
  const uint8_t* w = a.w + ((int64_t)e * a.N + n) * (a.K / 2);
  const uint16_t* x = (const uint16_t*)a.in.p + (int64_t)max(m, 0) * a.in.stride;
  float sum = 0.0f;
  for (int k = 2 * lane; k < a.K; k += 128) {
    const unsigned c = w[k / 2];
    float w0, w1, s;
    if (FMT == 1) {
      w0 = e2m1(c & 15);
      w1 = e2m1(c >> 4);
      s = __uint_as_float((unsigned)a.w_scale[((int64_t)e * a.N + n) * (a.K / 32) + k / 32] << 23);
    } else {
      w0 = (float)(int)(c & 15) - 8.0f;
      w1 = (float)(int)(c >> 4) - 8.0f;
      s = bf16_lo(((const uint16_t*)a.w_scale)[((int64_t)e * a.N + n) * (a.K / 128) + k / 128]);
    }
    if (m >= 0) sum += s * (w0 * bf16_lo(x[k]) + w1 * bf16_lo(x[k + 1]));
  }
  sum = wave_sum(sum);
  if (lane == 0) {
    const int64_t at = (int64_t)mo * a.out.stride + n;
    if (F32)
      ((float*)a.out.p)[at] = sum;
    else
      ((uint16_t*)a.out.p)[at] = (uint16_t)pack_bf16x2(sum, 0.0f);
  }
}

}  // namespace

bool launch_grouped_stream(int format, bool f32, hipStream_t st, const GroupedArgs& a) {
  const dim3 g(a.R, (a.N + 3) / 4);
  if (format == 1)
    f32 ? grouped_stream_kernel<1, true><<<g, 256, 0, st>>>(a) : grouped_stream_kernel<1, false><<<g, 256, 0, st>>>(a);
  else
    f32 ? grouped_stream_kernel<2, true><<<g, 256, 0, st>>>(a) : grouped_stream_kernel<2, false><<<g, 256, 0, st>>>(a);
  return true;
}

}  // namespace moe
