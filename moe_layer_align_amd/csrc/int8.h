// Rows to 8-bit integers with one scale per row, from bf16 values or from the
// gated activation: s = max|v|/127, q = round(v/s).
//
// A row is read once: its values wait in registers for the row's largest
// magnitude.  WPR waves hold a row, CH chunks of 16 values per lane; a
// workgroup has four rows where a wave holds one.  Bound by memory (bf16: 3
// bytes a value; activation: 5 bytes and the exponential).
#pragma once

#include "swiglu.h"

namespace moe {

constexpr int kInt8Chunk = 16;
constexpr int kInt8MaxRow = 1 << 16;

// Sixteen values at v -> codes.  127 v/top to the nearest integer, ties to even:
// for bf16 values 127 v is exact, and one correction of the quotient by its
// exact remainder makes a tie, which fp32 holds, come out as one; other
// quotients lie further from a tie (2^-9 of their size) than fp32's error.
__device__ __forceinline__ u32x4 int8_codes(const float (&v)[16], float top, float r) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = 127.0f * v[4 * i + j];
      float q = x * r;
      q = __builtin_fmaf(__builtin_fmaf(-q, top, x), r, q);
      w |= ((unsigned)(int)__builtin_rintf(q) & 0xffu) << (8 * j);
    }
    o[i] = w;
  }
  return o;
}

struct Int8Args {
  const uint8_t* in;
  int64_t stride;  // elements
  int R, K;        // K: codes of a row
  const float* weight;
  const int32_t* num_rows;
  uint8_t* codes;
  float* scales;
};

template <bool GATED, int WPR, int CH>
static __global__ __launch_bounds__(WPR < 4 ? 256 : 64 * WPR) void int8_rows_kernel(Int8Args a) {
  constexpr int kRows = WPR < 4 ? 4 / WPR : 1;  // per workgroup
  __shared__ unsigned part[WPR < 4 ? 4 : WPR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = ckpt_block() * kRows + wave / WPR, at = (wave % WPR) * 64 + lane;
  const int limit = a.num_rows ? min(a.R, *a.num_rows) : a.R;
  const bool in = row < limit;
  if (limit <= 0) return;  // uniform
  // every load in flight: addresses past the row or the last row are clamped
  constexpr int kLoads = GATED ? 4 : 2;
  u32x4 raw[CH][kLoads];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = min((c * 64 * WPR + at) * kInt8Chunk, a.K - kInt8Chunk);
    const uint8_t* p = a.in + (min(row, limit - 1) * a.stride + k) * 2;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw[c][i] = *(const u32x4*)(p + 16 * (i & 1) + (i >> 1) * (2 * (int64_t)a.K));
  }
  float v[CH][16];
  unsigned top = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const bool ok = (c * 64 * WPR + at) * kInt8Chunk < a.K;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float g[8], u[8];
      unpack8(raw[c][h], g);
      if constexpr (GATED) {
        unpack8(raw[c][2 + h], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = g[i] * sigmoid_fast(g[i]) * u[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][8 * h + i] = g[i];
        top = umax(top, ok ? __float_as_uint(g[i]) & 0x7fffffffu : 0u);
      }
    }
  }
  // magnitudes compare as their bits do; NaN above all
  top = umax(top, dpp_u32<kDppXor1>(top));
  top = umax(top, dpp_u32<kDppXor2>(top));
  top = umax(top, dpp_u32<kDppHalfMirror>(top));
  top = umax(top, dpp_u32<kDppMirror>(top));
  top = umax(top, dpp_u32<kDppBcast15, 0xA>(top));
  top = umax(top, dpp_u32<kDppBcast31, 0xC>(top));
  top = (unsigned)__builtin_amdgcn_readlane((int)top, 63);
  if constexpr (WPR > 1) {
    if (lane == 0) part[wave] = top;
    __syncthreads();
    top = part[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) top = umax(top, part[w]);
  }
  if (!in) return;
  const bool finite = top < 0x7f800000u, zero = top == 0;
  const float m = __uint_as_float(top);
  if (at == 0) {
    float s = zero ? 1.0f : m / 127.0f;
    if (a.weight) s *= a.weight[row];
    a.scales[row] = finite ? s : __uint_as_float(0x7fc00000u);
  }
  // neither 1/top nor 127 v may leave fp32's normal range
  const float f = m < 0x1p-100f ? 0x1p100f : (m > 0x1p100f ? 0x1p-100f : 1.0f);
  const float scaled = zero ? 1.0f : m * f;
  const float r = __builtin_amdgcn_rcpf(scaled);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * 64 * WPR + at) * kInt8Chunk;
    if (k >= a.K) continue;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[c][i] = finite ? v[c][i] * f : 0.0f;
    *(u32x4*)(a.codes + (int64_t)row * a.K + k) = int8_codes(v[c], scaled, r);
  }
}

template <bool GATED, int WPR, int CH>
inline void launch_int8_rows(const Int8Args& a, hipStream_t st) {
  constexpr int kRows = WPR < 4 ? 4 / WPR : 1, kThreads = WPR < 4 ? 256 : 64 * WPR;
  // a dimension of the grid holds fewer than 2^32 threads
  const int blocks = (a.R + kRows - 1) / kRows, x = blocks < (1 << 30) / kThreads ? blocks : (1 << 30) / kThreads;
  int8_rows_kernel<GATED, WPR, CH><<<dim3(x, (blocks + x - 1) / x), kThreads, 0, st>>>(a);
}

// Waves per row and chunks per lane by the row's length alone.
template <bool GATED>
inline void launch_int8_rows(const Int8Args& a, hipStream_t st) {
  const int K = a.K;
  if (K <= 1024)
    launch_int8_rows<GATED, 1, 1>(a, st);
  else if (K <= 2048)
    launch_int8_rows<GATED, 1, 2>(a, st);
  else if (K <= 4096)
    launch_int8_rows<GATED, 4, 1>(a, st);
  else if (K <= 8192)
    launch_int8_rows<GATED, 4, 2>(a, st);
  else if (K <= 16384)
    launch_int8_rows<GATED, 4, 4>(a, st);
  else if (K <= 32768)
    launch_int8_rows<GATED, 16, 2>(a, st);
  else
    launch_int8_rows<GATED, 16, 4>(a, st);
}

}  // namespace moe
