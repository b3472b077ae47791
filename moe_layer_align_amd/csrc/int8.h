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

// Largest value of a wave.  Magnitudes compare as their bits do, NaN above all.
__device__ __forceinline__ unsigned wave_umax(unsigned v) {
  v = umax(v, dpp_u32<kDppXor1>(v));
  v = umax(v, dpp_u32<kDppXor2>(v));
  v = umax(v, dpp_u32<kDppHalfMirror>(v));
  v = umax(v, dpp_u32<kDppMirror>(v));
  v = umax(v, dpp_u32<kDppBcast15, 0xA>(v));
  v = umax(v, dpp_u32<kDppBcast31, 0xC>(v));
  return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
}

// A row's scale, and what its codes are formed with, from its largest magnitude
// (fp32 bits, infinity or NaN where the row holds one).  f keeps 1/top and 127 v
// inside fp32's normal range.
struct RowScale {
  float s, f127, top, r;  // scale; 127 f; f top; its reciprocal
};
__device__ __forceinline__ RowScale row_scale(unsigned bits) {
  const float m = __uint_as_float(bits);
  const float f = m < 0x1p-100f ? 0x1p100f : (m > 0x1p100f ? 0x1p-100f : 1.0f);
  RowScale o;
  o.s = bits == 0 ? 1.0f : (bits < 0x7f800000u ? m / 127.0f : __uint_as_float(0x7fc00000u));
  o.top = bits == 0 ? 1.0f : m * f;
  o.r = __builtin_amdgcn_rcpf(o.top);
  o.f127 = 127.0f * f;
  return o;
}

// Sixteen values at v -> codes.  127 v/top to the nearest integer, ties to even:
// for bf16 values 127 v is exact, and one correction of the quotient by its
// exact remainder makes a tie, which fp32 holds, come out as one; the quotient of
// mantissas b and a (128 to 255), 127 b/(a 2^e), lies otherwise at least 1/(254 b)
// of its size from a tie, 2^-16, further than fp32's error of 2^-23.  The gated
// activation's values are fp32: their 127 v is rounded, and a value within that
// rounding of a tie may take either code.
// Adding 1.5 * 2^23 rounds to an integer and leaves its low byte in front.
__device__ __forceinline__ u32x4 int8_codes(const float (&v)[16], const RowScale& s) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unsigned b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = s.f127 * v[4 * i + j];
      const float q = x * s.r;
      b[j] = __float_as_uint(__builtin_fmaf(__builtin_fmaf(-q, s.top, x), s.r, q) + 0x1.8p23f);
    }
    // byte 0 of each
    o[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
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
  top = wave_umax(top);
  if constexpr (WPR > 1) {
    if (lane == 0) part[wave] = top;
    __syncthreads();
    top = part[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) top = umax(top, part[w]);
  }
  if (!in) return;
  const RowScale rs = row_scale(top);
  if (at == 0) a.scales[row] = a.weight ? rs.s * a.weight[row] : rs.s;
  const bool finite = top < 0x7f800000u;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * 64 * WPR + at) * kInt8Chunk;
    if (k < a.K) *(u32x4*)(a.codes + (int64_t)row * a.K + k) = finite ? int8_codes(v[c], rs) : u32x4{0, 0, 0, 0};
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
