// The gated activation with its inputs kept in 8 bits, and its gradient from
// them: h = w SiLU(g) u, with (g, u) as e4m3 codes under one power-of-two
// scale per 32 consecutive values.
//
// Both are bound by memory (a few tens of operations per 8 to 13 bytes).  A
// thread holds 8 gate values and the 8 up values of the same columns, so every
// access is 16 bytes (codes: 8) and the four lanes of a quad hold one scale
// group, whose largest magnitude two DPP quad permutations find.
//
// The scale is the smallest power of two under which the group's largest
// magnitude does not pass 448: unlike the layer's block scaling (exponent - 8,
// which clips mantissas above 1.75), no value is ever clipped, so each is
// within half a step, 2^-4 of its own size, of the value it stands for (down
// to the format's subnormals, 2^-15 of the group's largest).
#pragma once

#include "grouped.h"

namespace moe {

constexpr int kCkptGroup = 32;  // values per scale
constexpr int kCkptPer = 8;     // values per thread and half
constexpr int kCkptQuad = kCkptGroup / kCkptPer;

// Biased exponent of the scale for a largest finite magnitude with bits
// `amax`: exponent - 8, one more where the mantissa is above 1.75 (448 = 1.75
// * 2^8), at least 0.
__device__ __forceinline__ int ckpt_scale_code(unsigned amax) {
  const int c = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(c, 0);
}
// 2^(127 - code) and 2^(code - 127); code 0 stands for 2^-127, a subnormal.
__device__ __forceinline__ float pow2_recip(int code) { return __uint_as_float((unsigned)(254 - code) << 23); }
__device__ __forceinline__ float pow2_of(int code) {
  return __uint_as_float(code ? (unsigned)code << 23 : 0x400000u);
}

__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

// e4m3 codes of a thread's 8 values under the scale its quad shares; all
// lanes active.
__device__ __forceinline__ u32x2 encode8(const float (&v)[8], int* code) {
  unsigned m = 0, top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned b = __float_as_uint(v[i]) & 0x7fffffffu;
    top = umax(top, b);
    m = umax(m, b < 0x7f800000u ? b : 0u);
  }
  m = umax(m, dpp_u32<kDppXor1>(m));
  m = umax(m, dpp_u32<kDppXor2>(m));
  *code = ckpt_scale_code(m);
  const float r = pow2_recip(*code);
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * r, v[4 * i + 1] * r, 0, false);
    o[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * r, v[4 * i + 3] * r, w, true);
  }
  if (top >= 0x7f800000u) {  // NaN and infinities: the NaN code (the conversion's own is 0xff)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((__float_as_uint(v[i]) & 0x7fffffffu) >= 0x7f800000u)
        o[i >> 2] = (o[i >> 2] & ~(0xffu << 8 * (i & 3))) | 0x7fu << 8 * (i & 3);
  }
  return o;
}

__device__ __forceinline__ void decode8(u32x2 c, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    v[4 * i] = a[0] * s;
    v[4 * i + 1] = a[1] * s;
    v[4 * i + 2] = b[0] * s;
    v[4 * i + 3] = b[1] * s;
  }
}

__device__ __forceinline__ void unpack8(u32x4 w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// 1/(1+exp(-x)) with the hardware's exp2 and reciprocal, about an ulp each in
// fp32, against the 2^-9 of the results' rounding.
__device__ __forceinline__ float sigmoid_fast(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * 1.4426950408889634f));
}

// A launch's workgroups, in two rows of the grid where one would have 2^32
// threads, which a grid's dimension cannot hold.
inline dim3 ckpt_grid(int64_t blocks) {
  const unsigned y = blocks >> 23 ? 2 : 1;
  return dim3((unsigned)((blocks + y - 1) / y), y);
}
__device__ __forceinline__ int ckpt_block() { return (int)(blockIdx.x + blockIdx.y * gridDim.x); }

// Threads run over (row, chunk of 8 columns), the chunks of a row padded to
// whole quads.
static __global__ __launch_bounds__(256) void swiglu_checkpoint_kernel(const uint8_t* __restrict__ gu, int64_t stride,
                                                                const float* __restrict__ weight, int R, int I,
                                                                const int32_t* __restrict__ num_rows,
                                                                uint8_t* __restrict__ h, uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  const int groups = (I + kCkptGroup - 1) / kCkptGroup, per_row = groups * kCkptQuad;
  const int64_t base = (int64_t)ckpt_block() * 256;
  const int row0 = (int)(base / per_row);
  const unsigned local = (unsigned)(base - (int64_t)row0 * per_row) + threadIdx.x;
  const int row = row0 + (int)(local / (unsigned)per_row), chunk = (int)(local % (unsigned)per_row);
  const int limit = num_rows ? min(R, *num_rows) : R;
  const bool in_row = row < limit, ok = in_row && chunk * kCkptPer < I;
  float g[8] = {}, u[8] = {};
  if (ok) {
    const uint8_t* p = gu + ((int64_t)row * stride + chunk * kCkptPer) * 2;
    unpack8(*(const u32x4*)p, g);
    unpack8(*(const u32x4*)(p + 2 * (int64_t)I), u);
  }
  if (h && ok) {
    const float w = weight ? weight[row] : 1.0f;
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = g[i] * sigmoid_fast(g[i]) * u[i] * w;
    *(u32x4*)(h + ((int64_t)row * I + chunk * kCkptPer) * 2) = pack8(o);
  }
  if (!codes) return;
  int cg, cu;
  const u32x2 qg = encode8(g, &cg), qu = encode8(u, &cu);
  if (ok) {
    uint8_t* c = codes + (int64_t)row * 2 * I + chunk * kCkptPer;
    *(u32x2*)c = qg;
    *(u32x2*)(c + I) = qu;
  }
  if (in_row && chunk % kCkptQuad == 0) {
    uint8_t* s = scales + (int64_t)row * 2 * groups + chunk / kCkptQuad;
    s[0] = (uint8_t)cg;
    s[groups] = (uint8_t)cu;
  }
}

// WPR waves work on one row (so that its dweight is one sum in a fixed order),
// 512 columns per wave and step.
template <int WPR>
__global__ __launch_bounds__(WPR < 4 ? 256 : 64 * WPR) void swiglu_grad_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const uint8_t* __restrict__ dh,
    const float* __restrict__ weight, int R, int I, const int32_t* __restrict__ num_rows, uint8_t* __restrict__ dgu,
    uint8_t* __restrict__ h, float* __restrict__ dweight) {
  constexpr int kRows = WPR < 4 ? 4 / WPR : 1;  // rows per workgroup
  __shared__ float part[WPR * kRows];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row0 = ckpt_block() * kRows, row = row0 + wave / WPR, wr = wave % WPR;
  const int groups = (I + kCkptGroup - 1) / kCkptGroup;
  const int limit = num_rows ? min(R, *num_rows) : R;
  float sum = 0.0f;
  if (row < limit) {
    const float w = weight ? weight[row] : 1.0f;
    const uint8_t* c = codes + (int64_t)row * 2 * I;
    const uint8_t* s = scales + (int64_t)row * 2 * groups;
    const uint8_t* d = dh + (int64_t)row * I * 2;
    uint8_t* o = dgu + (int64_t)row * I * 4;
    for (int col = (wr * 64 + lane) * kCkptPer; col < I; col += WPR * 64 * kCkptPer) {
      float g[8], u[8], dv[8], og[8], ou[8], oh[8];
      decode8(*(const u32x2*)(c + col), pow2_of(s[col / kCkptGroup]), g);
      decode8(*(const u32x2*)(c + I + col), pow2_of(s[groups + col / kCkptGroup]), u);
      unpack8(*(const u32x4*)(d + 2 * (int64_t)col), dv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sg = sigmoid_fast(g[i]), silu = g[i] * sg, hv = silu * u[i], wd = w * dv[i];
        sum += dv[i] * hv;
        oh[i] = w * hv;
        ou[i] = wd * silu;
        og[i] = wd * u[i] * (sg * (1.0f + g[i] * (1.0f - sg)));
      }
      *(u32x4*)(o + 2 * (int64_t)col) = pack8(og);
      *(u32x4*)(o + 2 * ((int64_t)I + col)) = pack8(ou);
      if (h) *(u32x4*)(h + ((int64_t)row * I + col) * 2) = pack8(oh);
    }
  }
  if (!dweight) return;
  sum = wave_sum(sum);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  if (threadIdx.x < kRows && row0 + (int)threadIdx.x < limit) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) t += part[threadIdx.x * WPR + i];
    dweight[row0 + threadIdx.x] = t;
  }
}

inline void launch_swiglu_checkpoint(const uint8_t* gu, int64_t stride, const float* w, int R, int I,
                                     const int32_t* num_rows, uint8_t* h, uint8_t* codes, uint8_t* scales,
                                     hipStream_t st) {
  const int64_t threads = (int64_t)R * ((I + kCkptGroup - 1) / kCkptGroup) * kCkptQuad;
  swiglu_checkpoint_kernel<<<ckpt_grid((threads + 255) / 256), 256, 0, st>>>(gu, stride, w, R, I, num_rows, h, codes,
                                                                             scales);
}

inline void launch_swiglu_grad(const uint8_t* codes, const uint8_t* scales, const uint8_t* dh, const float* w, int R,
                               int I, const int32_t* num_rows, uint8_t* dgu, uint8_t* h, float* dweight,
                               hipStream_t st) {
  if (I <= 2048)
    swiglu_grad_kernel<1><<<ckpt_grid((R + 3) / 4), 256, 0, st>>>(codes, scales, dh, w, R, I, num_rows, dgu, h,
                                                                  dweight);
  else
    swiglu_grad_kernel<4><<<ckpt_grid(R), 256, 0, st>>>(codes, scales, dh, w, R, I, num_rows, dgu, h, dweight);
}

}  // namespace moe
