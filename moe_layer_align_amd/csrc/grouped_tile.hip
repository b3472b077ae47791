// Grouped expert products with bf16 weights, and their gradients: 64 x 64
// output tiles, operands staged through LDS as [index][contraction].
#include "grouped.h"

namespace moe {
namespace {

constexpr int kT = 64, kC = 32, kLd = kC + 8;

// 8 consecutive bf16 at p + off, zeros when !ok.
__device__ __forceinline__ u32x4 load8(const uint8_t* p, int64_t off, bool ok) {
  return ok ? *(const u32x4*)(p + 2 * off) : u32x4{0, 0, 0, 0};
}

// OP 0: out[i][n] = sum_k W[n][k] in[i][k]; OP 1: out[i][k] = sum_n W[n][k]
// in[i][n]; OP 2: dw[n][k] = sum_i dy[i][n] in[i][k].
template <int OP>
__device__ __forceinline__ void tile_product(const GroupedArgs& a, const GroupedWgradArgs& b, int e, int lo, int hi,
                                             int p0, int q0, f32x4 (&acc)[2][2]) {
  __shared__ __align__(16) uint16_t P[kT * kLd], Q[kT * kLd];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int N = OP == 2 ? b.N : a.N, K = OP == 2 ? b.K : a.K;
  const int len = OP == 0 ? K : (OP == 1 ? N : hi - lo);
  const uint8_t* w = OP == 2 ? nullptr : a.w + (int64_t)e * N * K * 2;
  const int wp = (wave >> 1) * 32, wq = (wave & 1) * 32;
  for (int c0 = 0; c0 < len; c0 += kC) {
    __syncthreads();
    {  // natural operand: index tid/4, chunk tid%4 of 8 along the contraction
      const int idx = tid >> 2, c = c0 + 8 * (tid & 3);
      if (OP == 0) {
        const int n = p0 + idx;
        *(u32x4*)(P + idx * kLd + 8 * (tid & 3)) = load8(w, (int64_t)n * K + c, n < N && c < len);
      }
      if (OP != 2) {
        const int i = q0 + idx, m = i < hi ? row_of(a.in, i) : -1;
        *(u32x4*)(Q + idx * kLd + 8 * (tid & 3)) = load8(a.in.p, (int64_t)m * a.in.stride + c, m >= 0 && c < len);
      }
    }
    {  // transposed operand: contraction row tid/8, chunk tid%8 of 8 indices
      const int c = c0 + (tid >> 3), x = 8 * (tid & 7);
      uint16_t v[8];
      if (OP == 1) {
        *(u32x4*)v = load8(w, (int64_t)c * K + p0 + x, c < len && p0 + x < K);
#pragma unroll
        for (int j = 0; j < 8; ++j) P[(x + j) * kLd + (tid >> 3)] = v[j];
      }
      if (OP == 2) {
        const int md = c < len ? row_of(b.dy, lo + c) : -1, mi = c < len ? row_of(b.in, lo + c) : -1;
        *(u32x4*)v = load8(b.dy.p, (int64_t)md * b.dy.stride + p0 + x, md >= 0 && mi >= 0 && p0 + x < N);
#pragma unroll
        for (int j = 0; j < 8; ++j) P[(x + j) * kLd + (tid >> 3)] = v[j];
        *(u32x4*)v = load8(b.in.p, (int64_t)mi * b.in.stride + q0 + x, md >= 0 && mi >= 0 && q0 + x < K);
#pragma unroll
        for (int j = 0; j < 8; ++j) Q[(x + j) * kLd + (tid >> 3)] = v[j];
      }
    }
    __syncthreads();
    u32x4 fp[2], fq[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fp[i] = *(const u32x4*)(P + (wp + 16 * i + (lane & 15)) * kLd + 8 * (lane >> 4));
      fq[i] = *(const u32x4*)(Q + (wq + 16 * i + (lane & 15)) * kLd + 8 * (lane >> 4));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16(fp[i], fq[j], acc[i][j]);
  }
}

template <int OP, bool F32>
__global__ __launch_bounds__(256) void grouped_tile_kernel(GroupedArgs a) {
  // row tile blockIdx.x -> expert
  int e = 0, lo = 0, hi = 0, q0 = -1, before = 0;
  for (e = 0; e < a.E; ++e) {
    group_range(a.offsets, e, a.R, &lo, &hi);
    const int nt = (hi - lo + kT - 1) / kT;
    if ((int)blockIdx.x < before + nt) {
      q0 = lo + ((int)blockIdx.x - before) * kT;
      break;
    }
    before += nt;
  }
  if (q0 < 0) return;
  f32x4 acc[2][2] = {};
  const int p0 = blockIdx.y * kT;
  tile_product<OP>(a, GroupedWgradArgs{}, e, lo, hi, p0, q0, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int width = OP == 0 ? a.N : a.K;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = q0 + (wave & 1) * 32 + 16 * j + (lane & 15);
    const int m = i < hi ? row_of(a.out, i) : -1;
    if (m < 0) continue;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int p = p0 + (wave >> 1) * 32 + 16 * t + 4 * (lane >> 4);
      if (p >= width) continue;
      const f32x4 c = acc[t][j];
      if (F32)
        *(f32x4*)(a.out.p + ((int64_t)m * a.out.stride + p) * 4) = c;
      else
        *(u32x2*)(a.out.p + ((int64_t)m * a.out.stride + p) * 2) = u32x2{pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3])};
    }
  }
}

template <bool F32, bool ACC>
__global__ __launch_bounds__(256) void grouped_wgrad_kernel(GroupedWgradArgs b) {
  const int e = blockIdx.z, p0 = blockIdx.y * kT, q0 = blockIdx.x * kT;
  int lo, hi;
  group_range(b.offsets, e, b.R, &lo, &hi);
  if (ACC && lo == hi) return;
  f32x4 acc[2][2] = {};
  tile_product<2>(GroupedArgs{}, b, e, lo, hi, p0, q0, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int k = q0 + (wave & 1) * 32 + 16 * j + (lane & 15);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int n = p0 + (wave >> 1) * 32 + 16 * t + 4 * (lane >> 4) + v;
        if (n >= b.N || k >= b.K) continue;
        const int64_t at = ((int64_t)e * b.N + n) * b.K + k;
        if (F32)
          ((float*)b.dw)[at] = acc[t][j][v] + (ACC ? ((float*)b.dw)[at] : 0.0f);
        else
          ((uint16_t*)b.dw)[at] = (uint16_t)pack_bf16x2(acc[t][j][v], 0.0f);
      }
  }
}

}  // namespace

bool launch_grouped_tile(bool dgrad, bool f32, hipStream_t st, const GroupedArgs& a) {
  const int width = dgrad ? a.K : a.N;
  const dim3 g(a.R / kT + (a.R < a.E ? a.R : a.E), (width + kT - 1) / kT);
  if (dgrad)
    f32 ? grouped_tile_kernel<1, true><<<g, 256, 0, st>>>(a) : grouped_tile_kernel<1, false><<<g, 256, 0, st>>>(a);
  else
    f32 ? grouped_tile_kernel<0, true><<<g, 256, 0, st>>>(a) : grouped_tile_kernel<0, false><<<g, 256, 0, st>>>(a);
  return true;
}

bool launch_grouped_wgrad(bool f32, bool accumulate, hipStream_t st, const GroupedWgradArgs& a) {
  const dim3 g((a.K + kT - 1) / kT, (a.N + kT - 1) / kT, a.E);
  if (f32 && accumulate)
    grouped_wgrad_kernel<true, true><<<g, 256, 0, st>>>(a);
  else if (f32)
    grouped_wgrad_kernel<true, false><<<g, 256, 0, st>>>(a);
  else
    grouped_wgrad_kernel<false, false><<<g, 256, 0, st>>>(a);
  return true;
}

}  // namespace moe
