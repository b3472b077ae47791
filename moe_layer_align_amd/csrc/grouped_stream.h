// What the streamed expert products share (a few rows per expert): buffer
// loads, the reads of a wave's LDS stage and the search for a workgroup's expert.
#pragma once

#include "grouped.h"
#include "mfma_tile.h"

namespace moe {
namespace {

constexpr unsigned kOob = 0xffc00000u;  // lane offset past every buffer
// a wave's weights of one step: 128 bytes of each of `ft` tiles of 16 weight rows
__host__ __device__ constexpr int stage_bytes(int ft) { return ft * 16 * 128; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, kBufferWord3);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, unsigned off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// A wave's fragments of a stage, from two addresses on (i = 0, 1).  Ahead of a
// read that it knows of, the compiler waits for all loads into LDS, those of the
// other stage too.
template <int FT>
__device__ __forceinline__ void read_stage(u32x4 (&w)[FT][2], unsigned a0, unsigned a1) {
  static_assert(FT == 2 || FT == 4, "tiles of a wave");
  if constexpr (FT == 4)
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
        "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
        "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
        "ds_read_b128 %6, %8 offset:6144\n\tds_read_b128 %7, %9 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(w[0][0]), "=&v"(w[0][1]), "=&v"(w[1][0]), "=&v"(w[1][1]), "=&v"(w[2][0]), "=&v"(w[2][1]),
          "=&v"(w[3][0]), "=&v"(w[3][1])
        : "v"(a0), "v"(a1)
        : "memory");
  else
    asm volatile(
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
        "ds_read_b128 %2, %4 offset:2048\n\tds_read_b128 %3, %5 offset:2048\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(w[0][0]), "=&v"(w[0][1]), "=&v"(w[1][0]), "=&v"(w[1][1])
        : "v"(a0), "v"(a1)
        : "memory");
}

// A workgroup's expert: blockIdx.y itself, or, with fewer rows than experts,
// the blockIdx.y-th that holds rows (e = E: none).  Thread i looks at experts i
// and i + 256.
struct Found {
  int e, lo, hi;
};
__device__ __forceinline__ Found find_expert(const int32_t* offsets, int R, int E) {
  __shared__ unsigned long long mask[kMaxExperts / 64];
  __shared__ int range[3];
  Found f = {(int)blockIdx.y, 0, 0};
  if (R >= E) {
    group_range(offsets, f.e, R, &f.lo, &f.hi);
  } else {
    const int tid = threadIdx.x, lane = tid & 63;
    int lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (tid + 256 * h < E) group_range(offsets, tid + 256 * h, R, &lo[h], &hi[h]);
      const unsigned long long m = __ballot(lo[h] < hi[h]);
      if (lane == 0) mask[4 * h + (tid >> 6)] = m;
    }
    if (tid == 0) range[0] = E;
    __syncthreads();
    int before[2] = {0, 0};  // experts with rows ahead of the thread's two
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const int n = __popcll(mask[w]);
      before[0] += w < (tid >> 6) ? n : 0;
      before[1] += w < 4 + (tid >> 6) ? n : 0;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (lo[h] < hi[h] &&
          before[h] + __popcll(mask[4 * h + (tid >> 6)] & lanemask_lt(lane)) == (int)blockIdx.y) {
        range[0] = tid + 256 * h;
        range[1] = lo[h];
        range[2] = hi[h];
      }
    __syncthreads();
    f = Found{range[0], range[1], range[2]};
  }
  return Found{__builtin_amdgcn_readfirstlane(f.e), __builtin_amdgcn_readfirstlane(f.lo),
               __builtin_amdgcn_readfirstlane(f.hi)};
}

}  // namespace
}  // namespace moe
