// What the LDS-tiled products share: the 32x32 MFMAs, direct-to-LDS load waits,
// the workgroup barrier of an LDS ring and its chunk swizzle.
#pragma once

#include "moe_device.h"

namespace moe {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

// 32x32x64 OCP e4m3 x e4m3 -> fp32, unit block scales.  A: lane l holds 32
// bytes of row l%32; B: 32 bytes of column l%32, at the same k positions.
// C: lane l holds column l%32, rows 8*(v/4) + 4*(l/32) + v%4, v = 0..15.
__device__ __forceinline__ f32x16 mfma32_fp8(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x16 c) {
  i32x8 a = __builtin_bit_cast(i32x8, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7));
  i32x8 b = __builtin_bit_cast(i32x8, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
}

// 32x32x16 bf16 -> fp32.  A: lane l holds 8 bf16 (16 bytes) of row l%32 at
// k = 8*(l/32); B: the same k of column l%32.  C as for mfma32_fp8.
__device__ __forceinline__ f32x16 mfma32_bf16(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}

// Wait until at most N vector-memory operations of this wave are
// outstanding (the LDS-DMA loads below are vector-memory operations whose
// destination the compiler does not track).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  // vmcnt[3:0] | expcnt 7 [6:4] | lgkmcnt 15 [11:8] | vmcnt[5:4] at [15:14]
  __builtin_amdgcn_s_waitcnt((N & 0xf) | (0x7 << 4) | (0xf << 8) | ((N >> 4) << 14));
}

// Workgroup barrier for the LDS ring: waits for this wave's own LDS reads
// only (lgkmcnt 0), not for its outstanding global-to-LDS loads, whose
// completion the K-loop waits for explicitly; the memory clobber keeps the
// compiler from moving LDS accesses across it.  (__syncthreads() would also
// wait for every vector-memory operation, draining the prefetch queue.)  The
// leading builtin repeats the LDS wait where the compiler's counter model
// sees it, so that it does not wait again for reads that already completed.
__device__ __forceinline__ void ring_barrier() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// third descriptor word of a raw byte buffer resource on CDNA (32-bit data
// format, no swizzle, no index stride)
constexpr int kBufferWord3 = 0x00020000;

// Chunk swizzle of operand rows of 128 bytes in LDS: the 16-byte chunk c of row
// r is stored at chunk position c ^ pf_mix(r), which makes 16-byte reads of
// one chunk of 16 consecutive rows free of bank conflicts.
__device__ __forceinline__ int pf_mix(int row) { return (row & 7) ^ ((row >> 3) & 1); }

}  // namespace moe
