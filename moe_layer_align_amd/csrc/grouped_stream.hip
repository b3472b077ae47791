// Grouped expert products with 4-bit weights, for the few rows per expert of
// decoding: bound by the stream of the weights.
//
// A workgroup multiplies a band of one expert's weight rows by that expert's
// rows, 16 or 32 of them per pass.  Weights go from HBM to registers, 16
// bytes (32 weights) per lane and load, are turned into bf16 there and
// multiplied by the 16x16x32 bf16 MFMA, rows as its A operand and weights as
// its B operand, so that a lane's four results are four rows' sums for one
// weight row, the one whose codes and scales the lane itself loads.
//
// A chunk is 128 of K: lane l holds the codes of weight row l%16 at k = 32 *
// (l/16) + 0..31, and its dword j (8 codes) meets the rows' elements at the
// same k in MFMA j: the order of a sum's terms is free as long as both
// operands agree.  Every element of a row is a bf16, every weight exact:
//   MXFP4: the conversion from e2m1 applies the lane's own E8M0 scale, a power
//     of two, exactly; sums run through the chunks in fp32.
//   int4: codes become 16 + q (four bits in a bf16's mantissa: one shift and
//     one and-or for two); a chunk is one scale group, whose sum starts from
//     -24 times the rows' own sum (one more MFMA with a constant operand, shared
//     by the band's tiles) and so ends as the sum of (q - 8) x; it is scaled in
//     fp32 when it joins the total.  (16 + q) - 24 loses at most a few bits of
//     24 (128 + q would lose eight); scaling the weights instead would round
//     each to bf16 and cost as much accuracy as the result's own rounding.
//
// WK waves of a workgroup split K (chunk by chunk, so that together they read
// 64 * WK consecutive bytes of a weight row), the others split the band;
// partial sums meet in LDS and are added in wave order.  Each wave holds FT
// tiles of 16 weight rows, which share the loads of the rows' elements: with
// one tile those are four times the weights' own.
#include "grouped.h"
#include "mfma_tile.h"

namespace moe {
namespace {

constexpr int kChunk = 128;              // K per chunk
constexpr unsigned kOob = 0xffc00000u;   // lane offset past every buffer
enum { kMxfp4 = 1, kInt4 = 2 };

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, kBufferWord3);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, unsigned off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// 8 codes -> 8 bf16 in the order k, or (int4) the pairs (0,4) (1,5) (2,6) (3,7).
template <int FMT>
__device__ __forceinline__ u32x4 dequant(unsigned w, unsigned scale) {
  u32x4 o;
  if constexpr (FMT == kMxfp4) {
    const float s = __uint_as_float(scale);
    o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else {
    constexpr unsigned mask = 0x00780078u, one = 0x41804180u;  // 16 + q: exponent of 16, q in mantissa bits 3..6
    o[0] = ((w << 3) & mask) | one;
    o[1] = ((w >> 1) & mask) | one;
    o[2] = ((w >> 5) & mask) | one;
    o[3] = ((w >> 9) & mask) | one;
  }
  return o;
}

// A row's 8 elements in the order of dequant's.
template <int FMT>
__device__ __forceinline__ u32x4 order(u32x4 x) {
  if constexpr (FMT == kMxfp4) return x;
  return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
               __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

template <int FMT, int FT, int NT>
struct Stage {  // one chunk's loads
  u32x4 w[FT], x[NT][4];
  unsigned s[FT];
};

// Grouped rows [i0, i0 + 16 NT) of expert e, of which those below hi are
// written.
template <int FMT, bool F32, int WK, int FT, int NT>
__device__ __forceinline__ void pass(const GroupedArgs& a, int e, int n0, int i0, int hi, lds_f32* red) {
  constexpr int kBand = 16 * FT * (4 / WK);  // weight rows of the workgroup
  constexpr int kLd = kBand + 4;             // row stride of the partial sums
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave % WK, wb = wave / WK;
  const int r16 = lane & 15, q = lane >> 4;
  const int nchunk = (a.K + kChunk - 1) / kChunk;
  const unsigned wrow = (unsigned)a.K / 2, srow = FMT == kMxfp4 ? (unsigned)a.K / 32 : (unsigned)a.K / 128 * 2;
  const __amdgpu_buffer_rsrc_t rw = buffer(a.w + (int64_t)e * a.N * wrow, (unsigned)a.N * wrow);
  const __amdgpu_buffer_rsrc_t rs = buffer(a.w_scale + (int64_t)e * a.N * srow, (unsigned)a.N * srow);
  const __amdgpu_buffer_rsrc_t rx =
      buffer(a.in.ids ? a.in.p : a.in.p + (int64_t)i0 * a.in.stride * 2, kOob);
  // weight rows at or past N lie past their buffer, and rows that are not read take kOob
  const unsigned n = (unsigned)(n0 + 16 * FT * wb + r16);
  const unsigned w0 = n * wrow + 16 * q, s0 = n * srow + (FMT == kMxfp4 ? q : 0);
  unsigned x0[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int i = i0 + 16 * t + r16;
    const int m = i < hi ? (a.in.ids ? row_of(a.in, i) : i - i0) : -1;
    x0[t] = m >= 0 ? (unsigned)m * (unsigned)(a.in.stride * 2) + 64 * q : kOob;
  }
  auto load = [&](Stage<FMT, FT, NT>& g, int c) {
    const bool ok = c * kChunk + 32 * q < a.K;  // past the end nothing is read: codes, scales and elements are zero
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      g.w[f] = load16(rw, ok ? w0 + 16 * f * wrow + c * 64 : kOob);
      if constexpr (FMT == kMxfp4)
        g.s[f] = (unsigned)__builtin_amdgcn_raw_buffer_load_b8(rs, (int)(ok ? s0 + 16 * f * srow + c * 4 : kOob), 0, 0) << 23;
      else
        g.s[f] = (unsigned)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)(ok ? s0 + 16 * f * srow + c * 2 : kOob), 0, 0) << 16;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) g.x[t][j] = load16(rx, ok ? x0[t] + c * (2 * kChunk) + 16 * j : kOob);
  };
  f32x4 acc[FT][NT] = {};
  auto multiply = [&](const Stage<FMT, FT, NT>& g) {
    u32x4 x[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[t][j] = order<FMT>(g.x[t][j]);
    if constexpr (FMT == kMxfp4) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int f = 0; f < FT; ++f) {
          const u32x4 w = dequant<FMT>(g.w[f][j], g.s[f]);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[f][t] = mfma_bf16(x[t][j], w, acc[f][t]);
        }
    } else {
      constexpr unsigned m24 = 0xc1c0c1c0u;  // a pair of bf16 -24
      f32x4 start[NT] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) start[t] = mfma_bf16(x[t][j], u32x4{m24, m24, m24, m24}, start[t]);
#pragma unroll
      for (int f = 0; f < FT; ++f) {
        f32x4 sum[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) sum[t] = start[t];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 w = dequant<FMT>(g.w[f][j], 0);
#pragma unroll
          for (int t = 0; t < NT; ++t) sum[t] = mfma_bf16(x[t][j], w, sum[t]);
        }
        const float s = __uint_as_float(g.s[f]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[f][t][v] += s * sum[t][v];
      }
    }
  };
  Stage<FMT, FT, NT> g0, g1;
  load(g0, wk);
  for (int c = wk; c < nchunk; c += 2 * WK) {  // loads past the last chunk read nothing
    load(g1, c + WK);
    multiply(g0);
    load(g0, c + 2 * WK);
    multiply(g1);
  }
  // partial sums: [wk][row][weight row]
  __syncthreads();  // the pass before may still be reading
#pragma unroll
  for (int f = 0; f < FT; ++f)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        red[(wk * 16 * NT + 16 * t + 4 * q + v) * kLd + 16 * (FT * wb + f) + r16] = acc[f][t][v];
  __syncthreads();
  constexpr int kPer = F32 ? 4 : 8;  // results per thread and store
  constexpr int kCols = kBand / kPer;
  for (int u = tid; u < 16 * NT * kCols; u += 256) {
    const int row = u / kCols, col = (u % kCols) * kPer, i = i0 + row;
    if (i >= hi || n0 + col >= a.N) continue;
    const int m = row_of(a.out, i);
    if (m < 0) continue;
    f32x4 v[kPer / 4];
#pragma unroll
    for (int h = 0; h < kPer / 4; ++h) {
      v[h] = *(const lds_f32x4*)(red + row * kLd + col + 4 * h);
#pragma unroll
      for (int k = 1; k < WK; ++k) v[h] += *(const lds_f32x4*)(red + (k * 16 * NT + row) * kLd + col + 4 * h);
    }
    const int64_t at = (int64_t)m * a.out.stride + n0 + col;
    if constexpr (F32)
      *(f32x4*)(a.out.p + at * 4) = v[0];
    else
      *(u32x4*)(a.out.p + at * 2) = u32x4{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]),
                                          pack_bf16x2(v[1][0], v[1][1]), pack_bf16x2(v[1][2], v[1][3])};
  }
}

template <int FMT, bool F32, int WK, int FT>
__global__ __launch_bounds__(256) void grouped_stream_kernel(GroupedArgs a) {
  constexpr int kBand = 16 * FT * (4 / WK);
  __shared__ __align__(16) float red[WK * 32 * (kBand + 4)];
  int lo, hi;
  group_range(a.offsets, blockIdx.y, a.R, &lo, &hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  const int n0 = blockIdx.x * kBand;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    if (hi - i0 <= 16)
      pass<FMT, F32, WK, FT, 1>(a, blockIdx.y, n0, i0, hi, (lds_f32*)red);
    else
      pass<FMT, F32, WK, FT, 2>(a, blockIdx.y, n0, i0, hi, (lds_f32*)red);
  }
}

template <int FMT, bool F32, int WK, int FT>
void launch(hipStream_t st, const GroupedArgs& a) {
  constexpr int kBand = 16 * FT * (4 / WK);
  grouped_stream_kernel<FMT, F32, WK, FT><<<dim3((a.N + kBand - 1) / kBand, a.E), 256, 0, st>>>(a);
}

// K is split over the workgroup's waves where it is long enough to keep every
// wave's two stages in flight; a wave holds four tiles where that still leaves
// two workgroups per CU, else one.
template <int FMT, bool F32>
void pick(hipStream_t st, const GroupedArgs& a) {
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int64_t rows = (int64_t)(a.R < a.E ? a.R : a.E) * a.N;  // weight rows that may be read
  if (chunks >= 8)
    rows >= 512 * 64 ? launch<FMT, F32, 4, 4>(st, a) : launch<FMT, F32, 4, 1>(st, a);
  else
    rows >= 512 * 128 ? launch<FMT, F32, 1, 2>(st, a) : launch<FMT, F32, 1, 1>(st, a);
}

}  // namespace

bool launch_grouped_stream(int format, bool f32, hipStream_t st, const GroupedArgs& a) {
  if (format == kMxfp4)
    f32 ? pick<kMxfp4, true>(st, a) : pick<kMxfp4, false>(st, a);
  else
    f32 ? pick<kInt4, true>(st, a) : pick<kInt4, false>(st, a);
  return true;
}

}  // namespace moe
