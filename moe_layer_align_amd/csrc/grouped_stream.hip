// Grouped expert products with 4-bit weights, for the few rows per expert of
// decoding: bound by the stream of the weights.
//
// A workgroup multiplies a band of one expert's weight rows by that expert's
// rows, 16 or 32 of them per pass.  Each wave streams its own part of the band
// through a private pair of LDS stages (no barrier in the loop): direct-to-LDS
// loads of 1 KB take eight whole lines of eight weight rows, where loads
// straight into the MFMA's layout (a lane per row) look up a line per lane and
// were held to 3 TB/s by it.  The fragments of a stage go to registers at once
// and its slot is loaded again, so that nearly two stages per wave are in
// flight.  64 tokens over 256 MXFP4 experts of 4096 x 7168 (2.7 GB): 424 to 458
// us by machine, 5.9 to 6.4 TB/s; one token through 8 of 28672 x 4096 (125 MB) 29 us, a third of it
// start and end of the launch and of its waves.
//
// A step is 256 of K.  In its chunk i (0, 1) of 128, lane l holds the codes of
// weight row l%16 at k = 128 i + 32 * (l/16) + 0..31, and its dword j (8 codes)
// meets the rows' elements at the same k in an MFMA of its own: the order of a
// sum's terms is free as long as both operands agree.  The weights are the B
// operand of the 16x16x32 bf16 MFMA and the rows its A operand, so that a lane's
// four results are four rows' sums for one weight row, the one whose codes and
// scales the lane itself holds.  Every element of a row is a bf16, every weight
// exact:
//   MXFP4: the conversion from e2m1 applies the lane's own E8M0 scale, a power
//     of two, exactly; sums run through the steps in fp32.
//   int4: codes become 16 + q (four bits in a bf16's mantissa: one shift and
//     one and-or for two); a chunk is one scale group, whose sum starts from
//     -24 times the rows' own sum (one more MFMA with a constant operand, shared
//     by the wave's tiles) and so ends as the sum of (q - 8) x; it is scaled in
//     fp32 when it joins the total.  (16 + q) - 24 loses at most a few bits of
//     24 (128 + q would lose eight); scaling the weights instead would round
//     each to bf16 and cost as much accuracy as the result's own rounding.
//
// Each wave holds two or four tiles of 16 weight rows, which share the loads of
// the rows' elements; WK waves split K, step by step, and the others the band;
// partial sums meet in LDS and are added in wave order.
#include <type_traits>

#include "grouped_stream.h"

namespace moe {
namespace {

constexpr int kStep = 256;               // K per step: 128 bytes of a weight row
enum { kMxfp4 = 1, kInt4 = 2 };

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

// int4: 16 + q is the exponent of 16 with q in mantissa bits 3..6.
constexpr unsigned kInt4One = 0x41804180u;

// 8 codes -> 8 bf16 in the order k, or (int4) the pairs (0,4) (1,5) (2,6) (3,7).
// `one` is kInt4One in a vector register: with both constants as literals the
// and-or would be two instructions.
template <int FMT>
__device__ __forceinline__ u32x4 dequant(unsigned w, unsigned scale, unsigned one) {
  u32x4 o;
  if constexpr (FMT == kMxfp4) {
    const float s = __uint_as_float(scale);
    o[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else {
    constexpr unsigned mask = 0x00780078u;
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

// What a wave holds in registers of a step beside its weights: the rows'
// elements and the scales, 8 codes (MXFP4) or 2 bf16 (int4) of each tile's
// weight row, in aligned dwords that start up to three bytes ahead of them.
template <int FMT, int FT, int NT>
struct Step {
  u32x4 x[NT][2][4];
  unsigned s[FT][FMT == kMxfp4 ? 3 : 2];
};

// Grouped rows [i0, i0 + 16 NT) of expert e, of which those below hi are
// written.
template <int FMT, bool F32, int WK, int FT, int NT>
__device__ __forceinline__ void pass(const GroupedArgs& a, int e, int n0, int i0, int hi, lds_u8* smem) {
  constexpr int kBand = 16 * FT * (4 / WK);  // weight rows of the workgroup
  constexpr int kLd = kBand + 4;              // row stride of the partial sums
  constexpr int kStage = stage_bytes(FT);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave % WK, wb = wave / WK;
  const int r16 = lane & 15, q = lane >> 4;
  const int nstep = (a.K + kStep - 1) / kStep;
  const unsigned wrow = (unsigned)a.K / 2, srow = FMT == kMxfp4 ? (unsigned)a.K / 32 : (unsigned)a.K / 128 * 2;
  const __amdgpu_buffer_rsrc_t rw = buffer(a.w + (int64_t)e * a.N * wrow, (unsigned)a.N * wrow);
  const __amdgpu_buffer_rsrc_t rx = buffer(a.in.ids ? a.in.p : a.in.p + (int64_t)i0 * a.in.stride * 2, kOob);
  // the expert's scales, in the aligned dwords that hold them
  const uint8_t* const sp = a.w_scale + (int64_t)e * a.N * srow;
  const unsigned slead = (unsigned)(uintptr_t)sp & 3;
  const __amdgpu_buffer_rsrc_t rs = buffer(sp - slead, ((unsigned)a.N * srow + slead + 3) & ~3u);
  lds_u8* const stage = smem + wave * (2 * kStage);
  const int nb = n0 + 16 * FT * wb;  // the wave's first weight row

  // weights: load d of a step takes rows nb + 8d + lane/8, lane l the 16-byte
  // chunk (l%8) ^ pf_mix(row) of their 128 bytes; rows at or past N lie past
  // the buffer, chunks past K take kOob
  const int wchunk = (lane & 7) ^ (lane >> 3);
  const unsigned w0 = (unsigned)(nb + (lane >> 3)) * wrow + (wchunk << 4);
  const unsigned w1 = (unsigned)(nb + (lane >> 3)) * wrow + ((wchunk ^ 1) << 4);
  auto load_w = [&](int c, int b) {
    const unsigned left = (unsigned)max(a.K / 2 - c * (kStep / 2), 0);  // bytes of a row from this step on
    const bool ok0 = (unsigned)(wchunk << 4) < left, ok1 = (unsigned)((wchunk ^ 1) << 4) < left;
#pragma unroll
    for (int d = 0; d < 2 * FT; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (void __attribute__((address_space(3)))*)(stage + b * kStage + d * 1024), 16,
          (int)((d & 1 ? ok1 : ok0) ? (d & 1 ? w1 : w0) + (unsigned)(8 * d) * wrow + c * (kStep / 2) : kOob), 0, 0, 0);
  };
  const unsigned s0 = (unsigned)(nb + r16) * srow + slead;
  unsigned x0[NT];
  auto load_rest = [&](Step<FMT, FT, NT>& g, int c) {
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      const unsigned at = c < nstep ? (s0 + 16 * f * srow + c * (FMT == kMxfp4 ? 8 : 4)) & ~3u : kOob;
      if constexpr (FMT == kMxfp4) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b96(rs, (int)at, 0, 0);
        g.s[f][0] = v[0];
        g.s[f][1] = v[1];
        g.s[f][2] = v[2];
      } else {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, (int)at, 0, 0);
        g.s[f][0] = v[0];
        g.s[f][1] = v[1];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          g.x[t][i][j] = load16(
              rx, c * kStep + 128 * i + 32 * q < a.K ? x0[t] + c * (2 * kStep) + 256 * i + 16 * j : kOob);
  };

  f32x4 acc[FT][NT] = {};
  unsigned one = kInt4One;
  if constexpr (FMT == kInt4) asm volatile("" : "+v"(one));
  auto multiply = [&](const Step<FMT, FT, NT>& g, const u32x4 (&w)[FT][2], int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u32x4 x[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[t][j] = order<FMT>(g.x[t][i][j]);
      // a scale past the row's end is another row's or none: zero.  The tiles
      // take turns: a tile's sums are a chain of dependent MFMAs.
      if constexpr (FMT == kMxfp4) {
        const bool ok = c * kStep + 128 * i + 32 * q < a.K;
        unsigned s[FT];
#pragma unroll
        for (int f = 0; f < FT; ++f) {
          const unsigned codes = __builtin_amdgcn_alignbyte(g.s[f][i + 1], g.s[f][i], (s0 + 16 * f * srow) & 3u);
          s[f] = ok ? ((codes >> (8 * q)) & 0xffu) << 23 : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < FT; ++f) {
            const u32x4 v = dequant<FMT>(w[f][i][j], s[f], one);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[f][t] = mfma_bf16(x[t][j], v, acc[f][t]);
          }
      } else {
        constexpr unsigned m24 = 0xc1c0c1c0u;  // a pair of bf16 -24
        f32x4 start[NT] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t) start[t] = mfma_bf16(x[t][j], u32x4{m24, m24, m24, m24}, start[t]);
        f32x4 sum[FT][NT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < FT; ++f) {
            const u32x4 v = dequant<FMT>(w[f][i][j], 0, one);
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[f][t] = mfma_bf16(x[t][j], v, j == 0 ? start[t] : sum[f][t]);
          }
#pragma unroll
        for (int f = 0; f < FT; ++f) {
          const unsigned pair = __builtin_amdgcn_alignbyte(g.s[f][1], g.s[f][0], (s0 + 16 * f * srow) & 3u);
          const float s = c * kStep + 128 * i < a.K ? (i ? bf16_hi(pair) : bf16_lo(pair)) : 0.0f;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[f][t][v] += s * sum[f][t][v];
        }
      }
    }
  };
  // Fragments of a stage: tile f's row at f * 2048, chunk 4 i + q.
  const unsigned frag = (unsigned)(uintptr_t)stage + r16 * 128;
  const unsigned frag0 = frag + ((q ^ pf_mix(r16)) << 4), frag1 = frag + (((4 + q) ^ pf_mix(r16)) << 4);

  // One step: its weights have landed when at most the loads issued after them
  // are outstanding, those of the next step (the loads are issued in this order
  // and kept in it by the fences).
  constexpr int kRest = FT + 8 * NT;             // load_rest's loads
  constexpr int kLater = 2 * FT + kRest;         // loads of a step
  static_assert(kLater < 64, "vmcnt range");
  auto fence = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  Step<FMT, FT, NT> g0, g1;
  auto step = [&](Step<FMT, FT, NT>& g, int c, int b, auto later, auto more) {
    fence();
    wait_vm<later()>();
    fence();
    u32x4 w[FT][2];
    read_stage<FT>(w, frag0 + b * kStage, frag1 + b * kStage);  // the stage is read: load it again
    fence();
    if constexpr (more()) load_w(c + 2 * WK, b);
    fence();
    multiply(g, w, c);
    fence();
    if constexpr (more()) load_rest(g, c + 2 * WK);
    fence();
  };
  constexpr std::integral_constant<int, kLater> next_in_flight{};
  constexpr std::integral_constant<int, 0> none_in_flight{};
  // The rows' ids first: loads return in order, and what follows from them
  // would wait for weights loaded ahead of them.
  constexpr int kPer = F32 ? 4 : 8;  // results per thread and store
  constexpr int kCols = kBand / kPer;
  constexpr int kStores = (16 * NT * kCols + 255) / 256;  // of the first threads
  const int last = hi - 1;
  int in_id[NT], out_id[kStores];
#pragma unroll
  for (int t = 0; t < NT; ++t) in_id[t] = a.in.ids ? a.in.ids[min(i0 + 16 * t + r16, last)] : 0;
#pragma unroll
  for (int u = 0; u < kStores; ++u) out_id[u] = a.out.ids ? a.out.ids[min(i0 + (u * 256 + tid) / kCols, last)] : 0;
  fence();
  load_w(wk, 0);
  fence();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int i = i0 + 16 * t + r16;
    const int m = i < hi ? (a.in.ids ? row_of(a.in, i, in_id[t]) : i - i0) : -1;
    x0[t] = m >= 0 ? (unsigned)m * (unsigned)(a.in.stride * 2) + 64 * q : kOob;
  }
  load_rest(g0, wk);
  fence();
  load_w(wk + WK, 1);
  fence();
  load_rest(g1, wk + WK);
  int c = wk;
  for (; c + 2 * WK < nstep; c += 2 * WK) {  // loads past the last step read nothing
    step(g0, c, 0, next_in_flight, std::true_type{});
    step(g1, c + WK, 1, next_in_flight, std::true_type{});
  }
  if (c < nstep) step(g0, c, 0, next_in_flight, std::false_type{});
  if (c + WK < nstep) step(g1, c + WK, 1, none_in_flight, std::false_type{});
  fence();
  wait_vm<0>();  // loads past the last step still write LDS
  lds_f32* const red = (lds_f32*)smem;
  // partial sums: [wk][row][weight row], over the stages
  __syncthreads();
#pragma unroll
  for (int f = 0; f < FT; ++f)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        red[(wk * 16 * NT + 16 * t + 4 * q + v) * kLd + 16 * (FT * wb + f) + r16] = acc[f][t][v];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kStores; ++u) {
    const int at_u = u * 256 + tid, row = at_u / kCols, col = (at_u % kCols) * kPer, i = i0 + row;
    if (row >= 16 * NT || i >= hi || n0 + col >= a.N) continue;
    const int m = row_of(a.out, i, out_id[u]);
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
  __syncthreads();  // the next pass loads over the partial sums
}

template <int FMT, bool F32, int WK, int FT, int NT>
__global__ __launch_bounds__(256, NT == 1 ? 2 : 1) void grouped_stream_kernel(GroupedArgs a) {
  constexpr int kBand = 16 * FT * (4 / WK);
  constexpr int kSums = WK * 16 * NT * (kBand + 4) * 4, kStages = 8 * stage_bytes(FT);
  __shared__ __align__(16) uint8_t smem[kStages];
  static_assert(kSums <= kStages, "the partial sums fit the stages");
  const Found f = find_expert(a.offsets, a.R, a.E);
  if (f.e >= a.E) return;
  for (int i0 = f.lo; i0 < f.hi; i0 += 16 * NT)
    pass<FMT, F32, WK, FT, NT>(a, f.e, blockIdx.x * kBand, i0, f.hi, (lds_u8*)smem);
}

template <int FMT, bool F32, int WK, int FT, int NT>
void launch(hipStream_t st, const GroupedArgs& a) {
  constexpr int kBand = 16 * FT * (4 / WK);
  grouped_stream_kernel<FMT, F32, WK, FT, NT>
      <<<dim3((a.N + kBand - 1) / kBand, a.R < a.E ? a.R : a.E), 256, 0, st>>>(a);
}

// Waves that split K, by its steps of 256 (1, 2, 4 waves): one where they are
// few (32 tokens over 128 experts, N 4096: K 1024 50, 50, 68 us; K 2048 96, 86,
// 91 us), four where they are many and one tile of rows leaves the registers
// (128 tokens over 32 experts of 4096 x 4096, two tiles: 86, 92, 105).  Four
// against two waves, medians of 14 rounds in turn whose quartiles lie within
// 0.5 % (int4 2 %), over 64 and 8 tokens top-8 of 256 experts with N 4096, 32
// tokens top-8 of 128 with N 2048 and one token top-2 of 8 with N 28672: time
// of four 1.01 to 1.21 of two's at 6 and 9 steps, 0.89 to 1.06 at 14 and 20, and
// at 24, 28 and 40 steps 0.89 to 0.99 (MXFP4) and 0.92 to 1.02 (int4); 8 tokens,
// K 6144, MXFP4: 138 against 153 us.  Few
// weight rows leave CUs idle: bands of 32 rows with K over four waves (one
// token, 8 experts of 4096 x 14336: 14 us against 21 with bands of 64 and 35 of
// 128).  Passes of 32 rows read the weights once where experts hold more than
// 8 rows on average; they need too many registers for two waves per SIMD.
template <int FMT, bool F32, int NT>
void pick(hipStream_t st, const GroupedArgs& a) {
  const int steps = (a.K + kStep - 1) / kStep;
  const int64_t rows = (int64_t)(a.R < a.E ? a.R : a.E) * a.N;  // weight rows that may be read
  if (rows < 256 * 64)
    launch<FMT, F32, 4, 2, NT>(st, a);
  else if (NT == 1 && steps >= 24)
    launch<FMT, F32, 4, 4, 1>(st, a);
  else if (steps >= 4)
    launch<FMT, F32, 2, 4, NT>(st, a);
  else
    launch<FMT, F32, 1, 4, NT>(st, a);
}

template <int FMT>
void pick(bool f32, hipStream_t st, const GroupedArgs& a) {
  if (a.R <= 8 * (int64_t)a.E)
    f32 ? pick<FMT, true, 1>(st, a) : pick<FMT, false, 1>(st, a);
  else
    f32 ? pick<FMT, true, 2>(st, a) : pick<FMT, false, 2>(st, a);
}

}  // namespace

bool launch_grouped_stream(int format, bool f32, hipStream_t st, const GroupedArgs& a) {
  if (format == kMxfp4)
    pick<kMxfp4>(f32, st, a);
  else
    pick<kInt4>(f32, st, a);
  return true;
}

}  // namespace moe
