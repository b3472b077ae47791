// Grouped expert products of 8-bit integers for the few rows per expert of
// decoding: bound by the stream of the weights.
//
// As in the 4-bit products a workgroup multiplies a band of one expert's weight
// rows by that expert's rows, 16, 32 or 64 of them per pass, and each wave streams
// its own part of the band through a private pair of LDS stages by direct-to-LDS
// loads of whole lines: 64 tokens over 256 experts of 4096 x 7168, of which 151
// hold rows (4.4 GB), 657 to 682 us by machine, 6.5 to 6.7 TB/s; one token through
// two of 28672 x 4096 (235 MB) 38 to 44 us.
//
// A step is 128 of K, 128 bytes of a weight row: lane l holds bytes 64 i + 16
// (l/16) .. + 15 (i = 0, 1) of weight row l%16, and the same of the rows' codes,
// so that 16x16x64 MFMAs multiply them as they lie.  The weights are the B
// operand: a lane's four results are four rows' sums for one weight row.  Sums
// are exact in int32; the scales join once, at the end.
//
// The four waves split K, step by step (wave w takes steps w, w + 4, ...), and
// their partial sums meet in LDS; where K has few steps each wave takes a band of
// its own instead.  Few weight rows take bands of 32 instead of 64, so that no CU
// is idle.
#include <type_traits>

#include "grouped_stream.h"
#include "int8.h"

namespace moe {
namespace {

constexpr int kStep = 128;  // K per step
constexpr int kFull = 1024;  // workgroups that fill the CUs, two on each, with some to spare
// bf16 rows become codes inside the product, which saves a launch and its codes'
// way through memory, where the weights that may be read are fewer bytes than this
// and the rows few, a call of one launch and of two (us): one token, top-2 of 8
// experts of 1024 x 1024 5.5 and 8.5, 14336 x 4096 24.2 and 26.3; 4 tokens, top-8
// of 128 of 1536 x 2048 21.5 and 20.5; one token, 28672 x 4096 50.5 and 50.5.
// Every band converts the rows anew: 125 rows per expert, 1024 x 1024, 35.6 and 12.9.
constexpr int64_t kOneLaunchBytes = (int64_t)1 << 27;
constexpr int kOneLaunchRows = 4;  // per expert, on average

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) int lds_i32;
typedef __attribute__((address_space(3))) unsigned lds_u32;
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// The largest magnitudes of grouped rows [i0, i0 + n) of bf16, as fp32 bits, to
// top[0..n): wave w takes rows w, w + 4, ...; rows at or beyond hi and masked ones
// have none.
__device__ __forceinline__ void row_tops(const GroupedInt8Args& a, int i0, int n, int hi, lds_u32* top) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  constexpr int kBatch = 8;  // loads in flight
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = a.K / 8;
  for (int r = wave; r < n; r += 4) {
    u16x2 m = {0, 0};
    const int row = i0 + r < hi ? row_of(a.in, i0 + r) : -1;
    if (row >= 0) {
      const u32x4* const p = (const u32x4*)(a.in.p + row * a.in.stride * 2);
      for (int c = lane; c < chunks; c += kBatch * kWave) {
        u32x4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) v[u] = p[min(c + u * kWave, chunks - 1)];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[u][w] & 0x7fff7fffu));
      }
    }
    const unsigned t = wave_umax(m[0] > m[1] ? m[0] : m[1]);
    if (lane == 0) top[r] = t << 16;
  }
}

// Grouped rows [i0, i0 + 16 NT) of expert e, of which those below hi are
// written.  BF16: the rows are bf16 and become codes here, on their way from
// memory to the MFMA, under the largest magnitude that a first look at them
// finds while the first weights are on their way.
template <bool BF16, bool F32, int WK, int FT, int NT>
__device__ __forceinline__ void pass(const GroupedInt8Args& a, int e, int n0, int i0, int hi, lds_u8* smem,
                                     lds_u32* top) {
  constexpr int kBand = 16 * FT * (4 / WK);  // weight rows of the workgroup
  constexpr int kLd = kBand + 4;              // row stride of the partial sums
  constexpr int kStage = stage_bytes(FT);
  constexpr int kEsz = BF16 ? 2 : 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int nstep = (a.K + kStep - 1) / kStep;
  const unsigned wrow = (unsigned)a.K;
  const __amdgpu_buffer_rsrc_t rw = buffer(a.w + (int64_t)e * a.N * wrow, (unsigned)a.N * wrow);
  const __amdgpu_buffer_rsrc_t rx = buffer(a.in.ids ? a.in.p : a.in.p + (int64_t)i0 * a.in.stride * kEsz, kOob);
  lds_u8* const stage = smem + wave * (2 * kStage);
  const int wk = wave % WK, wb = wave / WK, nb = n0 + 16 * FT * wb;  // the wave's first step and weight row

  // weights: load d of a step takes rows nb + 8d + lane/8, lane l the 16-byte
  // chunk (l%8) ^ pf_mix(row) of their 128 bytes; rows at or past N lie past
  // the buffer, chunks past K take kOob
  const int wchunk = (lane & 7) ^ (lane >> 3);
  const unsigned w0 = (unsigned)(nb + (lane >> 3)) * wrow + (wchunk << 4);
  const unsigned w1 = (unsigned)(nb + (lane >> 3)) * wrow + ((wchunk ^ 1) << 4);
  auto load_w = [&](int c, int b) {
    const int left = a.K - c * kStep;  // bytes of a row from this step on
    const bool ok0 = (wchunk << 4) < left, ok1 = ((wchunk ^ 1) << 4) < left;
#pragma unroll
    for (int d = 0; d < 2 * FT; ++d)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (void __attribute__((address_space(3)))*)(stage + b * kStage + d * 1024), 16,
          (int)((d & 1 ? ok1 : ok0) ? (d & 1 ? w1 : w0) + (unsigned)(8 * d) * wrow + c * kStep : kOob), 0, 0, 0);
  };
  unsigned x0[NT];
  struct Step {
    u32x4 x[NT][2][kEsz];
  };
  auto load_x = [&](Step& g, int c) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < kEsz; ++h)
          g.x[t][i][h] = load16(
              rx, c * kStep + 64 * i + 16 * q < a.K ? x0[t] + (unsigned)(c * kStep + 64 * i) * kEsz + 16 * h : kOob);
  };
  RowScale rs[NT];
  auto codes = [&](const Step& g, int t, int i) {
    if constexpr (BF16) {
      float lo[8], hi8[8], v[16];
      unpack8(g.x[t][i][0], lo);
      unpack8(g.x[t][i][kEsz - 1], hi8);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = lo[k];
        v[8 + k] = hi8[k];
      }
      return int8_codes(v, rs[t]);
    } else {
      return g.x[t][i][0];
    }
  };
  i32x4 acc[FT][NT] = {};
  // Fragments of a stage: tile f's row at f * 2048, chunk 4 i + q.
  const unsigned frag = (unsigned)(uintptr_t)stage + r16 * 128;
  const unsigned frag0 = frag + ((q ^ pf_mix(r16)) << 4), frag1 = frag + (((4 + q) ^ pf_mix(r16)) << 4);

  // One step: its loads have landed when at most those of the next step are
  // outstanding (they are issued in this order and kept in it by the fences).
  constexpr int kLater = 2 * FT + 2 * kEsz * NT;  // loads of a step
  static_assert(kLater < 64, "vmcnt range");
  auto fence = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  Step g0, g1;
  auto step = [&](Step& g, int c, int b, auto later, auto more) {
    fence();
    wait_vm<later()>();
    fence();
    u32x4 w[FT][2];
    read_stage<FT>(w, frag0 + b * kStage, frag1 + b * kStage);  // the stage is read: load it again
    fence();
    if constexpr (more()) load_w(c + 2 * WK, b);
    fence();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u32x4 x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t] = codes(g, t, i);
#pragma unroll
      for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[f][t] = mfma_i8(x[t], w[f][i], acc[f][t]);
    }
    fence();
    if constexpr (more()) load_x(g, c + 2 * WK);
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
  int in_id[NT], from_id[kStores], out_id[kStores];
#pragma unroll
  for (int t = 0; t < NT; ++t) in_id[t] = a.in.ids ? a.in.ids[min(i0 + 16 * t + r16, last)] : 0;
#pragma unroll
  for (int u = 0; u < kStores; ++u) {
    const int i = min(i0 + (u * 256 + tid) / kCols, last);
    from_id[u] = a.in.ids ? a.in.ids[i] : 0;
    out_id[u] = a.out.ids ? a.out.ids[i] : 0;
  }
  fence();
  load_w(wk, 0);
  fence();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int i = i0 + 16 * t + r16;
    const int m = i < hi ? (a.in.ids ? row_of(a.in, i, in_id[t]) : i - i0) : -1;
    x0[t] = m >= 0 ? ((unsigned)m * (unsigned)a.in.stride + 16 * q) * kEsz : kOob;
  }
  load_x(g0, wk);
  fence();
  // the scales of the thread's results
  float sa[kStores];
  f32x4 sw[kStores][kPer / 4];
#pragma unroll
  for (int u = 0; u < kStores; ++u) {
    const int at_u = u * 256 + tid, i = min(i0 + at_u / kCols, last), n = min(n0 + (at_u % kCols) * kPer, a.N - kPer);
    if constexpr (!BF16) {
      const int m = row_of(a.in, i, from_id[u]);
      sa[u] = m < 0 ? 0.0f : a.in_scale[m];
    }
#pragma unroll
    for (int h = 0; h < kPer / 4; ++h) sw[u][h] = *(const f32x4*)(a.w_scale + (int64_t)e * a.N + n + 4 * h);
  }
  fence();
  load_w(wk + WK, 1);
  fence();
  load_x(g1, wk + WK);
  if constexpr (BF16) {
    fence();
    row_tops(a, i0, 16 * NT, hi, top);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) rs[t] = row_scale(top[16 * t + r16]);
#pragma unroll
    for (int u = 0; u < kStores; ++u) sa[u] = row_scale(top[min((u * 256 + tid) / kCols, 16 * NT - 1)]).s;
  }
  int c = wk;
  for (; c + 2 * WK < nstep; c += 2 * WK) {  // loads past the last step read nothing
    step(g0, c, 0, next_in_flight, std::true_type{});
    step(g1, c + WK, 1, next_in_flight, std::true_type{});
  }
  if (c < nstep) step(g0, c, 0, next_in_flight, std::false_type{});
  if (c + WK < nstep) step(g1, c + WK, 1, none_in_flight, std::false_type{});
  fence();
  wait_vm<0>();  // loads past the last step still write LDS
  lds_i32* const red = (lds_i32*)smem;
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
      i32x4 s = *(const lds_i32x4*)(red + row * kLd + col + 4 * h);
#pragma unroll
      for (int k = 1; k < WK; ++k) s += *(const lds_i32x4*)(red + (k * 16 * NT + row) * kLd + col + 4 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[h][j] = (float)s[j] * sa[u] * sw[u][h][j];
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

// Most rows of a pass.  bf16 rows cost as much per row as the stream of the
// weights; wide bands need their registers for the results.
constexpr int pass_rows(bool bf16, int wk) { return bf16 || wk == 1 ? 32 : 64; }

// An expert's rows in passes of 64 (32), the last ones in one of 16 or 32 where
// that holds them: the weights are streamed once per pass, and the workgroups of
// a band (blockIdx.z) take its passes in turn.
template <bool BF16, bool F32, int WK, int FT>
__global__ __launch_bounds__(256, 2) void grouped_int8_kernel(GroupedInt8Args a) {
  constexpr int kBand = 16 * FT * (4 / WK), kRows = pass_rows(BF16, WK);
  constexpr int kSums = WK * kRows * (kBand + 4) * 4, kStages = 8 * stage_bytes(FT);
  __shared__ __align__(16) uint8_t smem[kStages > kSums ? kStages : kSums];
  __shared__ unsigned top[kRows];
  const Found f = find_expert(a.offsets, a.R, a.E);
  if (f.e >= a.E) return;
  const int n0 = blockIdx.x * kBand, step = gridDim.z * kRows;
  for (int i0 = f.lo + blockIdx.z * kRows; i0 < f.hi; i0 += step) {
    const int n = f.hi - i0;
    if (n <= 16)
      pass<BF16, F32, WK, FT, 1>(a, f.e, n0, i0, f.hi, (lds_u8*)smem, (lds_u32*)top);
    else if (n <= 32 || kRows == 32)
      pass<BF16, F32, WK, FT, 2>(a, f.e, n0, i0, f.hi, (lds_u8*)smem, (lds_u32*)top);
    else if constexpr (kRows == 64)
      pass<BF16, F32, WK, FT, 4>(a, f.e, n0, i0, f.hi, (lds_u8*)smem, (lds_u32*)top);
  }
}

template <bool BF16, bool F32, int WK, int FT>
void launch(hipStream_t st, const GroupedInt8Args& a) {
  constexpr int kBand = 16 * FT * (4 / WK), kRows = pass_rows(BF16, WK);
  const int bands = (a.N + kBand - 1) / kBand, experts = a.R < a.E ? a.R : a.E, passes = (a.R + kRows - 1) / kRows;
  // few bands: passes side by side, until the CUs are full
  const int64_t blocks = (int64_t)bands * experts;
  const int side = blocks >= kFull ? 1 : (int)((kFull + blocks - 1) / blocks);
  grouped_int8_kernel<BF16, F32, WK, FT>
      <<<dim3(bands, experts, side < passes ? side : passes), 256, 0, st>>>(a);
}

// K of few steps: four bands a workgroup against its four waves on one (us): 238
// experts of 13216 x 144 102.3 and 249.2, 256 of 4096 x 512 55.3 and 69.1, 128 of
// 1536 x 512 17.0 and 19.8, 105 of 5768 x 672 13.5 and 15.0, 128 of 1536 x 768 29.4
// and 28.8, 8 of 32768 x 1024 46.5 and 44.3.
constexpr int kShort = 640;

template <bool BF16, bool F32>
void pick(hipStream_t st, const GroupedInt8Args& a) {
  const int64_t rows = (int64_t)(a.R < a.E ? a.R : a.E) * a.N;  // weight rows that may be read
  if (rows < 256 * 64)
    launch<BF16, F32, 4, 2>(st, a);
  else if (a.K <= kShort)
    launch<BF16, F32, 1, 4>(st, a);
  else
    launch<BF16, F32, 4, 4>(st, a);
}

// Whether the passes over the bands are few: then each takes a workgroup of its
// own, all at once, where few tiles of 256 x 256 would leave most CUs idle
// (streamed and tiled, us): 66 passes over 5 experts of 184 x 7744 16.8 and 67.0;
// 384 of 1024 x 4096 23.5 and 39.7, 640 39.9 and 41.1; 640 of 1024 x 1024 14.7 and
// 19.3, 1136 25.4 and 20.3.  Of short K: 966 over 79 experts of 1736 x 256 12.4 and
// 21.1 (20.4 and 22.8 under a Zipf-like routing), 680 over 17 of 4096 x 512 14.3
// and 19.3, 1088 21.3 and 19.6.
bool few(int R, int E, int64_t N, int64_t K) {
  const int64_t experts = R < E ? R : E;
  return K <= kShort ? (R / 32 + experts) * ((N + 255) / 256) <= 960 : (R / 64 + experts) * ((N + 63) / 64) <= 640;
}

// Streamed or tiled otherwise, by the rows per expert on average (the same).  The
// stream has less to start and end: 402 MB of 128 experts of 1536 x 2048 with 2
// rows 60.6 and 74.6, 8 76.5 and 83.5, 16 78.7 and 87.3, 64 112.9 and 102.0; 268
// MB of 16 experts with 16 55.6 and 68.1.  It streams an expert's weights once per
// 64 rows, which costs where a few experts hold most rows, the more so the more
// there is to stream: under a Zipf-like routing of 16 rows 71.1 and 69.5, 63.1 and
// 77.3, but 505.7 and 367.2 for 3.8 GB (256 experts of 2048 x 7168), which even
// rows take as long in either form (2 rows 523.4 and 525.7, 16 718.6 and 719.4).
bool streamed(int R, int E, int64_t N, int64_t K) {
  const int rows = (R < E ? R : E) * N * K < ((int64_t)1 << 30) ? 16 : 4;
  return R <= rows * (int64_t)E || few(R, E, N, K);
}

}  // namespace

bool int8_rows_in_stream(int R, int E, int64_t N, int64_t K) {
  return streamed(R, E, N, K) && R <= kOneLaunchRows * (int64_t)E && (R < E ? R : E) * N * K < kOneLaunchBytes;
}

bool launch_grouped_int8(bool f32, hipStream_t st, const GroupedInt8Args& a) {
  if (!streamed(a.R, a.E, a.N, a.K)) return launch_grouped_tile_int8(f32, st, a);
  if (a.in_scale)
    f32 ? pick<false, true>(st, a) : pick<false, false>(st, a);
  else
    f32 ? pick<true, true>(st, a) : pick<true, false>(st, a);
  return true;
}

}  // namespace moe
