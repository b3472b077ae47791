// The tokens' way to their experts and back, with the gradients (include/moe.h):
// the copy of the hidden states to rows grouped by expert, the weighted sum of a
// token's rows, the gradient of that sum, and the gradient of the top-k softmax.
//
// All of it is bound by memory: a few operations per element, and what is read
// and written once sets the floor.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "grouped.h"
#include "moe.h"

using namespace moe;

namespace {

constexpr int kThreads = 256;

// 16 bytes of what a call reads once.  Kept out of the caches' way, the rows leave
// them to the results (fresh buffers each call): 4096 tokens, top-8, H 2048,
// combine_grad with the router's gradient 77.8 -> 57.6 us, dispatch 32.9 -> 30.4;
// 8192 tokens, top-2, H 4096, fp32 rows, combine 63.6 -> 60.4.
__device__ __forceinline__ u32x4 load_once(const uint8_t* p) { return __builtin_nontemporal_load((const u32x4*)p); }

// ---------------------------------------------------------------- dispatch
// A counting sort of the pairs by expert, stable in the pair index, and the copy
// of the tokens' rows to where it puts them, in one kernel: workgroup x owns
// `group` tokens, finds their pairs' rows and copies each token's row, which it
// reads once for all its pairs (a copy that runs over the sorted rows would read
// it again for every pair).
//
// How many pairs of each expert there are, and how many before a workgroup's
// own, comes by the number of pairs from
//   kCountAll   a count of all ids by every workgroup itself: one launch, for
//               decoding, where it takes less than a second launch would
//   kSumChunks  the counts of chunks of kChunk pairs, made by a launch before
//               this one: every workgroup adds up those of all chunks
//   kScanned    the same, added up by a launch between the two
// and in the latter two a count of the ids of its own chunk before its first.
enum Counts { kCountAll, kSumChunks, kScanned };

constexpr int kChunk = 1024;           // pairs per chunk of the counts
constexpr int kOwn = 64;               // pairs of a workgroup at most: one wave ranks them
constexpr int kCountAllPairs = 4096;   // at most so many pairs are counted by every workgroup
constexpr int kSumChunksCounts = 8192; // at most so many counts are added up by every workgroup

struct DispatchArgs {
  const uint8_t* x;
  int64_t x_stride;    // bytes
  const int32_t* ids;  // [M*k]
  int M, k, E, first, group;
  int row_bytes;       // multiple of 16
  uint8_t* rows;
  int64_t rows_stride;  // bytes
  int32_t* offsets;     // [E+1]
  int32_t* positions;   // [M*k]
  int32_t* pairs;       // [M*k]
  int32_t* counts;      // [chunks][E] counts, or (scanned) those of the chunks before, and [E] the totals behind them
  int chunks;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ bool local_expert(int id, int first, int E, int* e) {
  *e = __builtin_elementwise_sub_sat(id, first);  // negative for every id below `first` (first >= 0)
  return (unsigned)*e < (unsigned)E;
}

__global__ __launch_bounds__(kThreads) void count_chunks_kernel(const int32_t* __restrict__ ids, int P, int E,
                                                                int first, int32_t* __restrict__ counts) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kThreads) count[e] = 0;
  __syncthreads();
  const int f0 = blockIdx.x * kChunk + threadIdx.x;
  int id[kChunk / kThreads];
#pragma unroll
  for (int i = 0; i < kChunk / kThreads; ++i) id[i] = f0 + i * kThreads < P ? ids[f0 + i * kThreads] : 0;
#pragma unroll
  for (int i = 0; i < kChunk / kThreads; ++i) {
    int e;
    if (f0 + i * kThreads < P && local_expert(id[i], first, E, &e)) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) counts[(int64_t)blockIdx.x * E + e] = count[e];
}

// Each expert's counts become sums over the chunks before, a lane per expert
// (whole lines of experts at a step); the totals go behind the last chunk.
// The 16 waves of a workgroup split the chunks: their sums first, then the
// running sums from them on.
__global__ __launch_bounds__(1024) void scan_chunks_kernel(int32_t* __restrict__ counts, int chunks, int E) {
  __shared__ int sum[16][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * kWave + lane;
  const int per = (chunks + 15) / 16, c0 = min(wave * per, chunks), c1 = min(c0 + per, chunks);
  constexpr int kBatch = 8;  // loads in flight
  int n[kBatch], s = 0;
  auto load = [&](int c) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) n[i] = e < E && c + i < c1 ? counts[(int64_t)(c + i) * E + e] : 0;
  };
  for (int c = c0; c < c1; c += kBatch) {
    load(c);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) s += n[i];
  }
  sum[wave][lane] = s;
  __syncthreads();
  int run = 0, total = 0;
  for (int w = 0; w < 16; ++w) {
    run += w < wave ? sum[w][lane] : 0;
    total += sum[w][lane];
  }
  if (e >= E) return;
  for (int c = c0; c < c1; c += kBatch) {
    load(c);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (c + i < c1) counts[(int64_t)(c + i) * E + e] = run;
      run += n[i];
    }
  }
  if (wave == 0) counts[(int64_t)chunks * E + e] = total;
}

template <int COUNTS>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(DispatchArgs a) {
  __shared__ int total[kMaxExperts];   // pairs of each expert
  __shared__ int before[kMaxExperts];  // those ahead of the workgroup's own, then the expert's first free row
  __shared__ int wave_sum_[4];
  __shared__ int place[kOwn];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int P = a.M * a.k;
  const int t0 = blockIdx.x * a.group, t1 = min(t0 + a.group, a.M);
  const int f0 = t0 * a.k, f1 = t1 * a.k;  // the workgroup's own pairs
  const int chunk = f0 / kChunk;
  constexpr int kBatch = 8;  // loads in flight
  for (int e = tid; e < a.E; e += kThreads) {
    total[e] = COUNTS == kScanned ? a.counts[(int64_t)a.chunks * a.E + e] : 0;
    before[e] = COUNTS == kScanned ? a.counts[(int64_t)chunk * a.E + e] : 0;
  }
  __syncthreads();
  if constexpr (COUNTS == kSumChunks) {  // thread i: expert i % width of the chunks i / width, i / width + step, ...
    const int width = a.E < kThreads ? a.E : kThreads, step = kThreads / width;
    const int first = tid / width, of = tid - first * width;
    for (int e = of; e < a.E && first < step; e += width) {
      int n = 0, b = 0;
      for (int c = first; c < a.chunks; c += kBatch * step) {
        int v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = c + i * step < a.chunks ? a.counts[(c + i * step) * a.E + e] : 0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          n += v[i];
          b += c + i * step < chunk ? v[i] : 0;
        }
      }
      atomicAdd(&total[e], n);
      atomicAdd(&before[e], b);
    }
  }
  const int c0 = COUNTS == kCountAll ? 0 : chunk * kChunk, c1 = COUNTS == kCountAll ? P : f0;
  for (int f = c0 + tid; f < c1; f += kBatch * kThreads) {
    int id[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) id[i] = f + i * kThreads < c1 ? a.ids[f + i * kThreads] : 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      int e;
      if (f + i * kThreads >= c1 || !local_expert(id[i], a.first, a.E, &e)) continue;
      if constexpr (COUNTS == kCountAll) atomicAdd(&total[e], 1);
      if (COUNTS != kCountAll || f + i * kThreads < f0) atomicAdd(&before[e], 1);
    }
  }
  __syncthreads();
  // the experts' first rows: a scan of two experts a thread
  {
    const int e = 2 * tid;
    const int n0 = e < a.E ? total[e] : 0, n1 = e + 1 < a.E ? total[e + 1] : 0;
    const int incl = wave_incl_scan(n0 + n1);
    if (lane == 63) wave_sum_[wave] = incl;
    __syncthreads();
    int start = incl - n0 - n1;
#pragma unroll
    for (int w = 0; w < 4; ++w) start += w < wave ? wave_sum_[w] : 0;
    if (e < a.E) before[e] += start;
    if (e + 1 < a.E) before[e + 1] += start + n0;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      if (e < a.E) a.offsets[e] = start;
      if (e + 1 < a.E) a.offsets[e + 1] = start + n0;
      if (tid == 0) a.offsets[a.E] = wave_sum_[0] + wave_sum_[1] + wave_sum_[2] + wave_sum_[3];
    }
  }
  __syncthreads();
  const int held = wave_sum_[0] + wave_sum_[1] + wave_sum_[2] + wave_sum_[3];
  if (wave == 0) {  // a pair's row: its rank among the lanes of the same expert, by a match over the bits of its number
    const int f = f0 + lane;
    int e = 0;
    const bool ok = f < f1 && local_expert(a.ids[f], a.first, a.E, &e);
    unsigned long long same = __ballot(ok);
    for (int b = 0; (1 << b) < a.E; ++b) {
      const bool bit = ok && ((e >> b) & 1);
      const unsigned long long m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    const int p = ok ? before[e] + __popcll(same & lanemask_lt(lane)) : -1;
    place[lane] = p;
    if (blockIdx.y == 0 && f < f1) {
      a.positions[f] = p;
      if (ok) a.pairs[p] = f;
      if (f >= held) a.pairs[f] = -1;  // the rows behind the last expert's
    }
  }
  if (!a.rows) return;  // the layout alone
  __syncthreads();
  // the copy, only of tokens with a row here
  const int per_row = a.row_bytes / 16;
  if (per_row >= kWave) {
    // a wave takes 4 KB of a token's row at a time, for all its places
    const int parts = (per_row + 4 * kWave - 1) / (4 * kWave), n = (t1 - t0) * parts;
    for (int i = blockIdx.y * 4 + uniform(wave); i < n; i += gridDim.y * 4) {
      const int t = i / parts, c = (i - t * parts) * (4 * kWave) + lane;
      int p = lane < a.k ? place[t * a.k + lane] : -1;
      unsigned long long todo = __ballot(p >= 0);
      if (!todo) continue;
      const uint8_t* src = a.x + (t0 + t) * a.x_stride;
      u32x4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = load_once(src + min(c + u * kWave, per_row - 1) * 16);
      for (; todo; todo &= todo - 1) {
        uint8_t* dst = a.rows + __builtin_amdgcn_readlane(p, __ffsll(todo) - 1) * a.rows_stride;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + u * kWave < per_row) *(u32x4*)(dst + (c + u * kWave) * 16) = v[u];
      }
    }
  } else {
    const int n = (t1 - t0) * per_row;
    for (int i = blockIdx.y * kThreads + tid; i < n; i += gridDim.y * kThreads) {
      const int t = i / per_row, c = i - t * per_row;
      u32x4 v;
      bool have = false;
      for (int j = 0; j < a.k; ++j) {
        const int p = place[t * a.k + j];
        if (p < 0) continue;
        if (!have) v = load_once(a.x + (t0 + t) * a.x_stride + c * 16);
        have = true;
        *(u32x4*)(a.rows + p * a.rows_stride + c * 16) = v;
      }
    }
  }
}

// ---------------------------------------------------------------- combine
// Eight values from the 16 bytes, or (fp32) twice 16, that hold them.
template <bool F32>
__device__ __forceinline__ void unpack8(const u32x4* w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[F32 ? i : 2 * i] = F32 ? __uint_as_float(w[0][i]) : bf16_lo(w[0][i]);
    v[F32 ? 4 + i : 2 * i + 1] = F32 ? __uint_as_float(w[F32][i]) : bf16_hi(w[0][i]);
  }
}
__device__ __forceinline__ void store8(uint8_t* p, bool f32, const float (&v)[8]) {
  if (f32) {
    *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4*)(p + 16) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *(u32x4*)p = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
  }
}

// N consecutive 4-byte values, whose address is a multiple of 4.
template <typename T, int N>
__device__ __forceinline__ void load_dwords(T (&v)[N], const T* p) {
  typedef unsigned words __attribute__((ext_vector_type(N < 4 ? N : 4), aligned(4)));
  constexpr int kWords = N < 4 ? N : 4;
#pragma unroll
  for (int i = 0; i < N; i += kWords) {
    const words x = *(const words*)(p + i);
#pragma unroll
    for (int j = 0; j < kWords; ++j) v[i + j] = __builtin_bit_cast(T, (unsigned)x[j]);
  }
}

struct CombineArgs {
  const uint8_t* rows;
  int64_t rows_stride;  // bytes
  int R;
  const int32_t* positions;
  const float* weights;  // null: ones
  int M, k, H;
  uint8_t* y;
  int64_t y_stride;  // bytes
  int y_f32;
  int per_wg;  // tokens of a workgroup at a time
};

// Eight columns of a token per thread.  The loads of up to KB slots are in
// flight together; the sum runs over the slots in order, in fp32.
template <bool F32, int KB>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs a) {
  const int cols = a.H / 8;
  const int of = a.per_wg > 1 ? threadIdx.x / cols : 0;
  const int col = a.per_wg > 1 ? threadIdx.x - of * cols : blockIdx.y * kThreads + threadIdx.x;
  if (of >= a.per_wg || col >= cols) return;
  for (int t = blockIdx.x * a.per_wg + of; t < a.M; t += gridDim.x * a.per_wg) {
    const int32_t* pos = a.positions + (int64_t)t * a.k;
    const float* w = a.weights ? a.weights + (int64_t)t * a.k : nullptr;
    float sum[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      u32x4 raw[KB][F32 ? 2 : 1];
      int at[KB];
      float wj[KB];
      bool ok[KB];
      auto place = [&](int j) {
        at[j] = j0 + j < a.k ? pos[j0 + j] : -1;
        wj[j] = w && j0 + j < a.k ? w[j0 + j] : 1.0f;
      };
      // all places of four or eight slots ahead of their rows, whole batches by wide loads: top-8, 4096 tokens,
      // H 2048 29.7 -> 26.9 us; 32138 tokens, H 128, 8 of 27 experts here 13.3 -> 8.5; two slots lose 3 % by it
      if constexpr (KB > 2) {
        if (j0 + KB <= a.k) {
          load_dwords(at, pos + j0);
          if (w) load_dwords(wj, w + j0);
        } else {
#pragma unroll
          for (int j = 0; j < KB; ++j) place(j);
        }
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if constexpr (KB <= 2) place(j);
        const int p = at[j];
        ok[j] = (unsigned)p < (unsigned)a.R;
        if (!w) wj[j] = 1.0f;
        if (ok[j])
#pragma unroll
          for (int i = 0; i < (F32 ? 2 : 1); ++i)
            raw[j][i] = load_once(a.rows + p * a.rows_stride + (int64_t)col * (F32 ? 32 : 16) + 16 * i);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (!ok[j]) continue;
        float v[8];
        unpack8<F32>(raw[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += wj[j] * v[i];
      }
    }
    store8(a.y + t * a.y_stride + (int64_t)col * (a.y_f32 ? 32 : 16), a.y_f32, sum);
  }
}

struct CombineGradArgs {
  const uint8_t* dy;
  int64_t dy_stride;
  int dy_f32;
  const uint8_t* rows;  // null: dweights not wanted
  int64_t rows_stride;
  int R;
  const int32_t* positions;
  const float* weights;
  int M, k, H;
  uint8_t* drows;  // null: not wanted
  int64_t drows_stride;
  int drows_f32;
  float* dweights;
  int run;  // tokens at a time, run * k <= 64
};

// WPT waves work on one token (so that each of its dweights is one sum in a
// fixed order), 512 columns per wave and step, whose dy is read once for up to
// KB slots.  The loads of a step are issued before the step ahead of it is
// multiplied and stored: without that a wave's reads and writes take turns (4096
// tokens, top-8, H 2048, with the router's gradient, a wave per token and the
// results in one buffer: 73.2 -> 60.5 us).  Of four waves per token and one, in
// fresh buffers: 55.1 and 57.5.
//
// The waves take runs of tokens: one load has a run's places and weights, a lane
// each, and a ballot its tokens with rows.  The others, most of them where the
// experts are spread over many processes, cost no more than their zero weights,
// and their dy is not read (16384 tokens, top-8, H 2048, with the router's
// gradient, 8 of 256 experts here, against a workgroup per token that reads its
// dy: 88.4 -> 42.9 us; 32 here, uneven, 96.7 -> 68.6; all experts here, 4096
// tokens, 54.9 -> 53.5).
template <bool F32, int KB, int WPT>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGradArgs a) {
  constexpr int kRuns = 4 / WPT;  // per workgroup
  __shared__ float part[4][KB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wt = wave % WPT;
  const unsigned long long slots = ~0ull >> (64 - a.k);
  for (int64_t t0 = (int64_t)blockIdx.x * kRuns * a.run; t0 < a.M; t0 += (int64_t)gridDim.x * kRuns * a.run) {
    const int first = (int)t0 + wave / WPT * a.run;
    const int64_t pair = (int64_t)first * a.k + lane;
    const bool mine = lane < a.run * a.k && pair < (int64_t)a.M * a.k;
    int place = mine ? a.positions[pair] : -1;
    const float weight = mine && a.weights ? a.weights[pair] : 1.0f;
    if ((unsigned)place >= (unsigned)a.R) place = -1;
    unsigned long long left = __ballot(place >= 0);
    if (a.dweights && wt == 0 && mine && !(left >> (lane / a.k * a.k) & slots)) a.dweights[pair] = 0.0f;
    while (left) {
      const int at = (int)__builtin_ctzll(left) / a.k * a.k;
      left &= ~(slots << at);
      const int t = first + at / a.k;
      for (int j0 = 0; j0 < a.k; j0 += KB) {
        int p[KB];
        float w[KB], dot[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const int from = at + j0 + j;
          p[j] = j0 + j < a.k ? __builtin_amdgcn_readlane(place, from & 63) : -1;
          w[j] = __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(weight), from & 63));
          dot[j] = 0.0f;
        }
        bool any = false;
#pragma unroll
        for (int j = 0; j < KB; ++j) any |= p[j] >= 0;
        constexpr int kRaw = F32 ? 2 : 1;
        u32x4 d[2], next[KB][kRaw];
        const uint8_t* const dy = a.dy + (int64_t)t * a.dy_stride;
        auto load = [&](int col) {
          if (col >= a.H) return;
          d[0] = load_once(dy + (int64_t)col * (a.dy_f32 ? 4 : 2));
          if (a.dy_f32) d[1] = load_once(dy + (int64_t)col * 4 + 16);
          if (!a.rows) return;
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (p[j] >= 0)
#pragma unroll
              for (int i = 0; i < kRaw; ++i)
                next[j][i] = load_once(a.rows + p[j] * a.rows_stride + (int64_t)col * (F32 ? 4 : 2) + 16 * i);
        };
        const int col0 = (wt * 64 + lane) * 8;
        if (any) load(col0);
        if (any)
          for (int col = col0; col < a.H; col += WPT * 512) {
            float g[8];
            if (a.dy_f32)
              unpack8<true>(d, g);
            else
              unpack8<false>(d, g);
            u32x4 row[KB][kRaw];
#pragma unroll
            for (int j = 0; j < KB; ++j)
#pragma unroll
              for (int i = 0; i < kRaw; ++i) row[j][i] = next[j][i];
            load(col + WPT * 512);
#pragma unroll
            for (int j = 0; j < KB; ++j) {
              if (p[j] < 0) continue;
              if (a.rows) {
                float r[8];
                unpack8<F32>(row[j], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot[j] += g[i] * r[i];
              }
              if (a.drows) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = w[j] * g[i];
                store8(a.drows + p[j] * a.drows_stride + (int64_t)col * (a.drows_f32 ? 4 : 2), a.drows_f32, o);
              }
            }
          }
        if (!a.dweights) continue;
#pragma unroll
        for (int j = 0; j < KB; ++j) dot[j] = wave_sum(dot[j]);
        if constexpr (WPT > 1) {
          if (lane == 0)
#pragma unroll
            for (int j = 0; j < KB; ++j) part[wave][j] = dot[j];
          __syncthreads();
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            dot[j] = part[wave - wt][j];
#pragma unroll
            for (int i = 1; i < WPT; ++i) dot[j] += part[wave - wt + i][j];
          }
          __syncthreads();
        }
        if (wt == 0 && lane == 0)
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (j0 + j < a.k) a.dweights[(int64_t)t * a.k + j0 + j] = dot[j];
      }
    }
  }
}

// The same for rows of at most 8 LANES columns, a token per LANES lanes: a wave per
// token would leave most of its lanes idle (19047 tokens, top-6, H 96, with the
// router's gradient 37.7 -> 19.4 us; 32000, top-4, H 256 54.8 -> 39.3).
template <bool F32, int KB, int LANES>
__global__ __launch_bounds__(kThreads) void combine_grad_narrow_kernel(CombineGradArgs a) {
  constexpr int kTokens = kThreads / LANES;  // per workgroup
  const int l = threadIdx.x % LANES, col = l * 8;
  // whole groups of lanes take a token or none, so that their exchange below has all of them
  for (int t = blockIdx.x * kTokens + threadIdx.x / LANES; t < a.M; t += gridDim.x * kTokens) {
    const bool in = col < a.H;
    float g[8] = {};
    if (in) {
      const uint8_t* const dy = a.dy + t * a.dy_stride + col * (a.dy_f32 ? 4 : 2);
      u32x4 d[2] = {load_once(dy), {}};
      if (a.dy_f32) {
        d[1] = load_once(dy + 16);
        unpack8<true>(d, g);
      } else {
        unpack8<false>(d, g);
      }
    }
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      int p[KB];
      float w[KB], dot[KB];
      u32x4 raw[KB][F32 ? 2 : 1];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        p[j] = j0 + j < a.k ? a.positions[(int64_t)t * a.k + j0 + j] : -1;
        if (!in || (unsigned)p[j] >= (unsigned)a.R) p[j] = -1;
        w[j] = p[j] >= 0 && a.weights ? a.weights[(int64_t)t * a.k + j0 + j] : 1.0f;
        if (p[j] >= 0 && a.rows)
#pragma unroll
          for (int i = 0; i < (F32 ? 2 : 1); ++i)
            raw[j][i] = load_once(a.rows + p[j] * a.rows_stride + col * (F32 ? 4 : 2) + 16 * i);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        dot[j] = 0.0f;
        if (p[j] < 0) continue;
        if (a.rows) {
          float r[8];
          unpack8<F32>(raw[j], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot[j] += g[i] * r[i];
        }
        if (a.drows) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = w[j] * g[i];
          store8(a.drows + p[j] * a.drows_stride + col * (a.drows_f32 ? 4 : 2), a.drows_f32, o);
        }
      }
      if (!a.dweights) continue;
#pragma unroll
      for (int j = 0; j < KB; ++j) {
#pragma unroll
        for (int i = 1; i < LANES; i *= 2) dot[j] += __shfl_xor(dot[j], i);
        if (l == 0 && j0 + j < a.k) a.dweights[(int64_t)t * a.k + j0 + j] = dot[j];
      }
    }
  }
}

// ---------------------------------------------------------------- router
// dlogits of a token: w_j (dw_j - sum_i w_i dw_i) at its selected experts, zero
// at the others.  A wave per token: lane j holds slot j, every lane adds up the
// slots that name its experts (equal ids add up).  All lanes go through the
// experts together, and only the store is left out past the last one: a loop that
// lanes leave would let the compiler form g for the lanes in it alone, where the
// slots of the others are read too.
__global__ __launch_bounds__(kThreads) void route_grad_kernel(const int32_t* __restrict__ ids,
                                                              const float* __restrict__ w,
                                                              const float* __restrict__ dw, int M, int E, int k,
                                                              float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  for (int t = blockIdx.x * 4 + wave; t < M; t += gridDim.x * 4) {
    const int64_t at = (int64_t)t * k + lane;
    const int id = lane < k ? ids[at] : -1;
    const bool ok = (unsigned)id < (unsigned)E;
    const float wj = ok ? w[at] : 0.0f, dj = ok ? dw[at] : 0.0f;
    const float mean = wave_sum(wj * dj);
    const float g = wj * (dj - mean);
    for (int e0 = 0; e0 < E; e0 += kWave) {
      const int e = e0 + lane;
      float s = 0.0f;
      for (int j = 0; j < k; ++j) {
        const int ij = __builtin_amdgcn_readlane(id, j);
        const float gj = __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(g), j));
        s += ij == e ? gj : 0.0f;
      }
      if (e < E) dlogits[(int64_t)t * E + e] = s;
    }
  }
}

// ---------------------------------------------------------------- host side
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status_t launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE; }

constexpr int kMaxPairs = 1 << 26;
constexpr int64_t kMaxRowBytes = (int64_t)1 << 22;
constexpr int kMaxGrid = 1 << 22;

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
int grid_of(int64_t n) { return (int)(n < kMaxGrid ? n : kMaxGrid); }

bool routed(int M, int k) { return (int64_t)M * k < kMaxPairs && k <= kMaxTopK; }

// Rows of `width` elements of `esz` bytes, `stride` elements apart.
moe_status_t check_matrix(const void* p, int64_t stride, int64_t width, int esz) {
  if (!p || !aligned(p, 16) || stride < width || stride % 16 * esz % 16) return MOE_ERR_INVALID_ARG;
  return stride >= kMaxRowBytes / esz ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

bool known(moe_out_t t) { return t == MOE_OUT_BF16 || t == MOE_OUT_FP32; }
int size_of(moe_out_t t) { return t == MOE_OUT_FP32 ? 4 : 2; }

template <bool F32>
void launch_combine(int grid_y, hipStream_t st, const CombineArgs& a) {
  const dim3 grid(grid_of(cdiv(a.M, a.per_wg)), grid_y);
  if (a.k <= 2)
    combine_kernel<F32, 2><<<grid, kThreads, 0, st>>>(a);
  else if (a.k <= 4)
    combine_kernel<F32, 4><<<grid, kThreads, 0, st>>>(a);
  else
    combine_kernel<F32, 8><<<grid, kThreads, 0, st>>>(a);
}

// Runs of tokens of combine_grad.  More runs balance better where every token has
// rows, fewer cost less where most have none.  8192, 4096 and 2048 (us, with the
// router's gradient): 16384 tokens, top-8, H 2048, 8 of 256 experts here 44.3, 42.9
// and 43.0, 128 here 133.3, 139.3 and 144.0; 8192, top-2, H 4096, 1 of 8 here 18.9,
// 17.8 and 20.9.
constexpr int kGradRuns = 4096;

template <bool F32, int KB>
void launch_combine_grad(hipStream_t st, CombineGradArgs a) {
  const int runs = a.H <= 1024 ? 4 * kGradRuns : kGradRuns;
  a.run = a.M / runs < 1 ? 1 : a.M / runs < kWave / a.k ? a.M / runs : kWave / a.k;
  if (a.H <= 64)
    combine_grad_narrow_kernel<F32, KB, 8><<<grid_of(cdiv(a.M, kThreads / 8)), kThreads, 0, st>>>(a);
  else if (a.H <= 128)
    combine_grad_narrow_kernel<F32, KB, 16><<<grid_of(cdiv(a.M, kThreads / 16)), kThreads, 0, st>>>(a);
  else if (a.H <= 256)
    combine_grad_narrow_kernel<F32, KB, 32><<<grid_of(cdiv(a.M, kThreads / 32)), kThreads, 0, st>>>(a);
  else if (a.H <= 1024)
    combine_grad_kernel<F32, KB, 1><<<grid_of(cdiv(a.M, 4 * a.run)), kThreads, 0, st>>>(a);
  else
    combine_grad_kernel<F32, KB, 4><<<grid_of(cdiv(a.M, a.run)), kThreads, 0, st>>>(a);
}

}  // namespace

extern "C" {

size_t moe_dispatch_workspace_size(int32_t M, int32_t top_k, int32_t E) {
  if (M < 0 || top_k < 1 || E < 1 || E > kMaxExperts || !routed(M, top_k)) return 0;
  const int P = M * top_k;
  return P <= kCountAllPairs ? 0 : (size_t)(cdiv(P, kChunk) + 1) * E * 4;
}

moe_status_t moe_dispatch(const moe_dispatch_args_t* a, void* stream) {
  if (!a || a->M < 0 || a->E < 1 || a->top_k < 1 || a->first_expert < 0) return MOE_ERR_INVALID_ARG;
  const bool copy = a->x || a->rows;
  if (copy && a->row_bytes < 1) return MOE_ERR_INVALID_ARG;
  if (!routed(a->M, a->top_k) || a->E > kMaxExperts ||
      (copy && (a->row_bytes % 16 || a->row_bytes >= kMaxRowBytes)))
    return MOE_ERR_UNSUPPORTED;
  if (!a->offsets || !aligned(a->offsets, 4)) return MOE_ERR_INVALID_ARG;
  const hipStream_t st = (hipStream_t)stream;
  DispatchArgs d = {};
  d.M = a->M;
  d.k = a->top_k;
  d.E = a->E;
  d.first = a->first_expert;
  d.row_bytes = copy ? a->row_bytes : 0;
  d.offsets = a->offsets;
  d.group = 1;
  const int P = a->M * a->top_k;
  if (P > 0) {
    if (!a->ids || !aligned(a->ids, 4) || !a->positions || !aligned(a->positions, 4) || !a->pairs ||
        !aligned(a->pairs, 4))
      return MOE_ERR_INVALID_ARG;
    moe_status_t rc;
    if (copy && (rc = check_matrix(a->x, a->x_stride, a->row_bytes, 1)) != MOE_OK) return rc;
    if (copy && (rc = check_matrix(a->rows, a->rows_stride, a->row_bytes, 1)) != MOE_OK) return rc;
    d.x = (const uint8_t*)a->x;
    d.x_stride = a->x_stride;
    d.ids = a->ids;
    d.rows = (uint8_t*)a->rows;
    d.rows_stride = a->rows_stride;
    d.positions = a->positions;
    d.pairs = a->pairs;
    d.chunks = cdiv(P, kChunk);
    if (P > kCountAllPairs) {
      if (!a->workspace || !aligned(a->workspace, 16)) return MOE_ERR_INVALID_ARG;
      if (a->workspace_bytes < moe_dispatch_workspace_size(a->M, a->top_k, a->E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
      d.counts = (int32_t*)a->workspace;
    }
    // tokens of a workgroup: as many as one wave ranks, fewer where that would leave CUs idle
    const int most = kOwn / d.k, even = cdiv(d.M, 512);
    d.group = even < most ? even : most;
  }
  const int groups = P ? cdiv(d.M, d.group) : 1;
  // few workgroups share a token's row
  const int steps = cdiv((int64_t)d.group * (d.row_bytes / 16), 4 * kThreads);
  int split = 256 / groups < steps ? 256 / groups : steps;
  if (split < 1) split = 1;
  const dim3 grid(groups, split);
  if (P <= kCountAllPairs) {
    dispatch_kernel<kCountAll><<<grid, kThreads, 0, st>>>(d);
  } else {
    count_chunks_kernel<<<d.chunks, kThreads, 0, st>>>(d.ids, P, d.E, d.first, d.counts);
    if (d.chunks * (int64_t)d.E <= kSumChunksCounts) {
      dispatch_kernel<kSumChunks><<<grid, kThreads, 0, st>>>(d);
    } else {
      scan_chunks_kernel<<<cdiv(d.E, kWave), 1024, 0, st>>>(d.counts, d.chunks, d.E);
      dispatch_kernel<kScanned><<<grid, kThreads, 0, st>>>(d);
    }
  }
  return launch_status();
}

moe_status_t moe_combine(const moe_combine_args_t* a, void* stream) {
  if (!a || a->M < 0 || a->R < 0 || a->top_k < 1 || a->H < 1 || !known(a->rows_type) || !known(a->y_type))
    return MOE_ERR_INVALID_ARG;
  if (!routed(a->M, a->top_k) || a->R > kMaxPairs || a->H % 8) return MOE_ERR_UNSUPPORTED;
  if (a->M == 0) return MOE_OK;
  if (!a->positions || !aligned(a->positions, 4) || !aligned(a->weights, 4)) return MOE_ERR_INVALID_ARG;
  moe_status_t rc;
  if ((rc = check_matrix(a->rows, a->rows_stride, a->H, size_of(a->rows_type))) != MOE_OK) return rc;
  if ((rc = check_matrix(a->y, a->y_stride, a->H, size_of(a->y_type))) != MOE_OK) return rc;
  CombineArgs c = {};
  const int cols = a->H / 8;
  c.rows = (const uint8_t*)a->rows;
  c.rows_stride = a->rows_stride * size_of(a->rows_type);
  c.R = a->R;
  c.positions = a->positions;
  c.weights = a->weights;
  c.M = a->M;
  c.k = a->top_k;
  c.H = a->H;
  c.y = (uint8_t*)a->y;
  c.y_stride = a->y_stride * size_of(a->y_type);
  c.y_f32 = a->y_type == MOE_OUT_FP32;
  c.per_wg = cols < kThreads ? kThreads / cols : 1;
  const int grid_y = c.per_wg > 1 ? 1 : cdiv(cols, kThreads);
  if (a->rows_type == MOE_OUT_FP32)
    launch_combine<true>(grid_y, (hipStream_t)stream, c);
  else
    launch_combine<false>(grid_y, (hipStream_t)stream, c);
  return launch_status();
}

moe_status_t moe_combine_grad(const moe_combine_grad_args_t* a, void* stream) {
  if (!a || a->M < 0 || a->R < 0 || a->top_k < 1 || a->H < 1 || !known(a->dy_type) || !known(a->rows_type) ||
      !known(a->drows_type))
    return MOE_ERR_INVALID_ARG;
  if (!routed(a->M, a->top_k) || a->R > kMaxPairs || a->H % 8) return MOE_ERR_UNSUPPORTED;
  if (a->M == 0) return MOE_OK;
  if (!a->positions || !aligned(a->positions, 4) || !aligned(a->weights, 4) || !aligned(a->dweights, 4))
    return MOE_ERR_INVALID_ARG;
  if ((!a->drows && !a->dweights) || (a->rows != nullptr) != (a->dweights != nullptr)) return MOE_ERR_INVALID_ARG;
  moe_status_t rc;
  if ((rc = check_matrix(a->dy, a->dy_stride, a->H, size_of(a->dy_type))) != MOE_OK) return rc;
  if (a->rows && (rc = check_matrix(a->rows, a->rows_stride, a->H, size_of(a->rows_type))) != MOE_OK) return rc;
  if (a->drows && (rc = check_matrix(a->drows, a->drows_stride, a->H, size_of(a->drows_type))) != MOE_OK) return rc;
  CombineGradArgs c = {};
  c.dy = (const uint8_t*)a->dy;
  c.dy_stride = a->dy_stride * size_of(a->dy_type);
  c.dy_f32 = a->dy_type == MOE_OUT_FP32;
  c.rows = (const uint8_t*)a->rows;
  c.rows_stride = a->rows ? a->rows_stride * size_of(a->rows_type) : 0;
  c.R = a->R;
  c.positions = a->positions;
  c.weights = a->weights;
  c.M = a->M;
  c.k = a->top_k;
  c.H = a->H;
  c.drows = (uint8_t*)a->drows;
  c.drows_stride = a->drows ? a->drows_stride * size_of(a->drows_type) : 0;
  c.drows_f32 = a->drows_type == MOE_OUT_FP32;
  c.dweights = a->dweights;
  const hipStream_t st = (hipStream_t)stream;
  const bool f32 = a->rows_type == MOE_OUT_FP32;
  if (a->top_k <= 2)
    f32 ? launch_combine_grad<true, 2>(st, c) : launch_combine_grad<false, 2>(st, c);
  else
    f32 ? launch_combine_grad<true, 8>(st, c) : launch_combine_grad<false, 8>(st, c);
  return launch_status();
}

moe_status_t moe_route_topk_grad(const int32_t* topk_ids, const float* topk_weights, const float* dweights, int32_t M,
                                 int32_t E, int32_t top_k, float* dlogits, void* stream) {
  if (M < 0 || E < 1 || top_k < 1) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || !routed(M, top_k)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!topk_ids || !topk_weights || !dweights || !dlogits || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) ||
      !aligned(dweights, 4) || !aligned(dlogits, 4))
    return MOE_ERR_INVALID_ARG;
  route_grad_kernel<<<grid_of(cdiv(M, 4)), kThreads, 0, (hipStream_t)stream>>>(topk_ids, topk_weights, dweights, M, E,
                                                                               top_k, dlogits);
  return launch_status();
}

}  // extern "C"
