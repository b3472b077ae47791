// Grouped expert products with bf16 weights, and their gradients, as LDS-tiled
// MFMA products (gfx950).
//
// One kernel computes out[q][p] = sum_c P[p][c] Q[q][c] on 256 x 256 tiles:
//   OP 0, product        q: grouped rows, p: weight rows n,    c: k
//   OP 1, input gradient q: grouped rows, p: weight columns k, c: n
//   OP 2, weight gradient q: n (dy),      p: k (in),           c: the expert's rows
// P is the MFMA's A operand, so a lane ends with four consecutive p of one q,
// and p is the contiguous direction of every result.
//
// An operand is "natural" when c is contiguous in memory (weights of OP 0, rows
// of OP 0 and 1) and "transposed" when its own index is (weights of OP 1, both
// operands of OP 2).  Natural halves (128 indices x 64 c) lie in LDS as
// 128 rows of 128 bytes and are read as 16-byte fragments; transposed halves
// (64 c x 128 indices) lie as 64 rows of 256 bytes, as they come from memory,
// and are transposed by the LDS transpose reads (ds_read_b64_tr_b16: of a 4 x
// 16 block of 2-byte elements, lane i of 16 gets column i), so no operand is
// ever laid out twice.  Chunk swizzles keep both kinds of reads free of bank
// conflicts.
//
// Eight waves, two per SIMD, each own 64 p x 32 q of each of the tile's four
// 128 x 128 quadrants (128 fp32 accumulators per lane).  A 64-deep step has
// four phases, one quadrant each, in the order (0,0) (0,1) (1,1) (1,0), so
// that each phase needs only one operand half that the phase before did not
// have: it is read from LDS a phase ahead.  Each phase issues the direct-to-LDS
// loads of the half whose slot the phase before freed, six phases ahead of its
// use: about 100 KB are in flight per CU.  One barrier per phase (512 MFMA
// cycles per SIMD).
#include <atomic>
#include <type_traits>

#include "grouped.h"
#include "mfma_tile.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kThreads = 512;
constexpr int kC = 64;            // contraction per step
constexpr int kHalf = 128;        // indices of an operand half
constexpr int kTile = 256;
constexpr int kPiece = kHalf * kC * 2;  // 16 KB: one half of one step
constexpr int kLds = 8 * kPiece;  // 2 stages x 2 operands x 2 halves
// offset of a lane that loads nothing: past every buffer (their sizes are at
// most this), and far enough below 2^32 that an in-row offset added to it does
// not wrap
constexpr unsigned kOob = 0xffc00000u;

struct TileArgs {
  int R, E, N, K;
  const int32_t* offsets;
  RowsArg q;         // OP 0, 1: the input rows; OP 2: dy
  RowsArg p;         // OP 2: the product's input rows
  const uint8_t* w;  // OP 0, 1
  RowsArg out;       // OP 0, 1
  uint8_t* dw;       // OP 2
};

// One tile: expert e with rows [lo, hi), first q (a grouped row, or n) and
// first p.
struct Tile {
  int e, lo, hi, q0, p0;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Bytes from the first of `rows` rows `ld` bytes apart to the end of the last
// one's `width` bytes.
__device__ __forceinline__ unsigned extent(int64_t rows, int64_t ld, int64_t width) {
  return rows > 0 && width > 0 ? (unsigned)((rows - 1) * ld + width) : 0u;
}

// 16 bytes per lane from base + off (zeros past `bytes`) to dst + 16 * lane.
// The compiler makes a transpose read from LDS wait for every tracked load into
// LDS, which would empty the queue of loads in each phase: kernels with
// transposed operands issue theirs as untracked instructions (they write no
// register) and wait for them by count themselves.
template <bool TRACKED>
__device__ __forceinline__ void load_lds(const uint8_t* base, unsigned bytes, lds_u8* dst, unsigned off) {
  if constexpr (TRACKED) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)bytes, kBufferWord3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (void __attribute__((address_space(3)))*)dst, 16, (int)off, 0, 0, 0);
  } else {
    // the no-op is the wait that a vector load needs after its descriptor or m0
    // was written, which the compiler does not see here
    const uint64_t p = (uint64_t)base;
    const u32x4 r = {(unsigned)uniform((int)(unsigned)p), (unsigned)uniform((int)((unsigned)(p >> 32) & 0xffffu)),
                     (unsigned)uniform((int)bytes), (unsigned)kBufferWord3};
    const unsigned at = (unsigned)uniform((int)(unsigned)(uintptr_t)dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(r)
                 : "memory");  // m0: nothing else in these kernels uses it
  }
}

// Start of a phase: this wave's loads but the last N have landed and its LDS
// reads are done; then the barrier.
template <int N>
__device__ __forceinline__ void phase_begin() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), for the compiler's own count of LDS reads
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// A transposed operand's loads: the base moves with the steps, or, with row
// ids, the lane offsets do.  Wave w loads rows 8w + 4q + lane/16 (q = 0, 1) of
// a step's 64, lane l the 16-byte chunk (l%16) ^ 4*(l/16) of the half's 256
// bytes (so that the four rows of a transpose read lie in different banks).
struct TransLoads {
  const uint8_t* base;
  int64_t ld;         // row bytes
  int64_t width;      // bytes from the tile's first index to a row's end
  unsigned bytes;     // buffer size of the current step
  u32x2 off;
  // row ids
  const int32_t* ids;
  int rows, div, first, end;  // matrix rows; grouped rows [first, end)

  __device__ __forceinline__ static int row(int wave, int lane) { return 8 * wave + (lane >> 4); }
  __device__ __forceinline__ static unsigned chunk(int lane) {
    return (unsigned)((lane & 15) ^ (4 * (lane >> 4))) << 4;
  }
  __device__ __forceinline__ void lane_offsets(int wave, int lane) {
    const unsigned o = (unsigned)(row(wave, lane) * ld) + chunk(lane);
    off = u32x2{o, o + (unsigned)(4 * ld)};
  }
  // The wave's eight ids of step s by scalar loads (vector loads would be
  // waited for together with the loads into LDS), then the lane's two.
  __device__ __forceinline__ void fetch_ids(const int32_t* from, int s, int wave, int lane, int* id0, int* id1) const {
    const __attribute__((address_space(4))) int32_t* p = (const __attribute__((address_space(4))) int32_t*)from;
    const int r = first + kC * s + 8 * wave, g = lane >> 4;
    const int last = end - 1;
    const int a0 = p[min(r, last)], a1 = p[min(r + 1, last)], a2 = p[min(r + 2, last)], a3 = p[min(r + 3, last)];
    const int b0 = p[min(r + 4, last)], b1 = p[min(r + 5, last)], b2 = p[min(r + 6, last)], b3 = p[min(r + 7, last)];
    *id0 = g < 2 ? (g == 0 ? a0 : a1) : (g == 2 ? a2 : a3);
    *id1 = g < 2 ? (g == 0 ? b0 : b1) : (g == 2 ? b2 : b3);
  }
  __device__ __forceinline__ unsigned id_offset(int f, bool in, int lane) const {
    const unsigned m = div == 1 ? (unsigned)f : (unsigned)f / (unsigned)div;
    return in && f >= 0 && m < (unsigned)rows ? m * (unsigned)ld + chunk(lane) : kOob;
  }
  // Step s (steps are taken in order, from 0): `count` rows in all.
  __device__ __forceinline__ void step(int s, int count, int wave, int lane) {
    const bool by_id = ids != nullptr;
    u32x2 o = off;
    unsigned n = bytes;
    const uint8_t* at = base;
    if (by_id) {
      int f0, f1;
      fetch_ids(ids, s, wave, lane, &f0, &f1);
      const int r = kC * s + row(wave, lane);
      o = u32x2{id_offset(f0, r < count, lane), id_offset(f1, r + 4 < count, lane)};
    } else {
      if (s) at += kC * ld;
      n = extent(min(kC, count - kC * s), ld, width);
    }
    off = o;
    base = at;
    bytes = n;
  }
  __device__ __forceinline__ void issue(lds_u8* dst, int h) const {
    load_lds<false>(base, bytes, dst, off[0] + h * (kHalf * 2));
    load_lds<false>(base, bytes, dst + 1024, off[1] + h * (kHalf * 2));
  }
};

// Issue order of a phase: its MFMAs with the NDS fragment reads of the next
// phase spread between the first six of them and the NVM loads after the third
// and the last ones.  Reads or loads issued ahead of the MFMAs leave the matrix
// pipe idle while the LDS takes them from eight waves at once.
template <int NMF, int NDS, int NVM, int ID, int I = 0>
__device__ __forceinline__ void interleave() {
  if constexpr (I < NMF) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, ID);  // one MFMA
    constexpr int kOver = NMF * 3 / 4;
    if constexpr (I < kOver) {
      constexpr int n = NDS * (I + 1) / kOver - NDS * I / kOver;
      if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x100, n, ID);  // LDS reads
    }
    if constexpr (I >= kOver) {
      constexpr int v = NVM * (I + 1 - kOver) / (NMF - kOver) - NVM * (I - kOver) / (NMF - kOver);
      if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x020, v, ID);  // direct-to-LDS loads
    }
    interleave<NMF, NDS, NVM, ID, I + 1>();
  }
}

template <int OP, bool F32, bool ACC, bool HALF>
__device__ __forceinline__ void tile_product(const TileArgs& a, const Tile t, lds_u8* smem) {
  constexpr bool kTransP = OP != 0, kTransQ = OP == 2;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int wr = wave >> 2, wc = wave & 3;
  const int len = OP == 0 ? a.K : (OP == 1 ? a.N : t.hi - t.lo);  // contraction
  const int nk = (len + kC - 1) / kC;
  const int width = OP == 0 ? a.N : a.K;                           // of p

  // ---- loads.  Natural: wave w loads rows 16w + 8q + lane/8 (q = 0, 1), lane l
  // the logical chunk (l%8) ^ pf_mix(row) = (l%8) ^ (l/8) ^ q.
  const int nrow = 16 * wave + (lane >> 3);
  const int nchunk = (lane & 7) ^ (lane >> 3);
  const uint8_t* pbase = nullptr;
  unsigned pbytes = 0, poff[2];
  TransLoads tp, tq;
  if constexpr (!kTransP) {
    pbase = a.w + ((int64_t)t.e * a.N + t.p0) * a.K * 2;
    pbytes = extent(min(kTile, a.N - t.p0), (int64_t)a.K * 2, (int64_t)a.K * 2);
#pragma unroll
    for (int q = 0; q < 2; ++q) poff[q] = (unsigned)((nrow + 8 * q) * a.K * 2 + ((nchunk ^ q) << 4));
  } else if constexpr (OP == 1) {
    tp.ids = nullptr;
    tp.ld = (int64_t)a.K * 2;
    tp.width = (int64_t)(a.K - t.p0) * 2;
    tp.base = a.w + ((int64_t)t.e * a.N * a.K + t.p0) * 2;
    tp.lane_offsets(wave, lane);
  }
  auto rows_loads = [&](TransLoads& l, const RowsArg& r, int w, int x0) {  // OP 2
    l.ids = r.ids;
    l.ld = r.stride * 2;
    l.width = (int64_t)(w - x0) * 2;
    l.rows = r.rows;
    l.div = r.div;
    l.first = t.lo;
    l.end = t.hi;
    if (r.ids) {
      l.base = r.p + (int64_t)x0 * 2;
      l.bytes = extent(r.rows, l.ld, l.width);
    } else {
      l.base = r.p + t.lo * l.ld + (int64_t)x0 * 2;
      l.lane_offsets(wave, lane);
    }
  };
  const uint8_t* qbase = nullptr;
  unsigned qoff[2][2];
  if constexpr (kTransQ) {
    rows_loads(tp, a.p, a.K, t.p0);
    rows_loads(tq, a.q, a.N, t.q0);
  } else {
    qbase = a.q.ids ? a.q.p : a.q.p + t.q0 * a.q.stride * 2;
#pragma unroll
    for (int h = 0; h < (HALF ? 1 : 2); ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = kHalf * h + nrow + 8 * q;
        const int m = t.q0 + i < t.hi ? (a.q.ids ? row_of(a.q, t.q0 + i) : i) : -1;
        qoff[h][q] = m >= 0 ? (unsigned)m * (unsigned)(a.q.stride * 2) + ((nchunk ^ q) << 4) : kOob;
      }
  }
  auto p_slot = [&](int h, int b) { return smem + (2 * h + b) * kPiece; };
  auto q_slot = [&](int h, int b) { return smem + (4 + 2 * h + b) * kPiece; };
  auto step_p = [&](int s) {
    if constexpr (kTransP) tp.step(s, len, wave, lane);
  };
  auto step_q = [&](int s) {
    if constexpr (kTransQ) tq.step(s, len, wave, lane);
  };
  // half h of step s (b = s & 1); a natural chunk at or past the contraction's
  // end loads nothing (zeros)
  auto issue_p = [&](int h, int s, int b) {
    lds_u8* dst = p_slot(h, b) + wave * 2048;
    if constexpr (kTransP) {
      tp.issue(dst, h);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const unsigned off = poff[q] + (unsigned)(h * kHalf * a.K * 2 + s * (kC * 2));
        load_lds<true>(pbase, pbytes, dst + q * 1024, ((nchunk ^ q) << 3) < len - kC * s ? off : kOob);
      }
    }
  };
  auto issue_q = [&](int h, int s, int b) {
    lds_u8* dst = q_slot(h, b) + wave * 2048;
    if constexpr (kTransQ) {
      tq.issue(dst, h);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        load_lds<!kTransP>(qbase, kOob, dst + q * 1024,
                 ((nchunk ^ q) << 3) < len - kC * s ? qoff[h][q] + (unsigned)(s * (kC * 2)) : kOob);
    }
  };

  // ---- fragments: index base + 32*tile + lane%32, c = 16*kk + 8*(lane/32)..+7
  const int fr = lane & 31, hl = lane >> 5;
  auto trans_at = [&](int idx0) {
    const int r = 8 * hl + ((lane & 15) >> 2);  // its row of the step's 64, at kk = 0
    const int chunk = idx0 / 8 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    return r * 256 + ((chunk ^ (4 * (r & 3))) << 4) + 8 * (lane & 1);
  };
  // address at kk = 0 (natural: kk k flips bits 5 and 6 of it; transposed: kk
  // is a constant offset, tile 1 flips bit 6)
  int pa = kTransP ? trans_at(64 * wr) : (64 * wr + fr) * 128 + ((hl ^ pf_mix(fr)) << 4);
  int qa = kTransQ ? trans_at(32 * wc) : (32 * wc + fr) * 128 + ((hl ^ pf_mix(fr)) << 4);
  auto tr_frag = [&](const lds_u8* p) {  // rows r..r+3 and r+4..r+7 of one index each
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 256));
    const u32x2 l = __builtin_bit_cast(u32x2, lo), g = __builtin_bit_cast(u32x2, hi);
    return u32x4{l[0], l[1], g[0], g[1]};
  };
  // the empty asm keeps the compiler from holding every flipped address in a
  // register of its own across the loop
  auto read_p = [&](u32x4 (&f)[2][4], int h, int b) {
    const lds_u8* s = p_slot(h, b);
    asm volatile("" : "+v"(pa));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        f[i][kk] = kTransP ? tr_frag(s + (pa ^ (64 * i)) + kk * 4096) : *(const lds_u32x4*)(s + (pa ^ (32 * kk)) + i * 4096);
  };
  auto read_q = [&](u32x4 (&f)[4], int h, int b) {
    const lds_u8* s = q_slot(h, b);
    asm volatile("" : "+v"(qa));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      f[kk] = kTransQ ? tr_frag(s + qa + kk * 4096) : *(const lds_u32x4*)(s + (qa ^ (32 * kk)));
  };

  f32x16 acc[2][HALF ? 1 : 2][2];  // [P half][Q half][tile]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < (HALF ? 1 : 2); ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][k][v] = 0.0f;
  constexpr int kReadsP = kTransP ? 16 : 8, kReadsQ = kTransQ ? 8 : 4;  // LDS reads of a half
  u32x4 A0[2][4], A1[2][4], F0[4], F1[4];
  auto mma = [&](f32x16 (&c)[2], const u32x4 (&p)[2][4], const u32x4 (&q)[4]) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 2; ++i) c[i] = mfma32_bf16(p[i][kk], q[kk], c[i]);
  };

  if (nk > 0) {
    if constexpr (!HALF) {
      // A phase at time t waits until at most the loads of the last six phases
      // are outstanding: those it is about to read were issued seven phases ago.
      auto begin = [] { phase_begin<12>(); };
      auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
      step_p(0);
      issue_p(0, 0, 0);
      step_q(0);
      issue_q(0, 0, 0);
      issue_q(1, 0, 0);
      issue_p(1, 0, 0);
      step_p(1);
      issue_p(0, 1, 1);
      step_q(1);
      issue_q(0, 1, 1);
      issue_q(1, 1, 1);
      issue_p(1, 1, 1);
      begin();
      read_p(A0, 0, 0);
      read_q(F0, 0, 0);
      ring_barrier();
      step_p(2);
      issue_p(0, 2, 0);
      // X holds Q half 0 of the step on entry; Y takes half 1, then half 0 of the next step
      auto step = [&](int s, auto bt, u32x4 (&X)[4], u32x4 (&Y)[4]) {
        constexpr int b = decltype(bt)::value;
        begin();
        fence();
        read_q(Y, 1, b);
        step_q(s + 2);
        issue_q(0, s + 2, b);
        mma(acc[0][0], A0, X);
        interleave<8, kReadsQ, 2, 4 * b>();
        fence();
        begin();
        fence();
        read_p(A1, 1, b);
        issue_q(1, s + 2, b);
        mma(acc[0][HALF ? 0 : 1], A0, Y);
        interleave<8, kReadsP, 2, 4 * b + 1>();
        fence();
        begin();
        fence();
        read_p(A0, 0, b ^ 1);
        issue_p(1, s + 2, b);
        mma(acc[1][HALF ? 0 : 1], A1, Y);
        interleave<8, kReadsP, 2, 4 * b + 2>();
        fence();
        begin();
        fence();
        read_q(Y, 0, b ^ 1);
        step_p(s + 3);
        issue_p(0, s + 3, b ^ 1);
        mma(acc[1][0], A1, X);
        interleave<8, kReadsQ, 2, 4 * b + 3>();
        fence();
      };
      for (int s = 0; s < nk; s += 2) {
        step(s, std::integral_constant<int, 0>{}, F0, F1);
        if (s + 1 >= nk) break;
        step(s + 1, std::integral_constant<int, 1>{}, F1, F0);
      }
    } else {
      // At most 128 q: two phases per step, P half 1 is read in the first, P
      // half 0 and Q of the next step in the second.
      auto begin = [] { phase_begin<6>(); };
      auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
      step_p(0);
      issue_p(0, 0, 0);
      step_q(0);
      issue_q(0, 0, 0);
      issue_p(1, 0, 0);
      step_p(1);
      issue_p(0, 1, 1);
      step_q(1);
      issue_q(0, 1, 1);
      begin();
      read_p(A0, 0, 0);
      read_q(F0, 0, 0);
      ring_barrier();
      // the order of all later issues: P1(1), then P0(2) Q0(2), P1(2), ...
      issue_p(1, 1, 1);
      auto step = [&](int s, auto bt, u32x4 (&X)[4], u32x4 (&Y)[4]) {
        constexpr int b = decltype(bt)::value;
        begin();
        fence();
        read_p(A1, 1, b);
        step_p(s + 2);
        issue_p(0, s + 2, b);
        step_q(s + 2);
        issue_q(0, s + 2, b);
        mma(acc[0][0], A0, X);
        interleave<8, kReadsP, 4, 8 + 2 * b>();
        fence();
        begin();
        fence();
        read_p(A0, 0, b ^ 1);
        read_q(Y, 0, b ^ 1);
        issue_p(1, s + 2, b);
        mma(acc[1][0], A1, X);
        interleave<8, kReadsP + kReadsQ, 2, 9 + 2 * b>();
        fence();
      };
      for (int s = 0; s < nk; s += 2) {
        step(s, std::integral_constant<int, 0>{}, F0, F1);
        if (s + 1 >= nk) break;
        step(s + 1, std::integral_constant<int, 1>{}, F1, F0);
      }
    }
    phase_begin<0>();  // the loads past the last step (zeros) still write LDS
  }

  // ---- epilogue: each wave transposes its 64 p x 32 q of a quadrant through
  // its own LDS, so that a store writes whole 128-byte lines of a result row.
  const int rows = OP == 2 ? a.N - t.q0 : t.hi - t.q0;  // valid q
  lds_u8* ep = smem + wave * 8192;
  int el = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));  // the lane, again: nothing lives
  asm volatile("" : "+v"(el));                                                         // across the loop for this part
  const int ef = el & 31, eh = el >> 5;
#pragma unroll
  for (int j = 0; j < (HALF ? 1 : 2); ++j) {
    const int qb = kHalf * j + 32 * wc;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pb = t.p0 + kHalf * i + 64 * wr;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& c = acc[i][j][k];
          const f32x4 v = {c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
          if constexpr (F32)
            *(lds_f32x4*)(ep + ef * 256 + (((8 * k + 2 * g + eh) ^ (ef & 15)) << 4)) = v;
          else
            *(lds_u32x2*)(ep + ef * 128 + (((4 * k + g) ^ pf_mix(ef)) << 4) + 8 * eh) =
                u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
      constexpr int kLanes = F32 ? 16 : 8;   // lanes of a result row
      constexpr int kRows = 64 / kLanes;     // rows per store
      const int rl = el / kLanes, cl = el % kLanes;
      const int p = pb + cl * (F32 ? 4 : 8);
#pragma unroll
      for (int rr = 0; rr < 32 / kRows; ++rr) {
        const int x = kRows * rr + rl, q = qb + x;
        const u32x4 v = *(const lds_u32x4*)(ep + x * (F32 ? 256 : 128) + ((cl ^ (F32 ? x & 15 : pf_mix(x))) << 4));
        if (q >= rows || p >= width) continue;
        if constexpr (OP == 2) {
          u32x4* o = (u32x4*)(a.dw + (((int64_t)t.e * a.N + t.q0 + q) * a.K + p) * (F32 ? 4 : 2));
          if constexpr (ACC) {
            const f32x4 s = *(const f32x4*)o + __builtin_bit_cast(f32x4, v);
            *(f32x4*)o = s;
          } else {
            *o = v;
          }
        } else {
          const int m = row_of(a.out, t.q0 + q);
          if (m >= 0) *(u32x4*)(a.out.p + ((int64_t)m * a.out.stride + p) * (F32 ? 4 : 2)) = v;
        }
      }
    }
  }
}

// Row tile and p tile of grid position (XCD, index in XCD): row tiles are
// numbered expert by expert; an XCD takes an eighth of all tiles, in groups of
// four row tiles, p tiles outer, so that the ~32 workgroups that run together
// on an XCD share operands in its L2.
__device__ __forceinline__ bool map_tile(int NT, int PT, int* rt, int* pt) {
  const int T = NT * PT, per = (T + 7) >> 3, x = blockIdx.x & 7, j = blockIdx.x >> 3;
  const int L = x * per + j;
  if (j >= per || L >= T) return false;
  const int g = L / (4 * PT), r = L - g * 4 * PT, n = min(4, NT - 4 * g);
  *rt = 4 * g + r % n;
  *pt = r / n;
  return true;
}

template <int OP, bool F32>
__global__ __launch_bounds__(kThreads) void grouped_rows_kernel(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  // thread e: the row tiles of expert e, and their prefix sum
  __attribute__((address_space(3))) int* sc = (__attribute__((address_space(3))) int*)smem;
  const int tid = threadIdx.x, wave = tid >> 6;
  int lo = 0, hi = 0;
  if (tid < a.E) group_range(a.offsets, tid, a.R, &lo, &hi);
  const int nt = (hi - lo + kTile - 1) / kTile;
  const int incl = wave_incl_scan(nt);
  if ((tid & 63) == 63) sc[wave] = incl;
  __syncthreads();
  int before = incl - nt, NT = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int v = sc[w];
    before += w < wave ? v : 0;
    NT += v;
  }
  const int PT = ((OP == 0 ? a.N : a.K) + kTile - 1) / kTile;
  int rt, pt;
  if (!map_tile(uniform(NT), PT, &rt, &pt)) return;
  if (rt >= before && rt < before + nt) {
    sc[8] = tid;
    sc[9] = lo;
    sc[10] = hi;
    sc[11] = lo + (rt - before) * kTile;
  }
  __syncthreads();
  const Tile t = {uniform(sc[8]), uniform(sc[9]), uniform(sc[10]), uniform(sc[11]), pt * kTile};
  __syncthreads();
  if (t.hi - t.q0 <= kHalf)
    tile_product<OP, F32, false, true>(a, t, smem);
  else
    tile_product<OP, F32, false, false>(a, t, smem);
}

// Weight gradient: the tiles of an expert are split over the XCDs (experts
// differ in their contraction, so whole experts would not balance), each XCD
// taking a contiguous band; few tiles are dealt round robin.
template <bool F32, bool ACC>
__global__ __launch_bounds__(kThreads) void grouped_wgrad_kernel(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int QT = (a.N + kTile - 1) / kTile, PT = (a.K + kTile - 1) / kTile, T = QT * PT;
  const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
  int e, i;
  if (T >= 16) {
    const int per = (T + 7) >> 3;
    e = j / per;
    i = x * per + j % per;
  } else {
    e = (int)blockIdx.x / T;
    i = (int)blockIdx.x % T;
  }
  if (e >= a.E || i >= T) return;
  const int g = i / (4 * PT), r = i - g * 4 * PT, n = min(4, QT - 4 * g);
  Tile t = {e, 0, 0, (4 * g + r % n) * kTile, (r / n) * kTile};
  group_range(a.offsets, e, a.R, &t.lo, &t.hi);
  t.lo = uniform(t.lo);
  t.hi = uniform(t.hi);
  if (ACC && t.lo == t.hi) return;
  if (a.N - t.q0 <= kHalf)
    tile_product<2, F32, ACC, true>(a, t, (lds_u8*)smem_raw);
  else
    tile_product<2, F32, ACC, false>(a, t, (lds_u8*)smem_raw);
}

// Launch with kLds bytes of dynamic LDS; the kernel's ceiling is raised once
// per device.
template <typename Kernel>
bool launch(Kernel kernel, std::atomic<bool> (&lds_set)[64], int64_t grid, hipStream_t st, const TileArgs& a) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return false;
  if (dev >= 64 || !lds_set[dev].load(std::memory_order_acquire)) {
    if (hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds) != hipSuccess)
      return false;
    if (dev < 64) lds_set[dev].store(true, std::memory_order_release);
  }
  kernel<<<(unsigned)grid, kThreads, kLds, st>>>(a);
  return true;
}

template <int OP, bool F32>
bool launch_rows(int64_t grid, hipStream_t st, const TileArgs& a) {
  static std::atomic<bool> lds_set[64];
  return launch(grouped_rows_kernel<OP, F32>, lds_set, grid, st, a);
}

template <bool F32, bool ACC>
bool launch_weights(int64_t grid, hipStream_t st, const TileArgs& a) {
  static std::atomic<bool> lds_set[64];
  return launch(grouped_wgrad_kernel<F32, ACC>, lds_set, grid, st, a);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

bool launch_grouped_tile(bool dgrad, bool f32, hipStream_t st, const GroupedArgs& a) {
  TileArgs t = {};
  t.R = a.R;
  t.E = a.E;
  t.N = a.N;
  t.K = a.K;
  t.offsets = a.offsets;
  t.q = a.in;
  t.w = a.w;
  t.out = a.out;
  // row tiles: at most R/256 whole ones and one more per expert that holds rows
  const int64_t rows = a.R / kTile + (a.R < a.E ? a.R : a.E);
  const int64_t grid = 8 * cdiv(rows * cdiv(dgrad ? a.K : a.N, kTile), 8);
  if (dgrad) return f32 ? launch_rows<1, true>(grid, st, t) : launch_rows<1, false>(grid, st, t);
  return f32 ? launch_rows<0, true>(grid, st, t) : launch_rows<0, false>(grid, st, t);
}

bool launch_grouped_wgrad(bool f32, bool accumulate, hipStream_t st, const GroupedWgradArgs& a) {
  TileArgs t = {};
  t.R = a.R;
  t.E = a.E;
  t.N = a.N;
  t.K = a.K;
  t.offsets = a.offsets;
  t.q = a.dy;
  t.p = a.in;
  t.dw = a.dw;
  const int64_t tiles = cdiv(a.N, kTile) * cdiv(a.K, kTile);
  const int64_t grid = tiles >= 16 ? 8 * cdiv(tiles, 8) * a.E : 8 * cdiv(tiles * a.E, 8);
  if (f32) return accumulate ? launch_weights<true, true>(grid, st, t) : launch_weights<true, false>(grid, st, t);
  return launch_weights<false, false>(grid, st, t);
}

}  // namespace moe
