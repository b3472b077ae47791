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
//
// One persistent workgroup per CU walks the tiles, and its loads run on into
// the next tile: the queue stays full over a tile's epilogue, which transposes
// the results through LDS beside the ring.
//
// Rows of an expert past its last whole tile make a tile of 256 x 256 (more
// than 128 rows), 256 x 128 (more than 64) or several of 128 x 64, and each
// kind is run after the larger ones: the small ones are bound by the stream of
// the weights and fill the CUs that the large ones leave idle at the end.  Both
// together, 8 experts of about 1024 rows: product N 4096, K 14336 973 -> 816
// us, input gradient N 28672, K 4096 1966 -> 1709 us.  At most 64 rows in all
// that make few tiles have a kernel of their own (grouped_narrow_kernel below).
//
// Measured, 8 experts of 1024 rows, medians on two machines: product N 4096, K
// 14336 759 us (1.27 PFLOP/s; single launches from 720 to 844), N 28672, K 4096
// 1493 to 1508 us (1.28); its input gradient 1541 to 1549 us (1.24); weight
// gradient N 4096, K 14336 in fp32 1039 us (0.93), where 16 steps share an
// epilogue of 256 KB; with gathered rows each step also loads, divides and
// masks ids: 1069 us in place, 1184 with dy gathered, 1177 with `in`, 1296 with
// both (experts of about 1024 rows), and 1471 in place when it accumulates.  A
// library product of 8192 cubed takes 699 to 716 us (1.54 to 1.57 PFLOP/s).
// What bounds the steps is power: the first of these takes 566 us on zeros,
// and took 613 to 658 on random values without operand loads.  32 rows over
// 128 experts, N 1536, K 2048: 41 to 49 us by machine, bound by the weights in
// flight (4.5 TB/s over the experts used).
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
typedef __attribute__((address_space(4))) int32_t c_int32;  // read by scalar loads

constexpr int kThreads = 512;
constexpr int kC = 64;            // contraction per step
constexpr int kHalf = 128;        // indices of an operand half
constexpr int kTile = 256;
constexpr int kPiece = kHalf * kC * 2;  // 16 KB: one half of one step
constexpr int kRing = 8 * kPiece;       // 2 stages x 2 operands x 2 halves
// epilogue area of a wave: the weight gradient needs no table of tile counts
__host__ __device__ constexpr int epilogue_bytes(int op) { return op == 2 ? 4096 : 2048; }
constexpr int kTable = kRing + 8 * epilogue_bytes(0);  // tile counts of the experts
constexpr int lds_bytes(int op) {
  return op == 2 ? kRing + 8 * epilogue_bytes(2) : kTable + 2 * kMaxExperts * 4 + 64;
}
constexpr int kSlots = 32;              // most workgroups per XCD: one per CU
static_assert(lds_bytes(0) <= 160 * 1024 && lds_bytes(2) <= 160 * 1024, "LDS of one gfx950 CU");
// offset of a lane that loads nothing: past every buffer (their sizes are at
// most this), and far enough below 2^32 that an in-row offset added to it does
// not wrap
constexpr unsigned kOob = 0xffc00000u;
constexpr unsigned kMasked = kOob | 4;  // the same of a row without a place: offsets of others are multiples of 16

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

// Workgroups per XCD, the stride of a workgroup's items.
__device__ __forceinline__ int slots() { return (int)gridDim.x >> 3; }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The lane, made anew: what is derived from it is not held in registers across
// the loops around.
__device__ __forceinline__ int lane_now() {
  int l = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  asm volatile("" : "+v"(l));
  return l;
}

// Bytes from the first of `rows` rows `ld` bytes apart to the end of the last
// one's `width` bytes.
__device__ __forceinline__ unsigned extent(int64_t rows, int64_t ld, int64_t width) {
  return rows > 0 && width > 0 ? (unsigned)((rows - 1) * ld + width) : 0u;
}

#ifdef __OPTIMIZE__
constexpr bool kCountLoads = true;
#else  // an unoptimised build does not hold uniform values in scalar registers, which the instruction takes
constexpr bool kCountLoads = false;
#endif

// 16 bytes per lane from base + off (zeros past `bytes`) to dst + 16 * lane.
// The compiler makes a transpose read from LDS wait for every tracked load into
// LDS, which would empty the queue of loads in each phase: kernels with
// transposed operands issue theirs as untracked instructions (they write no
// register) and wait for them by count themselves.
template <bool TRACKED>
__device__ __forceinline__ void load_lds(const uint8_t* base, unsigned bytes, lds_u8* dst, unsigned off) {
  if constexpr (TRACKED || !kCountLoads) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (int)bytes, kBufferWord3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (void __attribute__((address_space(3)))*)dst, 16, (int)off, 0, 0, 0);
  } else {
    // the no-op is the wait that a vector load needs after its descriptor or m0
    // was written, which the compiler does not see here.  m0 is reserved: the
    // compiler keeps no value in it and does not take it as a clobber, but it
    // would not know that one it set for its own instruction is gone.  A kernel
    // has either these loads or its own, and a test of the assembly sees to it.
    const uint64_t p = (uint64_t)base;
    const u32x4 r = {(unsigned)uniform((int)(unsigned)p), (unsigned)uniform((int)((unsigned)(p >> 32) & 0xffffu)),
                     (unsigned)uniform((int)bytes), (unsigned)kBufferWord3};
    const unsigned at = (unsigned)uniform((int)(unsigned)(uintptr_t)dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(r)
                 : "memory");
  }
}

// Between a wave's LDS writes and its other lanes' reads of them: the hardware
// keeps a wave's LDS accesses in order, the compiler has to be told.
__device__ __forceinline__ void wave_exchange() {
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
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
template <bool IDS>
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
    const unsigned o = (unsigned)row(wave, lane) * (unsigned)ld + chunk(lane);
    off = u32x2{o, o + 4 * (unsigned)ld};
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
    return in && f >= 0 && m < (unsigned)rows ? m * (unsigned)ld + chunk(lane) : kMasked;
  }
  // Columns from x0 on of a rows operand, over the rows of tile t.
  __device__ __forceinline__ void rows_of(const RowsArg& r, int w, int x0, const Tile& t, int wave, int lane) {
    ids = IDS ? r.ids : nullptr;
    ld = r.stride * 2;
    width = (int64_t)(w - x0) * 2;
    rows = r.rows;
    div = r.div;
    first = t.lo;
    end = t.hi;
    base = r.p + (int64_t)x0 * 2 + (ids ? 0 : t.lo * ld);
    bytes = ids ? extent(rows, ld, width) : 0u;
    lane_offsets(wave, lane);
  }
  __device__ __forceinline__ void none() {
    ids = nullptr;
    bytes = 0;
  }
  // Step s (steps are taken in order, from 0): `count` rows in all, at least one.
  __device__ __forceinline__ void step(int s, int count, int wave, int lane) {
    if (IDS && ids) {
      int f0, f1;
      fetch_ids(ids, s, wave, lane, &f0, &f1);
      const int r = kC * s + row(wave, lane);
      off = u32x2{id_offset(f0, r < count, lane), id_offset(f1, r + 4 < count, lane)};
    } else {
      if (IDS) lane_offsets(wave, lane);  // the other operand's ids may have masked them
      base += s ? kC * ld : 0;
      const int left = min(kC, count - kC * s);
      bytes = left > 0 ? (unsigned)((left - 1) * ld + width) : 0u;
    }
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

template <int OP>
__device__ __forceinline__ int contraction(const TileArgs& a, const Tile& t) {
  return OP == 0 ? a.K : (OP == 1 ? a.N : t.hi - t.lo);
}
// Number of 64-deep steps of a tile.  The products' is even (a step past the
// end multiplies zeros), so that a step's stage is known to the compiler (1 %
// on long contractions); the weight gradient's may be odd (its contraction is an
// expert's rows: 8 experts of about 1024 3 %, 128 of about 64 10 % faster).
template <int OP>
__device__ __forceinline__ int steps_of(int len) {
  return OP == 2 ? (len + kC - 1) / kC : 2 * ((len + 2 * kC - 1) / (2 * kC));
}

// The loads of one workgroup's sequence of tiles, step by step.
template <int OP, bool HALF, bool IDS>
struct Loads {
  static constexpr bool kTransP = OP != 0, kTransQ = OP == 2;
  int s, nk, len;  // step of the current tile, its steps and its contraction
  const uint8_t* pbase;
  const uint8_t* qbase;
  unsigned pbytes;
  u32x2 poff;           // natural P: rows 16w + lane/8 and 8 more
  u32x2 qoff0, qoff1;   // natural Q: the same of half 0 and half 1
  TransLoads<OP == 2 && IDS> tp, tq;

  // Natural operands: wave w loads rows 16w + 8i + lane/8 (i = 0, 1) of a half,
  // lane l the logical chunk (l%8) ^ pf_mix(row) = (l%8) ^ (l/8) ^ i.
  __device__ __forceinline__ static int nrow(int wave, int lane) { return 16 * wave + (lane >> 3); }
  __device__ __forceinline__ static int nchunk(int lane) { return (lane & 7) ^ (lane >> 3); }

  __device__ __forceinline__ void init(const TileArgs& a, int wave, int lane) {
    if constexpr (!kTransP)
      poff = u32x2{(unsigned)(nrow(wave, lane) * a.K * 2 + (nchunk(lane) << 4)),
                   (unsigned)((nrow(wave, lane) + 8) * a.K * 2 + ((nchunk(lane) ^ 1) << 4))};
    if constexpr (OP == 1) {
      tp.ids = nullptr;
      tp.ld = (int64_t)a.K * 2;
      tp.lane_offsets(wave, lane);
    }
  }
  __device__ __forceinline__ unsigned row_offset(const TileArgs& a, const Tile& t, int i, int chunk) const {
    const int m = t.q0 + i < t.hi ? (a.q.ids ? row_of(a.q, t.q0 + i) : i) : -1;
    return m >= 0 ? (unsigned)m * (unsigned)(a.q.stride * 2) + (chunk << 4) : kOob;
  }
  // To the first step of a tile.
  __device__ __forceinline__ void tile(const TileArgs& a, const Tile& t, int wave) {
    const int lane = lane_now();
    len = contraction<OP>(a, t);
    nk = steps_of<OP>(len);
    s = 0;
    if constexpr (OP == 0) {
      pbase = a.w + ((int64_t)t.e * a.N + t.p0) * a.K * 2;
      pbytes = extent(min(kTile, a.N - t.p0), (int64_t)a.K * 2, (int64_t)a.K * 2);
    }
    if constexpr (OP == 1) {
      tp.width = (int64_t)(a.K - t.p0) * 2;
      tp.base = a.w + ((int64_t)t.e * a.N * a.K + t.p0) * 2;
    }
    if constexpr (!kTransQ) {
      qbase = a.q.ids ? a.q.p : a.q.p + t.q0 * a.q.stride * 2;
      const int r = nrow(wave, lane), c = nchunk(lane);
      qoff0 = u32x2{row_offset(a, t, r, c), row_offset(a, t, r + 8, c ^ 1)};
      if constexpr (!HALF) qoff1 = u32x2{row_offset(a, t, kHalf + r, c), row_offset(a, t, kHalf + r + 8, c ^ 1)};
    } else {
      tp.rows_of(a.p, a.K, t.p0, t, wave, lane);
      tq.rows_of(a.q, a.N, t.q0, t, wave, lane);
    }
    trans_step(wave, lane);
  }
  // The transposed operands to step s.  A row whose id masks it in one of the
  // weight gradient's operands is left out of the other too, where it may hold
  // an infinity or a NaN.
  __device__ __forceinline__ void trans_step(int wave, int lane) {
    if constexpr (kTransP) tp.step(s, len, wave, lane);
    if constexpr (kTransQ) tq.step(s, len, wave, lane);
    if constexpr (kTransQ && IDS) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool masked = tp.off[i] == kMasked || tq.off[i] == kMasked;
        tp.off[i] = masked ? kMasked : tp.off[i];
        tq.off[i] = masked ? kMasked : tq.off[i];
      }
    }
  }
  __device__ __forceinline__ void step(int wave) {  // to the next step of the tile
    const int lane = OP == 2 && IDS ? lane_now() : 0;
    ++s;
    trans_step(wave, lane);
  }
  __device__ __forceinline__ void end() {  // no more tiles: load nothing
    nk = 0x7fffffff;
    s = 0;
    len = 0;
    if constexpr (!kTransQ) qoff0 = qoff1 = u32x2{kOob, kOob};
    if constexpr (!kTransP) pbytes = 0;
    if constexpr (kTransP) tp.none();
    if constexpr (kTransQ) tq.none();
  }
  // Half h into its slot; a natural chunk at or past the contraction's end
  // loads nothing (zeros).
  __device__ __forceinline__ void issue_p(const TileArgs& a, lds_u8* dst, int h, int lane) const {
    if constexpr (kTransP) {
      tp.issue(dst, h);
    } else {
      const unsigned at = (unsigned)(h * kHalf * a.K * 2 + s * (kC * 2));
      load_lds<true>(pbase, pbytes, dst, nchunk(lane) << 3 < len - kC * s ? poff[0] + at : kOob);
      load_lds<true>(pbase, pbytes, dst + 1024, (nchunk(lane) ^ 1) << 3 < len - kC * s ? poff[1] + at : kOob);
    }
  }
  __device__ __forceinline__ void issue_q(lds_u8* dst, int h, int lane) const {
    if constexpr (kTransQ) {
      tq.issue(dst, h);
    } else {
      const u32x2 o = HALF || h == 0 ? qoff0 : qoff1;
      const unsigned at = (unsigned)(s * (kC * 2));
      load_lds<!kTransP>(qbase, kOob, dst, nchunk(lane) << 3 < len - kC * s ? o[0] + at : kOob);
      load_lds<!kTransP>(qbase, kOob, dst + 1024, (nchunk(lane) ^ 1) << 3 < len - kC * s ? o[1] + at : kOob);
    }
  }
};

// LDS address of a lane's transpose read of 32 indices from idx0 on, at kk = 0.
__device__ __forceinline__ int trans_at(int idx0, int lane) {
  const int r = 8 * (lane >> 5) + ((lane & 15) >> 2);  // its row of the step's 64
  const int chunk = idx0 / 8 + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  return r * 256 + ((chunk ^ (4 * (r & 3))) << 4) + 8 * (lane & 1);
}
__device__ __forceinline__ int natural_at(int idx0, int lane) {
  return (idx0 + (lane & 31)) * 128 + (((lane >> 5) ^ pf_mix(lane & 31)) << 4);
}
// Eight c of one index per lane: rows r..r+3 and r+4..r+7 of the transposed half.
__device__ __forceinline__ u32x4 tr_frag(const lds_u8* p) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 256));
  const u32x2 l = __builtin_bit_cast(u32x2, lo), g = __builtin_bit_cast(u32x2, hi);
  return u32x4{l[0], l[1], g[0], g[1]};
}

// Where a tile's result row q goes: nullptr for a row that is not written.
template <int OP, bool F32>
__device__ __forceinline__ uint8_t* out_row(const TileArgs& a, const Tile& t, int q) {
  constexpr int kEsz = F32 ? 4 : 2;
  if constexpr (OP == 2) {
    if (t.q0 + q >= a.N) return nullptr;
    return a.dw + ((int64_t)t.e * a.N + t.q0 + q) * a.K * kEsz;
  } else {
    const int m = t.q0 + q < t.hi ? row_of(a.out, t.q0 + q) : -1;
    return m < 0 ? nullptr : a.out.p + (int64_t)m * a.out.stride * kEsz;
  }
}

// All tiles of one kind (HALF: at most 128 q) of a workgroup: items(u, &tile)
// moves u to the next item from u on, or returns false.
template <int OP, bool F32, bool ACC, bool HALF, bool IDS, typename Items>
__device__ __forceinline__ void run_tiles(const TileArgs& a, lds_u8* smem, int& u, const Items& items) {
  constexpr bool kTransP = OP != 0, kTransQ = OP == 2;
  constexpr int kReadsP = kTransP ? 16 : 8, kReadsQ = kTransQ ? 8 : 4;  // LDS reads of a half
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wr = wave >> 2, wc = wave & 3;
  const int width = OP == 0 ? a.N : a.K;  // of p
  Tile t;
  if (!items(u, &t)) return;
  Loads<OP, HALF, IDS> L;
  Tile lt = t;  // the loads' tile
  int lu = u;
  L.init(a, wave, lane);
  auto load_tile = [&](bool have) {
    if (have)
      L.tile(a, lt, wave);
    else
      L.end();
  };
  // After a step: to the next tile where it was the last.  L.step itself is
  // scheduled among the MFMAs; past the last step it changes nothing that the
  // next tile keeps.
  auto load_next = [&] {
    if (L.s >= L.nk) {
      lu += slots();
      load_tile(items(lu, &lt));
    }
  };
  // Stage b (0, 1) of the ring: weight gradients add it to the addresses, as
  // a tile may have an odd number of steps (b: 0 this step's, 1 the next one's).
  constexpr bool kOdd = OP == 2;
  int stage = wave * 2048;
  auto dst = [&](int b) { return smem + (kOdd ? stage ^ (b * kPiece) : wave * 2048 + b * kPiece); };
  auto issue_p = [&](int h, int b) { L.issue_p(a, dst(b) + 2 * h * kPiece, h, lane); };
  auto issue_q = [&](int h, int b) { L.issue_q(dst(b) + (4 + 2 * h) * kPiece, h, lane); };

  // Fragments: index base + 32*tile + lane%32, c = 16*kk + 8*(lane/32)..+7.
  // Natural: kk flips bits 5 and 6 of the address; transposed: kk is a constant
  // offset, tile 1 flips bit 6.  The empty asm keeps the compiler from holding
  // every flipped address in a register of its own across the loop.
  int pa = kTransP ? trans_at(64 * wr, lane) : natural_at(64 * wr, lane);
  int qa = kTransQ ? trans_at(32 * wc, lane) : natural_at(32 * wc, lane);
  auto read_p = [&](u32x4 (&f)[2][4], int h, int b) {
    const lds_u8* s = smem + (2 * h + (kOdd ? 0 : b)) * kPiece;
    const int o = kOdd ? b * kPiece : 0;
    asm volatile("" : "+v"(pa));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        f[i][kk] = kTransP ? tr_frag(s + (pa ^ (64 * i + o)) + kk * 4096)
                           : *(const lds_u32x4*)(s + (pa ^ (32 * kk)) + i * 4096);
  };
  auto read_q = [&](u32x4 (&f)[4], int h, int b) {
    const lds_u8* s = smem + (4 + 2 * h + (kOdd ? 0 : b)) * kPiece;
    const int o = kOdd ? b * kPiece : 0;
    asm volatile("" : "+v"(qa));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      f[kk] = kTransQ ? tr_frag(s + (qa ^ o) + kk * 4096) : *(const lds_u32x4*)(s + (qa ^ (32 * kk)));
  };

  f32x16 acc[2][HALF ? 1 : 2][2];  // [P half][Q half][tile]
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < (HALF ? 1 : 2); ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][k][v] = 0.0f;
  };
  u32x4 A0[2][4], A1[2][4], F0[4], F1[4];
  auto mma = [&](f32x16 (&c)[2], const u32x4 (&p)[2][4], const u32x4 (&q)[4]) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 2; ++i) c[i] = mfma32_bf16(p[i][kk], q[kk], c[i]);
  };
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  // A phase waits until at most the loads of the last six phases (HALF: the
  // last three halves) are outstanding: those it is about to read were issued
  // before.
  constexpr int kAhead = HALF ? 6 : 12;
  auto begin = [] { phase_begin<kAhead>(); };

  // The order of all issues, by step: P0, Q0, Q1, P1 (HALF: P0, Q0, P1).
  load_tile(true);
  issue_p(0, 0);
  issue_q(0, 0);
  if constexpr (!HALF) issue_q(1, 0);
  issue_p(1, 0);
  L.step(wave);
  load_next();
  issue_p(0, 1);
  issue_q(0, 1);
  if constexpr (!HALF) issue_q(1, 1);
  if constexpr (!HALF) {
    issue_p(1, 1);
    L.step(wave);
    load_next();
  }
  begin();
  read_p(A0, 0, 0);
  read_q(F0, 0, 0);
  ring_barrier();
  if constexpr (HALF) {
    issue_p(1, 1);
    L.step(wave);
  } else {
    issue_p(0, 0);
  }
  // X holds Q half 0 of the step on entry; Y takes half 1, then half 0 of the next step
  auto step = [&](auto at, u32x4 (&X)[4], u32x4 (&Y)[4]) {
    constexpr int id = 4 * decltype(at)::value, b = kOdd ? 0 : decltype(at)::value;
    if constexpr (!HALF) {
      begin();
      fence();
      read_q(Y, 1, b);
      issue_q(0, b);
      mma(acc[0][0], A0, X);
      interleave<8, kReadsQ, 2, id>();
      fence();
      begin();
      fence();
      read_p(A1, 1, b);
      issue_q(1, b);
      mma(acc[0][HALF ? 0 : 1], A0, Y);
      interleave<8, kReadsP, 2, id + 1>();
      fence();
      begin();
      fence();
      read_p(A0, 0, b ^ 1);
      issue_p(1, b);
      L.step(wave);
      mma(acc[1][HALF ? 0 : 1], A1, Y);
      interleave<8, kReadsP, 2, id + 2>();
      fence();
      load_next();
      begin();
      fence();
      read_q(Y, 0, b ^ 1);
      issue_p(0, b ^ 1);
      mma(acc[1][0], A1, X);
      interleave<8, kReadsQ, 2, id + 3>();
      fence();
    } else {
      load_next();
      begin();
      fence();
      read_p(A1, 1, b);
      issue_p(0, b);
      issue_q(0, b);
      mma(acc[0][0], A0, X);
      interleave<8, kReadsP, 4, id>();
      fence();
      begin();
      fence();
      read_p(A0, 0, b ^ 1);
      read_q(Y, 0, b ^ 1);
      issue_p(1, b);
      L.step(wave);
      mma(acc[1][0], A1, X);
      interleave<8, kReadsP + kReadsQ, 2, id + 1>();
      fence();
    }
    if constexpr (kOdd) {
      stage ^= kPiece;
      pa ^= kPiece;
      qa ^= kPiece;
    }
  };

  while (true) {
    const int nk = steps_of<OP>(contraction<OP>(a, t));
    clear();
    for (int s = 1; s < nk; s += 2) {
      step(std::integral_constant<int, 0>{}, F0, F1);
      step(std::integral_constant<int, 1>{}, F1, F0);
    }
    if constexpr (kOdd) {
      if (nk & 1) {
        step(std::integral_constant<int, 2>{}, F0, F1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) F0[kk] = F1[kk];
      }
    }
    // Epilogue: each wave transposes its 64 p x 32 q of a quadrant through its
    // own LDS beside the ring, kQ result rows at a time, so that a store writes
    // whole 128-byte lines of a row.
    const int el = lane_now(), ef = el & 31, eh = el >> 5;
    constexpr int kArea = epilogue_bytes(OP);
    constexpr int kRowB = F32 ? 256 : 128;  // bytes of a quadrant's result row
    constexpr int kQ = kArea / kRowB;
    constexpr int kLanes = kRowB / 16;      // lanes of a result row
    constexpr int kX = kLanes - 1;          // chunk swizzle
    lds_u8* ep = smem + kRing + wave * kArea;
    const int rl = el / kLanes, cl = el % kLanes;
#pragma unroll
    for (int j = 0; j < (HALF ? 1 : 2); ++j)
#pragma unroll
      for (int z = 0; z < 32 / kQ; ++z)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (kQ == 32 || ef / kQ == z) {
            const int x = ef % kQ;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const f32x16& c = acc[i][j][k];
                const f32x4 v = {c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
                if constexpr (F32)
                  *(lds_f32x4*)(ep + x * kRowB + (((8 * k + 2 * g + eh) ^ (x & kX)) << 4)) = v;
                else
                  *(lds_u32x2*)(ep + x * kRowB + (((4 * k + g) ^ (x & kX)) << 4) + 8 * eh) =
                      u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
              }
          }
          wave_exchange();
          const int p = t.p0 + kHalf * i + 64 * wr + cl * (F32 ? 4 : 8);
#pragma unroll
          for (int rr = 0; rr < kQ * kLanes / 64; ++rr) {
            const int x = (64 / kLanes) * rr + rl;
            const u32x4 v = *(const lds_u32x4*)(ep + x * kRowB + ((cl ^ (x & kX)) << 4));
            uint8_t* o = out_row<OP, F32>(a, t, kHalf * j + 32 * wc + kQ * z + x);
            if (o && p < width) {
              u32x4* at = (u32x4*)(o + (int64_t)p * (F32 ? 4 : 2));
              if constexpr (ACC)
                *(f32x4*)at = *(const f32x4*)at + __builtin_bit_cast(f32x4, v);
              else
                *at = v;
            }
          }
          wave_exchange();
        }
    u += slots();
    if (!items(u, &t)) break;
  }
  phase_begin<0>();  // the loads past the last tile (zeros) still write LDS
}

// Tiles of at most 64 q: 128 p x 64 q, five steps of 24 KB in a ring, four of
// them in flight.  Wave w owns 32 p (w%4) x 32 q (w/4).
constexpr int kSmallQ = 64;
constexpr int kSmallStages = 5;
constexpr int kSmallStage = kPiece + kSmallQ * kC * 2;
static_assert(kSmallStages * kSmallStage <= kRing, "the small tiles' ring");

template <int OP, bool F32, typename Items>
__device__ __forceinline__ void run_small(const TileArgs& a, lds_u8* smem, int& u, const Items& items) {
  constexpr bool kTransP = OP != 0;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wp = wave & 3, wq = wave >> 2;
  const int width = OP == 0 ? a.N : a.K, len = OP == 0 ? a.K : a.N;
  const int nk = (len + kC - 1) / kC;
  Loads<OP, true, false> L;
  L.init(a, wave, lane);
  const int pa = kTransP ? trans_at(32 * wp, lane) : natural_at(32 * wp, lane);
  const int qa = natural_at(32 * wq, lane);
  const int qc = (lane & 7) ^ (lane >> 3) ^ (wave & 1);  // chunk of Q row 8w + lane/8
  for (Tile t; items(u, &t); u += slots()) {
    L.tile(a, t, wave);
    if constexpr (OP == 0) L.pbytes = extent(min(kHalf, a.N - t.p0), (int64_t)a.K * 2, (int64_t)a.K * 2);
    const unsigned qoff = L.row_offset(a, t, 8 * wave + (lane >> 3), qc);
    auto issue = [&](int stage) {  // step L.s, then on to the next
      lds_u8* dst = smem + stage * kSmallStage;
      L.issue_p(a, dst + wave * 2048, 0, lane);
      load_lds<!kTransP>(L.qbase, kOob, dst + kPiece + wave * 1024,
                         qc << 3 < len - kC * L.s ? qoff + (unsigned)(L.s * (kC * 2)) : kOob);
      L.step(wave);
    };
    f32x16 acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
    for (int i = 0; i < kSmallStages - 1; ++i) issue(i);
    int stage = 0;
    for (int s = 0; s < nk; ++s) {
      phase_begin<3 * (kSmallStages - 2)>();
      const lds_u8* at = smem + stage * kSmallStage;
      u32x4 p[4], q[4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        p[kk] = kTransP ? tr_frag(at + pa + kk * 4096) : *(const lds_u32x4*)(at + (pa ^ (32 * kk)));
        q[kk] = *(const lds_u32x4*)(at + kPiece + (qa ^ (32 * kk)));
      }
      issue(stage == 0 ? kSmallStages - 1 : stage - 1);  // the slot whose reads the barrier ended
      stage = stage == kSmallStages - 1 ? 0 : stage + 1;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) acc = mfma32_bf16(p[kk], q[kk], acc);
    }
    phase_begin<0>();  // the loads past the last step (zeros)
    uint8_t* o = out_row<OP, F32>(a, t, 32 * wq + (lane & 31));
    if (o)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int p = t.p0 + 32 * wp + 8 * g + 4 * (lane >> 5);
        if (p >= width) continue;
        const f32x4 v = {acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
        if constexpr (F32)
          *(f32x4*)(o + (int64_t)p * 4) = v;
        else
          *(u32x2*)(o + (int64_t)p * 2) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
  }
}

// Tiles of an expert with n rows: whole ones, and the kind of the rest.
__device__ __forceinline__ int full_tiles(int n) { return n / kTile + (n % kTile > kHalf); }
__device__ __forceinline__ bool half_tile(int n) { return n % kTile > kSmallQ && n % kTile <= kHalf; }
__device__ __forceinline__ bool small_tile(int n) { return n % kTile > 0 && n % kTile <= kSmallQ; }

typedef __attribute__((address_space(3))) int lds_int;

// Number of the E inclusive prefix sums tab[0..E) (shifted and masked) that are
// at most v: the expert of item v.
__device__ __forceinline__ int expert_of(const lds_int* tab, int E, int shift, int mask, int v, int lane) {
  int e = 0;
  for (int i = 0; i < E; i += 64) {
    const bool le = i + lane < E && ((tab[i + lane] >> shift) & mask) <= v;
    e += __popcll(__ballot(le));
  }
  return uniform(e);
}

// Product and input gradient.  Row tiles are numbered expert by expert, each
// kind on its own; an XCD takes an eighth of a kind's tiles, whole ones and
// halves in groups of four row tiles with p tiles outer, so that the ~32
// workgroups that run together on an XCD share operands in its L2.
template <int OP, bool F32>
__global__ __launch_bounds__(kThreads) void grouped_rows_kernel(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  lds_int* full = (lds_int*)(smem + kTable);  // [E] inclusive sums of whole tiles
  lds_int* rest = full + kMaxExperts;         // [E] of half tiles, and << 16 of small ones
  lds_int* part = rest + kMaxExperts;
  {
    const int tid = threadIdx.x, wave = tid >> 6;
    int lo = 0, hi = 0;
    if (tid < a.E) group_range(a.offsets, tid, a.R, &lo, &hi);
    const int f = full_tiles(hi - lo), r = (half_tile(hi - lo) ? 1 : 0) + (small_tile(hi - lo) ? 1 << 16 : 0);
    int fi = wave_incl_scan(f), ri = wave_incl_scan(r);
    if ((tid & 63) == 63) {
      part[wave] = fi;
      part[8 + wave] = ri;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      fi += w < wave ? part[w] : 0;
      ri += w < wave ? part[8 + w] : 0;
    }
    full[tid] = fi;
    rest[tid] = ri;
    __syncthreads();
  }
  // offsets that decrease could make experts overlap: no more tiles than R rows have
  const int NF = min(uniform(full[a.E - 1]), a.R / kTile + a.E);
  const int NR = uniform(rest[a.E - 1]), NH = NR & 0xffff, NS = NR >> 16;
  const int width = OP == 0 ? a.N : a.K;
  const int PT = (width + kTile - 1) / kTile, PS = (width + kHalf - 1) / kHalf;
  const int x = blockIdx.x & 7;
  const int lane = threadIdx.x & 63;
  // items of this XCD: [0, nf) whole tiles, [nf, nf + nh) halves, then small ones
  const int nf = (NF * PT + 7) >> 3, nh = (NH * PT + 7) >> 3, ns = (NS * PS + 7) >> 3;
  const c_int32* offsets = (const c_int32*)a.offsets;
  auto range = [&](Tile* t) {  // of expert t->e, by scalar loads
    const int lo = min(max(offsets[t->e], 0), a.R);
    t->lo = lo;
    t->hi = min(max(offsets[t->e + 1], lo), a.R);
  };
  auto raster = [&](int n, int rows, int j, int* rt, int* pt) {  // item j of this XCD's n
    const int i = x * n + j;
    if (j >= n || i >= rows * PT) return false;
    const int g = i / (4 * PT), r = i - g * 4 * PT, m = min(4, rows - 4 * g);
    *rt = 4 * g + r % m;
    *pt = r / m;
    return true;
  };
  auto whole = [&](int& u, Tile* t) {
    int rt, pt;
    if (u >= nf || !raster(nf, NF, u, &rt, &pt)) return false;
    t->e = expert_of(full, a.E, 0, -1, rt, lane);
    range(t);
    t->q0 = t->lo + (rt - (uniform(full[t->e]) - full_tiles(t->hi - t->lo))) * kTile;
    t->p0 = pt * kTile;
    return true;
  };
  auto half = [&](int& u, Tile* t) {
    int rt, pt;
    if (u >= nf + nh || !raster(nh, NH, u - nf, &rt, &pt)) return false;
    t->e = expert_of(rest, a.E, 0, 0xffff, rt, lane);
    range(t);
    t->q0 = t->lo + full_tiles(t->hi - t->lo) * kTile;
    t->p0 = pt * kTile;
    return true;
  };
  auto small = [&](int& u, Tile* t) {
    const int j = u - nf - nh, i = x * ns + j;
    if (j >= ns || i >= NS * PS) return false;
    t->e = expert_of(rest, a.E, 16, 0xffff, i / PS, lane);
    range(t);
    t->q0 = t->lo + full_tiles(t->hi - t->lo) * kTile;
    t->p0 = i % PS * kHalf;
    return true;
  };
  int u = blockIdx.x >> 3;
  run_tiles<OP, F32, false, false, true>(a, smem, u, whole);
  while (u < nf) u += slots();  // an XCD's last items can be missing
  run_tiles<OP, F32, false, true, true>(a, smem, u, half);
  while (u < nf + nh) u += slots();
  run_small<OP, F32>(a, smem, u, small);
}

// Weight gradient: the tiles of an expert are split over the XCDs (experts
// differ in their contraction, so whole experts would not balance), each XCD
// taking a contiguous band; few tiles are dealt round robin.  Experts without
// rows have no tiles.
template <bool F32, bool ACC, bool IDS>
__global__ __launch_bounds__(kThreads) void grouped_wgrad_kernel(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  const bool last_half = a.N % kTile > 0 && a.N % kTile <= kHalf;  // the last q tile is a half
  const int QT = (a.N + kTile - 1) / kTile - last_half, PT = (a.K + kTile - 1) / kTile;
  const int x = blockIdx.x & 7;
  const c_int32* offsets = (const c_int32*)a.offsets;
  auto range = [&](Tile* t) {
    const int lo = min(max(offsets[t->e], 0), a.R);
    t->lo = lo;
    t->hi = min(max(offsets[t->e + 1], lo), a.R);
  };
  const int T = QT * PT, per = (T + 7) >> 3;
  const int nf = T >= 16 ? per * a.E : (T * a.E + 7) >> 3, nh = last_half ? (PT * a.E + 7) >> 3 : 0;
  auto whole = [&](int& u, Tile* t) {
    for (; u < nf; u += slots()) {
      const int e = T >= 16 ? u / per : (u * 8 + x) / max(T, 1);
      const int i = T >= 16 ? x * per + u % per : (u * 8 + x) % max(T, 1);
      if (i >= T || e >= a.E) continue;
      const int g = i / (4 * PT), r = i - g * 4 * PT, n = min(4, QT - 4 * g);
      t->e = e;
      t->q0 = (4 * g + r % n) * kTile;
      t->p0 = (r / n) * kTile;
      range(t);
      if (t->lo < t->hi) return true;
    }
    return false;
  };
  auto half = [&](int& u, Tile* t) {
    for (; u < nf + nh; u += slots()) {
      const int i = (u - nf) * 8 + x;
      if (i >= PT * a.E) return false;
      t->e = i / PT;
      t->q0 = QT * kTile;
      t->p0 = i % PT * kTile;
      range(t);
      if (t->lo < t->hi) return true;
    }
    return false;
  };
  int u = blockIdx.x >> 3;
  run_tiles<2, F32, ACC, false, IDS>(a, smem, u, whole);
  while (u < nf) u += slots();
  run_tiles<2, F32, ACC, true, IDS>(a, smem, u, half);
  // experts without rows: zeros, or nothing to add
  if constexpr (!ACC) {
    const int64_t bytes = (int64_t)a.N * a.K * (F32 ? 4 : 2);
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      int lo = 0, hi = 1;
      if (e0 + lane < a.E) group_range(a.offsets, e0 + lane, a.R, &lo, &hi);
      for (unsigned long long m = __ballot(lo == hi); m; m &= m - 1) {
        uint8_t* o = a.dw + (e0 + __ffsll(m) - 1) * bytes;
        const int64_t step = (int64_t)gridDim.x * kThreads * 16;
        for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 16; i < bytes; i += step)
          *(u32x4*)(o + i) = u32x4{0, 0, 0, 0};
      }
    }
  }
}

// The product for at most 64 rows in all where tiles of 128 p would leave CUs
// idle: a workgroup per 64 p and expert with rows, whose waves also split each
// step's c in two (32 p x 32 q each), eight steps of 16 KB in a ring, seven of
// them in flight.  Against tiles of 128 p (medians of 14 rounds in turn, whose
// quartiles lie within 1 %): one token, top-2 of 8 experts, 4096 x 14336 63.9
// against 87.0 us; top-1, 144 x 2992 12.2 against 15.4; top-8 of 128, 1536 x 2048
// 11.7 against 12.9; 32 tokens, top-2 of 8, 2048 x 2048 13.5 against 14.0.  Near
// the rule's border it loses what the wider tiles save in rows' loads: two tokens,
// top-8 of 128, 1536 x 2048 (192 tiles of 128) 22.1 against 20.6; one token, top-2
// of 8, 14336 x 4096 (224) 51.9 against 51.3.
constexpr int kNarrow = 64;  // p and q of a tile
constexpr int kNarrowStages = 8;
constexpr int kNarrowStage = 2 * kNarrow * kC * 2;
constexpr int kNarrowLds = kNarrowStages * kNarrowStage + 64;

template <bool F32>
__global__ __launch_bounds__(kThreads) void grouped_narrow_kernel(TileArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  Tile t;
  {  // the blockIdx.y-th expert that holds rows
    lds_int* found = (lds_int*)(smem + kNarrowStages * kNarrowStage);  // e, lo, hi; rows per wave
    int lo = 0, hi = 0;
    if (tid < a.E) group_range(a.offsets, tid, a.R, &lo, &hi);
    const unsigned long long m = __ballot(lo < hi);
    if (lane == 0) found[4 + wave] = __popcll(m);
    if (tid == 0) found[0] = a.E;
    __syncthreads();
    int before = __popcll(m & lanemask_lt(lane));
#pragma unroll
    for (int w = 0; w < 8; ++w) before += w < wave ? found[4 + w] : 0;
    if (lo < hi && before == (int)blockIdx.y) {
      found[0] = tid;
      found[1] = lo;
      found[2] = hi;
    }
    __syncthreads();
    t.e = uniform(found[0]);
    if (t.e >= a.E) return;
    t.lo = t.q0 = uniform(found[1]);
    t.hi = uniform(found[2]);
    t.p0 = blockIdx.x * kNarrow;
  }
  const int wp = wave & 1, wq = (wave >> 1) & 1, wc = wave >> 2;
  // wave w loads rows 8w + lane/8 of both operands, lane l the chunk (l%8) ^ pf_mix(row)
  const int r = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ (lane >> 3) ^ (wave & 1);
  const int64_t ld = (int64_t)a.K * 2;
  const uint8_t* pbase = a.w + ((int64_t)t.e * a.N + t.p0) * ld;
  const unsigned pbytes = extent(min(kNarrow, a.N - t.p0), ld, ld);
  const unsigned poff = (unsigned)r * (unsigned)ld + (chunk << 4);
  const uint8_t* qbase = a.q.ids ? a.q.p : a.q.p + t.q0 * a.q.stride * 2;
  const int m = t.q0 + r < t.hi ? (a.q.ids ? row_of(a.q, t.q0 + r) : r) : -1;
  const unsigned qoff = m >= 0 ? (unsigned)m * (unsigned)(a.q.stride * 2) + (chunk << 4) : kOob;
  const int nk = steps_of<2>(a.K);
  auto issue = [&](int s, int stage) {
    lds_u8* dst = smem + stage * kNarrowStage + wave * 1024;
    const bool in = chunk << 3 < a.K - kC * s;
    load_lds<false>(pbase, pbytes, dst, in ? poff + (unsigned)(s * (kC * 2)) : kOob);
    load_lds<false>(qbase, kOob, dst + kNarrowStage / 2, in ? qoff + (unsigned)(s * (kC * 2)) : kOob);
  };
  const int pa = natural_at(32 * wp, lane) ^ (64 * wc), qa = natural_at(32 * wq, lane) ^ (64 * wc);
  f32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
  for (int i = 0; i < kNarrowStages - 1; ++i) issue(i, i);
  for (int s = 0; s < nk; ++s) {
    phase_begin<2 * (kNarrowStages - 2)>();
    const lds_u8* at = smem + s % kNarrowStages * kNarrowStage;
    u32x4 p[2], q[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      p[kk] = *(const lds_u32x4*)(at + (pa ^ (32 * kk)));
      q[kk] = *(const lds_u32x4*)(at + kNarrowStage / 2 + (qa ^ (32 * kk)));
    }
    issue(s + kNarrowStages - 1, (s + kNarrowStages - 1) % kNarrowStages);  // the slot whose reads the barrier ended
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) acc = mfma32_bf16(p[kk], q[kk], acc);
  }
  phase_begin<0>();  // the loads past the last step (zeros)
  // the two halves of c: [wave % 4][4 results][lane]
  lds_f32x4* sums = (lds_f32x4*)smem + (wave & 3) * 256 + lane;
  if (wc)
#pragma unroll
    for (int g = 0; g < 4; ++g) sums[64 * g] = f32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
  __syncthreads();
  if (wc) return;
  uint8_t* o = out_row<0, F32>(a, t, 32 * wq + (lane & 31));
  if (!o) return;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int p = t.p0 + 32 * wp + 8 * g + 4 * (lane >> 5);
    if (p >= a.N) continue;
    const f32x4 v = f32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]} + sums[64 * g];
    if constexpr (F32)
      *(f32x4*)(o + (int64_t)p * 4) = v;
    else
      *(u32x2*)(o + (int64_t)p * 2) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// Launch with `lds` bytes of dynamic LDS; the kernel's ceiling is raised once
// per device.
template <typename Kernel>
bool launch(Kernel kernel, int lds, std::atomic<bool> (&lds_set)[64], dim3 grid, hipStream_t st, const TileArgs& a) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return false;
  if (dev >= 64 || !lds_set[dev].load(std::memory_order_acquire)) {
    if (hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
      return false;
    if (dev < 64) lds_set[dev].store(true, std::memory_order_release);
  }
  kernel<<<grid, kThreads, lds, st>>>(a);
  return true;
}

template <int OP, bool F32>
bool launch_rows(int64_t grid, hipStream_t st, const TileArgs& a) {
  static std::atomic<bool> lds_set[64];
  return launch(grouped_rows_kernel<OP, F32>, lds_bytes(OP), lds_set, dim3((unsigned)grid), st, a);
}

template <bool F32>
bool launch_narrow(int experts, hipStream_t st, const TileArgs& a) {
  static std::atomic<bool> lds_set[64];
  return launch(grouped_narrow_kernel<F32>, kNarrowLds, lds_set, dim3((a.N + kNarrow - 1) / kNarrow, experts), st, a);
}

template <bool F32, bool ACC, bool IDS>
bool launch_weights(int64_t grid, hipStream_t st, const TileArgs& a) {
  static std::atomic<bool> lds_set[64];
  return launch(grouped_wgrad_kernel<F32, ACC, IDS>, lds_bytes(2), lds_set, dim3((unsigned)grid), st, a);
}
template <bool F32, bool ACC>
bool launch_weights(int64_t grid, hipStream_t st, const TileArgs& a) {
  return a.p.ids || a.q.ids ? launch_weights<F32, ACC, true>(grid, st, a)
                            : launch_weights<F32, ACC, false>(grid, st, a);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

namespace {

// One workgroup per CU: kSlots on each of the eight XCDs, fewer where there are
// fewer tiles than that.  An XCD's share of each of the up to three kinds of
// tiles is rounded up.
int64_t persistent_grid(int64_t tiles) {
  const int64_t slots = cdiv(tiles, 8) + 2;
  return 8 * (slots < kSlots ? slots : kSlots);
}

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
  // at most R/256 whole row tiles and one rest per expert that holds rows
  const int experts = a.R < a.E ? a.R : a.E;
  const int64_t rows = a.R / kTile + experts;
  if (!dgrad && a.R <= kNarrow && experts * cdiv(a.N, kHalf) < 8 * kSlots)
    return f32 ? launch_narrow<true>(experts, st, t) : launch_narrow<false>(experts, st, t);
  const int64_t grid = persistent_grid(rows * cdiv(dgrad ? a.K : a.N, kHalf));
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
  const int64_t grid = persistent_grid(cdiv(a.N, kTile) * cdiv(a.K, kTile) * a.E);
  if (f32) return accumulate ? launch_weights<true, true>(grid, st, t) : launch_weights<true, false>(grid, st, t);
  return launch_weights<false, false>(grid, st, t);
}

}  // namespace moe
