// Attention of a sequence's last tokens over its paged cache on the
// 5th-generation tensor cores: head dimension 128, pages of 16, 32, 64, ...
// keys, bfloat16 or 8-bit rows.
//
//   S = Q K^T       128 query rows x 128 keys, fp32 in TMEM
//   P = 2^(s - R)   R: the row's reference, near its running maximum
//   O += P V        128 query rows x 128 dims, fp32 in TMEM, P from TMEM
//
// Work.  A segment is a kv head's query rows (up to 256: token x head of the
// group, of one sequence, or of all sequences for the shared positions) with
// the keys they see, in tiles of 128 keys.  All segments' tiles are laid end
// to end and every CTA takes an equal share, so long and short sequences,
// heads and prefixes load all SMs alike whatever the lengths are, which only
// the device knows.  A segment that one CTA finishes is written by it;
// otherwise each CTA leaves (O, R, sum) and a second kernel joins them.
//
// Two streams share a CTA, so that one's softmax runs under the other's
// products: with up to 128 query rows both take the same rows and every
// second key tile (few rows are bound by the cache's bytes: what counts is
// how many are in flight); with more, each takes 128 of the rows and both
// read the same tiles (many rows are bound by the products: a tile in shared
// memory serves twice as many).
//
// Precision.  bfloat16: P goes in as bf16 high and low parts, two products
// with V, so that its rounding (2^-16) does not add to the output's.  8-bit:
// the codes are multiplied as they are, no byte of the cache is converted.
// q is split into an e4m3 and an e5m2 code (its 8 bits are 4 + 4, and what
// rounding to 4 leaves is one of 0 .. 8 units, which 3 bits hold: exact down
// to 2^-13 of the row's largest, within 2^-21 of the largest below) and P,
// times the key's value scale, an f16, into three e5m2 codes, which hold its
// 11 bits (2^-11 of each weight, or 2^-27 of the row's largest).  The scales of
// keys multiply the scores; those of values the weights.
//
// Warps: 0-3 and 4-7 softmax of stream 0 and 1 (thread = query row); 8 loads
// keys and values by TMA; 9 TMEM and MMA issue; 10 what a tile needs beside
// its rows: which 16-key groups exist, the scales, and, in tiles that hold
// keys which some row does not see, zeros for values that are not finite (a
// zero weight would turn them into NaN; rows that do see one are marked); 11
// the segments of this CTA, one ahead of the others, and their query rows.
// Loops over a tile are rolled where they can be: five roles' code shares the
// instruction cache, and unrolled it took most of the time to fetch.
//
// Measured.  32 x 8 tokens at contexts of 512 to 4096, 4 heads a kv head,
// bfloat16: 68 us, 4.5 TB/s of the cache; 256 x 7 at 8192, 8-bit: 592 us, 3.6
// TB/s.  Few rows are bound by a tile's chain of scores, softmax and weighted
// sums, of which a CTA has two under way (its values come late in the chain,
// so their bytes wait in shared memory).  Behind a shared prefix: 64 x 16
// tokens, 5 heads a kv head, 16384 keys, 8-bit: 0.54 ms (0.52 with weights of
// nine bits); 32 x 8, 8192 keys, bfloat16: 75 us; bound by the softmax's
// instructions, about 2000 cycles a tile of 256 rows with bfloat16 and 4500
// with 8-bit weights, beside products of 1280 to 1540.  (Two softmax warps for
// every 32 rows, 16 in all, were slower everywhere: 73, 593, 593 and 87 us,
// with weights of nine bits, where eight took 66, 565, 498 and 79.)
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kTile = 128;  // keys of a tile, query rows of a stream
constexpr int kD = 128;     // head dimension
constexpr int kSoftmax = 256;
constexpr int kThreads = kSoftmax + 128;
constexpr int kRowTile = 2 * kTile;  // query rows of a segment at most
constexpr int kSegs = 3;  // segments that warp 11 may be ahead (its query rows have two places)
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kMaxCtas = kMaxSM;
constexpr float kNone = -INFINITY;
// Least log2 of a value's scale that the reference of 8-bit weights follows:
// weights then stay below 2^(15 + 80), and their sums, of fewer than 2^31 keys,
// in a float's range.  Smaller values go into smaller codes: below 2^-84 the
// smallest of them are lost, below 2^-105 or so all.
constexpr int kLeastScale = -80;

// TMEM columns: scores (then weights) and accumulators of the two streams
__device__ constexpr uint32_t s_col(int j) { return 128u * j; }
__device__ constexpr uint32_t o_col(int j) { return 256u + 128u * j; }

struct TileInfo {
  float ks[kTile], vs[kTile];  // scales 2^(byte - 127) of keys and values
  float lv[kTile];             // log2 of the values' scales (at least kLeastScale)
  uint32_t bad[4];             // keys whose values were not finite and are zeros now
  uint32_t groups;             // bit i: 16-key group i exists
  float vmax;                  // the largest of lv
  uint32_t spoilt;             // some bit of `bad` is set
  uint32_t pad;
};

// A segment's share of this CTA, as its roles need it.
struct alignas(16) SegInfo {
  int tiles;            // 0: no more segments
  int first, end;       // position of its first tile; keys end before `end`
  int all_lo, all_hi;   // keys that every row sees
  int shared, s, h;     // the shared part's (s = 0), or sequence s; kv head
  int f0, rows;         // first query row (sequence, token, head of the group), their number
  int n, len;           // tokens and keys of sequence s
  int split;            // both streams take the same rows
  int copies;           // of the rows in the 128 of a stream (1, 2 or 4)
  int q;                // place of the query rows (split)
  int own_q;            // the softmax warps load the query rows: of many rows, and of the first segment
  int slot;             // place of the partial result, -1: the CTA finishes the segment
};

template <bool E4M3>
struct Smem {
  static constexpr int Q = 0;                          // [2][32 KB]
  static constexpr int SLOT = E4M3 ? 16384 : 32768;    // K or V of a tile
  static constexpr int SLOTS = E4M3 ? 9 : 5;
  static constexpr int RING = 65536;
  static constexpr int INFOS_AHEAD = 4;  // tiles that warp 10 may be ahead of the softmax
  static constexpr int INFO = RING + SLOTS * SLOT;
  static constexpr int INFOS = E4M3 ? (int)sizeof(TileInfo) : 32;  // bf16 keeps the tail of TileInfo only
  static constexpr int SEG = INFO + INFOS_AHEAD * INFOS;
  static constexpr int QSCALE = SEG + kSegs * (int)sizeof(SegInfo);  // float [kSegs][kRowTile], 8-bit only
  static constexpr int BAR = QSCALE + (E4M3 ? kSegs * kRowTile * 4 : 0);
  static constexpr size_t bytes = 1024 + BAR + (2 * SLOTS + 2 * INFOS_AHEAD + 2 * kSegs + 12) * 8 + 64;
  static_assert(bytes + 512 <= 227 * 1024, "shared memory");
};

struct Plan {
  AttendArgs a;
  int group, rows;     // query heads per kv head; query rows (n_tok * group) of a sequence
  int tiles_p;         // row tiles of the shared part (0: none)
  int tiles_s;         // row tiles of a sequence at most
  int slot_rows;       // rows of a sequence's partial slot
  int page_shift;      // page_size = 2^page_shift
  int seg_cost;
  int* head;           // workspace: all positions, tiles of the shared part, first position of each row tile
  float *part_p, *part_s;    // partial accumulators [slot][rows][kD] of the shared part and of the sequences
  float2 *ref_p, *ref_s;     // (R, sum) of their rows
};

// Lengths of sequence s, clamped to what the block table holds.
__device__ __forceinline__ int2 lengths(const AttendArgs& a, int s) {
  const int n = a.n_new ? min(max(a.n_new[s], 0), a.n_tok) : a.n_tok;
  const long long cap = (long long)a.max_pages * a.page_size;
  const int len = a.kv_len[s];
  return make_int2(n, len < 0 ? 0 : (int)min((long long)len, cap));
}
// Keys [x, y) that token t of a sequence sees.
__device__ __forceinline__ int2 sees(const AttendArgs& a, int2 nl, int t) {
  const int hi = a.causal ? nl.y - (nl.x - 1 - t) : nl.y;
  return make_int2(a.window > 0 ? max(0, hi - a.window) : 0, hi);
}

struct Segment {
  int rows;         // query rows
  int base, tiles;  // first key's position (a multiple of 16), key tiles
  int end;          // keys end before this position
};

// Row tile i of a sequence (positions from shared_len on).
__device__ __forceinline__ Segment segment_of(const AttendArgs& a, int group, int2 nl, int i) {
  Segment g = {0, 0, 0, 0};
  const int first = i * kRowTile, all = nl.x * group;
  if (first >= all) return g;
  g.rows = min(kRowTile, all - first);
  const int t0 = i == 0 ? 0 : first / group, t1 = first + g.rows == all ? nl.x - 1 : (first + g.rows - 1) / group;
  const int lo = max(sees(a, nl, t0).x, a.shared_len), hi = sees(a, nl, t1).y;
  if (hi <= lo) return g;
  g.base = lo & ~15;
  g.end = hi;
  g.tiles = (hi - g.base + kTile - 1) / kTile;
  return g;
}
// Cost of work in units of half a tile for up to 128 rows, near enough: a
// tile for more of them, and (seg_cost) a segment's start and end beside its
// tiles: measured, about 7 with bfloat16 rows and 16 with 8-bit ones.
__device__ __forceinline__ int weight_of(int rows) { return rows > kTile ? 4 : 2; }
__device__ __forceinline__ int cost_of(int seg_cost, int tiles, int w) { return tiles > 0 ? seg_cost + tiles * w : 0; }
// The tiles [x, y) of a segment at position `at` that the share [a, b) has:
// tile k counts as lying at at + seg_cost + k w.
__device__ __forceinline__ int2 tiles_in(int seg_cost, int at, int tiles, int w, int a, int b) {
  at += seg_cost;
  return make_int2(at >= a ? 0 : (a - at + w - 1) / w, b <= at ? 0 : min(tiles, (b - at + w - 1) / w));
}

// Share of CTA c of n: tiles whose position lies in [bound(c), bound(c + 1));
// the first units % n shares are one larger.  (Positions fit 31 bits: the
// host sees to it.)
__device__ __forceinline__ int bound_of(int units, int c, int n) { return units / n * c + min(c, units % n); }
__device__ __forceinline__ int owner_of(int units, int x, int n) {
  const int q = units / n, wide = units % n * (q + 1);
  return x < wide ? x / (q + 1) : units % n + (x - wide) / q;
}

// Place of a CTA's part of a segment.  With a shared part every segment has
// parts, and (segment, CTA) pairs in order take consecutive places; without,
// a CTA leaves at most two: of the segment in which its share starts, and of
// the one in which it ends.
__device__ __forceinline__ int slot_of(const Plan& p, int segment, int cta, bool from_start) {
  return p.tiles_p > 0 ? segment + cta : 2 * cta + from_start;
}

// A place in a ring of N slots and the parity of its round.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) {
      slot = 0;
      ++round;
    }
  }
  __device__ __forceinline__ Ring ahead(int n) const {  // n < N
    Ring r = *this;
    r.slot += n;
    if (r.slot >= N) {
      r.slot -= N;
      ++r.round;
    }
    return r;
  }
};

// A bounded wait that did not succeed at once.  Not inlined: the roles wait in
// many places.  The hardware suspends the thread for some microseconds a
// try (polling as fast as it goes took a third of all issued instructions,
// from the schedulers of the softmax warps); the clock is read now and then.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, uint32_t abort_flag, unsigned* status) {
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity), "r"(20000u)
          : "memory");
      if (ok) return true;
    }
    uint32_t given_up;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(given_up) : "r"(abort_flag) : "memory");
    if (given_up) return false;
    if (globaltimer() - t0 > kWaitNs) {
      asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort_flag), "r"(1u) : "memory");
      flag(status, DFLASH2_DEV_WAIT_TIMEOUT);
      return false;
    }
  }
}

// Waits, as long at most, until the count at `at` has come to n (counts differ
// by less than 2^31).
__device__ __noinline__ bool wait_count(uint32_t at, uint32_t n, uint32_t abort_flag, unsigned* status) {
  const uint64_t t0 = globaltimer();
  while (true) {
    uint32_t x;
    asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    if ((int)(x - n) >= 0) return true;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(x) : "r"(abort_flag) : "memory");
    if (x) return false;
    if (globaltimer() - t0 > kWaitNs) {
      asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort_flag), "r"(1u) : "memory");
      flag(status, DFLASH2_DEV_WAIT_TIMEOUT);
      return false;
    }
    __nanosleep(100);
  }
}

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ void bar_stream(int j) { asm volatile("bar.sync %0, 128;" ::"r"(2 + j) : "memory"); }
__device__ __forceinline__ bool bar_softmax_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, 1, 256, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// One lane of the warp.  The compiler knows that no other lane is active
// behind this: what the lane computes goes to uniform registers, where the
// tensor core's instructions take their operands.  (Behind `lane == 0` every
// operand is moved there instruction by instruction: 16 instructions a
// product, which the softmax warps of the same scheduler hold up: 2830 to
// 4970 cycles for 24 products beside busy warps, 1610 to 2570 this way, 1536
// in the tensor core.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// D (+)= A B, A from shared memory or from TMEM; kind::f16 or kind::f8f6f4.
template <bool E4M3>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    umma_bf16(d, a, b, idesc, acc);
}
template <bool E4M3>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ uint32_t bits2(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two f16 as three e5m2 each, in the upper bytes of the halves: an f16's
// upper byte is an e5m2, so round, subtract, round, subtract.  Rounding, and
// not cutting, makes three enough for the eleven bits: at most 2^7 units of
// the last place are left of the first code, 2^3 of the second, and three bits
// hold every such number.  That is exact from 2^-6 on; below, what is left may
// lie under an e5m2's smallest step, and rounding the last code too leaves out
// 2^-17 at most, 2^-27 of a row's largest weight.
__device__ __forceinline__ void split3(__half2 u, uint32_t (&h)[3]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t top = (*reinterpret_cast<const uint32_t*>(&u) + 0x00800080u) & 0xff00ff00u;
    h[q] = top;
    u = __hsub2(u, *reinterpret_cast<const __half2*>(&top));
  }
  h[2] = *reinterpret_cast<const uint32_t*>(&u) + 0x00800080u;
}

// Scales a row's accumulator (4 pieces of 32 columns, or none) and the
// weights of the tile's first `chunks` pieces of 32 keys by `by`, a power of
// two.  Rare, and so not inlined.
template <bool E4M3>
__device__ __noinline__ void rescale(uint32_t o, int pieces, uint32_t w, int chunks, float by) {
#pragma unroll 1
  for (int c = 0; c < pieces; ++c) {
    float x[32];
    tmem_ld32(o + 32 * c, x);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t r[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) r[b] = __float_as_uint(x[8 * i + b] * by);
      tmem_st8(o + 32 * c + 8 * i, r);
    }
  }
  tmem_st_wait();  // (and the weights stored before)
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t r[3][8];
    if (E4M3) {
      const __half2 by2 = __float2half2_rn(by);
      uint32_t n[3][8];
#pragma unroll
      for (int q = 0; q < 3; ++q) tmem_ld8_nowait(w + 32 * c + 8 * q, r[q]);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t h[2][3];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          __half2 u[3];
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            const uint32_t x = __byte_perm(r[q][i], 0u, b ? 0x3424 : 0x1404);
            u[q] = *reinterpret_cast<const __half2*>(&x);
          }
          split3(__hmul2(__hadd2(__hadd2(u[2], u[1]), u[0]), by2), h[b]);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) n[q][i] = __byte_perm(h[0][q], h[1][q], 0x7531);
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) tmem_st8(w + 32 * c + 8 * q, n[q]);
    } else {
      const __nv_bfloat162 by2 = __float2bfloat162_rn(by);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        tmem_ld8_nowait(w + 32 * c + 8 * q, r[0]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) r[0][i] = bits2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r[0][i]), by2));
        tmem_st8(w + 32 * c + 8 * q, r[0]);
      }
    }
  }
  tmem_st_wait();
}

// ------------------------------------------------------------------ query rows

// Rows [r0, r1) of a segment (r0 and r1 - r0 of one place of 128), by a warp,
// into the place at `dst`: K-major with the 128-byte swizzle.  bfloat16: two
// halves of 64 dims, 16 KB apart.  8-bit: the high codes (e4m3) and, 16 KB
// behind, the low ones (e5m2, whose smallest step is 2^7 times finer: small
// channels beside large ones keep their bits); a row's largest magnitude
// becomes 2^7 .. 2^8, and qscale[row] the factor that its scores take.
template <bool E4M3>
__device__ __forceinline__ void load_rows(const Plan& p, const SegInfo& g, int r0, int r1, uint8_t* dst, float* qscale) {
  const AttendArgs& a = p.a;
  constexpr int W = E4M3 ? 8 : 16;  // lanes of a row
  constexpr int STEP = 32 / W;
  const int lane = threadIdx.x & 31, c = lane & (W - 1);
  const int copy_rows = g.split ? kTile / g.copies : kTile;
  // this lane's row, stepped through the heads of the group, tokens and sequences without divisions
  int row = r0 + lane / W;
  int s = g.shared ? (g.f0 + row) / p.rows : g.s;
  int gq = g.f0 + row - s * p.rows, t = gq / p.group;
  gq -= t * p.group;
  int n = !a.n_new ? a.n_tok : s < a.batch ? a.n_new[s] : 0;
  auto source = [&]() {  // address of the row, or null; then the lane's next row
    const bool real = row < r1 && t < n;
    const bf16* src = a.q + ((size_t)s * a.n_tok + t) * a.q_stride + (size_t)(g.h * p.group + gq) * kD;
    row += STEP;
    gq += STEP;
    while (gq >= p.group) {
      gq -= p.group;
      if (++t == a.n_tok) {
        t = 0;
        ++s;
        if (a.n_new) n = s < a.batch ? a.n_new[s] : 0;
      }
    }
    return real ? src : nullptr;
  };
  if (!E4M3) {
#pragma unroll 2
    for (int x = r0; x < r1; x += STEP) {
      const int r = (x + lane / W) & (kTile - 1);
      const bf16* src = source();
      if (x + lane / W < r1)
        for (int cp = 0; cp < kTile; cp += copy_rows)  // (a row's place in 8 is the same in every copy)
          cp_async16(dst + (c >> 3) * 16384 + (cp + r) * 128 + (((c & 7) ^ (r & 7)) << 4), src ? src + c * 8 : a.q,
                     src != nullptr);
    }
    cp_async_commit();
    cp_async_wait<0>();
    return;
  }
#pragma unroll 1
  for (int x = r0; x < r1; x += 4 * STEP) {  // 16 rows: all their loads in flight, then their codes
    uint4 v[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bf16* src = source();
      v[u][0] = src ? reinterpret_cast<const uint4*>(src)[2 * c] : make_uint4(0u, 0u, 0u, 0u);
      v[u][1] = src ? reinterpret_cast<const uint4*>(src)[2 * c + 1] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int fr = x + u * STEP + lane / W, r = fr & (kTile - 1);
      const uint32_t w8[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w, v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(max(top, w8[i] & 0x7f800000u), (w8[i] << 16) & 0x7f800000u);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2^(134 - e), e the largest magnitude's exponent field (rows below
      // 2^-119 are not scaled up all the way, and keep their bits all the same)
      const uint32_t e = max(8u, top >= 0x7f800000u ? 254u : top >> 23);
      const float up = __uint_as_float((261u - e) << 23);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // (eight bits: an f16 holds the scaled value, and what the high code leaves of it, exactly)
        const __half2 x = __floats2half2_rn(__uint_as_float(w8[i] << 16) * up, __uint_as_float(w8[i] & 0xffff0000u) * up);
        const uint32_t h2 = __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
        const __half2 back(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h2, __NV_E4M3));
        const uint32_t l2 = __nv_cvt_halfraw2_to_fp8x2(__hsub2(x, back), __NV_SATFINITE, __NV_E5M2);
        hi[i >> 1] = (i & 1) ? hi[i >> 1] | (h2 << 16) : h2;
        lo[i >> 1] = (i & 1) ? lo[i >> 1] | (l2 << 16) : l2;
      }
      if (fr < r1) {
        for (int cp = 0; cp < kTile; cp += copy_rows) {
          uint8_t* q = dst + (cp + r) * 128 + ((c ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(q) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(q + 16384) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        // a row that is not finite has no result
        if (c == 0)
          qscale[fr] = top >= 0x7f800000u ? __int_as_float(0x7fffffff) : __uint_as_float((e - 7u) << 23);
      }
    }
  }
}

// ------------------------------------------------------------------ main kernel

template <bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) attend_tc_kernel(const __grid_constant__ Plan p,
                                                               const __grid_constant__ CUtensorMap tm_k,
                                                               const __grid_constant__ CUtensorMap tm_v) {
  using L = Smem<E4M3>;
  constexpr int NS = L::SLOTS, kInfo = L::INFOS_AHEAD;
  extern __shared__ uint8_t raw_smem[];
  // (an offset, not a cast address: the compiler keeps to shared-memory accesses)
  uint8_t* sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* full = bars;              // [NS] a K or V tile landed
  uint64_t* empty = full + NS;        // [NS] its products are done
  uint64_t* info_full = empty + NS;   // [kInfo] tile info is there (and V mended)
  uint64_t* info_empty = info_full + kInfo;
  uint64_t* seg_full = info_empty + kInfo;  // [kSegs] a segment and its query rows are there
  uint64_t* seg_empty = seg_full + kSegs;   // [kSegs] every role has read it (11 arrivals)
  uint64_t* s_full = seg_empty + kSegs;     // [2] scores of a stream's tile in TMEM
  uint64_t* p_ready = s_full + 2;           // [2] its weights in TMEM (4 arrivals)
  uint64_t* o_done = p_ready + 2;           // [2] a segment's last product of the stream is done
  uint64_t* q_empty = o_done + 2;           // [2] a place of query rows is free (8 arrivals)
  uint64_t* q_ready = q_empty + 2;          // query rows that the softmax warps load themselves (8 arrivals)
  uint64_t* q_full = q_ready + 1;           // [2] query rows that warp 11 loaded into a place
  uint64_t* drain = q_full + 2;             // every product issued is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* abort_flag = tmem_slot + 1;
  const uint32_t abort_at = smem_u32(abort_flag), issued_at = abort_at + 4;  // loads issued
  SegInfo* segs = reinterpret_cast<SegInfo*>(sm + L::SEG);
  __shared__ int scan[kThreads / 32], ends[kThreads / 32][2], start[3];

  const AttendArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, nctas = gridDim.x;
  pdl_launch_next();
  if (threadIdx.x < 2 * NS) mbar_init(bars + threadIdx.x, 1);
  else if (threadIdx.x == 32) {
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(info_full + i, 1);
      mbar_init(info_empty + i, 8);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(seg_full + i, 1);
      mbar_init(seg_empty + i, 11);
    }
  } else if (threadIdx.x == 64) {
    for (int j = 0; j < 2; ++j) {
      mbar_init(s_full + j, 1);
      mbar_init(p_ready + j, 4);
      mbar_init(o_done + j, 1);
      mbar_init(q_empty + j, 8);
      mbar_init(q_full + j, 1);
    }
    mbar_init(q_ready, 8);
    mbar_init(drain, 1);
    abort_flag[0] = abort_flag[1] = 0;
  }
  fence_barrier_init();
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();

  // ------------------------------------------------ shares of the work
  const int entries = a.batch * p.tiles_s;  // row tiles of the sequences
  const int per = (entries + kThreads - 1) / kThreads, e0 = min(entries, (int)threadIdx.x * per);
  const int e1 = min(entries, e0 + per);
  // units (tiles times cost) of row tile e, of all kv heads
  auto units_of = [&](int e, int2* nl) {
    const int s = p.tiles_s == 1 ? e : e / p.tiles_s;
    *nl = lengths(a, s);
    const Segment g = segment_of(a, p.group, *nl, p.tiles_s == 1 ? 0 : e % p.tiles_s);
    return cost_of(p.seg_cost, g.tiles, weight_of(g.rows)) * a.nkv;
  };
  int my_units = 0, lo = INT32_MAX, hi = 0;
  for (int e = e0; e < e1; ++e) {
    int2 nl;
    my_units += units_of(e, &nl);
    if (p.tiles_p > 0 && nl.x > 0) {
      lo = min(lo, sees(a, nl, 0).x);
      hi = max(hi, sees(a, nl, nl.x - 1).y);
    }
  }
  int before = my_units;  // block scan; minimum and maximum of the shared part's keys
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 31) {
    scan[warp] = before;
    ends[warp][0] = lo;
    ends[warp][1] = hi;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  before -= my_units;
  int total = 0;
  lo = INT32_MAX;
  hi = 0;
#pragma unroll 1
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += scan[i];
    total += scan[i];
    lo = min(lo, ends[i][0]);
    hi = max(hi, ends[i][1]);
  }
  hi = min(hi, a.shared_len);
  const int base_p = lo & ~15, end_p = hi;
  const int tiles_p = p.tiles_p > 0 && hi > lo ? (hi - base_p + kTile - 1) / kTile : 0;
  const int cost_p = cost_of(p.seg_cost, tiles_p, weight_of(kRowTile));  // (its last row tile may be cheaper: no matter)
  const int up = p.tiles_p * a.nkv * cost_p, units = up + total;
  const int share_a = bound_of(units, cta, nctas), share_b = bound_of(units, cta + 1, nctas);
  if (cta == 0) {  // for the joining kernel
    if (threadIdx.x == 0) {
      p.head[0] = units;
      p.head[1] = tiles_p;
    }
    int x = up + before;
    for (int e = e0; e < e1; ++e) {
      int2 nl;
      p.head[2 + e] = x;
      x += units_of(e, &nl);
      const int s = e / p.tiles_s;
      if (a.kv_len[s] != nl.y || (a.n_new && a.n_new[s] != nl.x)) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
    }
  }
  // the row tile and the position in which this CTA's share starts
  {
    const int x = share_a - up;
    if (share_a < share_b && x >= 0 && before <= x && x < before + my_units) {
      int y = before;
      for (int e = e0; e < e1; ++e) {
        int2 nl;
        const int all = units_of(e, &nl);
        if (x < y + all) {
          start[0] = e;
          start[1] = up + y;
          break;
        }
        y += all;
      }
    }
  }
  __syncthreads();

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(smem_u32(bar), parity) || wait_on(smem_u32(bar), parity, abort_at, a.status);
  };
  // The next segment (tiles = 0: none, or the kernel is giving up).
  Ring<kSegs> seg_at;
  auto next_segment = [&](SegInfo* g) {
    bool ok = __all_sync(0xffffffffu, wait(seg_full + seg_at.slot, seg_at.round & 1));
    if (warp < 8) ok = !bar_softmax_or(!ok);  // (their barriers need all of them, or none)
    *g = segs[seg_at.slot];
    if (!ok) g->tiles = 0;
    __syncwarp();
    if (!E4M3 || warp >= 8) {  // (the softmax warps of an 8-bit cache read the rows' scales first)
      if (lane == 0) mbar_arrive(seg_empty + seg_at.slot);
    }
    return g->tiles > 0;
  };

  if (warp == 11) {
    // ---------------------------------------------------------------- segments and their query rows
    int q_uses[2] = {0, 0}, q_next = 0;
    bool ok = true;
    // positions: `at` the current row tile's first, kv heads one behind the other
    int entry, at;
    bool shared = share_a < up;
    if (shared) {
      entry = share_a / (cost_p * a.nkv);
      at = entry * (cost_p * a.nkv);
    } else {
      entry = start[0];
      at = start[1];
    }
    if (share_a >= share_b) at = share_b;  // (no share: nothing has set `start`)
    while (at < share_b && ok) {
      SegInfo g;
      int base, tiles, w;
      if (shared) {
        g.s = 0;
        g.f0 = entry * kRowTile;
        g.rows = min(kRowTile, a.batch * p.rows - g.f0);
        base = base_p;
        tiles = tiles_p;
        w = weight_of(kRowTile);
        g.end = end_p;
        g.n = g.len = 0;
        // keys that all of its rows see
        const int s0 = g.f0 / p.rows, s1 = (g.f0 + g.rows - 1) / p.rows;
        int from = 0, to = a.shared_len;
        for (int s = s0 + lane; s <= s1; s += 32) {
          const int2 nl = lengths(a, s);
          if (nl.x == 0) continue;
          from = max(from, sees(a, nl, nl.x - 1).x);
          to = min(to, sees(a, nl, 0).y);
        }
        g.all_lo = __reduce_max_sync(0xffffffffu, from);
        g.all_hi = __reduce_min_sync(0xffffffffu, to);
      } else {
        g.s = p.tiles_s == 1 ? entry : entry / p.tiles_s;
        const int i = entry - g.s * p.tiles_s;
        const int2 nl = lengths(a, g.s);
        const Segment x = segment_of(a, p.group, nl, i);
        g.f0 = g.s * p.rows + i * kRowTile;
        g.rows = x.rows;
        base = x.base;
        tiles = x.tiles;
        w = weight_of(g.rows);
        g.end = x.end;
        g.n = nl.x;
        g.len = nl.y;
        g.all_lo = max(sees(a, nl, (i * kRowTile + g.rows - 1) / p.group).x, a.shared_len);
        g.all_hi = sees(a, nl, i * kRowTile / p.group).y;
      }
      g.shared = shared;
      g.split = g.rows <= kTile;
      g.copies = g.rows <= 32 ? 4 : g.rows <= 64 ? 2 : 1;
      for (int h = 0; h < a.nkv && ok; ++h, at += cost_of(p.seg_cost, tiles, w)) {
        if (tiles == 0 || at >= share_b) break;
        const int2 k = tiles_in(p.seg_cost, at, tiles, w, share_a, share_b);
        if (k.x >= k.y) continue;
        g.h = h;
        g.first = base + k.x * kTile;
        g.tiles = k.y - k.x;
        g.slot = k.x == 0 && k.y == tiles && p.tiles_p == 0 ? -1 : slot_of(p, entry * a.nkv + h, cta, k.x == 0);
        g.q = g.split ? q_next : 0;
        if (seg_at.round > 0) ok = wait(seg_empty + seg_at.slot, (seg_at.round - 1) & 1) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        g.own_q = !g.split || (seg_at.slot == 0 && seg_at.round == 0);
        if (lane == 0) segs[seg_at.slot] = g;
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_full + seg_at.slot);  // (its keys and values may be on their way before its rows)
        // query rows: the place (both, where the softmax warps load them) has to be free
        for (int b = g.split ? g.q : 0; b < (g.split ? g.q + 1 : 2); ++b) {
          if (q_uses[b] > 0) ok = wait(q_empty + b, (q_uses[b] - 1) & 1) && ok;
          ++q_uses[b];
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (g.split) q_next ^= 1;
        if (!g.own_q) {
          load_rows<E4M3>(p, g, 0, g.rows, sm + L::Q + g.q * 32768,
                          reinterpret_cast<float*>(sm + L::QSCALE) + seg_at.slot * kRowTile);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full + g.q);
        }
        seg_at.step();
      }
      // (after the last kv head `at` is the next row tile's first position)
      ++entry;
      if (shared && entry == p.tiles_p) {
        shared = false;
        entry = 0;
      }
    }
    // the end
    if (seg_at.round > 0) wait(seg_empty + seg_at.slot, (seg_at.round - 1) & 1);
    if (lane == 0) segs[seg_at.slot].tiles = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_full + seg_at.slot);
  } else if (warp == 8) {
    // ---------------------------------------------------------------- loads
    const uint64_t pol = policy_evict_first();
    const int absent = a.n_pages * a.page_size;  // a row past the pool: the copy fills zeros
    Ring<NS> at;
    bool ok = true;
    SegInfo g;
    for (; ok && next_segment(&g); seg_at.step()) {
      const int lead = g.split ? 2 : 1, x_h = g.h * (E4M3 ? 64 : 128);
      const int32_t* table = a.block_table + (size_t)g.s * a.max_pages;
      // lane 8 t + i: pool row of 16-key group i of tile t0 + t
      auto rows_of = [&](int t0) {
        const int t = t0 + (lane >> 3), pos = g.first + t * kTile + 16 * (lane & 7);
        int row = absent;
        if (t < g.tiles && pos < g.end) {
          const int page = table[pos >> p.page_shift];
          if (page >= 0 && page < a.n_pages) row = (page << p.page_shift) + (pos & (a.page_size - 1));
        }
        return row;
      };
      auto load = [&](int rows, int t, const void* map) {
        const int slot = at.slot;
        if (at.round > 0) ok = wait(empty + slot, (at.round - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        uint8_t* dst = sm + L::RING + slot * L::SLOT;
        if (lane == 0) {
          mbar_arrive_expect_tx(full + slot, L::SLOT);
          asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(issued_at), "r"(at.round * NS + slot + 1) : "memory");
        }
        const int row = __shfl_sync(0xffffffffu, rows, (t & 3) * 8 + (lane & 7));
        if (E4M3) {
          if (lane < 8) tma_load_2d(dst + lane * 2048, map, full + slot, x_h, row, pol);
        } else {
          if (lane < 16)
            tma_load_2d(dst + (lane >> 3) * 16384 + (lane & 7) * 2048, map, full + slot, x_h + (lane >> 3) * 64, row, pol);
        }
        at.step();
      };
      // keys' tiles are `lead` ahead of the values'; the rows of the next four
      // tiles are looked up while these are loaded
      int v_rows = rows_of(0), k_rows = v_rows, next = rows_of(4);
#pragma unroll 1
      for (int t = -lead; t < g.tiles && ok; ++t) {
        if (t > 0 && (t & 3) == 0) v_rows = k_rows;  // (the keys have moved on before, by lead < 4 tiles)
        if (t >= 0) load(v_rows, t, &tm_v);
        const int tk = t + lead;
        if (tk < g.tiles && ok) {
          if (tk > 0 && (tk & 3) == 0) {
            k_rows = next;
            next = rows_of(tk + 4);
          }
          load(k_rows, tk, &tm_k);
        }
      }
    }
    // copies in flight land before the CTA ends
    for (int i = 0; i < NS; ++i) {
      volatile int never = 0;
      if (i < at.slot) mbar_wait(full + i, at.round & 1, &never, kWaitNs);
      else if (at.round > 0) mbar_wait(full + i, (at.round - 1) & 1, &never, kWaitNs);
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_one()) {
      // shared addresses in the descriptors' 16-byte units; their upper words are constant
      const uint32_t ring = smem_u32(sm + L::RING) >> 4, qs = smem_u32(sm + L::Q) >> 4;
      constexpr uint64_t kKMajor =
          ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
      constexpr uint64_t kMnMajor =
          ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
      // A K-major, B = K rows K-major; B = V rows MN-major; 8-bit weights are
      // e5m2, and so are the low codes of q
      constexpr uint32_t id_s =
          E4M3 ? (1u << 4) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24) : idesc_bf16_f32(kTile, kTile);
      constexpr uint32_t id_o =
          (E4M3 ? (1u << 4) | (1u << 7) | ((kD >> 3) << 17) | ((kTile >> 4) << 24) : idesc_bf16_f32(kTile, kD)) |
          (1u << 16);
      Ring<NS> at;
      uint32_t n_p = 0, n_q = 0;  // parities: of the streams' weights; of the places' query rows and of q_ready
      bool ok = true;
      for (; ok; seg_at.step()) {
        if (!wait(seg_full + seg_at.slot, seg_at.round & 1)) break;
        const SegInfo& g = segs[seg_at.slot];
        const int nt = g.tiles, lead = g.split ? 2 : 1, g_q = g.q, g_own = g.own_q;
        const uint32_t q0 = qs + g_q * 2048;
        mbar_arrive(seg_empty + seg_at.slot);
        if (nt == 0) break;
        uint64_t* rows_there = g_own ? q_ready : q_full + g_q;
        const uint32_t bit = g_own ? 4u : 1u << g_q;
        if (!wait(rows_there, (n_q & bit) ? 1 : 0)) break;
        n_q ^= bit;
        // Work u: stream u % 2's products with a tile's values, and then its
        // scores of the next one.  With shared rows stream u % 2 takes tile u
        // and the slots go K0 K1 V0 K2 V1 K3 ...; otherwise both take tile
        // u / 2 and they go K0 V0 K1 V1 ...
        const int all = lead == 2 ? nt : 2 * nt;
#pragma unroll 1
        for (int u = -2; u < all; ++u) {
          const int j = u & 1;
          const bool release = lead == 2 || j == 1;
          const uint32_t pc = tmem + s_col(0) + 128u * j;
          if (u >= 0) {
            ok = wait(full + at.slot, at.round & 1) && wait(p_ready + j, (n_p >> j) & 1);
            if (!ok) break;
            n_p ^= 1u << j;
            tc_fence_after();
            const uint32_t vd = ring + at.slot * (L::SLOT >> 4), d = tmem + o_col(0) + 128u * j;
            const uint32_t acc = u >= 2 ? 1u : 0u;
            if (E4M3) {
#pragma unroll
              for (int x = 0; x < 12; ++x)  // 32 keys each, three parts
                mma_ts<true>(d, pc + 32 * (x / 3) + 8 * (x % 3), kMnMajor | (vd + (x / 3) * 256), id_o, x > 0 ? 1u : acc);
            } else {
#pragma unroll
              for (int x = 0; x < 16; ++x)  // 16 keys each, high and low parts
                mma_ts<false>(d, pc + 32 * (x >> 2) + 8 * ((x >> 1) & 1) + 16 * (x & 1), kMnMajor | (vd + (x >> 1) * 128),
                              id_o, x > 0 ? 1u : acc);
            }
            if (release) {
              umma_commit(empty + at.slot);
              at.step();
            }
            if (u + 2 >= all) umma_commit(o_done + j);
          }
          if (u + 2 < all) {
            const Ring<NS> k = u >= 0 && !release ? at.ahead(1) : at;
            ok = wait(full + k.slot, k.round & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t kd = ring + k.slot * (L::SLOT >> 4), qd = q0 + (lead == 1 ? 2048u * j : 0u);
#pragma unroll
            for (int x = 0; x < 8; ++x)  // 16 dims each; 8 bits: 32 dims each, with the high, then the low codes of q
              mma_ss<E4M3>(pc, kKMajor | (qd + (x >> 2) * 1024 + (x & 3) * 2),
                           kKMajor | (kd + (E4M3 ? 0 : (x >> 2) * 1024) + (x & 3) * 2),
                           E4M3 && x >= 4 ? id_s | (1u << 7) : id_s, x > 0 ? 1u : 0u);
            umma_commit(s_full + j);
            if (release) {
              umma_commit(empty + k.slot);
              at.step();
            }
          }
        }
      }
      umma_commit(drain);
      volatile int never = 0;
      if (!mbar_wait(drain, 0, &never, kWaitNs)) flag(a.status, DFLASH2_DEV_WAIT_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---------------------------------------------------------------- tile info
    Ring<NS> vat;  // slot of the next value tile
    Ring<kInfo> iat;
    bool ok = true;
    int rows4 = -1;
    uint32_t bytes[4][4];
    SegInfo g;
    for (; ok && next_segment(&g); seg_at.step()) {
      const int lead = g.split ? 2 : 1;
      const int32_t* table = a.block_table + (size_t)g.s * a.max_pages;
      for (int x = min(lead, g.tiles); x > 0; --x) vat.step();  // lead tiles of keys go first
      // lane 8 t + i: pool row of 16-key group i of tile t0 + t, or -1
      auto rows_of = [&](int t0) {
        const int t = t0 + (lane >> 3), pos = g.first + t * kTile + 16 * (lane & 7);
        int row = -1;
        if (t < g.tiles && pos < g.end) {
          const int page = table[pos >> p.page_shift];
          if (page >= 0 && page < a.n_pages) row = (page << p.page_shift) + (pos & (a.page_size - 1));
          else flag(a.status, DFLASH2_DEV_BAD_PAGE);
        }
        return row;
      };
      int next = rows_of(0);
      // Four tiles at a time: all their exponent bytes are asked for together
      // (keys' in the low halves, values' in the high ones; keys 32 i + lane).
#pragma unroll 1
      for (int t = 0; t < g.tiles && ok; ++t) {
        const int slot = iat.slot, k0 = g.first + t * kTile;
        if ((t & 3) == 0) {
          rows4 = next;
          next = rows_of(t + 4);
          if (E4M3) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = 32 * i + lane, r = __shfl_sync(0xffffffffu, rows4, 8 * u + (key >> 4));
                uint32_t b = 0;
                if (r >= 0 && k0 + u * kTile + key < g.end) {
                  const size_t x = ((size_t)r + (key & 15)) * a.nkv + g.h;
                  b = a.k_exp[x] | ((uint32_t)a.v_exp[x] << 16);
                }
                bytes[u][i] = b;
              }
          }
        }
        TileInfo* info;
        if (E4M3) info = reinterpret_cast<TileInfo*>(sm + L::INFO + slot * L::INFOS);
        else info = reinterpret_cast<TileInfo*>(sm + L::INFO + slot * L::INFOS - offsetof(TileInfo, bad));
        const uint32_t groups = (__ballot_sync(0xffffffffu, rows4 >= 0) >> (8 * (t & 3))) & 0xffu;
        const bool mixed = k0 < g.all_lo || k0 + kTile > g.all_hi || groups != 0xffu;
        if (iat.round > 0) ok = wait(info_empty + slot, (iat.round - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (E4M3) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = (t & 2) ? ((t & 1) ? bytes[3][i] : bytes[2][i]) : ((t & 1) ? bytes[1][i] : bytes[0][i]);
            const uint32_t kb = min(x & 0xffffu, 254u), vb = min(x >> 16, 254u);
            info->ks[32 * i + lane] = __uint_as_float(kb << 23);
            info->vs[32 * i + lane] = __uint_as_float(vb << 23);
            info->lv[32 * i + lane] = (float)max((int)vb - 127, kLeastScale);
            top = max(top, vb);
          }
          top = __reduce_max_sync(0xffffffffu, top);
          if (lane == 0) info->vmax = (float)max((int)top - 127, kLeastScale);
        }
        if (lane < 4) info->bad[lane] = 0;
        if (lane == 0) {
          info->groups = groups;
          info->spoilt = 0;
        }
        __syncwarp();
        if (mixed) {
          // (This warp may be more than a round of the ring ahead of the loads,
          // and a wait for a parity takes the phase before the last for the
          // right one: it waits for the load to be issued first.)
          ok = __all_sync(0xffffffffu, wait_count(issued_at, vat.round * NS + vat.slot + 1, abort_at, a.status) &&
                                           wait(full + vat.slot, vat.round & 1));
          if (!ok) break;
          uint8_t* v = sm + L::RING + vat.slot * L::SLOT;
          // keys below `to` and from `from` on are not seen by every row; behind
          // `past` a page holds what it held before (whole absent groups are zeros)
          const int to = min(kTile, g.all_lo - k0), past = g.end - k0, top = min(kTile, (past + 15) & ~15);
          int key0 = to > 0 ? 0 : max(0, g.all_hi - k0) & ~3;
          constexpr int W = E4M3 ? 8 : 16;  // lanes of a row, 16 bytes each
          uint32_t any = 0;
#pragma unroll 1
          while (key0 < top) {
            const int key = key0 + lane / W, c = lane & (W - 1);
            uint4* q = reinterpret_cast<uint4*>(v + (E4M3 ? 0 : (c >> 3) * 16384) + key * 128 + (c & 7) * 16);
            const bool in = key < top;
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (in) {
              const uint4 x = *q;
              w[0] = x.x;
              w[1] = x.y;
              w[2] = x.z;
              w[3] = x.w;
            }
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t gone = 0;
              if (E4M3) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                  if (((w[i] >> (8 * b)) & 0x7fu) == 0x7fu) gone |= 0xffu << (8 * b);
              } else {
                if ((w[i] & 0x7f80u) == 0x7f80u) gone |= 0xffffu;
                if ((w[i] & 0x7f800000u) == 0x7f800000u) gone |= 0xffff0000u;
              }
              bad |= gone != 0;
              w[i] &= ~gone;
            }
            const bool behind = key >= past;
            if (in && (bad || behind))
              *q = behind ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(w[0], w[1], w[2], w[3]);
            const uint32_t votes = __ballot_sync(0xffffffffu, bad && !behind);
            any |= votes;
            if (lane % W == 0 && ((votes >> lane) & ((1u << W) - 1u))) atomicOr(&info->bad[key >> 5], 1u << (key & 31));
            key0 += 32 / W;
            if (key0 >= to && key0 < ((g.all_hi - k0) & ~3)) key0 = (g.all_hi - k0) & ~3;
          }
          if (lane == 0) info->spoilt = any;
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(info_full + slot);
        iat.step();
        vat.step();
        if (t + lead < g.tiles) vat.step();  // the next key tile's
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int j = warp >> 2, r = threadIdx.x & 127;  // stream, row of its tile
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float scale = a.scale * 1.4426950408889634f;
    // how far a weight may pass 2^0: times the value's scale what an e5m2
    // holds; or little against a float's range, so that large values times
    // such weights stay finite where their mean does, and enough that a new
    // reference is rare
    const float head_room = E4M3 ? 15.f : 16.f;
    uint32_t n_s = 0, n_o = 0, n_q = 0, tiles = 0;
    SegInfo g;
    for (; next_segment(&g); seg_at.step()) {
      const int nt = g.tiles;
      const bool split = g.split != 0;  // the streams share the rows
      // With few rows the 128 hold copies of them, and each copy weighs a part
      // of a tile's keys, so that all four warps of a stream have work.
      const int copies = split ? g.copies : 1, copy_rows = kTile / copies;
      const int fr = split ? r & (copy_rows - 1) : j * kTile + r;
      const int c_lo = r / copy_rows * (4 / copies), c_hi = c_lo + 4 / copies;  // its pieces of 32 keys
      const bool mine = fr < g.rows;
      const int f = g.f0 + (mine ? fr : 0);
      const int s = g.shared ? f / p.rows : g.s, local = f - s * p.rows, t_row = local / p.group;
      const int head = g.h * p.group + local - t_row * p.group;
      if (g.own_q) {
        // (many rows are a long segment, and the first segment has nothing to
        // hide the loads behind; the places are free: this warp has been through
        // its last segment, and so has every other, by the vote)
        const int w0 = split ? warp * 16 : warp * 32, w1 = min(w0 + (split ? 16 : 32), g.rows);
        if (w0 < w1)
          load_rows<E4M3>(p, g, w0, w1, sm + L::Q + (split ? g.q : j) * 32768,
                          reinterpret_cast<float*>(sm + L::QSCALE) + seg_at.slot * kRowTile);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);
      }
      int2 see = make_int2(0, INT32_MAX);  // (rows that do not exist see everything: nothing to mask)
      bool real = mine;
      float rs = scale;  // factor of a row's scores
      if (mine) {
        const int2 nl = g.shared ? lengths(a, s) : make_int2(g.n, g.len);
        real = t_row < nl.x;
        see = real ? sees(a, nl, t_row) : make_int2(0, 0);
        if (g.shared) see.y = min(see.y, a.shared_len);
        else see.x = max(see.x, a.shared_len);
      }
      if (E4M3) {
        const int bit = g.own_q ? 2 : g.q;  // (the rows' scales are other warps' work)
        wait(g.own_q ? q_ready : q_full + g.q, (n_q >> bit) & 1);
        n_q ^= 1u << bit;
        if (mine) rs *= reinterpret_cast<const float*>(sm + L::QSCALE)[seg_at.slot * kRowTile + fr];
        if (rs < 1.17549435e-38f) rs = 1.17549435e-38f;  // (never 0: a hidden key's score is -inf times that)
      }
      if (E4M3) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + seg_at.slot);
      }
      const int first = g.first;
      float ref = kNone, sum = 0.f;
      bool poison = false;
      const bool idle = !__any_sync(0xffffffffu, mine);  // no row of this warp exists
      int done = 0;  // tiles of this stream in this segment
      for (int t = split ? j : 0; t < nt; t += split ? 2 : 1, ++done) {
        const uint32_t tile = tiles + t;
        const int slot = tile % kInfo;
        const TileInfo* info;
        if (E4M3) info = reinterpret_cast<const TileInfo*>(sm + L::INFO + slot * L::INFOS);
        else info = reinterpret_cast<const TileInfo*>(sm + L::INFO + slot * L::INFOS - offsetof(TileInfo, bad));
        wait(info_full + slot, (tile / kInfo) & 1);
        wait(s_full + j, n_s & 1);
        ++n_s;
        __syncwarp();
        tc_fence_after();
        if (!idle) {
          const int k0 = first + t * kTile;
          const int v0 = see.x - k0, v1 = see.y > k0 + kTile ? kTile : see.y - k0;  // keys of the tile that it sees
          const uint32_t groups = info->groups;
          // (a mended value is seen by rows that the whole tile is open to, too: other warps' rows made it a mended tile)
          const bool cut =
              __any_sync(0xffffffffu, mine && (v0 > 0 || v1 < kTile)) || groups != 0xffu || info->spoilt != 0;
          // bit i: key 32 c + i is seen
          auto seen = [&](int c) {
            const int from = min(32, max(0, v0 - 32 * c)), to = min(32, max(0, v1 - 32 * c));
            uint32_t m = (to == 32 ? 0xffffffffu : (1u << to) - 1u) & (from == 32 ? 0u : 0xffffffffu << from);
            if (!((groups >> (2 * c)) & 1)) m &= 0xffff0000u;
            if (!((groups >> (2 * c + 1)) & 1)) m &= 0x0000ffffu;
            return m;
          };
          uint64_t part[2] = {0ull, 0ull};  // sums of weights, two each
          const uint64_t rs2 = pack2(rs, rs);
          // 32 keys: their scores become weights in the same TMEM columns
          auto weigh = [&](int c, float (&x)[32]) {
            if (E4M3) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(info->ks + 32 * c + i);
                unpack2(mul2(pack2(x[i], x[i + 1]), k4.x), x[i], x[i + 1]);
                unpack2(mul2(pack2(x[i + 2], x[i + 3]), k4.y), x[i + 2], x[i + 3]);
              }
            }
            if (cut) {
              const uint32_t m = seen(c);
              poison |= (info->bad[c] & m) != 0;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((m >> i) & 1)) x[i] = kNone;
            }
            float y[11];
#pragma unroll
            for (int i = 0; i < 10; ++i) y[i] = max3(x[3 * i], x[3 * i + 1], x[3 * i + 2]);
            y[10] = fmaxf(x[30], x[31]);
            float top = max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), max3(max3(y[6], y[7], y[8]), y[9], y[10])) * rs;
            if (E4M3) top += info->vmax;
            bool over = __any_sync(0xffffffffu, mine && top > ref + head_room);
            if (E4M3 && over) {
              // (only a bound: the largest scale may be that of a key with a
              // small weight, or of one that the row does not see, whose page
              // may hold anything.  The reference comes from the keys' own.)
              top = kNone;
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const ulonglong2 l4 = *reinterpret_cast<const ulonglong2*>(info->lv + 32 * c + i);
                float a0, a1, a2, a3;
                unpack2(fma2(pack2(x[i], x[i + 1]), rs2, l4.x), a0, a1);
                unpack2(fma2(pack2(x[i + 2], x[i + 3]), rs2, l4.y), a2, a3);
                top = max3(max3(top, a0, a1), a2, a3);
              }
              over = __any_sync(0xffffffffu, mine && top > ref + head_room);
            }
            if (over) {
              // a new reference (a whole number, so that what is scaled to it
              // stays exact).  The products of the stream's last tile are
              // done: this tile's scores were issued behind them.
              const float now = fmaxf(ref, ceilf(top) - (E4M3 ? 11.f : 0.f));
              const float by = ref == kNone ? 0.f : ex2(ref - now);
              sum *= by;
              part[0] = mul2(part[0], pack2(by, by));
              part[1] = mul2(part[1], pack2(by, by));
              ref = now;
              rescale<E4M3>(lanes + o_col(j), done > 0 ? 4 : 0, lanes + s_col(j), c, by);
            }
            const float sub = ref == kNone ? 0.f : -ref;
            const uint64_t sub2 = pack2(sub, sub);
            if (E4M3) {
              uint32_t w[3][8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {  // four keys: a column of each part
                const ulonglong2 v4 = *reinterpret_cast<const ulonglong2*>(info->vs + 32 * c + 4 * i);
                uint32_t h[2][3];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  float p0, p1;
                  unpack2(fma2(pack2(x[4 * i + 2 * b], x[4 * i + 2 * b + 1]), rs2, sub2), p0, p1);
                  const uint64_t pp = pack2(ex2(p0), ex2(p1));
                  part[b] = add2(part[b], pp);
                  unpack2(mul2(pp, b ? v4.y : v4.x), p0, p1);
                  split3(__floats2half2_rn(p0, p1), h[b]);
                }
#pragma unroll
                for (int q = 0; q < 3; ++q) w[q][i] = __byte_perm(h[0][q], h[1][q], 0x7531);
              }
#pragma unroll
              for (int q = 0; q < 3; ++q) tmem_st8(lanes + s_col(j) + 32 * c + 8 * q, w[q]);
            } else {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {  // 16 keys: 8 columns of high and of low parts
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  float p0, p1;
                  unpack2(fma2(pack2(x[16 * hf + 2 * i], x[16 * hf + 2 * i + 1]), rs2, sub2), p0, p1);
                  p0 = ex2(p0);
                  p1 = ex2(p1);
                  const uint64_t pp = pack2(p0, p1);
                  part[i & 1] = add2(part[i & 1], pp);
                  const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                  hi[i] = __byte_perm(b0, b1, 0x7632);  // cut to the top 16 bits; what is left is exact
                  unpack2(add2(pp, pack2(__uint_as_float((b0 & 0xffff0000u) ^ 0x80000000u),
                                         __uint_as_float((b1 & 0xffff0000u) ^ 0x80000000u))), p0, p1);
                  lo[i] = bits2(__floats2bfloat162_rn(p0, p1));
                }
                tmem_st8(lanes + s_col(j) + 32 * c + 8 * hf, hi);
                tmem_st8(lanes + s_col(j) + 32 * c + 16 + 8 * hf, lo);
              }
            }
          };
          // One pass: a weight may be larger than 1, so the reference need not
          // be the maximum, only near enough.
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (c < c_lo || c >= c_hi) {  // (the whole warp: copies are of 32 rows or more)
              const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
              for (int q = 0; q < (E4M3 ? 3 : 4); ++q) tmem_st8(lanes + s_col(j) + 32 * c + 8 * q, none);
              continue;
            }
            float x[32];
            tmem_ld32(lanes + s_col(j) + 32 * c, x);
            tmem_ld_wait();
            weigh(c, x);
          }
          float s0, s1;
          unpack2(add2(part[0], part[1]), s0, s1);
          sum += s0 + s1;
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_ready + j);
          mbar_arrive_n(info_empty + slot, split ? 2 : 1);
        }
      }
      tiles += nt;
      // ------------------------------------------------ the segment's end
      const bool both = split && nt > 1;
      if (done > 0) {
        wait(o_done + j, n_o & 1);
        ++n_o;
      }
      if (poison) sum = __int_as_float(0x7fffffff);
      const bool whole = g.slot < 0;
      if (!split) {
        tc_fence_after();
        if (!idle) {
          float* part = nullptr;
          if (!whole) {
            const size_t row = (size_t)g.slot * (g.shared ? kRowTile : p.slot_rows) + fr;
            part = (g.shared ? p.part_p : p.part_s) + row * kD;
            if (mine) (g.shared ? p.ref_p : p.ref_s)[row] = make_float2(ref, sum);
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          bf16* orow = a.out + ((size_t)s * a.n_tok + t_row) * a.out_stride + (size_t)head * kD;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32(lanes + o_col(j) + 32 * c, o);
            tmem_ld_wait();
            if (whole) {
              if (real) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t w[4];
#pragma unroll
                  for (int b = 0; b < 4; ++b)
                    w[b] = sum == 0.f ? 0u : bits2(__floats2bfloat162_rn(o[8 * i + 2 * b] * inv, o[8 * i + 2 * b + 1] * inv));
                  reinterpret_cast<uint4*>(orow + 32 * c)[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            } else if (mine) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4*>(part + 32 * c)[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(q_empty);
          mbar_arrive(q_empty + 1);
        }
      } else {
        // A row's parts are in both streams and in every copy.  They meet in
        // the place of the query rows, whose products are done.
        float2* xch = reinterpret_cast<float2*>(sm + L::Q + g.q * 32768);
        bar_softmax();  // both streams' products
        xch[j * kTile + r] = make_float2(ref, sum);
        tc_fence_before();
        bar_softmax();
        tc_fence_after();
        // (a stream without tiles has no reference, and its accumulator is not read)
        const float mine0 = xch[r].x, mine1 = both ? xch[kTile + r].x : kNone;
        ref = kNone;
        sum = 0.f;
        for (int i = fr; i < 2 * kTile; i += copy_rows)
          if (i < kTile || both) ref = fmaxf(ref, xch[i].x);
        const float base = ref == kNone ? 0.f : ref;
        for (int i = fr; i < 2 * kTile; i += copy_rows)
          if (i < kTile || both) sum = fmaf(xch[i].y, ex2(xch[i].x - base), sum);
        const float w0 = ex2(mine0 - base), w1 = ex2(mine1 - base);
        if (!whole && j == 0 && r < copy_rows && mine) {
          const size_t row = (size_t)g.slot * (g.shared ? kRowTile : p.slot_rows) + fr;
          (g.shared ? p.ref_p : p.ref_s)[row] = make_float2(ref, sum);
        }
        // factor of the result: with `whole` the row's 1 / sum, in every copy
        const float fin = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        // Stream j's warps take dims 64 j .. 64 j + 63, 32 at a time: both
        // accumulators' into shared memory (pieces of 16 bytes at piece ^
        // row % 8), then the sums over the copies, out.
        float4* box = reinterpret_cast<float4*>(sm + L::Q + g.q * 32768 + j * 16384);
        const float f0 = sum == 0.f ? 0.f : w0 * fin, f1 = sum == 0.f ? 0.f : w1 * fin;
        bar_softmax();  // everyone has read the references and sums
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const int c = 2 * j + part;
          if (!idle) {
#pragma unroll 1
            for (int i = 0; i < 8; i += 2) {  // (small pieces: code that runs once a segment is slow to fetch)
              uint32_t o0[8], o1[8];
              float o[8];
              tmem_ld8_nowait(lanes + o_col(0) + 32 * c + 4 * i, o0);
              if (both) tmem_ld8_nowait(lanes + o_col(1) + 32 * c + 4 * i, o1);
              tmem_ld_wait();
#pragma unroll
              for (int b = 0; b < 8; ++b) {
                o[b] = __uint_as_float(o0[b]) * f0;
                if (both) o[b] = fmaf(__uint_as_float(o1[b]), f1, o[b]);
                if (sum == 0.f) o[b] = 0.f;
              }
              box[r * 8 + (i ^ (r & 7))] = make_float4(o[0], o[1], o[2], o[3]);
              box[r * 8 + ((i + 1) ^ (r & 7))] = make_float4(o[4], o[5], o[6], o[7]);
            }
          }
          bar_stream(j);
          for (int i = r; i < g.rows * 8; i += kTile) {
            const int row = i >> 3, piece = i & 7;
            float4 x = box[row * 8 + (piece ^ (row & 7))];
            for (int cp = copy_rows; cp < kTile; cp += copy_rows) {
              const float4 y = box[(cp + row) * 8 + (piece ^ (row & 7))];
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
            if (!whole) {
              const size_t at = ((size_t)g.slot * (g.shared ? kRowTile : p.slot_rows) + row) * kD + 32 * c + 4 * piece;
              *reinterpret_cast<float4*>((g.shared ? p.part_p : p.part_s) + at) = x;
            } else {  // (a sequence's own rows)
              const int lr = g.f0 + row - g.s * p.rows, t = lr / p.group;
              uint2 y;
              y.x = bits2(__floats2bfloat162_rn(x.x, x.y));
              y.y = bits2(__floats2bfloat162_rn(x.z, x.w));
              *reinterpret_cast<uint2*>(a.out + ((size_t)g.s * a.n_tok + t) * a.out_stride +
                                        (size_t)(g.h * p.group + lr - t * p.group) * kD + 32 * c + 4 * piece) = y;
            }
          }
          bar_stream(j);  // (the box has been read)
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty + g.q);
      }
      tc_fence_before();
      if (split) bar_softmax();  // both streams have read both accumulators
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ joining kernel

// A block per 32 rows of a segment of the sequences: the partial accumulators,
// weighted to a common reference.  Segments that one CTA finished are there
// already.  The CTAs that have parts of it are found by all threads at once,
// and a warp takes four rows at a time, so that their loads overlap.
constexpr int kJoinRows = 32;

__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ Plan p, int nctas) {
  __shared__ uint32_t has[3][(kMaxCtas + 31) / 32];  // CTAs with parts: the sequence's, and of two row tiles of the shared part
  pdl_launch_next();
  pdl_wait();
  const AttendArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int entry = blockIdx.x / a.nkv, h = blockIdx.x - entry * a.nkv;
  const int s = p.tiles_s == 1 ? entry : entry / p.tiles_s, i = entry - s * p.tiles_s;
  const int2 nl = lengths(a, s);
  const int units = p.head[0], tiles_p = p.head[1], start = p.head[2 + entry];
  const Segment g = segment_of(a, p.group, nl, i);
  const int rows = min(kRowTile, nl.x * p.group - i * kRowTile);
  if ((int)blockIdx.y * kJoinRows >= rows) return;
  const int w = weight_of(g.rows), wp = weight_of(kRowTile), f0 = s * p.rows + i * kRowTile;
  const int at = start + h * cost_of(p.seg_cost, g.tiles, w), ip = f0 / kRowTile, cost_p = cost_of(p.seg_cost, tiles_p, wp);
  // (a block looks at one CTA per thread)
  uint32_t mine = 0;
  // the CTA that has the segment's first tile
  const int c_first = g.tiles > 0 ? owner_of(units, at + p.seg_cost, nctas) : -1;
  {
    const int c = threadIdx.x;
    bool own = false, p0 = false, p1 = false;
    if (c < nctas) {
      const int lo = bound_of(units, c, nctas), hi = bound_of(units, c + 1, nctas);
      if (g.tiles > 0) {
        const int2 k = tiles_in(p.seg_cost, at, g.tiles, w, lo, hi);
        own = k.x < k.y && (p.tiles_p > 0 || k.x > 0 || k.y < g.tiles);
      }
      if (tiles_p > 0) {
        int2 k = tiles_in(p.seg_cost, (ip * a.nkv + h) * cost_p, tiles_p, wp, lo, hi);
        p0 = k.x < k.y;
        k = tiles_in(p.seg_cost, ((ip + 1) * a.nkv + h) * cost_p, tiles_p, wp, lo, hi);
        p1 = k.x < k.y;
      }
    }
    const uint32_t m0 = __ballot_sync(0xffffffffu, own), m1 = __ballot_sync(0xffffffffu, p0),
                   m2 = __ballot_sync(0xffffffffu, p1);
    if (lane == 0) {
      has[0][warp] = m0;
      has[1][warp] = m1;
      has[2][warp] = m2;
    }
    mine = m0;
  }
  const bool any = __syncthreads_or(mine);
  if (!any && g.tiles > 0 && p.tiles_p == 0) return;  // one CTA has written it (without tiles nobody has: zeros)
  constexpr int RW = kJoinRows / 8;
  {
    const int r0 = blockIdx.y * kJoinRows + warp;
    float ref[RW], sum[RW];
    float4 o[RW];
#pragma unroll
    for (int u = 0; u < RW; ++u) {
      ref[u] = kNone;
      sum[u] = 0.f;
      o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {
#pragma unroll 1
      for (int word = 0; word < (nctas + 31) / 32; ++word) {
        uint32_t m = has[kind][word];
        while (m) {
          const int c = word * 32 + __ffs(m) - 1;
          m &= m - 1;
          float2 rl[RW];
          float4 x[RW];
#pragma unroll
          for (int u = 0; u < RW; ++u) {
            const int r = r0 + 8 * u, f = f0 + r;
            // (rows of a segment may lie in two row tiles of the shared part)
            const bool in = r < rows && (kind == 0 || f / kRowTile == ip + kind - 1);
            rl[u] = make_float2(kNone, 0.f);
            x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) {
              const size_t row = kind == 0 ? (size_t)slot_of(p, entry * a.nkv + h, c, c == c_first) * p.slot_rows + r
                                           : (size_t)((ip + kind - 1) * a.nkv + h + c) * kRowTile + f % kRowTile;
              rl[u] = (kind == 0 ? p.ref_s : p.ref_p)[row];
              x[u] = reinterpret_cast<const float4*>((kind == 0 ? p.part_s : p.part_p) + row * kD)[lane];
            }
          }
#pragma unroll
          for (int u = 0; u < RW; ++u) {
            if (rl[u].y == 0.f) continue;
            const float now = fmaxf(ref[u], rl[u].x), base = now == kNone ? 0.f : now;
            const float fo = ex2(ref[u] - base), fx = ex2(rl[u].x - base);
            sum[u] = fmaf(sum[u], fo, rl[u].y * fx);
            o[u].x = fmaf(o[u].x, fo, x[u].x * fx);
            o[u].y = fmaf(o[u].y, fo, x[u].y * fx);
            o[u].z = fmaf(o[u].z, fo, x[u].z * fx);
            o[u].w = fmaf(o[u].w, fo, x[u].w * fx);
            ref[u] = now;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < RW; ++u) {
      const int r = r0 + 8 * u;
      if (r >= rows) continue;
      const int lr = i * kRowTile + r, t = lr / p.group;
      const float inv = sum[u] == 0.f ? 0.f : 1.f / sum[u];
      uint2 y;
      y.x = sum[u] == 0.f ? 0u : bits2(__floats2bfloat162_rn(o[u].x * inv, o[u].y * inv));
      y.y = sum[u] == 0.f ? 0u : bits2(__floats2bfloat162_rn(o[u].z * inv, o[u].w * inv));
      reinterpret_cast<uint2*>(a.out + ((size_t)s * a.n_tok + t) * a.out_stride + (size_t)(h * p.group + lr - t * p.group) * kD)[lane] = y;
    }
  }
}

// ------------------------------------------------------------------ host

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Sizes of a call's parts; `ctas` as large as any device's.
struct Sizes {
  int rows, tiles_p, tiles_s, slot_rows;
  size_t head, part_p, part_s, ref_p, ref_s, total;
};
bool sizes_of(int batch, int n_tok, int nq, int nkv, int shared_len, int ctas, Sizes* z) {
  const long long rows = (long long)n_tok * (nq / nkv);
  if (rows * batch >= (1ll << 31) - 512) return false;
  z->rows = (int)rows;
  const int rt = kRowTile;
  z->tiles_s = (int)((rows + rt - 1) / rt);
  z->tiles_p = shared_len > 0 ? (int)((rows * batch + rt - 1) / rt) : 0;
  z->slot_rows = (int)std::min<long long>(rt, rows);
  const long long segs_s = (long long)batch * z->tiles_s * nkv, segs_p = (long long)z->tiles_p * nkv;
  if (segs_s > (1 << 30) || segs_p > (1 << 30)) return false;
  const size_t n_s = (size_t)(z->tiles_p ? segs_s + ctas : 2 * ctas) * z->slot_rows, n_p = z->tiles_p ? (size_t)(segs_p + ctas) * rt : 0;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += align256(bytes);
    return x;
  };
  z->head = take((2 + (size_t)batch * z->tiles_s) * 4);
  z->ref_p = take(n_p * 8);
  z->ref_s = take(n_s * 8);
  z->part_p = take(n_p * kD * 4);
  z->part_s = take(n_s * kD * 4);
  z->total = at;
  return true;
}

template <bool E4M3>
int launch(const Plan& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Ctx& c) {
  // an attribute of the kernel on the current device: set on every call (a
  // flag of what was set would have to be kept per device)
  if (cudaFuncSetAttribute(attend_tc_kernel<E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)Smem<E4M3>::bytes) != cudaSuccess)
    return DFLASH2_ERR_CUDA;
  const int rc = launch_k(attend_tc_kernel<E4M3>, dim3(c.nsm), dim3(kThreads), Smem<E4M3>::bytes, c, p, tm_k, tm_v);
  if (rc != DFLASH2_OK) return rc;
  return launch_k(attend_join_kernel, dim3(p.a.batch * p.tiles_s * p.a.nkv, (p.slot_rows + kJoinRows - 1) / kJoinRows),
                  dim3(256), 0, c, p, c.nsm);
}

}  // namespace

bool attend_tc_fits(const AttendArgs& a) {
  if (a.d != kD || a.page_size < 16 || (a.page_size & (a.page_size - 1)) || (long long)a.n_pages * a.page_size >= (1ll << 31) - 256) return false;
  // positions of tiles are 32-bit: the most that the block table allows
  Sizes z;
  if (!sizes_of(a.batch, a.n_tok, a.nq, a.nkv, a.shared_len, kMaxCtas, &z)) return false;
  const long long each = ((long long)a.max_pages * a.page_size + 15) / kTile + 2;
  return ((long long)a.batch * z.tiles_s + z.tiles_p) * a.nkv * (each * 4 + 32) < (1ll << 31);
}

size_t attend_tc_workspace(int batch, int n_tok, int nq, int nkv, int shared_len) {
  Sizes z;
  return sizes_of(batch, n_tok, nq, nkv, shared_len, kMaxCtas, &z) ? z.total : 0;
}

int launch_attend_tc(const AttendArgs& a, void* workspace, const Ctx& c) {
  Sizes z;
  if (!sizes_of(a.batch, a.n_tok, a.nq, a.nkv, a.shared_len, kMaxCtas, &z)) return DFLASH2_ERR_SHAPE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Plan p = {};
  p.a = a;
  p.group = a.nq / a.nkv;
  p.rows = z.rows;
  p.tiles_p = z.tiles_p;
  p.tiles_s = z.tiles_s;
  p.slot_rows = z.slot_rows;
  p.seg_cost = a.e4m3 ? 16 : 7;
  while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
  p.head = reinterpret_cast<int*>(ws + z.head);
  p.part_p = reinterpret_cast<float*>(ws + z.part_p);
  p.part_s = reinterpret_cast<float*>(ws + z.part_s);
  p.ref_p = reinterpret_cast<float2*>(ws + z.ref_p);
  p.ref_s = reinterpret_cast<float2*>(ws + z.ref_s);
  // the pools as rows of 2-byte elements (8-bit rows: pairs of codes)
  const int cols = a.nkv * (a.e4m3 ? kD / 2 : kD);
  CUtensorMap tm_k, tm_v;
  const long long rows = (long long)a.n_pages * a.page_size;
  int rc = make_sw128_map(&tm_k, a.k, rows, cols, cols, 16);
  if (rc == DFLASH2_OK) rc = make_sw128_map(&tm_v, a.v, rows, cols, cols, 16);
  if (rc != DFLASH2_OK) return rc;
  return a.e4m3 ? launch<true>(p, tm_k, tm_v, c) : launch<false>(p, tm_k, tm_v, c);
}

}  // namespace df2
