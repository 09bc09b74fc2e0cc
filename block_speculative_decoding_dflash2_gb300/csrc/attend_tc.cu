// Attention of a sequence's last tokens over its paged cache on the
// 5th-generation tensor cores: head dimension 128, pages of whole 16-key
// groups, bfloat16 or 8-bit rows.
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
// with V, so that its rounding (2^-17) does not add to the output's.  8-bit:
// the codes are multiplied as they are, no byte of the cache is converted.
// q is split into two e4m3 codes (its 8 bits are 4 + 4: exact but for values
// below 2^-17 of the row's largest) and P, times the key's value scale, into
// three e5m2 codes (3 + 3 + 3 bits, 2^-9 of each weight over 2^30 of range).
// The scales of keys multiply the scores; those of values the weights.
//
// Warps: 0-3 and 4-7 softmax of stream 0 and 1 (thread = query row), 8 loads
// by TMA, 9 TMEM and MMA issue, 10 what a tile needs beside its rows: which
// 16-key groups exist, the scales, and, in tiles that hold keys which some
// row does not see, zeros for values that are not finite (a zero weight
// would turn them into NaN; rows that do see one are marked).
#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kTile = 128;  // keys of a tile, query rows of a stream
constexpr int kD = 128;     // head dimension
constexpr int kSoftmax = 256;
constexpr int kThreads = kSoftmax + 128;  // (the last warp only fills its group of four)
// registers a thread: 384 threads start with 168 (64512 in all), of which the
// softmax groups take 208 (53248) and the others keep 88 (11264)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kInfo = 4;  // tiles ahead of which warp 10 may run
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kMaxCtas = kMaxSM;
constexpr float kNone = -INFINITY;

// TMEM columns: scores (then weights) and accumulators of the two streams
__device__ constexpr uint32_t s_col(int j) { return 128u * j; }
__device__ constexpr uint32_t o_col(int j) { return 256u + 128u * j; }

struct TileInfo {
  float ks[kTile], vs[kTile];  // scales 2^(byte - 127) of keys and values
  uint32_t bad[4];             // keys whose values were not finite and are zeros now
  uint32_t groups;             // bit i: 16-key group i exists
  float vmax;                  // log2 of the largest value scale (at least -60)
  uint32_t mixed;              // some row does not see some key
  uint32_t pad;
};

template <bool E4M3, int QT>
struct Smem {
  static constexpr int Q = 0;                                  // [QT][32 KB]
  static constexpr int SLOT = E4M3 ? 16384 : 32768;            // K or V of a tile
  static constexpr int SLOTS = E4M3 ? (QT == 2 ? 9 : 11) : (QT == 2 ? 5 : 6);
  static constexpr int RING = QT * 32768;
  static constexpr int INFO = RING + SLOTS * SLOT;
  static constexpr int INFOS = E4M3 ? (int)sizeof(TileInfo) : 32;  // bf16 keeps the tail of TileInfo only
  static constexpr int BAR = INFO + kInfo * INFOS;
  static constexpr size_t bytes = 1024 + BAR + (2 * SLOTS + 2 * kInfo + 8) * 8 + 64;
  static_assert(bytes + 512 <= 227 * 1024, "shared memory");
};

struct Plan {
  AttendArgs a;
  int group, rows;     // query heads per kv head; query rows (n_tok * group) of a sequence
  int tiles_p;         // row tiles of the shared part (0: none)
  int tiles_s;         // row tiles of a sequence at most
  int row_weight;      // cost of a tile for more than 128 rows, in tiles for fewer
  int slot_rows;       // rows of a sequence's partial slot
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

// Row tile i of sequence s (positions from shared_len on).
template <int QT>
__device__ __forceinline__ Segment segment_of(const AttendArgs& a, int group, int2 nl, int i) {
  Segment g = {0, 0, 0, 0};
  const int first = i * (kTile * QT), all = nl.x * group;
  if (first >= all) return g;
  g.rows = min(kTile * QT, all - first);
  const int lo = max(sees(a, nl, first / group).x, a.shared_len);
  const int hi = sees(a, nl, (first + g.rows - 1) / group).y;
  if (hi <= lo) return g;
  g.base = lo & ~15;
  g.end = hi;
  g.tiles = (hi - g.base + kTile - 1) / kTile;
  return g;
}
__device__ __forceinline__ int weight_of(const Plan& p, int rows) { return rows > kTile ? p.row_weight : 1; }

// Share of CTA c of n: tiles whose position lies in [bound(c), bound(c + 1)).
// (positions fit 31 bits: the host sees to it)
__device__ __forceinline__ int bound_of(int units, int c, int n) { return (int)((long long)units * c / n); }
__device__ __forceinline__ int owner_of(int units, int x, int n) {
  return (int)((((long long)x + 1) * n - 1) / units);
}

// Walks a CTA's segments; every role walks for itself.
template <int QT>
struct Walk {
  const Plan* p;
  int a, b, at;  // this CTA's share; position of the current segment's first tile
  int base_p, tiles_p, end_p;
  int entry, h;        // row tile (shared part first) and kv head
  int2 nl;
  Segment g;
  int w;
  int k0, k1;  // this CTA's tiles of it

  __device__ __forceinline__ int s() const { return (entry - p->tiles_p) / p->tiles_s; }
  __device__ __forceinline__ bool shared() const { return entry < p->tiles_p; }
  __device__ __forceinline__ int first_row() const {  // flat query row (sequence, token, head of the group)
    return shared() ? entry * (kTile * QT) : s() * p->rows + (entry - p->tiles_p) % p->tiles_s * (kTile * QT);
  }
  __device__ __forceinline__ int ordinal() const { return (shared() ? entry : entry - p->tiles_p) * p->a.nkv + h; }
  __device__ __forceinline__ void load() {  // segment of `entry`
    if (shared()) {
      g.rows = (int)min((long long)kTile * QT, (long long)p->a.batch * p->rows - (long long)entry * (kTile * QT));
      g.base = base_p;
      g.tiles = tiles_p;
      g.end = end_p;
      w = QT == 2 ? p->row_weight : 1;
    } else {
      nl = lengths(p->a, s());
      g = segment_of<QT>(p->a, p->group, nl, (entry - p->tiles_p) % p->tiles_s);
      w = weight_of(*p, g.rows);
    }
  }
  // Moves to the next segment with tiles of this CTA; `fresh`: the first call.
  __device__ __forceinline__ bool next(bool fresh) {
    const int entries = p->tiles_p + p->a.batch * p->tiles_s;
    if (!fresh) {
      at += g.tiles * w;
      if (++h == p->a.nkv) {
        h = 0;
        ++entry;
        if (entry < entries) load();
      }
    } else if (entry < entries) {
      load();
    }
    while (at < b && entry < entries) {
      const int size = g.tiles * w;
      if (size == 0) {  // (all heads alike)
        h = 0;
        if (++entry < entries) load();
        continue;
      }
      if (at + size > a) {
        k0 = at >= a ? 0 : (a - at + w - 1) / w;
        k1 = min(g.tiles, (b - at + w - 1) / w);
        if (k0 < k1) return true;
      }
      at += size;
      if (++h == p->a.nkv) {
        h = 0;
        if (++entry < entries) load();
      }
    }
    return false;
  }
};

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

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// D += A B: A from TMEM or shared memory; kind::f16 or kind::f8f6f4
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

// ------------------------------------------------------------------ main kernel

template <bool E4M3, int QT>
__global__ void __launch_bounds__(kThreads, 1) attend_tc_kernel(const Plan p, const __grid_constant__ CUtensorMap tm_k,
                                                               const __grid_constant__ CUtensorMap tm_v) {
  using L = Smem<E4M3, QT>;
  constexpr int NS = L::SLOTS;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* full = bars;              // [NS] a K or V tile landed
  uint64_t* empty = full + NS;        // [NS] its products are done
  uint64_t* info_full = empty + NS;   // [kInfo] tile info is there (and V mended)
  uint64_t* info_empty = info_full + kInfo;
  uint64_t* s_full = info_empty + kInfo;  // [2] scores of a stream's tile in TMEM
  uint64_t* p_ready = s_full + 2;         // [2] its weights in TMEM (4 arrivals)
  uint64_t* o_done = p_ready + 2;         // [2] a segment's last product of the stream is done
  uint64_t* q_ready = o_done + 2;         // query rows in shared memory (8 arrivals)
  uint64_t* drain = q_ready + 1;          // every product issued is done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ int start_at[2];
  __shared__ int scan[kThreads / 32 + 1];
  __shared__ int start_entry;

  const AttendArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, nctas = gridDim.x;
  pdl_launch_next();
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(info_full + i, 1);
      mbar_init(info_empty + i, 8);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(s_full + j, 1);
      mbar_init(p_ready + j, 4);
      mbar_init(o_done + j, 1);
    }
    mbar_init(q_ready, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();

  // ------------------------------------------------ shares of the work
  Walk<QT> wk;
  wk.p = &p;
  const int entries = a.batch * p.tiles_s;  // row tiles of the sequences
  const int per = (entries + kThreads - 1) / kThreads, e0 = min(entries, (int)threadIdx.x * per);
  const int e1 = min(entries, e0 + per);
  {
    int sum = 0;
    int lo = INT32_MAX, hi = 0;
    for (int e = e0; e < e1; ++e) {
      const int s = e / p.tiles_s;
      const int2 nl = lengths(a, s);
      if (cta == 0 && e % p.tiles_s == 0 && (a.kv_len[s] < 0 || a.kv_len[s] != nl.y)) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
      const Segment g = segment_of<QT>(a, p.group, nl, e % p.tiles_s);
      sum += g.tiles * weight_of(p, g.rows) * a.nkv;
      if (nl.x > 0) {
        lo = min(lo, sees(a, nl, 0).x);
        hi = max(hi, sees(a, nl, nl.x - 1).y);
      }
    }
    // block scan of the sums; minimum and maximum of the shared part's keys
    int inc = sum;
    int mn = lo, mx = hi;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
      mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    int* ends = reinterpret_cast<int*>(sm);  // (the query rows' place, not in use yet)
    if (lane == 31) scan[warp + 1] = inc;
    if (lane == 0) {
      ends[2 * warp] = mn;
      ends[2 * warp + 1] = mx;
    }
    if (threadIdx.x == 0) {
      scan[0] = 0;
      start_entry = p.tiles_p + entries;
    }
    __syncthreads();
    int before = inc - sum, total = 0;
    mn = INT32_MAX;
    mx = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += scan[i + 1];
      total += scan[i + 1];
      mn = min(mn, ends[2 * i]);
      mx = max(mx, ends[2 * i + 1]);
    }
    mx = min(mx, a.shared_len);
    wk.base_p = mn & ~15;
    wk.end_p = mx;
    wk.tiles_p = p.tiles_p > 0 && mx > mn ? (mx - wk.base_p + kTile - 1) / kTile : 0;
    const int wp = QT == 2 ? p.row_weight : 1;
    const int up = p.tiles_p * a.nkv * wk.tiles_p * wp;
    const int units = up + total;
    wk.a = bound_of(units, cta, nctas);
    wk.b = bound_of(units, cta + 1, nctas);
    if (cta == 0) {  // for the joining kernel
      if (threadIdx.x == 0) {
        p.head[0] = units;
        p.head[1] = wk.tiles_p;
      }
      int x = up + before;
      for (int e = e0; e < e1; ++e) {
        p.head[2 + e] = x;
        const Segment g = segment_of<QT>(a, p.group, lengths(a, e / p.tiles_s), e % p.tiles_s);
        x += g.tiles * weight_of(p, g.rows) * a.nkv;
      }
    }
    // the entry and head in which this CTA's share starts
    if (wk.a < up) {
      const int each = wk.tiles_p * wp, seg = wk.a / each;
      if (threadIdx.x == 0) {
        start_entry = seg / a.nkv;
        start_at[0] = seg * each;
        start_at[1] = seg % a.nkv;
      }
    } else if (wk.a < wk.b) {
      const int x = wk.a - up;
      if (sum > 0 && before <= x && x < before + sum) {
        int y = before;
        for (int e = e0; e < e1; ++e) {
          const Segment g = segment_of<QT>(a, p.group, lengths(a, e / p.tiles_s), e % p.tiles_s);
          const int each = g.tiles * weight_of(p, g.rows);
          if (x < y + each * a.nkv) {
            const int hh = (x - y) / each;
            start_entry = p.tiles_p + e;
            start_at[0] = up + y + hh * each;
            start_at[1] = hh;
            break;
          }
          y += each * a.nkv;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wk.entry = start_entry;
  wk.at = start_at[0];
  wk.h = start_at[1];
  if (wk.a >= wk.b) wk.entry = p.tiles_p + entries;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity, abort_flag, kWaitNs)) return true;
    if (!*abort_flag) {
      *abort_flag = 1;
      flag(a.status, DFLASH2_DEV_WAIT_TIMEOUT);
    }
    return false;
  };
  // keys a tile of which is ahead of the weights': the streams' first tiles
  auto lead_of = [&]() { return QT == 2 && wk.g.rows > kTile ? 1 : 2; };

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 8) {
    // ---------------------------------------------------------------- loads
    const uint64_t pol = policy_evict_first();
    const int absent = a.n_pages * a.page_size;  // a row past the pool: the copy fills zeros
    Ring<NS> at;
    bool ok = true;
    for (bool more = wk.next(true); more && ok; more = wk.next(false)) {
      const int nt = wk.k1 - wk.k0, lead = lead_of();
      const int32_t* table = a.block_table + (size_t)(wk.shared() ? 0 : wk.s()) * a.max_pages;
      auto load = [&](int t, bool value) {
        const int slot = at.slot;
        int row = absent;
        if (lane < 8) {
          const int pos = wk.g.base + (wk.k0 + t) * kTile + 16 * lane;
          if (pos < wk.g.end) {
            const int page = table[pos / a.page_size];
            if (page >= 0 && page < a.n_pages) row = page * a.page_size + pos % a.page_size;
          }
        }
        if (at.round > 0) ok = wait(empty + slot, (at.round - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        uint8_t* dst = sm + L::RING + slot * L::SLOT;
        if (lane == 0) mbar_arrive_expect_tx(full + slot, L::SLOT);
        __syncwarp();
        const void* map = value ? &tm_v : &tm_k;
        if (E4M3) {
          if (lane < 8) tma_load_2d(dst + lane * 2048, map, full + slot, wk.h * 64, row, pol);
        } else {
          const int r = __shfl_sync(0xffffffffu, row, lane & 7);
          if (lane < 16)
            tma_load_2d(dst + (lane >> 3) * 16384 + (lane & 7) * 2048, map, full + slot, wk.h * 128 + (lane >> 3) * 64,
                        r, pol);
        }
        at.step();
      };
      for (int t = -lead; t < nt && ok; ++t) {
        if (t >= 0) load(t, true);
        if (t + lead < nt && ok) load(t + lead, false);
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
    if (lane == 0) {
      const uint32_t ring = smem_u32(sm + L::RING), qs = smem_u32(sm + L::Q);
      // A K-major, B = K rows K-major; B = V rows MN-major; 8-bit weights are e5m2
      const uint32_t id_s = E4M3 ? (1u << 4) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24) : idesc_bf16_f32(kTile, kTile);
      const uint32_t id_o =
          (E4M3 ? (1u << 4) | (1u << 7) | ((kD >> 3) << 17) | ((kTile >> 4) << 24) : idesc_bf16_f32(kTile, kD)) |
          (1u << 16);
      Ring<NS> at;
      uint32_t n_p = 0, segs = 0;  // bit j: parity of stream j's weights
      bool ok = true;
      for (bool more = wk.next(true); more && ok; more = wk.next(false)) {
        const int nt = wk.k1 - wk.k0, lead = lead_of();
        ok = wait(q_ready, segs & 1);
        ++segs;
        tc_fence_after();
        auto scores = [&](int j, int slot) {  // stream j's rows against the keys in a slot
          const uint64_t kd = sdesc_sw128(ring + slot * L::SLOT);
          const uint64_t qd = sdesc_sw128(qs + (lead == 1 ? j : 0) * 32768);
          const uint32_t d = tmem + s_col(j);
          if (E4M3) {
#pragma unroll
            for (int x = 0; x < 8; ++x)  // high, then low codes of q; 32 dims each
              mma_ss<true>(d, qd + (uint64_t)((x >> 2) * 1024 + (x & 3) * 2), kd + (uint64_t)((x & 3) * 2), id_s,
                           x > 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)  // 16 dims each
              mma_ss<false>(d, qd + (uint64_t)((x >> 2) * 1024 + (x & 3) * 2),
                            kd + (uint64_t)((x >> 2) * 1024 + (x & 3) * 2), id_s, x > 0 ? 1u : 0u);
          }
          umma_commit(s_full + j);
        };
        auto products = [&](int j, int slot, bool first) {
          const uint64_t vd = sdesc_mn_sw128(ring + slot * L::SLOT, 16384, 1024);
          const uint32_t d = tmem + o_col(j), pc = tmem + s_col(j);
          if (E4M3) {
#pragma unroll
            for (int x = 0; x < 4; ++x)  // 32 keys each, three parts
#pragma unroll
              for (int part = 0; part < 3; ++part)
                mma_ts<true>(d, pc + 32u * x + 8u * part, vd + (uint64_t)(x * 256), id_o,
                             (first && x == 0 && part == 0) ? 0u : 1u);
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)  // 16 keys each, high and low parts
#pragma unroll
              for (int part = 0; part < 2; ++part)
                mma_ts<false>(d, pc + 32u * (x >> 1) + 8u * (x & 1) + 16u * part, vd + (uint64_t)(x * 128), id_o,
                              (first && x == 0 && part == 0) ? 0u : 1u);
          }
        };
        auto landed = [&](const Ring<NS>& i) {
          ok = ok && wait(full + i.slot, i.round & 1);
          tc_fence_after();
        };
        auto weights = [&](int j) {
          ok = ok && wait(p_ready + j, (n_p >> j) & 1);
          n_p ^= 1u << j;
          tc_fence_after();
        };
        if (lead == 2) {
          // stream t % 2 takes tile t; slots in order K0 K1 V0 K2 V1 K3 ...
          for (int t = 0; t < min(2, nt) && ok; ++t) {
            landed(at);
            if (!ok) break;
            scores(t, at.slot);
            umma_commit(empty + at.slot);
            at.step();
          }
          for (int t = 0; t < nt && ok; ++t) {
            landed(at);
            weights(t & 1);
            if (!ok) break;
            products(t & 1, at.slot, t < 2);
            umma_commit(empty + at.slot);
            if (t + 2 >= nt) umma_commit(o_done + (t & 1));
            at.step();
            if (t + 2 < nt) {
              landed(at);
              if (!ok) break;
              scores(t & 1, at.slot);
              umma_commit(empty + at.slot);
              at.step();
            }
          }
        } else {
          // both streams take every tile; slots in order K0 V0 K1 V1 ...
          landed(at);
          if (!ok) break;
          scores(0, at.slot);
          scores(1, at.slot);
          umma_commit(empty + at.slot);
          at.step();
          for (int t = 0; t < nt && ok; ++t) {
            const Ring<NS> iv = at, ik = at.ahead(1);
            const bool again = t + 1 < nt;
            landed(iv);
            for (int j = 0; j < 2 && ok; ++j) {
              weights(j);
              if (!ok) break;
              products(j, iv.slot, t == 0);
              if (j == 1) umma_commit(empty + iv.slot);
              if (again) {
                if (j == 0) landed(ik);
                if (!ok) break;
                scores(j, ik.slot);
                if (j == 1) umma_commit(empty + ik.slot);
              } else {
                umma_commit(o_done + j);
              }
            }
            at.step();
            if (again) at.step();
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
    Ring<NS> vat;       // slot of the next value tile
    Ring<kInfo> iat;
    bool ok = true;
    for (bool more = wk.next(true); more && ok; more = wk.next(false)) {
      const int nt = wk.k1 - wk.k0, lead = lead_of();
      const int f0 = wk.first_row();
      const int32_t* table = a.block_table + (size_t)(wk.shared() ? 0 : wk.s()) * a.max_pages;
      // keys that all of the segment's rows see: [lo, hi)
      int lo = 0, hi = INT32_MAX;
      if (wk.shared()) {
        const int s0 = f0 / p.rows, s1 = (f0 + wk.g.rows - 1) / p.rows;
        for (int s = s0 + lane; s <= s1; s += 32) {
          const int2 nl = lengths(a, s);
          if (nl.x == 0) continue;
          lo = max(lo, sees(a, nl, nl.x - 1).x);
          hi = min(hi, sees(a, nl, 0).y);
        }
        lo = __reduce_max_sync(0xffffffffu, lo);
        hi = min(__reduce_min_sync(0xffffffffu, hi), a.shared_len);
      } else {
        const int r0 = f0 - wk.s() * p.rows;
        lo = max(sees(a, wk.nl, (r0 + wk.g.rows - 1) / p.group).x, a.shared_len);
        hi = sees(a, wk.nl, r0 / p.group).y;
      }
      for (int x = min(lead, nt); x > 0; --x) vat.step();  // lead tiles of keys go first
      for (int t = 0; t < nt && ok; ++t) {
        const int slot = iat.slot;
        TileInfo* info;
        if (E4M3) info = reinterpret_cast<TileInfo*>(sm + L::INFO + slot * L::INFOS);
        else info = reinterpret_cast<TileInfo*>(sm + L::INFO + slot * L::INFOS - offsetof(TileInfo, bad));
        const int k0 = wk.g.base + (wk.k0 + t) * kTile;
        bool there = false;
        int row = 0;
        if (lane < 8 && k0 + 16 * lane < wk.g.end) {
          const int pos = k0 + 16 * lane, page = table[pos / a.page_size];
          there = page >= 0 && page < a.n_pages;
          if (there) row = page * a.page_size + pos % a.page_size;
          else flag(a.status, DFLASH2_DEV_BAD_PAGE);
        }
        const uint32_t groups = __ballot_sync(0xffffffffu, there);
        const bool mixed = k0 < lo || k0 + kTile > hi || groups != 0xffu;
        float ks[4], vs[4];
        int top = 0;
        if (E4M3) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // keys 32 i + lane
            const int key = 32 * i + lane;
            const int r = __shfl_sync(0xffffffffu, row, key >> 4);
            const bool in = ((groups >> (key >> 4)) & 1) && k0 + key < wk.g.end;
            const size_t at = ((size_t)r + (key & 15)) * a.nkv + wk.h;
            const int kb = in ? min((int)a.k_exp[at], 254) : 0, vb = in ? min((int)a.v_exp[at], 254) : 0;
            ks[i] = __uint_as_float((uint32_t)kb << 23);
            vs[i] = __uint_as_float((uint32_t)vb << 23);
            top = max(top, vb);
          }
          top = __reduce_max_sync(0xffffffffu, top);
        }
        if (iat.round > 0) ok = wait(info_empty + slot, (iat.round - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (E4M3) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            info->ks[32 * i + lane] = ks[i];
            info->vs[32 * i + lane] = vs[i];
          }
        }
        if (lane < 4) info->bad[lane] = 0;
        if (lane == 0) {
          info->groups = groups;
          info->mixed = mixed;
          info->vmax = (float)max(top - 127, -60);
        }
        __syncwarp();
        if (mixed) {
          if (!wait(full + vat.slot, vat.round & 1)) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* v = sm + L::RING + vat.slot * L::SLOT;
          const int from = k0 + kTile > hi ? max(0, hi - k0) : kTile;  // keys from here on, and below `to`
          const int to = k0 < lo ? min(kTile, lo - k0) : 0;
          for (int key = 0; key < kTile; ++key) {
            if (key >= to && key < from) {
              key = from - 1;
              continue;
            }
            // keys past the end hold what the page held before
            const bool past = k0 + key >= wk.g.end;
            bool bad = false;
            if (E4M3) {
              uint32_t* q = reinterpret_cast<uint32_t*>(v + key * 128 + lane * 4);
              uint32_t x = *q, nan = 0;
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if (((x >> (8 * b)) & 0x7fu) == 0x7fu) nan |= 0xffu << (8 * b);
              bad = nan != 0;
              if (past || bad) *q = past ? 0u : x & ~nan;
            } else {
              uint2* q = reinterpret_cast<uint2*>(v + (lane >> 4) * 16384 + key * 128 + (lane & 15) * 8);
              uint2 x = *q;
              uint32_t w[2] = {x.x, x.y};
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                if ((w[b] & 0x7f80u) == 0x7f80u) {
                  bad = true;
                  w[b] &= 0xffff0000u;
                }
                if ((w[b] & 0x7f800000u) == 0x7f800000u) {
                  bad = true;
                  w[b] &= 0xffffu;
                }
              }
              if (past || bad) *q = past ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
            }
            if (__any_sync(0xffffffffu, bad && !past) && lane == 0) info->bad[key >> 5] |= 1u << (key & 31);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(info_full + slot);
        iat.step();
        vat.step();
        if (t + lead < nt) vat.step();  // the next key tile's
      }
    }
  }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int j = warp >> 2, r = threadIdx.x & 127;  // stream, row of its tile
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float scale = a.scale * 1.4426950408889634f;
    const float head_room = E4M3 ? 15.f : 8.f;  // how far a weight may pass 2^0 (E4M3: of weight times scale)
    uint32_t n_s = 0, n_o = 0, tiles = 0;
    bool ok = true;
    for (bool more = wk.next(true); more; more = wk.next(false)) {
      const int nt = wk.k1 - wk.k0;
      const bool split = lead_of() == 2;  // the streams share the rows
      const int fr = (split ? 0 : j * kTile) + r;
      const bool mine = fr < wk.g.rows;
      const int f = wk.first_row() + (mine ? fr : 0);
      const int s = f / p.rows, t_row = (f / p.group) % a.n_tok, head = wk.h * p.group + f % p.group;
      int2 see = make_int2(0, INT32_MAX);  // (rows that do not exist see everything: nothing to mask)
      bool real = mine;
      if (mine) {
        const int2 nl = wk.shared() ? lengths(a, s) : wk.nl;
        see = t_row < nl.x ? sees(a, nl, t_row) : make_int2(0, 0);
        real = t_row < nl.x;
        if (wk.shared()) see.y = min(see.y, a.shared_len);
        else see.x = max(see.x, a.shared_len);
      }
      bar_softmax();  // both streams are done with the last segment
      // query rows, K-major with the 128-byte swizzle
      float rs = scale;  // factor of a row's scores
      uint8_t* qdst = sm + L::Q + (split ? 0 : j) * 32768;
      const bf16* qrow = a.q + ((size_t)s * a.n_tok + t_row) * a.q_stride + (size_t)head * kD;
      if (E4M3) {
        // the row's largest magnitude becomes 2^7 .. 2^8; high codes at 0, low codes at 16 KB
        uint4 x[16];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          x[c] = real ? reinterpret_cast<const uint4*>(qrow)[c] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            top = max(top, w[i] & 0x7f800000u);
            top = max(top, (w[i] << 16) & 0x7f800000u);
          }
        }
        const int e = top >= 0x7f800000u ? 254 : max(1, (int)(top >> 23));
        // 2^(7 - (e - 127)) = 2^(134 - e), in two factors that are floats
        const int e_half = (134 - e) / 2;
        const float up0 = __uint_as_float((uint32_t)(127 + e_half) << 23);
        const float up1 = __uint_as_float((uint32_t)(127 + (134 - e) - e_half) << 23);
        rs = scale * __uint_as_float((uint32_t)(127 - e_half) << 23) *
             __uint_as_float((uint32_t)(127 - ((134 - e) - e_half)) << 23);
        if (top >= 0x7f800000u) rs = __int_as_float(0x7fffffff);  // a row that is not finite has no result
        if (!split || j == 0) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {  // 16 dims: 16 bytes of codes
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4& u = x[2 * c + (i >> 1)];
              const uint32_t w[2] = {(i & 1) ? u.z : u.x, (i & 1) ? u.w : u.y};
              uint32_t h2[2], l2[2];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const float v0 = __uint_as_float(w[b] << 16) * up0 * up1;
                const float v1 = __uint_as_float(w[b] & 0xffff0000u) * up0 * up1;
                h2[b] = __nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3);
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h2[b], __NV_E4M3);
                const float2 back = __half22float2(__half2(hr));
                l2[b] = __nv_cvt_float2_to_fp8x2(make_float2(v0 - back.x, v1 - back.y), __NV_SATFINITE, __NV_E4M3);
              }
              hi[i] = h2[0] | (h2[1] << 16);
              lo[i] = l2[0] | (l2[1] << 16);
            }
            const int at = r * 128 + ((c ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(qdst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(qdst + 16384 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      } else if (!split || j == 0) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint4 x = real ? reinterpret_cast<const uint4*>(qrow)[c] : make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(qdst + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);

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
        ok = wait(info_full + slot, (tile / kInfo) & 1) && ok;
        ok = wait(s_full + j, n_s & 1) && ok;
        ++n_s;
        __syncwarp();
        tc_fence_after();
        if (!idle) {
          float x[kTile];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(lanes + s_col(j) + 32 * c, x + 32 * c);
          tmem_ld_wait();
          if (E4M3) {
#pragma unroll
            for (int i = 0; i < kTile; i += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(info->ks + i);
              x[i] *= k4.x;
              x[i + 1] *= k4.y;
              x[i + 2] *= k4.z;
              x[i + 3] *= k4.w;
            }
          }
          const int k0 = wk.g.base + (wk.k0 + t) * kTile;
          const int v0 = see.x - k0, v1 = see.y > k0 + kTile ? kTile : see.y - k0;  // keys of the tile that it sees
          const uint32_t groups = info->groups;
          const bool cut = __any_sync(0xffffffffu, mine && (v0 > 0 || v1 < kTile)) || groups != 0xffu;
          if (cut) {
#pragma unroll
            for (int i = 0; i < kTile; ++i)
              if (i < v0 || i >= v1 || !((groups >> (i >> 4)) & 1)) x[i] = kNone;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int from = max(0, v0 - 32 * w), to = min(32, v1 - 32 * w);
              if (from < to) {
                const uint32_t m = (to == 32 ? 0xffffffffu : (1u << to) - 1u) & ~((1u << from) - 1u);
                poison |= (info->bad[w] & m) != 0;
              }
            }
          }
          float top = x[0];
#pragma unroll
          for (int i = 1; i < kTile; ++i) top = fmaxf(top, x[i]);
          top *= rs;
          if (E4M3) top += info->vmax;
          if (__any_sync(0xffffffffu, top > ref + head_room)) {
            // a new reference: what was summed up is scaled to it (the
            // products of the stream's last tile are done: its scores of this
            // tile were issued behind them)
            const float now = fmaxf(ref, E4M3 ? top - 11.f : top);
            const float by = ref == kNone ? 0.f : ex2(ref - now);
            sum *= by;
            ref = now;
            if (done > 0) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float o[32];
                tmem_ld32(lanes + o_col(j) + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t w[8];
#pragma unroll
                  for (int b = 0; b < 8; ++b) w[b] = __float_as_uint(o[8 * i + b] * by);
                  tmem_st8(lanes + o_col(j) + 32 * c + 8 * i, w);
                }
              }
            }
          }
          const float sub = ref == kNone ? 0.f : ref;
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (E4M3) {
              uint32_t w[3][8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {  // four keys: a column of each part
                const float4 v4 = *reinterpret_cast<const float4*>(info->vs + 32 * c + 4 * i);
                const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
                uint32_t h[2][3];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const float p0 = ex2(fmaf(x[32 * c + 4 * i + 2 * b], rs, -sub));
                  const float p1 = ex2(fmaf(x[32 * c + 4 * i + 2 * b + 1], rs, -sub));
                  part[2 * b] += p0;
                  part[2 * b + 1] += p1;
                  // the top byte of an f16 is an e5m2: cut, subtract, cut, subtract, round
                  __half2 u = __floats2half2_rn(p0 * vv[2 * b], p1 * vv[2 * b + 1]);
#pragma unroll
                  for (int q = 0; q < 2; ++q) {
                    const uint32_t cutoff = *reinterpret_cast<uint32_t*>(&u) & 0xff00ff00u;
                    h[b][q] = cutoff;
                    u = __hsub2(u, *reinterpret_cast<const __half2*>(&cutoff));
                  }
                  h[b][2] = *reinterpret_cast<uint32_t*>(&u) + 0x00800080u;
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
                  const float p0 = ex2(fmaf(x[32 * c + 16 * hf + 2 * i], rs, -sub));
                  const float p1 = ex2(fmaf(x[32 * c + 16 * hf + 2 * i + 1], rs, -sub));
                  part[(2 * i) & 3] += p0;
                  part[(2 * i + 1) & 3] += p1;
                  const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                  hi[i] = __byte_perm(b0, b1, 0x7632);  // cut to the top 16 bits
                  lo[i] = bits2(__floats2bfloat162_rn(p0 - __uint_as_float(b0 & 0xffff0000u),
                                                      p1 - __uint_as_float(b1 & 0xffff0000u)));
                }
                tmem_st8(lanes + s_col(j) + 32 * c + 8 * hf, hi);
                tmem_st8(lanes + s_col(j) + 32 * c + 16 + 8 * hf, lo);
              }
            }
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
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
        ok = wait(o_done + j, n_o & 1) && ok;
        ++n_o;
      }
      if (poison) sum = __int_as_float(0x7fffffff);
      float w0 = 1.f, w1 = 0.f;
      if (split) {
        // (R, sum) change hands in the scores' columns, which nothing uses any
        // more: the warps of a row in both streams have the same TMEM lanes
        uint32_t mine8[8] = {__float_as_uint(ref), __float_as_uint(sum)}, other8[8];
        tmem_st8(lanes + s_col(j), mine8);
        tmem_st_wait();
        tc_fence_before();
        bar_softmax();
        tc_fence_after();
        tmem_ld8_nowait(lanes + s_col(1 - j), other8);
        tmem_ld_wait();
        // (a stream without tiles has no reference, and its accumulator is not read)
        const float2 me = make_float2(ref, sum);
        const float2 you = make_float2(__uint_as_float(other8[0]), __uint_as_float(other8[1]));
        const float2 x0 = j ? you : me, x1 = j ? me : you;
        ref = fmaxf(x0.x, x1.x);
        const float base = ref == kNone ? 0.f : ref;
        w0 = ex2(x0.x - base);
        w1 = both ? ex2(x1.x - base) : 0.f;
        sum = x0.y * w0 + (both ? x1.y * w1 : 0.f);
      } else {
        tc_fence_after();
      }
      const bool whole = wk.k0 == 0 && wk.k1 == wk.g.tiles && p.tiles_p == 0;
      if (!idle) {
        float* part = nullptr;
        if (!whole) {
          const size_t row = (size_t)(wk.ordinal() + cta) * (wk.shared() ? kTile * QT : p.slot_rows) + fr;
          part = (wk.shared() ? p.part_p : p.part_s) + row * kD;
          if (mine && (!split || j == 0)) (wk.shared() ? p.ref_p : p.ref_s)[row] = make_float2(ref, sum);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        bf16* orow = a.out + ((size_t)s * a.n_tok + t_row) * a.out_stride + (size_t)head * kD;
        // streams that share rows take half of the dims each
#pragma unroll 1
        for (int c = split ? 2 * j : 0; c < (split ? 2 * j + 2 : 4); ++c) {
          float o[32];
          tmem_ld32(lanes + o_col(split ? 0 : j) + 32 * c, o);
          tmem_ld_wait();
          if (split) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= w0;
            if (both) {
              float o1[32];
              tmem_ld32(lanes + o_col(1) + 32 * c, o1);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], w1, o[i]);
            }
          }
          if (whole) {
            if (real) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int b = 0; b < 4; ++b)
                  w[b] = bits2(__floats2bfloat162_rn(sum == 0.f ? 0.f : o[8 * i + 2 * b] * inv,
                                                     sum == 0.f ? 0.f : o[8 * i + 2 * b + 1] * inv));
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
      tc_fence_before();
    }
    (void)ok;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ joining kernel

// A warp per query row: the partial accumulators of its segments, weighted
// to a common reference.  Rows that one CTA finished are there already.
template <int QT>
__global__ void __launch_bounds__(256) attend_join_kernel(const Plan p, int nctas) {
  pdl_launch_next();
  pdl_wait();
  const AttendArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (id >= (long long)a.batch * p.rows * a.nkv) return;
  const int h = (int)(id % a.nkv), f = (int)(id / a.nkv);
  const int s = f / p.rows, t = (f / p.group) % a.n_tok, local = f - s * p.rows;
  const int2 nl = lengths(a, s);
  if (t >= nl.x) return;
  const int units = p.head[0];
  const int i = local / (kTile * QT), entry = s * p.tiles_s + i;
  const Segment g = segment_of<QT>(a, p.group, nl, i);
  const int w = weight_of(p, g.rows);
  const int at = p.head[2 + entry] + h * g.tiles * w;
  if (p.tiles_p == 0 && g.tiles > 0 &&
      owner_of(units, at, nctas) == owner_of(units, at + (g.tiles - 1) * w, nctas))
    return;
  float ref = kNone, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto join = [&](int first, int tiles, int weight, int ordinal, int rows, int row, const float* part,
                  const float2* refs) {
    if (tiles == 0) return;
    const int c0 = owner_of(units, first, nctas), c1 = owner_of(units, first + (tiles - 1) * weight, nctas);
    for (int c = c0; c <= c1; ++c) {
      const int lo = bound_of(units, c, nctas), hi = bound_of(units, c + 1, nctas);
      const int k0 = first >= lo ? 0 : (lo - first + weight - 1) / weight;
      const int k1 = min(tiles, (hi - first + weight - 1) / weight);
      if (k0 >= k1) continue;  // no tile starts in this CTA's share
      const size_t at_row = (size_t)(ordinal + c) * rows + row;
      const float2 rl = refs[at_row];
      const float4 x = reinterpret_cast<const float4*>(part + at_row * kD)[lane];
      if (rl.y == 0.f) continue;
      const float now = fmaxf(ref, rl.x);
      const float base = now == kNone ? 0.f : now;
      const float fo = ex2(ref - base), fx = ex2(rl.x - base);
      sum = fmaf(sum, fo, rl.y * fx);
      o.x = fmaf(o.x, fo, x.x * fx);
      o.y = fmaf(o.y, fo, x.y * fx);
      o.z = fmaf(o.z, fo, x.z * fx);
      o.w = fmaf(o.w, fo, x.w * fx);
      ref = now;
    }
  };
  if (p.tiles_p > 0) {
    const int ip = f / (kTile * QT), tiles = p.head[1], ordinal = ip * a.nkv + h;
    const int wp = QT == 2 ? p.row_weight : 1;
    join(ordinal * tiles * wp, tiles, wp, ordinal, kTile * QT, f % (kTile * QT), p.part_p, p.ref_p);
  }
  join(at, g.tiles, w, entry * a.nkv + h, p.slot_rows, local % (kTile * QT), p.part_s, p.ref_s);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint2 out;
  out.x = sum == 0.f ? 0u : bits2(__floats2bfloat162_rn(o.x * inv, o.y * inv));
  out.y = sum == 0.f ? 0u : bits2(__floats2bfloat162_rn(o.z * inv, o.w * inv));
  reinterpret_cast<uint2*>(a.out + ((size_t)s * a.n_tok + t) * a.out_stride + (size_t)(h * p.group + f % p.group) * kD)[lane] = out;
}

// ------------------------------------------------------------------ host

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Sizes of a call's parts; `ctas` as large as any device's.
struct Sizes {
  int qt, rows, tiles_p, tiles_s, slot_rows;
  size_t head, part_p, part_s, ref_p, ref_s, total;
};
bool sizes_of(int batch, int n_tok, int nq, int nkv, int shared_len, int ctas, Sizes* z) {
  const long long rows = (long long)n_tok * (nq / nkv);
  if (rows * batch >= (1ll << 31) - 512) return false;
  z->rows = (int)rows;
  z->qt = rows > kTile || (shared_len > 0 && rows * batch > kTile) ? 2 : 1;
  const int rt = kTile * z->qt;
  z->tiles_s = (int)((rows + rt - 1) / rt);
  z->tiles_p = shared_len > 0 ? (int)((rows * batch + rt - 1) / rt) : 0;
  z->slot_rows = (int)std::min<long long>(rt, rows);
  const long long segs_s = (long long)batch * z->tiles_s * nkv, segs_p = (long long)z->tiles_p * nkv;
  if (segs_s > (1 << 30) || segs_p > (1 << 30)) return false;
  const size_t n_s = (size_t)(segs_s + ctas) * z->slot_rows, n_p = z->tiles_p ? (size_t)(segs_p + ctas) * rt : 0;
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

template <bool E4M3, int QT>
int launch(const Plan& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Ctx& c) {
  // an attribute of the kernel on the current device: set on every call (a
  // flag of what was set would have to be kept per device)
  if (cudaFuncSetAttribute(attend_tc_kernel<E4M3, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)Smem<E4M3, QT>::bytes) != cudaSuccess)
    return DFLASH2_ERR_CUDA;
  const int rc = launch_k(attend_tc_kernel<E4M3, QT>, dim3(c.nsm), dim3(kThreads), Smem<E4M3, QT>::bytes, c, p, tm_k, tm_v);
  if (rc != DFLASH2_OK) return rc;
  const long long rows = (long long)p.a.batch * p.rows * p.a.nkv;
  return launch_k(attend_join_kernel<QT>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, c, p, c.nsm);
}

}  // namespace

bool attend_tc_fits(const AttendArgs& a) {
  if (a.d != kD || a.page_size % 16 || (long long)a.n_pages * a.page_size >= (1ll << 31) - 256) return false;
  // positions of tiles are 32-bit: the most that the block table allows
  Sizes z;
  if (!sizes_of(a.batch, a.n_tok, a.nq, a.nkv, a.shared_len, kMaxCtas, &z)) return false;
  const long long each = ((long long)a.max_pages * a.page_size + 15) / kTile + 2;
  return ((long long)a.batch * z.tiles_s + z.tiles_p) * a.nkv * each * 2 < (1ll << 31);
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
  p.row_weight = a.e4m3 ? 2 : 1;
  p.slot_rows = z.slot_rows;
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
  if (a.e4m3) return z.qt == 2 ? launch<true, 2>(p, tm_k, tm_v, c) : launch<true, 1>(p, tm_k, tm_v, c);
  return z.qt == 2 ? launch<false, 2>(p, tm_k, tm_v, c) : launch<false, 1>(p, tm_k, tm_v, c);
}

}  // namespace df2
