// From a target's logits to tokens: temperature, top-k, top-p and min-p
// truncation, and on the truncated distribution the draw of a token, the
// distribution itself, or the verification of a draft ("Train a DFlash
// Drafter for Speculative Decoding": spec_generate's temperature, top_p and
// top_k truncate the TARGET's distribution, the one verification samples
// against).
//
// Definition, for a row z at temperature T > 0 with mass e_v =
// exp((z_v - max z) / T): order the tokens by (z descending, id ascending);
// keep the first top_k; of these the shortest prefix that holds top_p of
// their mass; of these the tokens with e_v >= min_p.  Every filter cuts the
// same order, so the kept tokens are a prefix of it, described by its last
// token (value, id).  T <= 0 keeps the first token alone.  Tokens at -inf or
// NaN have no mass and are never kept.
//
// Masses are whole numbers: e_v in units of 2^-lg, lg as large as a bound of the
// row's mass leaves room for in 62 bits (42 to 62), each good to about 2^-35 of
// itself and a unit.  Their 64-bit sums are exact and do not depend on the order
// of the additions, so draws and cuts are deterministic and sit within 2^-35 of
// the exact ones; in plain fp32 a cut or a draw next to a border falls on the wrong
// side about once in a thousand rows of a 150k vocabulary.  (Units of 2^-42 for
// every row would do for a flat one.  But errors of equal tokens add up: of a row
// with one token 14 above 150k equal ones, where a mass is 2^22 such units, 2 draws
// in 1000 gave another token.)
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

typedef unsigned long long u64;

constexpr int NT = 512, NW = NT / 32;
constexpr int NB = 1024;    // bins of a row's histogram
constexpr int CAP = 2048;   // tokens of a list
// Tokens of a list that is ranked (n^2 / 512 steps) instead of sorted.  With 128
// in its place top-k 96 takes 21.3 us for a row of 151936 instead of 17.1, and
// 29.1 for 64 rows instead of 23.3; the ranks' masses have room for 256.
constexpr int SMALL = 256;
constexpr int CMAX = 8;      // CTAs of a row's cluster
constexpr int PARTS = 1024;  // room for what a row's CTAs pick on their own: 128 each at CMAX
// Largest top-k whose tokens each CTA picks on its own: above 100 a peaked
// row's picks, which are at least top-k, soon do not fit their 128, and the
// histogram starts late.  Picked and by histogram, one row of 151936 takes (us)
// 11.2 and 14.5 at top-k 20, 13.1 and 14.8 at 64, 17.1 and 15.5 at 96, 20.7 and
// 15.9 at 120; 64 rows 16.9 and 24.1, 20.0 and 25.1, 23.3 and 26.2, 28.4 and 27.3.
constexpr int LOCAL_K = 100;
// Tokens each CTA picks to try for a top-p border alone, where a sample says that
// what was picked may hold it (0.9 of the nucleus by that estimate, which allows
// for the sample's error; trying always costs a flat row of 151936 60 us instead
// of 48, without the 0.9 the peaked row at top-p 0.99 takes 47 instead of 59).  One
// peaked row at top-p 0.9 takes 20.4 us with it and 34.4 without, 52 with 48 tokens
// (the row's picks no longer fit a ranked list) and 19.7 with 8; 64 such rows 80,
// 65, 49 and 107; a row whose nucleus is missed pays the try (0.99: 59 instead of
// 41).
constexpr int PROBE_K = 16;
constexpr int SUB = NT;       // finer bins of a list
constexpr int SLICE_BYTES = 19456 * 4;  // logits a CTA holds in shared memory, with two CTAs an SM
constexpr unsigned KEY_NINF = 0x007fffffu;  // order of -inf; NaN maps to 0

// Order-preserving map of a logit (a larger one has a larger key; -0 equals 0).
__device__ __forceinline__ unsigned okey(float z) {
  const unsigned u = __float_as_uint(z + 0.f);
  const unsigned k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return z != z ? 0u : k;
}
__device__ __forceinline__ float okey_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Powers of two for mass_of, rounded from 60 decimal digits: 2^(-j/32) in units
// of 2^-42, and 2^(-j/1024) as the whole number (1 - 2^(-j/1024)) 2^37 and as a
// float, for j = 0..31.
struct ExpConst {
  u64 pow32[32];
  unsigned drop[32];
  float pow1024[32];
};
__device__ const ExpConst c_exp = {
    {4398046511104ull, 4303805443529ull, 4211583767698ull, 4121338212211ull, 4033026432885ull,
     3946606992882ull, 3862039343274ull, 3779283804012ull, 3698301545306ull, 3619054569413ull,
     3541505692798ull, 3465618528697ull, 3391357470036ull, 3318687672730ull, 3247575039328ull,
     3177986203020ull, 3109888511975ull, 3043250014027ull, 2978039441675ull, 2914226197418ull,
     2851780339397ull, 2790672567345ull, 2730874208839ull, 2672357205845ull, 2615094101559ull,
     2559058027516ull, 2504222690988ull, 2450562362647ull, 2398051864490ull, 2346666558027ull,
     2296382332721ull, 2247175594673ull},
    {0u, 93001160u, 185939388u, 278814728u, 371627222u, 464376912u, 557063841u, 649688051u,
     742249585u, 834748485u, 927184793u, 1019558553u, 1111869805u, 1204118593u, 1296304959u, 1388428945u,
     1480490593u, 1572489946u, 1664427045u, 1756301933u, 1848114652u, 1939865243u, 2031553750u, 2123180213u,
     2214744675u, 2306247178u, 2397687764u, 2489066475u, 2580383352u, 2671638437u, 2762831773u, 2853963400u},
    {0x1p+0f, 0x1.ffa74ep-1f, 0x1.ff4eacp-1f, 0x1.fef61ap-1f, 0x1.fe9d96p-1f, 0x1.fe4522p-1f,
     0x1.fdecbep-1f, 0x1.fd9468p-1f, 0x1.fd3c22p-1f, 0x1.fce3ecp-1f, 0x1.fc8bc4p-1f, 0x1.fc33acp-1f,
     0x1.fbdba4p-1f, 0x1.fb83aap-1f, 0x1.fb2bcp-1f, 0x1.fad3e4p-1f, 0x1.fa7c18p-1f, 0x1.fa245cp-1f,
     0x1.f9ccaep-1f, 0x1.f9751p-1f, 0x1.f91d8p-1f, 0x1.f8c6p-1f, 0x1.f86e9p-1f, 0x1.f8172ep-1f,
     0x1.f7bfdap-1f, 0x1.f76898p-1f, 0x1.f71164p-1f, 0x1.f6ba3ep-1f, 0x1.f66328p-1f, 0x1.f60c2p-1f,
     0x1.f5b528p-1f, 0x1.f55e4p-1f}};
constexpr float FAR = 40.f;  // from here on masses are plain fp32
struct ExpTab {  // in shared memory
  u64 pow32[32];      // 2^(-k/32) in units of 2^-62
  uint2 pow1024[32];  // c_exp's drop, and its pow1024 as bits
};

// The row's exponent scale log2(e) / T as a float pair, and the masses' unit.
struct Scale {
  float zmax, hi, lo;
  bool odd;  // zmax or the temperature is infinite
  int lg;    // masses are in units of 2^-lg
};
// 2^n as a float, n in -126..127.
__device__ __forceinline__ float pow2f(int n) { return __int_as_float((127 + n) << 23); }
// x as a float pair.
__device__ __forceinline__ float2 pair_of(double x) {
  const float h = (float)x;
  return make_float2(h, (float)(x - (double)h));
}

// exp((z - zmax) / T) in units of 2^-lg, for z > -inf.  y = (zmax - z) log2(e) / T
// is held as p + e (the difference exact by two-sum, the product by fma) and
// cut into k/1024 + g + e with |g| <= 2^-11: 2^(-k/1024) is a product of two
// table entries in whole numbers and a shift, and the rest, 1 - 2^-(g+e) = w -
// w^2/2 with w = (g + e) ln 2 below 2^-11, is good to 2^-24 of itself in fp32:
// 2^-35 of the mass.  (A form good to 2^-37 takes about 10% longer; a draw's number
// has 24 bits, and a border next to which 2^-35 decides is met once in 10^5 rows of
// 150k tokens or less.)  From y = 40 on plain fp32 is good to 2^-58 of the largest
// mass.
__device__ __forceinline__ float y_of(float z, const Scale& s) {
  return __fmul_rn(s.zmax - z, s.hi);  // never contracted: its rounding error is formed below
}
__device__ __forceinline__ unsigned far_mass(float y, int lg) {  // below 2^23; 0 from y = 64 on, infinity and NaN included
  float f;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"((float)lg - y));
  return __float2uint_rn(f);
}
// No branch depends on one value, so the N evaluations overlap; with VOTE, a
// warp without far values skips their form (same results).
template <int N, bool VOTE>
__device__ __forceinline__ void masses_of(const float (&z)[N], const float (&p)[N], const Scale& s, const ExpTab& tab,
                                          u64 (&v)[N]) {
  bool far = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float dh = s.zmax - z[i], bb = dh - s.zmax;
    const float dl = (s.zmax - (dh - bb)) - (z[i] + bb);
    const float e = fmaf(dl, s.hi, fmaf(dh, s.lo, fmaf(dh, s.hi, -p[i])));
    // 1.5 2^23: rounds to a whole number of 1024ths (of far values only kept within the shift)
    const float kf = fmaf(fminf(p[i], FAR), 1024.f, 12582912.f);
    const unsigned k = __float_as_uint(kf) - 0x4b400000u;
    const float w = (fmaf(kf - 12582912.f, -0x1p-10f, p[i]) + e) * 0.693147182f;
    const float x = fmaf(-0.5f * w, w, w);
    const u64 a = tab.pow32[k >> 5 & 31];
    const uint2 t = tab.pow1024[k & 31];
    const unsigned a31 = (unsigned)(a >> 31);
    u64 b = a - ((u64)a31 * t.x >> 6);  // 2^(-(k mod 1024)/1024) in units of 2^-62
    const float bf = (float)a31 * __uint_as_float(t.y);  // the same in units of 2^-31
    asm("mad.wide.s32 %0, %1, -1048576, %0;" : "+l"(b) : "r"(__float2int_rn(bf * x * 2048.f)));
    v[i] = b >> ((k >> 10) + (62 - s.lg));
    far = far || !(p[i] < FAR);
  }
  if (!VOTE || __any_sync(0xffffffffu, far)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(p[i] < FAR)) v[i] = far_mass(p[i], s.lg);
  }
  // (a difference or a product without a value: an infinite maximum, which
  // shares the mass with its equals alone, or T = infinity)
  if (s.odd) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = z[i] == s.zmax || s.zmax < INFINITY ? 1ull << s.lg : 0ull;
  }
}
__device__ __forceinline__ u64 mass_of(float z, const Scale& s, const ExpTab& tab) {
  const float x[1] = {z}, y[1] = {y_of(z, s)};
  u64 v[1];
  masses_of<1, false>(x, y, s, tab, v);
  return v[0];
}

// The same to fp32 accuracy relative to the mass, however small.  Only written
// probabilities use it: two ulp of exp2f, one of the correction, then one of the
// fp32 reciprocal of the row's mass and half a one of the product, up to 8e-8 of a
// flat row's probabilities (rounded once from 64 bits they are off by 2.5e-8).
// What is kept, drawn and accepted is decided on the whole masses.
__device__ __forceinline__ float mass_f32(float z, const Scale& s) {
  if (z == s.zmax) return 1.f;
  if (s.odd) return s.zmax < INFINITY ? 1.f : 0.f;
  const float dh = s.zmax - z, p = __fmul_rn(dh, s.hi);
  if (!(p < 160.f)) return 0.f;
  const float bb = dh - s.zmax, dl = (s.zmax - (dh - bb)) - (z + bb);
  float e = fmaf(dh, s.hi, -p);
  e = fmaf(dh, s.lo, e);
  e = fmaf(dl, s.hi, e);
  const float f = exp2f(-p);  // (below 2^-126 a subnormal: the sum of a row is at least 1)
  return fmaf(f, -0.693147182f * e, f);
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------ clusters

__device__ __forceinline__ void st_cl(uint32_t addr, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cl(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned ld_cl(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ unsigned add_cl(uint32_t addr, unsigned v) {
  unsigned o;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(addr), "r"(v) : "memory");
  return o;
}

// The two halves of cluster_sync (every thread of the cluster, in turn).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The kept prefix of a row's order: every token with (key, id) ahead of or
// equal to (key, id) here.
struct Cut {
  unsigned key;
  int id;
};
__device__ __forceinline__ bool kept(unsigned k, int id, const Cut& c) {
  return k > c.key || (k == c.key && id <= c.id);
}

// The same on a logit, `zc` being the value of the cut's key.
__device__ __forceinline__ bool kept_z(float z, int id, float zc, int idc) { return z > zc || (z == zc && id <= idc); }

// The same as one comparison where every token at the cut's value stays.
struct CutZ {
  float below, at;  // kept: z > below, unless z == at and the id is past idc
  int idc;
  bool ties;  // some token at the cut's value does not stay
};
__device__ __forceinline__ CutZ cut_z(const Cut& c, int V) {
  // (the key below that of 0 is that of -0, which equals 0)
  return {okey_value(c.key - (c.key == 0x80000000u ? 2 : 1)), okey_value(c.key), c.id, c.id < V - 1};
}

// The masses of four logits (ids id .. id + 3), 0 for those the cut drops and
// for id x.  A warp whose kept logits are all far takes the short way.
__device__ __forceinline__ bool masses4(const float4& v, int id, const Scale& s, const ExpTab& tab, const CutZ& c,
                                        int x, u64 (&e)[4]) {
  const float z[4] = {v.x, v.y, v.z, v.w};
  bool keep[4], near = false;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) keep[j] = z[j] > c.below;
  if (c.ties) {
#pragma unroll
    for (int j = 0; j < 4; ++j) keep[j] = keep[j] && (z[j] > c.at || id + j <= c.idc);
  }
  if ((unsigned)(x - id) < 4u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) keep[j] = keep[j] && id + j != x;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = y_of(z[j], s);
    near = near || (keep[j] && !(y[j] >= FAR));
  }
  if (!__any_sync(0xffffffffu, near)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = keep[j] ? far_mass(y[j], s.lg) : 0u;
    return false;
  }
  masses_of<4, true>(z, y, s, tab, e);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (!keep[j]) e[j] = 0;
  return true;
}

// What the cluster's first CTA decides for the others.
enum { STEP_NONE = 0, STEP_LIST = 1, STEP_TOPK = 2, STEP_TOPP = 3, STEP_SLOW_K = 4, STEP_SLOW_P = 5 };
struct Decision {
  int step;
  int lo, hi;       // bins to gather
  unsigned before;  // tokens in bins ahead of lo
  Cut cut;
  unsigned total_lo, total_hi;  // mass of the cut, when known
};
constexpr int DW = sizeof(Decision) / 4;

struct Smem {
  ExpTab tab;     // copy of c_exp: lanes read different entries
  u64 cand[CAP];  // first CTA: gathered tokens, (key, ~id)
  unsigned hist[NB];
  u64 radix[SMALL];
  union {  // first CTA
    u64 parts[PARTS];  // what each CTA picked on its own, for a small top-k
    struct {
      float ecum[NB + 1];                 // estimated mass ahead of each bin
      unsigned sub[3][SUB];  // masses of a list's finer bins, 21 bits in each
    };
  };
  u64 wsum[NW], wsum2[NW];
  u64 wkept[NW];  // mass each warp's slice keeps of the bins that hold the top-p border
  u64 xm[2][CMAX], xg[2][CMAX];  // exchanged masses, two turns
  float xmax[CMAX], xmin[CMAX], xlow[CMAX], xub[CMAX];
  float2 xest[CMAX];
  int xid[CMAX];
  float fsum[NW], fmin[NW], fub[NW];
  float2 c_pair, off_pair;  // log2(e) / T and T ln(min_p)
  Decision mk;      // first CTA: the next decision
  Decision dec[2];  // the last one received, two turns
  struct {
    u64 total;
    Cut cut;
    int n;
  } sel[3];  // small lists: the kept tokens after top-k, top-p and min-p
  u64 bound;
  unsigned ncand, nlocal;  // tokens in the first CTA's list, and in this CTA's own
  unsigned sel_key;
  u64 sel_before;
  int pick, pick2;
};

// Adds a mass to bin b of a list's finer bins (2048 masses of 62 bits at most: no
// part overflows), and reads one.
__device__ __forceinline__ void sub_add(Smem& sm, int b, u64 e) {
  atomicAdd(&sm.sub[0][b], (unsigned)e & 0x1fffffu);
  atomicAdd(&sm.sub[1][b], (unsigned)(e >> 21) & 0x1fffffu);
  atomicAdd(&sm.sub[2][b], (unsigned)(e >> 42));
}
__device__ __forceinline__ u64 sub_get(const Smem& sm, int b) {
  return ((u64)sm.sub[2][b] << 42) + ((u64)sm.sub[1][b] << 21) + sm.sub[0][b];
}

// Sum over the threads before this one (and the block's total).
__device__ __forceinline__ u64 block_scan_u64(u64 mine, u64* total, Smem& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) sm.wsum[warp] = inc;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < warp) before += sm.wsum[i];
    all += sm.wsum[i];
  }
  *total = all;
  return before + inc - mine;
}

// Descending sort of the first n entries of `a` (n <= CAP, padded with zeros
// to a power of two; every entry is above zero).
__device__ __noinline__ void sort_desc(u64* a, int n) {
  int p = 32;
  while (p < n) p <<= 1;
  for (int i = n + threadIdx.x; i < p; i += NT) a[i] = 0;
  __syncthreads();
  for (int k = 2; k <= p; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int q = threadIdx.x; q < p / 2; q += NT) {
        const int i = ((q & ~(j - 1)) << 1) | (q & (j - 1));
        const u64 x = a[i], y = a[i + j];
        if ((x < y) == ((i & k) == 0)) a[i] = y, a[i + j] = x;
      }
      __syncthreads();
    }
}

// One CTA's slice of a row: ids [begin, begin + n).  Element i of the slice's
// storage is id first + i; storage is cut in groups of four that lie on
// 16-byte boundaries of the row for fp32 (8 bytes for bf16), and what it holds
// outside the slice reads as -inf.
template <typename T, bool RES>
struct Slice {
  static constexpr int U = 4;  // groups whose loads are in flight
  const T* row;
  T* zs;
  int begin, end, first, groups;
  __device__ __forceinline__ float4 get4(int i) const {
    auto four = [](const uint2& q) {  // of bf16
      return make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u), __uint_as_float(q.y << 16),
                         __uint_as_float(q.y & 0xffff0000u));
    };
    if constexpr (RES) {
      if constexpr (sizeof(T) == 4) return *reinterpret_cast<const float4*>(zs + 4 * i);
      else return four(*reinterpret_cast<const uint2*>(zs + 4 * i));
    }
    const int id = first + 4 * i;
    if (id >= begin && id + 4 <= end) {
      if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const float4*>(row + id));
      else return four(__ldg(reinterpret_cast<const uint2*>(row + id)));
    }
    float4 v;
    float* e = &v.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = id + j >= begin && id + j < end ? ld(row + id + j) : -INFINITY;
    return v;
  }
};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& v, float (&e)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void unpack16<float>(const uint4& v, float (&e)[4]) {
  e[0] = __uint_as_float(v.x), e[1] = __uint_as_float(v.y), e[2] = __uint_as_float(v.z), e[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void unpack16<bf16>(const uint4& v, float (&e)[8]) {
  const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[2 * i] = __uint_as_float(w[i] << 16);
    e[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Calls f(four logits, id of the first) on every group of the slice; every
// thread makes the same number of calls (elements outside read as -inf).
template <typename S, typename F>
__device__ __forceinline__ void for_each4(const S& s, F f) {
  for (int i0 = 0; i0 < s.groups; i0 += NT * S::U) {
    float4 v[S::U];
#pragma unroll
    for (int u = 0; u < S::U; ++u) {
      const int i = i0 + u * NT + threadIdx.x;
      v[u] = i < s.groups ? s.get4(i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
#pragma unroll
    for (int u = 0; u < S::U; ++u)
      if (u == 0 || i0 + u * NT < s.groups) f(v[u], s.first + 4 * (i0 + u * NT + (int)threadIdx.x));
  }
}
// The same for single elements.
template <typename S, typename F>
__device__ __forceinline__ void for_each(const S& s, F f) {
  for_each4(s, [&](const float4& v, int id) { f(v.x, id), f(v.y, id + 1), f(v.z, id + 2), f(v.w, id + 3); });
}

// A warp appends the tokens of its groups of four (ids id .. id + 3) that are
// marked to this CTA's list of room `most`, counted in `counter`.
__device__ __forceinline__ void append4(const float (&z)[4], const bool (&yes)[4], int id, unsigned* counter, u64* list,
                                        unsigned most) {
  const int lane = threadIdx.x & 31;
  unsigned m[4], n = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = __ballot_sync(0xffffffffu, yes[j]);
    n += __popc(m[j]);
  }
  if (!n) return;
  unsigned at = 0;
  if (lane == 0) at = atomicAdd(counter, n);
  at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const unsigned pos = at + __popc(m[j] & ((1u << lane) - 1));
    if (yes[j] && pos < most) list[pos] = ((u64)okey(z[j]) << 32) | (unsigned)~(id + j);
    at += __popc(m[j]);
  }
}
// The same for the slice's logits for which in(z) holds, all of them in [low, high].
template <typename S, typename F>
__device__ __forceinline__ void collect(const S& s, float low, float high, F in, unsigned* counter, u64* list,
                                        unsigned most) {
  for_each4(s, [&](const float4& v, int id) {
    const float z[4] = {v.x, v.y, v.z, v.w};
    bool yes[4], any = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) any = any || (z[j] >= low && z[j] <= high);
    if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) yes[j] = z[j] >= low && z[j] <= high && z[j] > -INFINITY && in(z[j]);
    append4(z, yes, id, counter, list, most);
  });
}

// The first token of the order, among those kept by `c`, at which the running
// sum of weights (1 each when by_count, else the masses) reaches `target`
// (>= 1, at most the total): radix selection on the key, 8 bits a level, then
// on the ids of equal keys.  By one CTA on the whole row: the way out for
// rows with more equal or nearly equal tokens than a list holds.
template <typename T>
__device__ __noinline__ Cut select_slow(const T* row, int V, Scale s, Cut c, bool by_count, u64 target, Smem& sm) {
  unsigned prefix = 0, mask = 0;
  u64 before = 0;  // weight ahead of the keys that match the prefix
  for (int level = 3; level >= 0; --level) {
    for (int i = threadIdx.x; i < 256; i += NT) sm.radix[i] = 0;
    __syncthreads();
    for (int v = threadIdx.x; v < V; v += NT) {
      const float z = ld(row + v);
      const unsigned k = okey(z);
      if ((k & mask) == prefix && kept(k, v, c))
        atomicAdd(&sm.radix[(k >> (8 * level)) & 255u], by_count ? 1ull : mass_of(z, s, sm.tab));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 b = before;
      int d = 255;
      while (d > 0 && b + sm.radix[d] < target) b += sm.radix[d--];
      sm.sel_key = prefix | ((unsigned)d << (8 * level));
      sm.sel_before = b;
    }
    __syncthreads();
    prefix = sm.sel_key;
    before = sm.sel_before;
    mask |= 255u << (8 * level);
    __syncthreads();
  }
  // equal keys: the need-th of them in id order (each has the same weight)
  const u64 w = by_count ? 1ull : mass_of(okey_value(prefix), s, sm.tab);
  const u64 need = w ? max(1ull, (target - before + w - 1) / w) : 1ull;
  const int per = (V + NT - 1) / NT;
  const int a = min(V, (int)threadIdx.x * per), b = min(V, a + per);
  u64 mine = 0, all;
  for (int v = a; v < b; ++v) {
    const unsigned k = okey(ld(row + v));
    mine += k == prefix && kept(k, v, c);
  }
  if (threadIdx.x == 0) sm.pick = c.key == prefix ? c.id : V - 1;
  const u64 ahead = block_scan_u64(mine, &all, sm);
  if (ahead < need && ahead + mine >= need) {
    u64 left = need - ahead;
    for (int v = a; v < b; ++v) {
      const unsigned k = okey(ld(row + v));
      if (k == prefix && kept(k, v, c) && --left == 0) sm.pick = v;
    }
  }
  __syncthreads();
  const Cut out = {prefix, sm.pick};
  __syncthreads();
  return out;
}

// floor(u total) and ceil(p total), exactly, for u and p in [0, 1) (in units
// of 2^-64: below 2^-41 a float's last bits are dropped).
__device__ __forceinline__ u64 units(float u) { return (u64)(fminf(fmaxf(u, 0.f), 0.99999994f) * 18446744073709551616.f); }
__device__ __forceinline__ u64 floor_share(float u, u64 total) { return __umul64hi(units(u), total); }
__device__ __forceinline__ u64 share_of(float p, u64 total) {
  const u64 q = units(p);
  const u64 t = __umul64hi(q, total) + (q * total != 0);
  return min(max(t, 1ull), total);
}

// The cut of min_p: max z + T ln(min_p), the second term as a pair, as the
// smallest float not below it.
__device__ __forceinline__ unsigned min_p_key(float zmax, float2 off) {
  const float t = zmax + off.x, bb = t - zmax;
  const float r = ((zmax - (t - bb)) + (off.x - bb)) + off.y;  // t + r: the exact sum to 2^-48
  if (!(fabsf(t) < INFINITY)) return okey(fminf(t, zmax));
  float f = t + r;
  if (f - t < r) f = nextafterf(f, INFINITY);
  return okey(fminf(f, zmax));
}

// The accepted prefix of a sequence, its emitted tokens and the counters, by
// one warp (lane i looks after row i).
__device__ void join_rows(const SamplingArgs& a, int s, int nd) {
  const int lane = threadIdx.x & 31, B = a.rows, D = B - 1;
  const int2 ro = lane <= nd ? __ldcg(a.rowout + (size_t)s * B + lane) : make_int2(0, -1);
  const int n = __ffs(~__ballot_sync(0xffffffffu, lane < nd && ro.x)) - 1;  // drafts accepted
  const int tok = __shfl_sync(0xffffffffu, ro.y, n);
  if (lane < B) a.out_tok[(size_t)s * B + lane] = lane < n ? a.path[(size_t)s * D + lane] : (lane == n ? tok : -1);
  u64* c = reinterpret_cast<u64*>(a.counters);
  if (c && lane < n) atomicAdd(c + 4 + B + lane, 1ull);
  if (lane == 0) {
    a.accept_len[s] = n;
    a.n_out[s] = n + 1;
    a.next_anchor[s] = tok;
    if (a.seq_len) a.seq_len[s] += n + 1;
    if (c) {
      atomicAdd(c + 0, 1ull);
      atomicAdd(c + 1, (u64)nd);
      atomicAdd(c + 2, (u64)n);
      atomicAdd(c + 3, (u64)(nd - n));
      atomicAdd(c + 4 + n, 1ull);
    }
  }
}

__global__ void __launch_bounds__(128) join_kernel(SamplingArgs a) {
  pdl_launch_next();
  pdl_wait();
  const int s = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (s < a.batch) join_rows(a, s, a.n_draft ? min(max(a.n_draft[s], 0), a.rows - 1) : a.rows - 1);
}

// One thread-block cluster per row, a slice of the row in each CTA's shared
// memory (RES; a vocabulary above 155,648 in fp32 stays in global memory): the
// logits are read from HBM once, and a row's steps are passes over shared
// memory joined by cluster barriers.
//   a small top-k    each CTA picks its candidates by its threads' largest
//                    logits, the first CTA ranks what they picked (no pass
//                    over all masses)
//   a top-p alone    the same with a few tokens, if a sample of the masses says
//                    that they may hold the nucleus; otherwise, as for a large
//                    top-k: a histogram of counts guesses the border's bins,
//                    and one pass over all masses takes their tokens, the mass
//                    ahead of them and the kept mass of each warp
//   neither          the kept mass of each warp decides which one holds the draw
// What bounds it: one row with a small top-k, the latency of those steps (151936
// fp32 logits with top-k 20 and top-p 0.95: 11.2 us); a nucleus over a flat row,
// 48 us, is passes of 19k tokens by each of its 8 CTAs.  Many rows, instructions,
// at 1.8 to 2.5 a cycle: 27 per token with top-k 20 (64 bf16 rows of 151936, 17
// us), 85 at a temperature alone (128 such rows, 84 us; 118 for 200 fp32 rows of
// 50257, 58 us), 164 for a nucleus (128 flat rows, 171 us; their bytes take 6 us at
// the copy's rate).  A mass is about 45 of them; the others are the load with its
// maximum, the histogram, the sums by warp and the lists.  Rows run in whole waves
// (128 rows of 151936 in clusters of 4 are 512 CTAs on 304 places), each CTA its
// steps one after the other.
template <typename T, bool RES>
__global__ void __launch_bounds__(NT, 2) sample_kernel(SamplingArgs a, int slice) {
  extern __shared__ uint4 zs_raw[];
  T* zs_buf = reinterpret_cast<T*>(zs_raw);
  __shared__ Smem sm;
  pdl_launch_next();
  pdl_wait();
  const int C = 1 << a.lg_cluster, row = blockIdx.x >> a.lg_cluster, rank = blockIdx.x & (C - 1), V = a.vocab;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seq = row / a.rows, i = row - seq * a.rows;  // sequence and its row
  int nd = a.rows - 1;
  if (a.kind == SAMPLING_VERIFY) {
    if (a.n_draft) nd = min(max(a.n_draft[seq], 0), nd);
    if (i > nd) return;  // the whole cluster
  }
  cluster_arrive();  // waited for before the first access to another CTA's memory
  const u64 pow32 = c_exp.pow32[lane];
  const uint2 pow1024 = make_uint2(c_exp.drop[lane], __float_as_uint(c_exp.pow1024[lane]));
  const T* z_row = static_cast<const T*>(a.logits) + (size_t)row * a.stride;
  const float temp = a.temperature ? a.temperature[seq] : 1.f;
  const int top_k = a.top_k ? a.top_k[seq] : 0;
  const float top_p = a.top_p ? a.top_p[seq] : 1.f, min_p = a.min_p ? a.min_p[seq] : 0.f;
  const bool greedy = !(temp > 0.f);
  // (64-bit floats are slow here: one lane each, while the logits load)
  // (a scale above fp32's range, from subnormal temperatures, is its largest value:
  // 0 times it is still 0)
  if (tid == 64) sm.c_pair = pair_of(fmin(1.4426950408889634074 / (greedy ? 1.0 : (double)temp), 3.4028234663852886e38));
  // (at an infinite temperature every mass is 1 and min(min_p, 1) drops none)
  if (tid == 96 && min_p > 0.f)
    sm.off_pair = temp == INFINITY ? make_float2(-INFINITY, 0.f) : pair_of((double)temp * log(fmin((double)min_p, 1.0)));

  int x = -1;          // the draft's token
  float zx = -INFINITY;  // and its logit
  if (a.kind == SAMPLING_VERIFY && i < nd) {
    x = a.path[(size_t)seq * (a.rows - 1) + i];
    if (x >= 0 && x < V) zx = ld(z_row + x);
  }

  // ---- 1. the slice into shared memory, its largest and smallest logit
  Slice<T, RES> s;
  s.row = z_row;
  s.zs = zs_buf;
  s.begin = min(V, rank * slice);
  s.end = min(V, s.begin + slice);
  constexpr int VEC = 16 / sizeof(T);
  const int mis = (int)((reinterpret_cast<uintptr_t>(z_row + s.begin) / sizeof(T)) % VEC);
  s.first = s.begin - mis;
  s.groups = s.end > s.begin ? (s.end - s.first + VEC - 1) / VEC * (VEC / 4) : 0;
  float mx = -INFINITY, mn = INFINITY;
  auto see = [&](float z) {
    if (z > -INFINITY) {  // (false for NaN)
      mx = fmaxf(mx, z);
      mn = fminf(mn, z);
    }
  };
  if constexpr (RES) {
    constexpr int U = 4;
    const int nv = s.groups / (VEC / 4);
    for (int v0 = tid; v0 < nv; v0 += U * NT) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT, id = s.first + v * VEC;
        if (v < nv && id >= s.begin && id + VEC <= s.end) q[u] = __ldg(reinterpret_cast<const uint4*>(z_row + id));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT, id = s.first + v * VEC;
        if (v >= nv) break;
        float e[VEC];
        if (id >= s.begin && id + VEC <= s.end) {
          unpack16<T>(q[u], e);
          zs_raw[v] = q[u];
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            e[j] = id + j >= s.begin && id + j < s.end ? ld(z_row + id + j) : -INFINITY;
            st(zs_buf + v * VEC + j, e[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) see(e[j]);
      }
    }
  } else {
    for_each(s, [&](float z, int) { see(z); });
  }
  for (int b = tid; b < NB; b += NT) sm.hist[b] = 0;
  if (warp == 0) {
    sm.tab.pow32[lane] = pow32 << 20;
    sm.tab.pow1024[lane] = pow1024;
  }
  if (tid == 0) {
    sm.ncand = sm.nlocal = 0;
    sm.pick = -1;
    sm.pick2 = 0x7fffffff;
  }
  const float thread_max = mx;
  mx = warp_max(mx);
  mn = -warp_max(-mn);
  if (lane == 0) {
    sm.fsum[warp] = mx;
    sm.fmin[warp] = mn;
  }
  __syncthreads();
  for (int w = 0; w < NW; ++w) {
    mx = fmaxf(mx, sm.fsum[w]);
    mn = fminf(mn, sm.fmin[w]);
  }
  float zmax = -INFINITY, zmin = INFINITY;
  // The mass of this thread's logits, relative to the CTA's largest, is at most
  // their number times that of the largest of them.
  auto bound = [&]() {
    const float per_thread = (float)((s.groups / (VEC / 4) + NT - 1) / NT * VEC);
    float ub = thread_max == mx ? 1.f : exp2f((thread_max - mx) * sm.c_pair.x);
    ub = warp_sum(thread_max > -INFINITY ? ub * per_thread : 0.f);
    if (lane == 0) sm.fub[warp] = ub;
  };
  auto tell_bound = [&]() {  // (by threads below C, after a barrier)
    float ub = 0.f;
    for (int w = 0; w < NW; ++w) ub += sm.fub[w];
    st_cl(dsmem_addr(&sm.xub[rank], tid), __float_as_uint(ub));
  };
  // A small top-k: each CTA picks its own candidates.  The k-th largest of its
  // threads' largest logits has at least k logits that are not below it, so no
  // token of the row's top k lies below it; few others do not.
  // (A top-p alone tries the same with a few tokens: the nucleus of a peaked
  // row is among them.)
  const bool by_k0 = !greedy && top_k > 0 && top_k < V, probe = !greedy && !by_k0 && top_p < 1.f;
  const int pick_k = by_k0 ? top_k : PROBE_K;
  bool local = probe || (by_k0 && top_k <= LOCAL_K);
  if (local) {
    const float range = fminf(mx - mn, 64.f);
    const float per = range > 0.f ? fminf((float)SUB / range, 1e30f) : 1.f;
    const int bin = thread_max == mx ? 0 : (int)fminf((mx - thread_max) * per, (float)(SUB - 1));
    if (thread_max > -INFINITY) atomicAdd(&sm.hist[bin], 1u);
    __syncthreads();
    u64 all;
    const unsigned c = sm.hist[tid];
    const u64 before = block_scan_u64(c, &all, sm);
    const bool enough = all >= (u64)pick_k;
    if (before < (u64)pick_k && (u64)pick_k <= before + c) sm.pick = tid;
    __syncthreads();
    float low = enough && thread_max > -INFINITY && bin <= sm.pick ? thread_max : INFINITY;
    low = -warp_max(-low);
    if (lane == 0) sm.fmin[warp] = low;
    __syncthreads();
    for (int w = 0; w < NW; ++w) low = fminf(low, sm.fmin[w]);
    if (!enough) low = -3.402823466e+38f;  // fewer logits than that: all of them
    const unsigned part = PARTS >> a.lg_cluster;
    cluster_wait();
    collect(s, low, INFINITY, [](float) { return true; }, &sm.nlocal, sm.cand, part);
    __syncthreads();
    for (unsigned e = tid; e < min(sm.nlocal, part); e += NT) st_cl(dsmem_addr(sm.parts + rank * part + e, 0), sm.cand[e]);
    if (probe) {
      // whether the picked tokens can hold the nucleus at all: their mass, and
      // that of the others from a sample (a group a thread), relative to this
      // CTA's largest logit; it only decides which way is tried
      float picked = 0.f, others = 0.f;
      const float c = sm.c_pair.x;
      for (unsigned e = tid; e < min(sm.nlocal, part); e += NT)
        picked += exp2f((okey_value((unsigned)(sm.cand[e] >> 32)) - mx) * c);
      if (tid < s.groups) {
        const float4 v = s.get4(tid);
        const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) others += z[j] < low ? exp2f((z[j] - mx) * c) : 0.f;
      }
      picked = warp_sum(picked);
      others = warp_sum(others) * (float)s.groups / (float)min(s.groups, NT);
      if (lane == 0) {
        sm.fsum[warp] = picked;
        sm.fmin[warp] = others;
      }
      bound();
      __syncthreads();
    }
    if (tid < C) {
      st_cl(dsmem_addr(&sm.xmax[rank], tid), __float_as_uint(mx));
      st_cl(dsmem_addr(&sm.xlow[rank], tid), __float_as_uint(low));
      st_cl(dsmem_addr(&sm.xid[rank], tid), sm.nlocal);
      if (probe) {
        float x = 0.f, y = 0.f;
        for (int w = 0; w < NW; ++w) x += sm.fsum[w], y += sm.fmin[w];
        st_cl(dsmem_addr(&sm.xest[rank].x, tid), __float_as_uint(x));
        st_cl(dsmem_addr(&sm.xest[rank].y, tid), __float_as_uint(y));
        tell_bound();
      }
    }
    cluster_sync();
    for (int r = 0; r < C; ++r) {
      zmax = fmaxf(zmax, sm.xmax[r]);
      local = local && sm.xid[r] <= (int)part;  // (else too many in one part: the ways below)
    }
    if (probe) {
      float picked = 0.f, all = 0.f;
      for (int r = 0; r < C; ++r) {
        const float f = sm.xmax[r] == zmax ? 1.f : exp2f((sm.xmax[r] - zmax) * sm.c_pair.x);
        picked += f * sm.xest[r].x;
        all += f * (sm.xest[r].x + sm.xest[r].y);
      }
      local = local && picked >= 0.9f * top_p * all;  // (false for NaN)
    }
  } else {
    cluster_wait();
  }
  auto full_range = [&]() {  // the row's range, and a clean start of the ways below
    for (int b = tid; b < NB; b += NT) sm.hist[b] = 0;
    if (tid == 0) {
      sm.ncand = 0;
      sm.pick = -1;
    }
    bound();
    __syncthreads();
    if (tid < C) {
      st_cl(dsmem_addr(&sm.xmax[rank], tid), __float_as_uint(mx));
      st_cl(dsmem_addr(&sm.xmin[rank], tid), __float_as_uint(mn));
      tell_bound();
    }
    cluster_sync();
    for (int r = 0; r < C; ++r) {
      zmax = fmaxf(zmax, sm.xmax[r]);
      zmin = fminf(zmin, sm.xmin[r]);
    }
  };
  if (!local) full_range();
  const bool empty = !(zmax > -INFINITY);
  const bool odd = zmax == INFINITY || sm.c_pair.x == 0.f;
  // The unit of the masses: 2^lg times the bound is at most 2^62 (a vocabulary is
  // at most 2^20, and so is what a small top-k's lists hold, 2^10).
  int lg = 42;
  if (local && by_k0) {
    static_assert(PARTS == 1 << 10, "tokens of such a list");
    lg = 52;
  } else if (!odd && !empty) {
    float ub = 0.f;
    for (int r = 0; r < C; ++r)
      ub += sm.xub[r] * (sm.xmax[r] == zmax ? 1.f : exp2f((sm.xmax[r] - zmax) * sm.c_pair.x));
    lg = min(max(61 - (int)(__float_as_uint(ub * 1.001f) >> 23) + 127, 42), 62);
  }
  const Scale sc = {zmax, sm.c_pair.x, sm.c_pair.y, odd, lg};

  Cut cut = {KEY_NINF + 1, V};  // everything above -inf
  u64 total = 0;                // mass of the cut, when known
  bool list = false;            // the kept tokens are the first `n_kept` of the first CTA's list,
  int n_kept = 0;               // sorted, or ranked if it is small (then `lanes` lanes hold a token)
  bool small = false;
  u64 lkey = 0, lmass = 0, lcum = 0;
  int lrank = 0, lanes = 1;

  // Each warp's range of the slice's groups, and the warp (of the cluster) that
  // has a token.
  const int g0 = (int)((long long)s.groups * warp / NW), g1 = (int)((long long)s.groups * (warp + 1) / NW);
  auto group4 = [&](int q) {
    return q < g1 ? s.get4(q) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  };
  auto warp_of = [&](int id) {
    const int r = id / slice, begin = r * slice;
    const int first = begin - (int)((reinterpret_cast<uintptr_t>(z_row + begin) / sizeof(T)) % VEC);
    const int groups = (min(V, begin + slice) - first + VEC - 1) / VEC * (VEC / 4);
    return r * NW + (((id - first) / 4 + 1) * NW - 1) / groups;
  };
  bool by_warp = false;  // known: the mass each warp keeps, g_warp + sm.wkept[warp]
  u64 g_warp = 0;

  // Broadcasts the first CTA's sm.mk.  (Two turns: a CTA that still reads one
  // decision is at least a cluster barrier ahead of the next but one.)
  int told = 0;
  auto broadcast = [&]() -> const Decision& {
    if (rank == 0) {
      __syncthreads();
      for (int w = tid; w < DW * C; w += NT)
        st_cl(dsmem_addr(reinterpret_cast<unsigned*>(&sm.dec[told]) + w % DW, w / DW),
              reinterpret_cast<const unsigned*>(&sm.mk)[w % DW]);
    }
    cluster_sync();
    const Decision& d = sm.dec[told];
    told ^= 1;
    return d;
  };
  // Sums two masses over the cluster.
  int turn = 0;
  auto exchange = [&](u64& m, u64& g) {
    m = warp_sum_u64(m);
    g = warp_sum_u64(g);
    __syncthreads();
    if (lane == 0) {
      sm.wsum[warp] = m;
      sm.wsum2[warp] = g;
    }
    __syncthreads();
    if (tid < C) {
      m = g = 0;
      for (int w = 0; w < NW; ++w) m += sm.wsum[w], g += sm.wsum2[w];
      st_cl(dsmem_addr(&sm.xm[turn][rank], tid), m);
      st_cl(dsmem_addr(&sm.xg[turn][rank], tid), g);
    }
    cluster_sync();
    m = g = 0;
    for (int r = 0; r < C; ++r) m += sm.xm[turn][r], g += sm.xg[turn][r];
    turn ^= 1;
  };
  auto mass_into = [&](u64& m) {  // adds this thread's share of the kept mass
    const CutZ cz = cut_z(cut, V);
    for_each4(s, [&](const float4& v, int id) {
      u64 e[4];
      if (masses4(v, id, sc, sm.tab, cz, -1, e)) m += (e[0] + e[1]) + (e[2] + e[3]);
      else m += ((unsigned)e[0] + (unsigned)e[1]) + ((unsigned)e[2] + (unsigned)e[3]);  // (below 2^26)
    });
  };
  auto mass_kept = [&]() {
    u64 m = 0, g = 0;
    mass_into(m);
    exchange(m, g);
    return m;
  };

  if (!empty && greedy) {
    int id0 = 0x7fffffff;
    for_each(s, [&](float z, int id) {
      if (z == zmax) id0 = min(id0, id);
    });
    id0 = __reduce_min_sync(0xffffffffu, id0);
    if (lane == 0 && id0 != 0x7fffffff) atomicMin(&sm.pick2, id0);
    __syncthreads();
    if (tid < C) st_cl(dsmem_addr(&sm.xid[rank], tid), (unsigned)sm.pick2);
    cluster_sync();
    id0 = 0x7fffffff;
    for (int r = 0; r < C; ++r) id0 = min(id0, sm.xid[r]);
    cut = {okey(zmax), id0};
    total = 1ull << lg;
  }

  // ---- 2. top-k and top-p: a histogram of the row's range finds the bins that
  // hold a border; their tokens are gathered and sorted by the first CTA
  const bool by_k = !empty && by_k0, by_p = !empty && !greedy && top_p < 1.f;
  if (by_k || by_p) {
    auto cut_at = [&](int p) { return Cut{(unsigned)(sm.cand[p] >> 32), (int)~(unsigned)sm.cand[p]}; };
    // masses of the list in order: this thread's four, and the mass before them
    u64 lm[CAP / NT], lbefore = 0, lall = 0;
    auto scan_list = [&](int n) {
      u64 sum = 0;
#pragma unroll
      for (int j = 0; j < CAP / NT; ++j) {
        const int p = tid * (CAP / NT) + j;
        lm[j] = p < n ? mass_of(okey_value((unsigned)(sm.cand[p] >> 32)), sc, sm.tab) : 0ull;
        sum += lm[j];
      }
      lbefore = block_scan_u64(sum, &lall, sm);
    };
    // first position of the list whose running mass, after `ahead`, reaches `want`
    auto find_mass = [&](int n, u64 ahead, u64 want) {
      if (tid == 0) sm.pick2 = n - 1;
      __syncthreads();
      u64 c = ahead + lbefore;
#pragma unroll
      for (int j = 0; j < CAP / NT; ++j) {
        if (c < want && want <= c + lm[j]) sm.pick2 = tid * (CAP / NT) + j;
        c += lm[j];
      }
      __syncthreads();
      const int p = sm.pick2;
      __syncthreads();
      return p;
    };
    // mass of the list up to position p
    auto mass_to = [&](int p) {
      u64 c = lbefore;
#pragma unroll
      for (int j = 0; j < CAP / NT; ++j) {
        c += lm[j];
        if (tid * (CAP / NT) + j == p) sm.sel_before = c;
      }
      __syncthreads();
      const u64 v = sm.sel_before;
      __syncthreads();
      return v;
    };

    // Small lists are not sorted: a token's lanes (a power of two of them, as
    // many as there are threads for) find by one pass over the list how many
    // tokens are not behind it, and their mass.
    auto rank_list = [&](int n) {
      lanes = 32;
      while (lanes > 1 && n * lanes > NT) lanes >>= 1;
      const int t = tid / lanes;
      lkey = t < n ? sm.cand[t] : 0;
      lmass = t < n ? mass_of(okey_value((unsigned)(lkey >> 32)), sc, sm.tab) : 0ull;
      if (t < n) sm.radix[t] = lmass;
      if (tid == 0) sm.pick2 = 0;
      __syncthreads();
      lrank = 0;  // tokens up to and with this one
      lcum = 0;
      if (t < n) {
#pragma unroll 4
        for (int j = tid & (lanes - 1); j < n; j += lanes) {
          const bool in = sm.cand[j] >= lkey;
          lrank += in;
          lcum += in ? sm.radix[j] : 0ull;
        }
      }
      for (int o = 1; o < lanes; o <<= 1) {
        lrank += __shfl_xor_sync(0xffffffffu, lrank, o);
        lcum += __shfl_xor_sync(0xffffffffu, lcum, o);
      }
    };
    // the lanes of the list's p-th token (from 1) tell the others
    auto tell = [&](int slot, bool mine, u64 ahead) {
      if (mine) {
        sm.sel[slot].total = ahead + lcum;
        sm.sel[slot].cut = {(unsigned)(lkey >> 32), (int)~(unsigned)lkey};
        sm.sel[slot].n = lrank;
      }
      __syncthreads();
      total = sm.sel[slot].total;
      cut = sm.sel[slot].cut;
      n_kept = sm.sel[slot].n;
    };

    // top-k and top-p of a list that holds the row's first tokens
    auto cut_list = [&](int n) {
      small = n <= SMALL;
      if (small) {
        rank_list(n);
        tell(0, lrank > 0 && lrank == min(top_k, n), 0);
        if (by_p) {
          const u64 want = share_of(top_p, total);
          tell(1, lrank > 0 && lcum >= want && lcum - lmass < want, 0);
        }
      } else {
        sort_desc(sm.cand, n);
        scan_list(n);
        n_kept = min(top_k, n);
        total = mass_to(n_kept - 1);
        if (by_p) {
          n_kept = min(n_kept, find_mass(n, 0, share_of(top_p, total)) + 1);
          total = mass_to(n_kept - 1);
        }
      }
    };
    auto merge_parts = [&]() {
      // The parts in one piece (in any order), without what lies below any of
      // their bounds.  Then, if that leaves several warps' worth, each full
      // warp sorts 32 of them: with F warps, at least top_k tokens are not
      // below the least of the warps' ceil(top_k / F)-th tokens.
      float low = -INFINITY;
      for (int r = 0; r < C; ++r) low = fmaxf(low, sm.xlow[r]);
      const unsigned low_key = okey(low), lg_part = 10 - a.lg_cluster;
      static_assert(PARTS == 1 << 10, "lg_part");
      if (tid == 0) {
        sm.ncand = 0;
        sm.bound = ~0ull;
      }
      __syncthreads();
      auto append = [&](bool yes, u64 v) {
        const unsigned m = __ballot_sync(0xffffffffu, yes);
        if (!m) return;
        unsigned at = 0;
        if (lane == 0) at = atomicAdd(&sm.ncand, __popc(m));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1));
        if (yes) sm.cand[at] = v;
      };
#pragma unroll
      for (int j = 0; j < PARTS / NT; ++j) {
        const unsigned e = tid + j * NT, r = e >> lg_part;
        const u64 v = e - (r << lg_part) < (unsigned)sm.xid[r] ? sm.parts[e] : 0ull;
        append((unsigned)(v >> 32) >= low_key && v, v);
      }
      if (tid == 0) sm.pick = -1;
      __syncthreads();
      int all = (int)sm.ncand;
      const int full = all / 32;
      if (by_k && full >= 2 && top_k <= 32 * full) {
        static_assert(PARTS <= 2 * NT, "two tokens a thread");
        u64 v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = tid + j * NT;
          v[j] = e < all ? sm.cand[e] : 0ull;
          if (warp + j * NW < full) {
            u64 y = v[j];
#pragma unroll
            for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
              for (int o = k >> 1; o > 0; o >>= 1) {
                const u64 w = __shfl_xor_sync(0xffffffffu, y, o);
                const bool larger = ((lane & o) == 0) == ((lane & k) == 0);
                y = larger ? (y > w ? y : w) : (y < w ? y : w);
              }
            y = __shfl_sync(0xffffffffu, y, (top_k + full - 1) / full - 1);
            if (lane == 0) atomicMin(&sm.bound, y);
          }
        }
        __syncthreads();
        if (tid == 0) sm.ncand = 0;
        const u64 bound = sm.bound;
        __syncthreads();
        append(v[0] >= bound && v[0], v[0]);
        append(v[1] >= bound && v[1], v[1]);
        __syncthreads();
        all = (int)sm.ncand;
      }
      return all;
    };
    if (local && by_k) {
      list = true;
      if (rank == 0) cut_list(merge_parts());
    } else if (local) {
      u64 m = 0, g = 0;
      mass_into(m);
      exchange(m, g);
      if (rank == 0) {
        const int n = merge_parts();
        small = n <= SMALL;
        bool found = false;
        if (small) {
          const u64 want = share_of(top_p, m);
          rank_list(n);
          tell(0, lrank > 0 && lrank == n, 0);
          found = want <= total;
          if (found) tell(1, lrank > 0 && lcum >= want && lcum - lmass < want, 0);
        }
        if (tid == 0) sm.mk.step = found ? STEP_LIST : STEP_NONE;
      }
      list = broadcast().step == STEP_LIST;
      if (!list) {
        cut = {KEY_NINF + 1, V};
        total = 0;
        full_range();
      }
    }
    if (!list) {
    // bins of equal width over [zmax - 64, zmax] or the row's own range if that
    // is smaller; what lies lower falls into the last bin
    const float range = fminf(zmax - zmin, 64.f);
    const float per = range > 0.f ? fminf((float)NB / range, 1e30f) : 1.f;
    auto bin_of = [&](float z) { return z == zmax ? 0 : (int)fminf((zmax - z) * per, (float)(NB - 1)); };
    for_each(s, [&](float z, int) {
      if (z > -INFINITY) atomicAdd(&sm.hist[bin_of(z)], 1u);
    });
    cluster_sync();
    unsigned c2[2] = {0, 0};  // the first CTA's threads: counts of bins 2 tid, 2 tid + 1, then of those before
    u64 n_all = 0, n_before = 0;
    if (rank == 0) {
      for (int r = 0; r < C; ++r) {
        c2[0] += ld_cl(dsmem_addr(&sm.hist[2 * tid], r));
        c2[1] += ld_cl(dsmem_addr(&sm.hist[2 * tid + 1], r));
      }
      n_before = block_scan_u64(c2[0] + c2[1], &n_all, sm);
      __syncthreads();
      sm.hist[2 * tid] = c2[0];  // from here on the row's counts
      sm.hist[2 * tid + 1] = c2[1];
      if (tid == 0) sm.mk.step = STEP_NONE;
      __syncthreads();
      if (by_k && (u64)top_k < n_all) {
        for (int h = 0; h < 2; ++h) {
          const u64 b0 = n_before + (h ? c2[0] : 0);
          if (b0 < (u64)top_k && (u64)top_k <= b0 + c2[h]) {  // one thread
            const int b = 2 * tid + h;
            sm.mk.lo = b;
            sm.mk.hi = b;
            sm.mk.before = (unsigned)b0;
            if (b0 + c2[h] <= CAP) {
              sm.mk.lo = 0;
              sm.mk.before = 0;
              sm.mk.step = STEP_LIST;
            } else {
              sm.mk.step = c2[h] <= CAP ? STEP_TOPK : STEP_SLOW_K;
            }
          }
        }
      }
    }
    Decision dec = broadcast();
    // Copies this CTA's own list behind one reservation in the first CTA's.
    auto deliver = [&]() {
      __syncthreads();
      const unsigned n = min(sm.nlocal, (unsigned)CAP);
      if (tid == 0) sm.sel_key = add_cl(dsmem_addr(&sm.ncand, 0), n);
      __syncthreads();
      const unsigned at = sm.sel_key;
      for (unsigned e = tid; e < n; e += NT)
        if (at + e < CAP) st_cl(dsmem_addr(sm.cand + at + e, 0), sm.cand[e]);
    };
    // Gathers the tokens of the decision's bins into the first CTA's list.
    auto gather = [&](int lo, int hi) {
      // (bounds beyond the bins' ends, roundings included, skip most)
      const float low = hi == NB - 1 ? -INFINITY : zmax - (float)(hi + 1) / per * 1.0001f;
      const float high = lo == 0 ? INFINITY : zmax - (float)lo / per * 0.9999f;
      auto in = [&](float z) { const int b = bin_of(z); return b >= lo && b <= hi; };
      if (rank == 0) {
        collect(s, low, high, in, &sm.ncand, sm.cand, CAP);
      } else {
        if (tid == 0) sm.nlocal = 0;
        __syncthreads();
        collect(s, low, high, in, &sm.nlocal, sm.cand, CAP);
        deliver();
      }
    };
    // The smallest logit in a bin ahead of bin b > 0 (bins fall as logits rise):
    // a search over the keys, 32 at a time, from a bracket around the bin's end.
    auto bin_end = [&](int b) {
      const float d = (float)b / per;
      unsigned lo = KEY_NINF + 1, hi = okey(zmax);
      const unsigned k0 = okey(zmax - d * 1.0001f), k1 = okey(zmax - d * 0.9999f);
      if (k0 > lo && k0 <= hi && bin_of(okey_value(k0)) >= b) lo = k0;
      if (k1 < hi && k1 >= lo && bin_of(okey_value(k1)) < b) hi = k1;
      while (lo < hi) {
        const unsigned step = (hi - lo + 31) >> 5, k = lo + min(step * lane, hi - lo);
        const unsigned yes = __ballot_sync(0xffffffffu, bin_of(okey_value(k)) < b);
        const int f = yes ? __ffs(yes) - 1 : 32;
        const unsigned last = __shfl_sync(0xffffffffu, k, max(f - 1, 0));
        const unsigned first = __shfl_sync(0xffffffffu, k, f & 31);
        if (f < 32) hi = first;
        if (f > 0) lo = last + 1;
      }
      return okey_value(hi);
    };

    if (dec.step == STEP_LIST) {
      gather(0, dec.hi);
      cluster_sync();
      list = true;
      if (rank == 0) cut_list((int)sm.ncand);
    } else {
      if (dec.step == STEP_TOPK) {
        gather(dec.lo, dec.hi);
        cluster_sync();
        if (rank == 0) {
          const int n = (int)sm.ncand;
          sort_desc(sm.cand, n);
          if (tid == 0) {
            sm.mk.cut = cut_at(top_k - (int)dec.before - 1);
            sm.ncand = 0;
          }
        }
        cut = broadcast().cut;
      } else if (dec.step == STEP_SLOW_K) {
        if (rank == 0) {
          const Cut c = select_slow(z_row, V, sc, cut, true, (u64)top_k, sm);
          if (tid == 0) sm.mk.cut = c;
        }
        cut = broadcast().cut;
      }
      if (by_p) {
        // The border's bin is guessed from the counts and each bin's middle;
        // the exact masses decide, and where they put the border elsewhere they
        // correct the next guess.
        float want_f = 0.f;
        int lo_least = 0, hi_most = NB - 1;  // bins the border may still be in
        if (rank == 0) {
          if (dec.step != STEP_NONE) hi_most = dec.lo;
          __syncthreads();
          float w2[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int b = 2 * tid + h;
            w2[h] = b <= hi_most && c2[h] ? (float)c2[h] * exp2f(-((float)b + 0.5f) / per * sc.hi) : 0.f;
          }
          float inc = w2[0] + w2[1];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
          }
          if (lane == 31) sm.fsum[warp] = inc;
          __syncthreads();
          float before = inc - w2[0] - w2[1], all = 0.f;
          for (int w = 0; w < NW; ++w) {
            if (w < warp) before += sm.fsum[w];
            all += sm.fsum[w];
          }
          sm.ecum[2 * tid] = before;
          sm.ecum[2 * tid + 1] = before + w2[0];
          if (tid == 0) sm.ecum[NB] = all;
          want_f = top_p * all;
        }
        const Cut given = cut;
        for (int tries = 0;; ++tries) {
          if (rank == 0) {
            if (tid == 0) sm.pick2 = lo_least;
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int b = 2 * tid + h;
              if (b > lo_least && b <= hi_most && sm.hist[b] && sm.ecum[b] < want_f) atomicMax(&sm.pick2, b);
            }
            __syncthreads();
            if (tid == 0) {
              int lo = sm.pick2, hi = lo;
              unsigned n = sm.hist[lo];
              bool up = true, down = true;
              // Widen by turns, by 16 bins a side at most, so that a guess that is
              // a few bins off still holds the border (not at all: one flat row
              // 44.6 us instead of 48.0, a peaked one whose border is in the
              // tail 73 instead of 59; by 64: 59 again, and 64 rows of a steep
              // distribution 106 instead of 95).
              for (int d = 0; d < 32 && (up || down); ++d) {
                bool& side = d & 1 ? up : down;
                if (!side) continue;
                const int b = d & 1 ? lo - 1 : hi + 1;
                side = b >= lo_least && b <= hi_most && n + sm.hist[b] <= CAP;
                if (!side) continue;
                n += sm.hist[b];
                lo = min(lo, b);
                hi = max(hi, b);
              }
              sm.mk.lo = lo;
              sm.mk.hi = hi;
              // (guesses corrected by exact masses: more than two were not seen to
              // matter, times are the same with 2; 8 bounds them)
              sm.mk.step = n <= CAP && tries < 8 ? STEP_TOPP : STEP_SLOW_P;
              sm.ncand = 0;
            }
          }
          dec = broadcast();
          const int lo = dec.lo, hi = dec.hi;
          // One pass: the kept mass, what of it lies ahead of the decision's bins
          // (by warp too, each a contiguous range of groups, for the draw), and
          // those bins' tokens into the first CTA's list.
          u64 m = 0, g = 0;
          const bool take = dec.step == STEP_TOPP;
          const float ahead = lo ? bin_end(lo) : NAN;
          const float least = !take ? NAN : hi == NB - 1 ? -3.402823466e+38f : bin_end(hi + 1);
          unsigned* counter = rank ? &sm.nlocal : &sm.ncand;
          if (tid == 0) sm.nlocal = 0;
          __syncthreads();
          const CutZ cz = cut_z(cut, V);
          for (int q0 = g0; q0 < g1; q0 += 32) {
            const float4 v = group4(q0 + lane);
            const float z[4] = {v.x, v.y, v.z, v.w};
            const int id = s.first + 4 * (q0 + lane);
            u64 e[4];
            masses4(v, id, sc, sm.tab, cz, -1, e);
            bool in[4], any = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool before = z[j] >= ahead;
              m += e[j];
              g += before ? e[j] : 0ull;
              in[j] = !before && z[j] >= least;
              any = any || in[j];
            }
            if (__any_sync(0xffffffffu, any)) append4(z, in, id, counter, sm.cand, CAP);
          }
          g_warp = warp_sum_u64(g);
          if (take && rank) deliver();
          exchange(m, g);
          if (rank == 0) {
            const u64 want = share_of(top_p, m);
            bool found = false, slow = dec.step == STEP_SLOW_P;
            if (!slow) {
              const int n = (int)sm.ncand;
              int n_list = n;
              small = n <= SMALL;
              u64 ga = g;  // mass ahead of the part of the list that is ranked
              u64 v[CAP / NT];
#pragma unroll
              for (int j = 0; j < CAP / NT; ++j) v[j] = tid + j * NT < n ? sm.cand[tid + j * NT] : 0ull;
              if (small) {
                rank_list(n);
                tell(0, lrank > 0 && lrank == n, 0);
                lall = n ? total : 0ull;
              } else if (lo > 0) {
                // finer bins find the border's few tokens; the rest is not needed
                const float top = zmax - (float)lo / per, fine = (float)SUB / ((float)(hi + 1 - lo) / per);
                int sb[CAP / NT];
                sm.sub[0][tid] = sm.sub[1][tid] = sm.sub[2][tid] = 0;
                __syncthreads();
#pragma unroll
                for (int j = 0; j < CAP / NT; ++j) {
                  const float z = okey_value((unsigned)(v[j] >> 32));
                  sb[j] = (int)fminf(fmaxf((top - z) * fine, 0.f), (float)(SUB - 1));
                  if (v[j]) sub_add(sm, sb[j], mass_of(z, sc, sm.tab));
                }
                __syncthreads();
                const u64 mine = sub_get(sm, tid);
                const u64 before = block_scan_u64(mine, &lall, sm);
                if (g + before < want && want <= g + before + mine) {
                  sm.pick2 = tid;
                  sm.sel_before = g + before;
                }
                __syncthreads();
                if (g < want && want <= g + lall) {
                  const int b = sm.pick2;
                  ga = sm.sel_before;
                  unsigned c = 0;
#pragma unroll
                  for (int j = 0; j < CAP / NT; ++j) c += v[j] && sb[j] == b;
                  u64 n2;
                  unsigned at = (unsigned)block_scan_u64(c, &n2, sm);
#pragma unroll
                  for (int j = 0; j < CAP / NT; ++j)
                    if (v[j] && sb[j] == b) sm.cand[at++] = v[j];
                  __syncthreads();
                  small = n2 <= SMALL;
                  if (small) {
                    rank_list((int)n2);
                  } else {
                    const u64 whole = lall;
                    sort_desc(sm.cand, (int)n2);
                    scan_list((int)n2);
                    lall = whole;
                  }
                  n_list = (int)n2;
                }
              } else {
                sort_desc(sm.cand, n);
                scan_list(n);
              }
              // (tokens of the last bin past the top-k cut stay behind the border:
              // the mass up to the cut is m, and want <= m)
              if (g < want && want <= g + lall) {
                found = true;
                if (small) {
                  tell(1, lrank > 0 && ga + lcum >= want && ga + lcum - lmass < want, ga);
                } else {
                  const int p = find_mass(n_list, ga, want);
                  total = ga + mass_to(p);
                  cut = cut_at(p);
                  n_kept = p + 1;
                }
                if (tid == 0) sm.mk.cut = cut;
                if (lo > 0 && a.kind != SAMPLING_PROBS) {
                  // what each warp of the cluster keeps of these bins
                  __syncthreads();
                  if (tid < CMAX * NW) sm.sub[0][tid] = sm.sub[1][tid] = sm.sub[2][tid] = 0;
                  __syncthreads();
#pragma unroll
                  for (int j = 0; j < CAP / NT; ++j) {
                    const unsigned key = (unsigned)(v[j] >> 32);
                    const int id = (int)~(unsigned)v[j];
                    if (v[j] && kept(key, id, cut)) sub_add(sm, warp_of(id), mass_of(okey_value(key), sc, sm.tab));
                  }
                  __syncthreads();
                  if (tid < C * NW) st_cl(dsmem_addr(&sm.wkept[tid % NW], tid / NW), sub_get(sm, tid));
                }
              } else {
                cut = given;  // not the list's
                const bool later = want > g;
                const u64 at = later ? g + lall : g;
                want_f = sm.ecum[later ? hi + 1 : lo] +
                         (float)((long long)want - (long long)at) * pow2f(-lg);
                if (later) lo_least = hi + 1;
                else hi_most = lo - 1;
                slow = lo_least > hi_most;
                __syncthreads();
              }
            }
            if (slow) {
              const Cut c = select_slow(z_row, V, sc, cut, false, want, sm);
              if (tid == 0) sm.mk.cut = c;
              total = 0;
            }
            if (tid == 0) {
              sm.mk.step = found && lo == 0 ? STEP_LIST : found || slow ? STEP_NONE : STEP_TOPP;
              sm.mk.total_lo = (unsigned)total;
              sm.mk.total_hi = (unsigned)(total >> 32);
            }
          }
          dec = broadcast();
          if (dec.step != STEP_TOPP) break;
        }
        cut = dec.cut;
        total = ((u64)dec.total_hi << 32) | dec.total_lo;
        list = dec.step == STEP_LIST;
        by_warp = total > 0;
      }
    }
    }
    if (list && rank == 0) {
      const unsigned mk = min_p > 0.f ? min_p_key(zmax, sm.off_pair) : 0u;
      if (small) {
        if (min_p > 0.f) {
          if (lrank > 0 && lrank <= n_kept && (unsigned)(lkey >> 32) >= mk) atomicMax(&sm.pick2, lrank);
          __syncthreads();
          tell(2, lrank > 0 && lrank == sm.pick2, 0);
        }
      } else {
        if (min_p > 0.f) {
          if (tid == 0) sm.pick2 = 0;
          __syncthreads();
          for (int p = tid; p < n_kept; p += NT)
            if ((unsigned)(sm.cand[p] >> 32) >= mk) atomicMax(&sm.pick2, p);
          __syncthreads();
          n_kept = sm.pick2 + 1;
          __syncthreads();
          total = mass_to(n_kept - 1);
        }
        cut = cut_at(n_kept - 1);
        __syncthreads();  // the list is reordered below
      }
    }
  }
  if (!list && !empty && !greedy && min_p > 0.f) {
    const unsigned mk = min_p_key(zmax, sm.off_pair);
    if (mk > cut.key) {
      cut = {mk, V};
      total = 0;
      by_warp = false;
    }
  }

  // ---- 3. the outputs
  if (empty && rank == 0 && tid == 0) flag(a.status, DFLASH2_DEV_EMPTY_ROW);
  if (a.kind == SAMPLING_PROBS) {
    if (list) {  // the others need the first CTA's cut
      if (rank == 0 && tid == 0) {
        sm.mk.cut = cut;
        sm.mk.total_lo = (unsigned)total;
        sm.mk.total_hi = (unsigned)(total >> 32);
      }
      const Decision dec = broadcast();
      cut = dec.cut;
      total = ((u64)dec.total_hi << 32) | dec.total_lo;
    } else if (!empty && total == 0) {
      total = mass_kept();
    }
    float* p = a.prob + (size_t)row * V;
    const float zc = okey_value(cut.key);
    const float inv = empty ? 0.f : pow2f(lg) / (float)total;
    for (int q = tid; q < 4 * s.groups; q += NT) {
      const int id = s.first + q;
      if (id < s.begin || id >= s.end) continue;
      const float z = RES ? ld(zs_buf + q) : ld(z_row + id);
      p[id] = !empty && kept_z(z, id, zc, cut.id) ? mass_f32(z, sc) * inv : 0.f;
    }
    return;
  }
  const bool verify = a.kind == SAMPLING_VERIFY;
  u64 x_mass = 0;  // kept mass of the draft's token
  if (list && rank != 0) return;  // the rest is the first CTA's
  if (!empty && x >= 0 && x < V && kept(okey(zx), x, cut)) x_mass = mass_of(zx, sc, sm.tab);
  auto passes = [&]() {
    return floor_share(a.u_accept[(size_t)seq * (a.rows - 1) + i], total) < x_mass;
  };
  auto threshold = [&](u64 sum) { return floor_share(a.u[seq], sum); };
  // One warp of the cluster ends the row; of a verified sequence's rows, the
  // last to end joins them.
  auto finish = [&](int token, bool pass) {
    if (!verify) {
      if (lane == 0) {
        a.token[row] = token;
        if (a.prob)
          a.prob[row] = token < 0 ? 0.f : mass_f32(ld(z_row + token), sc) * pow2f(lg) / (float)total;
      }
      return;
    }
    if (!a.arrived) {
      if (lane == 0) a.rowout[row] = make_int2(pass, token);
      return;
    }
    int last = 0;
    if (lane == 0) {
      a.rowout[row] = make_int2(pass, token);
      __threadfence();
      last = atomicAdd(a.arrived + seq, 1) == nd;
      if (last) a.arrived[seq] = 0;
      __threadfence();
    }
    last = __shfl_sync(0xffffffffu, last, 0);
    __syncwarp();  // what lane 0 has seen, the warp has (a shuffle orders no memory)
    if (last) join_rows(a, seq, nd);
  };
  if (empty) {
    if (rank == 0 && warp == 0) finish(-1, false);
    return;
  }
  if (greedy) {
    if (rank == 0 && warp == 0) finish(cut.id, verify && i < nd && x == cut.id);
    return;
  }
  if (list) {
    const bool pass = verify && i < nd && passes();
    if (!pass && small) {
      // the kept tokens in one piece (by rank), then the running mass in id
      // order at each of them, its lanes as many as there are threads for
      if (lrank > 0 && lrank <= n_kept) {
        sm.cand[CAP - 1 - lrank] = lkey;  // (the list itself lies below)
        sm.radix[lrank - 1] = (int)~(unsigned)lkey != x ? lmass : 0ull;
      }
      __syncthreads();
      lanes = 32;
      while (lanes > 1 && n_kept * lanes > NT) lanes >>= 1;
      const int t0 = tid / lanes;
      const u64* kept_list = sm.cand + CAP - 2;  // token of rank r + 1 at kept_list[-r]
      const unsigned me = t0 < n_kept ? (unsigned)kept_list[-t0] : 0u;
      const u64 e = t0 < n_kept ? sm.radix[t0] : 0ull;
      u64 c = 0;
      if (e) {
#pragma unroll 4
        for (int j = tid & (lanes - 1); j < n_kept; j += lanes) c += (unsigned)kept_list[-j] >= me ? sm.radix[j] : 0ull;
      }
      for (int o = 1; o < lanes; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      const u64 t = threshold(total - x_mass);
      if (e && c - e <= t && t < c) sm.pick = (int)~me;
      __syncthreads();
    } else if (!pass) {
      // the kept tokens in id order, and the first whose running mass exceeds the draw
      for (int p = tid; p < n_kept; p += NT) {
        const u64 v = sm.cand[p];
        sm.cand[p] = (v << 32) | (v >> 32);  // (~id, key): descending is ascending ids
      }
      __syncthreads();
      sort_desc(sm.cand, n_kept);
      u64 e[CAP / NT], sum = 0, all;
#pragma unroll
      for (int j = 0; j < CAP / NT; ++j) {
        const int p = tid * (CAP / NT) + j;
        e[j] = 0;
        if (p < n_kept && (int)~(unsigned)(sm.cand[p] >> 32) != x) e[j] = mass_of(okey_value((unsigned)sm.cand[p]), sc, sm.tab);
        sum += e[j];
      }
      u64 c = block_scan_u64(sum, &all, sm);
      if (all) {
        const u64 t = threshold(all);
#pragma unroll
        for (int j = 0; j < CAP / NT; ++j) {
          if (c <= t && t < c + e[j]) sm.pick = (int)~(unsigned)(sm.cand[tid * (CAP / NT) + j] >> 32);
          c += e[j];
        }
      }
      __syncthreads();
    }
    if (warp == 0) finish(pass ? -1 : sm.pick, pass);
    return;
  }
  // no list: masses by warp
  const CutZ cz = cut_z(cut, V);
  auto mass4 = [&](int q, u64 (&e)[4]) { masses4(group4(q), s.first + 4 * q, sc, sm.tab, cz, x, e); };
  u64 wm = 0;
  if (by_warp) {
    wm = g_warp + sm.wkept[warp];
    if (x_mass && x >= s.begin && x < s.end && warp_of(x) == rank * NW + warp) wm -= x_mass;
  } else {
    for (int q0 = g0; q0 < g1; q0 += 32) {
      u64 e[4];
      mass4(q0 + lane, e);
      wm += e[0] + e[1] + e[2] + e[3];
    }
    wm = warp_sum_u64(wm);
  }
  __syncthreads();
  if (lane == 0) sm.wsum[warp] = wm;
  __syncthreads();
  u64 before = 0, mine = 0;
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += sm.wsum[w];
    mine += sm.wsum[w];
  }
  if (tid < C) st_cl(dsmem_addr(&sm.xm[turn][rank], tid), mine);
  cluster_sync();
  u64 rest = 0;
  for (int r = 0; r < C; ++r) {
    if (r < rank) before += sm.xm[turn][r];
    rest += sm.xm[turn][r];
  }
  total = rest + x_mass;
  const bool pass = verify && i < nd && passes();
  if (pass || rest == 0) {
    if (rank == 0 && warp == 0) finish(-1, pass);
    return;
  }
  const u64 t = threshold(rest);
  if (!(before <= t && t < before + wm)) return;
  // this warp holds the token
  u64 c = before;
  for (int q0 = g0; q0 < g1; q0 += 32) {
    u64 e[4];
    mass4(q0 + lane, e);
    const u64 sum = e[0] + e[1] + e[2] + e[3];
    u64 inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const u64 step_sum = __shfl_sync(0xffffffffu, inc, 31);
    if (t < c + step_sum) {
      u64 d = c + inc - sum;
      int token = -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (d <= t && t < d + e[j]) token = s.first + 4 * (q0 + lane) + j;
        d += e[j];
      }
      const unsigned m = __ballot_sync(0xffffffffu, token >= 0);
      finish(__shfl_sync(0xffffffffu, token, __ffs(m) - 1), false);
      return;
    }
    c += step_sum;
  }
}

template <typename T, bool RES>
int launch_one(const SamplingArgs& a, int slice, const Ctx& c) {
  auto kern = sample_kernel<T, RES>;
  static std::atomic<unsigned long long> opted{0};  // devices whose kernel may use the largest size
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DFLASH2_ERR_CUDA;
  if (RES && !(opted.load(std::memory_order_relaxed) >> dev & 1)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SLICE_BYTES + 64) != cudaSuccess)
      return DFLASH2_ERR_CUDA;
    opted.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  const size_t smem = RES ? (size_t)((slice + 15 + 8) / 8 * 8) * sizeof(T) : 0;
  return launch_kx(kern, dim3((a.batch * a.rows) << a.lg_cluster), dim3(NT), smem, c, 1 << a.lg_cluster, a, slice);
}

// A row's cluster: as few CTAs as hold it in shared memory with two of them an
// SM, more while the rows leave SMs idle.  (64 bf16 rows of 151936 in clusters of
// 4 and 8, us: small top-k 18 and 28, flat nucleus 90 and 144, but settings of
// their own 82 and 62, the few rows of the long way taking half as long.
// Clusters of 3, 5, 6 or 7 where those suffice: 256 fp32 rows of 102400 77 to 309
// us against 87 to 354, but 64 to 200 rows of 50257 and 128256 2 to 9% longer.)
// (Rows shared out over one wave instead, up to one CTA a row that reads its logits again from L2 in every
// pass, took 315 us against 106 at 256 rows of 151936: the few rows without a
// small top-k keep their one CTA long after the others are done.)  What does
// not fit is read again from L2.
template <typename T>
int launch_rows(SamplingArgs a, const Ctx& c) {
  const long long rows = (long long)a.batch * a.rows;
  constexpr int SLICE = SLICE_BYTES / (int)sizeof(T);
  a.lg_cluster = 0;
  while (1 << a.lg_cluster < CMAX && (a.vocab > SLICE << a.lg_cluster ||
                                      (rows << a.lg_cluster < c.nsm && a.vocab > 4096 << a.lg_cluster)))
    ++a.lg_cluster;
  const int slice = ((a.vocab + (1 << a.lg_cluster) - 1 >> a.lg_cluster) + 7) / 8 * 8;
  return slice <= SLICE ? launch_one<T, true>(a, slice, c) : launch_one<T, false>(a, slice, c);
}

}  // namespace

int launch_sampling(const SamplingArgs& a, const Ctx& c) {
  const int rc = a.bf16_logits ? launch_rows<bf16>(a, c) : launch_rows<float>(a, c);
  if (rc != DFLASH2_OK || a.kind != SAMPLING_VERIFY || a.arrived) return rc;
  return launch_k(join_kernel, dim3((a.batch + 3) / 4), dim3(128), 0, c, a);
}

}  // namespace df2
