// Attention of a sequence's last tokens over its paged cache, in the general
// form: any page size, head dimension 64 or 128, bfloat16 or 8-bit rows.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(scale log2(e) q k_j - m)
//
// over the keys j that the token sees, with the running maximum m.  A block
// takes four query rows (token, head) of a kv head, so that a key loaded
// once serves all four; its key slots (8 lanes each, every lane holding d / 8
// of a key's values) walk the keys in turns, each with a maximum, a sum and
// an accumulator of its own.  Where blocks are few, a cluster of CTAs shares
// a block's keys.  Slots meet by shuffles, warps in shared memory, CTAs in
// each other's.  Hidden keys are stepped over, never multiplied by zero, so
// what lies in them (a NaN, an infinity) does not matter.
//
// What bounds it: for a few keys the chain lengths, block table, keys and
// values, meeting (5 us); then about 0.8 us for every 32 keys of a CTA, the
// latency of its loads and of scores, weights and sums in turn.  One token of
// 300 keys and 8 kv heads: 6.9 us (numbers one by one instead of by twos: 7.6; one CTA a block, and its slots meeting in
// shared memory: 18; tensor cores: 18).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kWarps = 8;
constexpr int kSlots = kWarps * 4;  // keys in flight
constexpr int kRows = 4;            // query rows of a block
constexpr int kMaxCluster = 8;      // CTAs that share the keys of a block

// A lane's part of a row as it lies in memory: D / 8 values.
template <int D, bool E4M3>
struct Piece {
  static constexpr int kWords = D / 8 * (E4M3 ? 1 : 2) / 4;
  uint32_t w[kWords];
  float s;
  __device__ __forceinline__ void load(const void* pool, const uint8_t* exps, size_t row, int sub) {
    const uint32_t* p = static_cast<const uint32_t*>(pool) + (row * 8 + sub) * kWords;
    if (kWords == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x;
      w[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i + 3 < kWords; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + i);
        w[i] = x.x;
        w[i + 1] = x.y;
        w[i + 2] = x.z;
        w[i + 3] = x.w;
      }
    }
    if (E4M3) s = __uint_as_float((uint32_t)exps[row] << 23);
  }
  __device__ __forceinline__ void widen(uint64_t (&x)[D / 16]) const {  // two numbers each
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      if (E4M3) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[i] = mul2(pack2(f.x, f.y), pack2(s, s));
      } else {
        x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      }
    }
  }
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) attend_rows_kernel(const __grid_constant__ AttendArgs a, int ctas) {
  constexpr int E = D / 8;  // values of a row per lane
  __shared__ __align__(16) float part[kWarps][kRows][D];
  __shared__ float2 part_ml[kWarps][kRows], ml[kRows];  // maximum and sum
  __shared__ __align__(16) float whole[kRows][D];
  pdl_launch_next();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7, slot = warp * 4 + (lane >> 3);
  const int block = blockIdx.x / ctas, rank = blockIdx.x - block * ctas;
  const int h = blockIdx.y, s = blockIdx.z, group = a.nq / a.nkv;
  const int n = a.n_new ? min(max(a.n_new[s], 0), a.n_tok) : a.n_tok;
  const int first = block * kRows;
  if (a.n_new && n != a.n_new[s] && threadIdx.x == 0) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
  if (first >= n * group) return;  // (all of its CTAs)
  int len = a.kv_len[s];
  if (len < 0 || (long long)len > (long long)a.max_pages * a.page_size) {
    if (threadIdx.x == 0) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
    len = len < 0 ? 0 : a.max_pages * a.page_size;
  }
  uint64_t q[kRows][E / 2], acc[kRows][E / 2];
  float m[kRows], l[kRows];
  int lo[kRows], hi[kRows];
  int from = len, to = 0, all_lo = 0, all_hi = len;  // keys that some and that all of the rows see
  const float scale = a.scale * 1.4426950408889634f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = min(first + r, n * group - 1), t = row / group;
    Piece<D, false> p;
    p.load(a.q + ((size_t)s * a.n_tok + t) * a.q_stride + (size_t)(h * group + row % group) * D, nullptr, 0, sub);
    p.widen(q[r]);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      q[r][i] = mul2(q[r][i], pack2(scale, scale));
      acc[r][i] = 0ull;
    }
    m[r] = -INFINITY;
    l[r] = 0.f;
    hi[r] = a.causal ? len - (n - 1 - t) : len;
    lo[r] = a.window > 0 ? max(0, hi[r] - a.window) : 0;
    from = min(from, lo[r]);
    to = max(to, hi[r]);
    all_lo = max(all_lo, lo[r]);
    all_hi = min(all_hi, hi[r]);
  }
  // page of key j (the shared positions are read through the first sequence's row)
  auto page_of = [&](int j) {
    if (j >= to) return -1;
    const int page = a.block_table[(size_t)(j < a.shared_len ? 0 : s) * a.max_pages + j / a.page_size];
    if (page >= 0 && page < a.n_pages) return page;
    flag(a.status, DFLASH2_DEV_BAD_PAGE);
    return -1;
  };
  // a key's rows are asked for while the one before is worked on, its page before that
  const int step = kSlots * ctas;
  Piece<D, E4M3> pk, pv, next_k, next_v;
  auto fetch = [&](int j, int page, Piece<D, E4M3>& k, Piece<D, E4M3>& v) {
    if (page < 0) return;
    const size_t row = ((size_t)page * a.page_size + j % a.page_size) * a.nkv + h;
    k.load(a.k, a.k_exp, row, sub);
    v.load(a.v, a.v_exp, row, sub);
  };
  int j = from + rank * kSlots + slot, page = page_of(j), next = page_of(j + step);
  fetch(j, page, pk, pv);
#pragma unroll 1
  for (int j0 = from + rank * kSlots; j0 < to; j0 += step) {
    const bool there = page >= 0;
    const int at = j;
    j += step;
    page = next;
    next = page_of(j + step);
    fetch(j, page, next_k, next_v);
    uint64_t x[E / 2];
    float dot[kRows];
    if (there) pk.widen(x);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      dot[r] = 0.f;
      if (there) {
        uint64_t two = 0ull;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) two = fma2(q[r][i], x[i], two);
        float even, odd;
        unpack2(two, even, odd);
        dot[r] = even + odd;
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], o);
    }
    if (there) pv.widen(x);
    auto raise = [&](int r) {  // the maximum, if the key's score is above it
      const float mn = fmaxf(m[r], dot[r]), f = ex2(m[r] - (mn == -INFINITY ? 0.f : mn));
      m[r] = mn;
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) acc[r][i] = mul2(acc[r][i], pack2(f, f));
    };
    auto add = [&](int r) {
      const float p = ex2(dot[r] - (m[r] == -INFINITY ? 0.f : m[r]));
      l[r] += p;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) acc[r][i] = fma2(pack2(p, p), x[i], acc[r][i]);
    };
    // (without branches between them the rows' chains run side by side)
    if (__all_sync(0xffffffffu, there && at >= all_lo && at < all_hi)) {
      bool up = false;
#pragma unroll
      for (int r = 0; r < kRows; ++r) up |= dot[r] > m[r];
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) raise(r);
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) add(r);
    } else {
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (there && at >= lo[r] && at < hi[r]) {
          raise(r);
          add(r);
        }
    }
    pk = next_k;
    pv = next_v;
  }
  // slots of a warp, warps of a CTA, CTAs of a cluster
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float top = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 8));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
    const float f = ex2(m[r] - (top == -INFINITY ? 0.f : top));
    l[r] *= f;
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
    if (lane == 0) part_ml[warp][r] = make_float2(top, l[r]);
    float o[E];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      unpack2(mul2(acc[r][i], pack2(f, f)), o[2 * i], o[2 * i + 1]);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        o[2 * i + b] += __shfl_xor_sync(0xffffffffu, o[2 * i + b], 8);
        o[2 * i + b] += __shfl_xor_sync(0xffffffffu, o[2 * i + b], 16);
      }
    }
    if (lane < 8)
#pragma unroll
      for (int i = 0; i < E; i += 4)
        *reinterpret_cast<float4*>(&part[warp][r][sub * E + i]) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
  }
  __syncthreads();
  auto store = [&](int r, int d, float sum, float2 o) {
    const int row = first + r;
    if (row >= n * group) return;
    const __nv_bfloat162 y = __floats2bfloat162_rn(sum == 0.f ? 0.f : o.x / sum, sum == 0.f ? 0.f : o.y / sum);
    *reinterpret_cast<__nv_bfloat162*>(a.out + ((size_t)s * a.n_tok + row / group) * a.out_stride +
                                       (size_t)(h * group + row % group) * D + d) = y;
  };
  constexpr int kPairs = kRows * D / 2;
  if ((int)threadIdx.x < kPairs) {
    const int r = threadIdx.x / (D / 2), d = threadIdx.x % (D / 2) * 2;
    float top = -INFINITY, sum = 0.f;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) top = fmaxf(top, part_ml[k][r].x);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float f = ex2(part_ml[k][r].x - ref);
      const float2 x = *reinterpret_cast<const float2*>(&part[k][r][d]);
      sum = fmaf(part_ml[k][r].y, f, sum);
      o.x = fmaf(x.x, f, o.x);
      o.y = fmaf(x.y, f, o.y);
    }
    if (ctas == 1) {
      store(r, d, sum, o);
    } else {
      *reinterpret_cast<float2*>(&whole[r][d]) = o;
      if (d == 0) ml[r] = make_float2(top, sum);
    }
  }
  if (ctas > 1) {
    cluster_sync();
    const int share = kPairs / ctas, i = rank * share + threadIdx.x;
    if ((int)threadIdx.x < share) {
      const int r = i / (D / 2), d = i % (D / 2) * 2;
      float2 from_ml[kMaxCluster], x[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        const int c = min(k, ctas - 1);
        from_ml[k] = ld_dsmem2(dsmem_addr(&ml[r], c));
        x[k] = ld_dsmem2(dsmem_addr(&whole[r][d], c));
        if (k >= ctas) from_ml[k] = make_float2(-INFINITY, 0.f);
      }
      float top = -INFINITY, sum = 0.f;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) top = fmaxf(top, from_ml[k].x);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k >= ctas) continue;
        const float f = ex2(from_ml[k].x - ref);
        sum = fmaf(from_ml[k].y, f, sum);
        o.x = fmaf(x[k].x, f, o.x);
        o.y = fmaf(x[k].y, f, o.y);
      }
      store(r, d, sum, o);
    }
    cluster_sync();  // (nobody leaves before its shared memory has been read)
  }
}

}  // namespace

static std::atomic<int> g_mode{0};
void attend_force_mode(int mode) { g_mode.store(mode); }

int launch_attend(const AttendArgs& a, void* workspace, const Ctx& c) {
  const int blocks = (a.n_tok * (a.nq / a.nkv) + kRows - 1) / kRows;
  const long long all = (long long)blocks * a.nkv * a.batch, cap = (long long)a.max_pages * a.page_size;
  // As many CTAs share a block's keys as find SMs, and keys: a CTA fills its
  // SM, and 16 clusters of 8 do not run at once (one token of 288 keys in 16
  // blocks: 13 us, with 4 CTAs each 8).
  int ctas = kMaxCluster;
  while (ctas > 1 && (all * ctas > (ctas == 8 ? c.nsm / 2 : c.nsm) || (ctas / 2) * kSlots >= cap)) ctas /= 2;
  // The tensor cores wherever their kernel goes, but for little work: theirs
  // starts late (plan, tiles, a second kernel; 13 to 20 us), this one takes 5
  // us and then 0.8 for every time a CTA goes over its slots, at most as often
  // as the block table allows.  us here and there, by times, bfloat16 and 8
  // heads of 4: 1 token (12 times: 2976 keys) 15 and 26, 4 sequences (12: 1536)
  // 15 and 22, 16 (15: 480) 16 and 23, (24: 768) 23 and 25, 32 (12: 192) 16 and
  // 24, (30: 480) 31 and 29; 8-bit, 16 (24: 768) 27 and 28.  (With 2 heads of 8
  // the tensor cores start some us earlier: 18 us at 16 sequences of 768, 12
  // times.)
  const long long times = (cap + kSlots * ctas - 1) / (kSlots * ctas) * ((all * ctas + c.nsm - 1) / c.nsm);
  const int mode = g_mode.load();
  if (mode != 1 && (times > 15 || mode == 2) && attend_tc_fits(a)) return launch_attend_tc(a, workspace, c);
  const dim3 grid(blocks * ctas, a.nkv, a.batch), block(32 * kWarps);
  if (a.d == 64)
    return a.e4m3 ? launch_kx(attend_rows_kernel<64, true>, grid, block, 0, c, ctas, a, ctas)
                  : launch_kx(attend_rows_kernel<64, false>, grid, block, 0, c, ctas, a, ctas);
  return a.e4m3 ? launch_kx(attend_rows_kernel<128, true>, grid, block, 0, c, ctas, a, ctas)
                : launch_kx(attend_rows_kernel<128, false>, grid, block, 0, c, ctas, a, ctas);
}

}  // namespace df2
