// Attention of a sequence's last tokens over its paged cache, in the general
// form: any page size, head dimension 64 or 128, bfloat16 or 8-bit rows.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(scale log2(e) q k_j - m)
//
// over the keys j that the token sees, with the running maximum m.  A block
// takes four query rows (token, head) of a kv head, so that a key loaded
// once serves all four; its key slots (8 lanes each, every lane holding d / 8
// of a key's values) walk the keys in turns, each with a maximum, a sum and
// an accumulator of its own, and are merged at the end.  Hidden keys are
// stepped over, never multiplied by zero, so what lies in them (a NaN, an
// infinity) does not matter.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kWarps = 8;
constexpr int kSlots = kWarps * 4;  // keys in flight
constexpr int kRows = 4;            // query rows of a block

template <int D, bool E4M3>
__device__ __forceinline__ void load_row(const void* pool, const uint8_t* exps, size_t row, int sub, float (&x)[D / 8]) {
  if (E4M3) {
    const uint8_t* p = static_cast<const uint8_t*>(pool) + row * D + sub * (D / 8);
    const float s = __uint_as_float((uint32_t)exps[row] << 23);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint2 c = *reinterpret_cast<const uint2*>(p + 8 * i);
      const uint32_t w[2] = {c.x, c.y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[8 * i + 2 * j] = f.x * s;
        x[8 * i + 2 * j + 1] = f.y * s;
      }
    }
  } else {
    const bf16* p = static_cast<const bf16*>(pool) + row * D + sub * (D / 8);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 c = *reinterpret_cast<const uint4*>(p + 8 * i);
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) attend_rows_kernel(AttendArgs a) {
  constexpr int E = D / 8;  // values of a row per lane
  __shared__ float sh[kSlots][D + 2];
  pdl_launch_next();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7, slot = warp * 4 + (lane >> 3);
  const int h = blockIdx.y, s = blockIdx.z, group = a.nq / a.nkv;
  const int n = a.n_new ? min(max(a.n_new[s], 0), a.n_tok) : a.n_tok;
  const int first = blockIdx.x * kRows;
  if (a.n_new && n != a.n_new[s] && threadIdx.x == 0) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
  if (first >= n * group) return;
  int len = a.kv_len[s];
  if (len < 0 || (long long)len > (long long)a.max_pages * a.page_size) {
    if (threadIdx.x == 0) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
    len = len < 0 ? 0 : a.max_pages * a.page_size;
  }
  float q[kRows][E], acc[kRows][E], m[kRows], l[kRows];
  int lo[kRows], hi[kRows];
  int from = len, to = 0;
  const float scale = a.scale * 1.4426950408889634f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = min(first + r, n * group - 1), t = row / group;
    const bf16* p = a.q + ((size_t)s * a.n_tok + t) * a.q_stride + (size_t)(h * group + row % group) * D + sub * E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      q[r][i] = __bfloat162float(p[i]) * scale;
      acc[r][i] = 0.f;
    }
    m[r] = -INFINITY;
    l[r] = 0.f;
    hi[r] = a.causal ? len - (n - 1 - t) : len;
    lo[r] = a.window > 0 ? max(0, hi[r] - a.window) : 0;
    from = min(from, lo[r]);
    to = max(to, hi[r]);
  }
  for (int j0 = from; j0 < to; j0 += kSlots) {
    const int j = j0 + slot;
    float x[E];
    int page = -1;
    if (j < to) {
      // the shared positions are read through the first sequence's row
      page = a.block_table[(size_t)(j < a.shared_len ? 0 : s) * a.max_pages + j / a.page_size];
      if (page < 0 || page >= a.n_pages) {
        flag(a.status, DFLASH2_DEV_BAD_PAGE);
        page = -1;
      }
    }
    const size_t row = page < 0 ? 0 : ((size_t)page * a.page_size + j % a.page_size) * a.nkv + h;
    if (page >= 0) load_row<D, E4M3>(a.k, a.k_exp, row, sub, x);
    float dot[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      dot[r] = 0.f;
      if (page >= 0)
#pragma unroll
        for (int i = 0; i < E; ++i) dot[r] = fmaf(q[r][i], x[i], dot[r]);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], o);
    }
    if (page < 0) continue;
    load_row<D, E4M3>(a.v, a.v_exp, row, sub, x);
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (j < lo[r] || j >= hi[r]) continue;
      const float mn = fmaxf(m[r], dot[r]);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[r] - ref), p = exp2f(dot[r] - ref);
      m[r] = mn;
      l[r] = fmaf(l[r], f, p);
#pragma unroll
      for (int i = 0; i < E; ++i) acc[r][i] = fmaf(acc[r][i], f, p * x[i]);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) sh[slot][sub * E + i] = acc[r][i];
    if (sub == 0) {
      sh[slot][D] = m[r];
      sh[slot][D + 1] = l[r];
    }
    __syncthreads();
    if (first + r < n * group && threadIdx.x < D) {
      float top = -INFINITY;
      for (int k = 0; k < kSlots; ++k) top = fmaxf(top, sh[k][D]);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f, o = 0.f;
      for (int k = 0; k < kSlots; ++k) {
        const float w = exp2f(sh[k][D] - ref);
        sum = fmaf(sh[k][D + 1], w, sum);
        o = fmaf(sh[k][threadIdx.x], w, o);
      }
      const int row = first + r;
      a.out[((size_t)s * a.n_tok + row / group) * a.out_stride + (size_t)(h * group + row % group) * D + threadIdx.x] =
          __float2bfloat16_rn(sum == 0.f ? 0.f : o / sum);
    }
  }
}

}  // namespace

int launch_attend(const AttendArgs& a, void* workspace, const Ctx& c) {
  // The tensor cores wherever their kernel goes (one token of 300 keys: 17 us
  // against 18 here; 32 x 8 tokens at contexts 512-4096: 66 against 1870).
  if (attend_tc_fits(a)) return launch_attend_tc(a, workspace, c);
  const dim3 grid((a.n_tok * (a.nq / a.nkv) + kRows - 1) / kRows, a.nkv, a.batch), block(32 * kWarps);
  if (a.d == 64)
    return a.e4m3 ? launch_k(attend_rows_kernel<64, true>, grid, block, 0, c, a)
                  : launch_k(attend_rows_kernel<64, false>, grid, block, 0, c, a);
  return a.e4m3 ? launch_k(attend_rows_kernel<128, true>, grid, block, 0, c, a)
                : launch_k(attend_rows_kernel<128, false>, grid, block, 0, c, a);
}

}  // namespace df2
