// Rows of keys and values written into a paged cache and read back, with
// the cache in bfloat16 or quantised as it is written.
//
// The 8-bit form keeps a head's row of d values as e4m3 codes and one
// exponent byte b, a code c standing for c * 2^(b - 127):
//   b = the smallest byte >= 1 with max|x| <= 448 * 2^(b - 127),
//   c = e4m3(x * 2^(127 - b))  (nearest, ties to even).
// The scale is a power of two, which costs a floating-point code no
// precision (at most one binade at the bottom of its range) and makes every
// product with it exact, so a row reads back as exactly what is stored.  The
// scaling itself is exact too, so the only rounding is the code's.
//
// Both directions are copies: what bounds them is memory, and for a few rows
// the latency of the chain offsets -> block table -> row.  A thread holds 8
// values (one 16-byte access of bf16), the d / 8 threads of a head form its
// maximum by shuffles, and a block takes `rpb` rows, whose destinations its
// threads find together while the values are on their way.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 16;  // rows of a block at most

// Row of the pool (pages laid end to end) of each of the block's rows, or -1.
__device__ __forceinline__ void find_rows(const CacheRowsArgs& a, int r0, int n, long long* place) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) place[i] = -1;
  __syncthreads();
  // every thread looks at some of the sequences for all rows of the block:
  // one trip to memory, where a search would take several
  for (int s = threadIdx.x; s < a.batch; s += blockDim.x) {
    const int lo = a.off[s], hi = a.off[s + 1];
    if (hi <= r0 || lo >= r0 + n) continue;
    const long long first = a.start ? a.start[s] : 0;
    for (int r = max(lo, r0); r < min(hi, r0 + n); ++r) {
      const long long p = first + (r - lo);
      if (p < 0 || p >= (long long)a.max_pages * a.page_size) {
        flag(a.status, DFLASH2_DEV_BAD_LENGTH);
        continue;
      }
      const int page = a.block_table[(size_t)s * a.max_pages + p / a.page_size];
      if (page < 0 || page >= a.n_pages) {
        flag(a.status, DFLASH2_DEV_BAD_PAGE);
        continue;
      }
      place[r - r0] = (long long)page * a.page_size + p % a.page_size;
    }
  }
  __syncthreads();
}

// 8 bf16 values -> 8 codes and the row's exponent byte; the threads of a row
// are `width` (8 or 16) neighbouring lanes.
__device__ __forceinline__ uint2 quantise8(const uint4& raw, int width, int* byte) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  uint32_t top = 0;  // bits of the largest finite magnitude
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __float_as_uint(x[i]) & 0x7fffffffu;
    if (m >= 0x7f800000u) x[i] = __int_as_float(0x7fffffff);  // infinities become NaN, which e4m3 has
    else top = max(top, m);
  }
  for (int o = width >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  // top = 1.m * 2^(e - 127) against 448 = 1.75 * 2^8
  const int b = max(1, (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
  *byte = b;
  const float inv = __uint_as_float((uint32_t)(254 - b) << 23);  // 2^(127 - b)
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h] * inv, x[4 * h + 1] * inv), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * h + 2] * inv, x[4 * h + 3] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    c[h] = lo | (hi << 16);
  }
  return make_uint2(c[0], c[1]);
}

__device__ __forceinline__ uint4 widen8(const uint2& c, int byte) {
  const float s = __uint_as_float((uint32_t)byte << 23);  // 2^(byte - 127)
  const uint32_t w[2] = {c.x, c.y};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool READ, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_rows_kernel(CacheRowsArgs a, int rpb) {
  __shared__ long long place[kMaxRows];
  pdl_launch_next();
  pdl_wait();
  const int r0 = blockIdx.x * rpb, n = min(rpb, a.rows - r0);
  const int vec = a.nkv * a.d / 8;  // 16-byte pieces of a row of keys or values
  const int items = n * vec * 2;
  const int width = a.d / 8;
  if (READ) {
    find_rows(a, r0, n, place);
    const int covered = a.off[a.batch];  // rows behind the last sequence are left as they are
    for (int i0 = 0; i0 < items; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      if (i >= items) break;
      const int part = i / (n * vec), j = i % (n * vec), r = j / vec, c = j % vec;
      if (r0 + r >= covered) continue;
      const long long p = place[r];
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      const void* pool = part ? a.v : a.k;
      if (p >= 0) {
        const size_t at = (size_t)p * vec + c;
        if (E4M3) {
          const int head = c / width;
          v = widen8(static_cast<const uint2*>(pool)[at], (part ? a.v_exp : a.k_exp)[(size_t)p * a.nkv + head]);
        } else {
          v = static_cast<const uint4*>(pool)[at];
        }
      }
      bf16* out = static_cast<bf16*>(part ? a.v_rows : a.k_rows);
      reinterpret_cast<uint4*>(out + (size_t)(r0 + r) * (part ? a.v_stride : a.k_stride))[c] = v;
    }
    return;
  }
  // the values do not depend on where they go: they are asked for first
  constexpr int kAhead = 8;
  uint4 x[kAhead];
  const int rounds = (items + kThreads - 1) / kThreads;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int i = u * kThreads + threadIdx.x;
    if (i < items) {
      const int part = i / (n * vec), j = i % (n * vec), r = j / vec, c = j % vec;
      const bf16* in = static_cast<const bf16*>(part ? a.v_rows : a.k_rows);
      x[u] = reinterpret_cast<const uint4*>(in + (size_t)(r0 + r) * (part ? a.v_stride : a.k_stride))[c];
    }
  }
  find_rows(a, r0, n, place);
  for (int u0 = 0; u0 < rounds; u0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = (u0 + u) * kThreads + threadIdx.x;
      const bool in_range = i < items;
      if (!__any_sync(0xffffffffu, in_range)) break;
      const int part = in_range ? i / (n * vec) : 0, j = in_range ? i % (n * vec) : 0, r = j / vec, c = j % vec;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (in_range) {
        if (u0 == 0) {
          v = x[u];
        } else {
          const bf16* in = static_cast<const bf16*>(part ? a.v_rows : a.k_rows);
          v = reinterpret_cast<const uint4*>(in + (size_t)(r0 + r) * (part ? a.v_stride : a.k_stride))[c];
        }
      }
      const long long p = in_range ? place[r] : -1;
      if (E4M3) {
        int byte;
        const uint2 q = quantise8(v, width, &byte);  // (whole warps: it shuffles)
        if (p >= 0) {
          static_cast<uint2*>(part ? a.v : a.k)[(size_t)p * vec + c] = q;
          if (c % width == 0) (part ? a.v_exp : a.k_exp)[(size_t)p * a.nkv + c / width] = (uint8_t)byte;
        }
      } else if (p >= 0) {
        static_cast<uint4*>(part ? a.v : a.k)[(size_t)p * vec + c] = v;
      }
    }
  }
}

}  // namespace

int launch_cache_rows(const CacheRowsArgs& a, bool read, const Ctx& c) {
  // rows of a block: enough that a thread has several accesses in flight,
  // few enough that the blocks cover the SMs
  const int vec = a.nkv * a.d / 8 * 2;
  int rpb = std::max(1, std::min(kMaxRows, 8 * kThreads / vec));
  while (rpb > 1 && (a.rows + rpb - 1) / rpb < 2 * c.nsm) --rpb;
  const dim3 grid((a.rows + rpb - 1) / rpb);
  if (read)
    return a.e4m3 ? launch_k(cache_rows_kernel<true, true>, grid, dim3(kThreads), 0, c, a, rpb)
                  : launch_k(cache_rows_kernel<true, false>, grid, dim3(kThreads), 0, c, a, rpb);
  return a.e4m3 ? launch_k(cache_rows_kernel<false, true>, grid, dim3(kThreads), 0, c, a, rpb)
                : launch_k(cache_rows_kernel<false, false>, grid, dim3(kThreads), 0, c, a, rpb);
}

}  // namespace df2
