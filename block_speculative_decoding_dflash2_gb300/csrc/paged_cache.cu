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
// the latency of the chain offsets -> block table -> row.  A warp takes a row,
// its keys and its values, 16 bytes of bfloat16 a lane and step; it finds the
// row's place by itself (32 offsets a look), so no warp waits for another,
// and the values to write are asked for before that.  33,500 rows of 8 heads
// of 128 quantised on their way in take 47 us (4.4 TB/s, bound by the
// conversion's instructions), 72,000 read back 81 us (5.5 TB/s); a few rows
// take 5.  (Blocks that shared their lookups, a division for every 16 bytes:
// 102 and 122 us.)
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 8;  // pieces of 16 bytes that a lane has in flight

// Row of the pool (pages laid end to end) of row r, or -1; *past: behind the
// last sequence.  All lanes of a warp, the same r.
__device__ __forceinline__ long long place_of(const CacheRowsArgs& a, int r, bool* past) {
  const int lane = threadIdx.x & 31;
  // the last sequence whose offset is not above r
  int lo = 0, n = a.batch;
  *past = false;
  while (true) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const int o = i < lo + n ? a.off[i] : INT32_MAX, end = n <= 32 ? (i < lo + n ? a.off[i + 1] : 0) : 0;
    const uint32_t below = __ballot_sync(0xffffffffu, i < lo + n && o <= r);
    if (!below) return -1;  // (offsets that do not start at 0)
    const int k = 31 - __clz(below);
    if (step == 1) {
      const int s = lo + k, first = __shfl_sync(0xffffffffu, o, k);
      if (r >= __shfl_sync(0xffffffffu, end, k)) {
        *past = true;
        return -1;
      }
      const long long p = (a.start ? a.start[s] : 0) + (long long)(r - first);
      if (p < 0 || p >= (long long)a.max_pages * a.page_size) {
        if (lane == 0) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
        return -1;
      }
      const int pi = (int)p / a.page_size, page = a.block_table[(size_t)s * a.max_pages + pi];
      if (page < 0 || page >= a.n_pages) {
        if (lane == 0) flag(a.status, DFLASH2_DEV_BAD_PAGE);
        return -1;
      }
      return (long long)page * a.page_size + ((int)p - pi * a.page_size);
    }
    lo += k * step;
    n = min(step, n - k * step);
  }
}

// 8 bf16 values -> 8 codes and the row's exponent byte; the lanes of a head
// are `width` (8 or 16) neighbours.
__device__ __forceinline__ uint2 quantise8(const uint4& raw, int width, int* byte) {
  uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  // the largest magnitude (NaN is passed over)
  __nv_bfloat162 m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = w[i] & 0x7fff7fffu;
    m[i] = *reinterpret_cast<const __nv_bfloat162*>(&x);
  }
  m[0] = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
  for (int o = width >> 1; o > 0; o >>= 1) {
    const uint32_t x = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&m[0]), o);
    m[0] = __hmax2(m[0], *reinterpret_cast<const __nv_bfloat162*>(&x));
  }
  uint32_t top = __float_as_uint(fmaxf(__low2float(m[0]), __high2float(m[0])));
  if (__any_sync(0xffffffffu, !(top < 0x7f800000u))) {
    // infinities or NaN alone: the largest finite magnitude, and NaN for the infinities, which e4m3 has not
    top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (w[i] << 16) & 0x7fffffffu, hi = w[i] & 0x7fff0000u;
      if (lo >= 0x7f800000u) w[i] |= 0x7fffu;
      else top = max(top, lo);
      if (hi >= 0x7f800000u) w[i] |= 0x7fff0000u;
      else top = max(top, hi);
    }
    for (int o = width >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  // top = 1.m * 2^(e - 127) against 448 = 1.75 * 2^8
  const int b = max(1, (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
  *byte = b;
  const float inv = __uint_as_float((uint32_t)(254 - b) << 23);  // 2^(127 - b)
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
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
__global__ void __launch_bounds__(32 * kWarps) cache_rows_kernel(const __grid_constant__ CacheRowsArgs a) {
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= a.rows) return;
  const int width = a.d / 8, lg_width = width == 16 ? 4 : 3;  // pieces of a head
  const int vec = a.nkv << lg_width;                          // pieces of a row of keys or values
  uint4* rows[2] = {reinterpret_cast<uint4*>(static_cast<bf16*>(a.k_rows) + (size_t)r * a.k_stride),
                    reinterpret_cast<uint4*>(static_cast<bf16*>(a.v_rows) + (size_t)r * a.v_stride)};
  // pieces 0 .. vec - 1 are the keys', vec .. 2 vec - 1 the values'
  uint4 x[kAhead];
  if (!READ) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int q = 32 * u + lane;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (q < 2 * vec) x[u] = __ldcs(q < vec ? rows[0] + q : rows[1] + (q - vec));
    }
  }
  bool past;
  const long long place = place_of(a, r, &past);
  if (READ ? past : place < 0) return;  // rows behind the last sequence are left as they are
  const size_t at = (size_t)max(place, 0ll) * vec;
  for (int q0 = 0; q0 < 2 * vec; q0 += 32 * kAhead) {
    if (READ) {
      int byte[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int q = q0 + 32 * u + lane;
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        byte[u] = 0;
        if (q < 2 * vec && place >= 0) {
          const bool v = q >= vec;
          const int c = v ? q - vec : q;
          if (E4M3) {
            const uint2 y = __ldcs(static_cast<const uint2*>(v ? a.v : a.k) + at + c);
            x[u].x = y.x;
            x[u].y = y.y;
            byte[u] = (v ? a.v_exp : a.k_exp)[(size_t)place * a.nkv + (c >> lg_width)];
          } else {
            x[u] = __ldcs(static_cast<const uint4*>(v ? a.v : a.k) + at + c);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int q = q0 + 32 * u + lane;
        if (q < 2 * vec)
          *(q < vec ? rows[0] + q : rows[1] + (q - vec)) = E4M3 ? widen8(make_uint2(x[u].x, x[u].y), byte[u]) : x[u];
      }
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int q = q0 + 32 * u + lane;
        if (q0 + 32 * u >= 2 * vec) break;  // (the whole warp)
        if (q0 > 0) {
          x[u] = make_uint4(0u, 0u, 0u, 0u);
          if (q < 2 * vec) x[u] = __ldcs(q < vec ? rows[0] + q : rows[1] + (q - vec));
        }
        const bool v = q >= vec;
        const int c = v ? q - vec : q;
        if (E4M3) {
          int byte;
          const uint2 y = quantise8(x[u], width, &byte);  // (whole warps: it shuffles)
          if (q < 2 * vec) {
            static_cast<uint2*>(v ? a.v : a.k)[at + c] = y;
            if ((c & (width - 1)) == 0) (v ? a.v_exp : a.k_exp)[(size_t)place * a.nkv + (c >> lg_width)] = (uint8_t)byte;
          }
        } else if (q < 2 * vec) {
          static_cast<uint4*>(v ? a.v : a.k)[at + c] = x[u];
        }
      }
    }
  }
}

}  // namespace

int launch_cache_rows(const CacheRowsArgs& a, bool read, const Ctx& c) {
  const dim3 grid((a.rows + kWarps - 1) / kWarps), block(32 * kWarps);
  if (read)
    return a.e4m3 ? launch_k(cache_rows_kernel<true, true>, grid, block, 0, c, a)
                  : launch_k(cache_rows_kernel<true, false>, grid, block, 0, c, a);
  return a.e4m3 ? launch_k(cache_rows_kernel<false, true>, grid, block, 0, c, a)
                : launch_k(cache_rows_kernel<false, false>, grid, block, 0, c, a);
}

}  // namespace df2
