// Changes that a request's settings make to rows of logits: penalties of
// tokens that were there already, biases, and a bit mask of what a grammar
// allows.
//
//   z' = z / rho (z > 0) or z rho   for seen tokens      (repetition)
//   z' = z - f c - p [c > 0]        c: count of a token  (frequency, presence)
//   z' = z + b                      the token's bias, then -inf where the mask has no bit
//
// Row i of a sequence counts the sequence's tokens and its first i drafts,
// so a block's rows are changed for verification as they would be one by
// one.  The work is one pass over the rows: what bounds it is memory.  A
// block takes a slice of the vocabulary of all rows of one sequence: it walks
// the sequence's tokens once, counts those of its slice in shared memory and
// lists them, streams the rows through the mask, and then goes through the
// list: the few tokens that have more to them than the mask do not slow the
// others down (looked up in the stream, they cost 130 us where 256 rows of
// 151936 bfloat16 take 40).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 5952;  // tokens of a slice at most: 48 KB of tables, four blocks an SM
constexpr int kMaxDrafts = 31;
constexpr int kAhead = 8;  // tokens of the history that a thread has in flight
constexpr int kRows = 4;  // rows whose loads a thread has in flight
constexpr uint32_t kSeen = 0x80000000u;

struct Row {
  float rho, presence, frequency;
};

// The new value of token v (slice entry e) in row i; `path` the sequence's drafts.
__device__ __forceinline__ float changed(const AdjustArgs& a, const Row& w, float z, int v, uint32_t count, int bias,
                                         const int32_t* path, int i, const float* bias_row) {
  bool seen = count & kSeen;
  int c = (int)(count & ~kSeen);
  for (int j = 0; j < i; ++j)
    if (path[j] == v) {
      seen = true;
      ++c;
    }
  if (seen) z = z > 0.f ? z / w.rho : z * w.rho;
  if (c > 0) z = (z - w.frequency * (float)c) - w.presence;
  if (bias > 0) z += bias_row[bias - 1];
  return z;
}

// -inf where `keep` has no bit: 4 floats or 8 bfloat16.
__device__ __forceinline__ void blank(uint4& x, uint32_t keep, float) {
  const uint32_t inf = 0xff800000u;
  if (!(keep & 1)) x.x = inf;
  if (!(keep & 2)) x.y = inf;
  if (!(keep & 4)) x.z = inf;
  if (!(keep & 8)) x.w = inf;
}
__device__ __forceinline__ uint32_t blank2(uint32_t x, uint32_t keep) {
  if (!(keep & 1)) x = (x & 0xffff0000u) | 0xff80u;
  if (!(keep & 2)) x = (x & 0xffffu) | 0xff800000u;
  return x;
}
__device__ __forceinline__ void blank(uint4& x, uint32_t keep, bf16) {
  x.x = blank2(x.x, keep);
  x.y = blank2(x.y, keep >> 2);
  x.z = blank2(x.z, keep >> 4);
  x.w = blank2(x.w, keep >> 6);
}

// R rows of nv tokens from v0 on, -inf where the mask has no bit; R x B loads
// of a thread are in flight together.  16-byte accesses where the rows are
// equally far from their border (R > 1: all of them), the rest one by one.
template <typename T, int R, int B>
__device__ __forceinline__ void copy_rows(const T* in, long long stride, T* out, long long out_stride,
                                          const uint32_t* mask, int words, int v0, int nv) {
  constexpr int E = 16 / sizeof(T);
  const bool even = (uintptr_t)in % 16 == (uintptr_t)out % 16;
  const int head = even ? min(nv, (E - (int)((uintptr_t)in % 16 / sizeof(T))) % E) : nv;
  const int body = (nv - head) / E, loose = nv - body * E;
  for (int x = threadIdx.x; x < loose * R; x += kThreads) {
    const int i = R == 1 ? 0 : x / loose, y = x - i * loose, e = y < head ? y : y + body * E;
    const bool keep = !mask || ((mask[i * (size_t)words + ((v0 + e) >> 5)] >> ((v0 + e) & 31)) & 1u);
    const T z = in[i * (size_t)stride + e];
    if (keep) out[i * (size_t)out_stride + e] = z;
    else st(out + i * (size_t)out_stride + e, -INFINITY);
  }
  for (int b0 = threadIdx.x; b0 < body; b0 += kThreads * B) {
    uint4 x[R * B];
    uint32_t keep[R * B];
#pragma unroll
    for (int u = 0; u < R * B; ++u) {
      const int i = u / B, b = b0 + u % B * kThreads, e = head + b * E;
      if (B > 1 && b >= body) continue;
      x[u] = __ldcs(reinterpret_cast<const uint4*>(in + i * (size_t)stride + e));
      keep[u] = 0xffffffffu;
      if (mask) {
        const uint32_t* m = mask + i * (size_t)words;
        keep[u] = __funnelshift_r(m[(v0 + e) >> 5], m[(v0 + e + E - 1) >> 5], (v0 + e) & 31);
      }
    }
#pragma unroll
    for (int u = 0; u < R * B; ++u) {
      const int i = u / B, b = b0 + u % B * kThreads;
      if (B > 1 && b >= body) continue;
      blank(x[u], keep[u], T());
      *reinterpret_cast<uint4*>(out + i * (size_t)out_stride + head + b * E) = x[u];
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) adjust_kernel(const __grid_constant__ AdjustArgs a, int slice) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ uint32_t sh[];
  uint32_t* count = sh;                                             // [slice] kSeen | count
  uint32_t* touched = count + slice;                                // [slice / 32] bits
  uint16_t* list = reinterpret_cast<uint16_t*>(touched + slice / 32);  // [slice] the entries with a bit
  uint16_t* bias_at = list + slice;                                    // [slice] last entry of the token + 1
  __shared__ int32_t path[kMaxDrafts + 1];
  __shared__ int listed;
  pdl_launch_next();
  pdl_wait();
  const int s = blockIdx.y, v0 = blockIdx.x * slice, nv = min(slice, a.vocab - v0);
  const bool biased = a.n_bias > 0;
  for (int i = threadIdx.x; i < slice; i += kThreads) {
    count[i] = 0;
    if (biased) bias_at[i] = 0;
  }
  for (int i = threadIdx.x; i < slice / 32; i += kThreads) touched[i] = 0;
  if (threadIdx.x == 0) listed = 0;
  auto touch = [&](int e) {
    const uint32_t bit = 1u << (e & 31);
    if (!(atomicOr(touched + (e >> 5), bit) & bit)) list[atomicAdd(&listed, 1)] = (uint16_t)e;
  };
  const Row w = {a.repetition ? a.repetition[s] : 1.f, a.presence ? a.presence[s] : 0.f,
                 a.frequency ? a.frequency[s] : 0.f};
  const bool penal = w.rho != 1.f || w.presence != 0.f || w.frequency != 0.f;
  __syncthreads();
  if (penal) {
    int n = a.n_tokens ? a.n_tokens[s] : 0;
    if (n < 0 || n > a.max_tokens) {
      if (threadIdx.x == 0) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
      n = n < 0 ? 0 : a.max_tokens;
    }
    const int prompt = a.prompt_len ? a.prompt_len[s] : 0;
    const int32_t* tok = a.tokens + (size_t)s * a.max_tokens;
    for (int i0 = 0; i0 < n; i0 += kAhead * kThreads) {
      int t[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads + threadIdx.x;
        t[u] = i < n ? tok[i] : v0 - 1;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads + threadIdx.x, e = t[u] - v0;
        if (i < n && (unsigned)t[u] >= (unsigned)a.vocab) flag(a.status, DFLASH2_DEV_BAD_TOKEN);
        else if ((unsigned)e < (unsigned)nv) {
          atomicOr(count + e, kSeen);
          if (i >= prompt) atomicAdd(count + e, 1u);
          touch(e);
        }
      }
    }
    if (a.path && threadIdx.x < a.rows - 1) {
      const int t = a.path[(size_t)s * (a.rows - 1) + threadIdx.x], e = t - v0;
      path[threadIdx.x] = t;
      if (t < -1 || t >= a.vocab) flag(a.status, DFLASH2_DEV_BAD_TOKEN);
      else if (t >= 0 && e >= 0 && e < nv) touch(e);
    }
  }
  if (biased) {
    // entries of the slice; of one token's several the last counts: 16-bit
    // halves have no maximum of their own, so the word is exchanged
    for (int i = threadIdx.x; i < a.n_bias; i += kThreads) {
      const int t = a.bias_id[(size_t)s * a.n_bias + i], e = t - v0;
      if (t < -1 || t >= a.vocab) {
        flag(a.status, DFLASH2_DEV_BAD_TOKEN);
      } else if (t >= 0 && e >= 0 && e < nv) {
        uint32_t* word = reinterpret_cast<uint32_t*>(bias_at) + (e >> 1);
        const int shift = 16 * (e & 1);
        uint32_t was = *word;
        while ((int)((was >> shift) & 0xffffu) < i + 1) {
          const uint32_t now = (was & ~(0xffffu << shift)) | ((uint32_t)(i + 1) << shift);
          const uint32_t got = atomicCAS(word, was, now);
          if (got == was) break;
          was = got;
        }
        touch(e);
      }
    }
  }
  __syncthreads();
  const float* bias_row = biased ? a.bias + (size_t)s * a.n_bias : nullptr;
  const int words = (a.vocab + 31) / 32;
  const T* in0 = static_cast<const T*>(a.logits) + (size_t)s * a.rows * (size_t)a.stride + v0;
  T* out0 = static_cast<T*>(a.out) + (size_t)s * a.rows * (size_t)a.out_stride + v0;
  const uint32_t* mask0 = a.mask ? a.mask + (size_t)s * a.rows * (size_t)words : nullptr;
  // the rows through the mask alone, kRows rows at a time, or the row
  for (int i = 0; i < a.rows;) {
    const T* in = in0 + i * (size_t)a.stride;
    T* out = out0 + i * (size_t)a.out_stride;
    const uint32_t* mask = mask0 ? mask0 + i * (size_t)words : nullptr;
    const bool many = a.rows - i >= kRows && a.stride % E == 0 && a.out_stride % E == 0;
    if (many) copy_rows<T, kRows, 1>(in, a.stride, out, a.out_stride, mask, words, v0, nv);
    else copy_rows<T, 1, 4>(in, a.stride, out, a.out_stride, mask, words, v0, nv);
    i += many ? kRows : 1;
  }
  // then the tokens that anything concerns, from the rows as they were (in
  // place too: the copy has changed only what the mask takes out)
  __syncthreads();
  const int all = listed * a.rows;
  for (int x0 = threadIdx.x; x0 < all; x0 += kAhead * kThreads) {
    float z[kAhead];
    bool keep[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int x = x0 + u * kThreads, k = x / a.rows, i = x - k * a.rows;
      keep[u] = x < all;
      if (keep[u]) {
        const int e = list[k];
        if (mask0) keep[u] = (mask0[i * (size_t)words + ((v0 + e) >> 5)] >> ((v0 + e) & 31)) & 1u;
        z[u] = ld(in0 + i * (size_t)a.stride + e);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (!keep[u]) continue;
      const int x = x0 + u * kThreads, k = x / a.rows, i = x - k * a.rows, e = list[k];
      st(out0 + i * (size_t)a.out_stride + e,
         changed(a, w, z[u], v0 + e, count[e], biased ? bias_at[e] : 0, path, penal && a.path ? i : 0, bias_row));
    }
  }
}

}  // namespace

int launch_adjust(const AdjustArgs& a, const Ctx& c) {
  const long long all = (long long)a.vocab * a.batch;
  const int per = (int)std::min<long long>(kMaxSlice, std::max<long long>(256, all / (4 * c.nsm)));
  const int slice = (per + 63) / 64 * 64;
  const size_t smem = (size_t)slice * 6 + slice / 8 + (a.n_bias > 0 ? (size_t)slice * 2 : 0);
  const dim3 grid((a.vocab + slice - 1) / slice, a.batch);
  return a.bf16_logits ? launch_k(adjust_kernel<bf16>, grid, dim3(kThreads), smem, c, a, slice)
                       : launch_k(adjust_kernel<float>, grid, dim3(kThreads), smem, c, a, slice);
}

}  // namespace df2
