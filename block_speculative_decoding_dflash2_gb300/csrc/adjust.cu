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
// the sequence's tokens once, counts those of its slice in shared memory, and
// streams the rows through.  A bit per token says whether anything but the
// mask concerns it, so for nearly all of them the counts are not read.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 8000;  // tokens of a slice at most: 48 KB of tables, four blocks an SM
constexpr int kMaxDrafts = 31;
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

template <typename T>
__global__ void __launch_bounds__(kThreads) adjust_kernel(AdjustArgs a, int slice) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ uint32_t sh[];
  uint32_t* count = sh;                                             // [slice] kSeen | count
  uint32_t* touched = count + slice;                                // [slice / 32 + 1] bits
  uint16_t* bias_at = reinterpret_cast<uint16_t*>(touched + slice / 32 + 1);  // [slice] last entry of the token + 1
  __shared__ int32_t path[kMaxDrafts + 1];
  pdl_launch_next();
  pdl_wait();
  const int s = blockIdx.y, v0 = blockIdx.x * slice, nv = min(slice, a.vocab - v0);
  const bool biased = a.n_bias > 0;
  for (int i = threadIdx.x; i < slice; i += kThreads) {
    count[i] = 0;
    if (biased) bias_at[i] = 0;
  }
  for (int i = threadIdx.x; i < slice / 32 + 1; i += kThreads) touched[i] = 0;
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
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int t = tok[i], e = t - v0;
      if (t < 0 || t >= a.vocab) {
        flag(a.status, DFLASH2_DEV_BAD_TOKEN);
      } else if (e >= 0 && e < nv) {
        atomicOr(count + e, kSeen);
        if (i >= prompt) atomicAdd(count + e, 1u);
        atomicOr(touched + (e >> 5), 1u << (e & 31));
      }
    }
    if (a.path && threadIdx.x < a.rows - 1) {
      const int t = a.path[(size_t)s * (a.rows - 1) + threadIdx.x], e = t - v0;
      path[threadIdx.x] = t;
      if (t < -1 || t >= a.vocab) flag(a.status, DFLASH2_DEV_BAD_TOKEN);
      else if (t >= 0 && e >= 0 && e < nv) atomicOr(touched + (e >> 5), 1u << (e & 31));
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
        atomicOr(touched + (e >> 5), 1u << (e & 31));
      }
    }
  }
  __syncthreads();
  const float* bias_row = biased ? a.bias + (size_t)s * a.n_bias : nullptr;
  const int words = (a.vocab + 31) / 32;
  for (int i = 0; i < a.rows; ++i) {
    const size_t row = (size_t)s * a.rows + i;
    const T* in = static_cast<const T*>(a.logits) + row * (size_t)a.stride + v0;
    T* out = static_cast<T*>(a.out) + row * (size_t)a.out_stride + v0;
    const uint32_t* mask = a.mask ? a.mask + row * (size_t)words : nullptr;
    const int drafts = penal && a.path ? i : 0;
    auto one = [&](int e, float z, uint32_t keep) {
      if ((touched[e >> 5] >> (e & 31)) & 1)
        z = changed(a, w, z, v0 + e, count[e], biased ? bias_at[e] : 0, path, drafts, bias_row);
      return keep ? z : -INFINITY;
    };
    // 16-byte accesses where the two rows are equally far from their border
    const int skew = (int)((uintptr_t)in % 16 / sizeof(T));
    const bool even = (uintptr_t)in % 16 == (uintptr_t)out % 16;
    const int head = even ? min(nv, (E - skew) % E) : nv;
    const int body = (nv - head) / E;
    for (int e = threadIdx.x; e < head + (nv - head - body * E); e += kThreads) {
      const int x = e < head ? e : e + body * E;
      const uint32_t keep = mask ? (mask[(v0 + x) >> 5] >> ((v0 + x) & 31)) & 1u : 1u;
      st(out + x, one(x, ld(in + x), keep));
    }
    for (int b = threadIdx.x; b < body; b += kThreads) {
      const int e = head + b * E;
      uint4 raw = *reinterpret_cast<const uint4*>(in + e);
      T* z = reinterpret_cast<T*>(&raw);
      uint32_t keep = 0xffffffffu;
      if (mask) {
        const int at = (v0 + e) >> 5, last = (v0 + e + E - 1) >> 5;
        keep = __funnelshift_r(mask[at], mask[last], (v0 + e) & 31);
      }
      const int at = e >> 5;
      const uint32_t any = __funnelshift_r(touched[at], touched[at + 1], e & 31) & ((1u << E) - 1u);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        if ((any >> k) & 1) st(z + k, one(e + k, ld(z + k), 1u));
        if (!((keep >> k) & 1)) st(z + k, -INFINITY);
      }
      *reinterpret_cast<uint4*>(out + e) = raw;
    }
  }
}

}  // namespace

int launch_adjust(const AdjustArgs& a, const Ctx& c) {
  const long long all = (long long)a.vocab * a.batch;
  const int per = (int)std::min<long long>(kMaxSlice, std::max<long long>(256, all / (4 * c.nsm)));
  const int slice = (per + 63) / 64 * 64;
  const size_t smem = (size_t)slice * 4 + (slice / 32 + 1) * 4 + (a.n_bias > 0 ? (size_t)slice * 2 : 0);
  const dim3 grid((a.vocab + slice - 1) / slice, a.batch);
  return a.bf16_logits ? launch_k(adjust_kernel<bf16>, grid, dim3(kThreads), smem, c, a, slice)
                       : launch_k(adjust_kernel<float>, grid, dim3(kThreads), smem, c, a, slice);
}

}  // namespace df2
