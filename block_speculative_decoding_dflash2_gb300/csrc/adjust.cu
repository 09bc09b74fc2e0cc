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
// one.  The work is one pass over the rows: what bounds it is memory.
//
// A block takes a slice of the vocabulary of all rows of one sequence.  Bulk
// copies bring the rows' slices into shared memory while the block walks the
// sequence's tokens, counts those of its slice in a table and lists them; the
// few listed tokens are then changed in place, the mask goes over the rest,
// and bulk copies take the slices out.  So the copies of some blocks run
// under the walks of others, and no token is read twice.  256 rows of 151936
// bfloat16 with 4000 tokens behind each sequence take 60 us (2.7 TB/s): 42 for
// the copies and the mask, 5 for the walks, 13 for the listed tokens, most of
// which lie in a few slices.  (Streamed through registers, the listed tokens
// changed in memory afterwards: 66.)
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 5952;        // tokens of a slice at most: 48 KB of tables
constexpr int kRows = 8;               // rows in shared memory at a time
constexpr int kRowBytes = 48 * 1024;   // their bytes at most
constexpr int kMaxDrafts = 31;
constexpr int kAhead = 8;              // tokens of the history that a thread has in flight
constexpr uint32_t kSeen = 0x80000000u;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kStaticBytes = 1024;     // more than the kernel's static shared memory (path, barrier, counters)

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

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Bytes of a row's slice that a bulk copy takes: whole 16 bytes from a
// 16-byte border, none where the row does not start on one.
__device__ __forceinline__ uint32_t bulk_bytes(const void* row, uint32_t bytes) {
  return (uintptr_t)row % 16 ? 0u : bytes & ~15u;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) adjust_kernel(const __grid_constant__ AdjustArgs a, int slice) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t sh[];
  const int group = min(kRows, a.rows);
  T* box = reinterpret_cast<T*>(sh);                                                  // [group][slice]
  uint32_t* count = reinterpret_cast<uint32_t*>(sh + (size_t)group * slice * sizeof(T));  // [slice] kSeen | count
  uint32_t* touched = count + slice;                                                  // [slice / 32] bits
  uint32_t* keep_at = touched + slice / 32;                                           // [group][slice / 32] mask words
  uint16_t* list = reinterpret_cast<uint16_t*>(keep_at + (a.mask ? group * (slice / 32) : 0));  // [slice] the entries with a bit
  uint16_t* bias_at = list + slice;                                                   // [slice] last entry of the token + 1
  __shared__ int32_t path[kMaxDrafts + 1];
  __shared__ int listed;
  __shared__ uint64_t bar;
  __shared__ int never;
  pdl_launch_next();
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_barrier_init();
    listed = 0;
    never = 0;
  }
  pdl_wait();
  const int s = blockIdx.y, v0 = blockIdx.x * slice, nv = min(slice, a.vocab - v0);
  const uint32_t bytes = (uint32_t)(nv * sizeof(T));
  const int words = (a.vocab + 31) / 32;
  // rows [i0, i0 + n) into the box: the bulk copies by one thread, what they leave by all
  auto fetch = [&](int i0, int n) {
    const T* in = static_cast<const T*>(a.logits) + ((size_t)s * a.rows + i0) * (size_t)a.stride + v0;
    if (threadIdx.x == 0) {
      uint32_t sum = 0;
      for (int i = 0; i < n; ++i) sum += bulk_bytes(in + i * (size_t)a.stride, bytes);
      mbar_arrive_expect_tx(&bar, sum);
      for (int i = 0; i < n; ++i) {
        const uint32_t b = bulk_bytes(in + i * (size_t)a.stride, bytes);
        if (b) bulk_g2s(box + i * slice, in + i * (size_t)a.stride, b, &bar);
      }
    }
    for (int i = 0; i < n; ++i) {
      const int from = (int)(bulk_bytes(in + i * (size_t)a.stride, bytes) / sizeof(T));
      for (int e = from + threadIdx.x; e < nv; e += kThreads) box[i * slice + e] = in[i * (size_t)a.stride + e];
    }
    if (a.mask) {
      const uint32_t* m = a.mask + ((size_t)s * a.rows + i0) * (size_t)words + v0 / 32;
      const int per = slice / 32, there = (nv + 31) / 32;
#pragma unroll 4
      for (int x = threadIdx.x; x < n * per; x += kThreads) {
        const int i = x / per, y = x - i * per;
        if (y < there) keep_at[x] = m[i * (size_t)words + y];
      }
    }
  };
  const bool biased = a.n_bias > 0;
  const float rho = a.repetition ? a.repetition[s] : 1.f, presence = a.presence ? a.presence[s] : 0.f,
              frequency = a.frequency ? a.frequency[s] : 0.f;
  const bool penal = rho != 1.f || presence != 0.f || frequency != 0.f;
  int n = a.n_tokens ? a.n_tokens[s] : 0;
  const int prompt = a.prompt_len ? a.prompt_len[s] : 0;
  __syncthreads();  // the barrier is there
  fetch(0, min(group, a.rows));
  for (int i = threadIdx.x; i < slice; i += kThreads) {
    count[i] = 0;
    if (biased) bias_at[i] = 0;
  }
  for (int i = threadIdx.x; i < slice / 32; i += kThreads) touched[i] = 0;
  auto touch = [&](int e) {
    const uint32_t bit = 1u << (e & 31);
    if (!(atomicOr(touched + (e >> 5), bit) & bit)) list[atomicAdd(&listed, 1)] = (uint16_t)e;
  };
  __syncthreads();
  if (n < 0 || n > a.max_tokens) {
    if (threadIdx.x == 0) flag(a.status, DFLASH2_DEV_BAD_LENGTH);
    n = n < 0 ? 0 : a.max_tokens;
  }
  const int32_t* tok = a.tokens + (size_t)s * a.max_tokens;
  if (!penal) {
    // nothing to count: the sequence's blocks share its ids, and only look whether they are any
    if (a.status)
      for (unsigned i = blockIdx.x * kThreads + threadIdx.x; i < (unsigned)n; i += gridDim.x * kThreads)
        if ((unsigned)tok[i] >= (unsigned)a.vocab) flag(a.status, DFLASH2_DEV_BAD_TOKEN);
  } else {
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
  }
  if (a.path && (int)threadIdx.x < a.rows - 1) {
    const int t = a.path[(size_t)s * (a.rows - 1) + threadIdx.x], e = t - v0;
    path[threadIdx.x] = t;
    if (t < -1 || t >= a.vocab) flag(a.status, DFLASH2_DEV_BAD_TOKEN);
    else if (penal && t >= 0 && e >= 0 && e < nv) touch(e);
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
  const bool drafts = penal && a.path;
  for (int i0 = 0, round = 0; i0 < a.rows; i0 += group, ++round) {
    const int rows = min(group, a.rows - i0);
    if (!mbar_wait(&bar, round & 1, &never, kWaitNs) && threadIdx.x == 0) flag(a.status, DFLASH2_DEV_WAIT_TIMEOUT);
    __syncthreads();  // the plain loads, the tables and the list
    for (int k = threadIdx.x; k < listed; k += kThreads) {
      const int e = list[k];
      uint32_t c = count[e];
      const int at = biased ? bias_at[e] : 0;
      const float bias = at > 0 ? a.bias[(size_t)s * a.n_bias + at - 1] : 0.f;
      if (drafts)  // those before the first row; each row then adds the draft before it
        for (int j = 0; j < i0 - 1; ++j)
          if (path[j] == v0 + e) c = (c + 1) | kSeen;
#pragma unroll 4
      for (int i = 0; i < rows; ++i) {
        if (drafts && i0 + i > 0 && path[i0 + i - 1] == v0 + e) c = (c + 1) | kSeen;
        float z = ld(box + i * slice + e);
        if (c & kSeen) z = z > 0.f ? z / rho : z * rho;
        if (c & ~kSeen) z = (z - frequency * (float)(c & ~kSeen)) - presence;
        if (at > 0) z += bias;
        st(box + i * slice + e, z);
      }
    }
    __syncthreads();
    if (a.mask) {
      const int vecs = (nv + E - 1) / E;  // (the last one's tail lies in the box, and goes nowhere)
      for (int i = 0; i < rows; ++i) {
        const uint32_t* m = keep_at + i * (slice / 32);
        for (int b = threadIdx.x; b < vecs; b += kThreads) {  // (E divides 32: one word has the bits)
          const uint32_t keep = m[b * E >> 5] >> (b * E & 31);
          if ((keep & ((1u << E) - 1u)) != (1u << E) - 1u) {
            uint4* x = reinterpret_cast<uint4*>(box + i * slice) + b;
            uint4 y = *x;
            blank(y, keep, T());
            *x = y;
          }
        }
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    T* out = static_cast<T*>(a.out) + ((size_t)s * a.rows + i0) * (size_t)a.out_stride + v0;
    if (threadIdx.x == 0) {
      for (int i = 0; i < rows; ++i) {
        const uint32_t b = bulk_bytes(out + i * (size_t)a.out_stride, bytes);
        if (b) bulk_s2g(out + i * (size_t)a.out_stride, box + i * slice, b);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    for (int i = 0; i < rows; ++i) {
      const int from = (int)(bulk_bytes(out + i * (size_t)a.out_stride, bytes) / sizeof(T));
      for (int e = from + threadIdx.x; e < nv; e += kThreads) out[i * (size_t)a.out_stride + e] = box[i * slice + e];
    }
    // the box is read out before it is filled again, or the block ends
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    if (i0 + group < a.rows) {
      __syncthreads();
      fetch(i0 + group, min(group, a.rows - i0 - group));
    }
  }
}

}  // namespace

int launch_adjust(const AdjustArgs& a, const Ctx& c) {
  // Slices: 18 blocks an SM in all (several times what runs at once, so that
  // the slices where most of the text's tokens lie do not decide), but up to
  // three times larger where the walk through the history is more than half
  // of a block's bytes, as far as the rows fit shared memory.
  const int group = std::min(kRows, a.rows), size = a.bf16_logits ? 2 : 4;
  const long long fill = (long long)a.vocab * a.batch / (18 * c.nsm);
  const long long walk = a.n_tokens ? 4ll * a.max_tokens / (a.rows * size) : 0;
  const int per = (int)std::min<long long>({kMaxSlice, kRowBytes / (group * size),
                                            std::max<long long>({256, fill, std::min(walk, 3 * fill)})});
  const int slice = per / 64 * 64;
  const size_t smem = (size_t)slice * (group * size + 6) + slice / 8 + (a.mask ? (size_t)group * slice / 8 : 0) +
                      (a.n_bias > 0 ? (size_t)slice * 2 : 0);
  const dim3 grid((a.vocab + slice - 1) / slice, a.batch);
  // (an attribute of the kernel on the current device, so on every call that
  // needs it; without it 48 KB hold the kernel's static bytes as well)
  const void* kernel = a.bf16_logits ? (const void*)adjust_kernel<bf16> : (const void*)adjust_kernel<float>;
  if (smem + kStaticBytes > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024) != cudaSuccess)
    return DFLASH2_ERR_CUDA;
  return a.bf16_logits ? launch_k(adjust_kernel<bf16>, grid, dim3(kThreads), smem, c, a, slice)
                       : launch_k(adjust_kernel<float>, grid, dim3(kThreads), smem, c, a, slice);
}

}  // namespace df2
