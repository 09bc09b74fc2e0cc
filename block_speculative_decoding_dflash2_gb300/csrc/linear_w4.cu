// Product with 4-bit weights and group scales:
//
//   y[n][m] = sum_g scale[m][g] * sum_{k in group g} (q[m][k] - 8) x[n][k]
//
// q are nibbles (byte j of a row holds elements 2j and 2j + 1), scale and x
// bf16, sums fp32, y fp32 or bf16 (rounded once).
//
// The weights are read once and decide the time while there are few
// activation rows, so they go from global memory straight into the registers
// of mma.sync.m16n8k16 as operand A: within a group the order of k is free as
// long as A and B agree, so each lane loads contiguous nibbles of its two rows
// (16, 8 or 4 bytes for groups of 128, 64 or 32: the four lanes of a row then
// always hold the same group) and the activations are stored in shared memory
// in the matching order, one 16-byte read per lane for two products.  A
// nibble becomes the bf16 value (q - 8) / 64 by a mask and a multiply-add (the
// 64 is put back at the end), so every product is exact; a group's fp32 sums are then scaled
// and added to the row's, which keeps the scale out of bf16.
//
// A CTA of 8 warps owns 128 weight rows at a time (16 a warp), or 256 where
// there are enough of them: two tiles of a warp share the activations' reads,
// which otherwise bound it (151936 x 4096 with groups of 64 and 8 rows: 76.9 us
// with 79% of the shared-memory cycles taken; 69.8 with two).  With few row blocks
// the inputs are split over a cluster of up to 8 CTAs, whose partial sums are
// added in rank order through distributed shared memory.
//
// What bounds it: 151936 x 4096 for one row takes 52 us with groups of 128 (6.2
// TB/s), where HBM needs 47; 68 and 109 with groups of 64 and 32, whose sums
// are scaled two and four times as often by the same 16 warps an SM (more do not
// fit beside the weights in flight); 54, 69 and 110 for 8 rows, 78, 98 and 138 for
// 16.  At 8 rows with groups of 64 shared memory and L1 are busy 75% of their
// cycles, DRAM 56%, and warps wait for loads most.  A small matrix takes its launch
// and two trips to memory: 704 x 256 for one row 2.7 us.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int WARPS = 8;
constexpr int CK = 128;                    // inputs of a chunk
constexpr int XS_MAX = 96 * 1024;          // activation bytes of a CTA (two CTAs share an SM)

struct Args {
  const uint8_t* codes;
  const bf16* scale;
  int M, K, chunks, slice;  // chunks of 128 inputs in all, and at most per CTA of a cluster
  int window;               // chunks whose activations are in shared memory at a time
  int blocks;               // row blocks
  int split;                // CTAs of a cluster
  const bf16* x;
  long long ldx;
  int N;  // up to 8 NT
  void* out;
  long long ldo;
  int accumulate;
};

// Nibbles e and e + 4 of a word (w8 = w >> 8) as bf16x2 (q - 8) / 64, exactly.
// A nibble's bits alone, at the bottom of a half or four above, are the values
// q 2^-133 and q 2^-129 (bf16 is linear up to 255 2^-133), so nothing is shifted
// but the word, once.
constexpr float UNSCALE = 64.f;
__device__ __forceinline__ uint32_t nib2(uint32_t w, uint32_t w8, int e) {
  const uint32_t r = (e < 2 ? w : w8) & (e & 1 ? 0x00f000f0u : 0x000f000fu);
  const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&r),
                                   __float2bfloat162_rn(e & 1 ? 0x1p+123f : 0x1p+127f), __float2bfloat162_rn(-0.125f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldw128(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldw64(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// First input of word i (8 nibbles) of lane-in-row t within a chunk.
template <int G>
__device__ __forceinline__ int word_k(int i, int t) {
  return G == 128 ? t * 32 + i * 8 : G == 64 ? (i >> 1) * 64 + t * 16 + (i & 1) * 8 : i * 32 + t * 8;
}

constexpr int U = 4;  // chunks whose scales are loaded together

// One lane's share of a chunk: 32 nibbles of two rows of each tile.
template <int R>
struct Chunk {
  uint32_t w[R][4];
};

// The group scales of four chunks of two rows: lane t of a row's four holds
// chunk t's (a request of 2-byte loads costs as much as one of 16-byte loads,
// so four chunks share it; the products fetch them by shuffles).
template <int G, int R>
struct Scales {
  float s[R][CK / G];
};
template <int G, int R>
__device__ __forceinline__ void load_scales(Scales<G, R>& c, const bf16* const (&srow)[R], int chunk, int K, int t) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < CK / G; ++i) {
      const int k = (chunk + t) * CK + i * G;
      c.s[r][i] = k < K ? __bfloat162float(srow[r][k / G]) : 0.f;
    }
}

template <int G, int R>
__device__ __forceinline__ void load_chunk(Chunk<R>& c, const uint8_t* const (&row)[R], int chunk, int K, int t) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint8_t* p = row[r] + (size_t)chunk * (CK / 2);
    if constexpr (G == 128) {
      const uint4 v = ldw128(p + t * 16);
      c.w[r][0] = v.x, c.w[r][1] = v.y, c.w[r][2] = v.z, c.w[r][3] = v.w;
    } else if constexpr (G == 64) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 v = make_uint2(0x88888888u, 0x88888888u);  // weight 0 past the row's end
        if (chunk * CK + h * 64 < K) v = ldw64(p + h * 32 + t * 8);
        c.w[r][2 * h] = v.x, c.w[r][2 * h + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c.w[r][i] = chunk * CK + i * 32 < K ? __ldg(reinterpret_cast<const uint32_t*>(p + i * 16 + t * 4)) : 0x88888888u;
    }
  }
}

template <int G, int NT, int MT, typename OutT>
__global__ void __launch_bounds__(WARPS * 32, 2) linear_w4_kernel(Args a) {
  constexpr int RB = WARPS * MT * 16;  // weight rows of a block
  constexpr int D = 4 / MT;            // chunks of weights in flight per warp
  extern __shared__ uint4 xs[];  // [window][4 words][NT][32 lanes], then the partial sums [NT * 8][RB]
  float* part = reinterpret_cast<float*>(xs + (size_t)a.window * 4 * NT * 32);
  pdl_launch_next();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % a.split;
  const int c_begin = min(a.chunks, rank * a.slice), c_end = min(a.chunks, c_begin + a.slice);
  const bool once = c_end - c_begin <= a.window;  // the activations stay for every row block

  // activations of chunks [c0, c1) in the order of the products
  auto stage = [&](int c0, int c1) {
    for (int i = threadIdx.x; i < (c1 - c0) * (NT * 8) * 16; i += WARPS * 32) {
      const int kb = i & 15, n = (i >> 4) % (NT * 8), c = (i >> 4) / (NT * 8);
      const int word = kb >> 2, tt = kb & 3;
      const int k = (c0 + c) * CK + word_k<G>(word, tt);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (n < a.N && k < a.K) v = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)n * a.ldx + k));
      const uint4 o = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                 __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
      xs[((c * 4 + word) * NT + (n >> 3)) * 32 + (n & 7) * 4 + tt] = o;
    }
  };
  if (once) {
    stage(c_begin, c_end);
    __syncthreads();
  }
  for (int blk = blockIdx.x / a.split; blk < a.blocks; blk += gridDim.x / a.split) {
    const int m0 = blk * RB + warp * (MT * 16) + g;
    const uint8_t* row[2 * MT];
    const bf16* srow[2 * MT];
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) {  // rows past the end read the last one and are not stored
      const size_t m = min(m0 + 8 * r, a.M - 1);
      row[r] = a.codes + m * (a.K / 2);
      srow[r] = a.scale + m * (a.K / G);
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int k = 0; k < MT; ++k)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][j][i] = 0.f;

    for (int w0 = c_begin; w0 < c_end; w0 += a.window) {
      const int w1 = min(c_end, w0 + a.window);
      if (!once) {
        __syncthreads();
        stage(w0, w1);
        __syncthreads();
      }
      Chunk<2 * MT> buf[D];
      Scales<G, 2 * MT> sc, sn;
      load_scales<G>(sn, srow, w0, a.K, t);
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (w0 + u < w1) load_chunk<G>(buf[u], row, w0 + u, a.K, t);
      for (int c0 = w0; c0 < w1; c0 += U) {
        sc = sn;
        if (c0 + U < w1) load_scales<G>(sn, srow, c0 + U, a.K, t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u;
          if (c >= w1) break;
          Chunk<2 * MT>& q = buf[u % D];
          float p[MT][NT][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i % (G / 32) == 0) {
#pragma unroll
              for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int e = 0; e < 4; ++e) p[k][j][e] = 0.f;
            }
            uint4 xv[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) xv[j] = xs[(((c - w0) * 4 + i) * NT + j) * 32 + lane];
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              const uint32_t wl = q.w[2 * k][i], wh = q.w[2 * k + 1][i];
              const uint32_t ul = wl >> 8, uh = wh >> 8;
              const uint32_t a0 = nib2(wl, ul, 0), a1 = nib2(wh, uh, 0), a2 = nib2(wl, ul, 1), a3 = nib2(wh, uh, 1);
              const uint32_t b0 = nib2(wl, ul, 2), b1 = nib2(wh, uh, 2), b2 = nib2(wl, ul, 3), b3 = nib2(wh, uh, 3);
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                mma16816(p[k][j], a0, a1, a2, a3, xv[j].x, xv[j].y);
                mma16816(p[k][j], b0, b1, b2, b3, xv[j].z, xv[j].w);
              }
            }
            if (i % (G / 32) == G / 32 - 1) {
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                const float s0 = __shfl_sync(0xffffffffu, sc.s[2 * k][i / (G / 32)], u, 4);
                const float s1 = __shfl_sync(0xffffffffu, sc.s[2 * k + 1][i / (G / 32)], u, 4);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  acc[k][j][0] = fmaf(s0, p[k][j][0], acc[k][j][0]);
                  acc[k][j][1] = fmaf(s0, p[k][j][1], acc[k][j][1]);
                  acc[k][j][2] = fmaf(s1, p[k][j][2], acc[k][j][2]);
                  acc[k][j][3] = fmaf(s1, p[k][j][3], acc[k][j][3]);
                }
              }
            }
          }
          if (c + D < w1) load_chunk<G>(q, row, c + D, a.K, t);
        }
      }
    }
    auto put = [&](int n, int m, float v) {
      if (n < a.N && m < a.M) {
        OutT* o = static_cast<OutT*>(a.out) + (size_t)n * a.ldo + m;
        st(o, a.accumulate ? fmaf(v, UNSCALE, ld(o)) : v * UNSCALE);
      }
    };
    if (a.split == 1) {
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) put(j * 8 + 2 * t + (e & 1), m0 + 16 * k + 8 * (e >> 1), acc[k][j][e]);
    } else {
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            part[(j * 8 + 2 * t + (e & 1)) * RB + warp * (MT * 16) + 16 * k + g + 8 * (e >> 1)] = acc[k][j][e];
      cluster_sync();
      // CTA `rank` adds a share of the block's sums, in rank order
      for (int i = rank * (WARPS * 32) + threadIdx.x; i < NT * 8 * RB / 4; i += a.split * WARPS * 32) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < a.split; ++r) {
          const float4 v = ld_dsmem4(dsmem_addr(part + i * 4, r));
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const int n = i * 4 / RB, m = blk * RB + i * 4 % RB;
        put(n, m, s.x), put(n, m + 1, s.y), put(n, m + 2, s.z), put(n, m + 3, s.w);
      }
      cluster_sync();  // every partial sum has been read
    }
  }
}

// Largest dynamic shared memory of an instantiation.
template <int NT, int MT>
constexpr int smem_most() {
  return XS_MAX + NT * 8 * (WARPS * MT * 16) * 4;
}

// Lets the kernel use that much on the current device, and counts the clusters
// of `split` CTAs that run at once on it (both once per device and size).
template <int G, int NT, int MT, typename OutT>
int wave_of(int split, int nsm) {
  static std::atomic<int> waves[64][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  int n = waves[dev][split].load(std::memory_order_relaxed);
  if (n) return n;
  auto kern = linear_w4_kernel<G, NT, MT, OutT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_most<NT, MT>()) != cudaSuccess)
    return -1;
  n = 2 * nsm;
  if (split > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split * 64);
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = smem_most<NT, MT>();
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = split;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      return -1;
    }
  }
  waves[dev][split].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs of a cluster: the most (up to 8) whose clusters hold every block in one
// wave with at least four chunks a CTA, but enough for the activations to fit.
// (Measured at 8 rows, groups of 128, us for splits of 1, 2, 4, 8: 6144 x 4096
// 13.3, 10.9, 7.6, 10.4 (48 blocks of 128 rows); 4096 x 12288 35, 34, 15, 10
// (32 blocks); 704 x 256 in 2 slices 3.1 against 2.2 in one.)
template <int G, int NT, int MT, typename OutT>
int split_of(int blocks, int chunks, int nsm) {
  constexpr int fit = XS_MAX / (NT * 8 * CK * 2);
  int split = std::min(8, (chunks + fit - 1) / fit);
  for (int s = std::min(8, chunks / 4); s > split; --s)
    if (wave_of<G, NT, MT, OutT>(s, nsm) >= blocks) return s;
  return split;
}

template <int G, int NT, int MT, typename OutT>
int launch(Args a, int split, const Ctx& c) {
  constexpr int RB = WARPS * MT * 16, per_chunk = NT * 8 * CK * 2, fit = XS_MAX / per_chunk;
  const int wave = wave_of<G, NT, MT, OutT>(split, c.nsm);
  if (wave < 1) return DFLASH2_ERR_CUDA;
  a.blocks = (a.M + RB - 1) / RB;
  a.split = split;
  a.slice = (a.chunks + a.split - 1) / a.split;
  a.window = std::min(a.slice, fit);
  const size_t smem = (size_t)a.window * per_chunk + (size_t)NT * 8 * RB * 4;
  const int clusters = std::min(wave, a.blocks);
  auto kern = linear_w4_kernel<G, NT, MT, OutT>;
  return launch_kx(kern, dim3(clusters * a.split), dim3(WARPS * 32), smem, c, a.split, a);
}

// Blocks of 256 rows unless blocks of 128 fill more of a wave; for more than 8
// activation rows, whose reads weigh more, also where those fill an SM each
// (16 rows, groups of 64, us with 256 and 128: 24576 x 4096 22.1, 28.7; 34816 x
// 5120 34.6, 37.7; but 12288 x 4096 16.0, 13.6).
template <int G, int NT, typename OutT>
int launch_m(const Args& a, const Ctx& c) {
  const int b2 = (a.M + 255) / 256, b1 = (a.M + 127) / 128, wave = 2 * c.nsm;
  const int s2 = split_of<G, NT, 2, OutT>(b2, a.chunks, c.nsm), s1 = split_of<G, NT, 1, OutT>(b1, a.chunks, c.nsm);
  const bool two = (NT == 2 && b1 >= c.nsm) || std::min(b2 * s2, wave) >= std::min(b1 * s1, wave);
  return two ? launch<G, NT, 2, OutT>(a, s2, c) : launch<G, NT, 1, OutT>(a, s1, c);
}

template <int G, typename OutT>
int launch_n(const Args& a, const Ctx& c) {
  return a.N <= 8 ? launch_m<G, 1, OutT>(a, c) : launch_m<G, 2, OutT>(a, c);
}

template <typename OutT>
int launch_g(int group, const Args& a, const Ctx& c) {
  return group == 32 ? launch_n<32, OutT>(a, c) : group == 64 ? launch_n<64, OutT>(a, c) : launch_n<128, OutT>(a, c);
}

}  // namespace

int launch_linear_w4(const W4Op& g, const Ctx& c) {
  // (entry points refuse these before their first launch)
  if ((uintptr_t)g.codes % 16 || (uintptr_t)g.x % 16 || (uintptr_t)g.scale % 2 || (g.N > 1 && g.ldx % 8) ||
      (uintptr_t)g.out % (g.out_bf16 ? 2 : 4))
    return DFLASH2_ERR_INVALID_ARG;
  const int most = 1 << 20;  // rows of a launch (its tiles are counted in ints)
  for (long long n = 0; n < g.N; n += most) {
    W4Op p = g;
    p.x = static_cast<const bf16*>(g.x) + n * g.ldx;
    p.N = (int)std::min<long long>(most, g.N - n);
    p.out = static_cast<char*>(g.out) + n * g.ldo * (g.out_bf16 ? 2 : 4);
    if (p.N > 16) {
      const int rc = launch_linear_w4_tc(p, c);
      if (rc != DFLASH2_OK) return rc;
      continue;
    }
    Args a = {};
    a.codes = static_cast<const uint8_t*>(p.codes);
    a.scale = static_cast<const bf16*>(p.scale);
    a.M = p.M;
    a.K = p.K;
    a.chunks = (p.K + CK - 1) / CK;
    a.x = static_cast<const bf16*>(p.x);
    a.ldx = p.ldx;
    a.N = p.N;
    a.out = p.out;
    a.ldo = p.ldo;
    a.accumulate = p.accumulate;
    const int rc = p.out_bf16 ? launch_g<bf16>(p.group, a, c) : launch_g<float>(p.group, a, c);
    if (rc != DFLASH2_OK) return rc;
  }
  return DFLASH2_OK;
}

}  // namespace df2
