// Product with 4-bit weights for many activation rows, on the 5th-generation
// tensor cores (the definition, and the kernel for few rows, are in
// linear_w4.cu).
//
// A 128-row weight tile is operand A of tcgen05.mma, held in TMEM, BN
// activation rows are operand B in shared memory, and every group of inputs is
// summed on its own: (q - 8) / 64 is exact in bf16, a group's fp32 sums lie in
// one of two to eight TMEM accumulators, and the epilogue warps read them,
// multiply them by the row's group scale and add them to the row's sums in
// registers while the tensor core fills the others.  (Scaled weights would need
// 11 bits, three more than bf16 has.)
//
// Warp roles (one CTA an SM):
//   warp 0       TMA producer of codes (one lane)
//   warp 1       MMA issuer (one lane) of even groups, and TMEM owner
//   then         epilogue: a set of four warps for every 32 columns
//   then 8       converters, in two groups of four on alternate chunks:
//                thread = weight row, its 64 bytes of codes -> 128 bf16 values
//                in 64 columns of its TMEM lane
//   last 2       MMA issuer of odd groups; TMA producer of activations
// Two issuers because a group's fences, waits and commits take one longer than
// its products (24576 x 4096 x 1024, with the activations' own producer: 187 us
// against 202).
// Operand A in TMEM because shared memory bounds the alternative: reading both
// operands of a 128 x 128 product takes all of its 128 bytes a cycle, and
// writing the converted tile as much again as a copy of the activations.
// With few tiles the inputs are split over a cluster, whose partial tiles are
// added in rank order through distributed shared memory.
//
// What it takes: 24576 x 4096 for 1024 rows 180 us (1.15 PFLOP/s), 5120 x 17408
// for 128 rows 27, the readout of 151936 x 4096 for 32, 64 and 128 rows 83, 103 and
// 136; groups of 64 and 32 double and quadruple the sums to scale (205 us at 128
// rows of that readout with 64).  What bounds it is known in part: it is not the
// products, the TMEM reads or the activations' copies (timed copies of the kernel
// with an eighth of the first, without the second or the third took 0 to 2% less),
// and the conversion's arithmetic is 15%.  At 5120 x 17408 x 128 a CTA issues 122k
// warp instructions, of which conversion (11 for 8 weights) and scaling (one for two
// sums) are 44k; the rest are its roles' loads, stores, polls and barriers.  That
// shape fills 120 of 152 SMs (40 tiles in clusters of 3).
//
// Every wait is bounded (1 s).  A wait that gives up records
// DFLASH2_DEV_WAIT_TIMEOUT (where the call has a status word) and lets the other
// roles bail out, the tile's outputs become NaN, and the kernel waits (bounded)
// for its own copies and products, frees TMEM and returns.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int BM = 128, BK = 128;  // weight rows of a tile, inputs of a chunk
constexpr int CONV_GROUPS = 2, CONV_GROUP = 128;
constexpr int CONV_THREADS = CONV_GROUPS * CONV_GROUP;
constexpr int SMEM_BUDGET = 227 * 1024 - 2048;  // 1 KB of alignment, 1 KB of barriers
constexpr uint64_t WAIT_NS = 1000000000ull;

constexpr int QC = 2;            // chunks of a block of codes (128 bytes of a row)
constexpr int A_COLS = BK / 2;   // TMEM columns of a chunk's operand A
constexpr uint32_t TMEM_COLS = 512;

// Rings: blocks of codes, which set how many bytes are on their way, and the
// operands of single chunks (A in TMEM, B in shared memory).
template <int BN>
struct Cfg {
  static constexpr int Q_BYTES = BM * BK / 2 * QC, B_BYTES = BN * BK * 2;
  static constexpr int S = 4, SB = BN == 128 ? 4 : 8, QS = 6;
  static constexpr int ACC = 256 / BN;           // accumulators
  static constexpr int COLS = 32;                // columns of an epilogue thread
  static constexpr int EPI_THREADS = BN / COLS * 128, THREADS = 128 + EPI_THREADS + CONV_THREADS;
  static constexpr int SMEM = QS * Q_BYTES + SB * B_BYTES + 2048;
  static_assert(SMEM <= SMEM_BUDGET + 2048, "shared memory");
  static_assert(S % 2 == 0 && SB % 2 == 0 && ACC % 2 == 0, "half of each to either parity");
  static_assert(ACC * BN + S * A_COLS <= (int)TMEM_COLS, "TMEM");
  static_assert(SB * B_BYTES >= BM * BN * 4, "the ring holds a partial tile");
};

struct Args {
  const bf16* scale;
  int M, K, N;
  int chunks, tiles, n_tiles, split, slice;  // chunks of 128 inputs; per CTA of a cluster (a multiple of QC)
  void* out;
  long long ldo;
  int accumulate;
  unsigned* status;   // or null
  uint64_t limit_ns;  // of a wait
  int x_tiles;        // tiles whose activations are copied: all, or none (a test's)
};

std::atomic<bool> g_withhold{false};

// 32 lanes x W consecutive TMEM columns -> W registers per thread.
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[W]) {
  static_assert(W == 16 || W == 32, "columns");
  if constexpr (W == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
  }
  tmem_ld_wait();
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Bounded wait for the phase of the given parity, given up too when *abort
// (nullable) becomes non-zero.  The clock, whose reading takes longer than most
// waits, is looked at every 256 tries.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  const uint32_t b = smem_u32(bar);
  uint64_t t0 = 0;
  for (unsigned i = 0;; ++i) {
    if (mbar_try_wait(b, parity)) return true;
    if ((i & 255) != 255) continue;
    if (abort && *abort) return false;
    const uint64_t t = globaltimer();
    if (t0 == 0) t0 = t;
    else if (t - t0 > limit_ns) return false;
  }
}

// 8 nibbles, in order, as bf16 values (q - 8) / 64: a nibble's bits alone are
// the subnormal q 2^-133, and q 2^-133 2^127 - 1/8 is exact.  (A byte's sign,
// 0, is what PRMT puts above it.  As (128 + q) - 136 a pair takes half a PRMT
// more: 5120 x 17408 for 128 rows took 28.3 us, and takes 26.9.)
constexpr float UNSCALE = 64.f;
__device__ __forceinline__ uint4 nibbles8(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  const __nv_bfloat162 up = __float2bfloat162_rn(0x1p+127f), off = __float2bfloat162_rn(-0.125f);
  auto two = [&](uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(lo), "r"(hi), "r"(sel));
    const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&r), up, off);
    return *reinterpret_cast<const uint32_t*>(&d);
  };
  return make_uint4(two(0xc480), two(0xd591), two(0xe6a2), two(0xf7b3));
}

// (a, b) += s (x, y), one instruction for both.
__device__ __forceinline__ void fma2(float& a, float& b, uint32_t x, uint32_t y, float s) {
  asm("{\n\t.reg .b64 d, e, f;\n\t"
      "mov.b64 d, {%0, %1};\n\t"
      "mov.b64 e, {%2, %3};\n\t"
      "mov.b64 f, {%4, %4};\n\t"
      "fma.rn.f32x2 d, e, f, d;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(x), "r"(y), "f"(s));
}

// D[tmem] (+)= A[tmem] * B[smem]^T: A's rows are lanes, two bf16 of a row a column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int BN, int G, typename OutT>
__global__ void __launch_bounds__(Cfg<BN>::THREADS, 1)
    linear_w4_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmX, Args a) {
  using C = Cfg<BN>;
  constexpr int S = C::S, SB = C::SB, QS = C::QS, ACC = C::ACC, EPI_THREADS = C::EPI_THREADS, THREADS = C::THREADS;
  constexpr int SP = S / 2, BP = SB / 2;  // of chunks of either parity
  constexpr int AP = ACC / 2;             // of either issuer
  constexpr bool EVERY = G < BK;          // both issuers work on every chunk
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stB = smem;
  uint8_t* stQ = stB + SB * C::B_BYTES;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(stQ + QS * C::Q_BYTES);  // a block of codes has landed
  uint64_t* q_empty = q_full + QS;
  uint64_t* full = q_empty + QS;  // a chunk's codes are converted
  uint64_t* empty = full + S;
  uint64_t* b_full = empty + S;  // a chunk's activations have landed
  uint64_t* b_empty = b_full + SB;
  uint64_t* acc_full = b_empty + SB;
  uint64_t* acc_empty = acc_full + ACC;
  uint64_t* drain = acc_empty + ACC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);  // then the abort flag, in one 8-byte word
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // (the shuffle tells the compiler that the warp index is uniform)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  pdl_launch_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < QS; ++s) {
      mbar_init(q_full + s, 1);
      mbar_init(q_empty + s, CONV_THREADS / 32);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, CONV_GROUP / 32);
      mbar_init(empty + s, EVERY ? 2 : 1);
    }
    for (int s = 0; s < SB; ++s) {
      mbar_init(b_full + s, 1);
      mbar_init(b_empty + s, EVERY ? 2 : 1);
    }
    for (int i = 0; i < ACC; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, EPI_THREADS / 32);
    }
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, tmem_a = tmem + ACC * BN;  // accumulators, then the A ring
  pdl_wait();

  auto fail = [&]() {
    *abort_flag = 1;
    flag(a.status, DFLASH2_DEV_WAIT_TIMEOUT);
  };

  const int rank = blockIdx.x % a.split, first = blockIdx.x / a.split, step = gridDim.x / a.split;
  const int c0 = min(a.chunks, rank * a.slice), c1 = min(a.chunks, c0 + a.slice);
  float* part = reinterpret_cast<float*>(smem);  // [BN][BM], in the idle ring

  const int nb = (c1 - c0 + QC - 1) / QC;  // blocks of codes of a tile
  // A group's products are the work of issuer 0 or 1 in turn: chunks alternate
  // where a chunk is one group, otherwise both issuers take their groups of
  // every chunk.  Each has accumulators of its own.  (On every barrier every
  // phase is waited for, by warps without which the next cannot complete: a
  // parity cannot tell two phases from none.)
  auto issue = [&](auto parity) {
    // The whole warp walks the chunks, so that descriptors stay in uniform
    // registers; one lane issues.
    constexpr int p = decltype(parity)::value;
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(BM, BN);
    int buf = p * AP;
    uint32_t acc_phase = 0, n[2] = {0, 0};  // n: chunks of either parity so far
    bool ok = true;
    auto products = [&](auto chunk_parity, uint32_t i) {
      constexpr int cp = decltype(chunk_parity)::value;
      const int stage = cp * SP + i % SP, slot = cp * BP + i % BP;
      const bool landed = wait_for(b_full + slot, i / BP & 1u, abort_flag, a.limit_ns);
      if (!__all_sync(0xffffffffu, landed && wait_for(full + stage, i / SP & 1u, abort_flag, a.limit_ns))) return false;
      tc_fence_after();
      const uint32_t at = tmem_a + (uint32_t)(stage * A_COLS);
      const uint64_t bd = sdesc_sw128(smem_u32(stB + slot * C::B_BYTES));
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk) {
        const bool begin = kk % (G / 16) == 0, end = kk % (G / 16) == G / 16 - 1;
        if (!EVERY || kk / (G / 16) % 2 == p) {
          if (begin) {
            if (!__all_sync(0xffffffffu, wait_for(acc_empty + buf, acc_phase ^ 1u, abort_flag, a.limit_ns))) return false;
            tc_fence_after();
          }
          if (leader)
            umma_bf16_ts(tmem + (uint32_t)(buf * BN), at + 8u * kk,
                         bd + (uint64_t)((kk >> 2) * (C::B_BYTES / 32) + 2 * (kk & 3)), idesc, begin ? 0u : 1u);
          if (end) {
            if (leader) umma_commit(acc_full + buf);
            if (++buf == (p + 1) * AP) {
              buf = p * AP;
              acc_phase ^= 1u;
            }
          }
        }
      }
      if (leader) {
        umma_commit(empty + stage);
        umma_commit(b_empty + slot);
      }
      return true;
    };
    for (int t = first; ok && t < a.tiles; t += step)
      for (int c = c0; ok && c < c1; c += 2) {
        if (EVERY || p == 0) ok = products(std::integral_constant<int, 0>(), n[0]++);
        if ((EVERY || p == 1) && c + 1 < c1) ok = ok && products(std::integral_constant<int, 1>(), n[1]++);
      }
    if (!ok) fail();
    if (leader) {
      umma_commit(drain);  // every product of this thread completes before TMEM can be freed
      if (!wait_for(drain, 0, nullptr, WAIT_NS)) fail();
    }
    __syncwarp();
  };
  if (warp == 0) {
    // codes (as the MMA warps: all lanes walk, one issues)
    const bool leader = elect_one();
    const uint64_t policy = policy_evict_first();
    int s = 0, issued = 0;  // issued: up to QS
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; ok && t < a.tiles; t += step)
      for (int b = 0; b < nb; ++b) {
        ok = __all_sync(0xffffffffu, wait_for(q_empty + s, phase ^ 1u, abort_flag, a.limit_ns));
        if (!ok) break;
        if (leader) {
          mbar_arrive_expect_tx(q_full + s, C::Q_BYTES);
          // (codes as pairs of bytes: 64 of them are 256 inputs)
          tma_load_2d(stQ + s * C::Q_BYTES, &tmQ, q_full + s, (c0 / QC + b) * (QC * BK / 4), t / a.n_tiles * BM, policy);
        }
        issued = min(issued + 1, QS);
        if (++s == QS) {
          s = 0;
          phase ^= 1u;
        }
      }
    if (!ok) fail();
    // every copy has landed before the CTA can end (consumers that gave up do not wait for theirs)
    for (; issued > 0; --issued) {
      if (s == 0) {
        s = QS;
        phase ^= 1u;
      }
      if (!wait_for(q_full + --s, phase, nullptr, WAIT_NS)) fail();
    }
    __syncwarp();
  } else if (warp == THREADS / 32 - 1) {
    // activations
    const bool leader = elect_one();
    const uint64_t policy = policy_evict_last();
    uint32_t j[2] = {0, 0};  // chunks of either parity so far
    bool ok = true;
    for (int t = first; ok && t < a.x_tiles; t += step) {
      const int nt = t % a.n_tiles;
      for (int b = 0; ok && b < nb; ++b) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int c = c0 + 2 * b + p, s = p * BP + j[p] % BP;
          if (!ok || c >= c1) break;
          ok = __all_sync(0xffffffffu, wait_for(b_empty + s, (j[p] / BP & 1u) ^ 1u, abort_flag, a.limit_ns));
          if (!ok) break;
          if (leader) {
            mbar_arrive_expect_tx(b_full + s, C::B_BYTES);
            // (two halves of 64 inputs, each in the 128-byte swizzle)
            tma_load_2d(stB + s * C::B_BYTES, &tmX, b_full + s, c * BK, nt * BN, policy);
            tma_load_2d(stB + s * C::B_BYTES + C::B_BYTES / 2, &tmX, b_full + s, c * BK + 64, nt * BN, policy);
          }
          ++j[p];
        }
      }
    }
    if (!ok) fail();
    for (int p = 0; p < 2; ++p)  // (as above)
      for (uint32_t i = j[p] - min(j[p], (uint32_t)BP); i != j[p]; ++i)
        if (!wait_for(b_full + p * BP + i % BP, i / BP & 1u, nullptr, WAIT_NS)) fail();
    __syncwarp();
  } else if (warp == 1) {
    issue(std::integral_constant<int, 0>());
  } else if (warp == THREADS / 32 - 2) {
    issue(std::integral_constant<int, 1>());
  } else if (warp >= 2 + EPI_THREADS / 32) {
    // converters: group cg takes chunk cg of every block; the codes lie in the
    // 128-byte swizzle (piece i of row r at i ^ (r & 7))
    const int cw = warp - 2 - EPI_THREADS / 32, cg = cw / 4, q = warp & 3, r = q * 32 + lane;
    int qs = 0;
    uint32_t q_phase = 0, j = 0;  // j: chunks of this group so far
    bool ok = true;
    for (int t = first; ok && t < a.tiles; t += step) {
      for (int b = 0; ok && b < nb; ++b) {
        bool got = wait_for(q_full + qs, q_phase, abort_flag, a.limit_ns);
        uint4 codes[4];
        if (got) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
            codes[h] = *reinterpret_cast<const uint4*>(stQ + qs * C::Q_BYTES + r * 128 + (((cg * 4 + h) ^ (r & 7)) << 4));
        }
        __syncwarp();
        if (got && lane == 0) mbar_arrive(q_empty + qs);
        if (b * QC + cg < c1 - c0) {
          // The slot is free when the products of this group's chunk j - SP are
          // done.  (Every phase of a barrier is waited for in turn: a parity
          // could not tell two phases from none.)
          const int stage = cg * SP + j % SP;
          static_assert(CONV_GROUPS == QC && QC == 2, "a group per chunk of a block");
          got = got && wait_for(empty + stage, (j / SP & 1u) ^ 1u, abort_flag, a.limit_ns);
          ++j;
          if (!__all_sync(0xffffffffu, got)) {  // TMEM stores are warp-wide
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dst = tmem_a + ((uint32_t)(q * 32) << 16) + (uint32_t)(stage * A_COLS);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t w[4] = {codes[h].x, codes[h].y, codes[h].z, codes[h].w};
            uint32_t v[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 x = nibbles8(w[j]);
              v[4 * j] = x.x, v[4 * j + 1] = x.y, v[4 * j + 2] = x.z, v[4 * j + 3] = x.w;
            }
            tmem_st16(dst + h * 16, v);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + stage);
        }
        ok = __all_sync(0xffffffffu, got);
        if (++qs == QS) {
          qs = 0;
          q_phase ^= 1u;
        }
      }
    }
    if (!ok) fail();
  } else {
    // epilogue
    constexpr int COLS = C::COLS;
    const int q = warp & 3, row = q * 32 + lane, set = (warp - 2) >> 2;
    const int g0 = c0 * BK / G, g1 = (c1 * BK + G - 1) / G, groups = a.K / G;
    uint32_t k0 = 0, k1 = 0;  // groups of either issuer so far
    bool ok = true;
    for (int t = first; t < a.tiles; t += step) {
      const int nt = t % a.n_tiles, mt = t / a.n_tiles, m = mt * BM + row;
      const bf16* srow = a.scale + (size_t)min(m, a.M - 1) * groups;
      float acc[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
      bf16 s_next = g0 < min(g1, groups) ? srow[g0] : __float2bfloat16(0.f);
      for (int g = g0; ok && g < g1; ++g) {
        const float s = __bfloat162float(s_next);  // (here, not behind its load: it has landed)
        s_next = g + 1 < min(g1, groups) ? srow[g + 1] : __float2bfloat16(0.f);
        const bool odd = (g - g0) & 1;
        const uint32_t k = odd ? k1++ : k0++, buf = (odd ? AP : 0) + k % AP;
        // (the whole warp goes on or gives up: TMEM reads are warp-wide)
        const bool got = wait_for(acc_full + buf, k / AP & 1u, abort_flag, a.limit_ns);
        if (!__all_sync(0xffffffffu, got)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN + set * COLS);
        constexpr int W = BN == 128 ? 16 : 32;  // columns of a TMEM read (with 896 threads, 72 registers each)
#pragma unroll
        for (int j0 = 0; j0 < COLS; j0 += W) {
          uint32_t v[W];
          tmem_ld<W>(d + j0, v);
          if (j0 + W == COLS) {  // the last read: the accumulator is free before its values are used
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + buf);
          }
#pragma unroll
          for (int j = 0; j < W; j += 2) fma2(acc[j0 + j], acc[j0 + j + 1], v[j], v[j + 1], s);
        }
      }
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = ok ? acc[j] * UNSCALE : __int_as_float(0x7fffffff);
      if (a.split == 1) {
        if (m < a.M) {
#pragma unroll
          for (int j = 0; j < COLS; ++j) {
            const int n = nt * BN + set * COLS + j;
            if (n < a.N) {
              OutT* o = static_cast<OutT*>(a.out) + (size_t)n * a.ldo + m;
              st(o, a.accumulate ? ld(o) + acc[j] : acc[j]);
            }
          }
        }
      } else {  // (one tile: every copy and product of it is done)
#pragma unroll
        for (int j = 0; j < COLS; ++j) part[(set * COLS + j) * BM + row] = acc[j];
      }
    }
  }
  if (a.split > 1) {
    cluster_sync();
    const int nt = first % a.n_tiles, mt = first / a.n_tiles;
    bool bad = false;  // a CTA of the cluster gave up
    for (int r = 0; r < a.split; ++r) bad = bad || __float_as_int(ld_dsmem2(dsmem_addr(tmem_slot, r)).y) != 0;
    for (int i = rank * THREADS + threadIdx.x; i < BN * BM / 4; i += a.split * THREADS) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r = 0; r < a.split; ++r) {
        const float4 v = ld_dsmem4(dsmem_addr(part + i * 4, r));
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      const float nan = __int_as_float(0x7fffffff);
      const float e[4] = {bad ? nan : s.x, bad ? nan : s.y, bad ? nan : s.z, bad ? nan : s.w};
      const int n = nt * BN + i * 4 / BM, m = mt * BM + i * 4 % BM;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n < a.N && m + j < a.M) {
          OutT* o = static_cast<OutT*>(a.out) + (size_t)n * a.ldo + m + j;
          st(o, a.accumulate ? ld(o) + e[j] : e[j]);
        }
    }
    cluster_sync();  // every partial tile has been read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

// Lets the kernel use its shared memory on the current device, and counts the
// clusters of `split` CTAs that run at once on it (both once per device and
// size).
template <int BN, int G, typename OutT>
int wave_of(int split, int nsm) {
  using C = Cfg<BN>;
  static std::atomic<int> waves[64][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  int n = waves[dev][split].load(std::memory_order_relaxed);
  if (n) return n;
  auto kern = linear_w4_tc_kernel<BN, G, OutT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return -1;
  n = nsm;
  if (split > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split * 64);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
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

template <int BN, int G, typename OutT>
int launch(const W4Op& g, const Ctx& c) {
  using C = Cfg<BN>;
  CUtensorMap mq, mx;
  int rc = make_sw128_map(&mq, g.codes, g.M, g.K / 4, g.K / 4, BM);
  if (rc) return rc;
  rc = make_sw128_map(&mx, g.x, g.N, g.K, g.ldx, BN);
  if (rc) return rc;
  Args a = {};
  a.scale = static_cast<const bf16*>(g.scale);
  a.M = g.M;
  a.K = g.K;
  a.N = g.N;
  a.chunks = (g.K + BK - 1) / BK;
  a.n_tiles = (g.N + BN - 1) / BN;
  a.tiles = (g.M + BM - 1) / BM * a.n_tiles;
  // Inputs split as far as all tiles' clusters run at once and a CTA has at
  // least 4 chunks.  (Clusters do not fill every group of SMs: 48 of 3 CTAs
  // need a second wave on 152 SMs, 6144 x 4096 x 17 took 16.6 us; 48 of 2, 9.9.)
  a.split = std::max(1, std::min({8, c.nsm / a.tiles, a.chunks / 4}));
  int wave;
  while ((wave = wave_of<BN, G, OutT>(a.split, c.nsm)) >= 0 && a.split > 1 && wave < a.tiles) --a.split;
  if (wave < 0) return DFLASH2_ERR_CUDA;
  a.slice = ((a.chunks + a.split - 1) / a.split + QC - 1) / QC * QC;
  a.out = g.out;
  a.ldo = g.ldo;
  a.accumulate = g.accumulate;
  a.status = c.status;
  const bool withhold = g_withhold.load(std::memory_order_relaxed);
  a.limit_ns = withhold ? 1000000 : WAIT_NS;
  a.x_tiles = withhold ? 0 : a.tiles;
  auto kern = linear_w4_tc_kernel<BN, G, OutT>;
  const int grid = a.split > 1 ? a.tiles * a.split : std::min(a.tiles, c.nsm);
  return launch_kx(kern, dim3(grid), dim3(C::THREADS), C::SMEM, c, a.split, mq, mx, a);
}

template <int G, typename OutT>
int launch_n(const W4Op& g, const Ctx& c) {
  if (g.N <= 32) return launch<32, G, OutT>(g, c);
  if (g.N <= 64) return launch<64, G, OutT>(g, c);
  return launch<128, G, OutT>(g, c);
}

template <typename OutT>
int launch_g(const W4Op& g, const Ctx& c) {
  return g.group == 32 ? launch_n<32, OutT>(g, c) : g.group == 64 ? launch_n<64, OutT>(g, c) : launch_n<128, OutT>(g, c);
}

}  // namespace

void linear_w4_withhold(bool on) { g_withhold.store(on); }

int launch_linear_w4_tc(const W4Op& g, const Ctx& c) {
  return g.out_bf16 ? launch_g<bf16>(g, c) : launch_g<float>(g, c);
}

}  // namespace df2
