// Product with 4-bit weights and group scales:
//
//   y[n][m] = sum_g scale[m][g] * sum_{k in group g} (q[m][k] - 8) x[n][k]
//
// q are nibbles (byte j of a row holds elements 2j and 2j + 1), scale and x
// bf16, sums fp32, y fp32 or bf16 (rounded once).
//
// One warp per weight row and up to NB activation rows; the lanes stride over
// the row's 16-byte pieces (32 weights, which lie in one group since a group
// is a multiple of 32), and a butterfly joins the 32 partial sums.
#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

constexpr int W4_WARPS = 8, NB = 4;

template <typename OutT>
__global__ void __launch_bounds__(W4_WARPS * 32)
    linear_w4_kernel(const uint8_t* __restrict__ codes, const bf16* __restrict__ scale, int lg_group, int M, int K,
                     const bf16* __restrict__ x, long long ldx, int N, OutT* __restrict__ out, long long ldo,
                     int accumulate) {
  pdl_launch_next();
  pdl_wait();
  const int m = blockIdx.x * W4_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int n0 = blockIdx.y * NB;
  if (m >= M) return;
  const uint4* row = reinterpret_cast<const uint4*>(codes + (size_t)m * (K / 2));
  const bf16* srow = scale + (size_t)m * (K >> lg_group);
  float acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = 0.f;
  for (int p = lane; p < K / 32; p += 32) {
    const uint4 q4 = __ldg(row + p);
    const uint32_t w[4] = {q4.x, q4.y, q4.z, q4.w};
    const float s = __bfloat162float(srow[(p * 32) >> lg_group]);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if (n0 + j >= N) break;
      const bf16* xr = x + (size_t)(n0 + j) * ldx + p * 32;
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        t = fmaf((float)((int)((w[i >> 3] >> (4 * (i & 7))) & 15u) - 8), __bfloat162float(xr[i]), t);
      acc[j] = fmaf(s, t, acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const float v = warp_sum(acc[j]);
    if (lane == 0 && n0 + j < N) {
      OutT* o = out + (size_t)(n0 + j) * ldo + m;
      st(o, accumulate ? ld(o) + v : v);
    }
  }
}

}  // namespace

int launch_linear_w4(const W4Op& g, const Ctx& c) {
  int lg = 0;
  while ((1 << lg) < g.group) ++lg;
  const dim3 grid((g.M + W4_WARPS - 1) / W4_WARPS, (g.N + NB - 1) / NB);
  const uint8_t* codes = static_cast<const uint8_t*>(g.codes);
  const bf16* scale = static_cast<const bf16*>(g.scale);
  const bf16* x = static_cast<const bf16*>(g.x);
  if (g.out_bf16)
    return launch_k(linear_w4_kernel<bf16>, grid, dim3(W4_WARPS * 32), 0, c, codes, scale, lg, g.M, g.K, x, g.ldx, g.N,
                    static_cast<bf16*>(g.out), g.ldo, (int)g.accumulate);
  return launch_k(linear_w4_kernel<float>, grid, dim3(W4_WARPS * 32), 0, c, codes, scale, lg, g.M, g.K, x, g.ldx, g.N,
                  static_cast<float*>(g.out), g.ldo, (int)g.accumulate);
}

}  // namespace df2
