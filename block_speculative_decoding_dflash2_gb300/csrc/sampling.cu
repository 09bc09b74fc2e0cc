// From a target's logits to tokens: temperature, top-k, top-p and min-p
// truncation, and on the truncated distribution the draw of a token, the
// distribution itself, or the verification of a draft ("Train a DFlash
// Drafter for Speculative Decoding": spec_generate's temperature, top_p and
// top_k truncate the TARGET's distribution, the one verification samples
// against).
//
// Definition, for a row z at temperature T > 0 with mass e_v =
// exp((z_v - max z) / T): order the tokens by (z descending, id ascending);
// keep the first top_k; of these the shortest prefix that holds top_p of
// their mass; of these the tokens with e_v >= min_p.  Every filter cuts the
// same order, so the kept tokens are a prefix of it, described by its last
// token (value, id).  T <= 0 keeps the first token alone.  Tokens at -inf or
// NaN have no mass and are never kept.
//
// Masses are whole numbers: e_v in units of 2^-42, from a two-float
// evaluation good to about 2^-37 of the mass.  Their 64-bit sums are exact
// and do not depend on the order of the additions, so draws and cuts are
// deterministic and sit within 2^-37 of the exact ones; in plain fp32 a cut
// or a draw next to a border falls on the wrong side about once in a
// thousand rows of a 150k vocabulary.
#include "common.cuh"
#include "internal.h"

namespace df2 {

namespace {

typedef unsigned long long u64;

constexpr int NT = 512, NW = NT / 32;
constexpr unsigned KEY_NINF = 0x007fffffu;  // order of -inf; NaN maps to 0

// Order-preserving map of a logit (a larger one has a larger key; -0 equals 0).
__device__ __forceinline__ unsigned okey(float z) {
  const unsigned u = __float_as_uint(z + 0.f);
  const unsigned k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return z != z ? 0u : k;
}
__device__ __forceinline__ float okey_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// 2^(-j/32) for j = -16..16, in units of 2^-42 and as a float pair (the
// table's values are those powers rounded from 50 decimal digits).
struct ExpTab {
  long long fix[33];
  float hi[33], lo[33];
};
__constant__ ExpTab c_exp = {
    {6219777023951ll, 6086500028053ll, 5956078883349ll, 5828452394836ll, 5703560678795ll,
     5581345134690ll, 5461748417677ll, 5344714411690ll, 5230188203118ll, 5118116055032ll,
     5008445381977ll, 4901124725294ll, 4796103728980ll, 4693333116055ll, 4592764665442ll,
     4494351189345ll, 4398046511104ll, 4303805443529ll, 4211583767698ll, 4121338212211ll,
     4033026432885ll, 3946606992882ll, 3862039343274ll, 3779283804012ll, 3698301545306ll,
     3619054569413ll, 3541505692798ll, 3465618528697ll, 3391357470036ll, 3318687672730ll,
     3247575039328ll, 3177986203020ll, 3109888511975ll},
    {0x1.6a09e60000000p+0f, 0x1.6247ec0000000p+0f, 0x1.5ab07e0000000p+0f, 0x1.5342b60000000p+0f, 0x1.4bfdae0000000p+0f, 0x1.44e0860000000p+0f,
     0x1.3dea640000000p+0f, 0x1.371a740000000p+0f, 0x1.306fe00000000p+0f, 0x1.29e9e00000000p+0f, 0x1.2387a60000000p+0f, 0x1.1d48740000000p+0f,
     0x1.172b840000000p+0f, 0x1.11301e0000000p+0f, 0x1.0b55860000000p+0f, 0x1.059b0e0000000p+0f, 0x1.0000000000000p+0f, 0x1.f507660000000p-1f,
     0x1.ea4afa0000000p-1f, 0x1.dfc9740000000p-1f, 0x1.d5818e0000000p-1f, 0x1.cb720e0000000p-1f, 0x1.c199be0000000p-1f, 0x1.b7f7700000000p-1f,
     0x1.ae89fa0000000p-1f, 0x1.a5503c0000000p-1f, 0x1.9c49180000000p-1f, 0x1.93737c0000000p-1f, 0x1.8ace540000000p-1f, 0x1.82589a0000000p-1f,
     0x1.7a11480000000p-1f, 0x1.71f75e0000000p-1f, 0x1.6a09e60000000p-1f},
    {0x1.9fcef40000000p-26f, -0x1.f8b5500000000p-25f, -0x1.5bd5ec0000000p-27f, -0x1.2c56100000000p-25f, -0x1.593abc0000000p-25f, 0x1.8624b40000000p-30f,
     0x1.8246840000000p-25f, -0x1.18aac60000000p-25f, 0x1.4636e20000000p-25f, -0x1.5c04240000000p-25f, 0x1.ceac480000000p-25f, -0x1.d2e8ca0000000p-25f,
     -0x1.c157420000000p-27f, -0x1.fdb4960000000p-25f, 0x1.9f31220000000p-25f, -0x1.9d4f520000000p-25f, 0x0.0p+0f, -0x1.246eb00000000p-27f,
     0x1.52486c0000000p-28f, -0x1.908c940000000p-26f, -0x1.822dbc0000000p-28f, -0x1.8837cc0000000p-28f, -0x1.3d56b20000000p-28f, -0x1.a094380000000p-26f,
     -0x1.a94b140000000p-27f, -0x1.b83b540000000p-26f, 0x1.51f8480000000p-28f, -0x1.e647440000000p-26f, 0x1.15506e0000000p-28f, -0x1.accc7c0000000p-27f,
     -0x1.829fd00000000p-26f, 0x1.1d8bee0000000p-26f, 0x1.9fcef40000000p-27f}};

// The row's exponent scale log2(e) / T as a float pair.
struct Scale {
  float zmax, hi, lo;
};
__device__ __forceinline__ Scale make_scale(float zmax, float T) {
  const double c = 1.4426950408889634074 / (double)T;
  Scale s;
  s.zmax = zmax;
  s.hi = (float)c;
  s.lo = (float)(c - (double)s.hi);
  return s;
}

// exp((z - zmax) / T) in units of 2^-42, for z > -inf.  With y = (zmax - z)
// log2(e) / T held as p + e (the difference exact by two-sum, the product by
// fma), y = n + j/32 + g + e, |g| <= 1/64, and 2^-(g+e) = 1 - (g + e) ln 2 +
// ..., whose linear term keeps its rounding error.
__device__ __forceinline__ u64 mass_of(float z, const Scale& s) {
  if (z == s.zmax || s.hi == 0.f) return 1ull << 42;
  const float dh = s.zmax - z;
  const float p = __fmul_rn(dh, s.hi);  // never contracted: its rounding error goes to e
  if (!(p < 44.f)) return 0ull;
  const float bb = dh - s.zmax;
  const float dl = (s.zmax - (dh - bb)) - (z + bb);
  float e = fmaf(dh, s.hi, -p);
  e = fmaf(dh, s.lo, e);
  e = fmaf(dl, s.hi, e);
  const float n = rintf(p), r = p - n;
  const float jf = rintf(r * 32.f), g = fmaf(jf, -0.03125f, r);
  const int j = (int)jf + 16;
  const float L1 = 0.693147182464599609f, L1lo = -1.90465429995776e-9f;  // ln 2
  const float gl = __fmul_rn(g, L1);
  const float glr = fmaf(g, L1lo, fmaf(e, L1, fmaf(g, L1, -gl)));
  const float x = (g + e) * L1;
  const float q = x * x * fmaf(x, fmaf(x, 0.0416666667f, -0.1666666667f), 0.5f) - glr;  // 2^-(g+e) - 1 + gl
  const float th = c_exp.hi[j], tl = c_exp.lo[j];
  const float m = __fmul_rn(th, gl);
  const float small = fmaf(th, q, -fmaf(th, gl, -m)) - tl * gl;
  const long long v = c_exp.fix[j] - ((long long)__float2int_rn(m * 68719476736.f) << 6) +
                      (long long)__float2int_rn(small * 4398046511104.f);
  const int sh = (int)n;  // 0..44
  return sh == 0 ? (u64)v : ((u64)v + (1ull << (sh - 1))) >> sh;
}

// The same to fp32 accuracy relative to the mass, however small.
__device__ __forceinline__ float mass_f32(float z, const Scale& s) {
  if (z == s.zmax || s.hi == 0.f) return 1.f;
  const float dh = s.zmax - z, p = __fmul_rn(dh, s.hi);
  if (!(p < 160.f)) return 0.f;
  const float bb = dh - s.zmax, dl = (s.zmax - (dh - bb)) - (z + bb);
  float e = fmaf(dh, s.hi, -p);
  e = fmaf(dh, s.lo, e);
  e = fmaf(dl, s.hi, e);
  const float f = exp2f(-p);
  return fmaf(f, -0.693147182f * e, f);
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Smem {
  unsigned cnt[256];
  u64 mass[256];
  u64 wsum[NW];
  float wmax[NW];
  unsigned sel_key;
  u64 sel_before;
  int pick;
};

__device__ __forceinline__ u64 block_sum_u64(u64 v, Smem& sm) {
  v = warp_sum_u64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.wsum[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = 0;
  for (int i = 0; i < NW; ++i) t += sm.wsum[i];
  return t;
}

// The kept prefix of a row's order: every token with (key, id) ahead of or
// equal to (key, id) here.
struct Cut {
  unsigned key;
  int id;
};
__device__ __forceinline__ bool kept(unsigned k, int id, const Cut& c) {
  return k > c.key || (k == c.key && id <= c.id);
}

// One step of a row's selection: among the tokens kept by `c`, the first one
// of the order whose running sum of weights (1 each when by_count, else the
// masses) reaches `target` (>= 1, at most the total).  Radix selection on the
// key, 8 bits a level, then on the ids of equal keys.
template <typename T>
__device__ Cut select_prefix(const T* row, int V, const Scale& s, Cut c, bool by_count, u64 target, Smem& sm) {
  unsigned prefix = 0, mask = 0;
  u64 before = 0;  // weight ahead of the keys that match the prefix
  for (int level = 3; level >= 0; --level) {
    for (int i = threadIdx.x; i < 256; i += NT) sm.mass[i] = 0;
    __syncthreads();
    for (int v = threadIdx.x; v < V; v += NT) {
      const float z = ld(row + v);
      const unsigned k = okey(z);
      if ((k & mask) == prefix && kept(k, v, c))
        atomicAdd(&sm.mass[(k >> (8 * level)) & 255u], by_count ? 1ull : mass_of(z, s));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      u64 b = before;
      int d = 255;
      while (d > 0 && b + sm.mass[d] < target) b += sm.mass[d--];
      sm.sel_key = prefix | ((unsigned)d << (8 * level));
      sm.sel_before = b;
    }
    __syncthreads();
    prefix = sm.sel_key;
    before = sm.sel_before;
    mask |= 255u << (8 * level);
    __syncthreads();
  }
  // equal keys: the need-th of them in id order (each has the same weight)
  const float zs = okey_value(prefix);
  const u64 w = by_count ? 1ull : mass_of(zs, s);
  u64 need = w ? (target - before + w - 1) / w : 1;
  if (need == 0) need = 1;
  const int per = (V + NT - 1) / NT;
  const int a = min(V, (int)threadIdx.x * per), b = min(V, a + per);
  unsigned mine = 0;
  for (int v = a; v < b; ++v) {
    const unsigned k = okey(ld(row + v));
    mine += k == prefix && kept(k, v, c);
  }
  unsigned inc = mine;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) sm.wsum[threadIdx.x >> 5] = inc;
  if (threadIdx.x == 0) sm.pick = c.key == prefix ? c.id : V - 1;
  __syncthreads();
  u64 ahead = inc - mine;
  for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) ahead += sm.wsum[i];
  if (ahead < need && ahead + mine >= need) {
    u64 left = need - ahead;
    for (int v = a; v < b; ++v) {
      const unsigned k = okey(ld(row + v));
      if (k == prefix && kept(k, v, c) && --left == 0) sm.pick = v;
    }
  }
  __syncthreads();
  Cut out;
  out.key = prefix;
  out.id = sm.pick;
  __syncthreads();
  return out;
}

struct Row {
  Scale s;
  Cut cut;
  u64 total;  // kept mass; 0: no token has any
  bool greedy;
};

// Everything the outputs need of one row.
template <typename T>
__device__ Row row_cut(const T* row, int V, float temp, int top_k, float top_p, float min_p, Smem& sm) {
  float mx = -INFINITY;
  for (int v = threadIdx.x; v < V; v += NT) {
    const float z = ld(row + v);
    mx = z > mx ? z : mx;
  }
  mx = warp_max(mx);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.wmax[threadIdx.x >> 5] = mx;
  __syncthreads();
  for (int i = 0; i < NW; ++i) mx = fmaxf(mx, sm.wmax[i]);
  Row r;
  r.greedy = !(temp > 0.f);
  r.s = make_scale(mx, r.greedy ? 1.f : temp);
  r.cut.key = KEY_NINF + 1;  // everything above -inf
  r.cut.id = V;
  r.total = 0;
  if (!(mx > -INFINITY)) return r;
  if (r.greedy) top_k = 1;
  if (top_k > 0 && top_k < V) {
    u64 n = 0;
    for (int v = threadIdx.x; v < V; v += NT) n += okey(ld(row + v)) > KEY_NINF;
    n = block_sum_u64(n, sm);
    if ((u64)top_k < n) r.cut = select_prefix(row, V, r.s, r.cut, true, (u64)top_k, sm);
  }
  auto sum = [&]() {
    u64 t = 0;
    for (int v = threadIdx.x; v < V; v += NT) {
      const float z = ld(row + v);
      const unsigned k = okey(z);
      if (kept(k, v, r.cut)) t += mass_of(z, r.s);
    }
    return block_sum_u64(t, sm);
  };
  r.total = sum();
  if (r.greedy) return r;
  if (top_p < 1.f) {
    const double want = (double)top_p * (double)r.total;
    u64 target = want > 0.0 ? (u64)ceil(want) : 1ull;
    if (target < 1) target = 1;
    if (target > r.total) target = r.total;
    r.cut = select_prefix(row, V, r.s, r.cut, false, target, sm);
    r.total = sum();
  }
  if (min_p > 0.f) {
    // z >= max z + T ln(min_p), as the smallest float that satisfies it
    const double zt = (double)mx + (double)temp * log((double)min_p);
    float zf = (float)zt;
    if ((double)zf < zt) zf = nextafterf(zf, INFINITY);
    zf = fminf(zf, mx);
    const unsigned k = okey(zf);
    if (k > r.cut.key) {
      r.cut.key = k;
      r.cut.id = V;
      r.total = sum();
    }
  }
  return r;
}

// First token in id order whose cumulative kept mass exceeds u times the
// total, without token x.  -1 when no mass is left.
template <typename T>
__device__ int row_draw(const T* row, int V, const Row& r, int x, float u, Smem& sm) {
  const int per = (V + NT - 1) / NT;
  const int a = min(V, (int)threadIdx.x * per), b = min(V, a + per);
  auto w = [&](int v) {
    const float z = ld(row + v);
    return v != x && kept(okey(z), v, r.cut) ? mass_of(z, r.s) : 0ull;
  };
  u64 mine = 0;
  for (int v = a; v < b; ++v) mine += w(v);
  const u64 total = block_sum_u64(mine, sm);
  if (total == 0) return -1;
  u64 inc = mine;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) sm.wsum[threadIdx.x >> 5] = inc;
  __syncthreads();
  u64 c = inc - mine;
  for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) c += sm.wsum[i];
  const u64 t = (u64)((double)fminf(fmaxf(u, 0.f), 0.99999994f) * (double)total);
  if (c <= t && t < c + mine)
    for (int v = a; v < b; ++v) {
      c += w(v);
      if (t < c) {
        sm.pick = v;
        break;
      }
    }
  __syncthreads();
  return sm.pick;
}

template <typename T>
__global__ void __launch_bounds__(NT) sample_kernel(SamplingArgs a) {
  __shared__ Smem sm;
  pdl_launch_next();
  pdl_wait();
  const int row = blockIdx.x, V = a.vocab;
  const int s = row / a.rows, i = row - s * a.rows;  // sequence and its row
  int nd = a.rows - 1;
  if (a.kind == SAMPLING_VERIFY) {
    if (a.n_draft) nd = min(max(a.n_draft[s], 0), nd);
    if (i > nd) return;
  }
  const T* z = static_cast<const T*>(a.logits) + (size_t)row * a.stride;
  const Row r = row_cut(z, V, a.temperature ? a.temperature[s] : 1.f, a.top_k ? a.top_k[s] : 0,
                        a.top_p ? a.top_p[s] : 1.f, a.min_p ? a.min_p[s] : 0.f, sm);
  if (r.total == 0 && threadIdx.x == 0) flag(a.status, DFLASH2_DEV_EMPTY_ROW);
  if (a.kind == SAMPLING_PROBS) {
    float* p = a.prob + (size_t)row * V;
    const float inv = r.total ? (float)(4398046511104.0 / (double)r.total) : 0.f;
    for (int v = threadIdx.x; v < V; v += NT) {
      const float zv = ld(z + v);
      p[v] = r.total && kept(okey(zv), v, r.cut) ? mass_f32(zv, r.s) * inv : 0.f;
    }
    return;
  }
  if (a.kind == SAMPLING_TOKEN) {
    const int t = r.total ? row_draw(z, V, r, -1, a.u[row], sm) : -1;
    if (threadIdx.x == 0) {
      a.token[row] = t;
      if (a.prob)
        a.prob[row] = t < 0 ? 0.f : mass_f32(ld(z + t), r.s) * (float)(4398046511104.0 / (double)r.total);
    }
    return;
  }
  // verification: whether draft i passes, and the token emitted if it does not
  bool pass = false;
  int x = -1;
  if (i < nd) {
    x = a.path[(size_t)s * (a.rows - 1) + i];
    if (r.total && x >= 0 && x < V) {
      const float zx = ld(z + x);
      const u64 mx = kept(okey(zx), x, r.cut) ? mass_of(zx, r.s) : 0ull;
      const float u = fminf(fmaxf(a.u_accept[(size_t)s * (a.rows - 1) + i], 0.f), 0.99999994f);
      pass = (double)u * (double)r.total < (double)mx;
    }
  }
  const int t = r.total && !pass ? row_draw(z, V, r, x, a.u[s], sm) : -1;
  if (threadIdx.x == 0) a.rowout[row] = make_int2(pass, t);
}

// The accepted prefix of each sequence, its emitted tokens and the counters.
__global__ void verify_rows_kernel(SamplingArgs a) {
  pdl_launch_next();
  pdl_wait();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= a.batch) return;
  const int B = a.rows, D = B - 1;
  const int nd = a.n_draft ? min(max(a.n_draft[s], 0), D) : D;
  const int2* ro = a.rowout + (size_t)s * B;
  int n = 0;
  while (n < nd && ro[n].x) ++n;
  const int tok = ro[n].y;
  for (int i = 0; i < B; ++i) a.out_tok[(size_t)s * B + i] = i < n ? a.path[(size_t)s * D + i] : (i == n ? tok : -1);
  a.accept_len[s] = n;
  a.n_out[s] = n + 1;
  a.next_anchor[s] = tok;
  if (a.seq_len) a.seq_len[s] += n + 1;
  if (a.counters) {
    u64* c = reinterpret_cast<u64*>(a.counters);
    atomicAdd(c + 0, 1ull);
    atomicAdd(c + 1, (u64)nd);
    atomicAdd(c + 2, (u64)n);
    atomicAdd(c + 3, (u64)(nd - n));
    atomicAdd(c + 4 + n, 1ull);
    for (int i = 0; i < n; ++i) atomicAdd(c + 4 + B + i, 1ull);
  }
}

}  // namespace

int launch_sampling(const SamplingArgs& a, const Ctx& c) {
  const dim3 grid(a.batch * a.rows);
  const int k = a.bf16_logits ? launch_k(sample_kernel<bf16>, grid, dim3(NT), 0, c, a)
                              : launch_k(sample_kernel<float>, grid, dim3(NT), 0, c, a);
  if (k != DFLASH2_OK || a.kind != SAMPLING_VERIFY) return k;
  return launch_k(verify_rows_kernel, dim3((a.batch + 127) / 128), dim3(128), 0, c, a);
}

}  // namespace df2
