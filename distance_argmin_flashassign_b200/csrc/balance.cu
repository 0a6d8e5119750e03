// balance.cu -- balance loss of rows routed to columns (experts, codes), with
// the per-column counts, and its gradient.
//
// For the n rows of a problem that take part (mask not 0, some logit above
// -inf), with M chosen columns each:
//   lse_i = ln sum_e exp z_ie      p_ie = exp(z_ie - lse_i)
//   P_e = (1/n) sum_i p_ie         f_e = count_e / (M n)
//   loss = coef E sum_e f_e P_e
//   dz_ie = g coef E / n  p_ie (f_e - sum_j f_j p_ij)
// One pass over the logits forward, one backward: a row lives in the
// registers of a team of lanes, its probabilities are added to the column
// sums that each lane keeps in registers over all of its rows, and blocks
// leave their sums in partial rows that a second kernel adds in block order.
// Counts are integers, so the shared-memory atomics that make them do not
// change the result.
#include <type_traits>

#include "chain.cuh"
#include "fk_internal.h"

namespace fk {

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// VL consecutive elements of T.
template <typename T, int VL> struct Pack {
  T e[VL];
};
template <typename T, int VL> __device__ __forceinline__ void ld_pack(const T *p, float *v) {
  constexpr int VB = VL * (int)sizeof(T);
  Pack<T, VL> k;
  if constexpr (VB == 16) {
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    memcpy(&k, &r, 16);
  } else {
    static_assert(VL == 1, "whole 16-byte packs or single elements");
    k.e[0] = *p;
  }
#pragma unroll
  for (int i = 0; i < VL; ++i) v[i] = to_f32<T>(k.e[i]);
}
template <typename T, int VL> __device__ __forceinline__ void st_pack(T *p, const float *v) {
  constexpr int VB = VL * (int)sizeof(T);
  Pack<T, VL> k;
#pragma unroll
  for (int i = 0; i < VL; ++i) k.e[i] = from_f32<T>(v[i]);
  if constexpr (VB == 16) {
    uint4 r;
    memcpy(&r, &k, 16);
    *reinterpret_cast<uint4 *>(p) = r;
  } else {
    *p = k.e[0];
  }
}

constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;
constexpr int kBalLane = 32;  // columns a lane holds at most

// Teams: a row belongs to G = 2^logg lanes of a warp, or (WIDE) to the whole
// block; lane l holds the packs l, l + G, l + 2G, ... of VL columns each.
struct Team {
  int logg, lane, row0, rows;  // lane in the team; the block's first row's team; teams a block
};
template <bool WIDE> __device__ __forceinline__ Team team_of(int logg) {
  Team t;
  if (WIDE) {
    t.logg = 8;
    t.lane = threadIdx.x;
    t.row0 = 0;
    t.rows = 1;
  } else {
    t.logg = logg;
    t.lane = threadIdx.x & ((1 << logg) - 1);
    t.row0 = threadIdx.x >> logg;
    t.rows = kBalThreads >> logg;
  }
  return t;
}

template <typename T, int VL, int P, bool WIDE>
__global__ void __launch_bounds__(kBalThreads) balance_rows_kernel(const T *__restrict__ Z,
                                                                   const int32_t *__restrict__ ids,
                                                                   const uint8_t *__restrict__ mask, int N, int E,
                                                                   int M, int logg, float *__restrict__ lse,
                                                                   float *__restrict__ psum, int *__restrict__ csum,
                                                                   int *__restrict__ tsum, int *status) {
  constexpr int NE = VL * P;
  extern __shared__ int smem[];
  int *hist = smem;                                   // [E] chosen columns of the block's rows
  float *cols = reinterpret_cast<float *>(smem + E);  // [E] column sums
  __shared__ float wm[2][kBalWarps], wsum[2][kBalWarps];
  __shared__ int taken[kBalWarps];
  const float ninf = __int_as_float(0xff800000);
  const Team t = team_of<WIDE>(logg);
  const int b = blockIdx.y, G = 1 << t.logg;
  const T *Zb = Z + (size_t)b * N * E;
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    hist[e] = 0;
    cols[e] = 0.f;
  }
  __syncthreads();
  wait_prior_grid();
  float acc[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) acc[i] = 0.f;
  int mytok = 0, buf = 0;
  bool bad = false;
  for (long long r0 = (long long)blockIdx.x * t.rows; r0 < N; r0 += (long long)gridDim.x * t.rows) {
    const long long r = r0 + t.row0;
    const bool live = r < N && (!mask || mask[(size_t)b * N + r] != 0);
    float z[NE];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + t.lane) * VL;
      if (live && c < E) {
        ld_pack<T, VL>(Zb + (size_t)r * E + c, z + p * VL);
      } else {
#pragma unroll
        for (int i = 0; i < VL; ++i) z[p * VL + i] = ninf;
      }
    }
    float m = ninf;
#pragma unroll
    for (int i = 0; i < NE; ++i) m = fmaxf(m, z[i]);
    for (int o = WIDE ? 16 : G >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // a team without a logit above -inf takes 0 for its maximum: its sum is 0 (or NaN)
    if (m == ninf) m = 0.f;
    const float m0 = m;
    if (fabsf(m) > 1e38f) {  // m log2(e) would overflow (a row of the type's lowest values)
#pragma unroll
      for (int i = 0; i < NE; ++i) z[i] -= m;
      m = 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      z[i] = exp2_fast(fmaf(z[i], kLog2e, -m * kLog2e));
      s += z[i];
    }
    for (int o = WIDE ? 16 : G >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    float factor;  // p_e = z[e] factor
    float l;
    if (WIDE) {
      // z holds exp(z - the warp's maximum): one exchange of the warps' maxima and sums
      if ((threadIdx.x & 31) == 0) {
        wm[buf][threadIdx.x >> 5] = s == 0.f ? ninf : m0;
        wsum[buf][threadIdx.x >> 5] = s;
      }
      __syncthreads();
      float M_ = ninf, S = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) M_ = fmaxf(M_, wm[buf][w]);
      if (M_ == ninf) M_ = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) S += wsum[buf][w] * (wsum[buf][w] == 0.f ? 0.f : exp2_fast((wm[buf][w] - M_) * kLog2e));
      buf ^= 1;
      factor = (s == 0.f ? 0.f : exp2_fast((m0 - M_) * kLog2e)) / S;  // NaN in every warp of a NaN row
      l = M_ + logf(S);
      s = S;
    } else {
      factor = 1.f / s;
      l = m0 + logf(s);
    }
    const bool on = live && s != 0.f;
    if (on) {
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] = fmaf(z[i], factor, acc[i]);
      for (int j = t.lane; j < M; j += G) {
        const int id = ids[((size_t)b * N + r) * M + j];
        if ((unsigned)id < (unsigned)E) atomicAdd(hist + id, 1);
        else bad |= id != -1;
      }
    }
    if (t.lane == 0) {
      mytok += on;
      if (lse && r < N) lse[(size_t)b * N + r] = on ? l : __int_as_float(0x7f800000);
    }
  }
  if (bad) record_status(status, kStBadLabel);
  // column sums: over the teams of a warp, then over the warps in order
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int c = (i / VL * G + t.lane) * VL + i % VL;
      if (c < E) cols[c] = acc[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      for (int o = G; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    for (int w = 0; w < kBalWarps; ++w) {
      if ((int)(threadIdx.x >> 5) == w && (threadIdx.x & 31) < G) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int c = (i / VL * G + t.lane) * VL + i % VL;
          if (c < E) cols[c] += acc[i];
        }
      }
      __syncthreads();
    }
  }
  for (int o = 16; o > 0; o >>= 1) mytok += __shfl_xor_sync(0xffffffffu, mytok, o);
  if ((threadIdx.x & 31) == 0) taken[threadIdx.x >> 5] = mytok;
  __syncthreads();
  const size_t part = (size_t)b * gridDim.x + blockIdx.x;
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    psum[part * E + e] = cols[e];
    csum[part * E + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < kBalWarps; ++w) n += taken[w];
    tsum[part] = n;
  }
}

// One block per problem: adds the blocks' partial rows in order, in fp64.
__global__ void __launch_bounds__(1024) balance_join_kernel(const float *__restrict__ psum,
                                                            const int *__restrict__ csum,
                                                            const int *__restrict__ tsum, int nparts, int E, int M,
                                                            float coef, float *__restrict__ loss,
                                                            int32_t *__restrict__ counts,
                                                            int32_t *__restrict__ tokens, float *__restrict__ meanp) {
  __shared__ double part[32];
  __shared__ int ntok;
  const int b = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  wait_prior_grid();
  if (w == 0) {
    int n = 0;
    for (int q = lane; q < nparts; q += 32) n += tsum[(size_t)b * nparts + q];
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) ntok = n;
  }
  __syncthreads();
  const int n = ntok;
  double mine = 0.0;
  for (int e = threadIdx.x; e < E; e += 1024) {
    double p = 0.0;
    int c = 0;
    for (int q = 0; q < nparts; ++q) {
      p += (double)psum[((size_t)b * nparts + q) * E + e];
      c += csum[((size_t)b * nparts + q) * E + e];
    }
    if (n > 0) p /= (double)n;
    counts[(size_t)b * E + e] = c;
    if (meanp) meanp[(size_t)b * E + e] = (float)p;
    mine += p * (double)c;
  }
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) part[w] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    for (int i = 0; i < 32; ++i) sum += part[i];
    loss[b] = n > 0 ? (float)((double)coef * E * sum / ((double)M * n)) : 0.f;
    tokens[b] = n;
  }
}

template <typename T, int VL, int P, bool WIDE>
__global__ void __launch_bounds__(kBalThreads) balance_grad_kernel(const T *Z, const int32_t *__restrict__ counts,
                                                                   const int32_t *__restrict__ tokens,
                                                                   const float *__restrict__ lse,
                                                                   const float *__restrict__ gloss, int N, int E,
                                                                   int M, float coef, int logg, T *dZ) {
  constexpr int NE = VL * P;
  __shared__ float wdot[2][kBalWarps];
  const Team t = team_of<WIDE>(logg);
  const int b = blockIdx.y, G = 1 << t.logg;
  const T *Zb = Z + (size_t)b * N * E;
  T *dZb = dZ + (size_t)b * N * E;
  wait_prior_grid();
  const int n = tokens[b] > 0 ? tokens[b] : 1;
  const float k = (gloss ? gloss[b] : 1.f) * (coef * (float)E / (float)n);
  float f[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int c = (i / VL * G + t.lane) * VL + i % VL;
    f[i] = c < E ? (float)counts[(size_t)b * E + c] / ((float)M * (float)n) : 0.f;
  }
  int buf = 0;
  for (long long r0 = (long long)blockIdx.x * t.rows; r0 < N; r0 += (long long)gridDim.x * t.rows) {
    const long long r = r0 + t.row0;
    const float l = r < N ? lse[(size_t)b * N + r] : 0.f;
    const bool on = r < N && l != __int_as_float(0x7f800000);
    float z[NE], dot = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * G + t.lane) * VL;
      if (on && c < E) {
        ld_pack<T, VL>(Zb + (size_t)r * E + c, z + p * VL);
#pragma unroll
        for (int i = 0; i < VL; ++i) z[p * VL + i] = exp2_fast((z[p * VL + i] - l) * kLog2e);
      } else {
#pragma unroll
        for (int i = 0; i < VL; ++i) z[p * VL + i] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) dot = fmaf(f[i], z[i], dot);
    for (int o = WIDE ? 16 : G >> 1; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (WIDE) {
      if ((threadIdx.x & 31) == 0) wdot[buf][threadIdx.x >> 5] = dot;
      __syncthreads();
      dot = 0.f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) dot += wdot[buf][w];
      buf ^= 1;
    }
    if (r < N) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int c = (p * G + t.lane) * VL;
        if (c < E) {
          float o[VL];
#pragma unroll
          for (int i = 0; i < VL; ++i) o[i] = on ? k * z[p * VL + i] * (f[p * VL + i] - dot) : 0.f;
          st_pack<T, VL>(dZb + (size_t)r * E + c, o);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host ---
// How a row of E logits is spread: whole 16-byte packs when the rows and the
// pointers are whole 16-byte pieces, else single elements; the fewest packs a
// lane with at most 32 lanes, or the whole block where a lane would hold more
// than kBalLane columns.
struct Spread {
  int VL, P, logg;
  bool wide;
  int rows;  // rows of a block's step
};
static Spread spread_of(int E, DType dt, bool aligned) {
  Spread p{};
  const int full = 16 / (int)dtype_size(dt);
  p.VL = aligned && E % full == 0 ? full : 1;
  const int packs = (E + p.VL - 1) / p.VL, most = kBalLane / p.VL;
  const int lanes = (packs + most - 1) / most > 32 ? kBalThreads : 32;
  p.wide = lanes > 32;
  p.P = 1;
  while (p.P * lanes < packs) p.P *= 2;
  while (!p.wide && (p.P << p.logg) < packs) ++p.logg;
  if (p.wide) p.logg = 8;
  p.rows = kBalThreads >> p.logg;
  return p;
}

// Blocks per problem: about 148 x 4 in all while there are rows for them,
// more where a team would add over 1,024 rows into one fp32 sum.
static int balance_blocks(int B, int64_t N, const Spread &p) {
  const int64_t steps = (N + p.rows - 1) / p.rows;
  int64_t nb = (148 * 4 + B - 1) / B;
  if (nb * 1024 < steps) nb = (steps + 1023) / 1024;
  return (int)(nb < steps ? nb : steps);
}

static size_t al256(size_t v) { return (v + 255) / 256 * 256; }
static size_t parts_bytes(int B, int64_t N, int E, const Spread &p) {
  const size_t parts = (size_t)B * balance_blocks(B, N, p);
  return 2 * al256(parts * E * 4) + al256(parts * 4);
}
// Enough for either alignment of Z.
size_t balance_workspace_bytes(int B, int64_t N, int E, DType dt) {
  const size_t a = parts_bytes(B, N, E, spread_of(E, dt, true)), u = parts_bytes(B, N, E, spread_of(E, dt, false));
  return a > u ? a : u;
}

// Calls f with the spread's template arguments.
template <typename T, typename F> static void with_spread(const Spread &p, F f) {
  constexpr int V = 16 / (int)sizeof(T);
#define FK_P(vl, n)                                                                              \
  if (p.VL == vl && p.P == n) {                                                                  \
    if (p.wide) return f(std::integral_constant<int, vl>(), std::integral_constant<int, n>(), std::true_type()); \
    return f(std::integral_constant<int, vl>(), std::integral_constant<int, n>(), std::false_type());            \
  }
  FK_P(V, 1) FK_P(V, 2) FK_P(V, 4)
  if constexpr (V == 4) { FK_P(V, 8) }
  FK_P(1, 1) FK_P(1, 2) FK_P(1, 4) FK_P(1, 8) FK_P(1, 16) FK_P(1, 32)
#undef FK_P
}

template <typename T> static cudaError_t balance_from(const BalanceArgs &a, void *ws, int *status, cudaStream_t s) {
  const Spread p = spread_of(a.E, a.dt, (uintptr_t)a.Z % 16 == 0);
  const int nb = balance_blocks(a.B, a.N, p);
  const size_t parts = (size_t)a.B * nb;
  float *psum = (float *)ws;
  int *csum = (int *)((char *)ws + al256(parts * a.E * 4));
  int *tsum = (int *)((char *)ws + 2 * al256(parts * a.E * 4));
  const size_t smem = (size_t)a.E * 8;
  cudaError_t e = cudaSuccess;
  with_spread<T>(p, [&](auto vl, auto np, auto wide) {
    const auto kernel = balance_rows_kernel<T, decltype(vl)::value, decltype(np)::value, decltype(wide)::value>;
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
      e = launch_chained(kernel, dim3(nb, a.B), dim3(kBalThreads), smem, s, (const T *)a.Z, a.ids, a.mask, a.N, a.E, a.M,
                         p.logg, a.lse, psum, csum, tsum, status);
  });
  if (e != cudaSuccess) return e;
  return launch_chained(balance_join_kernel, dim3(a.B), dim3(1024), 0, s, psum, csum, tsum, nb, a.E, a.M, a.coef, a.loss,
                        a.counts, a.tokens, a.meanp);
}
cudaError_t launch_balance(const BalanceArgs &a, void *ws, int *status, cudaStream_t s) {
  count_launches(2);
  return a.dt == kF32   ? balance_from<float>(a, ws, status, s)
         : a.dt == kF16 ? balance_from<__half>(a, ws, status, s)
                        : balance_from<__nv_bfloat16>(a, ws, status, s);
}

template <typename T> static cudaError_t balance_grad_from(const BalanceGradArgs &a, cudaStream_t s) {
  const Spread p = spread_of(a.E, a.dt, (uintptr_t)a.Z % 16 == 0 && (uintptr_t)a.dZ % 16 == 0);
  cudaError_t e = cudaSuccess;
  with_spread<T>(p, [&](auto vl, auto np, auto wide) {
    e = launch_chained(balance_grad_kernel<T, decltype(vl)::value, decltype(np)::value, decltype(wide)::value>,
                       dim3(balance_blocks(a.B, a.N, p), a.B), dim3(kBalThreads), 0, s, (const T *)a.Z, a.counts,
                       a.tokens, a.lse, a.gloss, a.N, a.E, a.M, a.coef, p.logg, (T *)a.dZ);
  });
  return e;
}
cudaError_t launch_balance_grad(const BalanceGradArgs &a, cudaStream_t s) {
  count_launches(1);
  return a.dt == kF32   ? balance_grad_from<float>(a, s)
         : a.dt == kF16 ? balance_grad_from<__half>(a, s)
                        : balance_grad_from<__nv_bfloat16>(a, s);
}

}  // namespace fk
