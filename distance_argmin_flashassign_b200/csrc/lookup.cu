// lookup.cu -- rows of a codebook by label, and the codebook's gradient.
//
//   Y[b,i]  = scale T[b, ids[b,i]]                    (fk_lookup)
//   dT[b,k] = scale sum over ids[b,i] = k of dY[b,i]  (fk_lookup_grad)
//
// The lookup is the assignment's inverse (points replaced by the centroids
// their labels name); its gradient is the sum part of the centroid update and
// runs on the same sorted order (label_sort.cu): no atomics, every sum in one
// fixed order.  A label of -1 names no row: a zero row of Y, no part in dT.
// The sums are fp32, as the update's are: n rows cost n 2^-24 of their magnitudes
// at worst (2 M rows of Zipf labels: 1.1e-7 of the result measured), two
// additions an instruction, and fp64 would halve the rows in flight.
#include <type_traits>

#include "chain.cuh"
#include "fk_internal.h"

namespace fk {

// ---------------------------------------------------------------- vectors --
// VB bytes moved by one instruction.
template <int VB> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = unsigned int; };
template <> struct Raw<2> { using type = unsigned short; };

template <int VB> __device__ __forceinline__ typename Raw<VB>::type ld_raw(const void *p) {
  return __ldg(reinterpret_cast<const typename Raw<VB>::type *>(p));
}
// Two 16-bit values of a word, and back (rounded to nearest even).
template <typename T> __device__ __forceinline__ void unpack2(uint32_t w, float *v) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    v[0] = f.x;
    v[1] = f.y;
  } else {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t w;
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    memcpy(&w, &h, 4);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    memcpy(&w, &h, 4);
  }
  return w;
}
template <typename T, int VB> __device__ __forceinline__ void unpack_raw(const typename Raw<VB>::type &r, float *v) {
  if constexpr (sizeof(T) == 4) {
    memcpy(v, &r, VB);
  } else if constexpr (VB == 2) {
    T e;
    memcpy(&e, &r, 2);
    v[0] = to_f32<T>(e);
  } else {
    uint32_t w[VB / 4];
    memcpy(w, &r, VB);
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) unpack2<T>(w[i], v + 2 * i);
  }
}
// n values rounded to nearest even and stored as one vector.
template <typename T, int n> __device__ __forceinline__ void st_vec(T *p, const float *v) {
  constexpr int VB = n * (int)sizeof(T);
  if constexpr (VB > 16) {
    st_vec<T, n / 2>(p, v);
    st_vec<T, n / 2>(p + n / 2, v + n / 2);
  } else {
    typename Raw<VB>::type r;
    if constexpr (sizeof(T) == 4) {
      memcpy(&r, v, VB);
    } else if constexpr (n == 1) {
      const T e = from_f32<T>(v[0]);
      memcpy(&r, &e, 2);
    } else {
      uint32_t w[n / 2];
#pragma unroll
      for (int i = 0; i < n / 2; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
      memcpy(&r, w, VB);
    }
    *reinterpret_cast<typename Raw<VB>::type *>(p) = r;
  }
}
template <typename T, int n> __device__ __forceinline__ void ld_vec(const T *p, float *v) {
  constexpr int VB = n * (int)sizeof(T);
  if constexpr (VB > 16) {
    ld_vec<T, n / 2>(p, v);
    ld_vec<T, n / 2>(p + n / 2, v + n / 2);
  } else {
    const typename Raw<VB>::type r = *reinterpret_cast<const typename Raw<VB>::type *>(p);
    unpack_raw<T, VB>(r, v);
  }
}

// ----------------------------------------------------------------- lookup --
// Vectors in flight per lane: the rows' round trip through L2 has to be covered
// (1 M x 128 fp16 rows of a 1,024-row table: 50 us; with the rows of a step
// loaded and stored before the next step's are asked for 58 us), with 4 blocks
// an SM.  Narrow vectors need more of them (50,001 x 1,002 fp32 to bf16, 8-byte
// loads: 39 us with 8, 47 with 4) and leave the registers for it, but a step has
// 32 rows at most, which rows of one to four lanes fill with four or fewer (2 M x 6
// bf16, three lanes: 19 us with 4, 27 with 8; 2 M x 10, five lanes: 33 and 31).
constexpr int look_depth(int epl, int lanes) { return epl <= 2 && lanes > 4 ? 8 : 4; }
// Groups of W = 2^logw lanes, one row at a time each; a lane has U vectors of
// EPL elements in flight: of U rows (W vectors cover a row), or, WIDE, of one
// row (slice blockIdx.y of its columns; one label and one address serve U
// vectors).  A warp takes 32 consecutive rows at a time: its lanes hold their
// labels, the next 32 labels are already on their way, and the rows of one
// step are loaded before those of the step before are scaled and stored, so
// that neither the labels' nor the rows' round trip is waited for in full.
template <typename TI, typename TO, int EPL, int U, bool WIDE>
__global__ void __launch_bounds__(256, 4) lookup_kernel(const TI *__restrict__ T, int K, int D,
                                                        const int32_t *__restrict__ ids, int rows, int N, int B,
                                                        float scale, TO *__restrict__ Y, int logw, int *status) {
  constexpr int VB = EPL * (int)sizeof(TI);
  using V = typename Raw<VB>::type;
  const int lane = threadIdx.x & 31;
  const int W = 1 << logw;
  const int col = ((WIDE ? U : 1) * (int)blockIdx.y * W + (lane & (W - 1))) * EPL;
  const int per = 32 >> logw, sub = lane >> logw;
  const int take = WIDE ? per : min(U * per, 32), steps = 32 / take;  // rows of a step, steps of 32 rows
  const long long stride = (long long)gridDim.x * (8 * 32);
  const TI *Tc = T + col;
  TO *Yc = Y + col;
  bool bad = false;
  // a label as the row of the B x K table it names, or -1
  auto row_of = [&](long long r) {
    if (r >= rows) return -1;
    const int id = __ldg(ids + r);
    const bool ok = (unsigned)id < (unsigned)K;
    bad |= !ok && id != -1;
    return ok ? (B > 1 ? (int)r / N * K + id : id) : -1;
  };
  auto load = [&](V *v, int k32, int j) {
    if (WIDE) {
      const int k = __shfl_sync(0xffffffffu, k32, j * take + sub);
      const TI *p = Tc + (size_t)(unsigned)max(k, 0) * (unsigned)D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = V();
        if (k >= 0 && col + u * W * EPL < D) v[u] = ld_raw<VB>(p + u * W * EPL);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = __shfl_sync(0xffffffffu, k32, (j * take + u * per + sub) & 31);
        v[u] = V();
        // (eight only with eight lanes a row or more: 32 rows)
        if ((U > 4 || u * per < take) && k >= 0 && col < D) v[u] = ld_raw<VB>(Tc + (size_t)(unsigned)k * (unsigned)D);
      }
    }
  };
  auto put = [&](const V &v, TO *p) {
    float f[EPL];
    unpack_raw<TI, VB>(v, f);
#pragma unroll
    for (int i = 0; i < EPL; ++i) f[i] *= scale;
    st_vec<TO, EPL>(p, f);
  };
  auto store = [&](const V *v, long long r32, int j) {
    if (WIDE) {
      const unsigned r = (unsigned)r32 + j * take + sub;  // below 2^31 + 32
      if (r < (unsigned)rows) {
        TO *p = Yc + (size_t)r * (unsigned)D;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (col + u * W * EPL < D) put(v[u], p + u * W * EPL);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = j * take + u * per + sub;
        if (u * per < take && col < D && r32 + at < rows)
          put(v[u], Yc + (size_t)(unsigned)((int)r32 + at) * (unsigned)D);
      }
    }
  };
  long long r32 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 32;
  if (r32 >= rows) return;
  int now = row_of(r32 + lane), next = row_of(r32 + stride + lane);
  V x[U], y[U];
  load(x, now, 0);
  int j = 0;
  auto turn = [&](V *cur, V *nxt) {  // loads the step after this one, stores this one
    const long long at = r32;
    const int jj = j;
    if (++j == steps) {
      j = 0;
      r32 += stride;
      now = next;
      load(nxt, now, 0);
      next = row_of(r32 + stride + lane);
    } else {
      load(nxt, now, j);
    }
    store(cur, at, jj);
  };
  while (r32 < rows) {
    turn(x, y);
    if (r32 >= rows) break;
    turn(y, x);
  }
  if (bad) record_status(status, kStBadLabel);
}

template <typename TI, typename TO, int EPL>
static void launch_lookup_as(const LookupArgs &a, int *status, cudaStream_t s) {
  constexpr int U = look_depth(EPL, 32), few = look_depth(EPL, 4);
  const int vecs = a.D / EPL;
  // WIDE from two lanes a row on: a lone lane's 16-byte stores would leave
  // half-written 32-byte sectors behind
  const bool wide = vecs >= 2 * U;
  const int each = wide ? (vecs + U - 1) / U : vecs;  // lanes that a row could use
  int logw = 0;
  while (logw < 5 && (1 << logw) < each) ++logw;
  const int slices = (each + (1 << logw) - 1) >> logw;
  const long long rows = (long long)a.B * a.N, need = (rows + 255) / 256;
  const long long wave = (148 * 4 + slices - 1) / slices;
  const dim3 grid((unsigned)(need < wave ? need : wave), slices);
  const auto kernel = wide        ? lookup_kernel<TI, TO, EPL, U, true>
                      : vecs <= 4 ? lookup_kernel<TI, TO, EPL, few, false>
                                  : lookup_kernel<TI, TO, EPL, U, false>;
  kernel<<<grid, 256, 0, s>>>((const TI *)a.T, a.K, a.D, a.ids, (int)rows, a.N, a.B, a.scale, (TO *)a.Y, logw, status);
}
template <typename TI, typename TO> static void launch_lookup_to(const LookupArgs &a, int *status, cudaStream_t s) {
  constexpr int widest = 16 / (int)(sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO));
  auto fits = [&](int n) {
    return a.D % n == 0 && (uintptr_t)a.T % (n * sizeof(TI)) == 0 && (uintptr_t)a.Y % (n * sizeof(TO)) == 0;
  };
  if (fits(widest)) launch_lookup_as<TI, TO, widest>(a, status, s);
  else if (fits(2)) launch_lookup_as<TI, TO, 2>(a, status, s);
  else launch_lookup_as<TI, TO, 1>(a, status, s);
}
template <typename TI> static void launch_lookup_from(const LookupArgs &a, int *status, cudaStream_t s) {
  if (a.dt_y == kF32) launch_lookup_to<TI, float>(a, status, s);
  else if (a.dt_y == kF16) launch_lookup_to<TI, __half>(a, status, s);
  else launch_lookup_to<TI, __nv_bfloat16>(a, status, s);
}
cudaError_t launch_lookup(const LookupArgs &a, int *status, cudaStream_t s) {
  if (a.dt == kF32) launch_lookup_from<float>(a, status, s);
  else if (a.dt == kF16) launch_lookup_from<__half>(a, status, s);
  else launch_lookup_from<__nv_bfloat16>(a, status, s);
  count_launches(1);
  return cudaGetLastError();
}

// --------------------------------------------------------------- gradient --
// Sorted positions per worker, eight at least (few rows: 1,000 x 64 bf16 13 us,
// 20 us with 32 at least), from the number of 16-byte pieces of dY alone,
// so that the order of a sum depends on the sizes and on nothing else.
// 148 SMs hold 113,664 lanes of the row-sum kernel (3 blocks of 256).
static int grad_rows_R(long long rows, int row_bytes) {
  const long long pieces = rows * ((row_bytes + 15) / 16);
  long long R = (pieces + 113663) / 113664;
  R = (R + 7) / 8 * 8;
  return (int)(R < 8 ? 8 : R > 512 ? 512 : R);
}

__device__ __forceinline__ void add2(float *a, const float *b) {  // two fp32 additions an instruction
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a[0]), "+f"(a[1])
      : "f"(b[0]), "f"(b[1]));
}
// Writes scale v (+ the row's own values) at columns [col, col + n) of row k.
template <int n>
__device__ __forceinline__ void put_grad(void *dT, int dt, size_t at, float *v, float scale, bool add) {
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] *= scale;
  float o[n];
  if (dt == kF32) {
    float *p = (float *)dT + at;
    if (add) {
      ld_vec<float, n>(p, o);
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] += o[i];
    }
    st_vec<float, n>(p, v);
  } else if (dt == kF16) {
    __half *p = (__half *)dT + at;
    if (add) {
      ld_vec<__half, n>(p, o);
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] += o[i];
    }
    st_vec<__half, n>(p, v);
  } else {
    __nv_bfloat16 *p = (__nv_bfloat16 *)dT + at;
    if (add) {
      ld_vec<__nv_bfloat16, n>(p, o);
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] += o[i];
    }
    st_vec<__nv_bfloat16, n>(p, v);
  }
}

// Worker = W lanes, one chunk of R sorted positions and one slice of W * EPL
// columns.  A segment (run of one label) inside the chunk goes straight to
// dT; the pieces of segments that cross the chunk's ends go to the chunk's
// two partial rows (0: the piece that starts the chunk, 1: the one that ends
// it).  `none` is the key of the points left out.  As in the lookup, the lanes
// hold W positions' keys and rows, the next W are on their way, and the rows
// of a step are loaded before those of the step before are added.
constexpr int kGradRows = 4;  // rows of a step
template <typename T, int VB, int W>
__global__ void __launch_bounds__(256, 3) grad_sum_kernel(const T *__restrict__ dY, int D,
                                                          const int32_t *__restrict__ skeys,
                                                          const int32_t *__restrict__ perm, int rows, int none, int R,
                                                          float scale, void *__restrict__ dT, int dt_t, int add,
                                                          float *__restrict__ parts) {
  constexpr int EPL = VB / (int)sizeof(T), U = kGradRows;
  using V = typename Raw<VB>::type;
  const int lw = threadIdx.x % W;
  const int col = (blockIdx.y * W + lw) * EPL;
  const bool mine = col < D;
  const T *Yc = dY + col;
  const long long wq = ((long long)blockIdx.x * 256 + threadIdx.x) / W;
  wait_prior_grid();
  const long long p0l = wq * R;
  const int p0 = p0l < rows ? (int)p0l : rows;
  const int p1 = rows - p0 < R ? rows : p0 + R;
  const bool live = p0 < p1;
  auto key_at = [&](long long pos) { return pos < p1 ? skeys[pos] : none; };
  auto row_at = [&](long long pos) { return pos < p1 ? perm[pos] : 0; };
  // the W positions at hand and the next W: key, and row (-1: left out)
  int kn = key_at((long long)p0 + lw), rn = row_at((long long)p0 + lw);
  int kx = key_at((long long)p0 + W + lw), rx = row_at((long long)p0 + W + lw);
  if (kn == none) rn = -1;
  int cur = live ? skeys[p0] : none, s = p0;
  const bool split_start = live && p0 > 0 && skeys[p0 - 1] == cur;
  const bool split_end = live && p1 < rows && skeys[p1] == skeys[p1 - 1];
  float a[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) a[i] = 0.f;
  auto flush = [&](int k, int sb, int se) {
    if (k == none || !mine) return;
    if ((sb == p0 && split_start) || (se == p1 && split_end))
      st_vec<float, EPL>(parts + ((size_t)wq * 2 + (sb == p0 ? 0 : 1)) * D + col, a);
    else
      put_grad<EPL>(dT, dt_t, (size_t)k * D + col, a, scale, add);
  };
  auto add_row = [&](const V &v) {
    float f[EPL];
    unpack_raw<T, VB>(v, f);
    if constexpr (EPL == 1) {
      a[0] += f[0];
    } else {
#pragma unroll
      for (int i = 0; i < EPL; i += 2) add2(a + i, f + i);
    }
  };
  struct Step {
    V v[U];
    int keys, first, last;  // the W positions' keys it is among; its first and last position's
  } x, y;
  auto load = [&](Step &n, int j) {  // step j of the W positions at hand
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = __shfl_sync(0xffffffffu, rn, j * U + u, W);
      if (row >= 0 && mine) n.v[u] = ld_raw<VB>(Yc + (size_t)(unsigned)row * (unsigned)D);
    }
    n.keys = kn;
    n.first = __shfl_sync(0xffffffffu, kn, j * U, W);
    n.last = __shfl_sync(0xffffffffu, kn, j * U + U - 1, W);
  };
  int j = 0, base = p0;  // the step to add: its place among its W positions, its first position
  auto turn = [&](Step &c, Step &n) {
    const int jc = j;
    if (++j == W / U) {
      j = 0;
      kn = kx;
      rn = kx == none ? -1 : rx;
      load(n, 0);
      kx = key_at((long long)base + U + W + lw);
      rx = row_at((long long)base + U + W + lw);
    } else {
      load(n, j);
    }
    // a label's positions are consecutive: equal ends, one label in between
    if (__all_sync(0xffffffffu, c.first == cur && c.last == cur && cur != none)) {
      if (mine)
#pragma unroll
        for (int u = 0; u < U; ++u) add_row(c.v[u]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = __shfl_sync(0xffffffffu, c.keys, jc * U + u, W);
        if (base + u < p1) {
          if (k != cur) {
            flush(cur, s, base + u);
            cur = k;
            s = base + u;
#pragma unroll
            for (int i = 0; i < EPL; ++i) a[i] = 0.f;
          }
          if (cur != none && mine) add_row(c.v[u]);
        }
      }
    }
    base += U;
  };
  load(x, 0);
  for (int i = 0; i < R; i += 2 * U) {  // the same for every worker: shuffles stay converged
    turn(x, y);
    turn(y, x);
  }
  if (live) flush(cur, s, p1);
}

// A segment that starts in chunk q and runs past its end is joined from its
// partial rows here, by the warp that looks at chunk q; where it has more than
// kHotPieces of them, by the block's 32 warps afterwards (warp w adds pieces
// w, w + 32, ..., then the 32 sums are added in warp order).  blockIdx.y:
// slice of kJoinCols columns, taken 128 at a time, four a lane (kept
// as a loop: 1 M x 128 rows of one label take 107 us for the whole gradient, and
// 147 where the same is written without one).
// Pieces: with 4 as the border 30,000 x 4,096 rows of 32 labels take 83 us for
// the whole gradient, with 16 or 64 73; with 64, 16,384 x 2,048 rows of Zipf labels
// take 94, with 16 79.  Columns: 500 x 1,024 rows of Zipf labels take 16 us with
// 64 or 128 a block, 24 with 512 (one block adds its slices of a hot label one
// after another); 1 M x 128 rows of 256 labels take 76 with 64, else 72.
constexpr int kHotPieces = 16, kJoinCols = 128;
__global__ void __launch_bounds__(1024) grad_join_kernel(const int32_t *__restrict__ skeys, int rows, int none, int R,
                                                         int D, const float *__restrict__ parts, float scale,
                                                         void *__restrict__ dT, int dt_t, int add) {
  __shared__ float red[32][129];
  __shared__ int hot_q[32], hot_np[32], hot_k[32], hot_first[32], nhot;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int nchunks = (rows + R - 1) / R, q = blockIdx.x * 32 + w;
  const int c0 = blockIdx.y * kJoinCols, c1 = min(D, c0 + kJoinCols);
  if (threadIdx.x == 0) nhot = 0;
  __syncthreads();
  wait_prior_grid();
  // pieces of the segment that ends chunk q: this chunk's and those of the
  // following chunks that start with its label (a label's positions are
  // consecutive, so these chunks are too); 1 where it does not start here or
  // does not run past the end
  int np = 1, k = none, first = 0;  // first: the chunk's partial row that holds its piece
  if (q < nchunks - 1) {
    const int p0 = q * R, p1 = p0 + R;
    k = skeys[p1 - 1];
    const int after = skeys[p1], before = p0 > 0 ? skeys[p0 - 1] : -1;
    first = skeys[p0] == k ? 0 : 1;
    if (k != none && after == k && before != k) {
      // the last such chunk: chunk lo starts with k, chunk hi does not.  32
      // chunks are looked at first, which is enough for most labels, then 32 of
      // the rest at equal distances, and so on
      int lo = q + 1, hi = nchunks;
      for (int step = 1; hi - lo > 1; step = (hi - lo + 31) / 32) {
        const int i = lo + step * (lane + 1);
        const unsigned in = __ballot_sync(0xffffffffu, i < hi && skeys[i < hi ? i * R : 0] == k);
        const int n = __popc(in);
        if (n < 32) hi = min(hi, lo + step * (n + 1));
        lo += step * n;
      }
      np = lo - q + 1;
    }
  }
  auto piece = [&](int q, int first, int i) { return parts + ((size_t)(q + i) * 2 + (i == 0 ? first : 0)) * D; };
  // adds pieces from, from + by, ... of columns c + lane + 32 j, four pieces loaded at a time
  auto add_pieces = [&](float *t, int q, int first, int from, int by, int np, int c) {
    for (int i0 = from; i0 < np; i0 += 4 * by) {
      float v[4][4];
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int i = i0 + ii * by;
        const float *row = piece(q, first, i < np ? i : 0) + c + lane;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) v[ii][jj] = i < np && c + lane + 32 * jj < c1 ? row[32 * jj] : 0.f;
      }
#pragma unroll
      for (int ii = 0; ii < 4; ++ii)
        if (i0 + ii * by < np) {
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) t[jj] += v[ii][jj];
        }
    }
  };
  if (np > kHotPieces) {
    if (lane == 0) {
      const int i = atomicAdd(&nhot, 1);  // any order: each is summed by itself
      hot_q[i] = q;
      hot_np[i] = np;
      hot_k[i] = k;
      hot_first[i] = first;
    }
  } else if (np > 1) {
    for (int c = c0; c < c1; c += 128) {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
      add_pieces(t, q, first, 0, 1, np, c);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
        if (c + lane + 32 * jj < c1) put_grad<1>(dT, dt_t, (size_t)k * D + c + lane + 32 * jj, t + jj, scale, add);
    }
  }
  __syncthreads();
  for (int h = 0; h < nhot; ++h) {
    const int hq = hot_q[h], hk = hot_k[h];
    for (int c = c0; c < c1; c += 128) {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
      add_pieces(t, hq, hot_first[h], w, 32, hot_np[h], c);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) red[w][lane + 32 * jj] = t[jj];
      __syncthreads();
      if (threadIdx.x < 128 && c + threadIdx.x < c1) {
        float sum[1] = {0.f};
        for (int ww = 0; ww < 32; ++ww) sum[0] += red[ww][threadIdx.x];
        put_grad<1>(dT, dt_t, (size_t)hk * D + c + threadIdx.x, sum, scale, add);
      }
      __syncthreads();
    }
  }
}

static size_t al256(size_t v) { return (v + 255) / 256 * 256; }

size_t lookup_grad_workspace_bytes(int64_t rows, int64_t Ktot, int B, int D, DType dt) {
  const int R = grad_rows_R(rows, D * (int)dtype_size(dt));
  return al256(label_sort_bytes(rows, Ktot, B, true)) + al256((size_t)((rows + R - 1) / R) * 2 * D * sizeof(float));
}

template <typename T, int VB, int W>
static void launch_grad_sum(const LookupGradArgs &a, const LabelSort &o, int rows, int none, int R, float *parts,
                            cudaStream_t s) {
  constexpr int EPL = VB / (int)sizeof(T);
  const long long chunks = ((long long)rows + R - 1) / R;
  const dim3 grid((unsigned)((chunks * W + 255) / 256), (a.D + W * EPL - 1) / (W * EPL));
  launch_chained(grad_sum_kernel<T, VB, W>, grid, dim3(256), 0, s, (const T *)a.dY, a.D, o.skeys, o.perm, rows, none, R,
                 a.scale, a.dT, (int)a.dt_t, a.accumulate, parts);
}
template <typename T>
static void launch_grad_from(const LookupGradArgs &a, const LabelSort &o, int rows, int none, int R, float *parts,
                             cudaStream_t s) {
  // the widest vector that the row length and both pointers allow
  auto fits = [&](int vb) {
    const int n = vb / (int)sizeof(T), out = n * (int)dtype_size(a.dt_t);
    return a.D % n == 0 && (uintptr_t)a.dY % vb == 0 && (uintptr_t)a.dT % (out < 16 ? out : 16) == 0;
  };
  if (fits(16)) {
    const int vecs = a.D * (int)sizeof(T) / 16;
    if (vecs <= 8) launch_grad_sum<T, 16, 8>(a, o, rows, none, R, parts, s);
    else if (vecs <= 16) launch_grad_sum<T, 16, 16>(a, o, rows, none, R, parts, s);
    else launch_grad_sum<T, 16, 32>(a, o, rows, none, R, parts, s);
  } else if (fits(8)) {
    launch_grad_sum<T, 8, 32>(a, o, rows, none, R, parts, s);
  } else if (sizeof(T) == 4 || fits(4)) {
    launch_grad_sum<T, 4, 32>(a, o, rows, none, R, parts, s);
  } else if constexpr (sizeof(T) == 2) {
    launch_grad_sum<T, 2, 32>(a, o, rows, none, R, parts, s);
  }
}

cudaError_t launch_lookup_grad(const LookupGradArgs &a, void *ws, int *status, cudaStream_t s) {
  const long long rows = (long long)a.B * a.N, Ktot = (long long)a.B * a.K;
  const size_t fill = a.accumulate ? 0 : (size_t)Ktot * a.D * dtype_size(a.dt_t);  // rows without a label
  if (rows == 0) return fill > 0 ? cudaMemsetAsync(a.dT, 0, fill, s) : cudaSuccess;
  LabelSort o;
  cudaError_t e = launch_label_sort_drop(a.ids, a.B, a.N, a.K, ws, status, s, &o, a.dT, fill);
  if (e != cudaSuccess) return e;
  float *parts = (float *)((char *)ws + al256(label_sort_bytes(rows, Ktot, a.B, true)));
  const int R = grad_rows_R(rows, a.D * (int)dtype_size(a.dt)), none = (int)Ktot, n = (int)rows;
  if (a.dt == kF32) launch_grad_from<float>(a, o, n, none, R, parts, s);
  else if (a.dt == kF16) launch_grad_from<__half>(a, o, n, none, R, parts, s);
  else launch_grad_from<__nv_bfloat16>(a, o, n, none, R, parts, s);
  const int nchunks = (n + R - 1) / R;
  count_launches(1);
  if (nchunks == 1) return cudaGetLastError();  // no segment runs past a chunk
  launch_chained(grad_join_kernel, dim3((nchunks + 31) / 32, (a.D + kJoinCols - 1) / kJoinCols), dim3(1024), 0, s,
                 o.skeys, n, none, R, a.D, parts, a.scale, a.dT, (int)a.dt_t, a.accumulate);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace fk
