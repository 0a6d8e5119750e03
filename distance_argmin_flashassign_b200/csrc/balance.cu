// balance.cu -- balance loss of rows routed to columns (experts, codes), with
// the per-column counts, and its gradient.
//
// For the n rows of a problem that take part (mask not 0, some logit above
// -inf), with M chosen columns each:
//   lse_i = ln sum_e exp z_ie      p_ie = exp(z_ie - lse_i)
//   P_e = (1/n) sum_i p_ie         f_e = count_e / (M n)
//   loss = coef E sum_e f_e P_e
//   dz_ie = g coef E / n  p_ie (f_e - sum_j f_j p_ij)
// One pass over the logits forward, one backward.  A row belongs to a team of
// lanes that hold its columns in registers; a warp (for long rows the block)
// is the owner of a run of rows, whose logits come to it through a ring of
// tiles in shared memory.  Forward, a team adds its rows' probabilities to
// column sums that its lanes keep in registers over all of their rows; blocks
// leave their sums in partial rows that a second small kernel adds in block
// order.  Counts are integers, so the shared-memory atomics that make them do
// not change the result.
//
// What bounds it (B200; shares of the HBM copy rate of 6,466 GB/s, whole calls
// back to back).  Forward, latency: with 16 warps an SM (some 120 registers) and
// chains of dependent operations per row (the maximum and its exchange, two
// exponentials, the sum's exchange) no unit is full: at 64 columns DRAM 28 %, issue
// slots 58 %, special-function unit 32 %; at 1,024 55 % each.  A bf16 logit takes
// 8 to 12 instructions with its share of the row's and the tile's.
//   16 x 32,768 x 64 bf16  31 us, 0.37     1 M x 128 bf16     80 us, 0.54
//   262,144 x 1,024 fp16  127 us, 0.65     65,536 x 2,048 bf16  93 us, 0.45
//   262,144 x 258 bf16     72 us, 0.30     32,768 x 8,192 bf16 227 us, 0.37
//   262,144 x 256 fp32     65 us, 0.66     100,003 x 515 fp32   61 us, 0.53
// Backward, HBM where rows are whole 16-byte pieces and there are enough of them,
// else 2- and 4-byte shared-memory accesses; at 64 columns latency again (DRAM
// 36 %, issue slots 54 %):
//   16 x 32,768 x 64 bf16  28 us, 0.76     1 M x 128 bf16    105 us, 0.80
//   262,144 x 1,024 fp16  205 us, 0.81     65,536 x 2,048 bf16 106 us, 0.78
//   262,144 x 258 bf16     80 us, 0.53     32,768 x 8,192 bf16 206 us, 0.81
//   262,144 x 256 fp32     97 us, 0.86     100,003 x 515 fp32   84 us, 0.76
// Pairs of fp32 operations in one instruction are worth 5 % of the forward pass.
//
// Rounding: everything is fp32 (blocks are joined in fp64).  2^x and 1/x are the
// approximate instructions, 2^-22 and 2^-23 of the result: as much as the
// rounded products before them cost, and one issue slot in place of several.  A
// lane adds at most 1,024 rows' probabilities into one fp32 sum, 2^-14 of it
// at worst; fp64 sums would hold twice the registers at 1/64 of the rate.
#include <atomic>
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
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 operations an instruction (a logit costs an unpack, half a maximum,
// half a product and sum each, and one ex2).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float warp_max(float v) {  // ignores NaN
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <typename T> constexpr bool kIsHalf = std::is_same<T, __half>::value;
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kIsHalf<T>) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float2 v) {
  uint32_t w;
  if constexpr (kIsHalf<T>) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    memcpy(&w, &h, 4);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    memcpy(&w, &h, 4);
  }
  return w;
}
template <typename T> __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // ignores NaN
  uint32_t w;
  if constexpr (kIsHalf<T>) asm("max.f16x2 %0, %1, %2;" : "=r"(w) : "r"(a), "r"(b));
  else asm("max.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(a), "r"(b));
  return w;
}

// The columns a lane holds of one row: P packs of VL consecutive elements (a
// whole 16 bytes, two of 16 bits, or a single element), as they lie in memory.
// A row of which nothing is looked at, and columns past E, count as -inf.
template <typename T, int VL, int P> struct Lane {
  static constexpr int NE = VL * P, NP = (NE + 1) / 2;  // columns, pairs of them
  static constexpr bool kWords = VL > 1 && sizeof(T) == 2;
  static constexpr int W = VL * (int)sizeof(T) / 4;  // 32-bit words of a pack
  uint32_t w[VL > 1 ? P * W : 1];
  float e[VL > 1 ? 1 : P];
  // p-th pack from column c of `row` in shared memory
  __device__ __forceinline__ void load(int p, const T *row, int c, bool ok) {
    if constexpr (VL == 1) {
      e[p] = ok ? to_f32<T>(row[c]) : neg_inf();
    } else {
      const uint32_t n = sizeof(T) == 4 ? 0xff800000u : kIsHalf<T> ? 0xfc00fc00u : 0xff80ff80u;
      if constexpr (W == 4) {
        uint4 v = make_uint4(n, n, n, n);
        if (ok) v = *reinterpret_cast<const uint4 *>(row + c);
        w[4 * p] = v.x;
        w[4 * p + 1] = v.y;
        w[4 * p + 2] = v.z;
        w[4 * p + 3] = v.w;
      } else {
        static_assert(W == 1, "whole 16-byte packs or pairs of 16 bits");
        w[p] = ok ? *reinterpret_cast<const uint32_t *>(row + c) : n;
      }
    }
  }
  __device__ __forceinline__ float max() const {
    float m = neg_inf();
    if constexpr (kWords) {
      uint32_t t = w[0];
#pragma unroll
      for (int i = 1; i < P * W; ++i) t = max2<T>(t, w[i]);
      const float2 f = unpack2<T>(t);
      m = fmaxf(m, fmaxf(f.x, f.y));
    } else {
      float2 z[NP];
      values(z);
#pragma unroll
      for (int i = 0; i < NP; ++i) m = fmaxf(m, fmaxf(z[i].x, z[i].y));
    }
    return m;
  }
  __device__ __forceinline__ void values(float2 *z) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (VL == 1) z[i] = make_float2(e[2 * i], 2 * i + 1 < P ? e[2 * i + 1] : neg_inf());
      else if constexpr (sizeof(T) == 4) z[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else z[i] = unpack2<T>(w[i]);
    }
  }
  // stores the p-th pack of z, or zeros, from column c of `row`
  __device__ __forceinline__ static void store(int p, const float2 *z, bool zero, T *row, int c) {
    if constexpr (VL == 1) {
      const float v = p & 1 ? z[p / 2].y : z[p / 2].x;
      row[c] = from_f32<T>(zero ? 0.f : v);
    } else if constexpr (W == 1) {
      *reinterpret_cast<uint32_t *>(row + c) = zero ? 0u : pack2<T>(z[p]);
    } else {
      uint4 o;
      if constexpr (sizeof(T) == 4) {
        o = make_uint4(__float_as_uint(z[2 * p].x), __float_as_uint(z[2 * p].y), __float_as_uint(z[2 * p + 1].x),
                       __float_as_uint(z[2 * p + 1].y));
      } else {
        o = make_uint4(pack2<T>(z[4 * p]), pack2<T>(z[4 * p + 1]), pack2<T>(z[4 * p + 2]), pack2<T>(z[4 * p + 3]));
      }
      if (zero) o = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(row + c) = o;
    }
  }
};

constexpr int kMaxSmem = 220 * 1024;  // of a block of these kernels, beside some 1 KB of static shared memory
constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;
constexpr int kBalLane = 32, kBalSome = 16;  // columns a lane holds at most, and where a warp has lanes to spare
// Lanes of a team, as a power of two, where the kernel is compiled for them:
constexpr int kWide = 6;      // from here on (64, 128, 256) several warps
constexpr int kAnyTeam = -1;  // up to a warp, known at run time

// Blocks that fit an SM next to a lane's columns in registers (three with 16
// or more columns a lane spill: 1 M x 128 bf16 100 us against 81 with two, 131,072 x
// 1,024 112 against 82).  With two, 28 of the 233 kernels still spill 12 to 64
// bytes, all of them single-element ones, with 28 or 32 columns a lane but for one.
constexpr int bal_blocks(int NE) { return NE <= 8 ? 3 : 2; }
template <int NE> constexpr int kBalBlocks = bal_blocks(NE);
// Rows a team works on at a time, so that one row's exchanges between lanes
// are not waited for alone (1 M x 128 bf16: 81 us, 89 with one).
constexpr int bal_rows(int NE) { return NE <= 16 ? 2 : 1; }
template <int NE> constexpr int kBalRows = bal_rows(NE);

// Rows go tile by tile to owners: a warp, whose G = 2^logg-lane teams take
// one row each, or for long rows (WIDE) two, four or eight warps as one team.
// Lane l of a team holds the packs l, l + G, l + 2G, ... of VL columns each.
template <int LOGG> struct Owner {
  static constexpr bool WIDE = LOGG >= kWide;
  static constexpr int kThreads = WIDE ? 1 << LOGG : 32, kWarps = kThreads / 32, kCount = kBalThreads / kThreads;
  int index;           // among the owners of the block
  int lane, row0, rows;  // lane in the team, the team's first row of a step, rows of a step
  int thread;
  __device__ __forceinline__ explicit Owner(int logg) {
    index = threadIdx.x / kThreads;
    thread = threadIdx.x % kThreads;
    lane = WIDE ? thread : threadIdx.x & ((1 << logg) - 1);
    row0 = WIDE ? 0 : (threadIdx.x & 31) >> logg;
    rows = WIDE ? 1 : 32 >> logg;
  }
  // (the warps are reconverged first and the barriers' per-thread forms are used)
  __device__ __forceinline__ void sync() const {
    __syncwarp();
    if constexpr (kThreads == kBalThreads) __syncthreads();
    else if constexpr (WIDE) asm volatile("barrier.sync %0, %1;" ::"r"(1 + index), "n"(kThreads) : "memory");
  }
  // sync, and whether any of the owner's threads says so
  __device__ __forceinline__ bool any(bool v) const {
    __syncwarp();
    if constexpr (kThreads == kBalThreads) {
      return __syncthreads_or(v) != 0;
    } else if constexpr (WIDE) {
      int r;
      asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.red.or.pred q, %2, %3, p;\n\t"
                   "selp.s32 %0, 1, 0, q;\n\t}"
                   : "=r"(r)
                   : "r"((int)v), "r"(1 + index), "n"(kThreads)
                   : "memory");
      return r != 0;
    } else {
      return __any_sync(0xffffffffu, v) != 0;
    }
  }
};

// ------------------------------------------------------------ row tiles ---
// Rows are consecutive in memory, so a tile of them is one range of bytes of
// each array.  One thread of an owner copies the ranges of a tile into its place
// in shared memory with bulk copies, a few tiles ahead of the owner's work: no
// registers wait for memory, and rows of any length and alignment arrive at the
// full rate.  A bulk copy moves whole aligned 16-byte pieces: a range is widened
// to them (its data then starts (address mod 16) bytes into its place), except
// at the very ends of the array, where what the pieces inside it leave is
// copied byte by byte.
struct Span {
  const char *lo;  // the whole pieces
  uint32_t bytes;
};
// The pieces of [a, a + n), which lies inside the array: with neighbours on
// both sides every piece that the range touches belongs to the array.
__device__ __forceinline__ Span span_inside(const char *a, uint32_t n) {
  const uint32_t skew = (uint32_t)(uintptr_t)a & 15;
  return {a - skew, (skew + n + 15) & ~15u};
}
// The same at the ends of the array [base, base + total): only whole pieces of
// it, and the bytes of the range that they do not cover copied to dst (the
// place of a's own piece).
__device__ __noinline__ Span span_at_ends(const char *a, uint32_t n, const char *base, size_t total, char *dst) {
  const char *from = (const char *)((uintptr_t)a & ~(uintptr_t)15), *end = a + n;
  const char *lo = from < base ? from + 16 : from;
  const char *hi = (const char *)(((uintptr_t)end + 15) & ~(uintptr_t)15);
  if (hi > base + total) hi -= 16;
  if (hi < lo) hi = lo;
  for (const char *q = a; q < end && q < lo; ++q) dst[q - from] = *q;
  for (const char *q = hi < a ? a : hi; q < end; ++q) dst[q - from] = *q;
  // the thread's next bulk copy into this place must not overtake these bytes
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return {lo, (uint32_t)(hi - lo)};
}
__device__ __forceinline__ void bulk_copy(const Span &v, const char *a, char *dst, uint32_t bar) {
  if (v.bytes == 0) return;
  const char *from = (const char *)((uintptr_t)a & ~(uintptr_t)15);
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst + (v.lo - from))),
               "l"(v.lo), "r"(v.bytes), "r"(bar)
               : "memory");
}
// Rows [r, r + n) of an array of `all` rows of `width` bytes into `dst`; the
// bytes of whole pieces are returned, to be expected by the barrier, and are
// copied by bulk_copy.
__device__ __forceinline__ Span span_of(const char *base, uint32_t width, size_t r, uint32_t n, size_t all, char *dst) {
  const char *a = base + r * width;
  // 16 rows hold at least 16 bytes
  if (r >= 16 && r + n + 16 <= all) return span_inside(a, n * width);
  return span_at_ends(a, n * width, base, all * width, dst);
}

// An owner has a run of consecutive rows.  Their logits pass through a ring of
// `stages` tiles of `rows` rows; what is small a row (labels or lse, mask)
// comes in batches of `batch` rows, whole tiles of at least 32 rows where the
// owner has them, in two places in turn, so that what is done once a row has a
// thread for each.  Places in bytes, whole 16-byte pieces.
struct Plan {
  int share;               // rows of an owner
  int rows, stages, z;     // of a tile; tiles; bytes of a tile's place
  int batch, mid, small;   // rows of a batch; bytes of its places
  __host__ __device__ int stats() const { return (batch * 8 + 15) / 16 * 16; }  // the rows' maxima and sums
  __host__ __device__ int bytes() const { return stages * z + 2 * (mid + small) + stats(); }
};
constexpr int kMaxStages = 4;
struct Bars {
  uint64_t tile[kMaxStages], side[2];
};
struct Rows {
  const char *Z, *mid, *small;
  uint32_t zrow, midrow;  // bytes of a row (small: 1)
  size_t all;             // rows of the arrays
  size_t first;           // the owner's first row in them
  int n, ntiles, nbatches;
  char *place;
  Bars *bar;
  Plan pl;
  __device__ __forceinline__ char *tile_at(int s) const { return place + s * pl.z; }
  __device__ __forceinline__ char *mid_at(int s) const { return place + pl.stages * pl.z + s * (pl.mid + pl.small); }
  __device__ __forceinline__ char *small_at(int s) const { return mid_at(s) + pl.mid; }
  __device__ __forceinline__ float2 *stats() const { return reinterpret_cast<float2 *>(mid_at(2)); }
  // where the data of a row lies in its array's place, from the row's own address
  __device__ __forceinline__ static uint32_t skew(const char *base, uint32_t width, size_t r) {
    return ((uint32_t)(uintptr_t)base + (uint32_t)r * width) & 15;
  }
  __device__ __forceinline__ int tile_rows(int k) const { return min(pl.rows, n - k * pl.rows); }
  __device__ __forceinline__ int batch_rows(int k) const { return min(pl.batch, n - k * pl.batch); }
  // one thread: tile k into ring place s; batch k into place s
  __device__ __forceinline__ void issue_tile(int k, int s) const {
    const size_t r = first + (size_t)(k * pl.rows);
    const uint32_t b = smem_u32(&bar->tile[s]);
    const Span v = span_of(Z, zrow, r, tile_rows(k), all, tile_at(s));
    mbar_arrive_expect_tx(b, v.bytes);
    bulk_copy(v, Z + r * zrow, tile_at(s), b);
  }
  __device__ __forceinline__ void issue_batch(int k, int s) const {
    const size_t r = first + (size_t)(k * pl.batch);
    const uint32_t b = smem_u32(&bar->side[s]), c = batch_rows(k);
    const Span v = span_of(mid, midrow, r, c, all, mid_at(s));
    Span m = {nullptr, 0};
    if (small) m = span_of(small, 1, r, c, all, small_at(s));
    mbar_arrive_expect_tx(b, v.bytes + m.bytes);
    bulk_copy(v, mid + r * midrow, mid_at(s), b);
    if (small) bulk_copy(m, small + r, small_at(s), b);
  }
  __device__ __forceinline__ void start() const {
    for (int i = 0; i < 2 && i < nbatches; ++i) issue_batch(i, i);
    for (int i = 0; i < pl.stages && i < ntiles; ++i) issue_tile(i, i);
  }
  // After a wait that ran out at batch kb, tile kt: let the copies in flight
  // land, within a second each.
  __device__ __forceinline__ void drain(int kb, int kt) const {
    for (int i = kb; i < kb + 2 && i < nbatches; ++i)
      mbar_wait_for(smem_u32(&bar->side[i & 1]), i >> 1 & 1, 1000000000ull);
    for (int i = kt; i < kt + pl.stages && i < ntiles; ++i)
      mbar_wait_for(smem_u32(&bar->tile[i % pl.stages]), i / pl.stages & 1, 1000000000ull);
  }
};

// The calling thread's owner: its rows of problem b and its places, with the
// barriers set up (visible after the block's next barrier).
template <int LOGG>
__device__ __forceinline__ Rows owned(const Owner<LOGG> &t, const Plan &pl, Bars *bar, char *smem, int b, int B,
                                            int N) {
  Rows v;
  const long long from = ((long long)blockIdx.x * t.kCount + t.index) * pl.share;
  v.n = from < N ? (int)min((long long)pl.share, N - from) : 0;
  v.first = (size_t)b * N + from;
  v.all = (size_t)B * N;
  v.ntiles = (v.n + pl.rows - 1) / pl.rows;
  v.nbatches = (v.n + pl.batch - 1) / pl.batch;
  v.place = smem + t.index * pl.bytes();
  v.bar = bar;
  v.pl = pl;
  if (t.thread == 0) {
    for (int i = 0; i < pl.stages; ++i) mbar_init(smem_u32(&bar->tile[i]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&bar->side[i]), 1);
    fence_mbar_init();
  }
  return v;
}

// Sum over the block of one double a thread, in a fixed order, to thread 0.
template <int WARPS> __device__ __forceinline__ double block_sum(double v, double *part) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double sum = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < WARPS; ++i) sum += part[i];
  return sum;
}

struct BalanceOut {
  float *loss;
  int32_t *counts, *tokens;
  float *meanp;
  float coef;
};
// Column e of problem b: its probability sum p and count c of the n rows; returns p / n * c.
__device__ __forceinline__ double put_column(const BalanceOut &o, int b, int E, int e, double p, int c, int n) {
  if (n > 0) p /= (double)n;
  o.counts[(size_t)b * E + e] = c;
  if (o.meanp) o.meanp[(size_t)b * E + e] = (float)p;
  return p * (double)c;
}
__device__ __forceinline__ void put_loss(const BalanceOut &o, int b, int E, int M, double sum, int n) {
  o.loss[b] = n > 0 ? (float)((double)o.coef * E * sum / ((double)M * n)) : 0.f;
  o.tokens[b] = n;
}

// With one block a problem the block writes the results itself; with more
// they leave partial rows for balance_join_kernel.
template <typename T, int VL, int P, int LOGG>
__global__ void __launch_bounds__(kBalThreads, kBalBlocks<VL * P>)
    balance_rows_kernel(const T *__restrict__ Z, const int32_t *__restrict__ ids, const uint8_t *__restrict__ mask,
                        int B, int N, int E, int M, int logg_, Plan pl, float *__restrict__ lse,
                        float *__restrict__ psum, int *__restrict__ csum, int *__restrict__ tsum, BalanceOut out,
                        DevCtl ctl) {
  constexpr bool WIDE = LOGG >= kWide;
  using L = Lane<T, VL, P>;
  constexpr int NE = L::NE, NP = L::NP, U = kBalRows<NE>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(8) Bars bars[Owner<LOGG>::kCount];
  __shared__ float wm[2][U][kBalWarps], wsum[2][U][kBalWarps];
  __shared__ int taken[kBalWarps], abort_flag;
  __shared__ double part[kBalWarps];
  const int logg = LOGG >= 0 ? LOGG : logg_;
  const Owner<LOGG> t(logg);
  const int b = blockIdx.y, G = 1 << logg;
  // the chosen columns of the block's rows [E], then the owners' places, where
  // the block's column sums [E] lie once the rows are done
  int *hist = reinterpret_cast<int *>(smem);
  char *places = smem + (E * 4 + 15) / 16 * 16;
  float *cols = reinterpret_cast<float *>(places);
  Rows v = owned(t, pl, &bars[t.index], places, b, B, N);
  v.Z = (const char *)Z;
  v.mid = (const char *)ids;
  v.small = (const char *)mask;
  v.zrow = (uint32_t)(E * sizeof(T));
  v.midrow = (uint32_t)M * 4;
  if (threadIdx.x == 0) abort_flag = 0;
  for (int e = threadIdx.x; e < E; e += kBalThreads) hist[e] = 0;
  __syncthreads();
  wait_prior_grid();
  if (t.thread == 0) v.start();

  float2 acc[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) acc[i] = both(0.f);
  int mytok = 0, buf = 0, at = 0, phase = 0, kt = 0, kb = 0;
  bool bad = false, gave_up = false;
  float2 *stat = v.stats();
  for (; kb < v.nbatches && !gave_up; ++kb) {
    mbar_wait(smem_u32(&v.bar->side[kb & 1]), kb >> 1 & 1, &abort_flag, ctl);
    const size_t rb = v.first + (size_t)kb * pl.batch;  // the batch's first row
    const int nrows = v.batch_rows(kb);
    const int *cs = reinterpret_cast<const int *>(v.mid_at(kb & 1) + v.skew(v.mid, v.midrow, rb));
    const uint8_t *ms = reinterpret_cast<const uint8_t *>(v.small_at(kb & 1) + v.skew(v.small, 1, rb));
    for (int in_batch = 0; in_batch < nrows; in_batch += pl.rows, ++kt) {
      mbar_wait(smem_u32(&v.bar->tile[at]), phase, &abort_flag, ctl);
      const int n = v.tile_rows(kt);
      const T *zs = reinterpret_cast<const T *>(v.tile_at(at) + v.skew(v.Z, v.zrow, v.first + (size_t)(kt * pl.rows)));
      // every team a row: probabilities into the column sums, maximum and sum kept
      for (int s0 = 0; s0 < n; s0 += U * t.rows) {
        L x[U];
        float own[U], off[U], m[U], s[U], sum[U];
        float2 z[U][NP];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = s0 + u * t.rows + t.row0;
          const bool live = r < n && (!mask || ms[in_batch + r] != 0);
          const T *row = zs + r * E;
#pragma unroll
          for (int p = 0; p < P; ++p) x[u].load(p, row, (p * G + t.lane) * VL, live && (p * G + t.lane) * VL < E);
          own[u] = m[u] = x[u].max();
        }
        // each lane's exponentials are of its own maximum, so that they need not
        // wait for the team's; a lane or team without a logit above -inf takes 0
        // for its maximum: its sum is 0 (or NaN)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (own[u] == neg_inf()) own[u] = 0.f;
          x[u].values(z[u]);
          float top = own[u];
          // a large maximum (a lane of masked columns): the rounding of its product
          // with log2(e) would be no small exponent any more
          if (!kIsHalf<T> && fabsf(top) > 65536.f) {
#pragma unroll
            for (int i = 0; i < NP; ++i) z[u][i] = add2(z[u][i], both(-top));
            top = 0.f;
          }
          float2 ss = both(0.f);
          const float2 shift = both(-top * kLog2e);
          off[u] = fmaf(top, kLog2e, shift.x);  // the shift's rounding, which the lane's exponentials share
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            z[u][i] = fma2(z[u][i], both(kLog2e), shift);
            z[u][i].x = exp2_fast(z[u][i].x);
            z[u][i].y = exp2_fast(z[u][i].y);
            ss = add2(ss, z[u][i]);
          }
          s[u] = ss.x + ss.y;
        }
        if constexpr (WIDE || LOGG == 5) {
#pragma unroll
          for (int u = 0; u < U; ++u) m[u] = warp_max(m[u]);
        } else {
#pragma unroll
          for (int o = G >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
        }
        float w[U];  // exp(own - m), less that rounding: the lane's sum and probabilities on the team's scale
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (m[u] == neg_inf()) m[u] = 0.f;
          w[u] = s[u] == 0.f ? 0.f : exp2_fast(fmaf(own[u] - m[u], kLog2e, -off[u]));
          s[u] *= w[u];
        }
#pragma unroll
        for (int o = WIDE ? 16 : G >> 1; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
        if (WIDE) {
          // one exchange of the warps' maxima and sums
          if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              wm[buf][u][threadIdx.x >> 5] = s[u] == 0.f ? neg_inf() : m[u];
              wsum[buf][u][threadIdx.x >> 5] = s[u];
            }
          t.sync();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = s0 + u * t.rows + t.row0;
          float factor;  // p_e = z_e w factor
          if (WIDE) {
            // lane l looks at the owner's warp l % kWarps
            constexpr int KW = Owner<LOGG>::kWarps;
            const int look = t.index * KW + threadIdx.x % KW;
            const float mw = wm[buf][u][look], sw = wsum[buf][u][look];
            float top = mw;
#pragma unroll
            for (int o = KW / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top == neg_inf()) top = 0.f;
            sum[u] = sw == 0.f ? 0.f : sw * exp2_fast((mw - top) * kLog2e);
#pragma unroll
            for (int o = KW / 2; o > 0; o >>= 1) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
            // NaN in every warp of a NaN row, 0 in every warp of a row left out
            factor = sum[u] == 0.f ? 0.f : (s[u] == 0.f ? 0.f : exp2_fast((m[u] - top) * kLog2e)) * rcp_fast(sum[u]);
            m[u] = top;
          } else {
            sum[u] = s[u];
            factor = sum[u] == 0.f ? 0.f : rcp_fast(sum[u]);
          }
#pragma unroll
          for (int i = 0; i < NP; ++i) acc[i] = fma2(z[u][i], both(w[u] * factor), acc[i]);
          if (t.lane == 0 && r < n) stat[in_batch + r] = make_float2(m[u], sum[u]);
        }
        buf ^= 1;
      }
      gave_up = t.any(*(volatile int *)&abort_flag);  // the tile has been read
      if (gave_up) break;
      if (t.thread == 0 && kt + pl.stages < v.ntiles) v.issue_tile(kt + pl.stages, at);
      if (++at == pl.stages) {
        at = 0;
        phase ^= 1;
      }
    }
    if (gave_up) break;
    // every thread a row: what is done once for each
    for (int r = t.thread; r < nrows; r += t.kThreads) {
      const float2 w = stat[r];
      const bool on = w.y != 0.f;  // a masked row has no sum either
      mytok += on;
      if (lse) lse[rb + r] = on ? w.x + logf(w.y) : __int_as_float(0x7f800000);
      if (on)
        for (int j = 0; j < M; ++j) {
          const int id = cs[r * M + j];
          if ((unsigned)id < (unsigned)E) atomicAdd(hist + id, 1);
          else bad |= id != -1;
        }
    }
    t.sync();  // the batch has been read
    if (t.thread == 0 && kb + 2 < v.nbatches) v.issue_batch(kb + 2, kb & 1);
  }
  if (gave_up && t.thread == 0) v.drain(kb, kt);
  if (bad) record_status(ctl.status, kStBadLabel);
  // column sums: over the teams of a warp, then over the owners in order
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kBalThreads) cols[e] = 0.f;
  __syncthreads();
  float sums[2 * NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    sums[2 * i] = acc[i].x;
    sums[2 * i + 1] = acc[i].y;
  }
  if (!WIDE)
#pragma unroll
    for (int o = G; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < NE; ++i) sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], o);
  for (int w = 0; w < t.kCount; ++w) {
    if (t.index == w && (WIDE || (int)(threadIdx.x & 31) < G)) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int c = (i / VL * G + t.lane) * VL + i % VL;
        if (c < E) cols[c] += sums[i];
      }
    }
    __syncthreads();
  }
  for (int o = 16; o > 0; o >>= 1) mytok += __shfl_xor_sync(0xffffffffu, mytok, o);
  if ((threadIdx.x & 31) == 0) taken[threadIdx.x >> 5] = mytok;
  __syncthreads();
  int ntok = 0;
#pragma unroll
  for (int w = 0; w < kBalWarps; ++w) ntok += taken[w];
  if (gridDim.x == 1) {
    double mine = 0.0;
    for (int e = threadIdx.x; e < E; e += kBalThreads) mine += put_column(out, b, E, e, cols[e], hist[e], ntok);
    const double sum = block_sum<kBalWarps>(mine, part);
    if (threadIdx.x == 0) put_loss(out, b, E, M, sum, ntok);
    return;
  }
  const size_t row = (size_t)b * gridDim.x + blockIdx.x;
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    psum[row * E + e] = cols[e];
    csum[row * E + e] = hist[e];
  }
  if (threadIdx.x == 0) tsum[row] = ntok;
}

// Adds the blocks' partial rows in block order, in fp64.  The CTAs of a
// cluster share a problem's columns and hand their parts of the loss to the
// first one through its shared memory; in a CTA, groups of threads share a
// column's partial rows.
constexpr int kJoinThreads = 1024, kJoinCluster = 8;
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(const float *__restrict__ psum,
                                                                    const int *__restrict__ csum,
                                                                    const int *__restrict__ tsum, int nparts, int E,
                                                                    int M, BalanceOut out) {
  __shared__ double part[kJoinThreads / 32], psub[kJoinThreads], shares[kJoinCluster];
  __shared__ int csub[kJoinThreads], ntok[kJoinThreads / 32];
  const int b = blockIdx.y, lane = threadIdx.x & 31, w = threadIdx.x >> 5, tid = threadIdx.x;
  const int ncta = gridDim.x, rank = blockIdx.x;
  if (ncta > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  wait_prior_grid();
  int n = 0;
  for (int q = tid; q < nparts; q += kJoinThreads) n += tsum[(size_t)b * nparts + q];
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) ntok[w] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) n += ntok[i];
  const int per = (E + ncta - 1) / ncta, e0 = rank * per, e1 = min(E, e0 + per);
  int tx = 32;  // columns at a time
  while (tx < per && tx < kJoinThreads) tx *= 2;
  const int ty = kJoinThreads / tx, g = tid / tx;
  double mine = 0.0;
  for (int base = e0; base < e1; base += tx) {
    const int e = base + tid % tx;
    double p = 0.0;
    int c = 0;
    if (e < e1) {
      const float *ps = psum + (size_t)b * nparts * E + e;
      const int *cs = csum + (size_t)b * nparts * E + e;
#pragma unroll 8
      for (int q = g; q < nparts; q += ty) {
        p += (double)ps[(size_t)q * E];
        c += cs[(size_t)q * E];
      }
    }
    psub[tid] = p;
    csub[tid] = c;
    __syncthreads();
    if (g == 0 && e < e1) {
      for (int i = 1; i < ty; ++i) {
        p += psub[i * tx + tid];
        c += csub[i * tx + tid];
      }
      mine += put_column(out, b, E, e, p, c, n);
    }
    __syncthreads();
  }
  const double sum = block_sum<kJoinThreads / 32>(mine, part);
  if (ncta == 1) {
    if (tid == 0) put_loss(out, b, E, M, sum, n);
    return;
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // the first CTA has started
  if (tid == 0) {
    uint32_t dst;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_u32(&shares[rank])));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(dst), "d"(sum) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (rank == 0 && tid == 0) {
    double all = 0.0;
    for (int i = 0; i < ncta; ++i) all += shares[i];
    put_loss(out, b, E, M, all, n);
  }
}

// A row's lse is an fp32 number, so exp(z - lse) is off by up to |lse| 2^-24 of
// itself: 2^-18 at the border here.  Far from 0 it is not a probability at all
// (a row filled with -1e9 has the lse -1e9, and exp(z - lse) = 1 in every
// column): such rows are normalised again.  The question, asked at each step
// (by rows of several warps once a batch of rows), costs 0 to 2 % (16 x 32,768 x 64
// bf16 27.2 us before, 27.7 with it; asked once a batch there too 29.0).
__device__ __forceinline__ bool far_lse(float l) {
  return fabsf(l) > 64.f && l != __int_as_float(0x7f800000);  // +inf: a row that takes no part
}

template <typename T, int VL, int P, int LOGG>
__global__ void __launch_bounds__(kBalThreads, kBalBlocks<VL * P>)
    balance_grad_kernel(const T *Z, const int32_t *__restrict__ counts, const int32_t *__restrict__ tokens,
                        const float *__restrict__ lse, const float *__restrict__ gloss, int B, int N, int E, int M,
                        float coef, int logg_, Plan pl, T *dZ, DevCtl ctl) {
  constexpr bool WIDE = LOGG >= kWide;
  using L = Lane<T, VL, P>;
  constexpr int NE = L::NE, NP = L::NP, U = kBalRows<NE>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(8) Bars bars[Owner<LOGG>::kCount];
  __shared__ float wdot[2][U][kBalWarps], wnorm[U][kBalWarps];
  __shared__ int abort_flag;
  const float inf = __int_as_float(0x7f800000);
  const int logg = LOGG >= 0 ? LOGG : logg_;
  const Owner<LOGG> t(logg);
  const int b = blockIdx.y, G = 1 << logg;
  Rows v = owned(t, pl, &bars[t.index], smem, b, B, N);
  v.Z = (const char *)Z;
  v.mid = (const char *)lse;
  v.small = nullptr;
  v.zrow = (uint32_t)(E * sizeof(T));
  v.midrow = 4;
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  wait_prior_grid();
  if (t.thread == 0) v.start();

  const int ntok = tokens[b] > 0 ? tokens[b] : 1;
  const float k = (gloss ? gloss[b] : 1.f) * (coef * (float)E / (float)ntok);
  float2 kf[NP];  // k f of the lane's columns
#pragma unroll
  for (int i = 0; i < 2 * NP; ++i) {
    const int c = (i / VL * G + t.lane) * VL + i % VL;
    const float v = i < NE && c < E ? k * ((float)counts[(size_t)b * E + c] / ((float)M * (float)ntok)) : 0.f;
    if (i & 1) kf[i / 2].y = v;
    else kf[i / 2].x = v;
  }
  int buf = 0, at = 0, phase = 0, kt = 0, kb = 0;
  bool gave_up = false;
  for (; kb < v.nbatches && !gave_up; ++kb) {
    mbar_wait(smem_u32(&v.bar->side[kb & 1]), kb >> 1 & 1, &abort_flag, ctl);
    const size_t rb = v.first + (size_t)kb * pl.batch;  // the batch's first row
    const int nrows = v.batch_rows(kb);
    const float *ls = reinterpret_cast<const float *>(v.mid_at(kb & 1) + v.skew(v.mid, 4, rb));
    // WIDE: whether some row of the batch is far, by a vote of the owner's threads,
    // so that all of them come to the norms' barrier or none does, even where the
    // wait above has run out and the copy lands while they read
    bool far_batch = false;
    if (WIDE) {
      for (int r = t.thread; r < nrows; r += t.kThreads) far_batch |= far_lse(ls[r]);
      far_batch = t.any(far_batch);
    }
    for (int in_batch = 0; in_batch < nrows; in_batch += pl.rows, ++kt) {
      mbar_wait(smem_u32(&v.bar->tile[at]), phase, &abort_flag, ctl);
      const int n = v.tile_rows(kt);
      const size_t r0 = rb + in_batch;
      const T *zs = reinterpret_cast<const T *>(v.tile_at(at) + v.skew(v.Z, v.zrow, r0));
      for (int s0 = 0; s0 < n; s0 += U * t.rows) {
        L x[U];
        float2 z[U][NP];
        float l[U], dot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = s0 + u * t.rows + t.row0;
          l[u] = r < n ? ls[in_batch + r] : inf;
          const T *row = zs + r * E;
#pragma unroll
          for (int p = 0; p < P; ++p) x[u].load(p, row, (p * G + t.lane) * VL, l[u] != inf && (p * G + t.lane) * VL < E);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[u].values(z[u]);
          float2 dd = both(0.f);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            // the difference first: a logit that is the row's whole sum has
            // probability 1 exactly, and so no gradient; past E -inf: 0
            z[u][i] = mul2(add2(z[u][i], both(-l[u])), both(kLog2e));
            z[u][i].x = exp2_fast(z[u][i].x);
            z[u][i].y = exp2_fast(z[u][i].y);
            dd = fma2(kf[i], z[u][i], dd);
          }
          dot[u] = dd.x + dd.y;
        }
#pragma unroll
        for (int o = WIDE ? 16 : G >> 1; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
        bool far = far_batch;
        if (!WIDE) {
#pragma unroll
          for (int u = 0; u < U; ++u) far |= far_lse(l[u]);
          far = __any_sync(0xffffffffu, far) != 0;
        }
        if (far) {
          // such a row's probabilities add up to some other number than 1: they and
          // the dot product of them are divided by it
          float norm[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float2 ss = both(0.f);
#pragma unroll
            for (int i = 0; i < NP; ++i) ss = add2(ss, z[u][i]);
            norm[u] = ss.x + ss.y;
          }
#pragma unroll
          for (int o = WIDE ? 16 : G >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) norm[u] += __shfl_xor_sync(0xffffffffu, norm[u], o);
          if (WIDE) {  // read before the exchange below, written again after it
            if ((threadIdx.x & 31) == 0)
#pragma unroll
              for (int u = 0; u < U; ++u) wnorm[u][threadIdx.x >> 5] = norm[u];
            t.sync();
#pragma unroll
            for (int u = 0; u < U; ++u) {
              norm[u] = 0.f;
#pragma unroll
              for (int w = 0; w < t.kWarps; ++w) norm[u] += wnorm[u][t.index * t.kWarps + w];
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float f = far_lse(l[u]) ? rcp_fast(norm[u]) : 1.f;
            dot[u] *= f;
#pragma unroll
            for (int i = 0; i < NP; ++i) z[u][i] = mul2(z[u][i], both(f));
          }
        }
        if (WIDE) {
          if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) wdot[buf][u][threadIdx.x >> 5] = dot[u];
          t.sync();
#pragma unroll
          for (int u = 0; u < U; ++u) {
            dot[u] = 0.f;
#pragma unroll
            for (int w = 0; w < t.kWarps; ++w) dot[u] += wdot[buf][u][t.index * t.kWarps + w];
          }
          buf ^= 1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = s0 + u * t.rows + t.row0;
#pragma unroll
          for (int i = 0; i < NP; ++i) z[u][i] = mul2(z[u][i], add2(kf[i], both(-dot[u])));
          T *row = dZ + (r0 + r) * E;
          if (r < n)
#pragma unroll
            for (int p = 0; p < P; ++p)
              if ((p * G + t.lane) * VL < E) L::store(p, z[u], l[u] == inf, row, (p * G + t.lane) * VL);
        }
      }
      gave_up = t.any(*(volatile int *)&abort_flag);  // the tile has been read, and of a batch's last tile the batch
      if (gave_up) break;
      if (t.thread == 0 && kt + pl.stages < v.ntiles) v.issue_tile(kt + pl.stages, at);
      if (++at == pl.stages) {
        at = 0;
        phase ^= 1;
      }
    }
    if (gave_up) break;
    if (t.thread == 0 && kb + 2 < v.nbatches) v.issue_batch(kb + 2, kb & 1);
  }
  if (gave_up && t.thread == 0) v.drain(kb, kt);
}

// ---------------------------------------------------------------- host ---
// How a row of E logits is spread: whole 16-byte packs when the rows and the
// pointers are whole 16-byte pieces, else pairs of 16-bit elements where they
// are whole 4-byte pieces (262,144 x 258 bf16: 72 us, element by element 89;
// backward 83 and 123), else single elements.  About 16 columns a lane where
// that needs no more than a warp: fewer lanes a row exchange less (524,288 x 64
// bf16 of an earlier version: 44 us with 16 columns a lane, 61 with 8).  Then up
// to kBalLane, and with more columns two, four or eight warps with up to
// kBalLane a lane (65,536 x 2,048 bf16: 93 us with two, 158 with eight).
struct Spread {
  int VL, P, logg;
  bool wide;
  int rows;      // rows of an owner's step
  int resident;  // blocks an SM
  int owners;    // of a block
};
static Spread spread_of(int E, DType dt, int aligned) {  // aligned: bytes, of the pointers
  Spread p{};
  const int row = E * (int)dtype_size(dt);
  const int unit = row % 16 == 0 && aligned % 16 == 0 ? 16 : row % 4 == 0 && aligned % 4 == 0 ? 4 : 2;
  p.VL = unit > (int)dtype_size(dt) ? unit / (int)dtype_size(dt) : 1;
  const int packs = (E + p.VL - 1) / p.VL, most = kBalLane / p.VL, some = kBalSome / p.VL;
  p.wide = packs > 32 * most;
  if (p.wide) p.logg = kWide;
  while ((p.wide || p.logg < 5) && ((p.wide ? most : some) << p.logg) < packs) ++p.logg;
  const int lanes = p.wide ? 1 << p.logg : 32;
  p.P = 1;
  // packs a lane: powers of two, and multiples of four (wide: eight) from eight on
  while (p.P << p.logg < packs) p.P += p.P < 8 ? p.P : p.wide ? 8 : 4;
  p.rows = (lanes >> p.logg) * bal_rows(p.VL * p.P);
  p.resident = bal_blocks(p.VL * p.P);
  p.owners = kBalThreads / lanes;
  return p;
}

static int place_of_columns(int E) { return (E * 4 + 15) / 16 * 16; }

// Blocks, and the plan of an owner's rows.  mid: bytes of labels (or lse) a
// row; extra: bytes a block keeps beside its owners' places.  One wave of
// blocks (more would leave most of the machine idle in a second one), fewer
// where an owner would not have a step's rows; a block takes its share of an
// SM's shared memory, an owner's tiles are as large as leaves three
// of them.
struct Grid {
  Plan pl;
  int blocks;  // per problem
  int smem;
};
static Grid grid_of(int B, int64_t N, int E, DType dt, int mid, int extra, const Spread &p) {
  Grid g{};
  auto place = [](int64_t bytes) { return (int)((bytes + 30 + 15) / 16 * 16); };  // both ends widened
  const int64_t zrow = (int64_t)E * dtype_size(dt);
  const int64_t wave = 148 * p.resident / B > 0 ? 148 * p.resident / B : 1;
  const int64_t room = ((225 * 1024 / p.resident - extra - 2048) / p.owners) / 16 * 16;
  int64_t share = (N + wave * p.owners - 1) / (wave * p.owners);
  share = (share + p.rows - 1) / p.rows * p.rows;
  // no team adds over 1,024 rows into one fp32 sum
  const int64_t most = 1024 * (p.rows / bal_rows(p.VL * p.P));
  if (share > most) share = most;
  // a batch of 32 rows (or the step's; fewer where many labels a row would take
  // over a third of the room) and the largest tile that leaves three of them;
  // then the batch whole tiles
  auto side = [&](int64_t batch) { return 2 * (place(batch * mid) + place(batch)) + (batch * 8 + 15) / 16 * 16; };
  int64_t batch = p.rows > 32 ? p.rows : 32;
  while (batch > 1 && side(batch) > room / 3) batch /= 2;
  int64_t rows = ((room - side(batch)) / 3 - 48) / zrow;
  if (rows > batch) rows = batch;
  if (rows > share) rows = share;
  rows = rows < p.rows ? rows : rows / p.rows * p.rows;
  if (rows < 1) rows = 1;
  batch = batch / rows * rows;
  g.pl.share = (int)share;
  g.pl.rows = (int)rows;
  g.pl.z = place(rows * zrow);
  g.pl.batch = (int)batch;
  g.pl.mid = place(batch * mid);
  g.pl.small = place(batch);
  const int64_t stages = (room - side(batch)) / g.pl.z, tiles = (share + rows - 1) / rows;
  g.pl.stages = (int)(stages < 2 ? 2 : stages > kMaxStages ? kMaxStages : stages);
  if (g.pl.stages > tiles) g.pl.stages = (int)tiles;
  g.blocks = (int)((N + share * p.owners - 1) / (share * p.owners));
  g.smem = p.owners * g.pl.bytes();
  if (g.smem < extra) g.smem = extra;  // the column sums' turn
  g.smem += extra;
  return g;
}

static size_t al256(size_t v) { return (v + 255) / 256 * 256; }
static size_t parts_bytes(int B, int64_t N, int E, DType dt, int aligned) {
  // the blocks do not depend on M
  const size_t parts = (size_t)B * grid_of(B, N, E, dt, 4, place_of_columns(E), spread_of(E, dt, aligned)).blocks;
  return 2 * al256(parts * E * 4) + al256(parts * 4);
}
// Enough for any alignment of Z.
size_t balance_workspace_bytes(int B, int64_t N, int E, DType dt) {
  size_t most = 0;
  for (int aligned : {16, 4, 2}) {
    const size_t n = parts_bytes(B, N, E, dt, aligned);
    if (n > most) most = n;
  }
  return most;
}
static int alignment(const void *p) { return (uintptr_t)p % 16 == 0 ? 16 : (uintptr_t)p % 4 == 0 ? 4 : 2; }

// Lets a kernel have `bytes` of dynamic shared memory; `allowed` remembers per
// device what it may have already.
template <typename K> static cudaError_t allow_smem(K kernel, int bytes, std::atomic<int> *allowed) {
  if (bytes <= 40 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && allowed[dev].load() >= bytes)) return e;
  // the most that any call may ask for, so that calls from two threads do not undo one another
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess && dev < 64) allowed[dev].store(kMaxSmem);
  return e;
}

// Calls f with the spread's template arguments: every spread that spread_of
// makes is listed.
template <typename T, typename F> static void with_spread(const Spread &p, F f) {
  constexpr int V = 16 / (int)sizeof(T);
#define FK_P(vl, n, lg)                                                                                           \
  if (p.VL == vl && p.P == n && (lg == kAnyTeam ? !p.wide : p.logg == lg))                                         \
    return f(std::integral_constant<int, vl>(), std::integral_constant<int, n>(), std::integral_constant<int, lg>());
  constexpr int H = kBalSome / V;  // packs a lane where a row takes more than one
  if constexpr (H == 4) { FK_P(V, 1, 0) }
  FK_P(V, H / 2, 0)
  FK_P(V, H, 0) FK_P(V, H, 1) FK_P(V, H, 2) FK_P(V, H, 3) FK_P(V, H, 4) FK_P(V, H, 5) FK_P(V, 2 * H, 5)
  FK_P(V, 2 * H, 6) FK_P(V, 2 * H, 7) FK_P(V, 2 * H, 8)
  if constexpr (V == 8) {
    FK_P(2, 1, 0) FK_P(2, 2, 0) FK_P(2, 4, 0) FK_P(2, 8, 0) FK_P(2, 8, 1) FK_P(2, 8, 2) FK_P(2, 8, 3) FK_P(2, 8, 4)
    FK_P(2, 8, 5) FK_P(2, 12, 5) FK_P(2, 16, 5)
    FK_P(2, 16, 6) FK_P(2, 16, 7) FK_P(2, 16, 8)
  }
  FK_P(1, 1, 0) FK_P(1, 2, 0) FK_P(1, 4, 0) FK_P(1, 8, 0) FK_P(1, 12, 5) FK_P(1, 16, 5)
  FK_P(1, 12, kAnyTeam) FK_P(1, 16, kAnyTeam)
  FK_P(1, 20, 5) FK_P(1, 24, 5) FK_P(1, 28, 5) FK_P(1, 32, 5)
  FK_P(1, 24, 6) FK_P(1, 32, 6) FK_P(1, 24, 7) FK_P(1, 32, 7) FK_P(1, 24, 8) FK_P(1, 32, 8)
#undef FK_P
}

template <typename T> static cudaError_t balance_from(const BalanceArgs &a, void *ws, DevCtl ctl, cudaStream_t s) {
  const Spread p = spread_of(a.E, a.dt, alignment(a.Z));
  const Grid g = grid_of(a.B, a.N, a.E, a.dt, 4 * a.M, place_of_columns(a.E), p);
  const int nb = g.blocks;
  const size_t parts = (size_t)a.B * nb;
  float *psum = (float *)ws;
  int *csum = (int *)((char *)ws + al256(parts * a.E * 4));
  int *tsum = (int *)((char *)ws + 2 * al256(parts * a.E * 4));
  const BalanceOut out{a.loss, a.counts, a.tokens, a.meanp, a.coef};
  cudaError_t e = cudaErrorNotSupported;
  with_spread<T>(p, [&](auto vl, auto np, auto lg) {
    const auto kernel = balance_rows_kernel<T, decltype(vl)::value, decltype(np)::value, decltype(lg)::value>;
    static std::atomic<int> allowed[64];
    e = allow_smem(kernel, g.smem, allowed);
    if (e == cudaSuccess)
      e = launch_chained(kernel, dim3(nb, a.B), dim3(kBalThreads), g.smem, s, (const T *)a.Z, a.ids, a.mask, a.B,
                         a.N, a.E, a.M, p.logg, g.pl, a.lse, psum, csum, tsum, out, ctl);
  });
  count_launches(1);
  if (e != cudaSuccess || nb == 1) return e;
  const int ncta = a.E <= 32 ? 1 : a.E >= 32 * kJoinCluster ? kJoinCluster : (a.E + 31) / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ncta, a.B);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ncta;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, balance_join_kernel, (const float *)psum, (const int *)csum, (const int *)tsum, nb, a.E,
                            a.M, out);
}
cudaError_t launch_balance(const BalanceArgs &a, void *ws, DevCtl ctl, cudaStream_t s) {
  return a.dt == kF32   ? balance_from<float>(a, ws, ctl, s)
         : a.dt == kF16 ? balance_from<__half>(a, ws, ctl, s)
                        : balance_from<__nv_bfloat16>(a, ws, ctl, s);
}

template <typename T> static cudaError_t balance_grad_from(const BalanceGradArgs &a, DevCtl ctl, cudaStream_t s) {
  const Spread p = spread_of(a.E, a.dt, alignment(a.Z) < alignment(a.dZ) ? alignment(a.Z) : alignment(a.dZ));
  const Grid g = grid_of(a.B, a.N, a.E, a.dt, 4, 0, p);
  cudaError_t e = cudaErrorNotSupported;
  with_spread<T>(p, [&](auto vl, auto np, auto lg) {
    const auto kernel = balance_grad_kernel<T, decltype(vl)::value, decltype(np)::value, decltype(lg)::value>;
    static std::atomic<int> allowed[64];
    e = allow_smem(kernel, g.smem, allowed);
    if (e == cudaSuccess)
      e = launch_chained(kernel, dim3(g.blocks, a.B), dim3(kBalThreads), g.smem, s, (const T *)a.Z, a.counts, a.tokens,
                         a.lse, a.gloss, a.B, a.N, a.E, a.M, a.coef, p.logg, g.pl, (T *)a.dZ, ctl);
  });
  return e;
}
cudaError_t launch_balance_grad(const BalanceGradArgs &a, DevCtl ctl, cudaStream_t s) {
  count_launches(1);
  return a.dt == kF32   ? balance_grad_from<float>(a, ctl, s)
         : a.dt == kF16 ? balance_grad_from<__half>(a, ctl, s)
                        : balance_grad_from<__nv_bfloat16>(a, ctl, s);
}

}  // namespace fk
