// label_sort.cu -- stable sort of points by label (the inverse map of the
// sort-inverse update and of the codebook gradient).
//
// Least-significant-digit radix sort of the keys b*K + label: 11-bit digits,
// one pass for up to 2,048 keys, two for up to 2^22; a batch of problems
// whose N is whole 4096-key tiles takes one pass on the label per problem.
// A pass is three kernels: per-tile digit histograms, a per-digit scan over
// tiles, and a scatter whose within-tile ranks come from shared-memory digit
// masks.  The sorted point ids are the inverse map (label -> its points); no
// global atomics, so the order is the same on every run.
#include "chain.cuh"
#include "fk_internal.h"

namespace fk {

constexpr int kSortThreads = 256;
constexpr int kSortItems = 16;
constexpr int kSortTile = kSortThreads * kSortItems;  // 4096 keys per tile
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 11;
constexpr int kMaxBins = 1 << kMaxDigitBits;

struct SortPlan {
  int npass;
  int shift[2], bits[2];
  int T;          // tiles
  int seg_tiles;  // > 0: one pass on the label digit, problems of seg_tiles whole tiles each
};

static int ceil_log2(long long v) {
  int b = 0;
  while ((1ll << b) < v) ++b;
  return b;
}

// A batch of B problems whose N is a whole number of tiles is sorted in one
// pass on the label alone when the key b*K + label would need two: the
// problems' points are already in problem order, and each tile belongs to
// one problem, so ranking a tile's points by label and placing problem b's
// runs at b*N gives the order of a stable sort by key.
// With `drop` there is one key more, B*K, for the points that name no row (in
// a pass on the label alone: digit K).
static SortPlan plan_sort(long long Ntot, long long Ktot, int B, bool drop) {
  SortPlan p{};
  int bits = ceil_log2(Ktot + drop);
  if (bits < 1) bits = 1;
  p.npass = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  const int w = (bits + p.npass - 1) / p.npass;
  int sh = 0;
  for (int i = 0; i < p.npass; ++i) {
    p.shift[i] = sh;
    p.bits[i] = (bits - sh) < w ? (bits - sh) : w;
    sh += p.bits[i];
  }
  p.T = (int)((Ntot + kSortTile - 1) / kSortTile);
  if (B > 1 && p.npass > 1 && (Ntot / B) % kSortTile == 0 && ceil_log2(Ktot / B + drop) <= kMaxDigitBits) {
    p.npass = 1;
    p.shift[0] = 0;
    p.bits[0] = ceil_log2(Ktot / B + drop) < 1 ? 1 : ceil_log2(Ktot / B + drop);
    p.seg_tiles = (int)(Ntot / B / kSortTile);
  }
  return p;
}

// --------------------------------------------------------------- sorting --
// Sort key of position pos from its label: b*K + label for problem b.  A
// label outside [0, K) counts as 0, or with DROP gets the key B*K of the
// points left out (-1 is a point that names no row, not an error); it sets
// `bad`, and the caller records that once, after all of its loads, so that
// no atomic sits between them.
template <bool DROP>
__device__ __forceinline__ int key_of_label(int lab, int pos, int N, int K, int B, bool &bad) {
  if ((unsigned)lab >= (unsigned)K) {
    if (DROP) {
      bad |= lab != -1;
      return B * K;
    }
    bad = true;
    lab = 0;
  }
  return B > 1 ? (pos / N) * K + lab : lab;
}

// Digit of a key in a pass on the label alone, in problem pb: the label, or K
// for the key of the points left out.
template <bool DROP> __device__ __forceinline__ int seg_digit(int key, int pb, int K) {
  const int d = key - pb * K;
  return DROP && d > K ? K : d;
}

// SEG: one pass per problem (the digit is the label), see plan_sort.
template <bool FIRST, bool SEG, bool DROP>
__global__ void __launch_bounds__(kSortThreads) radix_hist_kernel(const int32_t *__restrict__ keys, int Ntot,
                                                                  int N, int K, int B, int shift, int nbins,
                                                                  int T, int *__restrict__ H,
                                                                  int *status, int seg_tiles) {
  __shared__ int hist[kMaxBins + 1];
  for (int i = threadIdx.x; i <= nbins; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  wait_prior_grid();
  const int base = blockIdx.x * kSortTile;
  // all of the thread's keys are loaded before any is counted (16 loads in
  // flight), then counted with shared-memory atomics
  int v[kSortItems];
#pragma unroll
  for (int it = 0; it < kSortItems; ++it) {
    const int pos = base + it * kSortThreads + threadIdx.x;
    v[it] = pos < Ntot ? keys[pos] : 0;
  }
  bool bad = false;
#pragma unroll
  for (int it = 0; it < kSortItems; ++it) {
    const int pos = base + it * kSortThreads + threadIdx.x;
    int d = nbins;  // spare bin for positions past the end
    if (pos < Ntot) {
      const int key = FIRST ? key_of_label<DROP>(v[it], pos, N, K, B, bad) : v[it];
      // one pass per problem: the digit is the label (each tile lies in one problem)
      d = SEG ? seg_digit<DROP>(key, (int)blockIdx.x / seg_tiles, K) : (key >> shift) & (nbins - 1);
    }
    atomicAdd(&hist[d], 1);
  }
  if (bad) record_status(status, kStBadLabel);
  __syncthreads();
  for (int i = threadIdx.x; i < nbins; i += kSortThreads) H[(size_t)i * T + blockIdx.x] = hist[i];
}

// In place: row d of H becomes the exclusive prefix over tiles; totals[d] = row sum.
__global__ void __launch_bounds__(256) scan_rows_kernel(int *__restrict__ H, int T, int nbins,
                                                        int *__restrict__ totals) {
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  wait_prior_grid();
  if (w >= nbins) return;
  int *row = H + (size_t)w * T;
  int carry = 0;
  // 256 tiles per round: all of a lane's loads are issued before any is
  // scanned, so a round costs one memory round trip
  constexpr int kPerLane = 8;
  for (int t0 = 0; t0 < T; t0 += 32 * kPerLane) {
    int v[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int tt = t0 + 32 * i + lane;
      v[i] = tt < T ? row[tt] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      int incl = v[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
      }
      const int tt = t0 + 32 * i + lane;
      if (tt < T) row[tt] = carry + incl - v[i];
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (lane == 0) totals[w] = carry;
}

// ints of the region that holds the warps' digit masks while keys are
// ranked, then the tile's keys and values in sorted order
static __host__ __device__ int scatter_xbuf_ints(int nbins) {
  return 2 * kSortTile > kSortWarps * nbins ? 2 * kSortTile : kSortWarps * nbins;
}
static size_t scatter_smem_bytes(int nbins) {
  return (size_t)(2 * nbins + kSortWarps + scatter_xbuf_ints(nbins)) * 4 + (size_t)kSortWarps * (nbins + 1) * 4;
}

template <bool FIRST, bool SEG, bool DROP>
__global__ void __launch_bounds__(kSortThreads) radix_scatter_kernel(
    const int32_t *__restrict__ keys_in, const int32_t *__restrict__ vals_in, int32_t *__restrict__ keys_out,
    int32_t *__restrict__ vals_out, int Ntot, int N, int K, int B, int shift, int nbins, int T,
    const int *__restrict__ H, const int *__restrict__ totals, int *status, int seg_tiles) {
  extern __shared__ int sh[];
  const int stride = nbins + 1;
  int *dbase = sh;                                                   // [nbins]
  int *tstart = sh + nbins;                                          // [nbins]
  int *wsum = sh + 2 * nbins;                                        // [kSortWarps]
  int *keys_s = sh + 2 * nbins + kSortWarps;                         // [kSortTile]
  int *vals_s = keys_s + kSortTile;                                  // [kSortTile]
  unsigned *wmask = reinterpret_cast<unsigned *>(keys_s);            // [kSortWarps][nbins], same place
  int *wcnt = keys_s + scatter_xbuf_ints(nbins);                     // [kSortWarps][nbins + 1]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // one pass per problem (SEG): this tile's problem; the digit is the label
  // and the problem's runs start at pb * N
  const int pb = SEG ? (int)blockIdx.x / seg_tiles : 0;
  auto digit = [&](int key) { return SEG ? seg_digit<DROP>(key, pb, K) : (key >> shift) & (nbins - 1); };
  wait_prior_grid();
  // the warp's 512 consecutive keys and values are loaded first, so that
  // their latency overlaps the digit-base reads below
  int keyr[kSortItems], valr[kSortItems], locr[kSortItems];
  const int base = blockIdx.x * kSortTile + warp * (kSortItems * 32);
#pragma unroll
  for (int it = 0; it < kSortItems; ++it) {
    const int pos = base + it * 32 + lane;
    keyr[it] = pos < Ntot ? keys_in[pos] : 0;
    valr[it] = pos < Ntot ? (FIRST ? pos : vals_in[pos]) : 0;
  }

  // digit base of this tile = exclusive scan of digit totals + tile prefix;
  // both reads of a thread's digits are issued before either is used
  constexpr int kPer = kMaxBins / kSortThreads;  // digits per thread, at most
  const int per = (nbins + kSortThreads - 1) / kSortThreads;
  int tv[kPer], hv[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = tid * per + i;
    const bool ok = i < per && d < nbins;
    if (SEG) {
      // the problem's count of digit d and the count in its tiles before
      // this one, from the prefix over all tiles at the problem's bounds
      const int t0 = pb * seg_tiles, t1 = t0 + seg_tiles;
      const int p0 = ok ? H[(size_t)d * T + t0] : 0;
      const int p1 = ok ? (t1 < T ? H[(size_t)d * T + t1] : totals[d]) : 0;
      tv[i] = p1 - p0;
      hv[i] = (ok ? H[(size_t)d * T + blockIdx.x] : 0) - p0;
    } else {
      tv[i] = ok ? totals[d] : 0;
      hv[i] = ok ? H[(size_t)d * T + blockIdx.x] : 0;
    }
  }
  int s = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s += tv[i];
  int incl = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) wsum[warp] = incl;
  for (int i = tid; i < kSortWarps * stride; i += kSortThreads) wcnt[i] = 0;
  for (int i = tid; i < kSortWarps * nbins; i += kSortThreads) wmask[i] = 0u;
  __syncthreads();
  int run = incl - s + pb * N;
  for (int w = 0; w < warp; ++w) run += wsum[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int d = tid * per + i;
    if (i < per && d < nbins) dbase[d] = run + hv[i];
    run += tv[i];
  }

  // stable ranks within each warp's consecutive keys.  The lanes that hold
  // the same digit find each other through shared memory: each sets its bit
  // in the warp's mask word of its digit and reads the word back (on this
  // GPU much cheaper than a ballot per digit bit or match.any, whose cost
  // grows with the number of distinct digits).  The lowest of them clears
  // the word and adds the group's size to the warp's count of that digit;
  // the count before the add, broadcast after all of the warp's keys are
  // counted, is where the group starts.
  const unsigned lt_mask = (1u << lane) - 1u;
  int *mycnt = wcnt + warp * stride;
  unsigned *mymask = wmask + warp * nbins;
  unsigned peer[kSortItems];
  bool bad = false;
#pragma unroll
  for (int it = 0; it < kSortItems; ++it) {
    const int pos = base + it * 32 + lane;
    const bool valid = pos < Ntot;
    int d = 0;
    if (valid) {
      if (FIRST) keyr[it] = key_of_label<DROP>(keyr[it], pos, N, K, B, bad);
      d = digit(keyr[it]);
    }
    if (valid) atomicOr(mymask + d, 1u << lane);
    __syncwarp();
    const unsigned peers = valid ? mymask[d] : 0u;
    __syncwarp();
    int c = 0;
    if (valid && lane == __ffs(peers) - 1) {
      mymask[d] = 0u;
      c = atomicAdd(mycnt + d, __popc(peers));
    }
    __syncwarp();  // the next key's mask and add come after these
    peer[it] = peers;
    locr[it] = c;
  }
#pragma unroll
  for (int it = 0; it < kSortItems; ++it)
    locr[it] = __shfl_sync(0xffffffffu, locr[it], (__ffs(peer[it]) - 1) & 31) + __popc(peer[it] & lt_mask);
  if (bad) record_status(status, kStBadLabel);
  __syncthreads();  // masks done: the region holds keys and values from here on
  // per digit: exclusive prefix over warps (in place) and the tile's count,
  // then the exclusive scan of the tile's counts over digits: where each
  // digit's run starts in the tile's sorted order
  int cnt[kPer];
  int tsum = 0;
  for (int i = 0; i < per; ++i) {
    const int d = tid * per + i;
    int r = 0;
    if (d < nbins)
      for (int w = 0; w < kSortWarps; ++w) {
        const int t = wcnt[w * stride + d];
        wcnt[w * stride + d] = r;
        r += t;
      }
    cnt[i] = r;
    tsum += r;
  }
  int tincl = tsum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, tincl, o);
    if (lane >= o) tincl += n;
  }
  __syncthreads();  // everyone is done reading wsum (digit bases above)
  if (lane == 31) wsum[warp] = tincl;
  __syncthreads();
  int trun = tincl - tsum;
  for (int w = 0; w < warp; ++w) trun += wsum[w];
  for (int i = 0; i < per; ++i) {
    const int d = tid * per + i;
    if (d < nbins) tstart[d] = trun;
    trun += cnt[i];
  }
  __syncthreads();
  // exchange through shared memory into the tile's sorted order ...
#pragma unroll
  for (int it = 0; it < kSortItems; ++it) {
    const int pos = base + it * 32 + lane;
    if (pos < Ntot) {
      const int d = digit(keyr[it]);
      const int lp = tstart[d] + mycnt[d] + locr[it];
      keys_s[lp] = keyr[it];
      vals_s[lp] = valr[it];
    }
  }
  __syncthreads();
  // ... and write it out in that order: consecutive threads store
  // consecutive positions of a digit's run
  const int nvalid = (Ntot - blockIdx.x * kSortTile) < kSortTile ? (Ntot - blockIdx.x * kSortTile) : kSortTile;
#pragma unroll
  for (int it = 0; it < kSortItems; ++it) {
    const int idx = it * kSortThreads + tid;
    if (idx < nvalid) {
      const int key = keys_s[idx];
      const int d = digit(key);
      const int o = dbase[d] + (idx - tstart[d]);
      keys_out[o] = key;
      vals_out[o] = vals_s[idx];
    }
  }
}


static size_t al256(size_t v) { return (v + 255) / 256 * 256; }

// ------------------------------------------------- one launch, few points --
// Up to kFewPoints points are sorted by one cluster of CTAs in one launch (a
// whole gradient of 32,768 x 64 bf16 in a replayed graph: 33 us with 60,000
// labels, 39 us with the kernels above; with 65,536 points, eight CTAs are too
// few: 44 us and 39 us): the
// three kernels of a pass become two cluster barriers, the tiles' digit counts
// are read from the CTAs' shared memory, and the points change CTAs by stores
// to shared memory.  Digits of at most 9 bits: two passes up to 2^18 keys,
// three up to 2^22.  Meanwhile an array is zero-filled (the gradient's, whose
// rows without a point nobody else writes): a little by the grid's other
// clusters, more by a kernel of its own that runs beside the sort.
constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32, kFewCtas = 8, kFewItems = 8;
constexpr int kFewPoints = kFewThreads * kFewItems * kFewCtas;  // 32,768
constexpr size_t kFewFill = size_t(64) << 20;
constexpr int kFewBits = 9, kFewBins = 1 << kFewBits;

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, int a, int b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Zeroes [p, p + n), p aligned to its 2- or 4-byte elements; block `at` of `of`.
__device__ __forceinline__ void zero_fill(char *p, size_t n, int at, int of) {
  const size_t head = n < ((16 - (uintptr_t)p % 16) % 16) ? n : (16 - (uintptr_t)p % 16) % 16;
  const size_t body = (n - head) / 16, tail = n - head - body * 16;
  if (at == 0) {
    unsigned short *h = (unsigned short *)p, *t = (unsigned short *)(p + head + body * 16);
    if (threadIdx.x < head / 2) h[threadIdx.x] = 0;
    if (threadIdx.x < tail / 2) t[threadIdx.x] = 0;
  }
  uint4 *q = (uint4 *)(p + head);
#pragma unroll 4
  for (size_t i = (size_t)at * blockDim.x + threadIdx.x; i < body; i += (size_t)of * blockDim.x)
    q[i] = make_uint4(0, 0, 0, 0);
}

static int few_smem_bytes(int bins, int items) {
  return (2 * bins + kFewWarps + kFewWarps * bins + kFewWarps * (bins + 1) + 2 * kFewThreads * items) * 4;
}

// ITEMS points a thread; CTA c of the first cluster holds positions
// [c, c + 1) * kFewThreads * ITEMS.
template <int ITEMS>
__global__ void __launch_bounds__(kFewThreads) sort_few_kernel(const int32_t *__restrict__ labels, int rows, int N,
                                                               int K, int B, int npass, int bits, int bins,
                                                               int32_t *__restrict__ skeys,
                                                               int32_t *__restrict__ perm, char *fill, size_t fill_bytes,
                                                               int ncta, int *status) {
  constexpr int TILE = kFewThreads * ITEMS;
  extern __shared__ int sh[];
  wait_prior_grid();
  let_next_grid();  // fill_kernel, where there is one, may start (every other waits for this grid's end)
  if ((int)blockIdx.x >= ncta) {
    zero_fill(fill, fill_bytes, blockIdx.x - ncta, gridDim.x - ncta);
    return;
  }
  int2 *moved = reinterpret_cast<int2 *>(sh);                    // [TILE] key, row of the positions held
  int *total = sh + 2 * TILE;                                    // [bins] points of each digit here
  int *dbase = total + bins;                                     // [bins] where this CTA's points of a digit go
  int *wsum = dbase + bins;                                      // [kFewWarps]
  unsigned *wmask = reinterpret_cast<unsigned *>(wsum + kFewWarps);  // [kFewWarps][bins]
  int *wcnt = reinterpret_cast<int *>(wmask) + kFewWarps * bins;     // [kFewWarps][bins + 1]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x, stride = bins + 1;
  const int here = warp * (32 * ITEMS) + lane;  // of the thread's first item
  const int base = rank * TILE + here;
  int key[ITEMS], val[ITEMS], place[ITEMS];
  bool bad = false;
#pragma unroll
  for (int it = 0; it < ITEMS; ++it) {
    const int pos = base + it * 32;
    val[it] = pos;
    key[it] = pos < rows ? labels[pos] : 0;
  }
#pragma unroll
  for (int it = 0; it < ITEMS; ++it)
    if (base + it * 32 < rows) key[it] = key_of_label<true>(key[it], base + it * 32, N, K, B, bad);
  if (bad) record_status(status, kStBadLabel);
  int *mycnt = wcnt + warp * stride;
  unsigned *mymask = wmask + warp * bins;
  for (int pass = 0; pass < npass; ++pass) {
    const int shift = pass * bits;
    for (int i = tid; i < kFewWarps * stride; i += kFewThreads) wcnt[i] = 0;
    for (int i = tid; i < kFewWarps * bins; i += kFewThreads) wmask[i] = 0u;
    __syncthreads();
    // stable ranks within each warp's consecutive positions, as in radix_scatter_kernel
    unsigned peer[ITEMS];
#pragma unroll
    for (int it = 0; it < ITEMS; ++it) {
      const bool valid = base + it * 32 < rows;
      const int d = key[it] >> shift & (bins - 1);
      if (valid) atomicOr(mymask + d, 1u << lane);
      __syncwarp();
      const unsigned peers = valid ? mymask[d] : 0u;
      __syncwarp();
      int c = 0;
      if (valid && lane == __ffs(peers) - 1) {
        mymask[d] = 0u;
        c = atomicAdd(mycnt + d, __popc(peers));
      }
      __syncwarp();
      peer[it] = peers;
      place[it] = c;
    }
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
      place[it] = __shfl_sync(0xffffffffu, place[it], (__ffs(peer[it]) - 1) & 31) + __popc(peer[it] & ((1u << lane) - 1u));
    __syncthreads();
    if (tid < bins) {  // per digit: exclusive prefix over the warps, and the CTA's count
      int r = 0;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        const int t = wcnt[w * stride + tid];
        wcnt[w * stride + tid] = r;
        r += t;
      }
      total[tid] = r;
    }
    cluster_sync();  // every CTA has its counts, and has read the points it held
    int all = 0, before = 0;
    if (tid < bins)
#pragma unroll
      for (int c = 0; c < kFewCtas; ++c)
        if (c < ncta) {
          const int t = (int)ld_cluster(map_to_cta(smem_u32(&total[tid]), c));
          all += t;
          if (c < rank) before += t;
        }
    int incl = all;  // over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int run = incl - all + before;
    for (int w = 0; w < warp; ++w) run += wsum[w];
    if (tid < bins) dbase[tid] = run;
    __syncthreads();
    const bool last = pass == npass - 1;
#pragma unroll
    for (int it = 0; it < ITEMS; ++it)
      if (base + it * 32 < rows) {
        const int d = key[it] >> shift & (bins - 1);
        const int to = dbase[d] + mycnt[d] + place[it];
        if (last) {
          skeys[to] = key[it];
          perm[to] = val[it];
        } else {
          st_cluster2(map_to_cta(smem_u32(&moved[to % TILE]), to / TILE), key[it], val[it]);
        }
      }
    cluster_sync();  // the points have moved, and no CTA reads the others' counts any more
    if (!last)
#pragma unroll
      for (int it = 0; it < ITEMS; ++it) {
        const int2 p = moved[here + it * 32];
        key[it] = p.x;
        val[it] = p.y;
      }
  }
}

// Zero-fills beside the sort that was launched before it: it starts when the
// sort has (so everything before the sort is done), and ends when the sort
// has, so that what waits for it has waited for both.
__global__ void __launch_bounds__(512) fill_kernel(char *fill, size_t bytes) {
  zero_fill(fill, bytes, blockIdx.x, gridDim.x);
  wait_prior_grid();
}

static cudaError_t run_sort_few(const int32_t *labels, int B, int N, int K, void *ws, int *status, cudaStream_t s,
                                LabelSort *out, void *fill, size_t fill_bytes) {
  const int rows = B * N;
  const long long Ktot = (long long)B * K;
  int keybits = ceil_log2(Ktot + 1);
  if (keybits < 1) keybits = 1;
  const int npass = (keybits + kFewBits - 1) / kFewBits, bits = (keybits + npass - 1) / npass, bins = 1 << bits;
  // four points a thread and more CTAs before more points a thread
  int ncta = 1, items = 2;
  if (rows > kFewThreads * items) items = 4;
  while (ncta < kFewCtas && rows > kFewThreads * items * ncta) ncta *= 2;
  while (rows > kFewThreads * items * ncta) items *= 2;
  const auto kernel = items == 2 ? sort_few_kernel<2>
                      : items == 4 ? sort_few_kernel<4> : sort_few_kernel<8>;
  {
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !configured[dev]) {
      const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
      cudaError_t e = cudaFuncSetAttribute(sort_few_kernel<2>, at, few_smem_bytes(kFewBins, 2));
      if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_few_kernel<4>, at, few_smem_bytes(kFewBins, 4));
      if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_few_kernel<8>, at, few_smem_bytes(kFewBins, 8));
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  // beside the sort: one block of 512 threads an SM, with 32 KB to fill at
  // least, and no launch of its own, which is worth up to 3 us: a whole gradient
  // of 256 bf16 columns in a replayed graph takes 16.2 us with 500 labels and a
  // fill of 64 MiB, 18.7 with a kernel of its own; with 24,000 labels 32.3 and
  // 34.5 (with 6,000 and 32,768 the kernel is ahead by 1).  But the few fillers'
  // rate is lower: from 128 MiB on the kernel is ahead with more than some 4,000
  // labels (36.0 and 44.2 us with 6,000), at 512 MiB from 1,000 on (88 and 93;
  // 97 and 142 with 16,384).
  const bool apart = fill_bytes > kFewFill;
  long long fillers = apart ? 0 : (long long)((fill_bytes + 32767) / 32768);
  if (fillers > 148) fillers = 148;
  fillers = (fillers + ncta - 1) / ncta * ncta;
  int32_t *keys = (int32_t *)ws, *ids = (int32_t *)((char *)ws + al256((size_t)rows * 4));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ncta + (unsigned)fillers);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = few_smem_bytes(bins, items);
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, labels, rows, N, K, B, npass, bits, bins, keys, ids, (char *)fill,
                                     fill_bytes, ncta, status);
  count_launches(1);
  if (e == cudaSuccess && apart) {
    const size_t blocks = fill_bytes / (512 * 16 * 8) + 1;  // eight vectors a thread
    e = launch_chained(fill_kernel, dim3((unsigned)(blocks < (1u << 20) ? blocks : 1u << 20)), dim3(512), 0, s,
                       (char *)fill, fill_bytes);
    count_launches(1);
  }
  out->skeys = keys;
  out->perm = ids;
  return e;
}

// ---------------------------------------------------------------- host ---

struct SortWs {
  int32_t *kA, *vA, *kB, *vB;
  int *H, *totals;
  size_t bytes;
};
static SortWs carve_sort(void *base, long long Ntot, const SortPlan &sp) {
  int maxbins = 0;
  for (int i = 0; i < sp.npass; ++i) maxbins = (1 << sp.bits[i]) > maxbins ? (1 << sp.bits[i]) : maxbins;
  SortWs w{};
  char *p = (char *)base;
  size_t o = 0;
  auto take = [&](size_t n) { char *r = p ? p + o : nullptr; o += al256(n); return r; };
  w.kA = (int32_t *)take((size_t)Ntot * 4);
  w.vA = (int32_t *)take((size_t)Ntot * 4);
  w.kB = (int32_t *)take((size_t)Ntot * 4);
  w.vB = (int32_t *)take((size_t)Ntot * 4);
  w.H = (int *)take((size_t)maxbins * sp.T * 4);
  w.totals = (int *)take((size_t)maxbins * 4);
  w.bytes = o;
  return w;
}

size_t label_sort_bytes(int64_t Ntot, int64_t Ktot, int B, bool drop) {
  return carve_sort(nullptr, Ntot, plan_sort(Ntot, Ktot, B, drop)).bytes;
}

template <bool DROP>
static cudaError_t run_sort(const int32_t *labels, int B, int N, int K, void *ws, int *status, cudaStream_t s,
                            LabelSort *out) {
  const long long Ntot = (long long)B * N, Ktot = (long long)B * K;
  const SortPlan sp = plan_sort(Ntot, Ktot, B, DROP);
  const SortWs w = carve_sort(ws, Ntot, sp);
  {  // the scatter's tile exchange needs more than the default 48 KB of shared memory
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !configured[dev]) {
      const int most = (int)scatter_smem_bytes(kMaxBins);
      cudaFuncSetAttribute(radix_scatter_kernel<true, false, DROP>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      cudaFuncSetAttribute(radix_scatter_kernel<true, true, DROP>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      cudaFuncSetAttribute(radix_scatter_kernel<false, false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      configured[dev] = true;
    }
  }
  const int32_t *kin = labels, *vin = nullptr;
  int32_t *kout = w.kA, *vout = w.vA;
  int nl = 0;
  for (int pass = 0; pass < sp.npass; ++pass) {
    const int nbins = 1 << sp.bits[pass];
    const bool seg = sp.seg_tiles > 0;  // one pass, so pass == 0
    const auto hist = pass > 0 ? radix_hist_kernel<false, false, false>
                               : seg ? radix_hist_kernel<true, true, DROP> : radix_hist_kernel<true, false, DROP>;
    launch_chained(hist, dim3(sp.T), dim3(kSortThreads), 0, s, kin, (int)Ntot, N, K, B, sp.shift[pass], nbins, sp.T, w.H,
                   status, sp.seg_tiles);
    launch_chained(scan_rows_kernel, dim3((nbins + 7) / 8), dim3(256), 0, s, w.H, sp.T, nbins, w.totals);
    const auto scatter = pass > 0 ? radix_scatter_kernel<false, false, false>
                                  : seg ? radix_scatter_kernel<true, true, DROP> : radix_scatter_kernel<true, false, DROP>;
    launch_chained(scatter, dim3(sp.T), dim3(kSortThreads), scatter_smem_bytes(nbins), s, kin, vin, kout, vout, (int)Ntot,
                   N, K, B, sp.shift[pass], nbins, sp.T, w.H, w.totals, status, sp.seg_tiles);
    nl += 3;
    kin = kout;
    vin = vout;
    kout = (kout == w.kA) ? w.kB : w.kA;
    vout = (vout == w.vA) ? w.vB : w.vA;
  }
  out->skeys = kin;
  out->perm = vin;
  count_launches(nl);
  return cudaGetLastError();
}

cudaError_t launch_label_sort(const int32_t *labels, int B, int N, int K, void *ws, int *status, cudaStream_t s,
                              LabelSort *out) {
  return run_sort<false>(labels, B, N, K, ws, status, s, out);
}

cudaError_t launch_label_sort_drop(const int32_t *labels, int B, int N, int K, void *ws, int *status, cudaStream_t s,
                                   LabelSort *out, void *fill, size_t fill_bytes) {
  if ((long long)B * N <= kFewPoints) return run_sort_few(labels, B, N, K, ws, status, s, out, fill, fill_bytes);
  if (fill_bytes > 0) {
    const cudaError_t e = cudaMemsetAsync(fill, 0, fill_bytes, s);
    if (e != cudaSuccess) return e;
  }
  return run_sort<true>(labels, B, N, K, ws, status, s, out);
}

}  // namespace fk
