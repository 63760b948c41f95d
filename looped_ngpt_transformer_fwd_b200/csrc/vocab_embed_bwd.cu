// Gradient of the embedding lookup h_i = E[t_i] / |E[t_i]| by sorted tokens.
//   G_t = sum of dh_i over the rows with token t,
//   dE_t = (G_t - E_t (E_t . G_t) / |E_t|^2) / |E_t|
// (|E_t|^2 below 1e-20, where the lookup clamps the norm: dE_t = 1e10 G_t).
// The projection is linear, so it runs once per distinct token, after the sum.
//
// The tokens are sorted by (token, row), so equal tokens lie together; windows of
// the sorted list are summed independently, each finishing the runs that start
// in it, except that a long run is summed window by window and joined by a
// second kernel.  Every sum has a fixed order: at most 64 rows one after the other
// in 32 bits, the windows of a longer run in 64, rounded to 32 before the
// projection.
//
// Bound: HBM where the table is written: 32768 rows of 2048 into 131072 x 2048
// (tokens by frequency) 249 us, floor 212.  Adding to few rows is bound by the
// chain of launches: 4096 rows into the same table 30 us (floor 12), the sort 8,
// the sums 20 and the joining of long runs 10 of them when run alone from a cold
// cache; 32768 rows 141 (floor 78), the sort 30, the sums 100, the joining 14.
// 128 rows of 256 into 1024 x 256: 12 us.  Sums by atomics instead of the sort
// would neither repeat their bits nor allow one projection per token.
#include <string.h>

#include "kernels.h"
#include "vocab_ops.cuh"

namespace dory {

namespace {

// ------------------------------------------------------------- the launches
// A call is a chain of short kernels.  Each allows the next one to start early,
// and waits itself for the one before it (which has waited for the one before
// that) before it touches what they write.  What a kernel reads of them goes by
// plain loads, not by the read-only path.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
void launch_next(bool early, void (*kernel)(P...), int grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);   // an error stays for cudaGetLastError
}

// --------------------------------------------------------------- zero filling
// The sort's launches occupy a few SMs for some microseconds each: CTAs behind
// the sorting ones meanwhile write zeros over the table's last rows (whose
// tokens are the rare ones; the rows that do get a sum are written again).
struct Fill {
  float4* dst = nullptr;
  size_t n4 = 0;
};
constexpr size_t kFillBytes = 64 << 10;   // per CTA

__device__ __forceinline__ void fill_part(const Fill& f, int part) {
  const size_t first = part * (kFillBytes / 16);
  const size_t last = first + kFillBytes / 16 < f.n4 ? first + kFillBytes / 16 : f.n4;
  for (size_t i = first + threadIdx.x; i < last; i += blockDim.x) f.dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}
int fill_ctas(const Fill& f) { return static_cast<int>((f.n4 * 16 + kFillBytes - 1) / kFillBytes); }

// ------------------------------------------------------------------ the sort
// Up to kRankMax rows: a row's place is the number of (token, row) pairs below
// it, counted against all of them; n^2 comparisons over the whole GPU, one
// launch.  32 rows per CTA, a lane per row, each warp taking an eighth of the
// others: 8 us at 4096 rows, 16 at 8192, where the radix sort takes 23.
constexpr int kRankMax = 8192;
constexpr int kRankThreads = 256;
constexpr int kRankWarps = kRankThreads / 32;

__device__ __forceinline__ int32_t sort_key(int32_t t, int vocab) {
  return t < 0 || t >= vocab ? vocab : t;   // what is no token sorts behind all
}

__global__ void __launch_bounds__(kRankThreads)
    rank_sort_kernel(const int32_t* __restrict__ tokens, int n, int vocab,
                     int32_t* __restrict__ keys_out, int32_t* __restrict__ rows_out,
                     int32_t* __restrict__ n_long, uint32_t* status, int blocks, const Fill fill) {
  __shared__ __align__(16) int32_t key[kRankMax];
  __shared__ int below[kRankWarps][32];
  let_next_start();
  if (static_cast<int>(blockIdx.x) >= blocks) {
    fill_part(fill, blockIdx.x - blocks);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int padded = (n + 3) / 4 * 4;
  for (int i0 = threadIdx.x; i0 < padded; i0 += 8 * kRankThreads) {
    int32_t t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = i0 + j * kRankThreads < n ? tokens[i0 + j * kRankThreads] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kRankThreads;
      if (i < padded) key[i] = i < n ? sort_key(t[j], vocab) : 0x7FFFFFFF;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_long = 0;
  __syncthreads();
  const int first = blockIdx.x * 32, i = first + lane;
  const int mine = i < n ? key[i] : 0;
  // pairs with an earlier row count when their token is <= mine, later ones when < mine
  const int part = (padded / 4 + kRankWarps - 1) / kRankWarps * 4;
  const int lo = warp * part, hi = min(padded, lo + part);
  int c = 0;
  auto add = [&](int from, int to, int bar) {
#pragma unroll 4
    for (int j = from; j < to; j += 4) {
      const int4 k = *reinterpret_cast<const int4*>(key + j);
      c += ((k.x < bar) + (k.y < bar)) + ((k.z < bar) + (k.w < bar));
    }
  };
  add(lo, min(hi, first), mine + 1);
  for (int j = max(lo, first); j < min(hi, first + 32); ++j) c += key[j] < mine + (j < i);
  add(max(lo, first + 32), hi, mine);
  below[warp][lane] = c;
  __syncthreads();
  if (warp == 0 && i < n) {
    int at = 0;
#pragma unroll
    for (int w = 0; w < kRankWarps; ++w) at += below[w][lane];
    keys_out[at] = mine;
    rows_out[at] = i;
    const int32_t raw = tokens[i];
    if (raw != mine) report_status(status, kStatusBounds);
  }
}

// More rows: a stable radix sort, least significant digit first, two kernels a
// pass.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
// keys per thread: 4, so that more CTAs share few rows; 16 for many rows, as every
// CTA reads the counts of all others
constexpr int kFewBlocksMax = 1 << 18;
constexpr int kMaxBits = 9;
constexpr int kMaxBins = 1 << kMaxBits;

// counts[digit][block] of one pass
template <int kSortItems>
__global__ void __launch_bounds__(kSortThreads)
    digit_count_kernel(const int32_t* keys, int n, int vocab, int shift, int bits, int blocks,
                       int32_t* counts, int32_t* n_long, uint32_t* status, const Fill fill) {
  __shared__ int hist[kMaxBins];
  let_next_start();
  if (static_cast<int>(blockIdx.x) >= blocks) {
    fill_part(fill, blockIdx.x - blocks);
    return;
  }
  wait_for_previous();
  const int bins = 1 << bits;
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_long = 0;
  for (int i = threadIdx.x; i < bins; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  constexpr int kSortTile = kSortThreads * kSortItems;
  const int base = blockIdx.x * kSortTile;
  for (int i = base + threadIdx.x; i < min(n, base + kSortTile); i += kSortThreads) {
    const int32_t raw = keys[i], key = sort_key(raw, vocab);
    if (key != raw) report_status(status, kStatusBounds);
    atomicAdd(&hist[key >> shift & (bins - 1)], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSortThreads) counts[i * blocks + blockIdx.x] = hist[i];
}

// One stable pass.  A warp owns 32 kSortItems consecutive keys, 32 at a time; a
// key's place is the keys of smaller digits, those of its digit in earlier
// CTAs, earlier warps, earlier steps and lower lanes.
template <int kSortItems>
__global__ void __launch_bounds__(kSortThreads)
    digit_scatter_kernel(const int32_t* keys, const int32_t* rows, int n, int vocab, int shift,
                         int bits, int blocks, const int32_t* counts, int32_t* keys_out,
                         int32_t* rows_out, const Fill fill) {
  __shared__ int warp_hist[kSortWarps][kMaxBins];
  __shared__ int base[kMaxBins];
  __shared__ int scan[kSortWarps];
  let_next_start();
  if (static_cast<int>(blockIdx.x) >= blocks) {
    fill_part(fill, blockIdx.x - blocks);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bins = 1 << bits;
  for (int i = tid; i < kSortWarps * kMaxBins; i += kSortThreads) (&warp_hist[0][0])[i] = 0;
  wait_for_previous();
  // a thread per digit: its total, and its count in earlier CTAs
  int total = 0, before = 0;
  if (tid < bins)
#pragma unroll 8
    for (int b = 0; b < blocks; ++b) {
      const int c = counts[tid * blocks + b];
      total += c;
      if (b < static_cast<int>(blockIdx.x)) before += c;
    }
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int add = 0;
  for (int w = 0; w < warp; ++w) add += scan[w];
  if (tid < bins) base[tid] = add + incl - total + before;

  const int first = (blockIdx.x * kSortWarps + warp) * (32 * kSortItems);
  int32_t key[kSortItems], row[kSortItems];
  int place[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int i = first + j * 32 + lane;
    key[j] = i < n ? sort_key(keys[i], vocab) : -1;
    row[j] = i < n ? (rows ? rows[i] : i) : 0;
  }
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const int digit = key[j] >= 0 ? key[j] >> shift & (bins - 1) : -1;
    const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    int seen = 0;
    if (digit >= 0) seen = warp_hist[warp][digit];
    __syncwarp();
    if (digit >= 0 && rank == 0) warp_hist[warp][digit] = seen + __popc(peers);
    __syncwarp();
    place[j] = seen + rank;
  }
  __syncthreads();
  // exclusive over the warps, per digit
  if (tid < bins) {
    int sum = base[tid];
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = warp_hist[w][tid];
      warp_hist[w][tid] = sum;
      sum += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    if (key[j] < 0) continue;
    const int at = warp_hist[warp][key[j] >> shift & (bins - 1)] + place[j];
    keys_out[at] = key[j];
    rows_out[at] = row[j];
  }
}

// ------------------------------------------------------------------ the sums
constexpr int kMaxWindow = 32;
constexpr int kMaxLong = 64;
constexpr int kFillRows = 64;       // rows of the table per zero-filling CTA

__device__ __forceinline__ float2 block_sum2(float2 v, float2* part) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < (blockDim.x >> 5); ++w) {
    v.x += part[w].x;
    v.y += part[w].y;
  }
  return v;
}

// how many of the 64 entries from `at` on, in steps of `dir`, equal `key`
__device__ __forceinline__ int equal_run(const int* at, int dir, int key) {
  const int lane = threadIdx.x & 31;
  const uint32_t a = __ballot_sync(0xFFFFFFFFu, at[dir * lane] != key);
  const uint32_t b = __ballot_sync(0xFFFFFFFFu, at[dir * (lane + 32)] != key);
  return a ? __ffs(a) - 1 : b ? 31 + __ffs(b) : 64;
}

__device__ __forceinline__ void add4(float4& a, const float4 b) {
  a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}
__device__ __forceinline__ float4 unpack4(uint2 u) {
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

// d_emb[key] (+)= the projection of the sum g against the row h of the table;
// thread t holds float4 t, t + blockDim, ... of the row.
template <int NV>
__device__ __forceinline__ void finish_row(const float4 (&g)[NV], const uint2 (&h)[NV],
                                           const float4 (&was)[NV], bool add, float4* dst, int cols,
                                           float2* part) {
  float2 sums = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float4 e = unpack4(h[i]);
    sums.x += e.x * e.x + e.y * e.y + e.z * e.z + e.w * e.w;
    sums.y += e.x * g[i].x + e.y * g[i].y + e.z * g[i].z + e.w * g[i].w;
  }
  sums = block_sum2(sums, part);
  const bool clamped = sums.x < 1e-20f;
  const float inv = clamped ? 1e10f : 1.f / sqrtf(sums.x);
  const float proj = clamped ? 0.f : sums.y / sums.x;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = i * blockDim.x + threadIdx.x;
    if (col >= cols) continue;
    const float4 e = unpack4(h[i]);
    float4 o = make_float4((g[i].x - e.x * proj) * inv, (g[i].y - e.y * proj) * inv,
                           (g[i].z - e.z * proj) * inv, (g[i].w - e.w * proj) * inv);
    if (add) add4(o, was[i]);
    dst[col] = o;
  }
}

// Zeros into the rows of the table that no token points to: kFillRows rows a
// CTA, a binary search in the sorted tokens for each.
__device__ void fill_rows(const RunSumParams& p, int first, int* absent) {
  for (int r = threadIdx.x; r < kFillRows; r += blockDim.x) {
    int lo = 0, hi = p.n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.keys[mid] < first + r) lo = mid + 1;
      else hi = mid;
    }
    absent[r] = first + r < p.fill_rows && (lo == p.n || p.keys[lo] != first + r);
  }
  __syncthreads();
  for (int r = 0; r < kFillRows; ++r) {
    if (!absent[r]) continue;
    float4* dst = reinterpret_cast<float4*>(p.d_emb + static_cast<size_t>(first + r) * p.d);
    for (int i = threadIdx.x; i < p.d / 4; i += blockDim.x) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// One CTA per window [a, b) of the sorted list.  It finishes every run of at
// most `longest` rows that starts in the window, following it past b.  Of a
// longer run it sums its own entries only: into piece 2 w when the run comes
// from the left, into piece 2 w + 1 when it starts here (at most one does, as
// longest >= the window), and marks in more[w] whether a run from the left
// goes on to the right.  The rows a CTA reads are consecutive entries, so U of
// them (and the table rows of the runs that end among them) are loaded at once.
// Many CTAs matter more than many rows in flight in each: 64 registers a thread
// (adding spills 4 bytes of them; 16 of the 128 at four float4 a thread)
// and two rows take 249 us where 120 registers and four rows took 259 (32768 rows
// of 2048 into 131072 x 2048).
template <int NV, int U, bool Add>
__global__ void __launch_bounds__(256, NV == 1 ? (Add ? 3 : 4) : NV == 2 ? 4 : 2) run_sum_kernel(const RunSumParams p) {
  __shared__ int keys_s[kMaxWindow + 2 * kMaxLong];
  __shared__ int rows_s[kMaxWindow + kMaxLong];
  __shared__ float2 part[2][8];
  let_next_start();
  wait_for_previous();
  if (static_cast<int>(blockIdx.x) >= p.windows) {
    static_assert(kFillRows <= kMaxWindow + kMaxLong, "rows_s holds the flags");
    fill_rows(p, (blockIdx.x - p.windows) * kFillRows, rows_s);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31;
  const int a = blockIdx.x * p.window;
  int* key = keys_s + kMaxLong;            // key[i] = entry a + i, i in -64 .. window + 63
  for (int i = tid; i < p.window + 2 * kMaxLong; i += blockDim.x) {
    const int e = a + i - kMaxLong;
    const int k = e >= 0 && e < p.n ? p.keys[e] : -1;
    keys_s[i] = k < p.vocab ? k : -1;      // what is no token lies at the end: no entry
  }
  for (int i = tid; i < p.window + kMaxLong; i += blockDim.x)
    rows_s[i] = a + i < p.n ? p.rows[a + i] : 0;
  __syncthreads();
  const int size = __popc(__ballot_sync(0xFFFFFFFFu, lane < p.window && key[lane] >= 0));
  if (size == 0) return;
  // the run that comes from the left, and the one that holds the last entry
  const int from_left = equal_run(key - 1, -1, key[0]), here = equal_run(key, 1, key[0]);
  const bool left_long = from_left > 0 && from_left + here > p.longest;
  int e0 = 0, e1 = size;
  bool right_long = false;
  if (from_left > 0 && !left_long) e0 = min(here, size);   // an earlier window's
  if (here < size || from_left == 0) {
    const int last = size - 1;
    const int back = equal_run(key + last, -1, key[last]);
    const int ahead = equal_run(key + size, 1, key[last]);
    right_long = back + ahead > p.longest;
    if (!right_long) e1 = size + ahead;
  }
  if (tid == 0) {
    p.more[blockIdx.x] = left_long && here > size;
    if (right_long) {
      const int at = atomicAdd(p.n_long, 1);   // in any order: each run is summed by itself
      p.long_runs[at] = blockIdx.x;
      p.slices_done[at] = 0;
    }
  }

  const int cols = p.d / 4;
  float4 g[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  int turn = 0;
  for (int e = e0; e < e1; e += U) {
    float4 u[U][NV], was[U][NV];
    uint2 h[U][NV];
    // what each of the U entries ends: 0 nothing, 1 a run to finish, 2 / 3 a piece
    int ends[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int x = e + j;
      ends[j] = 0;
      if (x >= e1) continue;
      if (x == e1 - 1 || key[x] != key[x + 1])
        ends[j] = left_long && key[x] == key[0] ? 2 : right_long && x == e1 - 1 ? 3 : 1;
      const float4* src = reinterpret_cast<const float4*>(p.src + static_cast<size_t>(rows_s[x]) * p.d);
      const uint2* emb = reinterpret_cast<const uint2*>(p.emb + static_cast<size_t>(key[x]) * p.d);
      const float4* old = reinterpret_cast<const float4*>(p.d_emb + static_cast<size_t>(key[x]) * p.d);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = i * blockDim.x + tid;
        u[j][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        h[j][i] = make_uint2(0u, 0u);
        if (col < cols) {
          u[j][i] = src[col];
          if (ends[j] == 1) {
            h[j][i] = emb[col];
            if (Add) was[j][i] = old[col];
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (e + j >= e1) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i) add4(g[i], u[j][i]);
      if (ends[j] == 0) continue;
      if (ends[j] == 1) {
        finish_row<NV>(g, h[j], was[j], Add,
                       reinterpret_cast<float4*>(p.d_emb + static_cast<size_t>(key[e + j]) * p.d), cols,
                       part[turn++ & 1]);
      } else {
        float4* dst = reinterpret_cast<float4*>(
            p.pieces + (2 * static_cast<size_t>(blockIdx.x) + (ends[j] - 2)) * p.d);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int col = i * blockDim.x + tid;
          if (col < cols) dst[col] = g[i];
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// The long runs: 64 columns of one run's pieces a time, 16 threads across and 16
// down; the CTA that completes the run's last columns finishes the row.  The
// pieces are joined in 64 bits: a run may have n / 32 of them, and a chain of so
// many additions in 32 bits can drift by more than a window's sum ever does.
constexpr int kJoinThreads = 256;
constexpr int kJoinCols = 64;

struct Sum4 {
  double x = 0.0, y = 0.0, z = 0.0, w = 0.0;
  __device__ __forceinline__ void add(const float4 b) {
    x += b.x; y += b.y; z += b.z; w += b.w;
  }
};

template <int NV>
__global__ void __launch_bounds__(kJoinThreads) long_run_kernel(const RunSumParams p) {
  __shared__ double sums[16][4][16];
  __shared__ float2 part[8];
  __shared__ int n_pieces, last;
  wait_for_previous();
  const int tid = threadIdx.x, x = tid & 15, y = tid >> 4;
  const int slices = p.d / kJoinCols, items = *p.n_long * slices;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int run = item / slices, w = p.long_runs[run], col = (item - run * slices) * (kJoinCols / 4) + x;
    // pieces: 2 w + 1, then 2 j of the windows up to the first that is not passed through
    if (tid == 0) n_pieces = 0x7FFFFFFF;
    __syncthreads();
    for (int j = w + 1 + tid;; j += kJoinThreads) {
      const bool stop = j >= p.windows || !p.more[j];
      if (stop) atomicMin(&n_pieces, min(j, p.windows - 1) - w + 1);
      if (__syncthreads_or(stop)) break;
    }
    const int n = n_pieces;
    const float4* pieces = reinterpret_cast<const float4*>(p.pieces);
    const size_t cols = p.d / 4;
    Sum4 s;
    for (int k0 = y; k0 < n; k0 += 64) {
      float4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = k0 + q * 16;
        v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < n) v[q] = pieces[(2 * static_cast<size_t>(w + k) + (k == 0)) * cols + col];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) s.add(v[q]);
    }
    sums[y][0][x] = s.x;
    sums[y][1][x] = s.y;
    sums[y][2][x] = s.z;
    sums[y][3][x] = s.w;
    __syncthreads();
    if (y < 4) {   // a thread per column
      double sum = 0.0;
      for (int k = 0; k < 16; ++k) sum += sums[k][y][x];
      p.long_sums[static_cast<size_t>(run) * p.d + col * 4 + y] = static_cast<float>(sum);
      __threadfence();
    }
    __syncthreads();
    if (tid == 0) {
      // the count returns to zero with the last slice
      last = atomicInc(reinterpret_cast<unsigned int*>(p.slices_done + run), slices - 1) ==
             static_cast<unsigned int>(slices - 1);
      __threadfence();
    }
    __syncthreads();
    if (last) {
      const int key = p.keys[static_cast<size_t>(w + 1) * p.window];
      const float4* src = reinterpret_cast<const float4*>(p.long_sums) + static_cast<size_t>(run) * cols;
      const uint2* emb = reinterpret_cast<const uint2*>(p.emb + static_cast<size_t>(key) * p.d);
      float4* dst = reinterpret_cast<float4*>(p.d_emb + static_cast<size_t>(key) * p.d);
      float4 g[NV], was[NV];
      uint2 h[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * kJoinThreads + tid;
        g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        h[i] = make_uint2(0u, 0u);
        if (c < static_cast<int>(cols)) {
          g[i] = __ldcg(src + c);
          h[i] = emb[c];
          if (p.accumulate) was[i] = dst[c];
        }
      }
      finish_row<NV>(g, h, was, p.accumulate, dst, cols, part);
    }
    __syncthreads();   // shared memory is used again
  }
}

// Windows short enough to fill the GPU several times over with few rows, long
// enough that few runs are cut with many.
int run_window(int n, int num_sms) {
  int w = 4;
  while (w < kMaxWindow && n / w > 8 * num_sms) w *= 2;
  return w;
}

// Rows that one CTA still sums by itself: a longer run is spread over its windows.
int longest_run(int window) { return window * 2 < 16 ? 16 : window * 2; }

struct EmbedBwdLayout {
  size_t keys[2], rows[2], counts, n_long, long_runs, slices_done, more, pieces, long_sums;
  size_t total;
};
int sort_items(int n) { return n <= kFewBlocksMax ? 4 : 16; }
int sort_blocks(int n) { return (n + kSortThreads * sort_items(n) - 1) / (kSortThreads * sort_items(n)); }

EmbedBwdLayout embed_bwd_layout(int n, int d, int num_sms) {
  EmbedBwdLayout L;
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  const int window = run_window(n, num_sms), windows = (n + window - 1) / window;
  const int longs = n / (longest_run(window) + 1);    // at most so many long runs
  for (int i = 0; i < 2; ++i) {
    L.keys[i] = take(size_t(n) * 4);
    L.rows[i] = take(size_t(n) * 4);
  }
  L.counts = n > kRankMax ? take(size_t(sort_blocks(n)) * kMaxBins * 4) : 0;
  L.n_long = take(4);
  L.long_runs = take(size_t(longs) * 4);
  L.slices_done = take(size_t(longs) * 4);
  L.more = take(windows);
  L.pieces = take(size_t(2) * windows * d * 4);
  L.long_sums = take(size_t(longs) * d * 4);
  L.total = o;
  return L;
}

template <bool Add>
void run_sum_launch(const RunSumParams& p, bool early, int grid, int threads, cudaStream_t s) {
  switch ((p.d / 4 + threads - 1) / threads) {
    case 1: launch_next(early, run_sum_kernel<1, 4, Add>, grid, threads, s, p); break;
    case 2: launch_next(early, run_sum_kernel<2, 2, Add>, grid, threads, s, p); break;
    case 3: launch_next(early, run_sum_kernel<3, 2, Add>, grid, threads, s, p); break;
    default: launch_next(early, run_sum_kernel<4, 2, Add>, grid, threads, s, p); break;
  }
}

// Hands out parts of the region [0, rows) of the table, from its end.
struct FillPlan {
  float* table;
  int d;
  int rows;   // still to be filled
  Fill take(size_t bytes) {
    const size_t row = size_t(d) * 4;
    const int n = static_cast<int>(bytes / row < size_t(rows) ? bytes / row : size_t(rows));
    rows -= n;
    return {reinterpret_cast<float4*>(table + size_t(rows) * d), n * row / 16};
  }
};
// what is written while a launch of the sort runs
constexpr size_t kFillRank = 40u << 20, kFillCount = 16u << 20, kFillScatter = 40u << 20;

template <int Items>
void sort_pass(const int32_t* keys, const int32_t* rows, int n, int vocab, int shift, int bits,
               int blocks, int32_t* counts, int32_t* keys_out, int32_t* rows_out, int32_t* n_long,
               uint32_t* status, FillPlan& plan, bool early, bool first, cudaStream_t s) {
  Fill f = plan.take(kFillCount);
  launch_next(early && !first, digit_count_kernel<Items>, blocks + fill_ctas(f), kSortThreads, s, keys, n, vocab,
              shift, bits, blocks, counts, n_long, status, f);
  f = plan.take(kFillScatter);
  launch_next(early, digit_scatter_kernel<Items>, blocks + fill_ctas(f), kSortThreads, s, keys, rows, n, vocab,
              shift, bits, blocks, counts, keys_out, rows_out, f);
}

}  // namespace

size_t embed_bwd_workspace_bytes(int n, int d, int num_sms) {
  return embed_bwd_layout(n, d, num_sms).total;
}

cudaError_t launch_embed_bwd(const __nv_bfloat16* table, int vocab, int d, const int32_t* tokens,
                             int n, const float* dh, float* d_emb, int accumulate, void* ws,
                             int num_sms, uint32_t* status, cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  if (d % 128 != 0 || d > 4096) return cudaErrorInvalidValue;
  const EmbedBwdLayout L = embed_bwd_layout(n, d, num_sms);
  uint8_t* b = static_cast<uint8_t*>(ws);
  auto ints = [b](size_t at) { return reinterpret_cast<int32_t*>(b + at); };

  int32_t *keys = ints(L.keys[0]), *rows = ints(L.rows[0]), *n_long = ints(L.n_long);
  FillPlan plan{d_emb, d, accumulate ? 0 : vocab};
  // 32768 rows of 2048 added: 142 us for 150, from a few tokens 90 for 100.  Not
  // where zeros are written beside the sort (273 for 268: the next kernel's CTAs
  // take their place), and not after the rank sort (8192 rows 68 for 64: they come
  // to lie unevenly on the SMs it leaves).  The joining always starts early.
  const bool early = accumulate && n > kRankMax;
  if (n <= kRankMax) {
    const int blocks = (n + 31) / 32;
    const Fill f = plan.take(kFillRank);
    rank_sort_kernel<<<blocks + fill_ctas(f), kRankThreads, 0, s>>>(tokens, n, vocab, keys, rows, n_long,
                                                                    status, blocks, f);
  } else {
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;   // keys are 0..vocab
    const int passes = (bits + kMaxBits - 1) / kMaxBits, step = (bits + passes - 1) / passes;
    for (int i = 0; i < passes; ++i) {
      const int32_t *from = i ? keys : tokens, *from_rows = i ? rows : nullptr;
      keys = ints(L.keys[i & 1]);
      rows = ints(L.rows[i & 1]);
      (sort_items(n) == 4 ? sort_pass<4> : sort_pass<16>)(
          from, from_rows, n, vocab, i * step, step, sort_blocks(n), ints(L.counts), keys, rows,
          n_long, i == 0 ? status : nullptr, plan, early, i == 0, s);
    }
  }

  RunSumParams p;
  p.keys = keys;
  p.rows = rows;
  p.src = dh;
  p.n = n;
  p.d = d;
  p.vocab = vocab;
  p.emb = table;
  p.d_emb = d_emb;
  p.accumulate = accumulate;
  p.window = run_window(n, num_sms);
  p.windows = (n + p.window - 1) / p.window;
  p.longest = longest_run(p.window);
  p.n_long = n_long;
  p.long_runs = ints(L.long_runs);
  p.slices_done = ints(L.slices_done);
  p.more = b + L.more;
  p.pieces = reinterpret_cast<float*>(b + L.pieces);
  p.long_sums = reinterpret_cast<float*>(b + L.long_sums);
  // half the threads up to 1024 columns: barriers of fewer warps, twice the windows
  // in flight (32768 rows of 1024 added: 92 us for 100; a quarter of them 92)
  const int threads = d > 1024 ? 256 : d > 512 ? 128 : d / 4;
  p.fill_rows = plan.rows;   // the rest, beside the sums: rows without a token only
  const int grid = p.windows + (p.fill_rows + kFillRows - 1) / kFillRows;
  if (accumulate) run_sum_launch<true>(p, early, grid, threads, s);
  else run_sum_launch<false>(p, early, grid, threads, s);
  const long long items = static_cast<long long>(n / (p.longest + 1)) * (d / kJoinCols);
  if (items > 0) {
    const int blocks = static_cast<int>(items < 8 * num_sms ? items : 8 * num_sms);
    switch ((d / 4 + kJoinThreads - 1) / kJoinThreads) {
      case 1: launch_next(true, long_run_kernel<1>, blocks, kJoinThreads, s, p); break;
      case 2: launch_next(true, long_run_kernel<2>, blocks, kJoinThreads, s, p); break;
      case 3: launch_next(true, long_run_kernel<3>, blocks, kJoinThreads, s, p); break;
      default: launch_next(true, long_run_kernel<4>, blocks, kJoinThreads, s, p); break;
    }
  }
  return cudaGetLastError();
}

}  // namespace dory
