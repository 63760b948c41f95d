// The K largest logits of each row, with their tokens, and the row's
// log-sum-exp.  Order: value descending, token ascending among equal values
// (-0 equals +0); a NaN ranks below -inf.
//
// One pass over the row keeps the maximum of every group of consecutive logits.
// Let T be the K-th largest of these maxima.  K groups hold a value >= T, so the
// K-th largest logit is >= T, and a group whose maximum is below T holds none of
// the top K.  Of the groups with maximum exactly T only the first (by token) are
// needed: if c groups exceed T, at most K - c of the answers equal T, and each
// such group holds at least one.  So the logits of K groups decide the row,
// whatever its values.
//
// Bound: HBM, one read of the logits; with few rows the searches behind it, with
// short rows the instructions of the pass.  2048 rows of 131072: 1 answer 168 us,
// 64 answers 185, 256 answers 240 (floor 164: the reads of the K groups and the
// sort, one row's tail hidden by the other rows on its SM), 64 answers among ties
// 207; 4096 x 32768, 64 answers, 125 us (floor 82); one row of 131072 with 20
// answers 10 us, 148 of them 21 (floor 12).  Sorting or selecting on whole rows
// needs them read more than once or kept on chip; group maxima need a 32nd.
#include <string.h>

#include "kernels.h"
#include "vocab_ops.cuh"

namespace dory {

namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;

// log of a sum of exponentials; log2 s over the fp32 constant that scaled the
// differences, so that its rounding (nearly) cancels
__device__ __forceinline__ float log_of(const ExpSum& a) {
  return static_cast<float>(static_cast<double>(exp_ref(a.m)) +
                            static_cast<double>(log2f(a.s)) / static_cast<double>(kLog2e));
}

// A candidate: its key, then the lower token first.
__device__ __forceinline__ uint64_t word_of(uint32_t key, int token) {
  return static_cast<uint64_t>(key) << 32 | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ void put(float* values, int32_t* tokens, size_t at, uint64_t w) {
  values[at] = key_value(static_cast<uint32_t>(w >> 32));
  tokens[at] = static_cast<int32_t>(~static_cast<uint32_t>(w));
}

// One step of a bitonic sort into descending order, by kT threads.
template <int kT>
__device__ __forceinline__ void bitonic_step(uint64_t* list, int n, int size, int stride, int tid) {
  for (int i = tid; i < n / 2; i += kT) {
    const int a = 2 * i - (i & (stride - 1)), b = a + stride;
    const uint64_t x = list[a], y = list[b];
    if ((x < y) == ((a & size) == 0)) {
      list[a] = y;
      list[b] = x;
    }
  }
}

// Up to 32 kR words of a list into descending order in a warp's registers (lane l
// holds words l kR .. l kR + kR - 1), and the first k of them written.
template <int kR>
__device__ __noinline__ void sort_words(const uint64_t* list, int m, int k, float* values,
                                           int32_t* tokens, size_t at) {
  const int lane = threadIdx.x & 31;
  uint64_t w[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) w[r] = r * 32 + lane < m ? list[r * 32 + lane] : 0u;   // in any order
#pragma unroll
  for (int size = 2; size <= 32 * kR; size *= 2) {
#pragma unroll
    for (int d = size / 2; d > 0; d /= 2) {
      if (d >= kR) {
        const bool upper = lane & (d / kR);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const uint64_t y = __shfl_xor_sync(kFull, w[r], d / kR);
          const bool down = ((lane * kR + r) & size) == 0;
          w[r] = (w[r] < y) == (upper != down) ? y : w[r];
        }
      } else {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          if (r & d) continue;
          const bool down = ((lane * kR + r) & size) == 0;
          const uint64_t x = w[r], y = w[r | d];
          const bool swap = (x < y) == down;
          w[r] = swap ? y : x;
          w[r | d] = swap ? x : y;
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kR; ++r)
    if (lane * kR + r < k) put(values, tokens, at + lane * kR + r, w[r]);
}
// ------------------------------------------------------------- a warp per row
// Rows of at most 128 kNF logits stay in registers, as keys.  Up to kByGroup
// answers are found through groups of four; for more, the K-th largest logit
// itself.  No CTA barrier between a row's steps: 32768 rows of 1024 with 20
// answers take 74 us (floor 21; bound by instructions, mostly the threshold's
// search), 20000 of 1536 with 64 answers 103 (floor 20).
constexpr int kRowWarps = 4;    // per CTA
constexpr int kByGroup = 64;    // 4 * kByGroup candidates fit the list

// T: the highest threshold that at least k of the warp's keys reach, from the
// highest bit down, or one that exactly k reach; returns how many do.  `all` >= k
// keys are there, the others are 0.
template <int kN>
__device__ __forceinline__ int warp_kth(const uint32_t (&key)[kN], uint32_t lo, int all, int k, uint32_t& T) {
  uint32_t hi = 0u;
#pragma unroll
  for (int i = 0; i < kN; ++i) hi = max(hi, key[i]);
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi);
  T = lo;
  if (all == k || lo == hi) return all;
  int bit = 31 - __clz(lo ^ hi), reach = all;
  T = hi >> bit >> 1 << 1 << bit;
  for (; bit >= 0 && reach != k; --bit) {
    const uint32_t cand = T | 1u << bit;
    int c = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) c += key[i] >= cand;
    c = __reduce_add_sync(kFull, c);
    if (c >= k) {
      T = cand;
      reach = c;
    }
  }
  return reach;
}
// how many of the keys equal to T are wanted: all, or, where more than k reach
// T, what the larger ones leave of k
template <int kN>
__device__ __forceinline__ int warp_ties(const uint32_t (&key)[kN], uint32_t T, int reach, int k) {
  if (reach <= k) return 0x7FFFFFFF;
  int above = 0;
#pragma unroll
  for (int i = 0; i < kN; ++i) above += key[i] > T;
  return k - __reduce_add_sync(kFull, above);
}

template <int kNF>
__global__ void __launch_bounds__(kRowWarps * 32)
    top_warp_kernel(const float* __restrict__ logits, int n, int vocab, int k,
                    float* __restrict__ values, int32_t* __restrict__ tokens, float* __restrict__ lse) {
  __shared__ uint64_t lists[kRowWarps][kTopMax];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kRowWarps + warp;
  if (row >= n) return;
  uint64_t* list = lists[warp];
  const float* z = logits + static_cast<size_t>(row) * vocab;
  const int groups = vocab / 4;
  uint32_t key[4 * kNF], top[kNF], lo = kFull, lo_top = kFull;
  {
    float4 x[kNF];
#pragma unroll
    for (int i = 0; i < kNF; ++i) {
      const int g = i * 32 + lane;
      x[i] = g < groups ? reinterpret_cast<const float4*>(z)[g]
                        : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    ExpSum acc = {-INFINITY, 0.f};
    exp_add(acc, x, kLog2e);
    acc = warp_join(acc, kLog2e);
    if (lane == 0) lse[row] = log_of(acc);
#pragma unroll
    for (int i = 0; i < kNF; ++i) {
      const bool in = i * 32 + lane < groups;
      uint32_t* q = key + 4 * i;
      q[0] = in ? order_key(x[i].x) : 0u;
      q[1] = in ? order_key(x[i].y) : 0u;
      q[2] = in ? order_key(x[i].z) : 0u;
      q[3] = in ? order_key(x[i].w) : 0u;
      top[i] = max(max(q[0], q[1]), max(q[2], q[3]));
      if (in) {
        lo = min(lo, min(min(q[0], q[1]), min(q[2], q[3])));
        lo_top = min(lo_top, top[i]);
      }
    }
  }
  const uint32_t below = (1u << lane) - 1u;
  uint64_t pick = 0u;   // bit 4 i + q: the logit is a candidate
  int tied = 0;
  uint32_t T;
  if (k <= kByGroup) {
    const int reach = warp_kth(top, lo_top, groups, k, T), ties = warp_ties(top, T, reach, k);
#pragma unroll
    for (int i = 0; i < kNF; ++i) {
      const bool in = i * 32 + lane < groups, eq = in && top[i] == T;
      const uint32_t eqs = __ballot_sync(kFull, eq);
      if (in && (top[i] > T || (eq && tied + __popc(eqs & below) < ties))) {
#pragma unroll
        for (int q = 0; q < 4; ++q) pick |= static_cast<uint64_t>(key[4 * i + q] >= T) << (4 * i + q);
      }
      tied += __popc(eqs);
    }
  } else {
    const int reach = warp_kth(key, lo, vocab, k, T), ties = warp_ties(key, T, reach, k);
#pragma unroll
    for (int i = 0; i < kNF; ++i) {
      const bool in = i * 32 + lane < groups;
      uint32_t eqs[4];
      int before = tied;   // equal ones of smaller tokens
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        eqs[q] = __ballot_sync(kFull, in && key[4 * i + q] == T);
        before += __popc(eqs[q] & below);
        tied += __popc(eqs[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool eq = eqs[q] >> lane & 1u;
        if (in && (key[4 * i + q] > T || (eq && before < ties))) pick |= 1ull << (4 * i + q);
        before += eq;
      }
    }
  }
  int m = 0;
#pragma unroll
  for (int i = 0; i < kNF; ++i) {
    if (!__any_sync(kFull, (pick >> (4 * i) & 15u) != 0u)) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool take = pick >> (4 * i + q) & 1u;
      const uint32_t b = __ballot_sync(kFull, take);
      if (take) list[m + __popc(b & below)] = word_of(key[4 * i + q], (i * 32 + lane) * 4 + q);
      m += __popc(b);
    }
  }
  __syncwarp();
  const size_t at = static_cast<size_t>(row) * k;
  if (m > 128) {
    sort_words<8>(list, m, k, values, tokens, at);
  } else if (m > 64) {
    sort_words<4>(list, m, k, values, tokens, at);
  } else {
    // a word's place is the number of larger words
    for (int i = lane; i < m; i += 32) {
      const uint64_t w = list[i];
      int place = 0;
      for (int j = 0; j < m; ++j) place += list[j] > w;
      if (place < k) put(values, tokens, at + place, w);
    }
  }
}

// ------------------------------------- a CTA, or a cluster of CTAs, per row
constexpr int kGroup = 32;
constexpr int kMaxCluster = 8;
constexpr int kKeep = 16;       // group maxima per thread kept in registers
constexpr int kListMax = 512;   // candidates sorted at once; more are cut to k first

// Sum of a per-thread count over the CTA through slot[0..3], used in turn.
__device__ __forceinline__ int block_count(int c, int* slot, int turn) {
  c = __reduce_add_sync(kFull, c);
  if ((threadIdx.x & 31) == 0 && c) atomicAdd(&slot[turn & 3], c);
  if (threadIdx.x == 0) slot[(turn + 2) & 3] = 0;
  __syncthreads();
  return slot[turn & 3];
}

// the address of `local` in the first CTA of the cluster
__device__ __forceinline__ uint32_t in_first_cta(const void* local) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(local)));
  return a;
}

// Where the rows are few, a cluster of CTAs per row shares the pass over the
// logits and the first of them decides.  Rows of up to 16384 logits take 128
// threads, so that more of them are on an SM while each waits for its barriers
// (8192 x 16384, 64 answers: 139 us, floor 83), longer ones 256.
template <int kT, bool kCluster>
__global__ void __launch_bounds__(kT)
    top_kernel(const float* __restrict__ logits, int vocab, int k, int cluster,
               float* __restrict__ values, int32_t* __restrict__ tokens, float* __restrict__ lse) {
  constexpr int kWarps = kT / 32;
  extern __shared__ __align__(16) uint32_t gmax[];    // [groups]
  __shared__ uint64_t list[kListMax];
  __shared__ int glist[kTopMax];
  __shared__ float2 part[kWarps * (kCluster ? kMaxCluster : 1)];
  __shared__ uint32_t ends[2 * kWarps];
  __shared__ int slot[4];
  __shared__ int n_groups, n_list;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = vocab / kGroup;
  const int row = kCluster ? blockIdx.x / cluster : blockIdx.x;
  const int rank = kCluster ? blockIdx.x - row * cluster : 0;
  const float* z = logits + static_cast<size_t>(row) * vocab;
  if (kCluster) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // this CTA runs
  bool first_runs = !kCluster;
  const uint32_t gmax_at = kCluster ? in_first_cta(gmax) : 0u;
  if (tid == 0) {
    n_groups = 0;
    n_list = 0;
  }
  if (tid < 4) slot[tid] = 0;

  // A warp takes 1024 consecutive logits, 8 loads of 512 bytes; lane l holds four
  // of group 4 j + l / 8 of load j.  The 8 lanes of a group exchange halves of
  // their 8 maxima three times, so 7 shuffles finish 32 groups.
  ExpSum acc = {-INFINITY, 0.f};
  uint32_t lo = kFull, hi = 0u;
  for (int t0 = (rank * kWarps + warp) * 1024; t0 < vocab; t0 += kWarps * cluster * 1024) {
    float4 x[8];
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int v = t0 + j * 128 + lane * 4;
      x[j] = v < vocab ? *reinterpret_cast<const float4*>(z + v)
                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = max4(x[j]);
    exp_add(acc, x, kLog2e);
    const bool b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float give = b2 ? m[j] : m[j + 4], keep = b2 ? m[j + 4] : m[j];
      m[j] = fmaxf(keep, __shfl_xor_sync(kFull, give, 4));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float give = b1 ? m[j] : m[j + 2], keep = b1 ? m[j + 2] : m[j];
      m[j] = fmaxf(keep, __shfl_xor_sync(kFull, give, 2));
    }
    const float give = b0 ? m[0] : m[1], keep = b0 ? m[1] : m[0];
    const uint32_t key = order_key(fmaxf(keep, __shfl_xor_sync(kFull, give, 1)));
    const int g = t0 / kGroup + (lane & 7) * 4 + (lane >> 3);
    if (kCluster) {
      if (!first_runs) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      first_runs = true;
      if (g < groups) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(gmax_at + g * 4), "r"(key) : "memory");
    } else if (g < groups) {
      gmax[g] = key;
      lo = min(lo, key);
      hi = max(hi, key);
    }
  }
  acc = warp_join(acc, kLog2e);
  if (kCluster) {
    if (!first_runs) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (lane == 0)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(in_first_cta(&part[rank * kWarps + warp])),
                   "f"(acc.m), "f"(acc.s) : "memory");
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    for (int i = tid; i < groups; i += kT) {
      lo = min(lo, gmax[i]);
      hi = max(hi, gmax[i]);
    }
  } else if (lane == 0) {
    part[warp] = make_float2(acc.m, acc.s);
  }
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi);
  if (lane == 0) {
    ends[warp] = lo;
    ends[kWarps + warp] = hi;
  }
  __syncthreads();
  if (warp == kWarps - 1) {
    acc = {-INFINITY, 0.f};
    for (int w = lane; w < kWarps * cluster; w += 32) acc = exp_join(acc, {part[w].x, part[w].y}, kLog2e);
    acc = warp_join(acc, kLog2e);
    if (lane == 31) lse[row] = log_of(acc);
  }
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo = min(lo, ends[w]);
    hi = max(hi, ends[kWarps + w]);
  }

  // T: the highest threshold that at least k group maxima reach, from the highest
  // bit down, or one that exactly k reach
  uint32_t T = groups < k ? 0u : lo;
  int reach = groups;
  if (groups > k && lo != hi) {
    int bit = 31 - __clz(lo ^ hi);
    T = hi >> bit >> 1 << 1 << bit;
    uint32_t mine[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) mine[i] = i * kT + tid < groups ? gmax[i * kT + tid] : 0u;
    for (int turn = 0; bit >= 0 && reach != k; --bit, ++turn) {
      const uint32_t cand = T | 1u << bit;
      int c = 0;
#pragma unroll
      for (int i = 0; i < kKeep; ++i) c += mine[i] >= cand;
      for (int i = kKeep * kT + tid; i < groups; i += kT) c += gmax[i] >= cand;
      c = block_count(c, slot, turn);
      if (c >= k) {
        T = cand;
        reach = c;
      }
    }
  }
  if (reach <= k) {
    for (int g = tid; g < groups; g += kT)
      if (gmax[g] >= T) glist[atomicAdd(&n_groups, 1)] = g;
  } else {
    // more than k reach T, so T is the exact k-th maximum: the groups above it,
    // then the first ones equal to it
    for (int g = tid; g < groups; g += kT)
      if (gmax[g] > T) glist[atomicAdd(&n_groups, 1)] = g;
    __syncthreads();
    if (warp == 0) {
      int at = n_groups;
      for (int g0 = 0; g0 < groups && at < k; g0 += 32) {
        const bool eq = g0 + lane < groups && gmax[g0 + lane] == T;
        const uint32_t ball = __ballot_sync(kFull, eq);
        const int mine = at + __popc(ball & ((1u << lane) - 1u));
        if (eq && mine < k) glist[mine] = g0 + lane;
        at += __popc(ball);
      }
      if (lane == 0) n_groups = min(at, k);
    }
  }
  __syncthreads();

  // Their logits >= T.  A warp looks at every kWarps-th group of the list, 8 at a
  // time; what finds no room in the list is counted all the same.
  const int ng = n_groups;
  auto each_logit = [&](auto&& take) {
    for (int i = warp; i < ng; i += kWarps * 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = i + j * kWarps < ng ? z[glist[i + j * kWarps] * kGroup + lane] : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j * kWarps < ng) take(word_of(order_key(v[j]), glist[i + j * kWarps] * kGroup + lane));
    }
  };
  auto collect = [&](uint64_t bar) {
    each_logit([&](uint64_t w) {
      const bool take = w >= bar;
      const uint32_t ball = __ballot_sync(kFull, take);
      if (!ball) return;
      int base = 0;
      if (lane == 0) base = atomicAdd(&n_list, __popc(ball));
      base = __shfl_sync(kFull, base, 0) + __popc(ball & ((1u << lane) - 1u));
      if (take && base < kListMax) list[base] = w;
    });
    __syncthreads();
  };
  collect(static_cast<uint64_t>(T) << 32);
  int n = n_list;
  if (n > kListMax) {
    // answers crowded into few groups: cut to the k largest words, which all
    // differ, bit by bit over the groups' logits (read again, from L1 or L2)
    __syncthreads();
    if (tid < 4) slot[tid] = 0;
    if (tid == 0) n_list = 0;
    __syncthreads();
    int have = n;
    uint64_t bar = 0u;
    for (int bit = 63, turn = 0; bit >= 0 && have != k; --bit, ++turn) {
      const uint64_t cand = bar | 1ull << bit;
      int c = 0;
      each_logit([&](uint64_t w) { c += w >= cand; });
      c = block_count(c, slot, turn);
      if (c >= k) {
        bar = cand;
        have = c;
      }
    }
    collect(bar);
    n = n_list;
  }
  const size_t at = static_cast<size_t>(row) * k;
  if (n <= 128) {
    // a word's place is the number of larger words
    for (int i = tid; i < n; i += kT) {
      const uint64_t w = list[i];
      int place = 0;
      for (int j = 0; j < n; ++j) place += list[j] > w;
      if (place < k) put(values, tokens, at + place, w);
    }
    return;
  }
  int size = 256;
  while (size < n) size *= 2;
  for (int i = n + tid; i < size; i += kT) list[i] = 0u;
  __syncthreads();
  for (int s = 2; s <= size; s *= 2)
    for (int d = s / 2; d > 0; d /= 2) {
      bitonic_step<kT>(list, size, s, d, tid);
      __syncthreads();
    }
  for (int i = tid; i < k; i += kT) put(values, tokens, at + i, list[i]);
}

template <int kT, bool kCluster>
cudaError_t launch_row(const float* logits, int n, int vocab, int k, int cluster, float* values,
                       int32_t* tokens, float* lse, cudaStream_t s) {
  auto* kern = top_kernel<kT, kCluster>;
  static uint32_t attr_done = 0;   // per instantiation, one bit per device < 32
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(attr_done & (1u << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTopMaxVocab / kGroup * 4);
    if (e != cudaSuccess) return e;
    if (dev < 32) attr_done |= 1u << dev;
  }
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(n * cluster);
  cfg.blockDim = dim3(kT);
  cfg.dynamicSmemBytes = vocab / kGroup * 4;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, logits, vocab, k, cluster, values, tokens, lse);
}

template <int kNF>
cudaError_t launch_warps(const float* logits, int n, int vocab, int k, float* values,
                         int32_t* tokens, float* lse, cudaStream_t s) {
  top_warp_kernel<kNF><<<(n + kRowWarps - 1) / kRowWarps, kRowWarps * 32, 0, s>>>(
      logits, n, vocab, k, values, tokens, lse);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_top(const float* logits, int n, int vocab, int k, float* values,
                       int32_t* tokens, float* lse, int num_sms, cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  if (vocab % 256 != 0 || vocab > kTopMaxVocab || k < 1 || k > kTopMax || k > vocab)
    return cudaErrorInvalidValue;
  if (vocab <= 1024) return launch_warps<8>(logits, n, vocab, k, values, tokens, lse, s);
  if (vocab <= 2048) return launch_warps<16>(logits, n, vocab, k, values, tokens, lse, s);
  // as many CTAs per row as leave no SM without one, with at least 8192 logits each
  int cluster = 1;
  while (cluster < kMaxCluster && n * cluster < num_sms && vocab >= 2 * cluster * 8192) cluster *= 2;
  if (cluster > 1) return launch_row<256, true>(logits, n, vocab, k, cluster, values, tokens, lse, s);
  if (vocab <= 16384) return launch_row<128, false>(logits, n, vocab, k, 1, values, tokens, lse, s);
  return launch_row<256, false>(logits, n, vocab, k, 1, values, tokens, lse, s);
}

}  // namespace dory
