// Logits between the LM head and the sampler: penalties for repeated tokens,
// per-row biases and an allowed-token mask.
//   seen(v)  = token v occurs in the row's history, c(v) = times it occurs in
//              the part behind the prompt
//   z1 = seen ? (z > 0 ? z / r : z * r) : z
//   z2 = c > 0 ? z1 - (f c + p) : z1
//   z3 = z2 + sum of the row's biases of v
//   out = allowed(v) ? z3 : -inf
#include "kernels.h"
#include "vocab_ops.cuh"

namespace dory {

namespace {

constexpr int kLoads = 4;                // 16-byte history loads in flight per thread

// Start bringing `bytes` (a multiple of 16) from 16-byte aligned `src` into L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// What a table cell says of a token: 0 = not in the history, all ones = in the
// prompt only, otherwise its count behind the prompt.  16-bit cells serve
// histories of up to kMaxShort entries, so that a CTA's table spans twice the
// tokens; longer ones take 32 bits.
constexpr int kMaxShort = 0xFFFE;
template <typename Cell>
__device__ __forceinline__ void count_token(uint32_t* table, uint32_t at) {
  if (sizeof(Cell) == 4) atomicAdd(&table[at], 1u);
  else atomicAdd(&table[at >> 1], 1u << (at << 4 & 16));
}
template <typename Cell>
__device__ __forceinline__ uint4 cells4(const Cell* cell) {
  if (sizeof(Cell) == 4) return *reinterpret_cast<const uint4*>(cell);
  const uint2 c = *reinterpret_cast<const uint2*>(cell);
  return make_uint4(c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16);
}

// Branch-free, and a product with 1 / r in place of the division (one more
// rounding): with a long history nearly every warp has a token to change.
struct Penalty {
  float r, inv, f, p;
};
template <typename Cell>
__device__ __forceinline__ float penalised(float z, uint32_t c, const Penalty& w) {
  const float y = z * (z > 0.f ? w.inv : w.r);
  const float off = c != static_cast<Cell>(~Cell(0)) ? fmaf(w.f, static_cast<float>(c), w.p) : 0.f;
  return c ? y - off : z;
}

// `one` for entries [from, to) of a history, spread over the CTA; returns the
// thread's largest token.
template <int kThreads, typename Op>
__device__ __forceinline__ int for_entries(const int32_t* h, int from, int to, Op one) {
  if (from >= to) return -1;
  const int tid = threadIdx.x;
  h += from;
  const int len = to - from;
  // up to three entries before the first 16-byte boundary, then four at a time
  const int head = min(len, static_cast<int>(-(reinterpret_cast<uintptr_t>(h) >> 2) & 3));
  const int vecs = (len - head) / 4;
  const int4* h4 = reinterpret_cast<const int4*>(h + head);
  int top = -1;
  for (int i0 = tid; i0 < vecs; i0 += kThreads * kLoads) {
    int4 t[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = i0 + j * kThreads;
      t[j] = i < vecs ? h4[i] : make_int4(-1, -1, -1, -1);
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      top = max(max(max(top, one(t[j].x)), max(one(t[j].y), one(t[j].z))), one(t[j].w));
  }
  const int rest = head + vecs * 4;
  if (tid < head + len - rest) {
    const int i = tid < head ? tid : rest + tid - head;
    top = max(top, one(h[i]));
  }
  return top;
}

// One CTA per (row, chunk of kThreads * 4 * kVec tokens).  It asks for its logits
// (into L2), counts the history's tokens that fall into its chunk in shared
// memory, then passes over its logits once.  Every CTA of a row reads the row's
// whole history, from L2 after the first.
//
// Bound: HBM, the logits in and out.  256 rows x 131072 tokens without history
// take 49 us (floor 42), with up to 1000 tokens each 58, with 16k-32k tokens each
// and 64 biases 72 (floor 45): the counting, bound by latency, is only partly
// hidden.  With 16k-32k tokens and no biases it took 64 us in chunks of
// 32768 tokens on 1024 threads, two per SM, two loads in flight per thread (32
// registers; four spilled: 81 us); 512 threads and chunks of 16384 72 us, of
// 8192 94 us (more re-reading of the history), 65536 tokens on one CTA per SM
// 66 us; 32-bit cells in chunks of 16384 75 us.  Counting and streaming halves
// of one CTA working on different items took 110 us (the counting wants every
// warp); predicated atomics in place of the branch, and one pass over prompt and
// answer with a mark in the cell's top bit, gained nothing.
template <typename Cell, int kThreads, int kVec, int kMinBlocks, int kStep>
__global__ void __launch_bounds__(kThreads, kMinBlocks) adjust_kernel(const AdjustParams p) {
  constexpr int kChunk = kThreads * 4 * kVec;
  extern __shared__ __align__(16) uint32_t table[];   // [kChunk] cells where there is a history
  Cell* cell = reinterpret_cast<Cell*>(table);
  __shared__ __align__(16) int bias_tok[kAdjustMaxBias + 4];
  __shared__ float bias_val[kAdjustMaxBias];
  const int tid = threadIdx.x;
  const int row = blockIdx.x / p.chunks;
  const int chunk = blockIdx.x - row * p.chunks;
  const int lo = chunk * kChunk;
  const int size = min(kChunk, p.vocab - lo);
  const float* z = p.z + static_cast<size_t>(row) * p.vocab + lo;
  float* out = p.out + static_cast<size_t>(row) * p.vocab + lo;

  if (p.history) {
    if (tid == 0) prefetch_l2(z, size * 4);
    for (int i = tid; i < size * static_cast<int>(sizeof(Cell)) / 16; i += kThreads)
      reinterpret_cast<uint4*>(table)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // the row's biases, as offsets in the chunk
  for (int e = tid; e < p.n_bias; e += kThreads) {
    const int t = p.bias_tokens[static_cast<size_t>(row) * p.n_bias + e];
    bias_tok[e] = t - lo;
    bias_val[e] = p.bias_values[static_cast<size_t>(row) * p.n_bias + e];
    if (t >= p.vocab && chunk == 0) report_status(p.status, kStatusBounds);
  }
  if (tid < 3) bias_tok[p.n_bias + tid] = -1;   // up to whole groups of four
  __syncthreads();

  Penalty w = {1.f, 1.f, 0.f, 0.f};
  if (p.history) {
    int len = p.history_len[row];
    if (len < 0 || len > p.history_ld) {
      if (tid == 0 && chunk == 0) report_status(p.status, kStatusBounds);
      len = min(max(len, 0), p.history_ld);
    }
    const int prompt = p.prompt_len ? p.prompt_len[row] : 0;
    const int32_t* h = p.history + static_cast<size_t>(row) * p.history_ld;
    const int split = min(max(prompt, 0), len);
    int top = for_entries<kThreads>(h, split, len, [&](int t) {
      const uint32_t at = static_cast<uint32_t>(t - lo);
      if (at < static_cast<uint32_t>(size)) count_token<Cell>(table, at);
      return t;
    });
    __syncthreads();
    // a prompt's token marks an empty cell only (two entries of it write the same)
    const int top2 = for_entries<kThreads>(h, 0, split, [&](int t) {
      const uint32_t at = static_cast<uint32_t>(t - lo);
      if (at < static_cast<uint32_t>(size) && cell[at] == 0) cell[at] = ~Cell(0);
      return t;
    });
    top = max(top, top2);
    if (chunk == 0 && top >= p.vocab) report_status(p.status, kStatusBounds);
    if (p.repetition) w.r = p.repetition[row];
    if (p.frequency) w.f = p.frequency[row];
    if (p.presence) w.p = p.presence[row];
    w.inv = 1.f / w.r;
    __syncthreads();
  }

  const uint32_t* allowed =
      p.allowed ? p.allowed + (static_cast<size_t>(row) * p.vocab + lo) / 32 : nullptr;
#pragma unroll 1
  for (int v0 = tid * 4; v0 < size; v0 += kThreads * 4 * kStep) {
    float4 x[kStep];
    uint32_t bits[kStep];
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      const int v = v0 + i * kThreads * 4;
      if (v < size) x[i] = *reinterpret_cast<const float4*>(z + v);
      bits[i] = allowed && v < size ? allowed[v >> 5] >> (v & 31) : 0xFu;
    }
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      const int v = v0 + i * kThreads * 4;
      if (v >= size) continue;
      float4 y = x[i];
      if (p.history) {
        const uint4 c = cells4(cell + v);
        if (c.x | c.y | c.z | c.w) {
          y.x = penalised<Cell>(y.x, c.x, w);
          y.y = penalised<Cell>(y.y, c.y, w);
          y.z = penalised<Cell>(y.z, c.z, w);
          y.w = penalised<Cell>(y.w, c.w, w);
        }
      }
      if (!(bits[i] & 1u)) y.x = -INFINITY;
      if (!(bits[i] & 2u)) y.y = -INFINITY;
      if (!(bits[i] & 4u)) y.z = -INFINITY;
      if (!(bits[i] & 8u)) y.w = -INFINITY;
      *reinterpret_cast<float4*>(out + v) = y;
    }
  }
  // Biased tokens, on the values just written: the first entry of a token in the
  // list takes the sum of all its entries, in list order (a fixed order, no
  // atomics).
  if (p.n_bias > 0) {
    __syncthreads();
    for (int e = tid; e < p.n_bias; e += kThreads) {
      const int t = bias_tok[e];
      if (t < 0 || t >= size || (allowed && !(allowed[t >> 5] >> (t & 31) & 1u))) continue;
      int same = 0;
      for (int i = 0; i < p.n_bias; i += 4) {
        const int4 u = *reinterpret_cast<const int4*>(bias_tok + i);
        same += (u.x == t) + (u.y == t) + (u.z == t) + (u.w == t);
      }
      float sum = bias_val[e];
      if (same > 1) {
        bool first = true;
        sum = 0.f;
        for (int i = 0; i < p.n_bias; ++i) {
          if (bias_tok[i] != t) continue;
          first = first && i >= e;
          sum += bias_val[i];
        }
        if (!first) continue;
      }
      out[t] += sum;
    }
  }
}

template <typename Cell, int kThreads, int kVec, int kMinBlocks, int kStep>
cudaError_t adjust_launch(AdjustParams p, cudaStream_t s) {
  constexpr int kChunk = kThreads * 4 * kVec;
  auto* kern = adjust_kernel<Cell, kThreads, kVec, kMinBlocks, kStep>;
  p.chunks = (p.vocab + kChunk - 1) / kChunk;
  const long long grid = static_cast<long long>(p.n) * p.chunks;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const int cells = p.vocab < kChunk ? p.vocab : kChunk;
  static uint32_t attr_done = 0;   // per instantiation, one bit per device < 32
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(attr_done & (1u << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunk * sizeof(Cell));
    if (e != cudaSuccess) return e;
    if (dev < 32) attr_done |= 1u << dev;
  }
  kern<<<static_cast<unsigned>(grid), kThreads, p.history ? cells * sizeof(Cell) : 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adjust(AdjustParams p, int num_sms, cudaStream_t s) {
  if (p.n <= 0) return cudaSuccess;
  if (p.vocab % 256 != 0 || p.n_bias > kAdjustMaxBias) return cudaErrorInvalidValue;
  // The largest chunk that still gives every SM one (fewer re-reads of the
  // history), but none that a whole row does not half fill.  64 rows x 131072
  // with 4096 tokens of history: chunks of 32768 13 us, of 8192 17 us.
  // Cells go by the width of the history's rows, as their lengths are on the
  // device: rows wider than kMaxShort pay for 32-bit cells and chunks of 8192 with
  // few tokens too.  256 rows x 131072 with up to 1000 / 4096 / 32768 / 65534
  // tokens in rows of at most 65534 entries take 62 / 65 / 75 / 92 us, in wider
  // ones 68 / 76 / 103 / 142; 64 rows with up to 4096 21-23 and 25; one row 10 and 12.
  auto fits = [&](int chunk) {
    return p.vocab > chunk / 2 && static_cast<long long>(p.n) * ((p.vocab + chunk - 1) / chunk) >= num_sms;
  };
  if (p.history_ld > kMaxShort)
    return fits(8192) ? adjust_launch<uint32_t, 512, 4, 3, 4>(p, s)
                      : adjust_launch<uint32_t, 512, 1, 3, 1>(p, s);
  if (fits(32768)) return adjust_launch<uint16_t, 1024, 8, 2, 2>(p, s);
  if (fits(8192)) return adjust_launch<uint16_t, 512, 4, 3, 4>(p, s);
  return adjust_launch<uint16_t, 512, 1, 3, 1>(p, s);
}

}  // namespace dory
