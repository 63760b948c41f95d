// Distillation from a teacher's top logits: loss and gradient in one call.
//   p = softmax(t / T) over the valid entries of the row's list,
//   q = softmax(z / T) over the vocabulary,
//   loss = w T^2 sum_j p_j (log p_j - log q_{id_j}),
//   dz_v = g w T (q_v - sum_{j: id_j = v} p_j)   [times the logit scale s_v].
// A row without a valid entry, with only -inf logits on either side, or with
// w = 0 has loss 0 and gradient 0.
//
// The logits are read from memory once: between the sum and the gradient a row
// stays in its CTA's registers (vocabularies up to 16384) or in L2.
//
// Bound: HBM, the logits in and the gradient out.  bf16 gradient through the
// scale, 64 entries: 4096 x 131072 with weights 496 us (floor 410; 556 when
// called without a pause, as the clock falls to 1.57 GHz at the power limit),
// 4096 x 98304 423 (floor 369), 8192 x 49152 413 (370), 16000 x 24576 460 (362),
// 20000 x 16640 575 (307: two stages a row, the second nearly empty), 16384 x
// 16384 304 (247), 32768 x 4096 169 (126), 65536 x 1024 128 (67).  The loss alone
// of 3000 x 131072 231 (241: reads alone run above the copy rate).  Two CTAs of a cluster with half a row each, in
// registers or in a ring, were slower: their rows run in step, and memory waits
// while they join their sums.  Two CTAs of 544 threads leave the row kernel 56
// registers and 896 threads the ring 72; what does not fit goes to local memory
// (48-56 bytes a thread in the row kernel, 16-24 in the ring).
#include "kernels.h"
#include "vocab_ops.cuh"

namespace dory {

namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// Repeated tokens in a list are found with a table of twice as many places: a
// token goes to the upper bits of a product (multiplicative hashing) or to the
// next free place, unless it meets itself.  (Comparing all pairs instead took
// three times as long as the whole kernel does now at 65536 x 1024, 256 entries.)
constexpr int kSlots = 2 * kTopMax;
__device__ __forceinline__ int slot_of(int id) {
  return static_cast<int>((static_cast<uint32_t>(id) * 2654435769u) >> 16) & (kSlots - 1);
}
__device__ __forceinline__ void clear_slots(int* slot, int thread, int threads) {
  for (int i = thread; i < kSlots / 4; i += threads) reinterpret_cast<int4*>(slot)[i] = make_int4(-1, -1, -1, -1);
}
// `old`: what the token's first place held.  True if the list has it already.
__device__ __forceinline__ bool insert_rest(int* slot, int id, int old) {
  for (int at = slot_of(id); old != -1;) {
    if (old == id) return true;
    at = (at + 1) & (kSlots - 1);
    old = atomicCAS(slot + at, -1, id);
  }
  return false;
}
// Of a list with repeated tokens: whether entry e is the first of its token, and
// the sum of the token's probabilities in list order.
__device__ __forceinline__ bool first_of_token(const int* ids, const float* probs, int k, int e, float& target) {
  bool first = true;
  target = 0.f;
  for (int j = 0; j < k; ++j) {
    if (ids[j] != ids[e]) continue;
    first = first && j >= e;
    target += probs[j];
  }
  return first;
}

__device__ __forceinline__ float probability(float t, float c, const ExpSum& teacher) {
  return exp_term(t, c, exp_ref(teacher.m)) / teacher.s;
}
// An entry's part of the loss, in units of 1 / c, so that the rounding of c to
// fp32 nearly cancels.  The differences of the logits are formed in double
// precision: they cancel against the logarithm when the student is close to the
// teacher.
__device__ __forceinline__ double loss_term(float p, float t, float z, const ExpSum& teacher, const ExpSum& student,
                                            float c, float log2_ratio) {
  if (p == 0.f) return 0.0;
  const double d = (static_cast<double>(t) - teacher.m) - (static_cast<double>(z) - student.m);
  return static_cast<double>(p) * (d * static_cast<double>(c) + static_cast<double>(log2_ratio));
}
__device__ __forceinline__ double warp_sum_double(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
// streaming: what is written should not push the rows in flight out of L2
template <typename T>
__device__ __forceinline__ void store4(T* dst, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void store4<float>(float* dst, float a, float b, float c, float d) {
  __stcs(reinterpret_cast<float4*>(dst), make_float4(a, b, c, d));
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* dst, float a, float b, float c,
                                                      float d) {
  __stcs(reinterpret_cast<uint2*>(dst), make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d)));
}
__device__ __forceinline__ void store1(float* dst, float a) { *dst = a; }
__device__ __forceinline__ void store1(__nv_bfloat16* dst, float a) { *dst = __float2bfloat16_rn(a); }

// An entry's gradient, once the row's without the teacher is written.
template <typename Grad>
__device__ __forceinline__ void store_entry(Grad* dz, const DistillParams& p, int id, float z, float target, float w,
                                            const ExpSum& student) {
  const float coef = p.grad_scale * w;
  const float g = exp_term(z, p.exp_scale, exp_ref(student.m)) * (coef / student.s) - coef * target;
  store1(dz + id, p.col_scale ? g * __ldg(p.col_scale + id) : g);
}

// A thread's values x[] of a row -> exponentials relative to the thread's own
// maximum (but for the factor it returns), and their sum.
template <bool kNear, int NF>
__device__ __forceinline__ float exponentials_at(float4 (&x)[NF], float c, const ExpBase& b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    x[i] = exp4_at<kNear>(x[i], c, b);
    s += (x[i].x + x[i].y) + (x[i].z + x[i].w);
  }
  return s;
}
template <int NF>
__device__ __forceinline__ ExpSum exponentials(float4 (&x)[NF], float c, float& fix) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NF; ++i) top = fmaxf(top, max4(x[i]));
  const ExpBase b = exp_base(top, c);
  fix = b.fix;
  return {top, (b.near ? exponentials_at<true>(x, c, b) : exponentials_at<false>(x, c, b)) * b.fix};
}

template <typename Grad>
__device__ __forceinline__ void store_scaled(Grad* dst, const float4& e, float f, const float4& s, bool scaled) {
  const float2 ff = make_float2(f, f);
  float2 u = mul2(make_float2(e.x, e.y), ff), v = mul2(make_float2(e.z, e.w), ff);
  if (scaled) {
    u = mul2(u, make_float2(s.x, s.y));
    v = mul2(v, make_float2(s.z, s.w));
  }
  store4(dst, u.x, u.y, v.x, v.y);
}

// The teacher's list of a row: a warp's lanes keep their entries.
constexpr int kOwn = kTopMax / 32;
struct Entries {
  int id[kOwn];                      // -1 = unused
  float t[kOwn], z[kOwn], p[kOwn];   // the teacher's logit, the student's, the teacher's probability
};
// Read them; the sum over the list (s = 0: no entry with a finite logit).
__device__ __forceinline__ ExpSum load_entries(Entries& x, const DistillParams& p, int row) {
  const int lane = threadIdx.x & 31;
  const float c = p.exp_scale;
  const size_t at = static_cast<size_t>(row) * p.k;
  const float* z = p.logits + static_cast<size_t>(row) * p.vocab;
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int e = q * 32 + lane;
    x.id[q] = e < p.k ? p.teacher_tokens[at + e] : -1;
    x.t[q] = e < p.k ? p.teacher_logits[at + e] : -INFINITY;
  }
  ExpSum sum = {-INFINITY, 0.f};
  bool outside = false;
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    if (x.id[q] >= p.vocab) {
      outside = true;
      x.id[q] = -1;
    }
    x.z[q] = x.id[q] >= 0 ? z[x.id[q]] : 0.f;
    if (x.id[q] < 0) x.t[q] = -INFINITY;
    exp_raise(sum, x.t[q], c);
  }
  if (outside) report_status(p.status, kStatusBounds);
  const float ref = exp_ref(sum.m);
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    if (q * 32 >= p.k) break;
    sum.s += exp_term(x.t[q], c, ref);
  }
  sum = softmax_sum(warp_join(sum, c));
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    if (q * 32 >= p.k) break;
    x.p[q] = x.id[q] >= 0 ? probability(x.t[q], c, sum) : 0.f;
  }
  return sum;
}
// ------------------------------------------------- a row per CTA, in registers
constexpr int kNF = 8;                           // float4 per thread
constexpr int kRowThreads = 512;                 // at most, and a teacher warp
constexpr int kRowMax = kRowThreads * 4 * kNF;   // logits a CTA holds

struct RowShared {
  int id[kTopMax];                 // the teacher's list; -1 = unused
  float t[kTopMax], z[kTopMax], p[kTopMax];   // its logits, the student's, its probabilities
  __align__(16) int slot[kSlots];
  ExpSum sums[kRowThreads / 32], teacher;
  bool twice;                      // a token is repeated
};

// The threads keep their logits as exponentials relative to their own maximum
// between the sum and the gradient.  The last warp reads the teacher's list
// meanwhile, and finishes the loss; all of them then write the entries.  (With
// the list shared out from the start and no such warp: 388 us for 308 at
// 16384 x 16384, 64 entries.)
template <typename Grad>
__global__ void __launch_bounds__(kRowThreads + 32, 2) distill_row_kernel(const DistillParams p) {
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x - 32, warps = threads >> 5;
  const int row = blockIdx.x, V = p.vocab;
  const float* z = p.logits + static_cast<size_t>(row) * V;
  Grad* dz = p.grad ? static_cast<Grad*>(p.grad) + static_cast<size_t>(row) * V : nullptr;
  const float c = p.exp_scale;
  const float w = p.row_weight ? p.row_weight[row] : 1.f;
  if (w == 0.f) {
    if (tid == 0) p.loss[row] = 0.f;
    if (dz)
      for (int v = tid * 4; v < V; v += blockDim.x * 4) store4(dz + v, 0.f, 0.f, 0.f, 0.f);
    return;
  }
  float4 x[kNF];
  float own_m = -INFINITY, fix = 1.f;
  if (warp < warps) {
#pragma unroll
    for (int i = 0; i < kNF; ++i) {
      const int v = (i * threads + tid) * 4;
      x[i] = v < V ? *reinterpret_cast<const float4*>(z + v)
                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    const ExpSum own = exponentials<kNF>(x, c, fix);
    own_m = own.m;
    const ExpSum sum = warp_join(own, c);
    if (lane == 0) sh.sums[warp] = sum;
  } else {
    Entries y;
    const ExpSum sum = load_entries(y, p, row);
#pragma unroll
    for (int q = 0; q < kOwn; ++q) {
      if (q * 32 >= p.k) break;
      const int e = q * 32 + lane;
      sh.id[e] = y.id[q];
      sh.t[e] = y.t[q];
      sh.z[e] = y.z[q];
      sh.p[e] = y.p[q];
    }
    if (lane == 0) sh.teacher = sum;
    clear_slots(sh.slot, lane, 32);
  }
  __syncthreads();
  const ExpSum acc = softmax_sum(warp_join(lane < warps ? sh.sums[lane] : ExpSum{-INFINITY, 0.f}, c));
  const bool empty = acc.s == 0.f || sh.teacher.s == 0.f;
  const float inv = empty ? 0.f : p.grad_scale * w / acc.s;
  if (warp < warps && dz) {
    const float f = exp_term(own_m, c, exp_ref(acc.m)) * inv * fix;
#pragma unroll
    for (int i0 = 0; i0 < kNF; i0 += 4) {
      float4 s[4];
      if (p.col_scale) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = ((i0 + i) * threads + tid) * 4;
          if (v < V) s[i] = __ldg(reinterpret_cast<const float4*>(p.col_scale + v));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = ((i0 + i) * threads + tid) * 4;
        if (v >= V) continue;
        if (empty) store4(dz + v, 0.f, 0.f, 0.f, 0.f);
        else store_scaled(dz + v, x[i0 + i], f, s[i], p.col_scale != nullptr);
      }
    }
  }
  if (warp == warps) {
    double loss = 0.0;
    if (!empty) {
      const float ratio = log2f(acc.s / sh.teacher.s);
      for (int e = lane; e < p.k; e += 32) loss += loss_term(sh.p[e], sh.t[e], sh.z[e], sh.teacher, acc, c, ratio);
      loss = warp_sum_double(loss) * p.loss_scale * w;
    }
    if (lane == 0) p.loss[row] = static_cast<float>(loss);
    bool twice = false;
    if (dz && !empty)
      for (int e = lane; e < p.k; e += 32)
        if (const int id = sh.id[e]; id >= 0)
          twice = insert_rest(sh.slot, id, atomicCAS(sh.slot + slot_of(id), -1, id)) || twice;
    twice = __any_sync(kFull, twice);
    if (lane == 0) sh.twice = twice;
  }
  if (!dz || empty) return;
  __syncthreads();   // the row's stores come before the entries'
  for (int e = tid; e < p.k; e += blockDim.x) {
    const int id = sh.id[e];
    float target = sh.p[e];
    if (id < 0 || (sh.twice && !first_of_token(sh.id, sh.p, p.k, e, target))) continue;
    store_entry(dz, p, id, sh.z[e], target, w, acc);
  }
}

// ------------------------------------------- long rows, streamed through a ring
constexpr int kConsumers = 768;
constexpr int kConsumerWarps = kConsumers / 32;
constexpr int kTeachers = 3;   // teacher warps, one per row in turn
constexpr int kRingThreads = kConsumers + 32 * (1 + kTeachers);   // and a producer warp: 72 registers each
constexpr int kPer = 4;        // float4 per consumer and stage
constexpr int kStages = 4;
constexpr int kStageFloats = kConsumers * 4 * kPer;   // 48 KB

struct Teacher {
  int id[kTopMax];                 // written if a token is repeated
  float p[kTopMax];
  __align__(16) int slot[kSlots];
  ExpSum sum;                      // s = 0: no entry with a finite logit
  ExpSum student;                  // the row's own sum
};

// Whether no token stands twice in the list; if one does, the list is laid out
// for first_of_token.
__device__ __forceinline__ bool all_distinct(const Entries& x, Teacher& T, int k) {
  const int lane = threadIdx.x & 31;
  clear_slots(T.slot, lane, 32);
  __syncwarp();
  int old[kOwn];
#pragma unroll
  for (int q = 0; q < kOwn; ++q)
    old[q] = x.id[q] >= 0 && q * 32 < k ? atomicCAS(T.slot + slot_of(x.id[q]), -1, x.id[q]) : -1;
  bool twice = false;
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    if (q * 32 >= k) break;
    twice = insert_rest(T.slot, x.id[q], old[q]) || twice;
  }
  if (!__any_sync(kFull, twice)) return true;
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    if (q * 32 >= k) break;
    T.id[q * 32 + lane] = x.id[q];
    T.p[q * 32 + lane] = x.p[q];
  }
  __syncwarp();
  return false;
}
// Once the row's sum is known: its loss.
__device__ __forceinline__ void finish_loss(const Entries& x, const Teacher& T, const DistillParams& p, int row,
                                            float w, bool empty) {
  double loss = 0.0;
  if (!empty) {
    const float ratio = log2f(T.student.s / T.sum.s);
#pragma unroll
    for (int q = 0; q < kOwn; ++q) {
      if (q * 32 >= p.k) break;
      loss += loss_term(x.p[q], x.t[q], x.z[q], T.sum, T.student, p.exp_scale, ratio);
    }
    loss = warp_sum_double(loss) * p.loss_scale * w;
  }
  if ((threadIdx.x & 31) == 0) p.loss[row] = static_cast<float>(loss);
}
// Once the row's gradient without the teacher is written.
template <typename Grad>
__device__ __forceinline__ void finish_entries(const Entries& x, const Teacher& T, bool distinct,
                                               const DistillParams& p, Grad* dz, float w) {
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    if (q * 32 >= p.k) break;
    const int e = q * 32 + (threadIdx.x & 31), id = x.id[q];
    float target = x.p[q];
    if (id < 0 || (!distinct && !first_of_token(T.id, T.p, p.k, e, target))) continue;
    store_entry(dz, p, id, x.z[q], target, w, T.student);
  }
}

struct RingShared {
  Teacher teacher[kTeachers];
  ExpSum part[2][kConsumerWarps];
  uint64_t full[kStages], empty[kStages], tfull[kTeachers], tempty[kTeachers];
  int abort;
};
constexpr size_t kRingBytes = size_t(kStages) * kStageFloats * sizeof(float);
constexpr size_t kRingSmem = kRingBytes + sizeof(RingShared);

// The next stage of the ring.
struct RingAt {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1;
    }
  }
};

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// A consumer's share of a stage of `left` floats (or as many as fit).
__device__ __forceinline__ void load_stage(float4 (&x)[kPer], const float* src, int left) {
  const float4* src4 = reinterpret_cast<const float4*>(src) + threadIdx.x;
  if (left >= kStageFloats) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] = src4[j * kConsumers];
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      x[j] = (j * kConsumers + static_cast<int>(threadIdx.x)) * 4 < left
                 ? src4[j * kConsumers]
                 : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  }
}
// Hand a stage back to the producer once it has been read.
__device__ __forceinline__ void free_stage(const float4 (&x)[kPer], uint64_t* empty, bool ok) {
  uint32_t w = 0u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) w ^= __float_as_uint(x[j].x) ^ __float_as_uint(x[j].w);
  mbar_arrive_behind_loads(empty, w, ok);
}
template <bool kNear>
__device__ __forceinline__ void exp_stage(float4 (&x)[kPer], float c, const ExpBase& b) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) x[j] = exp4_at<kNear>(x[j], c, b);
}
template <bool kWhole, typename Grad>
__device__ __forceinline__ void store_stage(Grad* dst, const float4 (&x)[kPer], float f, const float4 (&s)[kPer],
                                            bool scaled, int left) {
  dst += threadIdx.x * 4;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (kWhole || (j * kConsumers + static_cast<int>(threadIdx.x)) * 4 < left)
      store_scaled(dst + j * kConsumers * 4, x[j], f, s[j], scaled);
}

// A row between its two passes: dz = f 2^(c (z - ref)) [s].
template <typename Grad>
struct Behind {
  Grad* dz = nullptr;   // null: no such row
  ExpBase base;
  float f;
  bool empty;
  int teacher;
};

// A consumer's share of the second pass over stage i of a row.
template <typename Grad>
__device__ __forceinline__ void gradient_step(const Behind<Grad>& b, const DistillParams& p, const float* ring,
                                              RingShared& sh, RingAt& at, bool& ok, int i) {
  const int v0 = i * kStageFloats, left = p.vocab - v0;
  float4 s[kPer], x[kPer];
  if (p.col_scale) load_stage(s, p.col_scale + v0, left);
  ok = ok && __all_sync(kFull, mbar_wait_bounded(&sh.full[at.stage], at.parity, &sh.abort, p.status));
  load_stage(x, ring + at.stage * kStageFloats, left);
  free_stage(x, &sh.empty[at.stage], ok);
  at.next();
  if (!ok) return;
  if (b.base.near) exp_stage<true>(x, p.exp_scale, b.base);
  else exp_stage<false>(x, p.exp_scale, b.base);
  if (b.empty) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (left >= kStageFloats) store_stage<true>(b.dz + v0, x, b.f, s, p.col_scale != nullptr, left);
  else store_stage<false>(b.dz + v0, x, b.f, s, p.col_scale != nullptr, left);
}

// One persistent CTA per SM: a producer thread streams every row twice, from
// memory for the sum and from L2 for the gradient, as far ahead as the ring is
// free.  The second pass over a row takes turns with the first one over the next,
// stage by stage, so that memory reads and writes mix all the time and the end
// of a sum delays nothing; it runs backwards, what came through L2 last first.
// (Keeping a row's last stages in the ring for the second pass instead was
// slower, 8192 x 49152 492 us for 410: nothing is fetched meanwhile.)
// A teacher warp per row reads its list ahead and finishes loss and entries
// behind.
template <typename Grad, bool kMix>
__global__ void __launch_bounds__(kRingThreads, 1) distill_ring_kernel(const DistillParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  float* ring = reinterpret_cast<float*>(smem);
  RingShared& sh = *reinterpret_cast<RingShared*>(smem + kRingBytes);
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = p.vocab, chunks = (V + kStageFloats - 1) / kStageFloats;
  const int first = blockIdx.x, step = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kConsumerWarps);
    }
    for (int i = 0; i < kTeachers; ++i) {
      mbar_init(&sh.tfull[i], 1);
      mbar_init(&sh.tempty[i], kConsumerWarps);
    }
    sh.abort = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t keep = l2_policy_evict_last(), drop = l2_policy_evict_first();
      RingAt at;
      int used = 0;
      bool ok = true;
      auto load = [&](int row, int i, uint64_t policy) {
        const int v = i * kStageFloats;
        const uint32_t bytes = min(kStageFloats, V - v) * 4;
        ok = ok && mbar_wait_bounded(&sh.empty[at.stage], at.parity ^ 1, abort_flag, p.status);
        if (!ok) return;
        mbar_arrive_expect_tx(&sh.full[at.stage], bytes);
        bulk_load(ring + at.stage * kStageFloats, p.logits + static_cast<size_t>(row) * V + v, bytes,
                  &sh.full[at.stage], policy);
        at.next();
        ++used;
      };
      float next_w = p.row_weight && first < p.n ? p.row_weight[first] : 1.f;
      int behind = -1;
      for (int row = first; row < p.n && ok; row += step) {
        const float w = next_w;
        if (p.row_weight && row + step < p.n) next_w = p.row_weight[row + step];
        if (w == 0.f) continue;
        for (int i = 0; i < chunks && ok; ++i) {
          if (kMix && behind >= 0) load(behind, chunks - 1 - i, drop);
          load(row, i, p.grad ? keep : drop);
        }
        if (p.grad && kMix) behind = row;
        if (p.grad && !kMix)
          for (int i = chunks - 1; i >= 0 && ok; --i) load(row, i, drop);
      }
      if (behind >= 0)
        for (int i = chunks - 1; i >= 0 && ok; --i) load(behind, i, drop);
      // shared memory outlives the copies in flight, after an abort too
      for (int u = used > kStages ? used - kStages : 0; u < used; ++u)
        drain_wait(&sh.full[u % kStages], u / kStages & 1);
    }
  } else if (warp > kConsumerWarps) {
    // ---------------------------------------------------------- teachers
    const int b = warp - kConsumerWarps - 1;
    Teacher& T = sh.teacher[b];
    uint32_t parity = 0;
    int turn = 0;   // of the rows with a weight
    float next_w = p.row_weight && first < p.n ? p.row_weight[first] : 1.f;
    for (int row = first; row < p.n; row += step) {
      const float w = next_w;
      if (p.row_weight && row + step < p.n) next_w = p.row_weight[row + step];
      if (w == 0.f || turn++ % kTeachers != b) continue;
      Entries x;
      const ExpSum sum = load_entries(x, p, row);
      if (lane == 0) T.sum = sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tfull[b]);
      const bool distinct = !p.grad || all_distinct(x, T, p.k);
      // the consumers have left the row's sum and written its gradient
      if (!__all_sync(kFull, mbar_wait_bounded(&sh.tempty[b], parity, abort_flag, p.status))) break;
      parity ^= 1;
      const bool empty = T.student.s == 0.f || T.sum.s == 0.f;
      finish_loss(x, T, p, row, w, empty);
      if (p.grad && !empty)
        finish_entries(x, T, distinct, p, static_cast<Grad*>(p.grad) + static_cast<size_t>(row) * V, w);
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------- consumers
    // A wait that ran out leaves its warp in step (the same CTA barriers) but
    // without effect, so that no other warp is left waiting for it.
    const float c = p.exp_scale;
    RingAt at;
    int used = 0;   // rows with a weight
    bool ok = true;
    float next_w = p.row_weight && first < p.n ? p.row_weight[first] : 1.f;
    Behind<Grad> behind;
    auto release = [&](int b) {
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&sh.tempty[b]);
    };
    for (int row = first; row < p.n; row += step) {
      Grad* dz = p.grad ? static_cast<Grad*>(p.grad) + static_cast<size_t>(row) * V : nullptr;
      const int b = used % kTeachers;
      const float w = next_w;
      if (p.row_weight && row + step < p.n) next_w = p.row_weight[row + step];
      if (w == 0.f) {
        if (dz)
          for (int v = tid * 4; v < V; v += kConsumers * 4) store4(dz + v, 0.f, 0.f, 0.f, 0.f);
        if (tid == 0) p.loss[row] = 0.f;
        continue;
      }
      ExpSum acc = {-INFINITY, 0.f};
      for (int i = 0; i < chunks; ++i) {
        if (kMix && behind.dz) gradient_step(behind, p, ring, sh, at, ok, chunks - 1 - i);
        ok = ok && __all_sync(kFull, mbar_wait_bounded(&sh.full[at.stage], at.parity, abort_flag, p.status));
        float4 x[kPer];
        load_stage(x, ring + at.stage * kStageFloats, V - i * kStageFloats);
        free_stage(x, &sh.empty[at.stage], ok);
        at.next();
        exp_add(acc, x, c);
      }
      if (kMix && behind.dz) release(behind.teacher);
      acc = warp_join(acc, c);
      if (lane == 0) sh.part[used & 1][warp] = acc;
      ok = ok && __all_sync(kFull, mbar_wait_bounded(&sh.tfull[b], used / kTeachers & 1, abort_flag, p.status));
      consumer_sync();
      acc = softmax_sum(warp_join(lane < kConsumerWarps ? sh.part[used & 1][lane] : ExpSum{-INFINITY, 0.f}, c));
      if (tid == 0) sh.teacher[b].student = acc;
      ++used;
      if (dz) {
        behind.dz = dz;
        behind.empty = acc.s == 0.f || sh.teacher[b].sum.s == 0.f;
        behind.base = exp_base(acc.m, c);
        behind.f = behind.empty ? 0.f : p.grad_scale * w / acc.s * behind.base.fix;
        behind.teacher = b;
        if (!kMix) {
          for (int i = chunks - 1; i >= 0; --i) gradient_step(behind, p, ring, sh, at, ok, i);
          release(b);
          behind.dz = nullptr;
        }
      } else {
        release(b);
      }
    }
    if (kMix && behind.dz) {
      for (int i = chunks - 1; i >= 0; --i) gradient_step(behind, p, ring, sh, at, ok, i);
      release(behind.teacher);
    }
  }
}

template <typename Grad, bool kMix>
cudaError_t launch_ring(const DistillParams& p, int num_sms, cudaStream_t s) {
  auto* kern = distill_ring_kernel<Grad, kMix>;
  static uint32_t attr_done = 0;   // per instantiation, one bit per device < 32
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(attr_done & (1u << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
    if (e != cudaSuccess) return e;
    if (dev < 32) attr_done |= 1u << dev;
  }
  kern<<<p.n < num_sms ? p.n : num_sms, kRingThreads, kRingSmem, s>>>(p);
  return cudaGetLastError();
}

template <typename Grad>
cudaError_t launch(const DistillParams& p, int num_sms, cudaStream_t s) {
  if (p.vocab <= kRowMax) {
    const int threads = (p.vocab / (4 * kNF) + 31) / 32 * 32 + 32;
    distill_row_kernel<Grad><<<p.n, threads, 0, s>>>(p);
    return cudaGetLastError();
  }
  // 402 M logits, turns taken or not, in us.  bf16 gradient through the scale (floor
  // 370): rows of 16640 710 and 696, 20480 600 and 603, 24576 483 and 565, 32768 489
  // and 524, 49152 425 and 458, 65536 447 and 470, 98304 481 and 440, 131072 538 and
  // 461: with turns the rows in flight, one and a half per SM, outgrow L2 in the end.
  // fp32 (floor 492): 16640 759 and 684, 24576 580 and 505, 49152 601 and 536, 65536
  // 648 and 545, 131072 707 and 632.
  if constexpr (sizeof(Grad) == 2)
    if (p.vocab <= 65536) return launch_ring<Grad, true>(p, num_sms, s);
  return launch_ring<Grad, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_distill(const DistillParams& p, int grad_bf16, int num_sms, cudaStream_t s) {
  if (p.n <= 0) return cudaSuccess;
  if (p.vocab % 256 != 0 || p.k < 1 || p.k > kTopMax) return cudaErrorInvalidValue;
  return grad_bf16 ? launch<__nv_bfloat16>(p, num_sms, s) : launch<float>(p, num_sms, s);
}

}  // namespace dory
