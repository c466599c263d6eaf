// Device code shared by the loss kernels: a row of logits as 16-byte words,
// the running maximum and sum of its softmax, and each loss's row values.
//
// Mathematics.  For a row z of V logits at temperature 1/c (c = 1 except in
// the distillation), with M = max z and s = sum exp(c (z_v - M)):
//   ln q_v = c (z_v - M) - ln s            log-softmax
//   lse    = M + ln s                      (c = 1)
// Maximum and sum come from one pass: a thread holds (m, s) of what it has
// seen, and on a new maximum m' its sum becomes s exp(c (m - m')) plus the new
// terms.  Two such pairs join the same way.  Every exponent is taken of a
// difference that is formed first, c (z - m) = log2(e) c (z - m) in base 2:
// z - m is exact or rounded once, so that the size of the logits costs the
// result nothing.
//
// A gradient row has the form g_v = coef (q_v - sum_k p_k [v = id_k]): one
// target with p = 1 for the label losses, k targets for the distillation.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "thd_loss_internal.h"

namespace thdcp {

typedef unsigned int Word4 __attribute__((ext_vector_type(4)));
typedef __bf16 Bf16x2 __attribute__((ext_vector_type(2)));
typedef float Float2v __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

struct Bf16 {
  uint16_t bits;
};
struct Fp16 {
  _Float16 v;
};

// Elements of one type in 16-byte words.
template <typename T>
struct Elem;

template <>
struct Elem<Bf16> {
  static constexpr int kPer = 8;
  static constexpr uint32_t kNegInfWord = 0xff80ff80u;
  static constexpr uint32_t kNanWord = 0x7fc07fc0u;
  static __device__ __forceinline__ float load(const Bf16* p) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(p->bits) << 16);
  }
  static __device__ __forceinline__ void unpack(Word4 w, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
    }
  }
  // rounded once, to nearest even
  static __device__ __forceinline__ Word4 pack(const float (&g)[8]) {
    Word4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Float2v f = {g[2 * i], g[2 * i + 1]};
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, Bf16x2));
    }
    return w;
  }
  static __device__ __forceinline__ Bf16 round(float g) {
    const Float2v f = {g, 0.0f};
    return Bf16{static_cast<uint16_t>(__builtin_bit_cast(uint32_t, __builtin_convertvector(f, Bf16x2)))};
  }
};

template <>
struct Elem<Fp16> {
  static constexpr int kPer = 8;
  static constexpr uint32_t kNegInfWord = 0xfc00fc00u;
  static constexpr uint32_t kNanWord = 0x7e007e00u;
  static __device__ __forceinline__ float load(const Fp16* p) { return static_cast<float>(p->v); }
  static __device__ __forceinline__ void unpack(Word4 w, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w[i])));
      x[2 * i + 1] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w[i] >> 16)));
    }
  }
  static __device__ __forceinline__ Word4 pack(const float (&g)[8]) {
    Word4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<_Float16>(g[2 * i]));
      const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<_Float16>(g[2 * i + 1]));
      w[i] = lo | (hi << 16);
    }
    return w;
  }
  static __device__ __forceinline__ Fp16 round(float g) { return Fp16{static_cast<_Float16>(g)}; }
};

template <>
struct Elem<float> {
  static constexpr int kPer = 4;
  static constexpr uint32_t kNegInfWord = 0xff800000u;
  static constexpr uint32_t kNanWord = 0x7fc00000u;
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void unpack(Word4 w, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = w[i];  // a copy: bit_cast of a vector element reads element 0
      x[i] = __builtin_bit_cast(float, bits);
    }
  }
  static __device__ __forceinline__ Word4 pack(const float (&g)[4]) {
    Word4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, g[i]);
    return w;
  }
  static __device__ __forceinline__ float round(float g) { return g; }
};

// A row as a head of single elements up to the first 16-byte boundary, whole
// words, and a tail of single elements: no access leaves the row.  Head and
// tail together ("edge") hold at most 2 (kPer - 1) elements; edge element i is
// held by thread i of the workgroup that owns the row's edge.
template <typename T>
struct RowCut {
  int32_t head, words, edge;
  __device__ __forceinline__ RowCut(const void* row, int32_t vocab) {
    constexpr int kPer = Elem<T>::kPer;
    const int32_t lead = static_cast<int32_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) /
                         static_cast<int32_t>(sizeof(T));
    head = min(lead, vocab);
    words = (vocab - head) / kPer;
    edge = vocab - words * kPer;
  }
  // column of edge element i
  __device__ __forceinline__ int32_t edge_column(int32_t i) const {
    return i < head ? i : i + words * Elem<T>::kPer;
  }
  // word that holds column v, or -1 for an edge element
  __device__ __forceinline__ int32_t word_of(int32_t v) const {
    const int32_t b = v - head;
    return b >= 0 && b < words * Elem<T>::kPer ? b / Elem<T>::kPer : -1;
  }
  __device__ __forceinline__ int32_t place_of(int32_t v) const { return (v - head) & (Elem<T>::kPer - 1); }
  __device__ __forceinline__ int32_t edge_of(int32_t v) const { return v < head ? v : v - words * Elem<T>::kPer; }
};

__device__ __forceinline__ Word4 load_word(const Word4* p) { return __builtin_nontemporal_load(p); }

// Where a gradient row goes.  It has the words of the logits' row when both
// start at the same place within 16 bytes, else its elements are stored one
// by one.
template <typename T>
struct OutRow {
  T* row;
  Word4* body;
  int32_t head;
  bool whole;
  __device__ __forceinline__ OutRow(T* out, const void* in, int32_t head_) : row(out), head(head_) {
    whole = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(in)) & 15) == 0;
    body = reinterpret_cast<Word4*>(out + head_);
  }
  __device__ __forceinline__ void store(int32_t word, const float (&g)[Elem<T>::kPer]) const {
    if (whole) {
      __builtin_nontemporal_store(Elem<T>::pack(g), body + word);
    } else {
#pragma unroll
      for (int e = 0; e < Elem<T>::kPer; ++e)
        row[head + static_cast<int64_t>(word) * Elem<T>::kPer + e] = Elem<T>::round(g[e]);
    }
  }
};

// Fills elements [0, n) of a row with one value (0 or NaN, given as a word of
// equal elements): rows that a mask leaves out, or whose target is not a
// column.
template <typename T>
__device__ __forceinline__ void fill_words(T* row, int32_t vocab, uint32_t value, int32_t w0, int32_t w1, bool edge,
                                           int32_t threads) {
  const RowCut<T> cut(row, vocab);
  const int32_t tid = threadIdx.x;
  Word4* body = reinterpret_cast<Word4*>(row + cut.head);
  const Word4 v = {value, value, value, value};
  for (int32_t w = w0 + tid; w < min(w1, cut.words); w += threads) __builtin_nontemporal_store(v, body + w);
  if (edge && tid < cut.edge) row[cut.edge_column(tid)] = __builtin_bit_cast(T, static_cast<
      typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type>(value));
}

// Running maximum and sum of exponentials.
struct Stat {
  float m = kNegInf;
  float s = 0.0f;
};

// The value to subtract: a maximum of -inf (nothing seen yet, or only -inf)
// would give -inf - -inf.
__device__ __forceinline__ float base_of(float m) { return m == kNegInf ? 0.0f : m; }

template <int N>
__device__ __forceinline__ void absorb(Stat& st, const float (&x)[N], float scale) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
  const float m = fmaxf(st.m, top);
  const float b = base_of(m);
  float s = st.s * exp2_fast((st.m - b) * scale);
#pragma unroll
  for (int i = 0; i < N; ++i) s += exp2_fast((x[i] - b) * scale);
  st.m = m;
  st.s = s;
}

// Joins the pairs of kWidth neighbouring lanes (a power of two); every lane
// of the group gets the same result.
template <int kWidth>
__device__ __forceinline__ Stat join_lanes(Stat st, float scale) {
  float m = st.m;
#pragma unroll
  for (int d = kWidth / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float b = base_of(m);
  // a NaN among the logits leaves its thread's maximum untouched and its sum
  // NaN, which this product keeps
  float s = st.s * exp2_fast((st.m - b) * scale);
#pragma unroll
  for (int d = kWidth / 2; d > 0; d >>= 1) s += __shfl_xor(s, d);
  return Stat{m, s};
}

// Joins the pairs of a workgroup in a fixed order.  s_red holds one pair per
// wave.  Contains one barrier; what threads wrote to LDS before it can be
// read after it.
template <int kThreads>
__device__ __forceinline__ Stat join_block(Stat st, float scale, float2* s_red) {
  constexpr int kWaves = kThreads / 64;
  st = join_lanes<64>(st, scale);
  const int lane = threadIdx.x & 63;
  if (lane == 0) s_red[threadIdx.x >> 6] = make_float2(st.m, st.s);
  __syncthreads();
  if constexpr (kWaves == 1) return st;
  const float2 r = s_red[lane & (kWaves - 1)];
  return join_lanes<kWaves>(Stat{r.x, r.y}, scale);
}

// ---- row values of the policy loss ----------------------------------------
// r = exp(logp - old), u = ref - logp:
//   L = w ( -min(r A, clip(r, low, high) A) + beta (exp(u) - u - 1) )
//   dL/dlogp = w ( -r A [not clipped] - beta (exp(u) - 1) )
// min takes the clipped branch when A > 0 and r is above the upper end, or A
// < 0 and r is below the lower one; the comparison is made on logp - old in 64
// bits against the ends' logarithms, as an error of the exponential there
// would switch a whole gradient row on or off.  exp(u) - u - 1 is a difference
// of near values for the usual small u: below 1/2 its series is summed.
struct PolicyRow {
  float loss, dlogp;
};

__device__ __forceinline__ float exp_minus_1_minus(float u) {
  if (fabsf(u) < 0.5f) {
    // u^2/2! + u^3/3! + ... + u^9/9!: the rest is below 2^-28 of the sum
    float t = 1.0f / 362880.0f;
    t = fmaf(t, u, 1.0f / 40320.0f);
    t = fmaf(t, u, 1.0f / 5040.0f);
    t = fmaf(t, u, 1.0f / 720.0f);
    t = fmaf(t, u, 1.0f / 120.0f);
    t = fmaf(t, u, 1.0f / 24.0f);
    t = fmaf(t, u, 1.0f / 6.0f);
    t = fmaf(t, u, 0.5f);
    return t * u * u;
  }
  return exp2_fast(u * kLog2e) - 1.0f - u;
}

__device__ __forceinline__ PolicyRow policy_row(const LossArgs& a, int64_t row, float logp) {
  const float adv = a.advantages[row];
  const double d = static_cast<double>(logp) - static_cast<double>(a.old_logp[row]);
  const bool clipped = adv >= 0.0f ? d > a.ln_high : d < a.ln_low;
  const float edge = adv >= 0.0f ? a.high : a.low;
  const float ratio = exp2_fast(static_cast<float>(d) * kLog2e);
  float loss = -(clipped ? edge : ratio) * adv;
  float g = clipped ? 0.0f : -ratio * adv;
  if (a.ref_logp) {
    const float u = a.ref_logp[row] - logp;
    const float k = exp_minus_1_minus(u);
    loss = fmaf(a.kl_coef, k, loss);
    g = fmaf(-a.kl_coef, k + u, g);
  }
  const float w = a.weights ? a.weights[row] : 1.0f;
  return PolicyRow{w * loss, w * g};
}

// ---- targets of the distillation -------------------------------------------
// Up to THD_MAX_TOPK teacher columns of one row, in LDS.  p = softmax(t / tau)
// over the given columns; a column given as -1, or with a logit of -inf, has no
// part in it.  Each column that occurs is listed once, with the sum of its
// probabilities in the order they are given, under the thread that holds the
// column's element, so that a gradient word costs its thread one bit test and a
// list walk only where a target falls into it.  The order of a thread's list
// depends on the lanes' order; no result does, as every element is in it once.
constexpr int kEdgeBit = 31;
constexpr int kRestBit = 30;  // words beyond the ones a thread holds in registers

template <int kThreads>
struct alignas(16) TargetList {
  int32_t id[THD_MAX_TOPK];    // column, -1: no part in the sum
  float p[THD_MAX_TOPK];       // its probability
  float ln_p[THD_MAX_TOPK];
  float z[THD_MAX_TOPK];       // the student's logit there
  float sum[THD_MAX_TOPK];     // the column's whole probability
  int32_t next[THD_MAX_TOPK];
  int32_t head[kThreads];
  uint32_t hit[kThreads];      // bit i: a target in the thread's word i
  int32_t state;               // RowState
};

enum RowState : int { kRowLive, kRowEmpty, kRowBad };

__device__ __forceinline__ void wave_sync_lds() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float load_any(const void* p, int64_t i, int32_t dtype) {
  if (dtype == THD_BF16) return Elem<Bf16>::load(static_cast<const Bf16*>(p) + i);
  if (dtype == THD_FP16) return Elem<Fp16>::load(static_cast<const Fp16*>(p) + i);
  return static_cast<const float*>(p)[i];
}

// Fills the list; run by wave 0 alone, its results are visible to the
// workgroup after the next barrier.  The workgroup holds the row's words
// [w0, w0 + n_words), word w0 + i in thread i % kThreads, of which a thread has
// a bit each for its first kHeld and one for the rest, and the row's edge if
// own_edge.  The student's logits are read from the row, or from z_saved
// where the row may be overwritten by then.
template <typename T, int kThreads, int kHeld>
__device__ __forceinline__ void list_targets(TargetList<kThreads>& l, const LossArgs& a, int64_t row, const T* in,
                                             const float* z_saved, const RowCut<T>& cut, int32_t vocab, int32_t w0,
                                             int32_t n_words, bool own_edge) {
  constexpr int kMine = THD_MAX_TOPK / 64;
  const int lane = threadIdx.x;
  const int64_t at = row * a.teacher_stride;
  int32_t id[kMine];
  float t[kMine], sum[kMine];
  bool first[kMine];
  bool bad = false;
  float top = kNegInf;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int32_t i = lane + 64 * j;
    id[j] = -1;
    t[j] = kNegInf;
    if (i < a.k) {
      const int64_t v = a.ids64 ? static_cast<const int64_t*>(a.teacher_ids)[at + i]
                                : static_cast<const int32_t*>(a.teacher_ids)[at + i];
      if (v < -1 || v >= vocab) bad = true;
      else if (v >= 0) {
        id[j] = static_cast<int32_t>(v);
        t[j] = load_any(a.teacher, at + i, a.teacher_dtype);
      }
    }
    top = fmaxf(top, t[j]);
  }
  for (int i = lane; i < kThreads; i += 64) {
    l.head[i] = -1;
    l.hit[i] = 0;
  }
  bad = __any(bad);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float base = base_of(top);
  float ts = 0.0f;
#pragma unroll
  for (int j = 0; j < kMine; ++j) ts += exp2_fast((t[j] - base) * a.inv_temperature * kLog2e);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) ts += __shfl_xor(ts, d);
  const float ln_ts = logf(ts);
  const float inv_ts = 1.0f / ts;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int32_t i = lane + 64 * j;
    const float x = (t[j] - base) * a.inv_temperature;
    const float p = exp2_fast(x * kLog2e) * inv_ts;
    if (p == 0.0f || bad) id[j] = -1;
    if (64 * j < a.k) {  // entries up to the next multiple of 64 are written
      l.id[i] = id[j];
      l.p[i] = id[j] >= 0 ? p : 0.0f;
      l.ln_p[i] = x - ln_ts;
      float z = 0.0f;
      if (id[j] >= 0) z = z_saved ? z_saved[row * a.k + i] : Elem<T>::load(in + id[j]);
      l.z[i] = z;
    }
  }
  if (lane == 0) l.state = bad ? kRowBad : (ts == 0.0f ? kRowEmpty : kRowLive);
  wave_sync_lds();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    sum[j] = 0.0f;
    first[j] = true;
    if (64 * j >= a.k) continue;
    const int32_t i = lane + 64 * j;
    for (int n = 0; n < a.k; n += 4) {
      const int4 o = *reinterpret_cast<const int4*>(l.id + n);
      const int32_t other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (other[e] == id[j]) {
          sum[j] += l.p[n + e];
          if (n + e < i) first[j] = false;
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int32_t i = lane + 64 * j;
    if (64 * j >= a.k || id[j] < 0 || !first[j]) continue;
    l.sum[i] = sum[j];
    int32_t owner, bit;
    const int32_t w = cut.word_of(id[j]);
    if (w < 0) {
      if (!own_edge) continue;
      owner = cut.edge_of(id[j]);
      bit = kEdgeBit;
    } else {
      const int32_t local = w - w0;
      if (local < 0 || local >= n_words) continue;
      owner = local % kThreads;
      bit = local / kThreads < kHeld ? local / kThreads : kRestBit;
    }
    l.next[i] = atomicExch(&l.head[owner], i);
    atomicOr(&l.hit[owner], 1u << bit);
  }
}

// Loss of the row from the filled list, on wave 0 (the same value in every
// lane): tau^2 w sum p (ln p - ln q).
template <int kThreads>
__device__ __forceinline__ float distill_loss(const TargetList<kThreads>& l, const LossArgs& a, float w, float m,
                                              float ln_s) {
  float loss = 0.0f;
  for (int i = threadIdx.x; i < a.k; i += 64) {
    if (l.id[i] < 0) continue;
    const float ln_q = (l.z[i] - m) * a.inv_temperature - ln_s;
    loss += l.p[i] * (l.ln_p[i] - ln_q);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) loss += __shfl_xor(loss, d);
  return a.temperature * a.temperature * w * loss;
}

// Takes a gradient word's targets from it: g[e] -= amount * sum.
template <typename T, int kThreads>
__device__ __forceinline__ void take_targets(const TargetList<kThreads>& l, const RowCut<T>& cut, int32_t word,
                                             float amount, float (&g)[Elem<T>::kPer]) {
  for (int32_t n = l.head[threadIdx.x]; n >= 0; n = l.next[n]) {
    const int32_t v = l.id[n];
    if (cut.word_of(v) != word) continue;
    const int32_t place = cut.place_of(v);
#pragma unroll
    for (int e = 0; e < Elem<T>::kPer; ++e)
      if (e == place) g[e] = fmaf(-amount, l.sum[n], g[e]);
  }
}

template <typename T, int kThreads>
__device__ __forceinline__ float take_edge_target(const TargetList<kThreads>& l, const RowCut<T>& cut, float amount,
                                                  float g) {
  for (int32_t n = l.head[threadIdx.x]; n >= 0; n = l.next[n]) {
    const int32_t v = l.id[n];
    if (cut.word_of(v) < 0) g = fmaf(-amount, l.sum[n], g);
  }
  return g;
}

}  // namespace thdcp
