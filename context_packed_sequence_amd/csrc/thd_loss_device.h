// Device code shared by the loss kernels: a row of logits as 16-byte words,
// the running maximum and sum of its softmax, and each loss's row values.
//
// Mathematics.  For a row z of V logits at temperature 1/c (c = 1 except in
// the distillation), with M = max z and s = sum exp(c (z_v - M)):
//   ln q_v = c (z_v - M) - ln s            log-softmax
//   lse    = M + ln s                      (c = 1)
// Maximum and sum come from one pass: a thread holds (m, s) of what it has
// seen, and on a new maximum m' its sum becomes s exp(c (m - m')) plus the new
// terms.  Two such pairs join the same way.  In base 2, with scale = log2(e) c,
// the exponents are either
//   (z - m) scale           z - m exact or rounded once (Stat), or
//   fma(z, scale, -top)     rounded once, where top is the rounded m scale
//                           (FastStat),
// so that the size of the logits costs the result nothing.  The second form
// takes one instruction less for every exponential and is used where those
// bound the kernel; its pair is relative to top itself, not to m, which makes
// the rounding of top cancel.  It does not hold logits of any size: rows whose
// top is beyond kHuge take the first form.
//
// A label's probability is near 1 for the tokens a model is sure of, and both
// ln q_y and 1 - q_y would be what is left of a difference: its column is kept
// out of the sum, rest = sum over v != y, and joins it at the end:
//   own = exp(c (z_y - M)),  ln q_y = -ln(1 + rest / own) where own >= rest,
//   1 - q_y = rest / (rest + own).
//
// A gradient row has the form g_v = coef (q_v - sum_k p_k [v = id_k]): one
// target with p = 1 for the label losses, k targets for the distillation.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "thd_device.h"
#include "thd_loss_internal.h"

namespace thdcp {

typedef unsigned int Word4 __attribute__((ext_vector_type(4)));
typedef __bf16 Bf16x2 __attribute__((ext_vector_type(2)));
typedef float Float2v __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

// Single instructions, within one step of the result.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float reciprocal(float x) { return __builtin_amdgcn_rcpf(x); }

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

// One element as it lies in memory, to be decoded later: decoding is the first
// use of a load, and waits for it and every load before it.
template <typename T>
__device__ __forceinline__ uint32_t load_raw(const T* p) {
  if constexpr (sizeof(T) == 2) return *reinterpret_cast<const uint16_t*>(p);
  else return *reinterpret_cast<const uint32_t*>(p);
}
template <typename T>
__device__ __forceinline__ float decode(uint32_t raw) {
  if constexpr (std::is_same_v<T, Bf16>) return __builtin_bit_cast(float, raw << 16);
  else if constexpr (std::is_same_v<T, Fp16>)
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(raw)));
  else return __builtin_bit_cast(float, raw);
}

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

// The words of a row behind a buffer resource of exactly their size: a load
// past either end gives zeros and a store there is dropped, both in hardware,
// so that the loops over a thread's words have no branches and every load of a
// row is issued before the first one is waited for.  Word w of the row belongs
// to thread (w + shift) mod threads, where shift puts a wave's 64 words on whole
// 128-byte lines of the row that is written: without it every wave of an
// unaligned row writes two part lines.
template <typename T>
struct RowWords {
  __amdgpu_buffer_rsrc_t rsrc;
  int32_t bytes;
  __device__ __forceinline__ RowWords(const void* body, int32_t words)
      : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(body), 0, 16 * words, kBufferWord3)),
        bytes(16 * words) {}
  // byte offsets: negative ones (as unsigned, huge) are out of range as well
  __device__ __forceinline__ Word4 load(int32_t at) const {
    return __builtin_bit_cast(Word4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, kStreamLoad));
  }
  // words that are read again soon: not past the caches
  __device__ __forceinline__ Word4 load_cached(int32_t at) const {
    return __builtin_bit_cast(Word4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, 0));
  }
  __device__ __forceinline__ void store(int32_t at, Word4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, at, 0, kStreamStorePolicy);
  }
  // 64 lanes' words straight to LDS, lane i's to to[i]; `to` is uniform
  __device__ __forceinline__ void load_to_lds(Word4* to, int32_t at) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(to)), 16, at, 0, 0,
        kStreamLoad);
  }
  static constexpr int kStreamLoad = 2;  // non-temporal
};

// Words by which a row's threads are shifted, from the place its body is
// written to.
__device__ __forceinline__ int32_t line_shift(const void* body) {
  return static_cast<int32_t>((reinterpret_cast<uintptr_t>(body) >> 4) & 7);
}

__device__ __forceinline__ bool same_place(const void* a, const void* b) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// Which of n tiles workgroup b takes.  Workgroup b runs on XCD b mod 8; the
// tiles are cut into chunks of 2^shift and XCD x takes chunks x, x + 8, ...
// front to back, so that each XCD streams through memory of its own (the
// remainder past the last 8 whole chunks in plain order).
__device__ __forceinline__ int32_t tile_of(int32_t b, int32_t n, int32_t shift) {
  const int32_t x = b & 7, j = b >> 3;
  const int32_t tile = ((((j >> shift) << 3) + x) << shift) + (j & ((1 << shift) - 1));
  const int32_t whole = (n >> (shift + 3)) << (shift + 3);
  return b < whole ? tile : b;
}

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

// The form with top = max(z) scale.  The exponent of the largest logit is what
// top was rounded by, up to 2^-24 of it: harmless in the result, but beyond the
// exponential's range from about 2^31 on.  So top starts at a value well within:
// a thread that has seen nothing, or nothing above it, has the sum 0 and needs
// no case of its own, and a row that ends there, or as far above, is huge.
constexpr float kLowestTop = -1.0e9f;
constexpr float kHuge = 0.9e9f;

struct FastStat {
  float top = kLowestTop;
  float s = 0.0f;
};

template <int N>
__device__ __forceinline__ void absorb(FastStat& st, const float (&x)[N], float scale) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, x[i]);
  const float top = fmaxf(st.top, m * scale);
  float s = st.s * exp2_fast(st.top - top);
#pragma unroll
  for (int i = 0; i < N; ++i) s += exp2_fast(fmaf(x[i], scale, -top));
  st.top = top;
  st.s = s;
}

// Maximum and sum over a wave, or over its first row of 16 lanes, on DPP lane
// moves (device helper dpp_move); the result is the same in every lane.
template <bool kRowOnly, typename Op>
__device__ __forceinline__ float wave_reduce(float x, float identity, Op op) {
  const auto move = [&](auto ctrl, auto mask) {
    const int32_t y = dpp_move<decltype(ctrl)::value, decltype(mask)::value>(
        __builtin_bit_cast(int32_t, x), __builtin_bit_cast(int32_t, identity));
    x = op(x, __builtin_bit_cast(float, y));
  };
  using std::integral_constant;
  move(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});
  move(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
  move(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
  move(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
  if constexpr (kRowOnly)
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, x), 15));
  move(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});
  move(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int32_t, x), 63));
}

struct FloatMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct FloatAdd {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
__device__ __forceinline__ float wave_max(float x) { return wave_reduce<false>(x, kNegInf, FloatMax{}); }
__device__ __forceinline__ float wave_add(float x) { return wave_reduce<false>(x, 0.0f, FloatAdd{}); }

// Joins the pairs of a wave's lanes (of its first 16 if kRowOnly).
template <bool kRowOnly>
__device__ __forceinline__ Stat join_lanes(Stat st, float scale) {
  const float m = wave_reduce<kRowOnly>(st.m, kNegInf, FloatMax{});
  const float b = base_of(m);
  // a NaN among the logits leaves its thread's maximum untouched and its sum
  // NaN, which this product keeps
  return Stat{m, wave_reduce<kRowOnly>(st.s * exp2_fast((st.m - b) * scale), 0.0f, FloatAdd{})};
}

template <bool kRowOnly>
__device__ __forceinline__ FastStat join_lanes(FastStat st, float) {
  const float top = wave_reduce<kRowOnly>(st.top, kLowestTop, FloatMax{});
  return FastStat{top, wave_reduce<kRowOnly>(st.s * exp2_fast(st.top - top), 0.0f, FloatAdd{})};
}

__device__ __forceinline__ float2 as_pair(Stat st) { return make_float2(st.m, st.s); }
__device__ __forceinline__ float2 as_pair(FastStat st) { return make_float2(st.top, st.s); }

// Joins the pairs of a workgroup in a fixed order.  s_red holds one pair per
// wave.  Contains one barrier; what threads wrote to LDS before it can be
// read after it.
template <int kThreads, typename S>
__device__ __forceinline__ S join_block(S st, float scale, float2* s_red) {
  constexpr int kWaves = kThreads / 64;
  static_assert(kWaves <= 16);
  st = join_lanes<false>(st, scale);
  const int lane = threadIdx.x & 63;
  if (lane == 0) s_red[threadIdx.x >> 6] = as_pair(st);
  __syncthreads();
  if constexpr (kWaves == 1) return st;
  S other;
  if (lane < kWaves) other = S{s_red[lane].x, s_red[lane].y};
  return join_lanes<true>(other, scale);
}

// The label's column joining the sum of the others.
struct LabelJoin {
  float logp, not_q;  // ln q_y, 1 - q_y
  float sum;          // of all columns, relative to the joined top
};

// ln(1 + x) for small x as ln(u) x / (u - 1) with u = 1 + x rounded (Kahan): the
// factor takes back what the rounding did to x.
__device__ __forceinline__ LabelJoin label_join(float rest, float own, float exponent) {
  const float sum = rest + own;
  const float x = rest * reciprocal(own), u = 1.0f + x;
  const float ln = logf(own >= rest ? u : sum);
  const float ln_1px = u == 1.0f ? x : ln * (x * reciprocal(u - 1.0f));
  return LabelJoin{own >= rest ? -ln_1px : exponent * kLn2 - ln, rest * reciprocal(sum), sum};
}

__device__ __forceinline__ LabelJoin join_label(FastStat& st, float z, float scale) {
  const float top = fmaxf(st.top, z * scale);
  const float rest = st.s * exp2_fast(st.top - top);
  const float exponent = fmaf(z, scale, -top);
  const LabelJoin j = label_join(rest, exp2_fast(exponent), exponent);
  st = FastStat{top, j.sum};
  return j;
}

__device__ __forceinline__ LabelJoin join_label(Stat& st, float z, float scale) {
  const float m = fmaxf(st.m, z);
  const float b = base_of(m);
  const float rest = st.s * exp2_fast((st.m - b) * scale);
  const float exponent = (z - b) * scale;
  const LabelJoin j = label_join(rest, exp2_fast(exponent), exponent);
  st = Stat{m, j.sum};
  return j;
}

// Log-sum-exp of a whole row.  A row of nothing but -inf has no softmax: NaN, not
// the -inf of the formula, which would make its gradient look like one.
__device__ __forceinline__ float log_sum_exp(Stat st) {
  return st.m == kNegInf ? __builtin_nanf("") : st.m + logf(st.s);
}

// Takes one element of a word out of the sum.
template <int N>
__device__ __forceinline__ void drop(float (&f)[N], int32_t place) {
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = e == place ? kNegInf : f[e];
}

// Maximum and sum of a whole row in the first form, element by element, without
// column `skip`: rows beyond kHuge.  Every thread of the workgroup calls it.
template <typename T, int kThreads>
__device__ __forceinline__ Stat row_stat(const T* in, int32_t vocab, int64_t skip, float scale, float2* s_red) {
  Stat st;
  for (int32_t v = threadIdx.x; v < vocab; v += kThreads) {
    const float f[1] = {v == skip ? kNegInf : Elem<T>::load(in + v)};
    absorb(st, f, scale);
  }
  __syncthreads();  // s_red may still be read
  return join_block<kThreads>(st, scale, s_red);
}

// The status word from a look at every row's targets (labels, or the teacher's
// columns), by one workgroup beside the rows': a launch that would set the word
// first costs more wherever the targets are few.
template <int kThreads>
__device__ __forceinline__ void scan_status(const LossArgs& a, int32_t rows, int32_t vocab) {
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  bool bad = false;
  constexpr int kEach = 8;  // loads in flight
  const int32_t n = a.k == 0 ? rows : rows * a.k;
  for (int32_t i0 = threadIdx.x; i0 < n; i0 += kEach * kThreads) {
    int64_t v[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int32_t i = i0 + j * kThreads;
      v[j] = 0;
      if (i >= n) continue;
      if (a.k == 0) {
        v[j] = a.labels[i];
      } else {
        const int64_t at = a.teacher_stride == a.k ? i : i / a.k * a.teacher_stride + i % a.k;
        v[j] = a.ids64 ? static_cast<const int64_t*>(a.teacher_ids)[at]
                       : static_cast<const int32_t*>(a.teacher_ids)[at];
      }
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (v[j] >= (a.k == 0 ? 0 : -1) && v[j] < vocab) continue;
      const int32_t t = (i0 + j * kThreads) / (a.k == 0 ? 1 : a.k);
      bad |= !a.mask || a.mask[t] != 0;
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (threadIdx.x == 0) *a.status = s_bad ? THD_ERR_LABEL : THD_OK;
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

// The KL term's exp(u) - 1 - u and its slope exp(u) - 1.  Each is formed on its
// own: for u far below 0 the term is -u, and the slope, which is -1 there, would
// not be found again in the term plus u.
struct KlTerm {
  float value, slope;
};

__device__ __forceinline__ KlTerm kl_term(float u) {
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
    const float value = t * u * u;
    return KlTerm{value, value + u};
  }
  const float slope = exp2_fast(u * kLog2e) - 1.0f;
  return KlTerm{slope - u, slope};
}

// What a row brings to it.
struct PolicyValues {
  float old_logp = 0.0f, ref_logp = 0.0f, advantage = 0.0f, weight = 1.0f;
};

__device__ __forceinline__ PolicyValues policy_values(const LossArgs& a, int64_t row) {
  PolicyValues v;
  v.old_logp = a.old_logp[row];
  v.advantage = a.advantages[row];
  if (a.ref_logp) v.ref_logp = a.ref_logp[row];
  if (a.weights) v.weight = a.weights[row];
  return v;
}

__device__ __forceinline__ PolicyRow policy_row(const LossArgs& a, const PolicyValues& v, float logp) {
  const float adv = v.advantage;
  const double d = static_cast<double>(logp) - static_cast<double>(v.old_logp);
  const bool clipped = adv >= 0.0f ? d > a.ln_high : d < a.ln_low;
  const float edge = adv >= 0.0f ? a.high : a.low;
  const float ratio = exp2_fast(static_cast<float>(d) * kLog2e);
  float loss = -(clipped ? edge : ratio) * adv;
  float g = clipped ? 0.0f : -ratio * adv;
  if (a.ref_logp) {
    const KlTerm k = kl_term(v.ref_logp - logp);
    loss = fmaf(a.kl_coef, k.value, loss);
    g = fmaf(-a.kl_coef, k.slope, g);
  }
  return PolicyRow{v.weight * loss, v.weight * g};
}

// ---- targets of the distillation -------------------------------------------
// Up to THD_MAX_TOPK teacher columns of one row, in LDS.  p = softmax(t / tau)
// over the given columns; a column given as -1, or with a logit of -inf, has no
// part in it.  A column is listed under the thread that holds its element, so
// that a gradient word costs its thread one bit test and a list walk only where
// a target falls into it.  The order of a list depends on the lanes' order; no
// result does, as every column is in it once: a column that is given more than
// once (found by walking the lists, which are short) makes the wave sum its
// probabilities, in the order they are given, into the first of its entries.
constexpr int kEdgeBit = 31;
constexpr int kRestBit = 30;  // words beyond the ones that have a bit each
constexpr int kMine = THD_MAX_TOPK / 64;

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

// A row's teacher entries as they lie in memory, entry lane + 64 j in lane's
// place j: issued early and decoded later, so that nothing waits for them.
struct TeacherRaw {
  uint32_t id_low[kMine], id_high[kMine], logit[kMine];
};

__device__ __forceinline__ void read_teacher(TeacherRaw& raw, const LossArgs& a, int64_t row) {
  const int64_t at = row * a.teacher_stride;
  const int64_t wide = a.ids64 ? 2 : 1;
  const uint32_t* ids = static_cast<const uint32_t*>(a.teacher_ids) + at * wide;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int32_t i = static_cast<int32_t>(threadIdx.x) + 64 * j;
    raw.id_low[j] = ~0u;
    raw.id_high[j] = ~0u;
    raw.logit[j] = 0;
    if (64 * j >= a.k) continue;
    if (i < a.k) {
      raw.id_low[j] = ids[i * wide];
      if (a.ids64) raw.id_high[j] = ids[i * wide + 1];
      if (a.teacher_dtype == THD_FP32) raw.logit[j] = static_cast<const uint32_t*>(a.teacher)[at + i];
      else raw.logit[j] = static_cast<const uint16_t*>(a.teacher)[at + i];
    }
  }
}

__device__ __forceinline__ float teacher_logit(uint32_t raw, int32_t dtype) {
  if (dtype == THD_BF16) return __builtin_bit_cast(float, raw << 16);
  if (dtype == THD_FP16) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(raw)));
  return __builtin_bit_cast(float, raw);
}

// Fills the list from the row's entries; run by wave 0 alone.  The workgroup
// holds the row's words [w0, w0 + n_words), word w in thread (w - w0 + shift) %
// kThreads, of which a thread has a bit each for its first kHeld and one for the
// rest, and the row's edge if own_edge.  Returns the lane's student logits in z
// (read from the row, or from z_saved where the row may be overwritten by
// then): store_logits puts them into the list once they are here.  The list is
// complete after the next barrier.
template <typename T, int kThreads, int kHeld>
__device__ __forceinline__ void list_targets(TargetList<kThreads>& l, const TeacherRaw& raw, float (&z)[kMine],
                                             const LossArgs& a, int64_t row, const T* in, const float* z_saved,
                                             const RowCut<T>& cut, int32_t vocab, int32_t w0, int32_t n_words,
                                             int32_t shift, bool own_edge) {
  const int lane = threadIdx.x;
  int32_t id[kMine];
  float t[kMine];
  bool bad = false;
  float top = kNegInf;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    id[j] = -1;
    t[j] = kNegInf;
    z[j] = 0.0f;
    if (64 * j >= a.k) continue;
    const int32_t low = static_cast<int32_t>(raw.id_low[j]);
    const int32_t high = a.ids64 ? static_cast<int32_t>(raw.id_high[j]) : low >> 31;
    const bool unused = low == -1 && high == -1;
    const bool column = high == 0 && low >= 0 && low < vocab;
    if (!unused && !column) bad = true;
    id[j] = column ? low : -1;
    t[j] = column ? teacher_logit(raw.logit[j], a.teacher_dtype) : kNegInf;
    if (id[j] >= 0) z[j] = z_saved ? z_saved[row * a.k + lane + 64 * j] : Elem<T>::load(in + id[j]);
    top = fmaxf(top, t[j]);
  }
  for (int i = lane; i < kThreads; i += 64) {
    l.head[i] = -1;
    l.hit[i] = 0;
  }
  bad = __any(bad);
  const float base = base_of(wave_max(top));
  float ts = 0.0f;
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (64 * j < a.k) ts += exp2_fast((t[j] - base) * a.inv_temperature * kLog2e);
  ts = wave_add(ts);
  const float ln_ts = logf(ts);
  const float inv_ts = 1.0f / ts;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (64 * j >= a.k) continue;  // entries up to the next multiple of 64 are written
    const int32_t i = lane + 64 * j;
    const float x = (t[j] - base) * a.inv_temperature;
    const float p = exp2_fast(x * kLog2e) * inv_ts;
    if (p == 0.0f || bad) id[j] = -1;
    l.id[i] = id[j];
    l.p[i] = l.sum[i] = id[j] >= 0 ? p : 0.0f;
    l.ln_p[i] = x - ln_ts;
  }
  if (lane == 0) l.state = bad ? kRowBad : (ts == 0.0f ? kRowEmpty : kRowLive);
  wave_sync_lds();

  bool listed[kMine];
  const auto insert = [&](int j) {
    const int32_t i = lane + 64 * j;
    int32_t owner, bit;
    const int32_t w = cut.word_of(id[j]);
    if (w < 0) {
      if (!own_edge) return false;
      owner = cut.edge_of(id[j]);
      bit = kEdgeBit;
    } else {
      if (w < w0 || w >= w0 + n_words) return false;
      const int32_t local = w - w0 + shift;
      owner = local % kThreads;
      bit = local / kThreads < kHeld ? local / kThreads : kRestBit;
    }
    l.next[i] = atomicExch(&l.head[owner], i);
    atomicOr(&l.hit[owner], 1u << bit);
    return true;
  };
#pragma unroll
  for (int j = 0; j < kMine; ++j) listed[j] = 64 * j < a.k && id[j] >= 0 && insert(j);
  wave_sync_lds();
  bool twice = false;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (!listed[j]) continue;
    for (int32_t n = l.next[lane + 64 * j]; n >= 0; n = l.next[n]) twice |= l.id[n] == id[j];
  }
  if (!__any(twice)) return;

  float sum[kMine];
  bool first[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    sum[j] = 0.0f;
    first[j] = true;
    if (64 * j >= a.k) continue;
    for (int n = 0; n < a.k; ++n) {
      if (l.id[n] != id[j]) continue;
      sum[j] += l.p[n];
      if (n < lane + 64 * j) first[j] = false;
    }
  }
  for (int i = lane; i < kThreads; i += 64) {
    l.head[i] = -1;
    l.hit[i] = 0;
  }
  wave_sync_lds();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    if (!listed[j] || !first[j]) continue;
    l.sum[lane + 64 * j] = sum[j];
    insert(j);
  }
}

__device__ __forceinline__ void store_logits(float* to, const float (&z)[kMine], int32_t k) {
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (64 * j < k) to[threadIdx.x + 64 * j] = z[j];
}

// Loss of the row from the filled list, on wave 0 (the same value in every
// lane): tau^2 w sum p (ln p - ln q).  exponent(z) is log2 of exp(z / tau) over
// the row's largest one.
template <int kThreads, typename F>
__device__ __forceinline__ float distill_loss(const TargetList<kThreads>& l, const LossArgs& a, float w, F exponent,
                                              float ln_s) {
  float loss = 0.0f;
  for (int i = threadIdx.x; i < a.k; i += 64) {
    if (l.id[i] < 0) continue;
    const float ln_q = exponent(l.z[i]) * kLn2 - ln_s;
    loss += l.p[i] * (l.ln_p[i] - ln_q);
  }
  // tau goes in on both sides of the sum: its square may lie outside 32 bits
  // where the loss does not
  return a.temperature * w * wave_add(loss) * a.temperature;
}

// Takes a gradient word's targets from it: g[e] -= amount * sum.
template <typename T, int kThreads>
__device__ __forceinline__ void take_targets(const TargetList<kThreads>& l, const RowCut<T>& cut, int32_t word,
                                             float amount, float (&g)[Elem<T>::kPer]) {
  for (int32_t n = l.head[threadIdx.x]; n >= 0; n = l.next[n]) {
    const int32_t v = l.id[n];
    if (cut.word_of(v) != word) continue;
    const int32_t place = cut.place_of(v);
    const float p = l.sum[n];
#pragma unroll
    for (int e = 0; e < Elem<T>::kPer; ++e)
      if (e == place) g[e] = fmaf(-amount, p, g[e]);
  }
}

template <typename T, int kThreads>
__device__ __forceinline__ float take_edge_target(const TargetList<kThreads>& l, const RowCut<T>& cut, float amount,
                                                  float g) {
  for (int32_t n = l.head[threadIdx.x]; n >= 0; n = l.next[n]) {
    const int32_t v = l.id[n];
    if (cut.word_of(v) < 0 && cut.edge_of(v) == static_cast<int32_t>(threadIdx.x)) g = fmaf(-amount, l.sum[n], g);
  }
  return g;
}

// Stores the targets' elements of a gradient row whose other elements are
// stored already: g = coef exp2((z - base) scale) - amount * sum.
template <typename T, int kThreads>
__device__ __forceinline__ void put_targets(const TargetList<kThreads>& l, T* out, float coef, float base,
                                            float scale, float amount) {
  for (int32_t n = l.head[threadIdx.x]; n >= 0; n = l.next[n]) {
    const float g = coef * exp2_fast((l.z[n] - base) * scale);
    out[l.id[n]] = Elem<T>::round(fmaf(-amount, l.sum[n], g));
  }
}

}  // namespace thdcp
