// One workgroup per row of logits: the policy loss and the distillation in one
// pass.  The row is read once into registers, its maximum and sum are formed as
// the words arrive, the gradient is computed from the registers and stored:
// one read and one write of the logits, the least the operation can move.
#pragma once

#include "thd_loss_device.h"

namespace thdcp {

constexpr int kJoinWords = 2;  // words absorbed at a time: 16 elements share one rescale

template <typename T, int kThreads, int kWords, LossKind kKind>
__global__ __launch_bounds__(kThreads, 4) void row_loss_kernel(LogitRows r, LossArgs a, int32_t row0) {
  constexpr int kPer = Elem<T>::kPer;
  static_assert(kWords % kJoinWords == 0 && kWords < kRestBit);
  struct NoList {
    int32_t state;
  };
  using List = typename std::conditional<kKind == kLossDistill, TargetList<kThreads>, NoList>::type;
  __shared__ float2 s_red[kThreads / 64];
  __shared__ List s_list;
  const int32_t tid = threadIdx.x;
  const int64_t row = static_cast<int64_t>(row0) + blockIdx.x;
  const T* in = static_cast<const T*>(r.in) + row * r.in_stride;
  T* out = static_cast<T*>(r.out) + row * r.out_stride;

  int64_t label = 0;
  if constexpr (kKind == kLossPolicy) label = a.labels[row];
  if (a.mask && a.mask[row] == 0) {
    fill_words<T>(out, r.vocab, 0u, 0, INT32_MAX, true, kThreads);
    if (tid == 0) {
      a.loss[row] = 0.0f;
      if (kKind == kLossPolicy) a.logp[row] = 0.0f;
    }
    return;
  }
  if (kKind == kLossPolicy && (label < 0 || label >= r.vocab)) {
    fill_words<T>(out, r.vocab, Elem<T>::kNanWord, 0, INT32_MAX, true, kThreads);
    if (tid == 0) {
      a.loss[row] = a.logp[row] = __builtin_nanf("");
      if (a.status) *a.status = THD_ERR_LABEL;
    }
    return;
  }

  const RowCut<T> cut(in, r.vocab);
  const Word4* body = reinterpret_cast<const Word4*>(in + cut.head);
  Word4 x[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int32_t w = k * kThreads + tid;
    x[k] = Word4{Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord};
    if (w < cut.words) x[k] = load_word(body + w);
  }
  float edge[1] = {kNegInf};
  if (tid < cut.edge) edge[0] = Elem<T>::load(in + cut.edge_column(tid));
  float z_label = 0.0f;
  if constexpr (kKind == kLossPolicy) z_label = Elem<T>::load(in + label);
  if constexpr (kKind == kLossDistill) {
    if (tid < 64) list_targets<T, kThreads, kWords>(s_list, a, row, in, nullptr, cut, r.vocab, 0, cut.words, true);
  }

  const float scale = kKind == kLossDistill ? a.inv_temperature * kLog2e : kLog2e;
  Stat st;
#pragma unroll
  for (int k = 0; k < kWords; k += kJoinWords) {
    float f[kJoinWords * kPer];
#pragma unroll
    for (int j = 0; j < kJoinWords; ++j) {
      float one[kPer];
      Elem<T>::unpack(x[k + j], one);
#pragma unroll
      for (int e = 0; e < kPer; ++e) f[j * kPer + e] = one[e];
    }
    absorb(st, f, scale);
  }
  for (int32_t w = kWords * kThreads + tid; w < cut.words; w += kThreads) {
    float f[kPer];
    Elem<T>::unpack(body[w], f);
    absorb(st, f, scale);
  }
  absorb(st, edge, scale);
  st = join_block<kThreads>(st, scale, s_red);
  // The words are unpacked a second time below.  Without this the compiler
  // keeps the 32-bit values of the first time instead: for 16-bit elements
  // twice the registers there are, spilled to memory.
#pragma unroll
  for (int k = 0; k < kWords; ++k) asm volatile("" : "+v"(x[k]));

  const float base = base_of(st.m);
  float coef, amount;  // of q, and of the targets
  if constexpr (kKind == kLossPolicy) {
    const float logp = (z_label - st.m) - logf(st.s);
    const PolicyRow p = policy_row(a, row, logp);
    if (tid == 0) {
      a.loss[row] = p.loss;
      a.logp[row] = logp;
    }
    amount = -p.dlogp;
  } else {
    if (s_list.state != kRowLive) {
      const bool bad = s_list.state == kRowBad;
      fill_words<T>(out, r.vocab, bad ? Elem<T>::kNanWord : 0u, 0, INT32_MAX, true, kThreads);
      if (tid == 0) {
        a.loss[row] = bad ? __builtin_nanf("") : 0.0f;
        if (bad && a.status) *a.status = THD_ERR_LABEL;
      }
      return;
    }
    const float w = a.weights ? a.weights[row] : 1.0f;
    if (tid < 64) {
      const float loss = distill_loss(s_list, a, w, st.m, logf(st.s));
      if (tid == 0) a.loss[row] = loss;
    }
    amount = a.temperature * w;
  }
  coef = amount / st.s;

  const OutRow<T> dst(out, in, cut.head);
  const int32_t label_word = kKind == kLossPolicy ? cut.word_of(static_cast<int32_t>(label)) : -1;
  const int32_t label_place = kKind == kLossPolicy ? cut.place_of(static_cast<int32_t>(label)) : 0;
  uint32_t hit = 0;
  if constexpr (kKind == kLossDistill) hit = s_list.hit[tid];

  auto gradient = [&](Word4 word, int32_t w, int bit) {
    float f[kPer], g[kPer];
    Elem<T>::unpack(word, f);
#pragma unroll
    for (int e = 0; e < kPer; ++e) g[e] = coef * exp2_fast((f[e] - base) * scale);
    if constexpr (kKind == kLossPolicy) {
      if (w == label_word) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (e == label_place) g[e] -= amount;
      }
    } else {
      if ((hit >> bit) & 1u) take_targets<T, kThreads>(s_list, cut, w, amount, g);
    }
    dst.store(w, g);
  };
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int32_t w = k * kThreads + tid;
    if (w < cut.words) gradient(x[k], w, k);
  }
  for (int32_t w = kWords * kThreads + tid; w < cut.words; w += kThreads) gradient(body[w], w, kRestBit);
  if (tid < cut.edge) {
    float g = coef * exp2_fast((edge[0] - base) * scale);
    if constexpr (kKind == kLossPolicy) {
      if (cut.edge_column(tid) == label) g -= amount;
    } else {
      if ((hit >> kEdgeBit) & 1u) g = take_edge_target<T, kThreads>(s_list, cut, amount, g);
    }
    out[cut.edge_column(tid)] = Elem<T>::round(g);
  }
}

// Launches in slices whose threads a grid can count (2^32).
template <typename T, int kThreads, int kWords, LossKind kKind>
hipError_t launch_rows_as(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  constexpr int32_t kSlice = static_cast<int32_t>((1LL << 31) / kThreads);
  for (int64_t row0 = 0; row0 < r.rows; row0 += kSlice) {
    const int32_t n = static_cast<int32_t>(r.rows - row0 < kSlice ? r.rows - row0 : kSlice);
    hipLaunchKernelGGL((row_loss_kernel<T, kThreads, kWords, kKind>), dim3(n), dim3(kThreads), 0, stream, r, a,
                       static_cast<int32_t>(row0));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, LossKind kKind>
hipError_t launch_rows(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  const int32_t words = r.vocab / Elem<T>::kPer;
  if (words <= 256) return launch_rows_as<T, 64, 4, kKind>(r, a, stream);
  if (words <= 1024) return launch_rows_as<T, 128, 8, kKind>(r, a, stream);
  if (words <= 2048) return launch_rows_as<T, 256, 8, kKind>(r, a, stream);
  if (words <= 4096) return launch_rows_as<T, 256, 16, kKind>(r, a, stream);
  if (words <= 8192) return launch_rows_as<T, 512, 16, kKind>(r, a, stream);
  if (words <= 16384) return launch_rows_as<T, 1024, 16, kKind>(r, a, stream);
  return launch_rows_as<T, 1024, 20, kKind>(r, a, stream);
}

template <LossKind kKind>
hipError_t launch_rows_dtype(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  switch (r.dtype) {
    case THD_BF16: return launch_rows<Bf16, kKind>(r, a, stream);
    case THD_FP16: return launch_rows<Fp16, kKind>(r, a, stream);
    default: return launch_rows<float, kKind>(r, a, stream);
  }
}

}  // namespace thdcp
