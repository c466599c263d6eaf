// Label log-probabilities and their gradient, and the two-pass form of the
// losses for few rows (each row cut into parts over many workgroups).
#include "thd_loss_device.h"

namespace thdcp {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;      // words a thread has in flight
constexpr int kMaxParts = 64;  // one per lane of the wave that joins them

__global__ void status_init_kernel(int32_t* status) { *status = THD_OK; }

// A part's words [w0, w1) of a row of `words` words cut into `parts`.
__device__ __forceinline__ void part_words(int32_t words, int32_t parts, int32_t part, int32_t* w0, int32_t* w1) {
  const int32_t per = (words + parts - 1) / parts;
  *w0 = min(part * per, words);
  *w1 = min(*w0 + per, words);
}

// Maximum and sum of a row's part.  With one part the row's log-probability
// and log-sum-exp are written, else the part's pair; part 0 also saves the
// logits of the row's targets, which the second pass may overwrite.
template <typename T, LossKind kKind>
__global__ __launch_bounds__(kThreads) void row_stats_kernel(LogitRows r, LossArgs a, LossParts p, int32_t row0) {
  constexpr int kPer = Elem<T>::kPer;
  __shared__ float2 s_red[kThreads / 64];
  const int32_t tid = threadIdx.x;
  const int64_t row = row0 + static_cast<int64_t>(blockIdx.x / p.parts);
  const int32_t part = blockIdx.x % p.parts;
  const T* in = static_cast<const T*>(r.in) + row * r.in_stride;
  // in the two-pass form only the second pass reports errors
  if (a.status && p.parts > 1 && blockIdx.x == 0 && row0 == 0 && tid == 0) *a.status = THD_OK;

  int64_t label = 0;
  if constexpr (kKind != kLossDistill) label = a.labels[row];
  if (a.mask && a.mask[row] == 0) {
    if (kKind == kLossLogp && p.parts == 1 && tid == 0) a.logp[row] = a.lse[row] = 0.0f;
    return;
  }
  if constexpr (kKind != kLossDistill) {
    if (label < 0 || label >= r.vocab) {
      if (kKind == kLossLogp && p.parts == 1 && tid == 0) {
        a.logp[row] = a.lse[row] = __builtin_nanf("");
        if (a.status) *a.status = THD_ERR_LABEL;
      }
      return;
    }
  }

  const RowCut<T> cut(in, r.vocab);
  const Word4* body = reinterpret_cast<const Word4*>(in + cut.head);
  int32_t w0, w1;
  part_words(cut.words, p.parts, part, &w0, &w1);
  float edge[1] = {kNegInf};
  float z_label = 0.0f;
  if (part == 0) {
    if (tid < cut.edge) edge[0] = Elem<T>::load(in + cut.edge_column(tid));
    if constexpr (kKind == kLossDistill) {
      if (tid < a.k) {
        const int64_t at = row * a.teacher_stride + tid;
        const int64_t v = a.ids64 ? static_cast<const int64_t*>(a.teacher_ids)[at]
                                  : static_cast<const int32_t*>(a.teacher_ids)[at];
        if (v >= 0 && v < r.vocab) p.targets[row * a.k + tid] = Elem<T>::load(in + v);
      }
    } else {
      z_label = Elem<T>::load(in + label);
    }
  }
  const float scale = kKind == kLossDistill ? a.inv_temperature * kLog2e : kLog2e;
  Stat st;
  int32_t w = w0 + tid;
  for (; w + (kAhead - 1) * kThreads < w1; w += kAhead * kThreads) {
    Word4 x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) x[k] = load_word(body + w + k * kThreads);
#pragma unroll
    for (int k = 0; k < kAhead; k += 2) {
      float f[2 * kPer], one[kPer];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Elem<T>::unpack(x[k + j], one);
#pragma unroll
        for (int e = 0; e < kPer; ++e) f[j * kPer + e] = one[e];
      }
      absorb(st, f, scale);
    }
  }
  for (; w < w1; w += kThreads) {
    float f[kPer];
    Elem<T>::unpack(load_word(body + w), f);
    absorb(st, f, scale);
  }
  absorb(st, edge, scale);
  st = join_block<kThreads>(st, scale, s_red);
  if (tid != 0) return;
  if (p.parts > 1) {
    p.stats[row * p.parts + part] = make_float2(st.m, st.s);
    if (kKind != kLossDistill && part == 0) p.targets[row] = z_label;
  } else {
    const float ln_s = logf(st.s);
    a.logp[row] = (z_label - st.m) - ln_s;
    a.lse[row] = st.m + ln_s;
  }
}

// Joins a row's parts; every lane of every wave gets the same result.
__device__ __forceinline__ Stat join_parts(const LossParts& p, int64_t row, float scale) {
  const int lane = threadIdx.x & 63;
  Stat st;
  if (lane < p.parts) {
    const float2 v = p.stats[row * p.parts + lane];
    st = Stat{v.x, v.y};
  }
  return join_lanes<64>(st, scale);
}

// Log-probability and log-sum-exp from the parts: one wave per row.
__global__ __launch_bounds__(64) void logp_join_kernel(LogitRows r, LossArgs a, LossParts p) {
  const int64_t row = blockIdx.x;
  const int64_t label = a.labels[row];
  const bool live = !a.mask || a.mask[row] != 0;
  const bool bad = live && (label < 0 || label >= r.vocab);
  float logp = 0.0f, lse = 0.0f;
  if (bad) {
    logp = lse = __builtin_nanf("");
    if (a.status && threadIdx.x == 0) *a.status = THD_ERR_LABEL;
  } else if (live) {
    const Stat st = join_parts(p, row, kLog2e);
    const float ln_s = logf(st.s);
    logp = (p.targets[row] - st.m) - ln_s;
    lse = st.m + ln_s;
  }
  if (threadIdx.x == 0) {
    a.logp[row] = logp;
    a.lse[row] = lse;
  }
}

// Gradient of a row's part: of the log-probabilities (given the row's
// log-sum-exp) or of a loss (given the parts of the first pass).
template <typename T, LossKind kKind>
__global__ __launch_bounds__(kThreads) void part_grad_kernel(LogitRows r, LossArgs a, LossParts p, int32_t row0) {
  constexpr int kPer = Elem<T>::kPer;
  struct NoList {
    int32_t state;
  };
  using List = typename std::conditional<kKind == kLossDistill, TargetList<kThreads>, NoList>::type;
  __shared__ List s_list;
  const int32_t tid = threadIdx.x;
  const int64_t row = row0 + static_cast<int64_t>(blockIdx.x / p.parts);
  const int32_t part = blockIdx.x % p.parts;
  const T* in = static_cast<const T*>(r.in) + row * r.in_stride;
  T* out = static_cast<T*>(r.out) + row * r.out_stride;

  const RowCut<T> cut(in, r.vocab);
  const Word4* body = reinterpret_cast<const Word4*>(in + cut.head);
  int32_t w0, w1;
  part_words(cut.words, p.parts, part, &w0, &w1);
  // 0: live, else the value that fills the part
  bool live = !a.mask || a.mask[row] != 0;
  bool bad = false;
  int64_t label = 0;
  if constexpr (kKind != kLossDistill) {
    label = a.labels[row];
    bad = live && (label < 0 || label >= r.vocab);
  }
  // the first words, read in the same round trip as the row's values
  Word4 x[kAhead];
  if (live) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (w0 + k * kThreads + tid < w1) x[k] = load_word(body + w0 + k * kThreads + tid);
  }
  if constexpr (kKind == kLossDistill) {
    if (live) {
      if (tid < 64)
        list_targets<T, kThreads, kRestBit>(s_list, a, row, in, p.targets, cut, r.vocab, w0, w1 - w0, part == 0);
      __syncthreads();
      bad = s_list.state == kRowBad;
      live = s_list.state == kRowLive;
    }
  }
  if (!live || bad) {
    // the gradient row's words, by its own alignment: the parts tile them too
    const RowCut<T> to(out, r.vocab);
    int32_t v0, v1;
    part_words(to.words, p.parts, part, &v0, &v1);
    fill_words<T>(out, r.vocab, bad ? Elem<T>::kNanWord : 0u, v0, v1, part == 0, kThreads);
    if (kKind != kLossLogp && part == 0 && tid == 0) {
      const float v = bad ? __builtin_nanf("") : 0.0f;
      a.loss[row] = v;
      if (kKind == kLossPolicy) a.logp[row] = v;
      if (bad && a.status) *a.status = THD_ERR_LABEL;
    }
    return;
  }

  const float scale = kKind == kLossDistill ? a.inv_temperature * kLog2e : kLog2e;
  float base, coef, amount;
  if constexpr (kKind == kLossLogp) {
    base = base_of(a.lse_in[row]);
    amount = -a.dlogp[row];
    coef = amount;
  } else {
    const Stat st = join_parts(p, row, scale);
    base = base_of(st.m);
    if constexpr (kKind == kLossPolicy) {
      const float logp = (p.targets[row] - st.m) - logf(st.s);
      const PolicyRow pr = policy_row(a, row, logp);
      amount = -pr.dlogp;
      if (part == 0 && tid == 0) {
        a.loss[row] = pr.loss;
        a.logp[row] = logp;
      }
    } else {
      const float w = a.weights ? a.weights[row] : 1.0f;
      amount = a.temperature * w;
      if (part == 0 && tid < 64) {
        const float loss = distill_loss(s_list, a, w, st.m, logf(st.s));
        if (tid == 0) a.loss[row] = loss;
      }
    }
    coef = amount / st.s;
  }

  const OutRow<T> dst(out, in, cut.head);
  const int32_t label_word = kKind != kLossDistill ? cut.word_of(static_cast<int32_t>(label)) : -1;
  const int32_t label_place = kKind != kLossDistill ? cut.place_of(static_cast<int32_t>(label)) : 0;
  uint32_t hit = 0;
  if constexpr (kKind == kLossDistill) hit = s_list.hit[tid];
  auto gradient = [&](Word4 word, int32_t w) {
    float f[kPer], g[kPer];
    Elem<T>::unpack(word, f);
#pragma unroll
    for (int e = 0; e < kPer; ++e) g[e] = coef * exp2_fast((f[e] - base) * scale);
    if constexpr (kKind != kLossDistill) {
      if (w == label_word) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (e == label_place) g[e] -= amount;
      }
    } else {
      const int bit = min((w - w0) / kThreads, kRestBit);
      if ((hit >> bit) & 1u) take_targets<T, kThreads>(s_list, cut, w, amount, g);
    }
    dst.store(w, g);
  };
  for (int32_t w = w0 + tid; w < w1; w += kAhead * kThreads) {
    if (w != w0 + tid) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (w + k * kThreads < w1) x[k] = load_word(body + w + k * kThreads);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (w + k * kThreads < w1) gradient(x[k], w + k * kThreads);
  }
  if (part == 0 && tid < cut.edge) {
    const int32_t v = cut.edge_column(tid);
    float g = coef * exp2_fast((Elem<T>::load(in + v) - base) * scale);
    if constexpr (kKind != kLossDistill) {
      if (v == label) g -= amount;
    } else {
      if ((hit >> kEdgeBit) & 1u) g = take_edge_target<T, kThreads>(s_list, cut, amount, g);
    }
    out[v] = Elem<T>::round(g);
  }
}

int32_t words_of(int32_t vocab, int32_t dtype) { return vocab / (dtype == THD_FP32 ? 4 : 8); }

int32_t clamp_parts(int64_t want, int32_t words) {
  const int64_t most = words / kThreads < kMaxParts ? words / kThreads : kMaxParts;
  if (want > most) want = most;
  return want < 1 ? 1 : static_cast<int32_t>(want);
}

// Slices of rows whose workgroups a grid can count (2^32 threads).
template <typename F>
hipError_t over_rows(int32_t rows, int32_t parts, F launch) {
  const int64_t slice = (1LL << 31) / kThreads / parts;
  for (int64_t row0 = 0; row0 < rows; row0 += slice) {
    const int64_t n = rows - row0 < slice ? rows - row0 : slice;
    launch(dim3(static_cast<unsigned>(n * parts)), static_cast<int32_t>(row0));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename F>
hipError_t by_dtype(int32_t dtype, F f) {
  switch (dtype) {
    case THD_BF16: return f(Bf16{});
    case THD_FP16: return f(Fp16{});
    default: return f(float{});
  }
}

template <LossKind kKind>
hipError_t launch_stats(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream) {
  return by_dtype(r.dtype, [&](auto t) {
    using T = decltype(t);
    return over_rows(r.rows, p.parts, [&](dim3 grid, int32_t row0) {
      hipLaunchKernelGGL((row_stats_kernel<T, kKind>), grid, dim3(kThreads), 0, stream, r, a, p, row0);
    });
  });
}

template <LossKind kKind>
hipError_t launch_part_grad(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream) {
  return by_dtype(r.dtype, [&](auto t) {
    using T = decltype(t);
    return over_rows(r.rows, p.parts, [&](dim3 grid, int32_t row0) {
      hipLaunchKernelGGL((part_grad_kernel<T, kKind>), grid, dim3(kThreads), 0, stream, r, a, p, row0);
    });
  });
}

}  // namespace

int32_t logp_parts(int32_t rows, int32_t vocab, int32_t dtype) {
  return rows < 1 ? 1 : clamp_parts(1024 / rows, words_of(vocab, dtype));
}

int32_t loss_parts(int32_t rows, int32_t vocab, int32_t dtype) {
  return rows < 1 ? 1 : clamp_parts(512 / rows, words_of(vocab, dtype));
}

hipError_t launch_status_init(int32_t* status, hipStream_t stream) {
  hipLaunchKernelGGL(status_init_kernel, dim3(1), dim3(1), 0, stream, status);
  return hipGetLastError();
}

hipError_t launch_token_logprobs(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream) {
  const hipError_t e = launch_stats<kLossLogp>(r, a, p, stream);
  if (e != hipSuccess || p.parts == 1) return e;
  hipLaunchKernelGGL(logp_join_kernel, dim3(r.rows), dim3(64), 0, stream, r, a, p);
  return hipGetLastError();
}

hipError_t launch_logp_backward(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  const int32_t words = words_of(r.vocab, r.dtype);
  LossParts p{};
  p.parts = words / (kAhead * kThreads) > 0 ? (words + kAhead * kThreads - 1) / (kAhead * kThreads) : 1;
  return launch_part_grad<kLossLogp>(r, a, p, stream);
}

hipError_t launch_policy_parts(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream) {
  const hipError_t e = launch_stats<kLossPolicy>(r, a, p, stream);
  if (e != hipSuccess) return e;
  return launch_part_grad<kLossPolicy>(r, a, p, stream);
}

hipError_t launch_distill_parts(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream) {
  const hipError_t e = launch_stats<kLossDistill>(r, a, p, stream);
  if (e != hipSuccess) return e;
  return launch_part_grad<kLossDistill>(r, a, p, stream);
}

}  // namespace thdcp
