// Label log-probabilities and their gradient, and the two-pass form of the
// losses for few rows (each row cut into parts over many workgroups).
//
// The log-probabilities read the logits once and write 8 bytes a row: 256
// threads stream a row with 8 words each in flight, the maximum and sum held
// as they go (32768 x 32000 bf16, a tenth masked: 275 us, 6.9 TB/s; a pure read
// stream 7.3).
#include <atomic>

#include "thd_loss_device.h"

namespace thdcp {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 16 * kThreads;  // bytes from one of a thread's words to the next
// The gradient of the log-probabilities has everything it needs with the row: a
// copy with an exponential per element.  8 KiB tiles (2 words a thread) in
// chunks of 16 tiles per XCD run at 6.4 TB/s, 95 % of a plain copy (16384 x
// 65536 bf16 637 us; 4 KiB tiles 709-716, 16 KiB 686-727, 32 KiB 714-730; plain
// order 666).
constexpr int kGradAhead = 2;
constexpr int kBackwardTurns = 2;
constexpr int kBackwardChunkShift = 4;
constexpr int kMaxParts = 64;         // one per lane of the wave that joins them

__global__ void status_init_kernel(int32_t* status) { *status = THD_OK; }

// Which row and part of it a workgroup has.  A part is `turns` turns of 256
// words, counted from the 128-byte line that holds the row's first word.
struct PartOf {
  int64_t row;
  int32_t part;
  __device__ __forceinline__ PartOf(const LossParts& p, int32_t row0, int32_t tiles) {
    const int32_t tile = tile_of(blockIdx.x, tiles, p.chunk_shift);
    row = row0 + static_cast<int64_t>(tile / p.parts);
    part = tile % p.parts;
  }
};

// Maximum and sum of a row's part.  With one part the row's log-probability
// and log-sum-exp are written, else the part's pair; part 0 also saves the
// logits of the row's targets, which the second pass may overwrite.
template <typename T, LossKind kKind, int kThreads>
__global__ __launch_bounds__(kThreads) void row_stats_kernel(LogitRows r, LossArgs a, LossParts p, int32_t row0) {
  constexpr int kPer = Elem<T>::kPer;
  constexpr int kStep = 16 * kThreads;
  constexpr int kStatsAhead = kThreads == 256 ? 8 : 4;  // words a thread has in flight
  __shared__ float2 s_red[kThreads / 64];
  const int32_t tid = threadIdx.x;
  if (a.scan && blockIdx.x == gridDim.x - 1) return scan_status<kThreads>(a, r.rows, r.vocab);
  const auto [row, part] = PartOf(p, row0, gridDim.x - a.scan);
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
        if (a.status && !a.scan) *a.status = THD_ERR_LABEL;
      }
      return;
    }
  }

  const RowCut<T> cut(in, r.vocab);
  const RowWords<T> words(in + cut.head, cut.words);
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
  const Word4 nothing = {Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord};
  const int32_t begin = part * p.turns * kStep - 16 * line_shift(in + cut.head);
  const int32_t end = min(begin + p.turns * kStep, words.bytes);
  // the label's column stays out of the sum until the end
  int32_t label_at = -1, label_place = 0;
  if constexpr (kKind != kLossDistill) {
    const int32_t w = cut.word_of(static_cast<int32_t>(label));
    if (w >= 0) label_at = 16 * w;
    label_place = cut.place_of(static_cast<int32_t>(label));
    if (part == 0 && tid < cut.edge && cut.edge_column(tid) == label) edge[0] = kNegInf;
  }
  Stat st;
  for (int32_t b0 = begin; b0 < end; b0 += kStatsAhead * kStep) {
    Word4 x[kStatsAhead];
    const int32_t b = b0 + 16 * tid;
#pragma unroll
    for (int k = 0; k < kStatsAhead; ++k) x[k] = words.load(b + k * kStep);
    if (b0 < 0 || b0 + kStatsAhead * kStep > end) {
#pragma unroll
      for (int k = 0; k < kStatsAhead; ++k)
        if (b + k * kStep < 0 || b + k * kStep >= end) x[k] = nothing;
    }
#pragma unroll
    for (int k = 0; k < kStatsAhead; k += 2) {
      if (b0 + k * kStep >= end) break;
      float f[2 * kPer], one[kPer];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Elem<T>::unpack(x[k + j], one);
        if (kKind != kLossDistill && b + (k + j) * kStep == label_at) drop(one, label_place);
#pragma unroll
        for (int e = 0; e < kPer; ++e) f[j * kPer + e] = one[e];
      }
      absorb(st, f, scale);
    }
  }
  absorb(st, edge, scale);
  st = join_block<kThreads>(st, scale, s_red);
  if (tid != 0) return;
  if (p.parts > 1) {
    p.stats[row * p.parts + part] = make_float2(st.m, st.s);
    if (kKind != kLossDistill && part == 0) p.targets[row] = z_label;
  } else {
    a.logp[row] = join_label(st, z_label, scale).logp;
    a.lse[row] = log_sum_exp(st);
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
  return join_lanes<false>(st, scale);
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
    Stat st = join_parts(p, row, kLog2e);
    logp = join_label(st, p.targets[row], kLog2e).logp;
    lse = log_sum_exp(st);
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
  const auto [row, part] = PartOf(p, row0, gridDim.x);
  const T* in = static_cast<const T*>(r.in) + row * r.in_stride;
  T* out = static_cast<T*>(r.out) + row * r.out_stride;

  const RowCut<T> cut(in, r.vocab);
  const RowWords<T> words(in + cut.head, cut.words);
  const int32_t shift = line_shift(out + cut.head);
  const int32_t begin = part * p.turns * kStep - 16 * shift;
  const int32_t end = min(begin + p.turns * kStep, words.bytes);
  bool live = !a.mask || a.mask[row] != 0;
  bool bad = false;
  int64_t label = 0;
  if constexpr (kKind != kLossDistill) {
    label = a.labels[row];
    bad = live && (label < 0 || label >= r.vocab);
  }
  TeacherRaw raw;
  if constexpr (kKind == kLossDistill) {
    if (live && tid < 64) read_teacher(raw, a, row);
  }
  // the row's values and its first words, read in one round trip
  PolicyValues values;
  if constexpr (kKind == kLossPolicy) values = policy_values(a, row);
  Word4 x[kGradAhead];
  if (live) {
#pragma unroll
    for (int k = 0; k < kGradAhead; ++k) x[k] = words.load(begin + 16 * tid + k * kStep);
  }
  if constexpr (kKind == kLossDistill) {
    if (live) {
      if (tid < 64) {
        float z[kMine];
        list_targets<T, kThreads, kRestBit>(s_list, raw, z, a, row, in, p.targets, cut, r.vocab,
                                            part * p.turns * kThreads - shift, p.turns * kThreads, 0, part == 0);
        store_logits(s_list.z, z, a.k);
      }
      __syncthreads();
      const int32_t state = __builtin_amdgcn_readfirstlane(s_list.state);
      bad = state == kRowBad;
      live = state == kRowLive;
    }
  }
  if (!live || bad) {
    // the gradient row's words, by its own place: the parts tile them too
    const int32_t v0 = part * p.turns * kThreads;
    const int32_t v1 = part == p.parts - 1 ? INT32_MAX : v0 + p.turns * kThreads;
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
  float label_gradient = 0.0f;
  if constexpr (kKind == kLossLogp) {
    base = a.lse_in[row];  // NaN where the row has no softmax
    amount = -a.dlogp[row];
    coef = amount;
  } else {
    Stat st = join_parts(p, row, scale);
    if constexpr (kKind == kLossPolicy) {
      const LabelJoin joined = join_label(st, p.targets[row], scale);
      base = base_of(st.m);
      const PolicyRow pr = policy_row(a, values, joined.logp);
      amount = -pr.dlogp;
      label_gradient = pr.dlogp * joined.not_q;
      if (part == 0 && tid == 0) {
        a.loss[row] = pr.loss;
        a.logp[row] = joined.logp;
      }
    } else {
      base = base_of(st.m);
      const float w = a.weights ? a.weights[row] : 1.0f;
      amount = a.temperature * w;
      if (part == 0 && tid < 64) {
        const float loss = distill_loss(s_list, a, w, [&](float z) { return (z - base) * scale; }, logf(st.s));
        if (tid == 0) a.loss[row] = loss;
      }
    }
    coef = amount * reciprocal(st.s);
  }

  // the label's element: from the sum of the others where that is known, else
  // the difference to its own probability
  const auto at_label = [&](float g) { return kKind == kLossPolicy ? label_gradient : g - amount; };
  uint32_t hit = 0;
  if constexpr (kKind == kLossDistill) hit = s_list.hit[tid];
  if (same_place(in, out)) {
    const RowWords<T> to(out + cut.head, cut.words);
    const int32_t label_word = kKind != kLossDistill ? cut.word_of(static_cast<int32_t>(label)) : -1;
    const int32_t label_at = label_word >= 0 ? 16 * label_word : -1;
    const int32_t label_place = kKind != kLossDistill ? cut.place_of(static_cast<int32_t>(label)) : 0;
    for (int32_t b = begin + 16 * tid; b < end; b += kGradAhead * kStep) {
      if (b != begin + 16 * tid) {
#pragma unroll
        for (int k = 0; k < kGradAhead; ++k) x[k] = words.load(b + k * kStep);
      }
#pragma unroll
      for (int k = 0; k < kGradAhead; ++k) {
        const int32_t at = b + k * kStep;
        if (at >= end) break;
        float f[kPer], g[kPer];
        Elem<T>::unpack(x[k], f);
#pragma unroll
        for (int e = 0; e < kPer; ++e) g[e] = coef * exp2_fast((f[e] - base) * scale);
        if constexpr (kKind != kLossDistill) {
          if (at == label_at) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
              if (e == label_place) g[e] = at_label(g[e]);
          }
        } else {
          const int bit = min((at - begin) / kStep, kRestBit);
          if ((hit >> bit) & 1u) take_targets<T, kThreads>(s_list, cut, at / 16, amount, g);
        }
        to.store(at, Elem<T>::pack(g));
      }
    }
    if (part == 0 && tid < cut.edge) {
      const int32_t v = cut.edge_column(tid);
      float g = coef * exp2_fast((Elem<T>::load(in + v) - base) * scale);
      if constexpr (kKind != kLossDistill) {
        if (v == label) g = at_label(g);
      } else {
        if ((hit >> kEdgeBit) & 1u) g = take_edge_target<T, kThreads>(s_list, cut, amount, g);
      }
      out[v] = Elem<T>::round(g);
    }
    return;
  }
  // a gradient row at another place within 16 bytes: element by element (of the
  // log-probabilities, 8192 x 50257 bf16: 554 us against 271 for rows alike). Every
  // element has one owner: the part that holds its word, or part 0 for the row's
  // edge, head and tail, whose targets it lists.
  const auto store = [&](int32_t v) {
    float g = coef * exp2_fast((Elem<T>::load(in + v) - base) * scale);
    if (kKind != kLossDistill && v == label) g = at_label(g);
    out[v] = Elem<T>::round(g);
  };
  const int32_t to_v = cut.head + end / 16 * kPer;
  for (int32_t v = cut.head + max(begin, 0) / 16 * kPer + tid; v < to_v; v += kThreads) store(v);
  if (part == 0 && tid < cut.edge) store(cut.edge_column(tid));
  if constexpr (kKind == kLossDistill) {
    __syncthreads();  // a target's element is stored again, after the first time
    put_targets<T, kThreads>(s_list, out, coef, base, scale, amount);
  }
}

int32_t words_of(int32_t vocab, int32_t dtype) { return vocab / (dtype == THD_FP32 ? 4 : 8); }

// Rows that 1024 threads each read faster than 256 do: where a compute unit has
// few (256 rows of 65536 bf16 8.4 us against 9.7; 32768 rows of 32000 columns
// 359 us against 275).
constexpr int kWideThreads = 1024;
bool wide_rows(int32_t rows, int32_t vocab, int32_t dtype) {
  return words_of(vocab, dtype) > 2048 && rows <= 2 * compute_units();
}

// About `want` parts a row: the turns of a part, and the parts that cover a
// row whose first word lies anywhere in its 128-byte line.
LossParts cut_row(int64_t want, int32_t vocab, int32_t dtype) {
  const int64_t turns = (words_of(vocab, dtype) + 7LL + kThreads - 1) / kThreads;
  if (want > kMaxParts) want = kMaxParts;
  if (want < 1) want = 1;
  LossParts p{};
  p.turns = static_cast<int32_t>((turns + want - 1) / want);
  p.parts = static_cast<int32_t>((turns + p.turns - 1) / p.turns);
  return p;
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
    if constexpr (kKind == kLossLogp) {
      if (p.parts == 1 && wide_rows(r.rows, r.vocab, r.dtype)) {
        LossParts whole = p;
        whole.turns = (words_of(r.vocab, r.dtype) + 7) / kWideThreads + 1;
        return over_rows(r.rows, kWideThreads / kThreads, [&](dim3, int32_t row0) {
          const int32_t slice = static_cast<int32_t>((1LL << 31) / kWideThreads);
          const int32_t n = r.rows - row0 < slice ? r.rows - row0 : slice;
          hipLaunchKernelGGL((row_stats_kernel<T, kKind, kWideThreads>), dim3(n + a.scan), dim3(kWideThreads), 0,
                             stream, r, a, whole, row0);
        });
      }
    }
    return over_rows(r.rows, p.parts, [&](dim3 grid, int32_t row0) {
      hipLaunchKernelGGL((row_stats_kernel<T, kKind, kThreads>), dim3(grid.x + a.scan), dim3(kThreads), 0,
                         stream, r, a, p, row0);
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

int32_t compute_units() {
  static std::atomic<int32_t> known[64];
  int device = 0;
  if (hipGetDevice(&device) != hipSuccess || device < 0 || device >= 64) return 256;
  int32_t n = known[device].load(std::memory_order_relaxed);
  if (n == 0) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || v < 1) return 256;
    n = v;
    known[device].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Two launches take about 2 us more than one, which they gain back where a row
// is long and the rows are few (bf16, us per call, two launches against one):
// log-probabilities of 65536 columns 5.5 / 5.9 for one row, 8.2 / 7.1 for 64;
// of 131072 columns 5.5 / 8.8, 9.5 / 11.0 for 64, 13.8 / 11.5 for 128; the
// policy loss of 32000 columns 6.8 / 6.4, of 50000 6.6 / 8.0, 8.0 / 8.6 for 32
// and 9.4 / 8.7 for 64, of 131072 6.7 / 13.9, 9.9 / 14.4 and 15.6 / 14.5.
LossParts logp_parts(int32_t rows, int32_t vocab, int32_t dtype) {
  return cut_row(rows < 1 || rows > 64 || words_of(vocab, dtype) <= 8192 ? 1 : 1024 / rows, vocab, dtype);
}

LossParts loss_parts(int32_t rows, int32_t vocab, int32_t dtype) {
  return cut_row(rows < 1 || rows > 48 || words_of(vocab, dtype) <= 4096 ? 1 : 512 / rows, vocab, dtype);
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
  const int64_t turns = (words_of(r.vocab, r.dtype) + 7LL + kThreads - 1) / kThreads;
  LossParts p{};
  p.turns = kBackwardTurns;
  p.parts = static_cast<int32_t>((turns + kBackwardTurns - 1) / kBackwardTurns);
  p.chunk_shift = kBackwardChunkShift;
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
