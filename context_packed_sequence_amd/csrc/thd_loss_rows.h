// One workgroup per row of logits: the policy loss and the distillation in one
// pass.  The row is read once into registers, its maximum and sum are formed as
// the words arrive, the gradient is computed from the registers and stored:
// one read and one write of the logits, the least the operation can move, and
// what the memory counters show (8192 x 131072 bf16, a tenth of the rows
// masked: 1.93 GB read, 2.15 GB written).
//
// What bounds it is memory.  A plain copy runs at 6.8 TB/s here; a workgroup
// that loads a whole row, waits, and stores it, with no arithmetic at all, at
// 5.7-6.3 TB/s (64-256 KiB rows), and this kernel at 6.1-6.5 TB/s for rows of
// up to 64 KiB, 5.6-5.9 for longer ones, where one or two workgroups fill a
// compute unit's registers.  Vector instructions are busy for 53 % of that time:
// 11.3 an element, 13.4 issue slots (an exponential, of which there are two, takes
// two).
//
// Tried and slower: workgroups that stay and load their next row into the
// registers as these are stored (loads and stores of a wave are counted in one
// order, so that the next row's words waited for this row's stores: 836 us
// against 748 for 8192 x 131072); starting the compute units apart from each
// other (no change); 512 threads with 32 words each (403 us against 380 for
// 4096 x 131072); a row's rest from cache instead of LDS (2047 x 200003: 341 us
// against 293).  Rows beyond registers and LDS do read their rest from cache:
// past it, 2048 x 262144 bf16 takes 431 us instead of 396.
#pragma once

#include "thd_loss_device.h"

namespace thdcp {

constexpr int kMostHeld = 1024 * (18 + 8);
constexpr int kRestWords = 4;  // words in flight of a row's part beyond the registers

// kWords words of a row per thread in registers, kLds more in LDS.  Up to 8 words
// leave room for 8 waves per SIMD, which runs faster than 4 waves of 16 words
// (8388 x 64000 bf16 356 us against 368); waves skip turns in which they have no
// word, so that a form serves any shorter row (134217 x 2000: 376 us without).
template <typename T, int kThreads, int kWords, int kLds, LossKind kKind>
__global__ __launch_bounds__(kThreads, kWords <= 8 ? 8 : 4) void row_loss_kernel(LogitRows r, LossArgs a, int32_t row0,
                                                               int32_t chunk_shift) {
  constexpr int kPer = Elem<T>::kPer;
  constexpr int kStep = 16 * kThreads;  // bytes from one of a thread's words to the next
  constexpr int kHeld = kWords + kLds;
  // the largest form takes rows of any length: what it cannot hold is read twice
  constexpr bool kAnyLength = kHeld * kThreads == kMostHeld;
  // words absorbed at a time, whose elements share one rescale
  constexpr int kJoinWords = kWords <= 8 ? 1 : 2;
  static_assert(kWords % kJoinWords == 0 && kHeld <= kRestBit);
  struct NoList {
    int32_t state;
  };
  using List = typename std::conditional<kKind == kLossDistill, TargetList<kThreads>, NoList>::type;
  __shared__ float2 s_red[kThreads / 64];
  __shared__ List s_list;
  extern __shared__ Word4 s_row[];  // [kLds][kThreads], each word used by its own thread alone
  const int32_t tid = threadIdx.x;
  if (a.scan && blockIdx.x == gridDim.x - 1) return scan_status<kThreads>(a, r.rows, r.vocab);
  const int64_t row = row0 + static_cast<int64_t>(tile_of(blockIdx.x, gridDim.x - a.scan, chunk_shift));
  const T* in = static_cast<const T*>(r.in) + row * r.in_stride;
  T* out = static_cast<T*>(r.out) + row * r.out_stride;
  const auto fill_row = [&](bool bad) {
    fill_words<T>(out, r.vocab, bad ? Elem<T>::kNanWord : 0u, 0, INT32_MAX, true, kThreads);
    if (tid == 0) {
      const float v = bad ? __builtin_nanf("") : 0.0f;
      a.loss[row] = v;
      if (kKind == kLossPolicy) a.logp[row] = v;
      if (bad && a.status && !a.scan) *a.status = THD_ERR_LABEL;
    }
  };

  // The row's own values and what its first columns need are issued before its
  // words: loads return in order, and these are wanted first.
  const uint8_t live = a.mask ? a.mask[row] : 1;
  int64_t label = 0;
  PolicyValues value;
  TeacherRaw raw;
  if constexpr (kKind == kLossPolicy) {
    label = a.labels[row];
    value = policy_values(a, row);
  } else {
    if (a.weights) value.weight = a.weights[row];
    if (tid < 64) read_teacher(raw, a, row);
  }
  if (!live) return fill_row(false);
  if (kKind == kLossPolicy && (label < 0 || label >= r.vocab)) return fill_row(true);

  const RowCut<T> cut(in, r.vocab);
  const RowWords<T> words(in + cut.head, cut.words);
  const int32_t shift = line_shift(out + cut.head);
  const int32_t at0 = 16 * (tid - shift);
  // turns in which this wave has a word of the row
  const int32_t wave0 = __builtin_amdgcn_readfirstlane(tid & ~63);
  const int32_t turns = (cut.words + shift - wave0 + kThreads - 1) / kThreads;
  constexpr uint32_t kNegInfRaw = sizeof(T) == 2 ? Elem<T>::kNegInfWord & 0xffffu : Elem<T>::kNegInfWord;
  uint32_t edge_raw = kNegInfRaw, label_raw = 0;
  if (tid < cut.edge) edge_raw = load_raw(in + cut.edge_column(tid));
  if constexpr (kKind == kLossPolicy) label_raw = load_raw(in + label);
  Word4 x[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) x[k] = words.load(at0 + k * kStep);
#pragma unroll
  for (int k = 0; k < kLds; ++k)
    words.load_to_lds(s_row + k * kThreads + wave0, at0 + (kWords + k) * kStep);

  float z_teacher[kMine];
  if constexpr (kKind == kLossDistill) {
    if (tid < 64)
      list_targets<T, kThreads, kHeld>(s_list, raw, z_teacher, a, row, in, nullptr, cut, r.vocab, 0, cut.words,
                                        shift, true);
  }

  int32_t label_turn = -1, label_thread = -1, label_place = 0;
  if constexpr (kKind == kLossPolicy) {
    const int32_t w = cut.word_of(label);
    if (w >= 0) {
      label_turn = (w + shift) / kThreads;
      label_thread = (w + shift) % kThreads;
      label_place = cut.place_of(label);
    }
  }
  const float scale = kKind == kLossDistill ? a.inv_temperature * kLog2e : kLog2e;
  const Word4 nothing = {Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord};
  FastStat fast;
#pragma unroll
  for (int k = 0; k < kWords; k += kJoinWords) {
    if (k >= turns) continue;
    if ((k == 0 && shift > 0) || (k + kJoinWords) * kThreads > cut.words + shift) {
      // words out of the row came as zeros
#pragma unroll
      for (int j = 0; j < kJoinWords; ++j)
        if (static_cast<uint32_t>(at0 + (k + j) * kStep) >= static_cast<uint32_t>(words.bytes)) x[k + j] = nothing;
    }
    float f[kJoinWords * kPer];
#pragma unroll
    for (int j = 0; j < kJoinWords; ++j) {
      float one[kPer];
      Elem<T>::unpack(x[k + j], one);
#pragma unroll
      for (int e = 0; e < kPer; ++e) f[j * kPer + e] = one[e];
    }
    if (label_turn >= k && label_turn < k + kJoinWords && tid == label_thread)
      drop(f, (label_turn - k) * kPer + label_place);
    absorb(fast, f, scale);
  }
  if constexpr (kLds > 0) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the words on their way to LDS
#pragma unroll
    for (int k = 0; k < kLds; ++k) {
      if (kWords + k >= turns) continue;
      float f[kPer];
      Elem<T>::unpack(at0 + (kWords + k) * kStep < words.bytes ? s_row[k * kThreads + tid] : nothing, f);
      if (kWords + k == label_turn && tid == label_thread) drop(f, label_place);
      absorb(fast, f, scale);
    }
  }
  for (int32_t b = at0 + kHeld * kStep, k = kHeld; kAnyLength && b < words.bytes; b += kRestWords * kStep, k += kRestWords) {
    Word4 y[kRestWords];
#pragma unroll
    for (int j = 0; j < kRestWords; ++j) y[j] = words.load_cached(b + j * kStep);
#pragma unroll
    for (int j = 0; j < kRestWords; ++j) {
      float f[kPer];
      Elem<T>::unpack(b + j * kStep < words.bytes ? y[j] : nothing, f);
      if (k + j == label_turn && tid == label_thread) drop(f, label_place);
      absorb(fast, f, scale);
    }
  }
  const float edge[1] = {decode<T>(edge_raw)};
  const bool label_on_edge = kKind == kLossPolicy && tid < cut.edge && cut.edge_column(tid) == label;
  absorb(fast, {label_on_edge ? kNegInf : edge[0]}, scale);
  if constexpr (kKind == kLossDistill) {
    if (tid < 64) store_logits(s_list.z, z_teacher, a.k);
  }
  fast = join_block<kThreads>(fast, scale, s_red);
  // The words are unpacked a second time below.  Without this the compiler
  // keeps the 32-bit values of the first time instead: for 16-bit elements
  // twice the registers there are, spilled to memory.
#pragma unroll
  for (int k = 0; k < kWords; ++k) asm volatile("" : "+v"(x[k]));

  // a row beyond the fast form: its sum, and below its gradient, are taken
  // element by element from memory
  LabelJoin joined;
  if constexpr (kKind == kLossPolicy) joined = join_label(fast, decode<T>(label_raw), scale);
  const bool huge = !(fabsf(fast.top) < kHuge);
  Stat st;
  if (huge) {
    st = row_stat<T, kThreads>(in, r.vocab, kKind == kLossPolicy ? label : -1, scale, s_red);
    if constexpr (kKind == kLossPolicy) joined = join_label(st, decode<T>(label_raw), scale);
  }
  const float sum = huge ? st.s : fast.s;
  const float base = base_of(st.m);
  float amount;  // factor of the targets
  int32_t state = kRowLive;
  if constexpr (kKind == kLossPolicy) {
    const PolicyRow p = policy_row(a, value, joined.logp);
    if (tid == 0) {
      a.loss[row] = p.loss;
      a.logp[row] = joined.logp;
    }
    amount = -p.dlogp;
  } else {
    state = __builtin_amdgcn_readfirstlane(s_list.state);
    if (tid < 64 && state == kRowLive) {
      // scale times the distance from the maximum
      const auto exponent = [&](float z) { return huge ? (z - base) * scale : fmaf(z, scale, -fast.top); };
      const float loss = distill_loss(s_list, a, value.weight, exponent, logf(sum));
      if (tid == 0) a.loss[row] = loss;
    }
    amount = a.temperature * value.weight;
  }
  const float coef = amount * reciprocal(sum);  // factor of the exponentials
  // in a row beyond the fast form no word is stored from the registers
  const RowWords<T> to(out + cut.head, huge ? 0 : cut.words);

  uint32_t hit = 0;
  if constexpr (kKind == kLossDistill) hit = s_list.hit[tid];
  const auto gradient = [&](Word4 word, int32_t b, int32_t k, int bit) {
    float f[kPer], g[kPer];
    Elem<T>::unpack(word, f);
#pragma unroll
    for (int e = 0; e < kPer; ++e) g[e] = coef * exp2_fast(fmaf(f[e], scale, -fast.top));
    if constexpr (kKind == kLossPolicy) {
      if (k == label_turn && tid == label_thread) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (e == label_place) g[e] = -amount * joined.not_q;
      }
    } else {
      if ((hit >> bit) & 1u) take_targets<T, kThreads>(s_list, cut, b / 16, amount, g);
    }
    to.store(b, Elem<T>::pack(g));
  };

  // the barriers keep each word's values in its own step: the scheduler would
  // gather them, and spill
  int32_t here = at0;
  asm volatile("" : "+v"(here));
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    if (k >= turns) continue;
    gradient(x[k], here, k, k);
    here += kStep;
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int k = kWords; k < kHeld; ++k) {
    if (k >= turns) continue;
    gradient(s_row[(k - kWords) * kThreads + tid], here, k, k);
    here += kStep;
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int32_t b = at0 + kHeld * kStep, k = kHeld; kAnyLength && b < words.bytes; b += kRestWords * kStep, k += kRestWords) {
    Word4 y[kRestWords];
#pragma unroll
    for (int j = 0; j < kRestWords; ++j) y[j] = words.load_cached(b + j * kStep);
#pragma unroll
    for (int j = 0; j < kRestWords; ++j) gradient(y[j], b + j * kStep, k + j, kRestBit);
  }
  if (tid < cut.edge && !huge) {
    const int32_t v = cut.edge_column(tid);
    float g = coef * exp2_fast(fmaf(edge[0], scale, -fast.top));
    if constexpr (kKind == kLossPolicy) {
      if (label_on_edge) g = -amount * joined.not_q;
    } else {
      if ((hit >> kEdgeBit) & 1u) g = take_edge_target<T, kThreads>(s_list, cut, amount, g);
    }
    out[v] = Elem<T>::round(g);
  }
  if (huge && state == kRowLive) {
    for (int32_t v = tid; v < r.vocab; v += kThreads) {
      float g = coef * exp2_fast((Elem<T>::load(in + v) - base) * scale);
      if (kKind == kLossPolicy && v == label) g = -amount * joined.not_q;
      out[v] = Elem<T>::round(g);
    }
    if constexpr (kKind == kLossDistill) {
      __syncthreads();  // a target's element is stored again, after the first time
      put_targets<T, kThreads>(s_list, out, coef, base, scale, amount);
    }
  }
  if (kKind == kLossDistill && state != kRowLive) {
    __syncthreads();  // over what was just stored
    fill_row(state == kRowBad);
  }
}

// The same for a gradient whose rows lie at another place within 16 bytes than
// the logits' rows: the row is read twice and the gradient stored element by
// element.  Right wherever a caller puts the gradient, and far from the memory's
// rate: 8192 x 50257 bf16 1488 us against 298 for rows that lie alike, 4096 x
// 100003 fp32 1756 against 604.  The Python calls place a gradient of their own
// alike.
template <typename T, LossKind kKind>
__global__ __launch_bounds__(256) void row_loss_apart_kernel(LogitRows r, LossArgs a) {
  constexpr int kThreads = 256;
  struct NoList {
    int32_t state;
  };
  using List = typename std::conditional<kKind == kLossDistill, TargetList<kThreads>, NoList>::type;
  __shared__ float2 s_red[kThreads / 64];
  __shared__ List s_list;
  const int32_t tid = threadIdx.x;
  if (a.scan && blockIdx.x == gridDim.x - 1) return scan_status<kThreads>(a, r.rows, r.vocab);
  for (int64_t row = blockIdx.x; row < r.rows; row += gridDim.x - a.scan) {
    const T* in = static_cast<const T*>(r.in) + row * r.in_stride;
    T* out = static_cast<T*>(r.out) + row * r.out_stride;
    const bool live = !a.mask || a.mask[row] != 0;
    int32_t state = live ? kRowLive : kRowEmpty;
    int64_t label = 0;
    if constexpr (kKind == kLossPolicy) {
      label = a.labels[row];
      if (live && (label < 0 || label >= r.vocab)) state = kRowBad;
    } else {
      if (live && tid < 64) {
        TeacherRaw raw;
        float z[kMine];
        const RowCut<T> cut(in, r.vocab);
        read_teacher(raw, a, row);
        list_targets<T, kThreads, kRestBit>(s_list, raw, z, a, row, in, nullptr, cut, r.vocab, 0, cut.words, 0, true);
        store_logits(s_list.z, z, a.k);
      }
      __syncthreads();
      if (live) state = __builtin_amdgcn_readfirstlane(s_list.state);
    }
    if (state != kRowLive) {
      fill_words<T>(out, r.vocab, state == kRowBad ? Elem<T>::kNanWord : 0u, 0, INT32_MAX, true, kThreads);
      if (tid == 0) {
        const float v = state == kRowBad ? __builtin_nanf("") : 0.0f;
        a.loss[row] = v;
        if (kKind == kLossPolicy) a.logp[row] = v;
        if (state == kRowBad && a.status && !a.scan) *a.status = THD_ERR_LABEL;
      }
    } else {
      const float scale = kKind == kLossDistill ? a.inv_temperature * kLog2e : kLog2e;
      Stat st = row_stat<T, kThreads>(in, r.vocab, kKind == kLossPolicy ? label : -1, scale, s_red);
      float amount;
      LabelJoin joined;
      if constexpr (kKind == kLossPolicy) {
        joined = join_label(st, Elem<T>::load(in + label), scale);
        const PolicyRow p = policy_row(a, policy_values(a, row), joined.logp);
        if (tid == 0) {
          a.loss[row] = p.loss;
          a.logp[row] = joined.logp;
        }
        amount = -p.dlogp;
      } else {
        const float w = a.weights ? a.weights[row] : 1.0f;
        if (tid < 64) {
          const float loss = distill_loss(s_list, a, w, [&](float z) { return (z - st.m) * scale; }, logf(st.s));
          if (tid == 0) a.loss[row] = loss;
        }
        amount = a.temperature * w;
      }
      const float coef = amount * reciprocal(st.s);
      const float base = base_of(st.m);
      for (int32_t v = tid; v < r.vocab; v += kThreads) {
        float g = coef * exp2_fast((Elem<T>::load(in + v) - base) * scale);
        if (kKind == kLossPolicy && v == label) g = -amount * joined.not_q;
        out[v] = Elem<T>::round(g);
      }
      if constexpr (kKind == kLossDistill) {
        __syncthreads();  // a target's element is stored again, after the first time
        put_targets<T, kThreads>(s_list, out, coef, base, scale, amount);
      }
    }
    __syncthreads();  // the next row reuses what is shared
  }
}

// Rows per chunk of an XCD's order: about 1 MiB, and at least 16 rows.  Against
// plain order: 67108 x 8000 bf16 354 us and 384, 16777 x 32000 365 and 377,
// 4096 x 131072 382 and 396; chunks of 4 rows are slower there (421 us).
inline int32_t row_chunk_shift(const LogitRows& r) {
  const int64_t bytes = static_cast<int64_t>(r.vocab) * (r.dtype == THD_FP32 ? 4 : 2);
  int32_t shift = 4;
  while (shift < 8 && (bytes << (shift + 1)) <= (1 << 20)) ++shift;
  return shift;
}

template <typename T, int kThreads, int kWords, int kLds, LossKind kKind>
hipError_t launch_rows_as(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  constexpr int32_t kSlice = static_cast<int32_t>((1LL << 31) / kThreads);  // a grid counts 2^32 threads
  for (int64_t row0 = 0; row0 < r.rows; row0 += kSlice) {
    const int32_t n = static_cast<int32_t>(r.rows - row0 < kSlice ? r.rows - row0 : kSlice);
    hipLaunchKernelGGL((row_loss_kernel<T, kThreads, kWords, kLds, kKind>), dim3(n + a.scan), dim3(kThreads),
                       kLds * kThreads * sizeof(Word4), stream, r, a, static_cast<int32_t>(row0), row_chunk_shift(r));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, LossKind kKind>
hipError_t launch_rows(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  const int64_t lag = reinterpret_cast<intptr_t>(r.out) - reinterpret_cast<intptr_t>(r.in);
  const int64_t pitch = r.rows > 1 ? r.out_stride * static_cast<int64_t>(sizeof(T)) : 0;
  const int64_t drift = r.rows > 1 ? pitch - r.in_stride * static_cast<int64_t>(sizeof(T)) : 0;
  if (lag % 16 != 0 || drift % 16 != 0) {
    const int32_t resident = compute_units() * 8;
    hipLaunchKernelGGL((row_loss_apart_kernel<T, kKind>), dim3((r.rows < resident ? r.rows : resident) + a.scan),
                       dim3(256), 0, stream, r, a);
    return hipGetLastError();
  }
  // rows that do not all start on a 128-byte line are shifted by up to 7 words
  const bool lines = reinterpret_cast<uintptr_t>(r.out) % 128 == 0 && pitch % 128 == 0;
  const int32_t words = r.vocab / Elem<T>::kPer + (lines ? 0 : 7);
  // 4 words a thread while 1024 threads hold the row (65536 x 4096 bf16 164 us,
  // with 8 words 177; 8388 x 32000 176 us with 4, 184 with 8 on half the
  // threads); then as many as it takes, two workgroups to a compute unit as long
  // as they fit (LDS from 8192 words on), then one.  Rows a few past a whole number
  // of rounds over the compute units pay for the last one: 131072 bf16 columns 39.5
  // us for 256 rows, 51.7 for 260, 64.9 for 512; 200003 columns 53, 71 and 88.
  if (words <= 64 * 4) return launch_rows_as<T, 64, 4, 0, kKind>(r, a, stream);
  if (words <= 128 * 4) return launch_rows_as<T, 128, 4, 0, kKind>(r, a, stream);
  if (words <= 256 * 4) return launch_rows_as<T, 256, 4, 0, kKind>(r, a, stream);
  if (words <= 512 * 4) return launch_rows_as<T, 512, 4, 0, kKind>(r, a, stream);
  if (words <= 1024 * 4) return launch_rows_as<T, 1024, 4, 0, kKind>(r, a, stream);
  if (words <= 1024 * 8) return launch_rows_as<T, 1024, 8, 0, kKind>(r, a, stream);
  if (words <= 1024 * 12) return launch_rows_as<T, 1024, 8, 4, kKind>(r, a, stream);
  if (words <= 1024 * 16) return launch_rows_as<T, 1024, 16, 0, kKind>(r, a, stream);
  return launch_rows_as<T, 1024, 18, 8, kKind>(r, a, stream);
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
