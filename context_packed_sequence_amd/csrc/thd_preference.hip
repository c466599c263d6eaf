// Preference loss over pairs of documents of a packed stream, and its gradient
// with respect to the tokens' log-probabilities.
//
//   S_d  = sum over the document's unmasked tokens of (logp - ref)
//   D    = beta (S_chosen - S_rejected)
//   L    = scale ((1 - e) ln(1 + exp(-D)) + e ln(1 + exp(D)))
//   dL/dlogp_t = +scale beta (e sigma(D) - (1 - e) sigma(-D)) on the chosen
//                document's tokens, its negative on the rejected one's.
//
// Two launches.  The stream is cut into tiles of 512 tokens, one wave each, so
// that one long document and many short ones spread alike.  Tile i and document
// d that overlap leave their partial sum at entry i + d of the workspace: along
// the stream either the tile or the document moves on, so no two overlaps share
// an entry, and a document's partial sums lie side by side.  The second launch
// adds them in that order (the result does not depend on timing), in 64 bits: a
// document's sum is a long sum of small differences.  It is bound by latency,
// not by its 13 bytes a token: every read of a tile is issued at once, and
// boundaries are searched 64 at a time.
#include "thd_loss_device.h"

namespace thdcp {
namespace {

constexpr int kTile = 512;
constexpr int kEach = kTile / 64;  // tokens per lane

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Slot that holds token t: the last one whose start is at or before it.  Each
// round probes 64 boundaries.  Some slot is returned for any list, so that a
// list that is not sorted stays in bounds.
__device__ __forceinline__ int32_t slot_of(const int32_t* cu, int32_t n_slots, int32_t t) {
  const int lane = threadIdx.x;
  int32_t lo = 0, n = n_slots;
  while (n > 1) {
    const int32_t step = (n + 63) / 64;
    const int32_t i = lane * step;
    const bool below = i < n && cu[lo + i] <= t;
    const int32_t last = max(__popcll(__ballot(below)) - 1, 0);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// Calls f(slot, begin, end) for every non-empty piece of a document inside
// tokens [t0, t1), in order; the arguments are the same in every lane.
template <typename F>
__device__ __forceinline__ void each_piece(const int32_t* cu, int32_t n_slots, int32_t t0, int32_t t1, F f) {
  const int lane = threadIdx.x;
  int32_t d0 = slot_of(cu, n_slots, t0);
  while (d0 < n_slots) {
    const int32_t mine = cu[min(d0 + lane, n_slots)];
    for (int i = 0; i < 63; ++i) {
      const int32_t d = d0 + i;
      const int32_t a = __shfl(mine, i), b = __shfl(mine, i + 1);
      if (d >= n_slots || a >= t1) return;
      const int32_t begin = max(a, t0), end = min(b, t1);
      if (begin < end) f(d, begin, end);
    }
    d0 += 63;
  }
}

__global__ __launch_bounds__(64) void preference_sums_kernel(PreferenceArgs a, int32_t tiles) {
  const int lane = threadIdx.x;
  if (static_cast<int32_t>(blockIdx.x) == tiles) {
    // the boundary list and the pairs, checked once
    int sev = 0;
    bool bad_pair = false;
    if (lane == 0) {
      if (a.cu[0] != 0) sev = kSevStart;
      if (a.cu[a.n_slots] != a.total) sev = max(sev, kSevTotal);
    }
    for (int32_t i = lane; i < a.n_slots; i += 64)
      if (a.cu[i + 1] < a.cu[i]) sev = max(sev, kSevMonotone);
    for (int32_t i = lane; i < a.n_pairs; i += 64) {
      const int32_t c = a.pairs[2 * i], r = a.pairs[2 * i + 1];
      const bool unused = c == -1 && r == -1;
      if (!unused && (c < 0 || c >= a.n_slots || r < 0 || r >= a.n_slots)) bad_pair = true;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sev = max(sev, __shfl_xor(sev, d));
    bad_pair = __any(bad_pair);
    if (lane == 0) {
      const int32_t code = severity_to_code(sev);
      *a.ws_code = code;
      if (a.status) *a.status = code != THD_OK ? code : (bad_pair ? THD_ERR_PAIR : THD_OK);
    }
    return;
  }
  const int32_t tile = blockIdx.x;
  const int32_t t0 = tile * kTile;
  const int32_t t1 = static_cast<int32_t>(min(static_cast<int64_t>(t0) + kTile, static_cast<int64_t>(a.total)));
  float lp[kEach], rp[kEach];
  uint8_t on[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int64_t t = static_cast<int64_t>(t0) + j * 64 + lane;
    lp[j] = rp[j] = 0.0f;
    on[j] = 0;
    if (t < t1) {
      on[j] = a.mask ? a.mask[t] : 1;
      lp[j] = a.logp[t];
      if (a.ref_logp) rp[j] = a.ref_logp[t];
    }
  }
  each_piece(a.cu, a.n_slots, t0, t1, [&](int32_t d, int32_t begin, int32_t end) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t t = static_cast<int64_t>(t0) + j * 64 + lane;
      if (on[j] && t >= begin && t < end) sum += static_cast<double>(lp[j]) - static_cast<double>(rp[j]);
    }
    sum = wave_sum(sum);
    if (lane == 0) a.ws_sums[static_cast<int64_t>(tile) + d] = sum;
  });
}

// Sum of a document's partial sums, on the whole wave.
__device__ __forceinline__ double document_sum(const PreferenceArgs& a, int32_t d) {
  const int32_t begin = a.cu[d], end = a.cu[d + 1];
  double sum = 0.0;
  if (begin < end) {
    const int32_t first = begin / kTile, last = (end - 1) / kTile;
    for (int32_t i = first + static_cast<int32_t>(threadIdx.x); i <= last; i += 64)
      sum += a.ws_sums[static_cast<int64_t>(i) + d];
  }
  return wave_sum(sum);
}

__device__ __forceinline__ double softplus(double x) { return log1p(exp(-fabs(x))) + (x > 0.0 ? x : 0.0); }

__global__ __launch_bounds__(64) void preference_loss_kernel(PreferenceArgs a, int32_t tiles) {
  const int lane = threadIdx.x;
  const int32_t code = *a.ws_code;
  if (code != THD_OK) return;
  if (static_cast<int32_t>(blockIdx.x) >= tiles) {
    const int32_t i = blockIdx.x - tiles;
    const int32_t c = a.pairs[2 * i], r = a.pairs[2 * i + 1];
    double loss = 0.0, won = 0.0, lost = 0.0;
    if (c >= 0 && c < a.n_slots && r >= 0 && r < a.n_slots) {
      won = a.beta * document_sum(a, c);
      lost = a.beta * document_sum(a, r);
      const double z = won - lost, e = a.smoothing;
      loss = 0.0;
      if (e < 1.0) loss += (1.0 - e) * softplus(-z);
      if (e > 0.0) loss += e * softplus(z);
      loss *= a.scale;
    } else if (c != -1 || r != -1) {
      loss = won = lost = __builtin_nan("");
    }
    if (lane == 0) {
      a.loss[i] = static_cast<float>(loss);
      a.rewards[2 * i] = static_cast<float>(won);
      a.rewards[2 * i + 1] = static_cast<float>(lost);
    }
    return;
  }
  const int32_t tile = blockIdx.x;
  const int32_t t0 = tile * kTile;
  const int32_t t1 = static_cast<int32_t>(min(static_cast<int64_t>(t0) + kTile, static_cast<int64_t>(a.total)));
  uint8_t on[kEach];
  float g[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int64_t t = static_cast<int64_t>(t0) + j * 64 + lane;
    g[j] = 0.0f;
    on[j] = t < t1 ? (a.mask ? a.mask[t] : 1) : 0;
  }
  each_piece(a.cu, a.n_slots, t0, t1, [&](int32_t d, int32_t begin, int32_t end) {
    // every pair that names the document, in order
    double coef = 0.0;
    for (int32_t p0 = 0; p0 < a.n_pairs; p0 += 64) {
      int32_t c = -1, r = -1;
      if (p0 + lane < a.n_pairs) {
        c = a.pairs[2 * (p0 + lane)];
        r = a.pairs[2 * (p0 + lane) + 1];
      }
      const bool valid = c >= 0 && c < a.n_slots && r >= 0 && r < a.n_slots;
      uint64_t named = __ballot(valid && c != r && (c == d || r == d));
      while (named) {
        const int l = __builtin_ctzll(named);
        named &= named - 1;
        const int32_t cc = __shfl(c, l), rr = __shfl(r, l);
        const double z = a.beta * document_sum(a, cc) -
                         a.beta * document_sum(a, rr);
        const double slope = a.smoothing - 1.0 / (1.0 + exp(z));
        coef += cc == d ? slope : -slope;
      }
    }
    const float v = static_cast<float>(coef * a.beta * a.scale);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int64_t t = static_cast<int64_t>(t0) + j * 64 + lane;
      if (t >= begin && t < end) g[j] = v;
    }
  });
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int64_t t = static_cast<int64_t>(t0) + j * 64 + lane;
    if (t < t1) a.dlogp[t] = on[j] ? g[j] : 0.0f;
  }
}

}  // namespace

int32_t preference_tiles(int32_t total) { return static_cast<int32_t>((static_cast<int64_t>(total) + kTile - 1) / kTile); }

hipError_t launch_preference(const PreferenceArgs& a, hipStream_t stream) {
  const int32_t tiles = preference_tiles(a.total);
  hipLaunchKernelGGL(preference_sums_kernel, dim3(tiles + 1), dim3(64), 0, stream, a, tiles);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || tiles + a.n_pairs == 0) return e;
  hipLaunchKernelGGL(preference_loss_kernel, dim3(tiles + a.n_pairs), dim3(64), 0, stream, a, tiles);
  return hipGetLastError();
}

}  // namespace thdcp
