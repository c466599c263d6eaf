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
// boundaries are searched 64 at a time (131072 tokens in 222 documents 6 and 8 us,
// 1048576 in 6 documents 5 and 8).
//
// The second launch forms each document's sum wherever it is wanted: once per
// tile and pair.  That saves a launch for a few tiles a document and grows with
// the square of a document's length times its pairs (two documents of 4M tokens
// together 64 us a call, of 16M 550 us); and every piece of a document within a
// tile looks through all pairs (65536 pairs over 131072 documents of 8 tokens
// 14.7 ms a call, 2048 over 4096 of 256 tokens 50 us).
#include "thd_loss_device.h"

namespace thdcp {
namespace {

constexpr int kTile = 512;
constexpr int kEach = kTile / 64;  // tokens per lane

// Sums of a wave's two halves of 32 lanes, each in every lane of its half:
// DPP moves within 16 lanes, then one exchange of the two rows of each half.
__device__ __forceinline__ double move_lanes(double x, int step) {
  const int64_t bits = __builtin_bit_cast(int64_t, x);
  switch (step) {  // 0x111, ...: row_shr by 1, 2, 4, 8; lanes without a source take 0
    case 1: return __builtin_bit_cast(double, dpp_move<0x111, 0xf>(bits, int64_t{0}));
    case 2: return __builtin_bit_cast(double, dpp_move<0x112, 0xf>(bits, int64_t{0}));
    case 4: return __builtin_bit_cast(double, dpp_move<0x114, 0xf>(bits, int64_t{0}));
    default: return __builtin_bit_cast(double, dpp_move<0x118, 0xf>(bits, int64_t{0}));
  }
}
__device__ __forceinline__ double lane_of(double x, int lane) {
  const int64_t bits = __builtin_bit_cast(int64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int32_t>(bits), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int32_t>(bits >> 32), lane);
  return __builtin_bit_cast(double, static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo));
}
struct HalfSums {
  double low, high;  // of lanes 0-31 and 32-63
};
__device__ __forceinline__ HalfSums half_sums(double v) {
  v += move_lanes(v, 1);
  v += move_lanes(v, 2);
  v += move_lanes(v, 4);
  v += move_lanes(v, 8);
  return HalfSums{lane_of(v, 15) + lane_of(v, 31), lane_of(v, 47) + lane_of(v, 63)};
}
__device__ __forceinline__ double wave_sum(double v) {
  const HalfSums h = half_sums(v);
  return h.low + h.high;
}

// Boundaries and pairs that fit are read into LDS with the tile's tokens, in one
// round trip; of longer lists each search round and each piece costs one.
constexpr int kLdsSlots = 1023;
constexpr int kLdsPairs = 512;

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

// A list on its way to LDS, by one wave: its first 64 * N words are issued with
// whatever else the tile reads, the rest follows.
template <int N>
struct Staged {
  int32_t v[N];
  __device__ __forceinline__ void issue(const int32_t* from, int32_t n) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t i = 64 * j + static_cast<int32_t>(threadIdx.x);
      v[j] = i < n ? from[i] : 0;
    }
  }
  __device__ __forceinline__ void finish(int32_t* to, const int32_t* from, int32_t n) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t i = 64 * j + static_cast<int32_t>(threadIdx.x);
      if (i < n) to[i] = v[j];
    }
    for (int32_t i = 64 * N + static_cast<int32_t>(threadIdx.x); i < n; i += 64) to[i] = from[i];
  }
};

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
    constexpr int kAhead = 4;  // entries in flight
    for (int32_t i0 = lane; i0 < max(a.n_slots, a.n_pairs); i0 += 64 * kAhead) {
      int32_t from[kAhead], to[kAhead], c[kAhead], r[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int32_t i = i0 + 64 * j;
        from[j] = to[j] = 0;
        c[j] = r[j] = -1;
        if (i < a.n_slots) {
          from[j] = a.cu[i];
          to[j] = a.cu[i + 1];
        }
        if (i < a.n_pairs) {
          c[j] = a.pairs[2 * i];
          r[j] = a.pairs[2 * i + 1];
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (to[j] < from[j]) sev = max(sev, kSevMonotone);
        const bool unused = c[j] == -1 && r[j] == -1;
        if (!unused && (c[j] < 0 || c[j] >= a.n_slots || r[j] < 0 || r[j] >= a.n_slots)) bad_pair = true;
      }
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
  __shared__ int32_t s_cu[kLdsSlots + 1];
  const int32_t tile = blockIdx.x;
  const int32_t t0 = tile * kTile;
  const int32_t t1 = static_cast<int32_t>(min(static_cast<int64_t>(t0) + kTile, static_cast<int64_t>(a.total)));
  const bool in_lds = a.n_slots <= kLdsSlots;
  Staged<4> bounds;
  if (in_lds) bounds.issue(a.cu, a.n_slots + 1);
  float lp[kEach], rp[kEach];
  uint8_t on[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int32_t t = min(t0 + j * 64 + lane, t1 - 1);  // past the tile: a token of it again, in no piece
    lp[j] = a.logp[t];
    rp[j] = a.ref_logp ? a.ref_logp[t] : 0.0f;
    on[j] = a.mask ? a.mask[t] : 1;
  }
  const int32_t* cu = a.cu;
  if (in_lds) {
    bounds.finish(s_cu, a.cu, a.n_slots + 1);
    __syncthreads();
    cu = s_cu;
  }
  each_piece(cu, a.n_slots, t0, t1, [&](int32_t d, int32_t begin, int32_t end) {
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

// Sums of two documents' partial sums, one on each half of the wave.
__device__ __forceinline__ HalfSums document_sums(const PreferenceArgs& a, const int32_t* cu, int32_t c, int32_t r) {
  const int half = threadIdx.x >> 5;
  const int32_t d = half ? r : c;
  const int32_t begin = cu[d], end = cu[d + 1];
  double sum = 0.0;
  if (begin < end) {
    constexpr int kAhead = 8;  // partial sums in flight
    const int32_t last = (end - 1) / kTile;
    for (int32_t i0 = begin / kTile + static_cast<int32_t>(threadIdx.x & 31); i0 <= last; i0 += 32 * kAhead) {
      double v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int32_t i = i0 + 32 * j;
        v[j] = a.ws_sums[static_cast<int64_t>(min(i, last)) + d];
        if (i > last) v[j] = 0.0;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) sum += v[j];
    }
  }
  return half_sums(sum);
}

__device__ __forceinline__ double softplus(double x) { return log1p(exp(-fabs(x))) + (x > 0.0 ? x : 0.0); }

__global__ __launch_bounds__(64) void preference_loss_kernel(PreferenceArgs a, int32_t tiles) {
  __shared__ int32_t s_cu[kLdsSlots + 1];
  __shared__ int32_t s_pairs[2 * kLdsPairs];
  const int lane = threadIdx.x;
  const int32_t code = *a.ws_code;
  if (static_cast<int32_t>(blockIdx.x) >= tiles) {
    if (code != THD_OK) return;
    const int32_t i = blockIdx.x - tiles;
    const int32_t c = a.pairs[2 * i], r = a.pairs[2 * i + 1];
    double loss = 0.0, won = 0.0, lost = 0.0;
    if (c >= 0 && c < a.n_slots && r >= 0 && r < a.n_slots) {
      const HalfSums sums = document_sums(a, a.cu, c, r);
      won = a.beta * sums.low;
      lost = a.beta * sums.high;
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
  const bool slots_in_lds = a.n_slots <= kLdsSlots, pairs_in_lds = a.n_pairs <= kLdsPairs;
  Staged<4> bounds, some_pairs;
  if (slots_in_lds) bounds.issue(a.cu, a.n_slots + 1);
  if (pairs_in_lds) some_pairs.issue(a.pairs, 2 * a.n_pairs);
  uint8_t on[kEach];
  float g[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    g[j] = 0.0f;
    on[j] = a.mask ? a.mask[min(t0 + j * 64 + lane, t1 - 1)] : 1;
  }
  if (code != THD_OK) return;
  const int32_t* cu = a.cu;
  const int32_t* pairs = a.pairs;
  if (slots_in_lds) {
    bounds.finish(s_cu, a.cu, a.n_slots + 1);
    cu = s_cu;
  }
  if (pairs_in_lds) {
    some_pairs.finish(s_pairs, a.pairs, 2 * a.n_pairs);
    pairs = s_pairs;
  }
  __syncthreads();
  each_piece(cu, a.n_slots, t0, t1, [&](int32_t d, int32_t begin, int32_t end) {
    // every pair that names the document, in order
    double coef = 0.0;
    for (int32_t p0 = 0; p0 < a.n_pairs; p0 += 64) {
      int32_t c = -1, r = -1;
      if (p0 + lane < a.n_pairs) {
        c = pairs[2 * (p0 + lane)];
        r = pairs[2 * (p0 + lane) + 1];
      }
      const bool valid = c >= 0 && c < a.n_slots && r >= 0 && r < a.n_slots;
      uint64_t named = __ballot(valid && c != r && (c == d || r == d));
      while (named) {
        const int l = __builtin_ctzll(named);
        named &= named - 1;
        const int32_t cc = __shfl(c, l), rr = __shfl(r, l);
        const HalfSums sums = document_sums(a, cu, cc, rr);
        const double z = a.beta * sums.low - a.beta * sums.high;
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
