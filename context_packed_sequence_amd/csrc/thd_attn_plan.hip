// Tiles of the attention kernels: which rows of which document each workgroup
// takes, laid out on the device from the boundaries, so that the host need not
// know them.
//
// One workgroup checks the boundaries (in the route build's order of rules),
// counts each slot's tiles, and writes every tile's description, the ones with
// most keys to look at first: the last workgroups to run are then the lightest.
// A tile's weight is held to 8 steps per power of two, and tiles of equal weight
// go where an LDS counter says, so their order may differ from run to run; a
// tile's result does not depend on its place.  Latency, of loads and barriers: 4 us
// for one document of 8192 tokens, 8 for 16384 tokens of short documents, 9 for 32768
// (with the boundaries in memory 12 and more).
#include "thd_attn_device.h"

namespace thdcp {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 256;
constexpr int kSlotsInLds = 4096;

__device__ __forceinline__ int32_t tiles_of(int32_t n, int32_t per) { return (n + per - 1) / per; }

// Buckets in order of falling weight; weight 0 last.
__device__ __forceinline__ int32_t bucket_of(int32_t weight) {
  if (weight <= 0) return kBuckets - 1;
  const uint32_t bits = __builtin_bit_cast(uint32_t, static_cast<float>(weight));
  return kBuckets - 2 - static_cast<int32_t>((bits >> 20) - 1016u);  // weights up to 2^31: 0..247
}

// The boundaries, and the tiles of all slots before each: in LDS where they fit.
struct Bounds {
  const int32_t *padded, *real;
  int32_t* first;
};

struct Slot {
  int32_t start, padded, real, first, chunk;
  __device__ __forceinline__ Slot(const AttnArgs& a, const Bounds& b, int32_t s) {
    start = b.padded[s];
    padded = b.padded[s + 1] - start;
    real = b.real[s + 1] - b.real[s];
    first = start / a.cp;
    chunk = a.cp == 1 ? padded : padded / (2 * a.cp);
  }
};

__device__ __forceinline__ int32_t query_tiles_of(const AttnArgs& a, const Slot& s) {
  return (a.cp == 1 ? 1 : 2) * tiles_of(s.chunk, kAttnRows / a.tile_heads);
}

// Tile t of a slot's query tiles, and its weight: the keys it looks at.
__device__ QueryTile query_tile(const AttnArgs& a, const Slot& s, int32_t t, int32_t* weight) {
  QueryTile q{};
  const int32_t tile_rows = kAttnRows / a.tile_heads;
  const int32_t per = tiles_of(s.chunk, tile_rows);
  const int32_t second = t >= per ? 1 : 0;
  const int32_t at = (t - second * per) * tile_rows;
  q.row = s.first + second * s.chunk + at;
  q.rows = min(tile_rows, s.chunk - at);
  q.pos = at + (a.cp == 1 ? 0 : second ? (2 * a.cp - 1 - a.rank) * s.chunk : a.rank * s.chunk);
  q.valid = max(0, min(q.rows, s.real - q.pos));
  q.doc = s.start;
  q.real = s.real;
  *weight = 0;
  if (q.valid > 0) {
    const Seen first(a, q.pos, q.real), last(a, q.pos + q.valid - 1, q.real);
    *weight = last.low + static_cast<int32_t>(last.span) - first.low;
  }
  return q;
}

// Tile t of a slot's key tiles, and its weight: the query rows that may see it.
__device__ KeyTile key_tile(const AttnArgs& a, const Slot& s, int32_t t, int32_t* weight) {
  KeyTile k{};
  k.key = t * kAttnKeys;
  k.keys = min(kAttnKeys, s.padded - k.key);
  k.valid = max(0, min(k.keys, s.real - k.key));
  k.doc = s.start;
  k.real = s.real;
  k.first = s.first;
  k.chunk = s.chunk;
  int32_t rows = 0;
  if (k.valid > 0) {
    const int32_t low = a.causal ? k.key : a.window ? max(0, k.key - a.window + 1) : 0;
    const int32_t high = a.window ? window_end(a, k.key + k.valid, s.real) : s.real;
    for (int second = 0; second < (a.cp == 1 ? 1 : 2); ++second) {
      const int32_t pos = a.cp == 1 ? 0 : second ? (2 * a.cp - 1 - a.rank) * s.chunk : a.rank * s.chunk;
      rows += max(0, min(high, pos + s.chunk) - max(low, pos));
    }
  }
  *weight = rows;
  return k;
}

// Exclusive prefix of count(slot) over all slots, in memory; returns the total.
template <typename Count>
__device__ int32_t slot_prefix(int32_t n_slots, int32_t* first, int32_t* s_wave, Count count) {
  int32_t carry = 0;
  for (int32_t base = 0; base < n_slots; base += kPlanThreads) {
    const int32_t s = base + threadIdx.x;
    const int32_t n = s < n_slots ? count(s) : 0;
    int32_t total;
    const int32_t before = block_exclusive_scan<kPlanThreads>(n, s_wave, &total);
    if (s < n_slots) first[s] = carry + before;
    carry += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) first[n_slots] = carry;
  __syncthreads();
  return carry;
}

__device__ __forceinline__ int32_t slot_of(const int32_t* first, int32_t n_slots, int32_t t) {
  int32_t low = 0, high = n_slots;  // first[low] <= t < first[high]
  while (high - low > 1) {
    const int32_t mid = (low + high) >> 1;
    if (first[mid] <= t) low = mid;
    else high = mid;
  }
  return low;
}

// Places n tiles by falling weight: make(t, &weight) describes tile t.  Places up to
// `most` hold no tile.
template <typename Tile, typename Make>
__device__ void place_tiles(int32_t n, int32_t most, Tile* out, int32_t* s_bucket, Make make) {
  for (int32_t t = n + threadIdx.x; t < most; t += kPlanThreads) out[t] = Tile{};
  for (int32_t b = threadIdx.x; b < kBuckets; b += kPlanThreads) s_bucket[b] = 0;
  __syncthreads();
  for (int32_t t = threadIdx.x; t < n; t += kPlanThreads) {
    int32_t weight;
    make(t, &weight);
    atomicAdd(&s_bucket[bucket_of(weight)], 1);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    int32_t c[kBuckets / 64], sum = 0;
#pragma unroll
    for (int i = 0; i < kBuckets / 64; ++i) {
      c[i] = s_bucket[threadIdx.x * (kBuckets / 64) + i];
      sum += c[i];
    }
    int32_t before = wave_inclusive_scan(sum, 0, ScanAdd{}) - sum;
#pragma unroll
    for (int i = 0; i < kBuckets / 64; ++i) {
      s_bucket[threadIdx.x * (kBuckets / 64) + i] = before;
      before += c[i];
    }
  }
  __syncthreads();
  for (int32_t t = threadIdx.x; t < n; t += kPlanThreads) {
    int32_t weight;
    const Tile tile = make(t, &weight);
    out[atomicAdd(&s_bucket[bucket_of(weight)], 1)] = tile;
  }
  __syncthreads();
}

template <bool kInLds>
__global__ __launch_bounds__(kPlanThreads) void attn_plan_kernel(AttnArgs a) {
  __shared__ int32_t s_wave[kPlanThreads / 64 + 1];
  __shared__ int32_t s_bucket[kBuckets];
  __shared__ int32_t s_severity;
  __shared__ int32_t s_bounds[kInLds ? 3 : 1][kInLds ? kSlotsInLds + 1 : 1];
  const AttnPlan& p = a.plan;
  Bounds bounds{a.cu_padded, a.cu_real ? a.cu_real : a.cu_padded, p.slot_first};
  if constexpr (kInLds) {
    for (int32_t s = threadIdx.x; s <= a.n_slots; s += kPlanThreads) {
      const int32_t padded = a.cu_padded[s], real = bounds.real[s];
      s_bounds[0][s] = padded;
      s_bounds[1][s] = real;
    }
    bounds = Bounds{s_bounds[0], s_bounds[1], s_bounds[2]};
  }
  if (threadIdx.x == 0) s_severity = 0;
  __syncthreads();
  int32_t severity = 0;
  if (threadIdx.x == 0) {
    if (bounds.padded[0] != 0 || bounds.real[0] != 0) severity = kSevStart;
    else if (bounds.padded[a.n_slots] != a.total) severity = kSevTotal;
  }
  for (int32_t s = threadIdx.x; s < a.n_slots; s += kPlanThreads) {
    const int64_t padded = static_cast<int64_t>(bounds.padded[s + 1]) - bounds.padded[s];
    const int64_t real = static_cast<int64_t>(bounds.real[s + 1]) - bounds.real[s];
    if (padded < 0 || real < 0) severity = max(severity, kSevMonotone);
    else if (a.cp > 1 && padded % (2 * a.cp) != 0) severity = max(severity, kSevDivisible);
    else if (real > padded) severity = max(severity, kSevRealGtPadded);
  }
  if (severity) atomicMax(&s_severity, severity);
  __syncthreads();
  const int32_t code = severity_to_code(s_severity);
  if (threadIdx.x == 0) {
    if (a.status) *a.status = code;
    p.header[kAttnCode] = code;
    p.header[kAttnMaxGrad] = 0;
    p.header[kAttnMaxValue] = 0;
  }
  if (code != THD_OK) {  // no tiles: nothing is written
    for (int32_t t = threadIdx.x; t < p.max_query_tiles; t += kPlanThreads) p.query_tiles[t] = QueryTile{};
    for (int32_t t = threadIdx.x; t < p.max_key_tiles; t += kPlanThreads) p.key_tiles[t] = KeyTile{};
    return;
  }
  const int32_t nq = slot_prefix(a.n_slots, bounds.first, s_wave,
                                 [&](int32_t s) { return query_tiles_of(a, Slot(a, bounds, s)); });
  place_tiles(nq, p.max_query_tiles, p.query_tiles, s_bucket, [&](int32_t t, int32_t* weight) {
    const int32_t s = slot_of(bounds.first, a.n_slots, t);
    return query_tile(a, Slot(a, bounds, s), t - bounds.first[s], weight);
  });
  if (p.key_tiles) {
    const int32_t nk = slot_prefix(a.n_slots, bounds.first, s_wave,
                                   [&](int32_t s) { return tiles_of(Slot(a, bounds, s).padded, kAttnKeys); });
    place_tiles(nk, p.max_key_tiles, p.key_tiles, s_bucket, [&](int32_t t, int32_t* weight) {
      const int32_t s = slot_of(bounds.first, a.n_slots, t);
      return key_tile(a, Slot(a, bounds, s), t - bounds.first[s], weight);
    });
  }
}

}  // namespace

hipError_t launch_attn_plan(const AttnArgs& a, hipStream_t stream) {
  if (a.n_slots <= kSlotsInLds) attn_plan_kernel<true><<<1, kPlanThreads, 0, stream>>>(a);
  else attn_plan_kernel<false><<<1, kPlanThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace thdcp
