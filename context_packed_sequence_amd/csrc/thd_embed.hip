// Embedding lookup on a packed stream, and the gradient of its table.
//
// The lookup is a copy of rows: every thread moves 16-byte words, four in flight.
//
// The gradient of row v of the table is the sum of drows[t] over the rows t that
// hold token v.  Atomic additions would add in an order of their own on each run, so
// the stream's rows are sorted by token first, stably, with digits of up to 9 bits:
// a wave finds a digit's rank among its 64 lanes from ballots, one per bit, and
// the counts of waves, workgroups and digits before it make it a place.  Then units
// of 16 to 128 sorted rows are summed, one thread per 16-byte column of a unit, in
// order: even however often a token occurs (the commonest of a text makes thousands of
// rows).  A token whose rows lie within one unit is stored at once;
// where its run passes a unit's border the sums go to a workspace, and the thread
// of the unit in which the run begins adds them up, in order, in the last launch.
// The rows of tokens that do not occur are cleared beside the sort of a small batch, or
// beside the sums of a large one.
//
// Long rows are bound by memory (32768 rows of 4096 bf16, table of 32000: 155 us, the sums
// 4.7 TB/s at random rows; 4099 of 1001 fp32, table of 100003: 85 us, 400 MB of it zeros),
// short ones by the launches that wait for each other: three up to 8192 rows (3090 of 178
// fp32 26 us), four to eight beyond (20510 of 10 fp16 49 us).
#include "thd_loss_device.h"
#include "thd_params_internal.h"

namespace thdcp {

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int64_t kFewSums = 8192, kMostShort = 2048;
constexpr int kEarlyRows = 4096;  // of the table, at most, that a workgroup beside the sort clears

// 16 bytes at any element's alignment: the hardware takes them as they lie.
struct __attribute__((packed, aligned(2))) LooseWord {
  uint32_t x[4];
};
__device__ __forceinline__ Word4 load_loose(const void* p) {
  const LooseWord w = *static_cast<const LooseWord*>(p);
  return Word4{w.x[0], w.x[1], w.x[2], w.x[3]};
}
__device__ __forceinline__ void store_loose(void* p, Word4 v) {
  *static_cast<LooseWord*>(p) = LooseWord{{v[0], v[1], v[2], v[3]}};
}

// Place of thread i of a workgroup that takes `each` of n x words places from
// `from` on: the row and the word, with one long division a workgroup.
struct FlatPlace {
  int64_t row0;
  int32_t rest;
  FastDiv by;
  __device__ __forceinline__ FlatPlace(int64_t from, int32_t words, FastDiv d) : by(d) {
    row0 = from / words;
    rest = static_cast<int32_t>(from - row0 * words);
  }
  __device__ __forceinline__ void operator()(int32_t i, int32_t words, int64_t* row, int32_t* word) const {
    const int32_t at = rest + i, r = by(at);
    *row = row0 + r;
    *word = at - r * words;
  }
};

// ---- lookup -----------------------------------------------------------------

constexpr int kLookupEach = 4;  // words of a thread

template <typename T>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a, int32_t words, FastDiv by_words) {
  constexpr int kPer = Elem<T>::kPer;
  if (a.scan && blockIdx.x == 0) {  // the workgroup that looks through all ids, the first to start
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    bool bad = false;
    constexpr int kAhead = 8;
    for (int64_t t0 = threadIdx.x; t0 < a.rows; t0 += kAhead * 256) {
      int64_t id[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) id[i] = t0 + i * 256 < a.rows ? a.ids[t0 + i * 256] : 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (t0 + i * 256 < a.rows && (id[i] < 0 || id[i] >= a.vocab)) bad |= !a.mask || a.mask[t0 + i * 256] != 0;
    }
    if (bad) s_bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) *a.status = s_bad ? THD_ERR_TOKEN : THD_OK;
    return;
  }
  const FlatPlace place((static_cast<int64_t>(blockIdx.x) - a.scan) * (256 * kLookupEach), words, by_words);
  int64_t row[kLookupEach], id[kLookupEach];
  int32_t word[kLookupEach];
  bool live[kLookupEach];
#pragma unroll
  for (int i = 0; i < kLookupEach; ++i) {
    place(i * 256 + threadIdx.x, words, &row[i], &word[i]);
    const bool in = row[i] < a.rows;
    live[i] = in && (!a.mask || a.mask[row[i]] != 0);
    id[i] = in ? a.ids[row[i]] : 0;
  }
  Word4 x[kLookupEach];
#pragma unroll
  for (int i = 0; i < kLookupEach; ++i) {
    x[i] = Word4{0, 0, 0, 0};
    if (!live[i]) continue;
    const bool good = id[i] >= 0 && id[i] < a.vocab;
    if (!good) {
      x[i] = Word4{Elem<T>::kNanWord, Elem<T>::kNanWord, Elem<T>::kNanWord, Elem<T>::kNanWord};
      if (!a.scan && a.status) *a.status = THD_ERR_TOKEN;
      continue;
    }
    const T* from = static_cast<const T*>(a.table) + id[i] * a.in_stride + word[i] * kPer;
    if (word[i] * kPer + kPer <= a.width) {
      x[i] = load_loose(from);
    } else {
      float v[kPer] = {};
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (word[i] * kPer + j < a.width) v[j] = Elem<T>::load(from + j);
      x[i] = Elem<T>::pack(v);
    }
  }
#pragma unroll
  for (int i = 0; i < kLookupEach; ++i) {
    if (row[i] >= a.rows) continue;
    float v[kPer];
    Elem<T>::unpack(x[i], v);
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] *= a.scale;
    T* to = static_cast<T*>(a.out) + row[i] * a.out_stride + word[i] * kPer;
    if (word[i] * kPer + kPer <= a.width) {
      store_loose(to, Elem<T>::pack(v));
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (word[i] * kPer + j < a.width) to[j] = Elem<T>::round(v[j]);
    }
  }
}

// ---- rows without a token ---------------------------------------------------

// The gradient's table for those who clear it: bytes are of a row, words its 16-byte
// ones.
struct ZeroRows {
  char* to;
  int64_t stride;
  int32_t bytes, words;
  FastDiv by_words, by_bytes;
  int32_t first, end;  // rows of the table
  int32_t each;        // of them to a workgroup
  bool run;            // rows follow one another without gaps, and are more than caches hold
  __device__ __forceinline__ int32_t row(int32_t block) const { return first + block * each; }
};

// Two bytes of a run of rows without gaps, unless their row's flag is set.
__device__ __forceinline__ void clear_pair(const ZeroRows& z, char* base, int32_t at, const uint8_t* s_taken) {
  if (!s_taken[z.by_bytes(at)]) *reinterpret_cast<uint16_t*>(base + at) = 0;
}

// Clears those of rows r0 .. r0 + n - 1 whose flag is not set.  A large table without gaps
// is cleared as one run, in 16-byte words from a line's start on whose stores pass the
// caches; a word that holds parts of rows with and without a token goes by twos of bytes.
// Other tables go row by row with plain stores, which meet in the caches at rows' ends and
// stay there.  fp32, few rows: 133106 x 1185 as a run 105 us, row by row 127; 100000 x 1024 73
// and 82; but 250000 x 250, which the 256 MB cache in front of memory holds, 50 and 44.
template <int kThreads>
__device__ __forceinline__ void clear_rows(const ZeroRows& z, int32_t r0, int32_t n, const uint8_t* s_taken) {
  if (z.run) {
    char* base = z.to + static_cast<int64_t>(r0) * z.stride;
    const int32_t size = n * z.bytes, lead = min(size, static_cast<int32_t>(-reinterpret_cast<uintptr_t>(base) & 127));
    const int32_t words = (size - lead) / 128 * 8, tail = lead + 16 * words;
    const StreamStore store(base + lead, 16 * words);
    for (int32_t w = threadIdx.x; w < words; w += kThreads) {
      const int32_t at = lead + 16 * w, first = z.by_bytes(at), last = z.by_bytes(at + 15);
      bool any = s_taken[first] != 0, all = any;
      for (int32_t r = first + 1; r <= last; ++r) {
        const bool taken = s_taken[r] != 0;
        any |= taken;
        all &= taken;
      }
      if (!any) {
        store(w, StoreW4{0, 0, 0, 0});
      } else if (!all) {
        for (int32_t b = 0; b < 16; b += 2) clear_pair(z, base, at + b, s_taken);
      }
    }
    for (int32_t at = 2 * threadIdx.x; at < lead; at += 2 * kThreads) clear_pair(z, base, at, s_taken);
    for (int32_t at = tail + 2 * threadIdx.x; at < size; at += 2 * kThreads) clear_pair(z, base, at, s_taken);
    return;
  }
  for (int32_t i = threadIdx.x; i < n * z.words; i += kThreads) {
    const int32_t r = z.by_words(i), at = 16 * (i - r * z.words);
    if (s_taken[r]) continue;
    char* to = z.to + (static_cast<int64_t>(r0) + r) * z.stride + at;
    if (at + 16 <= z.bytes) {
      store_loose(to, Word4{0, 0, 0, 0});
    } else {
      for (int32_t b = at; b < z.bytes; b += 2, to += 2) *reinterpret_cast<uint16_t*>(to) = 0;
    }
  }
}

// Which of rows r0 .. r0 + n - 1 occur in a small batch, by a look through its ids.
template <int kThreads>
__device__ __forceinline__ void find_taken(const EmbedArgs& a, int32_t r0, int32_t n, uint8_t* s_taken) {
  for (int32_t r = threadIdx.x; r < n; r += kThreads) s_taken[r] = 0;
  __syncthreads();
  constexpr int kAhead = 8;
  for (int32_t t0 = threadIdx.x; t0 < a.rows; t0 += kAhead * kThreads) {
    uint64_t row[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      row[i] = t0 + i * kThreads < a.rows ? static_cast<uint64_t>(a.ids[t0 + i * kThreads]) : ~uint64_t{0};
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      row[i] -= static_cast<uint64_t>(r0);
      if (row[i] < static_cast<uint64_t>(n) && (!a.mask || a.mask[t0 + i * kThreads] != 0)) s_taken[row[i]] = 1;
    }
  }
  __syncthreads();
}

// ---- sort -------------------------------------------------------------------

// Row t as it enters the sort, from its id and mask: rows that do not count come last.
__device__ __forceinline__ TokenRow token_row(const EmbedArgs& a, int32_t t, int64_t id, bool on, bool* bad) {
  const bool good = id >= 0 && id < a.vocab;
  *bad |= on && !good;
  return TokenRow{static_cast<uint32_t>(on && good ? id : a.vocab), static_cast<uint32_t>(t)};
}

// Rows t[i] as they enter the sort, where in[i]; ids and masks of all of them are on their
// way before the first is waited for.
template <int kEach>
__device__ __forceinline__ void token_rows(const EmbedArgs& a, const uint32_t (&t)[kEach], const bool (&in)[kEach],
                                           TokenRow (&item)[kEach], bool* bad) {
  // without a mask its places are read from the ids, and not looked at
  const uint8_t* mask = a.mask ? a.mask : reinterpret_cast<const uint8_t*>(a.ids);
  int64_t id[kEach];
  uint8_t on[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t at = in[i] ? t[i] : 0u;
    id[i] = a.ids[at];
    on[i] = mask[at];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    item[i] = in[i] ? token_row(a, static_cast<int32_t>(t[i]), id[i], !a.mask || on[i] != 0, bad) : TokenRow{0, 0};
}

// Ranks of a workgroup's items among those with the same digit: on return
// rank[i] counts the earlier ones of the thread's wave, and count[wave][digit] those
// of the waves before; total of each digit in s_total.  Item i of a thread is item
// (wave kEach + i) 64 + lane of the workgroup; `in` says whether it exists.
template <int kEach>
__device__ __forceinline__ void rank_digits(const uint32_t (&digit)[kEach], const bool (&in)[kEach], int32_t bits,
                                            int32_t (*s_count)[kSortBins], int32_t* s_total, int32_t (&rank)[kEach]) {
  const int32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int32_t bins = 1 << bits;
  for (int32_t i = threadIdx.x; i < kSortWaves * bins; i += kSortThreads) s_count[i >> bits][i & (bins - 1)] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    uint64_t peers = __ballot(in[i]);
    for (int32_t b = 0; b < bits; ++b) {
      const bool one = (digit[i] >> b) & 1;
      const uint64_t ones = __ballot(one);
      peers &= one ? ones : ~ones;
    }
    const int32_t lower = __popcll(peers & ((uint64_t{1} << lane) - 1));
    const int32_t before = s_count[wave][digit[i]];
    rank[i] = before + lower;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (in[i] && lower == 0) s_count[wave][digit[i]] = before + __popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  __syncthreads();
  for (int32_t d = threadIdx.x; d < kSortBins; d += kSortThreads) {
    int32_t sum = 0;
    if (d < bins) {
      int32_t n[kSortWaves];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) n[w] = s_count[w][d];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        s_count[w][d] = sum;
        sum += n[w];
      }
    }
    s_total[d] = sum;
  }
  __syncthreads();
}

// Up to kSortBlock rows: one workgroup, all passes in LDS, kEach rows a thread: what each
// costs in instructions is most of the time.  The others clear rows of tokens that do not occur meanwhile, having looked
// through the ids themselves.
template <int kEach>
__global__ __launch_bounds__(kSortThreads) void embed_sort_block_kernel(EmbedArgs a, EmbedSort s, ZeroRows z) {
  __shared__ int32_t s_count[kSortWaves][kSortBins];
  __shared__ int32_t s_total[kSortBins];
  __shared__ int32_t s_wave[kSortWaves + 1];
  __shared__ int s_bad;
  __shared__ TokenRow s_item[kEach * kSortThreads];
  if (blockIdx.x > 0) {
    static_assert(sizeof(s_item) >= kEarlyRows, "a byte a row");
    auto* s_taken = reinterpret_cast<uint8_t*>(s_item);
    const int32_t r0 = z.row(static_cast<int32_t>(blockIdx.x) - 1), n = min(z.each, z.end - r0);
    find_taken<kSortThreads>(a, r0, n, s_taken);
    clear_rows<kSortThreads>(z, r0, n, s_taken);
    return;
  }
  const int32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (threadIdx.x == 0) s_bad = 0;
  TokenRow item[kEach];
  uint32_t place[kEach];
  bool in[kEach], bad = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    place[i] = (wave * kEach + i) * 64 + lane;
    in[i] = place[i] < static_cast<uint32_t>(a.rows);
  }
  token_rows<kEach>(a, place, in, item, &bad);
  for (int32_t p = 0; p < s.passes; ++p) {
    uint32_t digit[kEach];
    int32_t rank[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) digit[i] = (item[i].key >> (p * s.bits)) & ((1u << s.bits) - 1);
    rank_digits<kEach>(digit, in, s.bits, s_count, s_total, rank);
    int32_t all;
    const int32_t n = threadIdx.x < kSortBins ? s_total[threadIdx.x] : 0;
    const int32_t first = block_exclusive_scan<kSortThreads>(n, s_wave, &all);
    if (threadIdx.x < kSortBins) s_total[threadIdx.x] = first;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (in[i]) s_item[s_total[digit[i]] + s_count[wave][digit[i]] + rank[i]] = item[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int32_t t = (wave * kEach + i) * 64 + lane;
      if (in[i]) item[i] = s_item[t];
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int32_t t = (wave * kEach + i) * 64 + lane;
    if (in[i]) s.a[t] = item[i];
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (threadIdx.x == 0 && a.status) *a.status = s_bad ? THD_ERR_TOKEN : THD_OK;
}

// One pass over more rows: each workgroup's digits counted ...
__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedArgs a, EmbedSort s, const TokenRow* from,
                                                                   int32_t shift) {
  __shared__ int32_t s_count[kSortBins];
  __shared__ int s_bad;
  if (threadIdx.x < kSortBins) s_count[threadIdx.x] = 0;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  // below 2^32: the first row is one
  const uint32_t first = blockIdx.x * static_cast<uint32_t>(s.turns) * kSortTile;
  const uint32_t end = min(static_cast<uint32_t>(a.rows), first + static_cast<uint32_t>(s.turns) * kSortTile);
  bool bad = false;
  constexpr int kEach = kSortTile / kSortThreads;
  for (uint32_t t0 = first + threadIdx.x; t0 < end; t0 += kSortTile) {
    TokenRow item[kEach];
    uint32_t t[kEach];
    bool in[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      t[i] = t0 + i * kSortThreads;
      in[i] = t[i] < end;
    }
    if (from) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) item[i] = from[in[i] ? t[i] : 0u];
    } else {
      token_rows<kEach>(a, t, in, item, &bad);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (in[i]) atomicAdd(&s_count[(item[i].key >> shift) & ((1u << s.bits) - 1)], 1);
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (threadIdx.x < kSortBins) s.counts[blockIdx.x * kSortBins + threadIdx.x] = s_count[threadIdx.x];
  if (threadIdx.x == 0 && !from) s.counts[kSortBlocks * kSortBins + blockIdx.x] = s_bad;
}

// ... and its rows placed: a digit's first place is that of all smaller digits
// and of the workgroups before, which every workgroup adds up for itself (counting all
// rows' digits in each of them instead of a launch before: 9000 rows 40 -> 38 us, 32768
// 50 -> 65).
__global__ __launch_bounds__(kSortThreads) void embed_place_kernel(EmbedArgs a, EmbedSort s, const TokenRow* from,
                                                                   TokenRow* to, int32_t shift) {
  constexpr int kEach = kSortTile / kSortThreads;
  __shared__ int32_t s_count[kSortWaves][kSortBins];
  __shared__ int32_t s_total[kSortBins], s_first[kSortBins];
  __shared__ int32_t s_wave[kSortWaves + 1];
  __shared__ int s_bad;
  const int32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t begin = blockIdx.x * static_cast<uint32_t>(s.turns) * kSortTile;
  bool bad = false;
  if (!from && a.status && blockIdx.x == 0) {
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    if (static_cast<int32_t>(threadIdx.x) < s.blocks && s.counts[kSortBlocks * kSortBins + threadIdx.x]) s_bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) *a.status = s_bad ? THD_ERR_TOKEN : THD_OK;
  }
  int32_t before = 0, all = 0;
  if (threadIdx.x < kSortBins) {
#pragma unroll 8
    for (int32_t b = 0; b < s.blocks; ++b) {
      const int32_t n = s.counts[b * kSortBins + threadIdx.x];
      all += n;
      if (b < static_cast<int32_t>(blockIdx.x)) before += n;
    }
  }
  int32_t sum;
  const int32_t smaller = block_exclusive_scan<kSortThreads>(all, s_wave, &sum);
  if (threadIdx.x < kSortBins) s_first[threadIdx.x] = smaller + before;
  __syncthreads();
  for (int32_t turn = 0; turn < s.turns; ++turn) {
    TokenRow item[kEach];
    uint32_t digit[kEach], t[kEach];
    bool in[kEach];
    int32_t rank[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      t[i] = begin + static_cast<uint32_t>(turn) * kSortTile + (wave * kEach + i) * 64 + lane;
      in[i] = t[i] < static_cast<uint32_t>(a.rows);
    }
    if (from) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) item[i] = in[i] ? from[t[i]] : TokenRow{0, 0};
    } else {
      token_rows<kEach>(a, t, in, item, &bad);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) digit[i] = (item[i].key >> shift) & ((1u << s.bits) - 1);
    rank_digits<kEach>(digit, in, s.bits, s_count, s_total, rank);
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (in[i]) to[s_first[digit[i]] + s_count[wave][digit[i]] + rank[i]] = item[i];
    __syncthreads();
    if (threadIdx.x < kSortBins) s_first[threadIdx.x] += s_total[threadIdx.x];
    __syncthreads();
  }
}

// ---- sums -------------------------------------------------------------------

// Stores columns [kPer word, ...) of row v of the gradient, or adds to them.
template <typename TI, typename TO>
__device__ __forceinline__ void finish_row(const EmbedArgs& a, uint32_t v, int32_t word,
                                           const float (&acc)[Elem<TI>::kPer]) {
  constexpr int kPer = Elem<TI>::kPer, kOut = Elem<TO>::kPer;
  TO* to = static_cast<TO*>(a.dtable) + static_cast<int64_t>(v) * a.out_stride + word * kPer;
  if (word * kPer + kPer <= a.width) {
#pragma unroll
    for (int part = 0; part < kPer; part += kOut) {
      float y[kOut];
#pragma unroll
      for (int j = 0; j < kOut; ++j) y[j] = a.scale * acc[part + j];
      if (a.accumulate) {
        float old[kOut];
        Elem<TO>::unpack(load_loose(to + part), old);
#pragma unroll
        for (int j = 0; j < kOut; ++j) y[j] += old[j];
      }
      store_loose(to + part, Elem<TO>::pack(y));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (word * kPer + j < a.width) {
      float y = a.scale * acc[j];
      if (a.accumulate) y += Elem<TO>::load(to + j);
      to[j] = Elem<TO>::round(y);
    }
}

// Partial sums: [unit][0: run from the unit before, 1: run into the next][partial_width].
template <int kPer>
__device__ __forceinline__ void store_partial(const EmbedSort& s, int32_t unit, int32_t slot, int32_t word,
                                              const float (&acc)[kPer]) {
  float* to = s.partial + (2 * static_cast<int64_t>(unit) + slot) * s.partial_width + word * kPer;
#pragma unroll
  for (int part = 0; part < kPer; part += 4)
    *reinterpret_cast<float4*>(to + part) = float4{acc[part], acc[part + 1], acc[part + 2], acc[part + 3]};
}

template <int kPer>
__device__ __forceinline__ void load_partial(const EmbedSort& s, int32_t unit, int32_t slot, int32_t word,
                                             float (&x)[kPer]) {
  const float* from = s.partial + (2 * static_cast<int64_t>(unit) + slot) * s.partial_width + word * kPer;
#pragma unroll
  for (int part = 0; part < kPer; part += 4) {
    const float4 f = *reinterpret_cast<const float4*>(from + part);
    x[part] = f.x, x[part + 1] = f.y, x[part + 2] = f.z, x[part + 3] = f.w;
  }
}

// A row's word of a thread.  Where the row ends inside the word, the 16 bytes that end
// with the row are loaded, and the elements of the word before dropped once all loads are
// on their way: element by element each row was waited for (20510 rows of 10 fp16 elements:
// the launch 61 us).  Rows shorter than a word go element by element.
template <typename T, bool kShort>
struct RowWord {
  static constexpr int kPer = Elem<T>::kPer, kBits = 128 / kPer;
  int32_t at, width;  // elements
  int32_t up, down;   // bits to shift by, to bring the word's own elements to their places
  __device__ __forceinline__ RowWord(int32_t row_width, int32_t word) : width(row_width) {
    at = kShort ? 0 : min(word * kPer, row_width - kPer);
    up = kShort ? kBits * (kPer - row_width) : 0;
    down = kShort ? up : kBits * (word * kPer - at);
  }
  // whether any word of a row has to be shifted
  __device__ __forceinline__ bool ragged() const { return width % kPer != 0; }
  __device__ __forceinline__ Word4 load(const T* row) const {
    if constexpr (!kShort) {
      return load_loose(row + at);
    } else {
      uint32_t x[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] = load_raw(row + min(j, width - 1));
      Word4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = kPer == 8 ? x[2 * i % kPer] | (x[(2 * i + 1) % kPer] << 16) : x[i];
      return w;
    }
  }
  // the word's own elements of what was loaded, zeros after the row
  __device__ __forceinline__ Word4 own(Word4 w) const {
    uint64_t low = w[0] | (static_cast<uint64_t>(w[1]) << 32), high = w[2] | (static_cast<uint64_t>(w[3]) << 32);
    if constexpr (kShort) {  // the elements after the row's go
      if (up >= 64) high = low << (up - 64), low = 0;
      else if (up > 0) high = (high << up) | (low >> (64 - up)), low <<= up;
    }
    if (down >= 64) low = high >> (down - 64), high = 0;
    else if (down > 0) low = (low >> down) | (high << (64 - down)), high >>= down;
    return Word4{static_cast<uint32_t>(low), static_cast<uint32_t>(low >> 32), static_cast<uint32_t>(high),
                 static_cast<uint32_t>(high >> 32)};
  }
};

template <typename TI, typename TO, bool kShort>
__global__ __launch_bounds__(256) void embed_sums_kernel(EmbedArgs a, EmbedSort s, int32_t words, FastDiv by_words,
                                                         int32_t unit_blocks, ZeroRows z) {
  constexpr int kPer = Elem<TI>::kPer;
  const auto none = static_cast<uint32_t>(a.vocab);
  if (static_cast<int32_t>(blockIdx.x) >= unit_blocks) {
    __shared__ uint8_t s_taken[256];
    const int32_t r0 = z.row(static_cast<int32_t>(blockIdx.x) - unit_blocks), n = min(z.each, z.end - r0);
    if (a.rows <= kSortBlock) {
      find_taken<256>(a, r0, n, s_taken);
    } else {
      if (static_cast<int32_t>(threadIdx.x) < n) {
        const auto v = static_cast<uint32_t>(r0 + threadIdx.x);
        int32_t low = 0, high = a.rows;  // first place whose key is not below v
        while (low < high) {
          const int32_t mid = low + ((high - low) >> 1);
          if (s.a[mid].key < v) low = mid + 1;
          else high = mid;
        }
        s_taken[threadIdx.x] = low < a.rows && s.a[low].key == v;
      }
      __syncthreads();
    }
    clear_rows<256>(z, r0, n, s_taken);
    return;
  }
  const FlatPlace place(static_cast<int64_t>(blockIdx.x) * 256, words, by_words);
  int64_t unit64;
  int32_t word;
  place(threadIdx.x, words, &unit64, &word);
  if (unit64 >= s.units) return;
  const auto unit = static_cast<int32_t>(unit64);
  const int32_t first = unit * s.unit, last = min(a.rows - first, s.unit) + first;
  const RowWord<TI, kShort> mine(a.width, word);
  constexpr int kBatch = 8;
  TokenRow item[kBatch], next[kBatch];
  const auto items = [&](int32_t from, TokenRow (&to)[kBatch]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) to[i] = s.a[from < a.rows - i ? from + i : a.rows - 1];
  };
  const uint32_t before = s.a[max(first - 1, 0)].key;
  items(first, item);
  uint32_t key = item[0].key;
  if (key == none) return;  // as are all after it
  bool open = first > 0 && before == key;  // the run began in a unit before
  float acc[kPer] = {};
  for (int32_t i0 = first; i0 < last && key != none; i0 += kBatch) {
    Word4 x[kBatch];
    items(i0 + kBatch < last ? i0 + kBatch : i0, next);  // ahead of the rows they are needed after
#pragma unroll
    for (int i = 0; i < kBatch; ++i)  // also rows that do not count, not looked at
      x[i] = mine.load(static_cast<const TI*>(a.drows) + static_cast<int64_t>(item[i].row) * a.in_stride);
    if (mine.ragged()) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) x[i] = mine.own(x[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i0 + i >= last || key == none) continue;
      if (item[i].key != key) {
        if (open) store_partial<kPer>(s, unit, 0, word, acc);
        else finish_row<TI, TO>(a, key, word, acc);
        open = false;
        key = item[i].key;
#pragma unroll
        for (int j = 0; j < kPer; ++j) acc[j] = 0.0f;
        if (key == none) continue;
      }
      float v[kPer];
      Elem<TI>::unpack(x[i], v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) acc[j] += v[j];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) item[i] = next[i];
  }
  if (key == none) return;
  if (open) store_partial<kPer>(s, unit, 0, word, acc);
  else if (last < a.rows && s.a[last].key == key) store_partial<kPer>(s, unit, 1, word, acc);
  else finish_row<TI, TO>(a, key, word, acc);
}

// Runs that pass a unit's border: the thread of the unit in which the run begins
// adds up its parts.
template <typename TI, typename TO>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedArgs a, EmbedSort s, int32_t words, FastDiv by_words) {
  constexpr int kPer = Elem<TI>::kPer;
  const auto none = static_cast<uint32_t>(a.vocab);
  const FlatPlace place(static_cast<int64_t>(blockIdx.x) * 256, words, by_words);
  int64_t unit64;
  int32_t word;
  place(threadIdx.x, words, &unit64, &word);
  if (unit64 >= s.units) return;
  const auto unit = static_cast<int32_t>(unit64);
  const int32_t first = unit * s.unit, last = min(a.rows - first, s.unit) + first;
  if (last >= a.rows) return;
  const uint32_t begin = s.a[first].key, before = s.a[max(first - 1, 0)].key;
  const uint32_t key = s.a[last - 1].key, next = s.a[last].key;
  if (key == none || next != key) return;
  if (first > 0 && begin == key && before == key) return;  // it began before
  float acc[kPer];
  load_partial<kPer>(s, unit, 1, word, acc);
  // Units whose first row holds the token have a part of the run; their keys come with
  // the parts, those past the run's end for nothing.
  constexpr int kBatch = 16;  // parts in flight
  bool more = true;
  for (int32_t u0 = unit + 1; more; u0 += kBatch) {
    float part[kBatch][kPer];
    uint32_t k[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int32_t u = min(u0 + i, s.units - 1);
      k[i] = s.a[static_cast<int64_t>(u) * s.unit].key;
      load_partial<kPer>(s, u, 0, word, part[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      more = more && u0 + i < s.units && k[i] == key;
#pragma unroll
      for (int j = 0; j < kPer; ++j) acc[j] += more ? part[i][j] : 0.0f;
    }
  }
  finish_row<TI, TO>(a, key, word, acc);
}

constexpr int64_t kCachedTable = 256 << 20;

// Rows [first, end) of the table, at most so many to a workgroup, and `bytes` of it: a
// quarter of that for a run and a few ids, which are looked through in no time.
ZeroRows zero_rows(const EmbedArgs& a, int32_t first, int32_t end, int64_t bytes, int32_t most_rows) {
  const int64_t size = a.out_dtype == THD_FP32 ? 4 : 2, row = a.width * size;
  ZeroRows z{};
  z.to = static_cast<char*>(a.dtable);
  z.stride = a.out_stride * size;
  z.bytes = static_cast<int32_t>(row);
  z.words = static_cast<int32_t>((row + 15) / 16);
  z.by_words = FastDiv::make(z.words);
  z.by_bytes = FastDiv::make(z.bytes);
  z.first = first;
  z.end = end;
  z.run = a.out_stride == a.width && row * a.vocab > kCachedTable;
  if (z.run && a.rows <= kSortThreads) bytes /= 4;
  const int64_t each = (bytes + row / 2) / row;
  z.each = static_cast<int32_t>(each < 1 ? 1 : each < most_rows ? each : most_rows);
  return z;
}
int64_t zero_blocks(const EmbedArgs& a, const ZeroRows& z) {
  return a.accumulate ? 0 : (static_cast<int64_t>(z.end) - z.first + z.each - 1) / z.each;
}
// Rows of the table that are cleared beside the sort of a small batch, which leaves most
// of the chip free; the others are, beside the sums.  What fits beside a sort is bytes: so
// many and so many more for each row that it has to sort.  A quarter of the table
// instead (in microseconds, fp32): 153 rows, table of 69994 x 267 29.8 against 24.2; 8000
// rows, 262000 x 64 41.0 and 33.7, 100000 x 500 56.6 and 48.3; 4099 rows, 100003 x 1001 95.6
// and 97.0; half as many bytes 24.4, 33.4, 50.7 and 99.6.
constexpr int64_t kEarlyBytes = 28000000, kEarlyBytesPerRow = 9000;
int32_t cleared_early(const EmbedArgs& a) {
  if (a.rows == 0 || a.rows > kSortBlock) return 0;
  const int64_t row = static_cast<int64_t>(a.width) * (a.out_dtype == THD_FP32 ? 4 : 2);
  const int64_t most = (kEarlyBytes + kEarlyBytesPerRow * a.rows) / row;
  return static_cast<int32_t>(most < a.vocab ? most : a.vocab);
}

template <typename TI, typename TO>
hipError_t sums(const EmbedArgs& a, const EmbedSort& s, hipStream_t stream) {
  const int32_t words = (a.width + Elem<TI>::kPer - 1) / Elem<TI>::kPer;
  const auto by_words = FastDiv::make(words);
  const auto unit_blocks = static_cast<int32_t>((static_cast<int64_t>(s.units) * words + 255) / 256);
  const ZeroRows z = zero_rows(a, cleared_early(a), a.vocab, 65536, 256);  // rows are searched for side by side
  const int64_t blocks = unit_blocks + zero_blocks(a, z);
  if (blocks > 0 && a.width < Elem<TI>::kPer)
    embed_sums_kernel<TI, TO, true>
        <<<static_cast<uint32_t>(blocks), 256, 0, stream>>>(a, s, words, by_words, unit_blocks, z);
  else if (blocks > 0)
    embed_sums_kernel<TI, TO, false>
        <<<static_cast<uint32_t>(blocks), 256, 0, stream>>>(a, s, words, by_words, unit_blocks, z);
  if (unit_blocks > 0 && s.units > 1)
    embed_join_kernel<TI, TO><<<unit_blocks, 256, 0, stream>>>(a, s, words, by_words);
  return hipGetLastError();
}

template <typename T>
hipError_t lookup(const EmbedArgs& a, hipStream_t stream) {
  const int32_t words = (a.width + Elem<T>::kPer - 1) / Elem<T>::kPer;
  const int64_t blocks = (static_cast<int64_t>(a.rows) * words + 256 * kLookupEach - 1) / (256 * kLookupEach);
  embed_kernel<T><<<static_cast<uint32_t>(blocks + a.scan), 256, 0, stream>>>(a, words, FastDiv::make(words));
  return hipGetLastError();
}

}  // namespace

EmbedSort embed_sort(int64_t rows, int64_t vocab, int64_t width) {
  EmbedSort s{};
  int32_t bits = 1;
  while ((int64_t{1} << bits) <= vocab) ++bits;  // keys 0..vocab
  s.passes = (bits + 8) / 9;
  s.bits = (bits + s.passes - 1) / s.passes;
  s.blocks = 1;
  if (rows > kSortBlock) {
    const int64_t tiles = (rows + kSortTile - 1) / kSortTile;
    s.turns = static_cast<int32_t>((tiles + kSortBlocks - 1) / kSortBlocks);
    s.blocks = static_cast<int32_t>((tiles + s.turns - 1) / s.turns);
  }
  // long units have fewer borders, short ones give few rows more threads (rows of 4096
  // bf16, units of 32, 64 and 128: 10000 rows 102, 114 and 142 us, 32768 163, 155 and
  // 162, 131072 385, 361 and 345)
  s.unit = rows <= kSortBlock ? 16 : rows < 16384 ? 32 : rows < 65536 ? 64 : 128;
  // Short rows leave few threads, and lanes of a wave then hold different units, whose
  // tokens end one by one: shorter units while there are fewer than kFewSums threads, but
  // no more than kMostShort units, as a run's parts are added one after the other (sums and
  // joining of 20510 rows of 10 fp16 44 -> 27 us, of 84222 of 94 72 -> 49, of 131072 of 20
  // bf16 88 -> 59; 131072 rows of one token in units of 16 688).
  const int64_t words = (width + 7) / 8;
  while (s.unit > 16 && rows / s.unit * words < kFewSums && rows / s.unit * 2 <= kMostShort) s.unit /= 2;
  s.units = static_cast<int32_t>((rows + s.unit - 1) / s.unit);
  return s;
}

hipError_t launch_embedding(const EmbedArgs& a, hipStream_t stream) {
  if (a.dtype == THD_BF16) return lookup<Bf16>(a, stream);
  return a.dtype == THD_FP16 ? lookup<Fp16>(a, stream) : lookup<float>(a, stream);
}

hipError_t launch_embedding_sort(const EmbedArgs& a, const EmbedSort& s, hipStream_t stream) {
  if (a.rows <= kSortBlock) {
    const ZeroRows z = zero_rows(a, 0, cleared_early(a), 131072, kEarlyRows);
    const auto blocks = static_cast<uint32_t>(1 + zero_blocks(a, z));
    if (a.rows <= kSortThreads) embed_sort_block_kernel<1><<<blocks, kSortThreads, 0, stream>>>(a, s, z);
    else if (a.rows <= 2 * kSortThreads) embed_sort_block_kernel<2><<<blocks, kSortThreads, 0, stream>>>(a, s, z);
    else if (a.rows <= 4 * kSortThreads) embed_sort_block_kernel<4><<<blocks, kSortThreads, 0, stream>>>(a, s, z);
    else embed_sort_block_kernel<kSortBlock / kSortThreads><<<blocks, kSortThreads, 0, stream>>>(a, s, z);
    return hipGetLastError();
  }
  const TokenRow* from = nullptr;
  for (int32_t p = 0; p < s.passes; ++p) {
    TokenRow* to = (s.passes - 1 - p) % 2 == 0 ? s.a : s.b;
    embed_count_kernel<<<s.blocks, kSortThreads, 0, stream>>>(a, s, from, p * s.bits);
    embed_place_kernel<<<s.blocks, kSortThreads, 0, stream>>>(a, s, from, to, p * s.bits);
    from = to;
  }
  return hipGetLastError();
}

hipError_t launch_embedding_sums(const EmbedArgs& a, const EmbedSort& s, hipStream_t stream) {
  if (a.dtype == THD_FP32) return sums<float, float>(a, s, stream);
  if (a.dtype == THD_BF16)
    return a.out_dtype == THD_FP32 ? sums<Bf16, float>(a, s, stream) : sums<Bf16, Bf16>(a, s, stream);
  return a.out_dtype == THD_FP32 ? sums<Fp16, float>(a, s, stream) : sums<Fp16, Fp16>(a, s, stream);
}

}  // namespace thdcp
