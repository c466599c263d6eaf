// Gradients of the attention inside documents.  With p as in the forward pass
// (formed again from q, k and the row's log-sum-exp):
//   dp_ij = dout_i . v_j,   delta_i = sum_j p_ij dp_ij = dout_i . out_i
//   dz_ij = p_ij (dp_ij - delta_i) (1 - (z_ij / cap)^2)       (cap > 0)
//   dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i dz_ij q_i,  dq_i = scale sum_j dz_ij k_j
//
// Query gradients and key gradients come from two kernels, each of which owns
// its rows and adds in a fixed order; scores and dp are formed in both, seven
// products instead of five, against atomic additions into 32-bit sums whose order
// would change the results.  Both hold a wave's own 32 rows (queries and dout, or
// keys and values) in registers as B operands, so that p and dz come out of the
// products as operands of the next ones, and move the other side's rows
// through LDS.  p and dz are rounded to the tensors' type as factors of those
// products; with delta from the rounded out (of rows with more keys than a block) that
// makes dq and dk differ from the formulas by about 1.6 roundings of their own elements
// (root mean square, bf16 2.7e-3 of the values; rounding the exact gradients alone
// 1.7e-3).
//
// bf16 takes delta in the query gradients' kernel, which runs first and leaves it for
// the key gradients: a launch and a reading of dout less (16384 tokens of short
// documents, 32 heads of 128: 54 us of 446).
//
// Bound as the forward pass is; one document of 8192 tokens, causal, 32 heads of 128
// over 8: dq 713 us (1157 TFLOP/s, matrix units busy 61 %, LDS 30 %), dk and dv 996 (1104,
// 53 %, 40 %) and 70 to add up their parts; with a cap 888 and 1202; in fp16 798 and 1124,
// and 46 for delta and the largest norms.
//
// fp16: p times 2^14 and dz times a power of two for which no dz passes the
// type's range (from the largest norms of a dout row and of a v row) keep small
// factors out of the subnormals; the sums are scaled back.
#include "thd_attn_device.h"

namespace thdcp {

namespace {

// Of fp16 probabilities, which are 1 at most.  Those from 2^-28 on keep all their bits.
constexpr float kProbabilityScale = 16384.0f;

// Power of two by which fp16 score gradients are held: |dz| <= 2 |dout| |v|.
__device__ __forceinline__ float gradient_scale(const AttnPlan& p) {
  const float bound = 2.0f * __builtin_bit_cast(float, p.header[kAttnMaxGrad]) *
                      __builtin_bit_cast(float, p.header[kAttnMaxValue]);
  if (!(bound > 0.0f) || !(bound < kAttnInf)) return 1.0f;
  return ldexpf(1.0f, 14 - ilogbf(bound) - 1);  // bound times it is below 2^14
}

// 16 lanes add up.
__device__ __forceinline__ float add_row16(float x) {
#pragma unroll
  for (int i = 1; i < 16; i <<= 1) x += __shfl_xor(x, i);
  return x;
}

// Rows that are not finite have no say in other rows' scale.
__device__ __forceinline__ float finite_or_zero(float x) { return x < kAttnInf ? x : 0.0f; }

// sum + x . y of eight elements
template <typename T>
__device__ __forceinline__ float dot_words(const U32x4& x, const U32x4& y, float sum) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u = x[k], v = y[k];
    sum = fmaf(T::low(u), T::low(v), sum);
    sum = fmaf(T::high(u), T::high(v), sum);
  }
  return sum;
}

// delta of a tile's rows, 16 lanes a row, and the largest norms, for fp16.
template <typename T>
__global__ __launch_bounds__(256) void attn_delta_kernel(AttnArgs a, int32_t query_blocks) {
  __shared__ float s_most[4];
  const int32_t l = threadIdx.x & 63, word = l & 15;
  const bool query = static_cast<int32_t>(blockIdx.x) < query_blocks;
  float most = 0.0f;
  if (query) {
    const int32_t parts = a.heads / a.tile_heads, first_head = blockIdx.x % parts * a.tile_heads;
    const QueryTile tile = a.plan.query_tiles[blockIdx.x / parts];
    if (tile.rows == 0) return;
    const int32_t tile_rows = kAttnRows / a.tile_heads;  // 32 and up: 16 rows are of one head
#pragma unroll
    for (int i = 0; i < kAttnRows / 16; ++i) {
      const int32_t head = first_head + 16 * i / tile_rows, row = 16 * i % tile_rows + (threadIdx.x >> 4);
      const RowsRead o(head_rows(a.out, tile.row, head), static_cast<int32_t>(2 * a.out.row), tile.valid, a.dim);
      const RowsRead g(head_rows(a.dout, tile.row, head), static_cast<int32_t>(2 * a.dout.row), tile.valid, a.dim);
      const U32x4 x = o.load(row, word, a.dim), y = g.load(row, word, a.dim);
      const float dot = add_row16(dot_words<T>(x, y, 0.0f));
      if (word == 0 && row < tile.valid)
        a.plan.delta[static_cast<int64_t>(head) * a.rows + tile.row + row] = dot;
      most = fmaxf(most, finite_or_zero(add_row16(dot_words<T>(y, y, 0.0f))));
    }
  } else {
    const int32_t b = blockIdx.x - query_blocks;
    const int32_t index = b / a.kv_heads, head = b % a.kv_heads;
    const KeyTile tile = a.plan.key_tiles[index];
    if (tile.keys == 0) return;
    const RowsRead v(head_rows(a.v, static_cast<int64_t>(tile.doc) + tile.key, head),
                     static_cast<int32_t>(2 * a.v.row), tile.valid, a.dim);
#pragma unroll
    for (int i = 0; i < kAttnKeys / 16; ++i) {
      const U32x4 x = v.load(16 * i + (threadIdx.x >> 4), word, a.dim);
      most = fmaxf(most, finite_or_zero(add_row16(dot_words<T>(x, x, 0.0f))));
    }
  }
#pragma unroll
  for (int i = 16; i < 64; i <<= 1) most = fmaxf(most, __shfl_xor(most, i));
  if (l == 0) s_most[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    most = sqrtf(fmaxf(fmaxf(s_most[0], s_most[1]), fmaxf(s_most[2], s_most[3])));
    // not negative: floats order as their bits do, and a maximum has no order
    if (most > 0.0f)
      atomicMax(a.plan.header + (query ? kAttnMaxGrad : kAttnMaxValue), __builtin_bit_cast(int32_t, most));
  }
}

// Sum of p dp over a block of scores (keys are registers), for both halves of a wave.
template <bool kCap, typename Visible>
__device__ __forceinline__ float block_delta(const AttnArgs& a, F32x16 s, const F32x16& dp, float lse,
                                             Visible visible) {
  const float factor = kCap ? 1.0f : a.scale * kAttnLog2e;
  if constexpr (kCap) attn_capped(a, s);
  float sum = 0.0f;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (visible(r)) sum = fmaf(attn_exp2(fmaf(s[r], factor, -lse)), dp[r], sum);
  return add_halves(sum);
}

// What both kernels make of a block of scores and dp (32 x 32, one row a
// register): p, and dz times `held`.  lse and delta are the registers' or the
// lane's, by the caller's functions of the register; scores not seen have p 0.
template <typename T, bool kCap, typename Lse, typename Delta, typename Visible>
__device__ __forceinline__ void score_gradients(const AttnArgs& a, F32x16 s, F32x16 dp, float held, Lse lse,
                                                Delta delta, Visible visible, U32x4 (&p16)[2], U32x4 (&dz16)[2]) {
  const float factor = kCap ? 1.0f : a.scale * kAttnLog2e;
  // the slope of the cap, held - (root s)^2
  const float root = kCap ? __builtin_sqrtf(held) / (a.cap * kAttnLog2e) : 0.0f;
  if constexpr (kCap) attn_capped(a, s);
#pragma unroll
  for (int r = 0; r < 16; r += 2) {
    if (kCap && r % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // few registers at a time
    float p[2], dz[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float z = s[r + e] * root, slope = kCap ? fmaf(-z, z, held) : held;
      float x = fmaf(s[r + e], factor, -lse(r + e));
      // 1 is p's most, which roundings of large scores pass, and fp16's range with it; NaN stays
      if (T::kNarrow) x = __builtin_elementwise_minimum(x, 0.0f);
      p[e] = visible(r + e) ? attn_exp2(x) : 0.0f;
      dz[e] = p[e] * (dp[r + e] - delta(r + e)) * slope;
      if (T::kNarrow) p[e] *= kProbabilityScale;
    }
    p16[r >> 3][(r & 7) >> 1] = T::pack(p[0], p[1]);
    dz16[r >> 3][(r & 7) >> 1] = T::pack(dz[0], dz[1]);
  }
}

// A number for each register's row of a C fragment, from this lane's first row on.
__device__ __forceinline__ F32x16 lds_rows(const float* at) {
  F32x16 r;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float4 x = *reinterpret_cast<const float4*>(at + 8 * g);
    r[4 * g] = x.x, r[4 * g + 1] = x.y, r[4 * g + 2] = x.z, r[4 * g + 3] = x.w;
  }
  return r;
}

// acc [dim][32] += (the 32 rows f was read from)^T b
template <typename T, int kDim>
__device__ __forceinline__ void add_columns(F32x16 (&acc)[kDim / 32], const U32x4 (&f)[kDim / 32][2],
                                            const U32x4 (&b)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int t = 0; t < kDim / 32; ++t) acc[t] = T::mfma(f[t][j], b[j], acc[t]);
}

// s += x bx^T and dp += y by^T for 32 rows of two tiles, a lane's place in them `row`.
// Reads go out four words at a time before the first is waited for.
template <typename T, int kDim>
__device__ __forceinline__ void row_products(const char* x, const char* y, int32_t row, const U32x4 (&bx)[kDim / 16],
                                             const U32x4 (&by)[kDim / 16], F32x16& s, F32x16& dp) {
  asm volatile("" : "+v"(row));  // words' places differ in single bits: not kept in registers
  constexpr int kRead = kDim % 64 == 0 ? 4 : 3;
#pragma unroll
  for (int i0 = 0; i0 < kDim / 16; i0 += kRead) {
    U32x4 fx[kRead], fy[kRead];
#pragma unroll
    for (int i = 0; i < kRead; ++i) {
      fx[i] = lds_read(x + (row ^ (32 * (i0 + i))), 0);
      fy[i] = lds_read(y + (row ^ (32 * (i0 + i))), 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kRead; ++i) {
      s = T::mfma(fx[i], bx[i0 + i], s);
      dp = T::mfma(fy[i], by[i0 + i], dp);
    }
  }
}

// Query gradients: 128 query rows a workgroup, as in the forward pass; 64 keys at a
// time, of which two workgroups' tiles fill a compute unit's LDS.
template <typename T, int kDim, bool kCap>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(AttnArgs a) {
  constexpr int kTile = kAttnStep * kRowBytes<kDim>;
  __shared__ __attribute__((aligned(16))) char s_tiles[4 * kTile];  // keys, values, and both again
  const AttnPlace place(blockIdx.x, a.kv_heads, a.group / a.tile_heads);
  if (place.tile >= a.plan.max_query_tiles) return;
  const QueryTile tile = a.plan.query_tiles[place.tile];
  if (tile.rows == 0) return;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t l = threadIdx.x & 63, c = l & 31, h = l >> 5;
  const WaveRows own(a, tile, place, wave);
  const int32_t pos = tile.pos + own.first;
  const float held = T::kNarrow ? gradient_scale(a.plan) : 1.0f;

  F32x16 dq[kDim / 32];
#pragma unroll
  for (int t = 0; t < kDim / 32; ++t) dq[t] = zero16();
  if (tile.valid > 0) {
    U32x4 q[kDim / 16], g[kDim / 16];
    const int32_t row_at = lds_word<kDim>(c, h);
    const uint32_t column_at[2] = {lds_address(s_tiles) + transposed_at<kDim>(0, 0),
                                   lds_address(s_tiles) + transposed_at<kDim>(0, 1)};
    const RowsRead queries(head_rows(a.q, tile.row + own.first, own.head), static_cast<int32_t>(2 * a.q.row),
                           own.valid, a.dim);
    const RowsRead grads(head_rows(a.dout, tile.row + own.first, own.head), static_cast<int32_t>(2 * a.dout.row),
                         own.valid, a.dim);
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) {
      q[i] = queries.load(c, 2 * i + h, a.dim);
      g[i] = grads.load(c, 2 * i + h, a.dim);
    }
    float lse = kAttnInf, delta = 0.0f;  // of a row that sees nothing: p 0
    if (c < own.valid) {
      const int64_t at = static_cast<int64_t>(own.head) * a.rows + tile.row + own.first + c;
      const float x = a.lse[at] * kAttnLog2e;
      lse = x == -kAttnInf ? kAttnInf : x;
      if constexpr (T::kNarrow) delta = a.plan.delta[at];
    }
    if constexpr (!T::kNarrow) {
      // here, where the rows of dout are at hand, for the key gradients' launch too
      const RowsRead outs(head_rows(a.out, tile.row + own.first, own.head), static_cast<int32_t>(2 * a.out.row),
                          own.valid, a.dim);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < kDim / 16; ++i) dot = dot_words<T>(outs.load(c, 2 * i + h, a.dim), g[i], dot);
      delta = add_halves(dot);
      if (l < own.valid) a.plan.delta[static_cast<int64_t>(own.head) * a.rows + tile.row + own.first + l] = delta;
    }
    const Seen first(a, tile.pos, tile.real), last(a, tile.pos + tile.valid - 1, tile.real);
    const int32_t end = last.low + static_cast<int32_t>(last.span);
    int32_t key = first.low & ~(kAttnStep - 1);
    const Seen seen(a, pos + c, tile.real);
    RowsWalk keys(a.k, static_cast<int64_t>(tile.doc) + key, place.kv_head, tile.real - key);
    RowsWalk values(a.v, static_cast<int64_t>(tile.doc) + key, place.kv_head, tile.real - key);
    const KeySteps steps(a, pos, 32, own.valid, tile.real);
    // Rows of which all keys stand in one block take delta from it, not from the rounded
    // out: with few keys dp - delta is a small difference of large numbers.
    const int32_t only = (max(steps.any, 0) + 31) & ~31;
    const bool alone = only + 32 >= steps.any_end;
    const auto load = [&](int32_t to) {
      keys.load<kDim, kAttnStep>(s_tiles + to, a.dim);
      values.load<kDim, kAttnStep>(s_tiles + to + kTile, a.dim);
    };
    const auto turn = [&](auto now, int32_t next) {
      lds_arrived();
      __syncthreads();
      if (key + kAttnStep < end) load(next);
#pragma unroll
      for (int b = 0; b < kAttnStep / 32; ++b) {
        const int32_t k0 = key + 32 * b, skip = 32 * b * kRowBytes<kDim>;
        if (k0 < steps.any || k0 >= steps.any_end) continue;
        F32x16 s = zero16(), dp = zero16();
        row_products<T, kDim>(s_tiles + now + skip, s_tiles + now + kTile + skip, row_at, q, g, s, dp);
        U32x4 p16[2], dz16[2];
        const bool all = k0 >= steps.all && k0 < steps.all_end;
        const auto sees = [&](int r) { return seen(k0 + 4 * h + (r & 3) + 8 * (r >> 2)); };
        if (alone) {
          delta = block_delta<kCap>(a, s, dp, lse, sees);
          if (l < own.valid) a.plan.delta[static_cast<int64_t>(own.head) * a.rows + tile.row + own.first + l] = delta;
        }
        const auto lane_lse = [&](int) { return lse; };
        const auto lane_delta = [&](int) { return delta; };
        if (all)
          score_gradients<T, kCap>(a, s, dp, held, lane_lse, lane_delta, [](int) { return true; }, p16, dz16);
        else
          score_gradients<T, kCap>(a, s, dp, held, lane_lse, lane_delta, sees, p16, dz16);
        U32x4 f[kDim / 32][2];
        read_columns<kDim, now>(column_at[0] + skip, column_at[1] + skip, f);
        add_columns<T, kDim>(dq, f, dz16);
      }
      key += kAttnStep;
    };
    load(0);
    while (key < end) {
      turn(Place<0>{}, 2 * kTile);
      if (key >= end) break;
      turn(Place<2 * kTile>{}, 0);
    }
    __syncthreads();
  }
  store_rows<T, kDim>(s_tiles + wave * kTile, dq, a.scale / held,
                      const_cast<char*>(head_rows(a.dq, tile.row + own.first, own.head)), 2 * a.dq.row, own.rows,
                      own.valid, a.dim);
}

// The query rows that a key tile's gradients come from: for each of the workgroup's
// heads, of each of the document's chunks the rows that see the tile, kStep at a time,
// from running addresses.
template <int kStep>
struct QueryWalk {
  int32_t head, heads_end, chunk;
  int32_t left = 0;                 // rows of the chunk that are still to come
  int32_t pos = 0;                  // position of the next one
  const char *q = nullptr, *grad = nullptr;
  int64_t number = 0;               // of its lse and delta
  __device__ __forceinline__ QueryWalk(const AttnArgs& a, const KeyTile& k, int32_t first_head, int32_t heads)
      : head(first_head), heads_end(first_head + heads), chunk(-1) {
    settle(a, k);
  }
  __device__ __forceinline__ bool done() const { return head >= heads_end; }
  // To the first row of the next chunk that has any.
  __device__ __forceinline__ void settle(const AttnArgs& a, const KeyTile& k) {
    while (left <= 0) {
      if (++chunk == (a.cp == 1 ? 1 : 2)) {
        chunk = 0;
        ++head;
      }
      if (done()) return;
      const int32_t start = a.cp == 1 ? 0 : chunk ? (2 * a.cp - 1 - a.rank) * k.chunk : a.rank * k.chunk;
      const int32_t valid = min(k.chunk, k.real - start);
      const int32_t low = a.causal ? k.key : a.window ? max(0, k.key - a.window + 1) : 0;
      const int32_t high = a.window ? window_end(a, k.key + k.valid, k.real) : k.real;
      const int32_t first = max(0, low - start);
      left = min(valid, high - start) - first;
      if (left <= 0) continue;
      pos = start + first;
      const int64_t row = static_cast<int64_t>(k.first) + chunk * k.chunk + first;
      q = head_rows(a.q, row, head);
      grad = head_rows(a.dout, row, head);
      number = static_cast<int64_t>(head) * a.rows + row;
    }
  }
  __device__ __forceinline__ void next(const AttnArgs& a, const KeyTile& k) {
    left -= kStep;
    pos += kStep;
    q += 2 * a.q.row * kStep;
    grad += 2 * a.dout.row * kStep;
    number += kStep;
    if (left <= 0) settle(a, k);
  }
};

// The steps of 32 rows, numbered by their first position, that see something of keys
// [k, k + valid), and that see everything of [k, k + 32).
struct RowSteps {
  int32_t any, any_end, all, all_end;
  __device__ __forceinline__ RowSteps(const AttnArgs& a, int32_t k, int32_t valid) {
    any = a.causal ? k - 31 : a.window ? k - a.window - 30 : INT32_MIN;
    any_end = valid <= 0 ? INT32_MIN : a.window ? window_end(a, k + valid, INT32_MAX) : INT32_MAX;
    all = a.causal ? k + 31 : a.window ? k + 32 - a.window : INT32_MIN;
    all_end = a.window ? window_end(a, k + 1, INT32_MAX) - 31 : INT32_MAX;
  }
};

// Number threadIdx.x of n, 0 past them.
__device__ __forceinline__ float load_number(const float* from, int32_t n) {
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(from), 0, 4 * n, kBufferWord3);
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsrc, 4 * threadIdx.x, 0, 0));
}

// A key row's sums of one part of a group's heads: [part][dk, dv][tokens][kv heads][dim].
__device__ __forceinline__ float* partial_sums(const AttnArgs& a, int32_t part, int32_t which, int64_t row,
                                               int32_t head) {
  return a.plan.partial + (((2 * static_cast<int64_t>(part) + which) * a.total + row) * a.kv_heads + head) * a.dim;
}

// A wave's accumulators [kDim][32 rows] in 32 bits; rows from `valid` on are zero.
template <int kDim>
__device__ __forceinline__ void store_sums(const AttnArgs& a, int32_t part, int32_t which,
                                           const F32x16 (&acc)[kDim / 32], float factor, int64_t row, int32_t head,
                                           int32_t rows, int32_t valid) {
  const int32_t c = threadIdx.x & 31, h = (threadIdx.x & 63) >> 5;
  if (c >= rows) return;
  float* to = partial_sums(a, part, which, row + c, head);
#pragma unroll
  for (int t = 0; t < kDim / 32; ++t)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int32_t d = 32 * t + 8 * g + 4 * h;
      float4 x = {acc[t][4 * g] * factor, acc[t][4 * g + 1] * factor, acc[t][4 * g + 2] * factor,
                  acc[t][4 * g + 3] * factor};
      if (c >= valid) x = float4{0.0f, 0.0f, 0.0f, 0.0f};
      if (d < a.dim) *reinterpret_cast<float4*>(to + d) = x;
    }
}

// Key and value gradients: 128 keys of one key head a workgroup, 32 a wave.
//
// A wave holds its keys' rows and both sums in registers.  With 128 elements a head
// that leaves no room for its values' rows beside two waves on each SIMD, of which one
// computes probabilities while the other multiplies; they are read from LDS instead,
// and query rows come 32 at a time, so that two workgroups share a compute unit's LDS.
//
// Where there are few key tiles, the heads of a group are dealt out over `parts`
// workgroups, each of which leaves its sums in 32 bits for attn_join_kernel.
template <typename T, int kDim, bool kCap>
__global__ __launch_bounds__(256, 2) void attn_dkv_kernel(AttnArgs a) {
  constexpr bool kHold = kDim <= 96;           // values in registers
  constexpr int kStep = kHold ? kAttnStep : 32;
  constexpr int kTile = kStep * kRowBytes<kDim>;
  // query rows, rows of dout, both again, values
  __shared__ __attribute__((aligned(16))) char s_tiles[4 * kTile + (kHold ? 0 : kAttnKeys * kRowBytes<kDim>)];
  __shared__ __attribute__((aligned(16))) float s_lse[2][kStep], s_delta[2][kStep];
  const AttnPlace place(blockIdx.x, a.kv_heads, a.key_parts);
  if (place.tile >= a.plan.max_key_tiles) return;
  const KeyTile tile = a.plan.key_tiles[place.tile];
  if (tile.keys == 0) return;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t l = threadIdx.x & 63, c = l & 31, h = l >> 5;
  const int32_t own_keys = min(32, max(0, tile.keys - 32 * wave));
  const int32_t own_valid = min(32, max(0, tile.valid - 32 * wave));
  const int32_t key = tile.key + 32 * wave;
  const int64_t stream = static_cast<int64_t>(tile.doc) + key;
  const float held = T::kNarrow ? gradient_scale(a.plan) : 1.0f;

  F32x16 dk[kDim / 32], dv[kDim / 32];
#pragma unroll
  for (int t = 0; t < kDim / 32; ++t) dk[t] = dv[t] = zero16();
  if (tile.valid > 0) {
    U32x4 k[kDim / 16], v[kHold ? kDim / 16 : 1];
    const int32_t row_at = lds_word<kDim>(c, h);
    const uint32_t column_at[2] = {lds_address(s_tiles) + transposed_at<kDim>(0, 0),
                                   lds_address(s_tiles) + transposed_at<kDim>(0, 1)};
    const RowsRead keys(head_rows(a.k, stream, place.kv_head), static_cast<int32_t>(2 * a.k.row), own_valid, a.dim);
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) k[i] = keys.load(c, 2 * i + h, a.dim);
    if constexpr (kHold) {
      const RowsRead values(head_rows(a.v, stream, place.kv_head), static_cast<int32_t>(2 * a.v.row), own_valid, a.dim);
#pragma unroll
      for (int i = 0; i < kDim / 16; ++i) v[i] = values.load(c, 2 * i + h, a.dim);
    } else {
      const RowsRead values(head_rows(a.v, static_cast<int64_t>(tile.doc) + tile.key, place.kv_head),
                            static_cast<int32_t>(2 * a.v.row), tile.valid, a.dim);
      load_tile<kDim, kAttnKeys>(s_tiles + 4 * kTile, values, a.dim);
    }
    const int32_t part_heads = a.group / a.key_parts;
    QueryWalk<kStep> walk(a, tile, place.kv_head * a.group + place.part * part_heads, part_heads);
    const RowSteps steps(a, key, own_valid);
    // positions that see key key + c
    const Seen seen(a.causal ? key + c : a.window ? key + c - a.window + 1 : 0,
                    a.window ? (a.causal ? a.window : 2u * a.window - 1u) : 0x7fffffffu);
    float next_lse = 0.0f, next_delta = 0.0f;
    // what scores start from, or (with a cap) is taken from their power of two
    const float lse_factor = kCap ? kAttnLog2e : -1.0f / a.scale;
    const auto load = [&](int32_t to) {
      const int32_t n = min(kStep, walk.left);
      // ahead of the tiles, which arrive after them; rows past the range are zero in all
      // four, and add nothing
      next_lse = load_number(a.lse + walk.number, n);
      next_delta = load_number(a.plan.delta + walk.number, n);
      load_tile<kDim, kStep>(s_tiles + to, RowsRead(walk.q, static_cast<int32_t>(2 * a.q.row), n, a.dim), a.dim);
      load_tile<kDim, kStep>(s_tiles + to + kTile, RowsRead(walk.grad, static_cast<int32_t>(2 * a.dout.row), n, a.dim),
                             a.dim);
    };
    const auto turn = [&](auto queries, int32_t mine, int32_t next) {
      if (threadIdx.x < kStep) {
        // a row that sees nothing: p 0
        s_lse[mine][threadIdx.x] = next_lse == -kAttnInf ? (kCap ? kAttnInf : -kAttnInf) : next_lse * lse_factor;
        s_delta[mine][threadIdx.x] = -next_delta;
      }
      lds_arrived();
      __syncthreads();
      const int32_t n = walk.left, pos = walk.pos;
      walk.next(a, tile);
      if (!walk.done()) load(next);
#pragma unroll
      for (int b = 0; b < kStep / 32; ++b) {
        const int32_t p0 = pos + 32 * b, skip = 32 * b * kRowBytes<kDim>;
        if (32 * b >= n || p0 < steps.any || p0 >= steps.any_end) continue;
        // the sums start at what is taken from them: -lse (as a score; with a cap, after it)
        // and -delta
        F32x16 s = kCap ? zero16() : lds_rows(&s_lse[mine][32 * b + 4 * h]);
        F32x16 dp = lds_rows(&s_delta[mine][32 * b + 4 * h]);
        const char* rows = s_tiles + queries + skip;
        if constexpr (kHold) {
          row_products<T, kDim>(rows, rows + kTile, row_at, k, v, s, dp);
        } else {
          int32_t row = row_at, value = row_at + 32 * wave * kRowBytes<kDim>;
          asm volatile("" : "+v"(row), "+v"(value));
#pragma unroll
          for (int i0 = 0; i0 < kDim / 16; i0 += 2) {
            U32x4 fx[2], fy[2], fv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              fx[i] = lds_read(rows + (row ^ (32 * (i0 + i))), 0);
              fy[i] = lds_read(rows + (row ^ (32 * (i0 + i))), kTile);
              fv[i] = lds_read(s_tiles + (value ^ (32 * (i0 + i))), 4 * kTile);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s = T::mfma(fx[i], k[i0 + i], s);
              dp = T::mfma(fy[i], fv[i], dp);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        U32x4 p16[2], dz16[2];
        const float* lse = &s_lse[mine][32 * b + 4 * h];
        const auto row_lse = [&](int r) { return kCap ? lse[(r & 3) + 8 * (r >> 2)] : 0.0f; };
        const auto no_delta = [](int) { return 0.0f; };
        // pads among the keys are other lanes' and are not stored
        if (p0 >= steps.all && p0 < steps.all_end)
          score_gradients<T, kCap>(a, s, dp, held, row_lse, no_delta, [](int) { return true; }, p16, dz16);
        else
          score_gradients<T, kCap>(a, s, dp, held, row_lse, no_delta,
                                   [&](int r) { return seen(p0 + 4 * h + (r & 3) + 8 * (r >> 2)); }, p16, dz16);
        __builtin_amdgcn_sched_barrier(0);
        U32x4 f[kDim / 32][2];
        read_columns<kDim, queries + kTile>(column_at[0] + skip, column_at[1] + skip, f);
        add_columns<T, kDim>(dv, f, p16);
        read_columns<kDim, queries>(column_at[0] + skip, column_at[1] + skip, f);
        add_columns<T, kDim>(dk, f, dz16);
      }
    };
    if (!walk.done()) load(0);
    while (!walk.done()) {
      turn(Place<0>{}, 0, 2 * kTile);
      if (walk.done()) break;
      turn(Place<2 * kTile>{}, 1, 0);
    }
    __syncthreads();
  }
  const float dv_factor = T::kNarrow ? 1.0f / kProbabilityScale : 1.0f;
  if (a.key_parts > 1) {
    store_sums<kDim>(a, place.part, 0, dk, a.scale / held, stream, place.kv_head, own_keys, own_valid);
    store_sums<kDim>(a, place.part, 1, dv, dv_factor, stream, place.kv_head, own_keys, own_valid);
    return;
  }
  // 32 rows of the results for each wave
  char* own = s_tiles + wave * kTile;
  store_rows<T, kDim>(own, dk, a.scale / held, const_cast<char*>(head_rows(a.dk, stream, place.kv_head)),
                      2 * a.dk.row, own_keys, own_valid, a.dim);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  store_rows<T, kDim>(own, dv, dv_factor, const_cast<char*>(head_rows(a.dv, stream, place.kv_head)), 2 * a.dv.row,
                      own_keys, own_valid, a.dim);
}

// Sums of the parts, in order, rounded once: 16 threads a row of a head, eight elements
// a thread.  Memory: 8192 tokens, 8 key heads of 128, four parts 70 us (4.3 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  if (a.plan.header[kAttnCode] != THD_OK) return;
  const int32_t word = threadIdx.x & 15, head = blockIdx.y;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (row >= a.total || 8 * word >= a.dim) return;
  for (int which = 0; which < 2; ++which) {
    float sum[8] = {};
    for (int32_t part = 0; part < a.key_parts; ++part) {
      const float4* from = reinterpret_cast<const float4*>(partial_sums(a, part, which, row, head) + 8 * word);
      const float4 x = from[0], y = from[1];
      sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
      sum[4] += y.x, sum[5] += y.y, sum[6] += y.z, sum[7] += y.w;
    }
    const AttnTensor& t = which ? a.dv : a.dk;
    *reinterpret_cast<U32x4*>(const_cast<char*>(head_rows(t, row, head)) + 16 * word) =
        U32x4{T::pack(sum[0], sum[1]), T::pack(sum[2], sum[3]), T::pack(sum[4], sum[5]), T::pack(sum[6], sum[7])};
  }
}

template <typename T, int kDim>
hipError_t dq(const AttnArgs& a, hipStream_t stream) {
  const int32_t units = a.plan.max_query_tiles * a.kv_heads;
  const dim3 grid((units + 7) / 8 * 8 * (a.group / a.tile_heads));
  if (a.cap > 0.0f) attn_dq_kernel<T, kDim, true><<<grid, 256, 0, stream>>>(a);
  else attn_dq_kernel<T, kDim, false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T, int kDim>
hipError_t dkv(const AttnArgs& a, hipStream_t stream) {
  const int32_t units = a.plan.max_key_tiles * a.kv_heads;
  const dim3 grid((units + 7) / 8 * 8 * a.key_parts);
  if (a.cap > 0.0f) attn_dkv_kernel<T, kDim, true><<<grid, 256, 0, stream>>>(a);
  else attn_dkv_kernel<T, kDim, false><<<grid, 256, 0, stream>>>(a);
  if (a.key_parts > 1) {
    const dim3 rows(static_cast<uint32_t>((static_cast<int64_t>(a.total) + 15) / 16), a.kv_heads);
    attn_join_kernel<T><<<rows, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t dq(const AttnArgs& a, hipStream_t stream) {
  return a.dim <= 64 ? dq<T, 64>(a, stream) : a.dim <= 96 ? dq<T, 96>(a, stream) : dq<T, 128>(a, stream);
}
template <typename T>
hipError_t dkv(const AttnArgs& a, hipStream_t stream) {
  return a.dim <= 64 ? dkv<T, 64>(a, stream) : a.dim <= 96 ? dkv<T, 96>(a, stream) : dkv<T, 128>(a, stream);
}

}  // namespace

hipError_t launch_attn_delta(const AttnArgs& a, hipStream_t stream) {
  const int32_t query_blocks = a.plan.max_query_tiles * (a.heads / a.tile_heads);
  const int32_t blocks = query_blocks + a.plan.max_key_tiles * a.kv_heads;
  attn_delta_kernel<AttnFp16><<<blocks, 256, 0, stream>>>(a, query_blocks);
  return hipGetLastError();
}

hipError_t launch_attn_dq(const AttnArgs& a, hipStream_t stream) {
  return a.dtype == THD_BF16 ? dq<AttnBf16>(a, stream) : dq<AttnFp16>(a, stream);
}

hipError_t launch_attn_dkv(const AttnArgs& a, hipStream_t stream) {
  return a.dtype == THD_BF16 ? dkv<AttnBf16>(a, stream) : dkv<AttnFp16>(a, stream);
}

}  // namespace thdcp
