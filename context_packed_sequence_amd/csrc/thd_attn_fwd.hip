// Attention inside documents: out = softmax(z) v and its log-sum-exp.
//
// One pass over the keys with the running maximum and sum of the softmax.  A
// workgroup owns 128 query rows, of one head or the same rows of the heads of a
// group, a wave 32 of them, and the four waves walk through the keys together,
// moved straight from memory to LDS while those before are worked on.  Scores are
// formed transposed, S^T = K Q^T, 32 keys at a time, so that a lane holds one query
// (its column) and 16 of the keys: the softmax needs one exchange between the two
// halves of a wave, the output's rescaling is by a lane's own factor, and the
// probabilities, rounded to the tensors' type as a factor of the matrix product (at
// most half a step of each, while their sum is held in 32 bits), are the second
// product's operand as they lie (O^T += V^T P^T, V read transposed).
//
// Probabilities are held relative to a reference of their row, and the output is
// rescaled only when some row's maximum grew by more than 2^8 beyond it: numbers up to
// 256 lose nothing in 32-bit sums, nor rounded to bf16.  fp16 has few exponents below 1:
// there the reference stands 2^9 below the maximum it was taken from, and may be
// outgrown by 2^6 more, which stays below the type's end.  Probabilities down to 2^-23 of
// that maximum keep all their bits, those down to 2^-34 some (without the 2^9, 2^-14 and
// 2^-25: a key 16 e-folds above all others and of value 0 put its row off by 6 %).
// 8192 tokens, 32 heads of 128 over 8, causal, fp16: 566 us against 563 without, 575 with
// 2^13 and 2^2.
//
// Long documents are bound by the matrix units and the vector units together, which hardly
// overlap: one of 8192 tokens, causal, 32 heads over 8, takes 524 us with heads of 128 (1050
// TFLOP/s; the matrix units busy for 57 % of the cycles, vector instructions for 47 %, LDS
// for 28 %), 429 with 96, 311 with 64, and 639 with 128 and a cap.  A large matrix product
// of the library reaches 1415 TFLOP/s.  Short ones are bound by starting and ending tiles
// (32768 tokens of documents of 64 to 1024: ten steps a tile, matrix units busy for 34 %),
// few long ones by the chain of a tile's steps (93 steps of 12 heads of 72: 0.95 us each).
#include "thd_attn_device.h"

namespace thdcp {

namespace {

// In powers of two: how far above a row's reference the maximum stands when it is taken,
// and how much further it may grow.
template <typename T>
constexpr float kLift = T::kNarrow ? 9.0f : 0.0f;
template <typename T>
constexpr float kGrowth = T::kNarrow ? 6.0f : 8.0f;
// Larger maxima have no bits to stand kLift above anything.
constexpr float kLiftUpTo = 0x1p22f;

template <typename T, int kDim, bool kCap>
struct ForwardWave {
  U32x4 q[kDim / 16];        // B: 32 queries
  F32x16 o[kDim / 32];       // [dim][query]
  float top = -kAttnInf;     // reference of the row's exponents, in powers of two
  float sum = 0.0f;          // of this lane's keys
  int32_t key_at;            // this lane's place in a tile
  uint32_t value_at[2];

  __device__ __forceinline__ explicit ForwardWave(const char* lds) {
    const int32_t l = threadIdx.x & 63;
    key_at = lds_word<kDim>(l & 31, l >> 5);
    value_at[0] = lds_address(lds) + transposed_at<kDim>(0, 0);
    value_at[1] = lds_address(lds) + transposed_at<kDim>(0, 1);
#pragma unroll
    for (int t = 0; t < kDim / 32; ++t) o[t] = zero16();
  }

  // Keys key0 .. key0 + 31, whose rows are at kKeys + skip in LDS and their values' at
  // kValues + skip; `partly`: the rows do not see all of them.
  template <int kKeys, int kValues>
  __device__ __forceinline__ void step(const AttnArgs& a, const char* lds, int32_t skip, int32_t key0, bool partly,
                                       const Seen& seen) {
    const int32_t h = (threadIdx.x & 63) >> 5;
    // places differ in single bits from word to word: one address, hidden from the
    // compiler so that it does not keep all of them in registers
    int32_t row = key_at;
    asm volatile("" : "+v"(row));
    F32x16 s = zero16();
    constexpr int kRead = kDim % 64 == 0 ? 4 : 3;
#pragma unroll
    for (int i0 = 0; i0 < kDim / 16; i0 += kRead) {
      U32x4 k[kRead];
#pragma unroll
      for (int i = 0; i < kRead; ++i) k[i] = lds_read(lds + skip + (row ^ (32 * (i0 + i))), kKeys);
      __builtin_amdgcn_sched_barrier(0);  // all on their way before the first is waited for
#pragma unroll
      for (int i = 0; i < kRead; ++i) s = T::mfma(k[i], q[i0 + i], s);
    }
    // scores in powers of two: s factor
    const float factor = kCap ? 1.0f : a.scale * kAttnLog2e;
    if constexpr (kCap) attn_capped(a, s);
    if (partly) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = seen(key0 + 4 * h + (r & 3) + 8 * (r >> 2)) ? s[r] : -kAttnInf;
    }
    float m = fmaxf(s[0], s[1]);
#pragma unroll
    for (int r = 2; r < 16; r += 2) m = fmaxf(fmaxf(m, s[r]), s[r + 1]);
    m = max_halves(m) * factor;
    if (__any(m - top > kLift<T> + kGrowth<T>)) {  // a difference: exact, however large they are
      const float to = fmaxf(top, m - (fabsf(m) < kLiftUpTo ? kLift<T> : 0.0f));
      const float shrink = to == -kAttnInf ? 1.0f : attn_exp2(top - to);
      top = to;
      sum *= shrink;
#pragma unroll
      for (int t = 0; t < kDim / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[t][r] *= shrink;
    }
    const float base = top == -kAttnInf ? 0.0f : top;
    U32x4 p[2];
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      const float x = attn_exp2(fmaf(s[r], factor, -base));
      const float y = attn_exp2(fmaf(s[r + 1], factor, -base));
      sum += x + y;
      p[r >> 3][(r & 7) >> 1] = T::pack(x, y);
    }
    U32x4 v[kDim / 32][2];
    read_columns<kDim, kValues>(value_at[0] + skip, value_at[1] + skip, v);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < kDim / 32; ++t) o[t] = T::mfma(v[t][j], p[j], o[t]);
  }
};

// Three waves a SIMD, one computing probabilities while another multiplies.  With heads
// above 64 that leaves room for 32 keys at a time (64 and two waves: 8192 tokens as above
// 553 us against 534, 32768 tokens of short documents 320 against 302; but a share of 1048
// workgroups, which fill two waves' places twice over, 1090 against 1145); smaller rows
// take 64, and half the barriers.
template <typename T, int kDim, bool kCap>
__global__ __launch_bounds__(256, 3) void attn_forward_kernel(AttnArgs a) {
  constexpr int kStep = kDim == 64 ? 64 : 32;
  constexpr int kTile = kStep * kRowBytes<kDim>;  // bytes
  __shared__ __attribute__((aligned(16))) char s_tiles[4 * kTile];  // keys, values, and both again
  const AttnPlace place(blockIdx.x, a.kv_heads, a.group / a.tile_heads);
  if (place.tile >= a.plan.max_query_tiles) return;
  const QueryTile tile = a.plan.query_tiles[place.tile];
  if (tile.rows == 0) return;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t l = threadIdx.x & 63, c = l & 31;
  const WaveRows own(a, tile, place, wave);
  const int32_t pos = tile.pos + own.first;

  ForwardWave<T, kDim, kCap> w(s_tiles);
  if (tile.valid > 0) {
    const RowsRead queries(head_rows(a.q, tile.row + own.first, own.head), static_cast<int32_t>(2 * a.q.row),
                           own.valid, a.dim);
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) w.q[i] = queries.load(c, 2 * i + (l >> 5), a.dim);

    const Seen first(a, tile.pos, tile.real), last(a, tile.pos + tile.valid - 1, tile.real);
    const int32_t end = last.low + static_cast<int32_t>(last.span);
    int32_t key = first.low & ~(kStep - 1);
    const Seen seen(a, pos + c, tile.real);
    RowsWalk keys(a.k, static_cast<int64_t>(tile.doc) + key, place.kv_head, tile.real - key);
    RowsWalk values(a.v, static_cast<int64_t>(tile.doc) + key, place.kv_head, tile.real - key);
    const KeySteps steps(a, pos, 32, own.valid, tile.real);
    const auto load = [&](int32_t to) {
      keys.load<kDim, kStep>(s_tiles + to, a.dim);
      values.load<kDim, kStep>(s_tiles + to + kTile, a.dim);
    };
    const auto turn = [&](auto now, int32_t next) {
      lds_arrived();
      __syncthreads();  // the tile is there, and nobody reads the one before
      if (key + kStep < end) load(next);
#pragma unroll
      for (int b = 0; b < kStep / 32; ++b) {
        const int32_t k0 = key + 32 * b;
        if (k0 >= steps.any && k0 < steps.any_end)
          w.template step<now, now + kTile>(a, s_tiles, 32 * b * kRowBytes<kDim>, k0, k0 < steps.all || k0 >= steps.all_end,
                                            seen);
      }
      key += kStep;
    };
    load(0);
    while (key < end) {
      turn(Place<0>{}, 2 * kTile);
      if (key >= end) break;
      turn(Place<2 * kTile>{}, 0);
    }
    __syncthreads();
  }
  const float sum = add_halves(w.sum);
  const float inverse = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // NaN stays
  store_rows<T, kDim>(s_tiles + wave * kTile, w.o, inverse,
                      const_cast<char*>(head_rows(a.out, tile.row + own.first, own.head)), 2 * a.out.row, own.rows,
                      own.valid, a.dim);
  if (l < own.rows)
    a.lse[static_cast<int64_t>(own.head) * a.rows + tile.row + own.first + l] =
        l < own.valid ? (w.top + __builtin_amdgcn_logf(sum)) * kAttnLn2 : -kAttnInf;
}

template <typename T, int kDim>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  const int32_t units = a.plan.max_query_tiles * a.kv_heads;
  const dim3 grid((units + 7) / 8 * 8 * (a.group / a.tile_heads));
  if (a.cap > 0.0f) attn_forward_kernel<T, kDim, true><<<grid, 256, 0, stream>>>(a);
  else attn_forward_kernel<T, kDim, false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  return a.dim <= 64 ? launch<T, 64>(a, stream) : a.dim <= 96 ? launch<T, 96>(a, stream) : launch<T, 128>(a, stream);
}

}  // namespace

hipError_t launch_attn_forward(const AttnArgs& a, hipStream_t stream) {
  return a.dtype == THD_BF16 ? launch<AttnBf16>(a, stream) : launch<AttnFp16>(a, stream);
}

}  // namespace thdcp
