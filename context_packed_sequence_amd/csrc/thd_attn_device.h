// Device code shared by the attention kernels: matrix fragments, tiles in LDS
// and the part of a document that a row sees.
//
// Fragments of v_mfma_f32_32x32x16 (lane l, h = l / 32, c = l mod 32):
//   A [32 rows][16]: lane holds row c, columns 8 h .. 8 h + 7
//   B [16][32 cols]: lane holds column c, rows 8 h .. 8 h + 7
//   C [32][32]:      lane holds column c, register r row (r & 3) + 8 (r >> 2) + 4 h
// A product's C is rounded and becomes the next product's B without leaving its
// lane: the sum over the shared index may run in any order, so register 8 j + e
// of C is called element e of B's block j, and the other operand is read in the
// same order: elements 0..3 from rows 16 j + 4 h.., 4..7 from 16 j + 8 + 4 h...
// ds_read_b64_tr_b16 gives just that: of 4 rows of 16 elements that 16 lanes
// point to, lane i gets column i.
//
// LDS tiles are rows of 64 or 128 16-bit elements in 16-byte words, word w of row r at
// place w ^ f(r).  f gives any 16 rows different places (reads of one word of 32
// rows, as A needs) and any 4 rows different quarters of the banks (transposing
// reads: 64 bytes of each of 4 rows), so neither read has bank conflicts.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "thd_attn_internal.h"
#include "thd_device.h"

namespace thdcp {

typedef unsigned int U32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int U32x2 __attribute__((ext_vector_type(2)));
typedef float F32x16 __attribute__((ext_vector_type(16)));
typedef float F32x2 __attribute__((ext_vector_type(2)));
typedef short I16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 Bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 Bf16p __attribute__((ext_vector_type(2)));
typedef _Float16 F16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 F16p __attribute__((ext_vector_type(2)));

constexpr float kAttnLog2e = 1.4426950408889634f;
constexpr float kAttnLn2 = 0.6931471805599453f;
constexpr float kAttnInf = __builtin_huge_valf();

struct AttnBf16 {
  static __device__ __forceinline__ F32x16 mfma(U32x4 a, U32x4 b, F32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Bf16x8, a), __builtin_bit_cast(Bf16x8, b), c, 0,
                                                   0, 0);
  }
  // rounded to nearest even
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const F32x2 f = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, Bf16p));
  }
  static __device__ __forceinline__ float low(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
  static __device__ __forceinline__ float high(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }
  static constexpr bool kNarrow = false;
};

struct AttnFp16 {
  static __device__ __forceinline__ F32x16 mfma(U32x4 a, U32x4 b, F32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(F16x8, a), __builtin_bit_cast(F16x8, b), c, 0, 0,
                                                  0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const F32x2 f = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, F16p));
  }
  static __device__ __forceinline__ float low(uint32_t w) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w)));
  }
  static __device__ __forceinline__ float high(uint32_t w) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(w >> 16)));
  }
  // 5 exponent bits: gradients of scores are held scaled by a power of two
  static constexpr bool kNarrow = true;
};

__device__ __forceinline__ F32x16 zero16() {
  F32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}

__device__ __forceinline__ float attn_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Capped scores in powers of two: s = cap log2(e) tanh(scale s / cap), element by
// element.  Scores are mostly well below their cap, and up to half of it s times an even
// polynomial, whose coefficients hold all the factors, takes six instructions an element;
// it also keeps its relative precision near 0, where 1 - 2 / (1 + e^(2x)) is off by up to
// 2^-23 of the cap.  Where a lane's score is larger, or the factors' powers do not fit 32
// bits, each element takes one of the two by its size.
__device__ __forceinline__ void attn_capped(const AttnArgs& a, F32x16& s) {
  float top = fmaxf(fabsf(s[0]), fabsf(s[1]));
#pragma unroll
  for (int r = 2; r < 16; r += 2) top = fmaxf(fmaxf(top, fabsf(s[r])), fabsf(s[r + 1]));
  if (!__any(top > a.curve_limit)) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float u = s[r] * s[r];
      float p = fmaf(u, a.curve[4], a.curve[3]);
      p = fmaf(u, p, a.curve[2]);
      p = fmaf(u, p, a.curve[1]);
      p = fmaf(u, p, a.curve[0]);
      s[r] *= p;
    }
    return;
  }
  const float most = a.cap * kAttnLog2e, in = a.scale / a.cap, slope = a.scale * kAttnLog2e;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    if (r % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // few registers at a time
    const float x = s[r] * in, u = x * x;
    float p = fmaf(u, kAttnTanh[4], kAttnTanh[3]);
    p = fmaf(u, p, kAttnTanh[2]);
    p = fmaf(u, p, kAttnTanh[1]);
    p = fmaf(u, p, 1.0f);
    const float large = fmaf(-2.0f * most, __builtin_amdgcn_rcpf(1.0f + attn_exp2(x * (2.0f * kAttnLog2e))), most);
    s[r] = fabsf(x) <= 0.5f ? s[r] * slope * p : large;
  }
}

// Value of lane l ^ 32, combined.
__device__ __forceinline__ float max_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])),
               __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
}
__device__ __forceinline__ float add_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, static_cast<uint32_t>(r[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(r[1]));
}

// Heads of up to 64, 96 or 128 elements (kDim) have kernels of their own; a row in LDS
// has room for 64 or 128.
template <int kDim>
constexpr int kRowBytes = kDim <= 64 ? 128 : 256;

template <int kDim>
__device__ __forceinline__ int32_t lds_swizzle(int32_t row) {
  if constexpr (kRowBytes<kDim> == 256) return ((row & 3) << 2) | ((row >> 2) & 3);
  else return ((row & 2) << 1) | ((row >> 2) & 3);  // two rows share a line of banks
}

// Byte address in a tile of word w of a row.
template <int kDim>
__device__ __forceinline__ int32_t lds_word(int32_t row, int32_t w) {
  return row * kRowBytes<kDim> + ((w ^ lds_swizzle<kDim>(row)) << 4);
}

__device__ __forceinline__ U32x4 lds_read(const char* tile, int32_t at) {
  return *reinterpret_cast<const U32x4*>(tile + at);
}

// Where a lane points to for a transposing read of rows 0..7 (second 0) or 8..15
// (second 1) of a tile, which are the summed index (in the order above), and columns
// 32 t .. 32 t + 31, the 32 rows of A.
template <int kDim>
__device__ __forceinline__ int32_t transposed_at(int32_t t, int32_t second) {
  const int32_t l = threadIdx.x & 63, i = l & 15;
  const int32_t row = 4 * (l >> 5) + (i >> 2) + 8 * second;
  const int32_t col = 32 * t + 16 * ((l >> 4) & 1) + 4 * (i & 3);
  return lds_word<kDim>(row, col >> 3) + 2 * (col & 7);
}
// A's fragments for 32 rows of a tile from kFrom on, all columns: [t][j] is columns
// 32 t .. 32 t + 31 of rows 16 j .. 16 j + 15.  `first` and `second` are the lane's LDS
// addresses transposed_at(0, 0) and (0, 1); other columns differ in single bits.  One
// block of reads with its wait: the compiler would wait for every load from memory to
// LDS before a transposing read, also for those of the tiles to come.
template <int kDim, int kFrom>
__device__ __forceinline__ void read_columns(uint32_t first, uint32_t second, U32x4 (&f)[kDim / 32][2]) {
  U32x2 x[kDim / 32][2], y[kDim / 32][2];
  if constexpr (kDim == 128) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %16 offset:%24\n"
        "ds_read_b64_tr_b16 %1, %20 offset:%24\n"
        "ds_read_b64_tr_b16 %2, %16 offset:%25\n"
        "ds_read_b64_tr_b16 %3, %20 offset:%25\n"
        "ds_read_b64_tr_b16 %4, %17 offset:%24\n"
        "ds_read_b64_tr_b16 %5, %21 offset:%24\n"
        "ds_read_b64_tr_b16 %6, %17 offset:%25\n"
        "ds_read_b64_tr_b16 %7, %21 offset:%25\n"
        "ds_read_b64_tr_b16 %8, %18 offset:%24\n"
        "ds_read_b64_tr_b16 %9, %22 offset:%24\n"
        "ds_read_b64_tr_b16 %10, %18 offset:%25\n"
        "ds_read_b64_tr_b16 %11, %22 offset:%25\n"
        "ds_read_b64_tr_b16 %12, %19 offset:%24\n"
        "ds_read_b64_tr_b16 %13, %23 offset:%24\n"
        "ds_read_b64_tr_b16 %14, %19 offset:%25\n"
        "ds_read_b64_tr_b16 %15, %23 offset:%25\n"
        "s_waitcnt lgkmcnt(0)\n"
        : "=&v"(x[0][0]), "=&v"(y[0][0]), "=&v"(x[0][1]), "=&v"(y[0][1]), "=&v"(x[1][0]), "=&v"(y[1][0]),
          "=&v"(x[1][1]), "=&v"(y[1][1]), "=&v"(x[2][0]), "=&v"(y[2][0]), "=&v"(x[2][1]), "=&v"(y[2][1]),
          "=&v"(x[3][0]), "=&v"(y[3][0]), "=&v"(x[3][1]), "=&v"(y[3][1])
        : "v"(first), "v"(first ^ 64), "v"(first ^ 128), "v"(first ^ 192), "v"(second), "v"(second ^ 64),
          "v"(second ^ 128), "v"(second ^ 192), "i"(kFrom), "i"(kFrom + 16 * kRowBytes<kDim>)
        : "memory");
  } else if constexpr (kDim == 96) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %12 offset:%18\n"
        "ds_read_b64_tr_b16 %1, %15 offset:%18\n"
        "ds_read_b64_tr_b16 %2, %12 offset:%19\n"
        "ds_read_b64_tr_b16 %3, %15 offset:%19\n"
        "ds_read_b64_tr_b16 %4, %13 offset:%18\n"
        "ds_read_b64_tr_b16 %5, %16 offset:%18\n"
        "ds_read_b64_tr_b16 %6, %13 offset:%19\n"
        "ds_read_b64_tr_b16 %7, %16 offset:%19\n"
        "ds_read_b64_tr_b16 %8, %14 offset:%18\n"
        "ds_read_b64_tr_b16 %9, %17 offset:%18\n"
        "ds_read_b64_tr_b16 %10, %14 offset:%19\n"
        "ds_read_b64_tr_b16 %11, %17 offset:%19\n"
        "s_waitcnt lgkmcnt(0)\n"
        : "=&v"(x[0][0]), "=&v"(y[0][0]), "=&v"(x[0][1]), "=&v"(y[0][1]), "=&v"(x[1][0]), "=&v"(y[1][0]),
          "=&v"(x[1][1]), "=&v"(y[1][1]), "=&v"(x[2][0]), "=&v"(y[2][0]), "=&v"(x[2][1]), "=&v"(y[2][1])
        : "v"(first), "v"(first ^ 64), "v"(first ^ 128), "v"(second), "v"(second ^ 64), "v"(second ^ 128), "i"(kFrom),
          "i"(kFrom + 16 * kRowBytes<kDim>)
        : "memory");
  } else {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8 offset:%12\n"
        "ds_read_b64_tr_b16 %1, %10 offset:%12\n"
        "ds_read_b64_tr_b16 %2, %8 offset:%13\n"
        "ds_read_b64_tr_b16 %3, %10 offset:%13\n"
        "ds_read_b64_tr_b16 %4, %9 offset:%12\n"
        "ds_read_b64_tr_b16 %5, %11 offset:%12\n"
        "ds_read_b64_tr_b16 %6, %9 offset:%13\n"
        "ds_read_b64_tr_b16 %7, %11 offset:%13\n"
        "s_waitcnt lgkmcnt(0)\n"
        : "=&v"(x[0][0]), "=&v"(y[0][0]), "=&v"(x[0][1]), "=&v"(y[0][1]), "=&v"(x[1][0]), "=&v"(y[1][0]),
          "=&v"(x[1][1]), "=&v"(y[1][1])
        : "v"(first), "v"(first ^ 64), "v"(second), "v"(second ^ 64), "i"(kFrom), "i"(kFrom + 16 * kRowBytes<kDim>)
        : "memory");
  }
#pragma unroll
  for (int t = 0; t < kDim / 32; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) f[t][j] = U32x4{x[t][j][0], x[t][j][1], y[t][j][0], y[t][j][1]};
}

// A place in LDS known when the code is compiled: it goes into reads' offset fields.
template <int kAt>
using Place = std::integral_constant<int, kAt>;

__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}

// Rows [0, valid) of one head, from `base` on, behind a buffer resource of
// exactly their size: a word past the last row, or past the head's elements, is
// read as zeros.  The resource is built anew for each tile, so that offsets stay
// within 32 bits however long the stream is.
struct RowsRead {
  __amdgpu_buffer_rsrc_t rsrc;
  int32_t stride;  // bytes
  __device__ __forceinline__ RowsRead(const void* base, int32_t stride_bytes, int32_t valid, int32_t dim)
      : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0,
                                               valid > 0 ? (valid - 1) * stride_bytes + 2 * dim : 0, kBufferWord3)),
        stride(stride_bytes) {}
  __device__ __forceinline__ int32_t at(int32_t row, int32_t w, int32_t dim) const {
    return 8 * w < dim ? row * stride + 16 * w : static_cast<int32_t>(0x80000000u);
  }
  __device__ __forceinline__ U32x4 load(int32_t row, int32_t w, int32_t dim) const {
    return __builtin_bit_cast(U32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at(row, w, dim), 0, 0));
  }
};

// First address of a head's rows, uniform over the workgroup.
__device__ __forceinline__ const char* head_rows(const AttnTensor& t, int64_t row, int32_t head) {
  return static_cast<const char*>(t.data) + 2 * (row * t.row + static_cast<int64_t>(head) * t.head);
}

// Moves kRows rows into an LDS tile, 16 bytes a lane and turn straight from
// memory (no registers in between); the caller waits (lds_arrived) before the
// barrier after which the tile is read.
template <int kDim, int kRows = kAttnStep>
__device__ __forceinline__ void load_tile(char* tile, const RowsRead& r, int32_t dim) {
  constexpr int kWords = kRowBytes<kDim> / 16;
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int j = 0; j < kRows * kWords / 256; ++j) {
    const int32_t s = j * 256 + threadIdx.x;
    const int32_t row = s / kWords;
    const int32_t w = (s % kWords) ^ lds_swizzle<kDim>(row);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r.rsrc,
        reinterpret_cast<__attribute__((address_space(3))) void*>(
            reinterpret_cast<uintptr_t>(tile + (j * 256 + wave * 64) * 16)),
        16, r.at(row, w, dim), 0, 0, 0);
  }
}
__device__ __forceinline__ void lds_arrived() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// End, within a document, of the positions that a window of one that ends at `end`
// reaches (in 32 bits without a sign: both are below 2^31).
__device__ __forceinline__ int32_t window_end(const AttnArgs& a, int32_t end, int32_t real) {
  const uint32_t to = static_cast<uint32_t>(end) + static_cast<uint32_t>(a.window) - 1u;
  return static_cast<int32_t>(to < static_cast<uint32_t>(real) ? to : static_cast<uint32_t>(real));
}

// Keys [low, low + span) of its document are what position `pos` sees.
struct Seen {
  int32_t low;
  uint32_t span;
  __device__ __forceinline__ Seen(const AttnArgs& a, int32_t pos, int32_t real) {
    low = a.window ? max(0, pos - a.window + 1) : 0;
    int32_t end = real;
    if (a.causal) end = min(real, pos + 1);
    else if (a.window) end = window_end(a, pos + 1, real);
    span = end > low ? static_cast<uint32_t>(end - low) : 0u;
  }
  __device__ __forceinline__ Seen(int32_t first, uint32_t n) : low(first), span(n) {}
  __device__ __forceinline__ bool operator()(int32_t key) const {
    return static_cast<uint32_t>(key) - static_cast<uint32_t>(low) < span;
  }
};

// Rows that a loop walks through, `step` at a time, from one running address: what a
// step costs beside the loads is a few scalar instructions.
struct RowsWalk {
  const char* at;
  int32_t left;      // rows from `at` on that hold tokens
  int32_t stride;    // bytes
  __device__ __forceinline__ RowsWalk(const AttnTensor& t, int64_t row, int32_t head, int32_t rows)
      : at(head_rows(t, row, head)), left(rows), stride(static_cast<int32_t>(2 * t.row)) {}
  template <int kDim, int kStep>
  __device__ __forceinline__ void load(char* tile, int32_t dim) {
    load_tile<kDim, kStep>(tile, RowsRead(at, stride, min(left, kStep), dim), dim);
    at += static_cast<int64_t>(stride) * kStep;
    left -= kStep;
  }
};

// The steps of 32 keys, numbered by their first key, that positions [p, p + np) see
// something of, and of which they see everything.
struct KeySteps {
  int32_t any, any_end, all, all_end;
  __device__ __forceinline__ KeySteps(const AttnArgs& a, int32_t p, int32_t np, int32_t valid, int32_t real) {
    const int32_t last = p + np - 1;
    any = a.window ? p - a.window - 30 : 0;   // k + 31 > p - window
    all = a.window ? last - a.window + 1 : 0;
    any_end = all_end = 0;
    if (valid <= 0) return;
    any_end = a.causal ? p + valid : a.window ? window_end(a, p + valid, real) : real;
    any_end = min(any_end, real);
    all_end = min(a.causal ? p + 1 : a.window ? window_end(a, p + 1, real) : real, real) - 31;
  }
};

// Tile and heads of workgroup b, which runs on XCD b mod 8: the workgroups of a group
// read the same keys, and stay on one XCD one after the other; tiles of a key head are
// dealt out so that, with 8 key heads, each XCD keeps to one of them.  `parts`:
// workgroups of a group.
struct AttnPlace {
  int32_t tile, kv_head, part;
  __device__ __forceinline__ AttnPlace(int32_t b, int32_t kv_heads, int32_t parts) {
    const int32_t j = b >> 3;
    const int32_t unit = (j / parts) * 8 + (b & 7);
    tile = unit / kv_heads;
    kv_head = unit % kv_heads;
    part = j % parts;
  }
};

// A wave's 32 query rows of a workgroup's tile.
struct WaveRows {
  int32_t head, first, rows, valid;  // first: within the tile
  __device__ __forceinline__ WaveRows(const AttnArgs& a, const QueryTile& tile, const AttnPlace& place, int32_t wave) {
    head = place.kv_head * a.group + place.part * a.tile_heads + wave % a.tile_heads;
    first = 32 * (wave / a.tile_heads);
    rows = min(32, max(0, tile.rows - first));
    valid = min(32, max(0, tile.valid - first));
  }
};

// Four waves' accumulators [kDim][32 rows] (rows are lanes) as rows of 16-bit
// elements, through LDS so that whole lines are stored; row r of the wave is
// multiplied by `factor` of its lane.  Rows from `valid` on are zero; rows from
// `rows` on, and columns from dim on, are not stored.
template <typename T, int kDim>
__device__ __forceinline__ void store_rows(char* lds, const F32x16 (&acc)[kDim / 32], float factor, char* base,
                                           int64_t stride_bytes, int32_t rows, int32_t valid, int32_t dim) {
  const int32_t l = threadIdx.x & 63, c = l & 31, h = l >> 5;
  const float f = c < valid ? factor : 0.0f;
#pragma unroll
  for (int t = 0; t < kDim / 32; ++t) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      U32x2 w;
      w[0] = T::pack(acc[t][4 * g] * f, acc[t][4 * g + 1] * f);
      w[1] = T::pack(acc[t][4 * g + 2] * f, acc[t][4 * g + 3] * f);
      if (c >= valid) w[0] = w[1] = 0u;  // whatever the pad's lane holds
      *reinterpret_cast<U32x2*>(lds + lds_word<kDim>(c, 4 * t + g) + 8 * h) = w;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  constexpr int kWords = kRowBytes<kDim> / 16;
#pragma unroll
  for (int j = 0; j < kWords / 2; ++j) {
    const int32_t s = j * 64 + l;
    const int32_t row = s / kWords, w = (s % kWords) ^ lds_swizzle<kDim>(row);
    const U32x4 x = lds_read(lds, s * 16);
    if (row < rows && 8 * w < dim) *reinterpret_cast<U32x4*>(base + row * stride_bytes + 16 * w) = x;
  }
}

}  // namespace thdcp
