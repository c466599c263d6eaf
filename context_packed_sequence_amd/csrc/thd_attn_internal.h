// Internal declarations of the attention on packed streams.  Not part of the
// public ABI (that is include/thd_attention.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "thd_attention.h"
#include "thd_internal.h"

namespace thdcp {

constexpr int kAttnRows = 128;   // query rows of a workgroup, over all its heads: 32 in each of its 4 waves
constexpr int kAttnKeys = 128;   // keys of a workgroup that computes their gradients
constexpr int kAttnStep = 64;    // keys (or query rows) that a workgroup moves through LDS at a time

// Heads of a group whose queries a workgroup takes together, the same rows of each: its
// waves then walk through the same keys to the same end, and a tile of few rows ends
// nearer to the diagonal and to the document's end (16384 tokens of short documents, 32
// heads over 8: forward 157 -> 123 us, dq 212 -> 173).
constexpr int32_t attn_tile_heads(int32_t group) { return group % 4 == 0 ? 4 : group % 2 == 0 ? 2 : 1; }

// tanh(x) / x on [-1/2, 1/2] as a polynomial in x^2, minimax: off by 1.5e-8 before rounding.
constexpr float kAttnTanh[5] = {1.0f, -0.33333144f, 0.13325879f, -0.05304552f, 0.01724153f};

// Query rows of one workgroup: a run of rows of one document's share.  Rows
// [valid, rows) are pads.
struct QueryTile {
  int32_t row;       // first row of the share
  int32_t rows;      // 1..kAttnRows / tile heads; 0: no tile
  int32_t valid;     // rows that hold tokens
  int32_t pos;       // position in the document of the first row
  int32_t doc;       // stream row of the document's first token
  int32_t real;      // the document's tokens
  int32_t unused[2];
};

// Keys of one workgroup of the key gradients, and where the share holds the
// document's queries: `first` is the share's first row of the document, chunk
// the length of each of its two zigzag chunks (the whole document if cp is 1).
struct KeyTile {
  int32_t key;       // position in the document of the first key
  int32_t keys;      // 1..kAttnKeys; 0: no tile
  int32_t valid;
  int32_t doc;
  int32_t real;
  int32_t first;
  int32_t chunk;
  int32_t unused;
};

// Workspace, written by the plan kernel.
enum AttnHeader : int { kAttnMaxGrad = 0, kAttnMaxValue = 1, kAttnCode = 2, kAttnHeaderWords = 16 };

struct AttnPlan {
  int32_t* header;         // [kAttnHeaderWords]
  int32_t* slot_first;     // [slots + 1] tiles of the slots before
  QueryTile* query_tiles;  // [max_query_tiles], heaviest first, those without rows last
  KeyTile* key_tiles;      // [max_key_tiles], null in the forward pass
  float* delta;            // [heads][rows], backward only
  float* partial;          // [key parts][2][tokens][kv heads][dim], with more than one part
  int32_t max_query_tiles;
  int32_t max_key_tiles;
};

// Elements between rows and heads of a [rows][heads][dim] tensor.
struct AttnTensor {
  void* data;
  int64_t row, head;
};

struct AttnArgs {
  AttnTensor q, k, v, out, dout, dq, dk, dv;
  float* lse;              // [heads][rows]
  const int32_t* cu_padded;
  const int32_t* cu_real;  // or null
  int32_t* status;         // or null
  int32_t n_slots, total, rows;
  int32_t heads, kv_heads, group, dim, dtype;
  int32_t tile_heads;      // heads of a group in a workgroup
  int32_t key_parts;       // workgroups that a group's heads are dealt out over for the key gradients
  int32_t causal, window;  // window 0: none
  int32_t cp, rank;
  float curve[5];          // with a cap: coefficients of the capped scores' polynomial in s^2,
  float curve_limit;       // for |s| up to this; -1: never
  float scale, cap;        // cap 0: none
  AttnPlan plan;
};

hipError_t launch_attn_plan(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_forward(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_delta(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_dq(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attn_dkv(const AttnArgs& a, hipStream_t stream);

}  // namespace thdcp
