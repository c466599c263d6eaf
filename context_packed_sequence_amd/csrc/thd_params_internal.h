// Internal declarations of the embedding table's and the gradients' operators.
// Not part of the public ABI (that is include/thd_params.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "thd_internal.h"
#include "thd_params.h"

namespace thdcp {

// ---- embedding --------------------------------------------------------------

struct EmbedArgs {
  const int64_t* ids;
  const uint8_t* mask;       // or null
  const void* table;         // lookup
  void* out;
  const void* drows;         // gradient
  void* dtable;
  int64_t in_stride, out_stride;  // elements
  int32_t rows, vocab, width;
  int32_t dtype, out_dtype;
  int32_t accumulate;
  float scale;
  int32_t* status;           // or null
  int32_t scan;              // 1: a workgroup of its own writes the status
};

// A row of the stream and the token it holds; key == vocab: none.
struct TokenRow {
  uint32_t key, row;
};

constexpr int32_t kSortBlock = 8192;    // rows that one workgroup sorts by itself
constexpr int32_t kSortTile = 4096;     // rows of a workgroup's turn where several sort
constexpr int32_t kSortBlocks = 256;    // at most
constexpr int32_t kSortBins = 512;

struct EmbedSort {
  TokenRow* a;               // [rows], sorted at the end
  TokenRow* b;               // [rows], null for one workgroup
  int32_t* counts;           // [blocks][kSortBins]
  int32_t blocks, turns;     // turns of kSortTile rows in a workgroup
  int32_t passes, bits;      // digits of `bits` bits
  float* partial;            // [units][2][partial_width]
  int32_t partial_width;     // width in whole words of any type
  int32_t unit;              // sorted rows of a unit
  int32_t units;
};

EmbedSort embed_sort(int64_t rows, int64_t vocab, int64_t width);

hipError_t launch_embedding(const EmbedArgs& a, hipStream_t stream);
hipError_t launch_embedding_sort(const EmbedArgs& a, const EmbedSort& s, hipStream_t stream);
hipError_t launch_embedding_sums(const EmbedArgs& a, const EmbedSort& s, hipStream_t stream);

// ---- gradients --------------------------------------------------------------

constexpr int32_t kListTensors = 96;          // tensors of one launch, passed by value
constexpr int32_t kNormBlocks = 2048;         // workgroups, and partial sums, of one launch
constexpr int32_t kGradChunkBytes = 32768;    // of a tensor's elements in a workgroup's turn

struct GradEntry {
  const void* in;
  void* out;
  int32_t tail;                               // elements of the last chunk
  int32_t types;                              // in, out << 8
};
struct GradList {
  GradEntry entry[kListTensors];
  int32_t first[kListTensors + 1];            // chunks of the tensors before
  int32_t tensors;
};
static_assert(sizeof(GradList) < 3584, "a launch takes 4 KiB of arguments");

struct ClipArgs {
  double scale, max_norm;
  const double* partial;     // sums of squares
  int32_t partials;
  const float* norm_in;      // or null: from the partial sums
  float* norm;               // or null
  int32_t* status;           // or null
};

// last: the tensors whose chunks are scaled first, as far as caches keep them.
hipError_t launch_norm(const GradList& l, double* partial, int32_t blocks, bool last, hipStream_t stream);
hipError_t launch_norm_finish(const ClipArgs& c, hipStream_t stream);
hipError_t launch_clip(const GradList& l, const ClipArgs& c, int32_t blocks, bool finish, hipStream_t stream);

}  // namespace thdcp
