// C ABI of the embedding table's and the gradients' operators: host-side
// argument checks and stream-ordered launches.  See include/thd_params.h.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "thd_loss_internal.h"
#include "thd_params_internal.h"

namespace {

int element_bytes(int32_t dtype) {
  switch (dtype) {
    case THD_BF16:
    case THD_FP16: return 2;
    case THD_FP32: return 4;
    default: return 0;
  }
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

struct Range {
  const void* p;
  int64_t bytes;
};

bool meet(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const auto x = reinterpret_cast<uintptr_t>(a.p);
  const auto y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uint64_t>(b.bytes) && y < x + static_cast<uint64_t>(a.bytes);
}

template <size_t N, size_t M>
bool apart(const Range (&outs)[N], const Range (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = i + 1; j < N; ++j)
      if (meet(outs[i], outs[j])) return false;
    for (size_t j = 0; j < M; ++j)
      if (meet(outs[i], ins[j])) return false;
  }
  return true;
}

// Bytes from the first to the last element of a row-major matrix; -1 if the
// stride does not fit.
int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t stride, int64_t element) {
  if (rows == 0) return 0;
  if (stride < cols || stride > (INT64_MAX / 16 - cols) / rows) return -1;
  return ((rows - 1) * stride + cols) * element;
}

bool sizes_ok(int64_t rows, int64_t vocab, int64_t width) {
  if (rows < 0 || rows > INT32_MAX || vocab < 1 || vocab > THD_MAX_VOCAB || width < 1 || width > THD_MAX_WIDTH)
    return false;
  // workgroups of a launch: the rows' (or units') words and the table's rows
  return rows * ((width + 3) / 4) / 256 + vocab < INT32_MAX - 2;
}

struct EmbedLayout {
  thdcp::EmbedSort sort;
  int64_t bytes;
};

EmbedLayout embed_layout(void* workspace, int64_t rows, int64_t vocab, int64_t width) {
  EmbedLayout l{thdcp::embed_sort(rows, vocab, width), 0};
  char* base = static_cast<char*>(workspace);
  const auto take = [&](int64_t n) {
    char* p = base + l.bytes;
    l.bytes += align_up(n, 16);
    return p;
  };
  l.sort.a = reinterpret_cast<thdcp::TokenRow*>(take(rows * static_cast<int64_t>(sizeof(thdcp::TokenRow))));
  if (rows > thdcp::kSortBlock) {
    l.sort.b = reinterpret_cast<thdcp::TokenRow*>(take(rows * static_cast<int64_t>(sizeof(thdcp::TokenRow))));
    l.sort.counts = reinterpret_cast<int32_t*>(take((thdcp::kSortBlocks * (thdcp::kSortBins + 1)) * 4LL));
  }
  l.sort.partial_width = static_cast<int32_t>(align_up(width, 8));
  l.sort.partial = reinterpret_cast<float*>(take(static_cast<int64_t>(l.sort.units) * 2 * l.sort.partial_width * 4));
  return l;
}

bool finite32(double x) { return std::isfinite(static_cast<float>(x)); }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int launched(hipError_t e) { return e == hipSuccess ? THD_OK : THD_ERR_HIP; }

int64_t lists_of(int64_t n_tensors) { return (n_tensors + thdcp::kListTensors - 1) / thdcp::kListTensors; }

int64_t chunks_of(int64_t elements, int32_t dtype) {
  const int64_t per = thdcp::kGradChunkBytes / element_bytes(dtype);
  return elements / per + (elements % per != 0);
}

bool tensors_ok(const void* const* grads, const int64_t* elements, const int32_t* dtypes, int32_t n) {
  if (n < 0 || n > THD_MAX_TENSORS) return false;
  if (n > 0 && (!grads || !elements || !dtypes)) return false;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int es = element_bytes(dtypes[i]);
    if (es == 0 || elements[i] < 0 || elements[i] > INT64_MAX / 64) return false;
    if (elements[i] > 0 && (!grads[i] || !aligned(grads[i], es))) return false;
    if (i % thdcp::kListTensors == 0) chunks = 0;
    chunks += chunks_of(elements[i], dtypes[i]);
    if (chunks > INT32_MAX / 2) return false;
  }
  return true;
}

// Tensors [from, ...) of the call as one launch's list.
thdcp::GradList list_of(const void* const* grads, void* const* outs, const int64_t* elements, const int32_t* dtypes,
                        const int32_t* out_dtypes, int32_t n, int32_t from) {
  thdcp::GradList l{};
  l.tensors = std::min(n - from, thdcp::kListTensors);
  for (int32_t i = 0; i < l.tensors; ++i) {
    const int64_t n = elements[from + i];
    const int64_t chunks = chunks_of(n, dtypes[from + i]);
    const int64_t per = thdcp::kGradChunkBytes / element_bytes(dtypes[from + i]);
    l.entry[i].in = grads[from + i];
    l.entry[i].out = outs ? outs[from + i] : nullptr;
    l.entry[i].tail = static_cast<int32_t>(chunks > 0 ? n - (chunks - 1) * per : 0);
    l.entry[i].types = dtypes[from + i] | (out_dtypes ? out_dtypes[from + i] << 8 : 0);
    l.first[i + 1] = l.first[i] + static_cast<int32_t>(chunks);
  }
  return l;
}

// Workgroups of a list's sums: one partial sum each.
int32_t blocks_of(const thdcp::GradList& l) { return std::min(l.first[l.tensors], thdcp::kNormBlocks); }

// Sums of squares of all tensors; *partials: how many.
int launch_sums(const void* const* grads, const int64_t* elements, const int32_t* dtypes, int32_t n, double* partial,
                int32_t* partials, void* stream) {
  *partials = 0;
  for (int32_t from = 0; from < n; from += thdcp::kListTensors) {
    const thdcp::GradList l = list_of(grads, nullptr, elements, dtypes, nullptr, n, from);
    if (l.first[l.tensors] == 0) continue;
    const int32_t blocks = blocks_of(l);
    const bool last = from + thdcp::kListTensors >= n;
    if (thdcp::launch_norm(l, partial + *partials, blocks, last, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
    *partials += blocks;
  }
  return THD_OK;
}

struct Piece {
  uintptr_t at, end;
  int32_t tensor;
  bool output;
};

// Whether an output meets another output, or a gradient other than the one it
// replaces.  Pieces in order of their addresses: one that starts before the
// furthest end so far meets a piece before it, and of such pairs only a gradient with
// its own output, or two gradients, are allowed.
int outputs_apart(std::vector<Piece>& pieces) {
  std::sort(pieces.begin(), pieces.end(), [](const Piece& a, const Piece& b) {
    return a.at != b.at ? a.at < b.at : a.tensor != b.tensor ? a.tensor < b.tensor : a.output < b.output;
  });
  uintptr_t in_end = 0, out_end = 0;     // furthest end of gradients and of outputs so far
  for (size_t i = 0; i < pieces.size(); ++i) {
    const Piece& p = pieces[i];
    if (!p.output) {
      if (p.at < out_end) return THD_ERR_ALIAS;
      // its own output may follow at the same place, and replaces it
      if (i + 1 < pieces.size() && pieces[i + 1].output && pieces[i + 1].tensor == p.tensor &&
          pieces[i + 1].at == p.at) {
        if (pieces[i + 1].end != p.end || p.at < in_end) return THD_ERR_ALIAS;
        out_end = std::max(out_end, p.end);
        ++i;
      }
      in_end = std::max(in_end, p.end);
    } else {
      if (p.at < out_end || p.at < in_end) return THD_ERR_ALIAS;
      out_end = std::max(out_end, p.end);
    }
  }
  return THD_OK;
}

}  // namespace

extern "C" {

int thd_embedding(const int64_t* ids, const uint8_t* mask, int64_t rows, const void* table, int32_t dtype,
                  int64_t vocab, int64_t width, int64_t table_stride, double scale, void* out, int64_t out_stride,
                  int32_t* status, void* stream) {
  const int es = element_bytes(dtype);
  if (es == 0 || !sizes_ok(rows, vocab, width) || !finite32(scale)) return THD_ERR_ARG;
  const int64_t in_bytes = matrix_bytes(vocab, width, table_stride, es);
  const int64_t out_bytes = matrix_bytes(rows, width, out_stride, es);
  if (in_bytes < 0 || out_bytes < 0 || !table || !aligned(table, es)) return THD_ERR_ARG;
  if (rows > 0 && (!ids || !out || !aligned(out, es))) return THD_ERR_ARG;
  const Range outs[] = {{out, out_bytes}, {status, 4}};
  const Range ins[] = {{table, in_bytes}, {ids, rows * 8}, {mask, rows}};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  thdcp::EmbedArgs a{};
  a.ids = ids;
  a.mask = mask;
  a.table = table;
  a.out = out;
  a.in_stride = table_stride;
  a.out_stride = out_stride;
  a.rows = static_cast<int32_t>(rows);
  a.vocab = static_cast<int32_t>(vocab);
  a.width = static_cast<int32_t>(width);
  a.dtype = dtype;
  a.scale = static_cast<float>(scale);
  a.status = status;
  // one workgroup looks through the ids beside the copy of the rows, which takes longer
  // than that if rows are long, or there are few; else a launch clears the status first
  const int64_t row_bytes = width * (dtype == THD_FP32 ? 4 : 2);
  a.scan = status && rows > 0 && (rows <= 8192 || row_bytes >= 4096);
  if (status && !a.scan && thdcp::launch_status_init(status, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
  if (rows == 0) return THD_OK;
  return launched(thdcp::launch_embedding(a, as_stream(stream)));
}

int64_t thd_embedding_workspace_bytes(int64_t rows, int64_t vocab, int64_t width) {
  if (!sizes_ok(rows, vocab, width)) return -1;
  return embed_layout(nullptr, rows, vocab, width).bytes;
}

int thd_embedding_backward(const void* drows, int32_t dtype, const int64_t* ids, const uint8_t* mask, int64_t rows,
                           int64_t vocab, int64_t width, int64_t row_stride, double scale, int32_t accumulate,
                           void* dtable, int32_t out_dtype, int64_t table_stride, int32_t* status, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  const int es = element_bytes(dtype), os = element_bytes(out_dtype);
  if (es == 0 || os == 0 || (out_dtype != dtype && out_dtype != THD_FP32)) return THD_ERR_ARG;
  if (!sizes_ok(rows, vocab, width) || !finite32(scale) || (accumulate != 0 && accumulate != 1)) return THD_ERR_ARG;
  const int64_t in_bytes = matrix_bytes(rows, width, row_stride, es);
  const int64_t out_bytes = matrix_bytes(vocab, width, table_stride, os);
  if (in_bytes < 0 || out_bytes < 0 || !dtable || !aligned(dtable, os)) return THD_ERR_ARG;
  if (rows > 0 && (!ids || !drows || !aligned(drows, es))) return THD_ERR_ARG;
  const EmbedLayout l = embed_layout(workspace, rows, vocab, width);
  if (l.bytes > 0 && (!workspace || workspace_bytes < l.bytes || !aligned(workspace, 16))) return THD_ERR_ARG;
  const Range outs[] = {{dtable, out_bytes}, {status, 4}, {workspace, l.bytes}};
  const Range ins[] = {{drows, in_bytes}, {ids, rows * 8}, {mask, rows}};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  thdcp::EmbedArgs a{};
  a.ids = ids;
  a.mask = mask;
  a.drows = drows;
  a.dtable = dtable;
  a.in_stride = row_stride;
  a.out_stride = table_stride;
  a.rows = static_cast<int32_t>(rows);
  a.vocab = static_cast<int32_t>(vocab);
  a.width = static_cast<int32_t>(width);
  a.dtype = dtype;
  a.out_dtype = out_dtype;
  a.accumulate = accumulate;
  a.scale = static_cast<float>(scale);
  a.status = status;
  if (rows == 0) {
    if (status && thdcp::launch_status_init(status, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
  } else if (thdcp::launch_embedding_sort(a, l.sort, as_stream(stream)) != hipSuccess) {
    return THD_ERR_HIP;
  }
  return launched(thdcp::launch_embedding_sums(a, l.sort, as_stream(stream)));
}

int64_t thd_gradients_workspace_bytes(int32_t n_tensors) {
  if (n_tensors < 0 || n_tensors > THD_MAX_TENSORS) return -1;
  return lists_of(n_tensors) * thdcp::kNormBlocks * 8;
}

int thd_gradient_norm(const void* const* grads, const int64_t* elements, const int32_t* dtypes, int32_t n_tensors,
                      double scale, float* norm, int32_t* status, void* workspace, int64_t workspace_bytes,
                      void* stream) {
  if (!tensors_ok(grads, elements, dtypes, n_tensors) || !finite32(scale) || !norm) return THD_ERR_ARG;
  const int64_t need = thd_gradients_workspace_bytes(n_tensors);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 8))) return THD_ERR_ARG;
  const Range outs[] = {{norm, 4}, {status, 4}, {workspace, need}};
  if (!apart(outs, {{nullptr, 0}})) return THD_ERR_ALIAS;
  for (int32_t i = 0; i < n_tensors; ++i)
    for (const Range& out : outs)
      if (meet(out, {grads[i], elements[i] * element_bytes(dtypes[i])})) return THD_ERR_ALIAS;
  thdcp::ClipArgs c{};
  c.scale = scale;
  c.partial = static_cast<double*>(workspace);
  c.norm = norm;
  c.status = status;
  const int rc = launch_sums(grads, elements, dtypes, n_tensors, static_cast<double*>(workspace), &c.partials, stream);
  return rc != THD_OK ? rc : launched(thdcp::launch_norm_finish(c, as_stream(stream)));
}

int thd_clip_gradients(const void* const* grads, void* const* outs, const int64_t* elements, const int32_t* dtypes,
                       const int32_t* out_dtypes, int32_t n_tensors, double max_norm, double scale,
                       const float* norm_in, float* norm, int32_t* status, void* workspace, int64_t workspace_bytes,
                       void* stream) {
  if (!tensors_ok(grads, elements, dtypes, n_tensors) || !finite32(scale) || !(max_norm > 0.0)) return THD_ERR_ARG;
  if (n_tensors > 0 && (!outs || !out_dtypes)) return THD_ERR_ARG;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (out_dtypes[i] != dtypes[i] && out_dtypes[i] != THD_FP32) return THD_ERR_ARG;
    if (elements[i] > 0 && (!outs[i] || !aligned(outs[i], element_bytes(out_dtypes[i])))) return THD_ERR_ARG;
  }
  const int64_t need = norm_in ? 0 : thd_gradients_workspace_bytes(n_tensors);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 8))) return THD_ERR_ARG;
  const Range own[] = {{norm, 4}, {status, 4}, {workspace, need}};
  const Range given[] = {{norm_in, 4}};
  if (!apart(own, given)) return THD_ERR_ALIAS;
  try {
    std::vector<Piece> pieces;
    pieces.reserve(2 * static_cast<size_t>(n_tensors) + 4);
    const auto add = [&](const void* p, int64_t bytes, int32_t tensor, bool output) {
      const auto at = reinterpret_cast<uintptr_t>(p);
      if (p && bytes > 0) pieces.push_back({at, at + static_cast<uintptr_t>(bytes), tensor, output});
    };
    for (int32_t i = 0; i < n_tensors; ++i) {
      add(grads[i], elements[i] * element_bytes(dtypes[i]), i, false);
      add(outs[i], elements[i] * element_bytes(out_dtypes[i]), i, true);
    }
    for (int32_t i = 0; i < 3; ++i) add(own[i].p, own[i].bytes, n_tensors + i, true);
    add(norm_in, 4, n_tensors + 3, false);
    const int rc = outputs_apart(pieces);
    if (rc != THD_OK) return rc;
  } catch (const std::bad_alloc&) {
    return THD_ERR_HIP;  // no memory for the check
  }
  thdcp::ClipArgs c{};
  c.scale = scale;
  c.max_norm = max_norm;
  c.partial = static_cast<double*>(workspace);
  c.norm_in = norm_in;
  c.norm = norm;
  c.status = status;
  if (!norm_in) {
    const int rc = launch_sums(grads, elements, dtypes, n_tensors, static_cast<double*>(workspace), &c.partials,
                               stream);
    if (rc != THD_OK) return rc;
  }
  // Few chunks: every workgroup adds up the partial sums for itself, and the first launch
  // writes the norm and the status.  Many: they are added up once, by a launch of their
  // own, and each chunk takes a workgroup: 6.3 TB/s for 1 GiB where 2048 workgroups that
  // go round reach 4.7.
  int64_t chunks = 0;
  for (int32_t i = 0; i < n_tensors; ++i) chunks += chunks_of(elements[i], dtypes[i]);
  bool finish = true;
  if (!norm_in && norm && chunks > thdcp::kNormBlocks) {
    if (thdcp::launch_norm_finish(c, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
    c.norm_in = norm;
    c.norm = nullptr;
    finish = false;
  }
  const bool each = c.norm_in != nullptr;
  for (int32_t from = (n_tensors - 1) / thdcp::kListTensors * thdcp::kListTensors; n_tensors > 0 && from >= 0;
       from -= thdcp::kListTensors) {
    const thdcp::GradList l = list_of(grads, outs, elements, dtypes, out_dtypes, n_tensors, from);
    if (l.first[l.tensors] == 0) continue;
    const int32_t blocks = each ? l.first[l.tensors] : blocks_of(l);
    if (thdcp::launch_clip(l, c, blocks, finish, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
    finish = false;
  }
  return finish ? launched(thdcp::launch_norm_finish(c, as_stream(stream))) : THD_OK;
}

}  // extern "C"
