// C ABI of the attention on packed streams: host-side argument checks and
// stream-ordered launches.  See include/thd_attention.h for the contract.
#include <cmath>

#include "thd_attn_internal.h"

namespace {

using thdcp::AttnArgs;
using thdcp::AttnTensor;

constexpr int64_t kMaxStride = 1 << 22;  // elements: 64 rows of a tile stay within 32-bit byte offsets

bool shape_ok(const thd_attention_shape* s) {
  if (!s || (s->dtype != THD_BF16 && s->dtype != THD_FP16)) return false;
  if (s->kv_heads < 1 || s->heads < s->kv_heads || s->heads % s->kv_heads != 0) return false;
  if (s->dim < 8 || s->dim > THD_MAX_HEAD_DIM || s->dim % 8 != 0) return false;
  if ((s->causal != 0 && s->causal != 1) || s->window < 0) return false;
  if (s->cp_size < 1 || s->cp_size > THD_MAX_CP || s->rank < 0 || s->rank >= s->cp_size) return false;
  // positions run a tile past the last token, and a window before the first, in 32 bits
  if (s->n_slots < 0 || s->n_slots == INT32_MAX) return false;
  if (s->total_tokens < 0 || s->total_tokens > THD_MAX_STREAM) return false;
  if (s->total_tokens % s->cp_size != 0) return false;
  // In 32 bits lse / scale has to be finite, products may end at 2^-126, which times scale
  // has to be nothing, and the gradients take up to 2^30 / cap and log2(e) cap.
  const auto scale = static_cast<float>(s->scale), cap = static_cast<float>(s->cap);
  if (!(scale >= std::ldexp(1.0f, -THD_SCALE_LOG2)) || !(scale <= std::ldexp(1.0f, THD_SCALE_LOG2))) return false;
  if (s->cap == 0.0) return true;
  if (!(cap >= std::ldexp(1.0f, -THD_CAP_LOG2)) || !std::isfinite(cap * 1.4426950408889634f)) return false;
  return std::isfinite(scale / cap) && scale / cap > 0.0f;
}

int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Parts that a group's heads are dealt out over for the key gradients.  A key tile of a
// long document has far more query rows to look at when it stands first than when it
// stands last, and up to 512 workgroups run at a time; smaller ones, more in number,
// fill in for each other.  Each part costs 16 bytes of sums a key element, written and
// read, which only long documents repay: wanted are half as many workgroups as the mean
// slot has tokens, up to 2048.  Backward of 32 heads of 128 over 8, causal, in one part
// and in this rule's: 8192 tokens in one document 1.70 and 1.11 ms (key gradients), in
// documents of 4096 1103 and 1016 us, of 512 205 us both (267 in two parts).
int32_t key_parts(const thd_attention_shape& s, int64_t key_tiles) {
  const int32_t group = s.heads / s.kv_heads;
  if (s.n_slots == 0) return 1;
  const int64_t half = s.total_tokens / s.n_slots / 2, wanted = half < 2048 ? half : 2048;
  int32_t parts = 1;
  while (parts < group && (group % parts != 0 || key_tiles * s.kv_heads * parts < wanted)) ++parts;
  return parts;
}

struct Layout {
  thdcp::AttnPlan plan;
  int32_t key_parts;
  int64_t bytes;  // -1: more workgroups than a launch takes
};

// Tiles are bounded by whole tiles plus one part tile for each run of rows; a launch
// has one at least.
int64_t most_tiles(int64_t rows, int64_t runs, int64_t per) {
  const int64_t n = rows / per + (runs < rows ? runs : rows);
  return n > 0 ? n : 1;
}

Layout layout(const thd_attention_shape& s, void* workspace, bool backward) {
  Layout l{};
  const int64_t rows = s.total_tokens / s.cp_size;
  const int64_t nq = most_tiles(rows, (s.cp_size > 1 ? 2LL : 1LL) * s.n_slots,
                                thdcp::kAttnRows / thdcp::attn_tile_heads(s.heads / s.kv_heads));
  const int64_t nk = backward ? most_tiles(s.total_tokens, s.n_slots, thdcp::kAttnKeys) : 0;
  const int32_t group = s.heads / s.kv_heads;
  l.key_parts = backward ? key_parts(s, nk) : 1;
  // workgroups of 256 threads, which a launch counts in 32 bits
  const int64_t query_blocks = (nq * s.kv_heads + 8) * (group / thdcp::attn_tile_heads(group));
  const int64_t key_blocks = (nk * s.kv_heads + 8) * l.key_parts;
  if (query_blocks + key_blocks > static_cast<int64_t>(UINT32_MAX / 256)) {
    l.bytes = -1;
    return l;
  }
  char* base = static_cast<char*>(workspace);
  int64_t at = 0;
  const auto take = [&](int64_t n) {
    char* p = base + at;
    at += align_up(n, 16);
    return p;
  };
  l.plan.header = reinterpret_cast<int32_t*>(take(thdcp::kAttnHeaderWords * 4));
  l.plan.slot_first = reinterpret_cast<int32_t*>(take((s.n_slots + 1LL) * 4));
  l.plan.query_tiles = reinterpret_cast<thdcp::QueryTile*>(take(nq * static_cast<int64_t>(sizeof(thdcp::QueryTile))));
  if (backward) {
    l.plan.key_tiles = reinterpret_cast<thdcp::KeyTile*>(take(nk * static_cast<int64_t>(sizeof(thdcp::KeyTile))));
    l.plan.delta = reinterpret_cast<float*>(take(rows * s.heads * 4));
    if (l.key_parts > 1)
      l.plan.partial = reinterpret_cast<float*>(take(8 * l.key_parts * s.total_tokens * s.kv_heads * s.dim));
  }
  l.plan.max_query_tiles = static_cast<int32_t>(nq);
  l.plan.max_key_tiles = static_cast<int32_t>(nk);
  l.bytes = at;
  return l;
}

// A tensor as rows x heads x dim elements of two bytes in memory.
struct Extent {
  uintptr_t at = 0;
  int64_t bytes = 0;              // from the first to the last element; 0: nothing
  int64_t outer = 0, inner = 0;   // bytes: step of the outer index, bytes that one step covers
};

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Whether t can be a tensor of these sizes (an output's elements are apart).
bool tensor_ok(const thd_heads* t, int64_t rows, int64_t heads, int64_t dim, bool output, Extent* e) {
  if (!t) return false;
  if (rows == 0) return true;
  if (!t->data || !aligned(t->data, 16) || t->row_stride % 8 != 0 || t->head_stride % 8 != 0) return false;
  if (t->row_stride < 0 || t->row_stride > kMaxStride || (rows > 1 && t->row_stride < dim)) return false;
  if (t->head_stride < 0 || t->head_stride > INT64_MAX / 64 / heads) return false;
  const bool rows_out = heads == 1 || (rows > 1 && t->row_stride >= t->head_stride);
  const int64_t n_out = rows_out ? rows : heads, n_in = rows_out ? heads : rows;
  const int64_t s_out = rows_out ? t->row_stride : t->head_stride, s_in = rows_out ? t->head_stride : t->row_stride;
  e->at = reinterpret_cast<uintptr_t>(t->data);
  e->inner = 2 * ((n_in - 1) * s_in + dim);
  e->outer = 2 * s_out;
  e->bytes = (n_out - 1) * e->outer + e->inner;
  if (!output) return true;
  return (n_in == 1 || s_in >= dim) && (n_out == 1 || e->outer >= e->inner);
}

bool meet(const Extent& a, const Extent& b) {
  if (a.bytes <= 0 || b.bytes <= 0) return false;
  if (!(a.at < b.at + static_cast<uint64_t>(b.bytes) && b.at < a.at + static_cast<uint64_t>(a.bytes))) return false;
  // interleaved rows of one buffer: apart if their parts of a step are
  if (a.outer != b.outer || a.outer == 0 || a.inner > a.outer || b.inner > b.outer) return true;
  const auto step = static_cast<uint64_t>(a.outer);
  const uint64_t ahead = (b.at - a.at) % step;  // of b's part after a's, around the step
  const uint64_t d = b.at >= a.at ? ahead : (step - (a.at - b.at) % step) % step;
  return !(d >= static_cast<uint64_t>(a.inner) && d + static_cast<uint64_t>(b.inner) <= step);
}

Extent flat(const void* p, int64_t bytes) {
  Extent e;
  e.at = reinterpret_cast<uintptr_t>(p);
  e.bytes = p ? bytes : 0;
  return e;
}

template <size_t N, size_t M>
bool apart(const Extent (&outs)[N], const Extent (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = i + 1; j < N; ++j)
      if (meet(outs[i], outs[j])) return false;
    for (size_t j = 0; j < M; ++j)
      if (meet(outs[i], ins[j])) return false;
  }
  return true;
}

// A single row has no step to the next; the kernels' row bounds need one that
// covers a row.
AttnTensor tensor(const thd_heads* t, int64_t rows, int64_t dim) {
  return {t->data, rows > 1 ? t->row_stride : dim, t->head_stride};
}

AttnArgs arguments(const thd_attention_shape& s, const Layout& l) {
  AttnArgs a{};
  a.cu_padded = s.cu_seqlens_padded;
  a.cu_real = s.cu_seqlens;
  a.n_slots = s.n_slots;
  a.total = static_cast<int32_t>(s.total_tokens);
  a.rows = static_cast<int32_t>(s.total_tokens / s.cp_size);
  a.heads = s.heads;
  a.kv_heads = s.kv_heads;
  a.group = s.heads / s.kv_heads;
  a.tile_heads = thdcp::attn_tile_heads(a.group);
  a.key_parts = l.key_parts;
  a.dim = s.dim;
  a.dtype = s.dtype;
  a.causal = s.causal;
  a.window = s.window >= s.total_tokens ? 0 : s.window;  // sees everything: no window
  a.cp = s.cp_size;
  a.rank = s.rank;
  a.scale = static_cast<float>(s.scale);
  a.cap = static_cast<float>(s.cap);
  a.plan = l.plan;
  a.curve_limit = -1.0f;
  const double in = s.cap > 0.0 ? s.scale / s.cap : 0.0;
  if (in >= 0x1p-12 && in <= 0x1p12 && s.scale >= 0x1p-24 && s.scale <= 0x1p24) {
    double c = s.scale * 1.4426950408889634;
    for (int i = 0; i < 5; ++i, c *= in * in) a.curve[i] = static_cast<float>(c * thdcp::kAttnTanh[i]);
    a.curve_limit = static_cast<float>(0.5 / in);
  }
  return a;
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int64_t thd_attention_workspace_bytes(const thd_attention_shape* shape, int32_t backward) {
  if (!shape_ok(shape) || (backward != 0 && backward != 1)) return -1;
  return layout(*shape, nullptr, backward != 0).bytes;
}

int thd_attention(const thd_attention_shape* shape, const thd_heads* q, const thd_heads* k, const thd_heads* v,
                  const thd_heads* out, float* lse, int32_t* status, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  if (!shape_ok(shape) || !shape->cu_seqlens_padded) return THD_ERR_ARG;
  const thd_attention_shape& s = *shape;
  const int64_t rows = s.total_tokens / s.cp_size;
  Extent eq, ek, ev, eo;
  if (!tensor_ok(q, rows, s.heads, s.dim, false, &eq) || !tensor_ok(k, s.total_tokens, s.kv_heads, s.dim, false, &ek) ||
      !tensor_ok(v, s.total_tokens, s.kv_heads, s.dim, false, &ev) ||
      !tensor_ok(out, rows, s.heads, s.dim, true, &eo) || (rows > 0 && !lse))
    return THD_ERR_ARG;
  const Layout l = layout(s, workspace, false);
  if (l.bytes < 0 || !workspace || workspace_bytes < l.bytes || !aligned(workspace, 16)) return THD_ERR_ARG;
  const int64_t cu = (s.n_slots + 1LL) * 4;
  const Extent outs[] = {eo, flat(lse, rows * s.heads * 4), flat(status, 4), flat(workspace, l.bytes)};
  const Extent ins[] = {eq, ek, ev, flat(s.cu_seqlens_padded, cu), flat(s.cu_seqlens, cu)};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  AttnArgs a = arguments(s, l);
  a.q = tensor(q, rows, s.dim);
  a.k = tensor(k, s.total_tokens, s.dim);
  a.v = tensor(v, s.total_tokens, s.dim);
  a.out = tensor(out, rows, s.dim);
  a.lse = lse;
  a.status = status;
  if (thdcp::launch_attn_plan(a, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
  if (rows == 0) return THD_OK;
  return thdcp::launch_attn_forward(a, as_stream(stream)) == hipSuccess ? THD_OK : THD_ERR_HIP;
}

int thd_attention_backward(const thd_attention_shape* shape, const thd_heads* q, const thd_heads* k,
                           const thd_heads* v, const thd_heads* out, const float* lse, const thd_heads* dout,
                           const thd_heads* dq, const thd_heads* dk, const thd_heads* dv, int32_t* status,
                           void* workspace, int64_t workspace_bytes, void* stream) {
  if (!shape_ok(shape) || !shape->cu_seqlens_padded) return THD_ERR_ARG;
  const thd_attention_shape& s = *shape;
  const int64_t rows = s.total_tokens / s.cp_size, tokens = s.total_tokens;
  Extent eq, ek, ev, eo, eg, edq, edk, edv;
  if (!tensor_ok(q, rows, s.heads, s.dim, false, &eq) || !tensor_ok(k, tokens, s.kv_heads, s.dim, false, &ek) ||
      !tensor_ok(v, tokens, s.kv_heads, s.dim, false, &ev) || !tensor_ok(out, rows, s.heads, s.dim, false, &eo) ||
      !tensor_ok(dout, rows, s.heads, s.dim, false, &eg) || !tensor_ok(dq, rows, s.heads, s.dim, true, &edq) ||
      !tensor_ok(dk, tokens, s.kv_heads, s.dim, true, &edk) ||
      !tensor_ok(dv, tokens, s.kv_heads, s.dim, true, &edv) || (rows > 0 && !lse))
    return THD_ERR_ARG;
  const Layout l = layout(s, workspace, true);
  if (l.bytes < 0 || !workspace || workspace_bytes < l.bytes || !aligned(workspace, 16)) return THD_ERR_ARG;
  const int64_t cu = (s.n_slots + 1LL) * 4;
  const Extent outs[] = {edq, edk, edv, flat(status, 4), flat(workspace, l.bytes)};
  const Extent ins[] = {eq, ek, ev, eo, eg, flat(lse, rows * s.heads * 4), flat(s.cu_seqlens_padded, cu),
                        flat(s.cu_seqlens, cu)};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  AttnArgs a = arguments(s, l);
  a.q = tensor(q, rows, s.dim);
  a.k = tensor(k, s.total_tokens, s.dim);
  a.v = tensor(v, s.total_tokens, s.dim);
  a.out = tensor(out, rows, s.dim);
  a.dout = tensor(dout, rows, s.dim);
  a.dq = tensor(dq, rows, s.dim);
  a.dk = tensor(dk, s.total_tokens, s.dim);
  a.dv = tensor(dv, s.total_tokens, s.dim);
  a.lse = const_cast<float*>(lse);
  a.status = status;
  if (thdcp::launch_attn_plan(a, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
  if (rows == 0) return THD_OK;
  // fp16 gradients are scaled by the largest norms, which come with delta; bf16 takes
  // delta in the query gradients' launch
  if (s.dtype == THD_FP16 && thdcp::launch_attn_delta(a, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
  if (thdcp::launch_attn_dq(a, as_stream(stream)) != hipSuccess) return THD_ERR_HIP;
  return thdcp::launch_attn_dkv(a, as_stream(stream)) == hipSuccess ? THD_OK : THD_ERR_HIP;
}

}  // extern "C"
