// Norm of many gradients together, and their scaling to a largest norm.
//
// Tensors come as a list passed by value with the launch (96 of them; more take
// more launches), each cut into chunks of 32 KiB.  Workgroups go round the chunks
// of all tensors, at most 2048 of them, and leave one sum of squares each; the
// workgroups that scale add those up for themselves, so that there is no launch in
// between.  Squares and sums are held in 64 bits: no gradient of 32 bits is too
// large to square, and the additions cost nothing beside the reads.  Chunks are
// scaled in the order opposite to the one they were read in, so that up to the last
// 256 MB come out of the cache instead of memory.
#include "thd_loss_device.h"
#include "thd_params_internal.h"

namespace thdcp {

namespace {

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

constexpr int kClipThreads = 256;

// The tensor that holds a chunk: lanes compare the list's prefix with it.
struct ListSearch {
  int32_t a, b;
  __device__ __forceinline__ explicit ListSearch(const GradList& l) {
    const int32_t lane = threadIdx.x & 63;
    a = lane < l.tensors ? l.first[lane] : INT32_MAX;
    b = lane + 64 < l.tensors ? l.first[min(lane + 64, kListTensors)] : INT32_MAX;
  }
  __device__ __forceinline__ int32_t operator()(int32_t chunk) const {
    return __popcll(__ballot(a <= chunk)) + __popcll(__ballot(b <= chunk)) - 1;
  }
};

__device__ __forceinline__ double block_sum(double x, double* s_wave) {
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) x += __shfl_xor(x, i);
  if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int i = 0; i < kClipThreads / 64; ++i) x += s_wave[i];
  return x;
}

// Elements of a type in a chunk.
__device__ __forceinline__ int32_t chunk_elements(int32_t type) {
  return type == THD_FP32 ? kGradChunkBytes / 4 : kGradChunkBytes / 2;
}

// A chunk: its tensor's type, its first element and how many it has.  The host says
// how many the last one has, so that no 64-bit minimum is formed here: hipcc (ROCm
// 7.2) took one that is uniform over a wave from a condition code it had overwritten,
// and read past the tensor.
struct Chunk {
  int32_t type, n;
  int64_t at;
  __device__ __forceinline__ Chunk(const GradList& l, int32_t t, int32_t chunk) : type(l.in_type[t]) {
    n = chunk + 1 == l.first[t + 1] ? l.tail[t] : chunk_elements(type);
    at = static_cast<int64_t>(chunk - l.first[t]) * chunk_elements(type);
  }
};

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int32_t n) {
  constexpr int kPer = Elem<T>::kPer, kWords = kGradChunkBytes / 16 / kClipThreads;
  double sum[2] = {0.0, 0.0};
  if (n == kWords * kClipThreads * kPer) {
    Word4 x[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) x[i] = load_loose(p + (i * kClipThreads + threadIdx.x) * kPer);
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      float v[kPer];
      Elem<T>::unpack(x[i], v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum[j & 1] = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), sum[j & 1]);
    }
    return sum[0] + sum[1];
  }
  const int32_t words = n / kPer;
  for (int32_t i = threadIdx.x; i < words; i += kClipThreads) {
    float v[kPer];
    Elem<T>::unpack(load_loose(p + i * kPer), v);
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum[j & 1] = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), sum[j & 1]);
  }
  const int32_t t = words * kPer + threadIdx.x;
  if (t < n) {
    const double v = Elem<T>::load(p + t);
    sum[0] = fma(v, v, sum[0]);
  }
  return sum[0] + sum[1];
}

__global__ __launch_bounds__(kClipThreads) void norm_kernel(GradList l, double* partial) {
  __shared__ double s_wave[kClipThreads / 64];
  const ListSearch search(l);
  double sum = 0.0;
  const int32_t chunks = l.first[l.tensors];
  for (int32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int32_t t = search(c);
    const Chunk k(l, t, c);
    if (k.type == THD_BF16) sum += chunk_squares(static_cast<const Bf16*>(l.in[t]) + k.at, k.n);
    else if (k.type == THD_FP16) sum += chunk_squares(static_cast<const Fp16*>(l.in[t]) + k.at, k.n);
    else sum += chunk_squares(static_cast<const float*>(l.in[t]) + k.at, k.n);
  }
  sum = block_sum(sum, s_wave);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm, as every workgroup forms it: in the same order, so the same bits.
__device__ __forceinline__ float norm_of(const ClipArgs& c, double* s_wave) {
  if (c.norm_in) return fabsf(*c.norm_in);
  double sum = 0.0;
#pragma unroll 4
  for (int32_t i = threadIdx.x; i < c.partials; i += kClipThreads) sum += c.partial[i];
  sum = block_sum(sum, s_wave);
  return static_cast<float>(fabs(c.scale) * sqrt(sum));
}

__device__ __forceinline__ void finish_norm(const ClipArgs& c, float norm) {
  if (threadIdx.x != 0) return;
  if (c.norm) *c.norm = norm;
  if (c.status) *c.status = fabsf(norm) < __builtin_huge_valf() ? THD_OK : THD_ERR_NORM;
}

__global__ __launch_bounds__(kClipThreads) void norm_finish_kernel(ClipArgs c) {
  __shared__ double s_wave[kClipThreads / 64];
  finish_norm(c, norm_of(c, s_wave));
}

template <typename TI, typename TO>
__device__ __forceinline__ void scale_chunk(const TI* p, TO* to, int32_t n, float f, bool zero) {
  constexpr int kPer = Elem<TI>::kPer, kOut = Elem<TO>::kPer, kWords = kGradChunkBytes / 16 / kClipThreads;
  const auto put = [&](int32_t word, Word4 x) {
    float v[kPer];
    Elem<TI>::unpack(x, v);
#pragma unroll
    for (int part = 0; part < kPer; part += kOut) {
      float y[kOut];
#pragma unroll
      for (int j = 0; j < kOut; ++j) y[j] = zero ? 0.0f : v[part + j] * f;
      store_loose(to + word * kPer + part, Elem<TO>::pack(y));
    }
  };
  if (n == kWords * kClipThreads * kPer) {
    Word4 x[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) x[i] = load_loose(p + (i * kClipThreads + threadIdx.x) * kPer);
#pragma unroll
    for (int i = 0; i < kWords; ++i) put(i * kClipThreads + threadIdx.x, x[i]);
    return;
  }
  const int32_t words = n / kPer;
  for (int32_t i = threadIdx.x; i < words; i += kClipThreads) put(i, load_loose(p + i * kPer));
  const int32_t t = words * kPer + threadIdx.x;
  if (t < n) to[t] = Elem<TO>::round(zero ? 0.0f : Elem<TI>::load(p + t) * f);
}

template <typename TI>
__device__ __forceinline__ void scale_tensor(const GradList& l, int32_t t, const Chunk& k, float f, bool zero) {
  const TI* from = static_cast<const TI*>(l.in[t]) + k.at;
  if (l.out_type[t] == THD_FP32) scale_chunk(from, static_cast<float*>(l.out[t]) + k.at, k.n, f, zero);
  else scale_chunk(from, static_cast<TI*>(l.out[t]) + k.at, k.n, f, zero);
}

__global__ __launch_bounds__(kClipThreads) void clip_kernel(GradList l, ClipArgs c, int32_t finish) {
  __shared__ double s_wave[kClipThreads / 64];
  const float norm = norm_of(c, s_wave);
  if (finish && blockIdx.x == 0) finish_norm(c, norm);
  const bool zero = !(fabsf(norm) < __builtin_huge_valf());
  // the factor in 64 bits, rounded once
  const double shrink = c.max_norm / (static_cast<double>(norm) + 1e-6);
  const auto f = static_cast<float>(c.scale * (shrink < 1.0 ? shrink : 1.0));
  const ListSearch search(l);
  const int32_t chunks = l.first[l.tensors];
  for (int32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const int32_t chunk = chunks - 1 - i;
    const int32_t t = search(chunk);
    if (l.in[t] == l.out[t] && f == 1.0f && !zero) continue;  // it holds the result
    const Chunk k(l, t, chunk);
    if (k.type == THD_BF16) scale_tensor<Bf16>(l, t, k, f, zero);
    else if (k.type == THD_FP16) scale_tensor<Fp16>(l, t, k, f, zero);
    else scale_tensor<float>(l, t, k, f, zero);
  }
}

}  // namespace

hipError_t launch_norm(const GradList& l, double* partial, int32_t blocks, hipStream_t stream) {
  norm_kernel<<<blocks, kClipThreads, 0, stream>>>(l, partial);
  return hipGetLastError();
}

hipError_t launch_norm_finish(const ClipArgs& c, hipStream_t stream) {
  norm_finish_kernel<<<1, kClipThreads, 0, stream>>>(c);
  return hipGetLastError();
}

hipError_t launch_clip(const GradList& l, const ClipArgs& c, int32_t blocks, bool finish, hipStream_t stream) {
  clip_kernel<<<blocks, kClipThreads, 0, stream>>>(l, c, finish ? 1 : 0);
  return hipGetLastError();
}

}  // namespace thdcp
