// Norm of many gradients together, and their scaling to a largest norm.
//
// Tensors come as a list passed by value with the launch (96 of them; more take
// more launches), each cut into chunks of 32 KiB.  Workgroups go round the chunks
// of all tensors, at most 2048 of them, and leave one sum of squares each; the
// workgroups that scale add those up for themselves, so that there is no launch in
// between.  Squares of a word are added in 32 bits and joined in 64, and formed in 64
// bits from the start where 32 cannot hold them: no gradient is too large or too small
// to square.  Chunks are scaled in the order opposite to the one they were read in, so
// that up to the last 192 MB come out of the cache instead of memory; what comes before
// is read past it.
//
// Bound by memory: 1 GiB of bf16 in 147 tensors takes 565 us, 157 of them for the norm
// and 398 for the scaling: 5.7 TB/s of two readings and a writing.
#include "thd_loss_device.h"
#include "thd_params_internal.h"

namespace thdcp {

namespace {

struct __attribute__((packed, aligned(2))) LooseWord {
  uint32_t x[4];
};
typedef unsigned int LooseVector __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ Word4 load_loose(const void* p) {
  const LooseWord w = *static_cast<const LooseWord*>(p);
  return Word4{w.x[0], w.x[1], w.x[2], w.x[3]};
}
__device__ __forceinline__ Word4 load_stream(const void* p) {
  return __builtin_nontemporal_load(static_cast<const LooseVector*>(p));
}
__device__ __forceinline__ void store_stream(void* p, Word4 v) {
  __builtin_nontemporal_store(v, static_cast<LooseVector*>(p));
}

constexpr int kClipThreads = 256;
constexpr int kKeptChunks = (192 << 20) / kGradChunkBytes;  // of 256 MB of cache in front of memory

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

// A chunk: where its first element is, how many it has.  The host says how many the
// last one has, so that no 64-bit minimum is formed here: hipcc (ROCm 7.2) took one
// that is uniform over a wave from a condition code it had overwritten, and read past
// the tensor.  A tensor's entry is one scalar load: kernel arguments are far from the
// compute units.
struct Chunk {
  const char* in = nullptr;
  char* out = nullptr;
  int32_t type = 0, out_type = 0, n = 0;      // n 0: no chunk
  bool own = false;                           // the output is the gradient itself
  __device__ __forceinline__ Chunk() {}
  __device__ __forceinline__ Chunk(const GradList& l, const ListSearch& search, int32_t chunk) {
    const int32_t t = search(chunk);
    const GradEntry e = l.entry[t];
    type = e.types & 255;
    out_type = e.types >> 8;
    const int32_t per = chunk_elements(type);
    const int64_t at = static_cast<int64_t>(chunk - l.first[t]) * per;
    n = chunk + 1 == l.first[t + 1] ? e.tail : per;
    own = e.in == e.out;
    in = static_cast<const char*>(e.in) + at * (type == THD_FP32 ? 4 : 2);
    out = static_cast<char*>(e.out) + at * (out_type == THD_FP32 ? 4 : 2);
  }
};

// Squares of a word's elements: in 32 bits where they can be (errors up to 2^-21 of a
// word, which average out over many), else in 64.  `odd` gathers what 32 bits cannot
// hold: a sum that is infinite or NaN, or so small that squares were lost below 2^-126.
template <typename T>
__device__ __forceinline__ float word_squares(Word4 x, bool* odd) {
  constexpr int kPer = Elem<T>::kPer;
  float v[kPer], sum = 0.0f;
  Elem<T>::unpack(x, v);
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum = fmaf(v[j], v[j], sum);
  *odd |= !(sum >= 0x1p-96f && sum < __builtin_huge_valf());
  return sum;
}
template <typename T>
__device__ __forceinline__ double word_squares64(Word4 x) {
  constexpr int kPer = Elem<T>::kPer;
  float v[kPer];
  double sum = 0.0;
  Elem<T>::unpack(x, v);
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), sum);
  return sum;
}

template <typename T, bool kStream>
__device__ __forceinline__ double chunk_squares(const T* p, int32_t n) {
  constexpr int kPer = Elem<T>::kPer, kWords = kGradChunkBytes / 16 / kClipThreads;
  if (n == kWords * kClipThreads * kPer) {
    Word4 x[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const T* at = p + (i * kClipThreads + threadIdx.x) * kPer;
      x[i] = kStream ? load_stream(at) : load_loose(at);
    }
    bool odd = false;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) sum += static_cast<double>(word_squares<T>(x[i], &odd));
    if (__any(odd)) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) sum += word_squares64<T>(x[i]);
    }
    return sum;
  }
  double sum = 0.0;
  const int32_t words = n / kPer;
  for (int32_t i = threadIdx.x; i < words; i += kClipThreads) sum += word_squares64<T>(load_loose(p + i * kPer));
  const int32_t t = words * kPer + threadIdx.x;
  if (t < n) {
    const double v = Elem<T>::load(p + t);
    sum = fma(v, v, sum);
  }
  return sum;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const Chunk& k, bool stream) {
  const T* p = reinterpret_cast<const T*>(k.in);
  return stream ? chunk_squares<T, true>(p, k.n) : chunk_squares<T, false>(p, k.n);
}

// Chunks before `kept` are read past the caches.
__global__ __launch_bounds__(kClipThreads) void norm_kernel(GradList l, double* partial, int32_t kept) {
  __shared__ double s_wave[kClipThreads / 64];
  const ListSearch search(l);
  double sum = 0.0;
  const int32_t chunks = l.first[l.tensors];
  int32_t c = blockIdx.x;
  Chunk k = c < chunks ? Chunk(l, search, c) : Chunk();
  while (k.n > 0) {
    const bool stream = c < kept;
    c += gridDim.x;
    const Chunk next = c < chunks ? Chunk(l, search, c) : Chunk();
    if (k.type == THD_BF16) sum += chunk_squares<Bf16>(k, stream);
    else if (k.type == THD_FP16) sum += chunk_squares<Fp16>(k, stream);
    else sum += chunk_squares<float>(k, stream);
    k = next;
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

// What gradients are multiplied by, rounded once from 64 bits: below 2^-126, where 32 bits
// have no room for a factor of 24 bits, a number from 1/2 to 1 and a power of two, else the
// factor itself and 2^0.
struct Factor {
  float f;
  int32_t power = 0;
  __device__ __forceinline__ explicit Factor(double x) {
    if (x != 0.0 && fabs(x) < 0x1p-126) x = frexp(x, &power);
    f = static_cast<float>(x);
  }
  __device__ __forceinline__ float operator()(float x) const { return ldexpf(x * f, power); }
  __device__ __forceinline__ bool one() const { return f == 1.0f && power == 0; }
};

// A chunk scaled.  Words lie as the tensors do: stores at any place within 16 bytes run
// as fast as words cut by the output (1 GiB of bf16, outputs 2 bytes past a word: 400
// us against 419).
template <typename TI, typename TO>
__device__ __forceinline__ void scale_chunk(const TI* p, TO* to, int32_t n, Factor f, bool zero) {
  constexpr int kPer = Elem<TI>::kPer, kOut = Elem<TO>::kPer, kWords = kGradChunkBytes / 16 / kClipThreads;
  const int32_t words = n / kPer;
  Word4 x[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const int32_t w = i * kClipThreads + threadIdx.x;
    if (w < words) x[i] = load_stream(p + w * kPer);
  }
  const int32_t edge = words * kPer + threadIdx.x;
  if (edge < n) to[edge] = Elem<TO>::round(zero ? 0.0f : f(Elem<TI>::load(p + edge)));
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    const int32_t w = i * kClipThreads + threadIdx.x;
    if (w >= words) continue;
    float v[kPer];
    Elem<TI>::unpack(x[i], v);
#pragma unroll
    for (int part = 0; part < kPer; part += kOut) {
      float y[kOut];
#pragma unroll
      for (int j = 0; j < kOut; ++j) y[j] = zero ? 0.0f : f(v[part + j]);
      store_stream(to + w * kPer + part, Elem<TO>::pack(y));
    }
  }
}

template <typename TI>
__device__ __forceinline__ void scale_tensor(const Chunk& k, Factor f, bool zero) {
  const TI* from = reinterpret_cast<const TI*>(k.in);
  if (k.out_type == THD_FP32) scale_chunk(from, reinterpret_cast<float*>(k.out), k.n, f, zero);
  else scale_chunk(from, reinterpret_cast<TI*>(k.out), k.n, f, zero);
}

__global__ __launch_bounds__(kClipThreads) void clip_kernel(GradList l, ClipArgs c, int32_t finish) {
  __shared__ double s_wave[kClipThreads / 64];
  const float norm = norm_of(c, s_wave);
  if (finish && blockIdx.x == 0) finish_norm(c, norm);
  const bool zero = !(fabsf(norm) < __builtin_huge_valf());
  const double shrink = c.max_norm / (static_cast<double>(norm) + 1e-6);
  const Factor f(c.scale * (shrink < 1.0 ? shrink : 1.0));
  const ListSearch search(l);
  const int32_t chunks = l.first[l.tensors];
  int32_t at = blockIdx.x;
  Chunk k = at < chunks ? Chunk(l, search, chunks - 1 - at) : Chunk();
  while (k.n > 0) {
    at += gridDim.x;
    const Chunk next = at < chunks ? Chunk(l, search, chunks - 1 - at) : Chunk();
    if (!k.own || !f.one() || zero) {  // else it holds the result
      if (k.type == THD_BF16) scale_tensor<Bf16>(k, f, zero);
      else if (k.type == THD_FP16) scale_tensor<Fp16>(k, f, zero);
      else scale_tensor<float>(k, f, zero);
    }
    k = next;
  }
}

}  // namespace

hipError_t launch_norm(const GradList& l, double* partial, int32_t blocks, bool last, hipStream_t stream) {
  const int32_t chunks = l.first[l.tensors];
  norm_kernel<<<blocks, kClipThreads, 0, stream>>>(l, partial, last ? chunks - kKeptChunks : chunks);
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
