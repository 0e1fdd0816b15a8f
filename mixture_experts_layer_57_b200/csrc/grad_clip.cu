// Global gradient norm over a list of tensors, and clipping by it.
//
//     norm   = sqrt( sum over all tensors and elements of g^2 )
//     out[i] = g[i] * min(1, max_norm / (norm + 1e-6))
//
// Two launches for a list: the norm needs every element before the first one can be scaled. Both
// are persistent grids over chunks of 8192 elements of one tensor; the list (addresses, lengths,
// first chunk of each tensor) travels in the kernel's parameters, so a captured launch keeps its
// own copy and nothing is staged in device memory. Bound by HBM: the norm reads every gradient
// once; the scaling reads and writes once, walking the list backwards, so that what the norm read
// last (up to the size of L2) is met there again.
//
// Sums: a thread adds the squares of its up to 32 elements of a chunk in fp32 and that sum to a
// double; blocks join in doubles, the last block to finish adds the blocks' sums in block order,
// so the result does not change from call to call. Where the fp32 sum of a chunk overflowed, or
// is so small that squares were lost below the normal range, the thread adds its elements again
// in double: norms are right for gradients of any finite size.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kChunk = 8192;
constexpr int kBlock = 256;

template <int N>
struct GradTable {
  const void* in[N];
  void* out[N];
  int64_t n[N];
  int first[N + 1];     // first chunk of each tensor; first[count] = all chunks
  uint8_t flags[N];     // bit 0: in is bf16, bit 1: out is bf16
  int count;
};
constexpr int kSmallList = 48, kLargeList = 1024;
static_assert(sizeof(GradTable<kLargeList>) + 64 <= 32764, "kernel parameter space");

template <int N>
__device__ __forceinline__ int tensor_of(const GradTable<N>& t, int chunk) {
  int lo = 0, hi = t.count;  // first[lo] <= chunk < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The elements of a chunk: a scalar head up to the first 16-byte boundary, 16-byte words, a
// scalar tail; one call of f per element, always the same elements to the same thread.
template <bool BF16, class F>
__device__ __forceinline__ void for_elements(const void* in, int64_t c0, int n, F f) {
  constexpr int VEC = BF16 ? 8 : 4;
  const uint8_t* base = reinterpret_cast<const uint8_t*>(in) + c0 * (BF16 ? 2 : 4);
  const int head = min(n, (int)(((16u - ((uint32_t)(uintptr_t)base & 15u)) & 15u) / (BF16 ? 2 : 4)));
  const int words = (n - head) / VEC;
  const int tail = head + words * VEC;
  if ((int)threadIdx.x < head) f(load_elem<BF16>(base, threadIdx.x));
  const uint4* v = reinterpret_cast<const uint4*>(base + head * (BF16 ? 2 : 4));
#pragma unroll 4
  for (int i = threadIdx.x; i < words; i += kBlock) {
    const uint4 q = v[i];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        f(__uint_as_float(w[j] << 16));
        f(__uint_as_float(w[j] & 0xffff0000u));
      } else {
        f(__uint_as_float(w[j]));
      }
    }
  }
  if ((int)threadIdx.x < n - tail) f(load_elem<BF16>(base, tail + threadIdx.x));
}

template <bool BF16>
__device__ __forceinline__ double chunk_squares(const void* in, int64_t c0, int n) {
  float s = 0.0f;
  uint32_t any = 0;
  for_elements<BF16>(in, c0, n, [&](float g) {
    s = fmaf(g, g, s);
    any |= __float_as_uint(g) << 1;  // zero for +-0 only
  });
  // from 2^-96 on, 32 squares lost below 2^-126 are less than 2^-25 of the sum
  if (any != 0 && !(s >= 1.262177448e-29f && s <= 3.0e38f)) {
    double d = 0.0;
    for_elements<BF16>(in, c0, n, [&](float g) { d = fma((double)g, (double)g, d); });
    return d;
  }
  return (double)s;
}

// Sum over the block; the result is valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0;
    for (int i = 0; i < kBlock / 32; ++i) v += sh[i];
  }
  return v;
}

// One block's sum per entry of partials; the last block to finish adds them in block order to the
// earlier launches' total (`first`: there is none) and, in the list's last launch, writes the norm.
template <int N>
__global__ void __launch_bounds__(kBlock)
    grad_norm_kernel(const __grid_constant__ GradTable<N> t, double* partials, double* total,
                     int first, int finish, unsigned* ticket, float* norm) {
  __shared__ double sh[kBlock / 32];
  __shared__ int last;
  pdl_wait();
  double sum = 0.0;
  const int chunks = t.first[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t c0 = (int64_t)(c - t.first[i]) * kChunk;
    const int n = (int)min((int64_t)kChunk, t.n[i] - c0);
    sum += (t.flags[i] & 1) ? chunk_squares<true>(t.in[i], c0, n)
                            : chunk_squares<false>(t.in[i], c0, n);
  }
  const double b = block_sum(sum, sh);
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = b;
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (last) {
    __threadfence();
    double s = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += kBlock) s += __ldcg(partials + i);
    s = block_sum(s, sh);
    if (threadIdx.x == 0) {
      if (!first) s += *total;
      *total = s;
      if (finish) *norm = (float)sqrt(s);
      *ticket = 0u;  // ready for the next launch
    }
  }
  pdl_trigger();
}

template <bool IN16, bool OUT16>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, int64_t c0, int n, float k) {
  constexpr int VEC = IN16 ? 8 : 4;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(in) + c0 * (IN16 ? 2 : 4);
  uint8_t* dst = reinterpret_cast<uint8_t*>(out) + c0 * (OUT16 ? 2 : 4);
  int done = 0;
  if ((((uintptr_t)src | (uintptr_t)dst) & 15u) == 0) {
    const int words = n / VEC;
#pragma unroll 4
    for (int i = threadIdx.x; i < words; i += kBlock) {
      const uint4 q = reinterpret_cast<const uint4*>(src)[i];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      float v[VEC];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (IN16) {
          v[2 * j] = k * __uint_as_float(w[j] << 16);
          v[2 * j + 1] = k * __uint_as_float(w[j] & 0xffff0000u);
        } else {
          v[j] = k * __uint_as_float(w[j]);
        }
      }
      if constexpr (OUT16) {
        uint32_t o[VEC / 2];
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j)
          o[j] = (uint32_t)f32_to_bf16_rn(v[2 * j]) | ((uint32_t)f32_to_bf16_rn(v[2 * j + 1]) << 16);
        if constexpr (IN16) reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[0], o[1], o[2], o[3]);
        else reinterpret_cast<uint2*>(dst)[i] = make_uint2(o[0], o[1]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC / 4; ++j)
          reinterpret_cast<float4*>(dst)[i * (VEC / 4) + j] =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
    }
    done = words * VEC;
  }
#pragma unroll 8
  for (int i = done + threadIdx.x; i < n; i += kBlock) {
    const float v = k * load_elem<IN16>(src, i);
    if constexpr (OUT16) reinterpret_cast<uint16_t*>(dst)[i] = f32_to_bf16_rn(v);
    else reinterpret_cast<float*>(dst)[i] = v;
  }
}

template <int N>
__global__ void __launch_bounds__(kBlock)
    grad_scale_kernel(const __grid_constant__ GradTable<N> t, const float* norm, float max_norm) {
  pdl_wait();
  const float c = max_norm / (*norm + 1e-6f);
  const float k = c > 1.0f ? 1.0f : c;  // NaN stays NaN
  const int chunks = t.first[t.count];
  for (int r = blockIdx.x; r < chunks; r += gridDim.x) {
    const int ch = chunks - 1 - r;
    const int i = tensor_of(t, ch);
    // a factor of 1 leaves a tensor that is scaled in place as it is
    if (k == 1.0f && t.in[i] == t.out[i]) continue;
    const int64_t c0 = (int64_t)(ch - t.first[i]) * kChunk;
    const int n = (int)min((int64_t)kChunk, t.n[i] - c0);
    switch (t.flags[i]) {
      case 0: scale_chunk<false, false>(t.in[i], t.out[i], c0, n, k); break;
      case 1: scale_chunk<true, false>(t.in[i], t.out[i], c0, n, k); break;
      case 2: scale_chunk<false, true>(t.in[i], t.out[i], c0, n, k); break;
      default: scale_chunk<true, true>(t.in[i], t.out[i], c0, n, k);
    }
  }
  pdl_trigger();
}

// Tensors from `from` on, as many as the table and its chunk numbers hold; returns the next one.
template <int N>
int64_t fill(GradTable<N>& t, const GradTensor* list, int64_t from, int64_t n_tensors) {
  int k = 0;
  int64_t chunks = 0, i = from;
  for (; i < n_tensors && k < N; ++i) {
    if (list[i].n == 0) continue;
    const int64_t c = (list[i].n + kChunk - 1) / kChunk;
    if (chunks + c >= INT32_MAX - kGradNormMaxBlocks) break;
    t.in[k] = list[i].in;
    t.out[k] = list[i].out;
    t.n[k] = list[i].n;
    t.first[k] = (int)chunks;
    t.flags[k] = (uint8_t)(list[i].in_bf16 | (list[i].out_bf16 << 1));
    chunks += c;
    ++k;
  }
  t.first[k] = (int)chunks;
  t.count = k;
  return i;
}

// Blocks of one launch: eight to an SM at most.
int grid_of(int chunks) { return std::min(chunks, std::min(8 * num_sms(), kGradNormMaxBlocks)); }

template <int N>
cudaError_t norm_lists(const GradTensor* list, int64_t n, double* partials, unsigned* ticket,
                       float* norm, cudaStream_t stream) {
  GradTable<N> t;
  int64_t at = 0;
  bool first = true;
  do {
    at = fill(t, list, at, n);
    const int grid = std::max(1, grid_of(t.first[t.count]));
    const cudaError_t e =
        launch_kernel(grad_norm_kernel<N>, dim3((unsigned)grid), dim3(kBlock), 0, stream, t,
                      partials + 1, partials, first ? 1 : 0, at >= n ? 1 : 0, ticket, norm);
    if (e != cudaSuccess) return e;
    first = false;
  } while (at < n);
  return cudaSuccess;
}

template <int N>
cudaError_t scale_lists(const GradTensor* list, int64_t n, const float* norm, float max_norm,
                        cudaStream_t stream) {
  GradTable<N> t;
  int64_t at = 0;
  while (at < n) {
    at = fill(t, list, at, n);
    if (t.count == 0) continue;
    const cudaError_t e = launch_kernel(grad_scale_kernel<N>, dim3((unsigned)grid_of(t.first[t.count])),
                                        dim3(kBlock), 0, stream, t, norm, max_norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t enqueue_grad_norm(const GradTensor* t, int64_t n_tensors, double* partials,
                              unsigned* ticket, float* norm, cudaStream_t stream) {
  return n_tensors <= kSmallList ? norm_lists<kSmallList>(t, n_tensors, partials, ticket, norm, stream)
                                 : norm_lists<kLargeList>(t, n_tensors, partials, ticket, norm, stream);
}

cudaError_t enqueue_grad_scale(const GradTensor* t, int64_t n_tensors, const float* norm,
                               float max_norm, cudaStream_t stream) {
  return n_tensors <= kSmallList ? scale_lists<kSmallList>(t, n_tensors, norm, max_norm, stream)
                                 : scale_lists<kLargeList>(t, n_tensors, norm, max_norm, stream);
}

}  // namespace moe
