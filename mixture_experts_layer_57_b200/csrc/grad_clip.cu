// Global gradient norm over a list of tensors, and clipping by it.
//
//     norm   = sqrt( sum over all tensors and elements of g^2 )
//     out[i] = g[i] * min(1, max_norm / (norm + 1e-6))
//
// Two launches for a list: the norm needs every element before the first one can be scaled. Both
// go by chunks of 8192 elements of one tensor; the list (addresses, lengths, first chunk of each
// tensor) travels in the kernel's parameters, so a captured launch keeps its own copy and nothing
// is staged in device memory. Bound by HBM: the norm reads every gradient once (persistent grid;
// 355 M fp32 elements: 233 us, 6.1 TB/s; 1.2 G bf16: 374 us, 6.4 TB/s), the scaling reads and
// writes once (a block per chunk; 355 M fp32 into odd places of a flat buffer: 423 us, 6.7 TB/s;
// 1.2 G bf16 into fp32: 1236 us, 5.8 TB/s).
//
// The scaling keeps few bytes in flight on purpose: with two or four words a thread, or as a
// persistent grid, the same work took 471 to 799 us (fp32) and 1341 to 2211 us (bf16 into fp32).
//
// Sums: a thread adds the squares of its up to 34 elements of a chunk in fp32, in two sums, and
// those to a double; blocks join in doubles, the last block to finish adds the blocks' sums in block order,
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
constexpr int kBlocksPerSm = 8;  // resident blocks per SM of the norm's persistent grid

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
// scalar tail; one call of one() per element of the ends and of four() per word, always the same
// elements to the same thread.
template <bool BF16, class One, class Four>
__device__ __forceinline__ void for_elements(const void* in, int64_t c0, int n, One one, Four four) {
  constexpr int VEC = BF16 ? 8 : 4, SIZE = BF16 ? 2 : 4;
  const uint8_t* base = reinterpret_cast<const uint8_t*>(in) + c0 * SIZE;
  const int head = min(n, (int)((16u - ((uint32_t)(uintptr_t)base & 15u)) & 15u) / SIZE);
  const int words = (n - head) / VEC;
  const int tail = head + words * VEC;
  if ((int)threadIdx.x < head) one(load_elem<BF16>(base, threadIdx.x));
  const uint4* v = reinterpret_cast<const uint4*>(base + head * SIZE);
#pragma unroll 4
  for (int i = threadIdx.x; i < words; i += kBlock) four(v[i]);
  if ((int)threadIdx.x < n - tail) one(load_elem<BF16>(base, tail + threadIdx.x));
}

template <bool BF16>
__device__ __forceinline__ double chunk_squares(const void* in, int64_t c0, int n) {
  float s0 = 0.0f, s1 = 0.0f;  // elements of even and odd place in a word
  uint32_t any = 0;            // bits of the values; without the signs, zero for +-0 only
  for_elements<BF16>(
      in, c0, n,
      [&](float g) {
        s0 = fmaf(g, g, s0);
        any |= __float_as_uint(g);
      },
      [&](const uint4& q) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        any |= (q.x | q.y) | (q.z | q.w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BF16) {
            const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
            s0 = fmaf(lo, lo, s0);
            s1 = fmaf(hi, hi, s1);
          } else {
            const float g = __uint_as_float(w[j]);
            float& s = j & 1 ? s1 : s0;
            s = fmaf(g, g, s);
          }
        }
      });
  const float s = s0 + s1;
  any &= BF16 ? 0x7fff7fffu : 0x7fffffffu;
  // from 2^-96 on, 32 squares lost below 2^-126 are less than 2^-25 of the sum
  if (any != 0 && !(s >= 1.262177448e-29f && s <= 3.0e38f)) {
    double d = 0.0;
    auto add = [&](float g) { d = fma((double)g, (double)g, d); };
    for_elements<BF16>(in, c0, n, add, [&](const uint4& q) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) add(__uint_as_float(w[j] << 16));
        add(__uint_as_float(BF16 ? w[j] & 0xffff0000u : w[j]));
      }
    });
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
__global__ void __launch_bounds__(kBlock, kBlocksPerSm)
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

// W consecutive 32-bit words that start `shift` bytes (even, below 16) into the 16-byte words from
// `a` on; every word read lies in the caller's range.
template <int W>
__device__ __forceinline__ void load_shifted(const uint8_t* a, int shift, uint32_t (&w)[W]) {
  if constexpr (W == 2) {
    // 8 bytes from a and, for a shift, from a + 8; the shift is below 8 here
    uint32_t q[4] = {0u, 0u, 0u, 0u};
    const uint2 lo = *reinterpret_cast<const uint2*>(a);
    q[0] = lo.x; q[1] = lo.y;
    if (shift != 0) {
      const uint2 hi = *reinterpret_cast<const uint2*>(a + 8);
      q[2] = hi.x; q[3] = hi.y;
    }
    if (shift & 4) { q[0] = q[1]; q[1] = q[2]; q[2] = q[3]; }
    if (shift & 2) {
      q[0] = __funnelshift_r(q[0], q[1], 16);
      q[1] = __funnelshift_r(q[1], q[2], 16);
    }
    w[0] = q[0]; w[1] = q[1];
  } else {
    uint32_t q[W + 4];
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(a)[i];
      q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
    }
    q[W] = q[W + 1] = q[W + 2] = q[W + 3] = 0u;
    if (shift != 0) {
      const uint4 v = reinterpret_cast<const uint4*>(a)[W / 4];
      q[W] = v.x; q[W + 1] = v.y; q[W + 2] = v.z; q[W + 3] = v.w;
    }
    if (shift & 8) {
#pragma unroll
      for (int i = 0; i < W + 2; ++i) q[i] = q[i + 2];
    }
    if (shift & 4) {
#pragma unroll
      for (int i = 0; i < W + 1; ++i) q[i] = q[i + 1];
    }
    if (shift & 2) {
#pragma unroll
      for (int i = 0; i < W; ++i) q[i] = __funnelshift_r(q[i], q[i + 1], 16);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = q[i];
  }
}

// n elements from c0 on, times k. The vectors are the output's 16-byte words; what they read
// starts anywhere in the input's words (a gradient's place in a flat buffer seldom shares the
// gradient's own alignment), so a thread reads the one or two words around its elements, the
// second mostly from L1, and shifts. Elements before the first and behind the last output word
// whose input words lie inside the chunk go one by one.
template <bool IN16, bool OUT16>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, int64_t c0, int n, float k) {
  constexpr int VEC = OUT16 ? 8 : 4;                  // elements of an output word
  constexpr int IS = IN16 ? 2 : 4;
  constexpr int W = VEC * IS / 4;                     // 32-bit input words of them
  constexpr int GRAIN = W == 2 ? 8 : 16;              // bytes of an input load
  const uint8_t* src = reinterpret_cast<const uint8_t*>(in) + c0 * IS;
  uint8_t* dst = reinterpret_cast<uint8_t*>(out) + c0 * (OUT16 ? 2 : 4);
  int head = (int)((16u - ((uint32_t)(uintptr_t)dst & 15u)) & 15u) / (OUT16 ? 2 : 4);
  const int shift = (int)((uintptr_t)(src + head * IS) & (GRAIN - 1));
  if (head * IS < shift) head += VEC;                 // the first input word starts in the chunk
  // the last input word ends in the chunk
  const int words = max(0, (n - head - (shift != 0 ? (GRAIN - shift) / IS : 0)) / VEC);
  const uint8_t* a = src + head * IS - shift;
  uint8_t* o = dst + head * (OUT16 ? 2 : 4);
#pragma unroll 1
  for (int i = threadIdx.x; i < words; i += kBlock) {
    uint32_t w[W];
    load_shifted<W>(a + (int64_t)i * VEC * IS, shift, w);
    float v[VEC];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (IN16) {
        v[2 * j] = k * __uint_as_float(w[j] << 16);
        v[2 * j + 1] = k * __uint_as_float(w[j] & 0xffff0000u);
      } else {
        v[j] = k * __uint_as_float(w[j]);
      }
    }
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (OUT16)
        r[j] = (uint32_t)f32_to_bf16_rn(v[2 * j]) | ((uint32_t)f32_to_bf16_rn(v[2 * j + 1]) << 16);
      else
        r[j] = __float_as_uint(v[j]);
    }
    reinterpret_cast<uint4*>(o)[i] = make_uint4(r[0], r[1], r[2], r[3]);
  }
  // both ends: fewer than 2 * 16 elements each, or the whole of a short chunk
  const int tail = words > 0 ? head + words * VEC : 0;
  const int singles = words > 0 ? head + n - tail : n;
  for (int i = threadIdx.x; i < singles; i += kBlock) {
    const int e = words > 0 && i >= head ? tail + i - head : i;
    const float v = k * load_elem<IN16>(src, e);
    if constexpr (OUT16) reinterpret_cast<uint16_t*>(dst)[e] = f32_to_bf16_rn(v);
    else reinterpret_cast<float*>(dst)[e] = v;
  }
}

template <int N>
__global__ void __launch_bounds__(kBlock, kBlocksPerSm)
    grad_scale_kernel(const __grid_constant__ GradTable<N> t, const float* norm, float max_norm) {
  pdl_wait();
  const float c = max_norm / (*norm + 1e-6f);
  const float k = c > 1.0f ? 1.0f : c;  // NaN stays NaN
  const int ch = (int)blockIdx.x;  // one block per chunk
  const int i = tensor_of(t, ch);
  const int64_t c0 = (int64_t)(ch - t.first[i]) * kChunk;
  const int n = (int)min((int64_t)kChunk, t.n[i] - c0);
  // a factor of 1 leaves a tensor that is scaled in place as it is
  if (k != 1.0f || t.in[i] != t.out[i]) {
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

template <int N>
cudaError_t norm_lists(const GradTensor* list, int64_t n, double* partials, unsigned* ticket,
                       float* norm, cudaStream_t stream) {
  GradTable<N> t;
  int64_t at = 0;
  bool first = true;
  do {
    at = fill(t, list, at, n);
    const int most = std::min(kBlocksPerSm * num_sms(), kGradNormMaxBlocks);
    const int grid = std::max(1, std::min(t.first[t.count], most));
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
    const cudaError_t e = launch_kernel(grad_scale_kernel<N>, dim3((unsigned)t.first[t.count]),
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
