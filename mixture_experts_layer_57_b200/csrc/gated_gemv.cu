// The gated expert FFN of a few rows of an fp32 layer (a decode step), forward:
//     h[r, i] = act(Wg[e][i] . x[r] + bg) * (Wu[e][i] . x[r] + bu),   y[r, m] = Wd[e][m] . h[r] + bd
//
// Bound by the weights' stream: each is read once, for all rows of its expert, and used for as many
// products as there are rows, which the FMA units keep up with for a few. A warp computes one hidden
// feature (a row of Wg and one of Wu) or one output (a row of Wd), its lanes side by side along the row,
// sums in fp32 and then over the lanes: no tiles to fill, so every SM takes part. Against the split-tf32
// tiles (us a call, weights that fit in L2 resident): 700 x 2000 of one expert, 1 row 14 and 32, 4 rows
// 27 and 33, 5 rows 27 and 33, 8 rows 38 and 33; 2048 x 8192, 1 row 66 and 149 (3.0 TB/s), 3 rows 148
// and 149, 5 rows 161 and 150, 8 rows 250 and 150; 8 rows of 512 x 1024 22 and 25; 8 rows over 8 experts
// of 1024 x 4096, 75 and 221. So experts with more than five rows go to the tiles unless the layer is
// small (gated_gemv_f32_suits). bf16 layers stay on their tiles, which stream as fast
// (when this form was tried there, one row of 2048 x 8192, weights cold: 43 us this way, 40 on the
// tiles; four rows 69 and 40).
//
// Launch overlap: both kernels let their successor start at once, and a single expert's weights are
// asked into L2 before the wait for what comes before.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 8;  // K elements of a lane whose weights are loaded together

struct GemvArgs {
  const int32_t* offsets;
  int E, K, n_out, act;
  int64_t rows_max;
  const float *in, *w0, *w1, *b0, *b1;
  float* out;
  int* status;
};

// The segment that starts at row blockIdx.y: its expert (-1: none, or bad offsets, which are
// flagged) and its rows.
__device__ __forceinline__ int segment_at(const GemvArgs& p, int& rows) {
  __shared__ int found[2], bad;
  if (threadIdx.x == 0) {
    found[0] = -1;
    bad = 0;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += 32 * kWarps) {
    const int a = p.offsets[e], b = p.offsets[e + 1];
    if (a < 0 || b < a || (int64_t)b > p.rows_max) {
      bad = 1;
    } else if (a == (int)blockIdx.y && b > a) {
      found[0] = e;
      found[1] = b - a;
    }
  }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) set_device_error(p.status, MOE_DEVERR_BAD_OFFSETS);
    return -1;
  }
  rows = found[1];
  return found[0];
}

__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// NR: rows a segment may have. UP: both projections, activation and product; else one matrix.
template <int NR, bool UP>
__global__ void __launch_bounds__(32 * kWarps) gated_gemv_kernel(const GemvArgs p) {
  const int lane = threadIdx.x & 31, f = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (p.E == 1 && f < p.n_out) {
    // the one expert's rows, asked for while the predecessor still runs (nothing is read yet)
    for (int k = lane * 32; k < p.K; k += 32 * 32) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w0 + (int64_t)f * p.K + k));
      if constexpr (UP) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w1 + (int64_t)f * p.K + k));
    }
  }
  pdl_wait();
  pdl_trigger();
  int rows = 0;
  const int e = segment_at(p, rows);
  if (e < 0 || f >= p.n_out) return;
  const int64_t at = ((int64_t)e * p.n_out + f) * p.K;
  const float* w0 = p.w0 + at;
  const float* w1 = UP ? p.w1 + at : nullptr;
  const float* in = p.in + (int64_t)blockIdx.y * p.K;
  float g[NR], u[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) g[r] = u[r] = 0.0f;
  // kAhead weights of each matrix are under way before the first is used; plain loads, as the rows may
  // be written until the wait above is over
  int k = lane;
  auto part = [&](auto n) {
    constexpr int N = decltype(n)::value;
    float a[N], b[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      a[j] = w0[k + 32 * j];
      b[j] = UP ? w1[k + 32 * j] : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (r < rows) {
        const float* x = in + (int64_t)r * p.K + k;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float v = x[32 * j];
          g[r] = fmaf(a[j], v, g[r]);
          if constexpr (UP) u[r] = fmaf(b[j], v, u[r]);
        }
      }
    }
    k += 32 * N;
  };
#pragma unroll 1
  while (k + 32 * (kAhead - 1) < p.K) part(std::integral_constant<int, kAhead>());
#pragma unroll 1
  while (k < p.K) part(std::integral_constant<int, 1>());
  const int64_t bi = (int64_t)e * p.n_out + f;
  const float bg = p.b0 != nullptr ? p.b0[bi] : 0.0f, bu = UP && p.b1 != nullptr ? p.b1[bi] : 0.0f;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (r >= rows) break;
    float v = lane_sum(g[r]) + bg;
    if constexpr (UP) {
      const float zu = lane_sum(u[r]) + bu;
      float a, da;
      gate_act(v, p.act, a, da);
      v = a * zu;
    }
    if (lane == 0) p.out[((int64_t)blockIdx.y + r) * p.n_out + f] = v;
  }
}

template <bool UP>
cudaError_t launch(const GemvArgs& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.n_out + kWarps - 1) / kWarps), (unsigned)p.rows_max);
  const dim3 block(32 * kWarps);
  if (p.rows_max == 1) return launch_kernel(gated_gemv_kernel<1, UP>, grid, block, 0, stream, p);
  if (p.rows_max == 2) return launch_kernel(gated_gemv_kernel<2, UP>, grid, block, 0, stream, p);
  if (p.rows_max <= 4) return launch_kernel(gated_gemv_kernel<4, UP>, grid, block, 0, stream, p);
  return launch_kernel(gated_gemv_kernel<kGatedGemvRows, UP>, grid, block, 0, stream, p);
}

}  // namespace

bool gated_gemv_f32_suits(const GatedFfn& g) {
  constexpr int64_t kExpertRows = 5, kSmall = 1 << 19;  // the figures at the top
  return g.rows_max <= kGatedGemvRows &&
         (std::min(g.capacity_hint, g.rows_max) <= kExpertRows || (int64_t)g.d * g.f <= kSmall);
}

cudaError_t enqueue_gated_gemv_f32(const GatedFfn& g, float* h, float* y, int* status,
                                   cudaStream_t stream) {
  const auto f32 = [](const void* p) { return (const float*)p; };
  GemvArgs p{g.offsets, g.E, g.d, g.f, g.act, g.rows_max, f32(g.x), f32(g.w_gate), f32(g.w_up),
             f32(g.b_gate), f32(g.b_up), h, status};
  const cudaError_t e = launch<true>(p, stream);
  if (e != cudaSuccess) return e;
  p.K = g.f;
  p.n_out = g.d;
  p.in = h;
  p.w0 = f32(g.w_down);
  p.b0 = f32(g.b_down);
  p.w1 = p.b1 = nullptr;
  p.out = y;
  return launch<false>(p, stream);
}

}  // namespace moe
