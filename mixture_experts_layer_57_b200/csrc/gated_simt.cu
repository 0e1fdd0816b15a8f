// The gated expert FFN (forward and backward) on fp32 FMA units, for fp32 layers (no TF32).
//
//     forward    h[r, i]  = act(zg) * zu,  zg = Wg[e][i] . x[r] + bg,  zu = Wu[e][i] . x[r] + bu
//                y[r, :]  = Wd[e] h[r, :] + bd
//     backward   dh[r, i] = sum_m dy[r, m] Wd[e][m, i],  du = dh act(zg),  dg = dh zu act'(zg)
//                dx[r, :] = Wg[e]^T dg[r, :] + Wu[e]^T du[r, :]
//                dWd[e] = dy^T h,  dWg[e] = dg^T x,  dWu[e] = du^T x   (sums over the rows of e)
//
// One tiled product serves all five: a block of 256 threads computes a BM x BN tile, each thread a
// (BM/16) x (BN/16) patch in registers as two column groups, from 16-deep slices of both operands
// in shared memory (k-major, so a thread reads its patch with 16-byte loads); the next slice is
// loaded into registers while the present one is multiplied. What bounds it: fp32 FMA issue.
// Every sum runs in index order in one thread, so results do not change from call to call.
#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kSliceK = 16;

// Which product; what A, B and the epilogue are.
constexpr int kOpUp = 0;      // A = x rows, B = Wg | Wu (half of the tile's columns each) -> h [, saved]
constexpr int kOpDown = 1;    // A = h rows, B = Wd -> y
constexpr int kOpHidden = 2;  // A = dy rows, B = Wd transposed -> dg, du
constexpr int kOpInput = 3;   // A = dg then du rows, B = Wg then Wu transposed -> dx
constexpr int kOpWeight = 4;  // A = dy | dg | du columns, B = h | x | x columns -> dWd | dWg | dWu

struct SimtArgs {
  const int32_t* offsets;
  int E, d, f, act;
  int64_t rows_max;
  const float *a0, *a1, *a2;   // A operands (row-major activations)
  const float *b0, *b1, *b2;   // B operands (weights, or activations for kOpWeight)
  const float *bias0, *bias1;
  const float *in0, *in1;      // kOpHidden: act(zg), zu act'(zg)
  float *out0, *out1, *out2;
  int* status;
};

template <int OP, int BM, int BN>
__global__ void __launch_bounds__(256) gated_simt_kernel(const SimtArgs p) {
  constexpr int TM = BM / 16, TN = BN / 16, HN = TN / 2;
  constexpr bool kAK = OP != kOpWeight;                 // A contiguous along k
  constexpr bool kBK = OP == kOpUp || OP == kOpDown;    // B contiguous along k
  constexpr int kCols = OP == kOpUp ? BN / 2 : BN;      // output columns per tile
  __shared__ __align__(16) float As[kSliceK][BM + 4];
  __shared__ __align__(16) float Bs[kSliceK][BN + 4];
  pdl_wait();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int d = p.d, f = p.f;

  // the tile: expert, column tile, and for kOpWeight the problem and row tile
  int e = blockIdx.z, n0 = blockIdx.x * kCols, which = 0, m_tile = blockIdx.y;
  if constexpr (OP == kOpWeight) {
    // problem 0: dWd [d, f]; problems 1 and 2: dWg, dWu [f, d]; tiles numbered in that order
    const int t0 = ((d + BM - 1) / BM) * ((f + BN - 1) / BN);
    const int t1 = ((f + BM - 1) / BM) * ((d + BN - 1) / BN);
    int t = blockIdx.x;
    if (t >= t0) {
      t -= t0;
      which = 1 + t / t1;
      t %= t1;
    }
    const int nt = ((which == 0 ? f : d) + BN - 1) / BN;
    m_tile = t / nt;
    n0 = (t - m_tile * nt) * BN;
    e = blockIdx.y;
  }
  int64_t s0 = p.offsets[e], s1 = p.offsets[e + 1];
  if (s0 < 0 || s1 < s0 || s1 > p.rows_max) {
    if (tid == 0) set_device_error(p.status, MOE_DEVERR_BAD_OFFSETS);
    s0 = s1 = 0;
  }
  const int64_t rows = s1 - s0;
  const int64_t M = OP == kOpWeight ? (which == 0 ? d : f) : rows;
  const int N = OP == kOpUp || OP == kOpHidden ? f
                : OP == kOpWeight              ? (which == 0 ? f : d)
                                               : d;
  const int64_t K = OP == kOpWeight ? rows : (OP == kOpUp || OP == kOpHidden ? d : f);
  constexpr int kPhases = OP == kOpInput ? 2 : 1;
  const int64_t slices = (K + kSliceK - 1) / kSliceK;
  const int64_t total = slices * kPhases;

  constexpr int kALoads = BM * kSliceK / 256, kBLoads = BN * kSliceK / 256;
  for (int64_t m0 = (int64_t)m_tile * BM; m0 < M;
       m0 += OP == kOpWeight ? M : (int64_t)gridDim.y * BM) {
    float acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = 0.0f;
    float ra[kALoads], rb[kBLoads];

    auto fetch = [&](int64_t s) {
      const int ph = kPhases == 2 && s >= slices ? 1 : 0;
      const int64_t k0 = (s - ph * slices) * kSliceK;
      const float* A = OP == kOpWeight ? (which == 0 ? p.a0 : (which == 1 ? p.a1 : p.a2))
                                       : (ph ? p.a1 : p.a0);
#pragma unroll
      for (int i = 0; i < kALoads; ++i) {
        const int id = tid + i * 256;
        const int mm = kAK ? id / kSliceK : id % BM, kk = kAK ? id % kSliceK : id / BM;
        const int64_t m = m0 + mm, k = k0 + kk;
        float v = 0.0f;
        if (m < M && k < K) v = kAK ? A[(s0 + m) * K + k] : A[(s0 + k) * M + m];
        ra[i] = v;
      }
#pragma unroll
      for (int i = 0; i < kBLoads; ++i) {
        const int id = tid + i * 256;
        const int nn = kBK ? id / kSliceK : id % BN, kk = kBK ? id % kSliceK : id / BN;
        const int64_t k = k0 + kk;
        float v = 0.0f;
        if constexpr (OP == kOpUp) {
          const int n = n0 + (nn < kCols ? nn : nn - kCols);
          if (n < N && k < K) v = (nn < kCols ? p.b0 : p.b1)[((int64_t)e * N + n) * K + k];
        } else {
          const int n = n0 + nn;
          if (n < N && k < K) {
            if constexpr (OP == kOpDown) v = p.b0[((int64_t)e * N + n) * K + k];
            else if constexpr (OP == kOpWeight)
              v = (which == 0 ? p.b0 : p.b1)[(s0 + k) * N + n];
            else v = (ph ? p.b1 : p.b0)[((int64_t)e * K + k) * N + n];
          }
        }
        rb[i] = v;
      }
    };
    auto put = [&]() {
#pragma unroll
      for (int i = 0; i < kALoads; ++i) {
        const int id = tid + i * 256;
        if constexpr (kAK) As[id % kSliceK][id / kSliceK] = ra[i];
        else As[id / BM][id % BM] = ra[i];
      }
#pragma unroll
      for (int i = 0; i < kBLoads; ++i) {
        const int id = tid + i * 256;
        if constexpr (kBK) Bs[id % kSliceK][id / kSliceK] = rb[i];
        else Bs[id / BN][id % BN] = rb[i];
      }
    };

    if (total > 0) fetch(0);
    for (int64_t s = 0; s < total; ++s) {
      __syncthreads();
      put();
      __syncthreads();
      if (s + 1 < total) fetch(s + 1);
#pragma unroll
      for (int kk = 0; kk < kSliceK; ++kk) {
        float av[TM], bv[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) av[i] = As[kk][ty * TM + i];
#pragma unroll
        for (int j = 0; j < HN; ++j) {
          bv[j] = Bs[kk][tx * HN + j];
          bv[HN + j] = Bs[kk][BN / 2 + tx * HN + j];
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
    }

#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = m0 + ty * TM + i;
      if (m >= M) continue;
      if constexpr (OP == kOpUp) {
#pragma unroll
        for (int j = 0; j < HN; ++j) {
          const int n = n0 + tx * HN + j;
          if (n >= N) continue;
          const float zg = acc[i][j] + (p.bias0 ? p.bias0[(int64_t)e * N + n] : 0.0f);
          const float zu = acc[i][HN + j] + (p.bias1 ? p.bias1[(int64_t)e * N + n] : 0.0f);
          float a, da;
          gate_act(zg, p.act, a, da);
          const int64_t o = (s0 + m) * N + n;
          p.out0[o] = a * zu;
          if (p.out1 != nullptr) {
            p.out1[o] = a;
            p.out2[o] = zu * da;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int n = n0 + (j < HN ? tx * HN + j : BN / 2 + tx * HN + j - HN);
          if (n >= N) continue;
          const float v = acc[i][j];
          if constexpr (OP == kOpDown) {
            p.out0[(s0 + m) * N + n] = v + (p.bias0 ? p.bias0[(int64_t)e * N + n] : 0.0f);
          } else if constexpr (OP == kOpHidden) {
            const int64_t o = (s0 + m) * N + n;
            const float a = p.in0[o], q = p.in1[o];
            p.out0[o] = v * q;  // dg
            p.out1[o] = v * a;  // du
          } else if constexpr (OP == kOpInput) {
            p.out0[(s0 + m) * N + n] = v;
          } else {
            float* out = which == 0 ? p.out0 : (which == 1 ? p.out1 : p.out2);
            out[((int64_t)e * M + m) * N + n] = v;
          }
        }
      }
    }
  }
  pdl_trigger();
}

// 128 x 128 tiles when they fill the SMs twice over, else 64 x 64: at 4 tiles of 128 the products
// of a small layer would use 4 SMs.
template <int OP>
cudaError_t launch_rows(const SimtArgs& p, int n_cols, int64_t capacity_hint, cudaStream_t stream) {
  if (p.rows_max == 0) return cudaSuccess;
  int64_t m_ext = capacity_hint < 1 ? 1 : capacity_hint;
  if (m_ext > p.rows_max) m_ext = p.rows_max;
  auto blocks = [&](int bm, int bn) {
    const int cols = OP == kOpUp ? bn / 2 : bn;
    int64_t my = (m_ext + bm - 1) / bm;
    if (my > 65535) my = 65535;
    return dim3((unsigned)((n_cols + cols - 1) / cols), (unsigned)my, (unsigned)p.E);
  };
  const dim3 big = blocks(128, 128);
  if ((int64_t)big.x * big.y * big.z >= 2 * num_sms())
    return launch_kernel(gated_simt_kernel<OP, 128, 128>, big, dim3(256), 0, stream, p);
  return launch_kernel(gated_simt_kernel<OP, 64, 64>, blocks(64, 64), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t enqueue_gated_up_f32(const GatedFfn& g, float* h, float* saved_a, float* saved_q,
                                 int* status, cudaStream_t stream) {
  SimtArgs p{};
  p.offsets = g.offsets; p.E = g.E; p.d = g.d; p.f = g.f; p.act = g.act; p.rows_max = g.rows_max;
  p.a0 = (const float*)g.x; p.b0 = (const float*)g.w_gate; p.b1 = (const float*)g.w_up;
  p.bias0 = (const float*)g.b_gate; p.bias1 = (const float*)g.b_up;
  p.out0 = h; p.out1 = saved_a; p.out2 = saved_q; p.status = status;
  return launch_rows<kOpUp>(p, g.f, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_down_f32(const GatedFfn& g, const float* h, float* y, int* status,
                                   cudaStream_t stream) {
  SimtArgs p{};
  p.offsets = g.offsets; p.E = g.E; p.d = g.d; p.f = g.f; p.rows_max = g.rows_max;
  p.a0 = h; p.b0 = (const float*)g.w_down; p.bias0 = (const float*)g.b_down;
  p.out0 = y; p.status = status;
  return launch_rows<kOpDown>(p, g.d, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_hidden_grad_f32(const GatedFfn& g, const float* dy, const float* saved_a,
                                          const float* saved_q, float* dg, float* du, int* status,
                                          cudaStream_t stream) {
  SimtArgs p{};
  p.offsets = g.offsets; p.E = g.E; p.d = g.d; p.f = g.f; p.rows_max = g.rows_max;
  p.a0 = dy; p.b0 = (const float*)g.w_down; p.in0 = saved_a; p.in1 = saved_q;
  p.out0 = dg; p.out1 = du; p.status = status;
  return launch_rows<kOpHidden>(p, g.f, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_input_grad_f32(const GatedFfn& g, const float* dg, const float* du,
                                         float* dx, int* status, cudaStream_t stream) {
  SimtArgs p{};
  p.offsets = g.offsets; p.E = g.E; p.d = g.d; p.f = g.f; p.rows_max = g.rows_max;
  p.a0 = dg; p.a1 = du; p.b0 = (const float*)g.w_gate; p.b1 = (const float*)g.w_up;
  p.out0 = dx; p.status = status;
  return launch_rows<kOpInput>(p, g.d, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_weight_grad_f32(const GatedFfn& g, const float* dy, const float* h,
                                          const float* dg, const float* du, float* dw_down,
                                          float* dw_gate, float* dw_up, int* status,
                                          cudaStream_t stream) {
  SimtArgs p{};
  p.offsets = g.offsets; p.E = g.E; p.d = g.d; p.f = g.f; p.rows_max = g.rows_max;
  p.a0 = dy; p.a1 = dg; p.a2 = du; p.b0 = h; p.b1 = (const float*)g.x;
  p.out0 = dw_down; p.out1 = dw_gate; p.out2 = dw_up; p.status = status;
  auto tiles = [&](int t) {
    const int64_t td = (g.d + t - 1) / t, tf = (g.f + t - 1) / t;
    return 3 * td * tf;
  };
  if (tiles(128) * g.E >= 2 * num_sms())
    return launch_kernel(gated_simt_kernel<kOpWeight, 128, 128>, dim3((unsigned)tiles(128), g.E),
                         dim3(256), 0, stream, p);
  return launch_kernel(gated_simt_kernel<kOpWeight, 64, 64>, dim3((unsigned)tiles(64), g.E),
                       dim3(256), 0, stream, p);
}

}  // namespace moe
