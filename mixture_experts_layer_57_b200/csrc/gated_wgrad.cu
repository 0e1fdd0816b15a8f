// Weight and bias gradients of the gated expert FFN (bf16 layers) on sm_100a tensor cores. For
// every expert e, over the rows r of its segment:
//     dWd[e][m][i] = sum_r dy[r][m] h[r][i]
//     dWg[e][i][j] = sum_r dg[r][i] x[r][j],   dWu[e][i][j] = sum_r du[r][i] x[r][j]
// in one persistent launch over the output tiles of all three. Both operands are read MN-major
// from the row-major activations (TMA boxes of 64 columns x 64 rows, 128-byte swizzle; no
// transposed copies). The last K block of a segment also holds rows of the next expert, whose
// values may be anything: the rows past the segment, up to the next multiple of 16, are cleared
// in shared memory and only the MMAs (K = 16 each) that cover the segment are issued. Experts
// without rows get zeros.
#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 256;
constexpr int kBK = 64;          // rows per stage
constexpr int kUmmaK = 16;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kBoxBytes = 64 * kBK * 2;  // one 64 x 64 bf16 box
constexpr int kEpiRowFloats = 36;        // 32 columns + 4 pad (16-byte aligned rows)
constexpr int kABytes = kBM * kBK * 2;
constexpr int kStageBytes = kABytes + kBN * kBK * 2;
constexpr int kEpiStageBytes = kEpiWarps * 32 * kEpiRowFloats * 4;
constexpr int kStages = (200 * 1024 - kEpiStageBytes) / kStageBytes;
constexpr int kTmemCols = 2 * kBN;
constexpr int kBarBytes = 8 * 32;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpiStageBytes + kBarBytes + 16;
static_assert(2 * kStages + 5 <= 32, "barrier area too small");
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct WgradMaps {
  CUtensorMap dy, h, dg, du, x;
};
struct WgradParams {
  const int32_t* offsets;
  int E, d, f;
  int64_t rows_max;
  void *dw_down, *dw_gate, *dw_up;
  int out_bf16;
  int* status;
};

// Output tile: problem (0 dWd, 1 dWg, 2 dWu), expert, first row and column, the problem's sizes,
// the segment's first row and row count.
struct WTile {
  int which, e, m0, n0, M, N, row0, rows;
};

__device__ __forceinline__ WTile decode(int t, const WgradParams& p, int t_down, int t_up) {
  WTile w;
  const int per_e = t_down + 2 * t_up;
  w.e = t / per_e;
  int u = t - w.e * per_e;
  int nt;
  if (u < t_down) {
    w.which = 0;
    w.M = p.d;
    w.N = p.f;
    nt = (p.f + kBN - 1) / kBN;
  } else {
    // the gate's and the up projection's tiles alternate: both read the same x columns
    u -= t_down;
    w.which = 1 + (u & 1);
    u >>= 1;
    w.M = p.f;
    w.N = p.d;
    nt = (p.d + kBN - 1) / kBN;
  }
  const int mt = u / nt;
  w.m0 = mt * kBM;
  w.n0 = (u - mt * nt) * kBN;
  int a = p.offsets[w.e], b = p.offsets[w.e + 1];
  if (a < 0 || b < a || (int64_t)b > p.rows_max) a = b = 0;  // invalid: treated as empty
  w.row0 = a;
  w.rows = b - a;
  return w;
}

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, int* status) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      set_device_error(status, MOE_DEVERR_TIMEOUT);
      return;
    }
  }
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    gated_wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_addr - raw_addr);
  float* epi_stage = reinterpret_cast<float*>(base + kStages * kStageBytes);
  uint8_t* aux = base + kStages * kStageBytes + kEpiStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(aux);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(aux + kBarBytes);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(aux + kBarBytes + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr int S = kStages;
  auto full_bar = [&](int s) { return smem_u32(&bars[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&bars[S + s]); };
  auto tfull_bar = [&](int a) { return smem_u32(&bars[2 * S + a]); };
  auto tempty_bar = [&](int a) { return smem_u32(&bars[2 * S + 2 + a]); };
  const uint32_t drain_bar = smem_u32(&bars[2 * S + 4]);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kEpiWarps * 32);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int t_down = ((p.d + kBM - 1) / kBM) * ((p.f + kBN - 1) / kBN);
  const int t_up = ((p.f + kBM - 1) / kBM) * ((p.d + kBN - 1) / kBN);
  const int total = p.E * (t_down + 2 * t_up);

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const WTile w = decode(t, p, t_down, t_up);
        const CUtensorMap* ma = w.which == 0 ? &maps.dy : (w.which == 1 ? &maps.dg : &maps.du);
        const CUtensorMap* mb = w.which == 0 ? &maps.h : &maps.x;
        for (int r = 0; r < w.rows; r += kBK) {
          if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t sa = base_addr + stage * kStageBytes;
          mbar_arrive_expect_tx(full_bar(stage), kStageBytes);
#pragma unroll
          for (int j = 0; j < kBM / 64; ++j)
            tma_load_2d(sa + j * kBoxBytes, ma, w.m0 + 64 * j, w.row0 + r, full_bar(stage));
#pragma unroll
          for (int j = 0; j < kBN / 64; ++j)
            tma_load_2d(sa + kABytes + j * kBoxBytes, mb, w.n0 + 64 * j, w.row0 + r,
                        full_bar(stage));
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      for (int i = max(0, issued - S); i < issued; ++i)
        wait_drain(full_bar(i % S), (uint32_t)((i / S) & 1), p.status);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer (whole warp)
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    const uint32_t idesc = idesc_bf16_f32_major(kBM, kBN, true, true);
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const WTile w = decode(t, p, t_down, t_up);
      if (!mbar_wait_bounded_warp(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kBN);
      for (int r = 0; r < w.rows; r += kBK) {
        if (!mbar_wait_bounded_warp(full_bar(stage), phase, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = base_addr + stage * kStageBytes;
        const int valid = min(kBK, w.rows - r);
        const int kend = (valid + kUmmaK - 1) & ~(kUmmaK - 1);
        if (valid < kend) {
          // a row of an MN-major box is 128 contiguous bytes; the swizzle permutes 16-byte
          // chunks inside it
          uint8_t* sp = base + stage * kStageBytes;
          const int chunks = (kend - valid) * 8;
          for (int i = lane; i < (kBM + kBN) / 64 * chunks; i += 32) {
            const int bx = i / chunks, c = i - bx * chunks;
            *reinterpret_cast<uint4*>(sp + bx * kBoxBytes + valid * 128 + c * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          const uint64_t adesc = smem_desc_sw128_mn(sa);
          const uint64_t bdesc = smem_desc_sw128_mn(sa + kABytes);
          for (int kk = 0; kk < kend / kUmmaK; ++kk)
            tc_mma_bf16(d_tmem, adesc + (uint64_t)(kk * (kMnKStepBytes >> 4)),
                        bdesc + (uint64_t)(kk * (kMnKStepBytes >> 4)), idesc,
                        (r | kk) != 0 ? 1u : 0u);
          tc_commit(empty_bar(stage));
        }
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) tc_commit(tfull_bar(acc));
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) {
      tc_commit(drain_bar);
      wait_drain(drain_bar, 0, p.status);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue (warps 2..9)
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    float* st = epi_stage + (warp - 2) * 32 * kEpiRowFloats;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const WTile w = decode(t, p, t_down, t_up);
      const bool empty = w.rows == 0;  // nothing was accumulated: the tile is zero
      uint8_t* out = reinterpret_cast<uint8_t*>(
          w.which == 0 ? p.dw_down : (w.which == 1 ? p.dw_gate : p.dw_up));
      if (!mbar_wait_bounded_warp(tfull_bar(acc), acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      const int mw = w.m0 + quarter * 32;  // first row of this warp
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kBN);
      for (int c0 = half * 32; c0 < kBN; c0 += 64) {
        uint32_t r0[16], r1[16];
        tmem_ld_32x32b_x16(taddr + (uint32_t)c0, r0);
        tmem_ld_32x32b_x16(taddr + (uint32_t)c0 + 16, r1);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t* r = q < 4 ? r0 : r1;
          const int o = 4 * (q & 3);
          *reinterpret_cast<float4*>(st + lane * kEpiRowFloats + 4 * q) =
              empty ? make_float4(0.f, 0.f, 0.f, 0.f)
                    : make_float4(__uint_as_float(r[o]), __uint_as_float(r[o + 1]),
                                  __uint_as_float(r[o + 2]), __uint_as_float(r[o + 3]));
        }
        __syncwarp();
        if (p.out_bf16) {
          const int n = w.n0 + c0 + 8 * (lane & 3);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2);
            const int m = mw + rr;
            if (m < w.M && n < w.N) {
              const float4 v0 = *reinterpret_cast<const float4*>(st + rr * kEpiRowFloats + 8 * (lane & 3));
              const float4 v1 = *reinterpret_cast<const float4*>(st + rr * kEpiRowFloats + 8 * (lane & 3) + 4);
              uint4 v;
              v.x = (uint32_t)f32_to_bf16_rn(v0.x) | ((uint32_t)f32_to_bf16_rn(v0.y) << 16);
              v.y = (uint32_t)f32_to_bf16_rn(v0.z) | ((uint32_t)f32_to_bf16_rn(v0.w) << 16);
              v.z = (uint32_t)f32_to_bf16_rn(v1.x) | ((uint32_t)f32_to_bf16_rn(v1.y) << 16);
              v.w = (uint32_t)f32_to_bf16_rn(v1.z) | ((uint32_t)f32_to_bf16_rn(v1.w) << 16);
              *reinterpret_cast<uint4*>(out + 2 * (((int64_t)w.e * w.M + m) * w.N + n)) = v;
            }
          }
        } else {
          const int n = w.n0 + c0 + 4 * (lane & 7);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3);
            const int m = mw + rr;
            if (m < w.M && n < w.N)
              *reinterpret_cast<float4*>(out + 4 * (((int64_t)w.e * w.M + m) * w.N + n)) =
                  *reinterpret_cast<const float4*>(st + rr * kEpiRowFloats + 4 * (lane & 7));
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      mbar_arrive(tempty_bar(acc));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// Column sums over each segment's rows of up to three matrices side by side (blockIdx.x walks
// their columns in groups of 256 threads x VEC), rows split S ways (blockIdx.z).
//   S == 1: written to out in its type; else partial[(e * S + s) * n_all + column].
struct BiasParams {
  const void* src[3];
  void* out[3];
  int n[3], blocks[3];
  const int32_t* offsets;
  int64_t rows_max;
  int n_all, S, out_bf16;
  float* partial;
};

template <bool BF16>
__device__ __forceinline__ void store_grad(void* out, int64_t i, float v, int out_bf16) {
  if (out_bf16) reinterpret_cast<uint16_t*>(out)[i] = f32_to_bf16_rn(v);
  else reinterpret_cast<float*>(out)[i] = v;
}

// bf16 rows are read eight columns to a thread (n % 8 == 0); fp32 rows one column to a thread.
template <bool BF16>
__global__ void __launch_bounds__(128) gated_bias_grad_kernel(const BiasParams p) {
  pdl_wait();
  constexpr int VEC = BF16 ? 8 : 1;
  int blk = blockIdx.x, i = 0, col0 = 0;
  while (i < 2 && blk >= p.blocks[i]) {
    blk -= p.blocks[i];
    col0 += p.n[i];
    ++i;
  }
  const int n = p.n[i];
  const int c = (blk * 128 + (int)threadIdx.x) * VEC;
  const int e = blockIdx.y, s = blockIdx.z;
  int64_t a = p.offsets[e], b = p.offsets[e + 1];
  if (a < 0 || b < a || b > p.rows_max) a = b = 0;
  const int64_t chunk = (b - a + p.S - 1) / p.S;
  const int64_t r0 = a + s * chunk, r1 = min(b, r0 + chunk);
  if (c < n) {
    float acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.0f;
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
      if constexpr (BF16) {
        const uint4 q = *reinterpret_cast<const uint4*>(
            reinterpret_cast<const uint16_t*>(p.src[i]) + r * n + c);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          acc[2 * v] += __uint_as_float(w[v] << 16);
          acc[2 * v + 1] += __uint_as_float(w[v] & 0xffff0000u);
        }
      } else {
        acc[0] += reinterpret_cast<const float*>(p.src[i])[r * n + c];
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      if (p.S == 1) store_grad<BF16>(p.out[i], (int64_t)e * n + c + v, acc[v], p.out_bf16);
      else p.partial[((int64_t)e * p.S + s) * p.n_all + col0 + c + v] = acc[v];
    }
  }
  pdl_trigger();
}

// The S row splits added in order.
__global__ void __launch_bounds__(256) gated_bias_join_kernel(const BiasParams p) {
  pdl_wait();
  const int col = blockIdx.x * 256 + threadIdx.x, e = blockIdx.y;
  if (col < p.n_all) {
    float acc = 0.0f;
    for (int s = 0; s < p.S; ++s) acc += p.partial[((int64_t)e * p.S + s) * p.n_all + col];
    int i = 0, c = col;
    while (i < 2 && c >= p.n[i]) c -= p.n[i++];
    store_grad<true>(p.out[i], (int64_t)e * p.n[i] + c, acc, p.out_bf16);
  }
  pdl_trigger();
}

// Row splits: enough blocks to fill the SMs a few times when there are few experts.
int bias_splits(int E, int64_t rows_max) {
  const int64_t per = (rows_max + 255) / 256;  // 256 rows to a split at least
  int64_t s = (64 + E - 1) / E;
  if (s > per) s = per;
  return (int)(s < 1 ? 1 : s);
}

}  // namespace

int64_t gated_bias_grad_partials(int E, int d, int f, int64_t rows_max) {
  const int S = bias_splits(E, rows_max);
  return S == 1 ? 0 : (int64_t)E * S * (d + 2 * (int64_t)f);
}

cudaError_t enqueue_gated_bias_grad(const GatedBiasGrad& b, bool bf16, bool out_bf16,
                                    const int32_t* offsets, int E, int64_t rows_max,
                                    float* partial, cudaStream_t stream) {
  BiasParams p{};
  const int per_block = 128 * (bf16 ? 8 : 1);
  int k = 0, blocks = 0;
  for (int i = 0; i < 3; ++i) {
    if (b.out[i] == nullptr) continue;
    p.src[k] = b.src[i];
    p.out[k] = b.out[i];
    p.n[k] = b.n[i];
    p.blocks[k] = (b.n[i] + per_block - 1) / per_block;
    p.n_all += b.n[i];
    blocks += p.blocks[k++];
  }
  if (k == 0) return cudaSuccess;
  p.offsets = offsets;
  p.rows_max = rows_max;
  p.S = bias_splits(E, rows_max);
  p.out_bf16 = out_bf16 ? 1 : 0;
  p.partial = partial;
  const dim3 grid((unsigned)blocks, (unsigned)E, (unsigned)p.S);
  cudaError_t e = bf16 ? launch_kernel(gated_bias_grad_kernel<true>, grid, dim3(128), 0, stream, p)
                       : launch_kernel(gated_bias_grad_kernel<false>, grid, dim3(128), 0, stream, p);
  if (e != cudaSuccess || p.S == 1) return e;
  return launch_kernel(gated_bias_join_kernel, dim3((unsigned)((p.n_all + 255) / 256), (unsigned)E),
                       dim3(256), 0, stream, p);
}

cudaError_t enqueue_gated_weight_grad_bf16(const GatedFfn& g, const void* dy, const void* h,
                                           const void* dg, const void* du, void* dw_down,
                                           void* dw_gate, void* dw_up, bool grad_bf16, int* status,
                                           cudaStream_t stream) {
  WgradMaps m;
  if (!make_bf16_map_2d(&m.dy, dy, g.rows_max, g.d, 64, kBK) ||
      !make_bf16_map_2d(&m.h, h, g.rows_max, g.f, 64, kBK) ||
      !make_bf16_map_2d(&m.dg, dg, g.rows_max, g.f, 64, kBK) ||
      !make_bf16_map_2d(&m.du, du, g.rows_max, g.f, 64, kBK) ||
      !make_bf16_map_2d(&m.x, g.x, g.rows_max, g.d, 64, kBK))
    return cudaErrorInvalidValue;
  WgradParams p{g.offsets, g.E, g.d, g.f, g.rows_max, dw_down, dw_gate, dw_up, grad_bf16 ? 1 : 0,
                status};
  static int attr_done[64] = {0};  // per device
  const cudaError_t e = ensure_dynamic_smem(gated_wgrad_kernel, kSmemBytes, attr_done);
  if (e != cudaSuccess) return e;
  return launch_kernel(gated_wgrad_kernel, dim3(num_sms()), dim3(kThreads), kSmemBytes, stream, m,
                       p);
}

}  // namespace moe
