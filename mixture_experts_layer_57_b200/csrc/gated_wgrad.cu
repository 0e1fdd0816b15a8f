// Weight and bias gradients of the gated expert FFN (bf16 layers) on sm_100a tensor cores. For
// every expert e, over the rows r of its segment:
//     dWd[e][m][i] = sum_r dy[r][m] h[r][i]
//     dWg[e][i][j] = sum_r dg[r][i] x[r][j],   dWu[e][i][j] = sum_r du[r][i] x[r][j]
// in one persistent launch over the output tiles of all three. Both operands are read MN-major
// from the row-major activations (TMA boxes of 64 columns x 64 rows, 128-byte swizzle; no
// transposed copies).
//
// With some 100 rows an expert the sums are short and writing the gradients bounds the kernel.
// A pair of CTAs computes a 256 x 256 tile (cta_group::2, 128 rows of it in each), so a tile costs
// each CTA 32 KB of loads per 64 rows; gradients leave through shared memory as TMA stores of whole
// 128-byte lines, two in flight per warp, while the next tile's MMAs run into a second accumulator.
// 128 experts of 128 rows, d 1024, f 4096: 964 us (3.7 GB at 3.8 TB/s; 870 with every tile written
// to one place, 680 without the stores: what is left is the MMAs of two blocks a tile and their
// hand-overs). One CTA a tile and rows written through fp32 staging: 1050 us. 16 epilogue warps with
// one buffer: 947, but 14% slower where the products bound (8 experts, d 4096, f 14336: 3.4 ms).
//
// The last K block of a segment is loaded in boxes of 16 rows, the last of which may also hold rows
// of the next expert, whose values may be anything: each CTA clears its own in shared memory before
// the MMAs (K = 16 each). A warp of its own does that as soon as such a tail has landed (its loads
// count on a barrier of their own CTA, those of other blocks on the first CTA's), long before the
// MMAs of the blocks before are issued, and reports to the first CTA's `tail` barrier.
// Experts without rows get zeros.
#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTile = 256;       // rows and columns of a pair's output tile
constexpr int kHalf = 128;       // A columns (tile rows) and B columns that one CTA loads
constexpr int kBK = 64;          // rows per stage
constexpr int kUmmaK = 16;
constexpr int kEpiSets = 2;     // epilogue warps for each quarter of a CTA's rows
constexpr int kEpiWarps = 4 * kEpiSets;
constexpr int kThreads = 96 + 32 * kEpiWarps;  // TMA, MMA, tails, epilogue
constexpr int kBoxBytes = 64 * kBK * 2;  // one 64 x 64 bf16 box
constexpr int kABytes = kHalf * kBK * 2;
constexpr int kStageBytes = 2 * kABytes;
constexpr int kOutBytes = 32 * 128;      // 32 tile rows of one 128-byte line each
constexpr int kEpiBytes = kEpiWarps * 2 * kOutBytes;
constexpr int kStages = 5;
constexpr int kGroup = 8;               // rows of tiles walked together
constexpr int kTmemCols = 2 * kTile;
constexpr int kBarBytes = 8 * 32;
constexpr int kSmemBytes =
    1024 + kStages * kStageBytes + kEpiBytes + kBarBytes + 16;
static_assert(4 * kStages + 5 <= 32, "barrier area too small");
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

struct WgradMaps {
  CUtensorMap a[3], b[2];    // dy, dg, du; h, x: boxes of 64 rows
  CUtensorMap ta[3], tb[2];  // the same in boxes of 16 rows
  CUtensorMap out[3];        // dWd, dWg, dWu
};
struct WgradParams {
  const int32_t* offsets;
  int E, d, f;
  int64_t rows_max;
  int out_bf16;
  int* status;
};

// Output tile: problem (0 dWd, 1 dWg, 2 dWu), expert, first row and column, the problem's sizes,
// the segment's first row and row count.
struct WTile {
  int which, e, m0, n0, M, N, row0, rows;
};

// The tiles of one pair: every `step`-th from `first` on. An expert's tiles are those of dWd, then
// those of dWg and dWu by turns (both read the same x columns); of a problem, kGroup rows of tiles
// at a time go column by column, so that the pairs at work share columns of both operands in L2.
// With short sums a tile is a microsecond's work: divisions are by multiplication and the segment's
// ends are kept while the expert stays.
struct Walk {
  int e = 0, step, row0 = 0, rows = 0;
  unsigned u, td, tf, per;  // u: tile within the expert; tiles along d and f and their product
  __device__ __forceinline__ Walk(const WgradParams& p, int first, int s) : step(s), u(first) {
    td = (unsigned)(p.d + kTile - 1) / kTile;
    tf = (unsigned)(p.f + kTile - 1) / kTile;
    per = td * tf;
    e = -1;
    u += 3 * per;  // settle() steps into expert 0
    settle(p);
  }
  __device__ __forceinline__ void settle(const WgradParams& p) {
    if (u < 3 * per) return;
    while (u >= 3 * per) {
      u -= 3 * per;
      ++e;
    }
    if (e < p.E) {
      int a = p.offsets[e], b = p.offsets[e + 1];
      if (a < 0 || b < a || (int64_t)b > p.rows_max) a = b = 0;  // invalid: treated as empty
      row0 = a;
      rows = b - a;
    }
  }
  __device__ __forceinline__ bool valid(const WgradParams& p) const { return e < p.E; }
  __device__ __forceinline__ void next(const WgradParams& p) {
    u += step;
    settle(p);
  }
  __device__ __forceinline__ WTile tile(const WgradParams& p) const {
    WTile w;
    w.e = e;
    w.row0 = row0;
    w.rows = rows;
    unsigned v = u, mt = td, nt = tf;
    w.which = 0;
    w.M = p.d;
    w.N = p.f;
    if (u >= per) {
      v = u - per;
      w.which = 1 + (int)(v & 1u);
      v >>= 1;
      w.M = p.f;
      w.N = p.d;
      mt = tf;
      nt = td;
    }
    // v < 2^24 in any gradients that fit in memory (256 x 256 elements to a tile, or widths up to 2^29)
    const unsigned band = kGroup * nt, g = div_small(v, band);
    v -= g * band;
    const unsigned high = min((unsigned)kGroup, mt - g * kGroup), n = div_small(v, high);
    w.m0 = (int)(g * kGroup + v - n * high) * kTile;
    w.n0 = (int)n * kTile;
    return w;
  }
  // v / by: a float quotient, exact to 2^-22 of it, so off by one step at most below 2^22, put right
  static __device__ __forceinline__ unsigned div_small(unsigned v, unsigned by) {
    unsigned q = (unsigned)__fdividef((float)v, (float)by);
    if (q * by > v) --q;
    if ((q + 1) * by <= v) ++q;
    return q;
  }
};

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, int* status) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      set_device_error(status, MOE_DEVERR_TIMEOUT);
      return;
    }
  }
}

// Whether a K block with `left` rows of its segment to go holds rows to clear.
__device__ __forceinline__ bool has_tail(int left) { return left < kBK && (left & (kUmmaK - 1)) != 0; }

// The uses of each stage by whole blocks and by tails, which count on different barriers: next()
// gives the parity of the next one's phase, last() that of the last one's.
struct Uses {
  uint32_t phase[2] = {0, 0}, any[2] = {0, 0};  // bits: stages
  __device__ __forceinline__ uint32_t next(int stage, bool tail) {
    const uint32_t parity = phase[tail] >> stage & 1u;
    phase[tail] ^= 1u << stage;
    any[tail] |= 1u << stage;
    return parity;
  }
  __device__ __forceinline__ uint32_t last(int stage, bool tail) const {
    return (phase[tail] >> stage & 1u) ^ 1u;
  }
};

// Clears this CTA's stage rows from `valid` to the next multiple of 16 (whole warp). A row of an
// MN-major box is 128 contiguous bytes; the swizzle permutes 16-byte chunks inside it.
__device__ __forceinline__ void clear_tail(uint8_t* stage, int valid, int lane) {
  const int chunks = (kUmmaK - valid % kUmmaK) * 8;
#pragma unroll
  for (int bx = 0; bx < kStageBytes / kBoxBytes; ++bx)
    for (int c = lane; c < chunks; c += 32)
      *reinterpret_cast<uint4*>(stage + bx * kBoxBytes + valid * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    gated_wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_addr - raw_addr);
  uint8_t* aux = base + kStages * kStageBytes + kEpiBytes;
  const uint32_t bars = smem_u32(aux);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(aux + kBarBytes);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(aux + kBarBytes + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  constexpr int S = kStages;
  auto full_bar = [&](int s) { return bars + 8u * s; };  // of the first CTA: both CTAs' loads
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto landed_bar = [&](int s) { return bars + 8u * (2 * S + s); };  // this CTA's loads of a tail
  auto tail_bar = [&](int s) { return bars + 8u * (3 * S + s); };  // of the first CTA: both cleared
  auto tfull_bar = [&](int a) { return bars + 8u * (4 * S + a); };
  auto tempty_bar = [&](int a) { return bars + 8u * (4 * S + 2 + a); };  // of the first CTA
  const uint32_t drain_bar = bars + 8u * (4 * S + 4);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(landed_bar(s), 1);
      mbar_init(tail_bar(s), 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      Uses uses;
      bool ok = true;
      for (Walk walk(p, first, step); walk.valid(p) && ok; walk.next(p)) {
        const WTile w = walk.tile(p);
        const int bi = w.which == 0 ? 0 : 1;
        const int m0 = w.m0 + rank * kHalf, n0 = w.n0 + rank * kHalf;
        for (int r = 0; r < w.rows; r += kBK) {
          if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t sa = base_addr + stage * kStageBytes;
          const int valid = w.rows - r;
          const uint32_t bytes = valid >= kBK ? kStageBytes : (uint32_t)(valid + 15) / 16 * 16 * 2 * kHalf * 2;
          const bool tail = has_tail(valid);
          const uint32_t bar = tail ? landed_bar(stage) : full_bar(stage);
          const uint32_t count_on = cluster_addr(bar, tail ? rank : 0);
          if (tail || rank == 0) mbar_arrive_expect_tx(bar, tail ? bytes : 2 * bytes);
          uses.next(stage, tail);
          const int rows16 = valid >= kBK ? 0 : (valid + 15) / 16;
#pragma unroll
          for (int j = 0; j < kHalf / 64; ++j) {
            const uint32_t da = sa + j * kBoxBytes, db = sa + kABytes + j * kBoxBytes;
            if (rows16 == 0) {
              tma_load_2d_pair(da, &maps.a[w.which], m0 + 64 * j, w.row0 + r, count_on);
              tma_load_2d_pair(db, &maps.b[bi], n0 + 64 * j, w.row0 + r, count_on);
            } else {
#pragma unroll 1
              for (int i = 0; i < rows16; ++i) {
                tma_load_2d_pair(da + i * 2048, &maps.ta[w.which], m0 + 64 * j, w.row0 + r + 16 * i, count_on);
                tma_load_2d_pair(db + i * 2048, &maps.tb[bi], n0 + 64 * j, w.row0 + r + 16 * i, count_on);
              }
            }
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // drain: the loads of the last uses may still be landing
      for (int s = 0; s < S; ++s) {
        if (rank == 0 && uses.any[0] >> s & 1u) wait_drain(full_bar(s), uses.last(s, false), p.status);
        if (uses.any[1] >> s & 1u) wait_drain(landed_bar(s), uses.last(s, true), p.status);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      int stage = 0, acc = 0;
      uint32_t acc_phase = 0;
      Uses uses;
      bool ok = true;
      const uint32_t idesc = idesc_bf16_f32_major(kTile, kTile, true, true);
      for (Walk walk(p, first, step); walk.valid(p) && ok; walk.next(p)) {
        if (!mbar_wait_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kTile);
        for (int left = walk.rows; left > 0; left -= kBK) {
          const bool tail = has_tail(left);
          const uint32_t parity = uses.next(stage, tail);
          ok = tail ? mbar_wait_cluster(tail_bar(stage), parity, abort_flag, p.status)
                    : mbar_wait_bounded(full_bar(stage), parity, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = base_addr + stage * kStageBytes;
          const uint64_t adesc = smem_desc_sw128_mn(sa);
          const uint64_t bdesc = smem_desc_sw128_mn(sa + kABytes);
#pragma unroll
          for (int kk = 0; kk < kBK / kUmmaK; ++kk)
            if (kk * kUmmaK < left)
              tc_mma_bf16_pair(d_tmem, adesc + (uint64_t)(kk * (kMnKStepBytes >> 4)),
                               bdesc + (uint64_t)(kk * (kMnKStepBytes >> 4)), idesc,
                               left != walk.rows || kk != 0 ? 1u : 0u);
          tc_commit_pair_both(empty_bar(stage), cluster_addr(empty_bar(stage), 1));
          if (++stage == S) stage = 0;
        }
        if (!ok) break;
        tc_commit_pair_both(tfull_bar(acc), cluster_addr(tfull_bar(acc), 1));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      tc_commit_pair_local(drain_bar);
      wait_drain(drain_bar, 0, p.status);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------- tails
    int stage = 0;
    Uses uses;
    bool ok = true;
    for (Walk walk(p, first, step); walk.valid(p) && ok; walk.next(p)) {
      for (int left = walk.rows; left > 0; left -= kBK) {
        if (has_tail(left)) {
          ok = mbar_wait_warp(landed_bar(stage), uses.next(stage, true), abort_flag, p.status);
          if (!ok) break;
          clear_tail(base + stage * kStageBytes, left, lane);
          if (lane == 0) mbar_arrive_cluster(cluster_addr(tail_bar(stage), 0));
        }
        if (++stage == S) stage = 0;
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    // this warp's 32 tile rows, every kEpiSets-th line of 128 bytes: each lane writes its row's 128
    // bytes into one of the warp's buffers, and one lane stores that
    const int quarter = warp & 3;
    const int set = (warp - 3) >> 2;
    const int cols = p.out_bf16 ? 64 : 32;  // of a line
    const int buf0 = kStages * kStageBytes + (warp - 3) * 2 * kOutBytes;
    int acc = 0, buf = 0;
    uint32_t acc_phase = 0;
    for (Walk walk(p, first, step); walk.valid(p); walk.next(p)) {
      const WTile w = walk.tile(p);
      const bool empty = w.rows == 0;  // nothing was accumulated: the tile is zero
      const int m = w.m0 + rank * kHalf + quarter * 32;  // first row of this warp
      if (!mbar_wait_warp(tfull_bar(acc), acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kTile);
      const int n_end = m < w.M ? min(kTile, w.N - w.n0) : 0;
      // the accumulator is free once this warp has read its last columns; one arrival per warp, as
      // the barrier takes arrivals one after another
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(tempty_bar(acc), 0));
      };
      if (set * cols >= n_end) release();
#pragma unroll 1
      for (int c0 = set * cols; c0 < n_end; c0 += kEpiSets * cols) {
        uint32_t line[32];
        if (p.out_bf16) {
          uint32_t r[4][16];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x16(taddr + (uint32_t)(c0 + 16 * q), r[q]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_ld_wait16(r[q]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              line[8 * q + i] = pack_bf16x2(__uint_as_float(r[q][2 * i]), __uint_as_float(r[q][2 * i + 1]));
          }
        } else {
          uint32_t r[2][16];
#pragma unroll
          for (int q = 0; q < 2; ++q) tmem_ld_32x32b_x16(taddr + (uint32_t)(c0 + 16 * q), r[q]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            tmem_ld_wait16(r[q]);
#pragma unroll
            for (int i = 0; i < 16; ++i) line[16 * q + i] = r[q][i];
          }
        }
        if (c0 + kEpiSets * cols >= n_end) release();
        if (lane == 0) bulk_wait_read<1>();  // the buffer's last store has read it
        __syncwarp();
        uint8_t* row = base + buf0 + buf * kOutBytes + lane * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(row + ((c ^ (lane & 7)) << 4)) =
              empty ? make_uint4(0u, 0u, 0u, 0u)
                    : make_uint4(line[4 * c], line[4 * c + 1], line[4 * c + 2], line[4 * c + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.out[w.which], base_addr + buf0 + buf * kOutBytes, w.n0 + c0, m, w.e);
          bulk_commit();
        }
        buf ^= 1;
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncwarp();
  cluster_sync();  // no commit or arrive targets the other CTA after this
  pdl_trigger();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
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
#pragma unroll 8
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

// Row splits: a thread adds its rows one after another, so few experts' rows are cut into some 200
// parts of 32 rows or more (17 experts, 1637 rows, 6520 columns:
// 16 us and 4 to join, 26 and 4 with parts of 256).
int bias_splits(int E, int64_t rows_max) {
  const int64_t per = (rows_max + 31) / 32;
  int64_t s = (200 + E - 1) / E;
  if (s > 64) s = 64;
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
  // gradients [E, M, N], stored in boxes of 32 rows of one 128-byte line
  auto grad_map = [&](CUtensorMap* map, const void* ptr, int M, int N) {
    const cuuint64_t size = grad_bf16 ? 2 : 4;
    const cuuint64_t extent[3] = {(cuuint64_t)N, (cuuint64_t)M, (cuuint64_t)g.E};
    const cuuint64_t stride[2] = {N * size, (cuuint64_t)M * N * size};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / size), 32, 1};
    return gated_tensor_map(map, ptr, grad_bf16, 3, extent, stride, box);
  };
  const void* acts[5] = {dy, dg, du, h, g.x};
  const int cols[5] = {g.d, g.f, g.f, g.f, g.d};
  for (int i = 0; i < 5; ++i)
    if (!make_bf16_map_2d(i < 3 ? &m.a[i] : &m.b[i - 3], acts[i], g.rows_max, cols[i], 64, kBK) ||
        !make_bf16_map_2d(i < 3 ? &m.ta[i] : &m.tb[i - 3], acts[i], g.rows_max, cols[i], 64, 16))
      return cudaErrorInvalidValue;
  if (!grad_map(&m.out[0], dw_down, g.d, g.f) || !grad_map(&m.out[1], dw_gate, g.f, g.d) ||
      !grad_map(&m.out[2], dw_up, g.f, g.d))
    return cudaErrorInvalidValue;
  const WgradParams p{g.offsets, g.E, g.d, g.f, g.rows_max, grad_bf16 ? 1 : 0, status};
  static int attr_done[64] = {0};  // per device
  const cudaError_t e = ensure_dynamic_smem(gated_wgrad_kernel, kSmemBytes, attr_done);
  if (e != cudaSuccess) return e;
  return launch_kernel(gated_wgrad_kernel, dim3(num_sms() / 2 * 2), dim3(kThreads), kSmemBytes, stream,
                       m, p);
}

}  // namespace moe
