// The gated expert FFN (forward and backward) of fp32 layers on sm_100a tensor cores.
//
//     up      h[r, i]  = act(zg) * zu,  zg = Wg[e][i] . x[r] + bg,  zu = Wu[e][i] . x[r] + bu
//     down    y[r, :]  = Wd[e] h[r, :] + bd
//     hidden  dh[r, i] = sum_m dy[r, m] Wd[e][m, i],  du = dh act(zg),  dg = dh zu act'(zg)
//     input   dx[r, :] = Wg[e]^T dg[r, :] + Wu[e]^T du[r, :]
//     weight  dWd[e] = dy^T h,  dWg[e] = dg^T x,  dWu[e] = du^T x   (sums over the rows of e)
//
// Sums as exact as fp32 arithmetic's. Every factor is split in two tf32 numbers, hi = x rounded to
// 11 bits and lo = x - hi rounded to 11, together within 2^-23 of x, and a product is hi hi + hi lo +
// lo hi: lo lo, which is left out, is 2^-22 of it at most, of either sign. The tensor cores cut each
// sum towards zero instead of rounding it (measured: 31 additions of 1.94 2^-24 to 1 leave 1), which
// over a long sum would cost several bits. So hi hi and the other two, 2^-11 of it, have accumulators
// of their own, 64 of K are summed in TMEM at a time, and the epilogue warps add those sums in
// registers, rounded to nearest. Measured against 64 bits, relative to the whole output (1000 rows,
// d 501, f 1334): 5e-7, where fp32 FMAs in index order gave 9e-7.
//
// Operands have any width, so rows start on any multiple of 4 bytes, which no TMA copy can do: eight
// warps load them (the next block's while they split this one's), split, and write both parts
// K-major in the swizzled layout of the MMA. The lanes of the accumulator are the output's
// contiguous index, so stores go out as whole lines. Tiles are of 128 features and 128 or 64 rows, or
// 64 rows with K over clusters of four CTAs that exchange their sums (launch_walk chooses). What
// bounds it: the loads and splits, some 4000 cycles for 32 of K and 128 rows, 2800 for 64 rows, of which
// the tensor pipe is at work for 850; 30% of the issue slots are taken (148 tiles of 128 rows, K 2048).
// 4 experts, 1000 rows, d 501, f 1334: up 61 us, down 52 (tiles of fp32 FMAs: 123 and 115).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace moe {
namespace {

enum Op { kUp = 0, kDown = 1, kHidden = 2, kInput = 3, kWeight = 4 };

constexpr int kBM = 128;
constexpr int kBK = 32;                  // fp32 of K per stage: one 128-byte swizzle row
constexpr int kChunk = 2;                // K blocks per sum in TMEM
constexpr int kLoadWarps = 8, kEpiWarps = 8;
// One warp of MMAs: 17 warps, for which the register file leaves 96 a thread.
constexpr int kThreads = 32 * (kLoadWarps + 1 + kEpiWarps);
constexpr int kAPart = kBM * kBK * 4;    // one part (hi or lo) of A
constexpr int kBarBytes = 8 * 16;

// BN: token columns of a tile. SPLIT: CTAs of a cluster that share a tile, each with its part of the
// K blocks; each then finishes every SPLIT-th part of every epilogue warp's columns, for which all
// write their sums into its shared memory.
template <int BN, int SPLIT>
struct Cfg {
  static constexpr int kBPart = BN * kBK * 4;
  static constexpr int kStageBytes = 2 * kAPart + 2 * kBPart;  // A hi, A lo, B hi, B lo
  static constexpr int kCols = BN / 2;                         // columns of an epilogue warp
  static constexpr int kOwn = kCols / SPLIT;                   // that this CTA finishes
  static constexpr int kExchange = SPLIT > 1 ? kEpiWarps * kCols * 32 * 4 : 0;
  static constexpr int kStages = BN == 128 || SPLIT > 1 ? 3 : 4;
  static constexpr int kAccCols = 2 * BN;                      // hi hi, and the small products
  static constexpr int kTmemCols = 2 * kAccCols;               // two of both
  static constexpr int kSmemBytes =
      1024 + kStages * kStageBytes + kExchange + kBarBytes + 16 + 2 * 4 * (MOE_MAX_EXPERTS + 1);
  static_assert(kSmemBytes <= 227 * 1024 && kOwn % 2 == 0, "shared memory budget, halves of kUp");
  static_assert(2 * kStages + 7 <= kBarBytes / 8, "barrier area too small");
};

struct Args {
  const int32_t* offsets;
  int E, act;
  int64_t rows_max;
  int n_out;                 // output features (kWeight: unused)
  int K;                     // of each product (kWeight: unused, the segment's rows)
  int d, f;
  const float *a0, *a1;      // weights; kWeight: h, x
  const float *b0, *b1, *b2; // token rows; kWeight: dy, dg, du
  const float *bias0, *bias1;
  const float *in0, *in1;    // kHidden: act(zg), zu act'(zg)
  float *out0, *out1, *out2;
  int* status;
};

// A tile: lanes are output features f0.., columns token rows row0.. (kWeight: rows row0.. of the
// gradient `which`), n_valid of them, of expert e; n_out features, sums over K (twice for kInput).
struct Tile {
  int e, f0, row0, n_valid, which, n_out, K, seg;
};

template <int OP, int BN>
__device__ __forceinline__ int tile_count(const Args& p, const int* prefix) {
  if constexpr (OP != kWeight) return prefix[p.E];
  const int t0 = ((p.f + kBM - 1) / kBM) * ((p.d + BN - 1) / BN);
  const int t1 = ((p.d + kBM - 1) / kBM) * ((p.f + BN - 1) / BN);
  return p.E * (t0 + 2 * t1);
}

template <int OP, int BN>
__device__ __forceinline__ Tile tile_at(const Args& p, int t, const int* prefix, const int* seg) {
  Tile w;
  if constexpr (OP == kWeight) {
    // dWd [d, f], then dWg and dWu [f, d]: features are a gradient row's elements
    const int t0 = ((p.f + kBM - 1) / kBM) * ((p.d + BN - 1) / BN);
    const int t1 = ((p.d + kBM - 1) / kBM) * ((p.f + BN - 1) / BN);
    w.e = t / (t0 + 2 * t1);
    int u = t - w.e * (t0 + 2 * t1);
    w.which = u < t0 ? 0 : 1 + (u - t0) / t1;
    if (w.which != 0) u = (u - t0) % t1;
    w.n_out = w.which == 0 ? p.f : p.d;
    const int rows = w.which == 0 ? p.d : p.f;
    const int nt = (rows + BN - 1) / BN;
    w.f0 = u / nt * kBM;
    w.row0 = u % nt * BN;
    w.n_valid = min(BN, rows - w.row0);
    int a = p.offsets[w.e], b = p.offsets[w.e + 1];
    if (a < 0 || b < a || (int64_t)b > p.rows_max) a = b = 0;  // flagged by the passes before
    w.seg = a;
    w.K = b - a;
  } else {
    int lo = 0, hi = p.E;  // prefix[lo] <= t < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int rows = seg[lo + 1] - seg[lo], ntt = (rows + BN - 1) / BN;
    const int local = t - prefix[lo], ft = local / ntt, jt = local - ft * ntt;
    w.e = lo;
    w.f0 = ft * (OP == kUp ? kBM / 2 : kBM);
    w.row0 = seg[lo] + jt * BN;
    w.n_valid = min(BN, rows - jt * BN);
    w.which = 0;
    w.n_out = p.n_out;
    w.K = p.K;
    w.seg = 0;
  }
  return w;
}

template <int OP>
__device__ __forceinline__ int k_blocks(const Tile& w) {
  return (OP == kInput ? 2 : 1) * ((w.K + kBK - 1) / kBK);
}

// One warp: seg[e] and the first tile of every expert; none if the offsets are not non-decreasing
// within [0, rows_max], which is flagged.
template <int BN>
__device__ __forceinline__ void build_tile_list(const Args& p, int n_ftiles, int* prefix, int* seg,
                                                int lane) {
  int run = 0;
  bool bad = false;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane;
    int tiles = 0;
    if (e < p.E) {
      const int a = p.offsets[e], b = p.offsets[e + 1];
      seg[e] = a;
      if (a < 0 || b < a || (int64_t)b > p.rows_max) bad = true;
      else tiles = n_ftiles * ((b - a + BN - 1) / BN);
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (e < p.E) prefix[e] = run + incl - tiles;
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    seg[p.E] = p.offsets[p.E];
    prefix[p.E] = bad ? 0 : run;
    if (bad && blockIdx.x == 0) set_device_error(p.status, MOE_DEVERR_BAD_OFFSETS);
  }
}

// How a load thread's 16 elements of one operand's K block lie: four units of four neighbours along
// k, 16 bytes of the stage each.
//   kWide    rows are contiguous along k and start on 16 bytes: a load per unit, eight lanes to a
//            row, 32 rows from one unit to the next
//   kNarrow  rows are contiguous along k and start anywhere: the same in single loads (a row to a
//            warp and 32 lanes along k took 109 us for what takes 74: addresses and stores)
//   kAcross  contiguous along the tile's rows: the lanes in neighbouring rows
enum Walk { kWide, kNarrow, kAcross };

// Of a tile of R rows, R / 32 units a thread: row and 16-byte place of unit i.
template <int W, int R>
__device__ __forceinline__ int row_of(int tid, int i) {
  return W == kAcross ? tid % R : (tid >> 3) + 32 * i;
}
template <int W, int R>
__device__ __forceinline__ int place_of(int tid, int i) {
  return W == kAcross ? tid / R + (256 / R) * i : tid & 7;
}

// at: row_of(tid, 0) at k = 0; step: to the next unit's row; ld: kAcross: from one k to the next;
// ok: bit i: row_of(tid, i) exists.
template <int W, int R>
__device__ __forceinline__ void load_block(float (&v)[R / 8], const float* at, int64_t step, uint32_t ok,
                                           int64_t ld, int k0, int K, int tid) {
#pragma unroll
  for (int i = 0; i < R / 32; ++i) {
    const int k = k0 + place_of<W, R>(tid, i) * 4;
    const float* from = W == kAcross ? at + k * ld : at + i * step + k;
    const bool mine = (ok >> i & 1u) != 0;
    if constexpr (W == kWide) {
      const float4 q = mine && k < K ? *reinterpret_cast<const float4*>(from)  // K % 4 == 0
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
    } else if (k0 + kBK <= K) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = mine ? from[W == kAcross ? j * ld : j] : 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[4 * i + j] = mine && k + j < K ? from[W == kAcross ? j * ld : j] : 0.0f;
    }
  }
}

// hi: x rounded to 11 bits (tf32), lo: the exact rest, rounded to 11. Where one of the four is 2^127
// or more, infinite or NaN, both are cut instead: hi does not overflow, and of a NaN, whose payload may
// be cut from hi, x - hi is a NaN that lo keeps (rounding up would carry it into -0). x - hi is NaN for
// an infinite x too, so its sums are NaN. (A NaN made quiet in hi instead: the forward pass of 1000
// rows, d 501, f 1334, takes 132 us for 108.)
__device__ __forceinline__ void split4(const float* x, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(x[j])));
  const uint32_t half = m < 1.7014118346e38f ? 0x1000u : 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    hi[j] = (__float_as_uint(x[j]) + half) & 0xffffe000u;
    lo[j] = (__float_as_uint(x[j] - __uint_as_float(hi[j])) + half) & 0xffffe000u;
  }
}

template <int W, int R>
__device__ __forceinline__ void put_block(const float (&v)[R / 8], uint8_t* part, int tid) {
#pragma unroll
  for (int i = 0; i < R / 32; ++i) {
    const int row = row_of<W, R>(tid, i), place = place_of<W, R>(tid, i);
    uint32_t hi[4], lo[4];
    split4(v + 4 * i, hi, lo);
    uint8_t* at = part + row * 128 + ((place ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + R * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

__device__ __forceinline__ void tc_mma_tf32(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// What becomes of N sums of this lane's feature, of tile columns c0.. on.
template <int OP, int N>
__device__ __forceinline__ void finish(const Args& p, const Tile& w, const float (&s)[N], int c0, int quarter,
                                       int lane) {
  if constexpr (OP == kUp) {
    // zg and zu of a feature lie half a warp apart: the lower lanes take the first half of the
    // columns, the upper ones the second
    const int hi = lane >> 4, f = w.f0 + quarter * 16 + (lane & 15);
    const bool f_ok = f < w.n_out;
    const int64_t bi = (int64_t)w.e * w.n_out + f;
    const float bg = p.bias0 != nullptr && f_ok ? p.bias0[bi] : 0.0f;
    const float bu = p.bias1 != nullptr && f_ok ? p.bias1[bi] : 0.0f;
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
      const float own = hi ? s[N / 2 + c] : s[c];
      const float got = __shfl_xor_sync(0xffffffffu, hi ? s[c] : s[N / 2 + c], 16);
      const int col = c0 + hi * (N / 2) + c;
      if (f_ok && col < w.n_valid) {
        const float zg = (hi ? got : own) + bg, zu = (hi ? own : got) + bu;
        float a, da;
        gate_act(zg, p.act, a, da);
        const int64_t o = (int64_t)(w.row0 + col) * w.n_out + f;
        p.out0[o] = a * zu;
        if (p.out1 != nullptr) {
          p.out1[o] = a;
          p.out2[o] = zu * da;
        }
      }
    }
  } else {
    const int f = w.f0 + quarter * 32 + lane;
    if (f >= w.n_out) return;
    const float b = OP == kDown && p.bias0 != nullptr ? p.bias0[(int64_t)w.e * w.n_out + f] : 0.0f;
    float* out = OP == kWeight ? (w.which == 0 ? p.out0 : (w.which == 1 ? p.out1 : p.out2)) : p.out0;
    // kWeight: a gradient row of this expert
    const int64_t first = OP == kWeight ? (int64_t)w.e * (w.which == 0 ? p.d : p.f) : 0;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (c0 + c >= w.n_valid) break;
      const int64_t o = (first + w.row0 + c0 + c) * w.n_out + f;
      if constexpr (OP == kHidden) {
        const float a = p.in0[o], q = p.in1[o];
        p.out0[o] = s[c] * q;  // dg
        p.out1[o] = s[c] * a;  // du
      } else {
        out[o] = s[c] + b;
      }
    }
  }
}

template <int OP, bool WIDE, int BN, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1) gated_tf32_kernel(const Args p) {
  using C = Cfg<BN, SPLIT>;
  constexpr int kAlongK = WIDE ? kWide : kNarrow;
  constexpr int kWalkA = OP == kUp || OP == kDown ? kAlongK : kAcross;
  constexpr int kWalkB = OP == kWeight ? kAcross : kAlongK;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_addr - raw_addr);
  float* exchange = reinterpret_cast<float*>(base + C::kStages * C::kStageBytes);
  uint8_t* aux = base + C::kStages * C::kStageBytes + C::kExchange;
  const uint32_t bars = smem_u32(aux);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(aux + kBarBytes);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(aux + kBarBytes + 4);
  int* prefix = reinterpret_cast<int*>(aux + kBarBytes + 16);
  int* seg = prefix + (MOE_MAX_EXPERTS + 1);
  constexpr int S = C::kStages;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
  auto tfull_bar = [&](int a) { return bars + 8u * (2 * S + a); };
  auto tempty_bar = [&](int a) { return bars + 8u * (2 * S + 2 + a); };
  const uint32_t drain_bar = bars + 8u * (2 * S + 4);
  const uint32_t sums_bar = bars + 8u * (2 * S + 5);  // SPLIT: every CTA's sums are in `exchange`
  const uint32_t free_bar = bars + 8u * (2 * S + 6);  // and every CTA has read this one's
  const int rank = SPLIT > 1 ? (int)cluster_ctarank() : 0;
  const int first = (int)blockIdx.x / SPLIT, step = (int)gridDim.x / SPLIT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), kLoadWarps);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    mbar_init(sums_bar, SPLIT * kEpiWarps);
    mbar_init(free_bar, SPLIT * kEpiWarps);
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == kLoadWarps) {
    tmem_alloc(smem_u32(tmem_holder), C::kTmemCols);
    tmem_relinquish();
  }
  if (OP != kWeight && warp == 0) {
    constexpr int feat = OP == kUp ? kBM / 2 : kBM;
    build_tile_list<BN>(p, (p.n_out + feat - 1) / feat, prefix, seg, lane);
  }
  tc_fence_before();
  if constexpr (SPLIT > 1) {
    __syncwarp();
    cluster_sync();
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total = tile_count<OP, BN>(p, prefix);
  // this CTA's K blocks of a tile
  auto from = [&](const Tile& w) { return k_blocks<OP>(w) * rank / SPLIT; };
  auto until = [&](const Tile& w) { return k_blocks<OP>(w) * (rank + 1) / SPLIT; };

  if (warp < kLoadWarps) {
    // ---------------------------------------------------------- loads and splits
    const int tid = threadIdx.x;
    const float *a_at = nullptr, *b_at = nullptr;  // this thread's first rows, for k = 0
    uint32_t a_ok = 0, b_ok = 0;
    int64_t a_ld = 0, b_ld = 0;
    Tile w{};
    int t = first, kb = 0, n_kb = 0, blocks1 = 0;
    bool in_tile = false;
    // makes (t, kb) the next K block there is; false if there is none
    auto settle = [&]() {
      while (t < total && kb >= n_kb) {
        if (in_tile) t += step;
        in_tile = true;
        if (t >= total) return false;
        w = tile_at<OP, BN>(p, t, prefix, seg);
        kb = from(w);
        n_kb = until(w);
        blocks1 = (w.K + kBK - 1) / kBK;
        if (kb >= n_kb) continue;
        a_ok = b_ok = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rows of the A tile: features in order, for kUp 16 of the gate's and 16 of the up
          // projection's by turns
          const int row = row_of<kWalkA, kBM>(tid, i);
          if ((OP == kUp ? w.f0 + (row >> 5) * 16 + (row & 15) : w.f0 + row) < w.n_out)
            a_ok |= 1u << i;
          if (row_of<kWalkB, BN>(tid, i) < w.n_valid) b_ok |= 1u << i;
        }
        const int row = row_of<kWalkA, kBM>(tid, 0), col = row_of<kWalkB, BN>(tid, 0);
        if constexpr (OP == kUp) {
          a_at = (row & 16 ? p.a1 : p.a0) + ((int64_t)w.e * p.n_out + w.f0 + (row & 15)) * p.K;
        } else if constexpr (OP == kDown) {
          a_at = p.a0 + ((int64_t)w.e * p.n_out + w.f0 + row) * p.K;
        } else if constexpr (OP == kWeight) {
          a_at = (w.which == 0 ? p.a0 : p.a1) + (int64_t)w.seg * w.n_out + w.f0 + row;
          a_ld = w.n_out;
        } else {
          a_at = p.a0 + (int64_t)w.e * p.K * p.n_out + w.f0 + row;
          a_ld = p.n_out;
        }
        if constexpr (OP == kWeight) {
          b_ld = w.which == 0 ? p.d : p.f;
          b_at = (w.which == 0 ? p.b0 : (w.which == 1 ? p.b1 : p.b2)) + w.seg * b_ld + w.row0 + col;
        } else {
          b_at = p.b0 + ((int64_t)w.row0 + col) * p.K;
        }
      }
      return t < total;
    };
    auto load = [&](float (&a)[kBM / 8], float (&b)[BN / 8]) {
      // kInput's second product: the same places of the other operands
      const bool second = OP == kInput && kb >= blocks1;
      const int k0 = (kb - (second ? blocks1 : 0)) * kBK;
      load_block<kWalkA, kBM>(a, second ? p.a1 + (a_at - p.a0) : a_at, (int64_t)(OP == kUp ? 16 : 32) * p.K,
                              a_ok, a_ld, k0, w.K, tid);
      load_block<kWalkB, BN>(b, second ? p.b1 + (b_at - p.b0) : b_at, (int64_t)32 * p.K, b_ok, b_ld, k0, w.K,
                             tid);
      ++kb;
    };
    float av[kBM / 8] = {}, bv[BN / 8] = {}, an[kBM / 8] = {}, bn[BN / 8] = {};
    int stage = 0;
    uint32_t phase = 0;
    bool have = settle();
    if (have) load(av, bv);
    while (have) {
      const bool more = settle();
      if (more) load(an, bn);
      if (!mbar_wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) break;
      uint8_t* to = base + stage * C::kStageBytes;
      put_block<kWalkA, kBM>(av, to, tid);
      put_block<kWalkB, BN>(bv, to + 2 * kAPart, tid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full_bar(stage));
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
      }
#pragma unroll
      for (int i = 0; i < kBM / 8; ++i) av[i] = an[i];
#pragma unroll
      for (int i = 0; i < BN / 8; ++i) bv[i] = bn[i];
      have = more;
    }
  } else if (warp == kLoadWarps) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        const Tile w = tile_at<OP, BN>(p, t, prefix, seg);
        const int kb0 = from(w), kb1 = until(w);
        // D fp32, A and B tf32, K-major, N = the tile's columns in groups of 16
        const uint32_t idesc = (1u << 4) | (2u << 7) | (2u << 10) |
                               ((uint32_t)(((w.n_valid + 15) & ~15) >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
        for (int kb = kb0; kb < kb1; ++kb) {
          const bool begins = (kb - kb0) % kChunk == 0;
          if (begins) {
            if (!(ok = mbar_wait_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.status))) break;
            tc_fence_after();
          }
          if (!(ok = mbar_wait_bounded(full_bar(stage), phase, abort_flag, p.status))) break;
          tc_fence_after();
          const uint32_t sa = base_addr + stage * C::kStageBytes;
          const uint64_t a_hi = smem_desc_sw128(sa), a_lo = smem_desc_sw128(sa + kAPart);
          const uint64_t b_hi = smem_desc_sw128(sa + 2 * kAPart);
          const uint64_t b_lo = smem_desc_sw128(sa + 2 * kAPart + C::kBPart);
          const uint32_t d = tmem_base + (uint32_t)(acc * C::kAccCols);
          const uint32_t more = begins ? 0u : 1u;
#pragma unroll
          for (int kk = 0; kk < kBK / 8; ++kk) {
            tc_mma_tf32(d, a_hi + 2 * kk, b_hi + 2 * kk, idesc, kk != 0 ? 1u : more);
            tc_mma_tf32(d + BN, a_lo + 2 * kk, b_hi + 2 * kk, idesc, kk != 0 ? 1u : more);
            tc_mma_tf32(d + BN, a_hi + 2 * kk, b_lo + 2 * kk, idesc, 1u);
          }
          tc_commit(empty_bar(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
          if ((kb - kb0) % kChunk == kChunk - 1 || kb == kb1 - 1) {
            tc_commit(tfull_bar(acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
          }
        }
      }
      // drain every MMA this thread issued before TMEM is released
      tc_commit(drain_bar);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(drain_bar, 0))
        if (global_timer_ns() - t0 > kWaitLimitNs) {
          set_device_error(p.status, MOE_DEVERR_TIMEOUT);
          break;
        }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- epilogue: half of the columns each
    const int quarter = warp & 3, c0 = (warp - kLoadWarps - 1) / 4 * C::kCols;
    int acc = 0;
    uint32_t acc_phase = 0, exchange_phase = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const Tile w = tile_at<OP, BN>(p, t, prefix, seg);
      const int chunks = (until(w) - from(w) + kChunk - 1) / kChunk;
      float s[C::kCols];
#pragma unroll
      for (int c = 0; c < C::kCols; ++c) s[c] = 0.0f;
      for (int k = 0; k < chunks; ++k) {
        if (!(ok = mbar_wait_warp(tfull_bar(acc), acc_phase, abort_flag, p.status))) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * C::kAccCols + c0);
#pragma unroll
        for (int g = 0; g < C::kCols / 16; ++g) {
          if (c0 + g * 16 < w.n_valid) {
            uint32_t r[16];
#pragma unroll
            for (int part = 1; part >= 0; --part) {
              tmem_ld_32x32b_x16(taddr + (uint32_t)(part * BN + g * 16), r);
              tmem_ld_wait16(r);
#pragma unroll
              for (int c = 0; c < 16; ++c) s[g * 16 + c] += __uint_as_float(r[c]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) break;
      if constexpr (SPLIT == 1) {
        if (c0 < w.n_valid) finish<OP, C::kCols>(p, w, s, c0, quarter, lane);
      } else {
        // [SPLIT senders][8 warps][kOwn columns][32 lanes] in the CTA that finishes the columns, once
        // all have read the tile before's
        if (!mbar_wait_cluster_warp(free_bar, exchange_phase ^ 1u, abort_flag, p.status)) break;
        const int ew = warp - kLoadWarps - 1;
        const uint32_t mine = smem_u32(exchange) + (uint32_t)((rank * kEpiWarps + ew) * C::kOwn * 32 + lane) * 4;
#pragma unroll
        for (int o = 0; o < SPLIT; ++o) {
          const uint32_t to = cluster_addr(mine, o);
#pragma unroll
          for (int c = 0; c < C::kOwn; ++c)
            st_cluster_u32(to + c * 128, __float_as_uint(s[o * C::kOwn + c]));
        }
        __syncwarp();
        if (lane == 0)
          for (int o = 0; o < SPLIT; ++o) mbar_arrive_cluster(cluster_addr(sums_bar, o));
        if (!mbar_wait_cluster_warp(sums_bar, exchange_phase, abort_flag, p.status)) break;
        float v[C::kOwn];
#pragma unroll
        for (int c = 0; c < C::kOwn; ++c) {
          v[c] = 0.0f;
#pragma unroll
          for (int o = 0; o < SPLIT; ++o)
            v[c] += exchange[((o * kEpiWarps + ew) * C::kOwn + c) * 32 + lane];
        }
        __syncwarp();
        if (lane == 0)
          for (int o = 0; o < SPLIT; ++o) mbar_arrive_cluster(cluster_addr(free_bar, o));
        exchange_phase ^= 1u;
        const int col = c0 + rank * C::kOwn;
        if (col < w.n_valid) finish<OP, C::kOwn>(p, w, v, col, quarter, lane);
      }
    }
  }

  tc_fence_before();
  if constexpr (SPLIT > 1) {
    __syncwarp();
    cluster_sync();  // no store or arrive targets another CTA after this
  } else {
    __syncthreads();
  }
  pdl_trigger();
  if (warp == kLoadWarps) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// Tiles of a kernel that run at once: one CTA to an SM, or as many clusters as the device holds (33 of
// four where 148 SMs would make 37); 0: such clusters do not fit.
template <int OP, bool WIDE, int BN, int SPLIT>
cudaError_t tiles_at_once(int* n) {
  auto kern = gated_tf32_kernel<OP, WIDE, BN, SPLIT>;
  constexpr int smem = Cfg<BN, SPLIT>::kSmemBytes;
  static int attr_done[64] = {0};  // per instantiation and device
  const cudaError_t e = ensure_dynamic_smem(kern, smem, attr_done);
  *n = num_sms();
  if (SPLIT == 1 || e != cudaSuccess) return e;
  static std::atomic<int> cache[kMaxDevices];
  return cluster_slots((const void*)kern, SPLIT, kThreads, smem, cache, n);
}

template <int OP, bool WIDE, int BN, int SPLIT>
cudaError_t launch_as(const Args& p, int64_t tiles, cudaStream_t stream) {
  auto kern = gated_tf32_kernel<OP, WIDE, BN, SPLIT>;
  constexpr int smem = Cfg<BN, SPLIT>::kSmemBytes;
  int at_once = 0;
  const cudaError_t e = tiles_at_once<OP, WIDE, BN, SPLIT>(&at_once);
  if (e != cudaSuccess) return e;
  const unsigned clusters = (unsigned)std::min<int64_t>(tiles, at_once);
  if constexpr (SPLIT == 1) return launch_kernel(kern, dim3(clusters), dim3(kThreads), smem, stream, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * SPLIT);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = SPLIT;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t l = cudaLaunchKernelEx(&cfg, kern, p);
  count_launch();
  return l;
}

template <int OP, bool WIDE>
cudaError_t launch_walk(const Args& p, int64_t capacity_hint, cudaStream_t stream) {
  // Rounds of tiles, as far as the host knows them, times a tile's K blocks; a block of 64 columns
  // counts as 0.65 of one of 128 (A is most of the loads), the exchange of sums as three. Measured,
  // tiles of 128, of 64, of 64 in clusters of four: 2048 rows, d 768, f 2048, down 88, 138, 180 us;
  // 777 rows of 3 experts, d 321, f 1027, input 120, 90, 59 us; hidden 49, 32, 63 us.
  auto over = [](int64_t n, int64_t by) { return (n + by - 1) / by; };
  const int64_t rows = std::max<int64_t>(1, std::min(capacity_hint, p.rows_max));
  auto tiles = [&](int bn) -> int64_t {
    if (OP == kWeight) return p.E * (over(p.f, kBM) * over(p.d, bn) + 2 * over(p.d, kBM) * over(p.f, bn));
    return std::min<int64_t>(p.E, p.rows_max) * over(rows, bn) * over(p.n_out, OP == kUp ? kBM / 2 : kBM);
  };
  const int64_t blocks = (OP == kInput ? 2 : 1) * over(OP == kWeight ? rows : p.K, kBK);
  int fours = 0;
  const cudaError_t e = tiles_at_once<OP, WIDE, 64, 4>(&fours);
  if (e != cudaSuccess) return e;
  const double t128 = (double)over(tiles(128), num_sms()) * blocks;
  const double t64 = over(tiles(64), num_sms()) * 0.65 * blocks;
  const double t64x4 = fours < 1 ? t128 : over(tiles(64), fours) * (0.65 * over(blocks, 4) + 3);
  if (t64x4 < t128 && t64x4 < t64) return launch_as<OP, WIDE, 64, 4>(p, tiles(64), stream);
  if (t64 < t128) return launch_as<OP, WIDE, 64, 1>(p, tiles(64), stream);
  return launch_as<OP, WIDE, 128, 1>(p, tiles(128), stream);
}

template <int OP>
cudaError_t launch(const Args& p, int64_t capacity_hint, cudaStream_t stream) {
  if (p.rows_max == 0) return cudaSuccess;
  // K % 4 == 0: rows that are contiguous along k start on 16 bytes
  if constexpr (OP != kWeight)
    if (p.K % 4 == 0) return launch_walk<OP, true>(p, capacity_hint, stream);
  return launch_walk<OP, false>(p, capacity_hint, stream);
}

Args args_of(const GatedFfn& g, int* status) {
  Args p{};
  p.offsets = g.offsets; p.E = g.E; p.d = g.d; p.f = g.f; p.act = g.act; p.rows_max = g.rows_max;
  p.status = status;
  return p;
}

}  // namespace

cudaError_t enqueue_gated_up_f32(const GatedFfn& g, float* h, float* saved_a, float* saved_q,
                                 int* status, cudaStream_t stream) {
  Args p = args_of(g, status);
  p.n_out = g.f; p.K = g.d;
  p.a0 = (const float*)g.w_gate; p.a1 = (const float*)g.w_up; p.b0 = (const float*)g.x;
  p.bias0 = (const float*)g.b_gate; p.bias1 = (const float*)g.b_up;
  p.out0 = h; p.out1 = saved_a; p.out2 = saved_q;
  return launch<kUp>(p, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_down_f32(const GatedFfn& g, const float* h, float* y, int* status,
                                   cudaStream_t stream) {
  Args p = args_of(g, status);
  p.n_out = g.d; p.K = g.f;
  p.a0 = (const float*)g.w_down; p.b0 = h; p.bias0 = (const float*)g.b_down; p.out0 = y;
  return launch<kDown>(p, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_hidden_grad_f32(const GatedFfn& g, const float* dy, const float* saved_a,
                                          const float* saved_q, float* dg, float* du, int* status,
                                          cudaStream_t stream) {
  Args p = args_of(g, status);
  p.n_out = g.f; p.K = g.d;
  p.a0 = (const float*)g.w_down; p.b0 = dy; p.in0 = saved_a; p.in1 = saved_q;
  p.out0 = dg; p.out1 = du;
  return launch<kHidden>(p, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_input_grad_f32(const GatedFfn& g, const float* dg, const float* du,
                                         float* dx, int* status, cudaStream_t stream) {
  Args p = args_of(g, status);
  p.n_out = g.d; p.K = g.f;
  p.a0 = (const float*)g.w_gate; p.a1 = (const float*)g.w_up; p.b0 = dg; p.b1 = du;
  p.out0 = dx;
  return launch<kInput>(p, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_weight_grad_f32(const GatedFfn& g, const float* dy, const float* h,
                                          const float* dg, const float* du, float* dw_down,
                                          float* dw_gate, float* dw_up, int* status,
                                          cudaStream_t stream) {
  Args p = args_of(g, status);
  p.a0 = h; p.a1 = (const float*)g.x; p.b0 = dy; p.b1 = dg; p.b2 = du;
  p.out0 = dw_down; p.out1 = dw_gate; p.out2 = dw_up;
  return launch<kWeight>(p, g.capacity_hint, stream);
}

}  // namespace moe
