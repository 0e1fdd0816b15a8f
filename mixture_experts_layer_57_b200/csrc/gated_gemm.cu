// The products of the gated expert FFN over expert-major rows on sm_100a tensor cores (tcgen05 +
// TMEM + TMA), forward and backward. For every row r of expert e's segment:
//     up      h[r, i] = act(zg) zu,  zg = Wg[e][i] . x[r] + bg[e, i],  zu likewise with Wu, bu
//             (training also writes a = act(zg) and q = zu act'(zg))
//     down    y[r, m] = Wd[e][m] . h[r] + bd[e, m]
//     hidden  dh[r, i] = sum_m dy[r, m] Wd[e][m, i];  dg = dh q,  du = dh a
//     input   dx[r, j] = sum_i dg[r, i] Wg[e][i, j] + du[r, i] Wu[e][i, j]
//
// The weights are the MMA's A operand (128 rows of M per tile and CTA) and the token rows its B
// operand (N = the tile's rows, so a segment of few rows costs no padding): the accumulator holds
// features in TMEM lanes and tokens in columns.
//
// Up projection: both weights meet in one accumulator. The 128 rows of an A tile are eight groups
// of 16: gate features f0..f0+15, up features f0..f0+15, gate f0+16.., and so on, each group one
// TMA box. A warp's 32 TMEM lanes then hold zg and zu of the same 16 features, half a warp apart;
// eight shuffles per 16 tokens give every lane zg and zu of one feature for eight tokens, so the
// activation and the product cost no extra pass, no extra accumulator and no shared memory.
//
// Schedule and roles as in the grouped GEMM: persistent CTAs walk tiles (expert, feature tile,
// token tile); warp 0 issues TMA into a ring of stages (64 of K each, 128-byte swizzle), one
// thread of warp 1 issues the MMAs into one of two accumulators, warps 2..9 are the epilogue of the
// tile before. Every wait is bounded; on expiry MOE_DEVERR_TIMEOUT is recorded, the other roles
// stop, in-flight copies and MMAs are drained and TMEM is freed.
#include <algorithm>

#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBM = 128;         // A rows per tile and CTA
constexpr int kBK = 64;          // K per stage: one 128-byte swizzle row of bf16
constexpr int kUmmaK = 16;       // K per tcgen05.mma (kind::f16)
constexpr int kThreads = 320;    // 10 warps: TMA, MMA, 8 epilogue
constexpr int kEpiWarps = 8;
constexpr int kEpiTileBytes = 16 * 32 * 4;  // per epilogue warp: 16 tokens x 32 features, fp32
constexpr int kBoxL = 64, kBoxS = 16;       // token rows of the two TMA box heights
constexpr int kRingBytes = 200 * 1024;

enum Op { kUp = 0, kDown = 1, kHidden = 2, kInput = 3 };

struct GemmParams {
  const int32_t* offsets;  // [E+1]
  int E;
  int n_out;               // output features per expert
  int K;                   // reduction length (of each of the two products of kInput)
  int64_t rows_max;
  const uint16_t *bias0, *bias1;
  void *out0, *out1, *out2;  // kUp: h, a, q; kDown, kInput: y or dx; kHidden: dg, du
  const uint16_t *in0, *in1; // kHidden: a, q
  int out_bf16;              // kDown, kInput
  int act;
  int* status;
};

// A and B of each product; the token operand with both box heights.
struct GemmMaps {
  CUtensorMap a0, a1, b0l, b0s, b1l, b1s;
};

// FT: A tiles of 128 rows per CTA tile, each with its own accumulator, that share the token rows
// of a stage.
template <int OP, int BN, int FT>
struct GemmCfg {
  static constexpr bool kAMn = OP == kHidden || OP == kInput;  // weights read MN-major
  static constexpr int kPhases = OP == kInput ? 2 : 1;
  static constexpr int kFeat = (OP == kUp ? kBM / 2 : kBM);    // output features per A tile
  static constexpr int kTileFeat = kFeat * FT;
  static constexpr int kABytes = FT * kBM * kBK * 2;
  static constexpr int kStageBytes = kABytes + BN * kBK * 2;
  static constexpr int kStagesFit = kRingBytes / kStageBytes;
  static constexpr int kStages = kStagesFit > 12 ? 12 : kStagesFit;
  static constexpr int kAccCols = FT * BN;
  static constexpr int kTmemCols = 2 * kAccCols < 32 ? 32 : 2 * kAccCols;
  static_assert(kTmemCols <= 512, "two accumulator buffers must fit TMEM");
  static constexpr int kBarBytes = 8 * 64;
  static constexpr int kAuxBytes = kBarBytes + 16 + 2 * 4 * (MOE_MAX_EXPERTS + 1);
  static constexpr int kSmemBytes =
      1024 + kStages * kStageBytes + kEpiWarps * kEpiTileBytes + kAuxBytes;
  static_assert(kStageBytes % 1024 == 0, "stage tiles must stay 1024-byte aligned");
  static_assert(2 * kStages + 5 <= 64, "barrier area too small");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

struct Tile {
  int e, f0, row0, n_valid;
};

// Tiles of one feature tile and all token tiles of an expert follow one another, so consecutive
// CTAs share a weight tile in L2.
template <int BN>
__device__ __forceinline__ Tile decode_tile(int t, const int* prefix, const int* seg, int E,
                                            int tile_feat) {
  int lo = 0, hi = E;  // prefix[lo] <= t < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int rows = seg[lo + 1] - seg[lo];
  const int ntt = (rows + BN - 1) / BN;
  const int local = t - prefix[lo];
  const int ft = local / ntt;
  const int jt = local - ft * ntt;
  return Tile{lo, ft * tile_feat, seg[lo] + jt * BN, min(BN, rows - jt * BN)};
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

// The mbarriers of one CTA: S stage-full, S stage-empty, 2 accumulator-full, 2 accumulator-empty
// and one drain barrier, 8 bytes each from `base`.
struct Bars {
  uint32_t base;
  int S;
  __device__ __forceinline__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return base + 8u * (S + s); }
  __device__ __forceinline__ uint32_t tfull(int a) const { return base + 8u * (2 * S + a); }
  __device__ __forceinline__ uint32_t tempty(int a) const { return base + 8u * (2 * S + 2 + a); }
  __device__ __forceinline__ uint32_t drain() const { return base + 8u * (2 * S + 4); }
};

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int S) {
    if (++stage == S) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Tile list in shared memory (one warp): seg[e] = first row of expert e, prefix[e] = its first
// tile, prefix[E] = the tile count (0 and a device error if the offsets are not non-decreasing
// within [0, rows_max]).
template <int BN>
__device__ __forceinline__ void build_tile_list(const GemmParams& p, int n_ftiles, int* prefix,
                                                int* seg, int lane) {
  const int E = p.E;
  const int chunk = (E + 31) / 32;
  const int e0 = min(E, lane * chunk), e1 = min(E, e0 + chunk);
  bool bad = false;
  int local = 0;
  for (int e = e0; e < e1; ++e) {
    const int a = p.offsets[e], b = p.offsets[e + 1];
    seg[e] = a;
    if (a < 0 || b < a || (int64_t)b > p.rows_max) bad = true;
    else local += n_ftiles * ((b - a + BN - 1) / BN);
  }
  if (lane == 0) seg[E] = p.offsets[E];
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int run = incl - local;
  for (int e = e0; e < e1; ++e) {
    prefix[e] = run;
    const int a = seg[e], b = p.offsets[e + 1];
    if (!(a < 0 || b < a || (int64_t)b > p.rows_max)) run += n_ftiles * ((b - a + BN - 1) / BN);
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  bad = __any_sync(0xffffffffu, bad);
  __syncwarp();
  if (lane == 0) {
    prefix[E] = bad ? 0 : total;
    if (bad && blockIdx.x == 0) set_device_error(p.status, MOE_DEVERR_BAD_OFFSETS);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return (uint32_t)f32_to_bf16_rn(lo) | ((uint32_t)f32_to_bf16_rn(hi) << 16);
}

// Loads the A tile(s) of one stage: feature f0 of expert e on, K block kb of product `ph`.
template <int OP, int FT>
__device__ __forceinline__ void load_a(uint32_t sa, const GemmMaps& m, const GemmParams& p, int ph,
                                       int e, int f0, int kb, uint32_t bar) {
#pragma unroll
  for (int i = 0; i < FT; ++i) {
    const uint32_t sai = sa + i * (kBM * kBK * 2);
    if constexpr (OP == kUp) {
      // rows past this expert's features belong to the next expert or are out of range; the
      // epilogue masks them
      const int w_row = e * p.n_out + f0 + i * (kBM / 2);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        tma_load_2d(sai + g * 4096, &m.a0, kb * kBK, w_row + g * 16, bar);
        tma_load_2d(sai + g * 4096 + 2048, &m.a1, kb * kBK, w_row + g * 16, bar);
      }
    } else if constexpr (OP == kDown) {
      tma_load_2d(sai, &m.a0, kb * kBK, e * p.n_out + f0 + i * kBM, bar);
    } else {
      const CUtensorMap* a = ph == 0 ? &m.a0 : &m.a1;
      // three dimensions, so that K rows past this expert's are zero and not the next expert's
      // (whose weights may be infinite or NaN)
      tma_load_3d(sai, a, f0 + i * kBM, kb * kBK, e, bar);
      tma_load_3d(sai + kBM * kBK, a, f0 + i * kBM + 64, kb * kBK, e, bar);
    }
  }
}

// Loads n token rows (a multiple of 16) from row0 on, in boxes of 64 rows and then of 16.
__device__ __forceinline__ void load_b(uint32_t sb, const CUtensorMap* l, const CUtensorMap* s,
                                       int kb, int row0, int n, uint32_t bar) {
  int r = 0;
  for (; r + kBoxL <= n; r += kBoxL) tma_load_2d(sb + r * 128, l, kb * kBK, row0 + r, bar);
  for (; r < n; r += kBoxS) tma_load_2d(sb + r * 128, s, kb * kBK, row0 + r, bar);
}

// Epilogue of one A tile (features f0 .. f0 + kFeat): this warp's lane quarter of the accumulator
// at acc, alternate 16-token chunks by `half`, staged through `st` so that rows leave in 16-byte
// stores.
template <int OP>
__device__ __forceinline__ void epilogue(const Tile& tl, int f0, const GemmParams& p, uint32_t acc,
                                         int quarter, int half, int lane, uint8_t* st) {
  const uint32_t taddr = acc + ((uint32_t)(quarter * 32) << 16);
  if constexpr (OP == kUp) {
    const int j = lane & 15, up = lane >> 4;
    const int fw = f0 + quarter * 16;  // first feature of this warp
    const int f = fw + j;
    const bool f_ok = f < p.n_out;
    const int64_t bi = (int64_t)tl.e * p.n_out + f;
    const float bg = p.bias0 != nullptr && f_ok ? bf16_to_f32(p.bias0[bi]) : 0.0f;
    const float bu = p.bias1 != nullptr && f_ok ? bf16_to_f32(p.bias1[bi]) : 0.0f;
    uint16_t* s16 = reinterpret_cast<uint16_t*>(st);  // [3][16 tokens][16 features]
    const bool save = p.out1 != nullptr;
    for (int c0 = half * 16; c0 < tl.n_valid; c0 += 32) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(taddr + (uint32_t)c0, r);
      tmem_ld_wait();
      const int nc = min(16, tl.n_valid - c0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // gate lanes keep tokens 0..7 and give 8..15, up lanes the other way round
        const float own = __uint_as_float(up ? r[8 + i] : r[i]);
        const float got = __shfl_xor_sync(0xffffffffu, __uint_as_float(up ? r[i] : r[8 + i]), 16);
        const float zg = (up ? got : own) + bg;
        const float zu = (up ? own : got) + bu;
        float a, da;
        gate_act<true>(zg, p.act, a, da);
        const int at = (up * 8 + i) * 16 + j;
        s16[at] = f32_to_bf16_rn(a * zu);
        if (save) {
          s16[256 + at] = f32_to_bf16_rn(a);
          s16[512 + at] = f32_to_bf16_rn(zu * da);
        }
      }
      __syncwarp();
      const int row = lane >> 1, ff = fw + 8 * (lane & 1);
      if (row < nc && ff < p.n_out) {
        const int64_t o = (int64_t)(tl.row0 + c0 + row) * p.n_out + ff;
        const uint4* s4 = reinterpret_cast<const uint4*>(st) + lane;
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out0) + o) = s4[0];
        if (save) {
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out1) + o) = s4[32];
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out2) + o) = s4[64];
        }
      }
      __syncwarp();
    }
  } else {
    const int fw = f0 + quarter * 32;
    const int f = fw + lane;
    const float bv = OP == kDown && p.bias0 != nullptr && f < p.n_out
                         ? bf16_to_f32(p.bias0[(int64_t)tl.e * p.n_out + f])
                         : 0.0f;
    float* s32 = reinterpret_cast<float*>(st);  // [16 tokens][32 features]
    for (int c0 = half * 16; c0 < tl.n_valid; c0 += 32) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(taddr + (uint32_t)c0, r);
      tmem_ld_wait();
      const int nc = min(16, tl.n_valid - c0);
#pragma unroll
      for (int c = 0; c < 16; ++c) s32[c * 32 + lane] = __uint_as_float(r[c]) + bv;
      __syncwarp();
      if (OP != kHidden && !p.out_bf16) {
#pragma unroll
        for (int id = lane; id < 128; id += 32) {
          const int row = id >> 3, ff = fw + 4 * (id & 7);
          if (row < nc && ff < p.n_out)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out0) +
                                       (int64_t)(tl.row0 + c0 + row) * p.n_out + ff) =
                *reinterpret_cast<const float4*>(st + id * 16);
        }
      } else {
        // 8 features of one token per lane
#pragma unroll
        for (int id = lane; id < 64; id += 32) {
          const int row = id >> 2, ff = fw + 8 * (id & 3);
          if (row < nc && ff < p.n_out) {
            const int64_t o = (int64_t)(tl.row0 + c0 + row) * p.n_out + ff;
            const float4 v0 = *reinterpret_cast<const float4*>(st + id * 32);
            const float4 v1 = *reinterpret_cast<const float4*>(st + id * 32 + 16);
            if constexpr (OP == kHidden) {
              auto times = [&](const uint16_t* in) {
                const uint4 s = *reinterpret_cast<const uint4*>(in + o);
                uint4 w;
                w.x = pack2(v0.x * __uint_as_float(s.x << 16), v0.y * __uint_as_float(s.x & 0xffff0000u));
                w.y = pack2(v0.z * __uint_as_float(s.y << 16), v0.w * __uint_as_float(s.y & 0xffff0000u));
                w.z = pack2(v1.x * __uint_as_float(s.z << 16), v1.y * __uint_as_float(s.z & 0xffff0000u));
                w.w = pack2(v1.z * __uint_as_float(s.w << 16), v1.w * __uint_as_float(s.w & 0xffff0000u));
                return w;
              };
              const uint4 du = times(p.in0), dg = times(p.in1);
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out0) + o) = dg;
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out1) + o) = du;
            } else {
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out0) + o) =
                  make_uint4(pack2(v0.x, v0.y), pack2(v0.z, v0.w), pack2(v1.x, v1.y), pack2(v1.z, v1.w));
            }
          }
        }
      }
      __syncwarp();
    }
  }
}

template <int OP, int BN, int FT>
__global__ void __launch_bounds__(kThreads, 1)
    gated_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmParams p) {
  using C = GemmCfg<OP, BN, FT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_addr - raw_addr);
  uint8_t* epi_tiles = base + C::kStages * C::kStageBytes;
  uint8_t* aux = epi_tiles + kEpiWarps * kEpiTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(aux);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(aux + C::kBarBytes);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(aux + C::kBarBytes + 4);
  int* prefix = reinterpret_cast<int*>(aux + C::kBarBytes + 16);
  int* seg = prefix + (MOE_MAX_EXPERTS + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr int S = C::kStages;
  const Bars B{smem_u32(bars), S};

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(B.full(s), 1);
      mbar_init(B.empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(B.tfull(a), 1);
      mbar_init(B.tempty(a), kEpiWarps * 32);
    }
    mbar_init(B.drain(), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), C::kTmemCols);
    tmem_relinquish();
  }
  const int n_ftiles = (p.n_out + C::kTileFeat - 1) / C::kTileFeat;
  if (warp == 2) build_tile_list<BN>(p, n_ftiles, prefix, seg, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total_tiles = prefix[p.E];
  const int n_kb = (p.K + kBK - 1) / kBK;
  const int n_blocks = C::kPhases * n_kb;
  auto tile_at = [&](int t) { return decode_tile<BN>(t, prefix, seg, p.E, C::kTileFeat); };

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      Ring ring;
      int issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total_tiles && ok; t += gridDim.x) {
        const Tile tl = tile_at(t);
        const int n_b = (tl.n_valid + 15) & ~15;
        for (int i = 0; i < n_blocks; ++i) {
          if (!mbar_wait_bounded(B.empty(ring.stage), ring.phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const int ph = C::kPhases == 2 && i >= n_kb ? 1 : 0;
          const int kb = i - ph * n_kb;
          const uint32_t sa = base_addr + ring.stage * C::kStageBytes;
          mbar_arrive_expect_tx(B.full(ring.stage), C::kABytes + n_b * 128);
          load_a<OP, FT>(sa, maps, p, ph, tl.e, tl.f0, kb, B.full(ring.stage));
          load_b(sa + C::kABytes, ph ? &maps.b1l : &maps.b0l, ph ? &maps.b1s : &maps.b0s, kb,
                 tl.row0, n_b, B.full(ring.stage));
          ++issued;
          ring.next(S);
        }
      }
      // drain: the last min(issued, S) loads may still be landing
      for (int i = max(0, issued - S); i < issued; ++i)
        wait_drain(B.full(i % S), (uint32_t)((i / S) & 1), p.status);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      Ring ring;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total_tiles && ok; t += gridDim.x) {
        if (!mbar_wait_bounded(B.tempty(acc), acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const Tile tl = tile_at(t);
        const uint32_t idesc =
            idesc_bf16_f32_major(kBM, (tl.n_valid + 15) & ~15, C::kAMn, false);
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * C::kAccCols);
        for (int i = 0; i < n_blocks; ++i) {
          if (!mbar_wait_bounded(B.full(ring.stage), ring.phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base_addr + ring.stage * C::kStageBytes;
          const uint64_t bdesc = smem_desc_sw128(sa + C::kABytes);
          constexpr uint64_t a_step = C::kAMn ? (kMnKStepBytes >> 4) : 2;
#pragma unroll
          for (int j = 0; j < FT; ++j) {
            const uint32_t saj = sa + j * (kBM * kBK * 2);
            const uint64_t adesc = C::kAMn ? smem_desc_sw128_mn(saj) : smem_desc_sw128(saj);
#pragma unroll
            for (int kk = 0; kk < kBK / kUmmaK; ++kk)
              tc_mma_bf16(d_tmem + (uint32_t)(j * BN), adesc + a_step * (uint64_t)kk,
                          bdesc + (uint64_t)(2 * kk), idesc, (i | kk) != 0 ? 1u : 0u);
          }
          tc_commit(B.empty(ring.stage));
          ring.next(S);
        }
        if (!ok) break;
        tc_commit(B.tfull(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      // drain every MMA this thread issued before TMEM is released
      tc_commit(B.drain());
      wait_drain(B.drain(), 0, p.status);
    }
  } else {
    // ---------------------------------------------------------- epilogue (warps 2..9)
    const int ew = warp - 2;
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    const int half = ew >> 2;
    uint8_t* st = epi_tiles + ew * kEpiTileBytes;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < total_tiles; t += gridDim.x) {
      if (!mbar_wait_bounded_warp(B.tfull(acc), acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      const Tile tl = tile_at(t);
#pragma unroll 1
      for (int j = 0; j < FT; ++j)
        epilogue<OP>(tl, tl.f0 + j * C::kFeat, p,
                     tmem_base + (uint32_t)(acc * C::kAccCols + j * BN), quarter, half, lane, st);
      tc_fence_before();
      mbar_arrive(B.tempty(acc));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- host side

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Weights [E, K, n] read MN-major in boxes of 64 features x 64 K rows of one expert.
bool weight_map_mn(CUtensorMap* m, const void* ptr, int E, int K, int n) {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  if (!fn) return false;
  cuuint64_t gdim[3] = {(cuuint64_t)n, (cuuint64_t)K, (cuuint64_t)E};
  cuuint64_t gstride[2] = {(cuuint64_t)n * 2, (cuuint64_t)n * K * 2};
  cuuint32_t box[3] = {64, kBK, 1};
  cuuint32_t estride[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), gdim, gstride, box,
            estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int OP, int BN, int FT>
cudaError_t launch_single(const GemmMaps& m, const GemmParams& p, cudaStream_t stream) {
  auto kern = gated_gemm_kernel<OP, BN, FT>;
  constexpr int smem = GemmCfg<OP, BN, FT>::kSmemBytes;
  static int attr_done[64] = {0};  // per instantiation and device
  const cudaError_t e = ensure_dynamic_smem(kern, smem, attr_done);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(num_sms()), dim3(kThreads), smem, stream, m, p);
}

template <int OP>
cudaError_t launch_op(const GemmMaps& m, const GemmParams& p, int64_t capacity_hint,
                      cudaStream_t stream) {
  if (capacity_hint <= 16) return launch_single<OP, 16, 2>(m, p, stream);
  if (capacity_hint <= 32) return launch_single<OP, 32, 2>(m, p, stream);
  if (capacity_hint <= 64) return launch_single<OP, 64, 2>(m, p, stream);
  if (capacity_hint <= 128) return launch_single<OP, 128, 2>(m, p, stream);
  return launch_single<OP, 256, 1>(m, p, stream);
}

// Both box heights of a token operand [rows, K].
bool token_maps(CUtensorMap* l, CUtensorMap* s, const void* ptr, int64_t rows, int K) {
  return make_bf16_map_2d(l, ptr, rows, K, kBK, kBoxL) &&
         make_bf16_map_2d(s, ptr, rows, K, kBK, kBoxS);
}

}  // namespace

cudaError_t enqueue_gated_up_bf16(const GatedFfn& g, void* h, void* saved_a, void* saved_q,
                                  int* status, cudaStream_t stream) {
  if (g.rows_max == 0) return cudaSuccess;
  GemmMaps m;
  if (!make_bf16_map_2d(&m.a0, g.w_gate, (int64_t)g.E * g.f, g.d, kBK, 16) ||
      !make_bf16_map_2d(&m.a1, g.w_up, (int64_t)g.E * g.f, g.d, kBK, 16) ||
      !token_maps(&m.b0l, &m.b0s, g.x, g.rows_max, g.d))
    return cudaErrorInvalidValue;
  m.b1l = m.b0l;
  m.b1s = m.b0s;
  GemmParams p{};
  p.offsets = g.offsets; p.E = g.E; p.n_out = g.f; p.K = g.d; p.rows_max = g.rows_max;
  p.bias0 = (const uint16_t*)g.b_gate; p.bias1 = (const uint16_t*)g.b_up;
  p.out0 = h; p.out1 = saved_a; p.out2 = saved_q; p.act = g.act; p.status = status;
  return launch_op<kUp>(m, p, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_down_bf16(const GatedFfn& g, const void* h, void* y, bool y_bf16,
                                    int* status, cudaStream_t stream) {
  if (g.rows_max == 0) return cudaSuccess;
  GemmMaps m;
  if (!make_bf16_map_2d(&m.a0, g.w_down, (int64_t)g.E * g.d, g.f, kBK, kBM) ||
      !token_maps(&m.b0l, &m.b0s, h, g.rows_max, g.f))
    return cudaErrorInvalidValue;
  m.a1 = m.a0;
  m.b1l = m.b0l;
  m.b1s = m.b0s;
  GemmParams p{};
  p.offsets = g.offsets; p.E = g.E; p.n_out = g.d; p.K = g.f; p.rows_max = g.rows_max;
  p.bias0 = (const uint16_t*)g.b_down; p.out0 = y; p.out_bf16 = y_bf16 ? 1 : 0; p.status = status;
  return launch_op<kDown>(m, p, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_hidden_grad_bf16(const GatedFfn& g, const void* dy, const void* saved_a,
                                           const void* saved_q, void* dg, void* du, int* status,
                                           cudaStream_t stream) {
  if (g.rows_max == 0) return cudaSuccess;
  GemmMaps m;
  if (!weight_map_mn(&m.a0, g.w_down, g.E, g.d, g.f) ||
      !token_maps(&m.b0l, &m.b0s, dy, g.rows_max, g.d))
    return cudaErrorInvalidValue;
  m.a1 = m.a0;
  m.b1l = m.b0l;
  m.b1s = m.b0s;
  GemmParams p{};
  p.offsets = g.offsets; p.E = g.E; p.n_out = g.f; p.K = g.d; p.rows_max = g.rows_max;
  p.out0 = dg; p.out1 = du; p.in0 = (const uint16_t*)saved_a; p.in1 = (const uint16_t*)saved_q;
  p.status = status;
  return launch_op<kHidden>(m, p, g.capacity_hint, stream);
}

cudaError_t enqueue_gated_input_grad_bf16(const GatedFfn& g, const void* dg, const void* du,
                                          void* dx, bool dx_bf16, int* status,
                                          cudaStream_t stream) {
  if (g.rows_max == 0) return cudaSuccess;
  GemmMaps m;
  if (!weight_map_mn(&m.a0, g.w_gate, g.E, g.f, g.d) ||
      !weight_map_mn(&m.a1, g.w_up, g.E, g.f, g.d) ||
      !token_maps(&m.b0l, &m.b0s, dg, g.rows_max, g.f) ||
      !token_maps(&m.b1l, &m.b1s, du, g.rows_max, g.f))
    return cudaErrorInvalidValue;
  GemmParams p{};
  p.offsets = g.offsets; p.E = g.E; p.n_out = g.d; p.K = g.f; p.rows_max = g.rows_max;
  p.out0 = dx; p.out_bf16 = dx_bf16 ? 1 : 0; p.status = status;
  return launch_op<kInput>(m, p, g.capacity_hint, stream);
}

}  // namespace moe
