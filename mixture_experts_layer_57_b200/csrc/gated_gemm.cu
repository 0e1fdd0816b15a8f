// The products of the gated expert FFN over expert-major rows on sm_100a tensor cores (tcgen05 +
// TMEM + TMA), forward and backward. For every row r of expert e's segment:
//     up      h[r, i] = act(zg) zu,  zg = Wg[e][i] . x[r] + bg[e, i],  zu likewise with Wu, bu
//             (training also writes a = act(zg) and q = zu act'(zg), as blocks of eight values)
//     down    y[r, m] = Wd[e][m] . h[r] + bd[e, m]
//     hidden  dh[r, i] = sum_m dy[r, m] Wd[e][m, i];  dg = dh q,  du = dh a
//     input   dx[r, j] = sum_i dg[r, i] Wg[e][i, j] + du[r, i] Wu[e][i, j]
//
// The weights are the MMA's A operand (128 rows of M per tile and CTA) and the token rows its B
// operand (N = the tile's rows, so a segment of few rows costs no padding): the accumulator holds
// features in TMEM lanes and tokens in columns.
//
// Up projection: both weights meet in one accumulator. Of the 128 rows of an A tile 64 are gate
// features and 64 up features, each a TMA box of its own tensor, so zg of a feature lies in one warp's
// TMEM lanes and zu in those of the warp two quarters on. The two exchange halves of every 16 tokens
// through shared memory (a kilobyte each way, handed over by mbarriers) and then both have zg and zu of
// 32 features for eight tokens: activation and product cost no extra pass and no extra accumulator.
// (Groups of 16 rows of each, which need no exchange but shuffles in the warp, are boxes of 2 KB: decode
// over 128 experts 647 us for 470. One tensor map over both weights, with their distance as a stride, is
// not sound: the memory between two allocations need not be mapped, and with the first tensor near the
// end of its allocation such loads ended in an illegal access, although every box lay inside the two
// tensors.)
//
// Hidden: the epilogue reads a and q, and loads them for its next 16 tokens while it works on these.
//
// Schedule and roles as in the grouped GEMM: persistent clusters walk tiles (expert, feature tile,
// token tile); warp 0 issues TMA into a ring of stages (64 of K each, 128-byte swizzle), one
// thread of warp 1 issues the MMAs into one of two accumulators, warps 2..13 are the epilogue of
// the tile before. Every wait is bounded; on expiry MOE_DEVERR_TIMEOUT is recorded, the other roles
// stop, in-flight copies and MMAs are drained and TMEM is freed.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "gated.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBM = 128;         // A rows per tile and CTA
constexpr int kBK = 64;          // K per stage: one 128-byte swizzle row of bf16
constexpr int kUmmaK = 16;       // K per tcgen05.mma (kind::f16)
constexpr int kEpiSets = 3;      // epilogue warps for each quarter of the accumulator's lanes
constexpr int kEpiWarps = 4 * kEpiSets;
constexpr int kThreads = 64 + 32 * kEpiWarps;  // TMA, MMA, epilogue
constexpr int kEpiTileBytes = 16 * 32 * 4;  // per epilogue warp: 16 tokens x 32 features, fp32
constexpr int kBoxL = 64, kBoxS = 16;       // token rows of the two TMA box heights
constexpr int kRingBytes = 193 * 1024;

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

// How CTAs share a tile.
//   kPair    two CTAs on two SMs, MMAs of M = 256 (cta_group::2): each holds 128 A rows, half of
//            the token rows and its half of the accumulator, so each token row is loaded once per
//            pair
//   kSplit   a cluster of S = 1 to 8 CTAs, each with its share of the K blocks; each CTA then
//            finishes every S-th group of 16 tokens, for which the others write their partial sums
//            into its shared memory
enum Mode { kPair = 0, kSplit = 1 };
constexpr int kMaxSplit = 8;
constexpr int kPartChunk = 16 * kBM * 4;  // partial sums of 16 tokens
constexpr int kPartChunks = 7;
// Partial sums that a CTA receives for one tile of `bn` tokens, in groups of 16.
__host__ __device__ constexpr int parts_of(int bn, int width) {
  return (width - 1) * ((bn / 16 + width - 1) / width);
}

// FT: A tiles of 128 rows per CTA tile, each with its own accumulator, that share the token rows
// of a stage. Two sets of accumulators: a tile's MMAs run while the one before is finished.
template <int OP, int BN, int FT, int MODE>
struct GemmCfg {
  static constexpr bool kAMn = OP == kHidden || OP == kInput;  // weights read MN-major
  static constexpr int kPhases = OP == kInput ? 2 : 1;
  static constexpr int kFeat = (OP == kUp ? kBM / 2 : kBM);    // output features per A tile
  static constexpr int kTileFeat = kFeat * FT * (MODE == kPair ? 2 : 1);
  static constexpr int kABytes = FT * kBM * kBK * 2;
  static constexpr int kBRows = MODE == kPair ? BN / 2 : BN;   // token rows per CTA and stage
  static constexpr int kStageBytes = kABytes + kBRows * kBK * 2;
  static constexpr int kPartBytes = MODE == kSplit ? kPartChunks * kPartChunk : 0;
  static constexpr int kStagesFit = (kRingBytes - kPartBytes) / kStageBytes;
  static constexpr int kStages = kStagesFit > 12 ? 12 : kStagesFit;
  static constexpr int kAccCols = FT * BN;
  static constexpr int kTmemCols = 2 * kAccCols;
  static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM");
  static_assert(MODE != kSplit || (FT == 1 && BN <= 128), "split tiles");
  static constexpr int kBarBytes = 8 * 64;
  static constexpr int kAuxBytes = kBarBytes + 16 + 2 * 4 * (MOE_MAX_EXPERTS + 1);
  static constexpr int kSmemBytes =
      1024 + kStages * kStageBytes + kPartBytes + kEpiWarps * kEpiTileBytes + kAuxBytes;
  static_assert(kStageBytes % 1024 == 0, "stage tiles must stay 1024-byte aligned");
  static_assert(kStages >= 3 && 2 * kStages + 7 + 2 * kEpiWarps <= 64, "stages, barriers");
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

// The mbarriers of one CTA: S stage-full, S stage-empty, 2 accumulator-full, 2 accumulator-empty,
// one drain barrier, and kSplit's two: the others' partial sums are written, and they have read
// this CTA's; kUp: two for every epilogue warp, its half of the exchange is written, and the other warp
// has read it. 8 bytes each from `base`.
struct Bars {
  uint32_t base;
  int S;
  __device__ __forceinline__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return base + 8u * (S + s); }
  __device__ __forceinline__ uint32_t tfull(int a) const { return base + 8u * (2 * S + a); }
  __device__ __forceinline__ uint32_t tempty(int a) const { return base + 8u * (2 * S + 2 + a); }
  __device__ __forceinline__ uint32_t drain() const { return base + 8u * (2 * S + 4); }
  __device__ __forceinline__ uint32_t part_full() const { return base + 8u * (2 * S + 5); }
  __device__ __forceinline__ uint32_t part_free() const { return base + 8u * (2 * S + 6); }
  __device__ __forceinline__ uint32_t given(int w) const { return base + 8u * (2 * S + 7 + 2 * w); }
  __device__ __forceinline__ uint32_t taken(int w) const { return base + 8u * (2 * S + 8 + 2 * w); }
};

// Position in the stage ring.
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

// One box into this CTA's shared memory, counted on `bar` (a pair's loads count on the barrier of
// its first CTA).
template <int MODE>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  if constexpr (MODE == kPair) tma_load_2d_pair(dst, m, x, y, bar);
  else tma_load_2d(dst, m, x, y, bar);
}
template <int MODE>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                        uint32_t bar) {
  if constexpr (MODE == kPair) tma_load_3d_pair(dst, m, x, y, z, bar);
  else tma_load_3d(dst, m, x, y, z, bar);
}

// Loads the A tile(s) of one stage: feature f0 of expert e on, K block kb of product `ph`.
template <int OP, int FT, int MODE>
__device__ __forceinline__ void load_a(uint32_t sa, const GemmMaps& m, const GemmParams& p, int ph,
                                       int e, int f0, int kb, uint32_t bar) {
#pragma unroll
  for (int i = 0; i < FT; ++i) {
    const uint32_t sai = sa + i * (kBM * kBK * 2);
    if constexpr (OP == kUp) {
      // rows past this expert's features belong to the next expert or are out of range; the
      // epilogue masks them
      const int w_row = e * p.n_out + f0 + i * (kBM / 2);
      load_2d<MODE>(sai, &m.a0, kb * kBK, w_row, bar);
      load_2d<MODE>(sai + kBM * kBK, &m.a1, kb * kBK, w_row, bar);
    } else if constexpr (OP == kDown) {
      load_2d<MODE>(sai, &m.a0, kb * kBK, e * p.n_out + f0 + i * kBM, bar);
    } else {
      const CUtensorMap* a = ph == 0 ? &m.a0 : &m.a1;
      // three dimensions, so that K rows past this expert's are zero and not the next expert's
      // (whose weights may be infinite or NaN)
      load_3d<MODE>(sai, a, f0 + i * kBM, kb * kBK, e, bar);
      load_3d<MODE>(sai + kBM * kBK, a, f0 + i * kBM + 64, kb * kBK, e, bar);
    }
  }
}

// Loads n token rows (a multiple of 16) from row0 on, in boxes of 64 rows and then of 16.
template <int MODE>
__device__ __forceinline__ void load_b(uint32_t sb, const CUtensorMap* l, const CUtensorMap* s,
                                       int kb, int row0, int n, uint32_t bar) {
  int r = 0;
#pragma unroll 1
  for (; r + kBoxL <= n; r += kBoxL) load_2d<MODE>(sb + r * 128, l, kb * kBK, row0 + r, bar);
#pragma unroll 1
  for (; r < n; r += kBoxS) load_2d<MODE>(sb + r * 128, s, kb * kBK, row0 + r, bar);
}

// Token columns of a tile's MMAs: its rows rounded up to what N allows (M = 256: multiples of 32).
template <int MODE>
__device__ __forceinline__ int mma_n(int n_valid) {
  return MODE == kPair ? (n_valid + 31) & ~31 : (n_valid + 15) & ~15;
}

// Which groups of 16 tokens of a tile this CTA finishes (kSplit: every `width`-th from `rank` on).
struct Share {
  int rank, width;
  const float* part;
  // groups of a full tile that one CTA finishes
  __device__ __forceinline__ int groups(int bn) const { return (bn / 16 + width - 1) / width; }
};

// What an epilogue warp of kHidden reads besides the accumulator: a and q of 16 tokens and 32
// features, eight features of one token to each of two loads a lane.
struct HiddenIn {
  uint4 a[2], q[2];
};
__device__ __forceinline__ void load_hidden_in(HiddenIn& in, const GemmParams& p, const Tile& tl,
                                               int fw, int c0, int lane) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int id = lane + 32 * u, row = c0 + (id >> 2), ff = fw + 8 * (id & 3);
    if (row < tl.n_valid && ff < p.n_out) {
      const int64_t o = (int64_t)(tl.row0 + row) * p.n_out + ff;
      in.a[u] = *reinterpret_cast<const uint4*>(p.in0 + o);
      in.q[u] = *reinterpret_cast<const uint4*>(p.in1 + o);
    }
  }
}

// The exchange of the up projection: this epilogue warp, the one that holds the other projection's
// pre-activations of the same 32 features, their staging tiles, and the phase of their barriers.
struct Exchange {
  Bars bars;
  int self, other;
  const float* theirs;
  uint32_t phase;
  bool up;  // this warp's accumulator lanes are up features
  volatile int* abort;
  int* status;
};

// Up projection: 16 tokens of this warp's 32 features of one projection. The warp of the gate features
// gives tokens 8..15 and finishes 0..7, the other one the other way round. False: a wait expired.
__device__ __forceinline__ bool finish_up(const Tile& tl, const GemmParams& p, const uint32_t (&r)[16],
                                          int fw, int c0, float bg, float bu, int lane, uint8_t* st,
                                          Exchange& x) {
  float* give = reinterpret_cast<float*>(st);            // [8 tokens][32 features]
  uint16_t* s16 = reinterpret_cast<uint16_t*>(st + 1024);  // h: the same
  float* s32 = reinterpret_cast<float*>(st + 1024);        // a, then q: the same
  if (!mbar_wait_warp(x.bars.taken(x.self), x.phase ^ 1u, x.abort, x.status)) return false;
#pragma unroll
  for (int i = 0; i < 8; ++i) give[i * 32 + lane] = __uint_as_float(x.up ? r[i] : r[8 + i]);
  __syncwarp();
  if (lane == 0) mbar_arrive(x.bars.given(x.self));
  if (!mbar_wait_warp(x.bars.given(x.other), x.phase, x.abort, x.status)) return false;
  float got[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) got[i] = x.theirs[i * 32 + lane];
  __syncwarp();
  if (lane == 0) mbar_arrive(x.bars.taken(x.other));
  x.phase ^= 1u;
  const bool save = p.out1 != nullptr;
  float a[8], q[8], h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float own = __uint_as_float(x.up ? r[8 + i] : r[i]);
    const float zg = (x.up ? got[i] : own) + bg;
    const float zu = (x.up ? own : got[i]) + bu;
    float da;
    gate_act<true>(zg, p.act, a[i], da);
    q[i] = zu * da;
    h[i] = a[i] * zu;
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t two = pack_bf16x2(h[i], h[i + 1]);
    s16[i * 32 + lane] = (uint16_t)two;
    s16[(i + 1) * 32 + lane] = (uint16_t)(two >> 16);
  }
  __syncwarp();
  // eight features of one token per lane
  const int token = lane >> 2, row = c0 + (x.up ? 8 : 0) + token, ff = fw + 8 * (lane & 3);
  const bool mine = row < tl.n_valid && ff < p.n_out;
  const int64_t o = (int64_t)(tl.row0 + row) * p.n_out + ff;
  if (mine)
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out0) + o) =
        reinterpret_cast<const uint4*>(s16)[lane];
  __syncwarp();
  if (save) {
    // the 16-byte halves in an order that spreads two tokens over all banks
    const float4* get = reinterpret_cast<const float4*>(s32) + 2 * lane;
    const int odd = token & 1;
    auto store = [&](void* out) {
      const float4 u = get[odd], w = get[odd ^ 1];
      const float4 lo = odd ? w : u, hi = odd ? u : w;
      const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      if (mine) *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + o) = pack_block8(v);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) s32[i * 32 + lane] = a[i];
    __syncwarp();
    store(p.out1);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) s32[i * 32 + lane] = q[i];
    __syncwarp();
    store(p.out2);
    __syncwarp();
  }
  return true;
}

// The other products: 16 tokens of this warp's 32 features, staged as fp32 so that rows leave in
// 16-byte stores.
template <int OP>
__device__ __forceinline__ void finish(const Tile& tl, const GemmParams& p, const uint32_t (&r)[16],
                                       int fw, int c0, float bv, const HiddenIn& in, int lane,
                                       uint8_t* st) {
  float* s32 = reinterpret_cast<float*>(st);  // [16 tokens][32 features]
#pragma unroll
  for (int c = 0; c < 16; ++c) s32[c * 32 + lane] = __uint_as_float(r[c]) + bv;
  __syncwarp();
  const int nc = min(16, tl.n_valid - c0);
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
    for (int u = 0; u < 2; ++u) {
      const int id = lane + 32 * u, row = id >> 2, ff = fw + 8 * (id & 3);
      if (row < nc && ff < p.n_out) {
        const int64_t o = (int64_t)(tl.row0 + c0 + row) * p.n_out + ff;
        const float4 v0 = *reinterpret_cast<const float4*>(st + id * 32);
        const float4 v1 = *reinterpret_cast<const float4*>(st + id * 32 + 16);
        if constexpr (OP == kHidden) {
          auto times = [&](const uint4& block) {
            float s[8];
            unpack_block8(block, s);
            return make_uint4(pack_bf16x2(v0.x * s[0], v0.y * s[1]), pack_bf16x2(v0.z * s[2], v0.w * s[3]),
                              pack_bf16x2(v1.x * s[4], v1.y * s[5]), pack_bf16x2(v1.z * s[6], v1.w * s[7]));
          };
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out0) + o) = times(in.q[u]);
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out1) + o) = times(in.a[u]);
        } else {
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out0) + o) =
              make_uint4(pack_bf16x2(v0.x, v0.y), pack_bf16x2(v0.z, v0.w), pack_bf16x2(v1.x, v1.y), pack_bf16x2(v1.z, v1.w));
        }
      }
    }
  }
  __syncwarp();
}

// Epilogue of a tile: this warp's lane quarter of its FT accumulators from acc on, every kEpiSets-th
// group of 16 tokens (kSplit: of this CTA's groups, with the other CTAs' partial sums added in rank
// order) from `set` on; false: a wait expired. The next group's accumulator columns, and for kHidden its a and q, are under
// way while a group is finished; kHidden's first ones come in `in`.
template <int OP, int BN, int FT, int MODE>
__device__ __forceinline__ bool epilogue(const Tile& tl, int f0, const GemmParams& p, uint32_t acc,
                                         int quarter, int set, int lane, uint8_t* st,
                                         const Share& sh, HiddenIn& in, Exchange& x) {
  using C = GemmCfg<OP, BN, FT, MODE>;
  const int first = (MODE == kSplit ? sh.rank + set * sh.width : set) * 16;
  const int next = (MODE == kSplit ? kEpiSets * sh.width : kEpiSets) * 16;
  if (first >= tl.n_valid) return true;
  const uint32_t taddr = acc + ((uint32_t)(quarter * 32) << 16);
  uint32_t r[16];
  tmem_ld_32x32b_x16(taddr + (uint32_t)first, r);
#pragma unroll 1
  for (int j = 0; j < FT; ++j) {
    const int fw = f0 + j * C::kFeat + (OP == kUp ? quarter & 1 : quarter) * 32;  // first of this warp
    const int f = fw + lane;
    const int64_t bi = (int64_t)tl.e * p.n_out + f;
    const bool f_ok = f < p.n_out;
    const float b0 = p.bias0 != nullptr && f_ok ? bf16_to_f32(p.bias0[bi]) : 0.0f;
    const float b1 = p.bias1 != nullptr && f_ok ? bf16_to_f32(p.bias1[bi]) : 0.0f;
    const float* part = MODE == kSplit ? sh.part + set * (kPartChunk / 4) + quarter * 32 + lane : nullptr;
#pragma unroll 1
    for (int c0 = first; c0 < tl.n_valid; c0 += next) {
      tmem_ld_wait16(r);
      uint32_t v[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) v[c] = r[c];
      const bool more = c0 + next < tl.n_valid;
      const int nj = more ? j : j + 1, nc0 = more ? c0 + next : first;
      if (nj < FT) tmem_ld_32x32b_x16(taddr + (uint32_t)(nj * BN + nc0), r);
      if constexpr (MODE == kSplit) {
        const int stride = sh.groups(BN) * (kPartChunk / 4);
#pragma unroll 1
        for (int s = 0; s + 1 < sh.width; ++s)
#pragma unroll
          for (int c = 0; c < 16; ++c)
            v[c] = __float_as_uint(__uint_as_float(v[c]) + part[s * stride + c * kBM]);
        part += kEpiSets * (kPartChunk / 4);
      }
      if constexpr (OP == kUp) {
        if (!finish_up(tl, p, v, fw, c0, b0, b1, lane, st, x)) return false;
      } else {
        const HiddenIn cur = in;
        if (OP == kHidden && nj < FT)
          load_hidden_in(in, p, tl, f0 + nj * C::kFeat + quarter * 32, nc0, lane);
        finish<OP>(tl, p, v, fw, c0, OP == kDown ? b0 : 0.0f, cur, lane, st);
      }
    }
  }
  return true;
}

template <int OP, int BN, int FT, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    gated_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmParams p) {
  using C = GemmCfg<OP, BN, FT, MODE>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_addr - raw_addr);
  float* part = reinterpret_cast<float*>(base + C::kStages * C::kStageBytes);
  uint8_t* epi_tiles = base + C::kStages * C::kStageBytes + C::kPartBytes;
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
  // CTAs that share a tile, this CTA's rank among them, and the tile walk's start and step
  const int width = (int)cluster_nctas();
  const int rank = (int)cluster_ctarank();
  const int first = (int)blockIdx.x / width, step = (int)gridDim.x / width;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(B.full(s), 1);
      mbar_init(B.empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(B.tfull(a), 1);
      mbar_init(B.tempty(a), (MODE == kPair ? 2 : 1) * kEpiWarps);
    }
    mbar_init(B.drain(), 1);
    for (int w = 0; OP == kUp && w < kEpiWarps; ++w) {
      mbar_init(B.given(w), 1);
      mbar_init(B.taken(w), 1);
    }
    mbar_init(B.part_full(), (width > 1 ? width - 1 : 1) * kEpiWarps);
    mbar_init(B.part_free(), (width > 1 ? width - 1 : 1) * kEpiWarps);
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == 1) {
    if constexpr (MODE == kPair) {
      tmem_alloc_pair(smem_u32(tmem_holder), C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_holder), C::kTmemCols);
      tmem_relinquish();
    }
  }
  const int n_ftiles = (p.n_out + C::kTileFeat - 1) / C::kTileFeat;
  if (warp == 2) build_tile_list<BN>(p, n_ftiles, prefix, seg, lane);
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // barriers initialised (and a pair's TMEM allocated) in every CTA
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int total_tiles = prefix[p.E];
  const int n_kb = (p.K + kBK - 1) / kBK;
  const int n_blocks = C::kPhases * n_kb;
  // this CTA's K blocks (of both products of kInput, one after the other)
  const int i0 = MODE == kSplit ? n_blocks * rank / width : 0;
  const int i1 = MODE == kSplit ? n_blocks * (rank + 1) / width : n_blocks;
  auto tile_at = [&](int t) { return decode_tile<BN>(t, prefix, seg, p.E, C::kTileFeat); };

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      Ring ring;
      int issued = 0;
      bool ok = true;
      for (int t = first; t < total_tiles && ok; t += step) {
        const Tile tl = tile_at(t);
        const int n_b = mma_n<MODE>(tl.n_valid) / (MODE == kPair ? 2 : 1);
        const int f0 = tl.f0 + (MODE == kPair ? rank * FT * C::kFeat : 0);
        const int row0 = tl.row0 + (MODE == kPair ? rank * n_b : 0);
        const uint32_t tx = C::kABytes + n_b * 128;
        for (int i = i0; i < i1; ++i) {
          if (!mbar_wait_bounded(B.empty(ring.stage), ring.phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const int ph = C::kPhases == 2 && i >= n_kb ? 1 : 0;
          const int kb = i - ph * n_kb;
          const uint32_t sa = base_addr + ring.stage * C::kStageBytes;
          uint32_t bar = B.full(ring.stage);
          if constexpr (MODE == kPair) {
            if (rank == 0) mbar_arrive_expect_tx(bar, 2 * tx);  // both CTAs' bytes
            bar = cluster_addr(bar, 0);
          } else {
            mbar_arrive_expect_tx(bar, tx);
          }
          load_a<OP, FT, MODE>(sa, maps, p, ph, tl.e, f0, kb, bar);
          load_b<MODE>(sa + C::kABytes, ph ? &maps.b1l : &maps.b0l, ph ? &maps.b1s : &maps.b0s, kb,
                       row0, n_b, bar);
          ++issued;
          ring.next(S);
        }
      }
      // drain: the last min(issued, S) loads may still be landing (a pair's first CTA counts both
      // CTAs' copies; the other stays resident until the cluster barrier below)
      if (MODE != kPair || rank == 0)
        for (int i = max(0, issued - S); i < issued; ++i)
          wait_drain(B.full(i % S), (uint32_t)((i / S) & 1), p.status);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0 && (MODE != kPair || rank == 0)) {
      Ring ring;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int t = first; t < total_tiles && ok; t += step) {
        if (!mbar_wait_bounded(B.tempty(acc), acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const Tile tl = tile_at(t);
        const uint32_t idesc = idesc_bf16_f32_major(MODE == kPair ? 2 * kBM : kBM,
                                                    mma_n<MODE>(tl.n_valid), C::kAMn, false);
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * C::kAccCols);
        for (int i = i0; i < i1; ++i) {
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
            for (int kk = 0; kk < kBK / kUmmaK; ++kk) {
              const uint32_t more = i != i0 || kk != 0 ? 1u : 0u;
              if constexpr (MODE == kPair)
                tc_mma_bf16_pair(d_tmem + (uint32_t)(j * BN), adesc + a_step * (uint64_t)kk,
                                 bdesc + (uint64_t)(2 * kk), idesc, more);
              else
                tc_mma_bf16(d_tmem + (uint32_t)(j * BN), adesc + a_step * (uint64_t)kk,
                            bdesc + (uint64_t)(2 * kk), idesc, more);
            }
          }
          if constexpr (MODE == kPair)
            tc_commit_pair_both(B.empty(ring.stage), cluster_addr(B.empty(ring.stage), 1));
          else
            tc_commit(B.empty(ring.stage));
          ring.next(S);
        }
        if (!ok) break;
        if constexpr (MODE == kPair)
          tc_commit_pair_both(B.tfull(acc), cluster_addr(B.tfull(acc), 1));
        else
          tc_commit(B.tfull(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      // drain every MMA this thread issued before TMEM is released
      if constexpr (MODE == kPair) tc_commit_pair_local(B.drain());
      else tc_commit(B.drain());
      wait_drain(B.drain(), 0, p.status);
    }
  } else {
    // ---------------------------------------------------------- epilogue (warps 2..13)
    const int ew = warp - 2;
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    const int set = ew >> 2;
    uint8_t* st = epi_tiles + ew * kEpiTileBytes;
    const int other = quarter < 2 ? ew - 2 : ew + 2;  // two quarters on (warps 2.. are quarters 2, 3, 0, 1)
    Exchange x{B, ew, other, reinterpret_cast<const float*>(epi_tiles + other * kEpiTileBytes), 0u,
               quarter >= 2, abort_flag, p.status};
    int acc = 0;
    uint32_t acc_phase = 0, part_phase = 0;
    for (int t = first; t < total_tiles; t += step) {
      const Tile tl = tile_at(t);
      const int f0 = tl.f0 + (MODE == kPair ? rank * FT * C::kFeat : 0);
      HiddenIn in = {};
      if constexpr (OP == kHidden)
        load_hidden_in(in, p, tl, f0 + quarter * 32,
                       (MODE == kSplit ? rank + set * width : set) * 16, lane);
      if (!mbar_wait_warp(B.tfull(acc), acc_phase, abort_flag, p.status)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + (uint32_t)(acc * C::kAccCols);
      const Share sh{rank, width, part};
      if (MODE == kSplit && width > 1) {
        // hand the others their groups, once they have read the tile before's
        if (!mbar_wait_cluster_warp(B.part_free(), part_phase ^ 1u, abort_flag, p.status)) break;
        const uint32_t taddr = d_tmem + ((uint32_t)(quarter * 32) << 16);
        const int groups = sh.groups(BN);
        for (int g = set; g * 16 < tl.n_valid; g += kEpiSets) {
          const int owner = g % width;
          if (owner == rank) continue;
          const int slot = (rank < owner ? rank : rank - 1) * groups + g / width;
          const uint32_t to = cluster_addr(smem_u32(part), owner) +
                              (uint32_t)(slot * kPartChunk + (quarter * 32 + lane) * 4);
          uint32_t r[16];
          tmem_ld_32x32b_x16(taddr + (uint32_t)(g * 16), r);
          tmem_ld_wait16(r);
#pragma unroll
          for (int c = 0; c < 16; ++c) st_cluster_u32(to + (uint32_t)(c * kBM * 4), r[c]);
        }
        __syncwarp();
        if (lane == 0)
          for (int s = 1; s < width; ++s)
            mbar_arrive_cluster(cluster_addr(B.part_full(), (rank + s) % width));
        if (!mbar_wait_cluster_warp(B.part_full(), part_phase, abort_flag, p.status)) break;
      }
      if (!epilogue<OP, BN, FT, MODE>(tl, f0, p, d_tmem, quarter, set, lane, st, sh, in, x)) break;
      if (MODE == kSplit && width > 1) {
        __syncwarp();
        if (lane == 0)
          for (int s = 1; s < width; ++s)
            mbar_arrive_cluster(cluster_addr(B.part_free(), (rank + s) % width));
      }
      part_phase ^= 1u;
      // one arrival per warp: the barrier takes arrivals one after another
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(B.tempty(acc), MODE == kPair ? 0 : rank));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before();
  __syncwarp();
  cluster_sync();  // no copy, commit, store or arrive targets another CTA after this
  pdl_trigger();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (MODE == kPair) tmem_dealloc_pair(tmem_base, C::kTmemCols);
    else tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- host side

bool encode_map(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* extent,
                const cuuint64_t* stride, const cuuint32_t* box) {
  return gated_tensor_map(m, ptr, true, rank, extent, stride, box);
}

// Weights [E, K, n] read MN-major in boxes of 64 features x 64 K rows of one expert.
bool weight_map_mn(CUtensorMap* m, const void* ptr, int E, int K, int n) {
  const cuuint64_t extent[3] = {(cuuint64_t)n, (cuuint64_t)K, (cuuint64_t)E};
  const cuuint64_t stride[2] = {(cuuint64_t)n * 2, (cuuint64_t)n * K * 2};
  const cuuint32_t box[3] = {64, kBK, 1};
  return encode_map(m, ptr, 3, extent, stride, box);
}

// One way of running a product: the kernel, its clusters (CTAs of each, and how many of them the
// device holds at once) and its shared memory.
struct Config {
  void (*kern)(GemmMaps, GemmParams);
  int smem, width, slots;
};

cudaError_t launch_clusters(const Config& c, int64_t tiles, cudaStream_t stream, const GemmMaps& m,
                            const GemmParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(tiles, c.slots) * c.width));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = c.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)c.width;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, c.kern, m, p);
  count_launch();
  return e;
}

// The kernel for a mode in clusters of `width`, with its slots on this device (asked once per
// kernel, width and device; 0: such clusters do not fit).
template <int OP, int BN, int FT, int MODE>
cudaError_t config_of(int width, Config* c) {
  *c = Config{gated_gemm_kernel<OP, BN, FT, MODE>, GemmCfg<OP, BN, FT, MODE>::kSmemBytes, width, 0};
  static int attr_done[64] = {0};  // per instantiation and device
  cudaError_t e = ensure_dynamic_smem(c->kern, c->smem, attr_done);
  if (e != cudaSuccess) return e;
  static std::atomic<int> cache[kMaxSplit + 1][kMaxDevices];
  return cluster_slots((const void*)c->kern, width, kThreads, c->smem, cache[width], &c->slots);
}

template <int OP, int BN>
cudaError_t config_of(int ft, int mode, int width, Config* c) {
  if constexpr (BN <= 128)
    if (mode == kSplit) return config_of<OP, BN, 1, kSplit>(width, c);
  if constexpr (BN <= 128)
    if (ft == 2) return config_of<OP, BN, 2, kPair>(2, c);
  return config_of<OP, BN, 1, kPair>(2, c);
}

template <int OP>
cudaError_t config_of(int bn, int ft, int mode, int width, Config* c) {
  switch (bn) {
    case 32: return config_of<OP, 32>(ft, mode, width, c);
    case 64: return config_of<OP, 64>(ft, mode, width, c);
    case 128: return config_of<OP, 128>(ft, mode, width, c);
    default: return config_of<OP, 256>(ft, mode, width, c);
  }
}

// Chooses how to run a product by an estimate of its time and launches it. Per K block a CTA takes
// the larger of its loads' time (75 bytes/ns) and its MMAs' (2 cycles a token column and A tile);
// rounds of tiles over the device's clusters multiply that; no way is faster than the weights come
// from HBM, and of equal ones the first wins. So come
//   - for many tiles of up to 128 rows, pairs with two A tiles, whose token rows cost the fewest
//     loads (128 experts of 86 rows, d 1024, f 4096, up: 386 us; one A tile 431, single CTAs 444);
//   - for more rows pairs with one A tile and 256 token columns (TMEM holds two sets of
//     accumulators only of one such tile; 128 rows an expert on average, 160 at most, up: 429 us;
//     two A tiles and one set, the epilogue not overlapped, 480);
//   - splits where tiles are fewer than SMs (8 rows, d 8192 -> 2048, weights cold: 18.8 us in clusters
//     of 6, 19.5 of 4, 25.5 of 2, 27.7 of 8, of which only 15 of 16 fit at once, 44 unsplit).
template <int OP>
cudaError_t launch_op(const GemmMaps& m, const GemmParams& p, int64_t capacity_hint,
                      cudaStream_t stream) {
  // rows of an expert and experts with rows, as far as the host knows
  const int64_t rows = std::max<int64_t>(1, std::min(capacity_hint, p.rows_max));
  const int64_t experts = std::min<int64_t>(p.E, p.rows_max);
  const int feat = OP == kUp ? kBM / 2 : kBM;
  const int64_t n_blocks = (int64_t)(OP == kInput ? 2 : 1) * ((p.K + kBK - 1) / kBK);
  const double hbm_ns = (double)experts * p.n_out * n_blocks * kBK * (OP == kUp ? 4 : 2) / 6500.0;
  Config best{};
  int64_t best_tiles = 0;
  double best_ns = 0;
  auto consider = [&](int bn, int ft, int mode, int width) -> cudaError_t {
    Config c{};
    const cudaError_t e = config_of<OP>(bn, ft, mode, width, &c);
    if (e != cudaSuccess) return e;
    if (c.slots < 1) return cudaSuccess;  // not on this device
    const int feats = feat * ft * (mode == kPair ? 2 : 1);
    const int64_t tiles = experts * ((rows + bn - 1) / bn) * ((p.n_out + feats - 1) / feats);
    const int64_t rounds = (tiles + c.slots - 1) / c.slots;
    const double n = (double)std::min<int64_t>((rows + 15) / 16 * 16, bn);
    const double load = (ft * kBM + (mode == kPair ? n / 2 : n)) * (kBK * 2) / 75.0;
    const double mma = ft * 2 * n / 1.7;
    const int ways = mode == kSplit ? width : 1;
    double ns = (double)(rounds * ((n_blocks + ways - 1) / ways)) * std::max(load, mma);
    if (mode == kSplit && width > 1) ns += 1500;  // the meeting of the partial sums
    ns = std::max(ns, hbm_ns);
    if (best.kern == nullptr || ns < best_ns) {
      best = c;
      best_tiles = tiles;
      best_ns = ns;
    }
    return cudaSuccess;
  };
  cudaError_t e = cudaSuccess;
  const int fit = rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
  if (fit <= 128) e = consider(fit, 2, kPair, 2);
  if (e == cudaSuccess) e = consider(fit, 1, kPair, 2);
  if (fit == 256 && e == cudaSuccess) e = consider(128, 1, kPair, 2);
  for (int width = 1; width <= kMaxSplit && n_blocks >= 4 * width; ++width)
    if (e == cudaSuccess && parts_of(std::min(fit, 128), width) <= kPartChunks)
      e = consider(std::min(fit, 128), 1, kSplit, width);
  if (e == cudaSuccess && best.kern == nullptr) e = consider(std::min(fit, 128), 1, kSplit, 1);
  if (e != cudaSuccess) return e;
  if (best.kern == nullptr) return cudaErrorLaunchOutOfResources;
  return launch_clusters(best, best_tiles, stream, m, p);
}

// Both box heights of a token operand [rows, K].
bool token_maps(CUtensorMap* l, CUtensorMap* s, const void* ptr, int64_t rows, int K) {
  return make_bf16_map_2d(l, ptr, rows, K, kBK, kBoxL) &&
         make_bf16_map_2d(s, ptr, rows, K, kBK, kBoxS);
}

}  // namespace

bool gated_tensor_map(CUtensorMap* m, const void* ptr, bool bf16, int rank, const cuuint64_t* extent,
                      const cuuint64_t* stride, const cuuint32_t* box) {
  using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                     const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                     const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn != nullptr &&
         fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
            (cuuint32_t)rank, const_cast<void*>(ptr), extent, stride, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t enqueue_gated_up_bf16(const GatedFfn& g, void* h, void* saved_a, void* saved_q,
                                  int* status, cudaStream_t stream) {
  if (g.rows_max == 0) return cudaSuccess;
  GemmMaps m;
  GemmParams p{};
  if (!make_bf16_map_2d(&m.a0, g.w_gate, (int64_t)g.E * g.f, g.d, kBK, kBM / 2) ||
      !make_bf16_map_2d(&m.a1, g.w_up, (int64_t)g.E * g.f, g.d, kBK, kBM / 2))
    return cudaErrorInvalidValue;
  if (!token_maps(&m.b0l, &m.b0s, g.x, g.rows_max, g.d)) return cudaErrorInvalidValue;
  m.b1l = m.b0l;
  m.b1s = m.b0s;
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
