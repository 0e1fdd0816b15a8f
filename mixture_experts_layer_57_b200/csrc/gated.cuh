// Gate activations of the gated expert FFN and their derivatives.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

// Coefficients of gate_act's fast Phi.
constexpr float kErfcP = 0.38f;
__device__ constexpr float kErfcC[7] = {0.214287281f,   0.216577843f, 0.180592224f, 0.247839555f,
                                        -0.0699200258f, 0.336040914f, -0.125418812f};

// a = act(z), da = act'(z).
//   SiLU: act = z s, act' = s (1 + z (1 - s)) with s = 1 / (1 + e^-z)
//   GeLU (erf form): act = z Phi(z), act' = Phi(z) + z phi(z)
// e^-z overflowing to infinity gives s = 0, the limit. FAST (bf16 layers) uses the approximate
// exponential and division, and Phi(-|z|) = e^(-x^2) / 2 times a polynomial without constant term in
// t = 1 / (1 + p x), x = |z| / sqrt 2: the form of Abramowitz and Stegun, Handbook of Mathematical
// Functions, 7.1.26, with the exponential that phi needs too, but with seven terms fitted here to the
// least largest RELATIVE error of erfc(x) e^(x^2) over [0, 13] (2^-19; 7.1.26 bounds the absolute one
// and is 0.4% off at z = -6, 1% at -8). With the exponential's own error act(z) is within 2^-15 of its
// value down to z = -12.5, far below the bf16 rounding that follows.
template <bool FAST = false>
__device__ __forceinline__ void gate_act(float z, int act, float& a, float& da) {
  if (act == MOE_GATE_SILU) {
    const float s = FAST ? __fdividef(1.0f, 1.0f + __expf(-z)) : 1.0f / (1.0f + expf(-z));
    a = z * s;
    da = s * (1.0f + z * (1.0f - s));
  } else if constexpr (FAST) {
    const float x = fabsf(z) * 0.70710678118654752440f;
    const float t = __fdividef(1.0f, fmaf(kErfcP, x, 1.0f));
    const float e = __expf(-x * x);
    float poly = kErfcC[6];
#pragma unroll
    for (int i = 5; i >= 0; --i) poly = fmaf(t, poly, kErfcC[i]);
    poly *= t;
    const float tail = 0.5f * poly * e;  // Phi(-|z|)
    const float cdf = z >= 0.0f ? 1.0f - tail : tail;
    a = z * cdf;
    da = fmaf(z * 0.39894228040143267794f, e, cdf);
  } else {
    // erfc, as 1 + erf cancels for negative z (nothing of act(-6) was left, 4% of act(-5) wrong)
    const float cdf = 0.5f * erfcf(z * -0.70710678118654752440f);
    a = z * cdf;
    da = cdf + z * 0.39894228040143267794f * expf(-0.5f * z * z);
  }
}

// Eight values in 8 x 16 bits with one exponent between them (what the forward pass of a bf16
// layer keeps for the backward pass): each is rounded to fp16 after scaling by the power of two, of
// even exponent, that brings the largest magnitude into [1/4, 1), which leaves bit 14 of every fp16
// zero; there go the eight bits of a code, one each. Bits 0..6 of it are half the exponent. Values
// within 2^-12 of the largest keep 11 bits where bf16 keeps 8 (plain bf16 copies of these two tensors
// raised the error of the weight gradients by a fifth), smaller ones an error of up to 2^-25 at that
// scale, which is bf16's half step at 2^-17. Where a value other than zero lies below 2^-17 there, all
// eight are scaled bf16 instead (bit 7 of the code; bit 14 of a bf16 below 1 is zero too): a gate that is
// shut beside one wide open keeps its 8 bits. Where a magnitude is 2^126 or more, infinite or NaN, bits
// 0..6 are all set and every value is the sign, the exponent and six bits of mantissa of its fp32 form.
__device__ __forceinline__ uint4 pack_block8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(v[i])));
  const uint32_t half = ((__float_as_uint(m) >> 23) + 1u) >> 1;
  uint32_t w[4];
  if (half >= 127u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t u = __float_as_uint(v[2 * i + j]);
        if ((u & 0x7fffffffu) > 0x7f800000u) u |= 0x00400000u;  // a NaN stays one when cut
        h[j] = ((u >> 16) & 0x8000u) | ((u >> 17) & 0x3fffu);
      }
      w[i] = h[0] | (h[1] << 16);
    }
  } else {
    const float scale = __uint_as_float((253u - 2u * half) << 23);  // 2^(126 - 2 half)
    float s[8], least = 1.0f;  // the smallest magnitude other than zero
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = v[i] * scale;
      least = fminf(least, v[i] != 0.0f ? fabsf(s[i]) : 1.0f);
    }
    const bool wide = least < 0x1p-17f;
    const uint32_t code = half | (wide ? 0x80u : 0u);
    const uint32_t bits = (code & 15u) | ((code >> 4) << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h;
      if (wide) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(s[2 * i + 1]), "f"(s[2 * i]));
      else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(s[2 * i + 1]), "f"(s[2 * i]));
      w[i] = h | (((bits >> i) << 14) & 0x40004000u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // code 127
  return make_uint4(w[0] | 0x40004000u, w[1] | 0x40004000u, w[2] | 0x40004000u, w[3] | 0x00004000u);
}
__device__ __forceinline__ void unpack_block8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bits |= ((w[i] & 0x40004000u) >> 14) << i;
  const uint32_t code = (bits | (bits >> 12)) & 0xffu, half = code & 0x7fu;
  if (half == 127u) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t h = w[i] >> (16 * j);
        v[2 * i + j] = __uint_as_float(((h & 0x8000u) << 16) | ((h & 0x3fffu) << 17));
      }
  } else {
    const float scale = __uint_as_float((2u * half + 1u) << 23);  // 2^(2 half - 126)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = w[i] & 0xbfffbfffu;
      float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
      if (code & 0x80u) f = make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
}

// Tiled bulk tensor copies global -> shared of three dimensions, completion counted on `bar` in bytes;
// the _pair form lands in this CTA and counts on an mbarrier of either CTA of a pair (a shared::cluster
// address).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, int32_t x,
                                                 int32_t y, int32_t z, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
      : "memory");
}

// Two values rounded to bf16 in one instruction (conversions are slow one by one: 64 a lane bounded
// the weight-gradient kernel's epilogue).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Waits for the tcgen05.ld into r; the operands keep every use of r behind it.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// mbar_wait_bounded_warp, with a first try before the timer is read.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                               int* status) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         mbar_wait_bounded_warp(bar, parity, abort, status);
}

// Store of a box from shared memory (what lies outside the tensor is not written), in this thread's
// current bulk group.
__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int32_t x, int32_t y,
                                             int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N of this thread's bulk groups have not read their shared memory yet / are not done.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Makes this thread's shared-memory writes visible to TMA and MMA reads that follow.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Clusters: the CTAs of this one, a store into another CTA's shared memory, and the bounded wait
// (whole warp) on a barrier that other CTAs arrive on, which also makes their stores visible.
__device__ __forceinline__ uint32_t cluster_nctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_smem, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_smem), "r"(v) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort,
                                                  int* status) {  // one thread
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      set_device_error(status, MOE_DEVERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool mbar_wait_cluster_warp(uint32_t bar, uint32_t parity,
                                                       volatile int* abort, int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (int it = 0;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait_cluster(bar, parity))) return true;
    int give_up = 0;
    if ((threadIdx.x & 31) == 0 && it >= 256)
      give_up = (*abort != 0) || (global_timer_ns() - t0 > kWaitLimitNs);
    give_up = __shfl_sync(0xffffffffu, give_up, 0);
    if (give_up) {
      if ((threadIdx.x & 31) == 0 && *abort == 0) {
        set_device_error(status, MOE_DEVERR_TIMEOUT);
        *abort = 1;
      }
      return false;
    }
  }
}

// A tensor map of the given extents (innermost first, in elements), byte strides of the outer
// dimensions and box, 128-byte swizzle (host).
bool gated_tensor_map(CUtensorMap* m, const void* ptr, bool bf16, int rank, const cuuint64_t* extent,
                      const cuuint64_t* stride, const cuuint32_t* box);

}  // namespace moe
