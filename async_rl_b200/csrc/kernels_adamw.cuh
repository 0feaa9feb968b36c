// kernels_adamw.cuh -- one AdamW step over many tensors, states in fp32 or in 8-bit blocks.
//
// The step is bound by HBM: 16 bytes of fp32 states (4 with 8-bit ones), the gradient, 8 bytes of
// master weights and 2 of the bf16 copy an element, against about 16 operations.  A warp takes 256
// consecutive elements at a time, eight a lane, so every lane's loads and stores are 8, 16 or 32
// bytes wide and a block of the 8-bit states is one warp's: its two maxima are shuffles, with
// nothing in shared memory.  The tensors' addresses travel as kernel parameters (at most 30 KB a
// launch), so a call copies nothing to the device and can be captured.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "bi_optim.h"
#include "sm100.cuh"

namespace bi {

constexpr int kAdamThreads = 256;
constexpr int kAdamUnit = 256;                      // elements of a warp's turn = a block of 8-bit states
constexpr int kAdamChunk = kAdamUnit * (kAdamThreads / 32);  // elements of a block
constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Inv = 1.0f / 448.0f;
constexpr float kF32Max = 3.4028235e38f;
constexpr float kE4m3Tiny = 0.001953125f;           // 2^-9, the smallest positive value

// Above these, states of 8 bits are not rounded to nearest.  A step moves m by 1 - beta1 and sqrt(v) by
// (1 - beta2) / 2 of itself; where that is less than half a code's step (1/18 of 9/8) nearest gives the old code
// back, and the state stands still.  beta1: the arithmetic bound.  beta2: the gradients' own scatter carries
// sqrt(v) over the edge for a while.  Measured as held over true sqrt(v), 10% and 90% quantiles, some thousand
// steps after 65,536 gradients changed their scales: nearest 0.91 and 1.10 (0.95), 0.90 and 1.11 (0.96), 0.90 and 1.20
// (0.98), 0.92 and 4.8 (0.99), 0.44 and 4.7 (0.999); dithered 0.87 and 1.15, 0.86 and 1.16, 0.84 and 1.19,
// 0.82 and 1.22, 0.79 and 1.26.  Dithering sqrt(v) costs 437 us for 357 of nearest (110 million elements; 447 and 480
// with five and four blocks an SM), both states 470.
constexpr double kNearestBeta1 = 17.0 / 18.0;
constexpr double kNearestBeta2 = 0.96;

struct AdamHyper {
  float b1, c1, b2, c2;   // beta1, 1 - beta1, beta2, 1 - beta2
  float rate, root, keep, eps;  // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t), 1 - lr wd, eps
};
struct AdamTensor {
  void* p;
  float* master;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
};
template <int kMax>
struct AdamTable {
  AdamTensor t[kMax];
  uint32_t first[kMax + 1];  // first block of each tensor
  uint32_t wide[(kMax + 31) / 32];  // bit i: tensor i's addresses allow vector access
  int32_t count;
};
struct AdamArgs {
  AdamHyper h;
  double lr, beta1, beta2;
  int64_t step;
  bool dither_m, dither_v;
  const float* grad_scale;
  const int64_t* step_dev;
  int32_t* status;
  int32_t set_status;  // this launch is the call's first
};

struct F8 {
  float x[8];
};
__device__ __forceinline__ F8 adam_ld_f32(const float* p) {
  uint32_t r[8];
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
  F8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f.x[e] = __uint_as_float(r[e]);
  return f;
}
__device__ __forceinline__ void adam_st_f32(float* p, const F8& f) {
  uint32_t r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(f.x[e]);
  st_global_v8(p, r);
}
__device__ __forceinline__ float bf16_up(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ F8 adam_ld_bf16(const uint16_t* p) {
  uint32_t r[4];
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "l"(p));
  F8 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f.x[2 * e] = bf16_up(r[e] & 0xffffu);
    f.x[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
  }
  return f;
}
__device__ __forceinline__ void adam_st_bf16(uint16_t* p, const F8& f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f.x[0], f.x[1]), pack_bf16x2(f.x[2], f.x[3]),
                                            pack_bf16x2(f.x[4], f.x[5]), pack_bf16x2(f.x[6], f.x[7]));
}
// Eight e4m3 codes, two at a time (a code is exact in fp16), and back (to nearest even, saturated).
__device__ __forceinline__ void e4m3_up8(const uint32_t (&w)[2], float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[e / 2] >> (16 * (e % 2))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t e4m3_down2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// 32 bits for element i of its tensor at step t: products with odd numbers from the fractions of irrational ones
// (the golden ratio, roots of 11, 2, 17, 3 and 13), high bits folded onto low ones in between.
__device__ __forceinline__ uint32_t adam_bits(int64_t i, int64_t t) {
  uint32_t x = static_cast<uint32_t>(i) * 0x9E3779B9u + static_cast<uint32_t>(i >> 32) * 0x510E527Fu +
               static_cast<uint32_t>(t) * 0x6A09E667u + static_cast<uint32_t>(t >> 32) * 0x1F83D9ABu;
  x ^= x >> 16;
  x *= 0xBB67AE85u;
  x ^= x >> 15;
  x *= 0x9B05688Du;
  return x ^ (x >> 16);
}
// y as the e4m3 value below or above it in magnitude, above with the odds of its place between them, r in
// [0, 65536).  |y| / spacing is below 16 and a power of two's multiple: exact; the sum is rounded.
__device__ __forceinline__ float adam_dither(float y, uint32_t r) {
  const uint32_t top = max(__float_as_uint(y) & 0x7f800000u, 0x3c800000u);  // 2^-6 and less: the spacing 2^-9
  const float spacing = __uint_as_float(top - (3u << 23)), inv = __uint_as_float((257u << 23) - top);
  const float c = floorf(__fadd_rn(__fmul_rn(fabsf(y), inv), __fmul_rn(static_cast<float>(r), 1.0f / 65536.0f)));
  return copysignf(__fmul_rn(c, spacing), y);
}

// One element; every operation is rounded, none contracted, so a plain evaluation in the same order
// gives the same bits (and with 8-bit states the same codes).
__device__ __forceinline__ void adam_one(const AdamHyper& h, float gs, float g, float& p, float& m, float& v, float& root) {
  g = __fmul_rn(g, gs);  // gs = 1 without a grad_scale: exact
  m = __fadd_rn(__fmul_rn(m, h.b1), __fmul_rn(g, h.c1));
  v = __fadd_rn(__fmul_rn(v, h.b2), __fmul_rn(__fmul_rn(g, g), h.c2));
  root = __fsqrt_rn(v);
  const float den = __fadd_rn(__fmul_rn(root, h.root), h.eps);
  p = __fsub_rn(__fmul_rn(p, h.keep), __fdiv_rn(__fmul_rn(m, h.rate), den));
}

__device__ __forceinline__ float adam_warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// kState: how states are held; kPBf16: bf16 params; kMaster: with fp32 masters; kGBf16: bf16 gradients
enum AdamState : int { kAdam32 = 0, kAdam8 = 1, kAdam8Dither = 2 };
template <int kMax, int kState, bool kPBf16, bool kMaster, bool kGBf16>
__global__ void __launch_bounds__(kAdamThreads, kState == kAdam32 ? 3 : 6)
    k_adamw(const __grid_constant__ AdamTable<kMax> tab, const AdamArgs a) {
  constexpr bool kState8 = kState != kAdam32;
  __shared__ AdamHyper sh;
  AdamHyper h = a.h;
  if (a.step_dev) {
    const int64_t t = *a.step_dev;
    if (t < 1) {
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 1 /* BI_ERR_INVALID_ARG */;
      return;
    }
    if (threadIdx.x == 0) {
      h.rate = static_cast<float>(a.lr / (1.0 - pow(a.beta1, static_cast<double>(t))));
      h.root = static_cast<float>(1.0 / sqrt(1.0 - pow(a.beta2, static_cast<double>(t))));
      sh = h;
    }
    __syncthreads();
    h = sh;
  }
  if (a.set_status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  // the block's tensor: the last one whose first block is not behind this one
  int lo = 0, hi = tab.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (tab.first[mid] <= blockIdx.x)
      lo = mid;
    else
      hi = mid - 1;
  }
  const AdamTensor& t = tab.t[lo];
  const bool wide = (tab.wide[lo / 32] >> (lo % 32)) & 1u;
  const int64_t n = t.n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x - tab.first[lo]) * kAdamChunk + warp * kAdamUnit;
  const int64_t i0 = unit + lane * 8;
  if (unit >= n) return;  // the whole warp
  float* pf = kMaster ? t.master : static_cast<float*>(t.p);
  uint16_t* pb = static_cast<uint16_t*>(t.p);
  const float* gf = static_cast<const float*>(t.g);
  const uint16_t* gb = static_cast<const uint16_t*>(t.g);
  // What a lane holds.  One unit a warp and, with 8-bit states, six blocks an SM: their step is bound by
  // the latency of its chain of conversions, roots and quotients, which warps hide better than loads ahead
  // (110 million elements, bf16 gradients, masters: 342 us when it was chosen, two units with both loads ahead 413, four
  // blocks 382; 357 now, and 413 with the step on the device, whose factors thread 0 of each block computes.)
  struct Held {
    F8 p, g, m, v;
    uint32_t mw[2], vw[2];
    float sm, sv;
  };
  auto load = [&](Held& x) {
    if (wide && i0 + 8 <= n) {
      x.g = kGBf16 ? adam_ld_bf16(gb + i0) : adam_ld_f32(gf + i0);
      x.p = (kPBf16 && !kMaster) ? adam_ld_bf16(pb + i0) : adam_ld_f32(pf + i0);
      if (!kState8) {
        x.m = adam_ld_f32(static_cast<const float*>(t.m) + i0);
        x.v = adam_ld_f32(static_cast<const float*>(t.v) + i0);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t i = i0 + e;
        const bool in = i < n;
        x.g.x[e] = !in ? 0.f : kGBf16 ? bf16_up(gb[i]) : gf[i];
        x.p.x[e] = !in ? 0.f : (kPBf16 && !kMaster) ? bf16_up(pb[i]) : pf[i];
        if (!kState8) {
          x.m.x[e] = in ? static_cast<const float*>(t.m)[i] : 0.f;
          x.v.x[e] = in ? static_cast<const float*>(t.v)[i] : 0.f;
        }
      }
    }
    if (kState8) {
      const uint8_t* mc = static_cast<const uint8_t*>(t.m) + i0;
      const uint8_t* vc = static_cast<const uint8_t*>(t.v) + i0;
      x.mw[0] = x.mw[1] = x.vw[0] = x.vw[1] = 0u;
      if (wide && i0 + 8 <= n) {
        const uint2 a2 = *reinterpret_cast<const uint2*>(mc), b2 = *reinterpret_cast<const uint2*>(vc);
        x.mw[0] = a2.x, x.mw[1] = a2.y, x.vw[0] = b2.x, x.vw[1] = b2.y;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i0 + e < n) {
            x.mw[e / 4] |= static_cast<uint32_t>(mc[e]) << (8 * (e % 4));
            x.vw[e / 4] |= static_cast<uint32_t>(vc[e]) << (8 * (e % 4));
          }
      }
      const int64_t block = unit / kAdamUnit;
      x.sm = t.ms[block];
      x.sv = t.vs[block];
    }
  };
  auto work = [&](Held& x) {
    const bool full = wide && i0 + 8 <= n;
    if (kState8) {
      e4m3_up8(x.mw, x.m.x);
      e4m3_up8(x.vw, x.v.x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x.m.x[e] = __fmul_rn(x.m.x[e], x.sm);
        const float r = __fmul_rn(x.v.x[e], x.sv);
        x.v.x[e] = __fmul_rn(r, r);
      }
    }
    float root[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) adam_one(h, gs, x.g.x[e], x.p.x[e], x.m.x[e], x.v.x[e], root[e]);
    if (kState8) {
      float mm = 0.f, mv = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // an infinity as the block's maximum would make NaN of all its elements: it becomes one itself (fmaxf
        // passes NaN over)
        x.m.x[e] = fabsf(x.m.x[e]) <= kF32Max ? x.m.x[e] : __int_as_float(0x7fffffff);
        root[e] = root[e] <= kF32Max ? root[e] : __int_as_float(0x7fffffff);
        if (i0 + e < n) {
          mm = fmaxf(mm, fabsf(x.m.x[e]));
          mv = fmaxf(mv, root[e]);
        }
      }
      mm = adam_warp_max(mm);
      mv = adam_warp_max(mv);
      // 448 / max is infinite for a maximum below 1.3e-36: zeros then, which a step with any eps to speak of would
      // not tell from it; sqrt(v) is never that small
      float im = __fmul_rn(__frcp_rn(mm), kE4m3Max);
      if (im > kF32Max) im = mm = 0.f;
      const float iv = mv > 0.f ? __fmul_rn(__frcp_rn(mv), kE4m3Max) : 0.f;
      uint32_t mw[2] = {}, vw[2] = {};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float r = __fmul_rn(root[e], iv);
        root[e] = root[e] > 0.f ? fmaxf(r, kE4m3Tiny) : r;
        x.m.x[e] = __fmul_rn(x.m.x[e], im);
        if (kState == kAdam8Dither) {
          const uint32_t bits = adam_bits(i0 + e, a.step_dev ? *a.step_dev : a.step);
          if (a.dither_m) x.m.x[e] = adam_dither(x.m.x[e], bits & 0xffffu);
          if (a.dither_v) root[e] = adam_dither(root[e], bits >> 16);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        mw[e / 4] |= e4m3_down2(x.m.x[e], x.m.x[e + 1]) << (8 * (e % 4));
        vw[e / 4] |= e4m3_down2(root[e], root[e + 1]) << (8 * (e % 4));
      }
      uint8_t* mc = static_cast<uint8_t*>(t.m) + i0;
      uint8_t* vc = static_cast<uint8_t*>(t.v) + i0;
      if (full) {
        *reinterpret_cast<uint2*>(mc) = make_uint2(mw[0], mw[1]);
        *reinterpret_cast<uint2*>(vc) = make_uint2(vw[0], vw[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i0 + e < n) {
            mc[e] = static_cast<uint8_t>(mw[e / 4] >> (8 * (e % 4)));
            vc[e] = static_cast<uint8_t>(vw[e / 4] >> (8 * (e % 4)));
          }
      }
      if (lane == 0) {
        const int64_t block = unit / kAdamUnit;
        t.ms[block] = __fmul_rn(mm, kE4m3Inv);
        t.vs[block] = __fmul_rn(mv, kE4m3Inv);
      }
    }
    if (full) {
      if (kPBf16) adam_st_bf16(pb + i0, x.p);
      if (!kPBf16 || kMaster) adam_st_f32(pf + i0, x.p);
      if (!kState8) {
        adam_st_f32(static_cast<float*>(t.m) + i0, x.m);
        adam_st_f32(static_cast<float*>(t.v) + i0, x.v);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t i = i0 + e;
        if (i >= n) continue;
        if (kPBf16) pb[i] = static_cast<uint16_t>(pack_bf16x2(x.p.x[e], 0.f) & 0xffffu);
        if (!kPBf16 || kMaster) pf[i] = x.p.x[e];
        if (!kState8) {
          static_cast<float*>(t.m)[i] = x.m.x[e];
          static_cast<float*>(t.v)[i] = x.v.x[e];
        }
      }
    }
  };
  Held x;
  load(x);
  work(x);
}

}  // namespace bi
