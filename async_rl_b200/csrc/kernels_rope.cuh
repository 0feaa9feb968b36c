// kernels_rope.cuh -- RMS norm of every query and key head with the rotation of its position in the
// same pass, and the gradient of both.
//
// With x one head's vector of D values, r = 1 / sqrt(mean(x^2) + eps), y = x r g and the first R
// values of y taken as R / 2 pairs (y_i, y_{i + R/2}) with the angles a_i = position * inv_freq_i:
//   z_i = y_i cos a_i - y_{i + R/2} sin a_i,   z_{i + R/2} = y_{i + R/2} cos a_i + y_i sin a_i,
// and z = y past R.  The gradient turns dz back by the same angles (dy), then
//   dg = sum over tokens and heads of dy n,  n = x r,   dx = r (dy g - n mean(dy g n)).
//
// Both are bound by HBM (4 and 6 bytes an element): everything between the loads and the stores
// stays in registers in fp32 and is rounded to bf16 once.  A head takes LH lanes of a warp, 16
// values a lane, as two 16-byte vectors that lie R / 2 apart, so a rotation needs no exchange
// between lanes.  The R / 2 cosines and sines of a token are computed once for all its heads, one
// or a few a lane, and shared through shared memory.  The angle is taken in turns in 64 bits
// (position * inv_freq / 2 pi, whole turns dropped), because a far position times a frequency has
// more than 24 significant bits; what is left, below half a turn, goes to sincospif in 32 bits.
// Measured: 76,239 tokens of 14 heads of 128 take 124 us (4.4 TB/s), 131,072 of 40 heads backward 795 us
// (5.1 TB/s).  The forward has 16 warps an SM (122 registers) with two slots of loads each in flight; three blocks an
// SM instead of two spill registers (162 us).  The backward's sums of both gains fill its 128 registers, and 116 bytes a
// thread spill.  Angles by a 64-bit fixed-point product measured the same.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "sm100.cuh"

namespace bi {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxD = 256;

struct RopeArgs {
  const uint16_t *q, *k;      // [T][Hq][D], [T][Hkv][D]: rows of q_ld, k_ld elements
  const uint16_t *dzq, *dzk;  // backward: gradients of the outputs
  uint16_t *oq, *ok;          // outputs (backward: gradients of q and k)
  const uint16_t *gq, *gk;    // [D] gains, or NULL: rotation only
  const int32_t* pos;         // [T]
  const float* inv_freq;      // [R / 2]
  int64_t q_ld, k_ld, dzq_ld, dzk_ld, oq_ld, ok_ld;
  int64_t T;
  int32_t Hq, Hkv, D, R;
  int32_t sb, nsb;            // slots of one warp's item, items of a token
  float eps;
  float* parts;               // backward: [blocks][2][D] partial gain gradients
  int32_t* status;
};

__device__ __forceinline__ uint4 rope_ld(const uint16_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
// Eight bf16 as four pairs of floats (pairs take one instruction where single values take two).
__device__ __forceinline__ void rope_unpack(const uint4& u, float2* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
}
__device__ __forceinline__ uint4 rope_pack(const float2* f) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                    pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ void rope_unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 rope_pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
// (x, y) turned: x c - y s and y c + x s, four pairs of each.
__device__ __forceinline__ void rope_turn(float2* x, float2* y, const float2* c, const float2* s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = x[e], b = y[e], p = mul2(a, c[e]);
    x[e] = make_float2(fmaf(-b.x, s[e].x, p.x), fmaf(-b.y, s[e].y, p.y));
    y[e] = fma2(b, c[e], mul2(a, s[e]));
  }
}
template <int LH>
__device__ __forceinline__ float rope_sum(float v) {
#pragma unroll
  for (int o = LH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The token's cosines and sines, by all lanes of the warp.
__device__ __forceinline__ void rope_angles(const RopeArgs& a, int64_t t, int lane, float2* cs) {
  constexpr double kInv2Pi = 0.15915494309189533577;
  const double p = static_cast<double>(__ldg(a.pos + t));
  __syncwarp();  // the previous token's readers are done
  for (int i = lane; i < a.R / 2; i += 32) {
    const double turns = p * (static_cast<double>(__ldg(a.inv_freq + i)) * kInv2Pi);
    float s, c;
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(c, s);
  }
  __syncwarp();
}

// A lane's two vectors of its head: rotated partners below R, neighbours past it.
struct RopeLane {
  int c0, c1;    // first element of each vector
  bool active;   // the lane has elements (D / 16 lanes of LH do)
  bool turns;    // they are rotated
};
__device__ __forceinline__ RopeLane rope_lane(const RopeArgs& a, int u) {
  RopeLane l;
  l.active = u < a.D / 16;
  l.turns = u < a.R / 16;
  l.c0 = l.turns ? 8 * u : a.R + 16 * (u - a.R / 16);
  l.c1 = l.turns ? a.R / 2 + 8 * u : l.c0 + 8;
  return l;
}

// A slot is the 32 / LH heads that a warp takes at a time; a token's slots are q's, then k's.
struct RopeSlots {
  int nq, n;  // of q, of both
};
template <int LH>
__device__ __forceinline__ RopeSlots rope_slots(const RopeArgs& a) {
  constexpr int HI = 32 / LH;
  const int nq = (a.Hq + HI - 1) / HI;
  return RopeSlots{nq, nq + (a.Hkv + HI - 1) / HI};
}

constexpr int kRopeFwdBlocks = 2;  // of an SM
template <int LH, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, kRopeFwdBlocks) k_qk_rope(const RopeArgs a) {
  __shared__ float2 cs_all[kRopeWarps][kRopeMaxD / 2];
  constexpr int HI = 32 / LH;  // heads at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2* cs = cs_all[warp];
  const RopeLane ln = rope_lane(a, lane % LH);
  const int sub = lane / LH;
  const RopeSlots sl = rope_slots<LH>(a);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  uint4 g[2][2] = {};  // gains of the lane's elements: [q, k][vector]
  if (kNorm && ln.active) {
    g[0][0] = *reinterpret_cast<const uint4*>(a.gq + ln.c0);
    g[0][1] = *reinterpret_cast<const uint4*>(a.gq + ln.c1);
    g[1][0] = *reinterpret_cast<const uint4*>(a.gk + ln.c0);
    g[1][1] = *reinterpret_cast<const uint4*>(a.gk + ln.c1);
  }
  const int64_t items = a.T * a.nsb;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kRopeWarps;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; it < items; it += nw) {
    const int64_t t = it / a.nsb;
    const int i0 = static_cast<int>(it - t * a.nsb) * a.sb;
    const int i1 = i0 + a.sb < sl.n ? i0 + a.sb : sl.n;
    auto load = [&](int i, uint4 (&x)[2]) {
      const bool q = i < sl.nq;
      const int h = (q ? i : i - sl.nq) * HI + sub;
      x[0] = x[1] = make_uint4(0u, 0u, 0u, 0u);
      if (ln.active && i < i1 && h < (q ? a.Hq : a.Hkv)) {
        const uint16_t* p = (q ? a.q + t * a.q_ld : a.k + t * a.k_ld) + static_cast<int64_t>(h) * a.D;
        x[0] = rope_ld(p + ln.c0);
        x[1] = rope_ld(p + ln.c1);
      }
    };
    uint4 nx[2][2];  // two slots ahead
    load(i0, nx[0]);
    load(i0 + 1, nx[1]);
    rope_angles(a, t, lane, cs);
    float2 c[4], s[4], gg[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = cs[ln.turns ? 8 * (lane % LH) + 2 * e : 0], w = cs[ln.turns ? 8 * (lane % LH) + 2 * e + 1 : 0];
      c[e] = ln.turns ? make_float2(v.x, w.x) : make_float2(1.f, 1.f);
      s[e] = ln.turns ? make_float2(v.y, w.y) : make_float2(0.f, 0.f);
    }
    if (kNorm) {
      rope_unpack(i0 < sl.nq ? g[0][0] : g[1][0], gg);
      rope_unpack(i0 < sl.nq ? g[0][1] : g[1][1], gg + 4);
    }
    auto slot = [&](int i, uint4 (&u)[2]) {
      float2 x[8];
      rope_unpack(u[0], x);
      rope_unpack(u[1], x + 4);
      load(i + 2, u);
      const bool q = i < sl.nq;
      const int h = (q ? i : i - sl.nq) * HI + sub;
      if (kNorm) {
        if (i == sl.nq) {
          rope_unpack(g[1][0], gg);
          rope_unpack(g[1][1], gg + 4);
        }
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fma2(x[e], x[e], ss);
        const float r = rsqrtf(fmaf(rope_sum<LH>(ss.x + ss.y), inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = mul2(mul2(x[e], make_float2(r, r)), gg[e]);
      }
      if (ln.turns) rope_turn(x, x + 4, c, s);
      if (ln.active && h < (q ? a.Hq : a.Hkv)) {
        uint16_t* o = (q ? a.oq + t * a.oq_ld : a.ok + t * a.ok_ld) + static_cast<int64_t>(h) * a.D;
        *reinterpret_cast<uint4*>(o + ln.c0) = rope_pack(x);
        *reinterpret_cast<uint4*>(o + ln.c1) = rope_pack(x + 4);
      }
    };
    for (int i = i0; i < i1; i += 2) {
      slot(i, nx[0]);
      if (i + 1 < i1) slot(i + 1, nx[1]);
    }
  }
}

// Gradient.  Each lane adds up the gain gradients of its 16 elements over all its items (fp32, a few
// hundred terms); the block joins its warps in order and writes one partial, and k_qk_gain adds the
// partials in block order: no atomics, the same bits for the same call.
template <int LH, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, 2) k_qk_rope_bwd(const RopeArgs a) {
  __shared__ float2 cs_all[kRopeWarps][kRopeMaxD / 2];
  __shared__ float sums[kNorm ? kRopeWarps : 1][2][kRopeMaxD];
  constexpr int HI = 32 / LH;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2* cs = cs_all[warp];
  const RopeLane ln = rope_lane(a, lane % LH);
  const int sub = lane / LH;
  const RopeSlots sl = rope_slots<LH>(a);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  uint4 g[2][2] = {};
  if (kNorm && ln.active) {
    g[0][0] = *reinterpret_cast<const uint4*>(a.gq + ln.c0);
    g[0][1] = *reinterpret_cast<const uint4*>(a.gq + ln.c1);
    g[1][0] = *reinterpret_cast<const uint4*>(a.gk + ln.c0);
    g[1][1] = *reinterpret_cast<const uint4*>(a.gk + ln.c1);
  }
  float acc[2][16] = {};
  const int64_t items = a.T * a.nsb;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kRopeWarps;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; it < items; it += nw) {
    const int64_t t = it / a.nsb;
    const int i0 = static_cast<int>(it - t * a.nsb) * a.sb;
    const int i1 = i0 + a.sb < sl.n ? i0 + a.sb : sl.n;
    float c[8], s[8];
    // the heads of one of the two tensors in [lo, hi)
    auto heads = [&](int lo, int hi, const uint16_t* xs, const uint16_t* dzs, uint16_t* os, const uint4 (&gg)[2],
                     float (&ac)[16], bool first) {
      uint4 nx[2] = {}, nz[2] = {};
      auto load = [&](int h) {
        nx[0] = nx[1] = nz[0] = nz[1] = make_uint4(0u, 0u, 0u, 0u);
        if (ln.active && h < hi) {
          const int64_t at = static_cast<int64_t>(h) * a.D;
          nz[0] = rope_ld(dzs + at + ln.c0);
          nz[1] = rope_ld(dzs + at + ln.c1);
          if (kNorm) {
            nx[0] = rope_ld(xs + at + ln.c0);
            nx[1] = rope_ld(xs + at + ln.c1);
          }
        }
      };
      load(lo + sub);
      if (first) {
        rope_angles(a, t, lane, cs);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = ln.turns ? cs[8 * (lane % LH) + e] : make_float2(1.f, 0.f);
          c[e] = v.x;
          s[e] = v.y;
        }
      }
      for (int hh = lo; hh < hi; hh += HI) {
        const int h = hh + sub;
        float x0[8], x1[8], d0[8], d1[8];
        rope_unpack8(nz[0], d0);
        rope_unpack8(nz[1], d1);
        rope_unpack8(nx[0], x0);
        rope_unpack8(nx[1], x1);
        load(h + HI);
        if (ln.turns) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y0 = d0[e], y1 = d1[e];
            d0[e] = fmaf(y0, c[e], y1 * s[e]);
            d1[e] = fmaf(y1, c[e], -(y0 * s[e]));
          }
        }
        if (kNorm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x0[e], x0[e], ss);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x1[e], x1[e], ss);
          ss = rope_sum<LH>(ss);
          const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
          float g0[8], g1[8];
          rope_unpack8(gg[0], g0);
          rope_unpack8(gg[1], g1);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x0[e] *= r;  // n
            x1[e] *= r;
            ac[e] = fmaf(d0[e], x0[e], ac[e]);
            ac[8 + e] = fmaf(d1[e], x1[e], ac[8 + e]);
            d0[e] *= g0[e];
            d1[e] *= g1[e];
            dot = fmaf(d0[e], x0[e], dot);
            dot = fmaf(d1[e], x1[e], dot);
          }
          dot = rope_sum<LH>(dot) * inv_d;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            d0[e] = r * fmaf(-x0[e], dot, d0[e]);
            d1[e] = r * fmaf(-x1[e], dot, d1[e]);
          }
        }
        if (ln.active && h < hi) {
          uint16_t* o = os + static_cast<int64_t>(h) * a.D;
          *reinterpret_cast<uint4*>(o + ln.c0) = rope_pack8(d0);
          *reinterpret_cast<uint4*>(o + ln.c1) = rope_pack8(d1);
        }
      }
    };
    const bool any_q = i0 < sl.nq;
    if (any_q)
      heads(i0 * HI, i1 * HI < a.Hq ? i1 * HI : a.Hq, kNorm ? a.q + t * a.q_ld : nullptr, a.dzq + t * a.dzq_ld,
            a.oq + t * a.oq_ld, g[0], acc[0], true);
    if (i1 > sl.nq) {
      const int from = any_q ? 0 : (i0 - sl.nq) * HI, to = (i1 - sl.nq) * HI;
      heads(from, to < a.Hkv ? to : a.Hkv, kNorm ? a.k + t * a.k_ld : nullptr, a.dzk + t * a.dzk_ld,
            a.ok + t * a.ok_ld, g[1], acc[1], !any_q);
    }
  }
  if (!kNorm) return;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = acc[w][e];
#pragma unroll
      for (int o = LH; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0 && ln.active) sums[warp][w][(e < 8 ? ln.c0 : ln.c1 - 8) + e] = v;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += kRopeThreads) {
    const int w = i / a.D, j = i - w * a.D;
    float v = 0.f;
#pragma unroll
    for (int x = 0; x < kRopeWarps; ++x) v += sums[x][w][j];
    a.parts[static_cast<int64_t>(blockIdx.x) * 2 * a.D + i] = v;
  }
}

// dg[i] = sum of the blocks' partials, i < 2 D: 16 strands of blocks in order, joined in order.
constexpr int kGainStrands = 16;
__global__ void __launch_bounds__(32 * kGainStrands)
    k_qk_gain(const float* __restrict__ parts, int nblk, int D, float* __restrict__ dgq, float* __restrict__ dgk) {
  __shared__ float sm[kGainStrands][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + x;
  float v = 0.f;
  if (i < 2 * D)
    for (int b = y; b < nblk; b += kGainStrands) v += parts[static_cast<int64_t>(b) * 2 * D + i];
  sm[y][x] = v;
  __syncthreads();
  if (y == 0 && i < 2 * D) {
#pragma unroll
    for (int s = 1; s < kGainStrands; ++s) v += sm[s][x];
    if (i < D)
      dgq[i] = v;
    else
      dgk[i - D] = v;
  }
}

}  // namespace bi
