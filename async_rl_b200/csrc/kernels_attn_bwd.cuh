// kernels_attn_bwd.cuh -- the gradient of softmax attention (kernels_attn.cuh has the forward).
//
// Mathematics.  With p_ij = exp(scale q_i . k_j - lse_i) on the visible pairs and the row's number
// delta_i = do_i . out_i:
//   dv_j = sum_i p_ij do_i,   ds_ij = p_ij (do_i . v_j - delta_i),
//   dk_j = scale sum_i ds_ij q_i,   dq_i = scale sum_j ds_ij k_j.
// p is recomputed from lse, so nothing of size queries x keys is ever stored.
//
// Two kernels.  k_attn_dkv holds 128 keys of one key/value head and runs over the query tiles that
// see them (4 products a tile pair); k_attn_dq holds 128 query rows and runs over the key tiles that
// they see (3 products).  One kernel for all three gradients needs 5 products, not 7, but has to add
// dQ up over CTAs: with atomics the order, and so the bits, would change from run to run, and 64 KB
// of fp32 additions a tile pair would go to L2.  Here every sum has a fixed order that depends on the
// places in the sequence only, so a sequence's gradients have the same bits in any batch.
//
// Both are bound by the tensor cores, with the exponentials (16 a clock and SM) next: 2048 and 1536
// clocks of products (D = 128) against 1024 of exponentials a pair of tiles.  Measured: a pair of tiles takes
// dK, dV 2700 clocks and dQ 1750; 64 packed causal sequences of 256..2048, 12/2 heads of 128: 591 and 514 us, with the
// plan's 22 and the rows' numbers' 100 in front of them (a call among others takes 1409); three of 4K..8K, 16/8 heads of
// 64: 676 and 474 us, 11 and 29 (1303).
//
// Rows behave as in the forward: a tile of 128 rows is floor(128 / G) tokens times the G heads that
// share a key/value head, so the gradients of shared heads are added up in the accumulators.
#pragma once

#include "kernels_attn.cuh"

namespace bi {

struct AttnBwdArgs {
  const AttnSeq* seqs;         // of this kernel's plan
  const AttnUnit* units;
  const AttnPlanHead* head;
  const AttnSeq* rows;         // of the dQ plan: unit0 counts its row tiles
  float* st;                   // [Hkv][tiles][2][128]: -lse log2(e) and -delta of each row of a tile
  int64_t tiles;
  const uint16_t *out, *dout;  // k_attn_pre
  const float* lse;
  int64_t do_ld, Tq;
  uint16_t *o0, *o1;           // dK and dV, or dQ
  int64_t ld0, ld1;
  int32_t Hq, Hkv, G, tpt;
  int32_t causal;
  float c;                     // scale log2(e)
  float scale;
  bool wide;                   // rows of the outputs start at 32-byte boundaries
  int32_t* status;
  uint64_t limit_ns;
};

// ----------------------------------------------------------------------------------------------
// rows' numbers
// ----------------------------------------------------------------------------------------------
// Bound by HBM (4 bytes an element of out).  A row of D values takes D / 8 lanes.  Rows of the tile
// that hold no query get -lse = -inf, which makes every p of theirs 0.
constexpr int kAtPreThreads = 256;
template <int D>
__global__ void __launch_bounds__(kAtPreThreads) k_attn_pre(const AttnBwdArgs a) {
  constexpr int L = D / 8;                    // lanes of a row
  constexpr int R = kAtPreThreads / L;        // rows at a time
  const int sub = threadIdx.x / L, lane = threadIdx.x % L;
  const int64_t n = static_cast<int64_t>(a.head->nunits) * a.Hkv;
  for (int64_t u = blockIdx.x; u < n; u += gridDim.x) {
    const AttnUnit w = a.units[u / a.Hkv];
    const int32_t h = static_cast<int32_t>(u % a.Hkv);
    const AttnSeq q = a.seqs[w.seq];
    float* st = a.st + (h * a.tiles + q.unit0 + w.t0 / a.tpt) * (2 * kAtTile);
#pragma unroll
    for (int r0 = 0; r0 < kAtTile; r0 += R) {
      const int r = r0 + sub;
      const int tok_in = r / a.G, g = r - tok_in * a.G;
      const bool valid = tok_in < a.tpt && w.t0 + tok_in < q.lq;
      const int64_t t = q.q0 + w.t0 + tok_in;
      const int32_t head = h * a.G + g;
      float sum = 0.f;
      if (valid) {
        const uint4 x = *reinterpret_cast<const uint4*>(a.out + (t * a.Hq + head) * D + lane * 8);
        const uint4 y = *reinterpret_cast<const uint4*>(a.dout + t * a.do_ld + head * D + lane * 8);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), sum);
          sum = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), sum);
        }
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        const float lse = valid ? a.lse[static_cast<int64_t>(head) * a.Tq + t] : -INFINITY;
        st[r] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;  // a row that sees nothing has no p
        st[kAtTile + r] = -sum;
      }
    }
  }
}

// ----------------------------------------------------------------------------------------------
// shared by both kernels
// ----------------------------------------------------------------------------------------------
// Warps 0-15: p and ds; 16: TMA; 17: MMA; 18: ragged tiles.  Four warps of each quarter of the SM hide one
// another's latencies: with two of them, and 64 columns a thread, p took 1300 clocks a tile, not 900.
constexpr int kAtBwdThreads = 608;
constexpr int kAtBwdProbs = 16;
constexpr int kAtSlotsA = 3, kAtSlotsB = 2;

template <int D>
struct AtBwdTile {
  static constexpr int tile_bytes = kAtTile * D * 2;
  static constexpr int ring_a = 2 * tile_bytes;                        // behind the two held tiles
  static constexpr int ring_b = ring_a + kAtSlotsA * tile_bytes;
  static constexpr int smem = ring_b + kAtSlotsB * tile_bytes;
};
struct AtBwdShared {
  float st[2][2][kAtTile];
  uint64_t held_full[2], held_empty[2];
  uint64_t a_full[kAtSlotsA], a_empty[kAtSlotsA];
  uint64_t b_full[kAtSlotsB], b_empty[kAtSlotsB];
  uint64_t st_full[2], st_empty[2];
  uint64_t s_full[2], dp_full;
  uint64_t p_full[2], ds_full[2];  // halves of the columns (dQ: ds_full[0] for both)
  uint64_t acc_full, done;
  uint64_t z_ask[2], z_full[2];    // a unit's ragged last tile (A and B ring): loading; has its zeros
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
  volatile uint32_t begun;  // units that the loading thread has begun
};
constexpr int kAtBwdSharedBytes = static_cast<int>((sizeof(AtBwdShared) + 127) / 128 * 128);

// A ring's slot and its phase.
template <int N>
struct AtRing {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() { ring_advance(slot, phase, N); }
  __device__ __forceinline__ void skip(uint32_t n) {
    phase ^= ((slot + n) / N) & 1u;
    slot = (slot + n) % N;
  }
};

struct AtStep {
  bool first, last, ragged;  // first and last tile of its unit; that has rows to clear
};
template <class Unit>
struct AtBwdWalk : AtWalk<AttnBwdArgs, Unit> {
  using AtWalk<AttnBwdArgs, Unit>::AtWalk;
  __device__ __forceinline__ bool step(AtStep& s) {
    if (!AtWalk<AttnBwdArgs, Unit>::step()) return false;
    s.first = this->i == 1;
    s.last = this->i == this->n;
    s.ragged = s.last && this->x.ragged;
    return true;
  }
};

// Warp roles' common start and end; returns the base of tensor memory.
__device__ __forceinline__ uint32_t at_bwd_begin(AtBwdShared& sh) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < kAtSlotsA; ++i) {
      mbar_init(&sh.a_full[i], 1);
      mbar_init(&sh.a_empty[i], 1);
    }
    for (int i = 0; i < kAtSlotsB; ++i) {
      mbar_init(&sh.b_full[i], 1);
      mbar_init(&sh.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.st_full[i], 1);
      mbar_init(&sh.held_full[i], 1);
      mbar_init(&sh.held_empty[i], 1);
      mbar_init(&sh.z_ask[i], 1);
      mbar_init(&sh.z_full[i], 1);
      mbar_init(&sh.st_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 32 * kAtBwdProbs);
      mbar_init(&sh.ds_full[i], 32 * kAtBwdProbs);
    }
    mbar_init(&sh.dp_full, 1);
    mbar_init(&sh.acc_full, 1);
    mbar_init(&sh.done, 1);
    sh.abort_flag = 0u;
    sh.begun = 0u;
    fence_mbar_init_cluster();
  }
  if (threadIdx.x / 32 == kAtBwdProbs + 1) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return sh.tmem_base;
}
__device__ __forceinline__ void at_bwd_end(AtBwdShared& sh, uint32_t tmem) {
  tc_fence_before();
  __syncthreads();
  if (sh.abort_flag != 0u) {  // on the error path a copy or a commit may still be in flight
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000u) {
    }
  }
  if (threadIdx.x / 32 == kAtBwdProbs + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// D[128 x 128] = A[128 x Dh] B[128 x Dh]^T, both K-major tiles in shared memory (one thread).
template <int D>
__device__ __forceinline__ void at_mma_ss(uint32_t d, uint64_t da, uint64_t db) {
  constexpr uint32_t idesc = idesc_bf16(128, 128, false, false);
  constexpr uint64_t blk = kAUnitBytes >> 4;
#pragma unroll
  for (int b = 0; b < D / 64; ++b)
#pragma unroll
    for (int k = 0; k < 4; ++k) umma_bf16(d, da + b * blk + 2 * k, db + b * blk + 2 * k, idesc, (b | k) ? 1u : 0u);
}
// Half of D[128 x Dh] += A[128 x 128] B[128 x Dh]: A in tensor memory as at_put leaves it, B a tile
// read along its rows (one thread).
template <int D>
__device__ __forceinline__ void at_mma_ts(uint32_t d, uint32_t a, uint64_t db, int half, bool first) {
  constexpr uint32_t idesc = idesc_bf16(128, D, false, true);
#pragma unroll
  for (int k = 4 * half; k < 4 * half + 4; ++k)
    umma_bf16_ta(d, a + k * 16, db + k * (2048 >> 4), idesc, (k > 0 || !first) ? 1u : 0u);
}

// A thread's columns of a 128-column tile: 16 of each half, [half * 64 + X * 16, +16), X its group of four
// warps.  Its bf16 results go into the first 8 of the 16 columns that it read.
__device__ __forceinline__ void at_get(uint32_t t, uint32_t (&s)[2][16]) {
  tmem_ld16(t, s[0]);
  tmem_ld16(t + 64, s[1]);
  tmem_ld_wait();
  tmem_ld_pin16(s[0]);
  tmem_ld_pin16(s[1]);
}
__device__ __forceinline__ void at_put(uint32_t t, const float2 (&p)[8]) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(p[e].x, p[e].y);  // bf16: what the tensor cores take
  tmem_st8(t, w);
}
// 16 columns of an accumulator, scaled, as bf16 (whole warp; stored where `valid`).
__device__ __forceinline__ void at_store16(uint32_t t, float scale, uint16_t* o, bool valid, bool wide) {
  uint32_t s[16], w[8];
  tmem_ld16(t, s);
  tmem_ld_wait();
  tmem_ld_pin16(s);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = pack_bf16x2(__uint_as_float(s[2 * e]) * scale, __uint_as_float(s[2 * e + 1]) * scale);
  if (valid) at_store32b(o, w, wide);
}
__device__ __forceinline__ void at_zero16(uint16_t* o) {
#pragma unroll
  for (int e = 0; e < 2; ++e) reinterpret_cast<uint4*>(o)[e] = make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ float2 at_pair(const uint32_t (&s)[16], int e) {
  return make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
}

// ----------------------------------------------------------------------------------------------
// dK, dV: keys are the lanes, query rows the columns
// ----------------------------------------------------------------------------------------------
// Tensor memory: S^T, dP^T, dV, dK.  P^T and dS^T replace the scores that they come from and are the
// A operands of dV and dK.  The issue order makes two phases: while the tensor cores work on
// dV += P_i dO_i and S_{i+1}, ds_i is computed; while they work on dK += dS_i Q_i and dP_{i+1},
// p_{i+1} is.
struct AtKvUnit {
  AttnSeq q;
  int32_t h, t0;
  int32_t i0, i1;   // query tiles that see a key of the unit
  int64_t tile0;    // of the sequence's first query tile
  int32_t rows;     // of the last query tile
  bool ragged;
  __device__ __forceinline__ int32_t tiles() const { return i1 - i0; }
  __device__ __forceinline__ void fetch(const AttnBwdArgs& a, int64_t u) {
    const AttnUnit w = a.units[u / a.Hkv];
    h = static_cast<int32_t>(u % a.Hkv);
    q = a.seqs[w.seq];
    t0 = w.t0;
    const int32_t first = attn_first_query(t0, q.lq, q.lk, a.causal);
    i1 = (q.lq + a.tpt - 1) / a.tpt;
    i0 = first >= q.lq ? i1 : first / a.tpt;
    tile0 = a.rows[w.seq].unit0;
    rows = (q.lq - (i1 - 1) * a.tpt) * a.G;
    ragged = rows < a.tpt * a.G;
  }
};

template <int D>
__device__ __forceinline__ void at_dkv_load(AtBwdShared& sh, const AttnBwdArgs& a, uint32_t smem, int64_t nu,
                                            const CUtensorMap* mq, const CUtensorMap* mk, const CUtensorMap* mv,
                                            const CUtensorMap* mdo) {
  using T = AtBwdTile<D>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  tma_prefetch_desc(mq);
  tma_prefetch_desc(mk);
  tma_prefetch_desc(mv);
  tma_prefetch_desc(mdo);
  const uint32_t bytes = static_cast<uint32_t>(a.tpt * a.G) * 128u * (D / 64);
  AtRing<kAtSlotsA> ra;
  AtRing<kAtSlotsB> rb;
  AtRing<2> rs;
  uint32_t hph = 0, begun = 0;
  AtBwdWalk<AtKvUnit> walk(a, nu);
  AtStep f;
  auto held = [&](int w, const CUtensorMap* m) {
    if (!mbar_wait<false>(&sh.held_empty[w], hph ^ 1u, wc)) return false;
    mbar_arrive_expect_tx(&sh.held_full[w], T::tile_bytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_3d(smem + w * T::tile_bytes + b * kAUnitBytes, m, &sh.held_full[w], b * 64, walk.x.h,
                  static_cast<int32_t>(walk.x.q.k0) + walk.x.t0);
    return true;
  };
  while (walk.step(f)) {
    const AtKvUnit& x = walk.x;
    const int32_t i = x.i0 + walk.i - 1;
    const int32_t row = static_cast<int32_t>(x.q.q0) + i * a.tpt;
    if (f.first) sh.begun = ++begun;
    if (f.first && !held(0, mk)) return;
    if (!mbar_wait<false>(&sh.a_empty[ra.slot], ra.phase ^ 1u, wc)) return;
    mbar_arrive_expect_tx(&sh.a_full[ra.slot], bytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_3d(smem + T::ring_a + ra.slot * T::tile_bytes + b * kAUnitBytes, mq, &sh.a_full[ra.slot], b * 64,
                  x.h * a.G, row);
    ra.next();
    if (f.ragged) mbar_arrive(&sh.z_ask[0]);
    if (!mbar_wait<false>(&sh.st_empty[rs.slot], rs.phase ^ 1u, wc)) return;
    mbar_arrive_expect_tx(&sh.st_full[rs.slot], 2 * kAtTile * 4);
    bulk_load(smem_u32(&sh.st[rs.slot][0][0]), a.st + (x.h * a.tiles + x.tile0 + i) * (2 * kAtTile), 2 * kAtTile * 4,
              &sh.st_full[rs.slot]);
    rs.next();
    if (f.first) {
      if (!held(1, mv)) return;
      hph ^= 1u;
    }
    if (!mbar_wait<false>(&sh.b_empty[rb.slot], rb.phase ^ 1u, wc)) return;
    mbar_arrive_expect_tx(&sh.b_full[rb.slot], bytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_3d(smem + T::ring_b + rb.slot * T::tile_bytes + b * kAUnitBytes, mdo, &sh.b_full[rb.slot], b * 64,
                  x.h * a.G, row);
    rb.next();
    if (f.ragged) mbar_arrive(&sh.z_ask[1]);
  }
}

template <int D>
__device__ __forceinline__ void at_dkv_mma(AtBwdShared& sh, const AttnBwdArgs& a, uint32_t smem, int64_t nu,
                                           uint32_t tmem) {
  using T = AtBwdTile<D>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  constexpr uint32_t ts = T::tile_bytes >> 4;
  const uint64_t dk = sdesc_k_sw128(smem), dv = sdesc_k_sw128(smem + T::tile_bytes);
  const uint64_t dq_k = sdesc_k_sw128(smem + T::ring_a), dq_mn = sdesc_mn_sw128(smem + T::ring_a, kAUnitBytes);
  const uint64_t do_k = sdesc_k_sw128(smem + T::ring_b), do_mn = sdesc_mn_sw128(smem + T::ring_b, kAUnitBytes);
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + D;
  AtRing<kAtSlotsA> ra, ra2;  // next tile to arrive, tile whose dK is next
  AtRing<kAtSlotsB> rb, rb2;
  AtRing<2> rs;
  uint32_t hph[2] = {0, 0}, zph[2] = {0, 0}, ph = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait<false>(bar, parity, wc);
    tc_fence_after();
    return ok;
  };
  // a new unit's held tile, and the zeros of a ragged one
  auto ready = [&](int w, const AtStep& f) {
    if (f.first) {
      if (!wait(&sh.held_full[w], hph[w])) return false;
      hph[w] ^= 1u;
    }
    if (f.ragged) {
      if (!wait(&sh.z_full[w], zph[w])) return false;
      zph[w] ^= 1u;
    }
    return true;
  };
  auto scores = [&](const AtStep& f) {
    if (!wait(&sh.a_full[ra.slot], ra.phase) || !ready(0, f)) return false;
    at_mma_ss<D>(t_s, dk, dq_k + ra.slot * ts);
    umma_commit(&sh.s_full[0]);
    if (f.last) umma_commit(&sh.held_empty[0]);
    ra.next();
    return true;
  };
  auto dprobs = [&](const AtStep& f) {
    if (!wait(&sh.b_full[rb.slot], rb.phase) || !ready(1, f)) return false;
    at_mma_ss<D>(t_dp, dv, do_k + rb.slot * ts);
    umma_commit(&sh.dp_full);
    if (f.last) umma_commit(&sh.held_empty[1]);
    rb.next();
    return true;
  };
  AtBwdWalk<AtKvUnit> walk(a, nu);
  AtStep f, fn;
  bool go = walk.step(f) && scores(f) && dprobs(f);
  while (go) {
    const bool next = walk.step(fn);
#pragma unroll
    for (int half = 0; half < 2 && go; ++half) {
      go = wait(&sh.p_full[half], ph);
      if (go) at_mma_ts<D>(t_dv, t_s, do_mn + rb2.slot * ts, half, f.first);
    }
    if (!go || (next && !scores(fn))) break;
    umma_commit(&sh.b_empty[rb2.slot]);
    rb2.next();
#pragma unroll
    for (int half = 0; half < 2 && go; ++half) {
      go = wait(&sh.ds_full[half], ph);
      if (go) at_mma_ts<D>(t_dk, t_dp, dq_mn + ra2.slot * ts, half, f.first);
    }
    if (!go) break;
    umma_commit(&sh.a_empty[ra2.slot]);
    umma_commit(&sh.st_empty[rs.slot]);
    if (f.last) umma_commit(&sh.acc_full);
    ra2.next();
    rs.next();
    ph ^= 1u;
    go = next && dprobs(fn);
    f = fn;
  }
  umma_commit(&sh.done);
  mbar_wait<false>(&sh.done, 0u, wc);
}

// Rows behind the sequence's last query may be another sequence's, or hold anything: zeros, before the
// products see them.  The loading thread asks for it with the tile's load; it is never two units ahead,
// because a unit's held tiles wait for the products with the last tiles of the unit before.
template <int D>
__device__ __forceinline__ void at_dkv_ragged(AtBwdShared& sh, const AttnBwdArgs& a, uint8_t* smem_p, int64_t nu) {
  using T = AtBwdTile<D>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  AtRing<kAtSlotsA> ra;
  AtRing<kAtSlotsB> rb;
  uint32_t ph = 0;
  for (int64_t r = 0, u; (u = at_turn(r)) < nu; ++r) {
    AtKvUnit x;
    x.fetch(a, u);
    if (x.i0 >= x.i1) continue;
    ra.skip(x.i1 - 1 - x.i0);
    rb.skip(x.i1 - 1 - x.i0);
    if (x.ragged) {
      if (!at_wait_behind(&sh.z_ask[0], ph, wc, &sh.begun) || !at_wait(&sh.a_full[ra.slot], ra.phase, wc)) return;
      at_zero_rows<D>(smem_p + T::ring_a + ra.slot * T::tile_bytes, x.rows);
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.z_full[0]);
      if (!at_wait(&sh.z_ask[1], ph, wc) || !at_wait(&sh.b_full[rb.slot], rb.phase, wc)) return;
      at_zero_rows<D>(smem_p + T::ring_b + rb.slot * T::tile_bytes, x.rows);
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.z_full[1]);
      ph ^= 1u;
    }
    ra.next();
    rb.next();
  }
}

template <int D>
__device__ __forceinline__ void at_dkv_probs(AtBwdShared& sh, const AttnBwdArgs& a, int64_t nu, uint32_t tmem) {
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int X = warp >> 2, key_in = (warp & 3) * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_s = tmem + lanes + X * 16, t_dp = t_s + 128;
  const int part = (X & 1) * (D / 2);  // groups 0 and 1 store a half of dK each, 2 and 3 of dV
  const uint32_t t_acc = tmem + lanes + 256 + (X < 2 ? D : 0) + part;
  uint32_t ph = 0, aph = 0;
  AtRing<2> rs;
  const float2 cc = make_float2(a.c, a.c);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return at_wait(bar, parity, wc); };
  // A unit's sums are stored when the next unit's first p is computed: its scores are there by then.
  uint16_t* done_o = nullptr;
  bool done_valid = false, pending = false;
  auto store = [&]() {
    if (!wait(&sh.acc_full, aph)) return false;
    aph ^= 1u;
#pragma unroll 1
    for (int b = 0; b < D / 32; ++b) at_store16(t_acc + b * 16, X < 2 ? a.scale : 1.f, done_o + b * 16, done_valid, a.wide);
    pending = false;
    return true;
  };
  for (int64_t r = 0, u; (u = at_turn(r)) < nu; ++r) {
    AtKvUnit x;
    x.fetch(a, u);
    const int32_t key = x.t0 + key_in;
    const bool valid = key < x.q.lk;
    uint16_t* o = (X < 2 ? a.o0 + (x.q.k0 + key) * a.ld0 : a.o1 + (x.q.k0 + key) * a.ld1) + x.h * D + part;
    if (x.i0 >= x.i1) {  // no query sees these keys
      if (valid)
#pragma unroll
        for (int b = 0; b < D / 32; ++b) at_zero16(o + b * 16);
      continue;
    }
    // this key's first query
    const int32_t from = a.causal ? key - (x.q.lk - x.q.lq) : 0;
    for (int32_t i = x.i0; i < x.i1; ++i) {
      // columns below `low` do not see this key
      const int64_t lw = (static_cast<int64_t>(from) - static_cast<int64_t>(i) * a.tpt) * a.G;
      const int low = lw > kAtTile ? kAtTile : static_cast<int>(lw < 0 ? 0 : lw);
      const bool masked = __any_sync(0xffffffffu, low > 0);
      if (!wait(&sh.st_full[rs.slot], rs.phase)) return;
      if (!wait(&sh.s_full[0], ph)) return;
      const float4* nl = reinterpret_cast<const float4*>(&sh.st[rs.slot][0][X * 16]);
      const float4* nd = reinterpret_cast<const float4*>(&sh.st[rs.slot][1][X * 16]);
      uint32_t s[2][16];
      float2 p[2][8];
      at_get(t_s, s);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (masked) {
          at_rare();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (half * 64 + X * 16 + e < low) s[half][e] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 l = nl[half * 16 + e / 2];
          const float2 y0 = fma2(at_pair(s[half], e), cc, make_float2(l.x, l.y));
          const float2 y1 = fma2(at_pair(s[half], e + 1), cc, make_float2(l.z, l.w));
          p[half][e] = at_ex2(e, y0);
          p[half][e + 1] = at_ex2(e + 1, y1);
        }
        if (pending && !store()) return;
        at_put(t_s + half * 64, p[half]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sh.p_full[half]);
      }
      if (!wait(&sh.dp_full, ph)) return;
      at_get(t_dp, s);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (masked) {
          at_rare();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (half * 64 + X * 16 + e < low) s[half][e] = 0u;  // p is 0 there; what v holds does not matter
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 d = nd[half * 16 + e / 2];
          p[half][e] = mul2(p[half][e], add2(at_pair(s[half], e), make_float2(d.x, d.y)));
          p[half][e + 1] = mul2(p[half][e + 1], add2(at_pair(s[half], e + 1), make_float2(d.z, d.w)));
        }
        at_put(t_dp + half * 64, p[half]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sh.ds_full[half]);
      }
      rs.next();
      ph ^= 1u;
    }
    pending = true;
    done_o = o;
    done_valid = valid;
  }
  if (pending) store();
}

// Rows [tpt G, 128) of every query tile are never loaded: zeros from the start.
template <int D>
__device__ __forceinline__ void at_zero_tails(uint8_t* ring, int slots, int rows) {
  for (int i = threadIdx.x; i < slots * (D / 64) * (kAtTile - rows) * 8; i += kAtBwdThreads) {
    const int v = i & 7, rest = i >> 3;
    const int r = rows + rest % (kAtTile - rows), blk = rest / (kAtTile - rows);
    *reinterpret_cast<uint4*>(ring + blk * kAUnitBytes + r * 128 + v * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D>
__global__ void __launch_bounds__(kAtBwdThreads, 1)
    k_attn_dkv(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, const AttnBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  AtBwdShared& sh = *reinterpret_cast<AtBwdShared*>(dsmem + AtBwdTile<D>::smem);
  const uint32_t smem = smem_u32(dsmem);
  at_zero_tails<D>(dsmem + AtBwdTile<D>::ring_a, kAtSlotsA + kAtSlotsB, a.tpt * a.G);
  fence_proxy_async_shared();
  const uint32_t tmem = at_bwd_begin(sh);
  const bool misaligned = (smem & 1023u) != 0;
  if (misaligned && threadIdx.x == 0) raise_status(a.status, 4 /* BI_ERR_CUDA */);
  const int64_t nu = misaligned ? 0 : static_cast<int64_t>(a.head->nunits) * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < kAtBwdProbs) {
    at_dkv_probs<D>(sh, a, nu, tmem);
  } else if (warp == kAtBwdProbs) {
    if (lane == 0) at_dkv_load<D>(sh, a, smem, nu, &mq, &mk, &mv, &mdo);
    __syncwarp();
  } else if (warp == kAtBwdProbs + 1) {
    if (elect_one()) at_dkv_mma<D>(sh, a, smem, nu, tmem);
    __syncwarp();
  } else {
    at_dkv_ragged<D>(sh, a, dsmem, nu);
  }
  at_bwd_end(sh, tmem);
}

// ----------------------------------------------------------------------------------------------
// dQ: query rows are the lanes, keys the columns
// ----------------------------------------------------------------------------------------------
// Tensor memory: S twice, dP, dQ.  dS replaces the scores and is the A operand of dQ.  S runs two
// tiles ahead, so the exponentials of a tile never wait for its products.
struct AtQUnit {
  AttnSeq q;
  int32_t h, t0;
  int32_t n;        // key tiles that a row of the unit sees
  int32_t rows;     // keys of the last one
  bool ragged;
  __device__ __forceinline__ int32_t tiles() const { return n; }
  __device__ __forceinline__ void fetch(const AttnBwdArgs& a, int64_t u) {
    const AttnUnit w = a.units[u / a.Hkv];
    h = static_cast<int32_t>(u % a.Hkv);
    q = a.seqs[w.seq];
    t0 = w.t0;
    const int32_t last = (t0 + a.tpt < q.lq ? t0 + a.tpt : q.lq) - 1;
    n = (attn_visible(last, q.lq, q.lk, a.causal) + kAtTile - 1) / kAtTile;
    rows = q.lk - (n - 1) * kAtTile;
    ragged = rows < kAtTile;
  }
};

template <int D>
__device__ __forceinline__ void at_dq_load(AtBwdShared& sh, const AttnBwdArgs& a, uint32_t smem, int64_t nu,
                                           const CUtensorMap* mq, const CUtensorMap* mk, const CUtensorMap* mv,
                                           const CUtensorMap* mdo) {
  using T = AtBwdTile<D>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  tma_prefetch_desc(mq);
  tma_prefetch_desc(mk);
  tma_prefetch_desc(mv);
  tma_prefetch_desc(mdo);
  const uint32_t bytes = static_cast<uint32_t>(a.tpt * a.G) * 128u * (D / 64);
  AtRing<kAtSlotsA> ra;
  AtRing<kAtSlotsB> rb;
  uint32_t hph = 0, begun = 0;
  AtBwdWalk<AtQUnit> walk(a, nu);
  AtStep f;
  auto held = [&](int w, const CUtensorMap* m) {
    if (!mbar_wait<false>(&sh.held_empty[w], hph ^ 1u, wc)) return false;
    mbar_arrive_expect_tx(&sh.held_full[w], bytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_3d(smem + w * T::tile_bytes + b * kAUnitBytes, m, &sh.held_full[w], b * 64, walk.x.h * a.G,
                  static_cast<int32_t>(walk.x.q.q0) + walk.x.t0);
    return true;
  };
  while (walk.step(f)) {
    const AtQUnit& x = walk.x;
    const int32_t key = static_cast<int32_t>(x.q.k0) + (walk.i - 1) * kAtTile;
    if (f.first) sh.begun = ++begun;
    if (f.first && !held(0, mq)) return;
    if (!mbar_wait<false>(&sh.a_empty[ra.slot], ra.phase ^ 1u, wc)) return;
    mbar_arrive_expect_tx(&sh.a_full[ra.slot], T::tile_bytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_3d(smem + T::ring_a + ra.slot * T::tile_bytes + b * kAUnitBytes, mk, &sh.a_full[ra.slot], b * 64, x.h, key);
    ra.next();
    if (f.ragged) mbar_arrive(&sh.z_ask[0]);
    if (f.first) {
      if (!held(1, mdo)) return;
      hph ^= 1u;
    }
    if (!mbar_wait<false>(&sh.b_empty[rb.slot], rb.phase ^ 1u, wc)) return;
    mbar_arrive_expect_tx(&sh.b_full[rb.slot], T::tile_bytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_3d(smem + T::ring_b + rb.slot * T::tile_bytes + b * kAUnitBytes, mv, &sh.b_full[rb.slot], b * 64, x.h, key);
    rb.next();
  }
}

template <int D>
__device__ __forceinline__ void at_dq_mma(AtBwdShared& sh, const AttnBwdArgs& a, uint32_t smem, int64_t nu,
                                          uint32_t tmem) {
  using T = AtBwdTile<D>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  constexpr uint32_t ts = T::tile_bytes >> 4;
  const uint64_t dq = sdesc_k_sw128(smem), ddo = sdesc_k_sw128(smem + T::tile_bytes);
  const uint64_t dk_k = sdesc_k_sw128(smem + T::ring_a), dk_mn = sdesc_mn_sw128(smem + T::ring_a, kAUnitBytes);
  const uint64_t dv_k = sdesc_k_sw128(smem + T::ring_b);
  const uint32_t t_dp = tmem + 256, t_dq = tmem + 384;
  AtRing<kAtSlotsA> ra, ra2;
  AtRing<kAtSlotsB> rb;
  AtRing<2> sb;                // score buffer of the next S
  uint32_t hph[2] = {0, 0}, zph = 0, ph = 0, cur = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait<false>(bar, parity, wc);
    tc_fence_after();
    return ok;
  };
  auto held = [&](int w, const AtStep& f) {
    if (!f.first) return true;
    hph[w] ^= 1u;
    return wait(&sh.held_full[w], hph[w] ^ 1u);
  };
  auto scores = [&](const AtStep& f) {
    if (!wait(&sh.a_full[ra.slot], ra.phase) || !held(0, f)) return false;
    if (f.ragged) {
      if (!wait(&sh.z_full[0], zph)) return false;
      zph ^= 1u;
    }
    at_mma_ss<D>(tmem + sb.slot * 128, dq, dk_k + ra.slot * ts);
    umma_commit(&sh.s_full[sb.slot]);
    if (f.last) umma_commit(&sh.held_empty[0]);
    ra.next();
    sb.next();
    return true;
  };
  auto dprobs = [&](const AtStep& f) {
    if (!wait(&sh.b_full[rb.slot], rb.phase) || !held(1, f)) return false;
    at_mma_ss<D>(t_dp, ddo, dv_k + rb.slot * ts);
    umma_commit(&sh.dp_full);
    umma_commit(&sh.b_empty[rb.slot]);
    if (f.last) umma_commit(&sh.held_empty[1]);
    rb.next();
    return true;
  };
  AtBwdWalk<AtQUnit> walk(a, nu);
  AtStep f, f1, f2;
  bool go = walk.step(f) && scores(f) && dprobs(f);
  bool n1 = go && walk.step(f1);
  if (n1) go = scores(f1);
  while (go) {
    const bool n2 = n1 && walk.step(f2);
    // One barrier for the whole tile: the next dP lets the next dS come, so nothing of this one may
    // still be waited for behind it.
    if (!wait(&sh.ds_full[0], ph) || (n1 && !dprobs(f1))) break;
#pragma unroll
    for (int half = 0; half < 2; ++half) at_mma_ts<D>(t_dq, tmem + cur * 128, dk_mn + ra2.slot * ts, half, f.first);
    umma_commit(&sh.a_empty[ra2.slot]);
    if (f.last) umma_commit(&sh.acc_full);
    ra2.next();
    cur ^= 1u;
    ph ^= 1u;
    if (n2 && !scores(f2)) break;
    go = n1;
    f = f1;
    f1 = f2;
    n1 = n2;
  }
  umma_commit(&sh.done);
  mbar_wait<false>(&sh.done, 0u, wc);
}

// The same for the keys behind a sequence's last one.
template <int D>
__device__ __forceinline__ void at_dq_ragged(AtBwdShared& sh, const AttnBwdArgs& a, uint8_t* smem_p, int64_t nu) {
  using T = AtBwdTile<D>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  AtRing<kAtSlotsA> ra;
  uint32_t ph = 0;
  for (int64_t r = 0, u; (u = at_turn(r)) < nu; ++r) {
    AtQUnit x;
    x.fetch(a, u);
    if (x.n == 0) continue;
    ra.skip(x.n - 1);
    if (x.ragged) {
      if (!at_wait_behind(&sh.z_ask[0], ph, wc, &sh.begun) || !at_wait(&sh.a_full[ra.slot], ra.phase, wc)) return;
      at_zero_rows<D>(smem_p + T::ring_a + ra.slot * T::tile_bytes, x.rows);
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.z_full[0]);
      ph ^= 1u;
    }
    ra.next();
  }
}

template <int D>
__device__ __forceinline__ void at_dq_probs(AtBwdShared& sh, const AttnBwdArgs& a, int64_t nu, uint32_t tmem) {
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int X = warp >> 2, row = (warp & 3) * 32 + lane;
  const int tok_in = row / a.G, g = row - tok_in * a.G;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t t_s = tmem + lanes + X * 16, t_dp = t_s + 256;
  uint32_t ph = 0, aph = 0;
  AtRing<2> sb;
  const float2 cc = make_float2(a.c, a.c);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return at_wait(bar, parity, wc); };
  // A unit's sum is stored when the next unit's first p is computed: its scores are there by then.
  uint16_t* done_o = nullptr;
  bool done_valid = false, pending = false;
  auto store = [&]() {
    if (!wait(&sh.acc_full, aph)) return false;
    aph ^= 1u;
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      at_store16(tmem + lanes + 384 + X * (D / 4) + b * 16, a.scale, done_o + b * 16, done_valid, a.wide);
    pending = false;
    return true;
  };
  for (int64_t r = 0, u; (u = at_turn(r)) < nu; ++r) {
    AtQUnit x;
    x.fetch(a, u);
    const int32_t tok = x.t0 + tok_in;
    const bool valid = tok_in < a.tpt && tok < x.q.lq;
    // rows without a query see all, so that they do not make their warp mask every tile
    const int32_t vis = valid ? attn_visible(tok, x.q.lq, x.q.lk, a.causal) : 0x7fffffff;
    uint16_t* o = a.o0 + (x.q.q0 + tok) * a.ld0 + static_cast<int64_t>(x.h * a.G + g) * D + X * (D / 4);
    if (x.n == 0) {  // no key to see
      if (valid)
#pragma unroll
        for (int b = 0; b < D / 64; ++b) at_zero16(o + b * 16);
      continue;
    }
    const float* st = a.st + (x.h * a.tiles + x.q.unit0 + x.t0 / a.tpt) * (2 * kAtTile) + row;
    const float2 nl = make_float2(st[0], st[0]), nd = make_float2(st[kAtTile], st[kAtTile]);
    for (int32_t j = 0; j < x.n; ++j) {
      const int32_t lim = vis - j * kAtTile;  // columns from here on are not seen
      const bool masked = __any_sync(0xffffffffu, lim < kAtTile);
      if (!wait(&sh.s_full[sb.slot], sb.phase)) return;
      uint32_t s[2][16];
      float2 p[2][8];
      at_get(t_s + sb.slot * 128, s);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (masked) {
          at_rare();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (half * 64 + X * 16 + e >= lim) s[half][e] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[half][e] = at_ex2(e, fma2(at_pair(s[half], e), cc, nl));
        }
      }
      if (pending && !store()) return;
      if (!wait(&sh.dp_full, ph)) return;
      at_get(t_dp, s);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (masked) {
          at_rare();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (half * 64 + X * 16 + e >= lim) s[half][e] = 0u;  // what v holds there does not matter
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) p[half][e] = mul2(p[half][e], add2(at_pair(s[half], e), nd));
        at_put(t_s + sb.slot * 128 + half * 64, p[half]);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sh.ds_full[0]);
      sb.next();
      ph ^= 1u;
    }
    pending = true;
    done_o = o;
    done_valid = valid;
  }
  if (pending) store();
}

template <int D>
__global__ void __launch_bounds__(kAtBwdThreads, 1)
    k_attn_dq(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, const AttnBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  AtBwdShared& sh = *reinterpret_cast<AtBwdShared*>(dsmem + AtBwdTile<D>::smem);
  const uint32_t smem = smem_u32(dsmem);
  const uint32_t tmem = at_bwd_begin(sh);
  const bool misaligned = (smem & 1023u) != 0;
  if (misaligned && threadIdx.x == 0) raise_status(a.status, 4 /* BI_ERR_CUDA */);
  const int64_t nu = misaligned ? 0 : static_cast<int64_t>(a.head->nunits) * a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < kAtBwdProbs) {
    at_dq_probs<D>(sh, a, nu, tmem);
  } else if (warp == kAtBwdProbs) {
    if (lane == 0) at_dq_load<D>(sh, a, smem, nu, &mq, &mk, &mv, &mdo);
    __syncwarp();
  } else if (warp == kAtBwdProbs + 1) {
    if (elect_one()) at_dq_mma<D>(sh, a, smem, nu, tmem);
    __syncwarp();
  } else {
    at_dq_ragged<D>(sh, a, dsmem, nu);
  }
  at_bwd_end(sh, tmem);
}

}  // namespace bi
