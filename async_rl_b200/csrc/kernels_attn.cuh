// kernels_attn.cuh -- softmax attention over packed sequences or key/value caches: the work plan and
// the forward pass.
//
// Mathematics.  For a query row with scores s_j = q . k_j (j over its visible keys) and
// c = scale log2(e), one pass over the keys keeps a reference m and
//   l = sum_j 2^(c s_j - m),   O = sum_j 2^(c s_j - m) v_j,
// multiplying l and O by 2^(m - m') when the reference is raised to m'.  out = O / l and
// lse = (m + log2 l) ln 2.  The reference follows the running maximum lazily: it is raised only by a
// tile whose maximum is more than 8 above it (every term stays below 2^8), which after the first
// tile of a row is rare.
//
// Fixed chunks.  The keys of a sequence are cut into chunks of 2048, counted from its first key.  A
// chunk starts from m = -inf, and chunks are joined in order:
//   m' = max(m, m_c),  O' = O 2^(m - m') + O_c 2^(m_c - m'),  l' likewise.
// Tiles of 128 keys, chunks and the order of every sum depend on the key's place in its sequence
// only, so a row's output has the same bits in a prefill, in a decode step over a cache and in any
// batch; a long cache with few rows is worked on by many SMs, one chunk each, joined by a second
// kernel with the same expressions.
//
// Rows.  The G = Hq / Hkv query heads of one key/value head share its keys: a tile of 128 rows holds
// floor(128 / G) tokens times G heads, so a decode step fills its tile with the group's heads and
// every key tile is read once for all of them.
//
// What bounds it.  A key tile takes a row tile 1024 clocks of products and, with every exponential on the
// special function unit, as many of those.  Its scores, softmax, P and product follow one another, so two row
// tiles take turns: one's products beside the other's softmax.  Measured, this kernel alone with pauses between
// (calls back to back, with plan and joining and at the clock they settle at, in brackets): one causal 8K sequence,
// 32/8 heads of 128: 475 us (1.16 PFLOP/s); 16K: 1.84 ms (2.14); 64 packed sequences of 256..2048, 12/2 heads:
// 431 us (484); decode over 64 caches of up to 8K keys: 201 us (225), 5.7 TB/s, where HBM is the bound.  Without
// any softmax, the 8K case takes 358 us: the issuing thread and the barriers.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "kernels_lm.cuh"

namespace bi {

constexpr int kAtTile = 128;                          // rows and keys of a tile
constexpr int kAtChunkTiles = 16;
constexpr int kAtChunk = kAtTile * kAtChunkTiles;     // keys of a chunk

struct AttnSeq {
  int64_t q0, k0;    // first query and key row
  int64_t part0;     // first of its partial rows (tokens x chunks), split forward only
  int32_t lq, lk;    // queries and keys
  int32_t unit0;     // first of its units before splitting
  int32_t nch;       // chunks of its keys, at least 1
};
struct AttnUnit {
  int32_t seq;
  int32_t t0;        // first query (forward, dQ) or key (dK, dV) of the unit
  int32_t c0, c1;    // chunks [c0, c1) (forward)
};
struct AttnPlanHead {
  int32_t nunits;
  int32_t split;     // units are single chunks; rows of sequences with several are joined later
};

// ----------------------------------------------------------------------------------------------
// plan: check the offsets, cut the sequences into units and list them, longest first
// ----------------------------------------------------------------------------------------------
enum AttnPlanMode : int { kPlanFwd = 0, kPlanDq = 1, kPlanDkv = 2 };
struct AttnPlanArgs {
  const int64_t *qo, *ko;
  const int32_t* kl;       // or NULL
  int64_t Tq, Tk;
  int32_t S, mode, causal;
  int32_t step;            // queries (keys) of a unit
  int32_t tpt;             // tokens of a 128-row tile
  int32_t sms, Hkv;
  int32_t cap_units;
  int64_t cap_part;        // partial rows the workspace holds
  AttnSeq* seqs;
  AttnUnit* units;
  AttnPlanHead* head;
  int32_t* status;         // written where not NULL
};

// Key tiles that the queries [.., last] see, and query tiles that see keys from `first` on.
__host__ __device__ __forceinline__ int32_t attn_visible(int32_t tok, int32_t lq, int32_t lk, int32_t causal) {
  const int32_t v = causal ? tok + lk - lq + 1 : lk;
  return v < 0 ? 0 : (v > lk ? lk : v);
}
__host__ __device__ __forceinline__ int32_t attn_first_query(int32_t key, int32_t lq, int32_t lk, int32_t causal) {
  const int32_t i = causal ? key - (lk - lq) : 0;
  return i < 0 ? 0 : i;
}
__device__ __forceinline__ int32_t attn_cost(const AttnPlanArgs& a, int32_t lq, int32_t lk, int32_t t0) {
  if (a.mode == kPlanDkv) {
    const int32_t first = attn_first_query(t0, lq, lk, a.causal);
    return first >= lq ? 0 : (lq + a.tpt - 1) / a.tpt - first / a.tpt;
  }
  const int32_t last = (t0 + a.step < lq ? t0 + a.step : lq) - 1;
  return (attn_visible(last, lq, lk, a.causal) + kAtTile - 1) / kAtTile;
}

constexpr int kPlanThreads = 1024;

// Inclusive scan over the block; `carry` is added and the block's total left in *total.
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  __syncthreads();  // the previous scan's readers are done
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t n = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += n;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kPlanThreads) k_attn_plan(const AttnPlanArgs p0, const AttnPlanArgs p1) {
  const AttnPlanArgs& a = blockIdx.x == 0 ? p0 : p1;
  __shared__ int64_t warp_sums[32];
  __shared__ int32_t hist[kPlanThreads];
  __shared__ int32_t sh_unit0[kPlanThreads], sh_lq[kPlanThreads], sh_lk[kPlanThreads];  // S <= kPlanThreads
  __shared__ int32_t longest;
  __shared__ unsigned long long work;
  const int tid = threadIdx.x;
  if (tid == 0) longest = 0, work = 0;
  hist[tid] = 0;
  __syncthreads();
  int64_t units = 0, parts = 0, split_units = 0;
  int bad = 0;
  for (int64_t base = 0; base < a.S; base += kPlanThreads) {
    const int64_t s = base + tid;
    int64_t n = 0, pr = 0, su = 0;
    AttnSeq q{};
    if (s < a.S) {
      const int64_t q0 = a.qo[s], q1 = a.qo[s + 1], k0 = a.ko[s], k1 = a.ko[s + 1];
      const int64_t lk = a.kl ? static_cast<int64_t>(a.kl[s]) : k1 - k0;
      if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk || lk < 0 || lk > k1 - k0) {
        bad = 1;
      } else {
        q.q0 = q0;
        q.k0 = k0;
        q.lq = static_cast<int32_t>(q1 - q0);
        q.lk = static_cast<int32_t>(lk);
        q.nch = q.lk > kAtChunk ? (q.lk + kAtChunk - 1) / kAtChunk : 1;
        const int32_t len = a.mode == kPlanDkv ? q.lk : q.lq;
        n = (len + a.step - 1) / a.step;
        if (a.mode == kPlanFwd) {
          pr = q.nch > 1 ? static_cast<int64_t>(q.lq) * q.nch : 0;
          su = n * q.nch;
        }
        if (n > 0) {
          const int32_t c0 = attn_cost(a, q.lq, q.lk, 0);
          const int32_t c1 = attn_cost(a, q.lq, q.lk, static_cast<int32_t>((n - 1) * a.step));
          atomicMax(&longest, c0 > c1 ? c0 : c1);
          atomicAdd(&work, static_cast<unsigned long long>(n) * (c0 + c1) / 2);
        }
      }
    }
    int64_t tn, tp, ts;
    const int64_t en = plan_scan(n, warp_sums, &tn) - n + units;
    const int64_t ep = plan_scan(pr, warp_sums, &tp) - pr + parts;
    plan_scan(su, warp_sums, &ts);
    if (s < a.S) {
      q.unit0 = static_cast<int32_t>(en);
      q.part0 = ep;
      a.seqs[s] = q;
      if (base == 0) {
        sh_unit0[tid] = q.unit0;
        sh_lq[tid] = q.lq;
        sh_lk[tid] = q.lk;
      }
    }
    units += tn;
    parts += tp;
    split_units += ts;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (tid == 0) {
      a.head->nunits = 0;
      a.head->split = 0;
      if (a.status) *a.status = 8 /* BI_ERR_BAD_OFFSETS */;
    }
    return;
  }
  // Splitting pays where the longest unit is a large part of an SM's share of the work: there the
  // other SMs would wait for it.  It costs a write and a read of the partial rows.
  const bool split = a.mode == kPlanFwd && parts > 0 && parts <= a.cap_part && split_units <= a.cap_units &&
                     2ull * static_cast<unsigned long long>(longest) * a.sms > work * static_cast<unsigned long long>(a.Hkv);
  const bool near = a.S <= kPlanThreads;
  // counting sort by cost, dearest first; the order within a cost is free (it decides which SM
  // works on a unit, never a result)
  for (int pass = 0; pass < 2; ++pass) {
    for (int64_t i = tid; i < units; i += kPlanThreads) {
      int32_t lo = 0, hi = a.S - 1;
      while (lo < hi) {  // the last sequence whose first unit is not behind i
        const int32_t mid = lo + (hi - lo + 1) / 2;
        if ((near ? sh_unit0[mid] : a.seqs[mid].unit0) <= i)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int32_t unit0 = near ? sh_unit0[lo] : a.seqs[lo].unit0;
      const int32_t lq = near ? sh_lq[lo] : a.seqs[lo].lq, lk = near ? sh_lk[lo] : a.seqs[lo].lk;
      const int32_t t0 = static_cast<int32_t>(i - unit0) * a.step;
      const int32_t cost = attn_cost(a, lq, lk, t0);
      const int32_t nc = split ? (cost + kAtChunkTiles - 1) / kAtChunkTiles : 1;
      for (int32_t c = 0; c < (nc > 0 ? nc : 1); ++c) {
        const int32_t left = cost - c * kAtChunkTiles;
        int32_t w = split && left > kAtChunkTiles ? kAtChunkTiles : left;
        w = w < kPlanThreads - 1 ? w : kPlanThreads - 1;
        const int32_t at = atomicAdd(&hist[w], 1);
        if (pass == 1) a.units[at] = AttnUnit{lo, t0, split ? c : 0, split ? c + 1 : 0x7fffffff / kAtChunkTiles};
      }
    }
    __syncthreads();
    if (pass == 0) {
      const int32_t w = kPlanThreads - 1 - tid;
      const int64_t n = hist[w];
      int64_t total;
      const int64_t e = plan_scan(n, warp_sums, &total) - n;
      hist[w] = static_cast<int32_t>(e);
      if (tid == 0) {
        a.head->nunits = static_cast<int32_t>(total);
        a.head->split = split ? 1 : 0;
        if (a.status) *a.status = 0;
      }
      __syncthreads();
    }
  }
}

// ----------------------------------------------------------------------------------------------
// forward
// ----------------------------------------------------------------------------------------------
struct AttnFwdArgs {
  const AttnSeq* seqs;
  const AttnUnit* units;
  const AttnPlanHead* head;
  uint16_t* out;       // [Tq][Hq][D]
  float* lse;          // [Hq][Tq]
  float* scratch;      // [CTAs][rows][D / 4][128][4]: running O of tiles with several chunks
  float* part;         // [partial rows][Hq][D]
  float2* part_ml;     // [partial rows][Hq]: (m, l)
  int64_t Tq;
  int32_t Hq, Hkv, G, tpt;
  int32_t rows;        // row tiles of a unit
  int32_t causal;
  float c;             // scale log2(e)
  bool wide;           // out starts at a 32-byte boundary
  int32_t* status;
  uint64_t limit_ns;
};

// kRows: row tiles of a unit.  Two share every key tile, and one's products run beside the other's softmax;
// single tokens fill one only, and two blocks of one row tile then share an SM.
// Warps 0-3 (and 4-7): softmax of the row tiles, a row to a thread; then TMA, MMA and ragged value tiles.
// A row's 128 scores stay in registers: the last four warps give up some of theirs (2 x 208 + 88 = 3 x 168
// and 168 + 88 = 2 x 128, what the block is launched with).
template <int D, int kRows>
struct AtFwdTile {
  static constexpr int tile_bytes = kAtTile * D * 2;       // Q, K and V tiles: D / 64 blocks of [128][64]
  static constexpr int slots = kRows == 2 ? (D == 128 ? 5 : 12) : (D == 128 ? 2 : 5);  // ring of K and V tiles
  static constexpr int smem = (kRows + slots) * tile_bytes;
  static constexpr int soft = 4 * kRows;                   // warps
  static constexpr int threads = 128 * kRows + 128;
  static constexpr int soft_regs = kRows == 2 ? 208 : 168, other_regs = 88;
  static constexpr int tmem = 256 * kRows;                 // columns: S of each row tile, then O
};
constexpr uint32_t kAtPairs = 8;    // more than a ring of tiles can hold
struct AtFwdShared {
  // Pair g of the tiles of a CTA: the values of its tile g - 1 and the keys of tile g, what the products
  // between two rounds of softmax read.
  uint64_t full[kAtPairs], empty[kAtPairs];
  uint64_t z_ask[kAtPairs], z_full[kAtPairs];  // its value tile is ragged: loading; has its zeros
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2][2], o_full[2];  // of the row tiles; P in halves of the keys
  uint64_t done;
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
  volatile uint32_t begun;  // units that the loading thread has begun
};
constexpr int kAtSharedBytes = static_cast<int>((sizeof(AtFwdShared) + 127) / 128 * 128);

// The difference by itself, whatever it is taken of: contracted with a product in one kernel and not in another
// it would give a row other bits in a prefill than in a decode step.
__device__ __forceinline__ float attn_join_scale(float from, float to) {
  return to == -INFINITY ? 0.f : ex2_approx(__fsub_rn(from, to));
}

// A CTA's r-th unit.  Units are listed dearest first; every other round runs backwards, so that a CTA
// that began with a dear one ends with a cheap one.
__device__ __forceinline__ int64_t at_turn(int64_t r) {
  return r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
// 32 bytes of a row.  Lanes hold rows of their own, so a warp's store touches 32 lines whatever its width: one
// wide store takes half the time of two.
__device__ __forceinline__ void at_store32b(uint16_t* o, const uint32_t* w, bool wide) {
  if (wide) {
    st_global_v8(o, w);
  } else {
    reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Keeps a rarely taken branch a branch: its selects are not to be executed everywhere.
__device__ __forceinline__ void at_rare() { asm volatile("" ::: "memory"); }

// 2^x, x below 128: x = j + f with j the nearest whole number, 2^f by the polynomial of degree 4 whose
// largest relative error on [-1/2, 1/2] is least (2^-18.5; found by Remez's exchange, the float32
// coefficients below), times 2^j put together from j's bits.  -127 and less give 0, NaN stays NaN.
__device__ __forceinline__ float2 ex2_poly(float2 x) {
  constexpr float kMagic = 12582912.f + 127.f;  // 1.5 2^23: adding it rounds to a whole number, j + 127 in the low bits
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(-127.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(-127.f));
  const float2 t = add2(x, make_float2(kMagic, kMagic));
  const float2 j = add2(t, make_float2(-kMagic, -kMagic));
  const float2 f = fma2(j, make_float2(-1.f, -1.f), x);
  float2 y = fma2(f, make_float2(0.009570102207362652f, 0.009570102207362652f),
                  make_float2(0.05591785907745361f, 0.05591785907745361f));
  y = fma2(y, f, make_float2(0.240247443318367f, 0.240247443318367f));
  y = fma2(y, f, make_float2(0.6931217908859253f, 0.6931217908859253f));
  y = fma2(y, f, make_float2(0.9999992847442627f, 0.9999992847442627f));
  return mul2(y, make_float2(__uint_as_float(__float_as_uint(t.x) << 23), __uint_as_float(__float_as_uint(t.y) << 23)));
}
// 2^x of a pair of columns.  The special function unit gives 16 results a clock and SM, as long for a
// tile's scores as its products take, so some columns of every 16 go to the FMA units instead; which
// ones is a matter of the column alone, so a row's bits do not depend on its batch.
// None, 1, 2, 3 or 4 of 8 pairs, whole calls: forward of one 8K sequence, 32/8 heads of 128: 511, 501, 488, 499 and
// 525 us, heads of 64: 440, 428, 433, 455 and 490; gradient: 1413, 1420, 1402, 1410 and 1442, heads of 64: 1146, 1129,
// 1144, 1146 and 1185; gradient of 16 sequences of 1024..2048, 12/2 heads of 128: 447, 450, 441, 443 and 460.
constexpr uint32_t kAtPoly = 0x94;  // pairs 2, 4 and 7 of 8
__device__ __forceinline__ float2 at_ex2(int pair, float2 x) {
  if ((kAtPoly >> (pair % 8)) & 1) return ex2_poly(x);
  return make_float2(ex2_approx(x.x), ex2_approx(x.y));
}

// A warp's wait for what MMAs left in tensor memory or what another role wrote.
__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, const WaitCtl& wc) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait<false>(bar, parity, wc));
  tc_fence_after();
  return ok;
}

// The ragged warp's wait: it has nothing to do with most units, and its next one may be the CTA's last.
__device__ __forceinline__ bool at_wait_behind(uint64_t* bar, uint32_t parity, const WaitCtl& wc,
                                               const volatile uint32_t* begun) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait_behind(bar, parity, wc, begun));
  tc_fence_after();
  return ok;
}

// What every role derives from a unit.
struct AtUnit {
  AttnSeq q;
  int32_t h;        // key/value head
  int32_t t0;
  int32_t jb;       // first key tile
  int32_t je0, je1;  // end of each row tile's key tiles
  int32_t n;        // end of the unit's
  __device__ __forceinline__ int32_t tiles() const { return n > jb ? n - jb : 0; }
  __device__ __forceinline__ int32_t je(int X) const { return X ? je1 : je0; }
  __device__ __forceinline__ bool ragged(int32_t j) const { return q.lk - j * kAtTile < kAtTile; }
  __device__ __forceinline__ void fetch(const AttnFwdArgs& a, int64_t u) {
    const AttnUnit w = a.units[u / a.Hkv];
    h = static_cast<int32_t>(u % a.Hkv);
    q = a.seqs[w.seq];
    t0 = w.t0;
    jb = w.c0 * kAtChunkTiles;
    const int32_t cap = w.c1 * kAtChunkTiles;
    auto end = [&](int32_t from) {
      const int32_t last = (from + a.tpt < q.lq ? from + a.tpt : q.lq) - 1;
      const int32_t m = last < from ? 0 : (attn_visible(last, q.lq, q.lk, a.causal) + kAtTile - 1) / kAtTile;
      return m < cap ? m : cap;
    };
    je0 = end(t0);
    je1 = a.rows == 2 ? end(t0 + a.tpt) : 0;
    n = je0 > je1 ? je0 : je1;
  }
};

// The tiles of a CTA's units one behind another.  The next unit's description is fetched a unit ahead,
// so that nothing waits for it at the turn.
template <class Args, class Unit>
struct AtWalk {
  const Args& a;
  const int64_t nu;
  int64_t r = 0;
  Unit x, nx;            // the current unit and the next one
  int32_t i = 0, n = 0;  // its tiles taken, and all of them
  bool more;
  __device__ __forceinline__ AtWalk(const Args& args, int64_t units) : a(args), nu(units) {
    more = at_turn(0) < nu;
    if (more) nx.fetch(a, at_turn(0));
  }
  __device__ __forceinline__ bool step() {
    while (i == n) {
      if (!more) return false;
      x = nx;
      i = 0;
      n = x.tiles();
      const int64_t u = at_turn(++r);
      more = u < nu;
      if (more) nx.fetch(a, u);
    }
    ++i;
    return true;
  }
};

template <int D, int kRows>
__device__ __forceinline__ void at_fwd_load(AtFwdShared& sh, const AttnFwdArgs& a, uint32_t smem, int64_t nu,
                                            const CUtensorMap* mq, const CUtensorMap* mk, const CUtensorMap* mv) {
  using T = AtFwdTile<D, kRows>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  tma_prefetch_desc(mq);
  tma_prefetch_desc(mk);
  tma_prefetch_desc(mv);
  const uint32_t ring = smem + kRows * T::tile_bytes;
  const uint32_t qbytes = static_cast<uint32_t>(a.tpt * a.G) * 128u * (D / 64);
  uint32_t qph = 0, g = 0, begun = 0;
  // tile `pos` of the ring (keys of tile g at 2 g, values at 2 g + 1), for pair `pair`
  auto load = [&](uint32_t pos, uint32_t pair, const CUtensorMap* m, int32_t h, int32_t row) {
    if (pos >= T::slots) {
      const uint32_t before = (pos - T::slots + 1) / 2;  // the pair that used the slot last
      if (!mbar_wait<false>(&sh.empty[before % kAtPairs], before / kAtPairs & 1u, wc)) return false;
    }
    uint64_t* bar = &sh.full[pair % kAtPairs];
    mbar_arrive_expect_tx(bar, T::tile_bytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_3d(ring + pos % T::slots * T::tile_bytes + b * kAUnitBytes, m, bar, b * 64, h, row);
    return true;
  };
  AtWalk<AttnFwdArgs, AtUnit> walk(a, nu);
  while (walk.step()) {
    const AtUnit& x = walk.x;
    const int32_t j = x.jb + walk.i - 1;
    if (walk.i == 1) {
      sh.begun = ++begun;
#pragma unroll
      for (int X = 0; X < kRows; ++X) {
        if (x.je(X) <= x.jb) continue;
        if (!mbar_wait<false>(&sh.q_empty[X], (qph >> X & 1u) ^ 1u, wc)) return;
        qph ^= 1u << X;
        mbar_arrive_expect_tx(&sh.q_full[X], qbytes);
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(smem + X * T::tile_bytes + b * kAUnitBytes, mq, &sh.q_full[X], b * 64, x.h * a.G,
                      static_cast<int32_t>(x.q.q0) + x.t0 + X * a.tpt);
      }
    }
    if (g == 0) mbar_arrive(&sh.full[0]);  // no values in the first pair
    const int32_t row = static_cast<int32_t>(x.q.k0) + j * kAtTile;
    if (!load(2 * g, g, mk, x.h, row) || !load(2 * g + 1, g + 1, mv, x.h, row)) return;
    ++g;
    if (x.ragged(j)) mbar_arrive(&sh.z_ask[g % kAtPairs]);
  }
  if (g > 0) mbar_arrive(&sh.full[g % kAtPairs]);  // no keys in the last one
}

// Rows [valid, 128) of a tile in shared memory become zeros (the whole warp): what lies behind a
// sequence's last key may be another sequence's or never written, and 0 x NaN would reach every row.
template <int D>
__device__ __forceinline__ void at_zero_rows(uint8_t* tile, int valid) {
  const int lane = threadIdx.x & 31;
  for (int r = valid + (lane >> 3); r < kAtTile; r += 4)
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      *reinterpret_cast<uint4*>(tile + b * kAUnitBytes + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_shared();
  __syncwarp();
}

// Value rows behind a sequence's last key, before the products see them.  The loading thread asks with the
// tile's load; until the tile is used up its slot, and with it the pair of barriers, belongs to it.
template <int D, int kRows>
__device__ __forceinline__ void at_fwd_ragged(AtFwdShared& sh, const AttnFwdArgs& a, uint8_t* smem_p, int64_t nu) {
  using T = AtFwdTile<D, kRows>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  uint32_t g = 0, used = 0;  // the unit's first tile, a phase for each pair of barriers
  for (int64_t r = 0, u; (u = at_turn(r)) < nu; ++r) {
    AtUnit x;
    x.fetch(a, u);
    const uint32_t tiles = static_cast<uint32_t>(x.tiles());
    if (tiles == 0) continue;
    g += tiles;
    if (!x.ragged(x.n - 1)) continue;
    const uint32_t b = g % kAtPairs;
    if (!at_wait_behind(&sh.z_ask[b], (used >> b) & 1u, wc, &sh.begun) || !at_wait(&sh.full[b], g / kAtPairs & 1u, wc)) return;
    used ^= 1u << b;
    at_zero_rows<D>(smem_p + (kRows + (2 * g - 1) % T::slots) * T::tile_bytes, x.q.lk - (x.n - 1) * kAtTile);
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.z_full[b]);
  }
}

// One thread.  A row tile's next scores go behind its product with the values, into the columns that held
// its P; the other row tile's softmax runs meanwhile.  The loop over a unit's tiles is kept short: what the
// thread does besides issuing has to fit into the time of 32 MMAs, 2048 clocks.
template <int D, int kRows>
__device__ __forceinline__ void at_fwd_mma(AtFwdShared& sh, const AttnFwdArgs& a, uint32_t smem, int64_t nu,
                                           uint32_t tmem) {
  using T = AtFwdTile<D, kRows>;
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
  constexpr uint32_t idesc_o = idesc_bf16(128, D, false, true);
  constexpr uint64_t blk = kAUnitBytes >> 4;
  constexpr uint32_t ts = T::tile_bytes >> 4;
  const uint64_t dq0 = sdesc_k_sw128(smem);
  const uint64_t dk0 = sdesc_k_sw128(smem + kRows * T::tile_bytes);
  const uint64_t dv0 = sdesc_mn_sw128(smem + kRows * T::tile_bytes, kAUnitBytes);
  using Row0 = std::integral_constant<int, 0>;
  using Row1 = std::integral_constant<int, 1>;
  uint32_t g = 0, kat = 0, vat = 0;      // pair; its tiles' slots times the tile's size
  uint32_t qph = 0, pph = 0, zph = 0;    // a phase for each row tile; for each pair of barriers
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait<false>(bar, parity, wc);
    tc_fence_after();
    return ok;
  };
  auto scores = [&](auto XC) {  // S_X = Q_X K^T
    constexpr int X = decltype(XC)::value;
    const uint64_t da = dq0 + X * ts, db = dk0 + kat;
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        umma_bf16(tmem + X * 128, da + b * blk + 2 * k, db + b * blk + 2 * k, idesc_s, (b | k) ? 1u : 0u);
    umma_commit(&sh.s_full[X]);
  };
  auto values = [&](auto XC, bool fresh) {  // O_X += P_X V
    constexpr int X = decltype(XC)::value;
    const uint64_t db = dv0 + vat;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (!wait(&sh.p_full[X][half], pph >> X & 1u)) return false;
#pragma unroll
      for (int k = 4 * half; k < 4 * half + 4; ++k)
        umma_bf16_ta(tmem + 128 * kRows + X * D, tmem + X * 128 + k * 8, db + k * (2048 >> 4), idesc_o, (k > 0 || !fresh) ? 1u : 0u);
    }
    pph ^= 1u << X;
    return true;
  };
  auto first1 = [&](const AtUnit& x, auto XC) {  // a unit's first scores
    constexpr int X = decltype(XC)::value;
    if (x.je(X) <= x.jb) return true;
    if (!wait(&sh.q_full[X], qph >> X & 1u)) return false;
    qph ^= 1u << X;
    scores(XC);
    if (x.je(X) == x.jb + 1) umma_commit(&sh.q_empty[X]);
    return true;
  };
  auto first = [&](const AtUnit& x) { return first1(x, Row0{}) && (kRows == 1 || first1(x, Row1{})); };
  auto turn = [&]() {  // on to the next pair
    umma_commit(&sh.empty[g % kAtPairs]);
    ++g;
    vat = kat + ts == T::slots * ts ? 0u : kat + ts;
    kat = vat + ts == T::slots * ts ? 0u : vat + ts;
  };
  AtUnit x, nx;
  int64_t r = 0;
  auto fetch = [&]() {  // the next unit that has tiles
    for (int64_t u; (u = at_turn(r)) < nu;) {
      ++r;
      nx.fetch(a, u);
      if (nx.tiles() > 0) return true;
    }
    return false;
  };
  bool next = fetch();
  bool go = next && wait(&sh.full[0], 0u) && first(nx);
  if (go) turn();
  while (go && next) {
    x = nx;
    next = fetch();
    const int32_t n = x.n - x.jb, e0 = x.je0 - x.jb, e1 = x.je1 - x.jb;
    for (int32_t i = 0; i + 1 < n && go; ++i) {
      go = wait(&sh.full[g % kAtPairs], g / kAtPairs & 1u);
      const bool fresh = i % kAtChunkTiles == 0, end = (i + 1) % kAtChunkTiles == 0;
      auto row = [&](auto XC, int32_t e) {
        constexpr int X = decltype(XC)::value;
        if (i < e) {
          go = go && values(XC, fresh);
          if (end || i + 1 == e) umma_commit(&sh.o_full[X]);
        }
        if (i + 1 < e) {
          scores(XC);
          if (i + 2 == e) umma_commit(&sh.q_empty[X]);
        }
      };
      row(Row0{}, e0);
      if (kRows == 2) row(Row1{}, e1);
      turn();
    }
    if (!go || !wait(&sh.full[g % kAtPairs], g / kAtPairs & 1u)) break;
    if (x.ragged(x.n - 1)) {
      const uint32_t b = g % kAtPairs;
      if (!wait(&sh.z_full[b], (zph >> b) & 1u)) break;
      zph ^= 1u << b;
    }
    auto row = [&](auto XC, int32_t e) {
      constexpr int X = decltype(XC)::value;
      if (e != n) return;
      go = go && values(XC, (n - 1) % kAtChunkTiles == 0);
      umma_commit(&sh.o_full[X]);
    };
    row(Row0{}, e0);
    if (kRows == 2) row(Row1{}, e1);
    if (go && next) go = first(nx);
    turn();
  }
  umma_commit(&sh.done);
  mbar_wait<false>(&sh.done, 0u, wc);
}

// Softmax and output of row tile X (128 threads, a row each).
template <int D, int kRows>
__device__ __forceinline__ void at_fwd_softmax(AtFwdShared& sh, const AttnFwdArgs& a, int X, int64_t nu, bool split,
                                               uint32_t tmem) {
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = warp * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t ts = tmem + X * 128 + lanes, to = tmem + 128 * kRows + X * D + lanes;
  const int tok_in = row / a.G, g = row - tok_in * a.G;
  float4* scr = reinterpret_cast<float4*>(a.scratch) + ((static_cast<int64_t>(blockIdx.x) * kRows + X) * (D / 4)) * 128 + row;
  uint32_t sph = 0, oph = 0;
  const float2 cc = make_float2(a.c, a.c);
  for (int64_t r = 0, u; (u = at_turn(r)) < nu; ++r) {
    AtUnit x;
    x.fetch(a, u);
    const int32_t tok = x.t0 + X * a.tpt + tok_in;
    const bool valid = tok_in < a.tpt && tok < x.q.lq;
    const bool warp_valid = __any_sync(0xffffffffu, valid);
    // rows without a query see all, so that they do not make their warp mask every tile
    const int32_t vis = valid ? attn_visible(tok, x.q.lq, x.q.lk, a.causal) : 0x7fffffff;
    const int32_t head = x.h * a.G + g;
    uint16_t* out = a.out + ((x.q.q0 + tok) * a.Hq + head) * D;
    float* lse = a.lse + static_cast<int64_t>(head) * a.Tq + x.q.q0 + tok;
    const bool joined = split && x.q.nch > 1;  // k_attn_join writes the rows of this sequence
    if (x.je(X) <= x.jb) {
      if (valid && !joined) {  // no key to see
#pragma unroll
        for (int e = 0; e < D / 8; ++e) reinterpret_cast<uint4*>(out)[e] = make_uint4(0u, 0u, 0u, 0u);
        *lse = -INFINITY;
      }
      continue;
    }
    float m = -INFINITY, l = 0.f;          // of the chunk
    float m_run = -INFINITY, l_run = 0.f;  // of the chunks before
    for (int32_t j = x.jb; j < x.je(X); ++j) {
      if (!at_wait(&sh.s_full[X], sph, wc)) return;
      sph ^= 1u;
      const bool first = j % kAtChunkTiles == 0;
      if (first) m = -INFINITY, l = 0.f;
      if (warp_valid) {
        uint32_t s[4][32];
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld32(ts + b * 32, s[b]);
        tmem_ld_wait();
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld_pin(s[b]);
        const int32_t lim = vis - j * kAtTile;
        if (__any_sync(0xffffffffu, lim < kAtTile)) {
          at_rare();
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (b * 32 + e >= lim) s[b][e] = 0xff800000u;  // -inf
        }
        float mx[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          mx[b] = __uint_as_float(s[b][0]);
#pragma unroll
          for (int e = 1; e < 31; e += 2)
            mx[b] = fmaxf(fmaxf(mx[b], __uint_as_float(s[b][e])), __uint_as_float(s[b][e + 1]));
          mx[b] = fmaxf(mx[b], __uint_as_float(s[b][31]));
        }
        const float top = __fmul_rn(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), a.c);  // rounded: see attn_join_scale
        if (first) {
          m = top;
        } else {
          const bool raise = top > __fadd_rn(m, 8.f);
          if (__any_sync(0xffffffffu, raise)) {
            at_rare();
            // S of this tile was issued behind the last product into O: O is complete
            const float alpha = raise ? attn_join_scale(m, top) : 1.f;
            if (raise) m = top;
            l = __fmul_rn(l, alpha);
#pragma unroll 1
            for (int b = 0; b < D / 16; ++b) {
              uint32_t o[16];
              tmem_ld16(to + b * 16, o);
              tmem_ld_wait();
              tmem_ld_pin16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st16(to + b * 16, o);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : -m;
        const float2 mm = make_float2(mu, mu);
        float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t(&c)[32] = s[2 * half + e / 16];
            const float2 v = make_float2(__uint_as_float(c[2 * (e % 16)]), __uint_as_float(c[2 * (e % 16) + 1]));
            const float2 y = at_ex2(e, fma2(v, cc, mm));
            sum[e % 2] = add2(sum[e % 2], y);
            p[e] = pack_bf16x2(y.x, y.y);  // bf16 terms: what the tensor cores take; l keeps fp32
          }
          tmem_st32(ts + half * 32, p);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&sh.p_full[X][half]);
        }
        l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      } else {
        mbar_arrive(&sh.p_full[X][0]);
        mbar_arrive(&sh.p_full[X][1]);
      }
      const bool last = j + 1 == x.je(X);
      if (!last && (j + 1) % kAtChunkTiles != 0) continue;
      // the chunk's end
      if (!at_wait(&sh.o_full[X], oph, wc)) return;
      oph ^= 1u;
      if (!warp_valid) continue;
      const bool fresh = j - x.jb < kAtChunkTiles;  // no chunk before it in this unit
      if (joined) {
        const int64_t pr = (x.q.part0 + static_cast<int64_t>(tok) * x.q.nch + j / kAtChunkTiles) * a.Hq + head;
        const bool mine = valid && vis > j / kAtChunkTiles * kAtChunk;
        if (mine) a.part_ml[pr] = make_float2(m, l);
#pragma unroll 1
        for (int b = 0; b < D / 32; ++b) {
          uint32_t o[32];
          tmem_ld32(to + b * 32, o);
          tmem_ld_wait();
          tmem_ld_pin(o);
          if (mine)
#pragma unroll
            for (int e = 0; e < 4; ++e) st_global_v8(a.part + pr * D + b * 32 + e * 8, o + e * 8);
        }
        continue;
      }
      const float m_new = fmaxf(m_run, m);
      const float ka = fresh ? 0.f : attn_join_scale(m_run, m_new), kb = fresh ? 1.f : attn_join_scale(m, m_new);
      l_run = fresh ? l : fmaf(l, kb, __fmul_rn(l_run, ka));
      m_run = m_new;
      const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
      if (fresh && last) {  // a row of one chunk: all of O at once
        uint32_t o[D / 32][32];
#pragma unroll
        for (int b = 0; b < D / 32; ++b) tmem_ld32(to + b * 32, o[b]);
        tmem_ld_wait();
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          tmem_ld_pin(o[b]);
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            p[e] = pack_bf16x2(__uint_as_float(o[b][2 * e]) * inv, __uint_as_float(o[b][2 * e + 1]) * inv);
          if (valid) {
            at_store32b(out + b * 32, p, a.wide);
            at_store32b(out + b * 32 + 16, p + 8, a.wide);
          }
        }
        if (valid) *lse = m_run == -INFINITY ? -INFINITY : fmaf(m_run, 0.69314718055994531f, logf(l_run));
        continue;
      }
#pragma unroll 1
      for (int b = 0; b < D / 32; ++b) {
        uint32_t o[32];
        tmem_ld32(to + b * 32, o);
        tmem_ld_wait();
        tmem_ld_pin(o);
        if (!fresh) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 q = scr[(b * 8 + e) * 128];
            o[4 * e] = __float_as_uint(fmaf(__uint_as_float(o[4 * e]), kb, q.x * ka));
            o[4 * e + 1] = __float_as_uint(fmaf(__uint_as_float(o[4 * e + 1]), kb, q.y * ka));
            o[4 * e + 2] = __float_as_uint(fmaf(__uint_as_float(o[4 * e + 2]), kb, q.z * ka));
            o[4 * e + 3] = __float_as_uint(fmaf(__uint_as_float(o[4 * e + 3]), kb, q.w * ka));
          }
        }
        if (!last) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            scr[(b * 8 + e) * 128] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                 __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        } else if (valid) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            p[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(out + b * 32 + e * 8) =
                make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]);
        }
      }
      if (last && valid)
        *lse = m_run == -INFINITY ? -INFINITY : fmaf(m_run, 0.69314718055994531f, logf(l_run));
    }
  }
}

template <int D, int kRows>
__global__ void __launch_bounds__(AtFwdTile<D, kRows>::threads, 3 - kRows)
    k_attn_fwd(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const AttnFwdArgs a) {
  // mq: Q [Tq][Hq][D], box {64, G, tpt}; mk, mv: [Tk][Hkv][D], box {64, 1, 128}; 128-byte swizzle
  using T = AtFwdTile<D, kRows>;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  AtFwdShared& sh = *reinterpret_cast<AtFwdShared*>(dsmem + T::smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < static_cast<int>(kAtPairs); ++i) {
      mbar_init(&sh.full[i], 2);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.z_ask[i], 1);
      mbar_init(&sh.z_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i][0], 128);
      mbar_init(&sh.p_full[i][1], 128);
      mbar_init(&sh.o_full[i], 1);
    }
    mbar_init(&sh.done, 1);
    sh.abort_flag = 0u;
    sh.begun = 0u;
    fence_mbar_init_cluster();
  }
  if (warp == T::soft + 1) {
    tmem_alloc(&sh.tmem_base, T::tmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  const uint32_t smem = smem_u32(dsmem);
  const bool misaligned = (smem & 1023u) != 0;
  if (misaligned && threadIdx.x == 0) raise_status(a.status, 4 /* BI_ERR_CUDA */);
  const int64_t nu = misaligned ? 0 : static_cast<int64_t>(a.head->nunits) * a.Hkv;
  const bool split = a.head->split != 0;
  if (warp < T::soft) {
    regs_take<T::soft_regs>();
    at_fwd_softmax<D, kRows>(sh, a, warp >> 2, nu, split, tmem);
  } else {
    regs_give<T::other_regs>();
    if (warp == T::soft) {
      if (lane == 0) at_fwd_load<D, kRows>(sh, a, smem, nu, &mq, &mk, &mv);
      __syncwarp();
    } else if (warp == T::soft + 1) {
      if (elect_one()) at_fwd_mma<D, kRows>(sh, a, smem, nu, tmem);
      __syncwarp();
    } else if (warp == T::soft + 2) {
      at_fwd_ragged<D, kRows>(sh, a, dsmem, nu);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (sh.abort_flag != 0u) {  // on the error path a copy or a commit may still be in flight
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000u) {
    }
  }
  if (warp == T::soft + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, T::tmem);
  }
}

// Joins the chunks of split rows, a warp a row: the expressions of the forward's own joining.
constexpr int kAtJoinThreads = 128;
template <int D>
__global__ void __launch_bounds__(kAtJoinThreads)
    k_attn_join(const AttnFwdArgs a, const int32_t S) {
  if (a.head->split == 0 || a.head->nunits == 0) return;
  const int lane = threadIdx.x & 31;
  constexpr int N = D / 32;
  const int64_t rows = a.Tq * a.Hq;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * (kAtJoinThreads / 32);
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * kAtJoinThreads + threadIdx.x) >> 5; r < rows; r += nw) {
    const int64_t t = r / a.Hq;
    const int32_t head = static_cast<int32_t>(r - t * a.Hq);
    int32_t lo = 0, hi = S - 1;
    while (lo < hi) {
      const int32_t mid = lo + (hi - lo + 1) / 2;
      if (a.seqs[mid].q0 <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    const AttnSeq q = a.seqs[lo];
    const int64_t tok = t - q.q0;
    if (q.nch <= 1 || tok < 0 || tok >= q.lq) continue;
    const int32_t vis = attn_visible(static_cast<int32_t>(tok), q.lq, q.lk, a.causal);
    const int32_t nch = (vis + kAtChunk - 1) / kAtChunk;
    float m_run = -INFINITY, l_run = 0.f, o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
    for (int32_t c = 0; c < nch; ++c) {
      const int64_t pr = (q.part0 + tok * q.nch + c) * a.Hq + head;
      const float2 ml = a.part_ml[pr];
      const float m_new = fmaxf(m_run, ml.x);
      const float ka = c == 0 ? 0.f : attn_join_scale(m_run, m_new), kb = c == 0 ? 1.f : attn_join_scale(ml.x, m_new);
      l_run = c == 0 ? ml.y : fmaf(ml.y, kb, __fmul_rn(l_run, ka));
      m_run = m_new;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float v = a.part[pr * D + e * 32 + lane];
        o[e] = c == 0 ? v : fmaf(v, kb, o[e] * ka);
      }
    }
    const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
    uint16_t* out = a.out + r * D;
#pragma unroll
    for (int e = 0; e < N; ++e) out[e * 32 + lane] = static_cast<uint16_t>(pack_bf16x2(o[e] * inv, 0.f) & 0xffffu);
    if (lane == 0)
      a.lse[static_cast<int64_t>(head) * a.Tq + t] =
          m_run == -INFINITY ? -INFINITY : fmaf(m_run, 0.69314718055994531f, logf(l_run));
  }
}

}  // namespace bi
