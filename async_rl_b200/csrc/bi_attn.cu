// bi_attn.cu -- entry points of softmax attention (include/bi_model.h).
#include <cmath>

#include "bi_model.h"
#include "host.h"
#include "kernels_attn_bwd.cuh"

namespace {

using namespace bi::host;

constexpr int kMaxSms = 160;
constexpr size_t kPartBytesMax = size_t{128} << 20;  // partial rows of a split forward, at most (below 2^19 of them)

struct Shape {
  int64_t Tq, Tk;
  int32_t S, Hq, Hkv, D;
  int32_t G, tpt;
};

bool shape_ok(Shape& z) {
  if (z.Hq <= 0 || z.Hkv <= 0 || z.Hq % z.Hkv != 0 || z.Hq / z.Hkv > bi::kAtTile || z.Hkv > 4096) return false;
  if (z.D != 64 && z.D != 128) return false;
  z.G = z.Hq / z.Hkv;
  z.tpt = bi::kAtTile / z.G;
  return true;
}
bool sizes_ok(const Shape& z) {
  return z.Tq >= 0 && z.Tk >= 0 && z.S >= 0 && z.Tq < (int64_t{1} << 31) - 512 && z.Tk < (int64_t{1} << 31) - 512;
}
// Units are counted in 32 bits: one for each sequence and tile at most, and the partial rows of a split forward.
bool units_ok(const Shape& z) {
  const int64_t most = (int64_t{1} << 31) - (int64_t{1} << 20);
  return z.S + z.Tq / z.tpt < most && z.S + z.Tk / bi::kAtTile < most;
}
bool rows_ok(const void* p, int64_t ld, int32_t heads, int32_t D) {
  return p && aligned16(p) && ld >= static_cast<int64_t>(heads) * D && ld % 8 == 0;
}

thread_local uint64_t g_wait_base_ns = 0;  // test hook

// Some roles wait for the length of a unit, which passes over all keys or all query rows of a sequence (none
// waits longer: the warps for ragged tiles, which pass units over, follow the units that the loading thread
// begins).  40 ns a key and row, against the 19 ns a key of the forward's two row tiles and the 13 ns a row of
// dK, dV (26 where only half of a tile's rows are used: groups of 65 heads).
uint64_t wait_limit(const Shape& z) {
  const uint64_t base = g_wait_base_ns ? g_wait_base_ns : kWaitLimitNs + 40ull * static_cast<uint64_t>(z.Tk + z.Tq * z.G);
  g_wait_base_ns = 0;
  return base;
}

// Workspace of the forward.  Partial rows are provided where the rows alone would leave SMs without
// work (fewer than four row tiles an SM), for sequences of up to twice the mean number of queries;
// where that is not enough the plan does not split, and the results are the same.
struct FwdLayout {
  size_t head, seqs, units, scratch, part, part_ml, total;
  int64_t cap_part;
  int32_t cap_units;
};
FwdLayout fwd_layout(const Shape& z) {
  FwdLayout L{};
  const int64_t S = z.S > 0 ? z.S : 1;
  const bool chunks = z.Tk > bi::kAtChunk;
  if (chunks && z.Tq * z.Hq < int64_t{4} * kMaxSms * bi::kAtTile) {
    const int64_t row = static_cast<int64_t>(z.Hq) * (z.D + 2) * 4;
    const int64_t want = 2 * ((z.Tq + S - 1) / S) * (S + z.Tk / bi::kAtChunk);
    const int64_t most = static_cast<int64_t>(kPartBytesMax) / row;
    L.cap_part = want < most ? want : most;
  }
  L.cap_units = static_cast<int32_t>(S + z.Tq / z.tpt + 1 + L.cap_part);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.head = take(sizeof(bi::AttnPlanHead));
  L.seqs = take(static_cast<size_t>(S) * sizeof(bi::AttnSeq));
  L.units = take(static_cast<size_t>(L.cap_units) * sizeof(bi::AttnUnit));
  L.scratch = take(chunks ? static_cast<size_t>(kMaxSms) * 2 * z.D * bi::kAtTile * 4 : 0);
  L.part = take(static_cast<size_t>(L.cap_part) * z.Hq * z.D * 4);
  L.part_ml = take(static_cast<size_t>(L.cap_part) * z.Hq * 8);
  L.total = o;
  return L;
}

struct BwdLayout {
  size_t head, seqs, units, seqs_kv, units_kv, st, total;
  int32_t cap_q, cap_kv;
};
BwdLayout bwd_layout(const Shape& z) {
  BwdLayout L{};
  const int64_t S = z.S > 0 ? z.S : 1;
  L.cap_q = static_cast<int32_t>(S + z.Tq / z.tpt + 1);
  L.cap_kv = static_cast<int32_t>(S + z.Tk / bi::kAtTile + 1);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.head = take(2 * sizeof(bi::AttnPlanHead));
  L.seqs = take(static_cast<size_t>(S) * sizeof(bi::AttnSeq));
  L.units = take(static_cast<size_t>(L.cap_q) * sizeof(bi::AttnUnit));
  L.seqs_kv = take(static_cast<size_t>(S) * sizeof(bi::AttnSeq));
  L.units_kv = take(static_cast<size_t>(L.cap_kv) * sizeof(bi::AttnUnit));
  L.st = take(static_cast<size_t>(z.Hkv) * L.cap_q * 2 * bi::kAtTile * 4);
  L.total = o;
  return L;
}

// [T][heads][D] bf16 with `ld` elements between tokens, box {64 columns, box_heads, box_rows}.
bool make_map_heads(CUtensorMap* m, const void* base, int64_t T, int32_t heads, int32_t D, int64_t ld, int box_heads,
                    int box_rows) {
  EncodeTiledFn f = encode_fn();
  if (!f) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(T > 0 ? T : 1)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int kRows>
bool grant_fwd() {
  return cudaFuncSetAttribute(bi::k_attn_fwd<D, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              bi::AtFwdTile<D, kRows>::smem + bi::kAtSharedBytes) == cudaSuccess;
}

// The current device's SM count, with the kernels' shared memory granted once.
int attn_device() {
  static std::mutex mu;
  static int ready[64] = {};
  int dev = 0;
  const int sms = sm_count();
  if (sms <= 0 || sms > kMaxSms || cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (!ready[dev]) {
    const int bwd128 = bi::AtBwdTile<128>::smem + bi::kAtBwdSharedBytes;
    const int bwd64 = bi::AtBwdTile<64>::smem + bi::kAtBwdSharedBytes;
    constexpr auto kSmem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if (cudaFuncSetAttribute(bi::k_attn_dkv<128>, kSmem, bwd128) != cudaSuccess ||
        cudaFuncSetAttribute(bi::k_attn_dkv<64>, kSmem, bwd64) != cudaSuccess ||
        cudaFuncSetAttribute(bi::k_attn_dq<128>, kSmem, bwd128) != cudaSuccess ||
        cudaFuncSetAttribute(bi::k_attn_dq<64>, kSmem, bwd64) != cudaSuccess ||
        !grant_fwd<128, 1>() || !grant_fwd<128, 2>() || !grant_fwd<64, 1>() || !grant_fwd<64, 2>())
      return 0;
    ready[dev] = 1;
  }
  return sms;
}

template <int D, int kRows>
bool launch_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const bi::AttnFwdArgs& a,
                unsigned grid, bool join, int32_t S, int sms, cudaStream_t s) {
  {
    ProfScope ps(kKAttnFwd, s);
    using T = bi::AtFwdTile<D, kRows>;
    bi::k_attn_fwd<D, kRows><<<grid, T::threads, T::smem + bi::kAtSharedBytes, s>>>(mq, mk, mv, a);
  }
  if (join) {
    const int64_t want = (a.Tq * a.Hq + bi::kAtJoinThreads / 32 - 1) / (bi::kAtJoinThreads / 32);
    const int64_t cap = static_cast<int64_t>(sms) * 16;
    ProfScope ps(kKAttnJoin, s);
    bi::k_attn_join<D><<<static_cast<unsigned>(want < cap ? want : cap), bi::kAtJoinThreads, 0, s>>>(a, S);
  }
  return cudaGetLastError() == cudaSuccess;
}

template <int D>
bool launch_bwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                const bi::AttnBwdArgs& dq, const bi::AttnBwdArgs& dkv, const BwdLayout& L, int sms, cudaStream_t s) {
  const auto grid = [&](int64_t units, int per_sm) {
    const int64_t n = units * dq.Hkv, cap = static_cast<int64_t>(sms) * per_sm;
    return static_cast<unsigned>(n < cap ? n : cap);
  };
  constexpr int smem = bi::AtBwdTile<D>::smem + bi::kAtBwdSharedBytes;
  {
    ProfScope ps(kKAttnPre, s);
    bi::k_attn_pre<D><<<grid(L.cap_q, 8), bi::kAtPreThreads, 0, s>>>(dq);
  }
  {
    ProfScope ps(kKAttnDkv, s);
    bi::k_attn_dkv<D><<<grid(L.cap_kv, 1), bi::kAtBwdThreads, smem, s>>>(mq, mk, mv, mdo, dkv);
  }
  {
    ProfScope ps(kKAttnDq, s);
    bi::k_attn_dq<D><<<grid(L.cap_q, 1), bi::kAtBwdThreads, smem, s>>>(mq, mk, mv, mdo, dq);
  }
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace

extern "C" {

void bi_debug_attn_wait_limit_once(uint64_t limit_ns) { g_wait_base_ns = limit_ns; }

size_t bi_attn_fwd_workspace_bytes(int64_t Tq, int64_t Tk, int32_t S, int32_t Hq, int32_t Hkv, int32_t D) {
  Shape z{Tq, Tk, S, Hq, Hkv, D, 0, 0};
  if (!sizes_ok(z) || !shape_ok(z) || !units_ok(z)) return 0;
  return fwd_layout(z).total;
}

bi_status bi_attn_fwd(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t q_ld, int64_t k_ld, int64_t v_ld,
                      const int64_t* q_offsets, const int64_t* k_offsets, const int32_t* k_lens, int32_t S, int64_t Tq,
                      int64_t Tk, int32_t Hq, int32_t Hkv, int32_t D, int32_t causal, float scale, uint16_t* out,
                      float* lse, int32_t* dev_status, void* ws, size_t ws_bytes, void* stream) {
  Shape z{Tq, Tk, S, Hq, Hkv, D, 0, 0};
  if (!dev_status || !sizes_ok(z) || !(scale > 0.f) || !std::isfinite(scale)) return BI_ERR_INVALID_ARG;
  if (!shape_ok(z)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!units_ok(z)) return BI_ERR_INVALID_ARG;
  if (S > 0 && (!q_offsets || !k_offsets)) return BI_ERR_INVALID_ARG;
  if (Tq > 0 && (!rows_ok(q, q_ld, Hq, D) || !out || !aligned16(out) || !lse))
    return BI_ERR_INVALID_ARG;
  if (Tk > 0 && (!rows_ok(k, k_ld, Hkv, D) || !rows_ok(v, v_ld, Hkv, D))) return BI_ERR_INVALID_ARG;
  const FwdLayout L = fwd_layout(z);
  if (!ws || ws_bytes < L.total || (reinterpret_cast<uintptr_t>(ws) & 255u)) return BI_ERR_WORKSPACE;
  if (aliased({span_rows(out, Tq, static_cast<int64_t>(Hq) * D, Hq, D), span(lse, static_cast<uint64_t>(Hq) * Tq * 4),
               span(dev_status, 4), span(ws, L.total)},
              {span_rows(q, Tq, q_ld, Hq, D), span_rows(k, Tk, k_ld, Hkv, D), span_rows(v, Tk, v_ld, Hkv, D),
               span(q_offsets, (S + int64_t{1}) * 8), span(k_offsets, (S + int64_t{1}) * 8), span(k_lens, S * int64_t{4})}))
    return BI_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (S == 0 || Tq == 0) return cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
  const int sms = attn_device();
  if (sms <= 0) return BI_ERR_CUDA;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  bi::AttnPlanArgs p{};
  p.qo = q_offsets;
  p.ko = k_offsets;
  p.kl = k_lens;
  p.Tq = Tq;
  p.Tk = Tk;
  p.S = S;
  p.mode = bi::kPlanFwd;
  p.causal = causal != 0;
  // One row tile a unit where the sequences' queries fill one at most on average (a decode step, a long chunk of
  // prompt among many single tokens).  One and two row tiles, 32/8 heads of 128 (32 tokens a tile): 64 single tokens
  // over caches of up to 8K keys 220 and 232 us, 16 tokens each 236 and 247, 33 tokens each 405 and 335, 64 tokens each
  // 374 and 300; 200 single tokens over up to 4K keys with a chunk of 2048, 4096 or 6000 tokens (11, 21 and 31 on
  // average) 396 and 423, 496 and 524, 659 and 653.
  const int rows = Tq <= static_cast<int64_t>(S) * z.tpt ? 1 : 2;
  const int blocks = rows == 1 ? 2 * sms : sms;
  p.step = rows * z.tpt;
  p.tpt = z.tpt;
  p.sms = blocks;
  p.Hkv = Hkv;
  p.cap_units = L.cap_units;
  p.cap_part = L.cap_part;
  p.seqs = reinterpret_cast<bi::AttnSeq*>(w8 + L.seqs);
  p.units = reinterpret_cast<bi::AttnUnit*>(w8 + L.units);
  p.head = reinterpret_cast<bi::AttnPlanHead*>(w8 + L.head);
  p.status = dev_status;
  // a call without keys reads none of them: any address serves the maps
  CUtensorMap mq, mk, mv;
  const void* kb = Tk > 0 ? static_cast<const void*>(k) : ws;
  const void* vb = Tk > 0 ? static_cast<const void*>(v) : ws;
  const int64_t kl = Tk > 0 ? k_ld : static_cast<int64_t>(Hkv) * D, vl = Tk > 0 ? v_ld : static_cast<int64_t>(Hkv) * D;
  if (!make_map_heads(&mq, q, Tq, Hq, D, q_ld, z.G, z.tpt) || !make_map_heads(&mk, kb, Tk, Hkv, D, kl, 1, bi::kAtTile) ||
      !make_map_heads(&mv, vb, Tk, Hkv, D, vl, 1, bi::kAtTile))
    return BI_ERR_CUDA;
  {
    ProfScope ps(kKAttnPlan, s);
    bi::k_attn_plan<<<1, bi::kPlanThreads, 0, s>>>(p, p);
  }
  bi::AttnFwdArgs a{};
  a.seqs = p.seqs;
  a.units = p.units;
  a.head = p.head;
  a.out = out;
  a.lse = lse;
  a.scratch = reinterpret_cast<float*>(w8 + L.scratch);
  a.part = reinterpret_cast<float*>(w8 + L.part);
  a.part_ml = reinterpret_cast<float2*>(w8 + L.part_ml);
  a.Tq = Tq;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = z.G;
  a.tpt = z.tpt;
  a.rows = rows;
  a.causal = p.causal;
  a.c = scale * bi::kLog2e;
  a.status = dev_status;
  a.wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  a.limit_ns = wait_limit(z);
  const int64_t most = static_cast<int64_t>(L.cap_units) * Hkv;
  const unsigned grid = static_cast<unsigned>(most < blocks ? most : blocks);
  const auto go = D == 128 ? (rows == 1 ? launch_fwd<128, 1> : launch_fwd<128, 2>)
                           : (rows == 1 ? launch_fwd<64, 1> : launch_fwd<64, 2>);
  const bool ok = go(mq, mk, mv, a, grid, L.cap_part > 0, S, sms, s);
  return ok ? BI_OK : BI_ERR_CUDA;
}

size_t bi_attn_bwd_workspace_bytes(int64_t Tq, int64_t Tk, int32_t S, int32_t Hq, int32_t Hkv, int32_t D) {
  Shape z{Tq, Tk, S, Hq, Hkv, D, 0, 0};
  if (!sizes_ok(z) || !shape_ok(z) || !units_ok(z)) return 0;
  return bwd_layout(z).total;
}

bi_status bi_attn_bwd(const uint16_t* dout, int64_t dout_ld, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                      int64_t q_ld, int64_t k_ld, int64_t v_ld, const uint16_t* out, const float* lse,
                      const int64_t* q_offsets, const int64_t* k_offsets, const int32_t* k_lens, int32_t S, int64_t Tq,
                      int64_t Tk, int32_t Hq, int32_t Hkv, int32_t D, int32_t causal, float scale, uint16_t* dq,
                      uint16_t* dk, uint16_t* dv, int64_t dq_ld, int64_t dk_ld, int64_t dv_ld, int32_t* dev_status,
                      void* ws, size_t ws_bytes, void* stream) {
  Shape z{Tq, Tk, S, Hq, Hkv, D, 0, 0};
  if (!dev_status || !sizes_ok(z) || !(scale > 0.f) || !std::isfinite(scale)) return BI_ERR_INVALID_ARG;
  if (!shape_ok(z)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!units_ok(z)) return BI_ERR_INVALID_ARG;
  if (S > 0 && (!q_offsets || !k_offsets)) return BI_ERR_INVALID_ARG;
  if (Tq > 0 && (!rows_ok(q, q_ld, Hq, D) || !rows_ok(dout, dout_ld, Hq, D) || !rows_ok(dq, dq_ld, Hq, D) || !out ||
                 !aligned16(out) || !lse))
    return BI_ERR_INVALID_ARG;
  if (Tk > 0 && (!rows_ok(k, k_ld, Hkv, D) || !rows_ok(v, v_ld, Hkv, D) || !rows_ok(dk, dk_ld, Hkv, D) ||
                 !rows_ok(dv, dv_ld, Hkv, D)))
    return BI_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(z);
  if (!ws || ws_bytes < L.total || (reinterpret_cast<uintptr_t>(ws) & 255u)) return BI_ERR_WORKSPACE;
  if (aliased({span_rows(dq, Tq, dq_ld, Hq, D), span_rows(dk, Tk, dk_ld, Hkv, D), span_rows(dv, Tk, dv_ld, Hkv, D),
               span(dev_status, 4), span(ws, L.total)},
              {span_rows(dout, Tq, dout_ld, Hq, D), span_rows(q, Tq, q_ld, Hq, D), span_rows(k, Tk, k_ld, Hkv, D),
               span_rows(v, Tk, v_ld, Hkv, D), span_rows(out, Tq, static_cast<int64_t>(Hq) * D, Hq, D),
               span(lse, static_cast<uint64_t>(Hq) * Tq * 4), span(q_offsets, (S + int64_t{1}) * 8),
               span(k_offsets, (S + int64_t{1}) * 8), span(k_lens, S * int64_t{4})}))
    return BI_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (S == 0 || (Tq == 0 && Tk == 0))
    return cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
  const int sms = attn_device();
  if (sms <= 0) return BI_ERR_CUDA;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  bi::AttnPlanArgs p{};
  p.qo = q_offsets;
  p.ko = k_offsets;
  p.kl = k_lens;
  p.Tq = Tq;
  p.Tk = Tk;
  p.S = S;
  p.mode = bi::kPlanDq;
  p.causal = causal != 0;
  p.step = z.tpt;
  p.tpt = z.tpt;
  p.sms = sms;
  p.Hkv = Hkv;
  p.cap_units = L.cap_q;
  p.seqs = reinterpret_cast<bi::AttnSeq*>(w8 + L.seqs);
  p.units = reinterpret_cast<bi::AttnUnit*>(w8 + L.units);
  p.head = reinterpret_cast<bi::AttnPlanHead*>(w8 + L.head);
  p.status = dev_status;
  bi::AttnPlanArgs pk = p;
  pk.mode = bi::kPlanDkv;
  pk.step = bi::kAtTile;
  pk.cap_units = L.cap_kv;
  pk.seqs = reinterpret_cast<bi::AttnSeq*>(w8 + L.seqs_kv);
  pk.units = reinterpret_cast<bi::AttnUnit*>(w8 + L.units_kv);
  pk.head = p.head + 1;
  pk.status = nullptr;
  // a call without queries or keys reads none of them: any address serves the maps
  CUtensorMap mq, mk, mv, mdo;
  const auto map = [&](CUtensorMap* m, const void* at, int64_t T, int32_t heads, int64_t ld, int bh, int br) {
    return T > 0 ? make_map_heads(m, at, T, heads, D, ld, bh, br)
                 : make_map_heads(m, ws, 0, heads, D, static_cast<int64_t>(heads) * D, bh, br);
  };
  if (!map(&mq, q, Tq, Hq, q_ld, z.G, z.tpt) || !map(&mdo, dout, Tq, Hq, dout_ld, z.G, z.tpt) ||
      !map(&mk, k, Tk, Hkv, k_ld, 1, bi::kAtTile) || !map(&mv, v, Tk, Hkv, v_ld, 1, bi::kAtTile))
    return BI_ERR_CUDA;
  {
    ProfScope ps(kKAttnPlan, s);
    bi::k_attn_plan<<<2, bi::kPlanThreads, 0, s>>>(p, pk);
  }
  bi::AttnBwdArgs a{};
  a.seqs = p.seqs;
  a.units = p.units;
  a.head = p.head;
  a.rows = p.seqs;
  a.st = reinterpret_cast<float*>(w8 + L.st);
  a.tiles = L.cap_q;
  a.out = out;
  a.dout = dout;
  a.lse = lse;
  a.do_ld = dout_ld;
  a.Tq = Tq;
  a.o0 = dq;
  a.ld0 = dq_ld;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = z.G;
  a.tpt = z.tpt;
  a.causal = p.causal;
  a.c = scale * bi::kLog2e;
  a.scale = scale;
  a.status = dev_status;
  a.limit_ns = wait_limit(z);
  a.wide = (reinterpret_cast<uintptr_t>(dq) & 31u) == 0 && dq_ld % 16 == 0;
  bi::AttnBwdArgs b = a;
  b.wide = ((reinterpret_cast<uintptr_t>(dk) | reinterpret_cast<uintptr_t>(dv)) & 31u) == 0 && dk_ld % 16 == 0 && dv_ld % 16 == 0;
  b.seqs = pk.seqs;
  b.units = pk.units;
  b.head = pk.head;
  b.o0 = dk;
  b.o1 = dv;
  b.ld0 = dk_ld;
  b.ld1 = dv_ld;
  const bool ok = D == 128 ? launch_bwd<128>(mq, mk, mv, mdo, a, b, L, sms, s)
                           : launch_bwd<64>(mq, mk, mv, mdo, a, b, L, sms, s);
  return ok ? BI_OK : BI_ERR_CUDA;
}

}  // extern "C"
