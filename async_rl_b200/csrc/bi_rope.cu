// bi_rope.cu -- entry points of the per-head norm with rotation (include/bi_model.h).
#include <cmath>

#include "bi_model.h"
#include "host.h"
#include "kernels_rope.cuh"

namespace {

using namespace bi::host;

bool shape_ok(int32_t Hq, int32_t Hkv, int32_t D, int32_t R) {
  return Hq > 0 && Hkv > 0 && Hq <= 4096 && Hkv <= 4096 && D > 0 && D % 16 == 0 && D <= bi::kRopeMaxD && R > 0 &&
         R % 16 == 0 && R <= D;
}
// rows of `heads` vectors, `ld` elements apart
bool rows_ok(const void* p, int64_t ld, int32_t heads, int32_t D) {
  return p && aligned16(p) && ld >= static_cast<int64_t>(heads) * D && ld % 8 == 0;
}
int lanes_of(int32_t D) {
  int n = 1;
  while (n < D / 16) n *= 2;
  return n;
}

// A warp takes a token with all its heads, so that its angles are computed once, where the tokens
// alone fill the SMs; with fewer tokens it takes one pass's heads, so that a decode step's few tokens
// do not queue their heads one behind another.
void split_heads(bi::RopeArgs& a, int lh, int sms) {
  const int at_once = 32 / lh;
  const int slots = (a.Hq + at_once - 1) / at_once + (a.Hkv + at_once - 1) / at_once;
  a.sb = a.T >= static_cast<int64_t>(sms) * 16 ? slots : 1;
  a.nsb = (slots + a.sb - 1) / a.sb;
}

unsigned grid_of(const bi::RopeArgs& a, int sms, int per_sm) {
  const int64_t items = a.T * a.nsb;
  const int64_t want = (items + bi::kRopeWarps - 1) / bi::kRopeWarps;
  const int64_t cap = static_cast<int64_t>(sms) * per_sm;
  return static_cast<unsigned>(want < cap ? want : cap);
}

constexpr int kBwdBlocksPerSm = 2;
constexpr int kMaxSms = 160;

}  // namespace

extern "C" {

size_t bi_qk_norm_rope_bwd_workspace_bytes(int32_t D) {
  if (D <= 0 || D % 16 != 0 || D > bi::kRopeMaxD) return 0;
  return static_cast<size_t>(kMaxSms) * kBwdBlocksPerSm * 2 * static_cast<size_t>(D) * sizeof(float);
}

bi_status bi_qk_norm_rope(const uint16_t* q, const uint16_t* k, int64_t q_ld, int64_t k_ld, const uint16_t* gq,
                          const uint16_t* gk, const int32_t* positions, const float* inv_freq, float eps, int64_t T,
                          int32_t Hq, int32_t Hkv, int32_t D, int32_t R, uint16_t* q_out, uint16_t* k_out,
                          int64_t q_out_ld, int64_t k_out_ld, int32_t* dev_status, void* stream) {
  if (!dev_status || T < 0 || T >= (int64_t{1} << 31) || !(eps >= 0.f) || !std::isfinite(eps)) return BI_ERR_INVALID_ARG;
  if (!shape_ok(Hq, Hkv, D, R)) return BI_ERR_UNSUPPORTED_SHAPE;
  if ((gq == nullptr) != (gk == nullptr) || !aligned16(gq) || !aligned16(gk) || !inv_freq) return BI_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !rows_ok(q, q_ld, Hq, D) || !rows_ok(k, k_ld, Hkv, D) || !rows_ok(q_out, q_out_ld, Hq, D) ||
                !rows_ok(k_out, k_out_ld, Hkv, D)))
    return BI_ERR_INVALID_ARG;
  const uint64_t gain_bytes = static_cast<uint64_t>(D) * 2;
  if (aliased({span_rows(q_out, T, q_out_ld, Hq, D), span_rows(k_out, T, k_out_ld, Hkv, D), span(dev_status, 4)},
              {span_rows(q, T, q_ld, Hq, D), span_rows(k, T, k_ld, Hkv, D), span(gq, gain_bytes), span(gk, gain_bytes),
               span(positions, T * 4), span(inv_freq, R * uint64_t{2})}))
    return BI_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return BI_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) return cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
  bi::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.oq = q_out;
  a.ok = k_out;
  a.gq = gq;
  a.gk = gk;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.q_ld = q_ld;
  a.k_ld = k_ld;
  a.oq_ld = q_out_ld;
  a.ok_ld = k_out_ld;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.R = R;
  a.eps = eps;
  a.status = dev_status;
  const int lh = lanes_of(D);
  split_heads(a, lh, sms);
  const unsigned grid = grid_of(a, sms, bi::kRopeFwdBlocks);
  ProfScope ps(kKQkRope, s);
#define BI_ROPE(LH_)                                                                   \
  if (lh == LH_) {                                                                     \
    if (gq)                                                                            \
      bi::k_qk_rope<LH_, true><<<grid, bi::kRopeThreads, 0, s>>>(a);                   \
    else                                                                               \
      bi::k_qk_rope<LH_, false><<<grid, bi::kRopeThreads, 0, s>>>(a);                  \
  }
  BI_ROPE(1) BI_ROPE(2) BI_ROPE(4) BI_ROPE(8) BI_ROPE(16)
#undef BI_ROPE
  return cudaGetLastError() == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

bi_status bi_qk_norm_rope_bwd(const uint16_t* dq_out, const uint16_t* dk_out, int64_t dq_out_ld, int64_t dk_out_ld,
                              const uint16_t* q, const uint16_t* k, int64_t q_ld, int64_t k_ld, const uint16_t* gq,
                              const uint16_t* gk, const int32_t* positions, const float* inv_freq, float eps, int64_t T,
                              int32_t Hq, int32_t Hkv, int32_t D, int32_t R, uint16_t* dq, uint16_t* dk, int64_t dq_ld,
                              int64_t dk_ld, float* dgq, float* dgk, int32_t* dev_status, void* ws, size_t ws_bytes,
                              void* stream) {
  if (!dev_status || T < 0 || T >= (int64_t{1} << 31) || !(eps >= 0.f) || !std::isfinite(eps)) return BI_ERR_INVALID_ARG;
  if (!shape_ok(Hq, Hkv, D, R)) return BI_ERR_UNSUPPORTED_SHAPE;
  if ((gq == nullptr) != (gk == nullptr) || !aligned16(gq) || !aligned16(gk) || !inv_freq) return BI_ERR_INVALID_ARG;
  if (gq && (!dgq || !dgk)) return BI_ERR_INVALID_ARG;
  if (T > 0 && (!positions || !rows_ok(dq_out, dq_out_ld, Hq, D) || !rows_ok(dk_out, dk_out_ld, Hkv, D) ||
                !rows_ok(dq, dq_ld, Hq, D) || !rows_ok(dk, dk_ld, Hkv, D)))
    return BI_ERR_INVALID_ARG;
  if (T > 0 && gq && (!rows_ok(q, q_ld, Hq, D) || !rows_ok(k, k_ld, Hkv, D))) return BI_ERR_INVALID_ARG;
  if (T > 0 && !gq && (dq == q || dk == k)) return BI_ERR_INVALID_ARG;  // not read, their strides may say nothing
  if (gq && (!ws || ws_bytes < bi_qk_norm_rope_bwd_workspace_bytes(D) || (reinterpret_cast<uintptr_t>(ws) & 255u)))
    return BI_ERR_WORKSPACE;
  const uint64_t gain_bytes = static_cast<uint64_t>(D) * 2, gain_grad = gq ? 2 * gain_bytes : 0;
  const int64_t read = gq ? T : 0;  // rows of q and k
  if (aliased({span_rows(dq, T, dq_ld, Hq, D), span_rows(dk, T, dk_ld, Hkv, D), span(dgq, gain_grad), span(dgk, gain_grad),
               span(dev_status, 4), span(ws, gq ? bi_qk_norm_rope_bwd_workspace_bytes(D) : 0)},
              {span_rows(dq_out, T, dq_out_ld, Hq, D), span_rows(dk_out, T, dk_out_ld, Hkv, D),
               span_rows(q, read, q_ld, Hq, D), span_rows(k, read, k_ld, Hkv, D), span(gq, gain_bytes),
               span(gk, gain_bytes), span(positions, T * 4), span(inv_freq, R * uint64_t{2})}))
    return BI_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0 || sms > kMaxSms) return BI_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (gq && (cudaMemsetAsync(dgq, 0, sizeof(float) * D, s) != cudaSuccess ||
               cudaMemsetAsync(dgk, 0, sizeof(float) * D, s) != cudaSuccess))
      return BI_ERR_CUDA;
    return cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
  }
  bi::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.dzq = dq_out;
  a.dzk = dk_out;
  a.oq = dq;
  a.ok = dk;
  a.gq = gq;
  a.gk = gk;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.q_ld = q_ld;
  a.k_ld = k_ld;
  a.dzq_ld = dq_out_ld;
  a.dzk_ld = dk_out_ld;
  a.oq_ld = dq_ld;
  a.ok_ld = dk_ld;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.R = R;
  a.eps = eps;
  a.parts = static_cast<float*>(ws);
  a.status = dev_status;
  const int lh = lanes_of(D);
  split_heads(a, lh, sms);
  const unsigned grid = grid_of(a, sms, kBwdBlocksPerSm);
  {
    ProfScope ps(kKQkRopeBwd, s);
#define BI_ROPE(LH_)                                                                       \
  if (lh == LH_) {                                                                         \
    if (gq)                                                                                \
      bi::k_qk_rope_bwd<LH_, true><<<grid, bi::kRopeThreads, 0, s>>>(a);                   \
    else                                                                                   \
      bi::k_qk_rope_bwd<LH_, false><<<grid, bi::kRopeThreads, 0, s>>>(a);                  \
  }
    BI_ROPE(1) BI_ROPE(2) BI_ROPE(4) BI_ROPE(8) BI_ROPE(16)
#undef BI_ROPE
  }
  if (gq) {
    ProfScope ps(kKQkGain, s);
    bi::k_qk_gain<<<static_cast<unsigned>((2 * D + 31) / 32), 32 * bi::kGainStrands, 0, s>>>(
        a.parts, static_cast<int>(grid), D, dgq, dgk);
  }
  return cudaGetLastError() == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

}  // extern "C"
