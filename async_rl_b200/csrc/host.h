// host.h -- what the host sides of the entry points share: the optional per-kernel timing, small
// helpers and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <vector>

namespace bi {
namespace host {

constexpr uint64_t kWaitLimitNs = 4000000000ull;  // 4 s for any single in-kernel wait

// ---------------------------------------------------------------------------------------------
// optional per-kernel timing (events around each launch; measurement tools only)
// ---------------------------------------------------------------------------------------------
enum KernelKind : int { kKPrep, kKRowmap, kKZeroRows, kKGather, kKLmFwd, kKLmFwdDH, kKLmDW, kKDwRows,
                        kKDwStream, kKSeqGate, kKRowParts, kKReduce, kKD3Partial, kKGemm, kKRmsNorm, kKLmZscan,
                        kKLmDecode1, kKD1Zero, kKQkRope, kKQkRopeBwd, kKQkGain, kKAttnPlan, kKAttnFwd, kKAttnJoin, kKAttnPre,
                        kKAttnDkv, kKAttnDq, kKAdamW, kNumKinds };
inline const char* const kKindNames[kNumKinds] = {"k_prep", "k_rowmap", "k_zero_prompt_rows", "k_gather_rows",
                                           "k_lm_fwd", "k_lm_fwd_dh", "k_lm_dw", "k_dw_rows", "k_dw_stream",
                                           "k_seq_gate", "k_row_parts", "k_reduce_parts", "k_d3_partial",
                                           "k_gemm_pair", "k_rmsnorm", "k_lm_zscan", "k_lm_decode1",
                                           "k_d1_zero", "k_qk_rope", "k_qk_rope_bwd", "k_qk_gain", "k_attn_plan", "k_attn_fwd",
                                           "k_attn_join", "k_attn_pre", "k_attn_dkv", "k_attn_dq", "k_adamw"};
struct Pending {
  int kind;
  cudaEvent_t a, b;
};
struct Profiler {
  bool on = false;
  bool failed = false;
  std::vector<Pending> pending;
  std::vector<cudaEvent_t> pool;
  double ms[kNumKinds] = {};
  int64_t n[kNumKinds] = {};
  cudaEvent_t get() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreate(&e) != cudaSuccess) failed = true;
    return e;
  }
};
inline thread_local Profiler g_prof;

struct ProfScope {  // records an event pair around one launch when profiling is on
  int kind;
  cudaStream_t s;
  cudaEvent_t a = nullptr;
  ProfScope(int k, cudaStream_t st) : kind(k), s(st) {
    if (g_prof.on) {
      a = g_prof.get();
      if (a) cudaEventRecord(a, s);
    }
  }
  ~ProfScope() {
    if (g_prof.on && a) {
      cudaEvent_t b = g_prof.get();
      if (b) {
        cudaEventRecord(b, s);
        g_prof.pending.push_back({kind, a, b});
      }
    }
  }
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---------------------------------------------------------------------------------------------
// tensor maps (driver entry point fetched through the runtime; no libcuda link dependency)
// ---------------------------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}


// What a call reads or writes: `rows` rows of `row` bytes, `ld` bytes apart (1 row: a plain array).
struct Span {
  uintptr_t at;
  uint64_t rows, row, ld;
};
inline Span span(const void* p, uint64_t bytes) {
  return Span{reinterpret_cast<uintptr_t>(p), p && bytes ? 1u : 0u, bytes, bytes};
}
// bf16 rows of `heads` heads, as the attention layer's tensors are
inline Span span_rows(const void* p, int64_t rows, int64_t ld, int64_t heads, int64_t D) {
  return Span{reinterpret_cast<uintptr_t>(p), p ? static_cast<uint64_t>(rows) : 0u, static_cast<uint64_t>(heads * D * 2),
              static_cast<uint64_t>(ld * 2)};
}
// Whether two of them share a byte.  Slices of one buffer have one stride: their rows keep their distance.  With
// two strides each row of one is held against the other's rows around it.
inline bool overlap(const Span& a, const Span& b) {
  if (a.rows == 0 || b.rows == 0) return false;
  const uintptr_t ae = a.at + (a.rows - 1) * a.ld + a.row, be = b.at + (b.rows - 1) * b.ld + b.row;
  if (ae <= b.at || be <= a.at) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  const Span &few = a.rows < b.rows ? a : b, &many = a.rows < b.rows ? b : a;
  // rows of `few` that reach into the range of `many`
  const uintptr_t ms = many.at, me = many.at + (many.rows - 1) * many.ld + many.row;
  uint64_t i = few.at + few.row <= ms && few.rows > 1 ? (ms - few.at - few.row) / few.ld + 1 : 0;
  for (uint64_t n = 0; i < few.rows && few.at + i * few.ld < me; ++i, ++n) {
    const uintptr_t lo = few.at + i * few.ld, hi = lo + few.row;
    if (hi <= ms) continue;
    // the first row of `many` that ends behind lo
    const uint64_t j = lo < ms + many.row ? 0 : (lo - ms - many.row) / many.ld + 1;
    if (j < many.rows && ms + j * many.ld < hi) return true;
    if (few.ld == many.ld && n > 0) return false;  // inside both, every row is like this one
  }
  return false;
}
// Outputs may share memory with no input and with no other output.
inline bool aliased(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* p = outs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return true;
    for (const Span& i : ins)
      if (overlap(*o, i)) return true;
  }
  return false;
}

// SMs of the current device (0 where that cannot be read), asked once per device.
inline int sm_count() {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0 && cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    known[dev] = 0;
  return known[dev];
}

}  // namespace host
}  // namespace bi
