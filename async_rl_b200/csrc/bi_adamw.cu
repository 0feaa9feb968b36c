// bi_adamw.cu -- entry point of the AdamW step (include/bi_optim.h).
#include <cmath>
#include <memory>
#include <new>

#include "bi_optim.h"
#include "host.h"
#include "kernels_adamw.cuh"

namespace {

using namespace bi::host;

// Tensors of one launch: the small tables keep the launch of a few tensors short, the large one fills
// the 32,764 bytes that kernel parameters may take.
constexpr int kSmall = 16;
constexpr int kMiddle = 96;
constexpr int kLarge = 440;
static_assert(sizeof(bi::AdamTable<kLarge>) + sizeof(bi::AdamArgs) <= 32764, "kernel parameters");

bool finite_nonneg(double x) { return x >= 0.0 && std::isfinite(x); }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int kMax>
bool launch(const bi_adamw_tensor* ts, int32_t& at, int32_t count, const bi_adamw_cfg& c, bool master, bi::AdamArgs& a,
            cudaStream_t s) {
  auto tab = std::unique_ptr<bi::AdamTable<kMax>>(new (std::nothrow) bi::AdamTable<kMax>());
  if (!tab) return false;
  uint64_t blocks = 0;
  int n = 0;
  for (; at < count && n < kMax; ++at) {
    const bi_adamw_tensor& t = ts[at];
    if (t.n == 0) continue;
    const uint64_t more = static_cast<uint64_t>((t.n + bi::kAdamChunk - 1) / bi::kAdamChunk);
    if (blocks + more > 0x7fffffffull) break;
    tab->t[n] = bi::AdamTensor{t.param, t.master, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scale, t.exp_avg_sq_scale, t.n};
    tab->first[n] = static_cast<uint32_t>(blocks);
    const bool state8 = c.state_bits == 8;
    const bool wide = aligned(t.param, c.param_bf16 ? 16 : 32) && aligned(t.master, 32) &&
                      aligned(t.grad, c.grad_bf16 ? 16 : 32) && aligned(t.exp_avg, state8 ? 8 : 32) &&
                      aligned(t.exp_avg_sq, state8 ? 8 : 32);
    if (wide) tab->wide[n / 32] |= 1u << (n % 32);
    blocks += more;
    ++n;
  }
  if (n == 0) return true;
  tab->first[n] = static_cast<uint32_t>(blocks);
  tab->count = n;
  const unsigned grid = static_cast<unsigned>(blocks);
  ProfScope ps(kKAdamW, s);
  const int held = c.state_bits == 32 ? bi::kAdam32 : a.dither_m || a.dither_v ? bi::kAdam8Dither : bi::kAdam8;
#define BI_ADAM(ST, PB, MA, GB)                                                                     \
  if (held == ST && (c.param_bf16 != 0) == PB && master == MA && (c.grad_bf16 != 0) == GB) \
    bi::k_adamw<kMax, ST, PB, MA, GB><<<grid, bi::kAdamThreads, 0, s>>>(*tab, a);
#define BI_ADAM_G(ST, PB, MA) BI_ADAM(ST, PB, MA, false) BI_ADAM(ST, PB, MA, true)
#define BI_ADAM_P(ST) BI_ADAM_G(ST, false, false) BI_ADAM_G(ST, true, false) BI_ADAM_G(ST, true, true)
  BI_ADAM_P(bi::kAdam32)
  BI_ADAM_P(bi::kAdam8)
  BI_ADAM_P(bi::kAdam8Dither)
#undef BI_ADAM_P
#undef BI_ADAM_G
#undef BI_ADAM
  a.set_status = 0;
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace

extern "C" bi_status bi_adamw_step(const bi_adamw_tensor* tensors, int32_t count, const bi_adamw_cfg* cfg,
                                   const float* grad_scale, const int64_t* step_dev, int32_t* dev_status, void* stream) {
  if (!cfg || !dev_status || count < 0 || (count > 0 && !tensors)) return BI_ERR_INVALID_ARG;
  const bi_adamw_cfg c = *cfg;
  if (c.state_bits != 8 && c.state_bits != 32) return BI_ERR_INVALID_ARG;
  if ((c.param_bf16 & ~1) || (c.grad_bf16 & ~1) || c.reserved != 0) return BI_ERR_INVALID_ARG;
  if (!finite_nonneg(c.lr) || !finite_nonneg(c.eps) || !finite_nonneg(c.weight_decay)) return BI_ERR_INVALID_ARG;
  if (!(c.beta1 >= 0.0 && c.beta1 < 1.0) || !(c.beta2 >= 0.0 && c.beta2 < 1.0)) return BI_ERR_INVALID_ARG;
  if (!step_dev && c.step < 1) return BI_ERR_INVALID_ARG;
  if (!aligned(grad_scale, 4) || !aligned(step_dev, 8)) return BI_ERR_INVALID_ARG;
  bool any = false, master = false;
  for (int32_t i = 0; i < count; ++i) {
    const bi_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > (int64_t{1} << 40)) return BI_ERR_INVALID_ARG;
    if (t.n == 0) continue;  // its pointers say nothing
    if (!any) master = t.master != nullptr;
    any = true;
    if ((t.master != nullptr) != master || (master && !c.param_bf16)) return BI_ERR_INVALID_ARG;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return BI_ERR_INVALID_ARG;
    if (!aligned(t.param, c.param_bf16 ? 2 : 4) || !aligned(t.master, 4) || !aligned(t.grad, c.grad_bf16 ? 2 : 4))
      return BI_ERR_INVALID_ARG;
    if (c.state_bits == 8) {
      if (!t.exp_avg_scale || !t.exp_avg_sq_scale || !aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))
        return BI_ERR_INVALID_ARG;
    } else if (!aligned(t.exp_avg, 4) || !aligned(t.exp_avg_sq, 4)) {
      return BI_ERR_INVALID_ARG;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bi::AdamArgs a{};
  a.h.b1 = static_cast<float>(c.beta1);
  a.h.c1 = static_cast<float>(1.0 - c.beta1);
  a.h.b2 = static_cast<float>(c.beta2);
  a.h.c2 = static_cast<float>(1.0 - c.beta2);
  a.h.keep = static_cast<float>(1.0 - c.lr * c.weight_decay);
  a.h.eps = static_cast<float>(c.eps);
  if (!step_dev) {
    a.h.rate = static_cast<float>(c.lr / (1.0 - std::pow(c.beta1, static_cast<double>(c.step))));
    a.h.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(c.beta2, static_cast<double>(c.step))));
  }
  a.lr = c.lr;
  a.beta1 = c.beta1;
  a.beta2 = c.beta2;
  a.step = c.step;
  a.dither_m = c.state_bits == 8 && c.beta1 > bi::kNearestBeta1;
  a.dither_v = c.state_bits == 8 && c.beta2 > bi::kNearestBeta2;
  a.grad_scale = grad_scale;
  a.step_dev = step_dev;
  a.status = dev_status;
  a.set_status = 1;
  int32_t at = 0;
  while (at < count)
    if (!(count - at <= kSmall    ? launch<kSmall>(tensors, at, count, c, master, a, s)
          : count - at <= kMiddle ? launch<kMiddle>(tensors, at, count, c, master, a, s)
                                  : launch<kLarge>(tensors, at, count, c, master, a, s)))
      return BI_ERR_CUDA;
  if (a.set_status && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess) return BI_ERR_CUDA;
  return BI_OK;
}
