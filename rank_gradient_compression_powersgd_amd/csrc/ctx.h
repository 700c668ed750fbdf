// What the files of the C ABI share: the context, errors, and checks of arguments.
#pragma once

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <memory>
#include <string>
#include <vector>

#include "../../include/psgd.h"
#include "psgd_internal.h"

struct psgd_plan;

struct psgd_ctx {
  int device = 0;
  int rank = 0;
  std::string err;
  std::vector<hipEvent_t> events;   // tracing hook: 2 per slot, empty when off
  char* scratch = nullptr;          // device address of this device's static scratch array
  std::unique_ptr<psgd_plan> noalloc_plan;   // host side of psgd_step_noalloc's transient plan
};

namespace {

psgd_status fail(psgd_ctx* ctx, psgd_status st, const char* fmt, ...) __attribute__((format(printf, 3, 4)));
inline psgd_status fail(psgd_ctx* ctx, psgd_status st, const char* fmt, ...) {
  if (ctx) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    ctx->err = buf;
  }
  return st;
}

inline psgd_status hip_fail(psgd_ctx* ctx, hipError_t e, const char* what) {
  (void)hipGetLastError();               // reported here: the next call's launches find none
  return fail(ctx, PSGD_EHIP, "%s: %s", what, hipGetErrorString(e));
}

#define HIPCHK(ctx, expr, what)                         \
  do {                                                  \
    hipError_t e_ = (expr);                             \
    if (e_ != hipSuccess) return hip_fail(ctx, e_, what); \
  } while (0)

inline int64_t rup(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Makes a context's device current for one call and gives the caller's back.
struct DeviceGuard {
  int prev = -1;
  hipError_t err;
  explicit DeviceGuard(int device) {
    err = hipGetDevice(&prev);
    if (err == hipSuccess && prev != device) err = hipSetDevice(device);
    else prev = -1;
  }
  ~DeviceGuard() { if (prev >= 0) (void)hipSetDevice(prev); }
};

inline int grad_type(psgd_dtype dt) {
  switch (dt) {
    case PSGD_F16: return psgd::G_F16;
    case PSGD_BF16: return psgd::G_BF16;
    case PSGD_F32: return psgd::G_F32;
  }
  return 0;
}
inline int type_size(int gt) { return gt == psgd::G_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

inline psgd_status check_hparams(psgd_ctx* ctx, const psgd_adam_hparams* hp) {
  if (!hp) return fail(ctx, PSGD_EINVAL, "hyperparameters are required");
  if (!(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) || !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f))
    return fail(ctx, PSGD_EINVAL, "betas must lie in [0, 1)");
  if (!(hp->eps >= 0.0f) || !(hp->lr >= 0.0f) || !(hp->weight_decay >= 0.0f) ||
      !std::isfinite(hp->eps) || !std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay))
    return fail(ctx, PSGD_EINVAL, "lr, eps and weight_decay must be finite and >= 0");
  return PSGD_OK;
}

}  // namespace
