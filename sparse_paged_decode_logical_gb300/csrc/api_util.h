// What the entry points that are not of the sparse path share: the device of a call, and the
// checks and constants of a score rule.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "dense.h"
#include "spd.h"

namespace spd {

// The device of a pointer made current for a call, the caller's afterwards.
class DeviceGuard {
 public:
  spd_status bind(int device) {
    if (cudaGetDevice(&prev_) != cudaSuccess) return SPD_ERR_CUDA;
    if (prev_ != device) {
      if (cudaSetDevice(device) != cudaSuccess) return SPD_ERR_CUDA;
      moved_ = true;
    }
    return SPD_OK;
  }
  ~DeviceGuard() {
    if (moved_) (void)cudaSetDevice(prev_);
  }

 private:
  int prev_ = -1;
  bool moved_ = false;
};

inline bool device_of(const void *p, int *device) {
  cudaPointerAttributes a{};
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess ||
      (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)) {
    (void)cudaGetLastError();
    return false;
  }
  *device = a.device;
  return true;
}

inline int sm_count(int device) {
  static std::atomic<int> known[64];
  const bool keep = device >= 0 && device < 64;
  int n = keep ? known[device].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return 152;
  }
  if (keep) known[device].store(n, std::memory_order_relaxed);
  return n;
}

inline const char *check_rule(const spd_score_rule *r) {
  if (!r) return nullptr;
  // (between the bounds every constant of the rule is an ordinary fp32 number)
  if (r->scale != 0.f && !(r->scale >= 1e-6f && r->scale <= 1e6f))
    return "scale must be 0 or in [1e-6, 1e6]";
  if (r->softcap != 0.f && !(r->softcap >= 1e-6f && r->softcap <= 1e6f))
    return "softcap must be 0 or in [1e-6, 1e6]";
  if (r->slopes && reinterpret_cast<uintptr_t>(r->slopes) % 4) return "slopes must be 4-byte aligned";
  return nullptr;
}

inline ScoreRule make_rule(const spd_score_rule *r, int d) {
  constexpr double kLog2e = 1.4426950408889634;
  ScoreRule x{};
  const double scale = r && r->scale > 0.f ? (double)r->scale : 1.0 / std::sqrt((double)d);
  x.scale_log2 = (float)(scale * kLog2e);
  if (r && r->softcap > 0.f) {
    x.z_in = (float)(scale / r->softcap);
    x.e_in = (float)(2.0 * kLog2e * scale / r->softcap);
    x.small = (float)(0.5999 * r->softcap / scale);
    x.cap_out = (float)(kLog2e * r->softcap);
    // tanh(z) / z in z^2, |z| <= 0.6 (dense_math.cuh)
    constexpr double kTanh[5] = {0.9999999403953552, -0.33332309126853943, 0.13310173153877258,
                                 -0.05210147798061371, 0.01547542680054903};
    for (int i = 0; i < 5; ++i) x.poly[i] = (float)(kLog2e * r->softcap * kTanh[i]);
  }
  x.slopes = r ? r->slopes : nullptr;
  x.rough = x.cap_out <= 256.f;
  if (x.cap_out > 0.f && r->softcap >= 30.f && !x.slopes && x.z_in > 1e-4f && x.z_in < 1e4f) {
    // (z_in^8 fits fp32)
    // tanh(z) / z in z^2, |z| <= 0.75, times scale log2(e) and in (q.k)^2
    constexpr double kTanh[5] = {0.999999463558197, -0.3332825005054474, 0.13258983194828033,
                                 -0.050056301057338715, 0.01292963046580553};
    double f = scale * kLog2e;
    const double z2 = scale / r->softcap * (scale / r->softcap);
    for (int i = 0; i < 5; ++i, f *= z2) x.quick_poly[i] = (float)(f * kTanh[i]);
    x.quick = (float)(0.7499 * r->softcap / scale);
    x.quick_floor = (float)(-0.25 * r->softcap / scale);
  }
  return x;
}

}  // namespace spd
