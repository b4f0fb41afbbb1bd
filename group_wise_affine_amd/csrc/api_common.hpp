// Shared by the files that implement the C ABI: the error message, pointer and
// stream checks, and the order of calls that share the library's scratch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>
#include <limits>
#include <mutex>

#include "../../include/libqmm.h"

namespace qmm_api {

inline thread_local char g_err[512] = "";

inline qmm_status fail(qmm_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline size_t elem_bytes(qmm_dtype dt) { return dt == QMM_F32 ? 4 : 2; }

// the stream (NULL: the current device's default stream) belongs to the
// current device, whose memory and static scratch the launch will use
inline qmm_status check_stream(const char* tag, void* stream) {
  if (!stream) return QMM_OK;
  int cur = -1;
  hipDevice_t sd = -1;
  if (hipGetDevice(&cur) != hipSuccess)
    return fail(QMM_E_LAUNCH, "%s: no current HIP device", tag);
  if (hipStreamGetDevice(static_cast<hipStream_t>(stream), &sd) != hipSuccess)
    return fail(QMM_E_ARG, "%s: stream is not a valid HIP stream", tag);
  if ((int)sd != cur)
    return fail(QMM_E_ARG, "%s: stream belongs to device %d, the current device is %d", tag,
                (int)sd, cur);
  return QMM_OK;
}

inline qmm_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess)
    return fail(QMM_E_LAUNCH, "%s: launch failed: %s", what,
                hipGetErrorString(e));
  g_err[0] = 0;
  return QMM_OK;
}

inline constexpr int64_t kI32 = std::numeric_limits<int32_t>::max();

// Calls whose kernels may use the device's static scratch (the split-K
// workspace, the tile counters, the MFMA GEMV's partial tiles and counters)
// are ordered across streams: a call queued on another stream than the
// previous such call on the device first waits for that call's work (one
// event per device, recorded after each call's launches), so calls from
// different streams or host threads do not race on the scratch. During
// stream capture nothing is waited for or recorded: a capturing caller
// orders its own work.
inline constexpr int kMaxDev = 64;
inline std::recursive_mutex g_ord_mu;
inline hipEvent_t g_ord_ev[kMaxDev] = {};
inline hipStream_t g_ord_st[kMaxDev] = {};
inline bool g_ord_used[kMaxDev] = {};

class ScratchOrder {
 public:
  // uses_scratch false: the call's kernels touch no scratch (the streaming
  // GEMV), so it neither waits nor records
  explicit ScratchOrder(void* stream, bool uses_scratch = true)
      : st_(static_cast<hipStream_t>(stream)) {
    if (!uses_scratch) return;
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(st_, &cs) != hipSuccess || cs != hipStreamCaptureStatusNone) return;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDev) return;
    g_ord_mu.lock();   // held until the launches are queued
    dev_ = dev;
    if (!g_ord_ev[dev] && hipEventCreateWithFlags(&g_ord_ev[dev], hipEventDisableTiming) != hipSuccess)
      g_ord_ev[dev] = nullptr;
    if (g_ord_ev[dev] && g_ord_used[dev] && g_ord_st[dev] != st_)
      (void)hipStreamWaitEvent(st_, g_ord_ev[dev], 0);
  }
  ~ScratchOrder() {
    if (dev_ < 0) return;
    if (g_ord_ev[dev_] && hipEventRecord(g_ord_ev[dev_], st_) == hipSuccess) {
      g_ord_st[dev_] = st_;
      g_ord_used[dev_] = true;
    }
    g_ord_mu.unlock();
  }
  ScratchOrder(const ScratchOrder&) = delete;
  ScratchOrder& operator=(const ScratchOrder&) = delete;

 private:
  hipStream_t st_;
  int dev_ = -1;
};

}  // namespace qmm_api
