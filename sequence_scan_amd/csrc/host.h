// What the C-ABI host units share: the calling thread's last error, argument
// checks, and the stream-ordered workspace.
#ifndef SSMSCAN_HOST_H
#define SSMSCAN_HOST_H

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>
#include <string>

#include "../../include/ssmscan.h"
#include "internal.h"

namespace ssmhost {

inline thread_local std::string g_last_error;

inline ssm_status fail(ssm_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline ssm_status ok() {
  return SSM_OK;
}

// A failed HIP runtime call also records its error as the calling thread's
// last error, which the launchers read back after their launches.  Once a
// call has reported such a failure itself, it clears that record, so the
// failure is not reported a second time by a later, valid call.
inline ssm_status fail_hip(const char* what, long long bytes, hipError_t e) {
  (void)hipGetLastError();
  if (bytes >= 0) return fail(SSM_ERR_HIP, "%s(%lld bytes) failed: %s", what, bytes, hipGetErrorString(e));
  return fail(SSM_ERR_HIP, "%s failed: %s", what, hipGetErrorString(e));
}

// Workspace memory.  A stream-ordered allocation from a device's default pool
// goes back to the system at the next synchronisation (that pool's release
// threshold is 0), so every call that follows one maps its workspace again:
// measured on MI355X, 21 ms for the 840 MB of the Mamba-2.8B-like layer's
// backward, ten times the kernels.  The library therefore allocates from a
// pool of its own per device whose freed memory stays reserved for the next
// call (ssm_trim_workspace hands it back).  Under stream capture the
// allocation is the stream's own (hipMallocAsync): the graph then owns it.
constexpr int kMaxDevices = 64;
inline std::mutex g_pool_mu;
inline hipMemPool_t g_pool[kMaxDevices] = {};
inline bool g_pool_tried[kMaxDevices] = {};

inline int stream_device(hipStream_t s) {
  if (s != nullptr) {
    const int d = hipGetStreamDeviceId(s);
    if (d >= 0) return d;
    (void)hipGetLastError();
  }
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) {
    (void)hipGetLastError();
    return -1;
  }
  return dev;
}

// The library's pool on `dev` (created on first use), or nullptr where the
// device offers none; then workspaces come from the default pool.
inline hipMemPool_t workspace_pool(int dev, bool create) {
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_pool_mu);
  if (create && !g_pool_tried[dev]) {
    g_pool_tried[dev] = true;
    hipMemPoolProps props{};
    props.allocType = hipMemAllocationTypePinned;
    props.handleTypes = hipMemHandleTypeNone;
    props.location.type = hipMemLocationTypeDevice;
    props.location.id = dev;
    hipMemPool_t pool = nullptr;
    if (hipMemPoolCreate(&pool, &props) == hipSuccess && pool != nullptr) {
      uint64_t keep = UINT64_MAX;
      if (hipMemPoolSetAttribute(pool, hipMemPoolAttrReleaseThreshold, &keep) == hipSuccess) g_pool[dev] = pool;
      else (void)hipMemPoolDestroy(pool);
    }
    (void)hipGetLastError();
  }
  return g_pool[dev];
}

inline hipError_t ws_alloc(void** p, int64_t bytes, hipStream_t s) {
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(s, &cs) != hipSuccess) {
    (void)hipGetLastError();
    cs = hipStreamCaptureStatusNone;
  }
  if (cs == hipStreamCaptureStatusNone) {
    if (hipMemPool_t pool = workspace_pool(stream_device(s), true))
      return hipMallocFromPoolAsync(p, (size_t)bytes, pool, s);
  }
  return hipMallocAsync(p, (size_t)bytes, s);
}

struct Range {
  const char* name;
  uintptr_t lo;
  uintptr_t hi;  // exclusive
};

inline Range range(const char* name, const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{name, lo, p ? lo + static_cast<uintptr_t>(bytes) : lo};
}

inline bool overlaps(const Range& a, const Range& b) {
  if (a.lo == 0 || b.lo == 0 || a.hi == a.lo || b.hi == b.lo) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t* r) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *r = a * b;
  return true;
}

// ceil(n / parts) for n >= 0 and parts >= 1, over their whole range.
inline int64_t ceil_div(int64_t n, int64_t parts) { return n / parts + (n % parts != 0); }

inline int64_t esize(ssm_dtype t) { return t == SSM_BF16 ? 2 : 4; }

inline bool valid_dtype(ssm_dtype t) { return t == SSM_F32 || t == SSM_BF16; }

inline ssm::DT to_dt(ssm_dtype t) { return t == SSM_BF16 ? ssm::DT::BF16 : ssm::DT::F32; }

inline ssm_status check_align(const char* name, const void* p, uintptr_t bytes = 16) {
  if (p != nullptr && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0)
    return fail(SSM_ERR_UNSUPPORTED, "%s is not %d-byte aligned", name, (int)bytes);
  return SSM_OK;
}

inline int device_simds() {
  int dev = 0;
  int cus = 0;
  // without a device the planner assumes MI355X's 256 CUs; the failed query's
  // error record is cleared (see fail_hip)
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) {
    (void)hipGetLastError();
    return 1024;
  }
  return cus * 4;
}

}  // namespace ssmhost

#endif  // SSMSCAN_HOST_H
