// What the host units of the block and model operators (api_block.cpp,
// api_model.cpp) share: checks of tensors, and workspaces that the caller may offer.
#ifndef SSMSCAN_HOST_BLOCK_H
#define SSMSCAN_HOST_BLOCK_H

#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "host.h"

namespace ssmhost {

struct Arg {
  const char* name;
  const void* p;
  int64_t bytes;     // extent that the kernels touch
  int64_t align;     // the element's size, or what vector accesses need
  bool required;
};

// Required pointers, alignment, and outputs that overlap an input or each
// other.  `same` lists pairs (output, input) that may be one buffer.
struct Same {
  const char* out;
  const char* in;
};
inline ssm_status check_args(std::initializer_list<Arg> ins, std::initializer_list<Arg> outs,
                             std::initializer_list<Same> same = {}) {
  ssm_status st;
  for (const auto* list : {&ins, &outs})
    for (const Arg& a : *list) {
      if (a.required && a.p == nullptr && a.bytes > 0)
        return fail(SSM_ERR_NULL_ARG, "required pointer %s is NULL", a.name);
      if ((st = check_align(a.name, a.p, (uintptr_t)a.align)) != SSM_OK) return st;
    }
  for (const Arg& o : outs) {
    const Range ro = range(o.name, o.p, o.bytes);
    for (const Arg& i : ins) {
      bool allowed = false;
      for (const Same& s : same)
        allowed |= o.p == i.p && o.bytes == i.bytes && std::strcmp(s.out, o.name) == 0 && std::strcmp(s.in, i.name) == 0;
      if (!allowed && overlaps(ro, range(i.name, i.p, i.bytes)))
        return fail(SSM_ERR_UNSUPPORTED, "%s overlaps input %s", o.name, i.name);
    }
    for (const Arg& q : outs)
      if (&q != &o && overlaps(ro, range(q.name, q.p, q.bytes)))
        return fail(SSM_ERR_UNSUPPORTED, "%s overlaps %s", o.name, q.name);
  }
  return SSM_OK;
}

// The memory that the calling thread offered for its next call (ssm_workspace),
// and the bytes that its last call wanted.
struct Offer {
  void* p;
  int64_t bytes;
};
inline thread_local Offer g_offer{nullptr, 0};
inline thread_local int64_t g_wanted = 0;

// A call's workspace: the offered memory, where it is large enough, or memory of
// the library's pool.  An offer is for one call, whatever comes of it.
class Workspace {
 public:
  Workspace() : offer_(g_offer) {
    g_offer = Offer{nullptr, 0};
    g_wanted = 0;
  }
  hipError_t get(void** p, int64_t bytes, hipStream_t s) {
    g_wanted = bytes;
    if (offer_.p != nullptr && bytes <= offer_.bytes) {
      *p = offer_.p;
      return hipSuccess;
    }
    const hipError_t e = ws_alloc(&own_, bytes, s);
    *p = own_;
    return e;
  }
  // After the call's launches: their status, or that of the release.
  hipError_t done(hipError_t launched, hipStream_t s) {
    if (own_ == nullptr) return launched;
    const hipError_t e = hipFreeAsync(own_, s);
    own_ = nullptr;
    return launched == hipSuccess ? e : launched;
  }

 private:
  Offer offer_;
  void* own_ = nullptr;
};

// A grid dimension holds fewer than 2^32 threads.
constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1024;

// Consecutive pieces of one workspace, each 16-byte aligned.
struct Pieces {
  int64_t floats = 0;
  bool fits = true;
  int64_t add(int64_t n) {
    const int64_t at = floats;
    if (n < 0 || n > (INT64_MAX / 4 - 4) - floats) fits = false;
    else floats += (n + 3) / 4 * 4;
    return at;
  }
};

}  // namespace ssmhost

#endif  // SSMSCAN_HOST_BLOCK_H
