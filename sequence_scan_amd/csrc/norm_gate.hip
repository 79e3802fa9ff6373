// gfx950 kernels of libssmscan: the gated norm after a block's mixer
// (norm_kernel.h).
#include <algorithm>

#include "norm_kernel.h"

namespace ssm {
namespace {

template <typename Tx>
void fwd(const NormArgs& a, hipStream_t s) {
  if (a.gate_last) launch_norm_fwd_t<kModeGateLast, Tx, float>(a, s);
  else launch_norm_fwd_t<kModeGate, Tx, float>(a, s);
}
template <typename Tx, typename Td>
void bwd(const NormArgs& a, hipStream_t s) {
  if (a.gate_last) launch_norm_bwd_t<kModeGateLast, Tx, Td>(a, s);
  else launch_norm_bwd_t<kModeGate, Tx, Td>(a, s);
}

}  // namespace

hipError_t launch_gated_norm(const NormArgs& a, DT in, hipStream_t s) {
  if (in == DT::F32) fwd<float>(a, s);
  else fwd<uint16_t>(a, s);
  return hipGetLastError();
}

hipError_t launch_gated_norm_bwd(const NormArgs& a, DT in, DT dout, hipStream_t s) {
  if (in == DT::F32 && dout == DT::F32) bwd<float, float>(a, s);
  else if (in == DT::F32) bwd<float, uint16_t>(a, s);
  else if (dout == DT::F32) bwd<uint16_t, float>(a, s);
  else bwd<uint16_t, uint16_t>(a, s);
  return hipGetLastError();
}

}  // namespace ssm
