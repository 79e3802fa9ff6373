// Host-only stand-ins for the block operators' kernel launchers (block.h), linked
// with fake_runtime.cpp: each reads the first and the last byte of every buffer and
// workspace region that the host layer hands to its kernel, at the extent that the
// kernel indexes.  Nothing is computed.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>

#include "../../sequence_scan_amd/csrc/block.h"

namespace {
long g_block_launches = 0;

void touch(const char* what, const void* p, int64_t n, int64_t esize) {
  if (n <= 0) return;
  if (!p) {
    std::fprintf(stderr, "launcher got NULL %s for %lld elements\n", what, (long long)n);
    std::abort();
  }
  const volatile unsigned char* c = static_cast<const volatile unsigned char*>(p);
  (void)c[0];
  (void)c[n * esize - 1];
}
void maybe(const char* what, const void* p, int64_t n, int64_t esize) {
  if (p) touch(what, p, n, esize);
}
int64_t es(ssm::DT t) { return t == ssm::DT::F32 ? 4 : 2; }
int64_t es16(int bf16) { return bf16 ? 2 : 4; }
int64_t wide(const ssm::NormArgs& a) { return (int64_t)a.groups * a.width; }
int64_t strided(const ssm::NormArgs& a, int64_t stride) { return (a.rows - 1) * stride + wide(a); }

void norm_common(const ssm::NormArgs& a) {
  if (a.rows < 1 || a.width < 1 || a.width > ssm::kNormMaxWidth || a.groups < 1 || a.groups > 65535 || a.cus < 1) std::abort();
  maybe("weight", a.w, wide(a), 4);
  maybe("bias", a.bias, wide(a), 4);
  maybe("scale", a.scale, wide(a), 4);
  if (a.part) touch("part", a.part, (int64_t)ssm::norm_row_blocks(a) * a.sums * wide(a), 4);
  ++g_block_launches;
}

// A walk's operands and outputs, over all of its rows.
void operand(const char* what, const ssm::LaOperand& o, const ssm::LaWalk& w) {
  if (o.share < 1 || w.nheads % o.share || o.row % 8) std::abort();
  touch(what, o.p, ((int64_t)w.batch * w.seqlen - 1) * o.row + (int64_t)(w.nheads / o.share) * o.head, 2);
}
void walk(const ssm::LaWalk& a, bool out) {
  const int64_t bn = (int64_t)a.batch * a.nheads, state = bn * a.xdim * a.cdim;
  if (a.n_chunks < 1 || (int64_t)a.n_chunks * a.chunk_len < a.seqlen || (int64_t)(a.n_chunks - 1) * a.chunk_len >= a.seqlen ||
      (a.n_chunks > 1 && a.chunk_len % ssm::kLaQ) || a.xdim > ssm::kLaMaxDim || a.cdim > ssm::kLaMaxDim) {
    std::fprintf(stderr, "inconsistent walk: %d chunks of %lld for %lld steps\n", a.n_chunks, (long long)a.chunk_len,
                 (long long)a.seqlen);
    std::abort();
  }
  operand("B", a.B, a);
  operand("X", a.X, a);
  touch("decay", a.decay, (a.batch - 1) * a.decay_b + (a.seqlen - 1) * a.decay_t + a.nheads, 4);
  maybe("first", a.first, state, 4);
  if (out) {
    operand("A", a.A, a);
    touch("out", a.out, bn * a.seqlen * a.xdim, es16(a.out_bf16));
    maybe("last", a.last, state, 4);
    if (a.n_chunks > 1) touch("chunk_states", a.chunk_states, state * a.n_chunks, 4);
    if (a.part) {
      touch("part", a.part, ((a.xdim + 63) / 64) * bn * a.seqlen, 4);
      operand("Z", a.Z, a);
    }
  }
  ++g_block_launches;
}
}  // namespace

extern "C" long fake_block_launches(void) { return g_block_launches; }

namespace ssm {

int norm_row_blocks(const NormArgs& a) { return a.rows < 7 ? (int)a.rows : 7; }

hipError_t launch_add_norm(const NormArgs& a, DT in, DT res, hipStream_t) {
  touch("x", a.x, strided(a, a.x_stride), es(in));
  maybe("residual", a.res, a.rows * wide(a), es(res));
  touch("out", a.out, a.rows * wide(a), es16(a.out_bf16));
  maybe("residual_out", a.res_out, a.rows * wide(a), es(res));
  norm_common(a);
  return hipSuccess;
}

hipError_t launch_add_norm_bwd(const NormArgs& a, DT in, DT res, hipStream_t) {
  const int64_t n = a.rows * wide(a);
  touch("dout", a.dout, n, es(in));
  touch("r", a.res, n, es(res));
  maybe("dres", a.dres, n, es(res));
  maybe("dx", a.out, n, es16(a.x_bf16));
  maybe("dresidual", a.res_out, n, es(res));
  if (a.part && a.sums == 3) touch("x", a.x, strided(a, a.x_stride), es16(a.x_bf16));
  norm_common(a);
  return hipSuccess;
}

hipError_t launch_gated_norm(const NormArgs& a, DT in, hipStream_t) {
  touch("x", a.x, strided(a, a.x_stride), es(in));
  if (a.z) touch("z", a.z, strided(a, a.z_stride), es(in));
  touch("out", a.out, a.rows * wide(a), es16(a.out_bf16));
  norm_common(a);
  return hipSuccess;
}

hipError_t launch_gated_norm_bwd(const NormArgs& a, DT in, DT dout, hipStream_t) {
  touch("x", a.x, strided(a, a.x_stride), es(in));
  touch("dout", a.dout, a.rows * wide(a), es(dout));
  touch("dx", a.out, a.rows * wide(a), es(in));
  if (a.z) {
    touch("z", a.z, strided(a, a.z_stride), es(in));
    touch("dz", a.dz, a.rows * wide(a), es(in));
  }
  norm_common(a);
  return hipSuccess;
}

hipError_t launch_norm_sums(const float* part, int blocks, int sums, int64_t width, float* const out[3], hipStream_t) {
  touch("part", part, (int64_t)blocks * sums * width, 4);
  for (int k = 0; k < sums; ++k) maybe("sum", out[k], width, 4);
  ++g_block_launches;
  return hipSuccess;
}

hipError_t launch_la_states(const LaWalk& a, bool, hipStream_t) {
  if (a.n_chunks < 2) std::abort();
  const int64_t bn = (int64_t)a.batch * a.nheads;
  touch("chunk_out", a.chunk_out, bn * a.n_chunks * a.xdim * a.cdim, 4);
  touch("chunk_decay", a.chunk_decay, bn * a.n_chunks, 4);
  walk(a, false);
  return hipSuccess;
}

hipError_t launch_la_fwd(const LaWalk& a, hipStream_t) {
  walk(a, true);
  return hipSuccess;
}

hipError_t launch_la_bwd(const LaBwd& a, hipStream_t) {
  const LaWalk& q = a.dq;
  const int64_t bn = (int64_t)q.batch * q.nheads, state = bn * q.xdim * q.cdim;
  walk(a.dq, true);
  walk(a.dk, true);
  walk(a.dv, true);
  if (q.n_chunks > 1) {
    touch("fwd_states", a.fwd_states, state * q.n_chunks, 4);
    touch("rev_states", a.rev_states, state * q.n_chunks, 4);
  }
  if (a.dlast) {
    touch("dlast", a.dlast, state, 4);
    touch("last_state", a.last_state, state, 4);
  }
  if (a.initial) {
    touch("initial", a.initial, state, 4);
    touch("dinitial", a.dinitial, state, 4);
  }
  const int64_t kept = bn * q.n_chunks * q.snap_slots * ((q.xdim + 63) / 64) * (q.cdim > 64 ? 8192 : 4096);
  if (!a.fixed_decay && q.snap_slots > 0) std::abort();
  touch("dq snaps", a.dq.snaps, kept, 4);
  touch("dk snaps", a.dk.snaps, kept, 4);
  touch("ddecay", a.ddecay, a.fixed_decay ? bn * q.n_chunks * 2 : bn * q.seqlen, 4);
  return hipSuccess;
}

hipError_t launch_la_group_sum(const float* in, void* out, bool out_bf16, int64_t rows, int ngroups, int share, int dim, hipStream_t) {
  touch("in", in, rows * ngroups * share * dim, 4);
  touch("out", out, rows * ngroups * dim, es16(out_bf16));
  ++g_block_launches;
  return hipSuccess;
}

hipError_t launch_la_decay_sum(const float* in, float* out, int64_t n, int nheads, hipStream_t) {
  touch("in", in, n * nheads * 2, 4);
  touch("out", out, nheads, 4);
  ++g_block_launches;
  return hipSuccess;
}

hipError_t launch_la_step(const LaStep& a, DT in, DT out, hipStream_t) {
  const int64_t bn = (int64_t)a.batch * a.nheads;
  touch("state", a.state, bn * a.dk * a.dv, 4);
  touch("state_out", a.state_out, bn * a.dk * a.dv, 4);
  touch("q", a.q, (int64_t)a.batch * a.ngroups * a.dk, es(in));
  touch("k", a.k, (int64_t)a.batch * a.ngroups * a.dk, es(in));
  touch("v", a.v, bn * a.dv, es(in));
  touch("decay", a.decay, (a.batch - 1) * a.decay_b + a.nheads, 4);
  touch("out", a.out, bn * a.dv, es(out));
  ++g_block_launches;
  return hipSuccess;
}

int64_t q4_image_bytes(const Q4Args& a) { return a.m > 16 ? (int64_t)a.m * a.k * 2 + 4096 : 0; }

hipError_t launch_q4(const Q4Args& a, hipStream_t) {
  if (a.m < 1 || a.n < 1 || a.cus < 1) std::abort();
  const int64_t groups = (int64_t)a.n * (a.k / a.group);
  if (a.k > 0) touch("x", a.x, (a.m - 1) * a.x_row + a.k, es16(a.x_bf16));
  touch("codes", a.codes, (int64_t)a.n * a.k / 2, 1);
  touch("scales", a.scales, groups, es16(a.scale_bf16));
  maybe("zeros", a.zeros, groups, 1);
  maybe("bias", a.bias, a.n, 4);
  touch("out", a.out, (int64_t)a.m * a.n, es16(a.out_bf16));
  if (const int64_t bytes = q4_image_bytes(a)) touch("image", a.image, bytes, 1);
  ++g_block_launches;
  return hipSuccess;
}

hipError_t launch_q4_quantize(const void* w, bool w_bf16, uint8_t* codes, void* scales, bool scale_bf16, uint8_t* zeros,
                              int64_t groups, int group, hipStream_t) {
  touch("w", w, groups * group, es16(w_bf16));
  touch("codes", codes, groups * group / 2, 1);
  touch("scales", scales, groups, es16(scale_bf16));
  touch("zeros", zeros, groups, 1);
  ++g_block_launches;
  return hipSuccess;
}

}  // namespace ssm
