// Internal interface between the host layer of the block operators
// (api_block.cpp) and their gfx950 kernels (norm_add.hip, norm_gate.hip,
// linattn.hip, q4.hip).  Not installed; not part of the ABI.
#pragma once

#include "internal.h"

namespace ssm {

constexpr int kNormMaxWidth = 8192;   // channels under one norm
constexpr int kNormMaxBlocks = 1024;   // row blocks whose column sums are joined

// The add norm (one group; x, res, scale, alpha) and the gated norm (z), each
// with its backward.  Widths are per group: column d of group g is
// g * width + d.
struct NormArgs {
  const void* x;          // block output (add; backward: nullable, for dscale) or mixer output (gate)
  const void* res;        // add: residual in (nullable), backward: the stored r
  const void* z;          // gate (nullable)
  const void* dout;       // backward
  const void* dres;       // add backward: gradient at the residual stream (nullable)
  const float* w;         // nullable
  const float* bias;      // nullable
  const float* scale;     // nullable
  void* out;              // forward: out; backward: dx (nullable)
  void* res_out;          // add: r (nullable), backward: dresidual (nullable)
  void* dz;               // gate backward
  float* part;            // backward: [blocks, sums, groups * width] column sums (nullable: none wanted)
  int64_t x_stride;
  int64_t z_stride;
  int64_t rows;
  float alpha;
  float eps;
  int32_t width;          // channels under one norm
  int32_t groups;
  int32_t center;
  int32_t gate_last;
  int32_t x_bf16;         // add backward: type of x and dx
  int32_t out_bf16;       // forward: type of out
  int32_t sums;           // backward: column sums kept: 2 (dweight, dbias), 3 (and dscale)
  int32_t cus;
};

// in: type of x (forward) or dout (backward); res: type of the residual stream.
// The backwards leave column sums of norm_row_blocks(a) row blocks in a.part.
hipError_t launch_add_norm(const NormArgs& a, DT in, DT res, hipStream_t s);
hipError_t launch_add_norm_bwd(const NormArgs& a, DT in, DT res, hipStream_t s);
hipError_t launch_gated_norm(const NormArgs& a, DT in, hipStream_t s);
hipError_t launch_gated_norm_bwd(const NormArgs& a, DT in, DT dout, hipStream_t s);
// Row blocks (workgroups along the rows) of a backward over these sizes, at
// most kNormMaxBlocks.
int norm_row_blocks(const NormArgs& a);
// Joins the column sums of `blocks` row blocks in a fixed order: out[k] receives
// sum k of every column (NULL: skipped).
hipError_t launch_norm_sums(const float* part, int blocks, int sums, int64_t width, float* const out[3],
                            hipStream_t s);

}  // namespace ssm
