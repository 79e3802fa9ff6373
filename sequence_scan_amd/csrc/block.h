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

// ------------------------------------------------------------ linear attention

constexpr int kLaQ = 32;            // steps per matrix chunk
constexpr int kLaBwdChunk = 2048;   // steps per time chunk of the backward, at most
constexpr int kLaSnap = 4;          // matrix chunks between two states kept for a fixed decay's gradient
constexpr int kLaSnapParts = kLaBwdChunk / kLaQ / kLaSnap;   // parts of a time chunk between them, at most
constexpr int kLaMaxDim = 128;      // dk and dv of the chunked form, multiples of 8
constexpr int kLaMaxStepDk = 256;   // dk of the single-token step, a multiple of 4

// A bf16 tensor of rows per token: head h of row (b, t) starts at
// p + (b * seqlen + t) * row + (h / share) * head.
struct LaOperand {
  const uint16_t* p;
  int64_t row;
  int32_t head;
  int32_t share;      // consecutive heads that read the same one
};

// One walk over the chunks (linattn_kernel.h): rows A, sources B, values X.
// States are [batch, nheads, dv, dk] fp32 whatever the walk's values are: value x
// and contracted column c of a head are at x * st_x + c * st_c.
struct LaWalk {
  LaOperand A, B, X, Z;
  const float* decay;         // log decay of (b, t, h): decay[b * decay_b + t * decay_t + h]
  int64_t decay_b, decay_t;
  void* out;                  // [batch, seqlen, nheads, xdim]
  const float* first;         // state that enters the walk (nullable)
  float* last;                // state that leaves it (nullable)
  const float* chunk_states;  // n_chunks > 1: [batch, n_chunks, nheads, ..], after the carry
  float* chunk_out;           // state pass: each time chunk's end state
  float* chunk_decay;         // state pass: [batch, n_chunks, nheads] summed log2 decay
  float* snaps;               // dq and dk walks, fixed decay: [batch, nheads, n_chunks, snap_slots, slices, 4096 or 8192]
  float* part;                // dq and dk walks: [slices, batch, nheads, seqlen]
  int64_t seqlen, chunk_len;
  int64_t st_x, st_c;
  int32_t n_chunks, batch, nheads;
  int32_t xdim, cdim;
  int32_t out_bf16;
  int32_t snap_slots;         // states kept within a time chunk: one less than its parts of kLaSnap matrix chunks
  float w_scale, row_scale, src_scale;
};

// The backward.  dq and dk walks write into fp32 workspaces where several heads
// share q and k (share > 1), joined by launch_la_group_sum.
struct LaBwd {
  LaWalk dq, dk, dv;
  const float* fwd_states;    // n_chunks > 1: state entering time chunk k + 1 in slot k
  const float* rev_states;    // n_chunks > 1: gradient of the state entering time chunk k in slot k
  const float* last_state;    // with dlast: the forward's last state
  const float* dlast;         // nullable
  const float* initial;       // nullable: the forward's initial state, and with it
  const float* dinitial;      // ... its gradient (left by the dk walk)
  float* ddecay;              // [batch, seqlen, nheads], or the partial sums [batch, n_chunks, nheads, 2]
  int32_t fixed_decay;
};

struct LaStep {
  const float* state;
  float* state_out;
  const void* q;
  const void* k;
  const void* v;
  const float* decay;         // of (b, h): decay[b * decay_b + h]
  int64_t decay_b;
  void* out;
  float scale;
  int32_t batch, nheads, ngroups, dk, dv;
};

// States entering every time chunk but the walk's first: the state pass and the
// carry (rev: walking back in time).
hipError_t launch_la_states(const LaWalk& a, bool rev, hipStream_t s);
hipError_t launch_la_fwd(const LaWalk& a, hipStream_t s);
// The three walks, then the decay's gradient (fixed_decay: its partial sums).
hipError_t launch_la_bwd(const LaBwd& a, hipStream_t s);
// out[row, g, d] = sum over the `share` heads of group g of in[row, g, i, d].
hipError_t launch_la_group_sum(const float* in, void* out, bool out_bf16, int64_t rows, int ngroups, int share, int dim,
                               hipStream_t s);
// out[h] = sum over n rows of in[n, h, 0] + in[n, h, 1].
hipError_t launch_la_decay_sum(const float* in, float* out, int64_t n, int nheads, hipStream_t s);
hipError_t launch_la_step(const LaStep& a, DT in, DT out, hipStream_t s);

// ------------------------------------------------------------ 4-bit products

struct Q4Args {
  const void* x;              // [m, k], rows x_row elements apart
  int64_t x_row;
  const uint8_t* codes;       // [n, k / 2], the low four bits first
  const void* scales;         // [n, k / group]
  const uint8_t* zeros;       // [n, k / group], or NULL: 8
  const float* bias;          // [n], nullable
  void* out;                  // [m, n]
  int32_t m, n, k, group;
  int32_t x_bf16, scale_bf16, out_bf16;
  int32_t cus;
  char* image;                // q4_image_bytes bytes of workspace, 16-byte aligned
  int32_t rows_per;           // set by the launcher: rows of x per workgroup
  int32_t terms;              // ... bf16 terms of x
};

int64_t q4_image_bytes(const Q4Args& a);
hipError_t launch_q4(const Q4Args& a, hipStream_t s);
// groups: n * k / group.
hipError_t launch_q4_quantize(const void* w, bool w_bf16, uint8_t* codes, void* scales, bool scale_bf16, uint8_t* zeros,
                              int64_t groups, int group, hipStream_t s);

}  // namespace ssm
