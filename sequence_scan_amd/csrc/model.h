// Internal interface between the host layer of the model operators
// (api_model.cpp) and their gfx950 kernels (gscan.hip, vocab.hip).  Not
// installed; not part of the ABI.
#pragma once

#include "internal.h"

namespace ssm {

// ------------------------------------------------------ gated linear recurrence

constexpr int kGsSegment = 32;    // steps between two stored states
constexpr int kGsFwdTile = 128;   // steps that a workgroup holds at a time
constexpr int kGsBwdTile = 64;

struct GscanArgs {
  const void* x;            // token (b, t)'s channels at (b * seqlen + t) * x_row
  const void* r;
  const void* i;            // nullable
  int64_t x_row, r_row, i_row;
  const float* rate;        // [width], nullable
  const float* initial;     // [batch, width], nullable; the step: the state before it
  const void* dout;         // backward: of type `out`
  const float* dlast;       // backward, nullable
  const float* states_in;   // backward: the states that the forward stored
  void* out;                // forward and step; contiguous, as all outputs
  float* last;              // forward, nullable; the step: the state behind it
  float* states;            // forward, nullable
  void* dx;                 // backward
  void* dr;
  void* di;
  float* drate;             // nullable
  float* dinitial;          // nullable
  float* part;              // backward with drate: [batch, tiles, width] sums over a tile's steps, and [gscan_sum_slices, width]
  char* work;               // gscan_chain_bytes bytes (gscan_plan.h), where a sequence has more than one tile
  int64_t batch, seqlen, width;
  int32_t lerp;
  int32_t out_bf16;         // type of out and dout
};

hipError_t launch_gscan_fwd(const GscanArgs& a, DT in, hipStream_t s);
hipError_t launch_gscan_bwd(const GscanArgs& a, DT in, hipStream_t s);
hipError_t launch_gscan_step(const GscanArgs& a, DT in, hipStream_t s);

// -------------------------------------------------- losses over a vocabulary

constexpr int kVocabTile = 256;   // of rows and columns; pieces of the vocabulary are multiples of it
constexpr int64_t kVocabPieceBytes = 268435456;   // of dz at a time, or kVocabPieceLeast columns
constexpr int64_t kVocabPieceLeast = 8192;
constexpr int64_t kVocabMaxLd = int64_t{1} << 22;   // elements between rows: 256 rows stay within 2^31 bytes

struct VocabArgs {
  const uint16_t* x;        // [rows, width] bf16, rows x_row apart
  const uint16_t* w;        // [vocab, width] bf16, rows w_row apart
  int64_t x_row, w_row;
  const int64_t* index;     // [rows, top] (cross entropy: the targets, top 1)
  const float* teacher;     // [rows, top]; NULL: cross entropy
  const float* dloss;       // backward: [rows]
  const float* lse_in;      // backward: [rows]
  const float* logits_in;   // backward of distillation: [rows, top]
  float* loss;              // forward
  float* lse;
  float* logits;            // forward: [rows, top] (cross entropy: workspace)
  uint16_t* dx;             // backward, each nullable
  uint16_t* dw;
  char* work;               // vocab_fwd_bytes or vocab_bwd_bytes bytes (vocab_plan.h)
  int32_t rows, width, vocab, top;
  float scale;              // z = scale x w^T (over the temperature)
  float z_loss;
  float temperature;        // distillation
  int32_t cus;
};

hipError_t launch_vocab_fwd(const VocabArgs& a, hipStream_t s);
hipError_t launch_vocab_bwd(const VocabArgs& a, hipStream_t s);

}  // namespace ssm
