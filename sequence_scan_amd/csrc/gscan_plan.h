// How the gated linear recurrence is cut into strips and tiles, and where its chain lies
// in the workspace.  No code for the device.
#ifndef SSMSCAN_GSCAN_PLAN_H
#define SSMSCAN_GSCAN_PLAN_H

#include <algorithm>
#include <cstdint>

#include "model.h"

namespace ssm {

struct Chain {
  uint64_t* parts;       // [strips][tiles][channels] (P, H)
  uint32_t* states;      // [strips][groups][channels]: the state that enters a group
  uint32_t* next;        // tiles handed out
  int32_t tiles, groups, strips;
  int32_t group;         // tiles of a group
  int32_t waves;         // wavefronts of a strip: all of a workgroup, or where one tile is enough and its sequence
                         // short a power of two of them, and the others of the workgroup the next strips
};
constexpr int kGsWaves = 8;       // of a workgroup

// Tiles of a group: few leave less to read of the tiles before, many make fewer hops along
// the chain.  Where workgroups are many, the hops hide behind them (us, with outputs stored
// through the caches):
//   8 x 2048 x 5120 (16 tiles): groups of 2 147.8, 4 147.2, 8 149.4
//   1 x 65537 x 2560 (513 tiles, 10260 workgroups): 8 200.9, 12 204.4, 16 208.9
//   1 x 60000 x 256, forward and back (469 and 938 tiles, 938 and 1876 workgroups): 8 155.7, 12 133.4, 16 126.8, 32 128.5
inline int group_of(int tiles, int strips) { return tiles <= 32 ? 4 : (int64_t)tiles * strips > 2048 ? 8 : 16; }

struct Layout {
  Chain c;
  int ch;
  int64_t blocks;    // workgroups
  int64_t bytes;     // of the chain's workspace
};
inline Layout gscan_layout(int64_t batch, int64_t seqlen, int64_t width, int64_t steps, int ch, char* work) {
  Layout l{};
  l.ch = ch;
  const int64_t each = 64 * ch;
  l.c.strips = (int32_t)(batch * ((width + each - 1) / each));
  l.c.tiles = (int32_t)((seqlen + steps - 1) / steps);
  l.c.group = group_of(l.c.tiles, l.c.strips);
  l.c.groups = (l.c.tiles + l.c.group - 1) / l.c.group;
  // Strips side by side where a sequence leaves wavefronts idle (us, one strip to a workgroup
  // and several: 4096 x 8 x 512 277 / 42, 2048 x 16 x 1024 287 / 59, 512 x 64 x 1024 83 / 57;
  // forward and back 607 / 115, 614 / 169, 188 / 163).
  l.c.waves = kGsWaves;
  while (l.c.tiles == 1 && l.c.waves > 1 && seqlen <= steps / kGsWaves * (l.c.waves / 2)) l.c.waves /= 2;
  const int64_t at_once = kGsWaves / l.c.waves;
  l.blocks = (l.c.strips + at_once - 1) / at_once * l.c.tiles;
  if (l.c.tiles > 1) {
    const int64_t parts = (int64_t)l.c.strips * l.c.tiles * each * 8, states = (int64_t)l.c.strips * l.c.groups * each * 4;
    l.c.parts = reinterpret_cast<uint64_t*>(work);
    l.c.states = reinterpret_cast<uint32_t*>(work + parts);
    l.c.next = reinterpret_cast<uint32_t*>(work + parts + states);
    l.bytes = parts + states + 16;
  }
  return l;
}

// Bytes of GscanArgs::work (0: none), a multiple of 16.
inline int64_t gscan_chain_bytes(int64_t batch, int64_t seqlen, int64_t width, bool backward) {
  // (strips of single channels are as many or more bytes than those of two)
  const int64_t steps = backward ? kGsBwdTile : kGsFwdTile;
  return std::max(gscan_layout(batch, seqlen, width, steps, 1, nullptr).bytes, gscan_layout(batch, seqlen, width, steps, 2, nullptr).bytes);
}

// Slices in which many rows of drate's sums are added first (1: all at once).
inline int64_t gscan_sum_slices(int64_t rows) { return rows < 2048 ? 1 : std::min<int64_t>(rows / 128, 64); }

}  // namespace ssm

#endif  // SSMSCAN_GSCAN_PLAN_H
