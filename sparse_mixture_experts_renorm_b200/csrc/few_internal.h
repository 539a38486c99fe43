// few_internal.h — the layer for a few tokens: limits, workspace and launcher
// (host-side declarations).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kFewTokens = MOE_FEW_TOKENS;  // two n8 tiles of an mma.sync step
constexpr int kFewMaxSplit = 8;                // parts of a down product's columns
constexpr int kFewTokPitch = 1024 + 64;        // bytes between token rows in shared memory and of hidden rows

// The workspace's first words: the call's status word, the plan from few_up to
// few_down, and a status word of each of few_up's blocks.
constexpr int kFewPlanAt = 4, kFewPlanWords = 764, kFewUpAt = 768, kFewUpWords = 256;

// Byte offsets inside the workspace.
struct FewWorkspace {
  size_t head;   // int32 [kFewUpAt + kFewUpWords], at 0
  size_t next;   // int32 [1] few_down's next item
  size_t done;   // int32 [blocks of 16 output columns] finished parts
  size_t h;      // hidden rows by expert and chunk of columns (few.cu, hidden_at)
  size_t y;      // fp32  [split, T*k, d] gated expert outputs
  size_t total;
  int split;     // parts that y has room for
};

struct FewArgs {
  const void *x, *wr, *wg, *wu, *wd;
  const float* br;
  int T, d, E, k, I, renorm;
  void* out;
  int32_t* idx;
  float* gate;
  int32_t* counts;  // NULL: not wanted
  float* aux;       // NULL: not wanted
  int32_t* head;
  int32_t* next;
  int32_t* done;
  void* h;
  float* y;
  int split;        // parts that y has room for
  int down_blocks;  // few_down's grid, set by the launcher
  int likely;       // nearly every expert will get tokens, set by the launcher
  // MOE_DEV_* bits go to *status. The call's own word (head[0]) is cleared by
  // few_up's first block, and no other knows when: what a wait there that gave up
  // has OR-ed in may be lost. So each block of few_up then keeps its bits in a
  // word of the head as well, and few_down, which starts when all of that is
  // done, adds them.
  int own;          // 1: the status word is the call's own; set to few_up's grid by the launcher
  int32_t* status;
  uint64_t limit_ns;
};

// Weight rows in boxes of 512 bytes: 8 rows of gate and up, 16 of down.
struct FewMaps {
  CUtensorMap wg, wu, wd;
};
bool make_tmap_few(CUtensorMap* map, const void* base, moe_dtype dtype, uint64_t rows, uint64_t cols, uint32_t box_rows);

FewWorkspace few_layout(int T, int d, int k, int I, moe_dtype dtype);
cudaError_t launch_few(moe_dtype dtype, const FewMaps& m, const FewArgs& a, cudaStream_t stream);

}  // namespace moe
