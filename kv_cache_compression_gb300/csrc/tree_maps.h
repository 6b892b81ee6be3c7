// Tensor maps of a tree attention's rows, for the kernels that load them by TMA.
#pragma once

#include <cuda.h>

#include "draft_internal.h"

namespace snapkv {

struct TreeMaps {
  CUtensorMap k, v, k_new, v_new;   // (the last two only where there are drafted rows)
  CUtensorMap q;                    // all query rows of a bf16 call as one list
};

// Boxes of `tile` cached rows, `fresh` drafted rows and `tile` query rows. bf16: 64 channels wide, 128-byte swizzle; 8-bit codes: whole
// rows, with the swizzle of their width. False: the driver refused.
bool tree_maps(TreeMaps* maps, const TreeJob& job, int tile, int fresh);

}  // namespace snapkv
