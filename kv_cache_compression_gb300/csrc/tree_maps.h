// Tensor maps of a tree attention's rows, for the kernels that load them by TMA.
#pragma once

#include <cuda.h>

#include "draft_internal.h"

namespace snapkv {

struct TreeMaps {
  CUtensorMap k, v, k_new, v_new;   // (the last two only where there are drafted rows)
};

// Boxes of `tile` cached rows and `fresh` drafted rows. bf16: 64 channels wide, 128-byte swizzle; 8-bit codes: whole
// rows, with the swizzle of their width. False: the driver refused.
bool tree_maps(TreeMaps* maps, const TreeJob& job, int tile, int fresh);

}  // namespace snapkv
