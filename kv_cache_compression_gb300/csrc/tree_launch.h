// Host side of the tree attention: how a call is cut, its workspace, and its launchers.
#pragma once

#include "draft_internal.h"

namespace snapkv {

namespace tree {
struct Args;
}

constexpr int kMaxTreeCtas = 320;     // of a first launch, at most (whatever the device's SM count): bounds the workspace
constexpr int kMaxTcCtas = 160;       // the same for the kernel whose passes have up to 256 rows
constexpr int kSimtRows = 32;         // query rows of a pass, at most

// The call's arguments, for passes of `tile_q` query rows.
tree::Args tree_args(const TreeJob& job, int tile_q);
// Cuts the call for at most `ctas` CTAs of one wave with tiles of `tile` cached and `fresh` drafted rows, and lays out
// its workspace, whose parts bound the grid.
cudaError_t tree_fill(tree::Args& a, const TreeJob& job, int tile, int fresh, int64_t ctas);

cudaError_t launch_tree_simt(const TreeJob& job);   // fp32 instructions: fp32 calls
cudaError_t launch_tree_mma(const TreeJob& job);    // mma.sync: bf16 calls of few query rows a KV head
cudaError_t launch_tree_tc(const TreeJob& job);     // tcgen05: bf16 calls of more

}  // namespace snapkv
