// Cuts calls of the tree attention as its launchers do (no GPU needed) and prints, per line of input, the CTAs of the grid and
// the bytes of the workspace that their parts end at. Input: batch q_heads heads head_dim tokens cap tile_q siblings tile fresh ctas.
#include <stdio.h>

#include "../kv_cache_compression_gb300/csrc/tree_schedule.cuh"
#include "../kv_cache_compression_gb300/csrc/tree_launch.h"

int main() {
  using namespace snapkv;
  TreeJob job = {};
  int tile_q, siblings, tile, fresh;
  long long cap, ctas;
  job.workspace = reinterpret_cast<void*>(4096);
  while (scanf("%d %d %d %d %d %lld %d %d %d %d %lld", &job.batch, &job.q_heads, &job.heads, &job.head_dim, &job.tokens, &cap, &tile_q, &siblings,
               &tile, &fresh, &ctas) == 11) {
    job.cap = cap;
    tree::Args a = tree_args(job, tile_q);
    a.siblings = siblings;
    if (tree_fill(a, job, tile, fresh, ctas) != cudaSuccess) return 1;
    const char* const end = reinterpret_cast<const char*>(a.parts) + (size_t)a.ctas * 2 * tile_q * (job.head_dim + 2) * sizeof(float);
    printf("%d %lld\n", a.ctas, a.direct ? 0LL : (long long)(end - static_cast<char*>(job.workspace)));
  }
  return 0;
}
