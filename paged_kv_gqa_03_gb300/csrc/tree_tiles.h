// tree_tiles.h — host side of the row-tile tensor-core kernels for a tree of
// drafted tokens (tree_tiles.cu, tree_tiles_fp8.cu): 16-bit and fp8 caches, any
// number of query rows.
#pragma once

#include "mq_decode.h"

namespace pkv {

constexpr int kTreeTileRows = 128;  // query rows of one CTA

struct TreeCut;
struct TreeTileParams {
  MqParams m;     // part_o / part_lse sized for this kernel (tree_tiles_ws_layout)
  TreeCut *cuts;  // [groups] workspace (MqWsLayout's `prefix`)
  int D;
  int RT;       // row tiles per (sequence, kv head): ceil(R / 128)
  int groups;   // ranges of the schedule; RT CTAs walk each in step
};

// Row tiles and ranges for R rows per kv head on `sms` SMs.
void tree_tiles_grid(int R, int sms, int *RT, int *groups);
// Workspace: the WsHeader at offset 0, then the fields (as MqWsLayout).
MqWsLayout tree_tiles_ws_layout(int D, int RT, int groups);
cudaError_t launch_tree_tiles(const TreeTileParams &p, int cache_dtype, int q_dtype, const CUtensorMap &tmK,
                              const CUtensorMap &tmV, cudaStream_t stream);
cudaError_t launch_tree_tiles_fp8(const TreeTileParams &p, int q_dtype, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                  cudaStream_t stream);

}  // namespace pkv
