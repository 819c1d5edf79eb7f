// tree_tiles.h — host side of the row-tile tensor-core kernels for a tree of
// drafted tokens (tree_tiles.cu, tree_tiles_fp8.cu): 16-bit and fp8 caches, any
// number of query rows.
#pragma once

#include "mq_decode.h"

namespace pkv {

constexpr int kTreeTileRows = 128;  // query rows of one CTA

// A cut of the schedule that falls within this many tiles of an item's end is
// moved there: the two groups' loads differ by as many tiles (1.3 - 1.5 us each),
// and the item needs no partials and no merge.
constexpr int kSnapTiles = 4;
constexpr int kUncutTiles = 2 * kSnapTiles + 1;  // items of up to this many tiles are never cut

struct TreeCut;
struct TreeTileParams {
  MqParams m;     // part_o / part_lse sized for this kernel (tree_tiles_ws_layout)
  uint8_t *cta_status;  // WsHeader::cta_status if no item can be cut (no merge follows), else null
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
