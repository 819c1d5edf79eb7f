// tree_tiles.h — host side of the row-tile tensor-core kernels for a tree of
// drafted tokens (tree_tiles.cu, tree_tiles_fp8.cu): 16-bit and fp8 caches, any
// number of query rows.
#pragma once

#include "mq_decode.h"

namespace pkv {

constexpr int kTreeTileRows = 128;  // query rows of one CTA

// A cut of the schedule that falls within this many tiles of an item's end is
// moved there: the two groups' loads differ by as many tiles (1.3 us each), and the
// item needs no partials.  0 / 1 / 2 / 3 / 4 tiles, us: 8 x 1000, 8 heads, 19.9 / 19.5 / 23.2 /
// 22.9 / 18.9; 16 x 1000 - 4000 52.5 / 51.8 / 51.8 / 52.2 / 53.0; 24 x 512 - 2048, 32 heads, 98.8 /
// 96.2 / 96.8 / 96.9 / 97.1; 1 x 333 14.3 / 12.9 / 12.3 / 11.6 / 11.8; 64 x 500, 32 heads, 130 /
// 129 / 125 / 125 / 124.
constexpr int kSnapTiles = 4;
constexpr int kUncutTiles = 2 * kSnapTiles + 1;  // items of up to this many tiles are never cut

struct TreeCut;
struct TreeTileParams {
  MqParams m;     // part_o / part_lse sized for this kernel (tree_tiles_ws_layout)
  const void *v_cache;
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
