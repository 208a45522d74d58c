// How the work of an attention call over pages is shared out (host code):
// which kernel, ranges of tiles, cuts.
#pragma once

#include "attend_pages_launch.h"

namespace hkv {

struct PageShare {
  int splits;              // > 0: the chunk kernel
  int ranges, min_tiles, part_rows;
  int64_t rows;            // partial rows in all
  int64_t items;           // of one request, at most
};

inline PageShare page_share_of(const Geometry& g, const hkv_requests& req, int32_t n_tokens,
                               int32_t n_q_heads, int dtype) {
  PageShare s = {};
  const int64_t queries = req.max_queries < n_tokens ? req.max_queries : n_tokens;
  const int64_t group = n_q_heads / g.n_heads;
  const int64_t rows = queries * group;
  const int64_t max_len = static_cast<int64_t>(req.max_blocks) * g.block_tokens;
  // Where requests have fewer rows on average than one of the chunk kernel's
  // workgroups, most of its workgroups would hold little: up to where the
  // join's workgroups, one for every row that a request might have, cost what
  // that spares, such steps take the rows kernel.
  const bool sparse = static_cast<int64_t>(n_tokens) * group < static_cast<int64_t>(kPageChunkRows) * req.n_requests &&
                      queries * n_q_heads * req.n_requests <= (1 << 19);
  if (rows > 128 && !sparse) {
    // One workgroup per 256 rows and key head; their tiles are cut where
    // these are too few for the CUs.
    s.items = (rows + kPageChunkRows - 1) / kPageChunkRows;
    int64_t most = static_cast<int64_t>(n_tokens) * group / kPageChunkRows + req.n_requests;
    const int64_t all = req.n_requests * s.items;
    most = (most < all ? most : all) * g.n_heads;
    const int64_t cuts = 256 / (most < 1 ? 1 : most);
    const int64_t long_enough = max_len / 512;
    s.splits = static_cast<int>(cuts < long_enough ? cuts : long_enough);
    s.splits = s.splits < 1 ? 1 : s.splits;
    s.rows = s.splits > 1 ? static_cast<int64_t>(s.splits) * n_tokens * n_q_heads : 0;
    return s;
  }
  const int64_t tiles = max_len < kPageRowsTile ? 1 : (max_len + kPageRowsTile - 1) / kPageRowsTile;
  s.items = (rows + kItemRows - 1) / kItemRows;
  s.min_tiles = kPageRowsWaves;
  s.part_rows = static_cast<int>(rows < kItemRows ? rows : kItemRows);
  const int64_t all = static_cast<int64_t>(req.n_requests) * s.items * tiles;
  // Requests of few tiles keep them to one workgroup per head and spare the
  // join, unless there are too few of them to keep more than a few CUs at work.
  const int64_t few = static_cast<int64_t>(req.n_requests) * g.n_heads >= 32 ? 32 : 16;
  if (req.n_requests <= kMaxDealtRequests && tiles > few && queries * n_q_heads <= (1 << 20) &&
      all < (int64_t{1} << 30)) {
    int64_t ranges = 512 / g.n_heads;
    const int64_t most = (all + s.min_tiles - 1) / s.min_tiles;
    ranges = ranges < 1 ? 1 : ranges;
    s.ranges = static_cast<int>(ranges < most ? ranges : most);
  }
  s.rows = static_cast<int64_t>(s.ranges) * 2 * g.n_heads * s.part_rows;
  (void)dtype;
  return s;
}

inline int64_t page_prefix_bytes(const hkv_requests& req) {
  return (static_cast<int64_t>(req.n_requests + 2) * 4 + 15) / 16 * 16;
}

inline int64_t page_share_bytes(const PageShare& s, const hkv_requests& req) {
  return s.rows > 0 ? page_prefix_bytes(req) + (s.rows * 8 + 15) / 16 * 16 + s.rows * HKV_HEAD_DIM * 4 : 0;
}

}  // namespace hkv
