// How the work of an attention call over pages is shared out (host code):
// which kernel, ranges of tiles, cuts.  (Times: 32 query heads, 8 key heads,
// bf16.)
#pragma once

#include "attend_pages_launch.h"

namespace hkv {

struct PageShare {
  int splits;              // > 0: the chunk kernel
  int ranges, min_tiles, part_rows;
  int64_t rows;            // partial rows in all
  int64_t items;           // of one request, at most
  int64_t index_bytes;     // of the workspace's first part
};

// slanted: the rows see very different numbers of tokens.
inline PageShare page_share_of(const Geometry& g, const hkv_requests& req, int32_t n_tokens,
                               int32_t n_q_heads, bool slanted) {
  PageShare s = {};
  const int64_t queries = req.max_queries < n_tokens ? req.max_queries : n_tokens;
  const int64_t group = n_q_heads / g.n_heads;
  const int64_t rows = queries * group;
  const int64_t all_rows = n_tokens * group;
  const int64_t max_len = static_cast<int64_t>(req.max_blocks) * g.block_tokens;
  // The rows kernel where requests have few rows on average: 16 requests over
  // 2,000 tokens with 8 queries (32 rows, one item) each take 33 us by it and 37 by
  // the chunk kernel, with 12 queries 43 and 37, 16 44 and 38, 40 110 and 55.
  // (Between 33 and 63 rows, which it takes for its weights of two parts, it is the
  // slower one.)  Also where the step as a whole is small, up to 256 rows a request:
  // 4 requests over 600 tokens with 40 queries each 17.5 and 21.6, but 16 of them,
  // not small any more, 36 and 25.  Both up to where the join's lanes, 16 for every
  // row that a request might have, cost what that spares.
  const bool few_rows = all_rows < int64_t{64} * req.n_requests;
  const bool small = all_rows < int64_t{256} * req.n_requests && max_len <= 1024 &&
                     all_rows * g.n_heads * max_len < 10'000'000;
  if (rows >= 64 && !((few_rows || small) && queries * n_q_heads * req.n_requests <= (1 << 19))) {
    // Two workgroups fit a CU.  Where the items, 128 rows of a key head each, are
    // too few for all CUs, their tiles are cut: 400 queries over 8,192 tokens take
    // 95 us with cuts for 512 workgroups, 112 with those for 256.  Where some rows
    // see far more than others, into twice as many, so that the short ones fill
    // up, unless the cuts would be shorter than 2,048 tokens: 1,229 of 8,192
    // tokens in the order of their positions, capped, take 175 us (254 uncut), a prompt
    // of 2,048 tokens 62, and 83 if it is cut in two.
    s.items = (rows + kPageChunkRows - 1) / kPageChunkRows;
    int64_t most = all_rows / kPageChunkRows + req.n_requests;
    const int64_t all = req.n_requests * s.items;
    most = (most < all ? most : all) * g.n_heads;
    most = most < 1 ? 1 : most;
    const int64_t cuts = (slanted ? 1024 : 512) / most;
    const int64_t long_enough = max_len / (slanted ? 2048 : 512);
    s.min_tiles = 8;
    s.splits = static_cast<int>(cuts < long_enough ? cuts : long_enough);
    s.splits = s.splits < 1 ? 1 : s.splits;
    if (s.splits > 1) {
      s.rows = static_cast<int64_t>(s.splits) * n_tokens * n_q_heads;
      s.index_bytes = (static_cast<int64_t>(n_tokens) * n_q_heads * 4 + 15) / 16 * 16;
    }
    return s;
  }
  const int64_t tiles = max_len < kPageRowsTile ? 1 : (max_len + kPageRowsTile - 1) / kPageRowsTile;
  const int64_t turns = (tiles + kPageRowsWaves - 1) / kPageRowsWaves;     // of a workgroup's waves
  s.items = (rows + kItemRows - 1) / kItemRows;
  s.min_tiles = kPageRowsWaves;
  s.part_rows = static_cast<int>(rows < kItemRows ? rows : kItemRows);
  const int64_t all = static_cast<int64_t>(req.n_requests) * s.items * turns * kPageRowsWaves;
  // Items of few tiles keep them to one workgroup and spare the join, unless
  // there are too few items to keep more than a few CUs at work: 64 requests over
  // up to 1,000 tokens take 34 us so and 50 with ranges, 8 over 777 21.8 and 23.6, 4
  // 21.9 and 17.4, one 21.5 and 17.1.
  const int64_t few = static_cast<int64_t>(req.n_requests) * s.items * g.n_heads >= 64 ? 32 : 16;
  if (req.n_requests <= kMaxDealtRequests && tiles > few && queries * n_q_heads <= (1 << 20) &&
      all < (int64_t{1} << 30)) {
    // One workgroup per CU: 512 instead of 256 take 117 us for 110 (32 requests of
    // up to 8,192 tokens, 64 query heads), 87 for 74 (16 of up to 4,096, 5 queries
    // each, fp32).
    int64_t ranges = 256 / g.n_heads;
    const int64_t most = (all + s.min_tiles - 1) / s.min_tiles;
    ranges = ranges < 1 ? 1 : ranges;
    s.ranges = static_cast<int>(ranges < most ? ranges : most);
  }
  s.rows = static_cast<int64_t>(s.ranges) * 2 * g.n_heads * s.part_rows;
  s.index_bytes = (static_cast<int64_t>(req.n_requests + 2) * 4 + 15) / 16 * 16;
  return s;
}

// How many lane groups of the join share a row: about two of its partial results
// each, or four where there are many rows (one request over 4,000 tokens takes
// 18 us in all, 31 with one group a row; 1,229 picked rows of 8,192 tokens, capped,
// 175, 180 with two results each).
constexpr int kJoinMostSets = 16;
inline int page_join_sets(const PageShare& s, int32_t n_requests) {
  const int64_t parts = s.splits > 0 ? s.splits : s.items > 0 ? s.ranges / (n_requests * s.items) : 0;
  const int64_t each = s.splits > 0 ? 4 : 2;
  int sets = 1;
  while (sets < kJoinMostSets && sets * each < parts) sets *= 2;
  return sets;
}

inline int64_t page_share_bytes(const PageShare& s) {
  return s.rows > 0 ? s.index_bytes + (s.rows * 8 + 15) / 16 * 16 + s.rows * HKV_HEAD_DIM * 4 : 0;
}

}  // namespace hkv
