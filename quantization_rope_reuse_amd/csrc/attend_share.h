// How the work of an attention call is shared out (host code): which kernel,
// heads and rows of a workgroup, ranges of tokens.
#pragma once

#include "attend_launch.h"

namespace hkv {

struct Share {
  int splits;              // > 0: the prompt kernel
  int hp, nt;              // heads per score tile, tiles of 16 rows: 16 nt / hp rows per item
  int set_heads, head_sets, ranges, min_tiles, part_rows;
  int64_t rows;            // partial rows in all
  int64_t items;           // of one request, at most
};

// How a call's work is shared out, from the sizes that the host knows.
inline Share share_of(int fmt, bool moved, const Geometry& g, const hkv_requests& req,
                      int32_t n_tokens, int32_t n_q_heads, int dtype) {
  Share s = {};
  const int64_t queries = req.max_queries < n_tokens ? req.max_queries : n_tokens;
  const int64_t rows = queries * (n_q_heads / g.n_heads);
  s.splits = 0;
  // The prompt kernel makes operands of codes once for 256 rows, the rows
  // kernel for 32; but its eight waves wait for each other every 64 tokens, and
  // a workgroup works as long on one row as on 256.  Of 32 query and 8 key
  // heads over INT4 in bf16, rows against prompt kernel in us: one request
  // behind 8,192 tokens, 50 queries 45 against 52, 100 queries 58 against 57,
  // 400 129 against 135, 1,000 289 against 265 (fp32 659 against 531); four
  // requests of 100 137 against 139 (FP8 168 against 139); eight first prompts
  // of 256 53 against 32, one 14 against 26: even where it is level from 400
  // rows on, the prompt kernel wins where it fills the CUs.
  // Where requests have fewer rows on average than one of its workgroups,
  // most of its workgroups hold little: 31 decodes of up to 8,192 tokens beside
  // a prompt of 100 queries 90 against 492, of 512 226 against 873, 128 decodes
  // of up to 2,048 called with 128 for the most queries 176 against 536.  Up to
  // where the join's workgroups, one for every row that a request might have,
  // cost what that spares (2^19 some 120 us).
  const bool sparse = static_cast<int64_t>(n_tokens) * (n_q_heads / g.n_heads) <
                          static_cast<int64_t>(kPromptRows) * req.n_requests &&
                      queries * n_q_heads * req.n_requests <= (1 << 19);
  if (rows > 384 && !sparse) {
    // One workgroup per 256 rows and key head; their tokens are cut where
    // these are too few for the CUs.
    s.items = (rows + kPromptRows - 1) / kPromptRows;
    int64_t most = static_cast<int64_t>(n_tokens) * (n_q_heads / g.n_heads) / kPromptRows + req.n_requests;
    const int64_t all = req.n_requests * s.items;
    most = (most < all ? most : all) * g.n_heads;
    const int64_t cuts = 256 / (most < 1 ? 1 : most);
    const int64_t long_enough = static_cast<int64_t>(req.max_blocks) * g.block_tokens / 512;
    s.splits = static_cast<int>(cuts < long_enough ? cuts : long_enough);
    s.splits = s.splits < 1 ? 1 : s.splits;
    s.hp = s.nt = 1;
    s.rows = s.splits > 1 ? static_cast<int64_t>(s.splits) * n_tokens * n_q_heads : 0;
    return s;
  }
  s.nt = dtype == HKV_F32 || moved || rows <= 16 ? 1 : 2;
  const int64_t max_len = static_cast<int64_t>(req.max_blocks) * g.block_tokens;
  const int64_t tiles = max_len < kTileTokens ? 1 : (max_len + kTileTokens - 1) / kTileTokens;
  // Two heads of at most 8 rows share a score tile, which halves the softmax
  // and the bookkeeping of each; and two INT4 heads of a token share a
  // 128-byte line, so one workgroup reads both.  Short work goes faster with
  // a workgroup for every head (one request of 777 tokens 11.6 against 12.4
  // us, of 3,000 12.6 against 12.9, of 8,000 16.9 against 15.1; 16 requests of
  // up to 1,000 16.4 against 20.5; 32 query and 8 key heads).
  const int64_t work = static_cast<int64_t>(req.n_requests) * g.n_heads * tiles;
  const bool paired = g.n_heads % 2 == 0 && (tiles > 32 ? work > 1024 : work > 8192);
  s.hp = paired && rows <= 8 ? 2 : 1;
  const int64_t item_rows = 16 * s.nt / s.hp;
  s.items = (rows + item_rows - 1) / item_rows;
  s.set_heads = s.hp == 1 && paired && fmt == HKV_INT4 ? 2 : 1;
  s.head_sets = g.n_heads / (s.set_heads * s.hp);
  const int64_t phases = kRowsWaves / s.set_heads;
  s.ranges = 0;
  s.min_tiles = static_cast<int>(phases);
  s.part_rows = static_cast<int>(rows < item_rows ? rows : item_rows);
  const int64_t all = static_cast<int64_t>(req.n_requests) * s.items * tiles;
  // Requests of few tiles keep them to one workgroup per head and spare the
  // join (16 requests of up to 1,000 tokens: 16.4 against 22.2 us), unless
  // there are too few of them to keep more than a few CUs at work (one request
  // of 777: 14.0 against 11.6).
  const int64_t few = static_cast<int64_t>(req.n_requests) * g.n_heads >= 32 ? 32 : 16;
  if (req.n_requests <= kMaxFlatRequests && tiles > few && queries * n_q_heads <= (1 << 20) &&
      all < (int64_t{1} << 30)) {
    int64_t ranges = 512 / s.head_sets;
    const int64_t most = (all + s.min_tiles - 1) / s.min_tiles;
    ranges = ranges < 1 ? 1 : ranges;
    s.ranges = static_cast<int>(ranges < most ? ranges : most);
  }
  s.rows = static_cast<int64_t>(s.ranges) * 2 * g.n_heads * s.part_rows;
  return s;
}

inline int64_t prefix_bytes(const hkv_requests& req) {
  return (static_cast<int64_t>(req.n_requests + 2) * 4 + 15) / 16 * 16;
}

inline int64_t share_bytes(const Share& s, const hkv_requests& req) {
  return s.rows > 0 ? prefix_bytes(req) + (s.rows * 8 + 15) / 16 * 16 + s.rows * HKV_HEAD_DIM * 4 : 0;
}

}  // namespace hkv
