// Parameters shared by the kernels of attention over pages.
#pragma once

#include "pages_launch.h"

namespace hkv {

constexpr int kItemRows = 32;              // rows of a wave
constexpr int kPageRowsWaves = 4;
constexpr int kPageRowsThreads = kPageRowsWaves * 64;
constexpr int kPageRowsTile = 32;          // tokens
constexpr int kMaxDealtRequests = 1024;    // requests whose tiles are dealt out evenly

constexpr int kPageChunkWaves = 4;
constexpr int kPageChunkThreads = kPageChunkWaves * 64;
constexpr int kPageChunkRows = kPageChunkWaves * kItemRows;

struct PageAttendParams {
  const char* k;
  const char* v;
  int64_t page, token, head;               // bytes
  int32_t num_pages, block_tokens, n_heads;
  uint64_t block_magic;    // token / block_tokens = token * magic >> shift, token < 2^31
  int32_t block_shift;
  int32_t grouped;         // groups of 16 (fp32: 8) tokens lie in one block, their offsets below 2^31
  int32_t n_requests;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t max_len;
  int32_t max_queries;
  int32_t n_tokens;
  const char* q;
  char* out;
  int64_t q_token, q_head, o_token, o_head;
  int32_t q_heads, group;
  float* lse;
  uint32_t q_keep, q_flip; // masks of the queries' bits (Queries::load)
  float scale, cap_log2;   // ScoreScale
  const float* slopes;
  int32_t f16;             // 16-bit elements are fp16, not bf16 (the join)
  int32_t causal, window;
  const int32_t* positions;
  const int32_t* begin;
  const int32_t* prefix;
  // how the work is shared out
  int32_t ranges;          // > 0: the rows kernel deals all tiles out over this many ranges
  int32_t min_tiles;       // least tiles of a range or cut
  int32_t part_rows;       // rows per head of a partial result
  int32_t splits;          // > 0: the chunk kernel runs, cutting each item's tiles into up to so many
  uint32_t* prefix_out;    // [n_requests + 2]: first tile of each request, total, tiles per range
  int32_t* part_n;         // [n_tokens][q_heads]: cuts of each row's item
  float2* part_ml;         // reference and sum of each partial row
  float* part_o;           // its output
};

hipError_t launch_page_rows_f32(const PageAttendParams& p, dim3 grid, hipStream_t stream);
hipError_t launch_page_rows_f16(const PageAttendParams& p, dim3 grid, hipStream_t stream);
hipError_t launch_page_rows_bf16(const PageAttendParams& p, dim3 grid, hipStream_t stream);
hipError_t launch_page_chunk_f32(const PageAttendParams& p, dim3 grid, hipStream_t stream);
hipError_t launch_page_chunk_f16(const PageAttendParams& p, dim3 grid, hipStream_t stream);
hipError_t launch_page_chunk_bf16(const PageAttendParams& p, dim3 grid, hipStream_t stream);

}  // namespace hkv
