// Parameters shared by the attention kernels (attend_rows.h, attend.hip).
#pragma once

#include "serve_launch.h"

namespace hkv {

constexpr int kTileTokens = 32;        // tokens of a step of the rows kernel
constexpr int kRowsWaves = 4;
constexpr int kRowsThreads = kRowsWaves * 64;
constexpr int kMaxFlatRequests = 1024; // requests whose tiles are dealt out evenly
constexpr int kWaveAreaBytes = 1280;   // LDS of a wave of the rows kernel

constexpr int kPromptWaves = 8;
constexpr int kPromptThreads = kPromptWaves * 64;
constexpr int kPromptRows = kPromptWaves * 32;   // rows of a workgroup of the prompt kernel

struct AttendParams {
  const uint8_t* rec;
  int64_t rec_block;
  int32_t n_blocks, block_tokens, n_heads, vecs;
  uint64_t block_magic;    // token / block_tokens = token * magic >> shift, token < 2^31
  int32_t block_shift;
  int32_t n_requests;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t max_len;
  int32_t max_queries;
  int32_t n_tokens;
  int32_t dtype, elem;
  const char* q;
  char* out;
  int64_t q_token, q_head, o_token, o_head;
  int32_t q_heads, group;
  float* lse;
  float scale_log2;        // sm_scale * log2(e)
  int32_t causal;
  const int32_t* delta;    // NULL: stored positions stand
  int32_t pairs;
  // the rows kernel's share of the work
  int32_t set_heads, head_sets;   // waves of different heads in a workgroup, sets of heads
  int32_t ranges;          // > 0: all tiles dealt out over this many ranges
  int32_t min_tiles;       // least tiles of a range
  int32_t part_rows;       // rows per head of a partial result
  int32_t splits;          // the prompt kernel's cuts of the tokens; 0: the rows kernel runs
  uint32_t* prefix_out;    // [n_requests + 2]: first tile of each request, total, tiles per range
  float* part_ml;          // reference and sum of each partial row
  float* part_o;           // its weighted values
  double theta[64];
};

hipError_t launch_rows_int4(const AttendParams& p, int hp, int nt, dim3 grid, size_t bytes,
                            hipStream_t stream);
hipError_t launch_rows_fp8(const AttendParams& p, int hp, int nt, dim3 grid, size_t bytes,
                           hipStream_t stream);
hipError_t launch_prompt_int4(const AttendParams& p, dim3 grid, hipStream_t stream);
hipError_t launch_prompt_fp8(const AttendParams& p, dim3 grid, hipStream_t stream);

}  // namespace hkv
