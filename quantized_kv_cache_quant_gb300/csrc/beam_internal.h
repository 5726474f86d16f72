// Launch interface between the host layer of the beam-search calls
// (beam_api.cu) and their kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace kvq {

constexpr int kBeamMaxWidth = 64;     // KVQ_BEAM_MAX_WIDTH
constexpr int kBeamMaxOut = 128;      // KVQ_BEAM_MAX_OUT
constexpr int kCopyMaxBuffers = 160;  // KVQ_COPY_MAX_BUFFERS

struct BeamSelectArgs {
  const void* logits;
  long long row_stride;
  const float* scores;
  const uint8_t* finished;  // or null
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int type, end_token, groups, width, vocab, n_out;
};
cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t s);

struct BlocksForkArgs {
  int32_t* block_table;
  int32_t* n_held;
  int32_t* seq_lens;
  const int32_t* parents;
  int32_t* shares;
  int32_t* free_blocks;
  int32_t* free_count;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* copy_count;
  int32_t* granted;        // or null
  int32_t* shared_blocks;  // or null
  uint32_t* bits;          // [ceil(num_blocks / 32)] blocks freed; 0 between calls
  int32_t* alike;          // [batch / width] max_blocks - first column that differs; 0 between calls
  int batch, max_blocks, width, block_tokens, num_blocks;
};
cudaError_t launch_blocks_fork(const BlocksForkArgs& a, cudaStream_t s);

struct BlocksCopyArgs {
  uint8_t* base[kCopyMaxBuffers];
  long long block_bytes[kCopyMaxBuffers];
  int32_t first_piece[kCopyMaxBuffers + 1];  // pieces of a block in the buffers before
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;  // or null
  int n_buffers, n_pairs, num_blocks;
};
constexpr int kCopyPiece = 4096;  // bytes a warp copies at a time
cudaError_t launch_blocks_copy(const BlocksCopyArgs& a, cudaStream_t s);

struct CompactState {
  int32_t movers, targets, done;
};
struct BlocksCompactArgs {
  int32_t* block_table;
  const int32_t* n_held;
  int32_t* shares;
  int32_t* free_blocks;
  int32_t* free_count;
  int32_t* moved_to;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* copy_count;
  int32_t* done;
  uint32_t* bits;        // [ceil(num_blocks / 32)] free blocks; 0 between calls
  int32_t* before;       // [ceil(num_blocks / 32)] free blocks below keep, used ones from keep on, in the words before
  CompactState* state;
  int batch, max_blocks, keep, num_blocks, max_copies;
};
cudaError_t launch_blocks_compact(const BlocksCompactArgs& a, cudaStream_t s);

}  // namespace kvq
