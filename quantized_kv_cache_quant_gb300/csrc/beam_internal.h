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

// Workspace of the block calls: [what compaction knows | 256 B][per request, 16 KB][by 64 words of 32 blocks each: words of
// freed blocks, words of free blocks, ranks before each word]. The place of a word is the same for pools of all sizes, so
// that what one call needs at 0 is never what another one left.
constexpr int kWordChunk = 64;
constexpr int kChunkStride = 3 * kWordChunk;
__host__ __device__ constexpr long long word_at(int i) {
  return static_cast<long long>(i / kWordChunk) * kChunkStride + i % kWordChunk;
}

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
  uint32_t* bits;          // word_at(0 .. ceil(num_blocks / 32) - 1): blocks freed; 0 between calls
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
  uint32_t* bits;        // word_at(0 .. ceil(num_blocks / 32) - 1): free blocks
  int32_t* before;       // the same: free blocks below keep, used ones from keep on, in the words before
  CompactState* state;
  int batch, max_blocks, keep, num_blocks, max_copies;
};
cudaError_t launch_blocks_compact(const BlocksCompactArgs& a, cudaStream_t s);

// What a pair of group attention left (group_plan.cuh): its number of parts,
// and, where there are several, the slot of the first.
struct GroupRecord {
  int parts, slot0;
};

// Partial results of a kind of pair (kind 0: shared blocks, 1: a sequence's
// own). Row `row` of a slot or of the pairs that one thread block took whole is
// `fold` partial rows that have to be joined too.
struct GroupPartials {
  GroupRecord* records;  // [requests, kv_heads, tiles]
  float* ml;             // [slots * tile_rows * fold, 2] (exponent, sum) of parts
  float* o;              // [slots * tile_rows * fold, D]
  float* whole_ml;       // [fold, batch * q_heads, 2]
  float* whole_o;        // [fold, batch * q_heads, D]
  int tile_rows, fold;
};

struct GroupArgs {
  const uint16_t* q;
  long long q_stride;  // fp16 elements between rows of q
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* shared_blocks;
  int batch, width, q_heads, kv_heads, head_dim, max_blocks, num_blocks, max_seq_len, per_head, fmt;
  int kinds;         // bit 0: this launch takes the shared blocks, bit 1: the own ones
  int blocks[2];     // thread blocks of the 16-row kernel that a kind can have work for
  float scale_log2;  // softmax scale * log2(e)
  void* out;
  int out_fp32;
  uint32_t* status;
  GroupPartials part[2];
};
// Rows of the partial results that the thread blocks of one launch leave in
// slots: two slots a block.
constexpr int kGroupMaxBlocks = 1024;       // of the 16-row kernel
constexpr int kGroupTcMaxBlocks = 160;      // of the tcgen05 kernel
constexpr int kGroupRows16 = 16, kGroupTcRows = 128;
// Query rows of a tile of shared blocks, as partial rows each: up to 16 rows a kv head the 16-row kernel, beyond the
// tcgen05 kernel, whose 128 rows hold 64 rows twice where that is enough. (us, 128 channels unless said otherwise:
//   16 rows, 8 x 4 sequences over 32K tokens   113 on mma.sync, 136 on tcgen05; 64 channels, 16 x 4 over 16K: 74, 109
//   32 rows, 32 x 4 sequences over 8K tokens   208 as two tiles on mma.sync, 163 held twice, 167 four times, 174 once
//   64 rows, 4 x 8 sequences over 128K tokens  664 as four tiles on mma.sync, 253 held twice, 273 once)
struct GroupTile {
  int rows, fold;
};
constexpr GroupTile group_tile(int rows_per_head) {
  return rows_per_head <= 16 ? GroupTile{16, 1} : rows_per_head <= 64 ? GroupTile{64, 2} : GroupTile{128, 1};
}
cudaError_t launch_group_attention(const GroupArgs& a, cudaStream_t s);
cudaError_t launch_group_tc(const GroupArgs& a, cudaStream_t s);  // the shared blocks on tcgen05

}  // namespace kvq
