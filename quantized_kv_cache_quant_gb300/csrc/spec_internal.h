// Launch interface between the host layer of the speculative-decoding calls
// (spec_api.cu) and their kernels.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace kvq {

constexpr int kSpecMaxBatch = 4096;  // KVQ_SPEC_MAX_BATCH
constexpr int kTreeMax = 256;        // KVQ_TREE_MAX

// A kernel's shared-memory limit, raised once per device (and its resident
// blocks per SM asked once): both calls cost more than a small launch. Two
// threads that come first together make the same call twice.
struct SharedMemoryOnce {
  static constexpr int kDevices = 64;
  std::atomic<int> per_sm[kDevices] = {};  // 0: not set yet
  template <class Kernel>
  cudaError_t set(Kernel kern, int smem, int threads = 0, int* blocks = nullptr) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = dev < kDevices ? per_sm[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      n = 1;
      if (threads > 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
      }
      if (dev < kDevices) per_sm[dev].store(n, std::memory_order_release);
    }
    if (blocks != nullptr) *blocks = n;
    return cudaSuccess;
  }
};

struct BlocksResizeArgs {
  int32_t* block_table;
  int32_t* n_held;
  const int32_t* target_tokens;
  int32_t* free_blocks;
  int32_t* free_count;
  int32_t* granted;  // or null
  const int32_t* shares;  // references of each block beyond the first, or null: every block has one
  int batch, max_blocks, block_tokens, num_blocks;
};
cudaError_t launch_blocks_resize(const BlocksResizeArgs& a, cudaStream_t s);

struct SlotMapArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* offsets;
  int64_t* slots;
  int32_t* seq_ids;    // or null
  int32_t* positions;  // or null
  int batch, max_blocks, block_tokens, num_blocks, n_rows;
};
cudaError_t launch_slot_map(const SlotMapArgs& a, cudaStream_t s);

struct Fp8AppendArgs {
  const uint16_t* k_new;
  const uint16_t* v_new;
  long long k_stride, v_stride;  // fp16 elements between tokens
  const int64_t* slots;
  int n_tokens, kv_heads, head_dim, num_blocks, per_head, fmt;
  uint8_t* k_pool;
  uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
};
cudaError_t launch_fp8_append(const Fp8AppendArgs& a, cudaStream_t s);

struct Fp8AcceptArgs {
  uint8_t* k_pool;
  uint8_t* v_pool;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* path;
  const int32_t* n_accepted;
  int32_t* new_lens;
  int batch, max_blocks, path_len, kv_heads, head_dim, num_blocks;
};
cudaError_t launch_fp8_accept(const Fp8AcceptArgs& a, cudaStream_t s);

// A pair of tree attention whose work several thread blocks shared (tree_plan.cuh).
struct TreeJoin {
  int parts;                // 0: none
  int slot0;                // of the first part; part i > 0 is in slot (slot0 & ~1) + 2 * i
  int rows, row0;           // rows of the tile, the tile's first row of the pair
  int b, h;
  int first, nodes, len;    // as TreeRequest's
};

struct TreeArgs {
  const uint16_t* q;
  long long q_stride;  // fp16 elements between rows of q
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* tree_offsets;
  const uint64_t* tree_mask;
  int mask_words;
  int n_tokens, batch, q_heads, kv_heads, head_dim, max_blocks, num_blocks, max_tree, max_seq_len, per_head, fmt;
  float scale_log2;  // softmax scale * log2(e)
  void* out;
  int out_fp32;
  uint32_t* status;
  TreeJoin* joins;  // [kTreeMaxBlocks]
  int* part_flag;   // [2 * kTreeMaxBlocks] NaN codes met
  float* part_ml;   // [2 * kTreeMaxBlocks, R, 2]
  float* part_o;    // [2 * kTreeMaxBlocks, R, D]
};
// Thread blocks of a tree attention launch at most (they leave two partial
// results each), and the rows of their partial results in all: R rows times
// two slots times the blocks of every kernel stay within kTreePartRows.
constexpr int kTreeMaxBlocks = 1024;
constexpr int kTreePartRows = 81920;
cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s);
// Joins the partial results that `blocks` thread blocks with tiles of `tile_rows` rows left.
cudaError_t launch_tree_join(const TreeArgs& a, int blocks, int tile_rows, cudaStream_t s);
// The same on tcgen05: 128 or 256 query rows a tile.
cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t s);

}  // namespace kvq
