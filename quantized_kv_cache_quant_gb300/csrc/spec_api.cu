// C-ABI host layer of the speculative-decoding calls (kvq_spec.h): argument
// checks and launches.
#include <climits>
#include <cmath>
#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_spec.h"
#include "spec_internal.h"

namespace {

static_assert(kvq::kSpecMaxBatch == KVQ_SPEC_MAX_BATCH, "the kernels' arrays hold what the checks let through");
static_assert(kvq::kTreeMax == KVQ_TREE_MAX, "the same");

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

kvq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

kvq_status check_pool(const fp8_pool* p) {
  if (p == nullptr || p->pool == nullptr || p->scale == nullptr) return KVQ_ERR_NULL;
  if (p->role != KVQ_ROLE_KEY && p->role != KVQ_ROLE_VALUE) return KVQ_ERR_ARG;
  if (p->fp8_format != 0 && p->fp8_format != 1) return KVQ_ERR_ARG;
  if (p->per_head != 0 && p->per_head != 1) return KVQ_ERR_ARG;
  if (p->num_blocks <= 0 || p->kv_heads <= 0) return KVQ_ERR_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(p->pool) || !aligned(p->scale)) return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

// Tree attention workspace: [status word | 256 B][what to join][flags of the
// partial results][(m, l) of their rows][o of their rows].
constexpr size_t kTreeJoins = kvq::kWsHeader;
constexpr size_t kTreeFlags = kTreeJoins + kvq::kTreeMaxBlocks * sizeof(kvq::TreeJoin);
constexpr size_t kTreePartials = kTreeFlags + 2 * kvq::kTreeMaxBlocks * sizeof(int);
static_assert(kTreePartials % 256 == 0, "the partial results are read as 16-byte vectors");

// A key pool and a value pool that belong together.
kvq_status check_pools(const fp8_pool* k, const fp8_pool* v) {
  kvq_status st = check_pool(k);
  if (st != KVQ_OK) return st;
  st = check_pool(v);
  if (st != KVQ_OK) return st;
  if (k->role != KVQ_ROLE_KEY || v->role != KVQ_ROLE_VALUE) return KVQ_ERR_ARG;
  if (k->fp8_format != v->fp8_format || k->per_head != v->per_head) return KVQ_ERR_ARG;
  if (k->num_blocks != v->num_blocks || k->kv_heads != v->kv_heads || k->head_dim != v->head_dim) return KVQ_ERR_SHAPE;
  if (k->kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

}  // namespace

kvq_status kv_blocks_resize(int32_t* block_table, int32_t batch, int32_t max_blocks, int32_t* n_held,
                            const int32_t* target_tokens, int32_t block_tokens, int32_t* free_blocks,
                            int32_t* free_count, int32_t num_blocks, int32_t* granted, void* stream) {
  if (!block_table || !n_held || !target_tokens || !free_blocks || !free_count) return KVQ_ERR_NULL;
  if (batch <= 0 || max_blocks <= 0 || block_tokens <= 0 || num_blocks <= 0) return KVQ_ERR_ARG;
  if (batch > KVQ_SPEC_MAX_BATCH || static_cast<long long>(batch) * max_blocks > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(block_table) || !aligned(n_held) || !aligned(target_tokens) || !aligned(free_blocks) ||
      !aligned(free_count) || !aligned(granted))
    return KVQ_ERR_ALIGN;
  kvq::BlocksResizeArgs a{};
  a.block_table = block_table;
  a.n_held = n_held;
  a.target_tokens = target_tokens;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.granted = granted;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.block_tokens = block_tokens;
  a.num_blocks = num_blocks;
  return from_cuda(kvq::launch_blocks_resize(a, static_cast<cudaStream_t>(stream)));
}

kvq_status kv_slot_map(const int32_t* block_table, int32_t batch, int32_t max_blocks, const int32_t* seq_lens,
                       const int32_t* new_lens, int32_t block_tokens, int32_t num_blocks, int32_t n_rows,
                       int32_t* offsets, int64_t* slots, int32_t* seq_ids, int32_t* positions, void* stream) {
  if (!block_table || !seq_lens || !new_lens || !offsets || !slots) return KVQ_ERR_NULL;
  if (batch <= 0 || max_blocks <= 0 || block_tokens <= 0 || num_blocks <= 0 || n_rows <= 0) return KVQ_ERR_ARG;
  if (batch > KVQ_SPEC_MAX_BATCH) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(block_table) || !aligned(seq_lens) || !aligned(new_lens) || !aligned(offsets) || !aligned(slots) ||
      !aligned(seq_ids) || !aligned(positions))
    return KVQ_ERR_ALIGN;
  kvq::SlotMapArgs a{};
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.offsets = offsets;
  a.slots = slots;
  a.seq_ids = seq_ids;
  a.positions = positions;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.block_tokens = block_tokens;
  a.num_blocks = num_blocks;
  a.n_rows = n_rows;
  return from_cuda(kvq::launch_slot_map(a, static_cast<cudaStream_t>(stream)));
}

kvq_status fp8_kv_append(const fp8_pool* k, const fp8_pool* v, const uint16_t* k_new, int64_t k_row_stride,
                         const uint16_t* v_new, int64_t v_row_stride, const int64_t* slots, int32_t n_tokens,
                         void* stream) {
  const kvq_status st = check_pools(k, v);
  if (st != KVQ_OK) return st;
  if (!k_new || !v_new || !slots) return KVQ_ERR_NULL;
  if (n_tokens <= 0) return KVQ_ERR_ARG;
  const int64_t row = static_cast<int64_t>(k->kv_heads) * k->head_dim;
  if (k_row_stride < row || v_row_stride < row || k_row_stride % 8 != 0 || v_row_stride % 8 != 0) return KVQ_ERR_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned(slots)) return KVQ_ERR_ALIGN;
  kvq::Fp8AppendArgs a{};
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.slots = slots;
  a.n_tokens = n_tokens;
  a.kv_heads = k->kv_heads;
  a.head_dim = k->head_dim;
  a.num_blocks = k->num_blocks;
  a.per_head = k->per_head;
  a.fmt = k->fp8_format;
  a.k_pool = k->pool;
  a.v_pool = v->pool;
  a.k_scale = k->scale;
  a.v_scale = v->scale;
  return from_cuda(kvq::launch_fp8_append(a, static_cast<cudaStream_t>(stream)));
}

kvq_status fp8_kv_accept(const fp8_pool* k, const fp8_pool* v, const int32_t* block_table, int32_t batch,
                         int32_t max_blocks, const int32_t* seq_lens, const int32_t* path, int32_t path_len,
                         const int32_t* n_accepted, int32_t* new_lens, void* stream) {
  const kvq_status st = check_pools(k, v);
  if (st != KVQ_OK) return st;
  if (!block_table || !seq_lens || !path || !n_accepted || !new_lens) return KVQ_ERR_NULL;
  if (batch <= 0 || max_blocks <= 0 || path_len <= 0) return KVQ_ERR_ARG;
  if (batch > KVQ_SPEC_MAX_BATCH || path_len > KVQ_TREE_MAX) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(block_table) || !aligned(seq_lens) || !aligned(path) || !aligned(n_accepted) || !aligned(new_lens))
    return KVQ_ERR_ALIGN;
  kvq::Fp8AcceptArgs a{};
  a.k_pool = k->pool;
  a.v_pool = v->pool;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.path = path;
  a.n_accepted = n_accepted;
  a.new_lens = new_lens;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.path_len = path_len;
  a.kv_heads = k->kv_heads;
  a.head_dim = k->head_dim;
  a.num_blocks = k->num_blocks;
  return from_cuda(kvq::launch_fp8_accept(a, static_cast<cudaStream_t>(stream)));
}

size_t fp8_tree_workspace_bytes(int32_t batch, int32_t kv_heads, int32_t q_heads, int32_t head_dim, int32_t max_tree) {
  if (batch <= 0 || batch > KVQ_SPEC_MAX_BATCH || kv_heads <= 0 || kv_heads > 65535 || q_heads <= 0 ||
      q_heads % kv_heads != 0 || q_heads / kv_heads > KVQ_TREE_MAX_GQA || (head_dim != 64 && head_dim != 128) ||
      max_tree <= 0 || max_tree > KVQ_TREE_MAX)
    return 0;
  return kTreePartials + static_cast<size_t>(kvq::kTreePartRows) * (head_dim + 2) * sizeof(float);
}

kvq_status fp8_tree_attention(const uint16_t* q, int64_t q_row_stride, int32_t n_tokens, const fp8_pool* k,
                              const fp8_pool* v, const int32_t* block_table, const int32_t* seq_lens,
                              const int32_t* tree_offsets, const uint64_t* tree_mask, int32_t mask_words, int32_t batch,
                              int32_t q_heads, int32_t max_blocks, int32_t max_tree, int32_t max_seq_len, void* out,
                              int32_t out_fp32, float softmax_scale, void* ws, size_t ws_bytes, void* stream) {
  const kvq_status st = check_pools(k, v);
  if (st != KVQ_OK) return st;
  if (!q || !block_table || !seq_lens || !tree_offsets || !tree_mask || !out) return KVQ_ERR_NULL;
  if (n_tokens <= 0 || batch <= 0 || q_heads <= 0 || max_blocks <= 0 || max_tree <= 0 || max_seq_len <= 0)
    return KVQ_ERR_ARG;
  const int kv_heads = k->kv_heads, head_dim = k->head_dim;
  if (max_tree > KVQ_TREE_MAX || batch > KVQ_SPEC_MAX_BATCH) return KVQ_ERR_UNSUPPORTED;
  if (q_heads % kv_heads != 0) return KVQ_ERR_SHAPE;
  if (q_heads / kv_heads > KVQ_TREE_MAX_GQA) return KVQ_ERR_UNSUPPORTED;
  if (mask_words <= 0 || static_cast<long long>(mask_words) * 64 < max_tree) return KVQ_ERR_ARG;
  if (q_row_stride < static_cast<int64_t>(q_heads) * head_dim || q_row_stride % 8 != 0) return KVQ_ERR_ARG;
  if (max_blocks > INT_MAX / 16) return KVQ_ERR_UNSUPPORTED;
  if (max_seq_len > max_blocks * 16) return KVQ_ERR_CAPACITY;
  if (!aligned16(q) || !aligned(block_table) || !aligned(seq_lens) || !aligned(tree_offsets) || !aligned(tree_mask) ||
      !aligned(out))
    return KVQ_ERR_ALIGN;
  if (ws == nullptr) return KVQ_ERR_WORKSPACE;
  if (!aligned(ws)) return KVQ_ERR_ALIGN;
  if (ws_bytes < fp8_tree_workspace_bytes(batch, kv_heads, q_heads, head_dim, max_tree)) return KVQ_ERR_WORKSPACE;
  if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale)) return KVQ_ERR_ARG;
  const float scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
  kvq::TreeArgs a{};
  a.q = q;
  a.q_stride = q_row_stride;
  a.k_pool = k->pool;
  a.v_pool = v->pool;
  a.k_scale = k->scale;
  a.v_scale = v->scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.tree_offsets = tree_offsets;
  a.tree_mask = tree_mask;
  a.mask_words = mask_words;
  a.n_tokens = n_tokens;
  a.batch = batch;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.max_blocks = max_blocks;
  a.num_blocks = k->num_blocks;
  a.max_tree = max_tree;
  a.max_seq_len = max_seq_len;
  a.per_head = k->per_head;
  a.fmt = k->fp8_format;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.out = out;
  a.out_fp32 = out_fp32;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  a.status = reinterpret_cast<uint32_t*>(base);
  a.joins = reinterpret_cast<kvq::TreeJoin*>(base + kTreeJoins);
  a.part_flag = reinterpret_cast<int*>(base + kTreeFlags);
  a.part_ml = reinterpret_cast<float*>(base + kTreePartials);
  a.part_o = a.part_ml + static_cast<size_t>(kvq::kTreePartRows) * 2;
  return from_cuda(kvq::launch_tree_attention(a, static_cast<cudaStream_t>(stream)));
}
