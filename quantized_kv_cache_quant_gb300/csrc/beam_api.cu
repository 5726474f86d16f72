// C-ABI host layer of the beam-search calls (kvq_beam.h): argument checks and
// launches.
#include <climits>
#include <cmath>
#include <cstdint>

#include "beam_internal.h"
#include "kvq_beam.h"
#include "kvq_device.cuh"
#include "pool_checks.h"
#include "spec_internal.h"

namespace {

using namespace kvq::checks;

static_assert(kvq::kBeamMaxWidth == KVQ_BEAM_MAX_WIDTH, "the kernels' arrays hold what the checks let through");
static_assert(kvq::kBeamMaxOut == KVQ_BEAM_MAX_OUT, "the same");
static_assert(kvq::kCopyMaxBuffers == KVQ_COPY_MAX_BUFFERS, "the same");

size_t padded(size_t n) { return (n + 255) / 256 * 256; }
// Offsets in the workspace of the block calls (beam_internal.h).
constexpr size_t kAlikeOffset = kvq::kWsHeader, kWordsOffset = kAlikeOffset + KVQ_SPEC_MAX_BATCH * sizeof(int32_t);
static_assert(kWordsOffset % 256 == 0, "the words are read 16 bytes at a time");

kvq_status check_workspace(const void* ws, size_t ws_bytes, int32_t groups, int32_t num_blocks) {
  if (ws == nullptr) return KVQ_ERR_WORKSPACE;
  if (!aligned(ws)) return KVQ_ERR_ALIGN;
  const size_t need = kv_blocks_workspace_bytes(groups, num_blocks);
  if (need == 0) return KVQ_ERR_UNSUPPORTED;
  return ws_bytes < need ? KVQ_ERR_WORKSPACE : KVQ_OK;
}

// Group attention workspace: [status word | 256 B][records of shared, of own pairs][slots of own pairs][slots of shared
// pairs][own pairs taken whole][shared pairs taken whole, each copy of a row].
struct GroupLayout {
  size_t records[2], slots[2], whole[2], bytes;  // offsets: kind 0 shared, 1 own
  size_t slot_rows[2], rows;
  kvq::GroupTile tile;
};
GroupLayout group_layout(int32_t batch, int32_t width, int32_t kv_heads, int32_t q_heads, int32_t head_dim) {
  GroupLayout l{};
  const int gq = q_heads / kv_heads;
  l.tile = kvq::group_tile(width * gq);
  l.rows = static_cast<size_t>(batch) * q_heads;
  const size_t pairs[2] = {static_cast<size_t>(batch / width) * kv_heads * ((width * gq + l.tile.rows - 1) / l.tile.rows),
                           static_cast<size_t>(batch) * kv_heads * ((gq + kvq::kGroupRows16 - 1) / kvq::kGroupRows16)};
  const bool tc = l.tile.rows != kvq::kGroupRows16;
  l.slot_rows[1] = 2 * kvq::kGroupMaxBlocks * kvq::kGroupRows16;
  l.slot_rows[0] = tc ? 2 * kvq::kGroupTcMaxBlocks * kvq::kGroupTcRows : l.slot_rows[1];
  size_t at = kvq::kWsHeader;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += padded(n);
    return here;
  };
  const size_t row = (static_cast<size_t>(head_dim) + 2) * sizeof(float);
  for (int kind = 0; kind < 2; ++kind) l.records[kind] = take(pairs[kind] * sizeof(kvq::GroupRecord));
  l.slots[1] = take(l.slot_rows[1] * row);
  l.slots[0] = take(l.slot_rows[0] * row);
  l.whole[1] = take(l.rows * row);
  l.whole[0] = take(l.rows * l.tile.fold * row);
  l.bytes = at;
  return l;
}

}  // namespace

kvq_status beam_select(const void* logits, int32_t logits_type, int64_t row_stride, const float* scores,
                       const uint8_t* finished, int32_t end_token, int32_t groups, int32_t width, int32_t vocab,
                       int32_t n_out, float* out_scores, int32_t* out_parents, int32_t* out_tokens, void* stream) {
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens) return KVQ_ERR_NULL;
  if (logits_type != KVQ_LOGITS_FP16 && logits_type != KVQ_LOGITS_FP32 && logits_type != KVQ_LOGITS_BF16) return KVQ_ERR_ARG;
  if (groups <= 0 || width <= 0 || vocab <= 0 || n_out <= 0 || n_out > vocab || row_stride < vocab) return KVQ_ERR_ARG;
  if (finished != nullptr && (end_token < 0 || end_token >= vocab)) return KVQ_ERR_ARG;
  if (width > KVQ_BEAM_MAX_WIDTH || n_out > KVQ_BEAM_MAX_OUT || vocab > (1 << 30) || groups > (1 << 24))
    return KVQ_ERR_UNSUPPORTED;
  const uintptr_t size = logits_type == KVQ_LOGITS_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size != 0) return KVQ_ERR_ALIGN;
  if (!aligned(scores) || !aligned(finished) || !aligned(out_scores) || !aligned(out_parents) || !aligned(out_tokens))
    return KVQ_ERR_ALIGN;
  kvq::BeamSelectArgs a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.scores = scores;
  a.finished = finished;
  a.out_scores = out_scores;
  a.out_parents = out_parents;
  a.out_tokens = out_tokens;
  a.type = logits_type;
  a.end_token = end_token;
  a.groups = groups;
  a.width = width;
  a.vocab = vocab;
  a.n_out = n_out;
  return from_cuda(kvq::launch_beam_select(a, static_cast<cudaStream_t>(stream)));
}

size_t kv_blocks_workspace_bytes(int32_t groups, int32_t num_blocks) {
  if (groups <= 0 || groups > KVQ_SPEC_MAX_BATCH || num_blocks <= 0 || num_blocks > INT_MAX - 31) return 0;
  const size_t words = (static_cast<size_t>(num_blocks) + 31) / 32;
  return kWordsOffset + (words + kvq::kWordChunk - 1) / kvq::kWordChunk * kvq::kChunkStride * sizeof(uint32_t);
}

kvq_status kv_blocks_fork(int32_t* block_table, int32_t batch, int32_t max_blocks, int32_t* n_held, int32_t* seq_lens,
                          const int32_t* parents, int32_t width, int32_t block_tokens, int32_t* shares,
                          int32_t* free_blocks, int32_t* free_count, int32_t num_blocks, int32_t* copy_src,
                          int32_t* copy_dst, int32_t* copy_count, int32_t* granted, int32_t* shared_blocks, void* ws,
                          size_t ws_bytes, void* stream) {
  if (!block_table || !n_held || !seq_lens || !parents || !shares || !free_blocks || !free_count || !copy_src ||
      !copy_dst || !copy_count)
    return KVQ_ERR_NULL;
  if (batch <= 0 || max_blocks <= 0 || width <= 0 || block_tokens <= 0 || num_blocks <= 0) return KVQ_ERR_ARG;
  if (batch > KVQ_SPEC_MAX_BATCH || width > KVQ_BEAM_MAX_WIDTH || static_cast<long long>(batch) * max_blocks > INT_MAX)
    return KVQ_ERR_UNSUPPORTED;
  if (batch % width != 0) return KVQ_ERR_SHAPE;
  if (!aligned(block_table) || !aligned(n_held) || !aligned(seq_lens) || !aligned(parents) || !aligned(shares) ||
      !aligned(free_blocks) || !aligned(free_count) || !aligned(copy_src) || !aligned(copy_dst) || !aligned(copy_count) ||
      !aligned(granted) || !aligned(shared_blocks))
    return KVQ_ERR_ALIGN;
  const kvq_status st = check_workspace(ws, ws_bytes, batch / width, num_blocks);
  if (st != KVQ_OK) return st;
  kvq::BlocksForkArgs a{};
  a.block_table = block_table;
  a.n_held = n_held;
  a.seq_lens = seq_lens;
  a.parents = parents;
  a.shares = shares;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.copy_count = copy_count;
  a.granted = granted;
  a.shared_blocks = shared_blocks;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  a.alike = reinterpret_cast<int32_t*>(base + kAlikeOffset);
  a.bits = reinterpret_cast<uint32_t*>(base + kWordsOffset);
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.width = width;
  a.block_tokens = block_tokens;
  a.num_blocks = num_blocks;
  return from_cuda(kvq::launch_blocks_fork(a, static_cast<cudaStream_t>(stream)));
}

kvq_status kv_blocks_resize_shared(int32_t* block_table, int32_t batch, int32_t max_blocks, int32_t* n_held,
                                   const int32_t* target_tokens, int32_t block_tokens, const int32_t* shares,
                                   int32_t* free_blocks, int32_t* free_count, int32_t num_blocks, int32_t* granted,
                                   void* stream) {
  if (!block_table || !n_held || !target_tokens || !shares || !free_blocks || !free_count) return KVQ_ERR_NULL;
  if (batch <= 0 || max_blocks <= 0 || block_tokens <= 0 || num_blocks <= 0) return KVQ_ERR_ARG;
  if (batch > KVQ_SPEC_MAX_BATCH || static_cast<long long>(batch) * max_blocks > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(block_table) || !aligned(n_held) || !aligned(target_tokens) || !aligned(shares) || !aligned(free_blocks) ||
      !aligned(free_count) || !aligned(granted))
    return KVQ_ERR_ALIGN;
  kvq::BlocksResizeArgs a{};
  a.block_table = block_table;
  a.n_held = n_held;
  a.target_tokens = target_tokens;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.granted = granted;
  a.shares = shares;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.block_tokens = block_tokens;
  a.num_blocks = num_blocks;
  return from_cuda(kvq::launch_blocks_resize(a, static_cast<cudaStream_t>(stream)));
}

kvq_status kv_blocks_copy(const kvq_block_buffer* buffers, int32_t n_buffers, int32_t num_blocks, const int32_t* src,
                          const int32_t* dst, int32_t n_pairs, const int32_t* count, void* stream) {
  if (!buffers || !src || !dst) return KVQ_ERR_NULL;
  if (n_buffers <= 0 || num_blocks <= 0 || n_pairs <= 0) return KVQ_ERR_ARG;
  if (n_buffers > KVQ_COPY_MAX_BUFFERS) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(src) || !aligned(dst) || !aligned(count)) return KVQ_ERR_ALIGN;
  kvq::BlocksCopyArgs a{};
  long long pieces = 0;
  for (int i = 0; i < n_buffers; ++i) {
    if (buffers[i].base == nullptr) return KVQ_ERR_NULL;
    if (buffers[i].block_bytes <= 0 || buffers[i].block_bytes % 16 != 0) return KVQ_ERR_ARG;
    if (buffers[i].block_bytes > LLONG_MAX / num_blocks) return KVQ_ERR_UNSUPPORTED;
    if (!aligned(buffers[i].base)) return KVQ_ERR_ALIGN;
    a.base[i] = static_cast<uint8_t*>(buffers[i].base);
    a.block_bytes[i] = buffers[i].block_bytes;
    a.first_piece[i] = static_cast<int32_t>(pieces);
    pieces += (buffers[i].block_bytes + kvq::kCopyPiece - 1) / kvq::kCopyPiece;
    if (pieces > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  }
  a.first_piece[n_buffers] = static_cast<int32_t>(pieces);
  a.src = src;
  a.dst = dst;
  a.count = count;
  a.n_buffers = n_buffers;
  a.n_pairs = n_pairs;
  a.num_blocks = num_blocks;
  return from_cuda(kvq::launch_blocks_copy(a, static_cast<cudaStream_t>(stream)));
}

kvq_status kv_blocks_compact(int32_t* block_table, int32_t batch, int32_t max_blocks, const int32_t* n_held,
                             int32_t keep_blocks, int32_t* shares, int32_t* free_blocks, int32_t* free_count,
                             int32_t num_blocks, int32_t* moved_to, int32_t* copy_src, int32_t* copy_dst,
                             int32_t max_copies, int32_t* copy_count, int32_t* done, void* ws, size_t ws_bytes,
                             void* stream) {
  if (!block_table || !n_held || !shares || !free_blocks || !free_count || !moved_to || !copy_src || !copy_dst ||
      !copy_count || !done)
    return KVQ_ERR_NULL;
  if (batch <= 0 || max_blocks <= 0 || num_blocks <= 0 || max_copies <= 0 || keep_blocks < 0 || keep_blocks > num_blocks)
    return KVQ_ERR_ARG;
  if (batch > KVQ_SPEC_MAX_BATCH || static_cast<long long>(batch) * max_blocks > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(block_table) || !aligned(n_held) || !aligned(shares) || !aligned(free_blocks) || !aligned(free_count) ||
      !aligned(moved_to) || !aligned(copy_src) || !aligned(copy_dst) || !aligned(copy_count) || !aligned(done))
    return KVQ_ERR_ALIGN;
  const kvq_status st = check_workspace(ws, ws_bytes, 1, num_blocks);
  if (st != KVQ_OK) return st;
  kvq::BlocksCompactArgs a{};
  a.block_table = block_table;
  a.n_held = n_held;
  a.shares = shares;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.moved_to = moved_to;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.copy_count = copy_count;
  a.done = done;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  a.state = reinterpret_cast<kvq::CompactState*>(base);
  a.bits = reinterpret_cast<uint32_t*>(base + kWordsOffset) + kvq::kWordChunk;
  a.before = reinterpret_cast<int32_t*>(base + kWordsOffset) + 2 * kvq::kWordChunk;
  a.batch = batch;
  a.max_blocks = max_blocks;
  a.keep = keep_blocks;
  a.num_blocks = num_blocks;
  a.max_copies = max_copies;
  return from_cuda(kvq::launch_blocks_compact(a, static_cast<cudaStream_t>(stream)));
}

size_t fp8_group_workspace_bytes(int32_t batch, int32_t width, int32_t kv_heads, int32_t q_heads, int32_t head_dim) {
  if (batch <= 0 || batch > KVQ_SPEC_MAX_BATCH || width <= 0 || width > KVQ_BEAM_MAX_WIDTH || batch % width != 0 ||
      kv_heads <= 0 || kv_heads > 65535 || q_heads <= 0 || q_heads % kv_heads != 0 ||
      q_heads / kv_heads > KVQ_TREE_MAX_GQA || static_cast<long long>(batch) * q_heads > INT_MAX ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return group_layout(batch, width, kv_heads, q_heads, head_dim).bytes;
}

kvq_status fp8_group_attention(const uint16_t* q, int64_t q_row_stride, const fp8_pool* k, const fp8_pool* v,
                               const int32_t* block_table, const int32_t* seq_lens, const int32_t* shared_blocks,
                               int32_t batch, int32_t width, int32_t q_heads, int32_t max_blocks, int32_t max_seq_len,
                               void* out, int32_t out_fp32, float softmax_scale, void* ws, size_t ws_bytes, void* stream) {
  const kvq_status st = check_pools(k, v);
  if (st != KVQ_OK) return st;
  if (!q || !block_table || !seq_lens || !shared_blocks || !out) return KVQ_ERR_NULL;
  if (batch <= 0 || width <= 0 || q_heads <= 0 || max_blocks <= 0 || max_seq_len <= 0) return KVQ_ERR_ARG;
  const int kv_heads = k->kv_heads, head_dim = k->head_dim;
  if (batch > KVQ_SPEC_MAX_BATCH || width > KVQ_BEAM_MAX_WIDTH) return KVQ_ERR_UNSUPPORTED;
  if (batch % width != 0 || q_heads % kv_heads != 0) return KVQ_ERR_SHAPE;
  if (q_heads / kv_heads > KVQ_TREE_MAX_GQA || static_cast<long long>(batch) * q_heads > INT_MAX) return KVQ_ERR_UNSUPPORTED;
  if (q_row_stride < static_cast<int64_t>(q_heads) * head_dim || q_row_stride % 8 != 0) return KVQ_ERR_ARG;
  if (max_blocks > INT_MAX / 16) return KVQ_ERR_UNSUPPORTED;
  if (max_seq_len > max_blocks * 16) return KVQ_ERR_CAPACITY;
  if (!aligned16(q) || !aligned(block_table) || !aligned(seq_lens) || !aligned(shared_blocks) || !aligned(out))
    return KVQ_ERR_ALIGN;
  if (ws == nullptr) return KVQ_ERR_WORKSPACE;
  if (!aligned(ws)) return KVQ_ERR_ALIGN;
  const GroupLayout l = group_layout(batch, width, kv_heads, q_heads, head_dim);
  if (ws_bytes < l.bytes) return KVQ_ERR_WORKSPACE;
  if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale)) return KVQ_ERR_ARG;
  const float scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
  kvq::GroupArgs a{};
  a.q = q;
  a.q_stride = q_row_stride;
  a.k_pool = k->pool;
  a.v_pool = v->pool;
  a.k_scale = k->scale;
  a.v_scale = v->scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.shared_blocks = shared_blocks;
  a.batch = batch;
  a.width = width;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.max_blocks = max_blocks;
  a.num_blocks = k->num_blocks;
  a.max_seq_len = max_seq_len;
  a.per_head = k->per_head;
  a.fmt = k->fp8_format;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.out = out;
  a.out_fp32 = out_fp32;
  uint8_t* const base = static_cast<uint8_t*>(ws);
  a.status = reinterpret_cast<uint32_t*>(base);
  for (int kind = 0; kind < 2; ++kind) {
    kvq::GroupPartials& p = a.part[kind];
    p.tile_rows = kind == 0 ? l.tile.rows : kvq::kGroupRows16;
    p.fold = kind == 0 ? l.tile.fold : 1;
    p.records = reinterpret_cast<kvq::GroupRecord*>(base + l.records[kind]);
    // (outputs first: their rows are whole 256 bytes)
    p.o = reinterpret_cast<float*>(base + l.slots[kind]);
    p.ml = p.o + l.slot_rows[kind] * head_dim;
    p.whole_o = reinterpret_cast<float*>(base + l.whole[kind]);
    p.whole_ml = p.whole_o + l.rows * p.fold * head_dim;
  }
  return from_cuda(kvq::launch_group_attention(a, static_cast<cudaStream_t>(stream)));
}
