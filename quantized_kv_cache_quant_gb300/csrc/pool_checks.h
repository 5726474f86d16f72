// Argument checks that the host layers of the paged FP8 calls share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kvq.h"

namespace kvq {
namespace checks {

inline bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline kvq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

inline kvq_status check_pool(const fp8_pool* p) {
  if (p == nullptr || p->pool == nullptr || p->scale == nullptr) return KVQ_ERR_NULL;
  if (p->role != KVQ_ROLE_KEY && p->role != KVQ_ROLE_VALUE) return KVQ_ERR_ARG;
  if (p->fp8_format != 0 && p->fp8_format != 1) return KVQ_ERR_ARG;
  if (p->per_head != 0 && p->per_head != 1) return KVQ_ERR_ARG;
  if (p->num_blocks <= 0 || p->kv_heads <= 0) return KVQ_ERR_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (!aligned(p->pool) || !aligned(p->scale)) return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

// A key pool and a value pool that belong together.
inline kvq_status check_pools(const fp8_pool* k, const fp8_pool* v) {
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

}  // namespace checks
}  // namespace kvq
