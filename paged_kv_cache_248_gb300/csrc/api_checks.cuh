// api_checks.cuh -- the argument checks that the C entries share.
#pragma once
#include "pkv_internal.cuh"

namespace pkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_cache(const pkv_cache_desc* c) {
  if (!c) return PKV_ERR_INVALID_ARG;
  if (c->block_size != PKV_BLOCK_SIZE || c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
    return PKV_ERR_INVALID_ARG;
  if (c->num_blocks > (int64_t(1) << 40)) return PKV_ERR_INVALID_ARG;
  if (c->dtype == PKV_F32 && (c->head_dim == 64 || c->head_dim == 128)) return PKV_OK;
  if (c->dtype == PKV_BF16 && c->head_dim == 128) return PKV_OK;
  return PKV_ERR_UNSUPPORTED;
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace pkv
