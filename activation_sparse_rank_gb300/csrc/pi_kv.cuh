// Argument checks of the key/value cache's entry points (pi_kv.cu, pi_attn.cu).
#pragma once

#include "pi_internal.cuh"

namespace pi {

pi_status check_cache(const pi_kv_cache *c);
pi_status check_tokens(const pi_kv_tokens *t);
// t with table_pages as the kernels use it.
inline pi_kv_tokens with_pages(pi_kv_tokens t) {
  if (t.table_pages == 0) t.table_pages = t.table_stride;
  return t;
}

}  // namespace pi
