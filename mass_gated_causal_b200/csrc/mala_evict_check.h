// mala_evict_check.h -- the host's checks of mala_evict_gather's arguments, on their own so
// that the torch side can make them before it starts the selection that comes first.
#pragma once

#include <algorithm>
#include <cstdint>

#include "../../include/mala.h"

namespace mala {

inline int check_gather(const void* k_pages, const void* v_pages, const void* block_table, const void* index,
                        const void* new_seqlens, const void* k_out_pages, const void* v_out_pages,
                        const void* out_table, int B, int Hkv, int budget, int num_pages, int num_out_pages,
                        int page_size, int max_pages_per_seq, int max_out_pages_per_seq, int d) {
  if (!k_pages || !v_pages || !block_table || !index || !new_seqlens || !k_out_pages || !v_out_pages || !out_table)
    return MALA_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || budget < 1 || num_pages < 1 || num_out_pages < 1 || max_pages_per_seq < 1 ||
      max_out_pages_per_seq < 1)
    return MALA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return MALA_ERR_UNSUPPORTED;
  if (page_size != 64 && page_size != 128) return MALA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_out_pages_per_seq) * page_size < budget) return MALA_ERR_INVALID_ARG;
  const long long most = std::max(num_pages, num_out_pages);
  if (static_cast<long long>(max_pages_per_seq) * page_size >= (1ll << 31) || most * page_size >= (1ll << 31) ||
      most * page_size * Hkv * d >= (1ll << 40) || B > 65535)
    return MALA_ERR_UNSUPPORTED;
  const void* ptrs[] = {k_pages, v_pages, k_out_pages, v_out_pages};
  for (const void* x : ptrs)
    if ((reinterpret_cast<uintptr_t>(x) & 15u) != 0) return MALA_ERR_UNSUPPORTED;
  return MALA_OK;
}

}  // namespace mala
