// Shared by the kernels of the attention tally (pkv_tally in include/pkv.h): where a
// token's entry lies, and how a weight enters it.
#pragma once

#include "common.cuh"

namespace pkv {

// Entry of (layer, page, KV head g, token of the page) in weight and origin: a page's
// entries of a head lie together, [NL][pages][Hkv][P].
__device__ __forceinline__ long long tally_at(const pkv_workspace &ws, int n_pages, int layer,
                                              int page, int g, int in_page) {
  return (((long long)layer * n_pages + page) * ws.n_kv_heads + g) * ws.page_size + in_page;
}

// A weight that is NaN or infinite counts as nothing: it would stay in its entry, and
// rank its token, for good.
__device__ __forceinline__ float tally_clean(float w) { return fabsf(w) < INFINITY ? w : 0.f; }

}  // namespace pkv
