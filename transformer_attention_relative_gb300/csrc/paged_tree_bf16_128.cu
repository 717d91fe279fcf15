// paged_tree_bf16_128.cu -- variants of the paged decode kernel for the nodes of a
// drafted tree, bf16 caches of head dimension 128.

#include "paged_decode.cuh"

namespace relpos {

PagedTreeVariant paged_tree_bf16_128(int rows8) {
  return rows8 == 1 ? paged_decode_variant<128, false, 1, 16, 2, PagedTreeParams>()
                    : paged_decode_variant<128, false, 2, 16, 2, PagedTreeParams>();
}

}  // namespace relpos
