// paged_tree_e4m3_64.cu -- variants of the paged decode kernel for the nodes of a
// drafted tree, e4m3 caches of head dimension 64.

#include "paged_decode.cuh"

namespace relpos {

PagedTreeVariant paged_tree_e4m3_64(int rows8) {
  return rows8 == 1 ? paged_decode_variant<64, true, 1, 32, 2, PagedTreeParams>()
                    : paged_decode_variant<64, true, 2, 32, 2, PagedTreeParams>();
}

}  // namespace relpos
