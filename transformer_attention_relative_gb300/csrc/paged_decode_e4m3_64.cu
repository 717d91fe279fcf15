// paged_decode_e4m3_64.cu -- variants of the paged decode kernel for e4m3 caches of
// head dimension 64.

#include "paged_decode.cuh"

namespace relpos {

PagedDecodeVariant paged_decode_e4m3_64(int rows8) {
  switch (rows8) {
    case 1: return paged_decode_variant<64, true, 1, 32, 2>();
    case 2: return paged_decode_variant<64, true, 2, 32, 2>();
    case 3: return paged_decode_variant<64, true, 3, 32, 2>();
    default: return paged_decode_variant<64, true, 4, 32, 2>();
  }
}

}  // namespace relpos
