// paged_decode_e4m3_128.cu -- variants of the paged decode kernel for e4m3 caches of
// head dimension 128.

#include "paged_decode.cuh"

namespace relpos {

PagedDecodeVariant paged_decode_e4m3_128(int rows8) {
  switch (rows8) {
    case 1: return paged_decode_variant<128, true, 1, 32, 2>();
    default: return paged_decode_variant<128, true, 2, 32, 2>();
  }
}

}  // namespace relpos
