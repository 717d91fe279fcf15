// paged_decode_bf16_128.cu -- variants of the paged decode kernel for bf16 caches of
// head dimension 128.

#include "paged_decode.cuh"

namespace relpos {

PagedDecodeVariant paged_decode_bf16_128(int rows8) {
  switch (rows8) {
    case 1: return paged_decode_variant<128, false, 1, 16, 2>();
    default: return paged_decode_variant<128, false, 2, 16, 2>();
  }
}

}  // namespace relpos
