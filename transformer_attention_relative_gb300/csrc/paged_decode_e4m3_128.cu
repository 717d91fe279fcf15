// paged_decode_e4m3_128.cu -- variants of the paged decode kernel for e4m3 caches of
// head dimension 128. Two ring stages: three took 1 to 5 percent longer (fewer
// blocks of an SM, the same bytes in flight).

#include "paged_decode.cuh"

namespace relpos {

PagedDecodeVariant paged_decode_e4m3_128(int rows8) {
  return rows8 == 1 ? paged_decode_variant<128, true, 1, 32, 2>() : paged_decode_variant<128, true, 2, 32, 2>();
}

}  // namespace relpos
