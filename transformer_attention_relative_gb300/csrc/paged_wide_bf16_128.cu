// paged_wide_bf16_128.cu -- variants of the wide tree kernel for bf16 caches of head
// dimension 128.

#include "paged_wide.cuh"

namespace relpos {

int paged_wide_bf16_128(const RelposPagedCache& cache, const PagedTreeParams& p, int blocks,
                        void (**combine)(PagedTreeParams), cudaStream_t stream) {
  return launch_wide<128, false>(cache, p, blocks, combine, stream);
}

}  // namespace relpos
