// paged_wide_bf16_64.cu -- variants of the wide tree kernel for bf16 caches of head
// dimension 64.

#include "paged_wide.cuh"

namespace relpos {

int paged_wide_bf16_64(const RelposPagedCache& cache, const PagedTreeParams& p, int blocks,
                        void (**combine)(PagedTreeParams), cudaStream_t stream) {
  return launch_wide<64, false>(cache, p, blocks, combine, stream);
}

}  // namespace relpos
