// paged_wide_e4m3_128.cu -- variants of the wide tree kernel for e4m3 caches of head
// dimension 128.

#include "paged_wide.cuh"

namespace relpos {

int paged_wide_e4m3_128(const RelposPagedCache& cache, const PagedTreeParams& p, int blocks,
                        void (**combine)(PagedTreeParams), cudaStream_t stream) {
  return launch_wide<128, true>(cache, p, blocks, combine, stream);
}

}  // namespace relpos
