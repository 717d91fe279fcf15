// paged_wide_e4m3_64.cu -- variants of the wide tree kernel for e4m3 caches of head
// dimension 64.

#include "paged_wide.cuh"

namespace relpos {

int paged_wide_e4m3_64(const RelposPagedCache& cache, const PagedTreeParams& p, int blocks,
                        void (**combine)(PagedTreeParams), cudaStream_t stream) {
  return launch_wide<64, true>(cache, p, blocks, combine, stream);
}

}  // namespace relpos
