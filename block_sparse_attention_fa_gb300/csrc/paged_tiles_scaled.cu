// paged_tiles_scaled.cu -- many rows over a cache held in 8 bits: not there yet.
#include "paged.cuh"

namespace fa {

cudaError_t launch_paged_tiles_scaled(const PagedScaledParams&, const CUtensorMap&, const CUtensorMap&, cudaStream_t) {
    return cudaErrorNotSupported;
}

}  // namespace fa
