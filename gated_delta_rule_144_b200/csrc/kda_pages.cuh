// Pages of a pool of states.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// Page dst[i] <- page src[i] (-1: zeros) of pool [layers][pages][page_bytes], i < n; dst[i] = -1
// does nothing. Conflicting or out-of-range pairs are left out and set DEV_BAD_INDEX.
cudaError_t launch_page_copy(void* pool, const int32_t* src, const int32_t* dst, int n, int layers,
                             int pages, long long page_bytes, unsigned* err, cudaStream_t stream);

}  // namespace kda
