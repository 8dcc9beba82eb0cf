// The batch attention's kernel for keys that many rows share.
#pragma once

#include "aq_batch.cuh"

namespace aq {

// row_tiles: 1 or 2 tiles of 128 query rows a CTA (2 only for D <= 128).
cudaError_t batch_shared(const BatchParams &p, int row_tiles, int grid, cudaStream_t stream);

}  // namespace aq
