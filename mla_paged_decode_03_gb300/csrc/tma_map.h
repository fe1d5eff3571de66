// Tensor maps of bf16 tensors for TMA tile loads with the 128-byte swizzle.
#pragma once

#include <stdint.h>

#include <cuda.h>

namespace mla {

// The driver encodes tensor maps (looked up once a process).
bool tile_maps_ok();

// A map of `rank` (2 or 3) dimensions, the innermost contiguous: sizes, byte strides of the outer
// ones (multiples of 16), box.  Elements outside the tensor are read as zeros.  False where the
// driver refuses it.
bool encode_tile_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box);

}  // namespace mla
