// Tensor maps of operands for TMA copies.
#pragma once
#include <cuda.h>

namespace sdv2 {

// Encodes a tiled bf16 map with the 128-byte swizzle: `rank` dimensions (elements, innermost first), the strides of
// all but the innermost in bytes, and the box that a copy brings.  Elements outside the tensor arrive as zeros.
bool encode_tensor_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box);

// The same for elements of another type, with or without the swizzle.
bool encode_tensor_map_of(CUtensorMapDataType type, CUtensorMapSwizzle swizzle, CUtensorMap* map, const void* base, int rank,
                          const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box);

}  // namespace sdv2
