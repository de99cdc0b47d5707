// Tensor maps of microscaled 4-bit matrices.
#pragma once
#include <cuda.h>
#include <cstdint>

namespace sdv2 {

// Codes of `rows` rows of `tiles` tiles: boxes of 128 bytes (256 columns) x box_rows rows, swizzled; what lies outside arrives as 0.
bool mx4_codes_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int tiles, int box_rows);

// Scales: boxes of a tile's 128 words x box_tiles tiles x box_row_tiles; tiles past the matrix's arrive as zeros.
bool mx4_scales_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int tiles, int box_tiles, int box_row_tiles);

}  // namespace sdv2
