// tensor_map.h - descriptors with which tiles of tokens are copied by one
// instruction.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace mcc1d {

// Tiles of 64 tokens and 64 values of a 16-bit tensor [S,B,heads,n] with these
// strides (S, B, heads; in elements); coordinates are (value, token, head, batch).
// `panels`: with a row's 16-byte pieces exchanged as tensor_core.cuh's panels have them.
// False where it cannot be described: rows off 16 bytes, strides of zero.
bool token_tiles(CUtensorMap *map, const void *at, int64_t S, int64_t B, int64_t heads, int64_t n, const int64_t (&strides)[3], bool panels);

}  // namespace mcc1d
