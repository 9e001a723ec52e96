// The tiled layout of a 4-bit matrix for the product of two such matrices: records of 128 rows x 256 elements, one after
// the other along a row of records.  A record is the shared-memory image that tcgen05 reads, so that one bulk copy brings
// it: 128 lines of 128 bytes of codes in the 128-byte swizzle (16-byte piece p of line r at p ^ (r % 8)), then for each 64
// elements 512 bytes of scales, the four of line r at (r % 32) * 16 + (r / 32) * 4.
#pragma once
#include <stddef.h>

namespace vh {

constexpr int kTileRows = 128;
constexpr int kTileElems = 256;
constexpr int kTileCodes = kTileRows * kTileElems / 2;
constexpr int kTileScales = kTileRows * kTileElems / 16;
constexpr int kTileBytes = kTileCodes + kTileScales;

__host__ __device__ constexpr int tiles_per_row(int H) { return (H + kTileElems - 1) / kTileElems; }
// Bytes of the codes and scale of a block of 16 elements (line r, block k) within the record.
__host__ __device__ constexpr int tile_code_at(int r, int k) { return r * 128 + (((k >> 1) ^ (r & 7)) << 4) + (k & 1) * 8; }
__host__ __device__ constexpr int tile_scale_at(int r, int k) {
    return kTileCodes + (k >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (k & 3);
}
inline size_t nvfp4_tiles_bytes(int rows, int H) {
    return ((size_t)rows + kTileRows - 1) / kTileRows * tiles_per_row(H) * kTileBytes;
}

}  // namespace vh
