// mx_copy.h -- where the MXFP4 tiles' copies read (mx_tile.h): the lane offset and the
// scalar offset of one raw buffer load, for the host compiler too.
//
// The range check of a raw buffer load looks at the lane offset; the scalar offset is
// added behind it. So token rows and their scales, which are copied two and four chunks at
// a time and may end inside such a unit, have their whole address in the lane offset: what lies
// behind the readable bytes is refused, and reads as zeros. A scalar offset is taken only
// by the weights, whose every piece lies whole inside the matrix.
#pragma once

#include <cstdint>

namespace moeblk {

constexpr uint32_t kMxPast = 1u << 31;  // a lane offset behind every buffer

struct MxCopy {
  uint32_t lane, scalar;
};

// n chunks from c0 on; `row`: the lane's offset to chunk 0 of its token, below 2^31

// chunks 2 u, 2 u + 1 of them, 64 bytes each
__host__ __device__ inline MxCopy mx_x_copy(uint32_t row, int c0, int n, int u) {
  return {row + (2 * u < n ? static_cast<uint32_t>(c0 + 2 * u) * 64u : kMxPast), 0};
}
// the scale words of chunks 4 v .. 4 v + 3
__host__ __device__ inline MxCopy mx_s_copy(uint32_t row, int c0, int n, int v) {
  return {row + (4 * v < n ? static_cast<uint32_t>(c0 + 4 * v) * 4u : kMxPast), 0};
}
// `lane`: the lane's offset in the piece that starts `piece` bytes into the tile of row
// block rb (the last of `blocks` at most), chunk k
__host__ __device__ inline MxCopy mx_w_copy(uint32_t lane, int c0, int n, int k, int Kc, int rb, int blocks,
                                            int tile_bytes, int piece) {
  const int c = c0 + k < Kc ? c0 + k : Kc - 1, b = rb < blocks ? rb : blocks - 1;
  return {lane + (k < n ? 0u : kMxPast), static_cast<uint32_t>((b * Kc + c) * tile_bytes + piece)};
}

}  // namespace moeblk
