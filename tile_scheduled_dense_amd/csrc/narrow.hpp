// narrow.hpp -- how much of a narrow matrix the LDS ring may copy.
#pragma once

namespace tg {

// Rows, of K, of a matrix `width` elements wide that the LDS ring takes (grouped_ring.hpp): it
// copies whole chunks of 16 bytes of every K tile but the last, which goes through registers
// element by element.  A chunk that passes a row's end brings the next rows, up to chunk - 1
// elements of them.  Of a width of half a chunk one further row covers them, and every last K
// tile has one; of less (rank 1 of 16 bits: 7 rows) a last tile that K cuts may not, so the
// ring ends with the whole tile before it, itself then through registers, and the cut one
// follows by itself.
constexpr int ring_rows(int K, int width, int tile_k, int chunk) { return 2 * width < chunk ? K - K % tile_k : K; }

}  // namespace tg
