// Which bytes a warp of the 4-bit product copies of a row of weights or scales.
// Plain C++, so that a test on the host goes through every piece.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SBT_COPY_FN __host__ __device__ __forceinline__
#else
#define SBT_COPY_FN inline
#endif

namespace sbt_matvec {

// Bytes of `tile` (at most) that a row of `row` bytes has from byte `at` on; `at` may be past its end.
SBT_COPY_FN int bytes_of(int64_t row, int64_t at, int tile) {
    const int64_t left = row - at;
    return left <= 0 ? 0 : left < tile ? (int)left : tile;
}

// Bytes of the 16-byte piece that starts `c` past the 16-byte boundary before a tile's row.  The row's own `bytes` start
// `shift` past the boundary; the first piece has those before them too, which lie in the same 16.  A row without bytes
// (columns past the last: its address may be past the array) has no piece.
SBT_COPY_FN int piece_of(int bytes, int shift, int c) {
    const int n = shift + bytes - c;
    return bytes == 0 || n <= 0 ? 0 : n < 16 ? n : 16;
}

}  // namespace sbt_matvec
