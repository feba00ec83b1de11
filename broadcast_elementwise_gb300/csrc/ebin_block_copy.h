// Which vectors of a row a lane copies to shared memory where rows lie off the vectors, as
// plain C++: ebin_block_unit.cuh follows it.
//
// A piece's copy begins on the vector that holds its first element, so the vectors at
// a row's two ends hold bytes of its neighbours, and those of a tensor's first and last rows
// bytes that are not the tensor's: such a vector goes element by element.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define EBIN_COPY_FN __device__ __forceinline__
#else
#define EBIN_COPY_FN inline
#endif

namespace ebin {

// Vectors from byte `at` of a row on: one, or two for the last lane of a chunk, of which
// each holds some of the row.
EBIN_COPY_FN int row_vectors(int at, int bytes, int row_bytes, bool last_lane) {
    return at >= row_bytes ? 0 : last_lane && at + bytes < row_bytes ? 2 : 1;
}

// Whether a vector of the row may leave the tensor.  Rows start two bytes apart at least and a
// vector passes an end of its row by at most 14, so from the eighth row on none begins before the
// first row, and none ends behind the last one but for the last eight.
EBIN_COPY_FN bool row_at_edge(int row, int rows) { return row < 8 || row >= rows - 8; }

// The vector at `low`, `bytes` long: whole() where it lies in [first, last), else one(byte) for
// each of its elements of `size` bytes there.
template <class Whole, class One>
EBIN_COPY_FN void copy_within(uintptr_t low, int bytes, int size, uintptr_t first, uintptr_t last,
                              const Whole &whole, const One &one) {
    if (low >= first && low + bytes <= last) {
        whole();
        return;
    }
    for (int b = 0; b < bytes; b += size)
        if (low + b >= first && low + b < last) one(b);
}

}  // namespace ebin
