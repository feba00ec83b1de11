// CPU model of the copies that bring rows off the vectors to shared memory, driven by the
// schedule the kernel follows (ebin_block_copy.h).  See test_row_copies.py.
#include <cstdint>
#include <vector>

#include "ebin_block_copy.h"

using namespace ebin;

// Rows of n elements of `size` bytes, `ld` apart from address `base` on; a lane copies pieces
// of C columns (8, or two of 4 that lie 128 apart), a chunk is 256 columns.  rule 0: the
// kernel's; 1: whole vectors everywhere; 2: only the first and the last row are looked at.
// outside: bytes read beyond the tensor; missing: bytes of rows that are not where a lane
// reads them.
extern "C" void row_copies(int size, int C, int64_t rows, int64_t n, int64_t ld, uintptr_t base,
                           int rule, int64_t *outside, int64_t *missing) {
    const int bytes = C * size, P = 8 / C;
    const uintptr_t first = base, last = base + ((rows - 1) * ld + n) * size;
    *outside = *missing = 0;
    for (int64_t r = 0; r < rows; ++r) {
        const uintptr_t row = base + r * ld * size;
        const bool edge = rule == 0 ? row_at_edge((int)r, (int)rows)
                        : rule == 2 && (r == 0 || r == rows - 1);
        for (int64_t chunk = 0; chunk < n; chunk += 256) {
            // what lies at each byte of the chunk's buffer: an address, or 0
            std::vector<uintptr_t> buffer(256 * size + 16, 0);
            int past = 0;
            for (int lane = 0; lane < 32; ++lane) {
                const uintptr_t mine = row + (chunk + lane * C) * size;
                past = (int)(mine & (uintptr_t)(bytes - 1));
                for (int q = 0; q < P; ++q) {
                    const int at = (int)(chunk + lane * C + q * 128) * size - past;
                    const int count = row_vectors(at, bytes, (int)n * size,
                                                  q == P - 1 && lane == 31);
                    for (int k = 0; k < count; ++k) {
                        const int to = lane * bytes + q * 128 * size + k * bytes;
                        const uintptr_t from = mine - past + q * 128 * size + k * bytes;
                        auto put = [&](int b, int count) {
                            for (int i = b; i < b + count; ++i) {
                                *outside += from + i < first || from + i >= last;
                                buffer[to + i] = from + i;
                            }
                        };
                        if (edge)
                            copy_within(from, bytes, size, first, last, [&] { put(0, bytes); },
                                        [&](int b) { put(b, size); });
                        else
                            put(0, bytes);
                    }
                }
            }
            // a lane reads the piece `past` bytes behind its place
            const int64_t columns = n - chunk < 256 ? n - chunk : 256;
            for (int64_t b = 0; b < columns * size; ++b)
                *missing += buffer[b + past] != row + chunk * size + b;
        }
    }
}
