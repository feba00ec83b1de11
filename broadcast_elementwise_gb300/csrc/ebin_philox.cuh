// The random words of dropout: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  Shared by the
// dropout kernels and the norms around a block.
#pragma once

#include <cmath>

#include "ebin_layer.h"

namespace ebin {

struct DropArgs {
    uint32_t least;      // words below it drop their element; 0: nothing is dropped
    float scale;         // 1 / (1 - least / 2^32)
    uint32_t key[20];    // the ten rounds' keys
    uint64_t offset;
    const uint64_t *offset_device;   // added to offset, or null
};

// Whether p is a probability that can be drawn, and its bound on words.
inline bool drop_bound(double p, uint32_t *least) {
    if (!(p >= 0.0) || !(p < 1.0)) return false;
    const double l = std::nearbyint(p * 4294967296.0);   // halves to even
    if (l > 4294967295.0) return false;
    *least = (uint32_t)l;
    return true;
}

inline DropArgs drop_args(uint32_t least, uint64_t seed, uint64_t offset,
                          const uint64_t *offset_device) {
    DropArgs d{};
    d.least = least;
    d.scale = (float)(1.0 / (1.0 - (double)least / 4294967296.0));
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    for (int r = 0; r < 10; ++r) {
        d.key[2 * r] = k0;
        d.key[2 * r + 1] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    d.offset = offset;
    d.offset_device = offset_device;
    return d;
}

#ifdef __CUDACC__
// The call's offset; after the wait for the launch before it.
__device__ __forceinline__ uint2 drop_offset(const DropArgs &d) {
    const uint64_t o = d.offset + (d.least && d.offset_device ? *d.offset_device : 0);
    return make_uint2((uint32_t)o, (uint32_t)(o >> 32));
}

// The words of columns 4 quad .. 4 quad + 3 of a row: 20 wide products and as
// many three-way exclusive ors, the keys read from the constant bank.
__device__ __forceinline__ uint4 drop_words(const DropArgs &d, uint32_t quad, uint32_t row,
                                            uint2 offset) {
    uint32_t c0 = quad, c1 = row, c2 = offset.x, c3 = offset.y;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ d.key[2 * r];
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ d.key[2 * r + 1];
        c3 = (uint32_t)a;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Four elements: what is kept times the scale, exactly 0 for what is dropped.
__device__ __forceinline__ void drop_quad(const DropArgs &d, uint32_t quad, uint32_t row,
                                          uint2 offset, float *x) {
    const uint4 w = drop_words(d, quad, row, offset);
    x[0] = w.x >= d.least ? x[0] * d.scale : 0.0f;
    x[1] = w.y >= d.least ? x[1] * d.scale : 0.0f;
    x[2] = w.z >= d.least ? x[2] * d.scale : 0.0f;
    x[3] = w.w >= d.least ? x[3] * d.scale : 0.0f;
}
#endif

}  // namespace ebin
