// Matrix products with bias, activation and residual in the epilogue.
#pragma once

#include "ebin_act.cuh"

namespace ebin {

struct GemmEpilogue {
    const void *bias;       // [n], or null
    const void *residual;   // [m][n], or null
    void *y;
    void *z;                // receives the pre-activation, or null
    int64_t ld_residual, ldy, ldz;
    int32_t bias_f32;
    int32_t act;
};

}  // namespace ebin
