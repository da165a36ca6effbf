// linear_few.cuh -- linear_forward for few tokens (a decoding step).
#pragma once

#include <cuda_runtime.h>

#include "linear.h"

namespace linear_few {

// Most tokens that run takes (FP32: beyond it, splitting the operands once for the
// product kernel costs less than splitting them in each CTA).
inline int max_tokens(int type) { return type == LINEAR_F32 ? 64 : 16; }

struct Few {
    int T, F, K;
    const void *x, *w, *bias, *residual;
    void *z, *out;
    long long ldx, ldw, ldr, ldz, ldo;
    int order, act;
    int sms, split;  // of the device; CTAs that share a tile's K (set by run)
};

cudaError_t run(int type, const Few &p, cudaStream_t stream);

}  // namespace linear_few
