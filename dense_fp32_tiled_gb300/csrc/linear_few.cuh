// linear_few.cuh -- linear_forward for few tokens (a decoding step).
#pragma once

#include <cuda_runtime.h>

#include "linear.h"

namespace linear_few {

struct Few {
    int T, F, K;
    const void *x, *w, *bias, *residual;
    void *z, *out;
    long long ldx, ldw, ldr, ldz, ldo;
    int order, act;
    int sms, split;  // of the device; CTAs that share a tile's K (set by run)
};

// Whether run does this product (its sizes, w, x and order are looked at).
bool takes(int type, const Few &p);
cudaError_t run(int type, const Few &p, cudaStream_t stream);

}  // namespace linear_few
