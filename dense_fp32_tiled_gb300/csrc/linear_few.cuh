// linear_few.cuh -- linear_forward for few tokens (a decoding step).
#pragma once

#include <cuda_runtime.h>

namespace linear_few {

constexpr int MAX_TOKENS = 16;

struct Few {
    int T, F, K;
    const void *x, *w, *bias, *residual;
    void *z, *out;
    long long ldx, ldw, ldr, ldz, ldo;
    int order, act;
};

cudaError_t run(int type, const Few &p, cudaStream_t stream);

}  // namespace linear_few
