// linear_prep.cuh -- what runs before the layer products: operands copied or
// split into what the tensor copies can read, and dz = dy * act'(z) with the
// bias gradient.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace linear_prep {

// `planes` matrices of `outer` rows of `inner` values (row stride ld, plane
// stride plane, in elements), to be copied to dst with rows of up8(inner)
// values.  FP32: as three bf16 pieces, piece i of matrix e at
// dst + (i*planes + e) * outer * up8(inner).
struct Copy {
    const void *src;
    long long ld, plane;
    int inner, outer, planes;
    void *dst;
};
// One or two of them in one launch.
cudaError_t copy_operands(int type, const Copy *copies, int n, cudaStream_t stream);

// Workspace of activation_gradient's column sums.
size_t sums_bytes(int M, int N, int E);

// dz = dy * act'(z) into dz (M rows of N, row stride lddz; FP32: three bf16
// pieces, M*lddz apart; NULL: not wanted), and dbias (E x N; E < 0: one group
// of all rows, no offsets) through the partial sums in `sums` (NULL: not
// wanted).
cudaError_t activation_gradient(int type, int act, int M, int N, int E, const int *offsets, const void *dy,
                                long long lddy, const void *z, long long ldz, void *dz, long long lddz, void *sums,
                                void *dbias, cudaStream_t stream);

}  // namespace linear_prep
