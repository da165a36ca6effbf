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

// Rows of a chunk: activation_gradient leaves, for the bias gradient, the column
// sums of each chunk's rows of each expert, expert e's rows of chunk c in row
// c + e of `sums` (which no other pair of the two shares, as both only grow
// along the rows).
constexpr int CHUNK = 64;

// Expert e's sum of column `col` from those, in chunk order (E < 0: one group).
__device__ __forceinline__ float column_sum(const float *sums, int M, int N, int E, const int *offsets, int e, int col,
                                            int first, int step) {
    int b = 0, end = M;
    if (E >= 0) {
        b = min(max(offsets[e], 0), M);
        end = min(max(offsets[e + 1], b), M);
    }
    float t = 0.0f;
    if (col < N && end > b) {
#pragma unroll 8
        for (int c = b / CHUNK + first; c <= (end - 1) / CHUNK; c += step) t += sums[static_cast<long long>(c + e) * N + col];
    }
    return t;
}

// Workspace of the column sums.
size_t sums_bytes(int M, int N, int E);

// dz = dy * act'(z) into dz (M rows of N, row stride lddz; FP32: three bf16
// pieces, M*lddz apart; NULL: not wanted), and the chunks' column sums into
// `sums` (E < 0: one group of all rows, no offsets; NULL: not wanted).
cudaError_t activation_gradient(int type, int act, int M, int N, int E, const int *offsets, const void *dy,
                                long long lddy, const void *z, long long ldz, void *dz, long long lddz, float *sums,
                                cudaStream_t stream);

// dbias (E x N, or N) from the column sums, where no product follows that adds them on the side.
cudaError_t column_sums(int type, int M, int N, int E, const int *offsets, const float *sums, void *dbias,
                        cudaStream_t stream);

}  // namespace linear_prep
