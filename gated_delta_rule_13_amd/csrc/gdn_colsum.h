// gdn_colsum.h -- the sum of partial gradients over the workgroups that left
// them, in a fixed order.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

// out[c] = sum over r of part[r][c], r ascending within each of 16 slices of
// the rows and the slices in order: a fixed order.  Columns [0, n0) go to
// out0, [n0, n0 + n1) to out1 (either may be null).
struct ColsumParams {
    const float* part;
    float* out0;
    float* out1;
    int64_t rows;
    int64_t n0, n1;
};
constexpr int kColsumSlices = 16;

static __global__ __launch_bounds__(64 * kColsumSlices) void gdn_colsum_kernel(ColsumParams p) {
    __shared__ float s[kColsumSlices][64];
    const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int64_t cols = p.n0 + p.n1;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    const int64_t per = (p.rows + kColsumSlices - 1) / kColsumSlices;
    const int64_t r1 = (slice + 1) * per < p.rows ? (slice + 1) * per : p.rows;
    float v = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = slice * per; r < r1; ++r) v += p.part[r * cols + c];
    }
    s[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < cols) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kColsumSlices; ++i) t += s[i][lane];
        if (c < p.n0) {
            if (p.out0) p.out0[c] = t;
        } else if (p.out1) {
            p.out1[c - p.n0] = t;
        }
    }
}

// Threads of a sum over `cols` columns (a launch counts them in 32 bits).
constexpr int64_t colsum_threads(int64_t cols) { return (cols + 63) / 64 * 64 * kColsumSlices; }

inline void launch_colsum(const float* part, int64_t rows, float* out0, int64_t n0, float* out1, int64_t n1,
                          hipStream_t st) {
    ColsumParams p{part, out0, out1, rows, n0, n1};
    hipLaunchKernelGGL(gdn_colsum_kernel, dim3((unsigned)((n0 + n1 + 63) / 64)), dim3(64 * kColsumSlices), 0, st, p);
}

}  // namespace gdn
