// gdn_lin_join.h -- what stands between and behind the passes of linear attention
// (gdn_lin.h): the chain of segments, and the sums of the gradient over tiles,
// heads and tokens.  Launched by the entry points alone, so that one object holds
// these kernels.
#pragma once
#include "gdn_layer.h"

namespace gdn {

// The states that segments start from, in the place of what each adds: X_{j+1}
// = a_j X_j + E_j from the first segment on, or backwards in time.
struct LinChainParams {
    float* sum;             // [B H, nseg, plane]
    const float* decay;     // [B H, nseg]
    const float* first;     // [B H, plane] or null
    int64_t plane;
    int nseg, rev;
};
static __global__ __launch_bounds__(256) void gdn_lin_chain_kernel(LinChainParams p, LinChainParams q) {
    const LinChainParams& c = blockIdx.z ? q : p;
    const int64_t i = blockIdx.x * 256ll + threadIdx.x, bh = blockIdx.y;
    if (i >= c.plane) return;
    float x = c.first ? c.first[bh * c.plane + i] : 0.f;
    for (int s = 0; s < c.nseg; ++s) {
        const int64_t j = bh * c.nseg + (c.rev ? c.nseg - 1 - s : s);
        const float e = c.sum[j * c.plane + i];
        c.sum[j * c.plane + i] = x;
        x = fmaf(exp2_hw(c.decay[j]), x, e);
    }
}

// The decay's gradient: the sums of the passes of dq and dk by tiles of columns.
struct LinDecayParams {
    const float* sums_q;    // [tiles, B H, T]
    const float* sums_k;
    const float* log_alpha;
    int64_t lsb, lsh, lst;
    const int32_t* lens;
    float* out;             // [B, H, T]
    int64_t tokens;         // B H T
    int H, T, tiles;
};
static __global__ __launch_bounds__(256) void gdn_lin_decay_kernel(LinDecayParams p) {
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= p.tokens) return;
    const int64_t bh = i / p.T;
    const int t = (int)(i - bh * p.T), b = (int)(bh / p.H), h = (int)(bh % p.H);
    float r = 0.f;
    // (behind a decay of 0 nothing is left to have a gradient)
    if (t < seq_len(p.lens, b, p.T) && !(p.log_alpha[b * p.lsb + h * p.lsh + t * p.lst] < -150.f / kLog2e)) {
        double s = 0;
        for (int k = 0; k < p.tiles; ++k) s += (double)p.sums_q[k * p.tokens + i] + p.sums_k[k * p.tokens + i];
        r = (float)s;
    }
    p.out[i] = r;
}

// Sums over sequences and tokens of one head's [B, H, T] numbers, in a fixed
// order.
static __global__ __launch_bounds__(1024) void gdn_lin_head_sum_kernel(const float* in, float* out, int B, int H, int T) {
    __shared__ double part[16];
    const int h = blockIdx.x;
    double s = 0;
    for (int b = 0; b < B; ++b)
        for (int t = threadIdx.x; t < T; t += 1024) s += in[((int64_t)b * H + h) * T + t];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double r = 0;
        for (int i = 0; i < 16; ++i) r += part[i];
        out[h] = (float)r;
    }
}

// Sums over the heads that share a head of queries or keys: [B, H, T, d] fp32
// to [B, H / rep, T, d].
struct LinGroupParams {
    const float* in;
    void* out;
    int64_t row;            // T d
    int64_t n;              // B (H / rep) T d
    int rep;
};
template <bool BF>
static __global__ __launch_bounds__(256) void gdn_lin_group_sum_kernel(LinGroupParams p) {
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    if (i >= p.n) return;
    const int64_t head = i / p.row, e = i - head * p.row;
    float s = 0.f;
    for (int r = 0; r < p.rep; ++r) s += p.in[(head * p.rep + r) * p.row + e];
    store_one<BF>(p.out, i, s);
}

}  // namespace gdn
