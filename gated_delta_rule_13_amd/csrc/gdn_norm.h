// gdn_norm.h -- normalisation of each head of each token with an activation
// or a gate, on gfx950.
//
//     n = (x - mean) / sqrt(var + eps),  p = n w + b,  y = p act(z) | act(p)
//
// and its gradient, with dp = dy act(z) (or dy act'(p)), dn = dp w:
//     dx = (dn - mean(dn) - n mean(dn n)) / sqrt(var + eps)
// (without the mean(dn) where x is not centred), dw = sum dp n, db = sum dp,
// dz = dy p act'(z).  One pass over x, z and y (and their gradients) bounds
// it: a group of L lanes holds a row of d numbers in registers, K pieces of V
// to a lane, so nothing is read twice; the row's sums are steps between
// neighbouring lanes (and between the waves, where the group is the whole
// workgroup).  L and K are chosen so that the pieces just cover the row (d =
// 192: 16 lanes with 3 pieces of four each, no lane idle); V is 4, or 1 where
// the size or the alignment of rows does not allow pieces.  Measured: 4 x 4096 x
// 16 x 128 from fp32 to bf16 with a gate, 55 us for 268 MB (4.9 TB/s, where a
// large copy reaches 5.1); the gradient at 2 x 1031 x 30 x 192 in bf16, 27 us
// for 119 MB (4.4 TB/s) and 4 us for the sum of the partial rows.  Number by
// number, in bf16 with a gate, 32M numbers in heads of 127 take 43 us where
// those of 128 take 34, and their gradient 102 for 66.
#pragma once
#include "gdn_layer.h"

namespace gdn {

struct NormParams {
    const void* x;
    const float* w;         // may be null
    const float* b;         // may be null
    const void* z;          // may be null
    void* y;
    int64_t xsb, xst, xsg;
    int64_t zsb, zst, zsg;
    int64_t rows;           // B T G
    int T, G, d;
    int center, per_group, silu;
    float eps;
};

struct NormBwdParams {
    NormParams f;
    const void* dy;
    void* dx;
    void* dz;               // may be null
    int64_t dsb, dst, dsg;  // strides of dx
    float* part;            // sums of a head's workgroups: rows of [w | b], see norm_partial
};

constexpr int kNormThreads = 256;
constexpr int kNormMaxD = 4096;

// Workgroups of the gradient that a compute unit holds at once, by the numbers
// in a lane (V K), where they lie two to a register or one, and their types: it
// is launched with as many.
constexpr int kNormResident = 4;
constexpr int norm_resident(bool bf16, int k, int v) {
    return k * v <= 6 || (k * v <= 8 && v == 4 && bf16) ? kNormResident : 3;
}

// Where workgroup blk leaves head g's sums for the weight (which 0) or the
// bias: rows [blk][w of all heads | b of all heads] for weights [G, d], and
// [blk, g][w | b] for weights [d], which are summed over the heads too.
__device__ __forceinline__ float* norm_partial(const NormBwdParams& q, int64_t blk, int g, int which) {
    const int64_t G = q.f.G, d = q.f.d;
    return q.part + (q.f.per_group ? (blk * 2 + which) * G + g : (blk * G + g) * 2 + which) * d;
}

__device__ __forceinline__ void act_both(float x, int act, float& val, float& slope) {
    if (act) {
        silu_both(x, val, slope);
    } else {
        val = x;
        slope = 1.f;
    }
}

// Sum over a group's lanes, in every lane.  Where the group is the workgroup
// the waves' sums are added in order, through two slots in turn: a wave that
// writes one again has passed the barrier behind the other, and so have all
// that read it.
template <int L>
struct GroupSum {
    float (*slots)[kNormThreads / 64];
    int turn = 0;
    __device__ __forceinline__ float operator()(float v) {
        if constexpr (L <= 64) return lanes_sum<L>(v);
        v = lanes_sum<64>(v);
        float* s = slots[turn];
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < kNormThreads / 64; ++i) v += s[i];
        return v;
    }
};

// The mean (0 if not centred) and 1 / sqrt(var + eps) of a row.
template <int L, int K, int V>
__device__ __forceinline__ void row_stats(const float (&x)[K][V], const NormParams& p, int j, GroupSum<L>& sum, float& mean,
                                          float& r) {
    const float inv = 1.f / (float)p.d;
    mean = 0.f;
    if (p.center) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) s += x[k][e];     // (pieces behind the row hold 0)
        mean = sum(s) * inv;
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const bool in = (k * L + j) * V < p.d;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float c = in ? x[k][e] - mean : 0.f;
            s = fmaf(c, c, s);
        }
    }
    r = 1.f / sqrtf(sum(s) * inv + p.eps);
}

// Where the rows of a group lie: it takes every `step`-th token of one head,
// token bt = b T + t, by additions (a division a row instead: 59 us for 52 at 30
// heads of 61 in bf16).
struct NormAt {
    int64_t bt, x, z, y, d; // elements of the row in x, z, y (dy, dz) and dx
    unsigned t;
    __device__ __forceinline__ NormAt(const NormParams& p, int64_t dsb, int64_t dst, int64_t dsg, int64_t token, int g) {
        const int64_t b = token / p.T;
        bt = token;
        t = (unsigned)(token - b * p.T);
        x = b * p.xsb + (int64_t)t * p.xst + g * p.xsg;
        z = b * p.zsb + (int64_t)t * p.zst + g * p.zsg;
        d = b * dsb + (int64_t)t * dst + g * dsg;
        y = (token * p.G + g) * p.d;
    }
};
struct NormStep {
    int64_t bt, x, z, y, d, wx, wz, wd;     // wx, wz, wd: where a sequence ends, on top
    unsigned t, T;
    __device__ __forceinline__ NormStep(const NormParams& p, int64_t dsb, int64_t dst, int64_t step) {
        const int64_t b = step / p.T, tt = step - b * p.T;
        bt = step;
        t = (unsigned)tt;
        T = (unsigned)p.T;
        x = b * p.xsb + tt * p.xst;
        z = b * p.zsb + tt * p.zst;
        d = b * dsb + tt * dst;
        y = step * p.G * p.d;
        wx = p.xsb - p.T * p.xst;
        wz = p.zsb - p.T * p.zst;
        wd = dsb - p.T * dst;
    }
    __device__ __forceinline__ void operator()(NormAt& r) const {
        r.bt += bt;
        r.t += t;
        const bool wrap = r.t >= T;
        r.t -= wrap ? T : 0;
        r.x += x + (wrap ? wx : 0);
        r.z += z + (wrap ? wz : 0);
        r.d += d + (wrap ? wd : 0);
        r.y += y;
    }
};

// One row as it lies in memory.
template <bool XB, bool OB, int L, int K, int V>
struct NormRow {
    Raw<XB, V> x[K];
    Raw<OB, V> z[K], dy[K];
    int64_t y0, d0;
    __device__ __forceinline__ void load(const NormParams& p, const void* dyp, const NormAt& at, int j) {
        y0 = at.y;
        d0 = at.d;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            x[k].zero();
            z[k].zero();
            dy[k].zero();
            if (c < p.d) {
                x[k].load(p.x, at.x + c);
                if (p.z) z[k].load(p.z, at.z + c);
                if (dyp) dy[k].load(dyp, at.y + c);
            }
        }
    }
};
template <int L, int K, int V>
__device__ __forceinline__ void load_columns(float (&w)[K][V], const float* src, const NormParams& p, int g, int j, float none) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + j) * V;
        const int wc = (p.per_group ? g * p.d : 0) + c;   // (weights [G, d] have 2^27 numbers at most)
#pragma unroll
        for (int e = 0; e < V; ++e) w[k][e] = src && c < p.d ? src[wc + e] : none;
    }
}

// A group of lanes takes every `tokens`-th token of one head, so that its
// columns of the weight stay in registers, with the next row in flight.
template <bool XB, bool OB, int L, int K, int V>
__global__ __launch_bounds__(kNormThreads) void gdn_norm_fwd_kernel(NormParams p, int64_t tokens) {
    __shared__ float slots[2][kNormThreads / 64];
    GroupSum<L> sum{slots};
    const int j = threadIdx.x % L;
    const int64_t grp = (int64_t)blockIdx.x * (kNormThreads / L) + threadIdx.x / L;
    const int g = (int)(grp % p.G);
    const int64_t bts = p.rows / p.G;
    int64_t bt = grp / p.G;
    if (bt >= tokens || bt >= bts) return;      // (a whole group of lanes)
    float w[K][V], b[K][V];
    load_columns<L, K, V>(w, p.w, p, g, j, 1.f);
    load_columns<L, K, V>(b, p.b, p, g, j, 0.f);
    NormRow<XB, OB, L, K, V> cur, next;
    NormAt at(p, 0, 0, 0, bt, g);
    const NormStep ahead(p, 0, 0, tokens);
    next.load(p, nullptr, at, j);
    for (; bt < bts; bt += tokens) {
        cur = next;
        ahead(at);
        if (at.bt < bts) next.load(p, nullptr, at, j);
        float x[K][V], mean, r;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) x[k][e] = cur.x[k].get(e);
        row_stats<L, K, V>(x, p, j, sum, mean, r);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            if (c < p.d) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float v = fmaf((x[k][e] - mean) * r, w[k][e], b[k][e]), gate = cur.z[k].get(e);
                    if (p.z) f[e] = v * (p.silu ? silu(gate) : gate);
                    else f[e] = p.silu ? silu(v) : v;
                }
                store_vec<OB, V>(p.y, cur.y0 + c, f);
            }
        }
    }
}

// A workgroup takes rows of one head, so that a lane's columns of the weight
// stay the same and their sums stay in registers until the end.
template <bool XB, bool OB, int L, int K, int V>
__global__ __launch_bounds__(kNormThreads, K * V <= 12 ? norm_resident(XB && OB, K, V) : 1) void gdn_norm_bwd_kernel(NormBwdParams q) {
    const NormParams& p = q.f;
    constexpr int kGroups = kNormThreads / L;
    __shared__ float red[kGroups][L * K * V];
    __shared__ float slots[2][kNormThreads / 64];
    GroupSum<L> sum{slots};
    const int j = threadIdx.x % L, grp = threadIdx.x / L;
    const int g = blockIdx.x % p.G;
    const int64_t blk = blockIdx.x / p.G, nblk = gridDim.x / p.G;
    const int64_t bts = p.rows / p.G, step = nblk * kGroups;
    const float inv = 1.f / (float)p.d;
    float w[K][V], b[K][V], sw[K][V], sb[K][V];
    load_columns<L, K, V>(w, p.w, p, g, j, 1.f);
    load_columns<L, K, V>(b, p.b, p, g, j, 0.f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) sw[k][e] = sb[k][e] = 0.f;
    int64_t bt = blk * kGroups + grp;
    NormRow<XB, OB, L, K, V> cur, next;
    NormAt at(p, q.dsb, q.dst, q.dsg, bt, g);
    const NormStep ahead(p, q.dsb, q.dst, step);
    if (bt < bts) next.load(p, q.dy, at, j);
    for (; bt < bts; bt += step) {
        cur = next;
        ahead(at);
        if (at.bt < bts) next.load(p, q.dy, at, j);
        float x[K][V], dn[K][V], mean, r;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) x[k][e] = cur.x[k].get(e);
        row_stats<L, K, V>(x, p, j, sum, mean, r);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            if (c < p.d) {
                float dz[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float n = (x[k][e] - mean) * r, pv = fmaf(n, w[k][e], b[k][e]), dy = cur.dy[k].get(e);
                    float val, slope;
                    act_both(p.z ? cur.z[k].get(e) : pv, p.silu, val, slope);
                    const float dp = dy * (p.z ? val : slope);
                    dz[e] = dy * pv * slope;
                    sw[k][e] = fmaf(dp, n, sw[k][e]);
                    sb[k][e] += dp;
                    x[k][e] = n;
                    dn[k][e] = dp * w[k][e];
                    s1 += dn[k][e];
                    s2 = fmaf(dn[k][e], n, s2);
                }
                if (p.z && q.dz) store_vec<OB, V>(q.dz, cur.y0 + c, dz);
            }
        }
        s1 = p.center ? sum(s1) * inv : 0.f;
        s2 = sum(s2) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            if (c < p.d) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = r * (dn[k][e] - s1 - x[k][e] * s2);
                store_vec<XB, V>(q.dx, cur.d0 + c, f);
            }
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) red[grp][(k * L + j) * V + e] = which ? sb[k][e] : sw[k][e];
        __syncthreads();
        float* out = norm_partial(q, blk, g, which);
        for (int c = threadIdx.x; c < p.d; c += kNormThreads) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) t += red[k][c];
            out[c] = t;
        }
    }
}

}  // namespace gdn
