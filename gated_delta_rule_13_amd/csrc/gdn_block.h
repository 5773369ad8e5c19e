// gdn_block.h -- the norms after and before a block, with the block's gate, the
// scale of its part and the residual stream between them, on gfx950.
//
//     n = o / sqrt(mean(o^2) + eps) w_post  (or n = o),   x' = x + s act(g) n
//     y = x' / sqrt(mean(x'^2) + eps) w_pre
//
// and the gradient, with rows x^ = x' r', o^ = o r (r, r' the factors 1 /
// sqrt(..)), from the gradients dx' and dy:
//     dX = dx' + r' (dy w_pre - x^ mean(dy w_pre x^))         (is dx)
//     ds = sum dX act(g) n,   dg = dX s n act'(g),   dn = dX s act(g)
//     do = r (dn w_post - o^ mean(dn w_post o^)),   dw_post = sum dn o^,   dw_pre = sum dy x^
// One pass over memory bounds both: 4 x 4096 x 2048 (x fp32, o bf16, gated) take
// 92 us for 470 MB (5.1 TB/s), the gradient 150 for 738 (4.9).  L lanes hold a row in registers, K pieces of
// V numbers to a lane, the next row's loads in flight, and their columns of the
// weights for all the rows that they take.
#pragma once
#include "gdn_layer.h"

namespace gdn {

struct BlockParams {
    const void* o;
    const void* x;          // the stream before the block; in the gradient behind it
    const void* g;          // may be null
    const float* w_post;    // may be null
    const float* scale;     // may be null
    const float* w_pre;     // may be null
    int64_t osb, ost, xsb, xst, gsb, gst;
    void* x_out;
    void* y;                // null: no norm before the next block
    int64_t rows;           // B T
    int T, D;
    int post, act;          // act: 0 the gate as it is, 1 sigmoid, 2 SiLU
    float eps;
};
struct BlockBwdParams {
    BlockParams f;
    const void* dx_out;     // may be null
    const void* dy;         // may be null
    void* dx;
    void* dO;
    void* dg;               // null without a gate
    float* part;            // [blocks][w_post | scale | w_pre][D]
};

constexpr int kBlockMaxD = 16384;
// Lanes to a row.
constexpr int block_lanes(int D) { return D <= 1024 ? 64 : D <= 4096 ? 256 : D <= 8192 ? 512 : 1024; }
template <int L>
constexpr int block_threads() { return L > 256 ? L : 256; }

// Sums of N numbers over a row's lanes, in every lane; where the row is the
// workgroup's, the waves' sums in order, through two slots in turn (a wave that
// writes one again has passed the barrier behind the other).
template <int L, int N>
struct BlockSum {
    float (*slots)[L / 64][N];
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lanes_sum<64>(v[i]);
        if constexpr (L > 64) {
            float (*s)[N] = slots[turn];
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) s[threadIdx.x >> 6][i] = v[i];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i] = 0.f;
#pragma unroll
                for (int k = 0; k < L / 64; ++k) v[i] += s[k][i];
            }
        }
    }
};

// act(g) and act'(g).
__device__ __forceinline__ void block_gate(float g, int act, float& val, float& slope) {
    if (act == 2) {
        silu_both(g, val, slope);
    } else if (act == 1) {
        // (from e^-|g|: no cancellation on either side)
        const float e = exp2_hw(-kLog2e * __builtin_fabsf(g)), r = rcp_hw(1.f + e), er = e * r;
        val = g < 0.f ? er : r;
        slope = er * r;
    } else {
        val = g;
        slope = 1.f;
    }
}

template <bool XB, bool OB, int L, int K, int V>
struct BlockRow {
    Raw<OB, V> o[K], g[K];
    Raw<XB, V> x[K];
    __device__ __forceinline__ void load(const BlockParams& p, int64_t row, int j) {
        const int64_t b = row / p.T, t = row - b * p.T;
        const char* po = row_at<OB>(p.o, b * p.osb + t * p.ost);
        const char* px = row_at<XB>(p.x, b * p.xsb + t * p.xst);
        const char* pg = p.g ? row_at<OB>(p.g, b * p.gsb + t * p.gst) : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            o[k].zero();
            g[k].zero();
            x[k].zero();
            if (c < p.D) {
                o[k].load_at(po, c * (OB ? 2 : 4));
                x[k].load_at(px, c * (XB ? 2 : 4));
                if (pg) g[k].load_at(pg, c * (OB ? 2 : 4));
            }
        }
    }
};
template <int L, int K, int V>
__device__ __forceinline__ void block_columns(float (&w)[K][V], const float* src, int D, int j) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * L + j) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) w[k][e] = src && c < D ? src[c + e] : 1.f;
    }
}

template <bool XB, bool OB, int L, int K, int V>
__global__ __launch_bounds__(block_threads<L>()) void gdn_block_fwd_kernel(BlockParams p) {
    constexpr int kGroups = block_threads<L>() / L;
    __shared__ float slots[2][L / 64][1];
    BlockSum<L, 1> sum{slots};
    const int j = threadIdx.x % L, grp = __builtin_amdgcn_readfirstlane(threadIdx.x / L);
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int64_t row = (int64_t)blockIdx.x * kGroups + grp;
    if (row >= p.rows) return;      // (a whole row's lanes)
    const float inv = 1.f / (float)p.D;
    float wp[K][V], sc[K][V], wn[K][V];
    block_columns<L, K, V>(wp, p.w_post, p.D, j);
    block_columns<L, K, V>(sc, p.scale, p.D, j);
    block_columns<L, K, V>(wn, p.w_pre, p.D, j);
    BlockRow<XB, OB, L, K, V> cur, next;
    next.load(p, row, j);
    for (; row < p.rows; row += step) {
        cur = next;
        if (row + step < p.rows) next.load(p, row + step, j);
        float s[1], r = 1.f;
        if (p.post) {
            s[0] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) s[0] = fmaf(cur.o[k].get(e), cur.o[k].get(e), s[0]);
            sum(s);
            r = 1.f / sqrtf(s[0] * inv + p.eps);
        }
        float x[K][V];
        s[0] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float a = 1.f, slope;
                if (p.g) block_gate(cur.g[k].get(e), p.act, a, slope);
                const float n = cur.o[k].get(e) * r * wp[k][e];
                x[k][e] = c < p.D ? fmaf(sc[k][e] * a, n, cur.x[k].get(e)) : 0.f;
                s[0] = fmaf(x[k][e], x[k][e], s[0]);
            }
            if (c < p.D) store_vec<XB, V>(p.x_out, row * p.D + c, x[k]);
        }
        if (p.y) {
            sum(s);
            r = 1.f / sqrtf(s[0] * inv + p.eps);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * L + j) * V;
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = x[k][e] * r * wn[k][e];
                if (c < p.D) store_vec<OB, V>(p.y, row * p.D + c, f);
            }
        }
    }
}

template <bool XB, bool OB, int L, int K, int V>
__global__ __launch_bounds__(block_threads<L>()) void gdn_block_bwd_kernel(BlockBwdParams q) {
    const BlockParams& p = q.f;
    constexpr int kGroups = block_threads<L>() / L;
    __shared__ float slots3[2][L / 64][3], slots1[2][L / 64][1];
    __shared__ float red[kGroups > 1 ? kGroups : 1][kGroups > 1 ? L * K * V : 1];
    BlockSum<L, 3> sum3{slots3};
    BlockSum<L, 1> sum1{slots1};
    const int j = threadIdx.x % L, grp = __builtin_amdgcn_readfirstlane(threadIdx.x / L);
    const int64_t step = (int64_t)gridDim.x * kGroups;
    const float inv = 1.f / (float)p.D;
    // (many numbers a lane in a large workgroup leave no registers for the
    // weights, which come from the caches again for each row, and then none for
    // the next row)
    constexpr bool kLean = (L == 512 && K * V > 12) || L > 512, kAhead = !kLean;
    float wp[K][V], sc[K][V], wn[K][V], ap[K][V], as[K][V], an[K][V];
    if constexpr (!kLean) {
        block_columns<L, K, V>(wp, p.w_post, p.D, j);
        block_columns<L, K, V>(sc, p.scale, p.D, j);
        block_columns<L, K, V>(wn, p.w_pre, p.D, j);
    }
    auto column = [&](const float* src, const float (&w)[K][V], int k, int e) __attribute__((always_inline)) {
        if constexpr (!kLean) return w[k][e];
        const int c = (k * L + j) * V;
        return src && c < p.D ? src[c + e] : 1.f;
    };
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) ap[k][e] = as[k][e] = an[k][e] = 0.f;
    int64_t row = (int64_t)blockIdx.x * kGroups + grp;
    BlockRow<XB, OB, L, K, V> cur, next;
    Raw<XB, V> dxc[K], dxn[K];
    Raw<OB, V> dyc[K], dyn[K];
    auto load = [&](int64_t r) __attribute__((always_inline)) {
        next.load(p, r, j);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            dxn[k].zero();
            dyn[k].zero();
            if (c < p.D) {
                if (q.dx_out) dxn[k].load(q.dx_out, r * p.D + c);
                if (q.dy) dyn[k].load(q.dy, r * p.D + c);
            }
        }
    };
    if (kAhead && row < p.rows) load(row);
    for (; row < p.rows; row += step) {
        if constexpr (!kAhead) load(row);
        cur = next;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            dxc[k] = dxn[k];
            dyc[k] = dyn[k];
        }
        if (kAhead && row + step < p.rows) load(row + step);
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float o = cur.o[k].get(e), x = cur.x[k].get(e);
                s[0] = fmaf(o, o, s[0]);
                s[1] = fmaf(x, x, s[1]);
                s[2] = fmaf(dyc[k].get(e) * column(p.w_pre, wn, k, e), x, s[2]);
            }
        sum3(s);
        const float r = p.post ? 1.f / sqrtf(s[0] * inv + p.eps) : 1.f;
        const float rn = 1.f / sqrtf(s[1] * inv + p.eps);
        const float mean = s[2] * rn * inv;     // of dy w_pre x^
        float d[K][V], t[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            float dx[V], dg[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float dy = dyc[k].get(e);
                float a = 1.f, slope = 0.f;
                if (p.g) block_gate(cur.g[k].get(e), p.act, a, slope);
                dx[e] = dxc[k].get(e);
                if (q.dy) {
                    const float xh = cur.x[k].get(e) * rn;
                    dx[e] = fmaf(rn, fmaf(-xh, mean, dy * column(p.w_pre, wn, k, e)), dx[e]);
                    an[k][e] = fmaf(dy, xh, an[k][e]);
                }
                const float oh = cur.o[k].get(e) * r, wpk = column(p.w_post, wp, k, e), n = oh * wpk;
                as[k][e] = fmaf(dx[e] * a, n, as[k][e]);
                const float dxs = dx[e] * column(p.scale, sc, k, e);
                dg[e] = dxs * n * slope;
                d[k][e] = dxs * a;
                if (p.post) {
                    ap[k][e] = fmaf(d[k][e], oh, ap[k][e]);
                    d[k][e] *= wpk;
                    t[0] = fmaf(c < p.D ? d[k][e] : 0.f, oh, t[0]);
                }
            }
            if (c < p.D) {
                store_vec<XB, V>(q.dx, row * p.D + c, dx);
                if (q.dg) store_vec<OB, V>(q.dg, row * p.D + c, dg);
            }
        }
        if (p.post) {
            sum1(t);
            t[0] *= inv;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * L + j) * V;
            if (p.post) {
#pragma unroll
                for (int e = 0; e < V; ++e) d[k][e] = r * fmaf(-cur.o[k].get(e) * r, t[0], d[k][e]);
            }
            if (c < p.D) store_vec<OB, V>(q.dO, row * p.D + c, d[k]);
        }
    }
    float* out = q.part + (int64_t)blockIdx.x * 3 * p.D;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        if (which == 0 ? !p.w_post : which == 1 ? !p.scale : !p.w_pre) continue;
        if constexpr (kGroups > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    red[grp][(k * L + j) * V + e] = which == 0 ? ap[k][e] : which == 1 ? as[k][e] : an[k][e];
            __syncthreads();
            for (int c = threadIdx.x; c < p.D; c += block_threads<L>()) {
                float v = 0.f;
#pragma unroll
                for (int k = 0; k < kGroups; ++k) v += red[k][c];
                out[(int64_t)which * p.D + c] = v;
            }
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * L + j) * V;
                if (c < p.D) store_vec<false, V>(out + (int64_t)which * p.D, c, which == 0 ? ap[k] : which == 1 ? as[k] : an[k]);
            }
        }
    }
}

}  // namespace gdn
