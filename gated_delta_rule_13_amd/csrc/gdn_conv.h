// gdn_conv.h -- the short causal convolution of each channel on gfx950.
//
//     p_t = bias + sum_{j < W} w_j x_{t-W+1+j},   y_t = silu(p_t)
//
// with the W-1 rows before the first token taken from the state.  Memory bounds
// it (x read once, y written once): a thread takes V neighbouring channels (16
// bytes of a row) down a tile of rows, holds the last W-1 rows in registers,
// and has the next kConvRows rows in flight while it works on the current ones.
// Measured at 4 x 4096 x 2048 in bf16, 4 taps: 30 us for 134 MB (4.5 TB/s, where
// a large copy reaches 5.1).
#pragma once
#include <type_traits>

#include "gdn_layer.h"

namespace gdn {

struct ConvParams {
    const void* x;
    const float* w;
    const float* bias;      // may be null
    const void* s0;         // may be null
    const int32_t* lens;    // may be null
    void* y;
    void* s1;               // may be null; may be s0
    int64_t sb, st;         // strides of x
    int B, T, D;
    int hd;                 // channels per head of y
    int nv;                 // vectors per row
    int tile, ntile;        // rows per thread, tiles per sequence
    int silu;
};

constexpr int kConvThreads = 256;
constexpr int kConvRows = 4;

// weights of V neighbouring channels
template <int W, int V>
struct ConvWeights {
    float w[W][V], b[V];
    __device__ __forceinline__ void load(const float* wp, const float* bp, int c) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = wp[(int64_t)(c + v) * W + j];
            b[v] = bp ? bp[c + v] : 0.f;
        }
    }
};

// the row at time t of sequence b: x for t >= 0, the state for t < 0
template <bool BF, int W, int V>
__device__ __forceinline__ void conv_row(Raw<BF, V>& r, const ConvParams& p, int b, int t, int c) {
    if (t >= 0) r.load(p.x, b * p.sb + t * p.st + c);
    else if (p.s0) r.load(p.s0, ((int64_t)b * (W - 1) + (t + W - 1)) * p.D + c);
    else r.zero();
}

template <bool BF, int W, int V>
__global__ __launch_bounds__(kConvThreads) void gdn_conv_fwd_kernel(ConvParams p) {
    const unsigned id = blockIdx.x * kConvThreads + threadIdx.x;
    const unsigned row_tile = id / (unsigned)p.nv;
    const int c = (int)(id % (unsigned)p.nv) * V;
    const int b = (int)(row_tile / (unsigned)p.ntile);
    if (b >= p.B) return;
    const int t0 = (int)(row_tile % (unsigned)p.ntile) * p.tile;
    const int n = seq_len(p.lens, b, p.T);
    const int tz = t0 + p.tile < p.T ? t0 + p.tile : p.T;
    const int t1 = tz < n ? tz : n;

    ConvWeights<W, V> wt;
    wt.load(p.w, p.bias, c);
    const int head = c / p.hd;
    const int64_t y0 = ((int64_t)b * (p.D / p.hd) + head) * p.T * p.hd + (c - head * p.hd);

    // rows t0 - W + 1 .. t0 - 1, then the chunk's
    Raw<BF, V> win[W - 1 + kConvRows], next[kConvRows];
    if (t0 < n || t0 == 0) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) conv_row<BF, W, V>(win[i], p, b, t0 - W + 1 + i, c);
    }
    // The thread of a sequence's first rows writes its final state too: it
    // alone reads the initial one, and has read it by now, so the two may be
    // the same buffer.
    Raw<BF, V> last[W - 1];
    if (t0 == 0 && p.s1) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int t = n - W + 1 + i;
            last[i] = win[0];
            if (t >= 0) last[i].load(p.x, b * p.sb + t * p.st + c);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                if (t + W - 1 == k) last[i] = win[k];
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float f[V];
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = last[i].get(v);
            store_vec<BF, V>(p.s1, ((int64_t)b * (W - 1) + i) * p.D + c, f);
        }
    }
    if (t0 < t1) {
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) next[i].load(p.x, b * p.sb + (t0 + i < t1 ? t0 + i : t1 - 1) * p.st + c);
    }
    for (int t = t0; t < t1; t += kConvRows) {
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) win[W - 1 + i] = next[i];
        if (t + kConvRows < t1) {
#pragma unroll
            for (int i = 0; i < kConvRows; ++i) {
                const int tt = t + kConvRows + i;
                next[i].load(p.x, b * p.sb + (tt < t1 ? tt : t1 - 1) * p.st + c);
            }
        }
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) {
            if (t + i < t1) {
                float f[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float a = wt.b[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) a = fmaf(wt.w[j][v], win[i + j].get(v), a);
                    const float act = silu(a);
                    f[v] = p.silu ? act : a;
                }
                store_vec<BF, V>(p.y, y0 + (int64_t)(t + i) * p.hd, f);
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) win[i] = win[kConvRows + i];
    }
    float zero[V];
#pragma unroll
    for (int v = 0; v < V; ++v) zero[v] = 0.f;
    for (int t = t0 > t1 ? t0 : t1; t < tz; ++t) store_vec<BF, V>(p.y, y0 + (int64_t)t * p.hd, zero);
}

// ---------------------------------------------------------------------------
// Gradient.  With dp_t = dy_t silu'(p_t) (zero outside the sequence):
//     dx_t = sum_j w_j dp_{t+W-1-j}   (t < 0: the initial state's rows)
//     dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t
// A wave takes 64 V channels down `tile` rows and W-1 more, whose dp its last
// rows need (computed again by the next tile's wave).  x and dy are read
// once and dx written once, which bounds it.  The sums over rows stay in
// registers, are added over the workgroup's tiles in LDS, and written as one
// row of partial sums for each workgroup.  Measured at 4 x 4096 x 2048 in bf16,
// 4 taps: 53 us for 201 MB and 5 us for the sum of the partial rows.  It moves
// 267 MB (5.0 TB/s, the rate of a large copy): 21 are the rows before and behind
// a tile, 41 cache lines that two workgroups share, whose L2s differ, where x's
// rows begin within a line (155 MB read for 196, and 45 us for 49 in one
// measurement, where they do not).  44 vector instructions an element keep the
// vector units busy 76 % of the time, so the waves matter too: two channels to a
// thread (119 registers, four waves on a vector unit) took 52 us where four (205
// registers) took 59 and eight spilled; branches on the activation and at the
// ends of tiles inside the row loop cost 8 us more.
struct ConvBwdParams {
    ConvParams f;
    const void* dy;
    const void* ds1;        // gradient of the final state, may be null
    void* dx;
    void* ds0;              // may be null
    float* part;            // [rows of workgroups][D * W + D]
};

constexpr int kConvBwdV = 2;                                 // channels per thread (wide)
constexpr int kConvBwdTiles = kConvThreads / 64;             // tiles per workgroup, one for each wave

template <bool BF, int W, int V>
__global__ __launch_bounds__(kConvThreads) void gdn_conv_bwd_kernel(ConvBwdParams q) {
    const ConvParams& p = q.f;
    constexpr uint32_t E = BF ? 2 : 4;
    __shared__ float red[kConvBwdTiles][64][(W + 1) * V + 1];
    const int ncb = (p.nv + 63) / 64;
    const int lane = threadIdx.x & 63, tl = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c0 = (int)(blockIdx.x % (unsigned)ncb) * 64 * V, c = c0 + lane * V;
    const int row_tile = (int)(blockIdx.x / (unsigned)ncb) * kConvBwdTiles + tl;

    float acc[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[j][v] = 0.f;

    if (c < p.D && row_tile < p.B * p.ntile) {
        const int b = row_tile / p.ntile;
        const int t0 = row_tile % p.ntile * p.tile;
        const int n = seq_len(p.lens, b, p.T);
        const int tz = t0 + p.tile < p.T ? t0 + p.tile : p.T;   // dx rows [t0, tz)
        const int t1 = tz < n ? tz : n;                         // tokens of its own
        const int t2 = tz + W - 1 < n ? tz + W - 1 : n;         // tokens whose dp it needs
        ConvWeights<W, V> wt;
        wt.load(p.w, p.bias, c);
        const int head = c / p.hd;
        const uint32_t off = (uint32_t)c * E;                   // (rows of 2 GiB are refused)
        const char* xr = row_at<BF>(p.x, b * p.sb);
        const int64_t xs = p.st * E;
        // dy: the lane's head starts p.T * p.hd elements after the one before
        const char* gr = row_at<BF>(q.dy, (int64_t)b * p.T * p.D);
        const int64_t goff = ((int64_t)head * p.T * p.hd + (c - head * p.hd)) * E;
        char* dr = row_at<BF>(q.dx, (int64_t)b * p.T * p.D);
        const int64_t gs = (int64_t)p.hd * E, ds = (int64_t)p.D * E;

        Raw<BF, V> win[W - 1 + kConvRows], nx[kConvRows], ng[kConvRows];
        float dp[W - 1 + kConvRows][V];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            if (t0 < t2) conv_row<BF, W, V>(win[i], p, b, t0 - W + 1 + i, c);
            else win[i].zero();
#pragma unroll
            for (int v = 0; v < V; ++v) dp[i][v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) {
            if (t0 < t2) {
                const int tt = t0 + i < t2 ? t0 + i : t2 - 1;
                nx[i].load_at(xr + tt * xs, off);
                ng[i].load(gr + tt * gs + goff, 0);
            } else {
                nx[i].zero();
                ng[i].zero();
            }
        }
        // dx rows t - W + 1 .. t - W + kConvRows follow from the dp up to t + kConvRows - 1
        for (int t = t0; t < tz + W - 1; t += kConvRows) {
            Raw<BF, V> g[kConvRows];
#pragma unroll
            for (int i = 0; i < kConvRows; ++i) {
                win[W - 1 + i] = nx[i];
                g[i] = ng[i];
            }
            if (t + kConvRows < t2) {
#pragma unroll
                for (int i = 0; i < kConvRows; ++i) {
                    const int tt = t + kConvRows + i < t2 ? t + kConvRows + i : t2 - 1;
                    nx[i].load_at(xr + tt * xs, off);
                    ng[i].load(gr + tt * gs + goff, 0);
                }
            }
            // EDGE: rows at the ends of the tile or the sequence are among them
            auto rows = [&](auto edge) {
                constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
                for (int i = 0; i < kConvRows; ++i) {
                    const int td = t + i - (W - 1);
                    // (rows behind t2 repeat the last one: their dp is 0)
                    const bool live = !EDGE || t + i < t2, mine = !EDGE || t + i < t1;
                    float f[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float a = wt.b[v], val, slope;
#pragma unroll
                        for (int j = 0; j < W; ++j) a = fmaf(wt.w[j][v], win[i + j].get(v), a);
                        silu_both(a, val, slope);
                        const float d = g[i].get(v) * (p.silu ? slope : 1.f);
                        dp[W - 1 + i][v] = live ? d : 0.f;
                        // (a row of another tile, or a repeated one, may be infinite: 0 in its
                        // place; a branch here takes the product into dbias' sum unrounded)
                        const float own = mine ? d : 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[j][v] = fmaf(own, mine ? win[i + j].get(v) : 0.f, acc[j][v]);
                        acc[W][v] += own;
                        f[v] = 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) f[v] = fmaf(wt.w[j][v], dp[i + W - 1 - j][v], f[v]);
                    }
                    if (!EDGE) {
                        store_at<BF, V>(dr + td * ds, off, f);
                    } else if (td >= t0 ? td < tz : (td < 0 && t0 == 0)) {
                        // the final state's rows are those at times n - W + 1 .. n - 1
                        const int k = td - (n - (W - 1));
                        if (q.ds1 && k >= 0 && td < n) {
                            Raw<BF, V> e;
                            e.load(q.ds1, ((int64_t)b * (W - 1) + k) * p.D + c);
#pragma unroll
                            for (int v = 0; v < V; ++v) f[v] += e.get(v);
                        }
                        if (td >= 0) store_at<BF, V>(dr + td * ds, off, f);
                        else if (q.ds0) store_vec<BF, V>(q.ds0, ((int64_t)b * (W - 1) + td + W - 1) * p.D + c, f);
                    }
                }
            };
            if (t >= t0 + W - 1 && t + kConvRows <= t1 && (!q.ds1 || t + kConvRows <= n - (W - 1))) rows(std::false_type());
            else rows(std::true_type());
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                win[i] = win[kConvRows + i];
#pragma unroll
                for (int v = 0; v < V; ++v) dp[i][v] = dp[kConvRows + i][v];
            }
        }
    }
    // [channel][tap], then the biases, summed over the workgroup's tiles
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j <= W; ++j) red[tl][lane][v * (W + 1) + j] = acc[j][v];
    __syncthreads();
    float* out = q.part + (int64_t)(blockIdx.x / (unsigned)ncb) * p.D * (W + 1);
    for (int i = threadIdx.x; i < 64 * V * (W + 1); i += kConvThreads) {
        const int ch = i / (W + 1), j = i % (W + 1);
        if (c0 + ch < p.D) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < kConvBwdTiles; ++k) t += red[k][ch / V][(ch % V) * (W + 1) + j];
            out[j < W ? (int64_t)(c0 + ch) * W + j : (int64_t)p.D * W + c0 + ch] = t;
        }
    }
}

}  // namespace gdn
