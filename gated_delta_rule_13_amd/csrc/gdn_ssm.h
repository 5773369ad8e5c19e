// gdn_ssm.h -- the selective state space recurrence on gfx950.
//
//     s_t = softplus(dt_t + dt_bias),  u_t = s_t x_t
//     h_t = exp(s_t A) h_{t-1} + u_t Bm_t          (N numbers per channel)
//     y_t = (C_t . h_t + Dskip x_t) silu(z_t)
//
// The decay differs for every channel and state, so a chunk of tokens is no
// product of matrices (unlike the delta rule's): the work is one exponential
// (two issue slots) and four multiply-adds for each (token, channel, state),
// on the vector units, against 8 bytes of memory for each (token, channel) in
// bf16.  With 16 states the vector units bound it: 96 issue slots a (token,
// channel) for the states and about 35 for the step size, gate and skip.
//
// A lane holds one channel with all its states in registers, so the sum over
// states needs no other lane.  Bm_t and C_t are the same for all channels of a
// group: the wave stages them in LDS as fp32, kTok tokens ahead, and every lane
// reads them at the same address (reading none of them changes nothing in the
// time).  A lane for each state instead (16 lanes a channel, no segments below)
// was built and took 231 us or more for what follows in 130, for the moves
// between lanes.
//
// Few channels on long sequences leave the chip empty, so the tokens are cut
// into segments.  The recurrence is linear in the state, and a segment acts
// on the state that enters it as h -> exp(A sum s) h + E, with E its end
// state from zero:
//   gdn_ssm_sum_kernel      E and sum s of every segment (all at once)
//   gdn_ssm_chain_kernel    the state that enters each segment, one after
//                           another
//   gdn_ssm_fwd_kernel      the outputs (all segments at once)
// which costs the exponentials twice.  Measured at 4 x 4096 x 2048 with 16
// states, bf16, gated: 97 + 8 + 130 us (24 segments), the last two thirds of
// what the vector units' issue rate would allow at 2.4 GHz, and at 1 x 32768 x
// 1024: 97 + 16 + 130 us.
#pragma once
#include <type_traits>

#include "gdn_layer.h"

namespace gdn {

struct SsmParams {
    const void* x;
    const void* dt;
    const float* A;
    const void* Bm;
    const void* C;
    const float* Dskip;     // may be null
    const void* z;          // may be null
    const float* dt_bias;   // may be null
    const float* h0;        // may be null
    const int32_t* lens;    // may be null
    void* y;
    float* h_final;         // may be null
    int64_t xsb, xst, dsb, dst, zsb, zst, bsb, bst, csb, cst;
    int B, T, D, N, G;
    int Dg;                 // channels per group
    int tpg;                // tiles of 64 channels per group
    int softplus;
    int wide, wide_out;     // A and h0, h_final in 16-byte pieces (N a multiple of 4, aligned)
    int seg_len, nseg;      // with segments a multiple of kTok
    // segment summaries, in units of (sequence, segment, tile):
    float* sum_e;           // [unit][NS][64]: E, then the state that enters
    float* sum_s;           // [unit][64]: sum of s
    // gradient
    const void* dy;
    const float* dh_final;  // may be null
    void* dx;
    void* ddt;
    void* dz;
    float* dh0;             // may be null
    float* sum_r;           // [unit][NS][64]: R, then the gradient that enters from behind
    float* keep_h;          // [unit][group 1 ..][NS][64]: state from zero at a group's start
    float* keep_s;          // [unit][group 1 ..][64]: sum of s up to there
    float* part_a;          // [sequence, segment][tile][NS][64]: dA
    float* part_d;          // [sequence, segment][tile][2][64]: dDskip, ddt_bias
    float* part_bc;         // [tile][sequence][token][2][NS]: dB, dC over a tile's channels
};

constexpr int kTok = 8;                              // tokens staged at a time (a group)

// Where a wave works: its sequence, segment and channels.
struct SsmPlace {
    int b, seg, tile, g, c;  // c: channel of the lane (clamped), of all D
    int c0;                  // the wave's first channel
    bool on;                 // the lane has a channel of its own
    int t0, t1, tz;          // tokens [t0, t1), padded rows [max(t0, t1), tz)
    int64_t unit;
};
__device__ __forceinline__ SsmPlace ssm_place(const SsmParams& p, unsigned id, int nseg, int lane) {
    SsmPlace w;
    const unsigned tiles = (unsigned)(p.G * p.tpg);
    w.tile = (int)(id % tiles);
    const unsigned bs = id / tiles;
    w.seg = (int)(bs % (unsigned)nseg);
    w.b = (int)(bs / (unsigned)nseg);
    w.g = w.tile / p.tpg;
    const int c = (w.tile % p.tpg) * 64 + lane;
    w.on = c < p.Dg;
    w.c = w.g * p.Dg + (w.on ? c : p.Dg - 1);
    w.c0 = w.g * p.Dg + (w.tile % p.tpg) * 64;
    const int n = seq_len(p.lens, w.b, p.T);
    w.t0 = w.seg * p.seg_len;
    w.tz = p.T - w.t0 < p.seg_len ? p.T : w.t0 + p.seg_len;
    w.t1 = w.tz < n ? w.tz : n;
    w.unit = ((int64_t)w.b * p.nseg + w.seg) * tiles + w.tile;
    return w;
}

// Bm and C of kTok tokens, spread over the wave's lanes: value i of lane l is
// number l + 64 i of [token][Bm | C][NS]; 0 behind the N states and behind t1.
template <bool BF, int NS>
struct StagedBC {
    static constexpr int kEach = kTok * 2 * NS / 64;
    Raw<BF, 1> v[kEach];
    __device__ __forceinline__ void load(const SsmParams& p, const SsmPlace& w, int t, int lane) {
        constexpr uint32_t E = BF ? 2 : 4;
        const buf_t bb = buffer_from(row_at<BF>(p.Bm, w.b * p.bsb + t * p.bst + w.g * p.N));
        const buf_t cb = buffer_from(row_at<BF>(p.C, w.b * p.csb + t * p.cst + w.g * p.N));
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = lane + 64 * i, n = k % NS, tok = k / (2 * NS);
            const bool in = n < p.N && t + tok < w.t1, c = (k / NS) & 1;
            // (strides are below 2^24 elements)
            const uint32_t bo = ((uint32_t)tok * (uint32_t)p.bst + n) * E, co = ((uint32_t)tok * (uint32_t)p.cst + n) * E;
            if constexpr (NS >= 64) {            // (a value of all lanes is of one of them)
                if (((64 * i) / NS) & 1) buf_load_one<BF>(v[i], cb, in ? co : kOutside);
                else buf_load_one<BF>(v[i], bb, in ? bo : kOutside);
            } else {
                Raw<BF, 1> other;
                buf_load_one<BF>(v[i], bb, in && !c ? bo : kOutside);
                buf_load_one<BF>(other, cb, in && c ? co : kOutside);
                v[i].w[0] |= other.w[0];
            }
        }
    }
    __device__ __forceinline__ void put(float* lds, int lane) const {
#pragma unroll
        for (int i = 0; i < kEach; ++i) lds[lane + 64 * i] = v[i].get(0);
    }
};

// One number of kTok tokens of the lane's channel; behind t1 the last one again.
template <bool BF>
struct Column {
    Raw<BF, 1> v[kTok];
    // base: element of the sequence's first row and the wave's first channel,
    // off: the lane's byte offset
    __device__ __forceinline__ void load(const void* p, int64_t base, int64_t st, uint32_t off, int t, int t1) {
        const buf_t rows = buffer_from(row_at<BF>(p, base + t * st));
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            buf_load_one<BF>(v[i], rows, off, (uint32_t)(t + i < t1 ? i : t1 - 1 - t) * (uint32_t)st * (BF ? 2 : 4));
    }
};

// NS states from n0 on of row `row` of A or h0 [.][N], 0 behind the N states.
// Lanes read rows of N numbers each, a cache line or more apart, so that a load
// costs by the lines it touches: 16-byte pieces take a quarter of the time
// (number by number, and before the first tokens' loads, the passes below took
// 101 and 135 us for 97 and 129, and 18 and 20 for 15 and 15 at 24 states).
template <int NS>
__device__ __forceinline__ void load_states(float (&v)[NS], const float* s, const SsmParams& p, int64_t row, int n0 = 0) {
    if (p.wide) {
#pragma unroll
        for (int n = 0; n < NS; n += 4) {
            const f32x4 q = n0 + n < p.N ? *reinterpret_cast<const f32x4*>(s + row * p.N + n0 + n) : zero4();
#pragma unroll
            for (int e = 0; e < 4; ++e) v[n + e] = q[e];
        }
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) v[n] = n0 + n < p.N ? s[row * p.N + n0 + n] : 0.f;
    }
}
// A log2(e) (0 behind the N states, which then stay 0 while x and the step size
// are finite)
template <int NS>
__device__ __forceinline__ void load_decay(float (&a)[NS], const SsmParams& p, int c, int n0 = 0) {
    load_states<NS>(a, p.A, p, c, n0);
#pragma unroll
    for (int n = 0; n < NS; ++n) a[n] *= kLog2e;
}
template <int NS>
__device__ __forceinline__ void load_sum(float (&h)[NS], const float* s, int64_t unit, int lane) {
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = s[(unit * NS + n) * 64 + lane];
}
template <int NS>
__device__ __forceinline__ void store_sum(float* s, const float (&h)[NS], int64_t unit, int lane) {
#pragma unroll
    for (int n = 0; n < NS; ++n) s[(unit * NS + n) * 64 + lane] = h[n];
}

// Pins the registers of v where it stands.  The kernels go through their
// staged tokens in an unrolled loop; without this the compiler reads every
// token's Bm and C at once, computes every decay first, leaves sums that are
// needed only at the end for last, and so holds hundreds of registers
// (the gradient's summaries: 403 registers and 178 us for 177 and 107).  The
// states of one token already are NS independent chains.
template <int N>
__device__ __forceinline__ void pin(float (&v)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) asm volatile("" : "+v"(v[n]) : : "memory");
}

// a + Dskip b.  Without a skip a itself: not 0 times what may be infinite.
__device__ __forceinline__ float ssm_skip(const SsmParams& p, float dskip, float b, float a) {
    return p.Dskip ? fmaf(dskip, b, a) : a;
}

__device__ __forceinline__ float ssm_step_size(float raw, bool soft) { return soft ? softplus(raw) : raw; }

// The state that enters a segment.
template <int NS>
__device__ __forceinline__ void load_entering(float (&h)[NS], const SsmParams& p, const SsmPlace& w, int lane) {
    if (p.nseg > 1) {
        load_sum<NS>(h, p.sum_e, w.unit, lane);
    } else if (p.h0) {
        load_states<NS>(h, p.h0, p, (int64_t)w.b * p.D + w.c);
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = 0.f;
    }
}

template <int NS>
__device__ __forceinline__ void store_final(const float (&h)[NS], const SsmParams& p, const SsmPlace& w) {
    float* out = p.h_final + ((int64_t)w.b * p.D + w.c) * p.N;
    if (p.wide_out) {
#pragma unroll
        for (int n = 0; n < NS; n += 4)
            if (n < p.N) *reinterpret_cast<f32x4*>(out + n) = f32x4{h[n], h[n + 1], h[n + 2], h[n + 3]};
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (n < p.N) out[n] = h[n];
    }
}

// The argument of a kernel that has no other, read again, and the workgroup's
// number as if it were new: so that what is done with them, in a case that is
// rare, takes no registers from what comes before.
__device__ __forceinline__ SsmParams argument_again(unsigned& id) {
    typedef const __attribute__((address_space(4))) SsmParams* Arg;
    Arg arg = (Arg)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(id), "+s"(arg));
    return *(const SsmParams*)arg;
}

// The outputs and the final state of a segment token by token, over the N states
// alone.
template <bool BF, int NS>
__device__ __forceinline__ void ssm_fwd_tokens(unsigned id, int lane) {
    const SsmParams p = argument_again(id);
    const SsmPlace w = ssm_place(p, id, p.nseg, lane);
    float a[NS], h[NS];
    load_entering<NS>(h, p, w, lane);
    load_decay<NS>(a, p, w.c);
    const float dskip = p.Dskip ? p.Dskip[w.c] : 0.f, bias = p.dt_bias ? p.dt_bias[w.c] : 0.f;
#pragma unroll 1
    for (int t = w.t0; t < w.t1; ++t) {
        const char* bm = row_at<BF>(p.Bm, w.b * p.bsb + t * p.bst + w.g * p.N);
        const char* cm = row_at<BF>(p.C, w.b * p.csb + t * p.cst + w.g * p.N);
        const float x = load_one<BF>(p.x, w.b * p.xsb + t * p.xst + w.c);
        const float s = ssm_step_size(load_one<BF>(p.dt, w.b * p.dsb + t * p.dst + w.c) + bias, p.softplus), u = s * x;
        float y = ssm_skip(p, dskip, x, 0.f);
        int N = p.N;
        asm volatile("" : "+s"(N));                  // (the comparisons stay here)
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            if (n < N) {
                h[n] = fmaf(exp2_hw(s * a[n]), h[n], u * load_one<BF>(bm, n));
                y = fmaf(h[n], load_one<BF>(cm, n), y);
            }
        }
        if (p.z) y *= silu(load_one<BF>(p.z, w.b * p.zsb + t * p.zst + w.c));
        if (w.on) store_one<BF>(p.y, ((int64_t)w.b * p.T + t) * p.D + w.c, y);
    }
    if (w.on && p.h_final && w.seg == p.nseg - 1) store_final<NS>(h, p, w);
}

// Tokens behind t1 take the step size 0 and x 0 (the last one's may be
// infinite): they leave the state as it is.  PAD: fewer than NS states.  The
// places behind them stay 0 by themselves unless u is infinite (u times their 0
// is NaN, and is in y): the last place shows it, and the segment is done again
// without them.  (Leaving the places out in the loop, state by state, took 316
// us for 270 at 4 x 2048 x 1024 with 48 states; clearing them there 297.)
template <bool BF, int NS, bool PAD>
__global__ __launch_bounds__(64, NS <= 16 ? 3 : 1) void gdn_ssm_fwd_kernel(SsmParams p) {
    __shared__ __align__(16) float bc[2][kTok][2][NS];
    const int lane = threadIdx.x;
    const SsmPlace w = ssm_place(p, blockIdx.x, p.nseg, lane);
    const int64_t xb = w.b * p.xsb + w.c0, db = w.b * p.dsb + w.c0;
    const int64_t yb = (int64_t)w.b * p.T * p.D + w.c, y0 = (int64_t)w.b * p.T * p.D + w.c0;
    // (without a gate x is loaded in its place, and not used)
    const void* zsrc = p.z ? p.z : p.x;
    const int64_t zb = p.z ? w.b * p.zsb + w.c0 : xb, zst = p.z ? p.zst : p.xst;
    const uint32_t off = (uint32_t)(w.c - w.c0) * (BF ? 2 : 4), out = w.on ? off : kOutside;
    float a[NS], h[NS];
    load_entering<NS>(h, p, w, lane);
    const float dskip = p.Dskip ? p.Dskip[w.c] : 0.f, bias = p.dt_bias ? p.dt_bias[w.c] : 0.f;

    if (w.t0 < w.t1) {
        StagedBC<BF, NS> nbc;
        Column<BF> nx, nd, nz;
        auto load = [&](int t) {
            nbc.load(p, w, t, lane);
            nx.load(p.x, xb, p.xst, off, t, w.t1);
            nd.load(p.dt, db, p.dst, off, t, w.t1);
            nz.load(zsrc, zb, zst, off, t, w.t1);
        };
        load(w.t0);
        load_decay<NS>(a, p, w.c);
        int buf = 0;
        for (int t = w.t0; t < w.t1; t += kTok, buf ^= 1) {
            nbc.put(&bc[buf][0][0][0], lane);
            float x[kTok], s[kTok], gate[kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const float raw = nd.v[i].get(0) + bias, soft = softplus(raw), open = silu(nz.v[i].get(0));
                x[i] = t + i < w.t1 ? nx.v[i].get(0) : 0.f;
                s[i] = t + i < w.t1 ? (p.softplus ? soft : raw) : 0.f;
                gate[i] = p.z ? open : 1.f;
            }
            load(t + kTok < w.t1 ? t + kTok : w.t0);      // (the last time for nothing)
            __syncthreads();
            const buf_t yr = buffer_from(row_at<BF>(p.y, y0 + (int64_t)t * p.D));
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const float u = s[i] * x[i];
                float y = ssm_skip(p, dskip, x[i], 0.f);
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    h[n] = fmaf(exp2_hw(s[i] * a[n]), h[n], u * bc[buf][i][0][n]);
                    y = fmaf(h[n], bc[buf][i][1][n], y);
                }
                buf_store_one<BF>(yr, t + i < w.t1 ? out : kOutside, (uint32_t)i * (uint32_t)p.D * (BF ? 2 : 4), y * gate[i]);
                pin(h);
            }
        }
    }
    const bool again = PAD && __any(__builtin_isnan(h[NS - 1]));
    if (w.on) {
        for (int t = w.t0 > w.t1 ? w.t0 : w.t1; t < w.tz; ++t) store_one<BF>(p.y, yb + (int64_t)t * p.D, 0.f);
        if (!again && p.h_final && w.seg == p.nseg - 1) store_final<NS>(h, p, w);
    }
    if (again) ssm_fwd_tokens<BF, NS>(blockIdx.x, lane);
}

// Summaries of the segments.  E = sum_t P_end / P_t u_t Bm_t, with P_t the
// product of the decays up to t, as the recurrence from zero.  For the
// gradient also R = sum_t P_t C_t dyg_t: what the segment's outputs add to the
// gradient of the state that enters it (dyg = dy silu(z)), and the state from
// zero after each group of kTok tokens, from which the gradient kernel goes
// on.
template <bool BF, int NS, bool GRAD>
__global__ __launch_bounds__(64, NS <= 16 && !GRAD ? 3 : 1) void gdn_ssm_sum_kernel(SsmParams p, int nseg) {
    __shared__ __align__(16) float bc[2][kTok][2][NS];
    const int lane = threadIdx.x;
    const SsmPlace w = ssm_place(p, blockIdx.x, nseg, lane);
    const int64_t xb = w.b * p.xsb + w.c0, db = w.b * p.dsb + w.c0, y0 = (int64_t)w.b * p.T * p.D + w.c0;
    const void* zsrc = p.z ? p.z : p.x;
    const int64_t zb = p.z ? w.b * p.zsb + w.c0 : xb, zst = p.z ? p.zst : p.xst;
    // (lanes without a channel read 0, and leave states of 0)
    const uint32_t off = w.on ? (uint32_t)(w.c - w.c0) * (BF ? 2 : 4) : kOutside;
    float a[NS], h[NS], pr[NS], r[NS], total = 0.f;
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = r[n] = 0.f, pr[n] = 1.f;
    const float bias = p.dt_bias && w.on ? p.dt_bias[w.c] : 0.f;
    if (w.t0 < w.t1) {
        StagedBC<BF, NS> nbc;
        Column<BF> nx, nd, nz, ng;
        auto load = [&](int t) {
            nbc.load(p, w, t, lane);
            nx.load(p.x, xb, p.xst, off, t, w.t1);
            nd.load(p.dt, db, p.dst, off, t, w.t1);
            if (GRAD) {
                nz.load(zsrc, zb, zst, off, t, w.t1);
                ng.load(p.dy, y0, p.D, off, t, w.t1);
            }
        };
        load(w.t0);
        load_decay<NS>(a, p, w.c);
        int buf = 0;
        for (int t = w.t0; t < w.t1; t += kTok, buf ^= 1) {
            nbc.put(&bc[buf][0][0][0], lane);
            float u[kTok], s[kTok], g[kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const bool in = t + i < w.t1;
                const float raw = nd.v[i].get(0) + bias, soft = softplus(raw);
                s[i] = in ? (p.softplus ? soft : raw) : 0.f;
                u[i] = in ? s[i] * nx.v[i].get(0) : 0.f;
                g[i] = 0.f;
                if (GRAD) {
                    const float dy = ng.v[i].get(0), open = silu(nz.v[i].get(0));
                    g[i] = in ? (p.z ? dy * open : dy) : 0.f;
                }
                total += s[i];
            }
            load(t + kTok < w.t1 ? t + kTok : w.t0);      // (the last time for nothing)
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    const float d = exp2_hw(s[i] * a[n]);
                    h[n] = fmaf(d, h[n], u[i] * bc[buf][i][0][n]);
                    if (GRAD) {
                        pr[n] *= d;
                        r[n] = fmaf(pr[n], g[i] * bc[buf][i][1][n], r[n]);
                    }
                }
                pin(h);
                if (GRAD) {
                    pin(pr);
                    pin(r);
                }
            }
            if (GRAD && t + kTok < w.t1) {
                const int64_t at = w.unit * (p.seg_len / kTok - 1) + (t - w.t0) / kTok;
                store_sum<NS>(p.keep_h, h, at, lane);
                p.keep_s[at * 64 + lane] = total;
            }
        }
    }
    store_sum<NS>(p.sum_e, h, w.unit, lane);
    p.sum_s[w.unit * 64 + lane] = total;
    if (GRAD) store_sum<NS>(p.sum_r, r, w.unit, lane);
}

// From the summaries, in their place: sum_e becomes the state that enters
// each segment; sum_r the gradient of the state that leaves it, from the last
// segment to the first (by the second half of the workgroups).  One wave for a
// (sequence, tile, state); the summaries of up to 32 segments are in flight, of
// 4 where there are no more (the gradient at 8 x 20 x 4000 with 16 states, one
// segment: 10 us, with 32 all the same 29).
constexpr int kChainThreads = 64;
template <int NS, bool GRAD>
__global__ __launch_bounds__(kChainThreads) void gdn_ssm_chain_kernel(SsmParams p) {
    const unsigned tiles = (unsigned)(p.G * p.tpg), all = (unsigned)p.B * tiles * NS;
    const int lane = threadIdx.x;
    const bool back = GRAD && blockIdx.x >= all;
    const unsigned id = back ? blockIdx.x - all : blockIdx.x;
    const int n = (int)(id % NS), tile = (int)(id / NS % tiles), b = (int)(id / NS / tiles);
    const int c = (tile % p.tpg) * 64 + lane, g = tile / p.tpg;
    const bool on = c < p.Dg && n < p.N;
    const int64_t ch = g * p.Dg + c, at = ((int64_t)b * p.D + ch) * p.N + n;
    const float a = on ? p.A[ch * p.N + n] * kLog2e : 0.f;
    // segment j of the way: j, or from the end
    const int64_t unit = ((int64_t)b * p.nseg + (back ? p.nseg - 1 : 0)) * tiles + tile;
    const int64_t ss = (back ? -1 : 1) * (int64_t)tiles * 64, se = ss * NS;
    float* e = (back ? p.sum_r : p.sum_e) + (unit * NS + n) * 64;
    const float* s = p.sum_s + unit * 64;
    const float* start = back ? p.dh_final : p.h0;
    float h = start && on ? start[at] : 0.f;
    auto run = [&](auto ahead) {
        constexpr int kAhead = decltype(ahead)::value;
        for (int k = 0; k < p.nseg; k += kAhead) {
            float ev[kAhead], sv[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                // (forward alone, the last segment has no summary: none is used)
                const int j = k + i < p.nseg - (GRAD ? 0 : 1) ? k + i : 0;
                ev[i] = e[j * se + lane];
                sv[i] = s[j * ss + lane];
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (k + i < p.nseg) {
                    // (0 where there is no state: an infinite x leaves NaN in the summaries there)
                    e[(k + i) * se + lane] = on ? h : 0.f;
                    h = fmaf(exp2_hw(sv[i] * a), h, ev[i]);
                }
            }
        }
    };
    if (p.nseg <= 4) run(std::integral_constant<int, 4>());
    else run(std::integral_constant<int, 32>());
    if (back && p.dh0 && on) p.dh0[at] = h;
}

// ---------------------------------------------------------------------------
// Sums over the lanes of many registers at once: each step between lanes
// halves the registers, a lane keeping the half that its own number selects,
// while there is more than one; then plain sums.  row_sums of R registers
// leaves value (lane % 32) / (32 / R) summed over the 32 lanes of each half.
// lanes whose `hi` is set keep b's sum with their partner, the others a's
template <int CTRL>
__device__ __forceinline__ float dpp_pair_add(float a, float b, bool hi) {
    const float keep = hi ? b : a, give = hi ? a : b;
    return keep + dpp_move<CTRL>(give);
}
template <int R>
__device__ __forceinline__ float row_sums(float (&v)[R], int lane) {
    static_assert(R >= 2 && R <= 32, "");
    constexpr int R2 = R / 2, R3 = R2 > 1 ? R2 / 2 : 1, R4 = R3 > 1 ? R3 / 2 : 1, R5 = R4 > 1 ? R4 / 2 : 1;
    // partners: lane ^ 16, the row rotated by 8, the half row mirrored (bits 0
    // to 2 flipped), lane ^ 2, lane ^ 1
#pragma unroll
    for (int i = 0; i < R2; ++i) v[i] = swap16_add(v[i], v[i + R2]);
    const bool b3 = lane & 8, b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
#pragma unroll
    for (int i = 0; i < R3; ++i) v[i] = R2 > 1 ? dpp_pair_add<0x128>(v[i], v[i + R3], b3) : v[i] + dpp_move<0x128>(v[i]);
#pragma unroll
    for (int i = 0; i < R4; ++i) v[i] = R3 > 1 ? dpp_pair_add<0x141>(v[i], v[i + R4], b2) : v[i] + dpp_move<0x141>(v[i]);
#pragma unroll
    for (int i = 0; i < R5; ++i) v[i] = R4 > 1 ? dpp_pair_add<0x4E>(v[i], v[i + R5], b1) : v[i] + dpp_move<0x4E>(v[i]);
    return R5 > 1 ? dpp_pair_add<0xB1>(v[0], v[1], b0) : v[0] + dpp_move<0xB1>(v[0]);
}

// Gradient.  With g_t the gradient of h_t (g_t = C_t dyg_t + a_{t+1} g_{t+1},
// a = exp(s A)), u = s x:
//     dC_t = sum over channels of dyg_t h_t,  dB_t = sum over channels of g_t u_t
//     du_t = sum over states of g_t Bm_t,     q_t = g_t a_t h_{t-1}
//     dx_t = Dskip dyg_t + s_t du_t,          ds_t = x_t du_t + sum over states of q_t A
//     ddt_t = ds_t sigmoid(dt_t + dt_bias),   dA = sum_t q_t s_t
//     dz_t = dy_t silu'(z_t) (C_t . h_t + Dskip x_t)
// A wave takes 64 channels of one segment and goes through its groups of kTok
// tokens from the last to the first: the state at the group's start (from zero,
// as the summaries left it, and the decayed state that entered the segment),
// the group's states and decays into registers, then the gradient backwards.
// The states are split over the workgroup's NB waves, NS each; what sums over
// states (du, ds, y) is added through LDS.  Measured at 2 x 4096 x 2048 with 16
// states, bf16, gated, all launches 345 us: summaries 96, chain 16, this
// kernel 220 (four states to a wave, held decays; computed again 238; eight
// states to a wave took 299 when four took 256, all 16 in one wave 322), the
// sums over tiles and segments 11.  The vector units are busy 93 % of the time:
// about 26 issue slots for a (token, channel, state) with its share
// of the rest, two fifths of them in the sums over channels.
//
// CLEAR: the places behind the N states and lanes without a channel are 0,
// whatever the inputs, and so are Bm and C behind a segment's last token, and dA
// before it.  The usual way does without that where it would cost time in the
// loop; an infinite step size, u, dyg, state, Bm or C then leaves NaN in dA of
// those places, lanes and tokens, or in the last state.  Returns whether there is
// any.  (p by value: a reference costs 2.6 % in the order of instructions.)
template <bool BF, int NS, int NB, bool PAD, bool CLEAR>
__device__ __forceinline__ bool ssm_bwd_segment(SsmParams p, unsigned id, float (&bc_all)[NB][kTok][2][NS],
                                                float (&el)[5][kTok][64], float (&start)[NB][NS][64],
                                                float (&cross)[NB > 1 ? NB : 1][NB > 1 ? 3 * kTok : 1][64]) {
    constexpr int NSA = NS * NB;                     // states of the layout
    constexpr bool HOLD = NS <= 4;                   // the group's decays stay in registers too
    enum { kS, kX, kGy, kZs, kSg };                  // step size, x, dy silu(z), dy silu'(z), slope of softplus
    const int lane = threadIdx.x & 63, blk = NB > 1 ? threadIdx.x >> 6 : 0;
    float(&bc)[kTok][2][NS] = bc_all[blk];
    const SsmPlace w = ssm_place(p, id, p.nseg, lane);
    const int n0 = blk * NS;
    const int states = CLEAR && w.on ? p.N - n0 : CLEAR ? 0 : NS;                // of the lane
    bool wild = false;
    const int64_t xb = w.b * p.xsb + w.c, db = w.b * p.dsb + w.c;
    const int64_t yb = (int64_t)w.b * p.T * p.D + w.c;
    const float dskip = p.Dskip ? p.Dskip[w.c] : 0.f, bias = p.dt_bias ? p.dt_bias[w.c] : 0.f;
    float a[NS], g[NS], da[NS], dd = 0.f, dbias = 0.f;
    load_decay<NS>(a, p, w.c, n0);
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        g[n] = p.sum_r[(w.unit * NSA + n0 + n) * 64 + lane];
        da[n] = 0.f;
    }
    // (without a gate z's loads read dy instead, and are not used)
    const void* zsrc = p.z ? p.z : p.dy;
    const int64_t zb = p.z ? w.b * p.zsb + w.c : yb, zst = p.z ? p.zst : p.D;
    const int groups = w.t1 > w.t0 ? (w.t1 - w.t0 + kTok - 1) / kTok : 0;
    for (int k = groups - 1; k >= 0; --k) {
        const int t = w.t0 + k * kTok;
        float h[NS];                                 // the state before the group (kept in LDS for its first token)
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = p.sum_e[(w.unit * NSA + n0 + n) * 64 + lane];
        if (k > 0) {
            const int64_t at = w.unit * (p.seg_len / kTok - 1) + k - 1;
            const float sk = p.keep_s[at * 64 + lane];
#pragma unroll
            for (int n = 0; n < NS; ++n)
                h[n] = fmaf(exp2_hw(sk * a[n]), h[n], p.keep_h[(at * NSA + n0 + n) * 64 + lane]);
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (CLEAR && n >= states) h[n] = 0.f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTok * 2 * NS / 64; ++i) {
            const int e = lane + 64 * i, n = n0 + e % NS;
            int tt = t + e / (2 * NS);
            tt = tt < w.t1 ? tt : w.t1 - 1;
            float v = 0.f;
            if (n < p.N)
                v = ((e / NS) & 1) ? load_one<BF>(p.C, w.b * p.csb + tt * p.cst + w.g * p.N + n)
                                   : load_one<BF>(p.Bm, w.b * p.bsb + tt * p.bst + w.g * p.N + n);
            (&bc[0][0][0])[e] = v;
        }
        if ((NS <= 4 || CLEAR) && t + kTok > w.t1) { // (behind the last token: an infinite C times dyg 0 is NaN)
#pragma unroll
            for (int i = 0; i < kTok * 2 * NS / 64; ++i) {
                const int e = lane + 64 * i;
                if (t + e / (2 * NS) >= w.t1) (&bc[0][0][0])[e] = 0.f;
            }
        }
        // What the tokens' channels need besides the states goes through LDS,
        // for the registers' sake, and so that each wave computes its share
        // of the tokens.
        constexpr int kMine = kTok / NB;
        Raw<BF, 1> rx[kMine], rd[kMine], rg[kMine], rz[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int tt = t + j * NB + blk < w.t1 ? t + j * NB + blk : w.t1 - 1;
            rx[j].load(p.x, xb + tt * p.xst);
            rd[j].load(p.dt, db + tt * p.dst);
            rg[j].load(p.dy, yb + (int64_t)tt * p.D);
            rz[j].load(zsrc, zb + tt * zst);
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int i = j * NB + blk;
            const bool in = t + i < w.t1;
            const float raw = rd[j].get(0) + bias, dy = rg[j].get(0);
            const float soft = softplus(raw), slope_soft = sigmoid(raw);
            float val, slope;
            silu_both(rz[j].get(0), val, slope);
            // (lanes without a channel add nothing to the sums over channels: their
            // states are 0, and these)
            el[kS][i][lane] = in && w.on ? (p.softplus ? soft : raw) : 0.f;
            el[kX][i][lane] = in && w.on ? rx[j].get(0) : 0.f;
            el[kGy][i][lane] = in && w.on ? (p.z ? dy * val : dy) : 0.f;
            el[kZs][i][lane] = in ? dy * slope : 0.f;
            el[kSg][i][lane] = p.softplus ? slope_soft : 1.f;
        }
        __syncthreads();
        float hs[kTok][NS], decays[kTok][HOLD ? NS : 1];
#pragma unroll
        for (int n = 0; n < NS; ++n) start[blk][n][lane] = h[n];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const float si = el[kS][i][lane], u = si * el[kX][i][lane];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const float decay = exp2_hw(si * a[n]);
                hs[i][n] = fmaf(decay, i > 0 ? hs[i > 0 ? i - 1 : 0][n] : h[n], u * bc[i][0][n]);
                if (CLEAR && n >= states) hs[i][n] = 0.f;
                if (HOLD) decays[i][HOLD ? n : 0] = decay;
            }
            pin(hs[i]);
        }
        if (PAD && k == groups - 1) {                // (the last state: the others' NaN comes into dA)
#pragma unroll
            for (int n = 0; n < NS; ++n) wild |= (n == NS - 1 || !w.on) && __builtin_isnan(hs[kTok - 1][n]);
        }
        // the outputs of token i of the lane's channel
        auto finish = [&](int i, float y, float du, float ds) {
            if (t + i < w.t1) {
                const float x = el[kX][i][lane], gy = el[kGy][i][lane];
                // (a holds A log2(e))
                const float dr = fmaf(x, du, ds * (1.f / kLog2e)) * el[kSg][i][lane];
                dbias += dr;
                dd = fmaf(gy, x, dd);
                if (w.on) {
                    const int64_t o = yb + (int64_t)(t + i) * p.D;
                    store_one<BF>(p.dx, o, ssm_skip(p, dskip, gy, el[kS][i][lane] * du));
                    store_one<BF>(p.ddt, o, dr);
                    if (p.z) store_one<BF>(p.dz, o, el[kZs][i][lane] * ssm_skip(p, dskip, x, y));
                }
            }
        };
        // kSum tokens' sums over the channels at once: 16 registers, after the
        // first step between lanes the terms of dB in the lower half of the
        // wave and of dC in the upper
        constexpr int kSum = 16 / NS;
#pragma unroll
        for (int i0 = kTok - kSum; i0 >= 0; i0 -= kSum) {
            float v[16];
#pragma unroll
            for (int i = i0 + kSum - 1; i >= i0; --i) {
                float y = 0.f, du = 0.f, ds = 0.f;
                const float si = el[kS][i][lane], gy = el[kGy][i][lane], u = si * el[kX][i][lane];
                // The places behind the last token came before it here.  They leave
                // g as it is, but their q, of an infinite state, times 0 is NaN.
                // (With eight states to a wave this branch costs 1.5 %, and the
                // segment is done again instead: there 0.3, here 1.8.)
                if ((NS <= 4 || CLEAR) && t + i == w.t1 - 1) {
#pragma unroll
                    for (int n = 0; n < NS; ++n) da[n] = 0.f;
                    pin(da);                         // (a branch, not a choice for every token)
                }
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    const float c = bc[i][1][n];
                    g[n] = fmaf(c, gy, g[n]);
                    if (CLEAR && n >= states) g[n] = 0.f;
                    v[(i - i0) * NS + n] = swap32_add(g[n] * u, gy * hs[i][n]);
                    y = fmaf(hs[i][n], c, y);
                    du = fmaf(g[n], bc[i][0][n], du);
                    g[n] *= HOLD ? decays[i][HOLD ? n : 0] : exp2_hw(si * a[n]);
                    if (CLEAR && n >= states) g[n] = 0.f;
                    const float q = g[n] * (i > 0 ? hs[i > 0 ? i - 1 : 0][n] : start[blk][n][lane]);
                    ds = fmaf(q, a[n], ds);
                    da[n] = fmaf(q, si, da[n]);
                }
                pin(g);
                pin(da);
                if (NB > 1) {
                    cross[blk][i][lane] = y;
                    cross[blk][kTok + i][lane] = du;
                    cross[blk][2 * kTok + i][lane] = ds;
                } else {
                    finish(i, y, du, ds);
                }
            }
            const float sum = row_sums<16>(v, lane);
            const int k = lane % 32 / 2, tt = t + i0 + k / NS;
            if (lane % 2 == 0 && tt < w.t1)
                p.part_bc[((((int64_t)w.tile * p.B + w.b) * p.T + tt) * 2 + lane / 32) * NSA + n0 + k % NS] = sum;
        }
        if (NB > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                if (i % NB != blk) continue;
                float y = 0.f, du = 0.f, ds = 0.f;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    y += cross[j][i][lane];
                    du += cross[j][kTok + i][lane];
                    ds += cross[j][2 * kTok + i][lane];
                }
                finish(i, y, du, ds);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) wild |= __builtin_isnan(da[n]);
    const unsigned tiles = (unsigned)(p.G * p.tpg);
    const int64_t at = ((int64_t)w.b * p.nseg + w.seg) * tiles + w.tile;
#pragma unroll
    for (int n = 0; n < NS; ++n) p.part_a[(at * NSA + n0 + n) * 64 + lane] = da[n];
    if (NB > 1) {                                    // (each wave finished some of the tokens)
        __syncthreads();
        cross[blk][0][lane] = dd;
        cross[blk][1][lane] = dbias;
        __syncthreads();
        dd = dbias = 0.f;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            dd += cross[j][0][lane];
            dbias += cross[j][1][lane];
        }
    }
    if (NB == 1 || blk == 0) {
        p.part_d[(at * 2) * 64 + lane] = dd;
        p.part_d[(at * 2 + 1) * 64 + lane] = dbias;
        if (w.on) {
            for (int t = w.t0 > w.t1 ? w.t0 : w.t1; t < w.tz; ++t) {
                const int64_t o = yb + (int64_t)t * p.D;
                store_one<BF>(p.dx, o, 0.f);
                store_one<BF>(p.ddt, o, 0.f);
                if (p.z) store_one<BF>(p.dz, o, 0.f);
            }
        }
    }
    return wild;
}

// PAD: fewer than NS NB states, or channels that fill no whole number of waves.
// A segment with such NaN is done again (clearing the places every time: 107.8
// us for 103.3 at 2 x 1024 x 1024 with 24 states).  One wave with both forms
// needs the registers of three on a vector unit (3 states: 44.8 us, in those of
// four 47.2).
template <bool BF, int NS, int NB, bool PAD>
__global__ __launch_bounds__(64 * NB, NS <= 4 && NB != 2 && !(PAD && NB == 1) ? 4 : 3) void gdn_ssm_bwd_kernel(SsmParams p) {
    __shared__ __align__(16) float bc[NB][kTok][2][NS];
    __shared__ float el[5][kTok][64];
    __shared__ float start[NB][NS][64];
    __shared__ float cross[NB > 1 ? NB : 1][NB > 1 ? 3 * kTok : 1][64];
    const bool wild = ssm_bwd_segment<BF, NS, NB, PAD, false>(p, blockIdx.x, bc, el, start, cross);
    if ((PAD || NS > 4) && __syncthreads_or(wild)) {
        unsigned id = blockIdx.x;
        const SsmParams again = argument_again(id);
        ssm_bwd_segment<BF, NS, NB, PAD, true>(again, id, bc, el, start, cross);
    }
}

// The gradients that sum over what the waves above share, in one launch.
//   Workgroups [0, bc): dB and dC, the sum of the tiles' parts of a group,
//     tiles ascending, rounded once; zero behind a sequence's end.
//   The others, one for a (tile, state) and two for a tile's dDskip and
//     ddt_bias: dA [D, N], dDskip [D], ddt_bias [D], the sum over sequences and
//     segments, in kSumSlices slices of them (ascending) and the slices in
//     order.
struct SsmSumParams {
    SsmParams f;
    void *dB, *dC;
    float *dA, *dD, *dbias;
    int ns;                 // states of the layout
    unsigned bc;
};
constexpr int kSumSlices = 8;
constexpr int kSumThreads = 64 * kSumSlices;

template <bool BF>
__global__ __launch_bounds__(kSumThreads) void gdn_ssm_grad_sum_kernel(SsmSumParams q) {
    const SsmParams& p = q.f;
    const int ns = q.ns;
    if (blockIdx.x < q.bc) {
        const int64_t id = (int64_t)blockIdx.x * kSumThreads + threadIdx.x;
        const int64_t per = (int64_t)p.B * p.T * p.G * 2 * ns;
        if (id >= per) return;
        const int n = (int)(id % ns), which = (int)(id / ns % 2);
        const int64_t btg = id / (2 * ns);
        const int g = (int)(btg % p.G);
        const int64_t bt = btg / p.G;
        if (n >= p.N) return;
        float v = 0.f;
        if (bt % p.T < seq_len(p.lens, (int)(bt / p.T), p.T)) {
            const float* src = p.part_bc + (((int64_t)g * p.tpg * p.B * p.T + bt) * 2 + which) * ns + n;
            const int64_t step = (int64_t)p.B * p.T * 2 * ns;
#pragma unroll 8
            for (int k = 0; k < p.tpg; ++k) v += src[k * step];
        }
        store_one<BF>(which ? q.dC : q.dB, (bt * p.G + g) * p.N + n, v);
        return;
    }
    __shared__ float sum[kSumSlices][64];
    const unsigned rows = (unsigned)ns + 2, id = blockIdx.x - q.bc;
    const int tiles = p.G * p.tpg;
    const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int n = (int)(id % rows), tile = (int)(id / rows);
    const float* src = n < ns ? p.part_a + ((int64_t)tile * ns + n) * 64 + lane
                              : p.part_d + ((int64_t)tile * 2 + n - ns) * 64 + lane;
    const int64_t step = (int64_t)tiles * (n < ns ? ns : 2) * 64;
    const int64_t all = (int64_t)p.B * p.nseg, per = (all + kSumSlices - 1) / kSumSlices;
    const int64_t end = (slice + 1) * per < all ? (slice + 1) * per : all;
    float v = 0.f;
#pragma unroll 8
    for (int64_t k = slice * per; k < end; ++k) v += src[k * step];
    sum[slice][lane] = v;
    __syncthreads();
    const int c = (tile % p.tpg) * 64 + lane;
    if (slice > 0 || c >= p.Dg) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < kSumSlices; ++k) v += sum[k][lane];
    const int64_t ch = (int64_t)(tile / p.tpg) * p.Dg + c;
    if (n < p.N) q.dA[ch * p.N + n] = v;
    else if (n == ns && q.dD) q.dD[ch] = v;
    else if (n == ns + 1 && q.dbias) q.dbias[ch] = v;
}

// ---------------------------------------------------------------------------
// One token: the state passes through memory once, which bounds it (measured at
// 64 sequences of 2048 channels and 16 states: 5.5 us for 18 MB; Bm and C
// loaded number by number 7.7, four sequences to a thread 6.5, without the
// non-temporal hint 5.8).  LP lanes share a channel, four states to a lane.
struct SsmStepParams {
    SsmParams f;
    float* h;
    int wide;               // states in 16-byte pieces (N a multiple of 4, aligned)
    int wide_bc;            // Bm and C in pieces of four (likewise)
};
constexpr int kStepThreads = 256;

template <bool BF, int LP>
__global__ __launch_bounds__(kStepThreads) void gdn_ssm_step_kernel(SsmStepParams q) {
    const SsmParams& p = q.f;
    const unsigned id = blockIdx.x * kStepThreads + threadIdx.x;
    const int d0 = (int)(id / LP), n0 = (int)(id % LP) * 4;
    const int64_t b = blockIdx.y;
    const bool on = d0 < p.D;
    const int d = on ? d0 : p.D - 1, g = d / p.Dg;
    const bool piece = q.wide && n0 < p.N;
    const int64_t hi = (b * p.D + d) * p.N + n0, ai = (int64_t)d * p.N + n0;
    const int64_t bi = b * p.bsb + (int64_t)g * p.N + n0, ci = b * p.csb + (int64_t)g * p.N + n0;
    f32x4 a = zero4(), h = zero4();
    float bm[4], cm[4];
    if (piece) {
        h = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(q.h + hi));
        a = *reinterpret_cast<const f32x4*>(p.A + ai);
    }
    if (q.wide_bc && n0 < p.N) {
        Raw<BF, 4> rb, rc;
        rb.load(p.Bm, bi);
        rc.load(p.C, ci);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bm[e] = rb.get(e);
            cm[e] = rc.get(e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = n0 + e < p.N;
            bm[e] = in ? load_one<BF>(p.Bm, bi + e) : 0.f;
            cm[e] = in ? load_one<BF>(p.C, ci + e) : 0.f;
        }
    }
    if (!piece) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = n0 + e < p.N;
            h[e] = in ? q.h[hi + e] : 0.f;
            a[e] = in ? p.A[ai + e] : 0.f;
        }
    }
    const float x = load_one<BF>(p.x, b * p.xsb + d);
    const float s = ssm_step_size(load_one<BF>(p.dt, b * p.dsb + d) + (p.dt_bias ? p.dt_bias[d] : 0.f), p.softplus);
    const float gate = p.z ? silu(load_one<BF>(p.z, b * p.zsb + d)) : 1.f;
    const float u = s * x;
    float y = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = fmaf(exp2_hw(s * (a[e] * kLog2e)), h[e], u * bm[e]);
        if (n0 + e >= p.N) h[e] = 0.f;           // (an infinite u leaves NaN behind the states)
        y = fmaf(h[e], cm[e], y);
    }
#pragma unroll
    for (int m = 1; m < LP; m *= 2) y += __shfl_xor(y, m, 64);
    if (!on) return;
    if (piece) {
        __builtin_nontemporal_store(h, reinterpret_cast<f32x4*>(q.h + hi));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + e < p.N) q.h[hi + e] = h[e];
    }
    if (n0 == 0) store_one<BF>(p.y, b * p.D + d, ssm_skip(p, p.Dskip ? p.Dskip[d] : 0.f, x, y) * gate);
}

}  // namespace gdn
