// gdn_lin.h -- linear attention with a decay for each head on gfx950: chunked
// passes over prompts, their gradient, and the step of a single token.
//
//     S_t = a_t S_{t-1} + v_t k_t^T,   o_t = s S_t q_t,   a_t = exp(log_alpha_t)
//
// Over a chunk of C tokens, with G_r the sum of log a from the chunk's first
// token to r and S the state before it:
//     o_r = s ( e^{G_r} S q_r + sum_{i <= r} e^{G_r - G_i} (q_r . k_i) v_i )
//     S  <- e^{G_C} S + sum_i e^{G_C - G_i} v_i k_i^T
// With D_t the gradient of S_t (D_t = a_{t+1} D_{t+1} + s do_t q_t^T) the
// gradients are dq_t = s S_t^T do_t, dk_t = D_t^T v_t, dv_t = D_t k_t, which are
// the same pass with other operands: dq that of (do, v, k) on S transposed, and
// backwards in time dk that of (v, do, q) and dv that of (k, q, do).  So one
// kernel serves all four: rows `a` meet rows `b` (over NK numbers), which
// contribute rows `c`.
//
// The decay's gradient a_t <D_t, S_{t-1}> is a sum over pairs of tokens, one
// that reads at or after t and one that writes before t.  Pairs around t's chunk:
// e^{G_C} <D, S> of the states on its two sides, for which the pass of dk leaves
// D behind each chunk and that of dq, which runs after it, reads it (32 KB to and
// fro for a chunk and 32 columns at 128); pairs with one token outside: q_r . dq_r
// for r >= t and k_i . dk_i for i < t without their chunk's part; pairs inside:
// their products M_ri, in t's tile of 16 tokens summed as a rectangle, with one
// token in another tile by rows (dq) and columns (dk), around the tile by whole
// tiles.  Every sum holds terms of the result alone: as differences of sums over
// q . dq and k . dk an early token's gradient would hold the rounding of every
// later one's, also where a document lies between them.
//
// Products on the matrix units: bf16 rows as they lie, and what is computed (the
// state, decayed values, products of rows times their decay) in two or three bf16
// numbers that add up to it (errors of 2^-17 or 2^-24), so that a bf16 output is
// rounded once, where it is stored; fp32 rows on the fp32 units.
//
// A workgroup has 32 columns of c and all of a head's tokens (or a segment's):
// the tiles of a head read the same rows a and b, from one XCD's L2, and the more
// columns a tile had, the fewer workgroups there were for 256 compute units.
// What bounds the passes is the chain of a chunk (reads from LDS, products,
// rounding, barrier: about 3000 clocks), with the matrix units busy 28 % of
// the time: 4 x 16 x 4096 of 128/128 in bf16 take 101 us (274 MB, 56 us at a
// copy's rate; 117 in calls without a pause), 1 x 8 x 32768 156 (of them 57 for
// the segments' sums and 8 for their chain), 32 x 16 x 256 of 64/64 33 (84 MB, 17),
// the gradient of 4 x 16 x 4096 406 (472 MB, 96; 240 for dk and dv, 160 for dq,
// of which moving D behind the chunks to and fro is some 60);
// 3 x 6 x 1021 of 72/40 in fp32 39, in three launches that each wait for few rows.
#pragma once
#include <type_traits>

#include "gdn_layer.h"

namespace gdn {

struct LinTensor {
    const void* p;
    int64_t sb, sh, st;     // elements between sequences, heads, tokens
    int rep;                // heads of values to one of its heads
    int wide;               // rows of 16-byte pieces
    int direct;             // and whole ones, near enough to go straight to LDS
};

// One pass: rows a, b of nk numbers, c (and x) of nv.
struct LinRole {
    LinTensor a, b, c;
    LinTensor x;            // gradient of the decay: q beside dq, k beside dk
    int nk, nv, tiles;
    const float* first;     // state to start from, or null
    const float* carry;     // states that segments start from [B H, nseg, d_v, d_k]
    float* last;            // state at the end, or null
    void* out;              // [B, H, T, nv]
    int out_bf16, out_wide; // out_wide: rows of pieces of 1, 4 or (bf16) 8 numbers
    // gradient of the decay
    float* sums;            // [tiles, B H, T]: this pass's part of it
    float* hold;            // [B H, chunks, tiles, NK * 32]: D behind each chunk, as
                            // the waves that keep it have it (dk writes, dq reads)
};

struct LinParams {
    LinRole r[3];
    const float* log_alpha; // or null
    int64_t lsb, lsh, lst;
    const int32_t* lens;    // or null
    float* seg_sum;         // [B H, nseg, d_v, d_k]: what each segment adds
    float* seg_decay;       // [B H, nseg]: log2 of its decay
    float* seg_sum_d;       // the same of D
    int64_t units;          // B H nseg
    int B, H, T, dk, dv, nseg, seg_len;
    float scale;
};

// (kLinDqSums, kLinDkSums: with the sums for the decay's gradient)
enum LinMode { kLinFwd, kLinDq, kLinDk, kLinDv, kLinDqSums, kLinDkSums, kLinSum, kLinSumD };

// Four waves form the outputs of a chunk, four keep the state and four move rows:
// all work on the same chunk at once, one wave of each kind to a SIMD.
constexpr int kLinRole = 256, kLinThreads = 3 * kLinRole;
constexpr int kLinTile = 32;        // columns of c to a workgroup
// Tokens to a chunk: as many as let two chunks' rows and two states lie in LDS.
constexpr int lin_chunk(bool bf16, int nk) { return bf16 && nk <= 128 ? 64 : 32; }
// A decay below 2^-kLinFloor counts as 0 (fp32 has none that is smaller).
constexpr float kLinFloor = 256.f;

typedef __attribute__((ext_vector_type(8))) float f32x8;
typedef __attribute__((address_space(3))) char lds_char;
template <typename V>
__device__ __forceinline__ V lds_get(const lds_char* p) {
    return *reinterpret_cast<const __attribute__((address_space(3))) V*>(p);
}
template <typename V>
__device__ __forceinline__ void lds_put(lds_char* p, V v) {
    *reinterpret_cast<__attribute__((address_space(3))) V*>(p) = v;
}

__device__ __forceinline__ lds_char* lds_at32(uint32_t a) { return (lds_char*)(uintptr_t)a; }

// Operands of a matrix product over 32 numbers: lane 16 g + n has row (or
// column) n and numbers 8 g .. 8 g + 7.
template <bool BF>
struct LinFrag;
template <>
struct LinFrag<true> {
    bf16x8 v;
    __device__ __forceinline__ f32x8 wide() const { return __builtin_convertvector(v, f32x8); }
};
template <>
struct LinFrag<false> {
    f32x8 v;
    __device__ __forceinline__ f32x8 wide() const { return v; }
};
__device__ __forceinline__ f32x4 lin_mma(const LinFrag<true>& a, const LinFrag<true>& b, f32x4 c) { return mfma_bf16(a.v, b.v, c); }
// (the fp32 unit takes four numbers at a time: one of each lane's eight)
__device__ __forceinline__ f32x4 lin_mma(const LinFrag<false>& a, const LinFrag<false>& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = mfma_f32(a.v[i], b.v[i], c);
    return c;
}
// Two numbers in bf16, and what they are short of: the dot product with (-1, 0)
// or (0, -1) takes one half from the number that it was rounded from, exactly,
// in one instruction.  (The empty asm keeps the compiler from converting each
// number again where it is widened.)
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;
__device__ __forceinline__ uint32_t lin_pack(float a, float b) {
    uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
    asm("" : "+v"(w));
    return w;
}
__device__ __forceinline__ void lin_rest(uint32_t w, float& a, float& b) {
    // (held in registers: as a literal, -1.0 stands for the upper half here)
    uint32_t first = 0xbf80u, second = 0xbf800000u;
    asm("" : "+s"(first), "+s"(second));
    const bf16x2 h = __builtin_bit_cast(bf16x2, w);
    a = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, first), a, false);
    b = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2, second), b, false);
}
// A computed operand: N bf16 numbers that add up to it, or fp32.
template <bool BF, int N>
struct LinSplit;
template <int N>
struct LinSplit<true, N> {
    LinFrag<true> part[N];
    __device__ __forceinline__ void set(f32x8 x) {
        u32x4 w[N];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                w[k][i] = lin_pack(a, b);
                if (k + 1 < N) lin_rest(w[k][i], a, b);
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) part[k].v = __builtin_bit_cast(bf16x8, w[k]);
    }
};
template <int N>
struct LinSplit<false, N> {
    LinFrag<false> part[1];
    __device__ __forceinline__ void set(f32x8 x) { part[0].v = x; }
};
template <bool BF, int N>
__device__ __forceinline__ f32x4 lin_mma(const LinFrag<BF>& a, const LinSplit<BF, N>& b, f32x4 c) {
#pragma unroll
    for (int k = 0; k < (BF ? N : 1); ++k) c = lin_mma(a, b.part[k], c);
    return c;
}

// Whether numbers are all finite: 0 times them is 0 (bf16: on the matrix units,
// which have time for it).
template <bool BF, int M, int N>
__device__ __forceinline__ bool lin_finite(const LinFrag<BF> (&f)[M][N]) {
    float z = 0.f;
    if constexpr (BF) {
        const LinFrag<true> none{};
        f32x4 d = zero4();
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int c = 0; c < N; ++c) d = lin_mma(f[m][c], none, d);
        z = (d[0] + d[1]) + (d[2] + d[3]);
    } else {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int c = 0; c < N; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) z = fmaf(f[m][c].v[j], 0.f, z);
    }
    return __builtin_amdgcn_ballot_w64(!(z == 0.f)) == 0;
}

// Rows of ROWB bytes in LDS, without padding between them; piece p (16 bytes)
// of row r lies at p ^ turn(r), so that what is read together covers all banks.
// As measured, an operand's read (16 bytes a lane) serves 16 lanes at a time
// from 64 banks: rows 0 .. 3 and 12 .. 15 of piece p with rows 4 .. 11 of piece
// p ^ 1 (fp32: p ^ 2), and the reverse; the transposing read serves 8 rows of a
// pair of pieces; a write serves one piece of 8 rows, on 32 banks.  So among rows
// that begin at the same bank the pairs (turn / 2) of rows 0 .. 7 differ, and
// those of 8 .. 15; two rows of one pair, which the first kind of read serves
// together, have its two pieces; and four rows of the 8 (where rows fill the
// banks) have the first, four the second.
template <int ROWB>
__device__ __forceinline__ int lin_turn(int r) {
    constexpr int SH = ROWB % 256 == 0 ? 0 : ROWB % 128 == 0 ? 1 : 2;
    return (((r & 7) ^ ((r >> 1) & 4)) >> SH) << 1 | ((r >> 2) & 1);
}
template <int ROWB>
__device__ __forceinline__ int lin_piece(int r, int p) { return r * ROWB + ((p ^ lin_turn<ROWB>(r)) << 4); }

// Where a lane reads operands from a tile, computed once: rows row0 + n (row0 a
// multiple of 16, which turns nothing), numbers 32 ks + 8 g ..
template <bool BF, int ROWB, int KS>
struct LinRows {
    static constexpr int kPer = BF ? 1 : 2;
    uint32_t o[KS * kPer];
    __device__ __forceinline__ LinRows(int n, int g) {
#pragma unroll
        for (int i = 0; i < KS * kPer; ++i) o[i] = lin_piece<ROWB>(n, BF ? 4 * i + g : 8 * (i / 2) + 2 * g + i % 2);
    }
    __device__ __forceinline__ LinRows(const LinRows& from, uint32_t base) {
#pragma unroll
        for (int i = 0; i < KS * kPer; ++i) {
            o[i] = from.o[i] + base;
            asm("" : "+v"(o[i]));       // (one register each, what is added to it goes into the reads)
        }
    }
    __device__ __forceinline__ LinFrag<BF> get(int tile, int row0, int ks) const {
        LinFrag<BF> f;
        if constexpr (BF) {
            f.v = lds_get<bf16x8>(lds_at32(o[ks]) + tile + row0 * ROWB);
        } else {
            const f32x4 a = lds_get<f32x4>(lds_at32(o[2 * ks]) + tile + row0 * ROWB), b = lds_get<f32x4>(lds_at32(o[2 * ks + 1]) + tile + row0 * ROWB);
            f.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    }
};
// Columns col0 + 16 i + n of tokens 32 m + 4 g + j and 32 m + 16 + 4 g + j: the
// order in which a product's result holds the rows of two tiles.
template <bool BF, int ROWB, int TILES>
struct LinCols {
    static constexpr int kPer = BF ? 1 : 4;
    uint32_t o[TILES * kPer];
    __device__ __forceinline__ LinCols(int col0, int n, int g) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            const int c = col0 + 16 * i;
            if constexpr (BF) {
                // (the transposing read: lane n of a group addresses four columns
                // of token n / 4 and receives four tokens of column n)
                o[i] = lin_piece<ROWB>(4 * g + (n >> 2), (c >> 3) + ((n & 3) >> 1)) + (n & 1) * 8;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i * 4 + j] = lin_piece<ROWB>(4 * g + j, (c + n) >> 2) + (n & 3) * 4;
            }
        }
    }
    __device__ __forceinline__ LinCols(const LinCols& from, uint32_t base) {
#pragma unroll
        for (int i = 0; i < TILES * kPer; ++i) {
            o[i] = from.o[i] + base;
            asm("" : "+v"(o[i]));
        }
    }
    __device__ __forceinline__ LinFrag<BF> get(int tile, int m, int i) const {
        LinFrag<BF> f;
        if constexpr (BF) {
            typedef __attribute__((ext_vector_type(4))) short s4;
            typedef __attribute__((address_space(3))) s4 lds_s4;
            const lds_char* at = lds_at32(o[i]) + tile + 32 * m * ROWB;
            const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)at);
            const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(at + 16 * ROWB));
            f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f.v[j] = lds_get<float>(lds_at32(o[i * 4 + (j & 3)]) + tile + (32 * m + 16 * (j >> 2)) * ROWB);
        }
        return f;
    }
};

// `rows` rows of `cols` numbers into a tile of C rows of ROWB bytes; the rest of
// the tile is 0.
template <bool BF, int ROWB, int C>
__device__ __forceinline__ void lin_stage(lds_char* tile, const char* src, int64_t stride, int rows, int cols, int wide) {
    constexpr int kEl = BF ? 8 : 4, kPieces = ROWB / 16, kBytes = BF ? 2 : 4;
    for (int i = threadIdx.x % kLinRole; i < C * kPieces; i += kLinRole) {
        const int r = i / kPieces, q = i % kPieces, c = q * kEl;
        u32x4 v = {0, 0, 0, 0};
        if (r < rows && c < cols) {
            const char* at = src + ((int64_t)r * stride + c) * kBytes;
            if (wide && c + kEl <= cols) {
                v = *reinterpret_cast<const u32x4*>(at);
            } else {
#pragma unroll
                for (int e = 0; e < kEl; ++e) {
                    if (c + e >= cols) break;
                    if constexpr (BF) {
                        const uint32_t x = reinterpret_cast<const unsigned short*>(at)[e];
                        v[e / 2] |= x << (16 * (e & 1));
                    } else {
                        v[e] = reinterpret_cast<const uint32_t*>(at)[e];
                    }
                }
            }
        }
        lds_put(tile + lin_piece<ROWB>(r, q), v);
    }
}

// Rows straight from memory into LDS, which the movers do: lane l of a wave
// writes 16 bytes (or 4) at `to` + 16 l (or 4 l).  The compiler knows nothing of these loads: lin_wait counts them.
// (M0, which holds the place, is no register that it keeps anything in.)
__device__ __forceinline__ void lin_direct16(uint32_t to, uint32_t off, const char* base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void lin_direct4(uint32_t to, const char* from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "memory");
}
// All waves: at most N of this wave's memory operations left under way (they end
// in order), its LDS writes done.
template <int N>
__device__ __forceinline__ void lin_wait() {
    static_assert(N < 64, "");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
// This wave's loads alone.
template <int N>
__device__ __forceinline__ void lin_arrived() {
    static_assert(N < 64, "");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The same for waves that wait for no loads.
__device__ __forceinline__ void lin_wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// Where this lane's pieces of a tile of C rows lie in memory (bytes from its
// first row) and whether they are inside the row.
template <bool BF, int ROWB, int C>
struct LinDirect {
    // (kSure: those that every wave makes)
    static constexpr int kPieces = ROWB / 16, kSure = C * kPieces / kLinRole, kLoads = (C * kPieces + kLinRole - 1) / kLinRole;
    uint32_t off[kLoads];
    uint32_t in;            // bit k: the piece of load k lies inside the row
    __device__ __forceinline__ void set(int64_t stride, int cols, int wave, int lane) {
        in = 0;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int i = (k * (kLinRole / 64) + wave) * 64 + lane, r = i / kPieces;
            const int q = (i % kPieces) ^ lin_turn<ROWB>(r);
            off[k] = (uint32_t)((int64_t)r * stride * (BF ? 2 : 4)) + q * 16;
            if (i < C * kPieces && q * (BF ? 8 : 4) < cols) in |= 1u << k;
        }
    }
    // ALL: every piece of every load lies inside
    template <bool ALL>
    __device__ __forceinline__ void load(uint32_t tile, const char* rows, int wave) const {
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            if ((ALL && kSure == kLoads) || (in & (1u << k))) lin_direct16(tile + (k * (kLinRole / 64) + wave) * 1024, off[k], rows);
    }
};

// Inclusive sums over the first C lanes in 64 bits.
template <int N>
__device__ __forceinline__ double lin_row_shr(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x110 + N, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), 0x110 + N, 0xf, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int N>
__device__ __forceinline__ float lin_row_shr(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x110 + N, 0xf, 0xf, false));
}
// Inclusive sums over rows of 16 lanes.
template <typename F>
__device__ __forceinline__ F lin_row_scan(F x) {
    x += lin_row_shr<1>(x);
    x += lin_row_shr<2>(x);
    x += lin_row_shr<4>(x);
    return x + lin_row_shr<8>(x);
}
__device__ __forceinline__ float lin_lane(float x, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
}
__device__ __forceinline__ double lin_lane(double x, int l) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, l), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lin_scan(double x, int lane) {
    x = lin_row_scan(x);
    const double a = lin_lane(x, 15), b = a + lin_lane(x, 31), c = b + lin_lane(x, 47);
    const int row = lane >> 4;
    return x + (row == 0 ? 0. : row == 1 ? a : row == 2 ? b : c);
}

// LDS of a pass.  kStages chunks of rows: the one at work and those under way.
template <bool BF, int NK, int C, int MODE>
struct LinPlan {
    static constexpr bool kOut = MODE < kLinSum, kGrad = MODE == kLinDqSums || MODE == kLinDkSums;
    static constexpr int kEl = BF ? 2 : 4;
    static constexpr int kRowA = NK * kEl, kRowC = kLinTile * kEl;
    // What is computed becomes an operand of bf16 rows in parts that add up to it:
    // decayed values three (their sums are the state, which stays fp32); the
    // state and the products of rows two, whose errors of 2^-17 a bf16 output's
    // own rounding hides (with one, 17 us less at 4 x 4096 x 16 x 128, every term
    // would be off by a rounding like the output's: 2.3e-3 in the mean for
    // 1.7e-3); the state three where the decay's gradient is taken from it, which
    // is fp32 (1.6e-7 off in the mean, and 1.5e-6 with two).
    static constexpr int kParts = !BF ? 1 : kGrad ? 3 : 2;
    static constexpr int kRowParts = 2;
    static constexpr int kValueParts = 3;
    static constexpr int kStateBytes = kParts * kLinTile * kRowA;
    static constexpr int kA = 0;
    static constexpr int kB = kA + (kOut ? C * kRowA : 0);
    static constexpr int kC = kB + C * kRowA;
    static constexpr int kX = kC + C * kRowC;
    static constexpr int kStageBytes = kX + (kGrad ? C * kRowC : 0);
    static constexpr int kVec = 0;                                  // of two chunks: see LinDecays
    static constexpr int kVecBytes = (6 * C + 4) * 4;
    static constexpr int kLog = kVec + 2 * kVecBytes;               // log_alpha of four chunks
    static constexpr int kSums = kLog + 4 * 64 * 4;                 // of two: see LinSums
    static constexpr int kSumBytes = kGrad ? (4 * C + 20) * 4 : 0;
    static constexpr int kState = (kSums + 2 * kSumBytes + 255) / 256 * 256;
    // The state lies in LDS twice, or once where only so two chunks' rows fit
    // beside it (bf16 rows of 256 numbers with the decay's gradient: 1038 us at
    // 2 x 16 x 4096 for 1690 with one chunk's); it is then written behind a barrier
    // of its own, which where both fit costs more than a third chunk's rows win
    // (4 x 16 x 4096 of 128: 446 us, and 421 with two states and two chunks).
    static constexpr bool fits(int states) { return kState + states * kStateBytes + 2 * kStageBytes <= 160 * 1024; }
    static constexpr int kStates = kOut && !fits(2) && fits(1) ? 1 : 2;
    static constexpr int kStage = kState + (kOut ? kStates * kStateBytes : 0);
    static constexpr int kRoom = 160 * 1024 - kStage;
    static constexpr int kStages = kRoom >= 3 * kStageBytes ? 3 : kRoom >= 2 * kStageBytes ? 2 : 1;
    static constexpr int kBytes = kStage + kStages * kStageBytes;
    static_assert(kBytes <= 160 * 1024, "");
};

// Sum over lanes 16 g + n of the groups before g.
__device__ __forceinline__ float lin_groups_before(float v, int g) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t even = r[0], odd = r[1];
    const uint32_t both = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, even) + __builtin_bit_cast(float, odd));
    const auto q = __builtin_amdgcn_permlane32_swap(both, both, false, false);
    const uint32_t low = q[0];
    return ((g & 1) ? __builtin_bit_cast(float, even) : 0.f) + (g >= 2 ? __builtin_bit_cast(float, low) : 0.f);
}
// Sum over lanes 16 g + n of all g, in each.
__device__ __forceinline__ float lin_sum_groups(float v) {
    v = swap16_add(v, v);
    return swap32_add(v, v);
}

// The decays of a chunk in LDS, C numbers each.  Where the chunk spans little, a
// decay between two tokens is the product of kOut of one and kIn of the other
// (from the middle of the span, 2^-48 to 2^48); else the exponential of the
// difference of G, which is kept in two numbers.
enum LinDecays { kLinOut, kLinIn, kLinGh, kLinGl, kLinFirst, kLinState, kLinWhole };
constexpr float kLinSpan = 48.f;
// The sums that a chunk leaves for the decay's gradient, C numbers each: pairs of
// a row with other tiles of its chunk, with tokens outside (by tile of columns),
// and of dq pairs around a token in its tile; then [reader's tile][token's tile]
// pairs around a tile, and the state's four waves' parts of those around the chunk.
enum LinSums { kLinOther, kLinOutside, kLinTileSum = 3, kLinAcross };

template <bool BF, int NK, int C, int MODE>
__device__ __forceinline__ void lin_pass(const LinParams& p, const LinRole& R, int64_t unit, int tile, char* shared) {
    typedef LinPlan<BF, NK, C, MODE> L;
    constexpr bool kRev = MODE == kLinDk || MODE == kLinDkSums || MODE == kLinDv || MODE == kLinSumD;
    constexpr bool kTurned = MODE == kLinDq || MODE == kLinDk || L::kGrad;      // the state transposed
    constexpr int RT = C / 16;                      // row tiles
    constexpr int CT = RT == 4 ? 2 : 1;             // column tiles of a wave
    constexpr int KS = NK / 32, KT = NK / 32;       // steps over nk; state tiles of a wave
    constexpr int EB = L::kEl;
    lds_char* lds = (lds_char*)shared;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const int wave12 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = wave12 & 3;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int64_t bh = unit / p.nseg;
    const int seg = (int)(unit % p.nseg);
    const int b = (int)(bh / p.H), h = (int)(bh % p.H);
    const int t0 = seg * p.seg_len, t1 = p.T - t0 > p.seg_len ? t0 + p.seg_len : p.T;
    int tl = seq_len(p.lens, b, p.T);
    tl = tl < t0 ? t0 : (tl > t1 ? t1 : tl);
    const int chunks = (tl - t0 + C - 1) / C;
    const int col0 = tile * kLinTile, cols = R.nv - col0 < kLinTile ? R.nv - col0 : kLinTile;
    constexpr int kStages = L::kStages, kAhead = kStages - 1;
    auto number = [&](int it) __attribute__((always_inline)) { return kRev ? chunks - 1 - it : it; };
    auto stage_of = [&](int it) __attribute__((always_inline)) { return lds0 + L::kStage + (kStages == 1 ? 0 : it % kStages) * L::kStageBytes; };
    // Whole chunks go straight to LDS; where their rows do not fill the tile, its
    // rest is 0 from the start.
    const bool direct = kAhead > 0 && R.b.direct && R.c.direct && (!L::kOut || R.a.direct) && (!L::kGrad || R.x.direct) && cols % (16 / EB) == 0;
    const bool all = R.nk == NK && cols == kLinTile, fill = direct && !all;
    const int64_t plane = (int64_t)p.dk * p.dv;
    const int64_t part = tile * (int64_t)p.B * p.H + bh;            // (rows of the partial sums)

    if (wave12 >= 8) {
        // ---- the waves that move rows ----
        // (few instructions that all others wait for)
        __builtin_amdgcn_s_setprio(3);
        auto head = [&](const LinTensor& x, int c) __attribute__((always_inline)) {
            return reinterpret_cast<const char*>(x.p) + (b * x.sb + (h / x.rep) * x.sh + c) * EB;
        };
        const float* la = p.log_alpha ? p.log_alpha + b * p.lsb + h * p.lsh : nullptr;
        // Rows of chunk number `it` into its stage, and its log_alpha, a chunk
        // earlier.  A whole chunk goes straight to LDS and keeps kLoads loads of
        // each wave under way.
        constexpr int kLoads = (L::kOut ? 2 : 1) * LinDirect<BF, L::kRowA, C>::kSure + (L::kGrad ? 2 : 1) * LinDirect<BF, L::kRowC, C>::kSure;
        LinDirect<BF, L::kRowA, C> da, db;
        LinDirect<BF, L::kRowC, C> dc, dx;
        if (direct) {
            if constexpr (L::kOut) da.set(R.a.st, R.nk, wave, lane);
            db.set(R.b.st, R.nk, wave, lane);
            dc.set(R.c.st, cols, wave, lane);
            if constexpr (L::kGrad) dx.set(R.x.st, cols, wave, lane);
            if (fill) {
                for (int i = threadIdx.x % kLinRole; i < kStages * L::kStageBytes / 16; i += kLinRole)
                    lds_put(lds + L::kStage + i * 16, u32x4{0, 0, 0, 0});
            }
        }
        auto is_full = [&](int it) __attribute__((always_inline)) { return direct && it < chunks && t0 + (number(it) + 1) * C <= tl; };
        auto load_log = [&](int it) __attribute__((always_inline)) {
            if (wave == 0 && la && it < chunks) {
                const int t = t0 + number(it) * C + lane;
                if (lane < C && t < tl) lin_direct4(lds0 + L::kLog + (it & 3) * 256, reinterpret_cast<const char*>(la + t * p.lst));
            }
        };
        // (called for one chunk after the other)
        const char *ra = L::kOut ? head(R.a, 0) : nullptr, *rb = head(R.b, 0), *rc = head(R.c, col0), *rx = L::kGrad ? head(R.x, col0) : nullptr;
        const int64_t first = t0 + (int64_t)number(0) * C, turn = kRev ? -C : C;
        if constexpr (L::kOut) ra += first * R.a.st * EB;
        rb += first * R.b.st * EB;
        rc += first * R.c.st * EB;
        if constexpr (L::kGrad) rx += first * R.x.st * EB;
        const int64_t sa = turn * R.a.st * EB, sb = turn * R.b.st * EB, sc = turn * R.c.st * EB, sx = turn * R.x.st * EB;
        auto load_all = [&](uint32_t at, auto whole) __attribute__((always_inline)) {
            constexpr bool ALL = decltype(whole)::value;
            if constexpr (L::kOut) da.template load<ALL>(at + L::kA, ra, wave);
            db.template load<ALL>(at + L::kB, rb, wave);
            dc.template load<ALL>(at + L::kC, rc, wave);
            if constexpr (L::kGrad) dx.template load<ALL>(at + L::kX, rx, wave);
        };
        auto load = [&](int it) __attribute__((always_inline)) {
            if (it >= chunks) return;
            const int tc = t0 + number(it) * C, rows = tl - tc < C ? tl - tc : C;
            const uint32_t stage = stage_of(it);
            if (direct && rows == C) {
                if (all) load_all(stage, std::true_type{});
                else load_all(stage, std::false_type{});
            } else {
                lds_char* to = lds_at32(stage);
                if constexpr (L::kOut) lin_stage<BF, L::kRowA, C>(to + L::kA, ra, R.a.st, rows, R.nk, R.a.wide);
                lin_stage<BF, L::kRowA, C>(to + L::kB, rb, R.b.st, rows, R.nk, R.b.wide);
                lin_stage<BF, L::kRowC, C>(to + L::kC, rc, R.c.st, rows, cols, R.c.wide);
                if constexpr (L::kGrad) lin_stage<BF, L::kRowC, C>(to + L::kX, rx, R.x.st, rows, cols, R.x.wide);
            }
            if constexpr (L::kOut) ra += sa;
            rb += sb;
            rc += sc;
            if constexpr (L::kGrad) rx += sx;
        };
        // the decays of chunk number `it`
        auto decays = [&](int it) __attribute__((always_inline)) {
            if (wave != 0 || it >= chunks) return;
            const int rows = tl - (t0 + number(it) * C);
            float l = la && lane < rows && lane < C ? lds_get<float>(lds + L::kLog + (it & 3) * 256 + lane * 4) * kLog2e : 0.f;
            l = l < -kLinFloor ? -kLinFloor : l;    // (NaN stays)
            const double G = lin_scan(l, lane), end = lin_lane(G, C - 1), mid = 0.5 * end;
            const float gh = (float)G, away = (float)(G - mid), gend = (float)end, gmid = (float)mid;
            // (a NaN is far, too)
            const bool far = __builtin_amdgcn_ballot_w64(!(__builtin_fabsf(away) <= kLinSpan)) != 0;
            const float from = exp2_hw(gh), to = exp2_hw((float)(end - G));
            lds_char* v = lds + L::kVec + (it & 1) * L::kVecBytes;
            if (lane < C) {
                lds_put(v + (kLinOut * C + lane) * 4, far ? 1.f : exp2_hw(kRev ? -away : away));
                lds_put(v + (kLinIn * C + lane) * 4, far ? 1.f : exp2_hw(kRev ? away : -away) * (kRev ? p.scale : 1.f));
                lds_put(v + (kLinGh * C + lane) * 4, gh);
                lds_put(v + (kLinGl * C + lane) * 4, (float)(G - gh));
                lds_put(v + (kLinFirst * C + lane) * 4, far ? (kRev ? to : from) : exp2_hw(gmid));
                lds_put(v + (kLinState * C + lane) * 4, kRev ? from * p.scale : to);
            }
            if (lane == 0) {
                lds_put(v + kLinWhole * C * 4, gend);
                lds_put(v + kLinWhole * C * 4 + 4, far ? 1.f : 0.f);
            }
        };
        // what a chunk left for the decay's gradient
        auto emit = [&](int it) __attribute__((always_inline)) {
            if constexpr (L::kGrad) {
                if (wave != 1) return;
                const lds_char* sums = lds + L::kSums + (it & 1) * L::kSumBytes;
                // (of dq lane 0 has the last token: sums from it on; of dk the
                // first, and sums up to the one before)
                const int c = kRev ? lane : C - 1 - lane, t = t0 + number(it) * C + c;
                float own = 0.f, x = 0.f;
                if (lane < C) {
                    x = lds_get<float>(sums + (kLinOutside * C + c) * 4);
                    if constexpr (RT == 2) x += lds_get<float>(sums + (kLinOutside * C + C + c) * 4);
                    own = lds_get<float>(sums + (kLinOther * C + c) * 4);
                }
                // (a tile is a row of lanes)
                float r = lin_row_scan(x + own);
                x = lin_row_scan(x);
                if constexpr (kRev) r = lin_row_shr<1>(r);
                float before = 0.f;
#pragma unroll
                for (int i = 0; i + 1 < RT; ++i) {
                    const float whole = lin_lane(x, 16 * i + 15);
                    if (lane >= 16 * i + 16) before += whole;
                }
                r += before;
                if constexpr (!kRev) {
                    if (lane < C) r += lds_get<float>(sums + (kLinTileSum * C + c) * 4);
#pragma unroll
                    for (int i = 2; i < RT; ++i)
#pragma unroll
                        for (int m = 1; m < i; ++m)
                            if (c / 16 == m) r += lds_get<float>(sums + (kLinAcross * C + 4 * i + m) * 4);
                    const f32x4 f = lds_get<f32x4>(sums + (kLinAcross * C + 16) * 4);
                    r += (f[0] + f[1]) + (f[2] + f[3]);
                }
                if (lane < C && t < tl) R.sums[part * p.T + t] = r;
            }
        };
        if (fill) lin_wait<0>();
        load_log(0);
        load_log(1);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            load(i);
            if (i + 1 < kAhead || kAhead == 1) load_log(i + 2);
        }
        // (log_alpha of the first chunk, which came first)
        if (kAhead > 0 && is_full(0) && is_full(kAhead - 1)) lin_arrived<kAhead * kLoads>();
        else lin_arrived<0>();
        decays(0);
        for (int it = 0; it < chunks; ++it) {
            // what chunk `it` needs has come; what was asked for since may be
            // under way
            if constexpr (kAhead == 0) {
                lin_wait<0>();
                load(it);
                load_log(it + 1);
                lin_wait<0>();
            } else {
                if (kAhead > 1 && is_full(it + kAhead - 1)) lin_wait<(kAhead - 1) * kLoads>();
                else lin_wait<0>();
                // (rows that are one chunk ahead come first, two ahead can wait)
                load_log(it + kAhead + 1);
                if constexpr (kAhead > 1) decays(it + 1);
                load(it + kAhead);
            }
            if constexpr (kAhead <= 1) decays(it + 1);
            if constexpr (L::kStates == 1) lin_wait_lds();
            if (it > 0) emit(it - 1);
        }
        if constexpr (L::kGrad) {
            __syncthreads();
            if (chunks > 0) emit(chunks - 1);
        }
        if constexpr (L::kOut) {
            // rows behind the last chunk
            const int64_t z0 = t0 + (int64_t)chunks * C;
            for (int64_t i = z0 * cols + (int)(threadIdx.x % kLinRole); i < (int64_t)t1 * cols; i += kLinRole) {
                const int64_t at = (bh * p.T + i / cols) * R.nv + col0 + i % cols;
                if (R.out_bf16) reinterpret_cast<__bf16*>(R.out)[at] = (__bf16)0.f;
                else reinterpret_cast<float*>(R.out)[at] = 0.f;
            }
        }
        return;
    }

    if (wave12 >= 4) {
        // ---- the waves that keep the state ----
        // Rows nk and columns nv: this wave's tiles are KT rows of tiles from kt0
        // and one column of tiles.
        const int nvt = wave & 1, kt0 = (wave >> 1) * KT;
        const int64_t sn = kTurned ? 1 : p.dk, sk = kTurned ? p.dk : 1;
        const int scol = col0 + nvt * 16 + n;
        const LinCols<BF, L::kRowA, KT> at_b(kt0 * 16, n, g);
        const LinCols<BF, L::kRowC, 1> at_c(nvt * 16, n, g);
        f32x4 S[KT];
        {
            const float* from = nullptr;
            if constexpr (L::kOut) from = R.carry ? R.carry + unit * plane : R.first ? R.first + bh * plane : nullptr;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = (kt0 + t) * 16 + 4 * g + j;
                    S[t][j] = from && k < R.nk && scol < R.nv ? from[k * sk + scol * sn] : 0.f;
                }
        }
        auto publish = [&](int buf) __attribute__((always_inline)) {
            lds_char* at = lds + L::kState + buf % L::kStates * L::kStateBytes;
            const int row = nvt * 16 + n;
            if constexpr (BF) {
                f32x4 x[KT];
#pragma unroll
                for (int t = 0; t < KT; ++t) x[t] = S[t];
#pragma unroll
                for (int k = 0; k < L::kParts; ++k) {
                    u32x2 w[KT];
#pragma unroll
                    for (int t = 0; t < KT; ++t) {
                        w[t] = u32x2{lin_pack(x[t][0], x[t][1]), lin_pack(x[t][2], x[t][3])};
                        if (k + 1 < L::kParts) {
                            float y[4] = {x[t][0], x[t][1], x[t][2], x[t][3]};
                            lin_rest(w[t][0], y[0], y[1]);
                            lin_rest(w[t][1], y[2], y[3]);
                            x[t] = f32x4{y[0], y[1], y[2], y[3]};
                        }
                    }
                    lds_char* to = at + k * kLinTile * L::kRowA;
                    // Two tiles at once, 16 bytes a lane: lanes of even g take
                    // their neighbour's numbers of the first, those of odd g
                    // theirs of the second.
#pragma unroll
                    for (int t = 0; t + 1 < KT; t += 2) {
                        const auto lo = __builtin_amdgcn_permlane16_swap(w[t][0], w[t + 1][0], false, false);
                        const auto hi = __builtin_amdgcn_permlane16_swap(w[t][1], w[t + 1][1], false, false);
                        lds_put(to + lin_piece<L::kRowA>(row, 2 * (kt0 + t + (g & 1)) + (g >> 1)), u32x4{lo[0], hi[0], lo[1], hi[1]});
                    }
                    if constexpr (KT % 2 == 1)
                        lds_put(to + lin_piece<L::kRowA>(row, 2 * (kt0 + KT - 1) + (g >> 1)) + (g & 1) * 8, w[KT - 1]);
                }
            } else {
#pragma unroll
                for (int t = 0; t < KT; ++t) lds_put(at + lin_piece<L::kRowA>(row, 4 * (kt0 + t) + g), S[t]);
            }
        };
        if constexpr (L::kOut) publish(0);
        // What the states on a chunk's two sides share: the pass of dk leaves D
        // behind chunk number `it`, that of dq reads it (a chunk ahead where
        // registers hold it) and multiplies by S before it.
        constexpr bool kEarly = KT <= 4;
        float* const hold = L::kGrad ? R.hold + ((bh * ((p.T + C - 1) / C) + t0 / C) * R.tiles + tile) * (NK * kLinTile) + (wave * 64 + lane) * 4 : nullptr;
        f32x4 behind[KT];
        float around = 0.f;
        auto load_behind = [&](int it) __attribute__((always_inline)) {
            if (it >= chunks) return;
            const float* at = hold + (int64_t)number(it) * R.tiles * (NK * kLinTile);
#pragma unroll
            for (int t = 0; t < KT; ++t) behind[t] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(at + t * 1024));
        };
        auto sides = [&](int it) __attribute__((always_inline)) {
            if (it >= chunks) return;
            if constexpr (MODE == kLinDkSums) {
                float* at = hold + (int64_t)number(it) * R.tiles * (NK * kLinTile);
#pragma unroll
                for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(at + t * 1024) = S[t];
            }
            if constexpr (MODE == kLinDqSums) {
                if constexpr (!kEarly) load_behind(it);
                around = 0.f;
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) around = fmaf(S[t][j], behind[t][j], around);
                if constexpr (kEarly) load_behind(it + 1);
            }
        };
        if constexpr (MODE == kLinDqSums && kEarly) load_behind(0);
        sides(0);
        if (fill) lin_wait_lds();
        float total = 0.f;      // log2 of the decay so far
        for (int it = 0; it < chunks; ++it) {
            lin_wait_lds();
            if constexpr (kAhead == 0) lin_wait_lds();
            const lds_char* vec = lds + L::kVec + (it & 1) * L::kVecBytes;
            const uint32_t stage = stage_of(it);
            const LinCols<BF, L::kRowA, KT> rb(at_b, stage);
            const LinCols<BF, L::kRowC, 1> rc(at_c, stage);
            LinFrag<BF> vals[C / 32], keys[C / 32][KT];
            f32x8 u[C / 32];
            const float gend = lds_get<float>(vec + kLinWhole * C * 4);
#pragma unroll
            for (int m = 0; m < C / 32; ++m) {
                vals[m] = rc.get(L::kC, m, 0);
                u[m] = __builtin_shufflevector(lds_get<f32x4>(vec + (kLinState * C + 32 * m + 4 * g) * 4),
                                               lds_get<f32x4>(vec + (kLinState * C + 32 * m + 16 + 4 * g) * 4), 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int m = 0; m < C / 32; ++m)
#pragma unroll
                for (int t = 0; t < KT; ++t) keys[m][t] = rb.get(L::kB, m, t);
            // (all reads on their way before anything waits for one)
            __builtin_amdgcn_sched_barrier(0);
            total += gend;
            const float whole = exp2_hw(gend);
#pragma unroll
            for (int t = 0; t < KT; ++t) S[t] *= whole;
#pragma unroll
            for (int m = 0; m < C / 32; ++m) {
                LinSplit<BF, L::kValueParts> fc;
                fc.set(vals[m].wide() * u[m]);
#pragma unroll
                for (int k = 0; k < (BF ? L::kValueParts : 1); ++k)
#pragma unroll
                    for (int t = 0; t < KT; ++t) S[t] = lin_mma(keys[m][t], fc.part[k], S[t]);
            }
            if constexpr (L::kStates == 1) lin_wait_lds();
            if constexpr (L::kOut) publish(it + 1);
            if constexpr (MODE == kLinDqSums) {
                const float f = lanes_sum<64>(around) * whole;
                if (lane == 0) lds_put(lds + L::kSums + (it & 1) * L::kSumBytes + (kLinAcross * C + 16 + wave) * 4, f);
            }
            sides(it + 1);
        }
        // the state at the end
        float* to = nullptr;
        if constexpr (MODE == kLinSum) to = p.seg_sum + unit * plane;
        if constexpr (MODE == kLinSumD) to = p.seg_sum_d + unit * plane;
        if constexpr (L::kOut) {
            if (R.last && seg == (kRev ? 0 : p.nseg - 1)) to = R.last + bh * plane;
        }
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = (kt0 + t) * 16 + 4 * g + j;
                if (to && k < R.nk && scol < R.nv) to[k * sk + scol * sn] = S[t][j];
            }
        if (MODE == kLinSum && tile == 0 && wave == 0 && lane == 0) p.seg_decay[unit] = total;
        if constexpr (L::kGrad) __syncthreads();
        return;
    }

    // ---- the waves that form the outputs ----
    if constexpr (!L::kOut) {
        // (as many barriers as the others pass)
        for (int it = 0; it < (fill ? 1 : 0) + chunks * (kAhead == 0 ? 2 : 1); ++it) lin_wait_lds();
        return;
    }
    const float oscale = kRev ? 1.f : p.scale;
    const int rt = RT == 4 ? wave : wave >> 1, ct0 = RT == 4 ? 0 : wave & 1;
    const int row = rt * 16 + n;
    // (steps whose reads go out together)
    constexpr int KB = KS < 4 ? KS : BF || NK <= 128 ? 4 : 2;
    // (of a state in parts one step, which is as many: prompts 107 us for 111)
    constexpr int KBS = L::kParts > 1 ? 1 : KB;
    const LinRows<BF, L::kRowA, KS> at_a(n, g);
    const LinRows<BF, L::kRowC, 1> at_x(n, g);
    const LinCols<BF, L::kRowC, CT> at_c(ct0 * 16, n, g);
    // A chunk's rows are stored during the next chunk, while that waits for its
    // reads.
    struct Rows {
        f32x4 c[CT];
    } done;
    float done_scale = 0.f;
    int done_at = 0;
    char* const out_base = reinterpret_cast<char*>(R.out) + (bh * p.T * R.nv + col0) * (R.out_bf16 ? 2 : 4);
    auto store = [&]() __attribute__((always_inline)) {
        if (done_at >= t1) return;
        // (rows behind the sequence's end inside its last chunk are 0)
        const bool live = done_at < tl;
        const int64_t first = (int64_t)done_at * R.nv;
        if (BF && CT == 2 && R.out_wide == 8 && cols == kLinTile) {
            // 16 bytes a lane: lanes of even g take their neighbour's columns of
            // the first tile, those of odd g theirs of the second
            const f32x4 a = live ? done.c[0] * done_scale : zero4(), b = live ? done.c[CT - 1] * done_scale : zero4();
            const auto lo = __builtin_amdgcn_permlane16_swap(lin_pack(a[0], a[1]), lin_pack(b[0], b[1]), false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap(lin_pack(a[2], a[3]), lin_pack(b[2], b[3]), false, false);
            *reinterpret_cast<u32x4*>(out_base + (first + (g & 1) * 16 + (g >> 1) * 8) * 2) = u32x4{lo[0], hi[0], lo[1], hi[1]};
            return;
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int col = (ct0 + c) * 16 + 4 * g;
            const f32x4 o = live ? done.c[c] * done_scale : zero4();
            const int64_t at = first + col;
            if (R.out_wide >= 4) {
                if (col < cols) {
                    if (R.out_bf16) *reinterpret_cast<bf16x4*>(out_base + at * 2) = __builtin_convertvector(o, bf16x4);
                    else *reinterpret_cast<f32x4*>(out_base + at * 4) = o;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < cols) {
                        if (R.out_bf16) *reinterpret_cast<__bf16*>(out_base + (at + j) * 2) = (__bf16)o[j];
                        else *reinterpret_cast<float*>(out_base + (at + j) * 4) = o[j];
                    }
            }
        }
    };
    if (fill) lin_wait_lds();
    for (int it = 0; it < chunks; ++it) {
        const int tc = t0 + number(it) * C;
        lin_wait_lds();
        if constexpr (kAhead == 0) lin_wait_lds();
        const lds_char* vec = lds + L::kVec + (it & 1) * L::kVecBytes;
        lds_char* sums = lds + L::kSums + (it & 1) * L::kSumBytes;
        const uint32_t stage = stage_of(it);
        const LinRows<BF, L::kRowA, KS> ra(at_a, stage), rs(at_a, lds0 + L::kState + it % L::kStates * L::kStateBytes);
        const LinCols<BF, L::kRowC, CT> rc(at_c, stage);
        // Reads go out together, as many as registers hold (KB steps), before
        // the products that wait for them.
        LinFrag<BF> fa[KS];
        Rows now;
        f32x4(&acc)[CT] = now.c;
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = zero4();
#pragma unroll
        for (int k0 = 0; k0 < KS; k0 += KBS) {
            LinFrag<BF> fs[L::kParts][CT][KBS];
#pragma unroll
            for (int ks = 0; ks < KBS; ++ks) {
                if (k0 + ks >= KS) break;
                fa[k0 + ks] = ra.get(L::kA, rt * 16, k0 + ks);
#pragma unroll
                for (int k = 0; k < L::kParts; ++k)
#pragma unroll
                    for (int c = 0; c < CT; ++c) fs[k][c][ks] = rs.get(k * kLinTile * L::kRowA, (ct0 + c) * 16, k0 + ks);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (k0 == 0 && it > 0) store();
#pragma unroll
            for (int ks = 0; ks < KBS; ++ks) {
                if (k0 + ks >= KS) break;
#pragma unroll
                for (int k = 0; k < L::kParts; ++k)
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[c] = lin_mma(fs[k][c][ks], fa[k0 + ks], acc[c]);
            }
        }
        if constexpr (L::kStates == 1) lin_wait_lds();
        // products of the rows with the pairs of tiles that hold any row on their
        // side of the diagonal, and what their decays need
        f32x4 pr[C / 16];
#pragma unroll
        for (int i = 0; i < C / 16; ++i) pr[i] = zero4();
#pragma unroll
        for (int i0 = 0; i0 < C / 16; i0 += 2) {
            if (kRev ? i0 + 1 < rt : i0 > rt) continue;
#pragma unroll
            for (int k0 = 0; k0 < KS; k0 += KB) {
                LinFrag<BF> fb[2][KB];
#pragma unroll
                for (int ks = 0; ks < KB; ++ks) {
                    if (k0 + ks >= KS) break;
#pragma unroll
                    for (int i = 0; i < 2; ++i) fb[i][ks] = ra.get(L::kB, (i0 + i) * 16, k0 + ks);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int ks = 0; ks < KB; ++ks) {
                    if (k0 + ks >= KS) break;
#pragma unroll
                    for (int i = 0; i < 2; ++i) pr[i0 + i] = lin_mma(fb[i][ks], fa[k0 + ks], pr[i0 + i]);
                }
            }
        }
        LinFrag<BF> fc[C / 32][CT];
#pragma unroll
        for (int m = 0; m < C / 32; ++m)
#pragma unroll
            for (int c = 0; c < CT; ++c) fc[m][c] = rc.get(L::kC, m, c);
        const bool finite = lin_finite(fc);
        const float out = lds_get<float>(vec + (kLinOut * C + row) * 4), before = lds_get<float>(vec + (kLinFirst * C + row) * 4);
        const bool far = __builtin_amdgcn_readfirstlane(lds_get<int>(vec + kLinWhole * C * 4 + 4)) != 0;
        f32x4 in[C / 16];
#pragma unroll
        for (int i = 0; i < C / 16; ++i) in[i] = lds_get<f32x4>(vec + (kLinIn * C + 16 * i + 4 * g) * 4);
        if (far) {
            const float gh = lds_get<float>(vec + (kLinGh * C + row) * 4), gl = lds_get<float>(vec + (kLinGl * C + row) * 4);
#pragma unroll
            for (int i = 0; i < C / 16; ++i) {
                const f32x4 ih = lds_get<f32x4>(vec + (kLinGh * C + 16 * i + 4 * g) * 4), il = lds_get<f32x4>(vec + (kLinGl * C + 16 * i + 4 * g) * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float d = (gh - ih[j]) + (gl - il[j]);
                    in[i][j] = exp2_hw(kRev ? -d : d) * (kRev ? p.scale : 1.f);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] *= before;
        const float scale = out * oscale;
#pragma unroll
        for (int i = 0; i < C / 16; ++i) {
            const int col = 16 * i + 4 * g;
#pragma unroll
            for (int j = 0; j < 4; ++j) pr[i][j] = (kRev ? col + j >= row : col + j <= row) ? pr[i][j] * in[i][j] : 0.f;
        }
        if constexpr (L::kGrad) {
            const LinRows<BF, L::kRowC, 1> rx(at_x, stage);
            const LinFrag<BF> mine = rx.get(L::kX, rt * 16, 0);
            f32x4 x[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int col = (ct0 + c) * 16 + 4 * g;
                const lds_char* at = lds_at32(stage) + L::kX + lin_piece<L::kRowC>(row, col * EB / 16) + col * EB % 16;
                if constexpr (BF) x[c] = __builtin_convertvector(lds_get<bf16x4>(at), f32x4);
                else x[c] = lds_get<f32x4>(at);
            }
            // (pairs in the row's own tile in the pass of dq, with other tiles in
            // both; what is no pair is left out, not multiplied by 0)
            float outside = 0.f, others = 0.f, across[RT] = {};
            f32x4 tile_sum = zero4();
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                if constexpr (MODE == kLinDqSums) {
                    // (tiles before this one, of the row's tile)
                    if (i > 0) across[i] = others;
                }
                if (kRev ? i <= rt : i > rt) continue;
                const f32x4 m = lin_mma(rx.get(L::kC, 16 * i, 0), mine, zero4()) * pr[i];
                if (kRev || i < rt) {
                    others += (m[0] + m[1]) + (m[2] + m[3]);
                } else {
                    float e[4], sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e[j] = sum;
                        sum += 4 * g + j < n ? m[j] : 0.f;
                    }
                    const float before_g = lin_groups_before(sum, g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) tile_sum[j] = lanes_sum<16>(4 * g + j <= n ? (before_g + e[j]) * scale : 0.f);
                }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) outside = fmaf(acc[c][j], x[c][j], outside);
            outside = lin_sum_groups(outside) * scale;
            if (g == 0) lds_put(sums + ((kLinOutside + ct0) * C + row) * 4, outside);
            if (ct0 == 0) {
                others *= scale;
                const float row_others = lin_sum_groups(others);
                if (g == 0) lds_put(sums + (kLinOther * C + row) * 4, row_others);
                if constexpr (MODE == kLinDqSums) {
                    if (n == 0) lds_put(sums + (kLinTileSum * C + rt * 16 + 4 * g) * 4, tile_sum);
#pragma unroll
                    for (int i = 1; i < RT; ++i) {
                        if (i >= rt) break;
                        const float a = lanes_sum<64>(across[i] * scale);
                        if (lane == 0) lds_put(sums + (kLinAcross * C + 4 * rt + i) * 4, a);
                    }
                }
            }
        }
        // What a row may not see it has times 0, which is not 0 of an infinite or
        // NaN number: a chunk that holds one is added up token by token, each to
        // the rows that see it.
        if (finite) {
#pragma unroll
            for (int m = 0; m < C / 32; ++m) {
                LinSplit<BF, L::kRowParts> pp;
                pp.set(__builtin_shufflevector(pr[2 * m], pr[2 * m + 1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[c] = lin_mma(fc[m][c], pp, acc[c]);
            }
        } else {
#pragma unroll
            for (int m = 0; m < C / 32; ++m)
#pragma unroll 1
                for (int i = 0; i < 32; ++i) {
                    LinFrag<BF> one[CT] = {};
                    f32x8 x = {};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (i != 16 * (j >> 2) + 4 * g + (j & 3)) continue;
                        x[j] = pr[2 * m + (j >> 2)][j & 3];
#pragma unroll
                        for (int c = 0; c < CT; ++c) one[c].v[j] = fc[m][c].v[j];
                    }
                    LinSplit<BF, L::kRowParts> pp;
                    pp.set(x);
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const f32x4 o = lin_mma(one[c], pp, zero4());
                        if (kRev ? 32 * m + i >= row : 32 * m + i <= row) acc[c] += o;
                    }
                }
        }
        done = now;
        done_scale = scale;
        done_at = tc + row;
    }
    if (chunks > 0) store();
    if constexpr (L::kGrad) __syncthreads();
}

// Workgroups: the tiles of a unit (a head of a sequence, or a segment of one)
// beside each other on one XCD, whose L2 then holds the rows that they share;
// neighbouring units too, whose heads may share queries and keys.
// (with the decay's gradient dk comes first, and dv with it or after)
enum LinSet { kLinSetFwd, kLinSetQk, kLinSetV, kLinSetAll, kLinSetKSums, kLinSetKvSums, kLinSetQSums, kLinSetSum, kLinSetSums };
constexpr int kXcds = 8;

constexpr int lin_most(int a, int b) { return a > b ? a : b; }
// LDS of a launch: the most that one of its passes takes.
template <bool BF, int NK, int SET>
struct LinBytes {
    static constexpr int C = lin_chunk(BF, NK);
    static constexpr int kRows = LinPlan<BF, NK, C, kLinFwd>::kBytes;
    static constexpr int kDq = LinPlan<BF, NK, C, kLinDqSums>::kBytes, kDk = LinPlan<BF, NK, C, kLinDkSums>::kBytes;
    static constexpr int value = SET == kLinSetSum || SET == kLinSetSums ? LinPlan<BF, NK, C, kLinSum>::kBytes
                                 : SET == kLinSetKSums                   ? kDk
                                 : SET == kLinSetKvSums                  ? lin_most(kDk, kRows)
                                 : SET == kLinSetQSums                   ? kDq
                                                                         : kRows;
    static_assert(LinPlan<BF, NK, C, kLinDq>::kBytes == kRows && LinPlan<BF, NK, C, kLinDk>::kBytes == kRows, "");
    static_assert(LinPlan<BF, NK, C, kLinDv>::kBytes == kRows && LinPlan<BF, NK, C, kLinSum>::kBytes == LinPlan<BF, NK, C, kLinSumD>::kBytes, "");
};

template <bool BF, int NK, int SET>
__global__ __launch_bounds__(kLinThreads) void gdn_lin_kernel(LinParams p) {
    __shared__ __align__(256) char lin_lds[LinBytes<BF, NK, SET>::value];
    constexpr int C = lin_chunk(BF, NK);
    constexpr int kRoles = SET == kLinSetAll ? 3 : SET == kLinSetQk || SET == kLinSetKvSums || SET == kLinSetSums ? 2 : 1;
    int tiles = 0;
#pragma unroll
    for (int i = 0; i < kRoles; ++i) tiles += p.r[i].tiles;
    const int64_t per = (p.units + kXcds - 1) / kXcds;
    const int64_t at = blockIdx.x / kXcds;
    const int64_t unit = (blockIdx.x % kXcds) * per + at / tiles;
    int tile = (int)(at % tiles);
    if (at / tiles >= per || unit >= p.units) return;
    // (the modes of a set's roles)
    constexpr LinMode k0 = SET == kLinSetFwd                               ? kLinFwd
                           : SET == kLinSetV                               ? kLinDv
                           : SET == kLinSetKSums || SET == kLinSetKvSums   ? kLinDkSums
                           : SET == kLinSetQSums                           ? kLinDqSums
                           : SET == kLinSetSum || SET == kLinSetSums       ? kLinSum
                                                                           : kLinDq;
    constexpr LinMode k1 = SET == kLinSetSums ? kLinSumD : SET == kLinSetKvSums ? kLinDv : kLinDk;
    if (kRoles == 1 || tile < p.r[0].tiles) {
        lin_pass<BF, NK, C, k0>(p, p.r[0], unit, tile, lin_lds);
        return;
    }
    if constexpr (kRoles > 1) {
        tile -= p.r[0].tiles;
        if (kRoles == 2 || tile < p.r[1].tiles) {
            lin_pass<BF, NK, C, k1>(p, p.r[1], unit, tile, lin_lds);
            return;
        }
        if constexpr (kRoles > 2) lin_pass<BF, NK, C, kLinDv>(p, p.r[2], unit, tile - p.r[1].tiles, lin_lds);
    }
}

// One token of every sequence, one pass over the state, which bounds it: 64 x 16
// states of 128 x 128 take 20 us, 135 MB, part of which the last level of cache
// holds from the call before.  A group of L lanes holds a row of the state (d_k
// numbers, V to a piece), kLinStepRows rows in turn: k and q are loaded once for
// them.
struct LinStepParams {
    LinTensor q, k, v;
    const float* log_alpha;
    int64_t lsb, lsh;
    float* S;
    void* out;
    int H, dk, dv, blocks, out_bf16;
    float scale;
};
constexpr int kLinStepThreads = 128;
constexpr int kLinStepRows = 4;
template <bool BF, int L, int J, int V>
__global__ __launch_bounds__(kLinStepThreads) void gdn_lin_step_kernel(LinStepParams p) {
    constexpr int kGroups = kLinStepThreads / L;
    const int m = threadIdx.x % L, grp = threadIdx.x / L;
    const int64_t bh = blockIdx.x / p.blocks;
    const int row0 = (int)(blockIdx.x % p.blocks) * kGroups * kLinStepRows + grp;
    const int b = (int)(bh / p.H), h = (int)(bh % p.H);
    const int64_t q0 = b * p.q.sb + (h / p.q.rep) * p.q.sh, k0 = b * p.k.sb + (h / p.k.rep) * p.k.sh;
    const int64_t v0 = b * p.v.sb + h * p.v.sh;
    Raw<false, V> S[kLinStepRows][J];
    Raw<BF, V> kr[J], qr[J];
#pragma unroll
    for (int r = 0; r < kLinStepRows; ++r) {
        const int row = row0 + r * kGroups;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (j * L + m) * V;
            S[r][j].zero();
            if (row < p.dv && c < p.dk) S[r][j].load(p.S, (bh * p.dv + row) * p.dk + c);
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (j * L + m) * V;
        kr[j].zero();
        qr[j].zero();
        if (c < p.dk) {
            kr[j].load(p.k.p, k0 + c);
            qr[j].load(p.q.p, q0 + c);
        }
    }
    const float a = p.log_alpha ? exp2_hw(p.log_alpha[b * p.lsb + h * p.lsh] * kLog2e) : 1.f;
#pragma unroll
    for (int r = 0; r < kLinStepRows; ++r) {
        const int row = row0 + r * kGroups;
        const float v = row < p.dv ? load_one<BF>(p.v.p, v0 + row) : 0.f;
        float o = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (j * L + m) * V;
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f[e] = fmaf(v, kr[j].get(e), a * S[r][j].get(e));
                o = fmaf(f[e], qr[j].get(e), o);
            }
            if (row < p.dv && c < p.dk) store_vec<false, V>(p.S, (bh * p.dv + row) * p.dk + c, f);
        }
        o = lanes_sum<L>(o) * p.scale;
        if (row < p.dv && m == 0) {
            if (p.out_bf16) reinterpret_cast<__bf16*>(p.out)[bh * p.dv + row] = (__bf16)o;
            else reinterpret_cast<float*>(p.out)[bh * p.dv + row] = o;
        }
    }
}

}  // namespace gdn
