// gdn_layer.h -- what the kernels around the recurrence share: element
// loads and stores of either dtype, and the activations.
#pragma once
#include "gdn_device.h"

namespace gdn {

// Vectors of V elements as they lie in memory (bf16: V in {1, 2, 4, 8}; float:
// V in {1, 2, 4}), kept raw until they are used so that nothing waits for a
// load that is only prefetched.
template <bool BF, int V>
struct Raw {
    static constexpr int kWords = BF ? (V + 1) / 2 : V;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    // element i of p (p + i aligned to V elements)
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if constexpr (BF && V == 1) {
            w[0] = reinterpret_cast<const unsigned short*>(p)[i];
        } else {
            typedef __attribute__((ext_vector_type(kWords))) uint32_t vec;
            const vec v = *reinterpret_cast<const vec*>(reinterpret_cast<const char*>(p) + i * (BF ? 2 : 4));
            if constexpr (kWords == 1) {
                w[0] = v[0];
            } else {
#pragma unroll
                for (int j = 0; j < kWords; ++j) w[j] = v[j];
            }
        }
    }
    // the elements at byte `off` of a row that the whole wave shares (its
    // address stays in scalar registers, and so does all arithmetic on it)
    __device__ __forceinline__ void load_at(const void* row, uint32_t off) {
        load(reinterpret_cast<const char*>(row) + off, 0);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (!BF) return __builtin_bit_cast(float, w[i]);
        return __builtin_bit_cast(float, (i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

template <bool BF, int V>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&f)[V]) {
    if constexpr (BF) {
        typedef __attribute__((ext_vector_type(V))) __bf16 vec;
        vec v;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = (__bf16)f[j];
        *reinterpret_cast<vec*>(reinterpret_cast<__bf16*>(p) + i) = v;
    } else {
        typedef __attribute__((ext_vector_type(V))) float vec;
        vec v;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = f[j];
        *reinterpret_cast<vec*>(reinterpret_cast<float*>(p) + i) = v;
    }
}

template <bool BF, int V>
__device__ __forceinline__ void store_at(void* row, uint32_t off, const float (&f)[V]) {
    store_vec<BF, V>(reinterpret_cast<char*>(row) + off, 0, f);
}
// Element i of a tensor as the address of a row.
template <bool BF>
__device__ __forceinline__ const char* row_at(const void* p, int64_t i) {
    return reinterpret_cast<const char*>(p) + i * (BF ? 2 : 4);
}
template <bool BF>
__device__ __forceinline__ char* row_at(void* p, int64_t i) {
    return reinterpret_cast<char*>(p) + i * (BF ? 2 : 4);
}

// One element through a buffer resource (gdn_device.h): at or behind its end,
// as kOutside is, a load gives 0 and a store writes nothing, so that neither
// needs a branch (one around a prefetch makes the compiler wait for it where
// the branch ends).
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ buf_t buffer_from(const void* base) { return buffer_over(base, 0x7fffffffu); }
// (row: a byte offset that the whole wave shares, which costs no vector
// instruction; off + row stays below 2^30)
template <bool BF>
__device__ __forceinline__ void buf_load_one(Raw<BF, 1>& r, buf_t b, uint32_t off, uint32_t row = 0) {
    if constexpr (BF) r.w[0] = (uint32_t)(unsigned short)__builtin_amdgcn_raw_buffer_load_b16(b, (int)off, (int)row, 0);
    else r.w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, (int)off, (int)row, 0);
}
template <bool BF>
__device__ __forceinline__ void buf_store_one(buf_t b, uint32_t off, uint32_t row, float v) {
    if constexpr (BF) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (__bf16)v), b, (int)off, (int)row, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), b, (int)off, (int)row, 0);
}

template <bool BF>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
    if constexpr (BF) return (float)reinterpret_cast<const __bf16*>(p)[i];
    return reinterpret_cast<const float*>(p)[i];
}
template <bool BF>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
    if constexpr (BF) reinterpret_cast<__bf16*>(p)[i] = (__bf16)v;
    else reinterpret_cast<float*>(p)[i] = v;
}

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// 1 / (1 + e^-x); e^-x overflows to infinity for x < -88.7, whose reciprocal
// is the right 0.
__device__ __forceinline__ float sigmoid(float x) { return rcp_hw(1.f + exp2_hw(-kLog2e * x)); }
// x, with -infinity as the lowest number (a NaN becomes a number: it is for
// products with what is NaN then too).
__device__ __forceinline__ float above_inf(float x) { return __builtin_amdgcn_fmed3f(x, -__FLT_MAX__, __builtin_inff()); }
// x sigmoid(x).  The bound keeps -infinity times 0 from being NaN; a NaN comes
// through sigmoid.
__device__ __forceinline__ float silu(float x) { return above_inf(x) * sigmoid(x); }
// silu(x) and silu'(x) = s + x s (1 - s), s = sigmoid(x), from e = e^-|x| and
// r = 1 / (1 + e): s is r or e r by x's sign, and s (1 - s) = e r^2 either way,
// with no cancellation.  At the infinities the limits (0 or x, 0 or 1).
__device__ __forceinline__ void silu_both(float x, float& val, float& slope) {
    const float e = exp2_hw(-kLog2e * __builtin_fabsf(x));
    const float r = rcp_hw(1.f + e), er = e * r;
    const float s = x < 0.f ? er : r;
    val = above_inf(x) * s;
    slope = fmaf(__builtin_amdgcn_fmed3f(x, -__FLT_MAX__, __FLT_MAX__), er * r, s);
}
// ln(1 + e^x) = max(x, 0) + ln(1 + e), e = e^-|x| <= 1.  With w = 1 + e as it
// was rounded and d = e - (w - 1) what that lost (exact), ln(1 + e) is ln(w) +
// d / w, and d / w is d to 2^-24 of the sum: small results keep their relative
// accuracy (ln(w) alone would leave steps of 1e-3 off by 6e-5).  v_log_f32 is
// accurate to its last bit near 1 too (measured: 1.9 x 2^-24 at most from 1 to
// 2), and the whole to the rounding of the exponent, 2^-24 |x| log2(e).
__device__ __forceinline__ float softplus(float x) {
    const float e = exp2_hw(-kLog2e * __builtin_fabsf(x));
    const float w = 1.f + e, d = e - (w - 1.f);
    // (max(x, 0) as integers: one instruction; a NaN is in d)
    const int bits = __builtin_bit_cast(int, x), top = bits > 0 ? bits : 0;
    return __builtin_bit_cast(float, top) + fmaf(__builtin_amdgcn_logf(w), 1.f / kLog2e, d);
}

// Moves and sums between lanes without LDS: DPP within a row of 16 lanes, and
// the lane-row swaps, which exchange halves of two registers in one
// instruction.  swap32_add(a, b) leaves a's sum over lane and lane ^ 32 in the
// lower 32 lanes and b's in the upper; swap16_add the same of lane ^ 16.
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float swap32_add(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t r0 = r[0], r1 = r[1];     // (a bit cast of a vector's element takes element 0)
    return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ float swap16_add(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t r0 = r[0], r1 = r[1];     // (a bit cast of a vector's element takes element 0)
    return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
}
// Sum over aligned groups of L lanes, in every lane (partners: lane ^ 1, lane ^
// 2, the half row mirrored, the row mirrored, then the other rows).
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    static_assert(L == 8 || L == 16 || L == 32 || L == 64, "");
    v += dpp_move<0xB1>(v);
    v += dpp_move<0x4E>(v);
    v += dpp_move<0x141>(v);
    if constexpr (L >= 16) v += dpp_move<0x140>(v);
    if constexpr (L >= 32) v = swap16_add(v, v);
    if constexpr (L >= 64) v = swap32_add(v, v);
    return v;
}

// The length of sequence b.
__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int T) {
    if (!lens) return T;
    const int n = lens[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

}  // namespace gdn
