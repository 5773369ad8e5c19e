// gdn_layer.h -- what the kernels around the recurrence share: element
// loads and stores of either dtype, and the activations.
#pragma once
#include "gdn_device.h"

namespace gdn {

// Vectors of V elements as they lie in memory (bf16: V in {1, 4, 8}; float:
// V in {1, 4}), kept raw until they are used so that nothing waits for a
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
// x sigmoid(x).  At x = -infinity the limit 0 (the product would be NaN).
__device__ __forceinline__ float silu(float x) {
    return x == -__builtin_inff() ? 0.f : x * sigmoid(x);
}
// silu(x) and silu'(x) = s + x s (1 - s), s = sigmoid(x), from e = e^-|x| and
// r = 1 / (1 + e): s is r or e r by x's sign, and s (1 - s) = e r^2 either way,
// with no cancellation.  At the infinities the limits (0 or x, 0 or 1).
__device__ __forceinline__ void silu_both(float x, float& val, float& slope) {
    const float e = exp2_hw(-kLog2e * __builtin_fabsf(x));
    const float r = rcp_hw(1.f + e);
    const float s = x < 0.f ? e * r : r;
    const bool inf = __builtin_isinf(x);
    val = inf && x < 0.f ? 0.f : x * s;
    slope = inf ? s : fmaf(x, e * r * r, s);
}
// ln(1 + e^x) = max(x, 0) + ln(1 + e), e = e^-|x| <= 1, and
// ln(1 + e) = 2 artanh(s), s = e / (2 + e) <= 1/3: the odd series in s to
// s^17 leaves 2 (1/3)^19 / 19 (1 - 1/9) < 1e-10 of the sum, and keeps the
// relative accuracy of small results (1 + e rounded first would not: steps of
// 1e-3 would be off by 6e-5).
__device__ __forceinline__ float softplus(float x) {
    const float e = exp2_hw(-kLog2e * __builtin_fabsf(x));
    const float s = e * rcp_hw(2.f + e);
    const float q = s * s;
    float r = 1.f / 17.f;
    r = fmaf(r, q, 1.f / 15.f);
    r = fmaf(r, q, 1.f / 13.f);
    r = fmaf(r, q, 1.f / 11.f);
    r = fmaf(r, q, 1.f / 9.f);
    r = fmaf(r, q, 1.f / 7.f);
    r = fmaf(r, q, 1.f / 5.f);
    r = fmaf(r, q, 1.f / 3.f);
    r = fmaf(r, q, 1.f);
    return __builtin_fmaxf(x, 0.f) + 2.f * s * r;
}

// The length of sequence b.
__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int T) {
    if (!lens) return T;
    const int n = lens[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

}  // namespace gdn
