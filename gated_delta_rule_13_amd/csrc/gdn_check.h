// gdn_check.h -- checks of arguments that the files with C entry points of the
// layer operators share.
#pragma once
#include <cstdint>
#include <initializer_list>
#include <string>

#include "gdn.h"
#include "gdn_error.h"

namespace gdn {

constexpr size_t kInvalid = (size_t)-1;
constexpr int64_t kMaxGrid = 0x7fffffff;
// A launch counts its threads in 32 bits.
inline bool threads_ok(long double n) { return n <= 4294967295.0L; }

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool dtype_ok(int t) { return t == GDN_BF16 || t == GDN_F32; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Every pointer that is given is aligned to its type.
struct Operand {
    const void* p;
    int dtype;
};
inline gdn_status check_aligned(std::initializer_list<Operand> ops) {
    for (const Operand& o : ops)
        if (o.p && !aligned(o.p, o.dtype == GDN_BF16 ? 2 : 4))
            return set_error(GDN_ERR_UNSUPPORTED, "tensor pointers must be aligned to their type");
    return GDN_OK;
}
// Whether 16-byte pieces of rows can be used for a tensor.
inline bool rows16(const void* p, int dtype, std::initializer_list<int64_t> strides) {
    if (!p) return true;
    if (!aligned(p, 16)) return false;
    for (int64_t s : strides)
        if (s % (dtype == GDN_BF16 ? 8 : 4) != 0) return false;
    return true;
}
// 16-byte pieces of fp32 rows and 8-byte ones of bf16 rows: four numbers.
inline bool rows4(const void* p, int dtype, std::initializer_list<int64_t> strides) {
    if (!p) return true;
    if (!aligned(p, dtype == GDN_BF16 ? 8 : 16)) return false;
    for (int64_t s : strides)
        if (s % 4 != 0) return false;
    return true;
}
// Pairs of a row's numbers.
inline bool rows2(const void* p, int dtype, std::initializer_list<int64_t> strides) {
    if (!p) return true;
    if (!aligned(p, dtype == GDN_BF16 ? 4 : 8)) return false;
    for (int64_t s : strides)
        if (s % 2 != 0) return false;
    return true;
}
// The memory of an operand, from its first element to its last: `rows` rows of
// `row` elements, `stride` apart.
struct Extent {
    const char* name;
    const void* p;
    uint64_t bytes;
    Extent(const char* what, const void* at, int dtype, uint64_t rows, uint64_t row, uint64_t stride)
        : name(what), p(at), bytes(((rows - 1) * stride + row) * (dtype == GDN_BF16 ? 2 : 4)) {}
    Extent(const char* what, const void* at, int dtype, uint64_t n) : Extent(what, at, dtype, 1, n, 0) {}
};
// A token's state is updated where it lies: nothing else that the call reads or
// writes may lie there.
inline gdn_status check_apart(const Extent& out, std::initializer_list<Extent> others) {
    const uint64_t a = reinterpret_cast<uintptr_t>(out.p);
    for (const Extent& o : others) {
        const uint64_t b = reinterpret_cast<uintptr_t>(o.p);
        if (o.p && a < b + o.bytes && b < a + out.bytes)
            return set_error(GDN_ERR_UNSUPPORTED, std::string(out.name) + " may not overlap " + o.name);
    }
    return GDN_OK;
}
inline gdn_status check_workspace(const void* ws, size_t given, size_t need, const char* query) {
    if (need == 0) return GDN_OK;
    if (!ws || given < need) return set_error(GDN_ERR_WORKSPACE, std::string("workspace smaller than ") + query);
    if (!aligned(ws, 256)) return set_error(GDN_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    return GDN_OK;
}
inline gdn_status check_counts(int64_t B, int64_t T, int64_t D) {
    if ((long double)B * T * D > 1.0e15L) return set_error(GDN_ERR_BAD_SHAPE, "tensor too large");
    return GDN_OK;
}

}  // namespace gdn
