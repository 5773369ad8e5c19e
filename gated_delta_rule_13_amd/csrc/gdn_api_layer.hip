// gdn_api_layer.hip -- C ABI of the operators around the recurrence: the
// short convolution, the selective state space recurrence and the head
// normalisation.  Validation, choice of launch shapes, dispatch.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "gdn.h"
#include "gdn_colsum.h"
#include "gdn_conv.h"
#include "gdn_error.h"
#include "gdn_launch.h"
#include "gdn_norm.h"
#include "gdn_ssm.h"

using gdn::set_error;

namespace {

constexpr size_t kInvalid = (size_t)-1;
constexpr int64_t kMaxGrid = 0x7fffffff;
// A launch counts its threads in 32 bits.
bool threads_ok(long double n) { return n <= 4294967295.0L; }

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int t) { return t == GDN_BF16 || t == GDN_F32; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Every pointer that is given is aligned to its type.
struct Operand {
    const void* p;
    int dtype;
};
gdn_status check_aligned(std::initializer_list<Operand> ops) {
    for (const Operand& o : ops)
        if (o.p && !aligned(o.p, o.dtype == GDN_BF16 ? 2 : 4))
            return set_error(GDN_ERR_UNSUPPORTED, "tensor pointers must be aligned to their type");
    return GDN_OK;
}
// Whether 16-byte pieces of rows can be used for a tensor.
bool rows16(const void* p, int dtype, std::initializer_list<int64_t> strides) {
    if (!p) return true;
    if (!aligned(p, 16)) return false;
    for (int64_t s : strides)
        if (s % (dtype == GDN_BF16 ? 8 : 4) != 0) return false;
    return true;
}
// 16-byte pieces of fp32 rows and 8-byte ones of bf16 rows: four numbers.
bool rows4(const void* p, int dtype, std::initializer_list<int64_t> strides) {
    if (!p) return true;
    if (!aligned(p, dtype == GDN_BF16 ? 8 : 16)) return false;
    for (int64_t s : strides)
        if (s % 4 != 0) return false;
    return true;
}
// Pairs of a row's numbers.
bool rows2(const void* p, int dtype, std::initializer_list<int64_t> strides) {
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
gdn_status check_apart(const Extent& out, std::initializer_list<Extent> others) {
    const uint64_t a = reinterpret_cast<uintptr_t>(out.p);
    for (const Extent& o : others) {
        const uint64_t b = reinterpret_cast<uintptr_t>(o.p);
        if (o.p && a < b + o.bytes && b < a + out.bytes)
            return set_error(GDN_ERR_UNSUPPORTED, std::string(out.name) + " may not overlap " + o.name);
    }
    return GDN_OK;
}
gdn_status check_workspace(const void* ws, size_t given, size_t need, const char* query) {
    if (need == 0) return GDN_OK;
    if (!ws || given < need) return set_error(GDN_ERR_WORKSPACE, std::string("workspace smaller than ") + query);
    if (!aligned(ws, 256)) return set_error(GDN_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    return GDN_OK;
}
gdn_status check_counts(int64_t B, int64_t T, int64_t D) {
    if ((long double)B * T * D > 1.0e15L) return set_error(GDN_ERR_BAD_SHAPE, "tensor too large");
    return GDN_OK;
}
// The convolution and the scan count a sequence's tokens in 32 bits, up to a
// tile of 64 and two groups of 8 past its end.
gdn_status check_tokens(int64_t T) {
    if (T > 0x80000000ll - 128) return set_error(GDN_ERR_UNSUPPORTED, "T must be at most 2^31 - 128");
    return GDN_OK;
}

// ---- short convolution ----
gdn_status validate(const gdn_conv_shape* s) {
    if (!s) return set_error(GDN_ERR_NULL_ARG, "shape is NULL");
    if (s->B < 1 || s->T < 1 || s->D < 1 || s->H < 1)
        return set_error(GDN_ERR_BAD_SHAPE, "B, T, D and H must be >= 1");
    if (s->D % s->H != 0) return set_error(GDN_ERR_BAD_SHAPE, "D must be a multiple of H");
    if (!dtype_ok(s->dtype)) return set_error(GDN_ERR_BAD_DTYPE, "dtype must be GDN_BF16 or GDN_F32");
    if (s->W < 2 || s->W > 4) return set_error(GDN_ERR_UNSUPPORTED, "W must be 2, 3 or 4");
    if (s->silu != 0 && s->silu != 1) return set_error(GDN_ERR_UNSUPPORTED, "silu must be 0 or 1");
    if (s->x_stride_b < 0 || s->x_stride_t < 0) return set_error(GDN_ERR_BAD_SHAPE, "strides must be >= 0");
    gdn_status st = check_counts(s->B, s->T, s->D);
    if (st == GDN_OK) st = check_tokens(s->T);
    if (st != GDN_OK) return st;
    if (s->D > (1 << 25)) return set_error(GDN_ERR_UNSUPPORTED, "D must be at most 2^25");
    return GDN_OK;
}

// Rows per thread: long tiles read the W - 1 rows before them less often, but
// the chip wants threads: the longest of 64, 32, 16, 8 that leaves `threads`
// of 16-byte pieces (whichever kernel runs).  Measured at 4 x 4096 x 2048 in
// bf16: the gradient 52 us with 32 rows (29 of its own), 58 with 64.
int conv_rows(const gdn_conv_shape& s, int64_t threads) {
    const int64_t pieces = ceil_div(s.D, s.dtype == GDN_BF16 ? 8 : 4);
    int rows = 64;
    while (rows > 8 && (int64_t)s.B * ceil_div(s.T, rows) * pieces < threads) rows /= 2;
    return rows;
}
int conv_fwd_tile(const gdn_conv_shape& s) { return conv_rows(s, 131072); }
int conv_bwd_tile(const gdn_conv_shape& s) { return conv_rows(s, 131072) - (s.W - 1); }

gdn::ConvParams conv_params(const gdn_conv_shape& s, const void* x, const float* w, const float* bias, const void* s0,
                            const int32_t* lens, int tile, int vec) {
    gdn::ConvParams p{};
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.s0 = s0;
    p.lens = lens;
    p.sb = s.x_stride_b;
    p.st = s.x_stride_t;
    p.B = s.B;
    p.T = s.T;
    p.D = s.D;
    p.hd = s.D / s.H;
    p.nv = s.D / vec;
    p.tile = tile;
    p.ntile = (int)ceil_div(s.T, tile);
    p.silu = s.silu;
    return p;
}

gdn_status conv_forward(const gdn_conv_shape* s, const void* x, const float* weight, const float* bias,
                        const void* state0, const int32_t* lens, void* y, void* state_out, void* stream) {
    if (!x || !weight || !y) return set_error(GDN_ERR_NULL_ARG, "x, weight and y are required");
    gdn_status st = check_aligned({{x, s->dtype}, {weight, GDN_F32}, {bias, GDN_F32}, {state0, s->dtype},
                                   {lens, GDN_F32}, {y, s->dtype}, {state_out, s->dtype}});
    if (st != GDN_OK) return st;
    const int64_t hd = s->D / s->H;
    const bool wide = rows16(x, s->dtype, {s->x_stride_b, s->x_stride_t, hd}) && rows16(y, s->dtype, {hd}) &&
                      rows16(state0, s->dtype, {hd}) && rows16(state_out, s->dtype, {hd});
    gdn::ConvParams p = conv_params(*s, x, weight, bias, state0, lens, conv_fwd_tile(*s),
                                    !wide ? 1 : s->dtype == GDN_BF16 ? 8 : 4);
    p.y = y;
    p.s1 = state_out;
    if ((long double)p.B * p.ntile * p.nv > kMaxGrid) return set_error(GDN_ERR_UNSUPPORTED, "tensor too large");
    gdn::conv_launcher(s->dtype == GDN_BF16, s->W, wide)(p, reinterpret_cast<hipStream_t>(stream));
    return gdn::launch_status();
}

// ---- selective state space recurrence ----
gdn_status validate(const gdn_ssm_shape* s) {
    if (!s) return set_error(GDN_ERR_NULL_ARG, "shape is NULL");
    if (s->B < 1 || s->T < 1 || s->D < 1 || s->N < 1 || s->G < 1)
        return set_error(GDN_ERR_BAD_SHAPE, "B, T, D, N and G must be >= 1");
    if (s->D % s->G != 0) return set_error(GDN_ERR_BAD_SHAPE, "D must be a multiple of G");
    if (!dtype_ok(s->dtype)) return set_error(GDN_ERR_BAD_DTYPE, "dtype must be GDN_BF16 or GDN_F32");
    if (s->N > 64) return set_error(GDN_ERR_UNSUPPORTED, "N must be at most 64");
    if (s->dt_softplus != 0 && s->dt_softplus != 1) return set_error(GDN_ERR_UNSUPPORTED, "dt_softplus must be 0 or 1");
    for (int64_t v : {s->x_stride_b, s->x_stride_t, s->dt_stride_b, s->dt_stride_t, s->z_stride_b, s->z_stride_t,
                      s->b_stride_b, s->b_stride_t, s->c_stride_b, s->c_stride_t})
        if (v < 0) return set_error(GDN_ERR_BAD_SHAPE, "strides must be >= 0");
    // (the kernels address the rows of a group of tokens by 32-bit offsets)
    constexpr int64_t kMaxRow = 1 << 24;
    if (s->D > kMaxRow) return set_error(GDN_ERR_UNSUPPORTED, "D must be at most 2^24");
    if (s->T > 1)
        for (int64_t v : {s->x_stride_t, s->dt_stride_t, s->z_stride_t, s->b_stride_t, s->c_stride_t})
            if (v > kMaxRow) return set_error(GDN_ERR_UNSUPPORTED, "strides of tokens must be at most 2^24");
    const gdn_status st = check_counts(s->B, s->T, (int64_t)s->D * s->N);
    return st != GDN_OK ? st : check_tokens(s->T);
}

// Segments of the forward pass.  One wave takes 64 channels of a segment; the
// chip has 1024 vector units, which hold three such waves each.  Segments cost
// the decays a second time, so there are none when the channels alone give
// that many waves, and as few as do otherwise; of 16 tokens at least, where
// what a segment costs besides its tokens is a fifth of it.  Two more launches
// pay from 64 tokens on (one sequence of 64, 16 states: 20 us either way), and
// with more states from 32 (2 x 33 x 1000 with 64 states: 53 us in one pass, 46
// in segments; 2 x 60: 83 and 47).  Measured at both sides of the number of
// waves, with 16 states: 1024 waves (16 x 2048 x 4096) 790 us in segments, 833
// in one pass; 2048 waves (32 x 1024 x 4096) 764 and 537, 2944 waves (46 x 1024
// x 4096) 959 and 718: from about 1500 on one pass would be faster.
struct SsmPlan {
    int seg_len, nseg;
    size_t off_s, bytes;
};
SsmPlan ssm_fwd_plan(const gdn_ssm_shape& s) {
    const int64_t tiles = (int64_t)s.G * ceil_div(s.D / s.G, 64), waves = s.B * tiles;
    SsmPlan pl{s.T, 1, 0, 0};
    const int64_t want = ceil_div(3 * 1024, waves);
    if (want > 1 && s.T >= (gdn::ssm_states(s.N) > 16 ? 32 : 64)) {
        const int64_t len = ceil_div(ceil_div(s.T, want), gdn::kTok) * gdn::kTok;
        pl.seg_len = (int)(len < 16 ? 16 : len);
        pl.nseg = (int)ceil_div(s.T, pl.seg_len);
    }
    if (pl.nseg > 1) {
        const size_t units = (size_t)waves * pl.nseg;
        pl.off_s = units * gdn::ssm_states(s.N) * 64 * 4;
        pl.bytes = pl.off_s + units * 64 * 4;
    }
    return pl;
}

gdn::SsmParams ssm_params(const gdn_ssm_shape& s, const void* x, const void* dt, const float* A, const void* Bm,
                          const void* C, const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                          const int32_t* lens) {
    gdn::SsmParams p{};
    p.x = x;
    p.dt = dt;
    p.A = A;
    p.Bm = Bm;
    p.C = C;
    p.Dskip = Dskip;
    p.z = z;
    p.dt_bias = dt_bias;
    p.h0 = h0;
    p.lens = lens;
    p.xsb = s.x_stride_b;
    p.xst = s.x_stride_t;
    p.dsb = s.dt_stride_b;
    p.dst = s.dt_stride_t;
    p.zsb = s.z_stride_b;
    p.zst = s.z_stride_t;
    p.bsb = s.b_stride_b;
    p.bst = s.b_stride_t;
    p.csb = s.c_stride_b;
    p.cst = s.c_stride_t;
    p.B = s.B;
    p.T = s.T;
    p.D = s.D;
    p.N = s.N;
    p.G = s.G;
    p.Dg = s.D / s.G;
    p.tpg = (int)ceil_div(p.Dg, 64);
    p.softplus = s.dt_softplus;
    p.wide = s.N % 4 == 0 && aligned(A, 16) && aligned(h0, 16);
    p.seg_len = s.T;
    p.nseg = 1;
    return p;
}

gdn_status ssm_check(const gdn_ssm_shape* s, const void* x, const void* dt, const float* A, const void* Bm, const void* C,
                     const float* Dskip, const void* z, const float* dt_bias, const float* h0, const int32_t* lens) {
    return check_aligned({{x, s->dtype}, {dt, s->dtype}, {A, GDN_F32}, {Bm, s->dtype}, {C, s->dtype}, {Dskip, GDN_F32},
                          {z, s->dtype}, {dt_bias, GDN_F32}, {h0, GDN_F32}, {lens, GDN_F32}});
}

// Parts of the gradient's workspace, in bytes from its start.
struct SsmGradPlan {
    int seg_len, nseg;
    size_t e, r, s, kh, ks, a, d, bc, bytes;
};
SsmGradPlan ssm_bwd_plan(const gdn_ssm_shape& s) {
    SsmGradPlan g{};
    const size_t tiles = (size_t)s.G * ceil_div(s.D / s.G, 64);
    // segments of 64 tokens, or 32 or 16 where those leave fewer than 1024 waves
    // of summaries (one for each vector unit)
    g.seg_len = 64;
    while (g.seg_len > 16 && (int64_t)s.B * tiles * ceil_div(s.T, g.seg_len) < 1024) g.seg_len /= 2;
    g.nseg = (int)ceil_div(s.T, g.seg_len);
    // (one segment: nothing is kept for groups that it does not have)
    if (g.nseg == 1) g.seg_len = (int)ceil_div(s.T, gdn::kTok) * gdn::kTok;
    const size_t units = (size_t)s.B * g.nseg * tiles, ns = gdn::ssm_states(s.N);
    g.e = 0;
    g.r = g.e + units * ns * 64 * 4;
    g.s = g.r + units * ns * 64 * 4;
    g.kh = g.s + units * 64 * 4;
    g.ks = g.kh + units * (g.seg_len / gdn::kTok - 1) * ns * 64 * 4;
    g.a = g.ks + units * (g.seg_len / gdn::kTok - 1) * 64 * 4;
    g.d = g.a + units * ns * 64 * 4;
    g.bc = g.d + units * 2 * 64 * 4;
    g.bytes = g.bc + up256(tiles * s.B * s.T * 2 * ns * 4);
    return g;
}
// Whether the launches of a plan fit: a wave for each segment of 64 channels,
// in the gradient up to eight; the chains, if there are any, a thread for each
// state of a lane, in the gradient both ways; and the gradient's sums, one for
// each number of dB and dC and a workgroup for 64 of the others.
gdn_status ssm_fits(const gdn_ssm_shape& s, int nseg, bool grad) {
    const int ns = gdn::ssm_states(s.N);
    const long double tiles = (long double)s.G * ceil_div(s.D / s.G, 64), lanes = tiles * s.B * 64;
    const bool waves = threads_ok(lanes * nseg * (grad ? 8 : 1));
    const bool chains = (nseg == 1 && !grad) || threads_ok(lanes * ns * (grad ? 2 : 1));
    const bool sums = !grad || threads_ok((long double)s.B * s.T * s.G * 2 * ns + (tiles * (ns + 2) + 1) * gdn::kSumThreads);
    if (!waves || !chains || !sums)
        return set_error(GDN_ERR_UNSUPPORTED, "tensor too large");
    return GDN_OK;
}

// ---- head normalisation ----
gdn_status validate(const gdn_norm_shape* s) {
    if (!s) return set_error(GDN_ERR_NULL_ARG, "shape is NULL");
    if (s->B < 1 || s->T < 1 || s->G < 1 || s->d < 1)
        return set_error(GDN_ERR_BAD_SHAPE, "B, T, G and d must be >= 1");
    if (!dtype_ok(s->x_dtype) || !dtype_ok(s->o_dtype))
        return set_error(GDN_ERR_BAD_DTYPE, "dtype must be GDN_BF16 or GDN_F32");
    if (s->d > gdn::kNormMaxD) return set_error(GDN_ERR_UNSUPPORTED, "d must be at most 4096");
    if ((s->center | s->w_per_group | s->silu) & ~1)
        return set_error(GDN_ERR_UNSUPPORTED, "center, w_per_group and silu must be 0 or 1");
    if (!(s->eps > 0.f)) return set_error(GDN_ERR_BAD_SHAPE, "eps must be > 0");
    for (int64_t v : {s->x_stride_b, s->x_stride_t, s->x_stride_g, s->z_stride_b, s->z_stride_t, s->z_stride_g})
        if (v < 0) return set_error(GDN_ERR_BAD_SHAPE, "strides must be >= 0");
    gdn_status st = check_counts((int64_t)s->B * s->T, s->G, s->d);
    if (st != GDN_OK) return st;
    // (a workgroup for each head, and the gradient's sums over w and b of all)
    if (s->G >= (1 << 24) || (s->w_per_group && (int64_t)s->G * s->d > (1 << 27)))
        return set_error(GDN_ERR_UNSUPPORTED, "G must be below 2^24, and G d at most 2^27 for weights [G, d]");
    return GDN_OK;
}
// Whether the gradient's sums over w and b fit a launch.
gdn_status norm_bwd_fits(const gdn_norm_shape& s) {
    const int64_t cols = 2 * (s.w_per_group ? (int64_t)s.G * s.d : s.d);
    if (!threads_ok(gdn::colsum_threads(cols)))
        return set_error(GDN_ERR_UNSUPPORTED, "G d must be below 2^27 in the gradient for weights [G, d]");
    return GDN_OK;
}
gdn::NormParams norm_params(const gdn_norm_shape& s, const void* x, const float* w, const float* b, const void* z) {
    gdn::NormParams p{};
    p.x = x;
    p.w = w;
    p.b = b;
    p.z = z;
    p.xsb = s.x_stride_b;
    p.xst = s.x_stride_t;
    p.xsg = s.x_stride_g;
    p.zsb = s.z_stride_b;
    p.zst = s.z_stride_t;
    p.zsg = s.z_stride_g;
    p.rows = (int64_t)s.B * s.T * s.G;
    p.T = s.T;
    p.G = s.G;
    p.d = s.d;
    p.center = s.center;
    p.per_group = s.w_per_group;
    p.silu = s.silu;
    p.eps = s.eps;
    return p;
}
// Workgroups that share a head's rows in the gradient, at most: over all heads
// as many as are resident at once on the chip's 256 compute units (measured at
// 2 x 1031 x 30 x 192 in bf16, three on each: 28.5 us; 2048 workgroups, which
// leave a last round half empty, 32.3; 512, 29.8).
int64_t norm_bwd_blocks(const gdn_norm_shape& s, int resident) {
    const int64_t bts = (int64_t)s.B * s.T, all = 256 * resident, most = s.G < all ? all / s.G : 1;
    return bts < most ? bts : most;
}

}  // namespace

extern "C" {

gdn_status gdn_conv_fwd(const gdn_conv_shape* s, const void* x, const float* weight, const float* bias,
                        const void* state0, const int32_t* lens, void* y, void* state_out, void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    return conv_forward(s, x, weight, bias, state0, lens, y, state_out, stream);
}

gdn_status gdn_conv_step(const gdn_conv_shape* s, const void* x, const float* weight, const float* bias, void* state,
                         void* y, void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    if (s->T != 1) return set_error(GDN_ERR_BAD_SHAPE, "T must be 1");
    if (!state) return set_error(GDN_ERR_NULL_ARG, "state is required");
    if (x && weight && y) {
        const int64_t D = s->D;
        const Extent ex("x", x, s->dtype, s->B, D, s->x_stride_b), ew("weight", weight, GDN_F32, D * s->W),
            eb("bias", bias, GDN_F32, D), es("state", state, s->dtype, s->B * (s->W - 1) * D), ey("y", y, s->dtype, s->B * D);
        st = check_apart(es, {ex, ew, eb, ey});
        if (st == GDN_OK) st = check_apart(ey, {ex, ew, eb});
        if (st != GDN_OK) return st;
    }
    return conv_forward(s, x, weight, bias, state, nullptr, y, state, stream);
}

size_t gdn_conv_bwd_workspace_bytes(const gdn_conv_shape* s) {
    gdn::clear_error();
    if (validate(s) != GDN_OK) return kInvalid;
    const int64_t row_tiles = s->B * ceil_div(s->T, conv_bwd_tile(*s));
    return up256((size_t)gdn::conv_bwd_part_rows(row_tiles) * s->D * (s->W + 1) * 4);
}

gdn_status gdn_conv_bwd(const gdn_conv_shape* s, const void* dy, const void* x, const float* weight, const float* bias,
                        const void* state0, const void* dstate_out, const int32_t* lens, void* dx, float* dweight,
                        float* dbias, void* dstate0, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    if (!dy || !x || !weight || !dx || !dweight)
        return set_error(GDN_ERR_NULL_ARG, "dy, x, weight, dx and dweight are required");
    st = check_aligned({{dy, s->dtype}, {x, s->dtype}, {weight, GDN_F32}, {bias, GDN_F32}, {state0, s->dtype},
                        {dstate_out, s->dtype}, {lens, GDN_F32}, {dx, s->dtype}, {dweight, GDN_F32}, {dbias, GDN_F32},
                        {dstate0, s->dtype}});
    if (st != GDN_OK) return st;
    st = check_workspace(workspace, workspace_bytes, gdn_conv_bwd_workspace_bytes(s), "gdn_conv_bwd_workspace_bytes");
    if (st != GDN_OK) return st;
    const int64_t hd = s->D / s->H;
    // (under 256 channels waves are few: 4 x 4096 x 192 in fp32 takes 18.1 us
    // number by number, 19.5 in pairs; 4 x 4096 x 1830 94 and 85, in bf16 72 and 62)
    static_assert(gdn::kConvBwdV == 2, "");
    const bool wide = s->D >= 256 && rows2(x, s->dtype, {s->x_stride_b, s->x_stride_t, hd}) && rows2(dy, s->dtype, {hd}) &&
                      rows2(dx, s->dtype, {hd}) && rows2(state0, s->dtype, {hd}) &&
                      rows2(dstate_out, s->dtype, {hd}) && rows2(dstate0, s->dtype, {hd});
    gdn::ConvBwdParams q{};
    q.f = conv_params(*s, x, weight, bias, state0, lens, conv_bwd_tile(*s), wide ? gdn::kConvBwdV : 1);
    q.dy = dy;
    q.ds1 = dstate_out;
    q.dx = dx;
    q.ds0 = dstate0;
    q.part = static_cast<float*>(workspace);
    const int64_t rows = gdn::conv_bwd_part_rows((int64_t)q.f.B * q.f.ntile);
    if (!threads_ok((long double)rows * ceil_div(q.f.nv, 64) * gdn::kConvThreads))
        return set_error(GDN_ERR_UNSUPPORTED, "tensor too large");
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    gdn::conv_bwd_launcher(s->dtype == GDN_BF16, s->W, wide)(q, hs);
    gdn::conv_bwd_sum(q.part, rows, s->D, s->W, dweight, dbias, hs);
    return gdn::launch_status();
}

size_t gdn_ssm_fwd_workspace_bytes(const gdn_ssm_shape* s) {
    gdn::clear_error();
    if (validate(s) != GDN_OK) return kInvalid;
    const SsmPlan pl = ssm_fwd_plan(*s);
    return ssm_fits(*s, pl.nseg, false) == GDN_OK ? pl.bytes : kInvalid;
}

gdn_status gdn_ssm_fwd(const gdn_ssm_shape* s, const void* x, const void* dt, const float* A, const void* Bm,
                       const void* C, const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                       const int32_t* lens, void* y, float* h_final, void* workspace, size_t workspace_bytes,
                       void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    const SsmPlan pl = ssm_fwd_plan(*s);
    st = ssm_fits(*s, pl.nseg, false);
    if (st != GDN_OK) return st;
    if (!x || !dt || !A || !Bm || !C || !y) return set_error(GDN_ERR_NULL_ARG, "x, dt, A, Bm, C and y are required");
    st = ssm_check(s, x, dt, A, Bm, C, Dskip, z, dt_bias, h0, lens);
    if (st != GDN_OK) return st;
    st = check_aligned({{y, s->dtype}, {h_final, GDN_F32}});
    if (st != GDN_OK) return st;
    st = check_workspace(workspace, workspace_bytes, pl.bytes, "gdn_ssm_fwd_workspace_bytes");
    if (st != GDN_OK) return st;
    gdn::SsmParams p = ssm_params(*s, x, dt, A, Bm, C, Dskip, z, dt_bias, h0, lens);
    p.y = y;
    p.h_final = h_final;
    p.wide_out = s->N % 4 == 0 && aligned(h_final, 16);
    p.seg_len = pl.seg_len;
    p.nseg = pl.nseg;
    p.sum_e = static_cast<float*>(workspace);
    p.sum_s = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_s);
    gdn::ssm_fwd_run(p, s->dtype == GDN_BF16, reinterpret_cast<hipStream_t>(stream));
    return gdn::launch_status();
}

gdn_status gdn_ssm_step(const gdn_ssm_shape* s, const void* x, const void* dt, const float* A, const void* Bm,
                        const void* C, const float* Dskip, const void* z, const float* dt_bias, float* h, void* y,
                        void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    if (s->T != 1) return set_error(GDN_ERR_BAD_SHAPE, "T must be 1");
    if (!x || !dt || !A || !Bm || !C || !h || !y)
        return set_error(GDN_ERR_NULL_ARG, "x, dt, A, Bm, C, h and y are required");
    st = ssm_check(s, x, dt, A, Bm, C, Dskip, z, dt_bias, h, nullptr);
    if (st != GDN_OK) return st;
    st = check_aligned({{y, s->dtype}});
    if (st != GDN_OK) return st;
    gdn::SsmStepParams q{};
    q.f = ssm_params(*s, x, dt, A, Bm, C, Dskip, z, dt_bias, nullptr, nullptr);
    q.f.y = y;
    q.h = h;
    q.wide = s->N % 4 == 0 && aligned(h, 16) && aligned(A, 16);
    q.wide_bc = s->N % 4 == 0 && rows4(Bm, s->dtype, {s->b_stride_b}) && rows4(C, s->dtype, {s->c_stride_b});
    // (the grid's second dimension counts sequences)
    if (s->B > 65535) return set_error(GDN_ERR_UNSUPPORTED, "B must be at most 65535");
    const int64_t B = s->B, D = s->D, bc = (int64_t)s->G * s->N;
    const Extent ex("x", x, s->dtype, B, D, s->x_stride_b), ed("dt", dt, s->dtype, B, D, s->dt_stride_b),
        eA("A", A, GDN_F32, D * s->N), eB("Bm", Bm, s->dtype, B, bc, s->b_stride_b), eC("C", C, s->dtype, B, bc, s->c_stride_b),
        eD("Dskip", Dskip, GDN_F32, D), ez("z", z, s->dtype, B, D, s->z_stride_b), eb("dt_bias", dt_bias, GDN_F32, D),
        eh("h", h, GDN_F32, B * D * s->N), ey("y", y, s->dtype, B * D);
    st = check_apart(eh, {ex, ed, eA, eB, eC, eD, ez, eb, ey});
    if (st == GDN_OK) st = check_apart(ey, {ex, ed, eA, eB, eC, eD, ez, eb});
    if (st != GDN_OK) return st;
    gdn::ssm_step_run(q, s->dtype == GDN_BF16, reinterpret_cast<hipStream_t>(stream));
    return gdn::launch_status();
}

size_t gdn_ssm_bwd_workspace_bytes(const gdn_ssm_shape* s) {
    gdn::clear_error();
    if (validate(s) != GDN_OK) return kInvalid;
    const SsmGradPlan pl = ssm_bwd_plan(*s);
    return ssm_fits(*s, pl.nseg, true) == GDN_OK ? pl.bytes : kInvalid;
}

gdn_status gdn_ssm_bwd(const gdn_ssm_shape* s, const void* dy, const void* x, const void* dt, const float* A,
                       const void* Bm, const void* C, const float* Dskip, const void* z, const float* dt_bias,
                       const float* h0, const float* dh_final, const int32_t* lens, void* dx, void* ddt, float* dA,
                       void* dBm, void* dC, float* dDskip, void* dz, float* ddt_bias, float* dh0, void* workspace,
                       size_t workspace_bytes, void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    const SsmGradPlan pl = ssm_bwd_plan(*s);
    st = ssm_fits(*s, pl.nseg, true);
    if (st != GDN_OK) return st;
    if (!dy || !x || !dt || !A || !Bm || !C || !dx || !ddt || !dA || !dBm || !dC)
        return set_error(GDN_ERR_NULL_ARG, "dy, x, dt, A, Bm, C, dx, ddt, dA, dBm and dC are required");
    if ((z != nullptr) != (dz != nullptr)) return set_error(GDN_ERR_NULL_ARG, "dz goes with z");
    st = ssm_check(s, x, dt, A, Bm, C, Dskip, z, dt_bias, h0, lens);
    if (st != GDN_OK) return st;
    st = check_aligned({{dy, s->dtype}, {dh_final, GDN_F32}, {dx, s->dtype}, {ddt, s->dtype}, {dA, GDN_F32},
                        {dBm, s->dtype}, {dC, s->dtype}, {dDskip, GDN_F32}, {dz, s->dtype}, {ddt_bias, GDN_F32},
                        {dh0, GDN_F32}});
    if (st != GDN_OK) return st;
    st = check_workspace(workspace, workspace_bytes, pl.bytes, "gdn_ssm_bwd_workspace_bytes");
    if (st != GDN_OK) return st;
    gdn::SsmParams p = ssm_params(*s, x, dt, A, Bm, C, Dskip, z, dt_bias, h0, lens);
    char* ws = static_cast<char*>(workspace);
    p.seg_len = pl.seg_len;
    p.nseg = pl.nseg;
    p.dy = dy;
    p.dh_final = dh_final;
    p.dx = dx;
    p.ddt = ddt;
    p.dz = dz;
    p.dh0 = dh0;
    p.sum_e = reinterpret_cast<float*>(ws + pl.e);
    p.sum_r = reinterpret_cast<float*>(ws + pl.r);
    p.sum_s = reinterpret_cast<float*>(ws + pl.s);
    p.keep_h = reinterpret_cast<float*>(ws + pl.kh);
    p.keep_s = reinterpret_cast<float*>(ws + pl.ks);
    p.part_a = reinterpret_cast<float*>(ws + pl.a);
    p.part_d = reinterpret_cast<float*>(ws + pl.d);
    p.part_bc = reinterpret_cast<float*>(ws + pl.bc);
    gdn::ssm_bwd_run(p, s->dtype == GDN_BF16, dA, dBm, dC, dDskip, ddt_bias, reinterpret_cast<hipStream_t>(stream));
    return gdn::launch_status();
}

gdn_status gdn_norm_fwd(const gdn_norm_shape* s, const void* x, const float* weight, const float* bias, const void* z,
                        void* y, void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    if (!x || !y) return set_error(GDN_ERR_NULL_ARG, "x and y are required");
    st = check_aligned({{x, s->x_dtype}, {weight, GDN_F32}, {bias, GDN_F32}, {z, s->o_dtype}, {y, s->o_dtype}});
    if (st != GDN_OK) return st;
    gdn::NormParams p = norm_params(*s, x, weight, bias, z);
    p.y = y;
    const bool wide = rows4(x, s->x_dtype, {s->d, s->x_stride_b, s->x_stride_t, s->x_stride_g}) &&
                      rows4(y, s->o_dtype, {s->d}) &&
                      rows4(z, s->o_dtype, {s->z_stride_b, s->z_stride_t, s->z_stride_g});
    gdn::NormLauncher fwd = nullptr;
    gdn::NormBwdLauncher bwd = nullptr;
    int resident = 0;
    gdn::norm_launchers(s->x_dtype == GDN_BF16, s->o_dtype == GDN_BF16, s->d, wide, &fwd, &bwd, &resident);
    fwd(p, reinterpret_cast<hipStream_t>(stream));
    return gdn::launch_status();
}

size_t gdn_norm_bwd_workspace_bytes(const gdn_norm_shape* s) {
    gdn::clear_error();
    if (validate(s) != GDN_OK || norm_bwd_fits(*s) != GDN_OK) return kInvalid;
    return up256((size_t)norm_bwd_blocks(*s, gdn::kNormResident) * 2 * s->G * s->d * 4);
}

gdn_status gdn_norm_bwd(const gdn_norm_shape* s, const void* dy, const void* x, const float* weight, const float* bias,
                        const void* z, void* dx, int64_t dx_stride_b, int64_t dx_stride_t, int64_t dx_stride_g,
                        float* dweight, float* dbias, void* dz, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::clear_error();
    gdn_status st = validate(s);
    if (st == GDN_OK) st = norm_bwd_fits(*s);
    if (st != GDN_OK) return st;
    if (!dy || !x || !dx) return set_error(GDN_ERR_NULL_ARG, "dy, x and dx are required");
    if ((z != nullptr) != (dz != nullptr)) return set_error(GDN_ERR_NULL_ARG, "dz goes with z");
    if ((s->B > 1 && dx_stride_b < s->d) || (s->T > 1 && dx_stride_t < s->d) || (s->G > 1 && dx_stride_g < s->d))
        return set_error(GDN_ERR_BAD_SHAPE, "the rows of dx may not overlap");
    st = check_aligned({{dy, s->o_dtype}, {x, s->x_dtype}, {weight, GDN_F32}, {bias, GDN_F32}, {z, s->o_dtype},
                        {dx, s->x_dtype}, {dweight, GDN_F32}, {dbias, GDN_F32}, {dz, s->o_dtype}});
    if (st != GDN_OK) return st;
    st = check_workspace(workspace, workspace_bytes, gdn_norm_bwd_workspace_bytes(s), "gdn_norm_bwd_workspace_bytes");
    if (st != GDN_OK) return st;
    gdn::NormBwdParams q{};
    q.f = norm_params(*s, x, weight, bias, z);
    q.dy = dy;
    q.dx = dx;
    q.dz = dz;
    q.dsb = dx_stride_b;
    q.dst = dx_stride_t;
    q.dsg = dx_stride_g;
    q.part = static_cast<float*>(workspace);
    const bool wide = rows4(x, s->x_dtype, {s->d, s->x_stride_b, s->x_stride_t, s->x_stride_g}) &&
                      rows4(dy, s->o_dtype, {s->d}) && rows4(dz, s->o_dtype, {s->d}) &&
                      rows4(dx, s->x_dtype, {dx_stride_b, dx_stride_t, dx_stride_g}) &&
                      rows4(z, s->o_dtype, {s->z_stride_b, s->z_stride_t, s->z_stride_g});
    gdn::NormLauncher fwd = nullptr;
    gdn::NormBwdLauncher bwd = nullptr;
    int resident = 0;
    gdn::norm_launchers(s->x_dtype == GDN_BF16, s->o_dtype == GDN_BF16, s->d, wide, &fwd, &bwd, &resident);
    const int nblk = (int)norm_bwd_blocks(*s, resident);
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    bwd(q, nblk, hs);
    gdn::norm_bwd_sum(q, nblk, dweight, dbias, hs);
    return gdn::launch_status();
}

}  // extern "C"
