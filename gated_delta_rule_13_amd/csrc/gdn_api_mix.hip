// gdn_api_mix.hip -- C ABI of linear attention with decay and of the norms
// around a block.  Validation, choice of launch shapes, dispatch.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "gdn.h"
#include "gdn_block.h"
#include "gdn_check.h"
#include "gdn_colsum.h"
#include "gdn_error.h"
#include "gdn_launch.h"
#include "gdn_lin.h"
#include "gdn_lin_join.h"

using namespace gdn;

namespace {

// ---- linear attention ----
gdn_status validate(const gdn_lin_shape* s) {
    if (!s) return set_error(GDN_ERR_NULL_ARG, "shape is NULL");
    if (s->B < 1 || s->H < 1 || s->T < 1 || s->Hq < 1 || s->Hk < 1 || s->d_k < 1 || s->d_v < 1)
        return set_error(GDN_ERR_BAD_SHAPE, "B, H, T, Hq, Hk, d_k and d_v must be >= 1");
    if (s->H % s->Hq != 0 || s->H % s->Hk != 0) return set_error(GDN_ERR_BAD_SHAPE, "H must be a multiple of Hq and of Hk");
    if (!dtype_ok(s->dtype) || !dtype_ok(s->o_dtype))
        return set_error(GDN_ERR_BAD_DTYPE, "dtype and o_dtype must be GDN_BF16 or GDN_F32");
    if (s->d_k > 256 || s->d_v > 256) return set_error(GDN_ERR_UNSUPPORTED, "d_k and d_v must be at most 256");
    if (s->per_head != 0 && s->per_head != 1) return set_error(GDN_ERR_UNSUPPORTED, "per_head must be 0 or 1");
    for (int64_t x : {s->q_stride_b, s->q_stride_h, s->q_stride_t, s->k_stride_b, s->k_stride_h, s->k_stride_t,
                      s->v_stride_b, s->v_stride_h, s->v_stride_t, s->a_stride_b, s->a_stride_h, s->a_stride_t})
        if (x < 0) return set_error(GDN_ERR_BAD_SHAPE, "strides must be >= 0");
    gdn_status st = check_counts((int64_t)s->B * s->H, s->T, 256);
    if (st != GDN_OK) return st;
    if (s->T > 0x80000000ll - 128) return set_error(GDN_ERR_UNSUPPORTED, "T must be at most 2^31 - 128");
    return GDN_OK;
}

int lin_rows(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : 256; }
int lin_tiles(int d) { return (int)ceil_div(d, kLinTile); }
LinLauncher lin_launcher(int dtype, int nk, int set) {
    const bool bf = dtype == GDN_BF16;
    switch (nk) {
        case 32: return bf ? lin_launcher_1_32(set) : lin_launcher_0_32(set);
        case 64: return bf ? lin_launcher_1_64(set) : lin_launcher_0_64(set);
        case 96: return bf ? lin_launcher_1_96(set) : lin_launcher_0_96(set);
        case 128: return bf ? lin_launcher_1_128(set) : lin_launcher_0_128(set);
        default: return bf ? lin_launcher_1_256(set) : lin_launcher_0_256(set);
    }
}
int64_t lin_blocks(int64_t units, int tiles) { return ceil_div(units, kXcds) * kXcds * tiles; }

// Segments: where the heads and tiles leave compute units idle, the tokens are
// cut, into 256 each at least, so that they have about two workgroups each, or in
// the gradient those of its smallest launch (the tiles of dq) one each.  They
// cost a pass over the rows for their sums, and win by the units that work:
// 1 x 8 x 32768 of 128/128 take 156 us, the same tokens as 64 heads 101 without;
// their gradient with decays 529 us, and 623 where its launches aim at two
// workgroups each together.  (Forward, 256 or 1024 workgroups measure alike.)
struct LinPlanSizes {
    int nseg, seg_len;
    int64_t units;
    size_t sum, sum_d, decay, sums_q, sums_k, hold, dla, dq, dk, bytes;
};
LinPlanSizes lin_plan(const gdn_lin_shape& s, bool grad) {
    LinPlanSizes pl{};
    const int64_t bh = (int64_t)s.B * s.H;
    const int64_t groups = bh * (lin_tiles(s.d_v) + (grad ? 2 * lin_tiles(s.d_k) : 0));
    int64_t nseg = groups >= 256 ? 1 : grad ? 256 / (bh * lin_tiles(s.d_k)) : ceil_div(512, groups);
    if (nseg > ceil_div(s.T, 256)) nseg = ceil_div(s.T, 256);
    pl.seg_len = (int)(ceil_div(ceil_div(s.T, nseg), 64) * 64);
    pl.nseg = (int)ceil_div(s.T, pl.seg_len);
    pl.units = bh * pl.nseg;
    size_t at = 0;
    auto take = [&](bool want, int64_t numbers) {
        const size_t here = at;
        if (want) at += up256((size_t)numbers * 4);
        return here;
    };
    const int64_t plane = (int64_t)s.d_k * s.d_v, tokens = bh * s.T, tiles = lin_tiles(s.d_k);
    const int C = lin_chunk(s.dtype == GDN_BF16, lin_rows(s.d_v));
    pl.sum = take(pl.nseg > 1, pl.units * plane);
    pl.decay = take(pl.nseg > 1, pl.units);
    if (grad) {
        pl.sum_d = take(pl.nseg > 1, pl.units * plane);
        pl.sums_q = take(true, tiles * tokens);
        pl.sums_k = take(true, tiles * tokens);
        pl.hold = take(true, tiles * bh * ceil_div(s.T, C) * lin_rows(s.d_v) * kLinTile);
        pl.dla = take(s.per_head, tokens);
        pl.dq = take(s.Hq < s.H, tokens * s.d_k);
        pl.dk = take(s.Hk < s.H, tokens * s.d_k);
    }
    pl.bytes = at;
    return pl;
}
gdn_status lin_fits(const gdn_lin_shape& s, bool grad) {
    const LinPlanSizes pl = lin_plan(s, grad);
    const int64_t bh = (int64_t)s.B * s.H;
    const int tiles = lin_tiles(s.d_v) + (grad ? 2 * lin_tiles(s.d_k) : 0);
    bool ok = threads_ok((long double)lin_blocks(pl.units, tiles) * kLinThreads);
    if (grad) {
        ok = ok && threads_ok((long double)bh * s.T + 256);
        if (s.Hq < s.H) ok = ok && threads_ok((long double)s.B * s.Hq * s.T * s.d_k + 256);
        if (s.Hk < s.H) ok = ok && threads_ok((long double)s.B * s.Hk * s.T * s.d_k + 256);
        ok = ok && threads_ok((long double)s.H * 1024);
    }
    return ok ? GDN_OK : set_error(GDN_ERR_UNSUPPORTED, "more workgroups than a launch holds");
}

LinTensor lin_tensor(const void* p, int dtype, int d, int64_t sb, int64_t sh, int64_t st, int rep) {
    LinTensor t{};
    t.p = p;
    t.sb = sb;
    t.sh = sh;
    t.st = st;
    t.rep = rep;
    t.wide = rows16(p, dtype, {sb, sh, st});
    // (a chunk's rows within 32 bits of its first)
    const int bytes = dtype == GDN_BF16 ? 2 : 4;
    t.direct = t.wide && d * bytes % 16 == 0 && st < (1ll << 31) / (64 * bytes);
    return t;
}
LinParams lin_params(const gdn_lin_shape& s, const LinPlanSizes& pl, const float* log_alpha, const int32_t* lens, char* ws) {
    LinParams p{};
    p.log_alpha = log_alpha;
    p.lsb = s.per_head ? 0 : s.a_stride_b;
    p.lsh = s.per_head ? 1 : s.a_stride_h;
    p.lst = s.per_head ? 0 : s.a_stride_t;
    p.lens = lens;
    p.units = pl.units;
    p.B = s.B;
    p.H = s.H;
    p.T = s.T;
    p.dk = s.d_k;
    p.dv = s.d_v;
    p.nseg = pl.nseg;
    p.seg_len = pl.seg_len;
    p.scale = s.scale;
    p.seg_sum = reinterpret_cast<float*>(ws + pl.sum);
    p.seg_sum_d = reinterpret_cast<float*>(ws + pl.sum_d);
    p.seg_decay = reinterpret_cast<float*>(ws + pl.decay);
    return p;
}
LinRole lin_role(const LinTensor& a, const LinTensor& b, const LinTensor& c, int nk, int nv, void* out, bool out_bf16) {
    LinRole r{};
    r.a = a;
    r.b = b;
    r.c = c;
    r.nk = nk;
    r.nv = nv;
    r.tiles = lin_tiles(nv);
    r.out = out;
    r.out_bf16 = out_bf16;
    r.out_wide = out_bf16 && rows16(out, GDN_BF16, {nv}) ? 8 : rows4(out, out_bf16 ? GDN_BF16 : GDN_F32, {nv}) ? 4 : 1;
    return r;
}
// What the segments add to the state (and to its gradient), and the states that
// they start from.
void lin_segments(const LinParams& base, const gdn_lin_shape& s, const LinTensor& q, const LinTensor& k, const LinTensor& v,
                  const LinTensor* dO, const float* S0, const float* dS_final, hipStream_t st) {
    LinParams p = base;
    p.r[0] = lin_role(q, k, v, s.d_k, s.d_v, nullptr, false);
    if (dO) p.r[1] = lin_role(k, q, *dO, s.d_k, s.d_v, nullptr, false);
    const int tiles = p.r[0].tiles * (dO ? 2 : 1);
    lin_launcher(s.dtype, lin_rows(s.d_k), dO ? kLinSetSums : kLinSetSum)(p, lin_blocks(p.units, tiles), st);
    const int64_t plane = (int64_t)s.d_k * s.d_v;
    const LinChainParams f{p.seg_sum, p.seg_decay, S0, plane, p.nseg, 0}, r{p.seg_sum_d, p.seg_decay, dS_final, plane, p.nseg, 1};
    hipLaunchKernelGGL(gdn_lin_chain_kernel, dim3((unsigned)ceil_div(plane, 256), (unsigned)(s.B * s.H), dO ? 2 : 1), dim3(256), 0, st,
                       f, r);
}

// ---- norms around a block ----
gdn_status validate(const gdn_block_norm_shape* s) {
    if (!s) return set_error(GDN_ERR_NULL_ARG, "shape is NULL");
    if (s->B < 1 || s->T < 1 || s->D < 1) return set_error(GDN_ERR_BAD_SHAPE, "B, T and D must be >= 1");
    if (!dtype_ok(s->dtype) || !dtype_ok(s->x_dtype))
        return set_error(GDN_ERR_BAD_DTYPE, "dtype and x_dtype must be GDN_BF16 or GDN_F32");
    if (s->D > kBlockMaxD) return set_error(GDN_ERR_UNSUPPORTED, "D must be at most 16384");
    if (s->post != 0 && s->post != 1) return set_error(GDN_ERR_UNSUPPORTED, "post must be 0 or 1");
    if (s->act < 0 || s->act > 2) return set_error(GDN_ERR_UNSUPPORTED, "act must be 0, 1 or 2");
    if (!(s->eps > 0.f)) return set_error(GDN_ERR_BAD_SHAPE, "eps must be > 0");
    for (int64_t x : {s->o_stride_b, s->o_stride_t, s->x_stride_b, s->x_stride_t, s->g_stride_b, s->g_stride_t})
        if (x < 0) return set_error(GDN_ERR_BAD_SHAPE, "strides must be >= 0");
    return check_counts(s->B, s->T, s->D);
}
BlockLaunchers block_launchers(const gdn_block_norm_shape& s, bool wide) {
    const bool xb = s.x_dtype == GDN_BF16, ob = s.dtype == GDN_BF16;
    if (xb) return ob ? block_launchers_1_1(s.D, wide) : block_launchers_1_0(s.D, wide);
    return ob ? block_launchers_0_1(s.D, wide) : block_launchers_0_0(s.D, wide);
}
// Workgroups, which stay for all rows: 1024 of 256 lanes forward (512 to 2048
// measure alike, 256 50 % slower at 4 x 4096 x 2048), 512 backward, each of which
// leaves a row of sums for the weights (152 us at that size; 1024 take 164, 256
// 179); fewer of more lanes.
int64_t block_groups(const gdn_block_norm_shape& s, bool grad) {
    const int lanes = block_lanes(s.D), threads = lanes < 256 ? 256 : lanes;
    const int64_t need = ceil_div((int64_t)s.B * s.T, threads / lanes), most = (grad ? 512 : 1024) * 256 / threads;
    return need < most ? need : most;
}
BlockParams block_params(const gdn_block_norm_shape& s, const void* o, const void* x, const void* g, const float* w_post,
                         const float* scale, const float* w_pre) {
    BlockParams p{};
    p.o = o;
    p.x = x;
    p.g = g;
    p.w_post = w_post;
    p.scale = scale;
    p.w_pre = w_pre;
    p.osb = s.o_stride_b;
    p.ost = s.o_stride_t;
    p.xsb = s.x_stride_b;
    p.xst = s.x_stride_t;
    p.gsb = s.g_stride_b;
    p.gst = s.g_stride_t;
    p.rows = (int64_t)s.B * s.T;
    p.T = s.T;
    p.D = s.D;
    p.post = s.post;
    p.act = s.act;
    p.eps = s.eps;
    return p;
}

}  // namespace

extern "C" {

size_t gdn_lin_fwd_workspace_bytes(const gdn_lin_shape* s) {
    clear_error();
    if (validate(s) != GDN_OK || lin_fits(*s, false) != GDN_OK) return kInvalid;
    return lin_plan(*s, false).bytes;
}

gdn_status gdn_lin_fwd(const gdn_lin_shape* s, const void* q, const void* k, const void* v, const float* log_alpha,
                       const float* S0, const int32_t* lens, void* O, float* S_final, void* workspace, size_t workspace_bytes,
                       void* stream) {
    clear_error();
    gdn_status st = validate(s);
    if (st == GDN_OK) st = lin_fits(*s, false);
    if (st != GDN_OK) return st;
    if (!q || !k || !v || !O) return set_error(GDN_ERR_NULL_ARG, "q, k, v and O are required");
    st = check_aligned({{q, s->dtype}, {k, s->dtype}, {v, s->dtype}, {log_alpha, GDN_F32}, {S0, GDN_F32}, {lens, GDN_F32},
                        {O, s->o_dtype}, {S_final, GDN_F32}});
    if (st != GDN_OK) return st;
    const LinPlanSizes pl = lin_plan(*s, false);
    st = check_workspace(workspace, workspace_bytes, pl.bytes, "gdn_lin_fwd_workspace_bytes");
    if (st != GDN_OK) return st;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const LinTensor tq = lin_tensor(q, s->dtype, s->d_k, s->q_stride_b, s->q_stride_h, s->q_stride_t, s->H / s->Hq),
                    tk = lin_tensor(k, s->dtype, s->d_k, s->k_stride_b, s->k_stride_h, s->k_stride_t, s->H / s->Hk),
                    tv = lin_tensor(v, s->dtype, s->d_v, s->v_stride_b, s->v_stride_h, s->v_stride_t, 1);
    LinParams p = lin_params(*s, pl, log_alpha, lens, static_cast<char*>(workspace));
    if (pl.nseg > 1) lin_segments(p, *s, tq, tk, tv, nullptr, S0, nullptr, hs);
    p.r[0] = lin_role(tq, tk, tv, s->d_k, s->d_v, O, s->o_dtype == GDN_BF16);
    p.r[0].first = S0;
    p.r[0].carry = pl.nseg > 1 ? p.seg_sum : nullptr;
    p.r[0].last = S_final;
    lin_launcher(s->dtype, lin_rows(s->d_k), kLinSetFwd)(p, lin_blocks(p.units, p.r[0].tiles), hs);
    return launch_status();
}

gdn_status gdn_lin_step(const gdn_lin_shape* s, const void* q, const void* k, const void* v, const float* log_alpha, float* S,
                        void* O, void* stream) {
    clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    if (s->T != 1) return set_error(GDN_ERR_BAD_SHAPE, "gdn_lin_step takes T = 1");
    if (!q || !k || !v || !S || !O) return set_error(GDN_ERR_NULL_ARG, "q, k, v, S and O are required");
    st = check_aligned({{q, s->dtype}, {k, s->dtype}, {v, s->dtype}, {log_alpha, GDN_F32}, {S, GDN_F32}, {O, s->o_dtype}});
    if (st != GDN_OK) return st;
    const int64_t bh = (int64_t)s->B * s->H;
    auto heads = [&](const char* name, const void* p, int dtype, int64_t sb, int64_t sh, int H, int d) {
        return Extent(name, p, dtype, 1, (uint64_t)((s->B - 1) * sb + (H - 1) * sh + d), 0);
    };
    const Extent eq = heads("q", q, s->dtype, s->q_stride_b, s->q_stride_h, s->Hq, s->d_k),
                 ek = heads("k", k, s->dtype, s->k_stride_b, s->k_stride_h, s->Hk, s->d_k),
                 ev = heads("v", v, s->dtype, s->v_stride_b, s->v_stride_h, s->H, s->d_v),
                 ea = heads("log_alpha", log_alpha, GDN_F32, s->per_head ? 0 : s->a_stride_b, s->per_head ? 1 : s->a_stride_h, s->H, 1),
                 eS("S", S, GDN_F32, (uint64_t)bh * s->d_v * s->d_k), eO("O", O, s->o_dtype, (uint64_t)bh * s->d_v);
    st = check_apart(eS, {eq, ek, ev, ea, eO});
    if (st == GDN_OK) st = check_apart(eO, {eq, ek, ev, ea});
    if (st != GDN_OK) return st;
    LinStepParams p{};
    p.q = lin_tensor(q, s->dtype, s->d_k, s->q_stride_b, s->q_stride_h, 0, s->H / s->Hq);
    p.k = lin_tensor(k, s->dtype, s->d_k, s->k_stride_b, s->k_stride_h, 0, s->H / s->Hk);
    p.v = lin_tensor(v, s->dtype, s->d_v, s->v_stride_b, s->v_stride_h, 0, 1);
    p.log_alpha = log_alpha;
    p.lsb = s->per_head ? 0 : s->a_stride_b;
    p.lsh = s->per_head ? 1 : s->a_stride_h;
    p.S = S;
    p.out = O;
    p.H = s->H;
    p.dk = s->d_k;
    p.dv = s->d_v;
    p.out_bf16 = s->o_dtype == GDN_BF16;
    p.scale = s->scale;
    const bool wide = rows4(S, GDN_F32, {s->d_k}) && rows4(q, s->dtype, {s->q_stride_b, s->q_stride_h}) &&
                      rows4(k, s->dtype, {s->k_stride_b, s->k_stride_h});
    int rows = 0;
    const LinStepLauncher run = s->dtype == GDN_BF16 ? lin_step_launcher_bf16(s->d_k, wide, &rows) : lin_step_launcher_f32(s->d_k, wide, &rows);
    p.blocks = (int)ceil_div(s->d_v, rows);
    if (!threads_ok((long double)bh * p.blocks * kLinStepThreads))
        return set_error(GDN_ERR_UNSUPPORTED, "more workgroups than a launch holds");
    run(p, bh, reinterpret_cast<hipStream_t>(stream));
    return launch_status();
}

size_t gdn_lin_bwd_workspace_bytes(const gdn_lin_shape* s) {
    clear_error();
    if (validate(s) != GDN_OK || lin_fits(*s, true) != GDN_OK) return kInvalid;
    return lin_plan(*s, true).bytes;
}

gdn_status gdn_lin_bwd(const gdn_lin_shape* s, const void* dO, const void* q, const void* k, const void* v, const float* log_alpha,
                       const float* S0, const float* dS_final, const int32_t* lens, void* dq, void* dk, void* dv,
                       float* dlog_alpha, float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    gdn_status st = validate(s);
    if (st == GDN_OK) st = lin_fits(*s, true);
    if (st != GDN_OK) return st;
    if (!dO || !q || !k || !v || !dq || !dk || !dv) return set_error(GDN_ERR_NULL_ARG, "dO, q, k, v, dq, dk and dv are required");
    if (dlog_alpha && !log_alpha) return set_error(GDN_ERR_NULL_ARG, "dlog_alpha goes with log_alpha");
    st = check_aligned({{dO, s->dtype}, {q, s->dtype}, {k, s->dtype}, {v, s->dtype}, {log_alpha, GDN_F32}, {S0, GDN_F32},
                        {dS_final, GDN_F32}, {lens, GDN_F32}, {dq, s->dtype}, {dk, s->dtype}, {dv, s->dtype},
                        {dlog_alpha, GDN_F32}, {dS0, GDN_F32}});
    if (st != GDN_OK) return st;
    const LinPlanSizes pl = lin_plan(*s, true);
    st = check_workspace(workspace, workspace_bytes, pl.bytes, "gdn_lin_bwd_workspace_bytes");
    if (st != GDN_OK) return st;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const LinTensor tq = lin_tensor(q, s->dtype, s->d_k, s->q_stride_b, s->q_stride_h, s->q_stride_t, s->H / s->Hq),
                    tk = lin_tensor(k, s->dtype, s->d_k, s->k_stride_b, s->k_stride_h, s->k_stride_t, s->H / s->Hk),
                    tv = lin_tensor(v, s->dtype, s->d_v, s->v_stride_b, s->v_stride_h, s->v_stride_t, 1),
                    td = lin_tensor(dO, s->dtype, s->d_v, (int64_t)s->H * s->T * s->d_v, (int64_t)s->T * s->d_v, s->d_v, 1);
    LinParams p = lin_params(*s, pl, log_alpha, lens, ws);
    if (pl.nseg > 1) lin_segments(p, *s, tq, tk, tv, &td, S0, dS_final, hs);
    const float* carry = pl.nseg > 1 ? p.seg_sum : nullptr;
    const float* carry_d = pl.nseg > 1 ? p.seg_sum_d : nullptr;
    const bool bf = s->dtype == GDN_BF16;
    auto sum = [&](size_t at) { return dlog_alpha ? reinterpret_cast<float*>(ws + at) : nullptr; };
    const bool gq = s->Hq < s->H, gk = s->Hk < s->H;
    LinRole rq = lin_role(td, tv, tk, s->d_v, s->d_k, gq ? ws + pl.dq : dq, bf && !gq);
    rq.x = tq;
    rq.first = S0;
    rq.carry = carry;
    rq.sums = sum(pl.sums_q);
    rq.hold = sum(pl.hold);
    LinRole rk = lin_role(tv, td, tq, s->d_v, s->d_k, gk ? ws + pl.dk : dk, bf && !gk);
    rk.x = tk;
    rk.first = dS_final;
    rk.carry = carry_d;
    rk.sums = sum(pl.sums_k);
    rk.hold = sum(pl.hold);
    LinRole rv = lin_role(tk, tq, td, s->d_k, s->d_v, dv, bf);
    rv.first = dS_final;
    rv.carry = carry_d;
    rv.last = dS0;
    const int rows_k = lin_rows(s->d_k), rows_v = lin_rows(s->d_v);
    auto pass = [&](LinSet set, int rows, std::initializer_list<LinRole> roles) {
        int tiles = 0, n = 0;
        for (const LinRole& r : roles) {
            p.r[n++] = r;
            tiles += r.tiles;
        }
        lin_launcher(s->dtype, rows, set)(p, lin_blocks(p.units, tiles), hs);
    };
    if (dlog_alpha) {
        if (rows_k == rows_v) {
            pass(kLinSetKvSums, rows_v, {rk, rv});
        } else {
            pass(kLinSetKSums, rows_v, {rk});
            pass(kLinSetV, rows_k, {rv});
        }
        pass(kLinSetQSums, rows_v, {rq});
    } else if (rows_k == rows_v) {
        pass(kLinSetAll, rows_v, {rq, rk, rv});
    } else {
        pass(kLinSetQk, rows_v, {rq, rk});
        pass(kLinSetV, rows_k, {rv});
    }
    auto groups = [&](bool want, size_t from, void* to, int heads) {
        if (!want) return;
        const int64_t row = (int64_t)s->T * s->d_k;
        const LinGroupParams g{reinterpret_cast<const float*>(ws + from), to, row, s->B * heads * row, s->H / heads};
        const dim3 grid((unsigned)ceil_div(g.n, 256));
        if (bf) hipLaunchKernelGGL((gdn_lin_group_sum_kernel<true>), grid, dim3(256), 0, hs, g);
        else hipLaunchKernelGGL((gdn_lin_group_sum_kernel<false>), grid, dim3(256), 0, hs, g);
    };
    groups(gq, pl.dq, dq, s->Hq);
    groups(gk, pl.dk, dk, s->Hk);
    if (dlog_alpha) {
        LinDecayParams d{};
        d.sums_q = rq.sums;
        d.sums_k = rk.sums;
        d.log_alpha = log_alpha;
        d.lsb = p.lsb;
        d.lsh = p.lsh;
        d.lst = p.lst;
        d.lens = lens;
        d.out = s->per_head ? reinterpret_cast<float*>(ws + pl.dla) : dlog_alpha;
        d.tokens = (int64_t)s->B * s->H * s->T;
        d.H = s->H;
        d.T = s->T;
        d.tiles = rq.tiles;
        hipLaunchKernelGGL(gdn_lin_decay_kernel, dim3((unsigned)ceil_div(d.tokens, 256)), dim3(256), 0, hs, d);
        if (s->per_head)
            hipLaunchKernelGGL(gdn_lin_head_sum_kernel, dim3((unsigned)s->H), dim3(1024), 0, hs, d.out, dlog_alpha, s->B, s->H, s->T);
    }
    return launch_status();
}

gdn_status gdn_block_norm_fwd(const gdn_block_norm_shape* s, const void* o, const void* x, const void* gate, const float* w_post,
                              const float* scale, const float* w_pre, void* x_out, void* y, void* stream) {
    clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    if (!o || !x || !x_out) return set_error(GDN_ERR_NULL_ARG, "o, x and x_out are required");
    if (w_post && !s->post) return set_error(GDN_ERR_UNSUPPORTED, "w_post goes with the norm after the block");
    if (w_pre && !y) return set_error(GDN_ERR_NULL_ARG, "w_pre goes with y");
    st = check_aligned({{o, s->dtype}, {x, s->x_dtype}, {gate, s->dtype}, {w_post, GDN_F32}, {scale, GDN_F32}, {w_pre, GDN_F32},
                        {x_out, s->x_dtype}, {y, s->dtype}});
    if (st != GDN_OK) return st;
    if (x_out == x && ((s->T > 1 && s->x_stride_t != s->D) || (s->B > 1 && s->x_stride_b != (int64_t)s->T * s->D)))
        return set_error(GDN_ERR_UNSUPPORTED, "x_out may be x only where x is contiguous");
    BlockParams p = block_params(*s, o, x, gate, w_post, scale, w_pre);
    p.x_out = x_out;
    p.y = y;
    const bool wide = rows4(o, s->dtype, {s->D, s->o_stride_b, s->o_stride_t}) && rows4(x, s->x_dtype, {s->x_stride_b, s->x_stride_t}) &&
                      rows4(gate, s->dtype, {s->g_stride_b, s->g_stride_t}) && rows4(x_out, s->x_dtype, {}) && rows4(y, s->dtype, {});
    const BlockLaunchers run = block_launchers(*s, wide);
    run.fwd(p, block_groups(*s, false), reinterpret_cast<hipStream_t>(stream));
    return launch_status();
}

size_t gdn_block_norm_bwd_workspace_bytes(const gdn_block_norm_shape* s) {
    clear_error();
    if (validate(s) != GDN_OK) return kInvalid;
    return up256((size_t)block_groups(*s, true) * 3 * s->D * 4);
}

gdn_status gdn_block_norm_bwd(const gdn_block_norm_shape* s, const void* dx_out, const void* dy, const void* x_out, const void* o,
                              const void* gate, const float* w_post, const float* scale, const float* w_pre, void* dx, void* dO,
                              void* dgate, float* dw_post, float* dscale, float* dw_pre, void* workspace, size_t workspace_bytes,
                              void* stream) {
    clear_error();
    gdn_status st = validate(s);
    if (st != GDN_OK) return st;
    if (!x_out || !o || !dx || !dO) return set_error(GDN_ERR_NULL_ARG, "x_out, o, dx and dO are required");
    if (!dx_out && !dy) return set_error(GDN_ERR_NULL_ARG, "dx_out or dy is required");
    if ((gate != nullptr) != (dgate != nullptr)) return set_error(GDN_ERR_NULL_ARG, "dgate goes with gate");
    if ((dw_post && !w_post) || (dscale && !scale) || (dw_pre && !w_pre))
        return set_error(GDN_ERR_NULL_ARG, "a weight's gradient goes with the weight");
    if (w_post && !s->post) return set_error(GDN_ERR_UNSUPPORTED, "w_post goes with the norm after the block");
    if (w_pre && !dy) return set_error(GDN_ERR_NULL_ARG, "w_pre goes with dy");
    st = check_aligned({{dx_out, s->x_dtype}, {dy, s->dtype}, {x_out, s->x_dtype}, {o, s->dtype}, {gate, s->dtype}, {w_post, GDN_F32},
                        {scale, GDN_F32}, {w_pre, GDN_F32}, {dx, s->x_dtype}, {dO, s->dtype}, {dgate, s->dtype}, {dw_post, GDN_F32},
                        {dscale, GDN_F32}, {dw_pre, GDN_F32}});
    if (st != GDN_OK) return st;
    st = check_workspace(workspace, workspace_bytes, gdn_block_norm_bwd_workspace_bytes(s), "gdn_block_norm_bwd_workspace_bytes");
    if (st != GDN_OK) return st;
    BlockBwdParams q{};
    q.f = block_params(*s, o, x_out, gate, w_post, scale, w_pre);
    q.dx_out = dx_out;
    q.dy = dy;
    q.dx = dx;
    q.dO = dO;
    q.dg = dgate;
    q.part = static_cast<float*>(workspace);
    const bool wide = rows4(o, s->dtype, {s->D, s->o_stride_b, s->o_stride_t}) && rows4(x_out, s->x_dtype, {s->x_stride_b, s->x_stride_t}) &&
                      rows4(gate, s->dtype, {s->g_stride_b, s->g_stride_t}) && rows4(dx_out, s->x_dtype, {}) && rows4(dy, s->dtype, {}) &&
                      rows4(dx, s->x_dtype, {}) && rows4(dO, s->dtype, {}) && rows4(dgate, s->dtype, {});
    const BlockLaunchers run = block_launchers(*s, wide);
    const int64_t blocks = block_groups(*s, true);
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    run.bwd(q, blocks, hs);
    if (dw_post || dscale || dw_pre) launch_colsum(q.part, blocks, dw_post, s->D, dscale, s->D, hs, dw_pre, s->D);
    return launch_status();
}

}  // extern "C"
