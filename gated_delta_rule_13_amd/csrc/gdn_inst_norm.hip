// gdn_inst_norm.hip -- instantiations of the head normalisation.
#include "gdn_colsum.h"
#include "gdn_launch.h"
#include "gdn_norm.h"

namespace gdn {
namespace {
// About four waves for each of the chip's 1024 vector units, all resident
// (measured at 4 x 4096 x 16 x 128, fp32 to bf16: 55 us; 8192 waves 60, 2048
// 58, one wave for every eight rows without the next row in flight 70).
constexpr int64_t kNormWaves = 4096;
template <bool XB, bool OB, int L, int K, int V>
void fwd(const NormParams& p, hipStream_t st) {
    const int64_t per = kNormThreads / L, bts = p.rows / p.G, most = (kNormWaves * 64 / L + p.G - 1) / p.G;
    const int64_t tokens = bts < most ? bts : most;
    hipLaunchKernelGGL((gdn_norm_fwd_kernel<XB, OB, L, K, V>), dim3((unsigned)((tokens * p.G + per - 1) / per)),
                       dim3(kNormThreads), 0, st, p, tokens);
}
template <bool XB, bool OB, int L, int K, int V>
void bwd(const NormBwdParams& q, int nblk, hipStream_t st) {
    hipLaunchKernelGGL((gdn_norm_bwd_kernel<XB, OB, L, K, V>), dim3((unsigned)nblk * q.f.G), dim3(kNormThreads), 0, st, q);
}

struct Pick {
    NormLauncher* f;
    NormBwdLauncher* b;
    int* resident;
    template <bool XB, bool OB, int L, int K, int V>
    void set() const {
        *f = fwd<XB, OB, L, K, V>;
        *b = bwd<XB, OB, L, K, V>;
        *resident = norm_resident(XB && OB, K, V);
    }
};
template <bool XB, bool OB, int L>
void pick(int K, const Pick& to) {
    switch (K) {
        case 1: return to.set<XB, OB, L, 1, 4>();
        case 2: return to.set<XB, OB, L, 2, 4>();
        case 3: return to.set<XB, OB, L, 3, 4>();
        default: return to.set<XB, OB, L, 4, 4>();
    }
}
template <bool XB, bool OB>
void pick_row(int d, bool wide, const Pick& to) {
    if (wide) {
        // the fewest lanes that cover a row with at most four pieces each
        const int pieces = d / 4;
        if (pieces <= 32) return pick<XB, OB, 8>((pieces + 7) / 8, to);
        if (pieces <= 64) return pick<XB, OB, 16>((pieces + 15) / 16, to);
        if (pieces <= 128) return pick<XB, OB, 32>((pieces + 31) / 32, to);
        if (pieces <= 256) return pick<XB, OB, 64>((pieces + 63) / 64, to);
        if (pieces <= 512) return to.set<XB, OB, 64, 8, 4>();
        return to.set<XB, OB, 256, 4, 4>();
    }
    // likewise with at most eight numbers each, while there are lanes (16
    // numbers to a lane: the gradient at 4 heads of 509 in bf16 143 us for 96)
    if (d <= 32) return to.set<XB, OB, 8, 4, 1>();
    if (d <= 64) return to.set<XB, OB, 16, 4, 1>();
    if (d <= 96) return to.set<XB, OB, 16, 6, 1>();
    if (d <= 128) return to.set<XB, OB, 16, 8, 1>();
    if (d <= 192) return to.set<XB, OB, 32, 6, 1>();
    if (d <= 256) return to.set<XB, OB, 32, 8, 1>();
    if (d <= 384) return to.set<XB, OB, 64, 6, 1>();
    if (d <= 512) return to.set<XB, OB, 64, 8, 1>();
    if (d <= 1024) return to.set<XB, OB, 256, 4, 1>();
    if (d <= 2048) return to.set<XB, OB, 256, 8, 1>();
    return to.set<XB, OB, 256, 16, 1>();
}
}  // namespace

void norm_launchers(bool x_bf16, bool o_bf16, int d, bool wide, NormLauncher* fwd, NormBwdLauncher* bwd,
                    int* resident) {
    const Pick to{fwd, bwd, resident};
    if (x_bf16) o_bf16 ? pick_row<true, true>(d, wide, to) : pick_row<true, false>(d, wide, to);
    else o_bf16 ? pick_row<false, true>(d, wide, to) : pick_row<false, false>(d, wide, to);
}

void norm_bwd_sum(const NormBwdParams& q, int nblk, float* dweight, float* dbias, hipStream_t st) {
    const NormParams& p = q.f;
    const int64_t rows = p.per_group ? nblk : (int64_t)nblk * p.G;
    const int64_t cols = p.per_group ? (int64_t)p.G * p.d : p.d;
    if (dweight || dbias) launch_colsum(q.part, rows, dweight, cols, dbias, cols, st);
}
}  // namespace gdn
