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
template <bool XB, bool OB, int L, int K>
void fwd(const NormParams& p, hipStream_t st) {
    const int64_t per = kNormThreads / L, bts = p.rows / p.G, most = (kNormWaves * (64 / L) + p.G - 1) / p.G;
    const int64_t tokens = bts < most ? bts : most;
    hipLaunchKernelGGL((gdn_norm_fwd_kernel<XB, OB, L, K>), dim3((unsigned)((tokens * p.G + per - 1) / per)),
                       dim3(kNormThreads), 0, st, p, tokens);
}
template <bool XB, bool OB>
void fwd_plain(const NormParams& p, hipStream_t st) {
    const int64_t per = kNormThreads / 64, most = 1 << 20;
    const int64_t all = (p.rows + per - 1) / per;
    hipLaunchKernelGGL((gdn_norm_fwd_plain_kernel<XB, OB>), dim3((unsigned)(all < most ? all : most)), dim3(kNormThreads),
                       0, st, p);
}
template <bool XB, bool OB, int L, int K>
void bwd(const NormBwdParams& q, int nblk, hipStream_t st) {
    hipLaunchKernelGGL((gdn_norm_bwd_kernel<XB, OB, L, K>), dim3((unsigned)nblk * q.f.G), dim3(kNormThreads), 0, st, q);
}
template <bool XB, bool OB>
void bwd_plain(const NormBwdParams& q, int nblk, hipStream_t st) {
    hipLaunchKernelGGL((gdn_norm_bwd_plain_kernel<XB, OB>), dim3((unsigned)nblk * q.f.G), dim3(64), 0, st, q);
}

template <bool XB, bool OB, int L>
void pick(int K, NormLauncher* f, NormBwdLauncher* b) {
    switch (K) {
        case 1: *f = fwd<XB, OB, L, 1>; *b = bwd<XB, OB, L, 1>; return;
        case 2: *f = fwd<XB, OB, L, 2>; *b = bwd<XB, OB, L, 2>; return;
        case 3: *f = fwd<XB, OB, L, 3>; *b = bwd<XB, OB, L, 3>; return;
        case 4: *f = fwd<XB, OB, L, 4>; *b = bwd<XB, OB, L, 4>; return;
    }
}
template <bool XB, bool OB>
void pick_row(int d, bool wide, NormLauncher* f, NormBwdLauncher* b) {
    const int pieces = d / 4;
    if (!wide || pieces > 512) {
        *f = fwd_plain<XB, OB>;
        *b = bwd_plain<XB, OB>;
        return;
    }
    if (pieces > 256) {
        *f = fwd<XB, OB, 64, 8>;
        *b = bwd<XB, OB, 64, 8>;
        return;
    }
    // the fewest lanes that cover a row with at most four pieces each
    if (pieces <= 32) pick<XB, OB, 8>((pieces + 7) / 8, f, b);
    else if (pieces <= 64) pick<XB, OB, 16>((pieces + 15) / 16, f, b);
    else if (pieces <= 128) pick<XB, OB, 32>((pieces + 31) / 32, f, b);
    else pick<XB, OB, 64>((pieces + 63) / 64, f, b);
}
}  // namespace

void norm_launchers(bool x_bf16, bool o_bf16, int d, bool wide, NormLauncher* fwd, NormBwdLauncher* bwd) {
    if (x_bf16) o_bf16 ? pick_row<true, true>(d, wide, fwd, bwd) : pick_row<true, false>(d, wide, fwd, bwd);
    else o_bf16 ? pick_row<false, true>(d, wide, fwd, bwd) : pick_row<false, false>(d, wide, fwd, bwd);
}

void norm_bwd_sum(const NormBwdParams& q, int nblk, float* dweight, float* dbias, hipStream_t st) {
    const NormParams& p = q.f;
    const int64_t rows = p.per_group ? nblk : (int64_t)nblk * p.G;
    const int64_t cols = p.per_group ? (int64_t)p.G * p.d : p.d;
    if (dweight || dbias) launch_colsum(q.part, rows, dweight, cols, dbias, cols, st);
}
}  // namespace gdn
