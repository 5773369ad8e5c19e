// gdn_inst_conv.hip -- instantiations of the short convolution.
#include "gdn_colsum.h"
#include "gdn_conv.h"
#include "gdn_launch.h"

namespace gdn {
namespace {
template <bool BF, int W, int V>
void fwd(const ConvParams& p, hipStream_t st) {
    const int64_t threads = (int64_t)p.B * p.ntile * p.nv;
    hipLaunchKernelGGL((gdn_conv_fwd_kernel<BF, W, V>), dim3((unsigned)((threads + kConvThreads - 1) / kConvThreads)),
                       dim3(kConvThreads), 0, st, p);
}
template <bool BF, int W, int V>
void bwd(const ConvBwdParams& q, hipStream_t st) {
    const int64_t ncb = (q.f.nv + 63) / 64;
    const int64_t rows = ((int64_t)q.f.B * q.f.ntile + kConvBwdTiles - 1) / kConvBwdTiles;
    hipLaunchKernelGGL((gdn_conv_bwd_kernel<BF, W, V>), dim3((unsigned)(ncb * rows)), dim3(kConvThreads), 0, st, q);
}
}  // namespace

#define GDN_CONV_PICK(FN, VB, VF)                                                                                  \
    switch (W) {                                                                                                   \
        case 2: return bf ? (wide ? FN<true, 2, VB> : FN<true, 2, 1>) : (wide ? FN<false, 2, VF> : FN<false, 2, 1>); \
        case 3: return bf ? (wide ? FN<true, 3, VB> : FN<true, 3, 1>) : (wide ? FN<false, 3, VF> : FN<false, 3, 1>); \
        case 4: return bf ? (wide ? FN<true, 4, VB> : FN<true, 4, 1>) : (wide ? FN<false, 4, VF> : FN<false, 4, 1>); \
    }                                                                                                              \
    return nullptr;

ConvLauncher conv_launcher(bool bf, int W, bool wide) { GDN_CONV_PICK(fwd, 8, 4) }
ConvBwdLauncher conv_bwd_launcher(bool bf, int W, bool wide) { GDN_CONV_PICK(bwd, kConvBwdV, kConvBwdV) }
#undef GDN_CONV_PICK

int64_t conv_bwd_part_rows(int64_t row_tiles) { return (row_tiles + kConvBwdTiles - 1) / kConvBwdTiles; }
void conv_bwd_sum(const float* part, int64_t rows, int D, int W, float* dweight, float* dbias, hipStream_t st) {
    launch_colsum(part, rows, dweight, (int64_t)D * W, dbias, D, st);
}
}  // namespace gdn
