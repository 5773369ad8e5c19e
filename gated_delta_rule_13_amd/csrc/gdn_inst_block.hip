// gdn_inst_block.hip -- instantiations of the norms around a block for one type
// of the stream (GDN_BLOCK_XB) and of the block (GDN_BLOCK_OB).
#include "gdn_block.h"
#include "gdn_launch.h"

namespace gdn {
namespace {
constexpr bool kXb = GDN_BLOCK_XB != 0, kOb = GDN_BLOCK_OB != 0;

template <int L, int K, int V>
void fwd(const BlockParams& p, int64_t blocks, hipStream_t st) {
    hipLaunchKernelGGL((gdn_block_fwd_kernel<kXb, kOb, L, K, V>), dim3((unsigned)blocks), dim3(block_threads<L>()), 0, st, p);
}
template <int L, int K, int V>
void bwd(const BlockBwdParams& q, int64_t blocks, hipStream_t st) {
    hipLaunchKernelGGL((gdn_block_bwd_kernel<kXb, kOb, L, K, V>), dim3((unsigned)blocks), dim3(block_threads<L>()), 0, st, q);
}
// Q: fours of numbers to a lane
template <int L, int Q>
BlockLaunchers fours(bool wide) {
    return wide ? BlockLaunchers{fwd<L, Q, 4>, bwd<L, Q, 4>} : BlockLaunchers{fwd<L, 4 * Q, 1>, bwd<L, 4 * Q, 1>};
}
// (rows that fewer lanes hold are theirs)
template <int L>
BlockLaunchers pick(int D, bool wide) {
    const int q = ((D + L - 1) / L + 3) / 4;
    if constexpr (L == 64) {
        if (q <= 1) return fours<L, 1>(wide);
    }
    if constexpr (L <= 256) {
        if (q <= 2) return fours<L, 2>(wide);
    }
    return q <= 3 ? fours<L, 3>(wide) : fours<L, 4>(wide);
}
}  // namespace

#define GDN_BLOCK_NAME2(xb, ob) block_launchers_##xb##_##ob
#define GDN_BLOCK_NAME(xb, ob) GDN_BLOCK_NAME2(xb, ob)
BlockLaunchers GDN_BLOCK_NAME(GDN_BLOCK_XB, GDN_BLOCK_OB)(int D, bool wide) {
    // the fewest lanes that hold a row with at most sixteen numbers each (a
    // thousand lanes leave the gradient too few registers: 4096 rows of 8192, bf16
    // on an fp32 stream, gated, take 532 us, and with 512 lanes 255; forward 91 and
    // 94)
    switch (block_lanes(D)) {
        case 64: return pick<64>(D, wide);
        case 256: return pick<256>(D, wide);
        case 512: return pick<512>(D, wide);
        default: return pick<1024>(D, wide);
    }
}

}  // namespace gdn
