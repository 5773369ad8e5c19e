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
template <int L>
BlockLaunchers pick(int numbers, bool wide) {
    BlockLaunchers r{};
    if (wide) {
        switch ((numbers + 3) / 4) {
            case 1: r.fwd = fwd<L, 1, 4>; r.bwd = bwd<L, 1, 4>; break;
            case 2: r.fwd = fwd<L, 2, 4>; r.bwd = bwd<L, 2, 4>; break;
            case 3: r.fwd = fwd<L, 3, 4>; r.bwd = bwd<L, 3, 4>; break;
            default: r.fwd = fwd<L, 4, 4>; r.bwd = bwd<L, 4, 4>; break;
        }
    } else {
        switch ((numbers + 3) / 4) {
            case 1: r.fwd = fwd<L, 4, 1>; r.bwd = bwd<L, 4, 1>; break;
            case 2: r.fwd = fwd<L, 8, 1>; r.bwd = bwd<L, 8, 1>; break;
            case 3: r.fwd = fwd<L, 12, 1>; r.bwd = bwd<L, 12, 1>; break;
            default: r.fwd = fwd<L, 16, 1>; r.bwd = bwd<L, 16, 1>; break;
        }
    }
    return r;
}
}  // namespace

#define GDN_BLOCK_NAME2(xb, ob) block_launchers_##xb##_##ob
#define GDN_BLOCK_NAME(xb, ob) GDN_BLOCK_NAME2(xb, ob)
BlockLaunchers GDN_BLOCK_NAME(GDN_BLOCK_XB, GDN_BLOCK_OB)(int D, bool wide) {
    // the fewest lanes that hold a row with at most sixteen numbers each (a
    // thousand lanes leave the gradient too few registers: 4096 rows of 8192, bf16
    // on an fp32 stream, take 529 us, and with 512 lanes 257; forward 68 and 78)
    switch (block_lanes(D)) {
        case 64: return pick<64>((D + 63) / 64, wide);
        case 256: return pick<256>((D + 255) / 256, wide);
        case 512: return pick<512>((D + 511) / 512, wide);
        default: return pick<1024>((D + 1023) / 1024, wide);
    }
}

}  // namespace gdn
