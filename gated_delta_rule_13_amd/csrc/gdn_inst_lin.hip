// gdn_inst_lin.hip -- instantiations of linear attention's passes for one type
// (GDN_LIN_BF16) and size of rows (GDN_LIN_NK), and, in the object of the first
// size, of its single-token step.
#include "gdn_launch.h"
#include "gdn_lin.h"

namespace gdn {
namespace {
constexpr bool kBf = GDN_LIN_BF16 != 0;
constexpr int kNk = GDN_LIN_NK;

template <int SET>
void run(const LinParams& p, int64_t blocks, hipStream_t st) {
    hipLaunchKernelGGL((gdn_lin_kernel<kBf, kNk, SET>), dim3((unsigned)blocks), dim3(kLinThreads), 0, st, p);
}
}  // namespace

#define GDN_LIN_NAME2(bf, nk) lin_launcher_##bf##_##nk
#define GDN_LIN_NAME(bf, nk) GDN_LIN_NAME2(bf, nk)
LinLauncher GDN_LIN_NAME(GDN_LIN_BF16, GDN_LIN_NK)(int set) {
    switch (set) {
        case kLinSetFwd: return run<kLinSetFwd>;
        case kLinSetQk: return run<kLinSetQk>;
        case kLinSetV: return run<kLinSetV>;
        case kLinSetAll: return run<kLinSetAll>;
        case kLinSetKSums: return run<kLinSetKSums>;
        case kLinSetKvSums: return run<kLinSetKvSums>;
        case kLinSetQSums: return run<kLinSetQSums>;
        case kLinSetSum: return run<kLinSetSum>;
        default: return run<kLinSetSums>;
    }
}

#if GDN_LIN_NK == 32
namespace {
template <int L, int J, int V>
void step(const LinStepParams& p, int64_t bhs, hipStream_t st) {
    hipLaunchKernelGGL((gdn_lin_step_kernel<kBf, L, J, V>), dim3((unsigned)(bhs * p.blocks)), dim3(kLinStepThreads), 0, st, p);
}
}  // namespace
#if GDN_LIN_BF16
LinStepLauncher lin_step_launcher_bf16(int dk, bool wide, int* rows)
#else
LinStepLauncher lin_step_launcher_f32(int dk, bool wide, int* rows)
#endif
{
    // pieces of four over eight lanes, or number by number over sixteen
    const int lanes = wide ? 8 : 16, per = lanes * (wide ? 4 : 1), J = (dk + per - 1) / per;
    *rows = kLinStepThreads / lanes * kLinStepRows;
    if (wide) {
        switch (J) {
            case 1: return step<8, 1, 4>;
            case 2: return step<8, 2, 4>;
            case 3: return step<8, 3, 4>;
            case 4: return step<8, 4, 4>;
            case 5: case 6: return step<8, 6, 4>;
            default: return step<8, 8, 4>;
        }
    }
    return J <= 4 ? step<16, 4, 1> : J <= 8 ? step<16, 8, 1> : step<16, 16, 1>;
}
#endif

}  // namespace gdn
