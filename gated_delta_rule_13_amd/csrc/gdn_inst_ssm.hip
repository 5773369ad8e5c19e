// gdn_inst_ssm.hip -- instantiations of the selective state space recurrence
// and its order of launches.  GDN_SSM_BF16 (0 or 1) picks the dtype.
#include "gdn_launch.h"
#include "gdn_ssm.h"

#if !defined(GDN_SSM_BF16)
#error "build with -DGDN_SSM_BF16=0 or 1"
#endif

namespace gdn {
namespace {
constexpr bool kBF = GDN_SSM_BF16 != 0;

unsigned blocks(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

template <int NS, bool GRAD>
void summaries(const SsmParams& p, int nseg_summed, hipStream_t st) {
    const int64_t tiles = (int64_t)p.G * p.tpg;
    if (nseg_summed > 0)
        hipLaunchKernelGGL((gdn_ssm_sum_kernel<kBF, NS, GRAD>), dim3((unsigned)(p.B * nseg_summed * tiles)), dim3(64), 0,
                           st, p, nseg_summed);
    hipLaunchKernelGGL((gdn_ssm_chain_kernel<NS, GRAD>), dim3((unsigned)((GRAD ? 2 : 1) * p.B * tiles * NS)),
                       dim3(kChainThreads), 0, st, p);
}

template <int NS>
void fwd(const SsmParams& p, hipStream_t st) {
    const int64_t tiles = (int64_t)p.G * p.tpg;
    if (p.nseg > 1) summaries<NS, false>(p, p.nseg - 1, st);
    const dim3 grid((unsigned)(p.B * p.nseg * tiles));
    if (p.N == NS) hipLaunchKernelGGL((gdn_ssm_fwd_kernel<kBF, NS, false>), grid, dim3(64), 0, st, p);
    else hipLaunchKernelGGL((gdn_ssm_fwd_kernel<kBF, NS, true>), grid, dim3(64), 0, st, p);
}

template <int NS, int NB>
void bwd(const SsmParams& p, float* dA, void* dBm, void* dC, float* dD, float* dbias, hipStream_t st) {
    constexpr int NSA = NS * NB;
    const int64_t tiles = (int64_t)p.G * p.tpg;
    summaries<NSA, true>(p, p.nseg, st);
    const dim3 grid((unsigned)(p.B * p.nseg * tiles));
    if (p.N == NSA && p.Dg % 64 == 0) hipLaunchKernelGGL((gdn_ssm_bwd_kernel<kBF, NS, NB, false>), grid, dim3(64 * NB), 0, st, p);
    else hipLaunchKernelGGL((gdn_ssm_bwd_kernel<kBF, NS, NB, true>), grid, dim3(64 * NB), 0, st, p);
    SsmSumParams q{p, dBm, dC, dA, dD, dbias, NSA, blocks((int64_t)p.B * p.T * p.G * 2 * NSA, kSumThreads)};
    hipLaunchKernelGGL((gdn_ssm_grad_sum_kernel<kBF>), dim3(q.bc + (unsigned)(tiles * (NSA + 2))), dim3(kSumThreads), 0, st,
                       q);
}

template <int LP>
void step(const SsmStepParams& q, hipStream_t st) {
    hipLaunchKernelGGL((gdn_ssm_step_kernel<kBF, LP>), dim3(blocks((int64_t)q.f.D * LP, kStepThreads), (unsigned)q.f.B),
                       dim3(kStepThreads), 0, st, q);
}
}  // namespace

#if GDN_SSM_BF16
#define GDN_SSM_NAME(name) name##_bf16
#else
#define GDN_SSM_NAME(name) name##_f32
#endif

void GDN_SSM_NAME(ssm_fwd_run)(const SsmParams& p, hipStream_t st) {
    switch (ssm_states(p.N)) {
        case 4: return fwd<4>(p, st);
        case 8: return fwd<8>(p, st);
        case 16: return fwd<16>(p, st);
        case 32: return fwd<32>(p, st);
        default: return fwd<64>(p, st);
    }
}
void GDN_SSM_NAME(ssm_bwd_run)(const SsmParams& p, float* dA, void* dBm, void* dC, float* dD, float* dbias, hipStream_t st) {
    switch (ssm_states(p.N)) {
        case 4: return bwd<4, 1>(p, dA, dBm, dC, dD, dbias, st);
        case 8: return bwd<4, 2>(p, dA, dBm, dC, dD, dbias, st);
        case 16: return bwd<4, 4>(p, dA, dBm, dC, dD, dbias, st);
        case 32: return bwd<8, 4>(p, dA, dBm, dC, dD, dbias, st);
        default: return bwd<8, 8>(p, dA, dBm, dC, dD, dbias, st);
    }
}
void GDN_SSM_NAME(ssm_step_run)(const SsmStepParams& q, hipStream_t st) {
    switch (ssm_states(q.f.N)) {
        case 4: return step<1>(q, st);
        case 8: return step<2>(q, st);
        case 16: return step<4>(q, st);
        case 32: return step<8>(q, st);
        default: return step<16>(q, st);
    }
}

#if GDN_SSM_BF16
int ssm_states(int N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
void ssm_fwd_run_f32(const SsmParams& p, hipStream_t st);
void ssm_bwd_run_f32(const SsmParams& p, float* dA, void* dBm, void* dC, float* dD, float* dbias, hipStream_t st);
void ssm_step_run_f32(const SsmStepParams& q, hipStream_t st);
void ssm_fwd_run(const SsmParams& p, bool bf, hipStream_t st) { bf ? ssm_fwd_run_bf16(p, st) : ssm_fwd_run_f32(p, st); }
void ssm_bwd_run(const SsmParams& p, bool bf, float* dA, void* dBm, void* dC, float* dD, float* dbias, hipStream_t st) {
    bf ? ssm_bwd_run_bf16(p, dA, dBm, dC, dD, dbias, st) : ssm_bwd_run_f32(p, dA, dBm, dC, dD, dbias, st);
}
void ssm_step_run(const SsmStepParams& q, bool bf, hipStream_t st) {
    bf ? ssm_step_run_bf16(q, st) : ssm_step_run_f32(q, st);
}
#endif
}  // namespace gdn
