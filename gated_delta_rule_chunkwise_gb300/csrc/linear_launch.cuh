// Launch of one product, for the translation units that hold its forms.
#pragma once
#include "linear_gemm.cuh"
#include "linear_plan.h"

namespace ldn {
namespace linear {

inline int sm_count()
{
    static int n[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!n[dev]) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        n[dev] = v;
    }
    return n[dev];
}

template <int BN, bool AMN, bool BMN, bool F8, bool EPI, bool PROMOTE>
cudaError_t launch(const Operand &A, const Operand &B, const Args &a, int sms, cudaStream_t st)
{
    using S = Tile<BN>;
    CUtensorMap ma, mb;
    // one row has no distance to a next one: any multiple of 16 bytes will do
    auto ld = [](const Operand &o) { return (uint64_t)(o.rows == 1 ? (o.width + 15) / 16 * 16 : o.ld); };
    auto plane = [&](const Operand &o) { return (uint64_t)(o.planes == 1 ? ld(o) : o.plane); };
    if (!make_tmap_rows(&ma, A.p, A.width, A.rows, A.planes, ld(A), plane(A), AMN ? 64 : kLanes, F8) ||
        !make_tmap_rows(&mb, B.p, B.width, B.rows, B.planes, ld(B), plane(B), BMN ? 64 : BN, F8))
        return cudaErrorInvalidValue;
    auto *k = gemm_kernel<BN, AMN, BMN, F8, EPI, PROMOTE>;
    // always the same value: a call between another's two lines changes nothing
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    const long long tiles = ((a.ni + kLanes - 1) / kLanes) * ((a.nj + BN - 1) / BN);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.split > 1 ? tiles * a.split : std::min<long long>(tiles, sms)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, k, ma, mb, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The product with the cut that plan_for gives.
template <bool AMN, bool BMN, bool F8, bool EPI, bool PROMOTE>
cudaError_t run(const Operand &A, const Operand &B, Args a, cudaStream_t st)
{
    const int sms = sm_count();
    a.status = status_word_ptr();
    if (!sms || !a.status) return cudaErrorUnknown;
    const Plan p = plan_for(a.ni, a.nj, a.kblocks, a.npairs, BMN ? 64 : 16, sms);
    a.split = p.split;
    if (!PROMOTE) a.chunk = a.kblocks;
    if constexpr (!BMN) {
        if (p.bn == 16) return launch<16, AMN, BMN, F8, EPI, PROMOTE>(A, B, a, sms, st);
        if (p.bn == 32) return launch<32, AMN, BMN, F8, EPI, PROMOTE>(A, B, a, sms, st);
    }
    if (p.bn == 64) return launch<64, AMN, BMN, F8, EPI, PROMOTE>(A, B, a, sms, st);
    if (p.bn == 128) return launch<128, AMN, BMN, F8, EPI, PROMOTE>(A, B, a, sms, st);
    return launch<256, AMN, BMN, F8, EPI, PROMOTE>(A, B, a, sms, st);
}

// k blocks of a chunk: 512 elements of 16 bits keep the sum within 5e-7 of its norm, and with fp32's six
// pairs of planes 256.
constexpr int kChunk = 8, kChunkPlanes = 4;

// Sums that an fp32 output would show are promoted; the others are rounded to bf16's 8 bits anyway.
template <bool AMN, bool BMN, bool F8, bool EPI>
cudaError_t run(const Operand &A, const Operand &B, Args a, cudaStream_t st)
{
    a.chunk = a.npairs > 1 ? kChunkPlanes : kChunk;
    if (a.out_f32 && a.kblocks * a.npairs > a.chunk) return run<AMN, BMN, F8, EPI, true>(A, B, a, st);
    return run<AMN, BMN, F8, EPI, false>(A, B, a, st);
}

}  // namespace linear
}  // namespace ldn
