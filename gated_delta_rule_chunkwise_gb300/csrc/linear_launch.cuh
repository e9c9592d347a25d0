// Launch of one product, for the translation units that hold its forms.
#pragma once
#include "linear_gemm.cuh"

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

template <bool AMN, bool BMN, bool F8, bool EPI, bool PROMOTE, bool PAIR>
cudaError_t launch(const Operand &A, const Operand &B, Args a, int sms, cudaStream_t st)
{
    // rows of whole 16-byte vectors; fp32 z leaves by the lanes, and so do bf16 results of promoted sums
    const long long row = a.ni * (a.out_f32 ? 4 : 2);
    auto vectors = [row](const void *p) { return ((uintptr_t)p & 15) == 0 && row % 16 == 0; };   // or null
    a.staged = a.split == 1 && vectors(a.out) && vectors(a.residual) &&
               (a.out_f32 ? !a.z : !PROMOTE && a.bn % 32 == 0 && !(a.z && a.residual) && vectors(a.z));
    const int cols = PAIR ? a.bn / 2 : a.bn, stage = stage_bytes(cols),
              beside = a.staged ? kStaging : part_bytes(a.bn, a.split);
    a.stages = std::min(kMostStages, (kStageBytes - beside) / stage);
    CUtensorMap ma, mb, mo, mz, mr;
    // one row has no distance to a next one: any multiple of 16 bytes will do
    auto ld = [](const Operand &o) { return (uint64_t)(o.rows == 1 ? (o.width + 15) / 16 * 16 : o.ld); };
    auto plane = [&](const Operand &o) { return (uint64_t)(o.planes == 1 ? ld(o) : o.plane); };
    if (!make_tmap_rows(&ma, A.p, A.width, A.rows, A.planes, ld(A), plane(A), AMN ? 64 : kLanes, F8) ||
        !make_tmap_rows(&mb, B.p, B.width, B.rows, B.planes, ld(B), plane(B), BMN ? 64 : cols, F8))
        return cudaErrorInvalidValue;
    mo = mz = mr = ma;   // where they are not used
    auto result = [&](CUtensorMap *m, const void *p) {
        return !p || (a.out_f32 ? make_tmap_f32(m, p, a.ni, a.nj, 16) : make_tmap_rows(m, p, a.ni, a.nj, 1, a.ni, a.ni, 32, false));
    };
    if (a.staged && (!result(&mo, a.out) || !result(&mz, a.z) || !result(&mr, a.residual))) return cudaErrorInvalidValue;
    auto *k = gemm_kernel<AMN, BMN, F8, EPI, PROMOTE, PAIR>;
    // always the most: a call between another's two lines changes nothing
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes + 1024);
    if (e != cudaSuccess) return e;
    constexpr int kTileLanes = PAIR ? 2 * kLanes : kLanes;
    const long long tiles = ((a.ni + kTileLanes - 1) / kTileLanes) * ((a.nj + a.bn - 1) / a.bn);
    const int blocks = PAIR ? 2 : a.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * (a.split > 1 ? tiles : std::min<long long>(tiles, sms / blocks))));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = a.stages * stage + beside + 1024;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // as launch_after
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, k, ma, mb, mo, mz, mr, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The product with the cut that plan_for gives.
template <bool AMN, bool BMN, bool F8, bool EPI, bool PROMOTE>
cudaError_t run(const Operand &A, const Operand &B, Args a, cudaStream_t st)
{
    const int sms = sm_count();
    a.status = status_word_ptr();
    if (!sms || !a.status) return cudaErrorUnknown;
    const Plan p = plan_for(a.ni, a.nj, a.kblocks, a.npairs, BMN, PROMOTE, sms);
    a.bn = p.bn;
    a.split = p.split;
    if (!PROMOTE) a.chunk = a.kblocks;
    if (p.pair) return launch<AMN, BMN, F8, EPI, PROMOTE, true>(A, B, a, sms, st);
    return launch<AMN, BMN, F8, EPI, PROMOTE, false>(A, B, a, sms, st);
}

// k blocks of a chunk, each four additions in tensor memory: of 16 products in 16 bits, of 32 in 8.  64 additions, 1024
// elements of 16 bits or 2048 of e4m3, keep a sum within 1.0e-6 of its norm (8.3e-7 where its products have one sign;
// of e4m3, whose products have few digits, 1.2e-7), and while a tile's results leave, the next one's products
// run two chunks ahead and no further (8192 x 4096 to 4096 onto an fp32 stream: 182 us, 204 with half as many).  With
// fp32's six pairs of planes 96 additions, of which the largest pair's are 16: 2.4e-7.
constexpr int kChunk = 16, kChunkPlanes = 4;
// For bf16 results, which are rounded by up to 3.9e-3: sums of one sign over 65536 elements of 16 bits come out 3.7e-4
// too small, and so do longer ones (over a million tokens 6.6e-3 without this, in 3640 us for 3620).
constexpr int kChunkRounded = 1024;

// Sums of more than one chunk are promoted.
template <bool AMN, bool BMN, bool F8, bool EPI>
cudaError_t run(const Operand &A, const Operand &B, Args a, cudaStream_t st)
{
    a.chunk = !a.out_f32 ? kChunkRounded : a.npairs > 1 ? kChunkPlanes : kChunk;
    if ((long long)a.kblocks * a.npairs > a.chunk) return run<AMN, BMN, F8, EPI, true>(A, B, a, st);
    return run<AMN, BMN, F8, EPI, false>(A, B, a, st);
}

}  // namespace linear
}  // namespace ldn
