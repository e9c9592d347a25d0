// The norms after a block and before the next one, with the block's gate and the residual's scale.
//
//   n = x rstd(x) wp  (wp absent: n = x),   g = gate or sigma(gate)  (absent: 1),
//   s = alpha r + g n  (stored in the residual's type),   y = s rstd(s) w,
//   rstd(v) = 1 / sqrt(mean_c v_c^2 + eps).
// The second norm is taken of s AS STORED, as in add_rmsnorm.cu.
//
// Every byte moves once: a row lives in registers (8 channels a thread and vector) through both of its
// sums, and the next rows are on their way meanwhile, in a ring in shared memory where there are many:
// two blocks of 512 threads hold 49 KB on their way in registers (16384 x 4096 in bf16 with a gate per
// token: 131 us), with a ring of 96 KB each 119, and in packed arithmetic 104 (6,450 GB/s).  Bound by HBM;
// 8192 x 2048 with an fp32 residual stream 34 us (5,920 GB/s), 57 % of the issue slots in use.
#include "norm_common.cuh"

namespace ldn {
namespace {

constexpr int kRingLeast = 1024;   // channels from which a row is worth its bulk copies

// s of 8 channels, as stored, from x g and r.  x g is exact in bf16 and the last product is not rounded:
// what rounding is left lets few sums fall to the other side of a border of the stored type.
template <typename TRes>
__device__ __forceinline__ V8 joined(const V8 &xg, const V8 &r, bool post, const V8 &wp, float rstd, float scale,
                                     const TRes *stored)
{
    return as_stored(post ? fma(xg, wp * rstd, r * scale) : fma(r, scale, xg), stored);
}
__device__ __forceinline__ float sum_of(float2 v) { return v.x + v.y; }

// A block walks rows blockIdx.x, + gridDim.x, ...  RING: they come through a ring in shared memory (rows
// of whole vectors), and a gate's row that several rows share is read where it changes; otherwise the
// next row is on its way into registers.
template <typename TIn, typename TRes, typename TG, int VPT, bool VEC, bool RING>
__global__ void __launch_bounds__(kMostThreads, VEC && VPT == 1 ? 2 : 1)
gated_kernel(const GatedNormArgs a, const RingPlan plan)
{
    constexpr bool KEEP = VPT <= 2;   // the weights stay in registers
    static_assert(KEEP || !RING, "a ring holds more than one row");
    extern __shared__ __align__(128) uint8_t ring_sm[];
    __shared__ __align__(16) Sums<1> sm[2][2];   // two a sum: the next row's pass no reader of these
    __shared__ uint64_t full[kRingMost];
    __shared__ int fail;
    const int nwarps = blockDim.x >> 5, D = a.D;
    const long long rows = a.rows;
    const unsigned shared = a.gate ? (unsigned)(a.rows / a.gate_rows) : 1u;   // rows that share a gate's
    const float inv_D = 1.f / (float)D;
    const TIn *x = (const TIn *)a.x;
    const TRes *r = (const TRes *)a.residual;
    const TG *gate = (const TG *)a.gate;
    const bool post = a.post_weight != nullptr, pre = a.weight != nullptr, own_gate = gate && shared == 1;
    RowRing<3> ring(ring_sm, full, &fail, plan);
    int at_r = 0, at_g = 0;
    if constexpr (RING) {
        ring.add<0>(x, D * sizeof(TIn));
        at_r = ring.add<1>(r, D * sizeof(TRes));
        at_g = ring.add<2>(gate, own_gate ? D * sizeof(TG) : 0);
    }
    for (int i = 0; i < 4; ++i) clear_sums<1>(sm[i >> 1][i & 1]);
    sm100::griddep_wait();   // before any memory of another kernel
    sm100::griddep_launch_dependents();
    V8 wp[KEEP ? VPT : 1], w[KEEP ? VPT : 1];
    if constexpr (KEEP)
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k);
            wp[k] = load8<VEC>(a.post_weight + c, post ? D - c : 0);
            w[k] = load8<VEC>(a.weight + c, pre ? D - c : 0);
        }
    __syncthreads();
    Raw<TIn, kE, VEC> rx[VPT];
    Raw<TRes, kE, VEC> rr[VPT];
    Raw<TG, kE, VEC> rg[VPT];
    long long held = -1;   // the gate's row in rg
    auto fetch_gate = [&](long long row) {
        if (!gate || row >= rows || (RING && own_gate)) return;
        const long long at = (unsigned)row / shared;
        if (at == held) return;
        held = at;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k);
            take8<VEC>(rg[k], gate + at * D + c, D - c);
        }
    };
    auto fetch = [&](long long row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), valid = row < rows ? D - c : 0;
            take8<VEC>(rx[k], x + row * D + c, valid);
            take8<VEC>(rr[k], r + row * D + c, valid);
        }
        fetch_gate(row);
    };
    const long long ahead = (long long)plan.stages * gridDim.x;
    if constexpr (RING) {
        if (ring.issues())
            for (int i = 0; i < plan.stages; ++i)
                if (blockIdx.x + (long long)i * gridDim.x < rows) ring.fill(i, blockIdx.x + (long long)i * gridDim.x);
    } else {
        fetch(blockIdx.x);
    }
    int turn = 0;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        if constexpr (RING) {
            fetch_gate(row);
            const uint8_t *in = ring.row();
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = place<VEC>(k);
                take8<VEC>(rx[k], (const TIn *)in + c, D - c);
                take8<VEC>(rr[k], (const TRes *)(in + at_r) + c, D - c);
                if (own_gate) take8<VEC>(rg[k], (const TG *)(in + at_g) + c, D - c);
            }
        }
        V8 v[VPT], q[VPT];
        float2 sum2 = dup(0.f);
        float rstd = 1.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            v[k] = widened(rx[k]);
            q[k] = widened(rr[k]);
            if (post) sum2 = dot(v[k], v[k], sum2);
        }
        if (gate)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                V8 g = widened(rg[k]);
                if (a.gate_sigmoid) g = sigmoid(g);
                v[k] = v[k] * g;
            }
        if constexpr (!RING && KEEP) fetch(row + gridDim.x);
        if (post) {
            float sum = sum_of(sum2);
            row_sums<1>(&sum, sm[turn][0], nwarps);
            rstd = root(fmaf(sum, inv_D, a.eps));
        } else if constexpr (RING) {
            __syncthreads();
        }
        if constexpr (RING) {   // every thread has read the stage
            if (ring.issues() && row + ahead < rows) ring.fill(ring.s, row + ahead);
            ring.step();
        }
        sum2 = dup(0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), at = KEEP ? k : 0;
            if constexpr (!KEEP) wp[0] = load8<VEC>(a.post_weight + c, post ? D - c : 0);
            v[k] = joined(v[k], q[k], post, wp[at], rstd, a.residual_scale, r);
            sum2 = dot(v[k], v[k], sum2);
            store8<VEC>((TRes *)a.residual_out + row * D + c, v[k], D - c);
        }
        if (pre) {
            float sum = sum_of(sum2);
            row_sums<1>(&sum, sm[turn][1], nwarps);
            rstd = root(fmaf(sum, inv_D, a.eps));
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = place<VEC>(k), at = KEEP ? k : 0;
                if constexpr (!KEEP) w[0] = load8<VEC>(a.weight + c, D - c);
                store8<VEC>((TIn *)a.y + row * D + c, v[k] * (w[at] * rstd), D - c);
            }
        }
        if constexpr (!RING && !KEEP) fetch(row + gridDim.x);
    }
    if constexpr (RING) ring.close(a.status);
}

// Vectors a thread: one where 512 threads hold the row (with two, and 256 threads of 116 registers,
// 16384 x 4096 took 152 us for 131).
int fwd_vpt(int D) { return D <= 4096 ? 1 : D <= 8192 ? 2 : 4; }

template <typename TIn, typename TRes, typename TG, int VPT>
cudaError_t gated_run(const GatedNormArgs &a, bool vec, cudaStream_t st)
{
    const int nt = norm_threads(a.D, VPT), per = (vec && VPT == 1 ? 1024 : 512) / nt;
    const dim3 grid((unsigned)std::min<long long>(a.rows, 152LL * per)), block(nt);
    if constexpr (VPT <= 2)
        if (vec && a.D >= kRingLeast && a.rows > 2LL * 152 * per) {
            const bool own = a.gate && a.gate_rows == a.rows;
            const RingPlan plan = ring_plan(a.D * (int)(sizeof(TIn) + sizeof(TRes) + (own ? sizeof(TG) : 0)), per);
            if (plan.stages) {
                auto *k = gated_kernel<TIn, TRes, TG, VPT, true, true>;
                // always the most: the attribute is the kernel's, shared by all host threads
                const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
                if (e != cudaSuccess) return e;
                return launch_after(k, grid, block, plan.stages * plan.stage, st, a, plan);
            }
        }
    return launch_after(vec ? gated_kernel<TIn, TRes, TG, VPT, true, false> : gated_kernel<TIn, TRes, TG, VPT, false, false>,
                        grid, block, 0, st, a, RingPlan{0, 0});
}

template <typename TIn, typename TRes, typename TG>
cudaError_t gated_pick(const GatedNormArgs &a, bool vec, cudaStream_t st)
{
    const int v = fwd_vpt(a.D);
    if (v == 1) return gated_run<TIn, TRes, TG, 1>(a, vec, st);
    if (v == 2) return gated_run<TIn, TRes, TG, 2>(a, vec, st);
    return gated_run<TIn, TRes, TG, 4>(a, vec, st);
}

}  // namespace

cudaError_t launch_gated_add_rmsnorm(const GatedNormArgs &a, cudaStream_t st)
{
    const bool vec = a.D % kE == 0 && vec16(a.x) && vec16(a.residual) && vec16(a.residual_out) && vec16(a.gate) &&
                     vec16(a.post_weight) && vec16(a.weight) && vec16(a.y);
    const bool wide_gate = a.gate_dtype == LDN_F32;
    using bf16 = __nv_bfloat16;
    if (a.dtype == LDN_F32) return gated_pick<float, float, float>(a, vec, st);
    if (a.res_dtype == LDN_F32)
        return wide_gate ? gated_pick<bf16, float, float>(a, vec, st) : gated_pick<bf16, float, bf16>(a, vec, st);
    return wide_gate ? gated_pick<bf16, bf16, float>(a, vec, st) : gated_pick<bf16, bf16, bf16>(a, vec, st);
}

}  // namespace ldn
