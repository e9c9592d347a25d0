// The norms after a block and before the next one, with the block's gate and the residual's scale.
//
//   n = x rstd(x) wp  (wp absent: n = x),   g = gate or sigma(gate)  (absent: 1),
//   s = alpha r + g n  (stored in the residual's type),   y = s rstd(s) w,
//   rstd(v) = 1 / sqrt(mean_c v_c^2 + eps).
// The second norm is taken of s AS STORED, as in add_rmsnorm.cu.
//
// Every byte moves once: a row lives in registers (8 channels a thread and vector) through both of its
// sums, and the next row's x, r and gate are on their way meanwhile.  Bound by HBM.
#include "norm_common.cuh"

namespace ldn {
namespace {

// A block walks rows blockIdx.x, + gridDim.x, ...
template <typename TIn, typename TRes, typename TG, int VPT, bool VEC>
__global__ void __launch_bounds__(kMostThreads)
gated_kernel(const GatedNormArgs a)
{
    constexpr int ST = kStep<VEC>;
    __shared__ float sm[2][2][32];
    const int nwarps = blockDim.x >> 5, D = a.D;
    const long long rows = a.rows, shared = a.gate ? a.rows / a.gate_rows : 1;   // rows that share a gate's
    const TIn *x = (const TIn *)a.x;
    const TRes *r = (const TRes *)a.residual;
    const TG *gate = (const TG *)a.gate;
    const bool post = a.post_weight != nullptr, pre = a.weight != nullptr;
    constexpr bool KEEP = VPT <= 2;   // the weights stay in registers, the next row comes ahead
    float wp[KEEP ? VPT : 1][kE], w[KEEP ? VPT : 1][kE];
    auto weights = [&](int k, int c) {
        load_n<kE, VEC, ST>(a.post_weight + c, wp[k], post ? D - c : 0);
        load_n<kE, VEC, ST>(a.weight + c, w[k], pre ? D - c : 0);
    };
    if constexpr (KEEP)
#pragma unroll
        for (int k = 0; k < VPT; ++k) weights(k, place<VEC>(k));
    Raw<TIn, kE, VEC> rx[VPT];
    Raw<TRes, kE, VEC> rr[VPT];
    Raw<TG, kE, VEC> rg[VPT];
    auto fetch_x = [&](long long row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k);
            rx[k].template load<VEC, ST>(x + row * D + c, row < rows ? D - c : 0);
        }
    };
    long long held = -1;   // the gate's row in rg
    auto fetch_rest = [&](long long row) {
        const long long at = row < rows ? row / shared : held;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), valid = row < rows ? D - c : 0;
            rr[k].template load<VEC, ST>(r + row * D + c, valid);
            if (gate && at != held) rg[k].template load<VEC, ST>(gate + at * D + c, D - c);
        }
        held = at;
    };
    fetch_x(blockIdx.x);
    fetch_rest(blockIdx.x);
    int turn = 0;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        float v[VPT][kE], sum = 0.f, rstd = 1.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            rx[k].widen(v[k]);
#pragma unroll
            for (int i = 0; i < kE; ++i) sum = fmaf(v[k][i], v[k][i], sum);
        }
        if constexpr (KEEP) fetch_x(row + gridDim.x);
        if (post) {
            block_sum<1>(&sum, sm[turn][0], nwarps);   // two buffers: the next row's sums pass no reader of these
            rstd = root(sum / (float)D + a.eps);
        }
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = place<VEC>(k), at = KEEP ? k : 0;
            if constexpr (!KEEP) load_n<kE, VEC, ST>(a.post_weight + c, wp[0], post ? D - c : 0);
            float q[kE];
            if (gate) {
                rg[k].widen(q);
#pragma unroll
                for (int i = 0; i < kE; ++i) v[k][i] *= a.gate_sigmoid ? sigmoid_fast(q[i]) : q[i];
            }
            rr[k].widen(q);
            // x g is exact in bf16, and the last product is not rounded: what is left lets few sums
            // fall to the other side of a border of the stored type
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                v[k][i] = as_stored(fmaf(v[k][i], post ? rstd * wp[at][i] : 1.f, a.residual_scale * q[i]), r);
                sum = fmaf(v[k][i], v[k][i], sum);
            }
            store_n<kE, VEC, ST>((TRes *)a.residual_out + row * D + c, v[k], D - c);
        }
        if constexpr (KEEP) fetch_rest(row + gridDim.x);
        if (pre) {
            block_sum<1>(&sum, sm[turn][1], nwarps);
            rstd = root(sum / (float)D + a.eps);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = place<VEC>(k), at = KEEP ? k : 0;
                if constexpr (!KEEP) load_n<kE, VEC, ST>(a.weight + c, w[0], D - c);
#pragma unroll
                for (int i = 0; i < kE; ++i) v[k][i] *= rstd * w[at][i];
                store_n<kE, VEC, ST>((TIn *)a.y + row * D + c, v[k], D - c);
            }
        }
        if constexpr (!KEEP) {
            fetch_x(row + gridDim.x);
            fetch_rest(row + gridDim.x);
        }
    }
}

int fwd_vpt(int D) { return D < 4096 ? 1 : D <= 8192 ? 2 : 4; }

template <typename TIn, typename TRes, typename TG, int VPT>
void gated_run(const GatedNormArgs &a, bool vec, cudaStream_t st)
{
    const int nt = norm_threads(a.D, VPT);
    const dim3 grid((unsigned)std::min<long long>(a.rows, 152LL * std::max(1, 768 / nt))), block(nt);
    if (vec) gated_kernel<TIn, TRes, TG, VPT, true><<<grid, block, 0, st>>>(a);
    else gated_kernel<TIn, TRes, TG, VPT, false><<<grid, block, 0, st>>>(a);
}

template <typename TIn, typename TRes, typename TG>
void gated_pick(const GatedNormArgs &a, bool vec, cudaStream_t st)
{
    const int v = fwd_vpt(a.D);
    if (v == 1) gated_run<TIn, TRes, TG, 1>(a, vec, st);
    else if (v == 2) gated_run<TIn, TRes, TG, 2>(a, vec, st);
    else gated_run<TIn, TRes, TG, 4>(a, vec, st);
}

}  // namespace

cudaError_t launch_gated_add_rmsnorm(const GatedNormArgs &a, cudaStream_t st)
{
    const bool vec = a.D % kE == 0 && vec16(a.x) && vec16(a.residual) && vec16(a.residual_out) && vec16(a.gate) &&
                     vec16(a.post_weight) && vec16(a.weight) && vec16(a.y);
    const bool wide_gate = a.gate_dtype == LDN_F32;
    using bf16 = __nv_bfloat16;
    if (a.dtype == LDN_F32) gated_pick<float, float, float>(a, vec, st);
    else if (a.res_dtype == LDN_F32)
        wide_gate ? gated_pick<bf16, float, float>(a, vec, st) : gated_pick<bf16, float, bf16>(a, vec, st);
    else wide_gate ? gated_pick<bf16, bf16, float>(a, vec, st) : gated_pick<bf16, bf16, bf16>(a, vec, st);
    return cudaGetLastError();
}

}  // namespace ldn
