// Gradient of gated_add_rmsnorm.cu, with rho the reciprocal roots and n, g as there:
//
//   dS = dsum + rho_s (w dy - s rho_s^2 mean_c(w dy s)),     dw = sum over rows of dy s rho_s,
//   dr = alpha dS,   dgate = dS n (times g (1 - g) behind a sigmoid), summed over the rows that share it,
//   dn = dS g,       dx = rho_x (wp dn - x rho_x^2 mean_c(wp dn x)),   dwp = sum over rows of dn x rho_x.
//
// Both roots and the first mean are one round of block sums, the second mean another.  The columns'
// sums stay on chip over all rows that a block walks and are joined by a second launch in a fixed
// order.  A block walks runs of rows that share a gate's row, so that the gate's sum is a column's too.
// Bound by HBM.
#include "norm_common.cuh"

namespace ldn {
namespace {

// How the rows are walked: `groups` of them, each cut into `cuts` runs; block b takes runs b, b + blocks, ...
struct Walk {
    int blocks, summed;   // summed: the gate's gradient is a sum over each group
    long long groups, cuts;
};

int bwd_vpt(int D) { return D <= 4096 ? 1 : D <= 8192 ? 2 : 4; }

Walk walk_of(long long rows, int D, long long gate_rows, bool dgate)
{
    if (rows == 0) return {0, dgate, gate_rows, 0};   // sums of nothing
    const int per = std::max(1, kMostThreads / norm_threads(D, bwd_vpt(D)));
    const long long most = std::min<long long>(rows, 152LL * per);
    Walk w{(int)most, dgate && gate_rows < rows, 1, most};
    if (w.summed) {
        w.groups = gate_rows;
        w.cuts = std::max(1LL, std::min(most / gate_rows, rows / gate_rows));
        w.blocks = (int)std::min(most, w.groups * w.cuts);
    }
    return w;
}

template <typename TIn, typename TRes, typename TG, int VPT, bool VEC>
__global__ void __launch_bounds__(kMostThreads)
gated_bwd_kernel(const GatedNormBwdArgs a, const Walk walk)
{
    constexpr int ST = kStep<VEC>;
    // one vector a thread: its weights and its columns' sums in registers, the next row on its way;
    // more: the sums in shared memory, each its thread's own
    constexpr bool ONE = VPT == 1;
    extern __shared__ float acc_sm[];
    __shared__ float sm[2][4 * 32];
    const int D = a.D, nt = blockDim.x, nwarps = nt >> 5;
    const TIn *x = (const TIn *)a.x, *dy = (const TIn *)a.dy;
    const TRes *s = (const TRes *)a.s, *dsum = (const TRes *)a.dsum;
    const TG *gate = (const TG *)a.gate;
    const bool post = a.post_weight != nullptr, pre = a.weight != nullptr, wants_gate = a.dgate != nullptr;
    const long long per = a.rows / walk.groups, shared = gate ? a.rows / a.gate_rows : 1;

    // the columns' sums: dweight, dpost_weight, dgate
    float acc[ONE ? 3 : 1][kE];
    auto add = [&](int which, int k, int i, float v) {
        if constexpr (ONE) acc[which][i] += v;
        else acc_sm[((which * VPT + k) * kE + i) * nt + threadIdx.x] += v;
    };
    auto sum_of = [&](int which, int k, float *v) {
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            if constexpr (ONE) v[i] = acc[which][i];
            else v[i] = acc_sm[((which * VPT + k) * kE + i) * nt + threadIdx.x];
        }
    };
    auto clear = [&](int which) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                if constexpr (ONE) acc[which][i] = 0.f;
                else acc_sm[((which * VPT + k) * kE + i) * nt + threadIdx.x] = 0.f;
            }
    };
    clear(0);
    clear(1);

    float w[ONE ? VPT : 1][kE], wp[ONE ? VPT : 1][kE];
    auto weights = [&](int k) {
        const int c = place<VEC>(k);
        load_n<kE, VEC, ST>(a.weight + c, w[ONE ? k : 0], pre ? D - c : 0);
        load_n<kE, VEC, ST>(a.post_weight + c, wp[ONE ? k : 0], post ? D - c : 0);
    };
    if constexpr (ONE) weights(0);

    Raw<TRes, kE, VEC> rs[VPT], rd[VPT];
    Raw<TIn, kE, VEC> ry[VPT], rx[VPT];
    Raw<TG, kE, VEC> rg[VPT];
    auto fetch = [&](int k, long long row) {   // row < 0: none
        const int c = place<VEC>(k), valid = row >= 0 ? D - c : 0;
        rs[k].template load<VEC, ST>(s + row * D + c, pre ? valid : 0);
        ry[k].template load<VEC, ST>(dy + row * D + c, pre ? valid : 0);
        rx[k].template load<VEC, ST>(x + row * D + c, valid);
        rd[k].template load<VEC, ST>(dsum + row * D + c, dsum ? valid : 0);
        rg[k].template load<VEC, ST>(gate + row / shared * D + c, gate ? valid : 0);
    };

    const long long runs = walk.groups * walk.cuts;
    long long run = blockIdx.x, row = 0, end = 0;
    auto open = [&]() {   // the run's rows
        const long long g = run / walk.cuts, q = run - g * walk.cuts;
        row = g * per + per * q / walk.cuts;
        end = g * per + per * (q + 1) / walk.cuts;
    };
    open();
    if constexpr (ONE) fetch(0, row);
    int turn = 0;
    while (run < runs) {
        if (walk.summed) clear(2);
        for (; row < end; ++row, turn ^= 1) {
            if constexpr (!ONE)
#pragma unroll
                for (int k = 0; k < VPT; ++k) fetch(k, row);
            float sums[3] = {0.f, 0.f, 0.f}, d[VPT][kE], xv[VPT][kE], sv[VPT][kE], gy[VPT][kE], gv[VPT][kE];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if constexpr (!ONE) weights(k);
                rs[k].widen(sv[k]);
                ry[k].widen(gy[k]);
                rx[k].widen(xv[k]);
                rd[k].widen(d[k]);
                rg[k].widen(gv[k]);
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    sums[0] = fmaf(sv[k][i], sv[k][i], sums[0]);
                    sums[1] = fmaf(w[ONE ? k : 0][i] * gy[k][i], sv[k][i], sums[1]);
                    sums[2] = fmaf(xv[k][i], xv[k][i], sums[2]);
                    if (!gate) gv[k][i] = 1.f;
                    else if (a.gate_sigmoid) gv[k][i] = sigmoid_fast(gv[k][i]);
                }
            }
            if constexpr (ONE) {
                long long next = row + 1;
                if (next == end) {   // the first row of this block's next run
                    const long long u = run + gridDim.x, g = u / walk.cuts, q = u - g * walk.cuts;
                    next = u < runs ? g * per + per * q / walk.cuts : -1;
                }
                fetch(0, next);
            }
            block_sum<3>(sums, sm[turn], nwarps);   // two buffers: the next row's sums pass no reader of these
            const float rho_s = root(sums[0] / (float)D + a.eps), m_s = rho_s * rho_s * (sums[1] / (float)D);
            const float rho_x = post ? root(sums[2] / (float)D + a.eps) : 1.f;
            float dot = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = place<VEC>(k), at = ONE ? k : 0;
                if constexpr (!ONE) weights(k);
                float out[kE];
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    if (pre) {
                        add(0, k, i, gy[k][i] * (sv[k][i] * rho_s));
                        d[k][i] = fmaf(rho_s, w[at][i] * gy[k][i] - sv[k][i] * m_s, d[k][i]);
                    }
                    out[i] = a.residual_scale * d[k][i];
                }
                if (a.dresidual) store_n<kE, VEC, ST>((TRes *)a.dresidual + row * D + c, out, D - c);
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    const float xh = xv[k][i] * rho_x, n = post ? xh * wp[at][i] : xh;
                    if (wants_gate) {
                        const float dg = d[k][i] * n;
                        if (walk.summed) add(2, k, i, dg);
                        else out[i] = a.gate_sigmoid ? dg * (gv[k][i] * (1.f - gv[k][i])) : dg;
                    }
                    d[k][i] *= gv[k][i];
                    if (post) {
                        add(1, k, i, d[k][i] * xh);
                        d[k][i] *= wp[at][i];
                        dot = fmaf(d[k][i], xv[k][i], dot);
                    }
                }
                if (wants_gate && !walk.summed) store_n<kE, VEC, ST>((TG *)a.dgate + row * D + c, out, D - c);
            }
            float m_x = 0.f;
            if (post) {
                block_sum<1>(&dot, sm[turn] + 96, nwarps);
                m_x = rho_x * rho_x * (dot / (float)D);
            }
            if (a.dx)
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int c = place<VEC>(k);
#pragma unroll
                    for (int i = 0; i < kE; ++i) d[k][i] = rho_x * (d[k][i] - xv[k][i] * m_x);
                    store_n<kE, VEC, ST>((TIn *)a.dx + row * D + c, d[k], D - c);
                }
        }
        if (walk.summed)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float v[kE];
                sum_of(2, k, v);
                const int c = place<VEC>(k);
                store_n<kE, VEC, ST>(a.part_gate + run * D + c, v, D - c);
            }
        run += gridDim.x;
        if (run < runs) open();
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        float v[kE];
        const int c = place<VEC>(k);
        if (pre) {
            sum_of(0, k, v);
            store_n<kE, VEC, ST>(a.part + (size_t)blockIdx.x * D + c, v, D - c);
        }
        if (post) {
            sum_of(1, k, v);
            store_n<kE, VEC, ST>(a.part_post + (size_t)blockIdx.x * D + c, v, D - c);
        }
    }
}

// blockIdx.y 0: dweight, 1: dpost_weight, from every block's share; 2 + g: the gate's row g from its
// runs'.  32 columns a block, kSumRows rows at a time.
constexpr int kSumRows = 32;
template <typename TG>
__global__ void __launch_bounds__(32 * kSumRows)
gated_sum_kernel(const GatedNormBwdArgs a, const Walk walk)
{
    __shared__ float sm[kSumRows][33];
    const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y, D = a.D;
    const long long which = blockIdx.y;
    for (long long u = which; u < 2 + (walk.summed ? walk.groups : 0); u += gridDim.y) {
        if ((u == 0 && !a.weight) || (u == 1 && !a.post_weight)) continue;
        const float *part = u == 0 ? a.part : u == 1 ? a.part_post : a.part_gate + (u - 2) * walk.cuts * D;
        const int n = u < 2 ? walk.blocks : (int)walk.cuts;
        float t = 0.f;
        if (c < D)
#pragma unroll 8
            for (int i = y; i < n; i += kSumRows) t += part[(size_t)i * D + c];
        sm[y][threadIdx.x] = t;
        __syncthreads();
        if (y == 0 && c < D) {
#pragma unroll
            for (int i = 1; i < kSumRows; ++i) t += sm[i][threadIdx.x];
            if (u == 0) a.dweight[c] = t;
            else if (u == 1) a.dpost_weight[c] = t;
            else {
                const long long at = (u - 2) * D + c;
                if (a.gate_sigmoid) {
                    const float g = sigmoid_fast((float)((const TG *)a.gate)[at]);
                    t *= g * (1.f - g);
                }
                store_n<1, false>((TG *)a.dgate + at, &t, 1);
            }
        }
        __syncthreads();
    }
}

template <typename TIn, typename TRes, typename TG, int VPT, bool VEC>
cudaError_t bwd_run(const GatedNormBwdArgs &a, const Walk &walk, cudaStream_t st)
{
    const int nt = norm_threads(a.D, VPT);
    auto *k = gated_bwd_kernel<TIn, TRes, TG, VPT, VEC>;
    size_t smem = 0;
    if constexpr (VPT > 1) {
        // always the most: the attribute is the kernel's, shared by all host threads
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   3 * VPT * kE * kMostThreads * (int)sizeof(float));
        if (e != cudaSuccess) return e;
        smem = (size_t)3 * VPT * kE * nt * sizeof(float);
    }
    k<<<walk.blocks, nt, smem, st>>>(a, walk);
    return cudaGetLastError();
}

template <typename TIn, typename TRes, typename TG>
cudaError_t bwd_pick(GatedNormBwdArgs a, const Walk &walk, bool vec, cudaStream_t st)
{
    const int v = bwd_vpt(a.D);
    cudaError_t e = cudaSuccess;
    if (a.rows) {
        if (v == 1) e = vec ? bwd_run<TIn, TRes, TG, 1, true>(a, walk, st) : bwd_run<TIn, TRes, TG, 1, false>(a, walk, st);
        else if (v == 2)
            e = vec ? bwd_run<TIn, TRes, TG, 2, true>(a, walk, st) : bwd_run<TIn, TRes, TG, 2, false>(a, walk, st);
        else e = vec ? bwd_run<TIn, TRes, TG, 4, true>(a, walk, st) : bwd_run<TIn, TRes, TG, 4, false>(a, walk, st);
        if (e != cudaSuccess) return e;
    }
    const long long sums = 2 + (walk.summed ? walk.groups : 0);
    gated_sum_kernel<TG><<<dim3((a.D + 31) / 32, (unsigned)std::min<long long>(sums, 65535)), dim3(32, kSumRows), 0, st>>>(
        a, walk);
    return cudaGetLastError();
}

}  // namespace

size_t gated_add_rmsnorm_bwd_floats(long long rows, int D, long long gate_rows)
{
    const Walk w = walk_of(rows, D, gate_rows ? gate_rows : rows, true);
    return ((size_t)2 * w.blocks + (w.summed ? (size_t)(w.groups * w.cuts) : 0)) * D;
}

cudaError_t launch_gated_add_rmsnorm_bwd(const GatedNormBwdArgs &given, cudaStream_t st)
{
    GatedNormBwdArgs a = given;
    const Walk walk = walk_of(a.rows, a.D, a.gate ? a.gate_rows : a.rows, a.dgate != nullptr);
    a.part_post = a.part + (size_t)walk.blocks * a.D;
    a.part_gate = a.part_post + (size_t)walk.blocks * a.D;
    const bool vec = a.D % kE == 0 && vec16(a.x) && vec16(a.dy) && vec16(a.s) && vec16(a.dsum) && vec16(a.gate) &&
                     vec16(a.post_weight) && vec16(a.weight) && vec16(a.dx) && vec16(a.dresidual) && vec16(a.dgate);
    const bool wide_gate = a.gate_dtype == LDN_F32;
    using bf16 = __nv_bfloat16;
    if (a.dtype == LDN_F32) return bwd_pick<float, float, float>(a, walk, vec, st);
    if (a.res_dtype == LDN_F32)
        return wide_gate ? bwd_pick<bf16, float, float>(a, walk, vec, st) : bwd_pick<bf16, float, bf16>(a, walk, vec, st);
    return wide_gate ? bwd_pick<bf16, bf16, float>(a, walk, vec, st) : bwd_pick<bf16, bf16, bf16>(a, walk, vec, st);
}

}  // namespace ldn
