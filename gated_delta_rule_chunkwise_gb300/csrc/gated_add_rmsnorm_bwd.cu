// Gradient of gated_add_rmsnorm.cu, with rho the reciprocal roots and n, g as there:
//
//   dS = dsum + rho_s (w dy - s rho_s^2 mean_c(w dy s)),     dw = sum over rows of dy s rho_s,
//   dr = alpha dS,   dgate = dS n (times g (1 - g) behind a sigmoid), summed over the rows that share it,
//   dn = dS g,       dx = rho_x (wp dn - x rho_x^2 mean_c(wp dn x)),   dwp = sum over rows of dn x rho_x.
//
// Both roots and the first mean are one round of block sums, the second mean another.  The columns'
// sums stay on chip over all rows that a block walks and are joined by a second launch in a fixed
// order.  A block walks runs of rows that share a gate's row, so that the gate's sum is a column's too.
// A row costs its latencies, of two rounds of sums and of the work between, with as few warps as the registers
// leave (three columns' sums, two weights, a row's five arrays): behind a ring a thread has two vectors and twice
// the registers, so that half the warps do as much between the sums.  8192 x 2048 in bf16 with an fp32 residual
// stream and a gate per sequence: 56 us (5,370 GB/s; 71 with one vector a thread, 64 with one thread to issue
// the copies and 64-bit rows), fp32 8192 x 4096 131 (6,140 GB/s; 255 with one vector).  One round of six sums in
// place of two took 65 for 64.  Single elements, where rows are no whole vectors: 3333 x 777 in fp32 25 us,
// bound by issue.
#include "norm_common.cuh"

namespace ldn {
namespace {

// How the rows are walked: `groups` of them, each cut into `cuts` runs; block b takes runs b, b + blocks, ...
// A group's run q has base rows, the first `extra` runs one more.
struct Walk {
    int blocks, summed;   // summed: the gate's gradient is a sum over each group
    unsigned groups, cuts, per, base, extra;
    // Rows of D floats in the workspace: two columns' sums of every block, and the gate's of every run.
    size_t shares() const { return (size_t)2 * blocks + (summed ? (size_t)groups * cuts : 0); }
};

constexpr int kRingLeast = 1024;    // channels from which a row is worth its bulk copies
constexpr int kRingThreads = 256;   // of two vectors each: they have the registers of 512 of one
int bwd_vpt(int D) { return D <= 4096 ? 1 : D <= 8192 ? 2 : 4; }

Walk walk_of(long long rows, int D, long long gate_rows, bool dgate)
{
    if (rows == 0) return {0, dgate, (unsigned)gate_rows, 0, 0, 0, 0};   // sums of nothing
    int per = std::max(1, kMostThreads / norm_threads(D, bwd_vpt(D)));
    if (D >= kRingLeast && D % kE == 0 && D <= 4096) per = std::min(per, kRingThreads / norm_threads(D, 2));
    const long long most = std::min<long long>(rows, 152LL * per);
    const bool summed = dgate && gate_rows < rows;
    const long long groups = summed ? gate_rows : 1, of = rows / groups,
                    cuts = summed ? std::max(1LL, std::min(most / groups, of)) : most;
    return {(int)std::min(most, groups * cuts), summed, (unsigned)groups, (unsigned)cuts, (unsigned)of,
            (unsigned)(of / cuts), (unsigned)(of % cuts)};
}

// RING: the rows come through a ring in shared memory, a stage being refilled once every thread has
// its values in registers, behind the first sums' barrier.
template <typename TIn, typename TRes, typename TG, int VPT, bool VEC, bool RING>
__global__ void __launch_bounds__(RING ? kRingThreads : kMostThreads, 1)
gated_bwd_kernel(const GatedNormBwdArgs a, const Walk walk, const RingPlan plan)
{
    // one vector a thread, or a ring: the weights and the columns' sums in registers, and the next row on its
    // way; more without one: the sums in shared memory, each its thread's own
    constexpr bool KEEP = VPT == 1 || RING;
    extern __shared__ float acc_sm[];
    __shared__ __align__(16) Sums<3> sm[2];
    __shared__ __align__(16) Sums<1> sm_x[2];
    const int D = a.D, nt = blockDim.x, nwarps = nt >> 5;
    const TIn *x = (const TIn *)a.x, *dy = (const TIn *)a.dy;
    const TRes *s = (const TRes *)a.s, *dsum = (const TRes *)a.dsum;
    const TG *gate = (const TG *)a.gate;
    const bool post = a.post_weight != nullptr, pre = a.weight != nullptr, wants_gate = a.dgate != nullptr;
    const unsigned shared = gate ? (unsigned)(a.rows / a.gate_rows) : 1u;
    const bool own_gate = gate && shared == 1;
    __shared__ uint64_t full[kRingMost];
    __shared__ int fail;
    RowRing<5> ring((uint8_t *)acc_sm, full, &fail, plan);
    int at_dy = 0, at_x = 0, at_d = 0, at_g = 0;
    if constexpr (RING) {
        ring.add<0>(s, pre ? D * sizeof(TRes) : 0);
        at_dy = ring.add<1>(dy, pre ? D * sizeof(TIn) : 0);
        at_x = ring.add<2>(x, D * sizeof(TIn));
        at_d = ring.add<3>(dsum, dsum ? D * sizeof(TRes) : 0);
        at_g = ring.add<4>(gate, own_gate ? D * sizeof(TG) : 0);
        __syncthreads();
    }

    const float inv_D = 1.f / (float)D;

    // the columns' sums over rows: of dy s rho_s (dweight), of dn x rho_x (dpost_weight) and of
    // dS x rho_x (dgate without its factor post_weight)
    V8 acc[KEEP ? 3 * VPT : 1];
    auto kept = [&](int which, int k) -> float4 * {   // a thread's own 8 in shared memory
        return (float4 *)acc_sm + ((which * VPT + k) * 2) * nt + threadIdx.x;
    };
    auto add = [&](int which, int k, const V8 &v, float f) {
        if constexpr (KEEP) {
            acc[which * VPT + k] = fma(v, f, acc[which * VPT + k]);
        } else {
            float4 *at = kept(which, k);
            V8 t{{{at[0].x, at[0].y}, {at[0].z, at[0].w}, {at[nt].x, at[nt].y}, {at[nt].z, at[nt].w}}};
            t = fma(v, f, t);
            at[0] = make_float4(t.p[0].x, t.p[0].y, t.p[1].x, t.p[1].y);
            at[nt] = make_float4(t.p[2].x, t.p[2].y, t.p[3].x, t.p[3].y);
        }
    };
    auto sum_of = [&](int which, int k) {
        if constexpr (KEEP) return acc[which * VPT + k];
        const float4 *at = kept(which, k);
        return V8{{{at[0].x, at[0].y}, {at[0].z, at[0].w}, {at[nt].x, at[nt].y}, {at[nt].z, at[nt].w}}};
    };
    auto clear = [&](int which) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if constexpr (KEEP) acc[which * VPT + k] = filled(0.f);
            else kept(which, k)[0] = kept(which, k)[nt] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    sm100::griddep_wait();   // before any memory of another kernel
    sm100::griddep_launch_dependents();
    clear(0);
    clear(1);
    for (int i = 0; i < 2; ++i) {
        clear_sums<3>(sm[i]);
        clear_sums<1>(sm_x[i]);
    }
    __syncthreads();

    V8 w[KEEP ? VPT : 1], wp[KEEP ? VPT : 1];
    auto weights = [&](int k) {
        const int c = place<VEC>(k), at = KEEP ? k : 0;
        w[at] = load8<VEC>(a.weight + c, pre ? D - c : 0);
        wp[at] = load8<VEC>(a.post_weight + c, post ? D - c : 0);
        if (!post) wp[at] = filled(1.f);
    };
    if constexpr (KEEP)
#pragma unroll
        for (int k = 0; k < VPT; ++k) weights(k);

    Raw<TRes, kE, VEC> rs[VPT], rd[VPT];
    Raw<TIn, kE, VEC> ry[VPT], rx[VPT];
    Raw<TG, kE, VEC> rg[VPT];
    auto fetch = [&](int k, long long row) {   // row < 0: none
        const int c = place<VEC>(k), valid = row >= 0 ? D - c : 0;
        const long long o = row * D + c;
        take8<VEC>(rs[k], s + o, pre ? valid : 0);
        take8<VEC>(ry[k], dy + o, pre ? valid : 0);
        take8<VEC>(rx[k], x + o, valid);
        take8<VEC>(rd[k], dsum + o, dsum ? valid : 0);
        if (gate && row >= 0) take8<VEC>(rg[k], gate + (unsigned)row / shared * (long long)D + c, D - c);
    };
    long long held = -1;   // RING: the gate's row in rg
    auto take = [&](int k, long long at_gate) {   // from the ring
        const int c = place<VEC>(k);
        const uint8_t *in = ring.row();
        take8<VEC>(rs[k], (const TRes *)in + c, pre ? D - c : 0);
        take8<VEC>(ry[k], (const TIn *)(in + at_dy) + c, pre ? D - c : 0);
        take8<VEC>(rx[k], (const TIn *)(in + at_x) + c, D - c);
        take8<VEC>(rd[k], (const TRes *)(in + at_d) + c, dsum ? D - c : 0);
        if (own_gate) take8<VEC>(rg[k], (const TG *)(in + at_g) + c, D - c);
        else if (gate && at_gate != held) take8<VEC>(rg[k], gate + at_gate * D + c, D - c);
    };

    // This block's rows one after another; `row` < 0 behind the last.
    // (int outside a ring spills more: 3333 x 777 in fp32 33 us, 28 with 64 bits)
    using Index = std::conditional_t<RING, int, long long>;
    struct Rows {
        unsigned run;
        Index row, end;
    };
    const unsigned runs = walk.groups * walk.cuts;   // fewer than 2^31, as rows
    auto open = [&](unsigned run) {
        const unsigned g = run / walk.cuts, q = run - g * walk.cuts, first = g * walk.per + q * walk.base + min(q, walk.extra);
        return run < runs ? Rows{run, (Index)first, (Index)(first + walk.base + (q < walk.extra))} : Rows{run, -1, -1};
    };
    auto after = [&](Rows r) {
        if (r.row >= 0 && ++r.row == r.end) r = open(r.run + gridDim.x);
        return r;
    };
    Rows at = open(blockIdx.x), ahead = at;   // ahead: the next to go into the ring
    if constexpr (RING) {
        if (ring.issues())
            for (int i = 0; i < plan.stages && ahead.row >= 0; ++i, ahead = after(ahead)) ring.fill(i, ahead.row);
    } else if constexpr (KEEP) {
        fetch(0, at.row);
    }
    int turn = 0;
    while (at.row >= 0) {
        if (walk.summed) clear(2);
        const unsigned run = at.run;
        for (; at.run == run && at.row >= 0; at = after(at), turn ^= 1) {
            const long long row = at.row;
            if constexpr (RING) {
                const long long at_gate = (unsigned)row / shared;
#pragma unroll
                for (int k = 0; k < VPT; ++k) take(k, at_gate);
                held = at_gate;
            } else if constexpr (!KEEP) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) fetch(k, row);
            }
            V8 d[VPT], xv[VPT], sv[VPT], gy[VPT], gv[VPT];
            float2 ss = dup(0.f), sy = dup(0.f), xx = dup(0.f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int at_w = KEEP ? k : 0;
                if constexpr (!KEEP) weights(k);
                xv[k] = widened(rx[k]);
                d[k] = widened(rd[k]);
                if (pre) {
                    sv[k] = widened(rs[k]);
                    gy[k] = widened(ry[k]);
                    ss = dot(sv[k], sv[k], ss);
                    sy = dot(w[at_w] * gy[k], sv[k], sy);
                }
                if (post) xx = dot(xv[k], xv[k], xx);
                if (gate) {
                    gv[k] = widened(rg[k]);
                    if (a.gate_sigmoid) gv[k] = sigmoid(gv[k]);
                }
            }
            float sums[3] = {ss.x + ss.y, sy.x + sy.y, xx.x + xx.y};
            if constexpr (KEEP && !RING) fetch(0, after(at).row);
            row_sums<3>(sums, sm[turn], nwarps);   // two buffers: the next row's sums pass no reader of these
            if constexpr (RING) {
                if (ring.issues() && ahead.row >= 0) {
                    ring.fill(ring.s, ahead.row);
                    ahead = after(ahead);
                }
                ring.step();
            }
            // rho^3 times a sum that is as large as 1 / rho is small: rho's cube alone would leave fp32's range for
            // rows above 4e12 or, without eps, below 2e-13
            const float rho_s = root(fmaf(sums[0], inv_D, a.eps)), m_s = rho_s * (rho_s * (rho_s * (sums[1] * inv_D)));
            const float rho_x = post ? root(fmaf(sums[2], inv_D, a.eps)) : 1.f;
            float2 dots = dup(0.f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = place<VEC>(k), at_w = KEEP ? k : 0;
                if constexpr (!KEEP) weights(k);
                if (pre) {
                    add(0, k, gy[k] * sv[k], rho_s);
                    d[k] = fma(sv[k], -m_s, fma(w[at_w] * gy[k], rho_s, d[k]));
                }
                if (a.dresidual) store8<VEC>((TRes *)a.dresidual + row * D + c, d[k] * a.residual_scale, D - c);
                V8 e = d[k] * xv[k];
                if (wants_gate) {
                    if (walk.summed) {
                        add(2, k, e, rho_x);
                    } else {
                        V8 out = e * (wp[at_w] * rho_x);
                        if (a.gate_sigmoid) out = out * (gv[k] * fma(gv[k], -1.f, filled(1.f)));
                        store8<VEC>((TG *)a.dgate + row * D + c, out, D - c);
                    }
                }
                if (gate) {
                    e = e * gv[k];
                    d[k] = d[k] * gv[k];
                }
                if (post) {
                    add(1, k, e, rho_x);
                    dots = dot(e, wp[at_w], dots);
                    d[k] = d[k] * (wp[at_w] * rho_x);
                }
            }
            float m_x = 0.f;
            if (post) {
                m_x = dots.x + dots.y;
                row_sums<1>(&m_x, sm_x[turn], nwarps);
                m_x = rho_x * (rho_x * (rho_x * (m_x * inv_D)));
            }
            if (a.dx)
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int c = place<VEC>(k);
                    store8<VEC>((TIn *)a.dx + row * D + c, post ? fma(xv[k], -m_x, d[k]) : d[k], D - c);
                }
        }
        if (walk.summed)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = place<VEC>(k);
                if constexpr (!KEEP) weights(k);
                store8<VEC>(a.part_gate + (long long)run * D + c, sum_of(2, k) * wp[KEEP ? k : 0], D - c);
            }
    }
    if constexpr (RING) ring.close(a.status);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = place<VEC>(k);
        if (pre) store8<VEC>(a.part + (size_t)blockIdx.x * D + c, sum_of(0, k), D - c);
        if (post) store8<VEC>(a.part_post + (size_t)blockIdx.x * D + c, sum_of(1, k), D - c);
    }
}

// blockIdx.y 0: dweight, 1: dpost_weight, from every block's share; 2 + g: the gate's row g from its
// runs'.  32 columns a block, kSumRows rows at a time.
constexpr int kSumRows = 32, kSumAhead = 10;   // 304 blocks' shares are one round of loads
template <typename TG>
__global__ void __launch_bounds__(32 * kSumRows)
gated_sum_kernel(const GatedNormBwdArgs a, const Walk walk)
{
    __shared__ float sm[kSumRows][33];
    sm100::griddep_wait();
    sm100::griddep_launch_dependents();
    const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y, D = a.D;
    for (long long u = blockIdx.y; u < 2 + (walk.summed ? walk.groups : 0); u += gridDim.y) {
        if ((u == 0 && !a.weight) || (u == 1 && !a.post_weight)) continue;
        const float *part = u == 0 ? a.part : u == 1 ? a.part_post : a.part_gate + (u - 2) * (long long)walk.cuts * D;
        const int n = u < 2 ? walk.blocks : (int)walk.cuts;
        float t = 0.f;
        if (c < D)
            for (int i = y; i < n; i += kSumRows * kSumAhead) {
                float v[kSumAhead];
#pragma unroll
                for (int q = 0; q < kSumAhead; ++q) v[q] = i + q * kSumRows < n ? part[(size_t)(i + q * kSumRows) * D + c] : 0.f;
#pragma unroll
                for (int q = 0; q < kSumAhead; ++q) t += v[q];
            }
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
    cudaError_t e = cudaSuccess;
    if constexpr (VPT == 1 && VEC)
        if (a.D >= kRingLeast && a.rows > 2LL * walk.blocks) {
            const bool own = a.gate && a.gate_rows == a.rows;
            const RingPlan plan = ring_plan(a.D * (int)((a.weight ? sizeof(TRes) + sizeof(TIn) : 0) + sizeof(TIn) +
                                                        (a.dsum ? sizeof(TRes) : 0) + (own ? sizeof(TG) : 0)),
                                            kRingThreads / norm_threads(a.D, 2));
            if (plan.stages) {
                auto *k = gated_bwd_kernel<TIn, TRes, TG, 2, true, true>;
                // always the most: the attribute is the kernel's, shared by all host threads
                e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
                if (e != cudaSuccess) return e;
                return launch_after(k, walk.blocks, norm_threads(a.D, 2), plan.stages * plan.stage, st, a, walk, plan);
            }
        }
    auto *k = gated_bwd_kernel<TIn, TRes, TG, VPT, VEC, false>;
    size_t smem = 0;
    if constexpr (VPT > 1) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 3 * VPT * kE * kMostThreads * (int)sizeof(float));
        if (e != cudaSuccess) return e;
        smem = (size_t)3 * VPT * kE * nt * sizeof(float);
    }
    return launch_after(k, walk.blocks, nt, smem, st, a, walk, RingPlan{0, 0});
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
    const long long sums = 2 + (walk.summed ? (long long)walk.groups : 0);
    return launch_after(gated_sum_kernel<TG>, dim3((a.D + 31) / 32, (unsigned)std::min<long long>(sums, 65535)),
                        dim3(32, kSumRows), 0, st, a, walk);
}

}  // namespace

// For either kind of call: without dgate a shared gate's groups do not bound the blocks, and the walk may have
// more of them (1530 rows of 2048 with 153 gates: 608 shares, 459 with dgate).
size_t gated_add_rmsnorm_bwd_floats(long long rows, int D, long long gate_rows)
{
    const long long gates = gate_rows ? gate_rows : rows;
    return std::max(walk_of(rows, D, gates, true).shares(), walk_of(rows, D, gates, false).shares()) * D;
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
