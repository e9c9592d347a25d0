// Gradient of the selective state space scan.
//
// With yb = dy silu(z) and g_t the gradient that reaches h_t,
//   g_t = C_t yb_t + a_{t+1} g_{t+1},        dC_t = sum_d yb_t h_t,   dB_t = sum_d g_t dt u,
//   q_t = sum_n g_t B_t,                     w_t = g_t a_t h_{t-1},
//   ddt = sum_n A w_t + u q_t,               du = dt q_t + D yb,
//   ddelta = ddt softplus'(delta + bias),    dz = dy silu'(z) (sum_n C h_t + D u),
//   dA = sum_t dt w_t,  dD = sum_t yb u,     dh0 = a_1 g_1.
//
// The forward saved the state entering every 32 tokens; a block takes those tiles in reverse
// order.  Inside a tile it first runs the states forward, keeping every fourth in shared
// memory, then takes four tokens at a time in reverse: their states and decays are formed
// again into registers and the gradients follow.  A lane owns two channels x 4 states, so the
// channel sums of dB and dC start in registers; the rest goes by halving exchanges, over the
// lanes of a channel for q, sum A w and sum C h (four tokens together), over the channels of a
// warp for dB and dC.  An update costs 15 fp32 operations and two exponentials (100 us for
// 2 x 2048 tokens of 4096 x 16 on the fp32 pipes alone) and takes 24 instructions, packed pairs
// counted once: the sums' shuffles, selections and additions are a quarter of them, broadcasts
// into pairs, loads and the elementwise work another.  350 us: two warps a scheduler run the
// recurrence and issue 53 % of the time.
//
// As in the forward a block is four warps of this recurrence and four helpers, which read the
// rows, form dt, dt u and yb a tile ahead, and turn the sums into du, ddelta, dz and the
// block's dB, dC a tile behind.  The recurrence needs most of the registers (states and decays
// of four tokens), so the block's are split: 152 a thread for it, 104 for the helpers.
//
// Sums across blocks (dB, dC over the channel blocks of a group; dA, dD and the bias over
// sequences and segments) go to the workspace and are added by a last launch in a fixed
// order: no atomics, the same bits on every call.  Few channels: the tokens are cut into
// segments; a first launch forms every segment's carry from zero (g alone, one exponential;
// in two parts where that launch would fill half the card: 46 us for 56 at the size above)
// and a block composes what reaches its end from the later ones.
#include <type_traits>

#include "ssm_common.cuh"

namespace ldn {
namespace {
using namespace ssm;

constexpr int kMain = 128, kThreads = 256, kWarps = 4, S = 4, KC = 2, SUB = 4;
// Registers a thread: what the block is launched with, and what its halves hold after the split.
constexpr int kRegs = 128, kRegsMain = 152, kRegsHelper = 104;
static_assert(kRegsMain + kRegsHelper == 2 * kRegs, "the halves share what the block has");

template <int N> constexpr int block_ch() { return kMain / (N / S) * KC; }
int block_channels(int N) { return kMain / (N / S) * KC; }

struct Plan {
    int n, len;      // segments per sequence, tokens of one (a multiple of TT)
    int gblocks;     // channel blocks per group
    int parts;       // parts of a segment whose carries are formed side by side
    __host__ __device__ int part_len() const { return ((len + parts - 1) / parts + TT - 1) / TT * TT; }
};

struct Work {
    float *bc;       // [gblocks][B * T][G][2][N]
    float *A;        // [B * n][D][N]
    float *D, *bias; // [B * n][D]
    float *carry;    // [B * n * parts][D][N]
    float *sums;     // [B * n * parts][D]
};

// Tiles are kept by warp, rows of the warp's WC channels.
template <int N>
struct Smem {
    static constexpr int WC = block_ch<N>() / kWarps, ROW = 2 * WC + 4;   // + 4: rows differ in banks
    float step[2][kWarps][TT * ROW];        // dt, dt u of a channel; then dt, q
    float yb[2][kWarps][TT * WC];           // yb; then sum C h
    float ww[kWarps][TT * WC];              // sum A2 w
    float B[2][TT * N], C[2][TT * N];
    float4 ckpt[TT / SUB - 1][KC][kMain];   // the state entering every SUB tokens but the last
    float red[kWarps][TT][2 * N];           // dB, dC summed over a warp's channels
};

struct Gate { float2 y, dy; };   // silu(z), silu'(z)
__device__ __forceinline__ Gate gate_of(float2 z)
{
    const float2 s = rcp(__fadd2_rn(ex2(__fmul2_rn(z, dup(-kLog2e))), dup(1.f)));
    const float2 one_minus = __ffma2_rn(s, dup(-1.f), dup(1.f));
    return {__fmul2_rn(z, s), __fmul2_rn(s, __ffma2_rn(z, one_minus, dup(1.f)))};
}

template <int ID> __device__ __forceinline__ void bar_arrive()
{
    asm volatile("barrier.cta.arrive %0, %1;" ::"n"(ID), "n"(kThreads) : "memory");
}
template <int ID> __device__ __forceinline__ void bar_sync()
{
    asm volatile("barrier.cta.sync %0, %1;" ::"n"(ID), "n"(kThreads) : "memory");
}
constexpr int kTaken = 1;   // the last tile's red and ww have been read

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// K neighbouring elements of a tile's B or C rows by each helper thread, widened to dst[TT][N].
template <typename T, int N>
__device__ __forceinline__ void rows_to_shared(float *dst, const T *src, long long ld, int rows, bool vec, int tid)
{
    constexpr int K = 4;
#pragma unroll
    for (int k = 0; k < (TT * N + kMain * K - 1) / (kMain * K); ++k) {
        const int i = (k * kMain + tid) * K, r = i / N;
        if (TT * N % (kMain * K) != 0 && i >= TT * N) continue;
        float v[K];
        const T *p = src + r * ld + i % N;
        if (vec) load_n<K, true>(p, v, r < rows ? K : 0);
        else load_n<K, false>(p, v, r < rows ? K : 0);
        *reinterpret_cast<float4 *>(dst + i) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

enum { kCarry = 0, kFull = 1 };

template <typename TIn, int N, bool VEC, int PHASE>
__global__ void __launch_bounds__(kThreads, 2)
ssm_backward_kernel(const SsmBwdArgs a, const Plan pl, const Work wk)
{
    constexpr int L = N / S, DB = block_ch<N>();
    extern __shared__ __align__(16) unsigned char smem_raw[];
    using Sm = Smem<N>;
    constexpr int WC = Sm::WC, ROW = Sm::ROW;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    const int Dg = a.D / a.G;
    const unsigned cblocks = (unsigned)pl.gblocks * a.G;
    const unsigned cb = blockIdx.x % cblocks, bs = blockIdx.x / cblocks;
    // kCarry: the parts of all segments but the first, whose carry nothing takes
    const int segs = PHASE == kCarry ? (pl.n - 1) * pl.parts : pl.n, b = (int)(bs / segs);
    const int part = PHASE == kCarry ? (int)(bs % segs) + pl.parts : 0;
    const int seg = PHASE == kCarry ? part / pl.parts : (int)(bs % segs);
    const int grp = (int)(cb / pl.gblocks), gb = (int)(cb % pl.gblocks), cg = gb * DB;
    const int c0 = grp * Dg + cg, cols = min(DB, Dg - cg);
    const bool helper = threadIdx.x >= kMain;
    const int tid = threadIdx.x % kMain, lane = tid & 31, warp = tid >> 5;
    const int len = seq_len(a.lens, b, a.T);
    const int plen = PHASE == kCarry ? pl.part_len() : pl.len;
    const int tb = seg * pl.len + (PHASE == kCarry ? part % pl.parts * plen : 0);
    const int te = min(min(tb + plen, (seg + 1) * pl.len), a.T);   // before tb: an empty part
    // tiles with rows of the sequence; through those behind its end g passes unchanged
    const int tiles = (max(min(len, te) - tb, 0) + TT - 1) / TT;
    const size_t row0 = (size_t)b * a.T + tb;   // the segment's first row
    const size_t bseg = PHASE == kCarry ? (size_t)b * pl.n * pl.parts + part : (size_t)b * pl.n + seg;
    auto rows_of = [&](int it) { return min(max(min(len, te) - tb - it * TT, 0), TT); };

    if (helper) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsHelper));
        constexpr int V = WC < 4 ? WC : 4, PR = WC / V;   // channels of a vector, vectors of a row
        static_assert(V == 4, "four channels a vector");
        const int w0 = warp * WC, ch = (lane % PR) * V, valid = cols - w0 - ch;
        const size_t cc = c0 + w0 + ch;
        const TIn *u = (const TIn *)a.u + row0 * a.ldu + cc;
        const TIn *dl = (const TIn *)a.delta + row0 * a.ldd + cc;
        const TIn *z = a.z ? (const TIn *)a.z + row0 * a.ldz + cc : nullptr;
        const TIn *dy = (const TIn *)a.dy + row0 * a.D + cc;
        const TIn *Bm = (const TIn *)a.Bm + row0 * a.ldb + (size_t)grp * N;
        const TIn *Cm = (const TIn *)a.Cm + row0 * a.ldc + (size_t)grp * N;
        auto whole = [](const TIn *p, long long ld) {
            return (((uintptr_t)p | (uintptr_t)(ld * (long long)sizeof(TIn))) & (4 * sizeof(TIn) - 1)) == 0;
        };
        const bool vB = whole(Bm, a.ldb), vC = whole(Cm, a.ldc);
        float2 bias[2], skip[2], accD[2] = {dup(0.f), dup(0.f)}, accb[2] = {dup(0.f), dup(0.f)};
        load_n<V, false>(a.bias + cc, reinterpret_cast<float *>(bias), a.bias ? valid : 0);
        load_n<V, false>(a.Dskip + cc, reinterpret_cast<float *>(skip), a.Dskip ? valid : 0);

        // A batch of rows is loaded before any of it is used: one latency for the batch.
        constexpr int ITEMS = TT * PR / 32, MOST = PHASE == kCarry && sizeof(TIn) == 2 ? 4 : 2,
                      BATCH = ITEMS < MOST ? ITEMS : MOST;
        using R4 = Raw<TIn, 4>;
        auto load_batch = [&](int t, int rows, int k0, R4 *ru, R4 *rd, R4 *ry, R4 *rz) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int row = ((k0 + k) * 32 + lane) / PR, n = row < rows ? valid : 0;
                const size_t at = t + row;
                if (PHASE == kFull) ru[k].template load<VEC>(u + at * a.ldu, n);
                rd[k].template load<VEC>(dl + at * a.ldd, n);
                ry[k].template load<VEC>(dy + at * a.D, n);
                if (z) rz[k].template load<VEC>(z + at * a.ldz, n);
            }
        };
        // A tile's lines to L2, one iteration before they are loaded: a thread a row of a tensor,
        // and of the entering states.
        auto announce = [&](int it) {
            const int rows = rows_of(it), row = tid % TT, which = tid / TT;
            if (row < rows) {
                const TIn *p = which == 0 ? dl : which == 1 ? dy : which == 2 ? z : u;
                const long long ld = which == 0 ? a.ldd : which == 1 ? a.D : which == 2 ? a.ldz : a.ldu;
                const int first = w0 + ch;   // p is this lane's place in the row
                if (p && (which < 3 || PHASE == kFull))
                    for (int c = 0; c < cols; c += 128 / (int)sizeof(TIn))
                        prefetch_l2(p - first + (size_t)(it * TT + row) * ld + c);
            }
            if (PHASE == kFull) {
                const size_t ck = (size_t)b * ((a.T + TT - 1) / TT) + tb / TT + it;
                for (int i = tid * 32; i < cols * N; i += kMain * 32) prefetch_l2(a.states + (ck * a.D + c0) * N + i);
            }
        };
        auto ready = [&](int it) {
            const int rows = rows_of(it), t = it * TT;
#pragma unroll 1
            for (int k0 = 0; k0 < ITEMS; k0 += BATCH) {
                R4 ru[BATCH], rd[BATCH], ry[BATCH], rz[BATCH];
                load_batch(t, rows, k0, ru, rd, ry, rz);
                if (k0 == 0) {
                    if (PHASE == kFull)
                        rows_to_shared<TIn, N>(sm.B[it & 1], Bm + (size_t)t * a.ldb, a.ldb, rows, vB, tid);
                    rows_to_shared<TIn, N>(sm.C[it & 1], Cm + (size_t)t * a.ldc, a.ldc, rows, vC, tid);
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int row = ((k0 + k) * 32 + lane) / PR;
                    float2 vu[2] = {dup(0.f), dup(0.f)}, vd[2], vy[2], vz[2];
                    if (PHASE == kFull) ru[k].widen(reinterpret_cast<float *>(vu));
                    rd[k].widen(reinterpret_cast<float *>(vd));
                    ry[k].widen(reinterpret_cast<float *>(vy));
                    if (z) rz[k].widen(reinterpret_cast<float *>(vz));
                    float4 *o = reinterpret_cast<float4 *>(sm.step[it & 1][warp] + row * ROW + 2 * ch);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float2 dt = __fadd2_rn(vd[c], bias[c]);
                        if (a.softplus) dt = softplus_accurate(dt);
                        if (row >= rows) dt = dup(0.f);   // a row past the end steps by zero: g stays
                        const float2 du = __fmul2_rn(dt, vu[c]);
                        o[c] = make_float4(dt.x, du.x, dt.y, du.y);
                        if (z) vy[c] = __fmul2_rn(vy[c], silu_fast(vz[c]));
                    }
                    *reinterpret_cast<float4 *>(sm.yb[it & 1][warp] + row * WC + ch) =
                        make_float4(vy[0].x, vy[0].y, vy[1].x, vy[1].y);
                }
            }
            __syncwarp();
        };
        auto finished = [&](int it) {
            const int rows = rows_of(it), t = it * TT, live = min(te - tb - t, TT);
            float *bc = wk.bc + (((size_t)gb * a.B * a.T + row0 + t) * a.G + grp) * (2 * N);
            TIn *du = (TIn *)a.du + (row0 + t) * a.D + cc, *dd = (TIn *)a.ddelta + (row0 + t) * a.D + cc;
            TIn *dz = z ? (TIn *)a.dz + (row0 + t) * a.D + cc : nullptr;
#pragma unroll 1
            for (int k0 = 0; k0 < ITEMS; k0 += BATCH) {
                R4 ru[BATCH], rd[BATCH], ry[BATCH], rz[BATCH];
                load_batch(t, rows, k0, ru, rd, ry, rz);
                if (k0 == 0)   // dB, dC of the block's channels, while the rows arrive
                    for (int i = tid; i < live * (2 * N / 4); i += kMain) {
                        const int row = i / (2 * N / 4), n = i % (2 * N / 4) * 4;
                        float4 s = *reinterpret_cast<const float4 *>(&sm.red[0][row][n]);
#pragma unroll
                        for (int k = 1; k < kWarps; ++k) {
                            const float4 q = *reinterpret_cast<const float4 *>(&sm.red[k][row][n]);
                            s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
                        }
                        // past the end sums of zeros, but where a state is NaN or infinite
                        if (row >= rows) s = make_float4(0.f, 0.f, 0.f, 0.f);
                        *reinterpret_cast<float4 *>(bc + (size_t)row * a.G * (2 * N) + n) = s;
                    }
                // the rows' du, ddelta, dz
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int row = ((k0 + k) * 32 + lane) / PR;
                    float2 vu[2], vd[2], vy[2], vz[2], pre[2], ww[2], oz[2], ou[2], od[2];
                    ru[k].widen(reinterpret_cast<float *>(vu));
                    rd[k].widen(reinterpret_cast<float *>(vd));
                    ry[k].widen(reinterpret_cast<float *>(vy));
                    if (z) rz[k].widen(reinterpret_cast<float *>(vz));
                    load_n<V, true>(sm.yb[it & 1][warp] + row * WC + ch, reinterpret_cast<float *>(pre));
                    load_n<V, true>(sm.ww[warp] + row * WC + ch, reinterpret_cast<float *>(ww));
                    const float4 *o = reinterpret_cast<const float4 *>(sm.step[it & 1][warp] + row * ROW + 2 * ch);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float4 s = o[c];
                        const float2 dt = make_float2(s.x, s.z), q = make_float2(s.y, s.w);
                        float2 yb = vy[c];
                        if (z) {
                            const Gate gt = gate_of(vz[c]);
                            oz[c] = __fmul2_rn(__fmul2_rn(vy[c], gt.dy), __ffma2_rn(skip[c], vu[c], pre[c]));
                            yb = __fmul2_rn(vy[c], gt.y);
                        }
                        ou[c] = __ffma2_rn(dt, q, __fmul2_rn(skip[c], yb));
                        od[c] = __ffma2_rn(ww[c], dup(kLn2), __fmul2_rn(vu[c], q));
                        if (a.softplus) {
                            const float2 x = __fadd2_rn(vd[c], bias[c]);
                            od[c] = __fmul2_rn(od[c], rcp(__fadd2_rn(ex2(__fmul2_rn(x, dup(-kLog2e))), dup(1.f))));
                        }
                        if (row >= rows) ou[c] = od[c] = oz[c] = yb = dup(0.f);
                        accD[c] = __ffma2_rn(yb, vu[c], accD[c]);
                        accb[c] = __fadd2_rn(accb[c], od[c]);
                    }
                    if (row < live) {
                        store_n<V, VEC>(du + (size_t)row * a.D, reinterpret_cast<float *>(ou), valid);
                        store_n<V, VEC>(dd + (size_t)row * a.D, reinterpret_cast<float *>(od), valid);
                        if (z) store_n<V, VEC>(dz + (size_t)row * a.D, reinterpret_cast<float *>(oz), valid);
                    }
                }
            }
            __syncwarp();
        };
        if (tiles > 0) ready(tiles - 1);
        if (tiles > 1) announce(tiles - 2);
        __syncthreads();
        for (int it = tiles - 1; it >= 0; --it) {
            if (PHASE == kFull) {
                if (it + 1 < tiles) finished(it + 1);
                bar_arrive<kTaken>();
            }
            if (it > 1) announce(it - 2);
            if (it > 0) ready(it - 1);
            __syncthreads();
        }
        if (PHASE == kFull) {
            if (tiles > 0) finished(0);
            // behind the end: no gradient (64 bits: a segment's vectors may outnumber an int)
            const float zeros[V] = {};
            for (long long i = (long long)tiles * TT * PR + lane; i < (long long)(te - tb) * PR; i += 32) {
                const size_t at = (row0 + i / PR) * a.D + cc;
                store_n<V, VEC>((TIn *)a.du + at, zeros, valid);
                store_n<V, VEC>((TIn *)a.ddelta + at, zeros, valid);
                if (z) store_n<V, VEC>((TIn *)a.dz + at, zeros, valid);
            }
            for (long long i = tid + (long long)tiles * TT * (2 * N / 4); i < (long long)(te - tb) * (2 * N / 4);
                 i += kMain)
                *reinterpret_cast<float4 *>(
                    wk.bc + (((size_t)gb * a.B * a.T + row0 + i / (2 * N / 4)) * a.G + grp) * (2 * N) +
                    i % (2 * N / 4) * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
            // dD and the bias over the lanes that share a vector's channels
#pragma unroll
            for (int o = 16; o >= PR; o >>= 1)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    accD[c].x += __shfl_xor_sync(0xffffffffu, accD[c].x, o);
                    accD[c].y += __shfl_xor_sync(0xffffffffu, accD[c].y, o);
                    accb[c].x += __shfl_xor_sync(0xffffffffu, accb[c].x, o);
                    accb[c].y += __shfl_xor_sync(0xffffffffu, accb[c].y, o);
                }
            if (lane < PR) {
                store_n<V, false>(wk.D + bseg * a.D + cc, reinterpret_cast<float *>(accD), valid);
                store_n<V, false>(wk.bias + bseg * a.D + cc, reinterpret_cast<float *>(accb), valid);
            }
        }
        return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMain));
    // The recurrence: lane l of a channel pair's L has states l S .. l S + S - 1 of channels
    // 2 slot and 2 slot + 1.
    const int l = tid % L, slot = tid / L, wch = 2 * slot - warp * WC;   // the pair's place in the warp
    // dA is summed tile by tile: 32 additions and then one a tile keep the sum of thousands of
    // tokens to a few roundings
    float2 A2[KC][2], g[KC][2], dA[KC][2], dAsum[KC][2];
    float sumdt[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int ch = KC * slot + k;
        const bool on = ch < cols;
        const size_t at = (size_t)(c0 + ch) * N + l * S;
        sumdt[k] = 0.f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            A2[k][s] = on ? make_float2(rate(a.A[at + 2 * s]), rate(a.A[at + 2 * s + 1])) : dup(0.f);
            g[k][s] = dA[k][s] = dAsum[k][s] = dup(0.f);
            if (PHASE == kFull && on && a.dh_final) {
                const float *p = a.dh_final + (size_t)b * a.D * N + at + 2 * s;
                g[k][s] = make_float2(p[0], p[1]);
            }
        }
        if (PHASE == kFull && on)
#pragma unroll 4
            for (int j = pl.n * pl.parts - 1; j >= (seg + 1) * pl.parts; --j) {   // through the later segments
                const size_t e = ((size_t)b * pl.n * pl.parts + j) * a.D + c0 + ch;
                const float sd = wk.sums[e];
                const float *p = wk.carry + e * N + l * S;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    g[k][s] = __ffma2_rn(decay(A2[k][s], sd), g[k][s],
                                         make_float2(p[2 * s], p[2 * s + 1]));
            }
    }
    __syncthreads();
    for (int it = tiles - 1; it >= 0; --it) {
        float *step = sm.step[it & 1][warp] + 2 * wch, *yb = sm.yb[it & 1][warp] + wch;
        const float *Br = sm.B[it & 1] + l * S, *Cr = sm.C[it & 1] + l * S;
        if constexpr (PHASE == kCarry) {
#pragma unroll 8
            for (int r = TT - 1; r >= 0; --r) {
                const float4 q = *reinterpret_cast<const float4 *>(step + r * ROW);
                const float2 y = *reinterpret_cast<const float2 *>(yb + r * WC);
                const float4 c = *reinterpret_cast<const float4 *>(Cr + r * N);
                const float2 Cv[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
                sumdt[0] += q.x;
                sumdt[1] += q.z;
#pragma unroll
                for (int k = 0; k < KC; ++k)
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        g[k][s] = __fmul2_rn(decay(A2[k][s], k ? q.z : q.x),
                                             __ffma2_rn(Cv[s], dup(k ? y.y : y.x), g[k][s]));
            }
        } else {
            float2 h[KC][2];
            const size_t ck = (size_t)b * ((a.T + TT - 1) / TT) + tb / TT + it;
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int ch = KC * slot + k;
                const float4 q = ch < cols
                    ? *reinterpret_cast<const float4 *>(a.states + (ck * a.D + c0 + ch) * N + l * S)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
                h[k][0] = make_float2(q.x, q.y);
                h[k][1] = make_float2(q.z, q.w);
            }
            // one token of the states: h = a h + dt u B, given its row of step and of B
            auto advance = [&](const float4 &q, const float4 &c, float2 (*av)[2], const float2 (*hi)[2],
                               float2 (*ho)[2]) {
                const float2 Bv[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
#pragma unroll
                for (int k = 0; k < KC; ++k)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        av[k][s] = decay(A2[k][s], k ? q.z : q.x);
                        ho[k][s] = __ffma2_rn(av[k][s], hi[k][s], __fmul2_rn(dup(k ? q.w : q.y), Bv[s]));
                    }
            };
#pragma unroll
            for (int sub = 0; sub < TT / SUB - 1; ++sub) {
                float4 q[SUB], c[SUB];
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
                    q[j] = *reinterpret_cast<const float4 *>(step + (sub * SUB + j) * ROW);
                    c[j] = *reinterpret_cast<const float4 *>(Br + (sub * SUB + j) * N);
                }
#pragma unroll
                for (int k = 0; k < KC; ++k)
                    sm.ckpt[sub][k][tid] = make_float4(h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y);
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
                    float2 av[KC][2];
                    advance(q[j], c[j], av, h, h);
                }
            }
            bar_sync<kTaken>();
#pragma unroll 1
            for (int sub = TT / SUB - 1; sub >= 0; --sub) {
                float4 q[SUB], bq[SUB], cq[SUB];
                float2 y[SUB];
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
                    const int r = sub * SUB + j;
                    q[j] = *reinterpret_cast<const float4 *>(step + r * ROW);
                    bq[j] = *reinterpret_cast<const float4 *>(Br + r * N);
                    cq[j] = *reinterpret_cast<const float4 *>(Cr + r * N);
                    y[j] = *reinterpret_cast<const float2 *>(yb + r * WC);
                }
                float2 hh[SUB + 1][KC][2], av[SUB][KC][2];   // states before each token, decays
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    if (sub < TT / SUB - 1) {
                        const float4 v = sm.ckpt[sub][k][tid];
                        h[k][0] = make_float2(v.x, v.y);
                        h[k][1] = make_float2(v.z, v.w);
                    }
                    hh[0][k][0] = h[k][0];
                    hh[0][k][1] = h[k][1];
                }
#pragma unroll
                for (int j = 0; j < SUB; ++j) advance(q[j], bq[j], av[j], hh[j], hh[j + 1]);
                float qs[SUB * KC], ws[SUB * KC], ps[SUB * KC];
#pragma unroll
                for (int j = SUB - 1; j >= 0; --j) {
                    const int r = sub * SUB + j;
                    const float2 Bv[2] = {make_float2(bq[j].x, bq[j].y), make_float2(bq[j].z, bq[j].w)};
                    const float2 Cv[2] = {make_float2(cq[j].x, cq[j].y), make_float2(cq[j].z, cq[j].w)};
                    float2 dB[2], dC[2];
#pragma unroll
                    for (int k = 0; k < KC; ++k) {
                        const float2 dt = dup(k ? q[j].z : q[j].x), du = dup(k ? q[j].w : q[j].y);
                        const float2 ybk = dup(k ? y[j].y : y[j].x);
                        float2 aq, aw, ap;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const float2 ht = hh[j + 1][k][s];
                            g[k][s] = __ffma2_rn(Cv[s], ybk, g[k][s]);
                            dB[s] = k ? __ffma2_rn(g[k][s], du, dB[s]) : __fmul2_rn(g[k][s], du);
                            dC[s] = k ? __ffma2_rn(ht, ybk, dC[s]) : __fmul2_rn(ht, ybk);
                            aq = s ? __ffma2_rn(g[k][s], Bv[s], aq) : __fmul2_rn(g[k][s], Bv[s]);
                            ap = s ? __ffma2_rn(ht, Cv[s], ap) : __fmul2_rn(ht, Cv[s]);
                            g[k][s] = __fmul2_rn(g[k][s], av[j][k][s]);
                            const float2 w = __fmul2_rn(g[k][s], hh[j][k][s]);
                            aw = s ? __ffma2_rn(A2[k][s], w, aw) : __fmul2_rn(A2[k][s], w);
                            dA[k][s] = __ffma2_rn(w, dt, dA[k][s]);
                        }
                        qs[j * KC + k] = aq.x + aq.y;
                        ws[j * KC + k] = aw.x + aw.y;
                        ps[j * KC + k] = ap.x + ap.y;
                    }
                    // over the warp's channels: lanes l, l + L, ...
                    constexpr int GR = 32 / L, HELD = 8 >= GR ? 8 / GR : 1, DUP = 8 >= GR ? 1 : GR / 8;
                    float v[8] = {dB[0].x, dB[0].y, dB[1].x, dB[1].y, dC[0].x, dC[0].y, dC[1].x, dC[1].y};
                    reduce_halving<8, 16, L>(v, lane);
                    const int gr = lane / L;
                    if (gr % DUP == 0)
#pragma unroll
                        for (int i = 0; i < HELD; ++i) {
                            const int idx = (gr / DUP) * HELD + i;
                            sm.red[warp][r][(idx >> 2) * N + l * S + (idx & 3)] = v[i];
                        }
                }
                // over a channel's lanes, four tokens together
                constexpr int V = SUB * KC, HELD = V >= L ? V / L : 1, DUP = V >= L ? 1 : L / V;
                reduce_halving<V, L / 2, 1>(qs, lane);
                reduce_halving<V, L / 2, 1>(ws, lane);
                reduce_halving<V, L / 2, 1>(ps, lane);
                __syncwarp();   // the rows written below have been read by all of a channel's lanes
                if (l % DUP == 0)
#pragma unroll
                    for (int i = 0; i < HELD; ++i) {
                        const int idx = (l / DUP) * HELD + i, r = sub * SUB + idx / KC, c = idx % KC;
                        step[r * ROW + 2 * c + 1] = qs[i];
                        yb[r * WC + c] = ps[i];
                        sm.ww[warp][r * WC + wch + c] = ws[i];
                    }
            }
#pragma unroll
            for (int k = 0; k < KC; ++k)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    dAsum[k][s] = __fadd2_rn(dAsum[k][s], dA[k][s]);
                    dA[k][s] = dup(0.f);
                }
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int ch = KC * slot + k;
        if (ch >= cols) continue;
        const size_t e = bseg * a.D + c0 + ch;
        const float4 gv = make_float4(g[k][0].x, g[k][0].y, g[k][1].x, g[k][1].y);
        if (PHASE == kCarry) {
            *reinterpret_cast<float4 *>(wk.carry + e * N + l * S) = gv;
            if (l == 0) wk.sums[e] = sumdt[k];
        } else {
            *reinterpret_cast<float4 *>(wk.A + e * N + l * S) =
                make_float4(dAsum[k][0].x, dAsum[k][0].y, dAsum[k][1].x, dAsum[k][1].y);
            if (seg == 0 && a.dh0)
                *reinterpret_cast<float4 *>(a.dh0 + ((size_t)b * a.D + c0 + ch) * N + l * S) = gv;
        }
    }
}

// The sums across blocks in a fixed order: dB, dC over the channel blocks of a group, four
// values a thread and kSlices threads a value (few rows are few threads, and one thread alone
// would wait for every block's load in turn); dA, dD and the bias over sequences and segments
// (np of them), a thread each.
constexpr int kSlices = 8, kSums = 32;   // 32 x 8 threads
template <typename TIn>
__global__ void __launch_bounds__(kSums * kSlices)
ssm_sum_kernel(const SsmBwdArgs a, const Work wk, int gblocks, int np, unsigned bc_blocks)
{
    __shared__ float4 sm[kSlices][kSums];
    const int N = a.N, x = threadIdx.x % kSums, y = threadIdx.x / kSums;
    if (blockIdx.x < bc_blocks) {
        const size_t n = (size_t)a.B * a.T * a.G * 2 * N, i = ((size_t)blockIdx.x * kSums + x) * 4;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n)
#pragma unroll 4
            for (int k = y; k < gblocks; k += kSlices) {
                const float4 q = *reinterpret_cast<const float4 *>(wk.bc + (size_t)k * n + i);
                t.x += q.x; t.y += q.y; t.z += q.z; t.w += q.w;
            }
        sm[y][x] = t;
        __syncthreads();
        if (y != 0 || i >= n) return;
#pragma unroll
        for (int k = 1; k < kSlices; ++k) {
            const float4 q = sm[k][x];
            t.x += q.x; t.y += q.y; t.z += q.z; t.w += q.w;
        }
        const size_t row = i / (2 * N);
        const int c = (int)(i % (2 * N));
        TIn *o = (c < N ? (TIn *)a.dB : (TIn *)a.dC) + row * N + (c < N ? c : c - N);
        const float v[4] = {t.x, t.y, t.z, t.w};
        store_n<4, false>(o, v);
        return;
    }
    const size_t i = (size_t)(blockIdx.x - bc_blocks) * (kSums * kSlices) + threadIdx.x, nA = (size_t)a.D * N;
    const float *src;
    float *dst;
    size_t per, o;
    if (i < nA) { src = wk.A; dst = a.dA; per = nA; o = i; }
    else if (i < nA + a.D) { src = wk.D; dst = a.dD; per = a.D; o = i - nA; }
    else if (i < nA + 2 * (size_t)a.D) { src = wk.bias; dst = a.dbias; per = a.D; o = i - nA - a.D; }
    else return;
    if (!dst) return;
    float t = 0.f;
#pragma unroll 4
    for (int k = 0; k < np; ++k) t += src[k * per + o];
    dst[o] = t;
}

constexpr int kSms = 152;
constexpr long long kMostSegs = 64;   // the first one composes all others, one after another

// Segments per sequence: enough to fill the SMs at two blocks each, of at least four tiles.
Plan bwd_plan(int B, int T, int D, int N, int G)
{
    const int db = block_channels(N), gblocks = (D / G + db - 1) / db;
    const long long blocks = (long long)B * G * gblocks;
    const int n = (int)std::max(1LL, std::min<long long>({kSms * 2 / blocks, T / (4 * TT), kMostSegs}));
    const int len = std::max(TT, (int)((((long long)T + n - 1) / n + TT - 1) / TT) * TT);
    const int segs = std::max(1, (T + len - 1) / len);
    // the carries' launch leaves half the card empty where it has one of two segments
    const int parts = segs > 1 && 2 * (segs - 1) * blocks <= kSms * 2 ? 2 : 1;
    return {segs, len, gblocks, parts};
}

size_t up4(size_t n) { return (n + 3) / 4 * 4; }

// The workspace's parts, every one a multiple of 16 bytes; their floats in all.
size_t lay_out(const Plan &p, int B, int T, int D, int N, int G, float *base, Work *w)
{
    const size_t np = (size_t)B * p.n;
    size_t at = 0;
    auto take = [&](size_t n) { float *q = base ? base + at : nullptr; at += up4(n); return q; };
    w->bc = take((size_t)p.gblocks * B * T * G * 2 * N);
    w->A = take(np * D * N);
    w->D = take(np * D);
    w->bias = take(np * D);
    w->carry = take(p.n > 1 ? np * p.parts * D * N : 0);
    w->sums = take(p.n > 1 ? np * p.parts * D : 0);
    return at;
}

template <typename TIn, int N, bool VEC, int PHASE>
cudaError_t bwd_launch(const SsmBwdArgs &a, const Plan &p, const Work &w, cudaStream_t st)
{
    constexpr int bytes = (int)sizeof(Smem<N>);
    auto *k = ssm_backward_kernel<TIn, N, VEC, PHASE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    // the split of the registers waits for what the launch has to hold
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, k);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kRegs) return cudaErrorInvalidConfiguration;
    const long long segs = PHASE == kCarry ? (p.n - 1) * p.parts : p.n;
    k<<<(unsigned)(p.gblocks * segs * a.G * a.B), kThreads, bytes, st>>>(a, p, w);
    return cudaGetLastError();
}

template <typename TIn, int N, bool VEC>
cudaError_t bwd_run(const SsmBwdArgs &a, cudaStream_t st)
{
    const Plan p = bwd_plan(a.B, a.T, a.D, a.N, a.G);
    Work w;
    lay_out(p, a.B, a.T, a.D, a.N, a.G, a.ws, &w);
    if (p.n > 1) {
        const cudaError_t e = bwd_launch<TIn, N, VEC, kCarry>(a, p, w, st);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = bwd_launch<TIn, N, VEC, kFull>(a, p, w, st);
    if (e != cudaSuccess) return e;
    const unsigned bcb = (unsigned)(((size_t)a.B * a.T * a.G * 2 * N / 4 + kSums - 1) / kSums);
    const unsigned pb = (unsigned)(((size_t)a.D * (N + 2) + kSums * kSlices - 1) / (kSums * kSlices));
    ssm_sum_kernel<TIn><<<bcb + pb, kSums * kSlices, 0, st>>>(a, w, p.gblocks, a.B * p.n, bcb);
    return cudaGetLastError();
}

template <typename TIn, int N>
cudaError_t bwd_pick(const SsmBwdArgs &a, cudaStream_t st)
{
    constexpr int E = 16 / sizeof(TIn);
    auto ok = [](const void *p) { return ((uintptr_t)p & 15u) == 0; };
    // every row that is loaded or stored in vectors: inputs and outputs
    const bool vec = (a.D / a.G) % E == 0 && a.ldu % E == 0 && a.ldd % E == 0 && ok(a.u) && ok(a.delta) && ok(a.dy) &&
                     ok(a.du) && ok(a.ddelta) && (!a.z || (a.ldz % E == 0 && ok(a.z) && ok(a.dz)));
    return vec ? bwd_run<TIn, N, true>(a, st) : bwd_run<TIn, N, false>(a, st);
}

// dh0 = dh_final (or zeros), parameter gradients zero: a call of no tokens.
__global__ void ssm_backward_empty_kernel(const SsmBwdArgs a)
{
    const size_t nh = (size_t)a.B * a.D * a.N, nA = (size_t)a.D * a.N, step = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < nh; i += step) {
        if (a.dh0) a.dh0[i] = a.dh_final ? a.dh_final[i] : 0.f;
        if (i < nA) a.dA[i] = 0.f;
        if (i < (size_t)a.D && a.dD) a.dD[i] = 0.f;
        if (i < (size_t)a.D && a.dbias) a.dbias[i] = 0.f;
    }
}

}  // namespace

size_t ssm_backward_workspace_bytes(int B, int T, int D, int N, int G)
{
    if (T == 0) return 0;
    Work w;
    return lay_out(bwd_plan(B, T, D, N, G), B, T, D, N, G, nullptr, &w) * sizeof(float);
}

cudaError_t launch_ssm_backward(const SsmBwdArgs &a, cudaStream_t st)
{
    if (a.T == 0) {
        const size_t blocks = std::min<size_t>(((size_t)a.B * a.D * a.N + 255) / 256, 1024);
        ssm_backward_empty_kernel<<<(unsigned)blocks, 256, 0, st>>>(a);
        return cudaGetLastError();
    }
    switch (a.N) {
    case 8: return a.dtype == LDN_F32 ? bwd_pick<float, 8>(a, st) : bwd_pick<__nv_bfloat16, 8>(a, st);
    case 16: return a.dtype == LDN_F32 ? bwd_pick<float, 16>(a, st) : bwd_pick<__nv_bfloat16, 16>(a, st);
    case 32: return a.dtype == LDN_F32 ? bwd_pick<float, 32>(a, st) : bwd_pick<__nv_bfloat16, 32>(a, st);
    case 64: return a.dtype == LDN_F32 ? bwd_pick<float, 64>(a, st) : bwd_pick<__nv_bfloat16, 64>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ldn
