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
// again into registers and the gradients follow.  A lane owns KC channels x 4 states, so the
// channel sums of dB and dC start in registers; the rest goes by halving exchanges, over the
// lanes of a channel for q, sum A w and sum C h (four tokens together), over the channels of a
// warp for dB and dC.  About 16 fp32 operations and two exponentials for every state: the
// kernel is bound by the fp32 pipe.
//
// Sums across blocks (dB, dC over the channel blocks of a group; dA, dD and the bias over
// sequences and segments) go to the workspace and are added by a last launch in a fixed
// order: no atomics, the same bits on every call.  Few channels: the tokens are cut into
// segments; a first launch forms every segment's carry from zero (g alone, one exponential)
// and a block composes what reaches its end from the later ones.
#include "ssm_common.cuh"

namespace ldn {
namespace {
using namespace ssm;

constexpr int kThreads = 128, kWarps = 4, S = 4, KC = 2, SUB = 4;

template <int N> constexpr int block_ch() { return kThreads / (N / S) * KC; }
int block_channels(int N) { return kThreads / (N / S) * KC; }

struct Plan {
    int n, len;      // segments per sequence, tokens of one (a multiple of TT)
    int gblocks;     // channel blocks per group
};

struct Work {
    float *bc;       // [gblocks][B * T][G][2][N]
    float *A;        // [B * n][D][N]
    float *D, *bias; // [B * n][D]
    float *carry;    // [B * n][D][N]
    float *sums;     // [B * n][D]
};

template <typename TIn, int N>
struct Smem {
    static constexpr int DB = block_ch<N>();
    // copies of the next tile in flight (bf16 rows; fp32 rows are read where they are used)
    __nv_bfloat16 raw[sizeof(TIn) == 2 ? 4 : 1][sizeof(TIn) == 2 ? TT * DB : 8];
    float4 step[TT][DB];                     // dt, dt u, yb, -; then dt, q, sum C h, sum A2 w
    float B[TT * N], C[TT * N];
    float4 ckpt[TT / SUB][KC][kThreads];     // the state entering every SUB tokens
    float red[kWarps][TT][2 * N];            // dB, dC summed over a warp's channels
    float bias[DB], skip[DB];
};

// e^x parts of a channel and token
struct Gate { float y, dy; };   // silu(z), silu'(z)
__device__ __forceinline__ Gate gate_of(float z)
{
    const float s = sigmoid_fast(z);
    return {z * s, s * fmaf(z, 1.f - s, 1.f)};
}

enum { kCarry = 0, kMain = 1 };

template <typename TIn, int N, bool VEC, int PHASE>
__global__ void __launch_bounds__(kThreads, 2)
ssm_backward_kernel(const SsmBwdArgs a, const Plan pl, const Work wk)
{
    constexpr int L = N / S, SL = kThreads / L, DB = SL * KC;
    constexpr bool STAGED = VEC && sizeof(TIn) == 2;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    using Sm = Smem<TIn, N>;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    const int Dg = a.D / a.G;
    const unsigned cblocks = (unsigned)pl.gblocks * a.G;
    const unsigned cb = blockIdx.x % cblocks, bs = blockIdx.x / cblocks;
    const int seg = (int)(bs % pl.n), b = (int)(bs / pl.n);
    const int grp = (int)(cb / pl.gblocks), gb = (int)(cb % pl.gblocks), cg = gb * DB;
    const int c0 = grp * Dg + cg, cols = min(DB, Dg - cg);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = tid % L, slot = tid / L;
    const int len = seq_len(a.lens, b, a.T);
    const int tb = seg * pl.len, te = min(tb + pl.len, a.T);
    const size_t row0 = (size_t)b * a.T;
    const TIn *u = (const TIn *)a.u + row0 * a.ldu + c0;
    const TIn *dl = (const TIn *)a.delta + row0 * a.ldd + c0;
    const TIn *z = a.z ? (const TIn *)a.z + row0 * a.ldz + c0 : nullptr;
    const TIn *dy = (const TIn *)a.dy + row0 * a.D + c0;
    const TIn *Bm = (const TIn *)a.Bm + row0 * a.ldb + (size_t)grp * N;
    const TIn *Cm = (const TIn *)a.Cm + row0 * a.ldc + (size_t)grp * N;

    for (int i = tid; i < DB; i += kThreads) {
        sm.bias[i] = a.bias && i < cols ? a.bias[c0 + i] : 0.f;
        sm.skip[i] = a.Dskip && i < cols ? a.Dskip[c0 + i] : 0.f;
    }
    float2 A2[KC][2], g[KC][2], dA[KC][2];
    float sumdt[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int ch = slot + k * SL;
        const bool on = ch < cols;
        const size_t at = (size_t)(c0 + ch) * N + l * S;
        sumdt[k] = 0.f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            A2[k][s] = on ? make_float2(a.A[at + 2 * s] * kLog2e, a.A[at + 2 * s + 1] * kLog2e) : dup(0.f);
            g[k][s] = dA[k][s] = dup(0.f);
            if (PHASE == kMain && on && a.dh_final) {
                const float *p = a.dh_final + (size_t)b * a.D * N + at + 2 * s;
                g[k][s] = make_float2(p[0], p[1]);
            }
        }
        if (PHASE == kMain && on)
            for (int j = pl.n - 1; j > seg; --j) {   // through the later segments
                const size_t e = ((size_t)b * pl.n + j) * a.D + c0 + ch;
                const float sd = wk.sums[e];
                const float *p = wk.carry + e * N + l * S;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    g[k][s] = __ffma2_rn(ex2(__fmul2_rn(A2[k][s], dup(sd))), g[k][s],
                                         make_float2(p[2 * s], p[2 * s + 1]));
            }
    }

    auto rows_of = [&](int t0) { return min(max(min(len, te) - t0, 0), TT); };
    auto fetch = [&](int t0) {
        if constexpr (STAGED) {
            const int rows = rows_of(t0);
            TIn(*raw)[TT * DB] = reinterpret_cast<TIn(*)[TT * DB]>(sm.raw);
            if (PHASE == kMain) load_rows<TIn, DB, DB, kThreads, true>(raw[0], u + (size_t)t0 * a.ldu, a.ldu, rows, cols);
            load_rows<TIn, DB, DB, kThreads, true>(raw[1], dl + (size_t)t0 * a.ldd, a.ldd, rows, cols);
            load_rows<TIn, DB, DB, kThreads, true>(raw[2], dy + (size_t)t0 * a.D, a.D, rows, cols);
            if (z) load_rows<TIn, DB, DB, kThreads, true>(raw[3], z + (size_t)t0 * a.ldz, a.ldz, rows, cols);
            cp_async_commit();
        }
    };
    // two neighbouring channels of a row, zeros outside
    auto pair = [&](const TIn *p, long long ld, int t0, int r, int c, bool live, float *v) {
        load_n<2, false>(p + (size_t)(t0 + r) * ld + c, v, live ? cols - c : 0);
    };
    constexpr int PER = DB / 2;
    static_assert(kThreads % PER == 0, "a thread keeps its channels in every pass over a tile");
    const int pc = (tid % PER) * 2;
    float accD[2] = {0.f, 0.f}, accb[2] = {0.f, 0.f};

    RowRegs<TIn, N, kThreads> rB, rC;
    const int vB = rB.alignment(Bm, a.ldb), vC = rC.alignment(Cm, a.ldc);
    const int last = tb + (te - 1 - tb) / TT * TT;   // the segment's last tile
    fetch(last);
    if (PHASE == kMain) rB.load(Bm + (size_t)last * a.ldb, a.ldb, rows_of(last), vB);
    rC.load(Cm + (size_t)last * a.ldc, a.ldc, rows_of(last), vC);
    for (int t0 = last; t0 >= tb; t0 -= TT) {
        const int rows = rows_of(t0);
        float4 h0[KC];
        if (PHASE == kMain) {
            const size_t ck = (size_t)b * ((a.T + TT - 1) / TT) + t0 / TT;
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int ch = slot + k * SL;
                h0[k] = ch < cols ? *reinterpret_cast<const float4 *>(a.states + (ck * a.D + c0 + ch) * N + l * S)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        if constexpr (STAGED) cp_async_wait<0>();
        __syncthreads();   // this tile has arrived; the last tile's readers are done
        if (PHASE == kMain) rB.store(sm.B, Bm + (size_t)t0 * a.ldb, a.ldb, rows, vB);
        rC.store(sm.C, Cm + (size_t)t0 * a.ldc, a.ldc, rows, vC);
        for (int i = tid; i < TT * PER; i += kThreads) {
            const int r = i / PER;
            const bool live = r < rows;
            float vu[2] = {0.f, 0.f}, vd[2], vy[2], vz[2];
            if constexpr (STAGED) {
                const TIn(*raw)[TT * DB] = reinterpret_cast<const TIn(*)[TT * DB]>(sm.raw);
                const int o = r * DB + pc;
                if (PHASE == kMain) load_n<2, false>(&raw[0][o], vu);
                load_n<2, false>(&raw[1][o], vd);
                load_n<2, false>(&raw[2][o], vy);
                if (z) load_n<2, false>(&raw[3][o], vz);
            } else {
                if (PHASE == kMain) pair(u, a.ldu, t0, r, pc, live, vu);
                pair(dl, a.ldd, t0, r, pc, live, vd);
                pair(dy, a.D, t0, r, pc, live, vy);
                if (z) pair(z, a.ldz, t0, r, pc, live, vz);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float dt = vd[k] + sm.bias[pc + k];
                if (a.softplus) dt = softplus_accurate(dt);
                if (!live) dt = 0.f;
                const float yb = z ? vy[k] * gate_of(vz[k]).y : vy[k];
                sm.step[r][pc + k] = make_float4(dt, live ? dt * vu[k] : 0.f, live ? yb : 0.f, 0.f);
            }
        }
        __syncthreads();
        if (t0 > tb) {
            fetch(t0 - TT);
            if (PHASE == kMain) rB.load(Bm + (size_t)(t0 - TT) * a.ldb, a.ldb, rows_of(t0 - TT), vB);
            rC.load(Cm + (size_t)(t0 - TT) * a.ldc, a.ldc, rows_of(t0 - TT), vC);
        }
        auto row4 = [&](const float *m, int r, float2 *v) {
            const float4 q = *reinterpret_cast<const float4 *>(&m[r * N + l * S]);
            v[0] = make_float2(q.x, q.y);
            v[1] = make_float2(q.z, q.w);
        };
        if constexpr (PHASE == kCarry) {
#pragma unroll 4
            for (int r = TT - 1; r >= 0; --r) {
                float2 Cv[2];
                row4(sm.C, r, Cv);
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    const float4 q = sm.step[r][slot + k * SL];
                    sumdt[k] += q.x;
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        g[k][s] = __fmul2_rn(ex2(__fmul2_rn(A2[k][s], dup(q.x))), __ffma2_rn(Cv[s], dup(q.z), g[k][s]));
                }
            }
        } else {
            float2 h[KC][2];
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                h[k][0] = make_float2(h0[k].x, h0[k].y);
                h[k][1] = make_float2(h0[k].z, h0[k].w);
            }
#pragma unroll 1
            for (int sub = 0; sub < TT / SUB; ++sub) {
#pragma unroll
                for (int k = 0; k < KC; ++k)
                    sm.ckpt[sub][k][tid] = make_float4(h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y);
                if (sub == TT / SUB - 1) break;
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
                    const int r = sub * SUB + j;
                    float2 Bv[2];
                    row4(sm.B, r, Bv);
#pragma unroll
                    for (int k = 0; k < KC; ++k) {
                        const float4 q = sm.step[r][slot + k * SL];
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            h[k][s] = __ffma2_rn(ex2(__fmul2_rn(A2[k][s], dup(q.x))), h[k][s],
                                                 __fmul2_rn(dup(q.y), Bv[s]));
                    }
                }
            }
#pragma unroll 1
            for (int sub = TT / SUB - 1; sub >= 0; --sub) {
                float2 hh[SUB + 1][KC][2], av[SUB][KC][2];   // states before each token, decays
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    const float4 q = sm.ckpt[sub][k][tid];
                    hh[0][k][0] = make_float2(q.x, q.y);
                    hh[0][k][1] = make_float2(q.z, q.w);
                }
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
                    const int r = sub * SUB + j;
                    float2 Bv[2];
                    row4(sm.B, r, Bv);
#pragma unroll
                    for (int k = 0; k < KC; ++k) {
                        const float4 q = sm.step[r][slot + k * SL];
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            av[j][k][s] = ex2(__fmul2_rn(A2[k][s], dup(q.x)));
                            hh[j + 1][k][s] = __ffma2_rn(av[j][k][s], hh[j][k][s], __fmul2_rn(dup(q.y), Bv[s]));
                        }
                    }
                }
                float qs[SUB * KC], ws[SUB * KC], ps[SUB * KC];
#pragma unroll
                for (int j = SUB - 1; j >= 0; --j) {
                    const int r = sub * SUB + j;
                    float2 Bv[2], Cv[2], dB[2], dC[2];
                    row4(sm.B, r, Bv);
                    row4(sm.C, r, Cv);
#pragma unroll
                    for (int k = 0; k < KC; ++k) {
                        const float4 q = sm.step[r][slot + k * SL];
                        float2 aq, aw, ap;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const float2 ht = hh[j + 1][k][s];
                            g[k][s] = __ffma2_rn(Cv[s], dup(q.z), g[k][s]);
                            dB[s] = k ? __ffma2_rn(g[k][s], dup(q.y), dB[s]) : __fmul2_rn(g[k][s], dup(q.y));
                            dC[s] = k ? __ffma2_rn(ht, dup(q.z), dC[s]) : __fmul2_rn(ht, dup(q.z));
                            aq = s ? __ffma2_rn(g[k][s], Bv[s], aq) : __fmul2_rn(g[k][s], Bv[s]);
                            ap = s ? __ffma2_rn(ht, Cv[s], ap) : __fmul2_rn(ht, Cv[s]);
                            g[k][s] = __fmul2_rn(g[k][s], av[j][k][s]);
                            const float2 w = __fmul2_rn(g[k][s], hh[j][k][s]);
                            aw = s ? __ffma2_rn(A2[k][s], w, aw) : __fmul2_rn(A2[k][s], w);
                            dA[k][s] = __ffma2_rn(w, dup(q.x), dA[k][s]);
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
                        const int idx = (l / DUP) * HELD + i;
                        float4 &o = sm.step[sub * SUB + idx / KC][slot + (idx % KC) * SL];
                        o.y = qs[i];
                        o.z = ps[i];
                        o.w = ws[i];
                    }
            }
            __syncthreads();
            // the tile's rows: du, ddelta, dz
            const int live_rows = min(te - t0, TT);
            TIn *du = (TIn *)a.du + (row0 + t0) * a.D + c0, *dd = (TIn *)a.ddelta + (row0 + t0) * a.D + c0;
            TIn *dz = a.dz ? (TIn *)a.dz + (row0 + t0) * a.D + c0 : nullptr;
            for (int i = tid; i < TT * PER; i += kThreads) {
                const int r = i / PER;
                if (r >= live_rows || pc >= cols) continue;
                const bool live = r < rows;
                float vu[2], vd[2], vy[2], vz[2], ou[2], od[2], oz[2];
                pair(u, a.ldu, t0, r, pc, live, vu);
                pair(dl, a.ldd, t0, r, pc, live, vd);
                pair(dy, a.D, t0, r, pc, live, vy);
                if (z) pair(z, a.ldz, t0, r, pc, live, vz);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 q = sm.step[r][pc + k];
                    float yb = vy[k];
                    oz[k] = 0.f;
                    if (z) {
                        const Gate gt = gate_of(vz[k]);
                        oz[k] = vy[k] * gt.dy * fmaf(sm.skip[pc + k], vu[k], q.z);
                        yb = vy[k] * gt.y;
                    }
                    ou[k] = fmaf(q.x, q.y, sm.skip[pc + k] * yb);
                    od[k] = fmaf(kLn2, q.w, vu[k] * q.y);
                    if (a.softplus) od[k] *= sigmoid_fast(vd[k] + sm.bias[pc + k]);
                    if (!live) ou[k] = od[k] = oz[k] = yb = 0.f;
                    accD[k] = fmaf(yb, vu[k], accD[k]);
                    accb[k] += od[k];
                }
                store_n<2, false>(du + (size_t)r * a.D + pc, ou, cols - pc);
                store_n<2, false>(dd + (size_t)r * a.D + pc, od, cols - pc);
                if (z) store_n<2, false>(dz + (size_t)r * a.D + pc, oz, cols - pc);
            }
            float *bc = wk.bc + (((size_t)gb * a.B * a.T + row0 + t0) * a.G + grp) * (2 * N);
            for (int i = tid; i < live_rows * 2 * N; i += kThreads) {
                const int r = i / (2 * N), n = i % (2 * N);
                float t = sm.red[0][r][n];
#pragma unroll
                for (int k = 1; k < kWarps; ++k) t += sm.red[k][r][n];
                bc[(size_t)r * a.G * (2 * N) + n] = t;
            }
        }
    }

    const size_t bseg = (size_t)b * pl.n + seg;
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int ch = slot + k * SL;
        if (ch >= cols) continue;
        const size_t e = bseg * a.D + c0 + ch;
        const float4 gv = make_float4(g[k][0].x, g[k][0].y, g[k][1].x, g[k][1].y);
        if (PHASE == kCarry) {
            *reinterpret_cast<float4 *>(wk.carry + e * N + l * S) = gv;
            if (l == 0) wk.sums[e] = sumdt[k];
        } else {
            *reinterpret_cast<float4 *>(wk.A + e * N + l * S) =
                make_float4(dA[k][0].x, dA[k][0].y, dA[k][1].x, dA[k][1].y);
            if (seg == 0 && a.dh0)
                *reinterpret_cast<float4 *>(a.dh0 + ((size_t)b * a.D + c0 + ch) * N + l * S) = gv;
        }
    }
    if constexpr (PHASE == kMain) {   // dD and the bias: over the threads that share a channel pair
        __syncthreads();
        float4 *t4 = reinterpret_cast<float4 *>(sm.red);
        t4[tid] = make_float4(accD[0], accD[1], accb[0], accb[1]);
        __syncthreads();
        if (tid < PER) {
            float4 t = t4[tid];
#pragma unroll
            for (int i = 1; i < kThreads / PER; ++i) {
                const float4 q = t4[tid + i * PER];
                t.x += q.x; t.y += q.y; t.z += q.z; t.w += q.w;
            }
            const size_t e = bseg * a.D + c0 + pc;
            if (pc < cols) { wk.D[e] = t.x; wk.bias[e] = t.z; }
            if (pc + 1 < cols) { wk.D[e + 1] = t.y; wk.bias[e + 1] = t.w; }
        }
    }
}

// The sums across blocks, each by one thread in order: dB, dC over the channel blocks of a
// group; dA, dD and the bias over sequences and segments (np of them).
template <typename TIn>
__global__ void __launch_bounds__(256)
ssm_sum_kernel(const SsmBwdArgs a, const Work wk, int gblocks, int np, unsigned bc_blocks)
{
    const int N = a.N;
    if (blockIdx.x < bc_blocks) {
        const size_t n = (size_t)a.B * a.T * a.G * 2 * N, i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
        if (i >= n) return;
        float4 t = *reinterpret_cast<const float4 *>(wk.bc + i);
        for (int k = 1; k < gblocks; ++k) {
            const float4 q = *reinterpret_cast<const float4 *>(wk.bc + (size_t)k * n + i);
            t.x += q.x; t.y += q.y; t.z += q.z; t.w += q.w;
        }
        const size_t row = i / (2 * N);
        const int c = (int)(i % (2 * N));
        TIn *o = (c < N ? (TIn *)a.dB : (TIn *)a.dC) + row * N + (c < N ? c : c - N);
        const float v[4] = {t.x, t.y, t.z, t.w};
        store_n<4, false>(o, v);
        return;
    }
    const size_t i = (size_t)(blockIdx.x - bc_blocks) * 256 + threadIdx.x, nA = (size_t)a.D * N;
    const float *src;
    float *dst;
    size_t per, o;
    if (i < nA) { src = wk.A; dst = a.dA; per = nA; o = i; }
    else if (i < nA + a.D) { src = wk.D; dst = a.dD; per = a.D; o = i - nA; }
    else if (i < nA + 2 * (size_t)a.D) { src = wk.bias; dst = a.dbias; per = a.D; o = i - nA - a.D; }
    else return;
    if (!dst) return;
    float t = 0.f;
    for (int k = 0; k < np; ++k) t += src[k * per + o];
    dst[o] = t;
}

constexpr int kSms = 152;

Plan bwd_plan(int B, int T, int D, int N, int G)
{
    const int db = block_channels(N), gblocks = (D / G + db - 1) / db;
    const long long blocks = (long long)B * G * gblocks, want = kSms * 2 * 3;   // two blocks an SM, three waves
    int n = (int)std::min<long long>((want + blocks - 1) / blocks, std::max(1, T / 64));
    n = std::max(1, std::min(n, 64));
    const int len = std::max(TT, (int)((((long long)T + n - 1) / n + TT - 1) / TT) * TT);
    return {std::max(1, (T + len - 1) / len), len, gblocks};
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
    w->carry = take(p.n > 1 ? np * D * N : 0);
    w->sums = take(p.n > 1 ? np * D : 0);
    return at;
}

template <typename TIn, int N, bool VEC, int PHASE>
cudaError_t bwd_launch(const SsmBwdArgs &a, const Plan &p, const Work &w, cudaStream_t st)
{
    constexpr int bytes = (int)sizeof(Smem<TIn, N>);
    auto *k = ssm_backward_kernel<TIn, N, VEC, PHASE>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k<<<(unsigned)((long long)p.gblocks * a.G * a.B * p.n), kThreads, bytes, st>>>(a, p, w);
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
    const cudaError_t e = bwd_launch<TIn, N, VEC, kMain>(a, p, w, st);
    if (e != cudaSuccess) return e;
    const unsigned bcb = (unsigned)(((size_t)a.B * a.T * a.G * 2 * N / 4 + 255) / 256);
    const unsigned pb = (unsigned)(((size_t)a.D * (N + 2) + 255) / 256);
    ssm_sum_kernel<TIn><<<bcb + pb, 256, 0, st>>>(a, w, p.gblocks, a.B * p.n, bcb);
    return cudaGetLastError();
}

template <typename TIn, int N>
cudaError_t bwd_pick(const SsmBwdArgs &a, cudaStream_t st)
{
    constexpr int E = 16 / sizeof(TIn);
    auto ok = [](const void *p) { return ((uintptr_t)p & 15u) == 0; };
    const bool vec = (a.D / a.G) % E == 0 && a.ldu % E == 0 && a.ldd % E == 0 && ok(a.u) && ok(a.delta) && ok(a.dy) &&
                     (!a.z || (a.ldz % E == 0 && ok(a.z)));
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
        ssm_backward_empty_kernel<<<(unsigned)std::min<size_t>(((size_t)a.B * a.D * a.N + 255) / 256, 1024), 256, 0, st>>>(a);
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
