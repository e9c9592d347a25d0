// Selective state space scan, forward over sequences and one token.
//
// Channel d, state n, token t:
//   dt = softplus(delta + bias) (or delta + bias),  a = e^{dt A},
//   h_t = a h_{t-1} + dt u_t B_t,   y_t = (sum_n C_t h_t + D u_t) silu(z_t).
//
// One update costs four fp32 operations (dt A, dt u B, a h + ., C h + .) and one exponential
// for every state of every channel and token: at N = 16 that outweighs the eight bytes a
// channel and token of traffic.  Per SM and cycle the GPU makes 128 fp32 results and 32
// exponentials (measured), so 32 updates: 54 us for 4 x 2048 tokens of 4096 x 16 at 2,060 MHz,
// against 40 us for their bytes.  What stands above that is everything else an update needs in
// registers -- each register written, by arithmetic or by a load, takes its turn at the register
// file, and at five results an update the operands' loads add two: a loop of the update alone, eight
// warps an SM as here, runs at 7.8 to 8.0 cycles an update and scheduler (7.3 to 7.5 with sixteen),
// which is 125 us on the SMs that hold two blocks -- and the elementwise work, the exchanges and the
// barriers, which are the other 59 us.
//
// L = N / S neighbouring lanes own one channel, S states each, in registers over the whole run;
// exponentials take e^x = 2^{x log2 e} with log2 e folded into A; products are packed pairs.
// A block is four warps of this recurrence and four helpers, a tile of 32 tokens the step: the
// helpers copy rows two tiles ahead (16-byte asynchronous copies), form dt and dt u a tile ahead,
// and add D u, apply the output gate and store a tile behind, while the recurrence reads its
// steps and the B, C rows (shared by all channels) from shared memory.  Each of the two has too
// few warps to cover its own latencies (one to two a scheduler at 4 x 4096 channels), so they
// cover each other's: 184 us, against 330 us for the same work one after another in one kind of
// warp.  One barrier a tile.  The sum over a channel's lanes is taken for 2 L tokens together (a
// halving exchange).
//
// Few channels for the card: the tokens are cut into segments that run side by side.  A first
// launch forms each segment's end state from zero and its sum of dt; in the second a segment
// composes what enters it, h <- e^{A sum dt} h + end, over the segments before it, and runs
// with its outputs.  The exponentials are then taken twice, so it is done only where whole
// sequences leave the card under-occupied (ssm_plan: 32768 tokens of 2048 x 16 in 556 us, 1737
// unsplit at the rate of 8192).
#include <type_traits>

#include "ssm_common.cuh"

namespace ldn {
namespace {
using namespace ssm;

enum { kWhole = 0, kEnds = 1, kFromEnds = 2 };

constexpr int kMain = 128, kThreads = 256;   // threads of the recurrence, of a block

// States of a lane, and the channels of a block.
constexpr int lane_states(int N) { return N == 8 ? 4 : 8; }
constexpr int block_channels(int N) { return kMain / (N / lane_states(N)); }

// Tiles are kept by warp, [warp][token][channel of the warp]: only B and C are shared.
template <typename TIn, int N>
struct Smem {
    static constexpr int WC = 32 / (N / lane_states(N)), WT = TT * WC;   // channels, elements of a warp
    static constexpr int ROW = WC + 2;   // a row of step: two pairs more, so that rows differ in banks
    TIn u[3][kMain / 32][WT], z[3][kMain / 32][WT], d[kMain / 32][WT];
    TIn rawB[TT * N], rawC[TT * N];
    // two rows more than a tile: the last tokens' loads run ahead into them, and go unused
    float B[2][(TT + 2) * N], C[2][(TT + 2) * N];
    float2 step[2][kMain / 32][(TT + 2) * ROW];   // dt, dt u; then a row's first WC floats the sums C h
};

struct Segs {
    int n, len;      // segments per sequence, tokens of one (a multiple of TT)
    float *ends;     // [B][n][D][N]
    float *sums;     // [B][n][D]
};

template <typename TIn, int N, bool VEC, int PHASE>
__global__ void __launch_bounds__(kThreads, 2)
ssm_scan_kernel(const SsmArgs a, const Segs sg, int gblocks)
{
    constexpr int S = lane_states(N), L = N / S, DB = block_channels(N);
    constexpr int TG = 2 * L;   // tokens of a group: two for every lane of a channel
    static_assert(TT % TG == 0, "whole groups");
    extern __shared__ __align__(16) unsigned char smem_raw[];
    using Sm = Smem<TIn, N>;
    constexpr int WC = Sm::WC, ROW = Sm::ROW;
    Sm &sm = *reinterpret_cast<Sm *>(smem_raw);
    const int Dg = a.D / a.G;
    const unsigned cblocks = (unsigned)gblocks * a.G;
    const unsigned cb = blockIdx.x % cblocks, bs = blockIdx.x / cblocks;
    const int segs = PHASE == kEnds ? sg.n - 1 : sg.n;   // nothing takes the last segment's end
    const int seg = (int)(bs % segs), b = (int)(bs / segs);
    const int grp = (int)(cb / gblocks), cg = (int)(cb % gblocks) * DB;
    const int c0 = grp * Dg + cg, cols = min(DB, Dg - cg);
    const bool helper = threadIdx.x >= kMain;
    const int tid = threadIdx.x % kMain, lane = tid & 31, warp = tid >> 5;
    const int len = seq_len(a.lens, b, a.T);
    const int tb = seg * sg.len, te = min(tb + sg.len, a.T);
    // tiles with rows of the sequence, and all of the segment's: behind the end the state stays
    const int tiles = (max(min(len, te) - tb, 0) + TT - 1) / TT, all = (te - tb + TT - 1) / TT;
    const size_t row0 = (size_t)b * a.T + tb;   // the segment's first row
    auto rows_of = [&](int it) { return min(max(min(len, te) - tb - it * TT, 0), TT); };

    if (helper) {
        // Copies, the elementwise work before the recurrence (prepare: dt, dt u) and after it
        // (finish: D u, the gate, the stores) for the channels of one recurrence warp, a tile
        // ahead of it and a tile behind it.  Vectors of PV and FV channels of a row; a lane's
        // channels stay the same.  FV channels are at most 16 bytes: VEC has groups of whole
        // 16-byte vectors, so that such a vector is inside its group or outside.
        constexpr int MOST = 16 / (int)sizeof(TIn);
        constexpr int PV = 4, FV = WC < MOST ? WC : MOST, PR = WC / PV, FR = WC / FV;
        const int w0 = warp * WC, wcols = cols - w0;   // the warp's channels
        const int pch = (lane % PR) * PV, fch = (lane % FR) * FV;
        const TIn *u = (const TIn *)a.u + row0 * a.ldu + c0 + w0;
        const TIn *dl = (const TIn *)a.delta + row0 * a.ldd + c0 + w0;
        const bool gated = a.z && PHASE != kEnds;
        const TIn *z = gated ? (const TIn *)a.z + row0 * a.ldz + c0 + w0 : nullptr;
        const TIn *Bm = (const TIn *)a.Bm + row0 * a.ldb + (size_t)grp * N;
        const TIn *Cm = (const TIn *)a.Cm + row0 * a.ldc + (size_t)grp * N;
        using Rows = SharedRows<TIn, N, kMain>;
        const int vB = Rows::alignment(Bm, a.ldb), vC = Rows::alignment(Cm, a.ldc);
        float2 bias[PV / 2], skip[FV / 2];
        load_n<PV, false>(a.bias + c0 + w0 + pch, reinterpret_cast<float *>(bias), a.bias ? wcols - pch : 0);
        load_n<FV, false>(a.Dskip + c0 + w0 + fch, reinterpret_cast<float *>(skip), a.Dskip ? wcols - fch : 0);

        // A tile whose rows and channels are all inside takes bodies without the tests.
        auto whole = [&](int it) { return rows_of(it) == TT && wcols >= WC; };
        auto copy = [&](int it, auto full) {
            constexpr bool F = decltype(full)::value;
            const int rows = rows_of(it), t = it * TT;
            warp_rows<TIn, WC, VEC, F>(sm.u[it % 3][warp], u + (size_t)t * a.ldu, a.ldu, rows, wcols);
            warp_rows<TIn, WC, VEC, F>(sm.d[warp], dl + (size_t)t * a.ldd, a.ldd, rows, wcols);
            if (gated) warp_rows<TIn, WC, VEC, F>(sm.z[it % 3][warp], z + (size_t)t * a.ldz, a.ldz, rows, wcols);
        };
        auto fetch = [&](int it) {
            const int rows = rows_of(it), t = it * TT;
            if (whole(it)) copy(it, std::true_type{});
            else copy(it, std::false_type{});
            Rows::fetch(sm.rawB, Bm + (size_t)t * a.ldb, a.ldb, rows, vB, tid);
            if (PHASE != kEnds) Rows::fetch(sm.rawC, Cm + (size_t)t * a.ldc, a.ldc, rows, vC, tid);
            cp_async_commit();
        };
        auto prepare = [&](int it, auto soft, auto full) {
            const int rows = rows_of(it);
            const TIn *td = sm.d[warp], *tu = sm.u[it % 3][warp];
#pragma unroll
            for (int k = 0; k < TT * PR / 32; ++k) {
                const int i = k * 32 + lane, r = i / PR;
                float2 v[PV / 2], w[PV / 2];
                load_n<PV, true>(td + i * PV, reinterpret_cast<float *>(v));
                load_n<PV, true>(tu + i * PV, reinterpret_cast<float *>(w));
                float4 *o = reinterpret_cast<float4 *>(sm.step[it & 1][warp] + r * ROW + pch);
#pragma unroll
                for (int c = 0; c < PV / 2; ++c) {
                    float2 dt = __fadd2_rn(v[c], bias[c]);
                    if (soft) dt = softplus_accurate(dt);
                    if (!full && r >= rows) dt = dup(0.f);   // a row past the end steps by zero: a = 1, no input
                    const float2 du = __fmul2_rn(dt, w[c]);
                    o[c] = make_float4(dt.x, du.x, dt.y, du.y);
                }
            }
        };
        auto ready = [&](int it) {   // tile `it` for the recurrence
            cp_async_wait<0>();
            const int rows = rows_of(it), t = it * TT;
            Rows::widen(sm.B[it & 1], sm.rawB, Bm + (size_t)t * a.ldb, a.ldb, rows, vB, tid);
            if (PHASE != kEnds) Rows::widen(sm.C[it & 1], sm.rawC, Cm + (size_t)t * a.ldc, a.ldc, rows, vC, tid);
            __syncwarp();
            if (!a.softplus) prepare(it, std::false_type{}, std::false_type{});
            else if (whole(it)) prepare(it, std::true_type{}, std::true_type{});
            else prepare(it, std::true_type{}, std::false_type{});
            __syncwarp();
        };
        auto finish = [&](int it, auto gate, auto full) {
            const int rows = rows_of(it), live = min(te - tb - it * TT, TT);
            const TIn *tu = sm.u[it % 3][warp], *tz = sm.z[it % 3][warp];
            const float *sums = reinterpret_cast<const float *>(sm.step[it & 1][warp]);
            TIn *y = (TIn *)a.y + (row0 + it * TT) * a.D + c0 + w0 + fch;
#pragma unroll
            for (int k = 0; k < TT * FR / 32; ++k) {
                const int i = k * 32 + lane, r = i / FR;
                float2 uu[FV / 2], zz[FV / 2], v[FV / 2];
                load_n<FV, true>(tu + i * FV, reinterpret_cast<float *>(uu));
                if (gate) load_n<FV, true>(tz + i * FV, reinterpret_cast<float *>(zz));
                load_n<FV, true>(sums + r * 2 * ROW + fch, reinterpret_cast<float *>(v));
#pragma unroll
                for (int c = 0; c < FV / 2; ++c) {
                    v[c] = __ffma2_rn(skip[c], uu[c], v[c]);
                    if (gate) v[c] = __fmul2_rn(v[c], silu_fast(zz[c]));
                    if (!full && r >= rows) v[c] = dup(0.f);   // a row past the sequence's end
                }
                if (full || r < live)
                    store_n<FV, VEC>(y + (size_t)r * a.D, reinterpret_cast<float *>(v), full ? FV : wcols - fch);
            }
            __syncwarp();
        };
        auto finished = [&](int it) {
            if constexpr (PHASE != kEnds) {
                if (!gated) finish(it, std::false_type{}, std::false_type{});
                else if (whole(it)) finish(it, std::true_type{}, std::true_type{});
                else finish(it, std::true_type{}, std::false_type{});
            }
        };
        if (tiles > 0) {
            fetch(0);
            ready(0);
            if (tiles > 1) fetch(1);
        }
        __syncthreads();
        for (int it = 0; it < tiles; ++it) {
            if (it > 0) finished(it - 1);
            if (it + 1 < tiles) ready(it + 1);
            if (it + 2 < tiles) fetch(it + 2);
            __syncthreads();
        }
        if (tiles > 0) finished(tiles - 1);
        if constexpr (PHASE != kEnds) {   // rows of the tiles behind the end
            // (64 bits: vectors of an unsplit sequence may outnumber an int)
            const float zeros[FV] = {};
            for (long long i = (long long)tiles * TT * FR + lane; i < (long long)(te - tb) * FR; i += 32)
                store_n<FV, VEC>((TIn *)a.y + (row0 + i / FR) * a.D + c0 + w0 + fch, zeros, wcols - fch);
        }
        return;
    }

    // The recurrence: lane l of a channel's L has states l S .. l S + S - 1.
    const int l = tid % L, slot = tid / L;
    const bool on = slot < cols;
    const size_t mine = (size_t)(c0 + slot) * N + l * S;
    float A2[S], h[S], sumdt = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        A2[s] = on ? rate(a.A[mine + s]) : 0.f;
        h[s] = PHASE != kEnds && on && a.h0 ? a.h0[(size_t)b * a.D * N + mine + s] : 0.f;
    }
    if (PHASE == kFromEnds && on)
#pragma unroll 4
        for (int j = 0; j < seg; ++j) {
            const size_t e = ((size_t)b * sg.n + j) * a.D + c0 + slot;
            const float sd = sg.sums[e];
            const float *p = sg.ends + e * N + l * S;
#pragma unroll
            for (int s = 0; s < S; ++s) h[s] = fmaf(decay(A2[s], sd), h[s], p[s]);
        }
    auto store_state = [&](float *p) {
#pragma unroll
        for (int s = 0; s < S; s += 4)
            *reinterpret_cast<float4 *>(p + s) = make_float4(h[s], h[s + 1], h[s + 2], h[s + 3]);
    };
    __syncthreads();
    for (int it = 0; it < tiles; ++it) {
        if (PHASE != kEnds && a.states && on)   // the state entering this tile
            store_state(a.states + ((size_t)b * ((a.T + TT - 1) / TT) + tb / TT + it) * a.D * N + mine);
        // Operands are loaded two tokens ahead and decays formed one token ahead, in the
        // source: a warp that loads and uses in one token waits for both latencies every token
        // (17 against 9 cycles an update with one warp a scheduler).
        float2 *step = sm.step[it & 1][warp];
        const float2 *sp = step + slot % WC;
        const float *Br = sm.B[it & 1] + l * S, *Cr = sm.C[it & 1] + l * S;
        float2 q[3];
        float bv[3][S], cv[3][S], e[2][S];
        auto load = [&](int t, int i) {
            q[i] = sp[t * ROW];
#pragma unroll
            for (int s = 0; s < S; s += 4) {
                *reinterpret_cast<float4 *>(&bv[i][s]) = *reinterpret_cast<const float4 *>(Br + t * N + s);
                if (PHASE != kEnds)
                    *reinterpret_cast<float4 *>(&cv[i][s]) = *reinterpret_cast<const float4 *>(Cr + t * N + s);
            }
        };
        auto decays = [&](int i, float *d) {
#pragma unroll
            for (int s = 0; s < S; s += 2) {
                const float2 x = decay(make_float2(A2[s], A2[s + 1]), q[i].x);
                d[s] = x.x;
                d[s + 1] = x.y;
            }
        };
        load(0, 0);
        load(1, 1);
        decays(0, e[0]);
        constexpr int UG = TG >= 4 ? 1 : 4 / TG;   // groups in one body: at least four tokens
#pragma unroll UG
        for (int tq = 0; tq < TT; tq += TG) {
            float yv[TG];
#pragma unroll
            for (int j = 0; j < TG; ++j) {
                load(tq + j + 2, 2);
                decays(1, e[1]);
                if (PHASE == kEnds) sumdt += q[0].x;
                float y0 = 0.f, y1 = 0.f;
#pragma unroll
                for (int s = 0; s < S; s += 2) {
                    const float2 in = __fmul2_rn(make_float2(bv[0][s], bv[0][s + 1]), dup(q[0].y));
                    const float2 x = __ffma2_rn(make_float2(e[0][s], e[0][s + 1]), make_float2(h[s], h[s + 1]), in);
                    h[s] = x.x;
                    h[s + 1] = x.y;
                    if (PHASE != kEnds) {
                        y0 = fmaf(cv[0][s], x.x, y0);
                        y1 = fmaf(cv[0][s + 1], x.y, y1);
                    }
                }
                yv[j] = y0 + y1;
                q[0] = q[1];
                q[1] = q[2];
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    e[0][s] = e[1][s];
                    bv[0][s] = bv[1][s]; bv[1][s] = bv[2][s];
                    cv[0][s] = cv[1][s]; cv[1][s] = cv[2][s];
                }
            }
            if constexpr (PHASE != kEnds) {
                // a lane gets the sums of two tokens, and writes them over steps that every lane
                // of the warp has read
                reduce_halving<TG, L / 2, 1>(yv, lane);
                __syncwarp();
                float *o = reinterpret_cast<float *>(step + (tq + 2 * l) * ROW) + slot % WC;
                o[0] = yv[0];
                o[2 * ROW] = yv[1];
            }
        }
        __syncthreads();
    }
    if (!on) return;
    if (PHASE != kEnds && a.states)
        for (int it = tiles; it < all; ++it)
            store_state(a.states + ((size_t)b * ((a.T + TT - 1) / TT) + tb / TT + it) * a.D * N + mine);
    if (PHASE == kEnds) {
        const size_t e = ((size_t)b * sg.n + seg) * a.D + c0 + slot;
        store_state(sg.ends + e * N + l * S);
        if (l == 0) sg.sums[e] = sumdt;
    } else if (seg == sg.n - 1 && a.h_final) {
        store_state(a.h_final + (size_t)b * a.D * N + mine);
    }
}

// One token for every sequence: a lane takes four states of one channel, the channel's lanes
// sum; h is read and written once, which is nearly all of the traffic.  A lane goes through
// kStepB sequences at once: their loads are in flight together, and A is read once for them
// (64 x 4096 x 16: 10.2 us; one sequence a lane 12.5, four 11.4, eight 14.7).
constexpr int kStepB = 2;

template <typename TIn, int N, bool VEC>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmArgs a)
{
    constexpr int L = N / 4;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x, unit = id / L;
    const int l = (int)(id % L);
    const long long groups = (a.B + kStepB - 1) / kStepB;
    const bool on = unit < groups * a.D;
    const int d = on ? (int)(unit % a.D) : 0, g = d / (a.D / a.G), b0 = on ? (int)(unit / a.D) * kStepB : 0;
    float Av[4], h[kStepB][4], Bv[kStepB][4], Cv[kStepB][4], u[kStepB], dt[kStepB], z[kStepB], y[kStepB];
    load_n<4, VEC>(a.A + (size_t)d * N + l * 4, Av);
    const float bias = a.bias ? a.bias[d] : 0.f, skip = a.Dskip ? a.Dskip[d] : 0.f;
#pragma unroll
    for (int k = 0; k < kStepB; ++k) {
        const int b = min(b0 + k, a.B - 1);   // past the last: that one again, not stored
        load_n<4, true>(a.h0 + ((size_t)b * a.D + d) * N + l * 4, h[k]);
        load_n<4, VEC>((const TIn *)a.Bm + (size_t)b * a.ldb + (size_t)g * N + l * 4, Bv[k]);
        load_n<4, VEC>((const TIn *)a.Cm + (size_t)b * a.ldc + (size_t)g * N + l * 4, Cv[k]);
        u[k] = load_in((const TIn *)a.u, (size_t)b * a.ldu + d);
        dt[k] = load_in((const TIn *)a.delta, (size_t)b * a.ldd + d) + bias;
        z[k] = a.z ? load_in((const TIn *)a.z, (size_t)b * a.ldz + d) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kStepB; ++k) {
        if (a.softplus) dt[k] = softplus_accurate(dt[k]);
        const float du = dt[k] * u[k];
        y[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[k][i] = fmaf(decay(rate(Av[i]), dt[k]), h[k][i], du * Bv[k][i]);
            y[k] = fmaf(Cv[k][i], h[k][i], y[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kStepB; ++k) {
        const bool mine = on && b0 + k < a.B;
        const size_t row = (size_t)(b0 + k) * a.D + d;
        if (mine) store_n<4, true>(a.h_final + row * N + l * 4, h[k]);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) y[k] += __shfl_xor_sync(0xffffffffu, y[k], o);
        if (mine && l == 0) {
            float v = fmaf(skip, u[k], y[k]);
            if (a.z) v *= z[k] * sigmoid_fast(z[k]);
            store_out((TIn *)a.y, row, v);
        }
    }
}

constexpr int kSms = 152;

// Blocks that carry the channels of every sequence.
long long channel_blocks(int B, int D, int N, int G)
{
    const int db = block_channels(N);
    return (long long)B * G * ((D / G + db - 1) / db);
}

struct Plan { int n, len; };
constexpr long long kMostSegs = 64;   // the last one composes all others, one after another

// Segments per sequence: as many as fill the SMs at two blocks each, from four on, of at least
// four tiles.  A split scan costs 1.6 times the work of a whole one, and whole sequences of one
// block an SM run 1.6 times as fast a token as of two.  2048 tokens of one sequence, whole and
// split: 64 channels 110 and 23 us, 2048 channels 111 and 50, 4096 channels (four segments) 111
// and 84, 6144 channels (three) 111 and 114.
Plan ssm_plan(int B, int T, int D, int N, int G)
{
    const long long blocks = channel_blocks(B, D, N, G);
    int n = (int)std::min<long long>({kSms * 2 / blocks, T / (4 * TT), kMostSegs});
    if (n < 4) n = 1;
    const int len = (int)((((long long)T + n - 1) / n + TT - 1) / TT) * TT;
    if (len <= 0) return {1, TT};
    return {std::max(1, (T + len - 1) / len), len};
}

size_t plan_bytes(const Plan &p, int B, int D, int N)
{
    return p.n > 1 ? (size_t)B * p.n * D * (N + 1) * sizeof(float) : 0;
}

template <typename TIn, int N, bool VEC, int PHASE>
cudaError_t scan_launch(const SsmArgs &a, const Segs &sg, cudaStream_t st)
{
    constexpr int DB = block_channels(N);
    constexpr int bytes = (int)sizeof(Smem<TIn, N>);
    auto *k = ssm_scan_kernel<TIn, N, VEC, PHASE>;
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    const int gblocks = (a.D / a.G + DB - 1) / DB;
    const long long segs = PHASE == kEnds ? sg.n - 1 : sg.n;
    k<<<(unsigned)(gblocks * segs * a.G * a.B), kThreads, bytes, st>>>(a, sg, gblocks);
    return cudaGetLastError();
}

template <typename TIn, int N, bool VEC>
cudaError_t scan_run(const SsmArgs &a, cudaStream_t st)
{
    const Plan p = ssm_plan(a.B, a.T, a.D, a.N, a.G);
    if (p.n > 1 && a.ws && a.ws_bytes >= plan_bytes(p, a.B, a.D, a.N)) {
        const Segs sg{p.n, p.len, a.ws, a.ws + (size_t)a.B * p.n * a.D * a.N};
        const cudaError_t e = scan_launch<TIn, N, VEC, kEnds>(a, sg, st);
        if (e != cudaSuccess) return e;
        return scan_launch<TIn, N, VEC, kFromEnds>(a, sg, st);
    }
    return scan_launch<TIn, N, VEC, kWhole>(a, Segs{1, std::max(TT, (a.T + TT - 1) / TT * TT), nullptr, nullptr}, st);
}

template <typename TIn, int N>
cudaError_t scan_pick(const SsmArgs &a, cudaStream_t st)
{
    constexpr int E = 16 / sizeof(TIn);
    auto ok = [](const void *p) { return ((uintptr_t)p & 15u) == 0; };
    const bool vec = (a.D / a.G) % E == 0 && a.ldu % E == 0 && a.ldd % E == 0 && ok(a.u) && ok(a.delta) && ok(a.y) &&
                     (!a.z || (a.ldz % E == 0 && ok(a.z)));
    return vec ? scan_run<TIn, N, true>(a, st) : scan_run<TIn, N, false>(a, st);
}

template <typename TIn, int N>
cudaError_t step_run(const SsmArgs &a, cudaStream_t st)
{
    constexpr int A = 4 * (int)sizeof(TIn);
    auto ok = [](const void *p, long long ld) {
        return (((uintptr_t)p | (uintptr_t)(ld * (long long)sizeof(TIn))) & (A - 1)) == 0;
    };
    const bool vec = ok(a.Bm, a.ldb) && ok(a.Cm, a.ldc) && ((uintptr_t)a.A & 15u) == 0;
    const long long n = (long long)((a.B + kStepB - 1) / kStepB) * a.D * (N / 4);
    const unsigned blocks = (unsigned)((n + 255) / 256);
    if (vec) ssm_step_kernel<TIn, N, true><<<blocks, 256, 0, st>>>(a);
    else ssm_step_kernel<TIn, N, false><<<blocks, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

#define LDN_BY_STATE(FN)                                                                           \
    switch (a.N) {                                                                                 \
    case 8: return a.dtype == LDN_F32 ? FN<float, 8>(a, st) : FN<__nv_bfloat16, 8>(a, st);         \
    case 16: return a.dtype == LDN_F32 ? FN<float, 16>(a, st) : FN<__nv_bfloat16, 16>(a, st);      \
    case 32: return a.dtype == LDN_F32 ? FN<float, 32>(a, st) : FN<__nv_bfloat16, 32>(a, st);      \
    case 64: return a.dtype == LDN_F32 ? FN<float, 64>(a, st) : FN<__nv_bfloat16, 64>(a, st);      \
    }                                                                                              \
    return cudaErrorInvalidValue

bool ssm_supported_n(int N) { return N == 8 || N == 16 || N == 32 || N == 64; }

size_t ssm_scan_workspace_bytes(int B, int T, int D, int N, int G)
{
    return plan_bytes(ssm_plan(B, T, D, N, G), B, D, N);
}

cudaError_t launch_ssm_scan(const SsmArgs &a, cudaStream_t st) { LDN_BY_STATE(scan_pick); }
cudaError_t launch_ssm_step(const SsmArgs &a, cudaStream_t st) { LDN_BY_STATE(step_run); }

}  // namespace ldn
