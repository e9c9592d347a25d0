// Selective state space scan, forward over sequences and one token.
//
// Channel d, state n, token t:
//   dt = softplus(delta + bias) (or delta + bias),  a = e^{dt A},
//   h_t = a h_{t-1} + dt u_t B_t,   y_t = (sum_n C_t h_t + D u_t) silu(z_t).
//
// One update costs four fp32 operations (dt A, dt u B, a h + ., C h + .) and one exponential
// for every state of every channel and token: at N = 16 that outweighs the eight bytes a
// channel and token of traffic, so the kernel is bound by the fp32 and exponential pipes, and
// what the layout minimises is everything else per update.  L = N / S neighbouring lanes own
// one channel, S states each, in registers over the whole run; exponentials take e^x = 2^{x
// log2 e} with log2 e folded into A.  A block walks tiles of 32 tokens: u, delta and z arrive
// by 16-byte asynchronous copies one tile ahead; a first step widens them and forms (dt, dt u)
// once per channel and token, doubled so that packed fp32x2 operands are one load; the scan
// step reads those and the B, C rows (shared by all channels) from shared memory; the sum
// over a channel's lanes is taken for four tokens together (a halving exchange); a last step
// adds D u, applies the output gate and stores whole rows.
//
// Few channels for the card: the tokens are cut into segments that run side by side.  A first
// launch forms each segment's end state from zero and its sum of dt; in the second a segment
// composes what enters it, h <- e^{A sum dt} h + end, over the segments before it, and runs
// with its outputs.  The exponentials are then taken twice, so it is done only where one wave
// of unsplit blocks leaves the card under-occupied (ssm_segments).
#include "ssm_common.cuh"

namespace ldn {
namespace {
using namespace ssm;

enum { kWhole = 0, kEnds = 1, kFromEnds = 2 };

template <int N> struct Shape;
template <> struct Shape<8> { static constexpr int S = 4, KC = 1; };
template <> struct Shape<16> { static constexpr int S = 4, KC = 1; };
template <> struct Shape<32> { static constexpr int S = 8, KC = 1; };
template <> struct Shape<64> { static constexpr int S = 8, KC = 1; };

constexpr int kThreads = 128;

// Channels per block.
constexpr int block_channels(int N) { return N == 8 ? 64 : N <= 32 ? 32 : 16; }

template <typename TIn, int DB, int N>
struct Smem {
    TIn u[2][TT * DB], d[2][TT * DB], z[2][TT * DB];
    float4 step[TT][DB];        // dt, dt, dt u, dt u
    float B[TT * N], C[TT * N];
    float y[TT][DB + 8];        // +8: the four token rows a warp stores differ in banks
    float bias[DB], skip[DB];
};

struct Segs {
    int n, len;      // segments per sequence, tokens of one (a multiple of TT)
    float *ends;     // [B][n][D][N]
    float *sums;     // [B][n][D]
};

template <typename TIn, int N, bool VEC, int PHASE>
__global__ void __launch_bounds__(kThreads)
ssm_scan_kernel(const SsmArgs a, const Segs sg, int gblocks)
{
    constexpr int S = Shape<N>::S, L = N / S, KC = Shape<N>::KC, SL = kThreads / L, DB = SL * KC;
    static_assert(DB == block_channels(N), "host and device agree on a block's channels");
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<TIn, DB, N> &sm = *reinterpret_cast<Smem<TIn, DB, N> *>(smem_raw);
    const int Dg = a.D / a.G;
    const unsigned cblocks = (unsigned)gblocks * a.G;
    const unsigned cb = blockIdx.x % cblocks, bs = blockIdx.x / cblocks;
    const int seg = (int)(bs % sg.n), b = (int)(bs / sg.n);
    const int grp = (int)(cb / gblocks), cg = (int)(cb % gblocks) * DB;
    const int c0 = grp * Dg + cg, cols = min(DB, Dg - cg);
    const int tid = threadIdx.x, lane = tid & 31, l = tid % L, slot = tid / L;
    const int len = seq_len(a.lens, b, a.T);
    const int tb = seg * sg.len, te = min(tb + sg.len, a.T);
    const size_t row0 = (size_t)b * a.T;
    const TIn *u = (const TIn *)a.u + row0 * a.ldu + c0;
    const TIn *dl = (const TIn *)a.delta + row0 * a.ldd + c0;
    const TIn *z = a.z && PHASE != kEnds ? (const TIn *)a.z + row0 * a.ldz + c0 : nullptr;
    const TIn *Bm = (const TIn *)a.Bm + row0 * a.ldb + (size_t)grp * N;
    const TIn *Cm = (const TIn *)a.Cm + row0 * a.ldc + (size_t)grp * N;

    for (int i = tid; i < DB; i += kThreads) {
        sm.bias[i] = a.bias && i < cols ? a.bias[c0 + i] : 0.f;
        sm.skip[i] = a.Dskip && i < cols ? a.Dskip[c0 + i] : 0.f;
    }
    float2 A2[KC][S / 2], h[KC][S / 2];
    float sumdt[KC];
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        const int ch = slot + k * SL;
        const bool on = ch < cols;
        const size_t at = (size_t)(c0 + ch) * N + l * S;
        sumdt[k] = 0.f;
#pragma unroll
        for (int s = 0; s < S / 2; ++s) {
            A2[k][s] = on ? make_float2(a.A[at + 2 * s] * kLog2e, a.A[at + 2 * s + 1] * kLog2e) : dup(0.f);
            h[k][s] = dup(0.f);
            if (PHASE != kEnds && on && a.h0) {
                const float *p = a.h0 + (size_t)b * a.D * N + at + 2 * s;
                h[k][s] = make_float2(p[0], p[1]);
            }
        }
        if constexpr (PHASE == kFromEnds) {
            if (on)
                for (int j = 0; j < seg; ++j) {
                    const size_t e = ((size_t)b * sg.n + j) * a.D + c0 + ch;
                    const float sd = sg.sums[e];
                    const float *p = sg.ends + e * N + l * S;
#pragma unroll
                    for (int s = 0; s < S / 2; ++s)
                        h[k][s] = __ffma2_rn(ex2(__fmul2_rn(A2[k][s], dup(sd))), h[k][s],
                                             make_float2(p[2 * s], p[2 * s + 1]));
                }
        }
    }

    auto rows_of = [&](int t0) { return min(max(min(len, te) - t0, 0), TT); };
    auto fetch = [&](int t0, int st) {
        const int rows = rows_of(t0);
        load_rows<TIn, DB, kThreads, VEC>(sm.u[st], u + (size_t)t0 * a.ldu, a.ldu, rows, cols);
        load_rows<TIn, DB, kThreads, VEC>(sm.d[st], dl + (size_t)t0 * a.ldd, a.ldd, rows, cols);
        if (z) load_rows<TIn, DB, kThreads, VEC>(sm.z[st], z + (size_t)t0 * a.ldz, a.ldz, rows, cols);
        cp_async_commit();
    };
    RowRegs<TIn, N, kThreads> rB, rC;
    if (tb < te) {
        fetch(tb, 0);
        rB.load(Bm + (size_t)tb * a.ldb, a.ldb, rows_of(tb));
        if (PHASE != kEnds) rC.load(Cm + (size_t)tb * a.ldc, a.ldc, rows_of(tb));
    }
    int st = 0;
    for (int t0 = tb; t0 < te; t0 += TT, st ^= 1) {
        const int rows = rows_of(t0);
        cp_async_wait<0>();
        __syncthreads();   // this tile has arrived; the last tile's readers are done
        rB.store(sm.B);
        if (PHASE != kEnds) rC.store(sm.C);
        if (t0 + TT < te) {
            fetch(t0 + TT, st ^ 1);
            rB.load(Bm + (size_t)(t0 + TT) * a.ldb, a.ldb, rows_of(t0 + TT));
            if (PHASE != kEnds) rC.load(Cm + (size_t)(t0 + TT) * a.ldc, a.ldc, rows_of(t0 + TT));
        }
        // (dt, dt u) of every channel and token; a row past the end steps by zero: a = 1, no input
        for (int i = tid; i < TT * DB; i += kThreads) {
            const int r = i / DB, c = i % DB;
            float dt = (float)sm.d[st][i] + sm.bias[c];
            if (a.softplus) dt = softplus_accurate(dt);
            if (r >= rows) dt = 0.f;
            const float du = r < rows ? dt * (float)sm.u[st][i] : 0.f;
            sm.step[r][c] = make_float4(dt, dt, du, du);
        }
        if (PHASE != kEnds && a.states) {   // the state entering this tile
            const size_t ck = (size_t)b * ((a.T + TT - 1) / TT) + t0 / TT;
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int ch = slot + k * SL;
                if (ch < cols) {
                    float4 *p = reinterpret_cast<float4 *>(a.states + (ck * a.D + c0 + ch) * N + l * S);
#pragma unroll
                    for (int s = 0; s < S / 4; ++s)
                        p[s] = make_float4(h[k][2 * s].x, h[k][2 * s].y, h[k][2 * s + 1].x, h[k][2 * s + 1].y);
                }
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int tq = 0; tq < TT; tq += 4) {
            float yv[4 * KC];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = tq + j;
                float2 Bv[S / 2], Cv[S / 2];
#pragma unroll
                for (int s = 0; s < S / 4; ++s) {
                    const float4 q = *reinterpret_cast<const float4 *>(&sm.B[r * N + l * S + 4 * s]);
                    Bv[2 * s] = make_float2(q.x, q.y);
                    Bv[2 * s + 1] = make_float2(q.z, q.w);
                    if (PHASE != kEnds) {
                        const float4 w = *reinterpret_cast<const float4 *>(&sm.C[r * N + l * S + 4 * s]);
                        Cv[2 * s] = make_float2(w.x, w.y);
                        Cv[2 * s + 1] = make_float2(w.z, w.w);
                    }
                }
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    const float4 q = sm.step[r][slot + k * SL];
                    const float2 dt = make_float2(q.x, q.y), du = make_float2(q.z, q.w);
                    if (PHASE == kEnds) sumdt[k] += q.x;
                    float2 acc = dup(0.f);
#pragma unroll
                    for (int s = 0; s < S / 2; ++s) {
                        const float2 e = ex2(__fmul2_rn(A2[k][s], dt));
                        h[k][s] = __ffma2_rn(e, h[k][s], __fmul2_rn(du, Bv[s]));
                        if (PHASE != kEnds) acc = s ? __ffma2_rn(Cv[s], h[k][s], acc) : __fmul2_rn(Cv[s], h[k][s]);
                    }
                    yv[j * KC + k] = acc.x + acc.y;
                }
            }
            if constexpr (PHASE != kEnds) {
                constexpr int V = 4 * KC;
                reduce_halving<V, L / 2, 1>(yv, lane);
                constexpr int HELD = V >= L ? V / L : 1, DUP = V >= L ? 1 : L / V;
                if (l % DUP == 0)
#pragma unroll
                    for (int i = 0; i < HELD; ++i) {
                        const int idx = (l / DUP) * HELD + i;
                        sm.y[tq + idx / KC][slot + (idx % KC) * SL] = yv[i];
                    }
            }
        }
        if constexpr (PHASE != kEnds) {
            __syncthreads();
            constexpr int E = VEC ? 16 / (int)sizeof(TIn) : 1, PER = DB / E;
            const int live = min(te - t0, TT);
            TIn *y = (TIn *)a.y + (row0 + t0) * a.D + c0;
            for (int i = tid; i < TT * PER; i += kThreads) {
                const int r = i / PER, e = (i % PER) * E;
                if (r >= live || e >= cols) continue;
                float v[E], uu[E], zz[E];
                load_n<E, VEC>(&sm.u[st][r * DB + e], uu);
                if (z) load_n<E, VEC>(&sm.z[st][r * DB + e], zz);
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    v[k] = fmaf(sm.skip[e + k], uu[k], sm.y[r][e + k]);
                    if (z) v[k] *= zz[k] * sigmoid_fast(zz[k]);
                    if (r >= rows) v[k] = 0.f;   // a row past the sequence's end
                }
                store_n<E, VEC>(y + (size_t)r * a.D + e, v);
            }
        }
    }

    if (PHASE == kEnds || (seg == sg.n - 1 && a.h_final)) {
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const int ch = slot + k * SL;
            if (ch >= cols) continue;
            const size_t e = (PHASE == kEnds ? (size_t)b * sg.n + seg : (size_t)b) * a.D + c0 + ch;
            float4 *p = reinterpret_cast<float4 *>((PHASE == kEnds ? sg.ends : a.h_final) + e * N + l * S);
#pragma unroll
            for (int s = 0; s < S / 4; ++s)
                p[s] = make_float4(h[k][2 * s].x, h[k][2 * s].y, h[k][2 * s + 1].x, h[k][2 * s + 1].y);
            if (PHASE == kEnds && l == 0) sg.sums[e] = sumdt[k];
        }
    }
}

// One token for every sequence: a lane takes four states of one channel, the channel's lanes
// sum; h is read and written once, which is nearly all of the traffic.
template <typename TIn, int N>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmArgs a)
{
    constexpr int L = N / 4;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long unit = id / L;
    const int l = (int)(id % L);
    const bool on = unit < (long long)a.B * a.D;
    const int b = on ? (int)(unit / a.D) : 0, d = on ? (int)(unit % a.D) : 0, g = d / (a.D / a.G);
    const TIn *Bm = (const TIn *)a.Bm + (size_t)b * a.ldb + g * N + l * 4;
    const TIn *Cm = (const TIn *)a.Cm + (size_t)b * a.ldc + g * N + l * 4;
    const size_t at = ((size_t)b * a.D + d) * N + l * 4;
    const float4 hv = *reinterpret_cast<const float4 *>(a.h0 + at);
    float h[4] = {hv.x, hv.y, hv.z, hv.w}, Av[4], y = 0.f;
    load_n<4, false>(a.A + (size_t)d * N + l * 4, Av);
    const float u = load_in((const TIn *)a.u, (size_t)b * a.ldu + d);
    float dt = load_in((const TIn *)a.delta, (size_t)b * a.ldd + d) + (a.bias ? a.bias[d] : 0.f);
    if (a.softplus) dt = softplus_accurate(dt);
    const float du = dt * u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(ex2(dt * (Av[i] * kLog2e)), h[i], du * load_in(Bm, i));
        y = fmaf(load_in(Cm, i), h[i], y);
    }
    if (on) *reinterpret_cast<float4 *>(a.h_final + at) = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (on && l == 0) {
        if (a.Dskip) y = fmaf(a.Dskip[d], u, y);
        if (a.z) {
            const float z = load_in((const TIn *)a.z, (size_t)b * a.ldz + d);
            y *= z * sigmoid_fast(z);
        }
        store_out((TIn *)a.y, (size_t)b * a.D + d, y);
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

// Segments per sequence.
Plan ssm_plan(int B, int T, int D, int N, int G)
{
    const long long blocks = channel_blocks(B, D, N, G);
    const long long want = kSms * 4;
    int n = 1;
    if (blocks * 2 <= kSms * 3) n = (int)std::min<long long>((want + blocks - 1) / blocks, std::min(T / 128, 64));
    n = std::max(n, 1);
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
    constexpr int bytes = (int)sizeof(Smem<TIn, DB, N>);
    auto *k = ssm_scan_kernel<TIn, N, VEC, PHASE>;
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    const int gblocks = (a.D / a.G + DB - 1) / DB;
    k<<<(unsigned)((long long)gblocks * a.G * a.B * sg.n), kThreads, bytes, st>>>(a, sg, gblocks);
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
    const long long n = (long long)a.B * a.D * (N / 4);
    ssm_step_kernel<TIn, N><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
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
