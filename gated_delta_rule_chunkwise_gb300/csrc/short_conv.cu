// Depthwise causal short convolution with a carried state: whole sequences, one token, and
// the gradient.
//
//   p_t[c] = b[c] + sum_{j<W} w[c][j] x_{t-W+1+j}[c],   y_t = silu(p_t) or p_t.
// Rows before t = 0 come from `state` (the W - 1 rows before the call; zeros when NULL);
// `state_out` gets the last W - 1 rows at each sequence's end.  With lengths, rows at and
// past a sequence's end are not read; their outputs (and gradients) are zeros.
//
//   dp_t = dy_t silu'(p_t),   dx_t = sum_j w[j] dp_{t+W-1-j} (+ dstate_out's row),
//   dw[j] = sum_t dp_t x_{t-W+1+j},   db = sum_t dp_t.
//
// Every direction streams its rows once: HBM is the floor (bf16, W = 4: 20 us for 4 x 2048 x
// 4096 forward, 15 us for the gradient at half the channels).  A lane owns four channels and
// walks a run of tokens with the last W rows in registers, so nothing goes through shared
// memory but the weights; rows are loaded a batch ahead and kept as loaded until used.  That
// takes 28 and 33 us: half the issue slots are used, and the rest is waiting for rows (loads
// in flight are bound by the registers that hold them) and for the taps' chains.
#include <type_traits>

#include "mixer_common.cuh"

namespace ldn {
namespace {

constexpr int kWarps = 4;   // runs per block, one warp each; all warps take the same channels
// Rows on their way at a time, and the registers a thread that leaves (blocks an SM): what
// measured fastest of 2, 3, 4 rows and 4 to 10 blocks at 4 x 2048 x 4096 (forward: 28 us, 33 at
// two rows, 42 with 16-byte loads and twice the registers).
constexpr int kBatch = 4, kBwdBatch = 3;
// Single elements (a word each on their way) leave room for fewer blocks.  More than four taps take
// registers: of 3, 4, 5, 6 blocks forward at 4 x 2048 x 4096 in bf16 W = 5 takes 36, 32, 31, 37 us and
// W = 8 39, 36, 54, 76; of 1, 2, 3, 4 in the gradient 123, 63, 63, 72 and 128, 92, 144, 254 (fp32, half
// the channels, W = 6: 61, 54, 46, 105).
constexpr int fwd_blocks(int W, bool vec) { return W > 4 ? 4 : vec ? 7 : 5; }
constexpr int bwd_blocks(int W, bool vec) { return W > 4 ? 2 : vec ? 4 : 3; }

// A lane owns 4 channels: consecutive ones where rows are whole vectors of 4, otherwise 32
// apart, so that a warp's single elements are neighbours (against one channel a lane: 4 x 2048
// x 1001 bf16 12.6 us for 14.2, gradient 29.7 for 31.9; 8 x 700 x 5003 30 for 41, gradient 87
// for 81; 2 x 100 x 301, which has too few lanes then, 4.5 for 3.1).
constexpr int kE = 4;
constexpr int step_of(bool vec) { return vec ? 1 : 32; }
__device__ __forceinline__ int place(bool vec, int t) { return vec ? t * kE : (t & ~31) * kE + (t & 31); }

__device__ __forceinline__ int seq_len(const int *lens, int b, int T)
{
    return lens ? min(max(lens[b], 0), T) : T;
}

// The weights of CH channels from c0 to shared memory, tap by tap: wsm[j][CH].  (Loaded one
// after another they cost a block 1 us: 300 x 512 3.6 us for 4.3, 4 x 2048 x 4096 27.5 for 28.4.)
template <int W, int CH>
__device__ __forceinline__ void load_taps(float *wsm, const float *w, int c0, int C)
{
    constexpr int EACH = CH * W / (32 * kWarps);
    float v[EACH];   // all on their way at once
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int i = k * 32 * kWarps + (int)threadIdx.x;
        v[k] = c0 + i / W < C ? __ldg(w + (size_t)c0 * W + i) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int i = k * 32 * kWarps + (int)threadIdx.x;
        wsm[i % W * CH + i / W] = v[k];
    }
    __syncthreads();
}

// A block is one run of tokens; its warps take neighbouring channels, so that it reads and
// writes 1 KB (bf16) of every row.
template <typename TIn, int W, bool VEC>
__global__ void __launch_bounds__(32 * kWarps, fwd_blocks(W, VEC))
short_conv_kernel(const ConvArgs a, int run, int runs, int cblocks)
{
    constexpr int E = kE, STEP = step_of(VEC), CH = 32 * kWarps * E;
    __shared__ __align__(16) float wsm[W * CH];
    const int cb = blockIdx.x % cblocks;
    const unsigned rb = blockIdx.x / cblocks;
    const int b = (int)(rb / runs), ri = (int)(rb % runs);
    load_taps<W, CH>(wsm, a.w, cb * CH, a.C);
    const int at = place(VEC, threadIdx.x), c = cb * CH + at, valid = a.C - c;
    if (valid <= 0) return;
    float wt[W][E], bias[E];
#pragma unroll
    for (int j = 0; j < W; ++j) load_n<E, VEC, STEP>(&wsm[j * CH + at], wt[j]);
    if (a.bias) load_n<E, false, STEP>(a.bias + c, bias, valid);
    else
#pragma unroll
        for (int i = 0; i < E; ++i) bias[i] = 0.f;
    const int len = seq_len(a.lens, b, a.T), t0 = ri * run, t1 = min(t0 + run, a.T);
    const TIn *x = (const TIn *)a.x + (size_t)b * a.T * a.ldx + c;
    TIn *y = (TIn *)a.y + (size_t)b * a.T * a.C + c;
    const TIn *st = a.state ? (const TIn *)a.state + (size_t)b * (W - 1) * a.C + c : nullptr;
    // row t of the sequence: the state's for t < 0, zeros at and past the end
    auto row = [&](int t, float *v) {
        if (t < 0) {
            if (st) load_n<E, VEC, STEP>(st + (size_t)(t + W - 1) * a.C, v, valid);
            else
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = 0.f;
        } else {
            load_n<E, VEC, STEP>(x + (size_t)t * a.ldx, v, t < len ? valid : 0);
        }
    };
    // win: the W - 1 rows before a batch, then the batch; the next batch is on its way as loaded
    float win[W - 1 + kBatch][E];
    Raw<TIn, E, VEC> next[kBatch];
    const int stop = min(len, t1);   // rows past it are not read
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row(t0 - (W - 1) + j, win[j]);
    // EDGE: some of the batch's rows or of the next one's may be outside
    auto batch = [&](int t, auto edge) {
        constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) next[k].widen(win[W - 1 + k]);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            next[k].template load<VEC, STEP>(x + (size_t)(t + kBatch + k) * a.ldx,
                                       !EDGE || t + kBatch + k < stop ? valid : 0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            float p[E];
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                float2 q = make_float2(bias[i], bias[i + 1]);
#pragma unroll
                for (int j = 0; j < W; ++j)
                    q = __ffma2_rn(make_float2(wt[j][i], wt[j][i + 1]),
                                   make_float2(win[k + j][i], win[k + j][i + 1]), q);
                if (a.act) q = silu_fast(q);
                p[i] = q.x;
                p[i + 1] = q.y;
            }
            if (EDGE && t + k >= len)
#pragma unroll
                for (int i = 0; i < E; ++i) p[i] = 0.f;
            if (!EDGE || t + k < t1) store_n<E, VEC, STEP>(y + (size_t)(t + k) * a.C, p, valid);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) win[j][i] = win[j + kBatch][i];
    };
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
        next[k].template load<VEC, STEP>(x + (size_t)(t0 + k) * a.ldx, t0 + k < stop ? valid : 0);
    // Two batches in one body leave half the window's moves from register to register: 28.3 us
    // for 29.7 at 4 x 2048 x 4096 in bf16; fp32 rows (22.9 us for 21.6 at half the channels) and
    // more than four taps (44 for 37 at W = 8) have no registers left for it.
    constexpr bool TWO = W <= 4 && sizeof(TIn) == 2;
    for (int t = t0; t < t1; t += kBatch) {
        if (TWO && t + 3 * kBatch <= stop) {
            batch(t, std::false_type{});
            batch(t += kBatch, std::false_type{});
        } else if (!TWO && t + 2 * kBatch <= stop) {
            batch(t, std::false_type{});
        } else {
            batch(t, std::true_type{});
        }
    }
    // The first run alone reads state rows (a run is at least W - 1 tokens), so its lanes may
    // write state_out over them once they have read the last rows.
    if (ri == 0 && a.state_out && W > 1) {
        float last[W][E];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) row(len - (W - 1) + j, last[j]);
        TIn *so = (TIn *)a.state_out + (size_t)b * (W - 1) * a.C + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_n<E, VEC, STEP>(so + (size_t)j * a.C, last[j], valid);
    }
}

// One token: E channels of one sequence per thread.
template <typename TIn, int W, int E, bool VEC>
__global__ void __launch_bounds__(128) short_conv_step_kernel(const ConvArgs a)
{
    const int per = (a.C + E - 1) / E;
    const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
    if (id >= (long long)a.B * per) return;
    const int b = (int)(id / per), c = (int)(id % per) * E, valid = a.C - c;
    float rows[W][E], p[E], wt[E * W];
    load_n<E * W, VEC>(a.w + (size_t)c * W, wt, min(valid, E) * W);   // taps of one channel after another
    const TIn *st = (const TIn *)a.state + (size_t)b * (W - 1) * a.C + c;
    TIn *so = (TIn *)a.state_out + (size_t)b * (W - 1) * a.C + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_n<E, VEC>(st + (size_t)j * a.C, rows[j], valid);
    load_n<E, VEC>((const TIn *)a.x + (size_t)b * a.ldx + c, rows[W - 1], valid);
    load_n<E, VEC>(a.bias + (a.bias ? c : 0), p, a.bias ? valid : 0);
#pragma unroll
    for (int i = 0; i < E; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) p[i] = fmaf(wt[i * W + j], rows[j][i], p[i]);
        if (a.act) p[i] *= sigmoid_fast(p[i]);
    }
    store_n<E, VEC>((TIn *)a.y + (size_t)b * a.C + c, p, valid);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_n<E, VEC>(so + (size_t)j * a.C, rows[j + 1], valid);
}

// The gradient.  A warp walks tokens t0 .. t1 + W - 2 of its run: dp_t from the window of x,
// then row t - (W - 1) of dx, whose last term dp_t is.  The first run also emits the state's
// rows (t < 0).  dw and db over the run's own tokens, summed over the block's warps, go to
// part [rblocks * B][W + 1][C].
template <typename TIn, int W, bool VEC>
__global__ void __launch_bounds__(32 * kWarps, bwd_blocks(W, VEC))
short_conv_bwd_kernel(const ConvBwdArgs a, int run, int runs, int cblocks)
{
    constexpr int E = kE, STEP = step_of(VEC);
    __shared__ __align__(16) float wsm[W * 32 * E];
    __shared__ float sums[kWarps][W + 1][32 * E];
    const int cb = blockIdx.x % cblocks;
    const unsigned rb = blockIdx.x / cblocks;
    const int rblocks = (runs + kWarps - 1) / kWarps;
    const int warp = threadIdx.x >> 5, at = place(VEC, threadIdx.x & 31);
    const int b = (int)(rb / rblocks), ri = (int)(rb % rblocks) * kWarps + warp;
    const int c0 = cb * 32 * E;
    load_taps<W, 32 * E>(wsm, a.w, c0, a.C);
    const int c = c0 + at, valid = a.C - c;
    float dw[W + 1][E];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) dw[j][i] = 0.f;
    if (ri < runs && valid > 0) {
        float wt[W][E], bias[E];
#pragma unroll
        for (int j = 0; j < W; ++j) load_n<E, VEC, STEP>(&wsm[j * 32 * E + at], wt[j]);
        if (a.bias) load_n<E, false, STEP>(a.bias + c, bias, valid);
        else
#pragma unroll
            for (int i = 0; i < E; ++i) bias[i] = 0.f;
        const int len = seq_len(a.lens, b, a.T), t0 = ri * run, t1 = min(t0 + run, a.T);
        const TIn *x = (const TIn *)a.x + (size_t)b * a.T * a.ldx + c;
        const TIn *dy = (const TIn *)a.dy + (size_t)b * a.T * a.C + c;
        TIn *dx = (TIn *)a.dx + (size_t)b * a.T * a.C + c;
        const size_t so = (size_t)b * (W - 1) * a.C + c;
        const TIn *st = a.state ? (const TIn *)a.state + so : nullptr;
        const TIn *dso = a.dstate_out ? (const TIn *)a.dstate_out + so : nullptr;
        TIn *dst = a.dstate ? (TIn *)a.dstate + so : nullptr;
        auto row = [&](int t, float *v) {
            if (t < 0) {
                if (st) load_n<E, VEC, STEP>(st + (size_t)(t + W - 1) * a.C, v, valid);
                else
#pragma unroll
                    for (int i = 0; i < E; ++i) v[i] = 0.f;
            } else {
                load_n<E, VEC, STEP>(x + (size_t)t * a.ldx, v, t < len ? valid : 0);
            }
        };
        // rows t-W+1 .. of x and of dp, a batch at a time; the next batch is on its way as loaded
        float win[W - 1 + kBwdBatch][E], dp[W - 1 + kBwdBatch][E];
        Raw<TIn, E, VEC> nx[kBwdBatch], ny[kBwdBatch];
        const int end = t1 + W - 1, stop = min(len, end);   // dp_t to end; rows past stop are not read
        auto fetch = [&](int t, auto edge) {
#pragma unroll
            for (int k = 0; k < kBwdBatch; ++k) {
                const int n = !decltype(edge)::value || t + k < stop ? valid : 0;
                nx[k].template load<VEC, STEP>(x + (size_t)(t + k) * a.ldx, n);
                ny[k].template load<VEC, STEP>(dy + (size_t)(t + k) * a.C, n);
            }
        };
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            row(t0 - (W - 1) + j, win[j]);
#pragma unroll
            for (int i = 0; i < E; ++i) dp[j][i] = 0.f;
        }
        // EDGE: some of the batch's rows, of those it finishes or of the next ones may be outside
        auto batch = [&](int t, auto edge) {
            constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
            for (int k = 0; k < kBwdBatch; ++k) {
                nx[k].widen(win[W - 1 + k]);
                ny[k].widen(dp[W - 1 + k]);
            }
            fetch(t + kBwdBatch, edge);
#pragma unroll
            for (int k = 0; k < kBwdBatch; ++k) {
                float *now = dp[W - 1 + k];
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    float2 d = make_float2(now[i], now[i + 1]);
                    if (a.act) {
                        float2 p = make_float2(bias[i], bias[i + 1]);
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            p = __ffma2_rn(make_float2(wt[j][i], wt[j][i + 1]),
                                           make_float2(win[k + j][i], win[k + j][i + 1]), p);
                        const float2 g = rcp(__fadd2_rn(ex2(__fmul2_rn(p, dup(-kLog2e))), dup(1.f)));
                        const float2 rest = __ffma2_rn(g, dup(-1.f), dup(1.f));
                        d = __fmul2_rn(d, __fmul2_rn(g, __ffma2_rn(p, rest, dup(1.f))));
                    }
                    if (EDGE && t + k >= len) d = dup(0.f);   // nothing flows from past the end, whatever p is
                    now[i] = d.x;
                    now[i + 1] = d.y;
                    if (!EDGE || t + k < min(t1, len)) {   // past the end d is 0, but a row of the window may be infinite
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            const float2 q = __ffma2_rn(d, make_float2(win[k + j][i], win[k + j][i + 1]),
                                                        make_float2(dw[j][i], dw[j][i + 1]));
                            dw[j][i] = q.x;
                            dw[j][i + 1] = q.y;
                        }
                        const float2 q = __fadd2_rn(d, make_float2(dw[W][i], dw[W][i + 1]));
                        dw[W][i] = q.x;
                        dw[W][i + 1] = q.y;
                    }
                }
                const int r = t + k - (W - 1);   // the row that dp_{t + k} completes
                if (!EDGE || (r < t1 && (r >= t0 || (ri == 0 && dst)))) {
                    float d[E];
                    const int j0 = r - (len - (W - 1));   // its place in state_out
                    if (EDGE && dso && j0 >= 0 && j0 < W - 1) load_n<E, VEC, STEP>(dso + (size_t)j0 * a.C, d, valid);
                    else
#pragma unroll
                        for (int i = 0; i < E; ++i) d[i] = 0.f;
#pragma unroll
                    for (int i = 0; i < E; i += 2) {
                        float2 q = make_float2(d[i], d[i + 1]);
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            q = __ffma2_rn(make_float2(wt[W - 1 - j][i], wt[W - 1 - j][i + 1]),
                                           make_float2(dp[k + j][i], dp[k + j][i + 1]), q);
                        if (EDGE && r >= len) q = dup(0.f);   // whatever the weights are
                        d[i] = q.x;
                        d[i + 1] = q.y;
                    }
                    if (!EDGE || r >= 0) store_n<E, VEC, STEP>(dx + (long long)r * a.C, d, valid);
                    else store_n<E, VEC, STEP>(dst + (size_t)(r + W - 1) * a.C, d, valid);
                }
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    win[j][i] = win[j + kBwdBatch][i];
                    dp[j][i] = dp[j + kBwdBatch][i];
                }
        };
        fetch(t0, std::true_type{});
        for (int t = t0; t < end; t += kBwdBatch) {
            if (t >= t0 + W - 1 && t + kBwdBatch <= t1 && t + 2 * kBwdBatch <= stop) batch(t, std::false_type{});
            else batch(t, std::true_type{});
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) sums[warp][j][at + i * STEP] = dw[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32 * E; i += 32 * kWarps) {
        const int j = i / (32 * E), cc = i % (32 * E);
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) t += sums[k][j][cc];
        if (c0 + cc < a.C) a.part[((size_t)rb * (W + 1) + j) * a.C + c0 + cc] = t;
    }
}

// dw [C][W] and db [C] from part [n][W + 1][C]: 32 columns a block, kSumRows rows at a time.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows)
conv_param_sum_kernel(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ db, int n, int W,
                      int C)
{
    __shared__ float sm[kSumRows][33];
    const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y, y = threadIdx.y;
    float t = 0.f;
    if (c < C)
#pragma unroll 8
        for (int i = y; i < n; i += kSumRows) t += part[((size_t)i * (W + 1) + j) * C + c];
    sm[y][threadIdx.x] = t;
    __syncthreads();
    if (y == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i) t += sm[i][threadIdx.x];
        if (j < W) dw[(size_t)c * W + j] = t;
        else if (db) db[c] = t;
    }
}

// Tokens of a run, of which a block has `per`; `units` blocks take a run of every sequence and
// channel.  Blocks come in waves of those that fit on the card, and a part wave takes as long
// as a whole one: of the runs that just fill one to four waves the one whose waves are shortest,
// a block's start and end counted as kStart tokens.  Against runs of 64, 32, 16 or 8 tokens,
// halved until there were 24 warps an SM: gradient of 4 x 2048 x 2048 33.2 us for 35.9, 3 x 3000
// x 2560 41 for 51, 7 x 777 x 1028 (fp32, W = 3) 16.6 for 24.5 and forward 9.4 for 11.4; where
// those runs happened to fill their waves the two are the same.
constexpr int kStart = 8;
int conv_run(long long units, int T, int W, int per, int blocks_sm)
{
    const long long fit = 152ll * blocks_sm;
    int best = 8;
    long long least = 0;
    for (int w = 1; w <= 4; ++w) {
        const long long rb = std::max(1ll, w * fit / std::max(1ll, units)), most = rb * per;
        const int run = (int)std::max(8ll, (T + most - 1) / most), runs = (T + run - 1) / run;
        const long long waves = (units * ((runs + per - 1) / per) + fit - 1) / fit;
        const long long cost = waves * (run + W - 1 + kStart);
        if (w == 1 || cost < least) best = run, least = cost;
    }
    return best;
}

// Runs of the gradient do not go by the alignment: the workspace's size follows them.
int conv_bwd_run(int B, int T, int C, int W)
{
    return conv_run((long long)B * ((C + 32 * kE - 1) / (32 * kE)), T, W, kWarps, bwd_blocks(W, true));
}

bool aligned_to(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename TIn, int W>
cudaError_t conv_fwd(const ConvArgs &a, cudaStream_t st)
{
    constexpr int E = kE, A = E * (int)sizeof(TIn);
    const bool vec = a.C % E == 0 && a.ldx % E == 0 && aligned_to(a.x, A) && aligned_to(a.y, A) &&
                     aligned_to(a.state, A) && aligned_to(a.state_out, A);
    constexpr int per = 32 * kWarps * E;
    const int cblocks = (a.C + per - 1) / per;
    const int run = conv_run((long long)a.B * cblocks, a.T, W, 1, fwd_blocks(W, vec));
    const int runs = std::max(1, (a.T + run - 1) / run);
    const long long blocks = (long long)cblocks * a.B * runs;
    if (vec) short_conv_kernel<TIn, W, true><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    else short_conv_kernel<TIn, W, false><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    return cudaGetLastError();
}

template <typename TIn, int W>
cudaError_t conv_step(const ConvArgs &a, cudaStream_t st)
{
    constexpr int E = kE, A = E * (int)sizeof(TIn);
    const bool vec = a.C % E == 0 && a.ldx % E == 0 && aligned_to(a.x, A) && aligned_to(a.y, A) &&
                     aligned_to(a.state, A) && aligned_to(a.state_out, A) && aligned_to(a.w, 16) &&
                     aligned_to(a.bias, 16);
    const long long n = (long long)a.B * ((a.C + (vec ? E : 1) - 1) / (vec ? E : 1));
    const unsigned blocks = (unsigned)((n + 127) / 128);
    if (vec) short_conv_step_kernel<TIn, W, E, true><<<blocks, 128, 0, st>>>(a);
    else short_conv_step_kernel<TIn, W, 1, false><<<blocks, 128, 0, st>>>(a);
    return cudaGetLastError();
}


template <typename TIn, int W>
cudaError_t conv_bwd(const ConvBwdArgs &a, cudaStream_t st)
{
    constexpr int A = kE * sizeof(TIn);
    const bool vec = a.C % kE == 0 && a.ldx % kE == 0 && aligned_to(a.x, A) && aligned_to(a.dy, A) &&
                     aligned_to(a.dx, A) && aligned_to(a.state, A) && aligned_to(a.dstate, A) &&
                     aligned_to(a.dstate_out, A);
    const int run = conv_bwd_run(a.B, a.T, a.C, W), runs = std::max(1, (a.T + run - 1) / run);
    const int cblocks = (a.C + 32 * kE - 1) / (32 * kE);
    const long long blocks = (long long)cblocks * a.B * ((runs + kWarps - 1) / kWarps);
    if (vec) short_conv_bwd_kernel<TIn, W, true><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    else short_conv_bwd_kernel<TIn, W, false><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int n = a.B * ((runs + kWarps - 1) / kWarps);
    conv_param_sum_kernel<<<dim3((a.C + 31) / 32, W + 1), dim3(32, kSumRows), 0, st>>>(a.part, a.dw, a.db, n, W, a.C);
    return cudaGetLastError();
}

}  // namespace

#define LDN_BY_WIDTH(FN)                                                                       \
    switch (a.W) {                                                                             \
    case 1: return a.dtype == LDN_F32 ? FN<float, 1>(a, st) : FN<__nv_bfloat16, 1>(a, st);     \
    case 2: return a.dtype == LDN_F32 ? FN<float, 2>(a, st) : FN<__nv_bfloat16, 2>(a, st);     \
    case 3: return a.dtype == LDN_F32 ? FN<float, 3>(a, st) : FN<__nv_bfloat16, 3>(a, st);     \
    case 4: return a.dtype == LDN_F32 ? FN<float, 4>(a, st) : FN<__nv_bfloat16, 4>(a, st);     \
    case 5: return a.dtype == LDN_F32 ? FN<float, 5>(a, st) : FN<__nv_bfloat16, 5>(a, st);     \
    case 6: return a.dtype == LDN_F32 ? FN<float, 6>(a, st) : FN<__nv_bfloat16, 6>(a, st);     \
    case 7: return a.dtype == LDN_F32 ? FN<float, 7>(a, st) : FN<__nv_bfloat16, 7>(a, st);     \
    case 8: return a.dtype == LDN_F32 ? FN<float, 8>(a, st) : FN<__nv_bfloat16, 8>(a, st);     \
    }                                                                                          \
    return cudaErrorInvalidValue

cudaError_t launch_short_conv(const ConvArgs &a, cudaStream_t st) { LDN_BY_WIDTH(conv_fwd); }
cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t st) { LDN_BY_WIDTH(conv_step); }
cudaError_t launch_short_conv_bwd(const ConvBwdArgs &a, cudaStream_t st) { LDN_BY_WIDTH(conv_bwd); }

size_t short_conv_bwd_workspace_bytes(int B, int T, int C, int W)
{
    const int run = conv_bwd_run(B, T, C, W), runs = std::max(1, (T + run - 1) / run);
    return (size_t)B * ((runs + kWarps - 1) / kWarps) * (W + 1) * C * sizeof(float);
}

}  // namespace ldn
