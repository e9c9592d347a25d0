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
// Every direction streams its rows once and is bound by HBM.  A lane owns 16 bytes of a row
// (8 bf16 / 4 fp32 channels; the gradient 4 channels) and walks a run of tokens with the last
// W rows in registers, so nothing goes through shared memory but the weights; a warp covers
// 512 contiguous bytes of every row.
#include "mixer_common.cuh"

namespace ldn {
namespace {

constexpr int kWarps = 4;   // runs per block, one warp each; all warps take the same channels
constexpr int kBatch = 4;   // rows on their way at a time

__device__ __forceinline__ int seq_len(const int *lens, int b, int T)
{
    return lens ? min(max(lens[b], 0), T) : T;
}

// The block's weights to shared memory, tap by tap: wsm[j][32 * E].
template <int W, int E>
__device__ __forceinline__ void load_taps(float *wsm, const float *w, int c0, int C)
{
    for (int i = threadIdx.x; i < 32 * E * W; i += blockDim.x) {
        const int c = i / W, j = i % W;
        wsm[j * 32 * E + c] = c0 + c < C ? __ldg(w + (size_t)(c0 + c) * W + j) : 0.f;
    }
    __syncthreads();
}

template <typename TIn, int W, int E, bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
short_conv_kernel(const ConvArgs a, int run, int runs, int cblocks)
{
    __shared__ __align__(16) float wsm[W * 32 * E];
    const int cb = blockIdx.x % cblocks;
    const unsigned rb = blockIdx.x / cblocks;
    const int rblocks = (runs + kWarps - 1) / kWarps;
    const int b = (int)(rb / rblocks), ri = (int)(rb % rblocks) * kWarps + (threadIdx.x >> 5);
    const int c0 = cb * 32 * E, lane = threadIdx.x & 31;
    load_taps<W, E>(wsm, a.w, c0, a.C);
    const int c = c0 + lane * E, valid = a.C - c;
    if (ri >= runs || valid <= 0) return;
    float wt[W][E], bias[E];
#pragma unroll
    for (int j = 0; j < W; ++j) load_n<E, (E % 4 == 0)>(&wsm[j * 32 * E + lane * E], wt[j]);
    if (a.bias) load_n<E, false>(a.bias + c, bias, valid);
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
            if (st) load_n<E, VEC>(st + (size_t)(t + W - 1) * a.C, v, valid);
            else
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = 0.f;
        } else {
            load_n<E, VEC>(x + (size_t)t * a.ldx, v, t < len ? valid : 0);
        }
    };
    // win: the W - 1 rows before a batch, then the batch; the next batch is on its way as loaded
    float win[W - 1 + kBatch][E];
    Raw<TIn, E> next[kBatch];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            next[k].template load<VEC>(x + (size_t)(t + k) * a.ldx, t + k < min(len, t1) ? valid : 0);
    };
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row(t0 - (W - 1) + j, win[j]);
    fetch(t0);
    for (int t = t0; t < t1; t += kBatch) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) next[k].widen(win[W - 1 + k]);
        fetch(t + kBatch);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            float p[E];
            if constexpr (E % 2 == 0) {
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
            } else {
                p[0] = bias[0];
#pragma unroll
                for (int j = 0; j < W; ++j) p[0] = fmaf(wt[j][0], win[k + j][0], p[0]);
                if (a.act) p[0] *= sigmoid_fast(p[0]);
            }
            if (t + k >= len)
#pragma unroll
                for (int i = 0; i < E; ++i) p[i] = 0.f;
            if (t + k < t1) store_n<E, VEC>(y + (size_t)(t + k) * a.C, p, valid);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < E; ++i) win[j][i] = win[j + kBatch][i];
    }
    // The first run alone reads state rows (a run is at least W - 1 tokens), so its lanes may
    // write state_out over them once they have read the last rows.
    if (ri == 0 && a.state_out && W > 1) {
        float last[W][E];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) row(len - (W - 1) + j, last[j]);
        TIn *so = (TIn *)a.state_out + (size_t)b * (W - 1) * a.C + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_n<E, VEC>(so + (size_t)j * a.C, last[j], valid);
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
    load_n<E * W, VEC>(a.w + (size_t)c * W, wt, valid * W);   // taps of one channel after another
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
template <typename TIn, int W, int E, bool VEC>
__global__ void __launch_bounds__(32 * kWarps)
short_conv_bwd_kernel(const ConvBwdArgs a, int run, int runs, int cblocks)
{
    __shared__ __align__(16) float wsm[W * 32 * E];
    __shared__ float sums[kWarps][W + 1][32 * E];
    const int cb = blockIdx.x % cblocks;
    const unsigned rb = blockIdx.x / cblocks;
    const int rblocks = (runs + kWarps - 1) / kWarps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = (int)(rb / rblocks), ri = (int)(rb % rblocks) * kWarps + warp;
    const int c0 = cb * 32 * E;
    load_taps<W, E>(wsm, a.w, c0, a.C);
    const int c = c0 + lane * E, valid = a.C - c;
    float dw[W + 1][E];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) dw[j][i] = 0.f;
    if (ri < runs && valid > 0) {
        float wt[W][E], bias[E];
#pragma unroll
        for (int j = 0; j < W; ++j) load_n<E, (E % 4 == 0)>(&wsm[j * 32 * E + lane * E], wt[j]);
        if (a.bias) load_n<E, false>(a.bias + c, bias, valid);
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
                if (st) load_n<E, VEC>(st + (size_t)(t + W - 1) * a.C, v, valid);
                else
#pragma unroll
                    for (int i = 0; i < E; ++i) v[i] = 0.f;
            } else {
                load_n<E, VEC>(x + (size_t)t * a.ldx, v, t < len ? valid : 0);
            }
        };
        // rows t-W+1 .. of x and of dp, a batch at a time; the next batch is on its way as loaded
        float win[W - 1 + kBatch][E], dp[W - 1 + kBatch][E];
        Raw<TIn, E> nx[kBatch], ny[kBatch];
        auto fetch = [&](int t) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int n = t + k < min(len, t1 + W - 1) ? valid : 0;
                nx[k].template load<VEC>(x + (size_t)(t + k) * a.ldx, n);
                ny[k].template load<VEC>(dy + (size_t)(t + k) * a.C, n);
            }
        };
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            row(t0 - (W - 1) + j, win[j]);
#pragma unroll
            for (int i = 0; i < E; ++i) dp[j][i] = 0.f;
        }
        fetch(t0);
        for (int t = t0; t < t1 + W - 1; t += kBatch) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                nx[k].widen(win[W - 1 + k]);
                ny[k].widen(dp[W - 1 + k]);
            }
            fetch(t + kBatch);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float *now = dp[W - 1 + k];
                if constexpr (E % 2 == 0) {
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
                        now[i] = d.x;
                        now[i + 1] = d.y;
                    }
                } else if (a.act) {
                    float p = bias[0];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(wt[j][0], win[k + j][0], p);
                    const float g = sigmoid_fast(p);
                    now[0] *= g * fmaf(p, 1.f - g, 1.f);
                }
                if (t + k >= len)   // nothing flows from past the end, whatever p is there
#pragma unroll
                    for (int i = 0; i < E; ++i) now[i] = 0.f;
                if (t + k < t1)
#pragma unroll
                    for (int i = 0; i < E; ++i) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][i] = fmaf(now[i], win[k + j][i], dw[j][i]);
                        dw[W][i] += now[i];
                    }
                const int r = t + k - (W - 1);
                if (r < t1 && (r >= t0 || (ri == 0 && dst))) {
                    float d[E];
                    const int j0 = r - (len - (W - 1));   // this row's place in state_out
                    load_n<E, VEC>(dso + (dso ? (long long)j0 * a.C : 0), d, dso && j0 >= 0 && j0 < W - 1 ? valid : 0);
#pragma unroll
                    for (int i = 0; i < E; ++i)
#pragma unroll
                        for (int j = 0; j < W; ++j) d[i] = fmaf(wt[W - 1 - j][i], dp[k + j][i], d[i]);
                    if (r >= 0) store_n<E, VEC>(dx + (size_t)r * a.C, d, valid);
                    else store_n<E, VEC>(dst + (size_t)(r + W - 1) * a.C, d, valid);
                }
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    win[j][i] = win[j + kBatch][i];
                    dp[j][i] = dp[j + kBatch][i];
                }
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) sums[warp][j][lane * E + i] = dw[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32 * E; i += 32 * kWarps) {
        const int j = i / (32 * E), cc = i % (32 * E);
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) t += sums[k][j][cc];
        if (c0 + cc < a.C) a.part[((size_t)rb * (W + 1) + j) * a.C + c0 + cc] = t;
    }
}

// dw [C][W] and db [C] from part [n][W + 1][C]: 32 columns a block, 8 rows in flight.
__global__ void __launch_bounds__(256)
conv_param_sum_kernel(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ db, int n, int W,
                      int C)
{
    __shared__ float sm[8][33];
    const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y, y = threadIdx.y;
    float t = 0.f;
    if (c < C)
        for (int i = y; i < n; i += 8) t += part[((size_t)i * (W + 1) + j) * C + c];
    sm[y][threadIdx.x] = t;
    __syncthreads();
    if (y == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += sm[i][threadIdx.x];
        if (j < W) dw[(size_t)c * W + j] = t;
        else if (db) db[c] = t;
    }
}

// Tokens of a run: long enough that the W - 1 rows read twice cost little, short enough that
// every SM has the 24 warps whose rows on their way (2 KB a warp) keep HBM busy.
int conv_run(int B, int T, int C, int e)
{
    const long long lanes = (long long)B * ((C + 32 * e - 1) / (32 * e));   // warps per token run
    int run = 64;
    while (run > 8 && lanes * ((T + run - 1) / run) < 152 * 24) run /= 2;
    return run;
}

bool aligned_to(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename TIn, int W>
cudaError_t conv_fwd(const ConvArgs &a, cudaStream_t st)
{
    constexpr int E = 16 / sizeof(TIn);
    const bool vec = a.C % E == 0 && a.ldx % E == 0 && aligned_to(a.x, 16) && aligned_to(a.y, 16) &&
                     aligned_to(a.state, 16) && aligned_to(a.state_out, 16);
    const int run = conv_run(a.B, a.T, a.C, vec ? E : 1), runs = std::max(1, (a.T + run - 1) / run);
    const int cblocks = (a.C + 32 * (vec ? E : 1) - 1) / (32 * (vec ? E : 1));
    const long long blocks = (long long)cblocks * a.B * ((runs + kWarps - 1) / kWarps);
    if (vec) short_conv_kernel<TIn, W, E, true><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    else short_conv_kernel<TIn, W, 1, false><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    return cudaGetLastError();
}

template <typename TIn, int W>
cudaError_t conv_step(const ConvArgs &a, cudaStream_t st)
{
    constexpr int E = 4, A = E * (int)sizeof(TIn);   // a token's work is latency: many small threads
    const bool vec = a.C % E == 0 && a.ldx % E == 0 && aligned_to(a.x, A) && aligned_to(a.y, A) &&
                     aligned_to(a.state, A) && aligned_to(a.state_out, A) && aligned_to(a.w, 16) &&
                     aligned_to(a.bias, 16);
    const long long n = (long long)a.B * ((a.C + (vec ? E : 1) - 1) / (vec ? E : 1));
    const unsigned blocks = (unsigned)((n + 127) / 128);
    if (vec) short_conv_step_kernel<TIn, W, E, true><<<blocks, 128, 0, st>>>(a);
    else short_conv_step_kernel<TIn, W, 1, false><<<blocks, 128, 0, st>>>(a);
    return cudaGetLastError();
}

constexpr int kBwdE = 4;

template <typename TIn, int W>
cudaError_t conv_bwd(const ConvBwdArgs &a, cudaStream_t st)
{
    constexpr int A = kBwdE * sizeof(TIn);
    const bool vec = a.C % kBwdE == 0 && a.ldx % kBwdE == 0 && aligned_to(a.x, A) && aligned_to(a.dy, A) &&
                     aligned_to(a.dx, A) && aligned_to(a.state, A) && aligned_to(a.dstate, A) &&
                     aligned_to(a.dstate_out, A);
    // the run goes by 4 channels a lane whatever the alignment: the workspace's size follows it
    const int run = conv_run(a.B, a.T, a.C, kBwdE), runs = std::max(1, (a.T + run - 1) / run);
    const int per = 32 * (vec ? kBwdE : 1), cblocks = (a.C + per - 1) / per;
    const long long blocks = (long long)cblocks * a.B * ((runs + kWarps - 1) / kWarps);
    if (vec) short_conv_bwd_kernel<TIn, W, kBwdE, true><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    else short_conv_bwd_kernel<TIn, W, 1, false><<<(unsigned)blocks, 32 * kWarps, 0, st>>>(a, run, runs, cblocks);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int n = a.B * ((runs + kWarps - 1) / kWarps);
    conv_param_sum_kernel<<<dim3((a.C + 31) / 32, W + 1), dim3(32, 8), 0, st>>>(a.part, a.dw, a.db, n, W, a.C);
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
    const int run = conv_run(B, T, C, kBwdE), runs = std::max(1, (T + run - 1) / run);
    return (size_t)B * ((runs + kWarps - 1) / kWarps) * (W + 1) * C * sizeof(float);
}

}  // namespace ldn
