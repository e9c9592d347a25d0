// C ABI of the operators around a token mixer: argument validation and dispatch of
// ldn_add_rmsnorm*, ldn_short_conv* and ldn_ssm_* (documented in include/ldn.h).
#include "ldn_internal.cuh"

using namespace ldn;

namespace {

constexpr long long kMostElements = 1LL << 40;

bool at(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool known(int dtype) { return dtype == LDN_F32 || dtype == LDN_BF16; }
size_t size_of(int dtype) { return dtype == LDN_BF16 ? 2 : 4; }
int status_of(cudaError_t e) { return e == cudaSuccess ? LDN_OK : LDN_ERR_CUDA; }

// A stretch of device memory (bytes 0: absent).
struct Span {
    const void *p;
    size_t bytes;
    bool hits(const Span &o) const
    {
        if (!p || !o.p || !bytes || !o.bytes) return false;
        const uintptr_t a = (uintptr_t)p, b = (uintptr_t)o.p;
        return a < b + o.bytes && b < a + bytes;
    }
};

// Whether some output overlaps an input or another output.
template <size_t NI, size_t NO>
bool overlapping(const Span (&in)[NI], const Span (&out)[NO])
{
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (out[i].hits(in[j])) return true;
        for (size_t j = 0; j < i; ++j)
            if (out[i].hits(out[j])) return true;
    }
    return false;
}

// Bytes from the first to the last element of `rows` rows of `width`, `ld` apart.
Span rows_span(const void *p, long long rows, long long ld, long long width, int dtype)
{
    return {p, p && rows > 0 ? (size_t)((rows - 1) * ld + width) * size_of(dtype) : 0};
}

}  // namespace

// ---- RMS norm with the residual's addition ----

static int norm_impl(const void *x, const void *residual, const float *weight, void *y, float *scale,
                     void *residual_out, long long rows, int D, int group, int dtype, int res_dtype, float eps,
                     bool eight, void *stream)
{
    if (!known(dtype) || !known(res_dtype)) return LDN_ERR_INVALID_ARG;
    if (rows < 0 || D < 1 || !(eps >= 0.f) || eps > 1e30f) return LDN_ERR_INVALID_ARG;
    if (eight && group != 0 && group != 128) return LDN_ERR_UNSUPPORTED;
    if (dtype == LDN_F32 && res_dtype != LDN_F32) return LDN_ERR_UNSUPPORTED;
    if (D > 32768 || rows > 0x7fffffffLL || rows * D > kMostElements) return LDN_ERR_UNSUPPORTED;
    if (rows == 0) return LDN_OK;
    if (!x || !weight || !y || (eight && !scale) || !residual != !residual_out) return LDN_ERR_INVALID_ARG;
    const size_t es = size_of(dtype), rs = size_of(res_dtype), n = (size_t)rows * D;
    if (!at(x, es) || !at(y, eight ? 1 : es) || !at(residual, rs) || !at(residual_out, rs) || !at(weight, 4) ||
        !at(scale, 4))
        return LDN_ERR_INVALID_ARG;
    const size_t nscale = !eight ? 0 : (size_t)rows * (group ? (D + 127) / 128 : 1);
    const Span in[] = {{x, n * es}, {weight, (size_t)D * 4},
                       {residual == residual_out ? nullptr : residual, n * rs}};   // the sum may replace the residual
    const Span out[] = {{y, n * (eight ? 1 : es)}, {scale, nscale * 4}, {residual_out, n * rs}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    const AddNormArgs a{x, residual, weight, y, eight ? scale : nullptr, residual_out, rows, D, group, dtype,
                        res_dtype, eps};
    return status_of(launch_add_rmsnorm(a, (cudaStream_t)stream));
}

extern "C" int ldn_add_rmsnorm(const void *x, const void *residual, const float *weight, void *y,
                               void *residual_out, long long rows, int D, int dtype, int residual_dtype, float eps,
                               void *stream)
{
    return norm_impl(x, residual, weight, y, nullptr, residual_out, rows, D, 0, dtype, residual_dtype, eps, false,
                     stream);
}

extern "C" int ldn_add_rmsnorm_e4m3(const void *x, const void *residual, const float *weight, void *q, float *scale,
                                    void *residual_out, long long rows, int D, int group, int dtype,
                                    int residual_dtype, float eps, void *stream)
{
    return norm_impl(x, residual, weight, q, scale, residual_out, rows, D, group, dtype, residual_dtype, eps, true,
                     stream);
}

static int check_norm_bwd(long long rows, int D)
{
    if (rows < 0 || D < 1) return LDN_ERR_INVALID_ARG;
    if (D > 32768 || rows > 0x7fffffffLL || rows * D > kMostElements) return LDN_ERR_UNSUPPORTED;
    return LDN_OK;
}

extern "C" size_t ldn_add_rmsnorm_backward_workspace_size(long long rows, int D)
{
    if (check_norm_bwd(rows, D) != LDN_OK) return 0;
    return (size_t)add_rmsnorm_bwd_blocks(rows, D) * D * sizeof(float);
}

extern "C" int ldn_add_rmsnorm_backward(const void *dy, const void *s, const float *weight, const void *dsum,
                                        void *dx, void *dresidual, float *dweight, long long rows, int D, int dtype,
                                        int residual_dtype, float eps, void *workspace, size_t workspace_bytes,
                                        void *stream)
{
    if (!known(dtype) || !known(residual_dtype) || !(eps >= 0.f) || eps > 1e30f) return LDN_ERR_INVALID_ARG;
    const int st = check_norm_bwd(rows, D);
    if (st != LDN_OK) return st;
    if (dtype == LDN_F32 && residual_dtype != LDN_F32) return LDN_ERR_UNSUPPORTED;
    if (!weight || !dweight || !at(weight, 4) || !at(dweight, 4)) return LDN_ERR_INVALID_ARG;
    const size_t need = ldn_add_rmsnorm_backward_workspace_size(rows, D), es = size_of(dtype),
                 rs = size_of(residual_dtype), n = (size_t)rows * D;
    if (rows > 0 && (!dy || !s || !workspace || workspace_bytes < need || !at(workspace, 16)))
        return LDN_ERR_INVALID_ARG;
    if (!at(dy, es) || !at(dx, es) || !at(s, rs) || !at(dsum, rs) || !at(dresidual, rs)) return LDN_ERR_INVALID_ARG;
    const Span in[] = {{dy, n * es}, {s, n * rs}, {weight, (size_t)D * 4}, {dsum, n * rs}};
    const Span out[] = {{dx, n * es}, {dresidual, n * rs}, {dweight, (size_t)D * 4}, {workspace, need}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    const AddNormBwdArgs a{dy, s, weight, dsum, dx, dresidual, dweight, (float *)workspace, rows, D, dtype,
                           residual_dtype, eps};
    return status_of(launch_add_rmsnorm_bwd(a, (cudaStream_t)stream));
}

// ---- Short causal convolution with a carried state ----

// Tokens of a sequence, and channels: runs, segments and blocks of channels may end a little past them.
constexpr int kMostInt = 0x7fffffff - (1 << 16);

static int check_conv(int B, int T, int C, int W, int dtype, long long ldx)
{
    if (!known(dtype) || B < 1 || T < 0 || C < 1 || W < 1 || ldx < C) return LDN_ERR_INVALID_ARG;
    if (W > 8 || T > kMostInt || C > kMostInt) return LDN_ERR_UNSUPPORTED;
    // elements from the first row to the last, and blocks of one launch (eight tokens of 32 channels each at least)
    if (ldx > kMostElements || (long long)B * std::max(T, W) > kMostElements / ldx) return LDN_ERR_UNSUPPORTED;
    if ((long long)B * ((T + 7LL) / 8) * ((C + 31) / 32) > 0x7fffffffLL) return LDN_ERR_UNSUPPORTED;
    return LDN_OK;
}

extern "C" int ldn_short_conv(const void *x, long long ldx, const float *weight, const float *bias,
                              const void *state, const int *lens, void *y, void *state_out, int B, int T, int C,
                              int width, int activation, int dtype, void *stream)
{
    const int st = check_conv(B, T, C, width, dtype, ldx);
    if (st != LDN_OK) return st;
    if (activation != 0 && activation != 1) return LDN_ERR_INVALID_ARG;
    if (!weight || (T > 0 && (!x || !y))) return LDN_ERR_INVALID_ARG;
    const size_t es = size_of(dtype), ns = (size_t)B * (width - 1) * C * es;
    if (!at(x, es) || !at(y, es) || !at(state, es) || !at(state_out, es) || !at(weight, 4) || !at(bias, 4) ||
        !at(lens, 4))
        return LDN_ERR_INVALID_ARG;
    if (T == 0 && !state_out) return LDN_OK;
    const Span in[] = {rows_span(x, (long long)B * T, ldx, C, dtype), {weight, (size_t)C * width * 4},
                       {bias, (size_t)C * 4}, {lens, (size_t)B * 4},
                       {state == state_out ? nullptr : state, ns}};   // the new state may replace the old one
    const Span out[] = {{y, (size_t)B * T * C * es}, {state_out, ns}};
    if (overlapping(in, out) || (state && Span{state, ns}.hits(out[0]))) return LDN_ERR_INVALID_ARG;
    const ConvArgs a{x, ldx, weight, bias, state, state_out, lens, y, B, T, C, width, activation, dtype};
    return status_of(launch_short_conv(a, (cudaStream_t)stream));
}

extern "C" int ldn_short_conv_step(const void *x, long long ldx, const float *weight, const float *bias,
                                   const void *state, void *y, void *state_out, int B, int C, int width,
                                   int activation, int dtype, void *stream)
{
    const int st = check_conv(B, 1, C, width, dtype, ldx);
    if (st != LDN_OK) return st;
    if (activation != 0 && activation != 1) return LDN_ERR_INVALID_ARG;
    if (!weight || !x || !y || (width > 1 && (!state || !state_out))) return LDN_ERR_INVALID_ARG;
    const size_t es = size_of(dtype), ns = (size_t)B * (width - 1) * C * es;
    if (!at(x, es) || !at(y, es) || !at(state, es) || !at(state_out, es) || !at(weight, 4) || !at(bias, 4))
        return LDN_ERR_INVALID_ARG;
    const Span in[] = {rows_span(x, B, ldx, C, dtype), {weight, (size_t)C * width * 4}, {bias, (size_t)C * 4},
                       {state == state_out ? nullptr : state, ns}};
    const Span out[] = {{y, (size_t)B * C * es}, {state_out, ns}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    const ConvArgs a{x, ldx, weight, bias, state, state_out, nullptr, y, B, 1, C, width, activation, dtype};
    return status_of(launch_short_conv_step(a, (cudaStream_t)stream));
}

extern "C" size_t ldn_short_conv_backward_workspace_size(int B, int T, int C, int width)
{
    if (check_conv(B, T, C, width, LDN_BF16, C) != LDN_OK) return 0;
    return short_conv_bwd_workspace_bytes(B, T, C, width);
}

extern "C" int ldn_short_conv_backward(const void *x, long long ldx, const float *weight, const float *bias,
                                       const void *state, const int *lens, const void *dy, const void *dstate_out,
                                       void *dx, float *dweight, float *dbias, void *dstate, int B, int T, int C,
                                       int width, int activation, int dtype, void *workspace,
                                       size_t workspace_bytes, void *stream)
{
    const int st = check_conv(B, T, C, width, dtype, ldx);
    if (st != LDN_OK) return st;
    if (activation != 0 && activation != 1) return LDN_ERR_INVALID_ARG;
    const size_t need = ldn_short_conv_backward_workspace_size(B, T, C, width);
    if (need == 0) return LDN_ERR_UNSUPPORTED;
    if (!weight || !dweight || (T > 0 && (!x || !dy || !dx))) return LDN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need || !at(workspace, 16)) return LDN_ERR_INVALID_ARG;
    const size_t es = size_of(dtype), ns = (size_t)B * (width - 1) * C * es, n = (size_t)B * T * C * es;
    if (!at(x, es) || !at(dy, es) || !at(dx, es) || !at(state, es) || !at(dstate, es) || !at(dstate_out, es) ||
        !at(weight, 4) || !at(bias, 4) || !at(lens, 4) || !at(dweight, 4) || !at(dbias, 4))
        return LDN_ERR_INVALID_ARG;
    const Span in[] = {rows_span(x, (long long)B * T, ldx, C, dtype), {weight, (size_t)C * width * 4},
                       {bias, (size_t)C * 4}, {lens, (size_t)B * 4}, {state, ns}, {dy, n}, {dstate_out, ns}};
    const Span out[] = {{dx, n}, {dweight, (size_t)C * width * 4}, {dbias, (size_t)C * 4}, {dstate, ns},
                        {workspace, need}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    const ConvBwdArgs a{x, ldx, weight, bias, state, lens, dy, dstate_out, dx, dweight, dbias, dstate,
                        (float *)workspace, B, T, C, width, activation, dtype};
    return status_of(launch_short_conv_bwd(a, (cudaStream_t)stream));
}

// ---- Selective state space scan ----

static int check_ssm(int B, int T, int D, int N, int G, int dtype)
{
    if (!known(dtype) || B < 1 || T < 0 || D < 1 || N < 1 || G < 1 || D % G != 0) return LDN_ERR_INVALID_ARG;
    if (!ssm_supported_n(N) || T > kMostInt || D > kMostInt) return LDN_ERR_UNSUPPORTED;
    // elements of [B][T][D], of [B][D][N], and blocks of one launch (32 tokens of 16 channels at least)
    if ((long long)B * std::max(T, N) > kMostElements / D) return LDN_ERR_UNSUPPORTED;
    if ((long long)B * ((T + 31LL) / 32 + 1) > 0x7fffffffLL / ((long long)G * (D / G / 16 + 1))) return LDN_ERR_UNSUPPORTED;
    return LDN_OK;
}

// Row distances: at least a row, and the tensor's extent within bounds.
static bool ssm_ld_ok(long long ld, long long width, long long rows)
{
    return ld >= width && ld <= kMostElements && rows <= kMostElements / ld;
}

extern "C" size_t ldn_ssm_scan_workspace_size(int B, int T, int D, int N, int G)
{
    if (check_ssm(B, T, D, N, G, LDN_BF16) != LDN_OK) return 0;
    return ssm_scan_workspace_bytes(B, T, D, N, G);
}

extern "C" int ldn_ssm_scan(const void *u, long long ldu, const void *delta, long long ld_delta, const float *A,
                            const void *Bm, long long ldb, const void *Cm, long long ldc, const float *Dskip,
                            const void *z, long long ldz, const float *delta_bias, const float *h0, const int *lens,
                            void *y, float *h_final, float *states, int B, int T, int D, int N, int G,
                            int delta_softplus, int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    const int st = check_ssm(B, T, D, N, G, dtype);
    if (st != LDN_OK) return st;
    if (delta_softplus != 0 && delta_softplus != 1) return LDN_ERR_INVALID_ARG;
    const long long rows = (long long)B * T, gn = (long long)G * N;
    if (!ssm_ld_ok(ldu, D, rows) || !ssm_ld_ok(ld_delta, D, rows) || !ssm_ld_ok(ldb, gn, rows) ||
        !ssm_ld_ok(ldc, gn, rows) || (z && !ssm_ld_ok(ldz, D, rows)))
        return LDN_ERR_INVALID_ARG;
    if (!A || (T > 0 && (!u || !delta || !Bm || !Cm || !y))) return LDN_ERR_INVALID_ARG;
    const size_t es = size_of(dtype), nh = (size_t)B * D * N * 4;
    if (!at(u, es) || !at(delta, es) || !at(Bm, es) || !at(Cm, es) || !at(z, es) || !at(y, es) || !at(A, 4) ||
        !at(Dskip, 4) || !at(delta_bias, 4) || !at(lens, 4) || !at(h0, 16) || !at(h_final, 16) || !at(states, 16) ||
        !at(workspace, 16))
        return LDN_ERR_INVALID_ARG;
    if (T == 0 && !h_final) return LDN_OK;
    const Span in[] = {rows_span(u, rows, ldu, D, dtype), rows_span(delta, rows, ld_delta, D, dtype),
                       {A, (size_t)D * N * 4}, rows_span(Bm, rows, ldb, gn, dtype),
                       rows_span(Cm, rows, ldc, gn, dtype), {Dskip, (size_t)D * 4}, rows_span(z, rows, ldz, D, dtype),
                       {delta_bias, (size_t)D * 4}, {h0, nh}, {lens, (size_t)B * 4}};
    // a workspace that is too small stays unused: the scan runs unsplit
    const size_t need = ldn_ssm_scan_workspace_size(B, T, D, N, G);
    if (workspace_bytes < need) workspace = nullptr;
    const Span out[] = {{y, (size_t)rows * D * es}, {h_final, nh},
                        {states, nh * (size_t)((T + kSsmChunk - 1) / kSsmChunk)}, {workspace, need}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    const SsmArgs a{u, delta, Bm, Cm, z, ldu, ld_delta, ldb, ldc, ldz, A, Dskip, delta_bias, h0, lens, y, h_final,
                    states, (float *)workspace, workspace ? workspace_bytes : 0, B, T, D, N, G, delta_softplus,
                    dtype};
    return status_of(launch_ssm_scan(a, (cudaStream_t)stream));
}

extern "C" int ldn_ssm_step(const void *u, long long ldu, const void *delta, long long ld_delta, const float *A,
                            const void *Bm, long long ldb, const void *Cm, long long ldc, const float *Dskip,
                            const void *z, long long ldz, const float *delta_bias, const float *h, float *h_out,
                            void *y, int B, int D, int N, int G, int delta_softplus, int dtype, void *stream)
{
    const int st = check_ssm(B, 1, D, N, G, dtype);
    if (st != LDN_OK) return st;
    if ((long long)B * D > 0x7fffffffLL * 256 / N) return LDN_ERR_UNSUPPORTED;
    if (delta_softplus != 0 && delta_softplus != 1) return LDN_ERR_INVALID_ARG;
    const long long gn = (long long)G * N;
    if (!ssm_ld_ok(ldu, D, B) || !ssm_ld_ok(ld_delta, D, B) || !ssm_ld_ok(ldb, gn, B) || !ssm_ld_ok(ldc, gn, B) ||
        (z && !ssm_ld_ok(ldz, D, B)))
        return LDN_ERR_INVALID_ARG;
    if (!A || !u || !delta || !Bm || !Cm || !y || !h || !h_out) return LDN_ERR_INVALID_ARG;
    const size_t es = size_of(dtype), nh = (size_t)B * D * N * 4;
    if (!at(u, es) || !at(delta, es) || !at(Bm, es) || !at(Cm, es) || !at(z, es) || !at(y, es) || !at(A, 4) ||
        !at(Dskip, 4) || !at(delta_bias, 4) || !at(h, 16) || !at(h_out, 16))
        return LDN_ERR_INVALID_ARG;
    const Span in[] = {rows_span(u, B, ldu, D, dtype), rows_span(delta, B, ld_delta, D, dtype),
                       {A, (size_t)D * N * 4}, rows_span(Bm, B, ldb, gn, dtype), rows_span(Cm, B, ldc, gn, dtype),
                       {Dskip, (size_t)D * 4}, rows_span(z, B, ldz, D, dtype), {delta_bias, (size_t)D * 4},
                       {h == h_out ? nullptr : h, nh}};   // in place: the state may replace itself
    const Span out[] = {{y, (size_t)B * D * es}, {h_out, nh}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    const SsmArgs a{u, delta, Bm, Cm, z, ldu, ld_delta, ldb, ldc, ldz, A, Dskip, delta_bias, h, nullptr, y, h_out,
                    nullptr, nullptr, 0, B, 1, D, N, G, delta_softplus, dtype};
    return status_of(launch_ssm_step(a, (cudaStream_t)stream));
}

extern "C" size_t ldn_ssm_backward_workspace_size(int B, int T, int D, int N, int G)
{
    if (check_ssm(B, T, D, N, G, LDN_BF16) != LDN_OK) return 0;
    return ssm_backward_workspace_bytes(B, T, D, N, G);
}

extern "C" int ldn_ssm_backward(const void *u, long long ldu, const void *delta, long long ld_delta, const float *A,
                                const void *Bm, long long ldb, const void *Cm, long long ldc, const float *Dskip,
                                const void *z, long long ldz, const float *delta_bias, const float *states,
                                const int *lens, const void *dy, const float *dh_final, void *du, void *ddelta,
                                float *dA, void *dB, void *dC, float *dD, void *dz, float *ddelta_bias, float *dh0,
                                int B, int T, int D, int N, int G, int delta_softplus, int dtype, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    const int st = check_ssm(B, T, D, N, G, dtype);
    if (st != LDN_OK) return st;
    if (delta_softplus != 0 && delta_softplus != 1) return LDN_ERR_INVALID_ARG;
    const long long rows = (long long)B * T, gn = (long long)G * N;
    if (!ssm_ld_ok(ldu, D, rows) || !ssm_ld_ok(ld_delta, D, rows) || !ssm_ld_ok(ldb, gn, rows) ||
        !ssm_ld_ok(ldc, gn, rows) || (z && !ssm_ld_ok(ldz, D, rows)))
        return LDN_ERR_INVALID_ARG;
    if (!A || !dA || !z != !dz || (T > 0 && (!u || !delta || !Bm || !Cm || !states || !dy || !du || !ddelta || !dB || !dC)))
        return LDN_ERR_INVALID_ARG;
    const size_t es = size_of(dtype), nh = (size_t)B * D * N * 4, n = (size_t)rows * D * es,
                 need = ldn_ssm_backward_workspace_size(B, T, D, N, G);
    if (T > 0 && (!workspace || workspace_bytes < need)) return LDN_ERR_INVALID_ARG;
    const void *elems[] = {u, delta, Bm, Cm, z, dy, du, ddelta, dB, dC, dz};
    for (const void *p : elems)
        if (!at(p, es)) return LDN_ERR_INVALID_ARG;
    if (!at(A, 4) || !at(Dskip, 4) || !at(delta_bias, 4) || !at(lens, 4) || !at(dA, 4) || !at(dD, 4) ||
        !at(ddelta_bias, 4) || !at(states, 16) || !at(dh_final, 16) || !at(dh0, 16) || !at(workspace, 16))
        return LDN_ERR_INVALID_ARG;
    const Span in[] = {rows_span(u, rows, ldu, D, dtype), rows_span(delta, rows, ld_delta, D, dtype),
                       {A, (size_t)D * N * 4}, rows_span(Bm, rows, ldb, gn, dtype),
                       rows_span(Cm, rows, ldc, gn, dtype), {Dskip, (size_t)D * 4}, rows_span(z, rows, ldz, D, dtype),
                       {delta_bias, (size_t)D * 4}, {lens, (size_t)B * 4}, {dy, n}, {dh_final, nh},
                       {states, nh * (size_t)((T + kSsmChunk - 1) / kSsmChunk)}};
    const Span out[] = {{du, n}, {ddelta, n}, {dA, (size_t)D * N * 4}, {dB, (size_t)(rows * gn) * es},
                        {dC, (size_t)(rows * gn) * es}, {dD, (size_t)D * 4}, {dz, n}, {ddelta_bias, (size_t)D * 4},
                        {dh0, nh}, {workspace, need}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    const SsmBwdArgs a{u, delta, Bm, Cm, z, ldu, ld_delta, ldb, ldc, ldz, A, Dskip, delta_bias, states, lens, dy,
                       dh_final, du, ddelta, dB, dC, dz, dA, dD, ddelta_bias, dh0, (float *)workspace, B, T, D, N, G,
                       delta_softplus, dtype};
    return status_of(launch_ssm_backward(a, (cudaStream_t)stream));
}
