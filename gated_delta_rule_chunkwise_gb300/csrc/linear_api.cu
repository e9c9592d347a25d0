// C ABI of the projections: argument validation, what is laid out in the workspace, and the
// products of ldn_linear, ldn_linear_e4m3 and ldn_linear_backward (documented in include/ldn.h).
#include "api_common.cuh"
#include "linear_common.cuh"

using namespace ldn;
using linear::Operand;

namespace {

constexpr size_t kAlign = 256;
constexpr long long kMostRow = 1LL << 38;   // elements between rows: TMA takes fewer than 2^40 bytes

// Places in the workspace, one after another.
struct Places {
    size_t bytes = 0;
    size_t take(size_t n)
    {
        const size_t p = bytes;
        bytes += (n + kAlign - 1) / kAlign * kAlign;
        return p;
    }
};

long long padded(long long width, int es) { return (width + 16 / es - 1) / (16 / es) * (16 / es); }

// Whether TMA can read these rows where they are: each begins at a 16-byte boundary.
bool readable(const void *p, long long ld, long long rows, int es)
{
    return at(p, 16) && (rows == 1 || ld * es % 16 == 0);
}

// Rows of an operand, where they are or (`copied`) at `place` of the workspace as planes or rows.
struct Source {
    const void *p;
    long long ld, rows;
    int width;
    bool copied;
    size_t place;
};

Source source(const void *p, long long ld, long long rows, int width, int dtype, int es, Places &ws)
{
    Source s{p, ld, rows, width, dtype == LDN_F32 || !readable(p, ld, rows, es), 0};
    if (s.copied)
        s.place = dtype == LDN_F32 ? ws.take((size_t)linear::kPlanes * rows * padded(width, 2) * 2)
                                   : ws.take((size_t)rows * padded(width, es) * es);
    return s;
}

// Lays out what is not taken where it lies.
cudaError_t prepare(const Source &a, const Source &b, int dtype, int es, char *ws, cudaStream_t st)
{
    if (dtype == LDN_F32) {
        auto split = [&](const Source &s) {
            return linear::Split{(const float *)s.p, ws + s.place, s.ld, padded(s.width, 2), s.copied ? s.rows : 0, s.width};
        };
        return a.copied || b.copied ? linear::split_rows(split(a), split(b), st) : cudaSuccess;
    }
    for (const Source *s : {&a, &b}) {
        if (!s->copied) continue;
        const cudaError_t e = linear::copy_rows(s->p, s->ld, ws + s->place, padded(s->width, es), s->rows, s->width, es, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

Operand operand(const Source &s, int dtype, int es, const char *ws)
{
    if (!s.copied) return {s.p, s.width, s.rows, s.ld, 0, 1};
    const long long ld = padded(s.width, dtype == LDN_F32 ? 2 : es);
    return {ws + s.place, s.width, s.rows, ld, ld * s.rows, dtype == LDN_F32 ? linear::kPlanes : 1};
}

// A product's k blocks and pairs of planes.
linear::Args product(long long ni, long long nj, long long k, int dtype, int es)
{
    linear::Args a = {};
    a.ni = ni;
    a.nj = nj;
    a.kblocks = (int)((k * (dtype == LDN_F32 ? 2 : es) + 127) / 128);
    if (dtype == LDN_F32) {   // mid mid, lo hi, hi lo, mid hi, hi mid, all all
        a.npairs = 6;
        a.pairs_a = 0x301021;
        a.pairs_b = 0x310201;
    } else {
        a.npairs = 1;
    }
    return a;
}

int check_sizes(long long rows, int K, int N, long long ldx, long long ldw, int activation)
{
    if (rows < 0 || K < 1 || N < 1 || ldx < K || ldw < K) return LDN_ERR_INVALID_ARG;
    if (activation < LDN_ACT_NONE || activation > LDN_ACT_GELU) return LDN_ERR_INVALID_ARG;
    constexpr long long most = 0x7fffffffLL - (1 << 16);   // tiles may end a little past the last row
    if (rows > most || K > most || N > most || ldx > kMostRow || ldw > kMostRow) return LDN_ERR_UNSUPPORTED;
    if (std::max(rows, 1LL) > kMostElements / ldx || N > kMostElements / ldw || rows > kMostElements / N)
        return LDN_ERR_UNSUPPORTED;
    // planes of an fp32 operand lie less than 2^40 bytes apart
    if (rows > (kMostElements >> 2) / K || N > (kMostElements >> 2) / K) return LDN_ERR_UNSUPPORTED;
    return LDN_OK;
}

// ---- the forward's ----

struct Forward {
    Places ws;
    Source x, w;
    Forward(const void *px, long long ldx, const void *pw, long long ldw, long long rows, int K, int N, int dtype, int es)
        : x(source(px, ldx, rows, K, dtype, es, ws)), w(source(pw, ldw, N, K, dtype, es, ws))
    {
    }
};

int forward(const void *x, long long ldx, const float *x_scale, const void *weight, long long ldw,
            const float *weight_scale, const void *bias, const void *residual, void *y, void *z, long long rows, int K,
            int N, int activation, int dtype, int out_dtype, bool eight, void *workspace, size_t workspace_bytes,
            void *stream)
{
    if (!known(dtype) || !known(out_dtype)) return LDN_ERR_INVALID_ARG;
    const int st = check_sizes(rows, K, N, ldx, ldw, activation);
    if (st != LDN_OK) return st;
    if (dtype == LDN_F32 && out_dtype != LDN_F32) return LDN_ERR_UNSUPPORTED;
    if (rows == 0) return LDN_OK;
    if (!x || !weight || !y || (eight && (!x_scale || !weight_scale))) return LDN_ERR_INVALID_ARG;
    const int es = eight ? 1 : (int)size_of(dtype);
    const size_t os = size_of(out_dtype), zs = size_of(dtype), n = (size_t)rows * N;
    if (!at(x, es) || !at(weight, es) || !at(bias, zs) || !at(residual, os) || !at(y, os) || !at(z, zs) ||
        !at(x_scale, 4) || !at(weight_scale, 4))
        return LDN_ERR_INVALID_ARG;
    const Forward f(x, ldx, weight, ldw, rows, K, N, dtype, es);
    if (f.ws.bytes && (!workspace || workspace_bytes < f.ws.bytes || !at(workspace, kAlign))) return LDN_ERR_INVALID_ARG;
    auto span = [es](const void *p, long long r, long long ld, long long width) {
        return Span{p, (size_t)((r - 1) * ld + width) * es};
    };
    const Span in[] = {span(x, rows, ldx, K), span(weight, N, ldw, K), {bias, (size_t)N * zs},
                       {x_scale, (size_t)rows * 4}, {weight_scale, (size_t)N * 4},
                       {residual == y ? nullptr : residual, n * os}};   // y may replace the residual
    const Span out[] = {{y, n * os}, {z, n * zs}, {f.ws.bytes ? workspace : nullptr, f.ws.bytes}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    char *ws = (char *)workspace;
    if (prepare(f.x, f.w, dtype, es, ws, s) != cudaSuccess) return LDN_ERR_CUDA;
    linear::Args a = product(N, rows, K, dtype, es);
    a.out = y;
    a.z = z;
    a.bias = bias;
    a.residual = residual;
    a.scale_i = weight_scale;
    a.scale_j = x_scale;
    a.out_f32 = out_dtype == LDN_F32;
    a.z_f32 = a.bias_f32 = dtype == LDN_F32;
    a.activation = activation;
    const Operand A = operand(f.w, dtype, es, ws), B = operand(f.x, dtype, es, ws);
    return status_of(eight ? linear_product_e4m3(A, B, a, s) : linear_product(A, B, a, s));
}

// ---- the gradients' ----

enum { kDx = 1, kDw = 2, kDb = 4 };

struct Backward {
    Places ws;
    Source x{}, w{};
    bool form = false;       // dz is formed: rounded, or laid out as planes or padded rows
    size_t dz = 0, part = 0;
    long long ld_dz = 0;
    Backward(const void *dy, const void *px, long long ldx, const void *pw, long long ldw, long long rows, int K, int N,
             int activation, int dtype, int dy_dtype, int want)
    {
        const int es = dtype == LDN_F32 ? 4 : 2;
        if (want & kDx) w = source(pw, ldw, N, K, dtype, es, ws);
        if (want & kDw) x = source(px, ldx, rows, K, dtype, es, ws);
        ld_dz = padded(N, 2);
        form = (want & (kDx | kDw)) &&
               (activation != LDN_ACT_NONE || dy_dtype == LDN_F32 || !readable(dy, N, rows, 2));
        if (form) dz = ws.take((size_t)(dtype == LDN_F32 ? linear::kPlanes : 1) * rows * ld_dz * 2);
        if (want & kDb) part = ws.take((size_t)linear::dz_runs(rows, N) * N * sizeof(float));
    }
};

}  // namespace

extern "C" int ldn_linear(const void *x, long long ldx, const void *weight, long long ldw, const void *bias,
                          const void *residual, void *y, void *z, long long rows, int K, int N, int activation,
                          int dtype, int out_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    return forward(x, ldx, nullptr, weight, ldw, nullptr, bias, residual, y, z, rows, K, N, activation, dtype,
                   out_dtype, false, workspace, workspace_bytes, stream);
}

extern "C" size_t ldn_linear_workspace_size(const void *x, long long ldx, const void *weight, long long ldw,
                                            long long rows, int K, int N, int dtype)
{
    if (!known(dtype) || check_sizes(rows, K, N, ldx, ldw, LDN_ACT_NONE) != LDN_OK || rows == 0) return 0;
    return Forward(x, ldx, weight, ldw, rows, K, N, dtype, (int)size_of(dtype)).ws.bytes;
}

extern "C" int ldn_linear_e4m3(const void *x, long long ldx, const float *x_scale, const void *weight, long long ldw,
                               const float *weight_scale, const void *bias, const void *residual, void *y,
                               long long rows, int K, int N, int activation, int out_dtype, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    return forward(x, ldx, x_scale, weight, ldw, weight_scale, bias, residual, y, nullptr, rows, K, N, activation,
                   LDN_BF16, out_dtype, true, workspace, workspace_bytes, stream);
}

extern "C" size_t ldn_linear_e4m3_workspace_size(const void *x, long long ldx, const void *weight, long long ldw,
                                                 long long rows, int K, int N)
{
    if (check_sizes(rows, K, N, ldx, ldw, LDN_ACT_NONE) != LDN_OK || rows == 0) return 0;
    return Forward(x, ldx, weight, ldw, rows, K, N, LDN_BF16, 1).ws.bytes;
}

extern "C" size_t ldn_linear_backward_workspace_size(const void *dy, const void *x, long long ldx, const void *weight,
                                                     long long ldw, long long rows, int K, int N, int activation,
                                                     int dtype, int dy_dtype, int want)
{
    if (!known(dtype) || !known(dy_dtype) || check_sizes(rows, K, N, ldx, ldw, activation) != LDN_OK || rows == 0)
        return 0;
    return Backward(dy, x, ldx, weight, ldw, rows, K, N, activation, dtype, dy_dtype, want).ws.bytes;
}

extern "C" int ldn_linear_backward(const void *dy, const void *x, long long ldx, const void *weight, long long ldw,
                                   const void *z, void *dx, void *dweight, void *dbias, long long rows, int K, int N,
                                   int activation, int dtype, int dy_dtype, void *workspace, size_t workspace_bytes,
                                   void *stream)
{
    if (!known(dtype) || !known(dy_dtype)) return LDN_ERR_INVALID_ARG;
    const int st = check_sizes(rows, K, N, ldx, ldw, activation);
    if (st != LDN_OK) return st;
    if (dtype == LDN_F32 && dy_dtype != LDN_F32) return LDN_ERR_UNSUPPORTED;
    const int es = (int)size_of(dtype);
    const size_t ys = size_of(dy_dtype), n = (size_t)rows * N;
    if (!at(dy, ys) || !at(x, es) || !at(weight, es) || !at(z, es) || !at(dx, es) || !at(dweight, es) || !at(dbias, es))
        return LDN_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {   // sums of nothing
        if (dweight && cudaMemsetAsync(dweight, 0, (size_t)N * K * es, s) != cudaSuccess) return LDN_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)N * es, s) != cudaSuccess) return LDN_ERR_CUDA;
        return LDN_OK;
    }
    const int want = (dx ? kDx : 0) | (dweight ? kDw : 0) | (dbias ? kDb : 0);
    if (!dy || (dx && !weight) || (dweight && !x) || (activation != LDN_ACT_NONE && want && !z)) return LDN_ERR_INVALID_ARG;
    const Backward b(dy, x, ldx, weight, ldw, rows, K, N, activation, dtype, dy_dtype, want);
    if (b.ws.bytes && (!workspace || workspace_bytes < b.ws.bytes || !at(workspace, kAlign))) return LDN_ERR_INVALID_ARG;
    const Span in[] = {{dy, n * ys}, rows_span(x, rows, ldx, K, dtype), rows_span(weight, N, ldw, K, dtype),
                       {activation ? z : nullptr, n * es}};
    const Span out[] = {{dx, (size_t)rows * K * es}, {dweight, (size_t)N * K * es}, {dbias, (size_t)N * es},
                        {b.ws.bytes ? workspace : nullptr, b.ws.bytes}};
    if (overlapping(in, out)) return LDN_ERR_INVALID_ARG;
    char *ws = (char *)workspace;
    const bool planes = dtype == LDN_F32;
    const long long plane = b.ld_dz * rows;
    if (b.form || dbias) {
        const cudaError_t e = linear::form_dz(dy, dy_dtype == LDN_F32, activation ? z : nullptr, activation,
                                              b.form ? ws + b.dz : nullptr, b.ld_dz, plane, planes,
                                              dbias ? (float *)(ws + b.part) : nullptr, dbias, planes, rows, N, s);
        if (e != cudaSuccess) return LDN_ERR_CUDA;
    }
    const Operand dz = b.form ? Operand{ws + b.dz, N, rows, b.ld_dz, plane, planes ? linear::kPlanes : 1}
                              : Operand{dy, N, rows, N, 0, 1};
    if (prepare(b.x, b.w, dtype, es, ws, s) != cudaSuccess) return LDN_ERR_CUDA;
    if (dx) {
        linear::Args a = product(K, rows, N, dtype, es);
        a.out = dx;
        a.out_f32 = planes;
        if (linear_product_dx(operand(b.w, dtype, es, ws), dz, a, s) != cudaSuccess) return LDN_ERR_CUDA;
    }
    if (dweight) {
        linear::Args a = product(K, N, rows, dtype, es);
        a.out = dweight;
        a.out_f32 = planes;
        if (linear_product_dw(operand(b.x, dtype, es, ws), dz, a, s) != cudaSuccess) return LDN_ERR_CUDA;
    }
    return LDN_OK;
}
