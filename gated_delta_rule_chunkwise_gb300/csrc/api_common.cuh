// Argument checks shared by the C entry points of the operators around a token mixer
// (mixer_api.cu, linear_api.cu).
#pragma once
#include "ldn_internal.cuh"

namespace ldn {
namespace {

constexpr long long kMostElements = 1LL << 40;

inline bool at(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool known(int dtype) { return dtype == LDN_F32 || dtype == LDN_BF16; }
inline size_t size_of(int dtype) { return dtype == LDN_BF16 ? 2 : 4; }
inline int status_of(cudaError_t e) { return e == cudaSuccess ? LDN_OK : LDN_ERR_CUDA; }

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
inline Span rows_span(const void *p, long long rows, long long ld, long long width, int dtype)
{
    return {p, p && rows > 0 ? (size_t)((rows - 1) * ld + width) * size_of(dtype) : 0};
}

}  // namespace
}  // namespace ldn
