// mx_checks.h -- argument checks of the C entry points that take matrices: sizes, pointers,
// distances of rows, and results that share memory with something else of the call.
#pragma once

#include "bitopt.h"
#include "launch.h"
#include "mx_overlap.h"

namespace bitopt {

constexpr int64_t kMaxDim = int64_t{1} << 30;    // sizes, rounded up to a tile, are int32 in the kernels

inline bool valid_dtype(int32_t d) { return d == BITOPT_F32 || d == BITOPT_F16 || d == BITOPT_BF16; }
inline uintptr_t elem_mask(int32_t d) { return d == BITOPT_F32 ? 3 : 1; }
inline bool aligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) == 0; }

inline int check_dim(int64_t v, const char* name, const char* fn) {
    if (v < 0) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s < 0", fn, name);
    if (v > kMaxDim) return api_fail(BITOPT_ERR_UNSUPPORTED, "%s: %s above %lld", fn, name, (long long)kMaxDim);
    return BITOPT_OK;
}

// A row-major matrix of elements: pointer, alignment to the element, distance of rows.
inline int check_matrix(const void* p, int32_t dtype, int64_t ld, int64_t rows, int64_t cols, const char* name, const char* fn) {
    if (!p) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (!aligned(p, elem_mask(dtype)))
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", fn, name);
    if (rows > 1 && ld < cols)
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: rows of %s are %lld elements apart but hold %lld", fn, name,
                        (long long)ld, (long long)cols);
    return BITOPT_OK;
}

inline int check_codes(const void* codes, const void* scales, const char* name, const char* fn) {
    if (!codes || !scales) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: NULL codes or scales of %s", fn, name);
    if (!aligned(codes, 15) || !aligned(scales, 15))
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: codes and scales of %s must be aligned to 16 bytes", fn, name);
    return BITOPT_OK;
}

// A matrix of a call, for the check that results share no memory with anything else of it.
struct Named {
    const char* name;
    ByteRows at;
};
inline Named elements(const char* name, const void* p, int32_t dtype, int64_t ld, int64_t rows, int64_t cols) {
    const int64_t es = dtype == BITOPT_F32 ? 4 : 2;
    // distances beyond 2^60 elements are no memory: one that still fits 64 bits stands for them
    return {name, {p, rows, cols * es, std::min<int64_t>(ld, int64_t{1} << 60) * es}};
}
inline Named packed(const char* name, const void* p, int64_t rows, int64_t width) { return {name, {p, rows, width, width}}; }

// The first `results` of the matrices are written: none may meet another.  The first `in_place` of
// those are laid out as the read matrices at `over` or `over2` and written item by item after the
// reads of the same items, so they may lie over the very same rows.
template <size_t N> int check_apart(const char* fn, size_t results, const Named (&m)[N], size_t in_place = 0,
                                    const void* over = nullptr, const void* over2 = nullptr) {
    for (size_t r = 0; r < results; ++r)
        for (size_t i = r + 1; i < N; ++i) {
            const ByteRows &a = m[r].at, &b = m[i].at;
            if (!rows_meet(a, b)) continue;
            if (r < in_place && i >= results && a.p == b.p && (b.p == over || b.p == over2) &&
                (a.rows == 1 || a.stride == b.stride))
                continue;
            return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, m[r].name, m[i].name);
        }
    return BITOPT_OK;
}

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace bitopt

#define BITOPT_TRY(call)          \
    do {                          \
        if (int rc = (call)) return rc; \
    } while (0)

