// f8_api.cpp -- the C ABI of the F8 operators (declared in include/bitopt.h): argument
// checks and dispatch.
#include "f8.h"
#include "mx_checks.h"

namespace {

using namespace bitopt;

constexpr int64_t kMaxK = int64_t{1} << 24;      // offsets within a tile of 256 rows stay below 2^32

int check_form(int32_t format, int32_t blocks, const char* fn) {
    if (format != BITOPT_F8_E4M3 && format != BITOPT_F8_E5M2)
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown F8 format %d", fn, format);
    if (blocks != BITOPT_F8_ROWS && blocks != BITOPT_F8_TILES)
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown blocks %d", fn, blocks);
    return BITOPT_OK;
}

int check_type(int32_t dtype, const char* fn) {
    return valid_dtype(dtype) ? BITOPT_OK : api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
}

int64_t scale_count(int64_t rows, int64_t cols, int32_t blocks) {
    return (blocks == BITOPT_F8_TILES ? f8_blocks(rows) : rows) * f8_blocks(cols);
}

Named codes_of(const char* name, const void* p, int64_t rows, int64_t cols) { return packed(name, p, rows, f8_padded(cols)); }
Named scales_of(const char* name, const void* p, int64_t rows, int64_t cols, int32_t blocks) {
    return packed(name, p, 1, 4 * scale_count(rows, cols, blocks));
}

}  // namespace

extern "C" {

int64_t bitopt_f8_code_bytes(int64_t cols) { return cols < 0 || cols > kMaxDim ? -1 : f8_padded(cols); }

int64_t bitopt_f8_scale_count(int64_t rows, int64_t cols, int32_t blocks) {
    if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return -1;
    return blocks == BITOPT_F8_ROWS || blocks == BITOPT_F8_TILES ? scale_count(rows, cols, blocks) : -1;
}

int bitopt_f8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, int32_t format,
                       int32_t blocks, uint8_t* codes, float* scales, uint8_t* codes_t, float* scales_t, void* stream) {
    const char* fn = "bitopt_f8_quantize";
    BITOPT_TRY(check_type(dtype, fn));
    BITOPT_TRY(check_form(format, blocks, fn));
    BITOPT_TRY(check_dim(rows, "rows", fn));
    BITOPT_TRY(check_dim(cols, "cols", fn));
    if (rows == 0 || cols == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_matrix(x, dtype, ldx, rows, cols, "x", fn));
    if ((codes || scales) || !(codes_t || scales_t)) BITOPT_TRY(check_codes(codes, scales, "x", fn));
    if (codes_t || scales_t) BITOPT_TRY(check_codes(codes_t, scales_t, "x transposed", fn));
    BITOPT_TRY(check_apart(fn, 4, {codes_of("codes", codes, rows, cols), scales_of("scales", scales, rows, cols, blocks),
                                   codes_of("codes of the transpose", codes_t, cols, rows),
                                   scales_of("scales of the transpose", scales_t, cols, rows, blocks),
                                   elements("x", x, dtype, ldx, rows, cols)}));
    F8CodecArgs a{};
    a.x = x; a.ldx = ldx; a.rows = rows; a.cols = cols;
    a.codes = codes; a.scales = scales; a.codes_t = codes_t; a.scales_t = scales_t;
    return api_status(launch_f8_quantize(a, dtype, format, blocks, as_stream(stream)), fn);
}

int bitopt_f8_dequantize(const uint8_t* codes, const float* scales, int32_t format, int32_t blocks, int64_t rows,
                         int64_t cols, void* out, int32_t dtype, int64_t ldo, void* stream) {
    const char* fn = "bitopt_f8_dequantize";
    BITOPT_TRY(check_type(dtype, fn));
    BITOPT_TRY(check_form(format, blocks, fn));
    BITOPT_TRY(check_dim(rows, "rows", fn));
    BITOPT_TRY(check_dim(cols, "cols", fn));
    if (rows == 0 || cols == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_codes(codes, scales, "the input", fn));
    BITOPT_TRY(check_matrix(out, dtype, ldo, rows, cols, "out", fn));
    BITOPT_TRY(check_apart(fn, 1, {elements("out", out, dtype, ldo, rows, cols), codes_of("codes", codes, rows, cols),
                                   scales_of("scales", scales, rows, cols, blocks)}));
    F8CodecArgs a{};
    a.out = out; a.ldo = ldo; a.rows = rows; a.cols = cols;
    a.codes = const_cast<uint8_t*>(codes); a.scales = const_cast<float*>(scales);
    return api_status(launch_f8_dequantize(a, dtype, format, blocks, as_stream(stream)), fn);
}

int bitopt_f8_matmul(const uint8_t* a_codes, const float* a_scales, int32_t a_format, const uint8_t* b_codes,
                     const float* b_scales, int32_t b_format, int32_t b_blocks, int64_t m, int64_t n, int64_t k, void* out,
                     int32_t out_dtype, int64_t ldo, int32_t accumulate, void* stream) {
    const char* fn = "bitopt_f8_matmul";
    BITOPT_TRY(check_type(out_dtype, fn));
    BITOPT_TRY(check_form(a_format, BITOPT_F8_ROWS, fn));
    BITOPT_TRY(check_form(b_format, b_blocks, fn));
    BITOPT_TRY(check_dim(m, "m", fn));
    BITOPT_TRY(check_dim(n, "n", fn));
    BITOPT_TRY(check_dim(k, "k", fn));
    if (k > kMaxK) return api_fail(BITOPT_ERR_UNSUPPORTED, "%s: k above %lld", fn, (long long)kMaxK);
    if (m == 0 || n == 0) return api_status(hipSuccess, fn);
    // a launch holds fewer than 2^32 threads: 512 for a tile of 256 x 128 or 16 columns of few rows
    const int64_t threads = m <= kF8FewRows ? (n + 15) / 16 * 512 : (m / 256 + 1) * (n / 128 + 1) * 512;
    if (threads > 0xffffffffll)
        return api_fail(BITOPT_ERR_UNSUPPORTED, "%s: %lld x %lld results are too many for one launch", fn, (long long)m,
                        (long long)n);
    BITOPT_TRY(check_matrix(out, out_dtype, ldo, m, n, "out", fn));
    if (k > 0) {
        BITOPT_TRY(check_codes(a_codes, a_scales, "a", fn));
        BITOPT_TRY(check_codes(b_codes, b_scales, "b", fn));
        BITOPT_TRY(check_apart(fn, 1, {elements("out", out, out_dtype, ldo, m, n), codes_of("a", a_codes, m, k),
                                       scales_of("a's scales", a_scales, m, k, BITOPT_F8_ROWS),
                                       codes_of("b", b_codes, n, k), scales_of("b's scales", b_scales, n, k, b_blocks)}));
    }
    F8GemmArgs g{};
    g.a = a_codes; g.a_scales = a_scales; g.b = b_codes; g.b_scales = b_scales;
    g.row_bytes = f8_padded(k);
    g.out = out; g.ldo = ldo; g.out_dtype = out_dtype; g.accumulate = accumulate != 0;
    g.M = (int32_t)m; g.N = (int32_t)n; g.K = (int32_t)k;
    if (m <= kF8FewRows) return api_status(launch_f8_few(g, a_format, b_format, b_blocks, as_stream(stream)), fn);
    // what the 8-bit instruction drops shows in fp16 (f8_gemm.h)
    if (out_dtype != BITOPT_BF16) return api_status(launch_f8_exact(g, a_format, b_format, b_blocks, as_stream(stream)), fn);
    return api_status(launch_f8_fast(g, a_format, b_format, b_blocks, as_stream(stream)), fn);
}

}  // extern "C"
