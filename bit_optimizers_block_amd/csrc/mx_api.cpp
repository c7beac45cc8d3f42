// mx_api.cpp -- the C ABI of the MX operators (declared in include/bitopt.h): argument
// checks and dispatch.
#include "bitopt.h"
#include "launch.h"
#include "mx_overlap.h"

namespace {

using bitopt::api_fail;
using bitopt::api_status;
using bitopt::MxGemmArgs;

constexpr int64_t kMaxDim = int64_t{1} << 30;    // sizes, rounded up to a tile, are int32 in the kernels
constexpr int64_t kMaxScaledK = int64_t{1} << 24;  // offsets within a tile of 256 rows stay below 2^32

bool valid_dtype(int32_t d) { return d == BITOPT_F32 || d == BITOPT_F16 || d == BITOPT_BF16; }
bool valid_format(int32_t f) { return f == BITOPT_MX_E2M1 || f == BITOPT_MX_E4M3; }
uintptr_t elem_mask(int32_t d) { return d == BITOPT_F32 ? 3 : 1; }
bool aligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) == 0; }

int check_dim(int64_t v, const char* name, const char* fn) {
    if (v < 0) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s < 0", fn, name);
    if (v > kMaxDim) return api_fail(BITOPT_ERR_UNSUPPORTED, "%s: %s above %lld", fn, name, (long long)kMaxDim);
    return BITOPT_OK;
}

// A row-major matrix of elements: pointer, alignment to the element, distance of rows.
int check_matrix(const void* p, int32_t dtype, int64_t ld, int64_t rows, int64_t cols, const char* name, const char* fn) {
    if (!p) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (!aligned(p, elem_mask(dtype)))
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", fn, name);
    if (rows > 1 && ld < cols)
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: rows of %s are %lld elements apart but hold %lld", fn, name,
                        (long long)ld, (long long)cols);
    return BITOPT_OK;
}

// A launch holds fewer than 2^32 threads.  Tiles of 256 x 256 take 512; smaller tiles are only
// taken for a few hundred of them.  The form for few rows has one workgroup of 256 for 64 columns
// where there are many.
int check_launch(int64_t rows, int64_t cols, bool few, const char* fn) {
    const int64_t threads = few ? (cols + 63) / 64 * 256 : (rows / 256 + 1) * (cols / 256 + 1) * 512;
    if (threads > 0xffffffffll)
        return api_fail(BITOPT_ERR_UNSUPPORTED, "%s: %lld x %lld results are too many for one launch", fn,
                        (long long)rows, (long long)cols);
    return BITOPT_OK;
}

int check_codes(const void* codes, const void* scales, const char* name, const char* fn) {
    if (!codes || !scales) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: NULL codes or scales of %s", fn, name);
    if (!aligned(codes, 15) || !aligned(scales, 15))
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: codes and scales of %s must be aligned to 16 bytes", fn, name);
    return BITOPT_OK;
}

int check_types(int32_t dtype, int32_t format, const char* fn) {
    if (!valid_dtype(dtype)) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
    if (!valid_format(format)) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown MX format %d", fn, format);
    return BITOPT_OK;
}

// The 16-bit products take fp16 and bf16.
int check_half(int32_t dtype, const char* fn) {
    if (dtype == BITOPT_F32) return api_fail(BITOPT_ERR_UNSUPPORTED, "%s: the input must be fp16 or bf16", fn);
    return BITOPT_OK;
}

// A matrix of a call, for the check that results share no memory with anything else of it.
struct Named {
    const char* name;
    bitopt::ByteRows at;
};
Named elements(const char* name, const void* p, int32_t dtype, int64_t ld, int64_t rows, int64_t cols) {
    const int64_t es = dtype == BITOPT_F32 ? 4 : 2;
    // distances beyond 2^60 elements are no memory: one that still fits 64 bits stands for them
    return {name, {p, rows, cols * es, std::min<int64_t>(ld, int64_t{1} << 60) * es}};
}
Named packed(const char* name, const void* p, int64_t rows, int64_t width) { return {name, {p, rows, width, width}}; }

// The first `results` of the matrices are written: none may meet another.  The first `in_place` of
// those are laid out as the read matrices at `over` or `over2` and written item by item after the
// reads of the same items, so they may lie over the very same rows.
template <size_t N> int check_apart(const char* fn, size_t results, const Named (&m)[N], size_t in_place = 0,
                                    const void* over = nullptr, const void* over2 = nullptr) {
    for (size_t r = 0; r < results; ++r)
        for (size_t i = r + 1; i < N; ++i) {
            const bitopt::ByteRows &a = m[r].at, &b = m[i].at;
            if (!bitopt::rows_meet(a, b)) continue;
            if (r < in_place && i >= results && a.p == b.p && (b.p == over || b.p == over2) &&
                (a.rows == 1 || a.stride == b.stride))
                continue;
            return api_fail(BITOPT_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, m[r].name, m[i].name);
        }
    return BITOPT_OK;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

#define BITOPT_TRY(call)          \
    do {                          \
        if (int rc = (call)) return rc; \
    } while (0)

extern "C" {

int64_t bitopt_mx_code_bytes(int64_t cols, int32_t format) {
    if (cols < 0 || cols > kMaxDim || !valid_format(format)) return -1;
    return bitopt::mx_code_bytes(cols, format);
}

int64_t bitopt_mx_scale_bytes(int64_t cols) {
    if (cols < 0 || cols > kMaxDim) return -1;
    return bitopt::mx_scale_bytes(cols);
}

int bitopt_mx_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, int32_t format,
                       uint8_t* codes, uint8_t* scales, void* stream) {
    const char* fn = "bitopt_mx_quantize";
    BITOPT_TRY(check_types(dtype, format, fn));
    BITOPT_TRY(check_dim(rows, "rows", fn));
    BITOPT_TRY(check_dim(cols, "cols", fn));
    if (rows == 0 || cols == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_matrix(x, dtype, ldx, rows, cols, "x", fn));
    BITOPT_TRY(check_codes(codes, scales, "x", fn));
    BITOPT_TRY(check_apart(fn, 2, {packed("codes", codes, rows, bitopt::mx_code_bytes(cols, format)),
                                   packed("scales", scales, rows, bitopt::mx_scale_bytes(cols)),
                                   elements("x", x, dtype, ldx, rows, cols)}));
    bitopt::MxCodecArgs a{};
    a.x = x; a.ldx = ldx; a.codes = codes; a.scales = scales; a.rows = rows; a.cols = cols;
    return api_status(bitopt::launch_mx_quantize(a, dtype, format, as_stream(stream)), fn);
}

int bitopt_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int32_t format, int64_t rows, int64_t cols,
                         void* out, int32_t dtype, int64_t ldo, void* stream) {
    const char* fn = "bitopt_mx_dequantize";
    BITOPT_TRY(check_types(dtype, format, fn));
    BITOPT_TRY(check_dim(rows, "rows", fn));
    BITOPT_TRY(check_dim(cols, "cols", fn));
    if (rows == 0 || cols == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_codes(codes, scales, "the input", fn));
    BITOPT_TRY(check_matrix(out, dtype, ldo, rows, cols, "out", fn));
    BITOPT_TRY(check_apart(fn, 1, {elements("out", out, dtype, ldo, rows, cols),
                                   packed("codes", codes, rows, bitopt::mx_code_bytes(cols, format)),
                                   packed("scales", scales, rows, bitopt::mx_scale_bytes(cols))}));
    bitopt::MxCodecArgs a{};
    a.out = out; a.ldo = ldo; a.rows = rows; a.cols = cols;
    a.codes = const_cast<uint8_t*>(codes); a.scales = const_cast<uint8_t*>(scales);
    return api_status(bitopt::launch_mx_dequantize(a, dtype, format, as_stream(stream)), fn);
}

int bitopt_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int32_t a_format, const uint8_t* b_codes,
                     const uint8_t* b_scales, int32_t b_format, int64_t m, int64_t n, int64_t k, void* out,
                     int32_t out_dtype, int64_t ldo, void* stream) {
    const char* fn = "bitopt_mx_matmul";
    BITOPT_TRY(check_types(out_dtype, a_format, fn));
    BITOPT_TRY(check_types(out_dtype, b_format, fn));
    BITOPT_TRY(check_dim(m, "m", fn));
    BITOPT_TRY(check_dim(n, "n", fn));
    BITOPT_TRY(check_dim(k, "k", fn));
    if (k > kMaxScaledK)
        return api_fail(BITOPT_ERR_UNSUPPORTED, "%s: k above %lld", fn, (long long)kMaxScaledK);
    if (m == 0 || n == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_launch(m, n, m <= bitopt::kMxSkinnyRows, fn));
    BITOPT_TRY(check_matrix(out, out_dtype, ldo, m, n, "out", fn));
    if (k > 0) {
        BITOPT_TRY(check_codes(a_codes, a_scales, "a", fn));
        BITOPT_TRY(check_codes(b_codes, b_scales, "b", fn));
        BITOPT_TRY(check_apart(fn, 1, {elements("out", out, out_dtype, ldo, m, n),
                                       packed("a", a_codes, m, bitopt::mx_code_bytes(k, a_format)),
                                       packed("a's scales", a_scales, m, bitopt::mx_scale_bytes(k)),
                                       packed("b", b_codes, n, bitopt::mx_code_bytes(k, b_format)),
                                       packed("b's scales", b_scales, n, bitopt::mx_scale_bytes(k))}));
    }
    MxGemmArgs g{};
    g.a = a_codes; g.a_scales = a_scales; g.b = b_codes; g.b_scales = b_scales;
    g.a_row_bytes = bitopt::mx_code_bytes(k, a_format); g.b_row_bytes = bitopt::mx_code_bytes(k, b_format);
    g.a_row_scales = g.b_row_scales = bitopt::mx_scale_bytes(k);
    g.out = out; g.ldo = ldo; g.out_dtype = out_dtype;
    g.M = (int32_t)m; g.N = (int32_t)n; g.K = (int32_t)k;
    if (m <= bitopt::kMxSkinnyRows)
        return api_status(bitopt::launch_mx_matmul_skinny(g, a_format, b_format, as_stream(stream)), fn);
    return api_status(bitopt::launch_mx_matmul(g, a_format, b_format, as_stream(stream)), fn);
}

int bitopt_mx_linear(const void* x, int32_t dtype, int64_t ldx, const uint8_t* w_codes, const uint8_t* w_scales,
                     int32_t format, int64_t tokens, int64_t n, int64_t k, void* out, int32_t out_dtype, int64_t ldo,
                     void* stream) {
    const char* fn = "bitopt_mx_linear";
    BITOPT_TRY(check_types(dtype, format, fn));
    BITOPT_TRY(check_types(out_dtype, format, fn));
    BITOPT_TRY(check_half(dtype, fn));
    BITOPT_TRY(check_dim(tokens, "tokens", fn));
    BITOPT_TRY(check_dim(n, "n", fn));
    BITOPT_TRY(check_dim(k, "k", fn));
    if (tokens == 0 || n == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_launch(tokens, n, tokens <= bitopt::kMxSkinnyRows, fn));
    BITOPT_TRY(check_matrix(out, out_dtype, ldo, tokens, n, "out", fn));
    if (k > 0) {
        BITOPT_TRY(check_matrix(x, dtype, ldx, tokens, k, "x", fn));
        BITOPT_TRY(check_codes(w_codes, w_scales, "w", fn));
        BITOPT_TRY(check_apart(fn, 1, {elements("out", out, out_dtype, ldo, tokens, n),
                                       elements("x", x, dtype, ldx, tokens, k),
                                       packed("w", w_codes, n, bitopt::mx_code_bytes(k, format)),
                                       packed("w's scales", w_scales, n, bitopt::mx_scale_bytes(k))}));
    }
    MxGemmArgs g{};
    g.a = x; g.lda = ldx; g.b = w_codes; g.b_scales = w_scales;
    g.b_row_bytes = bitopt::mx_code_bytes(k, format); g.b_row_scales = bitopt::mx_scale_bytes(k);
    g.out = out; g.ldo = ldo; g.out_dtype = out_dtype;
    g.M = (int32_t)tokens; g.N = (int32_t)n; g.K = (int32_t)k;
    if (tokens <= bitopt::kMxSkinnyRows)
        return api_status(bitopt::launch_mx_linear_skinny(g, dtype, format, as_stream(stream)), fn);
    return api_status(bitopt::launch_mx_linear(g, dtype, format, as_stream(stream)), fn);
}

int bitopt_mx_linear_grad_input(const void* dy, int32_t dtype, int64_t lddy, const uint8_t* w_codes,
                                const uint8_t* w_scales, int32_t format, int64_t tokens, int64_t n, int64_t k, void* dx,
                                int32_t out_dtype, int64_t lddx, void* stream) {
    const char* fn = "bitopt_mx_linear_grad_input";
    BITOPT_TRY(check_types(dtype, format, fn));
    BITOPT_TRY(check_types(out_dtype, format, fn));
    BITOPT_TRY(check_half(dtype, fn));
    BITOPT_TRY(check_dim(tokens, "tokens", fn));
    BITOPT_TRY(check_dim(n, "n", fn));
    BITOPT_TRY(check_dim(k, "k", fn));
    if (tokens == 0 || k == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_launch(tokens, k, false, fn));
    BITOPT_TRY(check_matrix(dx, out_dtype, lddx, tokens, k, "dx", fn));
    if (n > 0) {
        BITOPT_TRY(check_matrix(dy, dtype, lddy, tokens, n, "dy", fn));
        BITOPT_TRY(check_codes(w_codes, w_scales, "w", fn));
        BITOPT_TRY(check_apart(fn, 1, {elements("dx", dx, out_dtype, lddx, tokens, k),
                                       elements("dy", dy, dtype, lddy, tokens, n),
                                       packed("w", w_codes, n, bitopt::mx_code_bytes(k, format)),
                                       packed("w's scales", w_scales, n, bitopt::mx_scale_bytes(k))}));
    }
    MxGemmArgs g{};
    g.a = dy; g.lda = lddy; g.b = w_codes; g.b_scales = w_scales;
    g.b_row_bytes = bitopt::mx_code_bytes(k, format); g.b_row_scales = bitopt::mx_scale_bytes(k);
    g.out = dx; g.ldo = lddx; g.out_dtype = out_dtype;
    g.M = (int32_t)tokens; g.N = (int32_t)k; g.K = (int32_t)n;
    return api_status(bitopt::launch_mx_grad_input(g, dtype, format, as_stream(stream)), fn);
}

int bitopt_mx_linear_grad_weight(const void* dy, int32_t dtype, int64_t lddy, const uint8_t* x_codes,
                                 const uint8_t* x_scales, int32_t format, int64_t tokens, int64_t n, int64_t k, void* dw,
                                 int32_t out_dtype, int64_t lddw, int32_t accumulate, void* stream) {
    const char* fn = "bitopt_mx_linear_grad_weight";
    BITOPT_TRY(check_types(dtype, format, fn));
    BITOPT_TRY(check_types(out_dtype, format, fn));
    BITOPT_TRY(check_half(dtype, fn));
    BITOPT_TRY(check_dim(tokens, "tokens", fn));
    BITOPT_TRY(check_dim(n, "n", fn));
    BITOPT_TRY(check_dim(k, "k", fn));
    if (n == 0 || k == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_launch(n, k, false, fn));
    BITOPT_TRY(check_matrix(dw, out_dtype, lddw, n, k, "dw", fn));
    if (tokens > 0) {
        BITOPT_TRY(check_matrix(dy, dtype, lddy, tokens, n, "dy", fn));
        BITOPT_TRY(check_codes(x_codes, x_scales, "x", fn));
        BITOPT_TRY(check_apart(fn, 1, {elements("dw", dw, out_dtype, lddw, n, k),
                                       elements("dy", dy, dtype, lddy, tokens, n),
                                       packed("x", x_codes, tokens, bitopt::mx_code_bytes(k, format)),
                                       packed("x's scales", x_scales, tokens, bitopt::mx_scale_bytes(k))}));
    }
    MxGemmArgs g{};
    g.a = dy; g.lda = lddy; g.b = x_codes; g.b_scales = x_scales;
    g.b_row_bytes = bitopt::mx_code_bytes(k, format); g.b_row_scales = bitopt::mx_scale_bytes(k);
    g.out = dw; g.ldo = lddw; g.out_dtype = out_dtype; g.accumulate = accumulate != 0;
    g.M = (int32_t)n; g.N = (int32_t)k; g.K = (int32_t)tokens;
    return api_status(bitopt::launch_mx_grad_weight(g, dtype, format, as_stream(stream)), fn);
}

int bitopt_swiglu_forward_mx8(const void* gate, const void* up, int32_t dtype, int64_t rows, int64_t cols, int64_t ldg,
                              int64_t ldu, void* y, int64_t ldy, uint8_t* gate_codes, uint8_t* gate_scales,
                              uint8_t* up_codes, uint8_t* up_scales, void* stream) {
    const char* fn = "bitopt_swiglu_forward_mx8";
    BITOPT_TRY(check_types(dtype, BITOPT_MX_E4M3, fn));
    BITOPT_TRY(check_dim(rows, "rows", fn));
    BITOPT_TRY(check_dim(cols, "cols", fn));
    if (rows == 0 || cols == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_matrix(gate, dtype, ldg, rows, cols, "gate", fn));
    BITOPT_TRY(check_matrix(up, dtype, ldu, rows, cols, "up", fn));
    BITOPT_TRY(check_matrix(y, dtype, ldy, rows, cols, "y", fn));
    BITOPT_TRY(check_codes(gate_codes, gate_scales, "gate", fn));
    BITOPT_TRY(check_codes(up_codes, up_scales, "up", fn));
    BITOPT_TRY(check_apart(
        fn, 5,
        {elements("y", y, dtype, ldy, rows, cols), packed("gate's codes", gate_codes, rows, bitopt::mx_code_bytes(cols, BITOPT_MX_E4M3)),
         packed("gate's scales", gate_scales, rows, bitopt::mx_scale_bytes(cols)),
         packed("up's codes", up_codes, rows, bitopt::mx_code_bytes(cols, BITOPT_MX_E4M3)),
         packed("up's scales", up_scales, rows, bitopt::mx_scale_bytes(cols)),
         elements("gate", gate, dtype, ldg, rows, cols), elements("up", up, dtype, ldu, rows, cols)},
        1, gate, up));
    bitopt::SwigluArgs a{};
    a.gate = gate; a.up = up; a.y = y; a.ldg = ldg; a.ldu = ldu; a.ldy = ldy;
    a.gate_codes = gate_codes; a.gate_scales = gate_scales; a.up_codes = up_codes; a.up_scales = up_scales;
    a.rows = rows; a.cols = cols;
    return api_status(bitopt::launch_swiglu_forward(a, dtype, as_stream(stream)), fn);
}

int bitopt_swiglu_backward_mx8(const void* dy, int32_t dtype, int64_t rows, int64_t cols, int64_t lddy,
                               const uint8_t* gate_codes, const uint8_t* gate_scales, const uint8_t* up_codes,
                               const uint8_t* up_scales, void* dgate, int64_t lddg, void* dup, int64_t lddu,
                               void* stream) {
    const char* fn = "bitopt_swiglu_backward_mx8";
    BITOPT_TRY(check_types(dtype, BITOPT_MX_E4M3, fn));
    BITOPT_TRY(check_dim(rows, "rows", fn));
    BITOPT_TRY(check_dim(cols, "cols", fn));
    if (rows == 0 || cols == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_matrix(dy, dtype, lddy, rows, cols, "dy", fn));
    BITOPT_TRY(check_matrix(dgate, dtype, lddg, rows, cols, "dgate", fn));
    BITOPT_TRY(check_matrix(dup, dtype, lddu, rows, cols, "dup", fn));
    BITOPT_TRY(check_codes(gate_codes, gate_scales, "gate", fn));
    BITOPT_TRY(check_codes(up_codes, up_scales, "up", fn));
    BITOPT_TRY(check_apart(
        fn, 2,
        {elements("dgate", dgate, dtype, lddg, rows, cols), elements("dup", dup, dtype, lddu, rows, cols),
         elements("dy", dy, dtype, lddy, rows, cols), packed("gate's codes", gate_codes, rows, bitopt::mx_code_bytes(cols, BITOPT_MX_E4M3)),
         packed("gate's scales", gate_scales, rows, bitopt::mx_scale_bytes(cols)),
         packed("up's codes", up_codes, rows, bitopt::mx_code_bytes(cols, BITOPT_MX_E4M3)),
         packed("up's scales", up_scales, rows, bitopt::mx_scale_bytes(cols))},
        2, dy));
    bitopt::SwigluArgs a{};
    a.dy = dy; a.ldy = lddy; a.dgate = dgate; a.lddg = lddg; a.dup = dup; a.lddu = lddu;
    a.gate_codes = const_cast<uint8_t*>(gate_codes); a.gate_scales = const_cast<uint8_t*>(gate_scales);
    a.up_codes = const_cast<uint8_t*>(up_codes); a.up_scales = const_cast<uint8_t*>(up_scales);
    a.rows = rows; a.cols = cols;
    return api_status(bitopt::launch_swiglu_backward(a, dtype, as_stream(stream)), fn);
}

}  // extern "C"
