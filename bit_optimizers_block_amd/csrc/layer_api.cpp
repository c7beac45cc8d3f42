// layer_api.cpp -- the C ABI of dropout, the embedding lookup and its gradient (declared in
// include/bitopt.h): argument checks and dispatch.
#include <cmath>

#include "layer.h"
#include "mx_checks.h"

namespace {

using namespace bitopt;

int check_type(int32_t dtype, const char* fn) {
    return valid_dtype(dtype) ? BITOPT_OK : api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
}

int64_t token_bytes(int32_t type) { return type == BITOPT_TOKENS_I32 ? 4 : 8; }

int check_tokens(const void* tokens, int32_t type, const char* fn) {
    if (type != BITOPT_TOKENS_I32 && type != BITOPT_TOKENS_I64)
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown token type %d", fn, type);
    if (!tokens) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: tokens is NULL", fn);
    if (!aligned(tokens, token_bytes(type) - 1))
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: tokens is not aligned to its elements", fn);
    return BITOPT_OK;
}

int check_scale(float scale, const char* fn) {
    return std::isfinite(scale) ? BITOPT_OK : api_fail(BITOPT_ERR_INVALID_ARG, "%s: scale is not finite", fn);
}

// y is written from x and, where given, the residual; it may lie over either.
int dropout(const char* fn, const char* in, const char* out, const void* x, int32_t dtype, int64_t rows, int64_t cols,
            int64_t ldx, const void* residual, int64_t ldr, double p, uint64_t seed, uint64_t call, const uint64_t* counter,
            void* y, int64_t ldy, void* stream) {
    BITOPT_TRY(check_type(dtype, fn));
    BITOPT_TRY(check_dim(rows, "rows", fn));
    BITOPT_TRY(check_dim(cols, "cols", fn));
    if (!(p >= 0.0 && p <= 1.0)) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: p must lie in [0, 1]", fn);
    if (rows == 0 || cols == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_matrix(x, dtype, ldx, rows, cols, in, fn));
    BITOPT_TRY(check_matrix(y, dtype, ldy, rows, cols, out, fn));
    if (residual) BITOPT_TRY(check_matrix(residual, dtype, ldr, rows, cols, "residual", fn));
    if (!aligned(counter, 7)) return api_fail(BITOPT_ERR_INVALID_ARG, "%s: counter is not aligned to 8 bytes", fn);
    BITOPT_TRY(check_apart(fn, 1, {elements(out, y, dtype, ldy, rows, cols), elements(in, x, dtype, ldx, rows, cols),
                                   elements("residual", residual, dtype, ldr, rows, cols), packed("counter", counter, 1, 8)},
                           1, x, residual));
    DropoutArgs a{};
    a.x = x; a.residual = residual; a.y = y; a.ldx = ldx; a.ldr = ldr; a.ldy = ldy; a.rows = rows; a.cols = cols;
    a.seed = seed; a.call = call; a.counter = counter;
    a.threshold = (uint32_t)std::nearbyint(p * 65536.0);
    a.grow = a.threshold < 65536 ? (float)(65536.0 / (65536.0 - a.threshold)) : 0.0f;
    return api_status(launch_dropout(a, dtype, as_stream(stream)), fn);
}

}  // namespace

extern "C" {

int bitopt_dropout_forward(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, const void* residual,
                           int64_t ldr, double p, uint64_t seed, uint64_t call, const uint64_t* counter, void* y,
                           int64_t ldy, void* stream) {
    return dropout("bitopt_dropout_forward", "x", "y", x, dtype, rows, cols, ldx, residual, ldr, p, seed, call, counter, y,
                   ldy, stream);
}

int bitopt_dropout_backward(const void* dy, int32_t dtype, int64_t rows, int64_t cols, int64_t lddy, double p,
                            uint64_t seed, uint64_t call, const uint64_t* counter, void* dx, int64_t lddx, void* stream) {
    return dropout("bitopt_dropout_backward", "dy", "dx", dy, dtype, rows, cols, lddy, nullptr, 0, p, seed, call, counter,
                   dx, lddx, stream);
}

int bitopt_embedding_forward(const void* tokens, int32_t token_type, int64_t count, const void* table, int32_t dtype,
                             int64_t vocab, int64_t width, int64_t ldt, float scale, void* out, int32_t out_dtype,
                             int64_t ldo, void* stream) {
    const char* fn = "bitopt_embedding_forward";
    BITOPT_TRY(check_type(dtype, fn));
    BITOPT_TRY(check_type(out_dtype, fn));
    BITOPT_TRY(check_dim(count, "count", fn));
    BITOPT_TRY(check_dim(vocab, "vocab", fn));
    BITOPT_TRY(check_dim(width, "width", fn));
    BITOPT_TRY(check_scale(scale, fn));
    if (count == 0 || width == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_tokens(tokens, token_type, fn));
    if (vocab > 0) BITOPT_TRY(check_matrix(table, dtype, ldt, vocab, width, "table", fn));
    BITOPT_TRY(check_matrix(out, out_dtype, ldo, count, width, "out", fn));
    BITOPT_TRY(check_apart(fn, 1, {elements("out", out, out_dtype, ldo, count, width),
                                   packed("tokens", tokens, 1, count * token_bytes(token_type)),
                                   elements("table", table, dtype, ldt, vocab, width)}));
    EmbeddingArgs a{};
    a.tokens = tokens; a.count = count; a.wide = token_type == BITOPT_TOKENS_I64; a.table = table; a.ldt = ldt;
    a.out = out; a.ldo = ldo; a.vocab = vocab; a.width = width; a.scale = scale;
    return api_status(launch_embedding(a, dtype, out_dtype, as_stream(stream)), fn);
}

int bitopt_mx_embedding_forward(const void* tokens, int32_t token_type, int64_t count, const uint8_t* codes,
                                const uint8_t* scales, int32_t format, int64_t vocab, int64_t width, float scale,
                                void* out, int32_t out_dtype, int64_t ldo, void* stream) {
    const char* fn = "bitopt_mx_embedding_forward";
    BITOPT_TRY(check_type(out_dtype, fn));
    if (format != BITOPT_MX_E2M1 && format != BITOPT_MX_E4M3)
        return api_fail(BITOPT_ERR_INVALID_ARG, "%s: unknown MX format %d", fn, format);
    BITOPT_TRY(check_dim(count, "count", fn));
    BITOPT_TRY(check_dim(vocab, "vocab", fn));
    BITOPT_TRY(check_dim(width, "width", fn));
    BITOPT_TRY(check_scale(scale, fn));
    if (count == 0 || width == 0) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_tokens(tokens, token_type, fn));
    if (vocab > 0) BITOPT_TRY(check_codes(codes, scales, "the table", fn));
    BITOPT_TRY(check_matrix(out, out_dtype, ldo, count, width, "out", fn));
    BITOPT_TRY(check_apart(fn, 1, {elements("out", out, out_dtype, ldo, count, width),
                                   packed("tokens", tokens, 1, count * token_bytes(token_type)),
                                   packed("the table", codes, vocab, mx_code_bytes(width, format)),
                                   packed("the table's scales", scales, vocab, mx_scale_bytes(width))}));
    EmbeddingArgs a{};
    a.tokens = tokens; a.count = count; a.wide = token_type == BITOPT_TOKENS_I64; a.codes = codes; a.scales = scales;
    a.out = out; a.ldo = ldo; a.vocab = vocab; a.width = width; a.scale = scale;
    return api_status(launch_mx_embedding(a, format, out_dtype, as_stream(stream)), fn);
}

int64_t bitopt_embedding_workspace_bytes(int64_t count, int64_t vocab, int64_t width) {
    if (count < 0 || vocab < 0 || width < 0 || count > kMaxDim || vocab > kMaxDim || width > kMaxDim) return -1;
    return embedding_space(count, vocab, width).bytes;
}

int bitopt_embedding_backward(const void* dy, int32_t dtype, int64_t count, int64_t width, int64_t lddy,
                              const void* tokens, int32_t token_type, int64_t vocab, float scale, void* dtable,
                              int32_t out_dtype, int64_t ldd, int32_t accumulate, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    const char* fn = "bitopt_embedding_backward";
    BITOPT_TRY(check_type(dtype, fn));
    BITOPT_TRY(check_type(out_dtype, fn));
    BITOPT_TRY(check_dim(count, "count", fn));
    BITOPT_TRY(check_dim(vocab, "vocab", fn));
    BITOPT_TRY(check_dim(width, "width", fn));
    BITOPT_TRY(check_scale(scale, fn));
    if (vocab == 0 || width == 0 || (count == 0 && accumulate)) return api_status(hipSuccess, fn);
    BITOPT_TRY(check_matrix(dtable, out_dtype, ldd, vocab, width, "dtable", fn));
    EmbeddingGradArgs a{};
    a.out = dtable; a.ldo = ldd; a.vocab = vocab; a.width = width; a.count = count; a.accumulate = accumulate != 0;
    if (count > 0) {
        BITOPT_TRY(check_tokens(tokens, token_type, fn));
        BITOPT_TRY(check_matrix(dy, dtype, lddy, count, width, "dy", fn));
        a.at = embedding_space(count, vocab, width);
        if (!workspace || !aligned(workspace, 15) || workspace_bytes < a.at.bytes)
            return api_fail(BITOPT_ERR_INVALID_ARG, "%s: the workspace must be aligned to 16 bytes and hold %lld bytes", fn,
                            (long long)a.at.bytes);
        BITOPT_TRY(check_apart(fn, 2, {elements("dtable", dtable, out_dtype, ldd, vocab, width),
                                       packed("the workspace", workspace, 1, a.at.bytes),
                                       elements("dy", dy, dtype, lddy, count, width),
                                       packed("tokens", tokens, 1, count * token_bytes(token_type))}));
        a.tokens = tokens; a.wide = token_type == BITOPT_TOKENS_I64; a.dy = dy; a.lddy = lddy; a.scale = scale;
        a.work = static_cast<char*>(workspace);
    }
    return api_status(launch_embedding_grad(a, dtype, out_dtype, as_stream(stream)), fn);
}

}  // extern "C"
