// layer.h -- operators between the products of a training or decoding step: dropout, the
// embedding lookup and its gradient.  Argument blocks and launches.
#pragma once

#include <hip/hip_runtime.h>

#include "mx.h"

namespace bitopt {

struct DropoutArgs {
    const void* x; const void* residual; void* y;     // residual may be NULL
    int64_t ldx, ldr, ldy;
    int64_t rows, cols;
    uint64_t seed, call;
    const uint64_t* counter;             // device; added to call where given
    uint32_t threshold;                  // an element is kept when its 16 bits are not below it
    float grow;
};

struct EmbeddingArgs {
    const void* tokens; int64_t count;
    const void* table; int64_t ldt;      // elements, or
    const uint8_t* codes; const uint8_t* scales;      // an MX matrix
    void* out; int64_t ldo;
    int64_t vocab, width;
    float scale;
    bool wide;                           // 64-bit tokens
};

// Places in the workspace of an embedding's gradient, in bytes; every part is aligned to 16.
struct EmbeddingSpace {
    int64_t keys[2], order[2], digits, partial, bytes;
    int64_t span;                        // places of the sorted order in a window
};

struct EmbeddingGradArgs {
    const void* tokens; int64_t count;
    const void* dy; int64_t lddy;
    void* out; int64_t ldo;
    int64_t vocab, width;
    float scale;
    bool wide, accumulate;
    char* work;
    EmbeddingSpace at;
};

EmbeddingSpace embedding_space(int64_t count, int64_t vocab, int64_t width);

hipError_t launch_dropout(const DropoutArgs& a, int dtype, hipStream_t s);
hipError_t launch_embedding(const EmbeddingArgs& a, int dtype, int out_dtype, hipStream_t s);
hipError_t launch_mx_embedding(const EmbeddingArgs& a, int fmt, int out_dtype, hipStream_t s);
hipError_t launch_embedding_grad(const EmbeddingGradArgs& a, int dtype, int out_dtype, hipStream_t s);

}  // namespace bitopt
