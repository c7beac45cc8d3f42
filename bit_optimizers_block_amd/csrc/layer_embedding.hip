// Embedding lookup, from a table of elements or an MX matrix, and its gradient by sorted tokens.
//
// Gradient: out[v] (+)= scale * the sum of dy[t] over the tokens t with number v.  Tokens are
// sorted by number with a stable radix sort, so the rows of one number are a run of the sorted
// order, in their order in the batch: no atomics, and the same bits on every run.  A workgroup
// adds up to `span` rows of a run in registers; longer runs (a frequent token) leave their parts
// in the workspace, and a second kernel adds those.
#include "launch.h"
#include "layer.h"
#include "mx_rows.h"

namespace bitopt {

// ---------------------------------------------------------------------------- lookup

__device__ __forceinline__ int64_t token_at(const void* tokens, bool wide, int64_t t) {
    return wide ? gbl(reinterpret_cast<const int64_t*>(tokens))[t] : (int64_t)gbl(reinterpret_cast<const int32_t*>(tokens))[t];
}

// A token outside the table gets zeros.
template <int DT, int OUT> __global__ __launch_bounds__(kThreads) void k_embedding(EmbeddingArgs a, RowGrid g) {
    for_items(g, a.count, (int32_t)((a.width + 7) / 8), [&](int64_t row, int32_t item) {
        const int64_t e = 8 * (int64_t)item;
        const int n = (int)min((int64_t)8, a.width - e);
        const int64_t id = token_at(a.tokens, a.wide, row);
        float v[8] = {};
        if ((uint64_t)id < (uint64_t)a.vocab) ld_eight<DT, false>(a.table, id * a.ldt + e, n, e, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= a.scale;
        st_eight<OUT>(a.out, row * a.ldo + e, n, v);
    });
}

template <int FMT, int OUT> __global__ __launch_bounds__(kThreads) void k_mx_embedding(EmbeddingArgs a, RowGrid g) {
    const int64_t bytes = mx_code_bytes(a.width, FMT), blocks = mx_scale_bytes(a.width);
    for_items(g, a.count, (int32_t)((a.width + 7) / 8), [&](int64_t row, int32_t item) {
        const int64_t id = token_at(a.tokens, a.wide, row);
        float v[8] = {};
        if ((uint64_t)id < (uint64_t)a.vocab) {
            const float s = mx_scale_f32(gbl(a.scales)[id * blocks + item / 4]);
            const uint8_t* p = a.codes + id * bytes;
            if constexpr (FMT == kMxE2M1) {
                const uint32_t c = gbl(reinterpret_cast<const uint32_t*>(p))[item];
                mx_decode4_e2m1(c, s, v);
                mx_decode4_e2m1(c >> 16, s, v + 4);
            } else {
                const u32x2 c = gbl(reinterpret_cast<const u32x2*>(p))[item];
                mx_decode4_e4m3(c.x, s, v);
                mx_decode4_e4m3(c.y, s, v + 4);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= a.scale;
        st_eight<OUT>(a.out, row * a.ldo + 8 * (int64_t)item, (int)min((int64_t)8, a.width - 8 * (int64_t)item), v);
    });
}

// -------------------------------------------------------------------------- the sort

// A token's sort key: its number, or `vocab` where it is outside the table.
__device__ __forceinline__ uint32_t key_at(const EmbeddingGradArgs& a, int64_t t) {
    const int64_t id = token_at(a.tokens, a.wide, t);
    return (uint64_t)id < (uint64_t)a.vocab ? (uint32_t)id : (uint32_t)a.vocab;
}

constexpr int kDigits = 256, kSmallThreads = 1024, kTileItems = 4096;

// Ranks of a workgroup's items among those with their digit of the same wave, in the order (j,
// lane), and afterwards in counts[wave][digit] how many the wave has.  counts is zero before.
template <int IPT> __device__ __forceinline__ void rank_in_wave(const uint32_t d[IPT], volatile uint32_t* counts, uint32_t rank[IPT]) {
    const uint64_t below = (1ull << (threadIdx.x & 63)) - 1;
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        uint64_t same = ~0ull;                          // lanes with this lane's digit
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const bool bit = d[j] >> b & 1;
            const uint64_t with = __ballot(bit);
            same &= bit ? with : ~with;
        }
        const uint32_t had = counts[d[j]], before = __popcll(same & below);
        rank[j] = had + before;
        // a wave's LDS accesses take effect in order: the next item's read sees this
        if (before == 0) counts[d[j]] = had + (uint32_t)__popcll(same);
    }
}

// counts[wave][digit] -> the sum of all with a lower digit, or the same and a lower wave.
template <int WAVES> __device__ __forceinline__ void scan_counts(uint32_t* counts, uint32_t* sums) {
    constexpr int N = WAVES * kDigits / (WAVES * 64);   // counters of a thread: those of consecutive waves
    static_assert(WAVES % N == 0, "a thread's counters have one digit");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, d = tid / (WAVES / N), w0 = tid % (WAVES / N) * N;
    uint32_t c[N], total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = counts[(w0 + i) * kDigits + d];
        total += c[i];
    }
    uint32_t up = total;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
        const uint32_t v = __shfl_up(up, k);
        if (lane >= k) up += v;
    }
    if (lane == 63) sums[wave] = up;
    __syncthreads();
    uint32_t base = up - total;
    for (int w = 0; w < wave; ++w) base += sums[w];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        counts[(w0 + i) * kDigits + d] = base;
        base += c[i];
    }
}

// Zeros in every row of the gradient: `part` of `parts` workgroups.
template <int OUT> __device__ __forceinline__ void clear_rows(const EmbeddingGradArgs& a, int64_t part, int64_t parts) {
    const int32_t items = (int32_t)((a.width + 7) / 8);
    int lanes = 64;
    while (lanes < (int)blockDim.x && lanes < items) lanes *= 2;
    const int per = (int)blockDim.x / lanes;
    const float zero[8] = {};
    for (int64_t row = part * per + threadIdx.x / lanes; row < a.vocab; row += parts * per)
        for (int32_t item = threadIdx.x % lanes; item < items; item += lanes)
            st_eight<OUT>(a.out, row * a.ldo + 8 * (int64_t)item, (int)min((int64_t)8, a.width - 8 * (int64_t)item), zero);
}

__device__ __forceinline__ uint32_t* in_work(const EmbeddingGradArgs& a, int64_t at) { return reinterpret_cast<uint32_t*>(a.work + at); }

// Few tokens: one workgroup sorts them in LDS, each as its number above its place in the batch
// (`place` bits), while the others clear the gradient's rows.
template <int IPT, int OUT>
__global__ __launch_bounds__(kSmallThreads) void k_embedding_sort(EmbeddingGradArgs a, int place, int bits) {
    constexpr int WAVES = kSmallThreads / 64;
    __shared__ uint32_t buffer[kSmallThreads * IPT], counts[WAVES * kDigits], sums[WAVES];
    if (blockIdx.x > 0) {
        clear_rows<OUT>(a, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    const int tid = threadIdx.x, wave = tid >> 6, first = wave * 64 * IPT + (tid & 63);
    uint32_t v[IPT];
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const int t = first + 64 * j;
        v[j] = t < a.count ? key_at(a, t) << place | (uint32_t)t : ~0u;     // past the last: behind all others
    }
    for (int shift = place; shift < place + bits; shift += 8) {
        for (int i = tid; i < WAVES * kDigits; i += kSmallThreads) counts[i] = 0;
        __syncthreads();
        uint32_t d[IPT], rank[IPT];
#pragma unroll
        for (int j = 0; j < IPT; ++j) d[j] = v[j] >> shift & (kDigits - 1);
        rank_in_wave<IPT>(d, counts + wave * kDigits, rank);
        __syncthreads();
        scan_counts<WAVES>(counts, sums);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IPT; ++j) buffer[counts[wave * kDigits + d[j]] + rank[j]] = v[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < IPT; ++j) v[j] = buffer[first + 64 * j];
    }
    uint32_t *keys = in_work(a, a.at.keys[0]), *order = in_work(a, a.at.order[0]);
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const int t = first + 64 * j;
        if (t >= a.count) continue;
        keys[t] = v[j] >> place;
        order[t] = v[j] & ((1u << place) - 1);
    }
}

// Many tokens: passes of eight bits, each counting digits in tiles of 4096 tokens, adding up the
// counts and moving the tokens.  Pass p writes buffer p % 2 and reads the other, the first one the
// batch.
template <int OUT> __global__ __launch_bounds__(kThreads) void k_embedding_count(EmbeddingGradArgs a, int pass, int64_t tiles) {
    __shared__ uint32_t counts[kDigits];
    if (blockIdx.x >= tiles) {
        clear_rows<OUT>(a, blockIdx.x - tiles, gridDim.x - tiles);
        return;
    }
    const uint32_t* keys = in_work(a, a.at.keys[1 - (pass & 1)]);
    for (int i = threadIdx.x; i < kDigits; i += kThreads) counts[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kTileItems; i += kThreads) {
        const int64_t t = (int64_t)blockIdx.x * kTileItems + i;
        if (t < a.count) atomicAdd(&counts[(pass ? keys[t] : key_at(a, t)) >> 8 * pass & (kDigits - 1)], 1u);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kDigits; i += kThreads) in_work(a, a.at.digits)[i * tiles + blockIdx.x] = counts[i];
}

// Counts (digit by digit, tile by tile) -> the sum of all before each.
__global__ __launch_bounds__(kSmallThreads) void k_embedding_scan(EmbeddingGradArgs a, int64_t tiles) {
    __shared__ uint32_t sums[2][kSmallThreads / 64];
    uint32_t* c = in_work(a, a.at.digits);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t base = 0;
    for (int64_t i0 = 0, n = kDigits * tiles, turn = 0; i0 < n; i0 += 4 * kSmallThreads, turn ^= 1) {
        uint32_t v[4], total = 0;
        const int64_t i = i0 + 4 * tid;                 // n is a multiple of 256
        const u32x4 w = i < n ? *reinterpret_cast<const u32x4*>(c + i) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = total;
            total += w[k];
        }
        uint32_t up = total;
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
            const uint32_t x = __shfl_up(up, k);
            if (lane >= k) up += x;
        }
        if (lane == 63) sums[turn][wave] = up;
        __syncthreads();
        uint32_t mine = base + up - total;
        for (int k = 0; k < kSmallThreads / 64; ++k) {
            if (k < wave) mine += sums[turn][k];
            base += sums[turn][k];
        }
        if (i < n) *reinterpret_cast<u32x4*>(c + i) = u32x4{v[0] + mine, v[1] + mine, v[2] + mine, v[3] + mine};
    }
}

__global__ __launch_bounds__(kThreads) void k_embedding_move(EmbeddingGradArgs a, int pass, int64_t tiles) {
    constexpr int WAVES = kThreads / 64, IPT = kTileItems / kThreads;
    __shared__ uint32_t counts[WAVES * kDigits];
    const int to = pass & 1, from = 1 - to;
    const uint32_t *keys = in_work(a, a.at.keys[from]), *order = in_work(a, a.at.order[from]);
    uint32_t *keys_to = in_work(a, a.at.keys[to]), *order_to = in_work(a, a.at.order[to]);
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int i = tid; i < WAVES * kDigits; i += kThreads) counts[i] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kTileItems + wave * 64 * IPT + (tid & 63);
    uint32_t key[IPT], place[IPT], d[IPT], rank[IPT];
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        const int64_t t = first + 64 * j;
        const bool in = t < a.count;
        key[j] = !in ? ~0u : pass ? keys[t] : key_at(a, t);
        place[j] = !in ? 0u : pass ? order[t] : (uint32_t)t;
        d[j] = key[j] >> 8 * pass & (kDigits - 1);      // past the last: counted behind all others, not moved
    }
    rank_in_wave<IPT>(d, counts + wave * kDigits, rank);
    __syncthreads();
    static_assert(kThreads == kDigits, "a digit for each thread");
    uint32_t base = in_work(a, a.at.digits)[tid * tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const uint32_t c = counts[w * kDigits + tid];
        counts[w * kDigits + tid] = base;
        base += c;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
        if (first + 64 * j >= a.count) continue;
        const uint32_t at = counts[wave * kDigits + d[j]] + rank[j];
        keys_to[at] = key[j];
        order_to[at] = place[j];
    }
}

// -------------------------------------------------------------------------- the sums

// First place in [lo, hi) whose key is not below `key`; keys are sorted.
__device__ __forceinline__ int64_t first_not_below(const uint32_t* keys, int64_t lo, int64_t hi, uint32_t key) {
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (gbl(keys)[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <int OUT>
__device__ __forceinline__ void put_row(const EmbeddingGradArgs& a, uint32_t key, int32_t item, const float sum[8]) {
    const int64_t e = (int64_t)key * a.ldo + 8 * (int64_t)item;
    const int n = (int)min((int64_t)8, a.width - 8 * (int64_t)item);
    float v[8];
    if (a.accumulate) {
        ld_eight<OUT, false>(a.out, e, n, 8 * (int64_t)item, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += sum[j] * a.scale;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sum[j] * a.scale;
    }
    st_eight<OUT>(a.out, e, n, v);
}

// Parts of long runs: a whole part that begins at place i lies in row 2 (i / span) of the partial
// sums, a run's last one, if shorter, in the row behind it.  Two whole parts begin at least `span`
// places apart, and so do two short ones of long runs.
__device__ __forceinline__ float* part_row(const EmbeddingGradArgs& a, int64_t i, bool whole) {
    return reinterpret_cast<float*>(a.work + a.at.partial) + (2 * (i / a.at.span) + !whole) * ((a.width + 7) / 8 * 8);
}

// A place of the sorted order for each group of lanes: those where a part begins add up its rows.
template <int DT, int OUT> __global__ __launch_bounds__(kThreads) void k_embedding_sums(EmbeddingGradArgs a, RowGrid g, int buffer) {
    const uint32_t *keys = in_work(a, a.at.keys[buffer]), *order = in_work(a, a.at.order[buffer]);
    const int64_t span = a.at.span;
    for_items(g, a.count, (int32_t)((a.width + 7) / 8), [&](int64_t i, int32_t item) {
        const uint32_t key = gbl(keys)[i];
        if (key >= (uint32_t)a.vocab) return;
        bool whole_run = false;                         // the run is one part
        if (i == 0 || gbl(keys)[i - 1] != key) {
            whole_run = i + span >= a.count || gbl(keys)[i + span] != key;
        } else {
            if (i < span || gbl(keys)[i - span] != key) return;
            if ((i - first_not_below(keys, 0, i - span, key)) % span != 0) return;
        }
        const int64_t last = min(i + span, a.count);
        const int64_t end = gbl(keys)[last - 1] == key ? last : first_not_below(keys, i, last, key + 1);
        const int64_t e = 8 * (int64_t)item;
        const int n = (int)min((int64_t)8, a.width - e);
        float sum[8] = {};
        int64_t r = i;
        for (; r + 4 <= end; r += 4) {
            float v[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) ld_eight<DT, true>(a.dy, (int64_t)gbl(order)[r + k] * a.lddy + e, n, e, v[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += v[k][j];
        }
        for (; r < end; ++r) {
            float v[8];
            ld_eight<DT, true>(a.dy, (int64_t)gbl(order)[r] * a.lddy + e, n, e, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += v[j];
        }
        if (whole_run) {
            put_row<OUT>(a, key, item, sum);
        } else {
            float* p = part_row(a, i, end - i == span) + e;
            *gbl(reinterpret_cast<f32x4*>(p)) = f32x4{sum[0], sum[1], sum[2], sum[3]};
            *gbl(reinterpret_cast<f32x4*>(p + 4)) = f32x4{sum[4], sum[5], sum[6], sum[7]};
        }
    });
}

// `span` places of the sorted order for each workgroup: at most one run of more than a part begins
// there, and its parts are added up.
template <int OUT> __global__ __launch_bounds__(kThreads) void k_embedding_join(EmbeddingGradArgs a, int buffer) {
    __shared__ int64_t begins;
    const uint32_t* keys = in_work(a, a.at.keys[buffer]);
    const int64_t span = a.at.span, windows = (a.count + span - 1) / span;
    for (int64_t w = blockIdx.x; w < windows; w += gridDim.x) {
        __syncthreads();
        if (threadIdx.x == 0) begins = -1;
        __syncthreads();
        for (int64_t i = w * span + threadIdx.x; i < min((w + 1) * span, a.count - span); i += kThreads) {
            const uint32_t key = gbl(keys)[i];
            if (key < (uint32_t)a.vocab && (i == 0 || gbl(keys)[i - 1] != key) && gbl(keys)[i + span] == key) begins = i;
        }
        __syncthreads();
        if (begins < 0) continue;
        const int64_t first = begins;
        const uint32_t key = gbl(keys)[first];
        const int64_t end = first_not_below(keys, first, a.count, key + 1);
        for (int32_t item = threadIdx.x; item < (int32_t)((a.width + 7) / 8); item += kThreads) {
            float sum[8] = {};
            for (int64_t i = first; i < end; i += span) {
                const float* p = part_row(a, i, end - i >= span) + 8 * (int64_t)item;
                const f32x4 lo = *gbl(reinterpret_cast<const f32x4*>(p)), hi = *gbl(reinterpret_cast<const f32x4*>(p + 4));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[j] += lo[j];
                    sum[4 + j] += hi[j];
                }
            }
            put_row<OUT>(a, key, item, sum);
        }
    }
}

// ------------------------------------------------------------------------- launches

static int bits_of(int64_t v) {
    int b = 0;
    while (v >> b) ++b;
    return b;
}

// Tokens that one workgroup sorts, and whether their numbers and places fit 32 bits together.
static int place_bits(int64_t count) { return bits_of(std::max<int64_t>(count, 1) - 1); }
static bool small_sort(int64_t count, int64_t vocab) {
    return count <= 16 * kSmallThreads && place_bits(count) + bits_of(vocab) <= 32;
}

EmbeddingSpace embedding_space(int64_t count, int64_t vocab, int64_t width) {
    EmbeddingSpace s{};
    // a run of all tokens is twice as many parts as a part has rows, at most
    s.span = 32;
    while (4 * s.span * s.span < count) s.span *= 2;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t p = at;
        at += (bytes + 15) / 16 * 16;
        return p;
    };
    const bool small = small_sort(count, vocab);
    for (int b = 0; b < (small ? 1 : 2); ++b) {
        s.keys[b] = take(4 * count);
        s.order[b] = take(4 * count);
    }
    if (!small) s.digits = take(4 * kDigits * ((count + kTileItems - 1) / kTileItems));
    // not less than fewer tokens take, whose parts are shorter: a workspace for a count serves all below
    const int64_t parts = std::max<int64_t>(2 * ((count + s.span - 1) / s.span), s.span > 32 ? 4 * s.span : 0);
    if (count > s.span) s.partial = take(parts * ((width + 7) / 8 * 8) * 4);
    s.bytes = at;
    return s;
}

template <int OUT> static hipError_t sort_tokens(const EmbeddingGradArgs& a, int& buffer, hipStream_t s) {
    // 16 KB of rows for each clearing workgroup, on all CUs several times over at most
    const int64_t clear = a.accumulate ? 0 : std::max<int64_t>(1, std::min<int64_t>(a.vocab * a.width / 4096, 2048));
    const int bits = bits_of(a.vocab);
    buffer = 0;
    if (small_sort(a.count, a.vocab)) {
        const int place = place_bits(a.count);
        const dim3 grid((unsigned)(1 + clear));
        if (a.count <= kSmallThreads) hipLaunchKernelGGL((k_embedding_sort<1, OUT>), grid, dim3(kSmallThreads), 0, s, a, place, bits);
        else if (a.count <= 4 * kSmallThreads) hipLaunchKernelGGL((k_embedding_sort<4, OUT>), grid, dim3(kSmallThreads), 0, s, a, place, bits);
        else if (a.count <= 8 * kSmallThreads) hipLaunchKernelGGL((k_embedding_sort<8, OUT>), grid, dim3(kSmallThreads), 0, s, a, place, bits);
        else hipLaunchKernelGGL((k_embedding_sort<16, OUT>), grid, dim3(kSmallThreads), 0, s, a, place, bits);
        return hipGetLastError();
    }
    const int64_t tiles = (a.count + kTileItems - 1) / kTileItems;
    for (int pass = 0; 8 * pass < bits; ++pass) {
        const dim3 grid((unsigned)(tiles + (pass == 0 ? clear : 0)));
        hipLaunchKernelGGL((k_embedding_count<OUT>), grid, dim3(kThreads), 0, s, a, pass, tiles);
        hipLaunchKernelGGL(k_embedding_scan, dim3(1), dim3(kSmallThreads), 0, s, a, tiles);
        hipLaunchKernelGGL(k_embedding_move, dim3((unsigned)tiles), dim3(kThreads), 0, s, a, pass, tiles);
        if (hipError_t e = hipGetLastError()) return e;
        buffer = pass & 1;
    }
    return hipSuccess;
}

template <int OUT> static hipError_t embedding_grad(const EmbeddingGradArgs& a, int dtype, hipStream_t s) {
    int buffer;
    if (hipError_t e = sort_tokens<OUT>(a, buffer, s)) return e;
    if (a.count == 0) return hipSuccess;
    dim3 grid;
    const RowGrid g = row_grid(a.count, (a.width + 7) / 8, grid);
    if (dtype == kF32) hipLaunchKernelGGL((k_embedding_sums<kF32, OUT>), grid, dim3(kThreads), 0, s, a, g, buffer);
    else if (dtype == kF16) hipLaunchKernelGGL((k_embedding_sums<kF16, OUT>), grid, dim3(kThreads), 0, s, a, g, buffer);
    else hipLaunchKernelGGL((k_embedding_sums<kBF16, OUT>), grid, dim3(kThreads), 0, s, a, g, buffer);
    if (a.count > a.at.span) {
        const int64_t windows = (a.count + a.at.span - 1) / a.at.span;
        hipLaunchKernelGGL((k_embedding_join<OUT>), dim3((unsigned)std::min<int64_t>(windows, 65535)), dim3(kThreads), 0, s, a, buffer);
    }
    return hipGetLastError();
}

hipError_t launch_embedding_grad(const EmbeddingGradArgs& a, int dtype, int out_dtype, hipStream_t s) {
    return out_dtype == kF32 ? embedding_grad<kF32>(a, dtype, s)
                             : out_dtype == kF16 ? embedding_grad<kF16>(a, dtype, s) : embedding_grad<kBF16>(a, dtype, s);
}

template <int DT> static hipError_t embedding(const EmbeddingArgs& a, int out_dtype, hipStream_t s) {
    dim3 grid;
    const RowGrid g = row_grid(a.count, (a.width + 7) / 8, grid);
    if (out_dtype == kF32) hipLaunchKernelGGL((k_embedding<DT, kF32>), grid, dim3(kThreads), 0, s, a, g);
    else if (out_dtype == kF16) hipLaunchKernelGGL((k_embedding<DT, kF16>), grid, dim3(kThreads), 0, s, a, g);
    else hipLaunchKernelGGL((k_embedding<DT, kBF16>), grid, dim3(kThreads), 0, s, a, g);
    return hipGetLastError();
}

hipError_t launch_embedding(const EmbeddingArgs& a, int dtype, int out_dtype, hipStream_t s) {
    return dtype == kF32 ? embedding<kF32>(a, out_dtype, s) : dtype == kF16 ? embedding<kF16>(a, out_dtype, s) : embedding<kBF16>(a, out_dtype, s);
}

template <int FMT> static hipError_t mx_embedding(const EmbeddingArgs& a, int out_dtype, hipStream_t s) {
    dim3 grid;
    const RowGrid g = row_grid(a.count, (a.width + 7) / 8, grid);
    if (out_dtype == kF32) hipLaunchKernelGGL((k_mx_embedding<FMT, kF32>), grid, dim3(kThreads), 0, s, a, g);
    else if (out_dtype == kF16) hipLaunchKernelGGL((k_mx_embedding<FMT, kF16>), grid, dim3(kThreads), 0, s, a, g);
    else hipLaunchKernelGGL((k_mx_embedding<FMT, kBF16>), grid, dim3(kThreads), 0, s, a, g);
    return hipGetLastError();
}

hipError_t launch_mx_embedding(const EmbeddingArgs& a, int fmt, int out_dtype, hipStream_t s) {
    return fmt == kMxE2M1 ? mx_embedding<kMxE2M1>(a, out_dtype, s) : mx_embedding<kMxE4M3>(a, out_dtype, s);
}

}  // namespace bitopt
