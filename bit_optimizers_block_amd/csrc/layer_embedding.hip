// Embedding lookup, from a table of elements or an MX matrix, and its gradient by sorted tokens.
//
// Gradient: out[v] (+)= scale * the sum of dy[t] over the tokens t with number v.  Tokens are
// sorted by number with a stable radix sort, so the rows of one number are a run of the sorted
// order, in their order in the batch: no atomics, and the same bits on every run.  The order is
// cut into windows of `span` places, each added up by one group of lanes with eight rows in
// flight, whatever the runs' lengths; a run that lies in several windows (a frequent token)
// leaves its parts in the workspace, and a second kernel adds those in their order.
//
// Measured, 8192 bf16 rows of 2048 into 50257 fp32 rows: 95 us, of which 65 clear the table (6.3 TB/s;
// the sort, 17.6 by itself, runs beside that), 22 are the sums and 7 the parts; added to what is
// there 46.  The sums wait for three loads in turn (places, rows, the table's rows where added) and
// find the memory still busy with the cleared rows.  Clearing only 64 MB beside the sort and the
// rest, less the rows with a token, beside the sums: 128 us of a pass with the lookup against 121.
// Streamed stores of the zeros: 128 against 124.  The lookup (100 MB) takes 12.5 us.
#include "launch.h"
#include "layer.h"
#include "mx_rows.h"

namespace bitopt {

// ---------------------------------------------------------------------------- lookup

__device__ __forceinline__ int64_t token_at(const void* tokens, bool wide, int64_t t) {
    return wide ? gbl(reinterpret_cast<const int64_t*>(tokens))[t] : (int64_t)gbl(reinterpret_cast<const int32_t*>(tokens))[t];
}

// Elements of a lane: four where fp32 is written.
template <int OUT> constexpr int kEach = OUT == kF32 ? 4 : 8;

// A token outside the table gets zeros.
template <int DT, int OUT> __global__ __launch_bounds__(kThreads) void k_embedding(EmbeddingArgs a, RowGrid g) {
    constexpr int PER = kEach<OUT>;
    for_items(g, a.count, (int32_t)((a.width + PER - 1) / PER), [&](int64_t row, int32_t item) {
        const int64_t e = PER * (int64_t)item;
        const int n = (int)min((int64_t)PER, a.width - e);
        const int64_t id = token_at(a.tokens, a.wide, row);
        float v[PER] = {};
        if ((uint64_t)id < (uint64_t)a.vocab) ld_row<DT, PER>(a.table, id * a.ldt + e, n, e, v);
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] *= a.scale;
        st_row<OUT, PER>(a.out, row * a.ldo + e, n, v);
    });
}

template <int FMT, int OUT> __global__ __launch_bounds__(kThreads) void k_mx_embedding(EmbeddingArgs a, RowGrid g) {
    constexpr int PER = kEach<OUT>;
    const int64_t bytes = mx_code_bytes(a.width, FMT), blocks = mx_scale_bytes(a.width);
    for_items(g, a.count, (int32_t)((a.width + PER - 1) / PER), [&](int64_t row, int32_t item) {
        const int64_t id = token_at(a.tokens, a.wide, row);
        float v[PER] = {};
        if ((uint64_t)id < (uint64_t)a.vocab) {
            const float s = mx_scale_f32(gbl(a.scales)[id * blocks + item / (kMxBlock / PER)]);
            const uint8_t* p = a.codes + id * bytes + (int64_t)item * (FMT == kMxE2M1 ? PER / 2 : PER);
#pragma unroll
            for (int h = 0; h < PER / 4; ++h) {
                if constexpr (FMT == kMxE2M1) mx_decode4_e2m1(gbl(reinterpret_cast<const uint16_t*>(p))[h], s, v + 4 * h);
                else mx_decode4_e4m3(gbl(reinterpret_cast<const uint32_t*>(p))[h], s, v + 4 * h);
            }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] *= a.scale;
        const int64_t e = PER * (int64_t)item;
        st_row<OUT, PER>(a.out, row * a.ldo + e, (int)min((int64_t)PER, a.width - e), v);
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

// Zeros in every row of the gradient: `part` of `parts` workgroups.  Rows without gaps are one.
template <int OUT> __device__ __forceinline__ void clear_rows(const EmbeddingGradArgs& a, int64_t part, int64_t parts) {
    constexpr int PER = kPer<OUT>;
    const bool gaps = a.ldo != a.width;
    const int64_t rows = gaps ? a.vocab : 1, width = gaps ? a.width : a.vocab * a.width, items = (width + PER - 1) / PER;
    const float zero[PER] = {};
    if (!gaps) {
        for (int64_t i = part * blockDim.x + threadIdx.x; i < items; i += parts * blockDim.x)
            st_item<OUT, false>(a.out, PER * i, (int)min((int64_t)PER, width - PER * i), zero);
        return;
    }
    int lanes = 64;
    while (lanes < (int)blockDim.x && lanes < items) lanes *= 2;
    const int per = (int)blockDim.x / lanes;
    for (int64_t row = part * per + threadIdx.x / lanes; row < rows; row += parts * per)
        for (int64_t i = threadIdx.x % lanes; i < items; i += lanes)
            st_item<OUT, false>(a.out, row * a.ldo + PER * i, (int)min((int64_t)PER, width - PER * i), zero);
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

template <int OUT>
__device__ __forceinline__ void put_row(const EmbeddingGradArgs& a, uint32_t key, int32_t item, const float sum[8]) {
    const int64_t e = (int64_t)key * a.ldo + 8 * (int64_t)item;
    const int n = (int)min((int64_t)8, a.width - 8 * (int64_t)item);
    float v[8];
    if (a.accumulate) {
        ld_row<OUT, 8>(a.out, e, n, 8 * (int64_t)item, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += sum[j] * a.scale;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sum[j] * a.scale;
    }
    st_row<OUT, 8, false>(a.out, e, n, v);
}

// Window w's rows of partial sums: of the run that comes from the window before, and of one that
// begins in it and goes on in the next.
__device__ __forceinline__ float* part_row(const EmbeddingGradArgs& a, int64_t w, bool begins) {
    return reinterpret_cast<float*>(a.work + a.at.partial) + (2 * w + begins) * ((a.width + 7) / 8 * 8);
}

// Up to eight rows at a time, all of them and, where sums are added to it, the gradient's rows
// under way together.
template <int DT, int OUT, bool ADD>
__global__ __launch_bounds__(kThreads) void k_embedding_sums(EmbeddingGradArgs a, int lanes_log2, int buffer) {
    constexpr int U = 8;
    const uint32_t *keys = in_work(a, a.at.keys[buffer]), *order = in_work(a, a.at.order[buffer]);
    const int64_t span = a.at.span, windows = (a.count + span - 1) / span, per = kThreads >> lanes_log2;
    const int32_t item = (int32_t)(blockIdx.x << lanes_log2) + (threadIdx.x & ((1 << lanes_log2) - 1));
    const int64_t e = 8 * (int64_t)item, over = e + 8 - a.width;
    if (over >= 8) return;
    const uint32_t none = (uint32_t)a.vocab;
    for (int64_t w = per * blockIdx.y + (threadIdx.x >> lanes_log2); w < windows; w += per * gridDim.y) {
        const int64_t first = w * span, end = min(first + span, a.count);
        uint32_t run = gbl(keys)[first];
        // whether the run at hand began in this window
        bool begins = first == 0 || gbl(keys)[first - 1] != run;
        float sum[8] = {};
        for (int64_t i = first; i < end && run < none; i += U) {
            uint32_t key[U + 1], from[U];
            float v[U][8], old[ADD ? U : 1][8];
#pragma unroll
            for (int k = 0; k <= U; ++k) {
                const uint32_t at = gbl(keys)[min(i + k, a.count - 1)];
                key[k] = i + k < a.count ? at : none;
                if (k < U) from[k] = gbl(order)[min(i + k, end - 1)];
            }
            if (a.width >= 8) {
                Eight<DT> in[U];
                Eight<OUT> was[ADD ? U : 1];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    in[k].template load<false>(a.dy, (int64_t)from[k] * a.lddy, e, a.width);
                    if constexpr (ADD) was[k].template load<false>(a.out, (key[k] < none ? key[k] : 0) * a.ldo, e, a.width);
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    in[k].values(over, v[k]);
                    if constexpr (ADD) was[k].values(over, old[k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool in = j < a.width;
                        v[k][j] = in ? load1<DT>(a.dy, (int64_t)from[k] * a.lddy + j) : 0.0f;
                        if constexpr (ADD) old[k][j] = in ? load1<OUT>(a.out, (key[k] < none ? key[k] : 0) * a.ldo + j) : 0.0f;
                    }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (i + k >= end || key[k] >= none) break;
                run = key[k];
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] += v[k][j];
                if (key[k + 1] == run && i + k + 1 < end) continue;
                // the run's last row here
                if (begins && key[k + 1] != run) {
                    float y[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        y[j] = sum[j] * a.scale;
                        if constexpr (ADD) y[j] = old[k][j] + y[j];
                    }
                    st_row<OUT, 8, false>(a.out, run * a.ldo + e, (int)min((int64_t)8, a.width - e), y);
                } else {
                    float* p = part_row(a, w, begins) + e;
                    *gbl(reinterpret_cast<f32x4*>(p)) = f32x4{sum[0], sum[1], sum[2], sum[3]};
                    *gbl(reinterpret_cast<f32x4*>(p + 4)) = f32x4{sum[4], sum[5], sum[6], sum[7]};
                }
                begins = true;
                run = key[k + 1];
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
            }
        }
    }
}

constexpr int kJoinThreads = 512;

// Adds up the parts of the run that begins in a window and goes on in the next, if there is one:
// each group of lanes a stretch of them, the groups' sums in LDS in their order.
template <int OUT> __global__ __launch_bounds__(kJoinThreads) void k_embedding_join(EmbeddingGradArgs a, int lanes_log2, int buffer) {
    __shared__ f32x4 sums[2][kJoinThreads];
    const uint32_t* keys = in_work(a, a.at.keys[buffer]);
    const int64_t span = a.at.span, windows = (a.count + span - 1) / span;
    const int lanes = 1 << lanes_log2, groups = kJoinThreads >> lanes_log2;
    const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x >> lanes_log2;
    for (int64_t w = blockIdx.x; w + 1 < windows; w += gridDim.x) {
        const int64_t first = w * span;
        const uint32_t run = gbl(keys)[first + span];
        if (run >= (uint32_t)a.vocab || gbl(keys)[first + span - 1] != run) continue;
        if (first > 0 && gbl(keys)[first - 1] == run) continue;
        // windows that begin with the run: w + 1 and those behind it without a gap
        int64_t parts = 1;
        for (int64_t v = w + 1; v < windows; v += 64) {
            const int64_t at = (v + (threadIdx.x & 63)) * span;
            const uint64_t other = __ballot(at >= a.count || gbl(keys)[min(at, a.count - 1)] != run);
            parts += other ? __builtin_ctzll(other) : 64;
            if (other) break;
        }
        const int64_t stretch = (parts + groups - 1) / groups, lo = group * stretch, hi = min(lo + stretch, parts);
        for (int64_t c = lane; c < (int64_t)((a.width + 7) / 8 + lanes - 1) / lanes * lanes; c += lanes) {
            const bool in = c < (a.width + 7) / 8;
            f32x4 s0 = {0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
            if (in) {
#pragma unroll 8
                for (int64_t v = lo; v < hi; ++v) {
                    const float* p = part_row(a, w + v, v == 0) + 8 * c;
                    s0 += *gbl(reinterpret_cast<const f32x4*>(p));
                    s1 += *gbl(reinterpret_cast<const f32x4*>(p + 4));
                }
            }
            __syncthreads();                // the last columns' sums have been read
            sums[0][threadIdx.x] = s0;
            sums[1][threadIdx.x] = s1;
            __syncthreads();
            if (group == 0 && in) {
                for (int k = 1; k < groups && k * stretch < parts; ++k) {
                    s0 += sums[0][k * lanes + lane];
                    s1 += sums[1][k * lanes + lane];
                }
                const float sum[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                put_row<OUT>(a, run, (int32_t)c, sum);
            }
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
    // Eight places are one round of loads; more of them in a window, fewer parts to join.  us, added
    // gradient, with up to 2048, 1024, 768 and 512 windows (768 are 512 where count is a power of two): 8192
    // tokens, width 2048: 49.5, 49.4, 45.9, 46.5 (all the same token: 119, 118, 73, 73); 16384, 2048: 82, 73, 69,
    // 69; 32768, 1024: 86, 79, 81, 80; 65536, 512: 82, 83, 101, 101, where a workgroup takes four windows.
    const int64_t most = width > 512 ? 768 : 1024;
    s.span = 8;
    while (most * s.span < count) s.span *= 2;
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
    // not less than fewer tokens take, whose windows are shorter: a workspace for a count serves all below
    const int64_t parts = std::max<int64_t>(2 * ((count + s.span - 1) / s.span), s.span > 8 ? 2 * most : 0);
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

template <int DT, int OUT> static void sums(const EmbeddingGradArgs& a, dim3 grid, int lanes_log2, int buffer, hipStream_t s) {
    if (a.accumulate) hipLaunchKernelGGL((k_embedding_sums<DT, OUT, true>), grid, dim3(kThreads), 0, s, a, lanes_log2, buffer);
    else hipLaunchKernelGGL((k_embedding_sums<DT, OUT, false>), grid, dim3(kThreads), 0, s, a, lanes_log2, buffer);
}

template <int OUT> static hipError_t embedding_grad(const EmbeddingGradArgs& a, int dtype, hipStream_t s) {
    int buffer;
    if (hipError_t e = sort_tokens<OUT>(a, buffer, s)) return e;
    if (a.count == 0) return hipSuccess;
    const int64_t windows = (a.count + a.at.span - 1) / a.at.span, items = (a.width + 7) / 8;
    int lanes_log2 = 4;
    while (lanes_log2 < 8 && (1 << lanes_log2) < items) ++lanes_log2;
    const int64_t per = kThreads >> lanes_log2;
    const dim3 grid((unsigned)((items + (1 << lanes_log2) - 1) >> lanes_log2), (unsigned)std::min<int64_t>((windows + per - 1) / per, 65535));
    if (dtype == kF32) sums<kF32, OUT>(a, grid, lanes_log2, buffer, s);
    else if (dtype == kF16) sums<kF16, OUT>(a, grid, lanes_log2, buffer, s);
    else sums<kBF16, OUT>(a, grid, lanes_log2, buffer, s);
    if (windows > 1)
        hipLaunchKernelGGL((k_embedding_join<OUT>), dim3((unsigned)std::min<int64_t>(windows - 1, 65535)), dim3(kJoinThreads), 0, s, a,
                           lanes_log2, buffer);
    return hipGetLastError();
}

hipError_t launch_embedding_grad(const EmbeddingGradArgs& a, int dtype, int out_dtype, hipStream_t s) {
    return out_dtype == kF32 ? embedding_grad<kF32>(a, dtype, s)
                             : out_dtype == kF16 ? embedding_grad<kF16>(a, dtype, s) : embedding_grad<kBF16>(a, dtype, s);
}

template <int DT> static hipError_t embedding(const EmbeddingArgs& a, int out_dtype, hipStream_t s) {
    dim3 grid;
    const int per = out_dtype == kF32 ? 4 : 8;
    const RowGrid g = row_grid(a.count, (a.width + per - 1) / per, grid);
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
    const int per = out_dtype == kF32 ? 4 : 8;
    const RowGrid g = row_grid(a.count, (a.width + per - 1) / per, grid);
    if (out_dtype == kF32) hipLaunchKernelGGL((k_mx_embedding<FMT, kF32>), grid, dim3(kThreads), 0, s, a, g);
    else if (out_dtype == kF16) hipLaunchKernelGGL((k_mx_embedding<FMT, kF16>), grid, dim3(kThreads), 0, s, a, g);
    else hipLaunchKernelGGL((k_mx_embedding<FMT, kBF16>), grid, dim3(kThreads), 0, s, a, g);
    return hipGetLastError();
}

hipError_t launch_mx_embedding(const EmbeddingArgs& a, int fmt, int out_dtype, hipStream_t s) {
    return fmt == kMxE2M1 ? mx_embedding<kMxE2M1>(a, out_dtype, s) : mx_embedding<kMxE4M3>(a, out_dtype, s);
}

}  // namespace bitopt
