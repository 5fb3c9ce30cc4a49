// ls_experts.hip -- tokens to the rows of their experts and back (gfx950).
//
// A token t goes to `top` experts; pair p = t * top + j.  The sort is a stable counting sort of
// the pairs by expert: a histogram per tile of pairs, prefix sums over (expert, tile), and a
// rank among the pairs of the same expert in the tile, found 64 pairs at a time by comparing
// expert numbers bit by bit across the wave (one ballot a bit).  The moves of rows read each
// token's places once and go over its channels 16 bytes a lane: the gather reads a token's row
// once and writes it to all its places, the combination reads all its places and writes one
// row, its gradient reads both and writes both.  A place that is not a row (a pair over its
// expert's capacity) takes part in nothing.
#include "ls_elements.hpp"
#include "ls_internal.hpp"

namespace ls {

// ---------------------------------------------------------------- sort

// Pairs per turn and sort of 16384 x 8, 8192 x 4, 32768 x 8 and 131072 x 8 pairs by 256, 64, 128 and 256 experts: 2048 10.7, 8.5,
// 10.9, 28.4 us; 1024 10.8, 8.1, 11.2, 29.8; 4096 13.5, 11.4, 13.1, 27.5 (too few blocks but for the last).  What is left are
// two launches of a few microseconds: the counts, and each block's sums over the tiles' counts and its ranks.
constexpr int EX_BLOCK = 512;
constexpr int EX_WAVES = EX_BLOCK / 64;
constexpr int EX_STEPS = 4;                              // pairs per lane and turn
constexpr int EX_TURN = EX_BLOCK * EX_STEPS;             // pairs per block and turn
constexpr int EX_TILES = 128;                            // most tiles

struct ExpertsTiles {
    int64_t n, per_tile;  // pairs; pairs per tile, a multiple of EX_TURN
    int tiles;
};
static ExpertsTiles experts_tiles(int64_t n)
{
    const int64_t turns = n > 0 ? (n + EX_TURN - 1) / EX_TURN : 1;
    // two turns of one block are sooner done than a launch more: 2331 pairs 7.2 us against 8.2
    const int64_t per = turns <= 2 ? turns : (turns + EX_TILES - 1) / EX_TILES;
    return {n, per * EX_TURN, int((turns + per - 1) / per)};
}

// The expert of a pair, or `experts` for one that goes nowhere.
template <class I>
__device__ __forceinline__ uint32_t expert_of(const I* ids, int64_t p, int64_t n, int experts)
{
    if (p >= n)
        return uint32_t(experts);
    const int64_t e = ids[p];
    return e >= 0 && e < experts ? uint32_t(e) : uint32_t(experts);
}

// 16384 tokens of 8 choices of 256 experts: 4.7 us, and 8.1 for the places below; 256 pairs: the places alone, 4.6.
template <class I>
__global__ __launch_bounds__(EX_BLOCK) void experts_count_kernel(const I* ids, ExpertsTiles t, int experts, uint32_t* counts)
{
    extern __shared__ uint32_t count[];  // one per expert, and one for pairs without
    for (int e = threadIdx.x; e <= experts; e += EX_BLOCK)
        count[e] = 0;
    __syncthreads();
    const int64_t from = blockIdx.x * t.per_tile, to = from + t.per_tile < t.n ? from + t.per_tile : t.n;
    for (int64_t p = from + threadIdx.x; p < to; p += EX_BLOCK)
        atomicAdd(&count[expert_of(ids, p, t.n, experts)], 1u);
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += EX_BLOCK)
        counts[int64_t(blockIdx.x) * experts + e] = count[e];
}

// With one tile the counts are made here (counts == NULL).
template <class I>
__global__ __launch_bounds__(EX_BLOCK) void experts_place_kernel(const I* ids, ExpertsTiles t, int experts, int bits,
                                                                 const uint32_t* counts, int64_t* offsets, int32_t* order,
                                                                 int32_t* places)
{
    extern __shared__ uint32_t shared[];
    uint32_t* base = shared;                       // [experts + 1]: the next row of each expert
    uint32_t* seen = shared + experts + 1;         // [waves][experts + 1]
    __shared__ uint32_t wave_total[EX_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t from = blockIdx.x * t.per_tile, to = from + t.per_tile < t.n ? from + t.per_tile : t.n;
    if (counts == nullptr) {
        for (int e = tid; e <= experts; e += EX_BLOCK)
            seen[e] = 0;
        __syncthreads();
        for (int64_t p = from + tid; p < to; p += EX_BLOCK)
            atomicAdd(&seen[expert_of(ids, p, t.n, experts)], 1u);
        __syncthreads();
    }
    // each expert's pairs in all tiles and in the tiles in front, by several threads an expert where these are few
    uint32_t* before = shared + (1 + EX_WAVES) * (experts + 1);  // [experts]
    if (counts != nullptr) {
        for (int e = tid; e < experts; e += EX_BLOCK)
            seen[e] = before[e] = 0;
        __syncthreads();
        int wide = 64;
        while (wide < experts && wide < EX_BLOCK)
            wide *= 2;
        const int split = EX_BLOCK / wide, part = tid / wide;
        for (int e = tid % wide; e < experts; e += wide) {
            uint32_t total = 0, front = 0;
#pragma unroll 8
            for (int i = part; i < t.tiles; i += split) {
                const uint32_t c = counts[int64_t(i) * experts + e];
                total += c;
                front += i < int(blockIdx.x) ? c : 0;
            }
            atomicAdd(&seen[e], total);
            atomicAdd(&before[e], front);
        }
        __syncthreads();
    }
    // prefix sums over the experts, EX_BLOCK of them at a time
    uint32_t carry = 0;
    for (int e0 = 0; e0 < experts; e0 += EX_BLOCK) {
        const int e = e0 + tid;
        const uint32_t total = e < experts ? seen[e] : 0, front = e < experts && counts != nullptr ? before[e] : 0;
        const uint32_t incl = wave_inclusive_scan<SumU32>(total);
        if (lane == 63)
            wave_total[wave] = incl;
        __syncthreads();
        uint32_t first = carry;
        for (int w = 0; w < EX_WAVES; ++w) {
            first += w < wave ? wave_total[w] : 0;
            carry += wave_total[w];
        }
        if (e < experts) {
            base[e] = first + incl - total + front;
            if (blockIdx.x == 0)
                offsets[e] = first + incl - total;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0)
        offsets[experts] = carry;
    for (int64_t turn = from; turn < to; turn += EX_TURN) {
        for (int e = tid; e < EX_WAVES * (experts + 1); e += EX_BLOCK)
            seen[e] = 0;
        __syncthreads();
        // volatile: a lane reads what other lanes of its wave wrote a step before
        volatile uint32_t* mine = seen + wave * (experts + 1);
        uint32_t ex[EX_STEPS], rank[EX_STEPS];
        const int64_t p0 = turn + wave * (64 * EX_STEPS) + lane;
#pragma unroll
        for (int i = 0; i < EX_STEPS; ++i)
            ex[i] = expert_of(ids, p0 + i * 64, t.n, experts);
#pragma unroll
        for (int i = 0; i < EX_STEPS; ++i) {
            uint64_t peers = ~0ull;
            for (int b = 0; b < bits; ++b) {
                const bool on = (ex[i] >> b) & 1;
                const uint64_t m = __ballot(on);
                peers &= on ? m : ~m;
            }
            const uint32_t old = mine[ex[i]];
            const uint32_t lower = __builtin_popcountll(peers & ((1ull << lane) - 1));
            rank[i] = old + lower;
            if (lower == 0)
                mine[ex[i]] = old + uint32_t(__builtin_popcountll(peers));
        }
        __syncthreads();
        // where each wave's pairs of an expert begin
        for (int e = tid; e < experts; e += EX_BLOCK) {
            uint32_t next = base[e];
            for (int w = 0; w < EX_WAVES; ++w) {
                const uint32_t c = seen[w * (experts + 1) + e];
                seen[w * (experts + 1) + e] = next;
                next += c;
            }
            base[e] = next;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EX_STEPS; ++i) {
            const int64_t p = p0 + i * 64;
            if (p < to) {
                const bool routed = ex[i] < uint32_t(experts);
                const uint32_t row = mine[ex[i]] + rank[i];
                places[p] = routed ? int32_t(row) : -1;
                if (routed)
                    order[row] = int32_t(p);
            }
        }
        __syncthreads();
    }
    for (int64_t i = from + tid; i < to; i += EX_BLOCK)
        if (i >= carry)
            order[i] = -1;
}

size_t experts_workspace_bytes(int64_t pairs, int64_t experts)
{
    const ExpertsTiles t = experts_tiles(pairs);
    return 256 + (t.tiles > 1 ? size_t(t.tiles) * size_t(experts) * 4 : 0);
}

template <class I>
static hipError_t experts_sort_of(const I* ids, int64_t pairs, int experts, int64_t* offsets, int32_t* order, int32_t* places,
                                  void* ws, hipStream_t stream)
{
    const ExpertsTiles t = experts_tiles(pairs);
    uint32_t* counts = t.tiles > 1 ? reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + 256) : nullptr;
    int bits = 1;
    while ((1 << bits) <= experts)  // `experts` itself is a value too
        ++bits;
    const size_t row = size_t(experts + 1) * 4;
    if (counts != nullptr)
        experts_count_kernel<I><<<dim3(t.tiles), dim3(EX_BLOCK), row, stream>>>(ids, t, experts, counts);
    experts_place_kernel<I><<<dim3(t.tiles), dim3(EX_BLOCK), row * (2 + EX_WAVES), stream>>>(
        ids, t, experts, bits, counts, offsets, order, places);
    return hipGetLastError();
}

hipError_t launch_experts_sort(const void* ids, int id_bits, int64_t pairs, int64_t experts, int64_t* offsets, int32_t* order,
                               int32_t* places, void* ws, hipStream_t stream)
{
    if (id_bits == 32)
        return experts_sort_of(static_cast<const int32_t*>(ids), pairs, int(experts), offsets, order, places, ws, stream);
    return experts_sort_of(static_cast<const int64_t*>(ids), pairs, int(experts), offsets, order, places, ws, stream);
}

// ---------------------------------------------------------------- rows

// A block is `x` lanes over a row's parts of VEC channels by `y` tokens.  A launch holds less than 2^32
// threads along x, so a block may take several tokens.
constexpr int64_t EX_GRID = 1 << 20;
struct RowGrid {
    dim3 grid, block;
};
static RowGrid row_grid(int64_t tokens, int64_t parts, int most)
{
    int x = 8;
    while (x < most && x < parts)
        x *= 2;
    const int y = 256 / x;
    const int64_t blocks = (tokens + y - 1) / y;
    return {dim3(uint32_t(blocks < EX_GRID ? blocks : EX_GRID), uint32_t((parts + x - 1) / x)), dim3(x, y)};
}

constexpr int EX_FLIGHT = 8;  // rows on their way at once

// Of a token's pairs j0 .. j0 + N - 1: the rows (-1: none) and the weights.  All are loaded before any is looked
// at: one wait, where a look at each place before its weight took one for each pair.
template <int N>
__device__ __forceinline__ void pairs_of(const ExpertsRows& q, int64_t t, int j0, int64_t (&at)[N], float (&w)[N])
{
    int32_t place[N];
    uint32_t b[N];
    const int64_t first = t * q.top + j0;
    const int count = q.top - j0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        place[i] = -1;
        b[i] = 0;
        w[i] = 1.0f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < count)
            place[i] = q.places[first + i];
    if (q.weights != nullptr) {
        if (q.weight_type == LOGITS_F32) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < count)
                    b[i] = static_cast<const uint32_t*>(q.weights)[first + i];
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = from_bits<float>(b[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < count)
                    b[i] = static_cast<const uint16_t*>(q.weights)[first + i];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float v[1];
                if (q.weight_type == LOGITS_F16)
                    F16::unpack(b[i], v);
                else
                    BF16::unpack(b[i], v);
                w[i] = v[0];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        at[i] = place[i] >= 0 && place[i] < q.rows_count ? place[i] : -1;
}

// A thread's first token.  Where a wave has one token, in a scalar register: its places and weights are then
// scalar loads and branches.
template <bool WAVE>
__device__ __forceinline__ int64_t first_token()
{
    const uint32_t y = WAVE ? uint32_t(__builtin_amdgcn_readfirstlane(int(threadIdx.y))) : threadIdx.y;
    return int64_t(blockIdx.x) * blockDim.y + y;
}

// Bound by its writes: 16384 tokens to 8 rows of 2048 bfloat16 each, 604 MB, take 101 us (6.0 TB/s); 32 tokens 3.0.
template <class E, int VEC, bool WAVE, bool PAST>
__global__ __launch_bounds__(256) void experts_gather_kernel(ExpertsRows q)
{
    const int64_t c = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * VEC;
    if (c >= q.channels)
        return;
    for (int64_t t = first_token<WAVE>(); t < q.tokens; t += int64_t(gridDim.x) * blockDim.y) {
        Elements<E, VEC> v;
        v.load(static_cast<const char*>(q.x) + (t * q.x_row + c) * E::size);
        for (int j0 = 0; j0 < q.top; j0 += EX_FLIGHT) {
            float w[EX_FLIGHT];
            int64_t at[EX_FLIGHT];
            pairs_of(q, t, j0, at, w);
#pragma unroll
            for (int i = 0; i < EX_FLIGHT; ++i)
                if (at[i] >= 0)
                    v.template store<PAST>(static_cast<char*>(q.rows_out) + (at[i] * q.rows_out_row + c) * E::size);
        }
    }
}

// Bound by its reads: 8192 tokens of 8 rows of 4096 bfloat16, 604 MB, take 101 us (6.0 TB/s), 61 tokens of 6 rows of 5120 float16
// 3.6.  N rows at once, as many as a token has or EX_FLIGHT: with 8 for every call, 4096 tokens of 2 rows took 76 us against 65.
template <class E, int VEC, int N, bool WAVE, bool ONCE, bool PAST>
__global__ __launch_bounds__(256) void experts_combine_kernel(ExpertsRows q)
{
    const int64_t c = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * VEC;
    if (c >= q.channels)
        return;
    for (int64_t t = first_token<WAVE>(); t < q.tokens; t += int64_t(gridDim.x) * blockDim.y) {
        float sum[VEC] = {};
        for (int j0 = 0; j0 < q.top; j0 += N) {
            Elements<E, VEC> v[N];
            float w[N];
            int64_t at[N];
            pairs_of(q, t, j0, at, w);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at[i] >= 0)
                    v[i].template load<ONCE>(static_cast<const char*>(q.rows) + (at[i] * q.rows_row + c) * E::size);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at[i] >= 0) {
                    float f[VEC];
                    v[i].get(f);
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        sum[k] = __builtin_fmaf(w[i], f[k], sum[k]);
                }
        }
        Elements<E, VEC> o;
        o.set(sum);
        o.template store<PAST>(static_cast<char*>(q.out) + (t * q.out_row + c) * E::size);
    }
}

// The sum over the x lanes of a token (x a power of two up to 64), in every one of them.
__device__ __forceinline__ float sum_of_lanes(float v, int x)
{
    for (int step = 1; step < x; step *= 2)
        v += __shfl_xor(v, step);
    return v;
}

__device__ __forceinline__ void store_weight(void* weights, int type, int64_t p, float v)
{
    if (type == LOGITS_F32)
        static_cast<float*>(weights)[p] = v;
    else
        static_cast<uint16_t*>(weights)[p] = uint16_t(type == LOGITS_F16 ? F16::pack<1>({v}) : BF16::pack<1>({v}));
}

// The lanes of a token go over its channels together, so that its rows are read and written in long pieces (a
// wave a token, 1 KiB of each row at a time, took 241 us for 16384 tokens of 8 rows of 2048 bfloat16, and left most of
// the GPU idle with few tokens; as it is, 8192 tokens of 4 rows of 4096, 604 MB, take 116 us, 5.2 TB/s, as reads and writes mix; 128 lanes take 247 us for 8192 of 8 rows of 4096 against 230).  N as above: with 8 for every call,
// 16384 tokens of 2 rows of 2048 took 105 us against 60; with 4 for 8 rows of 4096, 240 against 230.
template <class E, int VEC, int N, bool WAVE, bool ONCE, bool PAST>
__global__ __launch_bounds__(256) void experts_combine_backward_kernel(ExpertsRows q)
{
    __shared__ float part[N][4];  // of each wave
    const int x = blockDim.x, y = blockDim.y, tx = threadIdx.x;
    const int ty = WAVE ? __builtin_amdgcn_readfirstlane(int(threadIdx.y)) : int(threadIdx.y);
    const int wave = (ty * x + tx) >> 6, waves = x > 64 ? x / 64 : 1;  // (of a token)
    for (int64_t t0 = int64_t(blockIdx.x) * y; t0 < q.tokens; t0 += int64_t(gridDim.x) * y) {
        const int64_t t = t0 + ty;
        const bool live = t < q.tokens;
        for (int j0 = 0; j0 < q.top; j0 += N) {
            float dot[N] = {}, w[N];
            int64_t at[N];
            pairs_of(q, live ? t : q.tokens - 1, j0, at, w);
            for (int64_t c = int64_t(tx) * VEC; live && c < q.channels; c += int64_t(x) * VEC) {
                Elements<E, VEC> d, v[N];
                d.template load<ONCE>(static_cast<const char*>(q.x) + (t * q.x_row + c) * E::size);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (at[i] >= 0)
                        v[i].template load<ONCE>(static_cast<const char*>(q.rows) + (at[i] * q.rows_row + c) * E::size);
                float df[VEC];
                d.get(df);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (at[i] >= 0) {
                        float f[VEC], g[VEC];
                        v[i].get(f);
#pragma unroll
                        for (int k = 0; k < VEC; ++k) {
                            dot[i] = __builtin_fmaf(f[k], df[k], dot[i]);
                            g[k] = w[i] * df[k];
                        }
                        v[i].set(g);
                        v[i].template store<PAST>(static_cast<char*>(q.rows_out) + (at[i] * q.rows_out_row + c) * E::size);
                    }
            }
            const int lanes = x < 64 ? x : 64;
#pragma unroll
            for (int i = 0; i < N; ++i)
                dot[i] = sum_of_lanes(dot[i], lanes);
            if (waves > 1) {
                if ((tx & 63) == 0) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        part[i][wave] = dot[i];
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    dot[i] = 0.0f;
                    for (int k = 0; k < waves; ++k)
                        dot[i] += part[i][ty * waves + k];
                }
                __syncthreads();
            }
            if (live && tx == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (j0 + i < q.top)
                        store_weight(q.dweights, q.weight_type, t * q.top + j0 + i, at[i] >= 0 ? dot[i] : 0.0f);
            }
        }
    }
}

// 16 bytes a lane where every row is aligned to that, else an element.
static bool wide_rows(const ExpertsRows& q, int size)
{
    const int64_t vec = 16 / size;
    const uintptr_t p = reinterpret_cast<uintptr_t>(q.x) | reinterpret_cast<uintptr_t>(q.rows) |
                        reinterpret_cast<uintptr_t>(q.rows_out) | reinterpret_cast<uintptr_t>(q.out);
    return q.channels % vec == 0 && p % 16 == 0 && q.x_row % vec == 0 && q.rows_row % vec == 0 && q.out_row % vec == 0 &&
           q.rows_out_row % vec == 0;
}

// How many rows a call moves decides how they pass the caches.
//   once: rows that are read once and are too many to be in the second-level caches still are loaded past them: 8192 tokens of 8
//     rows of 4096 bfloat16 are combined in 100 us against 120.  Rows shorter than 1 KiB gain nothing, and few rows, that the
//     experts' product has just written, lose (32 tokens' gradients 16.6 us against 11.9).
//   past: where the rows fill the memory-side cache, 256 MiB, a call writes past the caches, too.  Gather, and gather and
//     a product of all rows that follows it: 8192 tokens of 8 rows of 4096 bfloat16 101 and 268 us against 113 and 297, of 4
//     rows 55 and 144 against 68 and 156; the gradient 119 and 196 against 127 and 206.  Fewer rows the product finds in
//     that cache: 2560 tokens of 8 rows of 2048, 17 and 53 against 17 and 50, the gradient 41 and 78 against 38 and 68.
//     Sums, and sums and an addition to them: 8192 tokens of 8 rows of 4096 104 and 141 against 108 and 145; 4096 of 8 rows
//     of 2048, 26 and 37 against 28 and 36.
constexpr int64_t EX_ONCE_ROW = 1024, EX_ONCE_ALL = 64 << 20, EX_PAST_ALL = 256 << 20;
struct Caching {
    bool wave, once, past;  // a wave has one token; past: also once
};

template <class E, int VEC>
static void gather_of(const ExpertsRows& q, const RowGrid& g, const Caching& how, hipStream_t stream)
{
    if constexpr (VEC > 1)
        if (how.past) {
            experts_gather_kernel<E, VEC, true, true><<<g.grid, g.block, 0, stream>>>(q);
            return;
        }
    if (how.wave)
        experts_gather_kernel<E, VEC, true, false><<<g.grid, g.block, 0, stream>>>(q);
    else
        experts_gather_kernel<E, VEC, false, false><<<g.grid, g.block, 0, stream>>>(q);
}

template <class E, int VEC, int N>
static void combine_of(const ExpertsRows& q, const RowGrid& g, const Caching& how, hipStream_t stream)
{
    if constexpr (VEC > 1)
        if (how.once) {
            if (how.past)
                experts_combine_kernel<E, VEC, N, true, true, true><<<g.grid, g.block, 0, stream>>>(q);
            else
                experts_combine_kernel<E, VEC, N, true, true, false><<<g.grid, g.block, 0, stream>>>(q);
            return;
        }
    if (how.wave)
        experts_combine_kernel<E, VEC, N, true, false, false><<<g.grid, g.block, 0, stream>>>(q);
    else
        experts_combine_kernel<E, VEC, N, false, false, false><<<g.grid, g.block, 0, stream>>>(q);
}

template <class E, int VEC, int N>
static void combine_backward_of(const ExpertsRows& q, const RowGrid& g, const Caching& how, hipStream_t stream)
{
    const dim3 grid(g.grid.x);  // a block's lanes go over all channels
    if constexpr (VEC > 1)
        if (how.once) {
            if (how.past)
                experts_combine_backward_kernel<E, VEC, N, true, true, true><<<grid, g.block, 0, stream>>>(q);
            else
                experts_combine_backward_kernel<E, VEC, N, true, true, false><<<grid, g.block, 0, stream>>>(q);
            return;
        }
    if (how.wave)
        experts_combine_backward_kernel<E, VEC, N, true, false, false><<<grid, g.block, 0, stream>>>(q);
    else
        experts_combine_backward_kernel<E, VEC, N, false, false, false><<<grid, g.block, 0, stream>>>(q);
}

template <class E, int VEC>
static hipError_t rows_of(const ExpertsRows& q, ExpertsMove move, hipStream_t stream)
{
    const int64_t parts = (q.channels + VEC - 1) / VEC;
    const RowGrid g = row_grid(q.tokens, parts, 256);
    const int64_t row = q.channels * E::size, all = q.tokens * q.top * row;
    const bool wide = VEC > 1 && row >= EX_ONCE_ROW;
    const Caching how{g.block.x >= 64, wide && all >= EX_ONCE_ALL, wide && all >= EX_PAST_ALL};
    if (move == EXPERTS_GATHER)
        gather_of<E, VEC>(q, g, how, stream);
    else if (move == EXPERTS_COMBINE && q.top <= 2)
        combine_of<E, VEC, 2>(q, g, how, stream);
    else if (move == EXPERTS_COMBINE && q.top <= 4)
        combine_of<E, VEC, 4>(q, g, how, stream);
    else if (move == EXPERTS_COMBINE)
        combine_of<E, VEC, EX_FLIGHT>(q, g, how, stream);
    else if (q.top <= 2)
        combine_backward_of<E, VEC, 2>(q, g, how, stream);
    else if (q.top <= 4)
        combine_backward_of<E, VEC, 4>(q, g, how, stream);
    else
        combine_backward_of<E, VEC, EX_FLIGHT>(q, g, how, stream);
    return hipGetLastError();
}

template <class E>
static hipError_t rows_of_type(const ExpertsRows& q, ExpertsMove move, hipStream_t stream)
{
    return wide_rows(q, E::size) ? rows_of<E, 16 / E::size>(q, move, stream) : rows_of<E, 1>(q, move, stream);
}

hipError_t launch_experts_rows(const ExpertsRows& q, ExpertsMove move, int type, hipStream_t stream)
{
    if (q.tokens == 0 || (q.channels == 0 && move != EXPERTS_COMBINE_BACKWARD) || (q.top == 0 && move != EXPERTS_COMBINE))
        return hipSuccess;
    if (type == LOGITS_F32)
        return rows_of_type<F32>(q, move, stream);
    return type == LOGITS_F16 ? rows_of_type<F16>(q, move, stream) : rows_of_type<BF16>(q, move, stream);
}

}  // namespace ls
