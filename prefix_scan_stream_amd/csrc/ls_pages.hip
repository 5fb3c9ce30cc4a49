// ls_pages.hip -- the books of a paged cache: pages for new tokens, cache slots of
// this step's tokens, pages of finished requests back on the free list (gfx950).
//
// All three are one shape: request r makes c[r] outputs (pages or tokens), and output
// q belongs to the request whose run [U[r], U[r] + c[r]) of the exclusive prefix sum U
// contains it.  One launch does the prefix sum and the outputs: every block scans the
// requests' counts itself, PG_CHUNK requests at a time (32 KiB of lengths for 4096
// requests, from L2), keeps the chunk's prefix sums in LDS, and writes its share of the
// chunk's outputs, consecutive ones per turn.  Nothing is handed from block to
// block, so there is no workspace, no wait and no second launch; the price is that each
// block reads all counts, a few percent of the outputs' bytes at the sizes of a step.
// That is made for batches: up to 4096 requests 4-5 us for a step of a token each, then about
// 2.5 us more for each 4096 in the grid's every block (16384: 13 us; 65536: 37-57; 2^20: 0.54-0.84 ms).
// With few outputs bound by the latency of one scan (3.6-4.5 us against 2 of an empty kernel; a number of
// requests that is no multiple of eight loads its last ones one by one, 1 us).  With many (prompts, an
// emptied cache) 2-3.5 TB/s: each lane waits for an output's store before it loads the next.
#include "ls_wave64.hpp"
#include "ls_internal.hpp"

namespace ls {

// Measured for the outputs of 4096 prompts (2.7 M pages) / 2.6 M slots / 4.1 M released
// pages: 512 blocks of 512 threads 11.1 / 12.2 / 13.5 us; 256 blocks 12.4 / 14.8 / 18.8 (too
// few waves), 768 blocks 13.2 / 14.0 / 12.4 and 1024 13.7 / 13.2 / 15.9 (the registers, 88 / 90 / 74, leave a CU
// two blocks, of the last operator three, so later ones start late); 256 blocks of 1024 threads 10.0 / 13.1 / 13.1.  No
// grid is the best for all three; this one is kept for all, as the slots of every step have their best here.
constexpr int PG_BLOCK = 512;
constexpr int PG_WAVES = PG_BLOCK / 64;
constexpr int PG_CHUNK = 4096;                  // requests per scan
constexpr int PG_ITEMS = PG_CHUNK / PG_BLOCK;   // requests per thread
constexpr int PG_OUT = 4;                       // outputs per thread and turn, when there are many
constexpr int PG_MAX_GRID = 512;

// Division of 0 <= n < 2^31 by d >= 1: q = n * m >> (31 + s), s = ceil(log2 d),
// m = ceil(2^(31+s) / d) < 2^32.  m d exceeds 2^(31+s) by less than 2^s, so the error
// n (m d - 2^(31+s)) / (d 2^(31+s)) stays below 1/d for n < 2^31: exact.
struct PageDiv {
    uint32_t d, m, s;
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return uint32_t((uint64_t(n) * m) >> (31 + s)); }
    __device__ __forceinline__ uint32_t pages(uint32_t n) const { return n == 0 ? 0u : div(n - 1) + 1u; }
};

static PageDiv make_div(int64_t d)
{
    PageDiv p;
    p.d = uint32_t(d);
    p.s = 0;
    while ((uint64_t(1) << p.s) < uint64_t(d))
        ++p.s;
    const unsigned __int128 top = static_cast<unsigned __int128>(1) << (31 + p.s);
    p.m = uint32_t((top + uint64_t(d) - 1) / uint64_t(d));
    return p;
}

// Entries r .. r+7 of a vector of lengths, negative ones and those past the end as 0.
__device__ __forceinline__ void load_lens(const int32_t* p, int64_t r, int64_t n, uint32_t (&v)[PG_ITEMS])
{
    typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));
    static_assert(PG_ITEMS % 4 == 0, "128-bit loads");
    if (r + PG_ITEMS <= n) {
#pragma unroll
        for (int j = 0; j < PG_ITEMS; j += 4) {
            const i32x4 a = *reinterpret_cast<const i32x4*>(p + r + j);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[j + k] = uint32_t(a[k] < 0 ? 0 : a[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < PG_ITEMS; ++k) {
            const int32_t l = r + k < n ? p[r + k] : 0;
            v[k] = uint32_t(l < 0 ? 0 : l);
        }
    }
}

// Each operator below gives, for the requests r .. r+7 of a thread, what they make
// (`c`), what their outputs need to know of them (`info`, kept in LDS) and whether they
// can be served at all; writes output q, the i-th of request r; and writes the
// per-request results.

struct AppendOp {
    const int32_t *lens, *new_lens;
    int32_t* tables;
    const int32_t* free_pages;
    const int64_t* free_count;
    int64_t* count_out;
    uint8_t* granted;
    int64_t columns, stride, capacity;
    PageDiv page;
    static constexpr bool has_limit = true;

    __device__ __forceinline__ int64_t limit() const
    {
        const int64_t c = *free_count;
        return c < 0 ? 0 : (c > capacity ? capacity : c);
    }
    // pages asked for, pages held, and whether the table row has the columns
    __device__ __forceinline__ void count(int64_t r, int64_t n, uint32_t (&c)[PG_ITEMS], uint32_t (&info)[PG_ITEMS],
                                          bool (&fits)[PG_ITEMS]) const
    {
        uint32_t len[PG_ITEMS], add[PG_ITEMS];
        load_lens(lens, r, n, len);
        load_lens(new_lens, r, n, add);
#pragma unroll
        for (int k = 0; k < PG_ITEMS; ++k) {
            const uint32_t sum = len[k] + add[k];
            const uint32_t have = page.pages(len[k]), want = page.pages(sum & 0x7fffffffu);
            fits[k] = sum <= 0x7fffffffu && int64_t(want) <= columns;
            c[k] = fits[k] ? want - have : 0u;
            info[k] = have;
        }
    }
    __device__ __forceinline__ void emit(int64_t q, int64_t r, uint32_t i, uint32_t have, int64_t lim) const
    {
        tables[r * stride + have + i] = free_pages[lim - 1 - q];
    }
    __device__ __forceinline__ void request(int64_t r, uint32_t c, bool fits, int64_t upto, int64_t lim) const
    {
        granted[r] = fits && (c == 0 || upto <= lim) ? 1 : 0;
    }
    __device__ __forceinline__ void finish(int64_t taken, int64_t lim) const { *count_out = lim - taken; }
};

struct SlotsOp {
    const int32_t *lens, *new_lens, *tables;
    int64_t* slots;
    int32_t *positions, *requests;
    int64_t* offsets;
    int64_t columns, stride, n;
    PageDiv page;
    static constexpr bool has_limit = false;

    __device__ __forceinline__ int64_t limit() const { return n; }
    __device__ __forceinline__ void count(int64_t r, int64_t n, uint32_t (&c)[PG_ITEMS], uint32_t (&info)[PG_ITEMS],
                                          bool (&)[PG_ITEMS]) const
    {
        load_lens(new_lens, r, n, c);
        load_lens(lens, r, n, info);
    }
    __device__ __forceinline__ void emit(int64_t q, int64_t r, uint32_t i, uint32_t len, int64_t) const
    {
        const uint32_t at = len + i;
        int64_t slot = -1;
        if (at <= 0x7fffffffu) {
            const uint32_t col = page.div(at);
            const int32_t held = int64_t(col) < columns ? tables[r * stride + col] : -1;
            if (held >= 0)
                slot = int64_t(held) * page.d + (at - col * page.d);
        }
        slots[q] = slot;
        positions[q] = int32_t(at);
        requests[q] = int32_t(r);
    }
    __device__ __forceinline__ void request(int64_t r, uint32_t, bool, int64_t upto, int64_t) const
    {
        offsets[r + 1] = upto;
        if (r == 0)
            offsets[0] = 0;
    }
    __device__ __forceinline__ void pad(int64_t q) const
    {
        slots[q] = -1;
        positions[q] = 0;
        requests[q] = -1;
    }
};

struct ReleaseOp {
    const int32_t* lens;
    const uint8_t* finished;
    const int32_t* tables;
    int32_t* free_pages;
    const int64_t* free_count;
    int64_t* count_out;
    int64_t columns, stride, capacity;
    PageDiv page;
    static constexpr bool has_limit = false;

    // Where the pages go; those past the end of the free list are counted but not written.
    __device__ __forceinline__ int64_t limit() const
    {
        const int64_t c = *free_count;
        return c < 0 ? 0 : c;
    }
    __device__ __forceinline__ void count(int64_t r, int64_t n, uint32_t (&c)[PG_ITEMS], uint32_t (&info)[PG_ITEMS],
                                          bool (&)[PG_ITEMS]) const
    {
        uint32_t len[PG_ITEMS];
        load_lens(lens, r, n, len);
#pragma unroll
        for (int k = 0; k < PG_ITEMS; ++k) {
            const uint32_t held = page.pages(len[k]);
            c[k] = r + k >= n || finished[r + k] == 0 ? 0u : int64_t(held) < columns ? held : uint32_t(columns);
            info[k] = 0;
        }
    }
    __device__ __forceinline__ void emit(int64_t q, int64_t r, uint32_t i, uint32_t, int64_t base) const
    {
        if (q < capacity - base)
            free_pages[base + q] = tables[r * stride + i];
    }
    __device__ __forceinline__ void request(int64_t, uint32_t, bool, int64_t, int64_t) const {}
    __device__ __forceinline__ void finish(int64_t taken, int64_t base) const { *count_out = base + taken; }
};

// LDS place of request i's prefix: one entry of padding after eight spreads a wave's
// writes (8 entries per lane) over all banks.
__device__ __forceinline__ int place(int i) { return i + (i >> 3); }

// The last of n requests that starts at or before output `at`, by one wave: each step
// cuts the range into 64 parts, a lane each (two steps for 4096 requests).  n >= 1.
__device__ __forceinline__ int wave_find(const uint64_t* excl, int n, uint64_t at)
{
    const int lane = lane_id();
    int lo = 0;
    int step = PG_CHUNK / 64;
    static_assert(PG_CHUNK == 64 * 64, "two steps");
    for (int k = 0; k < 2; ++k) {
        const int i = lo + lane * step;
        const uint64_t in = __ballot(i < n && excl[place(i < n ? i : 0)] <= at);
        lo += (63 - __builtin_clzll(in | 1u)) * step;
        step = 1;
    }
    return lo;
}

// Outputs [base, end) of the chunk's n requests from r0, U consecutive ones per lane and
// turn; this block's first turn is `first_turn`.  A wave's share of a turn is
// consecutive, and the requests it spans are found once.
template <int U, class Op>
__device__ __forceinline__ void write_outputs(const Op& op, const uint64_t* excl, const uint32_t* info, int n,
                                              int64_t r0, int64_t base, int64_t end, int64_t first_turn,
                                              int64_t turns, int64_t lim)
{
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    for (int64_t q0 = base + (first_turn * PG_WAVES + wave) * (64 * U); q0 < end; q0 += turns * (PG_BLOCK * U)) {
        const int64_t q1 = q0 + 64 * U < end ? q0 + 64 * U : end;
        const int first = wave_find(excl, n, uint64_t(q0 - base));
        const int last = wave_find(excl, n, uint64_t(q1 - 1 - base));
        int lo[U], hi[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            lo[k] = first;
            hi[k] = last + 1;
        }
        // the last request that starts at or before the output (empty ones share their start with the next)
        for (int span = last - first; span > 0; span >>= 1) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int mid = (lo[k] + hi[k]) >> 1;
                const bool right = excl[place(mid)] <= uint64_t(q0 + k * 64 + lane - base);
                lo[k] = right ? mid : lo[k];
                hi[k] = right ? hi[k] : mid;
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t q = q0 + k * 64 + lane;
            if (q < q1)
                op.emit(q, r0 + lo[k], uint32_t(uint64_t(q - base) - excl[place(lo[k])]), info[lo[k]], lim);
        }
    }
}

template <class Op>
__global__ __launch_bounds__(PG_BLOCK) void expand_kernel(Op op, int64_t requests)
{
    __shared__ uint64_t s_excl[PG_CHUNK + PG_CHUNK / 8];  // outputs of the chunk before each of its requests
    __shared__ uint32_t s_info[PG_CHUNK];
    __shared__ uint64_t s_wave[PG_WAVES];
    __shared__ int64_t s_taken;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t grid = gridDim.x, block = blockIdx.x;
    const int64_t lim = op.limit();
    int64_t base = 0;      // outputs of earlier chunks
    int64_t taken = -1;    // AppendOp: the pages handed out, once the list has run out
    int64_t chunk = 0;

    for (int64_t r0 = 0; r0 < requests; r0 += PG_CHUNK, ++chunk) {
        const int n = requests - r0 < PG_CHUNK ? int(requests - r0) : PG_CHUNK;
        const int i0 = tid * PG_ITEMS;
        uint32_t c[PG_ITEMS] = {}, info[PG_ITEMS] = {};
        bool fits[PG_ITEMS] = {};
        if (i0 < n)
            op.count(r0 + i0, requests, c, info, fits);
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < PG_ITEMS; ++k)
            sum += c[k];
        const uint64_t incl = wave_inclusive_sum64(sum);
        if (lane == 63)
            s_wave[wave] = incl;
        if (tid == 0)
            s_taken = -1;
        __syncthreads();
        uint64_t excl = incl - sum, total = 0;
#pragma unroll
        for (int w = 0; w < PG_WAVES; ++w) {
            const uint64_t v = s_wave[w];
            excl += w < wave ? v : 0u;
            total += v;
        }
        const bool mine = block == chunk % grid;  // the block that writes this chunk's per-request results
        if (i0 < n) {
#pragma unroll
            for (int k = 0; k < PG_ITEMS; ++k) {
                const int64_t r = r0 + i0 + k;
                s_excl[place(i0 + k)] = excl;
                s_info[i0 + k] = info[k];
                const int64_t before = base + int64_t(excl);
                excl += c[k];
                const int64_t upto = base + int64_t(excl);
                if (mine && r < requests)
                    op.request(r, c[k], fits[k], upto, lim);
                if constexpr (Op::has_limit) {
                    // the first request whose pages the list does not hold: nothing is handed out from here on
                    if (before <= lim && upto > lim)
                        s_taken = before;
                }
            }
        }
        __syncthreads();
        int64_t end = base + int64_t(total);
        if constexpr (Op::has_limit) {
            if (taken < 0)
                taken = s_taken;
            if (taken >= 0 && end > taken)
                end = taken;
        } else if constexpr (__is_same(Op, SlotsOp)) {
            if (end > op.n)
                end = op.n;
        }
        // Turns of outputs are dealt to the blocks in turn, from another block in each chunk.  One output per
        // thread when that covers them (a shorter chain: 3.6 us against 4.8 for 256 tokens), else PG_OUT.
        const int64_t at = (block - chunk % grid + grid) % grid;
        if (end - base <= grid * PG_BLOCK)
            write_outputs<1>(op, s_excl, s_info, n, r0, base, end, at, grid, lim);
        else
            write_outputs<PG_OUT>(op, s_excl, s_info, n, r0, base, end, at, grid, lim);
        base += int64_t(total);
        __syncthreads();  // s_excl, s_info, s_wave and s_taken are rewritten by the next chunk
    }
    if constexpr (__is_same(Op, SlotsOp)) {
        for (int64_t q = base + block * PG_BLOCK + tid; q < op.n; q += grid * PG_BLOCK)
            op.pad(q);
        if (requests == 0 && block == 0 && tid == 0)
            op.offsets[0] = 0;
    } else {
        if (block == 0 && tid == 0)
            op.finish(taken >= 0 ? taken : base, lim);
    }
}

// Blocks for up to `outputs` outputs.
static unsigned expand_grid(int64_t outputs)
{
    const int64_t tiles = (outputs + PG_BLOCK - 1) / PG_BLOCK;
    return unsigned(tiles < 1 ? 1 : tiles > PG_MAX_GRID ? PG_MAX_GRID : tiles);
}

hipError_t launch_pages_append(const int32_t* lens, const int32_t* new_lens, int64_t requests, int32_t* tables,
                               int64_t columns, int64_t stride, const int32_t* free_pages, int64_t capacity,
                               const int64_t* free_count, int64_t page_size, int64_t* count_out, uint8_t* granted,
                               hipStream_t stream)
{
    const AppendOp op{lens, new_lens, tables, free_pages, free_count, count_out, granted, columns, stride, capacity,
                      make_div(page_size)};
    const int64_t cells = columns > 0 && requests > capacity / columns ? capacity : requests * columns;
    expand_kernel<AppendOp><<<expand_grid(cells), PG_BLOCK, 0, stream>>>(op, requests);
    return hipGetLastError();
}

hipError_t launch_slot_map(const int32_t* lens, const int32_t* new_lens, int64_t requests, const int32_t* tables,
                           int64_t columns, int64_t stride, int64_t page_size, int64_t n, int64_t* slots,
                           int32_t* positions, int32_t* request_ids, int64_t* offsets, hipStream_t stream)
{
    const SlotsOp op{lens, new_lens, tables, slots, positions, request_ids, offsets, columns, stride, n,
                     make_div(page_size)};
    expand_kernel<SlotsOp><<<expand_grid(n), PG_BLOCK, 0, stream>>>(op, requests);
    return hipGetLastError();
}

hipError_t launch_pages_release(const int32_t* lens, const uint8_t* finished, int64_t requests,
                                const int32_t* tables, int64_t columns, int64_t stride, int32_t* free_pages,
                                int64_t capacity, const int64_t* free_count, int64_t page_size, int64_t* count_out,
                                hipStream_t stream)
{
    const ReleaseOp op{lens, finished, tables, free_pages, free_count, count_out, columns, stride, capacity,
                       make_div(page_size)};
    const int64_t cells = columns > 0 && requests > capacity / columns ? capacity : requests * columns;
    expand_kernel<ReleaseOp><<<expand_grid(cells), PG_BLOCK, 0, stream>>>(op, requests);
    return hipGetLastError();
}

}  // namespace ls
