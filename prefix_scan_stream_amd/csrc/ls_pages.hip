// ls_pages.hip -- the books of a paged cache: pages for new tokens, cache slots of
// this step's tokens, pages of finished requests back on the free list (gfx950).
//
// All three are one shape: request r makes c[r] outputs (pages or tokens), and output
// q belongs to the request whose run [U[r], U[r] + c[r]) of the exclusive prefix sum U
// contains it.  One launch does the prefix sum and the outputs: every block scans the
// requests' counts itself, PG_CHUNK requests at a time (32 KiB of lengths for 4096
// requests, from L2), keeps the chunk's prefix sums in LDS, and writes its share of the
// chunk's outputs, PG_TILE consecutive ones per turn.  Nothing is handed from block to
// block, so there is no workspace, no wait and no second launch; the price is that each
// block reads all counts, a few percent of the outputs' bytes at the sizes of a step.
// Bound by the bytes of the outputs when there are many (prompts, an emptied cache), by
// the latency of one scan (two dependent loads and three barriers) when there are few.
#include "ls_device.hpp"
#include "ls_internal.hpp"

namespace ls {

constexpr int PG_BLOCK = 512;
constexpr int PG_WAVES = PG_BLOCK / 64;
constexpr int PG_ITEMS = 8;                     // requests per thread
constexpr int PG_CHUNK = PG_BLOCK * PG_ITEMS;   // requests per scan
constexpr int PG_OUT = 4;                       // outputs per thread and turn
constexpr int PG_TILE = PG_BLOCK * PG_OUT;
constexpr int PG_MAX_GRID = 1024;               // four blocks per CU

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

__device__ __forceinline__ int32_t at_least_0(int32_t v) { return v < 0 ? 0 : v; }

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
    // Pages request r asks for; `fits`: its table row has the columns.
    __device__ __forceinline__ uint32_t count(int64_t r, bool& fits) const
    {
        const uint32_t len = uint32_t(at_least_0(lens[r])), sum = len + uint32_t(at_least_0(new_lens[r]));
        const uint32_t have = page.pages(len), want = page.pages(sum & 0x7fffffffu);
        fits = sum <= 0x7fffffffu && int64_t(want) <= columns;
        return fits ? want - have : 0u;
    }
    __device__ __forceinline__ void emit(int64_t q, int64_t r, uint32_t i, int64_t lim) const
    {
        const uint32_t have = page.pages(uint32_t(at_least_0(lens[r])));
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
    __device__ __forceinline__ uint32_t count(int64_t r, bool& fits) const
    {
        fits = true;
        return uint32_t(at_least_0(new_lens[r]));
    }
    __device__ __forceinline__ void emit(int64_t q, int64_t r, uint32_t i, int64_t) const
    {
        const uint32_t at = uint32_t(at_least_0(lens[r])) + i;
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

    // Outputs past the end of the free list are counted but not written.
    __device__ __forceinline__ int64_t limit() const { return capacity; }
    __device__ __forceinline__ uint32_t count(int64_t r, bool& fits) const
    {
        fits = true;
        if (finished[r] == 0)
            return 0u;
        const uint32_t held = page.pages(uint32_t(at_least_0(lens[r])));
        return int64_t(held) < columns ? held : uint32_t(columns);
    }
    __device__ __forceinline__ void emit(int64_t q, int64_t r, uint32_t i, int64_t) const
    {
        const int64_t to = at_least_count() + q;
        if (to < capacity)
            free_pages[to] = tables[r * stride + i];
    }
    __device__ __forceinline__ int64_t at_least_count() const
    {
        const int64_t c = *free_count;
        return c < 0 ? 0 : c;
    }
    __device__ __forceinline__ void request(int64_t, uint32_t, bool, int64_t, int64_t) const {}
    __device__ __forceinline__ void finish(int64_t taken, int64_t) const { *count_out = at_least_count() + taken; }
};

template <class Op>
__global__ __launch_bounds__(PG_BLOCK) void expand_kernel(Op op, int64_t requests)
{
    __shared__ uint64_t s_excl[PG_CHUNK];  // outputs of the chunk before each of its requests
    __shared__ uint64_t s_wave[PG_WAVES];
    __shared__ int64_t s_taken;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t grid = gridDim.x, block = blockIdx.x;
    const int64_t lim = op.limit();
    int64_t base = 0;      // outputs of earlier chunks
    int64_t taken = -1;    // AppendOp: the pages handed out, once the list has run out
    int64_t chunk = 0;

    for (int64_t r0 = 0; r0 < requests; r0 += PG_CHUNK, ++chunk) {
        uint32_t c[PG_ITEMS];
        bool fits[PG_ITEMS];
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < PG_ITEMS; ++k) {
            const int64_t r = r0 + tid * PG_ITEMS + k;
            fits[k] = false;
            c[k] = r < requests ? op.count(r, fits[k]) : 0u;
            sum += c[k];
        }
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
#pragma unroll
        for (int k = 0; k < PG_ITEMS; ++k) {
            const int64_t r = r0 + tid * PG_ITEMS + k;
            s_excl[tid * PG_ITEMS + k] = excl;
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
        __syncthreads();
        int64_t end = base + int64_t(total);
        if constexpr (Op::has_limit) {
            if (taken < 0)
                taken = s_taken;
            if (taken >= 0 && end > taken)
                end = taken;
        } else {
            if (end > lim)
                end = lim;
        }
        // turns of PG_TILE outputs, dealt to the blocks in turn, from another block in each chunk
        for (int64_t q0 = base + (block - chunk % grid + grid) % grid * PG_TILE; q0 < end; q0 += grid * PG_TILE) {
#pragma unroll
            for (int k = 0; k < PG_OUT; ++k) {
                const int64_t q = q0 + k * PG_BLOCK + tid;
                if (q < end) {
                    const uint64_t at = uint64_t(q - base);
                    // the last request that starts at or before the output (empty ones share their start with the next)
                    int lo = 0, hi = PG_CHUNK;
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) >> 1;
                        if (s_excl[mid] <= at)
                            lo = mid;
                        else
                            hi = mid;
                    }
                    op.emit(q, r0 + lo, uint32_t(at - s_excl[lo]), lim);
                }
            }
        }
        base += int64_t(total);
        __syncthreads();  // s_excl, s_wave and s_taken are rewritten by the next chunk
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
    const int64_t tiles = (outputs + PG_TILE - 1) / PG_TILE;
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
