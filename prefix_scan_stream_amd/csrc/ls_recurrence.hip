// ls_recurrence.hip -- the gated linear recurrence h_t = a_t h_{t-1} + b_t over sequences,
// channel by channel, and its gradients (gfx950).
//
// A token is the affine map h -> a h + b of each channel, and maps compose:
//     (a1, b1) then (a2, b2)  =  (a2 a1, a2 b1 + b2),
// so the recurrence is a scan.  Channels lie beside each other in memory and are independent: a
// lane owns CPL neighbouring channels (4 bytes of a row), a wave some consecutive tokens of its
// 64 CPL channels, and a block's waves lie one behind the other in time.  Per tile (64 or 128 tokens):
//   1. every wave loads its rows (each load 256 consecutive bytes), makes a and b of them in
//      float32 and composes its map;
//   2. the waves' maps meet in LDS; every wave applies those in front of it to the value in
//      front of the tile and goes through its rows once more, from registers, writing h.
// So every byte is read once and written once.  The value in front of a tile comes from the
// block's last tile, where a block walks its sequence and the next tile's rows are on their
// way meanwhile, or through the workspace, where each tile is a block ("tiles as blocks").
//
// Backward, with mu_t = a_t lambda_t the gradient that h_{t-1} receives:
//     lambda_t = dh_t + mu_{t+1},   mu_t = a_t mu_{t+1} + a_t dh_t,
// the same maps' factors from the last token to the first.  A tile needs h again: it is
// made from x and gate, from the carries that the forward pass kept of every RC_PERIOD-th
// row, in 32 bits; the output h would cost as many bytes and is rounded.
//
// What bounds it: memory, three elements a token and channel forward and five backward, where blocks walk (64 sequences
// of 512 tokens of 2048 bfloat16 channels: 74-76 us forward, 5.4 TB/s, 132-141 backward, 4.8-5.1); and where tiles are
// blocks also the wait for the value in front, which holds a block's registers while nothing of it is
// under way (1 x 65536 x 2048, log: 184-192 and 308 us, 4.3 TB/s both; without the link, so with wrong values, 137 forward).
// Blocks of 8 waves that a CU holds, by their registers: forward with two channels a lane two (90-101 registers for tiles, 112-114
// for blocks that walk), with one three or four (53-60, 76-78); backward with two channels two with a sigmoid (82-86; packed with
// more than four chains 80: three), else three for more than four chains (78-80) and two for fewer (82-85), blocks that walk three or
// four (62-77); with one three (67-75; 16 bits, a sigmoid and packed 83: two).
// Tried for tiles and not kept: blocks that stay and load the next tile while they
// wait (230 to 365 us forward: one block a CU), raw rows kept and the maps made again for three or four blocks a CU (185 to 193:
// registers spill), one 16-bit channel a lane (backward 310, but 323 against 272 for 8 x 4096 x 4096).
//
// A sequence's first row takes its state in place of the carry, by selection and not by a
// factor of 0, so that an infinity in one sequence never reaches the next.
#include "ls_elements.hpp"
#include "ls_internal.hpp"
#include "ls_marks.hpp"

namespace ls {

constexpr int RC_TILE = 128;   // most tokens of a tile
constexpr int RC_PERIOD = 64;  // a carry is kept of every 64th row

// A lane's part of a row: 4 bytes, or one 16-bit element where rows are not aligned to two.
template <class E, int CPL>
constexpr bool whole_word = E::size * CPL == 4;

// once: past the caches
template <class E, int CPL, bool ONCE>
__device__ __forceinline__ uint32_t load_part(__amdgpu_buffer_rsrc_t rs, uint32_t voff)
{
    constexpr int policy = ONCE ? CACHE_NT : 0;
    if constexpr (whole_word<E, CPL>)
        return __builtin_amdgcn_raw_buffer_load_b32(rs, voff, 0, policy);
    else
        return uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rs, voff, 0, policy));
}
template <class E, int CPL>
__device__ __forceinline__ void store_part(__amdgpu_buffer_rsrc_t rs, uint32_t voff, const float (&v)[CPL])
{
    const uint32_t w = E::pack(v);
    if constexpr (whole_word<E, CPL>)
        __builtin_amdgcn_raw_buffer_store_b32(w, rs, voff, 0, STORE_POLICY);
    else
        __builtin_amdgcn_raw_buffer_store_b16(uint16_t(w), rs, voff, 0, STORE_POLICY);
}

// float32 rows of states and carries: the lane's CPL values.
template <int CPL>
__device__ __forceinline__ void load_state(__amdgpu_buffer_rsrc_t rs, uint32_t lane, float (&v)[CPL])
{
#pragma unroll
    for (int c = 0; c < CPL; ++c)
        v[c] = from_bits<float>(__builtin_amdgcn_raw_buffer_load_b32(rs, (lane * CPL + c) * 4, 0, 0));
}
template <int CPL>
__device__ __forceinline__ void store_state(__amdgpu_buffer_rsrc_t rs, uint32_t lane, const float (&v)[CPL])
{
#pragma unroll
    for (int c = 0; c < CPL; ++c)
        __builtin_amdgcn_raw_buffer_store_b32(to_bits(v[c]), rs, (lane * CPL + c) * 4, 0, 0);
}

// A row's window in a matrix: `bytes` of it from the block's first channel, none if it is not there.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_window(const void* p, bool there, uint32_t bytes)
{
    return make_rsrc(p, there ? bytes : 0u);
}

__device__ __forceinline__ uint64_t uniform(uint64_t v)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
    return (uint64_t(hi) << 32) | lo;
}

// Rows one after the other, of which `left` are there.  The compiler must not see through the
// address and the count: it would make all rows' windows at once, more than the scalar registers hold, and
// keep them in vector registers.
struct RowWalk {
    uint64_t at;
    int64_t row;  // bytes
    uint32_t bytes;
    int left;
    __device__ __forceinline__ RowWalk(const char* base, int64_t first, int64_t row_bytes, uint32_t width, int rows_left)
        : at(uniform(reinterpret_cast<uint64_t>(base) + uint64_t(first * row_bytes))), row(row_bytes), bytes(width),
          left(__builtin_amdgcn_readfirstlane(rows_left))
    {
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t window() const
    {
        return row_window(reinterpret_cast<const void*>(at), left > 0, bytes);
    }
    __device__ __forceinline__ void step(int64_t by)
    {
        at += uint64_t(by);
        asm volatile("" : "+s"(at));
    }
    __device__ __forceinline__ void next()
    {
        step(row);
        --left;
        asm volatile("" : "+s"(left));
    }
    // towards the first row: `left` counts what lies in front, this row among it
    __device__ __forceinline__ void previous(bool there)
    {
        step(-row);
        left = __builtin_amdgcn_readfirstlane(there ? 1 : 0);
        asm volatile("" : "+s"(left));
    }
};

// Rows from `row` on, at most `most`.
__device__ __forceinline__ int rows_left(int64_t rows, int64_t row, int most)
{
    const int64_t n = rows - row;
    return n < 0 ? 0 : n < most ? int(n) : most;
}

// ---------------------------------------------------------------- the gate

__device__ __forceinline__ float gate_exp(float g) { return __builtin_amdgcn_exp2f(g * 1.44269504088896340736f); }

// a = 1 / (1 + exp(-g)) and 1 - a, each to its own full precision: the smaller one is made first.
__device__ __forceinline__ void sigmoid_both(float g, float& a, float& rest)
{
    const float e = gate_exp(-__builtin_fabsf(g));
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    a = g >= 0.0f ? big : small;
    rest = g >= 0.0f ? small : big;
}

// a and b = what the token puts in, from the gate and x.
template <int GATING>
__device__ __forceinline__ void token_map(float g, float x, float& a, float& b)
{
    if constexpr (GATING == GATE_SIGMOID) {
        float rest;
        sigmoid_both(g, a, rest);
        b = x * rest;
    } else {
        a = GATING == GATE_LOG ? gate_exp(g) : g;
        b = x;
    }
}

// A decay in one register that gives a and 1 - a to full precision: of a sigmoid the smaller of the two, with a
// sign that says which.
template <int GATING>
struct Decay {
    float u;
    __device__ __forceinline__ void make(float g)
    {
        if constexpr (GATING == GATE_SIGMOID) {
            const float e = gate_exp(-__builtin_fabsf(g));
            const float small = e * __builtin_amdgcn_rcpf(1.0f + e);
            // not 0 for a >= 1/2, as 0 has no side (a gate beyond 87: 1 - a is below float32's range)
            u = g >= 0.0f ? __builtin_fmaxf(small, 1e-38f) : -small;
            u = g != g ? g : u;
        } else {
            u = GATING == GATE_LOG ? gate_exp(g) : g;
        }
    }
    __device__ __forceinline__ void nothing() { u = GATING == GATE_SIGMOID ? 1e-38f : 1.0f; }  // a = 1
    __device__ __forceinline__ float a() const { return GATING != GATE_SIGMOID ? u : u > 0.0f ? 1.0f - u : -u; }
    __device__ __forceinline__ float rest() const { return GATING != GATE_SIGMOID ? 1.0f : u > 0.0f ? u : 1.0f + u; }
};

// ---------------------------------------------------------------- maps

// A composed map (or, behind a sequence's start, h alone: the value itself).
template <int CPL>
struct alignas(8 * CPL) WaveMap {
    float a[CPL], h[CPL];
};

// ---------------------------------------------------------------- tiles as blocks of their own
// Where sequences and channels are too few to fill the GPU with blocks that walk, each tile is a
// block.  The tiles of a chain (a sequence, or the packed rows; and a group of channels) get their
// places in it from a counter, in the order blocks start, and a block only ever waits for lower
// places: for blocks that run or have run, however many of them fit and whatever else the GPU
// does.  (A block that stays to hand values to later places would not do: 256 chains filled the GPU
// with such blocks, and the later ones never started.)
//
// RC_GROUP places are a group, and groups a stretch.  A tile publishes its map, and a group's last tile the map of its
// group.  A tile composes the maps of the tiles in front of it in its group and of the groups in front of its own in
// the stretch (each wave fetches one of either), and applies them to the stretch's front, the value in front of its
// first place.  The stretch's last tile publishes the next one's front.  So a value passes a stretch with one store and one
// load, and a tile reads at most 2 (RC_GROUP - 1) maps.  A tile with a sequence's start (backward: end) does not depend on
// what is in front, and maps say so.
// A stretch is one group: with few chains, whose tiles are all under way at once, the steps from front to front are what
// takes the time, and there it is RC_GROUP groups.  65536 tokens of 128, 256, 384, 512, 768 and 2048 bfloat16 channels (128 a
// chain), forward and backward: one group 49 and 87, 50 and 91, 55 and 98, 58 and 105, 76 and 139, 187 and 345 us; eight 23 and
// 36, 33 and 57, 43 and 77, 57 and 104, 82 and 150, 207 and 376, as a tile waits once more.
// Groups of 4, 16 and 32: 512 channels 83 us forward with 4 against 58; 2048 channels 209 and 388 with 16.
//
// A word that is 0 is empty; values are made not to be 0 (a zero becomes -0, which shows in
// nothing but the sign of a zero).  A group counts the tiles that have read all they need, a stretch its groups, and the last
// one to sign off sets the words back to 0, the counter too; so does the last place with the chain's
// counter.  So a call leaves the workspace as it found it: all 0.

constexpr int RC_GROUP = 8;                   // a wave of a block for each: the link and one for every map
constexpr int RC_GROUP_SHIFT = 3;
constexpr int64_t RC_FEW = 4;                 // chains up to which a stretch is RC_GROUP groups; of more it is one
constexpr int RC_COUNTER = 32;                // 32-bit words from counter to counter: a line each
constexpr uint32_t RC_RESTART = 0x7fc0c0deu;  // for a factor: nothing passes (a NaN that no factor is)

constexpr int chain_levels(int64_t chains) { return chains <= RC_FEW ? 2 : 1; }

struct ChainLayout {
    int64_t chains, most, groups, stretches;  // most places of a chain, its groups and stretches
    size_t counts, maps, fronts, bytes;       // offsets
};
static ChainLayout chain_layout(int64_t chains, int64_t most, int lanes_channels)
{
    ChainLayout l;
    l.chains = chains;
    l.most = most;
    const int stretch_shift = RC_GROUP_SHIFT * chain_levels(chains);
    l.groups = ((most - 1) >> RC_GROUP_SHIFT) + 1;
    l.stretches = ((most - 1) >> stretch_shift) + 1;
    l.counts = sizeof(WsHeader) + size_t(chains) * RC_COUNTER * 4;
    l.maps = l.counts + size_t(chains) * size_t(l.groups) * 2 * RC_COUNTER * 4;
    l.fronts = l.maps + size_t(chains) * size_t(l.groups) * RC_GROUP * size_t(lanes_channels) * 8;
    l.bytes = l.fronts + size_t(chains) * size_t(l.stretches) * size_t(lanes_channels) * 4;
    return l;
}

// What a tile's waves fetch, in LDS: the maps of tiles [0] and of groups [1]; `arrived` starts at 0.
template <int CPL, int LEVELS>
struct ChainParts {
    WaveMap<CPL> maps[LEVELS][RC_GROUP - 1][64];
    float value[CPL][64];  // in front of the tile
    int restart[LEVELS][RC_GROUP - 1], arrived[2];
};

template <int CPL, int LEVELS>
struct Chain {
    WsHeader* header;
    uint32_t* counter;  // places given out
    uint32_t* counts;   // of each group: tiles that have read what they need; at a stretch's first also the groups that have
    uint64_t* maps;     // [place][64 CPL]: factor | value << 32; at a group's last place that of the group
    uint32_t* fronts;   // [stretch][64 CPL]
    int most, places;

    static constexpr int CH = 64 * CPL;
    static constexpr int STRETCH = 1 << (RC_GROUP_SHIFT * LEVELS);  // places

    __device__ __forceinline__ Chain() {}
    __device__ __forceinline__ Chain(void* ws, const ChainLayout& l, int64_t chain)
        : header(static_cast<WsHeader*>(ws)), most(int(l.most)), places(int(l.most))
    {
        char* p = static_cast<char*>(ws);
        counter = reinterpret_cast<uint32_t*>(p + sizeof(WsHeader)) + chain * RC_COUNTER;
        counts = reinterpret_cast<uint32_t*>(p + l.counts) + chain * l.groups * 2 * RC_COUNTER;
        maps = reinterpret_cast<uint64_t*>(p + l.maps) + chain * l.groups * RC_GROUP * CH;
        fronts = reinterpret_cast<uint32_t*>(p + l.fronts) + chain * l.stretches * CH;
    }

    // The block's place, in the order blocks start; `most`: the workspace is not as it should be.
    __device__ __forceinline__ int take_place(uint32_t& shared) const
    {
        if (most > 1 && threadIdx.x == 0) {
            const uint32_t t = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (t == uint32_t(most) - 1)
                __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (t >= uint32_t(most))
                flag_error(header, WS_ERR_BAD_TICKET);
            shared = t;
        }
        __syncthreads();
        if (most == 1)
            return 0;
        const uint32_t t = uint32_t(__builtin_amdgcn_readfirstlane(shared));
        return t < uint32_t(most) ? int(t) : most;
    }

    // Whether a wait is to end without what it waits for, for the whole wave: it has lasted too long, which is then on
    // record; or it has lasted a while and another one is on record (or a chain's waits would end one after the other).
    __device__ __forceinline__ bool gives_up(uint64_t start, int lane) const
    {
        const uint64_t ticks = uint64_t(wall_clock64()) - start;
        const bool late = ticks >= WAIT_LIMIT_TICKS;
        const bool given_up = ticks >= FALLBACK_TICKS &&
                              __hip_atomic_load(&header->error_flags, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != 0;
        if (__builtin_amdgcn_readfirstlane(int(late || given_up)) == 0)
            return false;
        if (late && lane == 0)
            flag_error(header, WS_ERR_WAIT_TIMEOUT);
        return true;
    }

    __device__ __forceinline__ void publish_map(uint64_t* p, int lane, const float (&a)[CPL], const float (&h)[CPL], bool restart) const
    {
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            // (a NaN of a gate's may have these bits)
            const uint32_t own = to_bits(a[c]) == RC_RESTART ? 0x7fc00000u : to_bits(a[c]), f = restart ? RC_RESTART : own;
            const uint64_t w = (uint64_t(to_bits(h[c])) << 32) | f;
            status_store(p + lane * CPL + c, w == 0 ? 0x80000000ull : w);
        }
    }

    // Two 32-bit words at once where a lane has two.
    __device__ __forceinline__ void store_front(int stretch, int lane, const uint32_t (&w)[CPL]) const
    {
        uint32_t* p = fronts + int64_t(stretch) * CH + lane * CPL;
        if constexpr (CPL == 2)
            status_store(reinterpret_cast<uint64_t*>(p), (uint64_t(w[1]) << 32) | w[0]);
        else
            __hip_atomic_store(p, w[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ void publish_front(int stretch, int lane, const float (&h)[CPL]) const
    {
        uint32_t w[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            w[c] = to_bits(h[c]) == 0 ? 0x80000000u : to_bits(h[c]);
        store_front(stretch, lane, w);
    }
    __device__ __forceinline__ void wait_front(int stretch, int lane, float (&h)[CPL]) const
    {
        const uint32_t* p = fronts + int64_t(stretch) * CH + lane * CPL;
        const uint64_t start = wait_start();
        for (;;) {
            bool there;
            if constexpr (CPL == 2) {
                const uint64_t w = status_load(reinterpret_cast<const uint64_t*>(p));
                h[0] = from_bits<float>(uint32_t(w));
                h[1] = from_bits<float>(uint32_t(w >> 32));
                there = uint32_t(w) != 0 && uint32_t(w >> 32) != 0;
            } else {
                const uint32_t w = __hip_atomic_load(const_cast<uint32_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                h[0] = from_bits<float>(w);
                there = w != 0;
            }
            if (__ballot(!there) == 0 || gives_up(start, lane))
                return;
            __builtin_amdgcn_s_sleep(2);
        }
    }

    // A map, once it is there (the whole wave).  Returns whether it restarts.
    __device__ __forceinline__ bool wait_map(const uint64_t* first, int lane, float (&a)[CPL], float (&h)[CPL]) const
    {
        const uint64_t* p = first + lane * CPL;
        uint64_t w[CPL];
        const uint64_t start = wait_start();
        for (;;) {
            bool there = true;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                w[c] = status_load(p + c);
                there &= w[c] != 0;
            }
            if (__ballot(!there) == 0 || gives_up(start, lane))
                break;
            __builtin_amdgcn_s_sleep(2);
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            a[c] = from_bits<float>(uint32_t(w[c]));
            h[c] = from_bits<float>(uint32_t(w[c] >> 32));
        }
        return uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(w[0]))) == RC_RESTART;
    }

    __device__ __forceinline__ static int stretch_of(int place) { return place / STRETCH; }
    // Tiles in front of this one in its group; groups in front of its own in the stretch.
    __device__ __forceinline__ static int tiles_before(int place) { return place % RC_GROUP; }
    __device__ __forceinline__ static int groups_before(int place) { return place % STRETCH / RC_GROUP; }
    __device__ __forceinline__ static bool ends_group(int place) { return place % RC_GROUP == RC_GROUP - 1; }
    __device__ __forceinline__ static bool ends_stretch(int place) { return place % STRETCH == STRETCH - 1; }
    __device__ __forceinline__ uint64_t* map_of(int place) const { return maps + int64_t(place) * CH; }
    __device__ __forceinline__ uint32_t* count_of(int place) const { return counts + int64_t(place / RC_GROUP) * 2 * RC_COUNTER; }

    // A tile's part in the chain.  One wave, the link, hands out the tile's map (a, h; cut: it restarts), ...
    __device__ __forceinline__ void hand_out(int place, int lane, const float (&a)[CPL], const float (&h)[CPL], bool cut) const
    {
        if (place == places - 1)
            return;
        if (!ends_group(place))
            publish_map(map_of(place), lane, a, h, cut);
        else if (cut)
            hand_out_group(place, lane, a, h, true);
    }
    // (a group's last tile) ... the group's, or, as the stretch's last, the next one's front, which a restart alone tells, ...
    __device__ __forceinline__ void hand_out_group(int place, int lane, const float (&a)[CPL], const float (&h)[CPL], bool cut) const
    {
        if (!ends_stretch(place))
            publish_map(map_of(place), lane, a, h, cut);
        else if (cut)
            publish_front(stretch_of(place) + 1, lane, h);
    }
    __device__ __forceinline__ void fetch(const uint64_t* map, int level, int which, int lane, ChainParts<CPL, LEVELS>& parts) const
    {
        WaveMap<CPL> m;
        const bool again = wait_map(map, lane, m.a, m.h);
        parts.maps[level][which][lane] = m;
        if (lane == 0)
            parts.restart[level][which] = again;
        // a wave's LDS accesses keep their order; the compiler is to keep it too
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        if (lane == 0)
            __hip_atomic_fetch_add(&parts.arrived[level], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    // ... each of the other waves (`which` of them, from 0) fetches one of the maps in front of it in its group and one of
    // the groups' in front, ...
    __device__ __forceinline__ void collect(int place, int which, int lane, ChainParts<CPL, LEVELS>& parts) const
    {
        const int tiles = tiles_before(place), groups = groups_before(place);
        if (which < tiles)
            fetch(map_of(place - tiles + which), 0, which, lane, parts);
        if (LEVELS > 1 && which < groups)
            fetch(map_of((place / RC_GROUP - groups + which) * RC_GROUP + RC_GROUP - 1), 1, which, lane, parts);
    }
    // Fetched maps composed, onto (a, h; cut).
    __device__ __forceinline__ void compose(int level, int count, int lane, ChainParts<CPL, LEVELS>& parts, float (&a)[CPL], float (&h)[CPL],
                                            bool& cut) const
    {
        // the collecting waves end their waits in any case
        while (__builtin_amdgcn_readfirstlane(__hip_atomic_load(&parts.arrived[level], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP)) <
               count)
            __builtin_amdgcn_s_sleep(1);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        for (int j = 0; j < count; ++j) {
            const WaveMap<CPL> o = parts.maps[level][j][lane];
            const bool again = __builtin_amdgcn_readfirstlane(parts.restart[level][j]) != 0;
            cut |= again;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                h[c] = again ? o.h[c] : __builtin_fmaf(o.a[c], h[c], o.h[c]);
                a[c] *= o.a[c];
            }
        }
    }
    // ... and the link makes of these and the stretch's front (the first one's: `v`) the value in front of the tile and hands on
    // what leaves it.  What can be done before the front is there is done by then: from front to front are two
    // multiply-adds.
    __device__ __forceinline__ void link(int place, int lane, const float (&a)[CPL], const float (&h)[CPL], bool cut,
                                         ChainParts<CPL, LEVELS>& parts, float (&v)[CPL], float (&leaves)[CPL]) const
    {
        bool group_cut = false, any_cut = false;
        float ga[CPL], gh[CPL], fa[CPL], fh[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            ga[c] = fa[c] = 1.0f;
            gh[c] = fh[c] = 0.0f;
        }
        compose(0, tiles_before(place), lane, parts, ga, gh, group_cut);
        if (LEVELS > 1 && !cut && ends_group(place) && place != places - 1) {
            float all_a[CPL], all_h[CPL];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                all_h[c] = __builtin_fmaf(a[c], gh[c], h[c]);
                all_a[c] = a[c] * ga[c];
            }
            hand_out_group(place, lane, all_a, all_h, group_cut);
        }
        if constexpr (LEVELS > 1) {
            compose(1, groups_before(place), lane, parts, fa, fh, any_cut);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                gh[c] = group_cut ? gh[c] : __builtin_fmaf(ga[c], fh[c], gh[c]);
                ga[c] *= fa[c];
            }
        }
        any_cut |= group_cut;
        if (stretch_of(place) > 0)
            wait_front(stretch_of(place), lane, v);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            v[c] = any_cut ? gh[c] : __builtin_fmaf(ga[c], v[c], gh[c]);
            leaves[c] = cut ? h[c] : __builtin_fmaf(a[c], v[c], h[c]);
        }
        if (!cut && !(LEVELS > 1 && group_cut) && ends_stretch(place) && place != places - 1)
            publish_front(stretch_of(place) + 1, lane, leaves);
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            parts.value[c][lane] = v[c];
    }

    // By one wave behind a barrier, when the tile has read all it needs: signs off.
    __device__ __forceinline__ uint32_t leave(int place, int lane) const
    {
        uint32_t before = 0;
        if (places > 1 && lane == 0)
            before = __hip_atomic_fetch_add(count_of(place), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return before;
    }
    __device__ __forceinline__ void clear_map(int place, int lane) const
    {
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            status_store(map_of(place) + lane * CPL + c, 0);
    }
    // Last step, some time later: whoever was the group's last to sign off (`before` of them) sets its words back, and
    // the last group's of a stretch those of the stretch.
    __device__ __forceinline__ void clear(int place, int lane, uint32_t before) const
    {
        const int first = place / RC_GROUP * RC_GROUP;
        const int in_group = places - first < RC_GROUP ? places - first : RC_GROUP;
        if (places == 1 || __builtin_amdgcn_readfirstlane(int(before)) != in_group - 1)
            return;
        const int start = stretch_of(place) * STRETCH;  // the stretch's first place
        const int behind = (places - 1) / RC_GROUP + 1 - start / RC_GROUP;
        const int in_stretch = behind < STRETCH / RC_GROUP ? behind : STRETCH / RC_GROUP;
        uint32_t groups = 0;
        if (lane == 0) {
            if (in_stretch > 1)
                groups = __hip_atomic_fetch_add(count_of(start) + RC_COUNTER, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(count_of(place), 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        for (int j = 0; j < in_group - 1; ++j)
            clear_map(first + j, lane);
        if (__builtin_amdgcn_readfirstlane(int(groups)) != in_stretch - 1)
            return;
        for (int j = 0; j < in_stretch - 1; ++j)
            clear_map(start + j * RC_GROUP + RC_GROUP - 1, lane);
        if (start > 0) {
            const uint32_t none[CPL] = {};
            store_front(stretch_of(place), lane, none);
        }
        if (in_stretch > 1 && lane == 0)
            __hip_atomic_store(count_of(start) + RC_COUNTER, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

// What a block works on.
template <int CPL, bool PACKED, bool CHAINED>
struct Work {
    static constexpr int CH = 64 * CPL;
    int lane, wave, waves, tile_rows, tile_shift;
    uint32_t chains, which, member, members;  // this block's chain, and which of the chain's blocks it is
    int64_t chain, c0;                        // sequence, first channel
    uint32_t here;                            // channels
    int64_t rows;                             // there are
    int places;                               // tiles with rows

    __device__ __forceinline__ Work(int rows_per_wave, int64_t sequences, int64_t call_rows, int64_t channels, const int64_t* offsets)
    {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        waves = blockDim.x >> 6;
        tile_rows = waves * rows_per_wave;
        tile_shift = __builtin_ctz(uint32_t(tile_rows));
        const uint32_t groups = uint32_t((channels + CH - 1) / CH);
        chains = (PACKED ? 1 : uint32_t(sequences)) * groups;
        which = CHAINED ? blockIdx.x % chains : blockIdx.x;
        member = CHAINED ? blockIdx.x / chains : 0;
        members = CHAINED ? gridDim.x / chains : 1;
        chain = which / groups;
        c0 = int64_t(which % groups) * CH;
        here = uint32_t(channels - c0 < CH ? channels - c0 : CH);
        rows = call_rows;
        if constexpr (PACKED) {
            const int64_t live = offsets[sequences];
            rows = int64_t(uniform(uint64_t(live < 0 ? 0 : live < rows ? live : rows)));
        }
        places = int((rows + tile_rows - 1) >> tile_shift);
    }
};

// ---------------------------------------------------------------- forward

template <class E, int CPL, int ROWS, int WAVES, int GATING, bool PACKED, int LEVELS, bool ONCE>
__global__ __launch_bounds__(64 * WAVES, 4) void recur_forward_kernel(RecurForward q, void* ws, ChainLayout layout)
{
    constexpr bool CHAINED = LEVELS > 0;
    static_assert(WAVES >= RC_GROUP && ROWS * WAVES <= RC_TILE, "each map of a group needs a wave");
    __shared__ WaveMap<CPL> maps[CHAINED ? 1 : 2][WAVES][64];
    __shared__ int restart[CHAINED ? 1 : 2][WAVES];
    __shared__ ChainParts<CPL, CHAINED ? LEVELS : 1> parts;
    __shared__ int head_seq[PACKED ? RC_TILE : 1], end_seq[PACKED ? RC_TILE : 1];
    __shared__ uint32_t place_shared;
    const Work<CPL, PACKED, CHAINED> w(ROWS, q.sequences, q.rows, q.channels, q.offsets);
    const int lane = w.lane, wave = w.wave, waves = w.waves;
    const int64_t chain = w.chain, c0 = w.c0, rows = w.rows;
    const uint32_t bytes = w.here * E::size, state_bytes = w.here * 4, voff = lane * CPL * E::size;
    const char* x = static_cast<const char*>(q.x) + (chain * q.x_sequence + c0) * E::size;
    const char* g = static_cast<const char*>(q.gate) + (chain * q.gate_sequence + c0) * E::size;
    const char* out = static_cast<const char*>(q.out) + (chain * q.out_sequence + c0) * E::size;
    const int64_t periods = (q.rows + RC_PERIOD - 1) / RC_PERIOD;

    uint32_t rx[ROWS], rg[ROWS];
    auto load_rows = [&](int64_t row) {
        const int n = rows_left(rows, row, ROWS);
        RowWalk wx(x, row, q.x_row * E::size, bytes, n), wg(g, row, q.gate_row * E::size, bytes, n);
#pragma unroll
        for (int j = 0; j < ROWS; ++j, wx.next(), wg.next()) {
            rx[j] = load_part<E, CPL, ONCE>(wx.window(), voff);
            rg[j] = load_part<E, CPL, ONCE>(wg.window(), voff);
        }
    };

    Chain<CPL, CHAINED ? LEVELS : 1> links;
    int place = 0;
    if constexpr (CHAINED) {
        links = Chain<CPL, LEVELS>(ws, layout, w.which);
        links.places = w.places;
        if (threadIdx.x < 2)
            parts.arrived[threadIdx.x] = 0;
        if constexpr (PACKED) {
            RowMarks<const int64_t*> marks(q.offsets, q.sequences, head_seq, end_seq);
            place = links.take_place(place_shared);
            marks.mark(q.offsets, q.sequences, int64_t(place) << w.tile_shift, w.tile_rows, head_seq, end_seq, lane);
            __syncthreads();
        } else {
            place = links.take_place(place_shared);
        }
    }
    // what is in front of the sequence; of a block that walks, of its next tile
    float carry[CPL] = {};
    if (!PACKED && q.state != nullptr && (!CHAINED || links.stretch_of(place) == 0))  // the first stretch's front
        load_state<CPL>(make_rsrc(q.state + chain * q.state_row + c0, state_bytes), lane, carry);
    if (place < w.places)
        load_rows((int64_t(place) << w.tile_shift) + wave * ROWS);
    for (int turn = 0; place < w.places; ++place, turn ^= 1) {
        const int64_t row0 = int64_t(place) << w.tile_shift, row = row0 + wave * ROWS;
        float a[ROWS][CPL], b[ROWS][CPL];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            float xv[CPL], gv[CPL];
            E::unpack(rx[j], xv);
            E::unpack(rg[j], gv);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                token_map<GATING>(gv[c], xv[c], a[j][c], b[j][c]);
        }
        const int have = rows_left(rows, row, ROWS);
        if (have < ROWS) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (j >= have) {
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        a[j][c] = 1.0f;
                        b[j][c] = 0.0f;
                    }
                }
        }
        if (!CHAINED && place + 1 < w.places)
            load_rows(row + w.tile_rows);
        uint32_t heads = 0, ends = 0;
        int hs = -1, es = -1;
        if constexpr (PACKED) {
            hs = head_seq[wave * ROWS + lane % ROWS];
            es = end_seq[wave * ROWS + lane % ROWS];
            heads = uint32_t(__ballot(lane < ROWS && hs >= 0));
            ends = uint32_t(__ballot(lane < ROWS && es >= 0));
            if (heads != 0 && q.state != nullptr) {
                // four rows' states on their way at a time
#pragma unroll
                for (int j0 = 0; j0 < ROWS; j0 += 4) {
                    float h0[4][CPL];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool head = (heads >> (j0 + j)) & 1;
                        const int64_t s = head ? read_lane(hs, j0 + j) : 0;
                        load_state<CPL>(row_window(q.state + c0 + s * q.state_row, head, state_bytes), lane, h0[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((heads >> (j0 + j)) & 1) {
#pragma unroll
                            for (int c = 0; c < CPL; ++c)
                                b[j0 + j][c] = __builtin_fmaf(a[j0 + j][c], h0[j][c], b[j0 + j][c]);
                        }
                }
            }
        }

        WaveMap<CPL> m;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            m.a[c] = 1.0f;
            m.h[c] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const bool head = PACKED && ((heads >> j) & 1);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                if (head)
                    m.h[c] = 0.0f;
                m.h[c] = __builtin_fmaf(a[j][c], m.h[c], b[j][c]);
                m.a[c] *= a[j][c];
            }
        }
        if constexpr (!PACKED) {
            // the state is here before the map goes out: the chain's end, or the wave that walked to the end, may write
            // it in place
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                asm volatile("" : "+v"(carry[c]));
        }
        maps[turn][wave][lane] = m;
        if (PACKED && lane == 0)
            restart[turn][wave] = heads != 0;
        __syncthreads();
        float h[CPL];
        uint32_t left = 0;
        if constexpr (!CHAINED) {
            for (int i = 0; i < waves; ++i) {
                const WaveMap<CPL> o = maps[turn][i][lane];
                const bool again = PACKED && __builtin_amdgcn_readfirstlane(restart[turn][i]) != 0;
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    if (i == wave)
                        h[c] = carry[c];
                    carry[c] = again ? o.h[c] : __builtin_fmaf(o.a[c], carry[c], o.h[c]);
                }
            }
        } else {
            // the waves in front, as a map
            WaveMap<CPL> before;
            bool cut = false;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                before.a[c] = 1.0f;
                before.h[c] = 0.0f;
            }
            for (int i = 0; i < wave; ++i) {
                const WaveMap<CPL> o = maps[0][i][lane];
                const bool again = PACKED && __builtin_amdgcn_readfirstlane(restart[0][i]) != 0;
                cut |= again;
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    before.h[c] = again ? o.h[c] : __builtin_fmaf(o.a[c], before.h[c], o.h[c]);
                    before.a[c] *= o.a[c];
                }
            }
            if (wave == waves - 1) {
                const bool any = cut || heads != 0;
                float leaves[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    m.h[c] = heads != 0 ? m.h[c] : __builtin_fmaf(m.a[c], before.h[c], m.h[c]);
                    m.a[c] *= before.a[c];
                }
                links.hand_out(place, lane, m.a, m.h, any);
                links.link(place, lane, m.a, m.h, any, parts, carry, leaves);
                if (!PACKED && place == w.places - 1)
                    store_state<CPL>(make_rsrc(q.state_out + chain * q.state_out_row + c0, state_bytes), lane, leaves);
            } else {
                links.collect(place, wave, lane, parts);
            }
            __syncthreads();
            if (wave == 0)
                left = links.leave(place, lane);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                h[c] = cut ? before.h[c] : __builtin_fmaf(before.a[c], parts.value[c][lane], before.h[c]);
        }
        if (q.carries != nullptr && row < rows && row % RC_PERIOD == 0)
            store_state<CPL>(make_rsrc(q.carries + (chain * periods + row / RC_PERIOD) * q.channels + c0, state_bytes), lane, h);
        RowWalk wo(out, row, q.out_row * E::size, bytes, have);
#pragma unroll
        for (int j = 0; j < ROWS; ++j, wo.next()) {
            const bool head = PACKED && ((heads >> j) & 1);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                h[c] = __builtin_fmaf(a[j][c], head ? 0.0f : h[c], b[j][c]);
            store_part<E, CPL>(wo.window(), voff, h);
            if (PACKED && ((ends >> j) & 1))
                store_state<CPL>(make_rsrc(q.state_out + read_lane(es, j) * q.state_out_row + c0, state_bytes), lane, h);
        }
        if constexpr (CHAINED) {
            if (wave == 0)
                links.clear(place, lane, left);
            break;
        }
    }
    if constexpr (!PACKED) {
        if (!CHAINED && wave == 0)
            store_state<CPL>(make_rsrc(q.state_out + chain * q.state_out_row + c0, state_bytes), lane, carry);
    } else if (q.state != q.state_out) {
        for (int64_t s = int64_t(w.member) * waves + wave; s < q.sequences; s += int64_t(w.members) * waves)
            if (q.offsets[s + 1] <= q.offsets[s]) {
                float h[CPL] = {};
                if (q.state != nullptr)
                    load_state<CPL>(make_rsrc(q.state + s * q.state_row + c0, state_bytes), lane, h);
                store_state<CPL>(make_rsrc(q.state_out + s * q.state_out_row + c0, state_bytes), lane, h);
            }
    }
}

// ---------------------------------------------------------------- backward

// A wave's map forward, and the gradient that leaves it in front when none comes from behind.
template <int CPL>
struct alignas(4 * CPL) WaveBack {
    float a[CPL], h[CPL], mu[CPL];
};

template <class E, int CPL, int ROWS, int WAVES, int GATING, bool PACKED, int LEVELS, bool ONCE>
__global__ __launch_bounds__(64 * WAVES, 4) void recur_backward_kernel(RecurBackward q, void* ws, ChainLayout layout)
{
    constexpr bool CHAINED = LEVELS > 0;
    static_assert(WAVES >= RC_GROUP && ROWS * WAVES <= RC_TILE && RC_PERIOD % ROWS == 0, "each map of a group needs a wave");
    __shared__ WaveBack<CPL> maps[CHAINED ? 1 : 2][WAVES][64];
    __shared__ int restart[CHAINED ? 1 : 2][WAVES][2];
    __shared__ ChainParts<CPL, CHAINED ? LEVELS : 1> parts;
    __shared__ int head_seq[PACKED ? RC_TILE : 1], end_seq[PACKED ? RC_TILE : 1];
    __shared__ uint32_t place_shared;
    const Work<CPL, PACKED, CHAINED> w(ROWS, q.sequences, q.rows, q.channels, q.offsets);
    const int lane = w.lane, wave = w.wave, waves = w.waves;
    const int64_t chain = w.chain, c0 = w.c0, rows = w.rows;
    const uint32_t bytes = w.here * E::size, state_bytes = w.here * 4, voff = lane * CPL * E::size;
    const char* x = static_cast<const char*>(q.x) + (chain * q.x_sequence + c0) * E::size;
    const char* g = static_cast<const char*>(q.gate) + (chain * q.gate_sequence + c0) * E::size;
    const char* dout = static_cast<const char*>(q.dout) + (chain * q.dout_sequence + c0) * E::size;
    const char* dx = static_cast<const char*>(q.dx) + (chain * q.dx_sequence + c0) * E::size;
    const char* dg = static_cast<const char*>(q.dgate) + (chain * q.dgate_sequence + c0) * E::size;
    const int64_t periods = (q.rows + RC_PERIOD - 1) / RC_PERIOD;

    // place 0 is the last tile
    auto first_row = [&](int place) { return int64_t(w.places - 1 - place) << w.tile_shift; };

    Chain<CPL, CHAINED ? LEVELS : 1> links;
    int place = 0;
    if constexpr (CHAINED) {
        links = Chain<CPL, LEVELS>(ws, layout, w.which);
        links.places = w.places;
        if (threadIdx.x < 2)
            parts.arrived[threadIdx.x] = 0;
        if constexpr (PACKED) {
            RowMarks<const int64_t*> marks(q.offsets, q.sequences, head_seq, end_seq);
            place = links.take_place(place_shared);
            marks.mark(q.offsets, q.sequences, first_row(place), w.tile_rows, head_seq, end_seq, lane);
            __syncthreads();
        } else {
            place = links.take_place(place_shared);
        }
    }
    float mu_carry[CPL] = {};
    if (!PACKED && q.dstate_out != nullptr && (!CHAINED || links.stretch_of(place) == 0))  // the first stretch's front
        load_state<CPL>(make_rsrc(q.dstate_out + chain * q.dstate_out_row + c0, state_bytes), lane, mu_carry);
    for (int turn = 0; place < w.places; ++place, turn ^= 1) {
        const int64_t row0 = first_row(place), row = row0 + wave * ROWS;
        const int have = rows_left(rows, row, ROWS);
        uint32_t rx[ROWS], rg[ROWS], rd[ROWS];
        float h[CPL];  // in front of the wave's period
        load_state<CPL>(row_window(q.carries + c0 + (chain * periods + row / RC_PERIOD) * q.channels, have > 0, state_bytes), lane, h);
        RowWalk wx(x, row, q.x_row * E::size, bytes, have), wg(g, row, q.gate_row * E::size, bytes, have),
            wd(dout, row, q.dout_row * E::size, bytes, have);
#pragma unroll
        for (int j = 0; j < ROWS; ++j, wx.next(), wg.next(), wd.next()) {
            rx[j] = load_part<E, CPL, ONCE>(wx.window(), voff);
            rg[j] = load_part<E, CPL, ONCE>(wg.window(), voff);
            rd[j] = load_part<E, CPL, ONCE>(wd.window(), voff);
        }
        uint32_t heads = 0, ends = 0;
        int hs = -1, es = -1;
        if constexpr (PACKED) {
            hs = head_seq[wave * ROWS + lane % ROWS];
            es = end_seq[wave * ROWS + lane % ROWS];
            heads = uint32_t(__ballot(lane < ROWS && hs >= 0));
            ends = uint32_t(__ballot(lane < ROWS && es >= 0));
        }
        auto state_of = [&](int j, float (&v)[CPL]) {
            const int64_t s = read_lane(hs, j);
            load_state<CPL>(row_window(q.state + c0 + s * q.state_row, q.state != nullptr, state_bytes), lane, v);
        };
        auto gradient_of = [&](int j, float (&v)[CPL]) {
            const int64_t s = read_lane(es, j);
            load_state<CPL>(row_window(q.dstate_out + c0 + s * q.dstate_out_row, q.dstate_out != nullptr, state_bytes), lane, v);
        };

        Decay<GATING> decay[ROWS][CPL];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            float gv[CPL];
            E::unpack(rg[j], gv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                decay[j][c].make(gv[c]);
                if (j >= have)
                    decay[j][c].nothing();
            }
        }
        // Each pass over the rows makes a and 1 - a again: kept, they would take twice the registers, and a CU hold
        // fewer blocks.
        auto forget = [&]() {
            if constexpr (GATING == GATE_SIGMOID) {
#pragma unroll
                for (int j = 0; j < ROWS; ++j)
#pragma unroll
                    for (int c = 0; c < CPL; ++c)
                        asm volatile("" : "+v"(decay[j][c].u));
            }
        };
        WaveBack<CPL> m;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            m.a[c] = 1.0f;
            m.h[c] = 0.0f;
            m.mu[c] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && ((heads >> j) & 1))
                state_of(j, m.h);
            float xv[CPL];
            E::unpack(rx[j], xv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const float a = decay[j][c].a();
                m.h[c] = __builtin_fmaf(a, m.h[c], decay[j][c].rest() * xv[c]);
                m.a[c] *= a;
            }
        }
        forget();
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j) {
            if (PACKED && ((ends >> j) & 1))
                gradient_of(j, m.mu);
            float dv[CPL];
            E::unpack(rd[j], dv);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                m.mu[c] = decay[j][c].a() * (dv[c] + m.mu[c]);
        }
        maps[turn][wave][lane] = m;
        if (PACKED && lane == 0) {
            restart[turn][wave][0] = heads != 0;
            restart[turn][wave][1] = ends != 0;
        }
        __syncthreads();
        // h in front of the wave, from its period's carry
        constexpr int PER = RC_PERIOD / ROWS;
        for (int i = wave / PER * PER; i < wave; ++i) {
            const WaveBack<CPL> o = maps[turn][i][lane];
            const bool again = PACKED && __builtin_amdgcn_readfirstlane(restart[turn][i][0]) != 0;
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                h[c] = again ? o.h[c] : __builtin_fmaf(o.a[c], h[c], o.h[c]);
        }
        float mu[CPL];
        uint32_t left = 0;
        if constexpr (!CHAINED) {
            for (int i = waves - 1; i >= 0; --i) {
                const WaveBack<CPL> o = maps[turn][i][lane];
                const bool again = PACKED && __builtin_amdgcn_readfirstlane(restart[turn][i][1]) != 0;
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    if (i == wave)
                        mu[c] = mu_carry[c];
                    mu_carry[c] = again ? o.mu[c] : __builtin_fmaf(o.a[c], mu_carry[c], o.mu[c]);
                }
            }
        } else {
            // the waves behind, as a map
            WaveMap<CPL> later;
            bool cut = false;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                later.a[c] = 1.0f;
                later.h[c] = 0.0f;
            }
            for (int i = waves - 1; i > wave; --i) {
                const WaveBack<CPL> o = maps[0][i][lane];
                const bool again = PACKED && __builtin_amdgcn_readfirstlane(restart[0][i][1]) != 0;
                cut |= again;
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    later.h[c] = again ? o.mu[c] : __builtin_fmaf(o.a[c], later.h[c], o.mu[c]);
                    later.a[c] *= o.a[c];
                }
            }
            if (wave == 0) {
                const bool any = cut || ends != 0;
                float leaves[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    m.mu[c] = ends != 0 ? m.mu[c] : __builtin_fmaf(m.a[c], later.h[c], m.mu[c]);
                    m.a[c] *= later.a[c];
                }
                links.hand_out(place, lane, m.a, m.mu, any);
                links.link(place, lane, m.a, m.mu, any, parts, mu_carry, leaves);
                if (!PACKED && place == w.places - 1)
                    store_state<CPL>(make_rsrc(q.dstate + chain * q.dstate_row + c0, state_bytes), lane, leaves);
            } else {
                links.collect(place, wave - 1, lane, parts);
            }
            __syncthreads();
            if (wave == 0)
                left = links.leave(place, lane);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                mu[c] = cut ? later.h[c] : __builtin_fmaf(later.a[c], parts.value[c][lane], later.h[c]);
        }
        float before[ROWS][CPL];
        forget();
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && ((heads >> j) & 1))
                state_of(j, h);
            float xv[CPL];
            E::unpack(rx[j], xv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                before[j][c] = h[c];
                h[c] = __builtin_fmaf(decay[j][c].a(), h[c], decay[j][c].rest() * xv[c]);
            }
        }
        forget();
        RowWalk ox(dx, row + ROWS - 1, q.dx_row * E::size, bytes, have == ROWS),
            og(dg, row + ROWS - 1, q.dgate_row * E::size, bytes, have == ROWS);
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j, ox.previous(j < have), og.previous(j < have)) {
            if (PACKED && ((ends >> j) & 1))
                gradient_of(j, mu);
            float dv[CPL], xv[CPL], gx[CPL], gg[CPL];
            E::unpack(rd[j], dv);
            E::unpack(rx[j], xv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const float a = decay[j][c].a(), lam = dv[c] + mu[c];
                mu[c] = a * lam;
                gx[c] = lam * decay[j][c].rest();
                gg[c] = GATING == GATE_SIGMOID ? gx[c] * a * (before[j][c] - xv[c])
                                               : (GATING == GATE_LOG ? mu[c] : lam) * before[j][c];
            }
            store_part<E, CPL>(ox.window(), voff, gx);
            store_part<E, CPL>(og.window(), voff, gg);
            if (PACKED && ((heads >> j) & 1))
                store_state<CPL>(make_rsrc(q.dstate + read_lane(hs, j) * q.dstate_row + c0, state_bytes), lane, mu);
        }
        if constexpr (CHAINED) {
            if (wave == 0)
                links.clear(place, lane, left);
            break;
        }
    }
    if constexpr (!PACKED) {
        if (!CHAINED && wave == 0)
            store_state<CPL>(make_rsrc(q.dstate + chain * q.dstate_row + c0, state_bytes), lane, mu_carry);
    } else {
        for (int64_t s = int64_t(w.member) * waves + wave; s < q.sequences; s += int64_t(w.members) * waves)
            if (q.offsets[s + 1] <= q.offsets[s]) {
                float v[CPL] = {};
                if (q.dstate_out != nullptr)
                    load_state<CPL>(make_rsrc(q.dstate_out + s * q.dstate_out_row + c0, state_bytes), lane, v);
                store_state<CPL>(make_rsrc(q.dstate + s * q.dstate_row + c0, state_bytes), lane, v);
            }
    }
}

// ---------------------------------------------------------------- one token a sequence

// VEC neighbouring channels per thread: 16 bytes of x, or one element where rows are not aligned.  One pass: x, gate and
// state in, out and state out; 256 sequences of 4096 bfloat16 channels take 4.7 us (14.7 MB: 2.4 at 6.2 TB/s and the launch's 2),
// one sequence of 2048 2.2.
template <class E, int VEC>
__global__ __launch_bounds__(256) void recur_step_kernel(RecurForward q)
{
    const int64_t parts = (q.channels + VEC - 1) / VEC;
    for (int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x; at < q.sequences * parts; at += int64_t(gridDim.x) * 256) {
        const int64_t s = at / parts, c = at % parts * VEC;
        Elements<E, VEC> ex, eg;
        Elements<F32, VEC> es;
        ex.load(static_cast<const char*>(q.x) + (s * q.x_sequence + c) * E::size);
        eg.load(static_cast<const char*>(q.gate) + (s * q.gate_sequence + c) * E::size);
        float h[VEC] = {}, a[VEC], b[VEC];
        if (q.state != nullptr) {
            es.load(q.state + s * q.state_row + c);
            es.get(h);
        }
        if (q.carries != nullptr)
            es.set(h), es.store(q.carries + s * q.channels + c);
        ex.get(b);
        eg.get(a);
    #pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if (q.gating == GATE_SIGMOID) {
                float rest;
                sigmoid_both(a[i], a[i], rest);
                b[i] *= rest;
            } else if (q.gating == GATE_LOG) {
                a[i] = gate_exp(a[i]);
            }
            h[i] = __builtin_fmaf(a[i], h[i], b[i]);
        }
        ex.set(h);
        ex.store(static_cast<char*>(q.out) + (s * q.out_sequence + c) * E::size);
        es.set(h);
        es.store(q.state_out + s * q.state_out_row + c);
    }
}

// ---------------------------------------------------------------- launches

// Blocks that walk keep the carry to themselves and load ahead; they take the call where the chains alone fill the
// GPU, or where a chain is one tile.  From 256 chains on: 8 x 4096 x 4096 (256) forward 151 us against 166, but 6 x 4096 x
// 8192 (384) 256 against 238, and backward slower in both; from 2048 on: 64 x 512 x 2048 (1024) 84 against 75.
// 512 such blocks run at once forward, so just above it the second round is nearly empty, and tiles would be faster: of 4096
// tokens of bfloat16, 512 chains walk in 289 and 526 us, 520 in 391 and 701 against 328 and 593 as tiles, 576 in 408 and 739
// against 366 and 662, 704 in 464 and 812 against 449 and 809, 768 in 462 and 798 against 514 and 912, 900 in 596 and 1076 against
// 575 and 1040, 1024 in 598 and 1103 against 669 and 1259, 2048 in 1228 and 2154 against 1348 and 2528.
constexpr int64_t RC_WALKERS = 512;

// Tokens per wave, and waves, of a tile.  1 x 65536 x 2048 forward with 8 tokens a wave 237 us against 183; backward of two
// channels a lane with 16 waves of 8 tokens 340 against 342, but 319 against 273 for 8 x 4096 x 4096.
template <int CPL>
struct ForwardShape {
    static constexpr int rows = 16, waves = 8;
};
template <int CPL>
struct BackwardShape {
    static constexpr int rows = CPL == 2 ? 8 : 16, waves = 8;
};

struct ChainPlan {
    bool chained;
    int waves;
    int64_t chains, tiles;
};
static constexpr ChainPlan chain_plan(int64_t sequences, int64_t rows, int64_t channels, bool packed, int per_lane, int wave_rows, int most_waves,
                            int least_waves)
{
    const int64_t chains = (packed ? 1 : sequences) * ((channels + 64 * per_lane - 1) / (64 * per_lane));
    int waves = most_waves;
    while (waves > least_waves && (waves / 2) * wave_rows >= rows)
        waves /= 2;
    const int64_t tiles = (rows + waves * wave_rows - 1) / (waves * wave_rows);
    return {packed || (tiles > 1 && chains < RC_WALKERS), waves, chains, tiles > 0 ? tiles : 1};
}

template <int CPL>
static constexpr ChainPlan plan_of(bool backward, int64_t sequences, int64_t rows, int64_t channels, bool packed)
{
    using F = ForwardShape<CPL>;
    using B = BackwardShape<CPL>;
    return backward ? chain_plan(sequences, rows, channels, packed, CPL, B::rows, B::waves, RC_PERIOD / B::rows)
                    : chain_plan(sequences, rows, channels, packed, CPL, F::rows, F::waves, 1);
}

// A block of fewer waves holds all rows in its one tile.  Of several tiles, each block has the link and a wave for
// every map that it collects: Chain::compose waits for them without a limit of its own.
template <int CPL>
static constexpr bool tiles_have_collectors()
{
    for (int64_t rows = 0; rows <= 4 * RC_TILE; ++rows)
        for (int which = 0; which < 4; ++which) {
            const ChainPlan p = plan_of<CPL>(which % 2 != 0, 1, rows, 64, which / 2 != 0);
            if (p.tiles > 1 && p.waves < RC_GROUP)
                return false;
        }
    return true;
}
static_assert(tiles_have_collectors<1>() && tiles_have_collectors<2>(), "a group's maps need a wave each");

template <int CPL>
static size_t chain_bytes(int64_t sequences, int64_t rows, int64_t channels, bool packed)
{
    size_t most = 0;
    for (int back = 0; back < 2; ++back) {
        const ChainPlan p = plan_of<CPL>(back != 0, sequences, rows, channels, packed);
        const size_t n = p.chained ? chain_layout(p.chains, p.tiles, 64 * CPL).bytes : 0;
        most = n > most ? n : most;
    }
    return most;
}

size_t recur_workspace_bytes(int64_t sequences, int64_t rows, int64_t channels, bool packed, int type)
{
    if (!packed && rows <= 1)
        return 0;
    size_t most = sizeof(WsHeader);
    const size_t one = chain_bytes<1>(sequences, rows, channels, packed);
    const size_t two = type == LOGITS_F32 ? 0 : chain_bytes<2>(sequences, rows, channels, packed);  // which one, the alignment tells
    most = one > most ? one : most;
    most = two > most ? two : most;
    return most;
}

int64_t recur_carry_rows(int64_t sequences, int64_t rows, bool packed)
{
    return (packed ? 1 : sequences) * ((rows + RC_PERIOD - 1) / RC_PERIOD);
}

namespace {

bool multiples(const void* p, int64_t a, int64_t b, int64_t to)
{
    return reinterpret_cast<uintptr_t>(p) % uintptr_t(to) == 0 && a % to == 0 && b % to == 0;
}

// x and gate that the memory-side cache (256 MiB) holds beside what the call writes are loaded as usual: it may have them,
// from the products that made them or from the forward pass.  More are loaded past the caches.  Forward and backward one after
// the other, loads as usual and past the caches, on five sets of inputs in turn and on the same inputs again: x and
// gate of 128 MiB (4 x 4096 x 2048 bfloat16) 135 and 128 us, 107 and 126; 41 MiB (3 x 1777 x 1001 float32) 52 and 60,
// 46 and 57; 256 MiB 264 and 250, 255 and 250; 512 MiB 486 and 453, 480 and 452.
constexpr int64_t RC_ONCE_ALL = 192 << 20;
template <class Q>
bool loads_once(const Q& q, int size, int per_lane)
{
    // few chains wait for each other more than for memory, and have kernels of their own
    const int64_t chains = (q.offsets != nullptr ? 1 : q.sequences) * ((q.channels + 64 * per_lane - 1) / (64 * per_lane));
    return chain_levels(chains) == 1 && (q.offsets != nullptr ? 1 : q.sequences) * q.rows * q.channels * size * 2 >= RC_ONCE_ALL;
}

// A launch holds less than 2^32 threads.  Of tiles as blocks, 2^23 - 1 of 512 threads: a call of more does not fit.
constexpr int64_t RC_BLOCKS = (int64_t(1) << 23) - 1;
// Of blocks that walk: most sequences of a launch of `groups` blocks each.  More are halved, so that each half still has chains
// enough to walk: what a call takes of its workspace goes by all its sequences.
int64_t sequences_at_once(int64_t groups) { return (int64_t(1) << 22) / groups > 0 ? (int64_t(1) << 22) / groups : 1; }

template <class E, int CPL, int GATING, bool ONCE>
hipError_t forward_of(const RecurForward& q, void* ws, hipStream_t stream)
{
    using S = ForwardShape<CPL>;
    const ChainPlan p = plan_of<CPL>(false, q.sequences, q.rows, q.channels, q.offsets != nullptr);
    const ChainLayout layout = chain_layout(p.chains, p.tiles, 64 * CPL);
    const dim3 blocks(uint32_t(p.chained ? p.chains * p.tiles : p.chains)), threads(64 * p.waves);
    if constexpr (!ONCE) {
        if (p.chained && chain_levels(p.chains) == 2) {
            if (q.offsets != nullptr)
                recur_forward_kernel<E, CPL, S::rows, S::waves, GATING, true, 2, false><<<blocks, threads, 0, stream>>>(q, ws, layout);
            else
                recur_forward_kernel<E, CPL, S::rows, S::waves, GATING, false, 2, false><<<blocks, threads, 0, stream>>>(q, ws, layout);
            return hipGetLastError();
        }
    }
    if (p.chained && q.offsets != nullptr)
        recur_forward_kernel<E, CPL, S::rows, S::waves, GATING, true, 1, ONCE><<<blocks, threads, 0, stream>>>(q, ws, layout);
    else if (p.chained)
        recur_forward_kernel<E, CPL, S::rows, S::waves, GATING, false, 1, ONCE><<<blocks, threads, 0, stream>>>(q, ws, layout);
    else
        recur_forward_kernel<E, CPL, S::rows, S::waves, GATING, false, 0, ONCE><<<blocks, threads, 0, stream>>>(q, ws, layout);
    return hipGetLastError();
}

template <class E, int CPL, bool ONCE>
hipError_t forward_by(const RecurForward& q, void* ws, hipStream_t stream)
{
    if (q.gating == GATE_DECAY)
        return forward_of<E, CPL, GATE_DECAY, ONCE>(q, ws, stream);
    if (q.gating == GATE_LOG)
        return forward_of<E, CPL, GATE_LOG, ONCE>(q, ws, stream);
    return forward_of<E, CPL, GATE_SIGMOID, ONCE>(q, ws, stream);
}

template <class E, int CPL>
hipError_t launch_forward(const RecurForward& q, void* ws, hipStream_t stream)
{
    const int64_t groups = (q.channels + 64 * CPL - 1) / (64 * CPL);
    if (q.offsets == nullptr && q.sequences > sequences_at_once(groups)) {
        const int64_t half = q.sequences / 2;
        RecurForward first = q, rest = q;
        first.sequences = half;
        rest.sequences -= half;
        rest.x = static_cast<const char*>(q.x) + half * q.x_sequence * E::size;
        rest.gate = static_cast<const char*>(q.gate) + half * q.gate_sequence * E::size;
        rest.out = static_cast<char*>(q.out) + half * q.out_sequence * E::size;
        if (q.state != nullptr)
            rest.state += half * q.state_row;
        rest.state_out += half * q.state_out_row;
        if (q.carries != nullptr)
            rest.carries += recur_carry_rows(half, q.rows, false) * q.channels;
        const hipError_t e = launch_forward<E, CPL>(first, ws, stream);
        return e != hipSuccess ? e : launch_forward<E, CPL>(rest, ws, stream);
    }
    return loads_once(q, E::size, CPL) ? forward_by<E, CPL, true>(q, ws, stream) : forward_by<E, CPL, false>(q, ws, stream);
}

template <class E, int CPL, int GATING, bool ONCE>
hipError_t backward_of(const RecurBackward& q, void* ws, hipStream_t stream)
{
    using S = BackwardShape<CPL>;
    const ChainPlan p = plan_of<CPL>(true, q.sequences, q.rows, q.channels, q.offsets != nullptr);
    const ChainLayout layout = chain_layout(p.chains, p.tiles, 64 * CPL);
    const dim3 blocks(uint32_t(p.chained ? p.chains * p.tiles : p.chains)), threads(64 * p.waves);
    if constexpr (!ONCE) {
        if (p.chained && chain_levels(p.chains) == 2) {
            if (q.offsets != nullptr)
                recur_backward_kernel<E, CPL, S::rows, S::waves, GATING, true, 2, false><<<blocks, threads, 0, stream>>>(q, ws, layout);
            else
                recur_backward_kernel<E, CPL, S::rows, S::waves, GATING, false, 2, false><<<blocks, threads, 0, stream>>>(q, ws, layout);
            return hipGetLastError();
        }
    }
    if (p.chained && q.offsets != nullptr)
        recur_backward_kernel<E, CPL, S::rows, S::waves, GATING, true, 1, ONCE><<<blocks, threads, 0, stream>>>(q, ws, layout);
    else if (p.chained)
        recur_backward_kernel<E, CPL, S::rows, S::waves, GATING, false, 1, ONCE><<<blocks, threads, 0, stream>>>(q, ws, layout);
    else
        recur_backward_kernel<E, CPL, S::rows, S::waves, GATING, false, 0, ONCE><<<blocks, threads, 0, stream>>>(q, ws, layout);
    return hipGetLastError();
}

template <class E, int CPL, bool ONCE>
hipError_t backward_by(const RecurBackward& q, void* ws, hipStream_t stream)
{
    if (q.gating == GATE_DECAY)
        return backward_of<E, CPL, GATE_DECAY, ONCE>(q, ws, stream);
    if (q.gating == GATE_LOG)
        return backward_of<E, CPL, GATE_LOG, ONCE>(q, ws, stream);
    return backward_of<E, CPL, GATE_SIGMOID, ONCE>(q, ws, stream);
}

template <class E, int CPL>
hipError_t launch_backward(const RecurBackward& q, void* ws, hipStream_t stream)
{
    const int64_t groups = (q.channels + 64 * CPL - 1) / (64 * CPL);
    if (q.offsets == nullptr && q.sequences > sequences_at_once(groups)) {
        const int64_t half = q.sequences / 2;
        RecurBackward first = q, rest = q;
        first.sequences = half;
        rest.sequences -= half;
        rest.dout = static_cast<const char*>(q.dout) + half * q.dout_sequence * E::size;
        rest.x = static_cast<const char*>(q.x) + half * q.x_sequence * E::size;
        rest.gate = static_cast<const char*>(q.gate) + half * q.gate_sequence * E::size;
        rest.dx = static_cast<char*>(q.dx) + half * q.dx_sequence * E::size;
        rest.dgate = static_cast<char*>(q.dgate) + half * q.dgate_sequence * E::size;
        if (q.state != nullptr)
            rest.state += half * q.state_row;
        if (q.dstate_out != nullptr)
            rest.dstate_out += half * q.dstate_out_row;
        rest.dstate += half * q.dstate_row;
        rest.carries += recur_carry_rows(half, q.rows, false) * q.channels;
        const hipError_t e = launch_backward<E, CPL>(first, ws, stream);
        return e != hipSuccess ? e : launch_backward<E, CPL>(rest, ws, stream);
    }
    return loads_once(q, E::size, CPL) ? backward_by<E, CPL, true>(q, ws, stream) : backward_by<E, CPL, false>(q, ws, stream);
}

// Channels a lane: a word of two 16-bit ones where every row is aligned to that.
int lane_channels(const RecurForward& q, int type)
{
    const bool pairs = type != LOGITS_F32 && q.channels % 2 == 0 && multiples(q.x, q.x_sequence * 2, q.x_row * 2, 4) &&
                       multiples(q.gate, q.gate_sequence * 2, q.gate_row * 2, 4) &&
                       multiples(q.out, q.out_sequence * 2, q.out_row * 2, 4);
    return pairs ? 2 : 1;
}
int lane_channels(const RecurBackward& q, int type)
{
    const bool pairs = type != LOGITS_F32 && q.channels % 2 == 0 && multiples(q.x, q.x_sequence * 2, q.x_row * 2, 4) &&
                       multiples(q.gate, q.gate_sequence * 2, q.gate_row * 2, 4) &&
                       multiples(q.dout, q.dout_sequence * 2, q.dout_row * 2, 4) &&
                       multiples(q.dx, q.dx_sequence * 2, q.dx_row * 2, 4) &&
                       multiples(q.dgate, q.dgate_sequence * 2, q.dgate_row * 2, 4);
    return pairs ? 2 : 1;
}

template <class E>
hipError_t launch_step(const RecurForward& q, hipStream_t stream)
{
    constexpr int VEC = 16 / E::size;
    const bool wide = q.channels % VEC == 0 && multiples(q.x, q.x_sequence * E::size, 0, 16) &&
                      multiples(q.gate, q.gate_sequence * E::size, 0, 16) && multiples(q.out, q.out_sequence * E::size, 0, 16) &&
                      multiples(q.state, q.state_row * 4, 0, 16) && multiples(q.state_out, q.state_out_row * 4, 0, 16) &&
                      multiples(q.carries, 0, 0, 16);
    const int64_t threads = q.sequences * (wide ? q.channels / VEC : q.channels);
    const dim3 blocks(uint32_t(threads < int64_t(1) << 31 ? (threads + 255) / 256 : 1 << 23));
    if (wide)
        recur_step_kernel<E, VEC><<<blocks, dim3(256), 0, stream>>>(q);
    else
        recur_step_kernel<E, 1><<<blocks, dim3(256), 0, stream>>>(q);
    return hipGetLastError();
}

template <class Q>
bool fits(const Q& q, int type, bool backward)
{
    const bool packed = q.offsets != nullptr;
    const ChainPlan p = lane_channels(q, type) == 2 ? plan_of<2>(backward, q.sequences, q.rows, q.channels, packed)
                                                    : plan_of<1>(backward, q.sequences, q.rows, q.channels, packed);
    return q.sequences == 0 || !p.chained || p.chains * p.tiles <= RC_BLOCKS;
}

}  // namespace

bool recurrence_fits(const RecurForward& q, int type) { return fits(q, type, false); }
bool recurrence_fits(const RecurBackward& q, int type) { return fits(q, type, true); }

hipError_t launch_recurrence(const RecurForward& q, int type, void* ws, hipStream_t stream)
{
    if (q.sequences == 0 || q.channels == 0)
        return hipSuccess;
    if (q.offsets == nullptr && q.rows == 1) {
        if (type == LOGITS_F32)
            return launch_step<F32>(q, stream);
        return type == LOGITS_F16 ? launch_step<F16>(q, stream) : launch_step<BF16>(q, stream);
    }
    if (type == LOGITS_F32)
        return launch_forward<F32, 1>(q, ws, stream);
    const bool pairs = lane_channels(q, type) == 2;
    if (type == LOGITS_F16)
        return pairs ? launch_forward<F16, 2>(q, ws, stream) : launch_forward<F16, 1>(q, ws, stream);
    return pairs ? launch_forward<BF16, 2>(q, ws, stream) : launch_forward<BF16, 1>(q, ws, stream);
}

hipError_t launch_recurrence_backward(const RecurBackward& q, int type, void* ws, hipStream_t stream)
{
    if (q.sequences == 0 || q.channels == 0)
        return hipSuccess;
    if (type == LOGITS_F32)
        return launch_backward<F32, 1>(q, ws, stream);
    const bool pairs = lane_channels(q, type) == 2;
    if (type == LOGITS_F16)
        return pairs ? launch_backward<F16, 2>(q, ws, stream) : launch_backward<F16, 1>(q, ws, stream);
    return pairs ? launch_backward<BF16, 2>(q, ws, stream) : launch_backward<BF16, 1>(q, ws, stream);
}

}  // namespace ls
