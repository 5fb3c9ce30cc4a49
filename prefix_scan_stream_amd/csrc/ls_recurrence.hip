// ls_recurrence.hip -- the gated linear recurrence h_t = a_t h_{t-1} + b_t over sequences,
// channel by channel, and its gradients (gfx950).
//
// A token is the affine map h -> a h + b of each channel, and maps compose:
//     (a1, b1) then (a2, b2)  =  (a2 a1, a2 b1 + b2),
// so the recurrence is a scan.  Channels lie beside each other in memory and are
// independent: a lane owns CPL neighbouring channels (4 bytes of a row), a wave RC_ROWS
// consecutive tokens of its 64 CPL channels, and a block's waves lie one behind the other
// in time.  Per tile (waves x RC_ROWS tokens):
//   1. every wave loads its rows (each load 256 consecutive bytes), makes a and b of them in
//      float32 and composes its map;
//   2. the waves' maps meet in LDS; every wave applies those in front of it to the tile's
//      carry and goes through its rows once more, from registers, writing h.
// The block walks the tiles of its sequence (packed rows: of all sequences) and keeps the
// carry in registers; the next tile's rows are on their way while a tile is finished.
//
// Backward, with mu_t = a_t lambda_t the gradient that h_{t-1} receives:
//     lambda_t = dh_t + mu_{t+1},   mu_t = a_t mu_{t+1} + a_t dh_t,
// the same maps' factors from the last token to the first.  A tile needs h again: it is
// made from x and gate, from the carries that the forward pass kept of every RC_PERIOD-th
// row, in 32 bits; the output h would cost as many bytes and is rounded.
//
// A sequence's first row takes its state in place of the carry, by selection and not by a
// factor of 0, so that an infinity in one sequence never reaches the next.
#include "ls_elements.hpp"
#include "ls_internal.hpp"

namespace ls {

constexpr int RC_ROWS = 16;    // tokens per wave and tile
constexpr int RC_WAVES = 8;
constexpr int RC_PERIOD = 64;  // a carry is kept of every 64th row
constexpr int RC_TILE = RC_WAVES * RC_ROWS;
static_assert(RC_TILE % RC_PERIOD == 0 && RC_PERIOD % RC_ROWS == 0, "tiles hold whole periods, periods whole waves");

// A lane's part of a row: 4 bytes, or one 16-bit element where rows are not aligned to two.
template <class E, int CPL>
constexpr bool whole_word = E::size * CPL == 4;

template <class E, int CPL>
__device__ __forceinline__ uint32_t load_part(__amdgpu_buffer_rsrc_t rs, uint32_t voff)
{
    if constexpr (whole_word<E, CPL>)
        return __builtin_amdgcn_raw_buffer_load_b32(rs, voff, 0, CACHE_NT);
    else
        return uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rs, voff, 0, CACHE_NT));
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
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_window(const void* base, int64_t offset, bool there, uint32_t bytes)
{
    return make_rsrc(static_cast<const char*>(base) + offset, there ? bytes : 0u);
}

// ---------------------------------------------------------------- the gate

// The decay of one token and channel, as a value that gives both a and 1 - a to full
// precision: sigmoid(-|g|) is the smaller of the two, its sign says which.
struct Decay {
    float u;
    __device__ __forceinline__ float keep(int gating) const
    {
        return gating != GATE_SIGMOID ? u : (u > 0.0f ? 1.0f - u : -u);
    }
};

__device__ __forceinline__ float gate_exp(float g) { return __builtin_amdgcn_exp2f(g * 1.44269504088896340736f); }

__device__ __forceinline__ void sigmoid_both(float g, float& a, float& rest)
{
    const float e = gate_exp(-__builtin_fabsf(g));
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    a = g >= 0.0f ? big : small;
    rest = g >= 0.0f ? small : big;
}

// a, and b = what the token puts in.
template <class E, int CPL>
__device__ __forceinline__ void token_maps(int gating, const uint32_t (&rx)[RC_ROWS], const uint32_t (&rg)[RC_ROWS],
                                           float (&a)[RC_ROWS][CPL], float (&b)[RC_ROWS][CPL])
{
#pragma unroll
    for (int j = 0; j < RC_ROWS; ++j) {
        E::unpack(rx[j], b[j]);
        E::unpack(rg[j], a[j]);
    }
    if (gating == GATE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j)
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                float rest;
                sigmoid_both(a[j][c], a[j][c], rest);
                b[j][c] *= rest;
            }
    } else if (gating == GATE_LOG) {
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j)
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                a[j][c] = gate_exp(a[j][c]);
    }
}

// ---------------------------------------------------------------- packed rows

// First s in [0, n) with offsets[s + 1] > row (n: none), the whole wave together: 64 probes a round.
__device__ __forceinline__ int64_t sequence_of_row(const int64_t* offsets, int64_t n, int64_t row, int lane)
{
    int64_t lo = 0, hi = n;  // the answer is in [lo, hi]
    while (hi - lo > 0) {
        const int64_t step = (hi - lo + 63) / 64;
        const int64_t at = lo + lane * step;
        const bool past = at < hi && offsets[at + 1] > row;
        const uint64_t found = __ballot(past);
        if (found == 0) {
            // the last probe in range stands before the answer
            const int64_t last = lo + (hi - 1 - lo) / step * step;
            lo = last + 1;
        } else {
            const int first = __builtin_ctzll(found);
            hi = lo + first * step;
            lo = first == 0 ? lo : lo + (first - 1) * step + 1;
        }
    }
    return lo;
}

// For each row of the tile the sequence that starts there and the one that ends there, or -1.
// Offsets out of order mark wrong rows, never ones outside the tile.
__device__ __forceinline__ void mark_rows(const int64_t* offsets, int64_t sequences, int64_t row0, int rows, int (&heads)[RC_TILE],
                                          int (&ends)[RC_TILE], int lane)
{
    const int tid = threadIdx.x, threads = blockDim.x;
    for (int i = tid; i < rows; i += threads)
        heads[i] = ends[i] = -1;
    const int64_t first = sequence_of_row(offsets, sequences, row0, lane);
    __syncthreads();
    for (int64_t s = first + tid; s < sequences; s += threads) {
        const int64_t from = offsets[s], to = offsets[s + 1];
        if (from >= row0 + rows)
            break;
        if (to > from) {
            if (from >= row0)
                heads[from - row0] = int(s);
            if (to > row0 && to <= row0 + rows)
                ends[to - 1 - row0] = int(s);
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- forward

// A wave's composed map (or, behind a sequence's start, the value itself).
template <int CPL>
struct alignas(8 * CPL) WaveMap {
    float a[CPL], h[CPL];
};

template <class E, int CPL, bool PACKED>
__global__ __launch_bounds__(RC_WAVES * 64) void recur_forward_kernel(RecurForward q)
{
    constexpr int CH = 64 * CPL;
    __shared__ WaveMap<CPL> maps[2][RC_WAVES][64];
    __shared__ int restart[2][RC_WAVES];
    __shared__ int head_seq[PACKED ? RC_TILE : 1], end_seq[PACKED ? RC_TILE : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int tile_rows = waves * RC_ROWS;
    const int64_t groups = (q.channels + CH - 1) / CH;
    const int64_t chain = blockIdx.x / groups, c0 = (blockIdx.x % groups) * CH;
    const uint32_t here = uint32_t(q.channels - c0 < CH ? q.channels - c0 : CH);  // channels of this block
    const uint32_t bytes = here * E::size, state_bytes = here * 4;
    const uint32_t voff = lane * CPL * E::size;
    int64_t rows = q.rows;
    if constexpr (PACKED) {
        const int64_t live = q.offsets[q.sequences];
        rows = live < 0 ? 0 : live < rows ? live : rows;
    }
    const char* x = static_cast<const char*>(q.x) + (chain * q.x_sequence + c0) * E::size;
    const char* g = static_cast<const char*>(q.gate) + (chain * q.gate_sequence + c0) * E::size;
    const char* out = static_cast<const char*>(q.out) + (chain * q.out_sequence + c0) * E::size;
    const int64_t x_row = q.x_row * E::size, g_row = q.gate_row * E::size, out_row = q.out_row * E::size;
    const int64_t periods = (q.rows + RC_PERIOD - 1) / RC_PERIOD;

    uint32_t rx[RC_ROWS], rg[RC_ROWS];
    auto load_rows = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j) {
            rx[j] = load_part<E, CPL>(row_window(x, (row + j) * x_row, row + j < rows, bytes), voff);
            rg[j] = load_part<E, CPL>(row_window(g, (row + j) * g_row, row + j < rows, bytes), voff);
        }
    };

    float carry[CPL] = {};
    if (!PACKED && q.state != nullptr)
        load_state<CPL>(make_rsrc(q.state + chain * q.state_row + c0, state_bytes), lane, carry);
    load_rows(wave * RC_ROWS);
    int turn = 0;
    for (int64_t row0 = 0; row0 < rows; row0 += tile_rows, turn ^= 1) {
        const int64_t row = row0 + wave * RC_ROWS;
        float a[RC_ROWS][CPL], b[RC_ROWS][CPL];
        token_maps<E, CPL>(q.gating, rx, rg, a, b);
        if (row0 + tile_rows < rows)
            load_rows(row + tile_rows);
        if (row + RC_ROWS > rows) {
#pragma unroll
            for (int j = 0; j < RC_ROWS; ++j)
                if (row + j >= rows) {
#pragma unroll
                    for (int c = 0; c < CPL; ++c) {
                        a[j][c] = 1.0f;
                        b[j][c] = 0.0f;
                    }
                }
        }
        uint32_t heads = 0, ends = 0;
        int hs = -1, es = -1;
        if constexpr (PACKED) {
            mark_rows(q.offsets, q.sequences, row0, tile_rows, head_seq, end_seq, lane);
            hs = head_seq[wave * RC_ROWS + lane % RC_ROWS];
            es = end_seq[wave * RC_ROWS + lane % RC_ROWS];
            heads = uint32_t(__ballot(lane < RC_ROWS && hs >= 0));
            ends = uint32_t(__ballot(lane < RC_ROWS && es >= 0));
            if (heads != 0 && q.state != nullptr) {
                float h0[RC_ROWS][CPL];
#pragma unroll
                for (int j = 0; j < RC_ROWS; ++j) {
                    const bool head = (heads >> j) & 1;
                    const int64_t s = head ? read_lane(hs, j) : 0;
                    load_state<CPL>(row_window(q.state + c0, s * q.state_row * 4, head, state_bytes), lane, h0[j]);
                }
#pragma unroll
                for (int j = 0; j < RC_ROWS; ++j)
                    if ((heads >> j) & 1) {
#pragma unroll
                        for (int c = 0; c < CPL; ++c)
                            b[j][c] = __builtin_fmaf(a[j][c], h0[j][c], b[j][c]);
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
        for (int j = 0; j < RC_ROWS; ++j) {
            const bool head = PACKED && ((heads >> j) & 1);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                if (head)
                    m.h[c] = 0.0f;
                m.h[c] = __builtin_fmaf(a[j][c], m.h[c], b[j][c]);
                m.a[c] *= a[j][c];
            }
        }
        maps[turn][wave][lane] = m;
        if (PACKED && lane == 0)
            restart[turn][wave] = heads != 0;
        __syncthreads();
        float h[CPL];
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
        if (q.carries != nullptr && row < rows && row % RC_PERIOD == 0)
            store_state<CPL>(make_rsrc(q.carries + (chain * periods + row / RC_PERIOD) * q.channels + c0, state_bytes), lane, h);
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j) {
            const bool head = PACKED && ((heads >> j) & 1);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                h[c] = __builtin_fmaf(a[j][c], head ? 0.0f : h[c], b[j][c]);
            store_part<E, CPL>(row_window(out, (row + j) * out_row, row + j < rows, bytes), voff, h);
            if (PACKED && ((ends >> j) & 1))
                store_state<CPL>(make_rsrc(q.state_out + read_lane(es, j) * q.state_out_row + c0, state_bytes), lane, h);
        }
    }
    if (!PACKED) {
        if (wave == 0)
            store_state<CPL>(make_rsrc(q.state_out + chain * q.state_out_row + c0, state_bytes), lane, carry);
    } else if (q.state != q.state_out) {
        for (int64_t s = wave; s < q.sequences; s += waves)
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

template <class E, int CPL, bool PACKED>
__global__ __launch_bounds__(RC_WAVES * 64) void recur_backward_kernel(RecurBackward q)
{
    constexpr int CH = 64 * CPL;
    __shared__ WaveBack<CPL> maps[2][RC_WAVES][64];
    __shared__ int restart[2][RC_WAVES][2];
    __shared__ int head_seq[PACKED ? RC_TILE : 1], end_seq[PACKED ? RC_TILE : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int tile_rows = waves * RC_ROWS;
    const int64_t groups = (q.channels + CH - 1) / CH;
    const int64_t chain = blockIdx.x / groups, c0 = (blockIdx.x % groups) * CH;
    const uint32_t here = uint32_t(q.channels - c0 < CH ? q.channels - c0 : CH);
    const uint32_t bytes = here * E::size, state_bytes = here * 4;
    const uint32_t voff = lane * CPL * E::size;
    int64_t rows = q.rows;
    if constexpr (PACKED) {
        const int64_t live = q.offsets[q.sequences];
        rows = live < 0 ? 0 : live < rows ? live : rows;
    }
    const char* x = static_cast<const char*>(q.x) + (chain * q.x_sequence + c0) * E::size;
    const char* g = static_cast<const char*>(q.gate) + (chain * q.gate_sequence + c0) * E::size;
    const char* dout = static_cast<const char*>(q.dout) + (chain * q.dout_sequence + c0) * E::size;
    const char* dx = static_cast<const char*>(q.dx) + (chain * q.dx_sequence + c0) * E::size;
    const char* dg = static_cast<const char*>(q.dgate) + (chain * q.dgate_sequence + c0) * E::size;
    const int64_t periods = (q.rows + RC_PERIOD - 1) / RC_PERIOD;

    float mu_carry[CPL] = {};
    if (!PACKED && q.dstate_out != nullptr)
        load_state<CPL>(make_rsrc(q.dstate_out + chain * q.dstate_out_row + c0, state_bytes), lane, mu_carry);
    int turn = 0;
    const int64_t last0 = rows > 0 ? (rows - 1) / tile_rows * tile_rows : -1;
    for (int64_t row0 = last0; row0 >= 0; row0 -= tile_rows, turn ^= 1) {
        const int64_t row = row0 + wave * RC_ROWS;
        uint32_t rx[RC_ROWS], rg[RC_ROWS], rd[RC_ROWS];
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j) {
            const bool there = row + j < rows;
            rx[j] = load_part<E, CPL>(row_window(x, (row + j) * q.x_row * E::size, there, bytes), voff);
            rg[j] = load_part<E, CPL>(row_window(g, (row + j) * q.gate_row * E::size, there, bytes), voff);
            rd[j] = load_part<E, CPL>(row_window(dout, (row + j) * q.dout_row * E::size, there, bytes), voff);
        }
        // h in front of the wave's period
        float h[CPL];
        const int64_t period = row / RC_PERIOD;
        load_state<CPL>(row_window(q.carries + c0, (chain * periods + period) * q.channels * 4, row < rows, state_bytes), lane, h);
        uint32_t heads = 0, ends = 0;
        int hs = -1, es = -1;
        if constexpr (PACKED) {
            mark_rows(q.offsets, q.sequences, row0, tile_rows, head_seq, end_seq, lane);
            hs = head_seq[wave * RC_ROWS + lane % RC_ROWS];
            es = end_seq[wave * RC_ROWS + lane % RC_ROWS];
            heads = uint32_t(__ballot(lane < RC_ROWS && hs >= 0));
            ends = uint32_t(__ballot(lane < RC_ROWS && es >= 0));
        }
        auto state_of = [&](int j, float (&v)[CPL]) {
            const int64_t s = read_lane(hs, j);
            load_state<CPL>(row_window(q.state + c0, s * q.state_row * 4, q.state != nullptr, state_bytes), lane, v);
        };
        auto gradient_of = [&](int j, float (&v)[CPL]) {
            const int64_t s = read_lane(es, j);
            load_state<CPL>(row_window(q.dstate_out + c0, s * q.dstate_out_row * 4, q.dstate_out != nullptr, state_bytes), lane, v);
        };

        // the decays, with 1 - a to full precision too (see Decay)
        Decay decay[RC_ROWS][CPL];
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j) {
            float gv[CPL];
            E::unpack(rg[j], gv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                float u = gv[c];
                if (q.gating == GATE_SIGMOID) {
                    const float e = gate_exp(-__builtin_fabsf(u));
                    const float small = e * __builtin_amdgcn_rcpf(1.0f + e);
                    // a gate so far out that the smaller one is 0 keeps its side
                    u = u >= 0.0f ? __builtin_fmaxf(small, 1e-38f) : -small;
                    if (gv[c] != gv[c])
                        u = gv[c];
                } else if (q.gating == GATE_LOG) {
                    u = gate_exp(u);
                }
                decay[j][c].u = row + j < rows ? u : (q.gating == GATE_SIGMOID ? 1e-38f : 1.0f);
            }
        }
        WaveBack<CPL> m;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            m.a[c] = 1.0f;
            m.h[c] = 0.0f;
            m.mu[c] = 0.0f;
        }
        const bool sigmoid = q.gating == GATE_SIGMOID;
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j) {
            if (PACKED && ((heads >> j) & 1))
                state_of(j, m.h);
            float xv[CPL];
            E::unpack(rx[j], xv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const float a = decay[j][c].keep(q.gating), u = decay[j][c].u;
                const float rest = sigmoid ? (u > 0.0f ? u : 1.0f + u) : 1.0f;
                m.h[c] = __builtin_fmaf(a, m.h[c], rest * xv[c]);
                m.a[c] *= a;
            }
        }
#pragma unroll
        for (int j = RC_ROWS - 1; j >= 0; --j) {
            if (PACKED && ((ends >> j) & 1))
                gradient_of(j, m.mu);
            float dv[CPL];
            E::unpack(rd[j], dv);
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                m.mu[c] = decay[j][c].keep(q.gating) * (dv[c] + m.mu[c]);
        }
        maps[turn][wave][lane] = m;
        if (PACKED && lane == 0) {
            restart[turn][wave][0] = heads != 0;
            restart[turn][wave][1] = ends != 0;
        }
        __syncthreads();
        // h in front of the wave, from its period's carry
        constexpr int PER = RC_PERIOD / RC_ROWS;
        for (int i = wave / PER * PER; i < wave; ++i) {
            const WaveBack<CPL> o = maps[turn][i][lane];
            const bool again = PACKED && __builtin_amdgcn_readfirstlane(restart[turn][i][0]) != 0;
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                h[c] = again ? o.h[c] : __builtin_fmaf(o.a[c], h[c], o.h[c]);
        }
        float mu[CPL];
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
        float before[RC_ROWS][CPL];
#pragma unroll
        for (int j = 0; j < RC_ROWS; ++j) {
            if (PACKED && ((heads >> j) & 1))
                state_of(j, h);
            float xv[CPL];
            E::unpack(rx[j], xv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                before[j][c] = h[c];
                const float a = decay[j][c].keep(q.gating), u = decay[j][c].u;
                const float rest = sigmoid ? (u > 0.0f ? u : 1.0f + u) : 1.0f;
                h[c] = __builtin_fmaf(a, h[c], rest * xv[c]);
            }
        }
#pragma unroll
        for (int j = RC_ROWS - 1; j >= 0; --j) {
            if (PACKED && ((ends >> j) & 1))
                gradient_of(j, mu);
            float dv[CPL], xv[CPL], gx[CPL], gg[CPL];
            E::unpack(rd[j], dv);
            E::unpack(rx[j], xv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const float a = decay[j][c].keep(q.gating), u = decay[j][c].u;
                const float rest = sigmoid ? (u > 0.0f ? u : 1.0f + u) : 1.0f;
                const float lam = dv[c] + mu[c];
                mu[c] = a * lam;
                gx[c] = lam * rest;
                gg[c] = sigmoid ? gx[c] * a * (before[j][c] - xv[c]) : (q.gating == GATE_LOG ? mu[c] : lam) * before[j][c];
            }
            const bool there = row + j < rows;
            store_part<E, CPL>(row_window(dx, (row + j) * q.dx_row * E::size, there, bytes), voff, gx);
            store_part<E, CPL>(row_window(dg, (row + j) * q.dgate_row * E::size, there, bytes), voff, gg);
            if (PACKED && ((heads >> j) & 1))
                store_state<CPL>(make_rsrc(q.dstate + read_lane(hs, j) * q.dstate_row + c0, state_bytes), lane, mu);
        }
    }
    if (!PACKED) {
        if (wave == 0)
            store_state<CPL>(make_rsrc(q.dstate + chain * q.dstate_row + c0, state_bytes), lane, mu_carry);
    } else {
        for (int64_t s = wave; s < q.sequences; s += waves)
            if (q.offsets[s + 1] <= q.offsets[s]) {
                float v[CPL] = {};
                if (q.dstate_out != nullptr)
                    load_state<CPL>(make_rsrc(q.dstate_out + s * q.dstate_out_row + c0, state_bytes), lane, v);
                store_state<CPL>(make_rsrc(q.dstate + s * q.dstate_row + c0, state_bytes), lane, v);
            }
    }
}

// ---------------------------------------------------------------- one token a sequence

// VEC neighbouring channels per thread: 16 bytes of x, or one element where rows are not aligned.
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

size_t recur_workspace_bytes(int64_t, int64_t rows, int64_t, bool packed, int)
{
    return packed || rows > 1 ? sizeof(WsHeader) : 0;
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

int waves_for(int64_t rows, int least)
{
    int w = RC_WAVES;
    while (w > least && (w / 2) * RC_ROWS >= rows)
        w /= 2;
    return w;
}

// A launch holds less than 2^32 threads: most sequences of a launch of `groups` blocks each.
int64_t sequences_at_once(int64_t groups) { return (int64_t(1) << 22) / groups > 0 ? (int64_t(1) << 22) / groups : 1; }

template <class E, int CPL>
hipError_t launch_forward(const RecurForward& q, hipStream_t stream)
{
    const int64_t groups = (q.channels + 64 * CPL - 1) / (64 * CPL), most = sequences_at_once(groups);
    if (q.offsets == nullptr && q.sequences > most) {
        RecurForward first = q, rest = q;
        first.sequences = most;
        rest.sequences -= most;
        rest.x = static_cast<const char*>(q.x) + most * q.x_sequence * E::size;
        rest.gate = static_cast<const char*>(q.gate) + most * q.gate_sequence * E::size;
        rest.out = static_cast<char*>(q.out) + most * q.out_sequence * E::size;
        if (q.state != nullptr)
            rest.state += most * q.state_row;
        rest.state_out += most * q.state_out_row;
        if (q.carries != nullptr)
            rest.carries += recur_carry_rows(most, q.rows, false) * q.channels;
        const hipError_t e = launch_forward<E, CPL>(first, stream);
        return e != hipSuccess ? e : launch_forward<E, CPL>(rest, stream);
    }
    const int64_t blocks = (q.offsets ? 1 : q.sequences) * groups;
    const dim3 threads(64 * waves_for(q.rows, 1));
    if (q.offsets)
        recur_forward_kernel<E, CPL, true><<<dim3(uint32_t(blocks)), threads, 0, stream>>>(q);
    else
        recur_forward_kernel<E, CPL, false><<<dim3(uint32_t(blocks)), threads, 0, stream>>>(q);
    return hipGetLastError();
}

template <class E, int CPL>
hipError_t launch_backward(const RecurBackward& q, hipStream_t stream)
{
    const int64_t groups = (q.channels + 64 * CPL - 1) / (64 * CPL), most = sequences_at_once(groups);
    if (q.offsets == nullptr && q.sequences > most) {
        RecurBackward first = q, rest = q;
        first.sequences = most;
        rest.sequences -= most;
        rest.dout = static_cast<const char*>(q.dout) + most * q.dout_sequence * E::size;
        rest.x = static_cast<const char*>(q.x) + most * q.x_sequence * E::size;
        rest.gate = static_cast<const char*>(q.gate) + most * q.gate_sequence * E::size;
        rest.dx = static_cast<char*>(q.dx) + most * q.dx_sequence * E::size;
        rest.dgate = static_cast<char*>(q.dgate) + most * q.dgate_sequence * E::size;
        if (q.state != nullptr)
            rest.state += most * q.state_row;
        if (q.dstate_out != nullptr)
            rest.dstate_out += most * q.dstate_out_row;
        rest.dstate += most * q.dstate_row;
        rest.carries += recur_carry_rows(most, q.rows, false) * q.channels;
        const hipError_t e = launch_backward<E, CPL>(first, stream);
        return e != hipSuccess ? e : launch_backward<E, CPL>(rest, stream);
    }
    const int64_t blocks = (q.offsets ? 1 : q.sequences) * groups;
    const dim3 threads(64 * waves_for(q.rows, RC_PERIOD / RC_ROWS));
    if (q.offsets)
        recur_backward_kernel<E, CPL, true><<<dim3(uint32_t(blocks)), threads, 0, stream>>>(q);
    else
        recur_backward_kernel<E, CPL, false><<<dim3(uint32_t(blocks)), threads, 0, stream>>>(q);
    return hipGetLastError();
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

}  // namespace

hipError_t launch_recurrence(const RecurForward& q, int type, void*, hipStream_t stream)
{
    if (q.sequences == 0 || q.channels == 0)
        return hipSuccess;
    if (q.offsets == nullptr && q.rows == 1) {
        if (type == LOGITS_F32)
            return launch_step<F32>(q, stream);
        return type == LOGITS_F16 ? launch_step<F16>(q, stream) : launch_step<BF16>(q, stream);
    }
    if (type == LOGITS_F32)
        return launch_forward<F32, 1>(q, stream);
    const bool pairs = q.channels % 2 == 0 && multiples(q.x, q.x_sequence * 2, q.x_row * 2, 4) &&
                       multiples(q.gate, q.gate_sequence * 2, q.gate_row * 2, 4) && multiples(q.out, q.out_sequence * 2, q.out_row * 2, 4);
    if (type == LOGITS_F16)
        return pairs ? launch_forward<F16, 2>(q, stream) : launch_forward<F16, 1>(q, stream);
    return pairs ? launch_forward<BF16, 2>(q, stream) : launch_forward<BF16, 1>(q, stream);
}

hipError_t launch_recurrence_backward(const RecurBackward& q, int type, void*, hipStream_t stream)
{
    if (q.sequences == 0 || q.channels == 0)
        return hipSuccess;
    if (type == LOGITS_F32)
        return launch_backward<F32, 1>(q, stream);
    const bool pairs = q.channels % 2 == 0 && multiples(q.x, q.x_sequence * 2, q.x_row * 2, 4) &&
                       multiples(q.gate, q.gate_sequence * 2, q.gate_row * 2, 4) &&
                       multiples(q.dout, q.dout_sequence * 2, q.dout_row * 2, 4) &&
                       multiples(q.dx, q.dx_sequence * 2, q.dx_row * 2, 4) &&
                       multiples(q.dgate, q.dgate_sequence * 2, q.dgate_row * 2, 4);
    if (type == LOGITS_F16)
        return pairs ? launch_backward<F16, 2>(q, stream) : launch_backward<F16, 1>(q, stream);
    return pairs ? launch_backward<BF16, 2>(q, stream) : launch_backward<BF16, 1>(q, stream);
}

}  // namespace ls
