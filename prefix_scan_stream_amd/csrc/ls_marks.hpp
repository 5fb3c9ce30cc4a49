// ls_marks.hpp -- where the sequences of packed rows begin and end in a tile of rows (gfx950).
// Offsets may be any pointer-like type that is indexed.
#pragma once
#include <stdint.h>

namespace ls {

// First s in [0, n) with offsets[s + 1] > row (n: none), the whole wave together: 64 probes a round.
template <class P>
__device__ __forceinline__ int64_t sequence_of_row(P offsets, int64_t n, int64_t row, int lane)
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

// For each row of a tile the sequence that starts there and the one that ends there, or -1.  Where the block has a
// thread for each sequence, its offsets are on their way before the tile is known; with more sequences they are searched
// for the tile's first.  Offsets out of order mark wrong rows, never ones outside the tile.
// Empty sequences stand at a row in any number, and a block goes over them at its threads' number a round: a wave
// that saw only such ones EMPTY_ROUNDS times searches for the next that is not.  2^30 of them would else hold the
// tile, and those that wait for it, for more than the second that a wait may last.
constexpr int EMPTY_ROUNDS = 16;

template <class P>
struct RowMarks {
    int64_t from, to;
    template <int TILE>
    __device__ __forceinline__ RowMarks(P offsets, int64_t sequences, int (&heads)[TILE], int (&ends)[TILE]) : from(0), to(0)
    {
        if (threadIdx.x < sequences) {
            from = offsets[threadIdx.x];
            to = offsets[threadIdx.x + 1];
        }
        for (int i = threadIdx.x; i < TILE; i += blockDim.x)
            heads[i] = ends[i] = -1;
    }
    // Between two barriers.
    template <int TILE>
    __device__ __forceinline__ void mark(P offsets, int64_t sequences, int64_t row0, int rows, int (&heads)[TILE], int (&ends)[TILE],
                                         int lane)
    {
        const int tid = threadIdx.x, threads = blockDim.x;
        int64_t s = tid;
        if (sequences > threads) {
            s += sequence_of_row(offsets, sequences, row0, lane);
            if (s < sequences) {
                from = offsets[s];
                to = offsets[s + 1];
            }
        }
        for (int idle = 0;;) {
            const bool in = s < sequences && from < row0 + rows, holds = in && to > from;
            if (__ballot(in) == 0)
                return;
            if (holds && from >= row0)
                heads[from - row0] = int(s);
            if (holds && to > row0 && to <= row0 + rows)
                ends[to - 1 - row0] = int(s);
            idle = __ballot(holds) == 0 ? idle + 1 : 0;
            s += threads;
            if (idle == EMPTY_ROUNDS) {
                // what follows lane 0's last one up to the first sequence that ends behind its row is empty, too
                const int64_t first = s - lane;
                const int64_t next = sequence_of_row(offsets, sequences, offsets[first - threads], lane);
                s += next > first ? (next - first) / threads * threads : 0;
                idle = 0;
            }
            if (s < sequences) {
                from = offsets[s];
                to = offsets[s + 1];
            }
        }
    }
};

}  // namespace ls
