// The marks of a tile's rows (ls_marks.hpp) run on the CPU: a block's threads are fibers, a wave's lanes meet in
// __ballot.  Offsets are read through a type that checks every index and counts the reads.
//
//     row_marks_model <sequences> <row0> <rows> <threads>  < offsets (int64)
// prints the reads of the busiest lane, then "row head end" for each row of the tile that has either.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <ucontext.h>
#include <vector>

#define __device__
#define __forceinline__ inline

struct Dim {
    unsigned x;
};
static Dim threadIdx, blockDim;

struct Fiber {
    ucontext_t at;
    std::vector<char> stack;
    bool done = false, asks = false, says = false;
    long reads = 0;
};
static std::vector<Fiber> fibers;
static std::vector<uint64_t> answer;  // of each wave's last ballot
static ucontext_t scheduler;
static unsigned running;

static uint64_t __ballot(bool v)
{
    Fiber& f = fibers[running];
    f.asks = true;
    f.says = v;
    swapcontext(&f.at, &scheduler);
    return answer[running / 64];
}

static std::vector<int64_t> values;
struct Offsets {
    int64_t operator[](int64_t i) const
    {
        if (i < 0 || i >= int64_t(values.size())) {
            std::printf("read at %lld of %zu offsets\n", (long long)i, values.size());
            std::exit(3);
        }
        ++fibers[running].reads;
        return values[size_t(i)];
    }
};

#include "ls_marks.hpp"

constexpr int TILE = 128;
static struct Guarded {
    int before[64], heads[TILE], between[64], ends[TILE], behind[64];
} marks;
static int64_t sequences, row0;
static int rows;

static void thread_main()
{
    {
        ls::RowMarks<Offsets> m(Offsets{}, sequences, marks.heads, marks.ends);
        __ballot(false);  // stands for the barrier in between
        m.mark(Offsets{}, sequences, row0, rows, marks.heads, marks.ends, int(threadIdx.x & 63));
    }
    fibers[running].done = true;
    swapcontext(&fibers[running].at, &scheduler);
}

static void run(unsigned i)
{
    running = i;
    threadIdx.x = i;
    swapcontext(&scheduler, &fibers[i].at);
}

int main(int, char** argv)
{
    sequences = std::atoll(argv[1]);
    row0 = std::atoll(argv[2]);
    rows = std::atoi(argv[3]);
    blockDim.x = unsigned(std::atoi(argv[4]));
    values.resize(size_t(sequences) + 1);
    if (std::fread(values.data(), 8, values.size(), stdin) != values.size())
        return 2;
    for (int i = 0; i < 64; ++i)
        marks.before[i] = marks.between[i] = marks.behind[i] = 77;
    fibers.resize(blockDim.x);
    answer.resize(blockDim.x / 64);
    for (Fiber& f : fibers) {
        f.stack.resize(1 << 16);
        getcontext(&f.at);
        f.at.uc_stack.ss_sp = f.stack.data();
        f.at.uc_stack.ss_size = f.stack.size();
        f.at.uc_link = nullptr;
        makecontext(&f.at, thread_main, 0);
    }
    // the whole block up to the barrier, then its waves in turn, a ballot after the other
    for (unsigned i = 0; i < blockDim.x; ++i)
        run(i);
    for (unsigned wave = 0; wave < blockDim.x / 64; ++wave)
        for (;;) {
            unsigned done = 0, asks = 0;
            uint64_t word = 0;
            for (unsigned l = 0; l < 64; ++l) {
                Fiber& f = fibers[wave * 64 + l];
                done += f.done;
                asks += f.asks;
                word |= uint64_t(f.asks && f.says) << l;
                f.asks = false;
            }
            if (done == 64)
                break;
            if (asks != 64) {
                std::printf("wave %u: %u lanes in a ballot, %u ended\n", wave, asks, done);
                return 4;
            }
            answer[wave] = word;
            for (unsigned l = 0; l < 64; ++l)
                run(wave * 64 + l);
        }
    long most = 0;
    for (const Fiber& f : fibers)
        most = f.reads > most ? f.reads : most;
    for (int i = 0; i < 64; ++i)
        if (marks.before[i] != 77 || marks.between[i] != 77 || marks.behind[i] != 77) {
            std::printf("a mark outside the tile\n");
            return 5;
        }
    std::printf("%ld\n", most);
    for (int i = 0; i < TILE; ++i)
        if (marks.heads[i] != -1 || marks.ends[i] != -1)
            std::printf("%d %d %d\n", i, marks.heads[i], marks.ends[i]);
    return 0;
}
