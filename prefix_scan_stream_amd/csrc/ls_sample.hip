// ls_sample.hip -- one token from each row of logits (gfx950).
//
// A row x of V logits, its largest value M, a temperature t:
//   w_i = exp((x_i - M) / t), the weight of token i; NaN counts as -inf, weight 0.
//   The order of tokens is by x descending, equal ones by index ascending.
//   top-k keeps the first k of that order; Z_k is their weight.
//   top-p keeps, of those, each whose weight before it is below p Z_k (the first always).
//   min-p keeps, of those, each with w_i >= min(1, min_p).
// Each cut keeps a prefix of the order, so the kept set is all elements up to one
// (value, index) pair, the cut.  The token is the first index, in index order, at which
// the running sum of the kept weights exceeds u Z (u the row's random number, Z the kept
// weight); its log-probability is (x - M)/t - ln Z.
//
// Neighbouring sums of a row lie about 2^-17 Z apart and u has 24 bits, so sums in 32
// bits would pick another token in some percents of the rows.  Weights and sums are in
// 64 bits: a double multiply-add issues at the rate of a single one here (5.5 cycles a
// wave and SIMD against 5.3, measured), and 2^f is a polynomial: of degree 10 where single
// weights count (exp2_poly, 2^-50.6), of degree 9 in the sums of a whole row (exp2_sum4,
// 2^-44.6), of degree 6 in the bins (fill_bins, 2^-48.9).  The bins' integers round more than that:
// to 2^-44.06 of a weight in rows of up to 2^17, and a bit more for each doubling (make_row).
//
// One launch.  A row is cut into segments, and its segments are shared out to blocks, so
// that few rows still use the whole GPU.  Every block leaves what its segments hold in
// the workspace; the block of a row that arrives last at the row's counter goes on alone.
//   No cuts (sample_all_kernel): the segments hold the sum of their weights, relative to a
//   value of theirs.  The last block has the running sums of the segments, so it knows the
//   one the token lies in, and reads only that again.
//   Cuts (sample_cut_kernel): the segments hold the largest values of their quarters.  The
//   k-th largest of the segments' values is at most the k-th largest logit, so for a small
//   k the candidates are the elements at or above it, which lie in a few more than k quarters:
//   these are read again and ordered in LDS.  min-p alone has its threshold from M the
//   same way.  Otherwise the cut is found by value without sorting the row (cut_row).
//
// Measured, in a graph, 131072 logits to a row:
//   1 row, bfloat16, top-k 50, top-p, min-p: 12.4 us, the latency of the chain of steps: 2 us the launch, 2 the
//   first read, 1 the counter, 4.5 the row's parameters (loaded one after the other) and one wave's search for the
//   candidates' quarters, 2 their reading, 3 order and sums.  64 rows, top-k 100, top-p, min-p: 15.6 us.
//   256 rows, bfloat16, top-p alone: 66 us, a row to a CU: 11 us the first read (6 TB/s over all), 25 the bins
//   (16.5 vector instructions a logit), 14 the bin's elements, the rest the steps between.
//   64 rows of flat logits (normal, a deviation of 0.5), top-p: 83 us, with two more readings for a bin of 13000.
//   512 rows, no cuts: bfloat16 and float16 51 us, bound by vector instructions (21 a logit by the counters, 47 us at
//   the measured rate); float32 57-62 us, 20 a logit with 268 MB to read beside them (4.3-4.7 TB/s).
#include <type_traits>

#include "ls_wave64.hpp"
#include "ls_internal.hpp"

namespace ls {

constexpr int SM_BLOCK = 1024;              // threads of a block that makes cuts
constexpr int SM_WAVES = SM_BLOCK / 64;
constexpr int SM_ALL_BLOCK = 256;           // without cuts
constexpr int SM_VEC = 8;                   // consecutive logits per lane and step
constexpr int SM_STEP = 64 * SM_VEC;        // consecutive logits per wave and step
constexpr int SM_PER_LANE = 8;              // segments of a row that one lane of a wave takes
constexpr int SM_SEGS = 64 * SM_PER_LANE;   // most segments of a row
constexpr int SM_PER_OCTAVE = 8;            // bins per halving of the weight
constexpr int SM_BINS = 512;
constexpr int SM_RANGES = 256;              // ranges of a refinement
constexpr int SM_LIST = 4096;               // elements of one bin kept in LDS
constexpr int SM_NOTES = 256;               // loads of one wave that hold such elements
constexpr int SM_SMALL = 512;               // elements that are ordered by counting
// More than these of a bin are divided by value once more before that, since counting takes the square
// of their number (512: 12 us, one division 3).  Top-p alone, 4 rows of 32000: 26.1 us with 64 or 128,
// 26.3 with 256, 38.5 with 512; 131072: 53.7, 50.6, 50.0, 48.8.
constexpr int SM_FEW = 256;
constexpr int SM_CUS = 256;                 // of an MI355X
constexpr int SM_ROWS = 4096;               // most rows of a launch
constexpr int SM_COUNTER = 32;              // 32-bit words from one row's counter to the next
// Most rows, and least steps of a row, for its bins to be made by SM_WAVES blocks in a launch of their
// own (sample_bins_kernel), which costs about 8 us and divides the bins' time by the waves.  Top-p alone,
// bfloat16, with it against without: 131072 logits 1 row 40.2 against 49.8 us, 32 rows 44.0 against 50.9,
// 64 rows 51.7 both, 128 rows 72 against 55; 64000 logits 1 row 31.5 against 32.8, 32 rows 34.4
// against 33.8; 32000 logits 1 row 27.8 against 25.7.
constexpr int SM_SPLIT_ROWS = 32;
constexpr int DPP_QUAD_SWAP1 = 0xb1, DPP_QUAD_SWAP2 = 0x4e;  // each lane of four its neighbour's value, the other pair's
constexpr int SM_FINE_SEGS = 32;  // segments of a row up to which its largest values are kept by sixteenths too
constexpr int SM_SPLIT_STEPS = 128;

constexpr double LOG2E = 0x1.71547652b82fep+0, LN2 = 0x1.62e42fefa39efp-1;
constexpr double TO_INT = 0x1.8p52;  // adding it rounds to the nearest integer, into the low word

// 2^f for |f| <= 1/2: interpolates at Chebyshev nodes with p(0) = 1; its largest
// relative error is 2^-50.6.
__device__ __forceinline__ double exp2_poly(double f)
{
    double p = 0x1.e5e9f548e5725p-28;
    p = __builtin_fma(p, f, 0x1.b6571de2f2351p-24);
    p = __builtin_fma(p, f, 0x1.62bfe46117445p-20);
    p = __builtin_fma(p, f, 0x1.ffcb76789860fp-17);
    p = __builtin_fma(p, f, 0x1.4309130378460p-13);
    p = __builtin_fma(p, f, 0x1.5d87fe908f88ap-10);
    p = __builtin_fma(p, f, 0x1.3b2ab6fba385fp-7);
    p = __builtin_fma(p, f, 0x1.c6b08d7044119p-5);
    p = __builtin_fma(p, f, 0x1.ebfbdff82c590p-3);
    p = __builtin_fma(p, f, 0x1.62e42fefa39f7p-1);
    return __builtin_fma(p, f, 1.0);
}

// 2^(d c + e) for -1000 <= d c <= 1 and a small e, with the exponent added in the high word.
__device__ __forceinline__ double exp2_fast(double d, double c, int e = 0)
{
    const double t = __builtin_fma(d, c, TO_INT);
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    u32x2 p = __builtin_bit_cast(u32x2, exp2_poly(__builtin_fma(d, c, TO_INT - t)));
    const uint32_t n = uint32_t(__builtin_bit_cast(uint64_t, t)) + uint32_t(e);
    // one instruction, where the compiler made five of a 64-bit addition
    asm("v_lshl_add_u32 %0, %1, 20, %2" : "=v"(p.y) : "v"(n), "v"(p.y));
    return __builtin_bit_cast(double, p);
}

// The sum of 2^(x c - R) over four logits, for an integer R given as k = TO_INT - R: rounding x c + k leaves
// the exponent in the low word, and the fraction x c less its nearest integer is one multiply-add
// with no subtraction of a reference from x.  The polynomial has one degree less than
// exp2_poly's, its relative error is 2^-44.6.  Four side by side, as a multiply-add's result
// is ready some issues later.
__device__ __forceinline__ double exp2_sum4(const double (&x)[4], double c, double k)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    constexpr double C[10] = {1.0,
                              0x1.62e42fefa39efp-1,
                              0x1.ebfbdff823cedp-3,
                              0x1.c6b08d7047e52p-5,
                              0x1.3b2ab7181b755p-7,
                              0x1.5d87fe86fe88ep-10,
                              0x1.4308ac85aa947p-13,
                              0x1.ffcb9515a8016p-17,
                              0x1.63d136366db24p-20,
                              0x1.b63880a30e9ffp-24};
    double t[4], f[4], p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        t[i] = __builtin_fma(x[i], c, k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __builtin_fma(x[i], c, k - t[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = __builtin_fma(C[9], f[i], C[8]);
#pragma unroll
    for (int j = 7; j >= 0; --j) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = __builtin_fma(p[i], f[i], C[j]);
        __builtin_amdgcn_sched_barrier(0);
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u32x2 w = __builtin_bit_cast(u32x2, p[i]);
        asm("v_lshl_add_u32 %0, %1, 20, %2" : "=v"(w.y) : "v"(uint32_t(__builtin_bit_cast(uint64_t, t[i]))), "v"(w.y));
        sum += __builtin_bit_cast(double, w);
    }
    return sum;
}

// 2^y for y <= 0 (NaN counts as -inf), 0 below 2^-1074.
__device__ __forceinline__ double exp2_exact(double y)
{
    y = __builtin_fmax(y, -1100.0);
    const double n = __builtin_rint(y);
    return __builtin_ldexp(exp2_poly(y - n), int(n));
}

// A value that is the same in all lanes, as a scalar.
template <class T>
__device__ __forceinline__ T uniform(T v)
{
    if constexpr (sizeof(T) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(b));
        const uint32_t hi = __builtin_amdgcn_readfirstlane(uint32_t(b >> 32));
        return __builtin_bit_cast(T, (uint64_t(hi) << 32) | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
    }
}

// Order-preserving keys of the logits: larger value, larger key; -0 and 0 are one.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = to_bits(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return from_bits<float>((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
constexpr uint32_t KEY_NEG_INF = 0x007fffffu;

// ---------------------------------------------------------------- a row's logits
typedef uint32_t u32x4_by4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_by2 __attribute__((ext_vector_type(4), aligned(2)));

// Eight consecutive logits as loaded; what lies past the row's end is -inf.
template <int TYPE>
struct Raw {
    static constexpr int WORDS = TYPE == LOGITS_F32 ? 8 : 4;
    static constexpr uint32_t NEG = TYPE == LOGITS_F32 ? 0xff800000u : TYPE == LOGITS_F16 ? 0xfc00fc00u : 0xff80ff80u;
    uint32_t w[WORDS];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < WORDS; ++k)
            w[k] = NEG;
    }
    using E = typename std::conditional<TYPE == LOGITS_F32, uint32_t, uint16_t>::type;
    using V = typename std::conditional<TYPE == LOGITS_F32, u32x4_by4, u32x4_by2>::type;
    __device__ __forceinline__ void load_all(const E* p)
    {
#pragma unroll
        for (int k = 0; k < WORDS; k += 4) {
            const V a = *reinterpret_cast<const V*>(reinterpret_cast<const uint32_t*>(p) + k);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[k + j] = a[j];
        }
    }
    // Logits idx .. idx+7; rows start at any multiple of the element's size.
    __device__ __forceinline__ void load(const void* row, int64_t idx, int64_t vocab)
    {
        const E* p = static_cast<const E*>(row) + idx;
        if (idx + SM_VEC <= vocab) {
            load_all(p);
        } else {
            // the row's end: one element at a time, last first (a loop: this code stands at every load)
#pragma unroll 1
            for (int k = SM_VEC - 1; k >= 0; --k) {
                const uint32_t e = idx + k < vocab ? uint32_t(p[k]) : NEG & (E(~E(0)));
#pragma unroll
                for (int j = WORDS - 1; j > 0; --j)
                    w[j] = TYPE == LOGITS_F32 ? w[j - 1] : (w[j] << 16) | (w[j - 1] >> 16);
                w[0] = TYPE == LOGITS_F32 ? e : (w[0] << 16) | e;
            }
        }
    }
    // A lane's logits of one step.  Whether the step is whole is the same for all lanes, so that whole ones
    // take a scalar address and no test per lane.
    __device__ __forceinline__ void load_step(const void* row, int step, int64_t vocab)
    {
        const int64_t first = int64_t(step) * SM_STEP;
        if (first + SM_STEP <= vocab)
            load_all(static_cast<const E*>(row) + first + uint32_t(lane_id()) * SM_VEC);
        else
            load(row, first + lane_id() * SM_VEC, vocab);
    }
    __device__ __forceinline__ void unpack(float (&x)[SM_VEC], bool inf) const
    {
#pragma unroll
        for (int k = 0; k < SM_VEC; ++k)
            x[k] = at(k);
        if (inf) {
            asm volatile("");  // a branch: hardly any row comes here
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k)
                x[k] = x[k] == __builtin_inff() ? 0.0f : -__builtin_inff();
        }
    }
    __device__ __forceinline__ float at(int k) const
    {
        if constexpr (TYPE == LOGITS_F32)
            return from_bits<float>(w[k]);
        else if constexpr (TYPE == LOGITS_BF16)
            return from_bits<float>(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
        else
            return float(__builtin_bit_cast(_Float16, uint16_t(k % 2 ? w[k / 2] >> 16 : w[k / 2])));
    }
};

// Where the row's largest value is +inf (`inf`), its elements are +inf or not: 0 or -inf.  NaN
// stays: it fails every comparison with a bound, and as a weight counts as far below.
__device__ __forceinline__ float clean(float x, bool inf)
{
    return inf ? (x == __builtin_inff() ? 0.0f : -__builtin_inff()) : x;
}

// One past the last kept element in the order: kept are keys above `key`, and equal
// ones up to `index`.
struct Cut {
    uint32_t key, index;
    __device__ __forceinline__ bool keeps(uint32_t k, uint32_t i) const { return k > key || (k == key && i <= index); }
};

// An infinite temperature makes all weights 1: so does this one, without 0 times infinity.
__device__ __forceinline__ double finite_temperature(float t) { return __builtin_fmin(double(t), 1e300); }

template <int TYPE>
struct Row {
    const void* p;
    int64_t vocab;
    int steps;       // of SM_STEP logits
    int index_bits;  // vocab <= 2^index_bits
    bool inf;        // see clean()
    float top;       // largest logit (after clean)
    double top64, c; // log2 w = (x - top) c, c = log2 e / t
    double far;      // -1000 / c: weights further down count as 2^-1000, next to nothing
    int frac;        // bits below the octave's unit in the bins' integers

    __device__ __forceinline__ void set_top(float t)
    {
        inf = t == __builtin_inff();
        top = inf ? 0.0f : t;
        top64 = uniform(double(top));
    }
    __device__ __forceinline__ void set_temperature(float t)
    {
        const double d = finite_temperature(t);
        c = uniform(LOG2E / d);
        far = uniform(-1000.0 * d / LOG2E);
    }
    // log2 of the weight: 0 for the largest, at most 0, monotone in x.  The subtraction comes first: folded into
    // one multiply-add it would leave the rounding of top c, 2e-12 for a logit of 400 at a temperature of 0.01,
    // in every weight.
    __device__ __forceinline__ double log2w(float x) const { return (double(x) - top64) * c; }
    __device__ __forceinline__ double weight(float x) const { return exp2_exact(log2w(x)); }
    // x - top in the range of exp2_fast; NaN counts as masked
    __device__ __forceinline__ double below(float x) const { return __builtin_fmax(double(x) - top64, far); }
    // bin: the nearest eighth of an octave below the largest weight
    __device__ __forceinline__ uint32_t bin(double d) const
    {
        const uint32_t b = uint32_t(__builtin_bit_cast(uint64_t, __builtin_fma(d, c * -double(SM_PER_OCTAVE), TO_INT)));
        return b < SM_BINS - 1 ? b : SM_BINS - 1;
    }
    // a weight in bin b as an integer of 2^-frac of the bin's octave, and back
    __device__ __forceinline__ uint64_t fixed(double d, uint32_t b) const
    {
        const double w = exp2_fast(d, c, int(b / SM_PER_OCTAVE) + frac) + 0x1p52;
        return __builtin_bit_cast(uint64_t, w) & ((uint64_t(1) << 52) - 1);
    }
    __device__ __forceinline__ double unfixed(uint64_t m, uint32_t b) const
    {
        return __builtin_ldexp(double(m), -(int(b / SM_PER_OCTAVE) + frac));
    }
    // f(x[8], index of x[0]) over steps first, first + stride, ... below end, by one wave, U loads at a time.
    // AHEAD: the next U are in flight while f works on these, for twice the registers.
    template <int U, bool AHEAD = true, class F>
    __device__ __forceinline__ void for_steps(int first, int end, int stride, F f) const
    {
        first = uniform(first);  // the same in all lanes, as the addresses want it
        end = uniform(end);
        Raw<TYPE> raw[U], next[U];
        const auto load = [&](Raw<TYPE>(&to)[U], int s) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u * stride < end)
                    to[u].load_step(p, s + u * stride, vocab);
        };
        if (AHEAD)
            load(raw, first);
        for (int s = first; s < end; s += U * stride) {
            if (AHEAD)
                load(next, s + U * stride);
            else
                load(raw, s);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = s + u * stride;
                if (at < end) {
                    float x[SM_VEC];
                    raw[u].unpack(x, inf);
                    f(x, uint32_t(at) * SM_STEP + uint32_t(lane_id() * SM_VEC));
                }
                __builtin_amdgcn_sched_barrier(0);  // one load's work at a time, for the registers
            }
            if (AHEAD) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    raw[u] = next[u];
            }
        }
    }
};

// ---------------------------------------------------------------- running sums
// The place of u in a sum: u <= 0 and NaN count as 0.  From 1 on it is past every running sum, whose rounding may
// be more than the last tokens weigh: the last positive weight is taken.
__device__ __forceinline__ double goal_of(double u, double total)
{
    return u > 0.0 ? (u < 1.0 ? u * total : double(__builtin_inff())) : 0.0;
}

// Sums of N values per lane: `incl` with the lanes before, `total` of all.
template <int N>
__device__ __forceinline__ void wave_sums(const double (&v)[N], double& incl, double& total)
{
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < N; ++k)
        sum += v[k];
    incl = wave_inclusive_sum64(sum);
    total = read_lane64(incl, 63);
}

// One wave, N values per lane in order (lane 0's first): the first at which `before` plus
// their running sum exceeds `goal` (`over`), the last positive one if none does, -1 if none
// is positive.  `incl`: the sum with the lanes before (wave_sums).  `before` becomes the sum
// in front of it.
template <int N>
__device__ __forceinline__ int wave_first_over(const double (&v)[N], double goal, double incl, double& before,
                                               bool& over)
{
    double r = before + dpp_move64<DPP_WAVE_SHR1, 0xf>(incl), at_hit = 0.0, at_last = 0.0;
    int hit = -1, last = -1;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const double up = r + v[k];
        if (v[k] > 0.0) {
            last = k;
            at_last = r;
            if (hit < 0 && up > goal) {
                hit = k;
                at_hit = r;
            }
        }
        r = up;
    }
    const uint64_t hits = __ballot(hit >= 0), any = __ballot(last >= 0);
    over = hits != 0;
    if (any == 0)
        return -1;
    const int l = over ? __builtin_ctzll(hits) : 63 - __builtin_clzll(any);
    before = read_lane64(over ? at_hit : at_last, l);
    return l * N + read_lane(over ? hit : last, l);
}

// One wave: the first index in steps [first, end) at which `run` and the running sum of
// f(x, index) exceed `goal`, or the last of positive weight; ~0 if there is none.
template <int U, int TYPE, class F>
__device__ __forceinline__ uint32_t wave_find_token(const Row<TYPE>& row, int first, int end, double run, double goal,
                                                    F f)
{
    uint32_t found = ~0u;
    bool over = false;
    row.template for_steps<U, false>(first, end, 1, [&](const float(&x)[SM_VEC], uint32_t idx) {
        if (over)
            return;
        double w[SM_VEC], incl, total, before = run;
#pragma unroll
        for (int k = 0; k < SM_VEC; ++k)
            w[k] = f(x[k], idx + k);
        wave_sums(w, incl, total);
        const int at = wave_first_over(w, goal, incl, before, over);
        if (at >= 0)
            found = uniform(idx) + uint32_t(at);
        run += total;
    });
    return found;
}

struct SharedSums {
    double sums[SM_BLOCK];
    uint32_t first, last, found, arrived;
};

// The block: the first index in the whole row, in index order, at which the running sum of
// f(x, index) exceeds u times the sum of all.  To all threads, with that sum.
template <int TYPE, class F>
__device__ __forceinline__ uint32_t find_in_order(const Row<TYPE>& row, SharedSums& sh, double u, F f, double& total)
{
    constexpr int N = SM_BLOCK / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (row.steps + SM_BLOCK - 1) / SM_BLOCK;  // steps per sum
    const int sums = (row.steps + per - 1) / per;
    __syncthreads();
    if (tid >= sums)
        sh.sums[tid] = 0.0;
    for (int s = wave; s < sums; s += SM_WAVES) {
        double sum = 0.0;
        row.template for_steps<1>(s * per, s * per + per < row.steps ? s * per + per : row.steps, 1,
                                  [&](const float(&x)[SM_VEC], uint32_t idx) {
#pragma unroll
                                      for (int k = 0; k < SM_VEC; ++k)
                                          sum += f(x[k], idx + k);
                                  });
        sum = wave_inclusive_sum64(sum);
        if (lane == 63)
            sh.sums[s] = sum;
    }
    __syncthreads();
    if (wave == 0) {
        double v[N], incl, before = 0.0;
        bool over;
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k] = sh.sums[lane * N + k];
        wave_sums(v, incl, total);
        const int over_at = wave_first_over(v, goal_of(u, total), incl, before, over), s = over_at < 0 ? 0 : over_at;
        const uint32_t token = wave_find_token<1>(row, s * per, s * per + per < row.steps ? s * per + per : row.steps,
                                               before, goal_of(u, total), f);
        if (lane == 0) {
            sh.found = token;
            sh.sums[0] = total;
        }
    }
    __syncthreads();
    total = uniform(sh.sums[0]);
    return uniform(sh.found);
}

// ---------------------------------------------------------------- handing a row on
// What a row's waves leave for the last of them: written and read at device scope, with
// the stores complete before the wave (or its block) counts itself in.
template <class T>
__device__ __forceinline__ void put(T* p, T v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get(const T* p)
{
    return __hip_atomic_load(const_cast<T*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Counts the caller in; whether it is the last of `parts`, which leaves the counter at 0.
// Additions to one 128-byte line take turns (about 10 ns each): a line to each row, and one
// addition to a block.  With counters side by side and one addition to a wave, 16 rows of
// 131072 without cuts took 54 us against 13.
__device__ __forceinline__ bool count_in(uint32_t* counter, uint32_t parts)
{
    const bool last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u == parts;
    if (last)
        put(counter, 0u);
    return last;
}

// The launch: part p of row r is block p * rows + r, so that the last blocks of the rows,
// which go on alone, lie on all XCDs (rows' blocks next to each other had put them on two
// of the eight: 416 us against 101 for 256 rows cut by mass).  Each wave of a block takes
// `per_wave` segments of seg_steps steps.
struct SampleGrid {
    uint32_t* counters;  // one per row, 0 between calls
    // rows x segs: each segment's largest value, or (with cuts) x 4: that of each quarter, and behind these where
    // a row has no more than SM_FINE_SEGS x 16: that of each four lanes
    float* tops;
    double* sums;        // rows x segs: without cuts, and its weights relative to that
    float* split_tops;   // rows: the largest value where sample_bins_kernel makes the cut, else NaN
    uint64_t* masses;    // rows x SM_WAVES x SM_BINS: the bins of each sixteenth of a row
    int steps, seg_steps, segs, per_wave, parts;
    bool split;
};

template <int TYPE>
__device__ __forceinline__ Row<TYPE> make_row(const SampleCall& call, const SampleGrid& g, int64_t r)
{
    Row<TYPE> row;
    row.p = static_cast<const char*>(call.logits) + r * call.stride * (TYPE == LOGITS_F32 ? 4 : 2);
    row.vocab = call.vocab;
    row.steps = g.steps;
    row.index_bits = call.vocab > 1 ? 32 - __builtin_clz(uint32_t(call.vocab - 1)) : 0;
    // A bin is a sum of up to vocab integers of at most 2^(frac + 1/16), a range of one (cut_in_bin) too.  Rounded to the
    // unit, a weight is off by 2^-(frac + 0.94) of itself in a bin and 2^-(frac + 0.06) in a range, always the same way
    // where logits are equal; 2^-44 up to 2^17 logits, 2^-(61 - index_bits) beyond.
    row.frac = 61 - row.index_bits < 44 ? 61 - row.index_bits : 44;
    row.inf = false;
    return row;
}

// One wave writes the row's result.
__device__ __forceinline__ void write_result(const SampleCall& call, int64_t r, int64_t token, double logprob)
{
    if (lane_id() == 0) {
        call.tokens[r] = token;
        if (call.logprobs != nullptr)
            call.logprobs[r] = float(logprob);
    }
}

template <int TYPE>
__device__ __forceinline__ void write_token(const SampleCall& call, int64_t r, const Row<TYPE>& row, uint32_t token,
                                            double total)
{
    token = token < row.vocab ? token : 0u;  // within the row, whatever the sums were
    if (lane_id() == 0) {
        float x;
        if constexpr (TYPE == LOGITS_F32)
            x = static_cast<const float*>(row.p)[token];
        else if constexpr (TYPE == LOGITS_BF16)
            x = from_bits<float>(uint32_t(static_cast<const uint16_t*>(row.p)[token]) << 16);
        else
            x = float(static_cast<const _Float16*>(row.p)[token]);
        call.tokens[r] = token;
        if (call.logprobs != nullptr)
            call.logprobs[r] = float(row.log2w(clean(x, row.inf)) * LN2 - ::log(total));
    }
}

// The largest values of a row's segments, in one wave's registers in order.
struct Tops {
    float v[SM_PER_LANE];
    int per_lane;
    __device__ __forceinline__ int seg(int k) const { return lane_id() * per_lane + k; }
    __device__ __forceinline__ float load(const SampleGrid& g, int64_t r)
    {
        per_lane = (g.segs + 63) / 64;
        float m = -__builtin_inff();
#pragma unroll
        for (int k = 0; k < SM_PER_LANE; ++k) {
            v[k] = -__builtin_inff();
            if (k < per_lane && seg(k) < g.segs)
                v[k] = get(&g.tops[r * g.segs + seg(k)]);
        }
#pragma unroll
        for (int k = 0; k < SM_PER_LANE; ++k)
            m = v[k] > m ? v[k] : m;
        return read_lane(wave_inclusive_scan<MaxF32>(m), 63);
    }
};

// With cuts: the largest values of the segments' quarters (16 lanes of each step), and of the
// segments.
struct QuarterTops : Tops {
    float quarter[SM_PER_LANE][4];
    __device__ __forceinline__ float load(const SampleGrid& g, int64_t r)
    {
        per_lane = (g.segs + 63) / 64;
        float m = -__builtin_inff();
        uint64_t w[SM_PER_LANE][2];
#pragma unroll
        for (int k = 0; k < SM_PER_LANE; ++k) {
            w[k][0] = w[k][1] = 0xff800000ff800000ull;
            if (k < per_lane && seg(k) < g.segs) {
                const uint64_t* p = reinterpret_cast<const uint64_t*>(g.tops) + (r * g.segs + seg(k)) * 2;
                w[k][0] = get(p);
                w[k][1] = get(p + 1);
            }
        }
#pragma unroll
        for (int k = 0; k < SM_PER_LANE; ++k) {
            v[k] = -__builtin_inff();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                quarter[k][q] = from_bits<float>(uint32_t(w[k][q / 2] >> (q % 2 * 32)));
                v[k] = quarter[k][q] > v[k] ? quarter[k][q] : v[k];
            }
            m = v[k] > m ? v[k] : m;
        }
        return read_lane(wave_inclusive_scan<MaxF32>(m), 63);
    }
};

// One wave: rows with nothing left, and the first index of the largest value where the
// temperature asks for it.  True when the row is done.
template <int TYPE>
__device__ __forceinline__ bool settle(const SampleCall& call, const SampleGrid& g, int64_t r, Row<TYPE>& row,
                                       const Tops& tops, float top)
{
    row.set_top(top);
    if (top == -__builtin_inff()) {
        write_result(call, r, -1, -double(__builtin_inff()));
        return true;
    }
    const float t = call.temperature[r];
    if (t > 0.0f) {
        row.set_temperature(t);
        return false;
    }
    uint32_t seg = ~0u;
#pragma unroll
    for (int k = SM_PER_LANE - 1; k >= 0; --k)
        if (tops.v[k] == top)
            seg = uint32_t(tops.seg(k));
    seg = read_lane(wave_inclusive_scan<MinU32>(seg), 63);
    const int s0 = int(seg) * g.seg_steps, s1 = s0 + g.seg_steps < g.steps ? s0 + g.seg_steps : g.steps;
    uint32_t first = ~0u;
    row.template for_steps<1>(s0, s1, 1, [&](const float(&x)[SM_VEC], uint32_t idx) {
#pragma unroll
        for (int k = SM_VEC - 1; k >= 0; --k)
            if (x[k] == row.top && idx + k < first)
                first = idx + k;
    });
    write_result(call, r, int64_t(read_lane(wave_inclusive_scan<MinU32>(first), 63)), 0.0);
    return true;
}

// ---------------------------------------------------------------- no cuts
// A segment's weights, relative to its own largest value `top`: two passes over its steps.
// For greedy rows only `top` is found.
template <int TYPE>
__device__ __forceinline__ double careful_sum(const Row<TYPE>& row, int s0, int s1, bool sums, double c, double far,
                                              float& top)
{
    float m = -__builtin_inff();
    row.template for_steps<TYPE == LOGITS_F32 ? 2 : 4, false>(s0, s1, 1, [&](const float(&x)[SM_VEC], uint32_t) {
#pragma unroll
        for (int k = 0; k < SM_VEC; ++k)
            m = x[k] > m ? x[k] : m;
    });
    top = read_lane(wave_inclusive_scan<MaxF32>(m), 63);
    if (!sums || top == -__builtin_inff())
        return 0.0;
    double sum = 0.0;
    row.template for_steps<1>(s0, s1, 1, [&](const float(&x)[SM_VEC], uint32_t) {
#pragma unroll
        for (int k = 0; k < SM_VEC; ++k) {
            const float y = clean(x[k], top == __builtin_inff());
            sum += exp2_fast(__builtin_fmax(double(y) - double(clean(top, top == __builtin_inff())), far), c);
        }
    });
    return sum;
}

// Waves work for themselves; the first of the row's last block finds its token.  A double
// reaches from 2^-1000 to 2^1000, so a wave's weights can be taken relative to the largest
// value of its first loads, whatever comes later: logits are held within 2^+-1000 of it, and a
// sum that leaves 2^-800 .. 2^800 (as one with NaN in it may) is made again with the
// segment's own largest value.  Bound by the logits' bytes in float32 and by the vector
// instructions (21 a logit, 18 of them for the weight) in 16 bits.
template <int TYPE>
__global__ __launch_bounds__(SM_ALL_BLOCK, 4) void sample_all_kernel(SampleCall call, SampleGrid g)
{
    constexpr float NEG = -__builtin_inff();
    constexpr int U = TYPE == LOGITS_F32 ? 2 : 4;
    constexpr int WAVES = SM_ALL_BLOCK / 64;
    const int lane = lane_id(), wave = uniform(int(threadIdx.x >> 6));
    const int64_t r = blockIdx.x % uint32_t(call.rows);
    const int part = int(blockIdx.x / uint32_t(call.rows));
    Row<TYPE> row = make_row<TYPE>(call, g, r);
    const float t = call.temperature[r];
    const bool sums = t > 0.0f;
    const double c = uniform(LOG2E / finite_temperature(t)), far = uniform(-1000.0 * finite_temperature(t) / LOG2E);
    const int seg0 = (part * WAVES + wave) * g.per_wave;
    const int seg1 = seg0 + g.per_wave < g.segs ? seg0 + g.per_wave : g.segs;
    const auto seg_end = [&](int seg) { return (seg + 1) * g.seg_steps < g.steps ? (seg + 1) * g.seg_steps : g.steps; };
    float ref = NEG, low = 0.0f, high = 0.0f;
    double k = TO_INT, scale = 1.0;  // sums are relative to 2^R; times `scale`, to ref's weight
    if (sums && seg0 < seg1) {
        // U steps at a time, the next ones on their way meanwhile, in two sets of registers by turns
        Raw<TYPE> set0[U], set1[U];
        const auto load = [&](Raw<TYPE>(&to)[U], int s, int end) {
            const int64_t first = int64_t(s) * SM_STEP;
            if (s + U <= end && first + U * SM_STEP <= row.vocab) {
                const auto* at = static_cast<const typename Raw<TYPE>::E*>(row.p) + first + uint32_t(lane) * SM_VEC;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    to[u].load_all(at + u * SM_STEP);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    to[u].clear();
                    if (s + u < end)
                        to[u].load_step(row.p, s + u, row.vocab);
                }
            }
        };
        int seg = seg0, s = seg0 * g.seg_steps, s1 = seg_end(seg0);
        double sum = 0.0;
        // adds up the loaded steps with the next ones under way; false after the last
        const auto turn = [&](Raw<TYPE>(&raw)[U], Raw<TYPE>(&next)[U]) {
            const bool ends = s + U >= s1;
            const int next_seg = ends ? seg + 1 : seg, next_s = ends ? next_seg * g.seg_steps : s + U;
            const int next_s1 = ends ? seg_end(next_seg) : s1;
            if (next_seg < seg1)
                load(next, next_s, next_s1);
            if (ref == NEG) {
                float m = NEG;
#pragma unroll
                for (int j = 0; j < SM_VEC; ++j)
                    m = raw[0].at(j) > m ? raw[0].at(j) : m;
                ref = read_lane(wave_inclusive_scan<MaxF32>(m), 63);
                low = uniform(float(double(ref) + far));
                high = uniform(float(double(ref) - far));
                const double whole = __builtin_rint(double(ref) * c), off = (double(low) - double(ref)) * c;
                k = uniform(TO_INT - whole);
                scale = uniform(exp2_exact(-__builtin_fma(double(ref), c, -whole)));
                // not so where there is no finite value to go by, no float near enough to 2^-1000 of it, or no
                // room for R beside the fractions (very low and high temperatures)
                if (!(off > -1010.0 && off < -900.0 && double(high) - double(ref) < -1.01 * far &&
                      __builtin_fabs(double(ref) * c) < 0x1p40))
                    scale = __builtin_nan("");
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s + u < s1) {
#pragma unroll
                    for (int j = 0; j < SM_VEC; j += 4) {
                        double x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = double(__builtin_amdgcn_fmed3f(raw[u].at(j + i), low, high));
                        sum += exp2_sum4(x, c, k);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);  // one load's work at a time, for the registers
            }
            if (ends) {
                sum = read_lane64(wave_inclusive_sum64(sum), 63) * scale;
                float top = ref;
                if (!(sum > 0x1p-800 && sum < 0x1p800)) {
                    sum = read_lane64(wave_inclusive_sum64(careful_sum(row, seg * g.seg_steps, s1, true, c, far, top)), 63);
                    if (scale != scale)
                        ref = NEG;  // the next loads may do
                }
                if (lane == 63) {
                    put(&g.tops[r * g.segs + seg], top);
                    put(&g.sums[r * g.segs + seg], sum);
                }
                sum = 0.0;
            }
            seg = next_seg;
            s = next_s;
            s1 = next_s1;
            return next_seg < seg1;
        };
        load(set0, s, s1);
        while (turn(set0, set1) && turn(set1, set0)) {
        }
    } else {
        for (int seg = seg0; seg < seg1; ++seg) {
            float top;
            careful_sum(row, seg * g.seg_steps, seg_end(seg), false, c, far, top);
            if (lane == 63)
                put(&g.tops[r * g.segs + seg], top);
        }
    }
    __shared__ uint32_t s_last;
    stores_done();
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = count_in(&g.counters[r * SM_COUNTER], uint32_t(g.parts)) ? 1u : 0u;
    __syncthreads();
    if (uniform(s_last) == 0u || wave != 0)
        return;

    Tops tops;
    const float top = tops.load(g, r);
    if (settle(call, g, r, row, tops, top))
        return;
    double v[SM_PER_LANE], incl, total, before = 0.0;
#pragma unroll
    for (int k = 0; k < SM_PER_LANE; ++k) {
        v[k] = 0.0;
        if (k < tops.per_lane && tops.v[k] != NEG)
            v[k] = get(&g.sums[r * g.segs + tops.seg(k)]) * row.weight(clean(tops.v[k], row.inf));
    }
    wave_sums(v, incl, total);
    const double goal = goal_of(double(call.uniforms[r]), total);
    bool over;
    const int at = wave_first_over(v, goal, incl, before, over);
    int seg = at < 0 ? 0 : at / SM_PER_LANE * tops.per_lane + at % SM_PER_LANE;
    // u >= 1: from the last segment back, since a segment's sum may be 0 where a weight is not (it is relative to
    // another logit), and the other way round
    const bool last = goal == double(__builtin_inff());
    if (last)
        seg = g.segs - 1;
    uint32_t token;
    do {
        const int s0 = seg * g.seg_steps, s1 = s0 + g.seg_steps < g.steps ? s0 + g.seg_steps : g.steps;
        token = wave_find_token<TYPE == LOGITS_F32 ? 2 : 4>(row, s0, s1, before, goal,
                                                            [&](float x, uint32_t) { return row.weight(x); });
    } while (last && token == ~0u && --seg >= 0);
    write_token(call, r, row, token, total);
}

// ---------------------------------------------------------------- cuts
struct Bin {
    uint32_t bin, key_lo, key_hi;
};

struct Pick {
    Bin bin;
    uint32_t above_count, reached, about;
    double above, goal;
};

struct SharedCuts {
    SharedSums s;
    uint64_t mass[SM_WAVES][SM_BINS];  // weight by bin of each sixteenth of the row, in 2^-frac of the bin's own
    double bin_weight[SM_BINS];        // that unit
    double bin_mass[SM_BINS];          // weight of the whole row
    uint32_t bin_count[SM_BINS];
    uint64_t range_mass[SM_RANGES];
    uint32_t range_count[SM_RANGES];
    uint32_t notes[SM_WAVES][SM_NOTES];  // indexes of loads that hold elements of a bin
    uint64_t list[SM_LIST];              // their places in the order: (largest key - key) << index_bits | index
    uint64_t small[SM_SMALL], sorted[SM_SMALL];
    double weight[SM_SMALL];
    double part_sum[SM_WAVES];
    uint64_t part_mass[SM_WAVES];
    uint32_t n_list, n_small, n_quarters, keep;
    uint32_t goes_on;  // whether the row's last block has more to do (a word of its own: s.arrived is still being read)
    float top, low;
    double kept;
    Pick pick;
    uint16_t quarters[SM_SEGS * 4];  // segment * 4 + quarter: those with candidates
};

// write(place, x[k], k) for each element with in(x[k], k), places counted on from a shared
// counter by one addition for the wave.
template <class P, class F>
__device__ __forceinline__ void wave_append(uint32_t* counter, const float (&x)[SM_VEC], P in, F write)
{
    uint64_t m[SM_VEC];
    int all = 0;
#pragma unroll
    for (int k = 0; k < SM_VEC; ++k) {
        m[k] = __ballot(in(x[k], k));
        all += __builtin_popcountll(m[k]);
    }
    if (all == 0)
        return;
    uint32_t at = 0;
    if (lane_id() == 0)
        at = atomicAdd(counter, uint32_t(all));
    at = uniform(at);
#pragma unroll
    for (int k = 0; k < SM_VEC; ++k) {
        if (m[k] != 0) {
            if (in(x[k], k))
                write(at + __builtin_amdgcn_mbcnt_hi(uint32_t(m[k] >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m[k]), 0u)),
                      x[k], k);
            at += uint32_t(__builtin_popcountll(m[k]));
        }
    }
}

// Orders the n <= SM_SMALL distinct places of `small` into `sorted`: each place's rank is the
// number of smaller ones, counted by a group of lanes.
__device__ __forceinline__ void order_small(SharedCuts& sh, uint32_t n)
{
    uint32_t group = 64;
    while (group > 1 && SM_BLOCK / group < n)
        group >>= 1;
    const uint32_t e = threadIdx.x / group, part = threadIdx.x & (group - 1);
    uint32_t rank = 0;
    const uint64_t v = e < n ? sh.small[e] : 0;
    if (e < n)
        for (uint32_t j = part; j < n; j += 4 * group) {
            uint64_t w[4];  // four at a time on their way
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                w[i] = sh.small[(j + i * group) % SM_SMALL];
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                rank += j + i * group < n && w[i] < v ? 1u : 0u;
        }
    for (uint32_t d = 1; d < group; d <<= 1)
        rank += __shfl_xor(rank, int(d));
    if (e < n && part == 0)
        sh.sorted[rank] = v;
    __syncthreads();
}

// One wave (all of them alike): the first of 64 N bins or ranges at which the running count
// reaches `want` (by_count) or the running weight `goal`, the last one that holds anything
// if none does.  above_count and above become what lies before it, `n` what it holds.
template <int N, class W>
__device__ __forceinline__ uint32_t pick(const uint32_t* counts, W weight_of, bool by_count, uint32_t want,
                                         double goal, uint32_t& above_count, double& above, uint32_t& n)
{
    const int first = lane_id() * N;
    uint32_t c[N], cs = 0;
    double m[N], ms = 0.0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        c[k] = counts[first + k];
        m[k] = weight_of(uint32_t(first + k));
        cs += c[k];
        ms += m[k];
    }
    uint32_t cr = above_count + wave_shift_up<SumU32>(wave_inclusive_scan<SumU32>(cs));
    uint32_t hit_c = 0, last_c = 0, hit_n = 0, last_n = 0;
    double mr = above + dpp_move64<DPP_WAVE_SHR1, 0xf>(wave_inclusive_sum64(ms)), hit_m = 0.0, last_m = 0.0;
    int hit = -1, last = -1;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t cu = cr + c[k];
        const double mu = mr + m[k];
        if (c[k] != 0) {
            last = k, last_c = cr, last_m = mr, last_n = c[k];
            if (hit < 0 && (by_count ? cu >= want : mu >= goal))
                hit = k, hit_c = cr, hit_m = mr, hit_n = c[k];
        }
        cr = cu;
        mr = mu;
    }
    const uint64_t hits = __ballot(hit >= 0), any = __ballot(last >= 0);
    const bool over = hits != 0;
    const int l = over ? __builtin_ctzll(hits) : any != 0 ? 63 - __builtin_clzll(any) : 0;
    above_count = read_lane(over ? hit_c : last_c, l);
    above = read_lane64(over ? hit_m : last_m, l);
    n = read_lane(over ? hit_n : last_n, l);
    const int k = read_lane(over ? hit : last, l);
    return uint32_t(l * N + (k < 0 ? 0 : k));
}

// The smallest key whose bin is at most b (all keys down to the lowest finite one for the
// last bin), by one wave: 64 tries a step, the first ones around where the bin ends by
// its formula.
template <int TYPE>
__device__ __forceinline__ uint32_t lowest_key(const Row<TYPE>& row, uint32_t b)
{
    uint32_t lo = KEY_NEG_INF, hi = key_of(row.top);  // lo is out, hi is in
    if (b >= SM_BINS - 1)
        return KEY_NEG_INF + 1;
    const float edge = float(row.top64 - (double(b) + 0.5) / SM_PER_OCTAVE / row.c);
    if (edge > -__builtin_inff() && edge < row.top) {
        const uint32_t key = uniform(key_of(edge)) - 32u + uint32_t(lane_id());
        const uint64_t in = __ballot(key >= hi || (key > lo && row.bin(row.below(value_of(key))) <= b));
        const int l = in != 0 ? __builtin_ctzll(in) : 64;
        const uint32_t first = uniform(key_of(edge)) - 32u;
        if (l > 0 && first > lo)
            lo = first + uint32_t(l) - 1u;  // out
        if (l < 64 && first + uint32_t(l) < hi)
            hi = first + uint32_t(l);
    }
    while (hi - lo > 1) {
        const uint32_t step = (hi - lo + 63) / 64, off = uint32_t(lane_id() + 1) * step;
        const uint32_t key = off < hi - lo ? lo + off : hi;
        const uint64_t in = __ballot(key == hi || row.bin(row.below(value_of(key))) <= b);
        const int l = __builtin_ctzll(in);
        const uint32_t first = read_lane(key, l), before = l > 0 ? read_lane(key, l - 1) : lo;
        lo = before;
        hi = first;
    }
    return hi;
}

template <int TYPE>
__device__ __forceinline__ Bin make_bin(const Row<TYPE>& row, uint32_t b)
{
    Bin bin;
    bin.bin = b;
    bin.key_lo = lowest_key(row, b);
    bin.key_hi = b > 0 ? lowest_key(row, b - 1) - 1 : key_of(row.top);
    return bin;
}

// A place in the order, relative to a bin's largest key.
template <int TYPE>
__device__ __forceinline__ uint64_t place_of(const Row<TYPE>& row, uint32_t key_hi, uint32_t key, uint32_t index)
{
    return (uint64_t(key_hi - key) << row.index_bits) | index;
}
template <int TYPE>
__device__ __forceinline__ uint32_t key_at(const Row<TYPE>& row, uint32_t key_hi, uint64_t place)
{
    return key_hi - uint32_t(place >> row.index_bits);
}
template <int TYPE>
__device__ __forceinline__ uint32_t index_at(const Row<TYPE>& row, uint64_t place)
{
    return uint32_t(place) & ((1u << row.index_bits) - 1u);
}

// x[k].  The values pass through an empty asm, or the compiler would index x itself, in memory.
__device__ __forceinline__ float choose(const float (&x)[SM_VEC], uint32_t k)
{
    float v = x[0];
#pragma unroll
    for (uint32_t i = 1; i < SM_VEC; ++i) {
        float y = x[i];
        asm("" : "+v"(y));
        v = k == i ? y : v;
    }
    return v;
}

// Collects a bin's elements with a place in [lo, hi] into the list; their number, or more than
// SM_LIST where they are too many.  First each wave notes which lanes' loads hold any of them
// (one test for eight elements: few hold any), then it reads only these again.
template <int TYPE>
__device__ __forceinline__ uint32_t collect(const Row<TYPE>& row, SharedCuts& sh, const Bin& bin, uint64_t lo,
                                            uint64_t hi)
{
    const uint32_t lane = uint32_t(lane_id());
    const int wave = uniform(int(threadIdx.x >> 6));
    const uint32_t k_lo = key_at(row, bin.key_hi, hi), k_hi = key_at(row, bin.key_hi, lo);
    const float x_lo = value_of(k_lo), x_hi = value_of(k_hi);
    // a range within one value is one of indexes; any other takes its values whole (cut_in_bin)
    const uint32_t i_lo = k_lo == k_hi ? index_at(row, lo) : 0u;
    const uint32_t i_hi = k_lo == k_hi ? index_at(row, hi) : ~0u - SM_VEC;
    const int begin = int(i_lo / SM_STEP);
    const int end = i_hi / SM_STEP < uint32_t(row.steps) ? int(i_hi / SM_STEP) + 1 : row.steps;
    // a little more than half the values' range about its middle, for the roundings of x - mid
    const float mid = uniform(0.5f * x_lo + 0.5f * x_hi);
    const float half = uniform((0.5f * x_hi - 0.5f * x_lo) * 1.000001f + (__builtin_fabsf(x_lo) + __builtin_fabsf(x_hi)) * 1e-6f + 1e-37f);
    __syncthreads();
    if (threadIdx.x == 0)
        sh.n_list = 0;
    uint32_t n = 0;
    uint32_t* notes = sh.notes[wave];
    row.template for_steps<TYPE == LOGITS_F32 ? 2 : 4, false>(begin + wave, end, SM_WAVES, [&](const float(&x)[SM_VEC], uint32_t idx) {
        float near = __builtin_inff();
#pragma unroll
        for (int k = 0; k < SM_VEC; ++k)
            near = __builtin_fminf(near, __builtin_fabsf(x[k] - mid));
        const uint64_t m = __ballot(near <= half && idx + SM_VEC > i_lo && idx <= i_hi);
        if (m == 0)
            return;
        const uint32_t at =
            n + __builtin_amdgcn_mbcnt_hi(uint32_t(m >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m), 0u));
        if ((m >> lane & 1u) && at < SM_NOTES)
            notes[at] = idx;
        n += uint32_t(__builtin_popcountll(m));
    });
    __syncthreads();
    if (n > SM_NOTES && lane == 0)
        atomicAdd(&sh.n_list, uint32_t(SM_LIST) + 1u);
    constexpr uint32_t U = TYPE == LOGITS_F32 ? 2 : 4;
    static_assert(SM_NOTES == 256, "64 at a time, U on their way");
#pragma unroll 1
    for (uint32_t j = 0; j < n && n <= SM_NOTES; j += 64 * U) {
        Raw<TYPE> raw[U];
        uint32_t note[U];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t at = j + u * 64 + lane;
            raw[u].clear();
            note[u] = at < n ? notes[at] : 0u;
            if (at < n)
                raw[u].load(row.p, note[u], row.vocab);
        }
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (j + u * 64 >= n)
                break;
            float x[SM_VEC];
            raw[u].unpack(x, row.inf);
            uint32_t in = 0;
#pragma unroll
            for (uint32_t k = 0; k < SM_VEC; ++k)
                in |= x[k] >= x_lo && x[k] <= x_hi && note[u] + k - i_lo <= i_hi - i_lo ? 1u << k : 0u;
            const uint32_t mine = uint32_t(__builtin_popcount(in)), incl = wave_inclusive_scan<SumU32>(mine);
            uint32_t at = 0;
            if (lane == 63)
                at = atomicAdd(&sh.n_list, incl);
            at = read_lane(at, 63) + incl - mine;
            while (in != 0) {
                const uint32_t k = uint32_t(__builtin_ctz(in));
                in &= in - 1;
                if (at < SM_LIST)
                    sh.list[at] = place_of(row, bin.key_hi, key_of(choose(x, k)), note[u] + k);
                ++at;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
    return uniform(sh.n_list);
}

// The element of a bin that makes the count reach `want` (by_count) or the weight reach
// `goal`, where above_count and above lie in front of the bin.  Its elements are
// collected; while they are too many, the range of places is cut into SM_RANGES and the
// one the cut lies in is kept.  A range is a power of two of places and starts at a multiple
// of it, so it is whole values, or indexes of one value.  At most eight bits of 64 go at a
// time, and one place is one element, so eight rounds and the one that collects suffice.
// `n`: about how many elements the bin holds.  Returns the place; `weight`: the weight up to and
// including it; `whole`: whether the list holds the whole bin.  What the bin holds before the list's range is
// left in sh.part_mass for each sixteenth of the row.
template <int TYPE>
__device__ __forceinline__ uint64_t cut_in_bin(const Row<TYPE>& row, SharedCuts& sh, const Bin& bin, bool by_count,
                                               uint32_t want, double goal, uint32_t above_count, double above,
                                               uint32_t n, double& weight, bool& whole)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(int(tid >> 6));
    const uint64_t all = place_of(row, bin.key_hi, bin.key_lo, (1u << row.index_bits) - 1u);
    uint64_t lo = 0, hi = all;
    bool in_list = false;
    uint64_t* const masses = &sh.list[wave * SM_RANGES];  // of the ranges in a sixteenth, while there is no list
    static_assert(SM_LIST >= SM_WAVES * SM_RANGES, "room in the list");
    whole = false;
    if (tid < SM_WAVES)
        sh.part_mass[tid] = 0;
    for (int round = 0; round < 10; ++round) {
        if (!in_list && n <= SM_LIST) {
            whole = lo == 0 && hi == all;
            n = collect(row, sh, bin, lo, hi);
            in_list = n <= SM_LIST;
            whole = whole && in_list;
        }
        if (in_list && n <= SM_FEW)
            break;
        const uint64_t span = hi - lo;
        const int bits = 64 - __builtin_clzll(span | 1u);
        const int shift = bits > 8 ? bits - 8 : 0;
        static_assert(SM_RANGES == 1 << 8, "eight bits of the span");
        if (tid < SM_RANGES) {
            sh.range_mass[tid] = 0;
            sh.range_count[tid] = 0;
        }
        if (!in_list)
            for (uint32_t i = lane; i < SM_RANGES; i += 64)
                masses[i] = 0;
        __syncthreads();
        // the lanes that agree with the first one make one addition: values that repeat, as a mask's lowest
        // one, would take turns (208 rows of 115258 logits, 82000 of a row masked so, top-k 75685: 491 us, so 318; 64 flat rows
        // of 131072 78 and 83)
        const auto add = [&](uint64_t v, float x, uint64_t* mass) {
            const uint32_t b = uint32_t((v - lo) >> shift), b0 = __builtin_amdgcn_readfirstlane(b);
            const bool same = b == b0 && x == uniform(x);
            const uint64_t all_same = __ballot(same);
            const uint32_t times = same ? uint32_t(__builtin_popcountll(all_same)) : 1u;
            if (!same || uint32_t(__builtin_ctzll(all_same)) == lane) {
                atomicAdd(&sh.range_count[b], times);
                atomicAdd(reinterpret_cast<unsigned long long*>(&mass[b]),
                          static_cast<unsigned long long>(row.fixed(row.below(x), bin.bin) * times));
            }
        };
        if (in_list) {
            for (uint32_t i = tid; i < sh.n_list; i += SM_BLOCK) {
                const uint64_t v = sh.list[i];
                if (v >= lo && v <= hi)
                    add(v, value_of(key_at(row, bin.key_hi, v)), sh.range_mass);
            }
        } else {
            const float x_lo = value_of(key_at(row, bin.key_hi, hi)), x_hi = value_of(key_at(row, bin.key_hi, lo));
            const int share = (row.steps + SM_WAVES - 1) / SM_WAVES, begin = wave * share;
            row.template for_steps<1>(begin, begin + share < row.steps ? begin + share : row.steps, 1, [&](const float(&x)[SM_VEC], uint32_t idx) {
                uint32_t in = 0;
#pragma unroll
                for (uint32_t k = 0; k < SM_VEC; ++k)
                    in |= x[k] >= x_lo && x[k] <= x_hi ? 1u << k : 0u;
                // few lanes have more than one or two: as many turns as the one with the most
                while (in != 0) {
                    const uint32_t k = uint32_t(__builtin_ctz(in));
                    in &= in - 1;
                    const float y = choose(x, k);
                    const uint64_t v = place_of(row, bin.key_hi, key_of(y), idx + k);
                    if (v >= lo && v <= hi)
                        add(v, y, masses);
                }
            });
            __syncthreads();
            if (tid < SM_RANGES) {
                uint64_t m = 0;
#pragma unroll
                for (int w = 0; w < SM_WAVES; ++w)
                    m += sh.list[w * SM_RANGES + tid];
                sh.range_mass[tid] = m;
            }
        }
        __syncthreads();
        const uint32_t b = pick<SM_RANGES / 64>(
            sh.range_count, [&](uint32_t i) { return row.unfixed(sh.range_mass[i], bin.bin); }, by_count, want, goal,
            above_count, above, n);
        if (!in_list) {
            uint64_t before = 0;
            for (uint32_t i = lane; i < b; i += 64)
                before += masses[i];
            if (before != 0)
                atomicAdd(reinterpret_cast<unsigned long long*>(&sh.part_mass[wave]),
                          static_cast<unsigned long long>(before));
        }
        lo += uint64_t(b) << shift;
        const uint64_t last = lo + ((uint64_t(1) << shift) - 1);
        hi = hi < last ? hi : last;
        __syncthreads();
    }
    if (tid == 0)
        sh.n_small = 0;
    __syncthreads();
    for (uint32_t i = tid; i < sh.n_list && i < SM_LIST; i += SM_BLOCK) {
        const uint64_t v = sh.list[i];
        if (v >= lo && v <= hi) {
            const uint32_t at = atomicAdd(&sh.n_small, 1u);
            if (at < SM_SMALL)
                sh.small[at] = v;
        }
    }
    __syncthreads();
    n = n < SM_SMALL ? n : SM_SMALL;
    order_small(sh, n);
    // 64 of the order at a time, by every wave for itself
    uint64_t place = 0;
    for (uint32_t i = 0; i < n; i += 64) {
        const uint32_t at = i + uint32_t(lane_id());
        place = at < n ? sh.sorted[at] : 0;
        const double w = at < n ? row.weight(value_of(key_at(row, bin.key_hi, place))) : 0.0;
        const double incl = above + wave_inclusive_sum64(w);
        const uint64_t hits =
            __ballot(at < n && (at == n - 1 || (by_count ? above_count + at + 1 >= want : incl >= goal)));
        if (hits != 0) {
            const int l = __builtin_ctzll(hits);
            place = read_lane64(place, l);
            weight = read_lane64(incl, l);
            break;
        }
        above = read_lane64(incl, 63);
    }
    return place;
}

// One wave: the bin in which the count reaches `want` (by_count) or the weight `goal` (of the
// whole row's weight, its share -goal where it is negative), into sh.pick; the whole
// weight into sh.kept.
template <int TYPE>
__device__ __forceinline__ void choose_bin(const Row<TYPE>& row, SharedCuts& sh, bool by_count, uint32_t want,
                                           double goal)
{
    constexpr int N = SM_BINS / 64;
    double all = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        all += sh.bin_mass[lane_id() * N + i];
    all = read_lane64(wave_inclusive_sum64(all), 63);
    goal = goal > 0.0 ? goal : -goal * all;
    uint32_t above_count = 0, n = 0;
    double above = 0.0;
    const uint32_t b = pick<N>(
        sh.bin_count, [&](uint32_t i) { return sh.bin_mass[i]; }, by_count, want, goal, above_count, above, n);
    const Bin bin = make_bin(row, b);
    sh.kept = all;
    sh.pick.bin = bin;
    sh.pick.above_count = above_count;
    sh.pick.above = above;
    sh.pick.goal = goal;
    sh.pick.reached = above_count + n >= want ? 1u : 0u;
    // its elements' number, to a sixteenth of an octave
    sh.pick.about = uint32_t(sh.bin_mass[b] / __builtin_ldexp(sh.bin_weight[b], row.frac));
}
__device__ __forceinline__ Bin uniform_bin(const SharedCuts& sh)
{
    return Bin{uniform(sh.pick.bin.bin), uniform(sh.pick.bin.key_lo), uniform(sh.pick.bin.key_hi)};
}

// The histogram of one wave's share of a row.  A weight is the weight 2^(-b/8) of its bin
// times 2^(z/8), |z| <= 1/2, and the bin counts the second factor in units of 2^-frac: a
// polynomial of degree 6 (relative error 2^-48.9) into whose last step the rounding to an
// integer is folded, with no exponent to insert.  Below 2^-63.9 weights count as 0, for at most
// vocab 2^-63.9 of the sum (2^-46.9 in a row of 2^17, a quarter of the integers' rounding in any row): added to
// the last bin they would take turns at one address (peaked rows: 200 of 42000 logits took 55 us, against 27).
template <bool COUNTS, int TYPE>
__device__ __forceinline__ void fill_bins(const Row<TYPE>& row, uint64_t* mass, uint32_t* count, int first, int end)
{
    const double one = __builtin_ldexp(1.0, row.frac);
    uint32_t beyond = 0;
    const double last = uniform(-double(SM_BINS - 1) / SM_PER_OCTAVE / row.c);  // the last bin's middle
    const double c8 = uniform(row.c * SM_PER_OCTAVE), c0 = uniform(one + 0x1p52);
    const double c1 = uniform(one * 0x1.62e42fefa3aefp-4), c2 = uniform(one * 0x1.ebfbdff82c5e7p-9);
    const double c3 = uniform(one * 0x1.c6b08d5e4bb3bp-14), c4 = uniform(one * 0x1.3b2ab6f5687a9p-19);
    const double c5 = uniform(one * 0x1.5d8dfde822453p-25), c6 = uniform(one * 0x1.430d3b3f37695p-31);
    row.template for_steps<TYPE == LOGITS_F32 ? 1 : 2>(first, end, 1, [&](const float(&x)[SM_VEC], uint32_t) {
#pragma unroll
        for (int j = 0; j < SM_VEC; ++j) {
            const double d = double(x[j]) - row.top64;
            const double t = __builtin_fma(d, -c8, TO_INT);
            const double z = __builtin_fma(d, c8, t - TO_INT);
            double w = __builtin_fma(c6, z, c5);
            w = __builtin_fma(w, z, c4);
            w = __builtin_fma(w, z, c3);
            w = __builtin_fma(w, z, c2);
            w = __builtin_fma(w, z, c1);
            w = __builtin_fma(w, z, c0);
            const uint32_t b = uint32_t(__builtin_bit_cast(uint64_t, t));
            if (COUNTS)
                beyond += uint32_t(__builtin_popcountll(__ballot(d <= last && x[j] > -__builtin_inff())));
            if (d > last) {
                atomicAdd(reinterpret_cast<unsigned long long*>(&mass[b]),
                          static_cast<unsigned long long>(__builtin_bit_cast(uint64_t, w) & ((uint64_t(1) << 52) - 1)));
                if (COUNTS)
                    atomicAdd(&count[b], 1u);
            }
        }
    });
    if (COUNTS && beyond != 0 && lane_id() == 0)
        atomicAdd(&count[SM_BINS - 1], beyond);
}

// The cuts of a row that are not settled by a few candidates: a histogram of weights (and
// counts, for top-k) by log2 w, eight bins to the octave, tells which bin the cut lies in,
// and only that bin's elements are collected and ordered.  Weights are added to bins as
// integers, so that sums do not depend on the order of the atomics.
// Each wave takes a sixteenth of the row and keeps its own bins: with the cut known, the
// kept weight of each sixteenth is known too, and only the one with the token is read
// for the running sums.  FILLED: the bins of the sixteenths are there (sample_bins_kernel).
template <bool FILLED, int TYPE>
__device__ __forceinline__ void cut_row(const SampleCall& call, int64_t r, const Row<TYPE>& row, SharedCuts& sh,
                                        uint32_t k, double p, double least)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int share = (row.steps + SM_WAVES - 1) / SM_WAVES;
    const bool by_k = int64_t(k) < row.vocab, by_p = p < 1.0;
    Cut cut{0u, ~0u};  // keeps all
    bool in_parts = false, whole = false;
    Bin bin{0, 0, 0};
    uint64_t place = 0;
    if (by_k || by_p) {
        if (!FILLED)
            for (int i = lane; i < SM_BINS; i += 64)
                sh.mass[wave][i] = 0;
        if (tid < SM_BINS) {
            sh.bin_count[tid] = 0;
            sh.bin_weight[tid] = exp2_exact(-double(tid) / SM_PER_OCTAVE - double(row.frac));
        }
        __syncthreads();
        if (!FILLED) {
            const int first = wave * share, end = first + share < row.steps ? first + share : row.steps;
            if (by_k)
                fill_bins<true>(row, sh.mass[wave], sh.bin_count, first, end);
            else
                fill_bins<false>(row, sh.mass[wave], sh.bin_count, first, end);
            __syncthreads();
        }
        if (tid < SM_BINS) {
            uint64_t m = 0;
#pragma unroll
            for (int w = 0; w < SM_WAVES; ++w)
                m += sh.mass[w][tid];
            sh.bin_mass[tid] = double(m) * sh.bin_weight[tid];
            if (!by_k)
                sh.bin_count[tid] = m != 0 ? 1u : 0u;
        }
        __syncthreads();
        // top-k's cut first, then top-p's by the weight up to it
        double kept = 0.0;
        for (int which = by_k ? 0 : 1; which < (by_p ? 2 : 1); ++which) {
            const Bin last_bin = bin;
            const uint64_t last_place = place;
            const Cut last_cut = cut;
            __syncthreads();
            if (wave == 0)
                choose_bin(row, sh, which == 0, k, which == 0 ? 0.0 : last_cut.key != 0 ? p * kept : -p);
            __syncthreads();
            if (which == 0) {
                kept = uniform(sh.kept);
                if (uniform(sh.pick.reached) == 0u)
                    continue;  // no more elements than k
            }
            bin = uniform_bin(sh);
            place = cut_in_bin(row, sh, bin, which == 0, k, uniform(sh.pick.goal), uniform(sh.pick.above_count),
                               uniform(sh.pick.above), uniform(sh.pick.about), kept, whole);
            in_parts = true;
            cut = Cut{key_at(row, bin.key_hi, place), index_at(row, place)};
            if (which == 1 && last_cut.key != 0 && cut.keeps(last_cut.key, last_cut.index)) {
                // no later than top-k's own cut, which rounding may have put first
                in_parts = whole && last_bin.bin == bin.bin;
                place = last_place;
                cut = last_cut;
            }
        }
    }
    // where the cut's own element has the weight that min-p asks for, min-p drops nothing more
    if (cut.key != 0 && row.weight(value_of(cut.key)) >= least)
        least = 0.0;
    const auto kept_weight = [&](float x, uint32_t i) {
        const double w = cut.keeps(key_of(x), i) ? row.weight(x) : 0.0;
        return w >= least ? w : 0.0;
    };
    double total;
    const double u = double(call.uniforms[r]);
    // (u <= 0 and u >= 1 ask for the first and last weight of all, which the bins may have left out)
    if (in_parts && least == 0.0 && u > 0.0 && u < 1.0) {
        for (uint32_t i = tid; i < sh.n_list; i += SM_BLOCK) {
            const uint64_t v = sh.list[i];
            if (v <= place)
                atomicAdd(reinterpret_cast<unsigned long long*>(
                              &sh.part_mass[index_at(row, v) / uint32_t(share * SM_STEP)]),
                          static_cast<unsigned long long>(
                              row.fixed(row.below(value_of(key_at(row, bin.key_hi, v))), bin.bin)));
        }
        double sum = 0.0;
        for (uint32_t b = lane; b < bin.bin; b += 64)
            sum += double(sh.mass[wave][b]) * sh.bin_weight[b];
        sum = wave_inclusive_sum64(sum);
        if (lane == 63)
            sh.part_sum[wave] = sum;
        __syncthreads();
        // every wave for itself: the sixteenth with the token
        double v[1] = {lane < SM_WAVES ? sh.part_sum[lane] + row.unfixed(sh.part_mass[lane], bin.bin) : 0.0};
        double incl, before = 0.0;
        bool over;
        wave_sums(v, incl, total);
        const double goal = goal_of(u, total);
        const int over_at = wave_first_over(v, goal, incl, before, over), part = over_at < 0 ? 0 : over_at;
        const int begin = part * share, end = begin + share < row.steps ? begin + share : row.steps;
        // a wave takes one step in sixteen of it, adds up and hands the sums round
        const int per = (share + SM_WAVES - 1) / SM_WAVES;
        const int mine = begin + wave * per, mine_end = mine + per < end ? mine + per : end;
        sum = 0.0;
        row.template for_steps<1>(mine, mine_end, 1, [&](const float(&x)[SM_VEC], uint32_t idx) {
#pragma unroll
            for (int j = 0; j < SM_VEC; ++j)
                sum += kept_weight(x[j], idx + j);
        });
        sum = wave_inclusive_sum64(sum);
        __syncthreads();
        if (lane == 63)
            sh.part_sum[wave] = sum;
        __syncthreads();
        double rest;
        v[0] = lane < SM_WAVES ? sh.part_sum[lane] : 0.0;
        wave_sums(v, incl, rest);
        if (wave_first_over(v, goal, incl, before, over) == wave)
            write_token(call, r, row, wave_find_token<1>(row, mine, mine_end, before, goal, kept_weight), total);
        return;
    }
    const uint32_t token = find_in_order(row, sh.s, u, kept_weight, total);
    if (wave == 0)
        write_token(call, r, row, token, total);
}

// In how many parts a segment's values are looked at for the k-th largest: 1, its quarters (4) or its
// sixteenths (16), the fewest that number more than k, as long as they are at most 512: more parts give fewer
// candidates, or allow more of k, and cost up to 0.7 us.  1 row, bfloat16, top-k 50, with segments only against so:
// 4000 logits 17.9 us to 12.7, 8192 18.7 to 12.6, 16384 21.2 to 13.2, 32000 25.5 to 12.2; top-k 100 of 64000 33.6 to 15.8.
// Keeping the sixteenths costs short rows with top-k 0.5 to 1 us where they are not asked for.
__device__ __forceinline__ uint32_t parts_of(const SampleGrid& g, uint32_t k)
{
    const uint64_t segs = uint64_t(g.segs), twice = uint64_t(k) * 2;
    if (g.segs <= SM_FINE_SEGS && twice > segs * 4)
        return 16;
    return g.segs <= 128 && twice > segs ? 4 : 1;
}

// One wave: where the candidates of a row begin.  few: at most the k-th largest logit, which is the
// k-th largest of the largest values of the segments or of parts of them, to 16 bits of its key; else a little below the
// smallest logit that min-p may keep.  The segments' quarters with candidates go into
// sh.quarters (a quarter is the most that is read for one candidate).
template <int TYPE>
__device__ __forceinline__ void find_segments(const SampleGrid& g, int64_t rows, int64_t r, const Row<TYPE>& row, SharedCuts& sh,
                                              const QuarterTops& tops, bool few, uint32_t k, double least)
{
    float low;
    if (few) {
        static_assert(SM_PER_LANE == 8, "two segments' quarters, or eight segments");
        const uint32_t parts = parts_of(g, k);
        uint32_t key[SM_PER_LANE], at = 0;
#pragma unroll
        for (int j = 0; j < SM_PER_LANE; ++j)
            key[j] = key_of(clean(parts == 4 ? tops.quarter[j / 4][j % 4] : tops.v[j], row.inf)) >> 16;
        if (__builtin_expect(parts == 16, 0)) {
            const float* const fine = g.tops + (rows * 4 + r * 16) * g.segs;
#pragma unroll
            for (int j = 0; j < SM_PER_LANE; ++j) {
                const int i = j * 64 + lane_id();
                key[j] = key_of(clean(i < g.segs * 16 ? get(&fine[i]) : -__builtin_inff(), row.inf)) >> 16;
            }
        }
        const auto count = [&](auto lanes, uint32_t v) {
            uint32_t n = 0;
#pragma unroll
            for (int j = 0; j < decltype(lanes)::value; ++j)
                n += uint32_t(__builtin_popcountll(__ballot(key[j] >= v)));
            return n;
        };
        // two bits of the key at a time: the three counts do not wait for each other
        const auto narrow = [&](auto lanes) {
            for (int bit = 14; bit >= 0; bit -= 2) {
                const uint32_t a = at | 1u << bit, b = at | 2u << bit, c = at | 3u << bit;
                const uint32_t na = count(lanes, a), nb = count(lanes, b), nc = count(lanes, c);
                at = nc >= k ? c : nb >= k ? b : na >= k ? a : at;
            }
        };
        if (uint32_t(g.segs) * parts <= 64u * 4)
            narrow(std::integral_constant<int, 4>{});
        else
            narrow(std::integral_constant<int, SM_PER_LANE>{});
        const uint32_t lowest = at << 16;
        low = value_of(lowest > KEY_NEG_INF ? lowest : KEY_NEG_INF + 1);
    } else {
        const double x = double(row.top) + ::log(least) * LOG2E / row.c;
        low = float(x - 1e-6 * (__builtin_fabs(x) + __builtin_fabs(double(row.top))) - 1e-30);
        low = low > -__builtin_inff() ? low : value_of(KEY_NEG_INF + 1);
    }
    uint32_t flags = 0;
#pragma unroll
    for (int j = 0; j < SM_PER_LANE; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            flags |= clean(tops.quarter[j][q], row.inf) >= low ? 1u << (j * 4 + q) : 0u;
    static_assert(SM_PER_LANE * 4 <= 32, "a lane's quarters are bits of one word");
    const uint32_t mine = uint32_t(__builtin_popcount(flags));
    const uint32_t incl = wave_inclusive_scan<SumU32>(mine);
    uint32_t q = incl - mine;
    for (; flags != 0; flags &= flags - 1) {
        const int bit = __builtin_ctz(flags);
        sh.quarters[q++] = uint16_t(tops.seg(bit / 4) * 4 + bit % 4);
    }
    if (lane_id() == 63)
        sh.n_quarters = incl;
    sh.low = low;
}

// Rows whose cut lies within a few candidates (find_segments).  False when they are more
// than SM_SMALL.
template <int TYPE>
__device__ __forceinline__ bool cut_candidates(const SampleCall& call, const SampleGrid& g, int64_t r,
                                               const Row<TYPE>& row, SharedCuts& sh, uint32_t k, double p,
                                               double least)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(int(tid >> 6));
    const float low = uniform(sh.low);
    const uint32_t key_hi = key_of(row.top);
    constexpr int U = TYPE == LOGITS_F32 ? 2 : 4;
    // four quarters to a load of the wave, 16 lanes each
    const int quarters = int(uniform(sh.n_quarters)), todo = (quarters + 3) / 4 * g.seg_steps;
    for (int i = wave; i < todo; i += U * SM_WAVES) {
        Raw<TYPE> raw[U];
        uint32_t idx[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int t = i + j * SM_WAVES, four = g.seg_steps == 1 ? t : t / g.seg_steps;
            const int q = four * 4 + int(lane >> 4);
            raw[j].clear();
            idx[j] = 0;
            if (t < todo && q < quarters) {
                const int at = sh.quarters[q], step = (at >> 2) * g.seg_steps + (t - four * g.seg_steps);
                idx[j] = uint32_t(step) * SM_STEP + uint32_t(at & 3) * (SM_STEP / 4) + (lane & 15) * SM_VEC;
                if (idx[j] < row.vocab)
                    raw[j].load(row.p, idx[j], row.vocab);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (i + j * SM_WAVES >= todo)
                break;
            float x[SM_VEC];
            raw[j].unpack(x, row.inf);
            wave_append(
                &sh.n_small, x, [&](float v, int) { return v >= low; },
                [&](uint32_t at, float v, int m) {
                    if (at < SM_SMALL)
                        sh.small[at] = place_of(row, key_hi, key_of(v), idx[j] + uint32_t(m));
                });
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
    const uint32_t n = uniform(sh.n_small);
    if (n > SM_SMALL)
        return false;
    order_small(sh, n);
    // one wave, 64 of the order at a time: the kept ones are its first `keep`, of weight `total`
    if (wave == 0) {
        uint32_t keep = k < n ? k : n;
        double total = 0.0;
        for (uint32_t i = 0; i < keep; i += 64) {
            const uint32_t at = i + lane;
            const double w = at < keep ? row.weight(value_of(key_at(row, key_hi, sh.sorted[at]))) : 0.0;
            if (at < keep)
                sh.weight[at] = w;
            total += w;
        }
        if (p < 1.0) {
            const double goal = p * read_lane64(wave_inclusive_sum64(total), 63);
            double run = 0.0;
            for (uint32_t i = 0; i < keep; i += 64) {
                const uint32_t at = i + lane;
                const double up = run + wave_inclusive_sum64(at < keep ? sh.weight[at] : 0.0);
                const uint64_t hits = __ballot(at < keep && up >= goal);
                if (hits != 0)
                    keep = i + uint32_t(__builtin_ctzll(hits)) + 1u;
                run = read_lane64(up, 63);
            }
        }
        total = 0.0;
        for (uint32_t i = 0; i < keep; i += 64) {
            const uint32_t at = i + lane;
            const double w = at < keep ? sh.weight[at] : 0.0;
            const uint64_t drops = __ballot(at > 0 && at < keep && !(w >= least));
            if (drops != 0)
                keep = i + uint32_t(__builtin_ctzll(drops));
            total += at < keep ? w : 0.0;
        }
        sh.keep = keep;
        sh.kept = read_lane64(wave_inclusive_sum64(total), 63);
    }
    __syncthreads();
    // running sums in index order, each by a group of lanes
    const uint32_t keep = uniform(sh.keep);
    const double total = uniform(sh.kept);
    uint32_t group = 64;
    while (group > 1 && SM_BLOCK / group < keep)
        group >>= 1;
    const uint32_t e = tid / group, part = tid & (group - 1);
    double run = 0.0;
    uint32_t index = 0;
    if (e < keep) {
        index = index_at(row, sh.sorted[e]);
        for (uint32_t j = part; j < keep; j += group)
            run += index_at(row, sh.sorted[j]) <= index ? sh.weight[j] : 0.0;
    }
    for (uint32_t d = 1; d < group; d <<= 1)
        run += __shfl_xor(run, int(d));
    if (e < keep && part == 0) {
        if (run > goal_of(double(call.uniforms[r]), total))
            atomicMin(&sh.s.found, index);
        if (sh.weight[e] > 0.0)
            atomicMax(&sh.s.last, index);
    }
    __syncthreads();
    if (wave == 0)
        write_token(call, r, row, sh.s.found != ~0u ? sh.s.found : sh.s.last, total);
    return true;
}

// What top-p and min-p ask for in row r.
__device__ __forceinline__ double share_of(const SampleCall& call, int64_t r)
{
    const double p = call.top_p != nullptr ? double(call.top_p[r]) : 1.0;
    return uniform(p > 0.0 ? p : 0.0);
}
__device__ __forceinline__ double least_of(const SampleCall& call, int64_t r)
{
    const float p = call.min_p != nullptr ? call.min_p[r] : 0.0f;
    return uniform(p > 0.0f ? __builtin_fmin(double(p), 1.0) : 0.0);
}

template <int TYPE>
__global__ __launch_bounds__(SM_BLOCK) void sample_cut_kernel(SampleCall call, SampleGrid g)
{
    __shared__ SharedCuts sh;
    constexpr float NEG = -__builtin_inff();
    constexpr int U = TYPE == LOGITS_F32 ? 2 : 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t r = blockIdx.x % uint32_t(call.rows);
    const int part = int(blockIdx.x / uint32_t(call.rows));
    Row<TYPE> row = make_row<TYPE>(call, g, r);
    for (int i = 0; i < g.per_wave; i += U) {
        float top[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            top[u] = NEG;
        for (int j = 0; j < g.seg_steps; ++j) {
            Raw<TYPE> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int seg = (part * g.per_wave + i + u) * SM_WAVES + wave, s = seg * g.seg_steps + j;
                if (i + u < g.per_wave && s < g.steps)
                    raw[u].load_step(row.p, s, row.vocab);
                else
                    raw[u].clear();
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < SM_VEC; ++k) {
                    const float x = raw[u].at(k);
                    top[u] = x > top[u] ? x : top[u];
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int seg = (part * g.per_wave + i + u) * SM_WAVES + wave;
            const float m = row16_inclusive_scan<MaxF32>(top[u]);
            if ((lane & 15) == 15 && i + u < g.per_wave && seg < g.segs)
                put(&g.tops[(r * g.segs + seg) * 4 + (lane >> 4)], m);
        }
    }
    // (out of the way of long rows: the same again for each four lanes, of loads that are in the L1 now)
    if (__builtin_expect(g.segs <= SM_FINE_SEGS && call.top_k != nullptr, 0)) {
#pragma unroll 1
        for (int i = 0; i < g.per_wave; ++i) {
            const int seg = (part * g.per_wave + i) * SM_WAVES + wave;
            if (seg >= g.segs)
                break;
            Raw<TYPE> raw;
            raw.load_step(row.p, seg, row.vocab);
            float four = NEG;
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k) {
                const float x = raw.at(k);
                four = x > four ? x : four;
            }
            four = MaxF32::apply(four, dpp_move<DPP_QUAD_SWAP1, 0xf>(NEG, four));
            four = MaxF32::apply(four, dpp_move<DPP_QUAD_SWAP2, 0xf>(NEG, four));
            if ((lane & 3) == 3)
                put(&g.tops[call.rows * g.segs * 4 + (r * g.segs + seg) * 16 + (lane >> 2)], four);
        }
    }
    stores_done();
    __syncthreads();
    if (tid == 0)
        sh.s.arrived = count_in(&g.counters[r * SM_COUNTER], uint32_t(g.parts)) ? 1u : 0u;
    __syncthreads();
    if (uniform(sh.s.arrived) == 0u)
        return;

    uint32_t k = ~0u;
    if (call.top_k != nullptr && call.top_k[r] > 0)
        k = uint32_t(call.top_k[r]);
    const double p = share_of(call, r), least = least_of(call, r);
    // few enough that the k-th largest of n parts' values leaves few candidates: of logits in any order
    // about -n ln(1 - k / n), which SM_SMALL has to hold (with k <= 3/4 n and 240 at most 440); in a
    // short row the bins take no longer from k = 128 on (200 of 16384: 21.2 us, with candidates 23.7)
    const uint32_t parts = parts_of(g, k), n = uint32_t(g.segs) * parts;
    const bool few = k <= (parts == 16 ? 128u : 240u) && k * 4 <= n * 3;
    const bool candidates = few || (p >= 1.0 && least > 0.0);
    // one wave (the others would only take its turns), then all
    if (wave == 0) {
        QuarterTops tops;
        const float top = tops.load(g, r);
        const bool done = settle(call, g, r, row, tops, top);
        sh.n_small = 0, sh.s.found = ~0u, sh.s.last = 0;
        const bool later = !done && g.split && p < 1.0;
        sh.goes_on = done || later ? 0u : 1u;
        sh.top = top;
        if (g.split && lane == 0)
            g.split_tops[r] = later ? top : __builtin_nanf("");
        if (!done && candidates)
            find_segments(g, call.rows, r, row, sh, tops, few, k, least);
    }
    __syncthreads();
    if (uniform(sh.goes_on) == 0u)
        return;
    row.set_top(uniform(sh.top));
    row.set_temperature(call.temperature[r]);
    if (!(candidates && cut_candidates(call, g, r, row, sh, k, p, least)))
        cut_row<false>(call, r, row, sh, k, p, least);
}

// A second launch for few rows with top-p alone: the rows' bins, each sixteenth of a row by a block,
// and the cut by the row's last one.  The bins are integers, so they are those that one block makes.
template <int TYPE>
__global__ __launch_bounds__(SM_BLOCK) void sample_bins_kernel(SampleCall call, SampleGrid g)
{
    __shared__ SharedCuts sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t r = blockIdx.x % uint32_t(call.rows);
    const int part = int(blockIdx.x / uint32_t(call.rows));
    const float top = uniform(g.split_tops[r]);
    if (top != top)
        return;
    Row<TYPE> row = make_row<TYPE>(call, g, r);
    row.set_top(top);
    row.set_temperature(call.temperature[r]);
    for (int i = lane; i < SM_BINS; i += 64)
        sh.mass[wave][i] = 0;
    __syncthreads();
    // a sixteenth of the row, as in cut_row, and a sixteenth of that to a wave
    const int share = (row.steps + SM_WAVES - 1) / SM_WAVES, begin = part * share;
    const int end = begin + share < row.steps ? begin + share : row.steps;
    const int per = (share + SM_WAVES - 1) / SM_WAVES, first = begin + wave * per;
    fill_bins<false>(row, sh.mass[wave], sh.bin_count, first, first + per < end ? first + per : end);
    __syncthreads();
    uint64_t* const masses = g.masses + r * (SM_WAVES * SM_BINS);
    if (tid < SM_BINS) {
        uint64_t m = 0;
#pragma unroll
        for (int w = 0; w < SM_WAVES; ++w)
            m += sh.mass[w][tid];
        put(&masses[part * SM_BINS + tid], m);
    }
    stores_done();
    __syncthreads();
    if (tid == 0) {
        sh.s.arrived = count_in(&g.counters[r * SM_COUNTER], uint32_t(SM_WAVES)) ? 1u : 0u;
        sh.n_small = 0, sh.s.found = ~0u, sh.s.last = 0;
    }
    __syncthreads();
    if (uniform(sh.s.arrived) == 0u)
        return;
#pragma unroll
    for (int i = 0; i < SM_WAVES * SM_BINS / SM_BLOCK; ++i)
        (&sh.mass[0][0])[i * SM_BLOCK + tid] = get(&masses[i * SM_BLOCK + tid]);
    cut_row<true>(call, r, row, sh, ~0u, share_of(call, r), least_of(call, r));
}

// ---------------------------------------------------------------- host side
static size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

static int64_t row_segs(int64_t vocab)
{
    const int64_t steps = (vocab + SM_STEP - 1) / SM_STEP;
    return steps < SM_SEGS ? steps : SM_SEGS;
}

// header | a counter for each row of a launch | 16 bytes for each segment: the segments' sums and
// behind them their largest values, or their quarters' largest values | 64 bytes more for each segment where a row has few | the largest value and the
// bins of the rows that sample_bins_kernel may take.  The counters' place is the same for every call, so that nothing else is ever written
// there and they stay 0 between calls of any sizes.
static size_t row_cells(int64_t rows, int64_t vocab)
{
    return size_t(rows < SM_ROWS ? rows : SM_ROWS) * size_t(row_segs(vocab));
}

static size_t fine_bytes(int64_t rows, int64_t vocab)
{
    return row_segs(vocab) <= SM_FINE_SEGS ? round256(row_cells(rows, vocab) * 64) : 0;
}
constexpr size_t SM_MASSES = size_t(SM_WAVES) * SM_BINS * 8;  // bytes of a row
static size_t split_rows(int64_t rows) { return size_t(rows < SM_SPLIT_ROWS ? rows : SM_SPLIT_ROWS); }

size_t sample_workspace_bytes(int64_t rows, int64_t vocab)
{
    const size_t cells = row_cells(rows, vocab);
    return 256 + SM_ROWS * SM_COUNTER * 4 + round256(cells * 16) + fine_bytes(rows, vocab) + SM_SPLIT_ROWS * 4 + split_rows(rows) * SM_MASSES;
}

template <int TYPE>
static void launch_type(const SampleCall& call, const SampleGrid& g, bool cuts, hipStream_t stream)
{
    const dim3 grid(unsigned(call.rows * g.parts));
    if (cuts) {
        sample_cut_kernel<TYPE><<<grid, SM_BLOCK, 0, stream>>>(call, g);
        if (g.split)
            sample_bins_kernel<TYPE><<<dim3(unsigned(call.rows * SM_WAVES)), SM_BLOCK, 0, stream>>>(call, g);
    } else {
        sample_all_kernel<TYPE><<<grid, SM_ALL_BLOCK, 0, stream>>>(call, g);
    }
}

hipError_t launch_sample(const SampleCall& call, int type, void* ws, hipStream_t stream)
{
    if (call.rows == 0)
        return hipSuccess;
    const bool cuts = call.top_k != nullptr || call.top_p != nullptr || call.min_p != nullptr;
    const int64_t rows = call.rows < SM_ROWS ? call.rows : SM_ROWS;  // of a launch
    SampleGrid g;
    g.steps = int((call.vocab + SM_STEP - 1) / SM_STEP);
    g.seg_steps = g.steps > SM_SEGS ? (g.steps + SM_SEGS - 1) / SM_SEGS : 1;
    // without cuts, where there are rows enough: four steps to a segment, for one sum across the wave to all four
    if (!cuts && rows * g.steps >= 4 * 8192 && g.seg_steps < 4)
        g.seg_steps = 4;
    g.segs = (g.steps + g.seg_steps - 1) / g.seg_steps;
    // Without cuts up to four segments to a wave, once that leaves 8192 waves.  With cuts no more blocks than CUs (the LDS holds one block a CU) where
    // that leaves each row one, in parts that fill the waves.
    if (cuts) {
        const int64_t blocks = rows < SM_CUS ? SM_CUS / rows : 1, shares = (g.segs + SM_WAVES - 1) / SM_WAVES;
        g.per_wave = int((shares + blocks - 1) / blocks);
    } else {
        g.per_wave = int(rows * g.segs >= 4 * 8192 ? 4 : rows * g.segs >= 2 * 8192 ? 2 : 1);
    }
    const int waves = cuts ? SM_WAVES : SM_ALL_BLOCK / 64;
    if (g.per_wave < 1)
        g.per_wave = 1;
    g.parts = (g.segs + waves * g.per_wave - 1) / (waves * g.per_wave);
    if (g.parts < 1)
        g.parts = 1;
    char* at = static_cast<char*>(ws) + 256;
    g.counters = reinterpret_cast<uint32_t*>(at);
    at += SM_ROWS * SM_COUNTER * 4;
    g.sums = reinterpret_cast<double*>(at);
    g.tops = reinterpret_cast<float*>(cuts ? at : at + size_t(rows) * size_t(g.segs) * 8);
    at += round256(row_cells(call.rows, call.vocab) * 16);
    at += fine_bytes(call.rows, call.vocab);
    g.split_tops = reinterpret_cast<float*>(at);
    g.masses = reinterpret_cast<uint64_t*>(at + SM_SPLIT_ROWS * 4);
    g.split = call.top_p != nullptr && call.top_k == nullptr && call.rows <= SM_SPLIT_ROWS && g.steps >= SM_SPLIT_STEPS;
    SampleCall now = call;
    for (int64_t r = 0; r < call.rows; r += rows) {
        now.rows = call.rows - r < rows ? call.rows - r : rows;
        if (type == LOGITS_F32)
            launch_type<LOGITS_F32>(now, g, cuts, stream);
        else if (type == LOGITS_F16)
            launch_type<LOGITS_F16>(now, g, cuts, stream);
        else
            launch_type<LOGITS_BF16>(now, g, cuts, stream);
        const int64_t size = type == LOGITS_F32 ? 4 : 2;
        now.logits = static_cast<const char*>(now.logits) + rows * now.stride * size;
        now.uniforms += rows;
        now.temperature += rows;
        now.top_k += now.top_k != nullptr ? rows : 0;
        now.top_p += now.top_p != nullptr ? rows : 0;
        now.min_p += now.min_p != nullptr ? rows : 0;
        now.tokens += rows;
        now.logprobs += now.logprobs != nullptr ? rows : 0;
    }
    return hipGetLastError();
}

}  // namespace ls
