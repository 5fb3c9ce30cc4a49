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
// 64 bits: a double multiply-add issues at the rate of a single one on this GPU, and 2^f
// is a polynomial of degree 10.
//
// The cuts are found by value, without sorting the row: a histogram of weights and
// counts over 2048 bins of log2 w (32 to the octave) tells which bin the cut lies in, and
// only that bin's elements are collected in LDS and sorted.  Weights are added to bins as
// integers of 2^-frac of the bin's octave, so that the sums do not depend on the order
// of the atomics.  A bin of more elements than the list holds is cut into 2048 ranges
// of its keys, and so on, until the list holds them or they are all equal.
#include "ls_device.hpp"
#include "ls_internal.hpp"

namespace ls {

constexpr int SM_BLOCK = 1024;
constexpr int SM_WAVES = SM_BLOCK / 64;
constexpr int SM_VEC = 8;                   // consecutive logits per lane and step
constexpr int SM_STEP = 64 * SM_VEC;        // consecutive logits per wave and step
constexpr int SM_SEGS = 1024;               // most segments of a row
constexpr int SM_BINS = 2048;
constexpr int SM_PER_OCTAVE = 32;
constexpr int SM_OCTAVES = SM_BINS / SM_PER_OCTAVE;
constexpr int SM_LIST = 4096;               // elements of one bin that are sorted in LDS
static_assert(SM_SEGS == SM_BLOCK && SM_BINS == 2 * SM_BLOCK, "one segment and two bins per thread");

// 2^y for y <= 0 (NaN counts as -inf): 2^n p(f), n the nearest integer, |f| <= 1/2.
// p interpolates 2^f at Chebyshev nodes (p(0) = 1); its largest relative error is
// 2^-50.6.  Results below 2^-1074 are 0.
__device__ __forceinline__ double exp2_neg(double y)
{
    y = __builtin_fmax(y, -1100.0);
    const double n = __builtin_rint(y);
    const double f = y - n;
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
    p = __builtin_fma(p, f, 1.0);
    return __builtin_ldexp(p, int(n));
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

template <int TYPE>
__device__ __forceinline__ float widen(uint32_t half)
{
    if constexpr (TYPE == LOGITS_BF16)
        return from_bits<float>(half << 16);
    else
        return float(__builtin_bit_cast(_Float16, uint16_t(half)));
}

// Logits idx .. idx+7 of a row, NaN and what lies past the end as -inf.  Rows start at any
// multiple of the element's size.
template <int TYPE>
__device__ __forceinline__ void load_logits(const void* row, int64_t idx, int64_t vocab, float (&x)[SM_VEC])
{
    constexpr float NEG = -__builtin_inff();
    if constexpr (TYPE == LOGITS_F32) {
        typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
        const float* p = static_cast<const float*>(row) + idx;
        if (idx + SM_VEC <= vocab) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = a[k];
                x[4 + k] = b[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k)
                x[k] = idx + k < vocab ? p[k] : NEG;
        }
    } else {
        typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(2)));
        const uint16_t* p = static_cast<const uint16_t*>(row) + idx;
        if (idx + SM_VEC <= vocab) {
            const u32x4a a = *reinterpret_cast<const u32x4a*>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = widen<TYPE>(a[k] & 0xffffu);
                x[2 * k + 1] = widen<TYPE>(a[k] >> 16);
            }
        } else {
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k)
                x[k] = idx + k < vocab ? widen<TYPE>(p[k]) : NEG;
        }
    }
#pragma unroll
    for (int k = 0; k < SM_VEC; ++k)
        x[k] = x[k] == x[k] ? x[k] : NEG;
}

// One past the last kept element in the order: kept are keys above `key`, and equal
// ones up to `index`.
struct Cut {
    uint32_t key;
    uint32_t index;
    __device__ __forceinline__ bool keeps(uint32_t k, uint32_t i) const { return k > key || (k == key && i <= index); }
};

struct SampleLds {
    uint64_t mass[SM_BINS];
    uint32_t count[SM_BINS];
    uint64_t list[SM_LIST];     // ~key << 32 | index: ascending is the order
    double seg[SM_SEGS];
    double wave_f64[SM_WAVES];
    uint32_t wave_u32[SM_WAVES];
    uint32_t n_list, bin, tie_index, best;
    double above, total;
    uint32_t above_count, key_lo, key_hi;
};

// What a block knows of its row.
template <int TYPE>
struct Row {
    const void* p;
    int64_t vocab;
    int seg_steps;   // steps per segment
    int segs;
    float top;
    double c;        // log2 e / t
    int frac;        // bits below the octave's unit in the bins' integers

    // log2 of the weight, at most 0; the same in every pass, and monotone in x
    __device__ __forceinline__ double log2w(float x) const
    {
        return x == top ? 0.0 : (double(x) - double(top)) * c;
    }
    __device__ __forceinline__ double weight(float x) const { return exp2_neg(log2w(x)); }
    __device__ __forceinline__ int bin(double y) const
    {
        const float s = float(__builtin_fmin(-y, double(SM_OCTAVES)));
        const int b = int(s * float(SM_PER_OCTAVE));
        return b < SM_BINS ? b : SM_BINS - 1;
    }
    __device__ __forceinline__ uint64_t fixed(double w, int b) const
    {
        return uint64_t(__builtin_ldexp(w, b / SM_PER_OCTAVE + frac) + 0.5);
    }
    __device__ __forceinline__ double unfixed(uint64_t m, int b) const
    {
        return __builtin_ldexp(double(m), -(b / SM_PER_OCTAVE + frac));
    }

    // f(x[8], index of x[0]) over the whole row: a wave takes every SM_WAVES-th segment
    template <class F>
    __device__ __forceinline__ void for_each(F f) const
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        for (int s = wave; s < segs; s += SM_WAVES) {
            for (int j = 0; j < seg_steps; ++j) {
                const int64_t idx = (int64_t(s) * seg_steps + j) * SM_STEP + lane * SM_VEC;
                if (idx >= vocab)
                    break;
                float x[SM_VEC];
                load_logits<TYPE>(p, idx, vocab, x);
                f(x, idx);
            }
        }
    }
};

__device__ __forceinline__ float wave_max(float v)
{
    for (int d = 32; d > 0; d >>= 1)
        v = __builtin_fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Running sums over the block's threads, in thread order; `total` to all.
__device__ __forceinline__ double block_inclusive_sum(double v, SampleLds& lds, double& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double incl = wave_inclusive_sum64(v);
    __syncthreads();
    if (lane == 63)
        lds.wave_f64[wave] = incl;
    __syncthreads();
    double before = 0.0;
    total = 0.0;
    for (int w = 0; w < SM_WAVES; ++w) {
        before = w == wave ? total : before;
        total += lds.wave_f64[w];
    }
    return before + incl;
}
__device__ __forceinline__ uint32_t block_inclusive_sum(uint32_t v, SampleLds& lds, uint32_t& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t incl = wave_inclusive_scan<SumU32>(v);
    __syncthreads();
    if (lane == 63)
        lds.wave_u32[wave] = incl;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
    for (int w = 0; w < SM_WAVES; ++w) {
        before = w == wave ? total : before;
        total += lds.wave_u32[w];
    }
    return before + incl;
}

// The first index, in index order, at which the running sum of f(x, index) exceeds
// goal(total); the last one of nonzero weight if none does.  total and that index to all.
template <int TYPE, class F, class G>
__device__ int64_t find_in_order(const Row<TYPE>& row, SampleLds& lds, F f, G goal_of, double& total)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __syncthreads();
    for (int s = wave; s < row.segs; s += SM_WAVES) {
        double sum = 0.0;
        for (int j = 0; j < row.seg_steps; ++j) {
            const int64_t idx = (int64_t(s) * row.seg_steps + j) * SM_STEP + lane * SM_VEC;
            if (idx < row.vocab) {
                float x[SM_VEC];
                load_logits<TYPE>(row.p, idx, row.vocab, x);
#pragma unroll
                for (int k = 0; k < SM_VEC; ++k)
                    sum += f(x[k], uint32_t(idx + k));
            }
        }
        sum = wave_inclusive_sum64(sum);
        if (lane == 63)
            lds.seg[s] = sum;
    }
    if (tid == 0) {
        lds.bin = ~0u;
        lds.best = 0;
    }
    __syncthreads();
    const double mine = tid < row.segs ? lds.seg[tid] : 0.0;
    const double incl = block_inclusive_sum(mine, lds, total);
    const double goal = goal_of(total);
    if (incl > goal)
        atomicMin(&lds.bin, uint32_t(tid));
    if (mine > 0.0)
        atomicMax(&lds.best, uint32_t(tid));
    lds.seg[tid] = incl;
    __syncthreads();
    const int s = int(lds.bin != ~0u ? lds.bin : lds.best);
    if (wave == 0) {
        double run = s > 0 ? lds.seg[s - 1] : 0.0;
        int64_t found = -1, last = 0;
        for (int j = 0; j < row.seg_steps && found < 0; ++j) {
            const int64_t idx = (int64_t(s) * row.seg_steps + j) * SM_STEP + lane * SM_VEC;
            float x[SM_VEC];
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k)
                x[k] = -__builtin_inff();
            if (idx < row.vocab)
                load_logits<TYPE>(row.p, idx, row.vocab, x);
            double w[SM_VEC], sum = 0.0;
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k) {
                w[k] = idx + k < row.vocab ? f(x[k], uint32_t(idx + k)) : 0.0;
                sum += w[k];
            }
            const double lane_incl = wave_inclusive_sum64(sum);
            double r = run + (lane_incl - sum);
            int hit = SM_VEC, end = -1;
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k) {
                r += w[k];
                if (w[k] > 0.0) {
                    end = k;
                    if (r > goal && hit == SM_VEC)
                        hit = k;
                }
            }
            const uint64_t hits = __ballot(hit < SM_VEC), ends = __ballot(end >= 0);
            const int64_t step0 = (int64_t(s) * row.seg_steps + j) * SM_STEP;
            if (hits != 0) {
                const int l = __builtin_ctzll(hits);
                found = step0 + l * SM_VEC + read_lane(hit, l);
            }
            if (ends != 0) {
                const int l = 63 - __builtin_clzll(ends);
                last = step0 + l * SM_VEC + read_lane(end, l);
            }
            run += read_lane64(lane_incl, 63);
        }
        if (lane == 0)
            lds.tie_index = uint32_t(found >= 0 ? found : last);
    }
    __syncthreads();
    return int64_t(lds.tie_index);
}

// Ascending sort of the list's first n entries.
__device__ void sort_list(SampleLds& lds, uint32_t n)
{
    uint32_t size = 2;
    while (size < n)
        size <<= 1;
    for (uint32_t i = n + threadIdx.x; i < size; i += SM_BLOCK)
        lds.list[i] = ~uint64_t(0);
    for (uint32_t run = 2; run <= size; run <<= 1) {
        for (uint32_t d = run >> 1; d > 0; d >>= 1) {
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < size / 2; i += SM_BLOCK) {
                const uint32_t a = 2 * i - (i & (d - 1)), b = a + d;
                const uint64_t va = lds.list[a], vb = lds.list[b];
                if ((va > vb) == ((a & run) == 0)) {
                    lds.list[a] = vb;
                    lds.list[b] = va;
                }
            }
        }
    }
    __syncthreads();
}

// Puts the bins' counts and weights together: picks the bin in which the running count
// reaches `want` (by_count) or the running weight reaches `goal`, into lds.bin, and what
// lies before it into lds.above / lds.above_count.  `total` and `elements` are the sums.
template <class W>
__device__ void pick_bin(SampleLds& lds, W weight_of, bool by_count, uint32_t want, double goal, double base,
                         double& total, uint32_t& elements)
{
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0)
        lds.bin = ~0u, lds.best = 0;
    const uint32_t n0 = lds.count[2 * tid], n1 = lds.count[2 * tid + 1];
    const double m0 = weight_of(lds.mass[2 * tid], 2 * tid), m1 = weight_of(lds.mass[2 * tid + 1], 2 * tid + 1);
    const uint32_t n_incl = block_inclusive_sum(n0 + n1, lds, elements);
    const double m_incl = block_inclusive_sum(m0 + m1, lds, total) + base;
    const uint32_t n_a = n_incl - n1, n_before = n_a - n0;
    const double m_a = m_incl - m1, m_before = m_a - m0;
    if (n1 != 0)
        atomicMax(&lds.best, uint32_t(2 * tid + 1));
    else if (n0 != 0)
        atomicMax(&lds.best, uint32_t(2 * tid));
    if (n0 != 0 && (by_count ? n_a >= want : m_a >= goal))
        atomicMin(&lds.bin, uint32_t(2 * tid));
    else if (n1 != 0 && (by_count ? n_incl >= want : m_incl >= goal))
        atomicMin(&lds.bin, uint32_t(2 * tid + 1));
    __syncthreads();
    if (tid == 0 && lds.bin == ~0u)
        lds.bin = lds.best;  // rounding at the very end of the sums
    __syncthreads();
    const int b = int(lds.bin);
    if (b / 2 == tid) {
        lds.above = b & 1 ? m_a : m_before;
        lds.above_count = b & 1 ? n_a : n_before;
    }
    __syncthreads();
}

// The cut inside one bin of the row's histogram (`bin`, holding `n` elements): the
// element that makes the count reach `want` (by_count) or the weight reach `goal`, where
// `above_count` and `above` lie in front of the bin.  Returns the weight up to and
// including the cut.
template <int TYPE>
__device__ Cut cut_in_bin(const Row<TYPE>& row, SampleLds& lds, int bin, uint32_t n, bool by_count, uint32_t want,
                          double goal, uint32_t above_count, double above, double& weight)
{
    const int tid = threadIdx.x;
    const double inf = __builtin_inf();
    uint32_t lo = 0, hi = ~0u;  // the keys looked at
    if (n > SM_LIST) {
        __syncthreads();
        if (tid == 0)
            lds.key_lo = ~0u, lds.key_hi = 0;
        __syncthreads();
        uint32_t klo = ~0u, khi = 0;
        row.for_each([&](const float(&x)[SM_VEC], int64_t) {
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k) {
                if (x[k] != -inf && row.bin(row.log2w(x[k])) == bin) {
                    const uint32_t key = key_of(x[k]);
                    klo = key < klo ? key : klo;
                    khi = key > khi ? key : khi;
                }
            }
        });
        atomicMin(&lds.key_lo, klo);
        atomicMax(&lds.key_hi, khi);
        __syncthreads();
        lo = lds.key_lo;
        hi = lds.key_hi;
    }
    while (n > SM_LIST && lo != hi) {
        const uint32_t span = hi - lo;
        const int bits = 32 - __builtin_clz(span);
        const int shift = bits > 11 ? bits - 11 : 0;  // 2048 ranges
        __syncthreads();
        for (int i = tid; i < SM_BINS; i += SM_BLOCK) {
            lds.mass[i] = 0;
            lds.count[i] = 0;
        }
        __syncthreads();
        row.for_each([&](const float(&x)[SM_VEC], int64_t) {
#pragma unroll
            for (int k = 0; k < SM_VEC; ++k) {
                const uint32_t key = key_of(x[k]);
                if (key >= lo && key <= hi) {
                    const uint32_t b = (hi - key) >> shift;
                    atomicAdd(&lds.count[b], 1u);
                    atomicAdd(reinterpret_cast<unsigned long long*>(&lds.mass[b]),
                              static_cast<unsigned long long>(row.fixed(row.weight(x[k]), bin)));
                }
            }
        });
        double total;
        uint32_t elements;
        pick_bin(
            lds, [&](uint64_t m, int) { return row.unfixed(m, bin); }, by_count, want - above_count, goal, above, total,
            elements);
        const uint32_t b = lds.bin;
        above = lds.above;
        above_count += lds.above_count;
        n = lds.count[b];
        hi -= b << shift;
        const uint32_t width = (1u << shift) - 1u;
        lo = hi - lo > width ? hi - width : lo;
        __syncthreads();
    }
    if (n > SM_LIST) {
        // equal values: the cut falls at a count of them, in index order
        const double w = row.weight(value_of(lo));
        uint32_t take = n;
        if (by_count) {
            take = want - above_count;
        } else if (w > 0.0) {
            const double m = __builtin_ceil((goal - above) / w);
            take = m < 1.0 ? 1u : (m < double(n) ? uint32_t(m) : n);
        }
        double ties;
        const uint32_t key = lo;
        const int64_t at = find_in_order(
            row, lds, [&](float x, uint32_t) { return key_of(x) == key ? 1.0 : 0.0; },
            [&](double) { return double(take) - 0.5; }, ties);
        weight = above + w * double(take);
        return Cut{key, uint32_t(at)};
    }
    __syncthreads();
    if (tid == 0)
        lds.n_list = 0, lds.best = ~0u;
    __syncthreads();
    row.for_each([&](const float(&x)[SM_VEC], int64_t idx) {
#pragma unroll
        for (int k = 0; k < SM_VEC; ++k) {
            const uint32_t key = key_of(x[k]);
            if (x[k] != -inf && key >= lo && key <= hi && row.bin(row.log2w(x[k])) == bin) {
                const uint32_t at = atomicAdd(&lds.n_list, 1u);
                if (at < SM_LIST)
                    lds.list[at] = (uint64_t(~key) << 32) | uint32_t(idx + k);
            }
        }
    });
    __syncthreads();
    n = lds.n_list < SM_LIST ? lds.n_list : SM_LIST;
    sort_list(lds, n);
    constexpr int PER = SM_LIST / SM_BLOCK;
    double w[PER], sum = 0.0, total;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const uint32_t i = tid * PER + k;
        w[k] = i < n ? row.weight(value_of(~uint32_t(lds.list[i] >> 32))) : 0.0;
        sum += w[k];
    }
    const double incl = block_inclusive_sum(sum, lds, total);
    double r = above + (incl - sum);
    uint32_t at = ~0u;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const uint32_t i = tid * PER + k;
        r += w[k];
        if (at == ~0u && i < n && (by_count ? above_count + i + 1 >= want : r >= goal))
            at = i;
    }
    if (at != ~0u)
        atomicMin(&lds.best, at);
    __syncthreads();
    at = lds.best != ~0u ? lds.best : n - 1;
    r = above + (incl - sum);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        r += w[k];
        if (uint32_t(tid * PER + k) == at)
            lds.total = r;
    }
    __syncthreads();
    weight = lds.total;
    const uint64_t e = lds.list[at];
    return Cut{~uint32_t(e >> 32), uint32_t(e)};
}

// One block per row.
template <int TYPE>
__global__ __launch_bounds__(SM_BLOCK) void sample_row_kernel(SampleCall call)
{
    __shared__ SampleLds lds;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const double inf = __builtin_inf();
    const int64_t r = blockIdx.x;
    constexpr int SIZE = TYPE == LOGITS_F32 ? 4 : 2;

    Row<TYPE> row;
    row.p = static_cast<const char*>(call.logits) + r * call.stride * SIZE;
    row.vocab = call.vocab;
    const int64_t steps = (call.vocab + SM_STEP - 1) / SM_STEP;
    row.seg_steps = int((steps + SM_SEGS - 1) / SM_SEGS);
    row.segs = row.seg_steps > 0 ? int((steps + row.seg_steps - 1) / row.seg_steps) : 0;
    int bits = 0;
    while (bits < 31 && (int64_t(1) << bits) < call.vocab)
        ++bits;
    row.frac = 62 - bits < 45 ? 62 - bits : 45;

    float top = -__builtin_inff();
    row.for_each([&](const float(&x)[SM_VEC], int64_t) {
#pragma unroll
        for (int k = 0; k < SM_VEC; ++k)
            top = x[k] > top ? x[k] : top;
    });
    top = wave_max(top);
    if (lane == 0)
        lds.wave_u32[wave] = to_bits(top);
    __syncthreads();
    for (int w = 0; w < SM_WAVES; ++w)
        top = __builtin_fmaxf(top, from_bits<float>(lds.wave_u32[w]));
    row.top = top;
    if (top == -__builtin_inff()) {
        if (tid == 0) {
            call.tokens[r] = -1;
            if (call.logprobs != nullptr)
                call.logprobs[r] = -__builtin_inff();
        }
        return;
    }
    const float t = call.temperature[r];
    if (!(t > 0.0f)) {
        if (tid == 0)
            lds.best = ~0u;
        __syncthreads();
        uint32_t first = ~0u;
        row.for_each([&](const float(&x)[SM_VEC], int64_t idx) {
#pragma unroll
            for (int k = SM_VEC - 1; k >= 0; --k)
                if (x[k] == top && uint32_t(idx + k) < first)
                    first = uint32_t(idx + k);
        });
        if (first != ~0u)
            atomicMin(&lds.best, first);
        __syncthreads();
        if (tid == 0) {
            call.tokens[r] = int64_t(lds.best);
            if (call.logprobs != nullptr)
                call.logprobs[r] = 0.0f;
        }
        return;
    }
    row.c = 0x1.71547652b82fep+0 / double(t);

    // the cuts in force
    uint32_t k = ~0u;
    if (call.top_k != nullptr && call.top_k[r] > 0)
        k = uint32_t(call.top_k[r]);
    double p = 2.0;
    if (call.top_p != nullptr) {
        p = double(call.top_p[r]);
        p = p > 0.0 ? p : 0.0;
    }
    double least = 0.0;
    if (call.min_p != nullptr && call.min_p[r] > 0.0f)
        least = __builtin_fmin(double(call.min_p[r]), 1.0);

    Cut cut{0u, ~0u};  // keeps all
    if (k < uint64_t(call.vocab) || p < 1.0) {
        __syncthreads();
        for (int i = tid; i < SM_BINS; i += SM_BLOCK) {
            lds.mass[i] = 0;
            lds.count[i] = 0;
        }
        __syncthreads();
        row.for_each([&](const float(&x)[SM_VEC], int64_t) {
#pragma unroll
            for (int j = 0; j < SM_VEC; ++j) {
                if (x[j] != -inf) {
                    const double y = row.log2w(x[j]);
                    const int b = row.bin(y);
                    atomicAdd(&lds.count[b], 1u);
                    if (p < 1.0)
                        atomicAdd(reinterpret_cast<unsigned long long*>(&lds.mass[b]),
                                  static_cast<unsigned long long>(row.fixed(exp2_neg(y), b)));
                }
            }
        });
        const auto in_bin = [&](uint64_t m, int b) { return row.unfixed(m, b); };
        double total;
        uint32_t elements;
        pick_bin(lds, in_bin, true, k, 0.0, 0.0, total, elements);
        const uint32_t kb = lds.bin, kn = lds.count[kb], k_above = lds.above_count;
        const double m_above = lds.above;
        const bool cut_k = k < elements;
        double pmass = total;
        uint32_t pb = 0, pn = 0, p_above = 0;
        double p_m_above = 0.0;
        // the histogram is reused by the refinements, so a cut by k that top-p follows keeps to its own copy:
        // the weight up to the k-th element comes from the refinement, then the histogram is made again
        if (cut_k) {
            cut = cut_in_bin(row, lds, int(kb), kn, true, k, 0.0, k_above, m_above, pmass);
            if (p < 1.0 && kn > SM_LIST) {
                __syncthreads();
                for (int i = tid; i < SM_BINS; i += SM_BLOCK) {
                    lds.mass[i] = 0;
                    lds.count[i] = 0;
                }
                __syncthreads();
                row.for_each([&](const float(&x)[SM_VEC], int64_t) {
#pragma unroll
                    for (int j = 0; j < SM_VEC; ++j) {
                        if (x[j] != -inf) {
                            const double y = row.log2w(x[j]);
                            const int b = row.bin(y);
                            atomicAdd(&lds.count[b], 1u);
                            atomicAdd(reinterpret_cast<unsigned long long*>(&lds.mass[b]),
                                      static_cast<unsigned long long>(row.fixed(exp2_neg(y), b)));
                        }
                    }
                });
            }
        }
        if (p < 1.0) {
            const double goal = p * pmass;
            pick_bin(lds, in_bin, false, 0, goal, 0.0, total, elements);
            pb = lds.bin;
            pn = lds.count[pb];
            p_above = lds.above_count;
            p_m_above = lds.above;
            double w;
            const Cut by_p = cut_in_bin(row, lds, int(pb), pn, false, 0, goal, p_above, p_m_above, w);
            if (cut.keeps(by_p.key, by_p.index))
                cut = by_p;
        }
    }

    double total;
    const double u = double(call.uniforms[r]);
    const int64_t token = find_in_order(
        row, lds,
        [&](float x, uint32_t i) {
            if (!cut.keeps(key_of(x), i))
                return 0.0;
            const double w = row.weight(x);
            return w >= least ? w : 0.0;
        },
        [&](double z) { return u > 0.0 ? u * z : 0.0; }, total);
    if (tid == 0) {
        call.tokens[r] = token;
        if (call.logprobs != nullptr) {
            float x;
            if constexpr (TYPE == LOGITS_F32)
                x = static_cast<const float*>(row.p)[token];
            else
                x = widen<TYPE>(static_cast<const uint16_t*>(row.p)[token]);
            call.logprobs[r] = float(row.log2w(x) * 0x1.62e42fefa39efp-1 - ::log(total));
        }
    }
}

size_t sample_workspace_bytes(int64_t, int64_t) { return 256; }

hipError_t launch_sample(const SampleCall& call, int type, void*, hipStream_t stream)
{
    if (call.rows == 0)
        return hipSuccess;
    const dim3 grid(static_cast<unsigned>(call.rows));
    if (type == LOGITS_F32)
        sample_row_kernel<LOGITS_F32><<<grid, SM_BLOCK, 0, stream>>>(call);
    else if (type == LOGITS_F16)
        sample_row_kernel<LOGITS_F16><<<grid, SM_BLOCK, 0, stream>>>(call);
    else
        sample_row_kernel<LOGITS_BF16><<<grid, SM_BLOCK, 0, stream>>>(call);
    return hipGetLastError();
}

}  // namespace ls
