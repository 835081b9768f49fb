// Sampling of ids from logits, with given uniform numbers.
//
// With w_i = 2^((x_i - max) log2(e) / T), ids in the order of their logits,
// largest first (equal logits: lowest id first):
//   top-k   keeps the first k ids;
//   top-p   keeps the shortest beginning of those whose weights sum to at
//           least p times the sum of all that top-k keeps;
//   min-p   keeps those of them with w_i >= min_p.
// What is kept is a beginning of the order: every id up to one element, the
// cut. The id drawn is the lowest kept one at which the running sum of kept
// weights, in the order of ids, exceeds u times their whole sum.
//
// Ids have to come out the same whatever the order in which partial sums
// meet, so weights are whole numbers: w_i in units of 2^-43 (the largest
// weight is 1), computed in f64 and summed in 64 bits, where 2^20 of them
// fit. f32 sums would move a border by 2^-24 of the whole, and with it the
// id of about one row in a hundred of a flat distribution over 2^16 ids; in
// these units a border moves by at most 2^-44 an id.
//
// A workgroup takes a row. Up to 2^16 ids its logits stay in registers (64 a
// lane at most), so the row is read once; larger vocabularies are read again
// from memory in each pass. A row is one CU's work, where an instruction for
// each logit of 2^16 costs half a microsecond: so the passes are few and
// short, and most rows form weights for a list only. The cut is found by
// spreading logits over bins of equal width below the largest: for a small
// top-k the largest logit of each thread, whose k-th bin bounds the cut's
// (at least k logits lie above its end); otherwise all of them, by count or
// by weight, looking into the bin where the sum crosses until all that lies
// above its end, or all that lies in it, is a list with an element for each
// thread. A list is sorted, and what is left is scans over it.
//
// Measured: one row of 32,256 f32 logits, top-k 50 and top-p 0.95: 15 us, of
// which 3 are the read and the largest, 4 the gather of the list, 5 the two
// sorts; top-p 0.9 alone, where every logit needs its weight, 19 to 43 us,
// top-k 1,000 with top-p 37. 512 rows of 64,256 (132 MB), each with settings of
// its own, greedy ones to top-k 5,000 with top-p: 129 us. A CU takes its two
// rows one after the other (128 registers a lane leave room for 16 waves);
// such a row takes 12 us (greedy: the read), 25 (top-k 50), 59 (top-p 0.9
// alone) to 74 us.
#pragma once

#include <type_traits>

#include "lanes.hpp"

namespace bpek {

constexpr int SM_UNIT = 43;                       // weights are multiples of 2^-43
constexpr uint32_t SM_BINS = 1024;
constexpr uint32_t SM_STEPS = 1024;               // powers of two from a table: 2^(j / 1024)
constexpr uint32_t SM_VEC = 2;                    // logits a lane takes at a time
constexpr uint32_t SM_IDS = (1u << 20) - 1u;        // ids are at most that
constexpr float SM_NEG = -__builtin_inff();
constexpr float SM_MOST = 3.402823466e38f;

struct Sampling {
    float temperature, top_p, min_p;              // for all rows, where the row arrays are null
    int32_t top_k;
    const float* temperatures;
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
};

// 2^f for |f| <= 1/2: the Taylor polynomial of e^(f ln 2) to degree 13, whose
// remainder is below 2^-57.
__device__ __forceinline__ double power_of_two(double f) {
    const double x = f * 0.6931471805599453094;
    double p = 1.0 / 6227020800.0;
    p = __builtin_fma(p, x, 1.0 / 479001600.0);
    p = __builtin_fma(p, x, 1.0 / 39916800.0);
    p = __builtin_fma(p, x, 1.0 / 3628800.0);
    p = __builtin_fma(p, x, 1.0 / 362880.0);
    p = __builtin_fma(p, x, 1.0 / 40320.0);
    p = __builtin_fma(p, x, 1.0 / 5040.0);
    p = __builtin_fma(p, x, 1.0 / 720.0);
    p = __builtin_fma(p, x, 1.0 / 120.0);
    p = __builtin_fma(p, x, 1.0 / 24.0);
    p = __builtin_fma(p, x, 1.0 / 6.0);
    p = __builtin_fma(p, x, 0.5);
    p = __builtin_fma(p, x, 1.0);
    return __builtin_fma(p, x, 1.0);
}

// 2^(t / 1024) in units of 2^-43 to the nearest whole number, for t <= 0 (0
// for NaN): the table's power times the Taylor polynomial of degree 3 of what
// is left, at most 1/2048 of a power, with a remainder below 2^-50.
__device__ __forceinline__ uint64_t weight_of(double t, const double* table) {
    constexpr double L = 0.6931471805599453094 / SM_STEPS;
    t = __builtin_fmax(t, -(SM_UNIT + 2.0) * SM_STEPS);  // below half a unit: 0 all the same
    const double n = __builtin_rint(t);
    const double r = t - n;
    double p = L * L * L / 6.0;
    p = __builtin_fma(p, r, L * L / 2.0);
    p = __builtin_fma(p, r, L);
    p = __builtin_fma(p, r, 1.0);
    const int i = (int)n;
    // p 2^(i / 1024 + 43) + 2^52: the sum's low 52 bits are the whole number
    const double unit = __hiloint2double(((i >> 10) + SM_UNIT + 1023) << 20, 0);
    const uint64_t bits = (uint64_t)__double_as_longlong(__builtin_fma(p * table[i & (SM_STEPS - 1)], unit, 0x1p52));
    return bits & ((uint64_t(1) << 52) - 1u);
}

// Plus infinity as the largest number (NaN stays: it compares with nothing,
// as minus infinity is above nothing).
__device__ __forceinline__ float finite(float a) { return a > SM_MOST ? SM_MOST : a; }

// SM_VEC logits from id on; those past the row are minus infinity.
template <typename T>
__device__ __forceinline__ void some_logits(const typename T::raw* p, uint32_t id, uint32_t v, float (&o)[SM_VEC]) {
    if (id + SM_VEC <= v) {
        load_n<T>(p + id, o);
    } else {
#pragma unroll
        for (int e = 0; e < SM_VEC; ++e) o[e] = id + e < v ? T::get(p[id + e]) : SM_NEG;
    }
#pragma unroll
    for (int e = 0; e < SM_VEC; ++e) o[e] = finite(o[e]);
}

template <typename T, int TPB, int N>  // N: vectors of logits a lane holds, 0 to read memory in each pass
struct Row {
    const typename T::raw* p;
    const double* table;
    uint32_t v, lane, wave, first, count;  // this wave's part starts at id first, in count vectors a lane
    typedef float Held __attribute__((ext_vector_type(N ? N : 2)));
    Held x[SM_VEC];
    float best;                             // the largest of this thread's
    float top;                              // of the row
    double c;                               // 1024 log2(e) / T

    __device__ __forceinline__ void open(const typename T::raw* row, uint32_t vocab) {
        p = row;
        v = vocab;
        lane = threadIdx.x & 63u;
        wave = threadIdx.x >> 6;
        count = N ? N : (vocab + TPB * SM_VEC - 1u) / (TPB * SM_VEC);
        first = wave * count * (64u * SM_VEC);
        best = SM_NEG;
        if (N) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float o[SM_VEC];
                some_logits<T>(p, first + (j * 64u + lane) * SM_VEC, v, o);
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) x[e][j] = o[e];
            }
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) best = fmaxf(best, x[e][j]);  // not a NaN
        } else {
            each([&](uint32_t, const float (&o)[SM_VEC]) {
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) best = fmaxf(best, o[e]);
            });
        }
    }
    // f(lowest id, its SM_VEC logits), ids rising. A loop over the registers
    // (its counter is uniform, so that they can be indexed by it), never
    // unrolled: this code runs once a row, and where it is long it is bound
    // by the fetch of its instructions.
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
        for (uint32_t j = 0; j < (N ? N : count); ++j) {
            const uint32_t id = first + (j * 64u + lane) * SM_VEC;
            float o[SM_VEC];
            if (N) {
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) o[e] = x[e][j];
            } else {
                some_logits<T>(p, id, v, o);
            }
            f(id, o);
        }
    }
    __device__ __forceinline__ double exponent(float a) const { return ((double)a - (double)top) * c; }
    __device__ __forceinline__ uint64_t weight(float a) const { return weight_of(exponent(a), table); }
};

struct Cut {
    float x;        // kept: logits above x, and equal ones up to id last
    uint32_t last;
    __device__ __forceinline__ bool keeps(float a, uint32_t id) const { return a > x || (a == x && id <= last); }
};

template <int TPB>
struct SampleShared {
    uint64_t mass[SM_BINS];
    uint32_t count[SM_BINS];
    uint64_t wave_a[TPB / 64];
    uint64_t wave_b[TPB / 64];
    float queue[TPB / 64][128];
    uint64_t key[TPB];      // a list: order of the logit << 32 | complement of the id
    double table[SM_STEPS];
    uint32_t list_n;
    uint32_t bin, lo, hi;
    uint64_t before_mass, before_count;
    Cut cut;
    uint32_t pick;
};

// Order-preserving bits of a float (no NaN; one zero).
__device__ __forceinline__ uint32_t order_bits(float a) {
    const uint32_t b = __builtin_bit_cast(uint32_t, a + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_order(uint32_t b) {
    return __builtin_bit_cast(float, b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

// The exclusive prefix of this thread's value over the workgroup, and the
// sum. The waves' sums lie in s; each wave scans them for itself.
template <int TPB>
__device__ __forceinline__ uint64_t block_prefix(uint64_t v, uint64_t* s, uint64_t* total) {
    auto add = [](uint64_t a, uint64_t b) { return a + b; };
    const uint32_t lane = threadIdx.x & 63u;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint64_t incl = wave_inclusive(v, uint64_t(0), add);
    lds_sync();
    if (lane == 63u) s[w] = incl;
    lds_sync();
    const uint64_t waves = wave_inclusive(lane < TPB / 64 ? s[lane] : uint64_t(0), uint64_t(0), add);
    *total = read_lane(waves, 63);
    return (w ? read_lane(waves, w - 1) : uint64_t(0)) + incl - v;
}
template <int TPB, typename V, typename Op>
__device__ __forceinline__ V block_all(V v, uint64_t* s, Op op) {  // op's identity is 0
    v = wave_all(v, V(0), op);
    const uint32_t lane = threadIdx.x & 63u;
    lds_sync();
    if (lane == 0) s[threadIdx.x >> 6] = v;
    lds_sync();
    return wave_all(lane < TPB / 64 ? (V)s[lane] : V(0), V(0), op);
}
template <int TPB, typename V>
__device__ __forceinline__ V block_sum(V v, uint64_t* s) {
    return block_all<TPB>(v, s, [](V a, V b) { return a + b; });
}

// The lowest id, in the order of ids, at which the running sum of f over
// the row exceeds target (below the whole sum). f(id, logit) is 0 for what
// does not count; sum is this thread's part. The wave in whose part it lies
// is known from the waves' sums, and all threads read that part again.
template <typename T, int TPB, int N, typename F>
__device__ __forceinline__ uint32_t pick_by_id(const Row<T, TPB, N>& row, uint64_t sum, F f, uint64_t target,
                                               SampleShared<TPB>& sh) {
    sum = wave_sum(sum);
    lds_sync();
    if (row.lane == 0) sh.wave_a[row.wave] = sum;
    lds_sync();
    const uint64_t waves = wave_inclusive(row.lane < TPB / 64 ? sh.wave_a[row.lane] : uint64_t(0), uint64_t(0),
                                          [](uint64_t a, uint64_t b) { return a + b; });
    const uint32_t w = (uint32_t)__popcll(__ballot(waves <= target));  // below the whole sum: some wave exceeds it
    uint64_t before = w ? read_lane(waves, (int)w - 1) : uint64_t(0);
    const uint32_t end = (w + 1u) * row.count * (64u * SM_VEC);
    for (uint32_t at = w * row.count * (64u * SM_VEC); at < end; at += TPB * SM_VEC) {
        const uint32_t id = at + threadIdx.x * SM_VEC;
        float o[SM_VEC];
        uint64_t g[SM_VEC], mine = 0, total;
        some_logits<T>(row.p, id, min(row.v, end), o);
#pragma unroll
        for (int e = 0; e < SM_VEC; ++e) mine += g[e] = f(id + e, o[e]);
        uint64_t run = before + block_prefix<TPB>(mine, sh.wave_b, &total);
        if (run <= target && run + mine > target) {
#pragma unroll
            for (int e = 0; e < SM_VEC; ++e) {
                if (run <= target && run + g[e] > target) sh.pick = id + e;
                run += g[e];
            }
        }
        before += total;
        if (before > target) break;
    }
    lds_sync();
    return sh.pick;
}

// Keys in falling order over the first n threads (bitonic; n is uniform).
// The rest have 0, and stay behind.
template <int TPB>
__device__ __forceinline__ uint64_t sort_keys(uint64_t key, uint32_t n, uint64_t* s) {
    const uint32_t t = threadIdx.x;
    uint32_t size = 2;
    while (size < n) size <<= 1;
#pragma unroll 1
    for (uint32_t run = 2; run <= size; run <<= 1) {
#pragma unroll 1
        for (uint32_t step = run >> 1; step > 0; step >>= 1) {
            uint64_t other;
            if (step >= 64) {
                lds_sync();
                s[t] = key;
                lds_sync();
                other = s[t ^ step];
            } else {
                other = (uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)(key >> 32), (int)step) << 32 |
                        (uint32_t)__shfl_xor((int)(uint32_t)key, (int)step);
            }
            // the larger key goes to the lower place, in rising runs the other way round
            const bool larger = ((t & step) == 0) == ((t & run) == 0);
            if (t < size && larger == (other > key)) key = other;
        }
    }
    return key;
}

template <typename T, int TPB, int N>
__global__ __launch_bounds__(TPB) void k_sample(const typename T::raw* __restrict__ logits, size_t stride, uint32_t v,
                                                const float* __restrict__ u, Sampling par, int32_t* __restrict__ ids,
                                                float* __restrict__ logp) {
    __shared__ SampleShared<TPB> sh;
    const uint32_t r = blockIdx.x, t = threadIdx.x;
    const float temperature = par.temperatures ? par.temperatures[r] : par.temperature;
    const int32_t top_k = par.top_ks ? par.top_ks[r] : par.top_k;
    const float top_p = par.top_ps ? par.top_ps[r] : par.top_p;
    const float min_p = par.min_ps ? par.min_ps[r] : par.min_p;
    const float draw = u[r];
    Row<T, TPB, N> row;
    row.table = sh.table;
    row.open(logits + r * stride, v);
    for (uint32_t i = t; i < SM_STEPS; i += TPB) sh.table[i] = power_of_two((double)i / SM_STEPS - 0.5) * 1.4142135623730950488;

    const uint32_t top_bits = block_all<TPB>(row.best > SM_NEG ? order_bits(row.best) : 0u, sh.wave_a,
                                             [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    if (top_bits == 0) {  // nothing to draw from
        if (t == 0) {
            ids[r] = -1;
            if (logp) logp[r] = SM_NEG;
        }
        return;
    }
    row.top = from_order(top_bits);
    // one id is left: T = 0 (or no number), top_k = 1, or no share for top_p
    if (!(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f) {
        uint32_t id = 0xFFFFFFFFu;
        if (row.best == row.top) {
            row.each([&](uint32_t i, const float (&o)[SM_VEC]) {
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e)
                    if (o[e] >= row.top) id = min(id, i + e);
            });
        }
        id = ~block_all<TPB>(~id, sh.wave_b, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
        if (t == 0) {
            ids[r] = (int32_t)id;
            if (logp) logp[r] = 0.0f;
        }
        return;
    }
    row.c = 1.4426950408889634074 * SM_STEPS / (double)temperature;
    const bool lowest = !(draw > 0.0f);  // the lowest kept id, however small its weight
    const bool by_min = min_p > 0.0f;
    const double least_t = by_min ? log2((double)fminf(min_p, 1.0f)) * SM_STEPS : 0.0;
    auto target_of = [&](uint64_t mass) {
        const double at = (double)draw * (double)mass;
        const uint64_t target = at < (double)mass ? (uint64_t)at : mass;
        return target < mass ? target : mass - 1u;
    };
    auto part_of = [&](uint64_t mass) {  // at least p of the mass: whole units, so the next whole number up
        const double part = __builtin_ceil((double)top_p * (double)mass);
        return part < 1.0 ? uint64_t(1) : (uint64_t)part;
    };
    auto answer = [&](uint32_t id, float a, uint64_t mass) {  // by one thread
        ids[r] = (int32_t)id;
        if (logp) {
            constexpr double LN2 = 0.6931471805599453094;
            logp[r] = (float)(row.exponent(finite(a)) * (LN2 / SM_STEPS) - log((double)mass) + SM_UNIT * LN2);
        }
    };

    bool by_k = top_k > 0 && (uint32_t)top_k < v;
    const bool by_p = top_p < 1.0f;
    Cut cut{SM_NEG, 0u};  // keeps all but minus infinity
    // min-p's smallest kept logit: the lowest of the four numbers about
    // top + least_t / c whose exponent reaches least_t
    float least_x = -SM_MOST;
    if (by_min && row.c > 0.0) {  // (at an infinite temperature all weights are 1)
        uint32_t g = order_bits(__double2float_rd((double)row.top + least_t / row.c));
        g = g > order_bits(-SM_MOST) + 2u ? g - 1u : order_bits(-SM_MOST);
        for (int i = 0; i < 3 && row.exponent(from_order(g)) < least_t; ++i) ++g;
        least_x = from_order(min(g, top_bits));
    }
    auto kept = [&](uint32_t id, float a) { return a >= least_x && cut.keeps(a, id); };
    // This thread's part of the weights that the cut keeps, of logits from
    // least on. A weight takes some thirty
    // instructions whether one lane wants it or all: where much is cut off,
    // a wave collects what is kept in LDS, and weighs it 64 at a time.
    auto kept_mass = [&](float least) {
        uint64_t mass = 0;
        if (cut.x > SM_NEG || least > -SM_MOST) {
            float* queue = sh.queue[row.wave];
            uint32_t n = 0;
            row.each([&](uint32_t id, const float (&o)[SM_VEC]) {
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) {
                    const bool keep = o[e] >= least && cut.keeps(o[e], id + e);
                    const uint64_t who = __ballot(keep);
                    if (!who) continue;
                    if (keep) queue[n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0u))] = o[e];
                    n += (uint32_t)__popcll(who);
                    if (n >= 64u) {
                        n -= 64u;
                        mass += row.weight(queue[n + row.lane]);
                    }
                }
            });
            if (row.lane < n) mass += row.weight(queue[row.lane]);
        } else {
            row.each([&](uint32_t id, const float (&o)[SM_VEC]) {
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) {
                    const uint64_t w = row.weight(o[e]);
                    mass += o[e] >= least ? w : uint64_t(0);
                }
            });
        }
        return mass;
    };
    // Draws from the list in sh.key, which holds everything down to the cut:
    // an element to a thread, first in falling order of logits, for the cuts,
    // then the kept ones in the order of ids. In one wave where that holds
    // the list: no barriers then.
    auto finish = [&](auto one_wave, uint32_t n_list, uint64_t need, bool by_mass) {
        constexpr bool WAVE = decltype(one_wave)::value;
        auto add = [](uint64_t a, uint64_t b) { return a + b; };
        auto prefix = [&](uint64_t v, uint64_t* s, uint64_t* total) {
            if constexpr (WAVE) {
                const uint64_t incl = wave_inclusive(v, uint64_t(0), add);
                *total = read_lane(incl, 63);
                return incl - v;
            } else {
                return block_prefix<TPB>(v, s, total);
            }
        };
        uint64_t key = sort_keys<TPB>(t < n_list ? sh.key[t] : 0u, n_list, sh.key);
        const uint32_t id = 0xFFFFFFFFu - (uint32_t)key;
        const float a = t < n_list ? from_order((uint32_t)(key >> 32)) : SM_NEG;
        const uint64_t w = row.weight(a);
        uint64_t mass, all;
        const uint64_t before = prefix(w, sh.wave_a, &all);
        bool keep = t < n_list && (by_mass ? before < need : t < (uint32_t)need);
        if (!by_mass && by_p) {
            uint64_t by_k_mass;
            if constexpr (WAVE) {
                by_k_mass = read_lane(before + w, __builtin_amdgcn_readfirstlane((int)need - 1));
            } else {
                if (t + 1u == (uint32_t)need) sh.before_mass = before + w;
                lds_sync();
                by_k_mass = sh.before_mass;
            }
            keep = keep && before < part_of(by_k_mass);
        }
        keep = keep && a >= least_x;
        (void)prefix(keep ? w : uint64_t(0), sh.wave_b, &mass);
        key = sort_keys<TPB>(keep ? (uint64_t)(SM_IDS - id) << (SM_UNIT + 1) | w : uint64_t(0), n_list, sh.key);
        const uint64_t g = key & ((uint64_t(1) << (SM_UNIT + 1)) - 1u);
        const uint64_t run = prefix(g, sh.wave_a, &all);
        const uint64_t target = target_of(mass);
        if (lowest ? t == 0 : run <= target && run + g > target) {
            const uint32_t drawn = SM_IDS - (uint32_t)(key >> (SM_UNIT + 1));
            answer(drawn, T::get(row.p[drawn]), mass);
        }
    };
    uint64_t need = by_k ? (uint64_t)top_k : 0;  // a count, or (0: not known yet) a weight
    // Top-k first; where it leaves too many for a list, top-p then works on
    // the row, with the weight that top-k's cut keeps.
    bool again = false;  // the bins of the turn before serve once more
    while (by_k || by_p) {
        const bool by_mass = !by_k;
        // where top-k leaves too many for a list, top-p needs their weight
        const bool weigh = by_mass || (by_p && need > TPB);
        // Logits below near have no weight in these units. (Bins over all the
        // row would leave one for all that counts beside a mask of very low
        // numbers.)
        const double far = (double)row.top - (SM_UNIT + 1.5) * 0.6931471805599453094 * (double)temperature;
        float hi = row.top, lo = far < (double)hi ? __double2float_rd(far) : hi;
        if (!(lo < hi)) lo = from_order(order_bits(hi) - 1u);
        lo = fmaxf(lo, -SM_MOST);
        uint64_t above_count = 0, above_mass = 0;  // of elements above hi
        uint32_t n_list = 0;
        enum { NONE, LIST, PART, EQUAL } found;
        bool maxima = !by_mass && need <= TPB / 2, deeper = false;
        for (;;) {
            if (!(lo < hi)) {
                found = EQUAL;
                break;
            }
            // Bins of equal width: hi is in bin 0 and lo in one of the last
            // two, so that a bin never holds both and every turn leaves
            // fewer. (Halves, so that the difference of any two numbers is
            // one; or, of neighbours of zero, a multiple.)
            const float f = hi - lo < 1e-30f ? 0x1p100f : 0.5f, f_hi = f * hi;
            const float k = (float)(SM_BINS - 1u) / __builtin_fmaf(-f, lo, f_hi);
            auto bin_of = [&](float a) { return min((uint32_t)fmaxf(__builtin_fmaf(-f, a, f_hi) * k, 0.0f), SM_BINS - 1u); };
            lds_sync();
            for (uint32_t i = t; i < SM_BINS && !again; i += TPB) {
                sh.count[i] = 0;
                if (weigh) sh.mass[i] = 0;
            }
            if (t == 0) {
                sh.bin = SM_BINS;
                sh.lo = 0xFFFFFFFFu;
                sh.hi = 0u;
                sh.list_n = 0;
            }
            lds_sync();
            uint32_t below = 0;
            if (again) {
                again = false;
            } else if (maxima) {
                if (row.best >= lo) atomicAdd(&sh.count[bin_of(row.best)], 1u);
            } else if (weigh) {
                row.each([&](uint32_t, const float (&o)[SM_VEC]) {
#pragma unroll
                    for (int e = 0; e < SM_VEC; ++e) {
                        const uint64_t w = row.weight(o[e]);  // of all: no branch holds up the next
                        if (o[e] >= lo && o[e] <= hi) {
                            const uint32_t b = bin_of(o[e]);
                            atomicAdd(&sh.count[b], 1u);
                            atomicAdd((unsigned long long*)&sh.mass[b], (unsigned long long)w);
                        }
                        below += o[e] < lo && o[e] > SM_NEG;
                    }
                });
            } else {
                row.each([&](uint32_t, const float (&o)[SM_VEC]) {
#pragma unroll
                    for (int e = 0; e < SM_VEC; ++e) {
                        const float a = o[e];
                        if (a >= lo && a <= hi) atomicAdd(&sh.count[bin_of(a)], 1u);
                        below += a < lo && a > SM_NEG;
                    }
                });
            }
            // scan the bins: a thread takes neighbouring ones
            constexpr uint32_t PER = SM_BINS / TPB;
            lds_sync();
            uint64_t sc = 0, sm = 0, all_count, all_mass = 0, m0 = 0;
#pragma unroll
            for (uint32_t i = 0; i < PER; ++i) {
                sc += sh.count[t * PER + i];
                if (weigh) sm += sh.mass[t * PER + i];
            }
            uint64_t c0 = above_count + block_prefix<TPB>(sc, sh.wave_a, &all_count);
            if (weigh) {
                m0 = above_mass + block_prefix<TPB>(sm, sh.wave_b, &all_mass);
                if (!need) need = part_of(all_mass);
            }
#pragma unroll
            for (uint32_t i = 0; i < PER; ++i) {
                const uint64_t c1 = c0 + sh.count[t * PER + i], m1 = weigh ? m0 + sh.mass[t * PER + i] : 0;
                if (by_mass ? (m0 < need && m1 >= need) : (c0 < need && c1 >= need)) {
                    sh.bin = t * PER + i;
                    sh.before_count = c0;
                    sh.before_mass = m0;
                }
                c0 = c1;
                m0 = m1;
            }
            lds_sync();
            const uint32_t bin = sh.bin;
            uint32_t in_bin;
            if (bin < SM_BINS) {
                in_bin = sh.count[bin];
                if (!maxima) {
                    above_count = sh.before_count;
                    above_mass = sh.before_mass;
                }
            } else if (maxima) {
                maxima = false;
                continue;
            } else {  // top-k reaches below near
                above_count += all_count;
                above_mass += all_mass;
                if (need > above_count + block_sum<TPB>(below, sh.wave_a)) {
                    found = NONE;
                    break;
                }
                in_bin = 0xFFFFFFFFu;
            }
            const bool whole = maxima || above_count + in_bin <= TPB;
            if (whole || in_bin <= TPB) {
                // a little below the bin's end: most vectors have nothing above it
                const float end = fmaxf(lo, (f_hi - ((float)bin + 1.5f) / k) / f);
                const float begin = whole ? SM_MOST : fminf(SM_MOST, (f_hi - ((float)bin - 0.5f) / k) / f);
                row.each([&](uint32_t id, const float (&o)[SM_VEC]) {
                    bool any = false;
#pragma unroll
                    for (int e = 0; e < SM_VEC; ++e) any = any || (o[e] >= end && o[e] <= begin);
                    if (!__ballot(any)) return;
#pragma unroll
                    for (int e = 0; e < SM_VEC; ++e) {
                        const float a = o[e];
                        const uint32_t b = bin_of(a);  // 0 above hi
                        const bool in = a >= lo && (whole ? b <= bin : b == bin && a <= hi);
                        const uint64_t who = __ballot(in);
                        if (!who) continue;
                        uint32_t at = 0;
                        if (row.lane == (uint32_t)__builtin_ctzll(who)) at = atomicAdd(&sh.list_n, (uint32_t)__popcll(who));
                        at = read_lane(at, __builtin_ctzll(who)) + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0u));
                        if (in && at < TPB) sh.key[at] = (uint64_t)order_bits(a) << 32 | (0xFFFFFFFFu - (id + e));
                    }
                });
                lds_sync();
                n_list = sh.list_n;
                if (n_list <= TPB) {
                    found = whole ? LIST : PART;
                    break;
                }
                maxima = false;  // more than a list above the bin in which the k-th thread's largest lies
                continue;
            }
            // on with the bin's own largest and smallest (bin SM_BINS: with what lies below near)
            uint32_t small = 0xFFFFFFFFu, large = 0u;
            row.each([&](uint32_t, const float (&o)[SM_VEC]) {
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) {
                    const float a = o[e];
                    if (bin < SM_BINS ? a >= lo && a <= hi && bin_of(a) == bin : a < lo && a > SM_NEG) {
                        small = min(small, order_bits(a));
                        large = max(large, order_bits(a));
                    }
                }
            });
            atomicMin(&sh.lo, small);
            atomicMax(&sh.hi, large);
            lds_sync();
            lo = from_order(sh.lo);
            hi = from_order(sh.hi);
            deeper = true;
        }
        if (found == LIST && n_list <= 64) {
            if (row.wave == 0) finish(std::true_type{}, n_list, need, by_mass);
            return;
        }
        if (found == LIST) {
            finish(std::false_type{}, n_list, need, by_mass);
            return;
        }
        if (found == PART) {
            const uint64_t key = sort_keys<TPB>(t < n_list ? sh.key[t] : 0u, n_list, sh.key);
            const float a = t < n_list ? from_order((uint32_t)(key >> 32)) : SM_NEG;
            const uint64_t w = row.weight(a);
            uint64_t all;
            const uint64_t before = block_prefix<TPB>(w, sh.wave_a, &all);
            if (by_mass ? above_mass + before < need && above_mass + before + w >= need : t + 1u == (uint32_t)(need - above_count)) {
                sh.cut.x = a;
                sh.cut.last = 0xFFFFFFFFu - (uint32_t)key;
                sh.before_mass = above_mass + before + w;
            }
            lds_sync();
            cut = sh.cut;
            above_mass = sh.before_mass;
        } else if (found == EQUAL) {
            uint64_t n = 0;
            row.each([&](uint32_t, const float (&o)[SM_VEC]) {
#pragma unroll
                for (int e = 0; e < SM_VEC; ++e) n += o[e] == hi;
            });
            const uint64_t there = block_sum<TPB>(n, sh.wave_b), w = row.weight(hi);
            if (by_mass && !need) need = part_of(there * w);  // a row of one value, the lowest there is
            const uint64_t nth = by_mass ? (need - above_mass + w - 1u) / w : need - above_count;
            cut.x = hi;
            cut.last = 0xFFFFFFFFu;
            if (nth <= there)
                cut.last = pick_by_id<T, TPB, N>(row, n, [&](uint32_t, float a) { return uint64_t(a == hi); }, nth - 1u, sh);
            above_mass += min(nth, there) * w;
        }
        if (!by_k) break;
        by_k = false;
        need = 0;
        if (found == NONE || !by_p) continue;
        // above_mass is what the cut keeps; without weights in the bins it is summed
        if (!weigh) above_mass = block_sum<TPB>(kept_mass(-SM_MOST), sh.wave_a);
        again = weigh && found == PART && !deeper;
        need = part_of(above_mass);
    }
    uint64_t mass, n = 0;
    if (lowest) {
        row.each([&](uint32_t id, const float (&o)[SM_VEC]) {
#pragma unroll
            for (int e = 0; e < SM_VEC; ++e) n += kept(id + e, o[e]);
        });
    }
    mass = kept_mass(least_x);
    const uint64_t all = block_sum<TPB>(mass, sh.wave_b);
    const uint32_t id = pick_by_id<T, TPB, N>(row, lowest ? n : mass, [&](uint32_t i, float a) {
        return !kept(i, a) ? uint64_t(0) : lowest ? uint64_t(1) : row.weight(a);
    }, lowest ? 0u : target_of(all), sh);
    if (t == 0) answer(id, T::get(row.p[id]), all);
}

}  // namespace bpek
