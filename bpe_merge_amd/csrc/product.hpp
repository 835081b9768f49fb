// Matrix product in 8-bit floating point with scales: logits of hidden rows
// over a vocabulary's output matrix.
//
//   out[m, n] = sum over blocks kb of 128 columns of
//               sa[m, kb] * sb[n / 128, kb] * sum over k in kb of a[m, k] * b[n, k]
//
// a [M, K] and b [N, K] are e4m3; a block's inner sum is scaled and added in
// f32. The inner sum itself has two forms:
//   e4m3 MFMA, one 16 x 16 x 128 instruction. Measured: of every 8
//     neighbouring products it drops what lies below 2^-13 of the largest
//     one's power of two; sums across these groups are f32. So a group is off
//     by less than 7 * 2^-13 of its largest product: below half a bfloat16 step
//     (2^-8) of that product, but more than a binary16 one's (2^-11), and all
//     of the result where the large products cancel. On normal data that is
//     1.5e-5 of the result's norm.
//   f16 MFMA, four 16 x 16 x 32 instructions on operands widened in
//     registers: e4m3 values are f16 values, their products are exact and
//     all sums f32. Half the matrix rate, and 16 conversions a fragment.
// Few rows are bound by reading b, where the exact form costs nothing. Many
// rows take it for f32 and binary16 results; bfloat16 ones take the e4m3 form,
// for its rate (2,048 x 65,536 x 4,096: 534 us against 960 in
// binary16), and callers who want f32 sums there ask for f32 results.
// b's rows are the MFMA's first operand and a's its second, so a lane of the
// result holds one row m and four neighbouring n: one scale factor per lane
// and tile, and vector stores.
#pragma once

#include <type_traits>

#include "lanes.hpp"
#include "plan.hpp"

namespace bpek {

constexpr uint32_t PR_BLOCK = 128;  // columns that share a scale, and the MFMA's depth

struct Product {
    const uint8_t* a;      // [m, k], row stride as
    const uint8_t* b;      // [n, k], row stride bs
    const float* sa;       // [m, blocks], row stride sas
    const float* sb;       // [ceil(n / 128), blocks], row stride sbs
    void* out;             // [m, n], row stride os
    size_t as, bs, sas, sbs, os;
    uint32_t m, n, k, blocks;
};

// 16 bytes at any address
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef int i32x4_words __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A lane's 32 e4m3 values of a fragment, as the inner sum's form takes them.
template <bool EXACT>
struct Fragment {
    i32x8 v;
    __device__ __forceinline__ Fragment() {}
    __device__ __forceinline__ explicit Fragment(i32x8 x) : v(x) {}
};
template <>
struct Fragment<true> {
    f16x8 v[4];
    __device__ __forceinline__ Fragment() {}
    __device__ __forceinline__ explicit Fragment(i32x8 x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * i + j], 1.0f, false);
                const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[2 * i + j], 1.0f, true);
                v[i][4 * j] = lo[0];
                v[i][4 * j + 1] = lo[1];
                v[i][4 * j + 2] = hi[0];
                v[i][4 * j + 3] = hi[1];
            }
        }
    }
};

// The inner sums of a 16 x 16 tile over a block.
__device__ __forceinline__ f32x4 inner(const Fragment<false>& x, const Fragment<false>& y) {
    // both operands e4m3; scale operands of 0 select the form without scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 inner(const Fragment<true>& x, const Fragment<true>& y) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.v[i], y.v[i], c, 0, 0, 0);
    return c;
}

// 16 bytes of a row from column c on, at any address.
__device__ __forceinline__ i32x4 piece(const uint8_t* __restrict__ row, uint32_t c) {
    i32x4 v;
    __builtin_memcpy(&v, row + c, 16);
    return v;
}
// The same with zeros from column k on.
__device__ __forceinline__ i32x4 piece(const uint8_t* __restrict__ row, uint32_t c, uint32_t k) {
    uint64_t q[2] = {0, 0};
    if (c + 16u <= k) {
        __builtin_memcpy(q, row + c, 16);
    } else if (c < k && k >= 16u) {
        // the row's last 16 bytes, moved down
        __builtin_memcpy(q, row + k - 16u, 16);
        const uint32_t s = (c + 16u - k) * 8u;
        q[0] = s < 64u ? q[0] >> s | q[1] << 1 << (63u - s) : q[1] >> (s - 64u);
        q[1] = s < 64u ? q[1] >> s : 0u;
    } else if (c < k) {
#pragma unroll
        for (uint32_t i = 0; i < 16u; ++i)
            if (c + i < k) q[i / 8] |= (uint64_t)row[c + i] << (8u * (i % 8));
    }
    return i32x4{(int)q[0], (int)(q[0] >> 32), (int)q[1], (int)(q[1] >> 32)};
}

__device__ __forceinline__ i32x8 join(i32x4 x, i32x4 y) {
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 32 bytes at any address, by loads of whole words (each of which holds at
// least one of them). Loads from between words take longer (1 x 32,256 x
// 4,095: 63 against 42 us; 61 x 4,256 x 4,353: 75 against 28).
__device__ __forceinline__ i32x8 words(const uint8_t* __restrict__ at) {
    const uint32_t off = (uint32_t)(uintptr_t)at & 3u;
    const uint8_t* first = at - off;
    const i32x8 v = join(*(const i32x4_words*)first, *(const i32x4_words*)(first + 16));
    const int after = *(const int*)(first + (off ? 32 : 28));
    i32x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (int)__builtin_amdgcn_alignbyte((uint32_t)(i < 7 ? v[i + 1] : after), (uint32_t)v[i], off);
    return r;
}

// Four neighbouring results of row m from column n on.
template <typename T>
__device__ __forceinline__ void put_four(const Product& p, uint32_t m, uint32_t n, f32x4 v) {
    typename T::raw* o = (typename T::raw*)p.out + m * p.os + n;
    if (n + 4u <= p.n) {
        const float f[4] = {v[0], v[1], v[2], v[3]};
        store_n<T>(o, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < p.n) o[i] = T::put(v[i]);
    }
}

// Few rows: memory bound by b. A workgroup takes NT * 16 rows of b and MT *
// 16 rows of a (the first from blockIdx.y on); its WAVES waves split the blocks of K, each streaming
// its part of b from memory straight into registers (every line is read by
// one wave, so LDS would only add a copy), and add up their sums in LDS at
// the end, in wave order. One row by 32,256 x 4,096: 25 us among other calls,
// 5.3 TB/s of b; 30 us alone, start and end included.
template <typename T, int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_product_rows(Product p) {
    __shared__ f32x4 s_acc[WAVES > 1 ? WAVES - 1 : 1][MT * NT][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t lr = lane & 15u, lg = lane >> 4;
    const uint32_t n0 = blockIdx.x * (NT * 16u), m0 = blockIdx.y * (MT * 16u);
    const uint32_t per = (p.blocks + WAVES - 1u) / WAVES;
    const uint32_t kb0 = wave * per, kb1 = min(p.blocks, kb0 + per);
    // rows past the end read the last row; their results are not stored
    const uint8_t* brow[NT];
    const float* sbrow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        brow[j] = p.b + min(n0 + j * 16u + lr, p.n - 1u) * p.bs;
        sbrow[j] = p.sb + (min(n0 + j * 16u, p.n - 1u) / PR_BLOCK) * p.sbs;
    }
    const uint8_t* arow[MT];
    const float* sarow[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const uint32_t m = min(m0 + i * 16u + lr, p.m - 1u);
        arow[i] = p.a + m * p.as;
        sarow[i] = p.sa + m * p.sas;
    }
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto work = [&](uint32_t kb, auto load) {  // load(row, column): 32 bytes
        const uint32_t c = kb * PR_BLOCK + lg * 32u;
        Fragment<true> bf[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) bf[j] = Fragment<true>(load(brow[j], c));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const Fragment<true> af(load(arow[i], c));
            const float s = sarow[i][kb];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const f32x4 v = inner(bf[j], af);
                const float f = s * sbrow[j][kb];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(v[e], f, acc[i][j][e]);
            }
        }
    };
    const uint32_t full = min(kb1, p.k / PR_BLOCK);  // blocks before this one are whole
    if ((((uintptr_t)p.a | (uintptr_t)p.b | (p.m > 1u ? p.as : 0u) | (p.n > 1u ? p.bs : 0u)) & 3u) == 0u) {
        for (uint32_t kb = kb0; kb < full; ++kb)
            work(kb, [](const uint8_t* row, uint32_t c) { return join(piece(row, c), piece(row, c + 16u)); });
    } else {
        for (uint32_t kb = kb0; kb < full; ++kb) work(kb, [](const uint8_t* row, uint32_t c) { return words(row + c); });
    }
    if (full < kb1 && full >= kb0)
        work(full, [&](const uint8_t* row, uint32_t c) { return join(piece(row, c, p.k), piece(row, c + 16u, p.k)); });
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) s_acc[wave - 1][i * NT + j][lane] = acc[i][j];
    }
    lds_sync();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int w = 0; w + 1 < WAVES; ++w) acc[i][j] += s_acc[w][i * NT + j][lane];
            const uint32_t m = m0 + i * 16u + lr, n = n0 + j * 16u + lg * 4u;
            if (m < p.m && n < p.n) put_four<T>(p, m, n, acc[i][j]);
        }
}

// Many rows: a tile of BN rows of b by BM rows of a per workgroup, WN x WM
// waves, both staged in LDS one block of K at a time, STAGES stages in turn.
// Up to some 64 rows it is bound by reading b (64 x 64,256 x 4,096: 52 us, 5.2
// TB/s), with many by the matrix unit and what feeds it: 2,048 x 65,536 x
// 4,096 takes 534 us, 2.06 PFLOP/s, where a library product of the same size
// with one scale in all takes 400 us. There the matrix unit works 45% of the
// time; without the scalings it took 6% less (measured on a copy), without
// the copies of the next blocks 30% less: those come from beyond the L2 (1.1
// GB a call) later than a block of work ago, and LDS has no room for a third
// stage of this tile.
// Rows that are not whole pieces, aligned, cannot be copied to LDS; they go
// through registers, one block ahead (700 x 32,256: K of 3,909 takes 215 us,
// of 3,904 142; 64 x 64,256: K of 4,095 78 us, of 4,096 52).
// A row's 8 pieces of 16 bytes are kept in an order of their own (piece c at
// c ^ turn(row)): the lanes of a fragment read a piece of 16 rows each, 16
// lanes at a time from 64 banks (256 bytes: two rows), and without it would
// meet in the same ones. Two rows share a turn, as they lie in different
// banks; row % 8 instead costs a conflict per read (measured: 4 cycles more).
__device__ __forceinline__ uint32_t turn(uint32_t row) { return (row >> 1) & 7u; }

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved; nothing else in these kernels uses it
// 16 bytes per lane from base + off into LDS at lds + 16 * lane (base and lds
// uniform). Inline assembly, so that the compiler does not wait for the copy
// before every LDS read; the caller waits for it (vmcnt) before its barrier.
__device__ __forceinline__ void copy_to_lds(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %0"
                 :
                 : "s"(base), "v"(off), "s"(lds)
                 : "m0");
}
// 4 bytes per lane likewise, at lds + 4 * lane.
__device__ __forceinline__ void copy_word_to_lds(const float* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(src), "s"(lds) : "m0");
}
#pragma clang diagnostic pop
// Waits until at most N of the wave's copies are left (they end in order).
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)p; }

template <typename T, bool EXACT, int BN, int BM, int WN, int WM, int STAGES, Pieces KIND>
__global__ __launch_bounds__(64 * WN * WM) void k_product_tile(Product p, uint32_t tiles_n, uint32_t tiles_m) {
    constexpr bool COPIED = copied(KIND);
    constexpr int TPB = 64 * WN * WM;
    constexpr int NT = BN / 16 / WN, MT = BM / 16 / WM;      // MFMA tiles of a wave
    constexpr int PIECES = (BN + BM) * 8 / TPB;          // 16-byte pieces a thread stages
    constexpr int B_PIECES = BN * 8 / TPB;
    constexpr uint32_t QB = BN / PR_BLOCK;                   // blocks of b's scales
    constexpr uint32_t STAGE = (BN + BM) * PR_BLOCK;
    static_assert(BN % PR_BLOCK == 0 && PR_BLOCK % (BN / WN) == 0, "a wave's rows of b share a scale");
    static_assert(BN * 8 % TPB == 0 && BM * 8 % TPB == 0 && TPB / 8 % 16 == 0, "threads stage whole rows");
    static_assert(BM % 64 == 0 && BM < TPB && QB <= 64, "whole waves bring the scales of a, the others those of b");
    static_assert(COPIED || STAGES == 2, "pieces that go through registers are one block ahead");
    static_assert(sizeof(typename T::raw) * BN * BM <= STAGES * STAGE, "the results fit the stages");
    __shared__ __align__(1024) uint8_t s_ab[STAGES][STAGE];
    __shared__ float s_sa[STAGES][BM];
    __shared__ float s_sb[STAGES][TPB - BM];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lr = lane & 15u, lg = lane >> 4;
    // Workgroups start round robin over the 8 dies; each die takes a
    // contiguous run of tiles, m fastest, so that the tiles that share rows
    // of b run together under one L2.
    const uint32_t tiles = tiles_n * tiles_m;
    const uint32_t die = blockIdx.x & 7u, slot = blockIdx.x >> 3;
    const uint32_t whole = tiles >> 3, rest = tiles & 7u;
    const uint32_t tile = die * whole + min(die, rest) + slot;
    const uint32_t n0 = tile / tiles_m * BN, m0 = tile % tiles_m * BM;
    const uint32_t wn = wave / WM, wm = wave % WM;

    // what this thread stages: piece threadIdx.x + j * TPB of the stage, at
    // offsets from the first row of b or of a (rows past the end read the
    // last row; their results are not stored)
    const uint8_t* b0 = p.b + n0 * p.bs;
    const uint8_t* a0 = p.a + m0 * p.as;
    const uint32_t col = ((threadIdx.x & 7u) ^ turn(threadIdx.x >> 3)) * 16u;  // one for all of them: TPB / 8 rows are 16s
    uint32_t off[PIECES];                                    // 256 rows lie within 2^31 bytes
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
        const uint32_t r = (threadIdx.x >> 3) + (j < B_PIECES ? j : j - B_PIECES) * (TPB / 8);
        off[j] = col + (j < B_PIECES ? min(r, p.n - 1u - n0) * (uint32_t)p.bs : min(r, p.m - 1u - m0) * (uint32_t)p.as);
        asm volatile("" : "+v"(off[j]));  // a register of its own, not half of a product's pair
    }
    // and a scale: the first BM threads one of a row of a, the others one of
    // a block of rows of b (those past the last block read it again)
    const bool of_a = wave < BM / 64;
    const float* scale = of_a ? p.sa + min(m0 + threadIdx.x, p.m - 1u) * p.sas
                              : p.sb + min(n0 / PR_BLOCK + min(lane, QB - 1u), (p.n - 1u) / PR_BLOCK) * p.sbs;
    float* s_scale = of_a ? &s_sa[0][wave * 64u] : &s_sb[0][wave * 64u - BM];
    const uint32_t next_scale = of_a ? BM : TPB - BM;        // from a stage's to the next one's

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Blocks are taken from a start of the tile's own, round to the one before
    // it: rows are often a power of two long, and workgroups that all worked
    // on the same columns would ask the same few memory channels for them
    // (256 x 64,256 x 4,096: 93 against 76 us). Dies start an eighth of a row
    // apart, the tiles of a die, which share rows through its L2, up to 7
    // blocks.
    const uint32_t start = (die * (p.blocks >> 3) + ((n0 / BN + m0 / BM) & 7u)) % p.blocks;
    auto place = [&](uint32_t kb) {
        kb = min(kb, p.blocks - 1u) + start;
        return __builtin_amdgcn_readfirstlane(kb < p.blocks ? kb : kb - p.blocks);
    };
    // Piece j of block kb into a stage, or into registers on its way there,
    // and with the last one the scale (past the last block the last one again:
    // no branch in the loop). A last block that is short is fetched as the
    // row's last 128 bytes; settle makes zeros of what of a belongs to the
    // block before.
    constexpr int COPIES = PIECES + 1;
    const uint32_t last = p.blocks - 1u, before = p.blocks * PR_BLOCK - p.k;
    [[maybe_unused]] i32x4 held[COPIED ? 1 : PIECES];
    [[maybe_unused]] float held_scale;
    auto fetch = [&](uint32_t kb, uint32_t stage, int j) {
        kb = place(kb);
        const uint8_t* base = (j < B_PIECES ? b0 : a0) + kb * PR_BLOCK;
        if ((KIND == PR_SHORT || KIND == PR_ODD) && kb == last) base -= before;
        if constexpr (COPIED) copy_to_lds(base, off[j], lds_address(&s_ab[stage][0]) + (wave * 64u + j * TPB) * 16u);
        else if constexpr (KIND == PR_ODD) held[j] = piece(base, off[j]);
        else held[j] = piece(base + (off[j] - col), col, p.k);
        if (j < PIECES - 1) return;
        if constexpr (COPIED) copy_word_to_lds(scale + kb, lds_address(s_scale) + stage * next_scale * 4u);
        else held_scale = scale[kb];
    };
    // What was fetched for block kb is in its stage after the next barrier,
    // but for what was fetched after it.
    auto settle = [&](uint32_t kb, uint32_t stage) {
        if constexpr (COPIED) {
            wait_copies<COPIES*(STAGES - 2)>();
            if (KIND == PR_SHORT && place(kb) == last && col < before) {
#pragma unroll
                for (int j = B_PIECES; j < PIECES; ++j) *(i32x4*)&s_ab[stage][(threadIdx.x + j * TPB) * 16u] = i32x4{0, 0, 0, 0};
            }
        } else {
            if (KIND == PR_ODD && place(kb) == last && col < before) {
                const uint32_t other = min(before - col, 16u);  // bytes of the block before
#pragma unroll
                for (int j = B_PIECES; j < PIECES; ++j)
#pragma unroll
                    for (uint32_t d = 0; d < 4; ++d)
                        held[j][d] &= other >= 4 * d + 4 ? 0u : other <= 4 * d ? ~0u : ~0u << (other - 4 * d) * 8u;
            }
#pragma unroll
            for (int j = 0; j < PIECES; ++j) *(i32x4*)&s_ab[stage][(threadIdx.x + j * TPB) * 16u] = held[j];
            s_scale[stage * next_scale + lane] = held_scale;
        }
    };
    const uint32_t swz0 = (lg ^ turn(lr)) * 16u, swz1 = ((lg + 4u) ^ turn(lr)) * 16u;
    const uint32_t n_in = wn * (BN / WN), m_in = wm * (BM / WM);

    // Copies run STAGES - 1 blocks ahead. (A block's data come from HBM in
    // about the time of a block's work, so one is not enough.)
#pragma unroll
    for (int b = 0; b < STAGES - 1; ++b)
#pragma unroll
        for (int j = 0; j < PIECES; ++j) fetch(b, b, j);
    settle(0, 0);
    lds_sync();
    uint32_t stage = 0;
    for (uint32_t kb = 0; kb < p.blocks; ++kb) {
        const uint32_t next = stage == 0 ? STAGES - 1 : stage - 1u;  // read in the turn before
        const uint8_t* bn = &s_ab[stage][(n_in + lr) * PR_BLOCK];
        const uint8_t* am = &s_ab[stage][(BN + m_in + lr) * PR_BLOCK];
        auto read = [&](const uint8_t* rows, int t) {
            return Fragment<EXACT>(join(*(const i32x4*)(rows + t * 16 * PR_BLOCK + swz0), *(const i32x4*)(rows + t * 16 * PR_BLOCK + swz1)));
        };
        Fragment<EXACT> af[MT];
        float f[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) af[i] = read(am, i);
        // a tile's sums are scaled while the matrix unit works on the next
        f32x4 sum[NT][MT];
#pragma unroll
        for (int j = 0; j <= NT; ++j) {
            if (j < NT) {
                const Fragment<EXACT> bf = read(bn, j);
#pragma unroll
                for (int i = 0; i < MT; ++i) sum[j][i] = inner(bf, af[i]);
                if (j == 0) {
#pragma unroll
                    for (int t = 0; t < MT; ++t) f[t] = s_sa[stage][m_in + t * 16 + lr];
                    const float fb = s_sb[stage][n_in / PR_BLOCK];
#pragma unroll
                    for (int t = 0; t < MT; ++t) f[t] *= fb;
                }
                // the next block's pieces, a few at a time, so that the
                // waves' other work is not held up behind them
#pragma unroll
                for (int c = 0; c < (KIND == PR_NARROW ? 0 : PIECES); ++c)
                    if (COPIED ? c * NT / PIECES == j : j == 0) fetch(kb + STAGES - 1u, next, c);
            }
            if (j > 0) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j - 1][e] = __builtin_fmaf(sum[j - 1][i][e], f[i], acc[i][j - 1][e]);
            }
        }
        if constexpr (KIND == PR_NARROW) break;
        stage = stage == STAGES - 1 ? 0 : stage + 1u;
        settle(kb + 1u, stage);
        lds_sync();
    }
    if constexpr (COPIED) wait_copies<0>();  // none may land in what follows
    // Results go through LDS, so that whole lines of a row leave together:
    // 16-byte pieces of row m are kept at piece ^ (m % 16).
    typedef typename T::raw raw;
    constexpr uint32_t PER = 16 / sizeof(raw);               // results in a piece
    raw* s_out = (raw*)&s_ab[0][0];
    lds_sync();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const uint32_t m = m_in + i * 16u + lr, n = n_in + j * 16u + lg * 4u;
            const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            store_n<T>(s_out + m * BN + (((n / PER) ^ (m & 15u)) * PER + n % PER), v);
        }
    lds_sync();
    constexpr uint32_t ROW = BN / PER;                       // pieces in a row
    for (uint32_t i = threadIdx.x; i < BM * ROW; i += TPB) {
        const uint32_t m = i / ROW, n = i % ROW * PER;
        if (m0 + m >= p.m) break;
        const raw* v = s_out + m * BN + ((i % ROW) ^ (m & 15u)) * PER;
        raw* o = (raw*)p.out + (size_t)(m0 + m) * p.os + n0 + n;
        if (n0 + n + PER <= p.n) {
            // results are not read again here: past the caches, which hold b
            __builtin_nontemporal_store(*(const i32x4*)v, (i32x4_any*)o);
        } else {
            for (uint32_t e = 0; n0 + n + e < p.n && e < PER; ++e) o[e] = v[e];
        }
    }
}

}  // namespace bpek
