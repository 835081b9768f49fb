// Ids back to text: the strings of a row of ids, one after another.
//
// A merge list's vocabulary gives id b < 256 the byte b and id 256 + k the
// string of merge k's left id followed by its right id's. On the device an
// id has one 16-byte entry: its length in the last byte and, up to 15 bytes
// of it, the string itself; a longer string's entry has its place in the
// pool of long strings. So one gather gives a token's length and, nearly
// always, its bytes.
//
// Lengths are data, so a token's place is a prefix sum. The tokens are cut
// into as many chunks as workgroups run together. A first pass sums the
// lengths of each chunk, from a table of bytes that lies in LDS (a gather of
// 64 lanes from memory takes 64 cycles, one from LDS a few); in the second,
// every workgroup adds up the sums of the chunks before its own, scans its
// tokens tile by tile, and writes each tile's bytes through LDS, where they
// are laid out as in memory, so that they leave in whole 16-byte pieces. A
// few tokens are one workgroup's work, in one launch.
//
// Measured: 8,000,003 ids of a vocabulary of 32,256 (58 MB of text): 15 us for
// the sums, 43 us for the text, where every id's entry is a gather from the L2
// (a line for 16 bytes of it); 64 ids: 7 us, 11 us until the host, which polls a
// word for the end, has their length (16 us where it waits for the stream).
#pragma once

#include "lanes.hpp"

namespace bpek {

constexpr uint32_t DC_INLINE = 15;            // string bytes an entry holds
constexpr uint32_t DC_LONG = 0xFFu;           // last byte of a longer string's entry
constexpr uint32_t DC_NONE = 0xFFFFFFFFu;     // the id that stands for no token: no bytes
constexpr int DC_TPB = 256;
constexpr int DC_ITEMS = 8;                   // tokens of a thread
constexpr uint32_t DC_TILE = DC_TPB * DC_ITEMS;
constexpr uint32_t DC_STAGE = 24 * 1024;      // text bytes staged in LDS; a tile with more writes directly
constexpr int DC_SUM_TPB = 1024;
constexpr uint32_t DC_CHUNKS = 1024;          // at most
// Up to this many chunks the last one to end tells the polling host, beyond it
// the host waits for the stream: every workgroup that tells writes back an L2
// (20,000 tokens: 21.4 against 25.1 us a call; 100,000: 22.6 against 25.4;
// 300,000: 27.1 against 26.2).
constexpr uint32_t DC_TELL = 64;
constexpr uint32_t DC_SUM_STEP = DC_SUM_TPB * 4;

struct DecTable {
    const uint4* entry;       // one for each id, and an empty one for no token
    const uint4* pool;        // long strings, each from a piece of 16 bytes on
    const uint8_t* length;    // of each id's string, DC_LONG where that is in its entry; padded to 16 bytes
    uint32_t n;               // ids
};

// A chunk's sum of lengths, and the lowest position in it of an id outside
// the vocabulary (all ones if there is none).
struct DecChunk {
    unsigned long long sum;
    unsigned long long bad;
};

// What a call reports to the host: the text's length, and the lowest
// position of an id outside the vocabulary (all ones if there is none).
struct DecResult {
    unsigned long long total;
    unsigned long long bad;
    unsigned long long ended;  // the last call of those that say so whose writes can all be seen
};

__device__ __forceinline__ uint32_t dec_length(const uint4& e) {
    const uint32_t l = e.w >> 24;
    return l == DC_LONG ? e.y : l;
}

__device__ __forceinline__ uint64_t dec_sum(const uint4 (&e)[DC_ITEMS]) {
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < DC_ITEMS; ++i) sum += dec_length(e[i]);
    return sum;
}

// Whether t is neither an id, tagged or not, nor no token.
__device__ __forceinline__ bool dec_bad(const DecTable& tab, uint32_t t) {
    return t != DC_NONE && ((t >> 17) != 0u || (t & 0xFFFFu) >= tab.n);
}

// The entries of a thread's tokens, which are good ones.
__device__ __forceinline__ void dec_entries(const DecTable& tab, const uint32_t (&t)[DC_ITEMS], uint4 (&e)[DC_ITEMS]) {
#pragma unroll
    for (int i = 0; i < DC_ITEMS; ++i) e[i] = tab.entry[t[i] == DC_NONE ? tab.n : t[i] & 0xFFFFu];
}
__device__ __forceinline__ void dec_tokens(const uint32_t* __restrict__ tokens, uint64_t at, uint64_t end,
                                           uint32_t (&t)[DC_ITEMS]) {
    if (at + DC_ITEMS <= end) {
        __builtin_memcpy(t, tokens + at, sizeof t);
    } else {
#pragma unroll
        for (int i = 0; i < DC_ITEMS; ++i) t[i] = at + i < end ? tokens[at + i] : DC_NONE;
    }
}

// The first l <= 16 bytes of v to p, of which room bytes are this thread's:
// all of v where there is room (what comes next takes the place of what is
// too much), else in pieces of 16, 8, 4, 2 and 1.
__device__ __forceinline__ void dec_bytes(uint4 v, uint32_t l, uint8_t* p, uint32_t room) {
    if (room >= 16u) {
        __builtin_memcpy(p, &v, 16);
        return;
    }
    uint64_t q = (uint64_t)v.y << 32 | v.x;
    if (l & 8u) {
        __builtin_memcpy(p, &q, 8);
        p += 8;
        q = (uint64_t)v.w << 32 | v.z;
    }
    if (l & 4u) {
        const uint32_t w = (uint32_t)q;
        __builtin_memcpy(p, &w, 4);
        p += 4;
        q >>= 32;
    }
    if (l & 2u) {
        const uint16_t w = (uint16_t)q;
        __builtin_memcpy(p, &w, 2);
        p += 2;
        q >>= 16;
    }
    if (l & 1u) *p = (uint8_t)q;
}

// A thread's strings from p on.
__device__ __forceinline__ void dec_write(const DecTable& tab, const uint4 (&e)[DC_ITEMS], uint64_t own, uint8_t* p) {
#pragma unroll
    for (int i = 0; i < DC_ITEMS; ++i) {
        const uint32_t l = e[i].w >> 24;
        if (l != DC_LONG) {
            dec_bytes(e[i], l, p, own < 16u ? (uint32_t)own : 16u);
            p += l;
            own -= l;
        } else {
            for (uint32_t at = 0; at < e[i].y; at += 16u) {
                const uint32_t part = min(16u, e[i].y - at);
                dec_bytes(tab.pool[e[i].x + at / 16u], part, p, own < 16u ? (uint32_t)own : 16u);
                p += part;
                own -= part;
            }
        }
    }
}

// Writes a tile's text: every thread's strings (of own bytes) from start (its
// place in the text of the whole call) on; begin and size say where the
// tile's text lies.
__device__ __forceinline__ void dec_emit(const DecTable& tab, const uint4 (&e)[DC_ITEMS], uint64_t own, uint64_t start,
                                         uint64_t begin, uint64_t size, uint8_t* __restrict__ out, uint8_t* stage) {
    uint8_t* dst = out + begin;
    const uint32_t skew = (uint32_t)((uintptr_t)dst & 15u);  // LDS and memory then break into the same pieces
    if (size + skew > DC_STAGE) {
        dec_write(tab, e, own, out + start);
        return;
    }
    dec_write(tab, e, own, stage + skew + (uint32_t)(start - begin));
    lds_sync();
    const uint32_t end = skew + (uint32_t)size;
    uint8_t* base = dst - skew;
    for (uint32_t b = threadIdx.x * 16u; b < end; b += DC_TPB * 16u) {
        if (b >= skew && b + 16u <= end) {
            *(uint4*)(base + b) = *(const uint4*)(stage + b);
        } else {
            for (uint32_t i = b < skew ? skew : b; i < end && i < b + 16u; ++i) base[i] = stage[i];
        }
    }
}

__device__ __forceinline__ void dec_offsets(const uint4 (&e)[DC_ITEMS], uint64_t at, uint64_t n, uint64_t start,
                                            int64_t* __restrict__ offsets) {
#pragma unroll
    for (int i = 0; i < DC_ITEMS; ++i) {
        if (at + i < n) offsets[at + i] = (int64_t)start;
        start += dec_length(e[i]);
    }
}

// Exclusive prefix of v over the workgroup's threads, and the total.
template <int TPB>
__device__ __forceinline__ uint64_t block_exclusive(uint64_t v, uint64_t* s_wave, uint64_t* total) {
    const uint32_t lane = threadIdx.x & 63u, w = threadIdx.x >> 6;
    const uint64_t incl = wave_inclusive(v, uint64_t(0), [](uint64_t a, uint64_t b) { return a + b; });
    if (lane == 63u) s_wave[w] = incl;
    lds_sync();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < TPB / 64; ++i) {
        before += i < (int)w ? s_wave[i] : 0;
        all += s_wave[i];
    }
    *total = all;
    return before + incl - v;
}

// A workgroup's last step: what it wrote can be seen by all, and once that
// holds for every workgroup, the host is told that this call has ended. left
// counts the workgroups that have not come so far. One wave writes back the
// L2 for all, once each has seen its own stores arrive there (a barrier alone
// does not wait for them).
__device__ __forceinline__ void dec_end(DecResult* res, unsigned long long call, unsigned* left) {
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    __syncthreads();
    if (threadIdx.x != 0) return;
    __threadfence_system();
    if (left && __hip_atomic_fetch_sub(left, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != 1u) return;
    __hip_atomic_store(&res->ended, call, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_SYSTEM);
}

// One workgroup does it all, for n <= DC_TILE.
__global__ __launch_bounds__(DC_TPB) void k_dec_small(DecTable tab, const uint32_t* __restrict__ tokens, uint32_t n,
                                                      uint8_t* __restrict__ out, uint64_t cap,
                                                      int64_t* __restrict__ offsets, DecResult* res,
                                                      unsigned long long call) {
    __shared__ uint64_t s_wave[DC_TPB / 64];
    __shared__ unsigned long long s_bad;
    __shared__ __align__(16) uint8_t stage[DC_STAGE];
    if (threadIdx.x == 0) s_bad = ~0ull;
    lds_sync();
    uint32_t t[DC_ITEMS];
    uint4 e[DC_ITEMS];
    const uint64_t at = (uint64_t)threadIdx.x * DC_ITEMS;
    dec_tokens(tokens, at, n, t);
#pragma unroll
    for (int i = 0; i < DC_ITEMS; ++i) {
        if (dec_bad(tab, t[i])) {
            atomicMin(&s_bad, (unsigned long long)(at + i));
            t[i] = DC_NONE;
        }
    }
    dec_entries(tab, t, e);
    const uint64_t own = dec_sum(e);
    uint64_t total;
    const uint64_t start = block_exclusive<DC_TPB>(own, s_wave, &total);  // its barrier also settles s_bad
    const bool good = s_bad == ~0ull;
    if (threadIdx.x == 0) {
        res->total = total;
        res->bad = s_bad;
    }
    if (good && offsets) {
        dec_offsets(e, at, n, start, offsets);
        if (threadIdx.x == 0) offsets[n] = (int64_t)total;
    }
    if (good && out && total <= cap) dec_emit(tab, e, own, start, 0, total, out, stage);
    dec_end(res, call, nullptr);
}

// The sum of lengths of chunk blockIdx.x: tokens [blockIdx.x * per, + per).
__global__ __launch_bounds__(DC_SUM_TPB) void k_dec_sum(DecTable tab, const uint32_t* __restrict__ tokens, uint64_t n,
                                                        uint64_t per, DecChunk* __restrict__ chunk,
                                                        unsigned* __restrict__ left) {
    extern __shared__ __align__(16) uint8_t s_length[];
    __shared__ uint64_t s_wave[DC_SUM_TPB / 64];
    __shared__ unsigned long long s_bad;
    if (threadIdx.x == 0) s_bad = ~0ull;
    for (uint32_t i = threadIdx.x * 16u; i < tab.n; i += DC_SUM_TPB * 16u)
        *(uint4*)(s_length + i) = *(const uint4*)(tab.length + i);
    lds_sync();
    const uint64_t end = min(n, (blockIdx.x + 1u) * per);
    uint64_t sum = 0;
    for (uint64_t at = blockIdx.x * per + threadIdx.x * 4u; at < end; at += DC_SUM_STEP) {
        uint32_t t[4];
        if (at + 4u <= end) {
            __builtin_memcpy(t, tokens + at, sizeof t);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = at + i < end ? tokens[at + i] : DC_NONE;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (dec_bad(tab, t[i])) {
                atomicMin(&s_bad, (unsigned long long)(at + i));
            } else if (t[i] != DC_NONE) {
                const uint32_t id = t[i] & 0xFFFFu, l = s_length[id];
                sum += l == DC_LONG ? tab.entry[id].y : l;
            }
        }
    }
    uint64_t total;
    (void)block_exclusive<DC_SUM_TPB>(sum, s_wave, &total);  // its barrier also settles s_bad
    if (threadIdx.x == 0) {
        chunk[blockIdx.x].sum = total;
        chunk[blockIdx.x].bad = s_bad;
        if (blockIdx.x == 0) *left = gridDim.x;
    }
}

// The text of chunk blockIdx.x, at the sum of those before it.
__global__ __launch_bounds__(DC_TPB) void k_dec_copy(DecTable tab, const uint32_t* __restrict__ tokens, uint64_t n,
                                                     uint64_t per, const DecChunk* __restrict__ chunk,
                                                     uint8_t* __restrict__ out, uint64_t cap,
                                                     int64_t* __restrict__ offsets, DecResult* res,
                                                     unsigned long long call, unsigned* left) {
    __shared__ uint64_t s_wave[2][DC_TPB / 64];
    __shared__ unsigned long long s_bad;
    __shared__ __align__(16) uint8_t stage[DC_STAGE];
    if (threadIdx.x == 0) s_bad = ~0ull;
    lds_sync();
    uint64_t mine = 0, before = 0, bad = ~0ull, total, begin;
    for (uint32_t c = threadIdx.x; c < gridDim.x; c += DC_TPB) {
        const DecChunk v = chunk[c];
        mine += v.sum;
        before += c < blockIdx.x ? v.sum : 0;
        bad = v.bad < bad ? v.bad : bad;
    }
    if (bad != ~0ull) atomicMin(&s_bad, (unsigned long long)bad);
    (void)block_exclusive<DC_TPB>(mine, s_wave[0], &total);
    (void)block_exclusive<DC_TPB>(before, s_wave[1], &begin);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        res->total = total;
        res->bad = s_bad;
    }
    const bool good = s_bad == ~0ull, write = good && out && total <= cap;
    // nothing to write: no tokens
    const uint64_t end = write || (good && offsets) ? min(n, (blockIdx.x + 1u) * per) : 0;
    uint32_t t[DC_ITEMS];
    dec_tokens(tokens, blockIdx.x * per + threadIdx.x * DC_ITEMS, end, t);
    for (uint64_t t0 = blockIdx.x * per; t0 < end; t0 += DC_TILE) {
        uint4 e[DC_ITEMS];
        const uint64_t at = t0 + threadIdx.x * DC_ITEMS;
        uint64_t size;
        dec_entries(tab, t, e);
        const uint64_t own = dec_sum(e);
        dec_tokens(tokens, at + DC_TILE, end, t);  // the next tile's, on their way meanwhile
        lds_sync();  // and the tile before has left the staging
        const uint64_t start = begin + block_exclusive<DC_TPB>(own, s_wave[0], &size);
        if (offsets) dec_offsets(e, at, end, start, offsets);
        if (write) dec_emit(tab, e, own, start, begin, size, out, stage);
        begin += size;
    }
    if (good && offsets && blockIdx.x == gridDim.x - 1u && threadIdx.x == 0) offsets[n] = (int64_t)total;
    if (call) dec_end(res, call, left);
}

}  // namespace bpek
