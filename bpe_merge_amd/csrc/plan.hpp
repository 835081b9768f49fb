// How calls of the operators between a hidden state and text are cut into
// launches, and which arrays may not share memory: host arithmetic on sizes
// alone, so that it can be checked without a device.
#pragma once

#include <stdint.h>

namespace bpek {

// A launch takes fewer than 2^32 threads in x and fewer than 2^16 workgroups in
// y. Rows that need more are launched in parts.
constexpr uint64_t groups_in_x(uint64_t threads) { return 0xFFFFFFFFull / threads; }
constexpr uint64_t GROUPS_IN_Y = 0xFFFF;

// Calls f(first row, rows, workgroups) for each part, where a workgroup takes
// group_rows rows and a launch at most most_groups workgroups.
template <typename F>
void in_parts(uint64_t rows, uint64_t group_rows, uint64_t most_groups, F f) {
    const uint64_t most = most_groups * group_rows;
    for (uint64_t at = 0; at < rows; at += most) {
        const uint64_t part = rows - at < most ? rows - at : most;
        f(at, uint32_t(part), uint32_t((part + group_rows - 1) / group_rows));
    }
}

// Whether two arrays of so many bytes share any.
inline bool share_bytes(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
    const uint64_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return a_bytes && b_bytes && p < q + b_bytes && q < p + a_bytes;
}

// The same for two arrays of rows of so many bytes, strides (in bytes) apart.
// Rows of one stride may lie between each other; of two they may not.
inline bool share_rows(const void* a, uint64_t a_stride, const void* b, uint64_t b_stride, uint64_t rows, uint64_t width) {
    if (!rows || !share_bytes(a, (rows - 1) * a_stride + width, b, (rows - 1) * b_stride + width)) return false;
    if (rows == 1 || a_stride != b_stride) return true;
    const uint64_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    const uint64_t off = (p < q ? q - p : p - q) % a_stride;
    return off < width || off + width > a_stride;
}

// ---------------------------------------------------------------- product

enum Pieces {
    PR_FULL,    // copied: rows of whole blocks, aligned to 16 bytes
    PR_SHORT,   // copied: rows of whole pieces (128 bytes at least), aligned to 16 bytes
    PR_ODD,     // through registers: rows of 128 bytes at least
    PR_NARROW   // through registers: rows of fewer, one block
};
constexpr bool copied(Pieces kind) { return kind == PR_FULL || kind == PR_SHORT; }

// The pieces of rows of k bytes.
constexpr Pieces pieces_of(uint64_t k, bool aligned_rows) {
    if (k < 128) return PR_NARROW;
    if (k % 16 != 0 || !aligned_rows) return PR_ODD;
    return k % 128 == 0 ? PR_FULL : PR_SHORT;
}

enum ProductKernel {
    PK_PARTS_16,            // streams over eight parts of K, rows of a to a workgroup
    PK_PARTS_32,
    PK_PARTS_64,
    PK_STREAM_16,           // streams over four
    PK_STREAM_32,
    PK_STREAM_64,
    PK_TILE_128_64,         // tiles of so many rows of b and of a
    PK_TILE_256_256,
    PK_TILE_256_128,
    PK_TILE_128_128_WAVES,  // eight waves instead of four
    PK_TILE_128_128,
    PK_COUNT
};

// Streams over eight parts of K: of the most rows of a that leave a workgroup
// to nearly every CU (rows of b x rows of a x K, 16, 32 or 64 rows of a to a
// workgroup: 456 x 128 x 8,192, 11, 17 or 27 us; 2,000 x 64 x 4,096, 11, 10 or
// 15; 456 x 500 x 4,091, 23, 20 or 18).
constexpr ProductKernel parts_kernel(uint64_t m, uint64_t n) {
    auto workgroups = [&](uint64_t rows) { return (n + 15) / 16 * ((m + rows - 1) / rows); };
    if (m > 32 && workgroups(64) >= 200) return PK_PARTS_64;
    if (m > 16 && workgroups(32) >= 200) return PK_PARTS_32;
    return PK_PARTS_16;
}

// Streams for any rows.
constexpr ProductKernel stream_kernel(uint64_t m, uint64_t n, uint64_t blocks) {
    if (n < 512 * 32 && blocks >= 16) return parts_kernel(m, n);
    return m <= 16 ? PK_STREAM_16 : m <= 32 ? PK_STREAM_32 : PK_STREAM_64;
}

// The tile for more than 64 rows, by the time a block of K takes (measured,
// in us): 256 x 256, one to a CU, 2.1; 256 x 128, one to a CU, 1.15; 128 x
// 128, 0.85 alone on a CU and 1.55 for two. On 2,048 x 65,536 x 4,096 they
// take 534, 620 and 775 us; on 1,024 x 8,192 x 8,192, where the widest leave
// half of the CUs idle, 106, 66 and 78 us. Exact sums (f32 and binary16 results)
// take 1.6 times as long in each, and have no 256 x 256, whose registers do not
// hold their fragments (nor anything but full blocks); 128 x 128 alone on a CU
// then takes 8 waves (128 x 32,256 x 4,096: 41 against 54 us). Pieces that go
// through registers take the last (700 x 32,256 x 3,909: 215 us, 235 in the
// second; 142 where rows are whole pieces). Where even of the last there are
// only a few, streams over parts of K keep more of the chip busy (128 x 456 x
// 8,192: 66 against 11 us; 1,000 x 456 x 8,191: 86 against 64).
constexpr ProductKernel tile_kernel(uint64_t m, uint64_t n, uint64_t blocks, Pieces kind, bool exact) {
    constexpr uint64_t CUS = 256;
    auto up = [](uint64_t a, uint64_t b) { return (a + b - 1) / b; };
    auto tiles = [&](uint64_t bn, uint64_t bm) { return up(n, bn) * up(m, bm); };
    const uint64_t wide = up(tiles(256, 256), CUS) * 210, mid = up(tiles(256, 128), CUS) * 115;
    if (tiles(128, 128) <= 40 && blocks >= 16) return parts_kernel(m, n);
    const uint64_t narrow = tiles(128, 128) <= CUS ? 85 : up(tiles(128, 128), 2 * CUS) * 155;
    if (!exact && kind == PR_FULL && wide <= mid && wide <= narrow) return PK_TILE_256_256;
    if (copied(kind) && mid <= narrow) return PK_TILE_256_128;
    if (exact && kind != PR_NARROW && tiles(128, 128) <= CUS) return PK_TILE_128_128_WAVES;
    return PK_TILE_128_128;
}

// Up to 64 rows. Streaming b costs a read of a's rows beside every read of
// b's, so that 4 rows already take longer than through LDS (64,256 x 4,096,
// 16 rows: 87 against 55 us; 4 rows: 62; 1 row: 50 us); but a tile is 128 rows
// of b, and where there are few of them streams over parts of K keep more busy
// (61 rows x 4,352: 23 against 27 us for 4,256 rows of b, 45 against 30 us for
// 16,256). Rows that are not whole pieces go through LDS one block ahead only,
// which pays from more 16 x 16 tiles on (streams against LDS: 60 x 8,256 x
// 1,001, 10 against 13 us; 5 x 32,256 x 4,001, 47 against 57; 61 x 16,256 x
// 4,353, 75 against 50; 16 x 64,256 x 4,095, 133 against 71).
constexpr ProductKernel few_kernel(uint64_t m, uint64_t n, uint64_t blocks, Pieces kind) {
    const bool tile = copied(kind) ? m > 3 && n >= 128 * 48 : m > 8 && (m + 15) / 16 * n >= 48000;
    return tile ? PK_TILE_128_64 : stream_kernel(m, n, blocks);
}

// The kernel for m x n results of so many blocks of K. exact: whether all
// inner sums are; tiled: whether a tile's rows lie within 32-bit offsets.
constexpr ProductKernel product_kernel(uint64_t m, uint64_t n, uint64_t blocks, Pieces kind, bool exact, bool tiled) {
    if (!tiled) return stream_kernel(m, n, blocks);
    return m <= 64 ? few_kernel(m, n, blocks, kind) : tile_kernel(m, n, blocks, kind, exact);
}

}  // namespace bpek
