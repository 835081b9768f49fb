// How calls of the operators between a hidden state and text are cut into
// launches: host arithmetic on sizes alone, so that it can be checked without
// a device.
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

}  // namespace bpek
