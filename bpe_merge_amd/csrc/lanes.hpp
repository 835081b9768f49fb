// Device helpers of the kernels between a model's last hidden state and
// text: moves between lanes of a wave by DPP (no LDS round trip), loads
// and stores of any alignment, and number types.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bpek {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// DPP controls: swaps inside a quad, reversal of 8 and of 16 lanes, shifts
// towards higher lanes inside a row of 16, and copies of a row's last lane.
constexpr int LN_SWAP1 = 0xB1, LN_SWAP2 = 0x4E, LN_MIRROR8 = 0x141, LN_MIRROR16 = 0x140;
constexpr int LN_SHR1 = 0x111, LN_SHR2 = 0x112, LN_SHR4 = 0x114, LN_SHR8 = 0x118;
constexpr int LN_BCAST15 = 0x142, LN_BCAST31 = 0x143;

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t lane_move(uint32_t ident, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)ident, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint64_t lane_move(uint64_t ident, uint64_t v) {
    return (uint64_t)lane_move<CTRL, ROWS>((uint32_t)(ident >> 32), (uint32_t)(v >> 32)) << 32 |
           lane_move<CTRL, ROWS>((uint32_t)ident, (uint32_t)v);
}
template <int CTRL>
__device__ __forceinline__ double lane_move(double v) {
    return __longlong_as_double((long long)lane_move<CTRL>(uint64_t(0), (uint64_t)__double_as_longlong(v)));
}

// Every lane of a row of 16 gets op over the row.
template <typename V, typename Op>
__device__ __forceinline__ V row_all(V v, Op op) {
    v = op(v, lane_move<LN_SWAP1>(v, v));
    v = op(v, lane_move<LN_SWAP2>(v, v));
    v = op(v, lane_move<LN_MIRROR8>(v, v));
    v = op(v, lane_move<LN_MIRROR16>(v, v));
    return v;
}

// Inclusive scan over the wave: op(a, b) is a then b, ident its identity.
template <typename V, typename Op>
__device__ __forceinline__ V wave_inclusive(V v, V ident, Op op) {
    v = op(lane_move<LN_SHR1>(ident, v), v);
    v = op(lane_move<LN_SHR2>(ident, v), v);
    v = op(lane_move<LN_SHR4>(ident, v), v);
    v = op(lane_move<LN_SHR8>(ident, v), v);
    v = op(lane_move<LN_BCAST15, 0xA>(ident, v), v);
    v = op(lane_move<LN_BCAST31, 0xC>(ident, v), v);
    return v;
}

__device__ __forceinline__ uint32_t read_lane(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
    return (uint64_t)read_lane((uint32_t)(v >> 32), lane) << 32 | read_lane((uint32_t)v, lane);
}

// op over the wave, in every lane (from the scan's last lane: uniform).
template <typename V, typename Op>
__device__ __forceinline__ V wave_all(V v, V ident, Op op) {
    return read_lane(wave_inclusive(v, ident, op), 63);
}

__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
    return wave_all(v, uint64_t(0), [](uint64_t a, uint64_t b) { return a + b; });
}
__device__ __forceinline__ double wave_sum(double v) {
    v += lane_move<LN_SWAP1>(v);
    v += lane_move<LN_SWAP2>(v);
    v += lane_move<LN_MIRROR8>(v);
    v += lane_move<LN_MIRROR16>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// A barrier for LDS alone: global loads and stores stay in flight.
__device__ __forceinline__ void lds_sync() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Element types of caller arrays, by the tag that the C ABI passes.
struct F32 {
    typedef float raw;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
struct F16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float get(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
    static __device__ __forceinline__ uint16_t put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct BF16 {
    typedef uint16_t raw;
    static __device__ __forceinline__ float get(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t put(float v) {
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};

// N elements from p, which is aligned to an element only (the hardware takes
// wide accesses at any address; they cost more only where they cross lines).
template <typename T, int N>
__device__ __forceinline__ void load_n(const typename T::raw* p, float (&v)[N]) {
    typename T::raw r[N];
    __builtin_memcpy(r, p, sizeof r);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = T::get(r[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_n(typename T::raw* p, const float (&v)[N]) {
    typename T::raw r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = T::put(v[i]);
    __builtin_memcpy(p, r, sizeof r);
}

}  // namespace bpek
