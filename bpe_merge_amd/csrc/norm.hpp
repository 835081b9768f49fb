// Residual addition, root-mean-square norm and 8-bit output with scales.
// Bound by memory: 16,384 rows of 8,192 bfloat16 with a residual take 174 us,
// 5.4 TB/s of the 944 MB they read and write (a copy of 1 GiB reaches 5.1);
// one row of 2,048 takes 2.6 us. Weights of 64,256 x 4,096 bfloat16 take 139 us,
// 5.7 TB/s.
//
//   h = x + r                       (f32; stored in x's type)
//   y = h * w / sqrt(mean(h^2) + eps)
//   s = max(max|y| / 448, 2^-126)   over each block of 128 columns
//   q = e4m3(y / s)                 (the f32 quotient, round to nearest even)
//
// One pass over memory: a row stays in registers between its sum of squares
// and its output, so each input is read once and each output written once.
// A lane holds 8 neighbouring columns, 16 lanes a block: the block's maximum
// is four DPP steps. Squares are summed in f64: f32 squares overflow from
// 1.8e19 on, and the f64 sum costs one conversion and one FMA per element in
// a kernel that memory bounds. The norm uses the sum before it is rounded
// for storage, so only stored values are rounded.
#pragma once

#include "lanes.hpp"

namespace bpek {

constexpr int NQ_BLOCK = 128;           // columns that share a scale
constexpr float NQ_MAX = 448.0f;        // largest e4m3 value
constexpr float NQ_TINY = 0x1p-126f;    // smallest scale: a block of zeros divides by it

// Two f32 values as e4m3 in the low (HIGH false) or high half of old.
template <bool HIGH>
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, uint32_t old) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HIGH);
}
__device__ __forceinline__ uint64_t to_e4m3(const float (&v)[8]) {
    uint32_t lo = to_e4m3<false>(v[0], v[1], 0u), hi = to_e4m3<false>(v[4], v[5], 0u);
    lo = to_e4m3<true>(v[2], v[3], lo);
    hi = to_e4m3<true>(v[6], v[7], hi);
    return (uint64_t)hi << 32 | lo;
}

// The scale of values whose largest magnitude has these bits. As unsigned
// numbers the bits of NaN are above those of infinity and of every value, so
// the maximum over them keeps a NaN, and the scale is then NaN.
__device__ __forceinline__ float scale_of(uint32_t max_bits) {
    const float s = __builtin_bit_cast(float, max_bits) / NQ_MAX;
    return s < NQ_TINY ? NQ_TINY : s;
}

// v / s, each as the f32 division gives it: the product with the rounded
// reciprocal, put right by what it leaves of v (exact in one FMA). 16 bits often
// lie half way between two codes, where the product alone falls to either side
// (one of 2,000 bfloat16 weights came out a code off). The division itself for
// each would cost 16,384 x 8,192 rows 182 us instead of 174, and 2,000 x 20,000
// 180 instead of 142.
__device__ __forceinline__ void divide(float (&v)[8], float s) {
    if (s < 0x1p-90f) {  // remainders of such numbers could leave the range of f32
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= 0x1p64f;
        s *= 0x1p64f;
    }
    const float inv = 1.0f / s, left = s < __builtin_inff() ? s : 0.0f;  // (by infinity: 0, and NaN for its own like)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = v[i] * inv;
        v[i] = __builtin_fmaf(-__builtin_fmaf(q, left, -v[i]), inv, q);
    }
}

// WAVES waves share a row (1: a workgroup takes 4 rows); a lane holds VPL
// vectors of 8 columns.
template <typename T, int WAVES, int VPL>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void k_norm_quant(
    const typename T::raw* x, size_t xs, const typename T::raw* r, size_t rs,
    const typename T::raw* __restrict__ w, uint32_t rows, uint32_t d, float eps, typename T::raw* sum, size_t ss,
    uint8_t* __restrict__ q, size_t qs, float* __restrict__ scales) {
    constexpr uint32_t TPR = 64u * WAVES;
    __shared__ double s_sum[WAVES];
    const uint32_t lane = threadIdx.x % TPR;
    const uint32_t row = WAVES == 1 ? blockIdx.x * 4u + threadIdx.x / 64u : blockIdx.x;
    if (WAVES == 1 && row >= rows) return;
    x += row * xs;
    if (r) r += row * rs;
    float h[VPL][8];
    double squares = 0.0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const uint32_t c = (j * TPR + lane) * 8u;
        if (c + 8u <= d) {
            load_n<T>(x + c, h[j]);
            if (r) {
                float t[8];
                load_n<T>(r + c, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] += t[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[j][i] = c + i < d ? T::get(x[c + i]) : 0.0f;
                if (r && c + i < d) h[j][i] += T::get(r[c + i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) squares += (double)h[j][i] * (double)h[j][i];
    }
    if (sum) {  // sum may be x or r itself: a lane writes only the columns that it has read
        sum += row * ss;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const uint32_t c = (j * TPR + lane) * 8u;
            if (c + 8u <= d) {
                store_n<T>(sum + c, h[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < d) sum[c + i] = T::put(h[j][i]);
            }
        }
    }
    squares = wave_sum(squares);
    if (WAVES > 1) {
        if (lane % 64u == 0) s_sum[lane / 64u] = squares;
        lds_sync();
        squares = 0.0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) squares += s_sum[i];
    }
    const double inv = 1.0 / sqrt(squares / (double)d + (double)eps);
    float inv_rms = (float)inv;
    if (inv > 0x1p100) {  // only with an eps of 0: past the range of f32, where the row itself is as near to zero
        inv_rms = (float)(inv * 0x1p-64);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) h[j][i] *= 0x1p64f;
    }
    const uint32_t blocks = (d + NQ_BLOCK - 1u) / NQ_BLOCK;
    q += row * qs;
    scales += (size_t)row * blocks;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        const uint32_t c = (j * TPR + lane) * 8u;
        float g[8];
        if (c + 8u <= d) {
            load_n<T>(w + c, g);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = c + i < d ? T::get(w[c + i]) : 0.0f;
        }
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // columns past d hold h = 0; they do not take part, whatever inv_rms is
            h[j][i] = h[j][i] * inv_rms * g[i];
            const uint32_t bits = c + i < d ? __builtin_bit_cast(uint32_t, h[j][i]) & 0x7FFFFFFFu : 0u;
            top = bits > top ? bits : top;
        }
        top = row_all(top, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
        const float s = scale_of(top);
        divide(h[j], s);  // at most 448 (1 + 2^-23): rounds to at most 448
        const uint64_t v = to_e4m3(h[j]);
        if (c + 8u <= d) {
            __builtin_memcpy(q + c, &v, 8);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < d) q[c + i] = (uint8_t)(v >> (8 * i));
        }
        if (lane % 16u == 0 && c < d) scales[c / NQ_BLOCK] = s;
    }
}

// A matrix in e4m3 with one scale for each 128 x 128 block (a workgroup
// takes a block: 256 threads, 64 elements each, in registers between the
// block's maximum and its output). Done once when weights are loaded.
template <typename T>
__global__ __launch_bounds__(256) void k_quant_weight(const typename T::raw* __restrict__ w, size_t ws, uint32_t n,
                                                      uint32_t k, uint8_t* __restrict__ q, size_t qs,
                                                      float* __restrict__ scales) {
    __shared__ uint32_t s_top[4];
    const uint32_t t = threadIdx.x, kb = blockIdx.x, nb = blockIdx.y;
    const uint32_t c = kb * NQ_BLOCK + (t % 16u) * 8u, r0 = nb * NQ_BLOCK + t / 16u;
    float v[8][8];
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t r = r0 + 16u * j;
        if (r < n && c + 8u <= k) {
            load_n<T>(w + r * ws + c, v[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = r < n && c + i < k ? T::get(w[r * ws + c + i]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = __builtin_bit_cast(uint32_t, v[j][i]) & 0x7FFFFFFFu;
            top = bits > top ? bits : top;
        }
    }
    top = wave_all(top, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    if (t % 64u == 0) s_top[t / 64u] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = s_top[i] > top ? s_top[i] : top;
    const float s = scale_of(top);
    if (t == 0) scales[(size_t)nb * gridDim.x + kb] = s;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t r = r0 + 16u * j;
        if (r >= n) break;
        divide(v[j], s);
        const uint64_t e = to_e4m3(v[j]);
        if (c + 8u <= k) {
            __builtin_memcpy(q + r * qs + c, &e, 8);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < k) q[r * qs + c + i] = (uint8_t)(e >> (8 * i));
        }
    }
}

}  // namespace bpek
