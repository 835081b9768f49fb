// Entry points of the operators between a model's last hidden state and
// text (include/bpe.h): norm with 8-bit output, scaled 8-bit product,
// sampling, and decoding of ids.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <chrono>
#include <cstring>
#include <initializer_list>
#include <new>
#include <type_traits>
#include <vector>

#include "../../include/bpe.h"
#include "host.hpp"
#include "decode.hpp"
#include "norm.hpp"
#include "plan.hpp"
#include "product.hpp"
#include "sample.hpp"

using bpeh::g_err;
using bpeh::set_err;

namespace {

struct Arg {
    const char* name;
    const void* p;
    bool optional;
};

// The device that holds all of these arrays; every one has to be device
// memory of that device.
bpe_status device_of(std::initializer_list<Arg> args, int* device) {
    int dev = -1;
    for (const Arg& a : args) {
        if (!a.p) {
            if (a.optional) continue;
            set_err("%s must be non-NULL", a.name);
            return BPE_EINVAL;
        }
        hipPointerAttribute_t at;
        if (hipPointerGetAttributes(&at, a.p) != hipSuccess ||
            (at.type != hipMemoryTypeDevice && at.type != hipMemoryTypeManaged)) {
            (void)hipGetLastError();
            set_err("%s must be device memory", a.name);
            return BPE_EINVAL;
        }
        if (dev >= 0 && at.device != dev) {
            set_err("%s is on device %d, arrays before it on device %d", a.name, at.device, dev);
            return BPE_EINVAL;
        }
        dev = at.device;
    }
    *device = dev;
    return BPE_OK;
}

// Whether an array of a call on this device is host memory or the device's
// own; memory of another device is an error.
bpe_status place_of(const char* name, const void* p, int device, bool* host) {
    hipPointerAttribute_t at;
    *host = true;
    if (hipPointerGetAttributes(&at, p) != hipSuccess) {
        (void)hipGetLastError();
        return BPE_OK;
    }
    if (at.type == hipMemoryTypeManaged) {
        *host = false;
    } else if (at.type == hipMemoryTypeDevice) {
        *host = false;
        if (at.device != device) {
            set_err("%s is on device %d, the call on device %d", name, at.device, device);
            return BPE_EINVAL;
        }
    }
    return BPE_OK;
}

// Makes a device current for a call, and puts the caller's back.
class OnDevice {
public:
    explicit OnDevice(int device) {
        if (hipGetDevice(&before_) == hipSuccess && before_ != device) moved_ = hipSetDevice(device) == hipSuccess;
    }
    ~OnDevice() {
        if (moved_) (void)hipSetDevice(before_);
    }
    OnDevice(const OnDevice&) = delete;
    OnDevice& operator=(const OnDevice&) = delete;

private:
    int before_ = 0;
    bool moved_ = false;
};

bool type_ok(bpe_type t) { return t == BPE_FLOAT || t == BPE_HALF || t == BPE_BFLOAT; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Calls f with the element type as a type.
template <typename F>
void with_type(bpe_type t, F f) {
    if (t == BPE_FLOAT) f(bpek::F32{});
    else if (t == BPE_HALF) f(bpek::F16{});
    else f(bpek::BF16{});
}
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
size_t size_of(bpe_type t) { return t == BPE_FLOAT ? 4 : 2; }

bool rows_overlap(size_t rows, size_t stride, size_t d) { return rows > 1 && stride < d; }

}  // namespace

extern "C" {

bpe_status bpe_norm_quant(const void* x, size_t x_stride, const void* residual, size_t residual_stride,
                          const void* weight, bpe_type type, size_t rows, size_t d, float eps, void* sum,
                          size_t sum_stride, uint8_t* q, size_t q_stride, float* scales, void* stream) {
    g_err.clear();
    if (!type_ok(type)) {
        set_err("type %d is none of BPE_FLOAT, BPE_HALF, BPE_BFLOAT", int(type));
        return BPE_EINVAL;
    }
    if (d == 0 || d > BPE_NORM_MAX_WIDTH || rows > 0x7FFFFFFFu) {
        set_err("d = %zu must be 1..%u and rows = %zu below 2^31", d, BPE_NORM_MAX_WIDTH, rows);
        return BPE_EINVAL;
    }
    if (!(eps >= 0.0f)) {
        set_err("eps must be 0 or more");
        return BPE_EINVAL;
    }
    if (rows == 0) return BPE_OK;
    if (rows_overlap(rows, x_stride, d) || (residual && rows_overlap(rows, residual_stride, d)) ||
        (sum && rows_overlap(rows, sum_stride, d)) || rows_overlap(rows, q_stride, d)) {
        set_err("a row stride is below d = %zu", d);
        return BPE_EINVAL;
    }
    if ((sum && sum == x && rows > 1 && sum_stride != x_stride) ||
        (sum && sum == residual && rows > 1 && sum_stride != residual_stride)) {
        set_err("a sum in place needs its input's row stride");
        return BPE_EINVAL;
    }
    const size_t es = size_of(type);
    if ((sum && sum != x && bpek::share_rows(sum, sum_stride * es, x, x_stride * es, rows, d * es)) ||
        (sum && residual && sum != residual &&
         bpek::share_rows(sum, sum_stride * es, residual, residual_stride * es, rows, d * es))) {
        set_err("a sum may be x or residual itself, or must share no memory with them");
        return BPE_EINVAL;
    }
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(weight, es) || !aligned(sum, es) || !aligned(scales, 4)) {
        set_err("an array is not aligned to its element type");
        return BPE_EINVAL;
    }
    int device = 0;
    bpe_status st = device_of({{"x", x, false}, {"residual", residual, true}, {"weight", weight, false},
                               {"sum", sum, true}, {"q", q, false}, {"scales", scales, false}}, &device);
    if (st != BPE_OK) return st;
    OnDevice on(device);
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_type(type, [&](auto tag) {
        using T = decltype(tag);
        using raw = typename T::raw;
        auto launch = [&](auto kernel, uint32_t group_rows, uint32_t tpb) {
            bpek::in_parts(rows, group_rows, bpek::groups_in_x(tpb), [&](size_t at, uint32_t part, uint32_t groups) {
                const raw* r = static_cast<const raw*>(residual);
                raw* h = static_cast<raw*>(sum);
                hipLaunchKernelGGL(kernel, dim3(groups), dim3(tpb), 0, s, static_cast<const raw*>(x) + at * x_stride, x_stride,
                                   r ? r + at * residual_stride : r, residual_stride, static_cast<const raw*>(weight), part,
                                   uint32_t(d), eps, h ? h + at * sum_stride : h, sum_stride, q + at * q_stride, q_stride,
                                   scales + at * ((d + 127) / 128));
            });
        };
        // A wave up to 1,024 columns (16 of them a lane; 4 rows in a
        // workgroup, no barrier), 4 waves up to 8,192 (32 a lane; more lanes
        // with fewer columns would wait for each other's sums more often),
        // 16 waves beyond (64 a lane).
        if (d <= 512) launch(bpek::k_norm_quant<T, 1, 1>, 4, 256);
        else if (d <= 1024) launch(bpek::k_norm_quant<T, 1, 2>, 4, 256);
        else if (d <= 2048) launch(bpek::k_norm_quant<T, 4, 1>, 1, 256);
        else if (d <= 4096) launch(bpek::k_norm_quant<T, 4, 2>, 1, 256);
        else if (d <= 8192) launch(bpek::k_norm_quant<T, 4, 4>, 1, 256);
        else launch(bpek::k_norm_quant<T, 16, 8>, 1, 1024);
    });
    HIP_TRY(hipGetLastError());
    return BPE_OK;
}

bpe_status bpe_quant_weight(const void* w, size_t w_stride, bpe_type type, size_t n, size_t k, uint8_t* q,
                            size_t q_stride, float* scales, void* stream) {
    g_err.clear();
    if (!type_ok(type)) {
        set_err("type %d is none of BPE_FLOAT, BPE_HALF, BPE_BFLOAT", int(type));
        return BPE_EINVAL;
    }
    if (n > BPE_PRODUCT_MAX || k > BPE_PRODUCT_MAX) {
        set_err("n = %zu and k = %zu must be at most %u", n, k, BPE_PRODUCT_MAX);
        return BPE_EINVAL;
    }
    if (n == 0 || k == 0) return BPE_OK;
    if (rows_overlap(n, w_stride, k) || rows_overlap(n, q_stride, k)) {
        set_err("a row stride is below k = %zu", k);
        return BPE_EINVAL;
    }
    if (!aligned(w, size_of(type)) || !aligned(scales, 4)) {
        set_err("an array is not aligned to its element type");
        return BPE_EINVAL;
    }
    int device = 0;
    bpe_status st = device_of({{"w", w, false}, {"q", q, false}, {"scales", scales, false}}, &device);
    if (st != BPE_OK) return st;
    OnDevice on(device);
    with_type(type, [&](auto tag) {
        using T = decltype(tag);
        hipLaunchKernelGGL(bpek::k_quant_weight<T>, dim3(uint32_t((k + 127) / 128), uint32_t((n + 127) / 128)),
                           dim3(256), 0, static_cast<hipStream_t>(stream), static_cast<const typename T::raw*>(w),
                           w_stride, uint32_t(n), uint32_t(k), q, q_stride, scales);
    });
    HIP_TRY(hipGetLastError());
    return BPE_OK;
}

}  // extern "C"

namespace {

// Results whose inner sums take the exact form for any number of rows.
template <typename T>
constexpr bool exact_sums = !std::is_same_v<T, bpek::BF16>;

template <typename T, int MT, int NT, int WAVES>
void launch_rows(const bpek::Product& p, hipStream_t s) {
    bpek::in_parts(p.m, MT * 16, bpek::GROUPS_IN_Y, [&](size_t at, uint32_t part, uint32_t groups) {
        bpek::Product here = p;
        here.a += at * p.as;
        here.sa += at * p.sas;
        here.out = static_cast<typename T::raw*>(p.out) + at * p.os;
        here.m = part;
        hipLaunchKernelGGL((bpek::k_product_rows<T, MT, NT, WAVES>), dim3((p.n + NT * 16 - 1) / (NT * 16), groups),
                           dim3(64 * WAVES), 0, s, here);
    });
}

template <typename T, bool EXACT, int BN, int BM, int WN, int WM, int STAGES, bpek::Pieces KIND>
void launch_tile(const bpek::Product& p, hipStream_t s) {
    const uint32_t tn = (p.n + BN - 1) / BN, tm = (p.m + BM - 1) / BM;
    hipLaunchKernelGGL((bpek::k_product_tile<T, EXACT, BN, BM, WN, WM, STAGES, KIND>), dim3(tn * tm), dim3(64 * WN * WM),
                       0, s, p, tn, tm);
}

// The kernel that product_kernel names.
template <typename T>
void launch_streams(bpek::ProductKernel kernel, const bpek::Product& p, hipStream_t s) {
    switch (kernel) {
        case bpek::PK_PARTS_64: return launch_rows<T, 4, 1, 8>(p, s);
        case bpek::PK_PARTS_32: return launch_rows<T, 2, 1, 8>(p, s);
        case bpek::PK_PARTS_16: return launch_rows<T, 1, 1, 8>(p, s);
        case bpek::PK_STREAM_16: return launch_rows<T, 1, 1, 4>(p, s);
        case bpek::PK_STREAM_32: return launch_rows<T, 2, 2, 4>(p, s);
        default: return launch_rows<T, 4, 2, 4>(p, s);
    }
}
template <typename T, bpek::Pieces KIND>
void launch_product(bpek::ProductKernel kernel, const bpek::Product& p, hipStream_t s) {
    constexpr bool EXACT = exact_sums<T>, COPIED = bpek::copied(KIND);
    switch (kernel) {
        case bpek::PK_TILE_128_64: return launch_tile<T, true, 128, 64, 2, 2, COPIED ? 3 : 2, KIND>(p, s);
        case bpek::PK_TILE_256_256:  // (product_kernel names no tile whose condition here does not hold)
            if constexpr (!EXACT && KIND == bpek::PR_FULL) return launch_tile<T, false, 256, 256, 2, 4, 2, KIND>(p, s);
            [[fallthrough]];
        case bpek::PK_TILE_256_128:
            if constexpr (COPIED) return launch_tile<T, EXACT, 256, 128, 4, 2, 3, KIND>(p, s);
            [[fallthrough]];
        case bpek::PK_TILE_128_128_WAVES:
            if constexpr (EXACT && KIND != bpek::PR_NARROW) return launch_tile<T, EXACT, 128, 128, 2, 4, COPIED ? 3 : 2, KIND>(p, s);
            [[fallthrough]];
        case bpek::PK_TILE_128_128: return launch_tile<T, EXACT, 128, 128, 2, 2, 2, KIND>(p, s);
        default: return launch_streams<T>(kernel, p, s);
    }
}

}  // namespace

extern "C" {

bpe_status bpe_matmul_scaled(const uint8_t* a, size_t a_stride, const float* a_scales, size_t a_scales_stride,
                             const uint8_t* b, size_t b_stride, const float* b_scales, size_t b_scales_stride,
                             size_t m, size_t n, size_t k, void* out, size_t out_stride, bpe_type out_type,
                             void* stream) {
    g_err.clear();
    if (!type_ok(out_type)) {
        set_err("type %d is none of BPE_FLOAT, BPE_HALF, BPE_BFLOAT", int(out_type));
        return BPE_EINVAL;
    }
    if (m > BPE_PRODUCT_MAX || n > BPE_PRODUCT_MAX || k > BPE_PRODUCT_MAX || k == 0) {
        set_err("m = %zu, n = %zu, k = %zu must be at most %u, and k at least 1", m, n, k, BPE_PRODUCT_MAX);
        return BPE_EINVAL;
    }
    if (m == 0 || n == 0) return BPE_OK;
    const size_t blocks = (k + 127) / 128;
    if (rows_overlap(m, a_stride, k) || rows_overlap(n, b_stride, k) || rows_overlap(m, out_stride, n) ||
        rows_overlap(m, a_scales_stride, blocks) || rows_overlap((n + 127) / 128, b_scales_stride, blocks)) {
        set_err("a row stride is below its row");
        return BPE_EINVAL;
    }
    if (!aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(out, size_of(out_type))) {
        set_err("an array is not aligned to its element type");
        return BPE_EINVAL;
    }
    int device = 0;
    bpe_status st = device_of({{"a", a, false}, {"a_scales", a_scales, false}, {"b", b, false},
                               {"b_scales", b_scales, false}, {"out", out, false}}, &device);
    if (st != BPE_OK) return st;
    OnDevice on(device);
    hipStream_t s = static_cast<hipStream_t>(stream);
    bpek::Product p;
    p.a = a;
    p.b = b;
    p.sa = a_scales;
    p.sb = b_scales;
    p.out = out;
    p.as = a_stride;
    p.bs = b_stride;
    p.sas = a_scales_stride;
    p.sbs = b_scales_stride;
    p.os = out_stride;
    p.m = uint32_t(m);
    p.n = uint32_t(n);
    p.k = uint32_t(k);
    p.blocks = uint32_t(blocks);
    // tiles need 256 rows within 32-bit offsets, copies whole aligned pieces
    // of 16 bytes
    const bool tiled = (m == 1 || a_stride < (1u << 23)) && (n == 1 || b_stride < (1u << 23));
    const bool aligned_rows = aligned(a, 16) && aligned(b, 16) && (m == 1 || a_stride % 16 == 0) && (n == 1 || b_stride % 16 == 0);
    const bpek::Pieces kind = bpek::pieces_of(k, aligned_rows);
    with_type(out_type, [&](auto tag) {
        using T = decltype(tag);
        const bpek::ProductKernel kernel = bpek::product_kernel(m, n, blocks, kind, exact_sums<T>, tiled);
        if (kind == bpek::PR_NARROW) launch_product<T, bpek::PR_NARROW>(kernel, p, s);
        else if (kind == bpek::PR_ODD) launch_product<T, bpek::PR_ODD>(kernel, p, s);
        else if (kind == bpek::PR_FULL) launch_product<T, bpek::PR_FULL>(kernel, p, s);
        else launch_product<T, bpek::PR_SHORT>(kernel, p, s);
    });
    HIP_TRY(hipGetLastError());
    return BPE_OK;
}

bpe_status bpe_sample(const void* logits, size_t stride, bpe_type type, size_t rows, size_t vocab, const float* u,
                      const bpe_sampling* how, int32_t* ids, float* logp, void* stream) {
    g_err.clear();
    if (!type_ok(type)) {
        set_err("type %d is none of BPE_FLOAT, BPE_HALF, BPE_BFLOAT", int(type));
        return BPE_EINVAL;
    }
    if (vocab == 0 || vocab > BPE_SAMPLE_MAX_VOCAB || rows > 0x7FFFFFFFu) {
        set_err("vocab = %zu must be 1..%u and rows = %zu below 2^31", vocab, BPE_SAMPLE_MAX_VOCAB, rows);
        return BPE_EINVAL;
    }
    if (!how) {
        set_err("the settings must be non-NULL");
        return BPE_EINVAL;
    }
    if (!how->temperatures && !(how->temperature >= 0.0f)) {
        set_err("temperature must be 0 or more");
        return BPE_EINVAL;
    }
    if (!how->top_ks && how->top_k < 0) {
        set_err("top_k must be 0 (off) or more");
        return BPE_EINVAL;
    }
    if (!how->top_ps && !(how->top_p > 0.0f && how->top_p <= 1.0f)) {
        set_err("top_p must be above 0 and at most 1 (off)");
        return BPE_EINVAL;
    }
    if (!how->min_ps && !(how->min_p >= 0.0f && how->min_p <= 1.0f)) {
        set_err("min_p must be 0 (off) to 1");
        return BPE_EINVAL;
    }
    if (rows == 0) return BPE_OK;
    if (rows_overlap(rows, stride, vocab)) {
        set_err("the row stride %zu is below vocab = %zu", stride, vocab);
        return BPE_EINVAL;
    }
    if (!aligned(logits, size_of(type)) || !aligned(u, 4) || !aligned(ids, 4) || !aligned(logp, 4) ||
        !aligned(how->temperatures, 4) || !aligned(how->top_ks, 4) || !aligned(how->top_ps, 4) ||
        !aligned(how->min_ps, 4)) {
        set_err("an array is not aligned to its element type");
        return BPE_EINVAL;
    }
    int device = 0;
    bpe_status st = device_of({{"logits", logits, false}, {"u", u, false}, {"temperatures", how->temperatures, true},
                               {"top_ks", how->top_ks, true}, {"top_ps", how->top_ps, true},
                               {"min_ps", how->min_ps, true}, {"ids", ids, false}, {"logp", logp, true}}, &device);
    if (st != BPE_OK) return st;
    OnDevice on(device);
    bpek::Sampling par;
    par.temperature = how->temperature;
    par.top_p = how->top_p;
    par.min_p = how->min_p;
    par.top_k = how->top_k;
    par.temperatures = how->temperatures;
    par.top_ks = how->top_ks;
    par.top_ps = how->top_ps;
    par.min_ps = how->min_ps;
    with_type(type, [&](auto tag) {
        using T = decltype(tag);
        auto launch = [&](auto kernel, uint32_t tpb) {
            bpek::in_parts(rows, 1, bpek::groups_in_x(tpb), [&](size_t at, uint32_t, uint32_t groups) {
                bpek::Sampling here = par;
                if (here.temperatures) here.temperatures += at;
                if (here.top_ks) here.top_ks += at;
                if (here.top_ps) here.top_ps += at;
                if (here.min_ps) here.min_ps += at;
                hipLaunchKernelGGL(kernel, dim3(groups), dim3(tpb), 0, static_cast<hipStream_t>(stream),
                                   static_cast<const typename T::raw*>(logits) + at * stride, stride, uint32_t(vocab), u + at,
                                   here, ids + at, logp ? logp + at : logp);
            });
        };
        if (vocab <= 2048) launch(bpek::k_sample<T, 256, 4>, 256);
        else if (vocab <= 8192) launch(bpek::k_sample<T, 256, 16>, 256);
        else if (vocab <= 32768) launch(bpek::k_sample<T, 1024, 16>, 1024);
        else if (vocab <= 65536) launch(bpek::k_sample<T, 1024, 32>, 1024);
        else launch(bpek::k_sample<T, 1024, 0>, 1024);
    });
    HIP_TRY(hipGetLastError());
    return BPE_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- decoding

struct bpe_decoder {
    int device = 0;
    hipStream_t stream = nullptr;          // used when the caller passes none
    uint4* entry = nullptr;
    uint4* pool = nullptr;
    uint8_t* length = nullptr;
    uint32_t n = 0, max_len = 0;
    bpek::DecChunk* chunk = nullptr;       // the chunks' sums of the last call
    unsigned* left = nullptr;              // and how many of them have not ended
    bpek::DecResult* said = nullptr;       // pinned host memory, written by the kernels
    unsigned long long calls = 0;          // that tell their end
    // pooled buffers, kept until bpe_decoder_free
    uint32_t* tok_buf = nullptr;           // device copies of host arrays
    size_t tok_cap = 0;
    uint8_t* text_buf = nullptr;
    size_t text_cap = 0;
    int64_t* off_buf = nullptr;
    size_t off_cap = 0;
};

namespace {

template <typename T>
bpe_status room(T** p, size_t* cap, size_t need) {
    if (*cap >= need) return BPE_OK;
    if (*p) HIP_TRY(hipFree(*p));
    *p = nullptr;
    *cap = 0;
    const size_t n = need + need / 2;
    if (hipMalloc(reinterpret_cast<void**>(p), n * sizeof(T)) != hipSuccess) {
        (void)hipGetLastError();
        set_err("hipMalloc of %zu bytes failed", n * sizeof(T));
        return BPE_ENOMEM;
    }
    *cap = n;
    return BPE_OK;
}

constexpr uint64_t DECODER_MAX_STRING_BYTES = uint64_t(1) << 27;  // as for the trie

// The vocabulary's entries and its pool of long strings.
bpe_status build_entries(const std::vector<bpe_merge>& merges, std::vector<uint4>* entry, std::vector<uint8_t>* pool,
                         uint32_t* max_len) {
    const uint32_t nv = BPE_BASE_VOCAB + uint32_t(merges.size());
    std::vector<uint64_t> off(nv + size_t(1), 0);
    for (uint32_t i = 0; i < nv; ++i) {
        uint64_t len = 1;
        if (i >= BPE_BASE_VOCAB) {
            const bpe_merge& g = merges[i - BPE_BASE_VOCAB];
            if (g.left >= i || g.right >= i) {
                set_err("merge %u (%u, %u) names an id that does not exist before it (ids < %u)", i - BPE_BASE_VOCAB,
                        g.left, g.right, i);
                return BPE_EINVAL;
            }
            len = (off[g.left + 1] - off[g.left]) + (off[g.right + 1] - off[g.right]);
        }
        off[i + 1] = off[i] + len;
        if (off[i + 1] > DECODER_MAX_STRING_BYTES) {
            set_err("the vocabulary's strings exceed %llu bytes", (unsigned long long)DECODER_MAX_STRING_BYTES);
            return BPE_EINVAL;
        }
    }
    std::vector<uint8_t> text(off[nv]);
    entry->assign(nv, uint4{0, 0, 0, 0});
    for (uint32_t i = 0; i < nv; ++i) {
        uint8_t* p = &text[off[i]];
        const uint32_t len = uint32_t(off[i + 1] - off[i]);
        if (i < BPE_BASE_VOCAB) {
            *p = uint8_t(i);
        } else {
            const bpe_merge& g = merges[i - BPE_BASE_VOCAB];
            const size_t l = off[g.left + 1] - off[g.left];
            std::memcpy(p, &text[off[g.left]], l);
            std::memcpy(p + l, &text[off[g.right]], len - l);
        }
        *max_len = std::max(*max_len, len);
        uint4& e = (*entry)[i];
        if (len <= bpek::DC_INLINE) {
            std::memcpy(&e, p, len);
            e.w |= len << 24;
        } else {
            e.x = uint32_t(pool->size() / 16);
            e.y = len;
            e.w = bpek::DC_LONG << 24;
            pool->insert(pool->end(), p, p + len);
            pool->resize(align_up(pool->size(), 16), 0);
        }
    }
    return BPE_OK;
}

// Whether the call's last workgroup says, within the time that a short call
// takes, that all have ended. Reading its word sees the end sooner than a wait
// for the stream, which takes over if the stream has more to do.
bool ended(const bpek::DecResult* said, unsigned long long call) {
    const auto until = std::chrono::steady_clock::now() + std::chrono::microseconds(100);
    do {
        for (int i = 0; i < 64; ++i)
            if (__atomic_load_n(&said->ended, __ATOMIC_ACQUIRE) == call) return true;
    } while (std::chrono::steady_clock::now() < until);
    return false;
}

}  // namespace

extern "C" {

bpe_status bpe_decoder_build(const bpe_merge* merges, uint32_t n_merges, bpe_decoder** out) {
    g_err.clear();
    if (!out || (!merges && n_merges)) {
        set_err("out must be non-NULL, and merges non-NULL when n_merges > 0");
        return BPE_EINVAL;
    }
    *out = nullptr;
    if (n_merges > BPE_MAX_MERGES) {
        set_err("%u merges exceed the id space (%u merges)", n_merges, BPE_MAX_MERGES);
        return BPE_EIDSPACE;
    }
    bpe_decoder* d = new (std::nothrow) bpe_decoder();
    if (!d) {
        set_err("out of host memory");
        return BPE_ENOMEM;
    }
    auto fail = [&](bpe_status s) {
        bpe_decoder_free(d);
        return s;
    };
    std::vector<uint4> entry;
    std::vector<uint8_t> pool, length;
    try {
        std::vector<bpe_merge> hm(n_merges);
        bpe_status st = bpeh::copy_merges(merges, n_merges, hm.data());
        if (st == BPE_OK) st = build_entries(hm, &entry, &pool, &d->max_len);
        if (st != BPE_OK) {
            delete d;
            return st;
        }
        length.assign(align_up(entry.size(), 16), 0);
        for (size_t i = 0; i < entry.size(); ++i) length[i] = uint8_t(entry[i].w >> 24);
        d->n = uint32_t(entry.size());
        entry.push_back(uint4{0, 0, 0, 0});  // no token
    } catch (const std::bad_alloc&) {
        delete d;
        set_err("out of host memory");
        return BPE_ENOMEM;
    }
    if (hipGetDevice(&d->device) != hipSuccess || hipStreamCreate(&d->stream) != hipSuccess) {
        (void)hipGetLastError();
        set_err("cannot create a stream");
        return fail(BPE_EHIP);
    }
    if (hipMalloc(reinterpret_cast<void**>(&d->entry), entry.size() * sizeof(uint4)) != hipSuccess ||
        hipMalloc(reinterpret_cast<void**>(&d->pool), pool.size() + 16) != hipSuccess ||
        hipMalloc(reinterpret_cast<void**>(&d->length), length.size()) != hipSuccess ||
        hipMalloc(reinterpret_cast<void**>(&d->chunk), sizeof(bpek::DecChunk) * bpek::DC_CHUNKS) != hipSuccess ||
        hipMalloc(reinterpret_cast<void**>(&d->left), sizeof(unsigned)) != hipSuccess ||
        hipHostMalloc(reinterpret_cast<void**>(&d->said), sizeof(bpek::DecResult), hipHostMallocCoherent) != hipSuccess) {
        (void)hipGetLastError();
        set_err("hipMalloc failed");
        return fail(BPE_ENOMEM);
    }
    if (hipMemcpy(d->entry, entry.data(), entry.size() * sizeof(uint4), hipMemcpyHostToDevice) != hipSuccess ||
        hipMemcpy(d->length, length.data(), length.size(), hipMemcpyHostToDevice) != hipSuccess ||
        (!pool.empty() && hipMemcpy(d->pool, pool.data(), pool.size(), hipMemcpyHostToDevice) != hipSuccess)) {
        (void)hipGetLastError();
        set_err("uploading the vocabulary failed");
        return fail(BPE_EHIP);
    }
    *d->said = bpek::DecResult{0, ~0ull, 0};
    *out = d;
    return BPE_OK;
}

bpe_status bpe_decoder_info(const bpe_decoder* d, uint32_t* vocab, uint32_t* max_len) {
    g_err.clear();
    if (!d) {
        set_err("decoder must be non-NULL");
        return BPE_EINVAL;
    }
    if (vocab) *vocab = d->n;
    if (max_len) *max_len = d->max_len;
    return BPE_OK;
}

bpe_status bpe_decoder_decode(bpe_decoder* d, const uint32_t* tokens, size_t n, void* stream, uint8_t* bytes,
                              size_t bytes_cap, int64_t* offsets, size_t* n_bytes) {
    g_err.clear();
    if (!d || !n_bytes || (n && !tokens)) {
        set_err("decoder and n_bytes must be non-NULL, and tokens non-NULL when n > 0");
        return BPE_EINVAL;
    }
    if (n > BPE_MAX_BYTES) {
        set_err("n = %zu exceeds the limit of %llu tokens", n, (unsigned long long)BPE_MAX_BYTES);
        return BPE_EINVAL;
    }
    if (!aligned(tokens, 4) || !aligned(offsets, 8)) {
        set_err("an array is not aligned to its element type");
        return BPE_EINVAL;
    }
    *n_bytes = 0;
    if (n == 0 && !offsets) return BPE_OK;
    OnDevice on(d->device);
    hipStream_t s = stream ? static_cast<hipStream_t>(stream) : d->stream;
    const bpek::DecTable tab{d->entry, d->pool, d->length, d->n};
    bool tokens_host = false, bytes_host = false, offsets_host = false;
    bpe_status st = BPE_OK;
    if (n && (st = place_of("tokens", tokens, d->device, &tokens_host)) != BPE_OK) return st;
    if (bytes && (st = place_of("bytes", bytes, d->device, &bytes_host)) != BPE_OK) return st;
    if (offsets && (st = place_of("offsets", offsets, d->device, &offsets_host)) != BPE_OK) return st;
    // The second pass reads the tokens while it writes, and writes where the
    // first pass's lengths say: on one device none may share memory. (What
    // lies in host memory is copied on the way.)
    const void* given[3] = {tokens, bytes, offsets};
    const uint64_t size[3] = {n * sizeof(uint32_t), bytes_cap, (n + 1) * sizeof(int64_t)};
    const bool there[3] = {n && !tokens_host, bytes && !bytes_host, offsets && !offsets_host};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (there[i] && there[j] && bpek::share_bytes(given[i], size[i], given[j], size[j])) {
                set_err("tokens, bytes and offsets must not share memory");
                return BPE_EINVAL;
            }
    const uint32_t* src = tokens;
    if (tokens_host) {
        if ((st = room(&d->tok_buf, &d->tok_cap, n)) != BPE_OK) return st;
        HIP_TRY(hipMemcpyAsync(d->tok_buf, tokens, n * sizeof(uint32_t), hipMemcpyHostToDevice, s));
        src = d->tok_buf;
    }
    int64_t* off = offsets;
    if (offsets_host) {
        if ((st = room(&d->off_buf, &d->off_cap, n + 1)) != BPE_OK) return st;
        off = d->off_buf;
    }
    // One pass over the tokens, with the text to dst (cap bytes) or nowhere.
    auto decode = [&](uint8_t* dst, size_t cap, int64_t* places) -> bpe_status {
        if (n <= bpek::DC_TILE) {
            hipLaunchKernelGGL(bpek::k_dec_small, dim3(1), dim3(bpek::DC_TPB), 0, s, tab, src, uint32_t(n), dst,
                               uint64_t(cap), places, d->said, ++d->calls);
            HIP_TRY(hipGetLastError());
            if (ended(d->said, d->calls)) return BPE_OK;
        } else {
            // whole tiles in a chunk, the same number in each but the last
            const uint64_t tiles = (n + bpek::DC_TILE - 1) / bpek::DC_TILE;
            const uint64_t per = (tiles + bpek::DC_CHUNKS - 1) / bpek::DC_CHUNKS * bpek::DC_TILE;
            const uint32_t chunks = uint32_t((n + per - 1) / per);
            const bool tell = chunks <= bpek::DC_TELL;
            hipLaunchKernelGGL(bpek::k_dec_sum, dim3(chunks), dim3(bpek::DC_SUM_TPB), align_up(d->n, 16), s, tab, src,
                               uint64_t(n), per, d->chunk, d->left);
            hipLaunchKernelGGL(bpek::k_dec_copy, dim3(chunks), dim3(bpek::DC_TPB), 0, s, tab, src, uint64_t(n), per,
                               d->chunk, dst, uint64_t(cap), places, d->said, tell ? ++d->calls : 0,
                               d->left);
            HIP_TRY(hipGetLastError());
            if (tell && ended(d->said, d->calls)) return BPE_OK;
        }
        HIP_TRY(hipStreamSynchronize(s));
        return BPE_OK;
    };
    if ((st = decode(bytes_host ? nullptr : bytes, bytes_cap, off)) != BPE_OK) return st;
    if (d->said->bad != ~0ull) {
        set_err("token %llu names no id of the vocabulary (%u ids)", (unsigned long long)d->said->bad, d->n);
        return BPE_EINVAL;
    }
    const size_t total = size_t(d->said->total);
    *n_bytes = total;
    if (offsets_host) HIP_TRY(hipMemcpy(offsets, off, (n + 1) * sizeof(int64_t), hipMemcpyDeviceToHost));
    if (bytes && total > bytes_cap) {
        set_err("the text takes %zu bytes, bytes_cap is %zu", total, bytes_cap);
        return BPE_EINVAL;
    }
    if (bytes_host && total) {  // the text's length is known now: room for it, and once more
        if ((st = room(&d->text_buf, &d->text_cap, total)) != BPE_OK) return st;
        if ((st = decode(d->text_buf, total, nullptr)) != BPE_OK) return st;
        HIP_TRY(hipMemcpy(bytes, d->text_buf, total, hipMemcpyDeviceToHost));
    }
    return BPE_OK;
}

void bpe_decoder_free(bpe_decoder* d) {
    if (!d) return;
    OnDevice on(d->device);
    if (d->stream) (void)hipStreamSynchronize(d->stream);
    if (d->entry) (void)hipFree(d->entry);
    if (d->pool) (void)hipFree(d->pool);
    if (d->tok_buf) (void)hipFree(d->tok_buf);
    if (d->text_buf) (void)hipFree(d->text_buf);
    if (d->off_buf) (void)hipFree(d->off_buf);
    if (d->length) (void)hipFree(d->length);
    if (d->chunk) (void)hipFree(d->chunk);
    if (d->left) (void)hipFree(d->left);
    if (d->said) (void)hipHostFree(d->said);
    if (d->stream) (void)hipStreamDestroy(d->stream);
    delete d;
}

}  // extern "C"
