// Rotary positions: query and key rows rotated by their tokens' positions, on
// their own (pa_rope) or on the way into the paged cache (pa_rope_append_kv).
//
// A row is taken as pairs of elements, and pair f of a token is turned by the
// angle that the caller's table holds for the token's position and frequency f:
// a' = a cos - b sin, b' = b cos + a sin. With several position axes (time,
// height and width of images and video) each frequency takes the position of
// one axis. Elements from rotary_dim on are copied.
//
// Bound by memory for many tokens (every row is read and written once; a token's
// row of the table serves all its heads), by latency for a step's few.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <vector>

#include "pa_internal.h"
#include "ptx.cuh"
#include "quantise.cuh"

namespace {

constexpr int kBlock = 16;
constexpr int kThreads = 64;
constexpr int kMaxAxes = 4;

// what happens to the rotated keys and the values
enum Sink { kRowsOnly = 0, kCopy = 1, kInt8 = 2, kFp8 = 3, kInt4 = 4 };

struct RopeParams {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;   // elements a token
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    int8_t* k_zp;
    int8_t* v_zp;
    const int64_t* slots;
    int64_t num_slots;
    const float* cos_sin;
    const int32_t* positions;
    const uint8_t* freq_axis;
    unsigned int* err;
    int max_positions;
    int num_axes;
    int rotary_dim;
    float turn;              // 1, or -1: the other way
    uint32_t num_tokens;
    uint32_t num_heads, num_kv_heads;
    uint32_t rows;           // of a token: query, key and value heads
    uint32_t slices;         // warps of a token
};

template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&x)[8]) {
    uint4 out;
    uint32_t* w = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (std::is_same<T, __half>::value) {
            const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return out;
}

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& raw, float (&x)[8]) {
    const T* h = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = pa::to_f32<T>(h[e]);
}

// Pairs of elements turned by the cosines and sines of 8 consecutive frequencies. Products
// and sums are rounded one by one, as a plain form does it, so a code does not depend on
// which of the two computed it (mul.rn.f32x2 and add.rn.f32x2 do not give that: with them
// some results are those of a fused operation).
template <bool kInterleaved>
__device__ __forceinline__ void rotate(float (&x)[8], float (&y)[8], const float (&c)[8],
                                       const float (&s)[8]) {
#pragma unroll
    for (int f = 0; f < 8; ++f) {
        // interleaved: x holds pairs 0..3 and y 4..7; else x the first elements, y the second
        float& a = kInterleaved ? (f < 4 ? x[2 * (f % 4)] : y[2 * (f % 4)]) : x[f];
        float& b = kInterleaved ? (f < 4 ? x[2 * (f % 4) + 1] : y[2 * (f % 4) + 1]) : y[f];
        const float u = __fsub_rn(__fmul_rn(a, c[f]), __fmul_rn(b, s[f]));
        b = __fadd_rn(__fmul_rn(b, c[f]), __fmul_rn(a, s[f]));
        a = u;
    }
}

// 16 elements a thread of a row (chunks of 8: a and b), head_dim / 16 threads a row; a
// warp takes kUnroll times 32 / (head_dim / 16) rows of one token, so that a thread's
// cosines and sines, read once, turn kUnroll rows and all its rows are on their way at
// once (8191 tokens of 32 heads of 128 cold: 29.8 us, 34.9 with one row a thread). CTAs of
// two warps, for those that quantise are slower than those that rotate (6001 tokens of 64 + 8
// + 8 heads into a 4-bit cache and read back: 58.5 us, 79 us with 8 warps, 60.5 with 4). Which 8
// frequencies a thread has does not depend on how pairs lie: chunks f / 8
// and (f + rotary_dim / 2) / 8 hold them, or chunks f / 4 and f / 4 + 1.
template <int kSink, int D, typename T, bool kInterleaved, int kUnroll>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kPer = D / 16;            // threads a row
    constexpr int kRows = 32 / kPer;        // rows a warp has at once
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t t = warp / p.slices;
    if (t >= p.num_tokens) return;
    pa::grid_dependency_wait();
    const uint32_t first = (warp - t * p.slices) * (kRows * kUnroll) + lane / kPer;
    const int c = lane % kPer, half = p.rotary_dim / 2, pairs = half / 8;
    const bool turned = c < pairs;
    const int a = kInterleaved ? 2 * c : turned ? c : 2 * c;
    const int b = kInterleaved || !turned ? a + 1 : c + pairs;

    uint4 ra[kUnroll], rb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t r = first + u * kRows;
        if (r >= p.rows) continue;
        const T* src;
        if (r < p.num_heads)
            src = static_cast<const T*>(p.q) + (int64_t)t * p.q_stride + (int64_t)r * D;
        else if (kSink == kRowsOnly || r < p.num_heads + p.num_kv_heads)
            src = static_cast<const T*>(p.k) + (int64_t)t * p.k_stride +
                  (int64_t)(r - p.num_heads) * D;
        else
            src = static_cast<const T*>(p.v) + (int64_t)t * p.v_stride +
                  (int64_t)(r - p.num_heads - p.num_kv_heads) * D;
        ra[u] = *(reinterpret_cast<const uint4*>(src) + a);
        rb[u] = *(reinterpret_cast<const uint4*>(src) + b);
    }
    int64_t slot = -1;
    if constexpr (kSink != kRowsOnly) slot = __ldg(p.slots + t);

    // cosines and sines of frequencies 8 c .. 8 c + 7
    float cs[8], sn[8];
    bool bad = false;
    auto load8 = [&](int pos) {
        const float4* row =
            reinterpret_cast<const float4*>(p.cos_sin + (int64_t)pos * p.rotary_dim) + 2 * c;
        const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row + half / 4),
                     s1 = __ldg(row + half / 4 + 1);
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
        cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
        sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    };
    if (p.num_axes == 1) {
        const int pos = __ldg(p.positions + t);
        bad = (uint32_t)pos >= (uint32_t)p.max_positions;
        if (turned && !bad) load8(pos);
    } else {
        int pos[kMaxAxes];
#pragma unroll
        for (int i = 0; i < kMaxAxes; ++i) {
            pos[i] = i < p.num_axes ? __ldg(p.positions + (int64_t)i * p.num_tokens + t) : 0;
            bad |= (uint32_t)pos[i] >= (uint32_t)p.max_positions;
        }
        if (turned) {
            const uint2 axes = __ldg(reinterpret_cast<const uint2*>(p.freq_axis) + c);
            const uint32_t x0 = axes.x & 255u;
            if (axes.x == axes.y && axes.x == x0 * 0x01010101u) {   // 8 frequencies of one axis
                bad |= x0 >= (uint32_t)p.num_axes;
                if (!bad) load8(x0 == 0 ? pos[0] : x0 == 1 ? pos[1] : x0 == 2 ? pos[2] : pos[3]);
            } else {
#pragma unroll
                for (int f = 0; f < 8; ++f) {
                    const uint32_t x = (f < 4 ? axes.x : axes.y) >> (8 * (f & 3)) & 255u;
                    bad |= x >= (uint32_t)p.num_axes;
                    const int at = x == 0 ? pos[0] : x == 1 ? pos[1] : x == 2 ? pos[2] : pos[3];
                    if (!bad) {
                        const float* row = p.cos_sin + (int64_t)at * p.rotary_dim + 8 * c + f;
                        cs[f] = __ldg(row);
                        sn[f] = __ldg(row + half);
                    }
                }
            }
        }
    }
    // a position outside the table, or a frequency without an axis: the token is left out
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0 && p.err) atomicOr(p.err, pa::ERR_BAD_SLOT);
        return;
    }
#pragma unroll
    for (int f = 0; f < 8; ++f) sn[f] = turned ? sn[f] * p.turn : 0.f;
    if (slot >= p.num_slots) {
        if (lane == 0 && p.err) atomicOr(p.err, pa::ERR_BAD_SLOT);
        slot = -1;
    }

#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t r = first + u * kRows;
        const bool is_q = r < p.num_heads;
        const bool is_k = !is_q && (kSink == kRowsOnly || r < p.num_heads + p.num_kv_heads);
        const bool in = r < p.rows;
        float x[8], y[8];
        if (in) {
            unpack16<T>(ra[u], x);
            unpack16<T>(rb[u], y);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
        }
        if (turned && (is_q || is_k)) {
            rotate<kInterleaved>(x, y, cs, sn);
            // what is not turned keeps its bits
            ra[u] = pack16<T>(x);
            rb[u] = pack16<T>(y);
        }
        if (in && is_q) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) +
                                                  (int64_t)t * p.q_out_stride + (int64_t)r * D);
            dst[a] = ra[u];
            dst[b] = rb[u];
        }
        const uint32_t g = is_k ? r - p.num_heads : r - p.num_heads - p.num_kv_heads;
        if (in && is_k && p.k_out) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.k_out) +
                                                  (int64_t)t * p.k_out_stride + (int64_t)g * D);
            dst[a] = ra[u];
            dst[b] = rb[u];
        }
        if constexpr (kSink != kRowsOnly) {
            // the shuffles below are the whole warp's: a warp of query rows alone leaves here
            if (slot < 0 || !__any_sync(0xffffffffu, in && !is_q)) continue;
            const bool put = in && !is_q;
            const int64_t row =
                ((slot / kBlock) * p.num_kv_heads + g) * kBlock + slot % kBlock;
            void* const cache = is_k ? p.k_cache : p.v_cache;
            if constexpr (kSink == kCopy) {
                if (put) {
                    uint4* dst = static_cast<uint4*>(cache) + row * (D / 8);
                    dst[a] = ra[u];
                    dst[b] = rb[u];
                }
            } else if constexpr (kSink == kFp8) {
                if (put) {
                    const float scale = __ldg((is_k ? p.k_scale : p.v_scale) + g);
                    uint2* dst = static_cast<uint2*>(cache) + row * (D / 8);
                    auto codes = [&](const float (&z)[8]) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 8; e += 2)
                            w[e / 2] = __nv_cvt_float2_to_fp8x2(
                                make_float2(__fdiv_rn(z[e], scale), __fdiv_rn(z[e + 1], scale)),
                                __NV_SATFINITE, __NV_E4M3);
                        return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
                    };
                    dst[a] = codes(x);
                    dst[b] = codes(y);
                }
            } else {
                // the range of what shares a scale: the row, or each 64 elements of it
                constexpr int kGroups = kSink == kInt4 ? D / PA_INT4_GROUP : 1;
                const int ga = kGroups > 1 ? a >> 3 : 0, gb = kGroups > 1 ? b >> 3 : 0;
                float mn[kGroups], mx[kGroups];
                float xn = 0.f, xx = 0.f, yn = 0.f, yx = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xn = fminf(xn, x[e]), xx = fmaxf(xx, x[e]);
                    yn = fminf(yn, y[e]), yx = fmaxf(yx, y[e]);
                }
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    mn[j] = fminf(ga == j ? xn : 0.f, gb == j ? yn : 0.f);
                    mx[j] = fmaxf(ga == j ? xx : 0.f, gb == j ? yx : 0.f);
#pragma unroll
                    for (int o = kPer / 2; o > 0; o >>= 1) {
                        mn[j] = fminf(mn[j], __shfl_xor_sync(0xffffffffu, mn[j], o));
                        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
                    }
                }
                if (put) {
                    using Quant = pa::Quantiser<kSink == kInt4 ? 15 : 255, kSink == kInt4 ? 0 : -128>;
                    float* const scales = (is_k ? p.k_scale : p.v_scale) + row * kGroups;
                    int8_t* const zps = (is_k ? p.k_zp : p.v_zp) + row * kGroups;
                    const Quant qa(ga ? mn[kGroups - 1] : mn[0], ga ? mx[kGroups - 1] : mx[0]);
                    if constexpr (kGroups == 1) {
                        if constexpr (kSink == kInt4) {
                            uint32_t* dst = static_cast<uint32_t*>(cache) + row * (D / 8);
                            dst[a] = qa.pack4(x);
                            dst[b] = qa.pack4(y);
                        } else {
                            uint2* dst = static_cast<uint2*>(cache) + row * (D / 8);
                            dst[a] = qa.pack8(x);
                            dst[b] = qa.pack8(y);
                        }
                        if (c == 0) {
                            scales[0] = qa.scale;
                            zps[0] = (int8_t)qa.zp;
                        }
                    } else {
                        const Quant qb(gb ? mn[1] : mn[0], gb ? mx[1] : mx[0]);
                        uint32_t* dst = static_cast<uint32_t*>(cache) + row * (D / 8);
                        dst[a] = qa.pack4(x);
                        dst[b] = qb.pack4(y);
                        // chunk 0 is the first thread's; chunk 8 starts the second group
                        if (a == 0 || a == 8) {
                            scales[ga] = qa.scale;
                            zps[ga] = (int8_t)qa.zp;
                        }
                        if (b == 8) {
                            scales[1] = qb.scale;
                            zps[1] = (int8_t)qb.zp;
                        }
                    }
                }
            }
        }
    }
}

template <int kSink, int D, typename T, bool kInterleaved, int kUnroll>
pa_status launch_as(RopeParams& p, cudaStream_t st) {
    constexpr uint32_t kAtOnce = 32 / (D / 16) * kUnroll;
    p.slices = (p.rows + kAtOnce - 1) / kAtOnce;
    const int64_t warps = (int64_t)p.num_tokens * p.slices;
    const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (warps > 0x7fffffff) return pa::fail(PA_ERR_UNSUPPORTED, "too many rows for one launch");
    return pa::cuda_status(
        pa::launch_pdl(rope_kernel<kSink, D, T, kInterleaved, kUnroll>, dim3((unsigned)grid),
                       dim3(kThreads), 0, st, p),
        "rope launch");
}

template <int kSink, int D, typename T>
pa_status launch_rows(RopeParams& p, bool interleaved, cudaStream_t st) {
    return interleaved ? launch_as<kSink, D, T, true, 4>(p, st)
                       : launch_as<kSink, D, T, false, 4>(p, st);
}

template <int kSink>
pa_status launch_rope(RopeParams& p, pa_dtype dtype, int head_dim, bool interleaved,
                      cudaStream_t st) {
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_rows<kSink, 128, __nv_bfloat16>(p, interleaved, st)
                               : launch_rows<kSink, 64, __nv_bfloat16>(p, interleaved, st);
    return head_dim == 128 ? launch_rows<kSink, 128, __half>(p, interleaved, st)
                           : launch_rows<kSink, 64, __half>(p, interleaved, st);
}

// rows of `heads` heads a token, `stride` elements from one token's to the next's
pa_status check_rows(const char* name, const void* rows, int64_t stride, int32_t heads,
                     int32_t head_dim) {
    if ((uintptr_t)rows % 16) return pa::fail(PA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (stride < (int64_t)heads * head_dim || stride % 8)
        return pa::fail(PA_ERR_INVALID_ARG,
                        "%s_stride %lld is not a multiple of 8 of at least %lld elements", name,
                        (long long)stride, (long long)heads * head_dim);
    return PA_OK;
}

// What both calls check of their rows and of the rotation.
pa_status check_rope(const void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
                     int32_t num_heads, pa_dtype dtype, const float* cos_sin,
                     int32_t max_positions, int32_t rotary_dim, const int32_t* positions,
                     int32_t num_axes, const uint8_t* freq_axis, int32_t num_tokens,
                     int32_t num_kv_heads, int32_t head_dim) {
    using pa::fail;
    if (dtype != PA_F16 && dtype != PA_BF16)
        return fail(PA_ERR_UNSUPPORTED, "dtype %d (F16 or BF16)", (int)dtype);
    if (head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d (64 or 128 supported)", head_dim);
    if (num_heads < 0 || num_kv_heads < 0 || num_heads > 65535 || num_kv_heads > 65535)
        return fail(PA_ERR_INVALID_ARG, "num_heads %d, num_kv_heads %d", num_heads, num_kv_heads);
    if (!cos_sin || !positions) return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    if (rotary_dim <= 0 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(PA_ERR_UNSUPPORTED, "rotary_dim %d (a multiple of 16 up to head_dim)",
                    rotary_dim);
    if (max_positions <= 0) return fail(PA_ERR_INVALID_ARG, "max_positions %d", max_positions);
    if (num_axes < 1 || num_axes > kMaxAxes)
        return fail(PA_ERR_UNSUPPORTED, "num_axes %d (1 to %d)", num_axes, kMaxAxes);
    if (num_axes > 1 && !freq_axis)
        return fail(PA_ERR_INVALID_ARG, "%d axes need freq_axis", num_axes);
    if (num_axes > 1 && (uintptr_t)freq_axis % 8)
        return fail(PA_ERR_INVALID_ARG, "freq_axis must be 8-byte aligned");
    if ((uintptr_t)cos_sin % 16) return fail(PA_ERR_INVALID_ARG, "cos_sin must be 16-byte aligned");
    if (num_heads > 0) {
        if (!q || !q_out) return fail(PA_ERR_INVALID_ARG, "NULL pointer");
        if (pa_status s = check_rows("q", q, q_stride, num_heads, head_dim)) return s;
        if (pa_status s = check_rows("q_out", q_out, q_out_stride, num_heads, head_dim)) return s;
        if (q == q_out && q_stride != q_out_stride)
            return fail(PA_ERR_INVALID_ARG, "q rotated in place needs q_out_stride %lld",
                        (long long)q_stride);
    }
    return PA_OK;
}

RopeParams rope_params(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
                       int32_t num_heads, void* k_out, int64_t k_out_stride, const void* k,
                       int64_t k_stride, int32_t num_kv_heads, const float* cos_sin,
                       int32_t max_positions, int32_t rotary_dim, const int32_t* positions,
                       int32_t num_axes, const uint8_t* freq_axis, int32_t num_tokens) {
    RopeParams p{};
    p.q = q, p.q_stride = q_stride, p.q_out = q_out, p.q_out_stride = q_out_stride;
    p.k = k, p.k_stride = k_stride, p.k_out = k_out, p.k_out_stride = k_out_stride;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.freq_axis = freq_axis;
    p.err = pa::device_error_word();
    p.max_positions = max_positions;
    p.num_axes = num_axes;
    p.rotary_dim = rotary_dim;
    p.turn = 1.f;
    p.num_tokens = (uint32_t)num_tokens;
    p.num_heads = (uint32_t)num_heads;
    p.num_kv_heads = (uint32_t)num_kv_heads;
    return p;
}

}  // namespace

extern "C" pa_status pa_rope(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride,
                             int32_t num_heads, void* k_out, int64_t k_out_stride, const void* k,
                             int64_t k_stride, int32_t num_kv_heads, pa_dtype dtype,
                             const float* cos_sin, int32_t max_positions, int32_t rotary_dim,
                             int32_t interleaved, const int32_t* positions, int32_t num_axes,
                             const uint8_t* freq_axis, int32_t inverse, int32_t num_tokens,
                             int32_t head_dim, void* stream) {
    using pa::fail;
    if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (num_tokens == 0) return PA_OK;
    if (pa_status s = check_rope(q_out, q_out_stride, q, q_stride, num_heads, dtype, cos_sin,
                                 max_positions, rotary_dim, positions, num_axes, freq_axis,
                                 num_tokens, num_kv_heads, head_dim))
        return s;
    if (num_heads + num_kv_heads == 0) return PA_OK;
    if (num_kv_heads > 0) {
        if (!k || !k_out) return fail(PA_ERR_INVALID_ARG, "NULL pointer");
        if (pa_status s = check_rows("k", k, k_stride, num_kv_heads, head_dim)) return s;
        if (pa_status s = check_rows("k_out", k_out, k_out_stride, num_kv_heads, head_dim)) return s;
        if (k == k_out && k_stride != k_out_stride)
            return fail(PA_ERR_INVALID_ARG, "k rotated in place needs k_out_stride %lld",
                        (long long)k_stride);
    }
    cudaStream_t st = (cudaStream_t)stream;
    if (pa::validate_enabled())
        if (pa_status s = pa::validate_positions(positions, num_axes, num_tokens, max_positions,
                                                 freq_axis, rotary_dim, st))
            return s;
    RopeParams p = rope_params(q_out, q_out_stride, q, q_stride, num_heads, k_out, k_out_stride, k,
                               k_stride, num_kv_heads, cos_sin, max_positions, rotary_dim,
                               positions, num_axes, freq_axis, num_tokens);
    p.rows = p.num_heads + p.num_kv_heads;
    p.turn = inverse ? -1.f : 1.f;
    return launch_rope<kRowsOnly>(p, dtype, head_dim, interleaved != 0, st);
}

extern "C" pa_status pa_rope_append_kv(
    void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, int32_t num_heads,
    void* key_out, int64_t key_out_stride, const void* key, int64_t key_stride, const void* value,
    int64_t value_stride, pa_dtype src_dtype, void* k_cache, void* v_cache, pa_dtype kv_dtype,
    float* k_scale, float* v_scale, int8_t* k_zp, int8_t* v_zp, const int64_t* slot_mapping,
    const float* cos_sin, int32_t max_positions, int32_t rotary_dim, int32_t interleaved,
    const int32_t* positions, int32_t num_axes, const uint8_t* freq_axis, int32_t num_tokens,
    int32_t num_blocks, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, void* stream) {
    using pa::fail;
    if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    if (pa_status s = pa::check_cache_args(k_cache, v_cache, kv_dtype, k_scale, v_scale, k_zp,
                                           v_zp, num_kv_heads, head_dim, block_size, num_blocks))
        return s;
    if (pa_status s = check_rope(q_out, q_out_stride, q, q_stride, num_heads, src_dtype, cos_sin,
                                 max_positions, rotary_dim, positions, num_axes, freq_axis,
                                 num_tokens, num_kv_heads, head_dim))
        return s;
    if ((kv_dtype == PA_F16 || kv_dtype == PA_BF16) && kv_dtype != src_dtype)
        return fail(PA_ERR_UNSUPPORTED, "a %s cache takes %s rows only",
                    kv_dtype == PA_F16 ? "F16" : "BF16", kv_dtype == PA_F16 ? "F16" : "BF16");
    if (pa_status s = check_rows("key", key, key_stride, num_kv_heads, head_dim)) return s;
    if (pa_status s = check_rows("value", value, value_stride, num_kv_heads, head_dim)) return s;
    if (key_out) {
        if (pa_status s = check_rows("key_out", key_out, key_out_stride, num_kv_heads, head_dim))
            return s;
        if (key == key_out && key_stride != key_out_stride)
            return fail(PA_ERR_INVALID_ARG, "key rotated in place needs key_out_stride %lld",
                        (long long)key_stride);
    }
    cudaStream_t st = (cudaStream_t)stream;
    if (pa::validate_enabled()) {
        if (pa_status s = pa::validate_slots(slot_mapping, num_tokens, num_blocks, st)) return s;
        if (pa_status s = pa::validate_positions(positions, num_axes, num_tokens, max_positions,
                                                 freq_axis, rotary_dim, st))
            return s;
    }
    RopeParams p = rope_params(q_out, q_out_stride, q, q_stride, num_heads, key_out,
                               key_out_stride, key, key_stride, num_kv_heads, cos_sin,
                               max_positions, rotary_dim, positions, num_axes, freq_axis,
                               num_tokens);
    p.v = value, p.v_stride = value_stride;
    p.k_cache = k_cache, p.v_cache = v_cache;
    p.k_scale = k_scale, p.v_scale = v_scale, p.k_zp = k_zp, p.v_zp = v_zp;
    p.slots = slot_mapping;
    p.num_slots = (int64_t)num_blocks * block_size;
    p.rows = p.num_heads + 2 * p.num_kv_heads;
    const bool il = interleaved != 0;
    switch (kv_dtype) {
        case PA_INT8: return launch_rope<kInt8>(p, src_dtype, head_dim, il, st);
        case PA_FP8_E4M3: return launch_rope<kFp8>(p, src_dtype, head_dim, il, st);
        case PA_INT4: return launch_rope<kInt4>(p, src_dtype, head_dim, il, st);
        default: return launch_rope<kCopy>(p, src_dtype, head_dim, il, st);
    }
}
