// KV-cache writes: append through a slot mapping (F16/BF16 copy, INT8, INT4
// or FP8 quantisation) and copy-on-write block copies; the read side of the
// same mapping, cached rows back as 16- or 32-bit rows.
//
// Append restates the decode workflow of "cs336 lecture 10" (KV Cache:
// append the new K, V to the cache) and the block table of "KV Cache ...
// PagedAttention" §七 (slot = physical block * 16 + offset). The INT8 path
// restates the same lecture's Quantization formula x_q = round(x/scale) +
// zero_point with one (scale, zero point) per (token, kv head) row, as
// "LLM推理优化深度实战" §5.2 asks (per head, not global). Block copies restate
// §2.1 of that page (copy a shared block only when it is modified).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_internal.h"
#include "ptx.cuh"

namespace {

constexpr int kBlock = 16;

// One thread per 16-byte vector of a (token, kv head) row, K and V together.
__global__ void append_kv16_kernel(const uint4* __restrict__ key, const uint4* __restrict__ value,
                                   uint4* __restrict__ k_cache, uint4* __restrict__ v_cache,
                                   const int64_t* __restrict__ slots, int num_tokens,
                                   int num_kv_heads, int vec_per_row, int64_t num_slots,
                                   unsigned int* err) {
    const int64_t per_token = (int64_t)num_kv_heads * vec_per_row;
    const int64_t total = (int64_t)num_tokens * per_token;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / per_token;
        const int64_t rem = i - t * per_token;
        const int64_t slot = __ldg(slots + t);
        if (slot < 0) continue;
        if (slot >= num_slots) {
            if (err) atomicOr(err, pa::ERR_BAD_SLOT);
            continue;
        }
        const int64_t blk = slot / kBlock, off = slot % kBlock;
        const int64_t g = rem / vec_per_row, v = rem - g * vec_per_row;
        const int64_t dst = ((blk * num_kv_heads + g) * kBlock + off) * vec_per_row + v;
        k_cache[dst] = __ldg(key + i);
        v_cache[dst] = __ldg(value + i);
    }
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
    return __bfloat162float(x);
}

// One warp per (token, kv head, K-or-V) row. EPL elements per lane
// (head_dim = 32 * EPL). Arithmetic is IEEE fp32: correctly rounded
// division (__fdiv_rn), round-half-to-even (rintf), no contraction.
template <typename T, int EPL>
__global__ void append_kv_int8_kernel(const T* __restrict__ key, const T* __restrict__ value,
                                      int8_t* __restrict__ k_cache, int8_t* __restrict__ v_cache,
                                      float* __restrict__ k_scale, float* __restrict__ v_scale,
                                      int8_t* __restrict__ k_zp, int8_t* __restrict__ v_zp,
                                      const int64_t* __restrict__ slots, int num_tokens,
                                      int num_kv_heads, int64_t num_slots, unsigned int* err) {
    constexpr int D = 32 * EPL;
    const int lane = threadIdx.x & 31;
    const int64_t warp = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
    const int64_t rows = (int64_t)num_tokens * num_kv_heads * 2;
    if (warp >= rows) return;
    const int which = (int)(warp & 1);          // 0 = K, 1 = V
    const int64_t tg = warp >> 1;               // token * num_kv_heads + g
    const int64_t t = tg / num_kv_heads;
    const int64_t g = tg - t * num_kv_heads;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (lane == 0 && err) atomicOr(err, pa::ERR_BAD_SLOT);
        return;
    }
    const T* src = (which ? value : key) + tg * D + lane * EPL;
    float x[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) x[e] = to_f32<T>(src[e]);
    // range widened to contain 0, as the oracle does
    float mn = 0.0f, mx = 0.0f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        mn = x[e] < mn ? x[e] : mn;
        mx = x[e] > mx ? x[e] : mx;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, mn, o);
        const float b = __shfl_xor_sync(0xffffffffu, mx, o);
        mn = a < mn ? a : mn;
        mx = b > mx ? b : mx;
    }
    float scale = __fdiv_rn(__fsub_rn(mx, mn), 255.0f);
    if (scale == 0.0f) scale = 1.0f;
    const float zf = __fsub_rn(-128.0f, rintf(__fdiv_rn(mn, scale)));
    int zp = (int)zf;
    zp = zp < -128 ? -128 : (zp > 127 ? 127 : zp);
    const int64_t blk = slot / kBlock, off = slot % kBlock;
    const int64_t row = (blk * num_kv_heads + g) * kBlock + off;
    uint32_t packed[(EPL + 3) / 4] = {};
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        int c = (int)rintf(__fdiv_rn(x[e], scale)) + zp;
        c = c < -128 ? -128 : (c > 127 ? 127 : c);
        packed[e / 4] |= (uint32_t)(uint8_t)(int8_t)c << (8 * (e % 4));
    }
    int8_t* dst = (which ? v_cache : k_cache) + row * D + lane * EPL;
    if constexpr (EPL == 4) {
        *reinterpret_cast<uint32_t*>(dst) = packed[0];
    } else {
        static_assert(EPL == 2, "head_dim 64 or 128");
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)packed[0];
    }
    if (lane == 0) {
        (which ? v_scale : k_scale)[row] = scale;
        (which ? v_zp : k_zp)[row] = (int8_t)zp;
    }
}

// FP8 E4M3 append ("LLM推理优化深度实战" §5.2: FP8 KV cache, one scale per
// KV head): one thread per 16 consecutive elements of a (token, kv head) row,
// K and V together. code = E4M3(x / scale[head]): the IEEE fp32 quotient
// (__fdiv_rn), converted with round-to-nearest-even and saturation at +-448.
template <typename T>
__global__ void append_kv_fp8_kernel(const T* __restrict__ key, const T* __restrict__ value,
                                     uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache,
                                     const float* __restrict__ k_scale,
                                     const float* __restrict__ v_scale,
                                     const int64_t* __restrict__ slots, int num_tokens,
                                     int num_kv_heads, int head_dim, int64_t num_slots,
                                     unsigned int* err) {
    const int per_row = head_dim / 16;
    const int64_t per_token = (int64_t)num_kv_heads * per_row;
    const int64_t total = (int64_t)num_tokens * per_token;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / per_token;
        const int64_t rem = i - t * per_token;
        const int64_t slot = __ldg(slots + t);
        if (slot < 0) continue;
        if (slot >= num_slots) {
            if (err) atomicOr(err, pa::ERR_BAD_SLOT);
            continue;
        }
        const int g = (int)(rem / per_row), c = (int)(rem - (int64_t)g * per_row);
        const int64_t blk = slot / kBlock, off = slot % kBlock;
        const int64_t src = (t * num_kv_heads + g) * head_dim + c * 16;
        const int64_t dst = ((blk * num_kv_heads + g) * kBlock + off) * head_dim + c * 16;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const T* in = (which ? value : key) + src;
            const float s = __ldg((which ? v_scale : k_scale) + g);
            const uint4 raw0 = __ldg(reinterpret_cast<const uint4*>(in));
            const uint4 raw1 = __ldg(reinterpret_cast<const uint4*>(in) + 1);
            const T* h0 = reinterpret_cast<const T*>(&raw0);
            const T* h1 = reinterpret_cast<const T*>(&raw1);
            uint32_t out[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t word = 0;
#pragma unroll
                for (int pr = 0; pr < 2; ++pr) {
                    const int e = 4 * w + 2 * pr;
                    const T* h = e < 8 ? h0 + e : h1 + (e - 8);
                    const float2 y = make_float2(__fdiv_rn(to_f32<T>(h[0]), s),
                                                 __fdiv_rn(to_f32<T>(h[1]), s));
                    const __nv_fp8x2_storage_t q =
                        __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                    word |= (uint32_t)q << (16 * pr);
                }
                out[w] = word;
            }
            *reinterpret_cast<uint4*>((which ? v_cache : k_cache) + dst) =
                make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
}

// Two fp32 numbers and the two-wide arithmetic on them (each operation rounds
// as its scalar form does).
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float lo, float hi) {
        asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    }
    __device__ __forceinline__ float lo() const {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
        return a;
    }
    __device__ __forceinline__ float hi() const {
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
        return b;
    }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// INT4 append: the formula of the INT8 path with 16 unsigned codes and one
// (scale, zero point) per 64 elements. 8 threads a row; a thread holds 8
// consecutive elements of every group of the K row and of the same V row (16-byte
// loads, 4-byte code stores), and a group's range is reduced over the 8 with
// shuffles. 2 bytes in and 0.58 out an element: bound by instruction issue before
// memory, so indexes are 32 bits wide (their 64-bit divisions alone cost a third of
// the kernel), a thread's index arithmetic serves every group of a row, and
// quotients come from one reciprocal a group; the rows are asked for before the
// slot is known. 16384 tokens of 8 heads of 128 elements, with the gather that reads
// them back: 32.8 us, 37.3 us with a thread a group, 59 us with a division an element.
template <typename T, int D>
__global__ void __launch_bounds__(256) append_kv_int4_kernel(
    const T* __restrict__ key, const T* __restrict__ value, uint8_t* __restrict__ k_cache,
    uint8_t* __restrict__ v_cache, float* __restrict__ k_scale, float* __restrict__ v_scale,
    int8_t* __restrict__ k_zp, int8_t* __restrict__ v_zp, const int64_t* __restrict__ slots,
    uint32_t total, uint32_t num_kv_heads, int64_t num_slots, unsigned int* err) {
    constexpr int kGroups = D / PA_INT4_GROUP;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    // total is a multiple of 8: the 8 threads of a row are all in range or all out of it
    pa::grid_dependency_wait();
    if (i >= total) return;
    const unsigned int peers = 0xffu << (threadIdx.x & 24);
    const uint32_t tg = i / 8, c = i % 8;
    const int64_t src = (int64_t)tg * (8 * kGroups) + c;
    uint4 raw[2][kGroups];
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        raw[0][j] = __ldcs(reinterpret_cast<const uint4*>(key) + src + 8 * j);
        raw[1][j] = __ldcs(reinterpret_cast<const uint4*>(value) + src + 8 * j);
    }
    const uint32_t t = tg / num_kv_heads, g = tg - t * num_kv_heads;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (c == 0 && err) atomicOr(err, pa::ERR_BAD_SLOT);
        return;
    }
    const int64_t row = ((slot / kBlock) * num_kv_heads + g) * kBlock + slot % kBlock;
#pragma unroll
    for (int w = 0; w < 2 * kGroups; ++w) {
        const int which = w / kGroups, j = w % kGroups;
        const T* h = reinterpret_cast<const T*>(&raw[which][j]);
        float x[8], mn = 0.0f, mx = 0.0f;   // the range is widened to contain 0
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = to_f32<T>(h[e]);
            mn = fminf(mn, x[e]);
            mx = fmaxf(mx, x[e]);
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            mn = fminf(mn, __shfl_xor_sync(peers, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(peers, mx, o));
        }
        const float range = __fsub_rn(mx, mn);
        float scale;
        uint32_t word;
        int zp;
        if (range > 1e-28f && range < 1e30f) {
            // Correctly rounded quotients by Markstein's theorem: with the correctly rounded
            // reciprocal y of b, q = a y and r = a - b q (exact in one fused operation),
            // q + r y is the rounded a / b. Then, adding 1.5 * 2^23 rounds to an integer in
            // the low bits, and the codes are put together from those bits as they are: the
            // excess of each over its code is the same number.
            constexpr float kFifteenth = 1.0f / 15.0f, kRound = 12582912.0f;
            const float s0 = __fmul_rn(range, kFifteenth);
            scale = __fmaf_rn(__fmaf_rn(-s0, 15.0f, range), kFifteenth, s0);
            const float inv = __frcp_rn(scale);
            const float z0 = __fmul_rn(mn, inv);
            const float z1 = __fmaf_rn(__fmaf_rn(-z0, scale, mn), inv, z0);
            const float zr = __fadd_rn(z1, kRound);
            zp = min(15, __float_as_int(kRound) - __float_as_int(zr));
            const float top = __int_as_float(__float_as_int(kRound) + 15 - zp);
            // no code is below 0: rounding keeps the order, and the zero point is -rint(mn / scale)
            word = 0;
#pragma unroll
            for (int e = 6; e >= 0; e -= 2) {
                const F2 v(x[e], x[e + 1]), q = v * F2(inv, inv);
                const F2 r = fma(q, F2(-scale, -scale), v);
                const F2 y = fma(r, F2(inv, inv), q) + F2(kRound, kRound);
                word = word * 16u + __float_as_uint(fminf(y.hi(), top));
                word = word * 16u + __float_as_uint(fminf(y.lo(), top));
            }
            word -= (uint32_t)(__float_as_int(kRound) - zp) * 0x11111111u;
        } else {                            // range 0, or too near the ends of fp32
            scale = __fdiv_rn(range, 15.0f);
            if (scale == 0.0f) scale = 1.0f;
            zp = (int)-rintf(__fdiv_rn(mn, scale));
            zp = zp < 0 ? 0 : min(15, zp);
            word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int q = (int)rintf(__fdiv_rn(x[e], scale)) + zp;
                word |= (uint32_t)(q < 0 ? 0 : min(15, q)) << (4 * e);
            }
        }
        reinterpret_cast<uint32_t*>(which ? v_cache : k_cache)[(row * kGroups + j) * 8 + c] = word;
        if (c == 0) {
            (which ? v_scale : k_scale)[row * kGroups + j] = scale;
            (which ? v_zp : k_zp)[row * kGroups + j] = (int8_t)zp;
        }
    }
}

// 8 consecutive cached elements (elements 8c .. 8c + 7 of cached row `row`) as
// stored, with what their codes are scaled by.
template <int KV, int D>
struct Cached8 {
    uint4 raw;
    float scale;
    int zp;
    __device__ __forceinline__ void load(const void* cache, const float* scales,
                                         const int8_t* zps, int64_t row, uint32_t g, uint32_t c) {
        constexpr int kPerRow = D / 8;
        if constexpr (KV == PA_F16 || KV == PA_BF16) {
            raw = __ldg(static_cast<const uint4*>(cache) + row * kPerRow + c);
        } else if constexpr (KV == PA_INT4) {
            raw.x = __ldg(static_cast<const uint32_t*>(cache) + row * kPerRow + c);
            scale = __ldg(scales + row * (D / PA_INT4_GROUP) + c / 8);
            zp = __ldg(zps + row * (D / PA_INT4_GROUP) + c / 8);
        } else {
            const uint2 u = __ldg(static_cast<const uint2*>(cache) + row * kPerRow + c);
            raw.x = u.x, raw.y = u.y;
            scale = __ldg(scales + (KV == PA_INT8 ? row : (int64_t)g));
            if constexpr (KV == PA_INT8) zp = __ldg(zps + row);
        }
    }
    // a code's value is one fp32 product
    __device__ __forceinline__ float value(int e) const {
        if constexpr (KV == PA_F16)
            return __half2float(reinterpret_cast<const __half*>(&raw)[e]);
        else if constexpr (KV == PA_BF16)
            return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(&raw)[e]);
        else if constexpr (KV == PA_INT4)   // 2^23 + code as its bits, less 2^23 + zero point
            return __fmul_rn(__fsub_rn(__uint_as_float((raw.x >> (4 * e) & 15u) | 0x4b000000u),
                                       8388608.0f + (float)zp),
                             scale);
        else if constexpr (KV == PA_INT8)
            return __fmul_rn((float)((int)reinterpret_cast<const int8_t*>(&raw)[e] - zp), scale);
        else
            return __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(
                                 reinterpret_cast<const uint8_t*>(&raw)[e], __NV_E4M3))),
                             scale);
    }
};

template <int KV, int D>
__device__ __forceinline__ void store8(float* dst, const Cached8<KV, D>& x) {
    __stcs(reinterpret_cast<float4*>(dst),
           make_float4(x.value(0), x.value(1), x.value(2), x.value(3)));
    __stcs(reinterpret_cast<float4*>(dst) + 1,
           make_float4(x.value(4), x.value(5), x.value(6), x.value(7)));
}
template <int KV, int D, typename T>
__device__ __forceinline__ void store8(T* dst, const Cached8<KV, D>& x) {
    constexpr bool half = std::is_same<T, __half>::value;
    uint4 out = x.raw;   // a 16-bit cache read as its own type
    if constexpr (KV != (half ? PA_F16 : PA_BF16)) {
        T* h = reinterpret_cast<T*>(&out);
        if constexpr (KV == PA_INT4) {   // value(), two at a time
            const float zero = -(8388608.0f + (float)x.zp);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const F2 code(__uint_as_float((x.raw.x >> (4 * e) & 15u) | 0x4b000000u),
                              __uint_as_float((x.raw.x >> (4 * e + 4) & 15u) | 0x4b000000u));
                const F2 v = (code + F2(zero, zero)) * F2(x.scale, x.scale);
                if constexpr (half)
                    *reinterpret_cast<__half2*>(h + e) = __floats2half2_rn(v.lo(), v.hi());
                else
                    *reinterpret_cast<__nv_bfloat162*>(h + e) = __floats2bfloat162_rn(v.lo(), v.hi());
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (half) h[e] = __float2half_rn(x.value(e));
                else h[e] = __float2bfloat16_rn(x.value(e));
            }
        }
    }
    __stcs(reinterpret_cast<uint4*>(dst), out);
}

// Cached rows read back through a slot mapping: the inverse of append, each
// row at the values the cache holds. 8 threads a row; a thread has 8 elements of
// every 64 of the K row and of the same V row. The streaming loads and stores here
// and in the append are worth 3 us of 36. Bound by memory: the cache's bytes in, the rows out.
template <int KV, int D, typename T>
__global__ void __launch_bounds__(256) gather_kv_kernel(
    T* __restrict__ key, T* __restrict__ value, const void* __restrict__ k_cache,
    const void* __restrict__ v_cache, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, const int8_t* __restrict__ k_zp,
    const int8_t* __restrict__ v_zp, const int64_t* __restrict__ slots, uint32_t total,
    uint32_t num_kv_heads, int64_t num_slots, unsigned int* err) {
    constexpr int kParts = D / 64;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;
    pa::grid_dependency_wait();
    if (i >= total) return;
    const uint32_t tg = i / 8, c = i % 8;
    const uint32_t t = tg / num_kv_heads, g = tg - t * num_kv_heads;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (c == 0 && err) atomicOr(err, pa::ERR_BAD_SLOT);
        return;
    }
    const int64_t row = ((slot / kBlock) * num_kv_heads + g) * kBlock + slot % kBlock;
    Cached8<KV, D> a[kParts], b[kParts];
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
        a[j].load(k_cache, k_scale, k_zp, row, g, c + 8 * j);
        b[j].load(v_cache, v_scale, v_zp, row, g, c + 8 * j);
    }
    const int64_t dst = (int64_t)tg * D + 8 * c;
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
        store8(key + dst + 64 * j, a[j]);
        store8(value + dst + 64 * j, b[j]);
    }
}

struct CopyParams {
    uint4* arrays[6];
    int64_t vecs_per_block[6];
};

// grid = (n_pairs, 6): one CTA copies one block of one array.
__global__ void copy_blocks_kernel(CopyParams p, const int32_t* __restrict__ pairs, int n_pairs,
                                   int64_t num_blocks, unsigned int* err) {
    const int pair = blockIdx.x, arr = blockIdx.y;
    uint4* base = p.arrays[arr];
    if (!base) return;
    const int64_t src = __ldg(pairs + 2 * pair), dst = __ldg(pairs + 2 * pair + 1);
    if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
        if (threadIdx.x == 0 && err) atomicOr(err, pa::ERR_BAD_BLOCK);
        return;
    }
    const int64_t n = p.vecs_per_block[arr];
    const uint4* s = base + src * n;
    uint4* d = base + dst * n;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) d[i] = s[i];
}

}  // namespace

namespace pa {

pa_status launch_append_kv(const AppendArgs& a) {
    unsigned int* err = device_error_word();
    const int64_t num_slots = (int64_t)a.num_blocks * a.block_size;
    if (a.kv_dtype == PA_INT4) {
        const int64_t total = (int64_t)a.num_tokens * a.num_kv_heads * 8;
        if (total > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "too many tokens for one launch");
#define PA_LAUNCH_Q4(T, D)                                                                     \
    return cuda_status(                                                                        \
        launch_pdl(append_kv_int4_kernel<T, D>, dim3((unsigned)((total + 255) / 256)),         \
                   dim3(256), 0, a.stream, static_cast<const T*>(a.key),                       \
                   static_cast<const T*>(a.value), static_cast<uint8_t*>(a.k_cache),           \
                   static_cast<uint8_t*>(a.v_cache), a.k_scale, a.v_scale, a.k_zp, a.v_zp,     \
                   a.slots, (uint32_t)total, (uint32_t)a.num_kv_heads, num_slots, err),        \
        "append_kv launch")
        if (a.src_dtype == PA_BF16) {
            if (a.head_dim == 128) PA_LAUNCH_Q4(__nv_bfloat16, 128);
            PA_LAUNCH_Q4(__nv_bfloat16, 64);
        }
        if (a.head_dim == 128) PA_LAUNCH_Q4(__half, 128);
        PA_LAUNCH_Q4(__half, 64);
#undef PA_LAUNCH_Q4
    } else if (a.kv_dtype == PA_FP8_E4M3) {
        const int64_t total = (int64_t)a.num_tokens * a.num_kv_heads * (a.head_dim / 16);
        const int threads = 256;
        const int64_t blocks = (total + threads - 1) / threads;
        const int grid = (int)(blocks < 65535 ? blocks : 65535);
        if (((uintptr_t)a.k_scale | (uintptr_t)a.v_scale) % 4)
            return fail(PA_ERR_INVALID_ARG, "k_scale / v_scale must be 4-byte aligned");
        if (a.src_dtype == PA_BF16)
            append_kv_fp8_kernel<__nv_bfloat16><<<grid, threads, 0, a.stream>>>(
                static_cast<const __nv_bfloat16*>(a.key),
                static_cast<const __nv_bfloat16*>(a.value), static_cast<uint8_t*>(a.k_cache),
                static_cast<uint8_t*>(a.v_cache), a.k_scale, a.v_scale, a.slots, a.num_tokens,
                a.num_kv_heads, a.head_dim, num_slots, err);
        else
            append_kv_fp8_kernel<__half><<<grid, threads, 0, a.stream>>>(
                static_cast<const __half*>(a.key), static_cast<const __half*>(a.value),
                static_cast<uint8_t*>(a.k_cache), static_cast<uint8_t*>(a.v_cache), a.k_scale,
                a.v_scale, a.slots, a.num_tokens, a.num_kv_heads, a.head_dim, num_slots, err);
    } else if (a.kv_dtype != PA_INT8) {
        const int vec_per_row = a.head_dim * 2 / 16;
        const int64_t total = (int64_t)a.num_tokens * a.num_kv_heads * vec_per_row;
        const int threads = 256;
        const int64_t blocks = (total + threads - 1) / threads;
        const int grid = (int)(blocks < 65535 ? blocks : 65535);
        append_kv16_kernel<<<grid, threads, 0, a.stream>>>(
            static_cast<const uint4*>(a.key), static_cast<const uint4*>(a.value),
            static_cast<uint4*>(a.k_cache), static_cast<uint4*>(a.v_cache), a.slots,
            a.num_tokens, a.num_kv_heads, vec_per_row, num_slots, err);
    } else {
        const int64_t rows = (int64_t)a.num_tokens * a.num_kv_heads * 2;
        const int threads = 256;
        const int64_t grid = (rows * 32 + threads - 1) / threads;
        if (grid > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "too many tokens for one launch");
#define PA_LAUNCH_Q8(T, EPL)                                                                   \
    append_kv_int8_kernel<T, EPL><<<(unsigned)grid, threads, 0, a.stream>>>(                   \
        static_cast<const T*>(a.key), static_cast<const T*>(a.value),                          \
        static_cast<int8_t*>(a.k_cache), static_cast<int8_t*>(a.v_cache), a.k_scale,           \
        a.v_scale, a.k_zp, a.v_zp, a.slots, a.num_tokens, a.num_kv_heads, num_slots, err)
        if (a.src_dtype == PA_BF16) {
            if (a.head_dim == 128) PA_LAUNCH_Q8(__nv_bfloat16, 4);
            else PA_LAUNCH_Q8(__nv_bfloat16, 2);
        } else {
            if (a.head_dim == 128) PA_LAUNCH_Q8(__half, 4);
            else PA_LAUNCH_Q8(__half, 2);
        }
#undef PA_LAUNCH_Q8
    }
    return cuda_status(cudaGetLastError(), "append_kv launch");
}

namespace {

template <int KV, int D, typename T>
pa_status gather_as(const GatherArgs& a, uint32_t total) {
    return cuda_status(
        launch_pdl(gather_kv_kernel<KV, D, T>, dim3((total + 255u) / 256u), dim3(256), 0, a.stream,
                   static_cast<T*>(a.key), static_cast<T*>(a.value), a.k_cache, a.v_cache,
                   a.k_scale, a.v_scale, a.k_zp, a.v_zp, a.slots, total, (uint32_t)a.num_kv_heads,
                   (int64_t)a.num_blocks * kBlock, device_error_word()),
        "gather_kv launch");
}

template <int KV, int D>
pa_status gather_from(const GatherArgs& a, uint32_t total) {
    if (a.out_dtype == PA_F32) return gather_as<KV, D, float>(a, total);
    if (a.out_dtype == PA_F16) return gather_as<KV, D, __half>(a, total);
    return gather_as<KV, D, __nv_bfloat16>(a, total);
}

template <int KV>
pa_status gather_dim(const GatherArgs& a, uint32_t total) {
    return a.head_dim == 128 ? gather_from<KV, 128>(a, total) : gather_from<KV, 64>(a, total);
}

}  // namespace

pa_status launch_gather_kv(const GatherArgs& a) {
    const int64_t total = (int64_t)a.num_tokens * a.num_kv_heads * 8;
    if (total > 0x7fffffff) return fail(PA_ERR_UNSUPPORTED, "too many tokens for one launch");
    const uint32_t n = (uint32_t)total;
    switch (a.kv_dtype) {
        case PA_F16: return gather_dim<PA_F16>(a, n);
        case PA_BF16: return gather_dim<PA_BF16>(a, n);
        case PA_INT8: return gather_dim<PA_INT8>(a, n);
        case PA_INT4: return gather_dim<PA_INT4>(a, n);
        default: return gather_dim<PA_FP8_E4M3>(a, n);
    }
}

pa_status launch_copy_blocks(const CopyArgs& a) {
    CopyParams p{};
    for (int i = 0; i < 6; ++i) {
        p.arrays[i] = static_cast<uint4*>(a.arrays[i]);
        p.vecs_per_block[i] = a.bytes_per_block[i] / 16;
    }
    dim3 grid(a.n_pairs, 6);
    copy_blocks_kernel<<<grid, 256, 0, a.stream>>>(p, a.pairs, a.n_pairs, a.num_blocks,
                                                   device_error_word());
    return cuda_status(cudaGetLastError(), "copy_blocks launch");
}

}  // namespace pa
