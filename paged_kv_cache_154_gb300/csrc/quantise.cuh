// The quantisers of a cached row, from fp32 values, and the two-wide fp32
// arithmetic that they use.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
    return __bfloat162float(x);
}

// Two fp32 numbers and the two-wide arithmetic on them (each operation rounds
// as its scalar form does, but a product that is only added to may be fused
// with the sum).
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

// 8 values as codes of kTop + 1 levels from kLow up (4 bits: 15, 0; 8 bits: 255, -128),
// given the range [mn, mx] of what shares their scale, widened to hold 0: scale =
// (mx - mn) / kTop (1 if 0), zp = clamp(kLow - rint(mn / scale)), code =
// clamp(rint(x / scale) + zp), quotients correctly rounded, ties to even.
template <int kTop, int kLow>
struct Quantiser {
    static constexpr float kRound = 12582912.0f;   // 1.5 * 2^23
    float scale, inv;
    int zp;
    bool quick;

    __device__ __forceinline__ Quantiser(float mn, float mx) {
        const float range = __fsub_rn(mx, mn);
        // not too near the ends of fp32, for the remainders below to be exact
        quick = range > 1e-28f && range < 1e30f;
        if (quick) {
            // Correctly rounded quotients by Markstein's theorem: with the correctly rounded
            // reciprocal y of b, q = a y and r = a - b q (exact in one fused operation),
            // q + r y is the rounded a / b. Then, adding 1.5 * 2^23 rounds to an integer in
            // the low bits.
            constexpr float kPart = 1.0f / (float)kTop;
            const float s0 = __fmul_rn(range, kPart);
            scale = __fmaf_rn(__fmaf_rn(-s0, (float)kTop, range), kPart, s0);
            inv = __frcp_rn(scale);
            const float z0 = __fmul_rn(mn, inv);
            const float z1 = __fmaf_rn(__fmaf_rn(-z0, scale, mn), inv, z0);
            const float zr = __fadd_rn(z1, kRound);
            zp = min(kLow + kTop, kLow + __float_as_int(kRound) - __float_as_int(zr));
        } else {
            scale = __fdiv_rn(range, (float)kTop);
            if (scale == 0.0f) scale = 1.0f;
            const int z = kLow + (int)-rintf(__fdiv_rn(mn, scale));
            zp = z < kLow ? kLow : min(kLow + kTop, z);
            inv = 0.0f;
        }
    }

    // x[e] + 1.5 * 2^23 rounded, no code above the top (none is below the bottom: rounding
    // keeps the order, and the zero point is kLow - rint(mn / scale)); its bits less those
    // of 1.5 * 2^23 are code - zp
    __device__ __forceinline__ void round2(const float* x, float& a, float& b) const {
        const float top = __int_as_float(__float_as_int(kRound) + kLow + kTop - zp);
        const F2 v(x[0], x[1]), q = v * F2(inv, inv);
        const F2 r = fma(q, F2(-scale, -scale), v);
        const F2 y = fma(r, F2(inv, inv), q) + F2(kRound, kRound);
        a = fminf(y.lo(), top);
        b = fminf(y.hi(), top);
    }
    __device__ __forceinline__ int slow_code(float x) const {
        const int q = (int)rintf(__fdiv_rn(x, scale)) + zp;
        return q < kLow ? kLow : min(kLow + kTop, q);
    }

    // 8 codes of 4 bits, element 0 lowest: put together from the bits as they are (the
    // excess of each over its code is the same number)
    __device__ __forceinline__ uint32_t pack4(const float (&x)[8]) const {
        uint32_t word = 0;
        if (quick) {
#pragma unroll
            for (int e = 6; e >= 0; e -= 2) {
                float a, b;
                round2(x + e, a, b);
                word = word * 16u + __float_as_uint(b);
                word = word * 16u + __float_as_uint(a);
            }
            word -= (uint32_t)(__float_as_int(kRound) - zp) * 0x11111111u;
        } else {                        // range 0, or too near the ends of fp32
#pragma unroll
            for (int e = 0; e < 8; ++e) word |= (uint32_t)slow_code(x[e]) << (4 * e);
        }
        return word;
    }
    // 8 codes of 8 bits
    __device__ __forceinline__ uint2 pack8(const float (&x)[8]) const {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                if (quick) {
                    float a, b;
                    round2(x + 4 * h + e, a, b);
                    c[e] = __float_as_uint(a) + (uint32_t)zp;   // the low byte is the code's
                    c[e + 1] = __float_as_uint(b) + (uint32_t)zp;
                } else {
                    c[e] = (uint32_t)slow_code(x[4 * h + e]);
                    c[e + 1] = (uint32_t)slow_code(x[4 * h + e + 1]);
                }
            }
            w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040),
                               0x5410);
        }
        return make_uint2(w[0], w[1]);
    }
};

}  // namespace pa
