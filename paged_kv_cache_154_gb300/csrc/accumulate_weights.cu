// The attention weight that each cached token gets from a run of queries, and
// its sum over calls: the quantity by which tokens are evicted from a cache.
//
// For sequence s, KV head g and token t
//
//   out[s][g][t] = in[s][g][t] + sum_i sum_h softmax_t'(scale q_ih . k_t')[t]
//
// over the run's queries i (query i of a run of r sees tokens 0 .. L - r + i)
// and the query heads h of the group ("KV Cache ... PagedAttention" §二, the
// softmax of the attention formula, without its product with V). A weight needs
// its row's sum over all tokens, so there are two kernels:
//
//   1. logits_kernel: logits of a tile of tokens, and each row's (m, l) over it
//      (m = largest logit in base-2 units, l = sum 2^(a - m));
//   2. the tiles' (m, l) merged into a row's, and out = in + sum over rows
//      2^(a - m) / l: from the logits that kernel 1 stored (stored_kernel, which
//      merges for itself), or from logits computed again (many_kernel for both
//      passes, rows_kernel between them where contexts are long).
//
// Storing costs 8 bytes a row and token, mostly within L2; computing again costs
// a second read of K and its products. So few rows are stored (up to 16 rows
// per KV head, while the buffer stays under 256 MB and the workspace has room for
// it), many are computed again.
//
// What bounds it: for few rows the read of K, which goes from global memory to
// operand registers directly: tokens stand in the M dimension of the warp-level
// product, and as the order of the dims is free (q is loaded in the same order), a
// lane's 16-byte load of its token is four operand registers with no staging in
// shared memory. The Llama-3-8B-shaped step (64 sequences of 512-4096 tokens, bf16,
// 325 MB) takes 63.2 us: 54 us at 82 % of the copy rate, and the sum; one 4-bit sequence
// of 100001 tokens (66 MB) 24.5 us, where the chain of a block counts as much as its
// bytes. For many rows it is the latency of load, product and exponential: a tile of
// K is staged in shared memory once, for warps of 16 rows of q each.
// Codes are made exact in fp16: code - zero point (INT8), E4M3 to fp16, masked
// nibbles as subnormals with the zero points taken out of the sums (INT4, as in
// the decode kernel); q goes to fp16 after an exact power-of-two scaling per row.
// Sums and softmax are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "pa_internal.h"
#include "ptx.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kUnit = 16777216.f;       // 2^24: masked nibbles are subnormals in units of 2^-24
constexpr int kBS = 16;                  // tokens per block
constexpr int kWarps = 4;                // warps per CTA
constexpr int kMaxTile = 2048;            // tokens of a logits CTA: a lane holds a block id
static_assert(kMaxTile / kBS / kWarps <= 32, "a lane holds a block id");
constexpr int kOutTokens = 1024;         // tokens of a stored CTA
constexpr int kManyWarps = 8;            // warps of a many_kernel CTA
constexpr int kMaxRows = 4096;           // query rows per KV head
constexpr int64_t kMaxStored = (int64_t)256 << 20;
constexpr int64_t kMaxWorkspace = (int64_t)1 << 40;

struct Params {
    float* out;
    const float* in;          // may be null: zeros
    const void* q;
    const void* k;
    const float* k_scale;
    const int8_t* k_zp;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* qsl;       // may be null: one query token per sequence
    float* logits;            // [num_seqs x H_kv][max tokens, a multiple of 16][row_pad], or null
    float2* stats;            // [num_seqs x H_kv][row_slots][tiles]: (m, l)
    float2* sums;             // [num_seqs x H_kv][row_slots]: see row_sum; computed again only,
                              // null: every warp makes its rows' from stats
    int row_warps;            // many_kernel: warps over chunks of 16 rows; the others split tokens
    int tile_tokens;          // of stats
    unsigned int* err;
    int64_t stride;           // of in and out, per KV head
    int num_seqs, num_q_tokens, max_q_len, num_heads, num_kv_heads, group, num_blocks, max_blocks;
    int max_len, tokens_pad, tiles, row_slots, row_pad;
    int q_bf16;
    float scale_log2;
};

// Context length and query run of a sequence, kept inside the call's bounds.
struct Seq {
    int L, r, q0;
    __device__ __forceinline__ Seq(const Params& p, int s) {
        L = max(0, min(__ldg(p.context_lens + s), p.max_len));
        q0 = s;
        r = 1;
        if (p.qsl) {
            q0 = __ldg(p.qsl + s);
            r = max(0, min(__ldg(p.qsl + s + 1) - q0, p.max_q_len));
        }
        if (q0 < 0 || q0 > p.num_q_tokens - r) r = 0;
    }
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {   // low 16 bits
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(d)
        : "r"(w));
    return d;
}

__device__ __forceinline__ float exp2i(int e) {   // 2^e for e in [-126, 127]
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// the product of mma_16816 on a zero accumulator
template <bool BF16>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// (m, l) of a pair of partial sums
__device__ __forceinline__ void merge(float& m, float& l, float m2, float l2) {
    const float top = fmaxf(m, m2);
    const float ref = top == -INFINITY ? 0.f : top;
    l = l * pa::ex2(m - ref) + l2 * pa::ex2(m2 - ref);
    m = top;
}

// The K operand. Per lane (quad = lane / 4, qc = lane % 4) and token half h
// (token quad + 8 h of a block): kWords 32-bit words of the token's row, loaded
// kVec words at a time; frag() makes the A registers of k-step kk.
template <int KV, int D>
struct KRows {
    static constexpr bool k16 = KV == PA_F16 || KV == PA_BF16;
    static constexpr int kRowBytes = KV == PA_INT4 ? D / 2 : k16 ? 2 * D : D;
    static constexpr int kWords = kRowBytes / 16;
    static constexpr int kVec = KV == PA_INT4 ? 2 : 4;    // a 4-bit load stays in one group
    static constexpr int kGroups = KV == PA_INT4 ? D / PA_INT4_GROUP : 1;
    static constexpr int kSteps = D / 16;
    static constexpr bool kScaled = KV == PA_INT8 || KV == PA_INT4;
    uint32_t w[2][kWords];
    float scale[2][kGroups];
    int zp[2][kGroups];

    __device__ __forceinline__ void load_scales(const Params& p, int64_t row, int quad) {
        if constexpr (kScaled) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t t = row + quad + 8 * h;
                if constexpr (kGroups == 2) {
                    const float2 f = __ldg(reinterpret_cast<const float2*>(p.k_scale) + t);
                    const uint16_t z = __ldg(reinterpret_cast<const uint16_t*>(p.k_zp) + t);
                    scale[h][0] = f.x, scale[h][1] = f.y;
                    zp[h][0] = z & 255, zp[h][1] = z >> 8;   // 0 .. 15
                } else {
                    scale[h][0] = __ldg(p.k_scale + t);
                    zp[h][0] = __ldg(p.k_zp + t);
                }
            }
        }
    }
    template <typename V, typename Load>
    __device__ __forceinline__ void put(int h, int j, Load load) {
        const V u = load();
        w[h][kVec * j] = u.x, w[h][kVec * j + 1] = u.y;
        if constexpr (kVec == 4) w[h][4 * j + 2] = u.z, w[h][4 * j + 3] = u.w;
    }
    using Vec = typename std::conditional<kVec == 4, uint4, uint2>::type;
    // from global memory: rows `row` (token 0 of the block) + quad, + quad + 8 of the cache
    __device__ __forceinline__ void load(const Params& p, int64_t row, int quad, int qc) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t* src =
                static_cast<const uint8_t*>(p.k) + (row + quad + 8 * h) * kRowBytes + 4 * kVec * qc;
#pragma unroll
            for (int j = 0; j < kWords / kVec; ++j)
                put<Vec>(h, j, [&] { return __ldg(reinterpret_cast<const Vec*>(src + 16 * kVec * j)); });
        }
        load_scales(p, row, quad);
    }
    // A staged row: its 16-byte chunks are exchanged so that the rows of one load fall into
    // different banks (rows of 32 bytes, and of 64 loaded 16 at a time, need none).
    __device__ __forceinline__ static int staged_chunk(int row, int chunk) {
        if constexpr (KV == PA_INT4) return kRowBytes == 64 ? chunk ^ (row & 2) : chunk;
        else return kRowBytes >= 128 ? chunk ^ ((row & 1) << 2) : chunk;
    }
    // A lane's place in a staged block (of 16 rows); a load further is an exclusive-or away.
    __device__ __forceinline__ static uint32_t staged_at(int quad, int qc) {
        const int at = 4 * kVec * qc;
        return quad * kRowBytes + 16 * staged_chunk(quad, at / 16) + at % 16;
    }
    __device__ __forceinline__ void load_staged(uint32_t at) {   // staged block + staged_at
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kWords / kVec; ++j) {
                const uint32_t src = (at + 8 * h * kRowBytes) ^ (16 * kVec * j);
                if constexpr (kVec == 4)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[h][4 * j]), "=r"(w[h][4 * j + 1]), "=r"(w[h][4 * j + 2]),
                                   "=r"(w[h][4 * j + 3])
                                 : "r"(src));
                else
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                 : "=r"(w[h][2 * j]), "=r"(w[h][2 * j + 1])
                                 : "r"(src));
            }
    }

    // a pair of dims of one token, in the low (hi = 0) or high columns of k-step kk; INT4: in
    // units of 2^-24 (hi = 0) and 2^-20
    __device__ __forceinline__ uint32_t pair(int h, int kk, int hi) const {
        if constexpr (k16) {
            return w[h][2 * kk + hi];
        } else if constexpr (KV == PA_INT8) {
            // (code ^ 0x80) in the mantissa of 1024.0, less 1152 + zp: code - zp exactly
            const uint32_t z = prmt((uint32_t)zp[h][0] ^ 0x80u, 0x64646464u, 0x4040u);
            return hsub2(prmt(w[h][kk] ^ 0x80808080u, 0x64646464u, hi ? 0x4342u : 0x4140u), z);
        } else if constexpr (KV == PA_INT4) {
            const uint32_t u = kk & 1 ? w[h][kk / 2] >> 8 : w[h][kk / 2];
            return u & (hi ? 0x00f000f0u : 0x000f000fu);
        } else {
            return e4m3x2_to_f16x2(hi ? w[h][kk] >> 16 : w[h][kk]);
        }
    }
    __device__ __forceinline__ void frag(int kk, uint32_t (&a)[4]) const {
        a[0] = pair(0, kk, 0), a[1] = pair(1, kk, 0);
        a[2] = pair(0, kk, 1), a[3] = pair(1, kk, 1);
    }
};

// 8 NR query rows of one (sequence, KV head) as B operands, in K's order of
// dims: row 8 nr + quad of the chunk that starts at row `first`. mul: what a
// product of rows 8 nr + 2 qc + e is multiplied by; bound: the last token that
// row sees (-1: none); qsum: INT4, the sum of a group's q in the products' units.
template <int KV, int D, int NR>
struct QRows {
    using K = KRows<KV, D>;
    static constexpr int kSums = KV == PA_INT4 ? K::kGroups : 1;
    uint32_t b[NR][K::kSteps][2];
    float mul[NR][2];
    int bound[NR][2];
    float qsum[NR][kSums][2];

    // OWN: mul, bound and qsum are those of rows 8 nr + quad instead, in [..][0]
    template <bool OWN = false>
    __device__ __forceinline__ void load(const Params& p, const Seq& sq, int g, int first,
                                         int quad, int qc) {
        const int rows = p.group * sq.r;
        float head = p.scale_log2;
        if constexpr (KV == PA_FP8_E4M3) head *= __ldg(p.k_scale + g);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = first + 8 * nr + quad;
            const bool on = row < rows;
            const int qi = on ? row / p.group : 0;
            const uint16_t* src =
                static_cast<const uint16_t*>(p.q) +
                ((int64_t)(sq.q0 + qi) * p.num_heads + g * p.group + (on ? row - qi * p.group : 0)) * D;
            float m = on ? head : 0.f, qs[kSums] = {};
            if constexpr (K::k16) {
#pragma unroll
                for (int j = 0; j < K::kSteps / 2; ++j) {
                    uint4 u = make_uint4(0u, 0u, 0u, 0u);
                    if (on) u = __ldg(reinterpret_cast<const uint4*>(src + 32 * j + 8 * qc));
                    b[nr][2 * j][0] = u.x, b[nr][2 * j][1] = u.y;
                    b[nr][2 * j + 1][0] = u.z, b[nr][2 * j + 1][1] = u.w;
                }
            } else {
                // the lane's dims 64 j + 16 qc .. + 15, then fp16 after scaling the row's largest
                // element into [2^14, 2^15)
                float v[D / 64][16], mx = 0.f;
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 u = make_uint4(0u, 0u, 0u, 0u);
                        if (on)
                            u = __ldg(reinterpret_cast<const uint4*>(src + 64 * j + 16 * qc + 8 * i));
                        const uint16_t* x = reinterpret_cast<const uint16_t*>(&u);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float f = p.q_bf16 ? __uint_as_float((uint32_t)x[e] << 16)
                                                     : __half2float(__ushort_as_half(x[e]));
                            v[j][8 * i + e] = f;
                            mx = fmaxf(mx, fabsf(f));
                        }
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                int ex = 0;
                if (mx > 0.f) {
                    ex = (int)((__float_as_uint(mx) >> 23) & 0xff) - 127;
                    ex = max(-100, min(100, ex));
                }
                const float up = exp2i(14 - ex);
                m *= exp2i(ex - 14);
                if constexpr (KV == PA_INT4) m *= kUnit;
#pragma unroll
                for (int kk = 0; kk < K::kSteps; ++kk)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float* x = v[kk / 4];
                        __half2 h;
                        if constexpr (KV == PA_INT4) {
                            // nibbles 0 and 4, 1 and 5 | 2 and 6, 3 and 7 of word kk / 2
                            const int i = 8 * (kk / 2 & 1) + 2 * (kk & 1) + e;
                            const float f = e ? up * 0.0625f : up;
                            h = __floats2half2_rn(x[i] * f, x[i + 4] * f);
                            const float2 r = __half22float2(h);
                            qs[kk / 4] += (r.x + r.y) * (e ? 16.f / kUnit : 1.f / kUnit);
                        } else {
                            const int i = 4 * (kk & 3) + 2 * e;
                            h = __floats2half2_rn(x[i] * up, x[i + 1] * up);
                        }
                        b[nr][kk][e] = *reinterpret_cast<const uint32_t*>(&h);
                    }
            }
            if constexpr (KV == PA_INT4) {
#pragma unroll
                for (int i = 0; i < kSums; ++i) {
                    qs[i] += __shfl_xor_sync(0xffffffffu, qs[i], 1);
                    qs[i] += __shfl_xor_sync(0xffffffffu, qs[i], 2);
                }
            }
            if constexpr (OWN) {
                mul[nr][0] = m;
#pragma unroll
                for (int i = 0; i < kSums; ++i) qsum[nr][i][0] = qs[i];
                bound[nr][0] = on ? min(sq.L - sq.r + qi, sq.L - 1) : -1;
                continue;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mul[nr][e] = __shfl_sync(0xffffffffu, m, 4 * (2 * qc + e));
#pragma unroll
                for (int i = 0; i < kSums; ++i)
                    qsum[nr][i][e] = __shfl_sync(0xffffffffu, qs[i], 4 * (2 * qc + e));
                const int mine = first + 8 * nr + 2 * qc + e;
                bound[nr][e] = mine < rows ? min(sq.L - sq.r + mine / p.group, sq.L - 1) : -1;
            }
        }
    }

    // logits (base-2 units) of the block whose first token is tok0: a[nr][2 h + e] of
    // token quad + 8 h and row 8 nr + 2 qc + e; -inf where the row does not see it
    // (masked: some row may not see all of it)
    __device__ __forceinline__ void logits(const K& k, int tok0, int quad, bool masked,
                                           float (&a)[NR][4]) const {
        float s[NR][K::kGroups][4];
#pragma unroll
        for (int kk = 0; kk < K::kSteps; ++kk) {
            uint32_t f[4];
            k.frag(kk, f);
            const int grp = kk * K::kGroups / K::kSteps;
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
                if (kk % (K::kSteps / K::kGroups) == 0)
                    mma_first<KV == PA_BF16>(s[nr][grp], f, b[nr][kk][0], b[nr][kk][1]);
                else
                    pa::mma_16816<KV == PA_BF16>(s[nr][grp], f, b[nr][kk][0], b[nr][kk][1]);
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = s[nr][0][2 * h + e];
                    if constexpr (KV == PA_INT4) v = fmaf(-(float)k.zp[h][0], qsum[nr][0][e], v);
                    if constexpr (K::kScaled) v *= k.scale[h][0];
                    if constexpr (K::kGroups == 2)
                        v = fmaf(fmaf(-(float)k.zp[h][1], qsum[nr][1][e], s[nr][1][2 * h + e]),
                                 k.scale[h][1], v);
                    a[nr][2 * h + e] = v * mul[nr][e];
                }
        if (masked) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tok0 + quad + 8 * (i >> 1) > bound[nr][i & 1]) a[nr][i] = -INFINITY;
        }
    }
};

// The running sums of a warp's rows: l = sum 2^(a - ref) over the tokens that the
// lane sees. The reference is the warp's (lanes of a row agree) and moves only when
// a logit passes it by 2^8; -inf: no token seen yet.
template <int NR>
struct RowSums {
    float ref[NR][2], l[NR][2];
    __device__ __forceinline__ void clear(const int (&bound)[NR][2]) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ref[nr][e] = bound[nr][e] < 0 ? 0.f : -INFINITY;   // rows that see nothing at all
                l[nr][e] = 0.f;
            }
    }
    __device__ __forceinline__ void add(const float (&a)[NR][4]) {
        float t[NR][4];
        bool raise = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) t[nr][i] = a[nr][i] - ref[nr][i & 1];
#pragma unroll
            for (int e = 0; e < 2; ++e) raise |= !(fmaxf(t[nr][e], t[nr][2 + e]) <= 8.f);
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(a[nr][e], a[nr][2 + e]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    if (mx > ref[nr][e] + 8.f) {
                        l[nr][e] *= pa::ex2(ref[nr][e] - mx);   // 0 while ref is -inf
                        ref[nr][e] = mx;
                    }
                    // still no token: nothing but -inf and NaN, which stays
                    const bool none = ref[nr][e] == -INFINITY;
#pragma unroll
                    for (int i = e; i < 4; i += 2)
                        t[nr][i] = none && a[nr][i] == -INFINITY ? -INFINITY
                                                                 : a[nr][i] - ref[nr][e];
                }
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) l[nr][e] += pa::ex2(t[nr][e]) + pa::ex2(t[nr][2 + e]);
    }
    // over the warp's tokens: (reference, sum) of rows 8 nr + 2 qc + e to part[]
    __device__ __forceinline__ void finish(float2* part, int quad, int qc) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nr][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (quad == 0) part[8 * nr + 2 * qc + e] = make_float2(ref[nr][e], sum);
            }
    }
};

__device__ __forceinline__ int block_of(const Params& p, int s, int i) {
    const int blk = __ldg(p.block_tables + (int64_t)s * p.max_blocks + i);
    if (blk >= 0 && blk < p.num_blocks) return blk;
    if (p.err) atomicOr(p.err, pa::ERR_BAD_BLOCK);
    return 0;
}

// Grid: (tiles of p.tile_tokens tokens, KV head, sequence): few rows, stored logits.
template <int KV, int D, int NR>
__global__ void __launch_bounds__(kWarps * 32) logits_kernel(const Params p) {
    // blocks of K in registers, on their way while one is multiplied (of 16-bit rows of 128,
    // 2: 64.1 us for the Llama-3-8B-shaped step, 3: 63.2; of smaller rows 5 are no better)
    constexpr int kDepth = KRows<KV, D>::kWords >= 16 ? 3 : 4;
    __shared__ float2 part[kWarps][8 * NR];
    // let the sum's kernel in only now: what ran before this one has ended, and that kernel
    // reads its inputs before it waits
    pa::grid_dependency_wait();
    pa::grid_dependents_launch();
    const int s = blockIdx.z, g = blockIdx.y, tile = blockIdx.x;
    const Seq sq(p, s);
    const int rows = p.group * sq.r;
    if (tile * p.tile_tokens >= sq.L || rows == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, qc = lane & 3;
    // this warp's blocks: b0 + warp, + kWarps, ...
    const int b0 = tile * (p.tile_tokens / kBS) + warp;
    const int nb = min((sq.L + kBS - 1) / kBS, (tile + 1) * (p.tile_tokens / kBS));
    // the same in all lanes, which a reduction tells the compiler too
    const int n = __reduce_max_sync(0xffffffffu, b0 < nb ? (nb - b0 + kWarps - 1) / kWarps : 0);
    int my_block = 0;
    if (lane < n) my_block = block_of(p, s, b0 + lane * kWarps);
    auto fetch = [&](KRows<KV, D>& k, int i) {   // past the last: the last again, not used
        const int64_t blk = __shfl_sync(0xffffffffu, my_block, min(i, n - 1));
        k.load(p, (blk * p.num_kv_heads + g) * kBS, quad, qc);
    };
    KRows<KV, D> k[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(k[i], i);
    QRows<KV, D, NR> q;
    q.load(p, sq, g, 0, quad, qc);
    RowSums<NR> sums;
    sums.clear(q.bound);
    // the lane's logits: rows 8 nr + 2 qc and + 1 of token quad, those that are kept
    float* keep = p.logits +
                  (((int64_t)s * p.num_kv_heads + g) * p.tokens_pad + b0 * kBS + quad) * p.row_pad +
                  2 * qc;
    const int half = 8 * p.row_pad, step = kWarps * kBS * p.row_pad;
    for (int i0 = 0; i0 < n; i0 += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            const int i = i0 + u;
            if (i >= n) break;
            fetch(k[(u + kDepth - 1) % kDepth], i + kDepth - 1);
            const int tok0 = (b0 + i * kWarps) * kBS;
            float a[NR][4];
            q.logits(k[u], tok0, quad, tok0 + kBS - 1 > sq.L - sq.r, a);
            sums.add(a);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
                if (8 * nr + 2 * qc < p.row_pad) {
                    *reinterpret_cast<float2*>(keep + 8 * nr) = make_float2(a[nr][0], a[nr][1]);
                    *reinterpret_cast<float2*>(keep + half + 8 * nr) = make_float2(a[nr][2], a[nr][3]);
                }
            keep += step;
        }
    }
    sums.finish(part[warp], quad, qc);
    __syncthreads();
    const int row = threadIdx.x;
    if (row < min(8 * NR, rows)) {
        float2 t = part[0][row];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) merge(t.x, t.y, part[w][row].x, part[w][row].y);
        p.stats[(((int64_t)s * p.num_kv_heads + g) * p.row_slots + row) * p.tiles + tile] = t;
    }
}

// What turns a row's logit a into its weight 2^(a - ref) * inv, from the (m, l)
// of its tiles, by LANES lanes: ref = m and inv = 1 / l, or 0 and 0 for a row that
// saw nothing.
template <int LANES>
__device__ __forceinline__ float2 row_sum(const Params& p, const Seq& sq, int64_t sg, int row,
                                          int lane) {
    const int tiles = (sq.L + p.tile_tokens - 1) / p.tile_tokens;
    const float2* src = p.stats + (sg * p.row_slots + row) * p.tiles;
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int i = lane; i < tiles; i += LANES) {
        const float2 t = __ldcg(src + i);   // the kernel before may have ended under this one
        merge(m, l, t.x, t.y);
    }
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1)
        merge(m, l, __shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, l, off));
    return make_float2(m == -INFINITY ? 0.f : m, l == 0.f ? 0.f : 1.f / l);
}

// Grid: (rows / kWarps, KV head, sequence): a warp a row, between many_kernel's passes.
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const Params p) {
    pa::grid_dependents_launch();
    pa::grid_dependency_wait();
    const int s = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 31;
    const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const Seq sq(p, s);
    if (row >= p.group * sq.r) return;
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const float2 t = row_sum<32>(p, sq, sg, row, lane);
    if (lane == 0) p.sums[sg * p.row_slots + row] = t;
}

// Grid: (tiles of kOutTokens tokens, KV head, sequence). RP: the rows a token
// has in the stored logits. Bound by latency (lengths, logits and row sums, output):
// the lengths and the weights so far are read before the logits are complete, and up to
// 6 CTAs share an SM (one 4-bit sequence of 100001 tokens: 24.5 us a call, 26.0 with 4
// CTAs, 26.5 without the early reads either).
template <int RP>
__global__ void __launch_bounds__(256, RP <= 4 ? 6 : RP == 8 ? 3 : 2) stored_kernel(const Params p) {
    __shared__ float2 sum[RP];
    const int s = blockIdx.z, g = blockIdx.y;
    const Seq sq(p, s);
    const int t0 = blockIdx.x * kOutTokens;
    if (t0 >= sq.L) {
        pa::grid_dependency_wait();
        return;
    }
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const int rows = p.group * sq.r;
    const int64_t base = sg * p.stride;
    constexpr int kEach = kOutTokens / 256;   // tokens of a thread, all asked for together
    float a[kEach][RP], before[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = t0 + i * 256 + threadIdx.x;
        before[i] = 0.f;
        if (t < sq.L && p.in) before[i] = __ldcg(p.in + base + t);
    }
    pa::grid_dependency_wait();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = t0 + i * 256 + threadIdx.x;
        if (t >= sq.L) continue;
        if (rows > 0) {
            const float* src = p.logits + (sg * p.tokens_pad + t) * RP;
            if constexpr (RP >= 4) {
#pragma unroll
                for (int j = 0; j < RP / 4; ++j)
                    *reinterpret_cast<float4*>(a[i] + 4 * j) =
                        __ldcs(reinterpret_cast<const float4*>(src) + j);
            } else {
#pragma unroll
                for (int j = 0; j < RP; ++j) a[i][j] = __ldcs(src + j);
            }
        }
    }
    for (int row = threadIdx.x >> 5; row < min(rows, RP); row += 8) {
        const float2 t = row_sum<32>(p, sq, sg, row, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0) sum[row] = t;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int t = t0 + i * 256 + threadIdx.x;
        if (t >= sq.L) continue;
        float w = 0.f;
#pragma unroll
        for (int j = 0; j < RP; ++j)
            if (j < rows) w = fmaf(pa::ex2(a[i][j] - sum[j].x), sum[j].y, w);
        p.out[base + t] = before[i] + w;
    }
}

// Tokens of a many_kernel tile: enough for the starts of its warps to be worth it
// (1.6 us less for the 8 prompts below than 128), 64 KB of K at most.
constexpr int kManyTokens = 256;

// 16 rows against the 16 tokens of two blocks, rows in the M dimension: the 16 bytes
// that a lane loads of a token are B operands as they come (with tokens in M an A operand
// mixes two tokens' words, which cost a move each), and the rows' A operands come from
// shared memory, one load for both blocks (kept in registers, they were copied for every
// product). Two blocks, since the chain of a block's load, products and vote is what a warp
// waits for. v[u][nr][h][e]: product of row 8 nr + quad and token 8 h + 2 qc + e of block u,
// without the row's factor.
template <int KV, int D>
struct ManyBlocks {
    using K = KRows<KV, D>;
    float v[2][2][2][2];
    __device__ __forceinline__ void run(const Params& p, const QRows<KV, D, 2>& q, uint32_t qa,
                                        const uint32_t (&staged)[2], const int64_t (&row)[2],
                                        int quad, int qc) {
        constexpr int G = K::kGroups;
        K k[2];
        float scale[2][2][2][G], zp[2][2][2][G];    // of tokens 8 h + 2 qc + e
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            k[u].load_staged(staged[u]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t t = row[u] + 8 * h + 2 * qc;
                float(&sc)[2][G] = scale[u][h];
                float(&z0)[2][G] = zp[u][h];
                if constexpr (KV == PA_INT8) {
                    sc[0][0] = __ldg(p.k_scale + t), sc[1][0] = __ldg(p.k_scale + t + 1);
                    k[u].zp[h][0] = __ldg(p.k_zp + row[u] + 8 * h + quad);
                } else if constexpr (G == 2) {
                    const float4 f = __ldg(reinterpret_cast<const float4*>(p.k_scale + 2 * t));
                    const uint32_t z = __ldg(reinterpret_cast<const uint32_t*>(p.k_zp + 2 * t));
                    sc[0][0] = f.x, sc[0][1] = f.y, sc[1][0] = f.z, sc[1][1] = f.w;
                    z0[0][0] = (float)(z & 255), z0[0][1] = (float)(z >> 8 & 255);
                    z0[1][0] = (float)(z >> 16 & 255), z0[1][1] = (float)(z >> 24);
                } else if constexpr (KV == PA_INT4) {
                    const float2 f = __ldg(reinterpret_cast<const float2*>(p.k_scale + t));
                    const uint16_t z = __ldg(reinterpret_cast<const uint16_t*>(p.k_zp + t));
                    sc[0][0] = f.x, sc[1][0] = f.y;
                    z0[0][0] = (float)(z & 255), z0[1][0] = (float)(z >> 8);
                }
            }
        }
        float s[2][2][G][4];
#pragma unroll
        for (int kk = 0; kk < K::kSteps; ++kk) {
            uint32_t a[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                         : "r"(qa + 512 * kk));
            const int g = kk * G / K::kSteps;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (kk % (K::kSteps / G) == 0)
                        mma_first<KV == PA_BF16>(s[u][h][g], a, k[u].pair(h, kk, 0),
                                                 k[u].pair(h, kk, 1));
                    else
                        pa::mma_16816<KV == PA_BF16>(s[u][h][g], a, k[u].pair(h, kk, 0),
                                                     k[u].pair(h, kk, 1));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int u = i / 8, nr = i / 4 % 2, h = i / 2 % 2, e = i % 2;
            float x = s[u][h][0][2 * nr + e];
            if constexpr (KV == PA_INT4) x = fmaf(-zp[u][h][e][0], q.qsum[nr][0][0], x);
            if constexpr (K::kScaled) x *= scale[u][h][e][0];
            if constexpr (G == 2)
                x = fmaf(fmaf(-zp[u][h][e][1], q.qsum[nr][1][0], s[u][h][1][2 * nr + e]),
                         scale[u][h][e][1], x);
            v[u][nr][h][e] = x;
        }
    }
    // logits (base-2 units) less ref, -inf where the row does not see the token
    __device__ __forceinline__ void relative(const QRows<KV, D, 2>& q, const float (&ref)[2],
                                             const int (&tok0)[2], int qc, bool masked,
                                             float (&t)[2][2][2][2]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int u = i / 8, nr = i / 4 % 2, h = i / 2 % 2, e = i % 2;
            t[u][nr][h][e] = fmaf(v[u][nr][h][e], q.mul[nr][0], -ref[nr]);
        }
        if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int u = i / 8, nr = i / 4 % 2, h = i / 2 % 2, e = i % 2;
                if (tok0[u] + 8 * h + 2 * qc + e > q.bound[nr][0]) t[u][nr][h][e] = -INFINITY;
            }
        }
    }
};

// The running sums of the lane's rows quad and quad + 8, as RowSums.
struct ManySums {
    float ref[2], l[2];
    template <int KV, int D>
    __device__ __forceinline__ void clear(const QRows<KV, D, 2>& q) {
#pragma unroll
        for (int nr = 0; nr < 2; ++nr) {
            ref[nr] = q.bound[nr][0] < 0 ? 0.f : -INFINITY;
            l[nr] = 0.f;
        }
    }
    __device__ __forceinline__ static float largest(const float (&t)[2][2][2][2], int nr) {
        return fmaxf(fmaxf(fmaxf(t[0][nr][0][0], t[0][nr][0][1]), fmaxf(t[0][nr][1][0], t[0][nr][1][1])),
                     fmaxf(fmaxf(t[1][nr][0][0], t[1][nr][0][1]), fmaxf(t[1][nr][1][0], t[1][nr][1][1])));
    }
    template <int KV, int D>
    __device__ __forceinline__ void add(const ManyBlocks<KV, D>& b, const QRows<KV, D, 2>& q,
                                        const int (&tok0)[2], int qc, bool masked) {
        float t[2][2][2][2];
        b.relative(q, ref, tok0, qc, masked, t);
        const bool raise = !(largest(t, 0) <= 8.f) || !(largest(t, 1) <= 8.f);
        if (__any_sync(0xffffffffu, raise)) {
            const float zero[2] = {0.f, 0.f};
            float a[2][2][2][2];
            b.relative(q, zero, tok0, qc, masked, a);
#pragma unroll
            for (int nr = 0; nr < 2; ++nr) {
                float mx = largest(a, nr);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (mx > ref[nr] + 8.f) {
                    l[nr] *= pa::ex2(ref[nr] - mx);   // 0 while ref is -inf
                    ref[nr] = mx;
                }
                // still no token: nothing but -inf and NaN, which stays
                const bool none = ref[nr] == -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = a[i / 4][nr][i / 2 % 2][i % 2];
                    t[i / 4][nr][i / 2 % 2][i % 2] = none && x == -INFINITY ? -INFINITY : x - ref[nr];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nr = 0; nr < 2; ++nr)
                l[nr] += (pa::ex2(t[u][nr][0][0]) + pa::ex2(t[u][nr][0][1])) +
                         (pa::ex2(t[u][nr][1][0]) + pa::ex2(t[u][nr][1][1]));
    }
    __device__ __forceinline__ void finish(float2* part, int quad, int qc) {
#pragma unroll
        for (int nr = 0; nr < 2; ++nr) {
            float sum = l[nr];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (qc == 0) part[8 * nr + quad] = make_float2(ref[nr], sum);
        }
    }
};

// Many rows. Grid: (tiles of kManyTokens, KV head, sequence). The tile's K is
// staged in shared memory once; warp (rc, tg) takes the row chunks rc, rc +
// row_warps, .. of 16 rows and the tile's blocks tg, tg + token_warps, ... SUM
// false: the rows' (m, l) over the tile; SUM true: the weights of the tile's
// tokens, summed over the rows (each warp keeps sums of its own, which are added
// up in a fixed order). Bound by the latency of a warp's pairs of blocks. 8 prompts
// of up to 4001 tokens, 128 rows, d = 64: 23.5 us a call; 3.5 us more with tokens in
// M, a block at a time, and 11 more again with K loaded from global memory for every
// chunk of rows.
template <int KV, int D, bool SUM>
__global__ void __launch_bounds__(32 * kManyWarps) many_kernel(const Params p) {
    constexpr int NR = 2, kTokens = kManyTokens, kBlocks = kTokens / kBS;
    constexpr int kRowBytes = KRows<KV, D>::kRowBytes, kChunks = kRowBytes / 16;
    // K, then SUM: float [row_warps][kTokens]; aligned to the span that staged rows exchange in
    extern __shared__ __align__(256) uint8_t tile_s[];
    __shared__ int blocks_s[kBlocks];
    __shared__ uint4 turn_s[kManyWarps][KRows<KV, D>::kSteps][32];
    __shared__ float2 part_s[kManyWarps][8 * NR];
    pa::grid_dependents_launch();
    pa::grid_dependency_wait();
    const int s = blockIdx.z, g = blockIdx.y, tile = blockIdx.x, t0 = tile * kTokens;
    const Seq sq(p, s);
    const int rows = p.group * sq.r;
    if (t0 >= sq.L || (!SUM && rows == 0)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, qc = lane & 3;
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const int nb = min(kBlocks, (sq.L - t0 + kBS - 1) / kBS);
    float* const sums = reinterpret_cast<float*>(tile_s + kTokens * kRowBytes);
    if (rows > 0) {
        if (tid < nb) blocks_s[tid] = block_of(p, s, t0 / kBS + tid);
        if (SUM)
            for (int i = tid; i < p.row_warps * kTokens; i += 32 * kManyWarps) sums[i] = 0.f;
        __syncthreads();
        for (int i = tid; i < nb * kBS * kChunks; i += 32 * kManyWarps) {
            const int t = i / kChunks, c = i % kChunks;
            const int64_t row = ((int64_t)blocks_s[t / kBS] * p.num_kv_heads + g) * kBS + t % kBS;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(pa::smem_addr(
                             tile_s + t * kRowBytes + 16 * KRows<KV, D>::staged_chunk(t, c))),
                         "l"(static_cast<const uint8_t*>(p.k) + row * kRowBytes + 16 * c)
                         : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    }
    const uint32_t staged = pa::smem_addr(tile_s) + KRows<KV, D>::staged_at(quad, qc);
    const int row_warps = p.row_warps, token_warps = kManyWarps / row_warps;
    const int rc = warp % row_warps, tg = warp / row_warps;
    const int rounds = (rows + 8 * NR * row_warps - 1) / (8 * NR * row_warps);
    for (int it = 0; it < rounds; ++it) {
        const int first = (it * row_warps + rc) * 8 * NR;
        // the last token that every row of the chunk sees (rows past the last see none)
        const int last_seen = first + 8 * NR <= rows ? sq.L - sq.r + first / p.group : -1;
        QRows<KV, D, NR> q;
        ManySums own;
        float ref[2], inv[2];
        if (first < rows) {              // warp-uniform
            q.template load<true>(p, sq, g, first, quad, qc);
#pragma unroll
            for (int kk = 0; kk < KRows<KV, D>::kSteps; ++kk)
                turn_s[warp][kk][lane] =
                    make_uint4(q.b[0][kk][0], q.b[1][kk][0], q.b[0][kk][1], q.b[1][kk][1]);
            __syncwarp();
            const uint32_t qa = pa::smem_addr(&turn_s[warp][0][lane]);
            own.clear(q);
            if constexpr (SUM) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    const int row = first + 8 * nr + quad;
                    float2 t = make_float2(0.f, 0.f);
                    if (p.sums) {
                        if (row < rows) t = __ldcg(p.sums + sg * p.row_slots + row);
                    } else {
                        t = row_sum<4>(p, sq, sg, min(row, rows - 1), qc);
                    }
                    ref[nr] = t.x, inv[nr] = t.y;
                }
            }
            for (int b = tg; b < nb; b += 2 * token_warps) {
                const int second = b + token_warps;
                const bool both = second < nb;      // else the first again, masked
                const int at[2] = {b, both ? second : b};
                uint32_t from[2];
                int64_t row[2];
                int tok0[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    from[u] = staged + at[u] * kBS * kRowBytes;
                    row[u] = KRows<KV, D>::kScaled
                                 ? ((int64_t)blocks_s[at[u]] * p.num_kv_heads + g) * kBS
                                 : 0;
                    tok0[u] = t0 + at[u] * kBS;
                }
                const bool masked = !both || tok0[1] + kBS - 1 > last_seen;
                if (!both) tok0[1] = INT_MAX / 2;
                ManyBlocks<KV, D> blocks;
                blocks.run(p, q, qa, from, row, quad, qc);
                if constexpr (!SUM) {
                    own.add(blocks, q, tok0, qc, masked);
                } else {
                    float t[2][2][2][2];
                    blocks.relative(q, ref, tok0, qc, masked, t);
                    // over the 8 lanes of a token, which split the eight tokens between them
                    const bool up = lane & 16, odd = lane & 8, far = lane & 4;
                    float w[2][4];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i / 4][i % 4] = fmaf(pa::ex2(t[i / 4][0][i / 2 % 2][i % 2]), inv[0],
                                               pa::ex2(t[i / 4][1][i / 2 % 2][i % 2]) * inv[1]);
                    float x[4], y[2];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = (up ? w[1][i] : w[0][i]) +
                               __shfl_xor_sync(0xffffffffu, up ? w[0][i] : w[1][i], 16);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        y[i] = (odd ? x[2 + i] : x[i]) +
                               __shfl_xor_sync(0xffffffffu, odd ? x[i] : x[2 + i], 8);
                    const float sum = (far ? y[1] : y[0]) +
                                      __shfl_xor_sync(0xffffffffu, far ? y[0] : y[1], 4);
                    if (both || !up)
                        sums[rc * kTokens + (up ? at[1] : at[0]) * kBS + (odd ? 8 : 0) + 2 * qc +
                             (far ? 1 : 0)] += sum;
                }
            }
        }
        if constexpr (!SUM) {
            if (first < rows) own.finish(part_s[warp], quad, qc);
            __syncthreads();
            const int c = tid / (8 * NR), i = tid % (8 * NR);
            const int row = (it * row_warps + c) * 8 * NR + i;
            if (c < row_warps && row < rows) {
                float2 t = part_s[c][i];
                for (int w = 1; w < token_warps; ++w)
                    merge(t.x, t.y, part_s[c + w * row_warps][i].x, part_s[c + w * row_warps][i].y);
                p.stats[(sg * p.row_slots + row) * p.tiles + tile] = t;
            }
            __syncthreads();
        }
    }
    if constexpr (SUM) {
        __syncthreads();
        const int64_t base = sg * p.stride + t0;
        for (int t = tid; t < min(kTokens, sq.L - t0); t += 32 * kManyWarps) {
            float w = 0.f;
            if (rows > 0)
                for (int c = 0; c < row_warps; ++c) w += sums[c * kTokens + t];
            p.out[base + t] = (p.in ? p.in[base + t] : 0.f) + w;
        }
    }
}

// Tokens of a logits CTA: one wave of four CTAs a SM where a tile of up to
// kMaxTile does that (fewer starts: 100001 tokens of 8 heads 41.7 us against 44.5
// with 512 in bf16, 24.6 against 29.8 in 4 bits), else 512, whose many waves even out
// a ragged batch (Llama-3-8B step: 63.4 us, 68.2 with 2048; 45.8 and 46.9 in 4 bits).
// Few long contexts or even ones would rather have 2048 there too (2 of 131072 tokens:
// 108.1 us, 103.1; 69.4 and 64.9 in 4 bits), but the host does not see the lengths.
constexpr int kMinTile = 128;
static_assert(kManyTokens >= kMinTile, "stats are sized for tiles of kMinTile");
int stored_tile(int64_t tokens) {
    const int64_t t = (tokens + 4 * 152 - 1) / (4 * 152);
    return t > kMaxTile ? 512 : (int)std::max<int64_t>(kMinTile, (t + 63) / 64 * 64);
}

// Up to as many tiles the warps of the last pass merge their rows' (m, l) themselves, by
// one batch of loads; beyond, a kernel between the passes does it once. 8 prompts, 4 heads
// of 128 rows, d = 64: of 3900 tokens (16 tiles) 36.4 us, 37.0 with that kernel; of 5000
// (20) 40.3 and 40.0; of 6000 (24) 42.2 and 41.4; of 8192 (32) 58.1 and 54.6. 2 prompts, 8
// heads of 64 rows, d = 128: of 3900 19.0 and 20.3, of 4300 (17) 19.8 and 20.5, of 5000 31.6
// and 31.1, of 6000 34.8 and 32.9.
constexpr int kFoldTiles = 16;

// A call computes its logits twice in a workspace of stats and sums, whose sizes grow
// with every argument, so that a buffer sized for the largest call serves them all;
// where the logits are worth storing and find room behind the stats it stores them.
struct Shape {
    int64_t rows;         // most query rows per KV head
    int row_pad, tokens_pad;
    int64_t stats_bytes;  // (m, l) of tiles of kMinTile tokens, the smallest
    int64_t sums_bytes;   // computed again
    int64_t logits_bytes; // stored; 0: not worth it
    bool fits;            // false: larger than a call may be, the rest is not set

    int64_t least_bytes() const { return stats_bytes + sums_bytes; }
    int64_t stored_bytes() const { return logits_bytes ? stats_bytes + logits_bytes : INT64_MAX; }
    int64_t bytes() const {
        return logits_bytes ? std::max(least_bytes(), stored_bytes()) : least_bytes();
    }
};

Shape shape_of(int num_seqs, int num_heads, int num_kv_heads, int max_q_len, int max_len) {
    Shape h{};
    h.rows = (int64_t)(num_heads / num_kv_heads) * max_q_len;
    // bounds that keep every product below in 64 bits
    if (num_seqs > 65535 || num_kv_heads > 65535 || h.rows > kMaxRows || max_len > pa::kMaxTokens)
        return h;
    h.tokens_pad = (max_len + kBS - 1) / kBS * kBS;
    const int64_t sg = (int64_t)num_seqs * num_kv_heads;
    h.row_pad = 2;            // two rows a store
    while (h.row_pad < h.rows) h.row_pad *= 2;
    if (h.rows <= 16 && sg * h.tokens_pad <= kMaxStored / (4 * h.row_pad))
        h.logits_bytes = sg * h.tokens_pad * h.row_pad * 4;
    const int64_t tiles = (max_len + kMinTile - 1) / kMinTile;
    if (sg * h.rows > kMaxWorkspace / 8 / tiles) return h;
    h.stats_bytes = (sg * h.rows * tiles * 8 + 255) / 256 * 256;
    if (max_len > kFoldTiles * kManyTokens) h.sums_bytes = (sg * h.rows * 8 + 255) / 256 * 256;
    h.fits = true;
    return h;
}

template <int RP>
pa_status launch_stored(const Params& p, cudaStream_t st) {
    return pa::cuda_status(
        pa::launch_pdl(stored_kernel<RP>,
                       dim3((p.max_len + kOutTokens - 1) / kOutTokens, p.num_kv_heads, p.num_seqs),
                       dim3(256), 0, st, p),
        "accumulate_weights sum launch");
}

template <int KV, int D>
pa_status launch_typed(Params& p, const Shape& h, void* workspace, bool stored, cudaStream_t st) {
    char* const ws = static_cast<char*>(workspace);
    p.stats = reinterpret_cast<float2*>(ws);
    p.tile_tokens =
        stored ? stored_tile((int64_t)p.num_seqs * p.num_kv_heads * p.max_len) : kManyTokens;
    p.tiles = (p.max_len + p.tile_tokens - 1) / p.tile_tokens;
    if (stored) {
        p.logits = reinterpret_cast<float*>(ws + h.stats_bytes);
        p.row_pad = h.row_pad;
        const dim3 grid(p.tiles, p.num_kv_heads, p.num_seqs);
        if (pa_status s = pa::cuda_status(
                h.rows <= 8
                    ? pa::launch_pdl(logits_kernel<KV, D, 1>, grid, dim3(kWarps * 32), 0, st, p)
                    : pa::launch_pdl(logits_kernel<KV, D, 2>, grid, dim3(kWarps * 32), 0, st, p),
                "accumulate_weights logits launch"))
            return s;
        switch (p.row_pad) {
            case 2: return launch_stored<2>(p, st);
            case 4: return launch_stored<4>(p, st);
            case 8: return launch_stored<8>(p, st);
            default: return launch_stored<16>(p, st);
        }
    }
    constexpr int kTokens = kManyTokens;
    if (h.sums_bytes) p.sums = reinterpret_cast<float2*>(ws + h.stats_bytes);
    p.row_warps = 1;
    while (p.row_warps < kManyWarps && 16 * p.row_warps < h.rows) p.row_warps *= 2;
    const int tile = kTokens * KRows<KV, D>::kRowBytes, sums = 4 * p.row_warps * kTokens;
    static std::atomic<uint64_t> allowed[2]{};
    if (pa_status s = pa::allow_smem(many_kernel<KV, D, false>, tile, allowed[0],
                                     "accumulate_weights: set shared memory size"))
        return s;
    if (pa_status s = pa::allow_smem(many_kernel<KV, D, true>, tile + 4 * kManyWarps * kTokens,
                                     allowed[1], "accumulate_weights: set shared memory size"))
        return s;
    const dim3 grid(p.tiles, p.num_kv_heads, p.num_seqs), block(32 * kManyWarps);
    if (pa_status s = pa::cuda_status(
            pa::launch_pdl(many_kernel<KV, D, false>, grid, block, (size_t)tile, st, p),
            "accumulate_weights logits launch"))
        return s;
    if (p.sums)
        if (pa_status s = pa::cuda_status(
                pa::launch_pdl(rows_kernel,
                               dim3((unsigned)((h.rows + kWarps - 1) / kWarps), p.num_kv_heads,
                                    p.num_seqs),
                               dim3(kWarps * 32), 0, st, p),
                "accumulate_weights row sums launch"))
            return s;
    return pa::cuda_status(
        pa::launch_pdl(many_kernel<KV, D, true>, grid, block, (size_t)(tile + sums), st, p),
        "accumulate_weights sum launch");
}

template <int D>
pa_status launch_kv(pa_dtype kv, Params& p, const Shape& h, void* workspace, bool stored,
                    cudaStream_t st) {
    switch (kv) {
        case PA_F16: return launch_typed<PA_F16, D>(p, h, workspace, stored, st);
        case PA_BF16: return launch_typed<PA_BF16, D>(p, h, workspace, stored, st);
        case PA_INT8: return launch_typed<PA_INT8, D>(p, h, workspace, stored, st);
        case PA_INT4: return launch_typed<PA_INT4, D>(p, h, workspace, stored, st);
        default: return launch_typed<PA_FP8_E4M3, D>(p, h, workspace, stored, st);
    }
}

}  // namespace

extern "C" size_t pa_accumulate_weights_workspace_size(int32_t num_seqs, int32_t num_q_tokens,
                                                       int32_t num_heads, int32_t num_kv_heads,
                                                       int32_t head_dim, int32_t max_q_len,
                                                       int32_t max_context_len) {
    if (num_seqs <= 0 || num_q_tokens <= 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || max_q_len <= 0 || max_context_len <= 0 || num_heads % num_kv_heads != 0)
        return 0;
    const Shape h = shape_of(num_seqs, num_heads, num_kv_heads, max_q_len, max_context_len);
    return h.fits ? (size_t)h.bytes() : 0;
}

extern "C" pa_status pa_accumulate_weights(
    float* scores_out, const float* scores_in, int64_t score_stride, const void* q,
    pa_dtype q_dtype, const void* k_cache, pa_dtype kv_dtype, const float* k_scale,
    const int8_t* k_zp, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
    int32_t num_q_tokens, int32_t max_q_len, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
    int32_t max_context_len, void* workspace, size_t workspace_bytes, void* stream) {
    using pa::fail;
    if (num_seqs < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs < 0");
    if (num_seqs == 0) return PA_OK;
    if (!scores_out) return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    // the shape rules of pa_decode; K stands in for V, the scores for its output
    if (pa_status s = pa::check_decode_args(
            scores_out, PA_F32, q, q_dtype, k_cache, k_cache, kv_dtype, k_scale, k_scale, k_zp,
            k_zp, block_tables, max_blocks_per_seq, context_lens, query_start_loc, num_seqs,
            num_q_tokens, &max_q_len, num_heads, num_kv_heads, head_dim, block_size, num_blocks,
            max_context_len))
        return s;
    if (score_stride < max_context_len)
        return fail(PA_ERR_INVALID_ARG, "score_stride %lld < max_context_len %d",
                    (long long)score_stride, max_context_len);
    if (((uintptr_t)scores_in | (uintptr_t)k_scale) % 4)
        return fail(PA_ERR_INVALID_ARG, "scores and k_scale must be 4-byte aligned");
    if (kv_dtype == PA_INT4 && ((uintptr_t)k_scale | (uintptr_t)k_zp) % 16)
        return fail(PA_ERR_INVALID_ARG, "k_scale and k_zp must be 16-byte aligned");
    const Shape h = shape_of(num_seqs, num_heads, num_kv_heads, max_q_len, max_context_len);
    if (!h.fits)
        return fail(PA_ERR_UNSUPPORTED,
                    "accumulate_weights call too large (%d sequences, %d KV heads, %lld query rows "
                    "per KV head, %d tokens; at most 65535, 65535, %d and %d)",
                    num_seqs, num_kv_heads, (long long)h.rows, max_context_len, kMaxRows,
                    pa::kMaxTokens);
    const size_t need = (size_t)h.least_bytes();
    if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)
        return fail(PA_ERR_INVALID_ARG, "workspace needs %zu bytes, 256-byte aligned (got %zu)",
                    need, workspace_bytes);
    cudaStream_t st = (cudaStream_t)stream;
    if (pa::validate_enabled())
        if (pa_status s = pa::validate_score_arrays(block_tables, max_blocks_per_seq, context_lens,
                                                    query_start_loc, num_seqs, num_q_tokens,
                                                    max_q_len, num_blocks, max_context_len, st))
            return s;
    Params p{};
    p.out = scores_out;
    p.in = scores_in;
    p.q = q;
    p.k = k_cache;
    p.k_scale = k_scale;
    p.k_zp = k_zp;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.qsl = query_start_loc;
    p.err = pa::device_error_word();
    p.stride = score_stride;
    p.num_seqs = num_seqs;
    p.num_q_tokens = num_q_tokens;
    p.max_q_len = max_q_len;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.max_len = max_context_len;
    p.tokens_pad = h.tokens_pad;
    p.row_slots = (int)h.rows;
    p.q_bf16 = q_dtype == PA_BF16;
    p.scale_log2 = scale * kLog2e;
    const bool stored = (int64_t)std::min<size_t>(workspace_bytes, INT64_MAX - 1) >= h.stored_bytes();
    return head_dim == 128 ? launch_kv<128>(kv_dtype, p, h, workspace, stored, st)
                           : launch_kv<64>(kv_dtype, p, h, workspace, stored, st);
}
