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
//      merges for itself), or from logits computed again (rows_kernel merges,
//      then again_kernel).
//
// Storing costs 8 bytes a row and token, mostly within L2; computing again costs
// a second read of K and its products. So few rows are stored (up to 16 rows
// per KV head, while the buffer stays under 256 MB), many are computed again.
//
// What bounds it: the read of K, once for few rows. K goes from global memory
// to operand registers directly: tokens stand in the M dimension of the
// warp-level product, and as the order of the dims is free (q is loaded in the
// same order), a lane's 16-byte load of its token is four operand registers
// with no staging in shared memory. Codes are made exact in fp16 as in the
// decode kernels: code - zero point (INT8, INT4), E4M3 to fp16; q goes to fp16
// after an exact power-of-two scaling per row. Sums and softmax are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "pa_internal.h"
#include "ptx.cuh"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBS = 16;                  // tokens per block
constexpr int kWarps = 4;                // warps per CTA
constexpr int kTileTokens = 512;         // tokens of a logits CTA: 8 blocks a warp
static_assert(kTileTokens / kBS / kWarps <= 32, "a lane holds a block id");
constexpr int kOutTokens = 1024;         // tokens of a stored CTA
constexpr int kAgainBlocks = 2;          // blocks of a warp of an again CTA
constexpr int kMaxRows = 4096;           // query rows per KV head: their sums fit shared memory
constexpr int64_t kMaxStored = (int64_t)256 << 20;

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
    float2* sums;             // [num_seqs x H_kv][row_slots]: see row_sum; computed again only
    unsigned int* err;
    int64_t stride;           // of in and out, per KV head
    int num_seqs, num_q_tokens, max_q_len, num_heads, num_kv_heads, group, num_blocks, max_blocks;
    int max_len, tokens_pad, tiles, row_slots, row_pad, chunks;
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

// The K operand. Per lane (quad = lane / 4, qc = lane % 4) and token half h
// (token quad + 8 h of a block): kWords 32-bit words of the token's row, loaded
// kVec words at a time; frag() makes the A registers of k-step kk, whose columns
// 2 qc, 2 qc + 1 and 2 qc + 8, 2 qc + 9 are the dims dim(kk, qc, 0 .. 3).
template <int KV, int D>
struct KRows {
    static constexpr bool k16 = KV == PA_F16 || KV == PA_BF16;
    static constexpr int kRowBytes = KV == PA_INT4 ? D / 2 : k16 ? 2 * D : D;
    static constexpr int kWords = kRowBytes / 16;
    static constexpr int kVec = KV == PA_INT4 ? 2 : 4;    // a 4-bit load stays in one group
    static constexpr int kGroups = KV == PA_INT4 ? D / PA_INT4_GROUP : 1;
    static constexpr int kSteps = D / 16;
    uint32_t w[2][kWords];
    float scale[2][kGroups];
    int zp[2][kGroups];

    __device__ __forceinline__ static int dim(int kk, int qc, int e) {
        if constexpr (k16) return 32 * (kk / 2) + 8 * qc + 4 * (kk & 1) + e;
        else if constexpr (KV == PA_INT4)      // nibble pairs (0,4), (1,5) | (2,6), (3,7)
            return 64 * (kk / 4) + 16 * qc + 8 * (kk / 2 & 1) + 2 * (kk & 1) + (e >> 1) +
                   4 * (e & 1);
        else return 64 * (kk / 4) + 16 * qc + 4 * (kk & 3) + e;
    }

    // rows `row` (token 0 of the block) + quad, + quad + 8 of the cache
    __device__ __forceinline__ void load(const Params& p, int64_t row, int quad, int qc) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t t = row + quad + 8 * h;
            const uint8_t* src = static_cast<const uint8_t*>(p.k) + t * kRowBytes;
#pragma unroll
            for (int j = 0; j < kWords / kVec; ++j) {
                if constexpr (kVec == 4) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + 64 * j + 16 * qc));
                    w[h][4 * j] = u.x, w[h][4 * j + 1] = u.y;
                    w[h][4 * j + 2] = u.z, w[h][4 * j + 3] = u.w;
                } else {
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(src + 32 * j + 8 * qc));
                    w[h][2 * j] = u.x, w[h][2 * j + 1] = u.y;
                }
            }
            if constexpr (KV == PA_INT8 || KV == PA_INT4)
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    scale[h][g] = __ldg(p.k_scale + t * kGroups + g);
                    zp[h][g] = __ldg(p.k_zp + t * kGroups + g);
                }
        }
    }

    // the pair (dims 0, 1 or 2, 3 of the step) of one token
    __device__ __forceinline__ uint32_t pair(int h, int kk, int hi) const {
        if constexpr (k16) {
            return w[h][2 * kk + hi];
        } else if constexpr (KV == PA_INT8) {
            // (code ^ 0x80) in the mantissa of 1024.0, less 1152 + zp: code - zp exactly
            const uint32_t z = prmt((uint32_t)zp[h][0] ^ 0x80u, 0x64646464u, 0x4040u);
            return hsub2(prmt(w[h][kk] ^ 0x80808080u, 0x64646464u, hi ? 0x4342u : 0x4140u), z);
        } else if constexpr (KV == PA_INT4) {
            const uint32_t z = (uint32_t)(zp[h][kk / 4] & 255) * 0x00010001u;
            const uint32_t u = kk & 1 ? w[h][kk / 2] >> 8 : w[h][kk / 2];
            return hi ? hsub2((u & 0x00f000f0u) | 0x54005400u, z * 16u + 0x54005400u)
                      : hsub2((u & 0x000f000fu) | 0x64006400u, z | 0x64006400u);
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
// row sees (-1: none).
template <int KV, int D, int NR>
struct QRows {
    using K = KRows<KV, D>;
    uint32_t b[NR][K::kSteps][2];
    float mul[NR][2];
    int bound[NR][2];

    __device__ __forceinline__ void load(const Params& p, const Seq& sq, int g, int first,
                                         int quad, int qc) {
        const int rows = p.group * sq.r;
        float head = p.scale_log2;
        if constexpr (KV == PA_FP8_E4M3) head *= __ldg(p.k_scale + g);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = first + 8 * nr + quad;
            const bool on = row < rows;
            const int64_t at = on ? ((int64_t)(sq.q0 + row / p.group) * p.num_heads +
                                     g * p.group + row % p.group) * D
                                  : 0;
            float m = on ? head : 0.f;
            if constexpr (K::k16) {
                const uint16_t* src = static_cast<const uint16_t*>(p.q) + at;
#pragma unroll
                for (int j = 0; j < K::kSteps / 2; ++j) {
                    uint4 u = make_uint4(0u, 0u, 0u, 0u);
                    if (on) u = __ldg(reinterpret_cast<const uint4*>(src + 32 * j + 8 * qc));
                    b[nr][2 * j][0] = u.x, b[nr][2 * j][1] = u.y;
                    b[nr][2 * j + 1][0] = u.z, b[nr][2 * j + 1][1] = u.w;
                }
            } else {
                // two rounds over the row: its largest element, then fp16 after scaling
                // that into [2^14, 2^15)
                const uint16_t* src = static_cast<const uint16_t*>(p.q) + at;
                auto element = [&](int kk, int e) {
                    const uint16_t u = on ? __ldg(src + K::dim(kk, qc, e)) : (uint16_t)0;
                    return p.q_bf16 ? __uint_as_float((uint32_t)u << 16)
                                    : __half2float(__ushort_as_half(u));
                };
                float mx = 0.f;
#pragma unroll
                for (int kk = 0; kk < K::kSteps; ++kk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(element(kk, e)));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                int ex = 0;
                if (mx > 0.f) {
                    ex = (int)((__float_as_uint(mx) >> 23) & 0xff) - 127;
                    ex = max(-100, min(100, ex));
                }
                const float up = exp2i(14 - ex);
                m *= exp2i(ex - 14);
#pragma unroll
                for (int kk = 0; kk < K::kSteps; ++kk)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const __half2 v = __floats2half2_rn(element(kk, 2 * e) * up,
                                                            element(kk, 2 * e + 1) * up);
                        b[nr][kk][e] = *reinterpret_cast<const uint32_t*>(&v);
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mul[nr][e] = __shfl_sync(0xffffffffu, m, 4 * (2 * qc + e));
                const int mine = first + 8 * nr + 2 * qc + e;
                bound[nr][e] = mine < rows ? min(sq.L - sq.r + mine / p.group, sq.L - 1) : -1;
            }
        }
    }

    // logits (base-2 units) of the block whose first token is tok0: a[nr][2 h + e] of
    // token quad + 8 h and row 8 nr + 2 qc + e; -inf where the row does not see it
    __device__ __forceinline__ void logits(const K& k, int tok0, int quad,
                                           float (&a)[NR][4]) const {
        float s[NR][K::kGroups][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int g = 0; g < K::kGroups; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nr][g][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < K::kSteps; ++kk) {
            uint32_t f[4];
            k.frag(kk, f);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
                pa::mma_16816<KV == PA_BF16>(s[nr][kk * K::kGroups / K::kSteps], f, b[nr][kk][0],
                                             b[nr][kk][1]);
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = s[nr][0][2 * h + e];
                    if constexpr (KV == PA_INT8 || KV == PA_INT4) v *= k.scale[h][0];
                    if constexpr (K::kGroups == 2) v = fmaf(s[nr][1][2 * h + e], k.scale[h][1], v);
                    v *= mul[nr][e];
                    if (tok0 + quad + 8 * h > bound[nr][e]) v = -INFINITY;
                    a[nr][2 * h + e] = v;
                }
    }
};

__device__ __forceinline__ int block_of(const Params& p, int s, int i) {
    const int blk = __ldg(p.block_tables + (int64_t)s * p.max_blocks + i);
    if (blk >= 0 && blk < p.num_blocks) return blk;
    if (p.err) atomicOr(p.err, pa::ERR_BAD_BLOCK);
    return 0;
}

// (m, l) of a pair of partial sums
__device__ __forceinline__ void merge(float& m, float& l, float m2, float l2) {
    const float top = fmaxf(m, m2);
    const float ref = top == -INFINITY ? 0.f : top;
    l = l * pa::ex2(m - ref) + l2 * pa::ex2(m2 - ref);
    m = top;
}

// Grid: (tiles of kTileTokens tokens, KV head x chunk of 8 NR rows, sequence).
template <int KV, int D, int NR>
__global__ void __launch_bounds__(kWarps * 32) logits_kernel(const Params p) {
    __shared__ float2 part[kWarps][8 * NR];
    pa::grid_dependents_launch();
    pa::grid_dependency_wait();
    const int s = blockIdx.z, g = blockIdx.y / p.chunks, c = blockIdx.y % p.chunks;
    const int tile = blockIdx.x, first = 8 * NR * c;
    const Seq sq(p, s);
    const int rows = p.group * sq.r;
    if (tile * kTileTokens >= sq.L || first >= rows) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, qc = lane & 3;
    // this warp's blocks: b0 + warp, + kWarps, ...
    const int b0 = tile * (kTileTokens / kBS) + warp;
    const int nb = min((sq.L + kBS - 1) / kBS, (tile + 1) * (kTileTokens / kBS));
    const int n = b0 < nb ? (nb - b0 + kWarps - 1) / kWarps : 0;
    int my_block = 0;
    if (lane < n) my_block = block_of(p, s, b0 + lane * kWarps);
    QRows<KV, D, NR> q;
    q.load(p, sq, g, first, quad, qc);
    float m[NR][2], l[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) m[nr][e] = -INFINITY, l[nr][e] = 0.f;
    auto fetch = [&](KRows<KV, D>& k, int i) {
        const int64_t blk = __shfl_sync(0xffffffffu, my_block, i);
        k.load(p, (blk * p.num_kv_heads + g) * kBS, quad, qc);
    };
    auto consume = [&](const KRows<KV, D>& k, int i) {
        const int tok0 = (b0 + i * kWarps) * kBS;
        float a[NR][4];
        q.logits(k, tok0, quad, a);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            if (p.logits) {   // stored calls have one chunk
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 8 * nr + 2 * qc;
                    float* dst = p.logits + ((int64_t)(s * p.num_kv_heads + g) * p.tokens_pad +
                                             tok0 + quad + 8 * h) * p.row_pad + row;
                    if (row + 1 < p.row_pad)
                        *reinterpret_cast<float2*>(dst) = make_float2(a[nr][2 * h],
                                                                      a[nr][2 * h + 1]);
                    else if (row < p.row_pad)
                        *dst = a[nr][2 * h];
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // the lane's own running sum: merged at the end
                const float mx = fmaxf(a[nr][e], a[nr][2 + e]);
                if (mx > m[nr][e]) {
                    l[nr][e] *= pa::ex2(m[nr][e] - mx);
                    m[nr][e] = mx;
                }
                const float ref = m[nr][e] == -INFINITY ? 0.f : m[nr][e];
                l[nr][e] += pa::ex2(a[nr][e] - ref) + pa::ex2(a[nr][2 + e] - ref);
            }
        }
    };
    KRows<KV, D> k0, k1;   // the next block's rows are on their way while one is multiplied
    if (n > 0) fetch(k0, 0);
    for (int i = 0; i < n; i += 2) {
        if (i + 1 < n) fetch(k1, i + 1);
        consume(k0, i);
        if (i + 1 == n) break;
        if (i + 2 < n) fetch(k0, i + 2);
        consume(k1, i + 1);
    }
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
                merge(m[nr][e], l[nr][e], __shfl_xor_sync(0xffffffffu, m[nr][e], off),
                      __shfl_xor_sync(0xffffffffu, l[nr][e], off));
            if (quad == 0) part[warp][8 * nr + 2 * qc + e] = make_float2(m[nr][e], l[nr][e]);
        }
    __syncthreads();
    const int row = threadIdx.x;
    if (row < min(8 * NR, rows - first)) {
        float2 t = part[0][row];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) merge(t.x, t.y, part[w][row].x, part[w][row].y);
        p.stats[((int64_t)(s * p.num_kv_heads + g) * p.row_slots + first + row) * p.tiles + tile] =
            t;
    }
}

// What turns a row's logit a into its weight 2^(a - ref) * inv, from the (m, l)
// of its tiles, by one warp: ref = m and inv = 1 / l, or 0 and 0 for a row that
// saw nothing.
__device__ __forceinline__ float2 row_sum(const Params& p, const Seq& sq, int64_t sg, int row,
                                          int lane) {
    const int tiles = (sq.L + kTileTokens - 1) / kTileTokens;
    const float2* src = p.stats + (sg * p.row_slots + row) * p.tiles;
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < tiles; i += 32) {
        const float2 t = __ldg(src + i);
        merge(m, l, t.x, t.y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        merge(m, l, __shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, l, off));
    return make_float2(m == -INFINITY ? 0.f : m, l == 0.f ? 0.f : 1.f / l);
}

// Grid: (rows / kWarps, KV head, sequence): a warp a row, for again_kernel.
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const Params p) {
    pa::grid_dependents_launch();
    pa::grid_dependency_wait();
    const int s = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 31;
    const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const Seq sq(p, s);
    if (row >= p.group * sq.r) return;
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const float2 t = row_sum(p, sq, sg, row, lane);
    if (lane == 0) p.sums[sg * p.row_slots + row] = t;
}

// Grid: (tiles of kOutTokens tokens, KV head, sequence). RP: the rows a token
// has in the stored logits.
template <int RP>
__global__ void __launch_bounds__(256) stored_kernel(const Params p) {
    __shared__ float2 sum[RP];
    pa::grid_dependency_wait();
    const int s = blockIdx.z, g = blockIdx.y;
    const Seq sq(p, s);
    const int t0 = blockIdx.x * kOutTokens;
    if (t0 >= sq.L) return;
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const int rows = p.group * sq.r;
    for (int row = threadIdx.x >> 5; row < min(rows, RP); row += 8) {
        const float2 t = row_sum(p, sq, sg, row, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0) sum[row] = t;
    }
    __syncthreads();
    const int64_t base = sg * p.stride;
    for (int t = t0 + threadIdx.x; t < min(sq.L, t0 + kOutTokens); t += 256) {
        float w = 0.f;
        if (rows > 0) {
            const float* src = p.logits + (sg * p.tokens_pad + t) * RP;
            float a[RP];
            if constexpr (RP >= 4) {
#pragma unroll
                for (int i = 0; i < RP / 4; ++i)
                    *reinterpret_cast<float4*>(a + 4 * i) =
                        __ldg(reinterpret_cast<const float4*>(src) + i);
            } else {
#pragma unroll
                for (int i = 0; i < RP; ++i) a[i] = __ldg(src + i);
            }
#pragma unroll
            for (int i = 0; i < RP; ++i)
                if (i < rows) w = fmaf(pa::ex2(a[i] - sum[i].x), sum[i].y, w);
        }
        p.out[base + t] = (p.in ? p.in[base + t] : 0.f) + w;
    }
}

// Grid: (tiles of kWarps x kAgainBlocks blocks, KV head, sequence); shared
// memory: the rows' sums.
template <int KV, int D>
__global__ void __launch_bounds__(kWarps * 32) again_kernel(const Params p) {
    constexpr int NR = 2;
    extern __shared__ float2 sum[];
    pa::grid_dependency_wait();
    const int s = blockIdx.z, g = blockIdx.y;
    const Seq sq(p, s);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, qc = lane & 3;
    const int t0 = blockIdx.x * kWarps * kAgainBlocks * kBS;
    if (t0 >= sq.L) return;
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const int rows = p.group * sq.r;
    for (int i = threadIdx.x; i < (rows + 15) / 16 * 16; i += kWarps * 32)
        sum[i] = i < rows ? __ldg(p.sums + sg * p.row_slots + i) : make_float2(0.f, 0.f);
    __syncthreads();
    KRows<KV, D> k[kAgainBlocks];
    float w[kAgainBlocks][2];
    int tok0[kAgainBlocks];
#pragma unroll
    for (int i = 0; i < kAgainBlocks; ++i) {
        w[i][0] = w[i][1] = 0.f;
        tok0[i] = t0 + (warp * kAgainBlocks + i) * kBS;
        if (tok0[i] < sq.L)
            k[i].load(p, ((int64_t)block_of(p, s, tok0[i] / kBS) * p.num_kv_heads + g) * kBS, quad,
                      qc);
    }
    for (int first = 0; first < rows; first += 8 * NR) {
        QRows<KV, D, NR> q;
        q.load(p, sq, g, first, quad, qc);
#pragma unroll
        for (int i = 0; i < kAgainBlocks; ++i) {
            if (tok0[i] >= sq.L) continue;   // warp-uniform
            float a[NR][4];
            q.logits(k[i], tok0[i], quad, a);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 x = sum[first + 8 * nr + 2 * qc + e];
                    w[i][0] = fmaf(pa::ex2(a[nr][e] - x.x), x.y, w[i][0]);
                    w[i][1] = fmaf(pa::ex2(a[nr][2 + e] - x.x), x.y, w[i][1]);
                }
        }
    }
    const int64_t base = sg * p.stride;
#pragma unroll
    for (int i = 0; i < kAgainBlocks; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x = w[i][h];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            const int t = tok0[i] + quad + 8 * h;
            if (qc == 0 && t < sq.L) p.out[base + t] = (p.in ? p.in[base + t] : 0.f) + x;
        }
}

struct Shape {
    int64_t rows;         // most query rows per KV head
    int nr, chunks, row_slots, row_pad, tiles, tokens_pad;
    int64_t stats_bytes, sums_bytes, logits_bytes;   // logits 0: computed again
};

Shape shape_of(int num_seqs, int num_heads, int num_kv_heads, int max_q_len, int max_len) {
    Shape h{};
    h.rows = (int64_t)(num_heads / num_kv_heads) * max_q_len;
    h.nr = h.rows <= 8 ? 1 : 2;
    h.chunks = (int)((h.rows + 8 * h.nr - 1) / (8 * h.nr));
    h.row_slots = (int)h.rows;
    h.tiles = (max_len + kTileTokens - 1) / kTileTokens;
    h.tokens_pad = (max_len + kBS - 1) / kBS * kBS;
    const int64_t sg = (int64_t)num_seqs * num_kv_heads;
    h.stats_bytes = (sg * h.rows * h.tiles * 8 + 255) / 256 * 256;
    if (h.rows <= 16) {
        h.row_pad = 1;
        while (h.row_pad < h.rows) h.row_pad *= 2;
        h.logits_bytes = sg * h.tokens_pad * h.row_pad * 4;
        if (h.logits_bytes > kMaxStored) h.logits_bytes = 0;
    }
    if (!h.logits_bytes) h.sums_bytes = (sg * h.rows * 8 + 255) / 256 * 256;
    return h;
}

template <int KV, int D, int NR>
pa_status launch_logits(const Params& p, cudaStream_t st) {
    return pa::cuda_status(
        pa::launch_pdl(logits_kernel<KV, D, NR>,
                       dim3(p.tiles, p.num_kv_heads * p.chunks, p.num_seqs), dim3(kWarps * 32), 0,
                       st, p),
        "accumulate_weights logits launch");
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
pa_status launch_typed(const Params& p, int nr, int64_t rows, cudaStream_t st) {
    if (pa_status s = nr == 1 ? launch_logits<KV, D, 1>(p, st) : launch_logits<KV, D, 2>(p, st))
        return s;
    if (p.logits) {
        switch (p.row_pad) {
            case 1: return launch_stored<1>(p, st);
            case 2: return launch_stored<2>(p, st);
            case 4: return launch_stored<4>(p, st);
            case 8: return launch_stored<8>(p, st);
            default: return launch_stored<16>(p, st);
        }
    }
    if (pa_status s = pa::cuda_status(
            pa::launch_pdl(rows_kernel,
                           dim3((unsigned)((rows + kWarps - 1) / kWarps), p.num_kv_heads,
                                p.num_seqs),
                           dim3(kWarps * 32), 0, st, p),
            "accumulate_weights row sums launch"))
        return s;
    const int tokens = kWarps * kAgainBlocks * kBS;
    return pa::cuda_status(
        pa::launch_pdl(again_kernel<KV, D>,
                       dim3((p.max_len + tokens - 1) / tokens, p.num_kv_heads, p.num_seqs),
                       dim3(kWarps * 32), (size_t)((rows + 15) / 16 * 16 * 8), st, p),
        "accumulate_weights sum launch");
}

template <int D>
pa_status launch_kv(pa_dtype kv, const Params& p, int nr, int64_t rows, cudaStream_t st) {
    switch (kv) {
        case PA_F16: return launch_typed<PA_F16, D>(p, nr, rows, st);
        case PA_BF16: return launch_typed<PA_BF16, D>(p, nr, rows, st);
        case PA_INT8: return launch_typed<PA_INT8, D>(p, nr, rows, st);
        case PA_INT4: return launch_typed<PA_INT4, D>(p, nr, rows, st);
        default: return launch_typed<PA_FP8_E4M3, D>(p, nr, rows, st);
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
    return (size_t)(h.stats_bytes + h.sums_bytes + h.logits_bytes);
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
    const Shape h = shape_of(num_seqs, num_heads, num_kv_heads, max_q_len, max_context_len);
    if (num_seqs > 65535 || (int64_t)num_kv_heads * h.chunks > 65535 || h.rows > kMaxRows)
        return fail(PA_ERR_UNSUPPORTED,
                    "accumulate_weights call too large (%d sequences, %d KV heads, %lld query rows "
                    "per KV head; at most 65535, and %d rows)",
                    num_seqs, num_kv_heads, (long long)h.rows, kMaxRows);
    const size_t need = (size_t)(h.stats_bytes + h.sums_bytes + h.logits_bytes);
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
    p.stats = static_cast<float2*>(workspace);
    char* const after = static_cast<char*>(workspace) + h.stats_bytes;
    if (h.logits_bytes) p.logits = reinterpret_cast<float*>(after);
    else p.sums = reinterpret_cast<float2*>(after);
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
    p.tiles = h.tiles;
    p.row_slots = h.row_slots;
    p.row_pad = h.row_pad;
    p.chunks = h.chunks;
    p.q_bf16 = q_dtype == PA_BF16;
    p.scale_log2 = scale * kLog2e;
    return head_dim == 128 ? launch_kv<128>(kv_dtype, p, h.nr, h.rows, st)
                           : launch_kv<64>(kv_dtype, p, h.nr, h.rows, st);
}
