// Paged decode attention over a 4-bit cache.
//
// A row holds unsigned 4-bit codes c with one fp32 scale s and zero point z
// per group of 64 elements; a value is (c - z) * s ("LLM推理优化深度实战" §5.2
// asks for scales finer than one per tensor; the affine form is "cs336 lecture
// 10", Quantization). softmax(Q K^T / sqrt(d)) V is computed without forming
// the dequantised values. With G groups in a row,
//
//   S[i][t] = sum_g ks[t][g] * sum_{j in g} q_ij (c[t][j] - kz[t][g])
//   O[i][j] = sum_t P[i][t] vs[t][g(j)] * (c[t][j] - vz[t][g(j)])
//
// c - z is an integer in [-15, 15], exact in fp16. Two codes become an fp16
// pair with one three-input logic operation: a code in mantissa bits 0-3 of
// 1024.0 is 1024 + c, in bits 4-7 of 64.0 it is 64 + c; subtracting 1024 + z
// or 64 + z is exact. q goes to fp16 after an exact power-of-two scaling per
// row, the V scale is folded into P against a running power-of-two reference
// per group, so the fp16 P never exceeds the softmax weight (at most 2^8 under
// the lazily moved maximum) and a new reference rescales O exactly. Products
// accumulate in fp32; the softmax maximum, sum and the scales are fp32.
//
// What bounds it: a (token, kv head) costs 148 bytes at d = 128, so the
// memory system delivers one every 7 cycles of an SM, in which its 256 codes
// must be unpacked and multiplied: issue slots, not bandwidth, are the scarce
// resource. So both products run transposed, S^T = K Q^T and O^T = V^T P^T,
// with the 16 tokens (or 16 dims) in the M dimension of the warp-level product
// and 8 query rows in N: up to 8 rows per KV head cost half of the products and
// accumulators that rows in M would. The 32-bit word of a K fragment
// (ldmatrix) is 8 consecutive dims of a token; the word of a transposed V
// fragment is 4 dims of 2 tokens: every masked nibble pair is an operand
// register, with no byte shuffles. P^T gets its operand layout from movmatrix.
//
// Work split: the balanced schedule (balanced.cuh) with the per-warp layout of
// the FP8 kernel: every warp streams its own share through its own ring (code
// tiles by TMA, scales and zero points by bulk copies on the same barrier);
// 8 or 16 query rows per tile, further rows as further chunks.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "balanced.cuh"
#include "pa_internal.h"
#include "ptx.cuh"

namespace {

using pa::sched::kBS;
using pa::sched::kWorkerWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazyMax = 8.f;    // base-2 headroom before the running max is moved
constexpr int kStages = 4;
// 16 warps a SM at 128 registers a thread; the accumulators of 16 rows at d =
// 128 need more, and get 12 warps at 168
constexpr int ctas_per_sm(int d, int nr) { return d == 128 && nr == 2 ? 3 : 4; }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// transpose of an 8x8 matrix of 16-bit elements held as one pair per lane
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

constexpr uint32_t kBase1024 = 0x64006400u, kBase64 = 0x54005400u;

// The zero points of two tokens (or of one, twice), as what the biased codes
// are reduced by: fp16 pairs 1024 + z and 64 + z.
struct ZeroPair {
    uint32_t z1024, z64;
    // zz: the two zero points in the low bytes of the two halves
    __device__ __forceinline__ explicit ZeroPair(uint32_t zz)
        : z1024(zz | kBase1024), z64(zz * 16u + kBase64) {}
};

// (code - z) of the nibble pairs of a word: nibbles 0 and 4 -> n[0], 1 and 5 ->
// n[1], 2 and 6 -> n[2], 3 and 7 -> n[3]
__device__ __forceinline__ void unpack(uint32_t w, const ZeroPair& z, uint32_t (&n)[4]) {
    const uint32_t h = w >> 8;
    n[0] = hsub2((w & 0x000f000fu) | kBase1024, z.z1024);
    n[1] = hsub2((w & 0x00f000f0u) | kBase64, z.z64);
    n[2] = hsub2((h & 0x000f000fu) | kBase1024, z.z1024);
    n[3] = hsub2((h & 0x00f000f0u) | kBase64, z.z64);
}

// smallest e with 2^e >= x, for a positive finite x (x = 0 gives -126)
__device__ __forceinline__ int ceil_log2(float x) {
    const uint32_t b = __float_as_uint(x);
    const int e = (int)((b >> 23) & 0xff) - 127;
    if (e < -126) return -126;
    return (b & 0x7fffff) ? e + 1 : e;
}

__device__ __forceinline__ float exp2i(int e) {   // 2^e for e in [-126, 127]
    e = max(-126, min(127, e));
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// byte offset of 16-byte chunk `chunk` (32 codes) of token row `row` in a code
// tile as the tensor map writes it: rows of 64 bytes under the 64-byte
// swizzle (d = 128), rows of 32 bytes under the 32-byte swizzle (d = 64)
template <int D>
__device__ __forceinline__ uint32_t tile4_offset(int row, int chunk) {
    if constexpr (D == 128) return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
    else return row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4);
}

// Per warp: kStages stages of (K codes, V codes), then the stages' scale
// areas (k scale, v scale [16][groups] fp32, k zero point, v zero point
// [16][groups]), padded so the next warp's ring starts on a 1024-byte boundary.
template <int D>
struct Q4Layout {
    static constexpr int kGroups = D / PA_INT4_GROUP;
    static constexpr int kTile = kBS * D / 2;             // one K (or V) code tile
    static constexpr int kStage = 2 * kTile;
    static constexpr int kScaleArea = kBS * kGroups * 4;
    static constexpr int kZpArea = kBS * kGroups;
    static constexpr int kMeta = 2 * (kScaleArea + kZpArea);
    static constexpr int kMetaAt = kStages * kStage;
    static constexpr int kWarp = (kMetaAt + kStages * kMeta + 1023) / 1024 * 1024;
    static_assert(kStage % 512 == 0 && kMeta % 16 == 0, "swizzle and bulk copy alignment");
    __host__ __device__ static int smem_bytes(int num_seqs) {
        return pa::sched::header_bytes(num_seqs, kStages) + kWorkerWarps * kWarp + 1024;
    }
};

struct Q4Extra {
    const float* k_scale;   // [num_blocks][num_kv_heads][16][D / 64]
    const float* v_scale;
    const int8_t* k_zp;
    const int8_t* v_zp;
};

// NR: tiles of 8 query rows (1: at most 8 rows per KV head; 2: chunks of 16)
template <typename TQ, int D, int NR>
__global__ void __launch_bounds__(kWorkerWarps * 32, ctas_per_sm(D, NR))
    paged_decode_int4_kernel(const __grid_constant__ CUtensorMap tmap_k,
                             const __grid_constant__ CUtensorMap tmap_v,
                             const pa::sched::Params p, const Q4Extra x) {
    using namespace pa::sched;
    using Lay = Q4Layout<D>;
    constexpr int S = kStages;
    constexpr int GR = Lay::kGroups;
    constexpr int CH = D / 32;           // 16-byte chunks of a row: 32 dims each

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = pa::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane >> 2, qc = lane & 3;
    const int mat = lane >> 3, mrow = lane & 7;
    const int ld_tok = (mat & 1) * 8 + mrow;   // m0, m2: tokens 0-7; m1, m3: tokens 8-15
    const int ld_chk = mat >> 1;               // m0, m1: chunk 2pp; m2, m3: chunk 2pp + 1
    const int hkv = p.num_kv_heads, G = p.group, n_seqs = p.num_seqs;
    int32_t* const cum = reinterpret_cast<int32_t*>(smem + kWorkerWarps * S * 8);
    uint8_t* const chunks = reinterpret_cast<uint8_t*>(cum + n_seqs + 1);
    const uint32_t bars = base + warp * S * 8;
    const int hdr = header_bytes(n_seqs, S);
    const uint32_t ring = base + hdr + warp * Lay::kWarp;
    const uint8_t* const meta = smem + hdr + warp * Lay::kWarp + Lay::kMetaAt;

    build_prefix(cum, chunks, p);
    const int64_t B = cum[n_seqs];
    const int64_t wid = (int64_t)blockIdx.x * kWorkerWarps + warp;
    const int64_t W = share_count(p, B);
    const int64_t f0 = share_start(wid, B, W);
    const int64_t f1 = share_start(wid + 1, B, W);
    const int n = (int)(f1 - f0);
    if (lane == 0) write_merge_record(p, wid, 0, 0, 0);   // none unless set at the end
    if (wid >= W || n <= 0) return;   // the grid's last CTA may have spare warps

    uint64_t pol_once = 0, pol_again = 0;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) pa::mbar_init(bars + 8 * i, 1);
        pa::fence_barrier_init();
        pa::prefetch_tensormap(&tmap_k);
        pa::prefetch_tensormap(&tmap_v);
        pol_once = pa::policy_evict_first();
        pol_again = pa::policy_evict_normal();
    }
    __syncwarp();

    // each lane keeps the (block x H_kv + kv head) tile of virtual block
    // win + lane and whether later row chunks read that block again
    int win = -32, my_tile = 0, my_once = 1;
    auto refresh = [&](int wbase) {
        win = wbase;
        const int64_t f = f0 + wbase + lane;
        my_tile = 0;
        my_once = 1;
        if (f < f1) {
            const Pos q = locate(p, cum, chunks, f);
            int blk = __ldg(p.block_tables + (int64_t)q.s * p.max_blocks + q.b);
            if (blk < 0 || blk >= p.num_blocks) {
                if (p.err) atomicOr(p.err, pa::ERR_BAD_BLOCK);
                blk = 0;
            }
            my_tile = blk * hkv + q.g;
            my_once = q.C == 1;
        }
    };
    auto issue = [&](int k) {   // warp-uniform
        if (k >= win + 32) refresh(k & ~31);
        const int tile = __shfl_sync(0xffffffffu, my_tile, k - win);
        const int once = __shfl_sync(0xffffffffu, my_once, k - win);
        if (lane == 0) {
            const uint32_t bar = bars + 8 * (k % S);
            const uint32_t dst = ring + (k % S) * Lay::kStage;
            const uint32_t sd = ring + Lay::kMetaAt + (k % S) * Lay::kMeta;
            const uint64_t pol = once ? pol_once : pol_again;
            const int64_t row = (int64_t)tile * (kBS * GR);
            pa::mbar_arrive_expect_tx(bar, 2 * Lay::kTile + Lay::kMeta);
            pa::tma_load_2d(dst, &tmap_k, 0, tile * kBS, bar, pol);
            pa::tma_load_2d(dst + Lay::kTile, &tmap_v, 0, tile * kBS, bar, pol);
            bulk_load(sd, x.k_scale + row, Lay::kScaleArea, bar);
            bulk_load(sd + Lay::kScaleArea, x.v_scale + row, Lay::kScaleArea, bar);
            bulk_load(sd + 2 * Lay::kScaleArea, x.k_zp + row, Lay::kZpArea, bar);
            bulk_load(sd + 2 * Lay::kScaleArea + Lay::kZpArea, x.v_zp + row, Lay::kZpArea, bar);
        }
    };
    int issued = 0;
    for (; issued < S && issued < n; ++issued) issue(issued);

    Pos cur = locate(p, cum, chunks, f0);
    // S^T / O^T fragments: the lane holds query rows 8 nr + 2 qc and + 1
    float o[NR][CH][2][4];               // [.][chunk][dims 4 quad + 2 j, + 1][(dim, row)]
    float m_run[NR][2], l_run[NR][2], rowmul[NR][2];
    int bound[NR][2];                    // last key each row sees
    uint32_t qb[NR][CH][4];              // row 8 nr + quad, dims 32 c + 8 qc .. + 7
    int ev[GR];                          // log2 of the running V-scale reference
    int L = 0, r = 1, q0 = 0, rows = 0, row_off = 0, seg_b0 = cur.b, last_q = 0;
    bool seg_first = true;

    // Segment start: this warp's q rows as fp16 B fragments, each row scaled
    // by 2^(14 - e_row), its dims paired as the nibbles of a K word are.
    auto start_segment = [&]() {
        L = __ldg(p.context_lens + cur.s);
        r = query_run(p.qsl, cur.s, &q0);
        last_q = L - r;
        row_off = cur.c * kBS;
        rows = min(kBS, G * r - row_off);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = 8 * nr + quad;
            float v[CH][8];
            if (row < rows) {
                const int gr = row_off + row;
                const TQ* src = static_cast<const TQ*>(p.q) +
                                ((int64_t)(q0 + gr / G) * p.num_heads + cur.g * G + gr % G) * D +
                                8 * qc;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + 32 * c));
                    const TQ* t = reinterpret_cast<const TQ*>(&u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[c][e] = (float)t[e];
                }
            } else {
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
            }
            float mx = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[c][e]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            int ex = 0;
            if (mx > 0.f) {
                ex = (int)((__float_as_uint(mx) >> 23) & 0xff) - 127;   // floor(log2 max|q|)
                ex = max(-100, min(100, ex));
            }
            const float up = exp2i(14 - ex);
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qb[nr][c][e] = pack_half2(v[c][e] * up, v[c][e + 4] * up);
            const float mul = row < rows ? p.scale_log2 * exp2i(ex - 14) : 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rowmul[nr][e] = __shfl_sync(0xffffffffu, mul, 4 * (2 * qc + e));
                bound[nr][e] = min(last_q + (row_off + 8 * nr + 2 * qc + e) / G, L - 1);
                m_run[nr][e] = -INFINITY;
                l_run[nr][e] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nr][c][j][e] = 0.f;
        }
#pragma unroll
        for (int g = 0; g < GR; ++g) ev[g] = -126;
    };

    // Segment end: the output rows (segment held whole) or the partial slot;
    // O of group g is in units of the V-scale reference 2^ev[g].
    auto finish_segment = [&](bool complete, int slot_idx, int tok_end) {
        Slot sl(p.slots + (2 * wid + slot_idx) * (int64_t)p.slot_bytes, p.rows_per_tile);
        if (!complete && lane == 0) {
            sl.hdr[0] = cur.s;
            sl.hdr[1] = cur.g;
            sl.hdr[2] = cur.c;
            sl.hdr[3] = seg_b0 * kBS;
            sl.hdr[4] = tok_end;
        }
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_run[nr][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int row = 8 * nr + 2 * qc + e;
                if (row >= rows) continue;
                int64_t obase = 0;
                if (complete) {
                    const int gr = row_off + row;
                    obase = ((int64_t)(q0 + gr / G) * p.num_heads + cur.g * G + gr % G) * D;
                } else if (quad == 0) {
                    sl.m[row] = m_run[nr][e];
                    sl.l[row] = l;
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const float vref = exp2i(ev[c * GR / CH]);
                    const float mul = complete ? vref / l : vref;
                    const float4 v = make_float4(o[nr][c][0][e] * mul, o[nr][c][0][2 + e] * mul,
                                                 o[nr][c][1][e] * mul, o[nr][c][1][2 + e] * mul);
                    const int col = 32 * c + 4 * quad;
                    if (!complete) {
                        *reinterpret_cast<float4*>(sl.o + (int64_t)row * D + col) = v;
                    } else if (p.out_f32) {
                        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + obase + col) = v;
                    } else {
                        TQ* o16 = static_cast<TQ*>(p.out) + obase + col;
                        if constexpr (std::is_same<TQ, __half>::value) {
                            *reinterpret_cast<__half2*>(o16) = __floats2half2_rn(v.x, v.y);
                            *reinterpret_cast<__half2*>(o16 + 2) = __floats2half2_rn(v.z, v.w);
                        } else {
                            *reinterpret_cast<__nv_bfloat162*>(o16) =
                                __floats2bfloat162_rn(v.x, v.y);
                            *reinterpret_cast<__nv_bfloat162*>(o16 + 2) =
                                __floats2bfloat162_rn(v.z, v.w);
                        }
                    }
                }
            }
    };

    start_segment();
    int consumed = 0;
    for (int k = 0; k < n; ++k) {
        const int st = k % S;
        if (!pa::mbar_wait(bars + 8 * st, (k / S) & 1, p.err, pa::ERR_WAIT_FULL)) break;
        consumed = k + 1;
        const uint32_t kb = ring + st * Lay::kStage, vb = kb + Lay::kTile;
        const float* ksc = reinterpret_cast<const float*>(meta + st * Lay::kMeta);
        const float* vsc = ksc + kBS * GR;
        const uint8_t* kzp = meta + st * Lay::kMeta + 2 * Lay::kScaleArea;
        const uint8_t* vzp = kzp + Lay::kZpArea;
        const int tok0 = cur.b * kBS;

        // scales of the lane's tokens quad and quad + 8
        float ks[2][GR], vs[2][GR];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = quad + 8 * h;
            if constexpr (GR == 2) {
                const float2 a = *reinterpret_cast<const float2*>(ksc + 2 * t);
                const float2 b = *reinterpret_cast<const float2*>(vsc + 2 * t);
                ks[h][0] = a.x, ks[h][1] = a.y, vs[h][0] = b.x, vs[h][1] = b.y;
            } else {
                ks[h][0] = ksc[t], vs[h][0] = vsc[t];
            }
            // scales past the context may hold anything: their weights must be 0
            if (tok0 + t >= L)
#pragma unroll
                for (int g = 0; g < GR; ++g) vs[h][g] = 0.f;
        }

        // ---- S^T = (K codes - z) Q^T: 16 tokens x 8 NR rows, one sum per group ----
        float s[NR][GR][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int g = 0; g < GR; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nr][g][e] = 0.f;
#pragma unroll
        for (int pp = 0; pp < CH / 2; ++pp) {
            uint32_t rr[4];
            pa::ldmatrix_x4(kb + tile4_offset<D>(ld_tok, 2 * pp + ld_chk), rr[0], rr[1], rr[2],
                            rr[3]);
            const int g = pp * 2 * GR / CH;
            const ZeroPair z0(kzp[quad * GR + g] * 0x00010001u);
            const ZeroPair z1(kzp[(quad + 8) * GR + g] * 0x00010001u);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t lo[4], hi[4];
                unpack(rr[2 * j], z0, lo);
                unpack(rr[2 * j + 1], z1, hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
                const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    const uint32_t(&q)[4] = qb[nr][2 * pp + j];
                    mma_f16(s[nr][g], a0, q[0], q[1]);
                    mma_f16(s[nr][g], a1, q[2], q[3]);
                }
            }
        }

        // ---- scales, mask, online softmax (lazy max) ----
        const bool need_mask = tok0 + kBS - 1 > last_q;
        float a[NR][4];                  // [.][2 h + e]: token quad + 8 h, row 2 qc + e
        bool raise = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = s[nr][0][2 * h + e] * ks[h][0];
                    if constexpr (GR == 2) v = fmaf(s[nr][1][2 * h + e], ks[h][1], v);
                    v *= rowmul[nr][e];
                    if (need_mask && tok0 + quad + 8 * h > bound[nr][e]) v = -INFINITY;
                    a[nr][2 * h + e] = v;
                    raise |= v > m_run[nr][e] + kLazyMax;
                }
        int evn[GR];
#pragma unroll
        for (int g = 0; g < GR; ++g) {
            evn[g] = ev[g];
            raise |= fmaxf(vs[0][g], vs[1][g]) > exp2i(ev[g]);
        }
        if (__any_sync(0xffffffffu, raise)) {   // rare: a row's maximum or a V reference moves
            float vfix[GR];
#pragma unroll
            for (int g = 0; g < GR; ++g) {
                float mx = fmaxf(vs[0][g], vs[1][g]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                evn[g] = max(ev[g], ceil_log2(mx));
                vfix[g] = exp2i(ev[g] - evn[g]);
                ev[g] = evn[g];
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(a[nr][e], a[nr][2 + e]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    float al = 1.f;
                    if (mx > m_run[nr][e] + kLazyMax) {
                        al = pa::ex2(m_run[nr][e] - mx);   // 0 while m_run is -inf
                        m_run[nr][e] = mx;
                    }
                    l_run[nr][e] *= al;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const float f = al * vfix[c * GR / CH];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            o[nr][c][j][e] *= f;
                            o[nr][c][j][2 + e] *= f;
                        }
                    }
                }
        }
        float vmul[2][GR];
#pragma unroll
        for (int g = 0; g < GR; ++g) {
            const float inv = exp2i(-ev[g]);
            vmul[0][g] = vs[0][g] * inv;
            vmul[1][g] = vs[1][g] * inv;
        }
        uint32_t pb[NR][GR][2];          // P^T operand: tokens 2 qc, + 1 / 2 qc + 8, + 9 of row quad
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float m_use = m_run[nr][e] == -INFINITY ? 0.f : m_run[nr][e];
                w[e] = pa::ex2(a[nr][e] - m_use);
                w[2 + e] = pa::ex2(a[nr][2 + e] - m_use);
                l_run[nr][e] += w[e] + w[2 + e];
            }
#pragma unroll
            for (int g = 0; g < GR; ++g)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    pb[nr][g][h] = movmatrix(
                        pack_half2(w[2 * h] * vmul[h][g], w[2 * h + 1] * vmul[h][g]));
        }

        // ---- O^T += (V codes - z)^T P^T ----
#pragma unroll
        for (int pp = 0; pp < CH / 2; ++pp) {
            uint32_t rr[4];
            pa::ldmatrix_x4_trans(vb + tile4_offset<D>(ld_tok, 2 * pp + ld_chk), rr[0], rr[1],
                                  rr[2], rr[3]);
            const int g = pp * 2 * GR / CH;
            // zero points of tokens 2 qc, 2 qc + 1 and 2 qc + 8, 2 qc + 9
            uint32_t y0, y1;
            if constexpr (GR == 2) {
                y0 = reinterpret_cast<const uint32_t*>(vzp)[qc];
                y1 = reinterpret_cast<const uint32_t*>(vzp)[qc + 4];
            } else {
                y0 = reinterpret_cast<const uint16_t*>(vzp)[qc];
                y1 = reinterpret_cast<const uint16_t*>(vzp)[qc + 4];
            }
            const uint32_t sel = GR == 2 ? (g == 0 ? 0x4240u : 0x4341u) : 0x4140u;
            const ZeroPair z0(prmt(y0, 0u, sel)), z1(prmt(y1, 0u, sel));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t lo[4], hi[4];
                unpack(rr[2 * j], z0, lo);
                unpack(rr[2 * j + 1], z1, hi);
                const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]};
                const uint32_t a1[4] = {lo[2], lo[3], hi[2], hi[3]};
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    mma_f16(o[nr][2 * pp + j][0], a0, pb[nr][g][0], pb[nr][g][1]);
                    mma_f16(o[nr][2 * pp + j][1], a1, pb[nr][g][0], pb[nr][g][1]);
                }
            }
        }
        __syncwarp();
        if (issued < n) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            issue(issued);
            ++issued;
        }
        ++cur.b;
        const bool seg_done = cur.b == cur.nbs;
        if (seg_done || k == n - 1) {
            finish_segment(seg_b0 == 0 && seg_done, seg_first ? 0 : 1, min(cur.b * kBS, L));
            if (k == n - 1) {
                if (lane == 0)
                    record_last_segment(p, wid, f1, B, seg_done, seg_b0, cur.nbs - cur.b,
                                        seg_first, q0, rows);
                break;
            }
            next_segment(p, cur, cum, chunks);
            seg_b0 = 0;
            seg_first = false;
            start_segment();
        }
    }
    // drain: no copy of this warp may still be in flight when it exits
    for (int k = consumed; k < issued; ++k)
        if (!pa::mbar_wait(bars + 8 * (k % S), (k / S) & 1, p.err, pa::ERR_WAIT_DRAIN)) break;
}

template <typename TQ, int D, int NR>
pa_status launch_int4(const pa::DecodeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                      pa::sched::Params prm, const Q4Extra& x) {
    using Lay = Q4Layout<D>;
    auto kern = paged_decode_int4_kernel<TQ, D, NR>;
    static bool attr_set = false;   // per instantiation; benign race (idempotent)
    if (!attr_set) {
        if (pa_status s = pa::cuda_status(
                cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     Lay::smem_bytes(pa::kBalancedMaxSeqs)),
                "int4 decode: set shared memory size"))
            return s;
        attr_set = true;
    }
    const int smem = Lay::smem_bytes(a.num_seqs);
    int dev = 0, sms = 0, ctas = 0;
    if (pa_status s = pa::cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return s;
    if (pa_status s = pa::cuda_status(
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count"))
        return s;
    if (pa_status s = pa::cuda_status(
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kern, kWorkerWarps * 32, smem),
            "occupancy query"))
        return s;
    if (ctas < 1) return pa::fail(PA_ERR_UNSUPPORTED, "int4 decode kernel does not fit on an SM");
    const pa::BalancedShape shape = pa::balanced_shape(a.num_seqs, a.num_heads, a.num_kv_heads,
                                                       a.head_dim, a.max_q_len, a.max_context_len,
                                                       pa::kTileInt4);
    const int64_t workers =
        std::min<int64_t>((int64_t)ctas * sms * kWorkerWarps, shape.workers);
    prm.workers = (int)workers;
    const int grid = (int)((workers + kWorkerWarps - 1) / kWorkerWarps);
    if (pa_status s = pa::cuda_status(
            pa::launch_pdl(kern, dim3(grid), dim3(kWorkerWarps * 32), smem, a.stream, mk, mv, prm,
                           x),
            "int4 decode launch"))
        return s;
    const int row_slots = (int)std::min<int64_t>(kBS, (int64_t)(a.num_heads / a.num_kv_heads) *
                                                          a.max_q_len);
    return pa::cuda_status(pa::sched::launch_segment_reduce<TQ, D>(prm, (int)shape.max_chunks,
                                                                    row_slots, a.stream),
                           "segment reduce launch");
}

template <typename TQ>
pa_status dispatch(const pa::DecodeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                   const pa::sched::Params& b, const Q4Extra& x) {
    const bool one = (int64_t)b.group * a.max_q_len <= 8;
    if (a.head_dim == 128)
        return one ? launch_int4<TQ, 128, 1>(a, mk, mv, b, x)
                   : launch_int4<TQ, 128, 2>(a, mk, mv, b, x);
    return one ? launch_int4<TQ, 64, 1>(a, mk, mv, b, x)
               : launch_int4<TQ, 64, 2>(a, mk, mv, b, x);
}

}  // namespace

namespace pa {

pa_status launch_decode_int4(const DecodeArgs& a) {
    if (a.partition_size != 0)
        return fail(PA_ERR_UNSUPPORTED, "INT4 caches use the balanced schedule (partition_size 0)");
    if (pa_status s = balanced_check(a)) return s;
    if (((uintptr_t)a.k_scale | (uintptr_t)a.v_scale | (uintptr_t)a.k_zp | (uintptr_t)a.v_zp) % 16)
        return fail(PA_ERR_INVALID_ARG, "scales and zero points must be 16-byte aligned");
    const BalancedShape shape = balanced_shape(a.num_seqs, a.num_heads, a.num_kv_heads,
                                               a.head_dim, a.max_q_len, a.max_context_len,
                                               kTileInt4);
    CUtensorMap mk, mv;   // rows of head_dim / 2 bytes
    if (pa_status s =
            cache_tensor_map(&mk, a.k_cache, a.num_blocks, a.num_kv_heads, a.head_dim / 2, 1))
        return s;
    if (pa_status s =
            cache_tensor_map(&mv, a.v_cache, a.num_blocks, a.num_kv_heads, a.head_dim / 2, 1))
        return s;
    pa::sched::Params b{};
    b.out = a.out;
    b.q = a.q;
    b.block_tables = a.block_tables;
    b.context_lens = a.context_lens;
    b.qsl = a.query_start_loc;
    b.cum_out = static_cast<int32_t*>(a.slots);
    b.slots = static_cast<uint8_t*>(a.slots) + shape.cum_bytes;
    b.err = device_error_word();
    b.max_blocks = a.max_blocks_per_seq;
    b.num_heads = a.num_heads;
    b.num_kv_heads = a.num_kv_heads;
    b.group = a.num_heads / a.num_kv_heads;
    b.num_seqs = a.num_seqs;
    b.num_blocks = a.num_blocks;
    b.rows_per_tile = shape.rows_per_tile;
    b.slot_bytes = (int)shape.slot_bytes;
    b.scale_log2 = a.scale * kLog2e;
    b.out_f32 = a.out_dtype == PA_F32;
    const Q4Extra x{a.k_scale, a.v_scale, a.k_zp, a.v_zp};
    return a.q_dtype == PA_BF16 ? dispatch<__nv_bfloat16>(a, mk, mv, b, x)
                                : dispatch<__half>(a, mk, mv, b, x);
}

}  // namespace pa
