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
// (the zero-point terms are taken out of the sums: z * sum_j q_ij of S, and of
// O the sum over tokens of P vs vz, one product more). A masked pair of codes IS
// an fp16 pair: a code in bits 0-3 of a half is the subnormal c * 2^-24, in bits
// 4-7 c * 2^-20, both exact, and the tensor cores multiply subnormals like any
// number; so a word of 8 codes costs one shift and four masks, and no
// conversion. The powers of two go into q, the output and the row's scale. q
// goes to fp16 after an exact power-of-two scaling per row, the V scale is
// folded into P against a running power of two per group that is no smaller
// than any V scale so far, in units of 2^-7 of it: the fp16 P is at most 2^7 times
// the softmax weight (2^8 under the lazily moved maximum), the largest power that
// stays finite, so that weights 2^-21 of the largest keep 11 bits and those of
// 2^-32 count; a new reference rescales O exactly. Products accumulate in fp32;
// the softmax maximum, sum and the scales are fp32.
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
// Work split: the balanced schedule (balanced.cuh): every warp streams its own
// share through its own stages; 8 or 16 query rows per tile, further rows as
// further chunks. Contexts of at most kWholeTokens are not cut.
//
// Measured, whole calls: 64 sequences of 512-4096 tokens, 32 query heads over 8
// (157 MB) 37.4 us, 4.2 TB/s; 4 sequences of 32768-131072 (324 MB) 64.0 us, 5.1
// TB/s, 75 % of the copy rate; a verify step of 16 to 40 rows per KV head (74 MB)
// 50.1 us. A block of 16 tokens takes 245 instructions, of which 70 mask, and the
// schedulers issue 0.57 a cycle.
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
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazyMax = 8.f;    // base-2 headroom before the running max is moved
constexpr int kPBits = 7;          // P is 2^kPBits weights: 2^(kLazyMax + kPBits) is finite in fp16
constexpr int kFoldBlocks = 64;    // blocks of a share between two folds of the zero points; 2^n
constexpr int kWholeTokens = 256;  // a warp walks them in the time of the merge's launch
// Warps of a CTA and CTAs of an SM, as many as the registers allow. One CTA of 12
// warps: its warps run at one pace, where of three CTAs of 4 the older ones ran ahead
// (a loop of 85, 98 and 113 thousand cycles for the same number of blocks) and left the
// SM to the last (68.3 us against 70.5 for the long-context step; with d = 64 28.2
// against 31.4 for a batch step, 55.2 and 56.4 for a long-context one). With 16 query rows
// two CTAs of 4 at d = 128, all that fits, where it made no such difference (55.0 us for
// the verify step, 55.8 in one CTA of 8); at d = 64 12 warps fit again (40.2 us in one CTA,
// 40.5 in three).
constexpr int ctas_per_sm(int d, int nr) { return d == 128 && nr == 2 ? 2 : 1; }
constexpr int worker_warps(int d, int nr) { return d == 128 && nr == 2 ? 4 : 12; }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "l"(policy)
                 : "memory");
}

// the same if `on` is not 0
__device__ __forceinline__ void copy16_if(uint32_t on, uint32_t dst, const void* src,
                                          uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "@p cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n\t}" ::"r"(dst),
        "l"(src), "l"(policy), "r"(on)
        : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the same on a zero accumulator
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

// The codes of a word as fp16 pairs: nibbles 0 and 4 -> n[0], 2 and 6 -> n[2] in
// units of 2^-24; 1 and 5 -> n[1], 3 and 7 -> n[3] in units of 2^-20.
constexpr float kUnit = 16777216.f;      // 2^24
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&n)[4]) {
    const uint32_t h = w >> 8;
    n[0] = w & 0x000f000fu;
    n[1] = w & 0x00f000f0u;
    n[2] = h & 0x000f000fu;
    n[3] = h & 0x00f000f0u;
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

// byte offset of 16-byte chunk `chunk` (32 codes) of token row `row` in a staged
// code tile: rows of 64 (d = 128) or 32 bytes, the chunks of a row exchanged so
// that the eight rows of an operand load fall into different banks
template <int D>
__device__ __forceinline__ uint32_t tile4_offset(int row, int chunk) {
    if constexpr (D == 128) return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
    else return row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4);
}

// Per warp: kStages stages of two blocks' (K codes, V codes), then the stages'
// scale areas, two blocks' (k scale, v scale [16][groups] fp32, k zero point, v
// zero point [16][groups]). Two blocks a stage: half the waits and issues of one.
template <int D>
struct Q4Layout {
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kGroups = D / PA_INT4_GROUP;
    static constexpr int kTile = kBS * D / 2;             // one K (or V) code tile
    static constexpr int kBlockCodes = 2 * kTile;
    static constexpr int kStage = 2 * kBlockCodes;
    static constexpr int kScaleArea = kBS * kGroups * 4;
    static constexpr int kZpArea = kBS * kGroups;
    static constexpr int kMeta = 2 * (kScaleArea + kZpArea);   // of one block
    static constexpr int kMetaAt = kStages * kStage;
    static constexpr int kWarp = kMetaAt + kStages * 2 * kMeta;
    static_assert(kTile % 512 == 0 && kMeta % 16 == 0, "alignment");
    __host__ __device__ static int header(int num_seqs) {   // cum, then chunks
        return ((num_seqs + 1) * 4 + num_seqs + 127) / 128 * 128;
    }
    __host__ __device__ static int smem_bytes(int num_seqs, int warps) {
        return header(num_seqs) + warps * kWarp;
    }
};

// share_start() in 32-bit arithmetic (B < 2^31, w <= W < 2^16): w B / W =
// w (B / W) + w (B mod W) / W; the 64-bit divisions are a quarter of a share's
// fixed cost.
__device__ __forceinline__ uint32_t share_begin(uint32_t w, uint32_t B, uint32_t W) {
    return w * (B / W) + w * (B % W) / W;
}

// The share that holds block f: the largest w with w B / W <= f, which is w B < (f + 1) W;
// an estimate in floating point, then exact steps.
__device__ __forceinline__ uint32_t share_with(uint32_t f, uint32_t B, uint32_t W) {
    const uint64_t end = ((uint64_t)f + 1) * W;
    uint32_t w = min(W - 1, (uint32_t)__fdividef(((float)f + 0.5f) * (float)W, (float)B));
    while ((uint64_t)w * B >= end) --w;
    while ((uint64_t)(w + 1) * B < end) ++w;
    return w;
}

// build_prefix() for tiles of RT rows: cum[s] = num_kv_heads * (blocks of all row chunks
// of the sequences before s), chunks[s] = row chunks of s.
template <int RT, int WARPS>
__device__ __forceinline__ void prefix_sums(int32_t* cum, uint8_t* chunks,
                                            const pa::sched::Params& p) {
    using namespace pa::sched;
    __shared__ int32_t totals[WARPS];
    pa::grid_dependents_launch();   // the merge may be scheduled early
    pa::grid_dependency_wait();     // inputs written by the previous kernel are visible
    const int n = p.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n + 32 * WARPS - 1) / (32 * WARPS);
    const int a = min(n, tid * per), b = min(n, a + per);
    int32_t own = 0;
    for (int i = a; i < b; ++i) {
        int q0;
        const int L = __ldg(p.context_lens + i), r = query_run(p.qsl, i, &q0);
        const int C = (p.group * r + RT - 1) / RT;
        int blocks = max(0, L + kBS - 1) / kBS;   // what one chunk sees: the run's last row sees all
        if (C != 1) {
            blocks = 0;
            for (int c = 0; c < C; ++c) blocks += chunk_blocks(p, L, r, 0, c);
        }
        chunks[i] = (uint8_t)C;
        cum[i] = p.num_kv_heads * blocks;
        own += p.num_kv_heads * blocks;
    }
    int32_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) totals[warp] = x;
    __syncthreads();
    const int32_t t = lane < WARPS ? totals[lane] : 0;
    int32_t run = x - own + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
    for (int i = a; i < b; ++i) {
        const int32_t v = cum[i];
        cum[i] = run;
        run += v;
    }
    if (tid == 32 * WARPS - 1) cum[n] = run;
    __syncthreads();
}

struct __align__(32) MergeRecord {
    int np;                 // pieces, in shares wid, wid + 1, ..; 0: nothing to merge
    int wid, first_slot;    // the first piece's worker and slot
    int q0, g, row0, rows;  // first query token, KV head, first query row and rows of the chunk
    int pad;
};

struct Q4Extra {
    const uint8_t* k;       // [num_blocks][num_kv_heads][16][D / 2]
    const uint8_t* v;
    const float* k_scale;   // [num_blocks][num_kv_heads][16][D / 64]
    const float* v_scale;
    const int8_t* k_zp;
    const int8_t* v_zp;
    int whole;              // a worker takes a whole segment instead of a share
    int max_chunks;
    // What the merge has to know of a cut segment, left by the worker of its first piece:
    // one per segment where there are no more segments than workers, else one per worker.
    MergeRecord* records;   // null with `whole`
    int by_segment;
};

// NR: tiles of 8 query rows (1: at most 8 rows per KV head; 2: chunks of 16)
template <typename TQ, int D, int NR>
__global__ void __launch_bounds__(worker_warps(D, NR) * 32, ctas_per_sm(D, NR))
    paged_decode_int4_kernel(const pa::sched::Params p, const Q4Extra x) {
    using namespace pa::sched;
    using Lay = Q4Layout<D>;
    constexpr int S = Lay::kStages;
    constexpr int GR = Lay::kGroups;
    constexpr int kRows = 8 * NR;
    constexpr int CH = D / 32;           // 16-byte chunks of a row: 32 dims each

    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane >> 2, qc = lane & 3;
    const int mat = lane >> 3, mrow = lane & 7;
    const int ld_tok = (mat & 1) * 8 + mrow;   // m0, m2: tokens 0-7; m1, m3: tokens 8-15
    const int ld_chk = mat >> 1;               // m0, m1: chunk 2pp; m2, m3: chunk 2pp + 1
    const int hkv = p.num_kv_heads, G = p.group, n_seqs = p.num_seqs;
    int32_t* const cum = reinterpret_cast<int32_t*>(smem);
    uint8_t* const chunks = reinterpret_cast<uint8_t*>(cum + n_seqs + 1);
    uint8_t* const mine = smem + Lay::header(n_seqs) + warp * Lay::kWarp;
    const uint32_t ring = pa::smem_addr(mine);
    const uint8_t* const meta = mine + Lay::kMetaAt;

    prefix_sums<kRows, worker_warps(D, NR)>(cum, chunks, p);
    const int64_t wid = (int64_t)blockIdx.x * worker_warps(D, NR) + warp;
    if (wid >= p.workers) return;     // the grid's last CTA may have spare warps
    if (x.records && !x.by_segment && lane == 0) x.records[wid].np = 0;
    int64_t f0, f1;
    if (x.whole) {                    // worker (s, g, c): its segment's blocks
        const int c = (uint32_t)wid % x.max_chunks, sg = (uint32_t)wid / x.max_chunks;
        const int s = sg / hkv, g = sg - s * hkv;
        if (c >= chunks[s]) return;
        int q0;
        const int r = query_run(p.qsl, s, &q0);
        const int L = __ldg(p.context_lens + s);
        f0 = cum[s] + (int64_t)g * ((cum[s + 1] - cum[s]) / hkv);
        for (int i = 0; i < c; ++i) f0 += chunk_blocks(p, L, r, 0, i);
        f1 = f0 + chunk_blocks(p, L, r, 0, c);
    } else {
        const int64_t B = cum[n_seqs], W = share_count(p, B);
        if (wid >= W) return;
        f0 = share_begin((uint32_t)wid, (uint32_t)B, (uint32_t)W);
        f1 = share_begin((uint32_t)wid + 1, (uint32_t)B, (uint32_t)W);
    }
    // the same in all lanes, which a reduction tells the compiler too
    const int n = __reduce_max_sync(0xffffffffu, (int)(f1 - f0));
    if (n <= 0) return;

    // read once, where no sequence has several row chunks; one policy a call, as its choice
    // by block took 14 of 285 instructions a block
    const uint64_t pol = x.max_chunks == 1 ? pa::policy_evict_first() : pa::policy_evict_normal();

    // each lane keeps the (block x H_kv + kv head) tile of virtual block win + lane
    int win = -32;
    uint32_t my_tile = 0;
    auto refresh = [&](int wbase) {
        win = wbase;
        const int64_t f = f0 + wbase + lane;
        my_tile = 0;
        Pos q{};
        if (f < f1) {
            q = locate(p, cum, chunks, f);
            int blk = __ldg(p.block_tables + (int64_t)q.s * p.max_blocks + q.b);
            if (blk < 0 || blk >= p.num_blocks) {
                if (p.err) atomicOr(p.err, pa::ERR_BAD_BLOCK);
                blk = 0;
            }
            my_tile = (uint32_t)(blk * hkv + q.g);
        }
        return q;
    };
    Pos cur = refresh(0);                // of block f0: lane 0's
    cur.s = __shfl_sync(0xffffffffu, cur.s, 0);
    cur.g = __shfl_sync(0xffffffffu, cur.g, 0);
    cur.c = __shfl_sync(0xffffffffu, cur.c, 0);
    cur.b = __shfl_sync(0xffffffffu, cur.b, 0);
    cur.nbs = __shfl_sync(0xffffffffu, cur.nbs, 0);
    cur.C = __shfl_sync(0xffffffffu, cur.C, 0);
    // A block is staged by 16-byte asynchronous copies, a lane each: one or two of
    // its K codes, as many of V, and one of its scales and zero points. (Bulk and
    // tensor copies take their operands from uniform registers, so six of them a
    // block cost 100 instructions where these cost 15, and issue slots are what
    // this kernel is short of.)
    const int row0 = lane / CH, chk0 = lane % CH;      // the lane's chunk of a code tile
    const uint32_t code_dst = ring + tile4_offset<D>(row0, chk0);
    constexpr int kS16 = Lay::kScaleArea / 16, kZ16 = Lay::kZpArea / 16;
    const uint8_t* const k_src = x.k + 16 * lane;
    const uint8_t* const v_src = x.v + 16 * lane;
    const uint8_t* meta_src = k_src;
    uint32_t meta_bytes = 0;                           // of a block, in the lane's array
    const uint32_t meta_dst = ring + Lay::kMetaAt + 16 * lane;
    if (lane < 2 * kS16) {
        meta_src = reinterpret_cast<const uint8_t*>(lane < kS16 ? x.k_scale : x.v_scale) +
                   16 * (lane % kS16);
        meta_bytes = Lay::kScaleArea;
    } else if (lane < 2 * (kS16 + kZ16)) {
        const int z = lane - 2 * kS16;
        meta_src = reinterpret_cast<const uint8_t*>(z < kZ16 ? x.k_zp : x.v_zp) + 16 * (z % kZ16);
        meta_bytes = Lay::kZpArea;
    }
    const int pairs = (n + 1) / 2;
    int issued = 0;                      // pairs of blocks asked for, every one a copy group
    uint32_t code_at = code_dst, meta_at = meta_dst;   // in the next pair's stage
    auto issue = [&](bool starting) {    // warp-uniform
        if (issued < pairs) {
            const int b0 = 2 * issued;
            if (!starting && b0 >= win + 32) refresh(b0 & ~31);
#pragma unroll
            for (int u = 0; u < 2; ++u) {   // a last block alone is staged twice
                const uint32_t tile = __shfl_sync(0xffffffffu, my_tile, min(b0 + u, n - 1) - win);
                const uint8_t* const k = k_src + (uint64_t)tile * Lay::kTile;
                const uint8_t* const v = v_src + (uint64_t)tile * Lay::kTile;
#pragma unroll
                for (int j = 0; j < Lay::kTile / 512; ++j) {
                    const uint32_t dst = code_at + u * Lay::kBlockCodes + 512 * j;
                    copy16(dst, k + 512 * j, pol);
                    copy16(dst + Lay::kTile, v + 512 * j, pol);
                }
                copy16_if(meta_bytes, meta_at + u * Lay::kMeta,
                          meta_src + (uint64_t)tile * meta_bytes, pol);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++issued;
        const bool wrap = code_at == code_dst + (S - 1) * Lay::kStage;
        code_at = wrap ? code_dst : code_at + Lay::kStage;
        meta_at = wrap ? meta_dst : meta_at + 2 * Lay::kMeta;
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) issue(true);

    // S^T / O^T fragments: the lane holds query rows 8 nr + 2 qc and + 1
    float o[NR][CH][2][4];               // [.][chunk][dims 4 quad + 2 j, + 1][(dim, row)]
    float oz[NR][GR][4];                 // sum of P vz: row 2 qc + e in [e], of lanes quad == 0
    float m_run[NR][2], l_run[NR][2], rowmul[NR][2];
    bool fresh = true;                   // no block of the segment done: m_run is not set yet
    float qsum[NR][GR][2];               // sum of the row's q over a group, as K products count it
    int bound[NR][2];                    // last key each row sees
    uint32_t qb[NR][CH][4];              // row 8 nr + quad, dims 32 c + 8 qc .. + 7
    float vtop[GR], vinv[GR];            // running top of the V scales, a power of two; 2^kPBits / it
    int L = 0, r = 1, q0 = 0, rows = 0, row_off = 0, seg_b0 = cur.b, last_q = 0;
    bool seg_first = true;
    // i / G for row numbers (i, G < 2^13): exact, as i times the rounding is under 2^32
    const uint32_t inv_g = 0xffffffffu / (uint32_t)G + 1u;
    auto query_of = [&](int i) { return G == 1 ? i : (int)__umulhi((uint32_t)i, inv_g); };

    // Segment start: this warp's q rows as fp16 B fragments, each row scaled
    // by 2^(14 - e_row), its dims paired as the nibbles of a K word are and the
    // odd ones, whose codes count 2^-20, by 2^-4 more.
    auto start_segment = [&](int left) {   // left: blocks of the share that are not done
        L = __ldg(p.context_lens + cur.s);
        r = query_run(p.qsl, cur.s, &q0);
        last_q = L - r;
        row_off = cur.c * kRows;
        rows = min(kRows, G * r - row_off);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = 8 * nr + quad;
            float v[CH][8];
            if (row < rows) {
                const int gr = row_off + row, qi = query_of(gr);
                const TQ* src = static_cast<const TQ*>(p.q) +
                                ((int64_t)(q0 + qi) * p.num_heads + cur.g * G + gr - qi * G) * D +
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
            const float up[2] = {exp2i(14 - ex), exp2i(10 - ex)};
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qb[nr][c][e] = pack_half2(v[c][e] * up[e & 1], v[c][e + 4] * up[e & 1]);
            // the sums over a group: the product with a K of codes 1
            float ones[GR][4];
            const uint32_t one[4] = {0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u};
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    float(&sum)[4] = ones[c * GR / CH];
                    if (e == 0 && c % (CH / GR) == 0)
                        mma_f16_first(sum, one, qb[nr][c][e], qb[nr][c][e + 1]);
                    else
                        mma_f16(sum, one, qb[nr][c][e], qb[nr][c][e + 1]);
                }
            const float mul = row < rows ? p.scale_log2 * exp2i(ex - 14) * kUnit : 0.f;
#pragma unroll
            for (int g = 0; g < GR; ++g) {
                qsum[nr][g][0] = ones[g][0], qsum[nr][g][1] = ones[g][1];
#pragma unroll
                for (int e = 0; e < 4; ++e) oz[nr][g][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rowmul[nr][e] = __shfl_sync(0xffffffffu, mul, 4 * (2 * qc + e));
                bound[nr][e] = min(last_q + query_of(row_off + 8 * nr + 2 * qc + e), L - 1);
                m_run[nr][e] = 0.f;
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
        for (int g = 0; g < GR; ++g) vtop[g] = exp2i(kPBits - 126), vinv[g] = exp2i(126);
        fresh = true;
        // the segment's merge record, by the worker that holds its first block
        if (lane == 0 && x.records && seg_b0 == 0 && cur.c < x.max_chunks) {
            const bool cut = cur.nbs > left;
            const int seg = (cur.s * hkv + cur.g) * x.max_chunks + cur.c;
            MergeRecord* const m = x.records + (x.by_segment ? seg : wid);
            if (cut) {                   // pieces up to the share of the segment's last block
                const uint32_t B = (uint32_t)cum[n_seqs], W = (uint32_t)share_count(p, B);
                const uint32_t wb = share_with((uint32_t)f1 + cur.nbs - left - 1, B, W);
                reinterpret_cast<int4*>(m)[0] =
                    make_int4((int)(wb - wid) + 1, (int)wid, seg_first ? 0 : 1, q0);
                reinterpret_cast<int4*>(m)[1] = make_int4(cur.g, row_off, rows, 0);
            } else if (x.by_segment) {
                m->np = 0;
            }
        }
    };

    // Segment end: the output rows (segment held whole) or the partial slot, whose O is the
    // average over the piece: a sum of values near the largest fp32 number would not be
    // finite. O of group g is in units of vtop[g] / 2^kPBits; vtop comes last, as neither
    // 2^24 vtop nor vtop / l need be a normal number.
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
                float z[GR];
#pragma unroll
                for (int g = 0; g < GR; ++g) z[g] = __shfl_sync(0xffffffffu, oz[nr][g][e], qc);
                const int row = 8 * nr + 2 * qc + e;
                if (row >= rows) continue;
                // a piece that the row sees nothing of (l = 0) is marked by its m, its O not read
                const float inv = __fdividef(kUnit / (1 << kPBits), l);
                int64_t obase = 0;
                if (complete) {
                    const int gr = row_off + row, qi = query_of(gr);
                    obase = ((int64_t)(q0 + qi) * p.num_heads + cur.g * G + gr - qi * G) * D;
                } else if (quad == 0) {
                    sl.m[row] = l == 0.f ? -INFINITY : m_run[nr][e];   // a row that saw nothing
                    sl.l[row] = l;
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    // dims 4 quad, + 2 count 2^-24, dims 4 quad + 1, + 3 count 2^-20
                    const float zc = z[c * GR / CH], top = vtop[c * GR / CH];
                    const float4 v = make_float4((o[nr][c][0][e] - zc) * inv * top,
                                                 fmaf(o[nr][c][0][2 + e], 0.0625f, -zc) * inv * top,
                                                 (o[nr][c][1][e] - zc) * inv * top,
                                                 fmaf(o[nr][c][1][2 + e], 0.0625f, -zc) * inv * top);
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

    // The zero points' sums taken out of O, as finish_segment does (both are linear in them).
    // The accumulators cut what they cannot hold of a product off, always downwards, and so in
    // proportion to the unsigned sum: over a share of 862 blocks even averages of either sign
    // were off by 5.6e-4 of their norm, with a fold every 64 blocks by 2.2e-4.
    auto fold_zero_points = [&]() {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int g = 0; g < GR; ++g) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float z = __shfl_sync(0xffffffffu, oz[nr][g][e], qc);
#pragma unroll
                    for (int c = g * CH / GR; c < (g + 1) * CH / GR; ++c)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            o[nr][c][j][e] -= z;
                            o[nr][c][j][2 + e] = fmaf(z, -16.f, o[nr][c][j][2 + e]);
                        }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) oz[nr][g][e] = 0.f;
            }
    };

    const uint32_t zsel = quad != 0 ? 0x4444u : GR == 2 ? 0x4240u : 0x4140u;
    // lane constants of the operand loads: a chunk further is 32 bytes in the swizzled row
    const uint32_t ld0 = tile4_offset<D>(ld_tok, ld_chk);
    int st = 0, half = 0;                // half: the stage's first block not yet done
    bool start = true;                   // (one copy of the start: it is long, and cold code)
    for (int k = 0; k < n;) {
        if (start) start_segment(n - k);
        start = false;
        if (half == 0) {                 // S groups are on their way: the oldest is here
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            __syncwarp();
        }
        // Both blocks of the stage at once; a block of another segment (or none) is masked
        // here and its segment comes back for it.
        const int take = min(2 - half, min(cur.nbs - cur.b, n - k));
        const uint32_t kb = ring + st * Lay::kStage + ld0;
        const uint8_t* const mt = meta + 2 * st * Lay::kMeta;
        const int tok0 = (cur.b - half) * kBS;   // of the stage's first block

        // scales of the lane's tokens quad and quad + 8 of each block
        float ks[2][2][GR], vs[2][2][GR];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float* ksc = reinterpret_cast<const float*>(mt + u * Lay::kMeta) + quad * GR;
            const float* vsc = ksc + kBS * GR;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (GR == 2) {
                    const float2 a = *reinterpret_cast<const float2*>(ksc + 16 * h);
                    const float2 b = *reinterpret_cast<const float2*>(vsc + 16 * h);
                    ks[u][h][0] = a.x, ks[u][h][1] = a.y, vs[u][h][0] = b.x, vs[u][h][1] = b.y;
                } else {
                    ks[u][h][0] = ksc[8 * h], vs[u][h][0] = vsc[8 * h];
                }
            }
        }

        // ---- S^T = K codes Q^T: 2 x 16 tokens x 8 NR rows, one sum per group; then
        // zero points and scales ----
        // a: logit less the running maximum, [.][.][2 h + e] of token quad + 8 h, row 2 qc + e
        float a[2][NR][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float s[NR][GR][4];
#pragma unroll
            for (int pp = 0; pp < CH / 2; ++pp) {
                uint32_t rr[4];
                pa::ldmatrix_x4((kb + u * Lay::kBlockCodes) ^ (32 * pp), rr[0], rr[1], rr[2], rr[3]);
                const int g = pp * 2 * GR / CH;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t lo[4], hi[4];
                    unpack(rr[2 * j], lo);
                    unpack(rr[2 * j + 1], hi);
                    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
                    const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        const uint32_t(&q)[4] = qb[nr][2 * pp + j];
                        if (j == 0 && (GR == CH / 2 || pp == 0))
                            mma_f16_first(s[nr][g], a0, q[0], q[1]);
                        else
                            mma_f16(s[nr][g], a0, q[0], q[1]);
                        mma_f16(s[nr][g], a1, q[2], q[3]);
                    }
                }
            }
            const uint8_t* kzp = mt + u * Lay::kMeta + 2 * Lay::kScaleArea + quad * GR;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float z[GR];
#pragma unroll
                for (int g = 0; g < GR; ++g) z[g] = (float)kzp[8 * GR * h + g];
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaf(-z[0], qsum[nr][0][e], s[nr][0][2 * h + e]) * ks[u][h][0];
                        if constexpr (GR == 2)
                            v = fmaf(fmaf(-z[1], qsum[nr][1][e], s[nr][1][2 * h + e]), ks[u][h][1],
                                     v);
                        a[u][nr][2 * h + e] = fmaf(v, rowmul[nr][e], -m_run[nr][e]);
                    }
            }
        }

        // ---- mask, online softmax (lazy max) ----
        if (take < 2 || tok0 + 2 * kBS - 1 > last_q) {   // the ends of a share or a context
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = tok0 + 16 * u + quad + 8 * h;
                    const bool here = u >= half && u < half + take;
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!here || t > bound[nr][e]) a[u][nr][2 * h + e] = -INFINITY;
                    // scales past the context may hold anything: their weights must be 0
                    if (!here || t >= L)
#pragma unroll
                        for (int g = 0; g < GR; ++g) vs[u][h][g] = 0.f;
                }
        }
        bool raise = fresh;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                raise |= fmaxf(fmaxf(a[0][nr][e], a[0][nr][2 + e]),
                               fmaxf(a[1][nr][e], a[1][nr][2 + e])) > kLazyMax;
#pragma unroll
        for (int g = 0; g < GR; ++g)
            raise |= fmaxf(fmaxf(vs[0][0][g], vs[0][1][g]), fmaxf(vs[1][0][g], vs[1][1][g])) >
                     vtop[g];
        if (__any_sync(0xffffffffu, raise)) {   // rare: a row's maximum or a V scale's top moves
            float vfix[GR];
#pragma unroll
            for (int g = 0; g < GR; ++g) {
                float mx = fmaxf(fmaxf(vs[0][0][g], vs[0][1][g]), fmaxf(vs[1][0][g], vs[1][1][g]));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float next = fmaxf(vtop[g], exp2i(ceil_log2(mx)));
                const int e = (int)(__float_as_uint(next) >> 23) - 127;   // powers of two: exact
                vinv[g] = exp2i(kPBits - e);
                vfix[g] = vtop[g] * exp2i(-e);
                vtop[g] = next;
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(fmaxf(a[0][nr][e], a[0][nr][2 + e]),
                                     fmaxf(a[1][nr][e], a[1][nr][2 + e]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    float al = 1.f;
                    if (mx > (fresh ? -INFINITY : kLazyMax)) {
                        al = fresh ? 0.f : pa::ex2(-mx);
                        m_run[nr][e] += mx;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = e; i < 4; i += 2) a[u][nr][i] -= mx;
                    }
                    l_run[nr][e] *= al;
#pragma unroll
                    for (int g = 0; g < GR; ++g) oz[nr][g][e] *= al * vfix[g];
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
            fresh = false;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t pb[NR][GR][2];      // P^T operand: tokens 2 qc, + 1 / 2 qc + 8, + 9 of row quad
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    w[e] = pa::ex2(a[u][nr][e]);
                    w[2 + e] = pa::ex2(a[u][nr][2 + e]);
                    l_run[nr][e] += w[e] + w[2 + e];
                }
#pragma unroll
                for (int g = 0; g < GR; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float m = vs[u][h][g] * vinv[g];
                        pb[nr][g][h] = movmatrix(pack_half2(w[2 * h] * m, w[2 * h + 1] * m));
                    }
            }
            // ---- O^T += V codes^T P^T, and the zero points' sums ----
            const uint32_t vb = kb + u * Lay::kBlockCodes + Lay::kTile;
#pragma unroll
            for (int pp = 0; pp < CH / 2; ++pp) {
                uint32_t rr[4];
                pa::ldmatrix_x4_trans(vb ^ (32 * pp), rr[0], rr[1], rr[2], rr[3]);
                const int g = pp * 2 * GR / CH;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t lo[4], hi[4];
                    unpack(rr[2 * j], lo);
                    unpack(rr[2 * j + 1], hi);
                    const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]};
                    const uint32_t a1[4] = {lo[2], lo[3], hi[2], hi[3]};
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        mma_f16(o[nr][2 * pp + j][0], a0, pb[nr][g][0], pb[nr][g][1]);
                        mma_f16(o[nr][2 * pp + j][1], a1, pb[nr][g][0], pb[nr][g][1]);
                    }
                }
            }
            // row 0 of a tile of its own: the zero points of tokens 2 qc, + 1 and 2 qc + 8, + 9
            const uint8_t* vzp = mt + u * Lay::kMeta + 2 * Lay::kScaleArea + Lay::kZpArea;
            uint32_t y0, y1;
            if constexpr (GR == 2) {
                y0 = reinterpret_cast<const uint32_t*>(vzp)[qc];
                y1 = reinterpret_cast<const uint32_t*>(vzp)[qc + 4];
            } else {
                y0 = reinterpret_cast<const uint16_t*>(vzp)[qc];
                y1 = reinterpret_cast<const uint16_t*>(vzp)[qc + 4];
            }
#pragma unroll
            for (int g = 0; g < GR; ++g) {
                // the two zero points' bytes into halves; all zero in the lanes of other rows
                const uint32_t sel = GR == 2 ? zsel + 0x0101u * g : zsel;
                const uint32_t az[4] = {prmt(y0, 0u, sel), 0u, prmt(y1, 0u, sel), 0u};
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    mma_f16(oz[nr][g], az, pb[nr][g][0], pb[nr][g][1]);
            }
        }
        k += take;
        half += take;
        if ((k ^ (k - take)) & kFoldBlocks) fold_zero_points();   // k passed a multiple of it
        if (half == 2) {
            __syncwarp();
            issue(false);                // into the stage just read
            half = 0;
            if (++st == S) st = 0;
        }
        cur.b += take;
        const bool seg_done = cur.b == cur.nbs;
        if (seg_done || k == n) {
            finish_segment(seg_b0 == 0 && seg_done, seg_first ? 0 : 1, min(cur.b * kBS, L));
            if (k == n) break;
            next_segment(p, cur, cum, chunks);
            seg_b0 = 0;
            seg_first = false;
            start = true;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Merges the pieces of the segments that share boundaries cut (log-sum-exp rule): the
// average of the pieces' averages O by their sums, 2^(m - M) l / den each.
// Grid: (query rows, merge records); a row is served by `wpr` of a CTA's warps,
// which take its pieces in turn and meet in shared memory. A warp asks for its
// first eight pieces' columns beside all of the row's (m, l), from which it gets
// the weights and the denominator. Bound by the latency of record, pieces and
// output in turn: the record saves every warp the arithmetic that finds a
// segment's shares (2.5, 5.1 and 1.9 us of the Llama-3-8B, verify and long-context
// steps, behind a launch of 1 us). Few long sequences are cut into a hundred pieces
// each: one warp a row waited for its loads 14 times over (14 us behind the
// long-context step), eight do twice. Merging in the decode kernel, by the last
// piece to finish, was slower (55.5 us against 48.8 for the Llama-3-8B step): equal
// shares end together, so nothing hides it, and a warp that folds all of a
// segment's rows waits longer than a grid of warps that fold one each.
constexpr int kMergeWarps = 8;
template <typename TQ, int D>
__global__ void __launch_bounds__(32 * kMergeWarps) int4_merge_kernel(const pa::sched::Params p,
                                                                      const Q4Extra x, int wpr) {
    using namespace pa::sched;
    constexpr int EPL = D / 32, kUnroll = 8;
    __shared__ __align__(16) float part[kMergeWarps][D];
    pa::grid_dependents_launch();
    pa::grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp & (wpr - 1);
    const int row = (blockIdx.x * (blockDim.x >> 5) + warp) / wpr;
    const int G = p.group, RT = p.rows_per_tile;
    const int4* const rec = reinterpret_cast<const int4*>(x.records + blockIdx.y);
    const int4 r0 = __ldcg(rec), r1 = __ldcg(rec + 1);
    bool live = true;
    if (x.by_segment) {                  // a segment without blocks leaves its record unset
        const int c = blockIdx.y % x.max_chunks, s = blockIdx.y / x.max_chunks / p.num_kv_heads;
        int q0;
        const int r = query_run(p.qsl, s, &q0), L = __ldg(p.context_lens + s);
        live = c * RT < G * r && chunk_blocks(p, L, r, 0, c) > 0;
    }
    const int np = live && row < r1.z ? r0.x : 0, wa = r0.y, first_slot = r0.z;
    if (wpr == 1 && np == 0) return;
    auto piece = [&](int i) {
        return Slot(p.slots + (2 * ((int64_t)wa + i) + (i == 0 ? first_slot : 0)) * p.slot_bytes, RT);
    };
    // a batch of this warp's pieces: m (or -inf), l and columns
    float w[kUnroll], ls[kUnroll], v[kUnroll][EPL];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int i = i0 + j * wpr;
            w[j] = -INFINITY;
            if (i >= np) continue;       // warp-uniform
            const Slot sl = piece(i);
            const float* src = sl.o + (int64_t)row * D + lane * EPL;
            if constexpr (EPL == 4) {
                const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
                v[j][0] = t.x, v[j][1] = t.y, v[j][2] = t.z, v[j][3] = t.w;
            } else {
                const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
                v[j][0] = t.x, v[j][1] = t.y;
            }
            w[j] = __ldcg(sl.m + row);   // -inf where the piece has no visible key
            ls[j] = __ldcg(sl.l + row);
        }
    };
    load(sub);                           // on the way beside the weights
    float M = -INFINITY, den = 0.f, acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
    for (int i = lane; i < np; i += 32) {
        const Slot sl = piece(i);
        const float l = __ldcg(sl.l + row), m = __ldcg(sl.m + row);
        if (m == -INFINITY && l == 0.f) continue;
        const float top = fmaxf(M, m);
        den = den * pa::ex2(M - top) + l * pa::ex2(m - top);
        M = top;
    }
    {
        float top = M;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        den *= M == -INFINITY ? 1.f : pa::ex2(M - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
        M = top;
    }
    const float inv = 1.f / den;
    for (int i0 = sub; i0 < np; i0 += kUnroll * wpr) {
        if (i0 != sub) load(i0);
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (i0 + j * wpr >= np || w[j] == -INFINITY) continue;
            const float f = pa::ex2(w[j] - M) * ls[j] * inv;
#pragma unroll
            for (int e = 0; e < EPL; ++e) acc[e] = fmaf(f, v[j][e], acc[e]);
        }
    }
    if (wpr > 1) {                       // the same for the whole grid
#pragma unroll
        for (int e = 0; e < EPL; ++e) part[warp][lane * EPL + e] = acc[e];
        __syncthreads();
        if (sub != 0 || np == 0) return;
        for (int i = 1; i < wpr; ++i)
#pragma unroll
            for (int e = 0; e < EPL; ++e) acc[e] += part[warp + i][lane * EPL + e];
    }
    if (np == 0) return;
    const int gr = r1.y + row;
    const int64_t out = ((int64_t)(r0.w + gr / G) * p.num_heads + r1.x * G + gr % G) * D + lane * EPL;
    if (p.out_f32) {
        float* dst = static_cast<float*>(p.out) + out;
        if constexpr (EPL == 4)
            *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else
            *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
        return;
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) store_out<TQ>(p.out, out + e, acc[e], 0);
}

template <typename TQ, int D, int NR>
pa_status launch_int4(const pa::DecodeArgs& a, pa::sched::Params prm, Q4Extra x) {
    using Lay = Q4Layout<D>;
    constexpr int kWorkerWarps = worker_warps(D, NR);
    auto kern = paged_decode_int4_kernel<TQ, D, NR>;
    static std::atomic<uint64_t> allowed{0};
    if (pa_status s = pa::allow_smem(kern, Lay::smem_bytes(pa::kBalancedMaxSeqs, kWorkerWarps),
                                     allowed,
                                     "int4 decode: set shared memory size"))
        return s;
    const int smem = Lay::smem_bytes(a.num_seqs, kWorkerWarps);
    // the answers of the last call's queries, which cost as much as a launch
    thread_local int last_dev = -1, last_smem = -1, sms = 0, ctas = 0;
    int dev = 0;
    if (pa_status s = pa::cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return s;
    if (dev != last_dev || smem != last_smem) {
        last_dev = -1;
        if (pa_status s = pa::cuda_status(
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count"))
            return s;
        if (pa_status s =
                pa::cuda_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                                    &ctas, kern, kWorkerWarps * 32, smem),
                                "occupancy query"))
            return s;
        last_dev = dev;
        last_smem = smem;
    }
    if (ctas < 1) return pa::fail(PA_ERR_UNSUPPORTED, "int4 decode kernel does not fit on an SM");
    const pa::BalancedShape shape = pa::balanced_shape(a.num_seqs, a.num_heads, a.num_kv_heads,
                                                       a.head_dim, a.max_q_len, a.max_context_len,
                                                       pa::kTileInt4);
    // Slots of 8 NR rows: with 8 the workspace, sized for 2048 workers' slots of 16 and
    // more rows, holds those of 16 warps on every SM.
    prm.rows_per_tile = 8 * NR;
    prm.slot_bytes = (int)pa::sched::slot_bytes(8 * NR, D);
    const int64_t rows = (int64_t)prm.group * a.max_q_len;
    const int chunks = (int)((rows + 8 * NR - 1) / (8 * NR));
    const int64_t segments = (int64_t)a.num_seqs * a.num_kv_heads * chunks;
    // Short contexts are not cut: a warp walks a segment of kWholeTokens in less than the
    // merge's launch takes.
    x.whole = a.max_context_len <= kWholeTokens;
    x.max_chunks = chunks;
    int64_t workers = segments;
    if (!x.whole) {
        workers = std::min((int64_t)ctas * sms * kWorkerWarps, shape.virtual_blocks);
        const int64_t record_bytes =
            (std::min(segments, workers) * (int64_t)sizeof(MergeRecord) + 255) / 256 * 256;
        x.records = reinterpret_cast<MergeRecord*>(prm.slots);
        prm.slots += record_bytes;
        const int64_t room = shape.workspace_bytes - shape.cum_bytes - record_bytes;
        workers = std::min(workers, room / (2 * prm.slot_bytes));
        x.by_segment = segments <= workers;
    }
    prm.workers = (int)workers;
    const int grid = (int)((workers + kWorkerWarps - 1) / kWorkerWarps);
    if (pa_status s = pa::cuda_status(
            pa::launch_pdl(kern, dim3(grid), dim3(kWorkerWarps * 32), smem, a.stream, prm, x),
            "int4 decode launch"))
        return s;
    if (x.whole) return PA_OK;
    // the workers of a segment, on average, decide how many warps share a row's merge
    const int row_slots = (int)std::min<int64_t>(8 * NR, rows);
    int wpr = 1;
    while (wpr < kMergeWarps && workers > 8 * wpr * segments) wpr *= 2;
    const int per = std::min(row_slots, kMergeWarps / wpr);   // rows of a CTA
    return pa::cuda_status(
        pa::launch_pdl(int4_merge_kernel<TQ, D>,
                       dim3((row_slots + per - 1) / per, (unsigned)std::min(segments, workers)),
                       dim3(32 * per * wpr), 0, a.stream, prm, x, wpr),
        "int4 merge launch");
}

template <typename TQ>
pa_status dispatch(const pa::DecodeArgs& a, const pa::sched::Params& b, const Q4Extra& x) {
    const bool one = (int64_t)b.group * a.max_q_len <= 8;
    if (a.head_dim == 128)
        return one ? launch_int4<TQ, 128, 1>(a, b, x)
                   : launch_int4<TQ, 128, 2>(a, b, x);
    return one ? launch_int4<TQ, 64, 1>(a, b, x)
               : launch_int4<TQ, 64, 2>(a, b, x);
}

}  // namespace

namespace pa {

pa_status launch_decode_int4(const DecodeArgs& a) {
    if (a.partition_size != 0)
        return fail(PA_ERR_UNSUPPORTED, "INT4 caches use the balanced schedule (partition_size 0)");
    // tile numbers have 31 bits; row chunks round the rows of the merge's grid up to twice
    // as many
    const int64_t segments = (int64_t)a.num_seqs * a.num_kv_heads;
    if ((int64_t)a.num_blocks * a.num_kv_heads > INT32_MAX ||
        segments * (a.num_heads / a.num_kv_heads) * a.max_q_len > 1 << 30)
        return fail(PA_ERR_UNSUPPORTED,
                    "int4 decode call too large (%d blocks x %d KV heads, %d sequences x %d heads x "
                    "%d queries; at most 2^31 - 1 and 2^30)",
                    a.num_blocks, a.num_kv_heads, a.num_seqs, a.num_heads, a.max_q_len);
    if (pa_status s = balanced_check(a)) return s;
    if (((uintptr_t)a.k_scale | (uintptr_t)a.v_scale | (uintptr_t)a.k_zp | (uintptr_t)a.v_zp) % 16)
        return fail(PA_ERR_INVALID_ARG, "scales and zero points must be 16-byte aligned");
    const BalancedShape shape = balanced_shape(a.num_seqs, a.num_heads, a.num_kv_heads,
                                               a.head_dim, a.max_q_len, a.max_context_len,
                                               kTileInt4);
    pa::sched::Params b{};
    b.out = a.out;
    b.q = a.q;
    b.block_tables = a.block_tables;
    b.context_lens = a.context_lens;
    b.qsl = a.query_start_loc;
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
    const Q4Extra x{static_cast<const uint8_t*>(a.k_cache),
                    static_cast<const uint8_t*>(a.v_cache), a.k_scale, a.v_scale, a.k_zp, a.v_zp,
                    0, 1, nullptr, 0};
    return a.q_dtype == PA_BF16 ? dispatch<__nv_bfloat16>(a, b, x)
                                : dispatch<__half>(a, b, x);
}

}  // namespace pa
