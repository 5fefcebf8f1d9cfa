// Eviction from the cache by accumulated attention weight: which tokens a
// budget keeps (pa_evict_select), and the row moves that close the holes
// (pa_move_tokens).
//
// For one sequence and KV head with L tokens, scores w and a budget n, the kept
// tokens are the protected ones (the first `sinks` and the last `recent`
// positions of the text) and then those of the largest score, equal ones in slot
// order. The slots 0 .. n - 1 are what remains: the i-th slot below n whose
// token is evicted takes the i-th kept token from above n. Attention does not
// depend on the order of the keys, so closing the holes is enough: a kept token
// below n stays where it is, each other one is read and written once, sources
// and destinations never meet, and every move can run at the same time. Moving
// the tokens up in order would instead rewrite everything behind the first hole.
// The price is that a slot no longer says where in the text its token stands;
// the positions array does.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "pa_internal.h"
#include "ptx.cuh"

namespace {

constexpr int kBS = 16;   // tokens per block

struct SelectParams {
    int2* moves;              // [num_seqs x H_kv][max_moves]: (source slot, destination slot)
    int32_t* move_counts;     // [num_seqs x H_kv]
    float* scores_out;
    int32_t* positions_out;
    const float* scores;
    const int32_t* positions; // may be null: every token in text order
    const int32_t* context_lens;
    const int32_t* new_lens;
    const int32_t* total_lens; // may be null: context_lens
    int64_t stride;
    int max_moves, num_kv_heads, max_len, sinks, recent;
};

// Scores as unsigned keys in their order: NaN lowest, -0 as +0, a protected
// token above every score.
constexpr uint32_t kProtected = 0xffffffffu;
__device__ __forceinline__ uint32_t score_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);   // -0 + 0 = +0
    if (w != w) return 0;
    return u >> 31 ? ~u : u | 0x80000000u;
}

// One row of scores: token j's position in the text and its key.
struct Row {
    const float* w;
    const int32_t* pos;
    int L, sinks, first_recent, shift;   // shift: text position of slot 0 where tokens are in order
    __device__ __forceinline__ int position(int j) const {
        const int q = pos ? pos[j] : -1;
        return q >= 0 ? q : shift + j;
    }
    __device__ __forceinline__ uint32_t key(int q, float x) const {
        return q < sinks || q >= first_recent ? kProtected : score_key(x);
    }
};

// Radix digits of a key, highest first: 11, 11 and 10 bits.
constexpr int kDigits = 3;
constexpr int kBins = 2048;
__device__ __forceinline__ int digit_shift(int d) { return d == 0 ? 21 : d == 1 ? 10 : 0; }
__device__ __forceinline__ int digit_bits(int d) { return d == 2 ? 10 : 11; }

constexpr int kMaxCluster = 8;
// shared memory of a CTA: one histogram a digit, then the keys of its slots
constexpr int kHistBytes = kDigits * kBins * 4;
constexpr int kMaxKeys = (200 * 1024 - kHistBytes) / 4;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of the cluster has arrived, and what each wrote before (shared or
// global memory) is visible to all.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the address of this CTA's shared variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(pa::smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t load_remote1(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 load_remote(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Four consecutive slots of a lane: `slots` of them are inside the row.
__device__ __forceinline__ void load4(const float* w, float (&v)[4], int j, int slots, bool aligned) {
    if (aligned && slots >= 4) {
        const float4 t = *reinterpret_cast<const float4*>(w + j);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < slots ? w[j + i] : 0.f;
    }
}
__device__ __forceinline__ void load4(const int32_t* p, int (&v)[4], int j, int slots, bool aligned) {
    if (aligned && slots >= 4) {
        const int4 t = *reinterpret_cast<const int4*>(p + j);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < slots ? p[j + i] : 0;
    }
}

// Of four bits a lane: how many are set in the lanes below, and in all of them.
__device__ __forceinline__ int before_lane(uint32_t bits, int lane, int& total) {
    int below = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t m = __ballot_sync(0xffffffffu, bits >> i & 1u);
        below += __popc(m & ((1u << lane) - 1u));
        total += __popc(m);
    }
    return below;
}

// A cluster of CTAs a (KV head, sequence), each CTA a contiguous part of the row
// (CL CTAs; 1: no cluster), each warp a contiguous range of that in pieces of 128
// slots, four a lane. One pass over scores and positions leaves keys in shared
// memory (KEYS; computed again from the scores when a part is too long for that).
// Then the n-th largest key by three radix steps, a walk that counts and one that
// emits the moves, ranks by a scan over the lanes, so that the lists come out in
// slot order. Bound by latency for short rows (barriers, the one read) and by
// issue slots for long ones: keys are read four at a time, the counting walk
// counts in registers, and the scan is one for 128 slots. A walk of 32 slots at a
// time with ballots took 43 us for 131072 tokens of 8 heads on 64 SMs, 274
// instructions for 32 slots, where pieces of 128 take 28 us; clusters of 16 took 85
// us, their barriers and remote reads outweigh the halved parts. Digits are 11 bits:
// the first holds the exponent and two more bits, so that like-sized scores spread over the
// histogram. Protected keys are above every score, so a first digit that falls on
// theirs ends the search.
template <int CL, int T, bool KEYS>   // CTAs a row, threads a CTA
__global__ void __launch_bounds__(T) evict_select_kernel(const SelectParams p) {
    constexpr int kWarps = T / 32, kPiece = 128;
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t* const hist = smem;                       // [kDigits][kBins]
    uint32_t* const keys = smem + kDigits * kBins;
    __shared__ __align__(16) int warp_counts[kWarps][4];   // gt, eq, gt below n, eq below n
    __shared__ __align__(16) int cta_counts[4];
    __shared__ uint32_t chunk_sums[kDigits][kBins / 128];
    __shared__ uint4 search_s[kDigits];
    const int s = blockIdx.z, g = blockIdx.y, part = CL == 1 ? 0 : (int)cluster_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pa::grid_dependents_launch();
    for (int i = tid; i < kDigits * kBins / 4; i += T)
        reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    pa::grid_dependency_wait();
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const int L = max(0, min(__ldg(p.context_lens + s), p.max_len));
    const int asked = __ldg(p.new_lens + s);
    const int n = asked < 0 ? L : min(asked, L);
    const int total = p.total_lens ? __ldg(p.total_lens + s) : L;
    const Row row{p.scores + sg * p.stride, p.positions ? p.positions + sg * p.stride : nullptr, L,
                  p.sinks, total - p.recent, total - L};
    float* const w_out = p.scores_out + sg * p.stride;
    int32_t* const pos_out = p.positions_out + sg * p.stride;
    int2* const moves = p.moves + sg * p.max_moves;
    const bool aligned =
        (((uintptr_t)row.w | (uintptr_t)row.pos | (uintptr_t)w_out | (uintptr_t)pos_out) & 15) == 0;
    // this CTA's slots, and this warp's of them: whole pieces, but for the row's last
    const int per = ((L + CL - 1) / CL + kPiece - 1) / kPiece * kPiece;
    const int a0 = min(L, part * per), a1 = min(L, a0 + per);
    const int seg = ((a1 - a0 + kWarps - 1) / kWarps + kPiece - 1) / kPiece * kPiece;
    const int j0 = min(a1, a0 + warp * seg), j1 = min(a1, j0 + seg);
    // scores and positions of slots j .. j + 3
    auto read4 = [&](int j, float (&w)[4], int (&pos)[4]) {
        load4(row.w, w, j, j1 - j, aligned);
        if (row.pos) load4(row.pos, pos, j, j1 - j, aligned);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pos[i] = row.pos && pos[i] >= 0 ? pos[i] : row.shift + j + i;
    };
    // their keys; 0 past the row
    auto keys4 = [&](int j, uint32_t (&k)[4]) {
        if constexpr (KEYS) {
            const uint4 t = *reinterpret_cast<const uint4*>(keys + (j - a0));
            k[0] = t.x, k[1] = t.y, k[2] = t.z, k[3] = t.w;
        } else {
            float w[4];
            int pos[4];
            read4(j, w, pos);
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = j + i < j1 ? row.key(pos[i], w[i]) : 0u;
        }
    };
    auto sync = [&]() {
        if constexpr (CL == 1) __syncthreads();
        else cluster_sync();
    };

    // key of the n-th token in the order, and how many tokens with that key stay
    uint32_t cut = 0, left = (uint32_t)n;
    const bool search = n > 0 && n < L;
    __syncthreads();                                   // the histograms are zero
#pragma unroll 4
    for (int b = j0; b < j1; b += kPiece) {            // warp-uniform
        const int j = b + 4 * lane;
        float w[4];
        int pos[4];
        read4(j, w, pos);
        uint32_t k[4], top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[i] = j + i < j1 ? row.key(pos[i], w[i]) : 0u;
            top = max(top, k[i]);
        }
        if (b + kPiece <= j1 && !__any_sync(0xffffffffu, top == kProtected)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) atomicAdd(hist + (k[i] >> 21), 1u);
        } else {                         // protected tokens come in runs: one addition a warp
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t safe = __ballot_sync(0xffffffffu, k[i] == kProtected);
                if (j + i < j1 && (k[i] != kProtected || lane == __ffs(safe) - 1))
                    atomicAdd(hist + (k[i] >> 21),
                              k[i] == kProtected ? (uint32_t)__popc(safe) : 1u);
            }
        }
        if (KEYS) *reinterpret_cast<uint4*>(keys + (j - a0)) = make_uint4(k[0], k[1], k[2], k[3]);
    }
    if (search) {
#pragma unroll 1
        for (int d = 0; d < kDigits; ++d) {
            uint32_t* const h = hist + d * kBins;
            const int shift = digit_shift(d), bins = 1 << digit_bits(d);
            if (d > 0) {
                const uint32_t mask = 0xffffffffu << (shift + digit_bits(d));
                for (int b = j0; b < j1; b += kPiece) {
                    const int j = b + 4 * lane;
                    uint32_t k[4];
                    keys4(j, k);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((k[i] & mask) == cut && j + i < j1)
                            atomicAdd(h + (k[i] >> shift & (bins - 1)), 1u);
                }
            }
            __syncthreads();
            // a warp sums a chunk of 128 bins (chunk 0 the highest); then the n-th key's chunk is
            // found from the chunks' sums, and its bin from that chunk's bins, by one warp, which
            // in a cluster reads both from all CTAs (the whole histograms would be 16 times as
            // much)
            const int chunks = bins / 128;
            for (int i = warp; i < chunks; i += kWarps) {
                const uint4 v = *reinterpret_cast<const uint4*>(h + bins - 128 * (i + 1) + 4 * lane);
                const uint32_t sum = __reduce_add_sync(0xffffffffu, v.x + v.y + v.z + v.w);
                if (lane == 0) chunk_sums[d][i] = sum;
            }
            sync();
            uint32_t bin = 0, above = 0, in_bin = 0;   // the bin, keys in higher ones, and in it
            if (warp == 0) {
                uint32_t upto = 0;
                if (lane < chunks) {
                    if constexpr (CL == 1) {
                        upto = chunk_sums[d][lane];
                    } else {
#pragma unroll
                        for (int c = 0; c < CL; ++c)
                            upto += load_remote1(remote(&chunk_sums[d][lane], c));
                    }
                }
                const uint32_t own = upto;
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                const int chunk =
                    __ffs(__ballot_sync(0xffffffffu, lane < chunks && upto >= left)) - 1;
                above = __shfl_sync(0xffffffffu, upto - own, chunk);
                const int top = bins - 128 * chunk - 4 * lane;   // the lane's bins: top - 1 .. - 4
                uint4 v;
                if constexpr (CL == 1) {
                    v = *reinterpret_cast<const uint4*>(h + top - 4);
                } else {
                    v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int c = 0; c < CL; ++c) {
                        const uint4 t = load_remote(remote(h + top - 4, c));
                        v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
                    }
                }
                const uint32_t mine = v.x + v.y + v.z + v.w;
                uint32_t run = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += y;
                }
                run += above;                          // keys in the lane's bins and higher ones
                const int owner = __ffs(__ballot_sync(0xffffffffu, run >= left)) - 1;
                uint32_t before = run - mine, found = v.w;
                int at = top - 1;
                if (before + found < left) {
                    before += found, found = v.z, --at;
                    if (before + found < left) {
                        before += found, found = v.y, --at;
                        if (before + found < left) before += found, found = v.x, --at;
                    }
                }
                above = __shfl_sync(0xffffffffu, before, owner);
                bin = __shfl_sync(0xffffffffu, (uint32_t)at, owner);
                in_bin = __shfl_sync(0xffffffffu, found, owner);
            }
            if (tid == 0) search_s[d] = make_uint4(bin, above, in_bin, 0u);
            __syncthreads();
            bin = search_s[d].x, above = search_s[d].y, in_bin = search_s[d].z;
            left -= above;
            cut |= bin << shift;
            if (in_bin == left) {                      // all of the bin stays: no need to split it
                --cut;                                 // (bin 0 whole would be the whole row)
                left = 0;
                break;
            }
            if (cut >> 21 == kProtected >> 21) {       // only protected keys are that high
                cut = kProtected;
                break;
            }
        }
    }
    // n == L: all stay (keys are at least 0, so all are above or at the cut 0, as many ties as
    // there are); n == 0: none does
    if (n == L) cut = 0, left = (uint32_t)L;
    if (n == 0) cut = kProtected, left = 0;

    // this warp's keys above and at the cut, all and those below n
    int c_gt = 0, c_eq = 0, c_gt_low = 0, c_eq_low = 0;
    const bool mixed = j0 < n && j1 > n;
    for (int b = j0; b < j1; b += kPiece) {
        const int j = b + 4 * lane;
        uint32_t k[4];
        keys4(j, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool is_eq = k[i] == cut && j + i < j1;
            c_gt += k[i] > cut;
            c_eq += is_eq;
            if (mixed) {
                c_gt_low += k[i] > cut && j + i < n;
                c_eq_low += is_eq && j + i < n;
            }
        }
    }
    if (j1 <= n) c_gt_low = c_gt, c_eq_low = c_eq;
    c_gt = __reduce_add_sync(0xffffffffu, c_gt), c_eq = __reduce_add_sync(0xffffffffu, c_eq);
    c_gt_low = __reduce_add_sync(0xffffffffu, c_gt_low);
    c_eq_low = __reduce_add_sync(0xffffffffu, c_eq_low);
    if (lane == 0)
        *reinterpret_cast<int4*>(warp_counts[warp]) = make_int4(c_gt, c_eq, c_gt_low, c_eq_low);
    __syncthreads();
    int4 c = make_int4(0, 0, 0, 0);
    if (lane < kWarps) c = *reinterpret_cast<const int4*>(warp_counts[lane]);
    int gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? c.x : 0);
    int eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? c.y : 0);
    int low = __reduce_add_sync(0xffffffffu, c.z), ties_low = __reduce_add_sync(0xffffffffu, c.w);
    if constexpr (CL > 1) {
        if (warp == 0) {
            const int gt = __reduce_add_sync(0xffffffffu, c.x);
            const int eq = __reduce_add_sync(0xffffffffu, c.y);
            if (lane == 0) *reinterpret_cast<int4*>(cta_counts) = make_int4(gt, eq, low, ties_low);
        }
        cluster_sync();
        uint4 v = make_uint4(0u, 0u, 0u, 0u);          // lane i: CTA i of the cluster
        if (lane < CL) v = load_remote(remote(cta_counts, lane));
        gt_before += __reduce_add_sync(0xffffffffu, lane < part ? (int)v.x : 0);
        eq_before += __reduce_add_sync(0xffffffffu, lane < part ? (int)v.y : 0);
        low = __reduce_add_sync(0xffffffffu, (int)v.z);
        ties_low = __reduce_add_sync(0xffffffffu, (int)v.w);
    }
    const int ties = (int)left;                       // tokens of key `cut` that stay
    const int kept_low = low + min(ties, ties_low);   // kept tokens below n
    const int count = n - kept_low;                   // holes, and tokens to fill them
    int kept = gt_before + min(ties, eq_before);      // kept tokens before the warp's next piece
    for (int b = j0; b < j1; b += kPiece) {
        const int j = b + 4 * lane;
        uint32_t k[4];
        keys4(j, k);
        uint32_t keep = 0, eq = 0;                     // a bit a slot
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            keep |= (uint32_t)(k[i] > cut) << i;
            eq |= (uint32_t)(k[i] == cut && j + i < j1) << i;
        }
        if (__any_sync(0xffffffffu, eq)) {             // ties: the first `ties` of the row stay
            int total = 0;
            int mine = eq_before + before_lane(eq, lane, total);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (eq >> i & 1u) {
                    keep |= (uint32_t)(mine < ties) << i;
                    ++mine;
                }
            eq_before += total;
        }
        int total = 0;
        int rank = kept + before_lane(keep, lane, total);   // kept tokens before the lane's slots
        kept += total;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool stays = keep >> i & 1u;
            if (stays && j + i >= n) moves[rank - kept_low].x = j + i;
            if (!stays && j + i < n && j + i < j1) moves[j + i - rank].y = j + i;
            rank += stays;
        }
    }
    // The slots below n as they are, shared by the row's CTAs; those of evicted tokens are
    // written again below. Keys come from shared memory by now, so that nobody reads what
    // this writes (a part whose keys are computed again copies its own slots).
    const int share = KEYS ? ((n + CL - 1) / CL + 3) / 4 * 4 : 0;
    const int c0 = KEYS ? min(n, part * share) + 4 * tid : min(j0, n) + 4 * lane;
    const int c1 = KEYS ? min(n, (part + 1) * share) : min(j1, n);
#pragma unroll 2
    for (int j = c0; j < c1; j += KEYS ? 4 * T : kPiece) {
        float w[4];
        int pos[4];
        load4(row.w, w, j, c1 - j, aligned);
        if (row.pos) load4(row.pos, pos, j, c1 - j, aligned);
#pragma unroll
        for (int i = 0; i < 4; ++i) pos[i] = row.pos && pos[i] >= 0 ? pos[i] : row.shift + j + i;
        if (aligned && j + 4 <= c1) {
            *reinterpret_cast<float4*>(w_out + j) = make_float4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<int4*>(pos_out + j) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j + i < c1) w_out[j + i] = w[i], pos_out[j + i] = pos[i];
        }
    }
    sync();                                            // the list is whole
    constexpr int kAhead = 4;                          // moves on the way together
    for (int i0 = part * T + tid; i0 < count; i0 += kAhead * CL * T) {
        int2 m[kAhead];                                // written by other CTAs of the cluster
        float w[kAhead];
        int pos[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i * CL * T < count) m[i] = __ldcg(moves + i0 + i * CL * T);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i * CL * T < count) w[i] = row.w[m[i].x], pos[i] = row.position(m[i].x);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i * CL * T < count) w_out[m[i].y] = w[i], pos_out[m[i].y] = pos[i];
    }
    if (part == 0 && tid == 0) p.move_counts[sg] = count;
    sync();                                            // entries from n on are read no more
    for (int j = max(n, a0) + tid; j < a1; j += T) {
        w_out[j] = 0.f;
        pos_out[j] = -1;
    }
}

struct MoveParams {
    uint4* code[2];           // K, V
    float* scale[2];          // null: rows carry no scales
    int8_t* zp[2];
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int2* moves;
    const int32_t* move_counts;
    unsigned int* err;
    int max_moves, num_kv_heads, max_len, num_blocks, max_blocks;
};

constexpr int kMoveWarps = 4;
constexpr int kMoveAhead = 4;   // copies on the way together, per warp: 8 were slower (67.5 us
                                // against 64.5 with the selection of 131072 tokens), 2 too
                                // (68.0), and so were loads ahead of the last stores (69)

// Grid: (parts, KV head, sequence); the warps of all parts share the row's moves.
// A lane looks up one move (its slots, their blocks) and copies its scales and
// zero points; then the warp copies the moves' K and V rows in 16-byte vectors,
// 32 / (2 VECS) moves at a time and kMoveAhead such loads on the way before the
// first store (no destination is a source, so the order is free). Bound by
// memory: each row in and out, in pieces of 256 bytes and less that lie apart; 25
// thousand moves of each of 8 heads (bf16, d = 128, 206 MB in and out) take 35 us
// alone. Caching loads rather than streaming ones: 63.3 us against 64.5 with the
// selection of 131072 tokens; a row's address from one base a lane: 64.5 against 68.6.
template <int VECS, int GROUPS>   // 16-byte vectors and scales of a row
__global__ void __launch_bounds__(32 * kMoveWarps) move_tokens_kernel(const MoveParams p) {
    constexpr int kPieces = 2 * VECS, kMoves = 32 / kPieces;   // moves of one warp-wide copy
    static_assert(kPieces <= 32, "a move fits a warp");
    // Kernels that read the cache may do so by loads that are not ordered after this one
    // until it has ended, so they are not let in early; nor is the list, which the kernel
    // before may have finished under this one, read that way.
    pa::grid_dependency_wait();
    const int s = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const int L = max(0, min(__ldg(p.context_lens + s), p.max_len));
    const int count = min(__ldcg(p.move_counts + sg), p.max_moves);
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
    const int warps = gridDim.x * kMoveWarps;
    // moves of a warp's turn: at most one a lane, and as many turns for every warp
    const int turns = max(1, (count + 32 * warps - 1) / (32 * warps));
    const int per = max(1, (count + turns * warps - 1) / (turns * warps));
    const int v = lane % kPieces >= VECS, c = lane % kPieces - v * VECS;
    // the lane's vector of row 0 of the KV head's tile in block 0
    uint4* const code = (v ? p.code[1] : p.code[0]) + (int64_t)g * kBS * VECS + c;
    const uint32_t block_vecs = (uint32_t)p.num_kv_heads * kBS * VECS;
    auto vec_at = [&](int blk, int off) {
        return code + ((uint64_t)(uint32_t)blk * block_vecs + off * VECS);
    };
    for (int64_t m0 = (int64_t)(blockIdx.x * kMoveWarps + (threadIdx.x >> 5)) * per; m0 < count;
         m0 += (int64_t)warps * per) {
        const int here = (int)min((int64_t)per, count - m0);
        int bs = -1, bd = -1, at = 0;    // blocks, and the offsets in them: source | destination << 4
        if (lane < here) {
            const int2 mv = __ldcg(p.moves + sg * p.max_moves + m0 + lane);
            if (mv.x < 0 || mv.x >= L || mv.y < 0 || mv.y >= L) {
                if (p.err) atomicOr(p.err, pa::ERR_BAD_SLOT);
            } else {
                bs = __ldg(table + mv.x / kBS), bd = __ldg(table + mv.y / kBS);
                at = mv.x % kBS | mv.y % kBS << 4;
                if (bs < 0 || bs >= p.num_blocks || bd < 0 || bd >= p.num_blocks) {
                    if (p.err) atomicOr(p.err, pa::ERR_BAD_BLOCK);
                    bs = -1;
                }
            }
        }
        auto row_of = [&](int blk, int off) {
            return ((int64_t)blk * p.num_kv_heads + g) * kBS + off;
        };
        if (GROUPS > 0 && bs >= 0) {
            const int64_t src = row_of(bs, at & 15) * GROUPS, dst = row_of(bd, at >> 4) * GROUPS;
            float sc[2][GROUPS > 0 ? GROUPS : 1];
            int8_t zp[2][GROUPS > 0 ? GROUPS : 1];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < GROUPS; ++j)
                    sc[i][j] = p.scale[i][src + j], zp[i][j] = p.zp[i][src + j];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < GROUPS; ++j)
                    p.scale[i][dst + j] = sc[i][j], p.zp[i][dst + j] = zp[i][j];
        }
        for (int i0 = 0; i0 < here; i0 += kMoves * kMoveAhead) {
            uint4 data[kMoveAhead];
            uint4* to[kMoveAhead];
#pragma unroll
            for (int k = 0; k < kMoveAhead; ++k) {
                const int m = i0 + k * kMoves + lane / kPieces;   // past the last: lanes with bs = -1
                const int from = __shfl_sync(0xffffffffu, bs, m & 31);
                const int dst = __shfl_sync(0xffffffffu, bd, m & 31);
                const int off = __shfl_sync(0xffffffffu, at, m & 31);
                const bool on = m < here && from >= 0;
                to[k] = on ? vec_at(dst, off >> 4) : nullptr;
                if (on) data[k] = *vec_at(from, off & 15);
            }
#pragma unroll
            for (int k = 0; k < kMoveAhead; ++k)
                if (to[k]) *to[k] = data[k];
        }
    }
}

template <int VECS, int GROUPS>
pa_status launch_move(const MoveParams& p, int num_seqs, cudaStream_t st) {
    // 8 CTAs a SM over the whole call, but no more than the moves could use
    const int64_t rows = (int64_t)num_seqs * p.num_kv_heads;
    const int64_t could = (p.max_moves + kMoveWarps - 1) / kMoveWarps;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(could, (152 * 8 + rows - 1) / rows));
    return pa::cuda_status(pa::launch_pdl(move_tokens_kernel<VECS, GROUPS>,
                                          dim3((unsigned)parts, p.num_kv_heads, num_seqs),
                                          dim3(32 * kMoveWarps), 0, st, p),
                           "move_tokens launch");
}

template <int CL, int T, bool KEYS>
pa_status launch_select_as(const SelectParams& p, int num_seqs, int keys, cudaStream_t st) {
    auto kern = evict_select_kernel<CL, T, KEYS>;
    static std::atomic<uint64_t> allowed{0};
    if (pa_status s = pa::allow_smem(kern, kHistBytes + 4 * kMaxKeys, allowed,
                                     "evict_select: set shared memory size"))
        return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL, p.num_kv_heads, num_seqs);
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = kHistBytes + (KEYS ? 4 * keys : 0);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL == 1 ? 1 : 2;
    return pa::cuda_status(cudaLaunchKernelEx(&cfg, kern, p), "evict_select launch");
}

template <int CL>
pa_status launch_select_cl(const SelectParams& p, int num_seqs, int keys, cudaStream_t st) {
    // four to five slots a thread where an SM then holds several CTAs, more in long parts
    if (keys <= 1280) return launch_select_as<CL, 256, true>(p, num_seqs, keys, st);
    if (keys <= 4096) return launch_select_as<CL, 512, true>(p, num_seqs, keys, st);
    return launch_select_as<CL, 1024, true>(p, num_seqs, keys, st);
}

// How many CTAs share a row: more while the rows alone leave SMs idle and a part
// stays worth its barriers (2048 slots), or while a part's keys do not fit shared
// memory.
pa_status launch_select(const SelectParams& p, int num_seqs, cudaStream_t st) {
    const int64_t rows = (int64_t)num_seqs * p.num_kv_heads;
    int cl = 1;
    while (cl < kMaxCluster && ((rows * cl < 152 && p.max_len / cl > 2048) ||
                                p.max_len / cl + 128 > kMaxKeys))
        cl *= 2;
    const int keys = ((p.max_len + cl - 1) / cl + 127) / 128 * 128;   // whole pieces
    if (keys > kMaxKeys) return launch_select_as<kMaxCluster, 1024, false>(p, num_seqs, keys, st);
    switch (cl) {
        case 1: return launch_select_cl<1>(p, num_seqs, keys, st);
        case 2: return launch_select_cl<2>(p, num_seqs, keys, st);
        case 4: return launch_select_cl<4>(p, num_seqs, keys, st);
        default: return launch_select_cl<8>(p, num_seqs, keys, st);
    }
}

}  // namespace

extern "C" pa_status pa_evict_select(int32_t* moves, int32_t max_moves, int32_t* move_counts,
                                     float* scores_out, int32_t* positions_out,
                                     const float* scores, const int32_t* positions,
                                     int64_t score_stride, const int32_t* context_lens,
                                     const int32_t* new_lens, const int32_t* total_lens,
                                     int32_t num_seqs, int32_t num_kv_heads,
                                     int32_t max_context_len, int32_t num_sinks,
                                     int32_t num_recent, void* stream) {
    using pa::fail;
    if (num_seqs < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs < 0");
    if (num_seqs == 0) return PA_OK;
    if (!moves || !move_counts || !scores_out || !positions_out || !scores || !context_lens ||
        !new_lens)
        return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    if (num_kv_heads <= 0) return fail(PA_ERR_INVALID_ARG, "num_kv_heads %d", num_kv_heads);
    if (max_context_len <= 0)
        return fail(PA_ERR_INVALID_ARG, "max_context_len %d", max_context_len);
    if (score_stride < max_context_len)
        return fail(PA_ERR_INVALID_ARG, "score_stride %lld < max_context_len %d",
                    (long long)score_stride, max_context_len);
    if (max_moves < 1 || max_moves < max_context_len / 2)
        return fail(PA_ERR_INVALID_ARG, "max_moves %d cannot hold %d moves", max_moves,
                    std::max(1, max_context_len / 2));
    if (num_sinks < 0 || num_recent < 0)
        return fail(PA_ERR_INVALID_ARG, "num_sinks %d, num_recent %d", num_sinks, num_recent);
    if (num_seqs > 65535 || num_kv_heads > 65535 || max_context_len > pa::kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED,
                    "more than 65535 sequences or KV heads, or %d tokens, in one call",
                    pa::kMaxTokens);
    if ((uintptr_t)moves % 8)
        return fail(PA_ERR_INVALID_ARG, "moves must be 8-byte aligned");
    cudaStream_t st = (cudaStream_t)stream;
    if (pa::validate_enabled())
        if (pa_status s = pa::validate_lengths(context_lens, new_lens, total_lens, num_seqs,
                                               max_context_len, st))
            return s;
    SelectParams p{};
    p.moves = reinterpret_cast<int2*>(moves);
    p.move_counts = move_counts;
    p.scores_out = scores_out;
    p.positions_out = positions_out;
    p.scores = scores;
    p.positions = positions;
    p.context_lens = context_lens;
    p.new_lens = new_lens;
    p.total_lens = total_lens;
    p.stride = score_stride;
    p.max_moves = max_moves;
    p.num_kv_heads = num_kv_heads;
    p.max_len = max_context_len;
    p.sinks = num_sinks;
    p.recent = num_recent;
    return launch_select(p, num_seqs, st);
}

extern "C" pa_status pa_move_tokens(void* k_cache, void* v_cache, pa_dtype kv_dtype,
                                    float* k_scale, float* v_scale, int8_t* k_zp, int8_t* v_zp,
                                    const int32_t* block_tables, int32_t max_blocks_per_seq,
                                    const int32_t* context_lens, const int32_t* moves,
                                    int32_t max_moves, const int32_t* move_counts,
                                    int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim,
                                    int32_t block_size, int32_t num_blocks,
                                    int32_t max_context_len, void* stream) {
    using pa::fail;
    if (num_seqs < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs < 0");
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !moves || !move_counts)
        return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    if (pa_status s = pa::check_cache_args(k_cache, v_cache, kv_dtype, k_scale, v_scale, k_zp,
                                           v_zp, num_kv_heads, head_dim, block_size, num_blocks))
        return s;
    if (max_moves < 1) return fail(PA_ERR_INVALID_ARG, "max_moves %d", max_moves);
    if (max_context_len <= 0 || (int64_t)max_blocks_per_seq * block_size < max_context_len)
        return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq %d, max_context_len %d",
                    max_blocks_per_seq, max_context_len);
    if (num_seqs > 65535 || num_kv_heads > 65535 || max_context_len > pa::kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED,
                    "more than 65535 sequences or KV heads, or %d tokens, in one call",
                    pa::kMaxTokens);
    if ((uintptr_t)moves % 8) return fail(PA_ERR_INVALID_ARG, "moves must be 8-byte aligned");
    cudaStream_t st = (cudaStream_t)stream;
    if (pa::validate_enabled())
        if (pa_status s = pa::validate_moves(block_tables, max_blocks_per_seq, context_lens, moves,
                                             max_moves, move_counts, num_seqs, num_kv_heads,
                                             num_blocks, max_context_len, st))
            return s;
    MoveParams p{};
    p.code[0] = static_cast<uint4*>(k_cache);
    p.code[1] = static_cast<uint4*>(v_cache);
    const int groups = pa::row_groups(kv_dtype, head_dim);
    if (groups) {
        p.scale[0] = k_scale, p.scale[1] = v_scale;
        p.zp[0] = k_zp, p.zp[1] = v_zp;
    }
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.moves = reinterpret_cast<const int2*>(moves);
    p.move_counts = move_counts;
    p.err = pa::device_error_word();
    p.max_moves = max_moves;
    p.num_kv_heads = num_kv_heads;
    p.max_len = max_context_len;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    const bool wide = head_dim == 128;
    switch (kv_dtype) {
        case PA_INT8:
            return wide ? launch_move<8, 1>(p, num_seqs, st) : launch_move<4, 1>(p, num_seqs, st);
        case PA_INT4:
            return wide ? launch_move<4, 2>(p, num_seqs, st) : launch_move<2, 1>(p, num_seqs, st);
        case PA_FP8_E4M3:
            return wide ? launch_move<8, 0>(p, num_seqs, st) : launch_move<4, 0>(p, num_seqs, st);
        default:
            return wide ? launch_move<16, 0>(p, num_seqs, st) : launch_move<8, 0>(p, num_seqs, st);
    }
}
