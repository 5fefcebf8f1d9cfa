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
    __device__ __forceinline__ uint32_t key(int j) const {
        const int q = position(j);
        return q < sinks || q >= first_recent ? kProtected : score_key(w[j]);
    }
};

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;

// A CTA a (KV head, sequence). The n-th largest key by four 8-bit radix steps,
// then one walk that counts and one that emits, each warp over a contiguous
// range of slots with ballots, so that lists come out in slot order.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const SelectParams p) {
    __shared__ uint32_t hist[kSelectWarps][256];
    __shared__ uint32_t digit_s, left_s;
    __shared__ int gt[kSelectWarps], eq[kSelectWarps], gt_low[kSelectWarps], eq_low[kSelectWarps];
    const int s = blockIdx.y, g = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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

    // key of the n-th token in the order, and how many tokens with that key stay
    uint32_t cut = 0, left = (uint32_t)n;
    if (n > 0 && n < L) {
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < kSelectWarps * 256; i += kSelectThreads) hist[0][i] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int j = tid; j < L; j += kSelectThreads) {
                const uint32_t k = row.key(j);
                if ((k & mask) == (cut & mask)) atomicAdd(&hist[warp][k >> shift & 255], 1u);
            }
            __syncthreads();
            if (tid < 256) {
                uint32_t t = 0;
#pragma unroll
                for (int i = 0; i < kSelectWarps; ++i) t += hist[i][tid];
                hist[0][tid] = t;
            }
            __syncthreads();
            if (warp == 0) {   // lane i: digits 255 - 8 i and the seven below
                uint32_t mine = 0;
                for (int d = 0; d < 8; ++d) mine += hist[0][255 - 8 * lane - d];
                uint32_t upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                uint32_t above = upto - mine;
                if (above < left && left <= upto)
                    for (int d = 0; d < 8; ++d) {
                        const uint32_t h = hist[0][255 - 8 * lane - d];
                        if (above + h >= left) {
                            digit_s = 255 - 8 * lane - d;
                            left_s = left - above;
                            break;
                        }
                        above += h;
                    }
            }
            __syncthreads();
            cut |= digit_s << shift;
            left = left_s;
        }
    }
    // n == L: all stay (every key is above no cut); n == 0: none does
    const bool all = n == L, none = n == 0;
    auto larger = [&](uint32_t k) { return all || (!none && k > cut); };
    auto equal = [&](uint32_t k) { return !all && !none && k == cut; };

    const int seg = ((L + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int j0 = min(L, warp * seg), j1 = min(L, j0 + seg);
    int c_gt = 0, c_eq = 0, c_gt_low = 0, c_eq_low = 0;
    for (int b = j0; b < j1; b += 32) {
        const int j = b + lane;
        const uint32_t k = j < j1 ? row.key(j) : 0u;
        const bool is_gt = j < j1 && larger(k), is_eq = j < j1 && equal(k);
        c_gt += __popc(__ballot_sync(0xffffffffu, is_gt));
        c_eq += __popc(__ballot_sync(0xffffffffu, is_eq));
        c_gt_low += __popc(__ballot_sync(0xffffffffu, is_gt && j < n));
        c_eq_low += __popc(__ballot_sync(0xffffffffu, is_eq && j < n));
    }
    if (lane == 0) gt[warp] = c_gt, eq[warp] = c_eq, gt_low[warp] = c_gt_low, eq_low[warp] = c_eq_low;
    __syncthreads();
    int eq_before = 0, gt_before = 0, low = 0, ties_low = 0;
    for (int i = 0; i < kSelectWarps; ++i) {
        if (i < warp) gt_before += gt[i], eq_before += eq[i];
        low += gt_low[i];
        ties_low += eq_low[i];
    }
    const int ties = (int)left;                       // tokens of key `cut` that stay
    const int kept_low = low + min(ties, ties_low);   // kept tokens below n
    const int count = n - kept_low;                   // holes, and tokens to fill them
    int kept = gt_before + min(ties, eq_before);      // kept tokens before the warp's next slot
    for (int b = j0; b < j1; b += 32) {
        const int j = b + lane;
        const uint32_t k = j < j1 ? row.key(j) : 0u;
        const bool is_eq = j < j1 && equal(k);
        const uint32_t eqs = __ballot_sync(0xffffffffu, is_eq);
        const uint32_t below = (1u << lane) - 1u;
        const bool keep = j < j1 && (larger(k) || (is_eq && eq_before + __popc(eqs & below) < ties));
        const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
        const int rank = kept + __popc(keeps & below);   // kept tokens before slot j
        if (j < j1) {
            if (keep && j >= n) {
                moves[rank - kept_low].x = j;
            } else if (keep) {
                w_out[j] = row.w[j];
                pos_out[j] = row.position(j);
            } else if (j < n) {
                moves[j - rank].y = j;
            }
        }
        eq_before += __popc(eqs);
        kept += __popc(keeps);
    }
    __syncthreads();
    for (int i = tid; i < count; i += kSelectThreads) {
        const int2 m = moves[i];
        w_out[m.y] = row.w[m.x];
        pos_out[m.y] = row.position(m.x);
    }
    if (tid == 0) p.move_counts[sg] = count;
    __syncthreads();
    for (int j = n + tid; j < L; j += kSelectThreads) {
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
    int row_vecs;             // 16-byte vectors of a row
    int groups;               // scales of a row
};

constexpr int kMoveThreads = 256;

// Grid: (parts, KV head, sequence); the parts stride over the row's moves. A
// thread copies one 16-byte vector of a K or V row, or one scale and zero point.
__global__ void __launch_bounds__(kMoveThreads) move_tokens_kernel(const MoveParams p) {
    const int s = blockIdx.z, g = blockIdx.y;
    const int64_t sg = (int64_t)s * p.num_kv_heads + g;
    const int L = max(0, min(__ldg(p.context_lens + s), p.max_len));
    const int count = min(__ldg(p.move_counts + sg), p.max_moves);
    const int vecs = 2 * p.row_vecs, pieces = vecs + 2 * p.groups;
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
    const int64_t items = (int64_t)count * pieces;
    for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < items;
         i += (int64_t)gridDim.x * kMoveThreads) {
        const int m = (int)(i / pieces), piece = (int)(i - (int64_t)m * pieces);
        const int2 mv = __ldg(p.moves + sg * p.max_moves + m);
        if (mv.x < 0 || mv.x >= L || mv.y < 0 || mv.y >= L) {
            if (p.err) atomicOr(p.err, pa::ERR_BAD_SLOT);
            continue;
        }
        const int bs = __ldg(table + mv.x / kBS), bd = __ldg(table + mv.y / kBS);
        if (bs < 0 || bs >= p.num_blocks || bd < 0 || bd >= p.num_blocks) {
            if (p.err) atomicOr(p.err, pa::ERR_BAD_BLOCK);
            continue;
        }
        const int64_t src = ((int64_t)bs * p.num_kv_heads + g) * kBS + mv.x % kBS;
        const int64_t dst = ((int64_t)bd * p.num_kv_heads + g) * kBS + mv.y % kBS;
        if (piece < vecs) {
            const int v = piece >= p.row_vecs, c = piece - v * p.row_vecs;
            uint4* code = p.code[v];
            code[dst * p.row_vecs + c] = code[src * p.row_vecs + c];
        } else {
            const int v = piece - vecs >= p.groups, c = piece - vecs - v * p.groups;
            p.scale[v][dst * p.groups + c] = p.scale[v][src * p.groups + c];
            p.zp[v][dst * p.groups + c] = p.zp[v][src * p.groups + c];
        }
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
    if (num_seqs > 65535)
        return fail(PA_ERR_UNSUPPORTED, "more than 65535 sequences in one call");
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
    evict_select_kernel<<<dim3(num_kv_heads, num_seqs), kSelectThreads, 0, st>>>(p);
    return pa::cuda_status(cudaGetLastError(), "evict_select launch");
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
    if (num_seqs > 65535 || num_kv_heads > 65535)
        return fail(PA_ERR_UNSUPPORTED, "more than 65535 sequences or KV heads in one call");
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
    p.groups = pa::row_groups(kv_dtype, head_dim);
    if (p.groups) {
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
    p.row_vecs = pa::cache_row_bytes(kv_dtype, head_dim) / 16;
    // about 16 CTAs a SM over the whole call, but no more than the moves could use
    const int64_t rows = (int64_t)num_seqs * num_kv_heads;
    const int64_t could = ((int64_t)max_moves * (2 * p.row_vecs + 2 * p.groups) + kMoveThreads - 1) /
                          kMoveThreads;
    const int64_t parts = std::max<int64_t>(1, std::min(could, 152 * 16 / rows));
    move_tokens_kernel<<<dim3((unsigned)parts, num_kv_heads, num_seqs), kMoveThreads, 0, st>>>(p);
    return pa::cuda_status(cudaGetLastError(), "move_tokens launch");
}
