// Causal attention over whole prompts, packed one after another, on the
// 5th-generation tensor cores (tcgen05, TMEM): q, k and v as a projection gives
// them, before anything is cached. out_i = sum over j <= i of softmax_j(scale
// q_i k_j) v_j within each prompt ("KV Cache ... PagedAttention" §二), query heads
// in contiguous groups per KV head ("cs336 lecture 10", GQA).
//
// A task is a run of a prompt's tokens and one KV head: two Q tiles of 128 rows,
// a row a (token, head of the group) pair, 128 / group tokens a tile, against the
// prompt's keys up to its last token in tiles of 128. Per tile:
//   S = Q K^T      M128 N128, both K-major in shared memory, S in TMEM
//   P = 2^(S - m)  one thread a row, P as 16 bits into TMEM
//   O += P V       M128 N = head_dim, P from TMEM, V MN-major in shared memory
// The reference m of a row is its maximum of some tiles ago. It moves, and O is scaled in
// TMEM, only when the weights of a tile's first 64 keys sum to more than 2^15 (a rise of 2^9
// to 2^15, by how many keys share it) or one of its last 64 keys' passes 2^15, which is rare (a
// bound of 2^8 was passed by ordinary scores of standard deviation 2 often enough to cost 8 %).
// Sums and O are fp32. P is rounded to the 16-bit type once, as the tensor cores take it, by at
// most half a step of a weight, 2^-8 bf16 and 2^-11 fp16: the size of the rounding of the
// output. (Two 16-bit parts, as the paged prefill has them, would be a third product.)
// fp16 has little room below 1: there weights are 2^8 times as large, so that those from 2^-22 of
// the largest on keep all their bits and the others are off by at most 2^-33 of it. (With the
// reference at 1 they were off by 2^-25: in a prompt whose first token takes e^18 of each other
// one, what the others give came out 75 % short.) The reference then moves from a rise of 2^7.75
// on. To keep that rare it starts from the maximum of the first 128 keys, not 32: 6 prompts of
// 16 heads of 64 take 132 us, 138 from 32 keys, 127 without the factor.
//
// A CTA a SM stays and works off its tasks: the longest first (a task's keys grow
// with its place in the prompt), dealt out to and fro over the CTAs. Its roles:
//   warps 0-3, 4-7   softmax of Q tile 0 and 1
//   warps 8-11       epilogue: O / l to global memory while the next task runs
//   warps 12, 15     issue the products of Q tile 0 and 1: the softmax of either tile
//                    has the other's products to run in
//   warp 13          TMA: Q tiles, K and V tiles into a ring
//   warp 14          finds the tasks
// Every wait is bounded: when the tasks stop being read, warp 14 ends every role's loop.
//
// What bounds it. head_dim 128: the tensor cores, 2048 of about 2250 cycles of a
// step (two Q tiles against 128 keys). One prompt of 8192 tokens, 32 heads over 8, bf16:
// 310 us, 1770 TFLOP/s; of 32768: 5.05 ms, 1740 TFLOP/s, at the power limit (5.3 ms where the
// scores' standard deviation is 2, not 1; every figure here without a workspace).
// head_dim 64: the softmax, 2200 cycles a step of which the products need 1024; the
// two warps of a quarter need 1100 for arithmetic alone (exponentials 1024), the
// rest are loads from TMEM and barriers. 16384 tokens, 32 heads over 8: 1.05 ms,
// 1045 TFLOP/s. Measured beside it, per step of head_dim 64: products waiting for P as
// at 128 (1.08 ms), four softmax warpgroups of half a tile's keys each (1.23 ms),
// halves of a tile one after another with the next one's maximum beside them (1.20
// ms), turns at the exponentials (1.18 ms).
// Short prompts: a task costs about 4000 cycles besides its steps: its first tile
// finds both softmaxes idle, its last is masked, and code that runs once a task comes
// from beyond the instruction caches (53 KB of code in all: 138 us, 46 KB: 128). 16
// prompts of 200 to 2000 tokens: 126 us, 1250 TFLOP/s (137 us at a standard deviation of 2).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <vector>

#include "pa_internal.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

#ifdef PA_TEST_HOOKS
// Test builds only (-DPA_TEST_HOOKS): the first CTA does not start the copy of its k-th K or V
// tile when k == g_test_skip_tile, so that the waits for that tile run out.
__device__ int g_test_skip_tile = -1;
extern "C" pa_status pa_test_skip_tile(int k) {
    return pa::cuda_status(cudaMemcpyToSymbol(g_test_skip_tile, &k, sizeof k), "test hook");
}
#endif

namespace {

constexpr int kRows = 128;               // rows of a Q tile
constexpr int kKeys = 128;               // keys of a K or V tile
constexpr int kThreads = 512;
constexpr int kLaunchSeqs = 256;         // prompts a launch: finding a task reads their lengths
constexpr int kMaxLen = 1 << 22;         // a task's products end well before a wait gives up
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSpan = 64;                // key tiles whose products are summed in TMEM, with a workspace
constexpr int kCtas = 152;               // that a workspace is sized for

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;                     // 128-byte wide parts of a row
    static constexpr int kTile = kKeys * D * 2;                // bytes of a K, V or Q tile
    static constexpr int kHalf = kKeys * 128;                  // bytes of one part
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kKVOff = 2 * kTile;
    static constexpr int kSumOff = kKVOff + kStages * kTile;   // l of both Q tiles' rows
    static constexpr int kOutOff = kSumOff + 2 * kRows * 4;    // an output tile on its way out
    static constexpr int kBarOff = kOutOff + kTile;
    // barriers
    static constexpr int kKVFull = 0, kKVEmpty = kStages, kClean = 2 * kStages,
                         kQFull = 3 * kStages, kQEmpty = kQFull + 2, kSFull = kQEmpty + 2,
                         kPFull = kSFull + 2 /* [tile][half] */, kSFree = kPFull + 4,
                         kOFree = kSFree + 2, kLFull = kOFree + 2, kOFull = kLFull + 2,
                         kODone = kOFull + 2, kTurn = kODone + 2, kTaskFull = kTurn + 2,
                         kTaskEmpty = kTaskFull + 2, kFin = kTaskEmpty + 2, kNumBars = kFin + 2;
    static constexpr int kTaskOff = (kBarOff + 8 * kNumBars + 15) / 16 * 16;   // two task records
    static constexpr int kFlagOff = kTaskOff + 2 * 16;            // TMEM address, abort flag
    static constexpr int kSmem = kFlagOff + 16 + 1024;            // + alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
    // TMEM columns: S of Q tile x at 128 x, O at 256 + D x. P goes over the last 64 columns of S
    // where O leaves no others; else it has its own, and the next S is there before this P is.
    static constexpr bool kApart = D == 64;
    static constexpr uint32_t kOCol = 256;
    __device__ static constexpr uint32_t p_col(int x) { return kApart ? 384 + 64 * x : 128 * x + 64; }
};
constexpr uint32_t kTmemCols = 512;

struct PromptParams {
    void* out;
    const int32_t* start;       // [num_seqs + 1] of this launch's prompts
    unsigned int* err;
    int64_t out_stride;
    int num_seqs;
    int num_tokens;
    int max_len;
    int num_kv_heads;
    int group;
    int tokens;                 // of a Q tile
    unsigned per_task_inv;      // 2^32 / (2 tokens) + 1
    int max_chunks;             // tasks of the longest prompt and one KV head
    float scale_log2;
    float* carry;               // sums of earlier spans, kept_floats() a CTA, or null: one span
};

// A CTA's part of the workspace: for either Q tile O as [column / 4][row][4], and the scale of
// each row of it.
constexpr int kept_floats(int head_dim) { return 2 * kRows * (head_dim + 1); }

template <int D>
__device__ __forceinline__ float* kept_sums(const PromptParams& p, int x) {
    return p.carry + (int64_t)blockIdx.x * kept_floats(D) + x * (kept_floats(D) / 2);
}

// Tokens off .. len - 1 of the prompt that starts at token `start`: what is behind them does
// not matter to the task. Chunks are counted back from the prompt's end, so that the one that
// may leave Q tile 1 empty is the one with the fewest keys.
// A product takes 16 keys at a time and may pass the prompt's end, from its last chunk and, with
// chunks of fewer tokens than that, from the ones before: the task says where the end is.
struct alignas(16) Task {
    int start, len, off;
    int head_rest;              // 16 x KV head + tokens of the prompt from len on, at most 15; -1: no more tasks
    __device__ __forceinline__ int head() const { return head_rest >> 4; }
    // the prompt's end, or a place that no product of the task reaches
    __device__ __forceinline__ int end() const { return len + (head_rest & 15); }
};

// What a task's Q tile x sees: the prompt's tokens [0, keys), in `tiles` tiles.
struct Span {
    int first, keys, tiles;
    __device__ __forceinline__ Span(const Task& t, int tokens, int x) {
        first = t.off + x * tokens;
        keys = min(first + tokens, t.len);
        tiles = (keys + kKeys - 1) / kKeys;
    }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// a * b + c of two neighbours, b and c the same for both
__device__ __forceinline__ void fma2(float& d0, float& d1, uint32_t a0, uint32_t a1, uint64_t b,
                                     uint64_t c) {
    asm("{\n\t.reg .b64 ra, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "fma.rn.f32x2 rd, ra, %4, %5;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "r"(a0), "r"(a1), "l"(b), "l"(c));
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void add2(uint64_t& d, float a0, float a1) {
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(pair(a0, a1)));
}
__device__ __forceinline__ float sum_of(uint64_t d) {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
    return a + b;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// 32 consecutive columns without a wait; wait_ld() then waits for all loads before it, and
// loaded() puts a use of these registers behind that wait.
__device__ __forceinline__ void ld_32cols_nowait(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// an arrival without a branch
__device__ __forceinline__ void arrive_if(uint32_t bar, bool p) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"((uint32_t)p)
        : "memory");
}
template <int kRegs>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(e));
    return e != 0;
}

// A place in the ring of K and V tiles, and the parity of its use.
template <int kStages>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ Ring next() const {
        Ring r;
        r.slot = slot + 1 == kStages ? 0 : slot + 1;
        r.phase = slot + 1 == kStages ? phase ^ 1 : phase;
        return r;
    }
    __device__ __forceinline__ void advance(uint32_t n) {
        const uint32_t at = slot + n;
        phase ^= (at / kStages) & 1;
        slot = at % kStages;
    }
};

// The rest of a wait whose first look failed, in few instructions (the roles' code takes turns
// in the instruction caches): false once the abort flag is set, which holds the error that ends
// the kernel. The scheduler's warp sets it, whose waits alone are timed: no role goes without
// reading the record that ends the tasks, and the scheduler waits for that.
__device__ __forceinline__ bool wait_longer(uint32_t bar, uint32_t parity,
                                            volatile uint32_t* abort_flag) {
#pragma unroll 1
    while (!pa::mbar_try_wait(bar, parity))
        if (*abort_flag != 0) return false;
    return true;
}

// A timed one: sets the flag after kWaitNs, counted in cycles of 2 GHz.
constexpr uint32_t kWaitClocks = pa::kWaitNs < 1000000000ull ? (uint32_t)(2 * pa::kWaitNs) : 2000000000u;

__device__ __forceinline__ uint32_t cycles() {
    uint32_t c;
    asm volatile("mov.u32 %0, %%clock;" : "=r"(c));
    return c;
}
__device__ __forceinline__ bool wait_timed(uint32_t bar, uint32_t parity,
                                           volatile uint32_t* abort_flag) {
    const uint32_t began = cycles();
#pragma unroll 1
    while (!pa::mbar_try_wait(bar, parity))
        if (cycles() - began > kWaitClocks) {
            *abort_flag = pa::ERR_WAIT_FULL;
            return false;
        }
    return true;
}

// Length of prompt s, cut to what the tensors hold.
__device__ __forceinline__ int length_of(const PromptParams& p, int s, int& start) {
    start = min(max(__ldg(p.start + s), 0), p.num_tokens);
    const int end = min(max(__ldg(p.start + s + 1), 0), p.num_tokens);
    return min(max(end - start, 0), p.max_len);
}

// kCarry is its own variant: 128 wide, what it adds to the softmax costs 6 to 8 % (16384 tokens, 32
// heads over 8, bf16: 1392 us with a workspace, 1300 without; 32768: 5.5 ms, 5.05); 64 wide,
// nothing (1040 us either way).
template <typename T, int D, bool kCarry>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v,
                            const __grid_constant__ PromptParams p) {
    using LY = Layout<D>;
    constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kStages = LY::kStages;
    // Weights are 2^kLift times as large; the reference moves when a key is kLazyMax orders above it
    // or the first 64 keys' weights sum to more than kLazySum: fp16 ends at 65504.
    constexpr float kLift = kBF16 ? 0.f : 8.f;
    constexpr float kLazyMax = kBF16 ? 15.f : 7.75f, kLazySum = kBF16 ? 32768.f : 60000.f;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = pa::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t bars = base + LY::kBarOff;
    float* const sums = reinterpret_cast<float*>(smem + LY::kSumOff);
    volatile Task* const tasks = reinterpret_cast<volatile Task*>(smem + LY::kTaskOff);
    uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(smem + LY::kFlagOff);
    volatile uint32_t* const abort_flag =
        reinterpret_cast<volatile uint32_t*>(smem + LY::kFlagOff + 8);
    auto bar = [&](int i) { return bars + 8u * i; };

    pa::grid_dependents_launch();
    if (threadIdx.x == 0) {
        for (int i = 0; i < LY::kNumBars; ++i) {
            // arrivals: P, S read, l, zeroed V rows and a free O from the four warps of a group; a
            // free K or V tile from both issuing warps; a task record from every warp that reads it
            const int n = (i >= LY::kPFull && i < LY::kOFull) || (i >= LY::kClean && i < LY::kQFull)
                              ? 4
                          : i >= LY::kKVEmpty && i < LY::kClean ? 2
                          : i >= LY::kTaskEmpty && i < LY::kFin ? 15
                                                               : 1;
            pa::mbar_init(bar(i), n);
        }
        *abort_flag = 0;
        pa::fence_barrier_init();
        pa::prefetch_tensormap(&map_q);
        pa::prefetch_tensormap(&map_k);
        pa::prefetch_tensormap(&map_v);
    }
    // Rows that no copy of Q writes (groups that do not divide 128): zeros, whose scores never move
    // a maximum. What an earlier kernel left there moved it in tile after tile (2 prompts of 4219
    // and 4271, groups of 7: 189 us, 164 with zeros).
    for (int e = p.tokens * p.group * 8 + threadIdx.x; e < kRows * 8; e += kThreads)
        for (int h = 0; h < 2 * LY::kHalves; ++h)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(base + h * LY::kHalf + 16 * e),
                         "r"(0u)
                         : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (warp == 12) {
        pa::tc::tmem_alloc(pa::smem_addr(tmem_holder), kTmemCols);
        pa::tc::tmem_relinquish();
    }
    pa::tc::fence_before_sync();
    __syncthreads();
    pa::tc::fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    pa::grid_dependency_wait();

    // a wait by one lane, or by the whole warp; false ends the role
    auto wait_one = [&](int b, uint32_t parity) -> bool {
        if (pa::mbar_try_wait(bar(b), parity)) return true;
        return wait_longer(bar(b), parity, abort_flag);
    };
    auto wait = [&](int b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_one(b, parity));
    };
    // what has to have ended before the CTA goes, also after a wait gave up
    auto drain = [&](int b, uint32_t parity) {
        if (!pa::mbar_wait(bar(b), parity, nullptr, 0) && p.err) atomicOr(p.err, pa::ERR_WAIT_DRAIN);
    };
    // the i-th task of this CTA
    auto read_task = [&](int i, Task& t) -> bool {
        if (!wait(LY::kTaskFull + (i & 1), (i >> 1) & 1)) return false;
        volatile Task& r = tasks[i & 1];
        t.start = r.start, t.len = r.len, t.off = r.off, t.head_rest = r.head_rest;
        __syncwarp();
        if (lane == 0) pa::mbar_arrive(bar(LY::kTaskEmpty + (i & 1)));
        return t.head_rest >= 0;
    };
    auto read_task_one = [&](int i, Task& t) -> bool {
        if (!wait_one(LY::kTaskFull + (i & 1), (i >> 1) & 1)) return false;
        volatile Task& r = tasks[i & 1];
        t.start = r.start, t.len = r.len, t.off = r.off, t.head_rest = r.head_rest;
        pa::mbar_arrive(bar(LY::kTaskEmpty + (i & 1)));
        return t.head_rest >= 0;
    };
    const int G = p.group, tokens = p.tokens;
    // whether the last products of both Q tiles reach V rows behind the prompt, in one tile:
    // then Q tile 0's softmax zeroes them, and Q tile 1's products wait for that
    auto first_cleans = [&](const Task& t) {
        const Span a(t, tokens, 0), b(t, tokens, 1);
        return b.keys > a.keys && a.tiles == b.tiles && ((a.keys + 15) & ~15) > t.end();
    };

    if (warp < 8) {
        // ---------------- softmax of Q tile x: one thread a row ----------------
        more_registers<176>();
        // 176 + 176 + 80 + 80: the 4 x 128 registers a thread of the launch
        const int x = warp >> 2;
        const int row = 32 * (warp & 3) + lane;
        const uint32_t lane_at = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_tm = tmem + lane_at + 128 * x, p_tm = tmem + lane_at + LY::p_col(x);
        const uint32_t o_tm = tmem + lane_at + LY::kOCol + D * x;
        const int token = row / G;                           // of the tile
        const uint64_t sl2 = pair(p.scale_log2, p.scale_log2);
        Ring<kStages> kv;                                    // the task's first K tile
        uint32_t n_s = 0, n_o = 0;                           // S tiles and tasks so far
        Task task;
        for (int i = 0; read_task(i, task); ++i) {
            const bool two = task.len - task.off > tokens;
            const Span all(task, tokens, two ? 1 : 0), span(task, tokens, x);
            if (x == 1 && !two) {
                kv.advance(2 * all.tiles);
                continue;
            }
            // rows past the tile's tokens or the prompt hold anything; they are not written
            const int bound = span.first + token;
            float m_run = -INFINITY, l_run = 0.f;
            float kept_scale = 0.f;                          // of the sums of earlier spans
            bool ok = true;
            uint64_t l4[2], nm;
            // 32 keys' weights, from their scores to P
            auto weights = [&](uint32_t (&c)[32], uint32_t p_at) {
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        float a, b;
                        fma2(a, b, c[j + q], c[j + q + 1], sl2, nm);
                        a = pa::ex2(a);
                        b = pa::ex2(b);
                        pk[(j + q) / 2] = pack2<T>(a, b);
                        add2(l4[q / 2], a, b);
                    }
                }
                pa::tc::st_16cols_nowait(p_at, pk);
            };
            auto max32 = [&](uint32_t (&c)[32], float (&m)[4]) {
#pragma unroll
                for (int j = 0; j < 32; j += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        m[q] = max3(m[q], __uint_as_float(c[j + 2 * q]),
                                    __uint_as_float(c[j + 2 * q + 1]));
            };
            auto scaled_max = [&](float (&m)[4]) {
                const float mx = fmaxf(max3(m[0], m[1], m[2]), m[3]);
                return mx == -INFINITY ? mx : mx * p.scale_log2;   // the scale is positive
            };
            auto mask = [&](uint32_t (&c)[32], int key0) {   // keys that a row must not see
                if (key0 + 31 > span.first) {
                    const int last = bound - key0;           // bits 0 .. last stay
                    const uint32_t seen = last < 0 ? 0u : 0xffffffffu >> (31 - min(last, 31));
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!(seen >> j & 1)) c[j] = 0xff800000u;    // -inf
                }
            };
            auto reference = [&]() {
                // rounded down: never more than the lift, also where scores are so large that it
                // is less than their fp32 step
                const float m = m_run == -INFINITY ? 0.f
                                : kLift == 0.f     ? -m_run
                                                   : __fadd_rd(kLift, -m_run);
                nm = pair(m, m);
            };
            auto scale_o = [&](float alpha) {
#pragma unroll 1
                for (int q = 0; q < D / 8; ++q) {
                    uint32_t ov[8];
                    pa::tc::ld_8cols(o_tm + 8 * q, ov);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                    pa::tc::st_8cols(o_tm + 8 * q, ov);
                }
            };
            // The tensor cores cut off what does not fit when they add to O: 2.5e-3 of a sum of one
            // sign over 524288 keys, 1.6e-4 over 32768. With a workspace O is added to the sums of
            // earlier spans after every 64 tiles (in fp32, to nearest), and the products start anew.
            auto keep = [&]() {
                float4* const at = reinterpret_cast<float4*>(kept_sums<D>(p, x)) + row;
#pragma unroll 1
                for (int q = 0; q < D / 8; ++q) {
                    uint32_t ov[8];
                    pa::tc::ld_8cols(o_tm + 8 * q, ov);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float4 v = make_float4(
                            __uint_as_float(ov[4 * e]), __uint_as_float(ov[4 * e + 1]),
                            __uint_as_float(ov[4 * e + 2]), __uint_as_float(ov[4 * e + 3]));
                        float4& sum = at[(2 * q + e) * kRows];
                        if (kept_scale != 0.f) {
                            const float4 old = sum;
                            v.x = fmaf(old.x, kept_scale, v.x), v.y = fmaf(old.y, kept_scale, v.y);
                            v.z = fmaf(old.z, kept_scale, v.z), v.w = fmaf(old.w, kept_scale, v.w);
                        }
                        sum = v;
                    }
                }
                kept_scale = 1.f;
            };
            auto publish = [&](int half) {
                pa::tc::wait_st();
                pa::tc::fence_before_sync();
                __syncwarp();
                arrive_if(bar(LY::kPFull + 2 * x + half), lane == 0);
            };
            // V rows behind the prompt that the last tile's product reaches may hold anything:
            // zeroed, so that a weight of 0 never meets a NaN. The first Q tile to reach them
            // does it.
            auto zero_behind = [&]() -> bool {
                const int end = task.end();
                if (((span.keys + 15) & ~15) <= end || (x == 1 && first_cleans(task))) return true;
                Ring<kStages> v = kv;
                v.advance(2 * span.tiles - 1);
                if (!wait(LY::kKVFull + v.slot, v.phase)) return false;
                const int z0 = end - (span.tiles - 1) * kKeys;
                const int n = (((span.keys + 15) & ~15) - end) * (D / 8);
                for (int e = row; e < n; e += kRows) {
                    const int r = z0 + e / (D / 8), ch = e % (D / 8);
                    const uint32_t dst = base + LY::kKVOff + v.slot * LY::kTile +
                                         (ch >> 3) * LY::kHalf + r * 128 + ((ch & 7) << 4);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0u)
                                 : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if (x == 0 && first_cleans(task)) {
                    __syncwarp();
                    if (lane == 0) pa::mbar_arrive(bar(LY::kClean + v.slot));
                }
                return true;
            };

            for (int t = 0; t < span.tiles; ++t, ++n_s) {
                ok = wait(LY::kSFull + x, n_s & 1);
                if (!ok) break;
                pa::tc::fence_after_sync();
                const int key0 = t * kKeys;
                const int in_tile = span.keys - key0;    // visible keys of this tile
                float alpha = 1.f;
                uint32_t c[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) ld_32cols_nowait(s_tm + 32 * i, c[i]);
                wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) loaded(c[i]);
                if (LY::kApart) {
                    // the next S may come; P of the last tile has been read
                    pa::tc::fence_before_sync();
                    __syncwarp();
                    arrive_if(bar(LY::kSFree + x), lane == 0);
                    if (n_s > 0) ok = wait(LY::kODone + x, (n_s - 1) & 1);
                    if (!ok) break;
                    pa::tc::fence_after_sync();
                }
                if (kCarry && t > 0 && t % kSpan == 0) keep();
                if (key0 + kKeys - 1 > span.first) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) mask(c[i], key0 + 32 * i);
                }
                if (t == 0) {                            // a first reference, not above the maximum
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    max32(c[0], m4);
                    if (!kBF16) max32(c[1], m4), max32(c[2], m4), max32(c[3], m4);
                    m_run = scaled_max(m4);
                }
                // Weights of the first 64 keys against the reference so far: a sum of them up to
                // kLazySum says that none is too large. The last 64 keys' maximum is found beside
                // them. In the rare case that either is, the maximum of all and once more. P may go
                // over the columns of the last 64 keys' S: they are in registers by now. (A
                // difference, not m_run + kLazyMax, which large scores would round up.)
                for (;;) {
                    reference();
                    l4[0] = l4[1] = 0;
                    weights(c[0], p_tm);
                    weights(c[1], p_tm + 16);
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    max32(c[2], m4);
                    max32(c[3], m4);
                    const bool look = sum_of(l4[0]) + sum_of(l4[1]) > kLazySum || m_run == -INFINITY ||
                                      scaled_max(m4) - m_run > kLazyMax;
                    if (!__any_sync(0xffffffffu, look)) break;
                    max32(c[0], m4);
                    max32(c[1], m4);
                    const float mx = scaled_max(m4);
                    const bool moved = look && mx > m_run;
                    if (!__any_sync(0xffffffffu, moved)) break;
                    if (moved) {
                        alpha = pa::ex2(m_run - mx);         // 0 while m_run is -inf
                        m_run = mx;
                        kept_scale *= alpha;
                    }
                    // O may be scaled now: S of this tile was issued behind the last P V, and the
                    // barrier says that both are done; the next P V waits for this P
                    if (t > 0) scale_o(alpha);
                }
                if (t == span.tiles - 1) ok = zero_behind();
                if (!ok) break;
                publish(0);
                if (in_tile > 64) {                      // else no product reads it
                    weights(c[2], p_tm + 32);
                    weights(c[3], p_tm + 48);
                }
                publish(1);
                l_run = l_run * alpha + (sum_of(l4[0]) + sum_of(l4[1]));
            }
            if (!ok) break;
            kv.advance(2 * all.tiles);
            // the sums of the last task have been read
            if (n_o > 0 && !wait(LY::kOFree + x, (n_o - 1) & 1)) break;
            ++n_o;
            sums[x * kRows + row] = l_run;
            if (kCarry) kept_sums<D>(p, x)[kRows * D + row] = kept_scale;
            __syncwarp();
            if (lane == 0) pa::mbar_arrive(bar(LY::kLFull + x));
        }
    } else if (warp < 12) {
        // ---------------- epilogue: O / l of each Q tile ----------------
        fewer_registers<80>();
        const int row = 32 * (warp & 3) + lane;
        const uint32_t lane_at = (uint32_t)(32 * (warp & 3)) << 16;
        const int token = row / G, head = row % G;
        constexpr int kChunks = D / 8;                       // 16-byte parts of a row
        uint4* const out = reinterpret_cast<uint4*>(smem + LY::kOutOff) + 32 * (warp & 3) * kChunks;
        uint32_t parity = 0;                                 // of Q tile x in bit x
        Task task;
        bool ok = true;
        for (int i = 0; ok && read_task(i, task); ++i) {
            const int nq = task.len - task.off > tokens ? 2 : 1;
#pragma unroll 1
            for (int x = 0; x < nq; ++x) {
                const int at = task.off + x * tokens + token;
                // where this lane's row goes, in units of 8 elements; -1: nowhere
                const int64_t mine =
                    token < tokens && at < task.len
                        ? ((int64_t)(task.start + at) * p.out_stride + (task.head() * G + head) * D) / 8
                        : -1;
                ok = wait(LY::kLFull + x, (parity >> x) & 1) &&
                     wait(LY::kOFull + x, (parity >> x) & 1);
                if (!ok) break;
                parity ^= 1u << x;
                pa::tc::fence_after_sync();
                const float l = sums[x * kRows + row];
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float* const kept = kCarry ? kept_sums<D>(p, x) : nullptr;
                const float kept_scale = kCarry ? kept[kRows * D + row] : 0.f;
                const uint32_t o_tm = tmem + lane_at + LY::kOCol + D * x;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    ld_32cols_nowait(o_tm + c, o);
                    wait_ld();
                    loaded(o);
                    if (kCarry && kept_scale != 0.f) {       // sums of earlier spans
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 v =
                                reinterpret_cast<const float4*>(kept)[(c + e) / 4 * kRows + row];
                            o[e] = __float_as_uint(fmaf(v.x, kept_scale, __uint_as_float(o[e])));
                            o[e + 1] = __float_as_uint(fmaf(v.y, kept_scale, __uint_as_float(o[e + 1])));
                            o[e + 2] = __float_as_uint(fmaf(v.z, kept_scale, __uint_as_float(o[e + 2])));
                            o[e + 3] = __float_as_uint(fmaf(v.w, kept_scale, __uint_as_float(o[e + 3])));
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint4 w;
                        w.x = pack2<T>(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                        w.y = pack2<T>(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                        w.z = pack2<T>(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                        w.w = pack2<T>(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                        out[lane * kChunks + (((c + e) / 8) ^ (lane % kChunks))] = w;
                    }
                }
                // all of O and l has been read
                pa::tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) pa::mbar_arrive(bar(LY::kOFree + x));
                // whole rows side by side (a lane a row of its own took 2700 cycles a tile, most
                // of them for 32 places a store)
#pragma unroll 4
                for (int r0 = 0; r0 < 32; r0 += 32 / kChunks) {
                    const int r = r0 + lane / kChunks, ch = lane % kChunks;
                    const int64_t to = __shfl_sync(0xffffffffu, mine, r);
                    if (to >= 0)
                        reinterpret_cast<uint4*>(p.out)[to + ch] = out[r * kChunks + (ch ^ (r % kChunks))];
                }
                __syncwarp();
            }
        }
    } else {
        fewer_registers<80>();
        if (warp == 12 || warp == 15) {
            // ---------------- the products of Q tile x, issued by one elected lane ----------------
            // One branch around everything: a product then issues in fewer cycles than it runs
            // (64 at N = 128; with an election around each it took 140 to 160). A warp a Q tile:
            // the waits of one overlap the products of the other. Both read every K and V tile
            // (or pass it on). The tensor cores run a thread's products in the order of their
            // issue, so that P V has read P before the next Q K^T takes its columns.
            if (elect_one()) {
                const int x = warp == 12 ? 0 : 1;
                constexpr uint32_t idesc_qk = pa::tc::idesc_f16(kBF16, false, false, kRows, kKeys);
                constexpr uint32_t idesc_pv = pa::tc::idesc_f16(kBF16, false, true, kRows, D);
                // the descriptor of address a + o is the one of a plus o >> 4
                const uint64_t dq = pa::tc::smem_desc_sw128(base + x * LY::kTile, 16, 1024);
                const uint64_t dk = pa::tc::smem_desc_sw128(base + LY::kKVOff, 16, 1024);
                const uint64_t dv = pa::tc::smem_desc_sw128(base + LY::kKVOff, LY::kHalf, 1024);
                const uint32_t s_tm = tmem + 128 * x, o_tm = tmem + LY::kOCol + D * x;
                Ring<kStages> kv;
                uint32_t n_s = 0, n_q = 0;
                uint32_t cleaned = 0;                        // parities of the ring's kClean
                // With two Q tiles their products take turns: P V and Q K'^T of one, then of the
                // other, or both softmaxes would come to run at once and then both products.
                // The turn goes over before the last products are issued, so that the pipe does
                // not wait for the other warp to wake up. (8192 tokens: 357 us, 410 without
                // turns.) Where P has columns of its own, softmaxes do not wait for products.
                uint32_t turns = 0;
                auto my_turn = [&](bool two) -> bool {
                    return LY::kApart || !two ||
                           wait_one(LY::kTurn + x, (turns++ & 1) ^ (x ^ 1));
                };
                auto pass_turn = [&](bool two) {
                    if (!LY::kApart && two) pa::mbar_arrive(bar(LY::kTurn + (x ^ 1)));
                };
                auto issue_qk = [&](bool two) {              // S = Q K^T
                    pa::tc::fence_after_sync();
                    const uint64_t b = dk + (uint64_t)((kv.slot * LY::kTile) >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t o = ((kk >> 2) * LY::kHalf + (kk & 3) * 32) >> 4;
                        pa::tc::mma_f16_ss(s_tm, dq + o, b + o, idesc_qk, kk > 0 ? 1u : 0u);
                        if (kk == D / 16 - 3) pass_turn(two);
                    }
                    pa::tc::commit(bar(LY::kSFull + x));
                    pa::tc::commit(bar(LY::kKVEmpty + kv.slot));
                    kv = kv.next();
                };
                auto issue_pv = [&](const Ring<kStages>& v, int half, int steps, bool more) {   // O += P V
                    pa::tc::fence_after_sync();
                    const uint64_t b = dv + (uint64_t)((v.slot * LY::kTile) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int kb = 4 * half + k;
                        if (kb < steps)
                            pa::tc::mma_f16_ts(o_tm, tmem + LY::p_col(x) + 8 * kb,
                                               b + (uint64_t)((kb * 16 * 128) >> 4), idesc_pv,
                                               more || kb > 0 ? 1u : 0u);
                    }
                };
                auto pass_on = [&](int n) -> bool {          // tiles that only the other one reads
                    for (int k = 0; k < n; ++k) {
                        if (!wait_one(LY::kKVFull + kv.slot, kv.phase)) return false;
                        pa::mbar_arrive(bar(LY::kKVEmpty + kv.slot));
                        kv = kv.next();
                    }
                    return true;
                };
                Task task, after;
                bool ok = true, go = read_task_one(0, task);
                // One place for each product, and the next task read while this one's last P is
                // waited for: code that runs once a task has left the instruction caches.
                for (int i = 0; ok && go; ++i, task = after) {
                    const bool two = task.len - task.off > tokens;
                    const int tiles = Span(task, tokens, two ? 1 : 0).tiles;
                    if (x == 1 && !two) {
                        ok = pass_on(2 * tiles);
                        go = read_task_one(i + 1, after);
                        continue;
                    }
                    const Span s(task, tokens, x);
                    const int both = two ? Span(task, tokens, 0).tiles : -1;  // tiles of either
#pragma unroll 1
                    for (int t = -1; t < s.tiles; ++t) {     // S of tile t + 1, O of tile t
                        const Ring<kStages> v = kv, next = t < 0 ? kv : kv.next();
                        const bool more = t + 1 < s.tiles, turn = t < both;
                        if (LY::kApart && more) {
                            // the next S, once this one has been read
                            ok = wait_one(LY::kKVFull + next.slot, next.phase) &&
                                 wait_one(t < 0 ? LY::kQFull + x : LY::kSFree + x,
                                          (t < 0 ? n_q : n_s) & 1);
                            if (!ok) break;
                            kv = next;
                            issue_qk(false);
                        }
                        if (LY::kApart && t < 0) continue;
                        if (!more) pa::tc::commit(bar(LY::kQEmpty + x));
                        // this V tile and the next K tile, or the first K tile and Q
                        ok = wait_one(LY::kKVFull + v.slot, v.phase);
                        if (!LY::kApart && more)
                            ok = ok && (t < 0 ? wait_one(LY::kQFull + x, n_q & 1)
                                              : wait_one(LY::kKVFull + next.slot, next.phase));
                        if (t == 0 && n_q > 0)               // O of the last task read
                            ok = ok && wait_one(LY::kOFree + x, (n_q - 1) & 1);
                        if (!more && x == 1 && first_cleans(task)) {
                            ok = ok && wait_one(LY::kClean + v.slot, (cleaned >> v.slot) & 1);
                            cleaned ^= 1u << v.slot;
                        }
                        ok = ok && my_turn(turn);
                        if (!ok) break;
                        if (!more) {
                            // the other one's next products need not wait for this task's last P
                            pass_turn(turn);
                            go = read_task_one(i + 1, after);
                        }
                        if (t >= 0) {
                            const int steps = (s.keys - t * kKeys + 15) >> 4;
                            ok = wait_one(LY::kPFull + 2 * x, n_s & 1);
                            if (!ok) break;
                            issue_pv(v, 0, steps, t > 0 && !(kCarry && t % kSpan == 0));
                            ok = wait_one(LY::kPFull + 2 * x + 1, n_s & 1);
                            if (!ok) break;
                            issue_pv(v, 1, steps, true);
                            if (LY::kApart) pa::tc::commit(bar(LY::kODone + x));
                            if (!more) pa::tc::commit(bar(LY::kOFull + x));
                            pa::tc::commit(bar(LY::kKVEmpty + v.slot));
                            if (!LY::kApart || !more) kv = next;
                            ++n_s;
                        }
                        if (!LY::kApart && more) issue_qk(turn);
                    }
                    ok = ok && pass_on(2 * (tiles - s.tiles));
                    ++n_q;
                }
                // every product and commit is done before TMEM and the CTA go
                pa::tc::commit(bar(LY::kFin + x));
                drain(LY::kFin + x, 0);
            }
            __syncwarp();
        } else if (warp == 13) {
            // ---------------- TMA: Q tiles, K and V tiles in turn ----------------
            if (elect_one()) {
                Ring<kStages> kv;
                uint32_t loaded = 0, n_q[2] = {0, 0};
                const uint32_t q_bytes = tokens * G * 128;
                Task task;
                for (int i = 0; read_task_one(i, task); ++i) {
                    const int nq = task.len - task.off > tokens ? 2 : 1;
                    const int tiles = Span(task, tokens, nq - 1).tiles;
                    auto load = [&](int k) -> bool {         // the task's k-th K (even) or V tile
                        if (loaded >= kStages &&
                            !wait_one(LY::kKVEmpty + kv.slot, kv.phase ^ 1))
                            return false;
                        const uint32_t b = bar(LY::kKVFull + kv.slot);
                        pa::mbar_arrive_expect_tx(b, LY::kTile);
#ifdef PA_TEST_HOOKS
                        if (blockIdx.x == 0 && (int)loaded == g_test_skip_tile) {
                            kv = kv.next();
                            ++loaded;
                            return true;
                        }
#endif
                        tma_load_4d(base + LY::kKVOff + kv.slot * LY::kTile,
                                    k & 1 ? &map_v : &map_k, 0, task.start + (k >> 1) * kKeys, 0,
                                    task.head(), b);
                        kv = kv.next();
                        ++loaded;
                        return true;
                    };
                    bool ok = load(0);
                    for (int x = 0; ok && x < nq; ++x) {
                        // Q of the last task has been read
                        if (n_q[x] > 0)
                            ok = wait_one(LY::kQEmpty + x, (n_q[x] - 1) & 1);
                        if (!ok) break;
                        const uint32_t b = bar(LY::kQFull + x);
                        pa::mbar_arrive_expect_tx(b, q_bytes * LY::kHalves);
                        for (int h = 0; h < LY::kHalves; ++h)
                            tma_load_3d(base + x * LY::kTile + h * LY::kHalf, &map_q, 64 * h,
                                        task.head() * G, task.start + task.off + x * tokens, b);
                        ++n_q[x];
                    }
                    for (int k = 1; ok && k < 2 * tiles; ++k) ok = load(k);
                    if (!ok) break;
                }
                // no copy may be in flight when the CTA ends (those whose tiles were consumed are
                // not; after a wait gave up, the last of the ring and of Q may be)
                if (*abort_flag) {
                    for (uint32_t u = loaded > kStages ? loaded - kStages : 0; u < loaded; ++u)
                        drain(LY::kKVFull + u % kStages, (u / kStages) & 1);
                    for (int x = 0; x < 2; ++x)
                        if (n_q[x] > 0) drain(LY::kQFull + x, (n_q[x] - 1) & 1);
                }
            }
            __syncwarp();
        } else if (warp == 14) {
            // ---------------- tasks ----------------
            // The tasks of all prompts in the order of their chunk's place, last first; among
            // equals by prompt, then by KV head. With n_s chunks of prompt s, F(c) = sum of
            // max(0, n_s - c) of them have a place of c or more: the chunk of task v is the
            // c with F(c + 1) <= v < F(c), its prompt the (v - F(c + 1))-th with n_s > c.
            const int per_task = 2 * tokens;
            auto chunks = [&](int len) -> int {              // ceil(len / per_task), len < 2^23
                return (int)__umulhi((unsigned)(len + per_task - 1), p.per_task_inv);
            };
            auto chunks_of = [&](int s) -> int {
                int start;
                return s < p.num_seqs ? chunks(length_of(p, s, start)) : 0;
            };
            const int n = chunks_of(lane);                   // further prompts' are read as needed
            auto at_least = [&](int c) -> unsigned {
                unsigned sum = (unsigned)max(0, n - c);
#pragma unroll 1
                for (int s = 32; s < p.num_seqs; s += 32)
                    sum += (unsigned)max(0, chunks_of(s + lane) - c);
                return __reduce_add_sync(0xffffffffu, sum);
            };
            const unsigned P = gridDim.x;
            // every role has read record i, or the flag is set
            auto all_read = [&](unsigned i) -> bool {
                return __all_sync(0xffffffffu, wait_timed(bar(LY::kTaskEmpty + (i & 1)), (i >> 1) & 1,
                                                          abort_flag));
            };
            for (unsigned i = 0;; ++i) {
                const unsigned v = i * P + (i & 1 ? P - 1 - blockIdx.x : blockIdx.x);
                const unsigned chunk = v / (unsigned)p.num_kv_heads;
                Task t;
                t.start = t.len = t.off = 0, t.head_rest = -1;
                int lo = -1, hi = p.max_chunks;              // F(lo) > chunk >= F(hi)
                unsigned above = 0;                          // F(hi)
#pragma unroll 1
                while (hi - lo > 1) {
                    const int mid = lo < 0 ? 0 : (lo + hi) >> 1;
                    const unsigned f = at_least(mid);
                    if (f > chunk) lo = mid;
                    else hi = mid, above = f;
                }
                if (lo >= 0) {                               // else there are no more
                    unsigned left = chunk - above;
                    int s = 0;
#pragma unroll 1
                    for (;; s += 32) {
                        const bool in = (s == 0 ? n : chunks_of(s + lane)) > lo;
                        const unsigned has = __ballot_sync(0xffffffffu, in);
                        const unsigned cnt = __popc(has);
                        if (left < cnt || s + 32 >= p.num_seqs) {
                            const bool here = in && __popc(has & ((1u << lane) - 1)) == left;
                            s += max(0, __ffs(__ballot_sync(0xffffffffu, here)) - 1);
                            break;
                        }
                        left -= cnt;
                    }
                    const int len = length_of(p, s, t.start);
                    // chunks behind this one (none, if the lengths changed under the kernel)
                    const int behind = max(0, chunks(len) - 1 - lo);
                    t.len = len - behind * per_task;
                    t.off = max(0, t.len - per_task);
                    t.head_rest = 16 * (int)(v - chunk * (unsigned)p.num_kv_heads) + min(15, len - t.len);
                }
                if (i >= 2 && !all_read(i - 2)) break;
                if (lane == 0) {
                    volatile Task& r = tasks[i & 1];
                    r.start = t.start, r.len = t.len, r.off = t.off, r.head_rest = t.head_rest;
                    pa::mbar_arrive(bar(LY::kTaskFull + (i & 1)));
                }
                __syncwarp();
                if (t.head_rest < 0) {
                    all_read(i);
                    break;
                }
            }
        }
    }
    pa::tc::fence_before_sync();
    __syncthreads();
    pa::tc::fence_after_sync();
    if (warp == 12) pa::tc::tmem_dealloc(tmem, kTmemCols);
    if (threadIdx.x == 0 && *abort_flag && p.err) atomicOr(p.err, *abort_flag);
}

template <typename T, int D, bool kCarry>
pa_status launch_as(const CUtensorMap* maps, const PromptParams& p, int64_t grid, cudaStream_t st) {
    auto kern = prompt_attention_kernel<T, D, kCarry>;
    static std::atomic<uint64_t> done{0};
    if (pa_status s = pa::allow_smem(kern, Layout<D>::kSmem, done, "prompt: shared memory size"))
        return s;
    return pa::cuda_status(pa::launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads),
                                          Layout<D>::kSmem, st, maps[0], maps[1], maps[2], p),
                           "prompt attention launch");
}

template <typename T, int D>
pa_status launch(const CUtensorMap* maps, const PromptParams& p, int64_t grid, cudaStream_t st) {
    return p.carry ? launch_as<T, D, true>(maps, p, grid, st)
                   : launch_as<T, D, false>(maps, p, grid, st);
}

pa_status check_rows(const char* name, const void* rows, int64_t stride, int32_t heads,
                     int32_t head_dim) {
    if ((uintptr_t)rows % 16) return pa::fail(PA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (stride < (int64_t)heads * head_dim || stride % 8)
        return pa::fail(PA_ERR_INVALID_ARG,
                        "%s_stride %lld is not a multiple of 8 of at least %lld elements", name,
                        (long long)stride, (long long)heads * head_dim);
    if (stride >= 1ll << 38)
        return pa::fail(PA_ERR_UNSUPPORTED, "%s_stride %lld", name, (long long)stride);
    return PA_OK;
}

}  // namespace

extern "C" size_t pa_prompt_attention_workspace_size(int32_t head_dim, int32_t max_seq_len) {
    if ((head_dim != 64 && head_dim != 128) || max_seq_len <= kSpan * kKeys || max_seq_len > kMaxLen)
        return 0;
    return sizeof(float) * kept_floats(head_dim) * kCtas;
}

extern "C" pa_status pa_prompt_attention(void* out, int64_t out_stride, const void* q,
                                         int64_t q_stride, const void* key, int64_t key_stride,
                                         const void* value, int64_t value_stride, pa_dtype dtype,
                                         const int32_t* seq_start, int32_t num_seqs,
                                         int32_t num_tokens, int32_t max_seq_len,
                                         int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                         float scale, void* workspace, size_t workspace_bytes,
                                         void* stream) {
    using pa::fail;
    if (num_seqs < 0 || num_tokens < 0)
        return fail(PA_ERR_INVALID_ARG, "num_seqs %d, num_tokens %d", num_seqs, num_tokens);
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !key || !value || !seq_start) return fail(PA_ERR_INVALID_ARG, "NULL pointer");
    if (dtype != PA_F16 && dtype != PA_BF16)
        return fail(PA_ERR_UNSUPPORTED, "dtype %d (F16 or BF16)", (int)dtype);
    if (head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d (64 or 128 supported)", head_dim);
    if (num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "num_heads %d is not a multiple of num_kv_heads %d",
                    num_heads, num_kv_heads);
    const int group = num_heads / num_kv_heads;
    if (group > kRows)
        return fail(PA_ERR_UNSUPPORTED, "%d query heads per KV head (at most %d)", group, kRows);
    if (max_seq_len < 1) return fail(PA_ERR_INVALID_ARG, "max_seq_len %d", max_seq_len);
    if (max_seq_len > kMaxLen)
        return fail(PA_ERR_UNSUPPORTED, "prompts of more than %d tokens", kMaxLen);
    if (num_heads > 65535) return fail(PA_ERR_UNSUPPORTED, "num_heads %d (at most 65535)", num_heads);
    if (!(scale >= 0.f) || isinf(scale * kLog2e)) return fail(PA_ERR_INVALID_ARG, "scale %g", (double)scale);
    if (pa_status s = check_rows("q", q, q_stride, num_heads, head_dim)) return s;
    if (pa_status s = check_rows("key", key, key_stride, num_kv_heads, head_dim)) return s;
    if (pa_status s = check_rows("value", value, value_stride, num_kv_heads, head_dim)) return s;
    if (pa_status s = check_rows("out", out, out_stride, num_heads, head_dim)) return s;
    if (workspace && (uintptr_t)workspace % 16)
        return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    const int64_t own = sizeof(float) * kept_floats(head_dim);   // a CTA's part of it
    const bool carry = max_seq_len > kSpan * kKeys && workspace;
    if (carry && (int64_t)workspace_bytes < own)
        return fail(PA_ERR_INVALID_ARG, "workspace of %zu bytes (%zu serve every SM)", workspace_bytes,
                    pa_prompt_attention_workspace_size(head_dim, max_seq_len));
    if (!workspace && max_seq_len > (dtype == PA_F16 ? 1 << 16 : 1 << 19))
        return fail(PA_ERR_INVALID_ARG, "prompts of up to %d tokens need a workspace", max_seq_len);
    cudaStream_t st = (cudaStream_t)stream;
    if (pa::validate_enabled())
        if (pa_status s = pa::validate_starts(seq_start, num_seqs, num_tokens, max_seq_len, st))
            return s;
    int dev = 0, sms = 0;
    if (pa_status s = pa::cuda_status(cudaGetDevice(&dev), "cudaGetDevice")) return s;
    if (pa_status s = pa::cuda_status(
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count"))
        return s;
    PromptParams p{};
    p.out = out;
    p.err = pa::device_error_word();
    p.out_stride = out_stride;
    p.num_tokens = num_tokens;
    p.max_len = max_seq_len;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.tokens = kRows / group;
    const int per_task = 2 * p.tokens;
    p.per_task_inv = (unsigned)((1ull << 32) / per_task) + 1;
    p.max_chunks = (max_seq_len + per_task - 1) / per_task;
    p.carry = carry ? static_cast<float*>(workspace) : nullptr;
    // not 0: a masked score of -inf stays one (a score of 2^100 still has a weight of 1)
    p.scale_log2 = fmaxf(scale * kLog2e, FLT_MIN);
    CUtensorMap maps[3];
    if (pa_status s = pa::rows_tensor_map_heads(&maps[0], q, num_tokens, q_stride, num_heads,
                                                head_dim, group, p.tokens))
        return s;
    if (pa_status s = pa::rows_tensor_map_tokens(&maps[1], key, num_tokens, key_stride,
                                                 num_kv_heads, head_dim, kKeys))
        return s;
    if (pa_status s = pa::rows_tensor_map_tokens(&maps[2], value, num_tokens, value_stride,
                                                 num_kv_heads, head_dim, kKeys))
        return s;
    for (int s0 = 0; s0 < num_seqs; s0 += kLaunchSeqs) {
        p.start = seq_start + s0;
        p.num_seqs = std::min(kLaunchSeqs, num_seqs - s0);
        // at most so many tasks
        const int64_t chunks = std::min((int64_t)p.num_seqs * p.max_chunks,
                                        (int64_t)num_tokens / per_task + p.num_seqs);
        if (chunks * num_kv_heads > 0x7fffffff)
            return fail(PA_ERR_UNSUPPORTED, "too many rows for one launch");
        int64_t grid = std::min<int64_t>(sms, chunks * num_kv_heads);
        if (carry) grid = std::min(grid, (int64_t)workspace_bytes / own);
        pa_status s;
        if (dtype == PA_BF16)
            s = head_dim == 128 ? launch<__nv_bfloat16, 128>(maps, p, grid, st)
                                : launch<__nv_bfloat16, 64>(maps, p, grid, st);
        else
            s = head_dim == 128 ? launch<__half, 128>(maps, p, grid, st)
                                : launch<__half, 64>(maps, p, grid, st);
        if (s) return s;
    }
    return PA_OK;
}
