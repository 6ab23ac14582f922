// Chunked causal prefill over a 4-bit pool on the 5th-generation tensor cores (head_dim 64 or 128, up to 128 q heads per
// kv head).
//
// One CTA computes two 128-row query tiles (a, b) of one (sequence, kv head), or one, with two CTAs on an SM that cover
// each other's start and end, where that serves better (plan_prefill_fp4): row r of a tile is token r / G, q head
// r % G of the G heads that share the kv head, so that every key is unpacked once for both. Keys come in tiles of
// 128. Of two tiles, twenty-four warps (of one: 0-11, two warps of each quadrant for the softmax):
//   0           owns the tensor memory and issues every MMA (kind::f16, fp16 operands, fp32 accumulation):
//               S = Q K^T, O += P V with P from tensor memory, in the order PV_a(j), QK_a(j+1), PV_b(j), QK_b(j+1), so
//               that the tensor cores serve one query tile while the other one's softmax runs
//   4-19        softmax, two threads per query row, each on 64 of the tile's 128 keys, online in the log2 domain, in one
//               pass over S against the reference of the tiles before. Where a score exceeds that by more than 2^8
//               (rarely), both threads of the row learn it at a barrier of their two warps, agree on a new reference,
//               do the tile again and rescale O
//   1-3, 20-23  unpack: a unit is 32 keys of K or of V, eight units a key tile, dealt to these warps in turn; a lane per
//               key reads the key's codes and scales a unit ahead, converts them (e2m1x2 -> f16x2, times the
//               scale, exact) and stores the row in the 128-byte-swizzled layout that the MMAs read; a key past the
//               sequence's end becomes zeros, whatever its cell holds
// Registers move from the other warps to the softmax ones (setmaxnreg; the shares add up to the launch's). Every form but bf16 with
// two tiles of head_dim 64 spills some: 36 to 64 bytes, fp32 at head_dim 64, whose running O has 32 of the 96 registers, 180 to 200.
//
// Query rows are brought to fp16 by a power of two per row, which the row's score factor takes back: bf16's 8 bits fit,
// and what is 2^-39 below the row's largest magnitude is lost. Weights are rounded to fp16, outputs once to bf16.
//
// fp32 queries: q and the weights are sums of two halves, 22 bits, so that S takes two Q K^T and O two P V; a CTA has one
// query tile (the second half lies where a second tile would), and its softmax reads S twice, for the maximum and for the
// weights, whose two halves take the place of the scores that they come from. 9 chunks of 90 to 300 on up to 1543 keys, 64 q
// / 16 kv heads of 64: 117 us (869 on the CUDA cores; 107 with O summed by the MMAs alone, which cut sums off); 4 of 17 to 96
// on up to 900, 12 q / 4 kv heads of 64: 19 (53); 16 of 256 on up to 4352, 32 q / 8 kv heads of 128: 419 (466 with 128
// registers for every warp). Bound: S, softmax and P V of a tile follow one another.
//
// Bound: the chain S -> softmax -> P -> P V, Q K^T -> next S of each query tile, about 3000 cycles a key tile of which 1024 are
// its own MMAs (both tiles' MMAs take 2048), and each CTA's start (5 us) and end (1.5). 16 sequences of 512 new rows on 512 to
// 4608 keys, 32 q / 8 kv heads of 128: 289 us, 1.07 PFLOP/s over visible pairs, 56 % of the measured bf16 rate. Forms that were
// slower there: a thread per row (8 softmax warps) in two passes 351 us, in one 352 to 378; the mask in every tile instead of in
// a copy of the loop 338; registers 56 / 88 instead of 48 / 96 (the softmax spills more) 318; three stages of K and two of V 302.
//
// Few rows on many keys: the key list is cut into runs (Split), one CTA each, and a second kernel merges their
// outputs by M = max m, out = sum 2^(m - M) o / sum 2^(m - M) l. Every wait is bounded; a timeout sets
// PA_DEVERR_WAIT_TIMEOUT and the CTA winds down.
#include <math.h>

#include <type_traits>

#include "fp4.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"
#include "scored.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;  // query rows per tile (M)
constexpr int kKeys = 128;  // keys per key tile (N of S = Q K^T, K of O += P V)
// Of a CTA of NQ query tiles: halves that make a number of q or a weight (fp32: two), CTAs on an SM, warps of softmax, of
// unpacking (three beside the MMA warp, and a warpgroup more in a CTA that has the SM to itself), threads; tensor
// memory columns of O, of all.
template <typename T, int D, int NQ>
struct Roles {
    static constexpr int pieces = std::is_same<T, float>::value ? 2 : 1, per_sm = NQ == 2 || pieces * D == 256 ? 1 : 2;
    static constexpr int soft = 8 * NQ, unpack = per_sm == 1 ? 7 : 3, threads = 32 * (soft + unpack + 1);
    // registers a thread: at launch, then of the softmax and of the other warps
    static constexpr int at_launch = pieces * D == 256 ? 128 : 80, soft_regs = at_launch == 128 ? 200 : 96, other_regs = at_launch == 128 ? 56 : 48;
    static_assert(32 * (soft * soft_regs + (unpack + 1) * other_regs) == threads * at_launch, "setmaxnreg's shares");
    static constexpr uint32_t o = NQ * 128, columns = NQ * 256;
};
constexpr uint32_t kHalf = 16384;         // 128 rows x 128 bytes (64 fp16 columns)
constexpr float kRescaleThreshold = 8.f;  // log2 units
// log2 of the weight of a score at the reference, so that weights far below it (and fp32's second halves) lie within fp16's
// range: 2^-25, which is lost, is 2^-32 of that, and many keys far below one add up to a part of the output. The largest
// weight, 2^(kAbove + kRescaleThreshold), is within fp16 too.
constexpr float kAbove = 7.f;
constexpr float kLowest = -3e38f;         // a maximum before the first score: finite, so that no difference is NaN
constexpr int kRankMax = 256;             // entries that each CTA ranks by their work
constexpr int kFewWaves = 4;              // grids of up to this many CTAs an SM are ordered pair by pair
constexpr size_t kSplitRowBytes = kRankMax * 16 * 16;  // Split::rows, in a workspace
constexpr int kMinPartTiles = 2;          // key tiles of a run, at least, when a list is split
// Contexts up to which a CTA has one query tile. Measured with one and two tiles: 16 chunks of 300, 16 heads of 64, 28.5 and
// 35.2 us, on 700 keys before them 73.9 and 68.0; 12 chunks of 100 on 20, 32 q / 8 kv heads of 128, 17.0 and 19.7, 8 of 500
// 58.2 and 52.6. A chunk that fits one tile has one in any case (64 of 20 rows on 30 keys 19.5 and 31.9, on 2020 136 and 139).
__host__ __device__ constexpr int short_keys(int D) { return D == 64 ? 768 : 192; }

template <typename T, int D, int NQ>
struct Smem {
    static constexpr int per_sm = Roles<T, D, NQ>::per_sm, pieces = Roles<T, D, NQ>::pieces;
    static constexpr int k_stages = per_sm == 2 ? 128 / D : D == 128 ? 2 : 4, v_stages = per_sm == 2 ? 128 / D : D == 128 ? 3 : 4;
    static constexpr uint32_t tile = (D / 64) * kHalf;  // 128 x D fp16
    static constexpr uint32_t q = 0;                    // query tiles; in the end the outputs on their way
    static constexpr uint32_t k = q + NQ * pieces * tile;
    static constexpr uint32_t v = k + k_stages * tile;
    static constexpr uint32_t bars = v + v_stages * tile;
    static constexpr int num_bars = 2 * k_stages + 2 * v_stages + 8;
    static constexpr uint32_t misc = bars + num_bars * 8;  // tmem base, abort flag
    static constexpr uint32_t total = misc + 16 + 1024;
};

// Few CTAs with long key lists: each list in up to `parts` runs, one CTA each. Their outputs (fp32, not
// yet divided by the sums) and (reference, sum) of every row go to the workspace for the merge kernel.
struct Split {
    int32_t parts;
    int4* rows;  // per CTA of the unsplit grid: first row of q, rows of tile a, of tile b, runs (0: nothing to merge)
    float4* o;   // [CTA][parts][D / 4][2 * kRows]
    float2* ml;  // [CTA][parts][2 * kRows]
};

struct Args {
    void* out;
    const void* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* query_start_loc;
    int32_t max_blocks, num_kv_heads, G, num_blocks, sub_log2, cap_tokens, max_chunk;
    int32_t sub;       // pairs of query tiles of an entry's chunk, or 1: a whole sequence
    uint32_t inv_sub;  // x / sub = x inv_sub / 2^16
    float c1;          // |scale| log2 e; the sign goes to the queries
    bool negate;
    float v_scale;
    Split split;
    uint32_t* err;
    uint64_t wait_limit_ns;
    int32_t drill;  // the CTA with the longest list: the first K tile's barrier waits for 16 bytes that nothing brings
};

// Instruction descriptor for kind::f16 with fp16 A and B and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t b_mn_major) {
    return (1u << 4) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_halves(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ int32_t read_flag(uint32_t flag) {
    int32_t v;
    asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(flag) : "memory");
    return v;
}
// Bounded wait; kSleep > 0: polls are that many ns apart, so that the many warps that wait leave the
// issue slots to those that compute (the MMA warp, alone on the critical path, polls at once).
template <uint32_t kSleep>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, uint32_t flag, const Args& a) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int k = 0; k < 64; ++k) {
            if (kSleep > 0) asm volatile("nanosleep.u32 %0;" ::"r"(kSleep));
            if (mbar_try_wait(bar, parity)) return true;
        }
        if (read_flag(flag)) return false;
        if (global_timer_ns() - t0 > a.wait_limit_ns) {
            raise_error(a.err, PA_DEVERR_WAIT_TIMEOUT);
            asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(flag) : "memory");
            return false;
        }
    }
}

// 16 columns of the warp's tensor-memory lanes; the wait takes the registers too, so that no use of them moves above it.
__device__ __forceinline__ void ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void wait_x16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// 8 columns, likewise.
__device__ __forceinline__ void ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void wait_x8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// A key's codes and scales.
template <int D>
struct RawRow {
    uint4 codes[D / 32];
    uint32_t scales[D / 64];  // 4 scales a word
};

template <typename T, int D, int NQ, bool SPLIT>
__global__ void __launch_bounds__(Roles<T, D, NQ>::threads, Roles<T, D, NQ>::per_sm)
    prefill_fp4_kernel(const __grid_constant__ Args a) {
    using L_ = Smem<T, D, NQ>;
    using Roles = Roles<T, D, NQ>;
    constexpr int kUnpackWarps = Roles::unpack, kPieces = Roles::pieces;
    constexpr uint32_t kO = Roles::o;
    constexpr uint32_t kTile = L_::tile;
    constexpr int kKStages = L_::k_stages, kVStages = L_::v_stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L_::bars);
    uint64_t* k_full = bars;                // [kKStages] K tile stored (4 units)
    uint64_t* k_empty = k_full + kKStages;  // [kKStages] the QKs that read the stage are done
    uint64_t* v_full = k_empty + kKStages;  // [kVStages]
    uint64_t* v_empty = v_full + kVStages;  // [kVStages] the PVs that read the stage are done
    uint64_t* s_full = v_empty + kVStages;  // [2] S of query tile a / b written
    uint64_t* p_full = s_full + 2;          // [2] its P written (8 softmax warps)
    uint64_t* o_done = p_full + 2;          // [2] its last PV finished
    uint64_t* q_full = o_done + 2;          // both query tiles stored (8 softmax warps a tile)
    uint64_t* idle = q_full + 1;            // every MMA issued has finished
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L_::misc);
    const uint32_t abort_flag = smem_u32(smem + L_::misc + 4);
    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2;

    // ---- barriers and tensor memory, while the entry is found -----------------------------------------
    // per query tile and quadrant: the last key tile (+ 1) whose scores exceed a reference; the one whose wait has given up
    __shared__ int32_t grow_at[2][4], stopped[2][4];
    if (tid == 64) *reinterpret_cast<volatile int32_t*>(smem + L_::misc + 4) = 0;
    if (tid >= 96 && tid < 104) grow_at[tid >> 2 & 1][tid & 3] = stopped[tid >> 2 & 1][tid & 3] = 0;
    if (warp == 1 && lane < L_::num_bars) {  // each once: an object in use must not be initialised again
        uint64_t* bar = bars + lane;
        const bool four = bar < k_empty || (bar >= v_full && bar < v_empty);
        mbar_init(bar, bar >= p_full && bar < o_done ? 8 : four ? 4 : bar == q_full ? 8 * NQ : 1);
        fence_mbarrier_init();
    }
    if (warp == 0) {
        umma::tmem_alloc(tmem_holder, Roles::columns);
        umma::tmem_relinquish();
    }
    umma::fence_before_sync();
    auto leave = [&]() {  // a CTA without work: all threads have passed a barrier since the allocation
        if (warp == 0) {
            umma::fence_after_sync();
            umma::tmem_dealloc(*tmem_holder, Roles::columns);
        }
    };

    __shared__ int4 chosen[2];  // the entry's sequence, pair, first row of q, rows; length
    __shared__ union {  // one after the other
        alignas(16) uint32_t rank_key[kRankMax];  // the entries' work
        float row[2][kRows];                      // per query tile: what the two threads of a row tell one another
    } shared;
    // A CTA's entry: one pair of query tiles of a sequence (sub = the pairs of a chunk) or, sub = 1, a
    // whole sequence, whose pairs and heads follow one another. Entries with the most keys come first:
    // work that a long CTA leaves to the end of the grid keeps one SM busy and the others idle.
    const int32_t G = a.G, TT = kRows / G, Hq = G * a.num_kv_heads, sub = a.sub;
    const int32_t place = blockIdx.z, n_entries = gridDim.z, h = blockIdx.y;
    int32_t seq, pair, q0, C, L;
    auto entry = [&](int32_t i) {
        seq = sub > 1 ? static_cast<int32_t>(i * a.inv_sub >> 16) : i;  // i / sub, for i < 256 exact
        pair = sub - 1 - (i - seq * sub);                                // a sequence's last tokens come first
        q0 = __ldg(a.query_start_loc + seq);
        C = __ldg(a.query_start_loc + seq + 1) - q0;
        L = __ldg(a.seq_lens + seq);
    };
    if (n_entries > 1 && n_entries <= kRankMax) {
        uint32_t mine = 0;
        if (tid < n_entries) {
            entry(tid);
            const int32_t first = NQ * pair * TT, rows = sub > 1 ? min(NQ * TT, C - first) : C;
            const int32_t keys = rows <= 0 ? 0 : L - C + first + rows;  // up to the last row's own
            // 24 bits of keys (all of them up to 2^24 tokens), and the number: no two alike
            mine = static_cast<uint32_t>(max(keys, 0)) >> max(8 - __clz(a.cap_tokens), 0) << 8 | (kRankMax - 1 - tid);
        }
        if (tid < kRankMax) shared.rank_key[tid] = mine;
        __syncthreads();
        if (tid < n_entries) {
            int32_t rank = 0;
#pragma unroll 4
            for (int32_t u = 0; u < n_entries; u += 4) {
                const uint4 k = *reinterpret_cast<const uint4*>(shared.rank_key + u);
                rank += (k.x > mine) + (k.y > mine) + (k.z > mine) + (k.w > mine);
            }
            if (rank == place) {
                chosen[0] = make_int4(seq, pair, q0, C);
                chosen[1].x = L;
            }
        }
        __syncthreads();
        const int4 c0 = chosen[0];
        seq = c0.x, pair = c0.y, q0 = c0.z, C = c0.w, L = chosen[1].x;
    } else {
        entry(place);
        __syncthreads();
    }
    umma::fence_after_sync();
    if (sub == 1) pair = SPLIT ? 0 : gridDim.x - 1 - blockIdx.x;
    const int32_t cta = place * a.num_kv_heads + h;
    if (SPLIT && tid == 0 && blockIdx.x == 0) a.split.rows[cta] = make_int4(0, 0, 0, 0);
    if (C < 0 || C > a.max_chunk || C > L || L > a.cap_tokens) {
        if (tid == 0 && pair == 0) raise_error(a.err, PA_DEVERR_LEN_RANGE);
        leave();
        return;
    }
    const int32_t t0a = NQ * pair * TT;
    if (t0a >= C) {  // uniform over the CTA
        leave();
        return;
    }
    const int32_t t0b = t0a + TT, P0 = L - C;

    // ---- key tiles of the CTA, and of each query tile: up to its last row's own key ---------------
    const int32_t all_a = (P0 + min(t0a + TT, C) - 1) / kKeys + 1;
    const int32_t all_b = NQ == 2 && t0b < C ? (P0 + min(t0b + TT, C) - 1) / kKeys + 1 : 0;
    int32_t n_kv = max(all_a, all_b), base = 0, n_parts = 1;
    if constexpr (SPLIT) {  // this CTA takes one of up to split.parts equal runs of the list
        const int32_t most = max(min(a.split.parts, n_kv / kMinPartTiles), 1), share = (n_kv + most - 1) / most;
        n_parts = (n_kv + share - 1) / share;
        if (static_cast<int32_t>(blockIdx.x) >= n_parts) {  // uniform over the CTA
            leave();
            return;
        }
        base = blockIdx.x * share;
        n_kv = min(share, n_kv - base);
        if (tid == 0 && blockIdx.x == 0 && n_parts > 1)
            a.split.rows[cta] = make_int4(q0 + t0a, min(TT, C - t0a) * G, NQ == 2 ? max(min(TT, C - t0b), 0) * G : 0, n_parts);
    }
    const int32_t n_a = min(max(all_a - base, 0), n_kv), n_b = min(max(all_b - base, 0), n_kv);

    // ---- roles ------------------------------------------------------------------------------------
    const bool softmax_warp = group >= 1 && group <= 2 * NQ;
    // softmax: query tile, half of the key tile, TMEM lane quadrant, row
    const int32_t x = NQ == 2 ? (group - 1) & 1 : 0, half = (NQ == 2 ? (group - 1) >> 1 : group - 1) & 1, quad = warp & 3, r = tid & 127;
    const uint32_t inv_G = 65536u / static_cast<uint32_t>(G) + 1;  // i / G = i inv_G / 2^16 for i, G <= 128
    constexpr int kLanes = D / 8 * kPieces, kPer = 32 / kLanes, kLoads = 16 / kPer;  // lanes of a query row, rows of a load, loads
    // Unit u: K (bit 2 clear) or V of key tile u / 8, keys 32 (u % 4) ..; this warp has every kUnpackWarps-th.
    const int32_t u_first = group == 0 ? warp - 1 : warp - (4 + Roles::soft) + 3, n_units = 8 * n_kv;
    const int32_t* table = a.block_table + static_cast<int64_t>(seq) * a.max_blocks;
    auto key_at = [&](int32_t u) { return (base + (u >> 3)) * kKeys + (u & 3) * 32 + lane; };
    // block id of this lane's key of unit u; -1: no such key
    auto block_of = [&](int32_t u) -> int32_t {
        const int32_t key = key_at(u);
        if (u >= n_units || key >= L) return -1;
        return __ldg(table + (key >> (4 + a.sub_log2)));  // (checked when it is used, so that nothing waits for it here)
    };
    auto load = [&](int32_t u, int32_t block, RawRow<D>& raw) {
        const bool held = u < n_units && key_at(u) < L;
        if (held && (block < 0 || block >= a.num_blocks)) {
            raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
            block = 0;
        }
        if (!held) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) raw.codes[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) raw.scales[i] = 0u;
            return;
        }
        const int32_t key = key_at(u), page = key >> 4;
        const uint8_t* p = (u & 4 ? a.v_cache : a.k_cache) +
                           fp4_page_at(block, a.num_kv_heads, h, a.sub_log2, page & ((1 << a.sub_log2) - 1), D);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw.codes[i] = __ldg(reinterpret_cast<const uint4*>(p + (key & 15) * (D / 2)) + i);
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            raw.scales[i] = __ldg(reinterpret_cast<const uint32_t*>(p + fp4_scales_at(D) + (key & 15) * (D / 16)) + i);
    };
    const bool unpack_warp = !softmax_warp && warp != 0;
    // tensor memory columns: S of tile x at 128 x (the P of each half of its keys, fp16 pairs, overwrites the first
    // 32 of the half's 64 columns once read; in two pieces, 16 keys' pairs of both overwrite their 16 columns), O of tile x
    // at kO + 128 x
    const uint32_t tmem = *tmem_holder;

    if (!softmax_warp) fewer_registers<Roles::other_regs>();
    if (unpack_warp) {
        // ======================================== unpack ========================================
        if (a.drill && tid == 32 && place == 0 && h == 0 && (SPLIT || sub > 1 ? blockIdx.x == 0 : pair == 0))
            mbar_expect_tx(&k_full[0], 16u);  // (before this warp stores its unit of the tile)
        RawRow<D> raw;
        load(u_first, block_of(u_first), raw);
        int32_t block_n = block_of(u_first + kUnpackWarps);  // of the next unit
        auto unit = [&](int32_t u) -> bool {  // unpacks u, and sends for this warp's next unit
            const int32_t j = u >> 3, r0 = (u & 3) * 32 + lane;
            const bool is_v = u & 4;
            const int32_t nst = is_v ? kVStages : kKStages, st = j % nst, use = j / nst;
            if (use > 0) {
                const bool ok = wait_or_abort<40>(is_v ? &v_empty[st] : &k_empty[st], static_cast<uint32_t>(use - 1) & 1u, abort_flag, a);
                if (!__all_sync(0xffffffffu, ok)) return false;
            }
            uint8_t* tile = smem + (is_v ? L_::v : L_::k) + st * kTile;
#pragma unroll
            for (int g = 0; g < D / 16; ++g) {
                const uint32_t s2 = e4m3x2_halves(static_cast<uint16_t>(raw.scales[g / 4] >> (16 * (g / 2 % 2))));
                const uint32_t m = __byte_perm(s2, 0u, g % 2 ? 0x3232u : 0x1010u);
                const uint4 w = raw.codes[g / 2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t y[4];
                    fp4_halves(g % 2 ? (c ? w.w : w.z) : (c ? w.y : w.x), y);
                    const int chunk = 2 * g + c;
                    *reinterpret_cast<uint4*>(tile + (chunk >> 3) * kHalf + sw128_offset(r0, chunk & 7)) =
                        make_uint4(hmul2(y[0], m), hmul2(y[1], m), hmul2(y[2], m), hmul2(y[3], m));
                }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(is_v ? &v_full[st] : &k_full[st]);
            const int32_t block = block_n;
            block_n = block_of(u + 2 * kUnpackWarps);
            load(u + kUnpackWarps, block, raw);
            return true;
        };
#pragma unroll 1
        for (int32_t u = u_first; u < n_units; u += kUnpackWarps)
            if (!unit(u)) break;
    } else if (warp == 0) {
        // ======================================= MMA issuer =====================================
        if (umma::elect_one()) {
            // One thread issues every MMA (a commit tracks those of its own thread) and does all the waiting.
            constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, 0);  // Q, K both K-major
            constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, 1);    // P (TMEM), V MN-major
            const uint64_t dq0 = umma::smem_desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t dk0 = umma::smem_desc_sw128(smem_u32(smem + L_::k), 16, 1024);
            const uint64_t dv0 = umma::smem_desc_sw128(smem_u32(smem + L_::v), kHalf, 1024);
            int32_t ks = 0, vs = 0;  // stages of the K tile of the last QK, of V tile j
            uint32_t k_use = 0, v_use = 0;
            // (descriptors are stepped where they are used: kept for the whole loop, they do not fit the registers)
            auto here = [](uint64_t& d) { asm volatile("" : "+l"(d)); };
            auto qk = [&](int x) {
                uint64_t dq = dq0 + static_cast<uint64_t>(x) * (kPieces * kTile >> 4), dk = dk0 + static_cast<uint64_t>(ks) * (kTile >> 4);
                here(dq);
                here(dk);
#pragma unroll
                for (int c = kPieces - 1; c >= 0; --c)  // the second halves first: the sums are cut off, so the small ones come early
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        const uint64_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
                        umma::mma_bf16(tmem + x * 128, dq + (c * kTile >> 4) + off, dk + off, idesc_qk, s > 0 || c < kPieces - 1);
                    }
                umma::commit(&s_full[x]);
            };
            auto pv = [&](int x, bool acc) {
                uint64_t dv = dv0 + static_cast<uint64_t>(vs) * (kTile >> 4);
                here(dv);
#pragma unroll
                for (int c = kPieces - 1; c >= 0; --c)
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)  // 16 keys per instruction: 8 P columns
                        umma::mma_bf16_tmem_a(tmem + kO + x * 128, tmem + x * 128 + (k >> 2) * 64 + (k & 3) * (8 * kPieces) + 8 * c,
                                              dv + static_cast<uint64_t>(k * (2048 >> 4)), idesc_pv,
                                              (acc && kPieces == 1) || k > 0 || c < kPieces - 1);
            };
            auto wait_k = [&]() {
                const bool ok = wait_or_abort<0>(&k_full[ks], k_use & 1u, abort_flag, a);
                umma::fence_after_sync();
                return ok;
            };
            bool ok = wait_or_abort<0>(q_full, 0, abort_flag, a) && wait_k();
            if (ok) {
                if (n_a > 0) qk(0);
                if (n_b > 0) qk(1);
                umma::commit(&k_empty[ks]);
            }
            for (int32_t j = 0; j < n_kv && ok; ++j) {
                const bool more = j + 1 < n_kv;
                if (more && ++ks == kKStages) {
                    ks = 0;
                    ++k_use;
                }
                ok = wait_or_abort<0>(&v_full[vs], v_use & 1u, abort_flag, a);
                if (ok && j < n_a) {  // P written, S read
                    ok = wait_or_abort<0>(&p_full[0], j & 1, abort_flag, a);
                    umma::fence_after_sync();
                    if (ok) pv(0, j > 0);
                    if (ok && j + 1 == n_a) umma::commit(&o_done[0]);
                }
                if (ok && more) ok = wait_k();
                if (ok && j + 1 < n_a) qk(0);
                if (ok && j < n_b) {
                    ok = wait_or_abort<0>(&p_full[1], j & 1, abort_flag, a);
                    umma::fence_after_sync();
                    if (ok) pv(1, j > 0);
                    if (ok && j + 1 == n_b) umma::commit(&o_done[1]);
                }
                if (ok) umma::commit(&v_empty[vs]);
                if (ok && j + 1 < n_b) qk(1);
                if (ok && more) umma::commit(&k_empty[ks]);
                if (++vs == kVStages) {
                    vs = 0;
                    ++v_use;
                }
            }
            umma::commit(idle);  // arrives once every MMA issued above has finished
            mbar_wait_timeout(idle, 0, a.wait_limit_ns);
        }
    } else {
        // ==================================== queries, softmax ==================================
        more_registers<Roles::soft_regs>();
        const int32_t tl = static_cast<int32_t>(r * inv_G >> 16), g = r - tl * G;
        const int32_t t_row = (x ? t0b : t0a) + tl, n_x = x ? n_b : n_a;
        const bool row_valid = tl < TT && t_row < C;
        const int32_t pair_bar = 1 + x * 4 + quad;  // the barrier of the two warps that share 32 rows
        {  // this warp's 16 rows to fp16, 16 bytes a lane: times 2^-e, so that the row's largest magnitude lies in [2^14, 2^15) and
           // what is small next to it, or its second halves, within fp16's range
            const int32_t c = lane & (kLanes - 1);
            uint8_t* sq = smem + x * (kPieces * kTile);
            uint4 q_raw[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int32_t rr = quad * 32 + half * 16 + k * kPer + lane / kLanes, tt = static_cast<int32_t>(rr * inv_G >> 16);
                const int32_t t = (x ? t0b : t0a) + tt;
                q_raw[k] = make_uint4(0u, 0u, 0u, 0u);
                if (tt < TT && t < C)
                    q_raw[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (static_cast<int64_t>(q0 + t) * Hq + h * G + (rr - tt * G)) * D) +
                                     (lane & (kLanes - 1)));
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const uint32_t w[4] = {q_raw[k].x, q_raw[k].y, q_raw[k].z, q_raw[k].w};
                const int32_t rr = quad * 32 + half * 16 + k * kPer + lane / kLanes;
                int32_t field;  // 141 + e
                if constexpr (kPieces == 1) {
                    uint32_t top = 0u;  // magnitudes as bf16 bits, two at a time
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = max_u16x2(top, w[i] & 0x7fff7fffu);
#pragma unroll
                    for (int off = 1; off < kLanes; off <<= 1) top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, off));
                    field = static_cast<int32_t>(max(top & 0xffffu, top >> 16) >> 7);
                } else {
                    uint32_t top = 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = max(top, w[i] & 0x7fffffffu);
#pragma unroll
                    for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
                    field = static_cast<int32_t>(top >> 23);
                }
                const int32_t e = field == 255 ? 0 : max(field, 15) - 141;  // (not finite: as it is; rows below 2^-112: times 2^126)
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23), f = a.negate ? -down : down;
                if constexpr (kPieces == 1) {
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = pack_halves(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
                    *reinterpret_cast<uint4*>(sq + (c >> 3) * kHalf + sw128_offset(rr, c & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {  // 4 dims: half of a 16-byte piece in each tile
                    uint8_t* at = sq + (c >> 4) * kHalf + sw128_offset(rr, c >> 1 & 7) + (c & 1) * 8;
                    float y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = __uint_as_float(w[i]) * f;
                    const uint32_t o0 = pack_halves(y[0], y[1]), o1 = pack_halves(y[2], y[3]);
                    const float2 h0 = halves_to_floats(o0), h1 = halves_to_floats(o1);
                    *reinterpret_cast<uint2*>(at) = make_uint2(o0, o1);
                    *reinterpret_cast<uint2*>(at + kTile) = make_uint2(pack_halves(y[0] - h0.x, y[1] - h0.y), pack_halves(y[2] - h1.x, y[3] - h1.y));
                }
                if (c == 0) shared.row[x][rr] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        named_barrier(pair_bar, 64);
        const float c1 = fmaxf(a.c1 * shared.row[x][r], 1e-37f);  // (a hidden score of -inf times it stays -inf)
        named_barrier(pair_bar, 64);
        const int32_t pos = row_valid ? P0 + t_row : L - 1;  // (rows without a query: zeros that go nowhere)
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tmem_s = tmem + x * 128 + half * 64 + lane_off;
        const uint32_t tmem_o = tmem + kO + x * 128 + half * (D / 2) + lane_off;  // the columns that it rescales and writes
        float m_ref = kLowest, l_sum = 0.f;  // the reference is the same in both threads of a row
        bool ok = true;
        int32_t keys = 0;  // of this half, those that the row sees are below this
        // P = 2^(s c1 - m) in fp16 pairs, 16 keys at a time, the next 16 on their way; the weights wait in registers
        // until the tile's maximum is known. Returns their sum; over: the largest exponent.
        auto weights = [&](auto masked, float& over, uint32_t (&pk)[32]) -> float {
            const uint64_t scale2 = pack2(c1, c1), shift2 = pack2(-m_ref, -m_ref);
            uint64_t psum[2] = {0ull, 0ull};
            float top[2] = {-INFINITY, -INFINITY};
            uint32_t raw[2][8];
            ld_x8(tmem_s, raw[0]);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                wait_x8(raw[c & 1]);
                if (c < 7) ld_x8(tmem_s + (c + 1) * 8, raw[(c + 1) & 1]);
                if constexpr (decltype(masked)::value) {  // hidden keys: -inf, so that their weight is exactly 0
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c * 8 + i >= keys) raw[c & 1][i] = __float_as_uint(-INFINITY);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x0, x1;
                    unpack2(fma2(pack2(__uint_as_float(raw[c & 1][2 * e]), __uint_as_float(raw[c & 1][2 * e + 1])), scale2, shift2), x0, x1);
                    top[e & 1] = max3(top[e & 1], x0, x1);
                    const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
                    psum[e & 1] = add2(psum[e & 1], pack2(p0, p1));
                    pk[c * 4 + e] = pack_halves(p0, p1);
                }
            }
            over = fmaxf(top[0], top[1]);
            float s0, s1;
            unpack2(add2(psum[0], psum[1]), s0, s1);
            return s0 + s1;
        };
        // f(the first half's value, the second's) of this row, for both of its threads
        auto both = [&](auto f, float mine) -> float {
            volatile float* row = &shared.row[x][r];
            if (half == 1) *row = mine;
            named_barrier(pair_bar, 64);
            if (half == 0) *row = mine = f(mine, *row);
            named_barrier(pair_bar, 64);
            return half == 0 ? mine : *row;
        };
        // The row's largest score of this tile, over both halves: the reference moves there if it is more than 2^8
        // above. Returns what sums and outputs so far are worth under the new one.
        auto move_reference = [&]() -> float {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            uint32_t raw[16];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                ld_x16(tmem_s + c * 16, raw);
                wait_x16(raw);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c * 16 + i < keys) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(raw[i]));
            }
            const float mine = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c1;
            const float m = both([](float p, float q) { return fmaxf(p, q); }, mine);
            const float m_new = m > m_ref + (kAbove + kRescaleThreshold) ? m - kAbove : m_ref, alpha = exp2_approx(m_ref - m_new);
            m_ref = m_new;
            return alpha;
        };
        // The weights of a tile as sums of two halves, in the place of their scores, 16 keys at a time. Returns their sum.
        auto weights_in_place = [&]() -> float {
            uint64_t psum = 0ull;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t raw[16], o[16];
                ld_x16(tmem_s + c * 16, raw);
                wait_x16(raw);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float x0 = fmaf(__uint_as_float(raw[2 * e]), c1, -m_ref), x1 = fmaf(__uint_as_float(raw[2 * e + 1]), c1, -m_ref);
                    if (c * 16 + 2 * e >= keys) x0 = -INFINITY;  // hidden: weight 0
                    if (c * 16 + 2 * e + 1 >= keys) x1 = -INFINITY;
                    const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
                    psum = add2(psum, pack2(p0, p1));
                    o[e] = pack_halves(p0, p1);
                    const float2 held = halves_to_floats(o[e]);
                    o[8 + e] = pack_halves(p0 - held.x, p1 - held.y);
                }
                umma::st_32x32b_x16(tmem_s + c * 16, o);
            }
            float s0, s1;
            unpack2(psum, s0, s1);
            return s0 + s1;
        };
        // Two pieces: O so far, in registers. The MMAs cut their sums off, always towards zero, which over 8000 keys is 2e-5 of an
        // output; a tile's part by itself, added here with rounding, leaves 3e-7.
        float o_sum[kPieces == 2 ? D / 2 : 1];
#pragma unroll
        for (float& o : o_sum) o = 0.f;
        auto collect = [&]() {
            if constexpr (kPieces == 2) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[16];
                    ld_x16(tmem_o + c * 16, o);
                    wait_x16(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o_sum[c * 16 + i] += __uint_as_float(o[i]);
                }
            }
        };
        for (int32_t j = 0; j < n_x; ++j) {
            ok = wait_or_abort<20>(&s_full[x], j & 1, abort_flag, a);
            if (!__all_sync(0xffffffffu, ok) && lane == 0) *const_cast<volatile int32_t*>(&stopped[x][quad]) = j + 1;
            umma::fence_after_sync();
            keys = pos - ((base + j) * kKeys + half * 64) + 1;
            float alpha = 1.f, sum;
            if constexpr (kPieces == 1) {
                const bool masked = __any_sync(0xffffffffu, keys < 64);  // the last tiles
                float over = 0.f;
                uint32_t pk[32];
                if (__any_sync(0xffffffffu, m_ref == kLowest)) alpha = move_reference();  // a row's first keys (alike in both warps)
                sum = masked ? weights(std::true_type(), over, pk) : weights(std::false_type(), over, pk);
                if (__any_sync(0xffffffffu, over > kAbove + kRescaleThreshold) && lane == 0)
                    *const_cast<volatile int32_t*>(&grow_at[x][quad]) = j + 1;
                named_barrier(pair_bar, 64);
                // both warps leave at the same tile, so that each meets the other at every barrier: a stop that the other warp
                // has met since, a tile later, does not count yet
                ok = *const_cast<volatile int32_t*>(&stopped[x][quad]) != j + 1;
                if (!ok) break;
                if (*const_cast<volatile int32_t*>(&grow_at[x][quad]) == j + 1) {
                    alpha *= move_reference();
                    sum = masked ? weights(std::true_type(), over, pk) : weights(std::false_type(), over, pk);
                }
                umma::st_32x32b_x32(tmem_s, pk);
            } else {  // the maximum first (a barrier of both warps), then the weights
                if (j > 0) collect();  // the PV of tile j - 1 finished before S of tile j was committed
                alpha = move_reference();
                ok = *const_cast<volatile int32_t*>(&stopped[x][quad]) != j + 1;
                if (!ok) break;
                sum = weights_in_place();
            }
            l_sum = l_sum * alpha + sum;
            if constexpr (kPieces == 2) {
#pragma unroll
                for (float& o : o_sum) o *= alpha;
            } else if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                // O holds the tiles before under the old reference; the PV of tile j - 1 finished
                // before S of tile j was committed, so O can be rescaled now
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[16];
                    ld_x16(tmem_o + c * 16, o);
                    wait_x16(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    umma::st_32x32b_x16(tmem_o + c * 16, o);
                }
            }
            umma::wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x]);
        }
        if (ok && n_x > 0) ok = wait_or_abort<20>(&o_done[x], 0, abort_flag, a);
        ok = __all_sync(0xffffffffu, ok);
        umma::fence_after_sync();
        if (n_x > 0) collect();
        l_sum = both([](float p, float q) { return p + q; }, l_sum);
        // columns half (D / 2) + 16 c .. of the row's output; a tile that no key tile of this CTA concerns (a run that only
        // the other tile sees) has no MMAs
        auto output = [&](int c, uint32_t(&o)[16]) {
            if constexpr (kPieces == 2) {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(o_sum[c * 16 + i]);
            } else if (n_x > 0) {
                ld_x16(tmem_o + c * 16, o);
                wait_x16(o);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0u;
            }
        };
        if (SPLIT && n_parts > 1) {
            if (ok) {
                const int64_t run = static_cast<int64_t>(cta) * a.split.parts + blockIdx.x;
                if (half == 0) a.split.ml[run * (2 * kRows) + x * kRows + r] = make_float2(m_ref, l_sum);
                float4* po = a.split.o + (run * (D / 4) + half * (D / 8)) * (2 * kRows) + x * kRows + r;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[16];
                    output(c, o);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        po[(c * 4 + v) * (2 * kRows)] =
                            make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                        __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                }
            }
        } else if (kPieces == 2 && ok && n_x > 0) {
            const float inv = l_sum == 0.f ? 0.f : a.v_scale / l_sum;
            float* to = static_cast<float*>(a.out) + (static_cast<int64_t>(q0 + t_row) * Hq + h * G + g) * D + half * (D / 2);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[16];
                output(c, o);
                if (!row_valid) continue;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    reinterpret_cast<float4*>(to)[c * 4 + v] =
                        make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                    __uint_as_float(o[4 * v + 2]) * inv, __uint_as_float(o[4 * v + 3]) * inv);
            }
        } else if (ok && n_x > 0) {
            const float inv = l_sum == 0.f ? 0.f : a.v_scale / l_sum;
            // this warp's rows x D / 2 columns through its own part of the query tile, which no MMA reads any more, so
            // that the stores go out whole lines at a time (a row's 16-byte pieces in different banks, lane by lane)
            constexpr int kChunks = D / 16;
            uint8_t* stage = smem + x * kTile + (half * 4 + quad) * (32 * D);
            const int32_t turn = D == 128 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[16];
                output(c, o);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(o[v * 8 + k]) * inv;
                    *reinterpret_cast<uint4*>(stage + lane * D + ((c * 2 + v) ^ turn) * 16) =
                        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
                }
            }
            __syncwarp();
            const int64_t to = row_valid ? (static_cast<int64_t>(q0 + t_row) * Hq + h * G + g) * D + half * (D / 2) : -1;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                const int32_t i = k * 32 + lane, rr = i / kChunks, c = i % kChunks;
                const int64_t off = __shfl_sync(0xffffffffu, to, rr);
                const int32_t t = D == 128 ? rr & 7 : (rr >> 1) & 3;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * D + (c ^ t) * 16);
                if (off >= 0) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + off + c * 8) = v;
            }
        }
    }

    // ---- wind down: the MMAs have retired (warp 0 waited for them) before tensor memory goes ------
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, Roles::columns);
    }
}

// Merges the runs of split key lists. Grid: four columns of head_dim x CTA of the unsplit grid; a thread has one row of
// the CTA's two tiles.
template <typename T, int D>
__global__ void __launch_bounds__(2 * kRows) prefill_fp4_merge_kernel(T* __restrict__ out,
                                                                      const __grid_constant__ Split split,
                                                                      int32_t num_kv_heads, int32_t G, float v_scale) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t c4 = blockIdx.x, cta = blockIdx.y, R = threadIdx.x;
    const int4 rows = split.rows[cta];
    const int32_t rr = R & (kRows - 1), n = R < kRows ? rows.y : rows.z;
    if (rows.w == 0 || rr >= n) return;
    const float2* ml = split.ml + static_cast<int64_t>(cta) * split.parts * (2 * kRows) + R;
    const float4* po = split.o + (static_cast<int64_t>(cta) * split.parts * (D / 4) + c4) * (2 * kRows) + R;
    float M = kLowest, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int32_t p = 0; p < rows.w; ++p) M = fmaxf(M, ml[p * (2 * kRows)].x);
#pragma unroll 8
    for (int32_t p = 0; p < rows.w; ++p) {
        const float2 x = ml[p * (2 * kRows)];
        const float4 o = po[static_cast<int64_t>(p) * (D / 4) * (2 * kRows)];
        const float w = exp2_approx(x.x - M);
        den = fmaf(w, x.y, den);
        acc.x = fmaf(w, o.x, acc.x), acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z), acc.w = fmaf(w, o.w, acc.w);
    }
    const float inv = den == 0.f ? 0.f : v_scale / den;
    const int32_t h = cta % num_kv_heads, TT = kRows / G, tt = rr / G, t = (R < kRows ? 0 : TT) + tt;
    T* to = out + (static_cast<int64_t>(rows.x + t) * G * num_kv_heads + h * G + (rr - tt * G)) * D + c4 * 4;
    if constexpr (std::is_same<T, float>::value)
        *reinterpret_cast<float4*>(to) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    else
        *reinterpret_cast<uint2*>(to) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// Grids of few waves are ordered pair by pair, others sequence by sequence.
bool few_waves(int64_t entries, int32_t num_kv_heads, int ctas_per_sm, int num_sms) {
    return entries <= kRankMax && entries * num_kv_heads <= static_cast<int64_t>(kFewWaves) * ctas_per_sm * num_sms;
}

template <typename T, int D, int NQ, bool SPLIT>
cudaError_t launch_impl(const PrefillArgs& p, float v_scale, const PrefillScoredPlan& plan, void* workspace, int num_sms,
                        cudaStream_t stream) {
    cudaError_t e = allow_smem<prefill_fp4_kernel<T, D, NQ, SPLIT>>(static_cast<int>(Smem<T, D, NQ>::total));
    if (e != cudaSuccess) return e;
    Args a{};
    a.out = p.out;
    a.q = p.q;
    a.k_cache = static_cast<const uint8_t*>(p.k_cache);
    a.v_cache = static_cast<const uint8_t*>(p.v_cache);
    a.block_table = p.block_table;
    a.seq_lens = p.seq_lens;
    a.query_start_loc = p.query_start_loc;
    a.max_blocks = p.max_blocks_per_seq;
    a.num_kv_heads = p.num_kv_heads;
    a.G = p.num_q_heads / p.num_kv_heads;
    a.num_blocks = p.num_blocks;
    a.sub_log2 = block_size_log2(p.block_size) - 4;
    a.cap_tokens = min(table_tokens(p.max_blocks_per_seq, a.sub_log2), p.max_seq_len);
    a.max_chunk = p.max_chunk_len;
    a.c1 = fabsf(p.scale) * kLog2e;
    a.negate = p.scale < 0.f;
    a.v_scale = v_scale;
    a.err = p.err;
    const WaitDrill drill = wait_drill();
    a.wait_limit_ns = drill.limit_ns;
    a.drill = drill.kind == kDrillPrefillKTile ? 1 : 0;
    const int32_t TT = kRows / a.G, pairs = (p.max_chunk_len - 1) / (NQ * TT) + 1;  // (rounded up, whatever the bound)
    const int64_t entries = static_cast<int64_t>(pairs) * p.num_seqs;
    const bool by_pair = few_waves(entries, p.num_kv_heads, Roles<T, D, NQ>::per_sm, num_sms);
    a.sub = by_pair ? pairs : 1;
    a.inv_sub = 65536u / a.sub + 1;
    const dim3 grid(SPLIT ? plan.parts : by_pair ? 1 : pairs, p.num_kv_heads, p.num_seqs * a.sub);
    if (SPLIT) {
        char* ws = static_cast<char*>(workspace);
        a.split.parts = plan.parts;
        a.split.rows = reinterpret_cast<int4*>(ws + kScoredCounterBytes);
        a.split.o = reinterpret_cast<float4*>(ws + kScoredCounterBytes + kSplitRowBytes);
        a.split.ml = reinterpret_cast<float2*>(a.split.o + entries * p.num_kv_heads * plan.parts * (D / 4) * (2 * kRows));
    }
    prefill_fp4_kernel<T, D, NQ, SPLIT><<<grid, Roles<T, D, NQ>::threads, Smem<T, D, NQ>::total, stream>>>(a);
    e = cudaGetLastError();
    if (!SPLIT || e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];  // the merge's CTAs may be set up while the last runs end
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / 4, static_cast<unsigned>(entries * p.num_kv_heads));
    cfg.blockDim = dim3(2 * kRows);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_fp4_merge_kernel<T, D>, static_cast<T*>(a.out), a.split, p.num_kv_heads, a.G, v_scale);
}

}  // namespace

PrefillScoredPlan plan_prefill_fp4(int32_t S, int32_t max_chunk, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_len,
                                   pa_dtype dtype, int num_sms) {
    PrefillScoredPlan plan{1, 2, 0};
    if (Hq / Hkv > kRows) return plan;
    const int32_t TT = kRows / (Hq / Hkv);
    if (dtype == PA_F32 || max_chunk <= TT || max_len <= short_keys(D)) plan.tiles = 1;
    const int64_t most = static_cast<int64_t>(max_len / kKeys + 1) / kMinPartTiles;  // runs of the longest list
    if (most < 2) return plan;
    // room for a wave of CTAs, whatever the chunks: a workspace serves every call up to its max_len
    plan.workspace_bytes = kScoredCounterBytes + kSplitRowBytes + static_cast<size_t>(num_sms) * (2 * kRows) * (D * 4 + 8);
    if (S < 1 || max_chunk < 1) return plan;
    const int32_t of_split = (dtype == PA_F32 ? 1 : 2) * TT;  // rows of a CTA whose keys are split
    const int64_t entries = (static_cast<int64_t>(max_chunk) + of_split - 1) / of_split * S;
    if (few_waves(entries, Hkv, 1, num_sms))  // one wave of CTAs, each with kMinPartTiles key tiles at least
        plan.parts = static_cast<int32_t>(max(min(num_sms / (entries * Hkv), most), static_cast<int64_t>(1)));
    return plan;
}

bool prefill_fp4_tc_ok(const PrefillArgs& a, const DeviceInfo& dev) {
    return a.num_q_heads / a.num_kv_heads <= kRows && a.num_seqs <= 65535 &&
           a.num_kv_heads <= 65535 && static_cast<int>(Smem<__nv_bfloat16, 128, 2>::total) <= dev.max_smem_optin;
}

cudaError_t launch_prefill_fp4_tc(const PrefillArgs& a, float v_scale, const PrefillScoredPlan& plan, void* workspace,
                                  int num_sms, cudaStream_t stream) {
    auto go = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (a.dtype == PA_F32)
            return plan.parts > 1 ? launch_impl<float, D, 1, true>(a, v_scale, plan, workspace, num_sms, stream)
                                  : launch_impl<float, D, 1, false>(a, v_scale, plan, workspace, num_sms, stream);
        using T = __nv_bfloat16;
        if (plan.parts > 1) return launch_impl<T, D, 2, true>(a, v_scale, plan, workspace, num_sms, stream);
        return plan.tiles == 1 ? launch_impl<T, D, 1, false>(a, v_scale, plan, workspace, num_sms, stream)
                               : launch_impl<T, D, 2, false>(a, v_scale, plan, workspace, num_sms, stream);
    };
    return a.head_dim == 128 ? go(std::integral_constant<int, 128>()) : go(std::integral_constant<int, 64>());
}

}  // namespace pa
