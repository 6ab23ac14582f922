// Scored chunked prefill on the 5th-generation tensor cores (bf16, head_dim 64 or 128, up to 128 q
// heads per kv head): attention of a chunk of new rows over the paged pool with scores that are
// capped by a tanh, biased by distance or masked (window, visible prefix, document start).
//
// One CTA computes two 128-row query tiles (a, b) of one (sequence, kv head), or one tile on short
// contexts and of short chunks (short_keys): row r of a tile is token r / G, q head r % G of the G heads
// that share the kv head, so every K/V tile is read once for both. Keys come in tiles of 128, and only
// the tiles that hold a key some row of the CTA sees (TileList: the prefix's tiles, then the window's).
// Of a CTA of two tiles (one tile: 8 softmax warps, then the same three):
//   warp 16    - K producer, warp 18 - V producer: block ids 32 pages ahead, TMA copies of 16-token
//                pages (128-byte swizzle) into rings of key tiles;
//   warp 17    - tensor-memory owner and MMA issuer: S = Q K^T, O += P V with P from tensor memory,
//                in the order PV_a(j), QK_a(j+1), PV_b(j), QK_b(j+1), so that the tensor cores
//                serve one query tile while the other one's softmax runs;
//   warps 0-15 - scores and softmax, two threads per query row, each on 64 of the tile's 128 keys
//                (four warps a scheduler to cover the arithmetic's and tensor memory's latencies).
//
// Chains of S -> softmax -> P -> P V -> next S run independently of one another: where a row's keys need
// no common maximum there are four, one per query tile and half of the key tile (64 keys), else two.
//
// Scores. Variants of the score arithmetic (Mode), all in the log2 domain:
//   plain      arg = s c1;                       online maximum, two passes over S
//   cap        arg = s Q(s^2) - ref;             no maximum: see below, one pass over S, four chains
//   distance   arg = s c1 - slope |p - j|;       online maximum, two passes
//   both       arg = s Q(s^2) - slope |p - j| - ref(row);  as cap
//   general    caps beyond the range of the fixed reference: online maximum, two passes, tanh by the identity
//   large cap  caps above kMaxIdentityCap: as general, small scores by the polynomial of scored.cuh
// At head_dim 64 tensor memory has room for an output per half of the keys: the modes with maxima then
// run four chains too, each half with its own maximum and output, merged at the end (8 sequences of 100
// to 1000 new rows on up to 2500 keys, 16 heads: 65.7 us, two chains 67.8).
// A capped score lies in [-cap, cap], so the weights 2^(arg - ref) against the fixed reference
// ref = cap log2(e) / 2 lie in [2^-112, 2^37] for caps up to kMaxFixedCap: no running maximum, no
// second pass over S and no rescaling of O are needed. tanh is the odd polynomial x Q(x^2) of degree
// 7, fitted to tanh on |x| <= 0.6 by Remez's minimax method (absolute error 2^-20.7, that times cap
// in the score, below the 2^-9 of the bf16 weights), evaluated on the FMA pipes two elements an
// instruction; a warp whose 32 scores of a row block hold a larger one takes
// tanh x = 1 - 2 / (1 + 2^(2 x log2 e)) for that block (absolute error 2^-20). P is rounded to bf16, the
// type in which the tensor cores multiply it by V (fp32 accumulation; the sums add the fp32 weights).
//
// Bound: the tensor cores, then the exponentials. 16 sequences of 512 new rows on 512 to 4608 keys, 32 q /
// 8 kv heads of 128, cap 50: 293 us, 1.06 PFLOP/s over visible pairs (54 % of the measured bf16 rate; a key
// tile takes 1.8 us against 1.35 of MMA time, its 64-wide S products being bound by shared memory), of
// which 20 % goes to each CTA's start (3 us), first S (1.5) and end (3.5). Forms that were slower: one
// persistent CTA per SM over equal cuts of all key tiles (399), key tiles sent for before the CTA's first
// barrier (304), raw maxima in pass one (no gain).
//
// Few rows on many keys: the key list is split (Split) so that a wave of CTAs shares it, and a second
// kernel merges their outputs.
//
// V rows of keys that no row of the CTA sees are zeroed in shared memory before P V (their pool
// cells may hold anything); their scores are masked. Every wait is bounded; a timeout sets
// PA_DEVERR_WAIT_TIMEOUT and the CTA winds down.
#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "pa_internal.h"
#include "pa_tcgen05.cuh"
#include "scored.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;  // query rows per tile (M)
constexpr int kKeys = 128;  // keys per key tile (N of S = Q K^T, K of O += P V)
// Warps of a CTA of NQ query tiles: softmax, K producer, MMA issuer, V producer.
template <int NQ>
struct Warps {
    static constexpr int soft = 8 * NQ, k = soft, mma = soft + 1, v = soft + 2, threads = 32 * (soft + 3);
};
constexpr uint32_t kHalf = 16384;         // 128 rows x 128 bytes (64 bf16 columns)
constexpr float kRescaleThreshold = 8.f;  // log2 units: O is rescaled only when the maximum grows by more
constexpr int kRankMax = 256;             // entries that each CTA ranks by their work
// Grids of up to this many CTAs an SM (CTAs without tokens counted) are ordered pair by pair. Measured at
// 512 CTAs of 1 to 16 key tiles: 58 us, against 65 ordered by sequence; at 864 CTAs of 1 to 3 key
// tiles, 504 of them without tokens: 49 us against 43, as ranking costs each CTA 0.6 us.
constexpr int kFewWaves = 4;
constexpr size_t kSplitRowBytes = kRankMax * 16 * 16;  // Split::rows, in a workspace
// Key tiles of a run, at least, when a list is split. Measured, 16 rows of one sequence on 4096 keys, 8 kv
// heads of 128: 16.4 us with 2, 17.7 with 4, 25.7 with 8, 63.8 not split; 256 rows on 32768 keys: 154 us, not
// split 531.
constexpr int kMinPartTiles = 2;
// Query tiles of a CTA: one, with two CTAs on an SM that cover each other's start and end, where one tile holds
// a chunk (64 chunks of 20 rows, 32 q / 8 kv heads of 128: on 30 keys 24.3 us against 38.1 with two tiles, on 2020
// keys 109 against 149) or the contexts are short (16 chunks of 300, 16 heads of 64: 33.1 against 40.0; 12 chunks
// of 100 on 120 keys, heads of 128: 12.8 against 19.0); else two, which share each K and V tile (16 chunks of 512
// on up to 4608 keys: 293 us, with one tile 419; the two meet near 1000 keys at head_dim 64, 200 at 128).
__host__ __device__ constexpr int short_keys(int D) { return D == 64 ? 768 : 192; }
// Caps with a fixed reference: 1.5 cap log2(e) <= 112. Measured, 16 sequences of 512 new rows on 2512 keys, 32 q / 8
// kv heads of 128: cap 50 302 us, not capped 330, cap 52 (general) 720.
constexpr float kMaxFixedCap = 51.f;
constexpr float kTopWeight = 48.f;  // with a distance bias: the largest weight's exponent

constexpr uint32_t kSleepProducer = 200, kSleepSoftmax = 40;  // ns between polls

// Caps up to which the identity alone serves: its error, 2^-20 cap, is then an eighth of the rounding of a weight to
// bf16. Measured, 16 sequences of 512 new rows on 2512 keys, 32 q / 8 kv heads of 128, scores of a few units: 728 us,
// with the polynomial for small scores 890; with scores that reach the cap 748 and 1419.
constexpr float kMaxIdentityCap = 256.f;

enum Mode : int { kPlain = 0, kCap = 1, kDistance = 2, kCapDistance = 3, kGeneral = 4, kLargeCap = 5 };

template <int D, int NQ>
struct Smem {
    static constexpr int k_stages = NQ == 1 ? 128 / D : D == 128 ? 3 : 4;
    static constexpr int v_stages = NQ == 1 ? 128 / D : D == 128 ? 2 : 4;
    static constexpr uint32_t tile = (D / 64) * kHalf;  // 128 x D bf16
    static constexpr uint32_t q = 0;                    // query tiles
    static constexpr uint32_t k = q + NQ * tile;
    static constexpr uint32_t v = k + k_stages * tile;
    static constexpr uint32_t bars = v + v_stages * tile;
    static constexpr int num_bars = 2 * k_stages + 2 * v_stages + 20;
    static constexpr uint32_t misc = bars + num_bars * 8;  // tmem base, abort flag
    static constexpr uint32_t total = misc + 16 + 1024;
};

// Keys that some valid row of one query tile sees: the two spans' unions.
struct SpanUnion {
    int32_t a0, a1, b0, b1;
    __device__ __forceinline__ bool covers(int32_t lo, int32_t hi) const {
        return (lo >= a0 && hi <= a1) || (lo >= b0 && hi <= b1);
    }
};

// Key tiles walked by the CTA: n_a from first_a, the rest from first_b.
struct TileList {
    int32_t first_a, n_a, first_b, n;
    int32_t base = 0;  // list position that the CTA's part begins with; positions below count from it
    __device__ __forceinline__ int32_t tile(int32_t i) const {
        i += base;
        return i < n_a ? first_a + i : first_b + (i - n_a);
    }
    __device__ __forceinline__ int32_t position(int32_t t) const {
        return (t < first_a + n_a ? t - first_a : n_a + (t - first_b)) - base;
    }
};

__device__ __forceinline__ TileList tile_list(const SpanUnion& u) {
    TileList l;
    l.first_a = u.a0 < u.a1 ? u.a0 / kKeys : 0;
    l.n_a = u.a0 < u.a1 ? (u.a1 + kKeys - 1) / kKeys - l.first_a : 0;
    l.first_b = u.b0 / kKeys;
    if (l.n_a > 0) l.first_b = max(l.first_b, l.first_a + l.n_a);
    const int32_t end = u.b0 < u.b1 ? (u.b1 + kKeys - 1) / kKeys : 0;
    l.n = l.n_a + max(0, end - l.first_b);
    return l;
}

__device__ __forceinline__ SpanUnion join(const SpanUnion& x, const SpanUnion& y) {
    SpanUnion u = x;
    if (y.a0 < y.a1) {
        u.a0 = x.a0 < x.a1 ? min(x.a0, y.a0) : y.a0;
        u.a1 = x.a0 < x.a1 ? max(x.a1, y.a1) : y.a1;
    }
    if (y.b0 < y.b1) {
        u.b0 = x.b0 < x.b1 ? min(x.b0, y.b0) : y.b0;
        u.b1 = x.b0 < x.b1 ? max(x.b1, y.b1) : y.b1;
    }
    return u;
}

// Few CTAs with long key lists: each list in up to `parts` runs, one CTA each. Their outputs (fp32, not
// yet divided by the sums) and (reference, sum) of every row go to the workspace for the merge kernel.
struct Split {
    int32_t parts;
    int4* rows;  // per CTA of the unsplit grid: first row of q, rows of tile a, of tile b, runs (0: nothing to merge)
    float4* o;   // [CTA][parts][D / 4][2 * kRows]
    float2* ml;  // [CTA][parts][2 * kRows]
};

// Score constants, log2 domain.
struct TcScore {
    float c1;       // scale log2 e
    float q[4];     // s Q(s^2) = cap log2(e) tanh(s scale / cap), coefficients of s, s^3, ..
    float s2_max;   // s^2 up to which the polynomial holds
    float two_k;    // 2 log2(e) scale / cap
    float cap_l2;   // cap log2 e
    float ref;      // fixed reference
    int32_t window;
    const float* slopes;
    const int32_t* key_start;
    const int32_t* prefix_len;
    bool causal;  // rows inside the prefix see no key behind themselves
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// The pair (x, x) of a value that every lane holds, through a shuffle: the compiler then keeps it in
// vector registers instead of moving it out of uniform ones for every group of keys.
__device__ __forceinline__ uint64_t hold2(float x) {
    const float v = __shfl_sync(0xffffffffu, x, 0);
    return pack2(v, v);
}
// Columns 2 e, 2 e + 1 of a group of 16 scores.
__device__ __forceinline__ uint64_t raw_pair(const uint32_t (&r)[16], int e) {
    return pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Floats as integers of the same order (no NaN), and back.
__device__ __forceinline__ int32_t ordered(float x) {
    const int32_t b = __float_as_int(x);
    return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int32_t b) { return __int_as_float(b ^ (b >> 31 & 0x7fffffff)); }

// 32 columns of the warp's tensor-memory lanes, and the wait that makes them valid, as one
// instruction group: nothing can use the registers before the wait.
__device__ __forceinline__ void ld_wait_x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// 16 columns; the wait takes the registers too, so that no use of them moves above it.
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

__device__ __forceinline__ void st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

__device__ __forceinline__ void sleep_ns(uint32_t ns) { asm volatile("nanosleep.u32 %0;" ::"r"(ns)); }
__device__ __forceinline__ int32_t read_flag(uint32_t flag) {
    int32_t v;
    asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(flag) : "memory");
    return v;
}
// Bounded wait; kSleep > 0: polls are that many ns apart, so that the many warps that wait leave the
// issue slots to those that compute (the MMA warp, alone on the critical path, polls at once).
template <uint32_t kSleep>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, uint32_t flag, uint32_t* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int k = 0; k < 64; ++k) {
            if (kSleep > 0) sleep_ns(kSleep);
            if (mbar_try_wait(bar, parity)) return true;
        }
        if (read_flag(flag)) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            raise_error(err, PA_DEVERR_WAIT_TIMEOUT);
            asm volatile("st.volatile.shared.s32 [%0], 1;" ::"r"(flag) : "memory");
            return false;
        }
    }
}

__device__ __forceinline__ void cp_async16(void* smem_dst, const void* src, bool zero) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(src),
                 "r"(zero ? 0 : 16)
                 : "memory");
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Bits i of a 32-key group whose keys base + i lie in [lo, hi).
__device__ __forceinline__ uint32_t span_bits(int32_t base, int32_t lo, int32_t hi) {
    const int32_t l = min(max(lo - base, 0), 32), h = min(max(hi - base, 0), 32);
    if (h <= l) return 0u;
    return (h == 32 ? 0xffffffffu : (1u << h) - 1u) & ~(l == 32 ? 0xffffffffu : (1u << l) - 1u);
}

template <int D, int MODE, int NQ, bool SPLIT>
__global__ void __launch_bounds__(Warps<NQ>::threads, 3 - NQ) prefill_scored_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ q, const int32_t* __restrict__ block_table,
    int32_t max_blocks, const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ query_start_loc,
    int32_t num_kv_heads, int32_t G, int32_t num_blocks, int32_t sub_log2, int32_t cap_tokens, int32_t max_chunk,
    int32_t sub, uint32_t inv_sub, const __grid_constant__ Split split, const __grid_constant__ TcScore sc, uint32_t* err) {
    using L_ = Smem<D, NQ>;
    constexpr int kSoftWarps = Warps<NQ>::soft, kKWarp = Warps<NQ>::k, kMmaWarp = Warps<NQ>::mma, kVWarp = Warps<NQ>::v;
    constexpr int kSoftThreads = 32 * kSoftWarps;
    constexpr uint32_t kO = NQ * 128;  // first tensor-memory column of O
    constexpr uint32_t kTile = L_::tile;
    constexpr int kKStages = L_::k_stages, kVStages = L_::v_stages;
    constexpr int kHalves = D / 64;
    // Chains of S -> softmax -> P -> PV -> next S that run independently of one another: one per query
    // tile, or, when no maximum ties the keys of a row together, one per query tile and half of the
    // key tile (chain c: query tile c & 1, half c >> 1), so that more MMA and softmax work overlaps.
    constexpr bool kFixed = MODE == kCap || MODE == kCapDistance;  // fixed reference
    constexpr bool kSplit = kFixed || D == 64;
    constexpr bool kOwnO = kSplit && !kFixed;  // each half of the keys has its own O and maximum
    constexpr int kChains = kSplit ? 2 * NQ : NQ;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L_::bars);
    uint64_t* k_full = bars;                // [kKStages] K tile landed
    uint64_t* k_empty = k_full + kKStages;  // [kKStages] the QKs that read the stage are done
    uint64_t* v_full = k_empty + kKStages;  // [kVStages]
    uint64_t* v_empty = v_full + kVStages;  // [kVStages] the PVs that read the stage are done
    uint64_t* s_full = v_empty + kVStages;  // [kChains] S of the chain written
    uint64_t* p_full = s_full + 4;          // [kChains] its P written (each softmax warp of the chain)
    uint64_t* o_done = p_full + 4;          // [2] last PV of tile a / b finished
    uint64_t* q_full = o_done + 2;          // query tiles in shared memory
    uint64_t* idle = q_full + 1;            // every MMA issued has finished
    uint64_t* mx_full = idle + 1;           // [2][4] both halves' maxima of a tile's 32 rows stored
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L_::misc);
    const uint32_t abort_flag = smem_u32(smem + L_::misc + 4);

    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ int4 chosen[2];  // the item's sequence, pair, first row of q, rows; length, prefix
    __shared__ int32_t red[2][4];    // per query tile: min a0, max a1, min b0, max b1
    __shared__ uint32_t seen_own[8];  // documents: the CTA's own positions that some row sees
    __shared__ union {  // one after the other
        alignas(16) uint32_t rank_key[kRankMax];  // the items' work
        int32_t row_top[2][kRows];                // per query tile: the rows' largest score so far, as an ordered integer
    } shared;
    // A CTA's entry: one pair of query tiles of a sequence (sub = the pairs of a chunk) or, sub = 1, a
    // whole sequence, whose pairs and heads follow one another. Entries with the most keys come first:
    // work that a long CTA leaves to the end of the grid keeps one SM busy and the others idle.
    const int32_t TT = kRows / G, Hq = G * num_kv_heads;
    const int32_t place = blockIdx.z, n_entries = gridDim.z, h = blockIdx.y;
    int32_t seq, pair, q0, C, L, prefix = 0;
    auto entry = [&](int32_t i) {
        seq = sub > 1 ? static_cast<int32_t>(i * inv_sub >> 16) : i;  // i / sub, for i < 256 exact
        pair = sub - 1 - (i - seq * sub);                              // a sequence's last tokens come first
        q0 = __ldg(query_start_loc + seq);
        C = __ldg(query_start_loc + seq + 1) - q0;
        L = __ldg(seq_lens + seq);
        if (sc.prefix_len) prefix = __ldg(sc.prefix_len + seq);
    };
    if (n_entries > 1 && n_entries <= kRankMax) {
        uint32_t mine = 0;
        if (tid < n_entries) {
            entry(tid);
            const int32_t first = NQ * pair * TT, rows = sub > 1 ? min(NQ * TT, C - first) : C;
            int32_t keys = L - C + first + rows;  // up to the last row's own
            if (sc.window > 0) keys = min(keys, min(sc.window, cap_tokens) + rows + min(max(prefix, 0), cap_tokens));
            if (rows <= 0) keys = 0;
            // 24 bits of keys (all of them up to 2^24 tokens), and the number: no two alike
            mine = static_cast<uint32_t>(max(keys, 0)) >> max(8 - __clz(cap_tokens), 0) << 8 | (kRankMax - 1 - tid);
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
                chosen[1] = make_int4(L, prefix, 0, 0);
            }
        }
        __syncthreads();
        const int4 c0 = chosen[0], c1 = chosen[1];
        seq = c0.x, pair = c0.y, q0 = c0.z, C = c0.w, L = c1.x, prefix = c1.y;
    } else {
        entry(place);
    }
    if (sub == 1) pair = SPLIT ? 0 : gridDim.x - 1 - blockIdx.x;
    const int32_t cta = place * num_kv_heads + h;
    if (SPLIT && tid == 0 && blockIdx.x == 0) split.rows[cta] = make_int4(0, 0, 0, 0);
    if (C < 0 || C > max_chunk || C > L || L > cap_tokens) {
        if (tid == 0 && pair == 0) raise_error(err, PA_DEVERR_LEN_RANGE);
        return;
    }
    const int32_t t0a = NQ * pair * TT, t0b = t0a + TT;
    if (t0a >= C) return;  // uniform over the CTA
    const int32_t P0 = L - C;

    // ---- rows of the softmax threads --------------------------------------------------------------
    const bool softmax_warp = warp < kSoftWarps;
    const int32_t xq = NQ == 2 ? (warp >> 2) & 1 : 0, half = (NQ == 2 ? warp >> 3 : warp >> 2) & 1;  // query tile and key half of a softmax warp
    const int32_t quad = warp & 3;                                // its TMEM lane quadrant
    const int32_t r = quad * 32 + lane;
    const uint32_t inv_G = 65536u / static_cast<uint32_t>(G) + 1;  // x / G = x inv_G / 2^16 for x, G <= 128
    const int32_t tl = static_cast<int32_t>(r * inv_G >> 16), g = r - tl * G;
    const int32_t t_row = (xq ? t0b : t0a) + tl;
    const bool row_valid = softmax_warp && tl < TT && t_row < C;
    const int32_t pos = P0 + t_row;
    // ---- query tiles: 16-byte copies into the swizzled K-major layout; rows without a query zero
    if (softmax_warp) {
        const int32_t ti = half * 128 + (tid & 127);
        uint8_t* sq = smem + xq * kTile;
        constexpr int kChunks = D / 8;  // 16-byte chunks of a row
        const int32_t t0 = xq ? t0b : t0a;
#pragma unroll
        for (int k = 0; k < kRows * kChunks / 256; ++k) {
            const int32_t i = ti + k * 256;
            const int32_t rr = i / kChunks, c16 = i % kChunks;
            const int32_t tt = static_cast<int32_t>(rr * inv_G >> 16), t = t0 + tt;
            const bool in = tt < TT && t < C;
            const __nv_bfloat16* src =
                in ? q + (static_cast<int64_t>(q0 + t) * Hq + h * G + (rr - tt * G)) * D + c16 * 8 : q;
            cp_async16(sq + (c16 >> 3) * kHalf + sw128_offset(rr, c16 & 7), src, !in);
        }
    }
    // ---- keys that the rows see ------------------------------------------------------------------
    KeySpans row{0, 0, 0, 0};
    if (row_valid)
        row = key_spans(L, pos, sc.key_start ? __ldg(sc.key_start + q0 + t_row) : 0, prefix, sc.window, sc.causal);
    SpanUnion ux[NQ];
    if (sc.key_start == nullptr) {  // rows' spans move with their position: the first and the last row tell
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int32_t t0 = x ? t0b : t0a, t1 = min(t0 + TT, C);
            if (t0 >= t1) {
                ux[x] = SpanUnion{0, 0, 0, 0};
                continue;
            }
            const KeySpans f = key_spans(L, P0 + t0, 0, prefix, sc.window, sc.causal);
            const KeySpans l = key_spans(L, P0 + t1 - 1, 0, prefix, sc.window, sc.causal);
            ux[x] = SpanUnion{f.a0, l.a1, f.b0, l.b1};
        }
    } else {
        if (tid < 8) {
            red[tid >> 2][tid & 3] = (tid & 1) ? 0 : 0x7fffffff;
            seen_own[tid] = 0u;
        }
        __syncthreads();
        if (softmax_warp && half == 0) {
            const bool in_a = row.a0 < row.a1, in_b = row.b0 < row.b1;
            const int32_t a0 = __reduce_min_sync(0xffffffffu, in_a ? row.a0 : 0x7fffffff);
            const int32_t a1 = __reduce_max_sync(0xffffffffu, in_a ? row.a1 : 0);
            const int32_t b0 = __reduce_min_sync(0xffffffffu, in_b ? row.b0 : 0x7fffffff);
            const int32_t b1 = __reduce_max_sync(0xffffffffu, in_b ? row.b1 : 0);
            if (lane == 0) {
                atomicMin(&red[xq][0], a0);
                atomicMax(&red[xq][1], a1);
                atomicMin(&red[xq][2], b0);
                atomicMax(&red[xq][3], b1);
            }
            if (g == 0) {
                // the CTA's own positions P0 + t0a + i that this row sees; a key before them that
                // any row's span reaches past is seen by the row with the lowest start
                const int32_t own = P0 + t0a;
                int32_t lo = max(row.a0 - own, 0), hi = in_a ? min(row.a1 - own, 256) : 0;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    for (int32_t w = lo >> 5; w * 32 < hi; ++w) atomicOr(&seen_own[w], span_bits(w * 32, lo, hi));
                    lo = max(row.b0 - own, 0), hi = in_b ? row.b1 - own : 0;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < NQ; ++x) ux[x] = SpanUnion{red[x][0], red[x][1], red[x][2], red[x][3]};
    }
    const SpanUnion uni = join(ux[0], ux[NQ - 1]);
    TileList tiles = tile_list(uni);
    int32_t n_kv = tiles.n, n_parts = 1;
    if constexpr (SPLIT) {  // this CTA takes one of up to split.parts equal runs of the list
        const int32_t most = max(min(split.parts, n_kv / kMinPartTiles), 1), share = max((n_kv + most - 1) / most, 1);
        n_parts = max((n_kv + share - 1) / share, 1);
        if (static_cast<int32_t>(blockIdx.x) >= n_parts) {  // uniform over the CTA
            asm volatile("cp.async.wait_all;" ::: "memory");
            return;
        }
        tiles.base = blockIdx.x * share;
        n_kv = min(share, n_kv - tiles.base);
        if (tid == 0 && blockIdx.x == 0 && n_parts > 1)
            split.rows[cta] = make_int4(q0 + t0a, min(TT, C - t0a) * G, max(min(TT, C - t0b), 0) * G, n_parts);
    }
    // list positions whose key tile query tile x uses: two ranges
    int32_t ra0[NQ], ra_n[NQ], rb0[NQ], rb_n[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        ra0[x] = ux[x].a0 / kKeys - tiles.first_a - tiles.base;
        ra_n[x] = ux[x].a0 < ux[x].a1 ? (ux[x].a1 - 1) / kKeys - tiles.first_a - tiles.base + 1 - ra0[x] : 0;
        rb0[x] = tiles.position(ux[x].b0 / kKeys);
        rb_n[x] = ux[x].b0 < ux[x].b1 ? tiles.position((ux[x].b1 - 1) / kKeys) + 1 - rb0[x] : 0;
    }
    auto used = [&](int32_t x, int32_t i) -> bool {
        return static_cast<uint32_t>(i - ra0[x]) < static_cast<uint32_t>(ra_n[x]) ||
               static_cast<uint32_t>(i - rb0[x]) < static_cast<uint32_t>(rb_n[x]);
    };
    const int32_t npages = (L + kPageTokens - 1) / kPageTokens;

    // Pool row of list page 8 i + s (page s of the i-th key tile); lane l of a producer warp holds
    // page 32 w + l of window w, fetched one window ahead.
    auto page_row = [&](int32_t lp) -> int32_t {
        int32_t phys = 0, pg = 0;
        if ((lp >> 3) < n_kv) {
            pg = tiles.tile(lp >> 3) * (kKeys / kPageTokens) + (lp & 7);
            if (pg < npages) {  // keys past the sequence end read the null block; masked
                phys = __ldg(block_table + static_cast<int64_t>(seq) * max_blocks + (pg >> sub_log2));
                if (phys < 0 || phys >= num_blocks) {
                    raise_error(err, PA_DEVERR_BLOCK_RANGE);
                    phys = 0;
                }
            }
        }
        return (((phys * num_kv_heads + h) << sub_log2) + (pg & ((1 << sub_log2) - 1))) * kPageTokens;
    };
    int32_t row_cur = 0, row_nxt = 0;
    if (warp == kKWarp || warp == kVWarp) {
        row_cur = page_row(lane);
        row_nxt = page_row(32 + lane);
    }
    if (tid == 0) {
        *reinterpret_cast<volatile int32_t*>(smem + L_::misc + 4) = 0;
        for (int i = 0; i < L_::num_bars; ++i) {  // each once: an object in use must not be initialised again
            uint64_t* bar = bars + i;
            const bool p = bar >= p_full && bar < p_full + kChains;
            mbar_init(bar, p ? kSoftWarps / kChains : bar >= mx_full ? 2 : bar == q_full ? kSoftThreads : 1);
        }
        fence_mbarrier_init();
    }
    if (!kSplit && softmax_warp && half == 0) shared.row_top[xq][r] = ordered(-INFINITY);  // (the ranking is over)
    if (warp == kMmaWarp) {
        umma::tmem_alloc(tmem_holder, 2 * kO);
        umma::tmem_relinquish();
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    // tensor memory columns: S of tile x at 128 x (the P of each half of its keys, bf16 pairs,
    // overwrites the first 32 of the half's 64 columns once read), O of tile x at kO + 128 x
    const uint32_t tmem = *tmem_holder;
    if (softmax_warp) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_shared();
        mbar_arrive(q_full);
    }

    int32_t last_j = -1;  // producers: last key tile issued
    if (warp == kKWarp || warp == kVWarp) {
        // ======================================= producers ======================================
        const bool is_v = warp == kVWarp;
        const int32_t nst = is_v ? kVStages : kKStages;
        const void* tm = is_v ? static_cast<const void*>(&tm_v) : static_cast<const void*>(&tm_k);
        uint64_t* full = is_v ? v_full : k_full;
        uint64_t* empty = is_v ? v_empty : k_empty;
        uint8_t* ring = smem + (is_v ? L_::v : L_::k);
        if (lane == 0) prefetch_tensormap(tm);
        for (int32_t j = 0; j < n_kv; ++j) {
            const int32_t st = j % nst;
            const uint32_t use = static_cast<uint32_t>(j / nst);
            if (j > 0 && (j & 3) == 0) {
                row_cur = row_nxt;
                row_nxt = page_row(32 * ((j >> 2) + 1) + lane);
            }
            bool ok = true;
            if (use > 0 && lane == 0) ok = wait_or_abort<kSleepProducer>(&empty[st], (use - 1) & 1u, abort_flag, err);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            uint8_t* dst = ring + st * kTile;
            if (lane == 0) mbar_arrive_expect_tx(&full[st], kTile);
            last_j = j;
            const int32_t rk = __shfl_sync(0xffffffffu, row_cur, (j & 3) * 8 + (lane & 7));
            __syncwarp();
            if (lane < 8 * kHalves)  // lane = (column half, page)
                tma_load_2d(dst + (lane >> 3) * kHalf + (lane & 7) * 2048u, tm, (lane >> 3) * 64, rk, &full[st]);
        }
    } else if (warp == kMmaWarp && umma::elect_one()) {
        // ======================================= MMA issuer =====================================
        // One thread issues every MMA (a commit tracks those of its own thread) and does all the waiting.
        constexpr int kChainKeys = kSplit ? 64 : 128;
        const uint32_t idesc_qk = umma::idesc_bf16_f32(128, kChainKeys, 0, 0);  // Q, K both K-major
        const uint32_t idesc_pv = umma::idesc_bf16_f32(128, D, 0, 1);           // P (TMEM), V MN-major
        const uint64_t dq0 = umma::smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk0 = umma::smem_desc_sw128(smem_u32(smem + L_::k), 16, 1024);
        const uint64_t dv0 = umma::smem_desc_sw128(smem_u32(smem + L_::v), kHalf, 1024);
        auto qk = [&](int c, int32_t j) {
            const int x = c % NQ, hf = c / NQ;
            const uint64_t dq = dq0 + static_cast<uint64_t>(x) * (kTile >> 4);
            const uint64_t dk = dk0 + static_cast<uint64_t>(j % kKStages) * (kTile >> 4) + hf * (64 * 128 >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                umma::mma_bf16(tmem + x * 128 + hf * 64, dq + off, dk + off, idesc_qk, ks > 0);
            }
            umma::commit(&s_full[c]);
        };
        auto pv = [&](int c, int32_t j, bool acc) {
            const int x = c % NQ, hf = c / NQ;
            const uint64_t dv = dv0 + static_cast<uint64_t>(j % kVStages) * (kTile >> 4);
#pragma unroll
            for (int k = 0; k < kChainKeys / 16; ++k) {  // 16 keys per instruction: 8 P columns
                const int kk = hf * 4 + k;
                umma::mma_bf16_tmem_a(tmem + kO + x * 128 + (kOwnO ? hf * D : 0), tmem + x * 128 + (kk >> 2) * 64 + (kk & 3) * 8,
                                      dv + static_cast<uint64_t>(kk * (2048 >> 4)), idesc_pv, (acc || k > 0));
            }
        };
        auto wait_k = [&](int32_t j) {
            const bool ok = wait_or_abort<0>(&k_full[j % kKStages], static_cast<uint32_t>(j / kKStages) & 1u, abort_flag, err);
            umma::fence_after_sync();
            return ok;
        };
        int32_t last[NQ], done[NQ] = {};  // last list position, and positions finished, per query tile
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            last[x] = n_kv - 1;
            while (last[x] >= 0 && !used(x, last[x])) --last[x];
        }
        bool ok = wait_or_abort<0>(q_full, 0, abort_flag, err);
        if (ok && n_kv > 0) ok = wait_k(0);
        if (ok && n_kv > 0) {
#pragma unroll
            for (int c = 0; c < kChains; ++c)
                if (used(c % NQ, 0)) qk(c, 0);
            umma::commit(&k_empty[0]);
        }
        for (int32_t j = 0; j < n_kv && ok; ++j) {
            const bool more = j + 1 < n_kv;
            ok = wait_or_abort<0>(&v_full[j % kVStages], static_cast<uint32_t>(j / kVStages) & 1u, abort_flag, err);
#pragma unroll
            for (int c = 0; c < kChains; ++c) {
                const int x = c % NQ;
                if (ok && used(x, j)) {  // P written, S read: O_x += P V(j)
                    ok = wait_or_abort<0>(&p_full[c], done[x] & 1, abort_flag, err);
                    umma::fence_after_sync();
                    if (ok) {
                        pv(c, j, done[x] > 0 || (!kOwnO && c >= NQ));
                        if (c >= kChains - NQ) {  // the query tile's last chain
                            ++done[x];
                            if (j == last[x]) umma::commit(&o_done[x]);
                        }
                    }
                }
                if (c == kChains - 1 && ok) umma::commit(&v_empty[j % kVStages]);
                if (c == 0 && ok && more) ok = wait_k(j + 1);
                if (ok && more && used(x, j + 1)) qk(c, j + 1);  // (used() knows the whole list, not where a run ends)
            }
            if (ok && more) umma::commit(&k_empty[(j + 1) % kKStages]);
        }
        umma::commit(idle);  // arrives once every MMA issued above has finished
        mbar_wait_timeout(idle, 0);
    } else if (softmax_warp) {
        // ==================================== scores and softmax ================================
        const int32_t chain = kSplit ? half * NQ + xq : xq;
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tmem_s = tmem + xq * 128 + half * 64 + lane_off;
        const uint32_t tmem_o = tmem + kO + xq * 128 + half * (kOwnO ? D : D / 2) + lane_off;  // columns it rescales
        const float slope = (MODE != kPlain && MODE != kCap) && sc.slopes && row_valid
                                ? __ldg(sc.slopes + h * G + g) * kLog2e
                                : 0.f;
        const uint64_t c1 = hold2(sc.c1);
        const uint64_t ref2 = hold2(-sc.ref);
        uint64_t tq[4];  // the polynomial's coefficients, kept in registers
#pragma unroll
        for (int k = 0; k < 4; ++k) tq[k] = hold2(sc.q[k]);
        const uint64_t step = pack2(8.f * slope, 8.f * slope);
        // fixed reference; under a distance bias, taken from the row's largest bias, so that the weight of the
        // key that has it lies in the range of the capped scores
        float fixed_shift = -sc.ref;
        if constexpr (MODE == kCapDistance) {
            const bool in_a = row.a0 < row.a1, in_b = row.b0 < row.b1;
            const int32_t lo = in_a ? row.a0 : row.b0, hi = (in_b ? row.b1 : row.a1) - 1;  // ends of what the row sees
            int32_t near = 0;  // b holds the row's own key, or is empty
            if (!in_b) near = max(max(lo - pos, pos - hi), 0);
            fixed_shift += slope * static_cast<float>(slope >= 0.f ? near : max(abs(pos - lo), abs(hi - pos)));
        }
        float m_ref = -INFINITY, l_sum = 0.f;
        bool ok = true;
        int32_t cnt = 0;  // key tiles this query tile has used
        for (int32_t i = 0; i < n_kv; ++i) {
            if (!used(xq, i)) continue;
            ok = wait_or_abort<kSleepSoftmax>(&s_full[chain], cnt & 1, abort_flag, err);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            umma::fence_after_sync();
            const int32_t ktile = tiles.tile(i) * kKeys, kbase = ktile + half * (kKeys / 2);
            const bool first = cnt == 0;
            ++cnt;
            // rows that see the whole tile need no mask (nor do rows without a query, whose Q is
            // zero and whose results go nowhere)
            const bool whole = !row_valid || (kbase >= row.a0 && kbase + kKeys / 2 <= row.a1) ||
                               (kbase >= row.b0 && kbase + kKeys / 2 <= row.b1);
            const bool mask = !__all_sync(0xffffffffu, whole);
            const bool behind = __any_sync(0xffffffffu, row_valid && kbase + kKeys / 2 - 1 > pos);
            const float d0 = static_cast<float>(kbase - pos);
            // Bits of the 16 keys of group c that the row sees.
            auto visible = [&](int c) -> uint32_t {
                return span_bits(kbase + c * 16, row.a0, row.a1) | span_bits(kbase + c * 16, row.b0, row.b1);
            };
            // Weight arguments (log2 domain), x = score + shift. A group of 16 keys is straight-line
            // code: begin_group sets up what its pairs share, pair_args does columns 2 e, 2 e + 1; what
            // differs by warp is branched on once per group (amend).
            float big[4];
            uint64_t away[4];
            auto begin_group = [&](int c, float shift) {
                if constexpr (kFixed || MODE == kLargeCap) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) big[k] = 0.f;
                }
                if constexpr (MODE == kDistance || MODE == kCapDistance) {  // -slope |p - j| = slope (j - p) for j <= p
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        away[k] = pack2(fmaf(slope, d0 + (c * 16 + 2 * k), shift), fmaf(slope, d0 + (c * 16 + 2 * k + 1), shift));
                }
            };
            auto pair_args = [&](uint64_t s, int c, int e, float shift, float& x0, float& x1) {
                if constexpr (MODE == kPlain) {
                    unpack2(fma2(s, c1, pack2(shift, shift)), x0, x1);
                } else if constexpr (kFixed) {
                    const uint64_t w = mul2(s, s);
                    uint64_t p = fma2(w, tq[3], tq[2]);
                    p = fma2(w, p, tq[1]);
                    p = fma2(w, p, tq[0]);
                    if constexpr (MODE == kCap) {
                        unpack2(fma2(s, p, ref2), x0, x1);
                    } else {
                        unpack2(fma2(s, p, away[e & 3]), x0, x1);
                        if (e < 4) away[e & 3] = add2(away[e & 3], step);
                    }
                    float w0, w1;
                    unpack2(w, w0, w1);
                    big[e & 3] = max3(big[e & 3], w0, w1);
                } else if constexpr (MODE == kDistance) {
                    unpack2(fma2(s, c1, away[e & 3]), x0, x1);
                    if (e < 4) away[e & 3] = add2(away[e & 3], step);
                } else {
                    float s0, s1;
                    unpack2(s, s0, s1);
                    const float y0 = s0 * sc.two_k, y1 = s1 * sc.two_k;
                    if constexpr (MODE == kGeneral) {
                        s0 = capped_far(y0, sc.cap_l2);
                        s1 = capped_far(y1, sc.cap_l2);
                    } else {
                        s0 = capped_near(s0, y0 * y0, sc.c1);
                        s1 = capped_near(s1, y1 * y1, sc.c1);
                        big[e & 3] = max3(big[e & 3], y0 * y0, y1 * y1);
                    }
                    x0 = fmaf(-slope, fabsf(d0 + (c * 16 + 2 * e)), s0) + shift;
                    x1 = fmaf(-slope, fabsf(d0 + (c * 16 + 2 * e + 1)), s1) + shift;
                }
            };
            // Scores beyond the polynomial's range, keys behind the row, masked keys.
            auto amend = [&](const uint32_t(&raw)[16], int c, float shift, float(&x)[16]) {
                bool redo = false;
                if constexpr (kFixed || MODE == kLargeCap)
                    redo = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])) > (kFixed ? sc.s2_max : kTanhY2);
                if constexpr (MODE == kDistance || MODE == kCapDistance) redo = redo || behind;
                if (redo || mask) {
                    if (redo) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float s = __uint_as_float(raw[k]);
                            if constexpr (MODE == kCap) x[k] = capped_far(s * sc.two_k, sc.cap_l2) + shift;
                            if constexpr (MODE == kCapDistance)
                                x[k] = capped_far(s * sc.two_k, sc.cap_l2) + fmaf(-slope, fabsf(d0 + (c * 16 + k)), shift);
                            if constexpr (MODE == kLargeCap) {
                                const float y = s * sc.two_k;
                                if (y * y > kTanhY2) x[k] = fmaf(-slope, fabsf(d0 + (c * 16 + k)), capped_far(y, sc.cap_l2)) + shift;
                            }
                            if constexpr (MODE == kDistance)
                                x[k] = fmaf(s, sc.c1, fmaf(-slope, fabsf(d0 + (c * 16 + k)), shift));
                        }
                    }
                    if (mask) {
                        const uint32_t vis = visible(c);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (!(vis >> k & 1u)) x[k] = -INFINITY;
                    }
                }
            };
            float alpha = 1.f, shift = fixed_shift;
            bool grow = false;
            if constexpr (!kFixed) {
                // pass 1: the tile's maximum over visible keys
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                uint32_t raw[2][16];
                ld_x16(tmem_s, raw[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    wait_x16(raw[c & 1]);
                    if (c < 3) ld_x16(tmem_s + (c + 1) * 16, raw[(c + 1) & 1]);
                    float x[16];
                    begin_group(c, 0.f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) pair_args(raw_pair(raw[c & 1], e), c, e, 0.f, x[2 * e], x[2 * e + 1]);
                    amend(raw[c & 1], c, 0.f, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e & 3] = max3(mx[e & 3], x[2 * e], x[2 * e + 1]);
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if constexpr (!kOwnO) {
                    // The row's other half of the keys is another thread's: both raise the row's maximum so far and
                    // read it. It is exact: rounded to fewer bits, a reference could lie so far above large
                    // scores that every weight of the row is 0. (The maximum so far exceeds m_ref + threshold just
                    // where the tile's does, and nobody raises it for the next tile before both have read
                    // it: the next S waits for both halves' P.)
                    atomicMax(&shared.row_top[xq][r], ordered(top));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&mx_full[xq * 4 + quad]);
                    ok = wait_or_abort<kSleepSoftmax>(&mx_full[xq * 4 + quad], (cnt - 1) & 1, abort_flag, err);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    top = unordered(*const_cast<volatile int32_t*>(&shared.row_top[xq][r]));
                }
                grow = top > m_ref + kRescaleThreshold;  // first visible keys: m_ref = -inf
                const float m_new = grow ? top : m_ref;
                alpha = grow ? exp2_approx(m_ref - m_new) : 1.f;
                m_ref = m_new;
                shift = m_new == -INFINITY ? 0.f : -m_new;  // nothing visible yet: weights are 0
            }
            if constexpr (!kFixed) {
                if (!first && __any_sync(0xffffffffu, grow)) {
                    // O holds the tiles before under the old reference; their last PV finished before
                    // this S was committed, so O can be rescaled now
#pragma unroll
                    for (int c = 0; c < (kOwnO ? D : D / 2) / 32; ++c) {
                        uint32_t o[32];
                        ld_wait_x32(tmem_o + c * 32, o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        umma::st_32x32b_x32(tmem_o + c * 32, o);
                    }
                    umma::wait_st();
                }
            }
            // keys that no row of the CTA sees: zero their V rows, in the chain's part of the key tile, by
            // the first query tile that uses it (thread r: 64 columns of one key row)
            const int32_t own = P0 + t0a;
            const bool gaps = !uni.covers(ktile, ktile + kKeys) || (sc.key_start != nullptr && ktile + kKeys > own);
            const int32_t zrow = kSplit ? half * 64 + (r & 63) : r, zhalf = kSplit ? r >> 6 : half;
            if (gaps && (xq == 0 || !used(0, i))) {
                const int32_t key = ktile + zrow;
                bool seen = (key >= uni.a0 && key < uni.a1) || (key >= uni.b0 && key < uni.b1);
                if (seen && sc.key_start != nullptr && static_cast<uint32_t>(key - own) < 256u)  // (behind: the prefix)
                    seen = (seen_own[(key - own) >> 5] >> ((key - own) & 31)) & 1u;
                const int32_t st = i % kVStages;
                const bool okv = wait_or_abort<kSleepSoftmax>(&v_full[st], static_cast<uint32_t>(i / kVStages) & 1u, abort_flag, err);
                if (okv && !seen && zhalf < kHalves) {
                    uint8_t* sv = smem + L_::v + st * kTile + zhalf * kHalf;
#pragma unroll
                    for (int c = 0; c < 8; ++c) *reinterpret_cast<int4*>(sv + zrow * 128u + c * 16u) = make_int4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();
            }
            // pass 2: P = 2^arg in bf16 pairs, 16 keys at a time (each group of S is read before
            // the P columns that overwrite part of it)
            uint64_t psum[4] = {0ull, 0ull, 0ull, 0ull};
            // One group ahead: the arithmetic of group c + 1 (FMA pipes) shares a block of code with
            // the exponentials of group c (MUFU), so that the two overlap within each warp.
            uint32_t raw[2][16];
            float x[2][16];
            ld_x16(tmem_s, raw[0]);
            wait_x16(raw[0]);
            ld_x16(tmem_s + 16, raw[1]);
            begin_group(0, shift);
#pragma unroll
            for (int e = 0; e < 8; ++e) pair_args(raw_pair(raw[0], e), 0, e, shift, x[0][2 * e], x[0][2 * e + 1]);
            amend(raw[0], 0, shift, x[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c < 3) {
                    wait_x16(raw[(c + 1) & 1]);
                    if (c < 2) ld_x16(tmem_s + (c + 2) * 16, raw[c & 1]);
                    begin_group(c + 1, shift);
                }
                uint32_t pk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (c < 3)
                        pair_args(raw_pair(raw[(c + 1) & 1], e), c + 1, e, shift, x[(c + 1) & 1][2 * e],
                                  x[(c + 1) & 1][2 * e + 1]);
                    const float p0 = exp2_approx(x[c & 1][2 * e]), p1 = exp2_approx(x[c & 1][2 * e + 1]);
                    psum[e & 3] = add2(psum[e & 3], pack2(p0, p1));
                    pk[e] = pack_bf16x2(p0, p1);
                }
                st_x8(tmem_s + c * 8, pk);
                if (c < 3) amend(raw[(c + 1) & 1], c + 1, shift, x[(c + 1) & 1]);
            }
            umma::wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[chain]);
            float s0, s1;
            unpack2(add2(add2(psum[0], psum[1]), add2(psum[2], psum[3])), s0, s1);
            l_sum = l_sum * alpha + (s0 + s1);
        }
        // The halves' sums meet in the query tile's shared memory, which no MMA reads any more and no thread's
        // copy still writes: o_done says both, as the MMAs waited for the copies. A query tile that no key tile of
        // the CTA uses (rows that see nothing, a run of keys that only the other tile sees) has no MMAs and
        // waits for all the copies itself. Every softmax thread of the tile comes here, aborted or not.
        if (ok) ok = wait_or_abort<kSleepSoftmax>(cnt > 0 ? &o_done[xq] : q_full, 0, abort_flag, err);
        float* sums = reinterpret_cast<float*>(smem + xq * kTile);
        __syncwarp();
        sums[half * kRows + r] = l_sum;
        if (kOwnO) sums[(2 + half) * kRows + r] = m_ref;
        named_barrier(1 + xq, 256);
        float w0 = 1.f, w1 = 1.f;  // weights of the halves' outputs: 1 under a common reference
        float top = kFixed ? 0.f : m_ref;
        if (kOwnO) {
            const float m0 = sums[2 * kRows + r], m1 = sums[3 * kRows + r];
            top = fmaxf(m0, m1);
            w0 = m0 == -INFINITY ? 0.f : exp2_approx(m0 - top);
            w1 = m1 == -INFINITY ? 0.f : exp2_approx(m1 - top);
        }
        l_sum = w0 * sums[r] + w1 * sums[kRows + r];
        // A row that sees one key is its V: its sum is the one weight, which P V took rounded to bf16.
        if (row.a1 - row.a0 + (row.b1 - row.b0) == 1) l_sum = __bfloat162float(__float2bfloat16_rn(l_sum));
        named_barrier(1 + xq, 256);
        ok = __all_sync(0xffffffffu, ok);
        // columns half (D / 2) + 32 c .. of the row's output, before the division; 0 where no key was used
        auto load_output = [&](int c, uint32_t(&o)[32]) {
            const uint32_t cols = tmem + kO + xq * 128 + half * (D / 2) + c * 32 + lane_off;
            if (cnt == 0) {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0u;
                return;
            }
            ld_wait_x32(cols, o);
            if constexpr (kOwnO) {
                uint32_t o1[32];
                ld_wait_x32(cols + D, o1);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = __float_as_uint(fmaf(w0, __uint_as_float(o[k]), w1 * __uint_as_float(o1[k])));
            }
        };
        if (SPLIT && n_parts > 1) {
            if (ok) {
                umma::fence_after_sync();
                const int64_t run = static_cast<int64_t>(cta) * split.parts + blockIdx.x;
                if (half == 0) split.ml[run * (2 * kRows) + xq * kRows + r] = make_float2(top, l_sum);
                float4* po = split.o + (run * (D / 4) + half * (D / 8)) * (2 * kRows) + xq * kRows + r;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t o[32];
                    load_output(c, o);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        po[(c * 8 + v) * (2 * kRows)] =
                            make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                        __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                }
            }
        } else if (ok) {
            umma::fence_after_sync();
            const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
            // this warp's rows x D / 2 columns through its own part of the tile's Q, so that the stores go
            // out whole lines at a time (a row's 16-byte pieces in different banks, lane by lane)
            constexpr int kPieces = D / 16;
            uint8_t* stage = smem + xq * kTile + (half * 4 + quad) * (32 * D);
            const int32_t turn = D == 128 ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t o[32];
                load_output(c, o);
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = l_sum == 0.f ? 0.f : __uint_as_float(o[v4 * 8 + k]) * inv;
                    *reinterpret_cast<uint4*>(stage + lane * D + ((c * 4 + v4) ^ turn) * 16) =
                        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                   pack_bf16x2(f[6], f[7]));
                }
            }
            __syncwarp();
            const int64_t row_off =
                row_valid ? (static_cast<int64_t>(q0 + t_row) * Hq + h * G + g) * D + half * (D / 2) : -1;
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const int32_t i = k * 32 + lane, rr = i / kPieces, c = i % kPieces;
                const int64_t off = __shfl_sync(0xffffffffu, row_off, rr);
                const int32_t t = D == 128 ? rr & 7 : (rr >> 1) & 3;
                const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * D + (c ^ t) * 16);
                if (off >= 0) *reinterpret_cast<uint4*>(out + off + c * 8) = v;
            }
        }
    }

    // ---- wind down: copies landed and MMAs retired before shared and tensor memory go ------
    if ((warp == kKWarp || warp == kVWarp) && lane == 0) {
        const int32_t nst = warp == kVWarp ? kVStages : kKStages;
        uint64_t* full = warp == kVWarp ? v_full : k_full;
        for (int32_t j = max(0, last_j - nst + 1); j <= last_j; ++j)
            mbar_wait_timeout(&full[j % nst], static_cast<uint32_t>(j / nst) & 1u);
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, 2 * kO);
    }
}

// Merges the runs of split key lists: M = max m, out = sum 2^(m - M) o / sum 2^(m - M) l. Grid: four
// columns of head_dim x CTA of the unsplit grid; a thread has one row of the CTA's two tiles.
template <int D>
__global__ void __launch_bounds__(2 * kRows) prefill_scored_merge_kernel(__nv_bfloat16* __restrict__ out,
                                                                         const __grid_constant__ Split split,
                                                                         int32_t num_kv_heads, int32_t G) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t c4 = blockIdx.x, cta = blockIdx.y, R = threadIdx.x;
    const int4 rows = split.rows[cta];
    const int32_t rr = R & (kRows - 1), n = R < kRows ? rows.y : rows.z;
    if (rows.w == 0 || rr >= n) return;
    const float2* ml = split.ml + static_cast<int64_t>(cta) * split.parts * (2 * kRows) + R;
    const float4* po = split.o + (static_cast<int64_t>(cta) * split.parts * (D / 4) + c4) * (2 * kRows) + R;
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int32_t p = 0; p < rows.w; ++p) M = fmaxf(M, ml[p * (2 * kRows)].x);
    const float ref = M == -INFINITY ? 0.f : M;  // no visible key in any run: weights are 0
#pragma unroll 8
    for (int32_t p = 0; p < rows.w; ++p) {
        const float2 x = ml[p * (2 * kRows)];
        const float4 o = po[static_cast<int64_t>(p) * (D / 4) * (2 * kRows)];
        const float w = exp2_approx(x.x - ref);
        den = fmaf(w, x.y, den);
        acc.x = fmaf(w, o.x, acc.x), acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z), acc.w = fmaf(w, o.w, acc.w);
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const int32_t h = cta % num_kv_heads, TT = kRows / G, tt = rr / G, t = (R < kRows ? 0 : TT) + tt;
    __nv_bfloat16* to = out + (static_cast<int64_t>(rows.x + t) * G * num_kv_heads + h * G + (rr - tt * G)) * D + c4 * 4;
    *reinterpret_cast<uint2*>(to) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// Minimax (Remez) coefficients of tanh x = x (t0 + t1 x^2 + t2 x^4 + t3 x^6) on |x| <= 0.6; absolute
// error 5.9e-7.
constexpr double kTanh[4] = {0.999991018, -0.332989742, 0.129745541, -0.0396112775};
constexpr float kTanhRange = 0.6f;

// Grids of few waves are ordered pair by pair, others sequence by sequence (kFewWaves).
// tiles: query tiles of a CTA; of one tile, two CTAs share an SM.
bool few_waves(int64_t entries, int32_t num_kv_heads, int tiles, int num_sms) {
    return entries <= kRankMax && entries * num_kv_heads <= static_cast<int64_t>(kFewWaves) * (3 - tiles) * num_sms;
}

template <int D, int MODE, int NQ, bool SPLIT>
cudaError_t launch_impl(const PrefillArgs& a, const TcScore& sc, const PrefillScoredPlan& plan,
                        void* workspace, int num_sms, cudaStream_t stream) {
    alignas(64) CUtensorMap tm_k, tm_v;
    const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.num_kv_heads * a.block_size;
    cudaError_t e = encode_bf16_2d_sw128(&tm_k, a.k_cache, D, rows, 64, kPageTokens);
    if (e != cudaSuccess) return e;
    e = encode_bf16_2d_sw128(&tm_v, a.v_cache, D, rows, 64, kPageTokens);
    if (e != cudaSuccess) return e;
    e = allow_smem<prefill_scored_kernel<D, MODE, NQ, SPLIT>>(static_cast<int>(Smem<D, NQ>::total));
    if (e != cudaSuccess) return e;
    const int32_t G = a.num_q_heads / a.num_kv_heads, TT = kRows / G;
    const int32_t sub_log2 = block_size_log2(a.block_size) - 4;
    const int32_t cap_tokens = min(table_tokens(a.max_blocks_per_seq, sub_log2), a.max_seq_len);
    const int32_t pairs = (a.max_chunk_len + NQ * TT - 1) / (NQ * TT);
    const int64_t entries = static_cast<int64_t>(pairs) * a.num_seqs;
    const bool by_pair = few_waves(entries, a.num_kv_heads, NQ, num_sms);
    const int32_t sub = by_pair ? pairs : 1;
    const dim3 grid(SPLIT ? plan.parts : by_pair ? 1 : pairs, a.num_kv_heads, a.num_seqs * sub);
    Split split{};
    if (SPLIT) {
        char* ws = static_cast<char*>(workspace);
        split.parts = plan.parts;
        split.rows = reinterpret_cast<int4*>(ws + kScoredCounterBytes);
        split.o = reinterpret_cast<float4*>(ws + kScoredCounterBytes + kSplitRowBytes);
        split.ml = reinterpret_cast<float2*>(split.o + entries * a.num_kv_heads * plan.parts * (D / 4) * (2 * kRows));
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    prefill_scored_kernel<D, MODE, NQ, SPLIT><<<grid, Warps<NQ>::threads, Smem<D, NQ>::total, stream>>>(
        tm_k, tm_v, out, static_cast<const __nv_bfloat16*>(a.q), a.block_table, a.max_blocks_per_seq, a.seq_lens,
        a.query_start_loc, a.num_kv_heads, G, a.num_blocks, sub_log2, cap_tokens, a.max_chunk_len, sub, 65536u / sub + 1,
        split, sc, a.err);
    e = cudaGetLastError();
    if (!SPLIT || e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];  // the merge's CTAs may be set up while the last runs end
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / 4, static_cast<unsigned>(entries * a.num_kv_heads));
    cfg.blockDim = dim3(2 * kRows);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_scored_merge_kernel<D>, out, split, a.num_kv_heads, G);
}

template <int D>
cudaError_t pick(const PrefillArgs& a, const TcScore& sc, Mode mode, const PrefillScoredPlan& plan, void* workspace,
                 int num_sms, cudaStream_t stream) {
    auto run = [&](auto m) {
        if (plan.parts > 1) return launch_impl<D, m, 2, true>(a, sc, plan, workspace, num_sms, stream);
        return plan.tiles == 1 ? launch_impl<D, m, 1, false>(a, sc, plan, workspace, num_sms, stream)
                               : launch_impl<D, m, 2, false>(a, sc, plan, workspace, num_sms, stream);
    };
    switch (mode) {
        case kPlain: return run(std::integral_constant<int, kPlain>{});
        case kCap: return run(std::integral_constant<int, kCap>{});
        case kDistance: return run(std::integral_constant<int, kDistance>{});
        case kCapDistance: return run(std::integral_constant<int, kCapDistance>{});
        case kGeneral: return run(std::integral_constant<int, kGeneral>{});
        default: return run(std::integral_constant<int, kLargeCap>{});
    }
}

}  // namespace

PrefillScoredPlan plan_prefill_scored(int32_t S, int32_t max_chunk, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_len,
                                      int num_sms) {
    PrefillScoredPlan plan{1, 2, 0};
    if (Hq / Hkv > kRows) return plan;
    const int32_t TT = kRows / (Hq / Hkv);
    if (max_chunk <= TT || max_len <= short_keys(D)) plan.tiles = 1;
    const int64_t most = static_cast<int64_t>(max_len / kKeys + 1) / kMinPartTiles;  // runs of the longest list
    if (most < 2) return plan;
    // room for a wave of CTAs, whatever the chunks: a workspace serves every call up to its max_len
    plan.workspace_bytes = kScoredCounterBytes + kSplitRowBytes + static_cast<size_t>(num_sms) * (2 * kRows) * (D * 4 + 8);
    if (S < 1 || max_chunk < 1) return plan;
    const int64_t entries = (static_cast<int64_t>(max_chunk) + 2 * TT - 1) / (2 * TT) * S;
    if (few_waves(entries, Hkv, 2, num_sms))  // one wave of CTAs, each with kMinPartTiles key tiles at least
        plan.parts = static_cast<int32_t>(max(min(num_sms / (entries * Hkv), most), static_cast<int64_t>(1)));
    return plan;
}

bool prefill_scored_tc_ok(const PrefillArgs& a, const DeviceInfo& dev) {
    return a.dtype == PA_BF16 && a.num_q_heads / a.num_kv_heads <= kRows && a.num_seqs <= 65535 &&
           a.num_kv_heads <= 65535 && static_cast<int>(Smem<128, 2>::total) <= dev.max_smem_optin;
}

cudaError_t launch_prefill_scored_tc(const PrefillArgs& a, const ScoreArgs& s, const PrefillScoredPlan& plan,
                                     void* workspace, int num_sms, cudaStream_t stream) {
    TcScore sc{};
    sc.c1 = a.scale * kLog2e;
    const bool capped = s.cap > 0.f;
    if (capped) {
        const double k = static_cast<double>(a.scale) / s.cap;
        double c = static_cast<double>(s.cap) * 1.4426950408889634 * k;
        for (int i = 0; i < 4; ++i, c *= k * k) sc.q[i] = static_cast<float>(c * kTanh[i]);
        sc.s2_max = static_cast<float>(kTanhRange * kTanhRange / (k * k));
        sc.two_k = static_cast<float>(fmin(fmax(2 * 1.4426950408889634 * k, -3e38), 3e38));
        sc.cap_l2 = fminf(s.cap * kLog2e, kLargestCapL2);
        sc.ref = s.slopes ? sc.cap_l2 - kTopWeight : 0.5f * sc.cap_l2;
    }
    sc.window = s.window;
    sc.slopes = s.slopes;
    sc.key_start = s.key_start;
    sc.prefix_len = s.prefix_len;
    sc.causal = s.causal;
    const Mode mode = !capped ? (s.slopes ? kDistance : kPlain)
                                 : s.cap > kMaxIdentityCap ? kLargeCap
                                 : s.cap > kMaxFixedCap || !isfinite(sc.q[3]) ? kGeneral  // (tiny caps: no polynomial)
                                 : s.slopes ? kCapDistance : kCap;
    return a.head_dim == 128 ? pick<128>(a, sc, mode, plan, workspace, num_sms, stream) : pick<64>(a, sc, mode, plan, workspace, num_sms, stream);
}

}  // namespace pa
