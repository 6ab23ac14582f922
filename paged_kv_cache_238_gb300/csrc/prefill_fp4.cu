// Chunked causal prefill over a 4-bit pool on the 5th-generation tensor cores (bf16 queries, head_dim 64 or 128, up
// to 128 q heads per kv head).
//
// One CTA computes two 128-row query tiles (a, b) of one (sequence, kv head): row r of a tile is token r / G, q head
// r % G of the G heads that share the kv head, so that every key is unpacked once for both. Keys come in tiles of
// 128. Five warpgroups:
//   0     warp 0 owns the tensor memory and issues every MMA (kind::f16, fp16 operands, fp32 accumulation):
//         S = Q K^T, O += P V with P from tensor memory, in the order PV_a(j), QK_a(j+1), PV_b(j), QK_b(j+1), so that
//         the tensor cores serve one query tile while the other one's softmax runs
//   1, 2  softmax of query tile a, of b: a thread per row (one lane of tensor memory), online in the log2 domain, in two
//         passes over S (maximum, exponentials); O is rescaled only where the maximum grows by more than 2^8
//   3, 4  unpack K tiles, V tiles: a thread per key reads the key's codes and scales two tiles ahead (block id), one
//         tile ahead (bytes), converts them (e2m1x2 -> f16x2, times the scale, exact) and stores the row in the
//         128-byte-swizzled layout that the MMAs read; a key past the sequence's end becomes zeros, whatever its cell holds
// Registers move from the unpacking warps to the softmax ones (setmaxnreg; the shares add up to the launch's).
//
// Query rows are brought to fp16 by a power of two per row, which the row's score factor takes back: bf16's 8 bits fit,
// and what is 2^-24 below the row's largest magnitude is lost. Weights are rounded to fp16, outputs once to bf16.
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
constexpr int kThreads = 640;
constexpr uint32_t kHalf = 16384;         // 128 rows x 128 bytes (64 fp16 columns)
constexpr float kRescaleThreshold = 8.f;  // log2 units
constexpr float kLowest = -3e38f;         // a maximum before the first score: finite, so that no difference is NaN
constexpr int kRankMax = 256;             // entries that each CTA ranks by their work
constexpr int kFewWaves = 4;              // grids of up to this many CTAs an SM are ordered pair by pair
constexpr size_t kSplitRowBytes = kRankMax * 16 * 16;  // Split::rows, in a workspace
constexpr int kMinPartTiles = 2;          // key tiles of a run, at least, when a list is split

template <int D>
struct Smem {
    static constexpr int k_stages = D == 128 ? 3 : 4, v_stages = D == 128 ? 2 : 4;
    static constexpr uint32_t tile = (D / 64) * kHalf;  // 128 x D fp16
    static constexpr uint32_t q = 0;                    // query tiles a, b; in the end the outputs on their way
    static constexpr uint32_t k = q + 2 * tile;
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
    __nv_bfloat16* out;
    const __nv_bfloat16* q;
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
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
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
            if (kSleep > 0) asm volatile("nanosleep.u32 %0;" ::"r"(kSleep));
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

// A key's codes and scales.
template <int D>
struct RawRow {
    uint4 codes[D / 32];
    uint32_t scales[D / 64];  // 4 scales a word
};

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) prefill_fp4_kernel(const __grid_constant__ Args a) {
    using L_ = Smem<D>;
    constexpr uint32_t kTile = L_::tile;
    constexpr int kKStages = L_::k_stages, kVStages = L_::v_stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L_::bars);
    uint64_t* k_full = bars;                // [kKStages] K tile stored (4 warps)
    uint64_t* k_empty = k_full + kKStages;  // [kKStages] the QKs that read the stage are done
    uint64_t* v_full = k_empty + kKStages;  // [kVStages]
    uint64_t* v_empty = v_full + kVStages;  // [kVStages] the PVs that read the stage are done
    uint64_t* s_full = v_empty + kVStages;  // [2] S of query tile a / b written
    uint64_t* p_full = s_full + 2;          // [2] its P written (4 softmax warps)
    uint64_t* o_done = p_full + 2;          // [2] its last PV finished
    uint64_t* q_full = o_done + 2;          // both query tiles stored (8 softmax warps)
    uint64_t* idle = q_full + 1;            // every MMA issued has finished
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L_::misc);
    const uint32_t abort_flag = smem_u32(smem + L_::misc + 4);
    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2;

    __shared__ int4 chosen[2];  // the entry's sequence, pair, first row of q, rows; length
    __shared__ alignas(16) uint32_t rank_key[kRankMax];  // the entries' work
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
            const int32_t first = 2 * pair * TT, rows = sub > 1 ? min(2 * TT, C - first) : C;
            const int32_t keys = rows <= 0 ? 0 : L - C + first + rows;  // up to the last row's own
            // 24 bits of keys (all of them up to 2^24 tokens), and the number: no two alike
            mine = static_cast<uint32_t>(max(keys, 0)) >> max(8 - __clz(a.cap_tokens), 0) << 8 | (kRankMax - 1 - tid);
        }
        if (tid < kRankMax) rank_key[tid] = mine;
        __syncthreads();
        if (tid < n_entries) {
            int32_t rank = 0;
#pragma unroll 4
            for (int32_t u = 0; u < n_entries; u += 4) {
                const uint4 k = *reinterpret_cast<const uint4*>(rank_key + u);
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
    }
    if (sub == 1) pair = SPLIT ? 0 : gridDim.x - 1 - blockIdx.x;
    const int32_t cta = place * a.num_kv_heads + h;
    if (SPLIT && tid == 0 && blockIdx.x == 0) a.split.rows[cta] = make_int4(0, 0, 0, 0);
    if (C < 0 || C > a.max_chunk || C > L || L > a.cap_tokens) {
        if (tid == 0 && pair == 0) raise_error(a.err, PA_DEVERR_LEN_RANGE);
        return;
    }
    const int32_t t0a = 2 * pair * TT, t0b = t0a + TT;
    if (t0a >= C) return;  // uniform over the CTA
    const int32_t P0 = L - C;

    // ---- key tiles of the CTA, and of each query tile: up to its last row's own key ---------------
    const int32_t all_a = (P0 + min(t0a + TT, C) - 1) / kKeys + 1;
    const int32_t all_b = t0b < C ? (P0 + min(t0b + TT, C) - 1) / kKeys + 1 : 0;
    int32_t n_kv = max(all_a, all_b), base = 0, n_parts = 1;
    if constexpr (SPLIT) {  // this CTA takes one of up to split.parts equal runs of the list
        const int32_t most = max(min(a.split.parts, n_kv / kMinPartTiles), 1), share = (n_kv + most - 1) / most;
        n_parts = (n_kv + share - 1) / share;
        if (static_cast<int32_t>(blockIdx.x) >= n_parts) return;  // uniform over the CTA
        base = blockIdx.x * share;
        n_kv = min(share, n_kv - base);
        if (tid == 0 && blockIdx.x == 0 && n_parts > 1)
            a.split.rows[cta] = make_int4(q0 + t0a, min(TT, C - t0a) * G, max(min(TT, C - t0b), 0) * G, n_parts);
    }
    const int32_t n_a = min(max(all_a - base, 0), n_kv), n_b = min(max(all_b - base, 0), n_kv);

    if (tid == 0) {
        *reinterpret_cast<volatile int32_t*>(smem + L_::misc + 4) = 0;
        for (int i = 0; i < L_::num_bars; ++i) {  // each once: an object in use must not be initialised again
            uint64_t* bar = bars + i;
            const bool four = bar < k_empty || (bar >= v_full && bar < v_empty) || (bar >= p_full && bar < o_done);
            mbar_init(bar, four ? 4 : bar == q_full ? 8 : 1);
        }
        fence_mbarrier_init();
    }
    if (warp == 0) {
        umma::tmem_alloc(tmem_holder, 512);
        umma::tmem_relinquish();
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    // tensor memory columns: S of tile x at 128 x (its P, fp16 pairs, overwrites the first 64 once read),
    // O of tile x at 256 + 128 x
    const uint32_t tmem = *tmem_holder;

    if (group >= 3) {
        // ================================ unpack: K (group 3), V ================================
        fewer_registers<64>();
        const bool is_v = group == 4;
        const int32_t nst = is_v ? kVStages : kKStages, r = tid & 127;  // this thread's key of each tile
        uint64_t* full = is_v ? v_full : k_full;
        uint64_t* empty = is_v ? v_empty : k_empty;
        uint8_t* ring = smem + (is_v ? L_::v : L_::k);
        const uint8_t* pool = is_v ? a.v_cache : a.k_cache;
        const int32_t* table = a.block_table + static_cast<int64_t>(seq) * a.max_blocks;
        // block id of this thread's key in tile j; -1: no such key
        auto block_of = [&](int32_t j) -> int32_t {
            const int32_t key = (base + j) * kKeys + r;
            if (j >= n_kv || key >= L) return -1;
            int32_t phys = __ldg(table + (key >> (4 + a.sub_log2)));
            if (phys < 0 || phys >= a.num_blocks) {
                raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
                phys = 0;
            }
            return phys;
        };
        auto load = [&](int32_t j, int32_t block, RawRow<D>& raw) {
            if (block < 0) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) raw.codes[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) raw.scales[i] = 0u;
                return;
            }
            const int32_t page = ((base + j) * kKeys + r) >> 4;
            const uint8_t* p = pool + fp4_page_at(block, a.num_kv_heads, h, a.sub_log2, page & ((1 << a.sub_log2) - 1), D);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) raw.codes[i] = __ldg(reinterpret_cast<const uint4*>(p + (r & 15) * (D / 2)) + i);
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                raw.scales[i] = __ldg(reinterpret_cast<const uint32_t*>(p + fp4_scales_at(D) + (r & 15) * (D / 16)) + i);
        };
        RawRow<D> raw;
        int32_t next = block_of(1);
        load(0, block_of(0), raw);
        int32_t st = 0;
        uint32_t use = 0;
        for (int32_t j = 0; j < n_kv; ++j) {
            if (use > 0) {
                const bool ok = wait_or_abort<40>(&empty[st], (use - 1) & 1u, abort_flag, a.err);
                if (!__all_sync(0xffffffffu, ok)) break;
            }
            uint8_t* tile = ring + st * kTile;
#pragma unroll
            for (int g = 0; g < D / 16; ++g) {
                const uint32_t s2 = e4m3x2_halves(static_cast<uint16_t>(raw.scales[g / 4] >> (16 * (g / 2 % 2))));
                const uint32_t m = __byte_perm(s2, 0u, g % 2 ? 0x3232u : 0x1010u);
                const uint4 w = raw.codes[g / 2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[4];
                    fp4_halves(g % 2 ? (c ? w.w : w.z) : (c ? w.y : w.x), x);
                    const int chunk = 2 * g + c;
                    *reinterpret_cast<uint4*>(tile + (chunk >> 3) * kHalf + sw128_offset(r, chunk & 7)) =
                        make_uint4(hmul2(x[0], m), hmul2(x[1], m), hmul2(x[2], m), hmul2(x[3], m));
                }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
            if (++st == nst) {
                st = 0;
                ++use;
            }
            const int32_t block = next;
            next = block_of(j + 2);
            load(j + 1, block, raw);
        }
    } else if (group == 0) {
        // ======================================= MMA issuer =====================================
        fewer_registers<32>();
        if (warp == 0 && umma::elect_one()) {
            // One thread issues every MMA (a commit tracks those of its own thread) and does all the waiting.
            constexpr uint32_t idesc_qk = idesc_f16_f32(128, 128, 0);  // Q, K both K-major
            constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, 1);    // P (TMEM), V MN-major
            const uint64_t dq0 = umma::smem_desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t dk0 = umma::smem_desc_sw128(smem_u32(smem + L_::k), 16, 1024);
            const uint64_t dv0 = umma::smem_desc_sw128(smem_u32(smem + L_::v), kHalf, 1024);
            int32_t ks = 0, vs = 0;  // stages of the K tile of the last QK, of V tile j
            uint32_t k_use = 0, v_use = 0;
            auto qk = [&](int x) {
                const uint64_t dq = dq0 + static_cast<uint64_t>(x) * (kTile >> 4), dk = dk0 + static_cast<uint64_t>(ks) * (kTile >> 4);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
                    umma::mma_bf16(tmem + x * 128, dq + off, dk + off, idesc_qk, s > 0);
                }
                umma::commit(&s_full[x]);
            };
            auto pv = [&](int x, bool acc) {
                const uint64_t dv = dv0 + static_cast<uint64_t>(vs) * (kTile >> 4);
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)  // 16 keys per instruction: 8 P columns
                    umma::mma_bf16_tmem_a(tmem + 256 + x * 128, tmem + x * 128 + k * 8, dv + static_cast<uint64_t>(k * (2048 >> 4)),
                                          idesc_pv, acc || k > 0);
            };
            auto wait_k = [&]() {
                const bool ok = wait_or_abort<0>(&k_full[ks], k_use & 1u, abort_flag, a.err);
                umma::fence_after_sync();
                return ok;
            };
            bool ok = wait_or_abort<0>(q_full, 0, abort_flag, a.err) && wait_k();
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
                ok = wait_or_abort<0>(&v_full[vs], v_use & 1u, abort_flag, a.err);
                if (ok && j < n_a) {  // P written, S read
                    ok = wait_or_abort<0>(&p_full[0], j & 1, abort_flag, a.err);
                    umma::fence_after_sync();
                    if (ok) pv(0, j > 0);
                    if (ok && j + 1 == n_a) umma::commit(&o_done[0]);
                }
                if (ok && more) ok = wait_k();
                if (ok && j + 1 < n_a) qk(0);
                if (ok && j < n_b) {
                    ok = wait_or_abort<0>(&p_full[1], j & 1, abort_flag, a.err);
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
            mbar_wait_timeout(idle, 0);
        }
    } else {
        // ==================================== queries, softmax ==================================
        more_registers<152>();
        const int32_t x = group - 1, quad = warp & 3, r = tid & 127;  // query tile, TMEM lane quadrant, row
        const uint32_t inv_G = 65536u / static_cast<uint32_t>(G) + 1;  // x / G = x inv_G / 2^16 for x, G <= 128
        const int32_t tl = static_cast<int32_t>(r * inv_G >> 16), g = r - tl * G;
        const int32_t t_row = (x ? t0b : t0a) + tl, n_x = x ? n_b : n_a;
        const bool row_valid = tl < TT && t_row < C;
        const int64_t row_off = (static_cast<int64_t>(q0 + t_row) * Hq + h * G + g) * D;
        float c1 = a.c1;
        {  // the row to fp16: times 2^-e with 2^e <= its largest magnitude < 2^(e + 1)
            auto chunk = [&](int c) {  // read twice, rather than held
                return row_valid ? __ldg(reinterpret_cast<const uint4*>(a.q + row_off) + c) : make_uint4(0u, 0u, 0u, 0u);
            };
            float top = 0.f;
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = chunk(c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = max3(top, fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u)));
            }
            const int32_t field = static_cast<int32_t>(__float_as_uint(top) >> 23);     // 127 + e
            const int32_t e = field == 255 ? 0 : min(max(field, 1), 253) - 127;         // (not finite: as it is)
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            c1 *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            c1 = fmaxf(c1, 1e-37f);  // a hidden score of -inf times it stays -inf
            const float f = a.negate ? -down : down;
            uint8_t* sq = smem + x * kTile;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = chunk(c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = pack_halves(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
                *reinterpret_cast<uint4*>(sq + (c >> 3) * kHalf + sw128_offset(r, c & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        const int32_t pos = row_valid ? P0 + t_row : L - 1;  // (rows without a query: zeros that go nowhere)
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tmem_s = tmem + x * 128 + lane_off, tmem_o = tmem + 256 + x * 128 + lane_off;
        float m_ref = kLowest, l_sum = 0.f;
        bool ok = true;
        for (int32_t j = 0; j < n_x; ++j) {
            ok = wait_or_abort<20>(&s_full[x], j & 1, abort_flag, a.err);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            umma::fence_after_sync();
            const int32_t kbase = (base + j) * kKeys;
            const bool diag = kbase + kKeys - 1 > pos;  // only these tiles need the causal mask
            // pass 1: row maximum of the raw scores (c1 > 0), eight independent chains
            float mxk[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mxk[k] = -INFINITY;
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
                uint32_t raw[2][32];
                umma::ld_32x32b_x32(tmem_s + c2 * 64, raw[0]);
                umma::ld_32x32b_x32(tmem_s + c2 * 64 + 32, raw[1]);
                umma::wait_ld();
                if (!diag) {
#pragma unroll
                    for (int i = 0; i < 64; i += 2)
                        mxk[(i >> 1) & 7] = max3(mxk[(i >> 1) & 7], __uint_as_float(raw[i >> 5][i & 31]),
                                                 __uint_as_float(raw[i >> 5][(i + 1) & 31]));
                } else {
#pragma unroll
                    for (int i = 0; i < 64; i += 2) {
                        const float x0 = kbase + c2 * 64 + i > pos ? -INFINITY : __uint_as_float(raw[i >> 5][i & 31]);
                        const float x1 =
                            kbase + c2 * 64 + i + 1 > pos ? -INFINITY : __uint_as_float(raw[i >> 5][(i + 1) & 31]);
                        mxk[(i >> 1) & 7] = max3(mxk[(i >> 1) & 7], x0, x1);
                    }
                }
            }
            const float mx = fmaxf(max3(max3(mxk[0], mxk[1], mxk[2]), mxk[3], mxk[4]), max3(mxk[5], mxk[6], mxk[7])) * c1;
            // reference: moved only when the tile's maximum exceeds it by more than 2^8
            const bool grow = mx > m_ref + kRescaleThreshold;
            const float m_new = grow ? mx : m_ref;
            const float alpha = exp2_approx(m_ref - m_new);
            const uint64_t scale2 = pack2(c1, c1), shift2 = pack2(-m_new, -m_new);
            // pass 2: P = 2^(s c1 - m) in fp16 pairs over the first 64 columns of S, 32 keys at a time (each group of S
            // is read before the P columns that overwrite part of it are written)
            uint64_t psum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
                uint32_t raw[32];
                umma::ld_32x32b_x32(tmem_s + c4 * 32, raw);
                umma::wait_ld();
                if (diag) {  // hidden keys: -inf, so that their weight is exactly 0
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (kbase + c4 * 32 + i > pos) raw[i] = __float_as_uint(-INFINITY);
                }
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x0, x1;
                    unpack2(fma2(pack2(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1])), scale2, shift2), x0, x1);
                    const float p0 = exp2_approx(x0), p1 = exp2_approx(x1);
                    psum[e & 3] = add2(psum[e & 3], pack2(p0, p1));
                    pk[e] = pack_halves(p0, p1);
                }
                umma::st_32x32b_x16(tmem_s + c4 * 16, pk);
            }
            umma::wait_st();
            float s0, s1;
            unpack2(add2(add2(psum[0], psum[1]), add2(psum[2], psum[3])), s0, s1);
            l_sum = l_sum * alpha + (s0 + s1);
            if (j > 0 && __any_sync(0xffffffffu, grow)) {
                // O holds the tiles before under the old reference; the PV of tile j - 1 finished
                // before S of tile j was committed, so O can be rescaled now
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t raw[32];
                    umma::ld_32x32b_x32(tmem_o + c * 32, raw);
                    umma::wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) * alpha);
                    umma::st_32x32b_x32(tmem_o + c * 32, raw);
                }
                umma::wait_st();
            }
            m_ref = m_new;
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x]);
        }
        if (ok && n_x > 0) ok = wait_or_abort<20>(&o_done[x], 0, abort_flag, a.err);
        // A tile that no key tile of this CTA concerns (a run that only the other tile sees) has no MMAs: its queries are
        // in shared memory by now, where nothing reads them.
        ok = __all_sync(0xffffffffu, ok);
        umma::fence_after_sync();
        if (SPLIT && n_parts > 1) {
            if (ok) {
                const int64_t run = static_cast<int64_t>(cta) * a.split.parts + blockIdx.x;
                a.split.ml[run * (2 * kRows) + x * kRows + r] = make_float2(m_ref, l_sum);
                float4* po = a.split.o + run * (D / 4) * (2 * kRows) + x * kRows + r;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (n_x > 0) {
                        umma::ld_32x32b_x32(tmem_o + c * 32, o);
                        umma::wait_ld();
                    }
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        po[(c * 8 + v) * (2 * kRows)] =
                            n_x == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                     : make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                   __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                }
            }
        } else {
            const float inv = l_sum == 0.f ? 0.f : a.v_scale / l_sum;
            // the warp's 32 rows through its own rows of the query tile, which no MMA reads any more, so that the
            // stores go out whole lines at a time (a row's 16-byte pieces in different banks, lane by lane)
            constexpr int kPieces = D / 8;
            uint8_t* stage = smem + x * kTile + quad * (32 * 2 * D);
            if (ok && n_x > 0) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    umma::ld_32x32b_x32(tmem_o + c * 32, o);
                    umma::wait_ld();
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        float f[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(o[v * 8 + k]) * inv;
                        *reinterpret_cast<uint4*>(stage + lane * (2 * D) + ((c * 4 + v) ^ (lane & 7)) * 16) =
                            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                       pack_bf16x2(f[6], f[7]));
                    }
                }
                __syncwarp();
                const int64_t to = row_valid ? row_off : -1;
#pragma unroll
                for (int k = 0; k < kPieces; ++k) {
                    const int32_t i = k * 32 + lane, rr = i / kPieces, c = i % kPieces;
                    const int64_t off = __shfl_sync(0xffffffffu, to, rr);
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * (2 * D) + (c ^ (rr & 7)) * 16);
                    if (off >= 0) *reinterpret_cast<uint4*>(a.out + off + c * 8) = v;
                }
            }
        }
    }

    // ---- wind down: the MMAs have retired (warp 0 waited for them) before tensor memory goes ------
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, 512);
    }
}

// Merges the runs of split key lists. Grid: four columns of head_dim x CTA of the unsplit grid; a thread has one row of
// the CTA's two tiles.
template <int D>
__global__ void __launch_bounds__(2 * kRows) prefill_fp4_merge_kernel(__nv_bfloat16* __restrict__ out,
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
    __nv_bfloat16* to = out + (static_cast<int64_t>(rows.x + t) * G * num_kv_heads + h * G + (rr - tt * G)) * D + c4 * 4;
    *reinterpret_cast<uint2*>(to) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// Grids of few waves are ordered pair by pair, others sequence by sequence.
bool few_waves(int64_t entries, int32_t num_kv_heads, int num_sms) {
    return entries <= kRankMax && entries * num_kv_heads <= static_cast<int64_t>(kFewWaves) * num_sms;
}

template <int D, bool SPLIT>
cudaError_t launch_impl(const PrefillArgs& p, float v_scale, const PrefillScoredPlan& plan, void* workspace, int num_sms,
                        cudaStream_t stream) {
    cudaError_t e = allow_smem<prefill_fp4_kernel<D, SPLIT>>(static_cast<int>(Smem<D>::total));
    if (e != cudaSuccess) return e;
    Args a{};
    a.out = static_cast<__nv_bfloat16*>(p.out);
    a.q = static_cast<const __nv_bfloat16*>(p.q);
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
    const int32_t TT = kRows / a.G, pairs = (p.max_chunk_len + 2 * TT - 1) / (2 * TT);
    const int64_t entries = static_cast<int64_t>(pairs) * p.num_seqs;
    const bool by_pair = few_waves(entries, p.num_kv_heads, num_sms);
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
    prefill_fp4_kernel<D, SPLIT><<<grid, kThreads, Smem<D>::total, stream>>>(a);
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
    return cudaLaunchKernelEx(&cfg, prefill_fp4_merge_kernel<D>, a.out, a.split, p.num_kv_heads, a.G, v_scale);
}

}  // namespace

PrefillScoredPlan plan_prefill_fp4(int32_t S, int32_t max_chunk, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_len,
                                   int num_sms) {
    PrefillScoredPlan plan{1, 2, 0};
    if (Hq / Hkv > kRows) return plan;
    const int32_t TT = kRows / (Hq / Hkv);
    const int64_t most = static_cast<int64_t>(max_len / kKeys + 1) / kMinPartTiles;  // runs of the longest list
    if (most < 2) return plan;
    // room for a wave of CTAs, whatever the chunks: a workspace serves every call up to its max_len
    plan.workspace_bytes = kScoredCounterBytes + kSplitRowBytes + static_cast<size_t>(num_sms) * (2 * kRows) * (D * 4 + 8);
    if (S < 1 || max_chunk < 1) return plan;
    const int64_t entries = (static_cast<int64_t>(max_chunk) + 2 * TT - 1) / (2 * TT) * S;
    if (few_waves(entries, Hkv, num_sms))  // one wave of CTAs, each with kMinPartTiles key tiles at least
        plan.parts = static_cast<int32_t>(max(min(num_sms / (entries * Hkv), most), static_cast<int64_t>(1)));
    return plan;
}

bool prefill_fp4_tc_ok(const PrefillArgs& a, const DeviceInfo& dev) {
    return a.dtype == PA_BF16 && a.num_q_heads / a.num_kv_heads <= kRows && a.num_seqs <= 65535 &&
           a.num_kv_heads <= 65535 && static_cast<int>(Smem<128>::total) <= dev.max_smem_optin;
}

cudaError_t launch_prefill_fp4_tc(const PrefillArgs& a, float v_scale, const PrefillScoredPlan& plan, void* workspace,
                                  int num_sms, cudaStream_t stream) {
    if (a.head_dim == 128)
        return plan.parts > 1 ? launch_impl<128, true>(a, v_scale, plan, workspace, num_sms, stream)
                              : launch_impl<128, false>(a, v_scale, plan, workspace, num_sms, stream);
    return plan.parts > 1 ? launch_impl<64, true>(a, v_scale, plan, workspace, num_sms, stream)
                          : launch_impl<64, false>(a, v_scale, plan, workspace, num_sms, stream);
}

}  // namespace pa
