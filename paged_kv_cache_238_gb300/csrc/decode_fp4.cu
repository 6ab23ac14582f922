// Decode over a 4-bit pool: one query row per sequence, on mma.sync in fp16 with pages staged by bulk copies. The pool's
// values (code * scale, 6 significant bits, fp4.cuh) are exact in fp16; a q head's row is brought to fp16 by a power of
// two; weights are rounded to fp16, everything else is fp32. fp32 queries and their weights are sums of two halves, which
// takes twice the MMAs but unpacks no more. The MMAs cut their sums off, always towards zero: over 8000 keys 3e-6 of an
// output. So the second halves are summed by themselves in S, and a page's part of O before it is added (4e-7).
//
// Work list, slices and joins are those of the scored decode kernel (decode_scored.cu): a unit is one page of 16
// tokens of one segment (sequence, kv head, chunk of up to 16 of the kv head's q heads); every CTA builds the list's
// prefix sums from seq_lens, takes an equal contiguous slice and gives each of its warps an equal contiguous part;
// pieces of cut segments meet in shared memory, those of segments cut between CTAs in the workspace, where the CTA
// that counts the last one joins them and puts the counter back to zero.
//
// Unpacking decides this kernel: at the full HBM rate an SM has about 3 thread instructions per element of K or V.
// So fragments are laid out for the codes as they lie in the pool (gid = lane / 4, tig = lane % 4):
//   K, the rows of S^T = K Q^T: a lane takes the D / 4 dims from tig D / 4 on of keys gid and gid + 8 (16 bytes at
//     D = 128, one load), 4 dims to a k16 step; Q's fragments are permuted alike. The dims lie in 2 groups (1 at 64).
//   V, the rows of O^T += V^T P^T: a lane takes the D / 8 dims from gid D / 8 on, one group's, of four keys, two to a
//     row of fragments. Codes of two keys are interleaved as nibbles first (one shift and one select per word), so
//     that the conversion of a byte gives the pair of keys that a fragment register holds.
//   Each register then costs one conversion (e2m1x2 to f16x2) and one product with the scales: 1 instruction an element.
// The four keys of tig are those of rows 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9 of S^T; row r of a page's S^T is key
// key_of(r), such that they are keys tig, tig + 4, tig + 8, tig + 12 and the loads of V meet two to a bank, not four.
// The softmax is online in the log2 domain against a reference that moves only when a score exceeds it by 2^kLag:
// most steps then need no reduction across lanes at all (a vote) and rescale nothing.
//
// Bound: the unpacking's issue slots and latencies, then HBM: 300 warp instructions a page of K and V at D = 128 (64
// conversions, 64 products with scales, 16 MMAs among them), 2.6 issued a cycle and SM. 8 sequences of 20000 to 32768 keys,
// 64 q / 8 kv heads of 128: 57 us, 4.2 TB/s, 62 % of the measured copy rate (32 sequences of 32768: 228 us, 78 %); 64 of 500
// to 16384, 32 q / 8 kv heads: 75 us (67 %), of which 4.4 pass until the first pages have come and 8 to 11 go to the slowest
// SM and the joins. 4 sequences of up to 700 keys: 9.1 us in a graph, a chain of latencies.
// fp32 queries (before on the CUDA cores): 8 of 8000 to 9000 keys, 16 q / 4 kv heads of 128, 21.7 us (54.8); 64 of 10 to
// 2000, 16 heads of 64, 22.3 (58.1); 24 of up to 777, 12 q / 4 kv heads of 64, 10.2 (12.1).
#include <math.h>

#include <type_traits>

#include "fp4.cuh"
#include "pa_internal.h"
#include "scored.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSeqs = 1024;  // sequences of one launch: their units live in shared memory
constexpr int kMaxHeads = 16;   // q heads of one segment
constexpr int kMinSlice = 4;    // units of a CTA's slice, at least
constexpr float kJoinWeight = 1.f / 1.5f;  // a segment of n units is cut into about sqrt(1.5 n) pieces at most
// A segment's start and end weigh as much as this many pages: 96 sequences of 16 to 2048 keys, 16 heads of 64, 24.8 us (1:
// 29.2, 2: 28.1, 7: 24.9); 64 of 500 to 16384, 32 q / 8 kv heads of 128, 75.2 us (1: 77.1).
constexpr int kSegmentUnits = 4;
constexpr float kLag = 8.f;                // log2 units
constexpr float kLowest = -3e38f;          // a reference before the first score: finite, so that no difference is NaN

// How q of type T and the weights come to fp16. bf16: q's row as it is once its largest magnitude lies in [2^14, 2^15), the
// weights rounded. fp32: both as sums of two halves, 22 bits. The row's top of 2^14 keeps what is small next to it within
// fp16's range (2^-39 of the largest is lost). A weight of 2^7 at the reference does that for the weights: those
// down to 2^-21 of the largest keep their 11 bits, and what is lost is 2^-32 of it; many keys far below one add up to a part
// of the output that 2^-25, with a weight of 1 there, would round away.
template <typename T>
struct Fp16Form {
    static constexpr bool kTwo = std::is_same<T, float>::value;
    static constexpr int kPieces = kTwo ? 2 : 1;
};
constexpr int kTop = 14;       // a row's largest magnitude: 2^kTop ..
constexpr float kAbove = 7.f;  // log2 of the weight of a score at the reference; 2^(kAbove + kLag) is within fp16

// Pages of one step of a warp, and room for one step: 64 sequences of 500 to 16384 keys 76 us, with steps of two pages and
// room for two or four of them 85.
constexpr int kStepPages = 4;
__host__ __device__ inline uint32_t up(uint32_t x, uint32_t a) { return (x + a - 1) / a * a; }

struct Layout {
    uint32_t ring_bytes, ring, piece0, piece_ml, weight, meta, bars, flags, prefix, lens, total;
};
// NW warps, hs q heads per segment, S sequences.
__host__ __device__ inline Layout layout(int NW, int hs, int D, int S) {
    Layout l;
    uint32_t o = 0;
    const uint32_t pages = 2u * fp4_page_bytes(D) * kStepPages, piece = static_cast<uint32_t>(hs) * D * 4u;
    l.ring_bytes = pages > piece ? pages : piece;  // a step's K pages, its V pages; in the end the warp's last piece
    l.ring = o;      o += static_cast<uint32_t>(NW) * l.ring_bytes;
    l.piece0 = o;    o += static_cast<uint32_t>(NW) * hs * D * 4u;       // each warp's first piece
    l.piece_ml = o;  o += static_cast<uint32_t>(NW) * 2u * hs * 8u;      // (max, sum) of both pieces
    l.weight = o;    o += static_cast<uint32_t>(NW) * 2u * hs * 12u;     // the pieces' weights, and (max, sum) of their run
    l.meta = up(o, 16u);  o = l.meta + static_cast<uint32_t>(NW) * 2u * 16u;  // segment of each piece
    l.bars = up(o, 16u);  o = l.bars + static_cast<uint32_t>(NW) * 2u * 8u;
    l.flags = o;     o += 32u;
    l.prefix = up(o, 16u);  o = l.prefix + up((S + 1) * 4u, 16u);
    l.lens = o;      o += static_cast<uint32_t>(S) * 4u;
    l.total = o + 128u;
    return l;
}

struct Params {
    void* out;
    const void* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* block_table;
    const int32_t* seq_lens;
    int32_t max_blocks, S, num_kv_heads, G, head_chunks, num_blocks, sub_log2, cap_tokens;
    float c1;          // scale log2 e
    float v_scale;
    int32_t* counter;  // [kScoredSegments] CTA pieces finished per segment; zero between calls
    float* piece_o;    // [C][2][hs][D]
    float2* piece_ml;  // [C][2][hs]
    uint32_t* err;
    uint64_t wait_limit_ns;
    int32_t drill;  // the warp of the list's first unit: its first K step waits for 16 bytes that no copy brings
};

__device__ __forceinline__ void bulk_copy_g2s(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar,
                                              uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(smem_dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint16_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// D = A(16x16, row) * B(16x8, col) + D, fp16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D = A B
__device__ __forceinline__ void mma_f16_fresh(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_halves(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float x, float y, float z, float w) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
}
__device__ __forceinline__ void store4(float* p, float x, float y, float z, float w) {
    *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
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
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t mask) { return (a & mask) | (b & ~mask); }

// The key, of a page's 16, in row r of S^T: rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 are keys t, t + 4, t + 8, t + 12.
__device__ __forceinline__ int32_t key_of(int32_t r) { return (r & 8) | ((r & 1) << 2) | ((r >> 1) & 3); }

// Sequence s with prefix[s] <= u < prefix[s + 1].
__device__ __forceinline__ int32_t find_seq(const int32_t* prefix, int32_t S, int32_t u) {
    int32_t lo = 0, hi = S;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (prefix[mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
}

// Position in the work list: sequence s, its segment h of nh, unit j: page j of np, or, from np on, one
// of the kSegmentUnits units without a page that stand for what a segment costs besides its pages.
struct Cursor {
    int32_t s, h, j, np, len;
    __device__ __forceinline__ void load(const int32_t* lens) {
        len = lens[s];
        np = (len + kPageTokens - 1) / kPageTokens;
    }
    __device__ __forceinline__ void at(const int32_t* prefix, const int32_t* lens, int32_t S, int32_t u) {
        s = find_seq(prefix, S, u);
        load(lens);
        const int32_t r = u - prefix[s], units = np + kSegmentUnits;
        h = r / units;
        j = r - h * units;
    }
    __device__ __forceinline__ void advance(int32_t pages, const int32_t* prefix, const int32_t* lens, int32_t S, int32_t nh) {
        j += pages;
        if (j < np + kSegmentUnits) return;
        j = 0;
        if (++h < nh) return;
        h = 0;
        do { ++s; } while (s < S && prefix[s + 1] == prefix[s]);
        if (s < S) load(lens);
    }
};

// A segment's piece: its segment number (-1: none), sequence, segment within the sequence, pages.
struct Piece {
    int32_t seg, s, h, np;
};

// NH: groups of 8 q heads of a segment (up to 8 NH heads).
template <typename T, int D, int NW, int NH>
__global__ void __launch_bounds__(NW * 32, 1)
    decode_fp4_kernel(const __grid_constant__ Params a) {
    constexpr uint32_t kPage = fp4_page_bytes(D), kScales = fp4_scales_at(D);
    constexpr int KS = D / 16, NMT = D / 16, SP = kStepPages, DL = D / 8;  // DL: dims of a lane's V rows
    constexpr int NTH = NW * 32;
    using F = Fp16Form<T>;
    constexpr int PC = F::kPieces, QW = 2 * PC;  // halves of a number; words of 4 elements of q
    T* const out = static_cast<T*>(a.out);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int32_t S = a.S, G = a.G, NHC = a.head_chunks, Hq = G * a.num_kv_heads;
    const int32_t hs = min(G, kMaxHeads), nh = a.num_kv_heads * NHC;  // heads and segments per sequence
    const Layout L = layout(NW, hs, D, S);
    float* piece0 = reinterpret_cast<float*>(smem + L.piece0);
    float2* piece_ml = reinterpret_cast<float2*>(smem + L.piece_ml);
    Piece* meta = reinterpret_cast<Piece*>(smem + L.meta);  // [2 NW]
    uint64_t* bars_all = reinterpret_cast<uint64_t*>(smem + L.bars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.flags);
    int32_t* cross = reinterpret_cast<int32_t*>(smem + L.flags + 8);  // [2] pieces of segments cut by the CTA's slice, [2] to join
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + L.prefix);
    int32_t* lens = reinterpret_cast<int32_t*>(smem + L.lens);
    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        *abort_flag = 0;
        cross[0] = cross[1] = -1;
        cross[2] = cross[3] = 0;
    }
    if (lane == 0) {
        meta[warp * 2].seg = meta[warp * 2 + 1].seg = -1;
        for (int i = 0; i < 2; ++i) mbar_init(&bars_all[warp * 2 + i], 1);
        fence_mbarrier_init();
    }
    // A programmatic launch: everything above ran beside the tail of the kernel before this one;
    // every input, output and the workspace are touched after this wait.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the work list: units of each sequence, block-wide exclusive scan ------------
    {
        __shared__ int32_t warp_tot[NW];
        const int32_t per = (S + NTH - 1) / NTH;
        const int32_t b = min(S, tid * per), e = min(S, b + per);
        int32_t local = 0;
        for (int32_t s = b; s < e; ++s) {
            int32_t len = __ldg(a.seq_lens + s);
            if (len < 0 || len > a.cap_tokens) {
                if (blockIdx.x == 0) raise_error(a.err, PA_DEVERR_LEN_RANGE);
                len = len < 0 ? 0 : a.cap_tokens;
            }
            lens[s] = len;
            const int32_t units = len > 0 ? ((len + kPageTokens - 1) / kPageTokens + kSegmentUnits) * nh : 0;
            prefix[s] = units;
            local += units;
        }
        int32_t incl = local;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) warp_tot[warp] = incl;
        __syncthreads();
        int32_t run = incl - local;
        for (int w = 0; w < warp; ++w) run += warp_tot[w];
        for (int32_t s = b; s < e; ++s) {
            const int32_t units = prefix[s];
            prefix[s] = run;
            run += units;
        }
        if (tid == NTH - 1) prefix[S] = run;
        __syncthreads();
    }
    const int32_t U = prefix[S];
    // slices of equal length, one per CTA, but not below kMinSlice, nor below where the time that n / chunk
    // pieces of a segment of n units take to join outweighs the shorter slices (about sqrt(n / 1.5))
    const float n_mean = static_cast<float>(U) / static_cast<float>(S * a.num_kv_heads * NHC);
    const int32_t chunk = max(max((U + static_cast<int32_t>(gridDim.x) - 1) / static_cast<int32_t>(gridDim.x), kMinSlice),
                              static_cast<int32_t>(sqrtf(n_mean * kJoinWeight)));
    // rows that see nothing are zero (spread over the CTAs)
    for (int32_t s = blockIdx.x; s < S; s += gridDim.x) {
        if (prefix[s + 1] != prefix[s]) continue;
        uint32_t* z = reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(s) * Hq * D);
        for (int32_t i = tid; i < Hq * D / 4 * QW; i += NTH) z[i] = 0u;
    }
    const int64_t first = static_cast<int64_t>(blockIdx.x) * chunk;
    if (first >= U) return;  // uniform over the CTA
    const int32_t u0 = static_cast<int32_t>(first), u1 = min(U, u0 + chunk);
    const int32_t per_warp = (u1 - u0 + NW - 1) / NW;
    const int32_t a_w = u0 + warp * per_warp, n = max(0, min(u1 - a_w, per_warp));
    uint8_t* ring = smem + L.ring + static_cast<uint32_t>(warp) * L.ring_bytes;
    const uint32_t ring_u32 = smem_u32(ring);
    uint64_t* bars = bars_all + warp * 2;  // a step's K has landed, its V
    const int32_t gid = lane >> 2, tig = lane & 3;

    if (n > 0) {
        // Page in the pool of unit a_w + 32 k + lane; -1: a unit without one.
        auto lane_page = [&](int32_t k) -> int32_t {
            if (32 * k + lane >= n) return -1;
            Cursor c;
            c.at(prefix, lens, S, a_w + 32 * k + lane);
            if (c.j >= c.np) return -1;
            int32_t phys = __ldg(a.block_table + static_cast<int64_t>(c.s) * a.max_blocks + (c.j >> a.sub_log2));
            if (phys < 0 || phys >= a.num_blocks) {
                raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
                phys = 0;
            }
            return ((phys * a.num_kv_heads + c.h / NHC) << a.sub_log2) + (c.j & ((1 << a.sub_log2) - 1));
        };
        // pages are read once per call: let them leave L2 first
        const uint64_t kv_policy = l2_policy_evict_first();
        // Step i holds units SP i .. of the part; lane x < SP copies the K or V page of unit x into its place. There is
        // room for one step: the next one's K is sent for when this one's scores are done, its V at the step's end.
        // Block ids come 32 units at a time, the next 32 on their way while these are used.
        int32_t k_steps = 0, v_steps = 0, id_cur = lane_page(0), id_nxt = n > 32 ? lane_page(1) : -1, step_id = -1;
        auto send = [&](const uint8_t* pool, uint8_t* to, uint64_t* bar, uint32_t more) {
            const bool mine = lane < SP && step_id >= 0 && !*abort_flag;
            const uint32_t copies = __ballot_sync(0xffffffffu, mine);
            if (lane == 0) mbar_arrive_expect_tx(bar, __popc(copies) * kPage + more);
            __syncwarp();
            if (mine) bulk_copy_g2s(to + lane * kPage, pool + static_cast<int64_t>(step_id) * kPage, kPage, bar, kv_policy);
        };
        auto send_k = [&]() {
            step_id = __shfl_sync(0xffffffffu, id_cur, (k_steps * SP + lane) & 31);
            send(a.k_cache, ring, &bars[0], a.drill && k_steps == 0 && a_w == 0 ? 16u : 0u);
            ++k_steps;
            if (((k_steps * SP) & 31) == 0) {
                id_cur = id_nxt;
                const int32_t k = k_steps * SP / 32 + 1;
                id_nxt = 32 * k < n ? lane_page(k) : -1;
            }
        };
        auto send_v = [&]() {
            send(a.v_cache, ring + SP * kPage, &bars[1], 0u);
            ++v_steps;
        };
        send_k();
        send_v();
        auto landed = [&](uint64_t* bar, int32_t step) {
            if (__all_sync(0xffffffffu, mbar_wait_bounded(bar, static_cast<uint32_t>(step) & 1u, abort_flag, a.wait_limit_ns)))
                return true;
            if (lane == 0) {
                if (!*abort_flag) raise_error(a.err, PA_DEVERR_WAIT_TIMEOUT);
                *abort_flag = 1;
            }
            __syncwarp();
            return false;
        };

        Cursor wc;
        wc.at(prefix, lens, S, a_w);
        // Fragment ownership (gid = lane / 4, tig = lane % 4):
        //   qb[f][c][ks] Q^T as B, piece c: head 8 f + gid, dims tig D / 4 + 4 ks .. + 3
        //   sc[i][f][e] S^T of page i: key key_of(gid + 8 (e / 2)), head 8 f + 2 tig + e % 2
        //   acc[f][mt]  O^T: head_dim gid D / 8 + 2 mt + e / 2, head 8 f + 2 tig + e % 2
        uint32_t qb[NH][PC][KS][2];
        float acc[NH][NMT][4], mh[NH][2], lh[NH][2], c1[NH][2];
        int32_t ng = 0, head0 = 0;
        bool cut_left = false;
        bool first_page = true;  // of a segment in this part
        const int32_t key_a = key_of(gid);  // and key_a + 8
        const float hidden = a.c1 < 0.f ? INFINITY : -INFINITY;  // a raw score whose weight is 0
        // this lane's places: K's codes and scales, V's
        const uint32_t at_k = ring_u32 + key_a * (D / 2) + tig * (D / 8);
        const uint32_t at_ks = ring_u32 + kScales + key_a * (D / 16) + tig * (D / 64);
        const uint32_t at_v = ring_u32 + SP * kPage + tig * (D / 2) + gid * (D / 16);
        const uint32_t at_vs = ring_u32 + SP * kPage + kScales + tig * (D / 16) + gid * DL / 16;
        // Pages slot .. of the step (`pages` of them, `left` keys from the first on). next: the step's last pages, and
        // another step follows, whose K is sent for behind the scores and whose V at the end. False: a wait gave up.
        auto attend = [&](auto pages, int32_t slot, int32_t left, bool wait_v, bool next) -> bool {
            constexpr int NP = decltype(pages)::value;
            const bool masked = left < NP * kPageTokens;
            // ---- S^T = K Q^T ----
            float sc[NP][NH][4];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                constexpr int WK = D / 32;  // words of a lane's dims of a key
                const uint32_t page = (slot + i) * kPage;
                uint32_t w0[WK], w1[WK], s0, s1;
                if constexpr (D == 128) {
                    const uint4 x = lds128(at_k + page), y = lds128(at_k + page + 8 * (D / 2));
                    w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
                    w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
                    s0 = e4m3x2_halves(lds16(at_ks + page));
                    s1 = e4m3x2_halves(lds16(at_ks + page + 8 * (D / 16)));
                } else {
                    const uint2 x = lds64(at_k + page), y = lds64(at_k + page + 8 * (D / 2));
                    w0[0] = x.x, w0[1] = x.y, w1[0] = y.x, w1[1] = y.y;
                    s0 = e4m3x2_halves(static_cast<uint16_t>(lds8(at_ks + page)));
                    s1 = e4m3x2_halves(static_cast<uint16_t>(lds8(at_ks + page + 8 * (D / 16))));
                }
                float low[NH][4];  // two pieces: the products of the second ones, which are small, by themselves
#pragma unroll
                for (int f = 0; f < NH; ++f)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[i][f][e] = low[f][e] = 0.f;
#pragma unroll
                for (int w = 0; w < WK; ++w) {  // two k16 steps
                    const uint32_t pick = w < 2 ? 0x1010u : 0x3232u;
                    const uint32_t m0 = __byte_perm(s0, 0u, pick), m1 = __byte_perm(s1, 0u, pick);
                    uint32_t h0[4], h1[4];
                    fp4_halves(w0[w], h0);
                    fp4_halves(w1[w], h1);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t fa[4] = {hmul2(h0[2 * x], m0), hmul2(h1[2 * x], m1), hmul2(h0[2 * x + 1], m0),
                                                hmul2(h1[2 * x + 1], m1)};
#pragma unroll
                        for (int f = 0; f < NH; ++f) {
                            if constexpr (F::kTwo) mma_f16(low[f], fa, qb[f][1][2 * w + x][0], qb[f][1][2 * w + x][1]);
                            mma_f16(sc[i][f], fa, qb[f][0][2 * w + x][0], qb[f][0][2 * w + x][1]);
                        }
                    }
                }
                if constexpr (F::kTwo) {
#pragma unroll
                    for (int f = 0; f < NH; ++f)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i][f][e] += low[f][e];
                }
            }
            if (next) {  // K has been read
                __syncwarp();
                send_k();
            }
            if (masked) {
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i * kPageTokens + key_a + 4 * (e & 2) >= left)
#pragma unroll
                            for (int f = 0; f < NH; ++f) sc[i][f][e] = hidden;
            }
            // ---- weights 2^(score - reference); the references move where a score exceeds one by more than kLag ----
            float x[NP][NH][4], top = -INFINITY;
            auto shifted = [&]() {
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int f = 0; f < NH; ++f)
#pragma unroll
                        for (int e = 0; e < 4; e += 2)
                            unpack2(fma2(pack2(sc[i][f][e], sc[i][f][e + 1]), pack2(c1[f][0], c1[f][1]), pack2(-mh[f][0], -mh[f][1])),
                                    x[i][f][e], x[i][f][e + 1]);
            };
            shifted();
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int f = 0; f < NH; ++f) top = max3(max3(top, x[i][f][0], x[i][f][1]), x[i][f][2], x[i][f][3]);
            if (__any_sync(0xffffffffu, top > kAbove + kLag)) {
#pragma unroll
                for (int f = 0; f < NH; ++f) {
                    float cc[2];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int i = 0; i < NP; ++i) mx = max3(mx, sc[i][f][hh] * c1[f][hh], sc[i][f][2 + hh] * c1[f][hh]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const float mn = fmaxf(mh[f][hh], mx - kAbove);
                        cc[hh] = exp2_approx(mh[f][hh] - mn);
                        mh[f][hh] = mn;
                        lh[f][hh] *= cc[hh];
                    }
#pragma unroll
                    for (int mt = 0; mt < NMT; ++mt) {
                        acc[f][mt][0] *= cc[0];
                        acc[f][mt][1] *= cc[1];
                        acc[f][mt][2] *= cc[0];
                        acc[f][mt][3] *= cc[1];
                    }
                }
                shifted();
            }
            uint32_t pb[NP][NH][PC][2];
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int f = 0; f < NH; ++f) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = exp2_approx(x[i][f][e]);
                    uint64_t l2 = pack2(lh[f][0], lh[f][1]);
                    l2 = add2(add2(l2, pack2(p[0], p[1])), pack2(p[2], p[3]));
                    unpack2(l2, lh[f][0], lh[f][1]);
#pragma unroll
                    for (int c = 0; c < PC; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t h = pack_halves(p[2 * e], p[2 * e + 1]);
                            pb[i][f][c][e] = movmatrix_trans(h);
                            if (c + 1 < PC) {  // what it leaves
                                const float2 held = halves_to_floats(h);
                                p[2 * e] -= held.x;
                                p[2 * e + 1] -= held.y;
                            }
                        }
                }
            // ---- O^T += V^T P^T ----
            if (wait_v && !landed(&bars[1], v_steps - 1)) return false;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                constexpr int WV = D / 64;  // words of a lane's dims of a key
                const uint32_t page = (slot + i) * kPage;
                uint32_t w[4][WV], sb[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {  // key tig + 4 x
                    if constexpr (D == 128) {
                        const uint2 v = lds64(at_v + page + 4 * x * (D / 2));
                        w[x][0] = v.x, w[x][1] = v.y;
                    } else {
                        w[x][0] = lds32(at_v + page + 4 * x * (D / 2));
                    }
                    sb[x] = lds8(at_vs + page + 4 * x * (D / 16));
                }
                if (masked) {  // a key that does not count may hold anything, a scale of NaN too; codes are numbers
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (i * kPageTokens + tig + 4 * x >= left) sb[x] = 0u;
                }
                const uint32_t m0 = e4m3x2_halves(static_cast<uint16_t>(__byte_perm(sb[0], sb[1], 0x0040u)));
                const uint32_t m1 = e4m3x2_halves(static_cast<uint16_t>(__byte_perm(sb[2], sb[3], 0x0040u)));
#pragma unroll
                for (int x = 0; x < WV; ++x) {
                    uint32_t e0[4], e1[4], o0[4], o1[4];  // even dims and odd dims of keys (0, 1) and (2, 3)
                    fp4_halves(select_bits(w[0][x], w[1][x] << 4, 0x0f0f0f0fu), e0);
                    fp4_halves(select_bits(w[0][x] >> 4, w[1][x], 0x0f0f0f0fu), o0);
                    fp4_halves(select_bits(w[2][x], w[3][x] << 4, 0x0f0f0f0fu), e1);
                    fp4_halves(select_bits(w[2][x] >> 4, w[3][x], 0x0f0f0f0fu), o1);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t fa[4] = {hmul2(e0[b], m0), hmul2(o0[b], m0), hmul2(e1[b], m1), hmul2(o1[b], m1)};
#pragma unroll
                        for (int f = 0; f < NH; ++f) {
                            float(&o)[4] = acc[f][4 * x + b];
                            if constexpr (F::kTwo) {  // the page's part by itself, added with rounding
                                float part[4];
                                mma_f16_fresh(part, fa, pb[i][f][1][0], pb[i][f][1][1]);
                                mma_f16(part, fa, pb[i][f][0][0], pb[i][f][0][1]);
#pragma unroll
                                for (int e = 0; e < 4; e += 2) unpack2(add2(pack2(o[e], o[e + 1]), pack2(part[e], part[e + 1])), o[e], o[e + 1]);
                            } else {
                                mma_f16(o, fa, pb[i][f][0][0], pb[i][f][0][1]);
                            }
                        }
                    }
                }
            }
            if (next) {  // V has been read
                __syncwarp();
                send_v();
            }
            return true;
        };
        for (int32_t t = 0, cnt; t < n; t += cnt) {
            // up to the end of the step, of the segment, of the part; or units without a page
            const int32_t slot = t & (SP - 1);
            const bool page_here = wc.j < wc.np;
            cnt = min(min(SP - slot, n - t), (page_here ? wc.np : wc.np + kSegmentUnits) - wc.j);
            const bool step_first = slot == 0, step_last = slot + cnt == SP;
            uint32_t raw[NH][KS][QW];  // 4 elements of q each
            const bool fresh = page_here && first_page;
            if (fresh) {  // a new segment: its query rows, on their way while the step's pages are waited for
                const int32_t hk = wc.h / NHC, g0 = (wc.h - hk * NHC) * kMaxHeads;
                ng = min(G - g0, kMaxHeads);
                head0 = hk * G + g0;
#pragma unroll
                for (int f = 0; f < NH; ++f) {
                    const T* row = static_cast<const T*>(a.q) + (static_cast<int64_t>(wc.s) * Hq + head0 + f * 8 + gid) * D + tig * (D / 4);
#pragma unroll
                    for (int ks = 0; ks < KS; ks += 4 / QW) {
                        const uint4 w = f * 8 + gid < ng ? __ldg(reinterpret_cast<const uint4*>(row + 4 * ks)) : make_uint4(0u, 0u, 0u, 0u);
                        raw[f][ks][0] = w.x, raw[f][ks][1] = w.y;
                        if constexpr (F::kTwo) raw[f][ks][2] = w.z, raw[f][ks][3] = w.w;
                        else raw[f][ks + 1][0] = w.z, raw[f][ks + 1][1] = w.w;
                    }
                }
            }
            if (step_first && !landed(&bars[0], k_steps - 1)) break;
            first_page = !page_here;
            if (!page_here) {
                if (step_last && t + cnt < n) send_k();
                if (step_first && !landed(&bars[1], v_steps - 1)) break;
                if (step_last && t + cnt < n) send_v();
                wc.advance(cnt, prefix, lens, S, nh);
                continue;
            }
            if (fresh) {
#pragma unroll
                for (int f = 0; f < NH; ++f) {
                    // the row to fp16: times 2^-e, so that its largest magnitude lies in [2^kTop, 2^(kTop + 1))
                    auto element = [&](int ks, int x) -> float {
                        if constexpr (F::kTwo) return __uint_as_float(raw[f][ks][x]);
                        else return __uint_as_float(x & 1 ? raw[f][ks][x / 2] & 0xffff0000u : raw[f][ks][x / 2] << 16);
                    };
                    float top = 0.f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int x = 0; x < 4; x += 2) top = max3(top, fabsf(element(ks, x)), fabsf(element(ks, x + 1)));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int32_t field = static_cast<int32_t>(__float_as_uint(top) >> 23);  // 127 + kTop + e
                    // (not finite: as it is; rows below 2^-112: times 2^126)
                    const int32_t e = field == 255 ? 0 : max(field, 1 + kTop) - 127 - kTop;
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    const float up2 = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float y0 = element(ks, 2 * x) * down, y1 = element(ks, 2 * x + 1) * down;
#pragma unroll
                            for (int c = 0; c < PC; ++c) {
                                const uint32_t h = pack_halves(y0, y1);
                                qb[f][c][ks][x] = h;
                                if (c + 1 < PC) {  // what it leaves, exactly
                                    const float2 held = halves_to_floats(h);
                                    y0 -= held.x;
                                    y1 -= held.y;
                                }
                            }
                        }
#pragma unroll
                    for (int mt = 0; mt < NMT; ++mt) acc[f][mt][0] = acc[f][mt][1] = acc[f][mt][2] = acc[f][mt][3] = 0.f;
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        mh[f][hh] = kLowest;
                        lh[f][hh] = 0.f;
                        c1[f][hh] = a.c1 * __shfl_sync(0xffffffffu, up2, (2 * tig + hh) * 4);
                        if (fabsf(c1[f][hh]) < 1e-37f) c1[f][hh] = copysignf(1e-37f, -hidden);  // times `hidden`: -inf, also for a scale of -0
                    }
                }
                cut_left = wc.j > 0;
            }
            // the step's pages at once, or those that this segment has of it one by one
            int32_t left = wc.len - wc.j * kPageTokens;  // keys from here on
            const bool more = step_last && t + cnt < n;
            bool ok = true;
            if (cnt == SP) {
                ok = attend(std::integral_constant<int, SP>(), 0, left, true, more);
            } else {
#pragma unroll 1
                for (int32_t x = 0; x < cnt && ok; ++x, left -= kPageTokens)
                    ok = attend(std::integral_constant<int, 1>(), slot + x, left, step_first && x == 0, more && x == cnt - 1);
            }
            if (!ok) break;

            if (t + cnt == n || wc.j + cnt == wc.np) {  // the part's last page of this segment
                float Lh[NH][2];
#pragma unroll
                for (int f = 0; f < NH; ++f) {
                    Lh[f][0] = lh[f][0];
                    Lh[f][1] = lh[f][1];
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
#pragma unroll
                    for (int f = 0; f < NH; ++f) {
                        Lh[f][0] += __shfl_xor_sync(0xffffffffu, Lh[f][0], off);
                        Lh[f][1] += __shfl_xor_sync(0xffffffffu, Lh[f][1], off);
                    }
                const bool inside = !cut_left && wc.j + cnt == wc.np;
                const int slot = cut_left ? 0 : 1;  // a piece cut on the left is the part's first, else its last
                __syncwarp();                           // slot 1 reuses the ring, idle after the last page
                float* pa_acc = slot == 0 ? piece0 + static_cast<uint32_t>(warp) * hs * D : reinterpret_cast<float*>(ring);
                T* o = out + (static_cast<int64_t>(wc.s) * Hq + head0) * D;
#pragma unroll
                for (int f = 0; f < NH; ++f)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int32_t head = f * 8 + tig * 2 + hh;
                        if (head >= ng) continue;
                        if (inside) {
                            const float inv = Lh[f][hh] == 0.f ? 0.f : a.v_scale / Lh[f][hh];
#pragma unroll
                            for (int c = 0; c < DL / 4; ++c)
                                store4(o + head * D + gid * DL + 4 * c, acc[f][2 * c][hh] * inv, acc[f][2 * c][2 + hh] * inv,
                                       acc[f][2 * c + 1][hh] * inv, acc[f][2 * c + 1][2 + hh] * inv);
                        } else {
#pragma unroll
                            for (int mt = 0; mt < NMT; ++mt)
                                *reinterpret_cast<float2*>(pa_acc + head * D + gid * DL + 2 * mt) =
                                    make_float2(acc[f][mt][hh], acc[f][mt][2 + hh]);
                            if (gid == 0) piece_ml[(warp * 2 + slot) * hs + head] = make_float2(mh[f][hh], Lh[f][hh]);
                        }
                    }
                if (!inside && lane == 0) meta[warp * 2 + slot] = Piece{wc.s * nh + wc.h, wc.s, wc.h, wc.np};
            }
            wc.advance(cnt, prefix, lens, S, nh);
        }
        // copies still in flight after an abort land before the CTA can exit
        if (*abort_flag && lane == 0) {
            mbar_wait_timeout(&bars[0], static_cast<uint32_t>(k_steps - 1) & 1u, a.wait_limit_ns);
            mbar_wait_timeout(&bars[1], static_cast<uint32_t>(v_steps - 1) & 1u, a.wait_limit_ns);
        }
    }
    __syncthreads();
    if (*abort_flag) return;

    // ---- pieces cut between this CTA's warps: runs of equal segments in list order -------------
    // First every (piece, head) weighs itself against its run: e_i / sum e_k l_k with e_i = 2^(m_i - M)
    // (pieces hold unnormalised outputs); then all threads add the pieces up. A lane stands for a piece; a place
    // without one counts to the run before it, so that runs are contiguous.
    constexpr int V4 = D / 4;
    float* weight = reinterpret_cast<float*>(smem + L.weight);            // [2 NW][hs]
    float2* run_ml = reinterpret_cast<float2*>(weight + 2 * NW * hs);     // [2 NW][hs] the run's (M, sum), at its first piece
    uint32_t held, starts;  // places with a piece; those whose predecessor belongs to another segment
    int32_t my_first;       // the first place of this lane's run
    {
        const int32_t seg = lane < 2 * NW ? meta[lane].seg : -1;
        held = __ballot_sync(0xffffffffu, seg >= 0);
        const uint32_t before = held & ((1u << lane) - 1u);
        const int32_t prev = __shfl_sync(0xffffffffu, seg, before ? 31 - __clz(before) : lane);
        starts = __ballot_sync(0xffffffffu, seg >= 0 && (before == 0u || prev != seg));
        const uint32_t upto = starts & (0xffffffffu >> (31 - lane));
        my_first = upto ? 31 - __clz(upto) : -1;
    }
    for (int32_t g = warp; g < hs; g += NW) {  // a warp per head
        const bool piece = (held >> lane & 1u) != 0u;
        const float2 ml = piece ? piece_ml[lane * hs + g] : make_float2(-INFINITY, 0.f);
        float M = ml.x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {  // over the run's places from here on
            const float o = __shfl_down_sync(0xffffffffu, M, off);
            const int32_t f = __shfl_down_sync(0xffffffffu, my_first, off);
            if (lane + off < 32 && f == my_first) M = fmaxf(M, o);
        }
        M = __shfl_sync(0xffffffffu, M, my_first < 0 ? lane : my_first);
        const float e = exp2_approx(ml.x - (M == -INFINITY ? 0.f : M));
        float den = e * ml.y;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float o = __shfl_down_sync(0xffffffffu, den, off);
            const int32_t f = __shfl_down_sync(0xffffffffu, my_first, off);
            if (lane + off < 32 && f == my_first) den += o;
        }
        den = __shfl_sync(0xffffffffu, den, my_first < 0 ? lane : my_first);
        if (piece) {
            weight[lane * hs + g] = den == 0.f ? 0.f : e / den;
            run_ml[lane * hs + g] = make_float2(M, den);
        }
    }
    __syncthreads();
    // the warps share the runs, and several warps share a run where there are few
    const int32_t runs = __popc(starts);
    for (int32_t run = runs > 0 ? warp % runs : 0; run < runs; run += NW) {
        uint32_t rest = starts;
        for (int32_t k = 0; k < run; ++k) rest &= rest - 1u;
        const int32_t i0 = __ffs(rest) - 1;
        rest &= rest - 1u;
        const uint32_t pieces = held & ~((1u << i0) - 1u) & (rest ? (1u << (__ffs(rest) - 1)) - 1u : 0xffffffffu);
        const int32_t shares = runs < NW ? (NW - 1 - run) / runs + 1 : 1, mine = runs < NW ? warp / runs : 0;
        const Piece pc = meta[i0];
        const int32_t seg_a = prefix[pc.s] + pc.h * (pc.np + kSegmentUnits);
        const bool complete = seg_a >= u0 && seg_a + pc.np <= u1;
        const int32_t hk = pc.h / NHC, g0 = (pc.h - hk * NHC) * kMaxHeads, heads = min(G - g0, kMaxHeads);
        const int32_t cslot = seg_a <= u0 ? 0 : 1;
        for (int32_t i = mine * 32 + lane; i < heads * V4; i += shares * 32) {
            const int32_t g = i / V4, d = (i - g * V4) * 4;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t left = pieces; left != 0u; left &= left - 1u) {
                const int32_t k = __ffs(left) - 1;
                const float* p = (k & 1) ? reinterpret_cast<const float*>(smem + L.ring + static_cast<uint32_t>(k >> 1) * L.ring_bytes)
                                         : piece0 + static_cast<uint32_t>(k >> 1) * hs * D;
                const float4 v = *reinterpret_cast<const float4*>(p + g * D + d);
                const float w = weight[k * hs + g];
                r.x = fmaf(w, v.x, r.x);
                r.y = fmaf(w, v.y, r.y);
                r.z = fmaf(w, v.z, r.z);
                r.w = fmaf(w, v.w, r.w);
            }
            if (complete) {
                store4(out + (static_cast<int64_t>(pc.s) * Hq + hk * G + g0 + g) * D + d, r.x * a.v_scale, r.y * a.v_scale,
                       r.z * a.v_scale, r.w * a.v_scale);
            } else {
                const int64_t pg = (static_cast<int64_t>(blockIdx.x) * 2 + cslot) * hs + g;
                *reinterpret_cast<float4*>(a.piece_o + pg * D + d) = r;
                if (d == 0) a.piece_ml[pg] = run_ml[i0 * hs + g];
            }
        }
        if (!complete && mine == 0 && lane == 0) cross[cslot] = i0;
    }
    __syncthreads();
    // ---- segments cut between CTAs: count this CTA's pieces; the last to count joins ------------
    if (tid < 2 && cross[tid] >= 0) {
        const Piece pc = meta[cross[tid]];
        const int32_t seg_a = prefix[pc.s] + pc.h * (pc.np + kSegmentUnits);
        const int32_t expected = (seg_a + pc.np - 1) / chunk - seg_a / chunk + 1;
        int32_t old;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(a.counter + pc.seg) : "memory");
        cross[2 + tid] = old == expected - 1 ? expected : 0;
        if (old == expected - 1) a.counter[pc.seg] = 0;
    }
    __syncthreads();
    // The join: a thread adds up a share of the pieces for 4 elements of a head, eight pieces' loads in
    // flight, and the shares are joined in order. The scratch is the ring, which nothing uses any more.
    float4* share_o = reinterpret_cast<float4*>(smem + L.ring);               // [NTH]
    float2* share_ml = reinterpret_cast<float2*>(smem + L.ring + 16u * NTH);  // [NTH]
    for (int32_t x = 0; x < 2; ++x) {
        const int32_t n_pieces = cross[2 + x];
        if (n_pieces == 0) continue;  // uniform over the CTA
        const Piece pc = meta[cross[x]];
        const int32_t seg_a = prefix[pc.s] + pc.h * (pc.np + kSegmentUnits), c_first = seg_a / chunk;
        const int32_t first_slot = seg_a == c_first * chunk ? 0 : 1;
        const int32_t hk = pc.h / NHC, g0 = (pc.h - hk * NHC) * kMaxHeads, heads = min(G - g0, kMaxHeads);
        const int32_t cols = heads * V4, shares = max(1, min(NTH / cols, n_pieces));
        auto add = [](float& M, float& den, float4& r, const float2 ml, const float4 v, float l) {
            // one piece (or share) more: its weight is l 2^(m - M), its sum ml.y 2^(m - M)
            const float Mn = fmaxf(M, ml.x), ref = Mn == -INFINITY ? 0.f : Mn;
            const float f = exp2_approx(M - ref), e = exp2_approx(ml.x - ref), w = e * l;
            M = Mn;
            den = fmaf(den, f, e * ml.y);
            r = make_float4(fmaf(w, v.x, r.x * f), fmaf(w, v.y, r.y * f), fmaf(w, v.z, r.z * f), fmaf(w, v.w, r.w * f));
        };
        auto put = [&](int32_t g, int32_t d, float den, const float4 r) {
            const float inv = den == 0.f ? 0.f : a.v_scale / den;
            store4(out + (static_cast<int64_t>(pc.s) * Hq + hk * G + g0 + g) * D + d, r.x * inv, r.y * inv, r.z * inv, r.w * inv);
        };
        for (int32_t i = tid; i < cols * shares; i += NTH) {  // one round unless a head chunk has more columns
            const int32_t sh = i / cols, col = i - sh * cols, g = col / V4, d = (col - g * V4) * 4;
            float M = -INFINITY, den = 0.f;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int32_t k0 = sh; k0 < n_pieces; k0 += 8 * shares) {
                float4 v[8];
                float2 ml[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int32_t k = k0 + j * shares;
                    const int64_t pg = (static_cast<int64_t>(c_first + k) * 2 + (k == 0 ? first_slot : 0)) * hs + g;
                    ml[j] = k < n_pieces ? __ldcg(a.piece_ml + pg) : make_float2(-INFINITY, 0.f);
                    v[j] = k < n_pieces ? __ldcg(reinterpret_cast<const float4*>(a.piece_o + pg * D + d))
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) add(M, den, r, ml[j], v[j], ml[j].y);  // pieces are normalised
            }
            if (shares == 1) {
                put(g, d, den, r);
            } else {
                share_o[i] = r;
                share_ml[i] = make_float2(M, den);
            }
        }
        __syncthreads();
        if (shares > 1 && tid < cols) {
            float M = -INFINITY, den = 0.f;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int32_t k = 0; k < shares; ++k) add(M, den, r, share_ml[k * cols + tid], share_o[k * cols + tid], 1.f);
            const int32_t g = tid / V4;
            put(g, (tid - g * V4) * 4, den, r);
        }
        __syncthreads();  // the scratch serves the other segment next
    }
}

template <typename T, int D, int NW, int NH>
cudaError_t launch_impl(const DecodeArgs& d, float v_scale, const DecodeScoredPlan& plan, cudaStream_t stream) {
    const int32_t G = d.num_q_heads / d.num_kv_heads, hs = G < kMaxHeads ? G : kMaxHeads;
    Params a{};
    a.k_cache = static_cast<const uint8_t*>(d.k_cache);
    a.v_cache = static_cast<const uint8_t*>(d.v_cache);
    a.max_blocks = d.max_blocks_per_seq;
    a.num_kv_heads = d.num_kv_heads;
    a.G = G;
    a.head_chunks = (G + kMaxHeads - 1) / kMaxHeads;
    a.num_blocks = d.num_blocks;
    a.sub_log2 = block_size_log2(d.block_size) - 4;
    a.cap_tokens = min(table_tokens(a.max_blocks, a.sub_log2), d.max_seq_len);
    a.c1 = d.scale * kLog2e;
    a.v_scale = v_scale;
    char* ws = static_cast<char*>(d.workspace);
    a.counter = reinterpret_cast<int32_t*>(ws);
    a.piece_o = reinterpret_cast<float*>(ws + kScoredCounterBytes);
    a.piece_ml = reinterpret_cast<float2*>(a.piece_o + static_cast<size_t>(plan.num_ctas) * 2 * hs * D);
    a.err = d.err;
    const WaitDrill drill = wait_drill();
    a.wait_limit_ns = drill.limit_ns;
    a.drill = drill.kind == kDrillDecodeStage ? 1 : 0;
    // Programmatic launch: the grid may be set up while the kernel before it drains.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.num_ctas);
    cfg.blockDim = dim3(NW * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    for (int32_t s0 = 0; s0 < d.num_seqs; s0 += plan.batch) {
        const int32_t S = d.num_seqs - s0 < plan.batch ? d.num_seqs - s0 : plan.batch;
        a.S = S;
        a.out = static_cast<T*>(d.out) + static_cast<int64_t>(s0) * d.num_q_heads * D;
        a.q = static_cast<const T*>(d.q) + static_cast<int64_t>(s0) * d.num_q_heads * D;
        a.block_table = d.block_table + static_cast<int64_t>(s0) * d.max_blocks_per_seq;
        a.seq_lens = d.seq_lens + s0;
        const Layout l = layout(NW, hs, D, S);
        cudaError_t e = allow_smem<decode_fp4_kernel<T, D, NW, NH>>(static_cast<int>(l.total));
        if (e != cudaSuccess) return e;
        cfg.dynamicSmemBytes = l.total;
        e = cudaLaunchKernelEx(&cfg, decode_fp4_kernel<T, D, NW, NH>, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Warps of a CTA, in fours for the four schedulers. Up to 8 heads, D = 128: 75 us with 12 (64 sequences of 500 to 16384 keys),
// 8: 101, 10: 86, 14: 84, 16 (spilled): 77; D = 64: 23.7 with 16 (96 of 16 to 2048), 12: 24.8. Twice the accumulators (more
// than 8 heads), or twice the queries (fp32, D = 128), leave registers for 8. fp32 spills 4 to 20 bytes, and 412 with more than 8
// heads of 128, both at once: 64 sequences of 2000 to 8000 keys, 64 q / 4 kv heads, 95 us (bf16 64; of 64 54 and 43).
constexpr int warps_of(int NH, int D, bool two_pieces) { return NH == 2 ? 8 : D == 64 ? 16 : two_pieces ? 8 : 12; }

template <typename T, int D>
cudaError_t pick(const DecodeArgs& a, float v_scale, const DecodeScoredPlan& plan, cudaStream_t stream) {
    constexpr bool two = Fp16Form<T>::kTwo;
    if (a.num_q_heads / a.num_kv_heads > 8) return launch_impl<T, D, warps_of(2, D, two), 2>(a, v_scale, plan, stream);
    return launch_impl<T, D, warps_of(1, D, two), 1>(a, v_scale, plan, stream);
}

}  // namespace

bool plan_decode_fp4(int32_t S, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_seq_len, pa_dtype dtype,
                     const DeviceInfo& dev, DecodeScoredPlan* plan) {
    const int32_t G = Hq / Hkv, hs = G < kMaxHeads ? G : kMaxHeads;
    const int64_t nh = static_cast<int64_t>(Hkv) * ((G + kMaxHeads - 1) / kMaxHeads);
    // sequences of one launch: their segments have counters, and units are counted in 32 bits
    int64_t batch = kScoredSegments / nh;
    const int64_t by_units = 0x70000000LL / (nh * (max_seq_len / kPageTokens + 1 + kSegmentUnits));  // (room for a slice past the end)
    if (by_units < batch) batch = by_units;
    if (batch > kMaxSeqs) batch = kMaxSeqs;
    if (batch < 1 || S < 1) return false;
    plan->batch = static_cast<int32_t>(batch < S ? batch : S);
    plan->num_ctas = dev.num_sms;
    plan->warps = warps_of(G > 8 ? 2 : 1, D, dtype == PA_F32);
    if (layout(plan->warps, hs, D, plan->batch).total + 64 > static_cast<uint32_t>(dev.max_smem_optin)) return false;
    plan->stages = 1;
    plan->workspace_bytes = kScoredCounterBytes + static_cast<size_t>(plan->num_ctas) * 2 * hs * (D * 4 + 8);
    return true;
}

cudaError_t launch_decode_fp4(const DecodeArgs& a, float v_scale, const DecodeScoredPlan& plan, cudaStream_t stream) {
    if (a.dtype == PA_F32)
        return a.head_dim == 128 ? pick<float, 128>(a, v_scale, plan, stream) : pick<float, 64>(a, v_scale, plan, stream);
    return a.head_dim == 128 ? pick<__nv_bfloat16, 128>(a, v_scale, plan, stream)
                             : pick<__nv_bfloat16, 64>(a, v_scale, plan, stream);
}

}  // namespace pa
