// Scored decode for bf16: one query row per sequence over the pages it sees, on mma.sync with TMA
// page staging. Memory bound: every visible page (16 tokens of K and of V of one kv head) is read
// once for all the q heads that share the kv head.
//
// Work list. A unit is one visible page of one segment; a segment is (sequence, kv head, chunk of up
// to 16 of the kv head's q heads). A sequence's pages are those its spans touch (scored.cuh), so a
// window or a document start shortens the list and balances with everything else. Every CTA builds
// the list's prefix sums from seq_lens (and key_start, prefix_len), takes an equal contiguous slice
// of it, and gives each of its warps an equal contiguous part.
//
// Streaming. Each warp owns a ring of stages; lane 0 copies a page's K and V (128-byte swizzle) by
// TMA, and with the first page of a segment its query rows; block ids are fetched 32 pages ahead.
// The arithmetic runs transposed: S^T = K Q^T puts the page's 16 keys in the 16 rows of
// m16n8k16 and 8 q heads in its columns, then O^T += V^T P^T with P^T brought into place by a
// register transpose; the softmax runs online in the log2 domain. Scores are transformed between
// the two (a tanh, by scored.cuh, a distance bias, masks); V rows of keys the row
// does not see are zeroed in shared memory.
//
// Joins, all by M = max m_i, w_i = l_i 2^(m_i - M), out = sum w_i o_i / sum w_i in a fixed order:
// a segment inside one warp's part goes straight to the output; pieces cut between the warps of a
// CTA meet in shared memory after one barrier, joined by all its threads; segments cut between CTAs
// leave one piece per CTA in the workspace, and the CTA that counts the last one joins them and
// puts the counter back to zero.
//
// Bound: HBM. 8 sequences of 20000 to 32768 keys, 64 q / 8 kv heads of 128, cap 30: 131 us, 6.5 TB/s, 96 % of
// the measured copy rate; 64 sequences of 500 to 16384 keys in a window of 4096: 110 us (94 %). Small batches
// are a chain of latencies (lengths, list, first pages, joins): 4 sequences of up to 700 keys 9.7 us in a graph.
#include <cuda.h>
#include <math.h>

#include "pa_internal.h"
#include "scored.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxSeqs = 1024;  // sequences of one launch: their spans live in shared memory
constexpr int kMaxHeads = 16;   // q heads of one segment
// Units of a CTA's slice, at least. Measured, 4 sequences of up to 700 keys, 8 kv heads of 128: 9.7 us with 4 or 2,
// 10.6 with 8, 14.3 with 32; 2 sequences of 1000 keys, one kv head: 9.8 with 4 or 8, 11.3 with 2, 14.2 with 1.
constexpr int kMinSlice = 4;
// One kv head of 128: 500 pages take 12.7, 14.2, 16.2, 20.3 us in 24, 48, 96, 125 pieces, 1250 pages 17.7, 16.7,
// 18.8, 22.2 us in 24, 48, 96, 152, 6250 pages 47.5, 31.9, 27.1, 27.4 us: best near sqrt(1.5 n) pieces.
constexpr float kJoinWeight = 1.f / 1.5f;
constexpr int kSegmentUnits = 1;  // a segment's start and end weigh as much as this many pages (96 sequences of 16
                                  // to 2048 keys, 16 heads of 64: 39.9 us, 52.3 when they weighed nothing)

// Pages of one step of a warp: 8 KB of K and V, so that what a step costs besides its pages
// (waits, reductions, the list) weighs alike at both head dims.
__host__ __device__ constexpr int step_pages(int D) { return 128 / D; }

__host__ __device__ inline uint32_t up(uint32_t x, uint32_t a) { return (x + a - 1) / a * a; }

struct Layout {
    uint32_t stage, ring, piece0, piece_ml, weight, meta, bars, flags, prefix, spans, total;
};
// NW warps, nst stages, hs q heads per segment, S sequences.
__host__ __device__ inline Layout layout(int NW, int nst, int hs, int D, int S) {
    Layout l;
    uint32_t o = 0;
    l.stage = up(2u * kPageTokens * D * 2u * step_pages(D) + static_cast<uint32_t>(hs) * D * 2u, 1024u);  // pages, query rows
    l.ring = o;      o += static_cast<uint32_t>(NW) * nst * l.stage;
    l.piece0 = o;    o += static_cast<uint32_t>(NW) * hs * D * 4u;       // each warp's first piece
    l.piece_ml = o;  o += static_cast<uint32_t>(NW) * 2u * hs * 8u;      // (max, sum) of both pieces
    l.weight = o;    o += static_cast<uint32_t>(NW) * 2u * hs * 12u;     // the pieces' weights, and (max, sum) of their run
    l.meta = up(o, 16u);  o = l.meta + static_cast<uint32_t>(NW) * 2u * 16u;  // segment of each piece
    l.bars = up(o, 16u);  o = l.bars + static_cast<uint32_t>(NW) * nst * 8u;
    l.flags = o;     o += 32u;
    l.prefix = up(o, 16u);  o = l.prefix + up((S + 1) * 4u, 16u);
    l.spans = o;     o += static_cast<uint32_t>(S) * 16u;
    l.total = o + 1024u;
    return l;
}

struct Params {
    __nv_bfloat16* out;
    const __nv_bfloat16* q;
    const int32_t* block_table;
    const int32_t* seq_lens;
    int32_t max_blocks, S, num_kv_heads, G, head_chunks, num_blocks, sub_log2, cap_tokens, nst;
    float c1;      // scale log2 e
    float two_k;   // 2 log2 e scale / cap
    float cap_l2;  // cap log2 e; 0: not capped
    ScoreArgs score;
    int32_t* counter;  // [kScoredSegments] CTA pieces finished per segment; zero between calls
    float* piece_o;    // [C][2][hs][D]
    float2* piece_ml;  // [C][2][hs]
    uint32_t* err;
};

__device__ __forceinline__ void bulk_copy_g2s(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(smem_dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

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
    int32_t s, h, j, np;
    KeySpans sp;
    PageList pl;
    __device__ __forceinline__ void load(const int4* spans) {
        const int4 v = spans[s];
        sp = KeySpans{v.x, v.y, v.z, v.w};
        pl = page_list(sp);
        np = pl.n;
    }
    __device__ __forceinline__ void at(const int32_t* prefix, const int4* spans, int32_t S, int32_t u) {
        s = find_seq(prefix, S, u);
        load(spans);
        const int32_t r = u - prefix[s], units = np + kSegmentUnits;
        h = r / units;
        j = r - h * units;
    }
    __device__ __forceinline__ void advance(int32_t pages, const int32_t* prefix, const int4* spans, int32_t S,
                                            int32_t nh) {
        j += pages;
        if (j < np + kSegmentUnits) return;
        j = 0;
        if (++h < nh) return;
        h = 0;
        do { ++s; } while (s < S && prefix[s + 1] == prefix[s]);
        if (s < S) load(spans);
    }
};

// A segment's piece: its segment number (-1: none), sequence, segment within the sequence, pages.
struct Piece {
    int32_t seg, s, h, np;
};

// NH: groups of 8 q heads of a segment (up to 8 NH heads).
template <int D, int NW, int NH>
__global__ void __launch_bounds__(NW * 32, 1)
    decode_scored_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ Params a) {
    constexpr uint32_t kPage = kPageTokens * D * 2;
    constexpr uint32_t kHalves = D / 64;
    constexpr int KS = D / 16, NMT = D / 16, SP = step_pages(D);
    constexpr int NTH = NW * 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int32_t S = a.S, G = a.G, nst = a.nst, NHC = a.head_chunks, Hq = G * a.num_kv_heads;
    const int32_t hs = min(G, kMaxHeads), nh = a.num_kv_heads * NHC;  // heads and segments per sequence
    const Layout L = layout(NW, nst, hs, D, S);
    float* piece0 = reinterpret_cast<float*>(smem + L.piece0);
    float2* piece_ml = reinterpret_cast<float2*>(smem + L.piece_ml);
    Piece* meta = reinterpret_cast<Piece*>(smem + L.meta);  // [2 NW]
    uint64_t* bars_all = reinterpret_cast<uint64_t*>(smem + L.bars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.flags);
    int32_t* cross = reinterpret_cast<int32_t*>(smem + L.flags + 8);  // [2] pieces of segments cut by the CTA's slice, [2] to join
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + L.prefix);
    int4* spans = reinterpret_cast<int4*>(smem + L.spans);
    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
        *abort_flag = 0;
        cross[0] = cross[1] = -1;
        cross[2] = cross[3] = 0;
    }
    if (lane == 0) {
        meta[warp * 2].seg = meta[warp * 2 + 1].seg = -1;
        for (int i = 0; i < nst; ++i) mbar_init(&bars_all[warp * nst + i], 1);
        fence_mbarrier_init();
    }
    // A programmatic launch: everything above ran beside the tail of the kernel before this one;
    // every input, output and the workspace are touched after this wait.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the work list: spans and units of each sequence, block-wide exclusive scan ------------
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
            const KeySpans sp = key_spans(len, len - 1, a.score.key_start ? __ldg(a.score.key_start + s) : 0,
                                          a.score.prefix_len ? __ldg(a.score.prefix_len + s) : 0, a.score.window,
                                          false);  // (the last row sees the whole prefix either way)
            spans[s] = make_int4(sp.a0, sp.a1, sp.b0, sp.b1);
            const int32_t pages = page_list(sp).n, units = pages > 0 ? (pages + kSegmentUnits) * nh : 0;
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
        uint32_t* z = reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(s) * Hq * D);
        for (int32_t i = tid; i < Hq * D / 2; i += NTH) z[i] = 0u;
    }
    const int64_t first = static_cast<int64_t>(blockIdx.x) * chunk;
    if (first >= U) return;  // uniform over the CTA
    const int32_t u0 = static_cast<int32_t>(first), u1 = min(U, u0 + chunk);
    const int32_t per_warp = (u1 - u0 + NW - 1) / NW;
    const int32_t a_w = u0 + warp * per_warp, n = max(0, min(u1 - a_w, per_warp));
    uint8_t* ring = smem + L.ring + static_cast<uint32_t>(warp) * nst * L.stage;
    const uint32_t ring_u32 = smem_u32(ring);
    uint64_t* bars = bars_all + warp * nst;
    const int32_t gid = lane >> 2, tig = lane & 3;

    if (n > 0) {
        int32_t t_i = 0, k_i = 0;  // pages and steps issued
        // Pool row of unit a_w + 32 k + lane.
        auto lane_row = [&](int32_t k) -> int32_t {
            if (32 * k + lane >= n) return 0;
            Cursor c;
            c.at(prefix, spans, S, a_w + 32 * k + lane);
            if (c.j >= c.np) return 0;
            const int32_t page = c.pl.page(c.j);
            int32_t phys = __ldg(a.block_table + static_cast<int64_t>(c.s) * a.max_blocks + (page >> a.sub_log2));
            if (phys < 0 || phys >= a.num_blocks) {
                raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
                phys = 0;
            }
            return ((((phys * a.num_kv_heads + c.h / NHC) << a.sub_log2) + (page & ((1 << a.sub_log2) - 1))) * kPageTokens);
        };
        int32_t kc = 0, id_cur = lane_row(0), id_nxt = 0;
        // pages are read once per call: let them leave L2 first
        const uint64_t kv_policy = l2_policy_evict_first();
        Cursor wi;
        wi.at(prefix, spans, S, a_w);
        // Step k_i (pages t_i .. of one segment, up to SP) into stage k_i % nst. Lane 2 i + kv copies the
        // K (kv = 0) or V of page i, lane 31 the query rows of a segment that begins here.
        bool q_due = true;  // the segment's query rows have not been copied yet
        auto next_block_ids = [&]() {
            if ((t_i >> 5) > kc) {  // the next 32 block ids, fetched while these are used
                ++kc;
                id_cur = id_nxt;
                id_nxt = 32 * (kc + 1) < n ? lane_row(kc + 1) : 0;
            }
        };
        auto skip = [&]() {  // to the next page of the part
            while (t_i < n && wi.j >= wi.np) {
                const int32_t none = min(wi.np + kSegmentUnits - wi.j, n - t_i);
                wi.advance(none, prefix, spans, S, nh);
                t_i += none;
                q_due = true;
                next_block_ids();
            }
        };
        auto issue = [&]() {
            const int32_t cnt = min(min(SP, wi.np - wi.j), n - t_i), st = k_i % nst;
            uint8_t* stage = ring + static_cast<uint32_t>(st) * L.stage;
            const bool seg_first = q_due;
            const int32_t hk = wi.h / NHC, g0 = (wi.h - hk * NHC) * kMaxHeads;
            const uint32_t qbytes = static_cast<uint32_t>(min(G - g0, kMaxHeads)) * D * 2u;
            const int32_t pg = t_i + (lane >> 1);
            const int32_t r0 = __shfl_sync(0xffffffffu, id_cur, pg & 31), r1 = __shfl_sync(0xffffffffu, id_nxt, pg & 31);
            const bool go = !*abort_flag;
            if (lane == 0 && go)
                mbar_arrive_expect_tx(&bars[st], static_cast<uint32_t>(cnt) * 2u * kPage + (seg_first ? qbytes : 0u));
            __syncwarp();
            if (lane < 2 * cnt && go) {
                const void* tm = (lane & 1) ? static_cast<const void*>(&tm_v) : static_cast<const void*>(&tm_k);
                uint8_t* dst = stage + static_cast<uint32_t>(lane) * kPage;
                const int32_t row = (pg >> 5) == kc ? r0 : r1;
                if constexpr (kHalves == 2) tma_load_3d_hint(dst, tm, 0, row, 0, &bars[st], kv_policy);  // both 64-column halves
                else tma_load_2d_hint(dst, tm, 0, row, &bars[st], kv_policy);
            }
            if (lane == 31 && seg_first && go)
                bulk_copy_g2s(stage + 2u * kPage * SP, a.q + (static_cast<int64_t>(wi.s) * Hq + hk * G + g0) * D, qbytes,
                              &bars[st]);
            wi.advance(cnt, prefix, spans, S, nh);
            t_i += cnt;
            ++k_i;
            q_due = false;
            next_block_ids();
            skip();
        };
        if (n > 32) id_nxt = lane_row(1);
        skip();
        for (int32_t i = 0; i < nst && t_i < n; ++i) issue();

        Cursor wc;
        wc.at(prefix, spans, S, a_w);
        // Fragment ownership (gid = lane / 4, tig = lane % 4):
        //   qb[f][ks]   Q^T as B: head 8 f + gid, dims 16 ks + 2 tig (+1) and + 8
        //   sc[i][f][e] S^T of page i: key gid + 8 (e / 2), head 8 f + 2 tig + e % 2
        //   acc[f][mt]  O^T: head_dim 16 mt + gid + 8 (e / 2), head 8 f + 2 tig + e % 2
        uint32_t qb[NH][KS][2];
        float acc[NH][NMT][4], mh[NH][2], lh[NH][2], slope[NH][2];
        int32_t ng = 0, head0 = 0;
        bool cut_left = false;
        int32_t k = 0;  // steps consumed
        bool first_page = true;  // of a segment in this part
        for (int32_t t = 0; t < n;) {
            if (wc.j >= wc.np) {  // units without a page
                const int32_t none = min(wc.np + kSegmentUnits - wc.j, n - t);
                wc.advance(none, prefix, spans, S, nh);
                t += none;
                first_page = true;
                continue;
            }
            const int32_t st = k % nst, cnt = min(min(SP, wc.np - wc.j), n - t);
            const bool landed = mbar_wait_bounded(&bars[st], static_cast<uint32_t>(k / nst) & 1u, abort_flag);
            if (!__all_sync(0xffffffffu, landed)) {
                if (lane == 0) {
                    if (!*abort_flag) raise_error(a.err, PA_DEVERR_WAIT_TIMEOUT);
                    *abort_flag = 1;
                }
                __syncwarp();
                break;
            }
            ++k;
            uint8_t* stage = ring + static_cast<uint32_t>(st) * L.stage;
            const uint32_t stage_u32 = ring_u32 + static_cast<uint32_t>(st) * L.stage;
            if (first_page) {  // a new segment: its query rows came with this step
                first_page = false;
                const int32_t hk = wc.h / NHC, g0 = (wc.h - hk * NHC) * kMaxHeads;
                ng = min(G - g0, kMaxHeads);
                head0 = hk * G + g0;
                const __nv_bfloat16* qs = reinterpret_cast<const __nv_bfloat16*>(stage + 2u * kPage * SP);
#pragma unroll
                for (int f = 0; f < NH; ++f) {
                    const bool valid = f * 8 + gid < ng;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const __nv_bfloat16* p = qs + (f * 8 + gid) * D + ks * 16 + tig * 2;
                        qb[f][ks][0] = valid ? *reinterpret_cast<const uint32_t*>(p) : 0u;
                        qb[f][ks][1] = valid ? *reinterpret_cast<const uint32_t*>(p + 8) : 0u;
                    }
#pragma unroll
                    for (int mt = 0; mt < NMT; ++mt) acc[f][mt][0] = acc[f][mt][1] = acc[f][mt][2] = acc[f][mt][3] = 0.f;
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        mh[f][hh] = -INFINITY;
                        lh[f][hh] = 0.f;
                        const int32_t head = f * 8 + tig * 2 + hh;
                        slope[f][hh] = a.score.slopes && head < ng ? __ldg(a.score.slopes + head0 + head) * kLog2e : 0.f;
                    }
                }
                cut_left = wc.j > 0;
            }
            // scores of the step's pages
            const uint32_t mat = lane >> 3, r8 = lane & 7;
            const int32_t pos = wc.sp.b1 - 1;
            float sc[SP][NH][4], mx[NH][2];
#pragma unroll
            for (int f = 0; f < NH; ++f) mx[f][0] = mx[f][1] = -INFINITY;
            bool zeroed = false;
#pragma unroll
            for (int i = 0; i < SP; ++i) {
                const uint32_t k_u32 = stage_u32 + 2u * i * kPage;
                const bool here = i < cnt;  // a missing page: its keys are masked, its K is not meant
                const int32_t key0 = wc.pl.page(wc.j + (here ? i : 0)) * kPageTokens;
                const bool whole = here && ((key0 >= wc.sp.a0 && key0 + kPageTokens <= wc.sp.a1) ||
                                            (key0 >= wc.sp.b0 && key0 + kPageTokens <= wc.sp.b1));
                if (here && !whole) {  // zero the V rows of keys the row does not see: a weight of 0 adds nothing
                    uint8_t* v = stage + (2u * i + 1u) * kPage;
                    for (int32_t c = lane; c < kPageTokens * 8 * static_cast<int32_t>(kHalves); c += 32) {
                        const int32_t hf = c / (kPageTokens * 8), rem = c % (kPageTokens * 8), rr = rem >> 3;
                        if (!wc.sp.sees(key0 + rr))
                            *reinterpret_cast<int4*>(v + hf * 2048u + rr * 128u + (rem & 7) * 16u) = make_int4(0, 0, 0, 0);
                    }
                    zeroed = true;
                    __syncwarp();
                }
                // S^T = K Q^T
#pragma unroll
                for (int f = 0; f < NH; ++f) sc[i][f][0] = sc[i][f][1] = sc[i][f][2] = sc[i][f][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint32_t key = r8 + 8u * (mat & 1u), c16 = ks * 2 + (mat >> 1);
                    uint32_t fa[4];
                    ldsm_x4(k_u32 + (c16 >> 3) * 2048u + sw128_offset(key, c16 & 7u), fa[0], fa[1], fa[2], fa[3]);
#pragma unroll
                    for (int f = 0; f < NH; ++f) mma_16816(sc[i][f], fa, qb[f][ks][0], qb[f][ks][1]);
                }
                // scores in the log2 domain
                const bool see0 = here && (whole || wc.sp.sees(key0 + gid)), see1 = here && (whole || wc.sp.sees(key0 + gid + 8));
                const float away0 = fabsf(static_cast<float>(pos - key0 - gid)), away1 = fabsf(static_cast<float>(pos - key0 - gid - 8));
                if (a.cap_l2 > 0.f) {  // the polynomial for all, the identity where a score is beyond it
                    float x[NH][4], big = 0.f;
#pragma unroll
                    for (int f = 0; f < NH; ++f)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float y = sc[i][f][e] * a.two_k;
                            x[f][e] = capped_near(sc[i][f][e], y * y, a.c1);
                            big = fmaxf(big, y * y);
                        }
                    if (__any_sync(0xffffffffu, big > kTanhY2)) {
#pragma unroll
                        for (int f = 0; f < NH; ++f)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float y = sc[i][f][e] * a.two_k;
                                if (y * y > kTanhY2) x[f][e] = capped_far(y, a.cap_l2);
                            }
                    }
#pragma unroll
                    for (int f = 0; f < NH; ++f)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i][f][e] = x[f][e];
                } else {
#pragma unroll
                    for (int f = 0; f < NH; ++f)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[i][f][e] *= a.c1;
                }
#pragma unroll
                for (int f = 0; f < NH; ++f) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[i][f][e] = (e < 2 ? see0 : see1) ? fmaf(-slope[f][e & 1], e < 2 ? away0 : away1, sc[i][f][e]) : -INFINITY;
                    mx[f][0] = fmaxf(mx[f][0], fmaxf(sc[i][f][0], sc[i][f][2]));
                    mx[f][1] = fmaxf(mx[f][1], fmaxf(sc[i][f][1], sc[i][f][3]));
                }
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
#pragma unroll
                for (int f = 0; f < NH; ++f) {
                    mx[f][0] = fmaxf(mx[f][0], __shfl_xor_sync(0xffffffffu, mx[f][0], off));
                    mx[f][1] = fmaxf(mx[f][1], __shfl_xor_sync(0xffffffffu, mx[f][1], off));
                }
            uint32_t pb[SP][NH][2];
#pragma unroll
            for (int f = 0; f < NH; ++f) {
                float cc[2], ref[2];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float mn = fmaxf(mh[f][hh], mx[f][hh]);
                    ref[hh] = mn == -INFINITY ? 0.f : mn;  // nothing above -inf yet: weights are 0, not NaN
                    cc[hh] = exp2_approx(mh[f][hh] - ref[hh]);
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
#pragma unroll
                for (int i = 0; i < SP; ++i) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = exp2_approx(sc[i][f][e] - ref[e & 1]);
                    lh[f][0] += p[0] + p[2];
                    lh[f][1] += p[1] + p[3];
                    pb[i][f][0] = movmatrix_trans(pack_bf16x2(p[0], p[1]));
                    pb[i][f][1] = movmatrix_trans(pack_bf16x2(p[2], p[3]));
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int i = 0; i < SP; ++i) {
                if (i >= cnt) break;
                const uint32_t v_u32 = stage_u32 + (2u * i + 1u) * kPage;
#pragma unroll
                for (int mt = 0; mt < NMT; ++mt) {
                    const uint32_t key = r8 + 8u * (mat >> 1), c16 = mt * 2 + (mat & 1u);
                    uint32_t fa[4];
                    ldsm_x4_trans(v_u32 + (c16 >> 3) * 2048u + sw128_offset(key, c16 & 7u), fa[0], fa[1], fa[2], fa[3]);
#pragma unroll
                    for (int f = 0; f < NH; ++f) mma_16816(acc[f][mt], fa, pb[i][f][0], pb[i][f][1]);
                }
            }

            if (t + cnt == n || wc.j + cnt == wc.np) {  // the warp's last page of this segment
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
                __nv_bfloat16* o = a.out + (static_cast<int64_t>(wc.s) * Hq + head0) * D;
#pragma unroll
                for (int f = 0; f < NH; ++f)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int32_t head = f * 8 + tig * 2 + hh;
                        if (head >= ng) continue;
                        if (inside) {
                            const float inv = Lh[f][hh] == 0.f ? 0.f : 1.f / Lh[f][hh];
#pragma unroll
                            for (int mt = 0; mt < NMT; ++mt) {
                                o[head * D + gid + mt * 16] = __float2bfloat16_rn(Lh[f][hh] == 0.f ? 0.f : acc[f][mt][hh] * inv);
                                o[head * D + gid + mt * 16 + 8] =
                                    __float2bfloat16_rn(Lh[f][hh] == 0.f ? 0.f : acc[f][mt][2 + hh] * inv);
                            }
                        } else {
#pragma unroll
                            for (int mt = 0; mt < NMT; ++mt) {
                                pa_acc[head * D + gid + mt * 16] = acc[f][mt][hh];
                                pa_acc[head * D + gid + mt * 16 + 8] = acc[f][mt][2 + hh];
                            }
                            if (gid == 0) piece_ml[(warp * 2 + slot) * hs + head] = make_float2(mh[f][hh], Lh[f][hh]);
                        }
                    }
                if (!inside && lane == 0) meta[warp * 2 + slot] = Piece{wc.s * nh + wc.h, wc.s, wc.h, wc.np};
            }
            __syncwarp();
            if (zeroed) fence_proxy_async_shared();  // generic writes before the next copy into the stage
            if (t_i < n) issue();
            wc.advance(cnt, prefix, spans, S, nh);
            t += cnt;
        }
        // after an abort: copies already issued land before the CTA can exit
        if (k < k_i && lane == 0)
            for (; k < k_i; ++k) mbar_wait_timeout(&bars[k % nst], static_cast<uint32_t>(k / nst) & 1u);
    }
    __syncthreads();
    if (*abort_flag) return;

    // ---- pieces cut between this CTA's warps: runs of equal segments in list order -------------
    // First every (piece, head) weighs itself against its run: e_i / sum e_k l_k with e_i = 2^(m_i - M)
    // (pieces hold unnormalised outputs); then all threads add the pieces up.
    constexpr int V4 = D / 4;
    float* weight = reinterpret_cast<float*>(smem + L.weight);            // [2 NW][hs]
    float2* run_ml = reinterpret_cast<float2*>(weight + 2 * NW * hs);     // [2 NW][hs] the run's (M, sum), at each piece
    for (int32_t g = warp; g < hs; g += NW) {  // a warp per head, a lane per piece
        const int32_t seg = lane < 2 * NW ? meta[lane].seg : -1;
        const float2 ml = seg >= 0 ? piece_ml[lane * hs + g] : make_float2(-INFINITY, 0.f);
        float M = -INFINITY, den = 0.f;
#pragma unroll 4
        for (int k = 0; k < 2 * NW; ++k) {
            const int32_t sk = __shfl_sync(0xffffffffu, seg, k);
            const float mk = __shfl_sync(0xffffffffu, ml.x, k);
            if (sk == seg) M = fmaxf(M, mk);
        }
        const float e = exp2_approx(ml.x - (M == -INFINITY ? 0.f : M)), el = e * ml.y;
#pragma unroll 4
        for (int k = 0; k < 2 * NW; ++k) {
            const int32_t sk = __shfl_sync(0xffffffffu, seg, k);
            const float lk = __shfl_sync(0xffffffffu, el, k);
            if (sk == seg) den += lk;
        }
        if (seg >= 0) {
            weight[lane * hs + g] = den == 0.f ? 0.f : e / den;
            run_ml[lane * hs + g] = make_float2(M, den);
        }
    }
    __syncthreads();
    // Runs begin at the pieces whose predecessor belongs to another segment; the warps share the runs,
    // and several warps share a run where there are few.
    uint32_t starts;
    {
        const int32_t seg = lane < 2 * NW ? meta[lane].seg : -1;
        const uint32_t held = __ballot_sync(0xffffffffu, seg >= 0);
        const uint32_t before = held & ((1u << lane) - 1u);
        const int32_t prev = __shfl_sync(0xffffffffu, seg, before ? 31 - __clz(before) : lane);
        starts = __ballot_sync(0xffffffffu, seg >= 0 && (before == 0u || prev != seg));
    }
    const int32_t runs = __popc(starts);
    for (int32_t run = runs > 0 ? warp % runs : 0; run < runs; run += NW) {
        const int32_t i0 = __fns(starts, 0, run + 1), i1 = run + 1 < runs ? __fns(starts, 0, run + 2) : 2 * NW;
        const int32_t shares = runs < NW ? (NW - 1 - run) / runs + 1 : 1, mine = runs < NW ? warp / runs : 0;
        const Piece pc = meta[i0];
        const int32_t seg_a = prefix[pc.s] + pc.h * (pc.np + kSegmentUnits);
        const bool complete = seg_a >= u0 && seg_a + pc.np <= u1;
        const int32_t hk = pc.h / NHC, g0 = (pc.h - hk * NHC) * kMaxHeads, heads = min(G - g0, kMaxHeads);
        const int32_t cslot = seg_a <= u0 ? 0 : 1;
        for (int32_t i = mine * 32 + lane; i < heads * V4; i += shares * 32) {
            const int32_t g = i / V4, d = (i - g * V4) * 4;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int32_t k = i0; k < i1; ++k) {
                if (meta[k].seg < 0) continue;
                const float* p = (k & 1) ? reinterpret_cast<const float*>(smem + L.ring + static_cast<uint32_t>(k >> 1) * nst * L.stage)
                                         : piece0 + static_cast<uint32_t>(k >> 1) * hs * D;
                const float4 v = *reinterpret_cast<const float4*>(p + g * D + d);
                const float w = weight[k * hs + g];
                r.x = fmaf(w, v.x, r.x);
                r.y = fmaf(w, v.y, r.y);
                r.z = fmaf(w, v.z, r.z);
                r.w = fmaf(w, v.w, r.w);
            }
            if (complete) {
                *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(pc.s) * Hq + hk * G + g0 + g) * D + d) =
                    make_uint2(pack_bf16x2(r.x, r.y), pack_bf16x2(r.z, r.w));
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
            const float inv = den == 0.f ? 0.f : 1.f / den;
            *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(pc.s) * Hq + hk * G + g0 + g) * D + d) =
                make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv));
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

template <int D, int NW, int NH>
cudaError_t launch_impl(const DecodeArgs& d, const ScoreArgs& score, const DecodeScoredPlan& plan, cudaStream_t stream) {
    alignas(64) CUtensorMap tm_k, tm_v;
    const uint64_t rows = static_cast<uint64_t>(d.num_blocks) * d.num_kv_heads * d.block_size;
    cudaError_t e;
    if (D == 128) {  // (column within a half, pool row, half): a page lands as two swizzled halves
        e = encode_bf16_3d_sw128(&tm_k, d.k_cache, 64, rows, 2, D * 2, 128, 64, kPageTokens, 2);
        if (e != cudaSuccess) return e;
        e = encode_bf16_3d_sw128(&tm_v, d.v_cache, 64, rows, 2, D * 2, 128, 64, kPageTokens, 2);
    } else {
        e = encode_bf16_2d_sw128(&tm_k, d.k_cache, D, rows, 64, kPageTokens);
        if (e != cudaSuccess) return e;
        e = encode_bf16_2d_sw128(&tm_v, d.v_cache, D, rows, 64, kPageTokens);
    }
    if (e != cudaSuccess) return e;
    const int32_t G = d.num_q_heads / d.num_kv_heads, hs = G < kMaxHeads ? G : kMaxHeads;
    Params a{};
    a.max_blocks = d.max_blocks_per_seq;
    a.num_kv_heads = d.num_kv_heads;
    a.G = G;
    a.head_chunks = (G + kMaxHeads - 1) / kMaxHeads;
    a.num_blocks = d.num_blocks;
    a.sub_log2 = block_size_log2(d.block_size) - 4;
    a.cap_tokens = min(table_tokens(a.max_blocks, a.sub_log2), d.max_seq_len);
    a.nst = plan.stages;
    a.c1 = d.scale * kLog2e;
    if (score.cap > 0.f) {
        a.two_k = static_cast<float>(fmin(fmax(2 * 1.4426950408889634 * d.scale / score.cap, -3e38), 3e38));
        a.cap_l2 = fminf(score.cap * kLog2e, kLargestCapL2);
    }
    char* ws = static_cast<char*>(d.workspace);
    a.counter = reinterpret_cast<int32_t*>(ws);
    a.piece_o = reinterpret_cast<float*>(ws + kScoredCounterBytes);
    a.piece_ml = reinterpret_cast<float2*>(a.piece_o + static_cast<size_t>(plan.num_ctas) * 2 * hs * D);
    a.err = d.err;
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
        a.out = static_cast<__nv_bfloat16*>(d.out) + static_cast<int64_t>(s0) * d.num_q_heads * D;
        a.q = static_cast<const __nv_bfloat16*>(d.q) + static_cast<int64_t>(s0) * d.num_q_heads * D;
        a.block_table = d.block_table + static_cast<int64_t>(s0) * d.max_blocks_per_seq;
        a.seq_lens = d.seq_lens + s0;
        a.score = score;
        if (score.key_start) a.score.key_start = score.key_start + s0;
        if (score.prefix_len) a.score.prefix_len = score.prefix_len + s0;
        const Layout l = layout(NW, plan.stages, hs, D, S);
        e = allow_smem<decode_scored_kernel<D, NW, NH>>(static_cast<int>(l.total));
        if (e != cudaSuccess) return e;
        cfg.dynamicSmemBytes = l.total;
        e = cudaLaunchKernelEx(&cfg, decode_scored_kernel<D, NW, NH>, tm_k, tm_v, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int D>
cudaError_t pick(const DecodeArgs& a, const ScoreArgs& score, const DecodeScoredPlan& plan, cudaStream_t stream) {
    const bool wide = a.num_q_heads / a.num_kv_heads > 8;
    if constexpr (D == 64)
        if (plan.warps == 10) return launch_impl<D, 10, 1>(a, score, plan, stream);
    if (plan.warps == 8) return wide ? launch_impl<D, 8, 2>(a, score, plan, stream) : launch_impl<D, 8, 1>(a, score, plan, stream);
    return wide ? launch_impl<D, 4, 2>(a, score, plan, stream) : launch_impl<D, 4, 1>(a, score, plan, stream);
}

}  // namespace

bool plan_decode_scored(int32_t S, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_seq_len, const DeviceInfo& dev,
                        DecodeScoredPlan* plan) {
    const int32_t G = Hq / Hkv, hs = G < kMaxHeads ? G : kMaxHeads;
    const int64_t nh = static_cast<int64_t>(Hkv) * ((G + kMaxHeads - 1) / kMaxHeads);
    // sequences of one launch: their segments have counters, and units are counted in 32 bits
    int64_t batch = kScoredSegments / nh;
    const int64_t by_units = 0x70000000LL / (nh * (max_seq_len / kPageTokens + 2));  // (room for a slice past the end)
    if (by_units < batch) batch = by_units;
    if (batch > kMaxSeqs) batch = kMaxSeqs;
    if (batch < 1 || S < 1) return false;
    plan->batch = static_cast<int32_t>(batch < S ? batch : S);
    plan->num_ctas = dev.num_sms;
    // 8 warps with as many stages as fit, else 4 warps (16 q heads of 128: the pieces take the room). At head_dim 64,
    // whose pages are half as long, 10 warps: 96 sequences of 16 to 2048 keys, 16 heads, 36.8 us (8 warps 40.0, 12 warps
    // 35.9); 300 of 100 keys 31.4 (34.6, 28.9); 96 of 1000 keys 70.2 (68.3, 72.0). At 128 10 warps lose: 64 sequences in a
    // window of 4096 119.7 us against 113.7.
    for (const int NW : {10, 8, 4})
        for (int nst = 4; nst >= 2; --nst) {
            if (NW == 10 && (D != 64 || G > 8)) continue;
            if (layout(NW, nst, hs, D, plan->batch).total + 64 > static_cast<uint32_t>(dev.max_smem_optin)) continue;
            plan->warps = NW;
            plan->stages = nst;
            plan->workspace_bytes = kScoredCounterBytes + static_cast<size_t>(plan->num_ctas) * 2 * hs * (D * 4 + 8);
            return true;
        }
    return false;
}

cudaError_t launch_decode_scored(const DecodeArgs& a, const ScoreArgs& score, const DecodeScoredPlan& plan,
                                 cudaStream_t stream) {
    return a.head_dim == 128 ? pick<128>(a, score, plan, stream) : pick<64>(a, score, plan, stream);
}

}  // namespace pa
