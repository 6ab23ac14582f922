// Scored attention on the CUDA cores: every type, head layout and score, decode and prefill.
//
// Grid: (query row, kv head x chunk of up to 4 q heads, partition of the row's visible pages). Four
// warps take the partition's 16-token pages in turn; a lane holds head_dim / 32 elements, dot
// products are reduced by shuffles, the softmax runs online per warp in the log2 domain, and the
// warps' (max, sum, output) meet in shared memory. Partitions of one row are merged by a second
// kernel with the same rule:
//   M = max_p m_p,  w_p = l_p 2^(m_p - M),  out = sum_p w_p o_p / sum_p w_p.
// The row's pages are those of its visible spans only, so a window or a document start costs no
// reads outside it. A page that a span cuts is read, and its invisible keys are skipped.
#include <math.h>

#include "pa_internal.h"
#include "scored.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHeads = 4;  // q heads per CTA
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t x) { return bf16_bits_to_float(x); }

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float x) {
    __nv_bfloat16 b = __float2bfloat16_rn(x);
    return *reinterpret_cast<uint16_t*>(&b);
}

struct SimtArgs {
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* query_start_loc;  // null: decode
    int32_t max_blocks, num_q_heads, num_kv_heads, num_blocks, sub_log2, cap_tokens, max_chunk;
    int32_t part_pages, num_parts, head_chunks;
    float scale;
    ScoreArgs score;
    float* ws_o;
    float* ws_ml;
    uint32_t* err;
};

// The query row of this CTA: its sequence, position and output row; false when it has none. A
// sequence whose length or chunk is out of range raises an error and has no rows (decode: clamps).
__device__ __forceinline__ bool locate(const SimtArgs& a, int32_t& s, int32_t& row, int32_t& len, int32_t& pos) {
    if (a.query_start_loc == nullptr) {
        s = row = blockIdx.x;
        len = __ldg(a.seq_lens + s);
        if (len < 0 || len > a.cap_tokens) {
            raise_error(a.err, PA_DEVERR_LEN_RANGE);
            len = len < 0 ? 0 : a.cap_tokens;
        }
        pos = len - 1;
        return true;
    }
    s = blockIdx.x / a.max_chunk;
    const int32_t r = blockIdx.x - s * a.max_chunk;
    const int32_t q0 = __ldg(a.query_start_loc + s), chunk = __ldg(a.query_start_loc + s + 1) - q0;
    len = __ldg(a.seq_lens + s);
    if (chunk < 0 || chunk > a.max_chunk || chunk > len || len > a.cap_tokens) {
        if (r == 0) raise_error(a.err, PA_DEVERR_LEN_RANGE);
        return false;
    }
    if (r >= chunk) return false;
    row = q0 + r;
    pos = len - chunk + r;
    return true;
}

__device__ __forceinline__ KeySpans row_spans(const SimtArgs& a, int32_t s, int32_t row, int32_t len, int32_t pos) {
    const int32_t start = a.score.key_start ? __ldg(a.score.key_start + row) : 0;
    const int32_t prefix = a.score.prefix_len ? __ldg(a.score.prefix_len + s) : 0;
    return key_spans(len, pos, start, prefix, a.score.window);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) scored_simt_kernel(T* __restrict__ out, const T* __restrict__ q,
                                                               const T* __restrict__ k_cache,
                                                               const T* __restrict__ v_cache,
                                                               const __grid_constant__ SimtArgs a) {
    constexpr int E = D / 32;
    int32_t s, row, len, pos;
    if (!locate(a, s, row, len, pos)) return;
    const int32_t hk = blockIdx.y / a.head_chunks, g0 = (blockIdx.y % a.head_chunks) * kHeads;
    const int32_t G = a.num_q_heads / a.num_kv_heads, ng = min(kHeads, G - g0);
    const int32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KeySpans sp = row_spans(a, s, row, len, pos);
    const PageList pl = page_list(sp);
    const int32_t parts = (pl.n + a.part_pages - 1) / a.part_pages;
    const int32_t p = blockIdx.z;
    if (p >= max(parts, 1)) return;

    float qv[kHeads][E], slope[kHeads];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
        const int32_t hq = hk * G + g0 + min(g, ng - 1);
        const T* qp = q + (static_cast<int64_t>(row) * a.num_q_heads + hq) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) qv[g][e] = widen<T>(qp[e]) * a.scale;
        slope[g] = a.score.slopes ? __ldg(a.score.slopes + hq) : 0.f;
    }
    float m[kHeads], l[kHeads], acc[kHeads][E];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[g][e] = 0.f;
    }
    const int32_t end = min(pl.n, (p + 1) * a.part_pages);
    for (int32_t i = p * a.part_pages + warp; i < end; i += kWarps) {
        const int32_t page = pl.page(i);
        const int32_t phys = __ldg(a.block_table + static_cast<int64_t>(s) * a.max_blocks + (page >> a.sub_log2));
        if (phys < 0 || phys >= a.num_blocks) {
            raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
            continue;
        }
        const int64_t base = ((((static_cast<int64_t>(phys) * a.num_kv_heads + hk) << a.sub_log2) +
                               (page & ((1 << a.sub_log2) - 1))) * kPageTokens) * D + lane * E;
        for (int32_t t = 0; t < kPageTokens; ++t) {
            const int32_t j = page * kPageTokens + t;
            if (!sp.sees(j)) continue;
            float kr[E], vr[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                kr[e] = widen<T>(k_cache[base + t * D + e]);
                vr[e] = widen<T>(v_cache[base + t * D + e]);
            }
            float z[kHeads];
#pragma unroll
            for (int g = 0; g < kHeads; ++g) {
                z[g] = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) z[g] = fmaf(qv[g][e], kr[e], z[g]);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                for (int g = 0; g < kHeads; ++g) z[g] += __shfl_xor_sync(0xffffffffu, z[g], off);
#pragma unroll
            for (int g = 0; g < kHeads; ++g) {
                if (a.score.cap > 0.f) z[g] = a.score.cap * tanhf(z[g] / a.score.cap);
                if (a.score.slopes) z[g] -= slope[g] * static_cast<float>(abs(pos - j));
                z[g] *= kLog2e;
                const float mn = fmaxf(m[g], z[g]);
                const float ref = mn == -INFINITY ? 0.f : mn;  // nothing finite yet: weights are 0, not NaN
                const float corr = exp2f(m[g] - ref), pj = exp2f(z[g] - ref);
                l[g] = l[g] * corr + pj;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[g][e] = fmaf(pj, vr[e], acc[g][e] * corr);
                m[g] = mn;
            }
        }
    }

    __shared__ float sm_acc[kWarps][kHeads][D];
    __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
#pragma unroll
        for (int e = 0; e < E; ++e) sm_acc[warp][g][lane * E + e] = acc[g][e];
        if (lane == 0) {
            sm_m[warp][g] = m[g];
            sm_l[warp][g] = l[g];
        }
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < ng * D; i += kThreads) {
        const int32_t g = i / D, d = i % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][g]);
        const float ref = M == -INFINITY ? 0.f : M;
        float num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(sm_m[w][g] - ref);  // a warp without keys: m = -inf, weight 0
            num = fmaf(sm_acc[w][g][d], f, num);
            den = fmaf(sm_l[w][g], f, den);
        }
        const float o = den == 0.f ? 0.f : num / den;
        const int64_t head = static_cast<int64_t>(row) * a.num_q_heads + hk * G + g0 + g;
        if (parts <= 1) {
            out[head * D + d] = narrow<T>(o);
        } else {
            const int64_t slot = head * a.num_parts + p;
            a.ws_o[slot * D + d] = o;
            if (d == 0) {
                a.ws_ml[2 * slot] = M;
                a.ws_ml[2 * slot + 1] = den;
            }
        }
    }
}

// Merges the partitions of decode rows that needed more than one (grid: sequence x q head).
template <typename T, int D>
__global__ void __launch_bounds__(D) scored_simt_merge_kernel(T* __restrict__ out, const __grid_constant__ SimtArgs a) {
    const int32_t s = blockIdx.x, hq = blockIdx.y, d = threadIdx.x;
    int32_t len = __ldg(a.seq_lens + s);
    len = len < 0 ? 0 : min(len, a.cap_tokens);
    const int32_t n = page_list(row_spans(a, s, s, len, len - 1)).n;
    const int32_t parts = (n + a.part_pages - 1) / a.part_pages;
    if (parts <= 1) return;
    const int64_t head = static_cast<int64_t>(s) * a.num_q_heads + hq, slot0 = head * a.num_parts;
    float M = -INFINITY;
    for (int32_t p = 0; p < parts; ++p) M = fmaxf(M, a.ws_ml[2 * (slot0 + p)]);
    const float ref = M == -INFINITY ? 0.f : M;
    float num = 0.f, den = 0.f;
    for (int32_t p = 0; p < parts; ++p) {
        const float w = a.ws_ml[2 * (slot0 + p) + 1] * exp2f(a.ws_ml[2 * (slot0 + p)] - ref);
        num = fmaf(w, a.ws_o[(slot0 + p) * D + d], num);
        den += w;
    }
    out[head * D + d] = narrow<T>(den == 0.f ? 0.f : num / den);
}

template <typename T, int D>
cudaError_t launch_decode_impl(const DecodeArgs& d, const ScoreArgs& score, const ScoredSimtPlan& plan,
                               cudaStream_t stream) {
    SimtArgs a{};
    a.block_table = d.block_table;
    a.seq_lens = d.seq_lens;
    a.max_blocks = d.max_blocks_per_seq;
    a.num_q_heads = d.num_q_heads;
    a.num_kv_heads = d.num_kv_heads;
    a.num_blocks = d.num_blocks;
    a.sub_log2 = block_size_log2(d.block_size) - 4;
    a.cap_tokens = min(table_tokens(a.max_blocks, a.sub_log2), d.max_seq_len);
    a.part_pages = plan.part_pages;
    a.num_parts = plan.num_parts;
    a.head_chunks = (d.num_q_heads / d.num_kv_heads + kHeads - 1) / kHeads;
    a.scale = d.scale;
    a.score = score;
    a.ws_o = reinterpret_cast<float*>(static_cast<char*>(d.workspace) + kScoredCounterBytes);
    a.ws_ml = a.ws_o + static_cast<size_t>(d.num_seqs) * d.num_q_heads * plan.num_parts * D;
    a.err = d.err;
    const dim3 grid(d.num_seqs, d.num_kv_heads * a.head_chunks, plan.num_parts);
    scored_simt_kernel<T, D><<<grid, kThreads, 0, stream>>>(static_cast<T*>(d.out), static_cast<const T*>(d.q),
                                                            static_cast<const T*>(d.k_cache),
                                                            static_cast<const T*>(d.v_cache), a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || plan.num_parts == 1) return e;
    scored_simt_merge_kernel<T, D><<<dim3(d.num_seqs, d.num_q_heads), D, 0, stream>>>(static_cast<T*>(d.out), a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_prefill_impl(const PrefillArgs& p, const ScoreArgs& score, cudaStream_t stream) {
    SimtArgs a{};
    a.block_table = p.block_table;
    a.seq_lens = p.seq_lens;
    a.query_start_loc = p.query_start_loc;
    a.max_blocks = p.max_blocks_per_seq;
    a.num_q_heads = p.num_q_heads;
    a.num_kv_heads = p.num_kv_heads;
    a.num_blocks = p.num_blocks;
    a.sub_log2 = block_size_log2(p.block_size) - 4;
    a.cap_tokens = min(table_tokens(a.max_blocks, a.sub_log2), p.max_seq_len);
    a.max_chunk = p.max_chunk_len;
    a.part_pages = 0x7fffffff;
    a.num_parts = 1;
    a.head_chunks = (p.num_q_heads / p.num_kv_heads + kHeads - 1) / kHeads;
    a.scale = p.scale;
    a.score = score;
    a.err = p.err;
    const dim3 grid(static_cast<unsigned>(p.num_seqs) * p.max_chunk_len, p.num_kv_heads * a.head_chunks, 1);
    scored_simt_kernel<T, D><<<grid, kThreads, 0, stream>>>(static_cast<T*>(p.out), static_cast<const T*>(p.q),
                                                            static_cast<const T*>(p.k_cache),
                                                            static_cast<const T*>(p.v_cache), a);
    return cudaGetLastError();
}

}  // namespace

int32_t scored_simt_head_chunks(int32_t group) { return (group + kHeads - 1) / kHeads; }

// Partitions so that (sequence, kv head, head chunk, partition) items fill the SMs about twice, of
// at least 4 pages each.
ScoredSimtPlan plan_scored_simt(int32_t S, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_seq_len, int num_sms) {
    ScoredSimtPlan p{};
    const int64_t items = static_cast<int64_t>(S) * Hkv * scored_simt_head_chunks(Hq / Hkv);
    const int32_t pages = max_seq_len / kPageTokens + 2;
    int64_t parts = items > 0 ? (2LL * num_sms + items - 1) / items : 1;
    parts = min(parts, static_cast<int64_t>((pages + 3) / 4));
    p.part_pages = static_cast<int32_t>((pages + parts - 1) / parts);
    p.num_parts = (pages + p.part_pages - 1) / p.part_pages;
    p.workspace_bytes =
        p.num_parts > 1
            ? kScoredCounterBytes + static_cast<size_t>(S) * Hq * p.num_parts * (D + 2) * sizeof(float)
            : 0;
    return p;
}

cudaError_t launch_scored_decode_simt(const DecodeArgs& a, const ScoreArgs& score, const ScoredSimtPlan& plan,
                                      cudaStream_t stream) {
    if (a.dtype == PA_F32)
        return a.head_dim == 128 ? launch_decode_impl<float, 128>(a, score, plan, stream)
                                 : launch_decode_impl<float, 64>(a, score, plan, stream);
    return a.head_dim == 128 ? launch_decode_impl<uint16_t, 128>(a, score, plan, stream)
                             : launch_decode_impl<uint16_t, 64>(a, score, plan, stream);
}

cudaError_t launch_scored_prefill_simt(const PrefillArgs& a, const ScoreArgs& score, cudaStream_t stream) {
    if (a.dtype == PA_F32)
        return a.head_dim == 128 ? launch_prefill_impl<float, 128>(a, score, stream)
                                 : launch_prefill_impl<float, 64>(a, score, stream);
    return a.head_dim == 128 ? launch_prefill_impl<uint16_t, 128>(a, score, stream)
                             : launch_prefill_impl<uint16_t, 64>(a, score, stream);
}

}  // namespace pa
