// Scored attention on the CUDA cores: every type, head layout and score, decode and prefill.
//
// A CTA takes up to R rows (R = 4 or 16) that share a kv head: the q heads of a decode row, or the
// q heads of R / G consecutive tokens of a chunk, so that each K and V element it reads serves all of
// them. Its eight warps take the 16-token pages that some row sees in turn. Scores: a lane holds one
// key and every other row (two lanes a key), so a score is one thread's dot product, q coming from
// shared memory by broadcast, and the page's maximum takes four shuffles a row. Then lanes change
// roles, through shared memory: a lane holds head_dim / 32 columns of the output of all R rows and
// walks the page's keys. The softmax runs online per warp in the log2 domain; the warps' (max, sum,
// output) meet in shared memory, and partitions of a decode row's pages in the workspace, where the
// last CTA to arrive merges them by the same rule:
//   M = max_p m_p,  w_p = l_p 2^(m_p - M),  out = sum_p w_p o_p / sum_p w_p.
// The pages are those of the rows' visible spans only, so a window or a document start costs no
// reads outside them. A page that a span cuts is read; its keys that no row sees are skipped in V.
#include <math.h>

#include "pa_internal.h"
#include "scored.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFewRows = 4, kManyRows = 16;  // R: rows of a CTA
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int32_t kFar = 0x7fffffff;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const uint16_t* p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}
// E consecutive elements (2 or 4).
__device__ __forceinline__ void load_n(const float* p, float (&x)[2]) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = v.x, x[1] = v.y;
}
__device__ __forceinline__ void load_n(const uint16_t* p, float (&x)[2]) {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(p));
    x[0] = __uint_as_float(v << 16), x[1] = __uint_as_float(v & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ void load_n(const T* p, float (&x)[4]) {
    const float4 v = load4(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}

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
    int32_t G, head_chunks, tokens, groups;  // q heads per kv head; chunks of R heads; tokens per CTA; CTAs per chunk
    int32_t part_pages, num_parts;
    float scale;
    ScoreArgs score;
    int32_t* counter;
    float* ws_o;
    float* ws_ml;
    uint32_t* err;
};

// Shared memory, in floats: the rows' q while pages are walked, then the warps' outputs.
template <int D, int R>
struct Smem {
    static constexpr int q_stride = D + 4;  // two rows in a broadcast lie in different banks
    static constexpr int q = 0;
    static constexpr int p = q + R * q_stride;             // [kWarps][16 keys][R]
    static constexpr int corr = p + kWarps * 16 * R;       // [kWarps][R]
    static constexpr int o = 0;                            // [kWarps][R][D]
    static constexpr int walk = corr + kWarps * R, join = o + kWarps * R * D;
    static constexpr int bytes = 4 * (walk > join ? walk : join);
};

template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads) scored_simt_kernel(T* __restrict__ out, const T* __restrict__ q,
                                                               const T* __restrict__ k_cache,
                                                               const T* __restrict__ v_cache,
                                                               const __grid_constant__ SimtArgs a) {
    constexpr int E = D / 32, RL = R / 2;
    using L = Smem<D, R>;
    extern __shared__ float4 smem4[];
    float* sm = reinterpret_cast<float*>(smem4);
    __shared__ KeySpans spans[R];
    __shared__ float slopes[R];
    __shared__ int32_t where[R];      // the rows' positions
    __shared__ KeySpans hull, inner;  // keys that some row sees (and what lies between them), that all rows see
    __shared__ float jm[kWarps][R], jl[kWarps][R], jM[R], jden[R];
    __shared__ int32_t last_part;
    const int32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // launched while the kernel before drains: nothing is read before it is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- the CTA's rows: row r is token t0 + r / heads, q head h0 + r % heads -------------------
    const int32_t hk = blockIdx.y / a.head_chunks, hc = blockIdx.y - hk * a.head_chunks;
    const int32_t heads = min(a.G - hc * R, min(a.G, R)), h0 = hk * a.G + hc * R;
    const bool decode = a.query_start_loc == nullptr;
    const int32_t s = decode ? blockIdx.x : blockIdx.x / a.groups, t0 = decode ? 0 : (blockIdx.x - s * a.groups) * a.tokens;
    int32_t len = __ldg(a.seq_lens + s), row0 = s, pos0, n_tok = 1;
    if (decode) {
        if (len < 0 || len > a.cap_tokens) {
            if (tid == 0) raise_error(a.err, PA_DEVERR_LEN_RANGE);
            len = len < 0 ? 0 : a.cap_tokens;
        }
        pos0 = len - 1;
    } else {
        const int32_t q0 = __ldg(a.query_start_loc + s), chunk = __ldg(a.query_start_loc + s + 1) - q0;
        if (chunk < 0 || chunk > a.max_chunk || chunk > len || len > a.cap_tokens) {
            if (tid == 0 && t0 == 0) raise_error(a.err, PA_DEVERR_LEN_RANGE);
            return;
        }
        if (t0 >= chunk) return;
        row0 = q0 + t0;
        pos0 = len - chunk + t0;
        n_tok = min(a.tokens, chunk - t0);
    }
    const int32_t n_rows = n_tok * heads;
    if (warp == 0) {
        KeySpans sp{0, 0, 0, 0};
        const bool valid = lane < n_rows;
        if (valid) {
            const int32_t tt = lane / heads, row = row0 + tt;
            sp = key_spans(len, pos0 + tt, a.score.key_start ? __ldg(a.score.key_start + row) : 0,
                           a.score.prefix_len ? __ldg(a.score.prefix_len + s) : 0, a.score.window);
            slopes[lane] = a.score.slopes ? __ldg(a.score.slopes + h0 + (lane - tt * heads)) * kLog2e : 0.f;
            where[lane] = pos0 + tt;
        } else if (lane < R) {
            slopes[lane] = 0.f;
            where[lane] = 0;
        }
        if (lane < R) spans[lane] = sp;
        const bool in_a = sp.a0 < sp.a1, in_b = sp.b0 < sp.b1;
        const int32_t ha0 = __reduce_min_sync(~0u, in_a ? sp.a0 : kFar), ha1 = __reduce_max_sync(~0u, in_a ? sp.a1 : 0);
        const int32_t hb0 = __reduce_min_sync(~0u, in_b ? sp.b0 : kFar), hb1 = __reduce_max_sync(~0u, in_b ? sp.b1 : 0);
        const int32_t ia0 = __reduce_max_sync(~0u, valid ? sp.a0 : 0), ia1 = __reduce_min_sync(~0u, valid ? sp.a1 : kFar);
        const int32_t ib0 = __reduce_max_sync(~0u, valid ? sp.b0 : 0), ib1 = __reduce_min_sync(~0u, valid ? sp.b1 : kFar);
        if (lane == 0) {
            hull = KeySpans{ha0 < ha1 ? ha0 : 0, ha0 < ha1 ? ha1 : 0, hb0 < hb1 ? hb0 : 0, hb0 < hb1 ? hb1 : 0};
            inner = KeySpans{ia0, ia1, ib0, ib1};
        }
    }
    // ---- q, scaled, rows without a query zero ---------------------------------------------------
    for (int32_t i = tid; i < R * D / 4; i += kThreads) {
        const int32_t r = i / (D / 4), c = i - r * (D / 4);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n_rows) {
            const int32_t tt = r / heads;
            v = load4(q + (static_cast<int64_t>(row0 + tt) * a.num_q_heads + h0 + (r - tt * heads)) * D + c * 4);
            v.x *= a.scale, v.y *= a.scale, v.z *= a.scale, v.w *= a.scale;
        }
        *reinterpret_cast<float4*>(sm + L::q + r * L::q_stride + c * 4) = v;
    }
    __syncthreads();

    const PageList pl = page_list(hull);
    const int32_t parts = (pl.n + a.part_pages - 1) / a.part_pages, part = blockIdx.z;
    if (part >= max(parts, 1)) return;  // uniform over the CTA
    const int32_t end = min(pl.n, (part + 1) * a.part_pages);
    const int32_t key = lane & 15, hh = lane >> 4;  // this lane's key of a page; its rows are 2 i + hh
    const int32_t* table = a.block_table + static_cast<int64_t>(s) * a.max_blocks;
    float* ps = sm + L::p + warp * 16 * R;    // [key][hh RL + i]: the weights
    float* corr = sm + L::corr + warp * R;    // [hh RL + i]: what the outputs so far are scaled by
    float m[RL], l[RL], acc[R][E];            // acc[hh RL + i]
#pragma unroll
    for (int i = 0; i < RL; ++i) m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
    int32_t i0 = part * a.part_pages + warp;
    int32_t phys = i0 < end ? __ldg(table + (pl.page(i0) >> a.sub_log2)) : 0;
    for (; i0 < end; i0 += kWarps) {
        const int32_t page = pl.page(i0), block = phys, j0 = page * kPageTokens, j = j0 + key;
        if (i0 + kWarps < end) phys = __ldg(table + (pl.page(i0 + kWarps) >> a.sub_log2));
        if (block < 0 || block >= a.num_blocks) {
            raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
            continue;
        }
        const int64_t base = ((((static_cast<int64_t>(block) * a.num_kv_heads + hk) << a.sub_log2) +
                               (page & ((1 << a.sub_log2) - 1))) * kPageTokens) * D;
        // ---- scores of (key, rows 2 i + hh) ----
        float z[RL];
#pragma unroll
        for (int i = 0; i < RL; ++i) z[i] = 0.f;
        const T* kp = k_cache + base + key * D;
        const float* qs = sm + L::q + hh * L::q_stride;
#pragma unroll
        for (int c0 = 0; c0 < D / 4; c0 += 8) {
            float4 kv[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) kv[c] = load4(kp + (c0 + c) * 4);
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int i = 0; i < RL; ++i) {
                    const float4 qv = *reinterpret_cast<const float4*>(qs + 2 * i * L::q_stride + (c0 + c) * 4);
                    z[i] = fmaf(qv.x, kv[c].x, z[i]);
                    z[i] = fmaf(qv.y, kv[c].y, z[i]);
                    z[i] = fmaf(qv.z, kv[c].z, z[i]);
                    z[i] = fmaf(qv.w, kv[c].w, z[i]);
                }
        }
        const bool whole = (j0 >= inner.a0 && j0 + kPageTokens <= inner.a1) || (j0 >= inner.b0 && j0 + kPageTokens <= inner.b1);
        uint32_t seen = 0xffffu;  // keys of the page that some row sees
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            if (a.score.cap > 0.f) z[i] = a.score.cap * tanhf(z[i] / a.score.cap);
            z[i] *= kLog2e;
            if (a.score.slopes) z[i] -= slopes[2 * i + hh] * static_cast<float>(abs(where[2 * i + hh] - j));
        }
        if (!whole) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                const bool sees = spans[2 * i + hh].sees(j);
                any |= sees;
                if (!sees) z[i] = -INFINITY;
            }
            seen = __ballot_sync(0xffffffffu, any);
            seen = (seen | seen >> 16) & 0xffffu;
            if (seen == 0u) continue;
        }
        // ---- weights against the rows' running maxima ----
        bool grow = false;
        float mn[RL];
#pragma unroll
        for (int i = 0; i < RL; ++i) mn[i] = z[i];
#pragma unroll
        for (int off = 8; off > 0; off >>= 1)
#pragma unroll
            for (int i = 0; i < RL; ++i) mn[i] = fmaxf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], off));
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            grow |= mn[i] > m[i];
            mn[i] = fmaxf(mn[i], m[i]);
            const float ref = mn[i] == -INFINITY ? 0.f : mn[i];  // nothing finite yet: weights are 0, not NaN
            z[i] = exp2f(z[i] - ref);
        }
        const bool rescale = __any_sync(0xffffffffu, grow);
        if (rescale) {
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                const float f = exp2f(m[i] - (mn[i] == -INFINITY ? 0.f : mn[i]));
                l[i] *= f;
                m[i] = mn[i];
                if (key == 0) corr[hh * RL + i] = f;
            }
        }
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            l[i] += z[i];
            ps[key * R + hh * RL + i] = z[i];
        }
        __syncwarp();
        if (rescale) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float f = corr[r];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[r][e] *= f;
            }
        }
        // ---- outputs: columns lane E .. of all rows ----
        const T* vp = v_cache + base + lane * E;
#pragma unroll
        for (int k0 = 0; k0 < kPageTokens; k0 += 8) {
            float vv[8][E];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (seen >> (k0 + k) & 1u) load_n(vp + (k0 + k) * D, vv[k]);
                else
#pragma unroll
                    for (int e = 0; e < E; ++e) vv[k][e] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(ps + (k0 + k) * R + r);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        acc[r][e] = fmaf(w.x, vv[k][e], acc[r][e]);
                        acc[r + 1][e] = fmaf(w.y, vv[k][e], acc[r + 1][e]);
                        acc[r + 2][e] = fmaf(w.z, vv[k][e], acc[r + 2][e]);
                        acc[r + 3][e] = fmaf(w.w, vv[k][e], acc[r + 3][e]);
                    }
                }
        }
        __syncwarp();
    }

    // ---- the warps' parts meet; row order hh RL + i -> row 2 i + hh -------------------------------
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < RL; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
    if (key == 0)
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            jm[warp][2 * i + hh] = m[i];
            jl[warp][2 * i + hh] = l[i];
        }
    __syncthreads();  // q and the weights are done with
    if (tid < R) {
        float M = -INFINITY, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, jm[w][tid]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(jm[w][tid] - ref);  // a warp without keys: m = -inf, weight 0
            den = fmaf(jl[w][tid], f, den);
            jm[w][tid] = f;
        }
        jM[tid] = M;
        jden[tid] = den;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float* o = sm + L::o + (warp * R + (i % RL) * 2 + i / RL) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = acc[i][e];
    }
    __syncthreads();
    for (int32_t i = tid; i < n_rows * D; i += kThreads) {
        const int32_t r = i / D, d = i - r * D;
        float num = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) num = fmaf(sm[L::o + (w * R + r) * D + d], jm[w][r], num);
        const float o = jden[r] == 0.f ? 0.f : num / jden[r];
        const int32_t tt = r / heads;
        const int64_t head = static_cast<int64_t>(row0 + tt) * a.num_q_heads + h0 + (r - tt * heads);
        if (parts <= 1) {
            out[head * D + d] = narrow<T>(o);
        } else {
            const int64_t slot = head * a.num_parts + part;
            __stcg(a.ws_o + slot * D + d, o);
            if (d == 0) __stcg(reinterpret_cast<float2*>(a.ws_ml) + slot, make_float2(jM[r], jden[r]));
        }
    }
    if (parts <= 1) return;
    // ---- a decode row in several partitions: the last CTA to arrive merges them --------------------
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        int32_t* c = a.counter + (s * static_cast<int32_t>(gridDim.y) + blockIdx.y);
        last_part = atomicAdd(c, 1) == parts - 1;
        if (last_part) *c = 0;  // ready for the next call
        __threadfence();
    }
    __syncthreads();
    if (!last_part) return;
    for (int32_t i = tid; i < n_rows * D; i += kThreads) {
        const int32_t r = i / D, d = i - r * D;
        const int64_t head = static_cast<int64_t>(row0) * a.num_q_heads + h0 + r, slot0 = head * a.num_parts;
        const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + slot0;
        float M = -INFINITY;
        for (int32_t p = 0; p < parts; ++p) M = fmaxf(M, __ldcg(ml + p).x);
        const float ref = M == -INFINITY ? 0.f : M;
        float num = 0.f, den = 0.f;
        for (int32_t p = 0; p < parts; ++p) {
            const float2 v = __ldcg(ml + p);
            const float w = v.y * exp2f(v.x - ref);
            num = fmaf(w, __ldcg(a.ws_o + (slot0 + p) * D + d), num);
            den += w;
        }
        out[head * D + d] = narrow<T>(den == 0.f ? 0.f : num / den);
    }
}

template <typename T, int D, int R>
cudaError_t launch_rows(void* out, const void* q, const void* k, const void* v, const SimtArgs& a, dim3 grid,
                        cudaStream_t stream) {
    constexpr int bytes = Smem<D, R>::bytes;
    if (bytes > 40960) {
        const cudaError_t e = cudaFuncSetAttribute(scored_simt_kernel<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_simt_kernel<T, D, R>, static_cast<T*>(out), static_cast<const T*>(q),
                              static_cast<const T*>(k), static_cast<const T*>(v), a);
}

template <typename T, int D>
cudaError_t launch_impl(void* out, const void* q, const void* k, const void* v, SimtArgs& a, int32_t num_seqs,
                        cudaStream_t stream) {
    const int32_t R = a.G * (a.query_start_loc ? a.max_chunk : 1) <= kFewRows ? kFewRows : kManyRows;
    a.head_chunks = (a.G + R - 1) / R;
    a.tokens = a.G < R ? R / a.G : 1;
    a.groups = a.query_start_loc ? (a.max_chunk + a.tokens - 1) / a.tokens : 1;
    const dim3 grid(static_cast<unsigned>(num_seqs) * a.groups, a.num_kv_heads * a.head_chunks, a.num_parts);
    return R == kFewRows ? launch_rows<T, D, kFewRows>(out, q, k, v, a, grid, stream)
                         : launch_rows<T, D, kManyRows>(out, q, k, v, a, grid, stream);
}

template <typename T>
cudaError_t launch_type(void* out, const void* q, const void* k, const void* v, SimtArgs& a, int32_t head_dim,
                        int32_t num_seqs, cudaStream_t stream) {
    return head_dim == 128 ? launch_impl<T, 128>(out, q, k, v, a, num_seqs, stream)
                           : launch_impl<T, 64>(out, q, k, v, a, num_seqs, stream);
}

// What DecodeArgs and PrefillArgs share.
template <typename A>
SimtArgs common_args(const A& d, const ScoreArgs& score) {
    SimtArgs a{};
    a.block_table = d.block_table;
    a.seq_lens = d.seq_lens;
    a.max_blocks = d.max_blocks_per_seq;
    a.num_q_heads = d.num_q_heads;
    a.num_kv_heads = d.num_kv_heads;
    a.num_blocks = d.num_blocks;
    a.sub_log2 = block_size_log2(d.block_size) - 4;
    a.cap_tokens = min(table_tokens(a.max_blocks, a.sub_log2), d.max_seq_len);
    a.G = d.num_q_heads / d.num_kv_heads;
    a.part_pages = 0x40000000;
    a.num_parts = 1;
    a.scale = d.scale;
    a.score = score;
    a.err = d.err;
    return a;
}

}  // namespace

int32_t scored_simt_head_chunks(int32_t group) {
    return group <= kFewRows ? 1 : (group + kManyRows - 1) / kManyRows;
}

// Partitions so that (sequence, kv head, head chunk, partition) items fill the SMs about twice, of
// at least kMinPages pages each.
ScoredSimtPlan plan_scored_simt(int32_t S, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_seq_len, int num_sms) {
    constexpr int64_t kMinPages = 2 * kWarps;
    ScoredSimtPlan p{};
    const int64_t items = static_cast<int64_t>(S) * Hkv * scored_simt_head_chunks(Hq / Hkv);
    const int32_t pages = max_seq_len / kPageTokens + 2;
    int64_t parts = items > 0 ? (2LL * num_sms + items - 1) / items : 1;
    parts = min(parts, (pages + kMinPages - 1) / kMinPages);
    p.part_pages = static_cast<int32_t>((pages + parts - 1) / parts);
    p.num_parts = (pages + p.part_pages - 1) / p.part_pages;
    p.workspace_bytes =
        p.num_parts > 1
            ? kScoredCounterBytes + static_cast<size_t>(S) * Hq * p.num_parts * (D + 2) * sizeof(float)
            : 0;
    return p;
}

cudaError_t launch_scored_decode_simt(const DecodeArgs& d, const ScoreArgs& score, const ScoredSimtPlan& plan,
                                      cudaStream_t stream) {
    SimtArgs a = common_args(d, score);
    a.part_pages = plan.part_pages;
    a.num_parts = plan.num_parts;
    a.counter = static_cast<int32_t*>(d.workspace);
    a.ws_o = reinterpret_cast<float*>(static_cast<char*>(d.workspace) + kScoredCounterBytes);
    a.ws_ml = a.ws_o + static_cast<size_t>(d.num_seqs) * d.num_q_heads * plan.num_parts * d.head_dim;
    return d.dtype == PA_F32 ? launch_type<float>(d.out, d.q, d.k_cache, d.v_cache, a, d.head_dim, d.num_seqs, stream)
                             : launch_type<uint16_t>(d.out, d.q, d.k_cache, d.v_cache, a, d.head_dim, d.num_seqs, stream);
}

cudaError_t launch_scored_prefill_simt(const PrefillArgs& p, const ScoreArgs& score, cudaStream_t stream) {
    SimtArgs a = common_args(p, score);
    a.query_start_loc = p.query_start_loc;
    a.max_chunk = p.max_chunk_len;
    return p.dtype == PA_F32 ? launch_type<float>(p.out, p.q, p.k_cache, p.v_cache, a, p.head_dim, p.num_seqs, stream)
                             : launch_type<uint16_t>(p.out, p.q, p.k_cache, p.v_cache, a, p.head_dim, p.num_seqs, stream);
}

}  // namespace pa
