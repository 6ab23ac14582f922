// Scored attention on the CUDA cores: every type, head layout and score, decode and prefill.
//
// A CTA takes up to R rows (R = 4 or 16) that share a kv head: the q heads of a decode row, or the
// q heads of R / G consecutive tokens of a chunk, so that each K and V element it reads serves all of
// them. Its warps (8 or 4) take the 16-token pages that some row sees in turn; each has room for one K and
// one V page, and the next K page is on its way while the V page is used, and the other way round.
// Scores: a lane multiplies 4 keys by 8 rows (R = 4: by 4) over a fourth (an eighth) of the columns, so
// that a value out of shared memory serves 4 or 8 products; a reduction that also scatters leaves each
// lane the scores of one key with half of the rows, and the page's maximum takes four shuffles a row.
// Then lanes change roles, through shared memory: a lane holds head_dim / 32 columns of the output of
// all R rows and walks the page's keys. Products run as packed pairs (two elements an instruction). The softmax runs online per warp in the log2 domain; the warps' (max, sum,
// output) meet in shared memory, and partitions of a decode row's pages in the workspace, where the
// last CTA to arrive merges them by the same rule:
//   M = max_p m_p,  w_p = l_p 2^(m_p - M),  out = sum_p w_p o_p / sum_p w_p.
// Pages of a 4-bit pool (fp4.cuh) land as they are, and their warp unpacks them into the room of an ordinary
// page, exactly, before it uses them. The pages are those of the rows' visible spans only, so a window or a document start costs no
// reads outside them. A page that a span cuts is read; its keys that no row sees are skipped in V.
//
// Bound: for a few rows the chain launch, lengths, block ids, pages, join (about 5 us: 24 sequences of up
// to 777 keys, 12 q / 4 kv heads of 64 in fp32: 5.8 us); for chunks the fp32 pipes (two products of a
// page take 2000 of 3100 cycles, one page and two warps per scheduler: 4 sequences of 17 to 96 rows in a
// window of 256 keys: 15.7 us). Loads of K and V straight into registers, a key per lane, took 27 us.
#include <math.h>

#include <type_traits>

#include "fp4.cuh"
#include "pa_internal.h"
#include "scored.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kFewRows = 4, kManyRows = 16;  // R: rows of a CTA
constexpr int kMaxParts = 128;  // partitions: the merge holds their weights in shared memory
constexpr float kLag = 8.f;  // log2 units
constexpr int kRawPairs = 3;  // 4-bit pools: page pairs of a warp on their way or at hand
constexpr int32_t kFar = 0x7fffffff;

// Four consecutive elements as two packed pairs.
struct Pairs {
    uint64_t lo, hi;
};
__device__ __forceinline__ Pairs load4(const float* p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    return Pairs{v.x, v.y};
}
__device__ __forceinline__ Pairs load4(const uint16_t* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return Pairs{pack2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u)),
                 pack2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u))};
}
// E consecutive elements (2 or 4), each twice.
__device__ __forceinline__ void load_twice(const float* p, uint64_t (&x)[2]) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = pack2(v.x, v.x), x[1] = pack2(v.y, v.y);
}
__device__ __forceinline__ void load_twice(const uint16_t* p, uint64_t (&x)[2]) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    const float lo = __uint_as_float(v << 16), hi = __uint_as_float(v & 0xffff0000u);
    x[0] = pack2(lo, lo), x[1] = pack2(hi, hi);
}
template <typename T>
__device__ __forceinline__ void load_twice(const T* p, uint64_t (&x)[4]) {
    const Pairs v = load4(p);
    float f[4];
    unpack2(v.lo, f[0], f[1]);
    unpack2(v.hi, f[2], f[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack2(f[e], f[e]);
}

__device__ __forceinline__ void cp_async16(void* smem_dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem_dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {  // all but the N groups committed last have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// Eight consecutive elements, 16-byte aligned.
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

struct SimtArgs {
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* query_start_loc;  // null: decode
    int32_t max_blocks, num_q_heads, num_kv_heads, num_blocks, sub_log2, cap_tokens, max_chunk;
    int32_t G, head_chunks, tokens, groups;  // q heads per kv head; chunks of R heads; tokens per CTA; CTAs per chunk
    int32_t part_pages, num_parts;
    float scale;
    float v_scale;  // 4-bit pools: the V pool's factor
    ScoreArgs score;
    int32_t* counter;
    float* ws_o;
    float* ws_ml;
    uint32_t* err;
};

// Shared memory in bytes: q, weights and pages while pages are walked, then the warps' outputs.
template <typename T, int D, int R, int kWarps, bool F4>
struct Smem {
    static constexpr int pad = 16 / sizeof(T);  // rows 16 bytes apart in bank: a lane reads its own row
    static constexpr int q_stride = D + 4;      // two rows in a broadcast lie in different banks
    static constexpr int q = 0;
    static constexpr int p = q + 4 * R * q_stride;                // [kWarps][16 keys][R]
    static constexpr int p_stride = R == 4 ? 4 : R + 4;           // lanes store their keys' weights in different banks
    static constexpr int corr = p + 4 * kWarps * 16 * p_stride;  // [kWarps][R]
    static constexpr int page = corr + 4 * kWarps * R;     // [kWarps] K page, V page
    static constexpr int k_stride = D + pad;
    static constexpr int k_bytes = 16 * k_stride * static_cast<int>(sizeof(T));
    static constexpr int raw = k_bytes + 16 * D * static_cast<int>(sizeof(T));  // 4-bit pools: pairs of a K and a V page
    static constexpr int page_bytes = raw + (F4 ? kRawPairs * 2 * fp4_page_bytes(D) : 0);
    static constexpr int walk = page + kWarps * page_bytes, join = 4 * kWarps * R * D;
    static constexpr int bytes = walk > join ? walk : join;
    static_assert(kMaxParts * R * 8 <= bytes, "the merge's weights");
};

template <typename T, int D, int R, int kWarps, bool F4>
__global__ void __launch_bounds__(32 * kWarps) scored_simt_kernel(T* __restrict__ out, const T* __restrict__ q,
                                                               const T* __restrict__ k_cache,
                                                               const T* __restrict__ v_cache,
                                                               const __grid_constant__ SimtArgs a) {
    constexpr int E = D / 32, RL = R / 2, kThreads = 32 * kWarps;
    using L = Smem<T, D, R, kWarps, F4>;
    extern __shared__ float4 smem4[];
    char* sm = reinterpret_cast<char*>(smem4);
    __shared__ KeySpans spans[R];
    __shared__ float slopes[R];
    __shared__ int32_t where[R];      // the rows' positions
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
    // every warp works out the rows' spans, so that its first pages can be on their way before the rows' q
    KeySpans sp{0, 0, 0, 0};
    const bool valid = lane < n_rows;
    if (valid) {
        const int32_t tt = lane / heads;
        sp = key_spans(len, pos0 + tt, a.score.key_start ? __ldg(a.score.key_start + row0 + tt) : 0,
                       a.score.prefix_len ? __ldg(a.score.prefix_len + s) : 0, a.score.window, a.score.causal);
    }
    if (warp == 0 && lane < R) {
        const int32_t tt = lane / heads;
        spans[lane] = sp;
        slopes[lane] = valid && a.score.slopes ? __ldg(a.score.slopes + h0 + (lane - tt * heads)) * kLog2e : 0.f;
        where[lane] = pos0 + tt;
    }
    const bool in_a = sp.a0 < sp.a1, in_b = sp.b0 < sp.b1;
    KeySpans hull, inner;  // keys that some row sees, with what lies between them; keys that all rows see
    hull.a0 = __reduce_min_sync(~0u, in_a ? sp.a0 : kFar);
    hull.a1 = __reduce_max_sync(~0u, in_a ? sp.a1 : 0);
    hull.b0 = __reduce_min_sync(~0u, in_b ? sp.b0 : kFar);
    hull.b1 = __reduce_max_sync(~0u, in_b ? sp.b1 : 0);
    if (hull.a0 == kFar) hull.a0 = 0;
    if (hull.b0 == kFar) hull.b0 = 0;
    inner.a0 = __reduce_max_sync(~0u, valid ? sp.a0 : 0);
    inner.a1 = __reduce_min_sync(~0u, valid ? sp.a1 : kFar);
    inner.b0 = __reduce_max_sync(~0u, valid ? sp.b0 : 0);
    inner.b1 = __reduce_min_sync(~0u, valid ? sp.b1 : kFar);
    const PageList pl = page_list(hull);
    const int32_t parts = (pl.n + a.part_pages - 1) / a.part_pages, part = blockIdx.z;
    if (part >= max(parts, 1)) return;  // uniform over the CTA
    const int32_t end = min(pl.n, (part + 1) * a.part_pages), first = part * a.part_pages + warp;
    const int32_t* table = a.block_table + static_cast<int64_t>(s) * a.max_blocks;
    T* k_page = reinterpret_cast<T*>(sm + L::page + warp * L::page_bytes);
    T* v_page = k_page + 16 * L::k_stride;
    uint8_t* const raw_pages = reinterpret_cast<uint8_t*>(k_page) + L::raw;  // F4: [kRawPairs] K, then V
    auto block_of = [&](int32_t i) { return i < end ? __ldg(table + (pl.page(i) >> a.sub_log2)) : 0; };
    auto in_pool = [&](int32_t block) { return block >= 0 && block < a.num_blocks; };
    // copy list page i of this warp, in this block, from a cache: 16 rows of D elements
    auto fetch = [&](const T* cache, T* dst, int32_t stride, int32_t i, int32_t block) {
        if (i < end && in_pool(block)) {
            const int64_t row = ((static_cast<int64_t>(block) * a.num_kv_heads + hk) << a.sub_log2) +
                                (pl.page(i) & ((1 << a.sub_log2) - 1));
            const T* src = cache + row * (kPageTokens * D);
            constexpr int kN = 16 / sizeof(T), kChunks = D / kN;  // 16-byte chunks of a row
#pragma unroll
            for (int c = lane; c < 16 * kChunks; c += 32) cp_async16(dst + c / kChunks * stride + c % kChunks * kN, src + c * kN);
        }
        cp_async_commit();
    };
    // F4: copy list page i of this warp, K and V, as they lie there
    auto fetch_pair = [&](int32_t slot, int32_t i, int32_t block) {
        if (i < end && in_pool(block)) {
            const int64_t at = (((static_cast<int64_t>(block) * a.num_kv_heads + hk) << a.sub_log2) +
                                (pl.page(i) & ((1 << a.sub_log2) - 1))) * fp4_page_bytes(D);
            uint8_t* to = raw_pages + slot * 2 * fp4_page_bytes(D);
#pragma unroll
            for (int c = lane; c < fp4_page_bytes(D) / 16; c += 32) {
                cp_async16(to + c * 16, reinterpret_cast<const uint8_t*>(k_cache) + at + c * 16);
                cp_async16(to + fp4_page_bytes(D) + c * 16, reinterpret_cast<const uint8_t*>(v_cache) + at + c * 16);
            }
        }
        cp_async_commit();
    };
    // F4: a page that has landed, as values of T times factor: a lane takes 8 dims of a key at a time
    auto unpack = [&](T* dst, int32_t stride, const uint8_t* raw, float factor) {
#pragma unroll
        for (int c = lane; c < 2 * D; c += 32) {
            const int key_row = c / (D / 8), d = c % (D / 8) * 8;
            const float s = halves_to_floats(e4m3x2_halves(raw[fp4_scales_at(D) + key_row * (D / 16) + d / 16])).x * factor;
            uint32_t h[4];
            fp4_halves(reinterpret_cast<const uint32_t*>(raw)[c], h);
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = halves_to_floats(h[e]);
                x[2 * e] = v.x * s, x[2 * e + 1] = v.y * s;
            }
            store8(dst + key_row * stride + d, x);
        }
        __syncwarp();
    };
    int32_t block = block_of(first), block_next = block_of(first + kWarps);
    int32_t block_third = F4 ? block_of(first + 2 * kWarps) : 0, slot = 0;
    if constexpr (F4) {
        static_assert(kRawPairs == 3, "the ids that the loop carries");
        fetch_pair(0, first, block);
        fetch_pair(1, first + kWarps, block_next);
        fetch_pair(2, first + 2 * kWarps, block_third);
    } else {
        fetch(k_cache, k_page, L::k_stride, first, block);
        fetch(v_cache, v_page, D, first, block);
    }
    // ---- q, scaled, rows without a query zero ---------------------------------------------------
    for (int32_t i = tid; i < R * D / 4; i += kThreads) {
        const int32_t r = i / (D / 4), c = i - r * (D / 4);
        Pairs v{0ull, 0ull};
        if (r < n_rows) {
            const int32_t tt = r / heads;
            v = load4(q + (static_cast<int64_t>(row0 + tt) * a.num_q_heads + h0 + (r - tt * heads)) * D + c * 4);
            const uint64_t scale = pack2(a.scale, a.scale);
            v.lo = mul2(v.lo, scale), v.hi = mul2(v.hi, scale);
        }
        *reinterpret_cast<Pairs*>(sm + L::q + 4 * (r * L::q_stride + c * 4)) = v;
    }
    __syncthreads();

    const int32_t key = lane & 15, hh = lane >> 4;  // the key of a page whose scores end here, with rows hh RL + i
    // products: keys key & ~3 .., RT rows from qrow, the ds-th of DS parts of the columns
    constexpr int RT = R == 4 ? 4 : R / 2, DS = R == 4 ? 8 : 4;
    const int32_t qrow = R == 4 ? 0 : hh * RL, ds = R == 4 ? (lane & 3) + 4 * hh : lane & 3;
    float* ps = reinterpret_cast<float*>(sm + L::p) + warp * 16 * L::p_stride;  // [key][row]: the weights
    float* corr = reinterpret_cast<float*>(sm + L::corr) + warp * R;  // [row]: what the outputs so far are scaled by
    float m[RL], l[RL];
    uint64_t acc[R / 2][E];  // outputs of rows 2 r, 2 r + 1
#pragma unroll
    for (int i = 0; i < RL; ++i) m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int r = 0; r < R / 2; ++r)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] = 0ull;
    for (int32_t i0 = first; i0 < end; i0 += kWarps) {
        const int32_t j0 = pl.page(i0) * kPageTokens, j = j0 + key;
        uint32_t seen = 0u;  // keys of the page that some row sees
        if (in_pool(block)) seen = 0xffffu;
        else if (lane == 0) raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
        cp_async_wait<F4 ? kRawPairs - 1 : 1>();
        __syncwarp();
        const uint8_t* raw_k = raw_pages + slot * 2 * fp4_page_bytes(D);
        if constexpr (F4) {
            if (seen) unpack(k_page, L::k_stride, raw_k, 1.f);
        }
        // ---- scores of (key, rows hh RL + i) ----
        float z[RL];
        if (seen) {
            uint64_t z2[4][RT];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < RT; ++i) z2[k][i] = 0ull;
#pragma unroll
            for (int c = 0; c < D / 4 / DS; ++c) {
                const int col = (c * DS + ds) * 4;
                Pairs kv[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) kv[k] = load4(k_page + ((key & 12) + k) * L::k_stride + col);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const Pairs qv = load4(reinterpret_cast<const float*>(sm + L::q) + (qrow + i) * L::q_stride + col);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        z2[k][i] = fma2(qv.lo, kv[k].lo, z2[k][i]);
                        z2[k][i] = fma2(qv.hi, kv[k].hi, z2[k][i]);
                    }
                }
            }
            // sum over the column parts: lanes that differ in bits 1, 0 (keys) and, R = 4, 4 (rows)
            float y[4][RT];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    float lo, hi;
                    unpack2(z2[k][i], lo, hi);
                    y[k][i] = lo + hi;
                }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const bool up = lane & 2, odd = lane & 1;
                const float s0 = up ? y[0][i] : y[2][i], s1 = up ? y[1][i] : y[3][i];
                const float k0 = (up ? y[2][i] : y[0][i]) + __shfl_xor_sync(0xffffffffu, s0, 2);
                const float k1 = (up ? y[3][i] : y[1][i]) + __shfl_xor_sync(0xffffffffu, s1, 2);
                y[0][i] = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
            }
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                z[i] = y[0][i];
                if constexpr (RT > RL)
                    z[i] = (hh ? y[0][i + RL] : y[0][i]) + __shfl_xor_sync(0xffffffffu, hh ? y[0][i] : y[0][i + RL], 16);
            }
        }
        __syncwarp();  // the K page has been read
        const int32_t block_after = block_of(i0 + (F4 ? kRawPairs : 2) * kWarps);
        if constexpr (!F4) fetch(k_cache, k_page, L::k_stride, i0 + kWarps, block_next);
        const bool whole = (j0 >= inner.a0 && j0 + kPageTokens <= inner.a1) || (j0 >= inner.b0 && j0 + kPageTokens <= inner.b1);
        if (seen) {
            if (a.score.cap > 0.f) {
#pragma unroll
                for (int i = 0; i < RL; ++i) z[i] = a.score.cap * tanhf(z[i] / a.score.cap);
            }
#pragma unroll
            for (int i = 0; i < RL; ++i) z[i] *= kLog2e;
            if (a.score.slopes) {
#pragma unroll
                for (int i = 0; i < RL; ++i) z[i] -= slopes[hh * RL + i] * static_cast<float>(abs(where[hh * RL + i] - j));
            }
            if (!whole) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < RL; ++i) {
                    const bool sees = spans[hh * RL + i].sees(j);
                    any |= sees;
                    if (!sees) z[i] = -INFINITY;
                }
                seen = __ballot_sync(0xffffffffu, any);
                seen = (seen | seen >> 16) & 0xffffu;
            }
        }
        bool rescale = false;
        if (seen) {
            // ---- weights against the rows' references: maxima of earlier pages, kept until one is
            // exceeded by more than kLag (the weights then stay below 2^kLag, and most pages rescale nothing)
            float mx[RL];
            bool grow = false;
#pragma unroll
            for (int i = 0; i < RL; ++i) mx[i] = z[i];
#pragma unroll
            for (int off = 8; off > 0; off >>= 1)
#pragma unroll
                for (int i = 0; i < RL; ++i) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], off));
#pragma unroll
            for (int i = 0; i < RL; ++i) grow |= mx[i] > m[i] + kLag;
            rescale = __any_sync(0xffffffffu, grow);
            if (rescale) {
#pragma unroll
                for (int i = 0; i < RL; ++i) {
                    const float up = fmaxf(mx[i], m[i]);
                    const float f = exp2_approx(m[i] - (up == -INFINITY ? 0.f : up));
                    l[i] *= f;
                    m[i] = up;
                    if (key == 0) corr[hh * RL + i] = f;
                }
            }
#pragma unroll
            for (int i = 0; i < RL; ++i)  // nothing finite yet: weights are 0, not NaN
                z[i] = exp2_approx(z[i] - (m[i] == -INFINITY ? 0.f : m[i]));
#pragma unroll
            for (int i = 0; i < RL; i += 2) {
                l[i] += z[i];
                l[i + 1] += z[i + 1];
                *reinterpret_cast<float2*>(ps + key * L::p_stride + hh * RL + i) = make_float2(z[i], z[i + 1]);
            }
        }
        if constexpr (!F4) cp_async_wait<1>();
        __syncwarp();
        if (seen) {
            if constexpr (F4) unpack(v_page, D, raw_k + fp4_page_bytes(D), a.v_scale);
            if (seen != 0xffffu) {  // keys that no row sees: their weights are 0, their V may be anything
                for (uint32_t w = ~seen & 0xffffu; w != 0u; w &= w - 1)
#pragma unroll
                    for (int e = 0; e < E; ++e) v_page[(__ffs(w) - 1) * D + lane * E + e] = T(0);
            }
            if (rescale) {
#pragma unroll
                for (int r = 0; r < R / 2; ++r) {
                    const uint64_t f = *reinterpret_cast<const uint64_t*>(corr + 2 * r);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[r][e] = mul2(acc[r][e], f);
                }
            }
            // ---- outputs: columns lane E .. of all rows (each lane reads what it zeroed itself) ----
#pragma unroll
            for (int k = 0; k < kPageTokens; ++k) {
                uint64_t vv[E];
                load_twice(v_page + k * D + lane * E, vv);
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const Pairs w = load4(ps + k * L::p_stride + r);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        acc[r / 2][e] = fma2(w.lo, vv[e], acc[r / 2][e]);
                        acc[r / 2 + 1][e] = fma2(w.hi, vv[e], acc[r / 2 + 1][e]);
                    }
                }
            }
        }
        __syncwarp();  // the V page and the weights have been read
        block = block_next;
        if constexpr (F4) {
            fetch_pair(slot, i0 + kRawPairs * kWarps, block_after);
            slot = slot + 1 == kRawPairs ? 0 : slot + 1;
            block_next = block_third;
            block_third = block_after;
        } else {
            fetch(v_cache, v_page, D, i0 + kWarps, block);
            block_next = block_after;
        }
    }

    // ---- the warps' parts meet -------------------------------
#pragma unroll
    for (int off = 8; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < RL; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
    if (key == 0)
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            jm[warp][hh * RL + i] = m[i];
            jl[warp][hh * RL + i] = l[i];
        }
    cp_async_wait<0>();
    __syncthreads();  // q, weights and pages are done with
    if (tid < R) {
        float M = -INFINITY, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, jm[w][tid]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_approx(jm[w][tid] - ref);  // a warp without keys: m = -inf, weight 0
            den = fmaf(jl[w][tid], f, den);
            jm[w][tid] = f;
        }
        jM[tid] = M;
        jden[tid] = den;
    }
    float* const joined = reinterpret_cast<float*>(sm);  // [kWarps][R][D]
#pragma unroll
    for (int i = 0; i < R; i += 2)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float x0, x1;
            unpack2(acc[i / 2][e], x0, x1);
            joined[(warp * R + i) * D + lane * E + e] = x0;
            joined[(warp * R + i + 1) * D + lane * E + e] = x1;
        }
    __syncthreads();
    const int32_t cta = blockIdx.x * gridDim.y + blockIdx.y;  // among those of one partition
    for (int32_t i = tid; i < n_rows * D; i += kThreads) {
        const int32_t r = i / D, d = i - r * D;
        float num = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) num = fmaf(joined[(w * R + r) * D + d], jm[w][r], num);
        const float o = jden[r] == 0.f ? 0.f : num / jden[r];
        const int32_t tt = r / heads;
        const int64_t head = static_cast<int64_t>(row0 + tt) * a.num_q_heads + h0 + (r - tt * heads);
        if (parts <= 1) {
            out[head * D + d] = narrow<T>(o);
        } else {
            const int64_t slot = (static_cast<int64_t>(cta) * R + r) * a.num_parts + part;
            __stcg(a.ws_o + slot * D + d, o);
            if (d == 0) __stcg(reinterpret_cast<float2*>(a.ws_ml) + slot, make_float2(jM[r], jden[r]));
        }
    }
    if (parts <= 1) return;
    // ---- several partitions: the last CTA to arrive merges them -----------------------------------
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        int32_t* c = a.counter + cta;
        last_part = atomicAdd(c, 1) == parts - 1;
        if (last_part) *c = 0;  // ready for the next call
        __threadfence();
    }
    __syncthreads();
    if (!last_part) return;
    // the partitions' (max, sum) of every row, then their weights, in shared memory: [part][row]
    float2* const w = reinterpret_cast<float2*>(sm);
    const int64_t slot0 = static_cast<int64_t>(cta) * R * a.num_parts;
    for (int32_t i = tid; i < parts * R; i += kThreads) {
        const int32_t p = i / R, r = i - p * R;
        if (r < n_rows) w[i] = __ldcg(reinterpret_cast<const float2*>(a.ws_ml) + slot0 + r * a.num_parts + p);
    }
    __syncthreads();
    if (tid < n_rows) {
        float M = -INFINITY, den = 0.f;
        for (int32_t p = 0; p < parts; ++p) M = fmaxf(M, w[p * R + tid].x);
        const float ref = M == -INFINITY ? 0.f : M;
        for (int32_t p = 0; p < parts; ++p) {
            const float2 v = w[p * R + tid];
            const float f = v.y * exp2_approx(v.x - ref);
            den += f;
            w[p * R + tid].x = f;
        }
        jden[tid] = den == 0.f ? 0.f : 1.f / den;
    }
    __syncthreads();
    for (int32_t i = tid; i < n_rows * (D / 4); i += kThreads) {
        const int32_t r = i / (D / 4), c = i - r * (D / 4);
        const float4* o = reinterpret_cast<const float4*>(a.ws_o + (slot0 + r * a.num_parts) * D) + c;
        float4 acc4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int32_t p = 0; p < parts; ++p) {
            const float4 v = __ldcg(o + p * (D / 4));
            const float f = w[p * R + r].x;
            acc4.x = fmaf(f, v.x, acc4.x), acc4.y = fmaf(f, v.y, acc4.y);
            acc4.z = fmaf(f, v.z, acc4.z), acc4.w = fmaf(f, v.w, acc4.w);
        }
        const int32_t tt = r / heads;
        T* to = out + (static_cast<int64_t>(row0 + tt) * a.num_q_heads + h0 + (r - tt * heads)) * D + c * 4;
        const float inv = jden[r];
        to[0] = narrow<T>(acc4.x * inv), to[1] = narrow<T>(acc4.y * inv);
        to[2] = narrow<T>(acc4.z * inv), to[3] = narrow<T>(acc4.w * inv);
    }
}

template <typename T, int D, int R, int kWarps, bool F4>
cudaError_t launch_rows(void* out, const void* q, const void* k, const void* v, const SimtArgs& a, dim3 grid,
                        cudaStream_t stream) {
    constexpr int bytes = Smem<T, D, R, kWarps, F4>::bytes;
    if (bytes > 40960) {  // with the static part, beyond what every kernel may use
        const cudaError_t e = allow_smem<scored_simt_kernel<T, D, R, kWarps, F4>>(bytes);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_simt_kernel<T, D, R, kWarps, F4>, static_cast<T*>(out), static_cast<const T*>(q),
                              static_cast<const T*>(k), static_cast<const T*>(v), a);
}

template <typename T, int D, bool F4>
cudaError_t launch_impl(void* out, const void* q, const void* k, const void* v, SimtArgs& a, const ScoredSimtPlan& p,
                        void* workspace, cudaStream_t stream) {
    a.head_chunks = p.head_chunks;
    a.tokens = p.tokens;
    a.groups = p.groups;
    a.part_pages = p.part_pages;
    a.num_parts = p.num_parts;
    if (p.num_parts > 1) {
        a.counter = static_cast<int32_t*>(workspace);
        a.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + kScoredCounterBytes);
        a.ws_ml = a.ws_o + static_cast<size_t>(p.grid_x) * a.num_kv_heads * p.head_chunks * p.rows * p.num_parts * D;
    }
    const dim3 grid(p.grid_x, a.num_kv_heads * a.head_chunks, a.num_parts);
    if (p.rows == kFewRows) return launch_rows<T, D, kFewRows, 8, F4>(out, q, k, v, a, grid, stream);
    return p.warps == 8 ? launch_rows<T, D, kManyRows, 8, F4>(out, q, k, v, a, grid, stream)
                        : launch_rows<T, D, kManyRows, 4, F4>(out, q, k, v, a, grid, stream);
}

template <bool F4, typename A>
cudaError_t launch_any(const A& d, SimtArgs& a, const ScoredSimtPlan& p, void* workspace, cudaStream_t stream) {
    auto run = [&](auto type, auto dim) {
        return launch_impl<decltype(type), decltype(dim)::value, F4>(d.out, d.q, d.k_cache, d.v_cache, a, p, workspace, stream);
    };
    using D128 = std::integral_constant<int, 128>;
    using D64 = std::integral_constant<int, 64>;
    if (d.dtype == PA_F32) return d.head_dim == 128 ? run(float(), D128()) : run(float(), D64());
    return d.head_dim == 128 ? run(uint16_t(), D128()) : run(uint16_t(), D64());
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
    a.scale = d.scale;
    a.score = score;
    a.err = d.err;
    return a;
}

}  // namespace

int32_t scored_simt_head_chunks(int32_t group) {
    return group <= kFewRows ? 1 : (group + kManyRows - 1) / kManyRows;
}

// max_chunk 0: decode. Partitions so that the CTAs fill the SMs once (two CTAs of 4 rows, one of 16 on an SM),
// of at least kMinPages pages each. Measured, 24 sequences of up to 777 keys, 4 kv heads of 64 in fp32: 9.1 us with 32 or 64 pages,
// 10.7 with 8 or 16.
ScoredSimtPlan plan_scored_simt(int32_t S, int32_t max_chunk, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_seq_len,
                                int num_sms) {
    constexpr int64_t kMinPages = 32;
    ScoredSimtPlan p{};
    const int32_t G = Hq / Hkv;
    // (24 sequences, 12 q / 4 kv heads of 64 in fp32: 5.8 us with 4 rows, 8.0 with 16; chunks of 17 to 96 rows, 8 q / 2
    // kv heads: 17.1 with 4, 15.7 with 16)
    p.rows = static_cast<int64_t>(G) * (max_chunk > 0 ? max_chunk : 1) <= kFewRows ? kFewRows : kManyRows;
    p.head_chunks = (G + p.rows - 1) / p.rows;
    p.tokens = G < p.rows ? p.rows / G : 1;
    p.groups = max_chunk > 0 ? (max_chunk - 1) / p.tokens + 1 : 1;
    p.grid_x = S * p.groups;
    const int64_t ctas = static_cast<int64_t>(p.grid_x) * Hkv * p.head_chunks, pages = max_seq_len / kPageTokens + 2;
    int64_t parts = ctas > 0 ? (p.rows == kFewRows ? 2LL : 1LL) * num_sms / ctas : 1;
    parts = max(min(min(parts, pages / kMinPages), static_cast<int64_t>(kMaxParts)), static_cast<int64_t>(1));
    p.part_pages = static_cast<int32_t>((pages + parts - 1) / parts);
    p.num_parts = static_cast<int32_t>((pages + p.part_pages - 1) / p.part_pages);
    // A CTA of 8 warps and 16 rows has an SM to itself; of 4 warps two fit, and hide each other's start and end.
    // Measured in fp32: 4 x 1024 rows, 16 q / 4 kv heads of 128: 659 us with 8, 541 with 4; 192 CTAs, 12 pages a
    // warp: 24.9 and 20.1; 192 CTAs of which 114 have rows (chunks of 17 to 96): 15.7 and 22.4.
    p.warps = p.rows == kFewRows || ctas * p.num_parts <= 2 * num_sms ? 8 : 4;
    // room for any number of rows: split grids have 2 num_sms CTAs at most
    if (pages >= 2 * kMinPages)
        p.workspace_bytes = kScoredCounterBytes + static_cast<size_t>(2 * num_sms) * kManyRows * (D + 2) * sizeof(float);
    return p;
}

cudaError_t launch_scored_decode_simt(const DecodeArgs& d, const ScoreArgs& score, const ScoredSimtPlan& plan,
                                      cudaStream_t stream) {
    SimtArgs a = common_args(d, score);
    return launch_any<false>(d, a, plan, d.workspace, stream);
}

cudaError_t launch_scored_prefill_simt(const PrefillArgs& p, const ScoreArgs& score, const ScoredSimtPlan& plan,
                                       void* workspace, cudaStream_t stream) {
    SimtArgs a = common_args(p, score);
    a.query_start_loc = p.query_start_loc;
    a.max_chunk = p.max_chunk_len;
    return launch_any<false>(p, a, plan, workspace, stream);
}

cudaError_t launch_fp4_decode_simt(const DecodeArgs& d, float v_scale, const ScoredSimtPlan& plan, cudaStream_t stream) {
    SimtArgs a = common_args(d, ScoreArgs{});
    a.v_scale = v_scale;
    return launch_any<true>(d, a, plan, d.workspace, stream);
}

cudaError_t launch_fp4_prefill_simt(const PrefillArgs& p, float v_scale, const ScoredSimtPlan& plan, void* workspace,
                                    cudaStream_t stream) {
    SimtArgs a = common_args(p, ScoreArgs{});
    a.v_scale = v_scale;
    a.query_start_loc = p.query_start_loc;
    a.max_chunk = p.max_chunk_len;
    return launch_any<true>(p, a, plan, workspace, stream);
}

}  // namespace pa
