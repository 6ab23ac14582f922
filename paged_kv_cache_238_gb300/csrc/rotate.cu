// New tokens on their way into the paged pool: q and k rotated by their positions, k and v written to
// their slots, in the pool's type or in 4 bits (fp4.cuh); and rows of a 4-bit pool read back.
//
// Rotation, with c, s the table's row at the token's position and R = rotary_dim:
//   halves       (x_i, x_(i + R/2))   -> (x_i c_i - x_(i + R/2) s_i,  x_(i + R/2) c_i + x_i s_i),  i < R / 2
//   interleaved  (x_2i, x_(2i + 1))   -> the same
// dims from R on stay. bf16 and fp32 results are rounded once. A k that goes into 4 bits is computed to
// about 45 bits first (each product as a rounded product and its error, summed with theirs), so that its
// rounding to fp32 and on to the call's type, and with it the code, is the exact result's.
//
// A thread owns 16 dims of a token's rows, as two chunks of 8 that rotate into one another (halves: chunk p and
// chunk R/16 + p), and walks up to 8 rows of one kind (q, k or v heads) with the table's 16 values in registers. In 4
// bits it owns the 16 dims of a group instead, and reads what they rotate with (again, from L1). A grid row per kind keeps
// a warp's threads on one path: with the kinds of a token side by side the pool's own type took 39 us and 4 bits 71.
//
// Bound: HBM in the pool's own type (8448 tokens, 32 q / 8 kv heads of 128, bf16: 34.4 us, 6.2 TB/s, 91 % of the measured copy
// rate; loads row by row 36.2); in 4 bits the latency of a group's loads at 24 warps an SM and its arithmetic, about 20 instructions an
// element of k and 7 of v (37.5 us of 48.5 with the read of the pool; with a division per element 58).
// 64 tokens: 2.2 us, in 4 bits and read back 4.5. fp32, 8448 tokens: 66.1 us; into 4 bits 61.9 (5.8 TB/s). Rows read back: 11.0 us
// (4.2 TB/s), as fp32 19.6 (4.2): loads of 4 bytes of codes and 1 of scales a thread, waited for at 42 warps an SM.
#include <type_traits>

#include "fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 128;

// Eight consecutive elements as they lie in memory, and as floats.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void load_plain(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        v = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void load_plain(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

template <typename T>
__device__ __forceinline__ float rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ float rounded<uint16_t>(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// a c + b s to about 45 bits, rounded once; what is not finite is the plain sum (its error terms are NaN).
__device__ __forceinline__ float turn_exact(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p), r = __fmul_rn(b, s), re = __fmaf_rn(b, s, -r);
    const float sum = __fadd_rn(p, r), z = __fsub_rn(sum, p);
    const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, z)), __fsub_rn(r, z));  // p + r = sum + e
    const float full = __fadd_rn(sum, __fadd_rn(e, __fadd_rn(pe, re)));
    return full == full ? full : sum;
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ void load4(const float* p, float* x) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
}

// The four pairs of a chunk.
template <typename T>
__device__ __forceinline__ void turn_pairs(Chunk<T>& v, const float* c, const float* s) {
    float x[8];
    v.get(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x0 = x[2 * i], x1 = x[2 * i + 1];
        x[2 * i] = fmaf(x0, c[i], -(x1 * s[i]));
        x[2 * i + 1] = fmaf(x1, c[i], x0 * s[i]);
    }
    v.put(x);
}

// Grid: y = kind (q, k, v), so that a warp's threads take one path; x = units of that kind (`per` heads of a token).
struct Shape {
    int32_t parts_log2;        // threads of a row: head_dim / 16
    int32_t q_units, k_units;  // units of a token
    int32_t q_per, k_per;
};

// Six CTAs an SM (80 registers) against five (96): the prompt 36.2 and 37.4 us; in 4 bits, where halves spill for it (76 bytes, fp32
// 148), 47.7 and 48.1.
template <typename T, bool F4, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 6) rotate_kernel(const __grid_constant__ RotateArgs a,
                                                          const __grid_constant__ Shape g) {
    // the kernel before may produce the inputs, or read the pool
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int kind = 2 - blockIdx.y;  // v, k, q: the longest come first
    const int32_t parts = 1 << g.parts_log2, p = static_cast<int32_t>(threadIdx.x) & (parts - 1);
    const uint32_t unit = (blockIdx.x * kThreads + threadIdx.x) >> g.parts_log2;  // (tokens x heads x parts fit 31 bits)
    const uint32_t of_token = max(kind == 0 ? g.q_units : g.k_units, 1);
    const int32_t t = static_cast<int32_t>(unit / of_token), u = static_cast<int32_t>(unit - t * of_token);
    if (t >= a.num_tokens) return;  // (the grid is as wide as its widest kind)
    if (kind == 0 && a.num_q_heads == 0) return;
    const int32_t heads = kind == 0 ? a.num_q_heads : a.num_kv_heads, per = kind == 0 ? g.q_per : g.k_per;
    const int32_t h0 = u * per, h1 = min(heads, h0 + per), D = a.head_dim, R = a.rotary_dim;

    const int64_t pos = __ldg(a.positions + t);
    if (pos < 0 || pos >= a.num_positions) {  // the token is left out
        if (p == 0 && u == 0) raise_error(a.err, PA_DEVERR_POSITION);
        return;
    }
    int64_t slot = 0;
    if (kind != 0) {
        slot = __ldg(a.slot_mapping + t);
        if (slot < 0) return;  // padding
        if (slot >= static_cast<int64_t>(a.num_blocks) << a.bs_log2) {
            if (p == 0 && u == 0) raise_error(a.err, PA_DEVERR_SLOT_RANGE);
            return;
        }
    }
    const int64_t block = slot >> a.bs_log2;
    const int32_t at = static_cast<int32_t>(slot & ((1 << a.bs_log2) - 1));
    const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                   static_cast<int64_t>(t) * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
    const float* turn = a.cos_sin + pos * R;

    if (F4 && kind != 0) {
        // ---- 4 bits: dims 16 p .. of each row -----------------------------------------------------
        uint8_t* pool = static_cast<uint8_t*>(kind == 1 ? a.k_cache : a.v_cache);
        const float unscale = kind == 1 ? a.k_unscale : a.v_unscale;  // a power of two: the product is exact
        const bool turned = kind == 1 && 16 * p < R;
        // halves: chunk j of the group is chunk 2 p + j of the row; its angles and the chunk it turns with
        float c[2][8], s[2][8];
        int32_t with[2] = {0, 0};
        bool upper[2] = {false, false};
        if (turned) {
            if (INTERLEAVED) {
                load8(turn + 8 * p, c[0]);
                load8(turn + R / 2 + 8 * p, s[0]);
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int32_t ch = 2 * p + j;
                    upper[j] = ch >= R / 16;
                    with[j] = upper[j] ? ch - R / 16 : ch + R / 16;
                    const int32_t i = (upper[j] ? with[j] : ch) * 8;
                    load8(turn + i, c[j]);
                    load8(turn + R / 2 + i, s[j]);
                }
            }
        }
#pragma unroll 2
        for (int32_t h = h0; h < h1; ++h) {
            const T* row = src + static_cast<int64_t>(h) * D;
            Chunk<T> own[2], other[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) own[j].load(row + 16 * p + 8 * j);
            if (turned && !INTERLEAVED) {
#pragma unroll
                for (int j = 0; j < 2; ++j) other[j].load(row + 8 * with[j]);
            }
            float y[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x[8];
                own[j].get(x);
                if (turned && INTERLEAVED) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float x0 = x[i], x1 = x[i + 1], ci = c[0][4 * j + i / 2], si = s[0][4 * j + i / 2];
                        x[i] = rounded<T>(turn_exact(x0, ci, -x1, si));
                        x[i + 1] = rounded<T>(turn_exact(x1, ci, x0, si));
                    }
                } else if (turned) {
                    float o[8];
                    other[j].get(o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = rounded<T>(turn_exact(x[i], c[j][i], upper[j] ? o[i] : -o[i], s[j][i]));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) y[8 * j + i] = x[i] * unscale;
            }
            uint32_t scale;
            const uint2 codes = fp4_pack16(y, &scale);
            uint8_t* page = pool + fp4_page_at(static_cast<int32_t>(block), a.num_kv_heads, h, a.bs_log2 - 4, at >> 4, D);
            *reinterpret_cast<uint2*>(page + (at & 15) * (D / 2) + 8 * p) = codes;
            page[fp4_scales_at(D) + (at & 15) * (D / 16) + p] = static_cast<uint8_t>(scale);
        }
        return;
    }

    // ---- the pool's own type, and q: two chunks of each row, the lanes' side by side -----------------------
    // halves: chunk p with chunk R / 16 + p; else p with p + parts; what lies behind a part that turns, in order
    const bool halves = !INTERLEAVED && kind != 2 && p < R / 16, behind = !INTERLEAVED && kind != 2 && !halves;
    const int32_t c0 = behind ? 2 * p : p, c1 = behind ? 2 * p + 1 : p + (halves ? R / 16 : parts);
    const bool turned0 = halves || (INTERLEAVED && kind != 2 && 8 * c0 < R), turned1 = halves || (INTERLEAVED && kind != 2 && 8 * c1 < R);
    float c[8], s[8];  // halves: of the pairs; interleaved: four of each chunk
    if (halves) {
        load8(turn + 8 * p, c);
        load8(turn + R / 2 + 8 * p, s);
    } else {
        if (turned0) {
            load4(turn + 4 * c0, c);
            load4(turn + R / 2 + 4 * c0, s);
        }
        if (turned1) {
            load4(turn + 4 * c1, c + 4);
            load4(turn + R / 2 + 4 * c1, s + 4);
        }
    }
    T* dst;
    int64_t step;  // between heads
    if (kind == 0) {
        dst = static_cast<T*>(a.q_out) + static_cast<int64_t>(t) * a.q_out_stride;
        step = D;
    } else {
        dst = static_cast<T*>(kind == 1 ? a.k_cache : a.v_cache) + (((block * a.num_kv_heads) << a.bs_log2) + at) * D;
        step = static_cast<int64_t>(D) << a.bs_log2;
    }
    // several rows' loads before their stores (fp32: two, whose 32 registers four in bf16 take as well): q_out may be q, so
    // these loads are ordinary ones, which the compiler does not move above the stores of rows before
    constexpr int kAhead = 8 / sizeof(T);
    for (int32_t h = h0; h < h1; h += kAhead) {
        Chunk<T> lo[kAhead], hi[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (h + x >= h1) continue;
            const T* row = src + static_cast<int64_t>(h + x) * D;
            lo[x].load_plain(row + 8 * c0);
            hi[x].load_plain(row + 8 * c1);
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (h + x >= h1) continue;
            if (halves) {
                float y0[8], y1[8];
                lo[x].get(y0);
                hi[x].get(y1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x0 = y0[i], x1 = y1[i];
                    y0[i] = fmaf(x0, c[i], -(x1 * s[i]));
                    y1[i] = fmaf(x1, c[i], x0 * s[i]);
                }
                lo[x].put(y0);
                hi[x].put(y1);
            } else if (INTERLEAVED) {
                if (turned0) turn_pairs(lo[x], c, s);
                if (turned1) turn_pairs(hi[x], c + 4, s + 4);
            }
            lo[x].store(dst + (h + x) * step + 8 * c0);
            hi[x].store(dst + (h + x) * step + 8 * c1);
        }
    }
}

template <typename T, bool F4, bool INTERLEAVED>
cudaError_t launch_rotate(const RotateArgs& a, const Shape& g, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t units = static_cast<int64_t>(a.num_tokens) * (g.q_units > g.k_units ? g.q_units : g.k_units);
    cfg.gridDim = dim3(static_cast<unsigned>(((units << g.parts_log2) + kThreads - 1) / kThreads), 3);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotate_kernel<T, F4, INTERLEAVED>, a, g);
}

// ---- rows of a 4-bit pool by slot, as values: a thread reads 8 dims of K and of V ---------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads) gather_fp4_kernel(const __grid_constant__ GatherFp4Args a, uint32_t chunks_log2,
                                                              uint32_t items) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= items) return;
    const uint32_t row = i >> chunks_log2, n = row / static_cast<uint32_t>(a.num_kv_heads);  // (slot, kv head)
    const int32_t c = static_cast<int32_t>(i & ((1u << chunks_log2) - 1)), h = static_cast<int32_t>(row - n * a.num_kv_heads);
    const int32_t D = a.head_dim;
    const int64_t slot = __ldg(a.slots + n);
    const bool in = slot >= 0 && slot < static_cast<int64_t>(a.num_blocks) << a.bs_log2;
    if (!in && slot >= 0 && c == 0 && h == 0) raise_error(a.err, PA_DEVERR_SLOT_RANGE);
    uint32_t codes[2] = {0u, 0u}, scale[2] = {0u, 0u};
    if (in) {
        const int32_t at = static_cast<int32_t>(slot & ((1 << a.bs_log2) - 1));
        const int64_t page = fp4_page_at(static_cast<int32_t>(slot >> a.bs_log2), a.num_kv_heads, h, a.bs_log2 - 4, at >> 4, D);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t* p = static_cast<const uint8_t*>(kv ? a.v_cache : a.k_cache) + page;
            codes[kv] = __ldg(reinterpret_cast<const uint32_t*>(p + (at & 15) * (D / 2)) + c);
            scale[kv] = __ldg(p + fp4_scales_at(D) + (at & 15) * (D / 16) + c / 2);
        }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float s = halves_to_floats(e4m3x2_halves(static_cast<uint16_t>(scale[kv]))).x * (kv ? a.v_scale : a.k_scale);
        uint32_t hv[4];
        fp4_halves(codes[kv], hv);
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = halves_to_floats(hv[e]);
            x[2 * e] = f.x * s;
            x[2 * e + 1] = f.y * s;
        }
        Chunk<T> o;
        o.put(x);
        o.store(static_cast<T*>(kv ? a.v_out : a.k_out) + static_cast<int64_t>(row) * D + 8 * c);
    }
}

template <typename T>
cudaError_t launch_gather(const GatherFp4Args& a, cudaStream_t stream) {
    const uint32_t chunks_log2 = a.head_dim == 128 ? 4 : 3;
    const uint32_t items = static_cast<uint32_t>(a.num_slots) * a.num_kv_heads << chunks_log2;  // (fit 31 bits)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((items + kThreads - 1) / kThreads);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gather_fp4_kernel<T>, a, chunks_log2, items);
}

}  // namespace

cudaError_t launch_rotate_and_cache(const RotateArgs& a, int num_sms, cudaStream_t stream) {
    // Heads of a unit: several, which share the angles and keep more loads in flight, where 16 CTAs an SM are left.
    // 8448 tokens, 32 q / 8 kv heads of 128: q by 8 37.4 us in all, by 4 38.8, by 2 46.4; k, v into 4 bits by 8 47.9 us (with
    // the read of the pool), by 4 51.2, by 1 58.3. 64 tokens into 4 bits by 1 4.2 us, by 4 6.7.
    auto per = [&](int32_t heads, bool packs) {
        const int64_t ctas = static_cast<int64_t>(a.num_tokens) * heads * (a.head_dim / 16) / kThreads;
        return ctas <= 16LL * num_sms ? 1 : packs || ctas > 96LL * num_sms ? 8 : 4;
    };
    Shape g;
    g.parts_log2 = a.head_dim == 128 ? 3 : 2;
    g.q_per = per(a.num_q_heads, false), g.k_per = per(a.num_kv_heads, a.fp4);
    g.q_units = (a.num_q_heads + g.q_per - 1) / g.q_per;
    g.k_units = (a.num_kv_heads + g.k_per - 1) / g.k_per;
    auto go = [&](auto type, auto f4) {
        using T = decltype(type);
        return a.interleaved ? launch_rotate<T, decltype(f4)::value, true>(a, g, stream)
                             : launch_rotate<T, decltype(f4)::value, false>(a, g, stream);
    };
    if (a.fp4) return a.dtype == PA_F32 ? go(float(), std::true_type()) : go(uint16_t(), std::true_type());
    return a.dtype == PA_F32 ? go(float(), std::false_type()) : go(uint16_t(), std::false_type());
}

cudaError_t launch_gather_fp4(const GatherFp4Args& a, cudaStream_t stream) {
    return a.dtype == PA_F32 ? launch_gather<float>(a, stream) : launch_gather<uint16_t>(a, stream);
}

}  // namespace pa
