// Scores of the scored attention kernels: the descriptor as the kernels take it, and which keys a
// query row sees.
//
//   z = scale q.k;  z = cap tanh(z / cap);  z -= slope |p - j|
//   visible(j) = j < L and j >= key_start and (j < prefix or (j <= p and j > p - window)),
//                causal prefix: (j <= p and (j < prefix or j > p - window))
//
// The visible keys are two spans without a common key, [a0, a1) (the prefix part) and [b0, b1)
// (the window part), so a kernel walks only their pages.
#pragma once

#include <atomic>
#include <mutex>

#include "pa_device.cuh"

namespace pa {

// Lets a kernel use this much dynamic shared memory on the current device. The runtime is asked once
// per kernel, device and larger size, not once per launch (it takes part of a microsecond).
template <auto* Kernel>
cudaError_t allow_smem(int bytes) {
    constexpr int kDevices = 64;
    static std::atomic<int> allowed[kDevices];
    static std::mutex mutex;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (allowed[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mutex);
    if (allowed[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) allowed[dev].store(bytes, std::memory_order_release);
    return e;
}

__device__ __forceinline__ float exp2_approx(float x) {  // relative error about 2^-22; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed fp32 pairs: one instruction for two elements.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Capped scores, cap log2(e) tanh(u) with u = s scale / cap, from y = 2 u log2(e) = s two_k and c1 = scale log2(e).
// Two forms, of which neither serves every cap: near u = 0 the identity cancels (an error of 2^-21 cap,
// whatever the score), and far from it a polynomial does not hold.
//   |u| <= 0.6  s c1 (1 + y^2 P(y^2)): tanh(u) / u fitted in its relative error (6.5e-8, minimax over a fine grid by
//               linear programming, the leading 1 held), so that a cap far above the scores leaves them alone;
//   beyond      cap (1 - 2 / (1 + 2^y)): relative error below 2^-20, and an absolute one below 2^-20 cap anywhere.
constexpr float kTanhP0 = -0.0400365926f, kTanhP1 = 0.00192027225f, kTanhP2 = -9.02627071e-05f, kTanhP3 = 3.21615289e-06f;
constexpr float kTanhY2 = 2.997171f;       // y^2 up to which the polynomial holds, (1.2 log2 e)^2
constexpr float kLargestCapL2 = 1.6e38f;  // cap log2(e) is held where twice of it is finite
__device__ __forceinline__ float capped_near(float s, float y2, float c1) {
    const float t = s * c1;
    return fmaf(t * y2, fmaf(y2, fmaf(y2, fmaf(y2, kTanhP3, kTanhP2), kTanhP1), kTanhP0), t);
}
__device__ __forceinline__ float capped_far(float y, float cap_l2) {
    return fmaf(-2.f * cap_l2, rcp_approx(1.f + exp2_approx(y)), cap_l2);
}

struct KeySpans {
    int32_t a0, a1, b0, b1;
    __device__ __forceinline__ bool sees(int32_t j) const { return (j >= a0 && j < a1) || (j >= b0 && j < b1); }
};

// Spans of a row at position p of a sequence with len keys (p < len). A row inside a causal prefix sees the prefix up
// to itself, and its window part is empty. Over the rows of a sequence, prefix parts lie before window parts.
__device__ __forceinline__ KeySpans key_spans(int32_t len, int32_t p, int32_t key_start, int32_t prefix,
                                              int32_t window, bool causal) {
    KeySpans s;
    const int32_t start = max(key_start, 0);
    s.a0 = start;
    s.a1 = max(start, min(prefix, causal ? p + 1 : len));
    s.b0 = max(start, window > 0 ? p + 1 - window : 0);
    if (s.a1 > s.a0) s.b0 = max(s.b0, s.a1);
    s.b1 = max(s.b0, p + 1);
    return s;
}

// The 16-token pages that hold the spans' keys, in ascending order: n_a pages from first_a, then
// the rest from first_b (a page that both spans touch is counted once).
struct PageList {
    int32_t first_a, n_a, first_b, n;
    __device__ __forceinline__ int32_t page(int32_t i) const { return i < n_a ? first_a + i : first_b + (i - n_a); }
};

__device__ __forceinline__ PageList page_list(const KeySpans& s) {
    PageList l;
    l.first_a = s.a0 / kPageTokens;
    l.n_a = s.a1 > s.a0 ? (s.a1 + kPageTokens - 1) / kPageTokens - l.first_a : 0;
    l.first_b = s.b0 / kPageTokens;
    if (l.n_a > 0) l.first_b = max(l.first_b, l.first_a + l.n_a);
    const int32_t end_b = s.b1 > s.b0 ? (s.b1 + kPageTokens - 1) / kPageTokens : 0;
    l.n = l.n_a + max(0, end_b - l.first_b);
    return l;
}

}  // namespace pa
