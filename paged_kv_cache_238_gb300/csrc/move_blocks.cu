// move_blocks: copies of pages between physical blocks in every layer's pools, and the rewrite of
// block tables to follow them. Pure data movement, bound by HBM: each moved byte is read and
// written once.
//
// Grid: x = pair, or a few of them where blocks are small (the last rows of CTAs after the pairs rewrite
// the table), y = pool, z = share of a block. A block of all kv heads is contiguous, so a whole-block copy is one run of 16-byte chunks; with
// `tokens` the copy is a run per head. A thread sends for eight chunks before it stores them, and blocks
// go to several CTAs where there are few: one chunk at a time and a CTA per block took 36 us for 6
// half-full blocks of 256 KB in 64 pools, this 14.6 (6.6 TB/s read and written); 960 blocks of 32 KB in 64
// pools: 565 us (7.1 TB/s, a plain copy of the same bytes 593). A table entry finds its pair by binary
// search over the ascending src ids.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 2432;   // copying CTAs below which a block is shared among several
constexpr int kInFlight = 8;  // 16-byte loads a thread issues before their stores

struct Pools {
    int4* p[kMoveMaxPools];
};

__device__ __forceinline__ bool in_pool(int32_t id, const MoveArgs& a) { return id >= 0 && id < a.num_blocks; }
__device__ __forceinline__ bool copied(int2 pr, const MoveArgs& a) {
    return in_pool(pr.x, a) && in_pool(pr.y, a) && pr.x != pr.y;
}
__device__ __forceinline__ void check_pair(const int2* pairs, int32_t i, const MoveArgs& a) {
    const int2 pr = __ldg(pairs + i);
    if (!in_pool(pr.x, a) || !in_pool(pr.y, a)) raise_error(a.err, PA_DEVERR_BLOCK_RANGE);
    if (a.block_table != nullptr && i > 0 && __ldg(&pairs[i - 1].x) >= pr.x) raise_error(a.err, PA_DEVERR_PAIR_ORDER);
}

__global__ void __launch_bounds__(kThreads) move_blocks_kernel(const __grid_constant__ Pools pools,
                                                               const __grid_constant__ MoveArgs a) {
    const int2* pairs = reinterpret_cast<const int2*>(a.pairs);
    const int32_t copying = (a.num_pairs + a.group - 1) / a.group;  // CTAs in x that copy
    if (static_cast<int32_t>(blockIdx.x) >= copying) {  // block-table rewrite
        if (blockIdx.y != 0 || blockIdx.z != 0) return;
        const int32_t ctas = static_cast<int32_t>(gridDim.x) - copying;
        const int64_t entries = static_cast<int64_t>(a.num_seqs) * a.max_blocks;
        for (int64_t i = (static_cast<int64_t>(blockIdx.x) - copying) * kThreads + threadIdx.x; i < entries;
             i += static_cast<int64_t>(ctas) * kThreads) {
            const int32_t s = static_cast<int32_t>(i / a.max_blocks), col = static_cast<int32_t>(i - static_cast<int64_t>(s) * a.max_blocks);
            if (static_cast<int64_t>(col) * a.block_size >= __ldg(a.seq_lens + s)) continue;
            const int32_t id = a.block_table[i];
            int32_t lo = 0, hi = a.num_pairs;
            while (lo < hi) {
                const int32_t mid = (lo + hi) >> 1;
                if (__ldg(&pairs[mid].x) < id) lo = mid + 1; else hi = mid;
            }
            if (lo < a.num_pairs && __ldg(&pairs[lo].x) == id) {
                const int32_t to = __ldg(&pairs[lo].y);
                if (to >= 0 && to < a.num_blocks) a.block_table[i] = to;
            }
        }
        return;
    }
    int4* pool = pools.p[blockIdx.y];  // null: a call that rewrites tables only
    const int32_t head = a.tokens ? a.block_size * a.row_chunks : a.block_chunks;  // chunks of a run, at most
    if (a.group > 1) {  // small blocks: several pairs a CTA, chunk i of which is chunk i % block_chunks of a pair
        const int32_t first = blockIdx.x * a.group, n_pairs = min(a.group, a.num_pairs - first);
        if (blockIdx.y == 0 && static_cast<int32_t>(threadIdx.x) < n_pairs) check_pair(pairs, first + threadIdx.x, a);
        if (pool == nullptr) return;
        const int32_t end = n_pairs * a.block_chunks;
        int4 v[kInFlight];
        int4* to[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int32_t i = threadIdx.x + k * kThreads, p = i / a.block_chunks, c = i - p * a.block_chunks;
            to[k] = nullptr;
            if (i >= end) continue;
            const int2 pr = __ldg(pairs + first + p);
            if (!copied(pr, a)) continue;
            if (a.tokens && c % head >= min(max(__ldg(a.tokens + first + p), 0), a.block_size) * a.row_chunks) continue;
            v[k] = pool[static_cast<int64_t>(pr.x) * a.block_chunks + c];
            to[k] = pool + static_cast<int64_t>(pr.y) * a.block_chunks + c;
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k)
            if (to[k]) *to[k] = v[k];
        return;
    }
    const int2 pr = __ldg(pairs + blockIdx.x);
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) check_pair(pairs, blockIdx.x, a);
    if (pool == nullptr || !copied(pr, a)) return;
    const int4* src = pool + static_cast<int64_t>(pr.x) * a.block_chunks;
    int4* dst = pool + static_cast<int64_t>(pr.y) * a.block_chunks;
    // runs of n chunks, one per head (whole blocks: one run); this CTA's share of all of them
    const int32_t n = a.tokens ? min(max(__ldg(a.tokens + blockIdx.x), 0), a.block_size) * a.row_chunks : head;
    const int32_t total = a.block_chunks / head * n;
    const int32_t share = (total + static_cast<int32_t>(gridDim.z) - 1) / static_cast<int32_t>(gridDim.z);
    const int32_t end = min(total, static_cast<int32_t>(blockIdx.z + 1) * share);
    int32_t c = static_cast<int32_t>(blockIdx.z) * share + threadIdx.x;
    for (; c < end; c += kInFlight * kThreads) {
        int4 v[kInFlight];
        int32_t at[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int32_t i = c + k * kThreads, h = i / n;
            at[k] = h * head + (i - h * n);
            if (i < end) v[k] = src[at[k]];
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k)
            if (c + k * kThreads < end) dst[at[k]] = v[k];
    }
}

}  // namespace

cudaError_t launch_move_blocks(const MoveArgs& a, void* const* pools, int32_t num_pools, cudaStream_t stream) {
    for (int32_t p0 = 0; p0 < num_pools || p0 == 0; p0 += kMoveMaxPools) {
        Pools ps{};
        const int32_t n = num_pools - p0 < kMoveMaxPools ? num_pools - p0 : kMoveMaxPools;
        for (int32_t i = 0; i < n; ++i) ps.p[i] = static_cast<int4*>(pools[p0 + i]);
        MoveArgs m = a;
        if (p0 > 0) m.block_table = nullptr;  // once
        const int64_t entries = m.block_table ? static_cast<int64_t>(m.num_seqs) * m.max_blocks : 0;
        const int64_t table_ctas = (entries + kThreads - 1) / kThreads < 512 ? (entries + kThreads - 1) / kThreads : 512;
        if (m.num_pairs + table_ctas == 0) return cudaSuccess;
        // small blocks: as many pairs a CTA as give its threads kInFlight chunks (575 blocks of 2 KB in 44 pools: 15.3 us,
        // 61 with a CTA per block)
        m.group = kThreads * kInFlight / m.block_chunks;
        if (m.group < 1) m.group = 1;
        const int64_t copying = (static_cast<int64_t>(m.num_pairs) + m.group - 1) / m.group;
        // few blocks: each goes to several CTAs, of at least kInFlight chunks a thread
        const int64_t whole = static_cast<int64_t>(m.num_pairs) * n, most = m.block_chunks / (kThreads * kInFlight);
        int64_t shares = whole > 0 ? (kCtas + whole - 1) / whole : 1;
        if (shares > most) shares = most;
        const dim3 grid(static_cast<unsigned>(copying + table_ctas), n > 0 ? n : 1, shares > 1 ? static_cast<unsigned>(shares) : 1);
        move_blocks_kernel<<<grid, kThreads, 0, stream>>>(ps, m);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace pa
