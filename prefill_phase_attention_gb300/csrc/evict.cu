// evict.cu -- eviction from a KV cache by accumulated attention weight.
//
// Per (sequence, KV head) of a cache of L tokens, L > budget: the first
// `sinks` and the last `recent` tokens stay, and of the tokens between them
// the m = budget - sinks - recent with the largest weight (ties: the lowest
// position first; NaN ranks above everything).  The kept rows of K and V move
// to positions 0 .. budget - 1 in their old order, in place.  L <= budget keeps
// every token.
//
// One launch, one cluster of 2, 4 or 8 CTAs per (sequence, head): each CTA
// moves one column part (64 bytes where the row has them) of K or of V, and
// together they choose the tokens:
//  - the m-th largest weight by a radix select, 8 bits of the weight's
//    order-preserving integer image per pass; up to kSoloTokens tokens every
//    CTA does it alone (a few thousand weights cost less than a cluster
//    barrier), beyond that each CTA takes its share of the positions and the
//    histograms are added through distributed shared memory;
//  - one pass over the positions then lists the kept ones in order (in shared
//    memory, or in global memory for the cluster).
// The move copies row list[j] to row j in increasing j, a chunk of rows in
// registers at a time.  list[j] >= j, so a chunk may be written once all of ITS
// sources are read: later chunks read at or past their own start, and the next
// chunk's loads are already in flight while this one is stored.  Column parts
// never touch one another's bytes, so no CTA waits for another here.
#include <cooperative_groups.h>

#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 4;            // 16-byte pieces per thread and chunk of the move
constexpr int kHeld = 8;           // weights a thread keeps in registers between passes
constexpr int kSoloTokens = kThreads * kHeld;

// Order-preserving image of a weight: larger weight, larger integer; -0 equals
// +0 and every NaN is the largest value.
__device__ __forceinline__ uint32_t rank_bits(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    if (u == 0x80000000u) u = 0;
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Cache row (over [slots or blocks, heads, rows]) of position pos of (b, h).
__device__ __forceinline__ size_t cache_row(const EvictArgs& a, int b, int h, int pos) {
    if (!a.block_table) return ((size_t)b * a.n_kv_heads + h) * a.max_cache_len + pos;
    const int blk = __ldg(a.block_table + (size_t)b * a.max_blocks + (pos >> a.block_log2));
    return (((size_t)blk * a.n_kv_heads + h) << a.block_log2) + (pos & ((1 << a.block_log2) - 1));
}

// Length of sequence b, or -1 when it is inconsistent or one of its blocks lies
// outside the pool (every CTA of the sequence comes to the same verdict).
__device__ int checked_length(const EvictArgs& a, int b) {
    const int len = a.lengths[b];
    bool bad = len < 0 || len > a.max_cache_len;
    if (!a.block_table) return bad ? -1 : len;
    if (!bad) {
        const int nb = (len + (1 << a.block_log2) - 1) >> a.block_log2;
#pragma unroll 4
        for (int i = threadIdx.x; i < nb; i += kThreads) {
            const int blk = __ldg(a.block_table + (size_t)b * a.max_blocks + i);
            bad |= blk < 0 || blk >= a.num_blocks;
        }
    }
    return __syncthreads_or(bad) ? -1 : len;
}

struct Shared {
    int hist[4][256];  // one per pass: no barrier between reading one and clearing the next
    int sums[256];
    int counts[2][kHeld * kWarps];  // certain and equal positions per block and warp, then ahead of them
    int total[2];        // ... of this CTA's share
    int total_batch[2];  // ... of a batch
    uint32_t digit;
    int need;
    int list[kSoloTokens];  // kept positions (one CTA alone)
};

// Moves a scalar per row (weights, row scales): dst row j = src row list[j].
__device__ void move_scalars(const EvictArgs& a, int b, int h, const float* src, float* dst, const int* list, int count) {
    for (int j0 = 0; j0 < count; j0 += kThreads * kHeld) {
        float x[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int j = j0 + i * kThreads + threadIdx.x;
            if (j < count) x[i] = src[cache_row(a, b, h, list[j])];
        }
        __syncthreads();  // in place: this chunk's sources are read
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int j = j0 + i * kThreads + threadIdx.x;
            if (j < count) dst[cache_row(a, b, h, j)] = x[i];
        }
    }
}

__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int bh = blockIdx.x / ranks;
    const int h = bh % a.n_kv_heads, b = bh / a.n_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = checked_length(a, b);
    if (len < 0) {
        if (tid == 0 && rank == 0 && h == 0) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
        return;
    }
    const bool coop = len > kSoloTokens;
    const int parts = coop ? ranks : 1, part = coop ? rank : 0;
    const int count = min(len, a.budget);
    const bool all = len <= a.budget;
    const int lo = a.sinks, hi = len - a.recent;  // the tokens that compete (when !all)
    int need = all ? 0 : a.budget - a.sinks - a.recent;
    // this CTA's positions: [p_lo, p_hi), thread t at p_lo + t, + kThreads, ...
    const int share = ((len + parts - 1) / parts + 31) & ~31;
    const int p_lo = min(len, part * share), p_hi = min(len, p_lo + share);
    uint32_t held[kHeld];
    uint32_t threshold = 0;
    int* const list = coop ? a.index + (size_t)bh * a.budget : sh.list;

    if (need > 0) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int p = p_lo + i * kThreads + tid;
            held[i] = p >= lo && p < min(p_hi, hi) ? rank_bits(a.weights[cache_row(a, b, h, p)]) : 0;
        }
        for (int i = tid; i < 4 * 256; i += kThreads) (&sh.hist[0][0])[i] = 0;
        __syncthreads();
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int p = p_lo + i * kThreads + tid;
                if (p >= lo && p < min(p_hi, hi) && (held[i] & mask) == threshold)
                    atomicAdd(&sh.hist[pass][(held[i] >> shift) & 255], 1);
            }
#pragma unroll 4
            for (int p = p_lo + kHeld * kThreads + tid; p < min(p_hi, hi); p += kThreads) {
                const uint32_t r = rank_bits(a.weights[cache_row(a, b, h, p)]);
                if (p >= lo && (r & mask) == threshold) atomicAdd(&sh.hist[pass][(r >> shift) & 255], 1);
            }
            if (coop)
                cluster.sync();
            else
                __syncthreads();
            // bin `tid` over the cluster; then how many weights lie in higher bins
            int mine = 0;
            if (tid < 256) {
                if (coop) {
#pragma unroll 8
                    for (int r = 0; r < ranks; ++r) mine += *cluster.map_shared_rank(&sh.hist[pass][tid], r);
                } else {
                    mine = sh.hist[pass][tid];
                }
                int above = mine;  // suffix sum within the warp
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_down_sync(0xffffffffu, above, o);
                    if (lane + o < 32) above += y;
                }
                sh.sums[tid] = above;
            }
            __syncthreads();
            if (tid < 256) {
                int above = sh.sums[tid] - mine;  // in higher bins
                for (int w = warp + 1; w < 8; ++w) above += sh.sums[w * 32];
                if (above < need && above + mine >= need) {
                    sh.digit = (uint32_t)tid;
                    sh.need = need - above;  // of this bin's
                }
            }
            __syncthreads();
            threshold |= sh.digit << shift;
            need = sh.need;
        }
    }
    // `need` is now how many weights equal to the threshold stay.
    const bool compete = !all && a.budget > a.sinks + a.recent;
    // 1: the position stays for certain, 2: its weight equals the threshold
    auto state = [&](int p, uint32_t r) -> int {
        if (p >= p_hi) return 0;
        if (all || p < lo || p >= hi) return 1;
        return !compete ? 0 : r > threshold ? 1 : r == threshold ? 2 : 0;
    };
    // a batch of kHeld blocks of kThreads positions from p0; the first is in `held`
    auto load_batch = [&](int p0) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int p = p0 + i * kThreads + tid;
            if (compete && p >= lo && p < min(p_hi, hi)) held[i] = rank_bits(a.weights[cache_row(a, b, h, p)]);
        }
    };
    int before = 0, equal_before = 0;  // kept positions and equal weights ahead of the batch
    if (coop) {
        int certain = 0, equal = 0;
        for (int p0 = p_lo; p0 < p_hi; p0 += kHeld * kThreads) {
            if (p0 > p_lo) load_batch(p0);
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int s = state(p0 + i * kThreads + tid, held[i]);
                certain += s == 1;
                equal += s == 2;
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            certain += __shfl_xor_sync(0xffffffffu, certain, o);
            equal += __shfl_xor_sync(0xffffffffu, equal, o);
        }
        if (lane == 0) sh.counts[0][warp] = certain, sh.counts[1][warp] = equal;
        __syncthreads();
        if (tid < 2) {
            int sum = 0;
            for (int w = 0; w < kWarps; ++w) sum += sh.counts[tid][w];
            sh.total[tid] = sum;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            before += *cluster.map_shared_rank(&sh.total[0], r);
            equal_before += *cluster.map_shared_rank(&sh.total[1], r);
        }
        before += min(equal_before, need);
        if (p_hi - p_lo > kHeld * kThreads) load_batch(p_lo);
    }
    // the kept positions, in order: warp w's part of block i comes after every
    // part of an earlier block and the earlier warps' parts of its own
    static_assert(kHeld * kWarps == 128, "four parts per lane of the scan");
    for (int p0 = p_lo; p0 < p_hi; p0 += kHeld * kThreads) {
        if (p0 > p_lo) load_batch(p0);
        int st[kHeld];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            st[i] = state(p0 + i * kThreads + tid, held[i]);
            const unsigned cm = __ballot_sync(0xffffffffu, st[i] == 1), em = __ballot_sync(0xffffffffu, st[i] == 2);
            if (lane == 0) sh.counts[0][i * kWarps + warp] = __popc(cm), sh.counts[1][i * kWarps + warp] = __popc(em);
        }
        __syncthreads();
        if (warp < 2) {  // warp 0 scans the certain ones, warp 1 the equal ones
            int c[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = sum;
                sum += sh.counts[warp][lane * 4 + i];
            }
            int inc = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sh.counts[warp][lane * 4 + i] = inc - sum + c[i];
            if (lane == 31) sh.total_batch[warp] = inc;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const unsigned cm = __ballot_sync(0xffffffffu, st[i] == 1), em = __ballot_sync(0xffffffffu, st[i] == 2);
            const unsigned below = (1u << lane) - 1;
            const int certain = sh.counts[0][i * kWarps + warp] + __popc(cm & below);
            const int equal = equal_before + sh.counts[1][i * kWarps + warp] + __popc(em & below);
            // kept ahead of p: the certain ones, and the equal ones that stay
            if (st[i] == 1 || (st[i] == 2 && equal < need))
                list[before + certain + min(equal, need) - min(equal_before, need)] = p0 + i * kThreads + tid;
        }
        before += sh.total_batch[0] + min(equal_before + sh.total_batch[1], need) - min(equal_before, need);
        equal_before += sh.total_batch[1];
    }
    __syncthreads();
    if (coop)
        cluster.sync();  // the list is whole, and every CTA has read the weights it needs
    else if (a.kept_weights == a.weights)
        cluster.sync();
    if (!coop && rank == 0)
        for (int i = tid; i < count; i += kThreads) a.index[(size_t)bh * a.budget + i] = list[i];
    if (rank == ranks - 1)
        for (int i = count + tid; i < a.budget; i += kThreads) a.index[(size_t)bh * a.budget + i] = -1;
    if (tid == 0 && rank == 0 && h == 0) a.kept_lengths[b] = count;
    if (rank == ranks - 1 && a.kept_weights && !(all && a.kept_weights == a.weights))
        move_scalars(a, b, h, a.weights, a.kept_weights, list, count);
    if (all) return;
    if (a.scale_k && rank < 2) {
        float* scale = rank ? a.scale_v : a.scale_k;
        move_scalars(a, b, h, scale, scale, list, count);
    }

    // K on even ranks, V on odd ones; column part rank / 2
    uint8_t* const cache = static_cast<uint8_t*>(rank & 1 ? a.cache_v : a.cache_k) + (rank >> 1) * a.part_bytes;
    const int log_pieces = a.part_bytes == 64 ? 2 : a.part_bytes == 32 ? 1 : 3;  // 16-byte pieces of a part
    const int rows = (kThreads * kVec) >> log_pieces;                           // of a chunk
    const int piece = tid & ((1 << log_pieces) - 1), row0 = tid >> log_pieces, step = kThreads >> log_pieces;
    auto sources = [&](int j0, int (&src)[kVec]) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int j = j0 + row0 + i * step;
            src[i] = j < count ? list[j] : -1;
            if (src[i] == j) src[i] = -1;  // already there
        }
    };
    auto load = [&](const int (&src)[kVec], uint4 (&x)[kVec]) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (src[i] >= 0)
                x[i] = *reinterpret_cast<const uint4*>(cache + cache_row(a, b, h, src[i]) * a.row_bytes + piece * 16);
    };
    uint4 x[kVec], y[kVec];
    int src[kVec], next[kVec];
    sources(0, src);
    load(src, x);
    for (int j0 = 0; j0 < count; j0 += rows) {
        sources(j0 + rows, next);
        load(next, y);
        __syncthreads();  // every source of this chunk is read
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (src[i] >= 0)
                *reinterpret_cast<uint4*>(cache + cache_row(a, b, h, j0 + row0 + i * step) * a.row_bytes + piece * 16) = x[i];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            x[i] = y[i];
            src[i] = next[i];
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& args, cudaStream_t stream) {
    EvictArgs a = args;
    a.part_bytes = a.row_bytes < 64 ? a.row_bytes : 64;
    const int ranks = 2 * (a.row_bytes / a.part_bytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ranks * a.num_seqs * a.n_kv_heads));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_kernel, a);
}

}  // namespace pa
