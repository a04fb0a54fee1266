// schedule.cuh -- device helpers shared by the tile schedulers.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace pa {

constexpr long long kL2GroupBytes = 48ll << 20;
// Batches of up to this many sequences keep the per-sequence tables the passes
// below hand to one another (SeqInfo, cost bin / list position, KV-head group)
// in shared memory; larger ones go through the workspace in global memory.
constexpr int kSmemSeqs = 1024;

// Sort key of a sequence: its total cost in log-spaced bins (exact below 64,
// then 64 bins per power of two), clamped to the histogram.
__device__ __forceinline__ int cost_bin(long long c) {
    if (c < 64) return (int)c;
    const int e = 63 - __clzll(c);  // >= 6
    const long long bin = 64 + (long long)(e - 6) * 64 + ((c >> (e - 6)) & 63);
    return bin < kCostBins - 1 ? (int)bin : kCostBins - 1;
}

// Block-wide exclusive scan of one int per thread (1024 threads); returns the
// exclusive prefix and writes the block total to *total.
__device__ __forceinline__ int block_exclusive_scan(int x, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;  // inclusive over warps
    }
    __syncthreads();
    const int excl = inc - x + (warp > 0 ? warp_sums[warp - 1] : 0);
    *total = warp_sums[31];
    __syncthreads();
    return excl;
}

// Sequence owning flattened query block i: the last b with seqs[b].pad <= i
// among sequences that have blocks (pad holds the first block index of b).
__device__ __forceinline__ int block_owner(const SeqInfo* seqs, int num_seqs, int i) {
    int lo = 0, hi = num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seqs[mid].pad <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// KV heads of a sequence whose units run together.  Every unit of a head
// streams that head's K/V from the start of the sequence, so while the CTAs
// work on a group of heads, the group's K/V (keys and values of P + n tokens,
// bf16) is what they re-read from L2; groups are sized to keep it within
// kL2GroupBytes (a share of the 129 MB L2 that leaves room for the q, out and
// cache-write streams and for the next group, which starts while the last
// units of a group run).  A group must also hold at least num_ctas times the
// sequence's longest unit of work (head_cost = the KV tiles of one head's
// units, longest = the most of one unit): a group's longest unit starts when
// the group does, so a smaller last group would end the launch on that one
// unit while the other SMs idle.  That bound wins over the L2 budget.  Short
// sequences keep all their heads in one group.
__device__ __forceinline__ int kv_head_group(const SeqInfo& si, int head_dim, int n_kv_heads, int num_ctas,
                                             long long head_cost, int longest) {
    const float head_bytes = (float)(si.P + si.n) * (float)(head_dim * 4);
    float g = floorf((float)kL2GroupBytes / fmaxf(head_bytes, 1.f));
    if (head_cost > 0) g = fmaxf(g, ceilf((float)num_ctas * (float)longest / (float)head_cost));
    return g >= (float)n_kv_heads ? n_kv_heads : (g < 1.f ? 1 : (int)g);
}

}  // namespace pa
