// plan4.cuh -- which sequences of a call over a 4-bit cache are expanded to bf16, and where to.
#pragma once

#include "cache4.cuh"
#include "kernels.h"

namespace pa {

// The attention kernel's tiles of a sequence's cached positions, which are the pool's blocks: [first,
// end) of them, the last one ends at position P - 1, so that block 0 may begin below 0.
__device__ __forceinline__ int end_block(const SeqInfo& s) { return (s.P + kBlock4 - 1) / kBlock4; }
__device__ __forceinline__ int block_start(const SeqInfo& s, int i) { return s.P - (end_block(s) - i) * kBlock4; }
__device__ __forceinline__ int first_block(const Expand4Params& p, const SeqInfo& s) {
    const int oldest = p.window > 0 ? max(0, s.P - p.window + 1) : 0;  // key that a query sees
    return (oldest - block_start(s, 0)) / kBlock4;
}

// Checks the sequences, and lays out the pool (one block of 1024 threads; ends with a barrier).
__device__ __forceinline__ void plan_expand4(const Expand4Params& p) {
    __shared__ int warp_sums[32], in_use;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Cache4& c = p.cache;
    if (tid == 0) in_use = 0;
    // a warp per sequence
    for (int b = warp; b < p.seqs.num_seqs; b += 32) {
        const SeqInfo s = stated_sequence(p.seqs, c.max_cache_len, b);
        bool bad = s.n < 0;
        if (c.block_table && s.n > 0) {
            const int end = ((s.P + s.n - 1) >> c.block_log2) + 1;
            const int32_t* table = c.block_table + (size_t)b * c.max_blocks;
#pragma unroll 8
            for (int i = lane; i < end; i += 32) bad |= (unsigned)__ldg(table + i) >= (unsigned)c.num_blocks;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            p.seqs.checked[b] = bad ? SeqInfo{0, 0, 0, 0} : s;
            if (bad) atomicOr(&p.seqs.hdr->error, PA_DEVERR_METADATA);
        }
    }
    __syncthreads();
    int base = 0;  // blocks of the sequences before
    for (int b0 = 0; b0 < p.seqs.num_seqs; b0 += 1024) {
        const int b = b0 + tid;
        SeqInfo s{0, 0, 0, 0};
        if (b < p.seqs.num_seqs) s = p.seqs.checked[b];
        const bool wanted = s.n > p.few_tokens;
        const int first = first_block(p, s);
        // (sums past the pool saturate: a sequence's blocks are at most 2^23)
        int need = wanted ? end_block(s) - first : 0, inc = need;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc = min(inc + y, 1 << 29);
        }
        if (lane == 31) warp_sums[warp] = inc;
        __syncthreads();
        int before = base;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) before = min(before + warp_sums[w], 1 << 29);
            base = min(base + warp_sums[w], 1 << 29);
        }
        const int at = min(before + inc, 1 << 29) - need;
        const bool fits = wanted && before + inc < 1 << 29 && at + need <= p.pool_blocks;
        if (b < p.seqs.num_seqs) {
            p.taken[b] = fits;
            p.base[b] = fits ? at * kBlock4 - block_start(s, first) : 0;
        }
        if (fits) atomicMax(&in_use, at + need);  // (those that fit are the first ones: no gaps)
        __syncthreads();
    }
    if (tid == 0) *p.blocks = in_use;
    for (int b = warp; b < p.seqs.num_seqs; b += 32) {
        if (!p.taken[b]) continue;
        const SeqInfo s = p.seqs.checked[b];
        const int first = first_block(p, s), end = end_block(s), at = (p.base[b] + block_start(s, first)) / kBlock4;
        for (int i = first + lane; i < end; i += 32) p.owners[at + i - first] = make_int2(b, block_start(s, i));
    }
    __threadfence_block();
    __syncthreads();
}

}  // namespace pa
