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
    __shared__ int warp_sums[32], first_out, base_there;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Cache4& c = p.cache;
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
    // In order, each sequence that fits in what is left of the pool: passes over 1024 of them, each of which
    // takes those before the first that does not fit, and leaves that one out.  (One pass where all fit.)
    int base = 0;  // blocks given away
    for (int b0 = 0; b0 < p.seqs.num_seqs; b0 += 1024) {
        const int b = b0 + tid;
        SeqInfo s{0, 0, 0, 0};
        if (b < p.seqs.num_seqs) s = p.seqs.checked[b];
        bool open = s.n > p.few_tokens, fits = false;
        const int first = first_block(p, s);
        const int need = end_block(s) - first;  // (0: a first prompt)
        int at = 0;
        for (;;) {
            open = open && need <= p.pool_blocks - base;
            // (sums past the pool saturate: a sequence's blocks are at most 2^23)
            int end = open ? need : 0;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end = min(end + y, 1 << 29);
            }
            if (lane == 31) warp_sums[warp] = end;
            if (tid == 0) first_out = 1024;
            __syncthreads();
            int before = base;
            int all = base;
            for (int w = 0; w < 32; ++w) {
                if (w < warp) before = min(before + warp_sums[w], 1 << 29);
                all = min(all + warp_sums[w], 1 << 29);
            }
            end = min(before + end, 1 << 29);
            if (open && end > p.pool_blocks) atomicMin(&first_out, tid);
            __syncthreads();
            const int out = first_out;
            if (open && tid < out) open = false, fits = true, at = end - need;
            if (tid == out) open = false, base_there = end - need;
            __syncthreads();
            base = out < 1024 ? base_there : all;
            if (out == 1024) break;
        }
        if (b < p.seqs.num_seqs) {
            p.taken[b] = fits;
            p.base[b] = fits ? at * kBlock4 - block_start(s, first) : 0;
        }
    }
    if (tid == 0) *p.blocks = base;
    __syncthreads();
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
