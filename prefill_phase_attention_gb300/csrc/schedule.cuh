// schedule.cuh -- device helpers shared by the tile schedulers.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"

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

// Whether entries [lo, hi) of a sequence's block table name a block outside the
// pool (one warp; 16 loads of a lane in flight).
__device__ __forceinline__ bool bad_blocks(const int32_t* table, int lo, int hi, int num_blocks, int lane) {
    bool bad = false;
    for (int L = lo + lane; L < hi; L += 32 * 16) {
        int blk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) blk[i] = L + 32 * i < hi ? __ldg(table + L + 32 * i) : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) bad |= (unsigned)blk[i] >= (unsigned)num_blocks;
    }
    return __any_sync(0xffffffffu, bad);
}

// The same for the blocks that a sequence's queries touch: those of its sink
// tiles, and those from its window's first tile to its last new token (one warp).
__device__ __forceinline__ bool bad_visible_blocks(const int32_t* table, const SeqInfo& si, int block_size,
                                                   int num_blocks, int causal, int window, int sinks, int lane) {
    if (si.n == 0) return false;
    const StreamGeo g = stream_geo(si.n, si.P, 0, si.n, causal, window, sinks, false, true);
    const int sink_end = min(g.nsink * kBlockN, si.P);
    const int first = g.lo < prefix_tiles(si.P) ? g.lo * kBlockN : si.P;
    return bad_blocks(table, 0, (sink_end + block_size - 1) / block_size, num_blocks, lane) |
           bad_blocks(table, first / block_size, (si.P + si.n - 1) / block_size + 1, num_blocks, lane);
}

// Sequence b of a call as its device metadata states it; n = -1 when that is inconsistent.
__device__ __forceinline__ SeqInfo checked_sequence(const ScheduleArgs& a, int b) {
    const int q_start = a.cu_seqlens_q[b], q_end = a.cu_seqlens_q[b + 1];
    const int lk = a.cu_seqlens_k[b + 1] - a.cu_seqlens_k[b];
    const int P = a.cache_offsets[b];
    const long long n = (long long)q_end - q_start;
    const bool ok = q_start >= 0 && n >= 0 && (long long)q_end <= a.total_q && P >= 0 &&
                    (long long)lk == (long long)P + n && (long long)P + n <= a.max_cache_len && (b > 0 || q_start == 0);
    return ok ? SeqInfo{q_start, (int)n, P, 0} : SeqInfo{0, -1, 0, 0};
}

// ---- batches of up to kFewSeqs sequences (the shared prefix among them) ----
//
// The counting sort of the general schedulers costs a one-CTA kernel most of its
// time (its passes run 32 warps through ~2000 instructions each).  A few
// sequences are ranked by comparing each with every other instead, one thread
// per sequence, in shared memory (launch lists, cold caches: one sequence 8.3 ->
// 5.0 us, 64 sequences over 16-token pages 19 -> 15).
constexpr int kFewSeqs = 256;
constexpr int kFewThreads = 512;

struct FewSeqs {
    SeqInfo seqs[kFewSeqs];  // pad: index of the sequence's first block
    float cost[kFewSeqs];
    int blocks[kFewSeqs];    // schedulable blocks per head
    int units[kFewSeqs];     // units in all
    int first[kFewSeqs];     // its first unit in the list
    int group[kFewSeqs];     // KV heads that run together
    int spans[kFewSeqs][2];  // table entries [0, x) and [y, end) to check: x, y
    int max_chunks;
    unsigned long long total;
};

// Loads and checks the sequences (and the prefix's table); f.seqs[b].n is 0 for a
// rejected one (which the lead CTA reports).  Ends with a barrier.  Returns
// whether the prefix is usable.
__device__ __forceinline__ bool load_few(const ScheduleArgs& a, FewSeqs& f, int sinks, const int32_t* prefix_table,
                                         int prefix_len, bool lead) {
    constexpr int kChunk = 16;  // table entries of a thread in flight
    const int tid = threadIdx.x;
    bool bad = false, prefix_ok = true;
    if (tid == 0) f.max_chunks = 0, f.total = 0;
    if (a.block_table) {
        __syncthreads();
        if (tid < a.num_seqs) {
            const SeqInfo si = checked_sequence(a, tid);
            f.seqs[tid] = si;
            int x = 0, y = 0, end = 0;
            if (si.n > 0) {
                const StreamGeo g = stream_geo(si.n, si.P, 0, si.n, a.causal, a.window, sinks, false, true);
                x = (min(g.nsink * kBlockN, si.P) + a.block_size - 1) / a.block_size;
                y = (g.lo < prefix_tiles(si.P) ? g.lo * kBlockN : si.P) / a.block_size;
                end = (si.P + si.n - 1) / a.block_size + 1;
            }
            x = min(x, y);  // the two ranges as one: entry i stands for i < x ? i : i - x + y
            f.spans[tid][0] = x;
            f.spans[tid][1] = y;
            f.blocks[tid] = end - y + x;  // entries to check
            atomicMax(&f.max_chunks, (end - y + x + kChunk - 1) / kChunk);
        }
        __syncthreads();
        const unsigned chunks = (unsigned)f.max_chunks;  // < 2^23, of at most 2^8 sequences
        for (unsigned w = tid; w < a.num_seqs * chunks; w += blockDim.x) {
            const int b = w / chunks, i0 = w % chunks * kChunk;
            const int n = f.blocks[b], x = f.spans[b][0], shift = f.spans[b][1] - x;
            const int32_t* row = a.block_table + (size_t)b * a.max_blocks;
            int blk[kChunk];
#pragma unroll
            for (int i = 0; i < kChunk; ++i) blk[i] = i0 + i < n ? __ldg(row + i0 + i + (i0 + i < x ? 0 : shift)) : 0;
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if ((unsigned)blk[i] >= (unsigned)a.num_blocks) f.seqs[b].n = -1;  // (several threads, one value)
        }
        if (prefix_len > 0) {
            const int nb = (prefix_len + a.block_size - 1) / a.block_size;
#pragma unroll 8
            for (int i = tid; i < nb; i += blockDim.x) bad |= (unsigned)__ldg(prefix_table + i) >= (unsigned)a.num_blocks;
        }
        prefix_ok = !__syncthreads_or(bad);
    }
    if (tid < a.num_seqs) {
        SeqInfo si = a.block_table ? f.seqs[tid] : checked_sequence(a, tid);
        if (si.n < 0 || !prefix_ok) {
            if (lead) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
            si = SeqInfo{0, 0, 0, 0};
        }
        f.seqs[tid] = si;
    } else if (tid == a.num_seqs && prefix_len > 0) {
        const int end = a.cu_seqlens_q[a.num_seqs];
        const int n = !prefix_ok || end < 0 ? 0 : (end < a.total_q ? end : a.total_q);
        f.seqs[tid] = SeqInfo{0, n, prefix_len, 0};
    }
    __syncthreads();
    return prefix_ok;
}

// From f.cost, f.blocks and f.units: each sequence's place in the list (by
// descending cost, then index) and the first-block numbers; where a list is
// `shared` between CTAs, its header and the sequences for the other kernels.
// Returns the blocks of all sequences.  Ends with a barrier.
__device__ __forceinline__ int rank_few(const ScheduleArgs& a, FewSeqs& f, int nseq, bool shared) {
    const int tid = threadIdx.x;
    if (tid < nseq) {
        const float mine = f.cost[tid];
        int first = 0, pad = 0, total = 0;
#pragma unroll 8
        for (int b = 0; b < nseq; ++b) {
            const float c = f.cost[b];
            const int u = f.units[b], n = f.blocks[b];
            first += c > mine || (c == mine && b < tid) ? u : 0;
            pad += b < tid ? n : 0;
            total += u;
        }
        f.first[tid] = first;
        f.seqs[tid].pad = pad;
        if (tid == nseq - 1) f.max_chunks = pad + f.blocks[tid];
        if (shared) a.seqs[tid] = f.seqs[tid];
        if (shared && tid == nseq - 1) {
            a.hdr->num_units = total < a.max_units ? total : a.max_units;
            a.hdr->counter = 0;
            a.hdr->max_units = a.max_units;
            if (total > a.max_units) atomicOr(&a.hdr->error, PA_DEVERR_OVERFLOW);
        }
    }
    __syncthreads();
    return f.max_chunks;
}

}  // namespace pa
