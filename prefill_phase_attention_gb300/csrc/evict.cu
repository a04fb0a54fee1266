// evict.cu -- eviction from a KV cache by accumulated attention weight.
//
// Per (sequence, KV head) of a cache of L tokens, L > budget: the first
// `sinks` and the last `recent` tokens stay, and of the tokens between them
// the m = budget - sinks - recent with the largest weight (ties: the lowest
// position first; NaN ranks above everything).  The kept rows of K and V move
// to positions 0 .. budget - 1 in their old order, in place.  L <= budget keeps
// every token.
//
// Choosing: the m-th largest weight by a radix select, 8 bits of the weight's
// order-preserving integer image per pass, until few enough weights share the
// digits chosen so far to be compared with one another.  One CTA does it alone while its
// threads can hold the weights in registers; beyond that the CTAs of a cluster
// each take a share of the positions and add their histograms through
// distributed shared memory.  One pass over the positions then lists the kept
// ones in order.
//
// Moving: row list[j] to row j in increasing j, a chunk of rows in registers at
// a time.  list[j] >= j, so a chunk may be written once all of ITS sources are
// read: later chunks read at or past their own start, and the next chunk's
// loads are already in flight while this one is stored.  A CTA moves one column
// part (64 bytes where the row has them) of K or of V; parts never touch one
// another's bytes, so no CTA waits for another.
//
// Two forms, picked by the number of CTAs.  While they all run at once, evict_kernel
// does both in one launch, a cluster of 2, 4 or 8 CTAs (its column parts) per
// (sequence, head).  With more of them a CTA that selects keeps one that moves from
// running: select_kernel runs first, one CTA (or a cluster) per (sequence, head), then
// move_kernel, which HBM bounds.  Measured (graph, 8 heads):
// 4 sequences of about 510 tokens to 384 7.8 us in one launch, 10.1 in two; 16 of
// 16384 to 4096 133 and 110 (select 19, move 85 at 6.3 TB/s); 64 of 700-4099 to
// 1024 in int8 pages 97 and 62.6.
// Few long caches take the first form too, and neither is near HBM there: a column
// part of a head is one CTA's, whatever its length, 8 KB fetched while 8 KB are
// written.
// Single cold passes, D = 128 bf16, to a quarter, one launch and two: one cache of
// 8192 tokens of 8 heads 34 and 38 us, of 32768 91 and 91 (0.75 TB/s), of 131072 333
// and 351; of 32768 tokens of 2 heads 91 and 89 (0.19 TB/s); four of 16384 of 8
// heads 59 and 67 (2.4 TB/s).
#include <cooperative_groups.h>

#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"
#include "ptx.cuh"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kVec = 2;  // 16-byte pieces per thread and chunk of the move
// one-launch form: threads, weights a thread holds (so tokens a CTA selects from alone)
constexpr int kFusedThreads = 256, kFusedHeld = 8;
// two-launch form (select CTAs of 512 threads: 70.0 us against 62.6 for 64 sequences
// of 700-4099 tokens in int8 pages, within 1 % for 16 of 16384, 32768 and 65536)
constexpr int kSelectThreads = 256, kSelectHeld = 16, kMoveThreads = 256;
// Weights crowd into a few digits: a histogram has this many copies, one per
// lane & 7, a bank apart, so that a warp's equal digits do not queue up.
constexpr int kCopies = 8;
// Once the bin that holds the m-th largest weight has at most this many, they are
// compared with one another instead of by further passes: after two of the four,
// for weights that are not nearly all alike.
constexpr int kCandidates = 128;

// Order-preserving image of a weight: larger weight, larger integer; -0 equals
// +0 and every NaN is the largest value.
__device__ __forceinline__ uint32_t rank_bits(float w) {
    const uint32_t u = __float_as_uint(__fadd_rn(w, 0.f));  // -0 + 0 = +0
    return w != w ? 0xffffffffu : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// Cache rows (over [slots or blocks, heads, rows]) of the positions of one (b, h).
struct Rows {
    const int32_t* table;  // nullptr: contiguous, rows base + pos
    size_t base;
    int log2, n_kv_heads, h;
    __device__ __forceinline__ Rows(const EvictArgs& a, int b, int head)
        : table(a.block_table ? a.block_table + (size_t)b * a.max_blocks : nullptr),
          base(((size_t)b * a.n_kv_heads + head) * a.max_cache_len),
          log2(a.block_log2),
          n_kv_heads(a.n_kv_heads),
          h(head) {}
    __device__ __forceinline__ size_t operator()(int pos) const {
        if (!table) return base + pos;
        const int head_block = __ldg(table + (pos >> log2)) * n_kv_heads + h;
        return ((size_t)head_block << log2) + (pos & ((1 << log2) - 1));
    }
};

// Length of sequence b, or -1 when it is inconsistent or one of its blocks lies
// outside the pool (every CTA of the sequence comes to the same verdict).
template <int kThreads>
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

template <int kThreads, int kHeld>
struct Shared {
    uint32_t copies[kCopies][257];
    int hist[4][256];  // this CTA's, one per pass: no barrier between the cluster's reads and the next pass
    int sums[256];
    int warp_counts[2][kThreads / 32];  // certain and equal positions per warp, then ahead of the warp
    int total[2];                       // ... of this CTA's share
    int batch[2];                       // ... of a batch
    uint32_t digit;
    int need, inside;                   // wanted from the chosen bin; weights in it
    int found;                          // candidates of this CTA's share
    uint32_t ranks[kThreads * (kHeld + 1)];  // a batch of rank_bits, one padding word per thread
};

// Moves a scalar per row (weights, row scales), kPerThread of a thread at a time:
// dst row j = src row list[j].
template <int kThreads, int kPerThread>
__device__ __forceinline__ void move_scalars(const Rows& rows, const float* src, float* dst, const int* list, int count) {
    for (int j0 = 0; j0 < count; j0 += kThreads * kPerThread) {
        float x[kPerThread];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int j = j0 + i * kThreads + threadIdx.x;
            if (j < count) x[i] = src[rows(list[j])];
        }
        __syncthreads();  // in place: this chunk's sources are read
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int j = j0 + i * kThreads + threadIdx.x;
            if (j < count) dst[rows(j)] = x[i];
        }
    }
}

// Lists the kept positions of (b, h) into `list`, ascending: this CTA's share of
// [0, len) when the cluster works together (coop), all of them otherwise.  Ends
// with a barrier of the CTA; a cluster's list is whole after a cluster barrier.
template <int kThreads, int kHeld>
__device__ __forceinline__ void select_tokens(const EvictArgs& a, Shared<kThreads, kHeld>& sh,
                                              const cg::cluster_group& cluster, int b, int h, int len, bool coop,
                                              int* list) {
    constexpr int kWarps = kThreads / 32;
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int parts = coop ? ranks : 1, part = coop ? rank : 0;
    const bool all = len <= a.budget;
    const int lo = a.sinks, hi = len - a.recent;  // the tokens that compete (when !all)
    int need = all ? 0 : a.budget - a.sinks - a.recent;
    // This CTA's positions [p_lo, p_hi), in batches; thread t has kHeld
    // consecutive ones of a batch in registers, read coalesced and handed over
    // through shared memory.  A rank of 0 (below every weight's) stands for a
    // position that does not compete.
    const int share = ((len + parts - 1) / parts + 31) & ~31;
    const int p_lo = min(len, part * share), p_hi = min(len, p_lo + share);
    constexpr int kBatch = kThreads * kHeld;
    const bool compete = need > 0;
    const Rows rows(a, b, h);
    uint32_t held[kHeld];
    uint32_t threshold = 0;
    auto load_batch = [&](int p0) {
        __syncthreads();
        // positions [lo, last) compete
        const unsigned span = compete ? (unsigned)max(0, min(p_hi, hi) - lo) : 0u;
        if (!rows.table) {
            const float* w = a.weights + rows.base + p0;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int x = i * kThreads + tid;
                sh.ranks[x + x / kHeld] = (unsigned)(p0 + x - lo) < span ? rank_bits(w[x]) : 0;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int x = i * kThreads + tid;
                sh.ranks[x + x / kHeld] = (unsigned)(p0 + x - lo) < span ? rank_bits(a.weights[rows(p0 + x)]) : 0;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int x = tid * kHeld + i;
            held[i] = x < p_hi - p0 ? sh.ranks[tid * (kHeld + 1) + i] : 0;
        }
    };
    const bool one_batch = p_hi - p_lo <= kBatch;
    load_batch(p_lo);

    if (compete) {
        uint32_t* const my_copy = sh.copies[lane & (kCopies - 1)];
        if (tid == 0) sh.found = 0;
        uint32_t mask = 0;  // the digits chosen so far
        int inside = len;   // weights that share them
        for (int pass = 0; pass < 4 && inside > kCandidates; ++pass) {
            const int shift = 24 - 8 * pass;
            for (int i = tid; i < kCopies * 257; i += kThreads) (&sh.copies[0][0])[i] = 0;
            __syncthreads();
            for (int p0 = p_lo; p0 < p_hi; p0 += kBatch) {
                if (!one_batch && (pass > 0 || p0 > p_lo)) load_batch(p0);
                if (p0 + warp * 32 * kHeld >= p_hi) continue;  // nothing of the batch is this warp's
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
                    // (ranks of 0 are the lowest: the digits chosen from above never reach them)
                    if ((held[i] & mask) == threshold) atomicAdd(&my_copy[(held[i] >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid < 256) {
                int sum = 0;
#pragma unroll
                for (int c = 0; c < kCopies; ++c) sum += (int)sh.copies[c][tid];
                sh.hist[pass][tid] = sum;
            }
            if (coop) cluster.sync();
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
                    sh.inside = mine;
                }
            }
            __syncthreads();
            threshold |= sh.digit << shift;
            mask |= 255u << shift;
            need = sh.need;
            inside = sh.inside;
        }
        if (mask != 0xffffffffu) {
            // the candidates of this CTA's share and of the cluster, where histograms were
            uint32_t *const own = sh.copies[0], *const every = sh.copies[1];
            __syncthreads();  // (sh.found)
            for (int p0 = p_lo; p0 < p_hi; p0 += kBatch) {
                if (!one_batch) load_batch(p0);
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
                    if (held[i] != 0 && (held[i] & mask) == threshold) own[atomicAdd(&sh.found, 1)] = held[i];
            }
            __syncthreads();
            const uint32_t* among = own;
            int n = sh.found;
            if (coop) {
                cluster.sync();
                n = 0;
                for (int r = 0; r < ranks; ++r) {
                    const int m = *cluster.map_shared_rank(&sh.found, r);
                    if (tid < m) every[n + tid] = *cluster.map_shared_rank(&own[tid], r);
                    n += m;
                }
                __syncthreads();
                among = every;
            }
            if (tid < n) {
                const uint32_t mine = among[tid];
                int above = 0, alike = 0;
#pragma unroll 8
                for (int i = 0; i < n; ++i) {
                    above += among[i] > mine;
                    alike += among[i] == mine;
                }
                if (above < need && above + alike >= need) {  // (equal ones write the same)
                    sh.digit = mine;
                    sh.need = need - above;
                }
            }
            __syncthreads();
            threshold = sh.digit;
            need = sh.need;
        }
    }
    // `need` is now how many weights equal to the threshold stay.  Of a thread's
    // positions: bit i of `certain` / `equal`: it stays for certain / its weight
    // equals the threshold.
    uint32_t certain = 0, equal = 0;
    auto classify = [&](int p0) {
        const int p = p0 + tid * kHeld;
        certain = equal = 0;
        if (p0 + warp * 32 * kHeld >= p_hi) return;
        if (compete) {  // a rank of 0 is neither above the threshold nor equal to it
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                certain |= held[i] > threshold ? 1u << i : 0u;
                equal |= held[i] == threshold ? 1u << i : 0u;
            }
        }
        if (all || p < lo || p + kHeld > hi) {  // some are forced, or past the share
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (p + i < p_hi && (all || p + i < lo || p + i >= hi)) certain |= 1u << i;
        }
    };
    int before = 0, equal_before = 0;  // kept positions and equal weights ahead of the batch
    if (coop) {
        int c = 0, e = 0;
        for (int p0 = p_lo; p0 < p_hi; p0 += kBatch) {
            if (!one_batch) load_batch(p0);
            classify(p0);
            c += __popc(certain);
            e += __popc(equal);
        }
        for (int o = 16; o > 0; o >>= 1) {
            c += __shfl_xor_sync(0xffffffffu, c, o);
            e += __shfl_xor_sync(0xffffffffu, e, o);
        }
        if (lane == 0) sh.warp_counts[0][warp] = c, sh.warp_counts[1][warp] = e;
        __syncthreads();
        if (tid < 2) {
            int sum = 0;
            for (int w = 0; w < kWarps; ++w) sum += sh.warp_counts[tid][w];
            sh.total[tid] = sum;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {
            before += *cluster.map_shared_rank(&sh.total[0], r);
            equal_before += *cluster.map_shared_rank(&sh.total[1], r);
        }
        before += min(equal_before, need);
    }
    for (int p0 = p_lo; p0 < p_hi; p0 += kBatch) {
        if (!one_batch) load_batch(p0);
        if (!one_batch || !coop) classify(p0);
        const int c = __popc(certain), e = __popc(equal);
        int c_inc = c, e_inc = e;  // inclusive over the warp
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, c_inc, o), y = __shfl_up_sync(0xffffffffu, e_inc, o);
            if (lane >= o) c_inc += x, e_inc += y;
        }
        __syncthreads();
        if (lane == 31) sh.warp_counts[0][warp] = c_inc, sh.warp_counts[1][warp] = e_inc;
        __syncthreads();
        if (warp < 2 && lane < kWarps) {  // warp 0 scans the certain ones, warp 1 the equal ones
            const unsigned active = (unsigned)((1ull << kWarps) - 1);
            const int x = sh.warp_counts[warp][lane];
            int inc = x;
            for (int o = 1; o < kWarps; o <<= 1) {
                const int y = __shfl_up_sync(active, inc, o);
                if (lane >= o) inc += y;
            }
            sh.warp_counts[warp][lane] = inc - x;
            if (lane == kWarps - 1) sh.batch[warp] = inc;
        }
        __syncthreads();
        int eq = equal_before + sh.warp_counts[1][warp] + e_inc - e;  // equal weights ahead of this thread
        int pos = before + sh.warp_counts[0][warp] + c_inc - c + min(eq, need) - min(equal_before, need);
        // the first need - eq of its equal weights stay
        uint32_t keep = certain;
        for (uint32_t left = equal; left != 0 && eq < need; left &= left - 1, ++eq) keep |= left & -left;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if ((keep >> i) & 1) list[pos++] = p0 + tid * kHeld + i;
        before += sh.batch[0] + min(equal_before + sh.batch[1], need) - min(equal_before, need);
        equal_before += sh.batch[1];
    }
    __syncthreads();
}

// The list where the caller wants it (with the -1s past the last kept position),
// and the length.
template <int kThreads>
__device__ __forceinline__ void write_index(const EvictArgs& a, int b, int h, int count, const int* list) {
    int* const index = a.index + ((size_t)b * a.n_kv_heads + h) * a.budget;
    if (list != index)
        for (int i = threadIdx.x; i < count; i += kThreads) index[i] = list[i];
    for (int i = count + threadIdx.x; i < a.budget; i += kThreads) index[i] = -1;
    if (threadIdx.x == 0 && h == 0) a.kept_lengths[b] = count;
}

// What goes with the rows: the kept weights (which = 0), K's (1) or V's row scales (2).
template <int kThreads, int kPerThread>
__device__ __forceinline__ void move_companions(const EvictArgs& a, int b, int h, int len, const int* list, int which) {
    const bool all = len <= a.budget;
    const float* const src = which == 0 ? a.weights : which == 1 ? a.scale_k : a.scale_v;
    float* const dst = which == 0 ? a.kept_weights : which == 1 ? a.scale_k : a.scale_v;
    if (!dst || (all && dst == src)) return;
    move_scalars<kThreads, kPerThread>(Rows(a, b, h), src, dst, list, min(len, a.budget));
}

// Moves column part `part` of the kept rows of K (which = 0) or V (1).
template <int kThreads>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int b, int h, int count, int which, int part,
                                          const int* list) {
    const int tid = threadIdx.x;
    const Rows row_of(a, b, h);
    uint8_t* const cache = static_cast<uint8_t*>(which ? a.cache_v : a.cache_k) + part * a.part_bytes;
    const int log_pieces = a.part_bytes == 64 ? 2 : 1;  // 16-byte pieces of a part (64 bytes, or a row of 32)
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
                x[i] = *reinterpret_cast<const uint4*>(cache + row_of(src[i]) * a.row_bytes + piece * 16);
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
                *reinterpret_cast<uint4*>(cache + row_of(j0 + row0 + i * step) * a.row_bytes + piece * 16) = x[i];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            x[i] = y[i];
            src[i] = next[i];
        }
    }
}

__global__ void __launch_bounds__(kFusedThreads, 4) evict_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ Shared<kFusedThreads, kFusedHeld> sh;
    __shared__ int s_list[kFusedThreads * kFusedHeld];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int bh = blockIdx.x / ranks, h = bh % a.n_kv_heads, b = bh / a.n_kv_heads;
    const int len = checked_length<kFusedThreads>(a, b);
    if (len < 0) {
        if (threadIdx.x == 0 && rank == 0 && h == 0) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
        return;
    }
    const bool coop = len > kFusedThreads * kFusedHeld;
    int* const list = coop ? a.index + (size_t)bh * a.budget : s_list;
    select_tokens(a, sh, cluster, b, h, len, coop, list);
    // the list is whole, and every CTA has read the weights it needs
    if (coop || a.kept_weights == a.weights) cluster.sync();
    if (rank == 0) write_index<kFusedThreads>(a, b, h, min(len, a.budget), list);
    if (rank == ranks - 1) move_companions<kFusedThreads, 8>(a, b, h, len, list, 0);
    if (rank < 2) move_companions<kFusedThreads, 8>(a, b, h, len, list, 1 + rank);
    if (len > a.budget) move_rows<kFusedThreads>(a, b, h, a.budget, rank & 1, rank >> 1, list);
}

__global__ void __launch_bounds__(kSelectThreads, 4) select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ Shared<kSelectThreads, kSelectHeld> sh;
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int bh = blockIdx.x / ranks, h = bh % a.n_kv_heads, b = bh / a.n_kv_heads;
    griddep_launch();
    const int len = checked_length<kSelectThreads>(a, b);
    if (len < 0) {
        if (threadIdx.x == 0 && rank == 0 && h == 0) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
        return;
    }
    const bool coop = ranks > 1 && len > kSelectThreads * kSelectHeld;
    int* const list = a.index + (size_t)bh * a.budget;
    if (coop || rank == 0) select_tokens(a, sh, cluster, b, h, len, coop, list);
    if (ranks > 1) cluster.sync();
    if (rank == 0) write_index<kSelectThreads>(a, b, h, min(len, a.budget), list);
}

// (out of line: inlined, it makes the movers' registers spill, which cost 30 us of 45)
__device__ __noinline__ void move_companions_of_movers(const EvictArgs& a, int b, int h, int len, const int* list,
                                                       int which) {
    move_companions<kMoveThreads, 4>(a, b, h, len, list, which);
}

// CTAs first for the column parts of K and V, of all heads, then for what goes with
// them (weights, K's scales, V's; `others` of the three).  (The select kernel moving
// these itself: 64 sequences in int8 pages 74.3 us a call against 62.7, 16 of 16384
// tokens 116.5 against 110.7.)
__global__ void __launch_bounds__(kMoveThreads, 7) move_kernel(const __grid_constant__ EvictArgs a, int parts, int others) {
    const int heads = a.num_seqs * a.n_kv_heads, movers = 2 * parts * heads;
    const bool mover = (int)blockIdx.x < movers;
    const int x = mover ? blockIdx.x : blockIdx.x - movers, per = mover ? 2 * parts : others;
    const int bh = x / per, what = x % per, h = bh % a.n_kv_heads, b = bh / a.n_kv_heads;
    const int len = checked_length<kMoveThreads>(a, b);
    griddep_wait();
    const int* const list = a.index + (size_t)bh * a.budget;
    if (!mover) {
        // (every weight has been read: they may move in place)
        const int first = a.kept_weights ? 0 : 1;
        if (len >= 0) move_companions_of_movers(a, b, h, len, list, what + first);
    } else if (len > a.budget) {
        move_rows<kMoveThreads>(a, b, h, a.budget, what / parts, what % parts, list);
    }
}

}  // namespace

// `sms`: SMs of the device; *launches: kernels enqueued.
cudaError_t launch_evict(const EvictArgs& args, int sms, int* launches, cudaStream_t stream) {
    EvictArgs a = args;
    a.part_bytes = a.row_bytes < 64 ? a.row_bytes : 64;
    const int parts = a.row_bytes / a.part_bytes, heads = a.num_seqs * a.n_kv_heads;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    if (2ll * parts * heads <= 2ll * sms) {
        attr[0].val.clusterDim.x = (unsigned)(2 * parts);
        cfg.gridDim = dim3((unsigned)(2 * parts * heads));
        cfg.blockDim = dim3(kFusedThreads);
        *launches = 1;
        return cudaLaunchKernelEx(&cfg, evict_kernel, a);
    }
    int ranks = 1;
    while (ranks < 8 && a.max_cache_len > ranks * kSelectThreads * kSelectHeld) ranks *= 2;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    cfg.gridDim = dim3((unsigned)(ranks * heads));
    cfg.blockDim = dim3(kSelectThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, a);
    if (e != cudaSuccess) return e;
    const int others = (a.kept_weights ? 1 : 0) + (a.scale_k ? 2 : 0);
    cfg.gridDim = dim3((unsigned)((2 * parts + others) * heads));
    cfg.blockDim = dim3(kMoveThreads);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    *launches = 2;
    return cudaLaunchKernelEx(&cfg, move_kernel, a, parts, others);
}

}  // namespace pa
