// schedule_long.cuh -- the plan of the long-context variant: how its units are cut
// and ordered.  A kernel of one CTA lays the list out (schedule_long.cu), or,
// for a few sequences, every CTA of the attention kernel works it out for itself
// and keeps the units that are its own.
//
// The list is laid out as in schedule.cu (sequences by descending cost, KV
// heads in L2-sized groups, blocks last to first), with two additions:
//  - a prefix that the batch shares is one more sequence, whose query blocks
//    are cut from the whole batch's tokens and see the prefix's tiles only;
//  - query blocks with many tiles are cut into pieces along the keys, so that
//    a few long rows still fill the GPU.  The pieces of a block write partial
//    results (fp32 output and log-sum-exp) into slabs that merge_kernel joins.
//
// Piece size (piece_tiles): with fewer units than CTAs, what makes one round of
// pieces; else the whole call's tiles over twice the CTAs; at least min_tiles.  A
// sequence that would gain less than kCutGain tiles by it is not cut, unless the
// call merges anyway.  (Decode rows of 8 KV heads, graph: one row of 10 tiles whole
// 16.3 us, in pieces of 4 14.8; of 34 tiles 36.3 and 17.5; eight rows of 34 tiles
// 40.4 and 34.2.)
// All blocks of a sequence get the same number of pieces (that of its longest
// block); a block with fewer tiles than pieces leaves holes in the list.  Of a
// prefix with more units than CTAs, whole rounds of units stay uncut and only the
// rest is cut, so that the last round is short (16 questions over an 8191-token
// prefix, 256 units of 64 tiles on 152 CTAs: 112 tiles for the busiest CTA where
// halves of every unit made it 128, for about the same partial results; 296 ->
// 285 us a call).
#pragma once

#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "schedule.cuh"

namespace pa {

constexpr int kCutGain = 4;

__device__ __forceinline__ int piece_tiles(unsigned long long tiles, unsigned long long units, int num_ctas, int min_tiles) {
    const unsigned long long over = units < (unsigned)num_ctas ? num_ctas - units / 2 : 2ull * (unsigned)num_ctas;
    const unsigned long long piece = (tiles + over - 1) / over;
    return max(min_tiles, (int)(piece < 0x7fffffffull ? piece : 0x7fffffffull));
}

// Pieces of a sequence whose longest block has mx tiles.
__device__ __forceinline__ int pieces_of(int mx, int piece, bool merged_anyway, int most) {
    if (!merged_anyway && mx <= piece + kCutGain) return 1;
    return max(1, min((mx + piece - 1) / piece, most));
}

// Writes the units of query block blk of sequence b and KV head kvh: the block's
// c tiles in its sequence's p pieces, or in one where the block is among the
// sequence's first `whole` ones.  emit(list position, unit, sequence); the lead
// CTA writes what the merge reads.
template <class Emit>
__device__ __forceinline__ void emit_block(const LongScheduleArgs& a, const SeqInfo& si, int b, int blk, int kvh,
                                           int nblk, int hg, int p, int whole, int first, int tpu, int c, bool lead,
                                           const Emit& emit) {
    const bool pre = b == a.num_seqs, partial = a.prefix_len > 0 || p > 1;
    const int g0 = kvh - kvh % hg, gsize = min(hg, a.n_kv_heads - g0);
    const int rank = g0 * nblk + (nblk - 1 - blk) * gsize + (kvh - g0);
    const int pos = first + (rank < whole ? rank : whole + (rank - whole) * p);
    if (rank < whole) p = 1;
    const int pb = min(p, c);  // pieces of this block
    for (int k = 0, s0 = 0; k < p && pos + k < a.max_units; ++k) {
        // c < 2^24 tiles and k <= 32 pieces: the product fits 32 bits
        const int s1 = k < pb ? (int)((unsigned)c * (unsigned)(k + 1) / (unsigned)pb) : s0;
        UnitX x;
        x.u = Unit{b, kvh, blk * tpu, s1 - s0};
        x.s0 = s0;
        x.slab = partial ? (pre ? a.max_pieces : 0) + k : -1;
        emit(pos + k, x, si);
        s0 = s1;
    }
    if (!lead) return;
    if (pre) a.pre_pieces[blk * a.n_kv_heads + kvh] = pb;
    if (a.tok_pieces && partial && !pre && kvh == 0)
        for (int t = blk * tpu; t < min(si.n, (blk + 1) * tpu); ++t) a.tok_pieces[si.q_start + t] = pb;
}

// How a prefix of U units of `tiles` each (U > CTAs) is cut: `whole` units stay
// uncut, the others get the pieces that make their rounds shortest (a piece
// costs about one tile more: its start, its partial results).
__device__ __forceinline__ int cut_rest(int units, int tiles, int num_ctas, int max_pieces, int min_tiles, int* whole) {
    *whole = units / num_ctas * num_ctas;
    const int rest = units - *whole;
    int best = 1, best_cost = 0x7fffffff;
    for (int p = 1; p <= max_pieces && (p == 1 || tiles >= p * min_tiles); ++p) {
        const int cost = (rest * p + num_ctas - 1) / num_ctas * ((tiles + p - 1) / p + 1);
        if (cost < best_cost) best = p, best_cost = cost;
    }
    return best;
}

// What planning for a few sequences (kFewSeqs, see schedule.cuh) keeps in shared memory.
struct LongPlan {
    FewSeqs f;
    int max[kFewSeqs], tiles[kFewSeqs], pieces[kFewSeqs];  // longest block, tiles per head, pieces
    int whole, units;
};

// Plans a call of a few sequences (one CTA of at least kFewSeqs threads): every
// unit goes to emit(list position, unit, sequence).  lead: this CTA writes what the
// merge reads and reports bad metadata; shared: the list is for other CTAs
// (its header and the sequences are written too).
template <class Emit>
__device__ __forceinline__ void plan_few(const LongScheduleArgs& a, LongPlan& plan, bool lead, bool shared,
                                         const Emit& emit) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tpu = a.unit_slots * (kBlockM / a.group);
    const bool shared_prefix = a.prefix_len > 0, paged = a.block_table != nullptr;
    const int nseq = a.num_seqs + (shared_prefix ? 1 : 0);
    if (lead && a.tok_pieces)
        for (int t = tid; t < a.total_q; t += blockDim.x) a.tok_pieces[t] = 0;
    FewSeqs& f = plan.f;
    load_few(a, f, a.sinks, a.prefix_table, a.prefix_len, lead);
    auto block_tiles = [&](const SeqInfo& si, int blk, bool pre) {
        const int q0 = blk * tpu, qe = q0 + tpu < si.n ? q0 + tpu : si.n;
        const StreamGeo g = stream_geo(si.n, si.P, q0, qe, a.causal, a.window, a.sinks, pre, paged);
        return g.nsink + g.hi - g.lo;
    };
    // tiles per head and longest block: by one thread, or by a warp where there are many blocks
    constexpr int kThreadBlocks = 4;
    if (tid == 0) plan.units = 0;
    __syncthreads();
    if (tid < nseq) {
        const SeqInfo si = f.seqs[tid];
        const int nblk = (si.n + tpu - 1) / tpu;
        f.blocks[tid] = nblk;
        atomicAdd(&plan.units, nblk * a.n_kv_heads);
        if (nblk <= kThreadBlocks) {
            int c = 0, mx = 0;
            for (int i = 0; i < nblk; ++i) {
                const int t = block_tiles(si, i, tid == a.num_seqs);
                c += t;
                mx = max(mx, t);
            }
            plan.tiles[tid] = c;
            plan.max[tid] = mx;
            if (c > 0) atomicAdd(&f.total, (unsigned long long)c * a.n_kv_heads);
        }
    }
    __syncthreads();
    for (int b = warp; b < nseq; b += blockDim.x / 32) {
        const int nblk = f.blocks[b];
        if (nblk <= kThreadBlocks) continue;
        const SeqInfo si = f.seqs[b];
        int c = 0, mx = 0;
        for (int i = lane; i < nblk; i += 32) {
            const int t = block_tiles(si, i, b == a.num_seqs);
            c += t;
            mx = max(mx, t);
        }
        for (int o = 16; o > 0; o >>= 1) {
            c += __shfl_xor_sync(0xffffffffu, c, o);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        if (lane == 0) {
            plan.tiles[b] = c;
            plan.max[b] = mx;
            atomicAdd(&f.total, (unsigned long long)c * a.n_kv_heads);
        }
    }
    __syncthreads();
    if (tid < nseq) {
        const int piece = piece_tiles(f.total, (unsigned)plan.units, a.num_ctas, a.min_tiles);
        const int c = plan.tiles[tid], mx = plan.max[tid];
        int p = pieces_of(mx, piece, shared_prefix, tid == a.num_seqs ? a.max_prefix_pieces : a.max_pieces);
        const int units = f.blocks[tid] * a.n_kv_heads;
        int whole = 0;
        if (tid == a.num_seqs) {
            if (units > a.num_ctas) p = cut_rest(units, mx, a.num_ctas, a.max_prefix_pieces, a.min_tiles, &whole);
            plan.whole = whole;
        }
        plan.pieces[tid] = p;
        f.units[tid] = whole + (units - whole) * p;
        f.cost[tid] = (float)c / (float)p;
        f.group[tid] =
            kv_head_group(f.seqs[tid], a.head_dim, a.n_kv_heads, a.num_ctas, (long long)c, (mx + p - 1) / p);
    }
    __syncthreads();
    const int total_blocks = rank_few(a, f, nseq, shared);
    for (int w = tid; w < total_blocks * a.n_kv_heads; w += blockDim.x) {
        const int i = w / a.n_kv_heads, kvh = w % a.n_kv_heads;
        const int b = block_owner(f.seqs, nseq, i);
        emit_block(a, f.seqs[b], b, i - f.seqs[b].pad, kvh, f.blocks[b], f.group[b], plan.pieces[b],
                   b == a.num_seqs ? plan.whole : 0, f.first[b], tpu,
                   block_tiles(f.seqs[b], i - f.seqs[b].pad, b == a.num_seqs), lead, emit);
    }
}

}  // namespace pa
