// schedule_long.cu -- tile scheduler and merge of the long-context variant (the
// plan itself: schedule_long.cuh).
#include <cuda_bf16.h>

#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"
#include "ptx.cuh"
#include "schedule.cuh"
#include "schedule_long.cuh"

namespace pa {

namespace {

__global__ void __launch_bounds__(1024) build_long_schedule_kernel(const __grid_constant__ LongScheduleArgs a) {
    __shared__ int hist[kCostBins];
    __shared__ int warp_sums[32];
    __shared__ unsigned long long s_total;
    __shared__ SeqInfo s_seqs[kSmemSeqs];
    __shared__ int s_scratch[kSmemSeqs], s_group[kSmemSeqs], s_pieces[kSmemSeqs];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nthr = blockDim.x, nwarps = nthr >> 5;
    const int tpu = a.unit_slots * (kBlockM / a.group);  // query tokens per unit
    const bool shared_prefix = a.prefix_len > 0;
    const int nseq = a.num_seqs + (shared_prefix ? 1 : 0);
    griddep_launch();
    const bool small = nseq <= kSmemSeqs;
    SeqInfo* const seqs = small ? s_seqs : a.seqs;
    int* const seq_scratch = small ? s_scratch : a.seq_scratch;
    int* const seq_group = small ? s_group : a.seq_group;
    int* const pieces = small ? s_pieces : a.seq_pieces;

    for (int i = tid; i < kCostBins; i += nthr) hist[i] = 0;
    if (tid == 0) s_total = 0;

    // Pass 1: sanitise each sequence (its metadata, then its table's blocks; a
    // bad block of the prefix rejects them all); number its query blocks.
    const bool paged = a.block_table != nullptr;
    for (int b = tid; b < a.num_seqs; b += nthr) seqs[b] = checked_sequence(a, b);
    bool bad_prefix = false;
    if (paged) {
        __threadfence_block();
        __syncthreads();
        for (int b = warp; b < a.num_seqs; b += nwarps) {
            const bool bad = bad_visible_blocks(a.block_table + (size_t)b * a.max_blocks, seqs[b], a.block_size,
                                                a.num_blocks, a.causal, a.window, a.sinks, lane);
            if (bad && lane == 0) seqs[b].n = -1;
        }
        if (shared_prefix) {
            const int nb = (a.prefix_len + a.block_size - 1) / a.block_size, part = (nb + nwarps - 1) / nwarps;
            bad_prefix = bad_blocks(a.prefix_table, warp * part, min(nb, (warp + 1) * part), a.num_blocks, lane);
        }
        __threadfence_block();
        bad_prefix = __syncthreads_or(bad_prefix);
    }
    int blocks_before = 0;
    for (int b0 = 0; b0 < nseq; b0 += nthr) {
        const int b = b0 + tid;
        SeqInfo si{0, 0, 0, 0};
        if (b < a.num_seqs) {
            si = seqs[b];
            if (si.n < 0 || bad_prefix) {
                atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
                si = SeqInfo{0, 0, 0, 0};
            }
        } else if (b == a.num_seqs && shared_prefix && !bad_prefix) {
            const int end = a.cu_seqlens_q[a.num_seqs];
            si.n = end < 0 ? 0 : (end < a.total_q ? end : a.total_q);
            si.P = a.prefix_len;
        }
        const int nblk = (si.n + tpu - 1) / tpu;
        int chunk_total;
        const int excl = block_exclusive_scan(nblk, warp_sums, &chunk_total);
        si.pad = blocks_before + excl;
        if (b < nseq) {
            a.seqs[b] = si;
            if (small) s_seqs[b] = si;
        }
        blocks_before += chunk_total;
    }
    const int total_blocks = blocks_before;
    if (a.tok_pieces)
        for (int t = tid; t < a.total_q; t += nthr) a.tok_pieces[t] = 0;
    __threadfence_block();
    __syncthreads();

    // tiles of the stream of query block blk of sequence si
    auto block_tiles = [&](const SeqInfo& si, int blk, bool pre) {
        const int q0 = blk * tpu, qe = q0 + tpu < si.n ? q0 + tpu : si.n;
        const StreamGeo g = stream_geo(si.n, si.P, q0, qe, a.causal, a.window, a.sinks, pre, paged);
        return g.nsink + g.hi - g.lo;
    };

    // Pass 2 (one warp per sequence): its tiles per head and its longest block.
    for (int b = warp; b < nseq; b += nwarps) {
        const SeqInfo si = seqs[b];
        const int nblk = (si.n + tpu - 1) / tpu;
        long long c = 0;
        int mx = 0;
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
            seq_scratch[b] = (int)(c < 0x7fffffffll ? c : 0x7fffffffll);
            seq_group[b] = mx;
            if (c > 0) atomicAdd(&s_total, (unsigned long long)c * a.n_kv_heads);
        }
    }
    __threadfence_block();
    __syncthreads();

    // Pieces per block, the sequence's cost bin and its KV-head group.
    const int piece = piece_tiles(s_total, (unsigned long long)total_blocks * a.n_kv_heads, a.num_ctas, a.min_tiles);
    for (int b = tid; b < nseq; b += nthr) {
        const SeqInfo si = seqs[b];
        const int nblk = (si.n + tpu - 1) / tpu;
        const int c = seq_scratch[b], mx = seq_group[b];
        const bool pre = b == a.num_seqs;
        const int p = pieces_of(mx, piece, shared_prefix, pre ? a.max_prefix_pieces : a.max_pieces);
        pieces[b] = p;
        if (nblk > 0) {
            const int bin = cost_bin((long long)c * a.n_kv_heads / p);
            seq_scratch[b] = bin;
            seq_group[b] = kv_head_group(si, a.head_dim, a.n_kv_heads, a.num_ctas, c, (mx + p - 1) / p);
            atomicAdd(&hist[bin], nblk * a.n_kv_heads * p);
        }
    }
    __threadfence_block();
    __syncthreads();

    // Exclusive scan in descending cost order.
    static_assert(kCostBins == 2 * 1024, "scan assumes two bins per thread");
    const int r0 = kCostBins - 1 - 2 * tid;
    const int h0 = hist[r0], h1 = hist[r0 - 1];
    int total;
    const int excl = block_exclusive_scan(h0 + h1, warp_sums, &total);
    hist[r0] = excl;
    hist[r0 - 1] = excl + h0;
    if (tid == 0) {
        a.hdr->num_units = total < a.max_units ? total : a.max_units;
        a.hdr->counter = 0;
        a.hdr->max_units = a.max_units;
        if (total > a.max_units) atomicOr(&a.hdr->error, PA_DEVERR_OVERFLOW);
    }
    __syncthreads();

    // Pass 3: each sequence claims its range of the list ...
    for (int b = tid; b < nseq; b += nthr) {
        const int nblk = (seqs[b].n + tpu - 1) / tpu;
        if (nblk > 0) seq_scratch[b] = atomicAdd(&hist[seq_scratch[b]], nblk * a.n_kv_heads * pieces[b]);
    }
    __threadfence_block();
    __syncthreads();

    // ... and its units go there.
    const int total_units = total_blocks * a.n_kv_heads;
    for (int w = tid; w < total_units; w += nthr) {
        const int i = w / a.n_kv_heads, kvh = w % a.n_kv_heads;
        const int b = block_owner(seqs, nseq, i);
        const SeqInfo si = seqs[b];
        emit_block(a, si, b, i - si.pad, kvh, (si.n + tpu - 1) / tpu, seq_group[b], pieces[b], 0, seq_scratch[b], tpu,
                   block_tiles(si, i - si.pad, b == a.num_seqs), true,
                   [&](int pos, const UnitX& x, const SeqInfo&) { a.xunits[pos] = x; });
    }
}

// The same for a few sequences (kFewSeqs).
__global__ void __launch_bounds__(kFewThreads) build_long_schedule_few_kernel(const __grid_constant__ LongScheduleArgs a) {
    __shared__ LongPlan plan;
    griddep_launch();
    plan_few(a, plan, true, true, [&](int pos, const UnitX& x, const SeqInfo&) { a.xunits[pos] = x; });
}

// One row (token, head) per D / 4 lanes.  The lanes fetch the row's log-sum-exps
// together (one load deep, whatever the number of slabs) and share their weights
// by shuffles; the slabs' outputs are fetched eight at a time, the first eight
// while the log-sum-exps are on their way.  The launch is bound by these latencies
// for a few rows and by L2 for many (the slabs were just written); many rows go
// four to a lane group, their slab counts looked up together.  (59000 rows of 3.5
// slabs on average, D = 128, cold caches: 35 us with one row each, 30 with four, 37
// with the first slabs of all four fetched ahead, at 80 registers; the whole call of
// 2048 rows 134 with one, 141 with four.)
template <int D, int kRows>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ MergeArgs a) {
    constexpr int kLanes = D / 4, kAtOnce = kRows == 1 ? 8 : 4, kGroups = 256 / kLanes;
    griddep_wait();
    const long long rows = (long long)a.total_q * a.n_heads;
    const long long first = (long long)blockIdx.x * (kRows * kGroups) + threadIdx.x / kLanes;
    const int l = threadIdx.x % kLanes;
    const unsigned lanes = kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1) << (threadIdx.x % 32 / kLanes * kLanes);
    int owns[kRows], all[kRows];  // slabs of the row: its token's own ones, and with its prefix unit's
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const long long row = first + k * kGroups;
        owns[k] = all[k] = 0;
        if (row >= rows) continue;
        const int token = (int)(row / a.n_heads), head = (int)(row % a.n_heads);
        owns[k] = a.tok_pieces[token];
        if (a.pre_pieces) all[k] = a.pre_pieces[token / a.tokens_per_block * (a.n_heads / a.group) + head / a.group];
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const long long row = first + k * kGroups;
        const int own = owns[k], n = own + all[k];
        if (own == 0) continue;  // not this call's, or written by its unit (the row's lanes agree)
        auto slab = [&](int i) { return (size_t)(i < own ? i : a.prefix_slab + i - own) * rows + row; };
        // (an empty piece's output was not written: whatever it holds gets no part)
        float4 o[kAtOnce];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (i0 + i < n) o[i] = *reinterpret_cast<const float4*>(a.part_o + slab(i0 + i) * D + 4 * l);
        };
        fetch(0);
        // lane l holds slabs l, l + kLanes, ...; at most kMaxSlabs in all
        constexpr int kHeld = (kMaxSlabs + kLanes - 1) / kLanes;
        float w[kHeld], m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            w[h] = h * kLanes + l < n ? a.part_lse[slab(h * kLanes + l)] : -INFINITY;
            m = fmaxf(m, w[h]);
        }
        for (int x = kLanes / 2; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, x));
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            w[h] = w[h] == -INFINITY ? 0.f : exp2f(w[h] - m);
            sum += w[h];
        }
        for (int x = kLanes / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(lanes, sum, x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        static_assert(kLanes % kAtOnce == 0, "the slabs fetched at once have their weights in one register");
#pragma unroll
        for (int i0 = 0; i0 < kMaxSlabs; i0 += kAtOnce) {
            if (i0 >= n) break;
            if (i0 > 0) fetch(i0);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float wi = __shfl_sync(lanes, w[i0 / kLanes], (i0 + i) % kLanes, kLanes);
                if (i0 + i >= n || wi == 0.f) continue;
                acc.x = fmaf(wi, o[i].x, acc.x);
                acc.y = fmaf(wi, o[i].y, acc.y);
                acc.z = fmaf(wi, o[i].z, acc.z);
                acc.w = fmaf(wi, o[i].w, acc.w);
            }
        }
        const float inv = 1.f / sum;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        const uint2 packed = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        *reinterpret_cast<uint2*>(a.out + row * D + 4 * l) = packed;
        if (l == 0 && a.lse) a.lse[row] = (m + log2f(sum)) * 0.69314718055994530942f;
    }
}

}  // namespace

cudaError_t launch_build_long_schedule(const LongScheduleArgs& a, cudaStream_t stream) {
    if (a.num_seqs + (a.prefix_len > 0 ? 1 : 0) <= kFewSeqs)
        build_long_schedule_few_kernel<<<1, kFewThreads, 0, stream>>>(a);
    else
        build_long_schedule_kernel<<<1, 1024, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_merge(const MergeArgs& a, int head_dim, int sms, cudaStream_t stream) {
    const long long threads = (long long)a.total_q * a.n_heads * (head_dim / 4), ctas = (threads + 255) / 256;
    const bool many = ctas >= 8ll * sms;  // more than run at once even so
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(many ? (ctas + 3) / 4 : ctas));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (head_dim) {
        case 32: return cudaLaunchKernelEx(&cfg, many ? merge_kernel<32, 4> : merge_kernel<32, 1>, a);
        case 64: return cudaLaunchKernelEx(&cfg, many ? merge_kernel<64, 4> : merge_kernel<64, 1>, a);
        default: return cudaLaunchKernelEx(&cfg, many ? merge_kernel<128, 4> : merge_kernel<128, 1>, a);
    }
}

}  // namespace pa
