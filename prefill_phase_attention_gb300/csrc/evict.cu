// evict.cu -- eviction from a KV cache by accumulated attention weight.
//
// Per (sequence, KV head) of a cache of L tokens, L > budget: the first
// `sinks` and the last `recent` tokens stay, and of the tokens between them
// the m = budget - sinks - recent with the largest weight (ties: the lowest
// position first; NaN ranks above everything).  The kept rows of K and V move
// to positions 0 .. budget - 1 in their old order, in place.  L <= budget keeps
// every token.
//
// select_kernel (one CTA per (sequence, head)): the m-th largest weight by a
// radix select, 8 bits of the order-preserving integer image per pass, then
// one pass over the positions that writes the kept positions in order, and the
// kept weights and row scales.
// move_kernel (one CTA per (sequence, head, K or V)): copies row index[j] to
// row j in increasing j.  index[j] >= j, so a chunk of rows may be written once
// all of ITS sources are read: later chunks read at or past their own start.
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveVec = 8;  // 16-byte pieces per thread and chunk

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
    if (a.block_table && !bad) {
        const int nb = (len + (1 << a.block_log2) - 1) >> a.block_log2;
        for (int i = threadIdx.x; i < nb; i += blockDim.x) {
            const int blk = a.block_table[(size_t)b * a.max_blocks + i];
            bad |= blk < 0 || blk >= a.num_blocks;
        }
    }
    return __syncthreads_or(bad) ? -1 : len;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int warp_sums[2][32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    griddep_launch();
    const int h = blockIdx.x % a.n_kv_heads, b = blockIdx.x / a.n_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int len = checked_length(a, b);
    if (len < 0) {
        if (tid == 0 && h == 0) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
        return;
    }
    int* index = a.index + (size_t)blockIdx.x * a.budget;
    const int count = min(len, a.budget);
    const bool all = len <= a.budget;
    const int lo = a.sinks, hi = len - a.recent;  // the tokens that compete (when !all)
    uint32_t threshold = 0;
    int need = a.budget - a.sinks - a.recent;  // of them kept
    if (!all && need > 0) {
        if (tid == 0) s_prefix = 0, s_need = need;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int p = lo + tid; p < hi; p += kSelThreads) {
                const uint32_t r = rank_bits(a.weights[cache_row(a, b, h, p)]);
                if ((r & mask) == prefix) atomicAdd(&hist[(r >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = s_need, bin = 255;
                while (bin > 0 && hist[bin] < left) left -= hist[bin--];
                s_prefix = prefix | ((uint32_t)bin << shift);
                s_need = left;  // how many with this digit (and, at the end, equal to the threshold)
            }
            __syncthreads();
        }
        threshold = s_prefix;
        need = s_need;
    }
    // kept positions in order: weights above the threshold, the first `need` equal to it
    int base = 0, equals = 0;
    for (int p0 = 0; p0 < len; p0 += kSelThreads) {
        const int p = p0 + tid;
        const bool in = p < len;
        size_t src = 0;
        float w = 0.f, sk = 0.f, sv = 0.f;
        if (in) {
            src = cache_row(a, b, h, p);
            w = a.weights[src];
            if (a.scale_k) sk = a.scale_k[src], sv = a.scale_v[src];
        }
        const bool forced = in && (all || p < lo || p >= hi);
        const uint32_t r = rank_bits(w);
        const bool compete = in && !forced && a.budget > a.sinks + a.recent;
        const bool eq = compete && r == threshold;
        const unsigned eqm = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) warp_sums[0][warp] = __popc(eqm);
        __syncthreads();
        int eq_before = equals, eq_total = 0;
        for (int i = 0; i < 32; ++i) {
            eq_before += i < warp ? warp_sums[0][i] : 0;
            eq_total += warp_sums[0][i];
        }
        eq_before += __popc(eqm & ((1u << lane) - 1));
        const bool keep = forced || (compete && r > threshold) || (eq && eq_before < need);
        const unsigned km = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) warp_sums[1][warp] = __popc(km);
        __syncthreads();
        int pos = base, total = 0;
        for (int i = 0; i < 32; ++i) {
            pos += i < warp ? warp_sums[1][i] : 0;
            total += warp_sums[1][i];
        }
        pos += __popc(km & ((1u << lane) - 1));
        if (keep) {
            index[pos] = p;
            const size_t dst = cache_row(a, b, h, pos);
            if (a.kept_weights) a.kept_weights[dst] = w;  // pos <= p: in place, this chunk was read above
            if (a.scale_k) a.scale_k[dst] = sk, a.scale_v[dst] = sv;
        }
        base += total;
        equals += eq_total;
        __syncthreads();
    }
    for (int i = count + tid; i < a.budget; i += kSelThreads) index[i] = -1;
    if (tid == 0 && h == 0) a.kept_lengths[b] = count;
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a) {
    griddep_wait();
    const int which = blockIdx.x & 1, bh = blockIdx.x >> 1;
    const int h = bh % a.n_kv_heads, b = bh / a.n_kv_heads;
    const int len = checked_length(a, b);
    if (len <= a.budget) return;  // rejected, or nothing to evict
    uint8_t* cache = static_cast<uint8_t*>(which ? a.cache_v : a.cache_k);
    const int* index = a.index + (size_t)bh * a.budget;
    const int pieces = a.row_bytes / 16;  // 2 .. 16, a power of two
    const int rows = kMoveThreads * kMoveVec / pieces;
    for (int j0 = 0; j0 < a.budget; j0 += rows) {
        uint4 x[kMoveVec];
        int j[kMoveVec];
#pragma unroll
        for (int i = 0; i < kMoveVec; ++i) {
            const int piece = threadIdx.x + i * kMoveThreads;
            j[i] = j0 + piece / pieces;
            if (j[i] < a.budget)
                x[i] = *reinterpret_cast<const uint4*>(cache + cache_row(a, b, h, index[j[i]]) * a.row_bytes +
                                                       (piece % pieces) * 16);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMoveVec; ++i) {
            const int piece = threadIdx.x + i * kMoveThreads;
            if (j[i] < a.budget)
                *reinterpret_cast<uint4*>(cache + cache_row(a, b, h, j[i]) * a.row_bytes + (piece % pieces) * 16) = x[i];
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    select_kernel<<<a.num_seqs * a.n_kv_heads, kSelThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * a.num_seqs * a.n_kv_heads));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, move_kernel, a);
}

}  // namespace pa
