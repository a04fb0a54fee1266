// cache4.cu -- writing keys and values into the 4-bit cache, reading them back, and
// the check of an attention call's sequences.
//
// Both copies are one pass over the rows, which the bytes bound: a lane takes 16
// channels (32 bytes of bf16, 8 of codes), head_dim / 16 lanes a row, and consecutive
// rows of lanes take consecutive tokens of one KV head, whose rows lie side by side in
// the cache.  A block takes 32 tokens and some heads of K and V; the tokens' sequences,
// positions and table entries are looked up once a block, in shared memory.  A block
// looks whether its sequences' tables are valid itself: a kernel ahead for that
// costs a small call more than all of it.
#include <algorithm>

#include "cache4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyTokens = 32;  // of a block
constexpr int kInFlight = 4;     // rows of a thread
constexpr int kCuInSmem = 1024;  // sequences whose boundaries are searched in shared memory

struct Places {
    int cu[kCuInSmem];
    int seq[kCopyTokens], pos[kCopyTokens];
    int last[kCopyTokens];        // of the token's sequence: its last position, its first token
    int first[kCopyTokens];

    size_t rows[kCopyTokens];     // row of KV head 0, ~0: none; another head's is `stride` rows on
};

// Where the rows of tokens [t0, t0 + kCopyTokens) are.  Ends with a barrier.
__device__ __forceinline__ void locate_tokens(const Sequences4& a, const Cache4& c, int t0, Places& at, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool in_smem = a.num_seqs <= kCuInSmem;
    if (in_smem) {
        for (int b = tid; b < a.num_seqs; b += kCopyThreads) at.cu[b] = a.cu_seqlens_q[b];
        __syncthreads();
    }
    if (tid < kCopyTokens) {
        const int t = t0 + tid;
        at.rows[tid] = ~size_t(0);
        at.seq[tid] = -1;
        
        if (t < a.total_q) {
            // the sequence owning token t: the last b with cu_seqlens_q[b] <= t
            int lo = 0, hi = a.num_seqs - 1;
            while (lo < hi) {
                const int mid = lo + (hi - lo + 1) / 2;
                if ((in_smem ? at.cu[mid] : a.cu_seqlens_q[mid]) <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const SeqInfo s = sequence4(a, c.max_cache_len, lo);
            if (t >= s.q_start && t < (long long)s.q_start + s.n) {
                at.seq[tid] = lo;
                at.pos[tid] = s.P + (t - s.q_start);
                at.first[tid] = s.P;
                at.last[tid] = s.P + s.n - 1;
                at.rows[tid] = row4(c, lo, 0, at.pos[tid]);
            }
        }
    }
    __syncthreads();
    if (c.block_table && !a.checked) {
        // a sequence with an entry outside the pool is skipped whole: the block's sequences,
        // a warp each
        for (int i = warp; i < kCopyTokens; i += kCopyThreads / 32) {
            const int b = at.seq[i];
            if (b < 0 || (i > 0 && at.seq[i - 1] == b)) continue;
            const int32_t* table = c.block_table + (size_t)b * c.max_blocks;
            const int end = (at.last[i] >> c.block_log2) + 1;
            bool bad = false;
#pragma unroll 8
            for (int e = (at.first[i] >> c.block_log2) + lane; e < end; e += 32)
                bad |= (unsigned)__ldg(table + e) >= (unsigned)c.num_blocks;
            if (!__any_sync(0xffffffffu, bad)) continue;
            if (lane == 0) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
            if (i + lane < kCopyTokens && at.seq[i + lane] == b) at.rows[i + lane] = ~size_t(0);
        }
        __syncthreads();
    }
    if (!a.checked && report)
        for (int b = tid; b < a.num_seqs; b += kCopyThreads)
            if (stated_sequence(a, c.max_cache_len, b).n < 0) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
}

// Rows of a block: heads [h0, h1) of K then V, 32 tokens each; a thread takes every
// kStep-th of them, `first` on, and channels [16 part, 16 part + 16).
template <int D>
struct Rows {
    static constexpr int kLanes = D / 16;
    static constexpr int kStep = kCopyThreads / kLanes;
    static_assert(kStep % kCopyTokens == 0 || kCopyTokens % kStep == 0, "a pass is whole heads or part of one");
    int part = threadIdx.x % kLanes, first = threadIdx.x / kLanes, h0, items;
    __device__ __forceinline__ Rows(int n_kv_heads, int heads, int heads_at) {
        h0 = heads_at * heads;
        items = (min(2 * n_kv_heads, h0 + heads) - h0) * kCopyTokens;
    }
    __device__ __forceinline__ int token(int it) const { return it % kCopyTokens; }
    __device__ __forceinline__ int head(int it) const { return h0 + it / kCopyTokens; }
};

// Tokens [32 tokens_at, ...) and heads [heads_at * p.heads, ...) of k and v into the cache.
template <int D>
__device__ __forceinline__ void write_rows4(const Copy4Params& p, Places& at, int tokens_at, int heads_at) {
    const int Hk = p.cache.n_kv_heads, groups = p.cache.groups, group_lanes = D / 16 / groups;
    const size_t stride = p.cache.block_table ? (size_t)1 << p.cache.block_log2 : (size_t)p.cache.max_cache_len;
    const int t0 = tokens_at * kCopyTokens;
    const Rows<D> r(Hk, p.heads, heads_at);
    constexpr int kStep = Rows<D>::kStep;
    uint4 x[kInFlight][2];
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int it = i0 + u * kStep, t = t0 + r.token(it), h = r.head(it);
            x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
            if (it < r.items && t < p.seqs.total_q) {
                const uint4* src =
                    reinterpret_cast<const uint4*>((h < Hk ? p.k : p.v) + ((size_t)t * Hk + (h < Hk ? h : h - Hk)) * D) + 2 * r.part;
                x[u][0] = __ldg(src);
                x[u][1] = __ldg(src + 1);
            }
        }
    };
    load(r.first);  // in flight while the tokens are located
    locate_tokens(p.seqs, p.cache, t0, at, tokens_at == 0 && heads_at == 0);
    // (whole warps go round: items and the steps are multiples of a warp's rows)
    for (int i0 = r.first; i0 < r.items; i0 += kInFlight * kStep) {
        if (i0 != r.first) load(i0);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int it = i0 + u * kStep, h = r.head(it);
            uint32_t codes[2], word;
            quantise(x[u], group_lanes, codes, &word);
            if (it >= r.items) continue;
            size_t row = at.rows[r.token(it)];
            if (row == ~size_t(0)) continue;
            row += (h < Hk ? h : h - Hk) * stride;
            reinterpret_cast<uint2*>((h < Hk ? p.cache.k : p.cache.v) + row * (D / 2))[r.part] = make_uint2(codes[0], codes[1]);
            if (r.part % group_lanes == 0) (h < Hk ? p.cache.kp : p.cache.vp)[row * groups + r.part / group_lanes] = word;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) write_cache4_kernel(const Copy4Params p) {
    __shared__ Places at;
    griddep_wait();
    write_rows4<D>(p, at, blockIdx.x, blockIdx.y);
}

// The values of 16 channels: a code as the low bits of 2^23; the product with s is exact, the sum
// rounds to fp32 and then once to bf16.
__device__ __forceinline__ void expand16(const uint2& codes, uint32_t word, uint4 (&out)[2]) {
    const float s = bf16_lo(word), m = bf16_hi(word);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t c = half ? codes.y : codes.x;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = __uint_as_float(0x4b000000u | ((c >> (8 * e)) & 15u)) - 8388608.f;
            const float b = __uint_as_float(0x4b000000u | ((c >> (8 * e + 4)) & 15u)) - 8388608.f;
            const __nv_bfloat162 v = __floats2bfloat162_rn(fmaf(a, s, m), fmaf(b, s, m));
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        out[half] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) read_cache4_kernel(const Copy4Params p) {
    __shared__ Places at;
    const int Hk = p.cache.n_kv_heads, groups = p.cache.groups, group_lanes = D / 16 / groups;
    const size_t stride = p.cache.block_table ? (size_t)1 << p.cache.block_log2 : (size_t)p.cache.max_cache_len;
    const int t0 = blockIdx.x * kCopyTokens;
    const Rows<D> r(Hk, p.heads, blockIdx.y);
    constexpr int kStep = Rows<D>::kStep;
    griddep_wait();
    locate_tokens(p.seqs, p.cache, t0, at, blockIdx.x == 0 && blockIdx.y == 0);
    for (int i0 = r.first; i0 < r.items; i0 += kInFlight * kStep) {
        uint2 codes[kInFlight];
        uint32_t word[kInFlight];
        bool there[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int it = i0 + u * kStep, h = r.head(it);
            size_t row = it < r.items ? at.rows[r.token(it)] : ~size_t(0);
            there[u] = row != ~size_t(0);
            codes[u] = make_uint2(0, 0);
            word[u] = 0;
            if (there[u]) {
                row += (h < Hk ? h : h - Hk) * stride;
                codes[u] = __ldg(reinterpret_cast<const uint2*>((h < Hk ? p.cache.k : p.cache.v) + row * (D / 2)) + r.part);
                word[u] = __ldg((h < Hk ? p.cache.kp : p.cache.vp) + row * groups + r.part / group_lanes);
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            if (!there[u]) continue;
            const int it = i0 + u * kStep, h = r.head(it);
            uint4* dst = reinterpret_cast<uint4*>((h < Hk ? p.k_out : p.v_out) +
                                                  ((size_t)(t0 + r.token(it)) * Hk + (h < Hk ? h : h - Hk)) * D) + 2 * r.part;
            uint4 out[2];
            expand16(codes[u], word[u], out);
            dst[0] = out[0];
            dst[1] = out[1];
        }
    }
}

// One block per sequence: its metadata, and the table entries of the call's tokens
// (whole: of all tokens up to its last).
__global__ void __launch_bounds__(128) check_sequences4_kernel(const Sequences4 a, const Cache4 c, bool whole) {
    const int b = blockIdx.x;
    griddep_launch();
    griddep_wait();
    const SeqInfo s = stated_sequence(a, c.max_cache_len, b);
    bool bad = s.n < 0;
    if (c.block_table && s.n > 0) {
        const int first = whole ? 0 : s.P >> c.block_log2, end = ((s.P + s.n - 1) >> c.block_log2) + 1;
        const int32_t* table = c.block_table + (size_t)b * c.max_blocks;
#pragma unroll 4
        for (int i = first + threadIdx.x; i < end; i += 128) bad |= (unsigned)__ldg(table + i) >= (unsigned)c.num_blocks;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.checked[b] = bad ? SeqInfo{0, 0, 0, 0} : s;
        if (bad) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
    }
}

// The first p.expanders blocks take 128 rows (a block of the pool, one head of K or V) at a time;
// the others write the call's new tokens into the cache, which nothing else of the call reads.
template <int D>
__global__ void __launch_bounds__(kCopyThreads) expand4_kernel(const Expand4Params p) {
    __shared__ Places places;
    griddep_wait();
    if ((int)blockIdx.x >= p.expanders) {
        const int x = blockIdx.x - p.expanders;
        write_rows4<D>(p.write, places, x % p.write_blocks, x / p.write_blocks);
        return;
    }
    constexpr int kLanes = D / 16, kStep = kCopyThreads / kLanes;
    constexpr int kPasses = kBlock4 / kStep > 0 ? kBlock4 / kStep : 1;
    const Cache4& c = p.cache;
    const int Hk = c.n_kv_heads, group_lanes = kLanes / c.groups;
    const int part = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
    const long long units = 2ll * Hk * *p.blocks;
    for (long long u = blockIdx.x; u < units; u += p.expanders) {
        const int block = (int)(u / (2 * Hk)), h = (int)(u % (2 * Hk)), kvh = h < Hk ? h : h - Hk;
        const int2 owner = p.owners[block];
        const int P = p.seqs.checked[owner.x].P;
        uint2 codes[kPasses];
        uint32_t word[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int pos = owner.y + i * kStep + first;
            codes[i] = make_uint2(0, 0);
            word[i] = 0;
            if (i * kStep + first < kBlock4 && pos < P) {
                const size_t row = row4(c, owner.x, kvh, pos);
                if (row == ~size_t(0)) continue;
                codes[i] = __ldg(reinterpret_cast<const uint2*>((h < Hk ? c.k : c.v) + row * (D / 2)) + part);
                word[i] = __ldg((h < Hk ? c.kp : c.vp) + row * c.groups + part / group_lanes);
            }
        }
        // row of the pool: its blocks' (a paged cache), or its one sequence's (contiguous)
        const size_t row0 = p.table ? ((size_t)block * Hk + kvh) * kBlock4
                                    : (size_t)kvh * p.table_blocks * kBlock4 + owner.y;
        __nv_bfloat16* const pool = (h < Hk ? p.k : p.v) + row0 * D;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kStep + first;
            if (r >= kBlock4 || owner.y + r >= P) continue;
            uint4 out[2];
            expand16(codes[i], word[i], out);
            uint4* dst = reinterpret_cast<uint4*>(pool + (size_t)r * D) + 2 * part;
            dst[0] = out[0];
            dst[1] = out[1];
        }
    }
}

template <class Kernel, class... Args>
cudaError_t launch_after(Kernel kernel, dim3 grid, unsigned threads, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_check_sequences4(const Sequences4& a, const Cache4& c, bool whole, cudaStream_t stream) {
    return launch_after(check_sequences4_kernel, dim3((unsigned)a.num_seqs), 128, stream, a, c, whole);
}

namespace {

// Heads of a block: enough blocks for the GPU first, then up to kMostRows channels of rows to a
// block, so that finding its tokens is little of its time.
constexpr long long kMostRows = 65536;
int heads_of_block(long long blocks, long long heads, int head_dim, int sms) {
    return (int)std::max(1ll, std::min(kMostRows / head_dim / kCopyTokens, blocks * heads / (8ll * sms)));
}

template <class Kernel>
cudaError_t launch_copy(Kernel kernel, Copy4Params p, int head_dim, int sms, cudaStream_t stream) {
    const long long blocks = ((long long)p.seqs.total_q + kCopyTokens - 1) / kCopyTokens;
    const long long heads = 2ll * p.cache.n_kv_heads;
    p.heads = heads_of_block(blocks, heads, head_dim, sms);
    return launch_after(kernel, dim3((unsigned)blocks, (unsigned)((heads + p.heads - 1) / p.heads)), kCopyThreads, stream, p);
}

}  // namespace

cudaError_t launch_write_cache4(const Copy4Params& p, int head_dim, int sms, cudaStream_t stream) {
    switch (head_dim) {
        case 32: return launch_copy(write_cache4_kernel<32>, p, 32, sms, stream);
        case 64: return launch_copy(write_cache4_kernel<64>, p, 64, sms, stream);
        default: return launch_copy(write_cache4_kernel<128>, p, 128, sms, stream);
    }
}

cudaError_t launch_read_cache4(const Copy4Params& p, int head_dim, int sms, cudaStream_t stream) {
    switch (head_dim) {
        case 32: return launch_copy(read_cache4_kernel<32>, p, 32, sms, stream);
        case 64: return launch_copy(read_cache4_kernel<64>, p, 64, sms, stream);
        default: return launch_copy(read_cache4_kernel<128>, p, 128, sms, stream);
    }
}

cudaError_t launch_expand4(Expand4Params p, int head_dim, int sms, cudaStream_t stream) {
    const long long blocks = ((long long)p.write.seqs.total_q + kCopyTokens - 1) / kCopyTokens;
    const long long heads = 2ll * p.cache.n_kv_heads;
    p.write.heads = heads_of_block(blocks, heads, head_dim, sms);
    p.write_blocks = (int)blocks;
    p.expanders = (int)std::min((long long)sms * 4, heads * p.pool_blocks);
    const dim3 grid((unsigned)(p.expanders + blocks * ((heads + p.write.heads - 1) / p.write.heads)));
    switch (head_dim) {
        case 32: return launch_after(expand4_kernel<32>, grid, kCopyThreads, stream, p);
        case 64: return launch_after(expand4_kernel<64>, grid, kCopyThreads, stream, p);
        default: return launch_after(expand4_kernel<128>, grid, kCopyThreads, stream, p);
    }
}

}  // namespace pa
