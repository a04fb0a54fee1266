// cache4.cu -- writing keys and values into the 4-bit cache, reading them back, and
// the check of a paged call's sequences.
//
// Both are one pass over the rows: a lane takes 8 channels (16 bytes of bf16, 4 of
// codes), head_dim / 8 lanes a row, and consecutive lanes of a warp take consecutive
// tokens of one KV head, whose rows lie side by side in the cache.  The bytes bound
// them; each thread has several rows in flight.
#include "cache4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyTokens = 32;  // of a block
constexpr int kInFlight = 4;     // rows of a thread

// Where the rows of a block's tokens are: the row of KV head 0 (~0: none); another
// head's is `stride` rows on.
__device__ __forceinline__ void locate_tokens(const Sequences4& a, const Cache4& c, long long t0, size_t* rows) {
    for (int i = threadIdx.x; i < kCopyTokens; i += kCopyThreads) {
        const long long t = t0 + i;
        size_t row = ~size_t(0);
        if (t < a.total_q) {
            // the sequence owning token t: the last b with cu_seqlens_q[b] <= t
            int lo = 0, hi = a.num_seqs - 1;
            while (lo < hi) {
                const int mid = lo + (hi - lo + 1) / 2;
                if (a.cu_seqlens_q[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const SeqInfo s = sequence4(a, c.max_cache_len, lo);
            if (t >= s.q_start && t < (long long)s.q_start + s.n) row = row4(c, lo, 0, s.P + (int)(t - s.q_start));
        }
        rows[i] = row;
    }
}

// Sequences whose metadata is inconsistent are reported by block 0 where no kernel checked them.
__device__ __forceinline__ void report_sequences(const Sequences4& a, int max_cache_len) {
    if (a.checked || blockIdx.x != 0) return;
    for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x)
        if (stated_sequence(a, max_cache_len, b).n < 0) atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) write_cache4_kernel(const Copy4Params p) {
    constexpr int kLanes = D / 8;  // of a row
    __shared__ size_t rows[kCopyTokens];
    const long long t0 = (long long)blockIdx.x * kCopyTokens;
    griddep_wait();
    locate_tokens(p.seqs, p.cache, t0, rows);
    report_sequences(p.seqs, p.cache.max_cache_len);
    __syncthreads();
    const int Hk = p.cache.n_kv_heads, groups = p.cache.groups, group_lanes = kLanes / groups;
    const size_t stride = p.cache.block_table ? (size_t)1 << p.cache.block_log2 : (size_t)p.cache.max_cache_len;
    const int part = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
    constexpr int kStep = kCopyThreads / kLanes;  // rows of a pass
    const int items = 2 * Hk * kCopyTokens;       // (k or v, head, token): a whole number of passes
    for (int i0 = first; i0 < items; i0 += kInFlight * kStep) {
        uint4 x[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int it = i0 + u * kStep, tt = it % kCopyTokens, h = it / kCopyTokens;
            x[u] = make_uint4(0, 0, 0, 0);
            if (it < items && rows[tt] != ~size_t(0)) {
                const __nv_bfloat16* src = h < Hk ? p.k : p.v;
                x[u] = __ldg(reinterpret_cast<const uint4*>(src + ((t0 + tt) * Hk + (h < Hk ? h : h - Hk)) * D) + part);
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int it = i0 + u * kStep, tt = it % kCopyTokens, h = it / kCopyTokens;
            uint32_t word;
            const uint32_t codes = quantise8(x[u], group_lanes, &word);
            if (it >= items || rows[tt] == ~size_t(0)) continue;
            const size_t row = rows[tt] + (h < Hk ? h : h - Hk) * stride;
            reinterpret_cast<uint32_t*>((h < Hk ? p.cache.k : p.cache.v) + row * (D / 2))[part] = codes;
            if (part % group_lanes == 0) (h < Hk ? p.cache.kp : p.cache.vp)[row * groups + part / group_lanes] = word;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) read_cache4_kernel(const Copy4Params p) {
    constexpr int kLanes = D / 8;
    __shared__ size_t rows[kCopyTokens];
    const long long t0 = (long long)blockIdx.x * kCopyTokens;
    griddep_wait();
    locate_tokens(p.seqs, p.cache, t0, rows);
    report_sequences(p.seqs, p.cache.max_cache_len);
    __syncthreads();
    const int Hk = p.cache.n_kv_heads, groups = p.cache.groups, group_lanes = kLanes / groups;
    const size_t stride = p.cache.block_table ? (size_t)1 << p.cache.block_log2 : (size_t)p.cache.max_cache_len;
    const int part = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
    constexpr int kStep = kCopyThreads / kLanes;
    const int items = 2 * Hk * kCopyTokens;
    for (int i0 = first; i0 < items; i0 += kInFlight * kStep) {
        uint32_t codes[kInFlight], word[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int it = i0 + u * kStep, tt = it % kCopyTokens, h = it / kCopyTokens;
            codes[u] = word[u] = 0;
            if (it < items && rows[tt] != ~size_t(0)) {
                const size_t row = rows[tt] + (h < Hk ? h : h - Hk) * stride;
                codes[u] = reinterpret_cast<const uint32_t*>((h < Hk ? p.cache.k : p.cache.v) + row * (D / 2))[part];
                word[u] = (h < Hk ? p.cache.kp : p.cache.vp)[row * groups + part / group_lanes];
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int it = i0 + u * kStep, tt = it % kCopyTokens, h = it / kCopyTokens;
            if (it >= items || rows[tt] == ~size_t(0)) continue;
            const float s = bf16_lo(word[u]), m = bf16_hi(word[u]);
            uint32_t out[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // the product is exact, the sum rounds to fp32 and then once to bf16
                const float a = fmaf((float)((codes[u] >> (8 * e)) & 15u), s, m);
                const float b = fmaf((float)((codes[u] >> (8 * e + 4)) & 15u), s, m);
                const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
                out[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            __nv_bfloat16* dst = h < Hk ? p.k_out : p.v_out;
            reinterpret_cast<uint4*>(dst + ((t0 + tt) * Hk + (h < Hk ? h : h - Hk)) * D)[part] =
                make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
}

// One block per sequence: its metadata, and the entries [first, end) of its table.
__global__ void __launch_bounds__(128) check_sequences4_kernel(const Sequences4 a, const Cache4 c, bool whole) {
    const int b = blockIdx.x;
    griddep_launch();
    griddep_wait();
    const SeqInfo s = stated_sequence(a, c.max_cache_len, b);
    bool bad = s.n < 0;
    if (c.block_table && s.n > 0) {
        // the blocks of the tokens it writes or reads; `whole`: of all tokens up to its last
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

template <class Kernel, class... Args>
cudaError_t launch_after(Kernel kernel, unsigned grid, unsigned threads, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
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
    return launch_after(check_sequences4_kernel, (unsigned)a.num_seqs, 128, stream, a, c, whole);
}

cudaError_t launch_write_cache4(const Copy4Params& p, int head_dim, cudaStream_t stream) {
    const unsigned grid = (unsigned)(((long long)p.seqs.total_q + kCopyTokens - 1) / kCopyTokens);
    switch (head_dim) {
        case 32: return launch_after(write_cache4_kernel<32>, grid, kCopyThreads, stream, p);
        case 64: return launch_after(write_cache4_kernel<64>, grid, kCopyThreads, stream, p);
        default: return launch_after(write_cache4_kernel<128>, grid, kCopyThreads, stream, p);
    }
}

cudaError_t launch_read_cache4(const Copy4Params& p, int head_dim, cudaStream_t stream) {
    const unsigned grid = (unsigned)(((long long)p.seqs.total_q + kCopyTokens - 1) / kCopyTokens);
    switch (head_dim) {
        case 32: return launch_after(read_cache4_kernel<32>, grid, kCopyThreads, stream, p);
        case 64: return launch_after(read_cache4_kernel<64>, grid, kCopyThreads, stream, p);
        default: return launch_after(read_cache4_kernel<128>, grid, kCopyThreads, stream, p);
    }
}

}  // namespace pa
