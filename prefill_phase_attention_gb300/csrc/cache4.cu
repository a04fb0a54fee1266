// cache4.cu -- writing keys and values into the 4-bit cache, reading them back, expanding
// a long chunk's cached ones, and the check of an attention call's sequences.
//
// Both copies are one pass over the rows, which the bytes bound: a lane takes 16
// channels (32 bytes of bf16, 8 of codes), head_dim / 16 lanes a row, and consecutive
// rows of lanes take consecutive tokens of one KV head, whose rows lie side by side in
// the cache.  A block takes 32 tokens and some heads of K and V; the tokens' sequences,
// positions and table entries are looked up once a block, in shared memory.  A block
// looks whether its sequences' tables are valid itself: a kernel ahead for that
// costs a small call more than all of it.  32768 tokens of 32 heads, d = 128, group 128: written in
// 115 us, read in 115 (6.0 TB/s; the floor at the copy rate is 101).  A lane that finds its rows by
// adding strides, and not anew, brought the first from 164; both 16-byte halves of 32 bytes in one
// store brought reading 16 x 16384 tokens of 8 heads, group 64, from 236 to 212 (floor 205).
#include <cuda_fp16.h>

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
    int first[kCopyTokens], last[kCopyTokens];  // positions of its sequence's first and last token
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

// A thread's rows: its token of the block's, heads first, first + kHeadStep, ... below end, and
// channels [16 part, 16 part + 16).
template <int D>
struct Rows {
    static constexpr int kLanes = D / 16;
    static constexpr int kHeadStep = kCopyThreads / kLanes / kCopyTokens;
    static_assert(kHeadStep >= 1 && kCopyThreads % (kLanes * kCopyTokens) == 0, "a pass is whole heads");
    int part = threadIdx.x % kLanes, token = threadIdx.x / kLanes % kCopyTokens, first, end;
    __device__ __forceinline__ Rows(int n_kv_heads, int heads, int slice) {
        first = slice * heads + threadIdx.x / (kLanes * kCopyTokens);
        end = min(n_kv_heads, (slice + 1) * heads);
    }
};

// Rows of the cache from one KV head to the next.
__device__ __forceinline__ size_t head_stride(const Cache4& c) {
    return c.block_table ? (size_t)1 << c.block_log2 : (size_t)c.max_cache_len;
}

// Tokens [32 tokens_at, ...) of a slice of the heads of k, or of v (the slices after those), into the
// cache.
template <int D, int kGroups>
__device__ __forceinline__ void write_rows4(const Copy4Params& p, Places& at, int tokens_at, int slice) {
    constexpr int kGroupLanes = D / 16 / kGroups, kStep = Rows<D>::kHeadStep;
    const int Hk = p.cache.n_kv_heads, t = tokens_at * kCopyTokens;
    const int slices = (Hk + p.heads - 1) / p.heads;
    const bool keys = slice < slices;
    const Rows<D> r(Hk, p.heads, keys ? slice : slice - slices);
    const bool there = t + r.token < p.seqs.total_q;
    const uint4* src = reinterpret_cast<const uint4*>((keys ? p.k : p.v) + ((size_t)(t + r.token) * Hk + r.first) * D) + 2 * r.part;
    uint4 x[kInFlight][2];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
            if (there && h + u * kStep < r.end) {
                x[u][0] = __ldg(src + u * kStep * (D / 8));
                x[u][1] = __ldg(src + u * kStep * (D / 8) + 1);
            }
        }
        src += kInFlight * kStep * (D / 8);
    };
    load(r.first);  // in flight while the tokens are located
    locate_tokens(p.seqs, p.cache, t, at, tokens_at == 0 && slice == 0);
    const size_t row = at.rows[r.token], stride = head_stride(p.cache) * kStep;
    const bool wanted = row != ~size_t(0);
    const size_t row0 = wanted ? row + r.first * head_stride(p.cache) : 0;
    uint2* codes_at = reinterpret_cast<uint2*>((keys ? p.cache.k : p.cache.v) + row0 * (D / 2)) + r.part;
    uint32_t* params_at = (keys ? p.cache.kp : p.cache.vp) + row0 * kGroups + r.part / kGroupLanes;
    // (whole warps go round: a warp's rows are of one head)
    for (int h = r.first; h < r.end; h += kInFlight * kStep) {
        if (h != r.first) load(h);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            uint32_t codes[2], word;
            quantise<kGroupLanes>(x[u], codes, &word);
            if (wanted && h + u * kStep < r.end) {
                *codes_at = make_uint2(codes[0], codes[1]);
                if (r.part % kGroupLanes == 0) *params_at = word;
            }
            codes_at += stride * (D / 16);
            params_at += stride * kGroups;
        }
    }
}

template <int D, int kGroups>
__global__ void __launch_bounds__(kCopyThreads, 4) write_cache4_kernel(const Copy4Params p) {
    __shared__ Places at;
    griddep_wait();
    write_rows4<D, kGroups>(p, at, blockIdx.x, blockIdx.y);
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

// 32 bytes, as one store where the tensor's alignment allows: of two stores each would fill half of
// every 32-byte sector that a warp touches.
__device__ __forceinline__ void store32(uint4* to, const uint4 (&x)[2], bool aligned) {
    if (aligned)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0].x), "r"(x[0].y),
                     "r"(x[0].z), "r"(x[0].w), "r"(x[1].x), "r"(x[1].y), "r"(x[1].z), "r"(x[1].w)
                     : "memory");
    else
        to[0] = x[0], to[1] = x[1];
}

// The values of 16 channels in fp16.
__device__ __forceinline__ void expand16_half(const uint2& codes, uint32_t word, uint4 (&out)[2]) {
    const float s = bf16_lo(word), m = bf16_hi(word);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t c = half ? codes.y : codes.x;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = __uint_as_float(0x4b000000u | ((c >> (8 * e)) & 15u)) - 8388608.f;
            const float b = __uint_as_float(0x4b000000u | ((c >> (8 * e + 4)) & 15u)) - 8388608.f;
            const __half2 v = __floats2half2_rn(fmaf(a, s, m), fmaf(b, s, m));
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        out[half] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The values of 16 channels as sums of two bf16 terms (to 2^-17 of their size: keys, whose scores
// go through an exponential).
__device__ __forceinline__ void expand16_two(const uint2& codes, uint32_t word, uint4 (&one)[2], uint4 (&two)[2]) {
    const float s = bf16_lo(word), m = bf16_hi(word);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t c = half ? codes.y : codes.x;
        uint32_t w[4], x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = fmaf(__uint_as_float(0x4b000000u | ((c >> (8 * e)) & 15u)) - 8388608.f, s, m);
            const float b = fmaf(__uint_as_float(0x4b000000u | ((c >> (8 * e + 4)) & 15u)) - 8388608.f, s, m);
            const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
            const __nv_bfloat162 r = __floats2bfloat162_rn(a - bf16_lo(w[e]), b - bf16_hi(w[e]));
            x[e] = *reinterpret_cast<const uint32_t*>(&r);
        }
        one[half] = make_uint4(w[0], w[1], w[2], w[3]);
        two[half] = make_uint4(x[0], x[1], x[2], x[3]);
    }
}

template <int D, int kGroups>
__global__ void __launch_bounds__(kCopyThreads) read_cache4_kernel(const Copy4Params p) {
    constexpr int kGroupLanes = D / 16 / kGroups, kStep = Rows<D>::kHeadStep;
    __shared__ Places at;
    const int Hk = p.cache.n_kv_heads, t = blockIdx.x * kCopyTokens;
    const Rows<D> r(Hk, p.heads, blockIdx.y);
    griddep_wait();
    locate_tokens(p.seqs, p.cache, t, at, blockIdx.x == 0 && blockIdx.y == 0);
    if (at.rows[r.token] == ~size_t(0)) return;
    const size_t row0 = at.rows[r.token] + r.first * head_stride(p.cache), stride = head_stride(p.cache) * kStep;
    const size_t to = ((size_t)(t + r.token) * Hk + r.first) * (D / 8) + 2 * r.part;
#pragma unroll 1
    for (int v = 0; v < 2; ++v) {  // K, then V: finding the tokens takes a block as long as either
        const uint2* codes_at = reinterpret_cast<const uint2*>((v ? p.cache.v : p.cache.k) + row0 * (D / 2)) + r.part;
        const uint32_t* params_at = (v ? p.cache.vp : p.cache.kp) + row0 * kGroups + r.part / kGroupLanes;
        uint4* dst = reinterpret_cast<uint4*>(v ? p.v_out : p.k_out) + to;
        for (int h = r.first; h < r.end; h += kInFlight * kStep) {
            uint2 codes[kInFlight];
            uint32_t word[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                codes[u] = make_uint2(0, 0);
                word[u] = 0;
                if (h + u * kStep < r.end) {
                    codes[u] = __ldg(codes_at);
                    word[u] = __ldg(params_at);
                }
                codes_at += stride * (D / 16);
                params_at += stride * kGroups;
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                uint4 out[2];
                expand16(codes[u], word[u], out);
                if (h + u * kStep < r.end) store32(dst, out, p.aligned32);
                dst += kStep * (D / 8);
            }
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
// Three bf16 planes are written for 1/6 of that read: 4096 positions and as many new tokens of 32
// heads take 38 us (136 MB read and 205 MB written: DRAM's time at 6.7 TB/s is 51, much of the pool
// stays in L2).  Expanding tiles in the attention kernel's own warps, for every query block again,
// took 659 us for both, 349 as two kernels (with keys in one term).
template <int D, int kGroups>
__global__ void __launch_bounds__(kCopyThreads, 4) expand4_kernel(const Expand4Params p) {
    __shared__ Places places;
    griddep_wait();
    if ((int)blockIdx.x >= p.expanders) {
        const int x = blockIdx.x - p.expanders;
        write_rows4<D, kGroups>(p.write, places, x % p.write_blocks, x / p.write_blocks);
        return;
    }
    constexpr int kLanes = D / 16, kStep = kCopyThreads / kLanes;
    constexpr int kPasses = kBlock4 / kStep > 0 ? kBlock4 / kStep : 1;
    const Cache4& c = p.cache;
    constexpr int kGroupLanes = kLanes / kGroups;
    const int Hk = c.n_kv_heads;
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
            if (i * kStep + first < kBlock4 && pos >= 0 && pos < P) {
                const size_t row = row4(c, owner.x, kvh, pos);
                if (row == ~size_t(0)) continue;
                codes[i] = __ldg(reinterpret_cast<const uint2*>((h < Hk ? c.k : c.v) + row * (D / 2)) + part);
                word[i] = __ldg((h < Hk ? c.kp : c.vp) + row * kGroups + part / kGroupLanes);
            }
        }
        const size_t at = ((size_t)kvh * p.pool_blocks + block) * kBlock4 * D;
        // Values are rounded to fp16, an eighth of bf16's error, where the largest of every row and group of
        // the block is within its range, with room for smaller ones (below 2^-14 they are off by 2^-25, which
        // is 2^-13 of their group's largest then), or 0.
        bool half = false;
        if (h >= Hk) {
            bool fits = true;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const float m = bf16_hi(word[i]), top = fmaxf(fabsf(m), fabsf(fmaf(15.f, bf16_lo(word[i]), m)));
                fits = fits && (top == 0.f || (top >= 0x1p-12f && top <= 0x1p15f));
            }
            half = __syncthreads_and(fits);
            if (threadIdx.x == 0) p.halves[(size_t)kvh * p.pool_blocks + block] = half;
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int r = i * kStep + first;
            if (r >= kBlock4) continue;  // (positions below 0 expand to zeros)
            const size_t to = at + (size_t)r * D + 16 * part;
            uint4 one[2], two[2];
            if (h < Hk) {
                expand16_two(codes[i], word[i], one, two);
                store32(reinterpret_cast<uint4*>(p.k + to), one, true);  // (the pool is the workspace's)
                store32(reinterpret_cast<uint4*>(p.k2 + to), two, true);
            } else {
                if (half)
                    expand16_half(codes[i], word[i], one);
                else
                    expand16(codes[i], word[i], one);
                store32(reinterpret_cast<uint4*>(p.v + to), one, true);
            }
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

// Heads of a block: enough blocks for the GPU first, then up to kMostChannels of a token to a block,
// so that finding its tokens is little of its time.
constexpr long long kMostChannels = 2048;

// kinds: 2 where K and V have blocks of their own.
int heads_of_block(long long blocks, int n_kv_heads, int head_dim, int kinds, int sms) {
    const long long wanted = blocks * kinds * n_kv_heads / (8ll * sms);
    const int most = (int)std::max(1ll, std::min({wanted, kMostChannels / head_dim, (long long)n_kv_heads}));
    const int slices = (n_kv_heads + most - 1) / most;
    return (n_kv_heads + slices - 1) / slices;
}

template <class Kernel>
cudaError_t launch_copy(Kernel kernel, Copy4Params p, int head_dim, int kinds, int sms, cudaStream_t stream) {
    const long long blocks = ((long long)p.seqs.total_q + kCopyTokens - 1) / kCopyTokens;
    p.heads = heads_of_block(blocks, p.cache.n_kv_heads, head_dim, kinds, sms);
    const int slices = kinds * ((p.cache.n_kv_heads + p.heads - 1) / p.heads);
    return launch_after(kernel, dim3((unsigned)blocks, (unsigned)slices), kCopyThreads, stream, p);
}

// f<head_dim, groups of a row>
#define PA_CACHE4_VARIANT(head_dim, groups, f)                    \
    head_dim == 32                    ? f<32, 1>                  \
    : head_dim == 64                  ? groups == 1 ? f<64, 1> : f<64, 2> \
    : groups == 1                     ? f<128, 1>                 \
    : groups == 2                     ? f<128, 2>                 \
                                      : f<128, 4>

}  // namespace

cudaError_t launch_write_cache4(const Copy4Params& p, int head_dim, int sms, cudaStream_t stream) {
    return launch_copy(PA_CACHE4_VARIANT(head_dim, p.cache.groups, write_cache4_kernel), p, head_dim, 2, sms, stream);
}

cudaError_t launch_read_cache4(const Copy4Params& p, int head_dim, int sms, cudaStream_t stream) {
    return launch_copy(PA_CACHE4_VARIANT(head_dim, p.cache.groups, read_cache4_kernel), p, head_dim, 1, sms, stream);
}

cudaError_t launch_expand4(Expand4Params p, int head_dim, int sms, cudaStream_t stream) {
    const long long blocks = ((long long)p.write.seqs.total_q + kCopyTokens - 1) / kCopyTokens;
    const int Hk = p.cache.n_kv_heads;
    p.write.heads = heads_of_block(blocks, Hk, head_dim, 2, sms);
    p.write_blocks = (int)blocks;
    p.expanders = (int)std::min((long long)sms * 4, 2ll * Hk * p.pool_blocks);
    const dim3 grid((unsigned)(p.expanders + blocks * 2 * ((Hk + p.write.heads - 1) / p.write.heads)));
    return launch_after(PA_CACHE4_VARIANT(head_dim, p.cache.groups, expand4_kernel), grid, kCopyThreads, stream, p);
}

#undef PA_CACHE4_VARIANT

}  // namespace pa
