// cache4.cuh -- the 4-bit KV cache: its format, and device helpers shared by the
// kernels that write, read and attend over it.
//
// A row (token, KV head) of head_dim channels is cut into groups of 32, 64 or 128
// channels.  A group's parameters are one 32-bit word, the scale s (low half) and the
// minimum m (high half) as bf16; its codes are 4 bits per channel, two to a byte, the
// even channel low.  A channel stands for m + code * s.  Of a group x of bf16 values
//     m = min x                       (a bf16 already: exact; 0 for -0)
//     s = bf16(fl(max x - m) * fl(1/15)), 0 when that is below 2^-126
//     code = min(15, rint(fl(fl(x - m) * r))), r = fl(1 / s), or 0 when s = 0
// where fl rounds to fp32 and rint ties to even.  The error is at most s / 2 and a few
// fp32 roundings, and 15 s / 2^9 more at the top of the range where s rounded down.
#pragma once

#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "common.cuh"
#include "prefill_attn.h"

namespace pa {

struct Cache4 {
    uint8_t* k;  // codes, [rows][head_dim / 2]
    uint8_t* v;
    uint32_t* kp;  // parameters, [rows][groups]
    uint32_t* vp;
    int groups;  // of a row
    int n_kv_heads, max_cache_len;
    // paged cache (block_table == nullptr: row (b * n_kv_heads + h) * max_cache_len + position)
    const int32_t* block_table;
    int block_log2, max_blocks, num_blocks;
};

// Metadata of a call's sequences.
struct Sequences4 {
    const int32_t* cu_seqlens_q;
    const int32_t* cu_seqlens_k;  // nullptr: a call without keys of its own
    const int32_t* cache_offsets;
    int num_seqs, total_q;
    SeqInfo* checked;  // where a kernel before wrote them; nullptr: none did
    WorkspaceHeader* hdr;
};

// Sequence b as its metadata states it; n = -1 when that is inconsistent.
__device__ __forceinline__ SeqInfo stated_sequence(const Sequences4& a, int max_cache_len, int b) {
    const int q_start = a.cu_seqlens_q[b], q_end = a.cu_seqlens_q[b + 1];
    const int P = a.cache_offsets[b];
    const long long n = (long long)q_end - q_start;
    bool ok = q_start >= 0 && n >= 0 && (long long)q_end <= a.total_q && P >= 0 && (long long)P + n <= max_cache_len &&
              (b > 0 || q_start == 0);
    if (a.cu_seqlens_k) ok = ok && (long long)a.cu_seqlens_k[b + 1] - a.cu_seqlens_k[b] == (long long)P + n;
    return ok ? SeqInfo{q_start, (int)n, P, 0} : SeqInfo{0, -1, 0, 0};
}

// The same from the kernel that checked it, if one did; n = 0 when it is to be skipped.
__device__ __forceinline__ SeqInfo sequence4(const Sequences4& a, int max_cache_len, int b) {
    SeqInfo s = a.checked ? a.checked[b] : stated_sequence(a, max_cache_len, b);
    if (s.n < 0) s.n = 0;
    return s;
}

// Cache row of a position, ~0 where the table names no block of the pool.
__device__ __forceinline__ size_t row4(const Cache4& c, int b, int kvh, int pos) {
    if (!c.block_table) return ((size_t)b * c.n_kv_heads + kvh) * c.max_cache_len + pos;
    const int blk = __ldg(c.block_table + (size_t)b * c.max_blocks + (pos >> c.block_log2));
    if ((unsigned)blk >= (unsigned)c.num_blocks) return ~size_t(0);
    return (((size_t)blk * c.n_kv_heads + kvh) << c.block_log2) + (pos & ((1 << c.block_log2) - 1));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Quantises 8 kWords channels (bf16 pairs x) of a row whose groups are spread over
// kLanes consecutive lanes each: codes[w] holds those of channels 8 w ..., *params the
// group's word (the same in its lanes).  All lanes of the warp.
template <int kLanes, int kWords>
__device__ __forceinline__ void quantise(const uint4 (&x)[kWords], uint32_t (&codes)[kWords], uint32_t* params) {
    uint32_t lo2 = x[0].x, hi2 = x[0].x;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        const uint32_t y[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
#pragma unroll
        for (int i = w == 0 ? 1 : 0; i < 4; ++i) lo2 = min_bf16x2(lo2, y[i]), hi2 = max_bf16x2(hi2, y[i]);
    }
    // (minimum, -maximum) of the lane, of the group
    hi2 ^= 0x80008000u;
    uint32_t ends = min_bf16x2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) ends = min_bf16x2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
    const float lo = __fadd_rn(bf16_lo(ends), 0.f), hi = -bf16_hi(ends);  // (a minimum of -0 is stored as 0)
    __nv_bfloat16 s = __float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
    const bool normal = __bfloat162float(s) >= 0x1p-126f;
    if (!normal) s = __float2bfloat16_rn(0.f);
    const float r = normal ? __frcp_rn(__bfloat162float(s)) : 0.f;
    // 2^23 + a value below 2^22 is rounded to an integer, ties to even, in the low bits.  None is
    // above 15: s is at least (1 - 2^-8) (hi - lo) / 15, so the largest is below 15.1.
    constexpr float kRound = 8388608.f;
    const float2 less = make_float2(-lo, -lo), times = make_float2(r, r);
    constexpr uint32_t kUnits = 0x4b000000u * 0x11111111u;  // what the eight numbers' upper bits add up to
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        const uint32_t y[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
        uint32_t sum = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            // (the last sum by halves: a product and a sum of pairs are fused, which rounds once)
            const float2 c = __fmul2_rn(__fadd2_rn(make_float2(bf16_lo(y[i]), bf16_hi(y[i])), less), times);
            sum = sum * 16 + __float_as_uint(__fadd_rn(c.y, kRound));
            sum = sum * 16 + __float_as_uint(__fadd_rn(c.x, kRound));
        }
        codes[w] = sum - kUnits;
    }
    *params = (uint32_t)__bfloat16_as_ushort(s) | (__float_as_uint(lo) & 0xffff0000u);
}

}  // namespace pa
