// cache4.cuh -- the 4-bit KV cache: its format, and device helpers shared by the
// kernels that write, read and attend over it.
//
// A row (token, KV head) of head_dim channels is cut into groups of 32, 64 or 128
// channels.  A group's parameters are one 32-bit word, the scale s (low half) and the
// minimum m (high half) as bf16; its codes are 4 bits per channel, two to a byte, the
// even channel low.  A channel stands for m + code * s.  Of a group x of bf16 values
//     m = min x                       (a bf16 already: exact)
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

// Quantises 8 channels (bf16 pairs x) of a row whose groups are spread over `lanes`
// consecutive lanes each: returns the 8 codes, *params the group's word (the same in
// its lanes).  All lanes of the warp.
__device__ __forceinline__ uint32_t quantise8(const uint4& x, int lanes, uint32_t* params) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
    for (int o = 1; o < lanes; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    __nv_bfloat16 s = __float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
    float sf = __bfloat162float(s);
    const float r = sf >= 0x1p-126f ? __frcp_rn(sf) : 0.f;
    if (!(sf >= 0x1p-126f)) s = __float2bfloat16_rn(0.f);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = __float2int_rn(__fmul_rn(__fsub_rn(v[i], lo), r));
        codes |= (uint32_t)(c < 15 ? c : 15) << (4 * i);
    }
    *params = (uint32_t)__bfloat16_as_ushort(s) | (__float_as_uint(lo) & 0xffff0000u);
    return codes;
}

}  // namespace pa
