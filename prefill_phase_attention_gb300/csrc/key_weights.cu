// key_weights.cu -- the attention weight that each cached key collects.
//
// weights[b, h, j] (+)= sum over the new queries i of sequence b and the query
// heads g of KV head h of exp(scale * q_{i,g} . k_j - lse_{i,g}), over the
// queries that see key j (causal mask, sliding window, sink tokens).  lse is
// the log-sum-exp that the attention call wrote, so the terms are the softmax
// probabilities.  Keys [0, P) come from the cache (their weights are added to),
// keys [P, P + n) from k (their weights are set).
//
// Simple form: one CTA of 128 threads per (sequence, KV head, 128 keys), one
// key per thread, the queries staged in shared memory a few rows at a time.
#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr int kKeys = 128;
constexpr int kQRows = 16;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__global__ void __launch_bounds__(kKeys) key_weights_simple_kernel(const __grid_constant__ KeyWeightsArgs a) {
    __shared__ float s_q[kQRows][D];
    __shared__ float s_lse[kQRows];
    const int tiles = (a.max_cache_len + kKeys - 1) / kKeys;
    for (long long unit = blockIdx.x; unit < (long long)tiles * a.n_kv_heads * a.num_seqs; unit += gridDim.x) {
        const int b = (int)(unit / ((long long)tiles * a.n_kv_heads)), h = (int)(unit / tiles % a.n_kv_heads);
        const int j0 = (int)(unit % tiles) * kKeys;
        const SeqInfo s = a.seqs[b];
        const int len = s.P + s.n;
        if (s.n == 0 || j0 >= len) continue;
        const int j = j0 + threadIdx.x;
        const bool in = j < len;
        float k[D];
        float ks = a.scale_log2;
        size_t row = 0;
        if (in) {
            if (a.block_table) {
                const int blk = a.block_table[(size_t)b * a.max_blocks + (j >> a.block_log2)];
                row = (((size_t)blk * a.n_kv_heads + h) << a.block_log2) + (j & ((1 << a.block_log2) - 1));
            } else {
                row = ((size_t)b * a.n_kv_heads + h) * a.max_cache_len + j;
            }
            if (j < s.P && a.scale_k) {
                const int8_t* c = static_cast<const int8_t*>(a.cache_k) + row * D;
#pragma unroll
                for (int d = 0; d < D; ++d) k[d] = (float)c[d];
                ks *= a.scale_k[row];
            } else {
                const __nv_bfloat16* c = j < s.P ? static_cast<const __nv_bfloat16*>(a.cache_k) + row * D
                                                 : a.k + ((size_t)(s.q_start + j - s.P) * a.n_kv_heads + h) * D;
#pragma unroll
                for (int d = 0; d < D; ++d) k[d] = __bfloat162float(c[d]);
            }
        }
        // query rows (token, head in group) from the first that may see a key of the tile
        const int first = a.causal ? max(0, j0 - s.P) : 0;
        float sum = 0.f;
        for (int r0 = first * a.group; r0 < s.n * a.group; r0 += kQRows) {
            __syncthreads();
            for (int i = threadIdx.x; i < kQRows * D; i += kKeys) {
                const int r = r0 + i / D;
                if (r < s.n * a.group)
                    s_q[i / D][i % D] = __bfloat162float(
                        a.q[((size_t)(s.q_start + r / a.group) * a.n_heads + h * a.group + r % a.group) * D + i % D]);
            }
            if (threadIdx.x < kQRows && r0 + threadIdx.x < s.n * a.group) {
                const int r = r0 + threadIdx.x;
                s_lse[threadIdx.x] =
                    a.lse[(size_t)(s.q_start + r / a.group) * a.n_heads + h * a.group + r % a.group] * kLog2e;
            }
            __syncthreads();
            const int rows = min(kQRows, s.n * a.group - r0);
            for (int r = 0; r < rows && in; ++r) {
                const int pos = s.P + (r0 + r) / a.group;
                const bool see = !a.causal || (j <= pos && (a.window == 0 || pos - j < a.window || j < a.sinks));
                if (!see) continue;
                float dot = 0.f;
#pragma unroll
                for (int d = 0; d < D; ++d) dot = fmaf(k[d], s_q[r][d], dot);
                sum += exp2f(fmaf(dot, ks, -s_lse[r]));
            }
        }
        if (in) a.weights[row] = (j < s.P ? a.weights[row] : 0.f) + sum;
    }
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsArgs& a, int head_dim, int sms, cudaStream_t stream) {
    const int tiles = (a.max_cache_len + kKeys - 1) / kKeys;
    const long long units = (long long)tiles * a.n_kv_heads * a.num_seqs;
    const unsigned grid = (unsigned)(units < 8ll * sms ? units : 8ll * sms);
    switch (head_dim) {
        case 32: key_weights_simple_kernel<32><<<grid, kKeys, 0, stream>>>(a); break;
        case 64: key_weights_simple_kernel<64><<<grid, kKeys, 0, stream>>>(a); break;
        default: key_weights_simple_kernel<128><<<grid, kKeys, 0, stream>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace pa
