// kernels.h -- launch interfaces of the device code (internal to the library).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache4.cuh"
#include "common.cuh"

namespace pa {

cudaError_t launch_build_schedule(const ScheduleArgs& a, cudaStream_t stream);

// Rotary embedding prologue: q_rot/k_rot = q/k rotated to each token's
// absolute position (runs after the scheduler, whose SeqInfo it reads).
struct RopeParams {
    const __nv_bfloat16* q;  // [T, H, d]
    const __nv_bfloat16* k;  // [T, Hk, d]
    __nv_bfloat16* q_rot;
    __nv_bfloat16* k_rot;
    const int32_t* cu_seqlens_q;
    const SeqInfo* seqs;
    int total_q, num_seqs, n_heads, n_kv_heads, head_dim;
    int pos0;            // position of a sequence's first cached token (tokens of a shared prefix)
    float inv_freq[64];  // inv_freq[i] = 1 / base^(2i / d), i < d/2
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream);



}  // namespace pa

#include <cuda.h>

namespace pa {

// Parameters of the warp-specialised tcgen05 attention kernel.  The tensor
// maps are encoded on the host per call.
struct FwdParams {
    CUtensorMap tm_q;        // q  [T, H, D]      viewed (D, H, T),        box (C, G, 128/G)
    CUtensorMap tm_k;        // k  [T, Hk, D]     viewed (D, Hk, T),       box (C, 1, 128)
    CUtensorMap tm_v;        // v  same as k
    CUtensorMap tm_ck;       // cache_k [B, Hk, cap, D] viewed (D, cap, B*Hk), box (C, 128, 1); paged:
                             // pool [NB, Hk, bs, D] viewed (D, bs, NB*Hk), box (C, min(bs, 128), 1)
    CUtensorMap tm_cv;       // cache_v same
    const __nv_bfloat16* k;  // raw pointers for the cache copy
    const __nv_bfloat16* v;
    __nv_bfloat16* cache_k;
    __nv_bfloat16* cache_v;
    __nv_bfloat16* out;
    float* lse;
    WorkspaceHeader* hdr;
    const SeqInfo* seqs;
    const Unit* units;
    int n_heads, n_kv_heads, group, max_cache_len;
    float scale_log2;        // scale * log2(e)
    int causal;
    int window;              // sliding window (0: none)
    // paged cache (block_table == nullptr: contiguous [B, Hk, cap, D] slots)
    const int32_t* block_table;  // [B][max_blocks]
    int block_log2;              // block_size = 1 << block_log2 (>= 8)
    int box_rows;                // min(block_size, 128): rows of one cache TMA box
    int max_blocks;
    int num_blocks;
    // int8 cache (kv_quant): cache_k/cache_v hold int8 codes, these the fp32
    // scale of each cache row ([B, Hk, cap])
    float* scale_k;
    float* scale_v;
    int kv_quant;
    int wait_timeout_test;  // test hook: CTA 0 waits on a barrier nothing completes
    // alternating variant (bf16 cache): units whose rows fit one Q tile split
    // their KV tiles between both softmax slots (even / odd) and merge the two
    // partial results; the host picks it for decode-heavy or small launches
    int alt;
    int unit_slots;  // Q tiles per unit the scheduler cut (2, or 1 in the alternating variant)
    int out_align32;  // out is 32-byte aligned: the epilogue stores whole 32-byte sectors
};

// Encodes the tensor maps of `p` (the pointer fields and sizes must be set).
// num_blocks: blocks in the pool when p.block_table is set (else unused).
cudaError_t encode_fwd_maps(FwdParams& p, const void* q, int total_q, int num_seqs, int head_dim, int num_blocks);
cudaError_t launch_attn_fwd(const FwdParams& p, int head_dim, int grid, cudaStream_t st);

// Cached keys in two bf16 terms (k + k2 to 2^-17 of their size) and values, expanded from a 4-bit
// cache: position x of sequence b is row base[b] + x of a pool [n_kv_heads][pool_blocks * 128][head_dim],
// where the tiles that end at its last position are whole blocks (zeros below position 0).  A block's
// values are fp16 where halves[kv head][block] is not 0, else bf16.
struct FwdParamsTwo : FwdParams {
    CUtensorMap tm_ck2;  // as tm_ck
    const int* base;
    const uint8_t* halves;
    int pool_blocks;
};
cudaError_t encode_pool_maps(FwdParamsTwo& p, int head_dim, const __nv_bfloat16* k, const __nv_bfloat16* k2,
                             const __nv_bfloat16* v, long long rows);
template <int D>
cudaError_t launch_attn_two_d(const FwdParamsTwo& p, int grid, cudaStream_t st);
template <>
cudaError_t launch_attn_two_d<32>(const FwdParamsTwo& p, int grid, cudaStream_t st);
template <>
cudaError_t launch_attn_two_d<64>(const FwdParamsTwo& p, int grid, cudaStream_t st);
template <>
cudaError_t launch_attn_two_d<128>(const FwdParamsTwo& p, int grid, cudaStream_t st);

// Scheduler of the long-context variant.
struct LongScheduleArgs : ScheduleArgs {
    UnitX* xunits;
    int* seq_pieces;  // [num_seqs + 1] scheduler scratch: pieces of each sequence's query blocks
    int* pre_pieces;  // [query blocks of the whole batch][n_kv_heads] pieces of each prefix unit
    int* tok_pieces;  // [total_q] slabs that the merge joins for a token (0: none); nullptr: no merge
    int sinks;
    int prefix_len;
    const int32_t* prefix_table;
    int max_pieces, max_prefix_pieces;  // slabs the workspace has for each
    int min_tiles;  // no piece smaller than this is cut
};
cudaError_t launch_build_long_schedule(const LongScheduleArgs& a, cudaStream_t stream);

// Parameters of the long-context variant: sink tokens, a prefix the batch
// shares, and units whose tiles are split between CTAs (pieces).
struct FwdParamsX : FwdParams {
    CUtensorMap tm_pk;  // contiguous shared prefix [Hk, prefix_cap, D] viewed (D, cap, Hk), box as tm_ck
    CUtensorMap tm_pv;
    const UnitX* xunits;          // instead of `units`
    int num_seqs;                 // Unit::b of a prefix unit (its SeqInfo: all tokens, P = prefix_len)
    int sinks;                    // sink tokens (0: none)
    int prefix_len;               // tokens of the shared prefix (0: none)
    int prefix_cap;               // rows per head of a contiguous prefix
    const int32_t* prefix_table;  // blocks of a paged prefix
    const float* prefix_scale_k;  // int8 contiguous prefix: fp32 scale of each row
    const float* prefix_scale_v;
    // partial results: slab s holds rows [s * slab_rows, ...), one per (token, head):
    // normalised fp32 output and log2-sum-exp2 over the keys of the piece
    float* part_o;
    float* part_lse;
    size_t slab_rows;             // total_q * n_heads
    // a few sequences of few units: no scheduler ran, every CTA plans for itself and
    // takes the units whose list position is its own modulo the grid
    int direct;
    LongScheduleArgs plan;
};
cudaError_t encode_prefix_maps(FwdParamsX& p, int head_dim, const void* prefix_k, const void* prefix_v);
template <int D>
cudaError_t launch_attn_long_d(const FwdParamsX& p, int grid, cudaStream_t st);
template <>
cudaError_t launch_attn_long_d<32>(const FwdParamsX& p, int grid, cudaStream_t st);
template <>
cudaError_t launch_attn_long_d<64>(const FwdParamsX& p, int grid, cudaStream_t st);
template <>
cudaError_t launch_attn_long_d<128>(const FwdParamsX& p, int grid, cudaStream_t st);

// Slabs of a row that the merge joins, at most: a sequence's own pieces and the prefix's.
constexpr int kMaxPieces = 32;
constexpr int kMaxSlabs = 2 * kMaxPieces;

// Joins the partial results of every (token, head): the token's own slabs
// [0, tok_pieces) and its prefix unit's, from prefix_slab on.
struct MergeArgs {
    const float* part_o;
    const float* part_lse;
    const int* tok_pieces;
    const int* pre_pieces;  // [token / tokens_per_block][n_kv_heads]; nullptr: no prefix
    int tokens_per_block, group;
    int prefix_slab;
    __nv_bfloat16* out;
    float* lse;
    int total_q, n_heads;
};
cudaError_t launch_merge(const MergeArgs& a, int head_dim, int sms, cudaStream_t stream);

// Weight each cached key collects from the new queries.
struct KeyScheduleArgs : ScheduleArgs {
    int sinks;
};
// units: Unit{sequence, KV head, first key tile of the sequence's stream, key tiles}.
cudaError_t launch_build_key_schedule(const KeyScheduleArgs& a, cudaStream_t stream);
// The attention kernel's parameters and tensor maps (its v, cache_v and out unused).
struct KeyWeightsParams : FwdParams {
    CUtensorMap tm_q1;  // q viewed as tm_q, box (C, G, 1): one token's heads
    float* weights;  // one per cache row
    int sinks;
};
cudaError_t encode_one_token_map(KeyWeightsParams& p, const void* q, int total_q, int head_dim);
cudaError_t launch_key_weights(const KeyWeightsParams& p, int head_dim, int grid, cudaStream_t stream);

// Eviction by weight, in place.
struct EvictArgs {
    void* cache_k;
    void* cache_v;
    int row_bytes;   // of one cached key or value
    int part_bytes;  // of it that one CTA moves (set by launch_evict)
    float* scale_k;
    float* scale_v;
    const float* weights;
    float* kept_weights;
    const int32_t* lengths;
    int32_t* kept_lengths;
    int32_t* index;  // [num_seqs, n_kv_heads, budget] kept positions, -1 past the last
    WorkspaceHeader* hdr;
    int num_seqs, n_kv_heads, max_cache_len, budget, sinks, recent;
    const int32_t* block_table;
    int block_log2, max_blocks, num_blocks;
};
cudaError_t launch_evict(const EvictArgs& a, int sms, int* launches, cudaStream_t stream);

// ---- the 4-bit cache ----

// Checks a call's sequences into a.checked (n = 0 for one that is skipped).  whole: every
// table entry up to a sequence's last token counts, else only those of the call's tokens.
cudaError_t launch_check_sequences4(const Sequences4& a, const Cache4& c, bool whole, cudaStream_t stream);

// Rows of packed tokens [total_q, n_kv_heads, head_dim] into the cache, or back.
struct Copy4Params {
    Sequences4 seqs;
    Cache4 cache;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    bool aligned32;  // k_out and v_out are 32-byte aligned
    int heads;       // of K and V that a block takes (set by the launch)
};
cudaError_t launch_write_cache4(const Copy4Params& p, int head_dim, int sms, cudaStream_t stream);
cudaError_t launch_read_cache4(const Copy4Params& p, int head_dim, int sms, cudaStream_t stream);

// Long chunks: their sequences' cached rows expanded for the attention kernel, in blocks of kBlock4
// rows of a pool [n_kv_heads][pool_blocks * kBlock4][head_dim] (FwdParamsTwo).
constexpr int kBlock4 = 128;
struct Expand4Params {
    Sequences4 seqs;  // checked: where the plan writes them
    Cache4 cache;
    int few_tokens;   // sequences of up to as many new tokens are not taken
    int window;
    int pool_blocks;
    int* taken;       // [num_seqs] 0: not taken
    int* base;        // [num_seqs] the pool's row of a taken sequence's position 0 (below 0 where the pool begins later)
    int2* owners;     // [pool_blocks] sequence and first position
    int* blocks;      // in use
    __nv_bfloat16* k;
    __nv_bfloat16* k2;
    __nv_bfloat16* v;  // or fp16:
    uint8_t* halves;   // [n_kv_heads][pool_blocks] whether a block's values are
    Copy4Params write;            // the call's new tokens, written by the same launch
    int expanders, write_blocks;  // blocks that expand, blocks of tokens to write (set by the launch)
};
// Checks the sequences (like launch_check_sequences4, whole), gives those that are taken their
// blocks, in order, until the pool is full, and builds the list of their work units.
cudaError_t launch_build_schedule4(const ScheduleArgs& a, const Expand4Params& x, cudaStream_t stream);
cudaError_t launch_expand4(Expand4Params p, int head_dim, int sms, cudaStream_t stream);

// Attention of few query rows per sequence over the 4-bit cache (attn_rows4.cu).
constexpr int kRows4Seqs = 256;  // sequences whose metadata a CTA keeps in shared memory
struct Rows4Params {
    Sequences4 seqs;
    Cache4 cache;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* out;
    float* lse;
    int n_heads, group;
    float scale_log2;
    int causal, window;
    const int* taken;  // sequences that another kernel takes (not 0); nullptr: none
    // partial results that CTAs hand one another: [grid][2] of 8 rows of D
    // floats, then as many (maximum, sum) pairs; arrivals[grid] is zero between calls
    float* part;
    int* arrivals;
    float* kept;  // [grid][kRows4Warps] of 8 rows of D floats: records of a CTA's warps
};
constexpr int kRows4Warps = 16, kRows4Grid = 256;  // at most
cudaError_t launch_attn_rows4(const Rows4Params& p, int head_dim, int grid, cudaStream_t stream);
cudaError_t launch_attn_rows4_128(const Rows4Params& p, int grid, cudaStream_t stream);

}  // namespace pa
