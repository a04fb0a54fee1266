// attn_rows4.cuh -- attention of few query rows per sequence over the 4-bit cache:
// decode rows, drafts, short chunks.
//
// A row block is 8 query rows (token, head of a KV head's group) of a sequence.  (16 rows, which
// share the expansion of the codes, leave registers for 8 warps at d = 128: 8192 keys by 64 tokens
// of 32 heads took 80 us so, 70 with blocks of 8.)
// Its keys come in tiles: 32 cached rows, or 8 new tokens (bf16; as many bytes), which
// follow them.  With a group's parameters (s, m) and codes c the score and output are
//     q . k_j   = sum_g s_jg (q_g . c_jg) + m_jg sum(q_g)
//     sum_j p_j v_j = sum_j (p_j s_jg) c_jg + sum_j p_j m_jg
// so the products of codes run on the tensor cores, in fp16 with exact codes, and the
// parameters multiply in fp32.  A code in the low bits of an fp16 number is c 2^-24, in the
// next four 16 c 2^-24, both subnormal and exact: one instruction a pair of codes, and
// one shift for every four.  (With bf16 operands it is a shift, a mask and a
// subtraction: 64 decode rows of 1024 to 16384 tokens 235 us.)  fp16's range is met by powers
// of two: a query is scaled so that its largest channel is in [2^14, 2^15), what falls
// below fp16 then is 2^-38 of that (2^-34 for odd codes' channels); and p s by a factor T per
// query and group that keeps its running maximum within 2^15 (see `shrink`): its rounding to fp16,
// 2^-11 or 2^-32 of the largest p s of the group so far, is the one that there is.
//
// What bounds it is HBM: 68 bytes of key or value (d = 128, one group) feed 8 rows, where
// 128-row MMA tiles would be 15/16 empty and want the codes expanded through shared
// memory, twice its bandwidth at this rate (80 bytes written and 80 read per clock and SM
// for 128).  So a warp keeps everything in registers: S^T = K Q^T and O^T = V^T P^T with
// keys (channels) as the rows of mma.m16n8k16, 8 queries as its columns.  ldmatrix hands
// out 4 codes as one 16-bit element: plain for K (a lane gets 8 channels of one key),
// transposed for V (4 channels of two keys), and (x >> 4 i) & 0x000f000f is then an
// operand's pair of codes; the channels' order inside an MMA is free, Q is laid out to
// match.  P^T becomes an operand by movmatrix.
//
// All tiles of a call form one list (sequence, KV head, row block, tile); a CTA takes an
// equal share of it, a warp an equal share of that, in a cp.async ring of its own that
// runs on across row blocks: no barrier and no wait between warps until the end.  A row
// block cut by a share's end leaves (maximum, sum, unnormalised output); the CTA joins
// those of its warps, and the CTA that comes last joins those of the CTAs, in list order
// whoever it is.
//
// 64 rows over 1024 to 16384 tokens (32/8 heads, d = 128, group 32): 144 us, 5.0 TB/s: about
// 88 % of the copy rate between the launch (4 us), the list's making (3), the first tiles' way (5), the
// spread of the ends (6) and the joins (7).
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "cache4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace pa {

namespace rows4 {

constexpr int kTileKeys = 32;  // cached rows of a tile
constexpr int kNewKeys = 8;    // new tokens of a tile
constexpr int kRows = 8;       // query rows of a row block: the columns of an MMA
// Beginning and ending a row block costs a warp as much as several tiles, so the list has
// as many places ahead of a row block's tiles that hold none: equal shares of places are equal
// shares of time.  (64 decode rows of 256 to 4096 tokens over pages, us, with 1 / 2 / 3 / 4 / 6
// places: 62 / 62 / 60 / 58 / 58.)
constexpr int kBlockCost = 4;

template <int D, int NG>
struct Cfg {
    // As many warps as registers (16: 128 a thread, 12: 168) allow: the
    // instructions of a tile take most of the time that its bytes do, so the issue slots
    // have to be filled.
    static constexpr int kWarps = NG == 4 ? 12 : 16;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kChunks = D / 32;
    static constexpr int kRowBytes = D / 2;
    static constexpr int kCodes = kTileKeys * kRowBytes;     // bytes of a tile's codes
    static constexpr int kParams = kTileKeys * NG * 4;       // bytes of a tile's parameters
    static constexpr int kTileBytes = 2 * (kCodes + kParams);
    static constexpr int kStages = D == 128 ? 3 : 4;
    // Places of a warp's row blocks: one per tile in the ring, which may each be a row block, and one
    // for the next row block, which the feeder enters as soon as it has issued a last tile.
    static constexpr int kItems = kStages + 1;
    static constexpr int kRecord = kRows * D * 4;  // bytes of a partial output
    static_assert(kStages * kTileBytes >= 2 * kRecord, "a warp's records end up in its ring");
    static_assert(2 * kWarps <= 32, "a lane per record");
};

// A sequence (n = 0: another kernel's, or skipped).
struct Seq {
    int q_start, n, P;  // as in SeqInfo
};

// A row block in a warp's share.
struct Item {
    Seq s;
    int b, kvh, block;
    int tiles;                // of the row block
    int start_hi, start_lo;   // list position of its first
};
// What a warp needs to know of a tile in its ring: the first position of a cached tile, or
// -1 - the index of the first new token; its item's slot (bits 8 on) and the flags.
struct Tile {
    int key, flags;
};
enum : int {
    kFirst = 1,      // of the row block, in this warp
    kLast = 2,       // of the row block, in this warp
    kFromBefore = 4, // the row block began before this warp's share
    kGoesOn = 8,     // and ends after it
    kEdge = 16,      // some of the tile's keys are hidden from some row
    kSlot = 8,       // shift
};

enum : uint8_t { kNoRecord, kKept, kInRing };  // a warp's record: none, in global memory, in the ring

// Tiles of the list that a sequence's row blocks have.
struct Extent {
    int first_tile;  // first cached tile that some query sees
    int cached, fresh;
    int blocks;  // row blocks
    __device__ __forceinline__ int tiles() const { return cached + fresh; }
    __device__ __forceinline__ int places() const { return blocks > 0 ? tiles() + kBlockCost : 0; }
};

__device__ __forceinline__ Seq sequence_of(const Rows4Params& p, int b) {
    const SeqInfo s = sequence4(p.seqs, p.cache.max_cache_len, b);
    return Seq{s.q_start, p.taken && p.taken[b] ? 0 : s.n, s.P};
}

// x / y and the remainder; 32 bits of x are enough nearly always.
__device__ __forceinline__ long long divide(long long x, int y, int& rest) {
    if ((x >> 32) == 0) {
        rest = (int)((unsigned)x % (unsigned)y);
        return (long long)((unsigned)x / (unsigned)y);
    }
    rest = (int)(x % y);
    return x / y;
}

__device__ __forceinline__ Extent extent(const Rows4Params& p, const Seq& s) {
    Extent e{0, 0, 0, 0};
    if (s.n == 0) return e;
    const int lo = p.causal && p.window > 0 ? max(0, s.P - p.window + 1) : 0;  // oldest key of the first token
    e.first_tile = lo / kTileKeys;
    e.cached = max(0, (s.P + kTileKeys - 1) / kTileKeys - e.first_tile);
    e.fresh = (s.n + kNewKeys - 1) / kNewKeys;
    e.blocks = (int)(((unsigned)s.n * (unsigned)p.group + kRows - 1) / kRows);  // n * group < 2^31
    return e;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
// The same, or zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(read ? kBytes : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// the same of fp16, and without a sum before
__device__ __forceinline__ void mma_half(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_half_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// 8x8 transpose of 16-bit elements held as a matrix fragment
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max of three (one instruction on sm_100+)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Codes i and i + 4 of a word (of each 16-bit half, code i) as a pair of fp16: times 2^-24
// for even i, 2^-20 for odd.
template <int i>
__device__ __forceinline__ uint32_t codes(uint32_t x) {
    return (i >= 2 ? x >> 8 : x) & (i & 1 ? 0x00f000f0u : 0x000f000fu);
}
constexpr float kCode = 0x1p-24f;    // unit of a code
// Largest factor of the weights: scales down to 2^-126 come to 2^-8, and it times a weight of up to
// 2^9 is finite (infinity times a scale of 0 would be NaN).
constexpr int kMostLogT = 118;
constexpr float kMostT = 0x1p118f;
constexpr float kMostWeight = 0x1p15f;

__device__ __forceinline__ float to_bf16(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

template <int D>
__device__ __forceinline__ int swizzle(int key) {  // of a row's 16-byte parts
    return D == 128 ? (key >> 1) & 3 : D == 64 ? (key >> 2) & 1 : 0;
}

// One row's four channels, and its log-sum-exp; nothing of a sequence whose table is bad.
template <int D>
__device__ __forceinline__ void store_row(const Rows4Params& p, const Item& t, bool bad, int row, int d, float4 o) {
    const int r = t.block * kRows + row;
    if (bad || r >= t.s.n * p.group) return;
    const size_t at = ((size_t)(t.s.q_start + r / p.group) * p.n_heads + t.kvh * p.group + r % p.group) * D + d;
    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack(o.x, o.y), pack(o.z, o.w));
}
__device__ __forceinline__ void store_lse(const Rows4Params& p, const Item& t, bool bad, int row, float m, float l) {
    const int r = t.block * kRows + row;
    if (bad || !p.lse || r >= t.s.n * p.group) return;
    p.lse[(size_t)(t.s.q_start + r / p.group) * p.n_heads + t.kvh * p.group + r % p.group] =
        (m + log2_approx(l)) * 0.69314718055994530942f;
}

// Where a warp is in the tile list; in shared memory, read and written where it is not
// simply at the next whole cached tile of its row block.
struct Walk {
    Seq s;
    Extent e;
    long long block_start;  // list position of the row block's first tile
    int b, kvh, block;      // row block: sequence, KV head, block of rows
    int fresh;              // tiles of new tokens that came
    int lo_most;            // largest first visible key of a row
};

// Walks the tile list from a sequence on, and starts the copies of one tile at a time.
template <int D, int NG>
struct Feeder {
    using C = Cfg<D, NG>;
    static constexpr int kParts = C::kRowBytes / 16;  // 16-byte parts of a row
    static constexpr int kPassRows = 32 / kParts;     // rows that the lanes copy at once
    const Rows4Params& p;
    const Seq* table;  // in shared memory, or nullptr
    Walk* walk;
    Item* items;
    Tile* tiles;
    uint32_t ring;    // this lane's place in the first stage
    uint32_t params;  // and its parameters'
    int lane;
    int left;         // places of the share that are still to come
    int count;        // tiles that came
    int key;          // next tile if it is cached
    int whole_until;  // tiles below are whole and have no edge
    unsigned row;     // contiguous cache: row of the next cached tile
    int flags;        // of the next tile: its item's slot, kFirst and kFromBefore
    unsigned rows, next_rows;  // paged: the pool's row of the lane's 8-row piece of this and the next 256 positions

    __device__ __forceinline__ Seq seq(int i) const {
        return table ? table[i] : sequence_of(p, i);
    }
    // Puts the feeder at list position `first`; `start` is that of sequence b0.
    __device__ __forceinline__ void seek(int b0, long long start, long long first, int places) {
        left = places;
        count = key = whole_until = 0;
        flags = (C::kItems - 1) << kSlot;
        if (left == 0) return;
        Walk w;
        w.b = b0;
        w.s = seq(w.b);
        w.e = extent(p, w.s);
        for (;;) {
            const long long all = (long long)w.e.places() * w.e.blocks * p.cache.n_kv_heads;
            if (first < start + all) break;
            start += all;
            ++w.b;  // the list's total says that there is one
            w.s = seq(w.b);
            w.e = extent(p, w.s);
        }
        int place;
        const int item = (int)divide(first - start, w.e.places(), place);
        w.kvh = item / w.e.blocks;
        w.block = item % w.e.blocks;
        w.block_start = first - place + kBlockCost;
        if (place < kBlockCost) left -= kBlockCost - place;
        if (left > 0) enter(w, max(0, place - kBlockCost));
        if (lane == 0) *walk = w;
        __syncwarp();
    }
    // Begins a row block at its tile j.
    __device__ __forceinline__ void enter(Walk& w, int j) {
        key = (w.e.first_tile + min(j, w.e.cached)) * kTileKeys;
        w.fresh = max(0, j - w.e.cached);
        w.lo_most = 0;
        if (p.causal && p.window > 0)
            w.lo_most = w.s.P + min((w.block * kRows + kRows - 1) / p.group, w.s.n - 1) - p.window + 1;
        const int slot = (flags >> kSlot) + 1 == C::kItems ? 0 : (flags >> kSlot) + 1;
        flags = slot << kSlot | kFirst | (j > 0 ? kFromBefore : 0);
        if (lane == 0)
            items[slot] = Item{w.s, w.b, w.kvh, w.block, w.e.tiles(), (int)(w.block_start >> 32), (int)w.block_start};
        if (p.cache.block_table) {
            rows = piece(w.b, w.kvh, w.s.P, key >> 8);
            next_rows = piece(w.b, w.kvh, w.s.P, (key >> 8) + 1);
        } else {
            row = (unsigned)((w.b * p.cache.n_kv_heads + w.kvh) * p.cache.max_cache_len + key);  // < 2^31
        }
        whole_until = key < w.lo_most ? 0 : w.s.P / kTileKeys * kTileKeys;
    }
    // The pool's row of the lane's 8-row piece.  (The bounds keep an entry that names no block of the
    // pool, which the CTA's check of the tables finds meanwhile, from becoming a stray read; a
    // pool has less than 2^32 rows.)
    __device__ __forceinline__ unsigned piece(int b, int kvh, int P, int window) const {
        const int pos = window * 256 + lane * 8;
        if (pos >= P) return 0;
        const int id = __ldg(p.cache.block_table + (size_t)b * p.cache.max_blocks + (pos >> p.cache.block_log2));
        const unsigned block = min((unsigned)id, (unsigned)p.cache.num_blocks - 1);
        return ((block * p.cache.n_kv_heads + kvh) << p.cache.block_log2) + (pos & ((1 << p.cache.block_log2) - 1));
    }
    // paged: the pool's row of the tile's row r
    __device__ __forceinline__ unsigned pool_row(int r) const {
        return __shfl_sync(0xffffffffu, rows, ((key & 255) >> 3) + (r >> 3)) + (r & 7);
    }
    __device__ __forceinline__ void advance() {
        key += kTileKeys;
        row += kTileKeys;
        if (p.cache.block_table && (key & 255) == 0) {
            rows = next_rows;
            next_rows = piece(walk->b, walk->kvh, walk->s.P, (key >> 8) + 1);
        }
    }
    __device__ __forceinline__ void issue(int stage) {
        if (left > 0) {
            if (key < whole_until)
                issue_whole(stage);
            else
                issue_any(stage);
        }
        cp_async_commit();
    }
    // (the swizzle is the same for rows a pass apart)
    __device__ __forceinline__ void issue_whole(int stage) {
        const uint32_t dst = ring + stage * C::kTileBytes, par = params + stage * C::kTileBytes;
        if (lane == 0) tiles[stage] = Tile{key, flags | (left == 1 ? kLast | kGoesOn : 0)};
        flags &= ~kFirst;
        --left;
        ++count;
        if (!p.cache.block_table) {
            const size_t from = (size_t)row * C::kRowBytes + lane * 16;
#pragma unroll
            for (int it = 0; it < kParts; ++it) {
                cp_async16(dst + it * 512, p.cache.k + from + it * 512);
                cp_async16(dst + C::kCodes + it * 512, p.cache.v + from + it * 512);
            }
            const size_t at = (size_t)(row + lane) * NG;
            if constexpr (NG == 4) {
                cp_async16(par, p.cache.kp + at);
                cp_async16(par + C::kParams, p.cache.vp + at);
            } else {
                cp_async_small<NG * 4>(par, p.cache.kp + at);
                cp_async_small<NG * 4>(par + C::kParams, p.cache.vp + at);
            }
        } else {
#pragma unroll
            for (int it = 0; it < kParts; ++it) {
                const size_t from = (size_t)pool_row(it * kPassRows + lane / kParts) * C::kRowBytes + lane % kParts * 16;
                cp_async16(dst + it * 512, p.cache.k + from);
                cp_async16(dst + C::kCodes + it * 512, p.cache.v + from);
            }
            const size_t at = (size_t)pool_row(lane) * NG;
            if constexpr (NG == 4) {
                cp_async16(par, p.cache.kp + at);
                cp_async16(par + C::kParams, p.cache.vp + at);
            } else {
                cp_async_small<NG * 4>(par, p.cache.kp + at);
                cp_async_small<NG * 4>(par + C::kParams, p.cache.vp + at);
            }
        }
        advance();
    }
    // A cached tile at an edge, with zeros past the sequence's cached rows, or new tokens.
    __device__ __forceinline__ void issue_any(int stage) {
        Walk w = *walk;
        const uint32_t dst = ring + stage * C::kTileBytes, par = params + stage * C::kTileBytes;
        const bool cached = w.fresh == 0 && key < (w.e.first_tile + w.e.cached) * kTileKeys;
        const int at = cached ? key : -1 - w.fresh * kNewKeys;
        if (cached) {
#pragma unroll 1
            for (int it = 0; it < kParts; ++it) {
                const int r = it * kPassRows + lane / kParts;
                const bool read = key + r < w.s.P;
                const size_t from_row = p.cache.block_table ? pool_row(r) : row + r;
                const size_t from = (read ? from_row : 0) * C::kRowBytes + lane % kParts * 16;
                cp_async16(dst + it * 512, p.cache.k + from, read);
                cp_async16(dst + C::kCodes + it * 512, p.cache.v + from, read);
            }
            const bool read = key + lane < w.s.P;
            const size_t from_row = p.cache.block_table ? pool_row(lane) : row + lane;
            const size_t from = (read ? from_row : 0) * NG;
            if constexpr (NG == 4) {
                cp_async16(par, p.cache.kp + from, read);
                cp_async16(par + C::kParams, p.cache.vp + from, read);
            } else {
                cp_async_small<NG * 4>(par, p.cache.kp + from, read);
                cp_async_small<NG * 4>(par + C::kParams, p.cache.vp + from, read);
            }
            advance();
            if (key >= w.lo_most) whole_until = w.s.P / kTileKeys * kTileKeys;
        } else {
            const uint32_t base = params + stage * C::kTileBytes - lane * NG * 4 - 2 * C::kCodes;
            constexpr int kNewParts = D / 8;  // 16-byte parts of a bf16 row
#pragma unroll 1
            for (int it = 0; it < kNewParts * kNewKeys / 32; ++it) {
                const int x = it * 32 + lane, tok = w.fresh * kNewKeys + x / kNewParts;
                const bool read = tok < w.s.n;
                const size_t from =
                    ((size_t)(w.s.q_start + (read ? tok : 0)) * p.cache.n_kv_heads + w.kvh) * D + x % kNewParts * 8;
                cp_async16(base + x * 16, p.k + from, read);
                cp_async16(base + C::kCodes + x * 16, p.v + from, read);
            }
            ++w.fresh;
        }
        --left;
        ++count;
        const bool ends = w.fresh == w.e.fresh;
        int f = flags | kEdge;
        if (ends || left == 0) f |= ends ? kLast : kLast | kGoesOn;
        if (lane == 0) tiles[stage] = Tile{at, f};
        flags &= ~kFirst;
        if (ends && left > 0) {
            w.block_start += w.e.places();
            if (++w.block == w.e.blocks) {
                w.block = 0;
                if (++w.kvh == p.cache.n_kv_heads) {
                    w.kvh = 0;
                    do {
                        ++w.b;
                        w.s = seq(w.b);
                        w.e = extent(p, w.s);
                    } while (w.e.blocks == 0);
                }
            }
            left -= kBlockCost;
            if (left > 0) enter(w, 0);
        }
        __syncwarp();
        if (lane == 0) *walk = w;
        __syncwarp();
    }
};

template <int D, int NG>
__global__ void __launch_bounds__(Cfg<D, NG>::kThreads, 1) attn_rows4_kernel(const Rows4Params p) {
    using C = Cfg<D, NG>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    constexpr int kGroupChunks = C::kChunks / NG;  // 32-channel chunks of a group
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Seq table[kRows4Seqs];
    __shared__ unsigned bad_tables[kRows4Seqs / 32];  // a bit per sequence of this CTA's share
    __shared__ Item items[kWarps][C::kItems];
    __shared__ Tile tiles[kWarps][C::kStages];
    __shared__ Walk walks[kWarps];
    __shared__ Item records[kWarps][2];
    __shared__ uint8_t record_kinds[kWarps][2];
    __shared__ float2 stats[kWarps][2][kRows];  // (maximum, sum) of a record's rows
    __shared__ __align__(16) float2 factors[NG > 1 ? kWarps : 1][4][NG];
    __shared__ long long warp_sums[kWarps];
    __shared__ long long start_of_first;
    __shared__ int first_seq, last_seq;
    __shared__ bool joins[2];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t4 = lane % 4;
    griddep_wait();

    // ---- the list: its length, and the sequence that this CTA's share begins in
    const bool in_table = p.seqs.num_seqs <= kRows4Seqs;
    if (in_table) {
        if (tid < p.seqs.num_seqs) {
            Seq s;
            if (p.seqs.checked) {
                s = sequence_of(p, tid);
            } else {
                const SeqInfo stated = stated_sequence(p.seqs, p.cache.max_cache_len, tid);
                if (blockIdx.x == 0 && stated.n < 0) atomicOr(&p.seqs.hdr->error, PA_DEVERR_METADATA);
                s = Seq{stated.q_start, max(stated.n, 0), stated.P};
            }
            table[tid] = s;
        }
        if (tid < kRows4Seqs / 32) bad_tables[tid] = 0;
    } else if (!p.seqs.checked && blockIdx.x == 0) {
        for (int b = tid; b < p.seqs.num_seqs; b += kThreads)
            if (stated_sequence(p.seqs, p.cache.max_cache_len, b).n < 0) atomicOr(&p.seqs.hdr->error, PA_DEVERR_METADATA);
    }
    auto places_of = [&](int b) -> long long {
        if (b >= p.seqs.num_seqs) return 0;
        const Extent e = extent(p, in_table ? table[b] : sequence_of(p, b));
        return (long long)e.places() * e.blocks * p.cache.n_kv_heads;
    };
    // exclusive prefix sum over the CTA; total: the sum
    auto scan = [&](long long x, long long& total) -> long long {
        long long inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) warp_sums[warp] = inc;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const long long y = warp_sums[w];
            if (w < warp) before += y;
            total += y;
        }
        __syncthreads();
        return before + inc - x;
    };
    long long all = 0, mine = 0, excl = 0;
    for (int b0 = 0; b0 < p.seqs.num_seqs; b0 += kThreads) {
        long long total;
        mine = places_of(b0 + tid);
        excl = all + scan(mine, total);
        all += total;
    }
    // shares of at least a place per warp
    int rest;
    const long long share = max((long long)kWarps, (long long)divide(all + gridDim.x - 1, gridDim.x, rest));
    const long long from = min(all, share * blockIdx.x), to = min(all, from + share);
    if (from >= to) return;  // (the whole CTA)
    const bool check_tables = in_table && p.cache.block_table && !p.seqs.checked;
    if (in_table) {
        if (mine > 0 && excl <= from && from < excl + mine) first_seq = tid, start_of_first = excl;
        if (mine > 0 && excl < to && to <= excl + mine) last_seq = tid;
    } else {
        long long before = 0;
        for (int b0 = 0; b0 < p.seqs.num_seqs && before <= from; b0 += kThreads) {
            long long total;
            const long long x = places_of(b0 + tid), ex = before + scan(x, total);
            if (x > 0 && ex <= from && from < ex + x) first_seq = b0 + tid, start_of_first = ex;
            before += total;
        }
    }
    if (tid < 2 * kWarps) record_kinds[tid / 2][tid % 2] = kNoRecord;
    __syncthreads();

    // ---- this warp's share
    uint8_t* const ring = smem + warp * C::kStages * C::kTileBytes;
    // a warp's first record, where its share goes on after it (at the end the ring has room)
    float* const kept = p.kept + ((size_t)blockIdx.x * kWarps + warp) * kRows * D;
    const long long len = to - from;
    const long long wfrom = from + len * warp / kWarps, wto = from + len * (warp + 1) / kWarps;
    constexpr int kParts = C::kRowBytes / 16;
    Feeder<D, NG> feed{p, in_table ? table : nullptr, &walks[warp], items[warp], tiles[warp],
                       ptx::smem_u32(ring) + lane / kParts * C::kRowBytes + (lane % kParts ^ swizzle<D>(lane / kParts)) * 16,
                       ptx::smem_u32(ring) + 2 * C::kCodes + lane * NG * 4, lane};
    feed.seek(first_seq, start_of_first, wfrom, (int)(wto - wfrom));  // (2^31 tiles of a warp would take an hour)
    uint32_t qf[C::kChunks][4];  // Q as the second operand: per chunk two 16-channel steps
    // sums of query g's channels by group, each as three bf16 terms, as the second operand of
    // the minima's product: places 0 .. NG - 1 the first terms, then the second, then the third
    uint32_t qsum[2];
    float o[C::kChunks][2][4];   // O^T: channels 32 c + 4 g + 2 e (+ 1), queries 2 t4, 2 t4 + 1
    float2 om[NG];               // sum of p m over this lane's keys
    float2 l;                    // sum of p over this lane's keys
    float2 scale;                // from scores as they are accumulated to log2 units
    float2 neg, most;            // less the running maximum m (log2 units; 0 before any key), (m + 8) / scale
    // Factor T of p s in the second product, and of O with it, of each group: one for all would leave the
    // weights of a group whose scales are 2^-20 of another's few bits.  They change seldom, so those
    // of more than one group are in shared memory (64 rows over 1024 to 16384 tokens, groups of 32: 154 us;
    // in registers, which spill, 185; one factor for all groups 157).
    float2 T_one;
    auto factor = [&](int a) -> float2 { return NG > 1 ? factors[NG > 1 ? warp : 0][t4][a] : T_one; };
    auto set_factor = [&](int a, const float2& t) {  // (between two meetings of the warp)
        if (NG == 1)
            T_one = t;
        else if (g == 0)
            factors[NG > 1 ? warp : 0][t4][a] = t;
    };
    auto all_factors = [&](float2 (&T)[NG]) {
        if constexpr (NG == 1) {
            T[0] = T_one;
        } else {
#pragma unroll
            for (int a = 0; a < NG; a += 2) {
                const float4 x = *reinterpret_cast<const float4*>(&factors[warp][t4][a]);
                T[a] = make_float2(x.x, x.y), T[a + 1] = make_float2(x.z, x.w);
            }
        }
    };

    // Whether a sequence is to be skipped whole because its table names a block outside the pool: the
    // CTA looks through the tables of the sequences in its share while the first tiles
    // come (a block id is clamped where it is used, so nothing faults meanwhile).
    auto bad_table = [&](int b) -> bool { return check_tables && (bad_tables[b / 32] >> b % 32 & 1) != 0; };

    int stage = 1;  // (the first pass fills stage 0)
#pragma unroll 1
    for (int i = 1 - C::kStages;; ++i, stage = stage + 1 == C::kStages ? 0 : stage + 1) {
        feed.issue(stage == 0 ? C::kStages - 1 : stage - 1);
        if (i < 0) continue;
        if (i == 0 && check_tables) {
            for (int b = first_seq; b <= last_seq; ++b) {
                const Seq s = table[b];
                const int end = s.n > 0 ? ((s.P + s.n - 1) >> p.cache.block_log2) + 1 : 0;
                const int32_t* entries = p.cache.block_table + (size_t)b * p.cache.max_blocks;
                bool bad = false;
#pragma unroll 4
                for (int x = tid; x < end; x += kThreads) bad |= (unsigned)__ldg(entries + x) >= (unsigned)p.cache.num_blocks;
                if (bad) {
                    atomicOr(&bad_tables[b / 32], 1u << b % 32);
                    atomicOr(&p.seqs.hdr->error, PA_DEVERR_METADATA);
                }
            }
            __syncthreads();
        }
        if (i >= feed.count) break;  // (the feeder is ahead)
        __syncwarp();
        const int flags = tiles[warp][stage].flags, key = tiles[warp][stage].key;
        const Item& t = items[warp][flags >> kSlot];
        const uint8_t* const tile = ring + stage * C::kTileBytes;
        const uint32_t tile_u32 = ptx::smem_u32(tile);

        if (flags & kFirst) {
            const Seq s = t.s;
            const int r = t.block * kRows + g;
            const bool there = r < s.n * p.group;
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + ((size_t)(s.q_start + (there ? r / p.group : 0)) * p.n_heads + t.kvh * p.group + (there ? r % p.group : 0)) * D);
            uint4 x[C::kChunks];  // channels 32 c + 8 t4 ...
            uint32_t top2 = 0;    // largest magnitude, of pairs
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                x[c] = there ? __ldg(src + 4 * c + t4) : make_uint4(0, 0, 0, 0);
                const uint32_t y[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) top2 = __vmaxu2(top2, y[i] & 0x7fff7fffu);
            }
            uint32_t top1 = max(top2 & 0xffffu, top2 >> 16);
            top1 = max(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
            top1 = max(top1, __shfl_xor_sync(0xffffffffu, top1, 2));
            // its largest channel goes to [2^14, 2^15)
            const int up = min(268 - (int)(top1 >> 7), 253);
            const float f = __int_as_float(up << 23);
            // (never 0: hidden keys' scores are -inf, and a query of zeros or a tiny scale leaves them so)
            const float un = fmaxf(__int_as_float((254 - up) << 23) * (p.scale_log2 / kCode), 0x1p-126f);
            float sum[NG];
#pragma unroll
            for (int a = 0; a < NG; ++a) sum[a] = 0.f;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                const float y[8] = {bf16_lo(x[c].x) * f, bf16_hi(x[c].x) * f, bf16_lo(x[c].y) * f, bf16_hi(x[c].y) * f,
                                    bf16_lo(x[c].z) * f, bf16_hi(x[c].z) * f, bf16_lo(x[c].w) * f, bf16_hi(x[c].w) * f};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = i & 1 ? 0.0625f : 1.f;  // odd codes come 16 times as large
                    qf[c][i] = pack_half(y[i] * w, y[i + 4] * w);
                    sum[c / kGroupChunks] += y[i] + y[i + 4];
                }
            }
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                sum[a] += __shfl_xor_sync(0xffffffffu, sum[a], 1);
                sum[a] += __shfl_xor_sync(0xffffffffu, sum[a], 2);  // of query g
                sum[a] *= kCode;
                om[a] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float term[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int place = 8 * h + 2 * t4 + e;
                    float x = 0.f;
#pragma unroll
                    for (int a = 0; a < NG; ++a) {
                        const float first = to_bf16(sum[a]), second = to_bf16(sum[a] - first);
                        if (place == a) x = first;
                        if (place == NG + a) x = second;
                        if (place == 2 * NG + a) x = sum[a] - first - second;
                    }
                    term[e] = x;
                }
                qsum[h] = pack(term[0], term[1]);
            }
            scale.x = __shfl_sync(0xffffffffu, un, 8 * t4);
            scale.y = __shfl_sync(0xffffffffu, un, 8 * t4 + 4);
            neg = l = make_float2(0.f, 0.f);
            most = both(-INFINITY);
#pragma unroll
            for (int a = 0; a < NG; ++a) set_factor(a, both(kMostT));
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[c][e / 4][e % 4] = 0.f;
        }
        cp_async_wait<C::kStages - 1>();  // (after the queries' loads: both come at once)
        __syncwarp();
        // keys [lo, hi] that row 2 t4 + e sees
        auto visible = [&](int e, int& lo, int& hi) {
            const int tok = min((t.block * kRows + 2 * t4 + e) / p.group, t.s.n - 1);
            hi = p.causal ? t.s.P + tok : t.s.P + t.s.n - 1;
            lo = p.causal && p.window > 0 ? t.s.P + tok - p.window + 1 : 0;
        };

        // The running maximum, from the largest score `top` of the lane's keys: it is raised, and
        // what was summed under it scaled, only when it falls behind by more than 2^8.  O keeps
        // its size, T is what grows.
        auto scale_o = [&](int a, float x, float y) {  // of a group's channels
#pragma unroll
            for (int c = 0; c < kGroupChunks; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[a * kGroupChunks + c][e / 4][e % 4] *= e & 1 ? y : x;
        };
        auto raise = [&](const float2& top) {
            if (!__any_sync(0xffffffffu, top.x > most.x || top.y > most.y)) return;
            float alpha[2], x[2] = {top.x, top.y};
            const float was[2] = {most.x, most.y}, less[2] = {neg.x, neg.y}, sc[2] = {scale.x, scale.y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 4));
                x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 8));
                x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 16));
                x[e] *= sc[e];
                const bool none = was[e] == -INFINITY;  // no key before
                if (!none) x[e] = fmaxf(x[e], -less[e]);
                alpha[e] = none ? 0.f : exp2_approx(-less[e] - x[e]);
            }
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                const float2 was_t = factor(a);
                const float t0[2] = {was_t.x, was_t.y};
                float t[2], less_o[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (t / t0 is 1 / alpha at most, which is finite: alpha is 2^-126 at least, or 0)
                    t[e] = alpha[e] == 0.f ? kMostT : fminf(__fdividef(t0[e], alpha[e]), kMostT);
                    less_o[e] = alpha[e] == 0.f ? 0.f : alpha[e] * (t[e] / t0[e]);
                }
                scale_o(a, less_o[0], less_o[1]);
                __syncwarp();
                set_factor(a, make_float2(t[0], t[1]));
                om[a].x *= alpha[0], om[a].y *= alpha[1];
            }
            __syncwarp();
            l.x *= alpha[0], l.y *= alpha[1];
            if (x[0] != -INFINITY) neg.x = -x[0], most.x = (x[0] + 8.f) / sc[0];
            if (x[1] != -INFINITY) neg.y = -x[1], most.y = (x[1] + 8.f) / sc[1];
        };
        // The factor of a group's weights that reach `top` without it: where one would pass kMostWeight,
        // the largest goes to [2^7, 2^8).
        auto shrink = [&](int a, const float2& top) {
            float t[2], x[2] = {top.x, top.y};
            const float2 was = factor(a);
            const float t0[2] = {was.x, was.y};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 4));
                x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 8));
                x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 16));
                x[e] = fminf(x[e], 0x1p127f);
                t[e] = x[e] * t0[e] > kMostWeight ? __int_as_float(min(261 - (__float_as_int(x[e]) >> 23), 127 + kMostLogT) << 23) : t0[e];
            }
            scale_o(a, t[0] / t0[0], t[1] / t0[1]);
            __syncwarp();
            set_factor(a, make_float2(t[0], t[1]));
        };

        if (key >= 0) {
            // ---- 32 cached keys: octet k of them in the matrix rows g of half k / 2
            // scores of key 8 k + g (accumulators 2 (k % 2) of half k / 2), queries 2 t4 and 2 t4 + 1:
            // first what the minima add
            float score[2][4];
            const uint32_t row_addr = tile_u32 + lane * C::kRowBytes;
            const uint32_t* kp = reinterpret_cast<const uint32_t*>(tile + 2 * C::kCodes) + g * NG;
            const uint32_t* vp = kp + kTileKeys * NG;
            constexpr int kPair = NG > 1 ? 2 : 1;  // groups of a lane's two places
            const uint32_t* const km = kp + kPair * (NG == 4 ? t4 & 1 : 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t a0 = __byte_perm(km[16 * h * NG], km[16 * h * NG + kPair - 1], 0x7632);
                const uint32_t a1 = __byte_perm(km[(16 * h + 8) * NG], km[(16 * h + 8) * NG + kPair - 1], 0x7632);
                mma_first(score[h], a0, a1, a0, a1, qsum[0], qsum[1]);
            }
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                // (one group: even and odd steps apart, two chains of dependent products for one)
                constexpr int kChains = NG == 1 && kGroupChunks > 1 ? 2 : 1;
                float acc[kChains][2][4];
#pragma unroll
                for (int cc = 0; cc < kGroupChunks; ++cc) {
                    const int c = a * kGroupChunks + cc;
                    uint32_t x[4];
                    ldmatrix4(row_addr + (c ^ swizzle<D>(lane)) * 16, x);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a0 = codes<0>(x[2 * h]), a1 = codes<0>(x[2 * h + 1]), a2 = codes<1>(x[2 * h]),
                                       a3 = codes<1>(x[2 * h + 1]), b0 = codes<2>(x[2 * h]), b1 = codes<2>(x[2 * h + 1]),
                                       b2 = codes<3>(x[2 * h]), b3 = codes<3>(x[2 * h + 1]);
                        if (cc == 0)
                            mma_half_first(acc[0][h], a0, a1, a2, a3, qf[c][0], qf[c][1]);
                        else
                            mma_half(acc[0][h], a0, a1, a2, a3, qf[c][0], qf[c][1]);
                        if (cc == 0 && kChains == 2)
                            mma_half_first(acc[kChains - 1][h], b0, b1, b2, b3, qf[c][2], qf[c][3]);
                        else
                            mma_half(acc[kChains - 1][h], b0, b1, b2, b3, qf[c][2], qf[c][3]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float sk = bf16_lo(kp[8 * k * NG + a]);
                    const int h = k / 2, i = 2 * (k & 1);
                    float2 qc = make_float2(acc[0][h][i], acc[0][h][i + 1]);
                    if (kChains == 2) qc = __fadd2_rn(qc, make_float2(acc[kChains - 1][h][i], acc[kChains - 1][h][i + 1]));
                    score[h][i] = fmaf(sk, qc.x, score[h][i]);
                    score[h][i + 1] = fmaf(sk, qc.y, score[h][i + 1]);
                }
            }
            float2 sc[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[k] = make_float2(score[k / 2][2 * (k & 1)], score[k / 2][2 * (k & 1) + 1]);
            if (flags & kEdge) {
                // the end of the cached keys, or an edge of a window
                const int P = t.s.P;
                int lo[2], hi;
                visible(0, lo[0], hi);
                visible(1, lo[1], hi);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int pos = key + 8 * k + g;
                    if (pos >= P || pos < lo[0]) sc[k].x = -INFINITY;
                    if (pos >= P || pos < lo[1]) sc[k].y = -INFINITY;
                }
            }
            float2 top;
            top.x = fmaxf(max3(sc[0].x, sc[1].x, sc[2].x), sc[3].x);
            top.y = fmaxf(max3(sc[0].y, sc[1].y, sc[2].y), sc[3].y);
            raise(top);
            float2 T[NG];
            all_factors(T);
            float sv[4][NG];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 x = __ffma2_rn(sc[k], scale, neg);
                const float2 pr = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                l = __fadd2_rn(l, pr);
                sc[k] = pr;
#pragma unroll
                for (int a = 0; a < NG; ++a) {
                    const uint32_t w = vp[8 * k * NG + a];
                    const float mv = bf16_hi(w);
                    sv[k][a] = bf16_lo(w);
                    om[a] = make_float2(fmaf(pr.x, mv, om[a].x), fmaf(pr.y, mv, om[a].y));
                }
            }
            uint32_t pt[NG][4];  // P^T times the values' scales and T, per octet
#pragma unroll 1
            for (int pass = 0;; ++pass) {
                float most_w = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int a = 0; a < NG; ++a) {
                        const float2 x = __fmul2_rn(sc[k], T[a]);
                        const float2 w = make_float2(x.x * sv[k][a], x.y * sv[k][a]);
                        most_w = max3(most_w, w.x, w.y);
                        pt[a][k] = pack_half(w.x, w.y);
                    }
                }
                if (pass > 0 || !__any_sync(0xffffffffu, most_w > kMostWeight)) break;
#pragma unroll
                for (int a = 0; a < NG; ++a) {
                    float2 top_w = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        top_w.x = fmaxf(top_w.x, sc[k].x * sv[k][a]);
                        top_w.y = fmaxf(top_w.y, sc[k].y * sv[k][a]);
                    }
                    shrink(a, top_w);
                }
                __syncwarp();
                all_factors(T);
            }
#pragma unroll
            for (int a = 0; a < NG; ++a)
#pragma unroll
                for (int k = 0; k < 4; ++k) pt[a][k] = movmatrix(pt[a][k]);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                const int a = c / kGroupChunks;
                uint32_t x[4];
                ldmatrix4_trans(row_addr + C::kCodes + (c ^ swizzle<D>(lane)) * 16, x);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a0 = codes<0>(x[2 * h]), a1 = codes<1>(x[2 * h]), a2 = codes<0>(x[2 * h + 1]),
                                   a3 = codes<1>(x[2 * h + 1]), b0 = codes<2>(x[2 * h]), b1 = codes<3>(x[2 * h]),
                                   b2 = codes<2>(x[2 * h + 1]), b3 = codes<3>(x[2 * h + 1]);
                    mma_half(o[c][0], a0, a1, a2, a3, pt[a][2 * h], pt[a][2 * h + 1]);
                    mma_half(o[c][1], b0, b1, b2, b3, pt[a][2 * h], pt[a][2 * h + 1]);
                }
            }
        } else {
            // ---- up to 8 new tokens, bf16: the matrix rows g of one tile.  Q goes back to bf16;
            // scores and outputs keep the units of the codes' products.
            auto as_bf16 = [](uint32_t h, float w) -> uint32_t {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
                return pack(x.x * w, x.y * w);
            };
            const int tok0 = -1 - key, tok = tok0 + g, many = t.s.n, P = t.s.P;
            float acc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = 0.f;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                const uint4 x = *reinterpret_cast<const uint4*>(tile + g * 2 * D + 64 * c + 16 * t4);
                mma(acc, __byte_perm(x.x, x.z, 0x5410), 0, __byte_perm(x.x, x.z, 0x7632), 0, as_bf16(qf[c][0], 1.f),
                    as_bf16(qf[c][1], 16.f));
                mma(acc, __byte_perm(x.y, x.w, 0x5410), 0, __byte_perm(x.y, x.w, 0x7632), 0, as_bf16(qf[c][2], 1.f),
                    as_bf16(qf[c][3], 16.f));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                int lo, hi;
                visible(e, lo, hi);
                acc[e] = tok >= many || P + tok > hi || P + tok < lo ? -INFINITY : acc[e] * kCode;
            }
            const float2 top = make_float2(acc[0], acc[1]);
            raise(top);
            // the weights here are p itself, at most: T is what scaled it to fp16's range so far
            constexpr float kOwn = 1.f / kCode;
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                const float2 T = factor(a);
                if (__any_sync(0xffffffffu, T.x > kOwn || T.y > kOwn)) {
                    const float2 t1 = make_float2(fminf(T.x, kOwn), fminf(T.y, kOwn));
                    scale_o(a, t1.x / T.x, t1.y / T.y);
                    set_factor(a, t1);  // (the lanes have met)
                }
            }
            __syncwarp();
            const float2 x = __ffma2_rn(top, scale, neg);
            const float2 pr = make_float2(exp2_approx(x.x), exp2_approx(x.y));
            l = __fadd2_rn(l, pr);
            uint32_t pt[NG];
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                const float2 T = factor(a);
                pt[a] = movmatrix(pack(pr.x * T.x * kCode, pr.y * T.y * kCode));
            }
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) {
                const uint8_t* v = tile + C::kCodes + 64 * c + 8 * g;
                const uint2 x = *reinterpret_cast<const uint2*>(v + 2 * t4 * 2 * D);
                const uint2 y = *reinterpret_cast<const uint2*>(v + (2 * t4 + 1) * 2 * D);
                // odd channels 16 times as large, as the codes' are
                auto odd = [](uint32_t lo, uint32_t hi) -> uint32_t { return pack(bf16_hi(lo) * 16.f, bf16_hi(hi) * 16.f); };
                const uint32_t v1 = odd(x.x, y.x), v3 = odd(x.y, y.y);
                mma(o[c][0], __byte_perm(x.x, y.x, 0x5410), v1, 0, 0, pt[c / kGroupChunks], 0);
                mma(o[c][1], __byte_perm(x.y, y.y, 0x5410), v3, 0, 0, pt[c / kGroupChunks], 0);
            }
            if (t.block == 0 && !bad_table(t.b)) {
                // their rows go into the cache, once per KV head
                constexpr int kLanes = D / 8, kStep = 32 / kLanes;
                constexpr int kGroupLanes = kLanes / NG;
                const int part = lane % kLanes;
                for (int r0 = 0; r0 < kNewKeys && tok0 + r0 < many; r0 += kStep) {
                    const int r = r0 + lane / kLanes;
                    uint32_t kw, vw, kc[1], vc[1];
                    const uint4 kx[1] = {*reinterpret_cast<const uint4*>(tile + r * 2 * D + part * 16)};
                    const uint4 vx[1] = {*reinterpret_cast<const uint4*>(tile + C::kCodes + r * 2 * D + part * 16)};
                    quantise<kGroupLanes>(kx, kc, &kw);
                    quantise<kGroupLanes>(vx, vc, &vw);
                    if (tok0 + r >= many) continue;
                    const size_t row = row4(p.cache, t.b, t.kvh, P + tok0 + r);
                    if (row == ~size_t(0)) continue;
                    reinterpret_cast<uint32_t*>(p.cache.k + row * C::kRowBytes)[part] = kc[0];
                    reinterpret_cast<uint32_t*>(p.cache.v + row * C::kRowBytes)[part] = vc[0];
                    if (part % kGroupLanes == 0) {
                        p.cache.kp[row * NG + part / kGroupLanes] = kw;
                        p.cache.vp[row * NG + part / kGroupLanes] = vw;
                    }
                }
                __syncwarp();
            }
        }

        if (flags & kLast) {
            const bool whole = !(flags & (kFromBefore | kGoesOn));
            const int slot = flags & kFromBefore ? 0 : 1;
            // where the share ends the ring is done with: its copies have landed
            const bool at_end = i + 1 >= feed.count;
            float* const rec = !at_end ? kept : reinterpret_cast<float*>(ring) + (slot == 0 ? kRows * D : 0);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = e ? l.y : l.x;
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                float add[NG];
#pragma unroll
                for (int a = 0; a < NG; ++a) {
                    float y = e ? om[a].y : om[a].x;
                    y += __shfl_xor_sync(0xffffffffu, y, 4);
                    y += __shfl_xor_sync(0xffffffffu, y, 8);
                    y += __shfl_xor_sync(0xffffffffu, y, 16);
                    add[a] = y;
                }
                const int row = 2 * t4 + e;
                const float f = whole ? 1.f / x : 1.f;
                // (-inf where the share's keys are all hidden from the row)
                const float m = (e ? most.y : most.x) == -INFINITY ? -INFINITY : -(e ? neg.y : neg.x);
#pragma unroll
                for (int c = 0; c < C::kChunks; ++c) {
                    const float2 T = factor(c / kGroupChunks);
                    const float un = f / (kCode * (e ? T.y : T.x)), odd = 0.0625f * un;
                    const float y = add[c / kGroupChunks] * f;
                    const float4 v = make_float4(fmaf(o[c][0][e], un, y), fmaf(o[c][0][2 + e], odd, y),
                                                 fmaf(o[c][1][e], un, y), fmaf(o[c][1][2 + e], odd, y));
                    if (whole)
                        store_row<D>(p, t, bad_table(t.b), row, 32 * c + 4 * g, v);
                    else
                        *reinterpret_cast<float4*>(rec + row * D + 32 * c + 4 * g) = v;
                }
                if (g == 0) {
                    if (whole)
                        store_lse(p, t, bad_table(t.b), row, m, x);
                    else
                        stats[warp][slot][row] = make_float2(m, x);
                }
            }
            if (!whole && lane == 0) {
                records[warp][slot] = t;
                record_kinds[warp][slot] = at_end ? kInRing : kKept;
            }
        }
        __syncwarp();
    }
    cp_async_wait<0>();
    constexpr int kElems = kRows * D;
    __syncwarp();
    if (record_kinds[warp][0] == kKept) {
        // the first record joins the second one in the ring
        float4* const to = reinterpret_cast<float4*>(ring) + kElems / 4;
#pragma unroll
        for (int x = 0; x < kElems / 128; ++x) to[32 * x + lane] = __ldcg(reinterpret_cast<const float4*>(kept) + 32 * x + lane);
    }
    __syncthreads();

    // ---- the CTA's records (one per lane), in list order: neighbours of one row block are joined
    auto record_data = [&](int i) -> const float* {
        return reinterpret_cast<const float*>(smem + i / 2 * C::kStages * C::kTileBytes) + (i & 1 ? 0 : kElems);
    };
    float2* const part_stats = reinterpret_cast<float2*>(p.part + (size_t)gridDim.x * 2 * kElems);
    unsigned valid, begins;  // of the records; where a row block's first one is
    {
        const bool have = lane < 2 * kWarps && record_kinds[lane / 2][lane & 1] != kNoRecord;
        valid = __ballot_sync(0xffffffffu, have);
        const int hi = have ? records[lane / 2][lane & 1].start_hi : 0, lo = have ? records[lane / 2][lane & 1].start_lo : 0;
        const unsigned before = valid & ((1u << lane) - 1);
        const int prev = before ? 31 - __clz(before) : lane;
        const int prev_hi = __shfl_sync(0xffffffffu, hi, prev), prev_lo = __shfl_sync(0xffffffffu, lo, prev);
        begins = __ballot_sync(0xffffffffu, have && !(before != 0 && prev_hi == hi && prev_lo == lo));
    }
    // the first record's row block may have begun in a CTA before, the last one's may go on
    auto start_of = [&](int i) -> long long {
        const Item& t = records[i / 2][i & 1];
        return ((long long)t.start_hi << 32) | (unsigned)t.start_lo;
    };
    if (begins == 0) return;  // (the whole CTA)
    int shared[2];            // records of the row blocks that other CTAs share: it began before, it goes on
    {
        const int i = __ffs(begins) - 1, k = 31 - __clz(begins);
        shared[0] = start_of(i) < from ? i : -1;
        shared[1] = start_of(k) >= from && start_of(k) + records[k / 2][k & 1].tiles > to ? k : -1;
    }
    // a warp takes 128 channels of a row block at a time
    constexpr int kUnits = kElems / 128;
    const int rank = __popc(begins & ((1u << lane) - 1)), row_blocks = __popc(begins);
    for (int u = warp; u < row_blocks * kUnits; u += kWarps) {
        const int i = __ffs(__ballot_sync(0xffffffffu, (begins >> lane & 1) && rank == u / kUnits)) - 1;
        const unsigned later = begins & ~((2u << i) - 1);
        unsigned members = valid & ~((1u << i) - 1) & (later ? (later & -later) - 1 : 0xffffffffu);
        const int x = u % kUnits * 128 + lane * 4, row = x / D;
        float top = -INFINITY;
        for (unsigned m = members; m != 0; m &= m - 1) {
            const int k = __ffs(m) - 1;
            top = fmaxf(top, stats[k / 2][k & 1][row].x);
        }
        float sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (; members != 0; members &= members - 1) {
            const int k = __ffs(members) - 1;
            const float2 st = stats[k / 2][k & 1][row];
            const float w = st.x == -INFINITY ? 0.f : exp2_approx(st.x - top);
            const float4 y = *reinterpret_cast<const float4*>(record_data(k) + x);
            sum = fmaf(w, st.y, sum);
            v.x = fmaf(w, y.x, v.x), v.y = fmaf(w, y.y, v.y), v.z = fmaf(w, y.z, v.z), v.w = fmaf(w, y.w, v.w);
        }
        if (i != shared[0] && i != shared[1]) {
            const Item& t = records[i / 2][i & 1];
            const float f = 1.f / sum;
            store_row<D>(p, t, bad_table(t.b), row, x % D, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
            if (x % D == 0) store_lse(p, t, bad_table(t.b), row, top, sum);
        } else {
            const size_t at = (size_t)blockIdx.x * 2 + (i == shared[0] ? 0 : 1);
            __stcg(reinterpret_cast<float4*>(p.part + at * kElems + x), v);
            if (x % D == 0) __stcg(part_stats + at * kRows + row, make_float2(top, sum));
        }
    }

    // ---- row blocks that several CTAs share: the last to arrive joins them, in list order
    if (shared[0] < 0 && shared[1] < 0) return;  // (the whole CTA)
    int c0[2], pieces[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (shared[k] < 0) continue;
        c0[k] = (int)(start_of(shared[k]) / share);
        pieces[k] = (int)((start_of(shared[k]) + records[shared[k] / 2][shared[k] & 1].tiles - 1) / share) - c0[k] + 1;
    }
    __syncthreads();
    if (tid == 0) {
        __threadfence();  // (what the CTA wrote, by way of the barrier)
        int old[2] = {-1, -1};
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (shared[k] >= 0) old[k] = atomicAdd(p.arrivals + c0[k], 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            joins[k] = shared[k] >= 0 && old[k] == pieces[k] - 1;
            if (joins[k]) p.arrivals[c0[k]] = 0;
        }
        __threadfence();
    }
    __syncthreads();
    for (int u = warp; u < 2 * kUnits; u += kWarps) {
        const int k = u / kUnits, x = u % kUnits * 128 + lane * 4, row = x / D;
        if (!joins[k]) continue;
        const int i = k == 0 ? shared[0] : shared[1], first = k == 0 ? c0[0] : c0[1], count = k == 0 ? pieces[0] : pieces[1];
        float top = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAtOnce = 8;
        for (int c = 0; c < count; c += kAtOnce) {
            float4 y[kAtOnce];
            float2 st[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                st[e] = make_float2(-INFINITY, 0.f);
                y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c + e < count) {
                    const size_t at = (size_t)(first + c + e) * 2 + (c + e == 0 ? 1 : 0);
                    st[e] = __ldcg(part_stats + at * kRows + row);
                    y[e] = __ldcg(reinterpret_cast<const float4*>(p.part + at * kElems + x));
                }
            }
            float most_here = top;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) most_here = fmaxf(most_here, st[e].x);
            const float use = most_here == -INFINITY ? 0.f : most_here;  // (no key yet: the weights are 0)
            const float f = exp2_approx(top - use);
            top = most_here;
            sum *= f;
            v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const float w = exp2_approx(st[e].x - use);
                sum = fmaf(w, st[e].y, sum);
                v.x = fmaf(w, y[e].x, v.x), v.y = fmaf(w, y[e].y, v.y), v.z = fmaf(w, y[e].z, v.z), v.w = fmaf(w, y[e].w, v.w);
            }
        }
        const Item& t = records[i / 2][i & 1];
        const float f = 1.f / sum;
        store_row<D>(p, t, bad_table(t.b), row, x % D, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        if (x % D == 0) store_lse(p, t, bad_table(t.b), row, top, sum);
    }
}

template <int D, int NG>
cudaError_t launch(const Rows4Params& p, int grid, cudaStream_t stream) {
    using C = Cfg<D, NG>;
    constexpr int kSmem = C::kWarps * C::kStages * C::kTileBytes;
    static_assert(kSmem <= 216 * 1024, "shared memory budget, beside the static part (11 KB at most)");
    static int configured_for[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !configured_for[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(attn_rows4_kernel<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured_for[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_rows4_kernel<D, NG>, p);
}

}  // namespace rows4

}  // namespace pa
