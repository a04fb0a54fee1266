// key_weights.cu -- the attention weight that each cached key collects.
//
// weights[b, h, j] (+)= sum over the new queries i of sequence b and the query
// heads g of KV head h of exp(scale * q_{i,g} . k_j - lse_{i,g}), over the
// queries that see key j (causal mask, sliding window, sink tokens).  lse is
// the log-sum-exp that the attention call wrote, so the terms are the softmax
// probabilities.  Keys [0, P) come from the cache (their weights are added to),
// keys [P, P + n) from k (their weights are set).
//
// The scores are computed transposed, S^T = K Q^T with 128 keys as the rows of
// the MMA: a key is then one TMEM lane, its sum over the queries is a sum over
// the columns that one thread reads, and no value crosses threads.  A row that
// holds no key of the sequence (before its first key, past its last one, stale
// rows of a cache block) only ever affects its own lane, which is not written.
//
// One persistent CTA per SM, 640 threads:
//   warp 0      fetches units, loads their K and Q tiles (rows = (token, head in
//               group)) into one ring of stages;
//   warps 1, 2  tcgen05 issuers (one's waits hide behind the other's MMAs);
//   warp 3      stages -lse * log2(e) of the Q tile's rows;
//   warps 4-19  four groups of four warps, an S buffer of 128 TMEM columns each:
//               the sums of exp2 over the columns, one key per thread.
//
// A wide unit is up to four key tiles against every Q tile that sees one of them:
// each Q tile brought into shared memory then feeds four MMAs (loading it for two
// key tiles at a time, the Q tiles alone -- with neither MMAs nor exponentials --
// took 164 of 270 us on an 8192-token prompt of 32 heads).  With four tiles, each
// group has a tile of its own; with one or two, two groups take a tile's Q tiles
// in turn and add their sums at the end.  Where four-tile units would leave SMs
// idle the scheduler cuts units of two.
//
// A sequence whose queries fit one Q tile (decode rows) has units that are longer
// runs of key tiles against that one Q tile, the tiles in turn to the groups; what
// bounds them is HBM.
//
// An int8 key tile is expanded in place by its group first (exact codes; the row
// scale multiplies the scores).  Every wait is bounded in time, as in the
// attention kernel.
//
// Measured (graph): 8192 tokens, 32 heads, D = 128: 208 us, 1.32 PFLOP/s; the
// tensor pipe and the exponentials are each in use 58 % of the time, for a group
// waits for its MMA and the MMA for the group's S buffer (all 512 TMEM columns are
// in use).  64 decode rows over 256-4096 cached tokens: 55 us, 6.1 TB/s in the
// kernel.
#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"
#include "ptx.cuh"
#include "schedule.cuh"

namespace pa {
using namespace ptx;

namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr int kThreads = 640;
constexpr int kLse = 3;      // Q tiles whose lse is staged
constexpr int kMaxRun = 32;  // key tiles of a unit of a one-Q-tile sequence, at most
constexpr int kGroups = 4;   // groups of sum warps = S buffers = key tiles of a wide unit, at most
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
    static constexpr int kChunkCols = D >= 64 ? 64 : 32;
    static constexpr int kChunks = D / kChunkCols;
    static constexpr int kRowBytes = kChunkCols * 2;
    static constexpr int kChunkBytes = 128 * kRowBytes;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr SmemSwizzle kSw = D >= 64 ? kSwizzle128B : kSwizzle64B;
    static constexpr int kSbo = 8 * kRowBytes;
    static constexpr int kGrpSbo = kChunks * kSbo;  // paged, two chunks: staged block by block
    static constexpr int kStages = 7;
};

struct UnitSlot {
    Unit u;  // q0: first tile (position in the sequence's stream), ntiles: key tiles
    SeqInfo s;
};

struct __align__(16) Ctrl {
    uint64_t full[7], empty[7];  // per ring stage
    uint64_t l_full[kLse], l_empty[kLse];
    uint64_t s_full[kGroups], s_empty[kGroups];  // S buffers
    uint64_t read[kGroups], conv[kGroups];       // int8 key tile of a group: codes read, tile expanded
    uint64_t pair_full[2], pair_empty[2];        // two groups on one tile: the second one's sums
    uint64_t mma_drain;
    uint64_t unit_full[2], unit_empty[2];
    UnitSlot slot[2];
    uint32_t tmem_base;
    int abort;
    alignas(16) float neg_lse[kLse][128];  // -lse * log2(e) of the Q tile's rows
    float pair[2][128];                    // two groups on one tile: the second one's sums
};

// The ring's stages in the order every role takes them: next() skips the stages
// of the resident tiles (the last unit's too while this unit's are chosen, if
// that leaves one).
struct Ring {
    int n, st = -1;
    uint32_t held = 0, before = 0, phase = 0;
    __device__ __forceinline__ explicit Ring(int stages) : n(stages) {}
    __device__ __forceinline__ void unit() {
        before = held;
        held = 0;
    }
    // The next tile's stage; `parity` of its use.
    __device__ __forceinline__ int next(bool resident, uint32_t& parity) {
        const uint32_t both = held | before;
        const uint32_t skip = resident && both != (1u << n) - 1 ? both : held;
        do {
            st = st + 1 == n ? 0 : st + 1;
        } while ((skip >> st) & 1);
        if (resident) held |= 1u << st;
        parity = (phase >> st) & 1;
        phase ^= 1u << st;
        return st;
    }
};

template <int D>
constexpr int smem_bytes() {
    using C = Cfg<D>;
    constexpr int n = C::kTileBytes * C::kStages + (int)sizeof(Ctrl);
    return n > 120 * 1024 ? n : 120 * 1024;  // one CTA per SM: it holds all 512 TMEM columns
}

__device__ __forceinline__ bool aborted(const Ctrl* c) { return *reinterpret_cast<const volatile int*>(&c->abort) != 0; }

__device__ __noinline__ bool wait_bar_slow(uint64_t* bar, uint32_t parity, Ctrl* c, WorkspaceHeader* hdr) {
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (aborted(c)) return false;
        if (globaltimer_ns() - t0 > kTimeoutNs) {
            *reinterpret_cast<volatile int*>(&c->abort) = 1;
            atomicOr(&hdr->error, PA_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Bounded wait of a converged warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Ctrl* c, WorkspaceHeader* hdr) {
    const bool ok = mbar_try_wait(bar, parity) || wait_bar_slow(bar, parity, c, hdr);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t pred = 0;
    asm volatile(
        "{\n\t.reg .pred P1;\n\t"
        "elect.sync _|P1, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, P1;\n\t}"
        : "+r"(pred));
    return pred != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four int8 codes (a word) as two words of bf16 pairs, exactly: code + 128 is
// the low mantissa byte of 2^23 + (code + 128).
__device__ __forceinline__ void expand4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const uint32_t x = codes ^ 0x80808080u;
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7540u + e)) - 8388736.0f;
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
}

// The key tiles a sequence's new queries see: stream positions [0, tiles), and
// the Q tiles of its queries.
struct SeqGeo {
    int np, nsink, gap, tiles, nq;
};

__device__ __forceinline__ SeqGeo seq_geo(const SeqInfo& s, int tps, int causal, int window, int sinks, bool paged) {
    SeqGeo g;
    g.np = prefix_tiles(s.P);
    const StreamGeo st = stream_geo(s.n, s.P, 0, s.n, causal, window, sinks, false, paged);
    g.nsink = st.nsink;
    g.gap = st.lo - st.nsink;
    g.tiles = st.nsink + st.hi - st.lo;
    g.nq = (s.n + tps - 1) / tps;
    return g;
}

// A key tile: its first row's position, and the positions [lo, hi) of the
// sequence that it holds.
struct KeyTile {
    int jt, kb, lo, hi;
};

template <bool kPaged>
__device__ __forceinline__ KeyTile key_tile_at(const SeqGeo& g, const SeqInfo& s, int x) {
    KeyTile k;
    k.jt = x < g.nsink ? x : x + g.gap;
    if (k.jt >= g.np) {
        k.kb = s.P + kBlockN * (k.jt - g.np);
        k.hi = min(k.kb + kBlockN, s.P + s.n);
    } else {
        k.kb = kPaged ? kBlockN * k.jt : s.P - kBlockN * (g.np - k.jt);
        k.hi = min(k.kb + kBlockN, s.P);
    }
    k.lo = max(k.kb, 0);
    return k;
}

// Q tiles [lo, hi) that see one of the key tiles first .. last of a unit.
struct QRange {
    int lo, hi;
};

__device__ __forceinline__ QRange unit_queries(const KeyTile& first, const KeyTile& last, const SeqInfo& s, int nq,
                                               int tps, int causal, int window, int sinks) {
    QRange r{0, nq};
    if (!causal) return r;
    if (first.lo > s.P) r.lo = (first.lo - s.P) / tps;
    if (window > 0 && first.lo >= sinks) {
        const int tok = window + (last.hi - 2 - s.P);  // last token that sees the last key
        r.hi = tok < 0 ? 0 : min(nq, tok / tps + 1);
    }
    return r;
}

// Q tiles [lo, hi) all of whose 128 columns count for every key of the tile.
__device__ __forceinline__ QRange full_queries(const KeyTile& k, const SeqInfo& s, int tps, int group, int causal,
                                               int window, int sinks) {
    QRange r{0, tps * group > kBlockN - 32 ? s.n / tps : 0};
    if (!causal) return r;
    if (k.hi - 1 > s.P) r.lo = (k.hi - 1 - s.P + tps - 1) / tps;
    if (window > 0 && k.hi > sinks) r.hi = min(r.hi, max(0, window + (k.lo - s.P)) / tps);
    return r;
}

// Key tiles of a unit of several Q tiles: four, or two where four would make fewer
// units than two per CTA (wide_tiles: the key tiles x KV heads of such sequences).
__device__ __forceinline__ int wide_length(unsigned long long wide_tiles, int num_ctas) {
    return wide_tiles >= 2ull * kGroups * (unsigned)num_ctas ? kGroups : 2;
}

// Key tiles of a unit of a sequence whose queries fit one Q tile: about three
// units per CTA of the `total` tiles of all of them (64 decode rows over 256-4096
// cached tokens, replayed: 55.0 us; 55.9 with four, 60.9 with eight, 56.4 with two).
// Single cold passes with two, three, four and eight: those rows in int8 pages 79,
// 79, 81 and 91 us; 8 rows over 16384 tokens 67, 65, 65 and 65; one row over 32768
// 28, 28, 31 and 30; 32 rows of 4 heads over 2048-32768 116, 115, 114 and 114; 256 rows
// over 128-1024 93 with each (a unit is a whole row of a head there).
__device__ __forceinline__ int run_length(unsigned long long total, int num_ctas) {
    const unsigned long long per = total / (3u * (unsigned)num_ctas);
    return per >= kMaxRun ? kMaxRun : (per < 2 ? 2 : (int)per & ~1);
}

// Writes unit x of sequence b and KV head kvh (its tiles in units of len).  A
// sequence's units: its KV heads in groups whose queries fit the L2 budget, and
// within a group the first keys first (under a causal mask the most expensive
// ones) with the group's heads adjacent.
__device__ __forceinline__ void emit_keys(const KeyScheduleArgs& a, const SeqInfo& si, int b, int x, int kvh, int tiles,
                                          int len, int units, int first) {
    // groups of one size, and none so small that its longest unit outlasts the
    // rest of it (a causal sequence's units average half its longest)
    const float head_bytes = (float)si.n * a.group * a.head_dim * 2;
    const float fit = fmaxf(floorf((float)kL2GroupBytes / fmaxf(head_bytes, 1.f)), 2.f * (float)a.num_ctas / (float)units);
    const int groups = fit >= (float)a.n_kv_heads ? 1 : (a.n_kv_heads + (int)fit - 1) / max(1, (int)fit);
    const int hg = (a.n_kv_heads + groups - 1) / groups;
    const int g0 = kvh - kvh % hg, gsize = min(hg, a.n_kv_heads - g0);
    const int pos = first + g0 * units + x * gsize + (kvh - g0);
    if (pos < a.max_units) a.units[pos] = Unit{b, kvh, x * len, min(len, tiles - x * len)};
}

__global__ void __launch_bounds__(1024) build_key_schedule_kernel(const __grid_constant__ KeyScheduleArgs a) {
    __shared__ int hist[kCostBins];
    __shared__ int warp_sums[32];
    __shared__ unsigned long long s_total, s_wide;
    __shared__ SeqInfo s_seqs[kSmemSeqs];
    __shared__ int s_first[kSmemSeqs], s_units[kSmemSeqs];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nthr = blockDim.x, nwarps = nthr >> 5;
    const int tps = kBlockM / a.group;
    griddep_launch();
    const bool small = a.num_seqs <= kSmemSeqs;
    SeqInfo* const seqs = small ? s_seqs : a.seqs;
    int* const seq_first = small ? s_first : a.seq_scratch;  // cost bin, then first unit of the sequence
    int* const seq_units = small ? s_units : a.seq_group;    // units per head
    for (int i = tid; i < kCostBins; i += nthr) hist[i] = 0;
    if (tid == 0) s_total = s_wide = 0;
    const bool paged = a.block_table != nullptr;
    for (int b = tid; b < a.num_seqs; b += nthr) seqs[b] = checked_sequence(a, b);
    __threadfence_block();
    __syncthreads();
    if (paged) {
        for (int b = warp; b < a.num_seqs; b += nwarps) {
            const bool bad = bad_visible_blocks(a.block_table + (size_t)b * a.max_blocks, seqs[b], a.block_size,
                                                a.num_blocks, a.causal, a.window, a.sinks, lane);
            if (bad && lane == 0) seqs[b].n = -1;
        }
        __threadfence_block();
        __syncthreads();
    }
    for (int b = tid; b < a.num_seqs; b += nthr) {
        SeqInfo si = seqs[b];
        if (si.n < 0) {
            atomicOr(&a.hdr->error, PA_DEVERR_METADATA);
            si = SeqInfo{0, 0, 0, 0};
            seqs[b] = si;
        }
        if (si.n > 0) {
            const SeqGeo g = seq_geo(si, tps, a.causal, a.window, a.sinks, paged);
            atomicAdd(g.nq == 1 ? &s_total : &s_wide, (unsigned long long)g.tiles * a.n_kv_heads);
        }
    }
    __threadfence_block();
    __syncthreads();
    const int run = run_length(s_total, a.num_ctas), wide = wide_length(s_wide, a.num_ctas);
    // units per sequence and head, numbered (SeqInfo::pad), and cost bins
    int before = 0;
    for (int b0 = 0; b0 < a.num_seqs; b0 += nthr) {
        const int b = b0 + tid;
        int units = 0;
        SeqInfo si{0, 0, 0, 0};
        SeqGeo g{};
        if (b < a.num_seqs) si = seqs[b];
        if (si.n > 0) {
            g = seq_geo(si, tps, a.causal, a.window, a.sinks, paged);
            const int len = g.nq == 1 ? run : wide;
            units = (g.tiles + len - 1) / len;
        }
        int chunk_total;
        const int excl = block_exclusive_scan(units, warp_sums, &chunk_total);
        if (b < a.num_seqs) {
            si.pad = before + excl;
            a.seqs[b] = si;
            if (small) s_seqs[b] = si;
            seq_units[b] = units;
            if (units > 0) {
                const int bin = cost_bin((long long)g.tiles * g.nq * a.n_kv_heads);
                seq_first[b] = bin;
                atomicAdd(&hist[bin], units * a.n_kv_heads);
            }
        }
        before += chunk_total;
    }
    __threadfence_block();
    __syncthreads();
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
    for (int b = tid; b < a.num_seqs; b += nthr)
        if (seq_units[b] > 0) seq_first[b] = atomicAdd(&hist[seq_first[b]], seq_units[b] * a.n_kv_heads);
    __threadfence_block();
    __syncthreads();
    for (int w = tid; w < before * a.n_kv_heads; w += nthr) {
        const int i = w / a.n_kv_heads, kvh = w % a.n_kv_heads;
        const int b = block_owner(seqs, a.num_seqs, i);
        const SeqInfo si = seqs[b];
        const SeqGeo g = seq_geo(si, tps, a.causal, a.window, a.sinks, paged);
        emit_keys(a, si, b, i - si.pad, kvh, g.tiles, g.nq == 1 ? run : wide, seq_units[b], seq_first[b]);
    }
}

// The same for a few sequences (kFewSeqs): see schedule.cuh.
__global__ void __launch_bounds__(kFewThreads) build_key_schedule_few_kernel(const __grid_constant__ KeyScheduleArgs a) {
    __shared__ FewSeqs f;
    __shared__ int s_tiles[kFewSeqs], s_len[kFewSeqs];
    __shared__ unsigned long long s_wide;
    const int tid = threadIdx.x, tps = kBlockM / a.group;
    const bool paged = a.block_table != nullptr;
    griddep_launch();
    if (tid == 0) s_wide = 0;
    load_few(a, f, a.sinks, nullptr, 0, true);
    SeqGeo g{};
    if (tid < a.num_seqs && f.seqs[tid].n > 0) {
        g = seq_geo(f.seqs[tid], tps, a.causal, a.window, a.sinks, paged);
        atomicAdd(g.nq == 1 ? &f.total : &s_wide, (unsigned long long)g.tiles * a.n_kv_heads);
    }
    __syncthreads();
    if (tid < a.num_seqs) {
        const int len = g.nq == 1 ? run_length(f.total, a.num_ctas) : wide_length(s_wide, a.num_ctas);
        s_tiles[tid] = g.tiles;
        s_len[tid] = len;
        f.blocks[tid] = (g.tiles + len - 1) / len;
        f.units[tid] = f.blocks[tid] * a.n_kv_heads;
        f.cost[tid] = (float)g.tiles * (float)g.nq;
    }
    __syncthreads();
    const int blocks = rank_few(a, f, a.num_seqs, true);
    for (int w = tid; w < blocks * a.n_kv_heads; w += kFewThreads) {
        const int i = w / a.n_kv_heads, kvh = w % a.n_kv_heads;
        const int b = block_owner(f.seqs, a.num_seqs, i);
        emit_keys(a, f.seqs[b], b, i - f.seqs[b].pad, kvh, s_tiles[b], s_len[b], f.blocks[b], f.first[b]);
    }
}

template <int D, bool kPaged, bool kQuant>
__global__ void __launch_bounds__(kThreads, 1) key_weights_kernel(const __grid_constant__ KeyWeightsParams p) {
    using C = Cfg<D>;
    constexpr bool kGrp = kPaged && !kQuant && C::kChunks == 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const bool misaligned = (smem_u32(smem_raw) & 1023u) != 0;
    uint8_t* const ring_smem = smem_raw;
    Ctrl* ctl = reinterpret_cast<Ctrl*>(ring_smem + C::kStages * C::kTileBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    WorkspaceHeader* hdr = p.hdr;
    const int G = p.group, tps = kBlockM / G;

    if (!misaligned && threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 2);  // the issuers: a commit, or an arrival
        }
        for (int i = 0; i < kLse; ++i) {
            mbar_init(&ctl->l_full[i], 1);
            mbar_init(&ctl->l_empty[i], 16);  // the sum warps
        }
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->s_empty[i], 4);  // the group's warps
            mbar_init(&ctl->read[i], 4);
            mbar_init(&ctl->conv[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->pair_full[i], 4);
            mbar_init(&ctl->pair_empty[i], 4);
        }
        mbar_init(&ctl->mma_drain, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->unit_full[i], 1);
            mbar_init(&ctl->unit_empty[i], kThreads / 32 - 1);  // every warp but the fetching one
        }
        ctl->abort = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tm_q);
        prefetch_tmap(&p.tm_q1);
        prefetch_tmap(&p.tm_k);
        prefetch_tmap(&p.tm_ck);
    }
    if (!misaligned && warp == 1) {
        tmem_alloc(&ctl->tmem_base, 512);
        tmem_relinquish();
    }
    griddep_wait();
    if (misaligned) {
        if (threadIdx.x == 0) atomicOr(&hdr->error, PA_DEVERR_SMEM_ALIGN);
        return;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    const int num_units = hdr->num_units;

    // On abort, let every copy this warp started land before the CTA exits.
    auto drain = [&](uint64_t* bars, uint32_t set, uint32_t par, int n) {
        const uint64_t t0 = globaltimer_ns();
        for (int i = 0; i < n; ++i)
            if ((set >> i) & 1)
                while (!mbar_try_wait(&bars[i], (par >> i) & 1) && globaltimer_ns() - t0 < kTimeoutNs) {
                }
    };
    // The next unit for a warp other than the fetching one (u.b < 0: no more); false: a wait gave up.
    auto next_unit = [&](int u_it, UnitSlot& us) -> bool {
        const int sl = u_it & 1;
        if (!warp_wait(&ctl->unit_full[sl], (u_it >> 1) & 1, ctl, hdr)) return false;
        us = ctl->slot[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->unit_empty[sl]);
        return us.u.b >= 0;
    };
    // The Q tiles of a wide unit.
    auto queries = [&](const SeqGeo& g, const SeqInfo& s, const Unit& u) {
        return unit_queries(key_tile_at<kPaged>(g, s, u.q0), key_tile_at<kPaged>(g, s, u.q0 + u.ntiles - 1), s, g.nq, tps,
                            p.causal, p.window, p.sinks);
    };
    // The Q tiles that see one key tile.
    auto seen_by = [&](const SeqGeo& g, const SeqInfo& s, const KeyTile& k) {
        return unit_queries(k, k, s, g.nq, tps, p.causal, p.window, p.sinks);
    };
    auto geo = [&](const SeqInfo& s) { return seq_geo(s, tps, p.causal, p.window, p.sinks, kPaged); };

    if (warp == 0) {
        // ---------------------------------------------- unit fetch, K and Q tiles
        Ring ring(C::kStages);
        uint32_t lp_set = 0, lp_par = 0;
        // waits for the next tile's stage to be free
        auto take = [&](bool resident, int& st) -> bool {
            uint32_t par;
            st = ring.next(resident, par);
            if (!warp_wait(&ctl->empty[st], par ^ 1, ctl, hdr)) return false;
            lp_set |= 1u << st;
            lp_par = (lp_par & ~(1u << st)) | (par << st);
            return true;
        };
        for (int u_it = 0;; ++u_it) {
            const int sl = u_it & 1;
            if (!warp_wait(&ctl->unit_empty[sl], ((u_it >> 1) & 1) ^ 1, ctl, hdr)) break;
            if (lane == 0) {
                const int idx = atomicAdd(&hdr->counter, 1);
                UnitSlot us;
                us.u.b = -1;
                if (idx < num_units) {
                    us.u = p.units[idx];
                    us.s = p.seqs[us.u.b];
                }
                ctl->slot[sl] = us;
                mbar_arrive(&ctl->unit_full[sl]);
            }
            __syncwarp();
            const Unit u = ctl->slot[sl].u;
            if (u.b < 0) break;
            const SeqInfo s = ctl->slot[sl].s;
            const SeqGeo g = geo(s);
            const bool single = g.nq == 1;
            ring.unit();
            auto load_q = [&](int qi) -> bool {
                // a decode row's Q tile is one token's heads; rows that no copy
                // fills are columns that no sum takes
                const bool one = s.n == 1;
                int st;
                if (!take(single, st)) return false;
                if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], G * (one ? 1 : tps) * C::kRowBytes * C::kChunks);
                __syncwarp();
                if (lane < C::kChunks)
                    tma_load_3d(ring_smem + st * C::kTileBytes + lane * C::kChunkBytes, one ? &p.tm_q1 : &p.tm_q,
                                &ctl->full[st], lane * C::kChunkCols, u.kvh * G, s.q_start + qi * tps);
                __syncwarp();
                return true;
            };
            bool ok = !single || load_q(0);
            for (int x = u.q0; x < u.q0 + u.ntiles && ok; ++x) {
                const KeyTile k = key_tile_at<kPaged>(g, s, x);
                const bool pre = k.jt < g.np;
                // paged prefix tile: this lane's block, fetched before the wait
                const int br = p.box_rows;
                const int boxes = kPaged && pre ? (k.hi - k.kb + br - 1) / br : 0;
                int blk = 0;
                if (kPaged && lane < boxes)
                    blk = __ldg(p.block_table + (size_t)u.b * p.max_blocks + ((k.kb + lane * br) >> p.block_log2));
                int st;
                if (!take(!single, st)) {
                    ok = false;
                    break;
                }
                uint8_t* stage = ring_smem + st * C::kTileBytes;
                uint64_t* full = &ctl->full[st];
                uint32_t bytes = C::kTileBytes;
                if (pre && kPaged) bytes = boxes * br * (kQuant ? D : C::kRowBytes * C::kChunks);
                else if (pre && kQuant) bytes = kBlockN * D;
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (!pre) {
                    if (lane < C::kChunks)
                        tma_load_3d(stage + lane * C::kChunkBytes, &p.tm_k, full, lane * C::kChunkCols, u.kvh,
                                    s.q_start + k.kb - s.P);
                } else if (kPaged) {
                    if (lane < boxes) {
                        const int row = (k.kb + lane * br) & ((1 << p.block_log2) - 1), z = blk * p.n_kv_heads + u.kvh;
                        if constexpr (kQuant) {
                            tma_load_3d(stage + C::kTileBytes / 2 + lane * br * D, &p.tm_ck, full, 0, row, z);
                        } else if constexpr (kGrp) {
                            tma_load_5d(stage + lane * br * C::kRowBytes * C::kChunks, &p.tm_ck, full, 0, 0, 0, row >> 3, z);
                        } else {
                            tma_load_3d(stage + lane * br * C::kRowBytes, &p.tm_ck, full, 0, row, z);
                        }
                    }
                } else {
                    const int z = u.b * p.n_kv_heads + u.kvh;
                    if constexpr (kQuant) {
                        if (lane == 0) tma_load_3d(stage + C::kTileBytes / 2, &p.tm_ck, full, 0, k.kb, z);
                    } else if (lane < C::kChunks) {
                        tma_load_3d(stage + lane * C::kChunkBytes, &p.tm_ck, full, lane * C::kChunkCols, k.kb, z);
                    }
                }
                __syncwarp();
            }
            if (ok && !single) {
                const QRange qr = queries(g, s, u);
                for (int qi = qr.lo; qi < qr.hi && ok; ++qi) ok = load_q(qi);
            }
            if (!ok) break;
        }
        if (lane == 0 && aborted(ctl)) drain(ctl->full, lp_set, lp_par, C::kStages);
    } else if (warp == 1 || warp == 2) {
        // --------------------------------------------------------- MMA issuers
        // Issuer me serves the S buffers me and me + 2.  Each stage's release takes
        // both: a commit by the one whose MMAs read it (both for a Q tile), an
        // arrival by the other -- which waits for the tile all the same, lest it
        // arrive for the stage's next use in this one's place.
        const int me = warp - 1;
        const bool leader = elect_one();
        const uint32_t addr = smem_u32(ring_smem);
        const uint64_t desc = smem_desc(addr, 16, C::kSbo, C::kSw);
        const uint64_t desc_g = smem_desc(addr, 16, C::kGrpSbo, C::kSw);  // staged block by block
        Ring ring(C::kStages);
        uint32_t used = 0;   // bit i: parity of the uses so far of S buffer me + 2 i
        uint32_t convs = 0;  // bit i: parity of the tiles expanded by group me + 2 i
        uint32_t nn = 0;             // tiles of one-Q-tile units so far
        bool ok = true;
        // S^T of the key tile at stage kst and the Q tile at stage qst into buffer buf
        auto issue = [&](int buf, int kst, bool grp, int qst, int cols) -> bool {
            if (!warp_wait(&ctl->s_empty[buf], ((used >> (buf >> 1)) & 1) ^ 1, ctl, hdr)) return false;
            used ^= 1u << (buf >> 1);
            tc_fence_after();
            // columns in use, rounded up to what an M = 128 MMA takes
            const uint32_t idesc = idesc_bf16_f32(kBlockM, 0, 0, 0) | ((uint32_t)((cols + 15) / 16) * 2 << 17);
            if (leader) {
                const uint64_t kd = (grp ? desc_g : desc) + ((kst * C::kTileBytes) >> 4);
                const uint64_t qd = desc + ((qst * C::kTileBytes) >> 4);
                const uint32_t kcs = grp ? C::kSbo : C::kChunkBytes;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ch = (kk * 16) / C::kChunkCols, in = ((kk * 16) % C::kChunkCols) * 2;
                    mma_ss(tmem + buf * 128, kd + ((ch * kcs + in) >> 4), qd + ((ch * C::kChunkBytes + in) >> 4), idesc,
                           kk > 0 ? 1u : 0u);
                }
                mma_commit(&ctl->s_full[buf]);
            }
            __syncwarp();
            return true;
        };
        // the key tile of group grp at stage st: landed, and expanded if it was codes
        auto wait_key = [&](int grp, bool codes, int st, uint32_t par) -> bool {
            if (!(kQuant && codes)) return warp_wait(&ctl->full[st], par, ctl, hdr);
            const bool got = warp_wait(&ctl->conv[grp], (convs >> (grp >> 1)) & 1, ctl, hdr);
            convs ^= 1u << (grp >> 1);
            return got;
        };
        auto release = [&](int st, bool mine) {
            if (leader) {
                if (mine)
                    mma_commit(&ctl->empty[st]);
                else
                    mbar_arrive(&ctl->empty[st]);
            }
            __syncwarp();
        };
        UnitSlot us;
        for (int u_it = 0; ok && next_unit(u_it, us); ++u_it) {
            const SeqInfo s = us.s;
            const SeqGeo g = geo(s);
            ring.unit();
            uint32_t par;
            if (g.nq == 1) {
                const int qst = ring.next(true, par);
                if (!warp_wait(&ctl->full[qst], par, ctl, hdr)) break;
                for (int x = us.u.q0; x < us.u.q0 + us.u.ntiles && ok; ++x, ++nn) {
                    const int kst = ring.next(false, par), grp = nn & 3;
                    const KeyTile k = key_tile_at<kPaged>(g, s, x);
                    const bool mine = (grp & 1) == me;
                    ok = mine ? wait_key(grp, k.jt < g.np, kst, par) && issue(grp, kst, kGrp && k.jt < g.np, qst, s.n * G)
                              : warp_wait(&ctl->full[kst], par, ctl, hdr);
                    if (ok) release(kst, mine);
                }
                if (ok) release(qst, true);
                continue;
            }
            const int nt = us.u.ntiles;
            const bool four = nt > 2;
            const QRange qr = queries(g, s, us.u);
            int kst[kGroups], st[2] = {0, 0};  // stages of the unit's tiles, of this issuer's tiles me and me + 2
            QRange mine[2] = {{0, 0}, {0, 0}};  // the Q tiles that see those
            bool grp[2] = {false, false};
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                kst[i] = 0;
                if (i >= nt) continue;
                kst[i] = ring.next(true, par);
                if ((i & 1) == me) {
                    const KeyTile k = key_tile_at<kPaged>(g, s, us.u.q0 + i);
                    st[i >> 1] = kst[i];
                    mine[i >> 1] = seen_by(g, s, k);
                    grp[i >> 1] = kGrp && k.jt < g.np;
                    ok = ok && wait_key(i, k.jt < g.np, kst[i], par);
                } else {
                    ok = ok && warp_wait(&ctl->full[kst[i]], par, ctl, hdr);
                }
            }
            for (int qi = qr.lo; qi < qr.hi && ok; ++qi) {
                const int cols = min(tps, s.n - qi * tps) * G;
                const int qst = ring.next(false, par);
                if (!warp_wait(&ctl->full[qst], par, ctl, hdr)) { ok = false; break; }
                bool any = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (qi < mine[i].lo || qi >= mine[i].hi || !ok) continue;
                    ok = issue(four ? me + 2 * i : me + 2 * (qi & 1), st[i], grp[i], qst, cols);
                    any = true;
                }
                if (ok) release(qst, any);
            }
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (i < nt) release(kst[i], (i & 1) == me);
        }
        // every MMA the issuers put in has finished before TMEM is released
        if (leader) {
            mma_commit(&ctl->mma_drain);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&ctl->mma_drain, 0) && globaltimer_ns() - t0 < kTimeoutNs) {
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        // --------------------------------------------------- lse of the Q tiles
        uint32_t lq = 0;
        bool ok = true;
        int col_tok[4], col_head[4];  // token and head in group of this lane's columns
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            col_tok[i] = (lane + 32 * i) / G;
            col_head[i] = (lane + 32 * i) % G;
        }
        UnitSlot us;
        for (int u_it = 0; ok && next_unit(u_it, us); ++u_it) {
            const SeqInfo s = us.s;
            const SeqGeo g = geo(s);
            const QRange qr = g.nq > 1 ? queries(g, s, us.u) : QRange{0, 1};
            float l[4];
            auto load_lse = [&](int qi) {
                const int q0 = qi * tps, qe = min(q0 + tps, s.n);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = q0 + col_tok[i];
                    // a column of no query adds exp2(-inf) = 0
                    l[i] = tok < qe && col_tok[i] < tps
                               ? -kLog2e * __ldg(p.lse + (size_t)(s.q_start + tok) * p.n_heads + us.u.kvh * G + col_head[i])
                               : -INFINITY;
                }
            };
            if (qr.lo < qr.hi) load_lse(qr.lo);
            for (int qi = qr.lo; qi < qr.hi; ++qi, ++lq) {
                const int st = lq % kLse;
                if (!warp_wait(&ctl->l_empty[st], ((lq / kLse) & 1) ^ 1, ctl, hdr)) { ok = false; break; }
#pragma unroll
                for (int i = 0; i < 4; ++i) ctl->neg_lse[st][lane + 32 * i] = l[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->l_full[st]);
                if (qi + 1 < qr.hi) load_lse(qi + 1);  // on its way during the next wait
            }
        }
    } else {
        // ------------------------------------------------------------ the sums
        const int group = (warp - 4) >> 2, sp = warp & 3;
        const int r = sp * 32 + lane;  // row of the key tile == TMEM lane
        const uint32_t col = tmem + ((uint32_t)(sp * 32) << 16) + group * 128;
        Ring ring(C::kStages);
        int lst = 0;                      // lse stage of the Q tile, and the parity of its use
        uint32_t lpar = 0, ns = 0, nn = 0;  // ns: S tiles of this group; nn: tiles of one-Q-tile units (of every group)
        uint32_t npair = 0, nread = 0;    // exchanges between two groups; tiles expanded
        bool ok = true;
        // done with the Q tile's lse
        auto next_lse = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->l_empty[lst]);
            if (++lst == kLse) {
                lst = 0;
                lpar ^= 1;
            }
        };
        // where the weight (and the scale) of key j of a tile of (b, kvh) lies
        auto weight_row = [&](const Unit& u, int j) -> size_t {
            if (kPaged) {
                const int blk = __ldg(p.block_table + (size_t)u.b * p.max_blocks + (j >> p.block_log2));
                return (((size_t)blk * p.n_kv_heads + u.kvh) << p.block_log2) + (j & ((1 << p.block_log2) - 1));
            }
            return ((size_t)u.b * p.n_kv_heads + u.kvh) * p.max_cache_len + j;
        };
        // Expands the codes (upper half of stage st) into the swizzled bf16 tile: the
        // group's warps read all of them before any writes.
        auto expand = [&](int st, uint32_t par) -> bool {
            uint8_t* stage = ring_smem + st * C::kTileBytes;
            if (!warp_wait(&ctl->full[st], par, ctl, hdr)) return false;
            constexpr int kPieces = D / 8;  // 8 codes each, per thread
            uint2 c[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                c[i] = *reinterpret_cast<const uint2*>(stage + C::kTileBytes / 2 + (r + 128 * i) * 8);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->read[group]);
            if (!warp_wait(&ctl->read[group], nread & 1, ctl, hdr)) return false;
            ++nread;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int idx = r + 128 * i, kr = idx / (D / 8), gr = idx % (D / 8);
                const int ch = gr / (C::kChunkCols / 8), gg = gr % (C::kChunkCols / 8);
                const int phys = D >= 64 ? (gg ^ (kr & 7)) : (gg ^ ((kr >> 1) & 3));
                uint4 o;
                expand4(c[i].x, o.x, o.y);
                expand4(c[i].y, o.z, o.w);
                *reinterpret_cast<uint4*>(stage + ch * C::kChunkBytes + kr * C::kRowBytes + phys * 16) = o;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->conv[group]);
            return true;
        };
        // Adds to `total` the exp2s of this group's next S tile: n columns, all of
        // them (whole), or of which this thread's key takes [lo, hi).
        auto add_tile = [&](const float* nl, int n, bool whole, int lo, int hi, float mul, float& total) -> bool {
            if (!warp_wait(&ctl->s_full[group], ns & 1, ctl, hdr)) return false;
            ++ns;
            tc_fence_after();
            float2 a0 = make_float2(0.f, 0.f), a1 = a0;
            if (whole) {
                // 32 columns are summed while the next 32 are on their way; of the
                // last 32, those past n (a group that does not divide 128) become 0,
                // and their lse is infinite
                const float2 mul2 = make_float2(mul, mul);
                uint32_t v[2][32];
                tmem_ld32(col, v[0]);
#pragma unroll
                for (int c = 0; c < kBlockN; c += 32) {
                    uint32_t (&x)[32] = v[(c / 32) & 1];
                    tmem_wait_ld();
                    reg_fence(x);
                    if (c + 32 < kBlockN) {
                        tmem_ld32(col + c + 32, v[(c / 32 + 1) & 1]);
                    } else {  // everything of the buffer is in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->s_empty[group]);
                        if (n < kBlockN) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (c + e >= n) x[e] = 0;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 l = *reinterpret_cast<const float4*>(nl + c + e);
                        const float2 s0 = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), mul2,
                                                     make_float2(l.x, l.y));
                        const float2 s1 = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])),
                                                     mul2, make_float2(l.z, l.w));
                        a0 = __fadd2_rn(a0, make_float2(ex2(s0.x), ex2(s0.y)));
                        a1 = __fadd2_rn(a1, make_float2(ex2(s1.x), ex2(s1.y)));
                    }
                }
            } else {
                for (int c = 0; c < n; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(col + c, v);
                    tmem_wait_ld();
                    reg_fence(v);
                    const int m = min(32, n - c);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        if (e >= m) break;
                        const float2 l = *reinterpret_cast<const float2*>(nl + c + e);
                        const float x0 = ex2(fmaf(__uint_as_float(v[e]), mul, l.x));
                        const float x1 = ex2(fmaf(__uint_as_float(v[e + 1]), mul, l.y));
                        a0.x += c + e >= lo && c + e < hi ? x0 : 0.f;
                        a0.y += c + e + 1 >= lo && c + e + 1 < hi ? x1 : 0.f;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->s_empty[group]);
            }
            total += (a0.x + a1.x) + (a0.y + a1.y);
            return true;
        };
        // columns [lo, hi) of the queries that see key j (columns are in token order)
        auto columns = [&](const SeqInfo& s, int j, int q0, int cols, int& lo, int& hi) {
            lo = 0;
            hi = cols;
            if (p.causal) {
                lo = max(0, j - s.P - q0) * G;
                // (clamped to a tile's tokens: a window times G may pass 32 bits)
                if (p.window > 0 && j >= p.sinks)
                    hi = min(hi, max(0, min(p.window + (j - s.P - q0), kBlockM)) * G);
            }
        };
        // key j's weight row, old weight and score factor; false: the row holds no key
        auto fetch = [&](const Unit& u, const SeqGeo& g, const KeyTile& k, size_t& row, float& old, float& mul) -> bool {
            const int j = k.kb + r;
            old = 0.f;
            mul = p.scale_log2;
            if (j < k.lo || j >= k.hi) return false;
            row = weight_row(u, j);
            if (k.jt < g.np) {
                old = p.weights[row];
                if (kQuant) mul *= __ldg(p.scale_k + row);
            }
            return true;
        };
        UnitSlot us;
        for (int u_it = 0; ok && next_unit(u_it, us); ++u_it) {
            const SeqInfo s = us.s;
            const Unit u = us.u;
            const SeqGeo g = geo(s);
            uint32_t par;
            if (kQuant) ring.unit();
            if (g.nq == 1) {
                // every fourth tile is this group's; its next tile's weights are
                // fetched one tile ahead
                if (kQuant) ring.next(true, par);
                if (!warp_wait(&ctl->l_full[lst], lpar, ctl, hdr)) break;
                const float* nl = ctl->neg_lse[lst];
                const int end = u.q0 + u.ntiles;
                int mine = u.q0 + (int)((group - nn) & 3);
                size_t row = 0, next_row = 0;
                float old = 0.f, next_old = 0.f, mul = 0.f, next_mul = 0.f;
                bool has = mine < end && fetch(u, g, key_tile_at<kPaged>(g, s, mine), row, old, mul), next_has = false;
                for (int x = u.q0; x < end; ++x, ++nn) {
                    const int kst = kQuant ? ring.next(false, par) : 0;
                    if (x != mine) continue;
                    mine += 4;
                    next_has = mine < end && fetch(u, g, key_tile_at<kPaged>(g, s, mine), next_row, next_old, next_mul);
                    const KeyTile k = key_tile_at<kPaged>(g, s, x);
                    if (kQuant && k.jt < g.np && !expand(kst, par)) { ok = false; break; }
                    int lo, hi;
                    columns(s, k.kb + r, 0, s.n * G, lo, hi);
                    float total = 0.f;
                    if (!add_tile(nl, s.n * G, false, lo, hi, mul, total)) { ok = false; break; }
                    if (has) p.weights[row] = old + total;
                    row = next_row;
                    has = next_has;
                    old = next_old;
                    mul = next_mul;
                }
                if (!ok) break;
                next_lse();
                continue;
            }
            const int nt = u.ntiles;
            const bool four = nt > 2;
            const int t = four ? group : group & 1, turn = group >> 1;  // this group's tile; its Q tiles' parity (if two)
            const bool here = t < nt;
            const QRange qr = queries(g, s, u);
            const KeyTile k = key_tile_at<kPaged>(g, s, u.q0 + (here ? t : 0));
            size_t row = 0;
            float old = 0.f, mul = 0.f, total = 0.f;
            const bool has = here && fetch(u, g, k, row, old, mul);
            if (kQuant) {
                for (int i = 0; i < nt; ++i) {
                    const int st = ring.next(true, par);
                    if (i == t && (four || turn == 0) && k.jt < g.np && !expand(st, par)) { ok = false; break; }
                }
            }
            const QRange mine = here ? seen_by(g, s, k) : QRange{0, 0};
            const QRange full = full_queries(k, s, tps, G, p.causal, p.window, p.sinks);
            for (int qi = qr.lo; qi < qr.hi && ok; ++qi) {
                if (kQuant) ring.next(false, par);
                ok = warp_wait(&ctl->l_full[lst], lpar, ctl, hdr);
                if (!ok) break;
                if (qi >= mine.lo && qi < mine.hi && (four || (qi & 1) == turn)) {
                    const int q0 = qi * tps, cols = min(tps, s.n - q0) * G;
                    int lo = 0, hi = 0;
                    const bool whole = qi >= full.lo && qi < full.hi;
                    if (!whole) columns(s, k.kb + r, q0, cols, lo, hi);
                    ok = add_tile(ctl->neg_lse[lst], cols, whole, lo, hi, mul, total);
                    if (!ok) break;
                }
                next_lse();
            }
            if (!ok) break;
            if (!four && here) {
                // the second group's sums join the first one's (bounded waits, both ways)
                if (turn) {
                    if (!warp_wait(&ctl->pair_empty[t], (npair & 1) ^ 1, ctl, hdr)) break;
                    ctl->pair[t][r] = total;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->pair_full[t]);
                } else {
                    if (!warp_wait(&ctl->pair_full[t], npair & 1, ctl, hdr)) break;
                    total += ctl->pair[t][r];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->pair_empty[t]);
                }
                ++npair;
            }
            if (has && (four || turn == 0)) p.weights[row] = old + total;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, bool kPaged, bool kQuant>
cudaError_t launch_d(const KeyWeightsParams& p, int grid, cudaStream_t st) {
    constexpr int kSmem = smem_bytes<D>();
    static_assert(kSmem <= 232448, "shared memory budget");
    static int configured_for[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !configured_for[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<D, kPaged, kQuant>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        configured_for[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, key_weights_kernel<D, kPaged, kQuant>, p);
}

template <int D>
cudaError_t launch_dim(const KeyWeightsParams& p, int grid, cudaStream_t st) {
    if (p.block_table) return p.kv_quant ? launch_d<D, true, true>(p, grid, st) : launch_d<D, true, false>(p, grid, st);
    return p.kv_quant ? launch_d<D, false, true>(p, grid, st) : launch_d<D, false, false>(p, grid, st);
}

}  // namespace

cudaError_t launch_build_key_schedule(const KeyScheduleArgs& a, cudaStream_t stream) {
    if (a.num_seqs <= kFewSeqs)
        build_key_schedule_few_kernel<<<1, kFewThreads, 0, stream>>>(a);
    else
        build_key_schedule_kernel<<<1, 1024, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_key_weights(const KeyWeightsParams& p, int head_dim, int grid, cudaStream_t stream) {
    switch (head_dim) {
        case 32: return launch_dim<32>(p, grid, stream);
        case 64: return launch_dim<64>(p, grid, stream);
        default: return launch_dim<128>(p, grid, stream);
    }
}

}  // namespace pa
