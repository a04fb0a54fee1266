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
// One persistent CTA per SM, 384 threads:
//   warp 0          fetches units, loads K tiles into a ring of four;
//   warp 1          tcgen05 issuer: per Q tile, S^T of both slots (two key tiles
//                   share every Q tile), two TMEM buffers per slot;
//   warp 2          loads Q tiles (rows = (token, head in group)) into a ring;
//   warp 3          stages -lse * log2(e) of the Q tile's rows;
//   warps 4-7, 8-11 slot 0 and slot 1: sum of exp2 over the columns, one key per
//                   thread; an int8 key tile is first expanded by its slot's
//                   warps (exact codes; the row scale multiplies the scores).
// A unit is a pair of key tiles against every Q tile that sees one of them; for
// a sequence whose queries fit one Q tile (decode rows) it is a longer run of
// key tiles, and the Q tile is loaded once.  Every wait is bounded in time, as
// in the attention kernel.
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
constexpr int kThreads = 384;
constexpr int kMaxRun = 8;   // key tiles of a unit of a one-Q-tile sequence, at most
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
    static constexpr int kStagesK = 4;
    static constexpr int kStagesQ = D == 128 ? 3 : 4;
};

struct UnitSlot {
    Unit u;  // q0: first tile (position in the sequence's stream), ntiles: key tiles
    SeqInfo s;
};

struct __align__(16) Ctrl {
    uint64_t k_full[4], k_empty[4], k_conv[4];
    uint64_t q_full[4], q_empty[4], l_full[4], l_empty[4];
    uint64_t s_full[2][2], s_empty[2][2];
    uint64_t mma_drain;
    uint64_t unit_full[2], unit_empty[2];
    UnitSlot slot[2];
    uint32_t tmem_base;
    int abort;
    alignas(16) float neg_lse[4][128];  // -lse * log2(e) of the Q tile's rows
};

template <int D>
constexpr int smem_bytes() {
    using C = Cfg<D>;
    constexpr int n = C::kTileBytes * (C::kStagesK + C::kStagesQ) + (int)sizeof(Ctrl);
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

// Barrier of one slot's four warps.
__device__ __forceinline__ void slot_sync(int slot) { asm volatile("bar.sync %0, 128;" ::"r"(slot + 1) : "memory"); }

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

// Whether some query of tokens [qs, qe) sees some key of the tile.
__device__ __forceinline__ bool tile_seen(const KeyTile& k, int P, int qs, int qe, int causal, int window, int sinks) {
    if (!causal) return true;
    if (P + qe - 1 < k.lo) return false;
    return window == 0 || P + qs - (k.hi - 1) < window || k.lo < sinks;
}

// Q tiles [lo, hi) that see a tile of the pair (k1.hi == 0: a pair of one).
struct QRange {
    int lo, hi;
};

__device__ __forceinline__ QRange pair_queries(const KeyTile& k0, const KeyTile& k1, bool two, const SeqInfo& s, int nq,
                                               int tps, int causal, int window, int sinks) {
    QRange r{0, nq};
    if (!causal) return r;
    if (k0.lo > s.P) r.lo = (k0.lo - s.P) / tps;
    if (window > 0 && k0.lo >= sinks) {
        const int last = window + (two ? k1.hi : k0.hi) - 2 - s.P;  // last token that sees the pair's last key
        r.hi = last < 0 ? 0 : min(nq, last / tps + 1);
    }
    return r;
}

// Key tiles of a unit of a sequence whose queries fit one Q tile: about eight
// units per CTA of the `total` tiles of all of them.
__device__ __forceinline__ int run_length(unsigned long long total, int num_ctas) {
    const unsigned long long per = total / (8u * (unsigned)num_ctas);
    return per >= kMaxRun ? kMaxRun : (per < 2 ? 2 : (int)per & ~1);
}

// Writes unit x of sequence b and KV head kvh (its tiles in units of len).  A
// sequence's units: its KV heads in groups whose queries fit the L2 budget, and
// within a group the first keys first (under a causal mask the most expensive
// ones) with the group's heads adjacent.
__device__ __forceinline__ void emit_keys(const KeyScheduleArgs& a, const SeqInfo& si, int b, int x, int kvh, int tiles,
                                          int len, int units, int first) {
    const float head_bytes = (float)si.n * a.group * a.head_dim * 2;
    const float fit = floorf((float)kL2GroupBytes / fmaxf(head_bytes, 1.f));
    const int hg = fit >= (float)a.n_kv_heads ? a.n_kv_heads : (fit < 1.f ? 1 : (int)fit);
    const int g0 = kvh - kvh % hg, gsize = min(hg, a.n_kv_heads - g0);
    const int pos = first + g0 * units + x * gsize + (kvh - g0);
    if (pos < a.max_units) a.units[pos] = Unit{b, kvh, x * len, min(len, tiles - x * len)};
}

__global__ void __launch_bounds__(1024) build_key_schedule_kernel(const __grid_constant__ KeyScheduleArgs a) {
    __shared__ int hist[kCostBins];
    __shared__ int warp_sums[32];
    __shared__ unsigned long long s_total;
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
    if (tid == 0) s_total = 0;
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
            if (g.nq == 1) atomicAdd(&s_total, (unsigned long long)g.tiles * a.n_kv_heads);
        }
    }
    __threadfence_block();
    __syncthreads();
    const int run = run_length(s_total, a.num_ctas);
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
            const int len = g.nq == 1 ? run : 2;
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
        emit_keys(a, si, b, i - si.pad, kvh, g.tiles, g.nq == 1 ? run : 2, seq_units[b], seq_first[b]);
    }
}

// The same for a few sequences (kFewSeqs): see schedule.cuh.
__global__ void __launch_bounds__(kFewThreads) build_key_schedule_few_kernel(const __grid_constant__ KeyScheduleArgs a) {
    __shared__ FewSeqs f;
    __shared__ int s_tiles[kFewSeqs], s_len[kFewSeqs];
    const int tid = threadIdx.x, tps = kBlockM / a.group;
    const bool paged = a.block_table != nullptr;
    griddep_launch();
    load_few(a, f, a.sinks, nullptr, 0);
    SeqGeo g{};
    if (tid < a.num_seqs && f.seqs[tid].n > 0) {
        g = seq_geo(f.seqs[tid], tps, a.causal, a.window, a.sinks, paged);
        if (g.nq == 1) atomicAdd(&f.total, (unsigned long long)g.tiles * a.n_kv_heads);
    }
    __syncthreads();
    if (tid < a.num_seqs) {
        const int len = g.nq == 1 ? run_length(f.total, a.num_ctas) : 2;
        s_tiles[tid] = g.tiles;
        s_len[tid] = len;
        f.blocks[tid] = f.units[tid] = (g.tiles + len - 1) / len;
        f.cost[tid] = (float)g.tiles * (float)g.nq;
    }
    __syncthreads();
    const int blocks = rank_few(a, f, a.num_seqs);
    for (int w = tid; w < blocks * a.n_kv_heads; w += kFewThreads) {
        const int i = w / a.n_kv_heads, kvh = w % a.n_kv_heads;
        const int b = block_owner(f.seqs, a.num_seqs, i);
        emit_keys(a, f.seqs[b], b, i - f.seqs[b].pad, kvh, s_tiles[b], s_len[b], f.units[b], f.first[b]);
    }
}

template <int D, bool kPaged, bool kQuant>
__global__ void __launch_bounds__(kThreads, 1) key_weights_kernel(const __grid_constant__ KeyWeightsParams p) {
    using C = Cfg<D>;
    constexpr bool kGrp = kPaged && !kQuant && C::kChunks == 2;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const bool misaligned = (smem_u32(smem_raw) & 1023u) != 0;
    uint8_t* k_smem = smem_raw;
    uint8_t* q_smem = k_smem + C::kStagesK * C::kTileBytes;
    Ctrl* ctl = reinterpret_cast<Ctrl*>(q_smem + C::kStagesQ * C::kTileBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    WorkspaceHeader* hdr = p.hdr;
    const int G = p.group, tps = kBlockM / G;

    if (!misaligned && threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&ctl->k_full[i], 1);
            mbar_init(&ctl->k_empty[i], 1);  // MMA commit
            mbar_init(&ctl->k_conv[i], 4);   // the slot's four warps
            mbar_init(&ctl->q_full[i], 1);
            mbar_init(&ctl->q_empty[i], 1);  // MMA commit
            mbar_init(&ctl->l_full[i], 1);
            mbar_init(&ctl->l_empty[i], 8);  // the sum warps
        }
        for (int s = 0; s < 2; ++s)
            for (int i = 0; i < 2; ++i) {
                mbar_init(&ctl->s_full[s][i], 1);
                mbar_init(&ctl->s_empty[s][i], 4);
            }
        mbar_init(&ctl->mma_drain, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->unit_full[i], 1);
            mbar_init(&ctl->unit_empty[i], 11);  // every warp but the fetching one
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
    // Q rows [tps * G, 128) belong to no token and no copy fills them
    if (!misaligned && tps * G < kBlockM) {
        for (int i = threadIdx.x; i < C::kStagesQ * C::kTileBytes / 16; i += kThreads)
            reinterpret_cast<uint4*>(q_smem)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
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
    auto geo = [&](const SeqInfo& s) { return seq_geo(s, tps, p.causal, p.window, p.sinks, kPaged); };

    if (warp == 0) {
        // ------------------------------------------------- unit fetch, K tiles
        uint32_t t = 0, lp_set = 0, lp_par = 0;
        bool short_units = true;
        for (int u_it = 0;; ++u_it) {
            const int sl = u_it & 1;
            if (!warp_wait(&ctl->unit_empty[sl], ((u_it >> 1) & 1) ^ 1, ctl, hdr)) break;
            // claim late: only when the ring has room for the unit's first tile,
            // so that the longest-first list still evens out the CTAs at its end
            // (not for decode rows, whose units are short and alike: there the
            // claim's latency would show)
            if (!short_units && !warp_wait(&ctl->k_empty[t % C::kStagesK], ((t / C::kStagesK) & 1) ^ 1, ctl, hdr)) break;
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
            short_units = g.nq == 1;
            bool ok = true;
            for (int x = u.q0; x < u.q0 + u.ntiles; ++x, ++t) {
                const KeyTile k = key_tile_at<kPaged>(g, s, x);
                const int st = t % C::kStagesK;
                const uint32_t ph = (t / C::kStagesK) & 1;
                uint8_t* stage = k_smem + st * C::kTileBytes;
                const bool pre = k.jt < g.np;
                // paged prefix tile: this lane's block, fetched before the wait
                const int br = p.box_rows;
                const int boxes = kPaged && pre ? (k.hi - k.kb + br - 1) / br : 0;
                int blk = 0;
                if (kPaged && lane < boxes)
                    blk = __ldg(p.block_table + (size_t)u.b * p.max_blocks + ((k.kb + lane * br) >> p.block_log2));
                if (!warp_wait(&ctl->k_empty[st], ph ^ 1, ctl, hdr)) {
                    ok = false;
                    break;
                }
                uint32_t bytes = C::kTileBytes;
                if (pre && kPaged) bytes = boxes * br * (kQuant ? D : C::kRowBytes * C::kChunks);
                else if (pre && kQuant) bytes = kBlockN * D;
                if (lane == 0) mbar_arrive_expect_tx(&ctl->k_full[st], bytes);
                __syncwarp();
                if (!pre) {
                    if (lane < C::kChunks)
                        tma_load_3d(stage + lane * C::kChunkBytes, &p.tm_k, &ctl->k_full[st], lane * C::kChunkCols, u.kvh,
                                    s.q_start + k.kb - s.P);
                } else if (kPaged) {
                    if (lane < boxes) {
                        const int row = (k.kb + lane * br) & ((1 << p.block_log2) - 1), z = blk * p.n_kv_heads + u.kvh;
                        if constexpr (kQuant) {
                            tma_load_3d(stage + C::kTileBytes / 2 + lane * br * D, &p.tm_ck, &ctl->k_full[st], 0, row, z);
                        } else if constexpr (kGrp) {
                            tma_load_5d(stage + lane * br * C::kRowBytes * C::kChunks, &p.tm_ck, &ctl->k_full[st], 0, 0, 0,
                                        row >> 3, z);
                        } else {
                            tma_load_3d(stage + lane * br * C::kRowBytes, &p.tm_ck, &ctl->k_full[st], 0, row, z);
                        }
                    }
                } else {
                    const int z = u.b * p.n_kv_heads + u.kvh;
                    if constexpr (kQuant) {
                        if (lane == 0) tma_load_3d(stage + C::kTileBytes / 2, &p.tm_ck, &ctl->k_full[st], 0, k.kb, z);
                    } else if (lane < C::kChunks) {
                        tma_load_3d(stage + lane * C::kChunkBytes, &p.tm_ck, &ctl->k_full[st], lane * C::kChunkCols, k.kb, z);
                    }
                }
                __syncwarp();
                lp_set |= 1u << st;
                lp_par = (lp_par & ~(1u << st)) | (ph << st);
            }
            if (!ok) break;
        }
        if (lane == 0 && aborted(ctl)) drain(ctl->k_full, lp_set, lp_par, C::kStagesK);
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint32_t k_addr = smem_u32(k_smem), q_addr = smem_u32(q_smem);
        const uint64_t k_desc = smem_desc(k_addr, 16, C::kSbo, C::kSw);
        const uint64_t k_desc_g = smem_desc(k_addr, 16, C::kGrpSbo, C::kSw);
        const uint64_t q_desc = smem_desc(q_addr, 16, C::kSbo, C::kSw);
        uint32_t t = 0, lq = 0;       // K tiles and Q tiles consumed so far
        uint32_t ns[2] = {0, 0};      // S^T tiles issued per slot
        uint32_t cpar = 0;            // parity of k_conv per stage
        bool ok = true;
        UnitSlot us;
        for (int u_it = 0; ok && next_unit(u_it, us); ++u_it) {
            const SeqInfo s = us.s;
            const SeqGeo g = geo(s);
            const bool single = g.nq == 1;
            if (single && !warp_wait(&ctl->q_full[lq % C::kStagesQ], (lq / C::kStagesQ) & 1, ctl, hdr)) break;
            for (int x = us.u.q0; x < us.u.q0 + us.u.ntiles && ok; x += 2) {
                const bool two = x + 1 < us.u.q0 + us.u.ntiles;
                const KeyTile kt[2] = {key_tile_at<kPaged>(g, s, x), key_tile_at<kPaged>(g, s, two ? x + 1 : x)};
                const QRange qr = single ? QRange{0, 1}
                                         : pair_queries(kt[0], kt[1], two, s, g.nq, tps, p.causal, p.window, p.sinks);
                bool ready[2] = {false, false};
                auto wait_k = [&](int i) -> bool {
                    const int st = (t + i) % C::kStagesK;
                    if (kQuant && kt[i].jt < g.np) {
                        const bool got = warp_wait(&ctl->k_conv[st], (cpar >> st) & 1, ctl, hdr);
                        cpar ^= 1u << st;
                        return got;
                    }
                    return warp_wait(&ctl->k_full[st], ((t + i) / C::kStagesK) & 1, ctl, hdr);
                };
                for (int qi = qr.lo; qi < qr.hi && ok; ++qi) {
                    const int qst = lq % C::kStagesQ;
                    const int q0 = qi * tps, qe = min(q0 + tps, s.n);
                    if (!single && !warp_wait(&ctl->q_full[qst], (lq / C::kStagesQ) & 1, ctl, hdr)) { ok = false; break; }
                    // columns in use, rounded up to what an M = 128 MMA takes
                    const uint32_t n16 = (uint32_t)((qe - q0) * G + 15) / 16;
                    const uint32_t idesc = (idesc_bf16_f32(kBlockM, 0, 0, 0)) | (n16 * 2 << 17);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i == 1 && !two) continue;
                        if (!tile_seen(kt[i], s.P, q0, qe, p.causal, p.window, p.sinks)) continue;
                        if (!ready[i]) {
                            if (!wait_k(i)) { ok = false; break; }
                            ready[i] = true;
                        }
                        const int buf = ns[i] & 1;
                        if (!warp_wait(&ctl->s_empty[i][buf], ((ns[i] >> 1) & 1) ^ 1, ctl, hdr)) { ok = false; break; }
                        tc_fence_after();
                        if (leader) {
                            const uint32_t koff = ((t + i) % C::kStagesK) * C::kTileBytes, qoff = qst * C::kTileBytes;
                            const bool grp = kGrp && kt[i].jt < g.np;
                            const uint64_t kd = grp ? k_desc_g : k_desc;
                            const uint32_t kcs = grp ? C::kSbo : C::kChunkBytes;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t ch = (kk * 16) / C::kChunkCols, in = ((kk * 16) % C::kChunkCols) * 2;
                                mma_ss(tmem + (i * 2 + buf) * 128, kd + ((koff + ch * kcs + in) >> 4),
                                       q_desc + ((qoff + ch * C::kChunkBytes + in) >> 4), idesc, kk > 0 ? 1u : 0u);
                            }
                            mma_commit(&ctl->s_full[i][buf]);
                        }
                        __syncwarp();
                        ++ns[i];
                    }
                    if (!ok) break;
                    if (!single) {
                        if (leader) mma_commit(&ctl->q_empty[qst]);
                        __syncwarp();
                        ++lq;
                    }
                }
                if (!ok) break;
                // a tile no query saw was still loaded (and expanded): take its turn
                for (int i = 0; i < (two ? 2 : 1) && ok; ++i) {
                    if (!ready[i]) ok = wait_k(i);
                    if (ok && leader) mma_commit(&ctl->k_empty[(t + i) % C::kStagesK]);
                    __syncwarp();
                }
                t += two ? 2 : 1;
            }
            if (!ok) break;
            if (single) {
                if (leader) mma_commit(&ctl->q_empty[lq % C::kStagesQ]);
                __syncwarp();
                ++lq;
            }
        }
        // every MMA this warp issued has finished before TMEM is released
        if (leader) {
            mma_commit(&ctl->mma_drain);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&ctl->mma_drain, 0) && globaltimer_ns() - t0 < kTimeoutNs) {
            }
        }
        __syncwarp();
    } else if (warp == 2 || warp == 3) {
        // ------------------------------- Q tiles (warp 2) and their lse (warp 3)
        uint32_t lq = 0, lp_set = 0, lp_par = 0;
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
            const bool single = g.nq == 1;
            const bool two = us.u.ntiles > 1;
            QRange qr{0, 1};
            if (!single)
                qr = pair_queries(key_tile_at<kPaged>(g, s, us.u.q0),
                                  key_tile_at<kPaged>(g, s, us.u.q0 + (two ? 1 : 0)), two, s, g.nq, tps, p.causal,
                                  p.window, p.sinks);
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
            if (warp == 3 && qr.lo < qr.hi) load_lse(qr.lo);
            for (int qi = qr.lo; qi < qr.hi; ++qi, ++lq) {
                const int st = lq % C::kStagesQ;
                const uint32_t ph = (lq / C::kStagesQ) & 1;
                const int q0 = qi * tps;
                if (warp == 2) {
                    if (!warp_wait(&ctl->q_empty[st], ph ^ 1, ctl, hdr)) { ok = false; break; }
                    // a decode row's Q tile is one token's heads: the rest of the
                    // stage keeps what it held, in columns that no sum takes
                    const bool one = s.n == 1;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&ctl->q_full[st], G * (one ? 1 : tps) * C::kRowBytes * C::kChunks);
                    __syncwarp();
                    if (lane < C::kChunks)
                        tma_load_3d(q_smem + st * C::kTileBytes + lane * C::kChunkBytes, one ? &p.tm_q1 : &p.tm_q, &ctl->q_full[st],
                                    lane * C::kChunkCols, us.u.kvh * G, s.q_start + q0);
                    __syncwarp();
                    lp_set |= 1u << st;
                    lp_par = (lp_par & ~(1u << st)) | (ph << st);
                } else {
                    if (!warp_wait(&ctl->l_empty[st], ph ^ 1, ctl, hdr)) { ok = false; break; }
#pragma unroll
                    for (int i = 0; i < 4; ++i) ctl->neg_lse[st][lane + 32 * i] = l[i];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->l_full[st]);
                    if (qi + 1 < qr.hi) load_lse(qi + 1);  // on its way during the next wait
                }
            }
        }
        if (warp == 2 && lane == 0 && aborted(ctl)) drain(ctl->q_full, lp_set, lp_par, C::kStagesQ);
    } else {
        // ------------------------------------------------------------ the sums
        const int slot = (warp - 4) >> 2, sp = warp & 3;
        const int r = sp * 32 + lane;  // row of the key tile == TMEM lane
        const uint32_t lane_off = (uint32_t)(sp * 32) << 16;
        uint32_t t = 0, lq = 0, ns = 0;
        bool ok = true;
        UnitSlot us;
        for (int u_it = 0; ok && next_unit(u_it, us); ++u_it) {
            const SeqInfo s = us.s;
            const SeqGeo g = geo(s);
            const bool single = g.nq == 1;
            if (single && !warp_wait(&ctl->l_full[lq % C::kStagesQ], (lq / C::kStagesQ) & 1, ctl, hdr)) break;
            for (int x = us.u.q0; x < us.u.q0 + us.u.ntiles && ok; x += 2) {
                const bool two = x + 1 < us.u.q0 + us.u.ntiles;
                const bool mine = slot == 0 || two;
                const KeyTile k0 = key_tile_at<kPaged>(g, s, x), k1 = key_tile_at<kPaged>(g, s, two ? x + 1 : x);
                const KeyTile k = slot ? k1 : k0;
                const QRange qr =
                    single ? QRange{0, 1} : pair_queries(k0, k1, two, s, g.nq, tps, p.causal, p.window, p.sinks);
                // this thread's key: its weight's row, its old weight
                const int j = k.kb + r;
                const bool has = mine && j >= k.lo && j < k.hi;
                const bool pre = k.jt < g.np;
                float* w = nullptr;
                float old = 0.f, mul = p.scale_log2;
                if (has) {
                    size_t row;
                    if (kPaged) {
                        const int blk = __ldg(p.block_table + (size_t)us.u.b * p.max_blocks + (j >> p.block_log2));
                        row = (((size_t)blk * p.n_kv_heads + us.u.kvh) << p.block_log2) + (j & ((1 << p.block_log2) - 1));
                    } else {
                        row = ((size_t)us.u.b * p.n_kv_heads + us.u.kvh) * p.max_cache_len + j;
                    }
                    w = p.weights + row;
                    if (pre) old = *w;
                    if (kQuant && pre) mul *= __ldg(p.scale_k + row);
                }
                if (kQuant && mine && pre) {
                    // expand the codes (upper half of the stage) into the swizzled
                    // bf16 tile: all of them are read before any is overwritten
                    const int st = (t + slot) % C::kStagesK;
                    uint8_t* stage = k_smem + st * C::kTileBytes;
                    if (!warp_wait(&ctl->k_full[st], ((t + slot) / C::kStagesK) & 1, ctl, hdr)) { ok = false; break; }
                    constexpr int kPieces = 128 * D / 8 / 128;  // 8 codes each, per thread
                    const int i0 = sp * 32 + lane;
                    uint2 c[kPieces];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        c[i] = *reinterpret_cast<const uint2*>(stage + C::kTileBytes / 2 + (i0 + 128 * i) * 8);
                    slot_sync(slot);
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int idx = i0 + 128 * i, row = idx / (D / 8), gr = idx % (D / 8);
                        const int ch = gr / (C::kChunkCols / 8), gg = gr % (C::kChunkCols / 8);
                        const int phys = D >= 64 ? (gg ^ (row & 7)) : (gg ^ ((row >> 1) & 3));
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t wd = e < 2 ? c[i].x : c[i].y;
                            const int sh = (e & 1) * 16;
                            const __nv_bfloat162 v =
                                __floats2bfloat162_rn((float)(int8_t)(wd >> sh), (float)(int8_t)(wd >> (sh + 8)));
                            o[e] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        *reinterpret_cast<uint4*>(stage + ch * C::kChunkBytes + row * C::kRowBytes + phys * 16) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->k_conv[st]);
                }
                const float2 mul2 = make_float2(mul, mul);
                float total = 0.f;
                for (int qi = qr.lo; qi < qr.hi; ++qi) {
                    const int qst = lq % C::kStagesQ;
                    const int q0 = qi * tps, qe = min(q0 + tps, s.n);
                    if (!single && !warp_wait(&ctl->l_full[qst], (lq / C::kStagesQ) & 1, ctl, hdr)) { ok = false; break; }
                    if (mine && tile_seen(k, s.P, q0, qe, p.causal, p.window, p.sinks)) {
                        const int buf = ns & 1;
                        if (!warp_wait(&ctl->s_full[slot][buf], (ns >> 1) & 1, ctl, hdr)) { ok = false; break; }
                        tc_fence_after();
                        const int cols = (qe - q0) * G;
                        // columns [clo, chi) of this key's queries (columns are in token order)
                        int clo = 0, chi = cols;
                        if (p.causal) {
                            clo = max(0, j - s.P - q0) * G;
                            if (p.window > 0 && j >= p.sinks) chi = min(chi, (p.window + j - s.P - q0) * G);
                        }
                        const bool whole = __all_sync(0xffffffffu, cols == kBlockN && (!has || (clo == 0 && chi == cols)));
                        const uint32_t col = tmem + lane_off + (slot * 2 + buf) * 128;
                        const float4* nl = reinterpret_cast<const float4*>(ctl->neg_lse[qst]);
                        float2 a0 = make_float2(0.f, 0.f), a1 = a0;
                        if (whole) {
                            // 32 columns are summed while the next 32 are on their way
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
                                    if (lane == 0) mbar_arrive(&ctl->s_empty[slot][buf]);
                                }
#pragma unroll
                                for (int e = 0; e < 32; e += 4) {
                                    const float4 l = nl[(c + e) / 4];
                                    const float2 s0 =
                                        __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), mul2,
                                                   make_float2(l.x, l.y));
                                    const float2 s1 =
                                        __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), mul2,
                                                   make_float2(l.z, l.w));
                                    a0 = __fadd2_rn(a0, make_float2(ex2(s0.x), ex2(s0.y)));
                                    a1 = __fadd2_rn(a1, make_float2(ex2(s1.x), ex2(s1.y)));
                                }
                            }
                        } else {
                            for (int c = 0; c < cols; c += 32) {
                                uint32_t v[32];
                                tmem_ld32(col + c, v);
                                tmem_wait_ld();
                                reg_fence(v);
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 l = reinterpret_cast<const float2*>(nl)[(c + e) / 2];
                                    const float x0 = ex2(fmaf(__uint_as_float(v[e]), mul, l.x));
                                    const float x1 = ex2(fmaf(__uint_as_float(v[e + 1]), mul, l.y));
                                    a0.x += c + e >= clo && c + e < chi ? x0 : 0.f;
                                    a0.y += c + e + 1 >= clo && c + e + 1 < chi ? x1 : 0.f;
                                }
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&ctl->s_empty[slot][buf]);
                        }
                        total += (a0.x + a1.x) + (a0.y + a1.y);
                        ++ns;
                    }
                    if (!single) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->l_empty[qst]);
                        ++lq;
                    }
                }
                if (!ok) break;
                if (has) *w = old + total;
                t += two ? 2 : 1;
            }
            if (!ok) break;
            if (single) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->l_empty[lq % C::kStagesQ]);
                ++lq;
            }
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
