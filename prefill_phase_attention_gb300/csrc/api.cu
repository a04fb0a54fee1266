// api.cu -- the C ABI (include/prefill_attn.h): argument checks, the
// per-(device, stream) schedule workspace, and the launch sequence.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <algorithm>
#include <exception>
#include <map>
#include <memory>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "common.cuh"
#include "kernels.h"
#include "prefill_attn.h"

namespace {

thread_local char g_last_error[512];
thread_local int g_last_launches = 0;
thread_local int g_last_schedule = 0;

pa_status fail(pa_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return s;
}

pa_status cuda_fail(cudaError_t e, const char* what) {
    return fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The status of the exception being handled.  Every C entry ends with it: an
// exception that left one would end the caller's process.
pa_status caught() noexcept {
    try {
        throw;
    } catch (const std::bad_alloc&) {
        return fail(PA_ERR_CUDA, "out of host memory");
    } catch (const std::exception& e) {
        return fail(PA_ERR_CUDA, "%s", e.what());
    } catch (...) {
        return fail(PA_ERR_CUDA, "unknown exception");
    }
}

struct Workspace {
    std::shared_ptr<std::mutex> mu;  // see StreamLock
    void* ptr = nullptr;
    size_t bytes = 0;
    int max_units = 0;
    int max_seqs = 0;
    void* rope = nullptr;  // rotated q/k copies (grown on demand)
    size_t rope_bytes = 0;
    void* aux = nullptr;   // lists and partial results of the long-context calls (grown on demand)
    size_t aux_bytes = 0;
    bool captured = false;  // a captured graph holds these addresses: outgrown blocks are kept, not freed
    std::vector<void*> old_headers;  // headers of outgrown blocks that a graph may still write errors to
    std::vector<void*> retired;      // outgrown blocks that a captured graph holds
};

std::mutex g_mu;
std::map<std::pair<int, cudaStream_t>, Workspace> g_ws;

// A stream's workspace and its lock, held by a call from its first look at the
// workspace to its last launch.  A call's kernels hand data to one another through
// that workspace, and a call may replace its blocks: two host threads that call on
// one stream must not mix their launches.  (g_mu is for the map; the lock outlives a
// release of the workspace.)
struct StreamLock {
    Workspace* ws;
    std::shared_ptr<std::mutex> mu;
    std::unique_lock<std::mutex> held;
    StreamLock(int dev, cudaStream_t st) : ws(of(dev, st)), mu(ws->mu), held(*mu) {}

    static Workspace* of(int dev, cudaStream_t st) {
        std::lock_guard<std::mutex> lock(g_mu);
        Workspace& w = g_ws[std::make_pair(dev, st)];  // (stays where it is)
        if (!w.mu) w.mu = std::make_shared<std::mutex>();
        return &w;
    }
};

// Room in `retired` for one more block, made before the block that replaces it is
// allocated: nothing throws in between.
void prepare_drop(Workspace& w) {
    if (w.captured) w.retired.reserve(w.retired.size() + 1);
}

// Gives up a block of a workspace that has been replaced by a larger one.
void drop_block(Workspace& w, void* ptr, cudaStream_t st) {
    if (!ptr) return;
    if (w.captured)
        w.retired.push_back(ptr);
    else
        cudaFreeAsync(ptr, st);
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// header | SeqInfo[max_seqs] | Unit[max_units] | int[2][max_seqs] (scheduler scratch)
size_t ws_bytes(int max_seqs, int max_units) {
    return align_up(sizeof(pa::WorkspaceHeader), 16) + (size_t)max_seqs * sizeof(pa::SeqInfo) +
           (size_t)max_units * sizeof(pa::Unit) + 2 * (size_t)max_seqs * sizeof(int);
}

pa::SeqInfo* ws_seqs(const Workspace& w) {
    return reinterpret_cast<pa::SeqInfo*>(static_cast<char*>(w.ptr) + align_up(sizeof(pa::WorkspaceHeader), 16));
}

pa::Unit* ws_units(const Workspace& w) { return reinterpret_cast<pa::Unit*>(ws_seqs(w) + w.max_seqs); }

int* ws_seq_scratch(const Workspace& w) { return reinterpret_cast<int*>(ws_units(w) + w.max_units); }

// True while `st` is being captured into a CUDA graph.
bool capturing(cudaStream_t st) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    return cudaStreamIsCapturing(st, &cs) == cudaSuccess && cs == cudaStreamCaptureStatusActive;
}

// Allocates (stream-ordered) a block of at least `need` bytes in place of one of
// `old`.  Where that one stays for a captured graph, the new one is at least twice
// its size (if there is room), so that all blocks which stay together are smaller
// than the newest.
cudaError_t alloc_block(const Workspace& w, size_t old, size_t need, cudaStream_t st, void** ptr, size_t* bytes) {
    *bytes = w.captured ? std::max(need, 2 * old) : need;
    cudaError_t e = cudaMallocAsync(ptr, *bytes, st);
    if (e == cudaErrorMemoryAllocation && *bytes > need) {
        cudaGetLastError();
        *bytes = need;
        e = cudaMallocAsync(ptr, need, st);
    }
    return e;
}

// Grows the workspace of a stream (stream-ordered) when needed; its lock is held, as
// in the next two.  Under graph capture nothing is allocated: the stream must already
// hold a workspace big enough (from a call outside the capture).
pa_status grow_workspace(Workspace& w, cudaStream_t st, int num_seqs, int max_units) {
    if (w.ptr && w.max_seqs >= num_seqs && w.max_units >= max_units) {
        if (!w.captured && capturing(st)) w.captured = true;
        return PA_OK;
    }
    if (capturing(st))
        return fail(PA_ERR_UNSUPPORTED,
                    "graph capture: the stream's workspace would have to grow (%d sequences, %d work units); "
                    "run a call of at least these sizes on this stream before capturing",
                    num_seqs, max_units);
    const int seqs = std::max(num_seqs, std::max(w.max_seqs, 64));
    int units = std::max(max_units, std::max(w.max_units, 4096));
    size_t bytes = 0;
    prepare_drop(w);
    if (w.captured) w.old_headers.reserve(w.old_headers.size() + 1);
    void* ptr = nullptr;
    cudaError_t e = alloc_block(w, w.bytes, ws_bytes(seqs, units), st, &ptr, &bytes);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMallocAsync(workspace)");
    // what is left of a larger block is room for units
    units = (int)std::min<size_t>(INT_MAX, units + (bytes - ws_bytes(seqs, units)) / sizeof(pa::Unit));
    e = cudaMemsetAsync(ptr, 0, sizeof(pa::WorkspaceHeader), st);
    if (e == cudaSuccess && w.ptr)  // keep sticky error bits across a regrow
        e = cudaMemcpyAsync(ptr, w.ptr, sizeof(int), cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) {
        cudaFreeAsync(ptr, st);
        return cuda_fail(e, "workspace init");
    }
    if (w.captured && w.ptr) w.old_headers.push_back(w.ptr);
    drop_block(w, w.ptr, st);
    w.ptr = ptr;
    w.bytes = bytes;
    w.max_seqs = seqs;
    w.max_units = units;
    return PA_OK;
}

// Grows (stream-ordered) the rotated-q/k scratch of a workspace to `bytes`.
pa_status get_rope_scratch(Workspace* w, cudaStream_t st, size_t bytes, void** out) {
    if (w->rope_bytes < bytes && capturing(st))
        return fail(PA_ERR_UNSUPPORTED,
                    "graph capture: the stream's rotary scratch would have to grow (%zu bytes); run a call with "
                    "rope_theta of at least these sizes on this stream before capturing",
                    bytes);
    if (w->rope_bytes < bytes) {
        prepare_drop(*w);
        void* nptr = nullptr;
        cudaError_t e = alloc_block(*w, w->rope_bytes, bytes, st, &nptr, &bytes);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMallocAsync(rotary scratch)");
        drop_block(*w, w->rope, st);
        w->rope = nptr;
        w->rope_bytes = bytes;
    }
    *out = w->rope;
    return PA_OK;
}

// Grows (stream-ordered) the auxiliary scratch of a workspace to `bytes`.
pa_status get_aux_scratch(Workspace* w, cudaStream_t st, size_t bytes, void** out) {
    if (w->aux_bytes < bytes && capturing(st))
        return fail(PA_ERR_UNSUPPORTED,
                    "graph capture: the stream's auxiliary scratch would have to grow (%zu bytes); run a call of at "
                    "least these sizes on this stream before capturing",
                    bytes);
    if (w->aux_bytes < bytes) {
        prepare_drop(*w);
        void* nptr = nullptr;
        cudaError_t e = alloc_block(*w, w->aux_bytes, bytes, st, &nptr, &bytes);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMallocAsync(auxiliary scratch)");
        drop_block(*w, w->aux, st);
        w->aux = nptr;
        w->aux_bytes = bytes;
    }
    *out = w->aux;
    return PA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pa_status check_args(const void* q, const void* k, const void* v, const int32_t* cu_q, const int32_t* cu_k,
                     const void* cache_k, const void* cache_v, const int32_t* off, const void* out,
                     const float* lse, int num_seqs, int total_q, int max_cache_len, int n_heads,
                     int n_kv_heads, int head_dim, float scale, int causal, bool paged = false) {
    if (num_seqs < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs must be >= 0 (got %d)", num_seqs);
    if (total_q < 0) return fail(PA_ERR_INVALID_ARG, "total_q must be >= 0 (got %d)", total_q);
    if (max_cache_len < 1) return fail(PA_ERR_INVALID_ARG, "max_cache_len must be >= 1 (got %d)", max_cache_len);
    if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARG, "n_heads (%d) must be a positive multiple of n_kv_heads (%d)", n_heads,
                    n_kv_heads);
    if (n_heads / n_kv_heads > pa::kBlockM)
        return fail(PA_ERR_UNSUPPORTED, "n_heads / n_kv_heads = %d exceeds %d", n_heads / n_kv_heads, pa::kBlockM);
    if (head_dim != 32 && head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim must be 32, 64 or 128 (got %d)", head_dim);
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(PA_ERR_INVALID_ARG, "scale must be finite and > 0 (got %g)", (double)scale);
    if (causal != 0 && causal != 1) return fail(PA_ERR_INVALID_ARG, "causal must be 0 or 1 (got %d)", causal);
    if (num_seqs == 0 || total_q == 0) return PA_OK;  // nothing is read or written
    const void* ptrs[] = {q, k, v, cu_q, cu_k, cache_k, cache_v, off, out};
    const char* names[] = {"q", "k", "v", "cu_seqlens_q", "cu_seqlens_k", "cache_k", "cache_v", "cache_offsets", "out"};
    for (int i = 0; i < 9; ++i) {
        if (!ptrs[i]) return fail(PA_ERR_INVALID_ARG, "%s is NULL", names[i]);
        if (i != 3 && i != 4 && i != 7 && !aligned16(ptrs[i]))
            return fail(PA_ERR_INVALID_ARG, "%s must be 16-byte aligned", names[i]);
    }
    if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k) | reinterpret_cast<uintptr_t>(off)) & 3u)
        return fail(PA_ERR_INVALID_ARG, "metadata arrays must be 4-byte aligned");
    if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return fail(PA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
    if (out == q || out == k || out == v) return fail(PA_ERR_INVALID_ARG, "out must not alias q, k or v");
    if (cache_k == k || cache_k == v || cache_v == k || cache_v == v || cache_k == cache_v)
        return fail(PA_ERR_INVALID_ARG, "caches must be distinct and must not alias k or v");
    // Row counts used by 32-bit kernel index arithmetic.
    if ((long long)total_q * n_heads >= (1LL << 31))
        return fail(PA_ERR_UNSUPPORTED, "total_q * n_heads must be < 2^31");
    if (!paged && (long long)num_seqs * n_kv_heads * max_cache_len >= (1LL << 31))
        return fail(PA_ERR_UNSUPPORTED, "num_seqs * n_kv_heads * max_cache_len must be < 2^31");
    return PA_OK;
}

struct Options {
    int window = 0;
    const int32_t* block_table = nullptr;  // paged cache when set
    int block_size = 0, max_blocks = 0, num_blocks = 0;
    float rope_theta = 0.f;                // rotary embedding when > 0
    int kv_quant = 0;                      // 1: int8 cache with fp32 row scales
    float* scale_k = nullptr;
    float* scale_v = nullptr;
    int wait_timeout_test = 0;
    int schedule = 0;  // pa_options.schedule (0: chosen per call)
};

// Reads the caller's options; fields past the caller's struct_size count as zero.
pa_status read_options(const pa_options* opts, int causal, Options* o) {
    *o = Options();
    if (!opts) return PA_OK;
    const size_t have = opts->struct_size;
    if (have < offsetof(pa_options, window) + sizeof(int32_t))
        return fail(PA_ERR_INVALID_ARG, "pa_options.struct_size %u is too small", (unsigned)opts->struct_size);
    o->window = opts->window;
    if (o->window < 0) return fail(PA_ERR_INVALID_ARG, "window must be >= 0 (got %d)", o->window);
    if (o->window > 0 && causal != 1) return fail(PA_ERR_INVALID_ARG, "a sliding window needs causal = 1");
    if (have >= offsetof(pa_options, reserved) + sizeof(int32_t)) {
        if (opts->reserved != 0) return fail(PA_ERR_INVALID_ARG, "pa_options.reserved must be 0");
    }
    if (have >= offsetof(pa_options, num_blocks) + sizeof(int32_t) && opts->block_table) {
        o->block_table = opts->block_table;
        o->block_size = opts->block_size;
        o->max_blocks = opts->max_blocks_per_seq;
        o->num_blocks = opts->num_blocks;
        const int bs = o->block_size;
        if (bs < 8 || bs > 4096 || (bs & (bs - 1)) != 0)
            return fail(PA_ERR_UNSUPPORTED, "block_size must be a power of two in [8, 4096] (got %d)", bs);
        if (o->max_blocks < 1 || o->num_blocks < 1)
            return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq (%d) and num_blocks (%d) must be >= 1", o->max_blocks,
                        o->num_blocks);
        if (reinterpret_cast<uintptr_t>(o->block_table) & 3u)
            return fail(PA_ERR_INVALID_ARG, "block_table must be 4-byte aligned");
    } else if (have >= offsetof(pa_options, block_table) + sizeof(void*) && opts->block_table) {
        return fail(PA_ERR_INVALID_ARG, "pa_options.struct_size %u does not cover the paged-cache fields",
                    (unsigned)opts->struct_size);
    }
    if (have >= offsetof(pa_options, rope_theta) + sizeof(float)) {
        o->rope_theta = opts->rope_theta;
        if (!(o->rope_theta >= 0.f) || !std::isfinite(o->rope_theta))
            return fail(PA_ERR_INVALID_ARG, "rope_theta must be finite and >= 0 (got %g)", (double)o->rope_theta);
    }
    if (have >= offsetof(pa_options, reserved2) + sizeof(int32_t) && opts->reserved2 != 0)
        return fail(PA_ERR_INVALID_ARG, "pa_options.reserved2 must be 0");
    if (have >= offsetof(pa_options, kv_quant) + sizeof(int32_t) && opts->kv_quant != 0) {
        if (have < offsetof(pa_options, cache_v_scale) + sizeof(float*))
            return fail(PA_ERR_INVALID_ARG, "pa_options.struct_size %u does not cover the scale pointers",
                        (unsigned)opts->struct_size);
        if (opts->kv_quant != 1) return fail(PA_ERR_INVALID_ARG, "kv_quant must be 0 or 1 (got %d)", opts->kv_quant);
        if (opts->reserved3 != 0) return fail(PA_ERR_INVALID_ARG, "pa_options.reserved3 must be 0");
        if (!opts->cache_k_scale || !opts->cache_v_scale)
            return fail(PA_ERR_INVALID_ARG, "kv_quant = 1 needs cache_k_scale and cache_v_scale");
        if ((reinterpret_cast<uintptr_t>(opts->cache_k_scale) | reinterpret_cast<uintptr_t>(opts->cache_v_scale)) & 3u)
            return fail(PA_ERR_INVALID_ARG, "cache scales must be 4-byte aligned");
        o->kv_quant = 1;
        o->scale_k = opts->cache_k_scale;
        o->scale_v = opts->cache_v_scale;
    }
    if (have >= offsetof(pa_options, schedule) + sizeof(int32_t)) {
        if (opts->wait_timeout_test != 0 && opts->wait_timeout_test != 1)
            return fail(PA_ERR_INVALID_ARG, "wait_timeout_test must be 0 or 1");
        o->wait_timeout_test = opts->wait_timeout_test;
        if (opts->schedule < 0 || opts->schedule > 3)
            return fail(PA_ERR_INVALID_ARG, "schedule must be 0 .. 3 (got %d)", opts->schedule);
        if ((opts->schedule == 1 || opts->schedule == 3) && (o->kv_quant || o->wait_timeout_test))
            return fail(PA_ERR_INVALID_ARG, "schedule %d needs a bf16 cache and wait_timeout_test = 0",
                        opts->schedule);
        o->schedule = opts->schedule;
    }
    return PA_OK;
}

// Checks that need both the options and the call's sizes.
pa_status check_paged(const Options& o, int max_cache_len, int n_kv_heads) {
    if (!o.block_table) return PA_OK;
    if ((long long)o.max_blocks * o.block_size != max_cache_len)
        return fail(PA_ERR_INVALID_ARG, "max_cache_len (%d) must equal max_blocks_per_seq (%d) * block_size (%d)",
                    max_cache_len, o.max_blocks, o.block_size);
    if ((long long)o.num_blocks * n_kv_heads >= (1LL << 31))
        return fail(PA_ERR_UNSUPPORTED, "num_blocks * n_kv_heads must be < 2^31");
    return PA_OK;
}

// The schedule of a call (pa_options.schedule 1 .. 3).  Two-tile units
// unless the launch is mostly decode rows (new tokens averaging under 64 per
// sequence: a decode unit then splits its KV tiles between both softmax slots
// so that the second does not idle) or is so small that two-tile units would
// not give every SM one (then one-tile units, twice as many, each splitting
// its tiles).  The splitting kernel variant runs other units a few per cent
// slower and one K/V tile then feeds one Q tile instead of two, so it is not
// taken for anything else.  Measured on GB300 (152 SMs), TFLOP/s with
// one-tile / two-tile units: a 512-token chunk over a 4096-token prefix, GQA
// 32/8 (64 two-tile units) 819 / 540; 1024-token prompts (128 units) 315 /
// 296 (MHA) and 318 / 309 (GQA-4); a 1536-token MHA prompt (192 units) 490 /
// 531.  bf16 caches only.
int auto_schedule(int total_q, int num_seqs, int n_heads, int n_kv_heads, bool kv_quant, int sms) {
    if (kv_quant) return 2;
    if ((long long)total_q < 64LL * num_seqs) return 3;
    const int tpu = pa::kSlots * (pa::kBlockM / (n_heads / n_kv_heads));
    const long long full_units = (long long)n_kv_heads * (total_q / tpu);
    return full_units <= sms ? 1 : 2;
}

// Upper bound on the work units of a call (host-side; device metadata unread).
long long unit_bound(int total_q, int num_seqs, int n_heads, int n_kv_heads, int slots) {
    const int group = n_heads / n_kv_heads;
    const int tpu = slots * (pa::kBlockM / group);  // query tokens per work unit
    return (long long)n_kv_heads * ((total_q + tpu - 1) / tpu + num_seqs);
}

int sm_count(int dev, pa_status* s) {
    int sms = 0;
    const cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    *s = e == cudaSuccess ? PA_OK : cuda_fail(e, "cudaDeviceGetAttribute");
    return sms;
}

// Device address of the allocation-free entry point's scratch array in the
// current context, or nullptr if that entry point has not run there yet.
void* noalloc_scratch_if_set_up();

struct Scratch {
    pa::WorkspaceHeader* hdr;
    pa::SeqInfo* seqs;
    pa::Unit* units;
    int max_units;
    int* seq_scratch;      // int[2][num_seqs] for the scheduler
    void* rope = nullptr;  // room for the rotated q and k when the rotary embedding is on
};

// Enqueues the rotary prologue; q and k then point at the rotated copies in `rope`.
cudaError_t rotate(const void*& q, const void*& k, const int32_t* cu_seqlens_q, const pa::SeqInfo* seqs, void* rope,
                   int total_q, int num_seqs, int n_heads, int n_kv_heads, int head_dim, float theta, int pos0,
                   cudaStream_t stream) {
    pa::RopeParams rp;
    rp.q = static_cast<const __nv_bfloat16*>(q);
    rp.k = static_cast<const __nv_bfloat16*>(k);
    rp.q_rot = static_cast<__nv_bfloat16*>(rope);
    rp.k_rot = rp.q_rot + (size_t)total_q * n_heads * head_dim;
    rp.cu_seqlens_q = cu_seqlens_q;
    rp.seqs = seqs;
    rp.total_q = total_q;
    rp.num_seqs = num_seqs;
    rp.n_heads = n_heads;
    rp.n_kv_heads = n_kv_heads;
    rp.head_dim = head_dim;
    rp.pos0 = pos0;
    for (int i = 0; i < head_dim / 2; ++i)
        rp.inv_freq[i] = 1.0f / std::pow(theta, (float)(2 * i) / (float)head_dim);
    q = rp.q_rot;
    k = rp.k_rot;
    return pa::launch_rope(rp, stream);
}

// The attention kernel's parameters except its tensor maps.
void fill_fwd(pa::FwdParams& p, const void* k, const void* v, void* cache_k, void* cache_v, void* out, float* lse,
              const Scratch& scr, int max_cache_len, int n_heads, int n_kv_heads, float scale, int causal,
              const Options& o, int sched) {
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.cache_k = static_cast<__nv_bfloat16*>(cache_k);
    p.cache_v = static_cast<__nv_bfloat16*>(cache_v);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.hdr = scr.hdr;
    p.seqs = scr.seqs;
    p.units = scr.units;
    p.n_heads = n_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = n_heads / n_kv_heads;
    p.max_cache_len = max_cache_len;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.causal = causal;
    p.window = o.window;
    p.block_table = o.block_table;
    p.block_log2 = 0;
    while (o.block_table && (1 << p.block_log2) < o.block_size) ++p.block_log2;
    p.box_rows = std::min(o.block_size, pa::kBlockN);
    p.max_blocks = o.max_blocks;
    p.num_blocks = o.num_blocks;
    p.kv_quant = o.kv_quant;
    p.wait_timeout_test = o.wait_timeout_test;
    p.alt = sched != 2;
    p.unit_slots = sched == 1 ? 1 : pa::kSlots;
    p.out_align32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    p.scale_k = o.scale_k;
    p.scale_v = o.scale_v;
}

void fill_schedule(pa::ScheduleArgs& sa, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                   const int32_t* cache_offsets, int num_seqs, int total_q, int max_cache_len, int n_heads,
                   int n_kv_heads, int head_dim, int causal, const Options& o, const Scratch& scr, int slots, int ctas) {
    sa.cu_seqlens_q = cu_seqlens_q;
    sa.cu_seqlens_k = cu_seqlens_k;
    sa.cache_offsets = cache_offsets;
    sa.hdr = scr.hdr;
    sa.seqs = scr.seqs;
    sa.units = scr.units;
    sa.seq_scratch = scr.seq_scratch;
    sa.seq_group = scr.seq_scratch + num_seqs;
    sa.num_seqs = num_seqs;
    sa.total_q = total_q;
    sa.max_cache_len = max_cache_len;
    sa.n_kv_heads = n_kv_heads;
    sa.head_dim = head_dim;
    sa.group = n_heads / n_kv_heads;
    sa.causal = causal;
    sa.window = o.window;
    sa.max_units = scr.max_units;
    sa.num_ctas = ctas;
    sa.unit_slots = slots;
    sa.block_table = o.block_table;
    sa.block_size = o.block_size;
    sa.max_blocks = o.max_blocks;
    sa.num_blocks = o.num_blocks;
}

// Enqueues the scheduler and the attention kernel (arguments already checked).
pa_status enqueue(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                  const int32_t* cu_seqlens_k, void* cache_k, void* cache_v, const int32_t* cache_offsets, void* out,
                  float* lse, int num_seqs, int total_q, int max_cache_len, int n_heads, int n_kv_heads,
                  int head_dim, float scale, int causal, const Options& o, const Scratch& scr, long long units_bound,
                  int sched, int sms, cudaStream_t stream) {
    const int slots = sched == 1 ? 1 : pa::kSlots;  // Q tiles per unit
    pa::ScheduleArgs sa;
    fill_schedule(sa, cu_seqlens_q, cu_seqlens_k, cache_offsets, num_seqs, total_q, max_cache_len, n_heads, n_kv_heads,
                  head_dim, causal, o, scr, slots, (int)std::min<long long>(sms, units_bound));
    cudaError_t e = pa::launch_build_schedule(sa, stream);
    if (e != cudaSuccess) return cuda_fail(e, "schedule launch");

    int launches = 2;
    if (o.rope_theta > 0.f) {
        e = rotate(q, k, cu_seqlens_q, scr.seqs, scr.rope, total_q, num_seqs, n_heads, n_kv_heads, head_dim,
                   o.rope_theta, 0, stream);
        if (e != cudaSuccess) return cuda_fail(e, "rotary prologue launch");
        launches = 3;
    }

    pa::FwdParams p;
    fill_fwd(p, k, v, cache_k, cache_v, out, lse, scr, max_cache_len, n_heads, n_kv_heads, scale, causal, o, sched);
    e = pa::encode_fwd_maps(p, q, total_q, num_seqs, head_dim, o.num_blocks);
    if (e != cudaSuccess) return cuda_fail(e, "tensor map encoding");
    const int grid = (int)std::min<long long>(sms, units_bound);
    e = pa::launch_attn_fwd(p, head_dim, grid, stream);
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
    g_last_launches = launches;
    g_last_schedule = sched;
    return PA_OK;
}

}  // namespace

extern "C" {


const char* prefill_attn_status_string(pa_status s) {
    switch (s) {
        case PA_OK: return "PA_OK";
        case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
        case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
        case PA_ERR_CUDA: return "PA_ERR_CUDA";
        case PA_ERR_DEVICE_TIMEOUT: return "PA_ERR_DEVICE_TIMEOUT";
        case PA_ERR_DEVICE_METADATA: return "PA_ERR_DEVICE_METADATA";
        case PA_ERR_DEVICE_LAYOUT: return "PA_ERR_DEVICE_LAYOUT";
    }
    return "PA_ERR_UNKNOWN";
}

const char* prefill_attn_last_error(void) { return g_last_error; }

int prefill_attn_last_launch_count(void) { return g_last_launches; }

int prefill_attn_last_schedule(void) { return g_last_schedule; }

int prefill_attn_auto_schedule(int total_q, int num_seqs, int n_heads, int n_kv_heads, int kv_quant, int num_sms) {
    if (total_q <= 0 || num_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || num_sms <= 0 ||
        n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > pa::kBlockM)
        return -1;
    return auto_schedule(total_q, num_seqs, n_heads, n_kv_heads, kv_quant != 0, num_sms);
}

pa_status prefill_attn_varlen(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                              const int32_t* cu_seqlens_k, void* cache_k, void* cache_v,
                              const int32_t* cache_offsets, void* out, float* lse, int num_seqs, int total_q,
                              int max_cache_len, int n_heads, int n_kv_heads, int head_dim, float scale,
                              int causal, pa_stream_t stream_) {
    return prefill_attn_varlen_ex(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                                  num_seqs, total_q, max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal,
                                  nullptr, stream_);
}

pa_status prefill_attn_varlen_ex(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                                 const int32_t* cu_seqlens_k, void* cache_k, void* cache_v,
                                 const int32_t* cache_offsets, void* out, float* lse, int num_seqs, int total_q,
                                 int max_cache_len, int n_heads, int n_kv_heads, int head_dim, float scale,
                                 int causal, const pa_options* opts, pa_stream_t stream_) try {
    g_last_error[0] = 0;
    g_last_launches = 0;
    g_last_schedule = 0;
    Options o;
    pa_status s = read_options(opts, causal, &o);
    if (s != PA_OK) return s;
    s = check_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, num_seqs,
                   total_q, max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal, o.block_table != nullptr);
    if (s != PA_OK) return s;
    s = check_paged(o, max_cache_len, n_kv_heads);
    if (s != PA_OK) return s;
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    const int sms = sm_count(dev, &s);
    if (s != PA_OK) return s;
    const int sched = o.schedule            ? o.schedule
                      : o.wait_timeout_test ? 2  // the hook's kernel
                                            : auto_schedule(total_q, num_seqs, n_heads, n_kv_heads, o.kv_quant != 0, sms);
    const int slots = sched == 1 ? 1 : pa::kSlots;
    const long long max_units_ll = unit_bound(total_q, num_seqs, n_heads, n_kv_heads, slots);
    if (max_units_ll >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "too many work units");
    const StreamLock lock(dev, stream);
    Workspace* const ws = lock.ws;
    s = grow_workspace(*ws, stream, num_seqs, (int)max_units_ll);
    if (s != PA_OK) return s;
    Scratch scr{static_cast<pa::WorkspaceHeader*>(ws->ptr), ws_seqs(*ws), ws_units(*ws), ws->max_units,
                ws_seq_scratch(*ws)};
    if (o.rope_theta > 0.f) {
        s = get_rope_scratch(ws, stream, (size_t)total_q * (n_heads + n_kv_heads) * head_dim * 2, &scr.rope);
        if (s != PA_OK) return s;
    }
    return enqueue(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, num_seqs, total_q,
                   max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal, o, scr, max_units_ll, sched, sms,
                   stream);
} catch (...) {
    return caught();
}

pa_status prefill_attn_varlen_validate(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                                       const int32_t* cu_seqlens_k, void* cache_k, void* cache_v,
                                       const int32_t* cache_offsets, void* out, float* lse, int num_seqs,
                                       int total_q, int max_cache_len, int n_heads, int n_kv_heads, int head_dim,
                                       float scale, int causal, pa_stream_t stream_) try {
    g_last_error[0] = 0;
    pa_status s = check_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                             num_seqs, total_q, max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal);
    if (s != PA_OK || num_seqs == 0) return s;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    std::vector<int32_t> cq((size_t)num_seqs + 1), ck((size_t)num_seqs + 1), of(num_seqs);
    cudaError_t e = cudaMemcpyAsync(cq.data(), cu_seqlens_q, cq.size() * 4, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaMemcpyAsync(ck.data(), cu_seqlens_k, ck.size() * 4, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaMemcpyAsync(of.data(), cache_offsets, of.size() * 4, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "reading metadata");
    if (cq[0] != 0) return fail(PA_ERR_INVALID_ARG, "cu_seqlens_q[0] = %d, must be 0", cq[0]);
    if (cq[num_seqs] != total_q)
        return fail(PA_ERR_INVALID_ARG, "cu_seqlens_q[num_seqs] = %d but total_q = %d", cq[num_seqs], total_q);
    for (int b = 0; b < num_seqs; ++b) {
        const long long n = (long long)cq[b + 1] - cq[b];
        if (n < 0) return fail(PA_ERR_INVALID_ARG, "cu_seqlens_q decreases at sequence %d", b);
        if (of[b] < 0) return fail(PA_ERR_INVALID_ARG, "cache_offsets[%d] = %d < 0", b, of[b]);
        if ((long long)ck[b + 1] - ck[b] != (long long)of[b] + n)
            return fail(PA_ERR_INVALID_ARG,
                        "sequence %d: cu_seqlens_k gives %lld keys, cache_offsets + seqlen_q = %lld", b,
                        (long long)ck[b + 1] - ck[b], (long long)of[b] + n);
        if ((long long)of[b] + n > max_cache_len)
            return fail(PA_ERR_INVALID_ARG, "sequence %d: %lld tokens exceed max_cache_len %d", b,
                        (long long)of[b] + n, max_cache_len);
    }
    return PA_OK;
} catch (...) {
    return caught();
}

pa_status prefill_attn_device_status(pa_stream_t stream_, int32_t* flags) try {
    g_last_error[0] = 0;
    if (flags) *flags = 0;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    const StreamLock own(dev, stream);  // (no call replaces the workspace meanwhile)
    // the workspace's word, outgrown ones that graphs use included
    std::vector<void*> words = own.ws->old_headers;
    words.push_back(own.ws->ptr);
    words.push_back(noalloc_scratch_if_set_up());
    int32_t word = 0;
    for (void* ptr : words) {
        if (!ptr) continue;
        int32_t w = 0, zero = 0;
        e = cudaMemcpy(&w, ptr, sizeof w, cudaMemcpyDeviceToHost);
        if (e == cudaSuccess && w != 0) e = cudaMemcpy(ptr, &zero, sizeof zero, cudaMemcpyHostToDevice);
        if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
        word |= w;
    }
    if (flags) *flags = word;
    if (word == 0) return PA_OK;
    if (word & PA_DEVERR_TIMEOUT) return fail(PA_ERR_DEVICE_TIMEOUT, "device error word 0x%x", word);
    if (word & PA_DEVERR_SMEM_ALIGN) return fail(PA_ERR_DEVICE_LAYOUT, "device error word 0x%x", word);
    return fail(PA_ERR_DEVICE_METADATA, "device error word 0x%x", word);
} catch (...) {
    return caught();
}

void prefill_attn_release(void) try {
    std::lock_guard<std::mutex> lock(g_mu);
    int cur = 0;
    cudaGetDevice(&cur);
    for (auto& kv : g_ws) {
        Workspace& w = kv.second;
        cudaSetDevice(kv.first.first);
        for (void* ptr : {w.ptr, w.rope, w.aux})
            if (ptr) cudaFree(ptr);
        for (void* ptr : w.retired) cudaFree(ptr);
    }
    cudaSetDevice(cur);
    g_ws.clear();
} catch (...) {
}


}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free variant: the scheduler scratch lives in a fixed device array.
// ---------------------------------------------------------------------------
namespace {

constexpr int kNoAllocMaxSeqs = 4096;
constexpr int kNoAllocMaxUnits = 61440;
constexpr size_t kNoAllocHeaderBytes = 16;
constexpr size_t kNoAllocBytes = kNoAllocHeaderBytes + (size_t)kNoAllocMaxSeqs * sizeof(pa::SeqInfo) +
                                 (size_t)kNoAllocMaxUnits * sizeof(pa::Unit) + 2 * (size_t)kNoAllocMaxSeqs * sizeof(int);
static_assert(sizeof(pa::WorkspaceHeader) <= kNoAllocHeaderBytes, "header size");

// In host code this name is only a stand-in for the array; its device address
// comes from cudaGetSymbolAddress, once per device.
__device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocBytes];

// The array's address is looked up once per CUDA context, keyed by the
// context's unique id: a device reset destroys the context (and the loaded
// device code with it), and the next context, even on the same device, gets an
// id of its own and so a fresh lookup.
std::mutex g_noalloc_mu;
std::map<unsigned long long, void*> g_noalloc_addr;

using CtxGetCurrentFn = CUresult (*)(CUcontext*);
using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long*);

// Unique id of the current context (false if there is none or the driver lacks the call).
bool current_context_id(unsigned long long* id) {
    static CtxGetCurrentFn get_current = nullptr;
    static CtxGetIdFn get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<CtxGetCurrentFn>(f);
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<CtxGetIdFn>(f);
    });
    CUcontext ctx = nullptr;
    if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx) return false;
    return get_id(ctx, id) == CUDA_SUCCESS;
}

pa_status noalloc_scratch(void** out) {
    unsigned long long id = 0;
    if (!current_context_id(&id)) return fail(PA_ERR_CUDA, "no current CUDA context");
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    auto it = g_noalloc_addr.find(id);
    if (it != g_noalloc_addr.end()) {
        *out = it->second;
        return PA_OK;
    }
    void* ptr = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&ptr, g_noalloc_scratch);  // in the current context
    if (e != cudaSuccess || !ptr) return cuda_fail(e, "cudaGetSymbolAddress(scratch)");
    g_noalloc_addr[id] = ptr;
    *out = ptr;
    return PA_OK;
}

}  // namespace

namespace {
void* noalloc_scratch_if_set_up() {
    unsigned long long id = 0;
    if (!current_context_id(&id)) return nullptr;
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    auto it = g_noalloc_addr.find(id);
    return it == g_noalloc_addr.end() ? nullptr : it->second;
}
}  // namespace

extern "C" pa_status prefill_attn_varlen_noalloc(const void* q, const void* k, const void* v,
                                                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                                                 void* cache_k, void* cache_v, const int32_t* cache_offsets,
                                                 void* out, float* lse, int num_seqs, int total_q,
                                                 int max_cache_len, int n_heads, int n_kv_heads, int head_dim,
                                                 float scale, int causal, pa_stream_t stream_) try {
    g_last_error[0] = 0;
    g_last_launches = 0;
    g_last_schedule = 0;
    pa_status s = check_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse,
                             num_seqs, total_q, max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal);
    if (s != PA_OK) return s;
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    const int sms = sm_count(dev, &s);
    if (s != PA_OK) return s;
    const int sched = auto_schedule(total_q, num_seqs, n_heads, n_kv_heads, false, sms);
    const long long units = unit_bound(total_q, num_seqs, n_heads, n_kv_heads, sched == 1 ? 1 : pa::kSlots);
    if (num_seqs > kNoAllocMaxSeqs)
        return fail(PA_ERR_UNSUPPORTED, "num_seqs %d exceeds the allocation-free limit %d", num_seqs, kNoAllocMaxSeqs);
    if (units > kNoAllocMaxUnits)
        return fail(PA_ERR_UNSUPPORTED, "up to %lld work units exceed the allocation-free limit %d", units,
                    kNoAllocMaxUnits);
    void* scratch = nullptr;
    s = noalloc_scratch(&scratch);
    if (s != PA_OK) return s;
    // the array keeps the previous call's contents: clear the header (error word, counters)
    e = cudaMemsetAsync(scratch, 0, kNoAllocHeaderBytes, stream);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the scratch header");
    pa::SeqInfo* seqs = reinterpret_cast<pa::SeqInfo*>(static_cast<unsigned char*>(scratch) + kNoAllocHeaderBytes);
    pa::Unit* units_ws = reinterpret_cast<pa::Unit*>(seqs + kNoAllocMaxSeqs);
    Scratch scr{static_cast<pa::WorkspaceHeader*>(scratch), seqs, units_ws, kNoAllocMaxUnits,
                reinterpret_cast<int*>(units_ws + kNoAllocMaxUnits)};
    return enqueue(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, num_seqs, total_q,
                   max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal, Options(), scr, units, sched, sms,
                   stream);
} catch (...) {
    return caught();
}

// ---------------------------------------------------------------------------
// Long-context calls: sink tokens, a shared prefix, key weights, eviction.
// ---------------------------------------------------------------------------
namespace {

// A prefix that every sequence of a call sees (pa_prefix, checked).
struct Prefix {
    int len = 0;
    const void* k = nullptr;
    const void* v = nullptr;
    int capacity = 0;
    const float* scale_k = nullptr;
    const float* scale_v = nullptr;
    const int32_t* block_table = nullptr;
};

pa_status read_prefix(const pa_prefix* prefix, const Options& o, Prefix* out) {
    *out = Prefix();
    if (!prefix) return fail(PA_ERR_INVALID_ARG, "prefix is NULL");
    if (prefix->struct_size < sizeof(pa_prefix))
        return fail(PA_ERR_INVALID_ARG, "pa_prefix.struct_size %u is too small", (unsigned)prefix->struct_size);
    if (prefix->reserved != 0) return fail(PA_ERR_INVALID_ARG, "pa_prefix.reserved must be 0");
    if (prefix->len < 0) return fail(PA_ERR_INVALID_ARG, "pa_prefix.len must be >= 0 (got %d)", prefix->len);
    out->len = prefix->len;
    if (prefix->len == 0) return PA_OK;  // nothing of it is read
    if (o.block_table) {
        if (!prefix->block_table) return fail(PA_ERR_INVALID_ARG, "a paged cache needs pa_prefix.block_table");
        if (reinterpret_cast<uintptr_t>(prefix->block_table) & 3u)
            return fail(PA_ERR_INVALID_ARG, "pa_prefix.block_table must be 4-byte aligned");
        out->block_table = prefix->block_table;
        return PA_OK;
    }
    if (!prefix->k || !prefix->v) return fail(PA_ERR_INVALID_ARG, "pa_prefix.k and pa_prefix.v must not be NULL");
    if (!aligned16(prefix->k) || !aligned16(prefix->v))
        return fail(PA_ERR_INVALID_ARG, "pa_prefix.k and pa_prefix.v must be 16-byte aligned");
    if (prefix->capacity < prefix->len)
        return fail(PA_ERR_INVALID_ARG, "pa_prefix.len (%d) exceeds its capacity (%d)", prefix->len, prefix->capacity);
    if (o.kv_quant) {
        if (!prefix->k_scale || !prefix->v_scale)
            return fail(PA_ERR_INVALID_ARG, "kv_quant = 1 needs pa_prefix.k_scale and pa_prefix.v_scale");
        if ((reinterpret_cast<uintptr_t>(prefix->k_scale) | reinterpret_cast<uintptr_t>(prefix->v_scale)) & 3u)
            return fail(PA_ERR_INVALID_ARG, "prefix scales must be 4-byte aligned");
        out->scale_k = prefix->k_scale;
        out->scale_v = prefix->v_scale;
    }
    out->k = prefix->k;
    out->v = prefix->v;
    out->capacity = prefix->capacity;
    return PA_OK;
}

// Rows are cut into as many pieces as have slabs of partial results within this many
// bytes, at most kMaxPieces: one bound for the sequences' own keys, one for the
// prefix's.  One slab (total_q rows of n_heads outputs) is the least that each part of a
// prefix call has, however large: two of 0.54 GB for 32768 new tokens of 32 heads, D = 128.
constexpr long long kPartialBytes = 64ll << 20, kPrefixPartialBytes = 256ll << 20;
using pa::kMaxPieces;
constexpr int kMinPieceTiles = 4;
constexpr int kUncutTiles = 8;
constexpr int kDirectSeqs = 64;
constexpr int kPieceWaves = 2;

pa_status check_unused(const Options& o, const char* what) {
    if (o.schedule || o.wait_timeout_test)
        return fail(PA_ERR_INVALID_ARG, "%s takes no schedule and no wait_timeout_test", what);
    return PA_OK;
}

// Enqueues a long-context attention call (arguments already checked).
pa_status enqueue_long(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                       const int32_t* cu_seqlens_k, void* cache_k, void* cache_v, const int32_t* cache_offsets,
                       void* out, float* lse, int num_seqs, int total_q, int max_cache_len, int n_heads,
                       int n_kv_heads, int head_dim, float scale, int causal, int sinks, const Prefix& pre,
                       const Options& o, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    pa_status s;
    const int sms = sm_count(dev, &s);
    if (s != PA_OK) return s;
    const int sched = o.schedule ? o.schedule
                                 : auto_schedule(total_q, num_seqs, n_heads, n_kv_heads, o.kv_quant != 0, sms);
    const int slots = sched == 1 ? 1 : pa::kSlots;
    const int tpu = slots * (pa::kBlockM / (n_heads / n_kv_heads));
    const long long blocks = ((long long)total_q + tpu - 1) / tpu;
    const long long own_units = (blocks + num_seqs) * n_kv_heads;
    const long long pre_units = pre.len > 0 ? blocks * n_kv_heads : 0;
    const long long target = (long long)kPieceWaves * sms;
    const long long slab_rows = (long long)total_q * n_heads;
    const long long slab_bytes = slab_rows * (head_dim + 1) * 4;
    const int fit = (int)std::max(1ll, std::min((long long)kMaxPieces, kPartialBytes / slab_bytes));
    // a row under a short window is not cut: its few tiles cost less than the merge's
    // launch (one row, window 256: 11.4 us whole, 12.9 in two pieces; 14 and 16 from Python)
    const long long most_tiles = o.window ? ((long long)o.window + sinks) / pa::kBlockN + 3 : LLONG_MAX;
    const int max_pieces = most_tiles <= kUncutTiles ? 1 : fit;
    // a prefix of fewer units than wanted is cut to make as many; of one with more
    // than CTAs only the units of the last round are, into at most four
    int max_prefix_pieces = 0;
    if (pre.len > 0) {
        const long long want = pre_units > sms ? 4 : std::min((long long)kMaxPieces, (target + pre_units - 1) / pre_units);
        max_prefix_pieces = (int)std::max(1ll, std::min(want, kPrefixPartialBytes / slab_bytes));
    }
    const bool merge = pre.len > 0 || max_pieces > 1;
    const long long slabs = merge ? max_pieces + max_prefix_pieces : 0;
    // pieces per block: at most 1 + tiles / piece size, so a call has at most its
    // blocks plus twice the wanted units (a causal sequence's blocks average at
    // least half its longest one); twice that again is room to spare
    const long long units =
        std::min(own_units * max_pieces + pre_units * std::max(1, max_prefix_pieces), own_units + pre_units + 4 * target);
    if (units >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "too many work units");
    const StreamLock lock(dev, stream);
    Workspace* const ws = lock.ws;
    s = grow_workspace(*ws, stream, num_seqs + 1, 0);
    if (s != PA_OK) return s;
    const size_t list_bytes = align_up((size_t)units * sizeof(pa::UnitX), 256);
    const size_t seq_bytes = align_up(((size_t)num_seqs + 1 + pre_units) * sizeof(int), 256);
    const size_t tok_bytes = merge ? align_up((size_t)total_q * sizeof(int), 256) : 0;
    const size_t lse_bytes = align_up((size_t)(slabs * slab_rows) * sizeof(float), 256);
    const size_t o_bytes = (size_t)(slabs * slab_rows) * head_dim * sizeof(float);
    void* aux = nullptr;
    s = get_aux_scratch(ws, stream, list_bytes + seq_bytes + tok_bytes + lse_bytes + o_bytes, &aux);
    if (s != PA_OK) return s;
    char* at = static_cast<char*>(aux);
    Scratch scr{static_cast<pa::WorkspaceHeader*>(ws->ptr), ws_seqs(*ws), nullptr, (int)units, ws_seq_scratch(*ws)};
    if (o.rope_theta > 0.f) {
        s = get_rope_scratch(ws, stream, (size_t)total_q * (n_heads + n_kv_heads) * head_dim * 2, &scr.rope);
        if (s != PA_OK) return s;
    }
    const int grid = (int)std::min<long long>(sms, units);

    pa::LongScheduleArgs sa;
    fill_schedule(sa, cu_seqlens_q, cu_seqlens_k, cache_offsets, num_seqs, total_q, max_cache_len, n_heads, n_kv_heads,
                  head_dim, causal, o, scr, slots, grid);
    sa.seq_group = scr.seq_scratch + num_seqs + 1;
    sa.xunits = reinterpret_cast<pa::UnitX*>(at);
    sa.seq_pieces = reinterpret_cast<int*>(at + list_bytes);
    sa.pre_pieces = sa.seq_pieces + num_seqs + 1;
    sa.tok_pieces = merge ? reinterpret_cast<int*>(at + list_bytes + seq_bytes) : nullptr;
    sa.sinks = sinks;
    sa.prefix_len = pre.len;
    sa.prefix_table = pre.block_table;
    sa.max_pieces = max_pieces;
    sa.max_prefix_pieces = max_prefix_pieces;
    sa.min_tiles = kMinPieceTiles;
    // Few sequences with at most one unit per SM before cutting (so at most a few
    // pieces per CTA): the attention kernel's CTAs plan for themselves, which saves
    // the scheduler's launch.  The rotary prologue needs the scheduler's sequences.
    const bool direct = num_seqs < kDirectSeqs && own_units + pre_units <= grid && o.rope_theta == 0.f;
    int launches = 1;
    if (!direct) {
        e = pa::launch_build_long_schedule(sa, stream);
        if (e != cudaSuccess) return cuda_fail(e, "schedule launch");
        ++launches;
    }
    if (o.rope_theta > 0.f) {
        e = rotate(q, k, cu_seqlens_q, scr.seqs, scr.rope, total_q, num_seqs, n_heads, n_kv_heads, head_dim,
                   o.rope_theta, pre.len, stream);
        if (e != cudaSuccess) return cuda_fail(e, "rotary prologue launch");
        ++launches;
    }

    pa::FwdParamsX p;
    fill_fwd(p, k, v, cache_k, cache_v, out, lse, scr, max_cache_len, n_heads, n_kv_heads, scale, causal, o, sched);
    p.xunits = sa.xunits;
    p.num_seqs = num_seqs;
    p.sinks = sinks;
    p.prefix_len = pre.len;
    p.prefix_cap = pre.capacity;
    p.prefix_table = pre.block_table;
    p.prefix_scale_k = pre.scale_k;
    p.prefix_scale_v = pre.scale_v;
    p.part_lse = reinterpret_cast<float*>(at + list_bytes + seq_bytes + tok_bytes);
    p.part_o = reinterpret_cast<float*>(at + list_bytes + seq_bytes + tok_bytes + lse_bytes);
    p.slab_rows = (size_t)slab_rows;
    p.direct = direct;
    p.plan = sa;
    e = pa::encode_fwd_maps(p, q, total_q, num_seqs, head_dim, o.num_blocks);
    if (e == cudaSuccess && pre.k) e = pa::encode_prefix_maps(p, head_dim, pre.k, pre.v);
    if (e != cudaSuccess) return cuda_fail(e, "tensor map encoding");
    e = head_dim == 32   ? pa::launch_attn_long_d<32>(p, grid, stream)
        : head_dim == 64 ? pa::launch_attn_long_d<64>(p, grid, stream)
                         : pa::launch_attn_long_d<128>(p, grid, stream);
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
    if (merge) {
        pa::MergeArgs ma{p.part_o, p.part_lse, sa.tok_pieces, pre.len > 0 ? sa.pre_pieces : nullptr, tpu,
                         n_heads / n_kv_heads, max_pieces, static_cast<__nv_bfloat16*>(out), lse, total_q, n_heads};
        e = pa::launch_merge(ma, head_dim, sms, stream);
        if (e != cudaSuccess) return cuda_fail(e, "merge launch");
        ++launches;
    }
    g_last_launches = launches;
    g_last_schedule = sched;
    return PA_OK;
}

// Whether [a, a + a_bytes) and [b, b + b_bytes) overlap.
bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + b_bytes && y < x + a_bytes;
}

// A buffer of a call, and whether the call writes it (at = nullptr: not given).
struct Span {
    const char* name;
    const void* at;
    size_t bytes;
    bool written;
};

// Rows of a call's cache (and of its scales and weights).
size_t cache_rows(const Options& o, int num_seqs, int max_cache_len, int n_kv_heads) {
    return o.block_table ? (size_t)o.num_blocks * n_kv_heads * o.block_size : (size_t)num_seqs * n_kv_heads * max_cache_len;
}

// What a call writes overlaps nothing else of it.
pa_status check_disjoint(const Span* s, size_t n) {
    for (size_t i = 0; i < n; ++i)
        for (size_t j = i + 1; j < n; ++j)
            if (s[i].at && s[j].at && (s[i].written || s[j].written) && overlap(s[i].at, s[i].bytes, s[j].at, s[j].bytes))
                return fail(PA_ERR_INVALID_ARG, "%s must not overlap %s", s[i].name, s[j].name);
    return PA_OK;
}

// The kernels' position arithmetic stays within 32 bits: positions and spans are
// at most kMaxTokens each, so the sum of two fits, and so do the schedulers' loops
// over as many sequences, which step 1024 at a time.  A window or sink count past
// the cache's capacity says the same as the capacity.
constexpr int kMaxTokens = 1 << 30;

pa_status check_capacity(int num_seqs, int max_cache_len, int prefix_len) {
    if (num_seqs > kMaxTokens) return fail(PA_ERR_UNSUPPORTED, "num_seqs (%d) must be at most 2^30", num_seqs);
    if (max_cache_len > kMaxTokens || prefix_len > kMaxTokens)
        return fail(PA_ERR_UNSUPPORTED, "max_cache_len (%d) and the prefix (%d tokens) must be at most 2^30",
                    max_cache_len, prefix_len);
    return PA_OK;
}

int clamp_span(int tokens, int max_cache_len) { return std::min(tokens, max_cache_len); }

int log2_of(int block_size) {
    int l = 0;
    while ((1 << l) < block_size) ++l;
    return l;
}

}  // namespace

extern "C" {

pa_status prefill_attn_varlen_sinks(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                                    const int32_t* cu_seqlens_k, void* cache_k, void* cache_v,
                                    const int32_t* cache_offsets, void* out, float* lse, int num_seqs, int total_q,
                                    int max_cache_len, int n_heads, int n_kv_heads, int head_dim, float scale,
                                    int sink_tokens, const pa_options* opts, pa_stream_t stream_) try {
    g_last_error[0] = 0;
    g_last_launches = 0;
    g_last_schedule = 0;
    Options o;
    pa_status s = read_options(opts, 1, &o);
    if (s != PA_OK) return s;
    if (o.window < 1) return fail(PA_ERR_INVALID_ARG, "sink tokens need a window (pa_options.window >= 1)");
    if (sink_tokens < 0) return fail(PA_ERR_INVALID_ARG, "sink_tokens must be >= 0 (got %d)", sink_tokens);
    if (o.wait_timeout_test) return fail(PA_ERR_INVALID_ARG, "wait_timeout_test is for prefill_attn_varlen_ex");
    s = check_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, num_seqs, total_q,
                   max_cache_len, n_heads, n_kv_heads, head_dim, scale, 1, o.block_table != nullptr);
    if (s != PA_OK) return s;
    s = check_paged(o, max_cache_len, n_kv_heads);
    if (s != PA_OK) return s;
    s = check_capacity(num_seqs, max_cache_len, 0);
    if (s != PA_OK) return s;
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    o.window = clamp_span(o.window, max_cache_len);
    return enqueue_long(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, num_seqs,
                        total_q, max_cache_len, n_heads, n_kv_heads, head_dim, scale, 1,
                        clamp_span(sink_tokens, max_cache_len), Prefix(), o,
                        reinterpret_cast<cudaStream_t>(stream_));
} catch (...) {
    return caught();
}

pa_status prefill_attn_varlen_prefix(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                                     const int32_t* cu_seqlens_k, void* cache_k, void* cache_v,
                                     const int32_t* cache_offsets, void* out, float* lse, int num_seqs, int total_q,
                                     int max_cache_len, int n_heads, int n_kv_heads, int head_dim, float scale,
                                     int causal, const pa_prefix* prefix, const pa_options* opts,
                                     pa_stream_t stream_) try {
    g_last_error[0] = 0;
    g_last_launches = 0;
    g_last_schedule = 0;
    Options o;
    pa_status s = read_options(opts, causal, &o);
    if (s != PA_OK) return s;
    if (o.window) return fail(PA_ERR_INVALID_ARG, "a shared prefix takes no sliding window");
    if (o.wait_timeout_test) return fail(PA_ERR_INVALID_ARG, "wait_timeout_test is for prefill_attn_varlen_ex");
    s = check_args(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, num_seqs, total_q,
                   max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal, o.block_table != nullptr);
    if (s != PA_OK) return s;
    s = check_paged(o, max_cache_len, n_kv_heads);
    if (s != PA_OK) return s;
    Prefix pre;
    s = read_prefix(prefix, o, &pre);
    if (s != PA_OK) return s;
    s = check_capacity(num_seqs, max_cache_len, pre.len);
    if (s != PA_OK) return s;
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    if (pre.k && (pre.k == out || pre.v == out || pre.k == cache_k || pre.k == cache_v || pre.v == cache_k ||
                  pre.v == cache_v))
        return fail(PA_ERR_INVALID_ARG, "the prefix must not alias out or the caches");
    if (pre.len > 0) {
        // the rows that are read: [0, len) of every head
        const size_t rows = pre.k ? (size_t)(n_kv_heads - 1) * pre.capacity + pre.len : 0;
        const size_t row_bytes = o.kv_quant ? head_dim : 2 * head_dim;
        const size_t blocks = pre.block_table ? ((size_t)pre.len + o.block_size - 1) / o.block_size : 0;
        const size_t out_rows = (size_t)total_q * n_heads;
        const Span spans[] = {{"out", out, out_rows * head_dim * 2, true},
                              {"lse", lse, out_rows * 4, true},
                              {"the prefix's k", pre.k, rows * row_bytes, false},
                              {"the prefix's v", pre.v, rows * row_bytes, false},
                              {"the prefix's k_scale", pre.scale_k, rows * 4, false},
                              {"the prefix's v_scale", pre.scale_v, rows * 4, false},
                              {"the prefix's block_table", pre.block_table, blocks * 4, false}};
        s = check_disjoint(spans, sizeof spans / sizeof *spans);
        if (s != PA_OK) return s;
    }
    return enqueue_long(q, k, v, cu_seqlens_q, cu_seqlens_k, cache_k, cache_v, cache_offsets, out, lse, num_seqs,
                        total_q, max_cache_len, n_heads, n_kv_heads, head_dim, scale, causal, 0, pre, o,
                        reinterpret_cast<cudaStream_t>(stream_));
} catch (...) {
    return caught();
}

pa_status prefill_attn_key_weights(const void* q, const void* k, const int32_t* cu_seqlens_q,
                                   const int32_t* cu_seqlens_k, const void* cache_k, const int32_t* cache_offsets,
                                   const float* lse, float* weights, int num_seqs, int total_q, int max_cache_len,
                                   int n_heads, int n_kv_heads, int head_dim, float scale, int causal,
                                   int sink_tokens, int prefix_len, const pa_options* opts, pa_stream_t stream_) try {
    g_last_error[0] = 0;
    g_last_launches = 0;
    g_last_schedule = 0;
    Options o;
    pa_status s = read_options(opts, causal, &o);
    if (s != PA_OK) return s;
    s = check_unused(o, "prefill_attn_key_weights");
    if (s != PA_OK) return s;
    if (sink_tokens < 0) return fail(PA_ERR_INVALID_ARG, "sink_tokens must be >= 0 (got %d)", sink_tokens);
    if (sink_tokens > 0 && o.window < 1)
        return fail(PA_ERR_INVALID_ARG, "sink tokens need a window (pa_options.window >= 1)");
    if (prefix_len < 0) return fail(PA_ERR_INVALID_ARG, "prefix_len must be >= 0 (got %d)", prefix_len);
    if (prefix_len > 0 && o.window) return fail(PA_ERR_INVALID_ARG, "a shared prefix takes no sliding window");
    // v, cache_v and out have no part here: stand-ins that satisfy the shared checks
    const void* none = reinterpret_cast<const void*>(uintptr_t(16));
    if (num_seqs > 0 && total_q > 0) {
        if (!lse) return fail(PA_ERR_INVALID_ARG, "lse is NULL");
        if (!weights) return fail(PA_ERR_INVALID_ARG, "weights is NULL");
        if (reinterpret_cast<uintptr_t>(weights) & 3u)
            return fail(PA_ERR_INVALID_ARG, "weights must be 4-byte aligned");
        if (static_cast<const void*>(weights) == lse || static_cast<const void*>(weights) == q ||
            static_cast<const void*>(weights) == k || static_cast<const void*>(weights) == cache_k)
            return fail(PA_ERR_INVALID_ARG, "weights must not alias an input");
    }
    s = check_args(q, k, none, cu_seqlens_q, cu_seqlens_k, cache_k, reinterpret_cast<const void*>(uintptr_t(32)),
                   cache_offsets, reinterpret_cast<const void*>(uintptr_t(48)), lse, num_seqs, total_q, max_cache_len,
                   n_heads, n_kv_heads, head_dim, scale, causal, o.block_table != nullptr);
    if (s != PA_OK) return s;
    s = check_paged(o, max_cache_len, n_kv_heads);
    if (s != PA_OK) return s;
    s = check_capacity(num_seqs, max_cache_len, prefix_len);
    if (s != PA_OK) return s;
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    const size_t rows = cache_rows(o, num_seqs, max_cache_len, n_kv_heads);
    const size_t q_rows = (size_t)total_q * n_heads, k_rows = (size_t)total_q * n_kv_heads;
    const Span spans[] = {{"weights", weights, rows * 4, true},
                          {"q", q, q_rows * head_dim * 2, false},
                          {"k", k, k_rows * head_dim * 2, false},
                          {"cache_k", cache_k, rows * head_dim * (o.kv_quant ? 1 : 2), false},
                          {"cache_k_scale", o.scale_k, rows * 4, false},
                          {"lse", lse, q_rows * 4, false},
                          {"cu_seqlens_q", cu_seqlens_q, ((size_t)num_seqs + 1) * 4, false},
                          {"cu_seqlens_k", cu_seqlens_k, ((size_t)num_seqs + 1) * 4, false},
                          {"cache_offsets", cache_offsets, (size_t)num_seqs * 4, false},
                          {"block_table", o.block_table, (size_t)num_seqs * o.max_blocks * 4, false}};
    s = check_disjoint(spans, sizeof spans / sizeof *spans);
    if (s != PA_OK) return s;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    const int sms = sm_count(dev, &s);
    if (s != PA_OK) return s;
    o.window = clamp_span(o.window, max_cache_len);
    sink_tokens = clamp_span(sink_tokens, max_cache_len);
    // units of at least two key tiles (or the sequence's last); prefix and new
    // keys are cut apart, so a sequence has at most one tile more than its rows need
    const long long tiles = ((long long)max_cache_len + pa::kBlockN - 1) / pa::kBlockN + 1;
    const long long units = (long long)num_seqs * n_kv_heads * ((tiles + 1) / 2);
    if (units >= (1LL << 31)) return fail(PA_ERR_UNSUPPORTED, "too many work units");
    const StreamLock lock(dev, stream);
    Workspace* const ws = lock.ws;
    s = grow_workspace(*ws, stream, num_seqs, (int)units);
    if (s != PA_OK) return s;
    Scratch scr{static_cast<pa::WorkspaceHeader*>(ws->ptr), ws_seqs(*ws), ws_units(*ws), ws->max_units,
                ws_seq_scratch(*ws)};
    if (o.rope_theta > 0.f) {
        s = get_rope_scratch(ws, stream, (size_t)total_q * (n_heads + n_kv_heads) * head_dim * 2, &scr.rope);
        if (s != PA_OK) return s;
    }
    const int grid = (int)std::min<long long>(sms, units);
    pa::KeyScheduleArgs sa;
    fill_schedule(sa, cu_seqlens_q, cu_seqlens_k, cache_offsets, num_seqs, total_q, max_cache_len, n_heads, n_kv_heads,
                  head_dim, causal, o, scr, pa::kSlots, grid);
    sa.sinks = sink_tokens;
    e = pa::launch_build_key_schedule(sa, stream);
    if (e != cudaSuccess) return cuda_fail(e, "schedule launch");
    int launches = 2;
    if (o.rope_theta > 0.f) {
        e = rotate(q, k, cu_seqlens_q, scr.seqs, scr.rope, total_q, num_seqs, n_heads, n_kv_heads, head_dim,
                   o.rope_theta, prefix_len, stream);
        if (e != cudaSuccess) return cuda_fail(e, "rotary prologue launch");
        ++launches;
    }
    pa::KeyWeightsParams p;
    fill_fwd(p, k, k, const_cast<void*>(cache_k), const_cast<void*>(cache_k), nullptr, const_cast<float*>(lse), scr,
             max_cache_len, n_heads, n_kv_heads, scale, causal, o, 2);
    p.weights = weights;
    p.sinks = sink_tokens;
    e = pa::encode_fwd_maps(p, q, total_q, num_seqs, head_dim, o.num_blocks);
    if (e == cudaSuccess) e = pa::encode_one_token_map(p, q, total_q, head_dim);
    if (e != cudaSuccess) return cuda_fail(e, "tensor map encoding");
    e = pa::launch_key_weights(p, head_dim, grid, stream);
    if (e != cudaSuccess) return cuda_fail(e, "key weight launch");
    g_last_launches = launches;
    return PA_OK;
} catch (...) {
    return caught();
}

pa_status prefill_attn_evict(void* cache_k, void* cache_v, const float* weights, const int32_t* lengths,
                             int32_t* kept_lengths, int32_t* kept_index, float* kept_weights, int num_seqs,
                             int max_cache_len, int n_kv_heads, int head_dim, int budget, int sink_tokens,
                             int recent_tokens, const pa_options* opts, pa_stream_t stream_) try {
    g_last_error[0] = 0;
    g_last_launches = 0;
    g_last_schedule = 0;
    Options o;
    pa_status s = read_options(opts, 1, &o);
    if (s != PA_OK) return s;
    s = check_unused(o, "prefill_attn_evict");
    if (s != PA_OK) return s;
    if (o.window) return fail(PA_ERR_INVALID_ARG, "prefill_attn_evict takes no window");
    if (o.rope_theta > 0.f) return fail(PA_ERR_INVALID_ARG, "prefill_attn_evict takes no rope_theta");
    if (num_seqs < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs must be >= 0 (got %d)", num_seqs);
    if (max_cache_len < 1) return fail(PA_ERR_INVALID_ARG, "max_cache_len must be >= 1 (got %d)", max_cache_len);
    if (n_kv_heads < 1) return fail(PA_ERR_INVALID_ARG, "n_kv_heads must be >= 1 (got %d)", n_kv_heads);
    if (head_dim != 32 && head_dim != 64 && head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim must be 32, 64 or 128 (got %d)", head_dim);
    if (budget < 1) return fail(PA_ERR_INVALID_ARG, "budget must be >= 1 (got %d)", budget);
    if (sink_tokens < 0 || recent_tokens < 0 || (long long)sink_tokens + recent_tokens > budget)
        return fail(PA_ERR_INVALID_ARG, "sink_tokens (%d) and recent_tokens (%d) must be >= 0 and fit the budget (%d)",
                    sink_tokens, recent_tokens, budget);
    s = check_paged(o, max_cache_len, n_kv_heads);
    if (s != PA_OK) return s;
    s = check_capacity(num_seqs, max_cache_len, 0);
    if (s != PA_OK) return s;
    // no sequence is longer than max_cache_len, so a larger budget says the same; only
    // a caller's index has an entry for each of its tokens
    if (!kept_index) budget = std::min(budget, max_cache_len);
    const long long heads = (long long)num_seqs * n_kv_heads;
    if (heads >= (1LL << 24)) return fail(PA_ERR_UNSUPPORTED, "num_seqs * n_kv_heads must be < 2^24");
    if (!o.block_table && heads * max_cache_len >= (1LL << 31))
        return fail(PA_ERR_UNSUPPORTED, "num_seqs * n_kv_heads * max_cache_len must be < 2^31");
    if (num_seqs == 0) return PA_OK;
    const void* ptrs[] = {cache_k, cache_v, weights, lengths, kept_lengths};
    const char* names[] = {"cache_k", "cache_v", "weights", "lengths", "kept_lengths"};
    for (int i = 0; i < 5; ++i) {
        if (!ptrs[i]) return fail(PA_ERR_INVALID_ARG, "%s is NULL", names[i]);
        if (i < 2 ? !aligned16(ptrs[i]) : (reinterpret_cast<uintptr_t>(ptrs[i]) & 3u) != 0)
            return fail(PA_ERR_INVALID_ARG, "%s must be %d-byte aligned", names[i], i < 2 ? 16 : 4);
    }
    if ((reinterpret_cast<uintptr_t>(kept_index) | reinterpret_cast<uintptr_t>(kept_weights)) & 3u)
        return fail(PA_ERR_INVALID_ARG, "kept_index and kept_weights must be 4-byte aligned");
    const size_t rows = cache_rows(o, num_seqs, max_cache_len, n_kv_heads);
    const size_t row_bytes = o.kv_quant ? head_dim : 2 * head_dim;
    const size_t index_bytes = (size_t)heads * budget * sizeof(int);
    if (overlap(cache_k, rows * row_bytes, cache_v, rows * row_bytes))
        return fail(PA_ERR_INVALID_ARG, "cache_k and cache_v must not overlap");
    if (kept_weights && kept_weights != weights && overlap(weights, rows * 4, kept_weights, rows * 4))
        return fail(PA_ERR_INVALID_ARG, "kept_weights must be weights itself or not overlap it");
    const Span spans[] = {{"kept_index", kept_index, index_bytes, true},
                          {"kept_lengths", kept_lengths, (size_t)num_seqs * 4, true},
                          {"kept_weights", kept_weights == weights ? nullptr : kept_weights, rows * 4, true},
                          {"cache_k", cache_k, rows * row_bytes, true},
                          {"cache_v", cache_v, rows * row_bytes, true},
                          {"cache_k_scale", o.scale_k, rows * 4, true},
                          {"cache_v_scale", o.scale_v, rows * 4, true},
                          {"weights", weights, rows * 4, kept_weights == weights},
                          {"lengths", lengths, (size_t)num_seqs * 4, false},
                          {"block_table", o.block_table, (size_t)num_seqs * o.max_blocks * 4, false}};
    s = check_disjoint(spans, sizeof spans / sizeof *spans);
    if (s != PA_OK) return s;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    const int sms = sm_count(dev, &s);
    if (s != PA_OK) return s;
    const StreamLock lock(dev, stream);
    Workspace* const ws = lock.ws;
    s = grow_workspace(*ws, stream, 0, 0);
    if (s != PA_OK) return s;
    void* aux = nullptr;
    if (!kept_index) {
        s = get_aux_scratch(ws, stream, index_bytes, &aux);
        if (s != PA_OK) return s;
    }
    pa::EvictArgs a;
    a.cache_k = cache_k;
    a.cache_v = cache_v;
    a.row_bytes = (int)row_bytes;
    a.part_bytes = 0;
    a.scale_k = o.kv_quant ? o.scale_k : nullptr;
    a.scale_v = o.kv_quant ? o.scale_v : nullptr;
    a.weights = weights;
    a.kept_weights = kept_weights;
    a.lengths = lengths;
    a.kept_lengths = kept_lengths;
    a.index = kept_index ? kept_index : static_cast<int*>(aux);
    a.hdr = static_cast<pa::WorkspaceHeader*>(ws->ptr);
    a.num_seqs = num_seqs;
    a.n_kv_heads = n_kv_heads;
    a.max_cache_len = max_cache_len;
    a.budget = budget;
    a.sinks = sink_tokens;
    a.recent = recent_tokens;
    a.block_table = o.block_table;
    a.block_log2 = log2_of(o.block_size);
    a.max_blocks = o.max_blocks;
    a.num_blocks = o.num_blocks;
    int launches = 0;
    e = pa::launch_evict(a, sms, &launches, stream);
    if (e != cudaSuccess) return cuda_fail(e, "eviction launch");
    g_last_launches = launches;
    return PA_OK;
} catch (...) {
    return caught();
}

}  // extern "C"
