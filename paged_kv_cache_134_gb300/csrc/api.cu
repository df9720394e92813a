// C ABI of the library: handle management, host-side validation, launches, error
// reporting and profiling.  Every computation happens in the kernels of append.cu,
// decode*.cu, rotary.cu, prefill.cu and blocks.cu.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "pkv_internal.h"

std::atomic<int64_t> g_pkv_launches{0};

namespace {
thread_local char g_msg[512] = "";

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_bytes(pkv_dtype d) { return d == PKV_INT4 ? 0 : d == PKV_FP8_E4M3 ? 1 : 2; }

bool supported_head_dim(int d) { return d == 64 || d == 128; }
bool supported_block_size(int b) { return b == 8 || b == 16 || b == 32; }
bool supported_group(int g) { return g == 1 || g == 2 || g == 4 || g == 8; }

// the argument checks the decode entry points share
int check_decode(const pkv_cache *c, const void *q, const int32_t *block_tables, int max_blocks_per_seq,
                 const int32_t *context_lens, int num_q_heads, float scale, const void *out) {
    if (num_q_heads <= 0 || num_q_heads % c->num_kv_heads)
        return pkv_fail(PKV_EINVAL, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                        c->num_kv_heads);
    if (!supported_group(num_q_heads / c->num_kv_heads))
        return pkv_fail(PKV_EUNSUPPORTED, "num_q_heads / num_kv_heads = %d not in {1, 2, 4, 8}",
                        num_q_heads / c->num_kv_heads);
    if (!q || !out || !context_lens || (!block_tables && max_blocks_per_seq > 0))
        return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(q) || !aligned16(out)) return pkv_fail(PKV_EINVAL, "q and out must be 16-byte aligned");
    if (!(scale == scale)) return pkv_fail(PKV_EINVAL, "scale is NaN");
    return PKV_OK;
}

bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// do n rows of na bytes, sa apart, share a byte with n rows of nb bytes, sb apart?  (Slices of one matrix do not; rows of
// different strides whose extents meet count as if they did.)
bool rows_overlap(const void *a, int64_t na, int64_t sa, const void *b, int64_t nb, int64_t sb, int64_t n) {
    if (na == 0 || nb == 0 || !overlap(a, (n - 1) * sa + na, b, (n - 1) * sb + nb)) return false;
    if (n == 1 || sa != sb || sa <= 0) return true;
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)), m = (d % sa + sa) % sa;
    return m < na || m + nb > sa;
}

int check_device(const pkv_cache *c) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return pkv_cuda_fail(e, "cudaGetDevice");
    if (dev != c->device) return pkv_fail(PKV_EINVAL, "cache lives on device %d but device %d is current", c->device, dev);
    return PKV_OK;
}

int ensure_workspace(pkv_cache *c, int64_t floats) {
    const int64_t bytes = floats * (int64_t)sizeof(float);
    if (bytes <= c->ws_bytes) return PKV_OK;
    if (c->ws) cudaFree(c->ws);
    c->ws = nullptr;
    c->ws_bytes = 0;
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(&c->ws), (size_t)bytes);
    if (e != cudaSuccess) {
        c->ws = nullptr;
        cudaGetLastError();
        return pkv_fail(PKV_ENOMEM, "decode workspace of %lld bytes: %s", (long long)bytes, cudaGetErrorString(e));
    }
    c->ws_bytes = bytes;
    return PKV_OK;
}
} // namespace

namespace {
// (an exception must not leave a C entry point)
bool room_for_one_more(std::vector<pkv_cache::StreamWs> &v) {
    try {
        v.reserve(v.size() + 1);
    } catch (...) {
        return false;
    }
    return true;
}

int64_t workspace_counters(const pkv_cache *c) { return (int64_t)1024 * c->num_kv_heads; } // rows of a launch

// Allocating and freeing are no part of a capture that this thread, or another, may be in.
struct RelaxedCapture {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
    ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// A workspace of `bytes` for partials and its zeroed counters, not tied to any stream's work: also while a
// stream is captured.
cudaError_t allocate_workspace(const pkv_cache *c, int64_t bytes, float **p) {
    RelaxedCapture relaxed;
    const int64_t tail = workspace_counters(c) * (int64_t)sizeof(int);
    cudaStream_t own = nullptr;
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(p), (size_t)(bytes + tail));
    if (e == cudaSuccess) {
        e = cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking);
        if (e == cudaSuccess) e = cudaMemsetAsync(reinterpret_cast<char *>(*p) + bytes, 0, (size_t)tail, own);
        if (e == cudaSuccess) e = cudaStreamSynchronize(own);
        if (own) cudaStreamDestroy(own);
        if (e != cudaSuccess) cudaFree(*p);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// One more workspace for the first stream or capture that needs one of at most its size.
int add_spare(pkv_cache *c, int64_t floats) {
    if (floats <= 0) return PKV_OK;
    pkv_cache::StreamWs b{0, 0, true, nullptr, (floats * (int64_t)sizeof(float) + 255) / 256 * 256};
    std::lock_guard<std::mutex> lk(c->ws_mu);
    if (!room_for_one_more(c->stream_ws)) return pkv_fail(PKV_ENOMEM, "out of host memory");
    cudaError_t e = allocate_workspace(c, b.bytes, &b.p);
    if (e != cudaSuccess)
        return pkv_fail(e == cudaErrorMemoryAllocation ? PKV_ENOMEM : PKV_ECUDA, "decode workspace of %lld bytes: %s",
                        (long long)b.bytes, cudaGetErrorString(e));
    c->stream_ws.push_back(b);
    return PKV_OK;
}
} // namespace

int pkv_stream_workspace(pkv_cache *c, cudaStream_t st, int64_t floats, PkvWorkspace *ws) {
    *ws = PkvWorkspace();
    if (floats <= 0) return PKV_OK;
    const int64_t bytes = (floats * (int64_t)sizeof(float) + 255) / 256 * 256;
    unsigned long long stream = 0, capture = 0;
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamGetCaptureInfo(st, &status, &capture);
    if (e == cudaSuccess && status == cudaStreamCaptureStatusActive) {
        stream = reinterpret_cast<uintptr_t>(st); // its id cannot be asked for now; the handle lives as long as the capture
    } else if (e == cudaSuccess) {
        capture = 0;
        e = cudaStreamGetId(st, &stream);
    }
    if (e != cudaSuccess) return pkv_cuda_fail(e, "stream query");
    auto use = [&](const pkv_cache::StreamWs &b) {
        ws->p = b.p;
        ws->floats = b.bytes / (int64_t)sizeof(float);
        ws->done = reinterpret_cast<int *>(reinterpret_cast<char *>(b.p) + b.bytes);
        ws->counters = workspace_counters(c);
        ws->clear = capture != 0;
        return PKV_OK;
    };
    auto &all = c->stream_ws;
    auto mine = [&](const pkv_cache::StreamWs &b) { return !b.spare && b.stream == stream && b.capture == capture; };
    int64_t most = 0;
    for (auto &b : all) {
        if (!mine(b)) continue;
        if (b.bytes >= bytes) return use(b);
        most = std::max(most, b.bytes);
    }
    // A spare one, or a new one.  What it replaces stays where it belongs to a capture (the graph's earlier nodes use it);
    // else it is freed once the stream's work, which alone uses it, is done.
    auto replace = [&](const pkv_cache::StreamWs &by) {
        if (capture || !most) return;
        RelaxedCapture relaxed;
        if (cudaStreamSynchronize(st) != cudaSuccess) {
            cudaGetLastError(); // (it stays for kv_cache_release_workspaces)
            return;
        }
        for (auto &b : all) {
            if (!mine(b) || b.p == by.p) continue;
            cudaFree(b.p);
            b.p = nullptr;
        }
        all.erase(std::remove_if(all.begin(), all.end(), [](const pkv_cache::StreamWs &b) { return !b.p; }), all.end());
    };
    pkv_cache::StreamWs *fit = nullptr; // the smallest: a decode leaves a larger one to the mass call it was reserved for
    for (auto &b : all)
        if (b.spare && b.bytes >= bytes && (!fit || b.bytes < fit->bytes)) fit = &b;
    if (fit) {
        fit->spare = false;
        fit->stream = stream;
        fit->capture = capture;
        const pkv_cache::StreamWs taken = *fit;
        replace(taken);
        return use(taken);
    }
    if (!room_for_one_more(all)) return pkv_fail(PKV_ENOMEM, "out of host memory");
    // half as much again as the last one, so that growing step by step is rare and what a capture outgrew stays little
    pkv_cache::StreamWs b{stream, capture, false, nullptr, std::max(bytes, (most + most / 2) / 256 * 256)};
    e = allocate_workspace(c, b.bytes, &b.p);
    if (e != cudaSuccess && b.bytes > bytes) {
        b.bytes = bytes;
        e = allocate_workspace(c, b.bytes, &b.p);
    }
    if (e != cudaSuccess)
        return pkv_fail(e == cudaErrorMemoryAllocation ? PKV_ENOMEM : PKV_ECUDA, "decode workspace of %lld bytes: %s",
                        (long long)bytes, cudaGetErrorString(e));
    all.push_back(b);
    replace(b);
    return use(b);
}

int pkv_fail(int status, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return status;
}

int pkv_cuda_fail(cudaError_t e, const char *what) {
    return pkv_fail(PKV_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

cudaError_t launch_decode_chunked(pkv_cache *c, DecodeLaunch d, cudaStream_t st) {
    const int G = d.num_q_heads / c->num_kv_heads;
    const int per = decode_seqs_per_launch(c, G);
    const int total = d.num_seqs;
    const int64_t row_bytes = (int64_t)d.num_q_heads * c->head_dim * 2; // q and out rows, 16-bit model dtype
    const char *q0 = static_cast<const char *>(d.q);
    char *out0 = static_cast<char *>(d.out);
    const int32_t *tables0 = d.tables, *lens0 = d.lens;
    CascadePrefixLaunch p;
    if (d.prefix) p = *d.prefix;
    for (int s0 = 0; s0 < total; s0 += per) {
        const int n = total - s0 < per ? total - s0 : per;
        d.q = q0 + s0 * row_bytes;
        d.out = out0 + s0 * row_bytes;
        d.tables = tables0 ? tables0 + (int64_t)s0 * d.max_blocks : nullptr;
        d.lens = lens0 + s0;
        d.num_seqs = n;
        if (d.prefix) {
            // the launch's own rows: its queries, its tables (every one names the shared prefix), and the
            // (m, l) half of the workspace right after its n * Hq * max_splits partial rows
            p.q = d.q;
            p.tables = d.tables;
            p.num_seqs = n;
            p.ws_ml = p.ws_o + (int64_t)n * d.num_q_heads * d.max_splits * c->head_dim;
            cudaError_t e = launch_cascade_prefix(c, p, st, 1);
            if (e != cudaSuccess) return e;
            d.prefix = &p;
        }
        cudaError_t e = launch_decode(c, d, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

PkvTimer::PkvTimer(pkv_cache *c_, int kind_, cudaStream_t st_) : c(c_), kind(kind_), st(st_) {
    if (!c || !c->profiling || !(c->profile_kinds & (1u << kind))) return;
    std::lock_guard<std::mutex> lk(c->mu);
    // sampled profiling: the launches in between run without events, so that their overlap with
    // the neighbouring kernels (programmatic dependent launch) is left as it is
    if (c->profile_seen[kind]++ % c->profile_every != 0) return;
    for (cudaEvent_t *ev : {&a, &b}) {
        if (!c->event_pool.empty()) {
            *ev = c->event_pool.back();
            c->event_pool.pop_back();
        } else if (cudaEventCreate(ev) != cudaSuccess) {
            *ev = nullptr;
        }
    }
    if (a) cudaEventRecord(a, st);
}

PkvTimer::~PkvTimer() {
    if (!c || !c->profiling || !a || !b) return;
    cudaEventRecord(b, st);
    std::lock_guard<std::mutex> lk(c->mu);
    c->events.push_back({kind, a, b});
}

extern "C" {

const char *pkv_last_error(void) { return g_msg; }

int64_t pkv_kernel_launches(void) { return g_pkv_launches.load(); }

int kv_cache_create(int64_t num_blocks, int block_size, int num_kv_heads, int head_dim, pkv_dtype kv_dtype,
                    pkv_dtype model_dtype, pkv_cache_t *out) {
    if (!out) return pkv_fail(PKV_EINVAL, "out is NULL");
    if (num_blocks <= 0 || num_kv_heads <= 0) return pkv_fail(PKV_EINVAL, "num_blocks and num_kv_heads must be > 0");
    if (kv_dtype < PKV_F16 || kv_dtype > PKV_INT4 || model_dtype < PKV_F16 || model_dtype > PKV_BF16)
        return pkv_fail(PKV_EINVAL, "bad dtype (kv %d, model %d)", (int)kv_dtype, (int)model_dtype);
    if (kv_dtype != PKV_FP8_E4M3 && kv_dtype != PKV_INT4 && kv_dtype != model_dtype)
        return pkv_fail(PKV_EINVAL, "a 16-bit cache must use its own dtype as model dtype");
    if (!supported_head_dim(head_dim)) return pkv_fail(PKV_EUNSUPPORTED, "head_dim %d not in {64, 128}", head_dim);
    if (!supported_block_size(block_size))
        return pkv_fail(PKV_EUNSUPPORTED, "block_size %d not in {8, 16, 32}", block_size);
    pkv_cache *c = new pkv_cache();
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device);
    if (e != cudaSuccess) {
        delete c;
        return pkv_cuda_fail(e, "device query");
    }
    c->num_blocks = num_blocks;
    c->block_size = block_size;
    c->num_kv_heads = num_kv_heads;
    c->head_dim = head_dim;
    c->kv_dtype = kv_dtype;
    c->model_dtype = model_dtype;
    c->elem_bytes = elem_bytes(kv_dtype); // 4-bit caches: 0, their strides are pkv_row_strides'
    c->tile_bytes = (int64_t)block_size * head_dim * c->elem_bytes;
    {
        int64_t block, head, v;
        pkv_row_strides(c, &block, &head, &v);
        c->pool_bytes = num_blocks * block;
    }
    e = cudaMalloc(&c->pool, (size_t)c->pool_bytes);
    if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void **>(&c->err), 16);
    if (e == cudaSuccess && kv_dtype == PKV_FP8_E4M3) {
        e = cudaMalloc(reinterpret_cast<void **>(&c->k_scale), sizeof(float) * num_kv_heads);
        if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void **>(&c->v_scale), sizeof(float) * num_kv_heads);
    }
    if (e == cudaSuccess) e = cudaMemset(c->pool, 0, (size_t)c->pool_bytes);
    if (e == cudaSuccess) e = cudaMemset(c->err, 0, 16);
    if (e == cudaSuccess) {
        // the no-alloc decode's fixed scratch is made resident on this device now, while the cache is
        // created, so that paged_decode_attention_noalloc never has to bring it in later
        if (int r = pkv_noalloc_scratch_prepare(c->device)) {
            kv_cache_destroy(c);
            return r;
        }
    }
    if (e == cudaSuccess && c->k_scale) {
        // default scale 1.0f (0x3F800000)
        float ones[256];
        for (float &x : ones) x = 1.0f;
        for (int h = 0; h < num_kv_heads && e == cudaSuccess; h += 256) {
            const int n = num_kv_heads - h < 256 ? num_kv_heads - h : 256;
            e = cudaMemcpy(c->k_scale + h, ones, n * sizeof(float), cudaMemcpyHostToDevice);
            if (e == cudaSuccess) e = cudaMemcpy(c->v_scale + h, ones, n * sizeof(float), cudaMemcpyHostToDevice);
        }
    }
    if (e != cudaSuccess) {
        const int st = (e == cudaErrorMemoryAllocation) ? PKV_ENOMEM : PKV_ECUDA;
        const long long bytes = c->pool_bytes;
        cudaGetLastError();
        kv_cache_destroy(c);
        return pkv_fail(st, "kv_cache_create (%lld bytes): %s", bytes, cudaGetErrorString(e));
    }
    *out = c;
    return PKV_OK;
}

int kv_cache_destroy(pkv_cache_t c) {
    if (!c) return PKV_OK;
    cudaDeviceSynchronize();
    if (c->pool) cudaFree(c->pool);
    if (c->err) cudaFree(c->err);
    if (c->k_scale) cudaFree(c->k_scale);
    if (c->v_scale) cudaFree(c->v_scale);
    if (c->ws) cudaFree(c->ws);
    if (c->plan) cudaFree(c->plan);
    for (auto &b : c->stream_ws) cudaFree(b.p);
    for (auto &ev : c->events) {
        cudaEventDestroy(ev.a);
        cudaEventDestroy(ev.b);
    }
    for (auto ev : c->event_pool) cudaEventDestroy(ev);
    delete c;
    return PKV_OK;
}

int kv_cache_set_scales(pkv_cache_t c, const float *k_scale, const float *v_scale, void *stream) {
    PKV_RANGE("kv_cache_set_scales");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (c->kv_dtype != PKV_FP8_E4M3) return pkv_fail(PKV_EINVAL, "scales apply to FP8 caches only");
    if (!k_scale || !v_scale) return pkv_fail(PKV_EINVAL, "scale pointer is NULL");
    if (int r = check_device(c)) return r;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t n = sizeof(float) * c->num_kv_heads;
    cudaError_t e = cudaMemcpyAsync(c->k_scale, k_scale, n, cudaMemcpyDeviceToDevice, st);
    if (e == cudaSuccess) e = cudaMemcpyAsync(c->v_scale, v_scale, n, cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return pkv_cuda_fail(e, "kv_cache_set_scales");
    return PKV_OK;
}

int kv_cache_view(pkv_cache_t c, void **base, int64_t strides_elems[5], int64_t *num_bytes) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    const int64_t tile = (int64_t)c->block_size * c->head_dim;
    if (base) *base = c->pool;
    if (strides_elems) {
        int64_t block, head, v;
        pkv_row_strides(c, &block, &head, &v);
        const bool i4 = c->kv_dtype == PKV_INT4; // elements are nibbles: two a byte
        strides_elems[0] = i4 ? 2 * block : 2 * c->num_kv_heads * tile;
        strides_elems[1] = i4 ? 0 : c->num_kv_heads * tile;
        strides_elems[2] = i4 ? 2 * head : tile;
        strides_elems[3] = i4 ? 0 : c->head_dim;
        strides_elems[4] = 1;
    }
    if (num_bytes) *num_bytes = c->pool_bytes;
    return PKV_OK;
}

int kv_cache_reserve(pkv_cache_t c, int max_seqs, int max_q_heads, int max_blocks_per_seq) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (max_seqs < 0 || max_q_heads < 0 || max_blocks_per_seq < 0) return pkv_fail(PKV_EINVAL, "negative size");
    if (int r = check_device(c)) return r;
    if (c->kv_dtype == PKV_INT4)
        return add_spare(c, decode_mma_workspace_floats(c, max_seqs, max_q_heads, max_blocks_per_seq, -1));
    const int bps = decode_split_blocks(c);
    const int max_splits = (max_blocks_per_seq + bps - 1) / bps;
    // consecutive launches of one call share the workspace: one launch's rows are enough
    int rows = max_seqs;
    if (max_q_heads > 0 && max_q_heads % c->num_kv_heads == 0 && supported_group(max_q_heads / c->num_kv_heads))
        rows = std::min(rows, decode_seqs_per_launch(c, max_q_heads / c->num_kv_heads));
    return ensure_workspace(c, decode_workspace_floats(c, rows, max_q_heads, max_splits));
}

int kv_cache_reserve_mass(pkv_cache_t c, int max_seqs, int max_q_heads, int max_blocks_per_seq, int64_t max_mass_len) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (max_seqs < 0 || max_q_heads < 0 || max_blocks_per_seq < 0 || max_mass_len < 0)
        return pkv_fail(PKV_EINVAL, "negative size");
    if (int r = check_device(c)) return r;
    return add_spare(c, decode_mma_workspace_floats(c, max_seqs, max_q_heads, max_blocks_per_seq, max_mass_len));
}

int kv_cache_reserve_window(pkv_cache_t c, int max_seqs, int max_q_heads, int max_blocks_per_seq, int max_window,
                            int max_sinks) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (max_seqs < 0 || max_q_heads < 0 || max_blocks_per_seq < 0 || max_sinks < 0)
        return pkv_fail(PKV_EINVAL, "negative size");
    if (max_window < 1) return pkv_fail(PKV_EINVAL, "window %d: window >= 1", max_window);
    if (max_q_heads % c->num_kv_heads || (max_q_heads > 0 && !supported_group(max_q_heads / c->num_kv_heads)))
        return pkv_fail(PKV_EUNSUPPORTED, "num_q_heads / num_kv_heads not in {1, 2, 4, 8}");
    if (int r = check_device(c)) return r;
    return add_spare(c, decode_window_workspace_floats(c, max_seqs, max_q_heads, max_blocks_per_seq, max_window, max_sinks));
}

int kv_cache_reserve_chunk(pkv_cache_t c, int max_seqs, int64_t max_tokens, int max_seqlen, int max_q_heads,
                           int max_blocks_per_seq) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (max_seqs < 0 || max_tokens < 0 || max_seqlen < 0 || max_q_heads < 0 || max_blocks_per_seq < 0)
        return pkv_fail(PKV_EINVAL, "negative size");
    if (max_q_heads % c->num_kv_heads || (max_q_heads > 0 && !supported_group(max_q_heads / c->num_kv_heads)))
        return pkv_fail(PKV_EUNSUPPORTED, "num_q_heads / num_kv_heads not in {1, 2, 4, 8}");
    if (int r = check_device(c)) return r;
    if (!max_seqs || !max_tokens || !max_seqlen || !max_q_heads) return PKV_OK;
    max_seqlen = (int)std::min<int64_t>(max_seqlen, max_tokens);
    return add_spare(c, chunk_workspace_floats(c, max_seqs, max_tokens, max_seqlen, max_q_heads, max_blocks_per_seq));
}

int kv_cache_release_workspaces(pkv_cache_t c, int graphs) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (int r = check_device(c)) return r;
    std::lock_guard<std::mutex> lk(c->ws_mu);
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return pkv_cuda_fail(e, "cudaDeviceSynchronize");
    for (auto &b : c->stream_ws) {
        if (b.capture && !graphs) continue;
        cudaFree(b.p);
        b.p = nullptr;
    }
    auto &all = c->stream_ws;
    all.erase(std::remove_if(all.begin(), all.end(), [](const pkv_cache::StreamWs &b) { return !b.p; }), all.end());
    return PKV_OK;
}

int kv_cache_check_error(pkv_cache_t c, int *device_code) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return pkv_cuda_fail(e, "cudaDeviceSynchronize");
    unsigned int v = 0;
    e = cudaMemcpy(&v, c->err, sizeof v, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(c->err, 0, sizeof v);
    if (e != cudaSuccess) return pkv_cuda_fail(e, "reading the device error word");
    if (device_code) *device_code = static_cast<int>(v);
    if (v) return pkv_fail(PKV_EDEVICE, "device error bits 0x%x", v);
    return PKV_OK;
}

int paged_slot_mapping(const int32_t *block_tables, int num_rows, int max_blocks_per_seq, const int32_t *seq_ids,
                       const int32_t *positions, int64_t num_tokens, int block_size, int64_t *slot_mapping,
                       void *stream) {
    PKV_RANGE("paged_slot_mapping");
    if (num_tokens < 0 || num_rows < 0 || max_blocks_per_seq < 0) return pkv_fail(PKV_EINVAL, "negative size");
    if (block_size <= 0) return pkv_fail(PKV_EINVAL, "block_size must be > 0");
    if (num_tokens == 0) return PKV_OK;
    if (!seq_ids || !positions || !slot_mapping || (!block_tables && num_rows > 0 && max_blocks_per_seq > 0))
        return pkv_fail(PKV_EINVAL, "NULL pointer");
    cudaError_t e = launch_slot_mapping(block_tables, num_rows, max_blocks_per_seq, seq_ids, positions, num_tokens,
                                        block_size, slot_mapping, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "slot mapping launch");
    return PKV_OK;
}

int paged_kv_append(pkv_cache_t c, const void *k, const void *v, const int64_t *slot_mapping, int64_t num_tokens,
                    void *stream) {
    PKV_RANGE("paged_kv_append");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_tokens < 0) return pkv_fail(PKV_EINVAL, "num_tokens < 0");
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(k) || !aligned16(v)) return pkv_fail(PKV_EINVAL, "k and v must be 16-byte aligned");
    if (int r = check_device(c)) return r;
    cudaError_t e = launch_append(c, k, v, slot_mapping, num_tokens, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "append launch");
    return PKV_OK;
}

int paged_kv_append_at(pkv_cache_t c, const void *k, const void *v, const int32_t *block_tables, int num_rows,
                       int max_blocks_per_seq, const int32_t *seq_ids, const int32_t *positions, int64_t num_tokens,
                       int64_t *slot_mapping, void *stream) {
    PKV_RANGE("paged_kv_append_at");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_tokens < 0 || num_rows < 0 || max_blocks_per_seq < 0) return pkv_fail(PKV_EINVAL, "negative size");
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !seq_ids || !positions || (!block_tables && num_rows > 0 && max_blocks_per_seq > 0))
        return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(k) || !aligned16(v)) return pkv_fail(PKV_EINVAL, "k and v must be 16-byte aligned");
    if (int r = check_device(c)) return r;
    cudaError_t e = launch_append_at(c, k, v, block_tables, num_rows, max_blocks_per_seq, seq_ids, positions,
                                     num_tokens, slot_mapping, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "append launch");
    return PKV_OK;
}

int paged_kv_append_rotary(pkv_cache_t c, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                           const void *v, int64_t v_stride, int num_q_heads, const int32_t *block_tables, int num_rows,
                           int max_blocks_per_seq, const int32_t *seq_ids, const int32_t *positions,
                           const int32_t *rotary_positions, int64_t num_tokens, const pkv_rotary_t *rotary,
                           const void *q_weight, const void *k_weight, float eps, void *q_out, int64_t q_out_stride,
                           int64_t *slot_mapping, void *stream) {
    PKV_RANGE("paged_kv_append_rotary");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_tokens < 0 || num_rows < 0 || max_blocks_per_seq < 0 || num_q_heads < 0)
        return pkv_fail(PKV_EINVAL, "negative size");
    if (num_q_heads > 4096 || c->num_kv_heads > 4096) return pkv_fail(PKV_EUNSUPPORTED, "more than 4096 heads");
    if (!rotary || !rotary->inv_freq) return pkv_fail(PKV_EINVAL, "rotary is NULL");
    if (rotary->rotary_dim < 16 || rotary->rotary_dim > c->head_dim || rotary->rotary_dim % 16)
        return pkv_fail(PKV_EUNSUPPORTED, "rotary_dim %d is not a multiple of 16 in [16, head_dim %d]",
                        rotary->rotary_dim, c->head_dim);
    if (!std::isfinite(rotary->gain)) return pkv_fail(PKV_EINVAL, "gain is not finite");
    for (int i = 0; i < rotary->rotary_dim / 2; ++i)
        if (!std::isfinite(rotary->inv_freq[i])) return pkv_fail(PKV_EINVAL, "inv_freq[%d] is not finite", i);
    if (!(eps >= 0.f)) return pkv_fail(PKV_EINVAL, "eps must be >= 0");
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !seq_ids || !positions || (!block_tables && num_rows > 0 && max_blocks_per_seq > 0) ||
        (num_q_heads > 0 && (!q || !q_out)))
        return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(k) || !aligned16(v) || (num_q_heads > 0 && (!aligned16(q) || !aligned16(q_out))) ||
        !aligned16(q_weight) || !aligned16(k_weight))
        return pkv_fail(PKV_EINVAL, "q, k, v, q_out and the weights must be 16-byte aligned");
    if ((k_stride | v_stride) % 8 || (num_q_heads > 0 && (q_stride | q_out_stride) % 8))
        return pkv_fail(PKV_EINVAL, "strides must be multiples of 8 elements");
    if (num_q_heads > 0 && num_tokens > 1 && q_out_stride < (int64_t)num_q_heads * c->head_dim)
        return pkv_fail(PKV_EINVAL, "q_out rows overlap");
    if (num_q_heads > 0) {
        const int64_t wq = (int64_t)num_q_heads * c->head_dim * 2, wk = (int64_t)c->num_kv_heads * c->head_dim * 2;
        const int64_t so = q_out_stride * 2;
        if ((!(q_out == q && (q_stride == q_out_stride || num_tokens == 1)) &&
             rows_overlap(q_out, wq, so, q, wq, q_stride * 2, num_tokens)) ||
            rows_overlap(q_out, wq, so, k, wk, k_stride * 2, num_tokens) ||
            rows_overlap(q_out, wq, so, v, wk, v_stride * 2, num_tokens))
            return pkv_fail(PKV_EINVAL, "q_out overlaps the inputs and is not q with q's stride");
    }
    if (int r = check_device(c)) return r;
    RotaryLaunch r{q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, num_q_heads, block_tables, num_rows,
                   max_blocks_per_seq, seq_ids, positions, rotary_positions, num_tokens, rotary,
                   num_q_heads > 0 ? q_weight : nullptr, k_weight, eps, slot_mapping};
    cudaError_t e = launch_append_rotary(c, r, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "append launch");
    return PKV_OK;
}

int paged_kv_gather(pkv_cache_t c, const int64_t *slot_mapping, int64_t num_tokens, void *k, void *v, void *stream) {
    PKV_RANGE("paged_kv_gather");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_tokens < 0) return pkv_fail(PKV_EINVAL, "num_tokens < 0");
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(k) || !aligned16(v)) return pkv_fail(PKV_EINVAL, "k and v must be 16-byte aligned");
    if (int r = check_device(c)) return r;
    cudaError_t e = launch_gather(c, slot_mapping, num_tokens, k, v, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "gather launch");
    return PKV_OK;
}

int paged_decode_attention_mass(const void *q, pkv_cache_t c, const int32_t *block_tables, int max_blocks_per_seq,
                                const int32_t *context_lens, int num_seqs, int num_q_heads, float scale, float decay,
                                float *attn_mass, int64_t mass_len, void *out, void *stream) {
    PKV_RANGE("paged_decode_attention_mass");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_seqs < 0 || max_blocks_per_seq < 0 || mass_len < 0) return pkv_fail(PKV_EINVAL, "negative size");
    if (num_seqs == 0) return PKV_OK;
    if (int r = check_decode(c, q, block_tables, max_blocks_per_seq, context_lens, num_q_heads, scale, out)) return r;
    if (!attn_mass && mass_len > 0) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!(decay >= 0.f && decay <= 1.f)) return pkv_fail(PKV_EINVAL, "decay must be in [0, 1]");
    if (int r = check_device(c)) return r;
    MmaDecodeLaunch d{q, out, block_tables, context_lens, max_blocks_per_seq, num_seqs, num_q_heads, scale,
                      attn_mass, mass_len, decay};
    return decode_mma_entry(c, d, nullptr, static_cast<cudaStream_t>(stream));
}

int paged_kv_evict(pkv_cache_t c, const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                   int num_seqs, const float *attn_mass, int64_t mass_len, int budget, int recent,
                   const int32_t *dst_block_tables, int max_dst_blocks_per_seq, int32_t *kept, int32_t *new_lens,
                   float *new_mass, int64_t new_mass_len, void *stream) {
    PKV_RANGE("paged_kv_evict");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_seqs < 0 || max_blocks_per_seq < 0 || max_dst_blocks_per_seq < 0 || mass_len < 0 || new_mass_len < 0)
        return pkv_fail(PKV_EINVAL, "negative size");
    if (budget < 1) return pkv_fail(PKV_EINVAL, "budget %d is less than 1", budget);
    if (recent < 0 || recent > budget) return pkv_fail(PKV_EINVAL, "recent %d is not in [0, budget %d]", recent, budget);
    if (num_seqs == 0) return PKV_OK;
    const int64_t cap = std::min<int64_t>(mass_len, (int64_t)max_blocks_per_seq * c->block_size);
    const int64_t most = std::min<int64_t>(cap, budget);
    if (cap > 1 << 30 || budget > 1 << 30)
        return pkv_fail(PKV_EUNSUPPORTED, "sequences and budgets of more than 2^30 tokens");
    if ((int64_t)max_dst_blocks_per_seq * c->block_size < most)
        return pkv_fail(PKV_EINVAL, "destination tables of %d blocks cannot hold %lld tokens", max_dst_blocks_per_seq,
                        (long long)most);
    if (new_mass_len < most)
        return pkv_fail(PKV_EINVAL, "new_mass rows of %lld cannot hold %lld tokens", (long long)new_mass_len,
                        (long long)most);
    if ((int64_t)num_seqs * c->num_kv_heads > 0x7FFFFFFF) return pkv_fail(PKV_EUNSUPPORTED, "too many rows");
    if (!context_lens || !kept || !new_lens || (most > 0 && (!block_tables || !attn_mass || !dst_block_tables)) ||
        (!new_mass && new_mass_len > 0))
        return pkv_fail(PKV_EINVAL, "NULL pointer");
    const int64_t rows = (int64_t)num_seqs * c->num_kv_heads;
    if (overlap(attn_mass, rows * mass_len * 4, new_mass, rows * new_mass_len * 4))
        return pkv_fail(PKV_EINVAL, "new_mass overlaps attn_mass");
    if (overlap(context_lens, (int64_t)num_seqs * 4, new_lens, (int64_t)num_seqs * 4))
        return pkv_fail(PKV_EINVAL, "new_lens overlaps context_lens");
    if (int r = check_device(c)) return r;
    EvictLaunch v{block_tables, dst_block_tables, context_lens, attn_mass, kept, new_lens, new_mass, mass_len,
                  new_mass_len, max_blocks_per_seq, max_dst_blocks_per_seq, num_seqs, budget, recent};
    cudaError_t e = launch_evict(c, v, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "eviction launch");
    return PKV_OK;
}

int paged_decode_attention(const void *q, pkv_cache_t c, const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int num_seqs, int num_q_heads, float scale, void *out,
                           void *stream) {
    PKV_RANGE("paged_decode_attention");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_seqs < 0 || max_blocks_per_seq < 0) return pkv_fail(PKV_EINVAL, "negative size");
    if (num_seqs == 0) return PKV_OK;
    if (int r = check_decode(c, q, block_tables, max_blocks_per_seq, context_lens, num_q_heads, scale, out)) return r;
    if (int r = check_device(c)) return r;
    if (c->kv_dtype == PKV_INT4) {
        MmaDecodeLaunch d{q, out, block_tables, context_lens, max_blocks_per_seq, num_seqs, num_q_heads, scale,
                          nullptr, -1, 1.f};
        return decode_mma_entry(c, d, nullptr, static_cast<cudaStream_t>(stream));
    }
    // a batch larger than one launch takes runs in consecutive launches that share the workspace
    const int per_launch = std::min(num_seqs, decode_seqs_per_launch(c, num_q_heads / c->num_kv_heads));
    DecodeLaunch d;
    d.q = q;
    d.out = out;
    d.tables = block_tables;
    d.lens = context_lens;
    d.max_blocks = max_blocks_per_seq;
    d.num_seqs = num_seqs;
    d.num_q_heads = num_q_heads;
    d.scale = scale;
    d.split_blocks = decode_split_blocks(c);
    d.max_splits = (max_blocks_per_seq + d.split_blocks - 1) / d.split_blocks;
    const int64_t ws = decode_workspace_floats(c, per_launch, num_q_heads, d.max_splits);
    if (int r = ensure_workspace(c, ws)) return r;
    d.ws_o = ws ? c->ws : nullptr;
    d.ws_ml = nullptr;
    cudaError_t e = launch_decode_chunked(c, d, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "decode launch");
    return PKV_OK;
}

int paged_decode_attention_window(const void *q, pkv_cache_t c, const int32_t *block_tables, int max_blocks_per_seq,
                                  const int32_t *context_lens, int num_seqs, int num_q_heads, float scale, int window,
                                  int sinks, void *out, void *stream) {
    PKV_RANGE("paged_decode_attention_window");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_seqs < 0 || max_blocks_per_seq < 0) return pkv_fail(PKV_EINVAL, "negative size");
    if (window < 1 || sinks < 0) return pkv_fail(PKV_EINVAL, "window %d and sinks %d: window >= 1, sinks >= 0", window, sinks);
    if (num_seqs == 0) return PKV_OK;
    if (int r = check_decode(c, q, block_tables, max_blocks_per_seq, context_lens, num_q_heads, scale, out)) return r;
    if (int r = check_device(c)) return r;
    sinks = std::min(sinks, 1 << 30); // (a block's rounding stays within 32 bits)
    MmaDecodeLaunch d{q, out, block_tables, context_lens, max_blocks_per_seq, num_seqs, num_q_heads, scale, nullptr, -1, 1.f,
                      window, sinks};
    return decode_mma_entry(c, d, nullptr, static_cast<cudaStream_t>(stream));
}

int paged_chunk_attention(const void *q, pkv_cache_t c, const int32_t *block_tables, int max_blocks_per_seq,
                          const int32_t *context_lens, const int32_t *cu_seqlens, int num_seqs, int max_seqlen,
                          int64_t total_tokens, int num_q_heads, float scale, int window, int sinks, void *out,
                          void *stream) {
    PKV_RANGE("paged_chunk_attention");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_seqs < 0 || max_seqlen < 0 || max_blocks_per_seq < 0 || total_tokens < 0)
        return pkv_fail(PKV_EINVAL, "negative size");
    if (window < 0 || sinks < 0 || (window == 0 && sinks > 0))
        return pkv_fail(PKV_EINVAL, "window %d and sinks %d: window >= 0 (0: none), sinks >= 0 and 0 without a window",
                        window, sinks);
    if (c->kv_dtype == PKV_INT4) return pkv_fail(PKV_EUNSUPPORTED, "the chunk attention does not read 4-bit caches");
    if (!(scale > 0.f) || !std::isfinite(scale)) return pkv_fail(PKV_EINVAL, "scale must be finite and > 0");
    if (num_seqs == 0 || max_seqlen == 0 || total_tokens == 0) return PKV_OK;
    max_seqlen = (int)std::min<int64_t>(max_seqlen, total_tokens); // (no piece of the call is longer)
    if (window >= (int64_t)max_blocks_per_seq * c->block_size) window = sinks = 0; // (no row has so many tokens before it)
    if (int r = check_decode(c, q, block_tables, max_blocks_per_seq, context_lens, num_q_heads, scale, out)) return r;
    if (!cu_seqlens) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (overlap(q, total_tokens * num_q_heads * c->head_dim * 2, out, total_tokens * num_q_heads * c->head_dim * 2))
        return pkv_fail(PKV_EINVAL, "out overlaps q");
    if (int r = check_device(c)) return r;
    ChunkLaunch p{q, out, block_tables, context_lens, cu_seqlens, max_blocks_per_seq, num_seqs, max_seqlen,
                  total_tokens, num_q_heads, window, std::min(sinks, 1 << 30), scale};
    return chunk_entry(c, p, static_cast<cudaStream_t>(stream));
}

static int prefill_entry(const void *q, const void *k, const void *v, const int32_t *cu_seqlens,
                         const int32_t *context_lens, int num_seqs, int max_seqlen, int64_t total_tokens,
                         const int32_t *block_tables, int max_blocks_per_seq, pkv_cache_t c, int num_q_heads,
                         float scale, void *out, void *stream) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_seqs < 0 || max_seqlen < 0 || max_blocks_per_seq < 0 || total_tokens < 0)
        return pkv_fail(PKV_EINVAL, "negative size");
    if (total_tokens > 0x7FFFFFFF) return pkv_fail(PKV_EUNSUPPORTED, "more than 2^31 - 1 packed tokens");
    if (num_seqs == 0 || max_seqlen == 0 || total_tokens == 0) return PKV_OK;
    if (num_q_heads <= 0 || num_q_heads % c->num_kv_heads)
        return pkv_fail(PKV_EINVAL, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                        c->num_kv_heads);
    if (!supported_group(num_q_heads / c->num_kv_heads))
        return pkv_fail(PKV_EUNSUPPORTED, "num_q_heads / num_kv_heads = %d not in {1, 2, 4, 8}",
                        num_q_heads / c->num_kv_heads);
    if (!q || !k || !v || !out || !cu_seqlens || !block_tables) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return pkv_fail(PKV_EINVAL, "q, k, v and out must be 16-byte aligned");
    if (int r = check_device(c)) return r;
    PrefillLaunch p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = out;
    p.cu = cu_seqlens;
    p.ctx = context_lens;
    p.tables = block_tables;
    p.num_seqs = num_seqs;
    p.max_seqlen = max_seqlen;
    p.total_tokens = total_tokens;
    p.max_blocks = max_blocks_per_seq;
    p.num_q_heads = num_q_heads;
    p.scale = scale;
    cudaError_t e = launch_prefill(c, p, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorNotSupported) return pkv_fail(PKV_EUNSUPPORTED, "prefill shape not supported");
    if (e != cudaSuccess) return pkv_cuda_fail(e, "prefill launch");
    return PKV_OK;
}

int paged_decode_attention_cascade(const void *q, pkv_cache_t c, const int32_t *block_tables, int max_blocks_per_seq,
                                   const int32_t *context_lens, int num_seqs, int num_q_heads, int shared_prefix_len,
                                   float scale, void *out, void *stream) {
    PKV_RANGE("paged_decode_attention_cascade");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (shared_prefix_len < 0 || shared_prefix_len % c->block_size)
        return pkv_fail(PKV_EINVAL, "shared_prefix_len %d is not a non-negative multiple of block_size %d",
                        shared_prefix_len, c->block_size);
    if (shared_prefix_len == 0)
        return paged_decode_attention(q, c, block_tables, max_blocks_per_seq, context_lens, num_seqs, num_q_heads,
                                      scale, out, stream);
    if (c->kv_dtype == PKV_INT4)
        return pkv_fail(PKV_EUNSUPPORTED, "the cascade's prefix phase does not read 4-bit caches");
    if (num_seqs < 0 || max_blocks_per_seq < 0) return pkv_fail(PKV_EINVAL, "negative size");
    if (num_seqs == 0) return PKV_OK;
    if ((int64_t)shared_prefix_len > (int64_t)max_blocks_per_seq * c->block_size)
        return pkv_fail(PKV_EINVAL, "shared prefix longer than the tables");
    if (num_q_heads <= 0 || num_q_heads % c->num_kv_heads)
        return pkv_fail(PKV_EINVAL, "num_q_heads %d is not a multiple of num_kv_heads %d", num_q_heads,
                        c->num_kv_heads);
    if (!supported_group(num_q_heads / c->num_kv_heads))
        return pkv_fail(PKV_EUNSUPPORTED, "num_q_heads / num_kv_heads = %d not in {1, 2, 4, 8}",
                        num_q_heads / c->num_kv_heads);
    if (!q || !out || !context_lens || !block_tables) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(q) || !aligned16(out)) return pkv_fail(PKV_EINVAL, "q and out must be 16-byte aligned");
    if (!(scale == scale)) return pkv_fail(PKV_EINVAL, "scale is NaN");
    if (int r = check_device(c)) return r;
    // a batch larger than one launch takes runs in consecutive launches (each reads the prefix once)
    const int per_launch = std::min(num_seqs, decode_seqs_per_launch(c, num_q_heads / c->num_kv_heads));
    const int split_tokens = cascade_split_tokens(c, per_launch, num_q_heads, shared_prefix_len);
    const int nps = (shared_prefix_len + split_tokens - 1) / split_tokens;
    const int pb = shared_prefix_len / c->block_size;
    DecodeLaunch d;
    d.q = q;
    d.out = out;
    d.tables = block_tables;
    d.lens = context_lens;
    d.max_blocks = max_blocks_per_seq;
    d.num_seqs = num_seqs;
    d.num_q_heads = num_q_heads;
    d.scale = scale;
    d.split_blocks = cascade_suffix_split_blocks(c);
    d.max_splits = nps + (max_blocks_per_seq - pb + d.split_blocks - 1) / d.split_blocks;
    d.start_block = pb;
    d.slot0 = nps;
    const int64_t rows = (int64_t)per_launch * num_q_heads * d.max_splits;
    if (int r = ensure_workspace(c, rows * (c->head_dim + 2))) return r;
    d.ws_o = c->ws;
    d.ws_ml = nullptr;
    CascadePrefixLaunch p;
    p.q = q;
    p.tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.prefix_tokens = shared_prefix_len;
    p.split_tokens = split_tokens;
    p.max_splits = d.max_splits;
    p.scale = scale;
    p.ws_o = c->ws;
    p.ws_ml = c->ws + rows * c->head_dim;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // launches, per run of sequences: the prefix phase's plan, the suffix decode, the prefix kernel,
    // the merge
    d.prefix = &p;
    cudaError_t e = launch_decode_chunked(c, d, st);
    if (e == cudaErrorNotSupported) return pkv_fail(PKV_EUNSUPPORTED, "cascade shape not supported");
    if (e != cudaSuccess) return pkv_cuda_fail(e, "cascade decode launch");
    return PKV_OK;
}

int packed_prefill_attention(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int num_seqs,
                             int max_seqlen, int64_t total_tokens, const int32_t *block_tables,
                             int max_blocks_per_seq, pkv_cache_t c, int num_q_heads, float scale, void *out,
                             void *stream) {
    PKV_RANGE("packed_prefill_attention");
    return prefill_entry(q, k, v, cu_seqlens, nullptr, num_seqs, max_seqlen, total_tokens, block_tables,
                         max_blocks_per_seq, c, num_q_heads, scale, out, stream);
}

int paged_prefill_attention(const void *q, const void *k, const void *v, const int32_t *cu_seqlens,
                            const int32_t *context_lens, int num_seqs, int max_seqlen, int64_t total_tokens,
                            const int32_t *block_tables, int max_blocks_per_seq, pkv_cache_t c, int num_q_heads,
                            float scale, void *out, void *stream) {
    PKV_RANGE("paged_prefill_attention");
    if (!context_lens && num_seqs > 0) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (c && c->kv_dtype == PKV_INT4)
        return pkv_fail(PKV_EUNSUPPORTED, "the prefill over a cached prefix does not read 4-bit caches");
    return prefill_entry(q, k, v, cu_seqlens, context_lens, num_seqs, max_seqlen, total_tokens, block_tables,
                         max_blocks_per_seq, c, num_q_heads, scale, out, stream);
}

int paged_block_copy(pkv_cache_t c, const int32_t *src_blocks, const int32_t *dst_blocks, int64_t num_pairs,
                     void *stream) {
    PKV_RANGE("paged_block_copy");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_pairs < 0) return pkv_fail(PKV_EINVAL, "num_pairs < 0");
    if (num_pairs == 0) return PKV_OK;
    if (!src_blocks || !dst_blocks) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (int r = check_device(c)) return r;
    cudaError_t e = launch_copy_blocks(c, c->pool, src_blocks, c->num_blocks, c->pool, dst_blocks, c->num_blocks,
                                       num_pairs, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "block copy launch");
    return PKV_OK;
}

int paged_block_swap_out(pkv_cache_t c, const int32_t *block_ids, int64_t num_ids, void *dst, void *stream) {
    PKV_RANGE("paged_block_swap_out");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_ids < 0) return pkv_fail(PKV_EINVAL, "num_ids < 0");
    if (num_ids == 0) return PKV_OK;
    if (!block_ids || !dst) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(dst)) return pkv_fail(PKV_EINVAL, "dst must be 16-byte aligned");
    if (int r = check_device(c)) return r;
    cudaError_t e = launch_copy_blocks(c, c->pool, block_ids, c->num_blocks, dst, nullptr, num_ids, num_ids,
                                       static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "swap-out launch");
    return PKV_OK;
}

int paged_block_swap_in(pkv_cache_t c, const int32_t *block_ids, int64_t num_ids, const void *src, void *stream) {
    PKV_RANGE("paged_block_swap_in");
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (num_ids < 0) return pkv_fail(PKV_EINVAL, "num_ids < 0");
    if (num_ids == 0) return PKV_OK;
    if (!block_ids || !src) return pkv_fail(PKV_EINVAL, "NULL pointer");
    if (!aligned16(src)) return pkv_fail(PKV_EINVAL, "src must be 16-byte aligned");
    if (int r = check_device(c)) return r;
    cudaError_t e = launch_copy_blocks(c, src, nullptr, num_ids, c->pool, block_ids, c->num_blocks, num_ids,
                                       static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return pkv_cuda_fail(e, "swap-in launch");
    return PKV_OK;
}

int kv_cache_profile_start(pkv_cache_t c, unsigned kinds) { return kv_cache_profile_start_sampled(c, kinds, 1); }

int kv_cache_profile_start_sampled(pkv_cache_t c, unsigned kinds, int every) {
    if (!c) return pkv_fail(PKV_EINVAL, "cache is NULL");
    if (every < 1) return pkv_fail(PKV_EINVAL, "every must be >= 1, got %d", every);
    // PKV_PROFILE_* bits map onto (1 << PKV_KIND_*)
    c->profile_kinds = ((kinds & PKV_PROFILE_DECODE) ? 1u << PKV_KIND_DECODE : 0u) |
                       ((kinds & PKV_PROFILE_PREFILL) ? 1u << PKV_KIND_PREFILL : 0u) |
                       ((kinds & PKV_PROFILE_APPEND) ? 1u << PKV_KIND_APPEND : 0u) |
                       ((kinds & PKV_PROFILE_MERGE) ? 1u << PKV_KIND_MERGE : 0u) |
                       ((kinds & PKV_PROFILE_COPY) ? 1u << PKV_KIND_COPY : 0u);
    std::lock_guard<std::mutex> lk(c->mu);
    for (auto &ev : c->events) {
        c->event_pool.push_back(ev.a);
        c->event_pool.push_back(ev.b);
    }
    c->events.clear();
    c->profile_every = every;
    for (int64_t &n : c->profile_seen) n = 0;
    c->profiling = true;
    return PKV_OK;
}

int kv_cache_profile_read(pkv_cache_t c, pkv_profile_t *out) {
    if (!c || !out) return pkv_fail(PKV_EINVAL, "NULL argument");
    std::lock_guard<std::mutex> lk(c->mu);
    c->profiling = false;
    std::memset(out, 0, sizeof *out);
    for (auto &ev : c->events) {
        cudaError_t e = cudaEventSynchronize(ev.b);
        float ms = 0.f;
        if (e == cudaSuccess) e = cudaEventElapsedTime(&ms, ev.a, ev.b);
        if (e != cudaSuccess) return pkv_cuda_fail(e, "profile events");
        if (ev.kind == PKV_KIND_DECODE) {
            out->decode_launches++;
            out->decode_ms += ms;
        } else if (ev.kind == PKV_KIND_PREFILL) {
            out->prefill_launches++;
            out->prefill_ms += ms;
        } else if (ev.kind == PKV_KIND_APPEND) {
            out->append_launches++;
            out->append_ms += ms;
        } else if (ev.kind == PKV_KIND_COPY) {
            out->copy_launches++;
            out->copy_ms += ms;
        } else {
            out->merge_launches++;
            out->merge_ms += ms;
        }
        c->event_pool.push_back(ev.a);
        c->event_pool.push_back(ev.b);
    }
    c->events.clear();
    return PKV_OK;
}

} // extern "C"
