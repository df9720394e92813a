// Eviction by accumulated attention mass.
//
// Per (sequence, KV head) of L tokens, budget B < L and R recent tokens (R <= B): the last R tokens stay,
// and of the other L - R the B - R of largest mass (equal masses: the lower position first).  What stays
// keeps its order and goes to positions 0 .. B - 1 of the destination table's blocks, with its mass; a
// sequence of at most B tokens is copied whole.  Attention does not depend on the order of keys whose
// positions are already in them, so a head may keep tokens of its own choice.
//
// select_kernel: one CTA per row finds the (B - R)-th largest mass by radix selection (four passes of
// 8-bit digits over keys whose unsigned order is the masses' order, histogram in shared memory), then
// writes the kept positions in order: each warp owns a run of positions, counts, and after a scan over
// the warps places its own.  The row is read from L2 after the first pass.
// move_kernel: the gather.  Bound by HBM: row_bytes read and written per kept token, K|V and head.
// Sources and destinations are different blocks, so rows move in any order.
#include <algorithm>

#include "device_common.cuh"
#include "int4.cuh"
#include "pkv_internal.h"

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

struct EvictArgs {
    char *pool;
    const int32_t *tables, *dst_tables, *lens;
    const float *mass;
    int32_t *kept, *new_lens;
    float *mass_out;
    unsigned int *err;
    int64_t num_blocks, mass_len, mass_out_len, cap;
    int64_t blk_stride, head_stride, v_off;
    int max_blocks, max_dst_blocks, hkv, bs, d, budget, recent;
};

// masses as unsigned numbers of the same order; NaN below every number, -0 as 0
PKV_DEV uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    if (x != x) return 0u;
    return (b >> 31) ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
    __shared__ int hist[256];
    __shared__ int wsum[2][kSelWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const int s = (int)(row / a.hkv), kvh = (int)(row - (int64_t)s * a.hkv);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int L = max(a.lens[s], 0);
    if (L > a.cap) {
        if (tid == 0) set_error(a.err, PKV_DEVERR_LENGTH);
        L = 0; // the sequence is skipped
    }
    const float *m = a.mass + row * a.mass_len;
    int32_t *kept = a.kept + row * a.budget;
    float *mo = a.mass_out + row * a.mass_out_len;
    const int len = min(L, a.budget);
    if (tid == 0 && kvh == 0) a.new_lens[s] = len;
    const int n = L > a.budget ? L - a.recent : 0; // candidates
    const int k = a.budget - a.recent;             // how many of them stay

    if (n > 0 && k > 0) {
        uint32_t prefix = 0; // the threshold's digits found so far
        int left = k;        // its rank among the keys that share them
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int t0 = 0; t0 < n; t0 += kSelThreads) {
                const int t = t0 + tid;
                uint32_t key = 0;
                bool in = t < n;
                if (in) {
                    key = order_key(m[t]);
                    in = shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8));
                }
                // one addition per digit and warp: most keys of a pass share a few digits
                const int digit = in ? (int)((key >> shift) & 255u) : 256;
                const unsigned same = __match_any_sync(0xffffffffu, digit);
                if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
            }
            __syncthreads();
            if (warp == 0) { // the digit whose suffix sum first reaches `left`
                int c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = hist[255 - (lane * 8 + i)], sum += c[i];
                int before = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += v;
                }
                before -= sum; // keys of larger digits, before this lane's eight
                if (before < left && left <= before + sum) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (before < left && left <= before + c[i]) {
                            s_prefix = prefix | ((uint32_t)(255 - (lane * 8 + i)) << shift);
                            s_left = left - before;
                        }
                        before += c[i];
                    }
                }
            }
            __syncthreads();
            prefix = s_prefix;
            left = s_left;
        }
        // prefix: the threshold; `left` of the keys equal to it stay, the first ones
        const int seg = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
        const int b = min(warp * seg, n), e = min(b + seg, n);
        int gt = 0, eq = 0;
        for (int t0 = b; t0 < e; t0 += 32) {
            const int t = t0 + lane;
            const uint32_t key = t < e ? order_key(m[t]) : 0u;
            gt += __popc(__ballot_sync(0xffffffffu, t < e && key > prefix));
            eq += __popc(__ballot_sync(0xffffffffu, t < e && key == prefix));
        }
        if (lane == 0) wsum[0][warp] = gt, wsum[1][warp] = eq;
        __syncthreads();
        int at = 0, eqb = 0; // larger keys and equal keys before this warp's run
        for (int w = 0; w < warp; ++w) at += wsum[0][w], eqb += wsum[1][w];
        at += min(eqb, left);
        for (int t0 = b; t0 < e; t0 += 32) {
            const int t = t0 + lane;
            const float v = t < e ? m[t] : 0.f;
            const uint32_t key = t < e ? order_key(v) : 0u;
            const unsigned be = __ballot_sync(0xffffffffu, t < e && key == prefix);
            const bool stay = t < e && (key > prefix || (key == prefix && eqb + __popc(be & ((1u << lane) - 1)) < left));
            const unsigned bs_ = __ballot_sync(0xffffffffu, stay);
            if (stay) {
                const int p = at + __popc(bs_ & ((1u << lane) - 1));
                kept[p] = t;
                mo[p] = v;
            }
            at += __popc(bs_);
            eqb += __popc(be);
        }
    }
    // the recent tokens (or a short sequence whole), then what lies behind
    const int first = n > 0 ? k : 0, from = n > 0 ? n - k : 0;
    for (int p = first + tid; p < len; p += kSelThreads) {
        kept[p] = p + from;
        mo[p] = m[p + from];
    }
    for (int p = len + tid; p < a.budget; p += kSelThreads) kept[p] = -1;
    for (int64_t p = len + tid; p < a.mass_out_len; p += kSelThreads) mo[p] = 0.f;
}

// LPT lanes move one token's K and V rows of one head, 16 bytes each; a 4-bit row's (s, z) words go by
// the two lanes behind them.
template <int LPT, bool I4>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a, int row_bytes) {
    pdl_trigger();
    pdl_wait();
    constexpr int kTokens = kMoveThreads / LPT;
    const int64_t row = blockIdx.x;
    const int s = (int)(row / a.hkv), kvh = (int)(row - (int64_t)s * a.hkv);
    const int lane = threadIdx.x % LPT, grp = threadIdx.x / LPT;
    const int32_t *kept = a.kept + row * a.budget;
    const int32_t *src_t = a.tables + (int64_t)s * a.max_blocks, *dst_t = a.dst_tables + (int64_t)s * a.max_dst_blocks;
    const int chunks = row_bytes / 16;
    const bool code = lane < 2 * chunks, par = I4 && !code && lane < 2 * chunks + 2;
    if (!code && !par) return;
    const int kv = code ? lane / chunks : lane - 2 * chunks;
    const int64_t base = kvh * a.head_stride;
    // bytes from a (block, head)'s start to this lane's piece of row `o`
    auto piece = [&](int o) -> int64_t {
        if (!I4) return kv * a.v_off + (int64_t)o * row_bytes + (lane - kv * chunks) * 16;
        return code ? int4_codes(kv, o, (lane - kv * chunks) * 16, a.d) : int4_params(kv, o, a.d);
    };
    const int lim = (int)min((int64_t)a.budget, a.cap);
    for (int j0 = blockIdx.y * kTokens * kMoveUnroll; j0 < lim; j0 += gridDim.y * kTokens * kMoveUnroll) {
        const char *from[kMoveUnroll];
        char *to[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int j = j0 + u * kTokens + grp;
            const int t = j < lim ? kept[j] : -1;
            from[u] = nullptr;
            if (t >= 0) {
                const int sb = src_t[t / a.bs], db = dst_t[j / a.bs];
                if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
                    if (lane == 0) set_error(a.err, PKV_DEVERR_BLOCK_ID);
                } else {
                    from[u] = a.pool + sb * a.blk_stride + base + piece(t % a.bs);
                    to[u] = a.pool + db * a.blk_stride + base + piece(j % a.bs);
                }
            }
        }
        if (code) {
            uint4 x[kMoveUnroll];
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u)
                if (from[u]) x[u] = __ldcs(reinterpret_cast<const uint4 *>(from[u]));
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u)
                if (from[u]) *reinterpret_cast<uint4 *>(to[u]) = x[u];
        } else {
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u)
                if (from[u]) *reinterpret_cast<uint32_t *>(to[u]) = *reinterpret_cast<const uint32_t *>(from[u]);
        }
    }
}

} // namespace

cudaError_t launch_evict(pkv_cache *c, const EvictLaunch &v, cudaStream_t st) {
    EvictArgs a;
    a.pool = static_cast<char *>(c->pool);
    a.tables = v.tables;
    a.dst_tables = v.dst_tables;
    a.lens = v.lens;
    a.mass = v.mass;
    a.kept = v.kept;
    a.new_lens = v.new_lens;
    a.mass_out = v.mass_out;
    a.err = c->err;
    a.num_blocks = c->num_blocks;
    a.mass_len = v.mass_len;
    a.mass_out_len = v.mass_out_len;
    a.cap = std::min<int64_t>(v.mass_len, (int64_t)v.max_blocks * c->block_size);
    pkv_row_strides(c, &a.blk_stride, &a.head_stride, &a.v_off);
    a.max_blocks = v.max_blocks;
    a.max_dst_blocks = v.max_dst_blocks;
    a.hkv = c->num_kv_heads;
    a.bs = c->block_size;
    a.d = c->head_dim;
    a.budget = v.budget;
    a.recent = v.recent;
    const unsigned rows = (unsigned)v.num_seqs * (unsigned)a.hkv;
    cudaError_t e;
    {
        PkvTimer timer(c, PKV_KIND_COPY, st);
        g_pkv_launches++;
        e = pdl_launch(select_kernel, dim3(rows), dim3(kSelThreads), 0, st, a);
    }
    if (e != cudaSuccess) return e;
    const bool i4 = c->kv_dtype == PKV_INT4;
    const int row_bytes = i4 ? a.d / 2 : a.d * c->elem_bytes;
    const int lanes = 2 * row_bytes / 16 + (i4 ? 2 : 0);
    const int lpt = lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
    const int64_t per = (int64_t)(kMoveThreads / lpt) * kMoveUnroll;
    const int64_t most = std::min<int64_t>(a.budget, a.cap);
    const dim3 grid(rows, (unsigned)std::max<int64_t>(1, std::min<int64_t>((most + per - 1) / per, 65535)));
    PkvTimer timer(c, PKV_KIND_COPY, st);
    g_pkv_launches++;
    auto kern = i4 ? (lpt == 8 ? move_kernel<8, true> : move_kernel<16, true>)
                   : lpt == 8 ? move_kernel<8, false> : lpt == 16 ? move_kernel<16, false> : move_kernel<32, false>;
    return pdl_launch(kern, grid, dim3(kMoveThreads), 0, st, a, row_bytes);
}
