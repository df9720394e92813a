// Eviction by accumulated attention mass.
//
// Per (sequence, KV head) of L tokens, budget B < L and R recent tokens (R <= B): the last R tokens stay,
// and of the other L - R the B - R of largest mass (equal masses: the lower position first).  What stays
// keeps its order and goes to positions 0 .. B - 1 of the destination table's blocks, with its mass; a
// sequence of at most B tokens is copied whole.  Attention does not depend on the order of keys whose
// positions are already in them, so a head may keep tokens of its own choice.
//
// Rows that keep few tokens for their number: one CTA takes a row; it selects, then moves, and rows that still
// select run beside rows that move already.  Else a CTA, or a cluster of 2 to 8 where rows are few and long, selects a
// row's tokens, and a second launch spreads the copies over all SMs (clusters do not land evenly: two CTAs on one SM, none on
// another; two sequences of 131071 tokens x 8 heads cut to 8191: 56 us, 60 with the clusters copying themselves).
//   * Selection.  Each CTA keeps its stretch of the row's keys (numbers whose unsigned order is the masses') in
//     shared memory, and the (B - R)-th largest is found by four passes of a radix selection (digits of 8 bits,
//     histograms in shared memory, summed over the cluster's: 11-bit digits take a pass less, but made the
//     CTAs spend 34 us on one another's histograms, 16 rows of 131071 positions, where these take 24 in all);
//     up to 160 candidates are ranked by comparing all with all instead, which takes one pass.  Each warp owns
//     a run of positions, counts what stays, and after a scan over warps and CTAs writes its kept positions in
//     order.  Bound by latency: sweeps over 16384 keys a CTA and the barriers between them.
//   * Moving.  A row's kept tokens are shared out evenly over its CTAs, 512 at a time: each thread looks up one
//     token's source and destination slot a chunk ahead, so that a row's copy waits for nothing but its own
//     bytes; a warp then moves four tokens' rows at once (K and V, 16 bytes a lane, all loaded before the first
//     is stored; eight at once spill: 164 us against 159 below).  Sources and destinations are different
//     blocks, so rows move in any order.  Bound by HBM: row_bytes read and written per kept token, K|V and
//     head.  1024 rows of up to 4096 fp16 tokens, D = 128, cut to 1024: 973 MB in 159 us, 6.1 TB/s.
#include <algorithm>

#include "device_common.cuh"
#include "int4.cuh"
#include "pkv_internal.h"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
// candidates that are ranked by comparing all with all (132 of them: 6.3 us, by digits 6.9; 263: 9.8 and 7.7)
constexpr int kAllPairs = 160;
constexpr int kMaxKeys = 24 * 1024; // keys of a CTA in shared memory; longer stretches are read again
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
    int max_blocks, max_dst_blocks, hkv, bs_log2, d, budget, recent;
    int ctas, keys; // CTAs of a row; keys of a CTA that fit its shared memory
    int row_bytes;
};

// masses as unsigned numbers of the same order; NaN below every number, -0 as 0
PKV_DEV uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    if (x != x) return 0u;
    return (b >> 31) ? ~b : b | 0x80000000u;
}

PKV_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// mass of an order key (-0 comes back as 0, any NaN as one NaN)
PKV_DEV float key_mass(uint32_t k) {
    return k == 0u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}
// what stands at the place of `p` in the shared memory of the cluster's CTA `rank` (no compiler barrier, so that several
// are under way at once; the cluster barriers are ones)
PKV_DEV uint32_t peer_at(const void *p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
PKV_DEV int peer_word(const void *p, int rank) {
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_at(p, rank)));
    return v;
}
// tokens of sequence s; one that does not fit is skipped
PKV_DEV int length_of(const EvictArgs &a, int s) {
    const int L = max(a.lens[s], 0);
    if (L <= a.cap) return L;
    if (threadIdx.x == 0) set_error(a.err, PKV_DEVERR_LENGTH);
    return 0;
}

// What stays of row `row` (L tokens of sequence s, KV head kvh), its mass and what lies behind, by CTA `rank`
// of the row's C (a cluster if CL).
template <bool CL>
PKV_DEV void select_row(const EvictArgs &a, int64_t row, int s, int kvh, int L, int rank, int C) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ int hist[2][kBins];
    __shared__ int wsum[2][kWarps];
    __shared__ int sums[2]; // this CTA's larger and equal keys
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float *m = a.mass + row * a.mass_len;
    int32_t *kept = a.kept + row * a.budget;
    float *mo = a.mass_out + row * a.mass_out_len;
    const int len = min(L, a.budget);
    if (tid == 0 && rank == 0 && kvh == 0) a.new_lens[s] = len;
    const int n = L > a.budget ? L - a.recent : 0; // candidates
    const int k = a.budget - a.recent;             // how many of them stay

    if (n > 0 && k > 0) {
        // this CTA's stretch [b, b + cnt)
        const int stretch = CL ? ((n + C - 1) / C + 31) & ~31 : n;
        const int b = min(rank * stretch, n), cnt = min(stretch, n - b);
        const bool held = stretch <= a.keys;
        const bool pairs = !CL && n <= kAllPairs && held;
        if (!pairs) { // the first pass's histogram is taken while the keys come in
            if (tid < kBins) hist[0][tid] = 0;
            __syncthreads();
        }
        constexpr int kLoad = 8;
        for (int i0 = tid; i0 < cnt; i0 += kLoad * kThreads) {
            float v[kLoad];
#pragma unroll
            for (int u = 0; u < kLoad; ++u)
                if (i0 + u * kThreads < cnt) v[u] = m[b + i0 + u * kThreads];
#pragma unroll
            for (int u = 0; u < kLoad; ++u) {
                const int i = i0 + u * kThreads;
                if (i >= cnt) break;
                const uint32_t key = order_key(v[u]);
                if (held) keys[i] = key;
                if (!pairs) atomicAdd(&hist[0][key >> 24], 1);
            }
        }
        // keys i .. i + 3 (i a multiple of 4; what lies behind the stretch is not meant)
        auto four = [&](int i) {
            if (held) return *reinterpret_cast<const uint4 *>(keys + i);
            const float *p = m + b + i;
            return make_uint4(order_key(p[0]), i + 1 < cnt ? order_key(p[1]) : 0u, i + 2 < cnt ? order_key(p[2]) : 0u,
                              i + 3 < cnt ? order_key(p[3]) : 0u);
        };
        uint32_t prefix = 0; // the threshold; `left` of the keys equal to it stay, the first ones
        int left = k;
        if (pairs) {
            if (tid >= n && tid < ((n + 3) & ~3)) keys[tid] = 0u; // (not larger than any)
            __syncthreads();
            if (tid < n) {
                const uint32_t mine = keys[tid];
                int larger = 0, same = 0; // same: equal ones before
#pragma unroll 4
                for (int i = 0; i < n; i += 4) {
                    const uint4 o = *reinterpret_cast<const uint4 *>(keys + i);
                    larger += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
                    same += (o.x == mine && i < tid) + (o.y == mine && i + 1 < tid) + (o.z == mine && i + 2 < tid) +
                            (o.w == mine && i + 3 < tid);
                }
                if (larger + same == k - 1) s_prefix = mine, s_left = same + 1;
            }
            __syncthreads();
            prefix = s_prefix;
            left = s_left;
        } else {
            for (int pass = 0; pass < 4; ++pass) {
                const int shift = 24 - 8 * pass;
                int *h = hist[pass & 1];
                if (pass > 0) {
                    if (tid < kBins) h[tid] = 0;
                    __syncthreads();
                    const uint32_t found = prefix >> (shift + 8);
                    for (int i = tid * 4; i < cnt; i += 4 * kThreads) {
                        const uint4 q = four(i);
                        const uint32_t k4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (i + u < cnt && (k4[u] >> (shift + 8)) == found)
                                atomicAdd(&h[(k4[u] >> shift) & (kBins - 1)], 1);
                    }
                }
                if (CL)
                    cluster_sync();
                else
                    __syncthreads();
                // a digit a thread, the largest first; the thread whose sum reaches `left` has the digit
                int c = 0;
                if (tid < kBins) {
                    const int *d = &h[kBins - 1 - tid];
                    if (CL) {
                        int part[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r) part[r] = r < C ? peer_word(d, r) : 0;
#pragma unroll
                        for (int r = 0; r < 8; ++r) c += part[r];
                    } else {
                        c = *d;
                    }
                }
                int before = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += v;
                }
                if (lane == 31) wsum[0][warp] = before;
                __syncthreads();
                for (int w = 0; w < warp; ++w) before += wsum[0][w];
                before -= c; // keys of larger digits
                if (before < left && left <= before + c) {
                    s_prefix = prefix | ((uint32_t)(kBins - 1 - tid) << shift);
                    s_left = left - before;
                }
                __syncthreads();
                prefix = s_prefix;
                left = s_left;
            }
        }
        // ---- each warp's run of the stretch: larger and equal keys, their sums before it, then the positions
        const int run = ((cnt + kWarps - 1) / kWarps + 127) & ~127;
        const int rb = min(warp * run, cnt), re = min(rb + run, cnt);
        int gt = 0, eq = 0;
        for (int i = rb + lane * 4; i < re; i += 128) {
            const uint4 q = four(i);
            const uint32_t k4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                gt += i + u < re && k4[u] > prefix;
                eq += i + u < re && k4[u] == prefix;
            }
        }
        gt = __reduce_add_sync(0xffffffffu, gt);
        eq = __reduce_add_sync(0xffffffffu, eq);
        __syncthreads(); // wsum has been read
        if (lane == 0) wsum[0][warp] = gt, wsum[1][warp] = eq;
        __syncthreads();
        int at = 0, eqb = 0; // larger and equal keys before this warp's run
        for (int w = 0; w < warp; ++w) at += wsum[0][w], eqb += wsum[1][w];
        if (CL) {
            if (tid == kThreads - 1) sums[0] = at + gt, sums[1] = eqb + eq;
            cluster_sync();
            for (int r = 0; r < rank; ++r) at += peer_word(&sums[0], r), eqb += peer_word(&sums[1], r);
        }
        at += min(eqb, left);
        for (int i0 = rb; i0 < re; i0 += 128) {
            const int i = i0 + lane * 4;
            const uint4 q = i < re ? four(i) : make_uint4(0, 0, 0, 0);
            const uint32_t k4[4] = {q.x, q.y, q.z, q.w};
            int g = 0, e = 0; // this lane's larger and equal keys
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                g += i + u < re && k4[u] > prefix;
                e += i + u < re && k4[u] == prefix;
            }
            int both = g | (e << 16); // summed over the lanes before, and over all
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, both, o);
                if (lane >= o) both += v;
            }
            const int all = __shfl_sync(0xffffffffu, both, 31);
            int e_at = eqb + (both >> 16) - e;
            // equal keys take a place while fewer than `left` of them have
            int p = at + (both & 0xFFFF) - g + min(e_at, left) - min(eqb, left);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool in = i + u < re, same = in && k4[u] == prefix;
                if (in && (k4[u] > prefix || (same && e_at < left))) {
                    kept[p] = b + i + u;
                    mo[p] = key_mass(k4[u]);
                    ++p;
                }
                e_at += same;
            }
            at += (all & 0xFFFF) + min(eqb + (all >> 16), left) - min(eqb, left);
            eqb += all >> 16;
        }
    }
    // ---- the recent tokens (or a short sequence whole), then what lies behind
    const int first = n > 0 ? k : 0, from = n > 0 ? n - k : 0;
    const int t0 = rank * kThreads + tid, step = C * kThreads;
    for (int p = first + t0; p < len; p += step) {
        kept[p] = p + from;
        mo[p] = m[p + from];
    }
    for (int p = len + t0; p < a.budget; p += step) kept[p] = -1;
#pragma unroll 4
    for (int64_t p = len + t0; p < a.mass_out_len; p += step) mo[p] = 0.f;
}

// Moves the `len` tokens of row `row` that stay, CTA `rank` of C a C-th of them.  LPT lanes move one token's
// K and V rows of one head, 16 bytes each; a 4-bit row's (s, z) words go by the two lanes behind them.
template <int LPT, bool I4>
PKV_DEV void move_row(const EvictArgs &a, int64_t row, int s, int kvh, int len, int rank, int C) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int32_t *kept = a.kept + row * a.budget;
    const int per = (len + C - 1) / C, end = min(len, (rank + 1) * per);
    constexpr int kGroups = kThreads / LPT;
    __shared__ uint2 slots[2][kThreads]; // source and destination slot of a chunk's tokens; none: -1
    const int part = lane % LPT, grp = tid / LPT;
    const int32_t *src_t = a.tables + (int64_t)s * a.max_blocks, *dst_t = a.dst_tables + (int64_t)s * a.max_dst_blocks;
    const int chunks = a.row_bytes / 16, bs = 1 << a.bs_log2;
    const bool code = part < 2 * chunks, par = I4 && !code && part < 2 * chunks + 2;
    const int kv = code ? part / chunks : part - 2 * chunks, in_row = (part - kv * chunks) * 16;
    char *head = a.pool + kvh * a.head_stride + (I4 ? 0 : kv * a.v_off + in_row);
    // this lane's piece of a slot's row
    auto place = [&](uint32_t slot) -> char * {
        const uint32_t o = slot & (bs - 1);
        char *p = head + (int64_t)(slot >> a.bs_log2) * a.blk_stride;
        if constexpr (!I4) return p + o * a.row_bytes;
        return p + (code ? int4_codes(kv, o, in_row, a.d) : int4_params(kv, o, a.d));
    };
    // a chunk's tokens, a thread each: the position two chunks ahead, its blocks one chunk ahead
    const int mine = rank * per + tid;
    auto kept_at = [&](int j) { return j < end ? kept[j] : -1; };
    auto blocks_at = [&](int j, int t) {
        return t < 0 ? make_int2(0, 0) : make_int2(src_t[t >> a.bs_log2], dst_t[j >> a.bs_log2]);
    };
    auto slots_of = [&](int j, int t, int2 b) {
        if (t < 0) return make_uint2(~0u, ~0u);
        if (b.x < 0 || b.x >= a.num_blocks || b.y < 0 || b.y >= a.num_blocks) {
            set_error(a.err, PKV_DEVERR_BLOCK_ID);
            return make_uint2(~0u, ~0u);
        }
        return make_uint2(((uint32_t)b.x << a.bs_log2) + (t & (bs - 1)), ((uint32_t)b.y << a.bs_log2) + (j & (bs - 1)));
    };
    int t1 = kept_at(mine), t2 = kept_at(mine + kThreads);
    slots[0][tid] = slots_of(mine, t1, blocks_at(mine, t1));
    __syncthreads();
    for (int j0 = rank * per, buf = 0; j0 < end; j0 += kThreads, buf ^= 1) {
        t1 = t2;
        const int j1 = j0 + kThreads + tid;
        const int2 b1 = blocks_at(j1, t1);
        t2 = kept_at(j1 + kThreads);
        const int here = min(kThreads, end - j0);
        if (code || par) {
            for (int i0 = grp; i0 < here; i0 += kGroups * kMoveUnroll) {
                uint2 sl[kMoveUnroll];
                uint4 x[kMoveUnroll];
#pragma unroll
                for (int u = 0; u < kMoveUnroll; ++u) {
                    const int i = i0 + u * kGroups;
                    sl[u] = i < here ? slots[buf][i] : make_uint2(~0u, ~0u);
                    if (sl[u].x == ~0u) continue;
                    if (code)
                        x[u] = __ldcs(reinterpret_cast<const uint4 *>(place(sl[u].x)));
                    else
                        x[u].x = *reinterpret_cast<const uint32_t *>(place(sl[u].x));
                }
#pragma unroll
                for (int u = 0; u < kMoveUnroll; ++u) {
                    if (sl[u].x == ~0u) continue;
                    if (code)
                        *reinterpret_cast<uint4 *>(place(sl[u].y)) = x[u];
                    else
                        *reinterpret_cast<uint32_t *>(place(sl[u].y)) = x[u].x;
                }
            }
        }
        slots[buf ^ 1][tid] = slots_of(j1, t1, b1);
        __syncthreads();
    }
}

template <int LPT, bool I4>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const EvictArgs a) {
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x / a.hkv, kvh = blockIdx.x - s * a.hkv, L = length_of(a, s);
    select_row<false>(a, blockIdx.x, s, kvh, L, 0, 1);
    __syncthreads();
    move_row<LPT, I4>(a, blockIdx.x, s, kvh, min(L, a.budget), 0, 1);
}

template <bool CL>
__global__ void __launch_bounds__(kThreads, 2) select_kernel(const EvictArgs a) {
    pdl_trigger();
    pdl_wait();
    const int row = CL ? blockIdx.x / a.ctas : blockIdx.x, s = row / a.hkv;
    select_row<CL>(a, row, s, row - s * a.hkv, length_of(a, s), blockIdx.x - row * a.ctas, a.ctas);
    if (CL) cluster_sync(); // nobody leaves while its sums are read
}

template <int LPT, bool I4>
__global__ void __launch_bounds__(kThreads, 2) move_kernel(const EvictArgs a) {
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x / a.ctas, s = row / a.hkv;
    move_row<LPT, I4>(a, row, s, row - s * a.hkv, min(length_of(a, s), a.budget), blockIdx.x - row * a.ctas, a.ctas);
}

template <bool CL>
cudaError_t launch_select(const EvictArgs &a, unsigned rows, size_t smem, cudaStream_t st) {
    static std::atomic<bool> have[64];
    cudaError_t e = pkv_allow_smem(reinterpret_cast<const void *>(select_kernel<CL>), have);
    if (e != cudaSuccess) return e;
    g_pkv_launches++;
    if constexpr (!CL) return pdl_launch(select_kernel<CL>, dim3(rows), dim3(kThreads), smem, st, a);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * a.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_kernel<CL>, a);
}

template <int LPT, bool I4>
cudaError_t launch_t(EvictArgs a, unsigned rows, bool apart, int sms, cudaStream_t st) {
    const size_t smem = a.keys * sizeof(uint32_t);
    if (!apart) {
        static std::atomic<bool> have[64];
        auto kern = evict_kernel<LPT, I4>;
        cudaError_t e = pkv_allow_smem(reinterpret_cast<const void *>(kern), have);
        if (e != cudaSuccess) return e;
        g_pkv_launches++;
        return pdl_launch(kern, dim3(rows), dim3(kThreads), smem, st, a);
    }
    cudaError_t e = a.ctas > 1 ? launch_select<true>(a, rows, smem, st) : launch_select<false>(a, rows, smem, st);
    if (e != cudaSuccess) return e;
    // two for each SM, and no more than 512 tokens for one
    a.ctas = (int)std::max<int64_t>((2 * sms + rows - 1) / rows, (std::min<int64_t>(a.cap, a.budget) + kThreads - 1) / kThreads);
    g_pkv_launches++;
    return pdl_launch(move_kernel<LPT, I4>, dim3(rows * a.ctas), dim3(kThreads), 0, st, a);
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
    a.bs_log2 = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
    a.d = c->head_dim;
    a.budget = v.budget;
    a.recent = v.recent;
    const bool i4 = c->kv_dtype == PKV_INT4;
    a.row_bytes = i4 ? a.d / 2 : a.d * c->elem_bytes;
    const unsigned rows = (unsigned)v.num_seqs * (unsigned)a.hkv;
    // a CTA per row, or a cluster while there are SMs for its CTAs and each gets 2048 positions or more (16 rows
    // of 131071 positions: clusters of 16 took 4 us more than clusters of 8, their barriers take longer)
    a.ctas = 1;
    while (a.ctas < 8 && (int64_t)rows * a.ctas * 2 <= c->num_sms && a.cap / (2 * a.ctas) >= 2048) a.ctas *= 2;
    const int64_t stretch = ((a.cap + a.ctas - 1) / a.ctas + 31) / 32 * 32;
    a.keys = (int)std::min<int64_t>(stretch, kMaxKeys);
    const int lanes = 2 * a.row_bytes / 16 + (i4 ? 2 : 0);
    PkvTimer timer(c, PKV_KIND_COPY, st);
    const int sms = c->num_sms;
    // Rows that keep many tokens for their number: the copies apart (8 rows that keep 600 bf16 tokens, D = 128:
    // 8.6 us against 13.2; 152 rows of very different lengths that keep up to 4566, 40 against 85; but 128 that
    // keep 300, 14 against 13, and 256 that keep 2000, 76 against 73)
    const bool apart = a.ctas > 1 || std::min<int64_t>(a.cap, a.budget) > 384 + 4 * (int64_t)rows;
    if (i4) return lanes <= 8 ? launch_t<8, true>(a, rows, apart, sms, st) : launch_t<16, true>(a, rows, apart, sms, st);
    if (lanes <= 8) return launch_t<8, false>(a, rows, apart, sms, st);
    return lanes <= 16 ? launch_t<16, false>(a, rows, apart, sms, st) : launch_t<32, false>(a, rows, apart, sms, st);
}
