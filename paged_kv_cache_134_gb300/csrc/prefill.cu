// Host side of the tensor-core attention of prefill_impl.cuh: the work-list kernel, the tiled-TMA maps
// and the launches of the packed prefill, the prefill over a cached prefix and the cascade decode's
// prefix phase.  The attention kernel itself is instantiated in prefill_packed.cu, prefill_paged.cu
// and prefill_cascade.cu (one translation unit each, compiled in parallel).
#include <algorithm>
#include <cstdlib>
#include <mutex>

#include "chunk_stream.cuh"

namespace pkv_prefill {

constexpr int kPlanThreads = 1024;

// in-place inclusive prefix sum of x[0, n) by the whole CTA (kPlanThreads threads)
PKV_DEV void cta_inclusive_scan(int *x, int n, int *warp_sums) {
    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int b = min((int)threadIdx.x * per, n), e = min(b + per, n);
    int own = 0;
    for (int i = b; i < e; ++i) own += x[i];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) warp_sums[w] = v;
    __syncthreads();
    if (w == 0) {
        int u = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) u += t;
        }
        warp_sums[lane] = u;
    }
    __syncthreads();
    int run = v - own + (w > 0 ? warp_sums[w - 1] : 0);
    for (int i = b; i < e; ++i) {
        run += x[i];
        x[i] = run;
    }
    __syncthreads();
}

// key tiles of pair p of sequence i (its two query tiles' key tiles added), from the item decoding
PKV_DEV int pair_cost(const Args &a, int i, int p) {
    const Item it = decode_item(a, i, p, 0);
    return it.t[0].n + it.t[1].n;
}

// The work list: every (sequence, pair of query tiles), heaviest first (a counting sort on the pair's
// key tiles, clamped to the histogram's range), so that the persistent CTAs, which take items in list
// order, end together.  The order inside one cost class is whatever the atomics give; it only decides
// which CTA computes an item, never what the item computes.  Also resets the next-item counter the
// attention kernel draws from.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Args a) {
    extern __shared__ int sh[];
    const int R = a.cost_bins;
    int *hist = sh; // hist[c] = #{pairs of cost c}, then #{pairs of cost <= c}
    int *cnt = sh + R;
    int *warp_sums = sh + 2 * R;
    pdl_trigger();
    pdl_wait();
    if (a.nps > 0) {
        // cascade: the items are the (tile of query rows, split pair) pairs, taken in order
        if (threadIdx.x == 0) {
            a.plan[0] = ((a.num_seqs + BM - 1) / BM) * ((a.nps + 1) / 2);
            a.plan[1] = 0;
        }
        return;
    }
    for (int x = threadIdx.x; x < R; x += kPlanThreads) {
        hist[x] = 0;
        cnt[x] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.num_seqs; i += kPlanThreads) {
        const int np = (seq_tiles(a, i, true) + 1) / 2;
        for (int p = 0; p < np; ++p) atomicAdd(&hist[min(pair_cost(a, i, p), R - 1)], 1);
    }
    __syncthreads();
    cta_inclusive_scan(hist, R, warp_sums); // hist[c] = #{pairs of cost <= c}
    const int total = hist[R - 1];
    int2 *list = reinterpret_cast<int2 *>(a.plan + 4);
    for (int i = threadIdx.x; i < a.num_seqs; i += kPlanThreads) {
        const int np = (seq_tiles(a, i, false) + 1) / 2;
        for (int p = 0; p < np; ++p) {
            const int c = min(pair_cost(a, i, p), R - 1);
            // descending cost: the pairs of cost c come after every pair of higher cost
            const int pos = total - hist[c] + atomicAdd(&cnt[c], 1);
            if (pos < a.plan_cap) list[pos] = make_int2(i, p);
        }
    }
    if (threadIdx.x == 0) {
        // sequences whose rows overlap make more pairs than the tokens allow: reported, list cut short
        if (total > a.plan_cap) set_error(a.err, PKV_DEVERR_CU_SEQLENS);
        a.plan[0] = (int)min((int64_t)total, a.plan_cap);
        a.plan[1] = 0;
    }
}

// The work list of a chunk call: every (sequence, row tile or pair of them, split), heaviest first as above.  As many
// lanes take a sequence as it can have row tiles (or pairs), up to a warp.
template <bool STREAM>
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const Args a) {
    extern __shared__ int sh[];
    const int R = a.cost_bins;
    int *hist = sh, *cnt = sh + R, *warp_sums = sh + 2 * R;
    pdl_trigger();
    pdl_wait();
    for (int x = threadIdx.x; x < R; x += kPlanThreads) hist[x] = cnt[x] = 0;
    __syncthreads();
    const int wide = a.max_groups >= 32 ? 32 : a.max_groups <= 1 ? 1 : 2 << (31 - __clz(a.max_groups - 1)); // lanes of a sequence
    const int lane = threadIdx.x & (wide - 1);
    int4 *list = reinterpret_cast<int4 *>(a.plan + 4);
    auto visit = [&](bool report, auto &&entry) {
        for (int i = threadIdx.x / wide; i < a.num_seqs; i += kPlanThreads / wide) {
            const int n = chunk_groups<!STREAM>(a, i, report && lane == 0);
            for (int g = lane; g < n; g += wide) {
                // (splits are of equal size but for the last one)
                const int parts = STREAM ? max(1, stream_unit(a, i, g, 0, 0).nsplit) : chunk_parts(chunk_item(a, i, g, 0, 0));
                for (int k = 0; k < parts; ++k) {
                    int cost;
                    if constexpr (STREAM) {
                        cost = stream_unit(a, i, g, k, 0).n;
                    } else {
                        const ChunkItem it = chunk_item(a, i, g, k, 0);
                        cost = it.t[0].n + it.t[1].n;
                    }
                    entry(i, g, k, min(cost, R - 1));
                }
            }
        }
    };
    visit(true, [&](int, int, int, int c) { atomicAdd(&hist[c], 1); });
    __syncthreads();
    cta_inclusive_scan(hist, R, warp_sums);
    const int total = hist[R - 1];
    visit(false, [&](int i, int g, int k, int c) {
        const int pos = total - hist[c] + atomicAdd(&cnt[c], 1);
        if (pos < a.plan_cap) list[pos] = make_int4(i, g, k, 0);
    });
    if (threadIdx.x == 0) {
        if (total > a.plan_cap) set_error(a.err, PKV_DEVERR_CU_SEQLENS); // rows that overlap: the list is cut short
        a.plan[0] = (int)min((int64_t)total, a.plan_cap);
        a.plan[1] = 0;
    }
}

// The rows of a chunk whose keys went in several splits: partials joined by their maxima, one warp a (token, head) row.
template <int D, int MT, bool STREAM>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const Args a) {
    using M = ModelT<MT>;
    constexpr int PER = D / 32;
    pdl_wait();
    const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int tok = blockIdx.x;
    if (h >= a.hq) return;
    const int64_t base = ((int64_t)tok * a.hq + h) * a.max_splits;
    const float2 *ml = reinterpret_cast<const float2 *>(a.ws_ml) + base;
    // (read while the row's sequence is looked for; what lies behind its splits is left aside below)
    const float2 early = lane < a.max_splits ? ml[lane] : make_float2(0.f, 0.f);
    // the sequence of the token: the last one that starts at or before it (the whole warp searches)
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < hi && a.cu[i] <= tok);
        if (!le) return; // (starts that do not ascend)
        lo += (31 - __clz(le)) * step;
        hi = min(hi, lo + step);
    }
    const int st = a.cu[lo], en = a.cu[lo + 1];
    if (tok < st || tok >= en || st < 0 || en > a.total_tokens || en - st > a.max_seqlen ||
        (int64_t)a.lens[lo] > (int64_t)a.max_blocks * a.bs)
        return;
    if (en - st <= a.few_rows >> a.lg_group) return;
    const int tile = (tok - st) / (BM >> a.lg_group);
    const int n = STREAM ? stream_unit(a, lo, tile, 0, 0).nsplit : chunk_splits(chunk_item(a, lo, tile / 2, 0, 0), tile & 1);
    if (n <= 1) return;
    float top = -INFINITY;
    for (int j = lane; j < n; j += 32) {
        const float2 v = j < 32 ? early : ml[j];
        if (v.y != 0.f) top = fmaxf(top, v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float num[PER], den = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) num[e] = 0.f;
    constexpr int U = 8; // splits whose loads go out together
    for (int j0 = 0; j0 < n; j0 += U) {
        float2 w[U];
        float v[U][PER];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            w[u] = make_float2(0.f, 0.f);
            if (j0 + u >= n) continue;
            w[u] = ml[j0 + u];
            const float *src = a.ws_o + (base + j0 + u) * D + lane * PER;
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                const float2 x = *reinterpret_cast<const float2 *>(src + e);
                v[u][e] = x.x;
                v[u][e + 1] = x.y;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (w[u].y == 0.f) continue; // no key of this split in sight (a NaN is a sum like any other)
            const float f = fast_exp2(w[u].x - top);
            den = fmaf(f, w[u].y, den);
#pragma unroll
            for (int e = 0; e < PER; ++e) num[e] = fmaf(f, v[u][e], num[e]);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<typename M::T *>(a.out) + ((int64_t)tok * a.hq + h) * D) + lane * (PER / 2);
#pragma unroll
    for (int e = 0; e < PER; e += 2) o[e / 2] = M::pack(num[e] * inv, num[e + 1] * inv);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// 2-D view [rows][cols] of a row-major matrix; box = 64 columns x box_rows rows, 128-byte swizzle.
// mt = PKV_FP8_E4M3: one-byte elements, boxes of 128 columns (one 128-byte swizzle row).
bool make_map(CUtensorMap *m, const void *base, int mt, int64_t rows, int64_t cols, int box_rows) {
    EncodeFn enc = encode_fn();
    if (!enc) return false;
    const bool bytes = mt == PKV_FP8_E4M3;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * (bytes ? 1 : 2)};
    const cuuint32_t box[2] = {bytes ? 128u : 64u, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType dt = bytes                ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : mt == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = enc(m, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// q or out [T][Hq][D] as tiles of 128 (or `rows`) (token, head of a group) rows: box = 64 dims x G heads x rows / G tokens
bool make_group_map(CUtensorMap *m, const void *base, int mt, int64_t tokens, int hq, int D, int G, int rows = BM) {
    EncodeFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)hq, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)hq * D * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)(rows / G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType dt = mt == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = enc(m, dt, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// E4M3 pool rows [rows][cols] of bytes, unswizzled: one box = box_rows whole rows (cols <= 256, a
// multiple of 16), landing as box_rows consecutive rows of cols bytes
bool make_code_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int box_rows) {
    EncodeFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols};
    const cuuint32_t box[2] = {(cuuint32_t)cols, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

cudaError_t launch_plan(const Args &a, cudaStream_t st) {
    const int smem = (2 * a.cost_bins + 32) * (int)sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return pdl_launch(plan_kernel, dim3(1), dim3(kPlanThreads), smem, st, a);
}

// the pool's map for the attention's key loads and the packed mode's block stores: 16-bit rows of D
// elements, box = bs rows x 64 dims, swizzled; E4M3 rows of D codes, box = bs whole rows, unswizzled
bool pool_map(CUtensorMap *m, const pkv_cache *c) {
    const int64_t pool_rows = c->num_blocks * 2 * c->num_kv_heads * c->block_size;
    if (c->kv_dtype == PKV_FP8_E4M3) return make_code_map(m, c->pool, pool_rows, c->head_dim, c->block_size);
    return make_map(m, c->pool, c->model_dtype, pool_rows, c->head_dim, c->block_size);
}

template <>
cudaError_t launch_stream_any<false, true>(int, int, const CUtensorMap &, const CUtensorMap &, const Args &, int, cudaStream_t);
template <>
cudaError_t launch_stream_any<false, false>(int, int, const CUtensorMap &, const CUtensorMap &, const Args &, int, cudaStream_t);
template <>
cudaError_t launch_stream_any<true, true>(int, int, const CUtensorMap &, const CUtensorMap &, const Args &, int, cudaStream_t);
template <>
cudaError_t launch_stream_any<true, false>(int, int, const CUtensorMap &, const CUtensorMap &, const Args &, int, cudaStream_t);

template <int MODE, bool KV8>
cudaError_t dispatch(int D, int mt, const Maps &m, const Args &a, int64_t max_ctas, int num_sms, cudaStream_t st) {
    if (D == 128)
        return mt == PKV_BF16 ? launch_attn<128, PKV_BF16, MODE, KV8>(m, a, max_ctas, num_sms, st)
                              : launch_attn<128, PKV_F16, MODE, KV8>(m, a, max_ctas, num_sms, st);
    if (D == 64)
        return mt == PKV_BF16 ? launch_attn<64, PKV_BF16, MODE, KV8>(m, a, max_ctas, num_sms, st)
                              : launch_attn<64, PKV_F16, MODE, KV8>(m, a, max_ctas, num_sms, st);
    return cudaErrorInvalidValue;
}

int lg2(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

Args base_args(pkv_cache *c, float scale) {
    Args a{};
    a.pool = static_cast<char *>(c->pool);
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.err = c->err;
    a.num_blocks = c->num_blocks;
    a.tile_elems = (int64_t)c->block_size * c->head_dim;
    a.hkv = c->num_kv_heads;
    a.bs = c->block_size;
    a.lg_bs = lg2(c->block_size);
    a.scale_log2 = scale * 1.4426950408889634f;
    return a;
}

} // namespace pkv_prefill

bool pkv_tmap_2d(CUtensorMap *m, const void *base, int mt, int64_t rows, int64_t cols, int box_rows) {
    return pkv_prefill::make_map(m, base, mt, rows, cols, box_rows);
}

bool pkv_tmap_kv_pairs_e4m3(CUtensorMap *m, const void *pool, int64_t num_blocks, int hkv, int bs) {
    using namespace pkv_prefill;
    EncodeFn enc = encode_fn();
    if (!enc || bs % 8 || bs / 8 > 256 || num_blocks < 1 || (int64_t)hkv * bs / 8 > 0x7FFFFFFFLL) return false;
    // the pool's E4M3 rows [(block, K|V, head, slot)][128 codes] seen as (code, slot % 8, K|V,
    // head * bs / 8 + slot / 8, block): a box of (128, 8, 2, bs / 8, 1) at (0, 0, 0, head * bs / 8,
    // block) is the K tile and the V tile of one (block, head) in one copy, landing as
    // [slot / 8][K, V][8 rows][128 bytes] (each 8-row group of K followed by the same rows of V)
    const cuuint64_t row = 128, kv = (cuuint64_t)hkv * bs * row;
    const cuuint64_t dims[5] = {128, 8, 2, (cuuint64_t)hkv * bs / 8, (cuuint64_t)num_blocks};
    const cuuint64_t strides[4] = {row, kv, 8 * row, 2 * kv};
    const cuuint32_t box[5] = {128u, 8u, 2u, (cuuint32_t)(bs / 8), 1u};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(pool), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool pkv_tmap_rows128_grouped(CUtensorMap *m, const void *base, int mt, int64_t rows, int box_rows) {
    using namespace pkv_prefill;
    EncodeFn enc = encode_fn();
    if (!enc || rows % 8 || box_rows % 8 || box_rows > 256 * 8) return false;
    // rows of 128 16-bit elements = 256 bytes, seen as (64 elements, row in its group of 8, half, group):
    // a box of (64, 8, 2, box_rows / 8) lands as [group][half][8 rows][128 bytes]
    const cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)(rows / 8)};
    const cuuint64_t strides[3] = {256, 128, 2048};
    const cuuint32_t box[4] = {64u, 8u, 2u, (cuuint32_t)(box_rows / 8)};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUtensorMapDataType dt = mt == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = enc(m, dt, 4, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

static cudaError_t ensure_plan(pkv_cache *c, int64_t bytes) {
    if (bytes <= c->plan_bytes) return cudaSuccess;
    if (c->plan) cudaFree(c->plan);
    c->plan = nullptr;
    c->plan_bytes = 0;
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(&c->plan), (size_t)bytes);
    if (e != cudaSuccess) {
        c->plan = nullptr;
        return e;
    }
    c->plan_bytes = bytes;
    return cudaSuccess;
}

cudaError_t launch_prefill(pkv_cache *c, const PrefillLaunch &p, cudaStream_t st) {
    using namespace pkv_prefill;
    if (p.total_tokens <= 0) return cudaSuccess;
    const int D = c->head_dim;
    const int mt = c->model_dtype;
    const bool kv8 = c->kv_dtype == PKV_FP8_E4M3, kv4 = c->kv_dtype == PKV_INT4;
    if (kv4 && p.ctx) return cudaErrorNotSupported;
    Args a = base_args(c, p.scale);
    a.k = static_cast<const char *>(p.k);
    a.v = static_cast<const char *>(p.v);
    a.out = p.out;
    a.cu = p.cu;
    a.ctx = p.ctx;
    a.tables = p.tables;
    a.total_tokens = p.total_tokens;
    a.num_seqs = p.num_seqs;
    a.max_seqlen = p.max_seqlen;
    a.max_blocks = p.max_blocks;
    a.hq = p.num_q_heads;
    a.write_pool = kv8 || kv4 ? 0 : 1;
    // (sequence, pair of query tiles) items: sum_i ceil(n_i / 2 BM) <= T / 2 BM + num_seqs
    const int64_t tiles_max = ((int64_t)p.max_seqlen + BM - 1) / BM;
    a.npairs_max = (int)((tiles_max + 1) / 2);
    const int64_t items = std::min<int64_t>((int64_t)a.npairs_max * p.num_seqs, p.total_tokens / (2 * BM) + p.num_seqs);
    if (items == 0) return cudaSuccess;
    if (items * p.num_q_heads > 0x7FFFFFFF) return cudaErrorNotSupported;
    // cost classes of the heaviest-first list: a pair's key tiles, at most 2 ceil((ctx + n) / BN); the
    // histogram's range is clamped (the order then only approximates heaviest first)
    const int64_t max_keys = p.ctx ? (int64_t)p.max_blocks * c->block_size : (int64_t)p.max_seqlen;
    a.cost_bins = (int)std::min<int64_t>(2 * ((max_keys + BN - 1) / BN) + 2, 16384);
    const int64_t plan_bytes = (4 + 2 * items) * (int64_t)sizeof(int);
    a.plan_cap = items;
    cudaError_t e = ensure_plan(c, plan_bytes);
    if (e != cudaSuccess) return e;
    a.plan = c->plan;
    // the pool as rows [(block, K|V, head, slot)][D] for the key loads and the tiled stores of whole
    // blocks; row coordinates are 32-bit
    const int64_t pool_rows = c->num_blocks * 2 * c->num_kv_heads * c->block_size;
    if (pool_rows > 0x7FFFFFFFLL) return cudaErrorNotSupported;
    Maps m;
    if (!make_map(&m.q, p.q, mt, p.total_tokens, (int64_t)p.num_q_heads * D, BM) ||
        !make_map(&m.k, p.k, mt, p.total_tokens, (int64_t)c->num_kv_heads * D, BN) ||
        !make_map(&m.v, p.v, mt, p.total_tokens, (int64_t)c->num_kv_heads * D, BN) ||
        // (a 4-bit pool has no rows of elements: the append writes it and no load of the packed mode reads it)
        !(kv4 ? make_map(&m.pool, p.k, mt, p.total_tokens, (int64_t)c->num_kv_heads * D, BN) : pool_map(&m.pool, c)) ||
        !make_map(&m.out, p.out, mt, p.total_tokens, (int64_t)p.num_q_heads * D, BM))
        return cudaErrorInvalidValue;
    if (p.ctx || kv8 || kv4) {
        // A cached prefix: the new tokens' K/V go to their slots first, then attention reads every key
        // through the block table.  An FP8 or 4-bit cache: the packed prefill's K/V write is the append's
        // (E4M3 or 4-bit codes), and the attention reads the packed k, v.
        e = launch_append_ranges(c, p.k, p.v, p.tables, p.num_seqs, p.max_blocks, p.cu, p.ctx, p.total_tokens, st);
        if (e != cudaSuccess) return e;
    }
    PkvTimer timer(c, PKV_KIND_PREFILL, st);
    e = launch_plan(a, st);
    g_pkv_launches++;
    if (e != cudaSuccess) return e;
    const int64_t max_ctas = items * p.num_q_heads;
    if (!p.ctx)
        e = dispatch<MODE_PACKED, false>(D, mt, m, a, max_ctas, c->num_sms, st);
    else if (kv8)
        e = dispatch<MODE_PAGED, true>(D, mt, m, a, max_ctas, c->num_sms, st);
    else
        e = dispatch<MODE_PAGED, false>(D, mt, m, a, max_ctas, c->num_sms, st);
    g_pkv_launches++;
    return e;
}

int cascade_split_tokens(const pkv_cache *c, int num_seqs, int num_q_heads, int prefix_tokens) {
    using namespace pkv_prefill;
    if (const char *v = std::getenv("PAGEDKV_CASCADE_SPLIT_TOKENS")) {
        // keys per prefix split, for tuning sweeps (rounded up to whole 128-key tiles)
        const int x = std::atoi(v);
        if (x > 0) return (x + BN - 1) / BN * BN;
    }
    // The prefix phase runs as one wave of items where it can: as many split pairs per (query-row tile,
    // head) as leave every item a CTA (one per SM; a split past one wave makes the whole phase wait for
    // a second), each split of at least 256 keys so that an item's fixed costs (Q load, epilogue,
    // partial write) stay small next to its key tiles, in whole 128-key tiles.
    const int64_t rows = (int64_t)((num_seqs + BM - 1) / BM) * num_q_heads;
    const int64_t pairs = std::max<int64_t>(1, (int64_t)c->num_sms / std::max<int64_t>(rows, 1));
    const int64_t nps = 2 * pairs;
    int64_t split = (prefix_tokens + nps - 1) / nps;
    split = std::max<int64_t>(split, 256);
    return (int)((split + BN - 1) / BN * BN);
}

cudaError_t launch_cascade_prefix(pkv_cache *c, const CascadePrefixLaunch &p, cudaStream_t st, int part) {
    using namespace pkv_prefill;
    if (p.num_seqs <= 0 || p.prefix_tokens <= 0) return cudaSuccess;
    const int D = c->head_dim;
    const int mt = c->model_dtype;
    const bool kv8 = c->kv_dtype == PKV_FP8_E4M3;
    Args a = base_args(c, p.scale);
    a.tables = p.tables;
    a.total_tokens = p.num_seqs;
    a.num_seqs = p.num_seqs;
    a.max_blocks = p.max_blocks;
    a.hq = p.num_q_heads;
    a.cost_bins = 1;
    a.ws_o = p.ws_o;
    a.ws_ml = p.ws_ml;
    a.max_splits = p.max_splits;
    a.prefix_tokens = p.prefix_tokens;
    a.split_tokens = p.split_tokens;
    a.nps = (p.prefix_tokens + p.split_tokens - 1) / p.split_tokens;
    const int64_t pairs = (int64_t)((p.num_seqs + BM - 1) / BM) * ((a.nps + 1) / 2);
    if (pairs * p.num_q_heads > 0x7FFFFFFF) return cudaErrorNotSupported;
    cudaError_t e = ensure_plan(c, 64);
    if (e != cudaSuccess) return e;
    a.plan = c->plan;
    const int64_t pool_rows = c->num_blocks * 2 * c->num_kv_heads * c->block_size;
    if (pool_rows > 0x7FFFFFFFLL) return cudaErrorNotSupported;
    // q [S][Hq][D] as rows of sequences: a box of 128 sequences x 64 dims of one head
    Maps m; // cascade: q and the pool (k, v, out unused)
    if (!make_map(&m.q, p.q, mt, p.num_seqs, (int64_t)p.num_q_heads * D, BM) || !pool_map(&m.pool, c))
        return cudaErrorInvalidValue;
    if (part == 1) {
        e = launch_plan(a, st);
        g_pkv_launches++;
        return e;
    }
    m.k = m.v = m.out = m.pool;
    e = kv8 ? dispatch<MODE_CASCADE, true>(D, mt, m, a, pairs * p.num_q_heads, c->num_sms, st)
            : dispatch<MODE_CASCADE, false>(D, mt, m, a, pairs * p.num_q_heads, c->num_sms, st);
    g_pkv_launches++;
    return e;
}

// ---------------------------------------------------------------- chunks of new tokens over the cache

namespace {
using namespace pkv_prefill;

// How a call of these sizes is cut: row tiles, key tiles of a split, splits of a row at most, items at most.
struct ChunkShape {
    bool stream;
    int split_steps, max_splits;
    int64_t groups, items; // (sequence, row tile or pair) at most; times the splits of each
    int max_groups;        // of a sequence
    // Few items: no list and no launch for it (one sequence of 2047 tokens: 16 us for 23).  Many: heaviest first from a list
    // (32 sequences of up to 4096 tokens, 32 heads, by turns: 224 us for 205).
    bool direct(const pkv_cache *c, int num_seqs) const { return rect(c, num_seqs) <= 2 * (int64_t)c->num_sms; }
    int64_t rect(const pkv_cache *c, int num_seqs) const {
        return (int64_t)num_seqs * max_groups * max_splits * c->num_kv_heads;
    }
    int64_t floats(const pkv_cache *c, int64_t tokens, int hq) const {
        const int64_t list = (4 + 4 * items + 63) / 64 * 64;
        return list + (max_splits > 1 ? tokens * hq * max_splits * (c->head_dim + 2) : 0);
    }
};

// Partial rows of a call of so many (token, head) rows over tables of so many key tiles, at most: what splits of 32 tiles
// need, or as many as fill the SMs (2 SMs / (row tiles KV heads) splits of tiles of at most 256 rows), and 2 GB.  A call
// whose q has more rows than its sequences can take (rows behind the last one, that nobody asks for) would be
// cut into more: it has few row tiles, but each split has room for all its rows.
int64_t most_partials(const pkv_cache *c, int64_t rows, int64_t steps) {
    const int64_t most = ((int64_t)1 << 29) / (c->head_dim + 2);
    if (rows >= most) return most;
    return std::min(most, rows * (steps / 32 + 3) + std::min<int64_t>(rows * steps, 2 * 256 * (int64_t)c->num_sms));
}
int64_t table_steps(const pkv_cache *c, int max_blocks) { return ((int64_t)max_blocks * c->block_size + BN - 1) / BN; }

ChunkShape chunk_shape(const pkv_cache *c, int num_seqs, int64_t tokens, int max_seqlen, int hq, int max_blocks, int window,
                       int sinks) {
    ChunkShape s;
    const int G = hq / c->num_kv_heads, bs = c->block_size;
    const int per = BM / G; // tokens of a row tile
    // One row tile a sequence: units by themselves, two at a time on an SM (chunk_stream.cuh).  More: tiles in pairs that share
    // their keys (prefill_impl.cuh), unless a sequence has two on average, so that most pairs would be half empty (64
    // sequences of 1 to 347 new tokens under a window, 2497 in all, G = 4: 137 us by themselves, 158 in pairs; 4 of 100 tokens
    // 164 and 123; one of 512 1185 and 1069).  Over E4M3 caches a pair's codes are widened once for both (512 tokens: 514
    // and 301).
    s.stream = max_seqlen <= per || (c->kv_dtype != PKV_FP8_E4M3 && tokens * G <= 2 * BM * (int64_t)num_seqs);
    const int group = s.stream ? per : 2 * per;
    const int64_t most = ((int64_t)max_seqlen + group - 1) / group; // of a sequence
    s.groups = std::min<int64_t>(num_seqs * most, tokens / group + num_seqs);
    int64_t keys = (int64_t)max_blocks * bs;
    if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window + std::min(max_seqlen, group) + sinks + 2 * bs);
    const int64_t steps = std::max<int64_t>(1, (keys + BN - 1) / BN);
    // splits of at most kMost key tiles, shorter where the items would not fill the SMs
    // (one sequence of 2047 tokens, 56 rows: 16 us with one tile a split, 20 with two, 25 with four; 512 tokens after
    // 131071: 1.11 ms with 32 tiles at most, 1.24 with 16, 1.16 with 64)
    constexpr int64_t kLeast = 1, kMost = 32;
    const int64_t places = (int64_t)c->num_sms * (s.stream ? 2 : 1);
    const int64_t share = (s.groups * c->num_kv_heads * steps + places - 1) / places;
    s.split_steps = (int)std::min(kMost, std::max(kLeast, share));
    s.max_splits = (int)((steps + s.split_steps - 1) / s.split_steps);
    // Longer ones where the partial rows of so many would be more than a call may have: their room follows from the
    // table's width, whatever the sequences hold (a piece of 8192 tokens, 64 heads, a table of 131072: 8.7 GB at 32).
    const int64_t fit = std::max<int64_t>(1, most_partials(c, tokens * hq, table_steps(c, max_blocks)) / (tokens * hq));
    if (s.max_splits > fit) {
        s.split_steps = (int)((steps + fit - 1) / fit);
        s.max_splits = (int)((steps + s.split_steps - 1) / s.split_steps);
    }
    s.max_groups = (int)most;
    s.items = s.groups * s.max_splits;
    return s;
}

template <bool STREAM>
cudaError_t launch_chunk_t(pkv_cache *c, const Args &a, const Maps &m, int64_t ctas, bool merge, cudaStream_t st) {
    const int D = c->head_dim, mt = c->model_dtype, smem = (2 * a.cost_bins + 32) * (int)sizeof(int);
    cudaError_t e;
    if (merge) {
        if (a.max_splits <= 1) return cudaSuccess;
        const dim3 grid((unsigned)a.total_tokens, (unsigned)((a.hq + 3) / 4));
        auto kern = D == 128 ? (mt == PKV_F16 ? chunk_merge_kernel<128, PKV_F16, STREAM> : chunk_merge_kernel<128, PKV_BF16, STREAM>)
                             : (mt == PKV_F16 ? chunk_merge_kernel<64, PKV_F16, STREAM> : chunk_merge_kernel<64, PKV_BF16, STREAM>);
        e = pdl_launch(kern, grid, dim3(128), 0, st, a);
        g_pkv_launches++;
        return e;
    }
    if (a.plan) {
        static std::atomic<bool> allowed[64] = {};
        e = pkv_allow_smem(reinterpret_cast<const void *>(chunk_plan_kernel<STREAM>), allowed);
        if (e != cudaSuccess) return e;
        e = pdl_launch(chunk_plan_kernel<STREAM>, dim3(1), dim3(kPlanThreads), smem, st, a);
        g_pkv_launches++;
        if (e != cudaSuccess) return e;
    }
    const bool kv8 = c->kv_dtype == PKV_FP8_E4M3;
    if constexpr (STREAM) {
        const bool few = (int64_t)a.max_seqlen << a.lg_group <= 64;
        const int grid = (int)std::min<int64_t>(ctas, c->num_sms);
        e = kv8 ? (few ? launch_stream_any<true, true>(D, mt, m.q, m.pool, a, grid, st)
                       : launch_stream_any<true, false>(D, mt, m.q, m.pool, a, grid, st))
                : (few ? launch_stream_any<false, true>(D, mt, m.q, m.pool, a, grid, st)
                       : launch_stream_any<false, false>(D, mt, m.q, m.pool, a, grid, st));
    } else {
        e = kv8 ? dispatch<MODE_CHUNK, true>(D, mt, m, a, ctas, c->num_sms, st)
                : dispatch<MODE_CHUNK, false>(D, mt, m, a, ctas, c->num_sms, st);
    }
    g_pkv_launches++;
    return e;
}

// Sequences of up to so many rows a KV head are taken apart from the others, by chunk_few.cuh beside the tcgen05 kernel; 0:
// none.  Where the longest piece is four times the mean one or more, as a batch of single tokens with a few pieces of prompts
// has it.  (Window 1024, 32/8 heads, 64 sequences of 1 to 347 new tokens: bf16 140 us by one kernel, 134 by two,
// 16 rows 136; one head a KV head 96 and 79; E4M3 133 and 107, 8 rows 115; 255 single tokens after 2048 and a piece of 128:
// bf16 391 and 344, E4M3 539 and 264.  16 bf16 sequences of that window 51 and 56.)
int rows_apart(const pkv_cache *c, const ChunkLaunch &p) {
    const bool fp8 = c->kv_dtype == PKV_FP8_E4M3;
    if (p.num_seqs < (fp8 ? 8 : 32) || (int64_t)p.num_seqs * p.max_seqlen < 4 * p.total_tokens) return 0;
    return fp8 ? 16 : 8;
}
} // namespace

int64_t chunk_workspace_floats(const pkv_cache *c, int num_seqs, int64_t tokens, int max_seqlen, int hq, int max_blocks) {
    // A call of fewer rows may be cut into more splits: what chunk_shape can make of any sizes up to these.
    const int64_t steps = table_steps(c, max_blocks), splits = steps / 32 + 3;
    const int64_t partials = most_partials(c, tokens > INT64_MAX / hq ? INT64_MAX : tokens * hq, steps);
    const int64_t groups = std::min<int64_t>(num_seqs * (((int64_t)max_seqlen + 15) / 16), tokens / 16 + num_seqs);
    const int64_t items = groups * splits + std::min<int64_t>(groups * steps, 2 * (int64_t)c->num_sms);
    // (a call may take the sequences of few rows apart from the others)
    return (4 + 4 * items + 63) / 64 * 64 + (partials * (c->head_dim + 2) + 63) / 64 * 64 +
           few_workspace_floats(c, num_seqs, max_blocks);
}

int chunk_entry(pkv_cache *c, const ChunkLaunch &p, cudaStream_t st) {
    const int hq = p.num_q_heads, D = c->head_dim, mt = c->model_dtype;
    int few = chunk_few_rows(c, p);
    if ((int64_t)p.max_seqlen * (hq / c->num_kv_heads) <= few) { // every sequence
        std::lock_guard<std::mutex> lk(c->ws_mu);
        PkvWorkspace ws;
        if (int r = pkv_stream_workspace(c, st, chunk_few_floats(c, p, few), &ws)) return r;
        PkvTimer timer(c, PKV_KIND_PREFILL, st);
        return chunk_few_launch(c, p, few, false, ws.p, st);
    }
    few = rows_apart(c, p);
    const ChunkShape s = chunk_shape(c, p.num_seqs, p.total_tokens, p.max_seqlen, hq, p.max_blocks, p.window, p.sinks);
    if (s.items * c->num_kv_heads > 0x7FFFFFFF || p.total_tokens > 1 << 30)
        return pkv_fail(PKV_EUNSUPPORTED, "too many rows for one call");
    if (p.window > 1 << 30) return pkv_fail(PKV_EUNSUPPORTED, "a window of more than 2^30 tokens in wider tables");
    const int64_t pool_rows = c->num_blocks * 2 * c->num_kv_heads * c->block_size;
    if (pool_rows > 0x7FFFFFFFLL) return pkv_fail(PKV_EUNSUPPORTED, "pools of more than 2^31 - 1 rows");
    Args a = base_args(c, p.scale);
    a.out = p.out;
    a.cu = p.cu;
    a.tables = p.tables;
    a.lens = p.lens;
    a.total_tokens = p.total_tokens;
    a.num_seqs = p.num_seqs;
    a.max_seqlen = p.max_seqlen;
    a.max_blocks = p.max_blocks;
    a.hq = hq;
    a.window = p.window;
    a.sinks = p.sinks;
    a.lg_group = lg2(hq / c->num_kv_heads);
    a.split_steps = s.split_steps;
    a.max_splits = s.max_splits;
    a.plan_cap = s.items;
    a.cost_bins = std::min(2 * s.split_steps + 2, 16384); // (the longest splits of the widest tables count alike)
    Maps m;
    const int G = hq / c->num_kv_heads, tile = s.stream && (int64_t)p.max_seqlen * G <= 64 ? 64 : BM;
    if (!make_group_map(&m.q, p.q, mt, p.total_tokens, hq, D, G, tile) ||
        (!s.stream && !make_group_map(&m.out, p.out, mt, p.total_tokens, hq, D, G)) || // (TMA stores of whole tiles)
        !(D == 128 && c->kv_dtype != PKV_FP8_E4M3 ? pkv_tmap_rows128_grouped(&m.pool, c->pool, mt, pool_rows, c->block_size)
                                                  : pool_map(&m.pool, c)))
        return pkv_fail(PKV_ECUDA, "tensor map");
    m.k = m.v = m.pool;
    std::lock_guard<std::mutex> lk(c->ws_mu);
    PkvWorkspace ws;
    const int64_t floats = (s.floats(c, p.total_tokens, hq) + 63) / 64 * 64;
    if (int r = pkv_stream_workspace(c, st, floats + (few ? chunk_few_floats(c, p, few) : 0), &ws)) return r;
    const bool direct = s.direct(c, p.num_seqs);
    a.plan = direct ? nullptr : reinterpret_cast<int *>(ws.p);
    a.max_groups = s.max_groups;
    if (direct) {
        a.max_parts = s.max_splits;
        a.rect = (int)s.rect(c, p.num_seqs);
    }
    a.ws_o = ws.p + (4 + 4 * s.items + 63) / 64 * 64;
    a.ws_ml = a.ws_o + p.total_tokens * hq * s.max_splits * D;
    PkvTimer timer(c, PKV_KIND_PREFILL, st);
    const int64_t ctas = direct ? a.rect : s.items * c->num_kv_heads;
    a.few_rows = few;
    for (const bool merge : {false, true}) {
        const cudaError_t e = s.stream ? launch_chunk_t<true>(c, a, m, ctas, merge, st) : launch_chunk_t<false>(c, a, m, ctas, merge, st);
        if (e != cudaSuccess) return pkv_cuda_fail(e, "chunk attention launch");
        if (few && !merge)
            if (int r = chunk_few_launch(c, p, few, true, ws.p + floats, st)) return r;
    }
    return PKV_OK;
}
