// Slot indexing and paged KV append.
//
// Slot indexing: token t of sequence s goes to physical block block_table[s][t / bs] at
// offset t % bs ("Paged KV Cache 与 Packed Sequence", discosf.com, section 2.2).
// Append: the new token's K/V is written at exactly that (block, offset) and nowhere else
// ("PagedAttention 与前缀缓存", 2kiu.com, section 4.1 step 3 and section 6.3).
//
// Both are HBM-bound scatter/gather work: 16-byte vector loads and stores, one thread per
// 16-byte source chunk, consecutive threads on consecutive chunks of a (token, K|V, head)
// row so that every warp moves whole contiguous 256-byte rows.  The fused variant computes
// each token's slot in the same kernel (and still returns the slots), which saves a launch
// per decode step.  All kernels are launched with programmatic dependent launch: they let the
// next kernel in the stream start its launch early and wait for their own predecessor before
// touching global memory.
//
// A 4-bit cache's rows are quantised on the way (append4_kernel, below); gather_kernel reads the rows
// of any cache back in the model's type.
#include "device_common.cuh"
#include "int4.cuh"
#include "pkv_internal.h"

namespace {

__global__ void slot_mapping_kernel(const int32_t *__restrict__ tables, int rows, int max_blocks,
                                    const int32_t *__restrict__ seq_ids, const int32_t *__restrict__ positions,
                                    int64_t n, int bs, int64_t *__restrict__ out) {
    pdl_trigger();
    pdl_wait();
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
        out[i] = slot_of(tables, rows, max_blocks, seq_ids[i], positions[i], bs);
}

struct AppendArgs {
    const uint4 *k, *v;   // [n][Hkv][D] model dtype, viewed as 16-byte chunks
    const int64_t *slots; // given slots (plain append) ...
    const int32_t *tables, *seq_ids, *positions; // ... or computed here (fused append)
    const int32_t *cu, *ctx; // ... or from packed ranges: token j of [cu[i], cu[i+1]) at position ctx[i] + j - cu[i]
                             // (ctx NULL: position j - cu[i])
    int64_t *slots_out;
    int rows, max_blocks;
    char *pool;
    const float *k_scale, *v_scale;
    unsigned int *err;
    int64_t n, num_slots;
    int hkv, bs, chunks_per_row; // chunks_per_row = D / 8
    int64_t tile_elems;          // bs * D
    int d, bs_log2;
};

// KVT: 0 = 16-bit cache (bit copy), 2 = E4M3 cache; MT = model dtype for the E4M3 path;
// MODE: 0 = slots given, 1 = slot from (table, sequence id, position) per token, 2 = sequence and
// position from packed ranges (cu_seqlens, context lengths), then the slot as in mode 1
enum { SLOTS_GIVEN = 0, SLOTS_AT = 1, SLOTS_RANGES = 2 };
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4; // chunks a thread loads before it stores any

// The slot of token j (mode-specific), or -1 for "skip".
template <int MODE>
PKV_DEV int64_t append_slot(const AppendArgs &a, int64_t j) {
    if constexpr (MODE == SLOTS_AT) {
        return slot_of(a.tables, a.rows, a.max_blocks, a.seq_ids[j], a.positions[j], a.bs);
    } else if constexpr (MODE == SLOTS_RANGES) {
        // sequence: the largest i with cu[i] <= j (a.rows = number of sequences)
        int lo = 0, hi = a.rows;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= j)
                lo = mid;
            else
                hi = mid;
        }
        const int64_t st = a.cu[lo], en = a.cu[lo + 1];
        const int c0 = a.ctx ? a.ctx[lo] : 0; // no context lengths: every sequence starts at position 0
        const int64_t pos = (int64_t)c0 + (j - st);
        return (j >= st && j < en && c0 >= 0 && pos <= 0x7FFFFFFF)
                   ? slot_of(a.tables, a.rows, a.max_blocks, lo, (int)pos, a.bs)
                   : -1;
    } else {
        return a.slots[j];
    }
}

// Token-major: a pass of the CTA covers whole tokens, tpg = max(1, threads / chunks per token) of
// them, so a token's slot is found once per thread rather than once per 16-byte chunk, and each
// thread issues the loads of up to kAppendUnroll chunks before it stores any of them.
template <int KVT, int MT, int MODE>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
    pdl_trigger();
    pdl_wait();
    const int row_chunks = a.hkv * a.chunks_per_row; // one (token, K|V) row over all heads
    const int per_token = 2 * row_chunks;
    const int tpg = per_token >= kAppendThreads ? 1 : kAppendThreads / per_token;
    const int lt = tpg > 1 ? (int)threadIdx.x / per_token : 0; // this thread's token in the pass
    const int r0 = tpg > 1 ? (int)threadIdx.x - lt * per_token : (int)threadIdx.x;
    const int rstep = tpg > 1 ? per_token : kAppendThreads;
    if (lt >= tpg) return; // threads past the last whole token of a pass
    for (int64_t j = (int64_t)blockIdx.x * tpg + lt; j < a.n; j += (int64_t)gridDim.x * tpg) {
        const int64_t slot = append_slot<MODE>(a, j);
        if (MODE != SLOTS_GIVEN && r0 == 0 && a.slots_out) a.slots_out[j] = slot;
        if (slot < 0) continue;
        if (slot >= a.num_slots) {
            if (r0 == 0) set_error(a.err, PKV_DEVERR_SLOT);
            continue;
        }
        const int64_t blk = slot / a.bs;
        const int off = static_cast<int>(slot - blk * a.bs);
        // element index of (blk, kv = 0, h = 0, off, 0) in the [NB][2][Hkv][bs][D] pool
        const int64_t e0 = blk * 2 * a.hkv * a.tile_elems + (int64_t)off * a.d;
        const uint4 *ksrc = a.k + j * row_chunks, *vsrc = a.v + j * row_chunks;
        for (int rb = r0; rb < per_token; rb += kAppendUnroll * rstep) {
            uint4 src[kAppendUnroll];
            int64_t dst[kAppendUnroll];
            int kvs[kAppendUnroll], hs[kAppendUnroll];
#pragma unroll
            for (int u = 0; u < kAppendUnroll; ++u) {
                const int r = rb + u * rstep;
                dst[u] = -1;
                if (r < per_token) {
                    const int kv = r >= row_chunks ? 1 : 0;
                    const int hc = r - kv * row_chunks;
                    const int h = hc / a.chunks_per_row;
                    const int c = hc - h * a.chunks_per_row;
                    src[u] = (kv ? vsrc : ksrc)[hc];
                    dst[u] = e0 + (int64_t)(kv * a.hkv + h) * a.tile_elems + c * 8;
                    kvs[u] = kv;
                    hs[u] = h;
                }
            }
#pragma unroll
            for (int u = 0; u < kAppendUnroll; ++u) {
                if (dst[u] < 0) continue;
                if constexpr (KVT != PKV_FP8_E4M3) {
                    reinterpret_cast<uint4 *>(a.pool)[dst[u] / 8] = src[u];
                } else {
                    float f[8];
                    cvt8<MT>(src[u], f);
                    const float sc = (kvs[u] ? a.v_scale : a.k_scale)[hs[u]];
                    uint2 o;
                    o.x = e4m3x2_from_f32(__fdiv_rn(f[0], sc), __fdiv_rn(f[1], sc)) |
                          (e4m3x2_from_f32(__fdiv_rn(f[2], sc), __fdiv_rn(f[3], sc)) << 16);
                    o.y = e4m3x2_from_f32(__fdiv_rn(f[4], sc), __fdiv_rn(f[5], sc)) |
                          (e4m3x2_from_f32(__fdiv_rn(f[6], sc), __fdiv_rn(f[7], sc)) << 16);
                    reinterpret_cast<uint2 *>(a.pool)[dst[u] / 8] = o;
                }
            }
        }
    }
}

// 4-bit append.  Per (token, K|V, KV head) row x[0 .. D): z = min x, s = RN((max x - min x) / 15) in the
// model's type, code = min(15, rint((x - z) / s)); int4.cuh has the layout and the border cases.  D / 16 lanes
// share a row, sixteen elements each (a 16-byte load from each half of the row, so that lanes lie side by side): the
// extremes meet by xor shuffles in the NaN-propagating forms, so a NaN anywhere reaches s, and each lane writes the four
// bytes of its codes in either half.  Bound by HBM (4 D bytes read and D + 8 written per token and head) and the
// ALU alike, 243 instructions a warp for sixteen elements a lane: with eight a lane the row's own work (range, step,
// reciprocal) cost as much as the codes, and reading tokens ahead into shared memory only added instructions.
// 5256 tokens x 32 heads, D = 128, written and read back: 43 us, 218 MB, 5.0 TB/s.
constexpr int kAppend4Ctas = 12; // of an SM, twice what fits: each takes several tokens (32: 44.1 us above, 6: 46.1)

template <int D, int MT, int MODE>
__global__ void __launch_bounds__(kAppendThreads) append4_kernel(AppendArgs a) {
    pdl_trigger();
    pdl_wait();
    constexpr int per_row = D / 16;
    const int side = a.hkv * per_row, per_token = 2 * side;
    const int tpg = per_token >= kAppendThreads ? 1 : kAppendThreads / per_token;
    const int lt = tpg > 1 ? (int)threadIdx.x / per_token : 0;
    const int r0 = tpg > 1 ? (int)threadIdx.x - lt * per_token : (int)threadIdx.x;
    const int rstep = tpg > 1 ? per_token : kAppendThreads;
    if (lt >= tpg) return;
    // the lanes that share a row: per_token, rstep and kAppendThreads are multiples of per_row (8 or 4), so they
    // take every branch below together
    const unsigned lanes = ((1u << per_row) - 1u) << ((threadIdx.x & 31) & ~(per_row - 1));
    for (int64_t j = (int64_t)blockIdx.x * tpg + lt; j < a.n; j += (int64_t)gridDim.x * tpg) {
        const int64_t slot = append_slot<MODE>(a, j);
        if (MODE != SLOTS_GIVEN && r0 == 0 && a.slots_out) a.slots_out[j] = slot;
        if (slot < 0) continue;
        if (slot >= a.num_slots) {
            if (r0 == 0) set_error(a.err, PKV_DEVERR_SLOT);
            continue;
        }
        const int64_t blk = slot >> a.bs_log2;
        const int off = static_cast<int>(slot) & (a.bs - 1);
        const uint4 *ksrc = a.k + j * side * 2, *vsrc = a.v + j * side * 2;
        for (int r = r0; r < per_token; r += rstep) {
            const uint4 *p = (r >= side ? vsrc - side * 2 : ksrc) + r / per_row * (2 * per_row) + r % per_row;
            const uint4 src[2] = {__ldcs(p), __ldcs(p + per_row)};
            const int kv = r >= side ? 1 : 0, hc = r - kv * side, h = hc / per_row, c = hc - h * per_row;
            const Int4Row row = int4_quantise<MT>(src, per_row, lanes);
            char *tile = a.pool + int4_head(blk, h, a.hkv, a.bs, D);
            *reinterpret_cast<uint32_t *>(tile + int4_codes(kv, off, c * 4, D)) = row.codes.x;
            *reinterpret_cast<uint32_t *>(tile + int4_codes(kv, off, D / 4 + c * 4, D)) = row.codes.y;
            if (c == 0) *reinterpret_cast<uint32_t *>(tile + int4_params(kv, off, D)) = row.params;
        }
    }
}

// Rows read back: token j's K and V at slots[j] in the model's type (a 4- or 8-bit row's values, rounded
// once; a 16-bit row's bits).  A negative slot gives a row of zeros, one past the pool zeros and
// PKV_DEVERR_SLOT.  Bound by HBM; sixteen elements a thread, half of them from either half of a row so that lanes lie side
// by side, two rows' loads before their stores (one: as fast for 4-bit rows; four: 45.4 us for 43.3 above).
struct GatherArgs {
    uint4 *k, *v;
    const int64_t *slots;
    const char *pool;
    const float *k_scale, *v_scale;
    unsigned int *err;
    int64_t n, num_slots;
    int hkv, bs_log2;
};
constexpr int kGatherUnroll = 2, kGatherCtas = 12; // CTAs of an SM, as kAppend4Ctas

template <int D, int KVT, int MT>
__global__ void __launch_bounds__(kAppendThreads) gather_kernel(GatherArgs a) {
    using M = ModelT<MT>;
    pdl_trigger();
    pdl_wait();
    constexpr int per_row = D / 16;
    constexpr int kWords = KVT == PKV_INT4 ? 2 : KVT == PKV_FP8_E4M3 ? 4 : 8; // of sixteen stored elements
    const int side = a.hkv * per_row, per_token = 2 * side, bs = 1 << a.bs_log2;
    const int tpg = per_token >= kAppendThreads ? 1 : kAppendThreads / per_token;
    const int lt = tpg > 1 ? (int)threadIdx.x / per_token : 0;
    const int r0 = tpg > 1 ? (int)threadIdx.x - lt * per_token : (int)threadIdx.x;
    const int rstep = tpg > 1 ? per_token : kAppendThreads;
    if (lt >= tpg) return;
    for (int64_t j = (int64_t)blockIdx.x * tpg + lt; j < a.n; j += (int64_t)gridDim.x * tpg) {
        int64_t slot = a.slots[j];
        if (slot >= a.num_slots) {
            if (r0 == 0) set_error(a.err, PKV_DEVERR_SLOT);
            slot = -1;
        }
        const int64_t blk = slot < 0 ? 0 : slot >> a.bs_log2;
        const int off = slot < 0 ? 0 : static_cast<int>(slot) & (bs - 1);
        for (int rb = r0; rb < per_token; rb += kGatherUnroll * rstep) {
            uint32_t x[kGatherUnroll][kWords], par[kGatherUnroll];
#pragma unroll
            for (int u = 0; u < kGatherUnroll; ++u) {
                const int r = rb + u * rstep;
                if (r >= per_token || slot < 0) continue;
                const int kv = r >= side ? 1 : 0, hc = r - kv * side, h = hc / per_row, c = hc - h * per_row;
                if constexpr (KVT == PKV_INT4) {
                    const char *tile = a.pool + int4_head(blk, h, a.hkv, bs, D);
                    x[u][0] = __ldcs(reinterpret_cast<const uint32_t *>(tile + int4_codes(kv, off, c * 4, D)));
                    x[u][1] = __ldcs(reinterpret_cast<const uint32_t *>(tile + int4_codes(kv, off, D / 4 + c * 4, D)));
                    par[u] = *reinterpret_cast<const uint32_t *>(tile + int4_params(kv, off, D));
                } else {
                    const char *p = a.pool + ((((blk * 2 + kv) * a.hkv + h) << a.bs_log2) + off) * (D * kWords / 4) +
                                    c * kWords * 2;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (KVT == PKV_FP8_E4M3) {
                            const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p + i * (D / 2)));
                            x[u][2 * i] = w.x;
                            x[u][2 * i + 1] = w.y;
                        } else {
                            const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p + i * D));
                            x[u][4 * i] = w.x;
                            x[u][4 * i + 1] = w.y;
                            x[u][4 * i + 2] = w.z;
                            x[u][4 * i + 3] = w.w;
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kGatherUnroll; ++u) {
                const int r = rb + u * rstep;
                if (r >= per_token) continue;
                const int kv = r >= side ? 1 : 0, hc = r - kv * side;
                uint4 o[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (slot >= 0) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (KVT == PKV_INT4) {
                            o[i] = int4_values<MT>(x[u][i], par[u]);
                        } else if constexpr (KVT == PKV_FP8_E4M3) {
                            const float sc = (kv ? a.v_scale : a.k_scale)[hc / per_row];
                            float f[8];
                            cvt8_e4m3(make_uint2(x[u][2 * i], x[u][2 * i + 1]), f);
                            o[i] = make_uint4(M::pack(f[0] * sc, f[1] * sc), M::pack(f[2] * sc, f[3] * sc),
                                              M::pack(f[4] * sc, f[5] * sc), M::pack(f[6] * sc, f[7] * sc));
                        } else {
                            o[i] = make_uint4(x[u][4 * i], x[u][4 * i + 1], x[u][4 * i + 2], x[u][4 * i + 3]);
                        }
                    }
                }
                uint4 *dst = (kv ? a.v : a.k) + j * side * 2 + hc / per_row * (2 * per_row) + hc % per_row;
                dst[0] = o[0];
                dst[per_row] = o[1];
            }
        }
    }
}

inline int grid_for(int64_t work, int threads, int num_sms) {
    const int64_t blocks = (work + threads - 1) / threads;
    const int64_t cap = (int64_t)num_sms * 16;
    return static_cast<int>(blocks < 1 ? 1 : (blocks > cap ? cap : blocks));
}

AppendArgs base_args(pkv_cache *c, const void *k, const void *v, int64_t n) {
    AppendArgs a{};
    a.k = static_cast<const uint4 *>(k);
    a.v = static_cast<const uint4 *>(v);
    a.pool = static_cast<char *>(c->pool);
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.err = c->err;
    a.n = n;
    a.num_slots = c->num_blocks * c->block_size;
    a.hkv = c->num_kv_heads;
    a.bs = c->block_size;
    a.chunks_per_row = c->head_dim / 8;
    a.tile_elems = (int64_t)c->block_size * c->head_dim;
    a.d = c->head_dim;
    a.bs_log2 = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
    return a;
}

template <int MODE>
cudaError_t launch_append_t(pkv_cache *c, const AppendArgs &a, cudaStream_t st) {
    // one CTA pass per tpg tokens (see append_kernel), up to 8 resident CTAs per SM
    const int per_token = 2 * a.hkv * a.chunks_per_row;
    const int tpg = per_token >= kAppendThreads ? 1 : kAppendThreads / per_token;
    const int64_t passes = (a.n + tpg - 1) / tpg;
    const int64_t cap = (int64_t)c->num_sms * (c->kv_dtype == PKV_INT4 ? kAppend4Ctas : 8);
    const dim3 grid((unsigned)(passes < 1 ? 1 : (passes > cap ? cap : passes)));
    PkvTimer timer(c, PKV_KIND_APPEND, st);
    cudaError_t e;
    if (c->kv_dtype == PKV_INT4) {
        auto kern = c->head_dim == 64
                        ? (c->model_dtype == PKV_F16 ? append4_kernel<64, PKV_F16, MODE> : append4_kernel<64, PKV_BF16, MODE>)
                        : (c->model_dtype == PKV_F16 ? append4_kernel<128, PKV_F16, MODE>
                                                     : append4_kernel<128, PKV_BF16, MODE>);
        e = pdl_launch(kern, grid, dim3(kAppendThreads), 0, st, a);
    } else if (c->kv_dtype != PKV_FP8_E4M3)
        e = pdl_launch(append_kernel<PKV_F16, PKV_F16, MODE>, grid, dim3(kAppendThreads), 0, st, a);
    else if (c->model_dtype == PKV_F16)
        e = pdl_launch(append_kernel<PKV_FP8_E4M3, PKV_F16, MODE>, grid, dim3(kAppendThreads), 0, st, a);
    else
        e = pdl_launch(append_kernel<PKV_FP8_E4M3, PKV_BF16, MODE>, grid, dim3(kAppendThreads), 0, st, a);
    g_pkv_launches++;
    return e;
}

} // namespace

cudaError_t launch_slot_mapping(const int32_t *tables, int rows, int max_blocks, const int32_t *seq_ids,
                                const int32_t *positions, int64_t n, int bs, int64_t *out, cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const cudaError_t e = pdl_launch(slot_mapping_kernel, dim3(grid_for(n, 256, sms)), dim3(256), 0, st, tables, rows,
                                     max_blocks, seq_ids, positions, n, bs, out);
    g_pkv_launches++;
    return e;
}

cudaError_t launch_append(pkv_cache *c, const void *k, const void *v, const int64_t *slots, int64_t n,
                          cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    AppendArgs a = base_args(c, k, v, n);
    a.slots = slots;
    return launch_append_t<SLOTS_GIVEN>(c, a, st);
}

cudaError_t launch_append_at(pkv_cache *c, const void *k, const void *v, const int32_t *tables, int rows,
                             int max_blocks, const int32_t *seq_ids, const int32_t *positions, int64_t n,
                             int64_t *slots_out, cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    AppendArgs a = base_args(c, k, v, n);
    a.tables = tables;
    a.rows = rows;
    a.max_blocks = max_blocks;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.slots_out = slots_out;
    return launch_append_t<SLOTS_AT>(c, a, st);
}

cudaError_t launch_append_ranges(pkv_cache *c, const void *k, const void *v, const int32_t *tables, int num_seqs,
                                 int max_blocks, const int32_t *cu, const int32_t *ctx, int64_t n, cudaStream_t st) {
    if (n == 0 || num_seqs <= 0) return cudaSuccess;
    AppendArgs a = base_args(c, k, v, n);
    a.tables = tables;
    a.rows = num_seqs;
    a.max_blocks = max_blocks;
    a.cu = cu;
    a.ctx = ctx;
    return launch_append_t<SLOTS_RANGES>(c, a, st);
}

cudaError_t launch_gather(pkv_cache *c, const int64_t *slots, int64_t n, void *k, void *v, cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    GatherArgs a{};
    a.k = static_cast<uint4 *>(k);
    a.v = static_cast<uint4 *>(v);
    a.slots = slots;
    a.pool = static_cast<const char *>(c->pool);
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.err = c->err;
    a.n = n;
    a.num_slots = c->num_blocks * c->block_size;
    a.hkv = c->num_kv_heads;
    a.bs_log2 = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
    const int per_token = 2 * a.hkv * (c->head_dim / 16);
    const int tpg = per_token >= kAppendThreads ? 1 : kAppendThreads / per_token;
    const int64_t passes = (n + tpg - 1) / tpg, cap = (int64_t)c->num_sms * kGatherCtas;
    const dim3 grid((unsigned)(passes > cap ? cap : passes)), block(kAppendThreads);
    const bool d64 = c->head_dim == 64, h = c->model_dtype == PKV_F16;
    PkvTimer timer(c, PKV_KIND_COPY, st);
    g_pkv_launches++;
    if (c->kv_dtype == PKV_INT4) {
        auto kern = d64 ? (h ? gather_kernel<64, PKV_INT4, PKV_F16> : gather_kernel<64, PKV_INT4, PKV_BF16>)
                        : (h ? gather_kernel<128, PKV_INT4, PKV_F16> : gather_kernel<128, PKV_INT4, PKV_BF16>);
        return pdl_launch(kern, grid, block, 0, st, a);
    }
    if (c->kv_dtype == PKV_FP8_E4M3) {
        auto kern = d64 ? (h ? gather_kernel<64, PKV_FP8_E4M3, PKV_F16> : gather_kernel<64, PKV_FP8_E4M3, PKV_BF16>)
                        : (h ? gather_kernel<128, PKV_FP8_E4M3, PKV_F16> : gather_kernel<128, PKV_FP8_E4M3, PKV_BF16>);
        return pdl_launch(kern, grid, block, 0, st, a);
    }
    return pdl_launch(d64 ? gather_kernel<64, PKV_F16, PKV_F16> : gather_kernel<128, PKV_F16, PKV_F16>, grid, block, 0, st, a);
}
