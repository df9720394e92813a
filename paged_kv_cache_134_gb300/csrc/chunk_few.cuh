// Chunk attention of few rows: up to 8 C query rows of a KV head (new tokens times the heads that share it), C = 1, 2, 3.
//
// out[r] = sum_t p_t V_t with p_t = softmax_t(scale * q_r . K_t) over the tokens t that row r sees: t <= p_r, and under a
// window t > p_r - window or t < sinks; rows r = (new token r / G, head r % G) of a sequence's KV head.
//
// decode_mma.cuh's kernel with C groups of eight columns: K and V tiles travel global -> shared -> register once and
// meet every group there (an E4M3 code is widened once for all rows).  Bound by the bytes of the cache for one group
// and by the tiles' chains beside it (scores, exponentials, products: eight to twelve warps an SM) for more: 32
// sequences of up to 4096 tokens, 5 new ones, 32 fp16 heads 161 us (1.01 GB, 6.3 TB/s); 256 log-normal ones of up to
// 8192, 32/8 heads, E4M3, 2 new tokens (one group) 99 us, 4 (two) 131 (455 MB).  P goes into the second product as a
// pair hi + lo, of fp16 (2^-22; weights of the base at 2^6 and at most at 2^14, so that they stay normal numbers down
// to 2^-20 of it) or bf16 (2^-16), or as one fp16 (2^-11) where an E4M3 cache's outputs are bf16 (2^-8); scores,
// statistics, sums and accumulators are fp32.  A tile is masked only where a row's end or its window's begin crosses
// it.  The four warps' sums meet in one buffer, added in turn (four barriers for four times the memory).
#pragma once

#include "decode_mma.cuh"

namespace pkv_mma {

// new tokens of sequence s; 0 where its numbers make no sense, or where it has more rows than this kernel's share
PKV_DEV int new_tokens(const FewArgs &a, int s, bool report = false) {
    const int64_t st = a.cu[s], n = a.cu[s + 1] - st;
    if (st < 0 || n < 0 || st + n > a.total || n > a.max_seqlen) {
        if (report) set_error(a.err, PKV_DEVERR_CU_SEQLENS);
        return 0;
    }
    if (n > 0 && (int64_t)a.lens[s] > a.cap) {
        if (report) set_error(a.err, PKV_DEVERR_LENGTH);
        return 0;
    }
    return n > a.most_rows >> a.lg_group ? 0 : (int)n;
}
PKV_DEV void report_row(const FewArgs &a, int s) { new_tokens(a, s, true); }
PKV_DEV bool has_rows(const FewArgs &a, int s) { return new_tokens(a, s) > 0; }
PKV_DEV int row_len(const FewArgs &a, int s) { return has_rows(a, s) ? max(a.lens[s], 0) : 0; }
// what the rows of a sequence see together
template <bool WIN>
PKV_DEV Reach sight_of(const FewArgs &a, int s, int L) {
    if (a.window == 0) return {L, 0, 0, 0, 0};
    return reach_of(L, a.window + new_tokens(a, s) - 1, a.sinks, 1 << a.bs_log2); // (the window is at most 2^30)
}

struct FewUnit : SeenUnit {
    int start, rows; // first token's row of q; rows (token, head)
    int c0;          // the last token that the first new token sees, in the order of what is in sight
};
PKV_DEV FewUnit few_unit(const FewArgs &a, const int *full, const int *part, int nfull, int u) {
    FewUnit r;
    static_cast<SeenUnit &>(r) = unit_of<true>(a, full, part, nfull, u);
    const int n = new_tokens(a, r.s);
    r.start = n > 0 ? a.cu[r.s] : 0;
    r.rows = n << a.lg_group;
    r.c0 = part[a.num_seqs + 1 + r.s] - n - (r.skip << a.bs_log2);
    return r;
}
// row r of a unit among all (token, head) rows
PKV_DEV int64_t few_row(const FewArgs &a, int start, int kvh, int r) {
    return (int64_t)(start + (r >> a.lg_group)) * a.hq + (kvh << a.lg_group) + (r & (a.group - 1));
}

// A split's first partial row.  (A split's rows side by side, as its unit writes them; a row's splits side by side
// instead: one sequence of 32768 tokens 29.4 us for 23.9, of 2047 15.2 for 12.8.)
PKV_DEV int64_t few_room(const FewArgs &a, int s, int kvh, int j) {
    return (((int64_t)s * a.hkv + kvh) * a.max_splits + j) * a.row_room;
}

// Joins one row's splits, 32 at a time in their order; a warp.  The partial rows of eight splits are on their way at once.
template <int D, int MT>
PKV_DEV void few_join(const FewArgs &a, int64_t room, int64_t row, int nsplit) {
    using M_ = ModelT<MT>;
    constexpr int N = D / 32, U = 8;
    using Vec = std::conditional_t<N == 4, float4, float2>;
    const int lane = threadIdx.x & 31;
    const float2 *ml = reinterpret_cast<const float2 *>(a.ws_ml) + room;
    const float *o = a.ws_o + room * D + lane * N;
    const int64_t step = (int64_t)a.row_room * D;
    float M = -INFINITY, den = 0.f, acc[N] = {};
    for (int j0 = 0; j0 < nsplit; j0 += 32) {
        const int n = min(32, nsplit - j0);
        const float2 v = lane < n ? __ldcg(ml + (int64_t)(j0 + lane) * a.row_room) : make_float2(-INFINITY, 0.f);
        float top = v.x;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        top = fmaxf(top, M);
        const float back = weight_of(M, top), w = lane < n ? weight_of(v.x, top) : 0.f;
        M = top;
        float sum = lane < n ? w * v.y : 0.f;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (j0 > 0) {
            den *= back;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] *= back;
        }
        den += sum;
        for (int j = 0; j < n; j += U) {
            Vec x[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (j + i < n) x[i] = __ldcg(reinterpret_cast<const Vec *>(o + (j0 + j + i) * step));
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float f = __shfl_sync(0xffffffffu, w, (j + i) & 31);
                if (j + i < n) {
                    acc[0] = fmaf(f, x[i].x, acc[0]);
                    acc[1] = fmaf(f, x[i].y, acc[1]);
                    if constexpr (N == 4) {
                        acc[2] = fmaf(f, x[i].z, acc[2]);
                        acc[3] = fmaf(f, x[i].w, acc[3]);
                    }
                }
            }
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<char *>(a.out) + (row * D + lane * N) * 2);
#pragma unroll
    for (int i = 0; i < N; i += 2) dst[i / 2] = den == 0.f ? 0u : M_::pack(acc[i] * inv, acc[i + 1] * inv);
}

// Rows of more than one split: a warp a row.  (A launch of its own, not the row's last CTA as in decode_mma.cuh: it joins up
// to 16 splits of up to 24 rows, 32 sequences of 5 new tokens, 32 fp16 heads: 161 us and 169; one of 2 tokens, 64/8 heads,
// 2047 before them: 12.6 and 15.7.)
template <int D, int MT>
__global__ void __launch_bounds__(kThreads) few_merge_kernel(const FewArgs a) {
    pdl_trigger();
    const int s = blockIdx.x / a.hkv, kvh = blockIdx.x - s * a.hkv, r = blockIdx.y * kWarps + (threadIdx.x >> 5);
    const int n = new_tokens(a, s), start = a.cu[s]; // (complete before the launch that this one follows began)
    const int nsplit = (sight_of<true>(a, s, row_len(a, s)).len + a.split_tokens - 1) / a.split_tokens;
    pdl_wait();
    if (r < n << a.lg_group && nsplit > 1) few_join<D, MT>(a, few_room(a, s, kvh, 0) + r, few_row(a, start, kvh, r), nsplit);
}

template <int D, int KV, int C>
using FewGeo = Geo<D, KV, (C > 1)>;
template <int D, int KV, int C>
constexpr int few_ctas() { return C > 1 ? 2 : FewGeo<D, KV, C>::kCtas; }

template <int D, int KV, int MT, int C>
__global__ void __launch_bounds__(kThreads, few_ctas<D, KV, C>()) few_kernel(const FewArgs a) {
    using G_ = FewGeo<D, KV, C>;
    using M_ = ModelT<MT>;
    constexpr int OT = KV == PKV_BF16 ? PKV_BF16 : PKV_F16; // operand type of the products
    using O = ModelT<OT>;
    constexpr int KS = D / 16; // k steps of the first product = m tiles of the second
    constexpr int ST = G_::kStages, R = 8 * C, LD = D + 4;
    constexpr bool PAIR = OT == PKV_BF16 || MT == PKV_F16; // (one fp16 weight would add 2^-11 to fp16 outputs' own)
    // A row's weights stand against a base that moves only when a score passes it by 2^kPast, to 2^kUp: few tiles move it,
    // and with it every sum, though sixteen rows have a new maximum in most (moving with every maximum: 143 us for 131 of
    // the E4M3 batch above).
    constexpr float kPast = 8.f, kUp = OT == PKV_BF16 ? 0.f : 14.f - kPast;
    extern __shared__ __align__(128) char smem[];
    __shared__ struct {
        float m[kWarps][R], l[kWarps][R], M[R];
    } J;
    __shared__ int sm_tmp[2 * kWarps];
    float *oacc = reinterpret_cast<float *>(smem + kWarps * ST * G_::kBytes); // [R][LD]
    const int tb_len = a.split_tokens >> a.bs_log2;
    char *qbuf = reinterpret_cast<char *>(oacc + R * LD); // two units' q rows and table entries
    int *tbuf = reinterpret_cast<int *>(qbuf + 2 * R * D * 2);
    int *full = tbuf + 2 * tb_len;
    int *part = full + a.num_seqs + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int bl = a.bs_log2, bs = 1 << bl;
    const uint32_t ring_u = smem_u32(smem + warp * ST * G_::kBytes);
    // late: beside the kernel of the sequences of more rows, which lets this one in once it has itself waited for what came
    // before; it fills the SMs as that one's CTAs leave them, and waits for it only before it exits.
    if (!a.late) pdl_wait();
    list_units<true>(a, full, part, sm_tmp);
    const int nfull = full[a.num_seqs] * a.hkv, nunits = nfull + part[a.num_seqs] * a.hkv;
    if ((int)blockIdx.x >= nunits) {
        if (a.late) pdl_wait();
        return;
    }

    // a unit's table entries and q rows on their way (rows without a query keep what was there: their columns are nobody's)
    auto stage = [&](const FewUnit &u, int *tb, char *qs) {
        const int nblk = blocks_of(a, u), b0 = u.t0 >> bl;
        const int32_t *row = a.tables + (int64_t)u.s * a.max_blocks;
        for (int i = threadIdx.x; i < nblk; i += kThreads) {
            const int at = b0 + i;
            cp4(smem_u32(tb + i), row + at + (at >= u.from ? u.skip : 0));
        }
        for (int i = threadIdx.x; i < u.rows * (D / 8); i += kThreads) {
            const int r = i / (D / 8), p = i % (D / 8);
            cp16(smem_u32(qs) + i * 16, static_cast<const char *>(a.q) + few_row(a, u.start, u.kvh, r) * (D * 2) + p * 16, 16);
        }
    };
    FewUnit u = few_unit(a, full, part, nfull, blockIdx.x);
    int par = 0; // which of the two buffers is this unit's
    int *tb = tbuf;
    stage(u, tb, qbuf);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    bool bad = __syncthreads_or(check_table(a, u, tb, threadIdx.x, kThreads));
    int nt = 0;   // this warp's tiles of the unit
    int slot = 0; // the slot of the next one

    auto issue = [&](int tile, int to) {
        const char *head = a.pool + u.kvh * a.head_stride;
        const int t0 = tile * kTile, left = u.n - t0; // left > 0
        const uint32_t dst = ring_u + to * G_::kBytes;
        const char *base[2];
        int lim[2], off[2]; // rows of each octet that exist, first row's offset in its block
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int t = t0 + 8 * o;
            const int b = t < u.n ? tb[t >> bl] : -1;
            off[o] = t & (bs - 1);
            base[o] = b >= 0 ? head + b * a.blk_stride : head;
            lim[o] = b >= 0 ? min(max(left - 8 * o, 0), 8) : 0;
            if (b < 0) off[o] = 0;
        }
#pragma unroll
        for (int i = 0; i < kTile * G_::kChunks / 32; ++i) {
            const int c = i * 32 + lane, r = c / G_::kChunks, p = c % G_::kChunks, o = r >> 3;
            const char *src = (o ? base[1] : base[0]) + ((o ? off[1] : off[0]) + (r & 7)) * G_::kRow + p * 16;
            int sz = (r & 7) < (o ? lim[1] : lim[0]) ? 16 : 0;
            if (u.t0 + t0 + r >= u.lo && u.t0 + t0 + r < u.hi) sz = 0; // (out of every row's sight: zeros)
            cp16(dst + place_k<D, KV>(r, p), src, sz);
            cp16(dst + G_::kV + place_v<D, KV>(r, p), src + a.v_off, sz);
        }
    };
    // a unit's first tiles, a group each (an empty one where there is no tile)
    auto start = [&]() {
        const int ntiles = (u.n + kTile - 1) / kTile;
        nt = ntiles > warp ? (ntiles - warp + kWarps - 1) / kWarps : 0;
        int to = slot;
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) {
            if (i < nt) issue(warp + i * kWarps, to);
            cp_commit();
            to = to == ST - 1 ? 0 : to + 1;
        }
    };
    start();

    for (int ui = blockIdx.x;;) {
        const int un = ui + gridDim.x;
        const bool more = un < nunits;
        FewUnit next = u;
        int *next_tb = tbuf + (par ^ 1) * tb_len;
        if (more) { // its needs ride in this unit's first group: they have landed with the last tile
            next = few_unit(a, full, part, nfull, un);
            stage(next, next_tb, qbuf + (par ^ 1) * R * D * 2);
        }
        // ---- q in the order of the K codes; per row: the score scale
        uint32_t qf[C][KS][2];
        float qs[C][2]; // of columns 2 t4 and 2 t4 + 1
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const char *q = qbuf + (par * R + 8 * c + g) * D * 2;
            float x[KS][4];
            if constexpr (G_::kBits == 16) {
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(q + (16 * k + 2 * t4 + 8 * i) * 2);
                        x[k][2 * i] = lo_f(w, MT);
                        x[k][2 * i + 1] = hi_f(w, MT);
                    }
            } else {
#pragma unroll
                for (int w = 0; w < D / 32; ++w) { // half a 16-code piece
                    const int d0 = 16 * (t4 + 4 * (w >> 1)) + 8 * (w & 1);
                    float f[8];
                    cvt8<MT>(*reinterpret_cast<const uint4 *>(q + d0 * 2), f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[2 * w + (i >> 2)][i & 3] = f[i];
                }
            }
            float s = a.qk_scale_log2;
            if constexpr (OT != MT) {
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(x[k][i]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // 2^(10 - exponent): the row's largest element goes to [2^10, 2^11)
                const int e = (int)(__float_as_uint(mx) >> 23); // biased
                const int sh = (e == 0 || e == 255) ? 0 : min(max(10 - (e - 127), -126), 126);
                const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[k][i] *= up;
                s *= __uint_as_float((uint32_t)(127 - sh) << 23);
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[c][k][0] = O::pack(x[k][0], x[k][1]);
                qf[c][k][1] = O::pack(x[k][2], x[k][3]);
            }
            if constexpr (KV == PKV_FP8_E4M3) s *= a.k_scale[u.kvh];
            qs[c][0] = __shfl_sync(0xffffffffu, s, 8 * t4);
            qs[c][1] = __shfl_sync(0xffffffffu, s, 8 * t4 + 4);
        }

        float m[C][2], mu[C][2], lim[C][2], l[C][2]; // bases; the finite numbers to subtract; where they move; sums
        float acc[C][KS][4];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m[c][0] = m[c][1] = lim[c][0] = lim[c][1] = -INFINITY;
            mu[c][0] = mu[c][1] = l[c][0] = l[c][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) acc[c][k][0] = acc[c][k][1] = acc[c][k][2] = acc[c][k][3] = 0.f;
        }
        const int last_c = u.c0 + (u.rows > 0 ? (u.rows - 1) >> a.lg_group : 0);
        for (int i = 0; i < nt; ++i) {
            cp_wait<ST - 2>();
            __syncwarp();
            {
                const int ahead = i + ST - 1;
                if (ahead < nt) issue(warp + ahead * kWarps, slot == 0 ? ST - 1 : slot - 1);
                cp_commit();
            }
            const uint32_t tile = ring_u + slot * G_::kBytes;
            slot = slot == ST - 1 ? 0 : slot + 1;
            const int t0 = (warp + i * kWarps) * kTile;
            const int at = u.t0 + t0; // first token, among those in sight

            // ---- scores: x[row group][token g, g + 8][row 2 t4, 2 t4 + 1]
            float x[C][4];
            {
                float s[C][2][4];
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[c][0][e] = s[c][1][e] = 0.f;
                if constexpr (KV == PKV_FP8_E4M3) {
#pragma unroll
                    for (int w = 0; w < D / 64; ++w) {
                        uint32_t ka[4], kb[4];
                        lds128(ka, tile + place_k<D, KV>(g, t4 + 4 * w));
                        lds128(kb, tile + place_k<D, KV>(g + 8, t4 + 4 * w));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t ha[2], hb[2];
                            widen8(ka[k], ha);
                            widen8(kb[k], hb);
#pragma unroll
                            for (int c = 0; c < C; ++c)
                                mma<OT>(s[c][k & 1], ha[0], hb[0], ha[1], hb[1], qf[c][4 * w + k][0], qf[c][4 * w + k][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t h[4]; // rows 0-7 / 8-15, columns 16 k .. + 7 / + 8 .. + 15
                        ldmatrix4(h, tile + place_k<D, KV>(lane & 15, 2 * k + (lane >> 4)));
#pragma unroll
                        for (int c = 0; c < C; ++c) mma<OT>(s[c][k & 1], h[0], h[1], h[2], h[3], qf[c][k][0], qf[c][k][1]);
                    }
                }
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[c][e] = (s[c][0][e] + s[c][1][e]) * qs[c][e & 1];
            }
            // (behind the sequence's end nothing is in any row's sight)
            if (at + kTile - 1 > u.c0 || (a.window > 0 && at <= last_c - a.window) || bad) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = at + g + 8 * (e >> 1), end = u.c0 + ((8 * c + 2 * t4 + (e & 1)) >> a.lg_group);
                        const bool sees = t <= end && (a.window == 0 || t > end - a.window || t < a.sinks);
                        if (!sees || (bad && tb[(t0 + g + 8 * (e >> 1)) >> bl] < 0)) x[c][e] = -INFINITY;
                    }
            }

            // ---- bases (one vote a tile)
            bool up = false;
#pragma unroll
            for (int c = 0; c < C; ++c) up = up || fmaxf(x[c][0], x[c][2]) > lim[c][0] || fmaxf(x[c][1], x[c][3]) > lim[c][1];
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float n = fmaxf(x[c][e], x[c][e + 2]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
                        n = n > lim[c][e] ? n : m[c][e]; // (whatever the other rows do, which may be nobody's)
                        f[e] = m[c][e] == n ? 1.f : fast_exp2(m[c][e] - n);
                        m[c][e] = n;
                        mu[c][e] = n == -INFINITY ? 0.f : n - kUp;
                        lim[c][e] = n + kPast;
                        l[c][e] *= f[e];
                    }
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[c][k][e] *= f[e & 1];
                }
            }
            // ---- P^T as the second product's B operand
            uint32_t b[C][2], lo[C][2];
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float w0 = fast_exp2(x[c][2 * r] - mu[c][0]), w1 = fast_exp2(x[c][2 * r + 1] - mu[c][1]);
                    l[c][0] += w0;
                    l[c][1] += w1;
                    if constexpr (PAIR) {
                        b[c][r] = movmatrix(pack_rz<OT>(w0, w1));
                        lo[c][r] = movmatrix(O::pack(w0 - kept_rz<OT>(w0), w1 - kept_rz<OT>(w1)));
                    } else {
                        b[c][r] = movmatrix(O::pack(w0, w1));
                        lo[c][r] = 0;
                    }
                }

            // ---- acc[dims][row] += V^T P^T
            const uint32_t vt = tile + G_::kV;
            auto product = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    mma<OT>(acc[c][k], a0, a1, a2, a3, b[c][0], b[c][1]);
                    if constexpr (PAIR) mma<OT>(acc[c][k], a0, a1, a2, a3, lo[c][0], lo[c][1]);
                }
            };
            if constexpr (G_::kBits == 16) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t h[4]; // tokens 0-7, dims 16 k .. + 7 | + 8 .. + 15, then tokens 8-15
                    ldmatrix4t(h, vt + place_v<D, KV>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
                    product(k, h[0], h[1], h[2], h[3]);
                }
            } else {
                // rows 2 t4, 2 t4 + 1, + 8: this thread's D / 8 dims of each
                constexpr int W = G_::kRow / 32; // words of D / 8 codes
                uint32_t v[4][W];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 2 * t4 + (r & 1) + (r >> 1) * 8;
                    if constexpr (W == 2)
                        lds64(v[r], vt + place_v<D, KV>(row, g >> 1) + (g & 1) * 8);
                    else
                        lds128(v[r], vt + place_v<D, KV>(row, g));
                }
#pragma unroll
                for (int w = 0; w < W; ++w) { // dims 4 w .. + 3 of the thread's: code pairs of tokens (2 t4, + 1) and (+ 8, + 9)
                    uint32_t h[2][4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t x0 = v[2 * r][w], x1 = v[2 * r + 1][w];
                        widen8(bytes_of(x0, x1, 0x5140), &h[r][0]);
                        widen8(bytes_of(x0, x1, 0x7362), &h[r][2]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) product(2 * w + k, h[0][2 * k], h[0][2 * k + 1], h[1][2 * k], h[1][2 * k + 1]);
                }
            }
        }
        cp_commit();
        cp_wait<0>();

        // ---- the next unit's first tiles, then this unit's join
        if (g == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) J.m[warp][8 * c + 2 * t4 + e] = m[c][e] - kUp;
        }
        const FewUnit cur = u;
        bad = __syncthreads_or(more && check_table(a, next, next_tb, threadIdx.x, kThreads)); // (each its own copies)
        u = next;
        tb = next_tb;
        par ^= 1;
        if (more) start();
        const float scale = KV == PKV_FP8_E4M3 ? a.v_scale[cur.kvh] : 1.f;
        float f[C][2];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * c + 2 * t4 + e;
                const float M = fmaxf(fmaxf(J.m[0][r], J.m[1][r]), fmaxf(J.m[2][r], J.m[3][r]));
                const float w = weight_of(J.m[warp][r], M);
                const float sum = row_sum(l[c][e]);
                if (g == 0) {
                    J.l[warp][r] = sum * w; // (a NaN comes through a weight of 0)
                    if (warp == 0) J.M[r] = M;
                }
                f[c][e] = w * scale;
            }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float *o = oacc + (8 * c + 2 * t4 + e) * LD;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            const int d0 = G_::kBits == 16 ? 16 * k + g : (D / 8) * g + 2 * k;
                            const int d1 = G_::kBits == 16 ? d0 + 8 : d0 + 1;
                            const float v0 = acc[c][k][e] * f[c][e], v1 = acc[c][k][e + 2] * f[c][e];
                            o[d0] = w ? o[d0] + v0 : v0;
                            o[d1] = w ? o[d1] + v1 : v1;
                        }
                    }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < cur.rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            const float4 v = *reinterpret_cast<const float4 *>(oacc + r * LD + d);
            const float den = ((J.l[0][r] + J.l[1][r]) + J.l[2][r]) + J.l[3][r];
            if (cur.nsplit > 1) {
                const int64_t part_row = few_room(a, cur.s, cur.kvh, cur.j) + r;
                if (d == 0) reinterpret_cast<float2 *>(a.ws_ml)[part_row] = make_float2(J.M[r], den);
                *reinterpret_cast<float4 *>(a.ws_o + part_row * D + d) = v;
            } else {
                const int64_t row = few_row(a, cur.start, cur.kvh, r);
                const float inv = den == 0.f ? 0.f : 1.f / den;
                *reinterpret_cast<uint2 *>(static_cast<char *>(a.out) + (row * D + d) * 2) =
                    den == 0.f ? make_uint2(0u, 0u) : make_uint2(M_::pack(v.x * inv, v.y * inv), M_::pack(v.z * inv, v.w * inv));
            }
        }
        __syncthreads();
        if (!more) break;
        ui = un;
    }
    if (a.late) pdl_wait();
    pdl_trigger();
}

template <int D, int KV, int C>
size_t few_smem(int seqs, int split, int bs_log2) {
    using G_ = FewGeo<D, KV, C>;
    return (size_t)kWarps * G_::kStages * G_::kBytes + 8 * C * (D + 4) * sizeof(float) + 2 * 8 * C * D * 2 +
           (3 * (seqs + 1) + 2 * (split >> bs_log2)) * sizeof(int);
}

template <int D, int KV, int MT, int C>
cudaError_t launch_few_t(const FewArgs &a, int sms, cudaStream_t st) {
    static std::atomic<bool> have[64];
    auto kern = few_kernel<D, KV, MT, C>;
    const size_t smem = few_smem<D, KV, C>(a.num_seqs, a.split_tokens, a.bs_log2);
    cudaError_t e = pkv_allow_smem(reinterpret_cast<const void *>(kern), have);
    if (e != cudaSuccess) return e;
    return pdl_launch(kern, dim3(grid_of(a, sms * ctas_of(few_ctas<D, KV, C>(), smem))), dim3(kThreads), smem, st, a);
}
template <int D, int KV, int MT>
cudaError_t launch_few_d(const FewArgs &a, int sms, bool merge, cudaStream_t st) {
    const int rows = min(a.most_rows >> a.lg_group, a.max_seqlen) << a.lg_group;
    if (merge)
        return pdl_launch(few_merge_kernel<D, MT>, dim3((unsigned)(a.num_seqs * a.hkv), (rows + kWarps - 1) / kWarps),
                          dim3(kThreads), 0, st, a);
    if (rows <= 8) return launch_few_t<D, KV, MT, 1>(a, sms, st);
    return rows <= 16 ? launch_few_t<D, KV, MT, 2>(a, sms, st) : launch_few_t<D, KV, MT, 3>(a, sms, st);
}
template <int KV, int MT>
cudaError_t launch_few(const FewArgs &a, int D, int sms, bool merge, cudaStream_t st) {
    return D == 64 ? launch_few_d<64, KV, MT>(a, sms, merge, st) : launch_few_d<128, KV, MT>(a, sms, merge, st);
}

} // namespace pkv_mma
