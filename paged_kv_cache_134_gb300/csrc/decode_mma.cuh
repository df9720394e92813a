// Decode attention over 16-bit and E4M3 caches, with attention mass or under a sliding window with sinks.
//
// out[s][h] = sum_t p_t V_t with p_t = softmax_t(scale * q[s][h] . K_t), and
// mass[s][g][t] := decay * mass[s][g][t] + sum_{h in group g} p[s][h][t].
//
// p needs the row's final maximum and sum, so the scores (fp32, a few per cent of the bytes of K and V, and
// mostly still in L2 when they are read) are kept until the row's last split is done.  Bound by the bytes of
// the cache.  K tile: A operand of mma.sync (16 tokens x D), q^T: B operand (D x 8 heads); V tile: A
// operand (16 dims x 16 tokens at a time, read transposed), P^T: B operand.  P goes from the first product's
// layout to the second's by movmatrix, as hi + lo parts (2^-22 relative for fp16 operands, 2^-16 for bf16):
// with up to four heads the lo part uses the four columns of B that are free anyway, with eight it takes a
// second product.  For fp16 operands the largest weight so far stands at 2^14, so that weights down to 2^-28 of it
// stay normal numbers and smaller ones lose 2^-39 of it at most (at 1, 20000 tokens beside one of e^16 times their
// weight lost 4e-4 of their sum); without mass, where the base stays while scores pass it by up to 2^8, it
// stands at 2^6: normal down to 2^-20 of it, smaller ones lose 2^-30.  E4M3 codes widen to fp16 in registers; bf16
// queries are then scaled by a power of two per head so that their largest element is in [2^10, 2^11).  Each warp
// has its own ring of 16-token tiles, filled by cp.async and swizzled on the way (no barrier between warps, no
// wait that could hang).
//
// Measured with mass_kernel: 32 fp16 sequences of up to 4096 tokens, 32 heads, 1.02 GB in 161 us, 6.4 TB/s.
#pragma once

#include "mma_common.cuh"

namespace pkv_mma {

constexpr int kTile = 16; // tokens of a tile

template <int D, int KV, bool G8 = false>
struct Geo {
    static constexpr int kBits = KV == PKV_FP8_E4M3 ? 8 : 16;
    static constexpr int kRow = D * kBits / 8; // bytes of one row's codes
    static constexpr int kChunks = kRow / 16;
    static constexpr int kV = kTile * kRow;                       // V codes behind K's
    static constexpr int kBytes = 2 * kTile * kRow;
    static constexpr int kStages = kBits == 8 ? (D == 128 ? 3 : 4) : G8 ? 2 : 3;
    static constexpr int kCtas = kBits == 8 ? 3 : 2; // per SM, as many as fit beside these rings
};

// Where 16-byte piece c of row r sits in a tile, chosen so that the reads below touch every bank once.
template <int D, int KV>
PKV_DEV int place_k(int r, int c) {
    constexpr int R = Geo<D, KV>::kRow;
    if constexpr (Geo<D, KV>::kBits == 16) return r * R + ((c ^ (r & 7)) << 4);
    if constexpr (R == 128) return r * R + ((c ^ ((r & 1) << 2)) << 4);
    return r * R + (c << 4);
}
template <int D, int KV>
PKV_DEV int place_v(int r, int c) {
    constexpr int R = Geo<D, KV>::kRow;
    if constexpr (Geo<D, KV>::kBits == 16) return r * R + ((c ^ (r & 7)) << 4);
    if constexpr (R == 128) return r * R + ((c ^ (r & 6)) << 4);
    const int p = (r & 8) | int4_place(r & 7); // even rows of an octet first
    return p * R + ((c ^ (p & 2)) << 4);
}

// MASS false, WIN: without the mass, under a sliding window with sinks (see Reach); a row's splits are joined as in
// decode_int4.cuh.  Bound by the bytes of the cache where windows are long, by a unit's fixed parts (finding it, the
// queries, the join: about 3 us) where they are not.  A window wants units of few tokens: against the plain decode's
// kernels under the same windows (CUDA cores for one head a KV head or D = 64, steps of 128 tokens on tcgen05 else)
// 32 sequences of 32 fp16 heads, window 1024, 474 MB: 73 us (80); 256 log-normal sequences, 32/8 heads, window 511, E4M3:
// 47 us (95), bf16 70 (89), of 64 dimensions 44 (90); one of 8192 tokens, bf16: 11 (13).  Only long windows of one head
// a KV head went as fast there (32 of 3000 tokens: 151 and 149).  The next unit's first tiles behind this one's last in the
// ring, its table checked at a barrier of its own, changed nothing (47.2; three CTAs an SM hide one another's joins).
template <int D, int KV, int MT, bool G8, bool MASS = true, bool WIN = false>
__global__ void __launch_bounds__(kThreads, Geo<D, KV>::kCtas) decode_mass_kernel(const Args a) {
    using G_ = Geo<D, KV, G8>;
    using M = ModelT<MT>;
    constexpr int OT = KV == PKV_BF16 ? PKV_BF16 : PKV_F16; // operand type of the products
    using O = ModelT<OT>;
    constexpr int KS = D / 16; // k steps of the first product = m tiles of the second
    constexpr int ST = G_::kStages;
    // Without mass the base moves only when a score passes it by 2^kPast, and with it every sum (see chunk_few.cuh).
    constexpr float kPast = MASS ? 0.f : 8.f;
    constexpr float kUp = OT == PKV_F16 ? 14.f - kPast : 0.f; // log2 of the base's weight (the largest: 2^14)
    extern __shared__ __align__(128) char smem[];
    __shared__ Join J;
    __shared__ int sm_tmp[2 * kWarps];
    constexpr int COLS = G8 ? 8 : 4, LD = D + 4;
    float *oacc = reinterpret_cast<float *>(smem + kWarps * ST * G_::kBytes); // [warp][COLS][LD]
    const int tb_len = a.split_tokens >> a.bs_log2;
    char *qbuf = reinterpret_cast<char *>(oacc + kWarps * COLS * LD); // two units' q rows and table entries
    int *tbuf = reinterpret_cast<int *>(qbuf + 2 * COLS * D * 2);
    int *full = tbuf + 2 * tb_len;
    int *part = full + a.num_seqs + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int G = a.group, bl = a.bs_log2, bs = 1 << bl;
    const uint32_t ring_u = smem_u32(smem + warp * ST * G_::kBytes);
    pdl_wait();
    list_units<WIN>(a, full, part, sm_tmp);
    const int nfull = full[a.num_seqs] * a.hkv, nunits = nfull + part[a.num_seqs] * a.hkv;
    if ((int)blockIdx.x >= nunits) return;

    UnitOf<WIN> u = unit_of<WIN>(a, full, part, nfull, blockIdx.x);
    int par = 0; // which of the two buffers is this unit's
    int *tb = tbuf;
    stage_unit<D>(a, u, tb, qbuf, threadIdx.x, kThreads);
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
            if constexpr (WIN) // (out of sight: zeros, as V is multiplied by the weight 0 there)
                if (u.t0 + t0 + r >= u.lo && u.t0 + t0 + r < u.hi) sz = 0;
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

    Unit prev = u;        // the last unit, if it still has to be counted (without mass)
    bool pending = false;
    for (int ui = blockIdx.x;;) {
        int before = 0;
        if (!MASS && pending && threadIdx.x == 0) before = count_unit(a, prev);
        const int un = ui + gridDim.x;
        const bool more = un < nunits;
        UnitOf<WIN> next = u;
        int *next_tb = tbuf + (par ^ 1) * tb_len;
        if (more) { // its needs ride in this unit's first group: they have landed with the last tile
            next = unit_of<WIN>(a, full, part, nfull, un);
            stage_unit<D>(a, next, next_tb, qbuf + (par ^ 1) * COLS * D * 2, threadIdx.x, kThreads);
        }
        const int n = u.n, s = u.s, kvh = u.kvh;
        // ---- q in the order of the K codes; per head: the score scale
        uint32_t qf[KS][2];
        float qs0, qs1; // of columns 2 t4 and 2 t4 + 1
        {
            const char *q = qbuf + (par * COLS + (G8 ? g : (g & 3) % G)) * D * 2;
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
            float qs = a.qk_scale_log2;
            if constexpr (OT != MT) {
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(x[k][i]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // 2^(10 - exponent): the head's largest element goes to [2^10, 2^11)
                const int e = (int)(__float_as_uint(mx) >> 23); // biased
                const int sh = (e == 0 || e == 255) ? 0 : min(max(10 - (e - 127), -126), 126);
                const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[k][i] *= up;
                qs *= __uint_as_float((uint32_t)(127 - sh) << 23);
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][0] = O::pack(x[k][0], x[k][1]);
                qf[k][1] = O::pack(x[k][2], x[k][3]);
            }
            if constexpr (KV == PKV_FP8_E4M3) qs *= a.k_scale[kvh];
            qs0 = __shfl_sync(0xffffffffu, qs, 8 * t4);
            qs1 = __shfl_sync(0xffffffffu, qs, 8 * t4 + 4);
        }

        float m0 = -INFINITY, m1 = -INFINITY, mu0 = 0.f, mu1 = 0.f; // running maxima; the finite numbers to subtract
        float l0 = 0.f, l1 = 0.f;
        const float lo_part = !G8 && t4 >= 2 ? 1.f : 0.f; // on the lanes whose columns carry the lo parts
        float acc[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
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
            const int left = n - t0;

            // ---- scores: x[token g, g + 8][column 2 t4, 2 t4 + 1]
            float c[2][4] = {};
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
                        mma<OT>(c[k & 1], ha[0], hb[0], ha[1], hb[1], qf[4 * w + k][0], qf[4 * w + k][1]);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t h[4]; // rows 0-7 / 8-15, columns 16 k .. + 7 / + 8 .. + 15
                    ldmatrix4(h, tile + place_k<D, KV>(lane & 15, 2 * k + (lane >> 4)));
                    mma<OT>(c[k & 1], h[0], h[1], h[2], h[3], qf[k][0], qf[k][1]);
                }
            }
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = c[0][e] + c[1][e];
            x[0] *= qs0;
            x[1] *= qs1;
            x[2] *= qs0;
            x[3] *= qs1;
            if (left < kTile || bad) {
                if (g >= left || (bad && tb[(t0 + g) >> bl] < 0)) x[0] = x[1] = -INFINITY;
                if (g + 8 >= left || (bad && tb[(t0 + g + 8) >> bl] < 0)) x[2] = x[3] = -INFINITY;
            }
            if constexpr (WIN) { // tokens out of sight among those in it
                const int lo = u.lo - u.t0 - t0, hi = u.hi - u.t0 - t0;
                if (g >= lo && g < hi) x[0] = x[1] = -INFINITY;
                if (g + 8 >= lo && g + 8 < hi) x[2] = x[3] = -INFINITY;
            }
            if constexpr (MASS) {
                float *dst = a.ws_x + (((int64_t)s * a.hkv + kvh) * a.cap + u.t0 + t0 + g) * G;
                if (G == 1) {
                    if (t4 == 0) {
                        if (g < left) dst[0] = x[0];
                        if (g + 8 < left) dst[8] = x[2];
                    }
                } else if (2 * t4 < G) {
                    if (g < left) *reinterpret_cast<float2 *>(dst + 2 * t4) = make_float2(x[0], x[1]);
                    if (g + 8 < left) *reinterpret_cast<float2 *>(dst + 8 * G + 2 * t4) = make_float2(x[2], x[3]);
                }
            }

            // ---- running maximum (moves rarely: one vote a tile)
            if (__any_sync(0xffffffffu, fmaxf(x[0], x[2]) > m0 + kPast || fmaxf(x[1], x[3]) > m1 + kPast)) {
                float n0 = fmaxf(x[0], x[2]), n1 = fmaxf(x[1], x[3]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
                    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
                }
                n0 = fmaxf(n0, m0);
                n1 = fmaxf(n1, m1);
                const float f0 = m0 == n0 ? 1.f : fast_exp2(m0 - n0), f1 = m1 == n1 ? 1.f : fast_exp2(m1 - n1);
                m0 = n0;
                m1 = n1;
                mu0 = m0 == -INFINITY ? 0.f : m0 - kUp;
                mu1 = m1 == -INFINITY ? 0.f : m1 - kUp;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    acc[k][0] *= f0;
                    acc[k][1] *= f1;
                    acc[k][2] *= f0;
                    acc[k][3] *= f1;
                }
            }
            float p[4];
            p[0] = fast_exp2(x[0] - mu0);
            p[1] = fast_exp2(x[1] - mu1);
            p[2] = fast_exp2(x[2] - mu0);
            p[3] = fast_exp2(x[3] - mu1);
            l0 += p[0] + p[2];
            l1 += p[1] + p[3];
            // ---- P^T as the second product's B operand: hi parts (cut) and lo parts (the rest, rounded to nearest)
            uint32_t b[2], lo[2] = {0, 0};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float w0 = p[2 * r], w1 = p[2 * r + 1];
                if constexpr (G8) {
                    b[r] = movmatrix(pack_rz<OT>(w0, w1));
                    lo[r] = movmatrix(O::pack(w0 - kept_rz<OT>(w0), w1 - kept_rz<OT>(w1)));
                } else { // columns 4..7 repeat the heads of columns 0..3: they carry the lo parts, 0..3 minus the hi parts
                    w0 = fmaf(w0, lo_part, -kept_rz<OT>(w0));
                    w1 = fmaf(w1, lo_part, -kept_rz<OT>(w1));
                    b[r] = movmatrix(O::pack(w0, w1));
                }
            }

            // ---- acc[dims][column] += V^T P^T
            const uint32_t vt = tile + G_::kV;
            auto product = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                mma<OT>(acc[k], a0, a1, a2, a3, b[0], b[1]);
                if constexpr (G8) mma<OT>(acc[k], a0, a1, a2, a3, lo[0], lo[1]);
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
                uint32_t h[2][D / 8]; // token pair (2 t4, + 1) and (+ 8, + 9): code pairs by dim
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint32_t x0 = v[2 * r][w], x1 = v[2 * r + 1][w];
                        widen8(bytes_of(x0, x1, 0x5140), &h[r][4 * w]);
                        widen8(bytes_of(x0, x1, 0x7362), &h[r][4 * w + 2]);
                    }
#pragma unroll
                for (int k = 0; k < KS; ++k) product(k, h[0][k], h[0][k + KS], h[1][k], h[1][k + KS]);
            }
        }
        cp_commit();
        cp_wait<0>();

        // ---- the next unit's first tiles, then this unit's join
        if (g == 0) {
            J.m[warp][2 * t4] = m0 - kUp;
            J.m[warp][2 * t4 + 1] = m1 - kUp;
        }
        const Unit cur = u;
        if (!MASS && threadIdx.x == 0) J.last = pending && before == prev.nsplit - 1;
        bad = __syncthreads_or(more && check_table(a, next, next_tb, threadIdx.x, kThreads)); // (each its own copies)
        u = next;
        tb = next_tb;
        par ^= 1;
        if (more) start();
        if constexpr (!MASS) {
            if (J.last) {
                __threadfence();
                join_row<D, MT>(a, prev, J);
            }
        }
        {
            const Weight w0 = warp_weight(J, warp, 2 * t4), w1 = warp_weight(J, warp, 2 * t4 + 1);
            l0 = row_sum(l0);
            l1 = row_sum(l1);
            if (g == 0) {
                J.l[warp][2 * t4] = l0 * w0.w; // (a NaN comes through a weight of 0)
                J.l[warp][2 * t4 + 1] = l1 * w1.w;
                if (warp == 0) {
                    J.M[2 * t4] = w0.M;
                    J.M[2 * t4 + 1] = w1.M;
                }
            }
            const float f = KV == PKV_FP8_E4M3 ? a.v_scale[cur.kvh] : 1.f;
            const float f0 = w0.w * f, f1 = w1.w * f;
            float *o0 = oacc + (warp * COLS + 2 * t4) * LD, *o1 = o0 + LD;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int d0 = G_::kBits == 16 ? 16 * k + g : (D / 8) * g + k;
                const int d1 = G_::kBits == 16 ? d0 + 8 : d0 + KS;
                if constexpr (!G8) { // hi and lo columns together
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[k][e] = __shfl_xor_sync(0xffffffffu, acc[k][e], 2) - acc[k][e];
                }
                if (2 * t4 < COLS) {
                    o0[d0] = acc[k][0] * f0;
                    o1[d0] = acc[k][1] * f1;
                    o0[d1] = acc[k][2] * f0;
                    o1[d1] = acc[k][3] * f1;
                }
            }
        }
        join_unit<D, COLS, MT, MASS, false>(a, cur, J, oacc);
        prev = cur;
        pending = !MASS && cur.nsplit > 1 && a.done;
        if (!more) break;
        ui = un;
    }
    if constexpr (!MASS) {
        if (pending) {
            if (threadIdx.x == 0) J.last = count_unit(a, prev) == prev.nsplit - 1;
            __syncthreads();
            if (J.last) {
                __threadfence();
                join_row<D, MT>(a, prev, J);
            }
        }
    }
    pdl_trigger();
}

template <int D, int KV, int MT, bool G8, bool MASS, bool WIN>
cudaError_t launch_mass_t(const Args &a, int sms, cudaStream_t st) {
    using G_ = Geo<D, KV, G8>;
    static std::atomic<bool> have[64];
    auto kern = decode_mass_kernel<D, KV, MT, G8, MASS, WIN>;
    constexpr int cols = G8 ? 8 : 4;
    const size_t smem = (size_t)kWarps * G_::kStages * G_::kBytes + kWarps * cols * (D + 4) * sizeof(float) +
                        2 * cols * D * 2 + (3 * (a.num_seqs + 1) + 2 * (a.split_tokens >> a.bs_log2)) * sizeof(int);
    cudaError_t e = pkv_allow_smem(reinterpret_cast<const void *>(kern), have);
    if (e != cudaSuccess) return e;
    return pdl_launch(kern, dim3(grid_of(a, sms * ctas_of(G_::kCtas, smem))), dim3(kThreads), smem, st, a);
}

// one cache type's kernels (one translation unit each)
template <int KV, int MT, bool MASS = true, bool WIN = false>
cudaError_t dispatch_mass(const Args &a, int D, int sms, bool merge, cudaStream_t st) {
    if (merge) return D == 64 ? launch_merge_t<64, MT, MASS, WIN>(a, sms, st) : launch_merge_t<128, MT, MASS, WIN>(a, sms, st);
    if (D == 64)
        return a.group == 8 ? launch_mass_t<64, KV, MT, true, MASS, WIN>(a, sms, st)
                            : launch_mass_t<64, KV, MT, false, MASS, WIN>(a, sms, st);
    return a.group == 8 ? launch_mass_t<128, KV, MT, true, MASS, WIN>(a, sms, st)
                        : launch_mass_t<128, KV, MT, false, MASS, WIN>(a, sms, st);
}

} // namespace pkv_mma
