// Decode attention of short rows, with or without attention mass, over every cache type.
//
//     x_t = scale * q[s][h] . K_t,   p_t = softmax_t(x),   out[s][h] = sum_t p_t V_t,
//     mass[s][g][t] := decay * mass[s][g][t] + sum_{h in group g} p[s][h][t].
//
// A warp takes a whole row (sequence, KV head) of at most kShortTokens tokens, so nothing is split or joined and the
// mass needs no second launch.  Scores: a token a lane, its K row read in pieces of eight elements, q as fp32 in
// shared memory (the same address for all lanes).  Outputs: a piece a lane, two or four tokens at a time, added over
// the warp at the end.  All in fp32; the weights are divided by their sum before the second product, so that the
// sums of a row's values stay in range.  A 4-bit row stays codes in both products, its step and offset two scalars.
// Bound by latency (length, table, rows, one after the other, once per row), which many rows an SM hide.
//
// Measured against the kernels of units, which take 2.5 to 6 us for a unit however short, on 256 x 32 rows of 16 tokens
// (one head, D = 128, bf16 model): 4-bit 13 us for 36, with mass 13 for 48; with mass over E4M3 15 for 110, over bf16
// 15 for 72.
#pragma once

#include "mma_common.cuh"

namespace pkv_mma {

constexpr int kShortWarps = 4;

// A piece of a row: eight stored elements in W words, and as fp32: a 16-bit row's numbers, the others' codes.
template <int KV>
struct Piece {
    static constexpr int W = KV == PKV_INT4 ? 1 : KV == PKV_FP8_E4M3 ? 2 : 4;
    uint32_t w[W];
    PKV_DEV void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    PKV_DEV void load(const char *p) {
        if constexpr (W == 1) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else if constexpr (W == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
    }
    template <int MT>
    PKV_DEV void widen(float *f) const {
        if constexpr (W == 1) {
            const uint32_t v = __byte_perm(w[0], 0, 0x2301);
            const uint32_t at3[4] = {w[0], w[0] >> 4, v, v >> 4};
#pragma unroll
            for (int i = 0; i < 4; ++i) { // elements i and i + 4 (int4_values)
                const uint32_t c = pair_add<PKV_F16>((at3[i] & 0x00780078u) | 0x58005800u, 0xD800D800u);
                f[i] = lo_f(c, PKV_F16);
                f[i + 4] = hi_f(c, PKV_F16);
            }
        } else if constexpr (W == 2) {
            cvt8_e4m3(make_uint2(w[0], w[1]), f);
        } else {
            cvt8<MT>(make_uint4(w[0], w[1], w[2], w[3]), f);
        }
    }
};

template <int D, int KV, int MT, int G>
__global__ void __launch_bounds__(kShortWarps * 32) short_kernel(const Args a) {
    using M_ = ModelT<MT>;
    constexpr int kRow = KV == PKV_INT4 ? D / 2 : KV == PKV_FP8_E4M3 ? D : 2 * D; // bytes of a row's codes
    constexpr int kPiece = kRow / (D / 8);
    __shared__ __align__(16) float sm_q[kShortWarps][G][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x * kShortWarps + warp;
    pdl_trigger();
    pdl_wait();
    if (row >= a.num_seqs * a.hkv) return;
    const int s = (int)(((uint64_t)(uint32_t)row * a.hkv_magic) >> a.hkv_shift), kvh = row - s * a.hkv;
    const int L = row_len(a, s);
    if (lane == 0 && kvh == 0 && (int64_t)a.lens[s] > a.cap) set_error(a.err, PKV_DEVERR_LENGTH);
    const int64_t q_row = ((int64_t)s * a.hq + kvh * G) * D;
    const int bs = 1 << a.bs_log2;
    auto head_of = [&](int b) { return a.pool + b * a.blk_stride + kvh * a.head_stride; };
    // the row's tokens, a lane each; -1: no token, or in no block
    int b = lane < L ? a.tables[(int64_t)s * a.max_blocks + (lane >> a.bs_log2)] : -1;
    if (lane < L && (b < 0 || b >= a.num_blocks)) {
        set_error(a.err, PKV_DEVERR_BLOCK_ID);
        b = -1;
    }
    // q; for codes with an offset also its sum
    float sum_q[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
        sum_q[h] = 0.f;
        if (lane < D / 8) {
            float f[8];
            cvt8<MT>(*reinterpret_cast<const uint4 *>(static_cast<const char *>(a.q) + (q_row + h * D + lane * 8) * 2), f);
            float4 *dst = reinterpret_cast<float4 *>(&sm_q[warp][h][lane * 8]);
            dst[0] = make_float4(f[0], f[1], f[2], f[3]);
            dst[1] = make_float4(f[4], f[5], f[6], f[7]);
            sum_q[h] = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
        if constexpr (KV == PKV_INT4) {
#pragma unroll
            for (int o = D / 16; o > 0; o >>= 1) sum_q[h] += __shfl_xor_sync(0xffffffffu, sum_q[h], o);
            sum_q[h] = __shfl_sync(0xffffffffu, sum_q[h], 0);
        }
    }
    __syncwarp();
    // V: lanes of a token share its row; kBatch tokens of a lane are on their way at once, the first ones from here
    constexpr int kLanes = D / 8, kStep = 32 / kLanes, kBatch = 8, kAll = kShortTokens / kStep;
    const int sub = lane / kLanes, piece = lane % kLanes;
    Piece<KV> v[kBatch];
    uint32_t sz[kBatch];
    auto load_v = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int t = (i0 + i) * kStep + sub, bt = __shfl_sync(0xffffffffu, b, t), off = t & (bs - 1);
            v[i].zero();
            sz[i] = 0;
            if (bt < 0) continue;
            const char *head = head_of(bt);
            if constexpr (KV == PKV_INT4) {
                v[i].load(head + int4_codes(1, off, piece * kPiece, D));
                sz[i] = *reinterpret_cast<const uint32_t *>(head + int4_params(1, off, D));
            } else {
                v[i].load(head + a.v_off + off * kRow + piece * kPiece);
            }
        }
    };
    load_v(0);
    // ---- scores
    float x[G];
#pragma unroll
    for (int h = 0; h < G; ++h) x[h] = -INFINITY;
    if (b >= 0) {
        const int off = lane & (bs - 1);
        const char *head = head_of(b);
        const char *k = KV == PKV_INT4 ? head + int4_codes(0, off, 0, D) : head + off * kRow;
        float dot[G];
#pragma unroll
        for (int h = 0; h < G; ++h) dot[h] = 0.f;
#pragma unroll
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
            Piece<KV> w[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) w[c].load(k + (c0 + c) * kPiece);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                float f[8];
                w[c].template widen<MT>(f);
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    const float4 q0 = *reinterpret_cast<const float4 *>(&sm_q[warp][h][(c0 + c) * 8]);
                    const float4 q1 = *reinterpret_cast<const float4 *>(&sm_q[warp][h][(c0 + c) * 8 + 4]);
                    dot[h] += fmaf(f[3], q0.w, fmaf(f[2], q0.z, fmaf(f[1], q0.y, f[0] * q0.x))) +
                              fmaf(f[7], q1.w, fmaf(f[6], q1.z, fmaf(f[5], q1.y, f[4] * q1.x)));
                }
            }
        }
        const float scale = KV == PKV_FP8_E4M3 ? a.qk_scale_log2 * a.k_scale[kvh] : a.qk_scale_log2;
        if constexpr (KV == PKV_INT4) {
            const uint32_t p = *reinterpret_cast<const uint32_t *>(head + int4_params(0, off, D));
#pragma unroll
            for (int h = 0; h < G; ++h) x[h] = fmaf(dot[h], lo_f(p, MT), sum_q[h] * hi_f(p, MT)) * scale;
        } else {
#pragma unroll
            for (int h = 0; h < G; ++h) x[h] = dot[h] * scale;
        }
    }
    // ---- weights, divided by their sum
    float all = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) {
        float m = x[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        x[h] = fast_exp2(x[h] - (m == -INFINITY ? 0.f : m));
        float l = x[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        x[h] *= l == 0.f ? 0.f : 1.f / l;
        all += x[h];
    }
    if (a.mass && lane < L) {
        float *m = a.mass + (int64_t)row * a.mass_len + lane;
        *m = fmaf(*m, a.decay, all);
    }
    // ---- outputs
    float acc[G][8], z[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
        z[h] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[h][i] = 0.f;
    }
#pragma unroll
    for (int i0 = 0; i0 < kAll; i0 += kBatch) {
        if (i0 * kStep >= L) break;
        if (i0 > 0) load_v(i0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float f[8];
            v[i].template widen<MT>(f);
            const float step = KV == PKV_INT4 ? lo_f(sz[i], MT) : 1.f, low = KV == PKV_INT4 ? hi_f(sz[i], MT) : 0.f;
#pragma unroll
            for (int h = 0; h < G; ++h) {
                const float p = __shfl_sync(0xffffffffu, x[h], (i0 + i) * kStep + sub), w = p * step;
                z[h] = fmaf(p, low, z[h]);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[h][e] = fmaf(w, f[e], acc[h][e]);
            }
        }
    }
    const float back = KV == PKV_FP8_E4M3 ? a.v_scale[kvh] : 1.f;
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) {
            if (KV == PKV_INT4) z[h] += __shfl_xor_sync(0xffffffffu, z[h], o);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[h][i] += __shfl_xor_sync(0xffffffffu, acc[h][i], o);
        }
        if (sub != h % kStep) continue;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = KV == PKV_INT4 ? acc[h][i] + z[h] : acc[h][i] * back;
        *reinterpret_cast<uint4 *>(static_cast<char *>(a.out) + (q_row + h * D + piece * 8) * 2) =
            make_uint4(M_::pack(y[0], y[1]), M_::pack(y[2], y[3]), M_::pack(y[4], y[5]), M_::pack(y[6], y[7]));
    }
}

template <int D, int KV, int MT>
cudaError_t launch_short_t(const Args &a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.num_seqs * (int64_t)a.hkv + kShortWarps - 1) / kShortWarps)), block(kShortWarps * 32);
    switch (a.group) {
    case 1: return pdl_launch(short_kernel<D, KV, MT, 1>, grid, block, 0, st, a);
    case 2: return pdl_launch(short_kernel<D, KV, MT, 2>, grid, block, 0, st, a);
    case 4: return pdl_launch(short_kernel<D, KV, MT, 4>, grid, block, 0, st, a);
    default: return pdl_launch(short_kernel<D, KV, MT, 8>, grid, block, 0, st, a);
    }
}

template <int KV, int MT>
cudaError_t dispatch_short(const Args &a, int D, cudaStream_t st) {
    return D == 64 ? launch_short_t<64, KV, MT>(a, st) : launch_short_t<128, KV, MT>(a, st);
}

} // namespace pkv_mma
