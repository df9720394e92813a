// Paged decode attention on warp-level matrix instructions: the 4-bit cache's decode, and the
// decode that accumulates attention mass for every cache type.
//
// What it computes, for sequence s, query head h of KV head g = h / G, L = context_lens[s]:
//     x_t = scale * q[s][h] . K_t,   p_t = exp(x_t) / sum_u exp(x_u),   out[s][h] = sum_t p_t V_t
// and, where asked, mass[s][g][t] := decay * mass[s][g][t] + sum_{h in group g} p[s][h][t].
// A 4-bit row stands for K_t = s_t c_t + z_t (c in 0..15, one s and z per row), so with the
// centred code c' = c - 8 and z' = z + 8 s
//     q . K_t = s_t (q . c'_t) + z'_t sum(q),     sum_t p_t V_t = sum_t (p_t s_t) c'_t + sum_t p_t z'_t:
// the matrix products run on the codes themselves, which fp16 holds exactly; steps and offsets are
// two scalars per token outside them.
//
// What bounds it: the bytes of the cache (68 B per row and head at 4 bits and D = 128).  At the
// measured 6.78 TB/s an SM gets 24 B = 47 codes per clock, too many to widen one by one: widening
// through shared memory for tcgen05 operands would write 94 B and read 94 B per clock of its 128,
// and one fp32 FMA per code would take 47 of the 128 lanes on top of the unpacking.  mma.sync takes
// its operands from registers, so a code travels global -> shared (asynchronous copy) -> register
// once, is widened there two at a time (9 instructions per 8 codes), and the products cost 16
// instructions per 16 tokens.
//
// Layout of the work:
//  * A unit is (sequence, KV head, split of split_tokens tokens); persistent CTAs of four warps walk
//    the units, whole splits first.  A warp takes every fourth 16-token tile of a split, with its own
//    ring of STAGES tiles filled by cp.async (no barrier between warps, no wait that could hang).
//  * K tile: A operand (16 tokens x D codes), q^T: B operand (D x 8 heads).  V tile: A operand
//    (16 dims x 16 tokens at a time), P^T: B operand (16 tokens x 8 heads).  The order of the summed
//    index is free, so each thread takes the codes of whole 16-byte pieces of a row as they lie, and q is laid
//    out once per unit in the same order.  P goes from the first product's layout to the second's by
//    movmatrix.
//  * The second product takes P as fp16 (bf16 for bf16 caches) hi + lo parts, so that rounding P
//    (2^-11 or 2^-8 relative) does not show: with up to four heads the lo part uses the four columns
//    of B that are free anyway; with eight heads it takes a second product.
//  * p_t s_t is divided by a power of two A >= every s_t seen (A moves with the accumulator like the
//    running maximum does), so that fp16 holds it whatever the steps' magnitude.
//  * bf16 queries over 4- and 8-bit caches are scaled by a power of two per head into fp16's range
//    (exact down to 2^-24 of the head's largest element, beyond that below 2^-34 of it).
//  * Scores, softmax statistics, sums and accumulators are fp32.
#pragma once

#include "device_common.cuh"
#include "pkv_internal.h"

namespace pkv_mma {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;       // tokens of a tile
constexpr int kMaxSeqs = 1024;  // sequences of a launch (their unit counts sit in shared memory)
constexpr int kMaxSplit = 1024; // tokens of a split

struct Args {
    const void *q;
    void *out;
    const char *pool;
    const float *k_scale, *v_scale; // E4M3 caches
    const int32_t *tables, *lens;
    float *ws_o, *ws_ml; // [S * Hq][max_splits][D], [S * Hq][max_splits][2]
    float *ws_x;         // mass: scores in log2 units, [S * Hkv][cap][G]
    float *mass;         // [S][Hkv][mass_len]
    unsigned int *err;
    int64_t num_blocks;
    int64_t blk_stride, head_stride, v_off; // bytes: block, head, V behind K
    int64_t mass_len, cap;                  // tokens of a mass row; tokens a sequence may have
    int max_blocks, num_seqs, hq, hkv, group, bs_log2;
    int split_tokens, max_splits;
    float qk_scale_log2; // scale * log2(e)
    float decay;
};

template <int D, int KV>
struct Geo {
    static constexpr int kBits = KV == PKV_INT4 ? 4 : KV == PKV_FP8_E4M3 ? 8 : 16;
    static constexpr int kRow = D * kBits / 8; // bytes of one row's codes
    static constexpr int kChunks = kRow / 16;
    static constexpr int kV = kTile * kRow;                       // V codes behind K's
    static constexpr int kPar = 2 * kTile * kRow;                 // (s, z) of K's rows, then of V's
    static constexpr int kBytes = kPar + (KV == PKV_INT4 ? 2 * kTile * 4 : 0);
    static constexpr int kStages = kBits == 4 ? 6 : kBits == 8 ? 4 : 3;
    static constexpr int kCtas = kBits == 4 ? 4 : kBits == 8 ? 3 : 2; // per SM
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
    const int p = (r & 8) | ((r & 7) >> 1) | ((r & 1) << 2); // even rows of an octet first
    if constexpr (R == 64) return p * R + ((c ^ (p & 2)) << 4);
    return p * R + (c << 4);
}

PKV_DEV void cp16(uint32_t dst, const char *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
PKV_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
PKV_DEV void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

PKV_DEV void lds64(uint32_t *w, uint32_t a) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
}
PKV_DEV void lds128(uint32_t *w, uint32_t a) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
}
PKV_DEV uint32_t lds32(uint32_t a) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(a));
    return w;
}
PKV_DEV void ldmatrix4(uint32_t *w, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a));
}
PKV_DEV void ldmatrix4t(uint32_t *w, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a));
}
PKV_DEV uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), operands fp16 or bf16
template <int OT>
PKV_DEV void mma(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (OT == PKV_F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

PKV_DEV uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (a & mask) | bits
template <uint32_t MASK, uint32_t BITS>
PKV_DEV uint32_t mask_or(uint32_t a) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "n"(MASK), "n"(BITS));
    return r;
}

// Nibbles 0..3 of each 16-bit half of w -> four fp16 pairs of c - 8 (low half, high half), exact:
// a nibble in the low bits of an fp16 of exponent 10 reads 1024 + c, one place up in an fp16 of
// exponent 6 reads 64 + c.
PKV_DEV void widen4(uint32_t w, uint32_t *h) {
    h[0] = hadd2(mask_or<0x000F000Fu, 0x64006400u>(w), 0xE408E408u);      // - 1032
    h[1] = hadd2(mask_or<0x00F000F0u, 0x54005400u>(w), 0xD480D480u);      // - 72
    const uint32_t v = w >> 8;
    h[2] = hadd2(mask_or<0x000F000Fu, 0x64006400u>(v), 0xE408E408u);
    h[3] = hadd2(mask_or<0x00F000F0u, 0x54005400u>(v), 0xD480D480u);
}
// two pairs of E4M3 codes (low 16 bits, high 16 bits) -> two fp16 pairs (exact)
PKV_DEV void widen8(uint32_t w, uint32_t *h) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(w));
}
PKV_DEV uint32_t bytes_of(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

PKV_DEV float lo_f(uint32_t w, int mt) {
    return mt == PKV_F16 ? __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu))) : __uint_as_float(w << 16);
}
PKV_DEV float hi_f(uint32_t w, int mt) {
    return mt == PKV_F16 ? __half2float(__ushort_as_half((unsigned short)(w >> 16))) : __uint_as_float(w & 0xFFFF0000u);
}

PKV_DEV int row_len(const Args &a, int s) {
    const int L = a.lens[s];
    return L <= 0 ? 0 : (int64_t)L > a.cap ? (int)a.cap : L;
}

// mass of tokens [t0, t1) of (sequence, KV head) row `row` from their stored scores, with the row's
// final maxima and reciprocal sums per head
PKV_DEV void add_mass(const Args &a, int64_t row, int t0, int t1, const float *M, const float *inv) {
    const float *x = a.ws_x + row * a.cap * a.group;
    float *m = a.mass + row * a.mass_len;
    for (int t = t0 + threadIdx.x; t < t1; t += kThreads) {
        float p = 0.f;
        for (int h = 0; h < a.group; ++h) p = fmaf(fast_exp2(x[(int64_t)t * a.group + h] - M[h]), inv[h], p);
        m[t] = fmaf(m[t], a.decay, p);
    }
}

// Block scan of the sequences' unit counts: full[s + 1], part[s + 1] hold the inclusive sums of whole
// splits and of partial ones (a sequence of length 0 has one partial unit, which writes its zero row).
PKV_DEV void list_units(const Args &a, int *full, int *part, int *tmp) {
    const int S = a.num_seqs, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int cf = 0, cp = 0; // sums of the sequences before this pass
    if (threadIdx.x == 0) full[0] = part[0] = 0;
    for (int s0 = 0; s0 < S; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        int f = 0, p = 0;
        if (s < S) {
            const int L = row_len(a, s);
            if (blockIdx.x == 0 && (int64_t)a.lens[s] > a.cap) set_error(a.err, PKV_DEVERR_LENGTH);
            f = L / a.split_tokens;
            p = (L % a.split_tokens != 0 || L == 0) ? 1 : 0;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int vf = __shfl_up_sync(0xffffffffu, f, o), vp = __shfl_up_sync(0xffffffffu, p, o);
            if (lane >= o) f += vf, p += vp;
        }
        if (lane == 31) tmp[warp] = f, tmp[kWarps + warp] = p;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) f += tmp[w], p += tmp[kWarps + w];
        }
        f += cf;
        p += cp;
        if (s < S) full[s + 1] = f, part[s + 1] = p;
        for (int w = 0; w < kWarps; ++w) cf += tmp[w], cp += tmp[kWarps + w];
        __syncthreads();
    }
}

PKV_DEV int find_row(const int *pref, int n, int k) { // largest i in [0, n) with pref[i] <= k
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pref[mid] <= k)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <int D, int KV, int MT, bool G8, bool MASS>
__global__ void __launch_bounds__(kThreads, Geo<D, KV>::kCtas) decode_kernel(const Args a) {
    using G_ = Geo<D, KV>;
    using M = ModelT<MT>;
    constexpr int OT = KV == PKV_BF16 ? PKV_BF16 : PKV_F16; // operand type of the products
    using O = ModelT<OT>;
    constexpr bool I4 = KV == PKV_INT4;
    constexpr int KS = D / 16; // k steps of the first product = m tiles of the second
    constexpr int ST = G_::kStages;
    extern __shared__ __align__(128) char smem[];
    __shared__ float sm_m[kWarps][8], sm_l[kWarps][8], sm_z[kWarps][8];
    __shared__ float sm_M[8], sm_inv[8], sm_w[kWarps][8];
    __shared__ int sm_tmp[2 * kWarps], sm_bad;
    int *full = reinterpret_cast<int *>(smem + kWarps * ST * G_::kBytes);
    int *part = full + a.num_seqs + 1;
    int *tb = part + a.num_seqs + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int G = a.group, bl = a.bs_log2, bs = 1 << bl;
    char *ring = smem + warp * ST * G_::kBytes;
    const uint32_t ring_u = smem_u32(ring);

    pdl_wait();
    list_units(a, full, part, sm_tmp);
    const int nfull = full[a.num_seqs] * a.hkv, nunits = nfull + part[a.num_seqs] * a.hkv;

    for (int u = blockIdx.x; u < nunits; u += gridDim.x) {
        // ---- which unit
        int s, kvh, j;
        if (u < nfull) {
            const int k = u / a.hkv;
            kvh = u - k * a.hkv;
            s = find_row(full, a.num_seqs, k);
            j = k - full[s];
        } else {
            const int k = (u - nfull) / a.hkv;
            kvh = (u - nfull) - k * a.hkv;
            s = find_row(part, a.num_seqs, k);
            j = full[s + 1] - full[s];
        }
        const int L = row_len(a, s);
        const int nsplit = (full[s + 1] - full[s]) + (part[s + 1] - part[s]);
        const int tb0 = j * a.split_tokens;                 // first token
        const int n = min(L - tb0, a.split_tokens);         // tokens of this unit
        const int nblk = (n + bs - 1) >> bl, ntiles = (n + kTile - 1) / kTile;
        if (threadIdx.x == 0) sm_bad = 0;
        __syncthreads(); // the last unit's shared memory is free
        for (int i = threadIdx.x; i < nblk; i += kThreads) {
            int b = a.tables[(int64_t)s * a.max_blocks + (tb0 >> bl) + i];
            if (b < 0 || b >= a.num_blocks) {
                set_error(a.err, PKV_DEVERR_BLOCK_ID);
                sm_bad = 1;
                b = -1;
            }
            tb[i] = b;
        }
        // ---- q in the order of the K codes; per head: sum(q) and the score scale
        uint32_t qf[KS][2];
        float sum0 = 0.f, sum1 = 0.f, qs0, qs1; // of columns 2 t4 and 2 t4 + 1
        {
            const int h = kvh * G + (G8 ? g : (g & 3) % G);
            const typename M::T *q = static_cast<const typename M::T *>(a.q) + ((int64_t)s * a.hq + h) * D;
            float x[KS][4];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                int d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (I4) {
                        // word k / 2 of the thread's quarter row: pairs (nibble p, nibble p + 4)
                        d[i] = t4 * (D / 4) + 8 * (k >> 1) + 2 * (k & 1) + (i >> 1) + 4 * (i & 1);
                    } else if constexpr (KV == PKV_FP8_E4M3) {
                        d[i] = 16 * (t4 + 4 * (k >> 2)) + 4 * (k & 3) + i;
                    } else {
                        d[i] = 16 * k + 2 * t4 + 8 * (i >> 1) + (i & 1);
                    }
                    x[k][i] = M::to_f(q[d[i]]);
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
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qf[k][0] = O::pack(x[k][0], x[k][1]);
                qf[k][1] = O::pack(x[k][2], x[k][3]);
                if constexpr (I4) sum += (x[k][0] + x[k][1]) + (x[k][2] + x[k][3]);
            }
            if constexpr (I4) {
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum0 = __shfl_sync(0xffffffffu, sum, 8 * t4);
                sum1 = __shfl_sync(0xffffffffu, sum, 8 * t4 + 4);
            }
            if constexpr (KV == PKV_FP8_E4M3) qs *= a.k_scale[kvh];
            qs0 = __shfl_sync(0xffffffffu, qs, 8 * t4);
            qs1 = __shfl_sync(0xffffffffu, qs, 8 * t4 + 4);
        }
        __syncthreads();
        const bool bad = sm_bad != 0;

        // ---- tiles of this warp: warp, warp + kWarps, ...
        const char *head = a.pool + kvh * a.head_stride;
        auto issue = [&](int tile, int slot) {
            const int t0 = tile * kTile, left = n - t0; // left > 0
            const uint32_t dst = ring_u + slot * G_::kBytes;
            const char *base[2];
            int lim[2], off[2]; // rows of each octet that exist, first row's offset in its block
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int t = t0 + 8 * o;
                const int b = t < n ? tb[t >> bl] : -1;
                off[o] = t & (bs - 1);
                base[o] = b >= 0 ? head + b * a.blk_stride : head;
                lim[o] = b >= 0 ? min(max(left - 8 * o, 0), 8) : 0;
                if (b < 0) off[o] = 0;
            }
#pragma unroll
            for (int i = 0; i < kTile * G_::kChunks / 32; ++i) {
                const int c = i * 32 + lane, r = c / G_::kChunks, p = c % G_::kChunks, o = r >> 3;
                const char *src = (o ? base[1] : base[0]) + ((o ? off[1] : off[0]) + (r & 7)) * G_::kRow + p * 16;
                const int sz = (r & 7) < (o ? lim[1] : lim[0]) ? 16 : 0;
                cp16(dst + place_k<D, KV>(r, p), src, sz);
                cp16(dst + G_::kV + place_v<D, KV>(r, p), src + a.v_off, sz);
            }
            if constexpr (I4) {
                if (lane < 8) { // 4 rows' (s, z) each: K rows 0..15, V rows 0..15
                    const int o = (lane >> 1) & 1, r = (lane & 1) * 4;
                    const char *src = (o ? base[1] : base[0]) + bs * D + (lane >> 2) * (bs * 4) +
                                      ((o ? off[1] : off[0]) + r) * 4;
                    cp16(dst + G_::kPar + lane * 16, src, min(max((o ? lim[1] : lim[0]) - r, 0), 4) * 4);
                }
            }
        };

        float m0 = -INFINITY, m1 = -INFINITY, mu0 = 0.f, mu1 = 0.f; // running maxima; the finite ones to subtract
        float l0 = 0.f, l1 = 0.f, z0 = 0.f, z1 = 0.f;
        float A = 0.f, invA = 1.f;
        float acc[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        const int nt = ntiles > warp ? (ntiles - warp + kWarps - 1) / kWarps : 0;
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) {
            if (i < nt) issue(warp + i * kWarps, i);
            cp_commit();
        }
        int slot = 0;
        for (int i = 0; i < nt; ++i) {
            cp_wait<ST - 2>();
            __syncwarp();
            {
                const int ahead = i + ST - 1;
                const int to = slot == 0 ? ST - 1 : slot - 1;
                if (ahead < nt) issue(warp + ahead * kWarps, to);
                cp_commit();
            }
            const uint32_t tile = ring_u + slot * G_::kBytes;
            slot = slot == ST - 1 ? 0 : slot + 1;
            const int t0 = (warp + i * kWarps) * kTile;
            const int left = n - t0;

            // ---- scores: x[token g, g + 8][column 2 t4, 2 t4 + 1]
            float c[2][4] = {};
            if constexpr (I4) {
                uint32_t ka[D / 32], kb[D / 32];
                if constexpr (D == 128) {
                    lds128(ka, tile + place_k<D, KV>(g, t4));
                    lds128(kb, tile + place_k<D, KV>(g + 8, t4));
                } else {
                    lds64(ka, tile + g * G_::kRow + t4 * 8);
                    lds64(kb, tile + (g + 8) * G_::kRow + t4 * 8);
                }
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    uint32_t ha[4], hb[4];
                    widen4(ka[w], ha);
                    widen4(kb[w], hb);
                    mma<OT>(c[0], ha[0], hb[0], ha[1], hb[1], qf[2 * w][0], qf[2 * w][1]);
                    mma<OT>(c[1], ha[2], hb[2], ha[3], hb[3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
                }
            } else if constexpr (KV == PKV_FP8_E4M3) {
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
            float vs0 = 1.f, vs1 = 1.f, vz0 = 0.f, vz1 = 0.f; // V's step and centred offset, rows g and g + 8
            if constexpr (I4) {
                const uint32_t p0 = lds32(tile + G_::kPar + g * 4), p1 = lds32(tile + G_::kPar + (g + 8) * 4);
                const float s0 = lo_f(p0, MT), s1 = lo_f(p1, MT);
                const float o0 = fmaf(8.f, s0, hi_f(p0, MT)), o1 = fmaf(8.f, s1, hi_f(p1, MT));
                x[0] = fmaf(s0, x[0], o0 * sum0) * qs0;
                x[1] = fmaf(s0, x[1], o0 * sum1) * qs1;
                x[2] = fmaf(s1, x[2], o1 * sum0) * qs0;
                x[3] = fmaf(s1, x[3], o1 * sum1) * qs1;
                const uint32_t v0 = lds32(tile + G_::kPar + 64 + g * 4), v1 = lds32(tile + G_::kPar + 64 + (g + 8) * 4);
                vs0 = lo_f(v0, MT);
                vs1 = lo_f(v1, MT);
                vz0 = fmaf(8.f, vs0, hi_f(v0, MT));
                vz1 = fmaf(8.f, vs1, hi_f(v1, MT));
            } else {
                x[0] *= qs0;
                x[1] *= qs1;
                x[2] *= qs0;
                x[3] *= qs1;
            }
            if (left < kTile || bad) {
                if (g >= left || (bad && tb[(t0 + g) >> bl] < 0)) x[0] = x[1] = -INFINITY;
                if (g + 8 >= left || (bad && tb[(t0 + g + 8) >> bl] < 0)) x[2] = x[3] = -INFINITY;
            }
            if constexpr (MASS) {
                float *dst = a.ws_x + (((int64_t)s * a.hkv + kvh) * a.cap + tb0 + t0 + g) * G;
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

            // ---- running maximum (moves rarely: one vote a tile) and the divisor of p s
            bool up = fmaxf(x[0], x[2]) > m0 || fmaxf(x[1], x[3]) > m1;
            if constexpr (I4) up = up || vs0 > A || vs1 > A;
            if (__any_sync(0xffffffffu, up)) {
                float n0 = fmaxf(x[0], x[2]), n1 = fmaxf(x[1], x[3]), ns = fmaxf(vs0, vs1);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
                    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
                    if constexpr (I4) ns = fmaxf(ns, __shfl_xor_sync(0xffffffffu, ns, o));
                }
                n0 = fmaxf(n0, m0);
                n1 = fmaxf(n1, m1);
                const float f0 = m0 == n0 ? 1.f : fast_exp2(m0 - n0), f1 = m1 == n1 ? 1.f : fast_exp2(m1 - n1);
                m0 = n0;
                m1 = n1;
                mu0 = m0 == -INFINITY ? 0.f : m0;
                mu1 = m1 == -INFINITY ? 0.f : m1;
                l0 *= f0;
                l1 *= f1;
                float r0 = f0, r1 = f1;
                if constexpr (I4) {
                    z0 *= f0;
                    z1 *= f1;
                    if (ns > A) { // the next power of two above the largest step (its reciprocal stays normal)
                        const int e = min(max((int)(__float_as_uint(ns) >> 23) + 1, 2), 252);
                        const float nA = __uint_as_float((uint32_t)e << 23);
                        const float ni = __uint_as_float((uint32_t)(254 - e) << 23);
                        r0 *= A * ni;
                        r1 *= A * ni;
                        A = nA;
                        invA = ni;
                    }
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    acc[k][0] *= r0;
                    acc[k][1] *= r1;
                    acc[k][2] *= r0;
                    acc[k][3] *= r1;
                }
            }
            float p[4];
            p[0] = fast_exp2(x[0] - mu0);
            p[1] = fast_exp2(x[1] - mu1);
            p[2] = fast_exp2(x[2] - mu0);
            p[3] = fast_exp2(x[3] - mu1);
            l0 += p[0] + p[2];
            l1 += p[1] + p[3];
            if constexpr (I4) {
                z0 = fmaf(p[0], vz0, fmaf(p[2], vz1, z0));
                z1 = fmaf(p[1], vz0, fmaf(p[3], vz1, z1));
                vs0 *= invA;
                vs1 *= invA;
                p[0] *= vs0;
                p[1] *= vs0;
                p[2] *= vs1;
                p[3] *= vs1;
            }
            // ---- P^T as the second product's B operand, hi and lo parts
            const uint32_t h0 = O::pack(p[0], p[1]), h1 = O::pack(p[2], p[3]);
            const uint32_t e0 = O::pack(p[0] - lo_f(h0, OT), p[1] - hi_f(h0, OT));
            const uint32_t e1 = O::pack(p[2] - lo_f(h1, OT), p[3] - hi_f(h1, OT));
            uint32_t b0, b1, b2 = 0, b3 = 0;
            if constexpr (G8) {
                b0 = movmatrix(h0);
                b1 = movmatrix(h1);
                b2 = movmatrix(e0);
                b3 = movmatrix(e1);
            } else { // columns 4..7 repeat the heads of columns 0..3: they carry the lo parts
                b0 = movmatrix(t4 >= 2 ? e0 : h0);
                b1 = movmatrix(t4 >= 2 ? e1 : h1);
            }

            // ---- acc[dims][column] += V^T P^T
            const uint32_t vt = tile + G_::kV;
            auto product = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                mma<OT>(acc[k], a0, a1, a2, a3, b0, b1);
                if constexpr (G8) mma<OT>(acc[k], a0, a1, a2, a3, b2, b3);
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
                    if constexpr (W == 1) v[r][0] = lds32(vt + place_v<D, KV>(row, g >> 2) + (g & 3) * 4);
                    if constexpr (W == 2) lds64(v[r], vt + place_v<D, KV>(row, g >> 1) + (g & 1) * 8);
                    if constexpr (W == 4) lds128(v[r], vt + place_v<D, KV>(row, g));
                }
                uint32_t h[2][D / 8]; // token pair (2 t4, + 1) and (+ 8, + 9): code pairs by dim
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint32_t x0 = v[2 * r][w], x1 = v[2 * r + 1][w];
                        if constexpr (I4) {
                            widen4(bytes_of(x0, x1, 0x5410), &h[r][8 * w]);
                            widen4(bytes_of(x0, x1, 0x7632), &h[r][8 * w + 4]);
                        } else {
                            widen8(bytes_of(x0, x1, 0x5140), &h[r][4 * w]);
                            widen8(bytes_of(x0, x1, 0x7362), &h[r][4 * w + 2]);
                        }
                    }
#pragma unroll
                for (int k = 0; k < KS; ++k) product(k, h[0][k], h[0][k + KS], h[1][k], h[1][k + KS]);
            }
        }
        cp_wait<0>();

        // ---- this warp's sums over its token rows, then the four warps' together
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            if constexpr (I4) {
                z0 += __shfl_xor_sync(0xffffffffu, z0, o);
                z1 += __shfl_xor_sync(0xffffffffu, z1, o);
            }
        }
        if (g == 0) {
            sm_m[warp][2 * t4] = m0;
            sm_m[warp][2 * t4 + 1] = m1;
            sm_l[warp][2 * t4] = l0;
            sm_l[warp][2 * t4 + 1] = l1;
            sm_z[warp][2 * t4] = z0;
            sm_z[warp][2 * t4 + 1] = z1;
        }
        __syncthreads(); // every warp is done with its ring: it holds the accumulators now
        float *oacc = reinterpret_cast<float *>(smem); // [warp][8 columns][D]
        {
            float f = I4 ? A : 1.f;
            if constexpr (KV == PKV_FP8_E4M3) f = a.v_scale[kvh];
            float *o0 = oacc + (warp * 8 + 2 * t4) * D, *o1 = o0 + D;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int d0 = G_::kBits == 16 ? 16 * k + g : (D / 8) * g + k;
                const int d1 = G_::kBits == 16 ? d0 + 8 : d0 + KS;
                o0[d0] = acc[k][0] * f;
                o1[d0] = acc[k][1] * f;
                o0[d1] = acc[k][2] * f;
                o1[d1] = acc[k][3] * f;
            }
        }
        if (threadIdx.x < G) { // per head: the warps' weights, the maximum, the sum
            const int h = threadIdx.x;
            float Mx = -INFINITY, den = 0.f;
            for (int w = 0; w < kWarps; ++w) Mx = fmaxf(Mx, sm_m[w][h]);
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm_m[w][h] == -INFINITY ? 0.f : sm_m[w][h] == Mx ? 1.f : fast_exp2(sm_m[w][h] - Mx);
                sm_w[w][h] = f;
                if (f != 0.f) den = fmaf(f, sm_l[w][h], den);
            }
            sm_M[h] = Mx == -INFINITY ? 0.f : Mx;
            sm_inv[h] = den == 0.f ? 0.f : 1.f / den;
            if (nsplit > 1) {
                float *ml = a.ws_ml + (((int64_t)s * a.hq + kvh * G + h) * a.max_splits + j) * 2;
                ml[0] = Mx;
                ml[1] = den;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < G * D; e += kThreads) {
            const int h = e / D, d = e % D;
            float num = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                float v = oacc[(w * 8 + h) * D + d];
                if constexpr (!G8) v += oacc[(w * 8 + h + 4) * D + d];
                if constexpr (I4) v += sm_z[w][h];
                if (sm_w[w][h] != 0.f) num = fmaf(sm_w[w][h], v, num);
            }
            const int64_t row = (int64_t)s * a.hq + kvh * G + h;
            if (nsplit > 1)
                a.ws_o[(row * a.max_splits + j) * D + d] = num;
            else
                static_cast<typename M::T *>(a.out)[row * D + d] = M::from_f(num * sm_inv[h]);
        }
        if constexpr (MASS) {
            if (nsplit == 1) add_mass(a, (int64_t)s * a.hkv + kvh, 0, L, sm_M, sm_inv);
        }
    }
    pdl_trigger();
}

// Joins the splits of each (sequence, KV head): out = sum_j w_j o_j / sum_j w_j l_j with
// w_j = 2^(m_j - max m), splits in order; MASS: block y also adds the mass of split y's tokens.
template <int D, int MT, bool MASS>
__global__ void __launch_bounds__(kThreads) merge_kernel(const Args a) {
    using M = ModelT<MT>;
    __shared__ float sm_M[8], sm_inv[8];
    extern __shared__ float wj[]; // [G][max_splits]
    pdl_wait();
    const int row = blockIdx.x, s = row / a.hkv, kvh = row - s * a.hkv, G = a.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = row_len(a, s);
    const int nsplit = (L + a.split_tokens - 1) / a.split_tokens;
    if (nsplit <= 1 || (MASS && (int)blockIdx.y >= nsplit)) return;
    for (int h = warp; h < G; h += kWarps) {
        const float2 *ml =
            reinterpret_cast<const float2 *>(a.ws_ml) + ((int64_t)s * a.hq + kvh * G + h) * a.max_splits;
        float Mx = -INFINITY, den = 0.f;
        for (int j = lane; j < nsplit; j += 32) Mx = fmaxf(Mx, ml[j].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, o));
        for (int j = lane; j < nsplit; j += 32) {
            const float2 v = ml[j];
            const float f = v.x == -INFINITY ? 0.f : v.x == Mx ? 1.f : fast_exp2(v.x - Mx);
            wj[h * a.max_splits + j] = f;
            if (f != 0.f) den = fmaf(f, v.y, den);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
        if (lane == 0) {
            sm_M[h] = Mx == -INFINITY ? 0.f : Mx;
            sm_inv[h] = den == 0.f ? 0.f : 1.f / den;
        }
    }
    __syncthreads();
    const int parts = MASS ? nsplit : gridDim.y;
    for (int e = blockIdx.y * kThreads + threadIdx.x; e < G * D; e += parts * kThreads) {
        const int h = e / D, d = e % D;
        const int64_t r = (int64_t)s * a.hq + kvh * G + h;
        const float *o = a.ws_o + r * a.max_splits * D + d;
        const float *w = wj + h * a.max_splits;
        float num = 0.f;
#pragma unroll 8
        for (int j = 0; j < nsplit; ++j) {
            const float v = o[(int64_t)j * D];
            if (w[j] != 0.f) num = fmaf(w[j], v, num);
        }
        static_cast<typename M::T *>(a.out)[r * D + d] = M::from_f(num * sm_inv[h]);
    }
    if constexpr (MASS) {
        const int t0 = blockIdx.y * a.split_tokens;
        add_mass(a, row, t0, min(L, t0 + a.split_tokens), sm_M, sm_inv);
    }
}

template <int D, int KV, int MT, bool G8, bool MASS>
cudaError_t launch_decode_t(const Args &a, int sms, cudaStream_t st) {
    auto kern = decode_kernel<D, KV, MT, G8, MASS>;
    using G_ = Geo<D, KV>;
    const size_t ring = (size_t)kWarps * G_::kStages * G_::kBytes;
    static_assert(kWarps * G_::kStages * G_::kBytes >= kWarps * 8 * D * 4, "the accumulators reuse the ring");
    const size_t smem = ring + (2 * (a.num_seqs + 1) + (a.split_tokens >> a.bs_log2)) * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.num_seqs * a.hkv * (a.max_splits > 0 ? a.max_splits : 1);
    const int64_t slots = (int64_t)sms * G_::kCtas;
    return pdl_launch(kern, dim3((unsigned)(units < slots ? units : slots)), dim3(kThreads), smem, st, a);
}

template <int D, int MT, bool MASS>
cudaError_t launch_merge_t(const Args &a, cudaStream_t st) {
    const unsigned y = MASS ? a.max_splits : (a.group * D + kThreads - 1) / kThreads;
    const size_t smem = (size_t)a.group * a.max_splits * sizeof(float);
    auto kern = merge_kernel<D, MT, MASS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return pdl_launch(kern, dim3((unsigned)(a.num_seqs * a.hkv), y), dim3(kThreads), smem, st, a);
}

// one cache type's kernels (one translation unit each)
template <int KV, int MT, bool MASS>
cudaError_t dispatch(const Args &a, int D, int sms, bool merge, cudaStream_t st) {
    if (merge) return D == 64 ? launch_merge_t<64, MT, MASS>(a, st) : launch_merge_t<128, MT, MASS>(a, st);
    if (D == 64)
        return a.group == 8 ? launch_decode_t<64, KV, MT, true, MASS>(a, sms, st)
                            : launch_decode_t<64, KV, MT, false, MASS>(a, sms, st);
    return a.group == 8 ? launch_decode_t<128, KV, MT, true, MASS>(a, sms, st)
                        : launch_decode_t<128, KV, MT, false, MASS>(a, sms, st);
}

} // namespace pkv_mma

cudaError_t pkv_mma_int4(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_int4_mass(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_fp8_mass(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_16bit_mass(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
