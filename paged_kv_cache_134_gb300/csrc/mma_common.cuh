// What the decode kernels of 4-bit caches and of the attention mass share (decode_int4.cuh, decode_mma.cuh, and for
// rows of a few tokens decode_short.cuh): arguments, PTX wrappers,
// the list of units, the join of a unit's warps and of a row's splits, the attention mass.
//
// A unit is (sequence, KV head, split of split_tokens tokens); persistent CTAs of four warps walk the units,
// whole splits first.  Each warp keeps the running maximum m, the sum l and the accumulator of its tokens;
// a unit's four are joined through shared memory in a fixed order.  A row's splits leave fp32 partials
// (m, l, o): up to kJoinSplits of them are joined by the CTA that finishes the row last (a counter per row
// that it sets back to 0), in split order, so the result does not depend on which CTA that is; more by
// merge_kernel, whose CTAs share them out.  With attention mass a second kernel, mass_kernel, walks the same
// units: it joins the splits and turns the stored scores into weights, which needs the row's final
// maximum and sum.  (Done by the row's last CTA instead, it kept one CTA busy with a whole row at the end:
// 65 us more on 32 fp16 sequences of up to 4096 tokens, 32 heads.)
#pragma once

#include <type_traits>

#include "device_common.cuh"
#include "int4.cuh"
#include "pkv_internal.h"

namespace pkv_mma {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSeqs = 1024;   // sequences of a launch (their unit counts sit in shared memory)
constexpr int kShortTokens = 32; // tokens of a row that one warp may take whole (decode_short.cuh): a lane each
constexpr int kJoinSplits = 16;  // splits of a row that its last CTA joins itself

struct Args {
    const void *q;
    void *out;
    const char *pool;
    const float *k_scale, *v_scale; // E4M3 caches
    const int32_t *tables, *lens;
    float *ws_o, *ws_ml; // [S * Hq][max_splits][D], [S * Hq][max_splits][2]
    float *ws_x;         // mass: scores in log2 units, [S * Hkv][cap][G]
    int *done;           // units finished per row, [S * Hkv], all 0 between launches; NULL: merge_kernel joins
    float *mass;         // [S][Hkv][mass_len]
    unsigned int *err;
    int64_t num_blocks;
    int64_t blk_stride, head_stride, v_off; // bytes: block, head, V behind K
    int64_t mass_len, cap;                  // tokens of a mass row; tokens a sequence may have
    int max_blocks, num_seqs, hq, hkv, group, bs_log2;
    int split_tokens, max_splits;
    uint32_t hkv_magic; // x / hkv = x * hkv_magic >> hkv_shift for 0 <= x < 2^31
    int hkv_shift;
    float qk_scale_log2; // scale * log2(e)
    float decay;
    int window, sinks; // WIN kernels: what is attended to (see Reach)
};

// attention of several new tokens a sequence (chunk_few.cuh)
struct FewArgs : Args {
    const int32_t *cu; // rows of sequence s: [cu[s], cu[s + 1])
    int64_t total;     // rows of q
    int max_seqlen, lg_group;
    int most_rows; // sequences of more rows a KV head are left aside
    int row_room;  // rows that a (sequence, KV head) has room for in the workspace: ws_o, ws_ml by (s, kvh, split, row)
    bool late;     // see few_kernel
};

// (the offset rides in the instruction: no address to compute)
template <int OFF = 0>
PKV_DEV void lds64(uint32_t *w, uint32_t a) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(w[0]), "=r"(w[1]) : "r"(a), "n"(OFF));
}
template <int OFF = 0>
PKV_DEV void lds128(uint32_t *w, uint32_t a) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a), "n"(OFF));
}
template <int OFF = 0>
PKV_DEV uint32_t lds32(uint32_t a) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(w) : "r"(a), "n"(OFF));
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

// c = a b
template <int OT>
PKV_DEV void mma_first(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    const float z = 0.f;
    if constexpr (OT == PKV_F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z));
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


template <int OT> // fp32 pair -> 16-bit pair, towards zero
PKV_DEV uint32_t pack_rz(float lo, float hi) {
    uint32_t r;
    if constexpr (OT == PKV_F16)
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// the part of x that pack_rz keeps (of a normal number)
template <int OT>
PKV_DEV float kept_rz(float x) {
    return __uint_as_float(__float_as_uint(x) & (OT == PKV_F16 ? 0xFFFFE000u : 0xFFFF0000u));
}

PKV_DEV int row_len(const Args &a, int s) {
    const int L = a.lens[s];
    return L <= 0 ? 0 : (int64_t)L > a.cap ? (int)a.cap : L;
}

// what sequence s shows, if it holds L tokens
template <bool WIN>
PKV_DEV Reach sight_of(const Args &a, int s, int L) {
    if constexpr (WIN) return reach_of(L, a.window, a.sinks, 1 << a.bs_log2);
    return {L, 0, 0, 0, 0};
}
PKV_DEV void report_row(const Args &a, int s) {
    if ((int64_t)a.lens[s] > a.cap) set_error(a.err, PKV_DEVERR_LENGTH);
}
PKV_DEV bool has_rows(const Args &, int) { return true; }

// Windows without splits, more units than CTAs: sequences of most tokens first, in eight classes, so that the CTAs, which take
// every gridDim-th unit, end together.  full[0 .. S) is then the order, full[S] = 0, part[S] = S.  (256 log-normal
// sequences, 32/8 heads, by order of the batch and by length: window 1024 over E4M3 64.7 and 59.6 us, bf16 101.0 and 96.4,
// of 64 dimensions 63.0 and 58.5; 511 over E4M3 46.7 and 46.5, bf16, where all SMs wait for memory anyway, 68.7 and 70.0.)
PKV_DEV bool by_length(const Args &a) {
    return a.max_splits == 1 && a.num_seqs >= 31 && (int64_t)a.num_seqs * a.hkv > (int64_t)gridDim.x;
}
template <typename A>
PKV_DEV void list_by_length(const A &a, int *full, int *part) {
    const int S = a.num_seqs, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = (S + 31) >> 5;
    int *len = part + S + 1, *count = part; // [class][chunk of 32 sequences]: 8 chunks <= S + 1 for S >= 31
    uint32_t classes = 0; // this lane's sequences', four bits each (at most 1024 sequences: 8 chunks a warp)
    for (int k = warp; k < chunks; k += kWarps) {
        const int s = k * 32 + lane;
        int cls = 8;
        if (s < S) {
            const int L = row_len(a, s), n = sight_of<true>(a, s, L).len;
            if (blockIdx.x == 0) report_row(a, s);
            len[s] = L;
            cls = 7;
#pragma unroll
            for (int i = 1; i < 8; ++i) cls -= 8 * (int64_t)n >= (int64_t)i * a.split_tokens;
        }
        classes = classes << 4 | cls;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = __popc(__ballot_sync(0xffffffffu, cls == i));
            if (lane == i) count[i * chunks + k] = n;
        }
    }
    __syncthreads();
    if (warp == 0) {
        int sum = 0;
        for (int i = 0; i < 8 * chunks; i += 32) {
            const int n = i + lane < 8 * chunks ? count[i + lane] : 0;
            int v = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += w;
            }
            if (i + lane < 8 * chunks) count[i + lane] = sum + v - n;
            sum += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    for (int k = warp; k < chunks; k += kWarps) {
        const int s = k * 32 + lane, cls = classes >> (4 * ((chunks - 1 - k) / kWarps)) & 15;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned same = __ballot_sync(0xffffffffu, cls == i);
            if (cls == i) full[count[i * chunks + k] + __popc(same & ((1u << lane) - 1))] = s;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        full[S] = 0;
        part[S] = S;
    }
    __syncthreads();
}

// Block scan of the sequences' unit counts: full[s + 1], part[s + 1] hold the inclusive sums of whole
// splits and of partial ones (a sequence of length 0 has one partial unit, which writes its zero row); the lengths lie
// behind part.  WIN: units of what is in sight (see Reach).
template <bool WIN = false, typename A = Args>
PKV_DEV void list_units(const A &a, int *full, int *part, int *tmp) {
    if constexpr (WIN)
        if (by_length(a)) return list_by_length(a, full, part);
    const int S = a.num_seqs, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *len = part + S + 1;
    int cf = 0, cp = 0; // sums of the sequences before this pass
    if (threadIdx.x == 0) full[0] = part[0] = 0;
    for (int s0 = 0; s0 < S; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        int f = 0, p = 0;
        if (s < S) {
            const int L = row_len(a, s);
            if (blockIdx.x == 0) report_row(a, s);
            len[s] = L;
            if (has_rows(a, s)) {
                const int n = sight_of<WIN>(a, s, L).len;
                f = n / a.split_tokens;
                p = (n % a.split_tokens != 0 || n == 0) ? 1 : 0;
            }
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

// Largest i in [0, n) with pref[i] <= k (pref[0] = 0 <= k, non-decreasing, n <= 1024): a warp looks at 32 places at once.
PKV_DEV int find_row(const int *pref, int n, int k) {
    const int lane = threadIdx.x & 31, stride = (n + 31) >> 5;
    const int at = lane * stride;
    const int block = __popc(__ballot_sync(0xffffffffu, at < n && pref[at] <= k)) - 1;
    const int i = block * stride + lane;
    return block * stride + __popc(__ballot_sync(0xffffffffu, lane < stride && i < n && pref[i] <= k)) - 1;
}

struct Unit {
    int s, kvh, j, nsplit;
    int t0, n; // first token, tokens
};

// WIN: t0 counts the tokens in sight; block i of them is logical block i, or i + skip from block `from` on, and [lo, hi) are
// hidden.
struct SeenUnit : Unit {
    int from, skip, lo, hi;
};
template <bool WIN>
using UnitOf = std::conditional_t<WIN, SeenUnit, Unit>;

// Unit u of the list (all lanes of a warp together, u the same for all).
template <bool WIN = false, typename A = Args>
PKV_DEV UnitOf<WIN> unit_of(const A &a, const int *full, const int *part, int nfull, int u) {
    UnitOf<WIN> r;
    const bool whole = u < nfull;
    const int v = whole ? u : u - nfull;
    const int k = (int)(((uint64_t)(uint32_t)v * a.hkv_magic) >> a.hkv_shift); // v / hkv
    r.kvh = v - k * a.hkv;
    const bool ordered = WIN && by_length(a);
    if (ordered) {
        r.s = full[k];
        r.j = 0;
    } else {
        r.s = find_row(whole ? full : part, a.num_seqs, k);
        r.j = whole ? k - full[r.s] : full[r.s + 1] - full[r.s];
    }
    int L = part[a.num_seqs + 1 + r.s];
    if constexpr (WIN) {
        const Reach rc = sight_of<true>(a, r.s, L);
        L = rc.len;
        r.from = rc.from;
        r.skip = rc.skip;
        r.lo = rc.lo;
        r.hi = rc.hi;
    }
    r.nsplit = ordered ? 1 : (full[r.s + 1] - full[r.s]) + (part[r.s + 1] - part[r.s]);
    r.t0 = r.j * a.split_tokens;
    r.n = min(L - r.t0, a.split_tokens);
    return r;
}

// What a unit needs besides its tiles: its table entries and its q rows (group x D, as they lie).
// They are copied to shared memory a unit ahead.
PKV_DEV int blocks_of(const Args &a, const Unit &u) { return (u.n + (1 << a.bs_log2) - 1) >> a.bs_log2; }

// Checks entries that have landed: an id that is no block becomes -1.  Returns whether this thread met one.
// i0, step: this thread's share
PKV_DEV bool check_table(const Args &a, const Unit &u, int *tb, int i0, int step) {
    bool bad = false;
    const int nblk = blocks_of(a, u);
    for (int i = i0; i < nblk; i += step) {
        const int b = tb[i];
        if (b < 0 || b >= a.num_blocks) {
            set_error(a.err, PKV_DEVERR_BLOCK_ID);
            bad = true;
            tb[i] = -1;
        }
    }
    return bad;
}

PKV_DEV void cp16(uint32_t dst, const char *src, int bytes) { // bytes < 16: zeros behind them
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
PKV_DEV void cp4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
PKV_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
PKV_DEV void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// issue only: the caller commits and waits
template <int D, typename U>
PKV_DEV void stage_unit(const Args &a, const U &u, int *tb, char *qs, int i0, int step) {
    const int nblk = blocks_of(a, u);
    const int32_t *row = a.tables + (int64_t)u.s * a.max_blocks + (u.t0 >> a.bs_log2);
    for (int i = i0; i < nblk; i += step) {
        int at = i;
        if constexpr (std::is_same_v<U, SeenUnit>) at += (u.t0 >> a.bs_log2) + i >= u.from ? u.skip : 0;
        cp4(smem_u32(tb + i), row + at);
    }
    const char *q = static_cast<const char *>(a.q) + ((int64_t)u.s * a.hq + u.kvh * a.group) * (D * 2);
    for (int i = i0; i < a.group * (D / 8); i += step) cp16(smem_u32(qs) + i * 16, q + i * 16, 16);
}

struct Join {
    float m[kWarps][8], l[kWarps][8], z[kWarps][8]; // per warp and column
    float M[8], inv[8];
    float wj[8][kJoinSplits];
    int last;
};

// The running maxima pass over NaN, so what saw nothing else keeps -inf and weighs 0: its sums are NaN, and are multiplied
// by their weight whatever that is, so that a row with a NaN score (or a NaN in V) comes out NaN however it was split.
PKV_DEV float weight_of(float m, float M) { return m == -INFINITY ? 0.f : m == M ? 1.f : fast_exp2(m - M); }

// Row (s, kvh)'s splits: maxima, reciprocal sums (M, inv) and the splits' weights w[h * ldw + j] per head.
// One warp per head; the caller synchronises.
PKV_DEV void split_weights(const Args &a, int s, int kvh, int nsplit, float *w, int ldw, float *M, float *inv) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int h = warp; h < a.group; h += blockDim.x / 32) {
        const float2 *ml =
            reinterpret_cast<const float2 *>(a.ws_ml) + ((int64_t)s * a.hq + kvh * a.group + h) * a.max_splits;
        const float2 none = make_float2(-INFINITY, 0.f);
        float2 v = lane < nsplit ? __ldcg(ml + lane) : none;
        float Mx = v.x, den = 0.f;
        for (int j = lane + 32; j < nsplit; j += 32) Mx = fmaxf(Mx, __ldcg(ml + j).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, o));
        for (int j = lane; j < nsplit; j += 32) {
            if (j >= 32) v = __ldcg(ml + j);
            const float f = weight_of(v.x, Mx);
            w[h * ldw + j] = f;
            den = fmaf(f, v.y, den);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
        if (lane == 0) {
            M[h] = Mx == -INFINITY ? 0.f : Mx;
            inv[h] = den == 0.f ? 0.f : 1.f / den;
        }
    }
}

// The end of a unit, in three steps.  1: each warp stores its columns' maxima (store_max); barrier.  2: it takes
// its weight 2^(m - max over the warps) per column and stores its sum, offsets' sum and accumulator already
// weighted.  3 (join_unit): barrier, the four warps' values added in a fixed order; leaves a barrier behind.
struct Weight {
    float M, w; // the unit's maximum of the column, this warp's weight
};
PKV_DEV Weight warp_weight(const Join &J, int warp, int column) {
    Weight r;
    r.M = fmaxf(fmaxf(J.m[0][column], J.m[1][column]), fmaxf(J.m[2][column], J.m[3][column]));
    r.w = weight_of(J.m[warp][column], r.M);
    return r;
}

// MASS: the unit's (m, l) is kept for mass_kernel even where the row is one unit.  I4: the accumulators are of
// codes that read 2^-21 (even elements) and 2^-17, without the offsets' sum.
template <int D, int COLS, int MT, bool MASS, bool I4>
PKV_DEV void join_unit(const Args &a, const Unit &u, Join &J, const float *oacc) {
    using M_ = ModelT<MT>;
    constexpr int LD = D + 4;
    const int G = a.group;
    __syncthreads();
    for (int e = threadIdx.x; e < G * (D / 4); e += kThreads) {
        const int h = e / (D / 4), d = e % (D / 4) * 4;
        const float *o = oacc + h * LD + d;
        float4 v[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v[w] = *reinterpret_cast<const float4 *>(o + w * COLS * LD);
        float n[4] = {((v[0].x + v[1].x) + v[2].x) + v[3].x, ((v[0].y + v[1].y) + v[2].y) + v[3].y,
                      ((v[0].z + v[1].z) + v[2].z) + v[3].z, ((v[0].w + v[1].w) + v[2].w) + v[3].w};
        const float den = ((J.l[0][h] + J.l[1][h]) + J.l[2][h]) + J.l[3][h];
        if constexpr (I4) {
            const float z = ((J.z[0][h] + J.z[1][h]) + J.z[2][h]) + J.z[3][h];
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = fmaf(n[i], i & 1 ? 131072.f : 2097152.f, z);
        }
        const int64_t row = (int64_t)u.s * a.hq + u.kvh * G + h;
        if ((MASS || u.nsplit > 1) && d == 0)
            reinterpret_cast<float2 *>(a.ws_ml)[row * a.max_splits + u.j] = make_float2(J.M[h], den);
        if (u.nsplit > 1) {
            *reinterpret_cast<float4 *>(a.ws_o + (row * a.max_splits + u.j) * D + d) = make_float4(n[0], n[1], n[2], n[3]);
        } else {
            const float inv = den == 0.f ? 0.f : 1.f / den;
            *reinterpret_cast<uint2 *>(static_cast<char *>(a.out) + (row * D + d) * 2) =
                den == 0.f ? make_uint2(0u, 0u)
                           : make_uint2(M_::pack(n[0] * inv, n[1] * inv), M_::pack(n[2] * inv, n[3] * inv));
        }
    }
    __syncthreads();
}

// A finished unit is counted when the next one starts (its partials have landed by then, and the counter's answer
// comes while that one runs).  Thread 0; after the barrier join_unit leaves.
PKV_DEV int count_unit(const Args &a, const Unit &u) {
    __threadfence(); // the unit's partials before its count
    const int before = atomicAdd(a.done + (int64_t)u.s * a.hkv + u.kvh, 1);
    return before;
}

// The row whose last unit u was: joins its splits.  All threads; starts and leaves with a barrier.
template <int D, int MT>
PKV_DEV void join_row(const Args &a, const Unit &u, Join &J) {
    using M_ = ModelT<MT>;
    const int G = a.group;
    const int64_t row = (int64_t)u.s * a.hkv + u.kvh;
    if (threadIdx.x == 0) a.done[row] = 0;
    split_weights(a, u.s, u.kvh, u.nsplit, &J.wj[0][0], kJoinSplits, J.M, J.inv);
    __syncthreads();
    for (int e = threadIdx.x; e < G * (D / 4); e += kThreads) {
        const int h = e / (D / 4), d = e % (D / 4) * 4;
        const int64_t r = (int64_t)u.s * a.hq + u.kvh * G + h;
        const float *o = a.ws_o + r * a.max_splits * D + d;
        float4 n = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int j = 0; j < u.nsplit; ++j) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(o + (int64_t)j * D));
            const float w = J.wj[h][j];
            n.x = fmaf(w, v.x, n.x);
            n.y = fmaf(w, v.y, n.y);
            n.z = fmaf(w, v.z, n.z);
            n.w = fmaf(w, v.w, n.w);
        }
        const float inv = J.inv[h];
        *reinterpret_cast<uint2 *>(static_cast<char *>(a.out) + (r * D + d) * 2) =
            make_uint2(M_::pack(n.x * inv, n.y * inv), M_::pack(n.z * inv, n.w * inv));
    }
    __syncthreads();
}

// sum over the lanes that share a column (the token rows)
PKV_DEV float row_sum(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Joins the splits of a row: block (row, y) takes every gridDim.y-th run of 32 outputs; each warp adds every
// kMergeWarps-th split in order, their sums are joined in warp order.  Rows come here with more than kJoinSplits
// splits: sixteen warps keep enough loads in flight.
constexpr int kMergeWarps = 16;
constexpr int kMassCtas = 8;

template <int D, int MT, bool WIN = false>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const Args a) {
    using M = ModelT<MT>;
    __shared__ float sm_M[8], sm_inv[8], sum[kMergeWarps][32];
    extern __shared__ float wj[]; // [G][max_splits]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int row = blockIdx.x, s = row / a.hkv, kvh = row - s * a.hkv;
    const int n = sight_of<WIN>(a, s, row_len(a, s)).len;
    const int nsplit = (n + a.split_tokens - 1) / a.split_tokens;
    if (nsplit <= 1) return;
    split_weights(a, s, kvh, nsplit, wj, a.max_splits, sm_M, sm_inv);
    __syncthreads();
    for (int e0 = blockIdx.y * 32; e0 < a.group * D; e0 += gridDim.y * 32) {
        const int h = e0 / D, d = e0 % D + lane;
        const int64_t r = (int64_t)s * a.hq + kvh * a.group + h;
        const float *o = a.ws_o + r * a.max_splits * D + d;
        const float *w = wj + h * a.max_splits;
        float num = 0.f;
#pragma unroll 8
        for (int j = warp; j < nsplit; j += kMergeWarps) {
            const float v = o[(int64_t)j * D];
            num = fmaf(w[j], v, num);
        }
        sum[warp][lane] = num;
        __syncthreads();
        if (warp == 0) {
            num = sum[0][lane];
#pragma unroll
            for (int w = 1; w < kMergeWarps; ++w) num += sum[w][lane];
            static_cast<typename M::T *>(a.out)[r * D + d] = M::from_f(num * sm_inv[h]);
        }
        __syncthreads();
    }
}

// After a decode that stored its scores: for every unit the mass of its tokens, and its share of the row's outputs
// where the row has several splits.  Persistent, the decode's list of units.  Bound by latency (the scores are mostly in L2):
// a unit waits once for its scores and the row's statistics together.  256 ragged sequences, 1.6 M (token, KV head)
// pairs of four heads: 13 us behind the decode's 61; a CTA needs 64 registers, more of them an SM were no faster.
struct MassShared {
    float M[8], inv[8];
    float4 part[kThreads];
    int tmp[2 * kWarps];
};

// G heads, U tokens a thread at a time; a unit's first scores are on their way while the row's splits are weighed.
template <int D, int MT, int G, int U>
PKV_DEV void mass_units(const Args &a, MassShared &sm, float *wj, const int *full, const int *part) {
    using M_ = ModelT<MT>;
    const int nfull = full[a.num_seqs] * a.hkv, nunits = nfull + part[a.num_seqs] * a.hkv;
    for (int ui = blockIdx.x; ui < nunits; ui += gridDim.x) {
        const Unit u = unit_of(a, full, part, nfull, ui);
        if (u.n <= 0) continue; // an empty sequence
        const int64_t row = (int64_t)u.s * a.hkv + u.kvh;
        const float *x = a.ws_x + (row * a.cap + u.t0) * G;
        float *m = a.mass + row * a.mass_len + u.t0;
        float xs[U][G], old[U];
        auto load = [&](int tb) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int t = tb + i * kThreads;
                if (t >= u.n) continue;
                const float *src = x + (int64_t)t * G;
                if constexpr (G == 1) {
                    xs[i][0] = __ldcg(src);
                } else if constexpr (G == 2) {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                    xs[i][0] = v.x;
                    xs[i][1] = v.y;
                } else {
#pragma unroll
                    for (int h = 0; h < G; h += 4) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + h));
                        xs[i][h] = v.x;
                        xs[i][h + 1] = v.y;
                        xs[i][h + 2] = v.z;
                        xs[i][h + 3] = v.w;
                    }
                }
                old[i] = m[t];
            }
        };
        load(threadIdx.x);
        split_weights(a, u.s, u.kvh, u.nsplit, wj, a.max_splits, sm.M, sm.inv);
        __syncthreads();
        float M[G], inv[G];
#pragma unroll
        for (int h = 0; h < G; ++h) M[h] = sm.M[h], inv[h] = sm.inv[h];
        for (int tb = threadIdx.x; tb < u.n; tb += kThreads * U) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int t = tb + i * kThreads;
                if (t >= u.n) continue;
                float p = 0.f;
#pragma unroll
                for (int h = 0; h < G; ++h) p = fmaf(fast_exp2(xs[i][h] - M[h]), inv[h], p);
                m[t] = fmaf(old[i], a.decay, p);
            }
            load(tb + kThreads * U);
        }
        if (u.nsplit > 1) {
            // the unit's share: c runs of four outputs, at most one a thread.  K threads a run take every K-th
            // split, their sums are added in order.
            constexpr int V = G * D / 4;
            const int i0 = V * u.j / u.nsplit, c = V * (u.j + 1) / u.nsplit - i0;
            if (c > 0) {
                const int K = min(kThreads / c, u.nsplit), k = threadIdx.x / c, i = i0 + threadIdx.x - k * c;
                const int h = i / (D / 4), d = i % (D / 4) * 4;
                const int64_t r = (int64_t)u.s * a.hq + u.kvh * G + h;
                if (k < K) {
                    const float *o = a.ws_o + r * a.max_splits * D + d, *w = wj + h * a.max_splits;
                    float4 n = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int j = k; j < u.nsplit; j += K) {
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(o + (int64_t)j * D));
                        n.x = fmaf(w[j], v.x, n.x);
                        n.y = fmaf(w[j], v.y, n.y);
                        n.z = fmaf(w[j], v.z, n.z);
                        n.w = fmaf(w[j], v.w, n.w);
                    }
                    sm.part[threadIdx.x] = n;
                }
                __syncthreads();
                if (k == 0) {
                    float4 n = sm.part[threadIdx.x];
                    for (int q = 1; q < K; ++q) {
                        const float4 v = sm.part[q * c + threadIdx.x];
                        n.x += v.x;
                        n.y += v.y;
                        n.z += v.z;
                        n.w += v.w;
                    }
                    const float f = sm.inv[h];
                    *reinterpret_cast<uint2 *>(static_cast<char *>(a.out) + (r * D + d) * 2) =
                        make_uint2(M_::pack(n.x * f, n.y * f), M_::pack(n.z * f, n.w * f));
                }
            }
        }
        __syncthreads();
    }
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, kMassCtas) mass_kernel(const Args a) {
    __shared__ MassShared sm;
    extern __shared__ float wj[]; // [G][max_splits], then the list of units
    int *full = reinterpret_cast<int *>(wj + a.group * a.max_splits), *part = full + a.num_seqs + 1;
    // (the lengths were complete before the decode began, so the list need not wait for its end)
    list_units(a, full, part, sm.tmp);
    pdl_wait();
    if (a.group == 1)
        mass_units<D, MT, 1, 8>(a, sm, wj, full, part);
    else if (a.group == 2)
        mass_units<D, MT, 2, 4>(a, sm, wj, full, part);
    else if (a.group == 4)
        mass_units<D, MT, 4, 4>(a, sm, wj, full, part);
    else
        mass_units<D, MT, 8, 2>(a, sm, wj, full, part);
}

// Resident CTAs per SM: `want`, or what the shared memory holds (228 KB an SM; a CTA has up to 1.5 KB of its own and 1 KB
// of the system's besides).  A CTA more would wait for a whole walk over the units to end.
inline int ctas_of(int want, size_t smem) {
    const int fit = (int)(233472 / (smem + 2560));
    return fit < 1 ? 1 : fit < want ? fit : want;
}

inline unsigned grid_of(const Args &a, int slots) {
    const int64_t units = (int64_t)a.num_seqs * a.hkv * (a.max_splits > 0 ? a.max_splits : 1);
    return (unsigned)(units < slots ? units : slots);
}

// the launch after the decode: merge_kernel, or mass_kernel
template <int D, int MT, bool MASS, bool WIN = false>
cudaError_t launch_merge_t(const Args &a, int sms, cudaStream_t st) {
    const size_t smem = (size_t)a.group * a.max_splits * sizeof(float);
    if constexpr (MASS) {
        return pdl_launch(mass_kernel<D, MT>, dim3(grid_of(a, kMassCtas * sms)), dim3(kThreads),
                          smem + 3 * (a.num_seqs + 1) * sizeof(int), st, a);
    } else {
        return pdl_launch(merge_kernel<D, MT, WIN>, dim3((unsigned)(a.num_seqs * a.hkv), a.group * D / 32),
                          dim3(kMergeWarps * 32),
                          smem, st, a);
    }
}

} // namespace pkv_mma

cudaError_t pkv_mma_int4(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_int4_window(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_16bit_window(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_fp8_window(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_int4_mass(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_fp8_mass(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_mma_16bit_mass(const pkv_mma::Args &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_few_16bit(const pkv_mma::FewArgs &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_few_e4m3(const pkv_mma::FewArgs &, int mt, int D, int sms, bool merge, cudaStream_t);
cudaError_t pkv_short_int4(const pkv_mma::Args &, int mt, int D, cudaStream_t);
cudaError_t pkv_short_fp8(const pkv_mma::Args &, int mt, int D, cudaStream_t);
cudaError_t pkv_short_16bit(const pkv_mma::Args &, int mt, int D, cudaStream_t);
