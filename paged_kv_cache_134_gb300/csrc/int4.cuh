// The 4-bit cache: layout and arithmetic of its rows.
//
// A (block, KV head) is one run of bs * (D + 8) bytes, an octet of 8 tokens after the other:
//     K codes [8][D / 2] | V codes [8][D / 2] | K (s, z) [8][2] | V (s, z) [8][2]
// so that the K and V of any 8 tokens of a head are one aligned run (one bulk copy brings a 16-token tile
// of a block), and a whole block, scales and all, is one run for block copy and swap.  s and z are in the
// model's type.  Elements 4 i .. 4 i + 3 of a row are the nibbles of its 16-bit word i, lowest first, the
// word rotated left by three bits: a nibble in bits 7..10 or 3..6 of an fp16 reads c 2^-17 or c 2^-21 (fp16
// numbers are evenly spaced up to bit 10), and exchanging the word's bytes brings the other two there.
// V's rows stand in the order 0 2 4 6 1 3 5 7, and at D = 128 those of places 2, 3, 6 and 7 with their
// halves swapped: the attention reads rows 0 2 4 6 (then 1 3 5 7) of 8 bytes each at once, and so finds
// them in different banks without copying them around.
//
// One step and one offset per (token, head) row: they then stand outside both matrix products of the
// attention (two scalars per token).  z is an element of the row, so the model's type holds it exactly;
// rounding s to the model's type moves the largest value by at most 15 * 2^-9 (bf16) of a step, against
// the half step of the codes.
//   * s is taken as 0 below 2^-126 (its reciprocal would overflow); s = 0 (a constant row) stores codes 0.
//   * A row that holds a NaN or an infinity, or whose range overflows fp32, gets s = z = NaN: it reads as
//     NaN throughout, as the attention over a 16-bit cache would return.
#pragma once

#include "device_common.cuh"

PKV_DEV int64_t int4_head(int64_t blk, int h, int hkv, int bs, int d) {
    return (blk * hkv + h) * ((int64_t)bs * (d + 8));
}
PKV_DEV int int4_place(int r) { return (r >> 1) | ((r & 1) << 2); } // V row r of an octet
// from a (block, head)'s start: byte `i` (a multiple of 4) of row `off`'s codes, and its (s, z)
PKV_DEV int int4_codes(int kv, int off, int i, int d) {
    const int oct = (off >> 3) * 8 * (d + 8), r = off & 7;
    if (kv == 0) return oct + r * (d / 2) + i;
    const int p = int4_place(r);
    return oct + 4 * d + p * (d / 2) + (d == 128 ? i ^ ((p & 2) << 4) : i);
}
PKV_DEV int int4_params(int kv, int off, int d) {
    return (off >> 3) * 8 * (d + 8) + 8 * d + kv * 32 + (off & 7) * 4;
}

struct Int4Row {
    uint2 codes;     // of this lane's two runs of eight
    uint32_t params; // s in the low half, z in the high half (the same on every lane of the row)
};

template <int MT>
PKV_DEV uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (MT == PKV_F16)
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int MT>
PKV_DEV uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (MT == PKV_F16)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int MT>
PKV_DEV float half_of(uint32_t w, int i) {
    if constexpr (MT == PKV_F16)
        return __half2float(__ushort_as_half((unsigned short)(i ? w >> 16 : w & 0xFFFFu)));
    else
        return __uint_as_float(i ? w & 0xFFFF0000u : w << 16);
}

// Sixteen elements of a row that the `per_row` lanes of `lanes` hold together (which sixteen is the caller's choice).
// Codes come from quotients d / s rounded as a division rounds them, so that a code does not hang on how it was
// computed.  They are q = d i, i an approximate 1 / s, corrected once by the remainder, q + (d - q s) i (Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, 1990): d - q s is exact, as s
// has at most 11 bits and q is off by a few units, and the sum is off by less than 2^-44 before it is rounded,
// while a quotient of 24 by 11 bits that is no float lies 2^-37 or more from a place where rounding turns.
// Rows with a step below 2^-90, whose remainders would be subnormal, divide; so do rows whose largest quotient passes 15.4
// (a step that the model's type holds to few bits), which are cut at 15.  The step is found the same way.
template <int MT>
PKV_DEV Int4Row int4_quantise(const uint4 (&src)[2], int per_row, unsigned lanes) {
    using M = ModelT<MT>;
    uint32_t lo = min2_nan<MT>(min2_nan<MT>(min2_nan<MT>(src[0].x, src[0].y), min2_nan<MT>(src[0].z, src[0].w)),
                               min2_nan<MT>(min2_nan<MT>(src[1].x, src[1].y), min2_nan<MT>(src[1].z, src[1].w)));
    uint32_t hi = max2_nan<MT>(max2_nan<MT>(max2_nan<MT>(src[0].x, src[0].y), max2_nan<MT>(src[0].z, src[0].w)),
                               max2_nan<MT>(max2_nan<MT>(src[1].x, src[1].y), max2_nan<MT>(src[1].z, src[1].w)));
    // the pair's least and largest as one word: two shuffles a step would carry two words
    lo = min2_nan<MT>(lo, __byte_perm(lo, lo, 0x1032));
    hi = max2_nan<MT>(hi, __byte_perm(hi, hi, 0x1032));
    uint32_t both = __byte_perm(lo, hi, 0x5410); // least low, largest high
    for (int o = 1; o < per_row; o <<= 1) {
        const uint32_t other = __shfl_xor_sync(lanes, both, o);
        both = __byte_perm(min2_nan<MT>(both, other), max2_nan<MT>(both, other), 0x7610);
    }
    const float z = half_of<MT>(both, 0), range = __fsub_rn(half_of<MT>(both, 1), z);
    Int4Row r;
    r.codes = make_uint2(0, 0);
    if (!(range < INFINITY)) { // NaN or overflow; an infinity in the row makes the range one or the other
        r.params = MT == PKV_F16 ? 0x7E007E00u : 0x7FC07FC0u;
        return r;
    }
    constexpr float kTiny = 8.0779357e-28f; // 2^-90
    float step = range * (1.f / 15.f);
    step = range < kTiny ? __fdiv_rn(range, 15.f) : fmaf(fmaf(step, -15.f, range), 1.f / 15.f, step);
    const uint32_t s16 = M::pack(step, 0.f) & 0xFFFFu;
    float s = half_of<MT>(s16, 0);
    if (s < 1.17549435e-38f) s = 0.f; // 2^-126
    r.params = (s == 0.f ? 0u : s16) | (both << 16);
    if (s == 0.f) return r;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s)); // (2^-126 <= s < 2^125: neither end is flushed)
    const float2 inv2 = make_float2(inv, inv), minus_z = make_float2(-z, -z), minus_s = make_float2(-s, -s),
                 zero = make_float2(0.f, 0.f), big = make_float2(12582912.f, 12582912.f);
    uint32_t w[4]; // four codes in the low 16 bits
    if (s < kTiny || range * inv > 15.4f) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float f[8];
            cvt8<MT>(src[u], f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[2 * u + i] = 0;
#pragma unroll
                for (int e = 3; e >= 0; --e)
                    w[2 * u + i] = w[2 * u + i] * 16 + (uint32_t)fminf(rintf(__fdiv_rn(__fsub_rn(f[4 * i + e], z), s)), 15.f);
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float f[8];
            cvt8<MT>(src[u], f);
            uint32_t t[8]; // codes in the low bits of 2^23 + 2^22 + them: the bits above drop out below
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 d = add2(make_float2(f[i], f[i + 1]), minus_z);
                float2 q = fma2(d, inv2, zero);
                q = fma2(fma2(q, minus_s, d), inv2, q);
                q = add2(q, big);
                t[i] = __float_as_uint(q.x);
                t[i + 1] = __float_as_uint(q.y);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[2 * u + i] = ((t[4 * i + 3] * 16 + t[4 * i + 2]) * 16 + t[4 * i + 1]) * 16 + t[4 * i];
        }
    }
    auto rotate = [](uint32_t c) { return ((c << 3) & 0xFFF8FFF8u) | ((c >> 13) & 0x00070007u); };
    r.codes = make_uint2(rotate(__byte_perm(w[0], w[1], 0x5410)), rotate(__byte_perm(w[2], w[3], 0x5410)));
    return r;
}

template <int MT>
PKV_DEV uint32_t pair_add(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (MT == PKV_F16)
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int MT>
PKV_DEV uint32_t pair_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    if constexpr (MT == PKV_F16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// The values s c + z of eight codes in the model's type, rounded once: a code in bits 3..6 of 128 (fp16) or 16 (bf16),
// where those bits count ones, that number taken off, a fused multiply-add.
template <int MT>
PKV_DEV uint4 int4_values(uint32_t codes, uint32_t params) {
    constexpr uint32_t kBase = MT == PKV_F16 ? 0x58005800u : 0x41804180u, kMinus = kBase | 0x80008000u;
    const uint32_t s = __byte_perm(params, 0, 0x1010), z = __byte_perm(params, 0, 0x3232);
    const uint32_t other = __byte_perm(codes, 0, 0x2301); // nibbles 2 and 3 where 0 and 1 are
    const uint32_t at3[4] = {codes, codes >> 4, other, other >> 4};
    uint32_t v[4]; // elements (i, i + 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair_fma<MT>(pair_add<MT>((at3[i] & 0x00780078u) | kBase, kMinus), s, z);
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                      __byte_perm(v[2], v[3], 0x7632));
}
