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
    uint32_t codes;  // this lane's eight
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

// Eight elements of a row that the `cpr` lanes of `lanes` hold together.
template <int MT>
PKV_DEV Int4Row int4_quantise(const uint4 &src, int cpr, unsigned lanes) {
    using M = ModelT<MT>;
    uint32_t lo = min2_nan<MT>(min2_nan<MT>(src.x, src.y), min2_nan<MT>(src.z, src.w));
    uint32_t hi = max2_nan<MT>(max2_nan<MT>(src.x, src.y), max2_nan<MT>(src.z, src.w));
    for (int o = 1; o < cpr; o <<= 1) {
        lo = min2_nan<MT>(lo, __shfl_xor_sync(lanes, lo, o));
        hi = max2_nan<MT>(hi, __shfl_xor_sync(lanes, hi, o));
    }
    lo = min2_nan<MT>(lo, __byte_perm(lo, lo, 0x1032));
    hi = max2_nan<MT>(hi, __byte_perm(hi, hi, 0x1032));
    const float z = half_of<MT>(lo, 0), range = __fsub_rn(half_of<MT>(hi, 0), z);
    Int4Row r;
    if (!(range < INFINITY)) { // NaN or overflow; an infinity in the row makes the range one or the other
        r.codes = 0;
        r.params = MT == PKV_F16 ? 0x7E007E00u : 0x7FC07FC0u;
        return r;
    }
    const uint32_t s16 = M::pack(__fdiv_rn(range, 15.f), 0.f) & 0xFFFFu;
    float s = half_of<MT>(s16, 0);
    if (s < 1.17549435e-38f) s = 0.f; // 2^-126
    r.params = (s == 0.f ? 0u : s16) | (lo << 16);
    r.codes = 0;
    if (s == 0.f) return r;
    float f[8];
    cvt8<MT>(src, f);
    const float inv = __frcp_rn(s);
    bool near_tie = false;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = __fsub_rn(f[i], z);
        y[i] = __fmul_rn(d, inv);
        const float t = __fsub_rn(__fadd_rn(y[i], 12582912.f), 12582912.f); // rint
        near_tie |= fabsf(y[i] - t) > 0.4999f;
        f[i] = d;
    }
    if (near_tie) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(f[i], s);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) // the low mantissa bits of y + 1.5 * 2^23 are rint(y)
        r.codes |= (__float_as_uint(__fadd_rn(fminf(y[i], 15.f), 12582912.f)) & 15u) << (4 * i);
    r.codes = ((r.codes << 3) & 0xFFF8FFF8u) | ((r.codes >> 13) & 0x00070007u);
    return r;
}

// values of eight codes (exact in fp32 but for the one rounding of the sum)
template <int MT>
PKV_DEV void int4_values(uint32_t codes, uint32_t params, float *f) {
    const float s = half_of<MT>(params, 0), z = half_of<MT>(params, 1);
    codes = ((codes >> 3) & 0x1FFF1FFFu) | ((codes << 13) & 0xE000E000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaf(s, (float)((codes >> (4 * i)) & 15u), z);
}
