// Decode attention over a 4-bit cache, with or without attention mass.
//
// What it computes, for sequence s, query head h of KV head g = h / G, L = context_lens[s]:
//     x_t = scale * q[s][h] . K_t,   p_t = exp(x_t) / sum_u exp(x_u),   out[s][h] = sum_t p_t V_t
// and, where asked, mass[s][g][t] := decay * mass[s][g][t] + sum_{h in group g} p[s][h][t].
// A row stands for K_t = s_t c_t + z_t (c in 0..15, one s and z per row), so
//     q . K_t = s_t (q . c_t) + z_t sum(q),     sum_t p_t V_t = sum_t (p_t s_t) c_t + sum_t p_t z_t:
// the matrix products run on the codes themselves; steps and offsets are two scalars per token outside them.
//
// What bounds it: the bytes of the cache (68 B per row and head at D = 128).  At the measured 6.78 TB/s an
// SM gets 24 B = 47 codes per clock, too many to widen one by one: widening through shared memory for
// tcgen05 operands would write 94 B and read 94 B per clock of its 128, and one fp32 FMA per code would take
// 47 of the 128 lanes on top of the unpacking.  mma.sync takes its operands from registers, so a code
// travels global -> shared (bulk copy) -> register once and is widened there.
//   * Codes as fp16: the stored words (int4.cuh) hold each nibble where an fp16 reads it as c 2^-21 or
//     c 2^-17, so widening is one AND per two codes and a byte exchange per eight: no bias to subtract.  The
//     products take such numbers exactly; their sums keep them to 2^-17 of a code step at the largest q
//     (2^-24 of the exponent that subnormal numbers count as), far below the half step of the codes.  The
//     powers of two go into q (a sixteenth for odd elements), the score and the accumulator.
//   * K tile: A operand (16 tokens x D codes), q^T: B operand (D x 8 heads).  V tile: A operand (16 dims x
//     16 tokens at a time), P^T: B operand (16 tokens x 8 heads).  The order of the summed index is free, so
//     each thread takes whole pieces of a row as they lie, and q is laid out once per unit in the same
//     order.  P goes from the first product's layout to the second's by movmatrix.
//   * The second product takes P as fp16 hi + lo parts (2^-22 relative), so that rounding P does not
//     show: with up to four heads the lo part uses the four columns of B that are free anyway; with eight it
//     takes a second product.  One head alone leaves every other column of its thread's two empty.
//   * Queries are scaled by a power of two per head so that their largest element is in [2^10, 2^11): fp16
//     then holds them (and a sixteenth of them) to 2^-31 of that element or better.
//   * Four warps share a unit's 32-token tiles, each with its own ring of tiles, no barrier between warps inside a
//     unit, and the next unit's first tiles on their way before this one is joined.  Which of the unit's four sums
//     a tile goes to depends on its number and the call's shapes alone, and so do the bits of a row: not on the other
//     sequences.  A tile is one run of the pool per block: one lane per block copies it, completion counted on an
//     mbarrier (bounded waits).  One warp in turn finds the next unit, fetches its table and q and lays q out for
//     all four.
//   * Two references a column.  The weights p stand against m, a running maximum of the scores that moves only when
//     a score passes it by 2^8.  The products p s that go into the second product are multiplied by F, a power of two
//     that puts the largest so far between 2^4 and 2^15: hi + lo hold them to 2^-22 of themselves or 2^-29 of the
//     largest, whatever tokens of great weight and small range, or of great range and no weight, stand among them
//     (F from the largest step alone: one token of e^-20 of the weight and 1024 times the range cost the others
//     1e-2 of the output).  Both move about once a unit (m by 2^4, F from 2^8: 62.7 us for the 61.6 of 256 ragged rows).
//   * Scores, softmax statistics, sums and accumulators are fp32.
//
// Measured: 32 sequences of up to 4096 tokens, 32 heads (7B batch), 268 MB in 59 us, 4.5 TB/s; 256 ragged ones of up to
// 8192, four heads to a KV head, 237 MB in 61 us, 3.9 TB/s; one of 131071 tokens, 143 MB in 37 us; 64 of up to 4096, eight
// heads to a KV head, 40 us.  Under a window (WIN, see Reach): of 1024 tokens and 4 sinks, the first of these 30.2 us (126 MB,
// floor 18.9); of 511 and 1, the second 35.5 (17.2).  Copies alone take 48 us of the first, arithmetic on data in L2 nearly all of it: four warps a
// scheduler, as many as 128 registers allow, hide the two and the dependent chain of a tile behind one another only in part.
#pragma once

#include <type_traits>

#include "mma_common.cuh"

namespace pkv_mma {

template <int D, int GC>
struct Geo4 {
    static constexpr int kOct = 8 * (D + 8);  // 8 tokens' K, V, (s, z), as in the pool
    static constexpr int kTile = 32;          // tokens
    static constexpr int kBytes = 4 * kOct;
    // four CTAs per SM, two tiles of 4 KB a warp on their way: with three CTAs of three the 7B batch below takes 62 us.
    // With eight heads the four warps' accumulators leave shared memory for three, and so 168 registers a thread (64
    // sequences of eight heads a group: 41.1 us; held to 128 registers, which spill, 43.5).
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kCtas = D == 128 && GC == 8 ? 3 : 4;
};

// Nibbles 0..3 of each 16-bit half of w -> four fp16 pairs (low half, high half): c 2^-21 for nibbles 0
// and 2, c 2^-17 for nibbles 1 and 3.  v is w with the bytes of each half exchanged.
PKV_DEV void widen4(uint32_t w, uint32_t v, uint32_t *h) {
    h[0] = w & 0x00780078u;
    h[1] = w & 0x07800780u;
    h[2] = v & 0x00780078u;
    h[3] = v & 0x07800780u;
}

PKV_DEV int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; } // of a positive number
PKV_DEV float power_of_two(int e) { return e < -126 ? 0.f : __uint_as_float((uint32_t)(127 + e) << 23); } // e < 128

// GC: 1 query head per KV head, 4 (two or four), 8
template <int D, int MT, int GC, bool MASS, bool WIN = false>
__global__ void __launch_bounds__(kThreads, Geo4<D, GC>::kCtas) decode_int4_kernel(const Args a) {
    using G_ = Geo4<D, GC>;
    constexpr int KS = D / 16;             // k steps of the first product = m tiles of the second
    constexpr int ST = G_::kStages, T = G_::kTile;
    constexpr int NC = GC == 1 ? 1 : 2;    // columns of a thread that count
    constexpr int COLS = GC, LD = D + 4;
    extern __shared__ __align__(128) char smem[];
    __shared__ Join J;
    __shared__ int sm_tmp[2 * kWarps];
    __shared__ uint64_t sm_bars[kWarps * ST];
    __shared__ UnitOf<WIN> sm_unit[2];
    __shared__ float sm_Q[2][8], sm_SQ[2][8]; // per column: the score's scale, sum(q) times it
    __shared__ int sm_bad[2];
    float *oacc = reinterpret_cast<float *>(smem + kWarps * ST * G_::kBytes); // [warp][COLS][LD]
    uint4 *frags = reinterpret_cast<uint4 *>(oacc + kWarps * COLS * LD);      // two units' q as B operands
    char *qraw = reinterpret_cast<char *>(frags + 2 * KS / 2 * 32);           // q rows as they lie
    const int tb_len = a.split_tokens >> a.bs_log2;
    int *tb = reinterpret_cast<int *>(qraw + COLS * D * 2); // two units' table entries
    int *full = tb + 2 * tb_len;
    int *part = full + a.num_seqs + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int G = a.group, bl = a.bs_log2, bs = 1 << bl;
    char *ring = smem + warp * ST * G_::kBytes;
    const uint32_t ring_u = smem_u32(ring);
    uint64_t *bars = sm_bars + warp * ST;
    uint32_t phase = 0; // of the slot being read, a bit per slot
    bool alive = true;  // false after a wait ran out: nothing more is copied or waited for
    if (lane < ST) mbar_init(&bars[lane], 1);
    fence_mbarrier_init();
    const uint64_t policy = l2_policy_evict_first();
    pdl_wait();
    list_units<WIN>(a, full, part, sm_tmp);
    const int nfull = full[a.num_seqs] * a.hkv, nunits = nfull + part[a.num_seqs] * a.hkv;
    if ((int)blockIdx.x >= nunits) return;

    // Tile `tile` of a unit (its tokens n, its table, its head's place in the pool) to slot `slot`, a lane per block:
    // whole octets (what lies behind the sequence's end is masked later: its codes are numbers, whatever they are).
    const int lane_t = lane << bl;                       // this lane's block's first token in a tile
    const uint32_t lane_bytes = (bs >> 3) * G_::kOct;    // bytes of a block's tile part
    const uint32_t lane_dst = lane * lane_bytes, blk_stride = (uint32_t)a.blk_stride;
    auto issue = [&](int n, const int *table, const char *head, int tile, int slot) {
        const int t = tile * T + lane_t;
        int b = -1;
        if (lane_t < T && t < n) b = table[t >> bl];
        const unsigned copies = __ballot_sync(0xffffffffu, b >= 0);
        if (lane == 0) mbar_arrive_expect_tx(&bars[slot], __popc(copies) * lane_bytes);
        __syncwarp();
        if (b >= 0)
            bulk_g2s_hint(ring + slot * G_::kBytes + lane_dst, head + (uint64_t)(uint32_t)b * blk_stride, lane_bytes,
                          &bars[slot], policy);
    };
    // One warp's work for a unit of buffer `par`: find it and start its copies ...
    auto fetch = [&](int ui, int par) {
        const UnitOf<WIN> v = unit_of<WIN>(a, full, part, nfull, ui);
        if (lane == 0) sm_unit[par] = v;
        stage_unit<D>(a, v, tb + par * tb_len, qraw, lane, 32);
        cp_commit();
    };
    // ... and when they have landed check the table and lay out q in the order of the K codes.
    auto prepare = [&](int par) {
        cp_wait<0>();
        __syncwarp();
        const bool bad = check_table(a, sm_unit[par], tb + par * tb_len, lane, 32);
        if (__any_sync(0xffffffffu, bad) && lane == 0) sm_bad[par] = 1;
        else if (lane == 0) sm_bad[par] = 0;
        const char *q = qraw + (GC == 8 ? g : GC == 1 ? 0 : (g & 3) % G) * D * 2;
        float x[KS][4];
        float mx = 0.f, sum = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) { // word w of the thread's quarter row
            float f[8];
            cvt8<MT>(*reinterpret_cast<const uint4 *>(q + (t4 * (D / 4) + 8 * w) * 2), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[2 * w + ((i & 3) >> 1)][2 * (i & 1) + (i >> 2)] = f[i]; // pairs (i, i + 4), two pairs a step
                mx = fmaxf(mx, fabsf(f[i]));
                sum += f[i];
            }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int e = (int)(__float_as_uint(mx) >> 23); // biased exponent of the head's largest element
        const int sh = (e == 0 || e == 255) ? 0 : min(max(10 - (e - 127), -100), 100);
        const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
        if (t4 == 0) {
            sm_Q[par][g] = a.qk_scale_log2 * __uint_as_float((uint32_t)(127 - sh) << 23) * 2097152.f; // 2^21
            sm_SQ[par][g] = sum * a.qk_scale_log2;
        }
#pragma unroll
        for (int k = 0; k < KS; k += 2) { // odd nibbles (second pairs) a sixteenth
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = i & 1 ? up * 0.0625f : up;
                w[i] = ModelT<PKV_F16>::pack(x[k + (i >> 1)][2 * (i & 1)] * f, x[k + (i >> 1)][2 * (i & 1) + 1] * f);
            }
            frags[(par * (KS / 2) + k / 2) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    };

    int par = 0; // which of the two buffers is this unit's
    if (warp == 0) {
        fetch(blockIdx.x, 0);
        prepare(0);
    }
    __syncthreads();
    UnitOf<WIN> u = sm_unit[0];
    int *table = tb;
    bool bad = sm_bad[0] != 0;
    int turn = 1; // the warp that prepares the next unit
    int slot = 0; // the slot of this warp's next tile
    int nt = 0;   // this warp's tiles of the unit
    // Whose tiles.  Evenly, tile 4 i + warp, where no CTA has two units, and with mass or eight heads (256 ragged
    // sequences with mass 71.9 us, 64 of eight heads 41.8).  Else the warp whose turn it is to prepare gets a tile less: the
    // others take one each before it gets its first, by their place behind it (73.9 and 42.6; but 256 ragged ones without
    // mass 61.1 for 62.1, 8192 rows of up to 500 tokens 80.7 for 83.1).  Also in a CTA's last unit, which prepares nothing:
    // the four sums are kept by that place (role), so that they do not depend on which warp's turn it was.
    const bool even = MASS || GC == 8 || (int64_t)gridDim.x == (int64_t)a.num_seqs * a.hkv * a.max_splits;
    int role = 0;
    int tile0 = 0, first = 0;
    const char *head = nullptr;
    auto tile_of = [&](int i) { return 4 * i + tile0 + (i == 0 ? first : 0); };
    auto start = [&]() {
        const int ntiles = (u.n + T - 1) / T, r = (warp - turn + kWarps - 1) & (kWarps - 1); // 3: this warp's turn
        role = even ? warp : r;
        if (even) {
            nt = max(0, ntiles + 3 - warp) / 4;
            tile0 = warp;
            first = 0;
        } else {
            nt = r == 3 ? max(0, ntiles - 3) / 4 : ntiles <= r ? 0 : 1 + max(0, ntiles - r) / 4;
            tile0 = r == 3 ? 6 : r - 1;
            first = r != 3;
        }
        head = a.pool + u.kvh * a.head_stride;
        if (!alive) return;
        int to = slot;
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            if (i < nt) issue(u.n, table, head, tile_of(i), to);
            to = to == ST - 1 ? 0 : to + 1;
        }
    };
    start();

    Unit prev = u;        // the last unit, if it still has to be counted
    bool pending = false;
    for (int ui = blockIdx.x;;) {
        int before = 0;
        if (!MASS && pending && threadIdx.x == 0) before = count_unit(a, prev);
        const int un = ui + gridDim.x;
        const bool more = un < nunits;
        if (warp == turn && more) fetch(un, par ^ 1);
        uint32_t qf[KS][2];
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
            const uint4 w = frags[(par * (KS / 2) + k / 2) * 32 + lane];
            qf[k][0] = w.x;
            qf[k][1] = w.y;
            qf[k + 1][0] = w.z;
            qf[k + 1][1] = w.w;
        }
        float Q[NC], SQ[NC]; // of columns 2 t4 (and 2 t4 + 1)
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            Q[k] = sm_Q[par][2 * t4 + k];
            SQ[k] = sm_SQ[par][2 * t4 + k];
        }

        // reference maxima; the finite ones to subtract; the scores above which they move
        float m[2] = {-INFINITY, -INFINITY}, mu[2] = {0.f, 0.f}, lim[2] = {-INFINITY, -INFINITY};
        float l[2] = {0.f, 0.f}, z[2] = {0.f, 0.f};
        float F[2] = {1.f, 1.f}, lim_s = 0.f; // of the products; the step above which they may pass 2^15
        float acc[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        // 1 on the lanes whose columns carry the lo parts (up to four heads: columns 4..7)
        const float lo_part = GC != 8 && t4 >= 2 ? 1.f : 0.f;

        for (int i = 0; i < nt; ++i) {
            const bool was_alive = alive;
            if (alive && !mbar_wait(&bars[slot], (phase >> slot) & 1)) {
                set_error(a.err, PKV_DEVERR_TIMEOUT);
                alive = false;
            }
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) {
                if (was_alive) // this warp's copies still on their way: its CTA must not end before them
                    for (int j = 0, at = slot; j < ST && i + j < nt; ++j, at = at == ST - 1 ? 0 : at + 1)
                        mbar_wait(&bars[at], (phase >> at) & 1);
                break;
            }
            phase ^= 1u << slot;
            const uint32_t tile = ring_u + slot * G_::kBytes;
            const uint32_t at_k = tile + g * (D / 2) + t4 * (D / 8), at_p = tile + 8 * D + g * 4;
            const int t0 = tile_of(i) * T;
            const int left = u.n - t0;

            // ---- scores of tokens g, g + 8, g + 16, g + 24 for the thread's columns
            float x[4][NC];
            float vs[4], vz[4]; // V's step and offset
            auto scores = [&](auto half) {
                constexpr int hh = decltype(half)::value;
                constexpr int O0 = 2 * hh * G_::kOct, O1 = O0 + G_::kOct;
                uint32_t ka[D / 32], kb[D / 32];
                if constexpr (D == 128) {
                    lds128<O0>(ka, at_k);
                    lds128<O1>(kb, at_k);
                } else {
                    lds64<O0>(ka, at_k);
                    lds64<O1>(kb, at_k);
                }
                float c[4];
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    uint32_t ha[4], hb[4];
                    widen4(ka[w], __byte_perm(ka[w], 0, 0x2301), ha);
                    widen4(kb[w], __byte_perm(kb[w], 0, 0x2301), hb);
                    if (w == 0)
                        mma_first<PKV_F16>(c, ha[0], hb[0], ha[1], hb[1], qf[2 * w][0], qf[2 * w][1]);
                    else
                        mma<PKV_F16>(c, ha[0], hb[0], ha[1], hb[1], qf[2 * w][0], qf[2 * w][1]);
                    mma<PKV_F16>(c, ha[2], hb[2], ha[3], hb[3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
                }
                const uint32_t kp[2] = {lds32<O0>(at_p), lds32<O1>(at_p)};
                const uint32_t vp[2] = {lds32<O0 + 32>(at_p), lds32<O1 + 32>(at_p)};
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float s = lo_f(kp[r], MT), o = hi_f(kp[r], MT);
#pragma unroll
                    for (int k = 0; k < NC; ++k) x[2 * hh + r][k] = fmaf(c[2 * r + k] * Q[k], s, o * SQ[k]);
                    vs[2 * hh + r] = lo_f(vp[r], MT);
                    vz[2 * hh + r] = hi_f(vp[r], MT);
                }
            };
            scores(std::integral_constant<int, 0>());
            scores(std::integral_constant<int, 1>());
            if (left < T || bad) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (g + 8 * r >= left || (bad && table[(t0 + g + 8 * r) >> bl] < 0)) {
#pragma unroll
                        for (int k = 0; k < NC; ++k) x[r][k] = -INFINITY;
                        vs[r] = vz[r] = 0.f;
                    }
            }
            if constexpr (WIN) { // tokens out of sight among those in it
                const int lo = u.lo - u.t0 - t0, hi = u.hi - u.t0 - t0;
                if (lo < T && hi > 0 && lo < hi) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (g + 8 * r >= lo && g + 8 * r < hi) {
#pragma unroll
                            for (int k = 0; k < NC; ++k) x[r][k] = -INFINITY;
                            vs[r] = vz[r] = 0.f;
                        }
                }
            }
            if constexpr (MASS) {
                float *dst = a.ws_x + (((int64_t)u.s * a.hkv + u.kvh) * a.cap + u.t0 + t0 + g) * G;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (g + 8 * r < left) {
                        if constexpr (GC == 1) {
                            if (t4 == 0) dst[8 * r] = x[r][0];
                        } else if (2 * t4 < G) {
                            *reinterpret_cast<float2 *>(dst + 8 * r * G + 2 * t4) = make_float2(x[r][0], x[r][NC - 1]);
                        }
                    }
            }

            // ---- references: one vote a tile, on its largest scores and its largest step
            float n_[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < NC; ++k) n_[k] = fmaxf(fmaxf(x[0][k], x[1][k]), fmaxf(x[2][k], x[3][k]));
            bool up = fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3])) > lim_s;
#pragma unroll
            for (int k = 0; k < NC; ++k) up = up || n_[k] > lim[k];
            if (__any_sync(0xffffffffu, up)) {
                float most[2] = {0.f, 0.f}; // the tile's largest product
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
                    for (int k = 0; k < NC; ++k) n_[k] = fmaxf(n_[k], __shfl_xor_sync(0xffffffffu, n_[k], o));
                }
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    n_[k] = fmaxf(n_[k], m[k]);
                    mu[k] = n_[k] == -INFINITY ? 0.f : n_[k];
#pragma unroll
                    for (int r = 0; r < 4; ++r) most[k] = fmaxf(most[k], fast_exp2(x[r][k] - mu[k]) * vs[r]);
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
#pragma unroll
                    for (int k = 0; k < NC; ++k) most[k] = fmaxf(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
                }
                float f[2] = {1.f, 1.f}; // of the accumulator
                lim_s = INFINITY;
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float d = m[k] == n_[k] ? 0.f : fminf(n_[k] - m[k], 300.f), whole = floorf(d);
                    const float part = fast_exp2(whole - d), back = part * power_of_two(-(int)whole);
                    l[k] *= back;
                    z[k] *= back;
                    // F against the new m, but for the fraction of the move, and what the tile asks for
                    const int e = exponent(F[k]) + (int)whole, q = exponent(most[k]);
                    int to = min(4 - q, 100);
                    if (m[k] != -INFINITY) {
                        to = e > 100 || e + q >= 15 ? min(to, e) : e;
                        f[k] = part * power_of_two(to - e);
                    }
                    F[k] = power_of_two(to);
                    m[k] = n_[k];
                    lim[k] = m[k] + 8.f;
                    if (m[k] != -INFINITY) lim_s = fminf(lim_s, power_of_two(7 - to)); // of p <= 2^8
                }
                if (i > 0) { // (nothing is summed before the first tile)
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        acc[k][0] *= f[0];
                        acc[k][1] *= f[1];
                        acc[k][2] *= f[0];
                        acc[k][3] *= f[1];
                    }
                }
            }
            // ---- P^T as the second product's B operand: minus the hi parts (columns 0..3) and the lo parts (4..7), or
            // for eight heads hi and lo one after the other.  hi is w cut to 11 bits; the rest, which is exact, is rounded
            // to nearest: cut as well, every weight would be low, and over zero-mean rows the sums of codes and of
            // offsets cancel (131071 tokens: 1.2e-3 of the bf16 output off an fp32 sum, for 5e-4).
            uint32_t b[4], bl_[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float w[2] = {0.f, 0.f};
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    const float p = fast_exp2(x[r][k] - mu[k]);
                    l[k] += p;
                    z[k] = fmaf(p, vz[r], z[k]);
                    w[k] = p * F[k] * vs[r]; // (in this order: F times a step may overflow where p is 0)
                }
                if constexpr (GC == 8) {
                    b[r] = movmatrix(pack_rz<PKV_F16>(w[0], w[1]));
                    bl_[r] = movmatrix(
                        ModelT<PKV_F16>::pack(w[0] - kept_rz<PKV_F16>(w[0]), w[1] - kept_rz<PKV_F16>(w[1])));
                } else {
#pragma unroll
                    for (int k = 0; k < NC; ++k) w[k] = fmaf(w[k], lo_part, -kept_rz<PKV_F16>(w[k]));
                    b[r] = movmatrix(ModelT<PKV_F16>::pack(w[0], w[1]));
                }
            }

            // ---- acc[dims][column] += V^T P^T: rows 2 t4, 2 t4 + 1 of each octet (places t4 and t4 + 4), this
            // thread's D / 8 codes of each
            const uint32_t at_v = D == 128 ? tile + t4 * 64 + ((g * 8) ^ ((t4 & 2) << 4)) : tile + t4 * 32 + g * 4;
            auto outputs = [&](auto half) {
                constexpr int hh = decltype(half)::value;
                constexpr int W = D / 64, O0 = 2 * hh * G_::kOct + 4 * D, O1 = O0 + G_::kOct, P4 = 4 * (D / 2);
                uint32_t v[4][W];
                if constexpr (W == 1) {
                    v[0][0] = lds32<O0>(at_v);
                    v[1][0] = lds32<O0 + P4>(at_v);
                    v[2][0] = lds32<O1>(at_v);
                    v[3][0] = lds32<O1 + P4>(at_v);
                } else {
                    lds64<O0>(v[0], at_v);
                    lds64<O0 + P4>(v[1], at_v);
                    lds64<O1>(v[2], at_v);
                    lds64<O1 + P4>(v[3], at_v);
                }
                uint32_t h[2][D / 8]; // token pairs of the two octets: code pairs by dim
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint32_t x0 = v[2 * r][w], x1 = v[2 * r + 1][w];
                        widen4(__byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x4501), &h[r][8 * w]);
                        widen4(__byte_perm(x0, x1, 0x7632), __byte_perm(x0, x1, 0x6723), &h[r][8 * w + 4]);
                    }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    mma<PKV_F16>(acc[k], h[0][k], h[0][k + KS], h[1][k], h[1][k + KS], b[2 * hh], b[2 * hh + 1]);
                    if constexpr (GC == 8)
                        mma<PKV_F16>(acc[k], h[0][k], h[0][k + KS], h[1][k], h[1][k + KS], bl_[2 * hh], bl_[2 * hh + 1]);
                }
            };
            outputs(std::integral_constant<int, 0>());
            outputs(std::integral_constant<int, 1>());
            __syncwarp(); // every lane has read the slot
            if (i + ST < nt) issue(u.n, table, head, 4 * (i + ST) + tile0, slot);
            slot = slot == ST - 1 ? 0 : slot + 1;
        }

        // ---- the next unit's first tiles, then this unit's join
        if (warp == turn && more) prepare(par ^ 1);
        turn = turn == kWarps - 1 ? 0 : turn + 1;
        if (g == 0) {
#pragma unroll
            for (int k = 0; k < NC; ++k) J.m[role][2 * t4 + k] = m[k];
        }
        if (!MASS && threadIdx.x == 0) J.last = pending && before == prev.nsplit - 1;
        __syncthreads();
        const Unit cur = u;
        const int me = role;
        par ^= 1;
        if (more) {
            u = sm_unit[par];
            bad = sm_bad[par] != 0;
            table = tb + par * tb_len;
            start();
        }
        if constexpr (!MASS) {
            if (J.last) {
                __threadfence();
                join_row<D, MT>(a, prev, J);
            }
        }
        {
            Weight w[NC];
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                w[k] = warp_weight(J, me, 2 * t4 + k);
                l[k] = row_sum(l[k]);
                z[k] = row_sum(z[k]); // (all lanes: the columns' weights differ)
                z[k] = w[k].w == 0.f ? 0.f : z[k] * w[k].w;
                if (g == 0) {
                    J.l[me][2 * t4 + k] = l[k] * w[k].w; // (a NaN comes through a weight of 0)
                    J.z[me][2 * t4 + k] = z[k];
                    if (warp == 0) J.M[2 * t4 + k] = w[k].M;
                }
                w[k].w *= power_of_two(-exponent(F[k]));
            }
            // hi and lo columns together; F and the warp's weight
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (NC == 1 && (e & 1)) continue;
                    float v = acc[k][e];
                    if constexpr (GC != 8) v = __shfl_xor_sync(0xffffffffu, v, 2) - v;
                    acc[k][e] = v * w[e & (NC - 1)].w;
                }
            if (2 * t4 < COLS) { // 16 (or 8) dims from (D / 8) g of each column
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float *o = oacc + (me * COLS + 2 * t4 + c) * LD + (D / 8) * g;
#pragma unroll
                    for (int k = 0; k < KS; k += 4) {
                        *reinterpret_cast<float4 *>(o + k) =
                            make_float4(acc[k][c], acc[k + 1][c], acc[k + 2][c], acc[k + 3][c]);
                        *reinterpret_cast<float4 *>(o + KS + k) =
                            make_float4(acc[k][c + 2], acc[k + 1][c + 2], acc[k + 2][c + 2], acc[k + 3][c + 2]);
                    }
                }
            }
        }
        join_unit<D, COLS, MT, MASS, true>(a, cur, J, oacc);
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

template <int D, int MT, int GC, bool MASS, bool WIN>
cudaError_t launch_int4_t(const Args &a, int sms, cudaStream_t st) {
    using G_ = Geo4<D, GC>;
    static std::atomic<bool> have[64];
    auto kern = decode_int4_kernel<D, MT, GC, MASS, WIN>;
    const size_t smem = (size_t)kWarps * G_::kStages * G_::kBytes + kWarps * GC * (D + 4) * sizeof(float) +
                        2 * (D / 32) * 32 * 16 + GC * D * 2 + (3 * (a.num_seqs + 1) + 2 * (a.split_tokens >> a.bs_log2)) * sizeof(int);
    cudaError_t e = pkv_allow_smem(reinterpret_cast<const void *>(kern), have);
    if (e != cudaSuccess) return e;
    return pdl_launch(kern, dim3(grid_of(a, sms * ctas_of(G_::kCtas, smem))), dim3(kThreads), smem, st, a);
}

template <int MT, bool MASS, bool WIN = false>
cudaError_t dispatch_int4(const Args &a, int D, int sms, bool merge, cudaStream_t st) {
    if (merge) return D == 64 ? launch_merge_t<64, MT, MASS, WIN>(a, sms, st) : launch_merge_t<128, MT, MASS, WIN>(a, sms, st);
#define PKV_INT4_CASE(DD, GC)                                                                                          \
    if (D == DD && (GC == 4 ? a.group == 2 || a.group == 4 : a.group == GC))                                           \
        return launch_int4_t<DD, MT, GC, MASS, WIN>(a, sms, st);
    PKV_INT4_CASE(64, 1)
    PKV_INT4_CASE(64, 4)
    PKV_INT4_CASE(64, 8)
    PKV_INT4_CASE(128, 1)
    PKV_INT4_CASE(128, 4)
    PKV_INT4_CASE(128, 8)
#undef PKV_INT4_CASE
    return cudaErrorNotSupported;
}

} // namespace pkv_mma
