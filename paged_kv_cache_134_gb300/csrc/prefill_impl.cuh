// Causal attention over packed or paged keys on the 5th-generation tensor cores: the packed prefill
// (with the paged K/V write fused in), the prefill over a cached prefix, and the prefix phase of the
// cascade decode.
//
// What it computes ("Paged KV Cache 与 Packed Sequence", discosf.com, sections 3.1-3.3, 4.2):
// sequences packed back to back, sequence i owning rows [cu[i], cu[i+1]); a query at in-sequence
// position r attends to the keys of its own sequence at positions c <= r (block-diagonal causal
// mask), out = softmax(scale q.k) v.  In packed mode every token's k/v is also written into the paged
// cache at block_table[i][r / bs], offset r % bs (the prompt-phase write of section 4.2, bounded by
// the sequence length so a partly filled tail block is never overrun).  In paged mode sequence i
// already holds ctx[i] tokens in its blocks ("PagedAttention 与前缀缓存", 2kiu.com, section 4.3): its
// rows sit at positions ctx[i] + r and every key is read from the pool through the block table.  In
// cascade mode the queries are the decode queries of a batch (one row per sequence) and the keys are
// a prefix shared by every table (section 3.3), cut into splits whose fp32 partials a merge combines.
// In chunk mode (paged_chunk_attention, pieces of prompts) the last n_i of a sequence's L_i cached tokens are its queries, the
// group's query heads of a token lie side by side in a tile's rows (a KV head's keys are read once for all of them), the
// keys may be cut into splits, and a window with sinks may hide keys: see ChunkItem.  512 tokens after 131071, 32/8 heads of
// 128 (1097 GFLOP, 575 us at the measured rate): bf16 1.11 ms (the pair makes 862 us of work; tensor pipe 72 % busy), fp16
// 0.91 (59 %), E4M3 1.04 (49 %; codes go through shared memory twice).  8 prompts of 4096 tokens, 577 us:
// 1.17, 0.92 and 1.06; under a window of 1024, 253 us: 728, 609 and 618.
//
// Design (one persistent CTA per SM, items taken from an atomic counter, heaviest first):
//  * An item is two 128-row query tiles A and B.  Packed and paged modes: consecutive tiles of one
//    (sequence, query head), which share every 128-key K/V tile (loaded once, used by both); cascade
//    mode: one tile of 128 sequences against two consecutive prefix splits (one Q tile, two key streams).
//  * Tensor memory (512 columns): S_A, S_B (128 fp32 columns each) and O_A, O_B (D columns each).  P
//    is written over S in place (fp16, or a bf16 hi + lo pair), and read by P V as the A operand from
//    tensor memory.
//  * Each tile has its own MMA-issuing warp, which issues per key step j: P V(j), then S(j+1).  While
//    one tile's softmax runs, the tensor pipe works on the other tile's products, so each softmax has
//    two MMAs' time (2 x 128 x 128 x D) to finish; S(j+1) of a tile is issued only after its P V(j),
//    which frees the S columns P occupies (tcgen05 operations of one thread complete in issue order).
//    Two issuing warps keep the pipe's queue fed while either waits for its softmax.
//  * Warp roles: 0 scheduler, Q loads and K loads; 2 V loads (each loader also writes the packed
//    mode's paged K/V rows, and widens the E4M3 tiles of FP8 caches); 1 and 3 the MMA issuers of tiles
//    A and B (warp 1 also owns tensor memory); 4-7 softmax of tile A, 8-11 softmax of tile B (one
//    thread per query row, tensor memory lane = row).
//  * O is rescaled in tensor memory only when a row's running maximum grows by more than 2^8 (the
//    exponent base stays fixed otherwise, which is exact algebra); the softmax thread does it, since
//    S(j) complete implies P V(j-1) complete.
//  * Item boundaries: the K loader issues the next item's first K tile, then its Q tiles as their
//    buffers free up; a tile's output (a whole tile of the sequence's rows) is staged in its own Q
//    buffer and written by TMA stores, and the Q buffer returns to the loader once they have read it.
//  * Every mbarrier wait is bounded; a timeout sets PKV_DEVERR_TIMEOUT and the CTA winds down.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "tcgen05.cuh"
#include "pkv_internal.h"

namespace pkv_prefill {

constexpr int BM = 128;          // query rows per tile (MMA M)
constexpr int BN = 128;          // keys per tile (MMA N of Q K^T, K of P V)
constexpr int kThreads = 384;    // 12 warps
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.0f; // log2 units
// Chunks over fp16 and E4M3 caches give their weights to P V as one fp16, as the prefill does over fp16 caches: fp16 outputs
// come to 1.35 times their own rounding (rms; 1.00 where chunk_few.cuh takes the rows, whose weights are pairs), bf16
// outputs to 1.006.  Pairs here: 1.00, and 28 % more time for 512 fp16 tokens after 131071 (894 us, 1145), 23 to 35 % for
// prompts of 4096, 6 to 11 % for tiles of 25 to 128 rows (44 over E4M3).  bf16 caches' weights are pairs: one bf16
// would cost outputs that have 2^-8 as much again.
// Of one fp16 a new base's weight is 2^kChunkUp and the largest 2^14, so that a weight stays a normal
// number down to 2^-20 of the base's and is nothing only below 2^-31.  (With the base at 1 those of 4000 tokens at 2^-25.2 of
// one token's came out as nothing, an output of 1e-4 as 0; over a long split that would be 2^-8 of the sum.)
constexpr float kChunkUp = 14.f - kRescale;
constexpr int kCodeOff = 16384;  // E4M3 codes of a stage: row r at stage + kCodeOff + r * D

enum { MODE_PACKED = 0, MODE_PAGED = 1, MODE_CASCADE = 2, MODE_CHUNK = 3 };

struct Args {
    const char *k, *v;  // packed [T][Hkv][D] (packed mode)
    void *out;          // packed [T][Hq][D]
    const int32_t *cu, *tables;
    char *pool;
    const float *k_scale, *v_scale; // FP8 caches: per KV head
    unsigned int *err;
    int *plan;          // [0] pair count, [1] next-item counter, [4 + 2i], [5 + 2i] = (sequence, pair) of list entry i
    const int32_t *ctx; // paged mode: tokens each sequence already holds in its blocks
    int64_t total_tokens, num_blocks, tile_elems;
    int num_seqs, max_seqlen, max_blocks, hq, hkv, bs, lg_bs, npairs_max, cost_bins;
    int64_t plan_cap;   // list entries the work list has room for
    int write_pool;     // packed mode: write K/V into the pool (16-bit caches; FP8 caches are written by the append)
    float scale_log2;
    // cascade mode: the decode queries of num_seqs sequences against a shared prefix of prefix_tokens
    // tokens (table row 0), cut into nps splits of split_tokens keys; each (sequence, query head, split)
    // leaves an fp32 partial (m, l, unnormalised o) in workspace slot split
    float *ws_o = nullptr, *ws_ml = nullptr;
    int max_splits = 0, prefix_tokens = 0, split_tokens = 0, nps = 0;
    // chunk mode and chunk_stream.cuh: tokens of each sequence, the new ones included; the last `window` keys (0: all) and the first
    // `sinks` are attended to; log2 of the query heads per KV head; key tiles of a split, about.  The window and a
    // call's rows are at most 2^30: a position less the window stays within 32 bits, also that of a row before the first token
    const int32_t *lens = nullptr;
    int window = 0, sinks = 0, lg_group = 0, split_steps = 0;
    int few_rows = 0; // sequences of at most so many rows a KV head are another kernel's (chunk_few.cuh)
    // without a list (plan NULL): row tiles (or pairs) of a sequence and splits (or pairs) of their keys, at most, and
    // sequences x those x KV heads
    int max_groups = 0, max_parts = 0, rect = 0;
};

// TMA descriptors of one launch: q (and out) as [rows][Hq * D] with 64-column boxes of BM rows; packed
// k and v as [T][Hkv * D] with boxes of BN rows; the pool's rows (16-bit: bs rows x 64 dims; E4M3: bs
// whole rows)
struct Maps {
    CUtensorMap q, k, v, pool, out;
};

// Shared memory: two Q tiles, the K ring and the V ring.  A 16-bit tile is [D/64 halves][rows][128 B],
// 128-byte swizzled.  FP8 caches: the codes of a K or V tile land at stage + kCodeOff (row r at r * D)
// and are widened into the 16-bit layout of the same stage: for D = 128 the codes are the upper half
// of the stage, which each row's widening thread reads whole before it writes it; for D = 64 they
// follow the 16 KB tile.
//
// ONE_Q (cascade): one Q tile, and the rings in halves, one per key stream (tile t has stages t, t + 2): a
// stage's barriers then see every phase waited for by one issuer.  (In one ring for both streams, an issuer would come
// back to a stage after two of its phases, and find the one before the other stream's, whose parity is the same,
// complete where its own tile is still on its way.)
template <int D, bool KV8, bool ONE_Q = false>
struct Layout {
    static constexpr int NKS = D == 128 && !ONE_Q ? 3 : 4; // K stages (a K stage frees once S of both tiles is done)
    static constexpr int NVS = D == 128 ? 2 : (ONE_Q ? 4 : 3); // V stages (a V stage frees after P V of both tiles)
    static constexpr int Q_TILE = BM * D * 2;
    static constexpr int TILE = BN * D * 2;
    static constexpr int STAGE = (KV8 && D == 64) ? TILE + BN * D : TILE;
    static constexpr int Q = 0;
    static constexpr int K0 = Q + (ONE_Q ? 1 : 2) * Q_TILE;
    static constexpr int V0 = K0 + NKS * STAGE;
    static constexpr int BAR = V0 + NVS * STAGE;
    static constexpr int NBARS = 4 + 4 + 2 + 2 + 4 * NKS + 4 * NVS + 2 + 2 + 2 + 2 + 2 + 2;
    static constexpr int MISC = BAR + (NBARS * 8 + 15) / 16 * 16; // TMEM slot, abort flag; item slots at + 16
    static constexpr int TOTAL = MISC + 16 + 64;
    static_assert(TOTAL + 1024 <= 232448, "shared memory");
    static_assert(!KV8 || D == 64 || kCodeOff + BN * D <= STAGE, "code region");
};

// two floats -> packed fp16/bf16 pair (round-to-nearest-even), `lo` in the low half
PKV_DEV uint32_t pack2(float lo, float hi, int mt) {
    uint32_t r;
    if (mt == PKV_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// two E4M3 codes (lo in bits 0-7) -> the model dtype's pair; exact (every E4M3 value is an fp16 and
// a bf16 value)
template <int MT>
PKV_DEV uint32_t widen2(uint32_t codes) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<unsigned short>(codes)));
    if constexpr (MT == PKV_F16) {
        return h2;
    } else {
        const float lo = __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xFFFFu)));
        const float hi = __half2float(__ushort_as_half(static_cast<unsigned short>(h2 >> 16)));
        return pack2(lo, hi, PKV_BF16);
    }
}

// Widen row r of an E4M3 tile (D codes at stage + kCodeOff + r * D) into the 128-byte-swizzled
// 16-bit layout of the same stage.  The whole code row is read before anything is written.
template <int D, int MT>
PKV_DEV void widen_row(uint8_t *stage, int r) {
    constexpr int NC = D / 16; // 16-byte chunks of codes
    uint4 c[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) c[i] = *reinterpret_cast<const uint4 *>(stage + kCodeOff + r * D + i * 16);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[2 * e] = widen2<MT>(w[e] & 0xFFFFu);
            o[2 * e + 1] = widen2<MT>(w[e] >> 16);
        }
        // codes 16 i .. 16 i + 15 = dims of two 8-element chunks u0 = 2 i, u0 + 1 (half = dims / 64)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int u = 2 * i + h, c2 = u >> 3, uu = u & 7;
            *reinterpret_cast<uint4 *>(stage + c2 * BN * 128 + r * 128 + ((uu ^ (r & 7)) << 4)) =
                make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
        }
    }
}

// E4M3 caches in chunk mode: four more warps widen the codes, so that the loads of the next tiles are on their way
// meanwhile (a loader that widened its own tiles, one row after another, took 16000 cycles for a pair of tiles that
// HBM brings in 2900).  Codes land in rings of their own, row r at r * D; the 16-bit tiles are fp16 whatever the model's type
// (exact; P then is one fp16 and not a pair), and a bf16 q is brought into fp16's range by a power of two for each
// row, which is left behind the layout for the softmax.
template <int D>
struct CodeLayout {
    static constexpr int NKS = D == 128 ? 2 : 3, NVS = NKS; // fp16 tiles
    static constexpr int NCS = D == 128 ? 1 : 3;            // code stages, of K and of V
    static constexpr int Q_TILE = BM * D * 2;
    static constexpr int TILE = BN * D * 2, STAGE = TILE, CODE = BN * D;
    static constexpr int Q = 0;
    static constexpr int K0 = Q + 2 * Q_TILE;
    static constexpr int V0 = K0 + NKS * STAGE;
    static constexpr int C0 = V0 + NVS * STAGE; // K codes, then V codes
    static constexpr int BAR = C0 + 2 * NCS * CODE;
    static constexpr int NBARS = 4 + 4 + 2 + 2 + 4 * NKS + 4 * NVS + 2 + 2 + 2 + 2 + 2 + 2 + 2;
    static constexpr int MISC = BAR + (NBARS * 8 + 15) / 16 * 16;
    static constexpr int TOTAL = MISC + 16 + 64;
    static_assert(NCS <= NKS && NCS <= NVS, "their barriers share the arrays");
};
template <int D, int MODE, bool KV8>
using LayoutOf = std::conditional_t<KV8 && MODE == MODE_CHUNK, CodeLayout<D>, Layout<D, KV8, MODE == MODE_CASCADE>>;
template <int D, int MODE, bool KV8>
constexpr int smem_total() {
    constexpr int n = LayoutOf<D, MODE, KV8>::TOTAL + (MODE == MODE_CHUNK && KV8 ? 4 * BM : 0);
    static_assert(n + 1024 <= 232448, "shared memory");
    return n;
}
template <int MODE, bool KV8>
constexpr int threads_of() {
    return KV8 && MODE == MODE_CHUNK ? kThreads + 128 : kThreads;
}

// row r of a tile of E4M3 codes -> fp16 in the 128-byte-swizzled layout (lanes take the row's sixteens in turn, so that
// neither the reads nor the writes of eight lanes meet in a bank)
template <int D>
PKV_DEV void widen_codes(const uint8_t *codes, uint8_t *tile, int r) {
    constexpr int NC = D / 16;
#pragma unroll 1 // (unrolled by four 8 % slower: the roles' code together outgrows the instruction cache)
    for (int i = 0; i < NC; ++i) {
        const int c = (i + r) & (NC - 1);
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + r * D + c * 16);
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[2 * e] = widen2<PKV_F16>(in[e] & 0xFFFFu);
            o[2 * e + 1] = widen2<PKV_F16>(in[e] >> 16);
        }
        uint8_t *row = tile + (c >> 2) * (BN * 128) + r * 128;
        const int u = 2 * (c & 3);
        *reinterpret_cast<uint4 *>(row + ((u ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(row + (((u + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// row r of a bf16 Q tile (128-byte swizzled) -> fp16 in place, times 2^-e; returns e.  The row's largest element comes to
// [2^14, 2^15); one that is smaller by 2^31 or more loses bits.
template <int D>
PKV_DEV int q_to_f16(uint8_t *tile, int r) {
    uint8_t *row = tile + r * 128;
    uint32_t top = 0;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const uint4 x = *reinterpret_cast<const uint4 *>(row + (i >> 3) * (BM * 128) + (((i & 7) ^ (r & 7)) << 4));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFF0000u, (w[e] << 16) & 0x7FFF0000u));
    }
    const int e = top == 0 ? 0 : max((int)(top >> 23) - 127, -100) - 14;
    const float f = __uint_as_float((uint32_t)(127 - e) << 23); // 2^-e, -114 <= -e <= 114
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        uint4 *at = reinterpret_cast<uint4 *>(row + (i >> 3) * (BM * 128) + (((i & 7) ^ (r & 7)) << 4));
        const uint4 x = *at;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = pack2(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f, PKV_F16);
        *at = make_uint4(o[0], o[1], o[2], o[3]);
    }
    return e;
}

// query tiles of sequence i (0 for a malformed cu_seqlens entry or context length, which is reported)
PKV_DEV int seq_tiles(const Args &a, int i, bool report) {
    const int st = a.cu[i], en = a.cu[i + 1];
    if (st < 0 || en < st || en > a.total_tokens || en - st > a.max_seqlen) {
        if (report) set_error(a.err, PKV_DEVERR_CU_SEQLENS);
        return 0;
    }
    if (a.ctx) {
        // paged mode: the cached tokens plus the new ones must fit the sequence's table
        const int64_t c0 = a.ctx[i];
        if (c0 < 0 || c0 + (en - st) > (int64_t)a.max_blocks * a.bs) {
            if (report) set_error(a.err, PKV_DEVERR_LENGTH);
            return 0;
        }
    }
    return (en - st + BM - 1) / BM;
}

// one tile of an item as the roles see it
struct Tile {
    int n;     // key tiles (0: the tile is absent)
    int q0;    // first query row of the tile (in-sequence row; cascade: 0)
    int qlast; // last valid query row
    int qpos0; // absolute position of the tile's row 0 (causal mask)
    int k0;    // absolute position of the first key
    int kend;  // keys at or past kend hold no token of the sequence (or of the prefix split)
};

struct Item {
    int seq, pr, h; // seq < 0: no more items.  Cascade: seq = tile of 128 sequences, pr = split pair
    int start;      // packed row of the sequence's first token (cascade: first sequence of the tile)
    int n;          // rows of the sequence (cascade: sequences in the tile)
    int trow;       // block-table row of the keys
    Tile t[2];
};

PKV_DEV Item decode_item(const Args &a, int seq, int pr, int h) {
    Item it;
    it.seq = seq;
    it.pr = pr;
    it.h = h;
    if (seq < 0) return it;
    if (a.nps > 0) {
        it.start = seq * BM;
        it.n = min(BM, a.num_seqs - it.start);
        it.trow = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int sp = 2 * pr + t;
            Tile &x = it.t[t];
            x.q0 = 0;
            x.qlast = it.n - 1;
            x.qpos0 = 0;
            x.k0 = sp * a.split_tokens;
            x.kend = min(x.k0 + a.split_tokens, a.prefix_tokens);
            x.n = sp < a.nps ? (x.kend - x.k0 + BN - 1) / BN : 0;
        }
        return it;
    }
    it.start = a.cu[seq];
    it.n = a.cu[seq + 1] - it.start;
    it.trow = seq;
    const int c0 = a.ctx ? a.ctx[seq] : 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        Tile &x = it.t[t];
        x.q0 = (2 * pr + t) * BM;
        x.qlast = min(x.q0 + BM, it.n) - 1;
        x.qpos0 = c0 + x.q0;
        x.k0 = 0;
        x.kend = c0 + it.n;
        x.n = x.q0 < it.n ? (c0 + x.qlast) / BN + 1 : 0; // key tiles up to the tile's last row
    }
    return it;
}

// Chunk mode: two row tiles A and B of one (sequence, KV head) over the same keys, one split of them.  Row r of a tile is token q0 + r / G, query head h G + r % G.  Keys are counted in "seen" order: the blocks
// that a row of the item can see, one after the other, as if nothing lay between (seen block i is logical block i, or
// i + skip from block `from` on).  Of them [lo, hi) are hidden from every row (the rest of the sinks' last block, and what
// lies before the first row's window); what else a row does not see is masked.
// How the keys are cut depends on the sequence's own lengths and the call's sizes, not on the other sequences.
struct ChunkItem : Item {
    int from, skip, lo, hi;
    int split;
    int ns[2];  // splits of each tile's keys (1: the tile's rows are final)
    bool zero;  // rows without keys: written as zeros by the first split's item
};

// key tiles of a split, of n in all: splits of equal size
PKV_DEV int steps_per_split(const Args &a, int n) {
    const int k = (n + a.split_steps - 1) / a.split_steps;
    return k > 1 ? (n + k - 1) / k : max(n, 1);
}

// What the window hides from every row from position p0 on, of a chunk: seen block i is logical block i, or i + skip from
// block `from` on, and of the seen keys [lo, hi) are hidden.
struct Hidden {
    int from, skip, lo, hi;
};
PKV_DEV Hidden hidden_from(const Args &a, int p0) {
    const int low = a.window > 0 ? max(p0 - a.window + 1, 0) : 0; // first key of the first row's window
    if (low <= a.sinks) return {0, 0, 0, 0};
    const int from = (a.sinks + a.bs - 1) >> a.lg_bs, skip = max((low >> a.lg_bs) - from, 0);
    return {from, skip, a.sinks, low - (skip << a.lg_bs)};
}

PKV_DEV ChunkItem chunk_item(const Args &a, int seq, int pr, int split, int h) {
    ChunkItem it;
    it.seq = seq;
    it.pr = pr;
    it.h = h;
    it.split = split;
    if (seq < 0) return it;
    const int per_tile = BM >> a.lg_group; // tokens
    it.start = a.cu[seq];
    it.n = a.cu[seq + 1] - it.start;
    it.trow = seq;
    const int before = max(a.lens[seq], 0) - it.n; // position of the first new token (negative: those rows see nothing)
    const int tok0 = 2 * pr * per_tile;
    const Hidden hid = hidden_from(a, before + tok0);
    it.from = hid.from;
    it.skip = hid.skip;
    it.lo = hid.lo;
    it.hi = hid.hi;
    int end[2], n[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        Tile &x = it.t[t];
        x.q0 = tok0 + t * per_tile;
        x.qlast = min(x.q0 + per_tile, it.n) - 1;
        x.qpos0 = before + x.q0;
        end[t] = x.q0 < it.n ? max(before + x.qlast + 1 - (it.skip << a.lg_bs), 0) : 0;
        n[t] = (end[t] + BN - 1) / BN;
    }
    const int per = steps_per_split(a, max(n[0], n[1]));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        Tile &x = it.t[t];
        x.k0 = split * per * BN;
        x.n = min(max(n[t] - split * per, 0), per);
        x.kend = min(max(end[0], end[1]), x.k0 + per * BN); // (one end for both tiles, whose loads they share)
        it.ns[t] = (n[t] + per - 1) / per;
    }
    it.zero = split == 0;
    return it;
}

// row tiles of sequence i, or (PAIRS) pairs of them; 0 where its numbers make no sense
template <bool PAIRS>
PKV_DEV int chunk_groups(const Args &a, int i, bool report) {
    const int st = a.cu[i], en = a.cu[i + 1];
    if (st < 0 || en < st || en > a.total_tokens || en - st > a.max_seqlen) {
        if (report) set_error(a.err, PKV_DEVERR_CU_SEQLENS);
        return 0;
    }
    if (en > st && (int64_t)a.lens[i] > (int64_t)a.max_blocks * a.bs) {
        if (report) set_error(a.err, PKV_DEVERR_LENGTH);
        return 0;
    }
    if (en - st <= a.few_rows >> a.lg_group) return 0;
    const int per = (PAIRS ? 2 : 1) * (BM >> a.lg_group);
    return (en - st + per - 1) / per;
}
// items of a group: at least the one that writes the rows without keys
PKV_DEV int chunk_parts(const ChunkItem &it) { return max(1, max(it.ns[0], it.ns[1])); }
// the next item of this CTA among all that the call's sizes allow, from `at` on: (sequence, group, KV head, part), -1 behind
// the last
PKV_DEV int4 direct_item(const Args &a, int &at) {
    for (; at < a.rect; at += gridDim.x) {
        const int h = at % a.hkv, r = at / a.hkv, part = r % a.max_parts, g = r / a.max_parts % a.max_groups;
        const int seq = r / a.max_parts / a.max_groups;
        if (g >= chunk_groups<true>(a, seq, h == 0 && part == 0 && g == 0)) continue;
        if (part > 0 && part >= chunk_parts(chunk_item(a, seq, g, 0, 0))) continue;
        at += gridDim.x;
        return make_int4(seq, g, h, part);
    }
    return make_int4(-1, 0, 0, 0);
}

// Loads of K (or V) tiles of an item, in their order.  Packed, paged and chunk modes share one key tile per step; cascade
// mode has one per tile and step.
template <bool SHARED>
PKV_DEV int ring_count(const Item &it) {
    return SHARED ? max(it.t[0].n, it.t[1].n) : it.t[0].n + it.t[1].n;
}
// the tile (0 or 1) that ring entry e of the item belongs to, and its key step
template <bool SHARED>
PKV_DEV void ring_entry(const Item &it, int e, int &t, int &j) {
    if constexpr (SHARED) {
        t = 0;
        j = e;
    } else {
        const int mn = min(it.t[0].n, it.t[1].n);
        if (e < 2 * mn) {
            t = e & 1;
            j = e >> 1;
        } else {
            t = it.t[0].n > mn ? 0 : 1;
            j = mn + (e - 2 * mn);
        }
    }
}

// bits 0 .. n - 1
PKV_DEV uint32_t ones_below(int n) { return n >= 32 ? 0xFFFFFFFFu : n > 0 ? (1u << n) - 1u : 0u; }

PKV_DEV int chunk_splits(const ChunkItem &it, int t) { return t ? it.ns[1] : it.ns[0]; }
PKV_DEV int chunk_splits(const Item &, int) { return 1; }

template <int D, int MT, int MODE, bool KV8>
__global__ void __launch_bounds__(threads_of<MODE, KV8>(), 1) attn_kernel(const __grid_constant__ Maps maps, const Args a) {
    const CUtensorMap &tq = maps.q, &tk = maps.k, &tv = maps.v, &tp = maps.pool, &to = maps.out;
    using L = LayoutOf<D, MODE, KV8>;
    constexpr bool PAGED = MODE != MODE_PACKED;    // keys from the pool through the block table
    constexpr bool CASCADE = MODE == MODE_CASCADE; // no causal mask, fp32 split partials out
    constexpr bool CHUNKED = MODE == MODE_CHUNK;
    constexpr bool ONE_Q = CASCADE;                // one Q tile, two key streams
    constexpr bool SHARED = !ONE_Q;                // both tiles use the same key tiles
    // K and V tiles of chunk mode at D = 128, 16-bit caches: one box a block brings both halves of its rows, as
    // [8 rows][half][8 rows][128 bytes]; else one box for each half, as [half][128 rows][128 bytes].  (A loader's warp needs
    // some 100 cycles for each box; with two a block, short chunks were bound by their loaders.)
    constexpr bool GROUPED = CHUNKED && D == 128 && !KV8;
    using It = std::conditional_t<CHUNKED, ChunkItem, Item>;
    constexpr bool WRITER = MODE == MODE_PACKED;   // the loaders write the item's K/V rows into the pool
    constexpr bool CODES = KV8 && CHUNKED;         // widened by warps of their own (CodeLayout)
    constexpr int OT = CODES ? (int)PKV_F16 : MT;  // the products' operands
    constexpr int NP = OT == PKV_BF16 ? 2 : 1;     // P parts (bf16: hi + lo)
    constexpr float kUp = CHUNKED && OT == PKV_F16 ? kChunkUp : 0.f;
    constexpr int EB = KV8 ? 1 : 2;                // pool bytes per element
    constexpr int NKS = L::NKS, NVS = L::NVS;
    extern __shared__ __align__(1024) uint8_t smem[];

    if (!CHUNKED || a.few_rows == 0) pdl_trigger();
    if (smem_u32(smem) & 1023u) return; // the swizzled tiles need 1024-byte alignment (always true)

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::BAR);
    // items go through a 4-slot ring: the scheduler publishes an item while the one before it is
    // still being loaded, so that nobody waits for the next item at an item boundary
    constexpr int kItemSlots = 4;
    uint64_t *item_full = bars, *item_empty = bars + kItemSlots;
    uint64_t *q_full = bars + 2 * kItemSlots, *q_empty = q_full + 2;
    uint64_t *k_full = q_empty + 2, *k_empty = k_full + NKS, *kc_full = k_empty + NKS, *k_spare = kc_full + NKS;
    uint64_t *v_full = k_spare + NKS, *v_empty = v_full + NVS, *vc_full = v_empty + NVS, *v_spare = vc_full + NVS;
    uint64_t *s_full = v_spare + NVS, *p_full = s_full + 2, *o_full = p_full + 2, *o_free = o_full + 2;
    uint64_t *fin = o_free + 2;
    uint64_t *epi = fin + 2; // a tile's output rows are staged (one arrival per softmax warp)
    uint64_t *qc_full = epi + 2; // CODES: a Q tile as fp16
    uint64_t *q_ready = CODES && MT == PKV_BF16 ? qc_full : q_full;
    int8_t *q_exp = reinterpret_cast<int8_t *>(smem + L::TOTAL); // CODES: [2 Q tiles][2 tiles][BM] exponents of q's rows
    (void)qc_full;
    (void)q_exp;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::MISC + 4);
    // exp phases the softmax of each tile has finished, counted per warp (4 per key step), monotonic
    int *sm_prog = reinterpret_cast<int *>(smem + L::MISC + 8); // [2]
    volatile int4 *item_slot = reinterpret_cast<volatile int4 *>(smem + L::MISC + 16); // [kItemSlots]
    (void)k_spare;
    (void)v_spare;
    // K / V tiles ready for the MMA: landed (16-bit) or landed and widened (E4M3)
    uint64_t *k_ready = KV8 ? kc_full : k_full;
    uint64_t *v_ready = KV8 ? vc_full : v_full;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // item consumers: V loader, the two MMA issuers, eight softmax warps (and four that widen)
    constexpr int kItemConsumers = CODES ? 15 : 11;
    // a K or V stage frees once every MMA warp whose tile reads it has released it (both tiles read
    // the shared key tiles of packed and paged modes; each cascade tile has key tiles of its own)
    constexpr int kStageReleasers = SHARED ? 2 : 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(item_full + s, 1);
            mbar_init(item_empty + s, kItemConsumers);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(q_full + s, 1);
            mbar_init(q_empty + s, ONE_Q ? 2 : 1); // cascade: one Q tile, read by both MMA warps
            mbar_init(s_full + s, 1);
            mbar_init(p_full + s, 4); // one arrival per softmax warp
            mbar_init(o_full + s, 1);
            mbar_init(o_free + s, 4);
        }
        for (int s = 0; s < NKS; ++s) {
            mbar_init(k_full + s, 1);
            mbar_init(k_empty + s, kStageReleasers);
            mbar_init(kc_full + s, CODES ? 4 : 1);
            if constexpr (CODES) mbar_init(k_spare + s, 4); // codes read (one arrival per warp that widens)
        }
        for (int s = 0; s < NVS; ++s) {
            mbar_init(v_full + s, 1);
            mbar_init(v_empty + s, kStageReleasers);
            mbar_init(vc_full + s, CODES ? 4 : 1);
            if constexpr (CODES) mbar_init(v_spare + s, 4);
        }
        if constexpr (CODES) {
            mbar_init(qc_full, 4);
            mbar_init(qc_full + 1, 4);
        }
        mbar_init(fin, 1);
        mbar_init(fin + 1, 1);
        mbar_init(epi, 4);
        mbar_init(epi + 1, 4);
        *abort_flag = 0;
        sm_prog[0] = 0;
        sm_prog[1] = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // everything above is private to this CTA; from here on global memory written by the previous
    // kernels on the stream (the work list, the inputs) is read.  Cascade mode runs right after the
    // suffix decode, which lets it launch once the decode itself has waited for its predecessors (the
    // plan of this call and everything before it): the prefix phase reads nothing the decode writes,
    // so it starts at once and fills the SMs the decode's CTAs leave, and waits for the decode only
    // before it exits (the merge after it then sees both).
    if constexpr (!CASCADE) pdl_wait();
    if (CHUNKED && a.few_rows > 0) pdl_trigger(); // (few_kernel reads what the list's launch, too, had waited for)

    const int G = a.hq / a.hkv;
    auto make_item = [&](int seq, int pr, int h, int split) -> It {
        (void)split;
        if constexpr (CHUNKED)
            return chunk_item(a, seq, pr, split, h);
        else
            return decode_item(a, seq, pr, h);
    };
    auto kv_head = [&](const It &it) -> int { return CHUNKED ? it.h : it.h / G; };
    auto fail = [&]() {
        set_error(a.err, PKV_DEVERR_TIMEOUT);
        *abort_flag = 1;
    };
    // the item in ring slot n % 4, once the scheduler has published it
    auto take_item = [&](int n, bool &ok) -> It {
        const int sl = n & (kItemSlots - 1);
        ok = mbar_wait_hint(item_full + sl, (n / kItemSlots) & 1);
        if (!ok) return make_item(-1, 0, 0, 0);
        return make_item(item_slot[sl].x, item_slot[sl].y, item_slot[sl].z, CHUNKED ? item_slot[sl].w : 0);
    };
    // the item's keys of ring entry e: key step j of tile t (packed / paged: one tile serves both)
    // (tiles are selected, not indexed, so that the item stays in registers)
    auto key_base = [&](const It &it, int e, int &t, int &j) -> int {
        ring_entry<SHARED>(it, e, t, j);
        return (t ? it.t[1].k0 : it.t[0].k0) + j * BN;
    };
    auto key_end = [&](const It &it, int t) -> int {
        return (SHARED || t == 0) ? it.t[0].kend : it.t[1].kend;
    };

    if constexpr (CODES) { // 128 x (80 + 2 x 176 + 80) = 512 x 128 registers
        if (warp < 4 || warp >= 12) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    } else {
        if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    }
    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------------- loaders
        // Warp 0: the scheduler (lane 0), Q loads and K loads; warp 2: V loads.  Packed mode: lane 0
        // loads each tile (one box per half of D).  Paged and cascade modes: lane l loads block l of
        // each tile; blocks full of the keys' tokens arrive as TMA boxes, and every other row of a V
        // tile is written with plain stores: the tokens of a partly filled last block copied from the
        // pool, zeros for slots past the keys' end and for unusable block ids (P is 0 on those rows,
        // but 0 * NaN is NaN, and the pool's unused slots may hold anything); K rows past the end are
        // masked by the softmax instead.  FP8 caches: the codes land in the stage's code region, and
        // the loader widens each tile once it has landed, before it issues the next one.  Packed mode:
        // the paged write of an item's own rows (the keys of its last tiles) leaves a stage just before
        // the loader refills it (whole blocks as tiled TMA stores, one lane per block and half of D;
        // the rows of a partly filled last block as plain 16-byte stores, so no slot past the sequence
        // is touched), or at the end.
        const bool isK = warp == 0;
        int ns = isK ? NKS : NVS, stage_bytes = L::STAGE, code_off = kCodeOff;
        uint8_t *ring = smem + (isK ? L::K0 : L::V0);
        uint64_t *const full = isK ? k_full : v_full;
        uint64_t *empty = isK ? k_empty : v_empty;
        if constexpr (CODES) { // codes, in their own stages
            ns = L::NCS;
            stage_bytes = L::CODE;
            code_off = 0;
            ring = smem + L::C0 + (isK ? 0 : L::NCS * L::CODE);
            empty = isK ? k_spare : v_spare;
        }
        uint64_t *const ready = isK ? kc_full : vc_full; // E4M3: widened
        const int kvsel = isK ? 0 : 1;                   // K or V half of a pool block
        constexpr int CPR = D * EB / 16;                  // 16-byte chunks per pool row
        constexpr int RPI = 32 / CPR;                     // rows per warp instruction (never two blocks: bs >= 8)
        const int cc = lane % CPR, rsub = lane / CPR;
        if (lane == 0) {
            if (isK) tc::prefetch_tmap(&tq);
            tc::prefetch_tmap(PAGED ? &tp : (isK ? &tk : &tv));
        }
        // packed mode: the pending pool write of the entry each stage holds (j < 0: none), with the
        // item's rows and (lane l) the table entry of its logical block lb0 + l
        int wj[4] = {-1, -1, -1, -1}, wq0[4] = {}, wql[4] = {}, wkvh[4] = {}, wblk[4] = {}, wpar[4] = {};
        auto flush_write = [&](int st) {
            if constexpr (WRITER) {
                if (wj[st] < 0) return;
                const uint8_t *src = ring + st * L::STAGE;
                // the tile has landed long ago (it was loaded ns entries back); the wait is for the
                // rare case the loader is about to refill a stage whose tile still flies
                mbar_wait_hint(full + st, (uint32_t)wpar[st]);
                const int j = wj[st], q0 = wq0[st], qlast = wql[st], kvh = wkvh[st], blkv = wblk[st];
                const int lb0 = q0 >> a.lg_bs;
                const int lo = max(j * BN, q0), hi = min(j * BN + BN - 1, qlast);
                if (lo <= hi) {
                    const int bfirst = lo >> a.lg_bs;           // lo is a multiple of bs
                    const int nfull = (hi + 1 - lo) >> a.lg_bs; // whole blocks among the rows
                    {
                        const int lb = bfirst + lane;
                        const int blk = __shfl_sync(0xffffffffu, blkv, min(lb - lb0, 31));
                        if (lane < nfull) {
                            if (blk < 0 || blk >= a.num_blocks) {
                                set_error(a.err, PKV_DEVERR_BLOCK_ID);
                            } else {
                                const uint8_t *box = src + ((lb << a.lg_bs) - j * BN) * 128;
                                const int y = ((blk * 2 + kvsel) * a.hkv + kvh) << a.lg_bs;
#pragma unroll
                                for (int c = 0; c < D / 64; ++c) tc::tma_store_2d(&tp, c * 64, y, box + c * BN * 128);
                                tc::bulk_commit();
                            }
                        }
                    }
                    const int c2 = cc >> 3, u = cc & 7;
                    for (int p0 = lo + (nfull << a.lg_bs); p0 <= hi; p0 += RPI) { // fewer than bs rows
                        const int pp = p0 + rsub;
                        const int lb = pp >> a.lg_bs;
                        const int blk = __shfl_sync(0xffffffffu, blkv, min(lb - lb0, 31));
                        if (pp > hi) continue;
                        if (blk < 0 || blk >= a.num_blocks) {
                            if (cc == 0) set_error(a.err, PKV_DEVERR_BLOCK_ID);
                            continue;
                        }
                        const int rr = pp - j * BN;
                        const uint4 xv = *reinterpret_cast<const uint4 *>(src + c2 * BN * 128 + rr * 128 +
                                                                          ((u ^ (rr & 7)) << 4));
                        const int64_t dst = ((int64_t)(blk * 2 + kvsel) * a.hkv + kvh) * a.tile_elems +
                                            (int64_t)(pp - (lb << a.lg_bs)) * D + cc * 8;
                        *reinterpret_cast<uint4 *>(a.pool + dst * 2) = xv;
                    }
                }
                tc::bulk_wait_read_all(); // the stores have read the stage; it may be refilled
                __syncwarp();
                wj[st] = -1;
            }
        };
        // The stage of the next load of tile t, and how often it was filled before: stages taken in turn, by all loads or
        // (ONE_Q) by those of each key stream; `g` counts all loads issued, `gt` those of each stream.
        int64_t g = 0;
        int gt[2] = {0, 0};
        auto next_stage = [&](int t, int &st, int &round) {
            if constexpr (ONE_Q) {
                const int c = t ? gt[1] : gt[0];
                st = t + 2 * (c % (ns / 2));
                round = c / (ns / 2);
            } else {
                st = (int)(g % ns);
                round = (int)(g / ns);
            }
        };
        // FP8: widen the tile in stage st (landed), then release it to the MMAs
        auto widen = [&](int st, uint32_t parity) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait_hint(full + st, parity))) return false;
            uint8_t *stage = ring + st * L::STAGE;
            for (int r = lane; r < BN; r += 32) widen_row<D, MT>(stage, r);
            fence_proxy_async_smem(); // the MMAs read the widened tile through the async proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(ready + st);
            return true;
        };
        const bool direct = CHUNKED && a.plan == nullptr; // few items: no list, every CTA looks for its own
        const int total = direct ? a.rect : a.plan[0] * (CHUNKED ? a.hkv : a.hq);
        int next_direct = blockIdx.x;
        (void)next_direct;
        int nq[2] = {0, 0}; // Q loads per buffer so far (warp 0)
        int pend = -1;      // FP8: the issued tile still to widen: its stage, and its phase's parity in bit 8
        // FP8: widen the pending tile; done before this warp can block on anything an MMA of that tile
        // may be holding up (the next tile's stage, the next item, the next item's Q buffer)
        auto widen_pending = [&]() -> bool {
            if constexpr (KV8 && !CODES) {
                if (pend >= 0) {
                    const bool w = widen(pend & 0xFF, (uint32_t)pend >> 8);
                    pend = -1;
                    return w;
                }
            }
            return true;
        };
        bool ok = true;
        // the scheduler (warp 0): take item m from the work list and publish it in ring slot m % 4
        auto publish = [&](int m, bool &pok) -> It {
            const int sl = m & (kItemSlots - 1);
            pok = true;
            if (m >= kItemSlots) pok = __all_sync(0xffffffffu, mbar_wait_hint(item_empty + sl, ((m / kItemSlots) - 1) & 1));
            int4 raw = make_int4(-1, 0, 0, 0);
            if (!pok) return make_item(-1, 0, 0, 0);
            if (lane == 0) {
                int idx = total;
                if (direct) {
                    if constexpr (CHUNKED) {
                        if (!*abort_flag) raw = direct_item(a, next_direct);
                    }
                } else if (!*abort_flag) {
                    idx = atomicAdd(a.plan + 1, 1);
                }
                if (idx < total) {
                    if constexpr (CASCADE) {
                        const int pair = idx / a.hq; // (tile of sequences, split pair)
                        const int npr = (a.nps + 1) / 2;
                        raw = make_int4(pair / npr, pair % npr, idx % a.hq, 0);
                    } else if constexpr (CHUNKED) {
                        const int4 e = reinterpret_cast<const int4 *>(a.plan + 4)[idx / a.hkv];
                        raw = make_int4(e.x, e.y, idx % a.hkv, e.z);
                    } else {
                        const int2 sq = reinterpret_cast<const int2 *>(a.plan + 4)[idx / a.hq];
                        raw = make_int4(sq.x, sq.y, idx % a.hq, 0);
                    }
                }
                item_slot[sl].x = raw.x;
                item_slot[sl].y = raw.y;
                item_slot[sl].z = raw.z;
                if constexpr (CHUNKED) item_slot[sl].w = raw.w;
                mbar_arrive(item_full + sl);
            }
            raw.x = __shfl_sync(0xffffffffu, raw.x, 0);
            raw.y = __shfl_sync(0xffffffffu, raw.y, 0);
            raw.z = __shfl_sync(0xffffffffu, raw.z, 0);
            if constexpr (CHUNKED) raw.w = __shfl_sync(0xffffffffu, raw.w, 0);
            return make_item(raw.x, raw.y, raw.z, raw.w);
        };
        for (int n = 0; ok; ++n) {
            It it;
            if (!isK && !widen_pending()) ok = false; // before waiting for the next item
            if (!ok) break;
            if (isK) {
                // ---- scheduler: take the next item and publish it (once the previous item's last K
                // tile is issued, a few key steps before that item ends)
                it = publish(n, ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (n > 0 && it.seq >= 0 && lane == 0) {
                    // the item's Q tiles load only once the previous item's last S of each tile is done:
                    // staged in L2 now, they then arrive from L2
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (ONE_Q ? b == 1 : it.t[b].n == 0) continue;
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            if constexpr (CHUNKED)
                                tc::tma_prefetch_3d(&tq, c * 64, it.h * G, it.start + it.t[b].q0);
                            else
                                tc::tma_prefetch_2d(&tq, it.h * D + c * 64, it.start + it.t[b].q0);
                        }
                    }
                }
            } else {
                it = take_item(n, ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            if (it.seq < 0) break;
            const int kvh = kv_head(it);
            if (isK && !widen_pending()) ok = false; // before the Q loads wait for their buffers
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            // ---- Q (warp 0): buffer b holds tile b (cascade: buffer 0 holds the one query tile of both
            // splits).  Each load waits for the previous item's last S of that tile, so the loads are
            // interleaved with the K tiles in the order their buffers free up: K tile 0 (its stage frees
            // a few key steps before the previous item ends), Q_A, K tile 1, Q_B, the rest.  The first S
            // of each tile then finds both operands in place.
            // query row of each buffer's tile, -1: nothing to load
            const int qrow0 = it.t[0].n > 0 ? it.start + it.t[0].q0 : -1;
            const int qrow1 = !ONE_Q && it.t[1].n > 0 ? it.start + it.t[1].q0 : -1;
            const int qcol = it.h * D;
            int qnext = 0; // next Q buffer to load
            auto issue_q = [&](int upto) {
                for (; qnext <= upto && qnext < 2 && ok; ++qnext) {
                    const int b = qnext;
                    const int row = b ? qrow1 : qrow0;
                    if (row < 0) continue;
                    if (lane == 0) {
                        const bool w = nq[b] < 1 || mbar_wait_hint(q_empty + b, (nq[b] - 1) & 1);
                        if (w) {
                            mbar_arrive_expect_tx(q_full + b, L::Q_TILE);
#pragma unroll
                            for (int c = 0; c < D / 64; ++c) {
                                uint8_t *dst = smem + L::Q + b * L::Q_TILE + c * BM * 128;
                                if constexpr (CHUNKED)
                                    tc::tma_load_3d(dst, &tq, c * 64, it.h * G, row, q_full + b);
                                else
                                    tc::tma_load_2d(dst, &tq, qcol + c * 64, row, q_full + b);
                            }
                        } else {
                            fail();
                        }
                        ok = w;
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    ++nq[b];
                }
            };
            const int ne = ring_count<SHARED>(it);
            // packed mode: this item writes the K/V of its own rows (the first query head of each KV
            // group does), from the key tiles that hold them
            const int q0 = it.t[0].q0, qlast = it.t[1].n > 0 ? it.t[1].qlast : it.t[0].qlast;
            const bool writes = WRITER && a.write_pool && it.h % G == 0;
            int blkv = -1;
            if (writes) {
                const int lb = (q0 >> a.lg_bs) + lane;
                if ((lb << a.lg_bs) <= qlast && lb < a.max_blocks) blkv = a.tables[(int64_t)it.seq * a.max_blocks + lb];
            }
            // paged / cascade: lane l's table entry of block l of ring entry e (-1: no token there)
            auto entry = [&](int e) -> int {
                int t, j;
                const int kb = key_base(it, e, t, j);
                const int lb = (kb >> a.lg_bs) + lane;
                int at = lb;
                if constexpr (CHUNKED) at += lb >= it.from ? it.skip : 0;
                return (lane < (BN >> a.lg_bs) && (lb << a.lg_bs) < key_end(it, t))
                           ? a.tables[(int64_t)it.trow * a.max_blocks + at]
                           : -1;
            };
            int nxt = PAGED && ne > 0 ? entry(0) : -1;
            for (int e = 0; e < ne && ok; ++e) {
                int tile = 0, step = 0, st, round;
                if constexpr (ONE_Q) ring_entry<SHARED>(it, e, tile, step);
                next_stage(tile, st, round);
                // FP8: the previous tile is widened first (an MMA waits for it), then this one loads
                if (!widen_pending()) ok = false;
                flush_write(st); // the stage's previous tile leaves for the pool before the refill
                if (ok && round >= 1) ok = __all_sync(0xffffffffu, mbar_wait_hint(empty + st, (round - 1) & 1));
                if (!ok || __any_sync(0xffffffffu, *abort_flag != 0)) break;
                uint8_t *stage = ring + st * stage_bytes;
                if constexpr (PAGED) {
                    int t, j;
                    const int kbase = key_base(it, e, t, j), send = key_end(it, t);
                    const int nbt = BN >> a.lg_bs;
                    int b = nxt;
                    if (e + 1 < ne) nxt = entry(e + 1);
                    const int lb = (kbase >> a.lg_bs) + lane;
                    const bool has = lane < nbt && (lb << a.lg_bs) < send;
                    const bool good = has && b >= 0 && b < a.num_blocks;
                    if (!isK && has && !good) set_error(a.err, PKV_DEVERR_BLOCK_ID);
                    // K: every usable block whole (rows past the end are masked); V: only full blocks
                    bool full_blk = good && (isK || ((lb + 1) << a.lg_bs) <= send);
                    if constexpr (CHUNKED) // (a block with tokens that no row sees: its other V rows one by one)
                        full_blk = full_blk && (isK || (lb << a.lg_bs) >= it.hi || ((lb + 1) << a.lg_bs) <= it.lo);
                    const unsigned fullmask = __ballot_sync(0xffffffffu, full_blk);
                    if (lane == 0) mbar_expect_tx(full + st, (uint32_t)__popc(fullmask) * (uint32_t)(a.bs * D * EB));
                    __syncwarp();
                    if (full_blk) {
                        const int y = ((b * 2 + kvsel) * a.hkv + kvh) << a.lg_bs;
                        if constexpr (KV8) {
                            tc::tma_load_2d(stage + code_off + (lane << a.lg_bs) * D, &tp, 0, y, full + st);
                        } else {
#pragma unroll
                            for (int c = 0; c < (GROUPED ? 0 : D / 64); ++c)
                                tc::tma_load_2d(stage + c * BN * 128 + ((lane << a.lg_bs) * 128), &tp, c * 64, y,
                                                full + st);
                            if constexpr (GROUPED)
                                tc::tma_load_4d(stage + (lane << a.lg_bs) * 256, &tp, 0, 0, 0, y >> 3, full + st);
                        }
                    }
                    const unsigned allmask = nbt == 32 ? 0xffffffffu : (1u << nbt) - 1u;
                    if (!isK) {
                        for (int r0 = 0; fullmask != allmask && r0 < BN; r0 += RPI) {
                            const int r = r0 + rsub, l = r >> a.lg_bs;
                            const int bl = __shfl_sync(0xffffffffu, good ? b : -1, l);
                            if ((fullmask >> l) & 1u) continue;
                            uint4 x = make_uint4(0u, 0u, 0u, 0u);
                            bool held = bl >= 0 && kbase + r < send;
                            if constexpr (CHUNKED) held = held && !(kbase + r >= it.lo && kbase + r < it.hi);
                            if (held)
                                x = *reinterpret_cast<const uint4 *>(
                                    a.pool + ((((int64_t)bl * 2 + 1) * a.hkv + kvh) * a.tile_elems +
                                              (int64_t)(r - (l << a.lg_bs)) * D) * EB + cc * 16);
                            if constexpr (KV8) {
                                *reinterpret_cast<uint4 *>(stage + code_off + r * D + cc * 16) = x;
                            } else {
                                const int c2 = cc >> 3, u = cc & 7;
                                uint8_t *at = GROUPED ? stage + (r >> 3) * 2048 + c2 * 1024 + (r & 7) * 128
                                                      : stage + c2 * BN * 128 + r * 128;
                                *reinterpret_cast<uint4 *>(at + ((u ^ (r & 7)) << 4)) = x;
                            }
                        }
                        if constexpr (!KV8) fence_proxy_async_smem(); // the plain stores are read by the MMA
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + st);
                } else {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(full + st, L::TILE);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tc::tma_load_2d(stage + c * BN * 128, isK ? &tk : &tv, kvh * D + c * 64, it.start + e * BN,
                                            full + st);
                    }
                    if (writes && e >= q0 / BN) {
                        // the tile holds some of the item's own rows: write them before the stage is refilled
                        wj[st] = e;
                        wq0[st] = q0;
                        wql[st] = qlast;
                        wkvh[st] = kvh;
                        wblk[st] = blkv;
                        wpar[st] = (int)(round & 1);
                    }
                }
                ++g;
                if constexpr (ONE_Q) ++(tile ? gt[1] : gt[0]);
                if constexpr (KV8 && !CODES) pend = st | (round & 1) << 8;
                if (isK && e < 2) issue_q(e); // Q_A after K tile 0, Q_B after K tile 1
            }
            if (isK) issue_q(1); // items of fewer than two key tiles
            if (!isK && lane == 0) mbar_arrive(item_empty + (n & (kItemSlots - 1)));
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        }
        // FP8: the last tile issued is widened too (an MMA may still be waiting for it)
        if (ok && !widen_pending() && lane == 0) fail();
        // pending pool writes leave now; every store has completed before the CTA exits
        for (int st = 0; st < ns; ++st) flush_write(st);
        if constexpr (WRITER) tc::bulk_wait_all();
        // the last loads must land before this CTA's shared memory goes away
        if (lane == 0) {
            if constexpr (ONE_Q) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    for (int c = max(gt[t] - ns / 2, 0); c < gt[t]; ++c)
                        if (!mbar_wait_hint(full + t + 2 * (c % (ns / 2)), (c / (ns / 2)) & 1)) set_error(a.err, PKV_DEVERR_TIMEOUT);
            } else {
                for (int64_t gg = g > ns ? g - ns : 0; gg < g; ++gg)
                    if (!mbar_wait_hint(full + gg % ns, (gg / ns) & 1)) set_error(a.err, PKV_DEVERR_TIMEOUT);
            }
            if (isK)
                for (int b = 0; b < 2; ++b)
                    if (nq[b] >= 1 && !mbar_wait_hint(q_full + b, (nq[b] - 1) & 1)) set_error(a.err, PKV_DEVERR_TIMEOUT);
        }
    } else if (warp == 1 || warp == 3) {
        // ---------------------------------------------------------------- MMA issuers
        // Warp 1 issues the products of tile A, warp 3 those of tile B, each from a converged warp with
        // one elected lane issuing (waits agreed with __all_sync).  Per tile: S(0), then per key step
        // j: P V(j), S(j+1).  S(j+1) follows P V(j) from the same thread, so it overwrites the S
        // columns only after P V(j) has read P from them.  Two issuers keep the tensor pipe's queue fed
        // while either waits for its softmax.  Commits track the issuing thread's own MMAs.
        const int t = warp == 1 ? 0 : 1;
        constexpr uint32_t IQK = tc::idesc_f16(OT == PKV_BF16 ? 1u : 0u, 0u, BM, BN);
        constexpr uint32_t IPV = tc::idesc_f16(OT == PKV_BF16 ? 1u : 0u, 1u, BM, D);
        // one descriptor per operand layout; the address field counts 16-byte units, so a tile at byte
        // offset `off` from the base is the base descriptor plus off / 16
        const uint64_t dQ = tc::smem_desc(smem_u32(smem + L::Q), 16, 1024);
        const uint64_t dK = tc::smem_desc(smem_u32(smem + L::K0), 16, GROUPED ? 2048 : 1024);
        const uint64_t dV = GROUPED ? tc::smem_desc(smem_u32(smem + L::V0), 1024, 2048)
                                    : tc::smem_desc(smem_u32(smem + L::V0), BN * 128, 1024);
        constexpr int kHalf = GROUPED ? 1024 : BN * 128, kKeys16 = GROUPED ? 4096 : 2048; // bytes between halves; of 16 keys
        const uint32_t tS = tmem + (uint32_t)(t * BN), tO = tmem + (uint32_t)(2 * BN + t * D);
        bool any_mma = false, ok = true;
        // ring cursors: the stage of the K (V) entry to look at next and the parity of its phase (ONE_Q: of the tile's own
        // half of the ring)
        constexpr int KN = ONE_Q ? NKS / 2 : NKS, VN = ONE_Q ? NVS / 2 : NVS;
        auto stage = [&](uint32_t st) -> uint32_t { return ONE_Q ? (uint32_t)t + 2 * st : st; };
        uint32_t kst = 0, kph = 0, vst = 0, vph = 0;
        uint32_t pph = 0, oph = 0, qph = 0; // phase parities of this tile's barriers
        bool o_used = false;
        auto adv = [](uint32_t &st, uint32_t &ph, int nstage) {
            if (++st == (uint32_t)nstage) {
                st = 0;
                ph ^= 1u;
            }
        };
        for (int n = 0; ok; ++n) {
            const It it = take_item(n, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || it.seq < 0) break;
            const int nt = t ? it.t[1].n : it.t[0].n;
            const int ne = ring_count<SHARED>(it);
            const int qb = ONE_Q ? 0 : t;
            // S(j) = Q K^T into the tile's S columns (its MMAs only; the caller commits)
            auto mmas_s = [&]() {
                const uint64_t a0 = dQ + (uint64_t)((qb * L::Q_TILE) >> 4);
                const uint64_t b0 = dK + (uint64_t)(stage(kst) * (L::STAGE >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int c = k >> 2, kk = k & 3;
                    tc::mma_f16_warp(tS, a0 + (uint64_t)((c * BM * 128 + kk * 32) >> 4),
                                     b0 + (uint64_t)((c * kHalf + kk * 32) >> 4), IQK, k > 0 ? 1u : 0u);
                }
            };
            // after S(j): S complete, this warp's share of the K stage, and Q after the tile's last S
            auto commit_s = [&](int j) {
                tc::commit_warp(s_full + t);
                tc::commit_warp(k_empty + stage(kst)); // this warp's share of the K stage
                adv(kst, kph, KN);
                if (j == nt - 1) {
                    // cascade: the last S of the tile has read Q (other modes: the epilogue, which stages
                    // the tile's output in the Q buffer, frees it)
                    if constexpr (ONE_Q) tc::commit_warp(q_empty + qb);
                    qph ^= 1u;
                }
            };
            // S(0): Q and the first K tile
            auto first_s = [&]() -> bool {
                if (!__all_sync(0xffffffffu, mbar_wait(k_ready + stage(kst), kph) && mbar_wait(q_ready + qb, qph))) return false;
                tc::fence_after_sync();
                any_mma = true;
                mmas_s();
                commit_s(0);
                return true;
            };
            // O += P(j) V(j), then S(j + 1) right behind it: the pipe gets both groups back to back.
            // P is read from tensor memory where the softmax left it (over S), and S(j + 1) overwrites
            // those columns only after P V(j) has read them (one thread's MMAs complete in order).
            auto step = [&](int j) -> bool {
                const bool more = j + 1 < nt;
                // the next K tile is normally in place already; checked first, so that nothing but the
                // softmax is waited for between the two groups
                if (more && !__all_sync(0xffffffffu, mbar_wait(k_ready + stage(kst), kph))) return false;
                bool w = mbar_wait(v_ready + stage(vst), vph) && mbar_wait(p_full + t, pph);
                // the previous item's epilogue of this tile has read O out of tensor memory
                if (j == 0 && o_used) w = w && mbar_wait(o_free + t, oph ^ 1u);
                if (!__all_sync(0xffffffffu, w)) return false;
                pph ^= 1u;
                tc::fence_after_sync();
                const uint64_t b0 = dV + (uint64_t)(stage(vst) * (L::STAGE >> 4));
#pragma unroll
                for (int part = 0; part < NP; ++part)
#pragma unroll
                    for (int k = 0; k < BN / 16; ++k)
                        tc::mma_f16_ts_warp(tO, tS + (uint32_t)(part * (BN / 2) + k * 8), b0 + (uint64_t)((k * kKeys16) >> 4),
                                            IPV, (j > 0 || k > 0 || part > 0) ? 1u : 0u);
                // the V stage share goes out before S(j + 1) is issued (a commit covers every earlier MMA of
                // this thread, so issued later it would hold the stage until S(j + 1) completes too); the
                // P V MMAs queued ahead keep the pipe busy meanwhile
                tc::commit_warp(v_empty + stage(vst)); // this warp's share of the V stage
                adv(vst, vph, VN);
                if (more) mmas_s();
                if (!more) {
                    tc::commit_warp(o_full + t); // the tile's O is complete once this commit arrives
                    oph ^= 1u;
                    o_used = true;
                } else {
                    commit_s(j + 1);
                }
                return true;
            };
            if (nt > 0) ok = first_s();
            for (int j = 0; j < nt && ok; ++j) ok = step(j);
            if constexpr (SHARED) {
                // Key tiles that only the other tile reads: this warp's share of their release, once they have landed.  (Passed
                // over without a wait, or released by the other tile's issuer for both, this warp could come to a stage
                // two of its phases ahead, and find the phase of the same parity before it complete.)
                for (int e = nt; e < ne && ok; ++e) {
                    ok = __all_sync(0xffffffffu, mbar_wait_hint(k_ready + kst, kph));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive(k_empty + kst);
                    adv(kst, kph, KN);
                    ok = __all_sync(0xffffffffu, mbar_wait_hint(v_ready + vst, vph));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive(v_empty + vst);
                    adv(vst, vph, VN);
                }
            } else {
                if (nt == 0 && ok) {
                    // cascade: no split for this tile; its share of the Q buffer once Q has landed
                    ok = __all_sync(0xffffffffu, mbar_wait_hint(q_ready + qb, qph));
                    if (ok && lane == 0) mbar_arrive(q_empty + qb);
                    qph ^= 1u;
                }
            }
            if (lane == 0) mbar_arrive(item_empty + (n & (kItemSlots - 1)));
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        }
        if (!ok && lane == 0) fail();
        // every MMA issued by this warp's elected lane has completed before TMEM is released (a warp that
        // issued none has nothing to wait for)
        if (any_mma) {
            tc::commit_warp(fin + t);
            if (!__all_sync(0xffffffffu, mbar_wait_hint(fin + t, 0)) && lane == 0) set_error(a.err, PKV_DEVERR_TIMEOUT);
        }
    } else if (CODES && warp >= 12) {
        // ---------------------------------------------------------------- widening (warps 12-15)
        // Thread r owns row r of every tile, K or V, K one tile ahead of V (a V tile waits for the products with the one
        // before it, the next K tile only for its own stage), and of every bf16 Q tile.
        if constexpr (CODES) {
            const int r = (warp - 12) * 32 + lane;
            bool ok = true;
            uint32_t g[2] = {0, 0};  // K, V tiles widened
            uint32_t nq[2] = {0, 0}; // Q tiles
            auto widen = [&](auto which) -> bool {
                constexpr int kv = decltype(which)::value;
                uint64_t *const land = kv ? v_full : k_full, *const read = kv ? v_spare : k_spare;
                uint64_t *const free = kv ? v_empty : k_empty, *const done = kv ? vc_full : kc_full;
                const uint32_t st = g[kv] % NKS, round = g[kv] / NKS;
                const uint32_t cs = g[kv] % L::NCS;
                bool w = mbar_wait_hint(land + cs, (g[kv] / L::NCS) & 1u);
                ++g[kv];
                if (w && round > 0) w = mbar_wait_hint(free + st, (round - 1) & 1u);
                if (!__all_sync(0xffffffffu, w)) return false;
                widen_codes<D>(smem + L::C0 + (kv * L::NCS + cs) * L::CODE, smem + (kv ? L::V0 : L::K0) + st * L::STAGE, r);
                fence_proxy_async_smem(); // the MMAs read the tile through the async proxy
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(read + cs);
                    mbar_arrive(done + st);
                }
                return true;
            };
            auto convert_q = [&](int b) -> bool {
                if constexpr (MT == PKV_BF16) {
                    const uint32_t n = b ? nq[1]++ : nq[0]++;
                    if (!__all_sync(0xffffffffu, mbar_wait_hint(q_full + b, n & 1u))) return false;
                    q_exp[((n & 1) * 2 + b) * BM + r] = (int8_t)q_to_f16<D>(smem + L::Q + b * L::Q_TILE, r);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(qc_full + b);
                }
                return true;
            };
            for (int n = 0; ok; ++n) {
                int n0, n1;
                {
                    const It it = take_item(n, ok);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok || it.seq < 0) break;
                    n0 = it.t[0].n;
                    n1 = it.t[1].n;
                }
                const int ne = max(n0, n1);
                // step -1: K tile 0 and Q_A; step e: K tile e + 1, (step 0: Q_B), V tile e
                for (int e = -1; e < ne && ok; ++e) {
                    if (e + 1 < ne) ok = widen(std::integral_constant<int, 0>());
                    if (ok && (e == -1 ? n0 > 0 : e == 0 && n1 > 0)) ok = convert_q(e + 1);
                    if (ok && e >= 0) ok = widen(std::integral_constant<int, 1>());
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(item_empty + (n & (kItemSlots - 1)));
                if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            }
            if (!ok && lane == 0) fail();
        }
    } else {
        if constexpr (CODES)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------------------------------------------------------- softmax, one thread per row
        const int t = (warp - 4) >> 2;          // tile A (warps 4-7) or B (warps 8-11)
        const int r = (warp & 3) * 32 + lane;   // query row of the tile = tensor-memory lane
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + (uint32_t)(t * BN);
        const uint32_t tO = tmem + lane_off + (uint32_t)(2 * BN + t * D);
        bool ok = true;
        int ns = 0, no = 0, nepi = 0, q_seen = 0; // q_seen: Q tiles of this tile's buffer in earlier items
        (void)q_seen;
        int steps0 = 0, steps1 = 0; // key steps of tiles A and B in earlier items
        // The two tiles' softmaxes take turns on the exponentials (they share the SMSPs and their
        // transcendental units; run together, each takes twice as long and the MMAs of both tiles
        // wait): in an item, A's step j follows B's step j - 1, and B's step j follows A's step j.
        // The wait reads the other tile's monotonic count of finished steps, polled with a bound.
        auto wait_turn = [&](int other, int target) -> bool {
            volatile int *prog = sm_prog + other;
            if (*prog >= target) return true;
            const uint64_t t0 = global_timer_ns();
            for (uint32_t i = 0; i < 0x80000000u; ++i) {
                if (*prog >= target) return true;
                __nanosleep(32);
                if ((i & 63u) == 0u && global_timer_ns() - t0 > PKV_WAIT_LIMIT_NS) return false;
            }
            return false;
        };
        for (int n = 0; ok; ++n) {
            const It it = take_item(n, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || it.seq < 0) break;
            const Tile x = t ? it.t[1] : it.t[0];
            const int n0 = it.t[0].n, n1 = it.t[1].n;
            if (x.n > 0) {
                const int kvh = kv_head(it);
                float sl = KV8 ? a.scale_log2 * a.k_scale[kvh] : a.scale_log2;
                const int qpos = x.qpos0 + (CHUNKED ? r >> a.lg_group : r); // absolute position of this row (causal modes)
                float m_use = -INFINITY, l = 0.f;
                for (int j = 0; j < x.n && ok; ++j) {
                    // (spinning: S complete is on the critical path; a suspended wait wakes later)
                    ok = __all_sync(0xffffffffu, mbar_wait(s_full + t, ns & 1));
                    if (!ok) break;
                    ++ns;
                    tc::fence_after_sync();
                    if constexpr (CODES && MT == PKV_BF16) {
                        // q's power of two: S is complete, so the row is converted; the next but one Q tile, which
                        // writes this slot again, waits for the next one's S, and that for this row's P
                        if (j == 0) sl *= exp2f((float)q_exp[((q_seen & 1) * 2 + t) * BM + r]);
                    }
                    uint32_t sr[BN];
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c)
                        tc::ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
                    tc::wait_ld();
                    const int kbase = x.k0 + j * BN;
                    if constexpr (CASCADE) {
                        // every query sees the whole split: only keys past its end are masked
                        if (kbase + BN > x.kend) {
                            const int lim = x.kend - kbase;
#pragma unroll
                            for (int c = 0; c < BN; ++c)
                                if (c >= lim) sr[c] = 0xFF800000u; // -inf
                        }
                    } else if constexpr (CHUNKED) {
                        // seen key kbase + c is at most this row's position up to c = upto - 1, inside its window from
                        // c = since on, a sink below c = first; only tiles on either edge of some row's sight
                        const int hidden = it.skip << a.lg_bs; // tokens between the sinks' blocks and the window's
                        const int plast = x.qpos0 + x.qlast - x.q0; // position of the tile's last row
                        const bool late = kbase + BN - 1 + hidden > x.qpos0;
                        const bool early = a.window > 0 && plast - a.window + 1 - hidden > kbase;
                        if (late || early) {
                            const int upto = qpos + 1 - hidden - kbase;
                            const int since = a.window > 0 ? qpos - a.window + 1 - hidden - kbase : 0;
                            const int first = min(a.sinks, qpos + 1) - kbase;
                            // (a word of seen keys at a time: tested one by one against three bounds they cost 70 registers)
#pragma unroll
                            for (int w = 0; w < BN / 32; ++w) {
                                const uint32_t in = (ones_below(upto - 32 * w) & ~ones_below(since - 32 * w)) | ones_below(first - 32 * w);
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    if (!(in & (1u << c))) sr[32 * w + c] = 0xFF800000u; // -inf
                            }
                        }
                    } else if (kbase + BN - 1 > x.qpos0) {
                        // causal mask, only on tiles that reach past the tile's first query row
                        const int lim = qpos - kbase + 1; // keys c < lim are at or before this row
#pragma unroll
                        for (int c = 0; c < BN; ++c)
                            if (c >= lim) sr[c] = 0xFF800000u; // -inf
                    }
                    // row maximum: eight independent chains of three-input maxima, then a short tree
                    float mc[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) mc[q] = __uint_as_float(sr[q]);
#pragma unroll
                    for (int c = 8; c < BN; c += 16) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) mc[q] = max3(mc[q], __uint_as_float(sr[c + q]), __uint_as_float(sr[c + 8 + q]));
                    }
                    const float mx = fmaxf(max3(mc[0], mc[1], mc[2]), max3(mc[3], mc[4], max3(mc[5], mc[6], mc[7]))) *
                                     sl; // scale > 0 keeps the order
                    const bool up = mx > m_use + (kRescale + kUp);
                    const float m_new = up ? mx - kUp : m_use;
                    const float alpha = up ? fast_exp2(m_use - m_new) : 1.f;
                    m_use = m_new;
                    const float nbase = m_use == -INFINITY ? 0.f : -m_use; // a row with no live key yet keeps p = 0
                    // O rescale (rows whose base moved): P V(j - 1) has completed, since S(j) has
                    if (j > 0 && __any_sync(0xffffffffu, up)) {
#pragma unroll
                        for (int cc = 0; cc < D / 16; ++cc) {
                            uint32_t o[16];
                            tc::ld16(tO + cc * 16, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tc::st16(tO + cc * 16, o);
                        }
                    }
                    // this tile's turn on the exponentials (see wait_turn)
                    if (t == 0 ? (j >= 1 && j - 1 < n1) : (j < n0)) {
                        const int target = 4 * (t == 0 ? steps1 + j : steps0 + j + 1);
                        ok = __all_sync(0xffffffffu, wait_turn(1 - t, target));
                        if (!ok) break;
                    }
                    float2 rs = make_float2(0.f, 0.f);
                    const float2 sc2 = make_float2(sl, sl), nb2 = make_float2(nbase, nbase);
                    // P over the S columns: packed pairs, key c in column c / 2 (bf16: lo parts from BN / 2)
                    // (keys per store: 32 for fp16 P, 16 for a bf16 hi + lo pair, to keep registers for S)
                    constexpr int KC = NP == 2 ? 16 : 32;
#pragma unroll
                    for (int q = 0; q < BN / KC; ++q) {
                        uint32_t phi[KC / 2], plo[NP == 2 ? KC / 2 : 1];
#pragma unroll
                        for (int c = 0; c < KC / 2; ++c) {
                            const int k = q * KC + 2 * c;
                            const float2 xx =
                                fma2(make_float2(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), sc2, nb2);
                            const float p0 = fast_exp2(xx.x), p1 = fast_exp2(xx.y);
                            rs = add2(rs, make_float2(p0, p1));
                            phi[c] = pack2(p0, p1, OT);
                            if constexpr (NP == 2) // remainders after bf16 rounding, themselves rounded to bf16
                                plo[c] = pack2(p0 - __uint_as_float(phi[c] << 16),
                                               p1 - __uint_as_float(phi[c] & 0xFFFF0000u), OT);
                        }
                        if constexpr (NP == 2) {
                            tc::stn<8>(tS + q * 8, phi);
                            tc::stn<8>(tS + BN / 2 + q * 8, plo);
                        } else {
                            tc::st16(tS + q * 16, phi);
                        }
                    }
                    l = l * alpha + (rs.x + rs.y);
                    tc::wait_st();
                    tc::fence_before_sync();
                    __syncwarp(); // every lane's P is stored; one arrival for the warp
                    if (lane == 0) {
                        mbar_arrive(p_full + t);
                        atomicAdd(sm_prog + t, 1); // this warp's exp phase of the step is done
                    }
                }
                // the tile's O is complete
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait_hint(o_full + t, no & 1));
                if (!ok) break;
                ++no;
                tc::fence_after_sync();
                using T = typename ModelT<MT>::T;
                const float vs = KV8 ? a.v_scale[kvh] : 1.f;
                if constexpr (CASCADE) {
                    // fp32 partial of (sequence it.start + r, head it.h, split 2 pr + t): unnormalised o
                    // and (m, l) with m the row's exponent base in log2 units, as the split merge expects
                    const bool valid = r < it.n;
                    const int64_t idx = ((int64_t)(it.start + r) * a.hq + it.h) * a.max_splits + 2 * it.pr + t;
                    float *wo = a.ws_o + idx * D;
                    uint32_t o[D]; // the whole row in one tensor-memory round trip
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) tc::ld32(tO + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[cc * 32]));
                    tc::wait_ld();
                    if (valid) {
                        float4 *dst = reinterpret_cast<float4 *>(wo);
#pragma unroll
                        for (int e = 0; e < D / 4; ++e)
                            dst[e] = make_float4(__uint_as_float(o[4 * e]) * vs, __uint_as_float(o[4 * e + 1]) * vs,
                                                 __uint_as_float(o[4 * e + 2]) * vs, __uint_as_float(o[4 * e + 3]) * vs);
                    }
                    if (valid) reinterpret_cast<float2 *>(a.ws_ml)[idx] = make_float2(m_use, l);
                } else if (CHUNKED && chunk_splits(it, t) > 1) {
                    if constexpr (CHUNKED) {
                        // fp32 partial of one of several splits, as in cascade mode; the Q buffer is not used
                        const int tok = x.q0 + (r >> a.lg_group);
                        const int64_t idx =
                            ((int64_t)(it.start + tok) * a.hq + it.h * G + (r & (G - 1))) * a.max_splits + it.split;
                        uint32_t o[D];
#pragma unroll
                        for (int cc = 0; cc < D / 32; ++cc) tc::ld32(tO + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[cc * 32]));
                        tc::wait_ld();
                        if ((warp & 3) == 0 && lane == 0) mbar_arrive(q_empty + t);
                        if (tok <= x.qlast) {
                            float4 *dst = reinterpret_cast<float4 *>(a.ws_o + idx * D);
#pragma unroll
                            for (int e = 0; e < D / 4; ++e)
                                dst[e] = make_float4(__uint_as_float(o[4 * e]) * vs, __uint_as_float(o[4 * e + 1]) * vs,
                                                     __uint_as_float(o[4 * e + 2]) * vs, __uint_as_float(o[4 * e + 3]) * vs);
                            reinterpret_cast<float2 *>(a.ws_ml)[idx] = make_float2(m_use, l);
                        }
                    }
                } else {
                    // (chunk mode: rows are (token, head) pairs, and one may see no key)
                    const int row = CHUNKED ? x.q0 + (r >> a.lg_group) : x.q0 + r;
                    const int tile_rows = CHUNKED ? BM >> a.lg_group : BM;
                    const float inv = CHUNKED && l == 0.f ? 0.f : vs / l;
                    uint32_t o[D]; // the whole row in one tensor-memory round trip
#pragma unroll
                    for (int cc = 0; cc < D / 32; ++cc) tc::ld32(tO + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[cc * 32]));
                    tc::wait_ld();
                    const bool lead = (warp & 3) == 0 && lane == 0;
                    if (x.q0 + tile_rows <= it.n) {
                        // a whole tile of the sequence's rows: staged in this tile's Q buffer (free, since the
                        // tile's last S has completed) in the Q tile's own 128-byte swizzled layout, then one TMA
                        // store per 64 columns writes coalesced rows; the buffer goes back to the Q loader once
                        // the stores have read it
                        uint8_t *stage = smem + L::Q + t * L::Q_TILE;
#pragma unroll
                        for (int cc = 0; cc < D / 8; ++cc) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack2(__uint_as_float(o[8 * cc + 2 * e]) * inv, __uint_as_float(o[8 * cc + 2 * e + 1]) * inv, MT);
                            const int h = cc >> 3, u = cc & 7;
                            *reinterpret_cast<uint4 *>(stage + h * BM * 128 + r * 128 + ((u ^ (r & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        fence_proxy_async_smem(); // the stores read the tile through the async proxy
                        __syncwarp();
                        if (lane == 0) mbar_arrive(epi + t);
                        if (lead) {
                            // the four warps' rows are staged (bounded wait: a warp that gave up never arrives)
                            if (mbar_wait(epi + t, nepi & 1)) {
#pragma unroll
                                for (int h = 0; h < D / 64; ++h) {
                                    if constexpr (CHUNKED)
                                        tc::tma_store_3d(&to, h * 64, it.h * G, it.start + x.q0, stage + h * BM * 128);
                                    else
                                        tc::tma_store_2d(&to, it.h * D + h * 64, it.start + x.q0, stage + h * BM * 128);
                                }
                                tc::bulk_commit();
                                tc::bulk_wait_read_all();
                                mbar_arrive(q_empty + t);
                            } else {
                                ok = false;
                            }
                        }
                        ++nepi;
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                    } else {
                        // the sequence's last, partial tile: row by row, so that no row of the next sequence is
                        // written; the Q buffer is not used here and is free already
                        if (lead) mbar_arrive(q_empty + t);
                        if (row < it.n) {
                            const int head = CHUNKED ? it.h * G + (r & (G - 1)) : it.h;
                            T *orow = static_cast<T *>(a.out) + ((int64_t)(it.start + row) * a.hq + head) * D;
#pragma unroll
                            for (int cc = 0; cc < D / 8; ++cc) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = pack2(__uint_as_float(o[8 * cc + 2 * e]) * inv,
                                                 __uint_as_float(o[8 * cc + 2 * e + 1]) * inv, MT);
                                reinterpret_cast<uint4 *>(orow)[cc] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free + t); // O has been read out; the tile's next first P V may overwrite it
            } else if constexpr (CHUNKED) {
                // rows that see no key at all
                const int tok = x.q0 + (r >> a.lg_group);
                if (it.zero && chunk_splits(it, t) == 0 && tok <= x.qlast) {
                    using T = typename ModelT<MT>::T;
                    uint4 *orow = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) +
                                                            ((int64_t)(it.start + tok) * a.hq + it.h * G + (r & (G - 1))) * D);
#pragma unroll
                    for (int cc = 0; cc < D / 8; ++cc) orow[cc] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            steps0 += n0;
            steps1 += n1;
            if (CODES && x.n > 0) ++q_seen;
            __syncwarp();
            if (lane == 0) mbar_arrive(item_empty + (n & (kItemSlots - 1)));
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        }
        if (!ok) fail();
        // the output tiles' TMA stores have completed before the CTA exits
        if (!CASCADE && (warp & 3) == 0 && lane == 0) tc::bulk_wait_all();
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
    if constexpr (CASCADE) pdl_wait(); // the grid completes after the suffix decode (see above)
}

// launch of one instantiation (prefill_packed.cu, prefill_paged.cu, prefill_cascade.cu)
template <int D, int MT, int MODE, bool KV8>
cudaError_t launch_attn(const Maps &m, const Args &a, int64_t max_ctas, int num_sms, cudaStream_t st) {
    auto kern = attn_kernel<D, MT, MODE, KV8>;
    const int smem = smem_total<D, MODE, KV8>();
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>(max_ctas, (int64_t)num_sms);
    return pdl_launch(kern, dim3((unsigned)grid), dim3(threads_of<MODE, KV8>()), smem, st, m, a);
}

#define PKV_ATTN_EXTERN(MODE, KV8)                                                                                     \
    extern template cudaError_t launch_attn<128, PKV_F16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t);  \
    extern template cudaError_t launch_attn<128, PKV_BF16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t); \
    extern template cudaError_t launch_attn<64, PKV_F16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t);   \
    extern template cudaError_t launch_attn<64, PKV_BF16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t);
#define PKV_ATTN_INSTANTIATE(MODE, KV8)                                                                         \
    template cudaError_t launch_attn<128, PKV_F16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t);  \
    template cudaError_t launch_attn<128, PKV_BF16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t); \
    template cudaError_t launch_attn<64, PKV_F16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t);   \
    template cudaError_t launch_attn<64, PKV_BF16, MODE, KV8>(const Maps &, const Args &, int64_t, int, cudaStream_t);

PKV_ATTN_EXTERN(MODE_PACKED, false)
PKV_ATTN_EXTERN(MODE_PAGED, false)
PKV_ATTN_EXTERN(MODE_PAGED, true)
PKV_ATTN_EXTERN(MODE_CASCADE, false)
PKV_ATTN_EXTERN(MODE_CASCADE, true)
PKV_ATTN_EXTERN(MODE_CHUNK, false)
PKV_ATTN_EXTERN(MODE_CHUNK, true)

} // namespace pkv_prefill
