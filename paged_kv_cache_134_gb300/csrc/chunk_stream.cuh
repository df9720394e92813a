// Attention of chunks of few rows over a paged cache (paged_chunk_attention where a sequence's new tokens times the query
// heads of a KV head fill one tile of 128 rows): drafted tokens, single tokens.
//
// The mathematics are those of prefill_impl.cuh: S = Q K^T and O += P V on tcgen05 with accumulators in tensor memory, an
// online softmax with a base that moves only when a row's maximum passes it by more than 2^8, one thread a row.
//
// (Weights of one fp16, or a pair of bf16: see kChunkUp.)
//
// A unit is (sequence, KV head, tile of rows, split of its keys): row r is token q0 + r / G, query head h G + r % G, so a
// KV head's keys are read once for all its query heads and all new tokens.  What bounds it is HBM (K and V once, 2 rows
// flops a byte), as long as copies stay in flight.  One unit's chain of products and softmax (S, exponentials, P V: about
// 3500 cycles for 128 keys, 64 KB of a 16-bit cache, that HBM brings to an SM in 2800) cannot keep it busy, and it
// stands still at every unit's end.  So a CTA runs two pipelines that share nothing but the SM: each has a loader, an MMA issuer,
// four softmax warps, its half of shared and of tensor memory, and takes units of its own from the list.  (Two splits
// of one unit side by side, sharing Q and ending together: 205 us on 32 sequences of up to 4096 tokens, 32 heads, 5 new
// tokens each, and 251 us on 256 ragged sequences over an E4M3 cache, 4 new tokens.)
//
// FEW (at most 64 rows, half a tile): both pipelines' rows lie in one Q tile, 0..63 and 64..127, and each multiplies all of
// it (the other's rows come out as garbage that nobody reads).  Their softmax warps then sit on different quarters of
// tensor memory, hence of the SM, and do not compete for the exponentials; of the four of a pipeline two have no rows and end,
// or widen codes.  The room goes to a third stage.
//
// K and V tiles take turns in one ring, K(0), V(0), K(1), ...: with three stages V(j + 1) loads once S(j) is done and K(j + 2)
// once P V(j) is, each about a step before it is needed.  (Rings of two for K and one for V: V(j + 1) could only follow
// P V(j), and its way from HBM was in the chain of every step.)
//
// E4M3 caches: codes land in a ring of their own, K and V in turn, and two more warps a pipeline (FEW: four) widen them to
// fp16 (see CodeLayout); a bf16 q is scaled into fp16 by the same warps.
//
// The loader works a unit out once and publishes it, while the unit before is being loaded, in a ring of four.
// Every wait is bounded; a timeout sets PKV_DEVERR_TIMEOUT and the CTA winds down.
#pragma once

#include "prefill_impl.cuh"

namespace pkv_prefill {

template <int D, bool KV8, bool FEW>
struct StreamLayout {
    static constexpr int NS = !KV8 && FEW ? 3 : 2;                     // stages of a pipeline, K and V in turn
    static constexpr int NC = KV8 ? (D == 64 ? 4 : FEW ? 2 : 1) : 0;   // code stages of a pipeline, K and V in turn
    static constexpr int Q_TILE = BM * D * 2, TILE = BN * D * 2, CODE = BN * D;
    static constexpr int NQ = FEW ? 1 : 2;
    static constexpr int Q = 0;
    static constexpr int T0 = Q + NQ * Q_TILE;           // [pipeline][stage]
    static constexpr int C0 = T0 + 2 * NS * TILE;        // [pipeline][stage]
    static constexpr int UNITS = C0 + 2 * NC * CODE;     // [pipeline][kUnitSlots] StreamUnit
    static constexpr int kUnitSlots = 4;
    static constexpr int EXP = UNITS + 2 * kUnitSlots * 64; // [pipeline][2 Q tiles][BM] exponents of q's rows (int8)
    static constexpr int BAR = EXP + (KV8 ? 2 * 2 * BM : 0);
    // a pipeline's barriers: units full, empty; Q full, empty, as fp16; tiles full, empty; codes landed, read; S full, P
    // full, O full, O free; end
    static constexpr int NBARS = 2 * kUnitSlots + 3 + 2 * NS + 2 * (NC ? NC : 1) + 4 + 1;
    static constexpr int kSoftmax = FEW ? 2 : 4;             // softmax warps of a pipeline
    static constexpr int kWiden = KV8 ? (FEW ? 4 : 2) : 0;   // warps that widen
    static constexpr int MISC = BAR + 2 * NBARS * 8; // tensor-memory address, abort flag
    static constexpr int TOTAL = MISC + 16;
    static_assert(TOTAL + 1024 <= 232448, "shared memory");
};

// a unit as its loader publishes it
struct StreamUnit {
    int n;         // key tiles; -1: no more units; 0: rows without keys
    int h;         // KV head
    int k0, kend;  // first seen key, and where the sequence's (the split's) seen keys end
    int hidden;    // tokens left out between the sinks' blocks and the window's: seen block i is i + hidden / bs from `from` on
    int from, lo, hi; // seen keys [lo, hi) are hidden from every row
    int trow;      // block-table row
    int qpos0;     // position of the tile's first row
    int row0, ntok; // packed row of its first token, tokens
    int split, nsplit;
    int pad[2];
};
static_assert(sizeof(StreamUnit) == 64, "a slot");

PKV_DEV StreamUnit stream_unit(const Args &a, int seq, int g, int split, int h) {
    StreamUnit u;
    u.n = -1;
    u.pad[0] = u.pad[1] = 0;
    if (seq < 0) return u;
    const int per_tile = BM >> a.lg_group, start = a.cu[seq], n = a.cu[seq + 1] - start, q0 = g * per_tile;
    const int before = max(a.lens[seq], 0) - n; // position of the first new token (negative: those rows see nothing)
    const int p0 = before + q0;                 // of the tile's first row
    const Hidden hid = hidden_from(a, p0);
    u.from = hid.from;
    u.lo = hid.lo;
    u.hi = hid.hi;
    u.h = h;
    u.hidden = hid.skip << a.lg_bs;
    u.trow = seq;
    u.qpos0 = p0;
    u.row0 = start + q0;
    u.ntok = min(per_tile, n - q0);
    const int end = max(p0 + u.ntok - u.hidden, 0), tiles = (end + BN - 1) / BN, per = steps_per_split(a, tiles);
    u.split = split;
    u.nsplit = (tiles + per - 1) / per;
    u.k0 = split * per * BN;
    u.n = min(max(tiles - split * per, 0), per);
    u.kend = min(end, u.k0 + per * BN);
    return u;
}

// the place `at` among all that the call's sizes allow, or the next of this pipeline's that holds a unit: (sequence, tile, split, KV head)
PKV_DEV int4 direct_unit(const Args &a, int &at, int stride) {
    for (; at < a.rect; at += stride) {
        const int h = at % a.hkv, r = at / a.hkv, part = r % a.max_parts, g = r / a.max_parts % a.max_groups;
        const int seq = r / a.max_parts / a.max_groups;
        if (g >= chunk_groups<false>(a, seq, h == 0 && part == 0 && g == 0)) continue;
        if (part > 0 && part >= stream_unit(a, seq, g, 0, 0).nsplit) continue;
        at += stride;
        return make_int4(seq, g, part, h);
    }
    return make_int4(-1, 0, 0, 0);
}

template <bool KV8>
__host__ __device__ constexpr int stream_threads() {
    return KV8 ? 512 : 384;
}

template <int D, int MT, bool KV8, bool FEW>
__global__ void __launch_bounds__(stream_threads<KV8>(), 1)
    stream_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tp, const Args a) {
    using L = StreamLayout<D, KV8, FEW>;
    constexpr int OT = KV8 ? (int)PKV_F16 : MT;  // the products' operands
    constexpr int NP = OT == PKV_BF16 ? 2 : 1;   // P parts (bf16: hi + lo)
    constexpr float kUp = OT == PKV_F16 ? kChunkUp : 0.f;
    constexpr int EB = KV8 ? 1 : 2;              // pool bytes per element
    constexpr bool GROUPED = D == 128 && !KV8;   // one box a block, [8 rows][half][8 rows][128 bytes] (see attn_kernel)
    constexpr bool SCALE_Q = KV8 && MT == PKV_BF16;
    constexpr int NS = L::NS, NC = L::NC, NU = L::kUnitSlots;
    constexpr int kRows = FEW ? 64 : 128;        // rows of a pipeline in the Q tile
    extern __shared__ __align__(1024) uint8_t smem[];

    if (a.few_rows == 0) pdl_trigger();
    if (smem_u32(smem) & 1023u) return; // the swizzled tiles need 1024-byte alignment (always true)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // loaders 0 and 2, issuers 1 and 3, softmax 4-7 and 8-11 (FEW: 4-5 and 10-11), widening 12-13 and 14-15 (FEW: and 6-7, 8-9)
    const int pipe = warp < 4 ? warp >> 1 : warp < 12 ? (warp - 4) >> 2 : (warp - 12) >> 1;
    const bool spare = FEW && warp >= 6 && warp < 10;
    uint64_t *const bars = reinterpret_cast<uint64_t *>(smem + L::BAR) + pipe * L::NBARS;
    uint64_t *const u_full = bars, *const u_empty = u_full + NU, *const q_full = u_empty + NU, *const q_empty = q_full + 1,
                    *const qc_full = q_empty + 1, *const t_full = qc_full + 1, *const t_empty = t_full + NS,
                    *const c_full = t_empty + NS,
                    *const c_empty = c_full + (NC ? NC : 1), *const s_full = c_empty + (NC ? NC : 1), *const p_full = s_full + 1,
                    *const o_full = p_full + 1, *const o_free = o_full + 1, *const fin = o_free + 1;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + L::MISC);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(smem + L::MISC + 4);
    StreamUnit *const slots = reinterpret_cast<StreamUnit *>(smem + L::UNITS) + pipe * NU;
    int8_t *const q_exp = reinterpret_cast<int8_t *>(smem + L::EXP) + pipe * 2 * BM;
    uint8_t *const q_tile = smem + L::Q + (FEW ? 0 : pipe * L::Q_TILE); // as the MMA reads it
    const int row_off = FEW ? pipe * 64 : 0;                            // the pipeline's first row in it
    uint8_t *const ring = smem + L::T0 + pipe * NS * L::TILE;
    uint8_t *const codes = smem + L::C0 + pipe * NC * L::CODE;

    if (threadIdx.x == 0) {
        for (int p = 0; p < 2; ++p) {
            uint64_t *b = reinterpret_cast<uint64_t *>(smem + L::BAR) + p * L::NBARS;
            for (int s = 0; s < NU; ++s) mbar_init(b++, 1);
            for (int s = 0; s < NU; ++s) mbar_init(b++, 1 + L::kSoftmax + L::kWiden); // the issuer's, too
            mbar_init(b++, 1);                                                        // Q full
            mbar_init(b++, 1);                                                        // Q empty
            mbar_init(b++, KV8 ? L::kWiden : 1);                                      // Q as fp16
            for (int s = 0; s < NS; ++s) mbar_init(b++, KV8 ? L::kWiden : 1);         // tile landed, or widened
            for (int s = 0; s < NS; ++s) mbar_init(b++, 1);
            for (int s = 0; s < (NC ? NC : 1); ++s) mbar_init(b++, 1);                // codes landed
            for (int s = 0; s < (NC ? NC : 1); ++s) mbar_init(b++, KV8 ? L::kWiden : 1); // codes read
            mbar_init(b++, 1);                                                        // S full
            mbar_init(b++, L::kSoftmax);                                              // P full
            mbar_init(b++, 1);                                                        // O full
            mbar_init(b++, L::kSoftmax);                                              // O free
            mbar_init(b++, 1);                                                        // end
        }
        *abort_flag = 0;
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
    pdl_wait(); // from here on global memory that the stream's earlier kernels wrote is read
    if (a.few_rows > 0) pdl_trigger(); // (few_kernel reads what the list's launch, too, had waited for)

    const int G = 1 << a.lg_group;
    auto fail = [&]() {
        set_error(a.err, PKV_DEVERR_TIMEOUT);
        *abort_flag = 1;
    };
    auto take = [&](int n) -> bool { return __all_sync(0xffffffffu, mbar_wait_hint(u_full + n % NU, (n / NU) & 1)); };
    auto give = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(u_empty + n % NU);
    };

    // ---------------------------------------------------------------- widening (E4M3)
    // A row of every tile a thread (two, where there are two warps), K and V in turn as they are loaded, and of every bf16 Q tile.
    auto widen_tiles = [&]() {
        if constexpr (KV8) {
            constexpr int kThreads = L::kWiden * 32;
            const int r = ((warp & 1) + (spare ? 2 : 0)) * 32 + lane;
            bool ok = true;
            int nt = 0, nq = 0; // tiles, Q tiles so far
            auto widen = [&]() -> bool {
                const int cs = nt % NC, st = nt % NS;
                bool w = mbar_wait_hint(c_full + cs, (nt / NC) & 1);
                if (w && nt >= NS) w = mbar_wait_hint(t_empty + st, (nt / NS - 1) & 1);
                if (!__all_sync(0xffffffffu, w)) return false;
#pragma unroll 1
                for (int x = r; x < BN; x += kThreads) widen_codes<D>(codes + cs * L::CODE, ring + st * L::TILE, x);
                fence_proxy_async_smem(); // the MMAs read the tile through the async proxy
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(c_empty + cs);
                    mbar_arrive(t_full + st);
                }
                ++nt;
                return true;
            };
            for (int n = 0; ok; ++n) {
                ok = take(n);
                if (!ok) break;
                const int tiles = slots[n % NU].n;
                if (tiles < 0) break;
                for (int j = 0; j < tiles && ok; ++j) {
                    ok = widen();
                    if (SCALE_Q && ok && j == 0) {
                        ok = __all_sync(0xffffffffu, mbar_wait_hint(q_full, nq & 1));
                        if (!ok) break;
#pragma unroll 1
                        for (int x = r; x < kRows; x += kThreads) q_exp[(nq & 1) * BM + row_off + x] = (int8_t)q_to_f16<D>(q_tile, row_off + x);
                        ++nq;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(qc_full);
                    }
                    ok = ok && widen();
                }
                give(n);
                if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
            }
            if (!ok && lane == 0) fail();
        }
    };

    if constexpr (KV8) { // 128 x (80 + 2 x 176 + 80) = 512 x 128 registers
        if (warp < 4 || warp >= 12) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    } else { // 128 x (104 + 2 x 200) <= 384 x 168
        if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    }
    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------------- loader
        // Lane l loads block l of each tile, one box (16-bit, D = 64: 64 dims x bs rows; E4M3: bs rows of codes).  K: every
        // usable block whole (the softmax masks what is not seen); V: blocks whose every row is seen by some row, the others' rows with plain
        // stores, zeros where no row may look (P is 0 there, but 0 NaN is NaN, and unused slots may hold anything).
        constexpr int CPR = D * EB / 16, RPI = 32 / CPR; // 16-byte chunks per pool row, rows per warp instruction
        const int cc = lane % CPR, rsub = lane / CPR, nbt = BN >> a.lg_bs;
        if (lane == 0) {
            tc::prefetch_tmap(&tq);
            tc::prefetch_tmap(&tp);
        }
        const bool direct = a.plan == nullptr;
        const int total = direct ? a.rect : a.plan[0] * a.hkv;
        int at = blockIdx.x + pipe * gridDim.x; // direct: the next place to look at
        int nt = 0, nq = 0;                     // tiles (or their codes) and Q tiles loaded so far
        bool ok = true;
        auto publish = [&](int n) {
            if (n >= NU && !__all_sync(0xffffffffu, mbar_wait_hint(u_empty + n % NU, (n / NU - 1) & 1))) {
                ok = false;
                return;
            }
            int4 raw = make_int4(-1, 0, 0, 0);
            if (lane == 0 && !*abort_flag) {
                if (direct) {
                    raw = direct_unit(a, at, 2 * gridDim.x);
                } else {
                    const int idx = atomicAdd(a.plan + 1, 1);
                    if (idx < total) {
                        raw = reinterpret_cast<const int4 *>(a.plan + 4)[idx / a.hkv];
                        raw.w = idx % a.hkv;
                    }
                }
            }
            raw.x = __shfl_sync(0xffffffffu, raw.x, 0);
            raw.y = __shfl_sync(0xffffffffu, raw.y, 0);
            raw.z = __shfl_sync(0xffffffffu, raw.z, 0);
            raw.w = __shfl_sync(0xffffffffu, raw.w, 0);
            const StreamUnit u = stream_unit(a, raw.x, raw.y, raw.z, raw.w);
            if (lane == 0) {
                slots[n % NU] = u;
                mbar_arrive(u_full + n % NU);
                if (u.n > 0 && n > 0)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) tc::tma_prefetch_3d(&tq, c * 64, u.h * G, u.row0);
            }
            __syncwarp(); // this warp reads the slot, too
        };
        for (int n = -1; ok; ++n) { // (a round before unit 0 publishes it and does nothing else)
            const StreamUnit *const u = slots + (n < 0 ? 0 : n % NU);
            const int tiles = n < 0 ? 0 : u->n;
            if (tiles < 0) break;
            const int h = u->h, k0 = u->k0, kend = u->kend, lo = u->lo, hi = u->hi, from = u->from;
            const int32_t *const trow = a.tables + (int64_t)u->trow * a.max_blocks;
            const int skip = u->hidden >> a.lg_bs;
            // lane l's table entry of block l of key tile j
            auto entry = [&](int j) -> int {
                const int lb = ((k0 + j * BN) >> a.lg_bs) + lane;
                return lane < nbt && (lb << a.lg_bs) < kend ? trow[lb + (lb >= from ? skip : 0)] : -1;
            };
            auto load = [&](bool isV, int j, int b) {
                constexpr int N = KV8 ? NC : NS;
                const int st = nt % N, round = nt / N;
                uint64_t *const full = (KV8 ? c_full : t_full) + st, *const empty = (KV8 ? c_empty : t_empty) + st;
                uint8_t *const stage = KV8 ? codes + st * L::CODE : ring + st * L::TILE;
                if (round > 0) ok = __all_sync(0xffffffffu, mbar_wait_hint(empty, (round - 1) & 1));
                if (!ok || __any_sync(0xffffffffu, *abort_flag != 0)) {
                    ok = false;
                    return;
                }
                ++nt;
                const int kbase = k0 + j * BN, lb = (kbase >> a.lg_bs) + lane;
                const bool has = lane < nbt && (lb << a.lg_bs) < kend;
                const bool good = has && b >= 0 && b < a.num_blocks;
                if (isV && has && !good) set_error(a.err, PKV_DEVERR_BLOCK_ID);
                const bool whole = good && (!isV || (((lb + 1) << a.lg_bs) <= kend &&
                                                     ((lb << a.lg_bs) >= hi || ((lb + 1) << a.lg_bs) <= lo)));
                const unsigned mask = __ballot_sync(0xffffffffu, whole);
                if (lane == 0) mbar_expect_tx(full, (uint32_t)__popc(mask) * (uint32_t)(a.bs * D * EB));
                __syncwarp();
                if (whole) {
                    const int y = ((b * 2 + (isV ? 1 : 0)) * a.hkv + h) << a.lg_bs;
                    if constexpr (KV8)
                        tc::tma_load_2d(stage + (lane << a.lg_bs) * D, &tp, 0, y, full);
                    else if constexpr (GROUPED)
                        tc::tma_load_4d(stage + (lane << a.lg_bs) * 256, &tp, 0, 0, 0, y >> 3, full);
                    else
                        tc::tma_load_2d(stage + (lane << a.lg_bs) * 128, &tp, 0, y, full);
                }
                if (isV) {
                    const unsigned all = nbt == 32 ? 0xffffffffu : (1u << nbt) - 1u;
                    for (int r0 = 0; mask != all && r0 < BN; r0 += RPI) {
                        const int r = r0 + rsub, l = r >> a.lg_bs;
                        const int bl = __shfl_sync(0xffffffffu, good ? b : -1, l);
                        if ((mask >> l) & 1u) continue;
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (bl >= 0 && kbase + r < kend && !(kbase + r >= lo && kbase + r < hi))
                            x = *reinterpret_cast<const uint4 *>(a.pool + ((((int64_t)bl * 2 + 1) * a.hkv + h) * a.tile_elems +
                                                                           (int64_t)(r - (l << a.lg_bs)) * D) * EB + cc * 16);
                        if constexpr (KV8) {
                            *reinterpret_cast<uint4 *>(stage + r * D + cc * 16) = x;
                        } else {
                            uint8_t *row = GROUPED ? stage + (r >> 3) * 2048 + (cc >> 3) * 1024 + (r & 7) * 128 : stage + r * 128;
                            *reinterpret_cast<uint4 *>(row + (((cc & 7) ^ (r & 7)) << 4)) = x;
                        }
                    }
                    if constexpr (!KV8) fence_proxy_async_smem(); // the plain stores are read by the MMA
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            };
            auto load_q = [&]() {
                if (nq > 0) ok = __all_sync(0xffffffffu, mbar_wait_hint(q_empty, (nq - 1) & 1));
                if (!ok) return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, kRows * D * 2);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        tc::tma_load_3d(q_tile + c * BM * 128 + row_off * 128, &tq, c * 64, h * G, u->row0, q_full);
                }
                __syncwarp();
                ++nq;
            };
            // K and V of tile j; Q behind the first K tile; the next unit published behind the second tile (the loads in flight
            // hide the reads that it takes)
            int e = tiles > 0 ? entry(0) : -1;
            for (int j = 0; ok; ++j) {
                if (j == min(tiles, 2)) {
                    publish(n + 1);
                    if (!ok) break;
                }
                if (j >= tiles) {
                    if (j >= 2) break;
                    continue;
                }
                const int e_next = j + 1 < tiles ? entry(j + 1) : -1;
                load(false, j, e);
                if (j == 0 && ok) load_q();
                if (ok) load(true, j, e);
                e = e_next;
            }
            if (!ok || __any_sync(0xffffffffu, *abort_flag != 0)) {
                if (!ok && lane == 0) fail();
                break;
            }
        }
        // the last loads must land before this CTA's shared memory goes away
        if (lane == 0) {
            constexpr int N = KV8 ? NC : NS;
            bool w = true;
            for (int c = max(nt - N, 0); c < nt; ++c) w = w && mbar_wait_hint((KV8 ? c_full : t_full) + c % N, (c / N) & 1);
            if (nq > 0) w = w && mbar_wait_hint(q_full, (nq - 1) & 1);
            if (!w) set_error(a.err, PKV_DEVERR_TIMEOUT);
        }
    } else if (warp == 1 || warp == 3) {
        // ---------------------------------------------------------------- MMA issuer
        // S(0), then per key tile j: P V(j), S(j + 1).  S(j + 1) follows P V(j) from the same thread, so it overwrites the
        // S columns only after P V(j) has read P from them.
        constexpr uint32_t IQK = tc::idesc_f16(OT == PKV_BF16 ? 1u : 0u, 0u, BM, BN);
        constexpr uint32_t IPV = tc::idesc_f16(OT == PKV_BF16 ? 1u : 0u, 1u, BM, D);
        const uint64_t dQ = tc::smem_desc(smem_u32(q_tile), 16, 1024);
        const uint64_t dK = tc::smem_desc(smem_u32(ring), 16, GROUPED ? 2048 : 1024);
        const uint64_t dV = GROUPED ? tc::smem_desc(smem_u32(ring), 1024, 2048) : tc::smem_desc(smem_u32(ring), BN * 128, 1024);
        constexpr int kHalf = GROUPED ? 1024 : BN * 128, kKeys16 = GROUPED ? 4096 : 2048;
        const uint32_t tS = tmem + (uint32_t)(pipe * BN), tO = tmem + (uint32_t)(2 * BN + pipe * D);
        uint64_t *const q_ready = SCALE_Q ? qc_full : q_full;
        bool any_mma = false, ok = true;
        int nt = 0, nq = 0, no = 0, np = 0; // tiles before the unit's; Q tiles, O tiles, P tiles so far
        for (int n = 0; ok; ++n) {
            ok = take(n);
            if (!ok) break;
            const int tiles = slots[n % NU].n;
            if (tiles < 0) break;
            // K(j) is tile nt + 2 j of the ring, V(j) the next one
            auto landed = [&](int c) { return mbar_wait(t_full + c % NS, (c / NS) & 1); };
            auto issue_s = [&](int j) {
                const int st = (nt + 2 * j) % NS;
                const uint64_t b0 = dK + (uint64_t)((st * L::TILE) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_f16_warp(tS, dQ + (uint64_t)(((k >> 2) * BM * 128 + (k & 3) * 32) >> 4),
                                     b0 + (uint64_t)(((k >> 2) * kHalf + (k & 3) * 32) >> 4), IQK, k > 0 ? 1u : 0u);
                tc::commit_warp(s_full);
                tc::commit_warp(t_empty + st);
                if (j + 1 == tiles) tc::commit_warp(q_empty);
            };
            if (tiles > 0) {
                ok = __all_sync(0xffffffffu, landed(nt) && mbar_wait(q_ready, nq & 1));
                ++nq;
                if (!ok) break;
                tc::fence_after_sync();
                any_mma = true;
                issue_s(0);
            }
            for (int j = 0; j < tiles && ok; ++j) {
                const bool more = j + 1 < tiles;
                // (three stages: the next K tile is normally in place already, and S(j + 1) goes out right behind P V(j); two: its
                // stage may still be this S's)
                bool w = (NS == 2 || !more || landed(nt + 2 * j + 2)) && landed(nt + 2 * j + 1) && mbar_wait(p_full, np & 1);
                if (j == 0 && no > 0) w = w && mbar_wait(o_free, (no - 1) & 1); // the unit before has been read out of O
                ok = __all_sync(0xffffffffu, w);
                if (!ok) break;
                ++np;
                tc::fence_after_sync();
                const int st = (nt + 2 * j + 1) % NS;
                const uint64_t b0 = dV + (uint64_t)((st * L::TILE) >> 4);
#pragma unroll
                for (int part = 0; part < NP; ++part)
#pragma unroll
                    for (int k = 0; k < BN / 16; ++k)
                        tc::mma_f16_ts_warp(tO, tS + (uint32_t)(part * (BN / 2) + k * 8), b0 + (uint64_t)((k * kKeys16) >> 4), IPV,
                                            (j > 0 || k > 0 || part > 0) ? 1u : 0u);
                tc::commit_warp(t_empty + st);
                if (!more) {
                    tc::commit_warp(o_full);
                    ++no;
                } else {
                    if (NS == 2) {
                        ok = __all_sync(0xffffffffu, landed(nt + 2 * j + 2));
                        if (!ok) break;
                        tc::fence_after_sync();
                    }
                    issue_s(j + 1);
                }
            }
            nt += 2 * tiles;
            give(n);
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        }
        if (!ok && lane == 0) fail();
        // every MMA issued by this warp has completed before tensor memory is released
        if (any_mma) {
            tc::commit_warp(fin);
            if (!__all_sync(0xffffffffu, mbar_wait_hint(fin, 0)) && lane == 0) set_error(a.err, PKV_DEVERR_TIMEOUT);
        }
    } else if (warp >= 12) {
        widen_tiles();
    } else {
        if constexpr (KV8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ---------------------------------------------------------------- softmax, one thread per row
        if (spare) { // (registers go to a warpgroup's warps alike, hence only here)
            widen_tiles();
        } else {
        const int tile_row = (warp & 3) * 32 + lane, r = tile_row - row_off; // row of the tile = tensor-memory lane; of the unit
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + (uint32_t)(pipe * BN), tO = tmem + lane_off + (uint32_t)(2 * BN + pipe * D);
        using T = typename ModelT<MT>::T;
        bool ok = true;
        int ns = 0, no = 0; // S tiles, O tiles so far (units with keys)
        for (int n = 0; ok; ++n) {
            ok = take(n);
            if (!ok) break;
            const StreamUnit *const u = slots + n % NU;
            const int tiles = u->n;
            if (tiles < 0) break;
            const int h = u->h, ntok = u->ntok, rows = ntok << a.lg_group, tok = r >> a.lg_group;
            const bool mine = r >= 0 && r < rows; // a row of the unit
            const int first = (warp & 3) * 32 - row_off;
            const bool live = first + 31 >= 0 && first < rows; // some row of this warp is
            // the row's place in q and out
            const int64_t row = (int64_t)(u->row0 + tok) * a.hq + h * G + (r & (G - 1));
            if (tiles == 0) {
                if (mine) { // rows that see no key
                    uint4 *orow = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * D);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0u, 0u, 0u, 0u);
                }
            } else if (!live) {
                for (int j = 0; j < tiles && ok; ++j, ++ns) {
                    ok = __all_sync(0xffffffffu, mbar_wait_hint(s_full, ns & 1));
                    if (ok && lane == 0) mbar_arrive(p_full);
                }
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait_hint(o_full, no & 1));
                if (!ok) break;
                ++no;
                if (lane == 0) mbar_arrive(o_free);
            } else {
                const int qpos = u->qpos0 + tok, plast = u->qpos0 + ntok - 1, hidden = u->hidden, qfirst = u->qpos0;
                float sl = KV8 ? a.scale_log2 * a.k_scale[h] : a.scale_log2;
                float m_use = -INFINITY, l = 0.f;
                int kbase = u->k0;
                for (int j = 0; j < tiles && ok; ++j, kbase += BN) {
                    ok = __all_sync(0xffffffffu, mbar_wait(s_full, ns & 1));
                    if (!ok) break;
                    ++ns;
                    tc::fence_after_sync();
                    if constexpr (SCALE_Q) {
                        // q's power of two: S is complete, so the row is converted; the next but one Q tile, which writes this
                        // slot again, waits for the next one's S, and that for this row's P
                        if (j == 0) sl *= exp2f((float)q_exp[(no & 1) * BM + tile_row]);
                    }
                    uint32_t sr[BN];
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) tc::ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
                    tc::wait_ld();
                    // seen key kbase + c is at most this row's position up to c = upto - 1, inside its window from c = since on,
                    // a sink below c = sink; only tiles on either edge of some row's sight
                    if (kbase + BN - 1 + hidden > qfirst || (a.window > 0 && plast - a.window + 1 - hidden > kbase)) {
                        const int upto = qpos + 1 - hidden - kbase;
                        const int since = a.window > 0 ? qpos - a.window + 1 - hidden - kbase : 0;
                        const int sink = min(a.sinks, qpos + 1) - kbase;
#pragma unroll
                        for (int w = 0; w < BN / 32; ++w) {
                            const uint32_t in = (ones_below(upto - 32 * w) & ~ones_below(since - 32 * w)) | ones_below(sink - 32 * w);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(in & (1u << c))) sr[32 * w + c] = 0xFF800000u; // -inf
                        }
                    }
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
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tc::ld16(tO + c * 16, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tc::st16(tO + c * 16, o);
                        }
                    }
                    float2 rs = make_float2(0.f, 0.f);
                    const float2 sc2 = make_float2(sl, sl), nb2 = make_float2(nbase, nbase);
                    // P over the S columns: packed pairs, key c in column c / 2 (bf16: lo parts from BN / 2)
                    constexpr int KC = NP == 2 ? 16 : 32;
#pragma unroll
                    for (int q = 0; q < BN / KC; ++q) {
                        uint32_t phi[KC / 2], plo[NP == 2 ? KC / 2 : 1];
#pragma unroll
                        for (int c = 0; c < KC / 2; ++c) {
                            const int k = q * KC + 2 * c;
                            const float2 xx = fma2(make_float2(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), sc2, nb2);
                            const float p0 = fast_exp2(xx.x), p1 = fast_exp2(xx.y);
                            rs = add2(rs, make_float2(p0, p1));
                            phi[c] = pack2(p0, p1, OT);
                            if constexpr (NP == 2) // remainders after bf16 rounding, themselves rounded to bf16
                                plo[c] = pack2(p0 - __uint_as_float(phi[c] << 16), p1 - __uint_as_float(phi[c] & 0xFFFF0000u), OT);
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
                    if (lane == 0) mbar_arrive(p_full);
                }
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait_hint(o_full, no & 1));
                if (!ok) break;
                ++no;
                tc::fence_after_sync();
                const float vs = KV8 ? a.v_scale[h] : 1.f;
                uint32_t o[D]; // the whole row in one tensor-memory round trip
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tc::ld32(tO + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[c * 32]));
                tc::wait_ld();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(o_free); // O has been read; the next unit's first P V may overwrite it
                if (mine && u->nsplit > 1) {
                    // fp32 partial: unnormalised o, and (m, l) with m the row's base in log2 units
                    const int64_t idx = row * a.max_splits + u->split;
                    float4 *dst = reinterpret_cast<float4 *>(a.ws_o + idx * D);
#pragma unroll
                    for (int e = 0; e < D / 4; ++e)
                        dst[e] = make_float4(__uint_as_float(o[4 * e]) * vs, __uint_as_float(o[4 * e + 1]) * vs,
                                             __uint_as_float(o[4 * e + 2]) * vs, __uint_as_float(o[4 * e + 3]) * vs);
                    reinterpret_cast<float2 *>(a.ws_ml)[idx] = make_float2(m_use, l);
                } else if (mine) {
                    const float inv = l == 0.f ? 0.f : vs / l; // (a row may see no key)
                    uint4 *orow = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * D);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack2(__uint_as_float(o[8 * c + 2 * e]) * inv, __uint_as_float(o[8 * c + 2 * e + 1]) * inv, MT);
                        orow[c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            give(n);
            if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        }
        if (!ok && lane == 0) fail();
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// launch of one instantiation (chunk_stream_*.cu)
template <int D, int MT, bool KV8, bool FEW>
cudaError_t launch_stream(const CUtensorMap &q, const CUtensorMap &pool, const Args &a, int grid, cudaStream_t st) {
    auto kern = stream_kernel<D, MT, KV8, FEW>;
    const int smem = StreamLayout<D, KV8, FEW>::TOTAL;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return pdl_launch(kern, dim3((unsigned)grid), dim3(stream_threads<KV8>()), smem, st, q, pool, a);
}
template <bool KV8, bool FEW>
cudaError_t launch_stream_any(int D, int mt, const CUtensorMap &q, const CUtensorMap &pool, const Args &a, int grid,
                              cudaStream_t st); // (one translation unit each)

#define PKV_STREAM_INSTANTIATE(KV8, FEW)                                                                               \
    template <>                                                                                                        \
    cudaError_t launch_stream_any<KV8, FEW>(int D, int mt, const CUtensorMap &q, const CUtensorMap &pool, const Args &a, \
                                            int grid, cudaStream_t st) {                                               \
        if (D == 128)                                                                                                  \
            return mt == PKV_BF16 ? launch_stream<128, PKV_BF16, KV8, FEW>(q, pool, a, grid, st)                       \
                                  : launch_stream<128, PKV_F16, KV8, FEW>(q, pool, a, grid, st);                       \
        return mt == PKV_BF16 ? launch_stream<64, PKV_BF16, KV8, FEW>(q, pool, a, grid, st)                            \
                              : launch_stream<64, PKV_F16, KV8, FEW>(q, pool, a, grid, st);                            \
    }

} // namespace pkv_prefill
