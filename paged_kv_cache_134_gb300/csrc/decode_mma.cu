// Host side of the matrix-instruction decodes (decode_int4.cuh, decode_mma.cuh): split size, workspace, launches.
#include "mma_common.cuh"

#include <algorithm>

namespace {

constexpr int kMaxSplit = 1024; // tokens

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// resident CTAs of the kernels of units
int64_t workers_of(const pkv_cache *c, int group) {
    const bool few = c->head_dim == 128 && group == 8; // Geo4::kCtas
    return (int64_t)c->num_sms * (c->kv_dtype == PKV_INT4 ? (few ? 3 : 4) : c->kv_dtype == PKV_FP8_E4M3 ? 3 : 2);
}

// sequences of a launch: over 16-bit caches the list of more would leave room for one CTA an SM instead of two
int most_seqs(const pkv_cache *c) {
    return c->kv_dtype == PKV_INT4 || c->kv_dtype == PKV_FP8_E4M3 ? pkv_mma::kMaxSeqs : 384;
}

// What one launch of at most `seqs` sequences looks like.
struct Plan {
    int64_t cap;    // tokens a sequence may have
    int split, max_splits, seqs;
    int64_t floats; // workspace
    bool is_short;  // a warp a row
};

bool plan_for(const pkv_cache *c, int num_seqs, int hq, int max_blocks, int64_t mass_len, Plan *p) {
    const bool mass = mass_len >= 0;
    p->cap = (int64_t)max_blocks * c->block_size;
    if (mass) p->cap = std::min(p->cap, mass_len);
    const bool i4 = c->kv_dtype == PKV_INT4;
    const int64_t workers = workers_of(c, hq / c->num_kv_heads);
    const int most = most_seqs(c);
    const int64_t rows = (int64_t)std::min(num_seqs, most) * c->num_kv_heads;
    // Short rows by a warp each, where two of three speak for it: the mass (which saves a launch), up to four heads (a
    // warp's work), more rows than CTAs.  4-bit, D = 128: 8 rows of four heads and 16 tokens, 5.4 us with mass
    // (units: 8.0), 5.7 without (5.1); 256 rows of eight heads and 32 tokens, 15.7 us with mass (9.4); many rows see
    // decode_short.cuh.
    p->is_short = p->cap <= pkv_mma::kShortTokens &&
                  (int)mass + (hq / c->num_kv_heads <= 4) + (rows > workers) >= 2;
    if (p->is_short) {
        p->split = p->max_splits = 1;
        p->seqs = (int)std::min<int64_t>(num_seqs, 0x7FFFFFFF / c->num_kv_heads);
        p->floats = 0;
        return true;
    }
    // Tokens of a split, a function of the call's shapes, never of the lengths (a result does not change with the other
    // sequences' lengths).  More than four waves of the largest: those, which have the least fixed costs (4-bit, 32
    // sequences of up to 4096 tokens and 256 of up to 8192: 59 and 61 us; 864 takes 3 more of both, 512 9 and 15).
    // Else the one with the least time at the table's full width by a model of it: waves of units, each of
    // so many rounds of the warps' tiles and a fixed part, and what joins the splits.  4-bit: rounds of 2.1 us, 1.2 a
    // unit, 3 for the last CTA's join, 5 for a merge launch; where a CTA has several units one warp prepares the next and
    // takes a tile less.  (Against two units per CTA, at least 64 tokens, over a hundred batches of 1 to 256
    // sequences: 0.5 to 1.1 of the time, 6 % less on average; one sequence of 131071 tokens 38.0 -> 37.1 us.)
    const int tile = i4 ? 32 : 16, round = 4 * tile;
    int64_t split = kMaxSplit;
    if (rows * ((p->cap + kMaxSplit - 1) / kMaxSplit) <= 4 * workers) {
        double least = 0.;
        for (int64_t k = i4 ? 1 : 2; k <= 2 * kMaxSplit / round; k += i4 ? 1 : 2) { // whole rounds, or a tile less
            const int64_t t = (k + 1) / 2 * round - (k % 2 ? tile : 0);
            const int64_t splits = std::max<int64_t>(1, (p->cap + t - 1) / t), units = rows * splits;
            if (units > 2 * workers + rows) continue; // (keeps the workspace within decode_mma_workspace_floats)
            const int64_t tiles = (std::min(t, p->cap) + tile - 1) / tile;
            const int64_t rounds = i4 && units > workers ? 1 + tiles / 4 : (tiles + 3) / 4;
            const double join = mass || splits == 1 ? 0. : splits <= pkv_mma::kJoinSplits ? 3. : 5.;
            const double time = (double)((units + workers - 1) / workers) * ((i4 ? 2.1 : 1.1) * rounds + (i4 ? 1.2 : 3.)) + join;
            if (least == 0. || time < least) {
                least = time;
                split = t;
            }
            if (splits == 1) break;
        }
    }
    split = std::max(split, round_up((p->cap + 1023) / 1024, 64));
    if (split / c->block_size > (i4 ? 1024 : 8192)) return false; // the split's table entries no longer fit shared memory
    p->split = (int)split;
    p->max_splits = (int)std::max<int64_t>(1, (p->cap + split - 1) / split);
    // (with mass a row of one split keeps its (m, l) too)
    const int64_t partials = p->max_splits > 1 || mass ? (int64_t)hq * p->max_splits * (c->head_dim + 2) : 0;
    const int64_t per_seq = partials + (mass ? (int64_t)hq * p->cap : 0);
    // ... and at most 2 GB of workspace unless one sequence needs more
    int64_t n = std::min(num_seqs, most);
    if (per_seq > 0) n = std::max<int64_t>(1, std::min<int64_t>(n, ((int64_t)1 << 29) / per_seq));
    p->seqs = (int)n;
    p->floats = n * per_seq;
    return true;
}

cudaError_t run_short(const pkv_cache *c, const pkv_mma::Args &a, cudaStream_t st) {
    const int mt = c->model_dtype, D = c->head_dim;
    if (c->kv_dtype == PKV_INT4) return pkv_short_int4(a, mt, D, st);
    return c->kv_dtype == PKV_FP8_E4M3 ? pkv_short_fp8(a, mt, D, st) : pkv_short_16bit(a, mt, D, st);
}

__global__ void clear_kernel(int *done, int n) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) done[i] = 0;
}

cudaError_t run(const pkv_cache *c, const pkv_mma::Args &a, bool mass, bool merge, cudaStream_t st) {
    const int mt = c->model_dtype, D = c->head_dim, sms = c->num_sms;
    if (!mass) return pkv_mma_int4(a, mt, D, sms, merge, st);
    if (c->kv_dtype == PKV_INT4) return pkv_mma_int4_mass(a, mt, D, sms, merge, st);
    if (c->kv_dtype == PKV_FP8_E4M3) return pkv_mma_fp8_mass(a, mt, D, sms, merge, st);
    return pkv_mma_16bit_mass(a, mt, D, sms, merge, st);
}

} // namespace

int64_t decode_mma_workspace_floats(const pkv_cache *c, int num_seqs, int hq, int max_blocks, int64_t mass_len) {
    // units of one launch: at most two waves and one more a row, or those of the largest split; with mass the scores
    // besides.  2 GB, unless one sequence (of at most 1024 splits) needs more.
    if (num_seqs <= 0 || hq <= 0) return 0;
    const int64_t seqs = std::min(num_seqs, most_seqs(c)), rows = seqs * c->num_kv_heads;
    int64_t cap = (int64_t)max_blocks * c->block_size, scores = 0; // of a sequence
    if (mass_len >= 0) {
        cap = std::min(cap, mass_len);
        scores = hq * cap;
    }
    const int64_t units = std::max(rows * ((cap + kMaxSplit - 1) / kMaxSplit), 2 * workers_of(c, 1) + rows);
    const int64_t row = std::max<int64_t>(hq / c->num_kv_heads, 1) * (c->head_dim + 2);
    return std::min(units * row + seqs * scores,
                    std::max<int64_t>((int64_t)1 << 29, 1024 * row * c->num_kv_heads + scores));
}

int decode_mma_entry(pkv_cache *c, const MmaDecodeLaunch &d, const PkvWorkspace *fixed, cudaStream_t st) {
    Plan p;
    if (!plan_for(c, d.num_seqs, d.num_q_heads, d.max_blocks, d.mass_len, &p))
        return pkv_fail(PKV_EUNSUPPORTED, "tables of %d blocks are wider than this decode takes", d.max_blocks);
    // a batch larger than one launch takes runs in consecutive launches that share the workspace: each
    // waits for the one before it.  Another host thread's call on this stream may use the same workspace, or replace
    // it: none of its own launches comes between this call's.
    std::lock_guard<std::mutex> lk(c->ws_mu);
    PkvWorkspace ws;
    if (!fixed) {
        if (int r = pkv_stream_workspace(c, st, p.floats, &ws)) return r;
    } else if (p.floats > fixed->floats) {
        return pkv_fail(PKV_EINVAL,
                        "no-alloc decode needs %lld bytes of scratch for %d sequences x %d query heads x %d splits; "
                        "its fixed scratch holds %lld bytes (use fewer sequences per call or paged_decode_attention)",
                        (long long)(p.floats * 4), p.seqs, d.num_q_heads, p.max_splits, (long long)(fixed->floats * 4));
    } else {
        ws = *fixed;
    }
    // few splits: the CTA that finishes a row last joins them (no second launch); many: merge_kernel
    const bool mass = d.mass_len >= 0;
    const bool join = !mass && p.max_splits <= pkv_mma::kJoinSplits && (int64_t)p.seqs * c->num_kv_heads <= ws.counters;
    pkv_mma::Args a;
    a.pool = static_cast<const char *>(c->pool);
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.err = c->err;
    a.num_blocks = c->num_blocks;
    pkv_row_strides(c, &a.blk_stride, &a.head_stride, &a.v_off);
    if (a.blk_stride > 0xFFFFFFFFll)
        return pkv_fail(PKV_EUNSUPPORTED, "blocks of %lld bytes are larger than this decode takes", (long long)a.blk_stride);
    a.mass_len = d.mass_len;
    a.cap = p.cap;
    a.max_blocks = d.max_blocks;
    a.hq = d.num_q_heads;
    a.hkv = c->num_kv_heads;
    a.group = d.num_q_heads / c->num_kv_heads;
    {
        int s = 0;
        while (((int64_t)1 << s) < a.hkv) ++s;
        a.hkv_shift = 31 + s;
        a.hkv_magic = (uint32_t)((((uint64_t)1 << a.hkv_shift) + a.hkv - 1) / a.hkv);
    }
    a.bs_log2 = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
    a.split_tokens = p.split;
    a.max_splits = p.max_splits;
    a.qk_scale_log2 = d.scale * 1.4426950408889634f;
    a.decay = d.decay;
    for (int s0 = 0; s0 < d.num_seqs; s0 += p.seqs) {
        const int n = std::min(p.seqs, d.num_seqs - s0);
        const int64_t rows = (int64_t)n * d.num_q_heads * (p.max_splits > 1 || mass ? p.max_splits : 0);
        const int64_t row_bytes = (int64_t)d.num_q_heads * c->head_dim * 2;
        a.q = static_cast<const char *>(d.q) + s0 * row_bytes;
        a.out = static_cast<char *>(d.out) + s0 * row_bytes;
        a.tables = d.tables ? d.tables + (int64_t)s0 * d.max_blocks : nullptr;
        a.lens = d.lens + s0;
        a.num_seqs = n;
        a.ws_o = ws.p;
        a.ws_ml = ws.p + rows * c->head_dim;
        a.ws_x = ws.p + rows * (c->head_dim + 2);
        a.done = join ? ws.done : nullptr;
        a.mass = mass ? d.mass + (int64_t)s0 * c->num_kv_heads * d.mass_len : nullptr;
        cudaError_t e;
        // The last launch left the counters at zero, but where its work may have met another's against the contract (the
        // fixed scratch; executables of one capture) a call does not rely on that: the damage would outlast both.
        // (0.6 to 1.1 us; joined by merge_kernel instead, without counters, the 7B batch takes 70 us for 59.)
        if (join && ws.clear) {
            const int counters = n * c->num_kv_heads;
            g_pkv_launches++;
            e = pdl_launch(clear_kernel, dim3((counters + 255) / 256), dim3(256), 0, st, ws.done, counters);
            if (e != cudaSuccess) return pkv_cuda_fail(e, "decode launch");
        }
        {
            PkvTimer timer(c, PKV_KIND_DECODE, st);
            g_pkv_launches++;
            e = p.is_short ? run_short(c, a, st) : run(c, a, mass, false, st);
        }
        if (e != cudaSuccess) return pkv_cuda_fail(e, "decode launch");
        if (!p.is_short && (mass || (p.max_splits > 1 && !join))) {
            PkvTimer timer(c, PKV_KIND_MERGE, st);
            g_pkv_launches++;
            e = run(c, a, mass, true, st);
        }
        if (e != cudaSuccess) return pkv_cuda_fail(e, "decode merge launch");
    }
    return PKV_OK;
}
