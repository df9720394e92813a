// Host side of the matrix-instruction decodes (decode_int4.cuh, decode_mma.cuh): split size, workspace, launches.
#include "mma_common.cuh"

#include <algorithm>

namespace {

constexpr int kMaxSplit = 1024; // tokens

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

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
    const int64_t workers = (int64_t)c->num_sms * (i4 ? 4 : c->kv_dtype == PKV_FP8_E4M3 ? 3 : 2);
    const int64_t rows = (int64_t)std::min(num_seqs, pkv_mma::kMaxSeqs) * c->num_kv_heads;
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
    // Two units per resident CTA at the table's full width: fewer leave SMs idle at the end, more make units so
    // short that their fixed costs (q, the join, the partial) show (one 4-bit sequence of 131071 tokens: 38 us, with
    // four 43).  At least 64 tokens, at most kMaxSplit (4-bit, 32 sequences of up to 4096 tokens and 256 of up to
    // 8192: 512 took 9 and 15 us more than 1024; 2048 took 2 and 14 more); more only to keep a row's splits within
    // 1024.  A function of the call's shapes, never of the lengths: a result does not change with the other
    // sequences' lengths.
    int64_t split = round_up((rows * p->cap + 2 * workers - 1) / (2 * workers), 64);
    split = std::max<int64_t>(64, std::min<int64_t>(split, kMaxSplit));
    split = std::max(split, round_up((p->cap + 1023) / 1024, 64));
    if (split / c->block_size > (i4 ? 1024 : 8192)) return false; // the split's table entries no longer fit shared memory
    p->split = (int)split;
    p->max_splits = (int)std::max<int64_t>(1, (p->cap + split - 1) / split);
    // (with mass a row of one split keeps its (m, l) too)
    const int64_t partials = p->max_splits > 1 || mass ? (int64_t)hq * p->max_splits * (c->head_dim + 2) : 0;
    const int64_t per_seq = partials + (mass ? (int64_t)hq * p->cap : 0);
    // sequences per launch: at most kMaxSeqs, and at most 2 GB of workspace unless one sequence needs more
    int64_t n = std::min<int64_t>(num_seqs, pkv_mma::kMaxSeqs);
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

cudaError_t run(const pkv_cache *c, const pkv_mma::Args &a, bool mass, bool merge, cudaStream_t st) {
    const int mt = c->model_dtype, D = c->head_dim, sms = c->num_sms;
    if (!mass) return pkv_mma_int4(a, mt, D, sms, merge, st);
    if (c->kv_dtype == PKV_INT4) return pkv_mma_int4_mass(a, mt, D, sms, merge, st);
    if (c->kv_dtype == PKV_FP8_E4M3) return pkv_mma_fp8_mass(a, mt, D, sms, merge, st);
    return pkv_mma_16bit_mass(a, mt, D, sms, merge, st);
}

} // namespace

int64_t decode_mma_workspace_floats(const pkv_cache *c, int num_seqs, int hq, int max_blocks) {
    Plan p;
    return plan_for(c, num_seqs, hq, max_blocks, -1, &p) ? p.floats : 0;
}

int decode_mma_entry(pkv_cache *c, const MmaDecodeLaunch &d, const PkvWorkspace *fixed, cudaStream_t st) {
    Plan p;
    if (!plan_for(c, d.num_seqs, d.num_q_heads, d.max_blocks, d.mass_len, &p))
        return pkv_fail(PKV_EUNSUPPORTED, "tables of %d blocks are wider than this decode takes", d.max_blocks);
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
    // a batch larger than one launch takes runs in consecutive launches that share the workspace: each
    // waits for the one before it.  Another host thread's call on this stream may use the same workspace: no launch of
    // its own comes between this call's.
    std::lock_guard<std::mutex> lk(c->ws_mu);
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
