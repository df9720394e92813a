// Host side of the matrix-instruction decodes (decode_int4.cuh, decode_mma.cuh): split size, workspace, launches.
#include "mma_common.cuh"

#include <algorithm>

namespace {

constexpr int kMaxSplit = 1024; // tokens
constexpr int kFewSplit = 1536; // of the chunk attention of few rows
constexpr int64_t kFewFloats = (int64_t)1 << 29; // partial rows of a launch of it

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// resident CTAs of the kernels of units
int64_t workers_of(const pkv_cache *c, int group) {
    const bool few = c->head_dim == 128 && group == 8; // Geo4::kCtas
    return (int64_t)c->num_sms * (c->kv_dtype == PKV_INT4 ? (few ? 3 : 4) : c->kv_dtype == PKV_FP8_E4M3 ? 3 : 2);
}

// sequences of a launch: over 16-bit caches the list of more would leave room for one CTA an SM instead of two (under a
// window, whose splits may be half as long again, of fewer)
int most_seqs(const pkv_cache *c, bool window = false) {
    return c->kv_dtype == PKV_INT4 || c->kv_dtype == PKV_FP8_E4M3 ? pkv_mma::kMaxSeqs : window ? 312 : 384;
}

// What one launch of at most `seqs` sequences looks like.
struct Plan {
    int64_t cap;    // tokens a sequence may have
    int split, max_splits, seqs;
    int64_t floats; // workspace
    bool is_short;  // a warp a row
};

// blocks of a sequence that a windowed query can see at most
int window_blocks(const pkv_cache *c, int max_blocks, int window, int sinks) {
    const int64_t bs = c->block_size, w = ((int64_t)window - 1 + bs - 1) / bs + 1, s = ((int64_t)sinks + bs - 1) / bs;
    return (int)std::min<int64_t>(max_blocks, w + s);
}

// (window: max_blocks are those that a window shows)
bool plan_for(const pkv_cache *c, int num_seqs, int hq, int max_blocks, int64_t mass_len, bool window, Plan *p) {
    const bool mass = mass_len >= 0;
    p->cap = (int64_t)max_blocks * c->block_size;
    if (mass) p->cap = std::min(p->cap, mass_len);
    const bool i4 = c->kv_dtype == PKV_INT4;
    const int64_t workers = workers_of(c, hq / c->num_kv_heads);
    const int most = most_seqs(c, window);
    const int64_t rows = (int64_t)std::min(num_seqs, most) * c->num_kv_heads;
    // Short rows by a warp each, where two of three speak for it: the mass (which saves a launch), up to four heads (a
    // warp's work), more rows than CTAs.  4-bit, D = 128: 8 rows of four heads and 16 tokens, 5.4 us with mass
    // (units: 8.0), 5.7 without (5.1); 256 rows of eight heads and 32 tokens, 15.7 us with mass (9.4); many rows see
    // decode_short.cuh.
    p->is_short = !window && p->cap <= pkv_mma::kShortTokens &&
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
    // Under a window the sequences' sight is mostly of one length, a little above a round number: splits of equal
    // size, and longer ones rather than one with a small rest (a window of 1024 and 4 sinks, 32 sequences of 32 fp16
    // heads: one split of 1056 74.0 us, two of 528 85.1, one of 1024 and a rest 83.2).
    const int tile = i4 ? 32 : 16, round = 4 * tile;
    const int64_t longest = window ? kMaxSplit + kMaxSplit / 2 : kMaxSplit;
    const int64_t parts = std::max<int64_t>(1, (p->cap + longest - 1) / longest);
    int64_t split = window ? round_up(std::max<int64_t>(1, (p->cap + parts - 1) / parts), 32) : kMaxSplit;
    if (rows * parts <= 4 * workers) {
        double least = 0.;
        for (int64_t k = i4 ? 1 : 2; k <= 2 * longest / round; k += i4 ? 1 : 2) { // whole rounds, or a tile less
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
    if (a.window > 0) {
        if (c->kv_dtype == PKV_INT4) return pkv_mma_int4_window(a, mt, D, sms, merge, st);
        if (c->kv_dtype == PKV_FP8_E4M3) return pkv_mma_fp8_window(a, mt, D, sms, merge, st);
        return pkv_mma_16bit_window(a, mt, D, sms, merge, st);
    }
    if (!mass) return pkv_mma_int4(a, mt, D, sms, merge, st);
    if (c->kv_dtype == PKV_INT4) return pkv_mma_int4_mass(a, mt, D, sms, merge, st);
    if (c->kv_dtype == PKV_FP8_E4M3) return pkv_mma_fp8_mass(a, mt, D, sms, merge, st);
    return pkv_mma_16bit_mass(a, mt, D, sms, merge, st);
}

// what follows from the cache and the heads alone
int pool_args(const pkv_cache *c, int hq, pkv_mma::Args *a) {
    a->pool = static_cast<const char *>(c->pool);
    a->k_scale = c->k_scale;
    a->v_scale = c->v_scale;
    a->err = c->err;
    a->num_blocks = c->num_blocks;
    pkv_row_strides(c, &a->blk_stride, &a->head_stride, &a->v_off);
    if (a->blk_stride > 0xFFFFFFFFll)
        return pkv_fail(PKV_EUNSUPPORTED, "blocks of %lld bytes are larger than this decode takes", (long long)a->blk_stride);
    a->hq = hq;
    a->hkv = c->num_kv_heads;
    a->group = hq / c->num_kv_heads;
    int s = 0;
    while (((int64_t)1 << s) < a->hkv) ++s;
    a->hkv_shift = 31 + s;
    a->hkv_magic = (uint32_t)((((uint64_t)1 << a->hkv_shift) + a->hkv - 1) / a->hkv);
    a->bs_log2 = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
    return PKV_OK;
}

// Splits of the chunk attention of few rows: tokens of one, for `units` = sequences times KV heads.  At least 128 tokens (a
// unit's fixed part costs about 100) and so few that the units fill the SMs twice; where there are more units than that,
// splits of equal size up to kFewSplit tokens.
int few_split(const pkv_cache *c, int64_t units, int64_t cap, int ctas) {
    const int64_t workers = (int64_t)c->num_sms * ctas, longest = kFewSplit;
    const int64_t parts = std::max<int64_t>(1, (cap + longest - 1) / longest);
    int64_t split = round_up(std::max<int64_t>(1, (cap + parts - 1) / parts), 32);
    if (units * parts <= 4 * workers) {
        double least = 0.;
        for (int64_t t = 128; t <= longest; t += 64) {
            const int64_t splits = std::max<int64_t>(1, (cap + t - 1) / t);
            if (units * splits > 2 * workers + units) continue; // (keeps the workspace within few_workspace_floats)
            const double join = splits == 1 ? 0. : 4.;
            const double time = (double)((units * splits + workers - 1) / workers) *
                                    (1.4 * (double)((std::min(t, cap) + 63) / 64) + 3.) + join;
            if (least == 0. || time < least) {
                least = time;
                split = t;
            }
            if (splits == 1) break;
        }
    }
    return (int)std::max(split, round_up((cap + 1023) / 1024, 64));
}

} // namespace

// tokens that the new ones of a sequence (rows at most) can see together, at most
static int64_t few_seen(const pkv_cache *c, const ChunkLaunch &p, int rows) {
    const int64_t bs = c->block_size, cap = p.max_blocks * bs;
    if (p.window == 0) return cap;
    const int64_t n = std::min(p.max_seqlen, rows / (p.num_q_heads / c->num_kv_heads));
    return std::min<int64_t>(cap, ((p.window + n - 2 + bs - 1) / bs + 1 + ((int64_t)p.sinks + bs - 1) / bs) * bs);
}
static int few_seqs(const pkv_cache *c, int num_seqs) { // of a launch (the list of more would leave room for one CTA an SM less)
    return std::min(num_seqs, c->kv_dtype == PKV_FP8_E4M3 ? pkv_mma::kMaxSeqs : 256);
}

// Up to 24 rows of a KV head: by chunk_few.cuh, but where long sequences fill the SMs many times over only up to 16 (E4M3)
// and 8; tcgen05 takes 64 rows in the time of one there.  (256 log-normal sequences of up to 8192 tokens, 32/8 heads, E4M3:
// 8 rows 99 us, tcgen05 168, 16 rows 131 and 174, 24 rows 172 and 179, 4 to 24 of them 172 and 167; bf16 8 rows 157 and
// 191, 16 rows 198 and 196, 24 rows 224 and 201.  The same under a window of 511: E4M3 16 rows 70 and 121, 24 rows 93 and
// 123, bf16 16 rows 96 and 154; 8 sequences of 4096, 24 rows: E4M3 26 and 46, bf16 34 and 50.)
int chunk_few_rows(const pkv_cache *c, const ChunkLaunch &p) {
    const int64_t parts = (few_seen(c, p, 24) + kFewSplit - 1) / kFewSplit;
    const bool some = parts <= 1 || (int64_t)few_seqs(c, p.num_seqs) * c->num_kv_heads * parts <= 8 * (int64_t)c->num_sms;
    return some ? 24 : c->kv_dtype == PKV_FP8_E4M3 ? 16 : 8;
}

// (seqs: of a launch, whose partial rows take at most 2 GB unless one sequence's need more)
static int few_plan(const pkv_cache *c, const ChunkLaunch &p, int rows, pkv_mma::FewArgs *a, int *seqs) {
    const int G = p.num_q_heads / c->num_kv_heads;
    const int64_t seen = few_seen(c, p, rows);
    a->most_rows = rows;
    a->row_room = std::min(p.max_seqlen, rows / G) * G;
    a->split_tokens = few_split(c, (int64_t)few_seqs(c, p.num_seqs) * c->num_kv_heads, seen,
                                c->kv_dtype == PKV_FP8_E4M3 && std::min<int64_t>(rows, (int64_t)p.max_seqlen * G) <= 8 ? 3 : 2);
    a->max_splits = (int)std::max<int64_t>(1, (seen + a->split_tokens - 1) / a->split_tokens);
    if (a->split_tokens / c->block_size > 8192)
        return pkv_fail(PKV_EUNSUPPORTED, "tables of %d blocks are wider than this call takes", p.max_blocks);
    const int64_t floats = (int64_t)c->num_kv_heads * a->row_room * a->max_splits * (c->head_dim + 2);
    *seqs = few_seqs(c, p.num_seqs);
    if (a->max_splits > 1) *seqs = (int)std::max<int64_t>(1, std::min<int64_t>(*seqs, kFewFloats / floats));
    return PKV_OK;
}

int64_t chunk_few_floats(const pkv_cache *c, const ChunkLaunch &p, int rows) {
    pkv_mma::FewArgs a;
    int seqs;
    if (few_plan(c, p, rows, &a, &seqs) || a.max_splits <= 1) return 0;
    return (int64_t)seqs * c->num_kv_heads * a.row_room * a.max_splits * (c->head_dim + 2);
}

int64_t few_workspace_floats(const pkv_cache *c, int num_seqs, int max_blocks) {
    // Rows of at most 24 a (sequence, KV head).  Splits: of at least 1024 tokens, or of at least 128 and so that a launch
    // has two waves of units (3 CTAs an SM) and one a row more.
    const int64_t cap = (int64_t)max_blocks * c->block_size, per_seq = (int64_t)c->num_kv_heads * 24;
    const int64_t rows = few_seqs(c, num_seqs) * per_seq;
    const int64_t most = std::min<int64_t>(rows * ((cap + 127) / 128), rows + 24 * 2 * 3 * (int64_t)c->num_sms);
    const int64_t floats = std::max(most, rows * ((cap + 1023) / 1024)) * (c->head_dim + 2);
    return std::min(floats, std::max(kFewFloats, per_seq * ((cap + 127) / 128) * (c->head_dim + 2)));
}

int chunk_few_launch(pkv_cache *c, const ChunkLaunch &p, int rows, bool late, float *ws, cudaStream_t st) {
    const int G = p.num_q_heads / c->num_kv_heads;
    int per;
    pkv_mma::FewArgs a;
    if (int r = pool_args(c, p.num_q_heads, &a)) return r;
    if (int r = few_plan(c, p, rows, &a, &per)) return r;
    a.q = p.q;
    a.out = p.out;
    a.ws_x = nullptr;
    a.mass = nullptr;
    a.mass_len = -1;
    a.decay = 1.f;
    a.done = nullptr;
    a.cap = (int64_t)p.max_blocks * c->block_size;
    a.max_blocks = p.max_blocks;
    a.qk_scale_log2 = p.scale * 1.4426950408889634f;
    a.window = std::min(p.window, 1 << 30);
    a.sinks = p.sinks;
    a.total = p.total_tokens;
    a.max_seqlen = p.max_seqlen;
    a.lg_group = G == 8 ? 3 : G == 4 ? 2 : G == 2 ? 1 : 0;
    const bool split = a.max_splits > 1;
    a.ws_o = split ? ws : nullptr;
    a.ws_ml = split ? ws + (int64_t)per * c->num_kv_heads * a.row_room * a.max_splits * c->head_dim : nullptr;
    for (int s0 = 0; s0 < p.num_seqs; s0 += per) {
        a.num_seqs = std::min(per, p.num_seqs - s0);
        a.tables = p.tables ? p.tables + (int64_t)s0 * p.max_blocks : nullptr;
        a.lens = p.lens + s0;
        a.cu = p.cu + s0;
        a.late = late && s0 == 0; // (later launches wait for the merge before them, whose room they use)
        for (int merge = 0; merge <= (split ? 1 : 0); ++merge) {
            g_pkv_launches++;
            const cudaError_t e = c->kv_dtype == PKV_FP8_E4M3 ? pkv_few_e4m3(a, c->model_dtype, c->head_dim, c->num_sms, merge, st)
                                                              : pkv_few_16bit(a, c->model_dtype, c->head_dim, c->num_sms, merge, st);
            if (e != cudaSuccess) return pkv_cuda_fail(e, "chunk attention launch");
        }
    }
    return PKV_OK;
}

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

int64_t decode_window_workspace_floats(const pkv_cache *c, int num_seqs, int hq, int max_blocks, int window, int sinks) {
    // (the decode's, of tables that hold what a window shows: its splits are no shorter and its launches of no more rows)
    return decode_mma_workspace_floats(c, num_seqs, hq, window_blocks(c, max_blocks, window, sinks), -1);
}

int decode_mma_entry(pkv_cache *c, const MmaDecodeLaunch &d, const PkvWorkspace *fixed, cudaStream_t st) {
    Plan p;
    const int seen = d.window > 0 ? window_blocks(c, d.max_blocks, d.window, d.sinks) : d.max_blocks;
    if (!plan_for(c, d.num_seqs, d.num_q_heads, seen, d.mass_len, d.window > 0, &p))
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
    if (int r = pool_args(c, d.num_q_heads, &a)) return r;
    a.mass_len = d.mass_len;
    a.cap = d.window > 0 ? (int64_t)d.max_blocks * c->block_size : p.cap;
    a.window = d.window;
    a.sinks = d.sinks;
    a.max_blocks = d.max_blocks;
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
