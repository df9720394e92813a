// New tokens' q, k and v on their way from the projections: norms of each head, position rotation, append.
//
// Per token j at position p and head row x of D elements (q and k):
//   y = x rsqrt(mean x^2 + eps) w                                            (optional, w per element)
//   (y_a, y_b) -> gain (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = p f_i
// for the pairs i of its first R elements, (a, b) = (i, i + R / 2) or (2 i, 2 i + 1); the others stay.  All of it in
// fp32, rounded once to the model's type: q goes to q_out, k and v to their slots as paged_kv_append stores them (so
// that a cache of few bits holds the codes of the k that the model's type holds, as the prefill that is given that k).
//
// The angle.  f_i comes as a 64-bit fraction of a turn, so p f_i modulo 2^64 is the angle modulo a turn (to 2^-31):
// two integer multiplications, no reduction of large arguments, the same error at position 100000 as at 1 (the leading 32 bits
// as a float, 2^-25 of a turn, then sincospif's own).  Nothing is read for it but the position, and a table of
// cosines for 131072 positions would be 64 MB.
//
// Bound by HBM (2 (Hq + 2 Hkv) D elements in, as many out) or, for a step's few tokens, by the launch and the chain
// position -> block table -> slot.  A pass of the CTA takes `tb` tokens: each (token, frequency) pair's cosine and sine is
// found by one thread and left in shared memory for all the token's heads (done by each thread for its own
// elements they are more instructions than the rest of the row), as are the slots.  Then D / 16 lanes share a row, sixteen
// elements each, chosen so that both members of a pair lie in the same lane: the runs of eight at 8 c and
// R / 2 + 8 c for halves, 16 c .. 16 c + 15 for neighbours.  A lane's cosines lie 16 bytes apart from its
// neighbours' (four reads of 16 bytes without bank conflicts).
//
// 5256 tokens of 32/32 heads: 46.1 us (floor of their bytes 38.7).  Into an E4M3 cache 51.4 (32.2), into a 4-bit one 44.2
// (29.2): those are bound by instructions (2.8 and 2.7 a cycle and SM of 4; sixteen IEEE divisions a lane, as the append
// has them, and the rows' extremes).
#include <algorithm>
#include <cmath>

#include "device_common.cuh"
#include "int4.cuh"
#include "pkv_internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4; // of a pass: 4 x 64 frequencies, one a thread
constexpr int kUnroll = 3;    // rows whose loads go out before any of them is worked on

// CTAs of an SM that fit together (64 registers a thread) and are launched.  5256 tokens of 32/32 heads, 8188 of 32/8 with
// norms: 46.4 and 40.8 us; one to three CTAs of the registers asked for 51.7 and 49.2, five 47.0 and 45.6 (spills), one or
// two rows at a time 47.3 and 43.9, 48.0 and 40.7.
constexpr int kCtas = 4, kGridCtas = 8;

struct RotaryArgs {
    const char *q, *k, *v; // token j's row at j * stride bytes
    char *q_out;
    int64_t q_stride, k_stride, v_stride, out_stride; // bytes
    const int32_t *tables, *seq_ids, *positions, *angles; // angles: positions of the rotation
    int64_t *slots_out;
    const void *wq, *wk;
    char *pool;
    const float *k_scale, *v_scale;
    unsigned int *err;
    int64_t n, num_slots, tile_elems;
    int rows, max_blocks, hq, hkv, bs, bs_log2;
    int per_token;        // rows of a token: hq + 2 hkv
    unsigned magic;       // ceil(2^32 / per_token)
    int pairs;            // R / 2
    int tb;
    float eps, gain;
    uint64_t freq[64]; // turns a position, times 2^64
};

template <int D, int KVT, int MT, bool NORM, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, kCtas) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    using M = ModelT<MT>;
    constexpr int LPR = D / 16, RPI = kThreads / LPR; // lanes a row, rows the CTA takes at once
    __shared__ float4 turn[2][kMaxTokens][4][8];      // [buffer][token][two of a lane's eight pairs][lane]: cos, sin twice
    __shared__ int64_t slot[2][kMaxTokens];
    const int tid = threadIdx.x, c = tid % LPR;
    const int my_token = tid / a.pairs, my_pair = tid - my_token * a.pairs;
    const uint64_t freq = a.freq[my_pair];
    // this lane's two runs of eight elements, and whether they are rotated
    const int turned = a.pairs / 8;
    const bool turns = c < turned;
    const int run0 = (INTERLEAVED || !turns) ? 2 * c : c, run1 = (INTERLEAVED || !turns) ? 2 * c + 1 : c + turned;
    pdl_trigger();
    pdl_wait();
    uint4 wq[2], wk[2]; // this lane's weights (as stored: widened they would take 32 registers)
    if constexpr (NORM) {
        const uint4 none = make_uint4(0, 0, 0, 0);
        wq[0] = a.wq ? static_cast<const uint4 *>(a.wq)[run0] : none;
        wq[1] = a.wq ? static_cast<const uint4 *>(a.wq)[run1] : none;
        wk[0] = a.wk ? static_cast<const uint4 *>(a.wk)[run0] : none;
        wk[1] = a.wk ? static_cast<const uint4 *>(a.wk)[run1] : none;
    }
    auto load_pos = [&](int64_t base) { // the position that this thread's angle is of
        const int64_t j = base + my_token;
        return my_token < a.tb && j < a.n ? a.angles[j] : 0;
    };
    auto prepare = [&](int buf, int64_t base, int pos) {
        if (my_token < a.tb) {
            const uint64_t t = (uint64_t)(int64_t)pos * freq;
            float s, co;
            sincospif((float)(int32_t)(t >> 32) * 4.656612873e-10f, &s, &co); // half turns: 2^-31
            // pair 8 l + e of lane l: word e / 2 of the lane, half e % 2
            reinterpret_cast<float2 *>(&turn[buf][my_token][(my_pair & 7) >> 1][my_pair >> 3])[my_pair & 1] =
                make_float2(co * a.gain, s * a.gain);
        }
        if (tid < a.tb && base + tid < a.n) {
            int64_t sl = slot_of(a.tables, a.rows, a.max_blocks, a.seq_ids[base + tid], a.positions[base + tid], a.bs);
            if (blockIdx.y == 0 && a.slots_out) a.slots_out[base + tid] = sl;
            if (sl >= a.num_slots) {
                set_error(a.err, PKV_DEVERR_SLOT);
                sl = -1;
            }
            slot[buf][tid] = sl;
        }
    };
    const int64_t step = (int64_t)gridDim.x * a.tb;
    int64_t base = (int64_t)blockIdx.x * a.tb;
    if (base >= a.n) return;
    prepare(0, base, load_pos(base));
    int next_pos = load_pos(base + step);
    __syncthreads();
    for (int buf = 0; base < a.n; base += step, buf ^= 1) {
        if (base + step < a.n) {
            prepare(buf ^ 1, base + step, next_pos);
            next_pos = load_pos(base + 2 * step);
        }
        const int total = (int)min((int64_t)a.tb, a.n - base) * a.per_token;
        const int stride = gridDim.y * RPI;
        // (every lane of a warp makes the same rounds: the norm's sums are exchanged by all of them)
        for (int r0 = blockIdx.y * RPI; r0 < total; r0 += kUnroll * stride) {
            uint4 x[kUnroll][2];
            int tok[kUnroll], head[kUnroll];
            bool live[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = r0 + u * stride + tid / LPR;
                live[u] = r < total;
                tok[u] = (int)__umulhi((unsigned)r, a.magic);
                head[u] = r - tok[u] * a.per_token;
                if (!live[u]) {
                    x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
                    continue;
                }
                const int64_t j = base + tok[u];
                const int hk = head[u] - a.hq;
                const char *p = hk < 0       ? a.q + j * a.q_stride + head[u] * (D * 2)
                                : hk < a.hkv ? a.k + j * a.k_stride + hk * (D * 2)
                                             : a.v + j * a.v_stride + (hk - a.hkv) * (D * 2);
                x[u][0] = __ldcs(reinterpret_cast<const uint4 *>(p) + run0);
                x[u][1] = __ldcs(reinterpret_cast<const uint4 *>(p) + run1);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int hk = head[u] - a.hq;
                const bool is_v = hk >= a.hkv;
                float f[16];
                cvt8<MT>(x[u][0], f);
                cvt8<MT>(x[u][1], f + 8);
                if constexpr (NORM) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    if (hk < 0 ? a.wq != nullptr : a.wk != nullptr) {
                        const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float w[8];
                            cvt8<MT>(hk < 0 ? wq[i] : wk[i], w);
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[8 * i + e] = f[8 * i + e] * inv * w[e];
                        }
                    }
                }
                if (!live[u]) continue;
                if (!is_v) {
                    if (turns) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float4 t = turn[buf][tok[u]][e >> 1][c];
                            const int a0 = INTERLEAVED ? 2 * e : e, b0 = INTERLEAVED ? 2 * e + 1 : e + 8;
                            const int a1 = INTERLEAVED ? 2 * e + 2 : e + 1, b1 = INTERLEAVED ? 2 * e + 3 : e + 9;
                            const float y0 = f[a0] * t.x - f[b0] * t.y, z0 = f[b0] * t.x + f[a0] * t.y;
                            const float y1 = f[a1] * t.z - f[b1] * t.w, z1 = f[b1] * t.z + f[a1] * t.w;
                            f[a0] = y0;
                            f[b0] = z0;
                            f[a1] = y1;
                            f[b1] = z1;
                        }
                    }
                    if (turns || NORM) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            x[u][i] = make_uint4(M::pack(f[8 * i], f[8 * i + 1]), M::pack(f[8 * i + 2], f[8 * i + 3]),
                                                 M::pack(f[8 * i + 4], f[8 * i + 5]), M::pack(f[8 * i + 6], f[8 * i + 7]));
                    }
                }
                if (hk < 0) {
                    uint4 *o = reinterpret_cast<uint4 *>(a.q_out + (base + tok[u]) * a.out_stride + head[u] * (D * 2));
                    o[run0] = x[u][0];
                    o[run1] = x[u][1];
                    continue;
                }
                const int64_t sl = slot[buf][tok[u]];
                if (sl < 0) continue;
                const int kv = is_v ? 1 : 0, h = hk - kv * a.hkv;
                const int64_t blk = sl >> a.bs_log2;
                const int off = (int)sl & (a.bs - 1);
                if constexpr (KVT == PKV_INT4) {
                    const unsigned lanes = ((1u << LPR) - 1u) << ((tid & 31) & ~(LPR - 1));
                    const Int4Row row = int4_quantise<MT>(x[u], LPR, lanes);
                    char *tile = a.pool + int4_head(blk, h, a.hkv, a.bs, D);
                    *reinterpret_cast<uint32_t *>(tile + int4_codes(kv, off, run0 * 4, D)) = row.codes.x;
                    *reinterpret_cast<uint32_t *>(tile + int4_codes(kv, off, run1 * 4, D)) = row.codes.y;
                    if (c == 0) *reinterpret_cast<uint32_t *>(tile + int4_params(kv, off, D)) = row.params;
                } else {
                    const int64_t e0 = ((blk * 2 + kv) * a.hkv + h) * a.tile_elems + off * D;
                    if constexpr (KVT == PKV_FP8_E4M3) {
                        const float sc = (kv ? a.v_scale : a.k_scale)[h];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float g[8];
                            cvt8<MT>(x[u][i], g);
                            uint2 o;
                            o.x = e4m3x2_from_f32(__fdiv_rn(g[0], sc), __fdiv_rn(g[1], sc)) |
                                  (e4m3x2_from_f32(__fdiv_rn(g[2], sc), __fdiv_rn(g[3], sc)) << 16);
                            o.y = e4m3x2_from_f32(__fdiv_rn(g[4], sc), __fdiv_rn(g[5], sc)) |
                                  (e4m3x2_from_f32(__fdiv_rn(g[6], sc), __fdiv_rn(g[7], sc)) << 16);
                            reinterpret_cast<uint2 *>(a.pool + e0)[i ? run1 : run0] = o;
                        }
                    } else {
                        uint4 *o = reinterpret_cast<uint4 *>(a.pool + e0 * 2);
                        o[run0] = x[u][0];
                        o[run1] = x[u][1];
                    }
                }
            }
        }
        __syncthreads();
    }
}

template <int D, int KVT, int MT>
cudaError_t launch_t(const RotaryArgs &a, bool norm, bool interleaved, dim3 grid, cudaStream_t st) {
    auto kern = norm ? (interleaved ? rotary_kernel<D, KVT, MT, true, true> : rotary_kernel<D, KVT, MT, true, false>)
                     : (interleaved ? rotary_kernel<D, KVT, MT, false, true> : rotary_kernel<D, KVT, MT, false, false>);
    return pdl_launch(kern, grid, dim3(kThreads), 0, st, a);
}

// x modulo one, times 2^64, cut
uint64_t part_bits(double x) {
    const double part = std::fmod(x, 1.0); // (exact, of x's sign)
    const uint64_t bits = (uint64_t)(std::fabs(part) * 18446744073709551616.0);
    return part < 0 ? 0 - bits : bits;
}
// radians as a fraction of a turn, modulo one, times 2^64: 1 / (2 pi) is two doubles and the product keeps its rounding
// error, so that 2^31 positions of it are right to 2^-31 of a turn for frequencies of up to 2^40.  (As one double product,
// right to 2^-53 of the turns of a position, position 2^31 - 1 was off by 2^-25 of a turn at a frequency of 1 and by a
// whole one at 1e8.)
uint64_t turn_bits(double radians) {
    constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    const double turns = radians * hi, rest = std::fma(radians, hi, -turns) + radians * lo;
    return part_bits(turns) + part_bits(rest);
}

} // namespace

cudaError_t launch_append_rotary(pkv_cache *c, const RotaryLaunch &r, cudaStream_t st) {
    if (r.n == 0) return cudaSuccess;
    RotaryArgs a{};
    a.q = static_cast<const char *>(r.q);
    a.k = static_cast<const char *>(r.k);
    a.v = static_cast<const char *>(r.v);
    a.q_out = static_cast<char *>(r.q_out);
    a.q_stride = r.q_stride * 2;
    a.k_stride = r.k_stride * 2;
    a.v_stride = r.v_stride * 2;
    a.out_stride = r.q_out_stride * 2;
    a.tables = r.tables;
    a.seq_ids = r.seq_ids;
    a.positions = r.positions;
    a.angles = r.rotary_positions ? r.rotary_positions : r.positions;
    a.slots_out = r.slots_out;
    a.wq = r.q_weight;
    a.wk = r.k_weight;
    a.pool = static_cast<char *>(c->pool);
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
    a.err = c->err;
    a.n = r.n;
    a.num_slots = c->num_blocks * c->block_size;
    a.tile_elems = (int64_t)c->block_size * c->head_dim;
    a.rows = r.rows;
    a.max_blocks = r.max_blocks;
    a.hq = r.num_q_heads;
    a.hkv = c->num_kv_heads;
    a.bs = c->block_size;
    a.bs_log2 = c->block_size == 8 ? 3 : c->block_size == 16 ? 4 : 5;
    a.per_token = a.hq + 2 * a.hkv;
    a.magic = (unsigned)((0x100000000ull + a.per_token - 1) / a.per_token);
    a.pairs = r.rotary->rotary_dim / 2;
    a.eps = r.eps;
    a.gain = r.rotary->gain;
    for (int i = 0; i < a.pairs; ++i) a.freq[i] = turn_bits(r.rotary->inv_freq[i]);
    // few tokens: one a pass, its rows over several CTAs; many: up to four a pass, the cosines of the next pass found
    // while this one's rows are on their way
    const int rows_at_once = kThreads / (c->head_dim / 16);
    a.tb = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxTokens, r.n / (c->num_sms * 2)));
    const int64_t passes = (r.n + a.tb - 1) / a.tb, cap = (int64_t)c->num_sms * kGridCtas;
    const unsigned gx = (unsigned)std::min(passes, cap);
    const unsigned gy = (unsigned)std::max<int64_t>(1, std::min<int64_t>((a.per_token * a.tb + rows_at_once - 1) / rows_at_once, cap / gx));
    const dim3 grid(gx, gy);
    const bool norm = r.q_weight || r.k_weight, il = r.rotary->interleaved != 0, h = c->model_dtype == PKV_F16;
    PkvTimer timer(c, PKV_KIND_APPEND, st);
    g_pkv_launches++;
#define PKV_CASE(DD)                                                                                                   \
    if (c->head_dim == DD) {                                                                                           \
        if (c->kv_dtype == PKV_INT4)                                                                                   \
            return h ? launch_t<DD, PKV_INT4, PKV_F16>(a, norm, il, grid, st) : launch_t<DD, PKV_INT4, PKV_BF16>(a, norm, il, grid, st); \
        if (c->kv_dtype == PKV_FP8_E4M3)                                                                               \
            return h ? launch_t<DD, PKV_FP8_E4M3, PKV_F16>(a, norm, il, grid, st)                                      \
                     : launch_t<DD, PKV_FP8_E4M3, PKV_BF16>(a, norm, il, grid, st);                                    \
        return h ? launch_t<DD, PKV_F16, PKV_F16>(a, norm, il, grid, st) : launch_t<DD, PKV_F16, PKV_BF16>(a, norm, il, grid, st); \
    }
    PKV_CASE(64)
    PKV_CASE(128)
#undef PKV_CASE
    return cudaErrorInvalidValue;
}
