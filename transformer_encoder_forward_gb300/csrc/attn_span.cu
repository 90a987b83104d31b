// Varlen attention with a window of its own to either side, a few first keys
// that stay visible, and a learned bias of relative position (sm_103a):
//
//     o[i, h] = sum_j softmax_j(scale * q[i, h] . k[j, g] + bias[bucket(j - i), h]) v[j, g]
//
// over the keys j of i's own sequence with
//     j <= i + right  and  (j >= i - left  or  j < sinks).
//
// The kernel is the flash form of attn.cu (128-query tiles, 128-key tiles, S
// and O in TMEM, one query row a softmax thread, the maximum moved lazily);
// what differs is the list of key tiles, the mask and the bias:
//   * key tiles: those that hold one of the first `sinks` keys, then those of
//     the window of the CTA's queries.  With two query tiles a CTA (hd = 128)
//     each tile takes part only in the key tiles that its own rows see: its S
//     and PV are not issued for the others and its softmax warps skip them;
//   * mask: a row's visible keys of a tile are four 32-bit words (a bit below
//     the last key and not below the first one, or below `sinks`), applied to
//     the scores in one pass; tiles that every row of a warp sees whole skip it;
//   * bias: a head's column of the table is spread over the distances once a
//     CTA, in shared memory, scaled by log2 e.  A row's thread then adds the
//     float at (key - row), neighbouring rows neighbouring words (no bank
//     conflicts), in the same FMA that scales the score.  Beyond `reach` all
//     distances of a side share one bucket: there the bias is one number for
//     the tile and goes into the exponent's offset, at no cost a key.
// A masked key has weight 0, but 0 x inf is not 0: the tensor core would spread
// a value that is not finite from a masked place.  So the rows of V behind a
// sequence's end (its neighbour's) are zeroed in shared memory, and an output
// row that comes out not finite all the same is computed again from its visible
// keys alone (mend_row), which finite inputs never reach.
// Every mbarrier wait is bounded, as in attn.cu.
#include <cuda.h>
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace tefwd {
namespace {

constexpr int BQ = 128;     // queries per tile (= TMEM lanes); TL tiles per CTA
constexpr int BKV = 128;    // keys per tile
constexpr int MAX_WORK = 640;   // work list entries carried in the launch parameters
constexpr int PAD = 160;    // distances past `reach` that a tile near it can still touch (158)
// as in attn.cu: K and V bytes that the CTA order treats as one group of heads
constexpr long long KV_ALL_BYTES = 48ll << 20;
constexpr long long KV_GROUP_BYTES = 24ll << 20;

__device__ int g_span_err;

struct SpanParams {
    CUtensorMap map;           // the bf16 q|k|v panel [T, ld], box 64 x 128
    __nv_bfloat16 *out;
    const __nv_bfloat16 *qkv;
    const int *cu;
    int nseq, total;
    int nwork;                 // > 0: work[i] = (sequence << 16) | query block, longest first
    int nq, hgroup;            // heads, and heads per group of the CTA order
    uint32_t work[MAX_WORK];
    long long ld, ldo;
    int q_off, k_off, v_off, group;
    int left, right, sinks;    // limits clipped to the longest sequence
    float scale_log2;
    // relative position bias
    const float *table;        // [buckets, ldt]
    long long ldt;
    int side, exact, reach, two_sided;   // buckets of a side, those of one distance each; clipped reach
    float grow;                // logarithmic buckets per unit of log2(distance / exact)
    uint16_t first[TE_RELPOS_MAX_BUCKETS];   // smallest distance of each bucket of a side
};

template <int HD, int TL>
struct SLayout {
    static constexpr int NB = HD / 64;              // 64-column boxes per tile row
    static constexpr int TILE = 128 * HD * 2;       // one 128-row tile
    static constexpr int Q_OFF = 0;                 // Q[TL]
    static constexpr int K_OFF = TL * TILE;         // K[2]
    static constexpr int V_OFF = K_OFF + 2 * TILE;  // V[2]
    static constexpr int BAR_OFF = V_OFF + 2 * TILE;
    static constexpr int NTHREADS = 32 * (4 * TL + 2);   // softmax warps, MMA warp, TMA warp
    static constexpr int MMA_WARP = 4 * TL, TMA_WARP = 4 * TL + 1;
    static constexpr int NBAR = 1 + 2 + 2 + 2 + 2 + 2 + 2 + 1 + 2 + 1;
    static constexpr int TAB_OFF = BAR_OFF + 8 * NBAR + 16;   // the head's table column, then the spread bias
    static constexpr int S_COL = 0;                 // S: TL x 128 f32 columns
    static constexpr int P_COL = TL == 1 ? 128 : 0; // TL = 1: 64 columns of its own; TL = 2: over S
    static constexpr int O_COL = TL == 1 ? 192 : TL * 128;   // O: TL x HD f32 columns
    static constexpr int COLS = TL == 1 ? 256 : 512;
    static_assert(TL == 2 || HD == 64, "one tile a CTA is the hd = 64 form");
    static_assert(O_COL + TL * HD <= COLS, "TMEM budget");
    // the widest bias: every distance to TE_RELPOS_MAX_DISTANCE to either side
    static_assert(TAB_OFF + 4 * (TE_RELPOS_MAX_BUCKETS + 2 * (TE_RELPOS_MAX_DISTANCE + PAD) + 1) + 1024 <= 227 * 1024,
                  "shared memory per CTA");
};

// Key tiles that rows [r0, r1] of a sequence of `len` see: tiles [0, sink) and
// [first, end).
struct KeyTiles {
    int sink, first, end;
    __device__ __forceinline__ bool has(int t) const { return t < end && (t >= first || t < sink); }
};
__device__ __forceinline__ KeyTiles key_tiles(const SpanParams &p, int r0, int r1, int len) {
    const int lo = r0 > p.left ? r0 - p.left : 0;
    const int hi = r1 + p.right + 1 < len ? r1 + p.right + 1 : len;
    const int first = lo / BKV;
    const int s = ((p.sinks < lo ? p.sinks : lo) + BKV - 1) / BKV;
    return {s < first ? s : first, first, (hi + BKV - 1) / BKV};
}

// bits 0 .. n-1 of a word (n clipped to 0 .. 32)
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}

// The bias of distance d (already clipped to the reach), in the table column col.
__device__ __forceinline__ float bias_of(const SpanParams &p, const float *col, int d) {
    const int a = p.two_sided ? (d < 0 ? -d : d) : (d < 0 ? -d : 0);
    int b = a;
    if (a >= p.exact) {
        // within one of the bucket by the f32 logarithm, then by the exact borders
        b = p.exact + (int)(__log2f((float)a / (float)p.exact) * p.grow);
        b = b < p.exact ? p.exact : (b > p.side - 1 ? p.side - 1 : b);
        if (b > p.exact && a < p.first[b]) --b;
        else if (b + 1 < p.side && a >= p.first[b + 1]) ++b;
    }
    return col[p.two_sided && d > 0 ? b + p.side : b];
}

// Scores of 64 keys to log2 units with their bias: v = v c + b[e] (ONE: + one).
template <bool ONE>
__device__ __forceinline__ void add_bias(uint32_t (&v)[64], uint64_t c2, const float *b, float one) {
#pragma unroll
    for (int e = 0; e < 64; e += 2) {
        const uint64_t b2 = ONE ? f2_pack(one, one) : f2_pack(b[e], b[e + 1]);
        float x, y;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2, b2), x, y);
        v[e] = __float_as_uint(x);
        v[e + 1] = __float_as_uint(y);
    }
}

// One output row from its visible keys alone, by one warp in f32: what the
// tiled form computes, without products of masked values.  It ends at once when
// all of the row is lost.
template <int HD, bool BIAS>
__device__ __noinline__ void mend_row(const SpanParams &p, const float *bias, int off, int len, int h, int qi) {
    constexpr int C = HD / 32;
    const int lane = threadIdx.x & 31, g = h / p.group;
    const __nv_bfloat16 *q = p.qkv + (long long)(off + qi) * p.ld + p.q_off + h * HD;
    const __nv_bfloat16 *kb = p.qkv + (long long)off * p.ld + p.k_off + g * HD;
    const __nv_bfloat16 *vb = p.qkv + (long long)off * p.ld + p.v_off + g * HD + lane * C;
    const int lo = qi > p.left ? qi - p.left : 0;
    const int hi = qi + p.right + 1 < len ? qi + p.right + 1 : len;
    float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
    for (int part = 0; part < 2; ++part) {
        const int from = part ? lo : 0, end = part ? hi : (p.sinks < lo ? p.sinks : lo);
        for (int k0 = from; k0 < end; k0 += 32) {
            const int key = k0 + lane;
            float s = -INFINITY;
            if (key < end) {
                const __nv_bfloat16 *k = kb + (long long)key * p.ld;
                float acc = 0.f;
                for (int c = 0; c < HD; ++c) acc = fmaf(__bfloat162float(q[c]), __bfloat162float(k[c]), acc);
                float b = 0.f;
                if (BIAS) {
                    const int d = key - qi;
                    b = bias[d < -p.reach ? -p.reach : (d > p.reach ? p.reach : d)];
                }
                s = fmaf(acc, p.scale_log2, b);
            }
            float wm = s;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, x));
            const float mn = fmaxf(m, wm), off2 = mn == -INFINITY ? 0.f : mn;
            const float alpha = hw_exp2(m - off2), pr = hw_exp2(s - off2);
            m = mn;
            l = l * alpha + warp_sum(pr);
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] *= alpha;
            for (int t = 0; t < 32 && k0 + t < end; ++t) {
                const float st = __shfl_sync(0xFFFFFFFFu, s, t), pt = __shfl_sync(0xFFFFFFFFu, pr, t);
                if (st == -INFINITY) continue;   // a bias of -inf masks too
                const __nv_bfloat16 *v = vb + (long long)(k0 + t) * p.ld;
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] = fmaf(pt, __bfloat162float(v[c]), o[c]);
            }
            bool lost = true;
#pragma unroll
            for (int c = 0; c < C; ++c) lost = lost && isnan(o[c]);
            if (__all_sync(0xFFFFFFFFu, lost)) {
                part = 2;
                break;
            }
        }
    }
    __nv_bfloat16 *orow = p.out + (long long)(off + qi) * p.ldo + h * HD + lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) orow[c] = __float2bfloat16_rn(l == 0.f ? 0.f : o[c] / l);
}

template <int HD, int TL, bool BIAS>
__global__ void __launch_bounds__(SLayout<HD, TL>::NTHREADS, TL == 1 ? 2 : 1)
    attn_span_kernel(const __grid_constant__ SpanParams p) {
    using L = SLayout<HD, TL>;
    constexpr int QB = TL * BQ;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_q = sb + L::BAR_OFF;
    const uint32_t bar_kf = bar_q + 8;             // [2] K loaded
    const uint32_t bar_vf = bar_kf + 16;           // [2] V loaded
    const uint32_t bar_kve = bar_vf + 16;          // [2] K and V read (TL = 1: V)
    const uint32_t bar_sf = bar_kve + 16;          // [2] S ready, per query tile
    const uint32_t bar_pf = bar_sf + 16;           // [2] P written, per query tile
    const uint32_t bar_pv = bar_pf + 16;           // [2] PV done, per query tile
    const uint32_t bar_fin = bar_pv + 16;
    const uint32_t bar_ke = bar_fin + 8;           // [2] TL = 1: K(j) read by S(j)
    const uint32_t bar_sfree = bar_ke + 16;        // TL = 1: the softmax has read S(j)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::BAR_OFF + 8 * L::NBAR);
    float *tab = reinterpret_cast<float *>(smem + L::TAB_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == L::TMA_WARP && lane == 0) {
        tma_prefetch_desc(&p.map);
        mbar_init(bar_q, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_kf + 8 * i, 1);
            mbar_init(bar_vf + 8 * i, 1);
            mbar_init(bar_kve + 8 * i, 1);
            mbar_init(bar_sf + 8 * i, 1);
            mbar_init(bar_pf + 8 * i, 4);
            mbar_init(bar_pv + 8 * i, 1);
            mbar_init(bar_ke + 8 * i, 1);
        }
        mbar_init(bar_sfree, 4);
        mbar_init(bar_fin, 1);
        fence_mbar_init();
    }
    if (warp == L::MMA_WARP) tmem_alloc(smem_u32(tmem_slot), L::COLS);
    // from here on global memory is touched
    prior_wait();

    int seq, qblk, h;
    if (p.nwork) {
        // CTAs take the heads in groups of hgroup: within a group, work items in
        // list order (most key tiles first), the group's heads fastest
        const int b = blockIdx.x;
        const int per = p.hgroup * p.nwork;
        const int g = b / per;
        const int r = b - g * per;
        const int h0 = g * p.hgroup;
        const int gn = p.nq - h0 < p.hgroup ? p.nq - h0 : p.hgroup;
        const int wi = r / gn;
        const uint32_t wv = p.work[wi];
        seq = (int)(wv >> 16);
        qblk = (int)(wv & 0xFFFFu);
        h = h0 + (r - wi * gn);
    } else {
        // many blocks: sequence s has the slots from cu[s] / QB + s on, at least
        // as many as it has query blocks
        const int slot = blockIdx.x / p.nq;
        h = blockIdx.x - slot * p.nq;
        int lo = 0, hi = p.nseq;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int at = lo + lane * step;
            const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < hi && p.cu[at] / QB + at <= slot);
            const int last = below ? 31 - __clz(below) : 0;
            lo += last * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        seq = lo;
        qblk = slot - (p.cu[seq] / QB + seq);
    }
    const int off = p.cu[seq], len = p.cu[seq + 1] - off;
    const int q0 = qblk * QB;
    // else: nothing to do, or a device table that is not the host's
    bool live = off >= 0 && len >= 1 && (long long)off + len <= p.total && qblk >= 0 && q0 < len;
    const int g = h / p.group;
    const int ntile = TL == 2 && q0 + BQ < len ? 2 : 1;   // tile B exists
    const int last_row = (q0 + QB < len ? q0 + QB : len) - 1;
    const KeyTiles all = key_tiles(p, q0, last_row, len);
    const int n = all.sink + all.end - all.first;
    auto tile_of = [&](int j) { return j < all.sink ? j : all.first + (j - all.sink); };
    // the key tiles of query tile w (TL = 1: every one)
    auto tiles_of = [&](int w) {
        const int r0 = q0 + w * BQ, r1 = r0 + BQ - 1;
        return TL == 1 ? all : key_tiles(p, r0, r1 < len ? r1 : len - 1, len);
    };

    if (warp == L::TMA_WARP && lane == 0) {
        // an earlier CTA gave up a wait: one thread's reading holds for the CTA
        live = live && *reinterpret_cast<volatile int *>(&g_span_err) == 0;
        tmem_slot[1] = live;
        if (live) mbar_arrive_expect_tx(bar_q, ntile * L::TILE);
        for (int w = 0; w < ntile && live; ++w)
            for (int c = 0; c < L::NB; ++c)
                tma_load_2d(sb + L::Q_OFF + w * L::TILE + c * 16384, &p.map, bar_q, p.q_off + h * HD + 64 * c,
                            off + q0 + w * BQ);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    next_go();
    const uint32_t tbase = tmem_slot[0];
    live = tmem_slot[1] != 0;
    bool ok = true;

    if (!live) {
    } else if (warp == L::TMA_WARP) {
        // ------------------------------------------------------ TMA producer
        // (the whole warp in step, one elected lane issues)
        const uint32_t e = elect_one();
        // K(i) into ring slot i & 1 once its previous occupant K(i - 2) is
        // free (TL = 1: read by S(i - 2); TL = 2: K and V free together after
        // PV(i - 2)); V(i) once PV(i - 2) is done
        auto load_k = [&](int i) -> bool {
            const int st = i & 1;
            const uint32_t fb = TL == 1 ? bar_ke : bar_kve;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(fb + 8 * st, ((i >> 1) & 1) ^ 1))) return false;
            mbar_arrive_expect_tx_e(bar_kf + 8 * st, L::TILE, e);
            for (int c = 0; c < L::NB; ++c)
                tma_load_2d_e(sb + L::K_OFF + st * L::TILE + c * 16384, &p.map, bar_kf + 8 * st,
                              p.k_off + g * HD + 64 * c, off + tile_of(i) * BKV, e);
            return true;
        };
        auto load_v = [&](int i) -> bool {
            const int st = i & 1;
            if (TL == 1 && !__all_sync(0xFFFFFFFFu, mbar_wait(bar_kve + 8 * st, ((i >> 1) & 1) ^ 1))) return false;
            mbar_arrive_expect_tx_e(bar_vf + 8 * st, L::TILE, e);
            for (int c = 0; c < L::NB; ++c)
                tma_load_2d_e(sb + L::V_OFF + st * L::TILE + c * 16384, &p.map, bar_vf + 8 * st,
                              p.v_off + g * HD + 64 * c, off + tile_of(i) * BKV, e);
            return true;
        };
        int nk = 0, nv = 0;   // K and V tiles issued
        if (TL == 1) {
            // K runs one tile ahead of V: S(j + 1) needs it while PV(j) waits for P(j)
            if (n > 0 && (ok = load_k(0))) nk = 1;
            for (; nv < n && ok; ++nv) {
                if (nk < n) {
                    if (!(ok = load_k(nk))) break;
                    ++nk;
                }
                if (!(ok = load_v(nv))) break;
            }
        } else {
            for (; nv < n && ok; ++nv) {
                if (!(ok = load_k(nv))) break;
                ++nk;
                ok = load_v(nv);
            }
        }
        // no copy of ours may still be landing when the CTA exits
        mbar_wait(bar_q, 0, 20000000ull);
        for (int i = nk - 2 < 0 ? 0 : nk - 2; i < nk; ++i) mbar_wait(bar_kf + 8 * (i & 1), (i >> 1) & 1, 20000000ull);
        for (int i = nv - 2 < 0 ? 0 : nv - 2; i < nv; ++i) mbar_wait(bar_vf + 8 * (i & 1), (i >> 1) & 1, 20000000ull);
    } else if (warp == L::MMA_WARP) {
        // ------------------------------------------------------- MMA issuer
        // (the whole warp in step, one elected lane issues)
        const uint32_t e = elect_one();
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, BKV);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, HD) | (1u << 16);   // B MN-major
        const uint64_t kd0 = smem_desc_sw128(sb + L::K_OFF), kd1 = smem_desc_sw128(sb + L::K_OFF + L::TILE);
        const uint64_t vd0 = smem_desc_mn_sw128(sb + L::V_OFF, 16384);
        const uint64_t vd1 = smem_desc_mn_sw128(sb + L::V_OFF + L::TILE, 16384);
        auto issue_s = [&](int w, int j) -> bool {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_kf + 8 * (j & 1), (j >> 1) & 1))) return false;
            tc_fence_after();
            const uint64_t k0 = (j & 1) ? kd1 : kd0;
            const uint64_t q0d = smem_desc_sw128(sb + L::Q_OFF + w * L::TILE);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                const uint32_t o = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                mma_ss_bf16_e(tbase + L::S_COL + w * 128, q0d + o, k0 + o, idesc_s, k > 0, e);
            }
            mma_commit_e(bar_sf + 8 * w, e);
            if (TL == 1) mma_commit_e(bar_ke + 8 * (j & 1), e);   // K(j) read
            return true;
        };
        auto issue_pv = [&](int w, int j, bool more) {
            const uint64_t v0 = (j & 1) ? vd1 : vd0;
#pragma unroll
            for (int s2 = 0; s2 < BKV / 16; ++s2)
                mma_ts_bf16_e(tbase + L::O_COL + w * HD, tbase + L::P_COL + w * 128 + 8 * s2,
                              v0 + (uint64_t)(128 * s2), idesc_pv, more || s2 != 0, e);
            mma_commit_e(bar_pv + 8 * w, e);
        };
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_q, 0));
        if (TL == 1) {
            ok = ok && issue_s(0, 0);
            // S(j+1) as soon as the softmax has read S(j) (P has columns of
            // its own), then PV(j) once P(j) is written
            for (int j = 0; j < n && ok; ++j) {
                if (j + 1 < n) {
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_sfree, j & 1))) { ok = false; break; }
                    tc_fence_after();
                    if (!(ok = issue_s(0, j + 1))) break;
                }
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_vf + 8 * (j & 1), (j >> 1) & 1)) ||
                    !__all_sync(0xFFFFFFFFu, mbar_wait(bar_pf, j & 1))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                issue_pv(0, j, j > 0);
                mma_commit_e(bar_kve + 8 * (j & 1), e);   // V(j) read
            }
        } else {
            // PV_A(j), S_A(j+1), PV_B(j), S_B(j+1), each only where the query
            // tile sees the key tile; S_w overwrites the P_w that PV_w reads
            // (not ordered by the tensor pipe): it waits for PV_w
            const KeyTiles kw[2] = {tiles_of(0), ntile == 2 ? tiles_of(1) : KeyTiles{0, 0, 0}};
            int done[2] = {0, 0};   // key tiles of each query tile whose PV is issued
            for (int w = 0; w < 2 && ok; ++w)
                if (kw[w].has(tile_of(0))) ok = issue_s(w, 0);
            for (int j = 0; j < n && ok; ++j) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_vf + 8 * (j & 1), (j >> 1) & 1))) { ok = false; break; }
                const int t = tile_of(j), tn = tile_of(j + 1);
                const bool b_too = kw[1].has(t);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (ok && kw[w].has(t)) {
                        if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar_pf + 8 * w, done[w] & 1))) { ok = false; break; }
                        tc_fence_after();
                        issue_pv(w, j, done[w] > 0);
                        ++done[w];
                    }
                    // K(j), V(j) are free once the last PV(j) is done
                    if (ok && w == (b_too ? 1 : 0)) mma_commit_e(bar_kve + 8 * (j & 1), e);
                    if (ok && j + 1 < n && kw[w].has(tn))
                        ok = (done[w] == 0 || __all_sync(0xFFFFFFFFu, mbar_wait(bar_pv + 8 * w, (done[w] - 1) & 1))) &&
                             issue_s(w, j + 1);
                }
            }
        }
        mma_commit_e(bar_fin, e);
        __all_sync(0xFFFFFFFFu, mbar_wait(bar_fin, 0, 20000000ull));
    } else if (warp < 4 * ntile) {
        // ---------------------------------------- softmax, one query per thread
        const int w = warp >> 2;                         // query tile of this warpgroup
        const int wq = warp & 3;                         // TMEM lane quadrant
        const int r0 = q0 + w * BQ + 32 * wq;            // the warp's first row
        const int qi = r0 + lane;
        const int rl = r0 + 31 < len - 1 ? r0 + 31 : len - 1;   // its last row
        const uint32_t tl = (uint32_t)(32 * wq) << 16;
        const uint32_t scol = tbase + tl + L::S_COL + w * 128;
        const uint32_t pcol = tbase + tl + L::P_COL + w * 128;
        const uint32_t ocol = tbase + tl + L::O_COL + w * HD;
        const float c = p.scale_log2;
        const KeyTiles mine = tiles_of(w);
        const float *bias = nullptr;                     // bias[d]: distance d, -(reach + PAD) .. reach + PAD
        if constexpr (BIAS) {
            // spread the head's bias over the distances while Q and K(0) are on their way
            const int nb = p.two_sided ? 2 * p.side : p.side, width = p.reach + PAD, nt = 128 * ntile;
            for (int b = threadIdx.x; b < nb; b += nt) {
                // log2 units; a finite bias stays finite (the type's lowest value still masks softly)
                const float t = p.table[(long long)b * p.ldt + h], t2 = t * 1.4426950408889634f;
                tab[b] = fabsf(t) <= FLT_MAX ? fminf(fmaxf(t2, -FLT_MAX), FLT_MAX) : t;
            }
            asm volatile("bar.sync 1, %0;" ::"r"(nt) : "memory");
            float *spread = tab + nb + width;
            for (int d = (int)threadIdx.x - width; d <= width; d += nt)
                spread[d] = bias_of(p, tab, d < -p.reach ? -p.reach : (d > p.reach ? p.reach : d));
            asm volatile("bar.sync 1, %0;" ::"r"(nt) : "memory");
            bias = spread;
        }
        float m_used = -INFINITY, l = 0.f;
        int jj = 0;                                      // key tiles done
        for (int j = 0; j < n; ++j) {
            const int t = tile_of(j);
            if (TL == 2 && !mine.has(t)) continue;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_sf + 8 * w, jj & 1));
            if (!ok) break;
            // TL = 2: S_w landed, so the PV_w before it is done: P_w and O_w may
            // be touched.  TL = 1: see below.
            tc_fence_after();
            const int kv0 = t * BKV;
            // the S row once into registers for all passes
            uint32_t v0[64], v1[64];
            tmem_ld64(scol, v0);
            tmem_ld64(scol + 64, v1);
            tmem_wait_ld();
            if (TL == 1) {
                // S(j) is in registers: the tensor core may compute S(j+1)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_sfree);
            }
            // scores in log2 units are s * cs + cb
            float cs = c, cb = 0.f;
            if constexpr (BIAS) {
                const int dlo = kv0 - (r0 + 31), dhi = kv0 + BKV - 1 - r0;   // the warp's distances
                const bool before = dhi <= -p.reach, behind = dlo >= p.reach;
                const uint64_t c2 = f2_pack(c, c);
                const float far = before || behind ? bias[before ? -p.reach : p.reach] : 0.f;
                if ((before || behind) && fabsf(far) <= 8192.f) {
                    cb = far;
                } else if (before || behind) {
                    // so large that it takes the scores' own digits, as it does beside a near tile
                    add_bias<true>(v0, c2, nullptr, far);
                    add_bias<true>(v1, c2, nullptr, far);
                    cs = 1.f;
                } else {
                    add_bias<false>(v0, c2, bias + (kv0 - qi), 0.f);
                    add_bias<false>(v1, c2, bias + (kv0 - qi) + 64, 0.f);
                    cs = 1.f;
                }
            }
            // some row of the warp does not see some key of the tile
            const bool whole = kv0 + BKV <= len && kv0 + BKV - 1 <= r0 + p.right &&
                               (kv0 >= rl - p.left || kv0 + BKV <= p.sinks);
            if (!whole) {
                const int hi = (qi + p.right < len ? qi + p.right + 1 : len) - kv0;   // keys below it are not too far
                const int lo = qi - p.left - kv0, sk = p.sinks - kv0;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t see =
                        bits_below(hi - 32 * x) & (~bits_below(lo - 32 * x) | bits_below(sk - 32 * x));
                    uint32_t *v = x < 2 ? v0 + 32 * x : v1 + 32 * (x - 2);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(see >> e & 1)) v[e] = 0xFF800000u;   // -inf
                }
            }
            // pass 1: the row maximum, eight partial ones
            float m8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = fmaxf(__uint_as_float(v0[i]), __uint_as_float(v1[i]));
#pragma unroll
            for (int e = 8; e < 64; ++e) m8[e & 7] = fmax3(m8[e & 7], __uint_as_float(v0[e]), __uint_as_float(v1[e]));
            const float mx = fmaf(fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                        fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7]))), cs, cb);
            if (TL == 1 && jj > 0) {
                // P and O are free once the PV before is done
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_pv, (jj - 1) & 1));
                if (!ok) break;
                tc_fence_after();
            }
            const bool resc = mx > m_used + 8.f;
            if (__any_sync(0xFFFFFFFFu, resc)) {
                const float alpha = resc ? hw_exp2(m_used - mx) : 1.f;
                if (resc) m_used = mx;
                l *= alpha;
                if (jj > 0) {
#pragma unroll
                    for (int cc = 0; cc < HD / 32; ++cc) {
                        uint32_t v[32];
                        tmem_ld32(ocol + 32 * cc, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                        tmem_st32(ocol + 32 * cc, v);
                    }
                    tmem_wait_st();
                }
            }
            // pass 2: P = 2^(s cs + cb - m) as bf16 and its row sum over the f32 values
            const float nm = cb - (m_used == -INFINITY ? 0.f : m_used);
            const uint64_t c2 = f2_pack(cs, cs), nm2 = f2_pack(nm, nm);
            uint64_t r4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r4[i] = f2_pack(0.f, 0.f);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const uint32_t (&v)[64] = hh ? v1 : v0;
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float a0, a1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, nm2), a0, a1);
                    const float p0 = hw_exp2(a0), p1 = hw_exp2(a1);
                    r4[e & 3] = f2_add(r4[e & 3], f2_pack(p0, p1));
                    pk[e] = pack_bf16x2(p0, p1);
                }
                tmem_st32(pcol + 32 * hh, pk);
            }
            float r8[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) f2_unpack(r4[i], r8[2 * i], r8[2 * i + 1]);
            l += ((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7]));
            if (kv0 + BKV > len) {
                // the last tile: V's rows behind the sequence become zeros, each
                // warp its share of them (a row is 128 bytes of each box)
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_vf + 8 * (j & 1), (j >> 1) & 1));
                if (!ok) break;
                for (int r = len - kv0 + 4 * wq + (lane >> 3); r < BKV; r += 16)
#pragma unroll
                    for (int cc = 0; cc < L::NB; ++cc)
                        *reinterpret_cast<uint4 *>(smem + L::V_OFF + (j & 1) * L::TILE + cc * 16384 + r * 128 +
                                                   (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_pf + 8 * w);
            ++jj;
        }
        // ---- epilogue: O / l, one row per thread (0 where nothing is visible)
        if (ok && jj > 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_pv + 8 * w, (jj - 1) & 1));
        if (ok) {
            tc_fence_after();
            const float inv = 1.f / l;
            float finite = l;                            // NaN once a value of the row is not finite
            __nv_bfloat16 *orow = p.out + (long long)(off + (qi < len ? qi : 0)) * p.ldo + h * HD;
#pragma unroll
            for (int cc = 0; cc < HD / 32; ++cc) {
                uint32_t v[32];
                tmem_ld32(ocol + 32 * cc, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) finite = fmaf(__uint_as_float(v[e]), 0.f, finite);
                if (qi < len) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4 u;
                        u.x = pack_bf16x2(__uint_as_float(v[8 * e + 0]) * inv, __uint_as_float(v[8 * e + 1]) * inv);
                        u.y = pack_bf16x2(__uint_as_float(v[8 * e + 2]) * inv, __uint_as_float(v[8 * e + 3]) * inv);
                        u.z = pack_bf16x2(__uint_as_float(v[8 * e + 4]) * inv, __uint_as_float(v[8 * e + 5]) * inv);
                        u.w = pack_bf16x2(__uint_as_float(v[8 * e + 6]) * inv, __uint_as_float(v[8 * e + 7]) * inv);
                        *reinterpret_cast<uint4 *>(orow + 32 * cc + 8 * e) = u;
                    }
                }
            }
            // rows whose sum is 0 or not finite, or that hold a value that is not
            uint32_t mend = __ballot_sync(0xFFFFFFFFu, qi < len && !(finite > 0.f && finite <= FLT_MAX));
            __syncwarp();
            while (mend) {
                const int r = __ffs(mend) - 1;
                mend &= mend - 1;
                mend_row<HD, BIAS>(p, bias, off, len, h, r0 + r);
            }
        }
    }
    if (!ok) atomicExch(&g_span_err, 1);
    tc_fence_before();
    __syncthreads();
    if (warp == L::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tbase, L::COLS);
    }
}

template <int HD, int TL, bool BIAS>
te_status launch(const SpanParams &p, cudaStream_t stream) {
    using L = SLayout<HD, TL>;
    constexpr int most = L::TAB_OFF + 1024 +
                         (BIAS ? 4 * (TE_RELPOS_MAX_BUCKETS + 2 * (TE_RELPOS_MAX_DISTANCE + PAD) + 1) : 0);
    const int nb = p.two_sided ? 2 * p.side : p.side;
    const int smem = L::TAB_OFF + 1024 + (BIAS ? 4 * (nb + 2 * (p.reach + PAD) + 1) : 0);
    static std::atomic<bool> ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cuda_fail(e, "attn: device");
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(attn_span_kernel<HD, TL, BIAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return cuda_fail(e, "attn: set shared memory size");
        ready[dev] = true;
    }
    const int64_t slots = p.nwork ? p.nwork : (int64_t)p.total / (TL * BQ) + p.nseq;
    if (slots * p.nq > 2147483647) return fail(TE_ESHAPE, "attn: too many query blocks and heads");
    e = launch_close(attn_span_kernel<HD, TL, BIAS>, dim3((unsigned)(slots * p.nq)), L::NTHREADS, smem, stream, 1, p);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "attn launch");
}

// --------------------------------------------- buckets of relative positions

// Whole numbers below 2^3072, for the borders of the buckets: products and
// comparisons only.
struct Whole {
    uint32_t w[96];
    int n;
    explicit Whole(uint32_t v) : n(1) { w[0] = v; }
    void times(uint32_t f) {
        uint64_t carry = 0;
        for (int i = 0; i < n; ++i) {
            carry += (uint64_t)w[i] * f;
            w[i] = (uint32_t)carry;
            carry >>= 32;
        }
        if (carry) w[n++] = (uint32_t)carry;
    }
    void times_power(uint32_t f, int k) {
        for (; k > 0; --k) times(f);
    }
    bool at_least(const Whole &o) const {
        if (n != o.n) return n > o.n;
        for (int i = n - 1; i >= 0; --i)
            if (w[i] != o.w[i]) return w[i] > o.w[i];
        return true;
    }
};

// Does distance d reach bucket exact + k of a side with n logarithmic buckets:
// (d / exact)^n >= (far / exact)^k, so d^n >= far^k exact^(n - k).  Factors are at
// most 2^11 and n at most 256: 2816 bits.
bool reaches(int d, int exact, int far, int n, int k) {
    Whole a(1), b(1);
    a.times_power((uint32_t)d, n);
    b.times_power((uint32_t)far, k);
    b.times_power((uint32_t)exact, n - k);
    return a.at_least(b);
}

te_status check_relpos(const te_relpos *plan, const char *name) {
    const int side = plan->two_sided ? plan->buckets / 2 : plan->buckets;
    bool good = (plan->two_sided == 0 || (plan->two_sided == 1 && plan->buckets % 2 == 0)) && side >= 2 &&
                plan->buckets <= TE_RELPOS_MAX_BUCKETS && plan->first[0] == 0 && plan->reach == plan->first[side - 1] &&
                plan->reach <= TE_RELPOS_MAX_DISTANCE;
    for (int b = 1; good && b < side; ++b) good = plan->first[b] >= plan->first[b - 1];
    return good ? TE_OK : fail(TE_EINVAL, "%s: the plan was not filled by te_relpos_init", name);
}

// The (sequence, query block) pairs, those with the most key tiles first; none
// when there are more than MAX_WORK (the kernel then finds its block itself).
int build_work(const int32_t *cu, int32_t nseq, const SpanParams &p, int qb, uint32_t *work) {
    int64_t n = 0;
    for (int32_t s = 0; s < nseq; ++s) {
        n += (cu[s + 1] - cu[s] + qb - 1) / qb;
        if (n > MAX_WORK) return 0;
    }
    uint64_t key[MAX_WORK];   // (most - cost) << 32 | place in packed order: a stable order by cost
    uint32_t at[MAX_WORK];
    int k = 0;
    for (int32_t s = 0; s < nseq; ++s) {
        const int32_t len = cu[s + 1] - cu[s];
        for (int32_t b = 0; b * qb < len; ++b, ++k) {
            const int64_t r0 = (int64_t)b * qb, r1 = std::min<int64_t>(r0 + qb, len) - 1;
            const int64_t lo = std::max<int64_t>(0, r0 - p.left), hi = std::min<int64_t>(len, r1 + p.right + 1);
            const int64_t keys = hi - lo + std::min<int64_t>(p.sinks, lo);
            const uint64_t cost = (uint64_t)(keys * std::min<int64_t>(r1 - r0 + 1, BQ));   // < 2^38
            key[k] = (((1ull << 40) - cost) << 20) | (uint64_t)k;
            at[k] = ((uint32_t)s << 16) | (uint32_t)b;
        }
    }
    std::sort(key, key + k);
    for (int i = 0; i < k; ++i) work[i] = at[key[i] & 0xFFFFF];
    return k;
}

te_status span_fwd(const char *name, const void *qkv, int64_t ld, int32_t q_off, int32_t k_off, int32_t v_off,
                   const int32_t *cu_host, const int32_t *cu_dev, int32_t nseq, int32_t nq, int32_t nkv, int32_t hd,
                   int32_t left, int32_t right, int32_t sinks, float scale, const te_relpos *plan, const float *table,
                   int64_t ldt, void *out, int64_t ldo, te_stream stream) {
    if (!qkv || !out) return fail(TE_EINVAL, "%s: NULL qkv or out", name);
    if (hd != 64 && hd != 128) return fail(TE_ESHAPE, "%s: hd=%d (64 or 128)", name, hd);
    if (nq < 1 || nkv < 1 || nq % nkv || nq > 65535)
        return fail(TE_ESHAPE, "%s: nq_heads=%d nkv_heads=%d (nq %% nkv == 0, at most 65535)", name, nq, nkv);
    if (left < -1 || right < -1 || sinks < 0)
        return fail(TE_EINVAL, "%s: left=%d right=%d sinks=%d (limits >= 0 or -1, sinks >= 0)", name, left, right, sinks);
    // a power of two to either side of which scores in log2 units stay normal numbers
    if (!(scale >= 0x1p-100f && scale <= 0x1p100f)) return fail(TE_EINVAL, "%s: scale=%g (2^-100 .. 2^100)", name, (double)scale);
    if (q_off < 0 || k_off < 0 || v_off < 0 || (int64_t)q_off + (int64_t)nq * hd > ld ||
        (int64_t)k_off + (int64_t)nkv * hd > ld || (int64_t)v_off + (int64_t)nkv * hd > ld)
        return fail(TE_ESHAPE, "%s: head columns run past ld=%lld", name, (long long)ld);
    if (ld > 2147483647) return fail(TE_ESHAPE, "%s: ld=%lld", name, (long long)ld);
    if (ldo < (int64_t)nq * hd || ldo > 2147483647) return fail(TE_ESHAPE, "%s: ldo=%lld, need nq_heads * hd or more", name, (long long)ldo);
    if (!aligned16(qkv) || !aligned16(out) || ld % 8 || ldo % 8 || q_off % 8 || k_off % 8 || v_off % 8)
        return fail(TE_EALIGN, "%s: rows and head offsets must be 16-byte aligned", name);
    int32_t total = 0, max_len = 0;
    te_status st = check_cu(cu_host, cu_dev, nseq, &total, &max_len);
    if (st != TE_OK) return st;
    if (max_len > (1 << 29)) return fail(TE_ESHAPE, "%s: a sequence of %d rows", name, max_len);
    if (plan) {
        if ((st = check_relpos(plan, name)) != TE_OK) return st;
        if (!table) return fail(TE_EINVAL, "%s: NULL table", name);
        if (ldt < nq) return fail(TE_ESHAPE, "%s: ldt=%lld < nq_heads=%d", name, (long long)ldt, nq);
        if (reinterpret_cast<uintptr_t>(table) & 3) return fail(TE_EALIGN, "%s: the table must be 4-byte aligned", name);
    }
    {
        const uintptr_t a0 = reinterpret_cast<uintptr_t>(qkv), a1 = a0 + (uintptr_t)total * ld * 2;
        const uintptr_t b0 = reinterpret_cast<uintptr_t>(out), b1 = b0 + (uintptr_t)total * ldo * 2;
        if (a0 < b1 && b0 < a1) return fail(TE_EINVAL, "%s: out overlaps qkv", name);
    }
    SpanParams p;
    memset(&p, 0, sizeof(p));
    st = make_map_2d(&p.map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, qkv, (uint64_t)ld, (uint64_t)total, (uint64_t)ld * 2,
                     64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TE_OK) return st;
    p.out = reinterpret_cast<__nv_bfloat16 *>(out);
    p.qkv = reinterpret_cast<const __nv_bfloat16 *>(qkv);
    p.cu = cu_dev;
    p.nseq = nseq;
    p.total = total;
    p.nq = nq;
    p.ld = ld;
    p.ldo = ldo;
    p.q_off = q_off;
    p.k_off = k_off;
    p.v_off = v_off;
    p.group = nq / nkv;
    // no limit and limits past every sequence are the same
    p.left = left < 0 || left > max_len ? max_len : left;
    p.right = right < 0 || right > max_len ? max_len : right;
    p.sinks = std::min(sinks, max_len);
    p.scale_log2 = scale * 1.4426950408889634f;
    if (plan) {
        p.table = table;
        p.ldt = ldt;
        p.two_sided = plan->two_sided;
        p.side = plan->two_sided ? plan->buckets / 2 : plan->buckets;
        p.exact = p.side / 2;
        // no pair is further apart than the longest sequence
        p.reach = std::min(plan->reach, max_len);
        p.grow = plan->grow;
        for (int b = 0; b < p.side; ++b) p.first[b] = (uint16_t)plan->first[b];
    }
    // hd = 64: one 128-query tile a CTA, two CTAs an SM; hd = 128: two tiles a CTA
    const int tl = hd == 64 ? 1 : 2;
    p.nwork = build_work(cu_host, nseq, p, tl * BQ, p.work);
    // heads per group: all when every head's K and V fit in KV_ALL_BYTES
    // together, else the kv heads whose K and V make about KV_GROUP_BYTES
    const int64_t kv_head = (int64_t)total * hd * 4;
    int64_t hg = nq;
    if (kv_head * nkv > KV_ALL_BYTES) hg = std::min<int64_t>(nq, std::max<int64_t>(1, KV_GROUP_BYTES / kv_head) * p.group);
    p.hgroup = (int)hg;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (hd == 64) return plan ? launch<64, 1, true>(p, s) : launch<64, 1, false>(p, s);
    return plan ? launch<128, 2, true>(p, s) : launch<128, 2, false>(p, s);
}

}  // namespace

int read_clear_attn_span_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_span_err, sizeof(int)) != cudaSuccess) return -1;
    if (v) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_span_err, &zero, sizeof(int));
    }
    return v;
}

}  // namespace tefwd

using namespace tefwd;

extern "C" te_status te_relpos_init(te_relpos *plan, int32_t buckets, int32_t max_distance, int32_t two_sided) {
    if (!plan) return fail(TE_EINVAL, "relpos_init: NULL plan");
    if (two_sided != 0 && two_sided != 1) return fail(TE_EINVAL, "relpos_init: two_sided=%d (0 or 1)", two_sided);
    if (buckets < (two_sided ? 4 : 2) || buckets > TE_RELPOS_MAX_BUCKETS || (two_sided && buckets % 2))
        return fail(TE_ESHAPE, "relpos_init: buckets=%d (%d to %d%s)", buckets, two_sided ? 4 : 2,
                    TE_RELPOS_MAX_BUCKETS, two_sided ? ", even" : "");
    const int side = two_sided ? buckets / 2 : buckets, exact = side / 2, n = side - exact;
    if (max_distance <= exact || max_distance > TE_RELPOS_MAX_DISTANCE)
        return fail(TE_ESHAPE, "relpos_init: max_distance=%d (%d to %d for these buckets)", max_distance, exact + 1,
                    TE_RELPOS_MAX_DISTANCE);
    te_relpos r;
    memset(&r, 0, sizeof(r));
    r.buckets = buckets;
    r.max_distance = max_distance;
    r.two_sided = two_sided;
    r.grow = (float)(n / log2((double)max_distance / exact));
    for (int b = 0; b <= exact; ++b) r.first[b] = b;
    for (int k = 1; k < n; ++k) {
        // from the power in f64, then to the border in whole numbers
        int d = (int)(exact * pow((double)max_distance / exact, (double)k / n));
        while (d > r.first[exact + k - 1] && reaches(d - 1, exact, max_distance, n, k)) --d;
        while (!reaches(d, exact, max_distance, n, k)) ++d;
        r.first[exact + k] = d;
    }
    r.reach = r.first[side - 1];
    *plan = r;
    return TE_OK;
}

extern "C" size_t te_relpos_size(void) { return sizeof(te_relpos); }

extern "C" te_status te_attn_sink_fwd(const void *qkv, int64_t ld, int32_t q_off, int32_t k_off, int32_t v_off,
                                      const int32_t *cu_host, const int32_t *cu_dev, int32_t nseq, int32_t nq_heads,
                                      int32_t nkv_heads, int32_t hd, int32_t left, int32_t right, int32_t sinks,
                                      float scale, void *out, int64_t ldo, te_stream stream) {
    return span_fwd("attn_sink", qkv, ld, q_off, k_off, v_off, cu_host, cu_dev, nseq, nq_heads, nkv_heads, hd, left,
                    right, sinks, scale, nullptr, nullptr, 0, out, ldo, stream);
}

extern "C" te_status te_attn_relbias_fwd(const void *qkv, int64_t ld, int32_t q_off, int32_t k_off, int32_t v_off,
                                         const int32_t *cu_host, const int32_t *cu_dev, int32_t nseq,
                                         int32_t nq_heads, int32_t nkv_heads, int32_t hd, int32_t left, int32_t right,
                                         int32_t sinks, float scale, const te_relpos *plan, const float *table,
                                         int64_t ldt, void *out, int64_t ldo, te_stream stream) {
    if (!plan) return fail(TE_EINVAL, "attn_relbias: NULL plan");
    return span_fwd("attn_relbias", qkv, ld, q_off, k_off, v_off, cu_host, cu_dev, nseq, nq_heads, nkv_heads, hd, left,
                    right, sinks, scale, plan, table, ldt, out, ldo, stream);
}
