// Products of 8-bit activations (a scale a token) with q8_row weights (a scale
// an output channel):
//
//     y[t, o] = (sx[t] * sum_j x[t, j] w[o, j]) * sw[o]  (+ bias) (+ residual)
//
// grouped over weights that share the activation, and the gated form
// act(g) * u.  The pages' projections ("cortiq-engine 0.7.6
// src/gpu_metal/zimage.rs" Enc::gemm, Enc::block SwiGLU; "cortiq-engine 0.8.39
// src/gpu_metal/egemma2.rs" Prog::mm) with the activation narrowed as the
// weights are.
#include <atomic>
#include <mutex>

#include "common.cuh"

namespace tefwd {
namespace {

constexpr int MAXZ = 4;

struct I8Item {
    const int8_t *w, *w2;          // w2: the up projection of the gated form
    const float *scale, *bias, *scale2, *bias2, *resid;
    void *y;
    long long ldy, ldr;
    int n, ydt, act;
    int tile0;                // first row group
};

struct I8Params {
    const int8_t *x;
    const float *xs;
    long long ldx;
    int m, k, z;
    int sms;                  // SMs of the device
    int ahead;                // small: bytes of each weight row asked for beforehand
    I8Item it[MAXZ];
};

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int j) { return j == 0 ? v.x : (j == 1 ? v.y : (j == 2 ? v.z : v.w)); }

// Few tokens: bound by the weights' bytes, which go from global memory
// straight into tensor-core fragments (the register form mma.sync: at this
// intensity a TMEM pipeline would only add latency).  A CTA takes MT x 16
// weight rows; its ks warps each take every ks-th 128 bytes of k.  The order
// of k inside a product is free as long as both operands share it, so lane
// 4 g + t loads 16 consecutive bytes of rows g and g + 8 at k + 16 t, and of
// tokens g, g + 8, ..., and word j of each is its share of the j-th 16-deep
// product.  Rows and tokens are widened to f16 in registers (exact), five
// instructions a word; D neighbouring slots of 128 bytes are in flight
// meanwhile (a step of all warps apart: 7 tokens, k 3840, n 11520 10.05 us, k
// 10240, n 3840 11.8; neighbours 9.6 and 11.0), and alternate products add into
// separate sums (a chain of dependent products would wait for each one's
// latency).  The warps' sums meet in shared memory, always in the same order.
// Gated: tile 0 is 16 gate rows, tile 1 the same features' up rows.
template <int NT, int MT, bool GATED, int D>
__global__ void __launch_bounds__(256) i8_small_kernel(const __grid_constant__ I8Params p) {
    static_assert(!GATED || MT == 2, "a gate tile and an up tile");
    extern __shared__ float part[];             // [ks][MT * 16 rows][NT * 8 tokens]
    constexpr int ROWS = MT * 16, TOK = NT * 8, F = GATED ? 16 : ROWS, PW = ROWS * TOK;
    constexpr int AS = 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ks = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    int zi = 0;
    while (zi + 1 < p.z && (int)blockIdx.x >= p.it[zi + 1].tile0) ++zi;
    const I8Item &it = p.it[zi];
    const int o0 = ((int)blockIdx.x - it.tile0) * F;
    const int8_t *wp[MT], *xp = p.x + (long long)g * p.ldx + 16 * t;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        wp[i] = (GATED && i == 1 ? it.w2 + (long long)(o0 + g) * p.k : it.w + (long long)(o0 + 16 * i + g) * p.k) + 16 * t;
    uint4 w[D][MT][2][2], x[D][NT][2];
    auto load = [&](uint4 (&wr)[MT][2][2], uint4 (&xr)[NT][2], int k0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = k0 + 64 * h < p.k;  // k is a multiple of 64
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    wr[i][r][h] = in ? __ldcs(reinterpret_cast<const uint4 *>(wp[i] + (long long)(8 * r) * p.k + k0 + 64 * h))
                                     : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                xr[n][h] = in && g + 8 * n < p.m
                               ? *reinterpret_cast<const uint4 *>(xp + (long long)(8 * n) * p.ldx + k0 + 64 * h)
                               : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    float acc[AS][MT][NT][4];
#pragma unroll
    for (int s = 0; s < AS; ++s)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[s][i][n][e] = 0.f;
    if (threadIdx.x < 16 * MT && p.ahead) {
        const int i = threadIdx.x >> 4, r = threadIdx.x & 15;
        l2_prefetch(GATED && i == 1 ? it.w2 + (long long)(o0 + r) * p.k : it.w + (long long)(o0 + 16 * i + r) * p.k,
                    p.ahead);
    }
    prior_wait();
    next_go();
    const int step = 128 * D * ks;
#pragma unroll
    for (int d = 0; d < D; ++d) load(w[d], x[d], 128 * D * warp + 128 * d);
    for (int k0 = 128 * D * warp; k0 < p.k; k0 += step) {
#pragma unroll
        for (int d = 0; d < D; ++d) {           // a slot past k holds zeros
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a[MT][4];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        widen4_f16(word(w[d][i][0][h], j), a[i][0], a[i][2]);
                        widen4_f16(word(w[d][i][1][h], j), a[i][1], a[i][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t b0, b1;
                        widen4_f16(word(x[d][n][h], j), b0, b1);
#pragma unroll
                        for (int i = 0; i < MT; ++i) mma_16x8x16(acc[j % AS][i][n], a[i], b0, b1);
                    }
                }
            if (k0 + step + 128 * d < p.k) load(w[d], x[d], k0 + step + 128 * d);
            else if (k0 + step < p.k) {     // the next pass runs, without this slot
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) w[d][i][0][h] = w[d][i][1][h] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }
#pragma unroll
    for (int s = 1; s < AS; ++s)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[0][i][n][e] += acc[s][i][n][e];
    // lane 4 g + t holds rows g and g + 8 of each tile for tokens 2 t, 2 t + 1
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                *reinterpret_cast<float2 *>(part + warp * PW + (16 * i + 8 * r + g) * TOK + 8 * n + 2 * t) =
                    make_float2(acc[0][i][n][2 * r], acc[0][i][n][2 * r + 1]);
    __syncthreads();
    // outputs, features fastest
    for (int e = threadIdx.x; e < F * p.m; e += blockDim.x) {
        const int f = e % F, tk = e / F, o = o0 + f;
        float a = 0.f, a2 = 0.f;
        for (int i = 0; i < ks; ++i) {
            a += part[i * PW + f * TOK + tk];
            if (GATED) a2 += part[i * PW + (16 + f) * TOK + tk];
        }
        const float sx = p.xs[tk];
        float y = fmaf(a * sx, it.scale[o], it.bias ? it.bias[o] : 0.f);
        if (GATED)
            y = apply_act(y, it.act) * fmaf(a2 * sx, it.scale2[o], it.bias2 ? it.bias2[o] : 0.f);
        else if (it.act != TE_EPI_NONE)
            y = apply_act(y, it.act - 1);
        if (it.resid) y += it.resid[tk * it.ldr + o];
        if (it.ydt == TE_F32)
            static_cast<float *>(it.y)[tk * it.ldy + o] = y;
        else
            static_cast<__nv_bfloat16 *>(it.y)[tk * it.ldy + o] = __float2bfloat16_rn(y);
    }
}

template <int NT, int MT, bool GATED, int D>
te_status small_go(I8Params &p, int groups, cudaStream_t s) {
    int ks = 1;
    while (ks < 8 && (long long)groups * ks < p.sms * 16 && 128 * D * ks < p.k) ks *= 2;
    const cudaError_t e = launch_close(i8_small_kernel<NT, MT, GATED, D>, dim3(groups), 32 * ks,
                                       ks * MT * 16 * NT * 8 * 4, s, 1, p);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "i8_linear launch");
}

// One CTA a group of MT x 16 rows, with as many warps as fill the device (16
// an SM) while each still has a pass of k.  Where eight warps a group do not
// fill it and have several passes, each keeps twice as much in flight (1 token,
// k 10240, n 3840: 10.7 -> 9.0 us; with 720 groups 9.4 -> 10.8).  The weights'
// first 14 MB are asked into L2 before the previous kernel has ended (7 tokens,
// k 3840: n 11520 10.9 -> 10.0 us, n 3840 6.2 -> 5.8; all 44 MB at once take
// 12.3).  Sixteen warps a group: 10.7 -> 12.8 at k 10240.
template <int NT, bool GATED>
struct Small {
    static constexpr int MT = GATED ? 2 : 1;            // tiles of 16 weight rows a group
    static constexpr int D = NT * MT == 1 ? 2 : 1;      // slots in flight
    static constexpr int D2 = NT * MT <= 2 ? 2 * D : D; // where warps are few
};
// The weight-row groups of all items; sets their places.
template <bool GATED>
int small_groups(I8Params &p) {
    int groups = 0;
    for (int i = 0; i < p.z; ++i) {
        p.it[i].tile0 = groups;
        groups += p.it[i].n / 16;
    }
    return groups;
}
template <int NT, bool GATED>
int small_slots(const I8Params &p, int groups) {
    using S = Small<NT, GATED>;
    return (long long)groups * 8 < p.sms * 16 && p.k > 128 * S::D * 8 ? S::D2 : S::D;
}
template <int NT, bool GATED>
te_status small_launch(I8Params &p, int slots, cudaStream_t s) {
    using S = Small<NT, GATED>;
    const int groups = small_groups<GATED>(p);
    const int ahead = (int)((14ll << 20) / ((long long)groups * 16 * S::MT)) & ~15;
    p.ahead = ahead < p.k ? ahead : p.k;
    return slots == S::D ? small_go<NT, S::MT, GATED, S::D>(p, groups, s) : small_go<NT, S::MT, GATED, S::D2>(p, groups, s);
}

// --------------------------------------------------- a middling token count
//
// Up to a few hundred tokens, or more with few features, the products are
// still bound by the weights' bytes or by latency: the wide tiles of the large
// pipeline (q8_linear.cu) leave SMs idle there, and its activation needs a
// widening pass of its own.  Here a CTA takes 128 weight rows (TMEM lanes) x N
// tokens x a share of k, in one launch and without a workspace:
//   * warp 0 streams stages of 128 k by TMA: the int8 weight rows and tokens
//     (128-byte swizzle);
//   * groups of four warps from warp 2 on, a lane quadrant a warp, take the stages in turn and
//     widen them to f16, exactly: the weights into TMEM (the MMA's A operand),
//     the tokens into shared memory in the MMA's 128-byte-swizzled layout (its
//     B operand); several groups, because one stage's chain of load, widening,
//     TMEM store and fence takes longer than its issue slots;
//   * warp 1 issues the MMAs (kind::f16, M = 128, N, K = 16; f32 sums in TMEM);
//   * the CTAs of a cluster share a tile and split k; at the end each sends
//     its partial sums for a run of tokens to the CTA that owns the run (through
//     distributed shared memory), which adds them in the order of k, scales
//     and stores.
// The split makes enough CTAs to fill the SMs, the ring (NS stages, two CTAs
// an SM up to N = 32) keeps enough bytes in flight for HBM.  Every wait is
// bounded; a wait that gives up sets the error word that te_check reads.
template <int N>
struct Mid {
    static constexpr int G = N <= 32 ? 2 : (N <= 64 ? 4 : 3);       // converter groups of 4 warps
    static constexpr int THREADS = 64 + 128 * G;
    static constexpr int NS = N <= 64 ? 4 : 3;              // int8 stages
    static constexpr int NA = N <= 32 ? 3 : G;              // widened stages
    static constexpr int CTAS = N <= 32 ? 2 : 1;            // an SM
    static constexpr int TMEM = 512 / CTAS;
    // A wait for a phase must know that the phase before it is over.  Slots
    // pass between the producer and one group only (NS a multiple of G), and a
    // widened stage's MMAs are complete in order, G of them a turn.
    static_assert(NS % G == 0 && NA >= G, "rings in phase with the groups");
    static constexpr int WBYTES = 128 * 128;                // int8 weights of a stage
    static constexpr int XBYTES = N * 128;                  // int8 tokens of a stage
    static constexpr int SBYTES = WBYTES + XBYTES;
    static constexpr int BBOX = N * 128;                    // 64 k of the widened tokens
    static constexpr int B_OFF = NS * SBYTES;
    static constexpr int BAR_OFF = B_OFF + NA * 2 * BBOX;
    static constexpr int NBAR = 2 * NS + 2 * NA + 1;
    static constexpr int BYTES = BAR_OFF + 8 * NBAR + 16;
    static_assert(SBYTES % 1024 == 0 && BBOX % 1024 == 0, "swizzled tiles stay 1024-byte aligned");
    static_assert(N * 128 * 4 <= B_OFF, "the partial sums reuse the ring");
    static_assert(N + 64 * NA <= TMEM, "TMEM columns");
    static_assert(BYTES + 1024 <= (CTAS == 2 ? 113 : 227) * 1024, "shared memory");
    // A CTA waits for its cluster's others while it holds TMEM.  So its SM must
    // have TMEM for all that fit there, or they end by themselves: two of these
    // (or one and attention's, which waits for nobody) have 256 columns each, and
    // beside the pairs of q8_gemm_kernel (from 179 KB) and mma_peak_kernel (160
    // KB), which hold 512 and wait for one another, there is no room for one.
    static_assert(BYTES + 1024 > 80 * 1024, "no CTA beside a pair's");
};

struct MidParams {
    CUtensorMap tx;                             // x int8 [m, k]
    CUtensorMap tw[MAXZ];                       // weights int8 [n, k]
    I8Item it[MAXZ];
    const float *xs;
    int *err;
    int m, k, z;
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int N, bool GATED>
__global__ void __launch_bounds__(Mid<N>::THREADS) i8_mid_kernel(const __grid_constant__ MidParams p) {
    using L = Mid<N>;
    constexpr int NA = L::NA, NS = L::NS;
    constexpr int F = GATED ? 64 : 128;         // features a tile
    extern __shared__ uint8_t smem_raw[];
    // the same offset in every CTA of a cluster: remote addresses agree
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_full = sb + L::BAR_OFF, bar_empty = bar_full + 8 * NS, bar_afull = bar_empty + 8 * NS,
                   bar_aempty = bar_afull + 8 * NA, bar_done = bar_aempty + 8 * NA;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::BAR_OFF + 8 * L::NBAR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank, csize;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    const int S = (int)csize;
    const int tile = (int)blockIdx.x / S;
    const int t0 = (int)blockIdx.y * N;
    int zi = 0;
    while (zi + 1 < p.z && tile >= p.it[zi + 1].tile0) ++zi;
    const I8Item &it = p.it[zi];
    const int o0 = (tile - it.tile0) * F;
    const int nkb = (p.k + 127) / 128;
    const int kb0 = (int)((long long)nkb * rank / S), cnt = (int)((long long)nkb * (rank + 1) / S) - kb0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 4);    // a group of converter warps
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(bar_afull + 8 * i, 4);
            mbar_init(bar_aempty + 8 * i, 1);   // the MMAs' commit
        }
        mbar_init(bar_done, 1);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), L::TMEM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    prior_wait();
    next_go();
    bool ok = true;

    if (warp == 0) {
        const uint32_t e = elect_one();
        for (int i = 0; i < cnt; ++i) {
            const int s = i % NS;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_empty + 8 * s, ((i / NS) & 1) ^ 1));
            if (!ok) break;
            const uint32_t fb = bar_full + 8 * s, dst = sb + s * L::SBYTES;
            const int k0 = (kb0 + i) * 128;
            mbar_arrive_expect_tx_e(fb, L::SBYTES, e);
            if (GATED) {                        // rows 0-63 gate, 64-127 up
                tma_load_2d_e(dst, &p.tw[0], fb, k0, o0, e);
                tma_load_2d_e(dst + L::WBYTES / 2, &p.tw[1], fb, k0, o0, e);
            } else {
                tma_load_2d_e(dst, &p.tw[zi], fb, k0, o0, e);
            }
            tma_load_2d_e(dst + L::WBYTES, &p.tx, fb, k0, t0, e);
        }
        // no copy of ours may land after the ring changes its use
        for (int j = cnt - NS < 0 ? 0 : cnt - NS; j < cnt; ++j)
            if (!mbar_wait(bar_full + 8 * (j % NS), (j / NS) & 1, 20000000ull)) ok = false;
    } else if (warp == 1) {
        const uint32_t e = elect_one();
        constexpr uint32_t idesc = idesc_f16_f32(128, N);
        for (int i = 0; i < cnt; ++i) {
            const int a = i % NA;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_afull + 8 * a, (i / NA) & 1));
            if (!ok) break;
            tc_fence_after();
            const uint64_t d0 = smem_desc_sw128(sb + L::B_OFF + a * 2 * L::BBOX);
            const uint32_t a0 = tbase + N + 64 * a;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                mma_ts_bf16_e(tbase, a0 + 8 * j, d0 + (uint64_t)(((j >> 2) * L::BBOX + (j & 3) * 32) >> 4), idesc,
                              (uint32_t)(i != 0 || j != 0), e);
            mma_commit_e(bar_aempty + 8 * a, e);
        }
        mma_commit_e(bar_done, e);              // every MMA issued above
        if (!mbar_wait(bar_done, 0, 20000000ull)) ok = false;
    } else {
        const int q = warp & 3, row = 32 * q + lane;
        for (int i = (warp - 2) >> 2; i < cnt; i += L::G) {
            const int s = i % NS, a = i % NA;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_full + 8 * s, (i / NS) & 1) &&
                                             mbar_wait(bar_aempty + 8 * a, ((i / NA) & 1) ^ 1));
            if (!ok) break;
            tc_fence_after();
            const uint8_t *st = smem + s * L::SBYTES;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(st + row * 128 + (((4 * h + c) ^ (row & 7)) << 4));
                    widen4_f16(v.x, r[8 * c + 0], r[8 * c + 1]);
                    widen4_f16(v.y, r[8 * c + 2], r[8 * c + 3]);
                    widen4_f16(v.z, r[8 * c + 4], r[8 * c + 5]);
                    widen4_f16(v.w, r[8 * c + 6], r[8 * c + 7]);
                }
                tmem_st32(tbase + ((uint32_t)(32 * q) << 16) + N + 64 * a + 32 * h, r);
            }
            // tokens: 16-byte piece c of row r becomes pieces 2c, 2c + 1 of
            // 128-byte rows, in the box of its half of k; the two halves' lanes
            // store in opposite order, so that no two hit one bank
#pragma unroll
            for (int j = 0; j < N / 16; ++j) {
                const int id = q * 2 * N + lane + 32 * j;
                const int xr = id >> 3, c = id & 7;
                const uint4 v = *reinterpret_cast<const uint4 *>(st + L::WBYTES + xr * 128 + ((c ^ (xr & 7)) << 4));
                uint4 lo, hi;
                widen4_f16(v.x, lo.x, lo.y);
                widen4_f16(v.y, lo.z, lo.w);
                widen4_f16(v.z, hi.x, hi.y);
                widen4_f16(v.w, hi.z, hi.w);
                uint8_t *box = smem + L::B_OFF + a * 2 * L::BBOX + (c >> 2) * L::BBOX + xr * 128;
                const int p0 = 2 * (c & 3), first = c >> 2;
                *reinterpret_cast<uint4 *>(box + (((p0 + first) ^ (xr & 7)) << 4)) = first ? hi : lo;
                *reinterpret_cast<uint4 *>(box + (((p0 + 1 - first) ^ (xr & 7)) << 4)) = first ? lo : hi;
            }
            fence_async_smem();                 // the B tile, visible to the MMA
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_afull + 8 * a);
                mbar_arrive(bar_empty + 8 * s);
            }
        }
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar_done, 0));
        tc_fence_after();
    }
    if (!ok && lane == 0) atomicExch(p.err, 1);
    __syncwarp();

    // Partial sums to the owners: token run d of TC tokens goes to CTA d, as
    // [source CTA][token][128 rows].  All pipelines are done with their rings first.
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const int tn = p.m - t0 < N ? p.m - t0 : N; // tokens of this tile
    const int TC = (tn + S - 1) / S;
    if (warp >= 2 && warp < 10 && cnt > 0) {
        const int q = warp & 3, h = (warp - 2) >> 2;
        int d = h * (N / 2) / TC, tl = h * (N / 2) - d * TC;    // owner and place of the next token
        const uint32_t mine = sb + (uint32_t)(((int)rank * TC * 128 + 32 * q + lane) * 4);
        uint32_t to = mapa_shared(mine, d < S ? d : 0);
        constexpr int LD = N >= 64 ? 4 : N / 16;    // TMEM loads in flight, 8 columns each
#pragma unroll
        for (int c8 = 0; c8 < N / 16; c8 += LD) {
            const int c0 = h * (N / 2) + 8 * c8;
            if (c0 >= tn) break;                // warp-uniform
            uint32_t v[LD][8];
#pragma unroll
            for (int i = 0; i < LD; ++i) tmem_ld8(tbase + ((uint32_t)(32 * q) << 16) + c0 + 8 * i, v[i]);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8 * LD; ++j) {
                if (c0 + j < tn) st_cluster_f32(to + 512 * tl, __uint_as_float(v[j / 8][j % 8]));
                if (++tl == TC) {
                    tl = 0;
                    to = mapa_shared(mine, ++d < S ? d : 0);
                }
            }
        }
    }
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, L::TMEM);
    }
    // Sums, scales and stores: a lane keeps 4 features (their scales and biases
    // in registers), a warp takes a token (gated: two) at a time.
    const int own = tn - (int)rank * TC < TC ? tn - (int)rank * TC : TC;
    constexpr int LPT = F / 4;                  // lanes a token
    const int f = 4 * (lane % LPT), o = o0 + f;
    if (o >= it.n) return;                      // n is a multiple of 32
    float4 sc, bi = make_float4(0.f, 0.f, 0.f, 0.f), sc2 = bi, bi2 = bi;
    sc = make_float4(it.scale[o], it.scale[o + 1], it.scale[o + 2], it.scale[o + 3]);
    if (it.bias) bi = make_float4(it.bias[o], it.bias[o + 1], it.bias[o + 2], it.bias[o + 3]);
    if (GATED) {
        sc2 = make_float4(it.scale2[o], it.scale2[o + 1], it.scale2[o + 2], it.scale2[o + 3]);
        if (it.bias2) bi2 = make_float4(it.bias2[o], it.bias2[o + 1], it.bias2[o + 2], it.bias2[o + 3]);
    }
    for (int tl = warp * (32 / LPT) + lane / LPT; tl < own; tl += (L::THREADS / 32) * (32 / LPT)) {
        const long long t = t0 + (int)rank * TC + tl;
        const float sx = p.xs[t];
        const float *b = reinterpret_cast<const float *>(smem) + tl * 128 + f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), u = a;
        for (int i = 0; i < S; ++i, b += TC * 128) {
            const float4 v = *reinterpret_cast<const float4 *>(b);
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
            if (GATED) {
                const float4 v2 = *reinterpret_cast<const float4 *>(b + 64);
                u.x += v2.x; u.y += v2.y; u.z += v2.z; u.w += v2.w;
            }
        }
        float y[4] = {fmaf(a.x * sx, sc.x, bi.x), fmaf(a.y * sx, sc.y, bi.y), fmaf(a.z * sx, sc.z, bi.z),
                      fmaf(a.w * sx, sc.w, bi.w)};
        if (GATED) {
            const float w[4] = {fmaf(u.x * sx, sc2.x, bi2.x), fmaf(u.y * sx, sc2.y, bi2.y),
                                fmaf(u.z * sx, sc2.z, bi2.z), fmaf(u.w * sx, sc2.w, bi2.w)};
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = apply_act(y[j], it.act) * w[j];
        } else if (it.act != TE_EPI_NONE) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = apply_act(y[j], it.act - 1);
        }
        if (it.resid) {
            const float4 r = *reinterpret_cast<const float4 *>(it.resid + t * it.ldr + o);
            y[0] += r.x; y[1] += r.y; y[2] += r.z; y[3] += r.w;
        }
        if (it.ydt == TE_F32)
            *reinterpret_cast<float4 *>(static_cast<float *>(it.y) + t * it.ldy + o) =
                make_float4(y[0], y[1], y[2], y[3]);
        else
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(it.y) + t * it.ldy + o) =
                make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
}

// A choice of token tile and split of k, and its time by the model below.
struct MidPlan {
    int n, split;
    double us;
};

// Device time of the mid kernel, fitted to single calls on cold weights: a
// wave of CTAs costs `start` us and `stage` us a stage of 128 k.  Splitting k
// shortens the stages of a CTA while the clusters still fit the device at once;
// clusters of `split` CTAs sit inside a GPC, so fewer CTAs are resident at
// larger splits (residents: asked of the runtime).
template <int N>
void mid_consider(MidPlan &best, int ftiles, int m, int nkb, const int *residents) {
    constexpr double start = N <= 16 ? 4.2 : (N <= 32 ? 4.6 : (N <= 64 ? 5.5 : 6.5));
    constexpr double stage = N <= 16 ? 0.5 : (N <= 32 ? 0.55 : (N <= 64 ? 0.65 : 0.8));
    const long long ttiles = ((long long)m + N - 1) / N, tiles = ftiles * ttiles;
    if (ttiles > 65535) return;                 // a grid's second axis
    for (int s = 1; s <= 8 && s <= nkb; s *= 2) {
        const int r = residents[s] > 0 ? residents[s] : 1;
        const double us = (double)((tiles + r - 1) / r) * (start + stage * ((nkb + s - 1) / s));
        if (us < best.us) best = {N, s, us};
    }
}

// Resident clusters of 1, 2, 4 and 8 CTAs of the kernel on the current device,
// asked for once (and its shared memory size set).  A device's row is read only
// once it is whole: first calls may come from several threads.
template <int N, bool GATED>
te_status mid_residents(const int *&out) {
    static int table[64][9] = {};
    static std::atomic<bool> whole[64] = {};
    static std::mutex filling;
    constexpr int smem = Mid<N>::BYTES + 1024;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cuda_fail(e, "i8_linear: device");
    int *t = table[dev];
    out = t;
    if (whole[dev].load(std::memory_order_acquire)) return TE_OK;
    const std::lock_guard<std::mutex> lock(filling);
    if (whole[dev].load(std::memory_order_relaxed)) return TE_OK;
    e = cudaFuncSetAttribute(i8_mid_kernel<N, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(e, "i8_linear: set shared memory size");
    for (int s = 8; s >= 1; s /= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(8 * sm_count(), 1, 1);
        cfg.blockDim = dim3(Mid<N>::THREADS, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = s;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, i8_mid_kernel<N, GATED>, &cfg);
        if (e != cudaSuccess || n < 1) return cuda_fail(e, "i8_linear: cluster occupancy");
        t[s] = n;
    }
    whole[dev].store(true, std::memory_order_release);
    return TE_OK;
}

template <bool GATED>
te_status mid_plan(MidPlan &best, int ftiles, int m, int k) {
    const int nkb = (k + 127) / 128;
    const int *r16, *r32, *r64, *r128;
    te_status st;
    if ((st = mid_residents<16, GATED>(r16)) != TE_OK || (st = mid_residents<32, GATED>(r32)) != TE_OK ||
        (st = mid_residents<64, GATED>(r64)) != TE_OK || (st = mid_residents<128, GATED>(r128)) != TE_OK)
        return st;
    best = {0, 1, 1e30};
    mid_consider<16>(best, ftiles, m, nkb, r16);
    mid_consider<32>(best, ftiles, m, nkb, r32);
    mid_consider<64>(best, ftiles, m, nkb, r64);
    mid_consider<128>(best, ftiles, m, nkb, r128);
    return TE_OK;
}

template <int N, bool GATED>
te_status mid_launch(const I8Params &q, int S, cudaStream_t s) {
    constexpr int F = GATED ? 64 : 128, smem = Mid<N>::BYTES + 1024;
    MidParams p;
    memset(&p, 0, sizeof(p));
    const int *residents;                       // asked for, so its shared memory size is set
    te_status st = mid_residents<N, GATED>(residents);
    if (st != TE_OK) return st;
    st = make_map_2d(&p.tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.x, (uint64_t)q.k, (uint64_t)q.m, (uint64_t)q.ldx, 128, N,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    int tiles = 0;
    for (int i = 0; i < q.z && st == TE_OK; ++i) {
        p.it[i] = q.it[i];
        p.it[i].tile0 = tiles;
        tiles += (q.it[i].n + F - 1) / F;
        st = make_map_2d(&p.tw[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, q.it[i].w, (uint64_t)q.k, (uint64_t)q.it[i].n,
                         (uint64_t)q.k, 128, F, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (GATED && st == TE_OK)
        st = make_map_2d(&p.tw[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, q.it[0].w2, (uint64_t)q.k, (uint64_t)q.it[0].n,
                         (uint64_t)q.k, 128, F, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TE_OK) return st;
    p.xs = q.xs;
    p.m = q.m;
    p.k = q.k;
    p.z = q.z;
    if ((st = gemm_error_word(&p.err)) != TE_OK) return st;
    const int ttiles = (q.m + N - 1) / N;
    const cudaError_t e = launch_close(i8_mid_kernel<N, GATED>, dim3(tiles * S, ttiles), Mid<N>::THREADS, smem, s, S, p);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "i8_linear launch");
}

// ------------------------------------------------ many tokens, short k (k <= 512)
//
// The widened weights of 128 features stay in shared memory (k x 256 bytes)
// while a CTA's run of token tiles passes: per tile it loads the int8 tokens
// only, widens them into TMEM and drains 128 x 128 outputs.  Against the large
// pipeline with its separate widening pass that saves the pass and its f16 copy
// of the tokens, which at short k cost as much as the product.  Tokens are the
// MMA's A operand (TMEM) and weights its B (shared memory): shared-memory
// bandwidth bounds the tile, and what is widened for every tile then costs a
// load and no store there.  (The other way round, weights in TMEM, a tile at
// k = 512 moved 512 KB through shared memory and took 5500 cycles.)
//   * persistent CTAs, one an SM; units are (128 features, 128 tokens), features
//     outermost; a CTA takes a contiguous run and reloads its weights where the
//     run crosses into the next features;
//   * warp 0: TMA, one ring of 128 x 128-byte chunks for weights and tokens;
//   * warps 2-9 widen every chunk together, in order: weights into shared memory
//     in the MMA's 128-byte-swizzled layout, tokens into a ring of TMEM stages
//     (two warps a lane quadrant);
//   * warp 1: MMAs, kind::f16, M = 128, N = 128, into alternating accumulators;
//   * warps 10-17 drain the other accumulator: lane = token, half of the features
//     a warp, scaled in f32 pairs, written to a staging block in the swizzled
//     layout of the TMA store that sends it (a reduce-add where y is its own
//     residual), two blocks in turn.
// Gated: columns 0-63 are gate features, 64-127 the same features' up rows, so
// a lane holds both of a pair.  Waits are bounded as everywhere.
struct ResParams {
    CUtensorMap tx;
    CUtensorMap tw[MAXZ];
    CUtensorMap ty[MAXZ];     // y_i: boxes of 32 features x 32 tokens
    I8Item it[MAXZ];
    const float *xs;
    int *err;
    int m, k, z, ttiles, units;
};
struct Res {
    static constexpr int NS = 4;                // int8 chunks
    static constexpr int NA = 4;                // TMEM stages of widened tokens
    static constexpr int CHUNK = 128 * 128;     // int8 chunk
    static constexpr int BBOX = 128 * 128;      // 64 k of 128 widened weight rows
    static constexpr int B_OFF = NS * CHUNK;
    static constexpr int FAC_OFF = B_OFF + 8 * BBOX;            // scale and bias of the tile's 128 columns
    static constexpr int STG_OFF = FAC_OFF + 2 * 128 * 4;
    static constexpr int STG = 4096;            // an output block of a draining warp (f32 32 x 32)
    static constexpr int BAR_OFF = STG_OFF + 8 * STG;
    static constexpr int NBAR = 2 * NS + 2 * NA + 2 + 4 + 2 + 1;
    static constexpr int BYTES = BAR_OFF + 8 * NBAR + 16;
    static constexpr int THREADS = 18 * 32;
    static constexpr int A_COL = 256;           // TMEM: two accumulators of 128 columns, then the stages
    static_assert(STG_OFF % 1024 == 0 && B_OFF % 1024 == 0, "swizzled tiles");
    static_assert(BYTES + 1024 <= 227 * 1024, "shared memory");
};

template <bool GATED>
__global__ void __launch_bounds__(Res::THREADS, 1) i8_res_kernel(const __grid_constant__ ResParams p) {
    using L = Res;
    constexpr int NS = L::NS, NA = L::NA, F = GATED ? 64 : 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar_full = sb + L::BAR_OFF, bar_empty = bar_full + 8 * NS, bar_afull = bar_empty + 8 * NS,
                   bar_aempty = bar_afull + 8 * NA, bar_wfull = bar_aempty + 8 * NA, bar_wempty = bar_wfull + 8,
                   bar_accfull = bar_wempty + 8, bar_accempty = bar_accfull + 16, bar_ffull = bar_accempty + 16,
                   bar_fempty = bar_ffull + 8, bar_done = bar_fempty + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::BAR_OFF + 8 * L::NBAR);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nkb = (p.k + 127) / 128;
    const int u0 = (int)((long long)p.units * blockIdx.x / gridDim.x);
    const int u1 = (int)((long long)p.units * (blockIdx.x + 1) / gridDim.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 8);
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(bar_afull + 8 * i, 8);
            mbar_init(bar_aempty + 8 * i, 1);
        }
        mbar_init(bar_wfull, 8);
        mbar_init(bar_wempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_accfull + 8 * i, 1);
            mbar_init(bar_accempty + 8 * i, 8);
        }
        mbar_init(bar_ffull, 8);
        mbar_init(bar_fempty, 8);
        mbar_init(bar_done, 1);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const int ft0 = u0 / p.ttiles, tt0 = u0 - ft0 * p.ttiles;
    auto item_of = [&](int ft) {
        int zi = 0;
        while (zi + 1 < p.z && ft >= p.it[zi + 1].tile0) ++zi;
        return zi;
    };
    // The tile's weights, by its first CTA (16238 x 512 x 512 f32: 14.0 -> 13.7 us;
    // by every CTA 14.1).
    if (threadIdx.x < 128 && u0 < u1 && tt0 == 0) {
        const I8Item &it = p.it[item_of(ft0)];
        const int r = threadIdx.x, o = (ft0 - it.tile0) * F + (GATED ? r & 63 : r);
        if (o < it.n) l2_prefetch((GATED && r >= 64 ? it.w2 : it.w) + (long long)o * p.k, p.k);
    }
    prior_wait();
    bool ok = true;
    // unit u is (feature tile ft, token tile tt); it brings new weights where a
    // run or a feature tile begins
    auto next = [&](int &ft, int &tt) {
        if (++tt == p.ttiles) {
            tt = 0;
            ++ft;
        }
    };

    if (warp == 0) {
        const uint32_t e = elect_one();
        if (e) tma_prefetch_desc(&p.tx);
        int ci = 0;
        auto slot = [&]() {                     // the next free chunk of the ring
            const int s = ci % NS;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_empty + 8 * s, ((ci / NS) & 1) ^ 1));
            if (ok) mbar_arrive_expect_tx_e(bar_full + 8 * s, L::CHUNK, e);
            return s;
        };
        for (int u = u0, ft = ft0, tt = tt0; u < u1 && ok; ++u, next(ft, tt)) {
            if (u == u0 || tt == 0) {
                const int zi = item_of(ft), o0 = (ft - p.it[zi].tile0) * F;
                for (int kb = 0; kb < nkb; ++kb, ++ci) {
                    const int s = slot();
                    if (!ok) break;
                    if (GATED) {                // rows 0-63 gate, 64-127 up
                        tma_load_2d_e(sb + s * L::CHUNK, &p.tw[0], bar_full + 8 * s, kb * 128, o0, e);
                        tma_load_2d_e(sb + s * L::CHUNK + L::CHUNK / 2, &p.tw[1], bar_full + 8 * s, kb * 128, o0, e);
                    } else {
                        tma_load_2d_e(sb + s * L::CHUNK, &p.tw[zi], bar_full + 8 * s, kb * 128, o0, e);
                    }
                }
            }
            if (u + 1 == u1) next_go();
            for (int kb = 0; kb < nkb && ok; ++kb, ++ci) {
                const int s = slot();
                if (ok) tma_load_2d_e(sb + s * L::CHUNK, &p.tx, bar_full + 8 * s, kb * 128, tt * 128, e);
            }
        }
        for (int j = ci - NS < 0 ? 0 : ci - NS; j < ci; ++j)    // no copy of ours lands after the CTA's end
            mbar_wait(bar_full + 8 * (j % NS), (j / NS) & 1, 20000000ull);
    } else if (warp == 1) {
        const uint32_t e = elect_one();
        constexpr uint32_t idesc = idesc_f16_f32(128, 128);
        int xi = 0, nfill = 0;
        for (int u = u0, ft = ft0, tt = tt0; u < u1 && ok; ++u, next(ft, tt)) {
            const int i = u - u0, b = i & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_accempty + 8 * b, ((i >> 1) & 1) ^ 1));
            if (ok && (u == u0 || tt == 0)) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_wfull, nfill++ & 1));
            for (int kb = 0; kb < nkb && ok; ++kb, ++xi) {
                const int s = xi % NA;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_afull + 8 * s, (xi / NA) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint64_t d0 = smem_desc_sw128(sb + L::B_OFF + kb * 2 * L::BBOX);
                const uint32_t a0 = tbase + L::A_COL + 64 * s;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    mma_ts_bf16_e(tbase + 128 * b, a0 + 8 * j, d0 + (uint64_t)(((j >> 2) * L::BBOX + (j & 3) * 32) >> 4),
                                  idesc, (uint32_t)(kb != 0 || j != 0), e);
                mma_commit_e(bar_aempty + 8 * s, e);
            }
            if (!ok) break;
            mma_commit_e(bar_accfull + 8 * b, e);
            // the last unit on these weights: they may be replaced
            if (u + 1 < u1 && tt + 1 == p.ttiles) mma_commit_e(bar_wempty, e);
        }
        mma_commit_e(bar_done, e);              // every MMA issued above
        if (!mbar_wait(bar_done, 0, 20000000ull)) ok = false;
    } else if (warp < 10) {
        const int q = warp & 3, h = (warp - 2) >> 2, row = 32 * q + lane;
        // Weights: the warp widens 16 rows of a chunk, lane l the 16-byte piece
        // c = l % 8 of rows l / 8 + 4 j.  Piece c becomes pieces 2c, 2c + 1 of
        // 128-byte rows in the box of its half of k, all swizzled by the row (row
        // + 4 flips bit 6 of the offset); the halves' lanes store in opposite
        // order, so that no two hit one bank.
        const int wr = 16 * (warp - 2) + (lane >> 3), wc = lane & 7, whi = wc >> 2;
        const int wrow = wr * 128, ws0 = (wc ^ (wr & 7)) << 4, wbox = whi * L::BBOX + wr * 128;
        const int wd0 = ((2 * (wc & 3) + whi) ^ (wr & 7)) << 4, wd1 = ((2 * (wc & 3) + 1 - whi) ^ (wr & 7)) << 4;
        int ci = 0, xi = 0, nfill = 0;
        for (int u = u0, ft = ft0, tt = tt0; u < u1 && ok; ++u, next(ft, tt)) {
            if (u == u0 || tt == 0) {
                // the factors of the tile's columns: this warp's 16, once the drain
                // of the features before is over
                if (nfill) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_fempty, (nfill - 1) & 1));
                if (!ok) break;
                {
                    const I8Item &it = p.it[item_of(ft)];
                    const int c = 16 * (warp - 2) + (lane & 15), o = (ft - it.tile0) * F + (GATED ? c & 63 : c);
                    const bool up = GATED && c >= 64;
                    const float *src = lane < 16 ? (up ? it.scale2 : it.scale) : (up ? it.bias2 : it.bias);
                    reinterpret_cast<float *>(smem + L::FAC_OFF)[(lane < 16 ? 0 : 128) + c] =
                        o < it.n && src ? src[o] : 0.f;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_ffull);
                }
                // the MMAs on the weights before are complete
                if (nfill) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_wempty, (nfill - 1) & 1));
                ++nfill;
                for (int kb = 0; kb < nkb && ok; ++kb, ++ci) {
                    const int s = ci % NS;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_full + 8 * s, (ci / NS) & 1));
                    if (!ok) break;
                    const uint8_t *src = smem + s * L::CHUNK + wrow;
                    uint8_t *dst = smem + L::B_OFF + kb * 2 * L::BBOX + wbox;
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = *reinterpret_cast<const uint4 *>(src + 512 * j + (ws0 ^ (64 * (j & 1))));
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint4 lo, hi;
                        widen4_f16(v[j].x, lo.x, lo.y);
                        widen4_f16(v[j].y, lo.z, lo.w);
                        widen4_f16(v[j].z, hi.x, hi.y);
                        widen4_f16(v[j].w, hi.z, hi.w);
                        *reinterpret_cast<uint4 *>(dst + 512 * j + (wd0 ^ (64 * (j & 1)))) = whi ? hi : lo;
                        *reinterpret_cast<uint4 *>(dst + 512 * j + (wd1 ^ (64 * (j & 1)))) = whi ? lo : hi;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_empty + 8 * s);
                }
                fence_async_smem();             // the weights, visible to the MMAs
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(bar_wfull);
            }
            for (int kb = 0; kb < nkb && ok; ++kb, ++ci, ++xi) {
                const int s = ci % NS, a = xi % NA;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_full + 8 * s, (ci / NS) & 1));
                if (!ok) break;
                uint32_t r[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(smem + s * L::CHUNK + row * 128 +
                                                                     (((4 * h + c) ^ (row & 7)) << 4));
                    widen4_f16(v.x, r[8 * c + 0], r[8 * c + 1]);
                    widen4_f16(v.y, r[8 * c + 2], r[8 * c + 3]);
                    widen4_f16(v.z, r[8 * c + 4], r[8 * c + 5]);
                    widen4_f16(v.w, r[8 * c + 6], r[8 * c + 7]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_empty + 8 * s);
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_aempty + 8 * a, ((xi / NA) & 1) ^ 1));
                if (!ok) break;
                tc_fence_after();
                tmem_st32(tbase + ((uint32_t)(32 * q) << 16) + L::A_COL + 64 * a + 32 * h, r);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_afull + 8 * a);
            }
        }
    } else {
        const int q = warp & 3, h = (warp - 10) >> 2;
        const float *fac = reinterpret_cast<const float *>(smem + L::FAC_OFF);
        uint8_t *stg = smem + L::STG_OFF + (warp - 10) * L::STG;
        int nfill = 0, last_bytes = 0, turn = 0;
        // The next staging block of `bytes` (2 KB blocks in two halves; a 4 KB
        // block, or a change of size, waits for all stores before).
        auto block = [&](int bytes) {
            if (lane == 0) {
                if (bytes == L::STG || bytes != last_bytes) bulk_wait_read_n<0>();
                else bulk_wait_read_n<1>();
            }
            __syncwarp();
            last_bytes = bytes;
            return stg + (bytes == L::STG ? 0 : (turn++ & 1) * (L::STG / 2));
        };
        const uint32_t trow = (uint32_t)(32 * q) << 16;
        float nts = tt0 * 128 + 32 * q + lane < p.m ? p.xs[tt0 * 128 + 32 * q + lane] : 0.f;
        for (int u = u0, ft = ft0, tt = tt0; u < u1 && ok; ++u, next(ft, tt)) {
            const int i = u - u0, b = i & 1;
            const int zi = item_of(ft);
            const I8Item &it = p.it[zi];
            const int tb = tt * 128 + 32 * q;   // this warp's tokens
            const int t = tb + lane;
            const bool f32 = it.ydt == TE_F32, inplace = it.resid != nullptr && it.resid == it.y;
            const float ts = nts;
            if (u + 1 < u1) {                   // the next tile's token scale
                int fn = ft, tn = tt;
                next(fn, tn);
                nts = tn * 128 + 32 * q + lane < p.m ? p.xs[tn * 128 + 32 * q + lane] : 0.f;
            }
            if (u == u0 || tt == 0) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_ffull, nfill++ & 1));
            if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar_accfull + 8 * b, (i >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const uint64_t ts2 = f2_pack(ts, ts);
            // (acc * ts) * scale + bias of v's columns, from column c on, in place
            auto scaled = [&](auto &v, int c) {
#pragma unroll
                for (int j = 0; j < (int)(sizeof(v) / 4); j += 4) {
                    const float4 s4 = *reinterpret_cast<const float4 *>(fac + c + j);
                    const float4 b4 = *reinterpret_cast<const float4 *>(fac + 128 + c + j);
                    const uint64_t y0 = f2_fma(f2_mul(f2_pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), ts2),
                                               f2_pack(s4.x, s4.y), f2_pack(b4.x, b4.y));
                    const uint64_t y1 = f2_fma(f2_mul(f2_pack(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), ts2),
                                               f2_pack(s4.z, s4.w), f2_pack(b4.z, b4.w));
                    float a0, a1, a2, a3;
                    f2_unpack(y0, a0, a1);
                    f2_unpack(y1, a2, a3);
                    v[j] = __float_as_uint(a0);
                    v[j + 1] = __float_as_uint(a1);
                    v[j + 2] = __float_as_uint(a2);
                    v[j + 3] = __float_as_uint(a3);
                }
            };
            // 32 tokens x 32 features as bf16: 64-byte rows, 64-byte swizzle
            auto send_bf16 = [&](const uint8_t *st, int fo) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&p.ty[zi], smem_u32(st), fo, tb);
                    bulk_commit();
                }
            };
            auto store_bf16 = [&](const uint32_t (&v)[32], int fo) {
                uint8_t *st = block(2048);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 w;
                    w.x = pack_bf16x2(__uint_as_float(v[8 * c]), __uint_as_float(v[8 * c + 1]));
                    w.y = pack_bf16x2(__uint_as_float(v[8 * c + 2]), __uint_as_float(v[8 * c + 3]));
                    w.z = pack_bf16x2(__uint_as_float(v[8 * c + 4]), __uint_as_float(v[8 * c + 5]));
                    w.w = pack_bf16x2(__uint_as_float(v[8 * c + 6]), __uint_as_float(v[8 * c + 7]));
                    *reinterpret_cast<uint4 *>(st + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = w;
                }
                send_bf16(st, fo);
            };
            const bool any = tb < p.m;          // warp-uniform
            if constexpr (GATED) {
                // 16 features at a time: with 32 the registers spill
                const int fo = (ft - it.tile0) * F + 32 * h;
                const bool out = any && fo < it.n;
                uint8_t *st = out ? block(2048) : stg;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t g[16], up[16];
                    if (any) {
                        tmem_ld16(tbase + trow + 128 * b + 32 * h + 16 * c, g);
                        tmem_ld16(tbase + trow + 128 * b + 64 + 32 * h + 16 * c, up);
                        tmem_wait_ld();
                        scaled(g, 32 * h + 16 * c);
                        scaled(up, 64 + 32 * h + 16 * c);
                    }
                    if (c == 1) {               // read, and the factors too
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_accempty + 8 * b);
                    }
                    if (!out) continue;
                    auto gate = [&](auto act_c) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const uint64_t a2 = act_pair<decltype(act_c)::value>(
                                f2_pack(__uint_as_float(g[j]), __uint_as_float(g[j + 1])));
                            float y0, y1;
                            f2_unpack(f2_mul(a2, f2_pack(__uint_as_float(up[j]), __uint_as_float(up[j + 1]))), y0, y1);
                            g[j / 2] = pack_bf16x2(y0, y1);
                        }
                    };
                    if (it.act == TE_ACT_GELU_TANH) gate(std::integral_constant<int, TE_ACT_GELU_TANH>{});
                    else gate(std::integral_constant<int, TE_ACT_SILU>{});
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *reinterpret_cast<uint4 *>(st + lane * 64 + (((2 * c + j) ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(g[4 * j], g[4 * j + 1], g[4 * j + 2], g[4 * j + 3]);
                }
                if (out) send_bf16(st, fo);
            } else {
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    const int col = 64 * h + 32 * c, fo = (ft - it.tile0) * F + col;
                    uint32_t v[32];
                    if (any) {
                        tmem_ld32(tbase + trow + 128 * b + col, v);
                        tmem_wait_ld();
                        scaled(v, col);
                    }
                    if (c == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_accempty + 8 * b);
                    }
                    if (!any || fo >= it.n) continue;       // n is a multiple of 32
                    if (it.act) act_block<true>(v, it.act - 1);
                    if (it.resid && !inplace && t < p.m) {
                        const float4 *rp = reinterpret_cast<const float4 *>(it.resid + (long long)t * it.ldr + fo);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 r4 = rp[j];
                            v[4 * j] = __float_as_uint(__uint_as_float(v[4 * j]) + r4.x);
                            v[4 * j + 1] = __float_as_uint(__uint_as_float(v[4 * j + 1]) + r4.y);
                            v[4 * j + 2] = __float_as_uint(__uint_as_float(v[4 * j + 2]) + r4.z);
                            v[4 * j + 3] = __float_as_uint(__uint_as_float(v[4 * j + 3]) + r4.w);
                        }
                    }
                    if (!f32) {
                        store_bf16(v, fo);
                        continue;
                    }
                    // f32: 128-byte rows, 128-byte swizzle
                    uint8_t *st = block(4096);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4 *>(st + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (inplace) tma_reduce_add_2d(&p.ty[zi], smem_u32(st), fo, tb);
                        else tma_store_2d(&p.ty[zi], smem_u32(st), fo, tb);
                        bulk_commit();
                    }
                }
            }
            // the last unit on these features: their factors may be replaced
            if (u + 1 < u1 && tt + 1 == p.ttiles) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_fempty);
            }
        }
        bulk_wait_all();                        // before the CTA's shared memory goes away
        __syncwarp();
    }
    if (!ok && lane == 0) atomicExch(p.err, 1);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

template <bool GATED>
te_status res_launch(const I8Params &q, cudaStream_t s) {
    constexpr int F = GATED ? 64 : 128, smem = Res::BYTES + 1024;
    static std::atomic<bool> ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cuda_fail(e, "i8_linear: device");
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(i8_res_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_fail(e, "i8_linear: set shared memory size");
        ready[dev] = true;
    }
    ResParams p;
    memset(&p, 0, sizeof(p));
    te_status st = make_map_2d(&p.tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.x, (uint64_t)q.k, (uint64_t)q.m, (uint64_t)q.ldx,
                               128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    int tiles = 0;
    for (int i = 0; i < q.z && st == TE_OK; ++i) {
        p.it[i] = q.it[i];
        p.it[i].tile0 = tiles;
        tiles += (q.it[i].n + F - 1) / F;
        st = make_map_2d(&p.tw[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, q.it[i].w, (uint64_t)q.k, (uint64_t)q.it[i].n,
                         (uint64_t)q.k, 128, F, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (GATED && st == TE_OK)
        st = make_map_2d(&p.tw[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, q.it[0].w2, (uint64_t)q.k, (uint64_t)q.it[0].n,
                         (uint64_t)q.k, 128, F, CU_TENSOR_MAP_SWIZZLE_128B);
    for (int i = 0; i < q.z && st == TE_OK; ++i) {
        const bool f32 = q.it[i].ydt == TE_F32;
        st = make_map_2d(&p.ty[i], f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q.it[i].y,
                         (uint64_t)q.it[i].n, (uint64_t)q.m, (uint64_t)q.it[i].ldy * (f32 ? 4 : 2), 32, 32,
                         f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    }
    if (st != TE_OK) return st;
    if ((st = gemm_error_word(&p.err)) != TE_OK) return st;
    p.xs = q.xs;
    p.m = q.m;
    p.k = q.k;
    p.z = q.z;
    p.ttiles = (q.m + 127) / 128;
    const long long units = (long long)p.ttiles * tiles;
    if (units > 0x7FFFFFFFll) return fail(TE_ESHAPE, "i8_linear: too many tiles");
    p.units = (int)units;
    e = launch_close(i8_res_kernel<GATED>, dim3(p.units < q.sms ? p.units : q.sms), Res::THREADS, smem, s, 1, p);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "i8_linear launch");
}

// x int8 [m, k] (rows ldx apart) widened to f16 [m, k], exactly: 16 values a
// thread, 16 bytes in and 32 out.
__global__ void __launch_bounds__(256) widen_kernel(const int8_t *x, long long ldx, __half *y,
                                                    long long total, int chunks) {
    prior_wait();
    next_go();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const long long r = i / chunks;
    const int c = (int)(i - r * chunks);
    const uint4 v = *reinterpret_cast<const uint4 *>(x + r * ldx + 16 * c);
    uint32_t out[8];
    widen4_f16(v.x, out[0], out[1]);
    widen4_f16(v.y, out[2], out[3]);
    widen4_f16(v.z, out[4], out[5]);
    widen4_f16(v.w, out[6], out[7]);
    uint4 *dst = reinterpret_cast<uint4 *>(y + 16 * i);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

te_status widen(const int8_t *x, int64_t ldx, void *y, int m, int k, cudaStream_t s) {
    const int chunks = k / 16;
    const long long total = (long long)m * chunks, blocks = (total + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return fail(TE_ESHAPE, "i8_linear: m * k too large");
    const cudaError_t e = launch_close(widen_kernel, dim3((unsigned)blocks), 256, 0, s, 1, x, ldx,
                                       static_cast<__half *>(y), total, chunks);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "i8_linear: widen launch");
}

constexpr int MAX_K = 65536, MAX_M = 0x7FFFFF00;   // token tiles end within an int

// Which kernel takes a call.  The measured device times (us, back to back in a
// graph, weights not in L2; n the output features in all):
//                      small    mid   resident   large (with its widening pass)
//   m = 8   k 3840 n 11520      9.7   14.9
//   m = 16  k 512  n 1536       2.4    3.6    6.3    6.7
//   m = 16  k 3840 n 3840       6.0    7.9          16.2
//   m = 16  k 10240 n 3840     12.1   12.6          33.9
//   m = 16  k 3840 n 11520     16.7   15.4
//   m = 32  k 768  n 2304       3.9    4.1           7.2
//   m = 32  k 2048 n 2048       5.3    4.6
//   m = 32  k 3840 n 3840       9.9    8.5          16.3
//   m = 64  k 3840 n 11520            22.3          17.8
//   m = 128 k 512  n 1536              4.6    6.7    8.0
//   m = 128 k 3840 n 3840             13.5          17.5
//   m = 128 k 10240 n 3840            21.1          35.7
//   m = 384 k 3840 n 11520            53.0          32.1
//   m = 600 k 512  n 1536              6.5    6.8    8.2
//   m = 1000 k 512 n 1536              9.7    7.0    8.7
//   m = 1000 k 768 n 2304             12.0          11.3
//   m = 4000 k 1024 n 128              6.5          12.7
//   m = 4000 k 1024 n 512             14.1          13.2
//   m = 8448 k 10240 n 256            59.0          85.0
//   m = 300 k 512  gated 2 x 2048      8.9    7.1    8.0
// Small: to 8 tokens; to 16 (32) tokens while the weights are under 40 M (2 M)
// values, beyond which its warps' widening of the tokens costs more than the
// TMEM pipeline's start.  Else mid where its modelled time (see mid_consider)
// is below that of what takes the larger counts: at k <= 512 the kernel with
// resident weights, 5.5 us and 1 + 0.45 us a stage for each round of its CTAs;
// beyond, large, 7 us (two launches), the widening pass's 3 bytes a value at 6
// TB/s and 0.39 us a stage of each wave of 256 x 128 units (fits of what was
// measured, to about 20 %; of the rows above and thirty others, one is given to
// a kernel slower by more than 2 %, 11.3 against 12.1 us).  Resident against large at 16238 tokens (us): k 512, n 1536 bf16 27.9
// and 34.2; n 512 f32 13.7 and 21.3; gated 2 x 2048 58.1 and 68.7; k 64, n 512
// f32 10.1 and 19.0.
template <bool GATED>
te_status rule(I8Params &p, te_i8_choice &c) {
    long long total = 0;
    int tiles = 0;                              // 128 weight rows (gated: 64 gate and 64 up)
    for (int i = 0; i < p.z; ++i) {
        total += GATED ? 2ll * p.it[i].n : p.it[i].n;
        tiles += GATED ? (p.it[i].n + 63) / 64 : (p.it[i].n + 127) / 128;
    }
    if (p.m <= 8 || (p.m <= 16 && total * p.k <= (40 << 20)) || (p.m <= 32 && total * p.k <= (2 << 20))) {
        const int groups = small_groups<GATED>(p);
        if (p.m <= 8) c = {TE_I8_FEW, 8, small_slots<1, GATED>(p, groups)};
        else if (p.m <= 16) c = {TE_I8_FEW, 16, small_slots<2, GATED>(p, groups)};
        else c = {TE_I8_FEW, 32, small_slots<4, GATED>(p, groups)};
        return TE_OK;
    }
    MidPlan plan;
    const te_status st = mid_plan<GATED>(plan, tiles, p.m, p.k);
    if (st != TE_OK) return st;
    const int nkb = (p.k + 127) / 128;
    const long long ttiles = (p.m + 127) / 128, sms = p.sms;
    double other;
    if (p.k <= 512) {
        c = {TE_I8_RESIDENT, 128, 1};
        const long long rounds = (tiles * ttiles + sms - 1) / sms;
        other = 5.5 + rounds * (1.0 + 0.45 * nkb);
    } else {
        c = {TE_I8_LARGE, 0, 0};
        const long long waves = ((tiles + 1) / 2 * ttiles + sms / 2 - 1) / (sms / 2);
        other = 7.0 + 0.39 * nkb * waves + (double)p.m * p.k * 3 / 6e6;
    }
    if (p.m <= 32 || plan.us < other) c = {TE_I8_MIDDLING, plan.n, plan.split};
    return TE_OK;
}

// te_i8_choose's choice, of this thread's calls.
thread_local bool g_chosen = false;
thread_local te_i8_choice g_choice;

// Whether a chosen kernel takes these sizes (the fields are a choice's, see te_i8_choose).
template <bool GATED>
te_status takes(const I8Params &p, const te_i8_choice &c) {
    bool ok;
    if (c.kernel == TE_I8_FEW) {
        ok = p.m <= c.tile && (c.tile == 8    ? c.split == Small<1, GATED>::D || c.split == Small<1, GATED>::D2
                               : c.tile == 16 ? c.split == Small<2, GATED>::D || c.split == Small<2, GATED>::D2
                                              : c.split == Small<4, GATED>::D);
    } else if (c.kernel == TE_I8_MIDDLING) {
        ok = c.split <= (p.k + 127) / 128 && ((long long)p.m + c.tile - 1) / c.tile <= 65535;
    } else {
        ok = c.kernel == TE_I8_RESIDENT ? p.k <= 512 : p.k > 512 && p.m > 8;
    }
    return ok ? TE_OK
              : fail(TE_ESHAPE, "i8_linear: the chosen kernel (%d, %d, %d) does not take m=%d k=%d", c.kernel, c.tile,
                     c.split, p.m, p.k);
}
template <bool GATED>
te_status choice_of(I8Params &p, te_i8_choice &c) {
    if (!g_chosen) return rule<GATED>(p, c);
    c = g_choice;
    return takes<GATED>(p, c);
}

// Launches the chosen kernel unless it is the large pipeline (the caller's).
template <bool GATED>
te_status go(I8Params &p, const te_i8_choice &c, cudaStream_t s) {
    if (c.kernel == TE_I8_RESIDENT) return res_launch<GATED>(p, s);
    if (c.kernel == TE_I8_FEW)
        return c.tile == 8    ? small_launch<1, GATED>(p, c.split, s)
               : c.tile == 16 ? small_launch<2, GATED>(p, c.split, s)
                              : small_launch<4, GATED>(p, c.split, s);
    if (c.tile == 16) return mid_launch<16, GATED>(p, c.split, s);
    if (c.tile == 32) return mid_launch<32, GATED>(p, c.split, s);
    return c.tile == 64 ? mid_launch<64, GATED>(p, c.split, s) : mid_launch<128, GATED>(p, c.split, s);
}
te_status check_x(const char *what, const void *x, int64_t ldx, const float *xs, int32_t m, int32_t k) {
    if (m > 0 && (!x || !xs)) return fail(TE_EINVAL, "%s: NULL x or x_scale", what);
    if (m < 0 || m > MAX_M || k < 64 || k > MAX_K || k % 64)
        return fail(TE_ESHAPE, "%s: m=%d k=%d (m 0..%d, k %% 64 == 0, 64..%d)", what, m, k, MAX_M, MAX_K);
    if (ldx < k || ldx % 16) return fail(TE_ESHAPE, "%s: ldx=%lld (>= k, multiple of 16)", what, (long long)ldx);
    if (!aligned16(x) || (reinterpret_cast<uintptr_t>(xs) & 3))
        return fail(TE_EALIGN, "%s: x 16-byte, x_scale 4-byte aligned", what);
    return TE_OK;
}

te_status check_w(const char *what, int i, const te_q8w &w, int32_t k) {
    if (!w.q || !w.scale) return fail(TE_EINVAL, "%s: item %d has a NULL q or scale", what, i);
    if (w.block_scale || w.col)
        return fail(TE_EINVAL, "%s: item %d: q8_row weights only (no block scales, no column field)", what, i);
    if (w.k != k) return fail(TE_ESHAPE, "%s: item %d has k=%d, x has %d", what, i, w.k, k);
    if (w.n < 32 || w.n % 32) return fail(TE_ESHAPE, "%s: item %d n=%d (multiple of 32)", what, i, w.n);
    if (!aligned16(w.q) || (reinterpret_cast<uintptr_t>(w.scale) & 3) ||
        (w.bias && (reinterpret_cast<uintptr_t>(w.bias) & 3)))
        return fail(TE_EALIGN, "%s: item %d: q 16-byte, scale and bias 4-byte aligned", what, i);
    return TE_OK;
}

te_status check_ws(const char *what, const void *ws, size_t have, size_t need) {
    if (have < need || (need && !ws))
        return fail(TE_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", what, ws ? have : (size_t)0, need);
    if (need && (reinterpret_cast<uintptr_t>(ws) & 255)) return fail(TE_EALIGN, "%s: workspace not 256-byte aligned", what);
    return TE_OK;
}

}  // namespace
}  // namespace tefwd

using namespace tefwd;

// the f16 activation of a call that may widen it beforehand, whatever n: no
// kernel for k <= 512 does
static size_t workspace_of(int32_t m, int32_t k) {
    return m <= 8 || m > MAX_M || k <= 512 ? 0 : ((size_t)m * k * 2 + 255) & ~(size_t)255;
}

extern "C" size_t te_i8_workspace(int32_t m, int32_t k, int32_t n) {
    return k < 64 || k > MAX_K || k % 64 || n < 32 ? 0 : workspace_of(m, k);
}

extern "C" te_status te_i8_linear(const int8_t *x, int64_t ldx, const float *x_scale, int32_t m,
                                  int32_t k, const te_q8_item *items, int32_t z, void *workspace,
                                  size_t ws_bytes, te_stream stream) {
    if (!items) return fail(TE_EINVAL, "i8_linear: NULL items");
    if (z < 1 || z > MAXZ) return fail(TE_ESHAPE, "i8_linear: z=%d (1..4)", z);
    te_status st = check_x("i8_linear", x, ldx, x_scale, m, k);
    if (st != TE_OK) return st;
    I8Params p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.xs = x_scale;
    p.ldx = ldx;
    p.m = m;
    p.k = k;
    p.z = z;
    p.sms = sm_count();
    int64_t n = 0;
    for (int i = 0; i < z; ++i) {
        const te_q8_item &src = items[i];
        if ((st = check_w("i8_linear", i, src.w, k)) != TE_OK) return st;
        if (m > 0 && !src.y) return fail(TE_EINVAL, "i8_linear: item %d has a NULL y", i);
        if (src.y_dtype != TE_F32 && src.y_dtype != TE_BF16) return fail(TE_EINVAL, "i8_linear: item %d bad y dtype", i);
        if (src.ldy < src.w.n) return fail(TE_ESHAPE, "i8_linear: item %d ldy < n", i);
        if (!aligned16(src.y) || (src.ldy * (src.y_dtype == TE_F32 ? 4 : 2)) % 16)
            return fail(TE_EALIGN, "i8_linear: item %d: y and its rows must be 16-byte aligned", i);
        if (src.epilogue < TE_EPI_NONE || src.epilogue > TE_EPI_SILU)
            return fail(TE_EINVAL, "i8_linear: item %d bad epilogue %d", i, src.epilogue);
        if (src.epilogue != TE_EPI_NONE && src.residual)
            return fail(TE_EINVAL, "i8_linear: item %d: an epilogue activation takes no residual", i);
        if (src.residual) {
            if (src.ldr < src.w.n) return fail(TE_ESHAPE, "i8_linear: item %d ldr < n", i);
            if (!aligned16(src.residual) || src.ldr % 4)
                return fail(TE_EALIGN, "i8_linear: item %d: residual rows must be 16-byte aligned", i);
            if (src.residual == src.y && (src.ldr != src.ldy || src.y_dtype != TE_F32))
                return fail(TE_EINVAL, "i8_linear: item %d: in-place residual needs f32 y and ldr == ldy", i);
        }
        I8Item &d = p.it[i];
        d.w = src.w.q;
        d.scale = src.w.scale;
        d.bias = src.w.bias;
        d.resid = src.residual;
        d.y = src.y;
        d.ldy = src.ldy;
        d.ldr = src.ldr;
        d.n = src.w.n;
        d.ydt = src.y_dtype;
        d.act = src.epilogue;
        n += src.w.n;
    }
    if (n > 0x7FFFFFFFll) return fail(TE_ESHAPE, "i8_linear: too many output features");
    if ((st = check_ws("i8_linear", workspace, ws_bytes, workspace_of(m, k))) != TE_OK) return st;
    if (m == 0) return TE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    te_i8_choice c;
    if ((st = choice_of<false>(p, c)) != TE_OK) return st;
    if (c.kernel != TE_I8_LARGE) return go<false>(p, c, s);
    if ((st = widen(x, ldx, workspace, m, k, s)) != TE_OK) return st;
    return i8_gemm_linear(workspace, x_scale, m, k, items, z, s);
}

extern "C" te_status te_i8_gated_linear(const int8_t *x, int64_t ldx, const float *x_scale, int32_t m,
                                        int32_t k, const te_q8w *wg, const te_q8w *wu, int32_t act,
                                        void *out, int64_t ldm, void *workspace, size_t ws_bytes,
                                        te_stream stream) {
    if (!wg || !wu || (m > 0 && !out)) return fail(TE_EINVAL, "i8_gated_linear: NULL wg, wu or out");
    if (act != TE_ACT_GELU_TANH && act != TE_ACT_SILU) return fail(TE_EINVAL, "i8_gated_linear: bad act");
    te_status st = check_x("i8_gated_linear", x, ldx, x_scale, m, k);
    if (st != TE_OK) return st;
    if ((st = check_w("i8_gated_linear", 0, *wg, k)) != TE_OK) return st;
    if ((st = check_w("i8_gated_linear", 1, *wu, k)) != TE_OK) return st;
    const int f = wg->n;
    if (wu->n != f) return fail(TE_ESHAPE, "i8_gated_linear: wg has n=%d, wu n=%d", f, wu->n);
    if (f > 0x3FFFFFFF) return fail(TE_ESHAPE, "i8_gated_linear: too many output features");
    if (ldm < f || ldm % 8) return fail(TE_ESHAPE, "i8_gated_linear: ldm=%lld (>= f, multiple of 8)", (long long)ldm);
    if (!aligned16(out)) return fail(TE_EALIGN, "i8_gated_linear: out not 16-byte aligned");
    if ((st = check_ws("i8_gated_linear", workspace, ws_bytes, workspace_of(m, k))) != TE_OK) return st;
    if (m == 0) return TE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    I8Params p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.xs = x_scale;
    p.ldx = ldx;
    p.m = m;
    p.k = k;
    p.z = 1;
    p.sms = sm_count();
    I8Item &d = p.it[0];
    d.w = wg->q;
    d.w2 = wu->q;
    d.scale = wg->scale;
    d.bias = wg->bias;
    d.scale2 = wu->scale;
    d.bias2 = wu->bias;
    d.y = out;
    d.ldy = ldm;
    d.n = f;
    d.ydt = TE_BF16;
    d.act = act;
    te_i8_choice c;
    if ((st = choice_of<true>(p, c)) != TE_OK) return st;
    if (c.kernel != TE_I8_LARGE) return go<true>(p, c, s);
    if ((st = widen(x, ldx, workspace, m, k, s)) != TE_OK) return st;
    return i8_gemm_gated(workspace, x_scale, m, k, wg, wu, act, out, ldm, s);
}

extern "C" te_status te_i8_choose(const te_i8_choice *choice) {
    if (choice) {
        const int32_t t = choice->tile, s = choice->split;
        bool ok = false;
        if (choice->kernel == TE_I8_FEW) ok = (t == 8 || t == 16 || t == 32) && (s == 1 || s == 2 || s == 4);
        if (choice->kernel == TE_I8_MIDDLING)
            ok = (t == 16 || t == 32 || t == 64 || t == 128) && (s == 1 || s == 2 || s == 4 || s == 8);
        if (choice->kernel == TE_I8_RESIDENT) ok = t == 128 && s == 1;
        if (choice->kernel == TE_I8_LARGE) ok = t == 0 && s == 0;
        if (!ok) return fail(TE_EINVAL, "i8_choose: no kernel (%d, %d, %d)", choice->kernel, t, s);
        g_choice = *choice;
    }
    g_chosen = choice != nullptr;
    return TE_OK;
}

extern "C" te_status te_i8_choice_of(int32_t m, int32_t k, const int32_t *n, int32_t z, int32_t gated,
                                     te_i8_choice *choice) {
    if (!n || !choice) return fail(TE_EINVAL, "i8_choice_of: NULL n or choice");
    if (z < 1 || z > (gated ? 1 : MAXZ) || m < 1 || m > MAX_M || k < 64 || k > MAX_K || k % 64)
        return fail(TE_ESHAPE, "i8_choice_of: m=%d k=%d z=%d", m, k, z);
    I8Params p;
    memset(&p, 0, sizeof(p));
    p.m = m;
    p.k = k;
    p.z = z;
    p.sms = sm_count();
    int ftiles = 0;
    for (int i = 0; i < z; ++i) {
        if (n[i] < 32 || n[i] % 32 || n[i] > 0x3FFFFFFF) return fail(TE_ESHAPE, "i8_choice_of: n=%d", n[i]);
        p.it[i].n = n[i];
        ftiles += gated ? (n[i] + 63) / 64 : (n[i] + 127) / 128;
    }
    te_i8_choice c;
    const te_status st = gated ? choice_of<true>(p, c) : choice_of<false>(p, c);
    if (st != TE_OK) return st;
    if (c.kernel == TE_I8_LARGE) i8_gemm_tile(m, k, ftiles, c.tile, c.split);
    *choice = c;
    return TE_OK;
}
