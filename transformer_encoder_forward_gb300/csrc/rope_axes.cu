// q/k norm and rotary positions with several axes (time, height, width, ...).
//
// Pair p of a head turns by pos[row, axis(p)] * f_p radians:
//     (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin).
// Angles are kept as 64-bit fixed-point fractions of a turn: f_p / (2 pi) as a
// word of 2^-64 turns (te_rope_axes.turn), times the position, modulo 2^64.
// The integer product wraps exactly where whole turns do, so the reduction
// loses nothing however far the position.  The word is the nearest one to
// f_p / (2 pi) for the f64 f_p of any size (see turn_word), so the product is within
// 2^-34 turns of pos * f_p at the furthest int32 positions; its top 32 bits
// (2^-32 turns), read as a signed fraction, give sine and cosine by sincospif.
// No table is read and no 64-bit float is touched on the device.
//
// Generalises the 1-D and 2-D rotation of "cortiq-engine 0.8.39
// src/gpu_metal/egemma2.rs" (Prog::qkv, EgQkv.sec) and "cortiq-engine 0.7.6
// src/gpu_metal/zimage.rs" (Enc::block) to axes of different widths.
#include <math.h>
#include <string.h>

#include <atomic>

#include "common.cuh"

namespace tefwd {
namespace {

struct RopeParams {
    const void *src;
    void *dst;
    const float *qn, *kn;
    const int32_t *pos;
    long long lds, ldd, ldp;
    int items;                // rows * cuts, those from `full` on in `fine` pieces of `sub` slots
    int full, fine, sub;
    int q_off, k_off, nq, nkv, hd;
    int hpi;                  // heads a slot
    int sq, slots;            // slots of the q heads, and with the k heads'
    int cuts, per;            // items a row's slots are cut into, slots an item
    float eps, q_mul, inv_hd;
    int pairs;
    // rope_vec_kernel: unit u of a head is 4 channels from c1[u] and 4 from
    // c2[u], its pairs p0[u].. (those past `pairs` do not turn).
    // rope_any_kernel: pair u is channels c1[u] and c2[u].
    uint8_t c1[TE_ROPE_MAX_PAIRS], c2[TE_ROPE_MAX_PAIRS], p0[32];
    uint8_t axis[TE_ROPE_MAX_PAIRS];
    unsigned long long turn[TE_ROPE_MAX_PAIRS];
};

// cos and sin of position * (turn / 2^64) turns
__device__ __forceinline__ float2 turn_cs(int pos, unsigned long long turn) {
    const unsigned long long a = (unsigned long long)(long long)pos * turn;
    const int top = (int)(a >> 32);                       // turns in [-1/2, 1/2) * 2^32
    float s, c;
    sincospif((float)top * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    return make_float2(c, s);
}

__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
// The 8 channels of a unit as loaded: 4 from c1, 4 from c2.  x1, x2: the first
// and second members of its four pairs, two pairs a 64-bit register; adjacent
// pairing takes them alternately from the 8, halves from the two pieces.
template <typename T> struct Unit;
template <> struct Unit<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p1, const float *p2) {
        a = *reinterpret_cast<const float4 *>(p1);
        b = *reinterpret_cast<const float4 *>(p2);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    template <bool ADJ> __device__ __forceinline__ void get(uint64_t (&x1)[2], uint64_t (&x2)[2]) const {
        x1[0] = ADJ ? f2_pack(a.x, a.z) : f2_pack(a.x, a.y);
        x1[1] = ADJ ? f2_pack(b.x, b.z) : f2_pack(a.z, a.w);
        x2[0] = ADJ ? f2_pack(a.y, a.w) : f2_pack(b.x, b.y);
        x2[1] = ADJ ? f2_pack(b.y, b.w) : f2_pack(b.z, b.w);
    }
};
template <> struct Unit<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p1, const __nv_bfloat16 *p2) {
        a = *reinterpret_cast<const uint2 *>(p1);
        b = *reinterpret_cast<const uint2 *>(p2);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint2(0u, 0u); }
    template <bool ADJ> __device__ __forceinline__ void get(uint64_t (&x1)[2], uint64_t (&x2)[2]) const {
        if (ADJ) {
            x1[0] = f2_pack(bf16_lo(a.x), bf16_lo(a.y));
            x1[1] = f2_pack(bf16_lo(b.x), bf16_lo(b.y));
            x2[0] = f2_pack(bf16_hi(a.x), bf16_hi(a.y));
            x2[1] = f2_pack(bf16_hi(b.x), bf16_hi(b.y));
        } else {
            x1[0] = f2_pack(bf16_lo(a.x), bf16_hi(a.x));
            x1[1] = f2_pack(bf16_lo(a.y), bf16_hi(a.y));
            x2[0] = f2_pack(bf16_lo(b.x), bf16_hi(b.x));
            x2[1] = f2_pack(bf16_lo(b.y), bf16_hi(b.y));
        }
    }
};
template <bool ADJ, typename T>
__device__ __forceinline__ void put_unit(T *p1, T *p2, const uint64_t (&y1)[2], const uint64_t (&y2)[2]) {
    float u[4], v[4];
    f2_unpack(y1[0], u[0], u[1]);
    f2_unpack(y1[1], u[2], u[3]);
    f2_unpack(y2[0], v[0], v[1]);
    f2_unpack(y2[1], v[2], v[3]);
    const float a[4] = {u[0], ADJ ? v[0] : u[1], ADJ ? u[1] : u[2], ADJ ? v[1] : u[3]};
    const float b[4] = {ADJ ? u[2] : v[0], ADJ ? v[2] : v[1], ADJ ? u[3] : v[2], v[3]};
    store4(p1, a);
    store4(p2, b);
}

// One item: a run of one row's slots; q heads first, then k heads, each part
// in slots of hpi heads.
struct Chunk {
    long long row;
    int s0, s1;
};
template <bool FINE>
__device__ __forceinline__ Chunk chunk_of(const RopeParams &p, unsigned item) {
    unsigned fine = 0;
    const bool last = FINE && p.fine > 1 && item >= (unsigned)p.full;
    if (last) {
        const unsigned r = item - p.full, b = r / (unsigned)p.fine;
        fine = r - b * p.fine;
        item = p.full + b;
    }
    const unsigned row = item / (unsigned)p.cuts;
    Chunk c;
    c.row = row;
    c.s0 = (int)(item - row * p.cuts) * p.per;
    c.s1 = c.s0 + p.per < p.slots ? c.s0 + p.per : p.slots;
    if (last) {
        c.s0 += (int)fine * p.sub;
        c.s1 = c.s0 + p.sub < c.s1 ? c.s0 + p.sub : c.s1;
    }
    return c;
}
// The heads [h0, h1) of part `k` (0: q, 1: k) in the chunk; empty where h0 >= h1.
__device__ __forceinline__ void part_heads(const RopeParams &p, const Chunk &c, int k, int &h0, int &h1) {
    const int lo = k ? (c.s0 > p.sq ? c.s0 - p.sq : 0) : c.s0, hi = k ? c.s1 - p.sq : (c.s1 < p.sq ? c.s1 : p.sq);
    const int n = k ? p.nkv : p.nq;
    h0 = lo * p.hpi;
    h1 = hi * p.hpi < n ? hi * p.hpi : n;
}

// A warp an item (persistent over items).  A head spans hd / 8 lanes, each with
// the two 4-channel pieces of one unit: both members of its four pairs
// (adjacent pairing: 8 neighbouring channels), so the rotation exchanges
// nothing between lanes and the norm is a reduction over the lane group (LPH
// lanes, or hd / 8 where that is no power of two: LPH == 0).  A lane's unit
// never changes, so its pairs' matrices serve all heads of a part.  The row's
// sines and cosines are worked out once by the whole warp.  All loads of a slot group go out before
// any arithmetic, which runs in f32 pairs.  Bound by HBM: registers are held to
// 64 (f32 80) for four (three) CTAs an SM, with the frequency words in shared
// memory; at 79 and two CTAs the 32760-row clip (1.0 GB) took 174 us instead of
// 158 (6.4 TB/s, 0.94 of the measured copy rate).  8448 rows (259 MB) take 46
// us, where a plain copy of as many bytes takes 41: a launch's start and end
// cost both.  Loads a step ahead in registers (fewer warps) took 55 us.  With few
// heads a row instructions bound it: 8448 rows of 12 + 4 heads of 96 take 18 us.
template <typename T, bool ADJ, bool PART, int LPH>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3) rope_vec_kernel(const __grid_constant__ RopeParams p) {
    constexpr int QU = 4;                       // load slots in flight
    // the row's cosines and sines, a warp's own; pairs past the last do not turn
    __shared__ __align__(16) float2 rows_cs[8][TE_ROPE_MAX_PAIRS + 4];
    __shared__ unsigned long long turns[TE_ROPE_MAX_PAIRS];
    __shared__ uint8_t axes[TE_ROPE_MAX_PAIRS];
    for (int i = threadIdx.x; i < TE_ROPE_MAX_PAIRS; i += 256) {
        turns[i] = i < p.pairs ? p.turn[i] : 0ull;
        axes[i] = i < p.pairs ? p.axis[i] : 0;
    }
    if (PART) {
        for (int i = threadIdx.x; i < 8 * (TE_ROPE_MAX_PAIRS + 4); i += 256) (&rows_cs[0][0])[i] = make_float2(1.f, 0.f);
    }
    __syncthreads();
    prior_wait();
    const int lane = threadIdx.x & 31;
    float2 *cs = rows_cs[threadIdx.x >> 5];
    const int lph = LPH ? LPH : p.hd / 8, hpi = LPH ? 32 / LPH : p.hpi;
    const int hl = lane / lph, u = lane - hl * lph;
    const bool on = LPH ? u < p.hd / 8 : hl < hpi;      // the other lanes idle
    const int uu = on ? u : 0;
    const int c1 = p.c1[uu], c2 = p.c2[uu], p0 = p.p0[uu];
    for (unsigned item = blockIdx.x * 8 + (threadIdx.x >> 5); item < (unsigned)p.items; item += gridDim.x * 8) {
        const Chunk ch = chunk_of<(LPH >= 16)>(p, item);
        bool turned = false;                    // the row's cosines and sines are there
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            int hbeg, hend;
            part_heads(p, ch, part, hbeg, hend);
            const int off = part ? p.k_off : p.q_off;
            const T *src = static_cast<const T *>(p.src) + ch.row * p.lds + off;
            T *dst = static_cast<T *>(p.dst) + ch.row * p.ldd + off;
            const float *nw = part ? p.kn : p.qn;
            // y1 = (x1 m11 - x2 m12) inv, y2 = (x2 m22 + x1 m21) inv: the rotation
            // with the norm's weights and q_mul multiplied into its matrix
            uint64_t m11[2], m12[2], m21[2], m22[2];
            for (int h0 = hbeg; h0 < hend; h0 += hpi * QU) {
                Unit<T> raw[QU];
#pragma unroll
                for (int i = 0; i < QU; ++i) {
                    const int hh = h0 + i * hpi + hl;
                    if (on && hh < hend) raw[i].load(src + (hh * p.hd + c1), src + (hh * p.hd + c2));
                    else raw[i].zero();
                }
                if (h0 == hbeg) {               // behind the first loads
                    if (!turned) {
                        turned = true;
                        const int32_t *pos = p.pos + ch.row * p.ldp;
                        __syncwarp();           // the last row's have been read
                        for (int i = lane; i < p.pairs; i += 32) cs[i] = turn_cs(pos[axes[i]], turns[i]);
                        __syncwarp();
                    }
                    float4 t4[2];
                    t4[0] = *reinterpret_cast<const float4 *>(cs + p0);
                    t4[1] = *reinterpret_cast<const float4 *>(cs + p0 + 2);
                    const float mul = part ? 1.f : p.q_mul;
                    float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
                    if (nw && on) {
                        load4(nw + c1, wa);
                        load4(nw + c2, wb);
                    }
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float r11[2], r12[2], r21[2], r22[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int pr = 2 * g + e;
                            const float w1 = (ADJ ? (pr < 2 ? wa[2 * pr] : wb[2 * pr - 4]) : wa[pr]) * mul;
                            const float w2 = (ADJ ? (pr < 2 ? wa[2 * pr + 1] : wb[2 * pr - 3]) : wb[pr]) * mul;
                            const float c = e ? t4[g].z : t4[g].x, sn = e ? t4[g].w : t4[g].y;
                            r11[e] = w1 * c;
                            r12[e] = -w2 * sn;
                            r21[e] = w1 * sn;
                            r22[e] = w2 * c;
                        }
                        m11[g] = f2_pack(r11[0], r11[1]);
                        m12[g] = f2_pack(r12[0], r12[1]);
                        m21[g] = f2_pack(r21[0], r21[1]);
                        m22[g] = f2_pack(r22[0], r22[1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < QU; ++i) {
                    if (h0 + i * hpi >= hend) break;    // warp-uniform: no head left
                    const int hh = h0 + i * hpi + hl;
                    uint64_t x1[2], x2[2], y1[2], y2[2];
                    raw[i].template get<ADJ>(x1, x2);
                    float inv = 1.f;
                    if (nw) {
                        const uint64_t q2 = f2_fma(x1[0], x1[0], f2_fma(x2[0], x2[0], f2_fma(x1[1], x1[1], f2_mul(x2[1], x2[1]))));
                        float q, qb;
                        f2_unpack(q2, q, qb);
                        q += qb;
                        if (LPH) {
#pragma unroll
                            for (int o = 1; o < LPH; o <<= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
                        } else {                // up to 32 lanes of any count: to the group's first, and back
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) {
                                const float r = __shfl_down_sync(0xFFFFFFFFu, q, o);
                                if (u + o < lph) q += r;
                            }
                            q = __shfl_sync(0xFFFFFFFFu, q, lane - u);
                        }
                        inv = rsqrtf(fmaf(q, p.inv_hd, p.eps));
                    }
                    const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint64_t s1 = f2_mul(x1[g], m11[g]), s2 = f2_mul(x2[g], m22[g]);
                        y1[g] = f2_fma(x2[g], m12[g], s1);
                        y2[g] = f2_fma(x1[g], m21[g], s2);
                        if (PART) {             // pairs that do not turn never see their neighbour
                            float a0, a1, b0, b1, u0, u1, v0, v1;
                            f2_unpack(y1[g], a0, a1);
                            f2_unpack(y2[g], b0, b1);
                            f2_unpack(s1, u0, u1);
                            f2_unpack(s2, v0, v1);
                            const bool t0 = p0 + 2 * g < p.pairs, t1 = p0 + 2 * g + 1 < p.pairs;
                            y1[g] = f2_pack(t0 ? a0 : u0, t1 ? a1 : u1);
                            y2[g] = f2_pack(t0 ? b0 : v0, t1 ? b1 : v1);
                        }
                        if (nw) {
                            y1[g] = f2_mul(y1[g], inv2);
                            y2[g] = f2_mul(y2[g], inv2);
                        }
                    }
                    if (on && hh < hend) put_unit<ADJ>(dst + (hh * p.hd + c1), dst + (hh * p.hd + c2), y1, y2);
                }
            }
        }
        if (item + gridDim.x * 8 >= (unsigned)p.items) next_go();
    }
}

// Any even sections: the heads of an item pass through shared memory, up to
// ANY_STG bytes at a time (16-byte loads and stores, single channels in
// between); lane l turns pairs l, l + 32, ... (NP of them) of each head, HU heads
// at once so that their chains of load, norm and rotation overlap.  (Four pairs
// a lane and several heads side by side in the warp: 8448 x 60 x 128 83 -> 138 us.)
constexpr int ANY_STG = 4096;

template <typename T, int NP>
__global__ void __launch_bounds__(256, NP == 4 ? 3 : 4) rope_any_kernel(const __grid_constant__ RopeParams p) {
    // heads at once: as many as the registers of four CTAs an SM hold (three
    // where a lane has four pairs: 2000 rows of 12 heads of 256 24.1 -> 17.9 us;
    // below, six or eight heads at three CTAs lose 5 to 25 %)
    constexpr int HU = NP == 4 ? 3 : 4;
    __shared__ __align__(16) uint8_t stage[8][ANY_STG];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    prior_wait();
    T *buf = reinterpret_cast<T *>(stage[warp]);
    constexpr int V = 16 / (int)sizeof(T);      // channels a 16-byte piece
    const int hb = ANY_STG / ((int)sizeof(T) * p.hd);   // heads a pass
    int c1[NP], c2[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int pr = lane + 32 * i;
        c1[i] = pr < p.hd / 2 ? p.c1[pr] : -1;
        c2[i] = pr < p.hd / 2 ? p.c2[pr] : -1;
    }
    for (unsigned item = blockIdx.x * 8 + warp; item < (unsigned)p.items; item += gridDim.x * 8) {
        const Chunk ch = chunk_of<false>(p, item);
        float2 cs[NP];
        const int32_t *pos = p.pos + ch.row * p.ldp;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int pr = lane + 32 * i;
            cs[i] = pr < p.pairs ? turn_cs(pos[p.axis[pr]], p.turn[pr]) : make_float2(1.f, 0.f);
        }
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            int hbeg, hend;
            part_heads(p, ch, part, hbeg, hend);
            const int off = part ? p.k_off : p.q_off;
            const T *src = static_cast<const T *>(p.src) + ch.row * p.lds + off;
            T *dst = static_cast<T *>(p.dst) + ch.row * p.ldd + off;
            const float *nw = part ? p.kn : p.qn;
            const float mul = part ? 1.f : p.q_mul;
            float w1[NP], w2[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                w1[i] = c1[i] >= 0 && nw ? nw[c1[i]] * mul : mul;
                w2[i] = c1[i] >= 0 && nw ? nw[c2[i]] * mul : mul;
            }
            for (int h0 = hbeg; h0 < hend; h0 += hb) {
                const int hn = hend - h0 < hb ? hend - h0 : hb;
                const int n16 = hn * p.hd / V;
                const uint4 *s16 = reinterpret_cast<const uint4 *>(src + (long long)h0 * p.hd);
                uint4 *d16 = reinterpret_cast<uint4 *>(dst + (long long)h0 * p.hd);
                uint4 *b16 = reinterpret_cast<uint4 *>(buf);
#pragma unroll
                for (int j = 0; j < ANY_STG / 512; ++j)
                    if (lane + 32 * j < n16) b16[lane + 32 * j] = s16[lane + 32 * j];
                __syncwarp();
                for (int h = 0; h < hn; h += HU) {
                    T *x = buf + h * p.hd;
                    float x1[HU][NP], x2[HU][NP], inv[HU];
#pragma unroll
                    for (int k = 0; k < HU; ++k) {
                        const bool have = h + k < hn;   // warp-uniform
                        float q = 0.f;
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            x1[k][i] = have && c1[i] >= 0 ? (float)x[k * p.hd + c1[i]] : 0.f;
                            x2[k][i] = have && c1[i] >= 0 ? (float)x[k * p.hd + c2[i]] : 0.f;
                            q = fmaf(x1[k][i], x1[k][i], fmaf(x2[k][i], x2[k][i], q));
                        }
                        inv[k] = q;
                    }
                    if (nw) {
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                            for (int k = 0; k < HU; ++k) inv[k] += __shfl_xor_sync(0xFFFFFFFFu, inv[k], o);
#pragma unroll
                        for (int k = 0; k < HU; ++k) inv[k] = rsqrtf(fmaf(inv[k], p.inv_hd, p.eps));
                    }
#pragma unroll
                    for (int k = 0; k < HU; ++k) {
                        if (h + k >= hn) break;
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            if (c1[i] < 0) continue;
                            float a = x1[k][i] * w1[i], b = x2[k][i] * w2[i];
                            if (nw) {
                                a *= inv[k];
                                b *= inv[k];
                            }
                            if (lane + 32 * i < p.pairs) {
                                const float y1 = fmaf(a, cs[i].x, -b * cs[i].y);
                                b = fmaf(b, cs[i].x, a * cs[i].y);
                                a = y1;
                            }
                            x[k * p.hd + c1[i]] = (T)a;
                            x[k * p.hd + c2[i]] = (T)b;
                        }
                    }
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < ANY_STG / 512; ++j)
                    if (lane + 32 * j < n16) d16[lane + 32 * j] = b16[lane + 32 * j];
                __syncwarp();                   // before the next pass overwrites the stage
            }
        }
        if (item + gridDim.x * 8 >= (unsigned)p.items) next_go();
    }
}

// Cuts the rows into items and launches one wave of warps over them.
template <auto KERN, bool FINE = false>
te_status launch(RopeParams &p, int rows, int hpi, cudaStream_t s) {
    // resident CTAs of the whole device, asked for once a kernel and device
    static std::atomic<int> resident[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cuda_fail(e, "qk_rope_axes: device");
    if (!resident[dev]) {
        int sms = 0, per = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, KERN, 256, 0);
        if (e != cudaSuccess || per < 1) return cuda_fail(e, "qk_rope_axes: occupancy");
        resident[dev] = sms * per;
    }
    const long long most = resident[dev], warps = 8 * most;
    // A row's slots (q heads, then k heads, hpi a slot) are cut into items of
    // about 16 slots, whose sines and cosines are then worth their while; with
    // few rows further, until every resident warp has an item.  (Cuts that even
    // out the last round of the warps cost more in repeated sines and cosines
    // than they gain: 47.7 -> 49.2 us at 8448 rows of 60 heads.)
    p.hpi = hpi;
    p.sq = (p.nq + hpi - 1) / hpi;
    p.slots = p.sq + (p.nkv + hpi - 1) / hpi;
    long long cuts = (p.slots + 8) / 16;
    if (cuts * rows < warps) cuts = warps / rows;
    if (cuts < 1) cuts = 1;
    if (cuts > p.slots) cuts = p.slots;
    p.per = (int)((p.slots + cuts - 1) / cuts);
    p.cuts = (p.slots + p.per - 1) / p.per;
    const long long items = (long long)rows * p.cuts;
    if (items > 0x7FFFFFFFll) return fail(TE_ESHAPE, "qk_rope_axes: rows=%d too many", rows);
    // What the last round of warps holds is cut finer, so that it occupies them
    // all: a round of whole items for a part of them would take as long (8448 rows
    // of 60 heads of 128, 3.5 rounds: 49.1 -> 45.9 us).  Pieces below 8 slots cost
    // more in repeated sines and cosines than they gain, and where a slot holds
    // three heads or more the index arithmetic alone does (16 heads of 72: 15.7 ->
    // 16.1 us).  Over many rounds the warps drift apart and even out by themselves
    // (32760 rows, 13.5 rounds: 159.3 -> 160.2 us with them).
    p.full = (int)(items / warps * warps);
    const long long rem = items - p.full;
    long long fine = FINE && p.full && p.full / warps < 8 && rem ? warps / rem : 1;
    if (fine > (p.per + 1) / 8) fine = (p.per + 1) / 8;
    if (fine < 1) fine = 1;
    p.sub = (int)((p.per + fine - 1) / fine);
    p.fine = (p.per + p.sub - 1) / p.sub;
    if (p.full + rem * p.fine > 0x7FFFFFFFll) p.fine = 1, p.sub = p.per;
    p.items = (int)(p.full + rem * p.fine);
    const long long need = ((long long)p.items + 7) / 8;
    e = launch_close(KERN, dim3((unsigned)(need < most ? need : most)), 256, 0, s, 1, p);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "qk_rope_axes launch");
}

template <typename T, bool ADJ, bool PART>
te_status launch_vec(RopeParams &p, int rows, cudaStream_t s) {
    // lanes a head: a power of two where as many heads fit the warp as without
    // the rounding (its norm takes half the instructions), else hd / 8
    const int nu = p.hd / 8;
    if (nu == 4) return launch<rope_vec_kernel<T, ADJ, PART, 4>>(p, rows, 8, s);
    if (nu == 7 || nu == 8) return launch<rope_vec_kernel<T, ADJ, PART, 8>>(p, rows, 4, s);
    if (nu >= 11 && nu <= 16) return launch<rope_vec_kernel<T, ADJ, PART, 16>, true>(p, rows, 2, s);
    if (nu >= 17) return launch<rope_vec_kernel<T, ADJ, PART, 32>, true>(p, rows, 1, s);
    return launch<rope_vec_kernel<T, ADJ, PART, 0>>(p, rows, 32 / nu, s);
}

template <typename T>
te_status run(RopeParams &p, const te_rope_axes &pl, int rows, cudaStream_t s) {
    const int rot = 2 * pl.pairs, hd = pl.hd;
    bool vec = true;                            // pieces of 4 channels, 4-aligned, on both sides of a pair
    if (pl.pairing == TE_ROPE_SECTION_HALVES)
        for (int a = 0; a < pl.axes; ++a) vec = vec && pl.sections[a] % 8 == 0;
    else if (pl.pairing == TE_ROPE_HEAD_HALVES)
        vec = rot % 8 == 0;
    if (vec) {
        int u = 0, pr = 0;
        auto unit = [&](int c1, int c2, int p0) {
            p.c1[u] = (uint8_t)c1;
            p.c2[u] = (uint8_t)c2;
            p.p0[u++] = (uint8_t)p0;
        };
        if (pl.pairing == TE_ROPE_ADJACENT) {
            for (; u < hd / 8;) unit(8 * u, 8 * u + 4, 4 * u);
        } else {
            const int n = pl.pairing == TE_ROPE_HEAD_HALVES ? 1 : pl.axes;
            for (int a = 0, start = 0; a < n; ++a) {
                const int sec = n == 1 ? rot : pl.sections[a];
                for (int i = 0; i < sec / 2; i += 4, pr += 4) unit(start + i, start + sec / 2 + i, pr);
                start += sec;
            }
            for (int c = rot; c < hd; c += 8) unit(c, c + 4, TE_ROPE_MAX_PAIRS);
        }
        if (pl.pairing == TE_ROPE_ADJACENT)
            return rot < hd ? launch_vec<T, true, true>(p, rows, s) : launch_vec<T, true, false>(p, rows, s);
        return rot < hd ? launch_vec<T, false, true>(p, rows, s) : launch_vec<T, false, false>(p, rows, s);
    }
    int pr = 0;
    for (int a = 0, start = 0; a < pl.axes; ++a) {
        const int sec = pl.sections[a];
        for (int i = 0; i < sec / 2; ++i, ++pr) {
            p.c1[pr] = (uint8_t)(pl.pairing == TE_ROPE_SECTION_HALVES ? start + i : pr);
            p.c2[pr] = (uint8_t)(pl.pairing == TE_ROPE_SECTION_HALVES ? start + i + sec / 2 : pr + rot / 2);
        }
        start += sec;
    }
    for (; pr < hd / 2; ++pr) {                 // the channels that do not turn
        p.c1[pr] = (uint8_t)(2 * pr);
        p.c2[pr] = (uint8_t)(2 * pr + 1);
    }
    if (hd <= 64) return launch<rope_any_kernel<T, 1>>(p, rows, 1, s);
    return hd <= 128 ? launch<rope_any_kernel<T, 2>>(p, rows, 1, s) : launch<rope_any_kernel<T, 4>>(p, rows, 1, s);
}

// f / (2 pi) in 2^-64 turns, modulo whole turns, to the nearest (f finite, >= 0).
// The method is Payne and Hanek's (1983): f = M 2^e with a 53-bit integer M, and
// of the bits of 1 / (2 pi) those left of e give whole turns, those right of
// e + 128 less than 2^-11 units; the 128 between, times M, are an exact integer
// product.  A product in f64 would be off by 2^-53 of f: 1e-4 turns at f = 1000
// and position 2^30.
uint64_t turn_word(double f) {
    // the fraction bits of 1 / (2 pi), first ones first (from Machin's formula)
    static const uint64_t bits[18] = {
        0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull, 0x7f9458eaf7aef158ull, 0x6dc91b8e909374b8ull,
        0x01924bba82746487ull, 0x3f877ac72c4a69cfull, 0xba208d7d4baed121ull, 0x3a671c09ad17df90ull, 0x4e64758e60d4ce7dull,
        0x272117e2ef7e4a0eull, 0xc7fe25fff7816603ull, 0xfbcbc462d6829b47ull, 0xdb4d9fb3c9f2c26dull, 0xd3d18fd9a797fa8bull,
        0x5d49eeb1faf97c5eull, 0xcf41ce7de294a4baull, 0x9afed7ec47e35742ull};
    int e;
    const uint64_t m = (uint64_t)ldexp(frexp(f, &e), 53);
    e -= 53;                                    // -1126 .. 971
    unsigned __int128 x = 0;                    // bits e .. e + 127 behind the point, zero ahead of it
    for (int i = 0; i < 18; ++i) {
        const int sh = e + 64 - 64 * i;         // word i's place: its last bit is worth 2^sh
        if (sh >= 128 || sh <= -64) continue;
        x += sh >= 0 ? (unsigned __int128)bits[i] << sh : (unsigned __int128)(bits[i] >> -sh);
    }
    const unsigned __int128 prod = x * m;       // modulo 2^128: whole turns go
    return (uint64_t)((prod + ((unsigned __int128)1 << 63)) >> 64);
}

// A plan whose fields the kernels may index by.
te_status check_plan(const te_rope_axes *pl, int32_t hd) {
    if (pl->hd != hd) return fail(TE_ESHAPE, "qk_rope_axes: plan for hd=%d, heads of %d", pl->hd, hd);
    if (hd < 8 || hd > 2 * TE_ROPE_MAX_PAIRS || hd % 8) return fail(TE_EINVAL, "qk_rope_axes: not an initialised plan");
    if (pl->axes < 1 || pl->axes > TE_ROPE_MAX_AXES || pl->pairing < TE_ROPE_SECTION_HALVES ||
        pl->pairing > TE_ROPE_ADJACENT)
        return fail(TE_EINVAL, "qk_rope_axes: not an initialised plan");
    int64_t rot = 0;
    for (int a = 0; a < pl->axes; ++a) {
        if (pl->sections[a] < 2 || pl->sections[a] % 2) return fail(TE_EINVAL, "qk_rope_axes: not an initialised plan");
        rot += pl->sections[a];
    }
    if (rot > hd || pl->pairs != rot / 2) return fail(TE_EINVAL, "qk_rope_axes: not an initialised plan");
    for (int i = 0; i < pl->pairs; ++i)
        if (pl->axis[i] >= pl->axes) return fail(TE_EINVAL, "qk_rope_axes: not an initialised plan");
    return TE_OK;
}

}  // namespace
}  // namespace tefwd

using namespace tefwd;

extern "C" size_t te_rope_axes_size(void) { return sizeof(te_rope_axes); }

extern "C" te_status te_rope_axes_init(te_rope_axes *plan, int32_t hd, int32_t axes,
                                       const int32_t *sections, double theta, int32_t whole,
                                       int32_t pairing, const double *freq) {
    if (!plan || !sections) return fail(TE_EINVAL, "rope_axes_init: NULL plan or sections");
    if (hd < 8 || hd > 2 * TE_ROPE_MAX_PAIRS || hd % 8)
        return fail(TE_ESHAPE, "rope_axes_init: hd=%d (hd %% 8 == 0, 8..%d)", hd, 2 * TE_ROPE_MAX_PAIRS);
    if (axes < 1 || axes > TE_ROPE_MAX_AXES)
        return fail(TE_ESHAPE, "rope_axes_init: axes=%d (1..%d)", axes, TE_ROPE_MAX_AXES);
    if (pairing < TE_ROPE_SECTION_HALVES || pairing > TE_ROPE_ADJACENT)
        return fail(TE_EINVAL, "rope_axes_init: bad pairing %d", pairing);
    if (!freq && !(theta > 0.0 && theta < HUGE_VAL))
        return fail(TE_EINVAL, "rope_axes_init: theta must be positive and finite");
    int64_t rot = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 2 || sections[a] % 2)
            return fail(TE_ESHAPE, "rope_axes_init: section %d is %d channels (even, >= 2)", a, sections[a]);
        rot += sections[a];
    }
    if (rot > hd) return fail(TE_ESHAPE, "rope_axes_init: sections hold %lld channels, a head %d", (long long)rot, hd);
    double f[TE_ROPE_MAX_PAIRS];
    int p = 0;
    for (int a = 0; a < axes; ++a)
        for (int i = 0; i < sections[a] / 2; ++i, ++p) {
            const double e = whole ? 2.0 * p / (double)rot : 2.0 * i / (double)sections[a];
            f[p] = freq ? freq[p] : pow(theta, -e);
            if (!(f[p] >= 0.0 && f[p] < HUGE_VAL))
                return freq ? fail(TE_EINVAL, "rope_axes_init: freq[%d] must be finite and >= 0", p)
                            : fail(TE_EINVAL, "rope_axes_init: theta^-%g is past an f64", e);
        }
    memset(plan, 0, sizeof(*plan));
    plan->hd = hd;
    plan->axes = axes;
    plan->pairs = (int32_t)(rot / 2);
    plan->pairing = pairing;
    p = 0;
    for (int a = 0; a < axes; ++a) {
        plan->sections[a] = sections[a];
        for (int i = 0; i < sections[a] / 2; ++i, ++p) {
            plan->axis[p] = (uint8_t)a;
            plan->turn[p] = turn_word(f[p]);
        }
    }
    return TE_OK;
}

extern "C" te_status te_qk_rope_axes(const void *src, int64_t ld_src, void *dst, int64_t ld_dst,
                                     int32_t dt, int32_t q_off, int32_t k_off, int32_t nq, int32_t nkv,
                                     int32_t hd, const float *qn, const float *kn, float eps,
                                     const te_rope_axes *plan, const int32_t *pos, int64_t ldp,
                                     float q_mul, int32_t rows, te_stream stream) {
    if (!plan || (rows > 0 && (!src || !dst || !pos)))
        return fail(TE_EINVAL, "qk_rope_axes: NULL src, dst, plan or pos");
    if (dt != TE_F32 && dt != TE_BF16) return fail(TE_EINVAL, "qk_rope_axes: bad dtype");
    const te_status ps = check_plan(plan, hd);
    if (ps != TE_OK) return ps;
    if (nq < 0 || nkv < 0 || rows < 0 || q_off < 0 || k_off < 0 || nq + (int64_t)nkv > 65535)
        return fail(TE_ESHAPE, "qk_rope_axes: negative size or offset, or more than 65535 heads");
    const int64_t ld_min = ld_src < ld_dst ? ld_src : ld_dst;
    if ((nq && (int64_t)q_off + (int64_t)nq * hd > ld_min) || (nkv && (int64_t)k_off + (int64_t)nkv * hd > ld_min))
        return fail(TE_ESHAPE, "qk_rope_axes: heads run past the row (ld %lld and %lld)", (long long)ld_src,
                    (long long)ld_dst);
    if (nq && nkv && (int64_t)q_off < (int64_t)k_off + (int64_t)nkv * hd && (int64_t)k_off < (int64_t)q_off + (int64_t)nq * hd)
        return fail(TE_ESHAPE, "qk_rope_axes: q and k heads overlap");
    if (ldp < plan->axes) return fail(TE_ESHAPE, "qk_rope_axes: ldp=%lld below %d axes", (long long)ldp, plan->axes);
    if (src == dst && ld_src != ld_dst) return fail(TE_EINVAL, "qk_rope_axes: in place needs ld_src == ld_dst");
    if ((qn == nullptr) != (kn == nullptr)) return fail(TE_EINVAL, "qk_rope_axes: give both qn and kn or neither");
    const int el = dt == TE_F32 ? 4 : 2;
    if (!aligned16(src) || !aligned16(dst) || (ld_src * el) % 16 || (ld_dst * el) % 16 || ((int64_t)q_off * el) % 16 ||
        ((int64_t)k_off * el) % 16 || (qn && !aligned16(qn)) || (kn && !aligned16(kn)) ||
        (reinterpret_cast<uintptr_t>(pos) & 3))
        return fail(TE_EALIGN, "qk_rope_axes: rows, head offsets and norm weights must be 16-byte aligned");
    if (rows == 0 || nq + nkv == 0) return TE_OK;
    RopeParams p;
    p.src = src;
    p.dst = dst;
    p.qn = qn;
    p.kn = kn;
    p.pos = pos;
    p.lds = ld_src;
    p.ldd = ld_dst;
    p.ldp = ldp;
    p.q_off = q_off;
    p.k_off = k_off;
    p.nq = nq;
    p.nkv = nkv;
    p.hd = hd;
    p.eps = eps;
    p.q_mul = q_mul;
    p.inv_hd = 1.f / (float)hd;
    p.pairs = plan->pairs;
    memcpy(p.axis, plan->axis, sizeof(p.axis));
    memcpy(p.turn, plan->turn, sizeof(p.turn));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dt == TE_F32 ? run<float>(p, *plan, rows, s) : run<__nv_bfloat16>(p, *plan, rows, s);
}
