// q/k norm and rotary positions with several axes (time, height, width, ...).
//
// Pair p of a head turns by pos[row, axis(p)] * f_p radians:
//     (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin).
// Angles are kept as 64-bit fixed-point fractions of a turn: f_p / (2 pi) as a
// word of 2^-64 turns (te_rope_axes.turn), times the position, modulo 2^64.
// The integer product wraps exactly where whole turns do, so the reduction
// loses nothing however far the position (the word itself is within 2^-53 of
// f_p, so 2^20 positions out an angle is off by about 2^-33 turns); its top
// 32 bits, read as a signed fraction, give sine and cosine by sincospif.  No
// table is read and no 64-bit float is touched on the device.
//
// Generalises the 1-D and 2-D rotation of "cortiq-engine 0.8.39
// src/gpu_metal/egemma2.rs" (Prog::qkv, EgQkv.sec) and "cortiq-engine 0.7.6
// src/gpu_metal/zimage.rs" (Enc::block) to axes of different widths.
#include <math.h>
#include <string.h>

#include "common.cuh"

namespace tefwd {
namespace {

struct RopeParams {
    const void *src;
    void *dst;
    const float *qn, *kn;
    const int32_t *pos;
    long long lds, ldd, ldp;
    int q_off, k_off, nq, nh, hd, rows, rot;
    float eps, q_mul;
    te_rope_axes plan;
};

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float *p, float v) { *p = v; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// cos and sin of position * (turn / 2^64) turns
__device__ __forceinline__ float2 turn_cs(int pos, unsigned long long turn) {
    const unsigned long long a = (unsigned long long)(long long)pos * turn;
    const int top = (int)(a >> 32);                       // turns in [-1/2, 1/2) * 2^32
    float s, c;
    sincospif((float)top * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    return make_float2(c, s);
}

// First and second channel of pair p.
__device__ __forceinline__ void pair_channels(const te_rope_axes &pl, int rot, int p, int &c1, int &c2) {
    if (pl.pairing == TE_ROPE_ADJACENT) {
        c1 = 2 * p;
        c2 = 2 * p + 1;
    } else if (pl.pairing == TE_ROPE_HEAD_HALVES) {
        c1 = p;
        c2 = p + rot / 2;
    } else {
        int start = 0, a = 0;
        while (a + 1 < pl.axes && p >= (start + pl.sections[a]) / 2) start += pl.sections[a++];
        c1 = start + (p - start / 2);
        c2 = c1 + pl.sections[a] / 2;
    }
}

// One warp per (row, head); lane l takes pairs l, l + 32, ... of the head and
// of the unrotated rest.
template <typename T>
__global__ void __launch_bounds__(256) rope_axes_kernel(const __grid_constant__ RopeParams p) {
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long row = item / p.nh;
    if (row >= p.rows) return;
    const int hh = (int)(item - row * p.nh);
    const bool isq = hh < p.nq;
    const int col = isq ? p.q_off + hh * p.hd : p.k_off + (hh - p.nq) * p.hd;
    const T *src = static_cast<const T *>(p.src) + row * p.lds + col;
    T *dst = static_cast<T *>(p.dst) + row * p.ldd + col;
    const int npairs = p.rot / 2;
    float x1[4], x2[4];
    int c1[4], c2[4];
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = lane + 32 * i;
        if (u < npairs) pair_channels(p.plan, p.rot, u, c1[i], c2[i]);
        else c1[i] = 2 * u, c2[i] = 2 * u + 1;          // unrotated
        if (u >= p.hd / 2) continue;
        x1[i] = ld(src + c1[i]);
        x2[i] = ld(src + c2[i]);
        q = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], q));
    }
    const float *nw = isq ? p.qn : p.kn;
    const float inv = nw ? rsqrtf(warp_sum(q) / (float)p.hd + p.eps) : 1.f;
    const float mul = isq ? p.q_mul : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = lane + 32 * i;
        if (u >= p.hd / 2) continue;
        float a = x1[i], b = x2[i];
        if (nw) {
            a *= inv * nw[c1[i]];
            b *= inv * nw[c2[i]];
        }
        if (u < npairs) {
            const float2 cs = turn_cs(p.pos[row * p.ldp + p.plan.axis[u]], p.plan.turn[u]);
            const float y1 = fmaf(a, cs.x, -b * cs.y), y2 = fmaf(b, cs.x, a * cs.y);
            a = y1;
            b = y2;
        }
        st(dst + c1[i], a * mul);
        st(dst + c2[i], b * mul);
    }
}

// A plan whose fields the kernels may index by.
te_status check_plan(const te_rope_axes *pl, int32_t hd) {
    if (pl->hd != hd) return fail(TE_ESHAPE, "qk_rope_axes: plan for hd=%d, heads of %d", pl->hd, hd);
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
    for (int p = 0; freq && p < rot / 2; ++p)
        if (!(freq[p] >= 0.0 && freq[p] < HUGE_VAL))
            return fail(TE_EINVAL, "rope_axes_init: freq[%d] must be finite and >= 0", p);
    memset(plan, 0, sizeof(*plan));
    plan->hd = hd;
    plan->axes = axes;
    plan->pairs = (int32_t)(rot / 2);
    plan->pairing = pairing;
    int p = 0;
    for (int a = 0; a < axes; ++a) {
        plan->sections[a] = sections[a];
        for (int i = 0; i < sections[a] / 2; ++i, ++p) {
            const double e = whole ? 2.0 * p / (double)rot : 2.0 * i / (double)sections[a];
            const double f = freq ? freq[p] : pow(theta, -e);
            const double turns = f * 0.15915494309189535;        // / 2 pi
            plan->axis[p] = (uint8_t)a;
            plan->turn[p] = (uint64_t)ldexp(turns - floor(turns), 64);   // < 2^64: an f64 below 1
        }
    }
    return TE_OK;
}

extern "C" te_status te_qk_rope_axes(const void *src, int64_t ld_src, void *dst, int64_t ld_dst,
                                     int32_t dt, int32_t q_off, int32_t k_off, int32_t nq, int32_t nkv,
                                     int32_t hd, const float *qn, const float *kn, float eps,
                                     const te_rope_axes *plan, const int32_t *pos, int64_t ldp,
                                     float q_mul, int32_t rows, te_stream stream) {
    if (!src || !dst || !plan || !pos) return fail(TE_EINVAL, "qk_rope_axes: NULL src, dst, plan or pos");
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
    p.nh = nq + nkv;
    p.hd = hd;
    p.rows = rows;
    p.rot = 2 * plan->pairs;
    p.eps = eps;
    p.q_mul = q_mul;
    p.plan = *plan;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const long long ctas = ((long long)rows * p.nh + 7) / 8;
    if (ctas > 0x7FFFFFFFll) return fail(TE_ESHAPE, "qk_rope_axes: rows * heads too large");
    if (dt == TE_F32) rope_axes_kernel<float><<<(unsigned)ctas, 256, 0, s>>>(p);
    else rope_axes_kernel<__nv_bfloat16><<<(unsigned)ctas, 256, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "qk_rope_axes launch");
}
