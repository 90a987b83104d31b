// Activations in 8 bits: each row (token) quantised with a scale of its own,
// alone (te_quant_rows) or behind the block's pre-norm (te_rownorm_quant).
//
//     a = max_j |v_j|,  scale = a / 127,  q_j = rint(v_j * (127 / a))
//
// with v = x, or v = Norm(pre * x) * w (+ b), times (1 + s).  Bound by HBM
// bandwidth: a row is read once (16-byte loads, all of a thread's chunks up
// front), stays in registers through the norm's reductions and the maximum,
// and leaves as 8-byte stores of q.  All arithmetic is f32; the normed value
// is not rounded to bf16 on the way, so the only rounding to fewer bits is
// the quantisation itself, at most half a step (scale / 2) a value.
//
// The maximum propagates NaNs, and its bit pattern, as an integer, orders like
// the values with infinities and NaNs above every finite one: one maximum finds
// the row's largest magnitude and whether any value is not finite.
#include <atomic>

#include "common.cuh"

namespace tefwd {
namespace {

enum QuantKind { QUANT_PLAIN = -1 };   // else a te_norm_kind

// Eight values of a row as loaded (read once: streaming loads).
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    }
};
// the per-feature vectors: shared by all rows, kept in cache
__device__ __forceinline__ void load8_vec(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// Largest magnitude of three, a NaN if any is one.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The WPR warps of a row meet: a barrier of their own.
template <int WPR>
__device__ __forceinline__ void row_bar(int slot) {
    if (WPR == 8) asm volatile("bar.sync 0;" ::: "memory");
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "n"(32 * WPR) : "memory");
}
// Sum / maximum of bit patterns over the warps of a row (every thread gets
// it).  `red` is one of two arrays used in turn: a reduction's readers are past
// it when the second next one writes it, by the barrier between.
template <int WPR>
__device__ __forceinline__ float row_sum(float x, float *red, int slot, int wr, int lane) {
    x = warp_sum(x);
    if (WPR == 1) return x;
    if (lane == 0) red[wr] = x;
    row_bar<WPR>(slot);
    float s = red[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) s += red[i];
    return s;
}
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x, float *red, int slot, int wr, int lane) {
    x = __reduce_max_sync(0xFFFFFFFFu, x);
    if (WPR == 1) return x;
    if (lane == 0) red[wr] = __uint_as_float(x);
    row_bar<WPR>(slot);
    uint32_t s = __float_as_uint(red[0]);
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
        const uint32_t o = __float_as_uint(red[i]);
        s = o > s ? o : s;
    }
    return s;
}

// WPR warps a row (8 / WPR rows a CTA at a time, persistent over rows), at most
// NV chunks of 8 columns a thread; the next row's loads are in flight while a
// row is worked on.  Registers are held to 2-4 CTAs an SM: rows in flight are
// what hides the row's chain of load, meetings, division and store (f32 8448 x
// 3840 behind an RMS norm: 28.0 us, 5.8 TB/s; LayerNorm 36.4; five CTAs with
// spills 41, one row a CTA without the loop 35).  The norm's factor is known
// before any value is scaled by it: a maximum found in the same meeting as the
// sum, over x w alone, saves 1 us there and rounds in another order than the
// norm does.
template <typename Tin, int NV, int WPR, bool NORM>
__global__ void __launch_bounds__(256, NV == 8 ? 2 : (NV == 4 || (NV == 2 && WPR == 1) ? 3 : 4))
    quant_kernel(const Tin *x, long long ldx, const float *w, const float *b, const float *ms, int kind, float eps, float pre,
                 int8_t *__restrict__ q, long long ldq, float *__restrict__ scale, int t, int d) {
    prior_wait();
    constexpr int TPR = 32 * WPR, RPC = 8 / WPR;
    __shared__ float red[2][8 / WPR][WPR];
    const int slot = threadIdx.x / TPR, tid = threadIdx.x % TPR;
    const int wr = tid >> 5, lane = tid & 31;
    int flip = 0;
    Raw8<Tin> nx[NV];
    auto fetch = [&](long long row) {
        const Tin *xr = x + row * ldx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tid) * 8;
            if (c < d) nx[i].load(xr + c);
            else nx[i].zero();
        }
    };
    long long row = (long long)blockIdx.x * RPC + slot;
    if (row < t) fetch(row);
    for (; row < t; row += (long long)gridDim.x * RPC) {   // uniform over the row's warps
        float v[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) nx[i].get(v[i]);
        const long long after = row + (long long)gridDim.x * RPC;
        if (after < t) fetch(after);
        if (NORM) {
            // te_rownorm_mod's steps in its order, each rounded as there: x pre,
            // (x - mean) inv, times w (plus b), times 1 + s
            if (pre != 1.f) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] *= pre;
            }
            if (kind == TE_NORM_LN) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s += v[i][e];
                const float mean = row_sum<WPR>(s, red[flip ^= 1][slot], slot, wr, lane) / (float)d;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if ((i * TPR + tid) * 8 < d)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[i][e] -= mean;
            }
            float s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) s2 = fmaf(v[i][e], v[i][e], s2);
            const float inv = rsqrtf(row_sum<WPR>(s2, red[flip ^= 1][slot], slot, wr, lane) / (float)d + eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + tid) * 8;
                if (c >= d) continue;
                float wv[8];
                load8_vec(w + c, wv);
                if (b) {
                    float bv[8];
                    load8_vec(b + c, bv);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = fmaf(v[i][e] * inv, wv[e], bv[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * inv * wv[e];
                }
                if (ms) {
                    load8_vec(ms + c, wv);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] *= 1.f + wv[e];
                }
            }
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 2) top = max3_abs_nan(top, v[i][e], v[i][e + 1]);
        const uint32_t mx = row_max<WPR>(__float_as_uint(top) & 0x7FFFFFFFu, red[flip ^= 1][slot], slot, wr, lane);
        // below 2^-120 the row counts as zero (127 / a would leave f32's range);
        // from the infinity's pattern up it holds a value that is not finite
        const bool finite = mx < 0x7F800000u, zero = mx < 0x03800000u;
        const float a = __uint_as_float(mx);
        const float up = finite && !zero ? __fdiv_rn(127.f, a) : 0.f;
        if (tid == 0) scale[row] = finite ? (zero ? 0.f : __fdiv_rn(a, 127.f)) : __uint_as_float(0x7FC00000u);
        int8_t *qr = q + row * ldq;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tid) * 8;
            if (c >= d) continue;
            uint32_t o[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // |v up| <= 127 (1 + 2^-22): rint cannot pass 127.  Adding 1.5 2^23
                // rounds to an integer (ties to even) and leaves it in the low byte.
                uint32_t r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r[e] = __float_as_uint(__fadd_rn(__fmul_rn(v[i][4 * h + e], up), 12582912.f));
                o[h] = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
            }
            *reinterpret_cast<uint2 *>(qr + c) = finite ? make_uint2(o[0], o[1]) : make_uint2(0u, 0u);
        }
        if (after >= t) next_go();
    }
}

template <typename Tin, auto KERN, int RPC>
te_status go(const void *x, int64_t ldx, const float *w, const float *b, const float *ms, int kind, float eps,
             float pre, int8_t *q, int64_t ldq, float *scale, int t, int d, cudaStream_t s) {
    // resident CTAs of the whole device, asked for once a kernel and device
    static std::atomic<int> resident[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cuda_fail(e, "quant: device");
    if (!resident[dev]) {
        int sms = 0, per = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, KERN, 256, 0);
        if (e != cudaSuccess || per < 1) return cuda_fail(e, "quant: occupancy");
        resident[dev] = sms * per;
    }
    const long long need = ((long long)t + RPC - 1) / RPC, most = resident[dev];
    e = launch_close(KERN, dim3((unsigned)(need < most ? need : most)), 256, 0, s, 1,
                     static_cast<const Tin *>(x), ldx, w, b, ms, kind, eps, pre, q, ldq, scale, t, d);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "quant launch");
}

template <typename Tin, bool NORM>
te_status launch(const void *x, int64_t ldx, const float *w, const float *b, const float *ms, int kind, float eps,
                 float pre, int8_t *q, int64_t ldq, float *scale, int t, int d, cudaStream_t s) {
    auto run = [&](auto f) { return f(x, ldx, w, b, ms, kind, eps, pre, q, ldq, scale, t, d, s); };
    if (d <= 256) return run(go<Tin, quant_kernel<Tin, 1, 1, NORM>, 8>);
    if (d <= 512) return run(go<Tin, quant_kernel<Tin, 2, 1, NORM>, 8>);
    if (d <= 1024) return run(go<Tin, quant_kernel<Tin, 1, 4, NORM>, 2>);
    if (d <= 2048) return run(go<Tin, quant_kernel<Tin, 1, 8, NORM>, 1>);
    if (d <= 4096) return run(go<Tin, quant_kernel<Tin, 2, 8, NORM>, 1>);
    if (d <= 8192) return run(go<Tin, quant_kernel<Tin, 4, 8, NORM>, 1>);
    return run(go<Tin, quant_kernel<Tin, 8, 8, NORM>, 1>);
}

te_status check(const char *what, const void *x, int32_t xdt, int64_t ldx, const int8_t *q, int64_t ldq,
                const float *scale, int32_t t, int32_t d) {
    if (t > 0 && (!x || !q || !scale)) return fail(TE_EINVAL, "%s: NULL x, q or scale", what);
    if (xdt != TE_F32 && xdt != TE_BF16) return fail(TE_EINVAL, "%s: bad dtype", what);
    if (t < 0 || d < 8 || d > 16384 || d % 8)
        return fail(TE_ESHAPE, "%s: t=%d d=%d (d %% 8 == 0, 8..16384)", what, t, d);
    if (ldx < d || ldq < d) return fail(TE_ESHAPE, "%s: leading dimension below d", what);
    if (!aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scale) & 3) ||
        ldx % (xdt == TE_F32 ? 4 : 8) || ldq % 16)
        return fail(TE_EALIGN, "%s: x, q and their rows must be 16-byte aligned, scale 4-byte", what);
    return TE_OK;
}

}  // namespace
}  // namespace tefwd

using namespace tefwd;

extern "C" te_status te_quant_rows(const void *x, int32_t xdt, int64_t ldx, int8_t *q, int64_t ldq,
                                   float *scale, int32_t t, int32_t d, te_stream stream) {
    const te_status st = check("quant_rows", x, xdt, ldx, q, ldq, scale, t, d);
    if (st != TE_OK) return st;
    if (t == 0) return TE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return xdt == TE_F32 ? launch<float, false>(x, ldx, nullptr, nullptr, nullptr, QUANT_PLAIN, 0.f, 1.f, q, ldq, scale,
                                                t, d, s)
                         : launch<__nv_bfloat16, false>(x, ldx, nullptr, nullptr, nullptr, QUANT_PLAIN, 0.f, 1.f, q, ldq,
                                                        scale, t, d, s);
}

extern "C" te_status te_rownorm_quant(const void *x, int32_t xdt, int64_t ldx, const float *w,
                                      const float *b, const float *mod_scale, int32_t kind, float eps,
                                      float pre, int8_t *q, int64_t ldq, float *scale, int32_t t,
                                      int32_t d, te_stream stream) {
    const te_status st = check("rownorm_quant", x, xdt, ldx, q, ldq, scale, t, d);
    if (st != TE_OK) return st;
    if (!w) return fail(TE_EINVAL, "rownorm_quant: NULL w");
    if (kind != TE_NORM_RMS && kind != TE_NORM_LN) return fail(TE_EINVAL, "rownorm_quant: bad kind");
    if (!aligned16(w) || (b && !aligned16(b)) || (mod_scale && !aligned16(mod_scale)))
        return fail(TE_EALIGN, "rownorm_quant: w, b and mod_scale must be 16-byte aligned");
    if (t == 0) return TE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const float *bias = kind == TE_NORM_LN ? b : nullptr;   // as te_rownorm: LN only
    return xdt == TE_F32
               ? launch<float, true>(x, ldx, w, bias, mod_scale, kind, eps, pre, q, ldq, scale, t, d, s)
               : launch<__nv_bfloat16, true>(x, ldx, w, bias, mod_scale, kind, eps, pre, q, ldq, scale, t, d, s);
}
