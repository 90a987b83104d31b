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
// The maximum is taken over the magnitudes' bit patterns as integers, whose
// order is the values' order with infinities and NaNs above every finite
// value: one integer maximum finds the row's largest magnitude and whether
// any value is not finite.
#include "common.cuh"

namespace tefwd {
namespace {

enum QuantKind { QUANT_PLAIN = -1 };   // else a te_norm_kind

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
}
// the per-feature vectors: shared by all rows, kept in cache
__device__ __forceinline__ void load8_vec(const float *p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sum / integer maximum over the WPR warps of a row (every thread gets it).
template <int WPR>
__device__ __forceinline__ float row_sum(float x, float (*red)[8], int slot, int wr, int lane) {
    x = warp_sum(x);
    if (WPR == 1) return x;
    __syncthreads();                    // earlier readers of red are done
    if (lane == 0) red[slot][wr] = x;
    __syncthreads();
    float s = red[slot][0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) s += red[slot][i];
    return s;
}
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x, float (*red)[8], int slot, int wr, int lane) {
    x = __reduce_max_sync(0xFFFFFFFFu, x);
    if (WPR == 1) return x;
    __syncthreads();
    if (lane == 0) red[slot][wr] = __uint_as_float(x);
    __syncthreads();
    uint32_t s = __float_as_uint(red[slot][0]);
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
        const uint32_t o = __float_as_uint(red[slot][i]);
        s = o > s ? o : s;
    }
    return s;
}

// WPR warps a row (8 / WPR rows a CTA), at most NV chunks of 8 columns a thread.
template <typename Tin, int NV, int WPR, bool NORM>
__global__ void __launch_bounds__(256)
    quant_kernel(const Tin *__restrict__ x, long long ldx, const float *__restrict__ w,
                 const float *__restrict__ b, const float *__restrict__ ms, int kind, float eps, float pre,
                 int8_t *__restrict__ q, long long ldq, float *__restrict__ scale, int t, int d) {
    constexpr int TPR = 32 * WPR;
    __shared__ float red[8][8];
    const int slot = threadIdx.x / TPR, tid = threadIdx.x % TPR;
    const int wr = tid >> 5, lane = tid & 31;
    const long long row = (long long)blockIdx.x * (8 / WPR) + slot;
    const bool active = row < t;        // idle threads still join the barriers
    const Tin *xr = x + (active ? row : 0) * ldx;
    float v[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tid) * 8;
        if (active && c < d) {
            load8(xr + c, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
        }
    }
    if (NORM) {
        float mean = 0.f;
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
            mean = row_sum<WPR>(s, red, slot, wr, lane) / (float)d;
        }
        float s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPR + tid) * 8 < d)
#pragma unroll
                for (int e = 0; e < 8; ++e) s2 += (v[i][e] - mean) * (v[i][e] - mean);
        const float inv = rsqrtf(row_sum<WPR>(s2, red, slot, wr, lane) / (float)d + eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tid) * 8;
            if (c >= d) continue;
            float wv[8];
            load8_vec(w + c, wv);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = (v[i][e] - mean) * inv * wv[e];
            if (b) {
                load8_vec(b + c, wv);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] += wv[e];
            }
            if (ms) {
                load8_vec(ms + c, wv);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] *= 1.f + wv[e];
            }
        }
    }
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t u = __float_as_uint(v[i][e]) & 0x7FFFFFFFu;
            mx = u > mx ? u : mx;
        }
    mx = row_max<WPR>(mx, red, slot, wr, lane);
    // below 2^-120 the row counts as zero (127 / a would leave f32's range);
    // from the infinity's pattern up it holds a value that is not finite
    const bool finite = mx < 0x7F800000u, zero = mx < 0x03800000u;
    const float a = __uint_as_float(mx);
    const float up = finite && !zero ? __fdiv_rn(127.f, a) : 0.f;
    if (!active) return;
    if (tid == 0) scale[row] = finite ? (zero ? 0.f : __fdiv_rn(a, 127.f)) : __uint_as_float(0x7FC00000u);
    int8_t *qr = q + row * ldq;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tid) * 8;
        if (c >= d) continue;
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // |v * up| <= 127 (1 + 2^-22): rint cannot pass 127
            const uint32_t b0 = __float2int_rn(__fmul_rn(v[i][4 * h + 0], up));
            const uint32_t b1 = __float2int_rn(__fmul_rn(v[i][4 * h + 1], up));
            const uint32_t b2 = __float2int_rn(__fmul_rn(v[i][4 * h + 2], up));
            const uint32_t b3 = __float2int_rn(__fmul_rn(v[i][4 * h + 3], up));
            o[h] = finite ? __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410) : 0u;
        }
        *reinterpret_cast<uint2 *>(qr + c) = make_uint2(o[0], o[1]);
    }
}

template <typename Tin, bool NORM>
void launch(const void *x, int64_t ldx, const float *w, const float *b, const float *ms, int kind, float eps,
            float pre, int8_t *q, int64_t ldq, float *scale, int t, int d, cudaStream_t s) {
    auto go = [&](auto kern, int rows) {
        kern<<<(unsigned)(((long long)t + rows - 1) / rows), 256, 0, s>>>(
            static_cast<const Tin *>(x), ldx, w, b, ms, kind, eps, pre, q, ldq, scale, t, d);
    };
    if (d <= 256) go(quant_kernel<Tin, 1, 1, NORM>, 8);
    else if (d <= 512) go(quant_kernel<Tin, 2, 1, NORM>, 8);
    else if (d <= 1024) go(quant_kernel<Tin, 1, 4, NORM>, 2);
    else if (d <= 2048) go(quant_kernel<Tin, 1, 8, NORM>, 1);
    else if (d <= 4096) go(quant_kernel<Tin, 2, 8, NORM>, 1);
    else if (d <= 8192) go(quant_kernel<Tin, 4, 8, NORM>, 1);
    else go(quant_kernel<Tin, 8, 8, NORM>, 1);
}

te_status check(const char *what, const void *x, int32_t xdt, int64_t ldx, const int8_t *q, int64_t ldq,
                const float *scale, int32_t t, int32_t d) {
    if (!x || !q || !scale) return fail(TE_EINVAL, "%s: NULL x, q or scale", what);
    if (xdt != TE_F32 && xdt != TE_BF16) return fail(TE_EINVAL, "%s: bad dtype", what);
    if (t < 0 || d < 8 || d > 16384 || d % 8)
        return fail(TE_ESHAPE, "%s: t=%d d=%d (d %% 8 == 0, 8..16384)", what, t, d);
    if (ldx < d || ldq < d) return fail(TE_ESHAPE, "%s: leading dimension below d", what);
    if (!aligned16(x) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scale) & 3) ||
        ldx % (xdt == TE_F32 ? 4 : 8) || ldq % 16)
        return fail(TE_EALIGN, "%s: x, q and their rows must be 16-byte aligned, scale 4-byte", what);
    return TE_OK;
}

te_status launched(const char *what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TE_OK : cuda_fail(e, what);
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
    if (xdt == TE_F32)
        launch<float, false>(x, ldx, nullptr, nullptr, nullptr, QUANT_PLAIN, 0.f, 1.f, q, ldq, scale, t, d, s);
    else
        launch<__nv_bfloat16, false>(x, ldx, nullptr, nullptr, nullptr, QUANT_PLAIN, 0.f, 1.f, q, ldq, scale, t,
                                     d, s);
    return launched("quant_rows launch");
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
    if (xdt == TE_F32)
        launch<float, true>(x, ldx, w, bias, mod_scale, kind, eps, pre, q, ldq, scale, t, d, s);
    else
        launch<__nv_bfloat16, true>(x, ldx, w, bias, mod_scale, kind, eps, pre, q, ldq, scale, t, d, s);
    return launched("rownorm_quant launch");
}
