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
#include "common.cuh"

namespace tefwd {
namespace {

constexpr int MAXZ = 4;

struct I8Item {
    const int8_t *w, *w2;          // w2: the up projection of the gated form
    const float *scale, *bias, *scale2, *bias2, *resid;
    void *y;
    long long ldy, ldr;
    int n, ydt, act, tile0;
};

struct I8Params {
    const int8_t *x;
    const float *xs;
    long long ldx;
    int m, k, z;
    I8Item it[MAXZ];
};

// 64 tokens x 64 features a CTA, 4 x 4 a thread, exact 32-bit integer sums by
// the 4-way byte dot product.
template <bool GATED>
__global__ void __launch_bounds__(256) i8_tile_kernel(const __grid_constant__ I8Params p) {
    __shared__ int xs[64][17], ws[GATED ? 128 : 64][17];
    int zi = 0;
    while (zi + 1 < p.z && (int)blockIdx.x >= p.it[zi + 1].tile0) ++zi;
    const I8Item &it = p.it[zi];
    const int o0 = ((int)blockIdx.x - it.tile0) * 64;
    const long long t0 = (long long)blockIdx.y * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {}, acc2[4][4] = {};
    for (int k0 = 0; k0 < p.k; k0 += 64) {
        const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 4;
        int4 v = make_int4(0, 0, 0, 0);
        if (t0 + r < p.m) v = *reinterpret_cast<const int4 *>(p.x + (t0 + r) * p.ldx + k0 + 4 * c);
        xs[r][c] = v.x; xs[r][c + 1] = v.y; xs[r][c + 2] = v.z; xs[r][c + 3] = v.w;
        v = make_int4(0, 0, 0, 0);
        if (o0 + r < it.n) v = *reinterpret_cast<const int4 *>(it.w + (long long)(o0 + r) * p.k + k0 + 4 * c);
        ws[r][c] = v.x; ws[r][c + 1] = v.y; ws[r][c + 2] = v.z; ws[r][c + 3] = v.w;
        if (GATED) {
            v = make_int4(0, 0, 0, 0);
            if (o0 + r < it.n) v = *reinterpret_cast<const int4 *>(it.w2 + (long long)(o0 + r) * p.k + k0 + 4 * c);
            ws[GATED ? 64 + r : 0][c] = v.x; ws[GATED ? 64 + r : 0][c + 1] = v.y;
            ws[GATED ? 64 + r : 0][c + 2] = v.z; ws[GATED ? 64 + r : 0][c + 3] = v.w;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    acc[a][b] = __dp4a(xs[ty + 16 * a][j], ws[tx + 16 * b][j], acc[a][b]);
                    if (GATED)
                        acc2[a][b] = __dp4a(xs[ty + 16 * a][j], ws[(GATED ? 64 : 0) + tx + 16 * b][j], acc2[a][b]);
                }
        __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const long long t = t0 + ty + 16 * a;
        if (t >= p.m) continue;
        const float sx = p.xs[t];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int o = o0 + tx + 16 * b;
            if (o >= it.n) continue;
            float y = fmaf((float)acc[a][b] * sx, it.scale[o], it.bias ? it.bias[o] : 0.f);
            if (GATED) y = apply_act(y, it.act) * fmaf((float)acc2[a][b] * sx, it.scale2[o], it.bias2 ? it.bias2[o] : 0.f);
            else if (it.act != TE_EPI_NONE) y = apply_act(y, it.act - 1);
            if (it.resid) y += it.resid[t * it.ldr + o];
            if (it.ydt == TE_F32) static_cast<float *>(it.y)[t * it.ldy + o] = y;
            else static_cast<__nv_bfloat16 *>(it.y)[t * it.ldy + o] = __float2bfloat16_rn(y);
        }
    }
}

// x int8 [m, k] (rows ldx apart) widened to f16 [m, k], exactly: 16 values a
// thread, 16 bytes in and 32 out.  q + 128 as the low byte of the f16 pattern
// 0x64xx reads 1024 + q + 128; subtracting 1152 leaves q.
__global__ void __launch_bounds__(256) widen_kernel(const int8_t *__restrict__ x, long long ldx,
                                                    __half *__restrict__ y, long long total, int chunks) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const long long r = i / chunks;
    const int c = (int)(i - r * chunks);
    const uint4 v = *reinterpret_cast<const uint4 *>(x + r * ldx + 16 * c);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u = in[j] ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
        out[2 * j] = *reinterpret_cast<const uint32_t *>(&l);
        out[2 * j + 1] = *reinterpret_cast<const uint32_t *>(&h);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(y + 16 * i);
    dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
    dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

te_status widen(const int8_t *x, int64_t ldx, void *y, int m, int k, cudaStream_t s) {
    const int chunks = k / 16;
    const long long total = (long long)m * chunks, blocks = (total + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return fail(TE_ESHAPE, "i8_linear: m * k too large");
    widen_kernel<<<(unsigned)blocks, 256, 0, s>>>(x, ldx, static_cast<__half *>(y), total, chunks);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "i8_linear: widen launch");
}

constexpr int SMALL_M = 8;
constexpr int MAX_K = 65536;

te_status check_x(const char *what, const void *x, int64_t ldx, const float *xs, int32_t m, int32_t k) {
    if (!x || !xs) return fail(TE_EINVAL, "%s: NULL x or x_scale", what);
    if (m < 0 || k < 64 || k > MAX_K || k % 64)
        return fail(TE_ESHAPE, "%s: m=%d k=%d (k %% 64 == 0, 64..%d)", what, m, k, MAX_K);
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

te_status launched(const char *what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TE_OK : cuda_fail(e, what);
}

}  // namespace
}  // namespace tefwd

using namespace tefwd;

extern "C" size_t te_i8_workspace(int32_t m, int32_t k, int32_t n) {
    if (m <= SMALL_M || k < 64 || k > MAX_K || k % 64 || n < 32) return 0;
    return ((size_t)m * k * 2 + 255) & ~(size_t)255;
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
    int tiles = 0;
    int64_t n = 0;
    for (int i = 0; i < z; ++i) {
        const te_q8_item &src = items[i];
        if ((st = check_w("i8_linear", i, src.w, k)) != TE_OK) return st;
        if (!src.y) return fail(TE_EINVAL, "i8_linear: item %d has a NULL y", i);
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
        d.tile0 = tiles;
        tiles += (src.w.n + 63) / 64;
        n += src.w.n;
    }
    if (n > 0x7FFFFFFFll) return fail(TE_ESHAPE, "i8_linear: too many output features");
    if ((st = check_ws("i8_linear", workspace, ws_bytes, te_i8_workspace(m, k, (int32_t)n))) != TE_OK) return st;
    if (m == 0) return TE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (m > SMALL_M) {
        if ((st = widen(x, ldx, workspace, m, k, s)) != TE_OK) return st;
        return i8_gemm_linear(workspace, x_scale, m, k, items, z, s);
    }
    i8_tile_kernel<false><<<dim3(tiles, (m + 63) / 64), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launched("i8_linear launch");
}

extern "C" te_status te_i8_gated_linear(const int8_t *x, int64_t ldx, const float *x_scale, int32_t m,
                                        int32_t k, const te_q8w *wg, const te_q8w *wu, int32_t act,
                                        void *out, int64_t ldm, void *workspace, size_t ws_bytes,
                                        te_stream stream) {
    if (!wg || !wu || !out) return fail(TE_EINVAL, "i8_gated_linear: NULL wg, wu or out");
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
    if ((st = check_ws("i8_gated_linear", workspace, ws_bytes, te_i8_workspace(m, k, 2 * f))) != TE_OK) return st;
    if (m == 0) return TE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (m > SMALL_M) {
        if ((st = widen(x, ldx, workspace, m, k, s)) != TE_OK) return st;
        return i8_gemm_gated(workspace, x_scale, m, k, wg, wu, act, out, ldm, s);
    }
    I8Params p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.xs = x_scale;
    p.ldx = ldx;
    p.m = m;
    p.k = k;
    p.z = 1;
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
    i8_tile_kernel<true><<<dim3((f + 63) / 64, (m + 63) / 64), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launched("i8_gated_linear launch");
}
