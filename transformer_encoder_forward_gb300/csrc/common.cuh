// Shared host and device helpers of the tefwd library (sm_103a).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>
#include <stdio.h>

#include "tefwd.h"

namespace tefwd {

// ------------------------------------------------------------------ host side

// Records a message for te_last_error() and returns `st`.
te_status fail(te_status st, const char *fmt, ...);
// Records a CUDA launch/runtime failure.
te_status cuda_fail(cudaError_t e, const char *what);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Validates host cu_seqlens: cu[0] == 0, strictly increasing.  Writes the
// total row count and the longest sequence.
te_status check_cu(const int32_t *cu_host, const int32_t *cu_dev, int32_t nseq,
                   int32_t *total, int32_t *max_len);

// Host validation of an encoder block descriptor (block.cu).
te_status check_block_desc(const te_block_desc *d);

// Encodes a 2-D tiled TMA descriptor (row-major, `inner` elements per row,
// `outer` rows, `row_bytes` apart) for a box of box_inner x box_outer.
te_status make_map_2d(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner,
                      uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                      CUtensorMapSwizzle sw);

// The tensor-core products of 8-bit activations (q8_linear.cu): xh is the
// activation widened to f16 [m, k], ts its token scales; arguments checked.
te_status i8_gemm_linear(const void *xh, const float *ts, int32_t m, int32_t k, const te_q8_item *items, int32_t z,
                         cudaStream_t s);
te_status i8_gemm_gated(const void *xh, const float *ts, int32_t m, int32_t k, const te_q8w *wg, const te_q8w *wu,
                        int32_t act, void *out, int64_t ldm, cudaStream_t s);

// The token tile and the tiles a unit of their first launch.
void i8_gemm_tile(int m, int k, int ftiles, int32_t &tokens, int32_t &tiles);

// SMs of the current device.
int sm_count();

// Bounded-wait error words: each translation unit with bounded waits owns one
// and exposes a reader that returns and clears it (0 = nothing happened).
int read_clear_gemm_error();
int read_clear_attn_error();
// Device address of the products' error word, for kernels of other
// translation units that report there.
te_status gemm_error_word(int **word);

// ---------------------------------------------------------------- device side

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Pairs of f32 in one 64-bit register for the paired f32x2 arithmetic of
// sm_100 and later (one instruction, two lanes of work, each rounded as the
// scalar operation would be).
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// max of three (one instruction)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The FFN gate activations: GELU with the tanh approximation,
// 0.5 g (1 + tanh(z)), z = sqrt(2/pi) (g + 0.044715 g^3), and SiLU,
// g / (1 + e^-g).  Both are written through the logistic function, using
// 0.5 (1 + tanh z) = 1 / (1 + e^-2z): g * sigma(2z) and g * sigma(g), with
// e^y = 2^(y log2 e) on the hardware exp2 and reciprocal (relative error
// ~1e-7, far below the bf16 rounding that follows).
__device__ __forceinline__ float hw_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float hw_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float apply_act(float g, int act) {
    // -2 z log2(e) for GELU-tanh; -g log2(e) for SiLU
    const float t = act == TE_ACT_GELU_TANH
                        ? g * fmaf(-0.10294324f, g * g, -2.3022082f)   // -2*log2e*sqrt(2/pi)*(1 + 0.044715 g^2)
                        : -1.4426950408889634f * g;
    // exp2 of a large t is +inf: g * rcp(inf) = g * 0 = 0, the right limit
    return g * hw_rcp(1.f + hw_exp2(t));
}

// The same activations through the hardware tanh, one special-function op
// instead of two: 0.5 g (1 + tanh z) for GELU-tanh, 0.5 g (1 + tanh(g/2))
// for SiLU (g sigma(g) = 0.5 g (1 + tanh(g/2))).  tanh.approx has a relative
// error near 2^-11, below the bf16 rounding of the result; the GEMM epilogue
// uses it, where the special-function unit bounds the drain of the gate.
__device__ __forceinline__ float hw_tanh(float x) {
    float y;
    asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float apply_act_tanh(float g, int act) {
    const float z = act == TE_ACT_GELU_TANH
                        ? g * fmaf(0.035677408f, g * g, 0.79788456f)   // sqrt(2/pi) (g + 0.044715 g^3)
                        : 0.5f * g;
    const float h = 0.5f * g;
    return fmaf(h, hw_tanh(z), h);
}

// Rounds to the nearest bfloat16 (ties to even) and back: the value a bf16
// store would keep.
__device__ __forceinline__ float round_bf16(float v) {
    return __bfloat162float(__float2bfloat16_rn(v));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ----------------------------------------------------------------- mbarrier

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for the phase of parity `parity` to complete.  Gives up after about
// `limit_ns` nanoseconds (default 200 ms, far above any legitimate wait inside
// one tile) and returns false, so that a broken pipeline ends the kernel with
// an error flag instead of hanging the GPU.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity,
                                          uint64_t limit_ns = 200000000ull) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 0 && globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// Cluster-scope variants, for barriers that receive arrivals from the peer
// CTA of a cluster (the peer's writes before its arrive are then visible).
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity,
                                                  uint64_t limit_ns = 200000000ull) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((it & 255u) == 0 && globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// The shared::cluster address of `local` (a shared::cta address of this CTA)
// in the shared memory of cluster CTA `rank`.
__device__ __forceinline__ uint32_t mapa_shared(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

// Arrives on an mbarrier given by its shared::cluster address (own or peer CTA).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}

// The same arrival without release semantics.  Only for signals whose payload
// is tensor-memory state the arriving thread has already waited for
// (tcgen05.wait::st / wait::ld, then tcgen05.fence::before_thread_sync): no
// generic-memory write has to be published with it, and a cluster-scope
// release costs about a microsecond.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}

// ----------------------------------------------------------------------- TMA

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void *map, uint32_t bar, int32_t c0,
                                            int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

// tma_load_2d / mbar_arrive_expect_tx issued by the lane whose `e` is set
// (the rest of the warp runs the same loop in step).
__device__ __forceinline__ void tma_load_2d_e(uint32_t dst, const void *map, uint32_t bar, int32_t c0,
                                              int32_t c1, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(e)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_e(uint32_t bar, uint32_t bytes, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(e)
        : "memory");
}

// Tensor store of a box from shared memory (plain layout, no swizzle) to
// global memory at element coordinates (c0 inner, c1 outer); rows past the
// tensor's extent are not written.  c0 * element size must be a multiple of
// 16 bytes and neither coordinate may be negative.
__device__ __forceinline__ void tma_store_2d(const void *map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
}

// As tma_store_2d, but adds the box into global memory (f32: one rounding).
__device__ __forceinline__ void tma_reduce_add_2d(const void *map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// Waits until the bulk stores committed so far have finished reading shared
// memory (the source buffer may be overwritten).
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Waits until at most N of the bulk store groups committed so far are still
// reading shared memory (N = 0: bulk_wait_read).
template <int N>
__device__ __forceinline__ void bulk_wait_read_n() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Waits until the bulk stores committed so far are complete.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Orders this thread's shared-memory writes before later bulk (async proxy) reads.
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Contiguous bulk copy global -> this CTA's shared memory, completing on
// `bar` (both addresses 16-byte aligned, bytes a multiple of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// bulk_load issued by the lane whose `e` is set.
__device__ __forceinline__ void bulk_load_e(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar,
                                            uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar), "r"(e)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_desc(const void *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ------------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Whole warp: allocates `ncols` TMEM columns, the base address lands in smem.
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

// D(tmem) (+)= A(tmem) * B(smem desc), kind::f16 (bf16 operands, f32 accumulate).
__device__ __forceinline__ void mma_ts_bf16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D(tmem) (+)= A(smem desc) * B(smem desc), kind::f16.
__device__ __forceinline__ void mma_ss_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a converged warp: 1 there, 0 elsewhere (elect.sync).  A warp
// that runs its issue loop in step and lets only the elected lane issue keeps
// the loop's values (descriptors, addresses) warp-uniform, so the tensor
// instructions take them straight from uniform registers.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e;
}

// mma_ss_bf16 / mma_ts_bf16 / mma_commit issued by the lane whose `e` is set.
__device__ __forceinline__ void mma_ss_bf16_e(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
        : "memory");
}
__device__ __forceinline__ void mma_ts_bf16_e(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(e)
        : "memory");
}
__device__ __forceinline__ void mma_commit_e(uint32_t bar, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(e)
        : "memory");
}

// Arrives on `bar` once every tcgen05.mma issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 lanes x 32 consecutive 32-bit columns: lane i of the warp gets TMEM lane
// (quadrant base + i), columns [col, col+32).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

// 32 lanes x 64 consecutive 32-bit columns (one wait covers all of them).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Shared-memory matrix descriptor of a K-major operand tile stored with the
// 128-byte swizzle (rows of 128 bytes, 8-row groups 1024 bytes apart; the
// tile base 1024-byte aligned).
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);         // start address
    d |= (uint64_t)1 << 16;                            // leading byte offset (unused here)
    d |= (uint64_t)(1024u >> 4) << 32;                 // stride byte offset: 8 rows
    d |= (uint64_t)1 << 46;                            // descriptor version
    d |= (uint64_t)2 << 61;                            // 128-byte swizzle
    return d;
}

// Instruction descriptor for kind::f16: bf16 A and B (K-major), f32 D.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
    return (1u << 4)                              // D format f32
           | (1u << 7)                            // A format bf16
           | (1u << 10)                           // B format bf16
           | ((uint32_t)(N >> 3) << 17)           // N / 8
           | ((uint32_t)(M >> 4) << 24);          // M / 16
}

// The same for f16 A and B.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
    return (1u << 4)                              // D format f32; A and B format 0: f16
           | ((uint32_t)(N >> 3) << 17)           // N / 8
           | ((uint32_t)(M >> 4) << 24);          // M / 16
}

// ------------------------------------------- launches that follow closely
//
// A kernel launched by launch_close may start once the CTAs of the stream's
// previous kernel have all ended or called next_go: its start (placement,
// barriers, TMEM) then overlaps the end of the other.  It has to call
// prior_wait, in every thread, before it touches global memory: that returns
// when the previous kernel has ended and all of its writes are to be seen, and
// since that one waited too, everything before it has ended as well.  So:
//   * next_go comes after the kernel's own prior_wait and after its TMEM
//     allocation (a later kernel's allocation must not be waited for);
//   * a kernel whose CTAs work through many rows calls it behind its last one
//     (32760 rotated rows: at the start 161.4 us, as the last row begins 159.3,
//     behind it 158.1; 8448 x 3840 f32 norm and quantisation: 29.7, 34.5, 29.3),
//     and the large pipeline not at all (a widening pass waiting beside its last
//     units: 12297 x 8768 gated 2 x 128 98 -> 108 us);
//   * nothing is read through the read-only path (__ldg, const __restrict__),
//     whose loads the compiler may move above the wait.
// The calls of a block follow one another at 1 to 3 us less each: 1023 rows of 16
// heads of 72 rotated 6.2 -> 3.7 us, 101 x 768 x 2304 8.2 -> 5.2, quantisation and
// product 16238 x 512 x 512 24.7 -> 20.4, norm, widening and product 2112 x 3840 x
// 11520 135 -> 130.
__device__ __forceinline__ void prior_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Asks for memory that the previous kernel may still write: nothing is read.
__device__ __forceinline__ void l2_prefetch(const void *p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
template <typename... P, typename... A>
cudaError_t launch_close(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// int8 x4 -> two f16x2 words, exactly.  u = q + 128 as the low byte of the f16
// pattern 0x64xx reads 1024 + q + 128; one paired subtraction of 1152 leaves
// q, which needs 8 of f16's 11 significant bits.
__device__ __forceinline__ void widen4_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&l);
    hi = *reinterpret_cast<const uint32_t *>(&h);
}

// --------------------------------------------- draining an accumulator block

// apply_act of two values, the same operations in f32 pairs where there are such.
template <int ACT>
__device__ __forceinline__ uint64_t act_pair(uint64_t g2) {
    const uint64_t one2 = f2_pack(1.f, 1.f);
    const uint64_t t2 = ACT == TE_ACT_GELU_TANH
                            ? f2_mul(g2, f2_fma(f2_pack(-0.10294324f, -0.10294324f), f2_mul(g2, g2),
                                                f2_pack(-2.3022082f, -2.3022082f)))
                            : f2_mul(g2, f2_pack(-1.4426950408889634f, -1.4426950408889634f));
    float t0, t1;
    f2_unpack(t2, t0, t1);
    f2_unpack(f2_fma(f2_pack(hw_exp2(t0), hw_exp2(t1)), one2, one2), t0, t1);
    return f2_mul(g2, f2_pack(hw_rcp(t0), hw_rcp(t1)));
}

// One 32-token block of the gated form, in a draining warp whose lanes 0-15
// hold the gate rows and 16-31 the up rows of its 16 features: v becomes the
// outputs yv, lane l's for tokens 0-15 of feature l and lane l + 16's for
// tokens 16-31.  Scale and bias, then gate lane l and up lane l + 16 swap half
// their tokens, then m = act(g) * u, in f32 pairs.  bf16 activations: both
// halves are rounded to bf16 before the gate, as a stored g|u panel would be,
// and the activation takes the hardware tanh (error below that rounding).
// 8-bit activations (ts: the block's 32 token scales in shared memory): g and
// u stay f32 and the activation is exact to f32 rounding, so that the output
// is rounded once.  act: a constant where the caller keeps a copy of the code
// an activation, a variable where one copy that selects is enough.
template <bool I8>
__device__ __forceinline__ void gate_block(const uint32_t (&v)[32], float sc, float bi, const float *ts, bool upper,
                                           int act, float (&yv)[16]) {
    const uint64_t sc2 = f2_pack(sc, sc), bi2 = f2_pack(bi, bi), half2 = f2_pack(0.5f, 0.5f);
    float gv[16], uv[16];
    float4 ta, tb;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        uint64_t v2 = f2_pack(__uint_as_float(v[j]), __uint_as_float(v[16 + j]));
        if constexpr (I8) {
            if ((j & 3) == 0) {
                ta = *reinterpret_cast<const float4 *>(ts + j);
                tb = *reinterpret_cast<const float4 *>(ts + 16 + j);
            }
            const float t0 = (j & 3) == 0 ? ta.x : ((j & 3) == 1 ? ta.y : ((j & 3) == 2 ? ta.z : ta.w));
            const float t1 = (j & 3) == 0 ? tb.x : ((j & 3) == 1 ? tb.y : ((j & 3) == 2 ? tb.z : tb.w));
            v2 = f2_mul(v2, f2_pack(t0, t1));
        }
        float lo, hi;
        f2_unpack(f2_fma(v2, sc2, bi2), lo, hi);
        if constexpr (!I8) {
            const uint32_t b2 = pack_bf16x2(lo, hi);
            lo = bf16_lo(b2);
            hi = bf16_hi(b2);
        }
        // the gate lane sends its token 16 + j, the up lane its token j
        const float got = __shfl_xor_sync(0xFFFFFFFFu, upper ? lo : hi, 16);
        // operands selected first: one activation per lane, no branch
        gv[j] = upper ? got : lo;
        uv[j] = upper ? hi : got;
    }
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        if constexpr (I8) {
            const uint64_t g2 = f2_pack(gv[j], gv[j + 1]);
            const uint64_t a2 = act == TE_ACT_GELU_TANH ? act_pair<TE_ACT_GELU_TANH>(g2) : act_pair<TE_ACT_SILU>(g2);
            f2_unpack(f2_mul(a2, f2_pack(uv[j], uv[j + 1])), yv[j], yv[j + 1]);
        } else {
            const uint64_t g2 = f2_pack(gv[j], gv[j + 1]);
            // GELU-tanh: z = g (0.79788456 + 0.035677408 g^2); SiLU: z = g / 2
            const uint64_t z2 = act == TE_ACT_GELU_TANH
                                    ? f2_mul(g2, f2_fma(f2_pack(0.035677408f, 0.035677408f), f2_mul(g2, g2),
                                                        f2_pack(0.79788456f, 0.79788456f)))
                                    : f2_mul(half2, g2);
            float z0, z1;
            f2_unpack(z2, z0, z1);
            const uint64_t h2 = f2_mul(half2, g2);
            const uint64_t a2 = f2_fma(h2, f2_pack(hw_tanh(z0), hw_tanh(z1)), h2);
            f2_unpack(f2_mul(a2, f2_pack(uv[j], uv[j + 1])), yv[j], yv[j + 1]);
        }
    }
}

// s*acc + b of one 32-token block in place (f32 bits), two tokens an
// instruction; 8-bit activations: (acc * ts) * s + b with the block's 32 token
// scales ts in shared memory.
template <bool I8>
__device__ __forceinline__ void scale_block(uint32_t (&v)[32], float sc, float bi, const float *ts) {
    const uint64_t sc2 = f2_pack(sc, sc), bi2 = f2_pack(bi, bi);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        uint64_t a2 = f2_pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
        uint64_t b2 = f2_pack(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
        if constexpr (I8) {
            const float4 t = *reinterpret_cast<const float4 *>(ts + j);
            a2 = f2_mul(a2, f2_pack(t.x, t.y));
            b2 = f2_mul(b2, f2_pack(t.z, t.w));
        }
        float y0, y1, y2, y3;
        f2_unpack(f2_fma(a2, sc2, bi2), y0, y1);
        f2_unpack(f2_fma(b2, sc2, bi2), y2, y3);
        v[j] = __float_as_uint(y0);
        v[j + 1] = __float_as_uint(y1);
        v[j + 2] = __float_as_uint(y2);
        v[j + 3] = __float_as_uint(y3);
    }
}

// The ungated MLP's activation of one block, act(bf16(y)); 8-bit activations:
// act(y) of the f32 value.
template <bool I8>
__device__ __forceinline__ void act_block(uint32_t (&v)[32], int act) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const float y = __uint_as_float(v[j]);
        v[j] = __float_as_uint(I8 ? apply_act(y, act) : apply_act_tanh(round_bf16(y), act));
    }
}

}  // namespace tefwd
