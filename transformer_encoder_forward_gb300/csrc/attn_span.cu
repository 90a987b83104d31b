// Varlen attention with a window of its own to either side, a few first keys
// that stay visible, and a learned bias of relative position (sm_103a):
//
//     o[i, h] = sum_j softmax_j(scale * q[i, h] . k[j, g] + bias[bucket(j - i), h]) v[j, g]
//
// over the keys j of i's own sequence with
//     j <= i + right  and  (j >= i - left  or  j < sinks).
//
// One pass over the keys: with m a reference that is moved to the row's maximum
// when there was none, or when the maximum grew by more than 2^20, P = 2^(s - m),
// l = sum P and O = P V are kept in f32 (P itself rounds to bf16, as the operand
// of its product; l adds the P before they round), and o = O / l at the end.
//
// What bounds it.  A key costs 4 hd multiply-adds on the tensor core and one
// exponential; bytes are few (q, k, v read once, o written: 30 % of the copy rate
// where windows are short, 10 % where they are not).  A step of 64 keys and all
// query tiles of a CTA takes the tensor core 1200 (hd 64, 3 tiles) and 1250 (hd
// 128, 2 tiles) clocks; alone, the softmax takes 1286 and 993 for it.  Both run
// at once and take about 1500 together: two pipes that wait on one another
// through barriers of about 100 clocks.  Without a window or bias, 2 x 4224 rows with
// 30 heads of 128 run at 1420 TFLOP/s; with a window, partly seen tiles and the masks of
// their pairs cost the rest.
//
// The form, and why:
//   * a CTA holds an SM and NT query tiles (128 rows, a row a softmax thread), as
//     many as TMEM, registers and shared memory hold: 3 at hd 64, 2 at hd 128.
//     The tiles share the K and V that are loaded, and one's softmax runs while
//     another's products do.  Key tiles are 64 keys: a row's scores of a tile are
//     64 registers, and a window is covered with less beside it than by 128
//     (two images with sinks: 268 us by 128, 222 by 64);
//   * each query tile has a warp that issues its products, a further warp
//     schedules, loads and spreads biases.  S of the next key tile is issued once
//     the softmax has this one's in registers; P goes to TMEM, half at a time, and
//     the next scores are read behind it (read before P's stores are waited for,
//     the long document takes 87 us instead of 81);
//   * a CTA that is done takes over the place of one that has not started
//     (cluster launch control), so that the next item's loads and first products
//     run under the last one's softmax and stores.  Items with the most keys go
//     first (up to MAX_WORK blocks; beyond that a CTA finds its block by a search
//     in the device's offsets).  Smaller items at the end would even out the last
//     turn, and cost what they gain: fewer query tiles in a step take longer each;
//   * key tiles: those that hold one of the first `sinks` keys, then those of
//     the window of the item's queries; a query tile takes part only in those
//     that its own rows see;
//   * mask: a row's visible keys of a tile are two 32-bit words (a bit below
//     the last key and not below the first one, or below `sinks`), applied to
//     the scores in one pass; tiles that every row of a warp sees whole skip it;
//   * bias: a head's column of the table is spread over the distances, in shared
//     memory, scaled by log2 e: the CTA's first by all softmax warps while Q and K
//     are on their way (two texts: 4.6 us instead of 6.8 by one warp), later ones
//     by the loading warp, ahead.  A row's thread then adds the float at (key -
//     row), neighbouring rows neighbouring words (no bank conflicts), in an FMA
//     that scales the score: a pass of its own, some 800 clocks a step of three tiles.
//     Where every tile is near (4 x 1024 rows of 12 heads of 64, 320 buckets to 800)
//     the call takes 25.7 us instead of the 18.2 without a bias.  Beyond `reach`
//     all distances of a side share one bucket: there the bias is one number for the tile
//     and goes into the exponent's offset, at no cost a key (32 buckets to 128: 19.9 us
//     there; two images 412 instead of 387; packed texts 42.3 instead of 35);
//   * one copy of each role's code, rare cases short rather than fast, no branch in
//     the softmax's loop that saves work only sometimes: the instruction caches and
//     the loop's one long schedule bound it (5 to 15 %: leaving out the exponentials
//     of tiles that a warp sees nothing of made even calls without such tiles slower).
// A masked key has weight 0, but 0 x inf is not 0: the tensor core would spread
// a value that is not finite from a masked place.  So the rows of V behind a
// sequence's end (its neighbour's) are zeroed in shared memory, and an output
// row that comes out not finite all the same is settled on its own (mend_rows), which
// finite inputs of ordinary size never reach.
// Every mbarrier wait is bounded, as in attn.cu; the limit grows with the keys that a row
// sees, as what is waited for does.
//
// Measured (a call among others; those of heads of 128 vary by 3 % with the clock):
// packed texts (32, 19 .. 955 rows, 8 heads of 64) with a window of 512 and 4 sinks 33.6
// us, with a bias 42.2; 30001 rows, 12 heads of 64, window 256, 64 sinks 82 us (645
// TFLOP/s of the visible pairs); grouped causal heads (8191 rows, 32 over 8 of 128, window
// 1023) 128 us (1010); two images of 4224 rows, 30 heads of 128: window 1056 and 32 sinks
// 209 us (1160), bias 416 us (1320, 70 % of the measured bf16 rate).
#include <cuda.h>
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace tefwd {
namespace {

constexpr int BQ = 128;     // queries per tile (= TMEM lanes)
constexpr int BKV = 64;     // keys per tile
constexpr int MAX_WORK = 640;   // work list entries carried in the launch parameters
constexpr int MAX_SMEM = 227 * 1024;
// A wait's limit, ns: far above what any takes, which is the steps of an item's key
// tiles (0.8 us for 64 keys) and, where rows have to be computed again, the 32 rows of
// a warp (1.8 us a key).
constexpr unsigned long long WAIT_NS = 200000000, WAIT_KEY_NS = 16000;
constexpr int PAD = 96;     // distances past `reach` that 32 rows and 64 keys near it can still touch (94)
// as in attn.cu: K and V bytes that the CTA order treats as one group of heads
constexpr long long KV_ALL_BYTES = 48ll << 20;
constexpr long long KV_GROUP_BYTES = 24ll << 20;

__device__ int g_span_err;

struct SpanParams {
    CUtensorMap map;           // the bf16 q|k|v panel [T, ld], box 64 x 64
    __nv_bfloat16 *out;
    const __nv_bfloat16 *qkv;
    const int *cu;
    int nseq, total;
    int nwork;                 // > 0: work[i] = (sequence << 16) | query block, longest first
    int nq, hgroup;            // heads, and heads per group of the CTA order
    uint32_t work[MAX_WORK];
    int starts[MAX_WORK + 1];  // with a list: the sequences' offsets (the device's array is not read)
    long long ld, ldo;
    int q_off, k_off, v_off, group;
    int left, right, sinks;    // limits clipped to the longest sequence
    unsigned long long wait_ns;   // limit of a wait
    float scale_log2;
    // relative position bias
    const float *table;        // [buckets, ldt]
    long long ldt;
    int side, exact, reach, two_sided;   // buckets of a side, those of one distance each; clipped reach
    float grow;                // logarithmic buckets per unit of log2(distance / exact)
    uint16_t first[TE_RELPOS_MAX_BUCKETS];   // smallest distance of each bucket of a side
};

// Several query tiles a CTA, four softmax warps each, and four warps that feed them.
template <int HD, int RING = HD == 64 ? 7 : 3>
struct SLayout {
    static constexpr int NB = HD / 64;              // 64-column boxes per tile row
    static constexpr int NT = HD == 64 ? 3 : 2;     // query tiles
    // pairs of a K and a V tile in flight: as many as fit.  Where there is a window the
    // first query tile is done with an item's keys while the last still needs
    // some; the ring lets it go on to the next item.
    static constexpr int R = RING;
    static constexpr int QTILE = BQ * HD * 2, TILE = BKV * HD * 2;
    static constexpr int QBOX = BQ * 128, BOX = BKV * 128;   // 64 columns of them
    static constexpr int Q_OFF = 0;                 // Q[NT]
    static constexpr int K_OFF = NT * QTILE;        // [R] K, V
    static constexpr int STG_OFF = K_OFF + R * 2 * TILE;     // a softmax warp's 32 rows of 32 outputs
    static constexpr int STG_WARP = 32 * 64;
    // warps: softmax (4 a query tile), one a query tile that issues its MMAs, and in
    // the same warpgroup one that schedules, loads and spreads the biases
    static constexpr int SOFTMAX_WARPS = 4 * NT, MMA_WARP = SOFTMAX_WARPS, TMA_WARP = MMA_WARP + 3;
    static constexpr int NTHREADS = 32 * (SOFTMAX_WARPS + 4);
    // registers a thread at launch, and after the softmax warps took over what the others do not need
    static constexpr int LAUNCH_REGS = HD == 64 ? 128 : 168, SOFTMAX_REGS = HD == 64 ? 144 : 208, OTHER_REGS = HD == 64 ? 80 : 88;
    static_assert(NT * SOFTMAX_REGS + OTHER_REGS <= (NT + 1) * LAUNCH_REGS && LAUNCH_REGS * NTHREADS <= 65536, "register split");
    static constexpr int BAR_OFF = STG_OFF + SOFTMAX_WARPS * STG_WARP;
    // barriers
    static constexpr int BAR_Q = 0;                      // [NT] Q loaded
    static constexpr int BAR_QE = BAR_Q + NT;            // [NT] Q read by the item's last S
    static constexpr int BAR_KV = BAR_QE + NT;      // [R] K and V loaded
    static constexpr int BAR_KVE = BAR_KV + R;           // [R] K and V read by every query tile
    static constexpr int BAR_SF = BAR_KVE + R;           // [NT] S ready
    static constexpr int BAR_SFREE = BAR_SF + NT;        // [NT] S is in registers
    static constexpr int BAR_PF = BAR_SFREE + NT;        // [NT] P written
    static constexpr int BAR_PV = BAR_PF + NT;           // [NT] its PV done
    static constexpr int BAR_OFREE = BAR_PV + NT;        // [NT] O is in registers
    static constexpr int BAR_REC = BAR_OFREE + NT;       // [4] item record written
    static constexpr int BAR_RECE = BAR_REC + 4;         // [4] item record read
    static constexpr int BAR_CLC = BAR_RECE + 4;         // the next CTA's place taken over, or not
    static constexpr int BAR_BF = BAR_CLC + 1;           // [2] bias spread
    static constexpr int BAR_BE = BAR_BF + 2;            // [2] bias no longer read
    static constexpr int BAR_B0 = BAR_BE + 2;            // the first bias spread, by the softmax warps
    static constexpr int BAR_FIN = BAR_B0 + 1;           // [NT] every MMA and commit of an MMA warp is done
    static constexpr int NBAR = BAR_FIN + NT;
    static constexpr int REC_OFF = (BAR_OFF + 8 * NBAR + 15) / 16 * 16;   // 4 records of 16 bytes, the taken place
    static constexpr int SLOT_OFF = REC_OFF + 80;        // TMEM base
    static constexpr int TAB_OFF = SLOT_OFF + 16;        // a head's table column, then two spread biases
    // TMEM columns of a query tile: S (64 f32), P (64 bf16), O (HD f32)
    static constexpr int P_COL = 64, O_COL = 96, TILE_COLS = 96 + HD;
    static_assert(NT * TILE_COLS <= 512, "TMEM budget");
    // shared memory besides the bias: nb of the table's column and two of 2 (reach + PAD) + 1 distances
    static constexpr int bytes(int nb, int reach) { return TAB_OFF + 1024 + 4 * (nb + 2 * (2 * (reach + PAD) + 1)); }
    static_assert(RING > (HD == 64 ? 7 : 3) || bytes(TE_RELPOS_MAX_BUCKETS, TE_RELPOS_MAX_DISTANCE) <= MAX_SMEM, "shared memory per CTA");
};

// Key tiles that rows [r0, r1] of a sequence of `len` see: tiles [0, sink) and
// [first, end).
struct KeyTiles {
    int sink, first, end;
    __device__ __forceinline__ bool has(int t) const { return t < end && (t >= first || t < sink); }
    __device__ __forceinline__ int count() const { return sink + end - first; }
    // the j-th of them, and the place of a tile among them
    __device__ __forceinline__ int tile(int j) const { return j < sink ? j : j + first - sink; }
    __device__ __forceinline__ int place(int t) const { return t < sink ? t : t - first + sink; }
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

// The bucket of distance d, which counts as the reach where it is further.
__device__ __forceinline__ int bucket_of(const SpanParams &p, int d) {
    int a = p.two_sided ? (d < 0 ? -d : d) : (d < 0 ? -d : 0);
    if (a > p.reach) a = p.reach;
    int b = a;
    if (a >= p.exact) {
        // within one of the bucket by the f32 logarithm, then by the exact borders
        b = p.exact + (int)(__log2f((float)a / (float)p.exact) * p.grow);
        b = b < p.exact ? p.exact : (b > p.side - 1 ? p.side - 1 : b);
        if (b > p.exact && a < p.first[b]) --b;
        else if (b + 1 < p.side && a >= p.first[b + 1]) ++b;
    }
    return p.two_sided && d > 0 ? b + p.side : b;
}

// A bias in log2 units; a finite one stays finite (the type's lowest value still masks softly).
__device__ __forceinline__ float bias_log2(float v) {
    const float v2 = v * 1.4426950408889634f;
    return fabsf(v) <= FLT_MAX ? fminf(fmaxf(v2, -FLT_MAX), FLT_MAX) : v;
}

// A whole warp waits for a phase, for limit_ns at most (then false); the loop out of
// the way of the code around it.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    if (__builtin_expect(__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)), 1)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)))
        if (__all_sync(0xFFFFFFFFu, globaltimer_ns() - t0 > limit_ns)) return false;
    return true;
}

// Arrives where `on` is set, without a branch.
__device__ __forceinline__ void arrive_if(uint32_t bar, bool on) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"((uint32_t)on)
                 : "memory");
}

// Shared-memory descriptors of the 128-byte swizzle differ in their low words
// alone (address, leading offset); the high word is the same for both operand forms.
constexpr uint32_t DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;

// Four MMAs along K = 64 as one block, issued by the lane whose e is set: the
// predicates are made once and the descriptors by adds to their low words.  First S = Q K^T, then O += P V.
__device__ __forceinline__ void mma_s4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a, {x, %6};\n\tmov.b64 b, {y, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a, {x, %6};\n\tmov.b64 b, {y, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a, {x, %6};\n\tmov.b64 b, {y, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(e), "n"(DESC_HI)
        : "memory");
}
__device__ __forceinline__ void mma_pv4(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 b, {y, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, 1;\n\t"
        "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 b, {y, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, 1;\n\t"
        "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 b, {y, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, 1;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(e), "n"(DESC_HI)
        : "memory");
}

__device__ __forceinline__ void arrive_n(uint32_t bar, int n, uint32_t e) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(n), "r"(e)
                 : "memory");
}

// Scores of 32 keys to log2 units with their bias: v = v c + b[e].
__device__ __forceinline__ void add_bias(uint32_t (&v)[32], uint64_t c2, const float *b) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const uint64_t b2 = f2_pack(b[e], b[e + 1]);
        float x, y;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2, b2), x, y);
        v[e] = __float_as_uint(x);
        v[e + 1] = __float_as_uint(y);
    }
}

// Waits for this thread's TMEM loads; the registers go through it, so that no use
// of theirs can come before.
__device__ __forceinline__ void wait_loaded(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Scores of 32 keys whose bit of `see` is 0 become -inf.
__device__ __forceinline__ void hide(uint32_t (&v)[32], uint32_t see) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!(see >> e & 1)) v[e] = 0xFF800000u;
}

// P = 2^(s cs + nm) of 32 keys as bf16, and its sums into r2.
__device__ __forceinline__ void exp_pass(const uint32_t (&v)[32], uint64_t c2, uint64_t nm2, uint64_t (&r2)[2],
                                         uint32_t (&pk)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float a0, a1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, nm2), a0, a1);
        const float p0 = hw_exp2(a0), p1 = hw_exp2(a1);
        r2[e & 1] = f2_add(r2[e & 1], f2_pack(p0, p1));
        pk[e] = pack_bf16x2(p0, p1);
    }
}

// Is one of a lane's bf16 values infinite or NaN?
template <int N>
__device__ __forceinline__ bool odd(const uint32_t (&w)[N]) {
    bool r = false;
#pragma unroll
    for (int i = 0; i < N; ++i) r |= ((w[i] & 0x7F80u) == 0x7F80u) | ((w[i] & 0x7F800000u) == 0x7F800000u);
    return r;
}
template <int N>
__device__ __forceinline__ void load_words(const __nv_bfloat16 *from, uint32_t (&w)[N]) {
    if constexpr (N == 1)
        w[0] = *reinterpret_cast<const uint32_t *>(from);
    else {
        const uint2 u = *reinterpret_cast<const uint2 *>(from);
        w[0] = u.x;
        w[1] = u.y;
    }
}

// Eight bf16 as f32.
__device__ __forceinline__ void widen(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}

// Output rows that the tiled form cannot give, by the warp that has them (bits of
// `rows`, from row r0 on).  Where a row's sum is good (bits of `good`) its finite
// channels are, too: a channel is lost to a value of V that is not finite, either one
// that the row sees, and then it is that infinity (NaN: both or a NaN), or one in a
// masked place of a tile (0 x inf).  One pass over the values that the warp's rows
// see tells which; a lane has the same channels of all of them, and for each channel
// the rows that see +inf and -inf.  Rows that this does not explain, and those
// whose sum is not good, are computed again from their visible keys alone, four at
// once, 32 keys at a time.
// No finite input of ordinary size comes here.  2048 rows, 12 heads of 64 (45 us): an
// infinite value that every row sees 162 us, a key of NaN 280; 256 keys to either side
// (22 us) and a NaN beside the sinks, in a tile of every row, 920 (36, 18 and 9 ms by a
// key at a time; one row at once 2.0 ms).  Not inlined, and the lane read anew: what is
// worked out from it would be kept through the loop over key tiles, whose registers are
// full (30001 rows, 12 heads of 64: 82 us, inlined 88).
template <int HD, bool BIAS>
__device__ __noinline__ void mend_rows(const SpanParams &p, const float *bias, int off, int len, int h, int r0, uint32_t rows,
                                          uint32_t good) {
    constexpr int C = HD / 32, W = C / 2;                // channels of a lane, words of them
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    int lane;
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
    const int g = (h / p.group) * HD;
    const __nv_bfloat16 *panel = p.qkv + (long long)off * p.ld;
    __nv_bfloat16 *out = p.out + (long long)(off + r0) * p.ldo + h * HD + lane * C;
    auto bias_of = [&](int d) { return BIAS ? bias[d < -p.reach ? -p.reach : (d > p.reach ? p.reach : d)] : 0.f; };
    // the keys of rows qa to qb: the first ns, and lo up to hi
    int lo, hi, ns;
    auto keys_of = [&](int qa, int qb) {
        lo = qa > p.left ? qa - p.left : 0;
        hi = qb + p.right + 1 < len ? qb + p.right + 1 : len;
        ns = p.sinks < lo ? p.sinks : lo;
    };
    auto key_of = [&](int j) { return j < ns ? j : j - ns + lo; };
    auto sees = [&](int qi, int key) {
        return key <= qi + p.right && (key >= qi - p.left || key < p.sinks) && (!BIAS || bias_of(key - qi) != -INFINITY);
    };

    if (good) {
        uint32_t plus[C] = {}, minus[C] = {}, again = 0;
        keys_of(r0 + __ffs(good) - 1, r0 + 31 - __clz(good));
        const int n = ns + hi - lo;
        const __nv_bfloat16 *v = panel + p.v_off + g + lane * C;
        bool known = false;                              // no later value changes anything
#pragma unroll 1
        for (int j = 0; j < n && !known; j += 8) {
            uint32_t eight[8 * W];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t w[W];
                load_words<W>(v + key_of(j + i < n ? j + i : n - 1) * p.ld, w);
#pragma unroll
                for (int y = 0; y < W; ++y) eight[i * W + y] = w[y];
            }
            if (!__any_sync(ALL, odd<8 * W>(eight))) continue;
#pragma unroll 1
            for (int i = j; i < j + 8 && i < n; ++i) {
                const int key = key_of(i);
                uint32_t w[W], k[W];
                load_words<W>(v + key * p.ld, w);
                if (!__any_sync(ALL, odd<W>(w))) continue;
                const uint32_t who = __ballot_sync(ALL, sees(r0 + lane, key)) & good;
                // (a key that is not finite may have scores of -inf, and then no weight)
                load_words<W>(panel + key * p.ld + p.k_off + g + lane * C, k);
                if (__any_sync(ALL, odd<W>(k))) again |= who;
                known = true;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint32_t x = w[c / 2] >> 16 * (c & 1);
                    if ((x & 0x7F80u) == 0x7F80u) {
                        const bool nan = x & 0x7Fu, neg = x & 0x8000u;
                        if (nan || !neg) plus[c] |= who;
                        if (nan || neg) minus[c] |= who;
                    }
                    known = known && (plus[c] & minus[c]) == good;
                }
                known = __all_sync(ALL, known);
            }
        }
#pragma unroll 1
        for (uint32_t left = good; left; left &= left - 1) {
            const int x = __ffs(left) - 1;
            __nv_bfloat16 *o = out + (long long)x * p.ldo;
            uint32_t w[W];
            load_words<W>(o, w);
            bool lost = again >> x & 1;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int at = 16 * (c & 1);
                if ((w[c / 2] >> at & 0x7F80u) == 0x7F80u) {
                    const bool a = plus[c] >> x & 1, b = minus[c] >> x & 1;
                    w[c / 2] = (w[c / 2] & ~(0xFFFFu << at)) | (a && b ? 0x7FFFu : b ? 0xFF80u : 0x7F80u) << at;
                    lost = lost || !(a || b);
                }
            }
            if (__any_sync(ALL, lost)) continue;
#pragma unroll
            for (int i = 0; i < W; ++i) reinterpret_cast<uint32_t *>(o)[i] = w[i];
            rows &= ~(1u << x);
        }
    }

    // R rows at once: they share their keys' loads and hide one another's latency
    constexpr int R = 4, G = HD / 8;                     // G lanes have a key's channels together, eight each
    const int at = lane % G * 8;
    int hint = -1;                                       // a key whose score lost the rows before
#pragma unroll 1
    while (rows) {
        int qi[R];
        float q[R][8], m[R], l[R], o[R][C];
#pragma unroll
        for (int r = 0; r < R; ++r) {                    // (the last one again where there are fewer)
            qi[r] = rows ? r0 + __ffs(rows) - 1 : qi[r > 0 ? r - 1 : 0];
            rows &= rows - 1;
            widen(*reinterpret_cast<const uint4 *>(panel + qi[r] * p.ld + p.q_off + h * HD + at), q[r]);
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) o[r][c] = 0.f;
        }
        keys_of(qi[0], qi[R - 1]);
        const int n = ns + hi - lo;
        // weights are taken down by a power of two above n, so that no sum of n values passes
        // the largest of them (by no more: tiny values would be lost)
        const int down = 32 - __clz(n);
        uint32_t lost = 0;                               // a bit a row
#pragma unroll 1
        for (int j = hint >= 0 ? -32 : 0; j < n && lost != (1u << R) - 1; j += 32) {
            const int key = j < 0 ? hint : key_of(j + lane < n ? j + lane : n - 1);
            float s[R];
#pragma unroll 4
            for (int i = 0; i < G; ++i) {
                float k[8];
                widen(*reinterpret_cast<const uint4 *>(panel + __shfl_sync(ALL, key, lane / G * G + i) * p.ld + p.k_off + g + at), k);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float d = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) d = fmaf(q[r][e], k[e], d);
#pragma unroll
                    for (int y = 1; y < G; y <<= 1) d += __shfl_xor_sync(ALL, d, y);
                    if (lane % G == i) s[r] = d;
                }
            }
            uint32_t take[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                // (a key that is masked takes nothing, whatever the score)
                s[r] = j + lane < n && sees(qi[r], key) ? fmaf(s[r], p.scale_log2, bias_of(key - qi[r])) : -INFINITY;
                // a score that is NaN or +inf loses the row, whatever else it sees
                const uint32_t bad = __ballot_sync(ALL, isnan(s[r]) || s[r] == INFINITY);
                if (bad) {
                    hint = __shfl_sync(ALL, key, __ffs(bad) - 1);
                    lost |= 1u << r;
                }
                take[r] = j < 0 ? 0 : __ballot_sync(ALL, s[r] > -INFINITY);
            }
            if (j < 0) continue;
            float pr[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mn = s[r];
#pragma unroll
                for (int y = 16; y > 0; y >>= 1) mn = fmaxf(mn, __shfl_xor_sync(ALL, mn, y));
                mn = fmaxf(m[r], mn);
                const float ref = mn == -INFINITY ? 0.f : mn, alpha = hw_exp2(m[r] - ref);
                pr[r] = hw_exp2(s[r] - ref);
                m[r] = mn;
                l[r] = l[r] * alpha + pr[r];
                pr[r] *= __int_as_float((127 - down) << 23);
#pragma unroll
                for (int c = 0; c < C; ++c) o[r][c] *= alpha;
            }
#pragma unroll 8
            for (int e = 0; e < 32; ++e) {
                uint32_t w[W];
                load_words<W>(panel + __shfl_sync(ALL, key, e) * p.ld + p.v_off + g + lane * C, w);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float we = __shfl_sync(ALL, pr[r], e);
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (take[r] >> e & 1)
                            o[r][c] = fmaf(we, __uint_as_float(c & 1 ? w[c / 2] & 0xFFFF0000u : w[c / 2] << 16), o[r][c]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int y = 16; y > 0; y >>= 1) l[r] += __shfl_xor_sync(ALL, l[r], y);
#pragma unroll
            for (int c = 0; c < C; ++c)
                out[(long long)(qi[r] - r0) * p.ldo + c] =
                    __float2bfloat16_rn(lost >> r & 1 ? NAN : l[r] == 0.f ? 0.f : o[r][c] / l[r] * __int_as_float((127 + down) << 23));
        }
    }
}

// The work of CTA `b` of the grid: which rows of which sequence, and the head.
struct Item {
    int off, len, q0, h;    // len 0: nothing
};
template <int QB>
__device__ __forceinline__ Item item_of(const SpanParams &p, int b, int lane) {
    int seq, qblk, h;
    long long off, len;
    if (p.nwork) {
        // CTAs take the heads in groups of hgroup: within a group, work items in
        // list order (most keys first), the group's heads fastest
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
        off = p.starts[seq];
        len = p.starts[seq + 1] - off;
    } else {
        // many blocks: sequence s has the slots from cu[s] / QB + s on, at least
        // as many as it has query blocks
        const int slot = b / p.nq;
        h = b - slot * p.nq;
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
        off = p.cu[seq];
        len = p.cu[seq + 1] - off;
        qblk = slot - (int)(off / QB + seq);
    }
    // nothing to do, or a device table that is not the host's: an item without rows
    const long long q0 = (long long)qblk * QB;
    const bool live = off >= 0 && len >= 1 && off + len <= p.total && q0 >= 0 && q0 < len;
    return {(int)off, live ? (int)len : 0, (int)q0, h};
}

// Takes over the place of a CTA of this grid that has not started yet; the
// answer (16 bytes) lands at dst and completes 16 bytes on bar.
__device__ __forceinline__ void take_next(uint32_t dst, uint32_t bar, uint32_t e) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n\t}" ::"r"(dst),
        "r"(bar), "r"(e)
        : "memory");
}
// The block index taken over, or -1: none was left.
__device__ __forceinline__ int taken(uint32_t src) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "mov.u32 %1, 0;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(src)
        : "memory");
    return got ? (int)x : -1;
}

template <int HD, bool BIAS, int RING>
__global__ void __launch_bounds__(SLayout<HD, RING>::NTHREADS, 1) attn_span_kernel(const __grid_constant__ SpanParams p) {
    using L = SLayout<HD, RING>;
    constexpr int NT = L::NT, QB = NT * BQ, R = L::R;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    auto bar = [&](int i) { return sb + L::BAR_OFF + 8 * i; };
    volatile int4 *rec = reinterpret_cast<volatile int4 *>(smem + L::REC_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::SLOT_OFF);
    float *tab = reinterpret_cast<float *>(smem + L::TAB_OFF);
    const int nb = p.two_sided ? 2 * p.side : p.side, width = p.reach + PAD;
    // the distance 0 of spread bias i
    auto spread_of = [&](int i) { return tab + nb + width + i * (2 * width + 1); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == L::TMA_WARP && lane == 0) {
        tma_prefetch_desc(&p.map);
        for (int i = 0; i < 2 * NT; ++i) mbar_init(bar(L::BAR_Q + i), 1);
        for (int i = 0; i < R; ++i) {
            mbar_init(bar(L::BAR_KV + i), 1);
            mbar_init(bar(L::BAR_KVE + i), NT);
        }
        for (int i = 0; i < NT; ++i) {
            mbar_init(bar(L::BAR_SF + i), 1);
            mbar_init(bar(L::BAR_SFREE + i), 4);
            mbar_init(bar(L::BAR_PF + i), 4);
            mbar_init(bar(L::BAR_PV + i), 1);
            mbar_init(bar(L::BAR_OFREE + i), 4);
            mbar_init(bar(L::BAR_FIN + i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(L::BAR_REC + i), 1);
            mbar_init(bar(L::BAR_RECE + i), L::SOFTMAX_WARPS + NT);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::BAR_BF + i), 1);
            mbar_init(bar(L::BAR_BE + i), L::SOFTMAX_WARPS);
        }
        mbar_init(bar(L::BAR_CLC), 1);
        mbar_init(bar(L::BAR_B0), L::SOFTMAX_WARPS);
        fence_mbar_init();
    }
    if (warp == L::MMA_WARP) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // from here on global memory is touched, by the loading warp once it knows its first item
    if (warp != L::TMA_WARP) {
        prior_wait();
        next_go();
    }
    const uint32_t tbase = tmem_slot[0];
    bool ok = true;
    // waits of a whole warp; false: given up
    auto wait = [&](int b, uint32_t parity) { return wait_on(bar(b), parity & 1, p.wait_ns); };
    // looks without waiting; what the look costs (its latency) the work up to its use hides
    auto test = [&](int b, uint32_t parity) { return mbar_test(bar(b), parity & 1); };
    // the record of the CTA's item number it, read by a whole warp
    auto get_record = [&](int it) {
        const volatile int4 *q = rec + (it & 3);
        return Item{q->x, q->y, q->z, q->w};
    };
    auto let_record = [&](int it) {
        __syncwarp();
        arrive_if(bar(L::BAR_RECE + (it & 3)), lane == 0);
    };
    auto read_record = [&](int it, Item &r) {
        if (!wait(L::BAR_REC + (it & 3), it >> 2)) return false;
        r = get_record(it);
        let_record(it);
        return true;
    };
    // the key tiles of an item in the order they are taken, and those of its query tile w
    auto tiles_of = [&](const Item &r) {
        return key_tiles(p, r.q0, r.q0 + QB < r.len ? r.q0 + QB - 1 : r.len - 1, r.len);
    };
    auto tiles_of_w = [&](const Item &r, int w) {
        const int r0 = r.q0 + w * BQ;
        return r0 < r.len ? key_tiles(p, r0, r0 + BQ < r.len ? r0 + BQ - 1 : r.len - 1, r.len) : KeyTiles{0, 0, 0};
    };
    // place and phase in a ring of R
    struct Ring {
        int at;
        uint32_t phase;
        __device__ __forceinline__ void step(int k = 1) {
            for (at += k; at >= R; at -= R) phase ^= 1;
        }
    };

    if (warp >= L::SOFTMAX_WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::OTHER_REGS));
        if (warp == L::TMA_WARP) {
            // ------------------------------------- scheduling and TMA producer
            // (the whole warp in step, one elected lane issues)
            const uint32_t e = elect_one();
            int next = *reinterpret_cast<volatile int *>(&g_span_err) == 0 ? (int)blockIdx.x : -1;
            next = __shfl_sync(0xFFFFFFFFu, next, 0);
            Ring kv = {0, 0};
            int kvn = 0;                                 // pairs of K and V issued in all
            int head = -1, built = 1;                    // the head whose bias was spread last, biases spread
            int asked = 0;                               // places asked for
            uint32_t qn[NT];                             // Q loads of each query tile
#pragma unroll
            for (int w = 0; w < NT; ++w) qn[w] = 0;
            // asks for the place of a CTA that has not started; after answer(), which reads it
            auto ask = [&]() {
                // the answer before was read: order that before it is overwritten
                fence_async_smem();
                __syncwarp();
                mbar_arrive_expect_tx_e(bar(L::BAR_CLC), 16, e);
                take_next(sb + L::REC_OFF + 64, bar(L::BAR_CLC), e);
                ++asked;
            };
            auto answer = [&]() {
                if (!wait(L::BAR_CLC, asked - 1)) { ok = false; return -1; }
                const int b = taken(sb + L::REC_OFF + 64);
                __syncwarp();
                return b;
            };
            // The next item with rows, from block `next` on; publishes its record
            // (len 0: no more) as the CTA's item number it.
            auto publish = [&](int it, Item &r) {
                r = {0, 0, 0, 0};
                if (!p.nwork) prior_wait();              // the offsets come from global memory
                while (next >= 0 && ok) {
                    r = item_of<QB>(p, next, lane);
                    if (r.len > 0) break;
                    ask();
                    next = answer();
                }
                if (!ok || !wait(L::BAR_RECE + (it & 3), (it >> 2) ^ 1)) { ok = false; return; }
                if (lane == 0) {
                    volatile int4 *q = rec + (it & 3);
                    q->x = r.off;
                    q->y = r.len;
                    q->z = r.q0;
                    q->w = r.h;
                    mbar_arrive(bar(L::BAR_REC + (it & 3)));
                }
                __syncwarp();
            };
            // Spreads a head's bias over the distances, in log2 units, ahead of its first item.
            auto spread_bias = [&](int h, float column) {
                if (h == head) return;
                head = h;
                const int buf = built & 1;
                if (!wait(L::BAR_BE + buf, (built >> 1) ^ 1)) { ok = false; return; }
                for (int b = lane; b < nb; b += 32)
                    tab[b] = bias_log2(b < 32 ? column : p.table[(long long)b * p.ldt + h]);
                __syncwarp();
                float *spread = spread_of(buf);
#pragma unroll 4
                for (int d = lane - width; d <= width; d += 32) spread[d] = tab[bucket_of(p, d)];
                __syncwarp();
                arrive_if(bar(L::BAR_BF + buf), lane == 0);
                ++built;
            };
            // Item number it is r, the one behind it r2; before the first there is an empty one.
            // The next item is published once the ring is full or the item's loads are out, and its
            // head's bias spread behind the load that follows.
            Item r = {0, 0, 0, 0}, r2 = r;
            int to_spread = -1;
            float column = 0.f;                          // its first 32 buckets, loaded ahead
            for (int it = -1; ok && (it < 0 || r.len > 0); ++it, r = r2) {
                const int g = r.h / p.group;
                KeyTiles tiles = {0, 0, 0}, kw[NT];
                if (it >= 0) tiles = tiles_of(r);
#pragma unroll
                for (int w = 0; w < NT; ++w) kw[w] = it >= 0 ? tiles_of_w(r, w) : KeyTiles{0, 0, 0};
                const int n = it >= 0 ? tiles.count() : 0;
                int qw = 0;                              // the query tile whose Q comes next
                for (int j = 0; ok; ++j) {
                    if (j == (n < R ? n : R)) {
                        if (it >= 0) next = answer();
                        if (ok) publish(it + 1, r2);
                        if (it < 0) {
                            prior_wait();
                            next_go();
                        }
                        if (BIAS && it < 0) head = r2.h;     // the softmax warps spread the first themselves
                        if (BIAS && it >= 0 && r2.len > 0) {
                            to_spread = r2.h;
                            column = lane < nb ? p.table[(long long)lane * p.ldt + to_spread] : 0.f;
                        }
                    }
                    if (!ok || j >= n) break;
                    const int t = tiles.tile(j);
                    int idle = 0, first = -1;            // query tiles that do not see this key tile; qw's first
#pragma unroll
                    for (int w = 0; w < NT; ++w) {
                        idle += kw[w].has(t) ? 0 : 1;
                        if (w == qw && kw[w].end > 0) first = kw[w].tile(0);
                    }
                    // a query tile's Q comes with the first key tile that it sees (later tiles
                    // see nothing sooner)
                    while (ok && t == first) {
                        uint32_t used = 0;
#pragma unroll
                        for (int w = 0; w < NT; ++w)
                            if (w == qw) used = qn[w]++;
                        if (!(ok = wait(L::BAR_QE + qw, used ^ 1))) break;
                        const uint32_t to = sb + L::Q_OFF + qw * L::QTILE, b = bar(L::BAR_Q + qw);
                        mbar_arrive_expect_tx_e(b, L::QTILE, e);
#pragma unroll
                        for (int c = 0; c < 2 * L::NB; ++c)   // 64 columns, 64 rows a box
                            tma_load_2d_e(to + c * L::BOX, &p.map, b, p.q_off + r.h * HD + 64 * (c >> 1),
                                          r.off + r.q0 + qw * BQ + BKV * (c & 1), e);
                        ++qw;
                        first = -1;
#pragma unroll
                        for (int w = 0; w < NT; ++w)
                            if (w == qw && kw[w].end > 0) first = kw[w].tile(0);
                    }
                    if (!ok || !(ok = wait(L::BAR_KVE + kv.at, kv.phase ^ 1))) break;
                    const uint32_t to = sb + L::K_OFF + kv.at * 2 * L::TILE, b = bar(L::BAR_KV + kv.at);
                    const int row = r.off + t * BKV;
                    mbar_arrive_expect_tx_e(b, 2 * L::TILE, e);
#pragma unroll
                    for (int c = 0; c < L::NB; ++c)
                        tma_load_2d_e(to + c * L::BOX, &p.map, b, p.k_off + g * HD + 64 * c, row, e);
#pragma unroll
                    for (int c = 0; c < L::NB; ++c)
                        tma_load_2d_e(to + L::TILE + c * L::BOX, &p.map, b, p.v_off + g * HD + 64 * c, row, e);
                    // those that do not see it have no need to say that they read it
                    if (idle) arrive_n(bar(L::BAR_KVE + kv.at), idle, e);
                    kv.step();
                    ++kvn;
                    if (j == 0) ask();
                    if (BIAS && to_spread >= 0) {
                        spread_bias(to_spread, column);
                        to_spread = -1;
                    }
                }
            }
            if (!ok) {
                // no copy of ours may still be landing when the CTA exits
#pragma unroll
                for (int w = 0; w < NT; ++w)
                    if (qn[w]) mbar_wait(bar(L::BAR_Q + w), (qn[w] - 1) & 1, 20000000ull);
                for (int i = kvn - R < 0 ? 0 : kvn - R; i < kvn; ++i) mbar_wait(bar(L::BAR_KV + i % R), (i / R) & 1, 20000000ull);
                if (asked) mbar_wait(bar(L::BAR_CLC), (asked - 1) & 1, 20000000ull);
            }
        } else if (warp - L::MMA_WARP < NT) {
            // ------------------------------------- MMA issuer of query tile w
            // (the whole warp in step, one elected lane issues)
            const int w = warp - L::MMA_WARP;
            const uint32_t e = elect_one();
            constexpr uint32_t idesc_s = idesc_bf16_f32(BQ, BKV);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(BQ, HD) | (1u << 16);   // B MN-major
            const uint32_t kd = (uint32_t)smem_desc_sw128(sb + L::K_OFF);
            const uint32_t vd = (uint32_t)smem_desc_mn_sw128(sb + L::K_OFF + L::TILE, L::BOX);
            const uint32_t q0 = (uint32_t)smem_desc_sw128(sb + L::Q_OFF) + w * (L::QTILE >> 4);
            const uint32_t stm = tbase + w * L::TILE_COLS;
            uint32_t sc = 0, pc = 0;                     // S and PV issued
            uint32_t items = 0;                          // items with rows before this one
            Ring kv = {0, 0};                            // the pair of K and V whose S comes next
            // S = Q K^T of the next key tile that this query tile sees.  A look at a parity tells a
            // phase from the one before it alone, and a pair that this warp passed unseen may, in
            // principle, still be landing when its place comes round; so first its release is looked for,
            // as by the loading warp: someone read it, so it landed, and the next cannot be released
            // without this warp.  (The passed pair was issued: an item's Q, which was waited for, comes
            // behind what was passed before it, and within an item fewer than R pairs are
            // passed.  So the pair before it was released, and the look is not off by two phases.
            // This warp's own part of the release is under way: the PV that is still to come
            // is of one of the last R - 1 pairs.)
            static_assert((NT - 1) * (BQ / BKV) + 1 <= R, "a query tile skips more than the ring holds");
            auto step_s = [&]() -> bool {
                const bool released = test(L::BAR_KVE + kv.at, kv.phase ^ 1);
                const bool there = test(L::BAR_KV + kv.at, kv.phase);
                // the softmax has the last S in registers (before the first there is nothing to wait for)
                const bool s_free = test(L::BAR_SFREE + w, sc + 1);
                if (__builtin_expect(!__all_sync(0xFFFFFFFFu, released && there && s_free), 0) &&
                    !(wait(L::BAR_KVE + kv.at, kv.phase ^ 1) && wait(L::BAR_KV + kv.at, kv.phase) && wait(L::BAR_SFREE + w, sc + 1)))
                    return false;
                tc_fence_after();
                const uint32_t k0 = kd + kv.at * (2 * L::TILE >> 4);
#pragma unroll
                for (int c = 0; c < L::NB; ++c)
                    mma_s4(stm, q0 + c * (L::QBOX >> 4), k0 + c * (L::BOX >> 4), idesc_s, c > 0, e);
                mma_commit_e(bar(L::BAR_SF + w), e);
                ++sc;
                return true;
            };
            // O += P V of the pair in ring place `at` (its S was waited for, so it is there); more: not the item's first
            auto step_pv = [&](int at, bool more) -> bool {
                const bool p_there = test(L::BAR_PF + w, pc);
                // an item's first overwrites O, whose last rows have been read
                const bool o_free = more ? true : test(L::BAR_OFREE + w, items + 1);
                if (__builtin_expect(!__all_sync(0xFFFFFFFFu, p_there && o_free), 0) &&
                    !((more || wait(L::BAR_OFREE + w, items + 1)) && wait(L::BAR_PF + w, pc)))
                    return false;
                tc_fence_after();
                mma_pv4(stm + L::O_COL, stm + L::P_COL, vd + at * (2 * L::TILE >> 4), idesc_pv, more, e);
                mma_commit_e(bar(L::BAR_PV + w), e);
                mma_commit_e(bar(L::BAR_KVE + at), e);
                ++pc;
                return true;
            };
            for (int it = 0; ok; ++it) {
                Item r;
                if (!(ok = read_record(it, r)) || r.len == 0) break;
                const KeyTiles all = tiles_of(r), mine = tiles_of_w(r, w);
                const int n = all.count(), m = mine.count();
                if (m == 0) {                            // the item has no rows of this query tile
                    kv.step(n);
                    continue;
                }
                // S of a key tile, then PV of the one before it; PV first where the next key tile
                // is so far on that it waits for that one's place in the ring
                int at_list = 0, si = 0;                 // where kv stands among the item's key tiles, S issued
                int at_s = 0, at_pv = 0;                 // ring places of the last S and of the PV that comes next
                ok = wait(L::BAR_Q + w, items);
                for (int i = 0; i < m && ok;) {
                    bool s_next = si < m && si <= i + 1;
                    int next = 0;
                    if (s_next) {
                        next = all.place(mine.tile(si));
                        s_next = si == i || next - at_list < R;
                    }
                    if (s_next) {
                        kv.step(next - at_list);
                        at_list = next;
                        at_pv = si == i ? kv.at : at_s;
                        at_s = kv.at;
                        ok = step_s();
                        // every S of the item is issued: its Q may be overwritten behind them
                        if (++si == m) mma_commit_e(bar(L::BAR_QE + w), e);
                    } else {
                        ok = step_pv(at_pv, i > 0);
                        at_pv = at_s;
                        ++i;
                    }
                }
                kv.step(n - at_list);
                ++items;
            }
            // nothing of ours may still be running when TMEM is given back
            mma_commit_e(bar(L::BAR_FIN + w), e);
            mbar_wait(bar(L::BAR_FIN + w), 0, 20000000ull);
        }
    } else {
        // ---------------------------------------- softmax, one query per thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::SOFTMAX_REGS));
        const int w = warp >> 2;                         // query tile
        const int wq = warp & 3;                         // TMEM lane quadrant: rows 32 wq ..
        const uint32_t scol = tbase + ((uint32_t)(32 * wq) << 16) + w * L::TILE_COLS;
        const float c = p.scale_log2;
        // Partial maxima of a row; whether S is given back behind them or as soon as it is in
        // registers; whether the next tile is looked over behind P or beside the second half.  All
        // only order the same work.  Measured, us (packed texts, images with sinks, the wide
        // reach, images with bias, causal window with bias): as here 33.6 204 25.5 407 92.9; two maxima
        // 33.7 204 26.1 406 92.5; S given back the other way 34.1 206 25.0 409 94.3; looked
        // over the other way 34.6 208 25.9 407 93.0.
        constexpr int NM = 3;
        constexpr bool FREE_LATE = HD == 64 || !BIAS;
        constexpr bool LOOK_LATE = HD == 64 || BIAS;
        uint32_t done = 0;                               // key tiles of this query tile, of all items
        uint32_t vbase = 0;                              // key tiles of the CTA's items before this one
        int head = -1, built = 0;                        // as where they are spread
        const float *bias = nullptr;                     // bias[d]: distance d, -(reach + PAD) .. reach + PAD
        for (int it = 0; ok; ++it) {
            if (!(ok = wait(L::BAR_REC + (it & 3), it >> 2))) break;
            Item r = get_record(it);                     // held until the item's end
            if (r.len == 0) break;
            const int len = r.len;
            if constexpr (BIAS) {
                if (r.h != head) {
                    // let go of the last head's bias, take this one's
                    if (head >= 0 && lane == 0) mbar_arrive(bar(L::BAR_BE + ((built - 1) & 1)));
                    head = r.h;
                    bias = spread_of(built & 1);
                    if (built == 0) {
                        // the CTA's first: by all softmax warps at once, while Q and K are on their way
                        for (int d = (int)threadIdx.x - width; d <= width; d += 32 * L::SOFTMAX_WARPS)
                            spread_of(0)[d] = bias_log2(p.table[(long long)bucket_of(p, d) * p.ldt + head]);
                        __syncwarp();
                        arrive_if(bar(L::BAR_B0), lane == 0);
                        if (!(ok = wait(L::BAR_B0, 0))) break;
                    } else if (!(ok = wait(L::BAR_BF + (built & 1), (built - 1) >> 1))) {
                        break;
                    }
                    ++built;
                }
            }
            const uint32_t vlast = vbase + tiles_of(r).count() - 1;   // the V tile of the item's last key tile
            vbase = vlast + 1;
            const int r0 = r.q0 + w * BQ + 32 * wq;      // the warp's first row
            if (r.q0 + w * BQ >= len) {                  // the item has no rows of this query tile
                let_record(it);
                continue;
            }
            const int qi = r0 + lane;
            const KeyTiles mine = tiles_of_w(r, w);
            float m_used = -INFINITY, nm0 = 0.f;         // nm0 = -m_used, 0 while there is none
            uint64_t r2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};   // partial row sums
            // Tiles whose first key is in [whole_from, whole_to], or which end within
            // the sinks, are seen whole by every row of the warp.  Near tiles begin
            // in (near_from, near_to); the others have one bias for all pairs.
            const int whole_from = (r0 + 31 < len - 1 ? r0 + 31 : len - 1) - p.left;
            const int whole_to = (r0 + p.right + 1 < len ? r0 + p.right + 1 : len) - BKV;
            const int near_from = r0 - (BKV - 1) - p.reach, near_to = r0 + 31 + p.reach;
            float far_before = 0.f, far_behind = 0.f;
            if constexpr (BIAS) {
                far_before = bias[-p.reach];
                far_behind = bias[p.reach];
            }
            // what the tile that begins at key kv0 needs: a mask or a bias of each pair
            // (special), else one bias cb for all its pairs
            bool special;
            float cb = 0.f;
            auto look = [&](int kv0) {
                special = kv0 > whole_to || (kv0 < whole_from && kv0 + BKV > p.sinks);
                if constexpr (BIAS) {
                    cb = kv0 <= near_from ? far_before : far_behind;
                    // a bias so large that it takes the scores' own digits is added to each, as in a near tile
                    special = special || (kv0 > near_from && kv0 < near_to) || !(fabsf(cb) <= 8192.f);
                }
            };
            int t = mine.sink > 0 ? 0 : mine.first;
            look(t * BKV);
            bool begun = false, more = true;
            // the tensor core may compute the next S
            auto free_s = [&]() {
                tc_fence_before();
                __syncwarp();
                arrive_if(bar(L::BAR_SFREE + w), lane == 0);
            };
            // the S row of a tile in two halves of 32 keys
            uint32_t va[32], vb[32];
            if (!(ok = wait(L::BAR_SF + w, done))) break;
            tc_fence_after();
            tmem_ld32(scol, va);
            tmem_ld32(scol + 32, vb);
            while (more) {
                wait_loaded(va);
                wait_loaded(vb);
                if (!FREE_LATE) free_s();
                // scores in log2 units are s * cs + cb
                float cs = c;
                if (special) {
                    const int kv0 = t * BKV;
                    if constexpr (BIAS) {
                        const bool near = kv0 > near_from && kv0 < near_to;
                        if (near || !(fabsf(cb) <= 8192.f)) {
                            // (64 distances past the reach hold a side's far bias)
                            const float *b = bias + (near ? kv0 - qi : kv0 <= near_from ? -p.reach - (BKV - 1) : p.reach);
                            const uint64_t c2 = f2_pack(c, c);
                            add_bias(va, c2, b);
                            add_bias(vb, c2, b + 32);
                            cs = 1.f;
                            cb = 0.f;
                        }
                    }
                    if (kv0 > whole_to || (kv0 < whole_from && kv0 + BKV > p.sinks)) {
                        const int hi = (qi + p.right < len ? qi + p.right + 1 : len) - kv0;   // keys below it are not too far
                        const int lo = qi - p.left - kv0, sk = p.sinks - kv0;
                        hide(va, bits_below(hi) & (~bits_below(lo) | bits_below(sk)));
                        hide(vb, bits_below(hi - 32) & (~bits_below(lo - 32) | bits_below(sk - 32)));
                    }
                    if (kv0 + BKV > len) {
                        // the last tile: V's rows behind the sequence become zeros, each
                        // warp its share of them (a row is 128 bytes of each box)
                        const uint32_t slot = vlast % R;
                        if (!(ok = wait(L::BAR_KV + slot, vlast / R))) break;
#pragma unroll 1
                        for (int x = len - kv0 + 4 * wq + (lane >> 3); x < BKV; x += 16)
#pragma unroll
                            for (int cc = 0; cc < L::NB; ++cc)
                                *reinterpret_cast<uint4 *>(smem + L::K_OFF + (2 * slot + 1) * L::TILE + cc * L::BOX + x * 128 +
                                                           (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                    }
                }
                if (FREE_LATE) free_s();
                // P is free once its last PV is done (there is none before the first)
                const bool p_free = test(L::BAR_PV + w, done - 1);
                // pass 1: the row maximum, a few partial ones; and beside it P = 2^(s cs + cb - m)
                // of the first half by the reference so far, which nearly always stays
                float mp[NM];
#pragma unroll
                for (int i = 0; i < NM; ++i) mp[i] = fmaxf(__uint_as_float(va[i]), __uint_as_float(vb[i]));
#pragma unroll
                for (int i = NM; i < 32; ++i) mp[i % NM] = fmax3(mp[i % NM], __uint_as_float(va[i]), __uint_as_float(vb[i]));
                const float mx = fmaf(fmax3(mp[0], mp[1], mp[2]), cs, cb);
                // it moves when a row grew by more than 2^20 (P, sums and O have f32's exponents to spare;
                // moves cost a pass over O: by 2^8 grouped causal heads take 129 us instead of 125, the causal
                // window with bias 102 instead of 93)
                const bool resc = mx > m_used + 20.f;
                const uint64_t c2 = f2_pack(cs, cs);
                uint64_t nm2 = f2_pack(cb + nm0, cb + nm0);
                uint64_t rt[2] = {r2[0], r2[1]};
                uint32_t pk[16];
                exp_pass(va, c2, nm2, rt, pk);
                if (__builtin_expect(!__all_sync(0xFFFFFFFFu, !resc && p_free), 0)) {
                    if (__any_sync(0xFFFFFFFFu, resc)) {
                        const float alpha = resc ? hw_exp2(m_used - mx) : 1.f;
                        if (resc) {
                            m_used = mx;
                            nm0 = -mx;
                        }
                        rt[0] = f2_mul(r2[0], f2_pack(alpha, alpha));
                        rt[1] = f2_mul(r2[1], f2_pack(alpha, alpha));
                        nm2 = f2_pack(cb + nm0, cb + nm0);
                        exp_pass(va, c2, nm2, rt, pk);
                        if (begun) {
                            // O is whole once the PV before is done
                            if (!(ok = wait(L::BAR_PV + w, done - 1))) break;
                            tc_fence_after();
#pragma unroll
                            for (int cc = 0; cc < HD / 16; ++cc) {   // (few columns at once: S holds the registers)
                                uint32_t o[16];
                                tmem_ld16(scol + L::O_COL + 16 * cc, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(scol + L::O_COL + 16 * cc, o);
                            }
                        }
                    }
                    if (!(ok = wait(L::BAR_PV + w, done - 1))) break;
                }
                tc_fence_after();
                tmem_st16(scol + L::P_COL, pk);
                // the second half; what the next tile needs is worked out beside it
                const bool s_there = test(L::BAR_SF + w, done + 1);
                exp_pass(vb, c2, nm2, rt, pk);
                r2[0] = rt[0];
                r2[1] = rt[1];
                t = t + 1 == mine.sink ? mine.first : t + 1;
                more = t < mine.end;
                if (!LOOK_LATE) look(t * BKV);
                tmem_st16(scol + L::P_COL + 16, pk);
                begun = true;
                ++done;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                arrive_if(bar(L::BAR_PF + w), lane == 0);
                if (LOOK_LATE) look(t * BKV);
                // (the next S may come only behind this tile's PV: P is out before it is waited for)
                if (more) {
                    if (!__all_sync(0xFFFFFFFFu, s_there))
                        if (!(ok = wait(L::BAR_SF + w, done))) break;
                    tc_fence_after();
                    tmem_ld32(scol, va);
                    tmem_ld32(scol + 32, vb);
                }
            }
            if (!ok) break;
            // ---- epilogue: O / l, one row per thread (0 where nothing is visible)
            float s0, s1, s2, s3;
            f2_unpack(r2[0], s0, s1);
            f2_unpack(r2[1], s2, s3);
            const float l = (s0 + s1) + (s2 + s3);
            const float inv = hw_rcp(l);                 // (2^-23 of itself, then rounded to bf16)
            float fin[4] = {l, 0.f, 0.f, 0.f};           // their sum is NaN once a value of the row is not finite
            r = get_record(it);
            let_record(it);
            // rows go out through shared memory, so that a store of the warp writes 8
            // pieces of 64 bytes instead of 32 of 16
            uint4 *stage = reinterpret_cast<uint4 *>(smem + L::STG_OFF + warp * L::STG_WARP);
            const int orow = lane >> 2, ochunk = lane & 3;   // what this lane stores: rows orow + 8 i
            __nv_bfloat16 *out = p.out + (long long)(r.off + r0 + orow) * p.ldo + r.h * HD + 8 * ochunk;
            if (!(ok = wait(L::BAR_PV + w, done - 1))) break;
            tc_fence_after();
#pragma unroll
            for (int cc = 0; cc < HD / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(scol + L::O_COL + 32 * cc, o);
                tmem_wait_ld();
                if (cc == HD / 32 - 1) {
                    // O is in registers: the next item's first PV may overwrite it
                    tc_fence_before();
                    __syncwarp();
                    arrive_if(bar(L::BAR_OFREE + w), lane == 0);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) fin[e & 3] = fmaf(__uint_as_float(o[e]), 0.f, fin[e & 3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint4 u;
                    u.x = pack_bf16x2(__uint_as_float(o[8 * e + 0]) * inv, __uint_as_float(o[8 * e + 1]) * inv);
                    u.y = pack_bf16x2(__uint_as_float(o[8 * e + 2]) * inv, __uint_as_float(o[8 * e + 3]) * inv);
                    u.z = pack_bf16x2(__uint_as_float(o[8 * e + 4]) * inv, __uint_as_float(o[8 * e + 5]) * inv);
                    u.w = pack_bf16x2(__uint_as_float(o[8 * e + 6]) * inv, __uint_as_float(o[8 * e + 7]) * inv);
                    stage[4 * lane + (e ^ (lane >> 1 & 3))] = u;   // no bank twice in eight lanes
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = orow + 8 * i;
                    const uint4 u = stage[4 * x + (ochunk ^ (x >> 1 & 3))];
                    if (r0 + x < len) *reinterpret_cast<uint4 *>(out + (long long)(8 * i) * p.ldo + 32 * cc) = u;
                }
                __syncwarp();
            }
            // rows that hold a value that is not finite, or whose sum is out of range: it is 1
            // to 2^49 but for scores past 2^24, which f32 holds so coarsely that a row's
            // weights are all off by one power of two (hw_rcp ends at 2^126)
            const float finite = (fin[0] + fin[1]) + (fin[2] + fin[3]);
            uint32_t mend = __ballot_sync(0xFFFFFFFFu, qi < len && !(finite >= 0x1p-64f && finite <= 0x1p80f));
            if (mend) {
                // no key was visible: a score of any would have set the reference, a NaN the sum
                const bool none = qi < len && l == 0.f && nm0 == 0.f;
                mend &= ~__ballot_sync(0xFFFFFFFFu, none);
                if (none) {
                    uint4 *row = reinterpret_cast<uint4 *>(p.out + (long long)(r.off + qi) * p.ldo + r.h * HD);
#pragma unroll 1
                    for (int i = 0; i < HD / 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
                }
                const uint32_t good = __ballot_sync(0xFFFFFFFFu, l >= 0x1p-64f && l <= 0x1p80f);
                if (mend) mend_rows<HD, BIAS>(p, bias, r.off, len, r.h, r0, mend, mend & good);
            }
        }
    }
    if (!ok) atomicExch(&g_span_err, 1);
    tc_fence_before();
    __syncthreads();
    if (warp == L::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

template <int HD, bool BIAS, int RING>
te_status launch(const SpanParams &p, cudaStream_t stream) {
    using L = SLayout<HD, RING>;
    constexpr int most = BIAS ? MAX_SMEM : L::TAB_OFF + 1024;
    const int smem = BIAS ? L::bytes(p.two_sided ? 2 * p.side : p.side, p.reach) : most;
    static std::atomic<bool> ready[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cuda_fail(e, "attn: device");
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(attn_span_kernel<HD, BIAS, RING>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return cuda_fail(e, "attn: set shared memory size");
        ready[dev] = true;
    }
    const int64_t slots = p.nwork ? p.nwork : (int64_t)p.total / (L::NT * BQ) + p.nseq;
    if (slots * p.nq > 2147483647) return fail(TE_ESHAPE, "attn: too many query blocks and heads");
    e = launch_close(attn_span_kernel<HD, BIAS, RING>, dim3((unsigned)(slots * p.nq)), L::NTHREADS, smem, stream, 1, p);
    return e == cudaSuccess ? TE_OK : cuda_fail(e, "attn launch");
}

// The deeper ring wherever the bias leaves room for it: with 4 pairs of K and V instead
// of 3 (hd 128) two images take 417 us instead of 423, with sinks 206 instead of 212; at hd 64 9
// instead of 7 change nothing.
template <int HD>
te_status launch(const SpanParams &p, const te_relpos *plan, cudaStream_t stream) {
    constexpr int DEEP = HD == 64 ? 7 : 4, WIDE = HD == 64 ? 7 : 3;
    if (!plan) return launch<HD, false, DEEP>(p, stream);
    if (SLayout<HD, DEEP>::bytes(p.two_sided ? 2 * p.side : p.side, p.reach) <= MAX_SMEM)
        return launch<HD, true, DEEP>(p, stream);
    return launch<HD, true, WIDE>(p, stream);
}

// --------------------------------------------- buckets of relative positions

// Whole numbers below 2^2880, for the borders of the buckets: products and
// comparisons only.
struct Whole {
    uint32_t w[90];
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
    uint64_t key[MAX_WORK];   // (most - keys) << 20 | place in packed order: a stable order by keys
    uint32_t at[MAX_WORK];
    int k = 0;
    for (int32_t s = 0; s < nseq; ++s) {
        const int32_t len = cu[s + 1] - cu[s];
        for (int32_t b = 0; b * qb < len; ++b, ++k) {
            const int64_t r0 = (int64_t)b * qb, r1 = std::min<int64_t>(r0 + qb, len) - 1;
            const int64_t lo = std::max<int64_t>(0, r0 - p.left), hi = std::min<int64_t>(len, r1 + p.right + 1);
            const int64_t keys = hi - lo + std::min<int64_t>(p.sinks, lo);
            key[k] = (((1ull << 40) - (uint64_t)keys) << 20) | (uint64_t)k;
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
    int32_t total = 0, max_len = 0;
    te_status st = check_attn_span(name, qkv, ld, q_off, k_off, v_off, cu_host, cu_dev, nseq, nq, nkv, hd, left, right,
                                   sinks, scale, plan, table, ldt, out, ldo, &total, &max_len);
    if (st != TE_OK) return st;
    SpanParams p;
    memset(&p, 0, sizeof(p));
    st = make_map_2d(&p.map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, qkv, (uint64_t)ld, (uint64_t)total, (uint64_t)ld * 2,
                     64, BKV, CU_TENSOR_MAP_SWIZZLE_128B);
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
    // the keys that a row may see bound what a wait can take
    p.wait_ns = WAIT_NS + WAIT_KEY_NS * (unsigned long long)std::min<int64_t>(max_len, (int64_t)p.left + p.right + 1 + p.sinks);
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
    p.nwork = build_work(cu_host, nseq, p, (hd == 64 ? SLayout<64>::NT : SLayout<128>::NT) * BQ, p.work);
    if (p.nwork) memcpy(p.starts, cu_host, sizeof(int32_t) * (nseq + 1));   // (no more sequences than blocks)
    // heads per group: all when every head's K and V fit in KV_ALL_BYTES
    // together, else the kv heads whose K and V make about KV_GROUP_BYTES
    const int64_t kv_head = (int64_t)total * hd * 4;
    int64_t hg = nq;
    if (kv_head * nkv > KV_ALL_BYTES) hg = std::min<int64_t>(nq, std::max<int64_t>(1, KV_GROUP_BYTES / kv_head) * p.group);
    p.hgroup = (int)hg;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return hd == 64 ? launch<64>(p, plan, s) : launch<128>(p, plan, s);
}

}  // namespace

// Host validation of te_attn_sink_fwd and (plan != NULL) te_attn_relbias_fwd;
// writes the row count and the longest sequence.
te_status check_attn_span(const char *name, const void *qkv, int64_t ld, int32_t q_off, int32_t k_off, int32_t v_off,
                          const int32_t *cu_host, const int32_t *cu_dev, int32_t nseq, int32_t nq, int32_t nkv, int32_t hd,
                          int32_t left, int32_t right, int32_t sinks, float scale, const te_relpos *plan, const float *table,
                          int64_t ldt, const void *out, int64_t ldo, int32_t *total_rows, int32_t *longest) {
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
    *total_rows = total;
    *longest = max_len;
    return TE_OK;
}

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
