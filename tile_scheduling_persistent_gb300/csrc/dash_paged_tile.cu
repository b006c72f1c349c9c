// dash_paged_tile.cu -- attention over a paged cache for sequences with many
// rows (more than few_most): chunks of prompts, drafted tokens of wide groups.
//
// The rows of a key/value head's group are packed: row r of a sequence is
// token r / G, head r % G, so that one read of a key tile serves the whole
// group.  An item is 2 matrix tiles of 128 / G tokens each (A and B, M = 128),
// one key/value head and a range of 128-key tiles:
//   S = Q K_j^T     (tcgen05, bf16, fp32 in tensor memory)
//   P = 2^(scale log2e S - m), bf16 (e4m3 caches: times 2^7, fp16) into the
//                   columns of S; l += row sums
//   O += P V_j      (A = P from tensor memory)
// A persistent CTA takes items from a counter (which CTA runs an item does not
// touch its bits).  The two tiles take turns: while the softmax warps work on
// one, the tensor core runs the other's products
//   ... PV_A(j) S_A(j+1) | PV_B(j) S_B(j+1) | PV_A(j+1) ...
// and both use each K and V tile once staged, so 256 rows share its reads.
// S_A(j+1) follows PV_A(j) in the tensor core's order, so one S/P buffer per
// tile suffices, and a completed S(j+1) says that O holds the sum through j:
// rescaling O (when a row's maximum has grown by more than 2^8) needs no
// further wait.  An item with one tile of rows uses the two buffers in turn,
// S(j+1) being issued before PV(j).
//
// bf16 caches: a warpgroup each for A and B, one row per thread (items of one
// tile go to the two in turn, so that one's epilogue overlaps the other's
// loop); the first half of P's keys is multiplied while the second is worked
// out.  e4m3 caches: scaling the scores comes on top, so the two share every
// tile by columns (keys 0-63 and 64-127; a thread has one row of A and the
// same row of B), which reads the scales once for both.  At D = 64 each half of
// the keys has an O, a maximum and a sum of its own, joined in the epilogue; at
// D = 128 tensor memory has room for one O, and its price is a vote of the 256
// threads for each tile (does any row outgrow its maximum?); the maxima
// themselves are exchanged only when one does.  (The votes cost 5% where they
// can be left out: 272 against 259 us for 2048 tokens over 8192 at D = 64.)
// Measured against a warpgroup for each row tile as for bf16 (the second 64
// scores read twice, for want of registers), Hq = 32, Hkv = 8, both with votes:
// 16 x 5 tokens over about 5000 keys 147 us against 165 (D = 128), 512 tokens
// over 8192 172 against 176, 2048 over 8192 370 against 360, and with D = 64 280
// against 282.
//
// Measured (Hq = 32, Hkv = 8): 4096 new tokens over 16384 keys, bf16, D = 128:
// 640 us, 1500 TFLOP/s (63% of the tensor core's cycles; what is left is the
// softmax between the products); 2048 over 8192: 190 us bf16, 363 to 376 us e4m3
// (votes, scaling, conversion: no unit is full); 16 x 5 tokens over to 5000 keys,
// bf16: 55 us, 3.2 TB/s (rounds of uneven items and their starts).  2048 over 8192, D = 64, e4m3: 259 us, 2000
// cycles for each matrix tile, of which the tensor core takes 512: 840 for the
// exponentials, 550 to read and scale the scores, 200 to 400 waiting for them.
//
// Warps: 0 producer (TMA: Q, and K / V pages of bf16 and E2M1 caches), 1 MMA issuer and
// tensor memory, 2 item scheduler, 3 idle, 4-7 and 8-11 softmax and epilogue,
// and for e4m3 and E2M1 caches 12-15 converters.
//
// e4m3 caches.  The converters read codes from the pages one tile ahead and
// store them, as TMA would a bf16 cache's tile, in fp16; the products then run
// in fp16.  K holds the codes themselves (exact), and the softmax multiplies
// the scores by the keys' scales in fp32: scores, maxima and sums lose nothing.
// V holds code * scale, rounded once to fp16 (2^-11, against 2^-8 of the
// output's bf16): a second scale for each column would cost the softmax as
// much again as its exponentials, since its reads of shared memory wait behind
// the tensor core's (K's are read once for A and B, while S is being formed).
// fp16's range is met with powers of two, undone in fp32: V by the largest scale so far in the item in [2^6, 2^7) (codes reach 448; when
// it grows, O is rescaled as for a grown maximum), Q by row, its largest value
// in [2^14, 2^15), converted in place.
//
// E2M1 caches.  The producer stages codes and scales as they lie in the pages (a
// ring of three K or V tiles, one bulk copy for each page's share), and the
// converters turn them into fp16 tiles of code * scale, exact, from shared memory:
// held in registers between the loads and the proxy fence, which waits for every
// access, the codes cost a trip to memory for each tile (2048 tokens over 8192:
// 635 us; 212 us so, 190 us for a bf16 cache).  Nothing is left to be scaled, so the
// softmax is the bf16 caches', a warpgroup for each row tile, with fp16 weights and
// queries as for e4m3; the cache's exponents join the scores' and the output's
// scale.  With half of the exponentials left out it is no faster either: the
// chain from a tile's scores to its weights bounds it as it does with bf16 caches.
//
// Tensor memory: S/P buffers at columns 0 and 128; O of A at 256, of B at 384 (e4m3 at
// D = 64: the second half of the keys 64 columns on).
#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

#include "dash_bwd.cuh"
#include "dash_internal.h"
#include "dash_paged.cuh"

namespace dash {

namespace {

constexpr int kKvStages = 4;   // K0 V0 K1 V1 ...
constexpr int kItemSlots = 2;

enum TileBar : int {
    T_Q_FULL = 0,                          // slots A, B
    T_Q_EMPTY = T_Q_FULL + 2,
    T_Q_READY = T_Q_EMPTY + 2,             // e4m3: a slot's queries are converted (T_Q_EMPTY keeps its uses apart)
    T_KV_FULL = T_Q_READY + 2,
    T_KV_EMPTY = T_KV_FULL + kKvStages,
    // [row tile or slot][buffer]: whoever waits for one of these sees every phase of it (parity cannot tell a phase from the
    // one after the next, and a warpgroup does not follow the items of the other)
    T_S_FULL = T_KV_EMPTY + kKvStages,
    T_P_READY = T_S_FULL + 4,              // [buffer][half of the keys]
    T_O_FULL = T_P_READY + 4,              // A, B
    T_PV_DONE = T_O_FULL + 2,              // items of one tile: every product with V
    T_ITEM_FULL,
    T_ITEM_EMPTY = T_ITEM_FULL + kItemSlots,
    T_PATCH = T_ITEM_EMPTY + kItemSlots,
    T_SCALES,                              // e4m3: the keys' scales of key tile t, slot t % 4
    T_RAW_FULL = T_SCALES + 4,             // E2M1: codes and scales of a K or V tile
    T_RAW_EMPTY = T_RAW_FULL + 3,
    T_COUNT = T_RAW_EMPTY + 3
};

// One item as its roles see it; the scheduler counts the uses of every barrier before it, so that no role has to
// follow items in which it has no part.
struct TileItem {
    int b;              // sequence, -1: no more items
    int hk, tok;        // key/value head; first token (row of q)
    int ntok;           // its tokens (tile A holds the first 128 / G)
    int pos;            // position of the first
    int lo, hi;         // keys that any row of the sequence sees
    int len;
    int t0, nk;         // key tiles t0 .. t0 + nk - 1
    int split;          // 1: the sequence's keys are split
    int tiles;          // 1 or 2
    int buf, slot;      // items of one tile: first S/P buffer; Q slot, O and (bf16) softmax warpgroup
    int kv, kt, qi;     // K and V stages, key tiles, items with keys before it
    int s_use[2], p_use[2], q_use[2], o_use[2], pv;   // [buffer] for S and P, [slot] for Q and O
    long long part;     // partial row of the item's first row
};

template <int D, int kType>
struct TileCfg {
    static constexpr bool kE4M3 = kType == DASH_CACHE_E4M3, kE2M1 = kType == DASH_CACHE_E2M1;
    static constexpr bool kConv = kType != DASH_CACHE_BF16;   // converters, and products in fp16
    static constexpr int kTile = D * 128 * 2;
    static constexpr int kNBox = D / 64;
    static constexpr bool kOwn = kE4M3 && D == 64;   // an O for each half of a tile's keys (tensor memory has room for four)
    static constexpr int OFF_Q = 0;                                  // A, B
    static constexpr int OFF_KV = 2 * kTile;
    static constexpr int OFF_MAX = OFF_KV + kKvStages * kTile;       // [A, B][column half][128 rows] fp32
    static constexpr int OFF_SUM = OFF_MAX + 4 * 128 * 4;            // the same
    static constexpr int OFF_QFAC = OFF_SUM + 4 * 128 * 4;           // converted: [2 items][A, B][128] fp32, 2^-a of each row
    static constexpr int OFF_KSC = OFF_QFAC + (kConv ? 2 * 2 * 128 * 4 : 0);    // [4 tiles][128] fp32, the keys' scales
    static constexpr int OFF_VFAC = OFF_KSC + (kE4M3 ? 4 * 128 * 4 : 0);        // [4 tiles] the factor of V
    static constexpr int OFF_RAW = OFF_VFAC + (kE4M3 ? 16 : 0);      // E2M1: [kRawStages] of codes [128][D / 2] and scales [128][D / 16]
    static constexpr int kRawStages = 3, kRawCodes = 128 * cell_bytes(kType, D), kRawStage = kRawCodes + 128 * scale_bytes(kType, D);
    static constexpr int OFF_ITEM = OFF_RAW + (kE2M1 ? kRawStages * kRawStage : 0);
    static constexpr int kItemBytes = 128;
    static constexpr int OFF_BAR = OFF_ITEM + kItemSlots * kItemBytes;
    static constexpr int OFF_CTL = OFF_BAR + T_COUNT * 8;            // tensor memory address, abort flag
    // at least ~117 KB, so that one CTA (and its 512 tensor memory columns) holds an SM
    static constexpr int kSmem = OFF_CTL + 16 > 120000 ? OFF_CTL + 16 : 120000;
    static constexpr int kThreads = kConv ? 512 : 384;
    // registers of the kinds of warpgroups (setmaxnreg), within what the launch grants
    static constexpr int kRegsLaunch = kConv ? 128 : 168, kRegsCtl = kE2M1 ? 48 : kE4M3 ? 56 : 72, kRegsConv = kE2M1 ? 64 : 120;
    static constexpr int kRegsSoftmax = kE2M1 ? 200 : kE4M3 ? 168 : 216;
    static_assert(128 * kRegsCtl + 256 * kRegsSoftmax + (kConv ? 128 * kRegsConv : 0) <= kThreads * kRegsLaunch, "register split");
    // dec must not raise and inc must not lower what the launch granted
    static_assert(kRegsCtl <= kRegsLaunch && (!kConv || kRegsConv <= kRegsLaunch) && kRegsSoftmax >= kRegsLaunch, "register split");
    static_assert(sizeof(TileItem) <= kItemBytes && kSmem <= 232448, "shared memory budget");
};

// One of two counts (an index that is not known when compiling would put the item into local memory).
__device__ __forceinline__ int pick(const int (&a)[2], int i) { return i ? a[1] : a[0]; }

struct TileWait {
    volatile int* abort;
    unsigned long long limit;
};

// Waits for a phase, at most the timeout; once a wait has run out (reported) no role waits any more and all reach their
// end: false.
// (Inlined: a call would take its caller's registers through the ABI's limits and spill the softmax.)
__device__ __forceinline__ bool tile_wait_slow(uint32_t bar, uint32_t parity, const TileWait& w) {
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*w.abort) return false;
        if (ptx::globaltimer() - t0 > w.limit) {
            serve_error(DASH_ERR_TIMEOUT, kOpAttn, blockIdx.x, 1, 0);
            *w.abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, const TileWait& w) {
    return ptx::mbar_try_wait(bar, parity) || tile_wait_slow(bar, parity, w);
}
// Every lane of a warp: all go on, or none.
__device__ __forceinline__ bool tile_wait_warp(uint32_t bar, uint32_t parity, const TileWait& w) {
    return __all_sync(0xffffffffu, tile_wait(bar, parity, w));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}
// Two codes as fp16 (exact).
__device__ __forceinline__ uint32_t half_codes(uint32_t codes, int upper) {
    uint32_t c;
    const uint16_t two = (uint16_t)(upper ? codes >> 16 : codes);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(c) : "h"(two));
    return c;
}
// Two values times a scale given as two fp16 parts (hi + lo, each twice): one rounding to fp16.
__device__ __forceinline__ uint32_t scaled_codes(uint32_t c, uint32_t hi, uint32_t lo) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tmul.rn.f16x2 t, %1, %3;\n\tfma.rn.f16x2 %0, %1, %2, t;\n\t}" : "=r"(r) : "r"(c), "r"(hi), "r"(lo));
    return r;
}
// 2^(k - e) and 2^(e - k) for x in [2^e, 2^(e+1)), k <= 14; both normal (a smaller x counts as 2^-112).
__device__ __forceinline__ void power_to(float x, int k, float& up, float& down) {
    const int e = min(max((int)(__float_as_uint(x) >> 23 & 255u) - 127, -112), 127);
    up = __uint_as_float((uint32_t)(127 + k - e) << 23);
    down = __uint_as_float((uint32_t)(127 - k + e) << 23);
}

// ---------------------------------------------------------------- products
// A product's 16 instructions have to leave in fewer cycles than the tensor core takes for them (64 each), from one warp.
// So the whole warp runs the issuer's code -- uniform control flow, values in uniform registers -- with the elected
// thread as a predicate of the instruction alone, and a shared-memory descriptor is one 32-bit addition: the upper half
// is constant (8-row groups 1024 bytes apart, version 1, 128-byte swizzle), the lower holds the address over 16 and, from
// bit 16, the distance between 64-column boxes over 16.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescK = 1u << 16;                       // K-major: no second distance
constexpr uint32_t kDescMn = ((uint32_t)kBox >> 4) << 16;   // MN-major

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
__device__ __forceinline__ void mma_ss_if(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(leader), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t leader, uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "r"(leader), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t leader, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
// S[128 x 128] = Q[128 x D] K[128 x D]^T, both K-major (lower descriptor halves)
// (kHalf: fp16 operands)
constexpr uint32_t kBf16Bits = (1u << 7) | (1u << 10);
template <int D, bool kHalf>
__device__ __forceinline__ void product_s(uint32_t leader, uint32_t d_tmem, uint32_t q_lo, uint32_t k_lo) {
    constexpr uint32_t idesc = ptx::idesc_bf16(128, 128, 0, 0) & ~(kHalf ? kBf16Bits : 0u);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (uint32_t)((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
        mma_ss_if(leader, d_tmem, q_lo + off, k_lo + off, idesc, kk > 0);
    }
}
// O[128 x D] (+)= P[128 x 64] (tensor memory, keys 64h ..) * V rows 64h .. (MN-major)
template <int D, bool kHalf>
__device__ __forceinline__ void product_pv(uint32_t leader, uint32_t d_tmem, uint32_t p_tmem, uint32_t v_lo, int h, uint32_t acc) {
    constexpr uint32_t idesc = ptx::idesc_bf16(128, D, 0, 1) & ~(kHalf ? kBf16Bits : 0u);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        mma_ts_if(leader, d_tmem, p_tmem + h * 64 + kk * 8, v_lo + (uint32_t)((4 * h + kk) * 2048 >> 4), idesc, kk > 0 ? 1u : acc);
}
// A vote of the 256 softmax threads; also their barrier.
__device__ __forceinline__ bool any_of_256(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

template <int D, int kType>
__global__ void __launch_bounds__(TileCfg<D, kType>::kThreads, 1) paged_tile_kernel(const __grid_constant__ PagedParams p) {
    using C = TileCfg<D, kType>;
    constexpr bool kE4M3 = C::kE4M3, kE2M1 = C::kE2M1, kConv = C::kConv;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile uint32_t* const tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_CTL);
    volatile int* const abort = reinterpret_cast<volatile int*>(smem + C::OFF_CTL + 4);
    auto BAR = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * (uint32_t)i; };
    const TileWait tw{abort, p.timeout_ns};
    const int tpt = 128 / p.G;   // tokens of a matrix tile
    const int trows = tpt * p.G;

    if (threadIdx.x == 0) {
        *abort = 0;
        for (int i = 0; i < T_COUNT; ++i) {
            int count = 1;
            if (kConv && ((i >= T_Q_READY && i < T_Q_READY + 2) || (i >= T_SCALES && i < T_RAW_FULL) || i >= T_RAW_EMPTY || (i >= T_KV_FULL && i < T_KV_FULL + kKvStages))) count = 4;   // converter warps
            if (i >= T_P_READY && i < T_P_READY + 4) count = 4;                                                         // a softmax warpgroup
            if (i >= T_ITEM_EMPTY && i < T_ITEM_EMPTY + kItemSlots) count = 10 + (kConv ? 4 : 0);
            ptx::mbar_init(BAR(i), count);
        }
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32((const void*)tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    wait_dependency();
    launch_dependents();

    // The items one after another: slot, its phase, and its release.
    int iu = 0;   // items taken
    auto next_item = [&](TileItem& it) -> bool {   // whole warps
        const int s = iu % kItemSlots;
        if (!tile_wait_warp(BAR(T_ITEM_FULL + s), (uint32_t)((iu / kItemSlots) & 1), tw)) return false;
        it = *reinterpret_cast<const TileItem*>(smem + C::OFF_ITEM + C::kItemBytes * s);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(BAR(T_ITEM_EMPTY + s));
        ++iu;
        return it.b >= 0;
    };
    auto parity = [](int uses) -> uint32_t { return (uint32_t)uses & 1u; };   // phase that the wait for use `uses` completes

    // Each warpgroup first re-sizes its registers, then runs its role.
    if (warp < 4) {
    ptx::setmaxnreg_dec<C::kRegsCtl>();
    if (warp == 0) {
        // ================================================== producer
        TileItem it;
        int patches = 0;
        bool ok = true;
        if (lane == 0) {
            ptx::prefetch_tensormap(&p.tm_q);
            if (!kE2M1 || p.gather) {   // (else there are none)
                ptx::prefetch_tensormap(&p.tm_k);
                ptx::prefetch_tensormap(&p.tm_v);
            }
        }
        const int page = p.c.page_size, rows = page < 128 ? page : 128, subs = 128 / rows;
        while (ok && next_item(it)) {
            if (it.nk <= 0) continue;
#pragma unroll 1
            for (int x = 0; ok && x < it.tiles; ++x) {
                const int slot = it.tiles == 2 ? x : it.slot;
                const int before = pick(it.q_use, slot);
                if (before > 0) ok = tile_wait_warp(BAR(T_Q_EMPTY + slot), parity(before - 1), tw);
                if (!ok) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(BAR(T_Q_FULL + slot), C::kNBox * trows * 128);
                    for (int bx = 0; bx < C::kNBox; ++bx)
                        tma_load_4d(sbase + C::OFF_Q + slot * C::kTile + bx * kBox, &p.tm_q, 64 * bx, 0, it.hk, it.tok + x * tpt,
                                    BAR(T_Q_FULL + slot));
                }
            }
            if (kE4M3) continue;
            if constexpr (kE2M1) {
                // codes and scales as they lie in the pages, K and V of a tile in turn: a lane for each page's share of either
                const int sub = lane >> 1, kind = lane & 1;
                const uint32_t size = (uint32_t)rows * (kind ? D / 16 : D / 2);
                const int t1 = it.t0 + it.nk;
                const int e0 = max(it.t0 * 128, it.lo) >> p.page_shift, e1 = (min(t1 * 128, it.hi) - 1) >> p.page_shift;
                int eb = (it.t0 * 128) >> p.page_shift, kv = it.kv;
                auto fetch = [&](int e) { return (e >= e0 && e <= e1) ? checked_page(p, it.b, e) : 0; };
                int pages = fetch(eb + lane), next = fetch(eb + 32 + lane);
                for (int t = it.t0; ok && t < t1; ++t) {
                    const int key = t * 128;
                    if ((key >> p.page_shift) - eb >= 32) {
                        eb += 32;
                        pages = next;
                        next = fetch(eb + 32 + lane);
                    }
                    const int k0 = key + sub * rows;
                    const bool need = sub < subs && k0 + rows > it.lo && k0 < it.hi;
                    const int pg = __shfl_sync(0xffffffffu, pages, ((k0 >> p.page_shift) - eb) & 31);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, need && kind == 0)) * (uint32_t)rows * (D / 2 + D / 16);
                    const long long cell = ((long long)pg * p.c.Hkv + it.hk) * page + (k0 & (page - 1));
                    int row[4];
                    if (p.gather) gather_rows(p, pages, eb, key + 64 * (sub & 1), it.hk, row);
#pragma unroll 1
                    for (int val = 0; val < 2; ++val, ++kv) {
                        const int st = kv % C::kRawStages;
                        if (kv >= C::kRawStages && !tile_wait_warp(BAR(T_RAW_EMPTY + st), parity(kv / C::kRawStages - 1), tw)) {
                            ok = false;
                            break;
                        }
                        const uint32_t dst = sbase + C::OFF_RAW + st * C::kRawStage;
                        if (lane == 0) ptx::mbar_arrive_expect_tx(BAR(T_RAW_FULL + st), p.gather ? (uint32_t)C::kRawStage : bytes);
                        __syncwarp();
                        if (p.gather) {   // (pages that no row sees are read as page 0)
                            if (sub < 2)
                                gather4(dst + (kind ? C::kRawCodes : 0) + 64 * sub * (kind ? D / 16 : D / 2),
                                        kind ? (val ? &p.tm_vs : &p.tm_ks) : (val ? &p.tm_v : &p.tm_k), row, BAR(T_RAW_FULL + st));
                            continue;
                        }
                        if (need) {
                            const void* from = kind ? (val ? p.c.v_scale : p.c.k_scale) : (val ? p.c.v : p.c.k);
                            bulk_load(dst + (kind ? C::kRawCodes : 0) + sub * size, (const uint8_t*)from + cell * (kind ? D / 16 : D / 2), size,
                                      BAR(T_RAW_FULL + st));
                        }
                    }
                }
                continue;
            }
            const int sub = lane / C::kNBox, box = lane % C::kNBox;
            const int t1 = it.t0 + it.nk;
            const int e0 = max(it.t0 * 128, it.lo) >> p.page_shift, e1 = (min(t1 * 128, it.hi) - 1) >> p.page_shift;
            int eb = (it.t0 * 128) >> p.page_shift, kv = it.kv;
            auto fetch = [&](int e) { return (e >= e0 && e <= e1) ? checked_page(p, it.b, e) : 0; };
            int pages = fetch(eb + lane), next = fetch(eb + 32 + lane);
            for (int t = it.t0; ok && t < t1; ++t) {
                const int key = t * 128;
                if ((key >> p.page_shift) - eb >= 32) {
                    eb += 32;
                    pages = next;
                    next = fetch(eb + 32 + lane);
                }
                const int k0 = key + sub * rows;
                const bool need = sub < subs && k0 + rows > it.lo && k0 < it.hi;
                const int pg = __shfl_sync(0xffffffffu, pages, ((k0 >> p.page_shift) - eb) & 31);
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, need)) * (uint32_t)rows * 128;
                const bool patch = key < it.lo || key + 128 > it.hi;
#pragma unroll 1
                for (int val = 0; val < 2; ++val, ++kv) {
                    const int st = kv % kKvStages;
                    if (kv >= kKvStages && !tile_wait_warp(BAR(T_KV_EMPTY + st), (uint32_t)((kv / kKvStages - 1) & 1), tw)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + C::OFF_KV + st * C::kTile;
                    // value rows that no row of the sequence sees (unwritten, freed) meet a zero weight: they must be
                    // zero, so such a tile lands on the producer's own barrier first
                    const bool own = patch && val;
                    const uint32_t bar = own ? BAR(T_PATCH) : BAR(T_KV_FULL + st);
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    if (need)
                        ptx::tma_load_3d(dst + box * kBox + sub * rows * 128, val ? &p.tm_v : &p.tm_k, 64 * box, k0 & (page - 1),
                                         pg * p.c.Hkv + it.hk, bar);
                    if (own) {
                        if (!tile_wait_warp(BAR(T_PATCH), (uint32_t)(patches & 1), tw)) {
                            ok = false;
                            break;
                        }
                        ++patches;
#pragma unroll 1
                        for (int i = lane; i < 128 * C::kNBox * 8; i += 32) {
                            const int r = (i >> 3) & 127;
                            if (key + r < it.lo || key + r >= it.hi) sts128(dst + (i >> 10) * kBox + (i & 1023) * 16, make_uint4(0, 0, 0, 0));
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(BAR(T_KV_FULL + st));
                    }
                }
            }
        }
        // a wait ran out: let the copies in flight land (bounded) before the CTA can end
        if (*abort) {
            const uint64_t t0 = ptx::globaltimer();
            while (ptx::globaltimer() - t0 < 1000000ull) {
            }
        }
    } else if (warp == 1) {
        // ================================================== MMA issuer
        TileItem it;
        const uint32_t leader = elect_one();
        const uint32_t lo0 = sbase >> 4;
        bool ok = true;
        while (ok && next_item(it)) {
            // through a shuffle: the compiler then knows them to be the same in every lane
            auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
            const int nk = uni(it.nk), tiles = uni(it.tiles), slot = uni(it.slot), kv0 = uni(it.kv);
            const int p_use[2] = {uni(it.p_use[0]), uni(it.p_use[1])};
            if (nk <= 0) continue;
            auto full = [&](int u) { return tile_wait_warp(BAR(T_KV_FULL + u % kKvStages), parity(u / kKvStages), tw); };
            auto stage = [&](int u) { return lo0 + ((C::OFF_KV + (u % kKvStages) * C::kTile) >> 4); };
            auto q_lo = [&](int x) { return lo0 + kDescK + ((C::OFF_Q + x * C::kTile) >> 4); };
            auto empty = [&](int u) { commit_if(leader, BAR(T_KV_EMPTY + u % kKvStages)); };
            auto scores = [&](int buf, int q, int u) {
                product_s<D, kConv>(leader, tmem + 128 * buf, q_lo(q), stage(u) + kDescK);
                commit_if(leader, BAR(T_S_FULL + 2 * q + buf));
            };
            // O_x (+)= P V_j.  bf16: in two halves of the keys, as the weights become ready.  e4m3: each half's warpgroup
            // also rescales its half of O's columns, so both have to be there.
            auto values = [&](int buf, int x, int u, int j, int use) -> bool {
                const uint32_t d = tmem + 256 + 128 * x, a = tmem + 128 * buf, b = stage(u) + kDescMn;
                if (!tile_wait_warp(BAR(T_P_READY + 2 * buf), parity(use), tw)) return false;
                // e4m3, one O: both warpgroups have scaled it by then
                if (kE4M3 && !C::kOwn && !tile_wait_warp(BAR(T_P_READY + 2 * buf + 1), parity(use), tw)) return false;
                ptx::tc_fence_after();
                product_pv<D, kConv>(leader, d, a, b, 0, j > 0 ? 1u : 0u);
                if (!kE4M3 || C::kOwn) {
                    if (!tile_wait_warp(BAR(T_P_READY + 2 * buf + 1), parity(use), tw)) return false;
                    ptx::tc_fence_after();
                }
                product_pv<D, kConv>(leader, d + (C::kOwn ? 64 : 0), a, b, 1, !C::kOwn || j > 0 ? 1u : 0u);
                return true;
            };
            for (int x = 0; ok && x < tiles; ++x) {
                const int q = tiles == 2 ? x : slot;
                ok = tile_wait_warp(BAR((kConv ? T_Q_READY : T_Q_FULL) + q), parity(pick(it.q_use, q)), tw);
            }
            ok = ok && full(kv0);
            if (!ok) break;
            ptx::tc_fence_after();
            if (tiles == 2) {
                scores(0, 0, kv0);
                scores(1, 1, kv0);
                empty(kv0);
                for (int j = 0; j < nk; ++j) {
                    const int uv = kv0 + 2 * j + 1, uk = uv + 1;
                    const bool more = j + 1 < nk;
                    if (!more) {   // after the last S
                        commit_if(leader, BAR(T_Q_EMPTY + 0));
                        commit_if(leader, BAR(T_Q_EMPTY + 1));
                    }
                    ok = full(uv) && values(0, 0, uv, j, p_use[0] + j);
                    if (!ok) break;
                    if (more) {
                        ok = full(uk);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        scores(0, 0, uk);
                    } else {
                        commit_if(leader, BAR(T_O_FULL + 0));
                    }
                    ok = values(1, 1, uv, j, p_use[1] + j);
                    if (!ok) break;
                    empty(uv);
                    if (more) {
                        scores(1, 1, uk);
                        empty(uk);
                    } else {
                        commit_if(leader, BAR(T_O_FULL + 1));
                    }
                }
            } else {
                int buf = uni(it.buf);
                scores(buf, slot, kv0);
                empty(kv0);
                for (int j = 0; j < nk; ++j, buf ^= 1) {
                    const int uv = kv0 + 2 * j + 1, uk = uv + 1;
                    if (j + 1 < nk) {
                        ok = full(uk);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        scores(buf ^ 1, slot, uk);
                        empty(uk);
                    } else {
                        commit_if(leader, BAR(T_Q_EMPTY + slot));
                    }
                    ok = full(uv) && values(buf, slot, uv, j, pick(p_use, buf) + (j >> 1));
                    if (!ok) break;
                    empty(uv);
                    commit_if(leader, BAR(T_PV_DONE));
                    if (j + 1 == nk) commit_if(leader, BAR(T_O_FULL + slot));
                }
            }
        }
        // after a wait that ran out, the products in flight end before tensor memory is freed (below, after the barrier);
        // otherwise every product has been waited for
        if (*abort) {
            const uint64_t t0 = ptx::globaltimer();
            while (ptx::globaltimer() - t0 < 1000000ull) {
            }
        }
    } else if (warp == 2) {
        // ================================================== scheduler
        const Plan* plan = p.plan;
        const int items = plan->items[p.nb];
        int buf = 0, slot = 0, kv = 0, kt = 0, qi = 0, pv = 0, s_use[2][2] = {{0, 0}, {0, 0}}, p_use[2] = {0, 0}, q_use[2] = {0, 0}, o_use[2] = {0, 0};
        for (int u = 0;; ++u) {
            int item = 0;
            if (lane == 0) item = atomicAdd(p.counter, 1);
            item = __shfl_sync(0xffffffffu, item, 0);
            const int s = u % kItemSlots;
            if (u >= kItemSlots && !tile_wait_warp(BAR(T_ITEM_EMPTY + s), (uint32_t)((u / kItemSlots - 1) & 1), tw)) break;
            TileItem it;
            it.b = -1;
            if (item < items) {
                int lo = 0, hi = p.nb;   // the last sequence with items[i] <= item (it has items of its own)
                while (hi - lo > 1) {
                    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
                    const unsigned le = __ballot_sync(0xffffffffu, at < hi && plan->items[at] <= item);
                    const int k = 31 - __clz(le);   // lane 0 always holds
                    lo += k * step;
                    hi = min(hi, lo + step);
                }
                const Seq q = plan->seq[lo];
                const Cut c = cut_many(p, q, tokens_per_item(p.G));
                const int local = item - plan->items[lo];
                const int per = p.c.Hkv * c.ns, row_tiles = c.items / per;
                const int rt = row_tiles - 1 - local / per;   // the longest causal rows first
                const int split = (local % per) / p.c.Hkv;
                const int i0 = rt * tokens_per_item(p.G);
                it.b = p.b0 + lo;
                it.hk = local % p.c.Hkv;
                it.tok = q.first + i0;
                it.ntok = min(tokens_per_item(p.G), q.n - i0);
                it.pos = q.len - q.n + i0;
                it.lo = c.lo;
                it.hi = c.hi;
                it.len = q.len;
                it.split = c.ns > 1;
                it.part = plan->rows[lo] + ((long long)split * p.c.Hkv + it.hk) * q.n * p.G + (long long)i0 * p.G;
                int klo, khi;   // keys seen by the item's rows
                seen_keys(p, q, i0, i0 + it.ntok, klo, khi);
                const int first = c.lo / 128 + split * c.st;
                it.t0 = max(first, klo / 128);
                it.nk = max(min(first + c.st, khi > klo ? (khi + 127) / 128 : 0) - it.t0, 0);
                it.tiles = it.ntok > tpt ? 2 : 1;
                it.buf = buf;
                it.slot = slot;
                it.kv = kv;
                it.kt = kt;
                it.qi = qi;
                it.pv = pv;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    it.s_use[x] = it.tiles == 2 ? s_use[x][x] : (slot ? s_use[1][x] : s_use[0][x]);
                    it.p_use[x] = p_use[x];
                    it.q_use[x] = q_use[x];
                    it.o_use[x] = o_use[x];
                }
                if (it.nk > 0) {
                    kv += 2 * it.nk;
                    kt += it.nk;
                    ++qi;
                    if (it.tiles == 2) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) s_use[x][x] += it.nk, p_use[x] += it.nk, ++q_use[x], ++o_use[x];
                    } else {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int uses = (it.nk + (x == buf ? 1 : 0)) / 2;
                            (slot ? s_use[1][x] : s_use[0][x]) += uses;
                            p_use[x] += uses;
                            q_use[x] += x == slot ? 1 : 0;
                            o_use[x] += x == slot ? 1 : 0;
                        }
                        pv += it.nk;
                        buf ^= it.nk & 1;
                        slot ^= 1;
                    }
                }
            }
            if (lane == 0) {
                *reinterpret_cast<TileItem*>(smem + C::OFF_ITEM + C::kItemBytes * s) = it;
                ptx::mbar_arrive(BAR(T_ITEM_FULL + s));
            }
            __syncwarp();
            if (it.b < 0) break;
        }
    }
    } else if (warp < 12) {
        ptx::setmaxnreg_inc<C::kRegsSoftmax>();
        // ================================================== softmax and epilogue
        // e4m3: this warpgroup w has keys 64 w .. of every key tile and columns D/2 w .. of O, of both row tiles (n = 0, 1);
        // bf16: everything of row tile w (n = 0).
        constexpr float kLift = kConv ? kLiftE4M3 : 0.f;   // maxima are held less this
        constexpr int kN = kE4M3 ? 2 : 1, kCols = kE4M3 ? 64 : 128, kOut = kE4M3 ? D / 2 : D;
        const int w = (warp - 4) >> 2;
        const int row = 32 * (warp & 3) + lane;
        const uint32_t tbase = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t out0 = 256u + (kE4M3 ? (uint32_t)((C::kOwn ? 64 : kOut) * w) : 0u);   // of O, what this warpgroup scales
        float* const mx_own = reinterpret_cast<float*>(smem + C::OFF_MAX) + 128 * w + row;
        float* const mx_other = reinterpret_cast<float*>(smem + C::OFF_MAX) + 128 * (w ^ 1) + row;
        for (int u = 0;; ++u) {
            // The item stays in its slot until the epilogue: what the loop over its key tiles needs is copied here.
            const int at_slot = u % kItemSlots;
            const TileItem& it = *reinterpret_cast<const TileItem*>(smem + C::OFF_ITEM + C::kItemBytes * at_slot);
            const bool more = tile_wait_warp(BAR(T_ITEM_FULL + at_slot), parity(u / kItemSlots), tw) && it.b >= 0;
            // e4m3: all eight warps take an item, or none: nobody is left alone at the votes below (after a wait that ran
            // out, the others just do not wait)
            if (kE4M3 ? any_of_256(!more) : !more) break;
            const int nk = it.nk, tiles = it.tiles, t0 = it.t0, kt = it.kt, qi = it.qi, pv = it.pv, slot = it.slot;
            const int use0 = it.s_use[0], use1 = it.s_use[1], buf0 = it.buf;
            // row tile of the item, and whether it is this warpgroup's
            auto tile = [&](int n) { return tiles == 1 ? 0 : kE4M3 ? n : w; };
            auto mine = [&](int n) { return kE4M3 ? n < tiles : tiles == 2 || slot == w; };
            auto o_of = [&](int n) { return tiles == 1 ? slot : tile(n); };
            // this row's keys, and the key tiles that every row of its tile sees whole
            int lo_r[kN], hi_r[kN], full_lo[kN], full_hi[kN];
            bool valid[kN];
            float m_ref[kN], l[kN], c[kN];
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                const int x = tile(n), pos_ = it.pos, ntok = it.ntok, len = it.len;
                const int i = x * tpt + row / p.G, pos = pos_ + i;
                valid[n] = row < trows && i < ntok;
                hi_r[n] = p.causal ? pos + 1 : len;
                lo_r[n] = (p.window && pos + 1 > p.window) ? pos + 1 - p.window : 0;
                const int first = pos_ + x * tpt, last = min(pos_ + ntok - 1, first + tpt - 1);
                full_hi[n] = p.causal ? first + 1 : len;
                full_lo[n] = (p.window && last + 1 > p.window) ? last + 1 - p.window : 0;
                m_ref[n] = -INFINITY;
                l[n] = 0.f;
                c[n] = p.scale_log2e;
            }
            float vfac = kE2M1 ? p.v_unit : 1.f;   // O holds the sum over vfac
            for (int j = 0; j < nk && mine(0); ++j) {
                const int key = (t0 + j) * 128 + (kE4M3 ? 64 * w : 0);   // the first of this thread's columns
                uint4 s4[8];                                              // e4m3: scales of 32 of them
                float grown = 1.f;                                        // of O, when the values' power of two has grown
                const uint32_t sc = sbase + C::OFF_KSC + ((kt + j) & 3) * 512 + 256 * w;
                if constexpr (kE4M3) {
                    const int t = kt + j;
                    tile_wait_warp(BAR(T_SCALES + (t & 3)), parity(t >> 2), tw);
                    const float f = reinterpret_cast<const float*>(smem + C::OFF_VFAC)[t & 3];
                    if (j == 0) vfac = f;
                    if (f != vfac) grown = vfac / f;
                    vfac = f;
                }
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    if (!mine(n)) continue;
                    const int buf = tiles == 2 ? tile(n) : (buf0 + j) & 1;
                    if (kE4M3) {   // read while the scores are formed
#pragma unroll
                        for (int k = 0; k < 8; ++k) s4[k] = lds128(sc + 16 * k);
                    }
                    const uint32_t tS = tbase + 128u * (uint32_t)buf + (kE4M3 ? 64u * (uint32_t)w : 0u);
                    const bool ready = tile_wait_warp(BAR(T_S_FULL + 2 * o_of(n) + buf), parity((buf ? use1 : use0) + (tiles == 2 ? j : j >> 1)), tw);
                    (void)ready;   // after a wait that ran out, values that nobody uses
                    ptx::tc_fence_after();
                    float y[kCols];
                    {
                        uint32_t r[kCols / 32][32];
#pragma unroll
                        for (int h = 0; h < kCols / 32; ++h) ptx::tmem_ld32(tS + 32 * h, r[h]);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < kCols; ++k) y[k] = __uint_as_float(r[k >> 5][k & 31]);
                    }
                    if constexpr (kConv) {
                        if (j == 0) {
                            c[n] *= reinterpret_cast<const float*>(
                                smem + C::OFF_QFAC)[((qi & 1) * 2 + (tiles == 2 ? tile(n) : slot)) * 128 + row];
                            if (kE2M1) c[n] = fminf(fmaxf(c[n], 0x1p-126f), 0x1p127f);   // (whatever k_exp: -inf times it stays -inf, zero zero)
                        }
                    }
                    if constexpr (kE4M3) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const uint4 f = s4[k & 7];
                            const ptx::f2 a = ptx::mul2({y[4 * k], y[4 * k + 1]}, {__uint_as_float(f.x), __uint_as_float(f.y)});
                            const ptx::f2 b = ptx::mul2({y[4 * k + 2], y[4 * k + 3]}, {__uint_as_float(f.z), __uint_as_float(f.w)});
                            y[4 * k] = a.x, y[4 * k + 1] = a.y, y[4 * k + 2] = b.x, y[4 * k + 3] = b.y;
                            if (k < 8) s4[k] = lds128(sc + 128 + 16 * k);
                        }
                    }
                    if (key < full_lo[n] || key + kCols > full_hi[n]) {
                        const int ka = lo_r[n] - key, kb = hi_r[n] - key;   // visible columns [ka, kb)
#pragma unroll
                        for (int k = 0; k < kCols; ++k)
                            if (k < ka || k >= kb) y[k] = -INFINITY;
                    }
                    // row maximum and sum over interleaved partials: short chains, one fixed order
                    float part[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) part[k] = fmaxf(y[2 * k], y[2 * k + 1]);
#pragma unroll
                    for (int k = 8; k < kCols; k += 2) part[(k >> 1) & 3] = fmaxf(fmaxf(part[(k >> 1) & 3], y[k]), y[k + 1]);
                    const float top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
                    float mx = kConv ? fmaf(c[n], top, -kLift) : c[n] * top;
                    const bool over = valid[n] && mx > m_ref[n] + 8.f;
                    const bool raise = kE4M3 && !C::kOwn ? any_of_256(over || grown != 1.f) : __any_sync(0xffffffffu, over || grown != 1.f);
                    if (raise) {
                        if (kE4M3 && !C::kOwn) {
                            *mx_own = mx;
                            any_of_256(false);
                            mx = fmaxf(mx, *mx_other);
                        }
                        const float m_new = fmaxf(m_ref[n], mx);
                        const float alpha = m_new == -INFINITY ? 1.f : ptx::ex2(m_ref[n] - m_new);
                        m_ref[n] = m_new;
                        l[n] *= alpha;
                        const float alpha_o = kE4M3 ? alpha * grown : alpha;
                        if (j > 0) {
                            // (one tile: S(j) was issued before PV(j-1))
                            if (tiles == 1) tile_wait_warp(BAR(T_PV_DONE), parity(pv + j - 1), tw);
                            ptx::tc_fence_after();
#pragma unroll 1
                            for (int cc = 0; cc < (C::kOwn ? D : kOut) / 16; ++cc) {
                                const uint32_t tO = tbase + out0 + 128u * (uint32_t)o_of(n) + (uint32_t)(16 * cc);
                                uint32_t r[16];
                                ptx::tmem_ld16(tO, r);
                                ptx::tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha_o);
                                ptx::tmem_st16(tO, r);
                            }
                        }
                    }
                    const float m_use = m_ref[n] == -INFINITY ? 0.f : m_ref[n];
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    // P rounded to bf16 (at most 2^8; e4m3 caches: fp16, lifted, at most 2^15), keys [0,64) -> columns [0,32), [64,128) -> [64,96)
#pragma unroll
                    for (int h = 0; h < kCols / 32; ++h) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const ptx::f2 e = ptx::fma2({y[32 * h + k], y[32 * h + k + 1]}, {c[n], c[n]}, {-m_use, -m_use});
                            const ptx::f2 v{ptx::ex2(e.x), ptx::ex2(e.y)};
                            const ptx::f2 s = ptx::add2({sum[k & 3], sum[(k + 1) & 3]}, v);
                            sum[k & 3] = s.x;
                            sum[(k + 1) & 3] = s.y;
                            pk[k >> 1] = kConv ? pack_half(v.x, v.y) : pack_bf16(v.x, v.y);
                        }
                        ptx::tmem_st16(tS + 64 * (h >> 1) + 16 * (h & 1), pk);
                        if (h & 1) {
                            ptx::tmem_st_wait();
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(BAR(T_P_READY + 2 * buf + (kE4M3 ? w : h >> 1)));
                        }
                    }
                    l[n] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
            }
            float total[kN], part0[kN], part1[kN];   // the row's sum; with an O for each half of the keys, what each is multiplied by
#pragma unroll
            for (int n = 0; n < kN; ++n) total[n] = l[n], part0[n] = part1[n] = 1.f;
            if constexpr (kE4M3) {   // over both halves of the columns, in one order
                float* const sums = reinterpret_cast<float*>(smem + C::OFF_SUM);
                float* const tops = reinterpret_cast<float*>(smem + C::OFF_MAX);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    sums[(2 * n + w) * 128 + row] = l[n];
                    if (C::kOwn) tops[(2 * n + w) * 128 + row] = m_ref[n];
                }
                any_of_256(false);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int at = 2 * n * 128 + row;
                    if (C::kOwn) {
                        m_ref[n] = fmaxf(tops[at], tops[at + 128]);
                        const float mu = m_ref[n] == -INFINITY ? 0.f : m_ref[n];
                        part0[n] = ptx::ex2(tops[at] - mu);
                        part1[n] = ptx::ex2(tops[at + 128] - mu);
                        total[n] = part0[n] * sums[at] + part1[n] * sums[at + 128];
                    } else {
                        total[n] = sums[at] + sums[at + 128];
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                if (!mine(n)) continue;
                const int o = o_of(n), i = tile(n) * tpt + row / p.G, g = row % p.G;
                if (nk > 0) {
                    tile_wait_warp(BAR(T_O_FULL + o), parity(pick(it.o_use, o)), tw);
                    ptx::tc_fence_after();
                }
                const bool split = it.split != 0;
                const long long at = (long long)(it.tok + i) * p.Hq + it.hk * p.G + g;   // row of o and lse
                const long long pr = it.part + (long long)i * p.G + g;
                const bool empty = total[n] == 0.f;   // no key; NaN stays NaN
                const float inv = vfac * (split || empty ? 1.f : 1.f / total[n]);
                const bool keep = split && valid[n] && pr < p.max_rows;
#pragma unroll
                for (int cc = 0; cc < kOut / 32; ++cc) {
                    const int col = (kE4M3 ? kOut * w : 0) + 32 * cc;
                    uint32_t r[32];
                    if (nk > 0) {
                        ptx::tmem_ld32(tbase + 256u + 128u * (uint32_t)o + (uint32_t)col, r);
                        if constexpr (C::kOwn) {
                            uint32_t r1[32];
                            ptx::tmem_ld32(tbase + 256u + 128u * (uint32_t)o + 64u + (uint32_t)col, r1);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                r[k] = __float_as_uint(part0[n] * __uint_as_float(r[k]) + part1[n] * __uint_as_float(r1[k]));
                        }
                        ptx::tmem_ld_wait();
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) r[k] = (nk <= 0 || empty) ? 0u : __float_as_uint(__uint_as_float(r[k]) * inv);
                    if (keep) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<uint4*>(p.part_o + pr * D + col + k) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
                    } else if (!split && valid[n]) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
                            *reinterpret_cast<uint4*>(p.o + at * D + col + k) =
                                make_uint4(pack_bf16(__uint_as_float(r[k]), __uint_as_float(r[k + 1])),
                                           pack_bf16(__uint_as_float(r[k + 2]), __uint_as_float(r[k + 3])),
                                           pack_bf16(__uint_as_float(r[k + 4]), __uint_as_float(r[k + 5])),
                                           pack_bf16(__uint_as_float(r[k + 6]), __uint_as_float(r[k + 7])));
                    }
                }
                const bool stats = !kE4M3 || w == 0;
                if (stats && keep)
                    p.part_ml[pr] = make_float2(empty ? -INFINITY : m_ref[n], empty ? 0.f : total[n]);
                else if (stats && !split && valid[n] && p.lse)
                    p.lse[at] = empty ? -INFINITY : (m_ref[n] + log2f(total[n])) * kLn2P;
            }
            ptx::tc_fence_before();   // O and S are read before the next item's products (its P_READY) overwrite them
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(BAR(T_ITEM_EMPTY + at_slot));
        }
    } else if (kConv) {
        ptx::setmaxnreg_dec<C::kRegsConv>();
        // ================================================== converters
        constexpr int kRows = 512 / D;          // keys that one load instruction of a warp covers (16 codes a lane)
        constexpr int kLoads = 32 / kRows;      // loads of a warp's 32 keys of a tile
        // A lane's 16 codes become two 16-byte chunks of the fp16 row.  Eight consecutive lanes hold four chunk pairs of two
        // neighbouring rows, whose swizzles differ in the lowest bit: no two of them meet in a bank.
        const int cw = warp - 12;
        const int chunk = D == 128 ? (lane & 3) | ((lane >> 3) & 1) << 2 : lane & 3;
        const int sub = D == 128 ? ((lane >> 2) & 1) | (lane >> 4) << 1 : lane >> 2;
        // offsets in a tile of the two chunks of key 32 cw + sub; kRows keys on, the row's swizzle flips chunk bit 2 (D = 128)
        // or stays (D = 64)
        const uint32_t line = (uint32_t)((2 * chunk) >> 3) * kBox + (uint32_t)(32 * cw + sub) * 128;
        const uint32_t to0 = line + ((((2 * chunk) & 7) ^ (sub & 7)) << 4), to1 = line + ((((2 * chunk + 1) & 7) ^ (sub & 7)) << 4);
        TileItem it;
        bool ok = true;
        while (ok && next_item(it)) {
            const int nk = it.nk;
            if (nk <= 0) continue;
            const int e0 = max(it.t0 * 128, it.lo) >> p.page_shift, e1 = (min((it.t0 + nk) * 128, it.hi) - 1) >> p.page_shift;
            int eb = (it.t0 * 128) >> p.page_shift;   // a lane holds the pages of entries eb + lane and eb + 32 + lane
            auto fetch = [&](int e) { return (kE4M3 && e >= e0 && e <= e1) ? checked_page(p, it.b, e) : 0; };
            int pages = fetch(eb + lane), next = fetch(eb + 32 + lane);
            // Unit u is K (even) or V (odd) of key tile t0 + u / 2.  This lane's addresses in it: first and second 16 keys of
            // the warp's 32 (a page holds at least 16), and which keys the sequence sees.
            long long cell[2] = {0, 0};
            int key0 = 0;
            auto aim = [&](int t) {
                if (((t * 128) >> p.page_shift) - eb >= 32) {
                    eb += 32;
                    pages = next;
                    next = fetch(eb + 32 + lane);
                }
                key0 = t * 128 + 32 * cw;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = key0 + 16 * h;
                    const int pg = __shfl_sync(0xffffffffu, pages, ((key >> p.page_shift) - eb) & 31);
                    cell[h] = ((long long)pg * p.c.Hkv + it.hk) * p.c.page_size + (key & (p.c.page_size - 1));
                }
            };
            [[maybe_unused]] auto load = [&](const void* base, uint4 (&w)[kLoads]) {
                const uint8_t* from[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) from[h] = (const uint8_t*)base + (cell[h] + sub) * D + 16 * chunk;
                if (key0 >= it.lo && key0 + 32 <= it.hi) {
#pragma unroll
                    for (int l = 0; l < kLoads; ++l)
                        w[l] = __ldg(reinterpret_cast<const uint4*>(from[l >= kLoads / 2] + (l & (kLoads / 2 - 1)) * (kRows * D)));
                } else {   // keys outside the sequence's read as zero
#pragma unroll
                    for (int l = 0; l < kLoads; ++l) {
                        const int key = key0 + kRows * l + sub;
                        w[l] = make_uint4(0, 0, 0, 0);
                        if (key >= it.lo && key < it.hi)
                            w[l] = __ldg(reinterpret_cast<const uint4*>(from[l >= kLoads / 2] + (l & (kLoads / 2 - 1)) * (kRows * D)));
                    }
                }
            };
            // Scales of a key tile (they come with K): the key's own of K, those of this warp's keys of V, and the largest of
            // V so far, for which every warp reads the whole tile's.
            float ks = 0.f, vs = 0.f, vtop = 0.f, v4[4];
            [[maybe_unused]] auto load_scales = [&](int t) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int key = t * 128 + 32 * c + lane;
                    const bool in = key >= it.lo && key < it.hi;
                    const int pg = __shfl_sync(0xffffffffu, pages, ((key >> p.page_shift) - eb) & 31);
                    const long long at = ((long long)pg * p.c.Hkv + it.hk) * p.c.page_size + (key & (p.c.page_size - 1));
                    v4[c] = in ? __ldg(p.c.v_scale + at) : 0.f;
                    if (c == cw) ks = in ? __ldg(p.c.k_scale + at) : 0.f;
                }
            };
            [[maybe_unused]] auto use_scales = [&]() {
                vs = cw == 0 ? v4[0] : cw == 1 ? v4[1] : cw == 2 ? v4[2] : v4[3];
                vtop = fmaxf(vtop, fmaxf(fmaxf(v4[0], v4[1]), fmaxf(v4[2], v4[3])));
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, d));
            };
            // With the first tile staged: the item's queries, one row per thread (of A, then of B)
            auto queries = [&]() -> bool {
#pragma unroll 1
                for (int x = 0; x < it.tiles; ++x) {
                    const int q = it.tiles == 2 ? x : it.slot;
                    if (!tile_wait_warp(BAR(T_Q_FULL + q), parity(pick(it.q_use, q)), tw)) return false;
                    const int row = 32 * cw + lane;
                    const uint32_t line = sbase + C::OFF_Q + q * C::kTile + row * 128;
                    float top = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        float f[8];
                        unpack_bf16(lds128(line + (c >> 3) * kBox + (((c & 7) ^ (row & 7)) << 4)), f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
                    }
                    float up, down;
                    power_to(top, 14, up, down);
                    reinterpret_cast<float*>(smem + C::OFF_QFAC)[((it.qi & 1) * 2 + q) * 128 + row] = down;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        const uint32_t at = line + (c >> 3) * kBox + (((c & 7) ^ (row & 7)) << 4);
                        float f[8];
                        unpack_bf16(lds128(at), f);
                        sts128(at, make_uint4(pack_half(f[0] * up, f[1] * up), pack_half(f[2] * up, f[3] * up),
                                              pack_half(f[4] * up, f[5] * up), pack_half(f[6] * up, f[7] * up)));
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(BAR(T_Q_READY + q));
                }
                return true;
            };
            // One unit: the codes `w` (loaded during the unit before it) into a stage; `next` (loaded first, so that the proxy
            // fence at the end, which waits for every access before it, finds them there) are the following unit's.
            [[maybe_unused]] auto unit = [&](int u, const uint4 (&w)[kLoads], uint4 (&next)[kLoads]) -> bool {
                const int kv = it.kv + u, st = kv % kKvStages;
                if (kv >= kKvStages && !tile_wait_warp(BAR(T_KV_EMPTY + st), parity(kv / kKvStages - 1), tw)) return false;
                const uint32_t dst = sbase + C::OFF_KV + st * C::kTile;
                float vup, vback;
                power_to(vtop, 6, vup, vback);
                const float scale = vs * vup;
                if (!(u & 1)) {
                    const int slot = (it.kt + (u >> 1)) & 3;
                    reinterpret_cast<float*>(smem + C::OFF_KSC)[slot * 128 + 32 * cw + lane] = ks;
                    if (cw == 0 && lane == 0) reinterpret_cast<float*>(smem + C::OFF_VFAC)[slot] = vback;
                }
                const bool more = u + 1 < 2 * nk;
                if (more && (u & 1)) {
                    aim(it.t0 + (u + 1) / 2);
                    load_scales(it.t0 + (u + 1) / 2);
                }
                if (more) load((u & 1) ? p.c.k : p.c.v, next);
                // fp16 parts of this lane's own key's scale (high part above, low part below)
                uint32_t parts = 0;
                if (u & 1) {
                    const uint32_t hi = pack_half(scale, scale) & 0xffffu;
                    parts = hi << 16 | (pack_half(scale - __half2float(__ushort_as_half((uint16_t)hi)), 0.f) & 0xffffu);
                }
#pragma unroll
                for (int l = 0; l < kLoads; ++l) {
                    const uint32_t c4[4] = {w[l].x, w[l].y, w[l].z, w[l].w};
                    uint32_t o[8];
                    if (u & 1) {
                        const uint32_t both = __shfl_sync(0xffffffffu, parts, kRows * l + sub);
                        const uint32_t hi = __byte_perm(both, 0u, 0x3232), lo = __byte_perm(both, 0u, 0x1010);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            o[2 * y] = scaled_codes(half_codes(c4[y], 0), hi, lo);
                            o[2 * y + 1] = scaled_codes(half_codes(c4[y], 1), hi, lo);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            o[2 * y] = half_codes(c4[y], 0);
                            o[2 * y + 1] = half_codes(c4[y], 1);
                        }
                    }
                    const uint32_t flip = D == 128 && (l & 1) ? 64u : 0u;
                    sts128(((dst + to0) ^ flip) + l * kRows * 128, make_uint4(o[0], o[1], o[2], o[3]));
                    sts128(((dst + to1) ^ flip) + l * kRows * 128, make_uint4(o[4], o[5], o[6], o[7]));
                }
                if (more && (u & 1)) use_scales();
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(BAR(T_KV_FULL + st));
                    if (!(u & 1)) ptx::mbar_arrive(BAR(T_SCALES + ((it.kt + (u >> 1)) & 3)));
                }
                return u != 1 || queries();
            };
            // E2M1: the producer has staged codes and scales; a lane's 16 codes are 8 bytes, with one scale.  K and V alike: values
            // code * scale, exact in fp16.
            [[maybe_unused]] auto unit4 = [&](int u) -> bool {
                const int kv = it.kv + u, st = kv % kKvStages, from = kv % C::kRawStages;
                if (!tile_wait_warp(BAR(T_RAW_FULL + from), parity(kv / C::kRawStages), tw)) return false;
                if (kv >= kKvStages && !tile_wait_warp(BAR(T_KV_EMPTY + st), parity(kv / kKvStages - 1), tw)) return false;
                const uint32_t dst = sbase + C::OFF_KV + st * C::kTile;
                const uint8_t* const raw = smem + C::OFF_RAW + from * C::kRawStage + (32 * cw + sub) * (D / 2) + 8 * chunk;
                const uint8_t* const scales = smem + C::OFF_RAW + from * C::kRawStage + C::kRawCodes + (32 * cw + sub) * (D / 16) + chunk;
                const int first = (it.t0 + (u >> 1)) * 128 + 32 * cw;
                const bool whole = first >= it.lo && first + 32 <= it.hi;
                uint2 w[kLoads];
                uint32_t f[kLoads];
#pragma unroll
                for (int l = 0; l < kLoads; ++l) {
                    w[l] = *reinterpret_cast<const uint2*>(raw + l * kRows * (D / 2));
                    f[l] = scales[l * kRows * (D / 16)];
                    const int key = first + kRows * l + sub;
                    if (!whole && (key < it.lo || key >= it.hi)) w[l] = make_uint2(0, 0), f[l] = 0;   // keys that no row sees: zero
                }
#pragma unroll
                for (int l = 0; l < kLoads; ++l) {
                    const uint32_t s = half2_of_e4m3x2(f[l] | f[l] << 8);
                    const uint32_t c2[2] = {w[l].x, w[l].y};
                    uint32_t o[8];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        o[4 * y] = mul_half2(half2_of_e2m1<0>(c2[y]), s);
                        o[4 * y + 1] = mul_half2(half2_of_e2m1<1>(c2[y]), s);
                        o[4 * y + 2] = mul_half2(half2_of_e2m1<2>(c2[y]), s);
                        o[4 * y + 3] = mul_half2(half2_of_e2m1<3>(c2[y]), s);
                    }
                    const uint32_t flip = D == 128 && (l & 1) ? 64u : 0u;
                    sts128(((dst + to0) ^ flip) + l * kRows * 128, make_uint4(o[0], o[1], o[2], o[3]));
                    sts128(((dst + to1) ^ flip) + l * kRows * 128, make_uint4(o[4], o[5], o[6], o[7]));
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(BAR(T_KV_FULL + st));
                    ptx::mbar_arrive(BAR(T_RAW_EMPTY + from));
                }
                return u != 1 || queries();
            };
            if constexpr (kE4M3) {
                uint4 wk[kLoads], wv[kLoads];
                aim(it.t0);
                load_scales(it.t0);
                load(p.c.k, wk);
                use_scales();
#pragma unroll 1
                for (int u = 0; ok && u < 2 * nk; u += 2) ok = unit(u, wk, wv) && unit(u + 1, wv, wk);
            } else {
#pragma unroll 1
                for (int u = 0; ok && u < 2 * nk; ++u) ok = unit4(u);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int D, int kType>
int launch_tile_t(const PagedParams& p, int grid, cudaStream_t s) {
    using C = TileCfg<D, kType>;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DASH_ERR_CUDA;
    if (dev < 0 || dev >= 64) return DASH_ERR_DEVICE;
    if (!ready[dev]) {
        cudaFuncAttributes a;
        if (cudaFuncSetAttribute(paged_tile_kernel<D, kType>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess ||
            cudaFuncGetAttributes(&a, paged_tile_kernel<D, kType>) != cudaSuccess)
            return DASH_ERR_CUDA;
        if (a.numRegs < C::kRegsLaunch) return DASH_ERR_LAUNCH;   // the softmax would wait for registers that are not there
        ready[dev] = true;
    }
    return launch_after(paged_tile_kernel<D, kType>, grid, C::kThreads, C::kSmem, p, s);
}

}  // namespace

int error_tile(int* out5, bool clear) { return serve_record(out5, clear); }

int launch_paged_many(const PagedParams& few, int grid, cudaStream_t s) {
    PagedParams p = few;
    const int rows = p.c.page_size < 128 ? p.c.page_size : 128;
    const long long heads = (long long)p.c.num_pages * p.c.Hkv;
    const bool bf16 = p.c.type == DASH_CACHE_BF16, d64 = p.c.D == 64;
    // (pages up to the few-rows kernel's stages have its maps)
    if ((bf16 && rows > kFewKeys && make_tmap_pages(&p.tm_k, &p.tm_v, p.c.k, p.c.v, heads, p.c.page_size, p.c.D, false, rows)) ||
        make_tmap_rows(&p.tm_q, p.q, p.T, p.q_t, p.c.Hkv, p.G, p.q_h, p.c.D, 128 / p.G))
        return DASH_ERR_CUDA;
    if (p.c.type == DASH_CACHE_E2M1)
        return d64 ? launch_tile_t<64, DASH_CACHE_E2M1>(p, grid, s) : launch_tile_t<128, DASH_CACHE_E2M1>(p, grid, s);
    if (p.c.type == DASH_CACHE_E4M3)
        return d64 ? launch_tile_t<64, DASH_CACHE_E4M3>(p, grid, s) : launch_tile_t<128, DASH_CACHE_E4M3>(p, grid, s);
    return d64 ? launch_tile_t<64, DASH_CACHE_BF16>(p, grid, s) : launch_tile_t<128, DASH_CACHE_BF16>(p, grid, s);
}

}  // namespace dash
