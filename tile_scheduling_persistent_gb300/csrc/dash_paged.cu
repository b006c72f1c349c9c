// dash_paged.cu -- attention of the newest tokens of each sequence over its
// paged key/value cache (dash_attn_paged): the entry points, the kernel for
// sequences with few rows, and the kernel that joins key ranges.
//
// Few rows (decoding, a few drafted tokens; few_most).  The work is reading the
// cache once: 4 n G D operations against 4 D bytes per key and head (2 D for
// e4m3) is 16 and 64 operations per byte at the most, where the GPU has 285 per
// byte of memory bandwidth.  So everything serves the stream of pages:
//   - one persistent CTA per SM with two or three independent groups, each a
//     producer warp and four consumers working through items of their own (8
//     query rows, a key/value head, a key range): while one group joins the
//     results of an item or waits for the next one's queries, the others
//     stream.  bf16 at D = 128 has shared memory for two;
//   - a group's producer walks its items and keeps a ring of 64-key stages (K
//     and V, 50 or 64 KB) full by TMA, across item boundaries, each lane
//     issuing one of a stage's copies (one per page, 64-value column and K/V:
//     pages of 16 tokens give 16 copies);
//   - each consumer warp takes 16 keys of a stage, all in registers, with the
//     keys (and the values' columns) on the 16-row side of m16n8k16 and the
//     query rows on its 8-column side: S^T = K Q^T, a running maximum and sum
//     per column, O^T += V^T P^T.  With the rows on the 16-row side, half of the
//     work would go to rows that a group of 8 heads does not have.  The wider
//     tcgen05 tiles (128 rows, 4 or 8 of them real) have nothing to add;
//   - more than 8 rows are several items over the same pages, one after another
//     in the order of items, so that all but the first find them in L2.  Two
//     such products in one item halve the reads from L2 and leave registers for
//     two groups only: 16 e4m3 sequences of 16 rows to 5000 keys took 53 us so,
//     43 us as two items (bf16: 71 and 75 us for 64 sequences at D = 64);
//   - at the end of an item the four warps' (O, m, l) are joined in shared
//     memory in a fixed order.
// Measured (Hq = 32, Hkv = 8, D = 128): 64 e4m3 sequences of 1 to 8192 tokens
// 99 us with the join, 5.7 TB/s; two bf16 sequences of 131071 (Hkv = 16) 298 us,
// 7.2 TB/s, as fast as memory goes; one of 1000 tokens 8.6 us.  With few or
// ragged sequences the last round of items is what keeps it from the first two.
//
// e4m3 caches.  Codes become fp16 pairs in registers (exact: e4m3 has 3
// fraction bits and exponents -9..8), so the products run in fp16: Q is scaled
// by a power of two per row so that its largest value lies in [2^14, 2^15) --
// values down to 2^-29 of it keep bf16's 8 bits -- and the scale returns in
// fp32 with the key's own scale: s = (Q 2^a . code) * ks * 2^-a.  The value's
// scale vs joins the weight before it is rounded: w = 2^(s + log2 vs - m' + 7),
// with m' the running maximum of s + log2 vs, so the largest contributions of
// a row lie near 2^7 whatever the scales (kLiftE4M3); the sum l keeps its own
// maximum m.
//
// Masked keys get s = -inf by a select, never by arithmetic, and value rows
// outside the visible keys (stale or unwritten cells, freed pages) are zeroed
// in shared memory before they meet a zero weight.
#include <math.h>
#include <string.h>

#include "dash_internal.h"
#include "dash_paged.cuh"

namespace dash {

namespace {

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit values in fragment layout.
__device__ __forceinline__ uint32_t transposed8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t codes, int upper) {
    uint32_t h;
    const uint16_t c = (uint16_t)(upper ? codes >> 16 : codes);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// The four consumer warps of one group.
__device__ __forceinline__ void consumer_barrier(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }

// ---------------------------------------------------------------- few rows
// kGroups: independent groups of four consumer warps and a producer.
template <int D, bool kE4M3, int kGroups>
struct FewCfg {
    static constexpr int kRows = kFewRows;
    static constexpr int kThreads = kGroups * 160;
    static constexpr int kElem = kE4M3 ? 1 : 2;
    static constexpr int kHalfStage = kFewKeys * D * kElem;   // K, then V
    static constexpr int kStage = 2 * kHalfStage;
    static constexpr int kRing = kGroups == 2 ? 65536 : 51200;                     // bytes of a group's stages
    static constexpr int kStages = (kRing / kStage) < 8 ? kRing / kStage : 8;      // of each group
    static_assert(kStages >= 2, "stage ring");
    static constexpr int kSlotRow = !kE4M3 ? D + 4 : D == 128 ? D + 16 : D + 8;   // floats; keeps the join free of bank conflicts
    static constexpr int OFF_SCALE = kGroups * kStages * kStage;   // [group][stage][K, V][kFewKeys] fp32
    static constexpr int OFF_SLOT = OFF_SCALE + (kE4M3 ? kGroups * kStages * 2 * kFewKeys * 4 : 0);   // [group][warp][row]
    static constexpr int OFF_M = OFF_SLOT + kGroups * 4 * kRows * kSlotRow * 4;   // [group][parity][warp][row]
    static constexpr int OFF_L = OFF_M + kGroups * 2 * 4 * kRows * 4;             // [group][warp][row]
    static constexpr int OFF_PLAN = OFF_L + kGroups * 4 * kRows * 4;
    static constexpr int OFF_BAR = (OFF_PLAN + (int)sizeof(Plan) + 15) / 16 * 16;
    static constexpr int OFF_ABORT = OFF_BAR + kGroups * 2 * kStages * 8;         // after [group][full, empty]
    static constexpr int kSmem = OFF_ABORT + 16;
    static_assert(kSmem <= 232448, "shared memory budget");
};

struct FewItem {
    Seq s;
    int lo, hi, ns;                 // keys seen by any row; key ranges
    int b, hk, split, r0, t0, t1;   // first row; key tiles [t0, t1)
};

// Item `item` of the launch; whole warps.  Its sequence is the last that begins at or before it, found by two votes over
// the plan's counts: an item's step to the next spans tens of short sequences.
__device__ __forceinline__ void find_item(const PagedParams& p, const Plan& plan, int item, FewItem& it) {
    constexpr int kMark = kMaxSeqs / 32;
    const int lane = threadIdx.x & 31;
    const int mark = __popc(__ballot_sync(0xffffffffu, kMark * lane < p.nb && plan.items[kMark * lane] <= item)) - 1;
    const int i = kMark * mark + lane;
    const int b = kMark * mark + __popc(__ballot_sync(0xffffffffu, lane < kMark && i < p.nb && plan.items[i] <= item)) - 1;
    it.s = plan.seq[b];
    it.b = p.b0 + b;
    const int st = plan.st[b], parts = few_parts(it.s.n, p.G);
    seen_keys(p, it.s, 0, it.s.n, it.lo, it.hi);
    const int first = it.lo / kFewKeys, tiles = it.hi > it.lo ? (it.hi - 1) / kFewKeys - first + 1 : 0;
    it.ns = tiles <= st ? 1 : (tiles + st - 1) / st;
    // the parts of a head and range come one after another: they share its cells in L2
    const uint32_t local = (uint32_t)(item - plan.items[b]);
    const int at = (int)(parts == 1 ? local : parts == 2 ? local / 2 : parts == 3 ? local / 3 : local / 4);
    it.r0 = kFewRows * ((int)local - at * parts);
    it.split = quick_div(at, p.c.Hkv, p.over_Hkv);
    it.hk = at - it.split * p.c.Hkv;
    it.t0 = first + it.split * st;
    it.t1 = min(it.t0 + st, first + tiles);
}

// Waits for a phase, at most timeout_ns; after a wait that ran out (reported) nothing waits any more, so that every
// role reaches its end.
__device__ __forceinline__ void few_wait(uint32_t bar, uint32_t parity, volatile int* abort, unsigned long long limit) {
    if (ptx::mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*abort) return;
        if (ptx::globaltimer() - t0 > limit) {
            serve_error(DASH_ERR_TIMEOUT, kOpAttn, blockIdx.x, 0, 0);
            *abort = 1;
            return;
        }
    }
}

template <int D, bool kE4M3, int kGroups>
__global__ void __launch_bounds__(kGroups * 160, 1) paged_few_kernel(const __grid_constant__ PagedParams p, int many) {
    using C = FewCfg<D, kE4M3, kGroups>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Plan& plan = *reinterpret_cast<Plan*>(smem + C::OFF_PLAN);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp < 4 * kGroups ? warp >> 2 : warp - 4 * kGroups;
    const uint32_t ring = sbase + group * C::kStages * C::kStage;
    const uint32_t bar_full = sbase + C::OFF_BAR + group * 16 * C::kStages, bar_empty = bar_full + 8 * C::kStages;

    if (threadIdx.x == 128 * kGroups) {
        *abort = 0;
        for (int s = 0; s < kGroups * C::kStages; ++s) {
            const uint32_t bar = sbase + C::OFF_BAR + (s / C::kStages) * 16 * C::kStages + 8 * (s % C::kStages);
            ptx::mbar_init(bar, 1);
            ptx::mbar_init(bar + 8 * C::kStages, 4);
        }
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&p.tm_k);
        ptx::prefetch_tensormap(&p.tm_v);
    }
    if (many && blockIdx.x == 0 && threadIdx.x == 0) *p.counter = 0;
    make_plan(p, plan, blockIdx.x == 0, many && blockIdx.x == 0 ? p.plan : nullptr);
    launch_dependents();
    const int items = plan.items[p.nb];
    FewItem it;

    if (warp >= 4 * kGroups) {
        // ================================================== producer
        const int page = p.c.page_size, rows = page < kFewKeys ? page : kFewKeys;
        const int subs = kFewKeys / rows;                 // copies of one kind along a stage's keys
        const int kinds = kE4M3 ? 4 : D / 32;             // K (per 64 values), V (same), or K, V and their scales
        const int sub = lane / kinds, kind = lane % kinds;
        const uint32_t sub_bytes = (uint32_t)rows * (2 * D * C::kElem + (kE4M3 ? 8 : 0));
        int tc = 0;                                       // stages used so far
        for (int item = group * gridDim.x + blockIdx.x; item < items; item += kGroups * gridDim.x) {
            find_item(p, plan, item, it);
            if (it.t0 >= it.t1) continue;
            const int e0 = max(it.t0 * kFewKeys, it.lo) >> p.page_shift;
            const int e1 = (min(it.t1 * kFewKeys, it.hi) - 1) >> p.page_shift;
            int eb = (it.t0 * kFewKeys) >> p.page_shift;   // a lane holds the pages of entries eb + lane and eb + 32 + lane
            auto fetch = [&](int e) { return (e >= e0 && e <= e1) ? checked_page(p, it.b, e) : 0; };
            int pages = fetch(eb + lane), next = fetch(eb + 32 + lane);
            for (int t = it.t0; t < it.t1; ++t, ++tc) {
                const int key = t * kFewKeys;
                if ((key >> p.page_shift) - eb >= 32) {
                    eb += 32;
                    pages = next;
                    next = fetch(eb + 32 + lane);
                }
                const int k0 = key + sub * rows;          // this lane's first key
                const bool need = sub < subs && k0 + rows > it.lo && k0 < it.hi;
                const int pg = __shfl_sync(0xffffffffu, pages, ((k0 >> p.page_shift) - eb) & 31);
                const int stage = tc % C::kStages;
                const uint32_t full = bar_full + 8 * stage;
                const int count = __popc(__ballot_sync(0xffffffffu, need && kind == 0));
                if (tc >= C::kStages) few_wait(bar_empty + 8 * stage, (uint32_t)((tc / C::kStages - 1) & 1), abort, p.timeout_ns);
                if (__any_sync(0xffffffffu, *abort)) break;
                if (lane == 0) ptx::mbar_arrive_expect_tx(full, count * sub_bytes);
                __syncwarp();
                if (need) {
                    const int y = k0 & (page - 1), head = pg * p.c.Hkv + it.hk;
                    const uint32_t base = ring + stage * C::kStage;
                    if (!kE4M3) {
                        constexpr int kBoxes = D / 64;
                        const int box = kind % kBoxes, val = kind / kBoxes;
                        ptx::tma_load_3d(base + val * C::kHalfStage + box * (kFewKeys * 128) + sub * rows * 128,
                                         val ? &p.tm_v : &p.tm_k, 64 * box, y, head, full);
                    } else if (kind < 2) {
                        ptx::tma_load_3d(base + kind * C::kHalfStage + sub * rows * D, kind ? &p.tm_v : &p.tm_k, 0, y, head, full);
                    } else {
                        const float* src = (kind == 3 ? p.c.v_scale : p.c.k_scale) + (long long)head * page + y;
                        bulk_load(sbase + C::OFF_SCALE + (((group * C::kStages + stage) * 2 + kind - 2) * kFewKeys + sub * rows) * 4, src,
                                  rows * 4, full);
                    }
                }
            }
            if (__any_sync(0xffffffffu, *abort)) break;
        }
        // let what was issued land before the CTA can end (the consumers have seen all of it unless a wait ran out)
        if (*abort)
            for (int u = max(tc - C::kStages, 0); u < tc; ++u) {
                const uint64_t t0 = ptx::globaltimer();
                while (!ptx::mbar_try_wait(bar_full + 8 * (u % C::kStages), (uint32_t)((u / C::kStages) & 1)) &&
                       ptx::globaltimer() - t0 < 100000000ull) {
                }
            }
        return;
    }

    // ================================================== consumers
    // Fragment of a lane: g = lane / 4, c = lane % 4.  S^T and P^T: keys g and g + 8 of the warp's 16, query rows
    // 2c and 2c + 1; O^T: columns of the values as commented below, the same query rows.
    const int g = lane >> 2, c4 = lane & 3;
    const int ws = warp & 3;
    // key of row n of an 8-key tile: e4m3 reads whole 16-byte chunks per lane, and this order keeps both the K reads
    // (rows n, n + 1 in one quarter of a warp) and the V reads (rows 2c) free of bank conflicts under the 128-byte swizzle
    auto perm = [](int n) { return kE4M3 ? (int)((0x36147250u >> (4 * n)) & 7u) : n; };
    float* const slots = reinterpret_cast<float*>(smem + C::OFF_SLOT) + group * 4 * C::kRows * C::kSlotRow;
    float* const mrow = reinterpret_cast<float*>(smem + C::OFF_M) + group * 2 * 4 * C::kRows;
    float* const lrow = reinterpret_cast<float*>(smem + C::OFF_L) + group * 4 * C::kRows;
    // Q^T: row g; k-step k holds values 16k + 2c, + 1 and + 8, + 9; e4m3: 64(k/4) + 16c + 4(k%4) + 0..3.  Loaded before the
    // join of the item before, which hides the wait.
    uint32_t qf[D / 16][2];
    auto load_queries = [&](const FewItem& x) {
        const int r = x.r0 + min(g, min(x.s.n * p.G - x.r0, kFewRows) - 1), i = quick_div(r, p.G, p.over_G);
        const __nv_bfloat16* q = p.q + (long long)(x.s.first + i) * p.q_t + (long long)(x.hk * p.G + r - i * p.G) * p.q_h;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            if (!kE4M3) {
                qf[k][0] = *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * c4);
                qf[k][1] = *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * c4 + 8);
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(q + 64 * (k >> 2) + 16 * c4 + 4 * (k & 3));
                qf[k][0] = w.x;
                qf[k][1] = w.y;
            }
        }
    };
    FewItem after;   // the next item
    const int first_item = group * gridDim.x + blockIdx.x, step = kGroups * gridDim.x;
    if (first_item < items) {
        find_item(p, plan, first_item, after);
        load_queries(after);
    }
    int tc = 0, parity = 0;
    for (int item = first_item; item < items; item += step, parity ^= 1) {
        it = after;
        const int all = it.s.n * p.G, R = min(all - it.r0, kFewRows);   // rows of the sequence, and of this item
        // keys [lo, hi) of this lane's query rows; key tiles in [full_lo, full_hi) are seen whole by every row
        int hi[2], lo[2], full_lo, full_hi, skip;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = quick_div(it.r0 + min(2 * c4 + e, R - 1), p.G, p.over_G);
            seen_keys(p, it.s, i, i + 1, lo[e], hi[e]);
        }
        seen_keys(p, it.s, 0, 1, skip, full_hi);
        seen_keys(p, it.s, it.s.n - 1, it.s.n, full_lo, skip);

        float qs[2];   // scale of the scores of rows 2c + e (log2 units)
        if (!kE4M3) {
            qs[0] = qs[1] = p.scale_log2e;
        } else {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[k][x] << 16)), fabsf(__uint_as_float(qf[k][x] & 0xffff0000u))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^a with 2^a * top in [2^14, 2^15); exponents kept where 2^a and 2^-a are normal
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -112), 127);
            const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            const float down = p.scale_log2e * __uint_as_float((uint32_t)(127 - 14 + e) << 23);
            qs[0] = __shfl_sync(0xffffffffu, down, 8 * c4);
            qs[1] = __shfl_sync(0xffffffffu, down, 8 * c4 + 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t w = qf[k][x];
                    qf[k][x] = pack_half(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                }
        }

        float o[D / 16][4], m[2], mv[2], l[2];
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[e] = mv[e] = -INFINITY;
            l[e] = 0.f;
        }

        for (int kt = it.t0; kt < it.t1; ++kt, ++tc) {
            const int stage = tc % C::kStages;
            few_wait(bar_full + 8 * stage, (uint32_t)((tc / C::kStages) & 1), abort, p.timeout_ns);
            __syncwarp();
            const uint32_t sk = ring + stage * C::kStage, sv = sk + C::kHalfStage;
            const int key0 = kt * kFewKeys + 16 * ws;   // this warp's first key
            const bool edge = key0 < full_lo || key0 + 16 > full_hi;
            if (edge) {   // value rows that no row sees: zero, whatever the cells hold
                const int r = lane >> 1;
                if (key0 + r < it.lo || key0 + r >= it.hi) {
                    const int row = 16 * ws + r;
                    constexpr int kRow = D * C::kElem / 2;   // bytes per lane
#pragma unroll
                    for (int x = 0; x < kRow; x += 16) {
                        const int byte = (lane & 1) * kRow + x;   // rows are zeroed whole: the swizzle stays inside a row
                        sts128(kE4M3 || D == 64 ? sv + row * (D * C::kElem) + byte
                                                : sv + (byte >> 7) * (kFewKeys * 128) + row * 128 + (byte & 127),
                               make_uint4(0, 0, 0, 0));
                    }
                }
                __syncwarp();
            }

            float s[4];   // (key g, rows 2c, 2c + 1), (key g + 8, the same)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = 0.f;
            if (!kE4M3) {
                const int row = 16 * ws + (lane & 15);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t a[4];
                    const int chunk = 2 * (k & 3) + (lane >> 4);
                    ldsm4(sk + (k >> 2) * (kFewKeys * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), a);
                    mma16816<false>(s, a, qf[k][0], qf[k][1]);
                }
            } else {
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const int chunk = 4 * h + c4;
                    uint32_t w[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int row = 16 * ws + 8 * n + perm(g);
                        const uint4 v = lds128(D == 128 ? sk + row * 128 + ((chunk ^ (row & 7)) << 4)
                                                        : sk + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
                        w[n][0] = v.x, w[n][1] = v.y, w[n][2] = v.z, w[n][3] = v.w;
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t a[4] = {half2_of_e4m3(w[0][x], 0), half2_of_e4m3(w[1][x], 0), half2_of_e4m3(w[0][x], 1),
                                               half2_of_e4m3(w[1][x], 1)};
                        mma16816<true>(s, a, qf[4 * h + x][0], qf[4 * h + x][1]);
                    }
                }
            }

            // scores in log2 units; lv = log2 of the value scales (e4m3)
            float ks[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
            if (kE4M3) {
                const float* sc = reinterpret_cast<const float*>(smem + C::OFF_SCALE) +
                                  (group * C::kStages + stage) * 2 * kFewKeys + 16 * ws + perm(g);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    ks[n] = sc[8 * n];
                    lv[n] = lg2(sc[kFewKeys + 8 * n]);
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) s[2 * n + e] *= kE4M3 ? qs[e] * ks[n] : qs[e];
            if (edge) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int key = key0 + 8 * n + perm(g);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (key < lo[e] || key >= hi[e]) s[2 * n + e] = -INFINITY;
                    if (key < it.lo || key >= it.hi) lv[n] = 0.f;
                }
            }
            // Running maxima (m of s; mv of s + lv, less the lift), raised only when a row outgrows them by 2^8.  Whether one does needs a
            // vote alone; the maxima over the warp's keys are formed only then.
            bool raise = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                raise = raise || fmaxf(s[e], s[2 + e]) > m[e] + 8.f;
                if (kE4M3) raise = raise || fmaxf(s[e] + lv[0], s[2 + e] + lv[1]) > mv[e] + (8.f + kLiftE4M3);
            }
            if (__any_sync(0xffffffffu, raise)) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[e], s[2 + e]), mw = kE4M3 ? fmaxf(s[e] + lv[0], s[2 + e] + lv[1]) : 0.f;
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) {
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        if (kE4M3) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, d));
                    }
                    const float nm = fmaxf(m[e], mx), nv = kE4M3 ? fmaxf(mv[e], mw - kLiftE4M3) : nm;
                    l[e] *= nm == -INFINITY ? 1.f : ptx::ex2(m[e] - nm);
                    f[e] = nv == -INFINITY ? 1.f : ptx::ex2((kE4M3 ? mv[e] : m[e]) - nv);
                    m[e] = nm;
                    mv[e] = nv;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    o[j][0] *= f[0];
                    o[j][1] *= f[1];
                    o[j][2] *= f[0];
                    o[j][3] *= f[1];
                }
            }
            uint32_t pb[2];   // P^T as the second operand: keys 2c, 2c + 1 (and + 8) of query row g
            float w[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mu = m[e] == -INFINITY ? 0.f : m[e], vu = mv[e] == -INFINITY ? 0.f : mv[e];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float x = s[2 * n + e];
                    const float pr = ptx::ex2(x - mu);
                    l[e] += pr;
                    w[2 * n + e] = kE4M3 ? ptx::ex2(x + (lv[n] - vu)) : pr;
                }
            }
            // rounded to the products' 16-bit type (bf16; fp16 with e4m3), the sum l from the unrounded weights
#pragma unroll
            for (int n = 0; n < 2; ++n)
                pb[n] = transposed8x8(kE4M3 ? pack_half(w[2 * n], w[2 * n + 1]) : pack_bf16(w[2 * n], w[2 * n + 1]));

            if (!kE4M3) {   // tile j of O^T: value columns 16j + g and + 8
                const int row = 16 * ws + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t a[4];
                    const int chunk = 2 * (j & 3) + ((lane >> 3) & 1);
                    ldsm4_t(sv + (j >> 2) * (kFewKeys * 128) + row * 128 + ((chunk ^ (row & 7)) << 4), a);
                    mma16816<false>(o[j], a, pb[0], pb[1]);
                }
            } else {        // tile j of O^T: value columns (D / 8) g + 2j and + 1
                const int r0 = 16 * ws + perm(2 * c4), r1 = 16 * ws + perm(2 * c4 + 1);
                constexpr int kWords = D / 32;   // words of a lane's D / 8 columns
                uint32_t w[4][kWords];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = (x & 1 ? r1 : r0) + 8 * (x >> 1);
                    if (D == 128) {
                        const uint4 v = lds128(sv + row * 128 + ((g ^ (row & 7)) << 4));
                        w[x][0] = v.x, w[x][1] = v.y, w[x][kWords - 2] = v.z, w[x][kWords - 1] = v.w;
                    } else {
                        const uint2 v = lds64(sv + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
                        w[x][0] = v.x, w[x][1] = v.y;
                    }
                }
#pragma unroll
                for (int y = 0; y < kWords; ++y)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {   // columns 4y + 2z, + 1: byte pairs of the two keys of each half
                        const uint32_t sel = z ? 0x7362u : 0x5140u;
                        const uint32_t lo2 = __byte_perm(w[0][y], w[1][y], sel), hi2 = __byte_perm(w[2][y], w[3][y], sel);
                        const uint32_t a[4] = {half2_of_e4m3(lo2, 0), half2_of_e4m3(lo2, 1), half2_of_e4m3(hi2, 0), half2_of_e4m3(hi2, 1)};
                        mma16816<true>(o[2 * y + z], a, pb[0], pb[1]);
                    }
            }
            if (edge) ptx::fence_proxy_async_smem();   // the zeroed rows before the next copy into the stage
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_empty + 8 * stage);
        }

        if (item + step < items) {
            find_item(p, plan, item + step, after);
            load_queries(after);
        }

        // ---------------------------------------------- join the four warps
        float* const mp = mrow + parity * 4 * C::kRows;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
            if (g == 0) mp[ws * C::kRows + 2 * c4 + e] = m[e];
        }
        consumer_barrier(group);
        float* const slot = slots + ws * C::kRows * C::kSlotRow;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * c4 + e;
            if (r >= R) continue;   // rows past R hold copies; they are neither joined nor stored
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) top = fmaxf(top, mp[w * C::kRows + r]);
            // outputs carry 2^-mv (weights with their scales), sums 2^-m
            const float fo = (top == -INFINITY || mv[e] == -INFINITY) ? 0.f : ptx::ex2((kE4M3 ? mv[e] : m[e]) - top);
            if (g == 0) lrow[ws * C::kRows + r] = l[e] * ((top == -INFINITY || m[e] == -INFINITY) ? 0.f : ptx::ex2(m[e] - top));
            float* row = slot + r * C::kSlotRow;
            if (!kE4M3) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    row[16 * j + g] = o[j][e] * fo;
                    row[16 * j + g + 8] = o[j][2 + e] * fo;
                }
            } else {
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {   // values (D / 8) g + 4k..: the chunk XOR c spreads the banks
                    const int chunk = ((D / 32) * g + k) ^ (D == 128 ? c4 : c4 >> 1);
                    *reinterpret_cast<float4*>(row + 4 * chunk) =
                        make_float4(o[2 * k][e] * fo, o[2 * k][2 + e] * fo, o[2 * k + 1][e] * fo, o[2 * k + 1][2 + e] * fo);
                }
            }
        }
        consumer_barrier(group);
        for (int i = threadIdx.x & 127; i < R * (D / 4); i += 128) {
            const int r = i / (D / 4), q4 = i % (D / 4), c = (r >> 1) & 3;
            const int chunk = kE4M3 ? q4 ^ (D == 128 ? c : c >> 1) : q4;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(slots + (w * C::kRows + r) * C::kSlotRow + 4 * chunk);
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                top = fmaxf(top, mp[w * C::kRows + r]);
                sum += lrow[w * C::kRows + r];
            }
            if (it.ns == 1) {
                const int token = quick_div(it.r0 + r, p.G, p.over_G), tok = it.s.first + token, h = it.hk * p.G + it.r0 + r - token * p.G;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;   // 0: no key; NaN stays NaN
                *reinterpret_cast<uint2*>(p.o + ((long long)tok * p.Hq + h) * D + 4 * q4) =
                    make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
                if (p.lse && q4 == 0) p.lse[(long long)tok * p.Hq + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2P;
            } else {
                const long long row = plan.rows[it.b - p.b0] + ((long long)it.split * p.c.Hkv + it.hk) * all + it.r0 + r;
                if (row < p.max_rows) {   // always, unless cu_q (reported) decreases somewhere
                    *reinterpret_cast<float4*>(p.part_o + row * D + 4 * q4) = a;
                    if (q4 == 0) p.part_ml[row] = make_float2(top, sum);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- joining key ranges
// o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the ns ranges of a row of a split sequence.  A block takes units:
// eight rows, one for each warp, which adds the ranges in ascending order; or one row of a sequence with many ranges
// (more than kWarpRanges, where one warp's chain of loads would take tens of microseconds), warp w adding ranges w,
// w + 8, ... and the eight sums added in order.  Which of the two depends on the row's own ns.  A block finds its first
// unit while the kernel before it runs.  It does not fit beside that kernel's CTA (its 18 or 24 thousand registers, where
// those hold 54 to 65 of an SM's 65 thousand), so this overlaps with the last CTAs only: blocks start on SMs whose CTA has ended.
constexpr int kWarpRanges = 48;

// Adds ranges s0, s0 + step, ... of the partial rows base, base + stride, ...: (sum l, sum o of this lane's D / 32 columns)
// relative to the maximum mu.
template <int D>
__device__ __forceinline__ void add_ranges(const PagedParams& p, long long base, long long stride, int s0, int step, int ns, float mu,
                                           float (&a)[D / 32], float& l) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
    for (int s = s0; s < ns; s += 8 * step) {   // eight loads at a time
        float2 ml[8];
        float v[8][E];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const long long at = base + (s + k * step) * stride;
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) v[k][e] = 0.f;
            if (s + k * step < ns) {
                ml[k] = p.part_ml[at];
                const float* o = p.part_o + at * D + E * lane;
                if (E == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(o);
                    v[k][0] = x.x, v[k][1] = x.y, v[k][E - 2] = x.z, v[k][E - 1] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(o);
                    v[k][0] = x.x, v[k][1] = x.y;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float f = ptx::ex2(ml[k].x - mu);
            l += f * ml[k].y;
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] += f * v[k][e];
        }
    }
}

template <int D>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ PagedParams p) {
    constexpr int E = D / 32, kSeqs = kMaxSeqs / 256;
    struct Unit {
        int first, n, ns, local;   // its sequence; the first (token, head) in it
        long long base;            // partial row of the sequence's first row
    };
    __shared__ Unit found[2];
    __shared__ int sums[2][8];
    __shared__ float part[8][D];
    __shared__ float part_l[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // this thread's sequences: units, partial rows, and the counts before
    Seq seq[kSeqs];
    int ns_[kSeqs], units = 0, parts = 0;
    const int per = p.nb > 256 ? kSeqs : 1;
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) seq[k] = Seq{0, 0, 0}, ns_[k] = 1;
    auto units_of = [&](int k) {
        const int rows = seq[k].n * p.Hq;
        return ns_[k] <= 1 ? 0 : ns_[k] <= kWarpRanges ? (rows + 7) / 8 : rows;
    };
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
        const int i = per * (int)threadIdx.x + k;
        if (k >= per || i >= p.nb) continue;
        seq[k] = load_seq(p, p.b0 + i, false);
        if (seq[k].n == 0) continue;
        ns_[k] = (few_rows(seq[k].n, p.G, p.c.type) ? cut_few(p, seq[k]) : cut_many(p, seq[k], tokens_per_item(p.G))).ns;
        units += units_of(k);
        if (ns_[k] > 1) parts += seq[k].n * p.Hq * ns_[k];
    }
    int su = units, sp = parts;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, su, d), y = __shfl_up_sync(0xffffffffu, sp, d);
        if (lane >= d) su += x, sp += y;
    }
    if (lane == 31) sums[0][warp] = su, sums[1][warp] = sp;
    __syncthreads();
    int total = 0;
    su -= units, sp -= parts;
    for (int w = 0; w < 8; ++w) {
        if (w < warp) su += sums[0][w], sp += sums[1][w];
        total += sums[0][w];
    }
    int turn = 0;
    for (int w = blockIdx.x; w < total; w += gridDim.x, turn ^= 1) {
        if (w >= su && w < su + units) {   // one thread of the block
            int u0 = su;
            long long p0 = sp;
#pragma unroll
            for (int k = 0; k < kSeqs; ++k) {
                const int here = units_of(k);
                if (w >= u0 && w < u0 + here)
                    found[turn] = Unit{seq[k].first, seq[k].n, ns_[k], (w - u0) * (ns_[k] <= kWarpRanges ? 8 : 1), p0};
                u0 += here;
                if (ns_[k] > 1) p0 += (long long)seq[k].n * p.Hq * ns_[k];
            }
        }
        __syncthreads();
        if (w == (int)blockIdx.x) wait_dependency();
        const Unit unit = found[turn];
        const bool alone = unit.ns <= kWarpRanges;
        const int local = unit.local + (alone ? warp : 0);
        const int i = local / p.Hq, h = local % p.Hq, hk = h / p.G;
        const int R = unit.n * p.G;
        const long long stride = (long long)p.c.Hkv * R, base = unit.base + (long long)hk * R + i * p.G + h % p.G;
        const long long at = (long long)(unit.first + i) * p.Hq + h;
        const bool real = i < unit.n && base + (unit.ns - 1) * stride < p.max_rows;   // (the second: unless cu_q, reported, decreases)
        float top = -INFINITY, l = 0.f, a[E];
        if (real) {
            for (int s = lane; s < unit.ns; s += 32) top = fmaxf(top, p.part_ml[base + s * stride].x);
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            add_ranges<D>(p, base, stride, alone ? 0 : warp, alone ? 1 : 8, unit.ns, top == -INFINITY ? 0.f : top, a, l);
        }
        if (!alone) {
            if (real) {
#pragma unroll
                for (int e = 0; e < E; ++e) part[warp][E * lane + e] = a[e];
                if (lane == 0) part_l[warp] = l;
            }
            __syncthreads();
            if (real && warp == 0) {
                l = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    l += part_l[v];
#pragma unroll
                    for (int e = 0; e < E; ++e) a[e] += part[v][E * lane + e];
                }
            }
            __syncthreads();
        }
        if (real && (alone || warp == 0)) {
            const float inv = l == 0.f ? 0.f : 1.f / l;   // 0: no key; NaN stays NaN
            __nv_bfloat16* o = p.o + at * D + E * lane;
            if (E == 4)
                *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(a[0] * inv, a[1] * inv), pack_bf16(a[E - 2] * inv, a[E - 1] * inv));
            else
                *reinterpret_cast<uint32_t*>(o) = pack_bf16(a[0] * inv, a[1] * inv);
            if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2P;
        }
    }
    if ((int)blockIdx.x >= total) wait_dependency();
}

// ---------------------------------------------------------------- host
int sm_count() {
    static int count[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!count[dev] && cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return count[dev];
}

template <int D, bool kE4M3, int kGroups>
int launch_few_t(const PagedParams& p, int many, int max_items, cudaStream_t s) {
    using C = FewCfg<D, kE4M3, kGroups>;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DASH_ERR_CUDA;
    if (dev < 0 || dev >= 64) return DASH_ERR_DEVICE;
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(paged_few_kernel<D, kE4M3, kGroups>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem) != cudaSuccess)
            return DASH_ERR_CUDA;
        ready[dev] = true;
    }
    const int sms = sm_count();
    if (sms <= 0) return DASH_ERR_CUDA;
    paged_few_kernel<D, kE4M3, kGroups><<<max_items < sms ? max_items : sms, C::kThreads, C::kSmem, s>>>(p, many);
    return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

// Three groups where their registers and stages allow it (few_workers counts on it).
int launch_few(const PagedParams& p, int many, int max_items, cudaStream_t s) {
    if (p.c.type == DASH_CACHE_E4M3)
        return p.c.D == 64 ? launch_few_t<64, true, 3>(p, many, max_items, s) : launch_few_t<128, true, 3>(p, many, max_items, s);
    return p.c.D == 64 ? launch_few_t<64, false, 3>(p, many, max_items, s) : launch_few_t<128, false, 2>(p, many, max_items, s);
}

// Its plan is made while the kernel before it in the stream runs.
template <int D>
int launch_combine(const PagedParams& p, long long max_rows, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return DASH_ERR_CUDA;
    // Three blocks for each SM, which holds that many at D = 64 and two at D = 128 (96 registers): each one makes the plan, so
    // more only repeat it (16 x 5 tokens over to 5000 bf16 keys, D = 128: 54 us with three, 56.5 with six, 62 with twelve, 55
    // with one; two were not tried).
    return launch_after(combine_kernel<D>, (unsigned)(max_rows < 3ll * sms ? max_rows : 3ll * sms), 256, 0, p, s);
}

// Bounds that the host knows of a launch of nb sequences, whatever the cache's type: items of the few-rows class, partial
// rows of both classes.
struct Bounds {
    long long few_items, rows;
};

Bounds bounds(int nb, long long T, int Hq, int Hkv, int max_q, long long max_kv) {
    const int G = Hq / Hkv;
    Bounds r{0, 0};
    const long long few_q = G > kFewMost ? 0 : (max_q < kFewMost / G ? max_q : kFewMost / G);   // tokens of a few-rows sequence
    const long long n_few = nb < T ? nb : T;
    if (few_q > 0) {
        const long long tiles = (max_kv + kFewKeys - 1) / kFewKeys;
        long long ns = 1;   // whichever of few_workers and few_parts a sequence has
        for (int parts = 1; parts <= kFewMost / kFewRows; ++parts)
            for (int workers : {kFewWorkers, kFewWorkers3}) {
                const long long most = few_most_ranges(tiles, workers, Hkv * parts);
                ns = ns < most ? most : ns;
            }
        r.few_items = n_few * Hkv * ns * (kFewMost / kFewRows);
        if (ns > 1) r.rows += (few_q * n_few < T ? few_q * n_few : T) * Hq * ns;
    }
    if ((long long)max_q * G > few_most(DASH_CACHE_BF16)) {
        const long long by_kv = max_kv / kTileSplitKeys + 2, by_heads = kTileSms / Hkv;   // ranges of a sequence
        const long long ns = by_kv < by_heads ? by_kv : by_heads;
        const long long least = few_most(DASH_CACHE_BF16) / G + 1;                       // tokens of the smallest many-rows sequence
        const long long n_many = T / least < nb ? T / least : nb;
        // a split sequence has at most kTileSms items, of at most kTileRows rows
        const long long by_items = n_many * kTileSms * kTileRows, by_len = ns > 1 ? T * Hq * ns : 0;
        r.rows += by_items < by_len ? by_items : by_len;
    }
    return r;
}

constexpr size_t kWsHeader = (256 + sizeof(Plan) + 255) / 256 * 256;   // the many-rows kernel's item counter and plan

}  // namespace

int error_paged(int* out5, bool clear) { return serve_record(out5, clear); }

}  // namespace dash

using namespace dash;

extern "C" int dash_attn_paged_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int64_t max_kv,
                                         size_t* bytes) {
    if (!bytes || B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 128 || (D != 64 && D != 128) ||
        max_q < 0 || max_kv < 0 || max_kv >= (1ll << 31) - 512 || (long long)T * Hq >= (1ll << 31))
        return DASH_ERR_ARG;
    *bytes = 0;
    if (B == 0 || T == 0) return DASH_OK;
    const Bounds b = bounds(B < kMaxSeqs ? B : kMaxSeqs, T, Hq, Hkv, max_q, max_kv);
    if (b.rows >= (1ll << 31) || b.few_items >= (1ll << 31)) return DASH_ERR_ARG;
    const bool many = (long long)max_q * (Hq / Hkv) > few_most(DASH_CACHE_BF16);
    if (b.rows || many) *bytes = kWsHeader + (size_t)b.rows * (D * sizeof(float) + sizeof(float2));
    return DASH_OK;
}

extern "C" int dash_attn_paged(const dash_bf16* q, int64_t q_stride_t, int64_t q_stride_h, const dash_kv_cache* cache,
                               const int32_t* block_table, int64_t table_stride, int max_pages,
                               const int32_t* kv_lens, const int32_t* cu_q, dash_bf16* o, float* lse, int B, int T,
                               int Hq, int max_q, int causal, int window, void* workspace, size_t workspace_bytes,
                               dash_stream_t stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (max_pages < 0 || table_stride < 0 || (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal) ||
        !serve_strides(q_stride_t, q_stride_h) || (T > 1 && q_stride_t == 0) || (Hq > 1 && q_stride_h == 0))
        return DASH_ERR_ARG;
    const int Hkv = cache->Hkv, D = cache->D;
    const int64_t max_kv = (int64_t)max_pages * cache->page_size;
    size_t need = 0;
    if ((rc = dash_attn_paged_workspace(B, T, Hq, Hkv, D, max_q, max_kv, &need))) return rc;
    if (B == 0 || T == 0) return DASH_OK;
    if (!serve_aligned(q) || !serve_aligned(o) || ((uintptr_t)lse & 3u) || !kv_lens || ((uintptr_t)kv_lens & 3u) ||
        ((uintptr_t)cu_q & 3u) || ((uintptr_t)block_table & 3u) || (max_pages > 0 && !block_table) ||
        (!cu_q && (T % B || T / B > max_q)) || (need && !serve_aligned(workspace)))
        return DASH_ERR_ARG;
    if (workspace_bytes < need) return DASH_ERR_SCRATCH;
    if ((rc = serve_check_device())) return rc;

    PagedParams prm;
    memset(&prm, 0, sizeof(prm));
    prm.c = *cache;
    prm.q = (const __nv_bfloat16*)q;
    prm.q_t = q_stride_t;
    prm.q_h = q_stride_h;
    prm.table_stride = table_stride;
    prm.table = block_table;
    prm.lens = kv_lens;
    prm.cu_q = cu_q;
    prm.o = (__nv_bfloat16*)o;
    prm.lse = lse;
    prm.timeout_ns = timeout_ns();
    prm.max_pages = max_pages;
    prm.B = B;
    prm.T = T;
    prm.Hq = Hq;
    prm.G = Hq / Hkv;
    prm.over_G = reciprocal(prm.G);
    prm.over_Hkv = reciprocal(Hkv);
    prm.max_q = max_q;
    prm.causal = causal;
    prm.window = window;
    while ((1 << prm.page_shift) < cache->page_size) ++prm.page_shift;
    prm.scale_log2e = (1.0f / sqrtf((float)D)) * kLog2eP;
    const bool e4m3 = cache->type == DASH_CACHE_E4M3;
    const int rows = cache->page_size < kFewKeys ? cache->page_size : kFewKeys;
    if (make_tmap_pages(&prm.tm_k, &prm.tm_v, cache->k, cache->v, (long long)cache->num_pages * Hkv, cache->page_size, D, e4m3, rows))
        return DASH_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    for (int b0 = 0; b0 < B; b0 += kMaxSeqs) {
        prm.b0 = b0;
        prm.nb = B - b0 < kMaxSeqs ? B - b0 : kMaxSeqs;
        const Bounds bd = bounds(prm.nb, T, Hq, Hkv, max_q, max_kv);
        if (need) {
            prm.counter = (int*)workspace;
            prm.plan = (Plan*)((char*)workspace + 256);
            prm.part_o = (float*)((char*)workspace + kWsHeader);
            prm.part_ml = (float2*)(prm.part_o + bd.rows * D);
            prm.max_rows = bd.rows;
        }
        const bool many = (long long)max_q * prm.G > few_most(cache->type);
        const int items = (int)(bd.few_items < 1 ? 1 : bd.few_items);   // at least one block: it checks the lengths
        rc = launch_few(prm, many, items, s);
        if (rc) return rc;
        if (many && (rc = launch_paged_many(prm, sm_count(), s))) return rc;
        if (bd.rows && (rc = D == 64 ? launch_combine<64>(prm, (long long)T * Hq, s) : launch_combine<128>(prm, (long long)T * Hq, s)))
            return rc;
    }
    return DASH_OK;
}
