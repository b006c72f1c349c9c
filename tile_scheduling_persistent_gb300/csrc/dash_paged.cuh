// dash_paged.cuh -- what the kernels of the paged attention share: how the
// sequences of a call are cut into work items, and the partial results of
// sequences whose keys are split.
//
// A sequence with n new tokens has n * G rows per key/value head (row r is
// token r / G, head r % G of the group: one row of queries reads the same keys
// for the whole group).  Two classes, by the sequence's own size:
//   few rows (few_most): memory bound; items of (8 rows, head, key range), dash_paged.cu
//   many rows: items of (256 rows, head, key range), dash_paged_tile.cu
// Every cut depends on the sequence's own lengths and on Hkv, G and D, never on
// the rest of the batch or on the number of SMs, so that a sequence's results
// are the same bits in any batch.
//
// A sequence cut into ns > 1 key ranges leaves, for each range and row, the
// unnormalised fp32 output, its maximum m (log2 units) and its sum l relative
// to m; combine_kernel joins the ranges in ascending order.
#pragma once
#include "dash_ptx.cuh"
#include "dash_serve.cuh"

namespace dash {

constexpr int kFewRows = 8;        // query rows of an item of the few-rows kernel
constexpr int kFewMost = 32;       // rows of a sequence of its class, at the most (few_most)
constexpr int kFewKeys = 64;       // keys per stage of the few-rows kernel
constexpr int kFewWholeTiles = 4;  // sequences of so many stages are not split: joining costs more than it gains
constexpr int kFewWorkers = 304;   // groups on a GB300's 152 SMs: two of each CTA,
constexpr int kFewWorkers3 = 456;  // or three
constexpr int kMaxSeqs = 512;      // sequences per launch (their plan lies in shared memory)
constexpr int kTileRows = 256;     // rows per item of the many-rows kernel
constexpr int kTileSplitKeys = 768;    // at least this many keys per range there (many_split)
constexpr int kTileSms = 152;          // items of one round of the many-rows kernel: a CTA on each SM
// e4m3 caches: weights become fp16 with 2^7 for the running maximum.  They exceed it by up to 2^8 before it is raised, and
// 2^15 is fp16's last whole binade; downwards each is held to 2^-11 of itself until 2^-21 of the largest, and to 2^-32 of
// the largest below.  (With 1 for the maximum, keys 2^24 below one whose value is small lost a fifth of their sum.)
constexpr float kLiftE4M3 = 7.f;
constexpr float kLog2eP = 1.4426950408889634f, kLn2P = 0.69314718055994531f;

struct Plan;

struct PagedParams {
    CUtensorMap tm_k, tm_v;        // [num_pages * Hkv][page_size][D], boxes of min(page_size, tile) rows
    CUtensorMap tm_q;              // many rows: [T][Hq][D]
    dash_kv_cache c;
    const __nv_bfloat16* q;
    long long q_t, q_h, table_stride;
    const int32_t *table, *lens, *cu_q;
    __nv_bfloat16* o;
    float* lse;
    float* part_o;                 // [rows of split sequences][D]
    float2* part_ml;               // (m, l) of each
    long long max_rows;            // rows that part_o and part_ml hold
    int* counter;                  // many rows: next item
    Plan* plan;                    // many rows: the launch's plan
    unsigned long long timeout_ns;
    int b0, nb;                    // the launch's sequences
    int max_pages, B, T, Hq, G, max_q, causal, window, page_shift;
    uint32_t over_G, over_Hkv;     // reciprocals (quick_div)
    float scale_log2e;
};

struct Seq {
    int first, n, len;             // n = 0: nothing to do
};

// x / d for launch constants d: floor(2^32 / d) + 1 times x, over 2^32, is exact while x * d < 2^32; 0 stands for no such
// number (d = 1, or too large).  A division costs some 80 cycles of latency, and an item took six.
inline uint32_t reciprocal(int d) { return d > 1 && d <= 4096 ? (uint32_t)((1ull << 32) / (unsigned)d) + 1u : 0u; }
__device__ __forceinline__ int quick_div(int x, int d, uint32_t over) {
    return over ? (int)__umulhi((uint32_t)x, over) : d == 1 ? x : x / d;
}

// What the device alone knows about sequence b, checked; report: this thread reports what is wrong.
__device__ __forceinline__ Seq load_seq(const PagedParams& p, int b, bool report) {
    const long long cap = (long long)p.max_pages * p.c.page_size;
    int c0, c1;
    if (p.cu_q) {
        c0 = p.cu_q[b];
        c1 = p.cu_q[b + 1];
    } else {
        const int n = p.T / p.B;
        c0 = b * n;
        c1 = c0 + n;
    }
    const int len = p.lens[b];
    Seq s{c0, c1 - c0, len};
    if (c0 < 0 || c1 < c0 || c1 > p.T) {
        if (report) serve_error(DASH_ERR_PAGE, kOpAttn, b, c0 < 0 ? c0 : c1, p.T);
        s.n = 0;
    } else if (s.n > p.max_q) {
        if (report) serve_error(DASH_ERR_PAGE, kOpAttn, b, s.n, p.max_q);
        s.n = 0;
    } else if (len < 0 || len > cap) {
        if (report) serve_error(DASH_ERR_PAGE, kOpAttn, b, len, cap);
        s.n = 0;
    }
    return s;
}

// The few-rows class ends where reading the pages once for every 8 rows (from L2 after the first time) costs more than
// the many-rows kernel's 128-row products, mostly of rows that do not exist.  Measured (us; 16 sequences to 5000 keys,
// Hq = 32, Hkv = 8; 5 tokens = 20 rows, 8 tokens = 32 rows, 12 tokens = 48 rows), few against many: e4m3, D = 128:
// 60 / 76 / 109 against 95 / 98 / 98; D = 64: 43 / 55 / 73 against 62 / 63 / 65; bf16, D = 128: 74 / 95 / 132 against
// 56 / 58 / 61.
__host__ __device__ inline int few_most(int type) { return type == DASH_CACHE_E4M3 ? kFewMost : 16; }
__host__ __device__ inline bool few_rows(int n, int G, int type) { return (long long)n * G <= few_most(type); }

// Keys [lo, hi) that rows i0 .. i1 - 1 (tokens) of a sequence see.
__device__ __forceinline__ void seen_keys(const PagedParams& p, const Seq& s, int i0, int i1, int& lo, int& hi) {
    const int p0 = s.len - s.n + i0, p1 = s.len - s.n + i1;   // first position, one past the last
    hi = p.causal ? (p1 < 0 ? 0 : p1) : s.len;
    lo = (p.window && p0 + 1 > p.window) ? p0 + 1 - p.window : 0;
}

// The most key ranges of a sequence: the least number of rounds of all workers (at most 4) that one sequence's items
// nearly fill (to 31/32), so that a long sequence alone, and any number of them, leave few workers idle in the last round.
__host__ __device__ inline int few_max_splits(int workers, int heads) {
    int best = 1, best_items = 0, best_rounds = 1;
    for (int rounds = 1; rounds <= 4; ++rounds) {
        const int ns = workers * rounds / heads, items = ns * heads;
        if (ns < 1) continue;
        if (items * best_rounds > best_items * rounds) best = ns, best_items = items, best_rounds = rounds;
        if (items * 32 >= workers * rounds * 31) break;
    }
    return best;
}

__host__ __device__ inline int few_parts(int n, int G) { return (n * G + kFewRows - 1) / kFewRows; }

// Groups that work through the items: three of a CTA, or two (launch_few).
__host__ __device__ inline int few_workers(int D, int type) {
    return type == DASH_CACHE_E4M3 || D == 64 ? kFewWorkers3 : kFewWorkers;
}

// Key ranges of a sequence: `tiles` stages cut into ns ranges of st stages.  A range costs its start, its queries and its
// share of the join: short ones serve a lone sequence, long ones a batch, whose other sequences fill the GPU.  Measured
// (us; Hq = 32, Hkv = 8, D = 128; 1000 bf16 keys, 4000 and 8192 e4m3 keys alone, 64 ragged e4m3 sequences to 8192, 256 to
// 2000), ranges of at least 2 stages: 8.3 11.8 15.1 136 149; 4: 9.6 10.3 13.2 107 117; 8: 12.5 11.7 12.7 99 109; 16: 17.6
// 15.5 16.3 97 111; growing with the sequence, as here: 8.5 11.9 12.7 100 129.
__host__ __device__ inline void few_split(int tiles, int workers, int heads, int& ns, int& st) {
    const int most = tiles <= kFewWholeTiles ? 1 : few_max_splits(workers, heads);
    const int least = tiles >= 64 ? 8 : tiles > 16 ? (tiles + 7) / 8 : 2;
    st = (tiles + most - 1) / most;
    st = st < least ? least : st;
    ns = (tiles + st - 1) / st;
    ns = ns < 1 ? 1 : ns;
}

// The most that few_split gives for up to `tiles` stages.
__host__ inline long long few_most_ranges(long long tiles, int workers, int Hkv) {
    const long long by_len = tiles <= kFewWholeTiles ? 1 : tiles < 16 ? (tiles + 1) / 2 : tiles < 64 ? 8 : (tiles + 7) / 8;
    const long long most = few_max_splits(workers, Hkv);
    return by_len < most ? by_len : most;
}

// The launch's plan in shared memory: sequences, and running counts.
struct Plan {
    Seq seq[kMaxSeqs];
    int items[kMaxSeqs + 1];   // items of the class before each sequence
    int rows[kMaxSeqs + 1];    // partial rows before each sequence (both classes)
    int st[kMaxSeqs];          // few rows: stages of a key range
    int warp_sum[3][16];
};

struct Cut {
    int lo, hi;                // keys seen by any row (few rows), tiles of them
    int tiles, ns, st;
    int items;                 // items of the sequence
    int parts;                 // few rows: items that share a head and a key range
};

__device__ __forceinline__ Cut cut_few(const PagedParams& p, const Seq& s) {
    Cut c;
    seen_keys(p, s, 0, s.n, c.lo, c.hi);
    c.tiles = c.hi > c.lo ? (c.hi - 1) / kFewKeys - c.lo / kFewKeys + 1 : 0;
    c.parts = few_parts(s.n, p.G);
    few_split(c.tiles, few_workers(p.c.D, p.c.type), p.c.Hkv * c.parts, c.ns, c.st);
    c.items = p.c.Hkv * c.ns * c.parts;
    return c;
}

// Many rows: a sequence of `full` (row tile, head) pairs over `tiles` key tiles alone on the GPU is cut into as many key
// ranges as one round of all SMs holds; never into a second round that is part empty: 256 and 512 new tokens over 8192
// and 16384 keys (Hq = 32, Hkv = 8, D = 128) took 67 and 160 us with as many items as fill two rounds, 49 and 122 us so.
// And only where that gains a sixteenth, in twentieths of a microsecond (a key tile 1.8 us, an item 3 us, joining 3 us and
// 0.05 us for each item): to a batch, which fills the GPU anyway, ranges are a cost.
// The least range likewise (us; 1, 16 and 64 sequences of 5 tokens over 5000 or to 5000 bf16 keys, 40 e4m3 tokens over 929):
// 512 keys 19.5 55.0 153 38, 768 keys 19.1 55.3 145 38, 1024 keys 22.6 54.1 142 44.
__host__ __device__ inline int many_split(int tiles, long long full) {
    const int most = (tiles + kTileSplitKeys / 128 - 1) / (kTileSplitKeys / 128);
    if (most <= 1 || 2 * full > kTileSms) return 1;
    const int want = kTileSms / (int)full, ns = want < most ? want : most;
    const int split = (tiles + ns - 1) / ns * 36 + 60 + 60 + (int)full * ns, whole = tiles * 36 + 60;
    return 16 * split < 15 * whole ? ns : 1;
}

// Key ranges of whole 128-key tiles of the sequence; row tiles of kTileRows rows.
__device__ __forceinline__ Cut cut_many(const PagedParams& p, const Seq& s, int tokens_per_tile) {
    Cut c;
    seen_keys(p, s, 0, s.n, c.lo, c.hi);
    c.tiles = c.hi > c.lo ? (c.hi - 1) / 128 - c.lo / 128 + 1 : 0;
    const int row_tiles = (s.n + tokens_per_tile - 1) / tokens_per_tile;
    const long long full = (long long)row_tiles * p.c.Hkv;
    c.ns = many_split(c.tiles, full);
    c.st = (c.tiles + c.ns - 1) / c.ns;
    c.ns = c.st > 0 ? (c.tiles + c.st - 1) / c.st : 1;
    c.items = (int)full * c.ns;
    return c;
}

// Tokens of one item of the many-rows kernel: two matrix tiles of 128 / G tokens.
__host__ __device__ inline int tokens_per_item(int G) { return 2 * (128 / G); }

// Fills plan (shared memory) for the launch's sequences: items of the few-rows class, and partial rows of both; `many`, if
// not null, is the same in global memory with the items of the many-rows class.  All threads of the block call it; at
// most 16 warps, at least kMaxSeqs / 2 threads.  Ends with a barrier.
__device__ __forceinline__ void make_plan(const PagedParams& p, Plan& plan, bool report, Plan* many) {
    const int per = (p.nb + (int)blockDim.x - 1) / (int)blockDim.x;
    const int t0 = (int)threadIdx.x * per;
    constexpr int kPer = 2;
    Seq seq[kPer];
    int count[kPer][3], st[kPer], own[3] = {0, 0, 0};   // items of few and of many rows, partial rows
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        count[k][0] = count[k][1] = count[k][2] = st[k] = 0;
        if (k >= per || t0 + k >= p.nb) continue;
        seq[k] = load_seq(p, p.b0 + t0 + k, report);
        if (seq[k].n == 0) continue;
        const bool f = few_rows(seq[k].n, p.G, p.c.type);
        const Cut c = f ? cut_few(p, seq[k]) : cut_many(p, seq[k], tokens_per_item(p.G));
        st[k] = c.st;
        count[k][0] = f ? c.items : 0;
        count[k][1] = f ? 0 : c.items;
        count[k][2] = c.ns > 1 ? seq[k].n * p.Hq * c.ns : 0;
#pragma unroll
        for (int x = 0; x < 3; ++x) own[x] += count[k][x];
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
    int sum[3] = {own[0], own[1], own[2]};
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const int v = __shfl_up_sync(0xffffffffu, sum[x], d);
            if (lane >= d) sum[x] += v;
        }
    if (lane == 31) {
#pragma unroll
        for (int x = 0; x < 3; ++x) plan.warp_sum[x][warp] = sum[x];
    }
    __syncthreads();
    int all[3] = {0, 0, 0};
#pragma unroll
    for (int x = 0; x < 3; ++x) sum[x] -= own[x];
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            const int v = plan.warp_sum[x][w];
            all[x] += v;
            if (w < warp) sum[x] += v;
        }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = t0 + k;
        if (k >= per || i >= p.nb) continue;
        plan.seq[i] = seq[k];
        plan.st[i] = st[k];
        plan.items[i] = sum[0];
        plan.rows[i] = sum[2];
        if (many) {
            many->seq[i] = seq[k];
            many->items[i] = sum[1];
            many->rows[i] = sum[2];
        }
#pragma unroll
        for (int x = 0; x < 3; ++x) sum[x] += count[k][x];
    }
    if (threadIdx.x == 0) {
        // (the host's bound holds for every cu_q that does not decrease; a row past it is not written, and its outputs neither)
        if (report && all[2] > p.max_rows) serve_error(DASH_ERR_SCRATCH, kOpAttn, p.b0, all[2], p.max_rows);
        plan.items[p.nb] = all[0];
        plan.rows[p.nb] = all[2];
        if (many) {
            many->items[p.nb] = all[1];
            many->rows[p.nb] = all[2];
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Page of key j of sequence b, checked: a bad entry is reported and read as page 0.
__device__ __forceinline__ int checked_page(const PagedParams& p, int b, int entry) {
    const int page = p.table[(long long)b * p.table_stride + entry];
    if (page < 0 || page >= p.c.num_pages) {
        serve_error(DASH_ERR_PAGE, kOpAttn, b, page, p.c.num_pages);
        return 0;
    }
    return page;
}

// Starts as the kernel before it in the stream ends, for which it waits itself (wait_dependency).
inline int launch_after(void (*kernel)(const PagedParams), unsigned grid, unsigned threads, size_t smem, const PagedParams& p,
                        cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

int launch_paged_many(const PagedParams& p, int max_items, cudaStream_t s);   // dash_paged_tile.cu

}  // namespace dash
