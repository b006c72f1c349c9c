// dash_pages.cu -- the pages of a paged cache: rows of a block table forked and
// dropped (dash_pages_fork), pages taken for new tokens (dash_pages_extend),
// the pages in use moved to the front of the pool (dash_pages_compact), and the
// cells that go with it copied (dash_kv_copy).
//
// The state is the caller's: the block table, the rows' lengths and refs[p],
// the number of table entries that hold page p (0: free).  Nothing here asks the
// host, so a decoding step that forks, extends and copies can be captured.
//
// What bounds them.  Tables and counts are small (64 rows of 512 entries and
// 65536 pages are 0.4 MB, a tenth of a microsecond of memory), so the first three
// are latency: a launch and a few dependent trips to memory.  Finding free pages
// in ascending order is a scan over the whole pool; one cluster of 8 CTAs does
// it in a single launch, each CTA its eighth of the pool, with counts exchanged
// through distributed shared memory and cluster barriers in place of a second
// and a third kernel (pools of up to 8192 pages: one CTA; pool_ctas).  The copy is
// memory bound: 601 MB in 98.6 us, 6.1 TB/s.
#include <string.h>

#include "dash_internal.h"
#include "dash_serve.cuh"

namespace dash {

namespace {

constexpr int kCluster = 8, kPoolThreads = 1024, kPoolTile = 4 * kPoolThreads;   // pages of a tile: four a thread
constexpr int kMaxRows = 4096;   // of dash_pages_extend: its rows lie in shared memory
constexpr long long kMostPairs = 1ll << 40;   // of dash_pages_fork: each old row looks at all parents (2^36 pairs take 60 ms)

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Each kernel here is started while the one before it in the stream ends (launch_next), waits for that one's end before it
// touches memory, and lets the next one start: two or three of them one after another are what a step launches.
__device__ __forceinline__ void take_turn() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
// All threads of the cluster; what they wrote before it, in shared or global memory, is seen after it.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same variable of CTA `rank` of the cluster.
__device__ __forceinline__ int remote_int(const int* p, uint32_t rank) {
    const uint32_t here = (uint32_t)__cvta_generic_to_shared(p);
    uint32_t there;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
    return v;
}

// Sum over the block's threads before this one, and over all of them.  `warps`: 32 words of shared memory; ends with a
// barrier.
template <typename T>
__device__ __forceinline__ T block_scan(T own, T* warps, T& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
    T sum = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    T mine = lane < n ? warps[lane] : T(0), w = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T v = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += v;
    }
    all = __shfl_sync(0xffffffffu, w, 31);
    const T before = __shfl_sync(0xffffffffu, w - mine, warp);
    __syncthreads();
    return before + sum - own;
}

struct PagesParams {
    const int32_t* table;
    int32_t* table_out;
    long long stride, stride_out;
    const int32_t *lens, *parents, *cu;
    int32_t *lens_out, *refs;
    const int32_t* refs_in;
    int64_t* slots;
    int32_t *positions, *copies, *counts, *rank;
    int rows, rows_out, max_pages, num_pages, page_size, page_shift, T;
};

__device__ __forceinline__ int pages_of(const PagesParams& p, int len) { return (len + p.page_size - 1) >> p.page_shift; }

// A row's length; one out of range is reported by the thread that asks for it, and counts as none.
__device__ __forceinline__ int checked_len(const PagesParams& p, int op, int row, int len, bool report) {
    const long long cap = (long long)p.max_pages << p.page_shift;
    if (len >= 0 && len <= cap) return len;
    if (report) serve_error(DASH_ERR_PAGE, op, row, len, cap);
    return 0;
}

// ---------------------------------------------------------------- fork
// Block i writes row i of the new table, and changes the counts of the pages of row i of the old one by its children
// less one: rows that go on as they are touch no count.
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ PagesParams p) {
    take_turn();
    const int i = blockIdx.x;
    if (i < p.rows_out) {
        int from = p.parents[i];
        if (from >= p.rows) {
            if (threadIdx.x == 0) serve_error(DASH_ERR_PAGE, kOpFork, i, from, p.rows);
            from = -1;
        }
        const int len = from < 0 ? 0 : checked_len(p, kOpFork, from, p.lens[from], threadIdx.x == 0);
        const int held = pages_of(p, len);
        for (int e = threadIdx.x; e < p.max_pages; e += blockDim.x) {
            int page = -1;
            if (e < held) {
                page = p.table[(long long)from * p.stride + e];
                if (page < 0 || page >= p.num_pages) serve_error(DASH_ERR_PAGE, kOpFork, from, page, p.num_pages);
            }
            p.table_out[(long long)i * p.stride_out + e] = page;
        }
        if (threadIdx.x == 0) p.lens_out[i] = len;
    }
    if (i < p.rows) {
        int children = 0;
        for (long long j0 = 0; j0 < p.rows_out; j0 += blockDim.x) {
            const long long j = j0 + threadIdx.x;
            children += __syncthreads_count(j < p.rows_out && p.parents[j] == i);
        }
        if (children == 1) return;
        const int held = pages_of(p, checked_len(p, kOpFork, i, p.lens[i], threadIdx.x == 0));
        for (int e = threadIdx.x; e < held; e += blockDim.x) {
            const int page = p.table[(long long)i * p.stride + e];
            if (page < 0 || page >= p.num_pages) {
                serve_error(DASH_ERR_PAGE, kOpFork, i, page, p.num_pages);
                continue;
            }
            const int was = atomicAdd(p.refs + page, children - 1);
            if (was + children - 1 < 0) serve_error(DASH_ERR_PAGE, kOpFork, i, was, children - 1);
        }
    }
}

// ---------------------------------------------------------------- extend
// Shared memory of the kernel: rows, and a hash table of the partly filled pages that rows go on in.
struct ExtendLayout {
    int rows, slots;   // hash slots: a power of two, at least twice the rows
    __host__ __device__ explicit ExtendLayout(int r) : rows(r), slots(64) {
        while (slots < 2 * r) slots *= 2;
    }
    __host__ __device__ int start() const { return 0; }                        // [rows + 1] pages needed by the rows before
    __host__ __device__ int len() const { return start() + rows + 1; }         // [rows]
    __host__ __device__ int cu() const { return len() + rows; }                // [rows + 1]
    __host__ __device__ int last() const { return cu() + rows + 1; }           // [rows] page to be copied from, or -1; -2: not extended
    __host__ __device__ int place() const { return last() + rows; }            // [rows] where its copy comes in the list
    __host__ __device__ int key() const { return place() + rows; }             // [slots]
    __host__ __device__ int count() const { return key() + slots; }            // [slots] rows that extend it
    __host__ __device__ int first() const { return count() + slots; }          // [slots] the first of them
    __host__ __device__ int words() const { return first() + slots; }
};

__global__ void __launch_bounds__(kPoolThreads) extend_kernel(const __grid_constant__ PagesParams p) {
    extern __shared__ int sm[];
    __shared__ int pool_free;
    __shared__ int scan_i[32];
    __shared__ long long scan_l[32];
    const ExtendLayout at(p.rows);
    int *const start = sm + at.start(), *const len = sm + at.len(), *const cu = sm + at.cu();
    int *const last = sm + at.last(), *const place = sm + at.place();
    int *const key = sm + at.key(), *const count = sm + at.count(), *const first = sm + at.first();
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const bool lead = rank == 0;
    const int tid = threadIdx.x, mask = at.slots - 1;
    take_turn();
    auto hash = [&](int page) { return (int)(((uint32_t)page * 2654435761u) >> 7) & mask; };

    // free pages of this CTA's part of the pool
    const int tiles = (p.num_pages + kPoolTile - 1) / kPoolTile, per = (tiles + (int)ctas - 1) / (int)ctas;
    const int t0 = min((int)rank * per, tiles), t1 = min(t0 + per, tiles);
    auto free_of = [&](int page0) -> unsigned {   // which of four pages are free
        unsigned m = 0;
        if (page0 + 4 <= p.num_pages) {
            const int4 r = *reinterpret_cast<const int4*>(p.refs + page0);
            m = (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3;
        } else {
            for (int k = 0; k < 4; ++k)
                if (page0 + k < p.num_pages && p.refs[page0 + k] == 0) m |= 1u << k;
        }
        return m;
    };
    int mine = 0;
    for (int t = t0; t < t1; ++t) mine += __popc(free_of(t * kPoolTile + 4 * tid));

    for (int s = tid; s < at.slots; s += kPoolThreads) key[s] = -1, count[s] = 0, first[s] = 0x7fffffff;
    for (int r = tid; r <= p.rows; r += kPoolThreads)
        cu[r] = p.cu ? p.cu[r] : p.rows ? r * (p.T / p.rows) : 0;
    __syncthreads();
    // rows: their lengths, and the partly filled page that a row goes on in
    for (int r = tid; r < p.rows; r += kPoolThreads) {
        const int l = p.lens[r], c0 = cu[r], c1 = cu[r + 1], n = c1 - c0;
        const long long cap = (long long)p.max_pages << p.page_shift;
        bool ok = true;
        int page = -1;
        if (c0 < 0 || n < 0 || c1 > p.T) {
            if (lead) serve_error(DASH_ERR_PAGE, kOpExtend, r, c0 < 0 ? c0 : c1, p.T);
            ok = false;
        } else if (l < 0 || l + (long long)n > cap) {
            if (lead) serve_error(DASH_ERR_PAGE, kOpExtend, r, l < 0 ? l : l + (long long)n, cap);
            ok = false;
        } else if (n > 0 && (l & (p.page_size - 1))) {
            page = p.table[(long long)r * p.stride + (l >> p.page_shift)];
            if (page < 0 || page >= p.num_pages) {
                if (lead) serve_error(DASH_ERR_PAGE, kOpExtend, r, page, p.num_pages);
                ok = false;
            } else if (p.refs[page] < 1) {   // held, and free: it may be another row's by the end of this call
                if (lead) serve_error(DASH_ERR_PAGE, kOpExtend, r, p.refs[page], 1);
                ok = false;
            } else {
                int s = hash(page);
                for (int was; (was = atomicCAS(key + s, -1, page)) != -1 && was != page;) s = (s + 1) & mask;
                atomicAdd(count + s, 1);
                atomicMin(first + s, r);
            }
        }
        len[r] = l;
        last[r] = ok ? page : -2;
    }
    __syncthreads();
    // A shared page is copied by every row that extends it; where nobody else holds it, by all but the first of them.  Where
    // it has fewer holders than that by its count, none of them goes on: the count would pass zero while others look for free
    // pages.
    // Needs and copies of the rows before, in one scan (of 48 and 16 bits: rows whose tokens overlap, as reported, may need more
    // pages than 32 bits count, and then get none).
    long long carry = 0;
    for (int r0 = 0; r0 < p.rows; r0 += kPoolThreads) {
        const int r = r0 + tid;
        long long own = 0;
        if (r < p.rows && last[r] != -2) {
            const int l = len[r], n = cu[r + 1] - cu[r];
            int copy = 0;
            if (last[r] >= 0) {
                int s = hash(last[r]);
                while (key[s] != last[r]) s = (s + 1) & mask;
                const int held = p.refs[last[r]];
                if (held < count[s]) {
                    if (lead) serve_error(DASH_ERR_PAGE, kOpExtend, r, held, count[s]);
                    last[r] = -2;
                } else {
                    copy = !(held == count[s] && first[s] == r);
                    if (!copy) last[r] = -1;
                }
            }
            if (last[r] != -2) own = (long long)(pages_of(p, l + n) - pages_of(p, l) + copy) | (long long)copy << 48;
        }
        long long all;
        const long long before = carry + block_scan(own, scan_l, all);
        if (r < p.rows) {
            start[r] = (int)before;
            place[r] = (int)(before >> 48);
        }
        carry += all;
    }
    const long long need = carry & 0xffffffffffffll;
    const int copies = (int)(carry >> 48);
    if (tid == 0) start[p.rows] = (int)need;
    int all_free;
    block_scan(mine, scan_i, all_free);
    if (tid == 0) pool_free = all_free;
    cluster_barrier();   // (from here on counts and tables change)
    int base = 0, total = 0;
    for (uint32_t r = 0; r < ctas; ++r) {
        const int v = remote_int(&pool_free, r);
        if (r < rank) base += v;
        total += v;
    }
    const bool enough = need <= total;
    if (!enough && lead && tid == 0) serve_error(DASH_ERR_NOMEM, kOpExtend, p.rows, need, total);
    if (lead && tid == 0) {
        p.counts[0] = enough ? copies : 0;
        p.counts[1] = enough ? (int)need : 0;
    }
    if (enough) {
        // the j-th free page goes to the row whose needs reach past j
        for (int t = t0; t < t1 && base < need; ++t) {
            const int page0 = t * kPoolTile + 4 * tid;
            const unsigned m = free_of(page0);
            int here;
            int j = base + block_scan(__popc(m), scan_i, here);
            base += here;
            for (int k = 0; k < 4 && j < need; ++k) {
                if (!(m >> k & 1)) continue;
                int lo = 0, hi = p.rows;   // the last row with start <= j
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (start[mid] <= j) lo = mid;
                    else hi = mid;
                }
                const int copy = last[lo] >= 0, nth = j - start[lo];
                const int entry = pages_of(p, len[lo]) + nth - copy;
                p.table_out[(long long)lo * p.stride + entry] = page0 + k;
                p.refs[page0 + k] = 1;
                if (copy && nth == 0) {
                    p.copies[2 * place[lo]] = last[lo];
                    p.copies[2 * place[lo] + 1] = page0 + k;
                    atomicSub(p.refs + last[lo], 1);
                }
                ++j;
            }
        }
    }
    cluster_barrier();   // tables are complete
    for (long long at_t = rank * kPoolThreads + tid; at_t < p.T; at_t += ctas * kPoolThreads) {
        const int t = (int)at_t;
        int lo = 0, hi = p.rows;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        long long slot = -1;
        int pos = 0;
        if (enough && p.rows > 0 && last[lo] != -2 && cu[lo] <= t && t < cu[lo + 1]) {
            pos = len[lo] + t - cu[lo];
            const int page = p.table_out[(long long)lo * p.stride + (pos >> p.page_shift)];
            slot = ((long long)page << p.page_shift) + (pos & (p.page_size - 1));
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
    if (enough && lead)
        for (int r = tid; r < p.rows; r += kPoolThreads)
            if (last[r] != -2) p.lens_out[r] = len[r] + cu[r + 1] - cu[r];
}

// ---------------------------------------------------------------- compact
// With L pages in use, the k-th of those from L on moves to the k-th free one below L.
__global__ void __launch_bounds__(kPoolThreads) compact_kernel(const __grid_constant__ PagesParams p) {
    __shared__ int pool_live, pool_below;
    __shared__ int scan[32];
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int tid = threadIdx.x;
    take_turn();
    const int tiles = (p.num_pages + kPoolTile - 1) / kPoolTile, per = (tiles + (int)ctas - 1) / (int)ctas;
    const int t0 = min((int)rank * per, tiles), t1 = min(t0 + per, tiles);
    auto counts_of = [&](int page0) -> int4 {
        int4 r = make_int4(0, 0, 0, 0);
        if (page0 + 4 <= p.num_pages) {
            r = *reinterpret_cast<const int4*>(p.refs_in + page0);
        } else {
            if (page0 < p.num_pages) r.x = p.refs_in[page0];
            if (page0 + 1 < p.num_pages) r.y = p.refs_in[page0 + 1];
            if (page0 + 2 < p.num_pages) r.z = p.refs_in[page0 + 2];
        }
        return r;
    };
    int mine = 0, all;
    for (int t = t0; t < t1; ++t) {
        const int4 r = counts_of(t * kPoolTile + 4 * tid);
        mine += (r.x != 0) + (r.y != 0) + (r.z != 0) + (r.w != 0);
    }
    block_scan(mine, scan, all);
    if (tid == 0) pool_live = all;
    cluster_barrier();
    int base = 0, live = 0;   // in use: before this CTA's part, and in all
    for (uint32_t r = 0; r < ctas; ++r) {
        const int v = remote_int(&pool_live, r);
        if (r < rank) base += v;
        live += v;
    }
    mine = 0;   // in use below `live`
    for (int t = t0; t < t1 && t * kPoolTile < live; ++t) {
        const int page0 = t * kPoolTile + 4 * tid;
        const int4 r = counts_of(page0);
        mine += (r.x != 0 && page0 < live) + (r.y != 0 && page0 + 1 < live) + (r.z != 0 && page0 + 2 < live) +
                (r.w != 0 && page0 + 3 < live);
    }
    block_scan(mine, scan, all);
    if (tid == 0) pool_below = all;
    cluster_barrier();
    int below = 0;
    for (uint32_t r = 0; r < ctas; ++r) below += remote_int(&pool_below, r);
    for (int t = t0; t < t1; ++t) {
        const int page0 = t * kPoolTile + 4 * tid;
        const int4 r4 = counts_of(page0);
        const int r[4] = {r4.x, r4.y, r4.z, r4.w};
        int here, seen = base + block_scan((r[0] != 0) + (r[1] != 0) + (r[2] != 0) + (r[3] != 0), scan, here);
        base += here;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = page0 + k;
            if (page >= p.num_pages) break;
            if (p.refs != p.refs_in) p.refs[page] = r[k];
            p.rank[page] = !r[k] ? -1 : page < live ? 0 : seen - below;   // which move takes it (-1: it was free)
            if (page >= live && r[k]) {
                p.copies[2 * (seen - below)] = page;
            } else if (page < live && !r[k]) {
                p.copies[2 * (page - seen) + 1] = page;
            }
            seen += r[k] != 0;
        }
    }
    cluster_barrier();
    const int moves = live - below;
    for (int i = (int)rank * kPoolThreads + tid; i < moves; i += (int)ctas * kPoolThreads) {
        const int from = p.copies[2 * i], to = p.copies[2 * i + 1];
        p.refs[to] = p.refs_in[from];
        p.refs[from] = 0;
    }
    if (rank == 0 && tid == 0) {
        p.counts[0] = moves;
        p.counts[1] = live;
    }
    cluster_barrier();   // (no CTA ends while others read its shared memory)
}

// The table with its pages renamed; blockIdx.y is the row.
__global__ void __launch_bounds__(256) rename_kernel(const __grid_constant__ PagesParams p) {
    take_turn();
    const int live = p.counts[1];
    for (long long r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const int held = pages_of(p, checked_len(p, kOpCompact, (int)r, p.lens[r], blockIdx.x == 0 && threadIdx.x == 0));
        for (int e = blockIdx.x * 256 + threadIdx.x; e < p.max_pages; e += gridDim.x * 256) {
            int page = p.table[r * p.stride + e];
            if (e < held) {
                const int k = page >= 0 && page < p.num_pages ? p.rank[page] : -1;
                if (k < 0) serve_error(DASH_ERR_PAGE, kOpCompact, r, page, p.num_pages);   // no such page, or a free one
                else if (page >= live) page = p.copies[2 * k + 1];
            }
            p.table_out[r * p.stride_out + e] = page;
        }
    }
}

// ---------------------------------------------------------------- copy
constexpr int kMostCaches = 64;        // of a launch
constexpr int kCopyThreads = 256, kCopyVectors = 8;
constexpr int kCopyChunk = kCopyThreads * kCopyVectors * 16;

struct CopyParams {
    uint8_t* base[kMostCaches][4];     // k, v, and their scales
    const int32_t *copies, *count;
    long long cells, scales;           // bytes of a page, and of its scales
    int caches, kinds, num_pages, most;
};

// Units of up to kCopyChunk bytes of one page, in the order of pairs.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
    take_turn();
    const int n = p.count ? min(max(*p.count, 0), p.most) : p.most;
    const int big = (int)((p.cells + kCopyChunk - 1) / kCopyChunk), small = (int)((p.scales + kCopyChunk - 1) / kCopyChunk);
    const int per_cache = 2 * big + (p.kinds > 2 ? 2 * small : 0);
    const long long units = (long long)n * p.caches * per_cache;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const long long of = u / per_cache;
        int part = (int)(u - of * per_cache);
        const int i = (int)(of / p.caches), cache = (int)(of - (long long)i * p.caches);
        const int from = p.copies[2ll * i], to = p.copies[2ll * i + 1];
        if (from < 0 || to < 0 || from >= p.num_pages || to >= p.num_pages) {
            if (threadIdx.x == 0 && part == 0 && cache == 0)
                serve_error(DASH_ERR_PAGE, kOpCopy, i, from < 0 || from >= p.num_pages ? from : to, p.num_pages);
            continue;
        }
        int kind = 0;
        if (part >= 2 * big) kind = 2, part -= 2 * big;
        const int pieces = kind ? small : big;
        if (part >= pieces) ++kind, part -= pieces;
        const long long bytes = kind < 2 ? p.cells : p.scales;
        const uint8_t* src = p.base[cache][kind] + from * bytes;
        uint8_t* dst = p.base[cache][kind] + to * bytes;
        const long long at = (long long)part * kCopyChunk + threadIdx.x * 16;
        uint4 w[kCopyVectors];
#pragma unroll
        for (int k = 0; k < kCopyVectors; ++k)
            if (at + k * kCopyThreads * 16 < bytes) w[k] = __ldcs(reinterpret_cast<const uint4*>(src + at + k * kCopyThreads * 16));
#pragma unroll
        for (int k = 0; k < kCopyVectors; ++k)
            if (at + k * kCopyThreads * 16 < bytes) __stcs(reinterpret_cast<uint4*>(dst + at + k * kCopyThreads * 16), w[k]);
    }
}

// ---------------------------------------------------------------- host
bool pool_ok(const int32_t* table, int64_t stride, const int32_t* lens, int rows, int max_pages, const int32_t* refs, int num_pages,
             int page_size) {
    if (rows < 0 || max_pages < 0 || stride < 0 || num_pages <= 0 || num_pages > (1 << 30)) return false;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return false;
    if ((long long)max_pages * page_size >= (1ll << 31) - 512 || (rows > 1 && stride < max_pages)) return false;
    return serve_aligned(refs) && (rows == 0 || (lens && !((uintptr_t)lens & 3u))) &&
           (rows == 0 || max_pages == 0 || (table && !((uintptr_t)table & 3u)));
}

PagesParams make_params(const int32_t* table, int64_t stride, const int32_t* lens, int rows, int max_pages, int32_t* refs, int num_pages,
                        int page_size) {
    PagesParams p;
    memset(&p, 0, sizeof(p));
    p.table = table;
    p.stride = stride;
    p.lens = lens;
    p.rows = rows;
    p.max_pages = max_pages;
    p.refs = refs;
    p.refs_in = refs;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.page_shift = __builtin_ctz((unsigned)page_size);
    return p;
}

// CTAs of the cluster that works through a pool.  A small one is one CTA's: its barriers cost less than the other seven bring.
// Measured (us; extend / compact, 160 rows), one CTA against eight: 64 pages 4.3 / 4.9 and 5.6 / 7.6, 2300 4.2 / 6.0 and
// 5.7 / 9.4, 8192 4.6 / 10.5 and 5.7 / 10.8, 16384 5.0 / 16.9 and 5.8 / 10.8, 65536 7.6 / 63 and 6.1 / 15.  (A thread's pages one
// after another, with one scan for all of them instead of one for each tile of 4096: 9.6 / 76 against 7.1 / 39 with 262144.)
unsigned pool_ctas(int num_pages) { return num_pages <= 2 * kPoolTile ? 1 : kCluster; }

template <typename P>
int launch_next(void (*kernel)(const P), dim3 grid, unsigned threads, size_t smem, const P& p, dash_stream_t stream, unsigned cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // namespace

int error_pages(int* out5, bool clear) { return serve_record(out5, clear); }

}  // namespace dash

using namespace dash;

extern "C" int dash_pages_fork(const int32_t* table, int64_t table_stride, const int32_t* lens, int rows, const int32_t* parents,
                               int32_t* table_out, int64_t out_stride, int32_t* lens_out, int rows_out, int max_pages, int32_t* refs,
                               int num_pages, int page_size, dash_stream_t stream) {
    if (!pool_ok(table, table_stride, lens, rows, max_pages, refs, num_pages, page_size) ||
        !pool_ok(table_out, out_stride, lens_out, rows_out, max_pages, refs, num_pages, page_size) ||
        (rows_out > 0 && (!parents || ((uintptr_t)parents & 3u))) ||
        (rows && rows_out && (lens == lens_out || (max_pages && table == table_out))) || (long long)rows * rows_out > kMostPairs)
        return DASH_ERR_ARG;
    if (rows == 0 && rows_out == 0) return DASH_OK;
    const int rc = serve_check_device();
    if (rc) return rc;
    PagesParams p = make_params(table, table_stride, lens, rows, max_pages, refs, num_pages, page_size);
    p.parents = parents;
    p.table_out = table_out;
    p.stride_out = out_stride;
    p.lens_out = lens_out;
    p.rows_out = rows_out;
    return launch_next(fork_kernel, dim3(rows > rows_out ? rows : rows_out), 256, 0, p, stream);
}

extern "C" int dash_pages_extend(int32_t* table, int64_t table_stride, int32_t* lens, int rows, int max_pages, int32_t* refs, int num_pages,
                                 int page_size, const int32_t* cu_new, int64_t* slots, int32_t* positions, int T, int32_t* copies,
                                 int32_t* counts, dash_stream_t stream) {
    if (!pool_ok(table, table_stride, lens, rows, max_pages, refs, num_pages, page_size) || rows > kMaxRows || T < 0 ||
        ((uintptr_t)cu_new & 3u) || (T > 0 && (!slots || ((uintptr_t)slots & 7u) || !positions || ((uintptr_t)positions & 3u))) ||
        (rows > 0 && (!copies || ((uintptr_t)copies & 3u))) || !counts || ((uintptr_t)counts & 3u) ||
        (!cu_new && (rows == 0 ? T > 0 : T % rows != 0)))
        return DASH_ERR_ARG;
    const int rc = serve_check_device();
    if (rc) return rc;
    PagesParams p = make_params(table, table_stride, lens, rows, max_pages, refs, num_pages, page_size);
    p.table_out = table;
    p.lens_out = lens;
    p.cu = cu_new;
    p.slots = slots;
    p.positions = positions;
    p.T = T;
    p.copies = copies;
    p.counts = counts;
    const int smem = ExtendLayout(rows).words() * 4;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DASH_ERR_CUDA;
    if (dev < 0 || dev >= 64) return DASH_ERR_DEVICE;
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ExtendLayout(kMaxRows).words() * 4) != cudaSuccess)
            return DASH_ERR_CUDA;
        ready[dev] = true;
    }
    const unsigned ctas = pool_ctas(num_pages);
    return launch_next(extend_kernel, dim3(ctas), kPoolThreads, smem, p, stream, ctas);
}

extern "C" int dash_pages_compact(const int32_t* table, int64_t table_stride, const int32_t* lens, int rows, int max_pages,
                                  const int32_t* refs, int num_pages, int page_size, int32_t* table_out, int64_t out_stride,
                                  int32_t* refs_out, int32_t* copies, int32_t* counts, void* workspace, size_t workspace_bytes,
                                  dash_stream_t stream) {
    if (!pool_ok(table, table_stride, lens, rows, max_pages, refs, num_pages, page_size) ||
        !pool_ok(table_out, out_stride, lens, rows, max_pages, refs_out, num_pages, page_size) ||
        (num_pages > 1 && (!copies || ((uintptr_t)copies & 3u))) || !counts || ((uintptr_t)counts & 3u) || !serve_aligned(workspace) ||
        (table == table_out && table_stride != out_stride))
        return DASH_ERR_ARG;
    if (workspace_bytes < (size_t)num_pages * 4) return DASH_ERR_SCRATCH;
    int rc = serve_check_device();
    if (rc) return rc;
    PagesParams p = make_params(table, table_stride, lens, rows, max_pages, refs_out, num_pages, page_size);
    p.refs_in = refs;
    p.table_out = table_out;
    p.stride_out = out_stride;
    p.copies = copies;
    p.counts = counts;
    p.rank = (int32_t*)workspace;
    const unsigned ctas = pool_ctas(num_pages);
    if ((rc = launch_next(compact_kernel, dim3(ctas), kPoolThreads, 0, p, stream, ctas)) || rows == 0 || max_pages == 0) return rc;
    const dim3 grid((unsigned)((max_pages + 255) / 256), (unsigned)(rows < 65535 ? rows : 65535));
    return launch_next(rename_kernel, grid, 256, 0, p, stream);
}

extern "C" int dash_kv_copy(const dash_kv_cache* caches, int n_caches, const int32_t* copies, const int32_t* n_copies, int max_copies,
                            dash_stream_t stream) {
    if (n_caches < 0 || max_copies < 0 || (n_caches > 0 && !caches) || ((uintptr_t)n_copies & 3u) ||
        (max_copies > 0 && (!copies || ((uintptr_t)copies & 3u))))
        return DASH_ERR_ARG;
    for (int i = 0; i < n_caches; ++i) {
        const int rc = check_cache(caches + i);
        if (rc) return rc;
        const dash_kv_cache &a = caches[i], &b = caches[0];
        if (a.type != b.type || a.num_pages != b.num_pages || a.page_size != b.page_size || a.Hkv != b.Hkv || a.D != b.D) return DASH_ERR_ARG;
    }
    if (n_caches == 0 || max_copies == 0) return DASH_OK;
    int rc = serve_check_device();
    if (rc) return rc;
    const dash_kv_cache& c = caches[0];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return DASH_ERR_CUDA;
    for (int i0 = 0; i0 < n_caches; i0 += kMostCaches) {
        CopyParams p;
        memset(&p, 0, sizeof(p));
        p.caches = n_caches - i0 < kMostCaches ? n_caches - i0 : kMostCaches;
        for (int i = 0; i < p.caches; ++i) {
            p.base[i][0] = (uint8_t*)caches[i0 + i].k;
            p.base[i][1] = (uint8_t*)caches[i0 + i].v;
            p.base[i][2] = (uint8_t*)caches[i0 + i].k_scale;
            p.base[i][3] = (uint8_t*)caches[i0 + i].v_scale;
        }
        p.cells = (long long)c.Hkv * c.page_size * cell_bytes(c.type, c.D);
        p.scales = (long long)c.Hkv * c.page_size * scale_bytes(c.type, c.D);
        p.kinds = p.scales ? 4 : 2;
        p.num_pages = c.num_pages;
        p.copies = copies;
        p.count = n_copies;
        p.most = max_copies;
        const long long units = (long long)max_copies * p.caches * 2 *
                                ((p.cells + kCopyChunk - 1) / kCopyChunk + (p.scales + kCopyChunk - 1) / kCopyChunk);
        if ((rc = launch_next(copy_kernel, dim3((unsigned)(units < 8ll * sms ? units : 8ll * sms)), kCopyThreads, 0, p, stream))) return rc;
    }
    return DASH_OK;
}
