// dash_paged.cu -- attention of the newest tokens of each sequence over its
// paged key/value cache (dash_attn_paged).
//
// One warp per (token, query head), its keys one after another with a running
// maximum m and sum l of the softmax:
//   m' = max(m, s),  l = l 2^(m - m') + 2^(s - m'),  o = o 2^(m - m') + 2^(s - m') v
// (scores in units of log2), o / l at the end.
#include <math.h>

#include "dash_internal.h"
#include "dash_serve.cuh"

namespace dash {

namespace {

constexpr float kLog2eP = 1.4426950408889634f, kLn2P = 0.69314718055994531f;

struct PagedParams {
    dash_kv_cache c;
    const __nv_bfloat16* q;
    long long q_t, q_h, table_stride;
    const int32_t *table, *lens, *cu_q;
    __nv_bfloat16* o;
    float* lse;
    int max_pages, B, T, Hq, max_q, causal, window;
};

template <int D, bool kE4M3>
__global__ void __launch_bounds__(256) paged_row_kernel(const __grid_constant__ PagedParams p) {
    constexpr int E = D / 32;   // values of a vector per lane
    const int lane = threadIdx.x & 31;
    const long long w = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
    const long long cap = (long long)p.max_pages * p.c.page_size;
    if (blockIdx.x == 0)   // what the host cannot see
        for (int b = threadIdx.x; b < p.B; b += 256) {
            const long long len = p.lens[b];
            if (len < 0 || len > cap) serve_error(DASH_ERR_PAGE, kOpAttn, b, len, cap);
            if (p.cu_q) {
                const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
                if (c0 < 0 || c1 < c0 || c1 > p.T) serve_error(DASH_ERR_PAGE, kOpAttn, b, c0 < 0 ? c0 : c1, p.T);
                if (c1 - c0 > p.max_q) serve_error(DASH_ERR_PAGE, kOpAttn, b, c1 - c0, p.max_q);
            }
        }
    const int row = (int)(w / p.Hq), h = (int)(w % p.Hq);
    if (row >= p.T) return;
    int b, first, n;
    if (p.cu_q) {
        int lo = 0, hi = p.B;   // the last b with cu_q[b] <= row
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (p.cu_q[mid] <= row ? lo : hi) = mid;
        }
        b = lo;
        first = p.cu_q[b];
        n = p.cu_q[b + 1] - first;
    } else {
        n = p.T / p.B;
        b = row / n;
        first = b * n;
    }
    if (first < 0 || row - first >= n || row < first) return;
    long long len = p.lens[b];
    len = len < 0 ? 0 : len > cap ? cap : len;
    const long long pos = len - n + (row - first);
    long long end = p.causal ? pos + 1 : len, begin = 0;
    if (p.window && pos + 1 > p.window) begin = pos + 1 - p.window;
    float q[E], o[E];
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[row * p.q_t + h * p.q_h + lane * E + e]) * (kLog2eP / sqrtf((float)D));
        o[e] = 0.f;
    }
    const int hk = h / (p.Hq / p.c.Hkv);
    float m = -INFINITY, l = 0.f;
    for (long long j = begin; j < end; ++j) {
        int page = p.table[b * p.table_stride + j / p.c.page_size];
        if (page < 0 || page >= p.c.num_pages) {
            if (lane == 0) serve_error(DASH_ERR_PAGE, kOpAttn, b, page, p.c.num_pages);
            page = 0;
        }
        const long long cell = ((long long)page * p.c.Hkv + hk) * p.c.page_size + j % p.c.page_size;
        float s = 0.f, v[E];
        for (int e = 0; e < E; e += 2) {
            const long long at = cell * D + lane * E + e;
            float2 k2, v2;
            if (kE4M3) {
                k2 = unpack_e4m3x2(*reinterpret_cast<const uint16_t*>((const uint8_t*)p.c.k + at));
                v2 = unpack_e4m3x2(*reinterpret_cast<const uint16_t*>((const uint8_t*)p.c.v + at));
            } else {
                k2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>((const __nv_bfloat16*)p.c.k + at));
                v2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>((const __nv_bfloat16*)p.c.v + at));
            }
            s += q[e] * k2.x + q[e + 1] * k2.y;
            v[e] = v2.x, v[e + 1] = v2.y;
        }
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        float vs = 1.f;
        if (kE4M3) {
            s *= p.c.k_scale[cell];
            vs = p.c.v_scale[cell];
        }
        const float m2 = fmaxf(m, s), a = exp2f(m - m2), w2 = exp2f(s - m2);
        l = l * a + w2;
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + w2 * vs * v[e];
        m = m2;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < E; ++e) p.o[((long long)row * p.Hq + h) * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
    if (p.lse && lane == 0) p.lse[(long long)row * p.Hq + h] = l > 0.f ? (m + log2f(l)) * kLn2P : -INFINITY;
}

}  // namespace

int take_error_paged(int* out5) { return take_serve_error(out5); }

}  // namespace dash

using namespace dash;

extern "C" int dash_attn_paged_workspace(int B, int T, int Hq, int Hkv, int D, int max_q, int64_t max_kv,
                                         size_t* bytes) {
    if (!bytes || B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hq / Hkv > 128 || (D != 64 && D != 128) ||
        max_q < 0 || max_kv < 0)
        return DASH_ERR_ARG;
    *bytes = 0;
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
        !serve_strides(q_stride_t, q_stride_h))
        return DASH_ERR_ARG;
    size_t need = 0;
    if ((rc = dash_attn_paged_workspace(B, T, Hq, cache->Hkv, cache->D, max_q, (int64_t)max_pages * cache->page_size,
                                        &need)))
        return rc;
    if (B == 0 || T == 0) return DASH_OK;
    if (!serve_aligned(q) || !serve_aligned(o) || ((uintptr_t)lse & 3u) || !kv_lens || ((uintptr_t)kv_lens & 3u) ||
        ((uintptr_t)cu_q & 3u) || ((uintptr_t)block_table & 3u) || (max_pages > 0 && !block_table) ||
        (!cu_q && (T % B || T / B > max_q)) || (need && !serve_aligned(workspace)))
        return DASH_ERR_ARG;
    if (workspace_bytes < need) return DASH_ERR_SCRATCH;
    if ((rc = serve_check_device())) return rc;
    PagedParams prm;
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
    prm.max_pages = max_pages;
    prm.B = B;
    prm.T = T;
    prm.Hq = Hq;
    prm.max_q = max_q;
    prm.causal = causal;
    prm.window = window;
    const long long blocks = ((long long)T * Hq + 7) / 8;
    if (blocks > 0x7fffffffll) return DASH_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (cache->type == DASH_CACHE_E4M3) {
        if (cache->D == 64) paged_row_kernel<64, true><<<(unsigned)blocks, 256, 0, s>>>(prm);
        else paged_row_kernel<128, true><<<(unsigned)blocks, 256, 0, s>>>(prm);
    } else {
        if (cache->D == 64) paged_row_kernel<64, false><<<(unsigned)blocks, 256, 0, s>>>(prm);
        else paged_row_kernel<128, false><<<(unsigned)blocks, 256, 0, s>>>(prm);
    }
    return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}
