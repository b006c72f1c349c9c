// dash_paged_tile.cu -- attention over a paged cache for sequences with many
// rows (n * G > 16).
//
// One warp per (token, query head), its keys one after another with a running
// maximum m and sum l of the softmax:
//   m' = max(m, s),  l = l 2^(m - m') + 2^(s - m'),  o = o 2^(m - m') + 2^(s - m') v
// (scores in units of log2), o / l at the end.
#include <math.h>

#include "dash_internal.h"
#include "dash_paged.cuh"

namespace dash {

namespace {

template <int D, bool kE4M3>
__global__ void __launch_bounds__(256) paged_row_kernel(const __grid_constant__ PagedParams p) {
    constexpr int E = D / 32;   // values of a vector per lane
    const int lane = threadIdx.x & 31;
    const long long w = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
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
    } else {
        b = row / (p.T / p.B);
    }
    const Seq q0 = load_seq(p, b, false);
    first = q0.first;
    n = q0.n;
    if (first < 0 || row - first >= n || row < first || few_rows(n, p.G) || b < p.b0 || b >= p.b0 + p.nb) return;
    long long len = q0.len;
    const long long pos = len - n + (row - first);
    long long end = p.causal ? pos + 1 : len, begin = 0;
    if (p.window && pos + 1 > p.window) begin = pos + 1 - p.window;
    float q[E], o[E];
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[row * p.q_t + h * p.q_h + lane * E + e]) * p.scale_log2e;
        o[e] = 0.f;
    }
    const int hk = h / p.G;
    float m = -INFINITY, l = 0.f;
    for (long long j = begin; j < end; ++j) {
        const int page = checked_page(p, b, (int)(j / p.c.page_size));
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

int take_error_tile(int* out5) { return take_serve_error(out5); }

int launch_paged_many(const PagedParams& p, int, cudaStream_t s) {
    const unsigned blocks = (unsigned)(((long long)p.T * p.Hq + 7) / 8);
    if (p.c.type == DASH_CACHE_E4M3) {
        if (p.c.D == 64) paged_row_kernel<64, true><<<blocks, 256, 0, s>>>(p);
        else paged_row_kernel<128, true><<<blocks, 256, 0, s>>>(p);
    } else {
        if (p.c.D == 64) paged_row_kernel<64, false><<<blocks, 256, 0, s>>>(p);
        else paged_row_kernel<128, false><<<blocks, 256, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // namespace dash
