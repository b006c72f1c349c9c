// dash_serve.cuh -- what the rotary, cache and paged attention kernels share:
// the per-device error record, vector conversions between bf16 / e4m3 and
// fp32, and argument checks of their entry points.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dash.h"

namespace dash {

enum ServeOp : int { kOpWrite = 1, kOpRead = 2, kOpAttn = 3 };

// First error of this translation unit's kernels on the device since it was
// last cleared: code, then info[4]; word 7 is claimed by the thread that writes
// them, and the code comes last, so that another stream's kernel is never seen
// half way.  A file-scope word needs no allocation, so the calls can be
// captured, and it stays valid for every replay.
static __device__ int g_serve_error[8];

static __device__ __noinline__ void serve_error(int code, int op, long long where, long long got, long long bound) {
    if (atomicCAS(&g_serve_error[7], 0, 1) == 0) {
        g_serve_error[1] = op;
        g_serve_error[2] = (int)where;
        g_serve_error[3] = (int)(got > 0x7fffffffll ? 0x7fffffffll : got < -0x80000000ll ? -0x80000000ll : got);
        g_serve_error[4] = (int)(bound > 0x7fffffffll ? 0x7fffffffll : bound);
        __threadfence();
        atomicExch(&g_serve_error[0], code);
    }
}

// This translation unit's record: read (out5[0] = DASH_OK: none), or cleared, which only one that was read is.
static inline int serve_record(int* out5, bool clear) {
    const int zero[8] = {0};
    if (clear) return cudaMemcpyToSymbol(g_serve_error, zero, sizeof(zero)) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
    int h[8] = {0};
    // (a code once seen, its info is there: the first copy may have read it too early)
    for (int i = 0; i < 2 && (i == 0 || h[0]); ++i)
        if (cudaMemcpyFromSymbol(h, g_serve_error, sizeof(h)) != cudaSuccess) return DASH_ERR_CUDA;
    for (int i = 0; i < 5; ++i) out5[i] = h[i];
    return DASH_OK;
}

// ---------------------------------------------------------------- conversions
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void unpack_bf16(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// Four fp32 values to four e4m3 codes (round to nearest even, saturating), lowest first.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Two e4m3 codes (exact).
__device__ __forceinline__ float2 unpack_e4m3x2(uint16_t codes) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(codes));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h2));
    return make_float2(lo, hi);
}
__device__ __forceinline__ void unpack_e4m3x8(const uint2& u, float (&x)[8]) {
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_e4m3x2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// ---------------------------------------------------------------- host checks
inline bool serve_aligned(const void* p) { return p && (((uintptr_t)p) & 15u) == 0; }
inline bool serve_strides(int64_t a, int64_t b) { return a >= 0 && b >= 0 && a % 8 == 0 && b % 8 == 0; }

inline int check_cache(const dash_kv_cache* c) {
    if (!c || !serve_aligned(c->k) || !serve_aligned(c->v)) return DASH_ERR_ARG;
    if (c->type != DASH_CACHE_BF16 && c->type != DASH_CACHE_E4M3) return DASH_ERR_ARG;
    if (c->type == DASH_CACHE_E4M3 ? (!serve_aligned(c->k_scale) || !serve_aligned(c->v_scale))
                                   : (c->k_scale || c->v_scale))
        return DASH_ERR_ARG;
    if (c->num_pages <= 0 || c->Hkv <= 0 || (c->D != 64 && c->D != 128)) return DASH_ERR_ARG;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return DASH_ERR_ARG;
    if ((long long)c->num_pages * c->Hkv >= (1ll << 31)) return DASH_ERR_ARG;
    return DASH_OK;
}

int serve_check_device();   // DASH_OK on sm_103 (dash_rope.cu)
// Records of the translation units (serve_record).
int error_rope(int* out5, bool clear);
int error_paged(int* out5, bool clear);
int error_tile(int* out5, bool clear);

}  // namespace dash
