// dash_rope.cu -- rotary positions and the paged cache's writer and reader
// (dash_rope, dash_kv_write, dash_kv_read; memory-bound kernels).
//
// Angles.  The rotation of pair i at position p is p * f_i radians modulo one
// turn.  p * f_i in fp32 would be off by p * f_i * 2^-24 (0.06 rad at a
// million), so the host turns f_i into the 64-bit fraction of a turn
// F_i = floor(f_i / 2pi * 2^64) mod 2^64, and the kernel forms p * F_i mod
// 2^64: an integer product whose wrap-around is the reduction modulo one turn.
// Its top 32 bits, as a signed number, are the angle in [-1/2, 1/2) turns; the
// error is p * 2^-64 turns from F_i (p * f_i * 2^-52 from the double f_i and its
// product with 1 / 2pi) and 2^-32 from the bits dropped, plus fp32's rounding of
// that fraction.  Two integer multiplies replace a
// 64-bit floating multiply and reduction.  The top bits also give the quadrant
// exactly, which leaves an angle of at most an eighth of a turn for a sine and a
// cosine of eleven operations together: polynomials in the angle's square that
// interpolate at Chebyshev nodes, off by 2^-24.2 at most (checked at two million
// angles).  The fast instructions (2^-21.4) are as quick, but an error in the
// rotation is an e4m3 cache's code off by a step wherever it crosses a boundary;
// sincospif took a third of the kernel's time with few heads.
//
// Work.  One thread owns 16 values of a vector as two chunks of 8, such that
// every chunk is one 16-byte access and the threads of a vector read
// consecutive chunks; for rotated values the chunks are 8j.. and rot/2 + 8j..,
// which hold both members of 8 pairs in either layout.  A thread forms the 8
// angles of its (token, chunk) once and uses them for a run of heads, four
// heads' loads at a time: these kernels only move data, and what limits them
// is how many bytes are on their way.
#include <math.h>

#include "dash_internal.h"
#include "dash_serve.cuh"

namespace dash {

namespace {

constexpr int kMaxPairs = 64;   // D / 2 at D = 128

struct Turns {
    unsigned long long f[kMaxPairs];   // fraction of a turn per position, times 2^64
    float factor;
    int rot, interleaved;
};

constexpr float kTurnHi = (float)1.4629180792671596e-9;                            // 2 pi / 2^32, in two parts
constexpr float kTurnLo = (float)(1.4629180792671596e-9 - (double)kTurnHi);

// cos and sin (times factor; sin negated for the inverse) of the 8 pairs of chunk j of a vector.
__device__ __forceinline__ void angles(const Turns& t, int j, long long pos, float sign, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // half layout: pairs 8j + e; interleaved: chunk 8j.. holds pairs 4j..4j+3, chunk rot/2 + 8j.. rot/4 + 4j..
        const int i = t.interleaved ? (e < 4 ? 4 * j + e : t.rot / 4 + 4 * j + e - 4) : 8 * j + e;
        const uint32_t turn = (uint32_t)(((unsigned long long)pos * t.f[i]) >> 32);
        const uint32_t quadrant = (turn + 0x20000000u) >> 30;                          // nearest quarter turn (mod 4)
        const float r = (float)(int)(turn - (quadrant << 30));
        const float x = fmaf(r, kTurnHi, r * kTurnLo), z = x * x;   // radians
        const float s0 = fmaf(x * z, fmaf(fmaf(-1.958784123e-4f, z, 8.332747966e-3f), z, -1.666666418e-1f), x);
        const float c0 = fmaf(fmaf(fmaf(fmaf(2.454789137e-5f, z, -1.388830249e-3f), z, 4.166666418e-2f), z, -0.5f), z, 1.f);
        const float s = (quadrant & 1u) ? c0 : s0, c = (quadrant & 1u) ? s0 : c0;
        cs[e] = ((quadrant + 1u) & 2u) ? -c * t.factor : c * t.factor;
        sn[e] = (quadrant & 2u) ? -s * (t.factor * sign) : s * (t.factor * sign);
    }
}

__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8],
                                       int interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = a[2 * e], y = a[2 * e + 1], u = b[2 * e], w = b[2 * e + 1];
            a[2 * e] = x * cs[e] - y * sn[e];
            a[2 * e + 1] = y * cs[e] + x * sn[e];
            b[2 * e] = u * cs[e + 4] - w * sn[e + 4];
            b[2 * e + 1] = w * cs[e + 4] + u * sn[e + 4];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = a[e], y = b[e];
            a[e] = x * cs[e] - y * sn[e];
            b[e] = y * cs[e] + x * sn[e];
        }
    }
}

// Where the two chunks of thread `unit` (of D / 16) start in a vector.
__device__ __forceinline__ void chunks(int unit, int rot, int& c0, int& c1) {
    const int ru = rot / 16;
    if (unit < ru) {
        c0 = 8 * unit;
        c1 = rot / 2 + 8 * unit;
    } else {
        c0 = rot + 16 * (unit - ru);
        c1 = c0 + 8;
    }
}

// 8 values as they lie in memory, and in fp32.
template <bool kF32>
struct Raw8 {
    uint4 w[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, long long at) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(base) + at * (kF32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) w[i] = __ldcs(p + i);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if (kF32) {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[kF32].x, w[kF32].y, w[kF32].z, w[kF32].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
        } else {
            unpack_bf16(w[0], x);
        }
    }
};
template <bool kF32>
__device__ __forceinline__ void store8(void* base, long long at, const float (&x)[8]) {
    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(base) + at * (kF32 ? 4 : 2));
    if (kF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            p[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
    } else {
        *p = pack_bf16x8(x);
    }
}

// ---------------------------------------------------------------- rope
struct RopeParams {
    dash_heads x[2], y[2];
    const int32_t* positions;
    long long pos_stride_b;
    Turns turns;
    float sign;
    int B, S, per;   // per: heads of a block
};

// Heads h0 .. h1 - 1 of one tensor, this thread's two chunks of each (at offsets c0, c1 from the vectors' start).
template <bool kXf, bool kYf>
__device__ __forceinline__ void turn_heads(const dash_heads& x, const dash_heads& y, long long from, long long to, int h0, int h1, int c0,
                                           int c1, bool turned, int interleaved, const float (&cs)[8], const float (&sn)[8]) {
    constexpr int kAtOnce = kXf ? 2 : 4;
    for (int h = h0; h < h1; h += kAtOnce) {
        Raw8<kXf> a[kAtOnce], b[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (h + i < h1) {
                a[i].load(x.data, from + (h + i) * x.stride_h + c0);
                b[i].load(x.data, from + (h + i) * x.stride_h + c1);
            }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (h + i < h1) {
                float u[8], v[8];
                a[i].get(u);
                b[i].get(v);
                if (turned) rotate(u, v, cs, sn, interleaved);
                store8<kYf>(y.data, to + (h + i) * y.stride_h + c0, u);
                store8<kYf>(y.data, to + (h + i) * y.stride_h + c1, v);
            }
    }
}

// blockIdx.z: the tensor; blockIdx.y: a run of its heads.
template <int D>
__global__ void __launch_bounds__(128, 6) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int U = D / 16;
    const dash_heads& x = p.x[blockIdx.z];
    const dash_heads& y = p.y[blockIdx.z];
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const long long token = i / U;
    const int unit = (int)(i % U);
    const int h0 = blockIdx.y * p.per, h1 = min(h0 + p.per, x.heads);
    if (token >= (long long)p.B * p.S || h0 >= h1) return;
    const int b = (int)(token / p.S), s = (int)(token - (long long)b * p.S);
    int c0, c1;
    chunks(unit, p.turns.rot, c0, c1);
    const bool turned = unit < p.turns.rot / 16;
    const long long from = b * x.stride_b + s * x.stride_s, to = b * y.stride_b + s * y.stride_s;
    const int il = p.turns.interleaved;
    float cs[8], sn[8];
    if (turned) {
        const long long pos = p.positions ? p.positions[b * p.pos_stride_b + s] : s;
        angles(p.turns, unit, pos, p.sign, cs, sn);
    }
    if (x.fp32) {
        if (y.fp32) turn_heads<true, true>(x, y, from, to, h0, h1, c0, c1, turned, il, cs, sn);
        else turn_heads<true, false>(x, y, from, to, h0, h1, c0, c1, turned, il, cs, sn);
    } else {
        if (y.fp32) turn_heads<false, true>(x, y, from, to, h0, h1, c0, c1, turned, il, cs, sn);
        else turn_heads<false, false>(x, y, from, to, h0, h1, c0, c1, turned, il, cs, sn);
    }
}

// ---------------------------------------------------------------- cache write
struct WriteParams {
    dash_kv_cache c;
    const __nv_bfloat16 *k, *v, *q;
    __nv_bfloat16* q_out;
    long long k_t, k_h, v_t, v_h, q_t, q_h, qo_t, qo_h;
    const int64_t* slots;
    const int32_t* positions;   // null: no rotation
    Turns turns;
    int T, Hq, page_shift, per; // Hq: 0 without queries; per: heads of a block
};

// fl(x / d) from inv = fl(1 / d) with one correction of the quotient (Markstein, IBM J. Res. Dev. 34, 1990): the quotient
// rounded correctly, at a third of a division's instructions, as one reciprocal serves a vector.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, d, x), inv, q);
}

// Heads of a token in the order queries, keys, values.  The threads of one
// vector are U consecutive lanes, whose maximum a butterfly forms.
template <int D, bool kE4M3>
__global__ void __launch_bounds__(128, 5) write_kernel(const __grid_constant__ WriteParams p) {
    constexpr int U = D / 16, kAtOnce = 4;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const bool live = i / U < p.T;   // whole vectors: lanes of one vector agree
    const long long token = live ? i / U : p.T - 1;
    const int unit = (int)(i % U);
    const int heads = p.Hq + 2 * p.c.Hkv;
    const int h0 = blockIdx.y * p.per, h1 = min(h0 + p.per, heads);
    const int rot = p.positions ? p.turns.rot : D;
    int c0, c1;
    chunks(unit, rot, c0, c1);
    const bool turned = p.positions && unit < rot / 16;
    float cs[8], sn[8];
    if (turned) angles(p.turns, unit, p.positions[token], 1.f, cs, sn);

    const long long slots = (long long)p.c.num_pages * p.c.page_size;
    long long slot = p.slots[token];
    if (slot >= slots && live && unit == 0 && blockIdx.y == 0)
        serve_error(DASH_ERR_PAGE, kOpWrite, token, slot, slots);
    const bool kept = live && slot >= 0 && slot < slots;
    if (!kept) slot = 0;
    const int page = (int)((unsigned long long)slot >> p.page_shift);
    const int off = (int)(slot & (p.c.page_size - 1));

    for (int hb = h0; hb < h1; hb += kAtOnce) {
        Raw8<false> ra[kAtOnce], rb[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int h = hb + k;
            if (h >= h1) continue;
            const int kind = h < p.Hq ? 0 : h < p.Hq + p.c.Hkv ? 1 : 2;
            const int hh = h - (kind == 0 ? 0 : kind == 1 ? p.Hq : p.Hq + p.c.Hkv);
            const __nv_bfloat16* base = kind == 0 ? p.q + token * p.q_t + hh * p.q_h
                                      : kind == 1 ? p.k + token * p.k_t + hh * p.k_h : p.v + token * p.v_t + hh * p.v_h;
            ra[k].load(base, c0);
            rb[k].load(base, c1);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int h = hb + k;
            if (h >= h1) continue;   // the same in all threads
            const int kind = h < p.Hq ? 0 : h < p.Hq + p.c.Hkv ? 1 : 2;
            float a[8], b[8];
            ra[k].get(a);
            rb[k].get(b);
            if (kind < 2 && turned) rotate(a, b, cs, sn, p.turns.interleaved);
            if (kind == 0) {
                if (live) {
                    __nv_bfloat16* to = p.q_out + token * p.qo_t + h * p.qo_h;
                    store8<false>(to, c0, a);
                    store8<false>(to, c1, b);
                }
                continue;
            }
            const bool val = kind == 2;
            const int hk = h - p.Hq - (val ? p.c.Hkv : 0);
            const long long cell = ((long long)page * p.c.Hkv + hk) * p.c.page_size + off;
            void* pages = val ? p.c.v : p.c.k;
            if (kE4M3) {
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(a[e]), fabsf(b[e])));
#pragma unroll
                for (int w = U / 2; w >= 1; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                const float scale = fmaxf(__fdiv_rn(m, 448.f), 0x1p-126f), inv = __frcp_rn(scale);
                uint32_t q[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    q[e] = pack_e4m3x4(quotient(a[4 * e], scale, inv), quotient(a[4 * e + 1], scale, inv),
                                       quotient(a[4 * e + 2], scale, inv), quotient(a[4 * e + 3], scale, inv));
                    q[2 + e] = pack_e4m3x4(quotient(b[4 * e], scale, inv), quotient(b[4 * e + 1], scale, inv),
                                           quotient(b[4 * e + 2], scale, inv), quotient(b[4 * e + 3], scale, inv));
                }
                if (kept) {
                    uint8_t* to = reinterpret_cast<uint8_t*>(pages) + cell * D;
                    *reinterpret_cast<uint2*>(to + c0) = make_uint2(q[0], q[1]);
                    *reinterpret_cast<uint2*>(to + c1) = make_uint2(q[2], q[3]);
                    if (unit == 0) (val ? p.c.v_scale : p.c.k_scale)[cell] = scale;
                }
            } else if (kept) {
                store8<false>(pages, cell * D + c0, a);
                store8<false>(pages, cell * D + c1, b);
            }
        }
    }
}

// ---------------------------------------------------------------- cache read
struct ReadParams {
    dash_kv_cache c;
    const int32_t* table;
    long long table_stride, stride_b, stride_h, stride_s;
    const int32_t* lens;
    __nv_bfloat16 *k, *v;
    int max_pages, B, S, page_shift;
};

// 8 values as bf16: a cell's codes times its scale, or the values themselves.
template <bool kE4M3>
struct Cell8 {
    uint4 w;
    float scale;
    __device__ __forceinline__ void load(const void* pages, const float* scales, long long cell, long long at) {
        if (kE4M3) {
            const uint2 u = __ldcs(reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(pages) + at));
            w.x = u.x, w.y = u.y;
            scale = scales[cell];
        } else {
            w = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(pages) + at));
        }
    }
    __device__ __forceinline__ uint4 get() const {
        if (!kE4M3) return w;
        float x[8];
        unpack_e4m3x8(make_uint2(w.x, w.y), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= scale;
        return pack_bf16x8(x);
    }
};

// D / 8 threads per token, 4 tokens of each thread at a time; blockIdx.y is the head, blockIdx.z the sequence.
template <int D, bool kE4M3>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int C = D / 8, kRows = 256 / C, kAtOnce = 4;
    const int d = 8 * (threadIdx.x % C), r = threadIdx.x / C;
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const long long cap = (long long)p.max_pages * p.c.page_size;
        long long given = p.lens[b];
        if (given > cap || given < 0) {
            if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
                serve_error(DASH_ERR_PAGE, kOpRead, b, given, cap);
            given = given < 0 ? 0 : cap;
        }
        const int len = (int)(given < p.S ? given : p.S);
        for (int h = blockIdx.y; h < p.c.Hkv; h += gridDim.y)
            for (int j0 = blockIdx.x * kRows * kAtOnce + r; j0 < len; j0 += gridDim.x * kRows * kAtOnce) {
                Cell8<kE4M3> k[kAtOnce], v[kAtOnce];
                bool ok[kAtOnce];
                int page[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int j = j0 + i * kRows;
                    page[i] = j < len ? p.table[b * p.table_stride + (j >> p.page_shift)] : 0;
                }
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int j = j0 + i * kRows;
                    ok[i] = j < len && page[i] >= 0 && page[i] < p.c.num_pages;
                    if (j < len && !ok[i]) serve_error(DASH_ERR_PAGE, kOpRead, b, page[i], p.c.num_pages);
                    if (!ok[i]) continue;
                    const long long cell = ((long long)page[i] * p.c.Hkv + h) * p.c.page_size + (j & (p.c.page_size - 1));
                    k[i].load(p.c.k, p.c.k_scale, cell, cell * D + d);
                    v[i].load(p.c.v, p.c.v_scale, cell, cell * D + d);
                }
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    if (!ok[i]) continue;
                    const long long to = b * p.stride_b + h * p.stride_h + (j0 + i * kRows) * p.stride_s + d;
                    *reinterpret_cast<uint4*>(p.k + to) = k[i].get();
                    *reinterpret_cast<uint4*>(p.v + to) = v[i].get();
                }
            }
    }
}

// ---------------------------------------------------------------- host
// inv_freq as 64-bit fractions of a turn; false when one is not finite.
bool make_turns(Turns* t, const double* inv_freq, int rot, int interleaved, float factor) {
    const double inv2pi = 0.15915494309189533577;   // 1 / (2 pi)
    for (int i = 0; i < rot / 2; ++i) {
        const double f = inv_freq[i];
        if (!(fabs(f) < 1e12)) return false;
        const double turns = f * inv2pi;
        double frac = turns - floor(turns);   // [0, 1], exact up to the product's rounding
        // two 32-bit halves: each step is exact in a double
        const double hi = floor(frac * 4294967296.0);
        const double lo = floor((frac * 4294967296.0 - hi) * 4294967296.0);
        t->f[i] = ((unsigned long long)hi << 32) + (unsigned long long)lo;
    }
    t->rot = rot;
    t->interleaved = interleaved;
    t->factor = factor;
    return true;
}

bool rope_args_ok(const double* inv_freq, int rot, int interleaved, float factor, int D) {
    return inv_freq && (D == 64 || D == 128) && rot >= 16 && rot <= D && rot % 16 == 0 &&
           (interleaved == 0 || interleaved == 1) && isfinite(factor);
}

// Written vectors: none may be another (a stride of 0 over more than one).
bool distinct(int64_t a, int64_t na, int64_t b, int64_t nb, int64_t c, int64_t nc) {
    return (na <= 1 || a > 0) && (nb <= 1 || b > 0) && (nc <= 1 || c > 0);
}

bool heads_ok(const dash_heads* t) {
    return serve_aligned(t->data) && (t->fp32 == 0 || t->fp32 == 1) && t->heads > 0 &&
           serve_strides(t->stride_b, t->stride_h) && serve_strides(t->stride_s, 0);
}

// Heads of a block: runs of at least 8 where there are so many, which share
// their angles, shorter ones only to have a few blocks for every SM.
int heads_per_block(long long blocks, int heads) {
    for (int per : {16, 8, 4, 2})
        if (per <= heads && blocks * ((heads + per - 1) / per) >= (per > 8 ? 4096 : 1024)) return per;
    return 1;
}

int launched() { return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA; }

}  // namespace

int serve_check_device() {
    static int known[64] = {};   // 1: sm_103
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DASH_ERR_CUDA;
    if (dev >= 0 && dev < 64 && known[dev]) return DASH_OK;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return DASH_ERR_CUDA;
    if (major != 10 || minor != 3) return DASH_ERR_DEVICE;
    if (dev >= 0 && dev < 64) known[dev] = 1;
    return DASH_OK;
}

int error_rope(int* out5, bool clear) { return serve_record(out5, clear); }

}  // namespace dash

using namespace dash;

extern "C" int dash_rope(const dash_heads* x, const dash_heads* y, const dash_heads* x2, const dash_heads* y2,
                         const int32_t* positions, int64_t pos_stride_b, const double* inv_freq, int rot,
                         int interleaved, float factor, int inverse, int B, int S, int D, dash_stream_t stream) {
    if (!x || !y || !x2 != !y2) return DASH_ERR_ARG;
    if (B < 0 || S < 0 || !rope_args_ok(inv_freq, rot, interleaved, factor, D) || (inverse != 0 && inverse != 1) ||
        pos_stride_b < 0 || ((uintptr_t)positions & 3u))
        return DASH_ERR_ARG;
    if (B == 0 || S == 0) return DASH_OK;
    RopeParams prm;
    for (int t = 0; t < (x2 ? 2 : 1); ++t) {
        const dash_heads* a = t ? x2 : x;
        const dash_heads* c = t ? y2 : y;
        if (!heads_ok(a) || !heads_ok(c) || a->heads != c->heads ||
            !distinct(c->stride_b, B, c->stride_h, c->heads, c->stride_s, S))
            return DASH_ERR_ARG;
        if (a->data == c->data && (a->fp32 != c->fp32 || a->stride_b != c->stride_b || a->stride_h != c->stride_h ||
                                   a->stride_s != c->stride_s))
            return DASH_ERR_ARG;
        prm.x[t] = *a;
        prm.y[t] = *c;
    }
    if ((long long)B * S * (D / 16) > (1ll << 31) * 127 || x->heads > 65535 || (x2 && x2->heads > 65535)) return DASH_ERR_ARG;
    if (!make_turns(&prm.turns, inv_freq, rot, interleaved, factor)) return DASH_ERR_ARG;
    const int rc = serve_check_device();
    if (rc) return rc;
    prm.positions = positions;
    prm.pos_stride_b = pos_stride_b;
    prm.sign = inverse ? -1.f : 1.f;
    prm.B = B;
    prm.S = S;
    const long long blocks = ((long long)B * S * (D / 16) + 127) / 128;
    const int most = x2 && x2->heads > x->heads ? x2->heads : x->heads;
    prm.per = heads_per_block(blocks, most);
    const dim3 grid((unsigned)blocks, (unsigned)((most + prm.per - 1) / prm.per), x2 ? 2 : 1);
    if (D == 64)
        rope_kernel<64><<<grid, 128, 0, (cudaStream_t)stream>>>(prm);
    else
        rope_kernel<128><<<grid, 128, 0, (cudaStream_t)stream>>>(prm);
    return launched();
}

extern "C" int dash_rope_freqs(int rot, double base, int scaling, double scale, int trained, double lo, double hi,
                               double* inv_freq, float* factor) {
    if (!inv_freq || !factor || rot < 4 || rot % 2 || !(base > 1.0) || !(scale >= 1.0) || !isfinite(base) ||
        !isfinite(scale) || scaling < DASH_ROPE_PLAIN || scaling > DASH_ROPE_RAMP)
        return DASH_ERR_ARG;
    const bool bands = scaling == DASH_ROPE_WAVE || scaling == DASH_ROPE_RAMP;
    if (bands && (trained < 1 || !(lo > 0.0) || !(hi > lo) || !isfinite(hi))) return DASH_ERR_ARG;
    const double two_pi = 6.28318530717958647693;
    if (scaling == DASH_ROPE_BASE) base *= pow(scale, (double)rot / (rot - 2));
    double first = 0, last = 0;
    if (scaling == DASH_ROPE_RAMP) {   // the pair indexes that make hi and lo turns over the trained length
        first = floor(rot * log(trained / (hi * two_pi)) / (2.0 * log(base)));
        last = ceil(rot * log(trained / (lo * two_pi)) / (2.0 * log(base)));
        first = first < 0 ? 0 : first;
        last = last > rot - 1 ? rot - 1 : last;
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot);
        double keep = 1.0;   // share of the unscaled frequency
        if (scaling == DASH_ROPE_LINEAR) keep = 0.0;
        if (scaling == DASH_ROPE_WAVE) keep = (trained * f / two_pi - lo) / (hi - lo);
        if (scaling == DASH_ROPE_RAMP) keep = 1.0 - (i - first) / (last - first > 1e-3 ? last - first : 1e-3);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        inv_freq[i] = scaling == DASH_ROPE_BASE ? f : f * (keep + (1.0 - keep) / scale);
    }
    *factor = (scaling == DASH_ROPE_RAMP && scale > 1.0) ? (float)(0.1 * log(scale) + 1.0) : 1.f;
    return DASH_OK;
}

extern "C" int dash_kv_write(const dash_kv_cache* cache, const dash_bf16* k, int64_t k_stride_t, int64_t k_stride_h,
                             const dash_bf16* v, int64_t v_stride_t, int64_t v_stride_h, const int64_t* slots, int T,
                             const dash_write_rope* rope, dash_stream_t stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (T < 0 || !serve_strides(k_stride_t, k_stride_h) || !serve_strides(v_stride_t, v_stride_h)) return DASH_ERR_ARG;
    if (rope && !rope_args_ok(rope->inv_freq, rope->rot, rope->interleaved, rope->factor, cache->D)) return DASH_ERR_ARG;
    if (T == 0) return DASH_OK;
    if (!serve_aligned(k) || !serve_aligned(v) || !slots || ((uintptr_t)slots & 7u)) return DASH_ERR_ARG;
    WriteParams prm;
    prm.c = *cache;
    prm.k = (const __nv_bfloat16*)k;
    prm.v = (const __nv_bfloat16*)v;
    prm.k_t = k_stride_t;
    prm.k_h = k_stride_h;
    prm.v_t = v_stride_t;
    prm.v_h = v_stride_h;
    prm.slots = slots;
    prm.positions = nullptr;
    prm.q = nullptr;
    prm.q_out = nullptr;
    prm.Hq = 0;
    prm.T = T;
    prm.page_shift = __builtin_ctz((unsigned)cache->page_size);
    prm.turns.interleaved = 0;
    if (rope) {
        if (!rope->positions || ((uintptr_t)rope->positions & 3u)) return DASH_ERR_ARG;
        if (!make_turns(&prm.turns, rope->inv_freq, rope->rot, rope->interleaved, rope->factor)) return DASH_ERR_ARG;
        prm.positions = rope->positions;
        if (rope->q) {
            if (!serve_aligned(rope->q) || !serve_aligned(rope->q_out) || rope->Hq <= 0 ||
                !serve_strides(rope->q_stride_t, rope->q_stride_h) ||
                !serve_strides(rope->q_out_stride_t, rope->q_out_stride_h) ||
                !distinct(rope->q_out_stride_t, T, rope->q_out_stride_h, rope->Hq, 0, 1))
                return DASH_ERR_ARG;
            if (rope->q == rope->q_out &&
                (rope->q_stride_t != rope->q_out_stride_t || rope->q_stride_h != rope->q_out_stride_h))
                return DASH_ERR_ARG;
            prm.q = (const __nv_bfloat16*)rope->q;
            prm.q_out = (__nv_bfloat16*)rope->q_out;
            prm.q_t = rope->q_stride_t;
            prm.q_h = rope->q_stride_h;
            prm.qo_t = rope->q_out_stride_t;
            prm.qo_h = rope->q_out_stride_h;
            prm.Hq = rope->Hq;
        }
    }
    if ((long long)prm.Hq + 2ll * cache->Hkv > 65535) return DASH_ERR_ARG;
    if ((rc = serve_check_device())) return rc;
    const int D = cache->D;
    const long long blocks = ((long long)T * (D / 16) + 127) / 128;
    prm.per = heads_per_block(blocks, prm.Hq + 2 * cache->Hkv);
    const dim3 grid((unsigned)blocks, (unsigned)((prm.Hq + 2 * cache->Hkv + prm.per - 1) / prm.per));
    cudaStream_t s = (cudaStream_t)stream;
    if (cache->type == DASH_CACHE_E4M3) {
        if (D == 64) write_kernel<64, true><<<grid, 128, 0, s>>>(prm);
        else write_kernel<128, true><<<grid, 128, 0, s>>>(prm);
    } else {
        if (D == 64) write_kernel<64, false><<<grid, 128, 0, s>>>(prm);
        else write_kernel<128, false><<<grid, 128, 0, s>>>(prm);
    }
    return launched();
}

extern "C" int dash_kv_read(const dash_kv_cache* cache, const int32_t* block_table, int64_t table_stride,
                            int max_pages, const int32_t* lens, dash_bf16* k, dash_bf16* v, int64_t stride_b,
                            int64_t stride_h, int64_t stride_s, int B, int S, dash_stream_t stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (B < 0 || S < 0 || S > (1 << 30) || max_pages < 0 || table_stride < 0 || !serve_strides(stride_b, stride_h) ||
        !serve_strides(stride_s, 0))
        return DASH_ERR_ARG;
    if (B == 0 || S == 0) return DASH_OK;
    if (!serve_aligned(k) || !serve_aligned(v) || !lens || ((uintptr_t)lens & 3u) || ((uintptr_t)block_table & 3u) ||
        (max_pages > 0 && !block_table) || !distinct(stride_b, B, stride_h, cache->Hkv, stride_s, S))
        return DASH_ERR_ARG;
    if ((rc = serve_check_device())) return rc;
    ReadParams prm;
    prm.c = *cache;
    prm.table = block_table;
    prm.table_stride = table_stride;
    prm.stride_b = stride_b;
    prm.stride_h = stride_h;
    prm.stride_s = stride_s;
    prm.lens = lens;
    prm.k = (__nv_bfloat16*)k;
    prm.v = (__nv_bfloat16*)v;
    prm.max_pages = max_pages;
    prm.B = B;
    prm.S = S;
    prm.page_shift = __builtin_ctz((unsigned)cache->page_size);
    const int D = cache->D;
    const long long x = ((long long)S + 4 * (2048 / D) - 1) / (4 * (2048 / D));   // 4 tokens of every thread
    const dim3 grid((unsigned)(x < 65536 ? x : 65536), (unsigned)(cache->Hkv < 65535 ? cache->Hkv : 65535),
                    (unsigned)(B < 65535 ? B : 65535));
    cudaStream_t s = (cudaStream_t)stream;
    if (cache->type == DASH_CACHE_E4M3) {
        if (D == 64) read_kernel<64, true><<<grid, 256, 0, s>>>(prm);
        else read_kernel<128, true><<<grid, 256, 0, s>>>(prm);
    } else {
        if (D == 64) read_kernel<64, false><<<grid, 256, 0, s>>>(prm);
        else read_kernel<128, false><<<grid, 256, 0, s>>>(prm);
    }
    return launched();
}

extern "C" int dash_get_status_paged(dash_stream_t stream, int* code, int* info) {
    if (!code) return DASH_ERR_ARG;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return DASH_ERR_CUDA;
    // one record per translation unit; all are read before one is cleared, and only the one reported is
    int (*const record[3])(int*, bool) = {error_rope, error_paged, error_tile};
    int r[3][5], pick = -1;
    for (int i = 0; i < 3; ++i) {
        const int rc = record[i](r[i], false);
        if (rc) return rc;
        if (r[i][0] && (pick < 0 || (r[i][0] == DASH_ERR_TIMEOUT && r[pick][0] != DASH_ERR_TIMEOUT))) pick = i;
    }
    if (pick >= 0) {
        const int rc = record[pick](nullptr, true);
        if (rc) return rc;
    }
    *code = pick < 0 ? DASH_OK : r[pick][0];
    if (info)
        for (int i = 0; i < 4; ++i) info[i] = pick < 0 ? 0 : r[pick][1 + i];
    return DASH_OK;
}
