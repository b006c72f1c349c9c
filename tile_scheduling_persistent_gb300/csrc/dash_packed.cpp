// dash_packed.cpp -- the serving calls with their arguments in one block of words (dash_packed), for callers that pay for
// every argument they pass: a foreign call from Python with 20 of them takes 1.6 us, one with a packed block 0.4 us.
#include "dash.h"

#include <stdint.h>

namespace {

// Words that are ints in the call itself, as bits, by call.
constexpr uint32_t kInts[] = {
    1u << 7,
    1u << 2 | 1u << 9 | 1u << 10,
    1u << 5 | 0x3fu << 10,
    1u << 3 | 1u << 8 | 1u << 9 | 1u << 11 | 1u << 12,
    1u << 3 | 1u << 4 | 1u << 6 | 1u << 7 | 1u << 11,
    1u << 3 | 1u << 4 | 1u << 6 | 1u << 7,
};

}  // namespace

extern "C" int dash_packed(int call, const int64_t* w, const dash_kv_cache* cache, const dash_write_rope* rope) {
    if (call < 0 || call >= (int)(sizeof(kInts) / sizeof(kInts[0])) || !w) return DASH_ERR_ARG;
    for (uint32_t m = kInts[call]; m; m &= m - 1) {
        const int64_t x = w[__builtin_ctz(m)];
        if (x != (int)x) return DASH_ERR_ARG;
    }
    auto num = [w](int i) { return (int)w[i]; };
    auto bf16 = [w](int i) { return (dash_bf16*)(uintptr_t)w[i]; };
    auto i32 = [w](int i) { return (int32_t*)(uintptr_t)w[i]; };
    auto any = [w](int i) { return (void*)(uintptr_t)w[i]; };
    switch (call) {
        case DASH_PACKED_KV_WRITE:
            return dash_kv_write(cache, bf16(0), w[1], w[2], bf16(3), w[4], w[5], (const int64_t*)any(6), num(7), rope, (dash_stream_t)any(8));
        case DASH_PACKED_KV_READ:
            return dash_kv_read(cache, i32(0), w[1], num(2), i32(3), bf16(4), bf16(5), w[6], w[7], w[8], num(9), num(10), (dash_stream_t)any(11));
        case DASH_PACKED_ATTN_PAGED:
            return dash_attn_paged(bf16(0), w[1], w[2], cache, i32(3), w[4], num(5), i32(6), i32(7), bf16(8), (float*)any(9), num(10), num(11),
                                   num(12), num(13), num(14), num(15), any(16), (size_t)w[17], (dash_stream_t)any(18));
        case DASH_PACKED_PAGES_FORK:
            return dash_pages_fork(i32(0), w[1], i32(2), num(3), i32(4), i32(5), w[6], i32(7), num(8), num(9), i32(10), num(11), num(12),
                                   (dash_stream_t)any(13));
        case DASH_PACKED_PAGES_EXTEND:
            return dash_pages_extend(i32(0), w[1], i32(2), num(3), num(4), i32(5), num(6), num(7), i32(8), (int64_t*)any(9), i32(10), num(11),
                                     i32(12), i32(13), (dash_stream_t)any(14));
        default:
            return dash_pages_compact(i32(0), w[1], i32(2), num(3), num(4), i32(5), num(6), num(7), i32(8), w[9], i32(10), i32(11), i32(12),
                                      any(13), (size_t)w[14], (dash_stream_t)any(15));
    }
}
