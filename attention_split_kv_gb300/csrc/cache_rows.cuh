// cache_rows.cuh -- what the cache kernels (cache.cu, latent_cache.cu) share: the sequence of a
// packed row, the place of a position in a cache, 4- and 8-element loads and stores.
#pragma once
#include <cuda_fp16.h>

#include "attn_internal.h"

namespace attn {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct Where {       // a packed row's place in its sequence
    int b;           // sequence, or -1: the row lies behind the last one
    int start, end;  // the sequence's rows
    int len;         // its kv_len
};

// The sequence of packed row t: the last b with start[b] <= t (so empty ones are
// passed over), by a 32-way search of the whole warp.  Its last step reads the
// lengths of its 32 candidates beside their starts, so up to 32 sequences cost
// one load's latency.
__device__ __forceinline__ Where find_row(const int32_t* __restrict__ start, const int32_t* __restrict__ kv_len,
                                          int B, int t, int lane) {
    int lo = 0, n = B;
    while (n > 32) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane * step < n && start[at] <= t;
        const int c = max(__popc(__ballot_sync(kFull, le)), 1) - 1;
        lo += c * step;
        n = min(step, n - c * step);
    }
    int s = 0, e = 0, len = 0;
    if (lane < n) {
        s = start[lo + lane];
        e = start[lo + lane + 1];
        len = kv_len[lo + lane];
    }
    const unsigned le = __ballot_sync(kFull, lane < n && s <= t);
    const int k = le ? 31 - __clz(le) : 0;
    Where w;
    w.b = lo + k;
    w.start = __shfl_sync(kFull, s, k);
    w.end = __shfl_sync(kFull, e, k);
    w.len = __shfl_sync(kFull, len, k);
    if (t < w.start || t >= w.end) w.b = -1;
    return w;
}

// 4 elements as they lie in memory, and as f32.
template <typename T>
struct Raw4;
template <>
struct Raw4<__half> {
    uint2 r;
    __device__ __forceinline__ void load(const __half* p) { r = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(float2* x) const {
        x[0] = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
        x[1] = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
    }
};
template <>
struct Raw4<float> {
    float4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(float2* x) const {
        x[0] = make_float2(r.x, r.y);
        x[1] = make_float2(r.z, r.w);
    }
};
__device__ __forceinline__ void load4(const float* p, float2* x) {
    Raw4<float> r;
    r.load(p);
    r.get(x);
}
__device__ __forceinline__ uint32_t pack2(float2 a) {
    const __half2 h = __floats2half2_rn(a.x, a.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store4(__half* p, const float2* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0]), pack2(x[1]));
}
__device__ __forceinline__ void store4(float* p, const float2* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
}
__device__ __forceinline__ void store8(__half* p, const float2 (&x)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
}
__device__ __forceinline__ void store8(float* p, const float2 (&x)[4]) {
    store4(p, x);
    store4(p + 4, x + 2);
}

// Where the cache keeps position p; false if its page id is outside the pool.
struct Slot {
    size_t slot;   // page or sequence
    int row;       // token within it
};
__device__ __forceinline__ bool find_slot(const CacheLayout& c, int b, long long p, Slot& s, int* err) {
    if (c.ring > 0) {
        s.slot = b;
        s.row = static_cast<int>(p % c.ring);
        return true;
    }
    if (!c.page_table) {
        s.slot = b;
        s.row = static_cast<int>(p);
        return true;
    }
    const int pg = c.page_table[static_cast<size_t>(b) * c.max_pages + (p >> c.log2P)];
    if (pg < 0 || pg >= c.n_pages) {
        atomicExch(err, kErrCachePage);
        return false;
    }
    s.slot = pg;
    s.row = static_cast<int>(p & (c.rows - 1));
    return true;
}

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

}  // namespace
}  // namespace attn
