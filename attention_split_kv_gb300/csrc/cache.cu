// cache.cu -- the steps on either side of the attention kernels: writing new
// tokens into a KV cache and reading cached tokens back.
//
// attn_append (doppler src/inference/pipelines/text/attention/run.js,
// runLayerAttentionGPU: per-head q/k RMS norm, RoPE from cos/sin tables, then
// the KV-cache update).  For a q or k head x in R^D of a token at position p:
//
//   y   = x * rsqrt(mean(x^2) + eps) * (w + offset)              (optional)
//   z_a = y_a cos(p, e) - y_b sin(p, e),  z_b = y_b cos(p, e) + y_a sin(p, e)
//         over the pairs (a, b) = (e, e + R/2) or (2e, 2e + 1), e < R/2
//
// in f32 with one rounding at the end: to f16, or for an int8 cache to codes
// with s = f16(max|z| / 127), code = rint(z / s).  v heads are only written.
//
// attn_kv_read is the way back: x = code * s (or the f16 value) as packed rows.
//
// Both move each byte once and compute a few operations on it, so they are
// bound by memory, and small calls by the chain of dependent loads (sequence ->
// length -> page -> slot).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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

// 8 elements as they lie in memory, and as f32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__half> {
    uint4 r;
    __device__ __forceinline__ void load(const __half* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    Raw8<T> r;
    r.load(p);
    r.get(x);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]),
                                              pack2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
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

// ------------------------------------------------------------------ append
// A CTA takes a token (blockIdx.x), or of few tokens a part of its heads (blockIdx.y of
// gridDim.y); a group of D/8 lanes a head at a time, 8 elements a lane (16-byte accesses).
// The norm, the largest magnitude and the half-split partner are shuffles inside the group.
// A lane's first two loads are issued before the search for the token's sequence, each
// later one before the head two back is worked on, so that the chain of dependent loads
// (sequence, page, table row) lies under them.
template <int D, typename T, typename TQ, bool INT8>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
    constexpr int LPR = D / 8;          // lanes a head
    constexpr int RPW = 32 / LPR;       // heads a warp
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x;
    const int sub = lane & (LPR - 1);   // lane within its head
    const int e0 = sub * 8;             // its first element
    const int n_heads = a.Hq + 2 * a.Hkv;
    const int step = static_cast<int>(gridDim.y * (blockDim.x >> 5)) * RPW;
    int h0 = static_cast<int>(blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5)) * RPW;
    auto fetch = [&](int h, Raw8<T>& r) {
        if (h >= n_heads) return;
        const T* p = h < a.Hq            ? static_cast<const T*>(a.q) + t * a.q_stride + h * D
                     : h < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + t * a.k_stride + (h - a.Hq) * D
                                        : static_cast<const T*>(a.v) + t * a.v_stride + (h - a.Hq - a.Hkv) * D;
        r.load(p + e0);
    };
    Raw8<T> raw[2];
    fetch(h0 + lane / LPR, raw[0]);
    fetch(h0 + step + lane / LPR, raw[1]);

    const Where w = find_row(a.q_start, a.kv_len, a.B, t, lane);
    if (w.b < 0) return;
    const long long p = static_cast<long long>(w.len) - w.end + t;   // kv_len - q_len + i
    const bool in_range = p >= 0 && p < a.cache.capacity && (a.rot == 0 || p < a.n_pos);
    if (!in_range) {
        if (threadIdx.x == 0) atomicExch(a.err, kErrAppendRange);
        return;
    }
    // a ring holds a sequence's newest tokens; what a longer chunk overwrites is not
    // written at all, so no two tokens of a call share a slot
    bool write = a.cache.ring == 0 || p >= static_cast<long long>(w.len) - a.cache.ring;
    Slot slot{0, 0};
    if (write) write = find_slot(a.cache, w.b, p, slot, a.err);

    float cs[8], sn[8];
    const int half = a.rot / 2;
    const bool rotates = e0 < a.rot;
    if (rotates) {
        const float* ct = a.cos + static_cast<size_t>(p) * half;
        const float* st = a.sin + static_cast<size_t>(p) * half;
        if (a.interleaved) {
            const float4 c4 = *reinterpret_cast<const float4*>(ct + e0 / 2);
            const float4 s4 = *reinterpret_cast<const float4*>(st + e0 / 2);
            cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
            sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
        } else {
            const int e = e0 < half ? e0 : e0 - half;
            load8(ct + e, cs);
            load8(st + e, sn);
        }
    }

    for (; h0 < n_heads; h0 += step) {   // uniform in the warp
        const int h = h0 + lane / LPR;
        const bool live = h < n_heads;
        const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;    // q, k, v
        const int hh = kind == 0 ? h : kind == 1 ? h - a.Hq : h - a.Hq - a.Hkv;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (live) raw[0].get(x);
        raw[0] = raw[1];
        fetch(h + 2 * step, raw[1]);
        const float* nw = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
        if (a.q_norm || a.k_norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            if (nw) {
                const float r = rsqrtf(ss * (1.0f / D) + a.eps);
                float g[8];
                load8(nw + e0, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (g[i] + a.offset);
            }
        }
        if (a.rot) {
            if (a.interleaved) {
                if (rotates && kind < 2) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = x[2 * i], v = x[2 * i + 1];
                        x[2 * i] = u * cs[i] - v * sn[i];
                        x[2 * i + 1] = v * cs[i] + u * sn[i];
                    }
                }
            } else {
                // the partner's 8 elements sit half / 8 lanes on (or back)
                const bool low = e0 < half;
                const int from = rotates ? lane + (low ? half / 8 : -(half / 8)) : lane;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(kFull, x[i], from);
                if (rotates && kind < 2) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = low ? x[i] * cs[i] - y[i] * sn[i] : x[i] * cs[i] + y[i] * sn[i];
                }
            }
        }
        float scale = 0.f;
        if constexpr (INT8) {
            // largest magnitude by its bits, which order NaN above infinity: a row with
            // either gets it as its scale
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
            scale = __half2float(__float2half_rn(__fdiv_rn(__uint_as_float(m), 127.0f)));
        }
        if (!live) continue;
        if (kind == 0) {
            store8(static_cast<TQ*>(a.q_out) + (static_cast<size_t>(t) * a.Hq + hh) * D + e0, x);
            continue;
        }
        if (!write) continue;
        const size_t row = slot.slot * a.cache.rows + slot.row;
        const size_t at = (row * a.Hkv + hh) * D + e0;
        if constexpr (INT8) {
            uint32_t c[2] = {0, 0};
            if (scale > 0.f && scale < INFINITY) {
                // x times 1 / scale is within 2^-23 * 127.1 < 2e-5 of x / scale, so it rounds
                // alike unless it lies that near to a tie: then the division decides
                const float inv = __fdiv_rn(1.0f, scale);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float q = x[i] * inv, r = rintf(q);
                    if (fabsf(q - r) > 0.4999f) r = rintf(__fdiv_rn(x[i], scale));
                    r = fminf(fmaxf(r, -127.f), 127.f);
                    c[i / 4] |= (static_cast<uint32_t>(static_cast<int>(r)) & 0xffu) << (8 * (i & 3));
                }
            }
            *reinterpret_cast<uint2*>(static_cast<int8_t*>(kind == 1 ? a.k_cache : a.v_cache) + at) =
                make_uint2(c[0], c[1]);
            if (sub == 0)
                static_cast<__half*>(kind == 1 ? a.k_scales : a.v_scales)[(slot.slot * a.Hkv + hh) * a.cache.rows +
                                                                           slot.row] = __float2half_rn(scale);
        } else {
            store8(static_cast<__half*>(kind == 1 ? a.k_cache : a.v_cache) + at, x);
        }
    }
}

template <int D, typename T, typename TQ>
void append_dispatch(const AppendArgs& a, bool int8, dim3 grid, int threads, cudaStream_t s) {
    if (int8) append_kernel<D, T, TQ, true><<<grid, threads, 0, s>>>(a);
    else append_kernel<D, T, TQ, false><<<grid, threads, 0, s>>>(a);
}
template <int D>
void append_types(const AppendLaunch& L, dim3 grid, int threads) {
    if (L.in_f32) {
        if (L.q_out_f32) append_dispatch<D, float, float>(L.args, L.int8, grid, threads, L.stream);
        else append_dispatch<D, float, __half>(L.args, L.int8, grid, threads, L.stream);
    } else {
        if (L.q_out_f32) append_dispatch<D, __half, float>(L.args, L.int8, grid, threads, L.stream);
        else append_dispatch<D, __half, __half>(L.args, L.int8, grid, threads, L.stream);
    }
}

// ------------------------------------------------------------------ read back
// A warp takes a row; a lane pieces of 16 elements (one 16-byte load of codes, two of f16),
// four at a time, all loads before the first store.
constexpr int kReadWarps = 8;

template <typename TO, bool INT8>
__global__ void __launch_bounds__(kReadWarps * 32) kv_read_kernel(const KvReadArgs a) {
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
    if (t >= a.total) return;
    const int log_d = a.D == 64 ? 2 : a.D == 128 ? 3 : 4;   // log2 of a head's pieces
    const int per = a.Hkv << log_d;                          // pieces of a token's K (or V)
    const Where w = find_row(a.out_start, a.kv_len, a.B, static_cast<int>(t), lane);
    if (w.b < 0) return;
    const long long p = (a.first ? static_cast<long long>(a.first[w.b]) : 0ll) + (t - w.start);
    bool held = p >= 0 && p < w.len && p < a.cache.capacity &&
                (a.cache.ring == 0 || p >= static_cast<long long>(w.len) - a.cache.ring);
    Slot slot{0, 0};
    if (held) held = find_slot(a.cache, w.b, p, slot, a.err);
    const size_t src = (slot.slot * a.cache.rows + slot.row) * a.Hkv * a.D;
    const size_t dst = static_cast<size_t>(t) * a.Hkv * a.D;
    for (int c0 = lane; c0 < 2 * per; c0 += 128) {
        uint4 raw[4][INT8 ? 1 : 2];
        __half sc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = c0 + 32 * u;
            const bool is_k = c < per;
            const int cc = is_k ? c : c - per;
            if (c >= 2 * per || !held) {
#pragma unroll
                for (int i = 0; i < (INT8 ? 1 : 2); ++i) raw[u][i] = make_uint4(0u, 0u, 0u, 0u);
                sc[u] = __float2half_rn(0.f);
            } else if constexpr (INT8) {
                raw[u][0] = *reinterpret_cast<const uint4*>(static_cast<const int8_t*>(is_k ? a.k_cache : a.v_cache) +
                                                            src + static_cast<size_t>(cc) * 16);
                sc[u] = static_cast<const __half*>(
                    is_k ? a.k_scales : a.v_scales)[(slot.slot * a.Hkv + (cc >> log_d)) * a.cache.rows + slot.row];
            } else {
                const uint4* s = reinterpret_cast<const uint4*>(
                    static_cast<const __half*>(is_k ? a.k_cache : a.v_cache) + src + static_cast<size_t>(cc) * 16);
                raw[u][0] = s[0];
                raw[u][1] = s[1];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = c0 + 32 * u;
            if (c >= 2 * per) break;
            const bool is_k = c < per;
            TO* out = static_cast<TO*>(is_k ? a.k_out : a.v_out) + dst + static_cast<size_t>(is_k ? c : c - per) * 16;
            float x[2][8];
            if constexpr (INT8) {
                const float s = __half2float(sc[u]);
                const uint32_t wd[4] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i / 8][i % 8] = static_cast<float>(static_cast<int8_t>(wd[i / 4] >> (8 * (i & 3)))) * s;
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Raw8<__half> r;
                    r.r = raw[u][i];
                    r.get(x[i]);
                }
            }
            store8(out, x[0]);
            store8(out + 8, x[1]);
        }
    }
}

}  // namespace

attn_status launch_append(const AppendLaunch& L) {
    const AppendArgs& a = L.args;
    // One CTA a token.  A call with fewer tokens than two an SM spreads each token's heads over
    // CTAs of one pass.
    const int lanes = (a.Hq + 2 * a.Hkv) * (L.D / 8);
    const int threads = lanes >= 256 ? 256 : (lanes + 31) / 32 * 32;
    const int parts = a.total_q >= 2 * sm_count() ? 1 : (lanes + threads - 1) / threads;
    const dim3 grid(a.total_q, parts);
    if (trace_enabled())
        trace("append_kernel<D=%d,in=%s,q_out=%s,int8=%d> grid=(%d,%d) block=%d B=%d Hq=%d Hkv=%d rot=%d", L.D,
              L.in_f32 ? "f32" : "f16", L.q_out_f32 ? "f32" : "f16", (int)L.int8, a.total_q, parts, threads, a.B, a.Hq,
              a.Hkv, a.rot);
    switch (L.D) {
        case 64: append_types<64>(L, grid, threads); break;
        case 128: append_types<128>(L, grid, threads); break;
        default: append_types<256>(L, grid, threads); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "append launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

attn_status launch_kv_read(const KvReadLaunch& L) {
    const KvReadArgs& a = L.args;
    const int grid = (a.total - 1) / kReadWarps + 1;
    if (trace_enabled())
        trace("kv_read_kernel<out=%s,int8=%d> grid=%d block=%d B=%d Hkv=%d D=%d", L.out_f32 ? "f32" : "f16",
              (int)L.int8, grid, kReadWarps * 32, a.B, a.Hkv, a.D);
    if (L.int8) {
        if (L.out_f32) kv_read_kernel<float, true><<<grid, kReadWarps * 32, 0, L.stream>>>(a);
        else kv_read_kernel<__half, true><<<grid, kReadWarps * 32, 0, L.stream>>>(a);
    } else {
        if (L.out_f32) kv_read_kernel<float, false><<<grid, kReadWarps * 32, 0, L.stream>>>(a);
        else kv_read_kernel<__half, false><<<grid, kReadWarps * 32, 0, L.stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "kv_read launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

}  // namespace attn
