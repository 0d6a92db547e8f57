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

__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
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
// One CTA a token, one group of D/8 lanes a head at a time (8 elements a lane,
// 16-byte accesses): the norm, the largest magnitude and the half-split partner
// are shuffles inside the group.
template <int D, typename T, typename TQ, bool INT8>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
    constexpr int LPR = D / 8;          // lanes a head
    constexpr int RPW = 32 / LPR;       // heads a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    const int t = blockIdx.x;
    const int sub = lane & (LPR - 1);   // lane within its head
    const int e0 = sub * 8;             // its first element
    const int n_heads = a.Hq + 2 * a.Hkv;
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

    for (int h0 = warp * RPW; h0 < n_heads; h0 += n_warps * RPW) {   // uniform in the warp
        const int h = h0 + lane / LPR;
        const bool live = h < n_heads;
        const int kind = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;    // q, k, v
        const int hh = kind == 0 ? h : kind == 1 ? h - a.Hq : h - a.Hq - a.Hkv;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (live) {
            const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                           static_cast<size_t>(t) * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                           hh * D + e0;
            load8(src, x);
        }
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
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float q = fminf(fmaxf(rintf(__fdiv_rn(x[i], scale)), -127.f), 127.f);
                    c[i / 4] |= (static_cast<uint32_t>(static_cast<int>(q)) & 0xffu) << (8 * (i & 3));
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
void append_dispatch(const AppendArgs& a, bool int8, int threads, cudaStream_t s) {
    if (int8) append_kernel<D, T, TQ, true><<<a.total_q, threads, 0, s>>>(a);
    else append_kernel<D, T, TQ, false><<<a.total_q, threads, 0, s>>>(a);
}
template <int D>
void append_types(const AppendLaunch& L, int threads) {
    if (L.in_f32) {
        if (L.q_out_f32) append_dispatch<D, float, float>(L.args, L.int8, threads, L.stream);
        else append_dispatch<D, float, __half>(L.args, L.int8, threads, L.stream);
    } else {
        if (L.q_out_f32) append_dispatch<D, __half, float>(L.args, L.int8, threads, L.stream);
        else append_dispatch<D, __half, __half>(L.args, L.int8, threads, L.stream);
    }
}

// ------------------------------------------------------------------ read back
// A warp takes 4 consecutive rows; a lane 16 elements at a time (one 16-byte load
// of codes, or two of f16).
constexpr int kReadRows = 4, kReadWarps = 8;

template <typename TO, bool INT8>
__global__ void __launch_bounds__(kReadWarps * 32) kv_read_kernel(const KvReadArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long t0 = (static_cast<long long>(blockIdx.x) * kReadWarps + warp) * kReadRows;
    const int per = a.Hkv * (a.D / 16);   // 16-element pieces of a token's K (or V)
    for (int r = 0; r < kReadRows; ++r) {
        if (t0 + r >= a.total) return;
        const int t = static_cast<int>(t0 + r);
        const Where w = find_row(a.out_start, a.kv_len, a.B, t, lane);
        if (w.b < 0) return;
        const long long p = (a.first ? static_cast<long long>(a.first[w.b]) : 0ll) + (t - w.start);
        bool held = p >= 0 && p < w.len && p < a.cache.capacity &&
                    (a.cache.ring == 0 || p >= static_cast<long long>(w.len) - a.cache.ring);
        Slot slot{0, 0};
        if (held) held = find_slot(a.cache, w.b, p, slot, a.err);
        const size_t row = slot.slot * a.cache.rows + slot.row;
        for (int c = lane; c < 2 * per; c += 32) {
            const bool is_k = c < per;
            const int cc = is_k ? c : c - per;
            const int hh = cc / (a.D / 16);
            float x[2][8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[0][i] = x[1][i] = 0.f;
            if (held) {
                const size_t at = row * a.Hkv * a.D + static_cast<size_t>(cc) * 16;
                if constexpr (INT8) {
                    const uint4 u = *reinterpret_cast<const uint4*>(
                        static_cast<const int8_t*>(is_k ? a.k_cache : a.v_cache) + at);
                    const float s = __half2float(static_cast<const __half*>(
                        is_k ? a.k_scales : a.v_scales)[(slot.slot * a.Hkv + hh) * a.cache.rows + slot.row]);
                    const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[i / 8][i % 8] = static_cast<float>(static_cast<int8_t>(wd[i / 4] >> (8 * (i & 3)))) * s;
                } else {
                    const __half* src = static_cast<const __half*>(is_k ? a.k_cache : a.v_cache) + at;
                    load8(src, x[0]);
                    load8(src + 8, x[1]);
                }
            }
            TO* dst = static_cast<TO*>(is_k ? a.k_out : a.v_out) + static_cast<size_t>(t) * a.Hkv * a.D +
                      static_cast<size_t>(cc) * 16;
            store8(dst, x[0]);
            store8(dst + 8, x[1]);
        }
    }
}

}  // namespace

attn_status launch_append(const AppendLaunch& L) {
    const AppendArgs& a = L.args;
    // one pass over the token's heads where 256 threads hold them
    const int lanes = (a.Hq + 2 * a.Hkv) * (L.D / 8);
    const int threads = lanes >= 256 ? 256 : (lanes + 31) / 32 * 32;
    if (trace_enabled())
        trace("append_kernel<D=%d,in=%s,q_out=%s,int8=%d> grid=%d block=%d B=%d Hq=%d Hkv=%d rot=%d", L.D,
              L.in_f32 ? "f32" : "f16", L.q_out_f32 ? "f32" : "f16", (int)L.int8, a.total_q, threads, a.B, a.Hq,
              a.Hkv, a.rot);
    switch (L.D) {
        case 64: append_types<64>(L, threads); break;
        case 128: append_types<128>(L, threads); break;
        default: append_types<256>(L, threads); break;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "append launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

attn_status launch_kv_read(const KvReadLaunch& L) {
    const KvReadArgs& a = L.args;
    const int rows = kReadRows * kReadWarps;
    const int grid = static_cast<int>((static_cast<long long>(a.total) + rows - 1) / rows);
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
