// latent_cache.cu -- the steps on either side of latent attention: writing new tokens'
// rows [c | rotated key part] into the cache and reading cached rows back.
//
// attn_latent_append, for a token at position p with latent vector c in R^R, key part k in
// R^64 and the query heads' parts q_h in R^64:
//
//   c'  = c * rsqrt(mean(c^2) + eps) * (w + offset)                 (optional)
//   z_a = y_a cos(p, e) - y_b sin(p, e),  z_b = y_b cos(p, e) + y_a sin(p, e)
//         for y = k and each q_h, over the pairs (e, e + 32) or (2e, 2e + 1), e < 32
//
// in f32 with one rounding to f16 at the end; row p of the cache is [c' | z of k].
//
// attn_latent_read is the way back, as packed c and key-part rows.
//
// Both move each byte once and compute a few operations on it: bound by memory, and small
// calls by the chain of dependent loads (sequence -> length -> page -> slot).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "cache_rows.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int E = 64;   // values of the rotated part

template <typename T>
struct Raw8 {
    Raw4<T> a, b;
    __device__ __forceinline__ void load(const T* p) {
        a.load(p);
        b.load(p + 4);
    }
    __device__ __forceinline__ void get(float2* x) const {
        a.get(x);
        b.get(x + 2);
    }
};
template <>
struct Raw8<__half> {
    uint4 r;
    __device__ __forceinline__ void load(const __half* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float2* x) const {
        x[0] = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
        x[1] = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
        x[2] = __half22float2(*reinterpret_cast<const __half2*>(&r.z));
        x[3] = __half22float2(*reinterpret_cast<const __half2*>(&r.w));
    }
};

// A CTA takes a token (blockIdx.x), or of few tokens a part of its turns (blockIdx.y of
// gridDim.y).  A warp's turn is the latent vector (a lane R/32 values of it, the norm a sum
// over the warp), or four rotated parts of 64 values (8 lanes each: the key's first, then the
// query heads'); a lane has both values of each pair it turns.
//
// Bound by latency (launch, and each warp's chain sequence, length, page, slot, table row): 2853
// tokens of 8 ragged chunks, 32 heads, f16: 6.8 us, 4.5 TB/s; 4096 f32 tokens of 16 heads 8.2 us,
// 4.9 TB/s; one token 2.0 us.
template <int R, typename T>
__global__ void __launch_bounds__(256) latent_append_kernel(const LatentAppendArgs a) {
    constexpr int NC = R / 256;      // 8-value pieces of the latent vector a lane
    const int lane = threadIdx.x & 31, t = blockIdx.x, sub = lane & 7;
    const int warps = blockDim.x >> 5, step = gridDim.y * warps;
    int turn = blockIdx.y * warps + (threadIdx.x >> 5);
    const int turns = 1 + (a.H + 1 + 3) / 4;
    const T* const ct = static_cast<const T*>(a.c) + t * a.c_stride;
    const T* const kt = static_cast<const T*>(a.k_rope) + t * a.k_stride;
    const T* const qt = static_cast<const T*>(a.q_rope) + t * a.q_stride;
    // elements of a lane's two quads
    const int ea = a.interleaved ? sub * 8 : sub * 4, eb = a.interleaved ? sub * 8 + 4 : E / 2 + sub * 4;
    // the first turn's loads go out before the search for the token's sequence, each later
    // turn's before the one before is worked on
    struct Pair {
        Raw4<T> a, b;
    } raw;
    Raw8<T> craw[NC];
    auto fetch = [&](int s) {
        if (s == 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) craw[i].load(ct + (i * 32 + lane) * 8);
        } else if (s < turns) {
            const int h = (s - 1) * 4 + (lane >> 3) - 1;   // -1: the key
            if (h < a.H) {
                const T* p = h < 0 ? kt : qt + h * a.q_head_stride;
                raw.a.load(p + ea);
                raw.b.load(p + eb);
            }
        }
    };
    fetch(turn);

    const Where w = find_row(a.q_start, a.kv_len, a.B, t, lane);
    if (w.b < 0) return;
    const long long p = static_cast<long long>(w.len) - w.end + t;   // kv_len - q_len + i
    if (p < 0) return;                   // no token: a padded batch's row
    if (p >= a.cache.capacity || (a.cos && p >= a.n_pos)) {
        if (threadIdx.x == 0) atomicExch(a.err, kErrAppendRange);
        return;
    }
    float2 cs[2], sn[2];
    if (a.cos) {
        const size_t at = static_cast<size_t>(p) * (E / 2) + sub * 4;
        load4(a.cos + at, cs);
        load4(a.sin + at, sn);
    }
    Slot slot{0, 0};
    const bool write = find_slot(a.cache, w.b, p, slot, a.err);
    __half* const x_row = static_cast<__half*>(a.x) + (slot.slot * a.cache.rows + slot.row) * (R + E);

    for (; turn < turns; turn += step) {   // uniform in the warp
        if (turn == 0) {
            float2 x[NC][4];
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                craw[i].get(x[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) s2 = ffma2(x[i][e], x[i][e], s2);
            }
            fetch(turn + step);
            if (a.c_norm) {
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
                const float r = rsqrtf(ss * (1.0f / R) + a.eps);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float2 g[4];
                    load4(a.c_norm + (i * 32 + lane) * 8, g);
                    load4(a.c_norm + (i * 32 + lane) * 8 + 4, g + 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[i][e] = fmul2(x[i][e], fmul2(fadd2(g[e], both(a.offset)), both(r)));
                }
            }
            if (write) {
#pragma unroll
                for (int i = 0; i < NC; ++i) store8(x_row + (i * 32 + lane) * 8, x[i]);
            }
            continue;
        }
        const int h = (turn - 1) * 4 + (lane >> 3) - 1;
        const bool live = h < a.H;
        float2 x[4] = {};
        if (live) {
            raw.a.get(x);
            raw.b.get(x + 2);
        }
        fetch(turn + step);
        if (a.cos) {
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c = (i & 1) ? cs[i / 2].y : cs[i / 2].x, n = (i & 1) ? sn[i / 2].y : sn[i / 2].x;
                    x[i] = ffma2(x[i], both(c), fmul2(make_float2(x[i].y, x[i].x), make_float2(-n, n)));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 u = x[i], v = x[2 + i], n = fmul2(v, sn[i]);
                    x[i] = ffma2(u, cs[i], make_float2(-n.x, -n.y));
                    x[2 + i] = ffma2(v, cs[i], fmul2(u, sn[i]));
                }
            }
        }
        if (live && (h >= 0 || write)) {
            __half* out = h < 0 ? x_row + R
                                : static_cast<__half*>(a.q_out) + t * a.q_out_stride + h * a.q_out_head_stride;
            store4(out + ea, x);
            store4(out + eb, x + 2);
        }
    }
}

// ------------------------------------------------------------------ read back
// A CTA takes `per` rows in a row: a lane each finds their places (a binary search over the
// sequences), then all threads copy 16-byte pieces, several at a time before their stores.  Bound
// by memory: 16 x 32768 tokens of 576 values to f16 179 us, 6.8 TB/s, what a copy takes, to f32 285 us,
// 6.35 TB/s; 37 tokens 2.5 us.  Few rows (less than 8 CTAs an SM of 32) are spread, 4 a CTA.
constexpr int kReadThreads = 256;
constexpr int kReadMost = 32;    // rows of a CTA
constexpr int kReadPieces = 4;   // pieces of a thread at a time

template <int R, typename TO>
__global__ void __launch_bounds__(kReadThreads) latent_read_kernel(const LatentReadArgs a, int per) {
    constexpr int PIECES = (R + E) / 8;
    __shared__ long long src[kReadMost];   // element offset of the row, -1: zeros, -2: not a row
    const long long t0 = static_cast<long long>(blockIdx.x) * per;
    const int n = static_cast<int>(min(static_cast<long long>(per), a.total - t0));
    if (static_cast<int>(threadIdx.x) < n) {
        const int t = static_cast<int>(t0) + threadIdx.x;
        int lo = 0, hi = a.B;            // the last sequence that starts at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.out_start[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int start = a.out_start[lo];
        long long at = -2;
        if (t >= start && t < a.out_start[lo + 1]) {
            const long long p = (a.first ? static_cast<long long>(a.first[lo]) : 0ll) + (t - start);
            Slot s{0, 0};
            at = -1;
            if (p >= 0 && p < a.kv_len[lo] && p < a.cache.capacity && find_slot(a.cache, lo, p, s, a.err))
                at = static_cast<long long>((s.slot * a.cache.rows + s.row) * (R + E));
        }
        src[threadIdx.x] = at;
    }
    __syncthreads();
    const __half* x = static_cast<const __half*>(a.x);
    for (int i0 = threadIdx.x; i0 < n * PIECES; i0 += kReadThreads * kReadPieces) {
        Raw8<__half> raw[kReadPieces];
        long long at[kReadPieces];
#pragma unroll
        for (int u = 0; u < kReadPieces; ++u) {
            const int i = i0 + u * kReadThreads;
            at[u] = i < n * PIECES ? src[i / PIECES] : -2;
            raw[u].r = make_uint4(0u, 0u, 0u, 0u);
            if (at[u] >= 0) raw[u].load(x + at[u] + (i % PIECES) * 8);
        }
#pragma unroll
        for (int u = 0; u < kReadPieces; ++u) {
            if (at[u] == -2) continue;
            const int i = i0 + u * kReadThreads, piece = i % PIECES;
            const long long t = t0 + i / PIECES;
            float2 v[4];
            raw[u].get(v);
            TO* out = piece < R / 8 ? static_cast<TO*>(a.c_out) + t * R + piece * 8
                                    : static_cast<TO*>(a.k_out) + t * E + (piece - R / 8) * 8;
            store8(out, v);
        }
    }
}

template <int R>
void append_types(const LatentAppendLaunch& L, dim3 grid, int threads) {
    if (L.in_f32) latent_append_kernel<R, float><<<grid, threads, 0, L.stream>>>(L.args);
    else latent_append_kernel<R, __half><<<grid, threads, 0, L.stream>>>(L.args);
}
template <int R>
void read_types(const LatentReadLaunch& L, int grid, int per) {
    if (L.out_f32) latent_read_kernel<R, float><<<grid, kReadThreads, 0, L.stream>>>(L.args, per);
    else latent_read_kernel<R, __half><<<grid, kReadThreads, 0, L.stream>>>(L.args, per);
}

}  // namespace

attn_status launch_latent_append(const LatentAppendLaunch& L) {
    const LatentAppendArgs& a = L.args;
    // A call of many tokens gives each a CTA of warps with up to 16 turns, or 4 of f32 (whose loads
    // are twice as many): 2853 f16 tokens of 10 turns take 9.2, 8.2, 7.6 and 6.8 us with up to 2, 4,
    // 8 and 16 turns a warp, 4096 f32 tokens of 6 turns 9.2, 8.2 and 8.8 with 2, 4 and 8 (several
    // tokens a CTA: no faster).  Of few tokens (fewer than two an SM) CTAs of at most 8 warps, a turn
    // each, several a token.
    const int turns = 1 + (a.H + 1 + 3) / 4, each = L.in_f32 ? 4 : 16;
    const bool many = a.total_q >= 2 * sm_count();
    const int most = many ? (turns + each - 1) / each : turns, warps = most < 8 ? most : 8;
    const int parts = many ? 1 : (turns + warps - 1) / warps;
    const dim3 grid(a.total_q, parts < 65535 ? parts : 65535);   // (gridDim.y; the rest in turn)
    if (trace_enabled())
        trace("latent_append_kernel<R=%d,in=%s> grid=(%u,%u) block=%d B=%d H=%d", L.R, L.in_f32 ? "f32" : "f16", grid.x,
              grid.y, warps * 32, a.B, a.H);
    if (L.R == 256) append_types<256>(L, grid, warps * 32);
    else append_types<512>(L, grid, warps * 32);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "latent append launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

attn_status launch_latent_read(const LatentReadLaunch& L) {
    const LatentReadArgs& a = L.args;
    const int per = a.total >= 8 * sm_count() * kReadMost ? kReadMost : 4;
    const int grid = (a.total - 1) / per + 1;
    if (trace_enabled())
        trace("latent_read_kernel<R=%d,out=%s> grid=%d block=%d rows=%d B=%d", L.R, L.out_f32 ? "f32" : "f16", grid,
              kReadThreads, per, a.B);
    if (L.R == 256) read_types<256>(L, grid, per);
    else read_types<512>(L, grid, per);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "latent read launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

}  // namespace attn
