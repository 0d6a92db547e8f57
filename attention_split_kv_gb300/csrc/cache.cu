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

#include <type_traits>

#include "attn_internal.h"
#include "cache_rows.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

// ------------------------------------------------------------------ append
// max(a, |b|, |c|), NaN if any is
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return d;
}

// Four codes of r = x / scale: rint(x * inv) sits in the low bits of x * inv + 1.5 * 2^23.
// x * inv is within 2^-24 * 127.1 < 1e-5 of x / scale, so it rounds alike unless it is that
// near to a tie; `tie` collects the distances from the integers.
__device__ __forceinline__ uint32_t codes4(const float2* x, float inv, float& tie) {
    constexpr float kMagic = 12582912.0f;
    float2 r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r[i] = ffma2(x[i], both(inv), both(kMagic));
        const float2 d = ffma2(x[i], both(inv), ffma2(r[i], both(-1.f), both(kMagic)));
        tie = fmaxf(tie, fmaxf(fabsf(d.x), fabsf(d.y)));
    }
    return __byte_perm(__byte_perm(__float_as_uint(r[0].x), __float_as_uint(r[0].y), 0x0040),
                       __byte_perm(__float_as_uint(r[1].x), __float_as_uint(r[1].y), 0x0040), 0x5410);
}
// The same by division, clamped (near a tie, or under a scale too small to be accurate).
__device__ __forceinline__ uint32_t codes4_exact(const float2* x, float scale) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = (i & 1) ? x[i / 2].y : x[i / 2].x;
        const float r = fminf(fmaxf(rintf(__fdiv_rn(v, scale)), -127.f), 127.f);
        c |= (static_cast<uint32_t>(static_cast<int>(r)) & 0xffu) << (8 * i);
    }
    return c;
}

// A CTA takes a token (blockIdx.x), or of few tokens a part of its heads (blockIdx.y of
// gridDim.y); a group of D/8 lanes a head at a time, a warp heads of one kind (q, k or v).
// A lane has two quads of 4 elements: those that half-split rotation pairs, or neighbours,
// so that a rotation stays inside a lane; the norm and the largest magnitude are shuffles
// inside the group.  A lane's first loads are issued before the search for the token's
// sequence, each later one before the head before is worked on, so that the chain of
// dependent loads (sequence, page, table row) lies under them (two heads ahead: no faster).
//
// Bound by instructions and by each warp's chain (load, two reductions over the lanes, two
// divisions, store): 2853 tokens of 32 + 2 x 8 heads (D = 128, f16 to int8 pages) take 22 us,
// 3.0 TB/s, with 217 instructions a warp's turn, issue slots 67% and DRAM 20% (half of the
// bytes stay in L2); 4096 tokens of 8 + 2 x 4 heads (D = 256, f32, ring) 20 us, 4.5 TB/s.
// With 48 registers (more warps, some spills) 24 and 24 us.
template <int D, typename T, typename TQ, bool INT8>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
    constexpr int LPR = D / 8;          // lanes a head
    constexpr int RPW = 32 / LPR;       // heads a warp
    const int lane = threadIdx.x & 31, t = blockIdx.x;
    const int sub = lane & (LPR - 1), hsub = lane / LPR;
    const int half = a.rot / 2;
    const bool rotates = sub * 8 < a.rot;
    // elements of the two quads: (e, e + R/2) for the first R/8 lanes of a half-split
    // rotation, else 8 in a row
    const bool split = !a.interleaved && rotates;
    const int ea = split ? sub * 4 : sub * 8, eb = split ? half + sub * 4 : sub * 8 + 4;

    const int nq = (a.Hq + RPW - 1) / RPW, nk = (a.Hkv + RPW - 1) / RPW, n_slots = nq + 2 * nk;
    const int step = gridDim.y * (blockDim.x >> 5);
    int slot_i = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const T* const qt = static_cast<const T*>(a.q) + t * a.q_stride;
    const T* const kt = static_cast<const T*>(a.k) + t * a.k_stride;
    const T* const vt = static_cast<const T*>(a.v) + t * a.v_stride;
    struct Pair {
        Raw4<T> a, b;
    };
    auto fetch = [&](int s, Pair& r) {
        const int kind = s < nq ? 0 : s < nq + nk ? 1 : 2;
        const int h = (s - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * RPW + hsub;
        if (s >= n_slots || h >= (kind == 0 ? a.Hq : a.Hkv)) return;
        const T* p = (kind == 0 ? qt : kind == 1 ? kt : vt) + h * D;
        r.a.load(p + ea);
        r.b.load(p + eb);
    };
    Pair raw;
    fetch(slot_i, raw);

    const Where w = find_row(a.q_start, a.kv_len, a.B, t, lane);
    if (w.b < 0) return;
    const long long p = static_cast<long long>(w.len) - w.end + t;   // kv_len - q_len + i
    if (p < 0) return;                   // no token: a padded batch's row
    if (p >= a.cache.capacity || (a.rot > 0 && p >= a.n_pos)) {
        if (threadIdx.x == 0) atomicExch(a.err, kErrAppendRange);
        return;
    }
    float2 cs[2], sn[2];
    if (rotates) {
        const size_t at = static_cast<size_t>(p) * half + sub * 4;
        load4(a.cos + at, cs);
        load4(a.sin + at, sn);
    }
    // a ring holds a sequence's newest tokens; what a longer chunk overwrites is not
    // written at all, so no two tokens of a call share a slot
    bool write = a.cache.ring == 0 || p >= static_cast<long long>(w.len) - a.cache.ring;
    Slot slot{0, 0};
    if (write) write = find_slot(a.cache, w.b, p, slot, a.err);
    const size_t row = (slot.slot * a.cache.rows + slot.row) * a.Hkv;        // in heads
    const size_t srow = slot.slot * a.Hkv * a.cache.rows + slot.row;         // of scales, head 0

    int g_kind = 2;
    float2 g[4];                         // the norm's weights, where g_kind has any
    for (; slot_i < n_slots; slot_i += step) {   // uniform in the warp, kind too
        const int kind = slot_i < nq ? 0 : slot_i < nq + nk ? 1 : 2;
        const int h = (slot_i - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * RPW + hsub;
        const bool live = h < (kind == 0 ? a.Hq : a.Hkv);
        float2 x[4] = {};
        if (live) {
            raw.a.get(x);
            raw.b.get(x + 2);
        }
        fetch(slot_i + step, raw);
        const float* nw = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
        if (nw) {
            if (g_kind != kind) {
                load4(nw + ea, g);
                load4(nw + eb, g + 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = fadd2(g[i], both(a.offset));
                g_kind = kind;
            }
            float2 s2 = fmul2(x[0], x[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) s2 = ffma2(x[i], x[i], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = fmul2(x[i], fmul2(g[i], both(r)));
        }
        if (kind < 2 && rotates) {
            if (split) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 u = x[i], v = x[2 + i], n = fmul2(v, sn[i]);
                    x[i] = ffma2(u, cs[i], make_float2(-n.x, -n.y));
                    x[2 + i] = ffma2(v, cs[i], fmul2(u, sn[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c = (i & 1) ? cs[i / 2].y : cs[i / 2].x, n = (i & 1) ? sn[i / 2].y : sn[i / 2].x;
                    x[i] = ffma2(x[i], both(c), fmul2(make_float2(x[i].y, x[i].x), make_float2(-n, n)));
                }
            }
        }
        if (kind == 0) {
            if (live) {
                TQ* out = static_cast<TQ*>(a.q_out) + (static_cast<size_t>(t) * a.Hq + h) * D;
                store4(out + ea, x);
                store4(out + eb, x + 2);
            }
            continue;
        }
        if constexpr (INT8) {
            // a head with an infinity or a NaN gets it as its scale
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max3_abs_nan(m, x[i].x, x[i].y);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = max3_abs_nan(m, __shfl_xor_sync(kFull, m, o), 0.f);
            const __half hs = __float2half_rn(__fdiv_rn(m, 127.0f));
            const float scale = __half2float(hs);
            uint32_t c0 = 0, c1 = 0;
            if (scale > 0.f && scale < INFINITY) {
                // an f16 scale with all its bits puts every code within 127.1
                float tie = 0.f;
                const float inv = __frcp_rn(scale);
                c0 = codes4(x, inv, tie);
                c1 = codes4(x + 2, inv, tie);
                if (tie > 0.4999f || scale < 0x1p-14f) {
                    c0 = codes4_exact(x, scale);
                    c1 = codes4_exact(x + 2, scale);
                }
            }
            if (live && write) {
                int8_t* out = static_cast<int8_t*>(kind == 1 ? a.k_cache : a.v_cache) + (row + h) * D;
                *reinterpret_cast<uint32_t*>(out + ea) = c0;
                *reinterpret_cast<uint32_t*>(out + eb) = c1;
                if (sub == 0)
                    static_cast<__half*>(kind == 1 ? a.k_scales : a.v_scales)[srow + static_cast<size_t>(h) * a.cache.rows] =
                        hs;
            }
        } else if (live && write) {
            __half* out = static_cast<__half*>(kind == 1 ? a.k_cache : a.v_cache) + (row + h) * D;
            store4(out + ea, x);
            store4(out + eb, x + 2);
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
// A warp takes a row, or 32 U pieces of one (ONE: no more than those); a lane pieces of E
// elements, one load each, U at a time, all loads before the first store.  Pieces of 16 codes
// become 32 bytes of f16, those of 8 codes or f16 values 16 or 32 bytes, so neighbouring lanes
// fill whole sectors.  Bound by DRAM: 16 x 32768 int8 tokens of 8 heads to f16 take 473 us,
// 6.8 TB/s, what a copy takes; 8 x 32768 f16 tokens to f32 478 us (555 with 64 bytes a lane);
// 4158 ring tokens of 4 heads (D = 256) to f32 12 us, the launch and the search included.
constexpr int kReadWarps = 8;
constexpr int kReadPieces = 4;   // U

template <bool INT8, typename TO>
constexpr int read_piece() { return INT8 && sizeof(TO) == 2 ? 16 : 8; }   // E

template <typename TO, bool INT8, bool ONE>
__global__ void __launch_bounds__(kReadWarps * 32) kv_read_kernel(const KvReadArgs a) {
    constexpr int E = read_piece<INT8, TO>(), U = kReadPieces;
    constexpr int W = INT8 ? E / 4 : E / 2;   // words of a piece
    using Raw = typename std::conditional<W == 4, uint4, uint2>::type;
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
    if (t >= a.total) return;
    const int log_d = (a.D == 64 ? 6 : a.D == 128 ? 7 : 8) - (E == 16 ? 4 : 3);   // log2 of a head's pieces
    const int per = a.Hkv << log_d;                                               // pieces of a token's K (or V)
    const Where w = find_row(a.out_start, a.kv_len, a.B, static_cast<int>(t), lane);
    if (w.b < 0) return;
    const long long p = (a.first ? static_cast<long long>(a.first[w.b]) : 0ll) + (t - w.start);
    bool held = p >= 0 && p < w.len && p < a.cache.capacity &&
                (a.cache.ring == 0 || p >= static_cast<long long>(w.len) - a.cache.ring);
    Slot slot{0, 0};
    if (held) held = find_slot(a.cache, w.b, p, slot, a.err);
    const size_t src = (slot.slot * a.cache.rows + slot.row) * a.Hkv * a.D;
    const size_t dst = static_cast<size_t>(t) * a.Hkv * a.D;
    for (int c0 = blockIdx.y * 32 * U + lane; c0 < 2 * per; c0 += 32 * U) {
        union {
            Raw v;
            uint32_t w[W];
        } raw[U];
        __half sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 32 * u;
            const bool is_k = c < per;
            const int cc = is_k ? c : c - per;
            sc[u] = __float2half_rn(0.f);
            if (c >= 2 * per || !held) {
                raw[u].v = Raw{};
            } else if constexpr (INT8) {
                raw[u].v = *reinterpret_cast<const Raw*>(static_cast<const int8_t*>(is_k ? a.k_cache : a.v_cache) + src +
                                                         static_cast<size_t>(cc) * E);
                sc[u] = static_cast<const __half*>(
                    is_k ? a.k_scales : a.v_scales)[(slot.slot * a.Hkv + (cc >> log_d)) * a.cache.rows + slot.row];
            } else {
                raw[u].v = *reinterpret_cast<const Raw*>(static_cast<const __half*>(is_k ? a.k_cache : a.v_cache) + src +
                                                         static_cast<size_t>(cc) * E);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 32 * u;
            if (c >= 2 * per) break;
            const bool is_k = c < per;
            TO* out = static_cast<TO*>(is_k ? a.k_out : a.v_out) + dst + static_cast<size_t>(is_k ? c : c - per) * E;
            const float2 s = both(__half2float(sc[u]));
#pragma unroll
            for (int e = 0; e < E; e += 8) {
                float2 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (INT8) {
                        const uint32_t w2 = raw[u].w[(e + 2 * i) / 4] >> (16 * (i & 1));
                        x[i] = fmul2(make_float2(static_cast<float>(static_cast<int8_t>(w2)),
                                                 static_cast<float>(static_cast<int8_t>(w2 >> 8))), s);
                    } else {
                        x[i] = __half22float2(*reinterpret_cast<const __half2*>(&raw[u].w[i]));
                    }
                }
                store8(out + e, x);
            }
        }
        if (ONE) break;
    }
}

template <typename TO, bool INT8>
void read_dispatch(const KvReadLaunch& L) {
    const KvReadArgs& a = L.args;
    // Few rows (less than two waves of warps) are shared by warps that load all of their pieces
    // at once: 13.5 us with a warp a row, 12.0 shared, for 4158 rows of 2 x 1024 f16 values to
    // f32; of 262144 rows of that size 478 and 517.  Rows of at most a piece a lane take the
    // form without a loop too, for its registers (more warps): 524288 rows of 32 pieces 200 us
    // with the loop, 167 without; of 64 pieces 277 and 288, of 128 pieces 473 and 540.
    const int pieces = 2 * a.Hkv * a.D / read_piece<INT8, TO>();
    const int passes = (pieces + 32 * kReadPieces - 1) / (32 * kReadPieces);
    const bool one = passes <= 65535 && (pieces <= 32 || a.total < 64 * sm_count());   // (gridDim.y)
    const dim3 grid((a.total - 1) / kReadWarps + 1, one ? passes : 1);
    if (trace_enabled())
        trace("kv_read_kernel<out=%s,int8=%d> one_pass=%d grid=(%u,%u) block=%d B=%d Hkv=%d D=%d", L.out_f32 ? "f32" : "f16",
              (int)INT8, (int)one, grid.x, grid.y, kReadWarps * 32, a.B, a.Hkv, a.D);
    if (one) kv_read_kernel<TO, INT8, true><<<grid, kReadWarps * 32, 0, L.stream>>>(a);
    else kv_read_kernel<TO, INT8, false><<<grid, kReadWarps * 32, 0, L.stream>>>(a);
}

}  // namespace

attn_status launch_append(const AppendLaunch& L) {
    const AppendArgs& a = L.args;
    // One CTA a token, of warps with 8 turns each: what a warp does once (the search, the
    // addresses) costs it as much as a turn and a half.  Ragged chunks of 48 heads: 25 us with 8
    // warps, 22 with 3; 4096 tokens of 16 wide f32 heads: 27 with 8, 20 with 2.  A call with
    // fewer tokens than two an SM has latency to lose instead: CTAs of at most 8 warps, a turn
    // each.
    const int rpw = 256 / L.D;
    const int turns = (a.Hq + rpw - 1) / rpw + 2 * ((a.Hkv + rpw - 1) / rpw);   // warps' worth of heads
    const bool many = a.total_q >= 2 * sm_count();
    const int most = many ? (turns + 7) / 8 : turns, warps = most < 8 ? most : 8, threads = warps * 32;
    const int parts = many ? 1 : min((turns + warps - 1) / warps, 65535);   // (gridDim.y; the rest in turn)
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
    if (L.int8) {
        if (L.out_f32) read_dispatch<float, true>(L);
        else read_dispatch<__half, true>(L);
    } else {
        if (L.out_f32) read_dispatch<float, false>(L);
        else read_dispatch<__half, false>(L);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "kv_read launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

}  // namespace attn
