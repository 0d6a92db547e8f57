// latent_run.cuh -- what the kernels of attn_latent_attend share: the call's arguments, a run's walk
// over its key tiles, where a segment's rows go, and the kernel that joins cut rows.
//
// The key tiles of all (sequence, group of row blocks) items, in that order, are cut into equal
// runs, one a unit (a CTA or a pair of CTAs).  A unit walks its run a segment, the part of one item,
// at a time; rows of items cut by a run's end go to the workspace.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int BN = 64;                      // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;
// A row's weights are 2^(logit - its offset), in f16 for the second product.  The offset lies kLift below the
// row's maximum when it is set, and is set again when a logit passes it by kRescaleThreshold (log2 units): the
// largest weight is 2^7 to 2^15 (f16 holds 65504), and of the others what is above 2^-25 is kept, 2^-32 or less
// of the largest.  (At offset 0 it was 2^-25: one key beside 65 thousand of e^-18 each lost all of their 0.1%.)
constexpr float kLift = 7.0f, kRescaleThreshold = 15.0f;
constexpr float kFastSumLimit = 32768.0f;   // weights that sum to at most this are at most 2^15
constexpr int kMaxCtas = 152;               // one CTA an SM
constexpr int kWholeTiles = 4;              // items of at most this many tiles are not cut
constexpr uint32_t kChunk = BN * 128;       // bytes of 64 values of a tile

struct Args {
    const int32_t *q_start, *kv_len, *page_table;
    __half* out;
    float* lse;
    float* part_o;       // [unit][2][NR][R]
    float2* part_ml;     // [unit][2][NR]
    int* meta;           // [unit][4]
    int* err;
    int B, total_q, max_q, H;
    int log2P, max_pages, n_slots, log_nb;   // 2^log_nb boxes a tile; slots: pages, or the contiguous cache's sequences
    int n_rb;            // row blocks of the longest chunk
    int side;            // row blocks of a sequence that neighbouring units take side by side
    int capacity;
    int whole;           // items are not cut
    float scale;
};

// One sequence's new tokens.  (Rows, tokens x heads, stay below 2^31: the host checks.)
struct Chunk {
    int q_base, n, pos0, L;   // first token row, tokens computed, position of token 0, cached keys
};
__device__ __forceinline__ Chunk load_chunk(const Args& a, int b) {
    Chunk c;
    c.q_base = a.q_start[b];
    const int n_q = max(a.q_start[b + 1] - c.q_base, 0), len = a.kv_len[b];
    c.n = min(n_q, a.max_q);
    c.pos0 = len - n_q;
    c.L = min(max(len, 0), a.capacity);
    return c;
}
// groups of row blocks that are taken side by side (more than one block only where every chunk
// is one token: one group)
template <int NR>
__device__ __forceinline__ int groups_of(const Args& a, const Chunk& c) {
    return a.side > 1 ? min(c.n, 1) : static_cast<int>((static_cast<uint32_t>(c.n * a.H) + NR - 1) / NR);
}
// keys that some row of the rows up to `end` (not included) keeps lie below this
__device__ __forceinline__ int key_end(const Args& a, const Chunk& c, uint32_t end) {
    const uint32_t last = min(end, static_cast<uint32_t>(c.n * a.H)) - 1;
    const long long token = c.n > 1 ? last / static_cast<uint32_t>(a.H) : 0;
    return static_cast<int>(max(0ll, min(static_cast<long long>(c.L), c.pos0 + token + 1)));
}
template <int NR>
__device__ __forceinline__ int group_tiles(const Args& a, const Chunk& c, int g) {
    return max((key_end(a, c, static_cast<uint32_t>(g + 1) * (a.side * NR)) + BN - 1) / BN, 1);
}

// A unit's run, walked a segment (part of one item) at a time; every warp walks for itself.  A run
// is a range of weights: an item weighs its key tiles and SEG before them.
struct Walk {
    int b, g;            // sequence, group of row blocks
    long long in, rem;   // where the run enters the item; its weight from there on
    int off, n, tiles;   // first key tile and key tiles of the segment; key tiles of the item
    Chunk c;
};
// (b, g, in, rem and the item's chunk and tiles are there)
template <int SEG>
__device__ __forceinline__ bool walk_item(const Args& a, Walk& w) {
    if (w.rem <= 0) return false;
    w.off = a.whole ? 0 : max(static_cast<int>(w.in) - SEG, 0);
    w.n = (a.whole ? w.tiles : static_cast<int>(min(static_cast<long long>(w.tiles), w.in + w.rem - SEG))) - w.off;
    return w.n > 0;
}
template <int NR, int SEG>
__device__ __forceinline__ bool walk_next(const Args& a, Walk& w) {
    w.rem -= w.tiles + SEG - w.in;
    w.in = 0;
    if (w.rem <= 0) return false;
    if (++w.g >= groups_of<NR>(a, w.c)) {
        w.g = 0;
        do {
            if (++w.b >= a.B) return false;
            w.c = load_chunk(a, w.b);
        } while (w.c.n == 0);
    }
    w.tiles = group_tiles<NR>(a, w.c, w.g);
    return walk_item<SEG>(a, w);
}
template <int NR, int SEG>
__device__ __forceinline__ bool walk_first(const Args& a, Walk& w) {
    const bool on = walk_item<SEG>(a, w);
    return on && a.whole && w.in > 0 ? walk_next<NR, SEG>(a, w) : on;   // (whole items: those that start in the run)
}

// What a run's start depends on, on its way into L2 before the kernels before this one have ended (nothing
// is read): a miss costs 2500 cycles, and three lie one behind another.  (With the chunk kept from the
// search: one token 6.7 to 6.5 us, 16 heads 35.1 to 34.7.)
__device__ __forceinline__ void prefetch_run(const Args& a, int threads) {
    for (int b = threadIdx.x; b <= a.B; b += threads) {
        prefetch_l2(a.q_start + b);
        if (b == a.B) break;
        prefetch_l2(a.kv_len + b);
        if (a.page_table) prefetch_l2(a.page_table + static_cast<size_t>(b) * a.max_pages);
    }
}

template <int THREADS>
constexpr int kRunWords = THREADS / 32 + 5;   // of 8 bytes: find_run's scratch
// The run of unit `unit` of `units`, found by the whole block of THREADS threads (two __syncthreads, the
// first with the tcgen05 fences for what the caller has set up).
template <int NR, int SEG, int THREADS>
__device__ __forceinline__ Walk find_run(const Args& a, int unit, int units, long long* sums) {
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    Walk run;
    constexpr int kWarps = THREADS / 32;   // sums: of the warps, then where the run starts
    int* first = reinterpret_cast<int*>(sums + kWarps + 1);
    const int max_g = a.side > 1 ? 1 : a.n_rb;
    const long long items = static_cast<long long>(a.B) * max_g, per = (items + THREADS - 1) / THREADS;
    const long long f0 = min(items, tid * per), f1 = min(items, f0 + per);
    // visits this thread's items in order until fn says stop
    auto visit = [&](auto fn) {
        if (f0 >= f1) return;
        int b = static_cast<int>(max_g == 1 ? f0 : f0 / max_g);
        int g = max_g == 1 ? 0 : static_cast<int>(f0 - static_cast<long long>(b) * max_g);
#pragma unroll 1
        for (long long left = f1 - f0; left > 0; ++b) {
            const Chunk c = load_chunk(a, b);
            const int end = static_cast<int>(min(static_cast<long long>(groups_of<NR>(a, c)), g + left));
#pragma unroll 1
            for (int i = g; i < end; ++i)
                if (!fn(b, i, group_tiles<NR>(a, c, i) + SEG)) return;
            left -= max_g - g;
            g = 0;
        }
    };
    long long mine = 0;
    visit([&](int, int, int weight) {
        mine += weight;
        return true;
    });
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) sums[warp] = before;
    before -= mine;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += sums[i];
        total += sums[i];
    }
    // as many runs as units, or fewer of a key tile at least (a run's weight is above SEG)
    const int runs = total >= static_cast<long long>(units) * (SEG + 1) ? units : max(1, static_cast<int>(total) / (SEG + 1));
    const long long each = total < (1ll << 31) ? static_cast<uint32_t>(total) / static_cast<uint32_t>(runs) : total / runs;
    const int more = static_cast<int>(total - each * runs);   // the first ones have one more
    const long long t = each * unit + min(unit, more);
    if (unit < runs && before <= t && t < before + mine) {
        long long at = before;
        visit([&](int b, int g, int weight) {
            if (at + weight <= t) {
                at += weight;
                return true;
            }
            sums[kWarps] = t - at;
            const Chunk c = load_chunk(a, b);
            first[0] = b;
            first[1] = g;
            first[2] = c.q_base;
            first[3] = c.n;
            first[4] = c.pos0;
            first[5] = c.L;
            first[6] = weight - SEG;
            return false;
        });
    }
    __syncthreads();
    run.b = first[0];
    run.g = first[1];
    run.c = Chunk{first[2], first[3], first[4], first[5]};
    run.tiles = first[6];
    run.in = sums[kWarps];
    run.rem = unit < runs && total > 0 ? each + (unit < more) : 0;
    return run;
}

// Where a segment's rows go: to out, or as a part to the workspace.
struct Out {
    long long row0;   // first row of out
    int n, part;      // rows written; place of the part
    bool whole;       // all of the item: to out
};
template <int NR>
__device__ __forceinline__ Out out_of(const Args& a, const Walk& w, uint32_t row0, int unit) {
    const long long live = static_cast<long long>(w.c.n) * a.H - row0, end = static_cast<long long>(a.total_q) * a.H;
    Out o;
    o.row0 = static_cast<long long>(w.c.q_base) * a.H + row0;
    o.n = o.row0 < 0 ? 0 : static_cast<int>(max(0ll, min(min(live, static_cast<long long>(NR)), end - o.row0)));
    o.part = unit * 2 + (w.off > 0 ? 0 : 1);
    o.whole = w.n == w.tiles;
    return o;
}

// Joins the partial rows of the items that run over a unit's boundary: block (c, y) takes the
// item that unit c leaves open, and of its rows those of chunk y.  A warp takes a row, or of few
// rows 128 values of one (join_width); all of its parts' loads are issued before the first is used.
constexpr int kJoinWarps = 4;
// 128-value blocks a warp (16 rows: 40.5 us with one, 42.5 with four; 64 rows: 70.0 and 66.0)
constexpr int join_width(int NP, int NR) { return NR >= 64 ? NP : 1; }

// (in the order they are written in: left to the compiler, each load is waited for before the next)
__device__ __forceinline__ float4 load_in_order(const float* p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

template <int NP, int NR>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const Args a, int n_units) {
    constexpr int R = NP * 128, NW = join_width(NP, NR), AT = NW == 1 ? 8 : 4;   // parts at a time
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the next call's attention waits for this kernel)
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for the whole of the attention kernel
    const int unit = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int row = unit * NW / NP, d0 = unit * NW % NP * 128 + lane * 4;
    const int4 meta = *reinterpret_cast<const int4*>(a.meta + blockIdx.x * 4);
    const size_t orow = static_cast<size_t>(static_cast<uint32_t>(meta.z)) + row;
    // The parts: the end of unit c's run, whole runs of the same item, the beginning of the last.  A
    // lane each reads their statistics (32 at a time), then all read their values.
    float2 o[2 * NW];
#pragma unroll
    for (int e = 0; e < 2 * NW; ++e) o[e] = make_float2(0.f, 0.f);
    float sum = 0.f, mx = -INFINITY;
    for (int c0 = blockIdx.x, ended = 0; !ended && c0 < n_units; c0 += 32 * a.side) {
        const int i = c0 + lane * a.side;
        const bool first = i == static_cast<int>(blockIdx.x);
        float2 x = make_float2(-INFINITY, 0.f);
        int end = 0;
        if (i < n_units) {
            x = a.part_ml[(static_cast<size_t>(i) * 2 + first) * NR + row];
            end = !first && a.meta[i * 4];
        }
        if (row >= meta.y) return;   // (looked at beside the first loads, whose addresses do not need it)
        const unsigned ends = __ballot_sync(0xffffffffu, end);
        int n = min(32, (n_units - c0 + a.side - 1) / a.side);
        if (ends) {
            n = min(n, __ffs(ends));
            ended = 1;
        }
        if (lane >= n) x = make_float2(-INFINITY, 0.f);
        float top = x.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        top = fmaxf(top, mx);
        const float old = mx == -INFINITY ? 0.f : ex2_approx(mx - top);
        const float f = x.x == -INFINITY ? 0.f : ex2_approx(x.x - top);
        mx = top;
        float part = f * x.y;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) part += __shfl_xor_sync(0xffffffffu, part, s);
        sum = fmaf(sum, old, part);
#pragma unroll
        for (int e = 0; e < 2 * NW; ++e) o[e] = fmul2(o[e], make_float2(old, old));
        for (int k0 = 0; k0 < n; k0 += AT) {
            float4 v[AT][NW];
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const int j = c0 + min(k0 + k, n - 1) * a.side;   // (past the last part: the last again, times 0)
                const float* src = a.part_o + ((static_cast<size_t>(j) * 2 + (j == static_cast<int>(blockIdx.x))) * NR + row) * R + d0;
#pragma unroll
                for (int e = 0; e < NW; ++e)
                    v[k][e] = load_in_order(src + e * 128);
            }
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const float g = __shfl_sync(0xffffffffu, k0 + k < n ? f : 0.f, (k0 + k) & 31);
#pragma unroll
                for (int e = 0; e < NW; ++e) {
                    o[2 * e] = ffma2(make_float2(v[k][e].x, v[k][e].y), make_float2(g, g), o[2 * e]);
                    o[2 * e + 1] = ffma2(make_float2(v[k][e].z, v[k][e].w), make_float2(g, g), o[2 * e + 1]);
                }
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < NW; ++e) {
        const __half2 h0 = __floats2half2_rn(o[2 * e].x * inv, o[2 * e].y * inv);
        const __half2 h1 = __floats2half2_rn(o[2 * e + 1].x * inv, o[2 * e + 1].y * inv);
        *reinterpret_cast<uint2*>(a.out + orow * R + d0 + e * 128) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    }
    if (a.lse && d0 == 0) a.lse[orow] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.6931471805599453f;
}

// Rows of a block, blocks of the longest chunk, and the workspace: partial rows, their
// statistics, a description a CTA.
struct Plan {
    int NR;
    long long n_rb;
    size_t off_ml, off_meta, bytes;
};
Plan make_plan(int max_q, int H, int R) {
    Plan p;
    const long long rows = static_cast<long long>(max_q) * H;
    p.NR = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    p.n_rb = (rows + p.NR - 1) / p.NR;
    const size_t slots = static_cast<size_t>(kMaxCtas) * 2 * p.NR;
    p.off_ml = slots * R * 4;
    p.off_meta = (p.off_ml + slots * 8 + 255) / 256 * 256;
    p.bytes = p.off_meta + (kMaxCtas * 16 + 255) / 256 * 256;
    return p;
}
// The kernels' arguments (all but those of the tensor maps).
void fill_args(const LatentAttendLaunch& L, const Plan& p, Args& a) {
    uint8_t* ws = static_cast<uint8_t*>(L.workspace);
    a.q_start = L.q_start;
    a.kv_len = L.kv_len;
    a.page_table = L.cache.page_table;
    a.n_slots = L.cache.page_table ? L.cache.n_pages : L.B;
    a.log_nb = 0;
    while (L.cache.page_table && (BN >> a.log_nb) > L.cache.rows) ++a.log_nb;
    a.out = static_cast<__half*>(L.out);
    a.lse = L.lse;
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + p.off_ml);
    a.meta = reinterpret_cast<int*>(ws + p.off_meta);
    a.err = L.err_word;
    a.B = L.B;
    a.total_q = L.total_q;
    a.max_q = L.max_q;
    a.H = L.H;
    a.log2P = L.cache.log2P;
    a.max_pages = L.cache.max_pages;
    a.capacity = static_cast<int>(L.cache.capacity < 0x7ffff000ll ? L.cache.capacity : 0x7ffff000ll);
    a.n_rb = static_cast<int>(p.n_rb);
    // One token of many heads: neighbouring units take its row blocks side by side, so that the second one
    // finds the cache's rows in L2
    a.side = L.max_q == 1 && p.n_rb <= 8 ? static_cast<int>(p.n_rb) : 1;
    a.scale = L.scale;
    // Short caches: items of few tiles are not cut, and nothing is to be joined.  That goes by what the cache
    // can hold, since the lengths are not known here (one token over 128 keys: 6.7 us in a table of 256
    // tokens, 9.6 with the second kernel in one of 32768)
    a.whole = a.capacity <= kWholeTiles * BN;
}

}  // namespace
}  // namespace attn
