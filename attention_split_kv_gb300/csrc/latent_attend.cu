// latent_attend.cu -- the absorbed form of latent attention (attn_latent_attend) on the
// sm_103a tensor cores: a token's key for every head is its cached row x_j = [c_j | r_j]
// (c the latent vector of R values, r the rotated part of 64), its value is c_j.
//
//   o_ih = sum_j softmax_j(scale q_ih . x_j) c_j      over the keys j <= pos_i
//
// The heads of a sequence's new tokens share the cache's rows, so (token, head) pairs are
// simply rows of one matrix, token-major as q lies in memory, cut into blocks of NR.
//
// The keys are the MMA's M side, the rows its N side:
//
//   S^T = X Q^T      128 keys x NR     (tcgen05.mma, X as it lies: K-major)
//   P^T = 2^(S^T scale log2e - m)      f16, to shared memory: a key's NR weights are one line
//   O^T += C^T P^T   R x NR            (C^T as X's same tile read MN-major, 128 values a block)
//
// so a tile of 128 keys comes from memory once and serves both products, few rows (one
// token of 16 heads) cost MMAs of N = 16 and not of 128 padded rows, and O^T of 512 values
// fits TMEM beside S^T for up to 64 rows (4 x 64 columns + 64).
//
// A row's weights lie along the lanes, so its maximum would be a reduction over 128 threads
// for every tile.  The running maximum m only has to be within 2^8 of the true one: a tile
// whose logits all stay below m + 8 (one vote) keeps m; the first tile of a segment and the
// rare others take the reduction and rescale O.  The row sums stay in the threads, over the
// rounded weights, and are reduced once a segment.
//
// Persistent CTAs: the key tiles of all (sequence, row block) items, in that order, are cut
// into equal runs, one a CTA; rows of items cut by a run's end go to the workspace and are
// joined by a second kernel.
//
// Roles (10 warps): 8 softmax warps (warp w: keys 32 (w % 4) .. + 31, the rows' half w / 4),
// a TMA warp, an MMA warp.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int BN = 128;                     // keys of a tile (TMEM lanes)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays at most 2^8
constexpr int kMaxCtas = 152;               // one CTA an SM
constexpr int kSegTiles = 1;                // a segment's fixed cost, in key tiles
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = (kSoftmaxWarps + 2) * 32;
constexpr uint32_t kPair = 2 * BN * 128;    // bytes of 128 values of a tile: two 64-value chunks
constexpr uint32_t kRope = BN * 128;        // of its rotated part, and of P

// instruction descriptors: f16 operands, f32 accumulation; A and B majors (1: MN)
__host__ __device__ constexpr uint32_t idesc(uint32_t N, uint32_t a_mn, uint32_t b_mn) {
    return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

// NP: blocks of 128 latent values; NR: rows of a block.
template <int NP, int NR>
struct Cfg {
    static constexpr int R = NP * 128, W = R + 64, NCH = 2 * NP + 1;
    static constexpr int NH = NR / 2;                      // rows of a softmax thread
    static constexpr uint32_t Q_CHUNK = NR * 128, Q_BYTES = NCH * Q_CHUNK;
    // where shared memory is short P takes the place of the tile's rotated part, which only S needs
    static constexpr bool ALIAS = NP == 4 && NR >= 32;
    static constexpr int NPS = NR == 64 ? 4 : 5;           // 128-value slots
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_PAIR = (Q_BYTES + 1023) / 1024 * 1024;
    static constexpr uint32_t OFF_ROPE = OFF_PAIR + NPS * kPair;
    static constexpr uint32_t OFF_P = ALIAS ? OFF_ROPE : OFF_ROPE + kRope;
    static constexpr uint32_t OFF_ROWS = OFF_P + kRope;    // lim, m, alpha, wmax[4], wl[4]: NR words each
    enum : int { A_LIM, A_M, A_ALPHA, A_WMAX, A_WL = A_WMAX + 4, N_ROWS = A_WL + 4 };
    static constexpr uint32_t OFF_FLAGS = OFF_ROWS + N_ROWS * NR * 4;   // [2][8] words
    static constexpr uint32_t OFF_SUMS = OFF_FLAGS + 64;   // the run's search
    enum : int {
        B_QFULL, B_QEMPTY, B_PAIR, B_PAIRFREE = B_PAIR + NPS, B_ROPE = B_PAIRFREE + NPS, B_ROPEFREE, B_S, B_P,
        B_DONE,      // a segment's last product is done
        B_GROUP,     // the softmax warps met
        B_TEARDOWN, N_BARS
    };
    static constexpr uint32_t OFF_BAR = OFF_SUMS + 24 * 8 + 32;
    static constexpr uint32_t OFF_MISC = OFF_BAR + N_BARS * 8;   // TMEM base, abort flag
    static constexpr uint32_t SMEM_ALLOC = OFF_MISC + 8 + 1024;
    static constexpr uint32_t COL_O = NR, COLS = NR + NP * NR;
    static constexpr uint32_t TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(2 * (SMEM_ALLOC + 1024) > 233472, "one CTA an SM: its TMEM allocation never waits");
    static_assert(OFF_SUMS % 8 == 0 && OFF_BAR % 8 == 0, "alignment");
};

struct Args {
    const int32_t *q_start, *kv_len, *page_table;
    __half* out;
    float* lse;
    float* part_o;       // [CTA][2][NR][R]
    float2* part_ml;     // [CTA][2][NR]
    int* meta;           // [CTA][4]
    int* err;
    int B, total_q, max_q, H;
    int log2P, max_pages, n_slots, box_rows;   // pages, or the contiguous cache's sequences
    int n_rb;            // row blocks of the longest chunk
    int side;            // row blocks of a sequence that neighbouring CTAs take side by side
    long long capacity;
    float scale;
};

// One sequence's new tokens.
struct Chunk {
    int q_base, n, pos0, L;   // first token row, tokens computed, position of token 0, cached keys
};
__device__ __forceinline__ Chunk load_chunk(const Args& a, int b) {
    Chunk c;
    c.q_base = a.q_start[b];
    const int n_q = max(a.q_start[b + 1] - c.q_base, 0), len = a.kv_len[b];
    c.n = min(n_q, a.max_q);
    c.pos0 = len - n_q;
    c.L = static_cast<int>(min(static_cast<long long>(max(len, 0)), a.capacity));
    return c;
}
// groups of row blocks that are taken side by side
template <int NR>
__device__ __forceinline__ int groups_of(const Args& a, const Chunk& c) {
    const long long blocks = (static_cast<long long>(c.n) * a.H + NR - 1) / NR;
    return static_cast<int>((blocks + a.side - 1) / a.side);
}
// keys that some row of the rows up to `end` (not included) keeps lie below this
__device__ __forceinline__ int key_end(const Args& a, const Chunk& c, long long end) {
    const long long last = min(end, static_cast<long long>(c.n) * a.H) - 1;
    return static_cast<int>(max(0ll, min(static_cast<long long>(c.L), c.pos0 + last / a.H + 1)));
}
template <int NR>
__device__ __forceinline__ int group_tiles(const Args& a, const Chunk& c, int g) {
    return max((key_end(a, c, static_cast<long long>(g + 1) * a.side * NR) + BN - 1) / BN, 1);
}

// A CTA's run of key tiles, walked a segment (part of one item) at a time.  Every warp walks
// for itself.
struct Walk {
    int b, g, off;       // sequence, group of row blocks, first key tile
    int n_g, n, tiles;   // groups of the sequence; key tiles of the segment and of the item
    long long rem;       // key tiles of the run from this segment on
    Chunk c;
};
template <int NR>
__device__ __forceinline__ bool walk_item(const Args& a, Walk& w) {
    if (w.rem <= 0) return false;
    w.c = load_chunk(a, w.b);
    w.n_g = groups_of<NR>(a, w.c);
    w.tiles = group_tiles<NR>(a, w.c, w.g);
    w.n = static_cast<int>(min(static_cast<long long>(w.tiles - w.off), w.rem));
    return w.n > 0;      // (lengths that changed under the call)
}
template <int NR>
__device__ __forceinline__ bool walk_next(const Args& a, Walk& w) {
    w.rem -= w.n;
    w.off = 0;
    if (w.rem <= 0) return false;
    if (++w.g >= w.n_g) {
        w.g = 0;
        do {
            if (++w.b >= a.B) return false;
        } while (load_chunk(a, w.b).n == 0);
    }
    return walk_item<NR>(a, w);
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N]) {
    if constexpr (N == 32) {
        tc_ld_32x32b_x32(addr, r);
    } else if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(addr));
    } else {
        static_assert(N == 8, "columns");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr));
    }
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[N]) {
    if constexpr (N == 32) {
        tc_st_32x32b_x32(addr, r);
    } else if constexpr (N == 16) {
        tc_st_32x32b_x16(addr, r);
    } else {
        static_assert(N == 8, "columns");
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    }
}

// N values of each lane reduced over the warp's lanes: lane l ends up with that of value
// l / (32 / N), in N - 1 + log2(32 / N) shuffles.
template <int N, typename Op>
__device__ __forceinline__ float reduce_lanes(const float (&x)[N], int lane, Op op) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[i];
    int o = 16;
#pragma unroll
    for (int w = N / 2; w > 0; w >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = up ? v[i + w] : v[i], send = up ? v[i] : v[i + w];
            v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
#pragma unroll
    for (; o > 0; o >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    return v[0];
}

template <int NP, int NR>
__global__ void __launch_bounds__(kThreads, 1)
latent_attend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_x, const Args a) {
    using C = Cfg<NP, NR>;
    constexpr int NH = C::NH, NPS = C::NPS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + C::OFF_BAR + i * 8; };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be set up meanwhile
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // A wait of a whole warp, with one answer for all of its lanes.
    auto wait = [&](int b, uint32_t parity, int code) -> bool {
        if (__all_sync(0xffffffffu, mbar_try_wait_for(bar(b), parity, 1000000))) return true;
        const uint64_t t0 = globaltimer();
        const uint64_t limit = *static_cast<volatile unsigned long long*>(&g_wait_limit_ns);
#pragma unroll 1
        do {
            if (__all_sync(0xffffffffu, mbar_try_wait_for(bar(b), parity, 1000000))) return true;
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
        } while (__any_sync(0xffffffffu, globaltimer() - t0 < limit));
        *abort_flag = 1;
        atomicExch(a.err, code);
        return false;
    };

    // ---- this CTA's run: sum the key tiles of every (sequence, group), then find where the
    // run starts
    Walk run;
    {
        constexpr int kWarps = kThreads / 32;
        long long* sums = reinterpret_cast<long long*>(smem + C::OFF_SUMS);   // [2][warps], then the run's ends
        int* first = reinterpret_cast<int*>(sums + 24);
        const int max_g = (a.n_rb + a.side - 1) / a.side;
        const long long pairs = static_cast<long long>(a.B) * max_g;
        const long long per = (pairs + kThreads - 1) / kThreads;
        const long long f0 = min(pairs, tid * per), f1 = min(pairs, f0 + per);
        // visits this thread's items in order until fn says stop
        auto visit = [&](auto fn) {
            if (f0 >= f1) return;
            int b = static_cast<int>(f0 / max_g), g = static_cast<int>(f0 - static_cast<long long>(b) * max_g);
            long long left = f1 - f0;
            while (left > 0) {
                const Chunk c = load_chunk(a, b);
                const int end = static_cast<int>(min(static_cast<long long>(groups_of<NR>(a, c)), g + left));
                for (int i = g; i < end; ++i)
                    if (!fn(b, i, group_tiles<NR>(a, c, i))) return;
                left -= max_g - g;
                g = 0;
                ++b;
            }
        };
        long long mine = 0, tiles = 0;         // weights, and key tiles alone
        visit([&](int, int, int t) {
            mine += t + kSegTiles;
            tiles += t;
            return true;
        });
        long long incl = mine, incl_t = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o), y = __shfl_up_sync(0xffffffffu, incl_t, o);
            if (lane >= o) {
                incl += x;
                incl_t += y;
            }
        }
        if (lane == 31) {
            sums[warp] = incl;
            sums[kWarps + warp] = incl_t;
        }
        if (tid == 0) {
            for (int i = 0; i < C::N_BARS; ++i)
                mbar_init(bar(i), i == C::B_P || i == C::B_GROUP ? kSoftmaxWarps : 1);
            *abort_flag = 0;
            first[3] = 0;
            fence_barrier_init();
        }
        if (warp == kSoftmaxWarps + 1) {
            tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        long long before = incl - mine, before_t = incl_t - tiles, total = 0, total_t = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) {
                before += sums[i];
                before_t += sums[kWarps + i];
            }
            total += sums[i];
            total_t += sums[kWarps + i];
        }
        // as many runs as CTAs, or fewer of a key tile at least (a run's weight is above kSegTiles)
        const int rank = static_cast<int>(blockIdx.x) / a.side;
        const long long runs = max(1ll, min(static_cast<long long>(gridDim.x / a.side), total / (kSegTiles + 1)));
        if (tid == 0) sums[20] = sums[21] = total_t;
        __syncthreads();
        if (rank < runs) {
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                const long long t = total * (rank + e) / runs;
                if (before > t || t >= before + mine) continue;
                long long acc = before, acc_t = before_t;
                visit([&](int b, int g, int n) {
                    if (acc + n + kSegTiles <= t) {
                        acc += n + kSegTiles;
                        acc_t += n;
                        return true;
                    }
                    const int off = max(static_cast<int>(t - acc) - kSegTiles, 0);
                    sums[20 + e] = acc_t + off;
                    if (e == 0) {
                        first[0] = b;
                        first[1] = g;
                        first[2] = off;
                    }
                    return false;
                });
            }
        }
        __syncthreads();
        run.b = first[0];
        run.g = first[1];
        run.off = first[2];
        run.rem = rank < runs ? sums[21] - sums[20] : 0;
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const int rb_in = static_cast<int>(blockIdx.x) % a.side;   // of the group's row blocks, this CTA's

    if (warp == kSoftmaxWarps) {
        // ------------------------------------------------------------ TMA: Q, then the tiles
        // Lane l brings box l % nb (a page, or a tile's part of one) of chunk l / nb of a
        // 128-value pair; the boxes of the rotated part are lanes 0 .. nb - 1.
        const int nb = BN / a.box_rows, bx = lane & (nb - 1), P = 1 << a.log2P;
        uint32_t n_pair = 0, n_tile = 0, n_seg = 0, n_q = 0;   // (copies posted)
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_x);
        }
        bool ok = true;
        Walk w = run;
        for (bool on = walk_item<NR>(a, w); on && ok; on = walk_next<NR>(a, w), ++n_seg) {
            const long long row0 = (static_cast<long long>(w.g) * a.side + rb_in) * NR;
            const int hi = key_end(a, w.c, row0 + NR);
            if (n_seg > 0 && !(ok = wait(C::B_QEMPTY, (n_seg - 1) & 1, kErrTimeoutSlot))) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(C::B_QFULL), C::Q_BYTES);
                const int q_row = static_cast<int>(static_cast<long long>(w.c.q_base) * a.H + row0);
                for (int c = 0; c < C::NCH; ++c)
                    tma_load_2d(sbase + C::OFF_Q + c * C::Q_CHUNK, &tm_q, bar(C::B_QFULL), c * 64, q_row);
            }
            ++n_q;
            // the place of this lane's box in tile j: page id (or sequence) and row
            int slot = 0;
            auto fetch = [&](int j) {
                const int kk = (w.off + j) * BN + bx * a.box_rows;
                slot = w.b;
                if (a.page_table)
                    slot = j < w.n && kk < hi
                               ? __ldg(&a.page_table[static_cast<size_t>(w.b) * a.max_pages + (kk >> a.log2P)]) : 0;
            };
            fetch(0);
            for (int j = 0; j < w.n; ++j, ++n_tile) {
                const int key0 = (w.off + j) * BN, kk = key0 + bx * a.box_rows;
                const int boxes = hi > key0 ? min(nb, (hi - key0 + a.box_rows - 1) / a.box_rows) : 0;
                const bool has = kk < hi;
                int row = kk;
                if (a.page_table) {
                    row = kk & (P - 1);
                    if (has && (slot < 0 || slot >= a.n_slots)) {
                        atomicExch(a.err, kErrLatentPage);   // never read: its keys are zeros
                        slot = a.n_slots;
                    }
                }
                const int cur = slot;
                fetch(j + 1);
                for (int p = 0; p < NP; ++p, ++n_pair) {
                    const uint32_t s = n_pair % NPS, round = n_pair / NPS;
                    if (round > 0 && !(ok = wait(C::B_PAIRFREE + s, (round - 1) & 1, kErrTimeoutSlot))) break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar(C::B_PAIR + s), static_cast<uint32_t>(2 * boxes * a.box_rows) * 128);
                    __syncwarp();
                    if (has && lane < 2 * nb) {
                        const int c = lane / nb;
                        tma_load_3d(sbase + C::OFF_PAIR + s * kPair + c * (BN * 128) + bx * a.box_rows * 128, &tm_x,
                                    bar(C::B_PAIR + s), p * 128 + c * 64, row, cur);
                    }
                }
                if (!ok) break;
                if (n_tile > 0 && !(ok = wait(C::B_ROPEFREE, (n_tile - 1) & 1, kErrTimeoutSlot))) break;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar(C::B_ROPE), static_cast<uint32_t>(boxes * a.box_rows) * 128);
                __syncwarp();
                if (has && lane < nb)
                    tma_load_3d(sbase + C::OFF_ROPE + bx * a.box_rows * 128, &tm_x, bar(C::B_ROPE), C::R, row, cur);
            }
        }
        if (!ok || __any_sync(0xffffffffu, *abort_flag)) {
            // let copies already in flight land before the CTA's shared memory goes away
            if (lane == 0) {
                if (n_q > 0) mbar_wait_drain(bar(C::B_QFULL), (n_q - 1) & 1, a.err, kErrTimeoutLoad);
                for (uint32_t i = n_pair > NPS ? n_pair - NPS : 0; i < n_pair; ++i)
                    mbar_wait_drain(bar(C::B_PAIR + i % NPS), (i / NPS) & 1, a.err, kErrTimeoutLoad);
                if (n_tile > 0) mbar_wait_drain(bar(C::B_ROPE), (n_tile - 1) & 1, a.err, kErrTimeoutLoad);
            }
        }
    } else if (warp == kSoftmaxWarps + 1) {
        // ------------------------------------------------------------ MMA issuer
        // (the whole warp runs the code; one lane issues)
        const uint32_t one = elect_one();
        constexpr uint32_t id_s = idesc(NR, 0, 0), id_o = idesc(NR, 1, 1);
        const uint64_t q_desc = smem_desc_sw128(sbase + C::OFF_Q, 16, 1024);
        const uint64_t x_desc = smem_desc_sw128(sbase + C::OFF_PAIR, 16, 1024);
        const uint64_t r_desc = smem_desc_sw128(sbase + C::OFF_ROPE, 16, 1024);
        const uint64_t c_desc = smem_desc_sw128(sbase + C::OFF_PAIR, BN * 128, 1024);   // MN-major: next 64 values
        const uint64_t p_desc = smem_desc_sw128(sbase + C::OFF_P, 16, 1024);
        bool stall = stall_first_tile(), ok = true;
        uint32_t n_tile = 0, n_seg = 0;
        Walk w = run;
        for (bool on = walk_item<NR>(a, w); on && ok; on = walk_next<NR>(a, w), ++n_seg) {
            if (!(ok = wait(C::B_QFULL, n_seg & 1, kErrTimeoutLoad))) break;
            for (int j = 0; j < w.n; ++j, ++n_tile) {
                const uint32_t pair0 = n_tile * NP;
                for (int p = 0; p < NP; ++p) {
                    const uint32_t s = (pair0 + p) % NPS;
                    if (!(ok = wait(C::B_PAIR + s, ((pair0 + p) / NPS) & 1, kErrTimeoutLoad))) break;
                    tc_fence_after();
                    const uint64_t xd = desc_advance(x_desc, s * kPair), qd = desc_advance(q_desc, p * 2 * C::Q_CHUNK);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_f16_ss_one(one, tmem, desc_advance(xd, c * (BN * 128) + kk * 32),
                                              desc_advance(qd, c * C::Q_CHUNK + kk * 32), id_s, (p | c | kk) != 0);
                }
                if (!ok || !(ok = wait(C::B_ROPE, n_tile & 1, kErrTimeoutLoad))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_f16_ss_one(one, tmem, desc_advance(r_desc, kk * 32),
                                      desc_advance(q_desc, 2 * NP * C::Q_CHUNK + kk * 32), id_s, 1);
                if (!C::ALIAS) tc_commit_one(one, bar(C::B_ROPEFREE));
                if (j == w.n - 1) tc_commit_one(one, bar(C::B_QEMPTY));
                if (!stall) tc_commit_one(one, bar(C::B_S));
                stall = false;
                if (!(ok = wait(C::B_P, n_tile & 1, kErrTimeoutSoftmax))) break;
                tc_fence_after();
                for (int p = 0; p < NP; ++p) {
                    const uint32_t s = (pair0 + p) % NPS;
                    const uint64_t cd = desc_advance(c_desc, s * kPair);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)   // 16 keys: 16 lines of 128 bytes
                        tc_mma_f16_ss_one(one, tmem + C::COL_O + p * NR, desc_advance(cd, kk * 2048),
                                          desc_advance(p_desc, kk * 2048), id_o, (j | kk) != 0);
                    tc_commit_one(one, bar(C::B_PAIRFREE + s));
                }
                if (C::ALIAS) tc_commit_one(one, bar(C::B_ROPEFREE));
                if (j == w.n - 1) tc_commit_one(one, bar(C::B_DONE));
            }
        }
        // all issued MMAs must retire before TMEM is released
        tc_commit_one(one, bar(C::B_TEARDOWN));
        if (lane == 0) mbar_wait_drain(bar(C::B_TEARDOWN), 0, a.err, kErrTimeoutMma);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax, and the rows out
        const int quarter = warp & 3, half = warp >> 2;
        const int key_in = quarter * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        float* rows = reinterpret_cast<float*>(smem + C::OFF_ROWS);
        int* lim = reinterpret_cast<int*>(rows + C::A_LIM * NR) + half * NH;   // this half's rows
        float* m = rows + C::A_M * NR + half * NH;
        float* alpha = rows + C::A_ALPHA * NR + half * NH;
        float* wmax = rows + C::A_WMAX * NR + half * NH;
        float* wl = rows + C::A_WL * NR + half * NH;
        volatile int* flags = reinterpret_cast<volatile int*>(smem + C::OFF_FLAGS);
        const float scale_log2 = a.scale * kLog2e;
        uint32_t n_meet = 0, n_tile = 0, n_seg = 0;
        // the 8 warps meet; writes to shared memory before it are seen after it
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_GROUP));
            return wait(C::B_GROUP, n_meet++ & 1, kErrTimeoutSoftmax);
        };
        if (tid == 0) a.meta[blockIdx.x * 4] = a.meta[blockIdx.x * 4 + 1] = 0;
        bool ok = true;
        Walk w = run;
        for (bool on = walk_item<NR>(a, w); on && ok; on = walk_next<NR>(a, w), ++n_seg) {
            const long long row0 = (static_cast<long long>(w.g) * a.side + rb_in) * NR;
            const int live = static_cast<int>(max(0ll, min(static_cast<long long>(NR), static_cast<long long>(w.c.n) * a.H - row0)));
            const int hi = key_end(a, w.c, row0 + NR);
            // keys below this are kept by every row of the block
            const int all_keep = live > 0 ? key_end(a, w.c, row0 + 1) : 0;
            if (tid < NR) reinterpret_cast<int*>(rows)[tid] = tid < live ? key_end(a, w.c, row0 + tid + 1) : 0;
            float l[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) l[i] = 0.f;
            if (!(ok = meet())) break;
            for (int j = 0; j < w.n; ++j, ++n_tile) {
                if (!(ok = wait(C::B_S, n_tile & 1, kErrTimeoutMma))) break;
                tc_fence_after();
                float x[NH];
                {
                    uint32_t r[NH];
                    tmem_load<NH>(lanes + half * NH, r);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < NH; ++i) x[i] = __uint_as_float(r[i]) * scale_log2;
                }
                const int key0 = (w.off + j) * BN, key = key0 + key_in;
                if (key0 + BN > all_keep) {
#pragma unroll
                    for (int i = 0; i < NH; i += 4) {
                        const int4 e = *reinterpret_cast<const int4*>(lim + i);
                        x[i] = key < e.x ? x[i] : -INFINITY;
                        x[i + 1] = key < e.y ? x[i + 1] : -INFINITY;
                        x[i + 2] = key < e.z ? x[i + 2] : -INFINITY;
                        x[i + 3] = key < e.w ? x[i + 3] : -INFINITY;
                    }
                }
                bool above = j == 0;
                if (j > 0) {
                    float over = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NH; i += 4) {
                        const float4 e = *reinterpret_cast<const float4*>(m + i);
                        over = fmaxf(fmaxf(over, x[i] - e.x), x[i + 1] - e.y);
                        over = fmaxf(fmaxf(over, x[i + 2] - e.z), x[i + 3] - e.w);
                    }
                    const int any = __any_sync(0xffffffffu, over > kRescaleThreshold);
                    if (lane == 0) flags[(n_tile & 1) * kSoftmaxWarps + warp] = any;
                    if (!(ok = meet())) break;
                    above = __any_sync(0xffffffffu, lane < kSoftmaxWarps && flags[(n_tile & 1) * kSoftmaxWarps + lane]);
                }
                if (above) {
                    // the rows' maxima over the tile: over the warp's lanes, then over the quarters
                    const float top = reduce_lanes<NH>(x, lane, [](float p, float q) { return fmaxf(p, q); });
                    if (lane % (32 / NH) == 0) wmax[quarter * NR + lane / (32 / NH)] = top;
                    if (!(ok = meet())) break;
                    if (quarter == 0 && lane < NH) {
                        const float t = fmaxf(fmaxf(wmax[lane], wmax[NR + lane]), fmaxf(wmax[2 * NR + lane], wmax[3 * NR + lane]));
                        const float old = j == 0 ? -INFINITY : m[lane];
                        float now = old, f = 1.f;
                        if (half * NH + lane >= live) {
                            now = INFINITY;   // not a row: no weight
                        } else if (t > old + kRescaleThreshold) {
                            now = t;
                            f = old == -INFINITY ? 0.f : ex2_approx(old - t);
                        }
                        m[lane] = now;
                        alpha[lane] = f;
                    }
                    if (!(ok = meet())) break;
                    if (j > 0) {
                        // (the product of the tile before is done: S of this one was issued after it)
                        float f[NH];
#pragma unroll
                        for (int i = 0; i < NH; ++i) {
                            f[i] = alpha[i];
                            l[i] *= f[i];
                        }
#pragma unroll 1
                        for (int p = 0; p < NP; ++p) {
                            uint32_t r[NH];
                            const uint32_t at = lanes + C::COL_O + p * NR + half * NH;
                            tmem_load<NH>(at, r);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < NH; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f[i]);
                            tmem_store<NH>(at, r);
                        }
                        tc_wait_st();
                    }
                }
                // weights: a key's line of P, swizzled as the MMA reads it
                uint32_t packed[NH / 2];
#pragma unroll
                for (int i = 0; i < NH; i += 4) {
                    float4 e = *reinterpret_cast<const float4*>(m + i);
                    // (a row that has kept no key yet: all of x is -inf)
                    e.x = e.x == -INFINITY ? 0.f : e.x;
                    e.y = e.y == -INFINITY ? 0.f : e.y;
                    e.z = e.z == -INFINITY ? 0.f : e.z;
                    e.w = e.w == -INFINITY ? 0.f : e.w;
                    const __half2 h0 = __floats2half2_rn(ex2_approx(x[i] - e.x), ex2_approx(x[i + 1] - e.y));
                    const __half2 h1 = __floats2half2_rn(ex2_approx(x[i + 2] - e.z), ex2_approx(x[i + 3] - e.w));
                    packed[i / 2] = *reinterpret_cast<const uint32_t*>(&h0);
                    packed[i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                    l[i] = add_f16_lo(l[i], packed[i / 2]);
                    l[i + 1] = add_f16_hi(l[i + 1], packed[i / 2]);
                    l[i + 2] = add_f16_lo(l[i + 2], packed[i / 2 + 1]);
                    l[i + 3] = add_f16_hi(l[i + 3], packed[i / 2 + 1]);
                }
                uint8_t* line = smem + C::OFF_P + key_in * 128;
#pragma unroll
                for (int u = 0; u < NH / 8; ++u)
                    *reinterpret_cast<uint4*>(line + (((half * (NH / 8) + u) ^ (key_in & 7)) << 4)) =
                        make_uint4(packed[4 * u], packed[4 * u + 1], packed[4 * u + 2], packed[4 * u + 3]);
                if (key0 + BN > hi) {
                    // keys that no row of the block keeps: their values are zeroed, since memory may
                    // hold anything there (or nothing was copied) and a weight of 0 must not meet a NaN
                    const int r0 = max(hi - key0, 0), per_chunk = (BN - r0) * 8;   // 16-byte units
                    for (int p = 0; p < NP; ++p) {
                        const uint32_t pr = n_tile * NP + p, s = pr % NPS;
                        if (!(ok = wait(C::B_PAIR + s, (pr / NPS) & 1, kErrTimeoutLoad))) break;
                        uint8_t* at = smem + C::OFF_PAIR + s * kPair;
                        for (int u = tid; u < 2 * per_chunk; u += kSoftmaxWarps * 32) {
                            const int c = u >= per_chunk, v = u - c * per_chunk;
                            *reinterpret_cast<uint4*>(at + c * (BN * 128) + r0 * 128 + v * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (!ok) break;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_P));
            }
            if (!ok) break;
            // the rows' sums
            const float sum = reduce_lanes<NH>(l, lane, [](float p, float q) { return p + q; });
            if (lane % (32 / NH) == 0) wl[quarter * NR + lane / (32 / NH)] = sum;
            if (!(ok = meet()) || !(ok = wait(C::B_DONE, n_seg & 1, kErrTimeoutMma))) break;
            tc_fence_after();
            const bool whole = w.n == w.tiles;
            const int part = static_cast<int>(blockIdx.x) * 2 + (w.off > 0 ? 0 : 1);
            const long long out0 = static_cast<long long>(w.c.q_base) * a.H + row0 + half * NH;
            const long long out_end = static_cast<long long>(a.total_q) * a.H;
            // this lane's row (the first lanes): its sum and maximum
            float my_inv = 0.f;
            if (lane < NH) {
                const float s = (wl[lane] + wl[NR + lane]) + (wl[2 * NR + lane] + wl[3 * NR + lane]);
                my_inv = !whole ? 1.f : s == 0.f ? 0.f : 1.0f / s;   // a row without keys: zeros; NaN stays NaN
                const bool mine = half * NH + lane < live && out0 + lane >= 0 && out0 + lane < out_end;
                if (quarter == 0 && mine) {
                    const float mx = m[lane];
                    if (!whole) a.part_ml[static_cast<size_t>(part) * NR + half * NH + lane] = make_float2(mx, s);
                    else if (a.lse)
                        a.lse[out0 + lane] = s == 0.f ? -INFINITY : (mx + __log2f(s)) * 0.6931471805599453f;
                }
            }
            // rows below this are written
            const int n_out = static_cast<int>(max(0ll, min(static_cast<long long>(live - half * NH), out_end - out0)));
            const bool in_out = out0 >= 0;
#pragma unroll 1
            for (int p = 0; p < NP; ++p) {
                uint32_t r[NH];
                tmem_load<NH>(lanes + C::COL_O + p * NR + half * NH, r);
                tc_wait_ld();
                const int d0 = p * 128 + quarter * 32;
                if (whole) {
                    // two lanes swap halves of two rows, so that a lane has two values of one row
#pragma unroll
                    for (int i = 0; i < NH; i += 2) {
                        const float v0 = __uint_as_float(r[i]) * __shfl_sync(0xffffffffu, my_inv, i);
                        const float v1 = __uint_as_float(r[i + 1]) * __shfl_sync(0xffffffffu, my_inv, i + 1);
                        const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v0 : v1, 1);
                        const __half2 h = (lane & 1) ? __floats2half2_rn(other, v1) : __floats2half2_rn(v0, other);
                        const int row = i + (lane & 1);
                        if (in_out && row < n_out)
                            *reinterpret_cast<__half2*>(a.out + static_cast<size_t>(out0 + row) * C::R + d0 + (lane & ~1)) = h;
                    }
                } else {
                    float* dst = a.part_o + (static_cast<size_t>(part) * NR + half * NH) * C::R + d0 + lane;
#pragma unroll
                    for (int i = 0; i < NH; ++i)
                        if (i < n_out) dst[static_cast<size_t>(i) * C::R] = __uint_as_float(r[i]);
                }
            }
            if (tid == 0) {
                // what the join needs of this CTA: [0] its run goes on after its first part (or
                // ends with it), [1] it leaves an item open, [2], [3] that item
                int* meta = a.meta + blockIdx.x * 4;
                if (w.off > 0) meta[0] = w.off + w.n == w.tiles;
                else if (!whole) {
                    meta[1] = 1;
                    meta[2] = w.b;
                    meta[3] = w.g;
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSoftmaxWarps + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the partial rows of the items that run over a CTA boundary: block (c, y) takes the
// item that CTA c leaves open, and of its rows those of chunk y, a warp a row.
constexpr int kJoinWarps = 8;

template <int NP, int NR>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const Args a, int n_ctas) {
    constexpr int R = NP * 128;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for the whole of latent_attend_kernel
    const int* meta = a.meta + blockIdx.x * 4;
    if (!meta[1]) return;
    const int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Chunk c = load_chunk(a, meta[2]);
    const long long at = (static_cast<long long>(meta[3]) * a.side + blockIdx.x % a.side) * NR + row;
    const long long orow = static_cast<long long>(c.q_base) * a.H + at;
    if (at >= static_cast<long long>(c.n) * a.H || orow < 0 || orow >= static_cast<long long>(a.total_q) * a.H) return;
    // the parts: the end of CTA c's run, whole runs of the same item, the beginning of the last
    float mx = a.part_ml[(static_cast<size_t>(blockIdx.x) * 2 + 1) * NR + row].x;
    int last = blockIdx.x;
    while (last + a.side < n_ctas) {
        last += a.side;
        mx = fmaxf(mx, a.part_ml[static_cast<size_t>(last) * 2 * NR + row].x);
        if (a.meta[last * 4]) break;
    }
    float2 o[NP * 2];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < NP * 2; ++e) o[e] = make_float2(0.f, 0.f);
    for (int i = blockIdx.x; i <= last; i += a.side) {
        const size_t p = (static_cast<size_t>(i) * 2 + (i == static_cast<int>(blockIdx.x) ? 1 : 0)) * NR + row;
        const float2 x = a.part_ml[p];
        const float f = x.x == -INFINITY ? 0.f : ex2_approx(x.x - mx);
        sum = fmaf(f, x.y, sum);
        const float4* src = reinterpret_cast<const float4*>(a.part_o + p * R) + lane;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const float4 v = src[e * 32];
            o[2 * e] = ffma2(make_float2(v.x, v.y), make_float2(f, f), o[2 * e]);
            o[2 * e + 1] = ffma2(make_float2(v.z, v.w), make_float2(f, f), o[2 * e + 1]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint2* dst = reinterpret_cast<uint2*>(a.out + static_cast<size_t>(orow) * R) + lane;
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        const __half2 h0 = __floats2half2_rn(o[2 * e].x * inv, o[2 * e].y * inv);
        const __half2 h1 = __floats2half2_rn(o[2 * e + 1].x * inv, o[2 * e + 1].y * inv);
        dst[e * 32] = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    }
    if (a.lse && lane == 0) a.lse[orow] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.6931471805599453f;
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

template <int NP, int NR>
attn_status launch(const LatentAttendLaunch& L, const Plan& p) {
    using C = Cfg<NP, NR>;
    CUtensorMap tq, tx;
    Args a;
    attn_status st;
    {
        const uint64_t dims[2] = {(uint64_t)C::W, (uint64_t)L.total_q * L.H};
        const uint64_t strides[1] = {(uint64_t)C::W * 2};
        const uint32_t box[2] = {64u, (uint32_t)NR};
        if ((st = encode_tmap_sw128(&tq, L.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, dims, strides, box)) != ATTN_OK)
            return st;
    }
    const int rows = L.cache.rows;
    a.n_slots = L.cache.page_table ? L.cache.n_pages : L.B;
    a.box_rows = L.cache.page_table && rows < BN ? rows : BN;
    {
        const uint64_t dims[3] = {(uint64_t)C::W, (uint64_t)rows, (uint64_t)a.n_slots};
        const uint64_t strides[2] = {(uint64_t)C::W * 2, (uint64_t)C::W * 2 * rows};
        const uint32_t box[3] = {64u, (uint32_t)a.box_rows, 1u};
        if ((st = encode_tmap_sw128(&tx, L.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, dims, strides, box)) != ATTN_OK)
            return st;
    }
    auto kernel = latent_attend_kernel<NP, NR>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC) != cudaSuccess)
            return set_error(ATTN_ECUDA, "cudaFuncSetAttribute(latent attend smem) failed");
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    uint8_t* ws = static_cast<uint8_t*>(L.workspace);
    a.q_start = L.q_start;
    a.kv_len = L.kv_len;
    a.page_table = L.cache.page_table;
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
    a.capacity = L.cache.capacity < 0x7ffff000ll ? L.cache.capacity : 0x7ffff000ll;
    a.n_rb = static_cast<int>(p.n_rb);
    // One token of many heads: neighbouring CTAs take its row blocks side by side, so that the
    // second one finds the cache's rows in L2
    a.side = L.max_q == 1 && p.n_rb <= 8 ? static_cast<int>(p.n_rb) : 1;
    a.scale = L.scale;
    const int sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    const int grid = sms / a.side * a.side;
    const dim3 join(grid, NR / kJoinWarps);
    if (trace_enabled())
        trace("latent_attend_kernel<R=%d,rows=%d> grid=%d block=%d smem=%u tmem_cols=%u row_blocks=%d side=%d B=%d "
              "total_q=%d H=%d box_rows=%d, then latent_join_kernel grid=(%u,%u)",
              C::R, NR, grid, kThreads, C::SMEM_ALLOC, C::TMEM_COLS, a.n_rb, a.side, L.B, L.total_q, L.H, a.box_rows,
              join.x, join.y);
    kernel<<<grid, kThreads, C::SMEM_ALLOC, L.stream>>>(tq, tx, a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        // set up while latent_attend_kernel runs: the join waits for its end itself
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = join;
        cfg.blockDim = dim3(kJoinWarps * 32);
        cfg.stream = L.stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, latent_join_kernel<NP, NR>, a, grid);
    }
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "latent attend launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

template <int NP>
attn_status launch_rows(const LatentAttendLaunch& L, const Plan& p) {
    switch (p.NR) {
        case 16: return launch<NP, 16>(L, p);
        case 32: return launch<NP, 32>(L, p);
        default: return launch<NP, 64>(L, p);
    }
}

}  // namespace

size_t latent_attend_workspace(int max_q, int H, int R) { return make_plan(max_q, H, R).bytes; }

attn_status launch_latent_attend(const LatentAttendLaunch& L) {
    const Plan p = make_plan(L.max_q, L.H, L.R);
    return L.R == 256 ? launch_rows<2>(L, p) : launch_rows<4>(L, p);
}

// Sets this translation unit's test controls (see ptx.cuh).
attn_status set_test_controls_latent_attend(unsigned long long wait_limit_ns, int stall) {
    if (cudaMemcpyToSymbol(g_wait_limit_ns, &wait_limit_ns, sizeof(wait_limit_ns)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_stall_first_tile, &stall, sizeof(stall)) != cudaSuccess)
        return set_error(ATTN_ECUDA, "test controls (latent attend): %s", cudaGetErrorString(cudaGetLastError()));
    return ATTN_OK;
}

}  // namespace attn
