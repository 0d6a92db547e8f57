// latent_pair.cu -- attn_latent_attend for many (token, head) rows over long caches, 512 latent values: a
// pair of CTAs (a cluster) takes blocks of 128 rows, each CTA one half of a cached row's values.
//
//   S_r = Q_r X_r^T    128 rows x 64 keys, over CTA r's half of the dims    (tcgen05.mma, M = 128)
//   S = S_0 + S_1      for 64 of the rows: the peer's part comes through shared memory
//   P = 2^(S scale log2e - m)   f16, to both CTAs' shared memory
//   O_r += P C_r       128 rows x R / 2 values      (C_r: the half tile as it lies, MN-major)
//
// Alone, a CTA has room for 64 rows of 512 values, whose M = 64 products run at half rate, and for
// two tiles beside their Q.  Halves of the dims make both products M = 128, and four half tiles fit
// beside Q, whose latent part (256 values of 128 rows) lies in TMEM: 512 columns are O (256), two S
// (128) and Q (128).  The rotated part (64 values) of a tile is CTA 0's or CTA 1's in turn.
//
// A row belongs to one CTA: 16 of each 32 rows (of a warp's lanes of TMEM) to CTA 0, the others to CTA
// 1, so that the four warps that own rows are on all four schedulers (on two: 2260 cycles a tile).
// Four more send the other rows' part of S to the peer, and four take what concerns the other rows'
// O: they wait for their P and rescale their O if their offset moved.
//
// What crosses to the peer goes without a release (one costs 1500 to 2300 cycles): S by st.async, 16 lines
// of P by a copy of 2 KB, both counted in bytes on the peer's barriers (a copy arrives 900 cycles later;
// st.async of P as well, after a transpose over four lanes, was no faster).
//
// Ordering between the CTAs: tile i's part of S is sent once the peer's weights of tile i - 2 are here
// (it has read that tile's part); P(i) is written once both CTAs' second products of tile i - 2 are done
// (each commits to both).  Neither CTA ends before the other's last store to it: they meet at the end.
//
// What bounds it: the chain from tile to tile.  A tile comes by every 1900 to 2000 cycles, of which the tensor
// cores work 1150; with a quarter of the products, no exponentials and a quarter of the copies it is 1700.
// Two tiles' P and S are under way at a time, and shared memory is full.  An owner's loop takes 2000 cycles
// for 16 rows; 8 rows an owner (19 warps) made 128 heads 57 to 61 us, owners that take every second
// tile 67.  32 sequences of 512 to 8192, 128 heads: 57.4 us, 660 TFLOP/s (59.4 with eight caches in turn, of which
// nothing stays in L2 from call to call); a chunk of 512 tokens of 128 heads
// on 4096: 475 us, 1180 TFLOP/s.
//
// Roles (15 warps): 4 owners, 4 senders, 4 that wait for the peer's P (and load Q into TMEM), a TMA warp,
// a warp that issues S and one that issues the others.  The first 12 write a segment's rows.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "latent_run.cuh"

namespace attn {
namespace {

constexpr int NP = 4;                       // blocks of 128 latent values, half of them a CTA's
constexpr int NR = 128;                     // rows of a block
constexpr int SEG = 8;   // a segment's fixed cost, in key tiles (128 heads: 66.0 us with 2, 61.9 with 4, 58.3 with 8, 58.6 with 12)
constexpr int kTmaWarp = 12, kSWarp = 13, kPvWarp = 14;   // and 4 each of owners, senders and others before them
constexpr int kThreads = (kPvWarp + 1) * 32;
constexpr uint32_t kRowsChunk = NR * 128;   // bytes of 64 values of a block's rows

struct Cfg {
    static constexpr int R = NP * 128, W = R + 64, HD = R / 2, DC = NP;   // DC: chunks of 64 values of a half
    static constexpr int NS = 4;                                          // tiles in the ring
    static constexpr uint32_t TILE = DC * kChunk;
    static constexpr uint32_t X_BYTES = NR / 2 * BN * 4;
    static constexpr uint32_t OFF_QR = 0;                                 // rotated part of Q
    static constexpr uint32_t OFF_RING = OFF_QR + kRowsChunk;
    static constexpr uint32_t OFF_ROT = OFF_RING + NS * TILE;             // rotated parts of every second tile
    static constexpr uint32_t OFF_P = OFF_ROT + NS / 2 * kChunk;          // of even and odd tiles
    static constexpr uint32_t OFF_X = OFF_P + 2 * kRowsChunk;             // the peer's part of S, as the threads hold it: [2][4 owners][8][32][16 bytes]
    static constexpr uint32_t OFF_FACTORS = OFF_X + 2 * X_BYTES;          // what to rescale the peer's rows by: [2][64]
    static constexpr uint32_t OFF_SUMS = OFF_FACTORS + 2 * 64 * 4;        // 1 / sum, of two segments: [2][128]
    static constexpr uint32_t OFF_RUN = OFF_SUMS + 2 * NR * 4;            // the run's search
    enum : int {
        B_QR,                            // rotated part of Q
        B_Q, B_QEMPTY,                   // Q is in TMEM; its last S is done
        B_FULL, B_FREE = B_FULL + NS,    // of the ring's places
        B_S = B_FREE + NS,               // S is there, of even and odd tiles
        B_READ = B_S + 2,                // S has been read
        B_X = B_READ + 2,                // the peer's part is there: [2][4 owners]
        B_THEIRS = B_X + 8,              // the peer's weights are there: [2][4 owners]
        B_P = B_THEIRS + 8,              // all weights are there, and O is rescaled
        B_PV = B_P + 2,                  // a tile's second product is done, in both CTAs
        B_SUM = B_PV + 2,                // sums are there, and the products are done, of even and odd segments
        B_OUT = B_SUM + 2,               // a segment's O has been read
        B_TEARDOWN,                      // of both issuers
        N_BARS = B_TEARDOWN + 2
    };
    static constexpr uint32_t OFF_BAR = OFF_RUN + kRunWords<kThreads> * 8;
    static constexpr uint32_t OFF_MISC = OFF_BAR + N_BARS * 8;   // TMEM base, abort flag
    static constexpr uint32_t SMEM_ALLOC = OFF_MISC + 8 + 1024;
    static constexpr uint32_t COL_O = 0, COL_S = HD, COL_Q = COL_S + 2 * BN, COLS = COL_Q + HD / 2;
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(COLS <= TMEM_COLS && NS % 2 == 0);
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(2 * (SMEM_ALLOC + 1024) > 233472, "one CTA an SM: its TMEM allocation never waits");
    static_assert(OFF_BAR % 8 == 0 && OFF_RUN % 8 == 0, "alignment");
};

// ---- the peer's shared memory
__device__ __forceinline__ uint32_t of_peer(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank ^ 1));
    return r;
}
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t x) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
// (counted on the peer's barrier, in bytes, when they are there)
__device__ __forceinline__ void peer_store4_async(uint32_t addr, uint32_t bar, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(addr),
                 "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void peer_store_async(uint32_t addr, uint32_t bar, float x) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %2, [%1];" ::"r"(addr), "r"(bar),
                 "r"(__float_as_uint(x))
                 : "memory");
}
// (commits to the barrier at this place in both CTAs)
__device__ __forceinline__ void commit_both(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "mov.b16 m, 3;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar),
        "r"(one)
        : "memory");
}
__device__ __forceinline__ void peer_copy(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// (sees what the peer stored before its arrival)
__device__ __forceinline__ bool try_wait_peer(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// This thread's row of O, every third 32 values from `first` on.
__device__ __forceinline__ void write_row(const Args& a, const Out& o, uint32_t o_tmem, int row, int d0, int first, float inv) {
    constexpr int R = NP * 128;
    const bool live = row < o.n;
#pragma unroll 1
    for (int q = first; q < NP * 2; q += 3) {
        uint32_t v[32];
        tc_ld_32x32b_x32(o_tmem + q * 32, v);
        tc_wait_ld();
        if (!live) continue;
        if (o.whole) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<size_t>(o.row0 + row) * R + d0 + q * 32);
            uint32_t h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const __half2 x = __floats2half2_rn(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
                h[i] = *reinterpret_cast<const uint32_t*>(&x);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
        } else {
            uint4* dst = reinterpret_cast<uint4*>(a.part_o + (static_cast<size_t>(o.part) * NR + row) * R + d0 + q * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
    }
}

// 16 lanes of O times a factor a row (a thread has values of rows lane / 4 and lane / 4 + 8).
__device__ __forceinline__ void rescale(uint32_t o_tmem, float f_a, float f_b) {
#pragma unroll 1
    for (int q = 0; q < NP * 2; ++q) {
        uint32_t v[16];
        tc_ld_16x256b_x4(o_tmem + q * 32, v);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * ((i & 2) ? f_b : f_a));
        tc_st_16x256b_x4(o_tmem + q * 32, v);
    }
    tc_wait_st();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
latent_pair_kernel(const __half* q, const __grid_constant__ CUtensorMap tm_qr, const __grid_constant__ CUtensorMap tm_half,
                   const __grid_constant__ CUtensorMap tm_box, const Args a) {
    using C = Cfg;
    constexpr int NS = C::NS, DC = C::DC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + C::OFF_BAR + i * 8; };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be set up meanwhile
    prefetch_run(a, kThreads);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = blockIdx.x & 1;
    if (tid == kTmaWarp * 32) {
        tma_prefetch_desc(&tm_qr);
        tma_prefetch_desc(&tm_half);
        tma_prefetch_desc(&tm_box);
    }
    // A wait of a whole warp, with one answer for all of its lanes.  A CTA that gives up tells the other.
    auto give_up = [&](int code) {
        *abort_flag = 1;
        peer_store(of_peer(sbase + C::OFF_MISC + 4, rank), 1u);
        atomicExch(a.err, code);
    };
    auto wait_for = [&](auto test, int code) -> bool {
        if (__all_sync(0xffffffffu, test())) return true;
        const uint64_t t0 = globaltimer();
        const uint64_t limit = *static_cast<volatile unsigned long long*>(&g_wait_limit_ns);
#pragma unroll 1
        do {
            if (__all_sync(0xffffffffu, test())) return true;
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
        } while (__any_sync(0xffffffffu, globaltimer() - t0 < limit));
        give_up(code);
        return false;
    };
    auto wait = [&](int b, uint32_t parity, int code) -> bool {
        return wait_for([&] { return mbar_try_wait(bar(b), parity); }, code);
    };
    auto wait_peer = [&](int b, uint32_t parity, int code) -> bool {
        return wait_for([&] { return try_wait_peer(bar(b), parity); }, code);
    };

    if (warp == 0) {
        for (int i = lane; i < C::N_BARS; i += 32) {
            int n = 1;   // arrivals
            if (i == C::B_Q) n = 4;                                     // warps
            if (i >= C::B_READ && i < C::B_READ + 2) n = 8;             // owners, senders
            if (i >= C::B_P && i < C::B_P + 2) n = 8;                   // owners, and those of the peer's rows
            if (i >= C::B_SUM && i < C::B_SUM + 2) n = 4;               // owners (and the peer's bytes)
            if (i >= C::B_PV && i < C::B_PV + 2) n = 2;                 // CTAs
            if (i == C::B_OUT) n = 12;
            mbar_init(bar(i), n);
        }
        if (lane == 0) *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kSWarp) {
        tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish();
    }
    __syncwarp();
    cluster_meet();   // (both CTAs' barriers are there)
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for what earlier calls wrote or still read

    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
    const Walk run = find_run<NR, SEG, kThreads>(a, pair / a.side, pairs / a.side, reinterpret_cast<long long*>(smem + C::OFF_RUN));
    const int rb_in = pair % a.side;   // of the group's row blocks, this pair's
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    auto row0_of = [&](const Walk& w) { return static_cast<uint32_t>(w.g * a.side + rb_in) * NR; };

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ TMA: Q's rotated part, then the half tiles
        // A half tile is one box where the tile lies in one page (or none), else a box a page and chunk.
        // (The whole warp runs the code and one lane issues.)
        const uint32_t one = elect_one();
        // Row blocks taken side by side, or one, read the cache once: the lines are the first to leave L2,
        // so that those of the partial rows stay.
        const uint64_t policy = a.n_rb <= a.side ? l2_policy_evict_first() : l2_policy_evict_normal();
        const int log_nb = a.log_nb, nb = 1 << log_nb, box_rows = BN >> log_nb, P = 1 << a.log2P;
        uint32_t n_tile = 0, n_seg = 0, s = 0, phase = 1;   // (the first round waits for no release)
        bool ok = true;
        Walk w = run;
        for (bool on = walk_first<NR, SEG>(a, w); on && ok; on = walk_next<NR, SEG>(a, w), ++n_seg) {
            const uint32_t row0 = row0_of(w);
            const int hi = key_end(a, w.c, row0 + NR);
            // the page of box `lane` of tile j, or the sequence: read a tile before its copies
            auto fetch = [&](int j) {
                const int kk = (w.off + j) * BN + lane * box_rows;
                if (!a.page_table) return w.b;
                return lane < nb && j < w.n && kk < hi
                           ? __ldg(&a.page_table[static_cast<size_t>(w.b) * a.max_pages + (kk >> a.log2P)]) : 0;
            };
            int slot = fetch(0);
            if (n_seg > 0 && !(ok = wait(C::B_QEMPTY, (n_seg - 1) & 1, kErrTimeoutSlot))) break;
            mbar_arrive_expect_tx_one(one, bar(C::B_QR), kRowsChunk);
            tma_load_3d_one(one, sbase + C::OFF_QR, &tm_qr, bar(C::B_QR), 0,
                            static_cast<int>(w.c.q_base * static_cast<uint32_t>(a.H) + row0), 2 * NP);
            int key0 = w.off * BN;
#pragma unroll 1
            for (int j = 0; j < w.n; ++j, key0 += BN) {
                const int boxes = hi > key0 ? min(nb, (hi - key0 + box_rows - 1) >> (6 - log_nb)) : 0;
                const int row = a.page_table ? key0 & (P - 1) : key0;   // (0 where a tile has several pages)
                if (a.page_table && (slot < 0 || slot >= a.n_slots)) {
                    atomicExch(a.err, kErrLatentPage);   // never read: its keys are zeros
                    slot = a.n_slots;
                }
                const int cur = slot;
                slot = fetch(j + 1);
                if (!(ok = wait(C::B_FREE + s, phase, kErrTimeoutSlot))) break;
                const bool rot = (s & 1) == rank;   // (an even number of places: the tile's parity)
                const uint32_t dst = sbase + C::OFF_RING + s * C::TILE, rot_dst = sbase + C::OFF_ROT + (s >> 1) * kChunk;
                const uint32_t full = bar(C::B_FULL + s);
                mbar_arrive_expect_tx_one(one, full, static_cast<uint32_t>(boxes * box_rows) * 128 * (DC + rot));
                if (log_nb == 0) {
                    const int at = __shfl_sync(0xffffffffu, cur, 0);
                    if (boxes) {
                        tma_load_4d_hint_one(one, dst, &tm_half, full, 0, row, rank * DC, at, policy);
                        if (rot) tma_load_4d_hint_one(one, rot_dst, &tm_box, full, 0, row, 2 * NP, at, policy);
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < boxes; ++i) {
                        const int page = __shfl_sync(0xffffffffu, cur, i);
#pragma unroll
                        for (int c = 0; c < DC; ++c)
                            tma_load_4d_hint_one(one, dst + c * kChunk + i * box_rows * 128, &tm_box, full, 0, 0, rank * DC + c,
                                                 page, policy);
                        if (rot) tma_load_4d_hint_one(one, rot_dst + i * box_rows * 128, &tm_box, full, 0, 0, 2 * NP, page, policy);
                    }
                }
                ++n_tile;
                if (++s == NS) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (!ok) {
                ++n_seg;   // (its Q is under way)
                break;
            }
        }
        if (!ok || __any_sync(0xffffffffu, *abort_flag)) {
            // let copies already in flight land before the CTA's shared memory goes away
            if (lane == 0) {
                if (n_seg > 0) mbar_wait_drain(bar(C::B_QR), (n_seg - 1) & 1, a.err, kErrTimeoutLoad);
                for (uint32_t i = n_tile > NS ? n_tile - NS : 0; i < n_tile; ++i)
                    mbar_wait_drain(bar(C::B_FULL + i % NS), (i / NS) & 1, a.err, kErrTimeoutLoad);
            }
        }
    } else if (warp == kSWarp || warp == kPvWarp) {
        // ------------------------------------------------------------ MMA issuers
        // (the whole warp runs the code; one lane issues)
        const uint32_t one = elect_one();
        bool ok = true;
        uint32_t n_tile = 0, n_seg = 0, s = 0, phase = 0;   // s, phase: the ring's place
        Walk w = run;
        if (warp == kSWarp) {
            constexpr uint32_t id_s = idesc_f16_f32(NR, BN, false);
            const uint64_t q_desc = smem_desc_sw128(sbase + C::OFF_QR, 16, 1024);
            const uint64_t x_desc = smem_desc_sw128(sbase, 16, 1024);
            const bool stall = stall_first_tile();
            for (bool on = walk_first<NR, SEG>(a, w); on && ok; on = walk_next<NR, SEG>(a, w), ++n_seg) {
                if (!(ok = wait(C::B_QR, n_seg & 1, kErrTimeoutLoad) && wait(C::B_Q, n_seg & 1, kErrTimeoutLoad))) break;
                for (int j = 0; j < w.n; ++j, ++n_tile) {
                    if (n_tile > 1 && !(ok = wait(C::B_READ + (n_tile & 1), ((n_tile >> 1) - 1) & 1, kErrTimeoutSoftmax))) break;
                    if (!(ok = wait(C::B_FULL + s, phase, kErrTimeoutLoad))) break;
                    tc_fence_after();
                    const uint32_t s_tmem = tmem + C::COL_S + (n_tile & 1) * BN;
                    const uint64_t xd = desc_advance(x_desc, C::OFF_RING + s * C::TILE);
#pragma unroll
                    for (int c = 0; c < DC; ++c)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // 16 values: 8 columns of Q
                            tc_mma_f16_ts_one(one, s_tmem, tmem + C::COL_Q + c * 32 + kk * 8, desc_advance(xd, c * kChunk + kk * 32),
                                              id_s, (c | kk) != 0);
                    if ((s & 1) == rank) {
                        const uint64_t rd = desc_advance(x_desc, C::OFF_ROT + (s >> 1) * kChunk);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_f16_ss_one(one, s_tmem, desc_advance(q_desc, kk * 32), desc_advance(rd, kk * 32), id_s, 1);
                    }
                    if (!(stall && n_tile == 0)) tc_commit_one(one, bar(C::B_S + (n_tile & 1)));
                    if (j == w.n - 1) tc_commit_one(one, bar(C::B_QEMPTY));
                    if (++s == NS) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
        } else {
            constexpr uint32_t id_o = idesc_f16_f32(NR, C::HD, true);
            const uint64_t c_desc = smem_desc_sw128(sbase + C::OFF_RING, kChunk, 1024);   // MN-major: next 64 values
            const uint64_t p_desc = smem_desc_sw128(sbase + C::OFF_P, 16, 1024);
            for (bool on = walk_first<NR, SEG>(a, w); on && ok; on = walk_next<NR, SEG>(a, w), ++n_seg) {
                if (n_seg > 0 && !(ok = wait(C::B_OUT, (n_seg - 1) & 1, kErrTimeoutSoftmax))) break;
                for (int j = 0; j < w.n; ++j, ++n_tile) {
                    if (!(ok = wait(C::B_P + (n_tile & 1), (n_tile >> 1) & 1, kErrTimeoutSoftmax))) break;
                    tc_fence_after();
                    const uint64_t pd = desc_advance(p_desc, (n_tile & 1) * kRowsChunk), cd = desc_advance(c_desc, s * C::TILE);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)   // 16 keys: 32 bytes of P's lines, 16 lines of C
                        tc_mma_f16_ss_one(one, tmem + C::COL_O, desc_advance(pd, kk * 32), desc_advance(cd, kk * 2048), id_o,
                                          (j | kk) != 0);
                    tc_commit_one(one, bar(C::B_FREE + s));
                    commit_both(one, bar(C::B_PV + (n_tile & 1)));
                    s = s + 1 == NS ? 0 : s + 1;
                }
            }
        }
        // all issued MMAs must retire before TMEM is released
        const int done = C::B_TEARDOWN + (warp - kSWarp);
        tc_commit_one(one, bar(done));
        if (lane == 0) mbar_wait_drain(bar(done), 0, a.err, kErrTimeoutMma);
        __syncwarp();
    } else {
        const int group = warp >> 2, unit = warp & 3;   // unit: its 32 lanes of TMEM
        const int row = unit * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(unit * 32) << 16);
        const uint32_t own = lanes + (rank * 16 << 16), others = lanes + ((rank ^ 1) * 16 << 16);   // 16 lanes each
        float* sums = reinterpret_cast<float*>(smem + C::OFF_SUMS);
        uint32_t n_tile = 0, n_seg = 0;
        bool ok = true;
        Walk w = run;
        if (rank == 0 && tid == 0) a.meta[pair * 4] = a.meta[pair * 4 + 1] = 0;
        // Q's latent part into TMEM, a row a thread
        auto load_q = [&](const Walk& v) {
            const long long at = static_cast<long long>(v.c.q_base) * a.H + row0_of(v) + row;
            const bool in = at >= 0 && at < static_cast<long long>(a.total_q) * a.H;
            const uint4* src = reinterpret_cast<const uint4*>(q + (in ? at : 0) * C::W + rank * C::HD);
#pragma unroll
            for (int c = 0; c < DC; c += 2) {
                uint32_t v0[32], v1[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint4 x = in ? __ldg(src + c * 8 + i) : make_uint4(0u, 0u, 0u, 0u);
                    uint32_t* to = i < 8 ? v0 + i * 4 : v1 + (i - 8) * 4;
                    to[0] = x.x;
                    to[1] = x.y;
                    to[2] = x.z;
                    to[3] = x.w;
                }
                tc_st_32x32b_x32(lanes + C::COL_Q + c * 32, v0);
                tc_st_32x32b_x32(lanes + C::COL_Q + c * 32 + 32, v1);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_Q));
        };
        const float scale_log2 = a.scale * kLog2e;
        bool on = walk_first<NR, SEG>(a, w);
        if (group == 2 && on) load_q(w);
        for (; on && ok; ++n_seg) {
            const uint32_t row0 = row0_of(w);
            const int hi = key_end(a, w.c, row0 + NR);
            const Out to = out_of<NR>(a, w, row0, pair);
            if (group == 0) {
                // ---------------------------------------------------- owners: 16 rows' weights
                const int first_row = unit * 32 + rank * 16;
                const int ra = first_row + (lane >> 2), rb = ra + 8;   // this thread's rows of the block
                const uint32_t at_p = sbase + C::OFF_P + first_row * 128, to_p = of_peer(at_p, rank);
                const uint32_t theirs = of_peer(bar(C::B_THEIRS + unit), rank);
                const uint32_t to_f = of_peer(sbase + C::OFF_FACTORS + (unit * 16 + (lane >> 2)) * 4, rank);
                const long long live = static_cast<long long>(w.c.n) * a.H - row0;
                // rows keep the keys below lim; no row of the warp drops a key below all_keep
                const int lim_a = key_end(a, w.c, row0 + ra + 1), lim_b = key_end(a, w.c, row0 + rb + 1);
                const int all_keep = key_end(a, w.c, row0 + first_row + 1);
                // offsets in log2 units; +inf for what is not a row of the block: no weight
                float m_a = ra < live ? -INFINITY : INFINITY, m_b = rb < live ? -INFINITY : INFINITY;
                float2 l_a = make_float2(0.f, 0.f), l_b = make_float2(0.f, 0.f);
                for (int j = 0; j < w.n; ++j, ++n_tile) {
                    const uint32_t par = n_tile & 1;
                    const int b_x = C::B_X + par * 4 + unit;
                    if (lane == 0) mbar_arrive_expect_tx(bar(b_x), C::X_BYTES / 4);
                    // S of both CTAs is there, and P of two tiles before has been read, here and at the peer
                    // (in one: each wait costs 100 cycles or more)
                    const uint32_t now = (n_tile >> 1) & 1;
                    if (!(ok = wait_for([&] {
                              return mbar_try_wait(bar(C::B_S + par), now) && try_wait_peer(bar(b_x), now) &&
                                     (n_tile < 2 || mbar_try_wait(bar(C::B_PV + par), now ^ 1));
                          }, kErrTimeoutMma))) break;
                    tc_fence_after();
                    // columns 8 i + 2 (lane % 4), + 1: row a in x[4 i], x[4 i + 1], row b in the next two
                    float x[32];
                    {
                        uint32_t r[32];
                        float4 y[8];
                        tc_ld_16x256b_x8(own + C::COL_S + par * BN, r);
                        const float4* part = reinterpret_cast<const float4*>(smem + C::OFF_X + par * C::X_BYTES) + unit * 256 + lane;
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = part[i * 32];
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 u = fadd2(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])), make_float2(y[i].x, y[i].y));
                            const float2 v = fadd2(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])), make_float2(y[i].z, y[i].w));
                            x[4 * i] = u.x;
                            x[4 * i + 1] = u.y;
                            x[4 * i + 2] = v.x;
                            x[4 * i + 3] = v.y;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_READ + par));
                    const int key0 = (w.off + j) * BN;
                    const bool masked = key0 + BN > all_keep;
                    const int drop_a = lim_a - key0 - 2 * (lane & 3), drop_b = lim_b - key0 - 2 * (lane & 3);
                    // a row's line of P is its 64 weights, swizzled as the MMA reads it (both rows alike,
                    // ra % 8 == rb % 8)
                    uint8_t* line = smem + C::OFF_P + par * kRowsChunk + ra * 128 + (lane & 3) * 4;
                    const float2 f2 = make_float2(scale_log2, scale_log2);
                    // weights against the offsets; returns their sums (of the rounded ones, so that an
                    // output is a convex combination of values)
                    auto weights = [&](float o_a, float o_b, float2& s_a, float2& s_b) {
                        s_a = s_b = make_float2(0.f, 0.f);
                        const float2 na = make_float2(-o_a, -o_a), nb2 = make_float2(-o_b, -o_b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float2 ya = ffma2(make_float2(x[4 * i], x[4 * i + 1]), f2, na);
                            float2 yb = ffma2(make_float2(x[4 * i + 2], x[4 * i + 3]), f2, nb2);
                            if (masked) {
                                if (8 * i >= drop_a) ya.x = -INFINITY;
                                if (8 * i + 1 >= drop_a) ya.y = -INFINITY;
                                if (8 * i >= drop_b) yb.x = -INFINITY;
                                if (8 * i + 1 >= drop_b) yb.y = -INFINITY;
                            }
                            const __half2 ha = __floats2half2_rn(ex2_approx(ya.x), ex2_approx(ya.y));
                            const __half2 hb = __floats2half2_rn(ex2_approx(yb.x), ex2_approx(yb.y));
                            const uint32_t pa = *reinterpret_cast<const uint32_t*>(&ha), pb = *reinterpret_cast<const uint32_t*>(&hb);
                            s_a.x = add_f16_lo(s_a.x, pa);
                            s_a.y = add_f16_hi(s_a.y, pa);
                            s_b.x = add_f16_lo(s_b.x, pb);
                            s_b.y = add_f16_hi(s_b.y, pb);
                            const int u = (i ^ (ra & 7)) << 4;
                            *reinterpret_cast<uint32_t*>(line + u) = pa;
                            *reinterpret_cast<uint32_t*>(line + u + 8 * 128) = pb;
                        }
                    };
                    // First against the running offsets, without the tile's maxima: weights of a thread that sum to
                    // at most 2^15 are each at most that.  A warp with any other (or a NaN, or a row that
                    // has kept no key so far) takes the tile's maxima.
                    float2 s_a, s_b;
                    float f_a = 1.f, f_b = 1.f;
                    bool moved = false, fast = __all_sync(0xffffffffu, m_a != -INFINITY && m_b != -INFINITY);
                    if (fast) {
                        weights(m_a, m_b, s_a, s_b);
                        fast = __all_sync(0xffffffffu, s_a.x + s_a.y <= kFastSumLimit && s_b.x + s_b.y <= kFastSumLimit);
                    }
                    if (!fast) {
                        float ta = -INFINITY, tb = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float ya = x[4 * i + e] * scale_log2, yb = x[4 * i + 2 + e] * scale_log2;
                                ta = fmaxf(ta, masked && 8 * i + e >= drop_a ? -INFINITY : ya);
                                tb = fmaxf(tb, masked && 8 * i + e >= drop_b ? -INFINITY : yb);
                            }
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) {
                            ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, o));
                            tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, o));
                        }
                        const bool need_a = ta - m_a > kRescaleThreshold, need_b = tb - m_b > kRescaleThreshold;
                        if (need_a) {
                            f_a = m_a == -INFINITY ? 0.f : ex2_approx(m_a - (ta - kLift));
                            l_a = fmul2(l_a, make_float2(f_a, f_a));
                            m_a = ta - kLift;
                        }
                        if (need_b) {
                            f_b = m_b == -INFINITY ? 0.f : ex2_approx(m_b - (tb - kLift));
                            l_b = fmul2(l_b, make_float2(f_b, f_b));
                            m_b = tb - kLift;
                        }
                        moved = __any_sync(0xffffffffu, need_a || need_b) && j > 0;
                        // (a row that has kept no key yet: all of its weights are 0)
                        weights(m_a == -INFINITY ? 0.f : m_a, m_b == -INFINITY ? 0.f : m_b, s_a, s_b);
                    }
                    l_a = fadd2(l_a, s_a);
                    l_b = fadd2(l_b, s_b);
                    fence_proxy_async_smem();
                    __syncwarp();
                    // 16 lines of P to the peer, and the rows' factors
                    if (lane == 0) peer_copy(to_p + par * kRowsChunk, at_p + par * kRowsChunk, 16 * 128, theirs + par * 32);
                    if ((lane & 3) == 0) {
                        peer_store_async(to_f + par * 256, theirs + par * 32, f_a);
                        peer_store_async(to_f + par * 256 + 32, theirs + par * 32, f_b);
                    }
                    if (moved) {
                        if (!(ok = wait(C::B_PV + (par ^ 1), ((n_tile - 1) >> 1) & 1, kErrTimeoutMma))) break;
                        tc_fence_after();
                        rescale(own + C::COL_O, f_a, f_b);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_P + par));
                }
                // (the products of the last two tiles: no commit of the peer's is on its way at the end)
                if (ok && n_tile > 1) ok = wait(C::B_PV + (n_tile & 1), ((n_tile >> 1) - 1) & 1, kErrTimeoutMma);
                if (!ok || !(ok = wait(C::B_PV + ((n_tile - 1) & 1), ((n_tile - 1) >> 1) & 1, kErrTimeoutMma))) break;
                float s_a = l_a.x + l_a.y, s_b = l_b.x + l_b.y;
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    s_a += __shfl_xor_sync(0xffffffffu, s_a, o);
                    s_b += __shfl_xor_sync(0xffffffffu, s_b, o);
                }
                if ((lane & 3) < 2) {
                    const bool first = (lane & 3) == 0;
                    const int r = first ? ra : rb, at = (n_seg & 1) * NR + r;
                    const float sum = first ? s_a : s_b, mx = first ? m_a : m_b;
                    const float inv = sum == 0.f ? 0.f : 1.0f / sum;   // a row without keys: zeros; NaN stays NaN
                    sums[at] = inv;
                    peer_store_async(of_peer(sbase + C::OFF_SUMS + at * 4, rank), of_peer(bar(C::B_SUM + (n_seg & 1)), rank), inv);
                    if (r < to.n) {
                        if (!to.whole) a.part_ml[static_cast<size_t>(to.part) * NR + r] = make_float2(mx, sum);
                        else if (a.lse)
                            a.lse[to.row0 + r] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.6931471805599453f;
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    if (unit == 0) mbar_arrive_expect_tx(bar(C::B_SUM + (n_seg & 1)), 64 * 4);
                    else mbar_arrive(bar(C::B_SUM + (n_seg & 1)));
                }
            } else if (group == 1) {
                // ---------------------------------------------------- senders: the peer's rows of S
                const uint32_t to_x = of_peer(sbase + C::OFF_X + unit * (C::X_BYTES / 4) + lane * 16, rank);
                const uint32_t to_b = of_peer(bar(C::B_X + unit), rank);
                for (int j = 0; j < w.n; ++j, ++n_tile) {
                    const uint32_t par = n_tile & 1;
                    // (the peer has read its part of S of two tiles before)
                    const uint32_t now = (n_tile >> 1) & 1;
                    if (!(ok = wait_for([&] {
                              return mbar_try_wait(bar(C::B_S + par), now) &&
                                     (n_tile < 2 || mbar_try_wait(bar(C::B_THEIRS + par * 4 + unit), now ^ 1));
                          }, kErrTimeoutMma))) break;
                    tc_fence_after();
                    uint32_t r[32];   // as the owner holds its part
                    tc_ld_16x256b_x8(others + C::COL_S + par * BN, r);
                    tc_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_READ + par));
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        peer_store4_async(to_x + par * C::X_BYTES + i * 512, to_b + par * 32, r[4 * i], r[4 * i + 1],
                                          r[4 * i + 2], r[4 * i + 3]);
                }
                if (!ok) break;
            } else {
                // ---------------------------------------------------- the peer's rows: their weights, their O
                const float* factors = reinterpret_cast<const float*>(smem + C::OFF_FACTORS);
                for (int j = 0; j < w.n; ++j, ++n_tile) {
                    const uint32_t par = n_tile & 1;
                    const int key0 = (w.off + j) * BN;
                    if (lane == 0) mbar_arrive_expect_tx(bar(C::B_THEIRS + par * 4 + unit), 16 * (128 + 4));
                    if (key0 + BN > hi) {
                        // keys that no row of the block keeps: their values are zeroed, since memory may
                        // hold anything there (or nothing was copied) and a weight of 0 must not meet a NaN
                        const uint32_t s = n_tile % NS;
                        if (!(ok = wait(C::B_FULL + s, (n_tile / NS) & 1, kErrTimeoutLoad))) break;
                        const int r0 = max(hi - key0, 0), per_chunk = (BN - r0) * 8;   // 16-byte units
                        uint8_t* at = smem + C::OFF_RING + s * C::TILE + r0 * 128;
                        for (int c = 0; c < DC; ++c)
                            for (int u = row; u < per_chunk; u += 128)
                                *reinterpret_cast<uint4*>(at + c * kChunk + u * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                    }
                    if (!(ok = wait_peer(C::B_THEIRS + par * 4 + unit, (n_tile >> 1) & 1, kErrTimeoutSoftmax))) break;
                    const float* f = factors + par * 64 + unit * 16 + (lane >> 2);
                    const float f_a = f[0], f_b = f[8];
                    if (__any_sync(0xffffffffu, f_a != 1.f || f_b != 1.f) && j > 0) {
                        if (!(ok = wait(C::B_PV + (par ^ 1), ((n_tile - 1) >> 1) & 1, kErrTimeoutMma))) break;
                        tc_fence_after();
                        rescale(others + C::COL_O, f_a, f_b);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_P + par));
                }
                if (!ok) break;
            }
            const Walk cur = w;
            on = walk_next<NR, SEG>(a, w);
            if (group == 2 && on) {
                if (!(ok = wait(C::B_QEMPTY, n_seg & 1, kErrTimeoutMma))) break;
                tc_fence_after();
                load_q(w);
            }
            if (!(ok = wait_peer(C::B_SUM + (n_seg & 1), (n_seg >> 1) & 1, kErrTimeoutSoftmax))) break;
            tc_fence_after();
            write_row(a, to, lanes + C::COL_O, row, rank * C::HD, group, sums[(n_seg & 1) * NR + row]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_OUT));
            if (rank == 0 && tid == 0) {
                // what the join needs of this pair: [0] the item its run goes on with ends in it; [1] the
                // rows to write of the item that it leaves open (0: none), [2] the first of them
                int* meta = a.meta + pair * 4;
                if (cur.off > 0) {
                    meta[0] = cur.off + cur.n == cur.tiles;
                } else if (!to.whole) {
                    meta[1] = to.n;
                    meta[2] = static_cast<int>(to.row0);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (*abort_flag) {
        // stores to the peer that nothing waited for: let them land (2 KB at most each, a few us)
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 100000) {}
    }
    __syncwarp();
    cluster_meet();   // (the peer may still store here)
}

attn_status launch(const LatentAttendLaunch& L, const Plan& p) {
    using C = Cfg;
    CUtensorMap tq, tx[2];
    Args a;
    attn_status st;
    fill_args(L, p, a);
    {
        const uint64_t dims[3] = {64u, (uint64_t)L.total_q * L.H, 2 * NP + 1};
        const uint64_t strides[2] = {(uint64_t)C::W * 2, 128u};
        const uint32_t box[3] = {64u, (uint32_t)NR, 1u};
        if ((st = encode_tmap_sw128(&tq, L.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, dims, strides, box)) != ATTN_OK)
            return st;
    }
    const int box_rows = BN >> a.log_nb;
    {
        // pages (or sequences) of rows of chunks of 64 values: boxes of half a tile's chunks, or of one
        const uint64_t rows = L.cache.rows, dims[4] = {64u, rows, 2 * NP + 1, (uint64_t)a.n_slots};
        const uint64_t strides[3] = {(uint64_t)C::W * 2, 128u, (uint64_t)C::W * 2 * rows};
        for (int i = 0; i < 2; ++i) {
            const uint32_t box[4] = {64u, (uint32_t)box_rows, i == 0 ? (uint32_t)C::DC : 1u, 1u};
            if ((st = encode_tmap_sw128(&tx[i], L.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, dims, strides, box)) != ATTN_OK)
                return st;
        }
    }
    auto kernel = latent_pair_kernel;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC) != cudaSuccess)
            return set_error(ATTN_ECUDA, "cudaFuncSetAttribute(latent pair smem) failed");
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    const int pairs = sms / 2 / a.side * a.side;
    const dim3 join(pairs, NR * NP / join_width(NP, NR) / kJoinWarps);
    if (trace_enabled())
        trace("latent_pair_kernel grid=%d block=%d smem=%u tmem_cols=%u row_blocks=%d side=%d B=%d total_q=%d H=%d "
              "box_rows=%d whole=%d, then latent_join_kernel grid=(%u,%u)",
              pairs * 2, kThreads, C::SMEM_ALLOC, C::TMEM_COLS, a.n_rb, a.side, L.B, L.total_q, L.H, box_rows, a.whole,
              a.whole ? 0 : join.x, a.whole ? 0 : join.y);
    // both are set up while the kernel before runs, and wait for its end themselves
    cudaError_t e = launch_dependent(kernel, dim3(pairs * 2), kThreads, C::SMEM_ALLOC, L.stream, static_cast<const __half*>(L.q),
                                     tq, tx[0], tx[1], a);
    if (e == cudaSuccess && !a.whole)
        e = launch_dependent(latent_join_kernel<NP, NR>, join, kJoinWarps * 32, 0, L.stream, a, pairs);
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "latent attend launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

}  // namespace

attn_status launch_latent_pair(const LatentAttendLaunch& L) {
    // (the workspace is that of blocks of 64 rows: half as many units, of twice the rows)
    Plan p = make_plan(L.max_q, L.H, L.R);
    p.n_rb = (p.n_rb + 1) / 2;
    return launch(L, p);
}

// Sets this translation unit's test controls (see ptx.cuh).
attn_status set_test_controls_latent_pair(unsigned long long wait_limit_ns, int stall) {
    if (cudaMemcpyToSymbol(g_wait_limit_ns, &wait_limit_ns, sizeof(wait_limit_ns)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_stall_first_tile, &stall, sizeof(stall)) != cudaSuccess)
        return set_error(ATTN_ECUDA, "test controls (latent pair): %s", cudaGetErrorString(cudaGetLastError()));
    return ATTN_OK;
}

}  // namespace attn
