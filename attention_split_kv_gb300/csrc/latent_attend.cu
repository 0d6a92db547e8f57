// latent_attend.cu -- the absorbed form of latent attention (attn_latent_attend) on the
// sm_103a tensor cores: a token's key for every head is its cached row x_j = [c_j | r_j]
// (c the latent vector of R values, r the rotated part of 64), its value is c_j.
//
//   o_ih = sum_j softmax_j(scale q_ih . x_j) c_j      over the keys j <= pos_i
//
// The heads of a sequence's new tokens share the cache's rows, so (token, head) pairs are
// simply rows of one matrix, token-major as q lies in memory, cut into blocks of NR.
//
//   S = Q X^T      rows x 64 keys     (tcgen05.mma, M = 64: rows past NR are not looked at)
//   P = 2^(S scale log2e - m)         f16, to shared memory
//   O^T += C^T P^T   R x NR           (C^T: the tile of X as it lies, read MN-major, 128 values a
//                                      block; N = NR)
//
// so a tile of 64 keys comes from memory once and serves both products, few rows (one token of
// 16 heads) cost products of N = 16 and not of 128 padded rows, and O^T of 512 values fits TMEM
// for up to 64 rows (4 x 64 columns) beside two S.  A row's logits lie in four threads, so its
// maximum and sum stay there; O is rescaled lazily (a weight is at most 2^15), a
// column a row, by all softmax warps.
//
// The S of a tile is made while the one before is in the softmax.  Tiles lie in a ring of halves
// that holds four of them, or of 512 values two (64 or 32 rows) or two and a half (16): a tile stays
// until its second product is done, so with tiles of 128 keys of 512 values the ring held one and the
// copies stood still meanwhile.
//
// Persistent CTAs: the key tiles of all (sequence, row block) items, in that order, are cut
// into equal runs, one a CTA; rows of items cut by a run's end go to the workspace and are
// joined by a second kernel.
//
// Roles (11 warps): 4 softmax warps (warp w: rows 16 w .. + 15; all four zero what a tile has
// too much and rescale O, 32 of O^T's lanes each), a TMA warp, a warp that issues the S products
// and one that issues the others: each waits for its own operands only (one warp for both,
// polling what is ready: 150 cycles a poll, 4500 a tile whatever its rows).  A segment's rows are
// written by the softmax warps and 4 that do only that.
//
// What bounds it.  Few heads: memory.  One token of 32 sequences of 512 to 8192 (137 thousand
// tokens of 576 values, 158 MB), 16 heads: 34.9 us with the join, 4.5 TB/s, of one cache again and again,
// of which some stays in L2; 38.2 us, 4.1 TB/s, with eight caches in turn (23.3 us at a copy's rate).
// Of the rest about 4 us go by before the first tile is there, 4 in the join, and the CTAs
// end 3 apart.  64-row blocks: the tensor cores, whose M = 64 products run at half rate: a tile
// takes 36 MMAs of 37 cycles and 16 of 47, 2080 in all, and comes by every 2600 to 3000, since
// with 64 rows' Q the ring holds two tiles and a tile's chain (copy, S, softmax, PV) is 6000
// long: 8 sequences of 4096, 128 heads, 27.0 us; 1 to 4 drafts of 32 heads of 16 x 32768 tokens 140
// us (89 at a copy's rate), tensor pipe 54%, DRAM 61%.  Many such blocks over long caches go to pairs
// of CTAs instead (latent_pair.cu).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "latent_run.cuh"

namespace attn {
namespace {

constexpr int kSoftmaxWarps = 4;
constexpr int kTmaWarp = kSoftmaxWarps, kSWarp = kTmaWarp + 1;   // and the PV warp
constexpr int kOutWarp = kSWarp + 2;
constexpr int kThreads = (kOutWarp + 4) * 32;

// instruction descriptor: f16 operands, f32 accumulation; A's major (1: MN), B K-major
__host__ __device__ constexpr uint32_t idesc(uint32_t M, uint32_t N, uint32_t a_mn) {
    return (1u << 4) | (a_mn << 15) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// NP: blocks of 128 latent values; NR: rows of a block.
template <int NP, int NR>
struct Cfg {
    static constexpr int R = NP * 128, W = R + 64, NCH = 2 * NP + 1;
    // a segment's fixed cost, in key tiles (128 heads: 69.0 us with 1, 68.0 with 2, 65.2 with 4, 67.0
    // with 6; 16 heads: 40.7, 40.6 and 40.4 with 1, 2 and 4)
    static constexpr int SEG = NR == 64 ? 4 : 2;
    static constexpr uint32_t Q_CHUNK = NR * 128, Q_BYTES = NCH * Q_CHUNK;
    // The ring's places hold half a tile each: NP chunks of 64 values, the second half's with the
    // rotated part behind them.  An even number is packed as tiles.
    static constexpr int NHS = NP == 2 ? 8 : NR == 16 ? 5 : 4;
    static constexpr uint32_t H0 = NP * kChunk, H1 = H0 + kChunk;
    static constexpr uint32_t RING_BYTES = NHS % 2 ? NHS * H1 : NHS / 2 * (H0 + H1);
    // 64 rows of 512 values: P takes the place of its tile's rotated part, which only S needs
    static constexpr bool ALIAS = NP == 4 && NR == 64;
    static constexpr uint32_t P_BYTES = NR * 128;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_RING = (Q_BYTES + 1023) / 1024 * 1024;
    static constexpr uint32_t OFF_P = OFF_RING + RING_BYTES;
    static constexpr uint32_t OFF_ROWS = OFF_P + (ALIAS ? 0 : 2 * P_BYTES);
    // words of the rows: rescale factors of two tiles, then 1 / sum of two segments
    static constexpr uint32_t OFF_FLAGS = OFF_ROWS + 4 * NR * 4;   // [2][4] words
    static constexpr uint32_t OFF_SUMS = OFF_FLAGS + 32;           // the run's search
    // of place s, from the ring's start
    __device__ static __forceinline__ uint32_t place(uint32_t s) {
        return NHS % 2 ? s * H1 : (s >> 1) * (H0 + H1) + (s & 1) * H0;
    }
    // P of tile i, from shared memory's start
    __device__ static __forceinline__ uint32_t p_of(uint32_t i) {
        return ALIAS ? OFF_RING + (i & 1) * (H0 + H1) + 2 * H0 : OFF_P + (i & 1) * P_BYTES;
    }
    static_assert(!ALIAS || NHS == 4, "P of tile i in place 2 i + 1");
    enum : int {
        B_QFULL, B_QEMPTY,
        B_FULL, B_FREE = B_FULL + NHS,   // of the ring's places
        B_S = B_FREE + NHS,
        B_P = B_S + 2,     // weights are there (and flags, factors), of even and odd tiles
        B_PV = B_P + 2,    // a tile's second product is done
        B_FIX = B_PV + 2,  // O is rescaled
        B_MEET,            // the softmax warps have a segment's sums, and its products are done
        B_OUT,             // the other four warps have read its O
        B_TEARDOWN,        // of both issuers
        N_BARS = B_TEARDOWN + 2
    };
    static constexpr uint32_t OFF_BAR = OFF_SUMS + kRunWords<kThreads> * 8;
    static constexpr uint32_t OFF_MISC = OFF_BAR + N_BARS * 8;   // TMEM base, abort flag
    static constexpr uint32_t SMEM_ALLOC = OFF_MISC + 8 + 1024;
    static constexpr uint32_t COL_O = 2 * BN, COLS = COL_O + NP * NR;
    static constexpr uint32_t TMEM_COLS = COLS <= 256 ? 256 : 512;
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(2 * (SMEM_ALLOC + 1024) > 233472, "one CTA an SM: its TMEM allocation never waits");
    static_assert(OFF_SUMS % 8 == 0 && OFF_BAR % 8 == 0, "alignment");
    // S's A operand is read as 64 rows: past NR those are whatever follows Q's chunk
    static_assert(OFF_Q + (NCH - 1) * Q_CHUNK + 64 * 128 <= OFF_ROWS, "Q's rows past NR");
    static_assert(NP % 2 == 0, "halves of whole blocks");
};

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// 32 of O^T's lanes (`quarter`) of every second group of rows, from `first` on.
template <int NP, int NR>
__device__ __forceinline__ void write_rows(const Args& a, const Out& o, uint32_t o_tmem, int quarter, int first,
                                           const float* inv_sum) {
    constexpr int R = NP * 128, EC = NR < 32 ? 16 : 32, NQ = NP * NR / EC;   // columns (rows) at a time
    const int lane = threadIdx.x & 31;
    const uint32_t lanes = o_tmem + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
    for (int q = first; q < NQ; q += 2) {
        const int c0 = (q * EC) % NR;       // the first of these rows
        const int d0 = q * EC / NR * 128 + quarter * 32, n_here = o.n - c0;
        if (n_here <= 0) continue;
        uint32_t v[EC];
        if constexpr (EC == 32) tc_ld_32x32b_x32(lanes + q * EC, v);
        else tmem_load16(lanes + q * EC, v);
        tc_wait_ld();
        if (o.whole) {
            // two lanes swap halves of two rows, so that a lane has two values of one row
            __half* dst = a.out + static_cast<size_t>(o.row0 + c0 + (lane & 1)) * R + d0 + (lane & ~1);
#pragma unroll
            for (int i = 0; i < EC; i += 2) {
                const float2 f = *reinterpret_cast<const float2*>(inv_sum + c0 + i);
                const float v0 = __uint_as_float(v[i]) * f.x, v1 = __uint_as_float(v[i + 1]) * f.y;
                const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v0 : v1, 1);
                const __half2 h = (lane & 1) ? __floats2half2_rn(other, v1) : __floats2half2_rn(v0, other);
                if (i + (lane & 1) < n_here) *reinterpret_cast<__half2*>(dst + i * R) = h;
            }
        } else {
            float* dst = a.part_o + (static_cast<size_t>(o.part) * NR + c0) * R + d0 + lane;
#pragma unroll
            for (int i = 0; i < EC; ++i)
                if (i < n_here) dst[i * R] = __uint_as_float(v[i]);
        }
    }
}

template <int NP, int NR>
__global__ void __launch_bounds__(kThreads, 1)
latent_attend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_h0,
                     const __grid_constant__ CUtensorMap tm_h1, const __grid_constant__ CUtensorMap tm_box, const Args a) {
    using C = Cfg<NP, NR>;
    constexpr int NHS = C::NHS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + C::OFF_BAR + i * 8; };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be set up meanwhile
    prefetch_run(a, kThreads);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == kSoftmaxWarps * 32) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(a.log_nb ? &tm_box : &tm_h0);
        tma_prefetch_desc(a.log_nb ? &tm_box : &tm_h1);
    }
    // A wait of a whole warp, with one answer for all of its lanes.
    auto wait = [&](int b, uint32_t parity, int code) -> bool {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar(b), parity))) return true;
        const uint64_t t0 = globaltimer();
        const uint64_t limit = *static_cast<volatile unsigned long long*>(&g_wait_limit_ns);
#pragma unroll 1
        do {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar(b), parity))) return true;
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
        } while (__any_sync(0xffffffffu, globaltimer() - t0 < limit));
        *abort_flag = 1;
        atomicExch(a.err, code);
        return false;
    };

    if (warp == 0) {
        for (int i = lane; i < C::N_BARS; i += 32)
            mbar_init(bar(i), (i >= C::B_P && i < C::B_P + 2) || i == C::B_FIX || i == C::B_MEET || i == C::B_OUT ? 4 : 1);
        if (lane == 0) *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kSWarp) {
        tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for what earlier calls wrote or still read

    const int cta = static_cast<int>(blockIdx.x);
    const Walk run = find_run<NR, C::SEG, kThreads>(a, cta / a.side, static_cast<int>(gridDim.x) / a.side,
                                                    reinterpret_cast<long long*>(smem + C::OFF_SUMS));
    const int rb_in = cta % a.side;   // of the group's row blocks, this CTA's
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);

    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ TMA: Q, then the tiles
        // Half a tile is one box where the tile lies in one page (or none), else a box a page and
        // chunk.  (The whole warp runs the code and one lane issues.)
        const uint32_t one = elect_one();
        // Row blocks taken side by side, or one, read the cache once: the lines are the first to leave L2,
        // so that those of the partial rows stay (32 sequences of 512 to 8192, eight caches in turn: 16 heads 38.6
        // to 38.2 us, 128 heads, in pairs, 61.2 to 59.4), and some of a cache that the next call reads again (one
        // cache: 38.5 to 36.9, 61.2 to 57.4).  Row blocks that come by at other times want them longer (1 to 4 drafts
        // of 16 x 32768: 139.5 to 141.3).
        const uint64_t policy = a.n_rb <= a.side ? l2_policy_evict_first() : l2_policy_evict_normal();
        const int log_nb = a.log_nb, nb = 1 << log_nb, box_rows = BN >> log_nb, P = 1 << a.log2P;
        uint32_t n_half = 0, n_seg = 0, n_q = 0;   // (copies posted)
        uint32_t s = 0, phase = 1;                 // place, and the phase of its release (the first round waits for none)
        bool ok = true;
        Walk w = run;
        for (bool on = walk_first<NR, C::SEG>(a, w); on && ok; on = walk_next<NR, C::SEG>(a, w), ++n_seg) {
            const uint32_t row0 = static_cast<uint32_t>(w.g * a.side + rb_in) * NR;
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
            mbar_arrive_expect_tx_one(one, bar(C::B_QFULL), C::Q_BYTES);
            tma_load_3d_one(one, sbase + C::OFF_Q, &tm_q, bar(C::B_QFULL), 0,
                            static_cast<int>(w.c.q_base * static_cast<uint32_t>(a.H) + row0), 0);
            ++n_q;
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
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!(ok = wait(C::B_FREE + s, phase, kErrTimeoutSlot))) break;
                    const uint32_t dst = sbase + C::OFF_RING + C::place(s), full = bar(C::B_FULL + s);
                    mbar_arrive_expect_tx_one(one, full, static_cast<uint32_t>(boxes * box_rows) * 128 * (NP + h));
                    if (log_nb == 0) {
                        if (boxes) tma_load_4d_hint_one(one, dst, h ? &tm_h1 : &tm_h0, full, 0, row, h * NP,
                                                        __shfl_sync(0xffffffffu, cur, 0), policy);
                    } else {
#pragma unroll 1
                        for (int i = 0; i < boxes; ++i) {
                            const int page = __shfl_sync(0xffffffffu, cur, i);
#pragma unroll
                            for (int c = 0; c < NP + h; ++c)
                                tma_load_4d_hint_one(one, dst + c * kChunk + i * box_rows * 128, &tm_box, full, 0, 0, h * NP + c, page,
                                                     policy);
                        }
                    }
                    ++n_half;
                    if (++s == NHS) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
            }
        }
        if (!ok || __any_sync(0xffffffffu, *abort_flag)) {
            // let copies already in flight land before the CTA's shared memory goes away
            if (lane == 0) {
                if (n_q > 0) mbar_wait_drain(bar(C::B_QFULL), (n_q - 1) & 1, a.err, kErrTimeoutLoad);
                for (uint32_t i = n_half > NHS ? n_half - NHS : 0; i < n_half; ++i)
                    mbar_wait_drain(bar(C::B_FULL + i % NHS), (i / NHS) & 1, a.err, kErrTimeoutLoad);
            }
        }
    } else if (warp >= kSWarp && warp < kOutWarp) {
        // ------------------------------------------------------------ MMA issuers
        // (the whole warp runs the code; one lane issues)
        const uint32_t one = elect_one();
        bool ok = true;
        uint32_t n_tile = 0, n_seg = 0, s = 0, phase = 0;   // s, phase: the ring's place
        Walk w = run;
        if (warp == kSWarp) {
            constexpr uint32_t id_s = idesc(64, BN, 0);
            const uint64_t q_desc = smem_desc_sw128(sbase + C::OFF_Q, 16, 1024);
            const uint64_t x_desc = smem_desc_sw128(sbase + C::OFF_RING, 16, 1024);
            const bool stall = stall_first_tile();
            for (bool on = walk_first<NR, C::SEG>(a, w); on && ok; on = walk_next<NR, C::SEG>(a, w), ++n_seg) {
                if (!(ok = wait(C::B_QFULL, n_seg & 1, kErrTimeoutLoad))) break;
                for (int j = 0; j < w.n; ++j, ++n_tile) {
                    // (the S of two tiles before has been read once its weights are written)
                    if (n_tile > 1 && !(ok = wait(C::B_P + (n_tile & 1), ((n_tile >> 1) - 1) & 1, kErrTimeoutSoftmax))) break;
                    const uint32_t s_tmem = tmem + (n_tile & 1) * BN;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!(ok = wait(C::B_FULL + s, phase, kErrTimeoutLoad))) break;
                        tc_fence_after();
                        const uint64_t xd = desc_advance(x_desc, C::place(s));
#pragma unroll
                        for (int c = 0; c < NP + h; ++c)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma_f16_ss_one(one, s_tmem, desc_advance(q_desc, (h * NP + c) * C::Q_CHUNK + kk * 32),
                                                  desc_advance(xd, c * kChunk + kk * 32), id_s, (h | c | kk) != 0);
                        if (++s == NHS) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    if (!(stall && n_tile == 0)) tc_commit_one(one, bar(C::B_S + (n_tile & 1)));
                    if (j == w.n - 1) tc_commit_one(one, bar(C::B_QEMPTY));
                }
            }
        } else {
            constexpr uint32_t id_o = idesc(128, NR, 1);
            const uint64_t c_desc = smem_desc_sw128(sbase + C::OFF_RING, kChunk, 1024);   // MN-major: next 64 values
            const uint64_t p_desc = smem_desc_sw128(sbase, 16, 1024);
            const int* flags = reinterpret_cast<const int*>(smem + C::OFF_FLAGS);
            uint32_t n_fix = 0;
            for (bool on = walk_first<NR, C::SEG>(a, w); on && ok; on = walk_next<NR, C::SEG>(a, w), ++n_seg) {
                if (n_seg > 0 && !(ok = wait(C::B_OUT, (n_seg - 1) & 1, kErrTimeoutSoftmax))) break;
                for (int j = 0; j < w.n; ++j, ++n_tile) {
                    if (!(ok = wait(C::B_P + (n_tile & 1), (n_tile >> 1) & 1, kErrTimeoutSoftmax))) break;
                    if (j > 0) {
                        const int* f = flags + (n_tile & 1) * kSoftmaxWarps;
                        if ((f[0] | f[1] | f[2] | f[3]) && !(ok = wait(C::B_FIX, n_fix++ & 1, kErrTimeoutSoftmax))) break;
                    }
                    tc_fence_after();
                    const uint64_t pd = desc_advance(p_desc, C::p_of(n_tile));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t cd = desc_advance(c_desc, C::place(s));
#pragma unroll
                        for (int p = 0; p < NP / 2; ++p)
#pragma unroll
                            for (int kk = 0; kk < BN / 16; ++kk)   // 16 keys: 16 lines of X, 32 bytes of P's
                                tc_mma_f16_ss_one(one, tmem + C::COL_O + (h * (NP / 2) + p) * NR,
                                                  desc_advance(cd, p * 2 * kChunk + kk * 2048), desc_advance(pd, kk * 32), id_o,
                                                  (j | kk) != 0);
                        tc_commit_one(one, bar(C::B_FREE + s));
                        s = s + 1 == NHS ? 0 : s + 1;
                    }
                    tc_commit_one(one, bar(C::B_PV + (n_tile & 1)));
                }
            }
        }
        // all issued MMAs must retire before TMEM is released
        const int done = C::B_TEARDOWN + (warp - kSWarp);
        tc_commit_one(one, bar(done));
        if (lane == 0) mbar_wait_drain(bar(done), 0, a.err, kErrTimeoutMma);
        __syncwarp();
    } else if (warp >= kOutWarp) {
        // ------------------------------------------------------------ half of the rows' values out
        uint32_t n_seg = 0;
        bool ok = true;
        Walk w = run;
        for (bool on = walk_first<NR, C::SEG>(a, w); on && ok; on = walk_next<NR, C::SEG>(a, w), ++n_seg) {
            const Out to = out_of<NR>(a, w, static_cast<uint32_t>(w.g * a.side + rb_in) * NR, cta);
            if (!(ok = wait(C::B_MEET, n_seg & 1, kErrTimeoutSoftmax))) break;
            tc_fence_after();
            write_rows<NP, NR>(a, to, tmem + C::COL_O, warp & 3, 1,
                               reinterpret_cast<const float*>(smem + C::OFF_ROWS) + (2 + (n_seg & 1)) * NR);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_OUT));
        }
    } else {
        // ------------------------------------------------------------ softmax, and the rows out
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const bool has_rows = warp * 16 < NR;
        const int ra = warp * 16 + (lane >> 2), rb = ra + 8;   // this thread's rows of the block
        float* factors = reinterpret_cast<float*>(smem + C::OFF_ROWS);   // [2][NR]
        volatile int* flags = reinterpret_cast<volatile int*>(smem + C::OFF_FLAGS);
        const float scale_log2 = a.scale * kLog2e;
        uint32_t n_tile = 0, n_meet = 0, n_seg = 0;
        // the 4 warps meet; writes to shared memory before it are seen after it
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_MEET));
            return wait(C::B_MEET, n_meet++ & 1, kErrTimeoutSoftmax);
        };
        // After tile i (not a segment's first): once all warps have written their weights, if a row
        // moved its maximum, every warp rescales its lanes of O before the tile's second product.
        auto fix = [&](uint32_t i) -> bool {
            if (!wait(C::B_P + (i & 1), (i >> 1) & 1, kErrTimeoutSoftmax)) return false;
            const int f = lane < kSoftmaxWarps ? flags[(i & 1) * kSoftmaxWarps + lane] : 0;
            if (!__any_sync(0xffffffffu, f)) return true;
            if (!wait(C::B_PV + ((i - 1) & 1), ((i - 1) >> 1) & 1, kErrTimeoutMma)) return false;
            tc_fence_after();
            const float* at = factors + (i & 1) * NR;
#pragma unroll 1
            for (int p = 0; p < NP * NR / 16; ++p) {
                uint32_t r[16];
                tmem_load16(lanes + C::COL_O + p * 16, r);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(at + (p * 16) % NR + e);
                    r[e] = __float_as_uint(__uint_as_float(r[e]) * x.x);
                    r[e + 1] = __float_as_uint(__uint_as_float(r[e + 1]) * x.y);
                    r[e + 2] = __float_as_uint(__uint_as_float(r[e + 2]) * x.z);
                    r[e + 3] = __float_as_uint(__uint_as_float(r[e + 3]) * x.w);
                }
                tc_st_32x32b_x16(lanes + C::COL_O + p * 16, r);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_FIX));
            return true;
        };
        if (tid == 0) a.meta[cta * 4] = a.meta[cta * 4 + 1] = 0;
        bool ok = true;
        Walk w = run;
        for (bool on = walk_first<NR, C::SEG>(a, w); on && ok; on = walk_next<NR, C::SEG>(a, w), ++n_seg) {
            const uint32_t row0 = static_cast<uint32_t>(w.g * a.side + rb_in) * NR;
            const int live = static_cast<int>(max(0ll, min(static_cast<long long>(NR), static_cast<long long>(w.c.n) * a.H - row0)));
            const int hi = key_end(a, w.c, row0 + NR);
            // rows keep the keys below lim; no row of the warp drops a key below all_keep
            const int lim_a = key_end(a, w.c, row0 + ra + 1), lim_b = key_end(a, w.c, row0 + rb + 1);
            const int all_keep = key_end(a, w.c, row0 + warp * 16 + 1);
            // offsets in log2 units; +inf for what is not a row of the block: no weight
            float m_a = ra < live ? -INFINITY : INFINITY, m_b = rb < live ? -INFINITY : INFINITY;
            float2 l_a = make_float2(0.f, 0.f), l_b = make_float2(0.f, 0.f);
            for (int j = 0; j < w.n; ++j, ++n_tile) {
                if (j > 1 && !(ok = fix(n_tile - 1))) break;
                if (!(ok = wait(C::B_S + (n_tile & 1), (n_tile >> 1) & 1, kErrTimeoutMma))) break;
                tc_fence_after();
                // (P of two tiles before must have been read)
                if (n_tile > 1 && !(ok = wait(C::B_PV + (n_tile & 1), ((n_tile >> 1) - 1) & 1, kErrTimeoutMma))) break;
                const int key0 = (w.off + j) * BN;
                if (has_rows) {
                    // columns 8 i + 2 (lane % 4), + 1: row a in x[4 i], x[4 i + 1], row b in the next two
                    float x[32];
                    {
                        uint32_t r[32];
                        tc_ld_16x256b_x8(lanes + (n_tile & 1) * BN, r);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
                    }
                    const bool masked = key0 + BN > all_keep;
                    const int drop_a = lim_a - key0 - 2 * (lane & 3), drop_b = lim_b - key0 - 2 * (lane & 3);
                    // a row's line of P is its 64 weights, swizzled as the MMA reads it (both rows alike,
                    // ra % 8 == rb % 8)
                    uint8_t* line = smem + C::p_of(n_tile) + ra * 128 + (lane & 3) * 4;
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
                    bool fast = __all_sync(0xffffffffu, m_a != -INFINITY && m_b != -INFINITY);
                    if (fast) {
                        weights(m_a, m_b, s_a, s_b);
                        fast = __all_sync(0xffffffffu, s_a.x + s_a.y <= kFastSumLimit && s_b.x + s_b.y <= kFastSumLimit);
                    }
                    int moved = 0;
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
                        float f_a = 1.f, f_b = 1.f;
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
                        if ((lane & 3) == 0) {
                            factors[(n_tile & 1) * NR + ra] = f_a;
                            factors[(n_tile & 1) * NR + rb] = f_b;
                        }
                        moved = __any_sync(0xffffffffu, need_a || need_b);
                        // (a row that has kept no key yet: all of its weights are 0)
                        weights(m_a == -INFINITY ? 0.f : m_a, m_b == -INFINITY ? 0.f : m_b, s_a, s_b);
                    } else if ((lane & 3) == 0) {
                        factors[(n_tile & 1) * NR + ra] = 1.f;
                        factors[(n_tile & 1) * NR + rb] = 1.f;
                    }
                    l_a = fadd2(l_a, s_a);
                    l_b = fadd2(l_b, s_b);
                    if (lane == 0) flags[(n_tile & 1) * kSoftmaxWarps + warp] = moved;
                } else if (lane == 0) {
                    flags[(n_tile & 1) * kSoftmaxWarps + warp] = 0;
                }
                if (key0 + BN > hi) {
                    // keys that no row of the block keeps: their values are zeroed, since memory may
                    // hold anything there (or nothing was copied) and a weight of 0 must not meet a NaN
                    const int r0 = max(hi - key0, 0), per_chunk = (BN - r0) * 8;   // 16-byte units
                    for (uint32_t i = 2 * n_tile; i < 2 * n_tile + 2; ++i) {
                        // (the wait, long over, orders these writes after the copies)
                        if (!(ok = wait(C::B_FULL + i % NHS, (i / NHS) & 1, kErrTimeoutLoad))) break;
                        uint8_t* at = smem + C::OFF_RING + C::place(i % NHS);
                        for (int u = tid; u < NP * per_chunk; u += kSoftmaxWarps * 32) {
                            const int c = u / per_chunk, v = u - c * per_chunk;
                            *reinterpret_cast<uint4*>(at + c * kChunk + r0 * 128 + v * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (!ok) break;
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_P + (n_tile & 1)));
            }
            if (!ok || (w.n > 1 && !(ok = fix(n_tile - 1)))) break;
            // the rows' sums, out of the threads that have them (two segments' in turn: another warp may
            // still read the last one's)
            float* inv_sum = factors + (2 + (n_seg & 1)) * NR;
            const Out to = out_of<NR>(a, w, row0, cta);
            if (has_rows) {
                float s_a = l_a.x + l_a.y, s_b = l_b.x + l_b.y;
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    s_a += __shfl_xor_sync(0xffffffffu, s_a, o);
                    s_b += __shfl_xor_sync(0xffffffffu, s_b, o);
                }
                if ((lane & 3) < 2) {
                    const bool first = (lane & 3) == 0;
                    const int row = first ? ra : rb;
                    const float s = first ? s_a : s_b, mx = first ? m_a : m_b;
                    inv_sum[row] = s == 0.f ? 0.f : 1.0f / s;   // a row without keys: zeros; NaN stays NaN
                    if (row < to.n) {
                        if (!to.whole) a.part_ml[static_cast<size_t>(to.part) * NR + row] = make_float2(mx, s);
                        else if (a.lse)
                            a.lse[to.row0 + row] = s == 0.f ? -INFINITY : (mx + __log2f(s)) * 0.6931471805599453f;
                    }
                }
            }
            if (!(ok = wait(C::B_PV + ((n_tile - 1) & 1), ((n_tile - 1) >> 1) & 1, kErrTimeoutMma)) || !(ok = meet())) break;
            tc_fence_after();
            write_rows<NP, NR>(a, to, tmem + C::COL_O, warp, 0, inv_sum);
            if (tid == 0) {
                // what the join needs of this CTA: [0] the item its run goes on with ends in it; [1] the
                // rows to write of the item that it leaves open (0: none), [2] the first of them
                int* meta = a.meta + cta * 4;
                if (w.off > 0) {
                    meta[0] = w.off + w.n == w.tiles;
                } else if (!to.whole) {
                    meta[1] = to.n;
                    meta[2] = static_cast<int>(to.row0);
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int NP, int NR>
attn_status launch(const LatentAttendLaunch& L, const Plan& p) {
    using C = Cfg<NP, NR>;
    CUtensorMap tq, tx[3];
    Args a;
    attn_status st;
    {
        // rows of 9 (5) chunks of 64 values, all chunks of a block in one box
        const uint64_t dims[3] = {64u, (uint64_t)L.total_q * L.H, (uint64_t)C::NCH};
        const uint64_t strides[2] = {(uint64_t)C::W * 2, 128u};
        const uint32_t box[3] = {64u, (uint32_t)NR, (uint32_t)C::NCH};
        if ((st = encode_tmap_sw128(&tq, L.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, dims, strides, box)) != ATTN_OK)
            return st;
    }
    fill_args(L, p, a);
    const int rows = L.cache.rows, box_rows = BN >> a.log_nb;
    {
        // the same: boxes of half a tile's chunks, or of one chunk of a page
        const uint64_t dims[4] = {64u, (uint64_t)rows, (uint64_t)C::NCH, (uint64_t)a.n_slots};
        const uint64_t strides[3] = {(uint64_t)C::W * 2, 128u, (uint64_t)C::W * 2 * rows};
        const uint32_t chunks[3] = {(uint32_t)NP, (uint32_t)NP + 1, 1u};
        for (int i = 0; i < 3; ++i) {
            const uint32_t box[4] = {64u, (uint32_t)box_rows, chunks[i], 1u};
            if ((st = encode_tmap_sw128(&tx[i], L.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, dims, strides, box)) != ATTN_OK)
                return st;
        }
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
    const int sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    const int grid = sms / a.side * a.side;
    const dim3 join(grid, NR * NP / join_width(NP, NR) / kJoinWarps);
    if (trace_enabled())
        trace("latent_attend_kernel<R=%d,rows=%d> grid=%d block=%d smem=%u tmem_cols=%u row_blocks=%d side=%d B=%d "
              "total_q=%d H=%d box_rows=%d whole=%d, then latent_join_kernel grid=(%u,%u)",
              C::R, NR, grid, kThreads, C::SMEM_ALLOC, C::TMEM_COLS, a.n_rb, a.side, L.B, L.total_q, L.H, box_rows,
              a.whole, a.whole ? 0 : join.x, a.whole ? 0 : join.y);
    // both are set up while the kernel before runs, and wait for its end themselves
    cudaError_t e = launch_dependent(kernel, dim3(grid), kThreads, C::SMEM_ALLOC, L.stream, tq, tx[0], tx[1], tx[2], a);
    if (e == cudaSuccess && !a.whole)
        e = launch_dependent(latent_join_kernel<NP, NR>, join, kJoinWarps * 32, 0, L.stream, a, grid);
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
    // Many blocks of 64 rows over long caches go to pairs of CTAs, which are faster a tile and slower to
    // start and to end (one GB300, here and in pairs: 32 sequences of 512 to 8192, 128 heads, 28 tiles an SM,
    // 61.4 and 57.3 us; 256 of 1024, 54 tiles, 124 and 110; a chunk of 512 tokens on 4096, 597 and 475; 8 sequences
    // of 4096, 7 tiles, 27.0 and 31.6; one of 3000 20.7 and 27.7; 256 latent values, 32 sequences of 4096: 33.7
    // and 41.6).  The two cross at 16 to 18 tiles an SM (128 heads, equal lengths, four caches in turn; 10, 14, 18
    // and 22 tiles: 32 sequences 35.7, 42.3, 48.1, 54.7 and 38.7, 43.3, 47.7, 52.3; 16 sequences 34.2, 40.3, 46.5, 52.8
    // and 37.0, 42.0, 46.3, 50.8).  Not chunks of one or two blocks, of which the shorter ones fill half a pair's (1
    // to 4 drafts of 32 heads of 16 x 32768: 141.7 and 145.5).  What the caches hold is not known here, only what
    // they can: short sequences in a wide table take the pairs' longer start and end (32 of 512 tokens, 128 heads:
    // 22.1 us in a table of 512, 26.4 in one of 32768).
    const long long blocks = L.B * p.n_rb;
    if (L.R == 512 && p.n_rb > (L.max_q == 1 ? 1 : 2) && blocks >= 32 &&
        blocks * ((L.cache.capacity + BN - 1) / BN) >= 16 * kMaxCtas)
        return launch_latent_pair(L);
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
