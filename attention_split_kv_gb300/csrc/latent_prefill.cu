// latent_prefill.cu -- the expanded form of latent attention (attn_latent_prefill) on the
// sm_103a tensor cores: packed sequences whose keys have a part of their own a head (128
// values) and a rotated part that all heads share (64), and values of 128.
//
//   o_ih = sum_j softmax_j(scale (q_ih[0:128] . k_jh + q_ih[128:192] . r_j)) v_jh
//
// over the keys j <= L - n + i (causal: the n queries are the last of the sequence's L
// tokens) or all of them.  The two parts are one product of depth 192 in the operands'
// chunks; the key is never put together in memory.
//
//   S  = Q K^T      128 queries x 128 keys, f32 in TMEM    (tcgen05.mma, 12 steps of 16)
//   P  = 2^(S scale log2e - m)     f16, over S in TMEM
//   O += P V        128 x 128, f32 in TMEM                 (P from TMEM, V MN-major)
//
// A CTA takes 256 queries of a head as two row tiles, each with its S/P and O (all 512 TMEM
// columns) and a softmax warpgroup; the two take turns on the tensor cores,
//
//   S0(0) S1(0) | PV0(j) S0(j+1) | PV1(j) S1(j+1) | ...
//
// so that one tile's softmax runs under the other's products (1280 cycles a turn at the
// tensor peak), and a key tile is read from shared memory's ring by both.  K and V lie in one
// ring of 16 KB chunks (64 values of 128 keys) in the order of their first use, which is also
// the order in which they are released: K(j) after S1(j), V(j) after PV1(j).
//
// A block of at most 128 queries has one row tile, which would wait for its own softmax.  Its even
// and odd key tiles are two streams instead, in the places of the two row tiles, each with its own
// offset, sum and O; the first stream's warps join them at the end.  (100 queries of 16 heads over
// 4096 keys 51.4 to 35.9 us, one query of 2 heads over 8000 keys 95 to 64.)  Where blocks of 256 would
// not fill the SMs, all blocks are of 128.
//
// What bounds it: a row tile's chain.  From S to the next S of the same row tile (430 cycles until
// the softmax has it, 230 to load it, 1550 for its weights, 180 until PV is issued, 540 and 680 of
// products) is 3600, for 2560 of products of both; 8192 tokens of 16 heads take 217 us, 1584
// TFLOP/s (84% of what a library's large product reaches here), tensor pipe 68%, in runs of 20 calls; under
// the power cap, which brings the SMs from 2070 to 1720 MHz, 237 us, 1450 TFLOP/s (86% of the library's there),
// and 240 with six inputs in turn.  Rows shared by
// two threads, 16 softmax warps, made it 243; a barrier a chunk instead of a tile (12 waits and 7
// commits a turn, not 4 and 4) 231; waits with a suspend-time hint 226.
//
// Roles (12 warps): 8 softmax warps (row tile w / 4), a TMA warp, an MMA warp, 2 idle.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int BM = 128, BN = 128;           // rows of a row tile, keys of a key tile
constexpr int HD = 128, RD = 64;            // a head's values, the rotated part's
constexpr float kLog2e = 1.4426950408889634f;
// A row's weights are 2^(logit - its offset) in f16: the offset lies kLift below the row's maximum when it is
// set, and is set again when a logit passes it by kRescaleThreshold (log2 units).  So the largest weight is 2^7
// to 2^15 (f16 holds 65504), and of the others what is above 2^-25 is kept, 2^-32 or less of the largest.
constexpr float kLift = 7.0f, kRescaleThreshold = 15.0f;
constexpr float kFastSumLimit = 32768.0f;   // a row whose p sum to at most this has every p <= 2^15
constexpr int kSoftmaxWarps = 8, kTmaWarp = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + 1;
// 3 warpgroups: 8 softmax warps, then the TMA warp, the MMA warp and two that only make up the
// third, which leaves registers to the others (launch: 384 x 168)
constexpr int kThreads = 384;
constexpr int kRegSoftmax = 208, kRegOther = 88;
static_assert(2 * kRegSoftmax + kRegOther == 3 * 168, "register split");
constexpr int kMaxRanked = 128;   // most (sequence, block) pairs that are ranked
constexpr int RING = 8, K_CHUNKS = 3, V_CHUNKS = 2, CHUNKS = K_CHUNKS + V_CHUNKS;
constexpr uint32_t kChunk = BN * 128;       // 64 values of 128 keys (or queries)
constexpr uint32_t OFF_Q = 0, OFF_RING = 2 * K_CHUNKS * kChunk, OFF_BAR = OFF_RING + RING * kChunk;
// barriers: of K tiles (even, odd), V tiles, their release; of each stream: S, weights, the last PV
// done; the second stream's rows are there
enum : int { B_Q, B_K = B_Q + 2, B_V = B_K + 2, B_KFREE = B_V + 2, B_VFREE = B_KFREE + 2, B_S = B_VFREE + 2, B_P = B_S + 2,
             B_DONE = B_P + 2, B_JOIN = B_DONE + 2, B_TEARDOWN, N_BARS };
constexpr uint32_t OFF_ML = (OFF_BAR + N_BARS * 8 + 15) / 16 * 16;   // the second stream's offsets and sums
constexpr uint32_t OFF_MISC = OFF_ML + BM * 8, SMEM_ALLOC = OFF_MISC + 8 + 1024;
constexpr uint32_t COL_O = 2 * BN, TMEM_COLS = 512;
static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
static_assert(2 * (SMEM_ALLOC + 1024) > 233472, "one CTA an SM: its TMEM allocation never waits");

struct Args {
    __half* out;
    float* lse;
    const int32_t *q_start, *kv_start;
    int total_q, max_q, H, causal;
    int B, blocks;   // sequences, blocks of the longest
    int rows;        // queries of a block: 128 or 256
    int ranked;      // the grid's CTAs take (sequence, block) pairs longest first
    float scale;
    int* err;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float row_max(const float (&t)[BN]) {
    float a[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = t[k];
#pragma unroll
    for (int i = 8; i + 16 <= BN; i += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = max3(a[k], t[i + k], t[i + 8 + k]);
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = fmaxf(a[k], t[BN - 8 + k]);
    return fmaxf(max3(a[0], a[1], a[2]), max3(a[3], a[4], max3(a[5], a[6], a[7])));
}

// What a CTA does: queries q0 .. of head h of one sequence.
struct Work {
    int h, q_base, k_base, q0, n_q;   // first rows of q and of the keys; queries of the sequence
    int L, pos0;                      // its keys, the position of query 0
    int n_keys;                       // key tiles
    int n_tiles[2];                   // steps of each stream
};

// The roles of a CTA's warps, after its barriers and tensor memory are set up.  SPLIT: a block of at
// most 128 queries has one row tile, which would wait for its own softmax; its even and odd key
// tiles are two streams instead, joined at the end.  Stream t's step i takes key tile j = 2 i + t;
// else it is row tile t, and j = i.
template <bool SPLIT>
__device__ __forceinline__ void run_roles(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_r,
                                          const CUtensorMap& tm_v, const Args& a, const Work& w, uint8_t* smem,
                                          uint32_t tmem) {
    const uint32_t sbase = smem_u32(smem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + OFF_BAR + i * 8; };
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int n = max(w.n_tiles[0], w.n_tiles[1]);   // steps
    auto key_tile = [&](int t, int i) { return SPLIT ? 2 * i + t : i; };
    // The ring's first chunk of K(j) and of V(j).  Streams first use K0 K1 V0 K2 V1 K3 V2 ..
    auto k_at = [&](int j) { return !SPLIT ? j * CHUNKS : j ? j * CHUNKS - 2 : 0; };
    auto v_at = [&](int j) { return !SPLIT || j == w.n_keys - 1 ? j * CHUNKS + K_CHUNKS : j * CHUNKS + 6; };

    // A wait of a whole warp, with one answer for all of its lanes.
    auto wait = [&](int i, uint32_t parity, int code) -> bool {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity))) return true;
        const uint64_t t0 = globaltimer();
        const uint64_t limit = *static_cast<volatile unsigned long long*>(&g_wait_limit_ns);
#pragma unroll 1
        do {
            if (__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity))) return true;
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
        } while (__any_sync(0xffffffffu, globaltimer() - t0 < limit));
        *abort_flag = 1;
        atomicExch(a.err, code);
        return false;
    };

    if (warp >= kSoftmaxWarps) {
    // (setmaxnreg is executed by all four warps of a warpgroup)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegOther));
    if (warp == kTmaWarp) {
        // ------------------------------------------------------------ TMA
        // (the whole warp runs the code; one lane issues)
        const uint32_t one = elect_one();
        int k_posted = 0, v_posted = 0;
        bool ok = true;
        const int n_q_tiles = !SPLIT && w.n_tiles[1] > 0 ? 2 : 1;
        for (int t = 0; t < n_q_tiles; ++t) {
            mbar_arrive_expect_tx_one(one, bar(B_Q + t), K_CHUNKS * kChunk);
            for (int c = 0; c < K_CHUNKS; ++c)
                tma_load_3d_one(one, sbase + OFF_Q + (t * K_CHUNKS + c) * kChunk, &tm_q, bar(B_Q + t), c * 64, w.h,
                                w.q_base + w.q0 + t * BM);
        }
        auto k_free = [&](int j) { return wait(B_KFREE + (j & 1), (j >> 1) & 1, kErrTimeoutSlot); };
        auto v_free = [&](int j) { return wait(B_VFREE + (j & 1), (j >> 1) & 1, kErrTimeoutSlot); };
        auto load_k = [&](int j) {
            uint32_t s = k_at(j) % RING;
            mbar_arrive_expect_tx_one(one, bar(B_K + (j & 1)), K_CHUNKS * kChunk);
            for (int c = 0; c < 2; ++c, s = (s + 1) % RING)
                tma_load_3d_one(one, sbase + OFF_RING + s * kChunk, &tm_k, bar(B_K + (j & 1)), c * 64, w.h, w.k_base + j * BN);
            tma_load_3d_one(one, sbase + OFF_RING + s * kChunk, &tm_r, bar(B_K + (j & 1)), 0, 0, w.k_base + j * BN);
            ++k_posted;
        };
        auto load_v = [&](int j) {
            uint32_t s = v_at(j) % RING;
            mbar_arrive_expect_tx_one(one, bar(B_V + (j & 1)), V_CHUNKS * kChunk);
            for (int c = 0; c < V_CHUNKS; ++c, s = (s + 1) % RING)
                tma_load_3d_one(one, sbase + OFF_RING + s * kChunk, &tm_v, bar(B_V + (j & 1)), c * 64, w.h, w.k_base + j * BN);
            ++v_posted;
        };
        if (!SPLIT) {
            // K(j) takes the places of K(j - 2)'s last chunk and V(j - 2), V(j) of K(j - 1)'s first two
            for (int j = 0; j < n; ++j) {
                if (j > 1 && !(ok = v_free(j - 2))) break;
                load_k(j);
                if (j > 0 && !(ok = k_free(j - 1))) break;
                load_v(j);
            }
        } else {
            // K(2) takes the places of K(0), a later K(j) of K(j - 2)'s last chunk and V(j - 3), V(j) of
            // K(j)'s own first two, the last V of K(j - 1)'s last chunk and V(j - 2)'s first
            load_k(0);
            for (int j = 1; j <= w.n_keys; ++j) {
                if (j < w.n_keys) {
                    if (j == 2 && !(ok = k_free(0))) break;
                    if (j > 2 && !(ok = v_free(j - 3))) break;
                    load_k(j);
                    if (j > 1 && !(ok = k_free(j - 1))) break;
                } else {
                    if (j == 2 && !(ok = k_free(0))) break;
                    if (j > 2 && !(ok = v_free(j - 3))) break;
                }
                load_v(j - 1);
            }
        }
        if (!ok || __any_sync(0xffffffffu, *abort_flag)) {
            // let copies already in flight land before the CTA's shared memory goes away
            if (lane == 0) {
                for (int t = 0; t < n_q_tiles; ++t) mbar_wait_drain(bar(B_Q + t), 0, a.err, kErrTimeoutLoad);
                for (int j = max(k_posted - 2, 0); j < k_posted; ++j)
                    mbar_wait_drain(bar(B_K + (j & 1)), (j >> 1) & 1, a.err, kErrTimeoutLoad);
                for (int j = max(v_posted - 2, 0); j < v_posted; ++j)
                    mbar_wait_drain(bar(B_V + (j & 1)), (j >> 1) & 1, a.err, kErrTimeoutLoad);
            }
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        // (the whole warp runs the code; one lane issues)
        const uint32_t one = elect_one();
        constexpr uint32_t id_s = idesc_f16_f32(BM, BN, false), id_o = idesc_f16_f32(BM, 64, true);
        const uint64_t q_desc = smem_desc_sw128(sbase + OFF_Q, 16, 1024);
        const uint64_t x_desc = smem_desc_sw128(sbase + OFF_RING, 16, 1024);
        const bool stall = stall_first_tile();
        bool ok = true;
        // Row tile 1 finds what row tile 0 has taken, and releases it.
        auto issue_s = [&](int t, int i) -> bool {
            const int j = key_tile(t, i);
            if (i < w.n_tiles[t]) {
                if (i == 0 && (t == 0 || !SPLIT) && !wait(B_Q + t, 0, kErrTimeoutLoad)) return false;
                if ((SPLIT || t == 0 || i >= w.n_tiles[0]) && !wait(B_K + (j & 1), (j >> 1) & 1, kErrTimeoutLoad)) return false;
                tc_fence_after();
                const uint64_t q = desc_advance(q_desc, SPLIT ? 0 : t * K_CHUNKS * kChunk);
                uint32_t s = k_at(j) % RING;
#pragma unroll
                for (int c = 0; c < K_CHUNKS; ++c, s = (s + 1) % RING) {
                    const uint64_t kd = desc_advance(x_desc, s * kChunk);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_f16_ss_one(one, tmem + t * BN, desc_advance(q, c * kChunk + kk * 32), desc_advance(kd, kk * 32),
                                          id_s, (c | kk) != 0);
                }
                if (!(stall && i == 0)) tc_commit_one(one, bar(B_S + t));
            }
            if (SPLIT ? i < w.n_tiles[t] : t == 1 && i < n) tc_commit_one(one, bar(B_KFREE + (j & 1)));
            return true;
        };
        auto issue_pv = [&](int t, int i) -> bool {
            const int j = key_tile(t, i);
            if (i < w.n_tiles[t]) {
                if (!wait(B_P + t, i & 1, kErrTimeoutSoftmax)) return false;
                if ((SPLIT || t == 0 || i >= w.n_tiles[0]) && !wait(B_V + (j & 1), (j >> 1) & 1, kErrTimeoutLoad)) return false;
                tc_fence_after();
                uint32_t s = v_at(j) % RING;
#pragma unroll
                for (int c = 0; c < V_CHUNKS; ++c, s = (s + 1) % RING) {
                    const uint64_t vd = desc_advance(x_desc, s * kChunk);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)   // 16 keys: 8 columns of P, 16 lines of V
                        tc_mma_f16_ts_one(one, tmem + COL_O + t * HD + c * 64, tmem + t * BN + kk * 8,
                                          desc_advance(vd, kk * 2048), id_o, (i | kk) != 0);
                }
                if (i == w.n_tiles[t] - 1) tc_commit_one(one, bar(B_DONE + t));
            }
            if (SPLIT ? i < w.n_tiles[t] : t == 1) tc_commit_one(one, bar(B_VFREE + (j & 1)));
            return true;
        };
        ok = issue_s(0, 0) && issue_s(1, 0);
        for (int i = 0; ok && i < n; ++i) ok = issue_pv(0, i) && issue_s(0, i + 1) && issue_pv(1, i) && issue_s(1, i + 1);
        // all issued MMAs must retire before TMEM is released
        tc_commit_one(one, bar(B_TEARDOWN));
        if (lane == 0) mbar_wait_drain(bar(B_TEARDOWN), 0, a.err, kErrTimeoutMma);
        __syncwarp();
    }
    } else {
        // ------------------------------------------------------------ softmax, and the rows out
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax));
        const int t = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const int qi = w.q0 + (SPLIT ? 0 : t * BM) + row;       // this thread's query
        const int keep = a.causal ? min(w.L, w.pos0 + qi + 1) : w.L;   // it keeps the keys below this
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t s_addr = lanes + t * BN, o_addr = lanes + COL_O + t * HD;
        const int my_tiles = w.n_tiles[t];
        // logits are raw products times scale > 0 in the exponent; another scale goes in first
        const bool raw = a.scale > 0.f;
        const float to_log2 = raw ? a.scale * kLog2e : 1.f;
        float m = -INFINITY, l = 0.f;      // m: the offset, of the products times to_log2
        bool ok = true;
        for (int i = 0; i < my_tiles; ++i) {
            const int j = key_tile(t, i);
            if (!(ok = wait(B_S + t, i & 1, kErrTimeoutMma))) break;
            tc_fence_after();
            float x[BN];
            {
                uint32_t r[BN];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c)
                    tc_ld_32x32b_x32(s_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(r + c * 32));
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < BN; ++i) x[i] = __uint_as_float(r[i]);
            }
            if (!raw) {
#pragma unroll
                for (int i = 0; i < BN; ++i) x[i] *= a.scale * kLog2e;
            }
            const int key0 = j * BN;
            if (key0 + BN > keep) {
#pragma unroll
                for (int i = 0; i < BN; ++i)
                    if (key0 + i >= keep) x[i] = -INFINITY;
            }
            // weights against the offset m_off, rounded to f16 and stored over S; returns their sum
            // (of the rounded ones, so that a row stays a convex combination of values)
            auto exps = [&](float m_off) -> float {
                float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                const float2 f2 = make_float2(to_log2, to_log2), nm2 = make_float2(-m_off, -m_off);
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t packed[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 y = ffma2(make_float2(x[c * 32 + i], x[c * 32 + i + 1]), f2, nm2);
                        const __half2 hp = __floats2half2_rn(ex2_approx(y.x), ex2_approx(y.y));
                        packed[i / 2] = *reinterpret_cast<const uint32_t*>(&hp);
                        const int k = (i / 2) & 3;
                        ls[2 * k] = add_f16_lo(ls[2 * k], packed[i / 2]);
                        ls[2 * k + 1] = add_f16_hi(ls[2 * k + 1], packed[i / 2]);
                    }
                    tc_st_32x32b_x16(s_addr + c * 16, packed);
                }
                return ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
            };
            // First against the running offset, without the tile's maximum: a warp with a row whose
            // weights sum to more than 2^15 (or a NaN, or no key so far) takes that.
            bool fast = false;
            if (__all_sync(0xffffffffu, m != -INFINITY)) {
                const float s = exps(m);
                fast = __all_sync(0xffffffffu, s <= kFastSumLimit);
                if (fast) l += s;
            }
            if (!fast) {
                const float top = row_max(x) * to_log2;
                const bool need = top - m > kRescaleThreshold;   // (no key so far: m -inf)
                const bool rescale = __any_sync(0xffffffffu, need) && i > 0;
                float alpha = 1.f;
                if (need) {
                    alpha = m == -INFINITY ? 0.f : ex2_approx(m - (top - kLift));
                    l *= alpha;
                    m = top - kLift;
                }
                l += exps(m == -INFINITY ? 0.f : m);
                if (rescale) {
                    // (PV of the tile before is done: S of this one was issued after it)
#pragma unroll 1
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t r[32];
                        tc_ld_32x32b_x32(o_addr + c * 32, r);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                        tc_st_32x32b_x32(o_addr + c * 32, r);
                    }
                }
            }
            if (key0 + BN > w.L) {
                // rows behind the sequence's keys are another's, or nothing: their values are zeroed,
                // since a weight of 0 must not meet a NaN.  (Both row tiles do it, each before its PV.)
                const int r0 = max(w.L - key0, 0), units = (BN - r0) * 8;   // 16 bytes each
                if (!(ok = wait(B_V + (j & 1), (j >> 1) & 1, kErrTimeoutLoad))) break;
                for (int c = 0; c < V_CHUNKS; ++c) {
                    uint8_t* at = smem + OFF_RING + (v_at(j) + c) % RING * kChunk + r0 * 128;
                    for (int u = tid & 127; u < units; u += 128) *reinterpret_cast<uint4*>(at + u * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + t));
        }
        if (ok && my_tiles > 0) ok = wait(B_DONE + t, 0, kErrTimeoutMma);
        // of two streams the first one's warps join the rows
        float2* ml = reinterpret_cast<float2*>(smem + OFF_ML);
        float f0 = 1.f, f1 = 0.f;
        if (ok && SPLIT) {
            if (t == 1) {
                ml[row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_JOIN));
            } else if ((ok = wait(B_JOIN, 0, kErrTimeoutSoftmax) && wait(B_DONE + 1, 0, kErrTimeoutMma))) {
                const float2 other = ml[row];
                const float top = fmaxf(m, other.x);
                f0 = m == -INFINITY ? 0.f : ex2_approx(m - top);
                f1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - top);
                l = f0 * l + f1 * other.y;
                m = top;
            }
        }
        if (ok && my_tiles > 0 && !(SPLIT && t == 1)) {
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.0f / l;   // no key: zeros; NaN stays NaN
            f0 *= inv;
            f1 *= inv;
            const int orow = w.q_base + qi;
            const bool live = qi < w.n_q && orow >= 0 && orow < a.total_q;
            __half* dst = a.out + (static_cast<size_t>(live ? orow : 0) * a.H + w.h) * HD;
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
                float o[32];
                {
                    uint32_t r[32];
                    tc_ld_32x32b_x32(o_addr + c * 32, r);
                    tc_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(r[i]) * f0;
                    if (SPLIT) {
                        tc_ld_32x32b_x32(o_addr + HD + c * 32, r);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(__uint_as_float(r[i]), f1, o[i]);
                    }
                }
                uint32_t hv[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const __half2 p2 = __floats2half2_rn(o[2 * i], o[2 * i + 1]);
                    hv[i] = *reinterpret_cast<const uint32_t*>(&p2);
                }
                if (live) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<uint4*>(dst + c * 32)[i] = make_uint4(hv[4 * i], hv[4 * i + 1], hv[4 * i + 2], hv[4 * i + 3]);
                }
            }
            if (a.lse && live)
                a.lse[static_cast<size_t>(orow) * a.H + w.h] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
        }
    }
}

// STREAMS: with the code for blocks of one row tile.
template <bool STREAMS>
__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v, const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + OFF_BAR + i * 8; };
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

    const int rows = STREAMS ? a.rows : 2 * BM;   // of a block
    // Heads fastest, then blocks of 256 (or 128) queries: of few sequences all of them ranked by the work
    // they are, the most first (8 chunks of 33 to 700 tokens over 739 to 3900: 103 us in the
    // sequences' order), else sequence by sequence from the last block (the longest when causal).
    int h = blockIdx.x, b = blockIdx.z, block = static_cast<int>(gridDim.y - 1 - blockIdx.y);
    if (a.ranked) {
        int* work = reinterpret_cast<int*>(smem + OFF_Q);   // before any copy
        const int n_pairs = a.B * a.blocks, want = static_cast<int>(blockIdx.x) / a.H;
        int mine = -1;                           // no queries: last
        if (tid < n_pairs) {
            const int bb = tid / a.blocks, first = tid % a.blocks * rows;
            const int all = max(a.q_start[bb + 1] - a.q_start[bb], 0), keys = max(a.kv_start[bb + 1] - a.kv_start[bb], 0);
            const int nq = min(all, a.max_q);
            if (first < nq) {
                const int end = min(first + rows, nq);
                const int hi = a.causal ? max(min(keys, keys - all + end), 0) : keys;
                mine = (hi / BN + 1) * (end - first > BM ? 2 : 1);   // (a key tile for one row tile: half the time)
            }
            work[tid] = mine;
        }
        __syncthreads();
        if (tid < n_pairs) {
            int rank = 0;
            for (int i = 0; i < n_pairs; ++i) rank += work[i] > mine || (work[i] == mine && i < tid);
            if (rank == want) work[kMaxRanked] = tid;   // (ranks are a permutation: one writer)
        }
        __syncthreads();
        const int pair = work[kMaxRanked];
        b = pair / a.blocks;
        block = pair % a.blocks;
        h = static_cast<int>(blockIdx.x) % a.H;
        fence_proxy_async_smem();
        __syncthreads();                         // (before Q is copied over it)
    }
    const int q_base = a.q_start[b], k_base = a.kv_start[b];
    const int n_all = max(a.q_start[b + 1] - q_base, 0), L = max(a.kv_start[b + 1] - k_base, 0);
    const int n_q = min(n_all, a.max_q);
    const int q0 = block * rows;
    if (q0 >= n_q) return;                       // a shorter sequence: no queries for this CTA
    const int pos0 = L - n_all;                  // position of query 0
    // key tiles of each row tile (at least one where it has rows)
    int n_tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = q0 + t * BM, last = min(first + BM, n_q) - 1;
        const int hi = a.causal ? max(min(L, pos0 + last + 1), 0) : L;
        n_tiles[t] = first < n_q && t * BM < rows ? max((hi + BN - 1) / BN, 1) : 0;
    }
    const int n_keys = max(n_tiles[0], n_tiles[1]);
    const bool split = STREAMS && n_tiles[1] == 0 && n_keys > 1;
    if (split) {
        n_tiles[1] = n_keys / 2;
        n_tiles[0] = n_keys - n_tiles[1];
    }
    if (tid == 0) {
        for (int i = 0; i < N_BARS; ++i) mbar_init(bar(i), i == B_P || i == B_P + 1 || i == B_JOIN ? 4 : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_holder), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);

    const Work w{h, q_base, k_base, q0, n_q, L, pos0, n_keys, {n_tiles[0], n_tiles[1]}};
    if constexpr (STREAMS) {
        if (split) run_roles<true>(tm_q, tm_k, tm_r, tm_v, a, w, smem, tmem);
        else run_roles<false>(tm_q, tm_k, tm_r, tm_v, a, w, smem, tmem);
    } else {
        run_roles<false>(tm_q, tm_k, tm_r, tm_v, a, w, smem, tmem);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// f16 rows [rows, H, n] with strides in elements, in boxes of 64 values of 128 rows of a head.
attn_status rows_map(CUtensorMap* m, const void* base, int n, int H, int rows, long long head_stride, long long stride) {
    const uint64_t dims[3] = {(uint64_t)n, (uint64_t)H, (uint64_t)rows};
    const uint64_t strides[2] = {(uint64_t)head_stride * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64u, 1u, (uint32_t)BN};
    return encode_tmap_sw128(m, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, dims, strides, box);
}

}  // namespace

attn_status launch_latent_prefill(const LatentPrefillLaunch& L) {
    CUtensorMap tq, tk, tr, tv;
    attn_status st;
    if ((st = rows_map(&tq, L.q, HD + RD, L.H, L.total_q, HD + RD, L.q_stride)) != ATTN_OK) return st;
    if ((st = rows_map(&tk, L.k, HD, L.H, L.total_kv, L.k_head_stride, L.k_stride)) != ATTN_OK) return st;
    if ((st = rows_map(&tv, L.v, HD, L.H, L.total_kv, L.v_head_stride, L.v_stride)) != ATTN_OK) return st;
    if ((st = rows_map(&tr, L.k_rope, RD, 1, L.total_kv, RD, L.k_rope_stride)) != ATTN_OK) return st;
    // Blocks of 256 queries that do not fill the SMs are halved, each half with its keys in two streams (one
    // sequence of 16 heads: 300 queries over 4096 keys 61 to 37 us, a prompt of 1024 tokens 21 to 15, of 2048
    // 36 to 28; of 3000, 192 blocks, 49 to 51, and 8 ragged chunks, 304 blocks, 69 to 71).
    const long long most = (static_cast<long long>(L.total_q) / (2 * BM) + L.B) * L.H;
    const int rows = most <= sm_count() ? BM : 2 * BM;
    // A lone sequence of more blocks has at most one short one, beside full ones that take longer, and runs
    // faster without the streams' code (8192 tokens of 16 heads 217 us, with it 225); several with it (8
    // ragged chunks 78.6 us, without 79.5).
    const bool streams = rows == BM || L.B > 1 || L.max_q <= BM;
    auto kernel = streams ? latent_prefill_kernel<true> : latent_prefill_kernel<false>;
    static bool attr_set[2][64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[streams][dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC) != cudaSuccess)
            return set_error(ATTN_ECUDA, "cudaFuncSetAttribute(latent prefill smem) failed");
        if (dev >= 0 && dev < 64) attr_set[streams][dev] = true;
    }
    Args a;
    a.out = static_cast<__half*>(L.out);
    a.lse = L.lse;
    a.q_start = L.q_start;
    a.kv_start = L.kv_start;
    a.total_q = L.total_q;
    a.max_q = L.max_q;
    a.H = L.H;
    a.causal = L.causal;
    a.scale = L.scale;
    a.err = L.err_word;
    a.B = L.B;
    a.rows = rows;
    a.blocks = (L.max_q - 1) / rows + 1;
    a.ranked = L.B > 1 && static_cast<long long>(L.B) * a.blocks <= kMaxRanked;
    const dim3 grid = a.ranked ? dim3(L.B * a.blocks * L.H) : dim3(L.H, a.blocks, L.B);
    if (trace_enabled())
        trace("latent_prefill_kernel grid=(%u,%u,%u) block=%d smem=%u tmem_cols=%u total_q=%d total_kv=%d H=%d causal=%d ranked=%d streams=%d rows=%d",
              grid.x, grid.y, grid.z, kThreads, SMEM_ALLOC, TMEM_COLS, L.total_q, L.total_kv, L.H, L.causal, a.ranked, (int)streams, rows);
    kernel<<<grid, kThreads, SMEM_ALLOC, L.stream>>>(tq, tk, tr, tv, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "latent prefill launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

// Sets this translation unit's test controls (see ptx.cuh).
attn_status set_test_controls_latent_prefill(unsigned long long wait_limit_ns, int stall) {
    if (cudaMemcpyToSymbol(g_wait_limit_ns, &wait_limit_ns, sizeof(wait_limit_ns)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_stall_first_tile, &stall, sizeof(stall)) != cudaSuccess)
        return set_error(ATTN_ECUDA, "test controls (latent prefill): %s", cudaGetErrorString(cudaGetLastError()));
    return ATTN_OK;
}

}  // namespace attn
