// prefill_int8.cu -- a chunk of new tokens of every sequence over its int8 paged
// cache (attn_prefill_paged_ex with ATTN_KV_INT8) on the sm_103a tensor cores.
//
//   o_i = sum_j softmax_j(cap(scale ks_j q_i . kc_j)) vs_j vc_j
//
// over the keys j <= pos_i (and pos_i - j < W), with codes kc, vc and one scale
// ks_j, vs_j a (token, kv head).  Codes are integers of at most 8 bits, so they are
// exact as f16 operands and neither K nor V is rounded:
//
//   S   = Q Kc^T                                 (tcgen05.mma, f32 in TMEM)
//   y_j = S_j (ks_j scale log2e) + log2 vs_j     (one packed fma)
//   P_j = f16(2^(y_j - m)),  m the running maximum of y
//   O  += P Vc,   l += r(2^(y_j - m)) / vs_j     (tcgen05.mma; f32)
//
// so the value's scale sits in its weight, and the weight is rounded once, relative
// to the row's largest weighted scale.  out = O / l, lse = (m + log2 l) / log2e.
// r rounds to the 11 bits that f16 keeps, with f32's exponents: the sum is then over the
// weights that the product uses, so out is a convex combination of values and a dominant
// key gives its value exactly (with the unrounded weights: off by up to 2^-11 of it).  f16
// itself will not do for the sum, because a key of a small value scale can have a weight
// far below f16's normal range and still most of the row's mass.  The rounding costs 8
// chunks of 512 tokens 8% (303 us without it) and calls of few rows at most 1%.
//
// Rows are packed: the query heads that share a kv head are rows of one tile beside
// its queries (row r is query r / HG, head r % HG), so a decode step or a few draft
// tokens read their cache once.  A group of rows is one 128-row tile, or two.
//
// Persistent CTAs: the key tiles of all (sequence, row group, head) items, in that
// order, are cut into equal runs, one a CTA.  An item inside one run is written
// directly; one that runs over a boundary leaves unnormalised partial rows in the
// workspace, which a second kernel joins.  Long caches with few rows and short ones
// with many are balanced by the same cut, without the host knowing any length.
//
// Roles (20 warps): a K and a V warp bring code tiles into a ring of stages (TMA, a box a
// page); 8 converter warps turn codes into f16 operands (128-byte swizzle) in a ring of 3;
// one warp issues the MMAs; one walks the run, loads Q and writes the per-key factors; 8
// softmax warps.  D = 64/128 keep two streams, each with its S (P overwrites it) and O in
// TMEM and 4 softmax warps, which take turns on the tensor cores: the two row tiles of a
// group, or for a single tile the even and the odd key tiles, joined at the end.  D = 256
// has one O (its 256 columns) and tiles of 64 keys, with two S and P buffers beside it; all
// 8 softmax warps, 16 rows each, take every tile.
//
// What bounds it: shared memory.  Codes are written by TMA, read, stored at twice the size
// and read by the MMA, so a 128-key tile of one row tile (D = 128) takes 2170 wavefronts of
// 128 bytes (LSU 1150, MMA operands 768, TMA 256) in 2650 to 2790 cycles: 524288 cached
// tokens of 8 kv heads and 4 new ones of 32 heads take 304 us, 3.6 TB/s (HBM alone: 161 us);
// 1 to 8 new tokens of 32 sequences of 512 to 8192, 98 us, 3.0 TB/s.  With two row tiles one
// conversion serves both, and the softmax's chain (S, 3500 cycles of softmax, PV, the next S)
// comes to the front: 8 chunks of 512 tokens on 1 to 7680 cached ones (32/8 heads) take
// 319 us, 744 TFLOP/s, tensor pipe 33%, issue slots 53%, shared memory 61%.  16 softmax warps
// of 16 rows do not shorten it (305 to 307 us): a 16-byte factor load takes 4 wavefronts, and
// with half the rows a load serves half as much.  D = 256 with a softcap and a window of 1024
// keys: 70 us, 432 TFLOP/s: shared memory (3200 wavefronts a 64-key tile: Q is read anew for
// each) and each segment's fixed part.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int BM = 128;                     // rows of a tile (TMEM lanes)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays at most 2^8
constexpr int kMaxCtas = 152;               // one CTA an SM
constexpr int kMinTiles = 2;                // least key tiles of a run
// 5 warpgroups.  Registers at launch: 640 x 96; the softmax warpgroups then take
// theirs from the last one's and the converters'.
constexpr int kThreads = 640;
constexpr int kRegSoftmax = 152, kRegConvert = 56, kRegOther = 64;
static_assert(2 * kRegSoftmax + 2 * kRegConvert + kRegOther == 5 * 96, "register split");

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// x rounded to 11 significant bits (to nearest even, as f16 rounds in its normal range).
__device__ __forceinline__ float2 round11(float2 x) {
    uint32_t a, b;
    asm("cvt.rn.tf32.f32 %0, %1;" : "=r"(a) : "f"(x.x));
    asm("cvt.rn.tf32.f32 %0, %1;" : "=r"(b) : "f"(x.y));
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}
// One arrival of a whole warp: its lanes' earlier writes are ordered before it.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// Per-key factors of a key tile, laid out as the softmax threads read them (a pair
// of keys a time), and the sign of the value's scale for the converters.
template <int BN>
struct KeyFactors {
    float4 a[BN / 2];      // {ks, ks', log2 vs, log2 vs'}: ks times scale (and log2e, or 1 / cap)
    float2 b[BN / 2];      // {1 / vs, 1 / vs'}
    uint32_t sign[BN];     // f16x2 of 1, -1, or 0 for a value that counts as zero
};

template <int D, int NT>
struct Cfg {
    static constexpr int BN = D == 256 ? 64 : 128;       // keys a tile
    static constexpr int NCH = D / 64;                   // 128-byte chunks of a row of f16
    static constexpr int NS = D == 256 ? 1 : 2;          // streams (O accumulators)
    static constexpr int NSM = 8, NCV = 8;               // softmax and converter warps
    static constexpr int K_WARP = 16, MMA_WARP = 17, V_WARP = 18;   // 19: per-key factors and Q
    static constexpr int RING = 3;                       // f16 operand tiles
    // staged code tiles: what shared memory leaves beside Q and the operand ring
    static constexpr int NST = D == 64 ? 8 : D == 128 ? (NT == 1 ? 5 : 3) : 3;
    static constexpr int NTAB = 4;                       // key-factor tables
    // what a segment costs beside its key tiles (filling the pipeline, writing its rows), in
    // key tiles.  8 x 512 chunks (D = 128): 337 us unweighted, 304 with 2, 302 with 3, 305 with
    // 4; the sum of eight D = 256 calls (prompts, chunks, drafts): 620, 611, 616, 620 and 631 us
    // with 1, 2, 3, 4 and 6
    static constexpr int SEG_TILES = D == 256 ? 2 : 3;
    static constexpr int SEGS = 4;                       // segment descriptions
    static constexpr uint32_t Q_TILE = NCH * BM * 128;
    static constexpr uint32_t OP_CHUNK = BN * 128, OP_BYTES = NCH * OP_CHUNK;
    static constexpr int IDS = 8, SCALES = 4;            // rings of prefetched page ids and scales (tiles)
    static constexpr uint32_t CODE_BYTES = BN * D, SCALE_BYTES = 2 * BN * 2;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_OP = OFF_Q + NT * Q_TILE;
    static constexpr uint32_t OFF_CODE = OFF_OP + RING * OP_BYTES;
    static constexpr uint32_t OFF_SCALE = OFF_CODE + NST * CODE_BYTES;
    static constexpr uint32_t OFF_IDS = OFF_SCALE + SCALES * SCALE_BYTES;
    // (of the factor, the K and the V warp: one a box)
    static constexpr uint32_t OFF_TAB = OFF_IDS + 3 * IDS * 16 * 4;
    static constexpr uint32_t OFF_ML = OFF_TAB + NTAB * sizeof(KeyFactors<BN>);
    static constexpr uint32_t OFF_BAR = OFF_ML + 2 * BM * 8;   // row statistics [warpgroup][row]
    enum : int {
        B_SFULL_ST = 0,                    // stage: codes are there
        B_SEMPTY_ST = B_SFULL_ST + NST,    // stage: converted
        B_OPFULL = B_SEMPTY_ST + NST,      // operand tile: converted
        B_OPEMPTY = B_OPFULL + RING,       // operand tile: its MMAs are done
        B_TAB = B_OPEMPTY + RING,          // key factors are there
        B_TABEMPTY = B_TAB + NTAB,         // their tile's P are done, and its V is converted
        B_SEG = B_TABEMPTY + NTAB,         // segment descriptions
        B_SEGFREE = B_SEG + SEGS,          // no warp needs it any more
        B_QFULL = B_SEGFREE + SEGS,
        B_QEMPTY,
        B_S,                               // S of buffer 0, 1
        B_SFREE = B_S + 2,                 // it has been read (D = 256)
        B_P = B_SFREE + 2,                 // P of buffer 0, 1
        B_PV = B_P + 2,                    // its PV is done (D = 64/128: of the tile's first 64 keys)
        B_PH = B_PV + 2,                   // P of the first 64 keys (D = 64/128)
        B_DONE = B_PH + 2,                 // a segment's last PV is done
        B_OFREE,                           // its O has been read
        B_ML,                              // its row statistics are in shared memory
        B_TEARDOWN,
        N_BARS
    };
    static constexpr uint32_t OFF_MISC = OFF_BAR + N_BARS * 8;   // TMEM base, abort flag, start
    static constexpr uint32_t OFF_FILLS = OFF_MISC + 8;
    static constexpr uint32_t OFF_SEG = (OFF_FILLS + NST * 4 + 7) / 8 * 8;
    static constexpr uint32_t SMEM_ALLOC = OFF_SEG + (SEGS + 1) * 80 + 1024;   // 80: sizeof(Seg)
    // TMEM: S of two units, P (D = 64/128: over the S it was made from), then O
    static constexpr bool OVER = D <= 128;
    static constexpr uint32_t COL_P = OVER ? 0 : 2 * BN, P_STRIDE = OVER ? BN : BN / 2;
    static constexpr uint32_t COL_O = OVER ? 2 * BN : 2 * BN + BN;
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(OFF_SEG % 8 == 0, "alignment");
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(2 * (SMEM_ALLOC + 1024) > 233472, "one CTA an SM: its TMEM allocation never waits");
    static_assert(COL_O + NS * D <= TMEM_COLS, "TMEM budget");
    static_assert(D != 256 || NT == 1, "one O");
};

struct Args8 {
    const int32_t *q_start, *kv_len, *page_table;
    const __half *k_scales, *v_scales;
    __half* out;
    float* lse;
    float* part_o;       // [CTA][2][rows][D]
    float2* part_ml;     // [CTA][2][rows]
    int* meta;           // [CTA][8]
    int* err;
    int B, total_q, max_q, Hq, Hkv, G, HG, n_hg, QT1, QTG;   // QT1 queries a row tile, QTG a group
    int hg_mul;          // 2^22 / HG, up
    int QQ;              // queries a quarter of the tile's rows (32 of them), or 0: rows one after the other
    int hp, n_hb;        // heads (kv heads x head groups) taken side by side, batches of them
    int P, log2P, max_pages, n_pages, box_rows, window, slot_rows;
    long long capacity;
    int max_rg;
    float scale, softcap;
};

// The query of a tile's row (row / HG, exact for rows and HG up to 143: row * HG < 2^22), and
// its packed row, query * HG + head; -1 where the tile has none.
__device__ __forceinline__ int query_of(const Args8& a, int row) {
    return a.QQ ? (row >> 5) * a.QQ + (((row & 31) * a.hg_mul) >> 22) : (row * a.hg_mul) >> 22;
}
__device__ __forceinline__ int packed_row(const Args8& a, int row) {
    if (!a.QQ) return row < a.QT1 * a.HG ? row : -1;
    return (row & 31) < a.QQ * a.HG ? (row >> 5) * a.QQ * a.HG + (row & 31) : -1;
}

// One sequence's chunk, and one of its row groups.
struct Chunk {
    int q_base, n_rows, pos0, L;   // first packed row, rows computed, position of query 0, cached keys
};
__device__ __forceinline__ Chunk load_chunk(const Args8& a, int b) {
    Chunk c;
    c.q_base = a.q_start[b];
    const int n_q = max(a.q_start[b + 1] - c.q_base, 0), len = a.kv_len[b];
    c.n_rows = min(n_q, a.max_q);
    c.pos0 = len - n_q;
    c.L = static_cast<int>(min(static_cast<long long>(max(len, 0)), a.capacity));
    return c;
}
struct Span {
    int lo, hi, jt0, tiles;   // keys some row of the group keeps lie in [lo, hi); its key tiles (at least one)
};
template <int BN>
__device__ __forceinline__ Span group_span(const Args8& a, const Chunk& c, int rg) {
    const long long first = static_cast<long long>(c.pos0) + rg * a.QTG;
    const long long last = static_cast<long long>(c.pos0) + min(rg * a.QTG + a.QTG, c.n_rows) - 1;
    Span s;
    s.hi = static_cast<int>(max(min(static_cast<long long>(c.L), last + 1), 0ll));
    s.lo = a.window > 0 ? static_cast<int>(max(0ll, first - a.window + 1)) : 0;
    if (s.lo >= s.hi) s.lo = s.hi = 0;   // no row keeps a key: one tile, all masked
    s.jt0 = s.lo / BN;
    s.tiles = max((s.hi + BN - 1) / BN - s.jt0, 1);
    return s;
}

// A CTA's run of key tiles as segments, each of one item.  One lane walks it and leaves
// the segments in shared memory for all warps (the walk's code in each role would push the
// roles' own code out of the instruction caches).
struct Seg {
    int b, rg, hb, off, n_rg;
    int head, kv, hg0;        // kv head and head group; kv head; the group's first query head of it
    int n, tiles;             // key tiles of this segment and of its item
    int lo, hi, key0;         // keys some row keeps; the segment's first key
    int q_base, n_rows, pos0;
    int two;                  // two row tiles (every key tile is used twice), or one
    long long rem;            // key tiles of the run from this segment on; 0: the end
};
static_assert(sizeof(Seg) == 80, "shared memory budget");
template <int BN>
__device__ __forceinline__ void seg_item(const Args8& a, Seg& s) {
    const Chunk c = load_chunk(a, s.b);
    const Span sp = group_span<BN>(a, c, s.rg);
    s.n_rg = (c.n_rows + a.QTG - 1) / a.QTG;
    s.tiles = sp.tiles;
    s.lo = sp.lo;
    s.hi = sp.hi;
    s.key0 = (sp.jt0 + s.off) * BN;
    s.q_base = c.q_base;
    s.n_rows = c.n_rows;
    s.pos0 = c.pos0;
    s.two = a.QTG > a.QT1 && c.n_rows - s.rg * a.QTG > a.QT1;
    s.n = static_cast<int>(min(static_cast<long long>(s.tiles - s.off), s.rem));
}
// The first segment (b, rg, hb, off and rem are set), or the next one.  Returns false
// at the end of the run.
template <int BN>
__device__ __forceinline__ void seg_step(const Args8& a, Seg& s, bool first) {
    for (;; first = false) {
        if (!first) {
            s.rem -= s.n;
            s.off = 0;
            if (s.rem > 0 && ++s.hb == a.n_hb) {
                s.hb = 0;
                if (++s.rg >= s.n_rg) {
                    s.rg = 0;
                    do {
                        if (++s.b >= a.B) s.rem = 0;   // (q_start changed under the call)
                    } while (s.rem > 0 && load_chunk(a, s.b).n_rows == 0);
                }
            }
        }
        if (s.rem <= 0) return;
        seg_item<BN>(a, s);
        s.head = s.hb * a.hp + static_cast<int>(blockIdx.x) % a.hp;
        s.kv = s.head / a.n_hg;
        s.hg0 = (s.head - s.kv * a.n_hg) * a.HG;
        if (s.kv < a.Hkv) return;   // the last batch may have fewer heads
    }
}
// The order in which a segment of n key tiles loads them, which is the order the
// MMAs first need them in: with two row tiles K0 V0 K1 V1 ..; with one, S of the next
// tile runs before PV of this one: K0 K1 V0 K2 V1 .. .
__device__ __forceinline__ int item_k(bool two, int j) { return two ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int item_v(bool two, int j, int n) { return two ? 2 * j + 1 : j == n - 1 ? 2 * n - 1 : 2 * j + 2; }
__device__ __forceinline__ bool item_of(bool two, int i, int n, int& j) {   // true: K
    if (two) {
        j = i >> 1;
        return (i & 1) == 0;
    }
    if (i == 0) {
        j = 0;
        return true;
    }
    if (i == 2 * n - 1) {
        j = n - 1;
        return false;
    }
    j = (i & 1) ? (i + 1) >> 1 : (i >> 1) - 1;
    return (i & 1) != 0;
}

// Four int8 codes to two f16 pairs: a code's byte with its sign bit flipped is code +
// 128, the low byte of the f16 number 1024 + 128 + code; fma(x, s, -1152 s) is then
// s * code exactly for s = 1, -1 or 0.
__device__ __forceinline__ void codes_to_f16(uint32_t w, __half2 s, __half2 off, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&a), s, off);
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b), s, off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

template <int D, int NT, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
prefill8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const Args8 a) {
    using C = Cfg<D, NT>;
    constexpr int BN = C::BN, NCH = C::NCH, NST = C::NST, RING = C::RING;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    volatile uint32_t* fills = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_FILLS);   // of each stage
    Seg* segs = reinterpret_cast<Seg*>(smem + C::OFF_SEG);
    Seg& walk = segs[C::SEGS];     // the walk's own state
    KeyFactors<BN>* tab = reinterpret_cast<KeyFactors<BN>*>(smem + C::OFF_TAB);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);   // [warpgroup][row]
    auto bar = [&](int i) { return sbase + C::OFF_BAR + i * 8; };
    // The bounded wait of ptx.cuh (mbar_wait) in less code (it is in all of this kernel's
    // roles, which together run close to the instruction caches' size), and suspended up to
    // 1 ms a try: 20 warps that poll slow down the ones that work.
    const uint32_t limit = static_cast<uint32_t>(
        min(*static_cast<volatile unsigned long long*>(&g_wait_limit_ns), 0xffffffffull));
    auto wait = [limit](uint32_t b, uint32_t parity, volatile int* abort_flag, int* err, int code) -> bool {
        if (mbar_try_wait_for(b, parity, 1000000)) return true;
        const uint32_t t0 = globaltimer_lo();
#pragma unroll 1
        do {
            if (mbar_try_wait_for(b, parity, 1000000)) return true;
            if (*abort_flag) return false;
        } while (globaltimer_lo() - t0 < limit);
        *abort_flag = 1;
        atomicExch(err, code);
        return false;
    };
    // The same for a whole warp, with one answer for all of its lanes, so that a warp whose loop
    // has warp-wide steps leaves it as a whole: a lane that gave up alone would never meet the
    // others there.  (A vote on the answers of separate waits instead: 300 -> 316 to 326 us for 4
    // tokens of 16 long contexts; in this form 304, and 8 chunks of 512 tokens 328 -> 319, since
    // no lanes have to be brought together after a wait.  Slower for the softmax warps: 312.)
    auto wait_warp = [limit](uint32_t b, uint32_t parity, volatile int* abort_flag, int* err, int code) -> bool {
        if (__all_sync(0xffffffffu, mbar_try_wait_for(b, parity, 1000000))) return true;
        const uint32_t t0 = globaltimer_lo();
#pragma unroll 1
        do {
            if (__all_sync(0xffffffffu, mbar_try_wait_for(b, parity, 1000000))) return true;
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
        } while (__any_sync(0xffffffffu, globaltimer_lo() - t0 < limit));
        *abort_flag = 1;
        atomicExch(err, code);
        return false;
    };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be set up meanwhile
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    // ---- this CTA's run: sum the key tiles of every (sequence, row group), then find
    // where the run starts
    {
        long long* sums = reinterpret_cast<long long*>(tab);   // before any table
        static_assert(sizeof(KeyFactors<BN>) >= 66 * 8, "scratch");
        const long long pairs = static_cast<long long>(a.B) * a.max_rg;
        const long long per = (pairs + kThreads - 1) / kThreads;
        const long long f0 = min(pairs, tid * per), f1 = min(pairs, f0 + per);
        // visits this thread's pairs in order until fn says stop
        auto visit = [&](auto fn) {
            if (f0 >= f1) return;
            int b = static_cast<int>(f0 / a.max_rg), rg = static_cast<int>(f0 - static_cast<long long>(b) * a.max_rg);
            long long left = f1 - f0;
            while (left > 0) {
                const Chunk c = load_chunk(a, b);
                const int n_rg = (c.n_rows + a.QTG - 1) / a.QTG;
                const int end = static_cast<int>(min(static_cast<long long>(n_rg), rg + left));
                for (int r = rg; r < end; ++r)
                    if (!fn(b, r, group_span<BN>(a, c, r).tiles)) return;
                left -= a.max_rg - rg;
                rg = 0;
                ++b;
            }
        };
        long long mine = 0, tiles = 0;         // weights, and key tiles alone
        visit([&](int, int, int t) {
            mine += t + C::SEG_TILES;
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
            sums[32 + warp] = incl_t;
        }
        if (tid == 0) {
            for (int i = 0; i < NST; ++i) {
                mbar_init(bar(C::B_SFULL_ST + i), 1);
                mbar_init(bar(C::B_SEMPTY_ST + i), C::NCV);
            }
            for (int i = 0; i < RING; ++i) {
                mbar_init(bar(C::B_OPFULL + i), C::NCV);
                mbar_init(bar(C::B_OPEMPTY + i), 1);
            }
            for (int i = 0; i < C::SEGS; ++i) {
                mbar_init(bar(C::B_SEG + i), 1);
                mbar_init(bar(C::B_SEGFREE + i), kThreads / 32);
            }
            for (int i = 0; i < C::NTAB; ++i) {
                mbar_init(bar(C::B_TAB + i), 1);
                mbar_init(bar(C::B_TABEMPTY + i), 1);
            }
            mbar_init(bar(C::B_QFULL), 1);
            mbar_init(bar(C::B_QEMPTY), 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(C::B_S + i), 1);
                mbar_init(bar(C::B_SFREE + i), C::NSM / C::NS);
                mbar_init(bar(C::B_P + i), C::NSM / C::NS);
                mbar_init(bar(C::B_PV + i), 1);
                mbar_init(bar(C::B_PH + i), C::NSM / C::NS);
            }
            mbar_init(bar(C::B_DONE), 1);
            mbar_init(bar(C::B_OFREE), C::NSM);
            mbar_init(bar(C::B_ML), C::NSM);
            mbar_init(bar(C::B_TEARDOWN), 1);
            *abort_flag = 0;
            for (int i = 0; i < NST; ++i) fills[i] = 0;
            fence_barrier_init();
        }
        if (warp == C::MMA_WARP) {
            tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
            tmem_relinquish();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        long long sw = lane < kThreads / 32 ? sums[lane] : 0, sw_t = lane < kThreads / 32 ? sums[32 + lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, sw, o), y = __shfl_up_sync(0xffffffffu, sw_t, o);
            if (lane >= o) {
                sw += x;
                sw_t += y;
            }
        }
        const long long total = __shfl_sync(0xffffffffu, sw, 31), total_t = __shfl_sync(0xffffffffu, sw_t, 31);
        long long before = __shfl_sync(0xffffffffu, sw, max(warp - 1, 0)), before_t = __shfl_sync(0xffffffffu, sw_t, max(warp - 1, 0));
        if (warp == 0) before = before_t = 0;
        before += incl - mine;
        before_t += incl_t - tiles;
        // as many runs as CTAs for each of the hp heads, or fewer of kMinTiles.  A run's weight is
        // more than SEG_TILES, so it has a key tile at least.
        const long long all = total * a.n_hb;
        const int rank = static_cast<int>(blockIdx.x) / a.hp;
        const long long runs =
            max(1ll, min(static_cast<long long>(gridDim.x / a.hp), all / (C::SEG_TILES + kMinTiles)));
        // where weight t lies: the thread that has it leaves the key tiles before it, and for the
        // run's start the item
        auto locate = [&](long long t, long long* pos, bool start) {
            if (before * a.n_hb > t || t >= (before + mine) * a.n_hb) return;
            long long acc = before, acc_t = before_t;
            visit([&](int b, int rg, int n) {
                const int weight = n + C::SEG_TILES;
                if ((acc + weight) * a.n_hb <= t) {
                    acc += weight;
                    acc_t += n;
                    return true;
                }
                const long long in = t - acc * a.n_hb;
                const int hb = static_cast<int>(in / weight);
                const int off = max(static_cast<int>(in - static_cast<long long>(hb) * weight) - C::SEG_TILES, 0);
                *pos = acc_t * a.n_hb + static_cast<long long>(hb) * n + off;
                if (start) {
                    walk.b = b;
                    walk.rg = rg;
                    walk.hb = hb;
                    walk.off = off;
                }
                return false;
            });
        };
        if (rank < runs) {
            const long long mine_t = all * (rank + (lane & 1)) / runs;   // the run's start and end
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                const long long t = __shfl_sync(0xffffffffu, mine_t, e);
                if (t < all) locate(t, &sums[64 + e], e == 0);
                else if (tid == 0) sums[64 + e] = total_t * a.n_hb;
                __syncwarp();
            }
        } else if (tid == 0) {
            sums[64] = sums[65] = 0;
        }
        __syncthreads();
        // (the walking warp, which is also the one that writes the tables; 0: no run)
        if (warp == C::V_WARP + 1 && lane == 0) walk.rem = sums[65] - sums[64];
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    // Segment `seg` of the run, once it is known; false at the run's end.  leave(): this warp
    // needs segment `seg` no more.
    auto enter = [&](uint32_t seg, const Seg*& w) -> bool {
        const bool known = wait(bar(C::B_SEG + seg % C::SEGS), (seg / C::SEGS) & 1, abort_flag, a.err, kErrTimeoutSlot);
        w = &segs[seg % C::SEGS];
        return known && w->rem > 0;
    };
    auto leave = [&](uint32_t seg) { mbar_arrive(bar(C::B_SEGFREE + seg % C::SEGS)); };

    // (setmaxnreg is executed by all four warps of a warpgroup)
    if (warp >= C::K_WARP) {
    regs_dec<kRegOther>();
    if (warp == C::K_WARP || warp == C::V_WARP) {
        // ------------------------------------------------------------ codes
        // One warp brings K tiles, one V tiles; lanes 0-15, lane i the box of the tile's
        // i-th page (one box inside a page that is longer than the tile).  Page ids come
        // 4 tiles ahead by asynchronous copies; lane 0 waits for the stage and posts the
        // byte count.
        if (lane < 16) {
            const unsigned gmask = 0x0000ffffu;
            const bool leader = lane == 0, mine_k = warp == C::K_WARP;
            const CUtensorMap* tm = mine_k ? &tm_k : &tm_v;
            if (leader) tma_prefetch_desc(tm);
            const int R = a.box_rows;
            const bool has_box = lane * R < BN;
            const uint32_t ids = C::OFF_IDS + (mine_k ? 1 : 2) * (C::IDS * 16 * 4) + lane * 4;
            // (A parity wait is right only for a barrier at most one phase behind.  This warp's
            // own items are at most 3 apart, and the converters free stages in item order, so
            // the one it waited for last vouches for every earlier phase of any stage.)
            static_assert(NST >= 3, "stage waits");
            uint32_t base = 0;                     // items before this segment
            int ok = 1;
            const Seg* w;
            for (uint32_t seg = 0; ok && __any_sync(gmask, enter(seg, w)); ++seg) {
                const bool two = NT == 2 && w->two;
                const int n = w->n, lo = w->lo, hi = w->hi, k0 = w->key0 + lane * R;
                const int g = w->kv;
                const int32_t* table = a.page_table + static_cast<size_t>(w->b) * a.max_pages;
                __syncwarp(gmask);
                if (leader) leave(seg);
                auto in_use = [&](int kk) { return has_box && kk >= lo - R + 1 && kk < hi; };
                auto fetch = [&](int j) {
                    const int kk = k0 + j * BN;
                    if (j < n && in_use(kk)) cp_async4(sbase + ids + (j % C::IDS) * 64, &table[kk >> a.log2P]);
                    cp_async_commit();
                };
                for (int j = 0; j < 4; ++j) fetch(j);
                for (int j = 0; j < n; ++j) {
                    const uint32_t gi = base + (mine_k ? item_k(two, j) : item_v(two, j, n)), st = gi % NST;
                    fetch(j + 4);
                    cp_async_wait<4>();
                    if (gi >= NST) {
                        if (leader)
                            ok = wait(bar(C::B_SEMPTY_ST + st), ((gi / NST) - 1) & 1, abort_flag, a.err, kErrTimeoutSlot);
                        ok = __shfl_sync(gmask, ok, 0);
                        if (!ok) break;
                    }
                    // boxes without a key of [lo, hi), and pages outside the pool, take the page
                    // coordinate n_pages, so that the copy fills zeros
                    const int kk = k0 + j * BN;
                    int page = a.n_pages, row = 0;
                    if (in_use(kk)) {
                        const int pg = *reinterpret_cast<const int*>(smem + ids + (j % C::IDS) * 64);
                        if (pg >= 0 && pg < a.n_pages) {
                            page = pg;
                            row = kk & (a.P - 1);
                        } else {
                            atomicExch(a.err, kErrChunkPage);
                        }
                    }
                    if (leader) {
                        fills[st] = gi / NST + 1;
                        mbar_arrive_expect_tx(bar(C::B_SFULL_ST + st), C::CODE_BYTES);
                    }
                    __syncwarp(gmask);
                    if (has_box)
#pragma unroll
                        for (int c = 0; c < D; c += 128)   // 128-byte columns
                            tma_load_4d(sbase + C::OFF_CODE + st * C::CODE_BYTES + c * BN + lane * R * min(D, 128), tm,
                                        bar(C::B_SFULL_ST + st), c, g, row, page);
                }
                cp_async_wait<0>();
                base += 2 * n;
            }
            cp_async_wait<0>();
            if (leader && *abort_flag)   // copies in flight land before the CTA's shared memory goes away
                for (int i = 0; i < NST; ++i)
                    if (const uint32_t f = fills[i])
                        mbar_wait_drain(bar(C::B_SFULL_ST + i), (f - 1) & 1, a.err, kErrTimeoutLoad);
        }
    } else if (warp == C::MMA_WARP) {
        // ------------------------------------------------------------ MMA issuer
        // The whole warp runs it, one lane issues.
        // Unit u of a segment is a key tile with a row tile: of two row tiles, key tile u / 2 and
        // row tile u % 2, else key tile u.  Where P lies over S, S of unit u + 2 is issued right
        // after PV of unit u (MMAs of one thread run in the order of their issue); else before
        // it, as soon as S of unit u has been read.
        constexpr uint32_t idesc_s = idesc_f16_f32(BM, BN, false);
        constexpr uint32_t idesc_o = idesc_f16_f32(BM, D, true);
        const uint64_t q_desc = smem_desc_sw128(sbase + C::OFF_Q, 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(sbase + C::OFF_OP, 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(sbase + C::OFF_OP, C::OP_CHUNK, 1024);
        const uint32_t one = elect_one();
        // testing hook: hold back the signal of the first S tile
        const bool stall = stall_first_tile();
        uint32_t base = 0, jt = 0, u0 = 0;   // items, key tiles and units before this segment
        auto wait_all = [&](int b, uint32_t parity, int code) -> bool {
            return wait_warp(bar(b), parity & 1, abort_flag, a.err, code);
        };
        bool ok = true;
        const Seg* w;
        for (uint32_t seg = 0; ok && __any_sync(0xffffffffu, enter(seg, w)); ++seg) {
            const bool two = NT == 2 && __shfl_sync(0xffffffffu, w->two, 0);
            const int n = __shfl_sync(0xffffffffu, w->n, 0), U = two ? 2 * n : n;
            if (one) leave(seg);
            ok = wait_all(C::B_QFULL, seg, kErrTimeoutLoad);
            auto issue_s = [&](int u) -> bool {
                const uint32_t gi = base + item_k(two, two ? u >> 1 : u), slot = gi % RING, gu = u0 + u, buf = gu & 1;
                if (!wait_all(C::B_OPFULL + slot, gi / RING, kErrTimeoutLoad)) return false;
                if (!C::OVER && gu >= 2 && !wait_all(C::B_SFREE + buf, (gu >> 1) - 1, kErrTimeoutSoftmax)) return false;
                tc_fence_after();
                const uint64_t kd = desc_advance(k_desc, slot * C::OP_BYTES);
                const uint64_t qd = desc_advance(q_desc, two ? (u & 1) * C::Q_TILE : 0);
#pragma unroll
                for (int c = 0; c < NCH; ++c)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_f16_ss_one(one, tmem + buf * BN, desc_advance(qd, c * (BM * 128) + kk * 32),
                                          desc_advance(kd, c * C::OP_CHUNK + kk * 32), idesc_s, (c | kk) != 0);
                if (!(stall && gu == 0)) tc_commit_one(one, bar(C::B_S + buf));
                if (!two || (u & 1)) tc_commit_one(one, bar(C::B_OPEMPTY + slot));
                if (u == U - 1) tc_commit_one(one, bar(C::B_QEMPTY));
                return true;
            };
            // (units -2 and -1 only issue S of units 0 and 1)
            for (int u = -2; ok && u < U; ++u) {
                if ((!C::OVER || u < 0) && u + 2 < U && !(ok = issue_s(u + 2))) break;
                if (u < 0) continue;
                const uint32_t gu = u0 + u, buf = gu & 1;
                const int j = two ? u >> 1 : u;
                const uint32_t gi = base + item_v(two, j, n), slot = gi % RING;
                ok = wait_all(C::OVER ? C::B_PH + buf : C::B_P + buf, gu >> 1, kErrTimeoutSoftmax) &&
                     wait_all(C::B_OPFULL + slot, gi / RING, kErrTimeoutLoad);
                // O still holds the segment before until its rows have been read
                if (ok && u == 0 && seg > 0) ok = wait_all(C::B_OFREE, seg - 1, kErrTimeoutSoftmax);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = desc_advance(v_desc, slot * C::OP_BYTES);
                const uint32_t o_tmem = tmem + C::COL_O + (C::NS == 2 ? buf * D : 0);
                // (D = 64/128: the first half's products run while the second's P are made)
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) {
                    if (C::OVER && kk == BN / 32) {
                        tc_commit_one(one, bar(C::B_PV + buf));
                        if (!(ok = wait_all(C::B_P + buf, gu >> 1, kErrTimeoutSoftmax))) break;
                        tc_fence_after();
                    }
                    tc_mma_f16_ts_one(one, o_tmem, tmem + C::COL_P + buf * C::P_STRIDE + kk * 8,
                                      desc_advance(vd, kk * 16 * 128), idesc_o, u >= C::NS || kk > 0 ? 1u : 0u);
                }
                if (!ok) break;
                if (!C::OVER) tc_commit_one(one, bar(C::B_PV + buf));
                if (!two || (u & 1)) {
                    tc_commit_one(one, bar(C::B_OPEMPTY + slot));
                    if (one) mbar_arrive(bar(C::B_TABEMPTY + (jt + j) % C::NTAB));   // its P are done
                }
                if (C::OVER && u + 2 < U && !(ok = issue_s(u + 2))) break;
            }
            if (ok) tc_commit_one(one, bar(C::B_DONE));
            base += 2 * n;
            jt += n;
            u0 += U;
        }
        tc_commit_one(one, bar(C::B_TEARDOWN));   // all MMAs retire before TMEM is released
        mbar_wait_drain(bar(C::B_TEARDOWN), 0, a.err, kErrTimeoutMma);
    } else {
        // ------------------------------------------------------------ per-key factors, Q
        // A lane takes a pair of keys (D = 64/128: two).  Its page ids come 4 tiles ahead
        // and its scales 2 tiles ahead, by asynchronous copies of its own.
        if (lane == 0) tma_prefetch_desc(&tm_q);
        const float kf = CAP ? a.scale / a.softcap : a.scale * kLog2e;
        const uint32_t ids = C::OFF_IDS, scl = C::OFF_SCALE + lane * 4;
        const int R = a.box_rows;
        uint32_t jt = 0, seg = 0, known = 0;   // key tiles before this segment; segments published
        bool ok = true;
        const Seg* w;
        for (;; ++seg) {
            // this warp also walks the run: two segments ahead of its own, as far as the
            // descriptions' ring has room
            if (lane == 0) {
                while (ok && known <= seg + 2 && (known == 0 || walk.rem > 0)) {
                    const uint32_t e = known % C::SEGS;
                    if (known >= C::SEGS)
                        ok = wait(bar(C::B_SEGFREE + e), (known / C::SEGS - 1) & 1, abort_flag, a.err, kErrTimeoutSlot);
                    if (!ok) break;
                    seg_step<BN>(a, walk, known == 0);
                    segs[e] = walk;
                    if (known == 0) {
                        int* m = a.meta + blockIdx.x * 8;
                        m[0] = walk.rem > 0 && walk.n == walk.tiles - walk.off;   // ends the item it begins in
                        m[1] = 0;                                                 // ends inside another (set below)
                    }
                    mbar_arrive(bar(C::B_SEG + e));
                    ++known;
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !__any_sync(0xffffffffu, enter(seg, w))) break;
            const int n = w->n, lo = w->lo, hi = w->hi, k0 = w->key0 + 2 * lane;
            const int g = w->kv;
            const int32_t* table = a.page_table + static_cast<size_t>(w->b) * a.max_pages;
            if (lane == 0) {
                if (seg > 0) ok = wait(bar(C::B_QEMPTY), (seg - 1) & 1, abort_flag, a.err, kErrTimeoutSlot);
                if (ok) {
                    const int nt = NT == 2 && w->two ? 2 : 1;
                    const int h0 = g * a.G + w->hg0;
                    const int q0 = w->q_base + w->rg * a.QTG;
                    mbar_arrive_expect_tx(bar(C::B_QFULL), nt * NCH * a.HG * a.QT1 * 128);
                    // a box a row tile, or a quarter of one, and 64 columns
                    const int boxes = a.QQ ? 4 : nt, queries = a.QQ ? a.QQ : a.QT1;
                    const uint32_t apart = a.QQ ? 32 * 128 : C::Q_TILE;
                    for (int t = 0; t < boxes; ++t)
#pragma unroll 1
                        for (int c = 0; c < NCH; ++c)
                            tma_load_3d(sbase + C::OFF_Q + t * apart + c * (BM * 128), &tm_q, bar(C::B_QFULL), c * 64, h0,
                                        q0 + t * queries);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // page ids: lane i < 16 that of the tile's i-th box
            auto fetch_ids = [&](int j) {
                const int kk = w->key0 + j * BN + lane * R;
                if (j < n && lane * R < BN && kk >= lo - R + 1 && kk < hi)
                    cp_async4(sbase + ids + (j % C::IDS) * 64 + lane * 4, &table[kk >> a.log2P]);
            };
            auto fetch_scales = [&](int j) {
                __syncwarp();             // ids that other lanes brought
#pragma unroll
                for (int x = 0; x < BN / 64; ++x) {
                    const int kk = k0 + j * BN + x * 64;
                    if (!(j < n && kk + 1 >= lo && kk < hi)) continue;
                    const int pg = *reinterpret_cast<const int*>(smem + ids + (j % C::IDS) * 64 + (2 * lane + x * 64) / R * 4);
                    const uint32_t dst = scl + (j % C::SCALES) * C::SCALE_BYTES + x * 128;
                    if (pg >= 0 && pg < a.n_pages) {
                        const size_t at = (static_cast<size_t>(pg) * a.Hkv + g) * a.P + (kk & (a.P - 1));
                        cp_async4(sbase + dst, a.k_scales + at);
                        cp_async4(sbase + dst + BN * 2, a.v_scales + at);
                    } else {   // its codes are zeros too
                        *reinterpret_cast<uint32_t*>(smem + dst) = 0u;
                        *reinterpret_cast<uint32_t*>(smem + dst + BN * 2) = 0u;
                    }
                }
            };
            for (int j = 0; j < 4; ++j) fetch_ids(j);
            cp_async_commit();
            cp_async_wait<0>();
            fetch_scales(0);
            cp_async_commit();
            fetch_scales(1);
            cp_async_commit();
            for (int j = 0; j < n; ++j) {
                cp_async_wait<1>();       // scales of tile j, ids up to tile j + 2
                fetch_scales(j + 2);
                fetch_ids(j + 4);
                cp_async_commit();
                const uint32_t tb = (jt + j) % C::NTAB;
                if (jt + j >= C::NTAB)
                    ok = wait(bar(C::B_TABEMPTY + tb), ((jt + j) / C::NTAB - 1) & 1, abort_flag, a.err, kErrTimeoutSoftmax);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                KeyFactors<BN>& t = tab[tb];
                const uint8_t* sc = smem + scl + (j % C::SCALES) * C::SCALE_BYTES;
#pragma unroll 1
                for (int x = 0; x < BN / 64; ++x) {
                    const int pr = x * 32 + lane;
                    const float2 ks2 = __half22float2(*reinterpret_cast<const __half2*>(sc + x * 128));
                    const float2 vs2 = __half22float2(*reinterpret_cast<const __half2*>(sc + x * 128 + BN * 2));
                    float f[2], lv[2], iv[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = k0 + j * BN + x * 64 + e;
                        const float ks = e ? ks2.y : ks2.x, vs = e ? vs2.y : vs2.x;
                        const bool in = key >= lo && key < hi;
                        const bool fin = isfinite(ks) && isfinite(vs);
                        // a value scale of 0 counts as the smallest f16 with codes of 0; a scale
                        // that is not finite makes the logit NaN, which only rows that keep the
                        // key take; keys outside [lo, hi) get factors that cannot spoil anything
                        const float av = in && fin ? fmaxf(fabsf(vs), 0x1p-24f) : 1.f;
                        f[e] = !in ? 0.f : fin ? ks * kf : __int_as_float(0x7fc00000);
                        lv[e] = log2f(av);
                        iv[e] = 1.f / av;
                        t.sign[2 * pr + e] = !in || !fin || vs == 0.f ? 0u : vs > 0.f ? 0x3c003c00u : 0xbc00bc00u;
                    }
                    t.a[pr] = make_float4(f[0], f[1], lv[0], lv[1]);
                    t.b[pr] = make_float2(iv[0], iv[1]);
                }
                warp_arrive(bar(C::B_TAB + tb), lane);
            }
            cp_async_wait<0>();
            jt += n;
            warp_arrive(bar(C::B_SEGFREE + seg % C::SEGS), lane);
        }
        cp_async_wait<0>();
        if (lane == 0 && *abort_flag && seg > 0) mbar_wait_drain(bar(C::B_QFULL), (seg - 1) & 1, a.err, kErrTimeoutLoad);
    }
    } else if (warp >= C::NSM) {
        // ------------------------------------------------------------ converters
        regs_dec<kRegConvert>();
        // A thread takes pieces of 16 codes: one 16-byte load, two 16-byte stores of f16.
        // Staged rows of 128 bytes are swizzled by their TMA copy (16-byte unit u of row r at
        // u ^ (r & 7)), operand rows by what the MMA reads; 4 lanes take a row's 64 bytes, and
        // the 8 lanes of an access phase the rows r and r ^ 5, whose units fall into distinct
        // banks in the load and in both stores (64-byte rows: r and r + 1, not swizzled).
        constexpr int ROWS = BN / C::NCV;             // of a warp
        constexpr int GROUPS = ROWS / 8;              // 8 rows, a quad of lanes each
        constexpr int HALVES = D / 64;                // 64-byte pieces of a row
        const int cw = warp - C::NSM, quad = lane >> 2;
        const int r8 = D == 64 ? quad : (quad & 1) ? (quad >> 1) ^ 5 : quad >> 1;   // row of 8
        const int row0 = cw * ROWS + r8;
        const uint32_t src0 = D == 64 ? row0 * 64 + (lane & 3) * 16 : row0 * 128 + (((lane & 3) ^ r8) << 4);
        const uint32_t dst0 = row0 * 128 + (((lane & 3) * 2 ^ r8) << 4);     // and dst0 ^ 16
        uint32_t st = 0, st_par = 0, slot = 0, slot_par = 1, jt = 0;   // rings, and key tiles before this segment
        bool ok = true;
        const Seg* w;
        for (uint32_t seg = 0; ok && __any_sync(0xffffffffu, enter(seg, w)); ++seg) {
            const bool two = NT == 2 && w->two;
            const int n = w->n;
            warp_arrive(bar(C::B_SEGFREE + seg % C::SEGS), lane);
            for (int i = 0; i < 2 * n; ++i) {
                int j;
                const bool is_k = item_of(two, i, n, j);
                const KeyFactors<BN>& t = tab[(jt + j) % C::NTAB];
                ok = wait_warp(bar(C::B_SFULL_ST + st), st_par, abort_flag, a.err, kErrTimeoutLoad);
                if (ok && !is_k)   // the signs of this tile's value scales
                    ok = wait_warp(bar(C::B_TAB + (jt + j) % C::NTAB), ((jt + j) / C::NTAB) & 1, abort_flag, a.err,
                              kErrTimeoutLoad);
                if (!ok) break;
                const uint8_t* src = smem + C::OFF_CODE + st * C::CODE_BYTES;
                uint8_t* dst = smem + C::OFF_OP + slot * C::OP_BYTES + dst0;
                uint4 v[GROUPS][HALVES];
                uint32_t sg[GROUPS];
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
                        v[g][h] = *reinterpret_cast<const uint4*>(
                            src + ((src0 + g * 8 * (D == 64 ? 64 : 128)) ^ ((h & 1) * 64)) + (h >> 1) * (BN * 128));
                    sg[g] = is_k ? 0x3c003c00u : t.sign[row0 + g * 8];
                }
                // (a fresh barrier's "phase before" counts as complete: the first RING waits pass)
                ok = wait_warp(bar(C::B_OPEMPTY + slot), slot_par, abort_flag, a.err, kErrTimeoutMma);
                if (!ok) break;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    const __half2 s = *reinterpret_cast<const __half2*>(&sg[g]);
                    const __half2 off = __hmul2(s, __float2half2_rn(-1152.f));
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        uint4 x, y;
                        codes_to_f16(v[g][h].x, s, off, x.x, x.y);
                        codes_to_f16(v[g][h].y, s, off, x.z, x.w);
                        codes_to_f16(v[g][h].z, s, off, y.x, y.y);
                        codes_to_f16(v[g][h].w, s, off, y.z, y.w);
                        uint8_t* d = dst + g * 1024 + h * C::OP_CHUNK;
                        *reinterpret_cast<uint4*>(d) = x;
                        *reinterpret_cast<uint4*>(smem + ((d - smem) ^ 16)) = y;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::B_OPFULL + slot));
                    mbar_arrive(bar(C::B_SEMPTY_ST + st));
                }
                if (++st == NST) st = 0, st_par ^= 1;
                if (++slot == RING) slot = 0, slot_par ^= 1;
            }
            jt += n;
        }
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<kRegSoftmax>();
        // Each warpgroup takes the units of its stream, a warp 32 rows (one stream: both take
        // every unit, a warp 16 rows), 64 keys a time.  Of every 16-row half a thread holds
        // rows lane / 4 and lane / 4 + 8, and of every 8 columns the pair 2 (lane % 4), so that
        // a 16- and an 8-byte load of per-key factors serve 2 keys of 4 rows; a row a thread
        // would take 4 times the loads.  Where row groups have one row tile the halves go one
        // after the other, so that the second one, often without rows, can be left out.
        constexpr int HL = C::NS;                  // 16-row halves of a warp
        constexpr int HN = NT == 2 ? 2 : 1;        // taken at once
        static_assert(HN <= HL, "halves");
        const int ws = warp >> 2;
        const int quarter = warp & 3;
        const int row0 = quarter * 32 + (HL == 1 ? ws * 16 : 0);   // the warp's first row
        const uint32_t lanes = tmem + (static_cast<uint32_t>(row0) << 16);
        const float cap_log2 = a.softcap * kLog2e;
        const int W = a.window > 0 ? min(a.window, 0x3fffffff) : 0;
        uint32_t u0 = 0, jt = 0, seg = 0;
        bool ok = true;
        const Seg* wp;
        for (; ok && __any_sync(0xffffffffu, enter(seg, wp)); ++seg) {
            const Seg& w = *wp;
            const bool two = NT == 2 && w.two;
            const int n = w.n, U = two ? 2 * n : n, k0 = w.key0, hi = w.hi;
            const int first_u = C::NS == 1 ? 0 : static_cast<int>((ws ^ u0) & 1);
            const int rt = two ? first_u : 0;      // this warpgroup's row tile
            const int q0 = w.rg * a.QTG + rt * a.QT1;
            // rows row0 + 8 x + lane / 4, at positions that ascend
            int pos[2 * HL];
            float m[2 * HL], l[2 * HL];
#pragma unroll
            for (int x = 0; x < 2 * HL; ++x) {
                pos[x] = w.pos0 + q0 + query_of(a, row0 + x * 8 + (lane >> 2));
                m[x] = -INFINITY;
                l[x] = 0.f;
            }
            // keys in [all_lo, all_hi) are kept by each of the warp's rows
            const int all_hi = min(hi, w.pos0 + q0 + query_of(a, row0) + 1);
            const int all_lo = W ? w.pos0 + q0 + query_of(a, row0 + 16 * HL - 1) - W + 1 : 0;
            // without a query among its rows a warp only keeps step (its rows of P are what TMEM
            // holds: rows of the products do not mix)
            const bool idle = w.n_rows - q0 <= query_of(a, row0);
            const int nh = HL == HN || a.QQ ? 1 : w.n_rows - q0 <= query_of(a, row0 + 16) ? 1 : 2;   // halves in turn
            for (int u = first_u; ok && u < U; u += C::NS) {
                const int j = two ? u >> 1 : u;
                const uint32_t gu = u0 + u, buf = gu & 1, tb = (jt + j) % C::NTAB;
                ok = wait(bar(C::B_TAB + tb), ((jt + j) / C::NTAB) & 1, abort_flag, a.err, kErrTimeoutLoad) &&
                     wait(bar(C::B_S + buf), (gu >> 1) & 1, abort_flag, a.err, kErrTimeoutMma);
                ok = __all_sync(0xffffffffu, ok);   // tcgen05 loads and stores need whole warps
                if (!ok) break;
                tc_fence_after();
                // PV of unit g is done (D = 64/128: that of its first 64 keys): its P may be
                // overwritten, its O rescaled.  Where P lies over S, S of unit g + 2 came after all of it.
                auto pv_done = [&](uint32_t g) -> bool {
                    const bool done = wait(bar(C::B_PV + (g & 1)), (g >> 1) & 1, abort_flag, a.err, kErrTimeoutMma);
                    tc_fence_after();
                    return __all_sync(0xffffffffu, done);
                };
                if (idle) warp_arrive(bar((C::OVER ? C::B_PH : C::B_SFREE) + buf), lane);
                if (!C::OVER && gu >= 2 && !(ok = pv_done(gu - 2))) break;
#pragma unroll 1
                for (int it = 0; it < BN / 64 * nh && !idle; ++it) {   // 64 keys, a half or both
                    const int c = nh == 2 ? it >> 1 : it;
                    const uint32_t half = nh == 2 ? static_cast<uint32_t>((it & 1) * 16) << 16 : 0u;
                    const float4* fa = tab[tb].a + c * 32 + (lane & 3);
                    const float2* fb = tab[tb].b + c * 32 + (lane & 3);
                    const int key0 = k0 + j * BN + c * 64;
                    const uint32_t p_addr = lanes + half + C::COL_P + buf * C::P_STRIDE;
                    float2 y[2 * HN][8];           // [row][8-column group]
                    {
                        uint32_t r[HN][32];
#pragma unroll
                        for (int hf = 0; hf < HN; ++hf)
                            tc_ld_16x256b_x8(lanes + half + buf * BN + c * 64 + (static_cast<uint32_t>(hf * 16) << 16), r[hf]);
                        tc_wait_ld();
#pragma unroll
                        for (int x = 0; x < 2 * HN; ++x)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                y[x][i] = make_float2(__uint_as_float(r[x / 2][4 * i + 2 * (x & 1)]),
                                                      __uint_as_float(r[x / 2][4 * i + 2 * (x & 1) + 1]));
                    }
                    if (!C::OVER) {
                        tc_fence_before();
                        warp_arrive(bar(C::B_SFREE + buf), lane);
                    }
                    if constexpr (CAP) {
                        // c tanh(x) in log2 units: an odd polynomial for |x| <= 1/4 (the dropped
                        // x^9 term is below 8.4e-8), else the exponential form for the whole warp
                        const float k1 = cap_log2 * (-1.0f / 3.0f), k2 = cap_log2 * (2.0f / 15.0f),
                                    k3 = cap_log2 * (-17.0f / 315.0f);
                        float ax = 0.f;
                        float2 lv[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = fa[4 * i];
                            lv[i] = make_float2(f.z, f.w);
#pragma unroll
                            for (int x = 0; x < 2 * HN; ++x) {
                                y[x][i] = fmul2(y[x][i], make_float2(f.x, f.y));
                                ax = max3(ax, fabsf(y[x][i].x), fabsf(y[x][i].y));
                            }
                        }
                        if (__all_sync(0xffffffffu, ax <= 0.25f)) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
#pragma unroll
                                for (int x = 0; x < 2 * HN; ++x) {
                                    const float2 v = y[x][i], z = fmul2(v, v);
                                    float2 q = ffma2(z, make_float2(k3, k3), make_float2(k2, k2));
                                    q = ffma2(q, z, make_float2(k1, k1));
                                    q = ffma2(q, z, make_float2(cap_log2, cap_log2));
                                    y[x][i] = ffma2(v, q, lv[i]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
#pragma unroll
                                for (int x = 0; x < 2 * HN; ++x)
                                    y[x][i] = make_float2(fmaf(cap_log2, tanh_abs_accurate(y[x][i].x), lv[i].x),
                                                          fmaf(cap_log2, tanh_abs_accurate(y[x][i].y), lv[i].y));
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = fa[4 * i];
#pragma unroll
                            for (int x = 0; x < 2 * HN; ++x)
                                y[x][i] = ffma2(y[x][i], make_float2(f.x, f.y), make_float2(f.z, f.w));
                        }
                    }
                    if (key0 < all_lo || key0 + 64 > all_hi) {   // a row keeps the keys [klo, khi)
#pragma unroll
                        for (int x = 0; x < 2 * HN; ++x) {
                            const int khi = min(hi, pos[x] + 1), klo = W ? max(0, pos[x] - W + 1) : 0;
                            const int from = klo - key0 - 2 * (lane & 3);
                            const unsigned count = max(khi - klo, 0);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (static_cast<unsigned>(8 * i - from) >= count) y[x][i].x = -INFINITY;
                                if (static_cast<unsigned>(8 * i + 1 - from) >= count) y[x][i].y = -INFINITY;
                            }
                        }
                    }
                    // P = f16(2^(y - m)), sums of it / vs.  A row keeps its m while no y
                    // exceeds it by more than the threshold (P stays at most 2^8), so its 4
                    // lanes need not agree on every tile's maximum
                    float mx[2 * HN];
                    bool over = false;
#pragma unroll
                    for (int x = 0; x < 2 * HN; ++x) {
                        float q[2] = {fmaxf(y[x][0].x, y[x][0].y), fmaxf(y[x][1].x, y[x][1].y)};
#pragma unroll
                        for (int i = 2; i < 8; ++i) q[i & 1] = max3(q[i & 1], y[x][i].x, y[x][i].y);
                        mx[x] = fmaxf(q[0], q[1]);
                        over = over || mx[x] > m[x] + kRescaleThreshold;   // m = -inf: any kept key
                    }
                    if (__any_sync(0xffffffffu, over)) {
                        float alpha[2 * HN];
#pragma unroll
                        for (int x = 0; x < 2 * HN; ++x) {
                            float v = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                            alpha[x] = 1.f;
                            if (v > m[x] + kRescaleThreshold) {
                                alpha[x] = m[x] == -INFINITY ? 0.f : ex2_approx(m[x] - v);
                                l[x] *= alpha[x];
                                m[x] = v;
                            }
                        }
                        // what O holds was weighted with the old maxima: one stream: after PV of the
                        // unit before; two: after PV of the tile's first 64 keys, for the second
                        if (u >= C::NS || c > 0) {
                            if ((C::NS == 1 || c > 0) && !(ok = pv_done(C::NS == 1 ? gu - 1 : gu))) break;
                            const uint32_t o_addr = lanes + half + C::COL_O + (C::NS == 2 ? buf * D : 0);
#pragma unroll 1
                            for (int e = 0; e < D; e += 32) {
#pragma unroll
                                for (int hf = 0; hf < HN; ++hf) {
                                    const uint32_t at = o_addr + e + (static_cast<uint32_t>(hf * 16) << 16);
                                    uint32_t r[16];
                                    tc_ld_16x256b_x4(at, r);
                                    tc_wait_ld();
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha[2 * hf + ((i >> 1) & 1)]);
                                    tc_st_16x256b_x4(at, r);
                                }
                            }
                        }
                    }
                    float2 nm[2 * HN];
#pragma unroll
                    for (int x = 0; x < 2 * HN; ++x) {
                        const float mu = m[x] == -INFINITY ? 0.f : -m[x];
                        nm[x] = make_float2(mu, mu);
                    }
                    // (32 keys a time: 16 columns of P)
#pragma unroll
                    for (int i0 = 0; i0 < 8; i0 += 4) {
                        uint32_t packed[HN][8];
#pragma unroll
                        for (int i = i0; i < i0 + 4; ++i) {
#pragma unroll
                            for (int x = 0; x < 2 * HN; ++x) {
                                const float2 d = fadd2(y[x][i], nm[x]);
                                y[x][i] = make_float2(ex2_approx(d.x), ex2_approx(d.y));
                                const __half2 hp = __floats2half2_rn(y[x][i].x, y[x][i].y);
                                packed[x / 2][2 * (i - i0) + (x & 1)] = *reinterpret_cast<const uint32_t*>(&hp);
                            }
                        }
#pragma unroll
                        for (int hf = 0; hf < HN; ++hf)
                            tc_st_16x128b_x4(p_addr + c * 32 + i0 * 4 + (static_cast<uint32_t>(hf * 16) << 16), packed[hf]);
                    }
                    // P goes off before the sums are taken; their factors are read first, since
                    // the tile's last P frees its table
                    float2 iv[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) iv[i] = fb[4 * i];
                    const bool last = c == BN / 64 - 1;
                    if ((C::OVER || last) && (nh == 1 || (it & 1))) {
                        tc_wait_st();
                        tc_fence_before();
                        warp_arrive(bar((last ? C::B_P : C::B_PH) + buf), lane);
                    }
#pragma unroll
                    for (int x = 0; x < 2 * HN; ++x) {
                        float2 ls = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) ls = ffma2(round11(y[x][i]), iv[i], ls);
                        l[x] += ls.x + ls.y;
                    }
                    if constexpr (HL > HN) {
                        if (nh == 2) {   // the other half's state to the front
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float fm = m[x], fl = l[x];
                                const int ip = pos[x];
                                m[x] = m[x + 2];
                                l[x] = l[x + 2];
                                pos[x] = pos[x + 2];
                                m[x + 2] = fm;
                                l[x + 2] = fl;
                                pos[x + 2] = ip;
                            }
                        }
                    }
                }
                if (!ok) break;
                if (idle) warp_arrive(bar(C::B_P + buf), lane);
            }
            // -------------------------------------------------------- the segment's rows
            if (ok) ok = wait(bar(C::B_DONE), seg & 1, abort_flag, a.err, kErrTimeoutMma);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < 2 * HL; ++x) {
                float v = l[x];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if ((lane & 3) == 0) ml[(HL == 2 ? ws * BM : 0) + row0 + x * 8 + (lane >> 2)] = make_float2(m[x], v);
            }
            warp_arrive(bar(C::B_ML), lane);
            ok = __all_sync(0xffffffffu, wait(bar(C::B_ML), seg & 1, abort_flag, a.err, kErrTimeoutSoftmax));
            if (!ok) break;
            {
                // A warp writes its quarter's 32 rows: of two row tiles each warpgroup one, of a
                // single one half of the columns, where the two streams are joined.
                const bool join = C::NS == 2 && !two && n > 1, whole = w.off == 0 && n == w.tiles;
                const int cols = two ? D : D / 2, c0 = two ? 0 : ws * (D / 2);
                // stream of this row tile, or of the segment's first unit; the other one
                const int s0 = C::NS == 1 ? 0 : two ? ws : static_cast<int>(u0 & 1);
                const uint32_t o_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + C::COL_O + c0;
                const uint32_t o0 = o_tmem + s0 * D, o1 = o_tmem + (C::NS == 2 ? (s0 ^ 1) * D : 0);
                const int slot = blockIdx.x * 2 + (w.off > 0 ? 0 : 1);
                float w0[4], w1[4];
                char* dst[4];                      // of this lane's part of each row; null: not a row of the call
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = quarter * 32 + x * 8 + (lane >> 2);
                    const float2 a0 = ml[s0 * BM + row];
                    float mx = a0.x, sum = a0.y;
                    w0[x] = 1.f;
                    w1[x] = 0.f;
                    if (join) {
                        const float2 a1 = ml[(s0 ^ 1) * BM + row];
                        mx = fmaxf(a0.x, a1.x);
                        w0[x] = a0.x == -INFINITY ? 0.f : ex2_approx(a0.x - mx);
                        w1[x] = a1.x == -INFINITY ? 0.f : ex2_approx(a1.x - mx);
                        sum = w0[x] * a0.y + w1[x] * a1.y;
                    }
                    const int pr = packed_row(a, row), qr = query_of(a, row), qi = q0 + qr, gh = w.hg0 + pr - qr * a.HG;
                    const int orow = w.q_base + qi;
                    const bool live = pr >= 0 && qi < w.n_rows && gh < a.G && orow >= 0 && orow < a.total_q;
                    const size_t at = static_cast<size_t>(orow) * a.Hq + w.kv * a.G + gh;
                    const size_t part = static_cast<size_t>(slot) * a.slot_rows + rt * a.QT1 * a.HG + pr;
                    if (whole) {
                        // a sum of 0 is a row without keys (0, -inf); NaN stays NaN
                        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
                        w0[x] *= inv;
                        w1[x] *= inv;
                    }
                    dst[x] = !live ? nullptr
                             : whole ? reinterpret_cast<char*>(a.out + at * D + c0 + 8 * (lane & 3))
                                     : reinterpret_cast<char*>(a.part_o + part * D + c0 + 2 * (lane & 3));
                    if (live && c0 == 0 && (lane & 3) == 0) {
                        if (!whole) a.part_ml[part] = make_float2(mx, sum);
                        else if (a.lse)
                            a.lse[at] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.6931471805599453f;
                    }
                }
#pragma unroll 1
                for (int c = 0; c < cols; c += 32) {
                    __syncwarp();
                    float o[2][16];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t r[16];
                        tc_ld_16x256b_x4(o0 + c + (static_cast<uint32_t>(hf * 16) << 16), r);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[hf][e] = __uint_as_float(r[e]) * w0[2 * hf + ((e >> 1) & 1)];
                        if (join) {
                            tc_ld_16x256b_x4(o1 + c + (static_cast<uint32_t>(hf * 16) << 16), r);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[hf][e] = fmaf(__uint_as_float(r[e]), w1[2 * hf + ((e >> 1) & 1)], o[hf][e]);
                        }
                    }
                    if (whole) {
                        // the 4 lanes of a row hold 2 of every 8 columns: after a 4 x 4 transpose a
                        // lane has 8 in a row, and the row's store is 64 bytes
                        const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t v[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const __half2 h2 = __floats2half2_rn(o[x / 2][4 * i + 2 * (x & 1)],
                                                                     o[x / 2][4 * i + 2 * (x & 1) + 1]);
                                v[i] = *reinterpret_cast<const uint32_t*>(&h2);
                            }
#pragma unroll
                            for (int i = 0; i < 4; i += 2) {
                                const uint32_t g = __shfl_xor_sync(0xffffffffu, b0 ? v[i] : v[i + 1], 1);
                                if (b0) v[i] = g;
                                else v[i + 1] = g;
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t g = __shfl_xor_sync(0xffffffffu, b1 ? v[i] : v[i + 2], 2);
                                if (b1) v[i] = g;
                                else v[i + 2] = g;
                            }
                            if (dst[x]) *reinterpret_cast<uint4*>(dst[x] + c * 2) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (dst[x]) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    *reinterpret_cast<float2*>(dst[x] + (c + 8 * i) * 4) =
                                        make_float2(o[x / 2][4 * i + 2 * (x & 1)], o[x / 2][4 * i + 2 * (x & 1) + 1]);
                            }
                    }
                }
                if (tid == 0 && w.off == 0 && !whole) {
                    int* meta = a.meta + blockIdx.x * 8;
                    meta[1] = 1;
                    meta[2] = w.b;
                    meta[3] = w.rg;
                    meta[4] = w.head;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(C::B_OFREE));
                leave(seg);
            }
            u0 += U;
            jt += n;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Joins the partial rows of the items that run over a CTA boundary: block (c, y) takes
// the item that CTA c leaves unfinished, and of its rows those of chunk y, a warp a row.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill8_join_kernel(const Args8 a, int n_ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // for the whole of prefill8_kernel
    const int* meta = a.meta + blockIdx.x * 8;
    if (!meta[1]) return;
    const int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Chunk c = load_chunk(a, meta[2]);
    const int rg = meta[3], head = meta[4];
    const int per = a.QT1 * a.HG;
    const int qi = rg * a.QTG + (row / per) * a.QT1 + (row % per) / a.HG;
    const int gh = (head % a.n_hg) * a.HG + (row % per) % a.HG, orow = c.q_base + qi;
    if (qi >= c.n_rows || qi >= (rg + 1) * a.QTG || gh >= a.G || orow < 0 || orow >= a.total_q) return;
    // the parts: the end of CTA c's run, whole runs of the same head, the beginning of the last
    float mx = a.part_ml[(static_cast<size_t>(blockIdx.x) * 2 + 1) * a.slot_rows + row].x;
    int last = blockIdx.x;
    while (last + a.hp < n_ctas) {
        last += a.hp;
        mx = fmaxf(mx, a.part_ml[static_cast<size_t>(last) * 2 * a.slot_rows + row].x);
        if (a.meta[last * 8]) break;
    }
    float o[D / 32], sum = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
    for (int i = blockIdx.x; i <= last; i += a.hp) {
        const size_t at = (static_cast<size_t>(i) * 2 + (i == blockIdx.x ? 1 : 0)) * a.slot_rows + row;
        const float2 x = a.part_ml[at];
        const float w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - mx);
        sum = fmaf(w, x.y, sum);
        const float* src = a.part_o + at * D + lane * (D / 32);
#pragma unroll
        for (int e = 0; e < D / 32; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(src + e);
            o[e] = fmaf(w, v.x, o[e]);
            o[e + 1] = fmaf(w, v.y, o[e + 1]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    const size_t at = static_cast<size_t>(orow) * a.Hq + (head / a.n_hg) * a.G + gh;
    __half2* dst = reinterpret_cast<__half2*>(a.out + at * D + lane * (D / 32));
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) dst[e / 2] = __floats2half2_rn(o[e] * inv, o[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * 0.6931471805599453f;
}

// Row packing and the workspace: partial rows, their statistics, a description a CTA.
struct Plan {
    int G, HG, n_hg, QT1, NT, QTG, QQ, slot_rows;
    size_t off_ml, off_meta, bytes;
};
Plan make_plan(int max_q, int Hq, int Hkv, int D) {
    Plan p;
    p.G = Hq / Hkv;
    p.HG = p.G < BM ? p.G : BM;
    p.n_hg = (p.G + p.HG - 1) / p.HG;
    p.QT1 = BM / p.HG;
    p.NT = D <= 128 && max_q > p.QT1 ? 2 : 1;   // D = 256: one O fills TMEM
    // A few queries fill the 16-row halves of the tile's quarters first, so that a softmax warp
    // has one of them and not two in turn (1 to 8 drafts of 32 sequences, up to 32 rows: 112 us
    // one after the other, 96 by quarters)
    const int half = 16 / p.HG;   // queries
    p.QQ = D <= 128 && max_q > half && max_q <= 4 * half ? half : 0;
    if (p.QQ) p.QT1 = 4 * p.QQ;
    p.QTG = p.NT * p.QT1;
    p.slot_rows = (max_q < p.QTG ? max_q : p.QTG) * p.HG;
    const size_t rows = static_cast<size_t>(kMaxCtas) * 2 * p.slot_rows;
    p.off_ml = (rows * D * 4 + 255) / 256 * 256;
    p.off_meta = (p.off_ml + rows * 8 + 255) / 256 * 256;
    p.bytes = p.off_meta + kMaxCtas * 32;
    return p;
}

template <int D, int NT, bool CAP>
attn_status launch(const Prefill8Launch& L, const Plan& p) {
    using C = Cfg<D, NT>;
    CUtensorMap tq, tk, tv;
    Args8 a;
    a.box_rows = L.page_size < C::BN ? L.page_size : C::BN;
    attn_status st;
    {
        // q [total_q, Hq, D]: boxes of HG heads of QT1 queries, packed rows in row order
        const uint64_t dims[3] = {(uint64_t)D, (uint64_t)L.Hq, (uint64_t)L.total_q};
        const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)D * 2 * L.Hq};
        const uint32_t box[3] = {64u, (uint32_t)p.HG, (uint32_t)(p.QQ ? p.QQ : p.QT1)};
        if ((st = encode_tmap_sw128(&tq, L.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, dims, strides, box)) != ATTN_OK)
            return st;
    }
    {
        const uint64_t dims[4] = {(uint64_t)D, (uint64_t)L.Hkv, (uint64_t)L.page_size, (uint64_t)L.n_pages};
        const uint64_t strides[3] = {(uint64_t)D, (uint64_t)D * L.Hkv, (uint64_t)D * L.Hkv * L.page_size};
        const uint32_t box[4] = {(uint32_t)(D < 128 ? D : 128), 1u, (uint32_t)a.box_rows, 1u};
        auto encode = D == 64 ? encode_tmap_plain : encode_tmap_sw128;
        if ((st = encode(&tk, L.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, dims, strides, box)) != ATTN_OK) return st;
        if ((st = encode(&tv, L.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, dims, strides, box)) != ATTN_OK) return st;
    }
    auto kernel = prefill8_kernel<D, NT, CAP>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC) != cudaSuccess)
            return set_error(ATTN_ECUDA, "cudaFuncSetAttribute(prefill int8 smem) failed");
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    uint8_t* ws = static_cast<uint8_t*>(L.workspace);
    a.q_start = L.q_start;
    a.kv_len = L.kv_len;
    a.page_table = L.page_table;
    a.k_scales = static_cast<const __half*>(L.k_scales);
    a.v_scales = static_cast<const __half*>(L.v_scales);
    a.out = static_cast<__half*>(L.out);
    a.lse = L.lse;
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + p.off_ml);
    a.meta = reinterpret_cast<int*>(ws + p.off_meta);
    a.err = L.err_word;
    a.B = L.B;
    a.total_q = L.total_q;
    a.max_q = L.max_q;
    a.Hq = L.Hq;
    a.Hkv = L.Hkv;
    a.G = p.G;
    a.HG = p.HG;
    a.n_hg = p.n_hg;
    a.hg_mul = (1 << 22) / p.HG + 1;
    a.QQ = p.QQ;
    a.QT1 = p.QT1;
    a.QTG = p.QTG;
    a.P = L.page_size;
    a.log2P = 0;
    while ((1 << a.log2P) < L.page_size) ++a.log2P;
    a.max_pages = L.max_pages;
    a.n_pages = L.n_pages;
    a.window = L.window;
    a.slot_rows = p.slot_rows;
    const long long cap = static_cast<long long>(L.max_pages) * L.page_size;
    a.capacity = cap < 0x7ffff000ll ? cap : 0x7ffff000ll;
    a.max_rg = (L.max_q - 1) / p.QTG + 1;
    a.scale = L.scale;
    a.softcap = L.softcap;
    // The CTAs of one run take its hp heads side by side, so that they read neighbouring
    // rows of the same pages at the same time.  hp: the count that leaves the fewest CTAs
    // without work (152 CTAs: 8 heads as 19 x 8, 16 as the same in 2 batches, 100 in 2 batches as
    // 3 x 50; 7 one after the other, since 21 x 7 would leave 5 CTAs idle)
    const int sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    const int heads = L.Hkv * p.n_hg;
    double best = 0.;
    const int nb0 = (heads + sms - 1) / sms;
    for (int nb = nb0; nb <= heads && nb < nb0 + 32; ++nb) {
        const int hp = (heads + nb - 1) / nb;
        const double use = static_cast<double>(sms / hp) * hp / sms * heads / (static_cast<double>(hp) * nb);
        if (use > best * 1.02) {
            best = use;
            a.hp = hp;
            a.n_hb = nb;
        }
    }
    const int grid = sms / a.hp * a.hp;
    const dim3 join(grid, (p.slot_rows + kJoinWarps - 1) / kJoinWarps);
    if (trace_enabled())
        trace("prefill8_kernel<D=%d,row_tiles=%d,cap=%d> grid=%d block=%d smem=%u key_tile=%d stages=%d heads_per_row_tile=%d heads_side_by_side=%d "
              "queries_per_group=%d B=%d total_q=%d Hq=%d Hkv=%d page=%d window=%d, then prefill8_join_kernel grid=(%u,%u)",
              D, NT, (int)CAP, grid, kThreads, C::SMEM_ALLOC, C::BN, C::NST, p.HG, a.hp, p.QTG, L.B, L.total_q, L.Hq, L.Hkv,
              L.page_size, L.window, join.x, join.y);
    kernel<<<grid, kThreads, C::SMEM_ALLOC, L.stream>>>(tq, tk, tv, a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        // set up while prefill8_kernel runs: the join waits for its end itself
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = join;
        cfg.blockDim = dim3(kJoinWarps * 32);
        cfg.stream = L.stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, prefill8_join_kernel<D>, a, grid);
    }
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "prefill (int8) launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

template <int D, int NT>
attn_status launch_cap(const Prefill8Launch& L, const Plan& p) {
    return L.softcap > 0.f ? launch<D, NT, true>(L, p) : launch<D, NT, false>(L, p);
}

}  // namespace

size_t prefill8_workspace(int max_q, int Hq, int Hkv, int D) { return make_plan(max_q, Hq, Hkv, D).bytes; }

attn_status launch_prefill8(const Prefill8Launch& L) {
    const Plan p = make_plan(L.max_q, L.Hq, L.Hkv, L.D);
    switch (L.D) {
        case 64: return p.NT == 2 ? launch_cap<64, 2>(L, p) : launch_cap<64, 1>(L, p);
        case 128: return p.NT == 2 ? launch_cap<128, 2>(L, p) : launch_cap<128, 1>(L, p);
        default: return launch_cap<256, 1>(L, p);
    }
}

// Sets this translation unit's test controls (see ptx.cuh).
attn_status set_test_controls_prefill8(unsigned long long wait_limit_ns, int stall) {
    if (cudaMemcpyToSymbol(g_wait_limit_ns, &wait_limit_ns, sizeof(wait_limit_ns)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_stall_first_tile, &stall, sizeof(stall)) != cudaSuccess)
        return set_error(ATTN_ECUDA, "test controls (prefill int8): %s", cudaGetErrorString(cudaGetLastError()));
    return ATTN_OK;
}

}  // namespace attn
