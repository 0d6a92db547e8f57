// prefill_int8.cu -- a chunk of new tokens of every sequence over its int8 paged
// cache (attn_prefill_paged_ex with ATTN_KV_INT8).
//
//   o_i = sum_j softmax_j(cap(scale * ks_j * q_i . kcode_j)) f16(vcode_j * vs_j)
//
// over the keys j <= pos_i (and pos_i - j < W).  One CTA a (packed query, head),
// a thread a key of a 128-key tile for the logits and a column for the sum, in
// f32 with a running maximum and sum.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"

namespace attn {
namespace {

constexpr int kTile = 128;

struct Args8 {
    Prefill8Launch L;
    int log2P;
};

__device__ __forceinline__ float dequant(int8_t c, __half s) {
    return __half2float(__float2half_rn(static_cast<float>(c) * __half2float(s)));
}

template <int D>
__global__ void __launch_bounds__(kTile) prefill8_kernel(const Args8 a) {
    __shared__ float q[D];
    __shared__ float pr[kTile];
    __shared__ int page[kTile];
    __shared__ float red[8];
    const Prefill8Launch& L = a.L;
    const int t = blockIdx.x, h = blockIdx.y, g = h / (L.Hq / L.Hkv), tid = threadIdx.x;
    int b = 0;
    while (b < L.B && L.q_start[b + 1] <= t) ++b;
    if (b >= L.B || t < L.q_start[b]) return;
    const long long pos = static_cast<long long>(L.kv_len[b]) - L.q_start[b + 1] + t;
    const long long cap = static_cast<long long>(L.max_pages) * L.page_size;
    const long long hi = min(min(pos + 1, cap), static_cast<long long>(max(L.kv_len[b], 0)));
    const long long lo = L.window > 0 ? max(0ll, pos - L.window + 1) : 0;
    const size_t row = static_cast<size_t>(t) * L.Hq + h;
    for (int i = tid; i < D; i += kTile) q[i] = __half2float(static_cast<const __half*>(L.q)[row * D + i]);
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[D / kTile > 0 ? D / kTile : 1] = {};
    for (long long j0 = lo; j0 < hi; j0 += kTile) {
        const long long j = j0 + tid;
        float s = -INFINITY;
        int pg = -1;
        if (j < hi) {
            pg = L.page_table[static_cast<size_t>(b) * L.max_pages + (j >> a.log2P)];
            if (pg < 0 || pg >= L.n_pages) {
                atomicExch(L.err_word, kErrBadPage);
                pg = -1;
            }
            float d = 0.f;
            if (pg >= 0) {
                const int r = static_cast<int>(j & (L.page_size - 1));
                const int8_t* kp = static_cast<const int8_t*>(L.k) +
                                   ((static_cast<size_t>(pg) * L.page_size + r) * L.Hkv + g) * D;
                const __half ks = static_cast<const __half*>(L.k_scales)[(static_cast<size_t>(pg) * L.Hkv + g) * L.page_size + r];
                for (int i = 0; i < D; ++i) d = fmaf(q[i], static_cast<float>(kp[i]), d);
                // a scale that is not finite makes the logit, and so the row, NaN
                const float vs = __half2float(static_cast<const __half*>(
                    L.v_scales)[(static_cast<size_t>(pg) * L.Hkv + g) * L.page_size + r]);
                d = isfinite(__half2float(ks)) && isfinite(vs) ? d * __half2float(ks) : NAN;
            }
            s = d * L.scale;
            if (L.softcap > 0.f) s = L.softcap * tanhf(s / L.softcap);
        }
        page[tid] = pg;
        float mx = s;
        for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float off = mn == -INFINITY ? 0.f : mn;
        const float p = expf(s - off);
        pr[tid] = p;
        float sum = p;
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if ((tid & 31) == 0) red[4 + (tid >> 5)] = sum;
        __syncthreads();
        const float alpha = m == -INFINITY ? 0.f : expf(m - off);
        l = l * alpha + ((red[4] + red[5]) + (red[6] + red[7]));
        m = mn;
        const int n = static_cast<int>(min(hi - j0, static_cast<long long>(kTile)));
        for (int c = 0; c * kTile < D; ++c) {
            const int col = c * kTile + tid;
            float acc = o[c] * alpha;
            if (col < D)
                for (int x = 0; x < n; ++x) {
                    const int pgx = page[x];
                    if (pgx < 0) continue;
                    const int r = static_cast<int>((j0 + x) & (L.page_size - 1));
                    const int8_t cv = static_cast<const int8_t*>(
                        L.v)[((static_cast<size_t>(pgx) * L.page_size + r) * L.Hkv + g) * D + col];
                    acc = fmaf(pr[x], dequant(cv, static_cast<const __half*>(L.v_scales)[(static_cast<size_t>(pgx) * L.Hkv + g) *
                                                                                    L.page_size + r]), acc);
                }
            o[c] = acc;
        }
        __syncthreads();
    }
    for (int c = 0; c * kTile < D; ++c) {
        const int col = c * kTile + tid;
        if (col < D) static_cast<__half*>(L.out)[row * D + col] = __float2half_rn(hi > lo ? o[c] / l : 0.f);
    }
    if (L.lse && tid == 0) L.lse[row] = hi > lo ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t prefill8_workspace(int, int, int, int) { return 256; }

attn_status launch_prefill8(const Prefill8Launch& L) {
    Args8 a;
    a.L = L;
    a.log2P = 0;
    while ((1 << a.log2P) < L.page_size) ++a.log2P;
    const dim3 grid(L.total_q, L.Hq);
    if (trace_enabled()) trace("prefill8_kernel<D=%d> grid=(%u,%u) block=%d", L.D, grid.x, grid.y, kTile);
    if (L.D == 64) prefill8_kernel<64><<<grid, kTile, 0, L.stream>>>(a);
    else if (L.D == 128) prefill8_kernel<128><<<grid, kTile, 0, L.stream>>>(a);
    else prefill8_kernel<256><<<grid, kTile, 0, L.stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return set_error(ATTN_ECUDA, "prefill (int8) launch failed: %s", cudaGetErrorString(e));
    return ATTN_OK;
}

}  // namespace attn
