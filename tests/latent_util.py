"""Plain 64-bit forms of latent attention for its tests, and bounds of what the kernels may be
off by, derived from the roundings they make."""
import math

import torch

F16 = torch.finfo(torch.float16).eps / 2   # largest relative rounding of a normal f16 (2^-11)
# Norm and rotation in f32: a sum of R <= 512 squares (16 serial and 5 pairwise additions), a
# product with 1/R, an rsqrt (2 ulp), at most 6 products and sums: under 32 roundings of 2^-24
# each, relative to |a| + |b| of a rotated pair.
F32_CHAIN = 32 * 2.0 ** -24
# Logits: products of f16 values are exact in f32; sums of up to 576 of them in the tensor cores
# (each partial sum off by at most 2^-21 of the magnitudes added, 36 steps of 16), the scale's
# product, the offset's subtraction and 2^x (2 ulp).  Relative to scale * sum |q| |x|.
LOGIT = 40 * 2.0 ** -22


def starts(lens, device="cpu"):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=device)


def rows_of(case, b, n):
    """The first n cached rows of sequence b, 64-bit; a page id outside the pool gives zeros."""
    if case.page_table is None:
        return case.cache[b, :n].double()
    P, pages = case.page_size, case.cache.shape[0]
    ids = case.page_table[b, : -(-n // P)].long()
    good = (ids >= 0) & (ids < pages)
    x = torch.where(good[:, None, None], case.cache[ids.clamp(0, pages - 1)].double(), 0.0)
    return x.flatten(0, 1)[:n]


def _softmax_rows(t, keep, values, mags):
    """Softmax of logits t [..., n, L] over the kept keys applied to values [L, d]: (out, lse, bound of
    the output's error).  mags: bound of each row's logits' errors [..., n, 1]."""
    t = t.masked_fill(~keep, -math.inf)
    lse = torch.logsumexp(t, -1)
    some = torch.isfinite(lse)[..., None]
    p = torch.where(some & keep, torch.exp(t - torch.where(some, lse[..., None], 0.0)), 0.0)
    out = p @ values
    # The weights' roundings d_j (f16: at most 2^-11 each, or 2^-25 of the row's largest) and the
    # logits' errors move the output by sum p_j d_j (v_j - out) / (1 + ..), and
    # sum p_j |v_j - out| <= sqrt(sum p_j v_j^2 - out^2) (Cauchy); the sum is over the rounded weights.
    spread = torch.sqrt(torch.clamp(p @ values.square() - out.square(), min=0.0))
    top = p.amax(-1, keepdim=True)
    tiny = 2.0 ** -25 * top * (keep.double() @ values.abs() + keep.sum(-1, keepdim=True) * out.abs())
    bound = 1.01 * ((F16 + 2 * mags) * spread + tiny + F16 * out.abs()) + 2.0 ** -24
    return out, lse, bound


def attend_reference(case, q, q_lens, max_q=None):
    """attn_latent_attend in 64 bits: (out [T, H, R], lse [T, H], bound of the output's error)."""
    T, H, W = q.shape
    R, dev = W - 64, q.device
    out = torch.zeros(T, H, R, dtype=torch.float64, device=dev)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    bound = torch.full((T, H, R), 2.0 ** -24, dtype=torch.float64, device=dev)
    cap = case.cache.shape[1] if case.page_table is None else case.max_pages * case.page_size
    a = 0
    for b, n in enumerate(q_lens):
        full = int(case.kv_len[b])
        L = max(0, min(full, cap))
        m = n if max_q is None else min(n, max_q)
        if m and L:
            x = rows_of(case, b, L)
            qq = q[a:a + m].double()
            t = case.scale * torch.einsum("ihd,jd->ihj", qq, x)
            mags = LOGIT * abs(case.scale) * torch.einsum("ihd,jd->ihj", qq.abs(), x.abs()).amax(-1, keepdim=True)
            pos = full - n + torch.arange(m, device=dev)
            keep = (torch.arange(L, device=dev)[None] <= pos[:, None])[:, None].expand(m, H, L)
            out[a:a + m], lse[a:a + m], bound[a:a + m] = _softmax_rows(t, keep, x[:, :R], mags)
        a += n
    return out, lse, bound


def prefill_reference(q, k, v, k_rope, q_lens, kv_lens, scale, causal=True):
    """attn_latent_prefill in 64 bits: (out [T, H, 128], lse [T, H], bound of the output's error)."""
    T, H = q.shape[:2]
    dev = q.device
    out = torch.zeros(T, H, 128, dtype=torch.float64, device=dev)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    bound = torch.full((T, H, 128), 2.0 ** -24, dtype=torch.float64, device=dev)
    a = c = 0
    for n, L in zip(q_lens, kv_lens):
        if n and L:
            pos = L - n + torch.arange(n, device=dev)
            j = torch.arange(L, device=dev)
            keep = j[None] <= pos[:, None] if causal else torch.ones(n, L, dtype=torch.bool, device=dev)
            for h in range(H):
                qq = q[a:a + n, h].double()
                kk = torch.cat((k[c:c + L, h], k_rope[c:c + L]), -1).double()
                mags = LOGIT * abs(scale) * (qq.abs() @ kk.abs().T).amax(-1, keepdim=True)
                o, s, e = _softmax_rows(scale * (qq @ kk.T), keep, v[c:c + L, h].double(), mags)
                out[a:a + n, h], lse[a:a + n, h], bound[a:a + n, h] = o, s, e
        a, c = a + n, c + L
    return out, lse, bound


def assert_within(got, ref, bound, what=""):
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all()), "%s: non-finite output" % what
    worst = (err / bound).max() if err.numel() else torch.tensor(0.0)
    assert float(worst) <= 1.0, "%s: error %.3g of the bound (max-abs %.3g)" % (what, worst, err.max())


def assert_lse(got, ref, what=""):
    # the sum is over rounded weights (2^-11 relative), the logarithm's argument and log2 approximate
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin) and bool((got[~fin] == ref[~fin]).all()), "%s: lse of empty rows" % what
    if fin.any():
        err = (got.double() - ref)[fin].abs()
        assert float((err - 2.0 ** -20 * ref[fin].abs()).max()) <= 2 * F16, "%s: lse max-abs %.3g" % (what, err.max())
