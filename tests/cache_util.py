"""Plain 64-bit forms of the cache operators (append, read back, int8 chunks)
for their tests, on the CPU, and the caches they run on."""
import math

import torch

import seeded_inputs as si

F16_HALF = torch.finfo(torch.float16).eps / 2     # largest relative rounding of a normal f16
F16_TINY = 2.0 ** -25                             # half a step of subnormal f16
# f32 arithmetic of norm and rotation: a sum of D <= 256 squares in 8 serial and 5
# pairwise additions, a division, an rsqrt (2 ulp) and at most 6 products and sums:
# under 32 roundings of at most 2^-24 each, relative to |a| + |b| of the rotated pair
F32_CHAIN = 32 * 2.0 ** -24


class Cache:
    """A cache of any layout: what attn.append / attn.kv_read take as their case."""

    def __init__(self, layout, B, Hkv, D, cap, *, int8=False, page_size=16, ring=0, seed=0, fill=False, device="cpu"):
        self.layout, self.batch, self.n_kv_heads, self.head_dim, self.int8 = layout, B, Hkv, D, int8
        self.page_table, self.page_size, self.max_pages, self.ring = None, 0, 0, 0
        if layout == "paged":
            self.page_size = P = page_size
            self.max_pages = -(-cap // P)
            n_pages = B * self.max_pages + 2
            perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))
            self.page_table = perm[: B * self.max_pages].view(B, self.max_pages).to(torch.int32)
            slots, rows = n_pages, P
        else:
            self.ring = ring if layout == "ring" else 0
            slots, rows = B, ring if layout == "ring" else -(-cap // 8) * 8
        self.cap = self.max_pages * self.page_size if layout == "paged" else rows
        x = [si.f16_normal((slots, rows, Hkv, D), seed * 10 + i) for i in (1, 2)]
        self.k_scales = self.v_scales = None
        if int8:
            codes = [si.quantize_int8_rows(y) for y in x]
            self.k, self.v = (c for c, _ in codes)
            self.k_scales, self.v_scales = (s.permute(0, 2, 1).contiguous() for _, s in codes)
        else:
            self.k, self.v = x
        if not fill:   # recognisable contents of what no token was written to
            for t in (self.k, self.v):
                t.fill_(77)
            if int8:
                self.k_scales.fill_(0.5)
                self.v_scales.fill_(0.5)

    def to(self, device):
        import copy
        c = copy.copy(self)
        for name in ("k", "v", "k_scales", "v_scales", "page_table", "kv_len"):
            t = getattr(self, name, None)
            if t is not None:
                setattr(c, name, t.to(device).clone())
        return c

    def where(self, b, p):
        """(slot, row) of position p of sequence b."""
        if self.layout == "paged":
            return int(self.page_table[b, p // self.page_size]), p % self.page_size
        return b, p % self.ring if self.ring else p

    def head(self, name, b, p, h):
        """The 64-bit value of one cached head."""
        s, r = self.where(b, p)
        x = getattr(self, name)[s, r, h].double()
        return x * getattr(self, name + "_scales")[s, h, r].double() if self.int8 else x


def norm_rotate(x, w, eps, offset, cos, sin, p, interleaved):
    """One head in 64 bits, and |a| + |b| of each value's pair (the scale of its f32 error)."""
    x = x.double()
    if w is not None:
        x = x / math.sqrt(float((x * x).mean()) + eps) * (w.double() + offset)
    out, mag = x.clone(), x.abs()
    if cos is not None:
        R = 2 * cos.shape[1]
        for e in range(R // 2):
            i, j = (2 * e, 2 * e + 1) if interleaved else (e, e + R // 2)
            c, s = float(cos[p, e]), float(sin[p, e])
            out[i], out[j] = x[i] * c - x[j] * s, x[j] * c + x[i] * s
            mag[i] = mag[j] = x[i].abs() + x[j].abs()
    return out, mag


def tables(n_pos, R, base=10000.0):
    inv = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def chunk_reference(case):
    """attn_prefill_paged_ex in 64 bits on code * scale: (out [total_q, Hq, D], lse [total_q, Hq])."""
    T, Hq, Hkv, D, P = case.q.shape[0], case.n_heads, case.n_kv_heads, case.head_dim, case.page_size
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    for b in range(case.batch):
        r0, r1 = int(case.q_start[b]), int(case.q_start[b + 1])
        L = max(0, min(int(case.kv_len[b]), case.max_pages * P))
        if r1 <= r0 or L == 0:
            continue
        pages = case.page_table[b, : -(-L // P)].long()
        k, v = ((x[pages].double() * s[pages].double().transpose(1, 2)[..., None]).flatten(0, 1)[:L]
                for x, s in ((case.k, case.k_scales), (case.v, case.v_scales)))
        pos = int(case.kv_len[b]) - (r1 - r0) + torch.arange(r1 - r0)
        j = torch.arange(L)
        keep = j[None] <= pos[:, None]
        if case.window:
            keep &= pos[:, None] - j[None] < case.window
        some = keep.any(1)
        for h in range(Hq):
            t = case.scale * (case.q[r0:r1, h].double() @ k[:, h // (Hq // Hkv)].T)
            if case.softcap:
                t = case.softcap * torch.tanh(t / case.softcap)
            t = t.masked_fill(~keep, -math.inf)
            lse[r0:r1, h] = torch.logsumexp(t, 1)
            w = torch.where(some[:, None], torch.softmax(torch.where(some[:, None], t, 0.0), 1), 0.0)
            w = torch.where(keep, w, 0.0)
            vv = v[:, h // (Hq // Hkv)]
            out[r0:r1, h] = w @ torch.where(keep.any(0)[:, None], vv, 0.0)
    return out, lse
