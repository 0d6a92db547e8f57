"""Measured workloads of the cache operators: attn_append (per-head q/k norm,
rotary positions and the cache write in one pass, f16 or int8), attn_kv_read
(cache tokens back as rows) and attn_prefill_paged_ex (a chunk of new tokens
over an int8 paged cache).

``run`` takes what ``prepare`` made through one pass: the operators' plain form
in elementary torch operations, or with ``own`` the library's entry points.
``exact`` is the same in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def _append(name, **kw):
    c = dict(op="append", name=name, B=1, q_lo=1, q_hi=1, kv_lo=1, kv_hi=128, Hq=4, Hkv=2, D=64, page=0, ring=0,
             int8=False, f32=False, norm=True, offset=0.0, rot=64, interleaved=False, lens=1)
    c.update(kw)
    return c


def _read(name, **kw):
    c = dict(op="read", name=name, B=1, n_lo=1, n_hi=1, kv_lo=1, kv_hi=128, Hkv=2, D=64, page=0, ring=0, int8=True,
             f32=False, lens=2)
    c.update(kw)
    return c


def _chunk(name, **kw):
    c = dict(op="chunk", name=name, B=1, q_lo=1, q_hi=1, kv_lo=128, kv_hi=128, Hq=4, Hkv=2, D=64, page=16, window=0,
             softcap=0.0, scale=0.0, lens=3)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of the smallest model: its latency is a launch
        _append("append_tiny_decode", kv_lo=128, kv_hi=128),
        # one decode step of 32 sequences of a grouped-query model over int8 pages, read back
        _append("append_decode_int8_pages", B=32, kv_lo=512, kv_hi=8192, Hq=32, Hkv=8, D=128, rot=128, page=16,
                int8=True, lens=11),
        # chunks of ragged lengths (some short, one near 700) of the same model: the prefill of a server's step
        _append("append_chunks_int8_pages", B=8, q_lo=33, q_hi=700, kv_lo=701, kv_hi=8192, Hq=32, Hkv=8, D=128,
                rot=128, page=16, int8=True, lens=12),
        # a whole prompt of a sliding-window model with wide heads, f32 activations, (1 + w) norms, ring cache
        _append("append_prompt_f32_ring", q_lo=4096, q_hi=4096, kv_lo=4096, kv_hi=4096, Hq=8, Hkv=4, D=256, rot=256,
                ring=1024, f32=True, offset=1.0, lens=13),
        # a partial page of one short sequence back as rows
        _read("read_37_tokens", n_lo=37, n_hi=37, kv_lo=101, kv_hi=101, page=16, lens=21),
        # every token of a long-context int8 batch back as f16 (leaving the cache for another tier)
        _read("read_long_int8", B=16, n_lo=32768, n_hi=32768, kv_lo=32768, kv_hi=32768, Hkv=8, D=128, lens=22),
        # what wide-head ring caches hold, as f32 rows
        _read("read_ring_f32", B=5, n_lo=700, n_hi=1024, kv_lo=1024, kv_hi=5000, Hkv=4, D=256, ring=1024, int8=False,
              f32=True, lens=23),
        # one new token of the smallest model over its int8 pages
        _chunk("chunk_tiny_one_token"),
        # 1 to 8 draft tokens of each of 32 sequences checked against their caches
        _chunk("chunk_verify_drafts", B=32, q_lo=1, q_hi=8, kv_lo=512, kv_hi=8192, Hq=32, Hkv=8, D=128, lens=31),
        # 4 draft tokens of each of 16 long contexts: the cache's bytes are the cost
        _chunk("chunk_verify_long", B=16, q_lo=4, q_hi=4, kv_lo=32768, kv_hi=32768, Hq=32, Hkv=8, D=128, lens=32),
        # prefill chunks of 512 tokens of 8 sequences over ragged contexts: the products are the cost
        _chunk("chunk_prefill_512", B=8, q_lo=512, q_hi=512, kv_lo=513, kv_hi=8192, Hq=32, Hkv=8, D=128, lens=33),
        # a 4096-token prompt with soft-capped logits, a window of 1024 and wide heads
        _chunk("chunk_softcap_window", q_lo=4096, q_hi=4096, kv_lo=4096, kv_hi=4096, Hq=8, Hkv=4, D=256, window=1024,
               softcap=50.0, scale=1.0 / 16.0, lens=34),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    B = _log_int(rng, 1, 32)
    lens = rng.randrange(1, 1 << 20)
    op = rng.choice(["append", "read", "chunk", "chunk"])
    if op == "append":
        q_hi = _log_int(rng, 1, 4096)
        kv_hi = q_hi + _log_int(rng, 1, 8192)
        while B > 1 and B * q_hi > 6000:
            B = (B + 1) // 2
        while B > 1 and B * kv_hi * Hkv * D > (1 << 26):
            B = (B + 1) // 2
        while Hkv > 1 and B * q_hi * (G + 2) * Hkv * D > (1 << 24):
            Hkv = (Hkv + 1) // 2
        layout = rng.choice(["plain", "page", "ring"])
        int8 = rng.random() < 0.5
        return _append("", B=B, q_lo=max(1, q_hi // 3), q_hi=q_hi, kv_lo=q_hi, kv_hi=kv_hi, Hq=G * Hkv, Hkv=Hkv, D=D,
                       page=rng.choice([8, 16, 32, 64, 256]) if layout == "page" else 0,
                       ring=16 * _log_int(rng, 1, 100) if layout == "ring" else 0, int8=int8, f32=rng.random() < 0.3,
                       norm=rng.random() < 0.7, offset=rng.choice([0.0, 1.0]), rot=rng.choice([0, 16, 32, D // 2, D, D]),
                       interleaved=rng.random() < 0.4, lens=lens)
    if op == "read":
        kv_hi = _log_int(rng, 16, 16384)
        while B > 1 and B * kv_hi * Hkv * D > (1 << 27):
            B = (B + 1) // 2
        layout = rng.choice(["plain", "page", "ring"])
        n_hi = _log_int(rng, 1, kv_hi)
        return _read("", B=B, n_lo=max(1, n_hi // 4), n_hi=n_hi, kv_lo=n_hi, kv_hi=kv_hi, Hkv=Hkv, D=D,
                     page=rng.choice([8, 16, 32, 64, 256]) if layout == "page" else 0,
                     ring=16 * _log_int(rng, 1, 100) if layout == "ring" else 0, int8=rng.random() < 0.7,
                     f32=rng.random() < 0.3, lens=lens)
    q_hi = _log_int(rng, 1, 1024)
    kv_hi = q_hi + _log_int(rng, 16, 16384)
    while B > 1 and (B * kv_hi * Hkv * D > (1 << 27) or B * G * Hkv * q_hi * kv_hi > (1 << 29)):
        B = (B + 1) // 2
    while Hkv > 1 and (B * kv_hi * Hkv * D > (1 << 27) or B * G * Hkv * q_hi * kv_hi > (1 << 29)):
        Hkv = (Hkv + 1) // 2
    return _chunk("", B=B, q_lo=max(1, q_hi // 4), q_hi=q_hi, kv_lo=q_hi + (kv_hi - q_hi) // 8, kv_hi=kv_hi, Hq=G * Hkv,
                  Hkv=Hkv, D=D, page=rng.choice([8, 16, 32, 64, 256]),
                  window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), softcap=rng.choice([0.0, 0.0, 30.0]), lens=lens)


def _lengths(case):
    """(new or read tokens, cached tokens) of each sequence: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    lo, hi = ("n_lo", "n_hi") if case["op"] == "read" else ("q_lo", "q_hi")
    n = [r.randint(case[lo], case[hi]) for _ in range(case["B"])]
    kv = [r.randint(max(case["kv_lo"], x), max(case["kv_hi"], x)) for x in n]
    if case["op"] == "read" and case["ring"]:
        n = [min(x, case["ring"]) for x in n]
    return n, kv


# ------------------------------------------------------------------ the inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _codes(g, *shape):
    # codes of rows of normal values: their largest is near 127 / 3.5 times the deviation of one value
    return (_normal(g, *shape) * 36.0).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, *shape):
    return (0.0276 * (1.0 + 0.2 * torch.rand(shape, generator=g, device=DEV))).to(torch.float16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    n, kv = _lengths(case)
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    total = sum(n)
    start = torch.tensor([0] + list(torch.tensor(n).cumsum(0).tolist()), dtype=torch.int32, device=DEV)
    s = dict(case=case, B=B, Hkv=Hkv, D=D, total=total, max_q=max(n), max_kv=max(kv), start=start,
             kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV), int8=case.get("int8", True), table=None, max_pages=0, n_pages=0,
             page=case["page"], ring=case.get("ring", 0), k_scales=None, v_scales=None)
    if s["page"]:
        P = s["page"]
        need = [-(-x // P) for x in kv]
        s["max_pages"], s["n_pages"] = max(need), sum(need) + 3
        perm = torch.randperm(s["n_pages"], generator=g, device=DEV).to(torch.int32).cpu()
        table, at = torch.full((B, s["max_pages"]), -1, dtype=torch.int32), 0
        for b in range(B):
            table[b, : need[b]] = perm[at : at + need[b]]
            at += need[b]
        s["table"] = table.to(DEV)
        slots, rows = s["n_pages"], P
    else:
        slots, rows = B, s["ring"] or -(-max(kv) // 8) * 8
    s["cap"] = rows
    shape = (slots, rows, Hkv, D)
    # an append starts from an empty cache; the others find a full one
    if s["int8"]:
        full = case["op"] != "append"
        for x in ("k", "v"):
            s[x] = _codes(g, *shape) if full else torch.zeros(shape, dtype=torch.int8, device=DEV)
            s[x + "_scales"] = (_scales(g, slots, Hkv, rows) if full
                                else torch.zeros((slots, Hkv, rows), dtype=torch.float16, device=DEV))
    else:
        for x in ("k", "v"):
            s[x] = (_normal(g, *shape).to(torch.float16) if case["op"] != "append"
                    else torch.zeros(shape, dtype=torch.float16, device=DEV))
    dt = torch.float32 if case.get("f32") else torch.float16
    if case["op"] == "append":
        Hq, R = case["Hq"], case["rot"]
        # one projection's output: q, k and v rows side by side
        s["qkv"] = _normal(g, total, (Hq + 2 * Hkv) * D).mul_(1.5).to(dt)
        s["q_norm"] = 1.0 - case["offset"] + 0.1 * _normal(g, D) if case["norm"] else None
        s["k_norm"] = 1.0 - case["offset"] + 0.1 * _normal(g, D) if case["norm"] else None
        s["cos"] = s["sin"] = None
        if R:
            inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
            angle = torch.arange(max(kv), dtype=torch.float64, device=DEV)[:, None] * inv
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["q_out"] = torch.empty((total, Hq, D), dtype=torch.float16, device=DEV)
    if case["op"] == "chunk":
        s["q"] = _normal(g, total, case["Hq"], D).to(torch.float16)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = case["scale"] or 1.0 / math.sqrt(D)
    if case["op"] == "read" or (case["op"] == "append" and s["int8"]):
        ot = torch.float32 if case["op"] == "read" and case["f32"] else torch.float16
        s["k_out"] = torch.empty((total, Hkv, D), dtype=ot, device=DEV)
        s["v_out"] = torch.empty((total, Hkv, D), dtype=ot, device=DEV)
        # the read takes the last tokens; after an append those are the ones it wrote
        first = [a - b for a, b in zip(kv, n)]
        s["first"] = torch.tensor(first, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ the plain forms
def _where(s):
    """Of each packed row: its sequence, position, whether the cache keeps it, and its (slot, row)."""
    t = torch.arange(s["total"], device=DEV)
    b = (t[:, None] >= s["start"][None, 1:]).sum(1)
    pos = s["kv_len"][b] - s["start"][b + 1] + t
    keep = torch.ones_like(pos, dtype=torch.bool)
    if s["page"]:
        return b, pos, keep, s["table"][b, pos // s["page"]].long(), pos % s["page"]
    if s["ring"]:
        keep = pos >= s["kv_len"][b] - s["ring"]
        return b, pos, keep, b, pos % s["ring"]
    return b, pos, keep, b, pos


def _norm_rotate(x, w, pos, s):
    c, R = s["case"], s["case"]["rot"]
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (w + c["offset"])
    if R:
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        if c["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., : R // 2], x[..., R // 2 : R]
            rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        x = torch.cat((rot, x[..., R:]), -1)
    return x


def _quantise(x):
    scale = (x.abs().amax(-1) / 127.0).to(torch.float16)
    wide = scale.float()[..., None]
    codes = torch.where(wide > 0, (x / wide).round().clamp(-127, 127), torch.zeros_like(x))
    return codes.to(torch.int8), scale


def _plain_append(s):
    c, Hkv, D = s["case"], s["Hkv"], s["D"]
    Hq = c["Hq"]
    b, pos, keep, slot, row = _where(s)
    x = s["qkv"].float().view(s["total"], Hq + 2 * Hkv, D)
    q = _norm_rotate(x[:, :Hq], s["q_norm"], pos, s).to(torch.float16)
    k = _norm_rotate(x[:, Hq : Hq + Hkv], s["k_norm"], pos, s)
    v = x[:, Hq + Hkv :]
    kept, slot, row = keep.nonzero()[:, 0], slot[keep], row[keep]
    if not s["int8"]:
        s["k"][slot, row] = k[kept].to(torch.float16)
        s["v"][slot, row] = v[kept].to(torch.float16)
        return {"q": q, "k_cache": s["k"], "v_cache": s["v"]}
    s["k"][slot, row], ks = _quantise(k[kept])
    s["v"][slot, row], vs = _quantise(v[kept])
    s["k_scales"][slot, :, row] = ks
    s["v_scales"][slot, :, row] = vs
    k, v = _plain_read(s, torch.float16)
    return {"q": q, "k": k, "v": v}


def _plain_read(s, dtype):
    b, pos, keep, slot, row = _where(s)
    k, v = s["k"][slot, row].float(), s["v"][slot, row].float()
    if s["int8"]:
        k = k * s["k_scales"][slot, :, row].float()[..., None]
        v = v * s["v_scales"][slot, :, row].float()[..., None]
    zero = torch.zeros((), device=DEV)
    keep = keep[:, None, None]
    return torch.where(keep, k, zero).to(dtype), torch.where(keep, v, zero).to(dtype)


def _rows_of(s, x, scales):
    """All cached tokens of every sequence, in order and padded: [B, Hkv, max_kv, D]."""
    j = torch.arange(s["max_kv"], device=DEV)
    pages = s["table"][:, j // s["page"]].long().clamp_min(0)
    rows = x[pages, j % s["page"]].float() * scales[pages, :, j % s["page"]].float()[..., None]
    return torch.where((j < s["kv_len"][:, None])[..., None, None], rows, torch.zeros((), device=DEV)).transpose(1, 2)


def _plain_chunk(s):
    c, B, Hkv, D = s["case"], s["B"], s["Hkv"], s["D"]
    G, n = c["Hq"] // Hkv, s["max_q"]
    q_len = s["start"][1:] - s["start"][:-1]
    i = torch.arange(n, device=DEV)
    at = (s["start"][:-1, None] + i).clamp_max(s["total"] - 1)
    q = s["q"].float()[at].view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    t = torch.matmul(q, _rows_of(s, s["k"], s["k_scales"]).transpose(2, 3)).view(B, Hkv, G, n, s["max_kv"]) * s["scale"]
    if c["softcap"]:
        t = c["softcap"] * torch.tanh(t / c["softcap"])
    pos = (s["kv_len"] - q_len)[:, None] + i
    j = torch.arange(s["max_kv"], device=DEV)
    keep = j <= pos[..., None]
    if c["window"]:
        keep = keep & (pos[..., None] - j < c["window"])
    keep = (keep & (j < s["kv_len"][:, None, None]))[:, None, None]
    t = t.masked_fill(~keep, -math.inf)
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    del t
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * n, -1), _rows_of(s, s["v"], s["v_scales"])).view(B, Hkv, G, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hkv * G, D)
    return o[i < q_len[:, None]].to(torch.float16)


# ------------------------------------------------------------------ the library's calls
def _own_read(attn, s):
    attn.attn_kv_read(s["k"], s["v"], s["kv_len"], s["first"], s["start"], s["table"], s["page"], s["max_pages"],
                      s["n_pages"], s["cap"], s["ring"], s["k_scales"], s["v_scales"],
                      attn.ATTN_KV_INT8 if s["int8"] else attn.ATTN_KV_F16, s["B"], s["total"], s["Hkv"], s["D"],
                      s["k_out"], s["v_out"], attn.ATTN_F32 if s["k_out"].dtype == torch.float32 else attn.ATTN_F16)
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_append(attn, s):
    c, Hkv, D = s["case"], s["Hkv"], s["D"]
    Hq, qkv = c["Hq"], s["qkv"]
    attn.attn_append(qkv, qkv[:, Hq * D :], qkv[:, (Hq + Hkv) * D :], attn.ATTN_F32 if c["f32"] else attn.ATTN_F16,
                     qkv.stride(0), qkv.stride(0), qkv.stride(0), s["q_norm"], s["k_norm"], 1e-6, c["offset"],
                     s["cos"], s["sin"], 0 if s["cos"] is None else s["cos"].shape[0], c["rot"], c["interleaved"],
                     s["start"], s["kv_len"], s["k"], s["v"], s["table"], s["page"], s["max_pages"], s["n_pages"],
                     s["cap"], s["ring"], s["k_scales"], s["v_scales"],
                     attn.ATTN_KV_INT8 if s["int8"] else attn.ATTN_KV_F16, s["B"], s["total"], Hq, Hkv, D,
                     s["q_out"], attn.ATTN_F16)
    if not s["int8"]:
        return {"q": s["q_out"], "k_cache": s["k"], "v_cache": s["v"]}
    return {"q": s["q_out"], **_own_read(attn, s)}


def _own_chunk(attn, s):
    c = s["case"]
    if "workspace" not in s:
        size = attn.attn_prefill_paged_workspace_size(s["B"], s["max_q"], c["Hq"], s["Hkv"], s["D"], attn.ATTN_KV_INT8)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    attn.attn_prefill_paged_ex(s["q"], s["k"], s["v"], s["start"], s["kv_len"], s["table"], s["page"], s["max_pages"],
                               s["n_pages"], s["k_scales"], s["v_scales"], attn.ATTN_KV_INT8, s["B"], s["total"],
                               s["max_q"], c["Hq"], s["Hkv"], s["D"], c["window"], c["softcap"], s["scale"], s["out"],
                               None, s["workspace"], s["workspace"].numel())
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        import attention_split_kv_gb300 as attn

        return (_own_append if op == "append" else _own_read if op == "read" else _own_chunk)(attn, state)
    if op == "append":
        return _plain_append(state)
    if op == "read":
        k, v = _plain_read(state, torch.float32 if state["case"]["f32"] else torch.float16)
        return {"k": k, "v": v}
    return _plain_chunk(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    n, kv = _lengths(case)
    B, Hkv, D, T = case["B"], case["Hkv"], case["D"], sum(n)
    lens = 8 * B + 4
    if case["op"] == "append":
        e = 4 if case["f32"] else 2
        Hq, R = case["Hq"], case["rot"]
        kept = sum(min(x, case["ring"]) if case["ring"] else x for x in n)
        token = Hkv * 2 * ((D + 2) if case["int8"] else 2 * D)
        size = T * ((Hq + 2 * Hkv) * D * e + R * 4 + Hq * D * 2) + kept * token + lens
        if case["int8"]:
            size += kept * token + T * Hkv * D * 4
        return {"bytes": size, "flops": T * (Hq + 2 * Hkv) * D * 8}
    if case["op"] == "read":
        token = Hkv * 2 * ((D + 2) if case["int8"] else 2 * D)
        return {"bytes": T * (token + Hkv * D * 2 * (4 if case["f32"] else 2)) + lens, "flops": 2 * T * Hkv * D}
    W, pairs, used = case["window"], 0, 0
    for a, L in zip(n, kv):
        first = L - a
        pairs += sum(min(p + 1, W) if W else p + 1 for p in range(first, L))
        used += L - (max(0, first - W + 1) if W else 0)
    return {"bytes": used * Hkv * 2 * (D + 2) + T * case["Hq"] * D * 4 + lens, "flops": 4 * D * pairs * case["Hq"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_heads(s, x, w, positions):
    """Norm and rotation of [T, H, D] rows: the rotation as a product with 2 x 2 matrices."""
    c, R = s["case"], s["case"]["rot"]
    x = x.double()
    if w is not None:
        mean = torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / x.shape[-1]
        x = x / (mean + 1e-6).sqrt() * (w.double() + c["offset"])
    if R:
        x = x.clone()
        first = torch.arange(0, R, 2, device=DEV) if c["interleaved"] else torch.arange(R // 2, device=DEV)
        second = first + 1 if c["interleaved"] else first + R // 2
        z = torch.complex(x[..., first], x[..., second])
        turn = torch.complex(s["cos"].double()[positions], s["sin"].double()[positions])[:, None]
        z = z * turn
        x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_int8(x):
    """The values that a row's codes stand for."""
    step = (x.abs().max(-1, keepdim=True).values / 127).to(torch.float16).double()
    live = step > 0
    return torch.round(x / torch.where(live, step, 1.0)).clamp(-127, 127) * step * live


def exact(case, seed):
    s = prepare(case, seed)
    n, kv = _lengths(case)
    Hkv, D = s["Hkv"], s["D"]
    seq = torch.tensor([b for b, x in enumerate(n) for _ in range(x)], device=DEV)
    pos = torch.tensor([L - x + i for x, L in zip(n, kv) for i in range(x)], device=DEV)
    length = torch.tensor(kv, device=DEV)[seq]
    held = pos >= length - s["ring"] if s["ring"] else pos >= 0
    if s["page"]:
        slot, row = s["table"].long()[seq, torch.div(pos, s["page"], rounding_mode="floor")], pos % s["page"]
    else:
        slot, row = seq, pos % s["ring"] if s["ring"] else pos
    if case["op"] == "append":
        q, k, v = s["qkv"].view(len(seq), -1, D).split((case["Hq"], Hkv, Hkv), 1)
        out = {"q": _exact_heads(s, q, s["q_norm"], pos)}
        k, v = _exact_heads(s, k, s["k_norm"], pos), v.double()
        if s["int8"]:
            return {**out, "k": _exact_int8(k) * held[:, None, None], "v": _exact_int8(v) * held[:, None, None]}
        for name, x in (("k_cache", k), ("v_cache", v)):
            cache = torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV)
            cache[slot[held], row[held]] = x[held]
            out[name] = cache
        return out
    if case["op"] == "read":
        out = {}
        for name in ("k", "v"):
            x = s[name][slot, row].double()
            if s["int8"]:
                x = x * s[name + "_scales"].transpose(1, 2)[slot, row].double()[..., None]
            out[name] = x * held[:, None, None]
        return out
    G = case["Hq"] // Hkv
    outs = []
    for b in range(s["B"]):  # one sequence at a time
        L, m = kv[b], n[b]
        pages = s["table"][b, : -(-L // s["page"])].long()
        k, v = ((s[x][pages].double() * s[x + "_scales"][pages].double().transpose(1, 2)[..., None]).flatten(0, 1)[:L] for x in ("k", "v"))
        p = torch.arange(L - m, L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None]
        hide = j > p
        if case["window"]:
            hide = hide | (j <= p - case["window"])
        a = int(s["start"][b])
        q = s["q"][a : a + m].double()
        heads = []
        for h in range(case["Hq"]):
            t = s["scale"] * (q[:, h] @ k[:, h // G].T)
            if case["softcap"]:
                t = case["softcap"] * torch.tanh(t / case["softcap"])
            heads.append(torch.softmax(t.masked_fill(hide, -math.inf), -1) @ v[:, h // G])
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)
