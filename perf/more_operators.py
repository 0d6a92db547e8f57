"""Measured workloads of latent attention, where a token's keys and values for all
heads come from one cached vector [c | k_rope] (c normed, k_rope rotated):

* attn_latent_append: the new tokens' latent vectors normed, their key parts and the
  queries' parts rotated, and the rows written to the cache, in one pass;
* attn_latent_read: cached rows back as c and k_rope (what the expanded form multiplies);
* attn_latent_attend: the absorbed form, queries in the latent space against the cache;
* attn_latent_prefill: the expanded form, packed prompts with a key part a head, the key
  part that heads share, and a value a head.

``run`` takes what ``prepare`` made through one pass: the operators' plain form in
elementary torch operations, or with ``own`` the library's entry points.  ``exact`` is
the same in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

DEV = "cuda"
ROPE = 64      # rotated values of a key
HEAD = 128     # values of a head beside them in the expanded form (and of its value)


# ------------------------------------------------------------------ the cases
def _append(name, **kw):
    c = dict(op="append", name=name, B=1, q_lo=1, q_hi=1, kv_lo=128, kv_hi=128, H=16, R=512, page=64, f32=False,
             norm=True, offset=0.0, interleaved=True, lens=1)
    c.update(kw)
    return c


def _read(name, **kw):
    c = dict(op="read", name=name, B=1, n_lo=1, n_hi=1, kv_lo=128, kv_hi=128, R=512, page=64, f32=False, lens=2)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(op="attend", name=name, B=1, q_lo=1, q_hi=1, kv_lo=128, kv_hi=128, H=16, R=512, page=64, lens=3)
    c.update(kw)
    return c


def _prefill(name, **kw):
    c = dict(op="prefill", name=name, B=1, q_lo=37, q_hi=37, kv_lo=37, kv_hi=37, H=8, causal=True, lens=4)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of one sequence: its latency is a launch
        _append("append_one_token", H=8, R=256, page=16),
        # one decode step of 32 sequences, all heads on one GPU
        _append("append_decode_step", B=32, kv_lo=512, kv_hi=4096, H=128, lens=11),
        # chunks of ragged lengths (33 to 700 tokens) of 8 sequences: the prefill of a server's step
        _append("append_chunks", B=8, q_lo=33, q_hi=700, kv_lo=701, kv_hi=8192, H=32, lens=12),
        # a whole prompt with f32 activations, (1 + w) norms and half-split rotation, no pages
        _append("append_prompt_f32", q_lo=4096, q_hi=4096, kv_lo=4096, kv_hi=4096, H=16, page=0, f32=True, offset=1.0,
                interleaved=False, lens=13),
        # a partial page of one short sequence back as rows
        _read("read_37_tokens", n_lo=37, n_hi=37, kv_lo=101, kv_hi=101, R=256, page=16),
        # every token of a long-context batch back (to be expanded, or to leave for another tier)
        _read("read_long", B=16, n_lo=32768, n_hi=32768, kv_lo=32768, kv_hi=32768, lens=22),
        # one new token of a small model over a short context
        _attend("attend_tiny", H=8, R=256, page=16),
        # one decode step of 32 sequences with the 16 heads that one of several GPUs keeps
        _attend("attend_decode_16_heads", B=32, kv_lo=512, kv_hi=8192, lens=31),
        # the same step with all 128 heads
        _attend("attend_decode_128_heads", B=32, kv_lo=512, kv_hi=8192, H=128, lens=31),
        # 1 to 4 draft tokens of each of 16 long contexts checked against their caches
        _attend("attend_drafts_long", B=16, q_lo=1, q_hi=4, kv_lo=32768, kv_hi=32768, H=32, lens=32),
        # chunks of ragged lengths of 8 sequences behind cached prefixes, expanded
        _prefill("prefill_chunks", B=8, q_lo=33, q_hi=700, kv_lo=701, kv_hi=4096, H=16, lens=41),
        # a long prompt: the products are the cost
        _prefill("prefill_prompt", q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, H=16, lens=42),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "prefill"])
    B = _log_int(rng, 1, 32)
    lens = rng.randrange(1, 1 << 20)
    R = rng.choice([256, 512, 512])
    H = rng.choice([1, 2, 5, 8, 16, 20, 32, 64, 128])
    page = rng.choice([0, 8, 16, 32, 64, 128, 256])
    if op == "append":
        q_hi = _log_int(rng, 1, 4096)
        kv_hi = q_hi + _log_int(rng, 1, 8192)
        while B > 1 and (B * q_hi > 6000 or B * kv_hi > 1 << 17):
            B = (B + 1) // 2
        while H > 1 and B * q_hi * H > 1 << 17:
            H = (H + 1) // 2
        return _append("", B=B, q_lo=max(1, q_hi // 3), q_hi=q_hi, kv_lo=q_hi, kv_hi=kv_hi, H=H, R=R, page=page,
                       f32=rng.random() < 0.3, norm=rng.random() < 0.8, offset=rng.choice([0.0, 1.0]),
                       interleaved=rng.random() < 0.6, lens=lens)
    if op == "read":
        kv_hi = _log_int(rng, 16, 32768)
        while B > 1 and B * kv_hi > 1 << 18:
            B = (B + 1) // 2
        n_hi = _log_int(rng, 1, kv_hi)
        return _read("", B=B, n_lo=max(1, n_hi // 4), n_hi=n_hi, kv_lo=n_hi, kv_hi=kv_hi, R=R, page=page,
                     f32=rng.random() < 0.4, lens=lens)
    if op == "attend":
        q_hi = _log_int(rng, 1, 256)
        kv_hi = q_hi + _log_int(rng, 16, 32768)
        while q_hi > 1 and q_hi * H * kv_hi > 1 << 26:
            q_hi = (q_hi + 1) // 2
        while B > 1 and (B * q_hi * H * kv_hi > 1 << 26 or B * kv_hi > 1 << 18):
            B = (B + 1) // 2
        return _attend("", B=B, q_lo=max(1, q_hi // 4), q_hi=q_hi, kv_lo=q_hi + (kv_hi - q_hi) // 8, kv_hi=kv_hi, H=H,
                       R=R, page=page, lens=lens)
    q_hi = _log_int(rng, 1, 4096)
    kv_hi = q_hi + rng.choice([0, _log_int(rng, 1, 4096)])
    while H > 1 and q_hi * H * kv_hi > 1 << 28:
        H = (H + 1) // 2
    while B > 1 and B * q_hi * H * kv_hi > 1 << 28:
        B = (B + 1) // 2
    return _prefill("", B=B, q_lo=max(1, q_hi // 4), q_hi=q_hi, kv_lo=q_hi, kv_hi=kv_hi, H=H,
                    causal=rng.random() < 0.8, lens=lens)


def _lengths(case):
    """(new or read tokens, tokens in all) of each sequence: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    lo, hi = ("n_lo", "n_hi") if case["op"] == "read" else ("q_lo", "q_hi")
    n = [r.randint(case[lo], case[hi]) for _ in range(case["B"])]
    return n, [r.randint(max(case["kv_lo"], x), max(case["kv_hi"], x)) for x in n]


# ------------------------------------------------------------------ the inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _starts(n):
    at = [0]
    for x in n:
        at.append(at[-1] + x)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    n, kv = _lengths(case)
    op, B = case["op"], case["B"]
    total = sum(n)
    s = dict(case=case, B=B, total=total, max_q=max(n), max_kv=max(kv), start=_starts(n))
    if op == "prefill":
        H, keys = case["H"], sum(kv)
        s["kv_start"], s["keys"] = _starts(kv), keys
        s["q"] = _normal(g, total, H, HEAD + ROPE).to(torch.float16)
        # one product gives a head's key part and its value side by side
        s["kv"] = _normal(g, keys, H, 2 * HEAD).to(torch.float16)
        s["k_rope"] = _normal(g, keys, ROPE).to(torch.float16)
        s["out"] = torch.empty((total, H, HEAD), dtype=torch.float16, device=DEV)
        s["scale"] = 1.0 / math.sqrt(HEAD + ROPE)
        return s
    R, P = case["R"], case["page"]
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["page"], s["table"], s["max_pages"], s["n_pages"] = P, None, 0, 0
    if P:
        need = [-(-x // P) for x in kv]
        s["max_pages"], s["n_pages"] = max(need), sum(need) + 3
        perm = torch.randperm(s["n_pages"], generator=g, device=DEV).to(torch.int32).cpu()
        table, at = torch.full((B, s["max_pages"]), -1, dtype=torch.int32), 0
        for b in range(B):
            table[b, : need[b]] = perm[at : at + need[b]]
            at += need[b]
        s["table"] = table.to(DEV)
    shape = (s["n_pages"], P, R + ROPE) if P else (B, max(kv), R + ROPE)
    s["cap"] = shape[1]
    # an append starts from an empty cache; the others find a full one
    s["cache"] = (torch.zeros(shape, dtype=torch.float16, device=DEV) if op == "append"
                  else _normal(g, *shape).to(torch.float16))
    if op == "append":
        H, dt = case["H"], torch.float32 if case["f32"] else torch.float16
        # the projections' outputs: a token's latent vector beside its key part, and the query heads
        s["ckr"] = _normal(g, total, R + ROPE).mul_(1.5).to(dt)
        s["qh"] = _normal(g, total, H, HEAD + ROPE).to(dt)
        s["norm"] = 1.0 - case["offset"] + 0.1 * _normal(g, R) if case["norm"] else None
        inv = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device=DEV) / ROPE)
        angle = torch.arange(max(kv), dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        # the queries that attn_latent_attend takes; its first R values come from another product
        s["q_out"] = torch.zeros((total, H, R + ROPE), dtype=torch.float16, device=DEV)
    elif op == "read":
        dt = torch.float32 if case["f32"] else torch.float16
        s["c_out"] = torch.empty((total, R), dtype=dt, device=DEV)
        s["k_out"] = torch.empty((total, ROPE), dtype=dt, device=DEV)
        s["first"] = torch.tensor([a - b for a, b in zip(kv, n)], dtype=torch.int32, device=DEV)
    else:
        H = case["H"]
        s["q"] = _normal(g, total, H, R + ROPE).to(torch.float16)
        s["out"] = torch.empty((total, H, R), dtype=torch.float16, device=DEV)
        s["scale"] = 1.0 / math.sqrt(HEAD + ROPE)
    return s


# ------------------------------------------------------------------ the plain forms
def _place(s):
    """Of each packed row: its position, and its (slot, row) in the cache."""
    t = torch.arange(s["total"], device=DEV)
    b = (t[:, None] >= s["start"][None, 1:]).sum(1)
    pos = s["kv_len"][b] - s["start"][b + 1] + t
    if s["page"]:
        return pos, s["table"][b, pos // s["page"]].long(), pos % s["page"]
    return pos, b, pos


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x[..., : ROPE // 2], x[..., ROPE // 2 :]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_append(s):
    c, R = s["case"], s["case"]["R"]
    pos, slot, row = _place(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    x = s["ckr"].float()
    y = x[:, :R]
    if s["norm"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * (s["norm"] + c["offset"])
    k = _rotate(x[:, R:], cos, sin, c["interleaved"])
    s["cache"][slot, row] = torch.cat((y, k), -1).to(torch.float16)
    q = _rotate(s["qh"][..., HEAD:].float(), cos[:, None], sin[:, None], c["interleaved"])
    s["q_out"][..., R:] = q.to(torch.float16)
    return {"q": s["q_out"], "cache": s["cache"]}


def _plain_read(s):
    R = s["case"]["R"]
    _, slot, row = _place(s)
    x = s["cache"][slot, row].to(s["c_out"].dtype)
    return {"c": x[:, :R].contiguous(), "k_rope": x[:, R:].contiguous()}


def _softmax(t):
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, torch.zeros_like(p))


def _plain_attend(s):
    c, B, n = s["case"], s["B"], s["max_q"]
    H, R = c["H"], c["R"]
    j = torch.arange(s["max_kv"], device=DEV)
    if s["page"]:
        rows = s["cache"][s["table"][:, j // s["page"]].long().clamp_min(0), j % s["page"]].float()
    else:
        rows = s["cache"].float()
    rows = torch.where((j < s["kv_len"][:, None])[..., None], rows, torch.zeros((), device=DEV))
    q_len = s["start"][1:] - s["start"][:-1]
    i = torch.arange(n, device=DEV)
    at = (s["start"][:-1, None] + i).clamp_max(s["total"] - 1)
    q = s["q"].float()[at].view(B, n * H, R + ROPE)
    t = torch.matmul(q, rows.transpose(1, 2)).view(B, n, H, -1) * s["scale"]
    pos = (s["kv_len"] - q_len)[:, None] + i
    t = t.masked_fill((j > pos[..., None])[:, :, None], -math.inf)
    o = torch.matmul(_softmax(t).view(B, n * H, -1), rows[..., :R]).view(B, n, H, R)
    return o[i < q_len[:, None]].to(torch.float16)


def _plain_prefill(s):
    n, kv = _lengths(s["case"])
    outs, a, b = [], 0, 0
    for m, L in zip(n, kv):  # one sequence at a time
        q = s["q"][a : a + m].float().transpose(0, 1)
        k = s["kv"][b : b + L].float().transpose(0, 1)
        t = torch.matmul(q[..., :HEAD], k[..., :HEAD].transpose(1, 2))
        t += torch.matmul(q[..., HEAD:], s["k_rope"][b : b + L].float().T)
        t *= s["scale"]
        if s["case"]["causal"]:
            pos = L - m + torch.arange(m, device=DEV)
            t = t.masked_fill(torch.arange(L, device=DEV) > pos[:, None], -math.inf)
        outs.append(torch.matmul(_softmax(t), k[..., HEAD:]).transpose(0, 1))
        a, b = a + m, b + L
    return torch.cat(outs).to(torch.float16)


# ------------------------------------------------------------------ the library's calls
def _own_append(attn, s):
    c = s["case"]
    H, R = c["H"], c["R"]
    attn.attn_latent_append(s["ckr"], s["ckr"][:, R:], s["qh"][..., HEAD:], attn.ATTN_F32 if c["f32"] else attn.ATTN_F16,
                            s["ckr"].stride(0), s["ckr"].stride(0), s["qh"].stride(0), s["qh"].stride(1), s["norm"],
                            1e-6, c["offset"], s["cos"], s["sin"], s["cos"].shape[0], c["interleaved"], s["start"],
                            s["kv_len"], s["cache"], s["table"], s["page"], s["max_pages"], s["n_pages"], s["cap"],
                            s["B"], s["total"], H, R, ROPE, s["q_out"][..., R:], s["q_out"].stride(0),
                            s["q_out"].stride(1))
    return {"q": s["q_out"], "cache": s["cache"]}


def _own_read(attn, s):
    attn.attn_latent_read(s["cache"], s["kv_len"], s["first"], s["start"], s["table"], s["page"], s["max_pages"],
                          s["n_pages"], s["cap"], s["B"], s["total"], s["case"]["R"], ROPE, s["c_out"], s["k_out"],
                          attn.ATTN_F32 if s["c_out"].dtype == torch.float32 else attn.ATTN_F16)
    return {"c": s["c_out"], "k_rope": s["k_out"]}


def _own_attend(attn, s):
    c = s["case"]
    if "workspace" not in s:
        size = attn.attn_latent_workspace_size(s["B"], s["max_q"], c["H"], c["R"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    attn.attn_latent_attend(s["q"], s["cache"], s["start"], s["kv_len"], s["table"], s["page"], s["max_pages"],
                            s["n_pages"], s["cap"], s["B"], s["total"], s["max_q"], c["H"], c["R"], ROPE, s["scale"],
                            s["out"], None, s["workspace"], s["workspace"].numel())
    return s["out"]


def _own_prefill(attn, s):
    c, kv = s["case"], s["kv"]
    attn.attn_latent_prefill(s["q"], kv, kv[..., HEAD:], s["k_rope"], s["q"].stride(0), kv.stride(0), kv.stride(1),
                             kv.stride(0), kv.stride(1), s["k_rope"].stride(0), s["start"], s["kv_start"], s["B"],
                             s["total"], s["keys"], s["max_q"], c["H"], HEAD, ROPE, c["causal"], s["scale"], s["out"],
                             None)
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        import attention_split_kv_gb300 as attn

        calls = {"append": _own_append, "read": _own_read, "attend": _own_attend, "prefill": _own_prefill}
        return calls[op](attn, state)
    plain = {"append": _plain_append, "read": _plain_read, "attend": _plain_attend, "prefill": _plain_prefill}
    return plain[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(n, kv, causal=True):
    if not causal:
        return sum(a * L for a, L in zip(n, kv))
    return sum(a * (L - a) + a * (a + 1) // 2 for a, L in zip(n, kv))


def work(case):
    n, kv = _lengths(case)
    op, B, T = case["op"], case["B"], sum(n)
    lens = 8 * B + 4
    if op == "prefill":
        H, keys = case["H"], sum(kv)
        size = T * H * (2 * HEAD + ROPE) * 2 + keys * (2 * H * HEAD + ROPE) * 2 + 2 * (4 * B + 4)
        return {"bytes": size, "flops": 2 * _pairs(n, kv, case["causal"]) * H * (2 * HEAD + ROPE)}
    R = case["R"]
    row = R + ROPE
    if op == "append":
        e, H = 4 if case["f32"] else 2, case["H"]
        size = T * (row + H * ROPE) * (e + 2) + T * ROPE * 4 + (4 * R if case["norm"] else 0) + lens
        return {"bytes": size, "flops": T * (5 * R + 3 * (H + 1) * ROPE)}
    if op == "read":
        return {"bytes": T * row * (2 + (4 if case["f32"] else 2)) + lens, "flops": 0}
    H = case["H"]
    return {"bytes": sum(kv) * row * 2 + T * H * (row + R) * 2 + lens, "flops": 2 * _pairs(n, kv) * H * (row + R)}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turn(x, angles, interleaved):
    """Rotation of the last axis as a complex product."""
    first = torch.arange(0, ROPE, 2, device=DEV) if interleaved else torch.arange(ROPE // 2, device=DEV)
    second = first + 1 if interleaved else first + ROPE // 2
    z = torch.complex(x[..., first], x[..., second]) * angles
    y = torch.empty_like(x)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    n, kv = _lengths(case)
    if case["op"] == "prefill":
        outs, a, b = [], 0, 0
        for m, L in zip(n, kv):
            hide = torch.arange(L, device=DEV)[None] > torch.arange(L - m, L, device=DEV)[:, None]
            heads = []
            for h in range(case["H"]):
                q = s["q"][a : a + m, h].double()
                k = torch.cat((s["kv"][b : b + L, h, :HEAD], s["k_rope"][b : b + L]), -1).double()
                t = s["scale"] * (q @ k.T)
                if case["causal"]:
                    t = t.masked_fill(hide, -math.inf)
                heads.append(torch.softmax(t, -1) @ s["kv"][b : b + L, h, HEAD:].double())
            outs.append(torch.stack(heads, 1))
            a, b = a + m, b + L
        return torch.cat(outs)
    R, P = case["R"], s["page"]
    seq = torch.tensor([b for b, x in enumerate(n) for _ in range(x)], device=DEV)
    pos = torch.tensor([L - x + i for x, L in zip(n, kv) for i in range(x)], device=DEV)
    slot = s["table"].long()[seq, torch.div(pos, P, rounding_mode="floor")] if P else seq
    row = pos % P if P else pos
    if case["op"] == "append":
        turn = torch.complex(s["cos"].double(), s["sin"].double())[pos]
        x = s["ckr"].double()
        y = x[:, :R]
        if s["norm"] is not None:
            mean = torch.linalg.vector_norm(y, dim=-1, keepdim=True).square() / R
            y = y / (mean + 1e-6).sqrt() * (s["norm"].double() + case["offset"])
        cache = torch.zeros(s["cache"].shape, dtype=torch.float64, device=DEV)
        cache[slot, row] = torch.cat((y, _exact_turn(x[:, R:], turn, case["interleaved"])), -1)
        q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
        q[..., R:] = _exact_turn(s["qh"][..., HEAD:].double(), turn[:, None], case["interleaved"])
        return {"q": q, "cache": cache}
    if case["op"] == "read":
        x = s["cache"][slot, row].double()
        return {"c": x[:, :R], "k_rope": x[:, R:]}
    outs, a = [], 0
    for b, (m, L) in enumerate(zip(n, kv)):
        rows = s["cache"][s["table"][b, : -(-L // P)].long()].flatten(0, 1) if P else s["cache"][b]
        rows = rows[:L].double()
        q = s["q"][a : a + m].double()
        t = s["scale"] * torch.einsum("ihd,jd->ihj", q, rows)
        hide = torch.arange(L, device=DEV)[None] > torch.arange(L - m, L, device=DEV)[:, None]
        t = t.masked_fill(hide[:, None], -math.inf)
        outs.append(torch.einsum("ihj,jd->ihd", torch.softmax(t, -1), rows[:, :R]))
        a += m
    return torch.cat(outs)
