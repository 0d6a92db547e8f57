"""attn_latent_append and attn_latent_read against their formulas in 64 bits, the operators of
latent attention one after the other, and the failure path of their waits."""
import math

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from cache_util import tables
from latent_util import F16, F32_CHAIN, assert_within, attend_reference, prefill_reference, rows_of, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    assert attn.attn_device_status() == attn.ATTN_OK
    yield
    assert attn.attn_testing_set_waits(0, 0) == attn.ATTN_OK
    assert attn.attn_device_status() == attn.ATTN_OK


def _rotate(x, cos, sin, pos, interleaved):
    """64-bit rotation of [T, .., 64] rows at positions pos, and |a| + |b| of each value's pair."""
    x = x.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    shape = (len(pos),) + (1,) * (x.dim() - 2) + (32,)
    c, s = cos[pos].double().view(shape), sin[pos].double().view(shape)
    out, mag = (a * c - b * s, b * c + a * s), a.abs() + b.abs()
    if interleaved:
        return torch.stack(out, -1).flatten(-2), torch.stack((mag, mag), -1).flatten(-2)
    return torch.cat(out, -1), torch.cat((mag, mag), -1)


def _norm(c, w, eps, offset):
    c = c.double()
    return c * torch.rsqrt(c.square().mean(-1, keepdim=True) + eps) * (w.double() + offset)


def _round_bound(ref, mag):
    return 1.01 * (F16 * ref.abs() + 2 * F32_CHAIN * mag) + 2.0 ** -25


def _positions(q_lens, kv_lens):
    seq = [b for b, n in enumerate(q_lens) for _ in range(n)]
    pos = [L - n + i for n, L in zip(q_lens, kv_lens) for i in range(n)]
    return seq, pos


def _place(case, b, p):
    return (int(case.page_table[b, p // case.page_size]), p % case.page_size) if case.page_size else (b, p)


def _append_case(q_lens, kv_lens, R, page, H, dtype, seed=1, cap=0, tail=2, n_pos=0):
    case = si.make_latent_case(kv_lens, R, seed, page_size=page, cap=cap, fill=77.0, device="cuda")
    T = sum(q_lens) + tail
    g = torch.Generator(device="cuda").manual_seed(seed)
    ckr = (torch.randn(T, R + 64, generator=g, device="cuda") * 1.5).to(dtype)
    qh = torch.randn(T, max(H, 1), 192, generator=g, device="cuda").to(dtype)
    cos, sin = (t.cuda() for t in tables(n_pos or max(kv_lens + [1]), 64))
    w = 0.1 * torch.randn(R, generator=g, device="cuda")
    return case, ckr, qh, cos, sin, w


def _check_append(case, ckr, qh, cos, sin, w, q_lens, kv_lens, R, H, offset, interleaved, q_out=None, skip=()):
    T = sum(q_lens)
    q_rope = qh[..., 128:] if H else None
    packed = torch.full((ckr.shape[0], max(H, 1), R + 64), 7.0, dtype=torch.float16, device="cuda")
    out = q_out if q_out is not None else packed[..., R:] if H else None
    src = qh.clone()
    attn.latent_append(case, ckr[:, :R], ckr[:, R:], starts(q_lens, "cuda"), q_rope=q_rope, c_norm=w, norm_offset=offset,
                       rope_cos=cos, rope_sin=sin, rope_interleaved=interleaved, q_out=out)
    seq, pos = _positions(q_lens, kv_lens)
    live = [t for t in range(T) if pos[t] >= 0 and t not in skip]
    at = torch.tensor([pos[t] for t in live], device="cuda", dtype=torch.long)
    rows = torch.tensor(live, device="cuda", dtype=torch.long)
    c = ckr[rows, :R].double() if w is None else _norm(ckr[rows, :R], w, 1e-6, offset)
    k, kmag = (ckr[rows, R:].double(), ckr[rows, R:].double().abs()) if cos is None else _rotate(ckr[rows, R:], cos, sin, at, interleaved)
    ref, mag = torch.cat((c, k), -1), torch.cat((c.abs(), kmag), -1)
    places = [_place(case, seq[t], pos[t]) for t in live]
    if live:
        s, r = (torch.tensor(x, device="cuda") for x in zip(*places))
        assert_within(case.cache[s, r], ref, _round_bound(ref, mag), "cache rows")
        case.cache[s, r] = 77.0
    assert bool((case.cache == 77).all()), "rows of no new token were written"
    if H:
        ref, mag = (src[rows, :, 128:].double(),) * 2 if cos is None else _rotate(src[rows, :, 128:], cos, sin, at, interleaved)
        assert_within(out[rows], ref, _round_bound(ref, mag.abs()), "q")
        rest = torch.ones(ckr.shape[0], dtype=torch.bool, device="cuda")
        rest[rows] = False
        if q_out is None:
            assert bool((packed[..., :R] == 7).all()) and bool((packed[rest] == 7).all()), "q_out beside the heads' parts"
    assert torch.equal(src[..., :128], qh[..., :128])


LENS = [([1], [1]), ([1] * 5, [1, 64, 65, 300, 17]), ([3, 0, 40, 1], [3, 9, 200, 128]), ([400, 129], [500, 129])]


@pytest.mark.parametrize("q_lens,kv_lens", LENS, ids=str)
@pytest.mark.parametrize("R,page,H", [(512, 64, 16), (512, 0, 128), (256, 8, 5), (256, 0, 1), (512, 256, 0), (256, 1024, 3)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=["f16", "f32"])
@pytest.mark.parametrize("interleaved", [True, False])
def test_append(q_lens, kv_lens, R, page, H, dtype, interleaved):
    case, ckr, qh, cos, sin, w = _append_case(q_lens, kv_lens, R, page, H, dtype)
    offset = 1.0 if interleaved else 0.0
    _check_append(case, ckr, qh, cos, sin, w + (1.0 - offset), q_lens, kv_lens, R, H, offset, interleaved)


@pytest.mark.parametrize("rope,norm", [(False, True), (True, False), (False, False)])
def test_append_without_norm_or_rotation(rope, norm):
    q_lens, kv_lens = [2, 33], [50, 33]
    case, ckr, qh, cos, sin, w = _append_case(q_lens, kv_lens, 512, 16, 8, torch.float32)
    _check_append(case, ckr, qh, cos if rope else None, sin if rope else None, w + 1 if norm else None, q_lens, kv_lens,
                  512, 8, 0.0, True)


def test_append_rotates_q_in_place():
    q_lens, kv_lens = [5, 1], [70, 33]
    case, ckr, qh, cos, sin, w = _append_case(q_lens, kv_lens, 256, 16, 12, torch.float16)
    _check_append(case, ckr, qh, cos, sin, w + 1, q_lens, kv_lens, 256, 12, 0.0, False, q_out=qh[..., 128:])


def test_append_leaves_out_a_padded_batchs_rows():
    # sequences of length 0, and more rows than tokens: negative positions are no tokens
    q_lens, kv_lens = [2, 3, 1], [0, 1, 40]
    case, ckr, qh, cos, sin, w = _append_case(q_lens, kv_lens, 512, 16, 4, torch.float16)
    _check_append(case, ckr, qh, cos, sin, w + 1, q_lens, kv_lens, 512, 4, 0.0, True)


@pytest.mark.parametrize("what", ["capacity", "tables", "page"])
def test_append_reports_what_it_leaves_out(what):
    q_lens, kv_lens = [3, 2], [34, 20]
    page = 16 if what == "page" else 0
    case, ckr, qh, cos, sin, w = _append_case(q_lens, kv_lens, 256, page, 4, torch.float16)
    skip = ()
    if what == "capacity":     # (the contiguous cache holds 33 tokens a sequence)
        case.cache = case.cache[:, :33].contiguous()
        skip = (2,)
    elif what == "tables":
        cos, sin = cos[:33].contiguous(), sin[:33].contiguous()
        skip = (2,)
    else:
        case.page_table[1, 1] = case.cache.shape[0]   # positions 18, 19 of sequence 1
    if what != "page":
        _check_append(case, ckr, qh, cos, sin, w + 1, q_lens, kv_lens, 256, 4, 0.0, True, skip=skip)
    else:
        before = case.cache.clone()
        out = attn.latent_append(case, ckr[:, :256], ckr[:, 256:], starts(q_lens, "cuda"), q_rope=qh[..., 128:], rope_cos=cos,
                                 rope_sin=sin)
        ref, mag = _rotate(qh[:5, :, 128:], cos, sin, torch.tensor([31, 32, 33, 18, 19], device="cuda"), True)
        assert_within(out[:5], ref, _round_bound(ref, mag))   # q is written all the same
        changed = (case.cache != before).flatten(1).any(1).nonzero()[:, 0].tolist()
        assert sorted(changed) == sorted({int(case.page_table[0, 1]), int(case.page_table[0, 2])})
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS


@pytest.mark.parametrize("R,page", [(512, 64), (512, 0), (256, 8), (256, 1024)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kv_lens,first,n", [
    ([1], [0], [1]), ([37, 0, 300], [0, 0, 5], [37, 0, 295]), ([100, 50], [90, 0], [20, 51]), ([64, 9], [-3, 2], [10, 3]),
    ([3000, 2000], [0, 1], [3000, 1999])], ids=str)
def test_read(R, page, f32, kv_lens, first, n):
    case = si.make_latent_case(kv_lens, R, 3, page_size=page, device="cuda")
    T = sum(n)
    st = starts(n, "cuda")
    dt = torch.float32 if f32 else torch.float16
    c = torch.full((T + 3, R), 7.0, dtype=dt, device="cuda")
    k = torch.full((T + 3, 64), 7.0, dtype=dt, device="cuda")
    rows, cap = (page, case.max_pages) if page else (0, 0)
    attn.attn_latent_read(case.cache, case.kv_len, torch.tensor(first, dtype=torch.int32, device="cuda"), st, case.page_table,
                          rows, cap, case.cache.shape[0], case.cache.shape[1], case.batch, T + 3, R, 64, c, k,
                          attn.ATTN_F32 if f32 else attn.ATTN_F16)
    ref = torch.zeros(T, R + 64, dtype=torch.float64, device="cuda")
    at = 0
    for b, (a, m, L) in enumerate(zip(first, n, kv_lens)):
        x = rows_of(case, b, L)
        lo, hi = max(a, 0), min(a + m, L)
        if hi > lo:
            ref[at + lo - a: at + hi - a] = x[lo:hi]
        at += m
    assert torch.equal(c[:T].double(), ref[:, :R]) and torch.equal(k[:T].double(), ref[:, R:])
    assert bool((c[T:] == 7).all()) and bool((k[T:] == 7).all())


def test_read_reports_a_page_outside_the_pool():
    case = si.make_latent_case([100], 512, 3, page_size=16, device="cuda")
    case.page_table[0, 2] = -1
    c, k = attn.latent_read(case, starts([100], "cuda"), 100, out_f32=True)
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    assert bool((c[32:48] == 0).all()) and bool((k[32:48] == 0).all())
    assert torch.equal(torch.cat((c, k), 1).double(), rows_of(case, 0, 100))


def test_offsets_past_32_bits():
    pages = (1 << 32) // (64 * 576) + 8
    case = si.LatentCase(cache=torch.zeros(pages, 64, 576, dtype=torch.float16, device="cuda"),
                         kv_len=torch.tensor([70], dtype=torch.int32, device="cuda"), batch=1,
                         page_table=torch.tensor([[pages - 3, pages - 1]], dtype=torch.int32, device="cuda"), page_size=64,
                         max_pages=2)
    x = torch.randn(70, 576, device="cuda").half()
    attn.latent_append(case, x[:, :512], x[:, 512:], starts([70], "cuda"))
    assert torch.equal(case.cache[pages - 3], x[:64]) and torch.equal(case.cache[pages - 1, :6], x[64:])
    c, k = attn.latent_read(case, starts([70], "cuda"), 70)
    assert torch.equal(torch.cat((c, k), 1), x)


# ------------------------------------------------------------------ together, as a model uses them
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("R,H", [(512, 16), (256, 5)])
def test_prompt_then_chunk_then_tokens_in_both_forms(R, H, page):
    """Tokens appended as a prompt, a chunk and single steps; each step attended in the absorbed form
    (queries times W_uk) and in the expanded one (cached rows times W_uk, W_uv): the absorbed output
    times W_uv is the expanded output, up to the roundings both make."""
    g = torch.Generator(device="cuda").manual_seed(R + H + page)
    B, scale = 2, 1.0 / math.sqrt(192.0)
    w_uk = torch.randn(H, 128, R, generator=g, device="cuda").double() / math.sqrt(R)
    w_uv = torch.randn(H, R, 128, generator=g, device="cuda").double() / math.sqrt(R)
    steps = [[70, 33], [20, 1], [1, 1], [1, 1]]
    total = [sum(s[b] for s in steps) for b in range(B)]
    case = si.make_latent_case(total, R, 5, page_size=page, fill=float("nan"), device="cuda")
    cos, sin = (t.cuda() for t in tables(max(total), 64))
    w = 1.0 + 0.1 * torch.randn(R, generator=g, device="cuda")
    done = [0, 0]
    for n in steps:
        T = sum(n)
        done = [d + x for d, x in zip(done, n)]
        case.kv_len.copy_(torch.tensor(done, dtype=torch.int32))
        start = starts(n, "cuda")
        proj = torch.randn(T, R + 64, generator=g, device="cuda").half()
        q = torch.randn(T, H, 192, generator=g, device="cuda").half()
        # the projections' absorbed query, and its rotated part written beside it by the append
        qa = torch.empty(T, H, R + 64, dtype=torch.float16, device="cuda")
        qa[..., :R] = torch.einsum("thd,hdr->thr", q[..., :128].double(), w_uk).half()
        attn.latent_append(case, proj[:, :R], proj[:, R:], start, q_rope=q[..., 128:], c_norm=w, rope_cos=cos, rope_sin=sin,
                           q_out=qa[..., R:])
        q[..., 128:] = qa[..., R:]
        oa = attn.latent_attend(case, qa, start, max(n))
        ref, _, bound = attend_reference(case, qa, n)
        assert_within(oa, ref, bound, "absorbed")
        kv_start = starts(done, "cuda")
        c, r = attn.latent_read(case, kv_start, sum(done))
        k = torch.einsum("tr,hdr->thd", c.double(), w_uk).half()
        v = torch.einsum("tr,hrd->thd", c.double(), w_uv).half()
        oe = attn.latent_prefill(q, k, v, r, start, kv_start, max(n), scale)
        ref_e, _, bound_e = prefill_reference(q, k, v, r, n, done, scale)
        assert_within(oe, ref_e, bound_e, "expanded")
        # Both forms against each other: beside the kernels' own errors, the absorbed query, the
        # expanded keys and the values are each rounded to f16 (2^-11 of N(0, 1)-sized values), which
        # moves a logit by about 2^-11 sqrt(192) |q| |k| scale / sqrt(192) at random, under 2^-7 at
        # most here, and an output by that share of the values' spread (under 4).
        a = torch.einsum("thr,hrd->thd", oa.double(), w_uv)
        assert float((a - oe.double()).abs().max()) <= 4 * 2.0 ** -7


@pytest.mark.parametrize("R,H", [(512, 16), (512, 128), (256, 20)])
def test_attend_timeout_reports_and_recovers(R, H):
    case = si.make_latent_case([700, 3, 1300], R, 9, page_size=16, device="cuda")
    q = si.f16_normal((3, H, R + 64), 4, "cuda")
    start = starts([1, 1, 1], "cuda")
    assert attn.attn_testing_set_waits(20_000_000, 1) == attn.ATTN_OK
    try:
        attn.latent_attend(case, q, start, 1)
        assert attn.attn_device_status() == attn.ATTN_ETIMEOUT
    finally:
        assert attn.attn_testing_set_waits(0, 0) == attn.ATTN_OK
    ref, _, bound = attend_reference(case, q, [1, 1, 1])
    assert_within(attn.latent_attend(case, q, start, 1), ref, bound)


@pytest.mark.parametrize("n", [100, 300, 900])
def test_prefill_timeout_reports_and_recovers(n):
    q, k, v = (si.f16_normal((n, 4, d), d, "cuda") for d in (192, 128, 128))
    r = si.f16_normal((n, 64), 6, "cuda")
    st = starts([n], "cuda")
    assert attn.attn_testing_set_waits(20_000_000, 1) == attn.ATTN_OK
    try:
        attn.latent_prefill(q, k, v, r, st, st, n, 0.07)
        assert attn.attn_device_status() == attn.ATTN_ETIMEOUT
    finally:
        assert attn.attn_testing_set_waits(0, 0) == attn.ATTN_OK
    ref, _, bound = prefill_reference(q, k, v, r, [n], [n], 0.07)
    assert_within(attn.latent_prefill(q, k, v, r, st, st, n, 0.07), ref, bound)


@pytest.mark.parametrize("what", ["append", "read", "attend", "prefill"])
def test_calls_on_another_stream(what):
    case = si.make_latent_case([300, 40], 512, 9, page_size=16, device="cuda")
    start = starts([2, 1], "cuda")
    q = si.f16_normal((3, 16, 576), 4, "cuda")
    kv = si.f16_normal((340, 16, 256), 5, "cuda")
    rows = si.f16_normal((3, 576), 6, "cuda")
    kv_start = starts([300, 40], "cuda")
    calls = {
        "append": lambda **s: (attn.latent_append(case, rows[:, :512], rows[:, 512:], start, q_rope=q[..., 512:], **s), case.cache),
        "read": lambda **s: attn.latent_read(case, kv_start, 340, **s),
        "attend": lambda **s: (attn.latent_attend(case, q, start, 2, **s),),
        "prefill": lambda **s: (attn.latent_prefill(q[..., :192].contiguous(), kv[..., :128], kv[..., 128:],
                                                    q[0, 0].new_zeros(340, 64), start, kv_start, 2, 0.07, **s),),
    }
    want = [t.clone() for t in calls[what]()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        got = calls[what](stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
