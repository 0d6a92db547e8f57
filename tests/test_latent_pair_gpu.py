"""attn_latent_attend in pairs of CTAs: many rows of 512 latent values over caches that can be long."""
import math
import os
import subprocess
import sys

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from latent_util import assert_lse, assert_within, attend_reference, starts

pytestmark = pytest.mark.gpu

# tokens and sequences for which single tokens of more than 64 rows, and chunks of more than 128, are taken in pairs
ROOM, SEQS = 4864, 16


@pytest.fixture(autouse=True)
def _status():
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _case(q_lens, kv_lens, H, page, seed=1, tail=0, R=512):
    # (sequences without new tokens between and behind the others)
    more = max(SEQS - len(q_lens), 0)
    q_lens, kv_lens = q_lens[:1] + [0] * (more // 2) + q_lens[1:] + [0] * (more - more // 2), \
        kv_lens[:1] + [7] * (more // 2) + kv_lens[1:] + [7] * (more - more // 2)
    case = si.make_latent_case(kv_lens, R, seed, page_size=page, cap=ROOM, device="cuda")
    return case, si.f16_normal((sum(q_lens) + tail, H, R + 64), seed + 100, "cuda"), q_lens


def _check(case, q, q_lens, what="", max_q=None):
    T = sum(q_lens)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = torch.full((*q.shape[:2], 512), 7.0, dtype=torch.float16, device="cuda")
    top = max_q if max_q is not None else max(q_lens)
    attn.latent_attend(case, q, starts(q_lens, "cuda"), top, out=out, lse_out=lse)
    ref, ref_lse, bound = attend_reference(case, q[:T], q_lens, max_q)
    done = torch.cat([torch.arange(n, device="cuda") < top for n in q_lens])
    assert bool((out[T:] == 7).all()) and bool((out[:T][~done] == 7).all()), "rows of no token were written"
    assert bool((lse[T:] == 7).all())
    assert_within(out[:T][done], ref[done], bound[done], what)
    assert_lse(lse[:T][done], ref_lse[done], what)


@pytest.mark.parametrize("q_lens,kv_lens,H", [
    ([1, 1], [2500, 3], 65), ([1], [900], 127), ([1, 1, 1], [64, 700, 0], 129), ([1, 1], [4864, 40], 300), ([1], [300], 1100),
    ([1] * 5, [1, 63, 64, 65, 128], 128), ([1] * 20, list(range(100, 2100, 100)), 128),
    ([3, 1, 4], [700, 20, 3000], 50), ([9, 2], [1500, 2], 16), ([130], [130], 1), ([2, 3], [65, 1000], 100),
    ([1, 0, 3, 1], [64, 0, 130, 5], 50), ([40, 7], [40, 555], 17),
], ids=str)
@pytest.mark.parametrize("page", [0, 8, 16, 64, 256])
def test_against_the_formula(q_lens, kv_lens, H, page):
    case, q, q_lens = _case(q_lens, kv_lens, H, page, tail=1)
    _check(case, q, q_lens)


def test_more_tokens_than_cached_and_a_chunk_that_is_cut():
    case, q, q_lens = _case([9, 4], [5, 300], 20, 16)
    _check(case, q, q_lens)
    case, q, q_lens = _case([9, 4], [500, 300], 40, 16)
    _check(case, q, q_lens, max_q=6)


@pytest.mark.parametrize("page", [0, 16])
def test_what_no_query_keeps_is_never_used(page):
    case, q, q_lens = _case([1, 2, 1], [70, 200, 1], 80, page)
    ref, _, bound = attend_reference(case, q, q_lens)
    slots = case.cache.shape[0]
    if page:
        used = torch.zeros(slots, page, dtype=torch.bool, device="cuda")
        for b, n in enumerate(case.kv_len.tolist()):
            for t in range(n):
                used[case.page_table[b, t // page], t % page] = True
    else:
        used = torch.arange(ROOM, device="cuda")[None] < case.kv_len[:, None]
    case.cache[~used] = math.nan
    assert_within(attn.latent_attend(case, q, starts(q_lens, "cuda"), 2), ref, bound)


def test_page_ids_outside_the_pool_read_as_zeros_and_are_reported():
    case, q, q_lens = _case([1, 1], [700, 300], 128, 64)
    first, second = [b for b, n in enumerate(q_lens) if n]
    case.page_table[first, 3] = case.cache.shape[0]
    case.page_table[second, 0] = -5
    lse = torch.empty(q.shape[:2], device="cuda")
    out = attn.latent_attend(case, q, starts(q_lens, "cuda"), 1, lse_out=lse)
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    ref, ref_lse, bound = attend_reference(case, q, q_lens)
    assert_within(out, ref, bound)
    assert_lse(lse, ref_lse)


@pytest.mark.parametrize("H,n", [(128, 1), (50, 3)])
@pytest.mark.parametrize("step", [0.5, 12.0])
def test_logits_that_keep_growing(H, n, step):
    # keys of one direction, growing along the sequence, and queries along it and against it in turn: the
    # maxima of some rows move in (nearly) every tile, of others never
    L = 2000
    case, q, q_lens = _case([n, 1], [L, 777], H, 0)
    g = torch.Generator(device="cuda").manual_seed(3)
    d = torch.randn(576, generator=g, device="cuda")
    d /= d.norm()
    for b, (m, length) in enumerate(zip(q_lens, case.kv_len.tolist())):
        rows = torch.arange(length, device="cuda")[:, None] / 128.0 * step / (case.scale * 24.0) * d
        case.cache[b, :length] = (rows + 0.3 * torch.randn(length, 576, generator=g, device="cuda")).half()
    along = torch.where(torch.arange(H, device="cuda") % 3 == 1, -24.0, 24.0)[None, :, None] * d
    q.copy_((along + 0.2 * torch.randn(q.shape, generator=g, device="cuda")).half())
    _check(case, q, q_lens)


def test_a_query_of_nan_or_infinity_stays_in_its_row():
    # (of either CTA's half of the rows and of the values, and of the rotated part)
    case, q, q_lens = _case([1, 3], [700, 300], 100, 16)
    ref, _, bound = attend_reference(case, q, q_lens)
    q[0, 5, 3], q[0, 80, 300], q[2, 30, 540], q[3, 99, 511] = math.nan, math.inf, math.nan, math.nan
    out = attn.latent_attend(case, q, starts(q_lens, "cuda"), 3)
    good = torch.ones(4, 100, dtype=torch.bool)
    for t, h in ((0, 5), (0, 80), (2, 30), (3, 99)):
        assert bool(out[t, h].isnan().all())
        good[t, h] = False
    assert_within(out[good], ref[good], bound[good])


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-20])
def test_scales(scale):
    case, q, q_lens = _case([1, 2], [200, 333], 70, 64)
    case.scale = scale
    _check(case, q, q_lens)


def test_again_and_again():
    # the same bits from call to call, and from a captured one between others; then with other lengths
    case, q, q_lens = _case([1, 4, 2, 1], [3000, 700, 70, 4800], 64, 32)
    start = starts(q_lens, "cuda")
    first = attn.latent_attend(case, q, start, 4)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(first)
    with torch.cuda.graph(graph):
        attn.latent_attend(case, q, start, 4, out=out)
        attn.latent_attend(case, q, start, 4, out=out)
    for _ in range(20):
        assert torch.equal(attn.latent_attend(case, q, start, 4), first)
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    case.kv_len.sub_(torch.tensor([n > 1 for n in case.kv_len.tolist()], dtype=torch.int32, device="cuda"))
    graph.replay()
    ref, _, bound = attend_reference(case, q, q_lens)
    assert_within(out, ref, bound)


def test_two_streams_at_once():
    cases = [_case([1, 2], [4000 + i, 900], 100, 16, seed=i) for i in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    start = starts(cases[0][2], "cuda")
    refs = [attend_reference(c, q, n) for c, q, n in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for (c, q, _), s in zip(cases, streams):
            outs.append(attn.latent_attend(c, q, start, 2, stream=s))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert_within(out, refs[i % 2][0], refs[i % 2][2])


def test_offsets_past_32_bits():
    case, q, q_lens = _case([1, 2], [150, 70], 70, 64)
    pages = (1 << 32) // (64 * 576) + 8
    pool = torch.zeros(pages, 64, 576, dtype=torch.float16, device="cuda")
    far = case.page_table.clone()
    used = case.page_table >= 0
    far[used] = pages - 1 - case.page_table[used]
    pool[far[used].long()] = case.cache[case.page_table[used].long()]
    ref, _, bound = attend_reference(case, q, q_lens)
    case.cache, case.page_table = pool, far
    assert_within(attn.latent_attend(case, q, starts(q_lens, "cuda"), 2), ref, bound)


def test_a_timeout_is_reported_and_the_next_call_is_right():
    case, q, q_lens = _case([1, 3], [700, 1300], 128, 16)
    start = starts(q_lens, "cuda")
    assert attn.attn_testing_set_waits(20_000_000, 1) == attn.ATTN_OK
    try:
        attn.latent_attend(case, q, start, 3)
        assert attn.attn_device_status() == attn.ATTN_ETIMEOUT
    finally:
        assert attn.attn_testing_set_waits(0, 0) == attn.ATTN_OK
    ref, _, bound = attend_reference(case, q, q_lens)
    assert_within(attn.latent_attend(case, q, start, 3), ref, bound)


TRACE = r"""
import torch
import attention_split_kv_gb300 as attn
import seeded_inputs as si
from tests.latent_util import starts
attn.load()
for B, cap, H, R, n in ((16, 4864, 128, 512, 1), (16, 4800, 128, 512, 1), (15, 4864, 128, 512, 1), (16, 4864, 128, 256, 1),
                        (32, 4864, 64, 512, 1), (16, 4864, 300, 512, 1), (16, 4864, 32, 512, 4), (16, 4864, 32, 512, 5)):
    case = si.make_latent_case([9] * B, R, 1, page_size=16, cap=cap, device="cuda")
    attn.latent_attend(case, si.f16_normal((B * n, H, R + 64), 2, "cuda"), starts([n] * B, "cuda"), n)
torch.cuda.synchronize()
assert attn.attn_device_status() == attn.ATTN_OK
"""


def test_trace_names_the_form():
    # many rows of 512 values over caches that can be long: in pairs; else alone
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", TRACE], cwd=root, env=dict(os.environ, ATTN_TRACE="1"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [x for x in r.stderr.splitlines() if x.startswith("[libattn]")]
    assert ["latent_pair_kernel " in x for x in lines] == [True, False, False, False, False, True, False, True]
    assert "side=1" in lines[0] and "side=3" in lines[5]


def test_steps_of_append_and_attend():
    # each step's q and cache rows are written by the append directly before, q in place of the last step's
    H, B = 128, 16
    lens = [3, 700, 64, 1500] * 4
    room = si.make_latent_case([n + 8 for n in lens], 512, 3, page_size=32, cap=ROOM, device="cuda")
    start = starts([1] * B, "cuda")
    q = si.f16_normal((B, H, 576), 9, "cuda")
    outs = []
    for step in range(6):
        c = si.f16_normal((B, 512), 20 + step, "cuda")
        kr, qr = si.f16_normal((B, 64), 40 + step, "cuda"), si.f16_normal((B, H, 64), 60 + step, "cuda")
        kv_len = torch.tensor([n + 1 + step for n in lens], dtype=torch.int32, device="cuda")
        attn.latent_append(room, c, kr, start, kv_len=kv_len, q_rope=qr, q_out=q[..., 512:])
        outs.append((attn.latent_attend(room, q, start, 1, kv_len=kv_len), q.clone(), kv_len, c, kr, qr))
    for out, used, kv_len, c, kr, qr in outs:
        assert torch.equal(used[..., 512:], qr)
        room.kv_len = kv_len
        ref, _, bound = attend_reference(room, used, [1] * B)
        assert_within(out, ref, bound)
