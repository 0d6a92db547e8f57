"""attn_latent_attend (the absorbed form of latent attention) against its formula in 64 bits."""
import math

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from latent_util import assert_lse, assert_within, attend_reference, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    assert attn.attn_device_status() == attn.ATTN_OK
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _case(q_lens, kv_lens, H, R, page, seed=1, cap=0, tail=0):
    case = si.make_latent_case(kv_lens, R, seed, page_size=page, cap=cap, device="cuda")
    q = si.f16_normal((sum(q_lens) + tail, H, R + 64), seed + 100, "cuda")
    return case, q, starts(q_lens, "cuda")


def _check(case, q, q_lens, what="", max_q=None):
    T = sum(q_lens)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = torch.full((*q.shape[:2], q.shape[2] - 64), 7.0, dtype=torch.float16, device="cuda")
    top = max_q if max_q is not None else max(q_lens)
    attn.latent_attend(case, q, starts(q_lens, "cuda"), top, out=out, lse_out=lse)
    ref, ref_lse, bound = attend_reference(case, q[:T], q_lens, max_q)
    done = torch.cat([torch.arange(n, device="cuda") < top for n in q_lens])
    assert bool((out[T:] == 7).all()) and bool((out[:T][~done] == 7).all()), "rows of no token were written"
    assert bool((lse[T:] == 7).all())
    assert_within(out[:T][done], ref[done], bound[done], what)
    assert_lse(lse[:T][done], ref_lse[done], what)
    return out


LENS = [
    ([1], [1]), ([1], [128]), ([1], [129]), ([1], [2500]),
    ([1] * 5, [1, 127, 128, 700, 2049]),
    ([1, 0, 3, 1], [64, 0, 130, 5]),
    ([3, 5, 2], [300, 5, 1023]),
    ([40, 7], [40, 555]),
]


@pytest.mark.parametrize("q_lens,kv_lens", LENS, ids=str)
@pytest.mark.parametrize("H", [1, 5, 16, 20, 64, 128])
@pytest.mark.parametrize("R,page", [(512, 64), (512, 0), (256, 16), (256, 0)])
def test_against_the_formula(q_lens, kv_lens, H, R, page):
    case, q, _ = _case(q_lens, kv_lens, H, R, page, tail=2)
    _check(case, q, q_lens)


@pytest.mark.parametrize("page", [8, 32, 128, 256, 1024])
@pytest.mark.parametrize("R", [256, 512])
def test_page_sizes(page, R):
    case, q, _ = _case([2, 1, 9], [700, 1500, 9], 16, R, page)
    _check(case, q, [2, 1, 9])
    flat = si.make_latent_case([700, 1500, 9], R, 1, device="cuda")
    for b, n in enumerate([700, 1500, 9]):   # the same rows without pages: the same bits
        ids = case.page_table[b, : -(-n // page)].long()
        flat.cache[b, :n] = case.cache[ids].flatten(0, 1)[:n]
    a, b = (attn.latent_attend(c, q, starts([2, 1, 9], "cuda"), 9) for c in (case, flat))
    assert torch.equal(a, b)


@pytest.mark.parametrize("page", [0, 16, 256])
def test_what_no_query_keeps_is_never_used(page):
    # pages that end inside a tile, slots past the sequence, pages of no sequence: all NaN
    kv, q_lens = [1, 130, 517, 64], [1, 2, 4, 1]
    case, q, _ = _case(q_lens, kv, 16, 512, page, cap=600)
    clean = case.cache.clone()
    case.cache.fill_(math.nan)
    for b, n in enumerate(kv):
        for p in range(n):
            at = (b, p) if not page else (int(case.page_table[b, p // page]), p % page)
            case.cache[at] = clean[at]
    _check(case, q, q_lens)


def test_rows_without_keys_and_padded_batches():
    # more new tokens than cached ones (the first keep nothing), no cached token at all, no new token
    case, q, _ = _case([4, 1, 0, 2], [2, 0, 9, -3], 20, 256, 16)
    out = _check(case, q, [4, 1, 0, 2])
    assert bool((out[:2] == 0).all()) and bool((out[4:] == 0).all())


def test_lengths_above_the_capacity_are_clamped():
    case, q, _ = _case([1, 2], [200, 130], 8, 256, 0)
    case.kv_len = torch.tensor([1000, 130], dtype=torch.int32, device="cuda")
    _check(case, q, [1, 2])


def test_a_chunk_longer_than_max_q_is_cut():
    case, q, _ = _case([9, 3], [300, 200], 16, 512, 64)
    _check(case, q, [9, 3], max_q=4)


def test_page_ids_outside_the_pool_read_as_zeros_and_are_reported():
    case, q, _ = _case([1, 2], [700, 300], 16, 512, 64)
    case.page_table[0, 3] = case.cache.shape[0]
    case.page_table[1, 0] = -5
    lse = torch.empty(q.shape[:2], device="cuda")
    out = attn.latent_attend(case, q, starts([1, 2], "cuda"), 2, lse_out=lse)
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    ref, ref_lse, bound = attend_reference(case, q, [1, 2])
    assert_within(out, ref, bound)
    assert_lse(lse, ref_lse)


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("step", [0.5, 12.0])
def test_logits_that_keep_growing(H, step):
    # keys of one direction, growing along the sequence: the running maximum moves in (nearly) every
    # tile; the last tokens then carry the mass
    L = 2000
    case, q, _ = _case([1, 3], [L, 777], H, 512, 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    d = torch.randn(576, generator=g, device="cuda")
    d /= d.norm()
    for b, n in enumerate([L, 777]):
        rows = torch.arange(n, device="cuda")[:, None] / 128.0 * step / (case.scale * 24.0) * d
        rows = rows + 0.3 * torch.randn(n, 576, generator=g, device="cuda")
        ids = case.page_table[b, : -(-n // 64)].long()
        pad = torch.zeros(len(ids) * 64, 576, device="cuda")
        pad[:n] = rows
        case.cache[ids] = pad.view(-1, 64, 576).to(torch.float16)
    q.copy_((24.0 * d + 0.2 * torch.randn(q.shape, generator=g, device="cuda")).to(torch.float16))
    _check(case, q, [1, 3])


def test_one_dominant_key_gives_its_value():
    case, q, _ = _case([1], [1000], 16, 512, 16)
    where = int(case.page_table[0, 333 // 16]), 333 % 16
    row = case.cache[where]
    q[:] = (row.float() * 4).to(torch.float16)
    out = attn.latent_attend(case, q, starts([1], "cuda"), 1)
    assert torch.equal(out, row[:512].expand_as(out))


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_scales(scale):
    case, q, _ = _case([1, 4], [300, 1000], 16, 256, 64)
    case.scale = scale
    _check(case, q, [1, 4])


def test_a_nan_query_stays_in_its_row():
    case, q, _ = _case([1, 1], [300, 1000], 20, 512, 64)
    q[0, 3, 5] = math.nan
    q[1, 7, 575] = math.inf
    out = attn.latent_attend(case, q, starts([1, 1], "cuda"), 1)
    assert bool(out[0, 3].isnan().all()) and bool(out[1, 7].isnan().all())
    good = torch.ones(2, 20, dtype=torch.bool)
    good[0, 3] = good[1, 7] = False
    ref, _, bound = attend_reference(case, torch.nan_to_num(q, 0.0, 0.0, 0.0), [1, 1])
    assert_within(out[good], ref[good], bound[good])


def test_long_contexts_split_over_all_ctas():
    case, q, _ = _case([1, 2], [40000, 20001], 32, 512, 64)
    _check(case, q, [1, 2])


def test_many_sequences():
    kv = [(37 * i) % 300 for i in range(700)]
    case, q, _ = _case([1] * 700, kv, 8, 256, 16)
    _check(case, q, [1] * 700)


def test_the_same_call_gives_the_same_bits():
    case, q, start = _case([1, 3, 1], [3000, 700, 9000], 128, 512, 64)
    a = attn.latent_attend(case, q, start, 3)
    for _ in range(3):
        assert torch.equal(a, attn.latent_attend(case, q, start, 3))


def test_captured_and_replayed_with_other_lengths():
    case, q, start = _case([1] * 4, [900, 20, 300, 4000], 16, 512, 64)
    ws = torch.empty(attn.attn_latent_workspace_size(4, 1, 16, 512), dtype=torch.uint8, device="cuda")
    out = torch.empty(4, 16, 512, dtype=torch.float16, device="cuda")
    attn.latent_attend(case, q, start, 1, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.latent_attend(case, q, start, 1, out=out, workspace=ws)
    for kv in ([900, 20, 300, 4000], [1, 20, 0, 3999], [130, 1, 299, 7]):
        case.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, device="cuda"))
        graph.replay()
        ref, _, bound = attend_reference(case, q, [1] * 4)
        assert_within(out, ref, bound, str(kv))


def test_offsets_past_32_bits():
    # rows whose element offset needs 33 bits: a pool of 2^32 elements, three of its last pages used
    case, q, start = _case([1, 2], [150, 70], 16, 512, 64)
    pages = (1 << 32) // (64 * 576) + 8
    pool = torch.zeros(pages, 64, 576, dtype=torch.float16, device="cuda")
    far = case.page_table.clone()
    used = case.page_table >= 0
    far[used] = pages - 1 - case.page_table[used]
    pool[far[used].long()] = case.cache[case.page_table[used].long()]
    ref, _, bound = attend_reference(case, q, [1, 2])
    case.cache, case.page_table = pool, far
    assert_within(attn.latent_attend(case, q, start, 2), ref, bound)


TRACE = r"""
import torch
import attention_split_kv_gb300 as attn
import seeded_inputs as si
from tests.latent_util import starts
attn.load()
for kv, cap, H in ((100, 256, 16), (100, 257, 16), (300, 0, 40), (300, 0, 128)):
    case = si.make_latent_case([kv], 512, 1, cap=cap, device="cuda")
    attn.latent_attend(case, si.f16_normal((1, H, 576), 2, "cuda"), starts([1], "cuda"), 1)
q = si.f16_normal((300, 4, 192), 3, "cuda")
st = starts([200, 100], "cuda")
attn.latent_prefill(q, q[..., :128], q[..., 64:], q[:, 0, :64], st, st, 200, 0.07)
torch.cuda.synchronize()
assert attn.attn_device_status() == attn.ATTN_OK
"""


def test_trace_names_the_forms():
    # short caches are not cut (and not joined); rows choose the block; several blocks go side by side
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", TRACE], cwd=root, env=dict(os.environ, ATTN_TRACE="1"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [x for x in r.stderr.splitlines() if x.startswith("[libattn]")]
    assert len(lines) == 5
    for line, part in zip(lines, ("rows=16> ", "rows=16> ", "rows=64> ", "rows=64> ", "latent_prefill_kernel ")):
        assert part in line, line
    assert "whole=1" in lines[0] and all("whole=0" in x for x in lines[1:4])
    assert "side=1" in lines[2] and "side=2" in lines[3] and "ranked=1" in lines[4]
