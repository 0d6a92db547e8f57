"""attn_latent_attend where a CTA (or pair) walks many whole items, as caches of at most 256 tokens are
taken, and where more row blocks than two of a token go side by side or one after the other."""
import os
import subprocess
import sys

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from latent_util import assert_lse, assert_within, attend_reference, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _check(q_lens, kv_lens, H, R, page, cap=0, seed=1):
    case = si.make_latent_case(kv_lens, R, seed, page_size=page, cap=cap, device="cuda")
    T = sum(q_lens)
    q = si.f16_normal((T + 1, H, R + 64), seed + 100, "cuda")
    out = torch.full((T + 1, H, R), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T + 1, H), 7.0, device="cuda")
    attn.latent_attend(case, q, starts(q_lens, "cuda"), max(q_lens), out=out, lse_out=lse)
    ref, ref_lse, bound = attend_reference(case, q[:T], q_lens)
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all()), "rows of no token were written"
    assert_within(out[:T], ref, bound)
    assert_lse(lse[:T], ref_lse)


# 0 to 256 tokens, whole tiles and odd ones in any order
MANY = [(37 * i) % 257 for i in range(700)]


@pytest.mark.parametrize("H,R", [(5, 512), (16, 512), (16, 256), (20, 256), (40, 512), (128, 256), (200, 256)])
@pytest.mark.parametrize("page", [0, 16, 256])
def test_many_single_tokens(H, R, page):
    _check([1] * 700, MANY, H, R, page, cap=256)


@pytest.mark.parametrize("page", [0, 16])
def test_many_single_tokens_and_sequences_without_one(page):
    _check([int(i % 3 != 1) for i in range(700)], MANY, 16, 512, page, cap=256)


@pytest.mark.parametrize("H,R", [(16, 512), (8, 256)])
@pytest.mark.parametrize("page", [0, 64])
def test_many_chunks(H, R, page):
    q_lens = [(13 * i) % 30 for i in range(60)]
    _check(q_lens, [max(n, (41 * i) % 257) for i, n in enumerate(q_lens)], H, R, page, cap=256)


@pytest.mark.parametrize("page", [0, 16, 64])
def test_pairs_of_single_tokens(page):
    _check([1] * 320, MANY[:320], 128, 512, page, cap=256)


def test_pairs_of_single_tokens_and_sequences_without_one():
    _check([int(i % 3 != 1) for i in range(330)], MANY[:330], 128, 512, 16, cap=256)


@pytest.mark.parametrize("page", [0, 32])
def test_pairs_of_prompts(page):
    _check([256, 0, 190], [256, 9, 256], 128, 512, page, cap=256)


@pytest.mark.parametrize("H", [129, 192, 300, 400, 512, 513, 1100])
@pytest.mark.parametrize("page", [0, 16])
def test_many_row_blocks(H, page):
    _check([1, 1], [2500, 3], H, 256, page)                              # cut and joined
    _check([1] * 5, [1, 63, 64, 65, 700], H, 256, page)
    _check([1, 0, 1], [200, 5, 130], H, 256, page)                       # whole
    if H <= 512:
        _check([1, 1, 1], [1900, 64, 1], H, 512, page)
        _check([1, 1, 1], [90, 256, 0], H, 512, page)


TRACE = r"""
import torch
import attention_split_kv_gb300 as attn
import seeded_inputs as si
from tests.latent_util import starts
attn.load()
for B, n, cap, H, R in ((700, 1, 256, 16, 512), (700, 1, 256, 200, 256), (320, 1, 256, 128, 512), (3, 256, 256, 128, 512),
                        (2, 1, 2500, 512, 256), (2, 1, 2500, 513, 256), (3, 1, 1900, 300, 512)):
    case = si.make_latent_case([9] * B, R, 1, page_size=16, cap=cap, device="cuda")
    attn.latent_attend(case, si.f16_normal((B * n, H, R + 64), 2, "cuda"), starts([n] * B, "cuda"), n)
torch.cuda.synchronize()
assert attn.attn_device_status() == attn.ATTN_OK
"""


def test_trace_names_the_forms():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", TRACE], cwd=root, env=dict(os.environ, ATTN_TRACE="1"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [x for x in r.stderr.splitlines() if x.startswith("[libattn]")]
    assert len(lines) == 7
    for line, pair, side, whole in zip(lines, (0, 0, 1, 1, 0, 0, 0), (1, 4, 1, 1, 8, 1, 5), (1, 1, 1, 1, 0, 0, 0)):
        assert ("latent_pair_kernel " in line) == bool(pair), line
        assert "side=%d " % side in line and "whole=%d" % whole in line, line
