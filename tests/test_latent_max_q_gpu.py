"""max_q of the latent calls is an upper bound of the sequences' new tokens, however loose."""
import math
import os
import subprocess
import sys

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from latent_util import assert_lse, assert_within, attend_reference, prefill_reference, starts

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)
MOST = 65535 * 256   # of attn_latent_prefill


@pytest.fixture(autouse=True)
def _status():
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


@pytest.mark.parametrize("q_lens,kv_lens", [([100], [130]), ([1], [700]), ([300], [300]), ([40, 0, 7], [40, 9, 300]),
                                            ([200, 1, 129], [333, 1, 129])], ids=str)
@pytest.mark.parametrize("max_q", [1000, 70000, MOST // 2 + 200, MOST])
def test_prefill(q_lens, kv_lens, max_q):
    T = sum(q_lens)
    q = si.f16_normal((T + 2, 2, 192), 1, "cuda")
    kv, r = si.f16_normal((sum(kv_lens), 2, 256), 2, "cuda"), si.f16_normal((sum(kv_lens), 64), 3, "cuda")
    out = torch.full((T + 2, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T + 2, 2), 7.0, device="cuda")
    args = (q, kv[..., :128], kv[..., 128:], r, starts(q_lens, "cuda"), starts(kv_lens, "cuda"))
    attn.latent_prefill(*args, max_q, SCALE, out=out, lse_out=lse)
    ref, ref_lse, bound = prefill_reference(q[:T], *args[1:4], q_lens, kv_lens, SCALE)
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all()), "rows of no token were written"
    assert_within(out[:T], ref, bound)
    assert_lse(lse[:T], ref_lse)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [700, 3, 64]), ([3, 0, 5, 1], [300, 9, 5, 64])], ids=str)
@pytest.mark.parametrize("H,R", [(1, 512), (16, 512), (16, 256), (80, 512)])
@pytest.mark.parametrize("max_q", [6, 33, 5000])
def test_attend(q_lens, kv_lens, H, R, max_q):
    # (the bound chooses the block of rows, and pairs of CTAs where it and the capacity are large)
    T = sum(q_lens)
    case = si.make_latent_case(kv_lens, R, 1, page_size=16, cap=8192, device="cuda")
    q = si.f16_normal((T + 1, H, R + 64), 2, "cuda")
    out = torch.full((T + 1, H, R), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T + 1, H), 7.0, device="cuda")
    attn.latent_attend(case, q, starts(q_lens, "cuda"), max_q, out=out, lse_out=lse)
    ref, ref_lse, bound = attend_reference(case, q[:T], q_lens)
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all()), "rows of no token were written"
    assert_within(out[:T], ref, bound)
    assert_lse(lse[:T], ref_lse)


TRACE = r"""
import torch
import attention_split_kv_gb300 as attn
import seeded_inputs as si
from tests.latent_util import starts
attn.load()
for lens in ([100], [30, 50, 20]):
    q = si.f16_normal((100, 2, 192), 3, "cuda")
    st = starts(lens, "cuda")
    for max_q in (100, 101, 131072, 65535 * 200):
        attn.latent_prefill(q, q[..., :128], q[..., 64:], q[:, 0, :64], st, st, max_q, 0.07)
torch.cuda.synchronize()
assert attn.attn_device_status() == attn.ATTN_OK
"""


def test_prefill_launches_no_blocks_for_a_loose_bound():
    # a sequence has at most all queries: the launch is that of this bound, with the same ranking
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", TRACE], cwd=root, env=dict(os.environ, ATTN_TRACE="1"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [x for x in r.stderr.splitlines() if "latent_prefill_kernel " in x]
    assert len(lines) == 8 and len(set(lines[:4])) == 1 and len(set(lines[4:])) == 1, lines
    assert "ranked=1" in lines[4]
