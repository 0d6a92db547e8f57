"""One dominant key beside many faint ones: the weights go to the products in f16, whose range has to
hold the faint ones too."""
import math

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from latent_util import F16, starts

pytestmark = pytest.mark.gpu
GAP = 18.0   # of the logits: the faint keys' weights are e^-18 = 2^-25.97 of the dominant one's


@pytest.fixture(autouse=True)
def _status():
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _check(out, lse, faint):
    # values: 0 of the dominant key, 1 of the others; logits GAP and 0
    w = faint * math.exp(-GAP)
    ref, ref_lse = w / (1.0 + w), GAP + math.log1p(w)
    # A faint weight is rounded to a multiple of 2^-24 (f16's least value) of a scale on which the
    # dominant one is 2^7 at least: off by at most 2^-32 of it.
    tiny = faint * 2.0 ** -32
    # Beside that, relative: the logit's error with the exponential's; the products' sums, 16 keys a step of
    # the tensor cores, which may cut (2^-23 each); the weights' sum, an addition a tile of 64 keys or more;
    # the output's rounding.
    logit, steps, adds = GAP * 2.0 ** -18, faint / 16 * 2.0 ** -23, faint / 64 * 2.0 ** -24
    err = (out.double() - ref).abs().max()
    assert float(err) <= tiny + ref * (logit + steps + adds + 2 * F16), (float(err), ref)
    # (the dominant weight is a power of two: rounded to itself, or off by the logit's error)
    err = (lse.double() - ref_lse).abs().max()
    assert float(err) <= tiny + logit + adds + 2.0 ** -18, (float(err), ref_lse)


# one CTA (or pair of them) walks a sequence whole where there are more sequences than of those; all of
# them read the same pages
@pytest.mark.parametrize("B,H,R,n", [(160, 8, 256, 131072), (160, 16, 512, 65536), (160, 60, 256, 65536),
                                     (160, 128, 256, 65536), (90, 128, 512, 65536)])
def test_attend(B, H, R, n):
    case = si.make_latent_case([n], R, 1, page_size=256, fill=0.0, device="cuda")
    case.cache[..., :R] = 1.0
    first = int(case.page_table[0, 0])
    case.cache[first, 0, :R] = 0.0
    case.cache[first, 0, R] = 1.0
    case.batch, case.scale = B, GAP
    case.page_table = case.page_table.expand(B, -1).contiguous()
    case.kv_len = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, H, R + 64, dtype=torch.float16, device="cuda")
    q[..., R] = 1.0
    lse = torch.empty(B, H, device="cuda")
    out = attn.latent_attend(case, q, starts([1] * B, "cuda"), 1, lse_out=lse)
    _check(out, lse, n - 1)


@pytest.mark.parametrize("n_q,H,n", [(1, 1, 131072), (100, 2, 65536), (300, 152, 65536)])
@pytest.mark.parametrize("where", ["first", "last"])
def test_prefill(n_q, H, n, where):
    # (two streams of key tiles, or two row tiles); not causal: every query keeps every key
    k = torch.zeros(n, 1, 128, dtype=torch.float16, device="cuda").expand(n, H, 128).contiguous()
    v = torch.ones(n, 1, 128, dtype=torch.float16, device="cuda").expand(n, H, 128).contiguous()
    r = torch.zeros(n, 64, dtype=torch.float16, device="cuda")
    at = 0 if where == "first" else n - 1
    v[at], r[at, 0] = 0.0, 1.0
    q = torch.zeros(n_q, H, 192, dtype=torch.float16, device="cuda")
    q[..., 128] = 1.0
    lse = torch.empty(n_q, H, device="cuda")
    out = attn.latent_prefill(q, k, v, r, starts([n_q], "cuda"), starts([n], "cuda"), n_q, GAP, causal=False, lse_out=lse)
    _check(out, lse, n - 1)
