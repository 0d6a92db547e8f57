"""attn_latent_read of many rows, whose CTAs take 32 each: several rounds of copies, sequences' ends
inside a CTA, a last CTA that is not full."""
import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from latent_util import rows_of, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,page", [(256, 16), (256, 0), (512, 64)])
@pytest.mark.parametrize("f32", [False, True])
def test_many_rows(R, page, f32):
    # 45 thousand rows, and 3 that are not a sequence's; tokens below 0 and past the lengths are zeros
    kv_lens = [9000, 0, 1, 20001, 33, 0, 15, 17000]
    first = [0, 0, 0, 100, -3, 2, 0, 5]
    n = [9000, 0, 1, 19001, 40, 3, 15, 16999]
    case = si.make_latent_case(kv_lens, R, 3, page_size=page, device="cuda")
    T = sum(n)
    dt = torch.float32 if f32 else torch.float16
    c, k = (torch.full((T + 3, w), 7.0, dtype=dt, device="cuda") for w in (R, 64))
    attn.attn_latent_read(case.cache, case.kv_len, torch.tensor(first, dtype=torch.int32, device="cuda"), starts(n, "cuda"),
                          case.page_table, page, case.max_pages, case.cache.shape[0], case.cache.shape[1], case.batch, T + 3, R, 64,
                          c, k, attn.ATTN_F32 if f32 else attn.ATTN_F16)
    ref = torch.zeros(T, R + 64, dtype=torch.float64, device="cuda")
    at = 0
    for b, (a, m, L) in enumerate(zip(first, n, kv_lens)):
        lo, hi = max(a, 0), min(a + m, L)
        if hi > lo:
            ref[at + lo - a:at + hi - a] = rows_of(case, b, L)[lo:hi]
        at += m
    assert torch.equal(c[:T].double(), ref[:, :R]) and torch.equal(k[:T].double(), ref[:, R:])
    assert bool((c[T:] == 7).all()) and bool((k[T:] == 7).all())
    assert attn.attn_device_status() == attn.ATTN_OK
