"""attn_latent_prefill (the expanded form of latent attention) against its formula in 64 bits."""
import math

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from latent_util import assert_lse, assert_within, prefill_reference, starts

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    assert attn.attn_device_status() == attn.ATTN_OK
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _inputs(q_lens, kv_lens, H, seed=1, tail=0):
    q = si.f16_normal((sum(q_lens) + tail, H, 192), seed, "cuda")
    kv = si.f16_normal((sum(kv_lens) + tail, H, 256), seed + 1, "cuda")
    r = si.f16_normal((sum(kv_lens) + tail, 64), seed + 2, "cuda")
    return q, kv[..., :128], kv[..., 128:], r


def _check(q, k, v, r, q_lens, kv_lens, scale=SCALE, causal=True, what=""):
    T = sum(q_lens)
    out = torch.full((*q.shape[:2], 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    attn.latent_prefill(q, k, v, r, starts(q_lens, "cuda"), starts(kv_lens, "cuda"), max(q_lens), scale, causal, out=out,
                        lse_out=lse)
    ref, ref_lse, bound = prefill_reference(q[:T], k, v, r, q_lens, kv_lens, scale, causal)
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all()), "rows of no token were written"
    assert_within(out[:T], ref, bound, what)
    assert_lse(lse[:T], ref_lse, what)
    return out


LENS = [
    ([1], [1]), ([1], [300]), ([37], [37]), ([128], [128]), ([129], [129]), ([256], [256]), ([300], [700]),
    ([1, 0, 130, 257, 5], [1, 9, 130, 400, 128]),
    ([64, 200], [64, 1000]), ([513, 255], [513, 511]),
]


@pytest.mark.parametrize("q_lens,kv_lens", LENS, ids=str)
@pytest.mark.parametrize("H", [1, 3, 16])
@pytest.mark.parametrize("causal", [True, False])
def test_against_the_formula(q_lens, kv_lens, H, causal):
    _check(*_inputs(q_lens, kv_lens, H, tail=3), q_lens, kv_lens, causal=causal)


def test_more_queries_than_keys():
    out = _check(*_inputs([10, 300, 4], [4, 40, 0], 4, tail=1), [10, 300, 4], [4, 40, 0])
    assert bool((out[:6] == 0).all()) and bool((out[310:314] == 0).all())


def test_what_lies_behind_a_sequence_is_never_used():
    # the next sequence's rows, and rows of no sequence, are NaN for the first one
    q_lens, kv_lens = [70, 20], [70, 20]
    q, k, v, r = _inputs(q_lens, kv_lens, 4, tail=90)
    ref, _, bound = prefill_reference(q, k, v, r, q_lens, kv_lens, SCALE)
    for t in (k, v, r):
        t[70:] = math.nan
    out = attn.latent_prefill(q, k, v, r, starts(q_lens, "cuda"), starts(kv_lens, "cuda"), 70, SCALE)
    assert_within(out[:70], ref[:70], bound[:70])
    assert bool(out[70:90].isnan().all())


@pytest.mark.parametrize("step", [0.5, 12.0])
@pytest.mark.parametrize("causal", [True, False])
def test_logits_that_keep_growing(step, causal):
    q_lens, kv_lens = [300, 65], [900, 65]
    q, k, v, r = _inputs(q_lens, kv_lens, 2)
    g = torch.Generator(device="cuda").manual_seed(5)
    d = torch.randn(192, generator=g, device="cuda")
    d /= d.norm()
    pos = torch.cat([torch.arange(n, device="cuda") for n in kv_lens])[:, None]
    rows = pos / 128.0 * step / (SCALE * 14.0) * d
    k.copy_((rows[:, None, :128] + 0.3 * torch.randn(k.shape, generator=g, device="cuda")).half())
    r.copy_((rows[:, 128:] + 0.3 * torch.randn(r.shape, generator=g, device="cuda")).half())
    q.copy_((14.0 * d + 0.2 * torch.randn(q.shape, generator=g, device="cuda")).half())
    _check(q, k, v, r, q_lens, kv_lens, causal=causal)


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.4])
def test_scales(scale):
    _check(*_inputs([200], [333], 2), [200], [333], scale=scale)


def test_strides():
    # q of wider rows, k and v apart and with rows of padding, k_rope a slice of the latent rows
    q_lens, kv_lens = [140, 9], [300, 9]
    q = si.f16_normal((149, 5 * 192 + 64), 3, "cuda")[:, :960].view(149, 5, 192)
    k = si.f16_normal((309, 5, 136), 4, "cuda")[..., :128]
    v = si.f16_normal((309, 5, 128), 5, "cuda")
    r = si.f16_normal((309, 576), 6, "cuda")[:, 512:]
    _check(q, k, v, r, q_lens, kv_lens)


def test_a_chunk_longer_than_max_q_is_cut():
    q, k, v, r = _inputs([400, 50], [400, 50], 2)
    out = torch.full((450, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    attn.latent_prefill(q, k, v, r, starts([400, 50], "cuda"), starts([400, 50], "cuda"), 130, SCALE, out=out)
    ref, _, bound = prefill_reference(q, k, v, r, [400, 50], [400, 50], SCALE)
    assert_within(out[:130], ref[:130], bound[:130])
    assert bool((out[130:400] == 7).all())
    assert_within(out[400:], ref[400:], bound[400:])


def test_a_dominant_key_gives_its_value():
    q, k, v, r = _inputs([1], [300], 4)
    q[0, :, :128], q[0, :, 128:] = 8 * k[77], 8 * r[77]
    out = attn.latent_prefill(q, k, v, r, starts([1], "cuda"), starts([300], "cuda"), 1, SCALE)
    assert torch.equal(out[0], v[77])


def test_the_same_call_gives_the_same_bits_and_can_be_captured():
    q_lens, kv_lens = [300, 1, 60], [800, 5, 60]
    q, k, v, r = _inputs(q_lens, kv_lens, 8)
    args = (q, k, v, r, starts(q_lens, "cuda"), starts(kv_lens, "cuda"), 300, SCALE)
    a = attn.latent_prefill(*args)
    out = torch.empty_like(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.latent_prefill(*args, out=out)
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        assert torch.equal(a, out)


def test_a_long_prompt():
    q, k, v, r = _inputs([3000], [3000], 2)
    _check(q, k, v, r, [3000], [3000])


@pytest.mark.parametrize("n", [1, 5, 127, 128])
@pytest.mark.parametrize("L", [128, 129, 256, 257, 384, 500, 1100, 2000])
@pytest.mark.parametrize("causal", [True, False])
def test_few_queries_over_many_keys(n, L, causal):
    # blocks of one row tile take even and odd key tiles as two streams
    _check(*_inputs([n, 3], [L, 200], 2, tail=1), [n, 3], [L, 200], causal=causal)


def test_a_stream_without_a_key():
    # 100 queries, the last of 130 keys: in the second key tile only the last two keep any; and with
    # fewer keys than queries
    _check(*_inputs([100, 128], [130, 140], 2), [100, 128], [130, 140])
    _check(*_inputs([128, 100], [129, 40], 2), [128, 100], [129, 40])


@pytest.mark.parametrize("n", [300, 100])
def test_a_nan_query_stays_in_its_row(n):
    q, k, v, r = _inputs([n], [700], 3)
    ref, _, bound = prefill_reference(q, k, v, r, [n], [700], SCALE)
    q[7, 1, 5], q[40, 2, 150] = math.nan, math.inf
    out = attn.latent_prefill(q, k, v, r, starts([n], "cuda"), starts([700], "cuda"), n, SCALE)
    assert bool(out[7, 1].isnan().all()) and bool(out[40, 2].isnan().all())
    good = torch.ones(n, 3, dtype=torch.bool)
    good[7, 1] = good[40, 2] = False
    assert_within(out[good], ref[good], bound[good])


# Blocks of 256 queries are taken where they fill the SMs: sequences without tokens behind the others (ranked, and
# too many to be ranked), or one sequence of many heads.
WIDE = [
    ([256], [256]), ([300], [700]), ([129, 1], [129, 400]), ([1, 0, 130, 257, 5], [1, 9, 130, 400, 128]),
    ([513, 255], [513, 511]), ([700], [64]),
]


@pytest.mark.parametrize("q_lens,kv_lens", WIDE, ids=str)
@pytest.mark.parametrize("H,seqs", [(16, 12), (1, 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks_of_256(q_lens, kv_lens, H, seqs, causal):
    more = [0] * (seqs - len(q_lens))
    _check(*_inputs(q_lens, kv_lens, H, tail=3), q_lens + more, kv_lens + more, causal=causal)


@pytest.mark.parametrize("n,L", [(129, 129), (256, 300), (300, 700), (600, 513)])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks_of_256_of_one_sequence(n, L, causal):
    _check(*_inputs([n], [L], 160, tail=2), [n], [L], causal=causal)


@pytest.mark.parametrize("n,H", [(300, 160), (300, 20)])
def test_logits_that_keep_growing_in_both_row_tiles(n, H):
    q, k, v, r = _inputs([n], [900], H)
    g = torch.Generator(device="cuda").manual_seed(5)
    d = torch.randn(192, generator=g, device="cuda")
    d /= d.norm()
    rows = torch.arange(900, device="cuda")[:, None] / 128.0 * 12.0 / (SCALE * 14.0) * d
    k.copy_((rows[:, None, :128] + 0.3 * torch.randn(k.shape, generator=g, device="cuda")).half())
    r.copy_((rows[:, 128:] + 0.3 * torch.randn(r.shape, generator=g, device="cuda")).half())
    q.copy_((14.0 * d + 0.2 * torch.randn(q.shape, generator=g, device="cuda")).half())
    _check(q, k, v, r, [n], [900])


@pytest.mark.parametrize("n,H", [(300, 160), (300, 3)])
def test_rows_behind_a_long_sequence_and_nan_queries(n, H):
    q, k, v, r = _inputs([n], [700], H, tail=80)
    ref, _, bound = prefill_reference(q[:n], k, v, r, [n], [700], SCALE)
    for t in (k, v, r):
        t[700:] = math.nan
    q[7, 1, 5], q[260, 2, 150] = math.nan, math.inf
    st = starts([n], "cuda"), starts([700], "cuda")
    out = attn.latent_prefill(q, k, v, r, *st, n, SCALE)[:n]
    assert bool(out[7, 1].isnan().all()) and bool(out[260, 2].isnan().all())
    good = torch.ones(n, H, dtype=torch.bool)
    good[7, 1] = good[260, 2] = False
    assert_within(out[good], ref[good], bound[good])


@pytest.mark.parametrize("n,H", [(300, 160), (300, 16)])
def test_a_timeout_in_either_block_size(n, H):
    q, k, v, r = _inputs([n], [n], H)
    st = starts([n], "cuda")
    assert attn.attn_testing_set_waits(20_000_000, 1) == attn.ATTN_OK
    try:
        attn.latent_prefill(q, k, v, r, st, st, n, SCALE)
        assert attn.attn_device_status() == attn.ATTN_ETIMEOUT
    finally:
        assert attn.attn_testing_set_waits(0, 0) == attn.ATTN_OK
    _check(q, k, v, r, [n], [n])
