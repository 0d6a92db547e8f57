"""Refusals of attn_append, attn_kv_read and attn_prefill_paged_ex that need no
GPU (every check is made on the host before a launch), and the plain forms their
GPU tests compare with, pinned to closed forms."""
import math

import pytest
import torch

import attention_split_kv_gb300 as attn
import oracle
import seeded_inputs as si
from cache_util import Cache, chunk_reference, norm_rotate, tables

FAKE = 1 << 20   # a non-null, aligned address never dereferenced on the host
LAYOUT = dict(page_table=None, page_size=0, max_pages=0, n_pages=0, max_kv=128, ring_size=0, k_scales=None,
              v_scales=None, kv_dtype=attn.ATTN_KV_F16)
APPEND = dict(q=FAKE, k=FAKE, v=FAKE, in_dtype=attn.ATTN_F16, q_stride=512, k_stride=512, v_stride=512, q_norm=FAKE,
              k_norm=FAKE, norm_eps=1e-6, norm_offset=0.0, rope_cos=FAKE, rope_sin=FAKE, rope_positions=128,
              rope_dim=64, rope_interleaved=False, q_start=FAKE, kv_len=FAKE, k_cache=FAKE, v_cache=FAKE, **LAYOUT,
              batch=1, total_q=4, n_heads=4, n_kv_heads=2, head_dim=64, q_out=FAKE, q_out_dtype=attn.ATTN_F16, stream=0)
READ = dict(k_cache=FAKE, v_cache=FAKE, kv_len=FAKE, first=None, out_start=FAKE, **LAYOUT, batch=1, total=4,
            n_kv_heads=2, head_dim=64, k_out=FAKE, v_out=FAKE, out_dtype=attn.ATTN_F16, stream=0)
CHUNK = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, q_start=FAKE, kv_len=FAKE, page_table=FAKE, page_size=16, max_pages=8,
             n_pages=8, k_scales=FAKE, v_scales=FAKE, kv_dtype=attn.ATTN_KV_INT8, batch=1, total_q=4, max_q=4,
             n_heads=4, n_kv_heads=2, head_dim=64, window=0, softcap=0.0, scale=0.125, out=FAKE, lse_out=None,
             workspace=FAKE, workspace_bytes=1 << 30, stream=0)
INT8 = dict(kv_dtype=attn.ATTN_KV_INT8, k_scales=FAKE, v_scales=FAKE)
PAGED = dict(page_table=FAKE, page_size=16, max_pages=8, n_pages=8)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()


def _refused(call, args, kw, status):
    with pytest.raises(attn.AttnError) as e:
        call(**{**args, **kw})
    assert e.value.status == status
    assert attn.attn_last_error()


LAYOUT_REFUSALS = [
    (dict(k_cache=None), attn.ATTN_EINVAL),
    (dict(v_cache=None), attn.ATTN_EINVAL),
    (dict(k_cache=FAKE + 8), attn.ATTN_EINVAL),
    (dict(n_kv_heads=0), attn.ATTN_EINVAL),
    (dict(head_dim=96, rope_dim=0), attn.ATTN_EUNSUPPORTED),
    (dict(kv_dtype=3), attn.ATTN_EINVAL),
    (dict(kv_dtype=attn.ATTN_KV_INT8), attn.ATTN_EINVAL),
    (dict(INT8, k_scales=None), attn.ATTN_EINVAL),
    (dict(INT8, v_scales=FAKE + 2), attn.ATTN_EINVAL),
    (dict(INT8, max_kv=100), attn.ATTN_EUNSUPPORTED),
    (dict(max_kv=0), attn.ATTN_EINVAL),
    (dict(ring_size=24), attn.ATTN_EUNSUPPORTED),
    (dict(ring_size=-16), attn.ATTN_EUNSUPPORTED),
    (dict(PAGED, ring_size=16), attn.ATTN_EINVAL),
    (dict(PAGED, page_size=12), attn.ATTN_EUNSUPPORTED),
    (dict(PAGED, page_size=2048), attn.ATTN_EUNSUPPORTED),
    (dict(PAGED, **INT8, page_size=4), attn.ATTN_EUNSUPPORTED),
    (dict(PAGED, max_pages=0), attn.ATTN_EINVAL),
    (dict(PAGED, n_pages=0), attn.ATTN_EINVAL),
    (dict(batch=0), attn.ATTN_EINVAL),
    (dict(kv_len=None), attn.ATTN_EINVAL),
]


@pytest.mark.parametrize("kw,status", LAYOUT_REFUSALS + [
    (dict(k=None), attn.ATTN_EINVAL),
    (dict(v=None), attn.ATTN_EINVAL),
    (dict(q=None), attn.ATTN_EINVAL),
    (dict(q_out=None), attn.ATTN_EINVAL),
    (dict(q_start=None), attn.ATTN_EINVAL),
    (dict(in_dtype=2), attn.ATTN_EINVAL),
    (dict(q_out_dtype=-1), attn.ATTN_EINVAL),
    (dict(total_q=-1), attn.ATTN_EINVAL),
    (dict(n_heads=0), attn.ATTN_EINVAL),
    (dict(n_heads=70000, q_stride=1 << 40), attn.ATTN_EUNSUPPORTED),
    (dict(q_stride=255), attn.ATTN_EINVAL),
    (dict(k_stride=64), attn.ATTN_EINVAL),
    (dict(v_stride=-512), attn.ATTN_EINVAL),
    (dict(v_stride=130), attn.ATTN_EUNSUPPORTED),
    (dict(in_dtype=attn.ATTN_F32, k_stride=130), attn.ATTN_EUNSUPPORTED),
    (dict(norm_eps=-1.0), attn.ATTN_EINVAL),
    (dict(norm_eps=NAN), attn.ATTN_EINVAL),
    (dict(norm_offset=INF), attn.ATTN_EINVAL),
    (dict(rope_dim=-16), attn.ATTN_EINVAL),
    (dict(rope_dim=80), attn.ATTN_EINVAL),
    (dict(rope_dim=24), attn.ATTN_EUNSUPPORTED),
    (dict(rope_cos=None), attn.ATTN_EINVAL),
    (dict(rope_positions=0), attn.ATTN_EINVAL),
    (dict(rope_sin=FAKE + 4), attn.ATTN_EINVAL),
    (dict(q_norm=FAKE + 4), attn.ATTN_EINVAL),
    (dict(k=FAKE + 2), attn.ATTN_EINVAL),
])
def test_append_refuses_on_host(kw, status):
    _refused(attn.attn_append, APPEND, kw, status)


@pytest.mark.parametrize("kw,status", [(dict((k, x) for k, x in d.items() if k != "rope_dim"), s)
                                       for d, s in LAYOUT_REFUSALS] + [
    (dict(out_start=None), attn.ATTN_EINVAL),
    (dict(k_out=None), attn.ATTN_EINVAL),
    (dict(v_out=FAKE + 8), attn.ATTN_EINVAL),
    (dict(out_dtype=5), attn.ATTN_EINVAL),
    (dict(total=-1), attn.ATTN_EINVAL),
])
def test_read_refuses_on_host(kw, status):
    _refused(attn.attn_kv_read, READ, kw, status)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), attn.ATTN_EINVAL),
    (dict(page_table=None), attn.ATTN_EINVAL),
    (dict(kv_dtype=9), attn.ATTN_EINVAL),
    (dict(k_scales=None), attn.ATTN_EINVAL),
    (dict(v_scales=FAKE + 2), attn.ATTN_EINVAL),
    (dict(page_size=4), attn.ATTN_EUNSUPPORTED),
    (dict(page_size=24), attn.ATTN_EUNSUPPORTED),
    (dict(n_heads=5), attn.ATTN_EINVAL),
    (dict(head_dim=80), attn.ATTN_EUNSUPPORTED),
    (dict(batch=70000), attn.ATTN_EUNSUPPORTED),
    (dict(window=-1), attn.ATTN_EINVAL),
    (dict(softcap=-2.0), attn.ATTN_EINVAL),
    (dict(scale=INF), attn.ATTN_EINVAL),
    (dict(workspace=None), attn.ATTN_EINVAL),
    (dict(workspace_bytes=16), attn.ATTN_EINVAL),
    (dict(workspace=FAKE + 16), attn.ATTN_EINVAL),
    (dict(out=FAKE + 2), attn.ATTN_EINVAL),
])
def test_chunk_refuses_on_host(kw, status):
    _refused(attn.attn_prefill_paged_ex, CHUNK, kw, status)


@pytest.mark.parametrize("kw", [dict(q_stride=512), dict(q_stride=256, k_stride=512, q_out_dtype=attn.ATTN_F32),
                                dict(q_stride=256, in_dtype=attn.ATTN_F32), dict(total_q=1, q_out_dtype=attn.ATTN_F32)],
                         ids=str)
def test_the_entry_point_refuses_q_out_over_other_rows(kw):
    _refused(attn.attn_append, APPEND, {**dict(q=1 << 21, q_out=1 << 21), **kw}, attn.ATTN_EINVAL)


@pytest.mark.parametrize("kw", [dict(q_stride=256), dict(total_q=1, q_stride=512), dict(q_out=1 << 22, q_stride=512)],
                         ids=str)
def test_the_entry_point_takes_q_out_over_the_rows_it_read(kw):
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    # every check passes: what remains is the missing GPU
    _refused(attn.attn_append, APPEND, {**dict(q=1 << 21, q_out=1 << 21), **kw}, attn.ATTN_ECUDA)


def test_no_rows_is_a_call_that_does_nothing():
    attn.attn_append(**{**APPEND, "total_q": 0})
    attn.attn_kv_read(**{**READ, "total": 0})
    attn.attn_prefill_paged_ex(**{**CHUNK, "total_q": 0, "max_q": 0})


def test_chunk_workspace_sizes():
    size = attn.attn_prefill_paged_workspace_size
    assert size(4, 512, 32, 8, 128, attn.ATTN_KV_INT8) > 0
    assert size(4, 512, 32, 8, 128, attn.ATTN_KV_F16) > 0
    for bad in [(0, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 1, 5, 2, 64), (1, 1, 4, 2, 80), (70000, 1, 4, 2, 64)]:
        assert size(*bad, attn.ATTN_KV_INT8) == 0
    assert size(1, 1, 4, 2, 64, 7) == 0


# ---- the plain forms
def test_plain_rotation_is_a_rotation():
    cos, sin = tables(50, 64)
    x = torch.randn(64, generator=torch.Generator().manual_seed(1))
    for inter in (False, True):
        y, _ = norm_rotate(x, None, 0, 0, cos, sin, 0, inter)
        assert torch.equal(y, x.double())                       # position 0
        y, mag = norm_rotate(x, None, 0, 0, cos, sin, 49, inter)
        assert abs(float(y.norm()) - float(x.double().norm())) < 1e-5   # lengths stay (tables are f32)
        assert bool((mag + 1e-9 >= y.abs()).all())
        # the product of two rotated heads depends on the distance alone
        a, _ = norm_rotate(x, None, 0, 0, cos, sin, 11, inter)
        b, _ = norm_rotate(x, None, 0, 0, cos, sin, 49 - 11, inter)
        z, _ = norm_rotate(x, None, 0, 0, cos, sin, 0, inter)
        c, _ = norm_rotate(x, None, 0, 0, cos, sin, 27, inter)
        assert abs(float(a @ b) - float(z @ c)) < 1e-4


def test_plain_norm_has_unit_mean_square():
    x = torch.randn(128, generator=torch.Generator().manual_seed(2))
    y, _ = norm_rotate(x, torch.zeros(128), 0.0, 1.0, None, None, 0, False)
    assert abs(float((y * y).mean()) - 1) < 1e-12


def test_plain_chunk_agrees_with_the_oracle_on_f16_values():
    # codes with a power-of-two scale are f16 values exactly, so the f16 oracle takes the same cache
    case = si.make_chunked_case(3, 4, 2, 64, [5, 0, 20], [30, 7, 0], seed=5, page_size=8, window=9, softcap=3.0,
                                int8=True)
    case.k_scales.fill_(1 / 32)
    case.v_scales.fill_(1 / 64)
    out, lse = chunk_reference(case)
    f16 = si.make_chunked_case(3, 4, 2, 64, [5, 0, 20], [30, 7, 0], seed=5, page_size=8, window=9, softcap=3.0)
    f16.k, f16.v = (case.k.double() / 32).half(), (case.v.double() / 64).half()
    ref, ref_lse = oracle.prefill_paged(f16)
    assert float((out.flatten(0, 1) - torch.from_numpy(ref)).abs().max()) < 1e-9
    assert float((lse.flatten() - torch.from_numpy(ref_lse)).abs().max()) < 1e-9


def test_cache_layouts_address_every_token_once():
    for layout in ("plain", "paged", "ring"):
        c = Cache(layout, 3, 1, 64, 40, ring=48, page_size=8)
        spots = {c.where(b, p) for b in range(3) for p in range(40)}
        assert len(spots) == 120
    assert math.isclose(float(Cache("plain", 1, 1, 64, 8, int8=True, fill=False).head("k", 0, 3, 0)[5]), 38.5)
