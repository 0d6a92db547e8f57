"""What append, kv_read and prefill_paged refuse before any entry point is called:
tensors that do not agree with the cache or with one another, which the kernels would
address out of range.  The tensors are on the CPU and nothing is launched."""
import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from cache_util import Cache, tables

_names = "-".join   # of a dict's keys
ENTRIES = ("attn_append", "attn_kv_read", "attn_prefill_paged_ex")


@pytest.fixture(autouse=True)
def called(monkeypatch):
    """The entry points replaced by ones that note their call."""
    calls = []
    for name in ENTRIES:
        monkeypatch.setattr(attn, name, lambda *args, name=name: calls.append((name, args)))
    monkeypatch.setattr(attn, "attn_prefill_paged_workspace_size", lambda *args: 256)
    return calls


def _refuses(call, called):
    with pytest.raises(attn.AttnError) as e:
        call()
    assert e.value.status == attn.ATTN_EINVAL and not called


def _append_args(**kw):
    cos, sin = tables(40, 64)
    x = torch.zeros(5, 8, 64, dtype=torch.float16)
    args = dict(q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], q_start=torch.tensor([0, 2, 5], dtype=torch.int32),
                kv_len=torch.tensor([2, 30], dtype=torch.int32), q_norm=torch.ones(64), k_norm=torch.ones(64),
                rope_cos=cos, rope_sin=sin, q_out=torch.zeros(5, 4, 64, dtype=torch.float16))
    args.update(kw)
    return args


def _f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _i32(n):
    return torch.zeros(n, dtype=torch.int32)


CACHES = [dict(layout="plain"), dict(layout="paged", page_size=8), dict(layout="ring", ring=32)]


@pytest.mark.parametrize("layout", CACHES, ids=lambda d: d["layout"])
@pytest.mark.parametrize("int8", [False, True])
def test_tensors_that_agree_are_taken(layout, int8, called):
    cache = Cache(B=2, Hkv=2, D=64, cap=40, int8=int8, **layout)
    attn.append(cache, **_append_args())
    attn.append(cache, **_append_args(q=None, q_out=None, q_norm=None, rope_cos=None, rope_sin=None))
    q = _f16(5, 4, 64)
    assert attn.append(cache, **_append_args(q=q, q_out=q)) is q
    attn.append(cache, **_append_args(q_start=_i32(9), kv_len=_i32(7)))      # buffers of a larger batch
    attn.kv_read(cache, _i32(3), 6, first=_i32(2), kv_len=_i32(2))
    assert [c[0] for c in called] == ["attn_append"] * 4 + ["attn_kv_read"]


@pytest.mark.parametrize("kw", [
    dict(q=_f16(4, 4, 64)), dict(q=_f16(6, 4, 64)), dict(q=_f16(5, 4, 128)), dict(q=_f16(5, 256)),
    dict(k=_f16(5, 1, 64)), dict(k=_f16(5, 2, 128)), dict(k=_f16(5, 3, 64), v=_f16(5, 3, 64)),
    dict(k=_f16(5, 2, 128), v=_f16(5, 2, 128), q=_f16(5, 4, 128), q_out=None),
    dict(v=_f16(4, 2, 64)), dict(v=_f16(5, 1, 64)), dict(v=_f16(5, 2, 32)),
    dict(q_start=_i32(2)), dict(kv_len=_i32(1)),
    dict(q_norm=torch.ones(32)), dict(k_norm=torch.ones(128)), dict(q_norm=torch.ones(128)[::2]),
    dict(rope_sin=tables(39, 64)[1]), dict(rope_sin=tables(40, 32)[1]), dict(rope_sin=None), dict(rope_cos=None),
    dict(rope_cos=torch.ones(2560), rope_sin=torch.ones(2560)),
    dict(q_out=_f16(4, 4, 64)), dict(q_out=_f16(5, 256)), dict(q_out=_f16(5, 8, 64)[:, :4]),
    dict(q_out=_f16(5, 64, 4).transpose(1, 2)), dict(q_out=torch.zeros(5, 4, 64, dtype=torch.bfloat16)),
    dict(v=torch.zeros(5, 2, 64, dtype=torch.float16, device="meta")),
    dict(q_start=torch.zeros(3, dtype=torch.int32, device="meta")),
], ids=_names)
def test_append_refuses_tensors_that_do_not_agree(kw, called):
    _refuses(lambda: attn.append(Cache("plain", 2, 2, 64, 40), **_append_args(**kw)), called)


def test_append_refuses_to_rotate_a_slice_in_place(called):
    # q_out is packed: written over a slice of a projection's rows it would fall on other tokens' q, k and v
    x = _f16(5, 8, 64)
    args = _append_args(q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], q_out=x[:, :4])
    _refuses(lambda: attn.append(Cache("plain", 2, 2, 64, 40), **args), called)


BAD_CACHES = [
    dict(v=_f16(2, 40, 2, 32)), dict(v=torch.zeros(2, 40, 2, 64, dtype=torch.int8)),
    dict(k=torch.zeros(2, 40, 2, 64), v=torch.zeros(2, 40, 2, 64)),
    dict(k=_f16(2, 40, 128), v=_f16(2, 40, 128)), dict(k=_f16(2, 80, 2, 64)[:, ::2]),
    dict(batch=3), dict(n_kv_heads=3), dict(head_dim=128), dict(ring=32),
    dict(page_table=_i32(6).view(2, 3), page_size=16, max_pages=3),
    dict(page_table=_i32(2).view(1, 2), page_size=40, max_pages=2),
    dict(page_table=_i32(6).view(2, 3), page_size=40, max_pages=2),
    dict(page_table=_i32(12).view(2, 6)[:, :2], page_size=40, max_pages=2),
    dict(page_table=_i32(4).view(2, 2).long(), page_size=40, max_pages=2),
]


@pytest.mark.parametrize("kw", BAD_CACHES, ids=_names)
def test_caches_that_do_not_agree_are_refused(kw, called):
    cache = Cache("plain", 2, 2, 64, 40)
    cache.__dict__.update(kw)
    _refuses(lambda: attn.append(cache, **_append_args()), called)
    _refuses(lambda: attn.kv_read(cache, _i32(3), 4, kv_len=_i32(2)), called)


@pytest.mark.parametrize("kw", [dict(k_scales=None), dict(v_scales=_f16(2, 40, 2)), dict(k_scales=torch.zeros(2, 2, 40)),
                                dict(v_scales=_f16(2, 40, 2).transpose(1, 2))], ids=_names)
def test_scales_that_do_not_agree_are_refused(kw, called):
    cache = Cache("plain", 2, 2, 64, 40, int8=True)
    cache.__dict__.update(kw)
    _refuses(lambda: attn.append(cache, **_append_args()), called)
    _refuses(lambda: attn.kv_read(cache, _i32(3), 4, kv_len=_i32(2)), called)


@pytest.mark.parametrize("kw", [dict(out_start=_i32(2)), dict(first=_i32(1)), dict(kv_len=_i32(1)),
                                dict(first=_i32(4)[::2])], ids=_names)
def test_read_refuses_short_lengths(kw, called):
    args = dict(out_start=_i32(3), total=4, first=_i32(2), kv_len=_i32(2))
    _refuses(lambda: attn.kv_read(Cache("plain", 2, 2, 64, 40), **{**args, **kw}), called)


@pytest.mark.parametrize("kw", [dict(q=_f16(10, 4, 64)), dict(q=_f16(11, 4, 128)[..., :64]), dict(q=torch.zeros(11, 4, 64)),
                                dict(k_scales=_f16(9, 2, 8)), dict(q_start=_i32(2)), dict(kv_len=_i32(1)),
                                dict(page_size=8), dict(n_kv_heads=1), dict(v_scales=None)], ids=_names)
def test_int8_chunks_refuse_tensors_that_do_not_agree(kw, called):
    case = si.make_chunked_case(2, 4, 2, 64, [5, 6], [9, 30], seed=1, page_size=16, int8=True)
    attn.prefill_paged(case)
    assert called.pop()[0] == "attn_prefill_paged_ex"
    _refuses(lambda: attn.prefill_paged(case, out=_f16(10, 4, 64)), called)
    _refuses(lambda: attn.prefill_paged(case, lse_out=_f16(11, 4)), called)
    case.__dict__.update(kw)
    _refuses(lambda: attn.prefill_paged(case), called)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("max_q", [0, 7])
def test_a_step_without_new_tokens_does_nothing(int8, max_q, monkeypatch):
    # a server's step in which no sequence has a new token, with max_q as counted or as a fixed bound
    monkeypatch.undo()
    attn.build()
    case = si.make_chunked_case(2, 4, 2, 64, [0, 0], [9, 30], seed=1, page_size=16, int8=int8)
    case.q, case.max_q = _f16(0, 4, 64), max_q
    out, lse = _f16(3, 4, 64) + 5, torch.full((3, 4), 5.0)
    assert attn.prefill_paged(case).shape == (0, 4, 64)
    assert attn.prefill_paged(case, out=out, lse_out=lse) is out
    assert bool((out == 5).all()) and bool((lse == 5).all())
    for layout in CACHES:
        cache = Cache(B=2, Hkv=2, D=64, cap=40, int8=int8, **layout)
        q, k = _f16(0, 4, 64), _f16(0, 2, 64)
        got = attn.append(cache, q, k, k, _i32(3), _i32(2), rope_cos=tables(40, 64)[0], rope_sin=tables(40, 64)[1])
        assert got.shape == (0, 4, 64) and got.dtype == torch.float16
        assert attn.append(cache, None, k, k, _i32(3), _i32(2)) is None
        k, v = attn.kv_read(cache, _i32(3), 0, kv_len=_i32(2), out_f32=True)
        assert k.shape == v.shape == (0, 2, 64) and k.dtype == torch.float32


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_the_current_stream_without_torch_s_short_cut(missing, monkeypatch):
    # torch's own way to a raw stream is used where it is there, and not needed
    class Now:
        cuda_stream = 12345

    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Now)
    monkeypatch.delattr(torch._C, missing, raising=False)
    assert attn._stream(None) == 12345
    assert attn._stream(77) == 77 and attn._stream(Now) == 12345
