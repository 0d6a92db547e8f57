"""What the latent attention calls refuse on the host, before anything is launched: bad arguments
(C ABI) and tensors that do not agree (binding).  No GPU is needed."""
import ctypes

import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si

FAKE = 1 << 20   # a non-null, aligned address never dereferenced on the host
EINVAL, EUNSUPPORTED = attn.ATTN_EINVAL, attn.ATTN_EUNSUPPORTED
PAGED = dict(page_table=FAKE, page_size=16, max_pages_per_seq=4, n_pages=9, max_kv=0)
CACHE = dict(cache=FAKE, page_table=None, page_size=0, max_pages_per_seq=0, n_pages=0, max_kv=128)
ORDER = {
    "attn_latent_append": "c k_rope q_rope in_dtype c_stride k_rope_stride q_stride q_head_stride c_norm norm_eps norm_offset "
                          "rope_cos rope_sin rope_positions rope_interleaved q_start kv_len cache page_table page_size "
                          "max_pages_per_seq n_pages max_kv batch total_q n_heads latent_dim rope_dim q_out q_out_stride "
                          "q_out_head_stride stream",
    "attn_latent_read": "cache kv_len first out_start page_table page_size max_pages_per_seq n_pages max_kv batch total "
                        "latent_dim rope_dim c_out k_rope_out out_dtype stream",
    "attn_latent_attend": "q cache q_start kv_len page_table page_size max_pages_per_seq n_pages max_kv batch total_q max_q "
                          "n_heads latent_dim rope_dim scale out lse_out workspace workspace_bytes stream",
    "attn_latent_prefill": "q k v k_rope q_stride k_stride k_head_stride v_stride v_head_stride k_rope_stride q_start kv_start "
                           "batch total_q total_kv max_q n_heads head_dim rope_dim causal scale out lse_out stream",
}
GOOD = {
    "attn_latent_append": dict(c=FAKE, k_rope=FAKE, q_rope=FAKE, in_dtype=attn.ATTN_F16, c_stride=576, k_rope_stride=576,
                               q_stride=4 * 192, q_head_stride=192, c_norm=FAKE, norm_eps=1e-6, norm_offset=0.0, rope_cos=FAKE,
                               rope_sin=FAKE, rope_positions=128, rope_interleaved=1, q_start=FAKE, kv_len=FAKE, batch=1,
                               total_q=0, n_heads=4, latent_dim=512, rope_dim=64, q_out=2 * FAKE, q_out_stride=4 * 576,
                               q_out_head_stride=576, **CACHE),
    "attn_latent_read": dict(kv_len=FAKE, first=None, out_start=FAKE, batch=1, total=0, latent_dim=512, rope_dim=64, c_out=FAKE,
                             k_rope_out=FAKE, out_dtype=attn.ATTN_F16, **CACHE),
    "attn_latent_attend": dict(q=FAKE, q_start=FAKE, kv_len=FAKE, batch=1, total_q=0, max_q=1, n_heads=4, latent_dim=512,
                               rope_dim=64, scale=0.1, out=FAKE, lse_out=None, workspace=FAKE, workspace_bytes=1 << 30, **CACHE),
    "attn_latent_prefill": dict(q=FAKE, k=FAKE, v=FAKE, k_rope=FAKE, q_stride=4 * 192, k_stride=1024, k_head_stride=256,
                                v_stride=1024, v_head_stride=256, k_rope_stride=64, q_start=FAKE, kv_start=FAKE, batch=1,
                                total_q=0, total_kv=5, max_q=1, n_heads=4, head_dim=128, rope_dim=64, causal=1, scale=0.1,
                                out=FAKE, lse_out=None),
}


def _call(name, **kw):
    args = dict(GOOD[name], stream=0)
    args.update(kw)
    return getattr(attn.load(), name)(*[args[k] for k in ORDER[name].split()])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()


@pytest.mark.parametrize("name", sorted(GOOD))
def test_calls_without_a_token_do_nothing(name):
    assert _call(name) == attn.ATTN_OK
    if "cache" in GOOD[name]:
        assert _call(name, **PAGED) == attn.ATTN_OK


CACHE_BAD = [
    (dict(cache=None), EINVAL), (dict(cache=FAKE + 2), EINVAL), (dict(max_kv=0), EINVAL), (dict(batch=0), EINVAL),
    (dict(batch=65536), EUNSUPPORTED), (dict(latent_dim=128), EUNSUPPORTED), (dict(latent_dim=576), EUNSUPPORTED),
    (dict(rope_dim=32), EUNSUPPORTED), (dict(PAGED, page_size=4), EUNSUPPORTED), (dict(PAGED, page_size=24), EUNSUPPORTED),
    (dict(PAGED, page_size=2048), EUNSUPPORTED), (dict(PAGED, n_pages=0), EINVAL), (dict(PAGED, max_pages_per_seq=0), EINVAL),
]


@pytest.mark.parametrize("name", ["attn_latent_append", "attn_latent_read", "attn_latent_attend"])
@pytest.mark.parametrize("kw,status", CACHE_BAD, ids=str)
def test_bad_caches(name, kw, status):
    assert _call(name, **kw) == status and attn.attn_last_error().startswith(name)


@pytest.mark.parametrize("name,kw,status", [
    ("append", dict(c=None), EINVAL), ("append", dict(k_rope=None), EINVAL), ("append", dict(q_rope=None), EINVAL),
    ("append", dict(q_out=None), EINVAL), ("append", dict(in_dtype=2), EINVAL), ("append", dict(total_q=-1), EINVAL),
    ("append", dict(n_heads=0), EINVAL), ("append", dict(n_heads=65536), EUNSUPPORTED), ("append", dict(c_stride=504), EINVAL),
    ("append", dict(c_stride=580), EUNSUPPORTED), ("append", dict(k_rope_stride=63), EINVAL),
    ("append", dict(q_head_stride=56), EINVAL), ("append", dict(q_stride=3 * 192), EINVAL),
    ("append", dict(q_head_stride=196, q_stride=1024), EUNSUPPORTED), ("append", dict(q_out_stride=576), EINVAL),
    ("append", dict(q_out_head_stride=580, q_out_stride=4096), EUNSUPPORTED), ("append", dict(norm_eps=-1.0), EINVAL),
    ("append", dict(norm_eps=float("nan")), EINVAL), ("append", dict(norm_offset=float("inf")), EINVAL),
    ("append", dict(rope_sin=None), EINVAL), ("append", dict(rope_positions=0), EINVAL), ("append", dict(c=FAKE + 4), EINVAL),
    ("append", dict(q_out=FAKE), EINVAL),      # q_rope, with other strides
    ("append", dict(q_out=FAKE, in_dtype=attn.ATTN_F32, q_out_stride=768, q_out_head_stride=192), EINVAL),
    ("read", dict(out_start=None), EINVAL), ("read", dict(c_out=None), EINVAL), ("read", dict(k_rope_out=FAKE + 8), EINVAL),
    ("read", dict(out_dtype=5), EINVAL), ("read", dict(total=-1), EINVAL),
    ("attend", dict(q=None), EINVAL), ("attend", dict(out=None), EINVAL), ("attend", dict(workspace=None), EINVAL),
    ("attend", dict(total_q=1, workspace_bytes=256), EINVAL), ("attend", dict(workspace=FAKE + 128), EINVAL),
    ("attend", dict(scale=float("inf")), EINVAL), ("attend", dict(n_heads=0), EINVAL), ("attend", dict(max_q=-1), EINVAL),
    ("attend", dict(total_q=1 << 20, n_heads=4096), EUNSUPPORTED), ("attend", dict(q=FAKE + 8), EINVAL),
    ("prefill", dict(v=None), EINVAL), ("prefill", dict(kv_start=None), EINVAL), ("prefill", dict(total_kv=0), EINVAL),
    ("prefill", dict(head_dim=64), EUNSUPPORTED), ("prefill", dict(rope_dim=32), EUNSUPPORTED),
    ("prefill", dict(causal=2), EINVAL), ("prefill", dict(scale=float("nan")), EINVAL),
    ("prefill", dict(q_stride=760), EINVAL), ("prefill", dict(k_head_stride=120), EINVAL),
    ("prefill", dict(v_stride=512), EINVAL), ("prefill", dict(k_rope_stride=68), EUNSUPPORTED),
    ("prefill", dict(k_rope_stride=56), EINVAL), ("prefill", dict(k_rope=FAKE + 2), EINVAL),
    ("prefill", dict(batch=65536), EUNSUPPORTED), ("prefill", dict(n_heads=-1), EINVAL),
], ids=lambda x: str(x))
def test_bad_arguments(name, kw, status):
    assert _call("attn_latent_" + name, **kw) == status
    assert attn.attn_last_error().startswith("attn_latent_" + name)


def test_q_may_be_rotated_in_place_only_as_it_lies():
    assert _call("attn_latent_append", q_out=FAKE, q_out_stride=768, q_out_head_stride=192) == attn.ATTN_OK


def test_workspace_sizes():
    size = attn.attn_latent_workspace_size
    assert size(1, 1, 16, 512) > 0 and size(1, 1, 16, 512) % 256 == 0
    assert size(1, 1, 16, 512) < size(1, 1, 32, 512) < size(1, 1, 64, 512) == size(9, 500, 128, 512)
    for bad in ((0, 1, 16, 512), (1, 0, 16, 512), (1, 1, 0, 512), (1, 1, 16, 128), (70000, 1, 16, 512), (1, 1 << 20, 4096, 512)):
        assert size(*bad) == 0


# ------------------------------------------------------------------ the binding
def _f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _i32(n):
    return torch.zeros(n, dtype=torch.int32)


@pytest.fixture
def called(monkeypatch):
    calls = []
    for name in GOOD:
        monkeypatch.setattr(attn, name, lambda *args, name=name: calls.append((name, args)))
    return calls


def _refuses(call, called):
    with pytest.raises(attn.AttnError) as e:
        call()
    assert e.value.status == EINVAL and not called


def _case(**kw):
    case = si.make_latent_case([20, 9], 256, 1, page_size=kw.pop("pages", 0))
    case.__dict__.update(kw)
    return case


def _append(case, **kw):
    x = _f16(5, 320)
    args = dict(c=x[:, :256], k_rope=x[:, 256:], q_start=_i32(3), q_rope=_f16(5, 4, 192)[..., 128:], c_norm=torch.ones(256),
                rope_cos=torch.ones(20, 32), rope_sin=torch.ones(20, 32), q_out=_f16(5, 4, 320)[..., 256:])
    args.update(kw)
    return attn.latent_append(case, **args)


@pytest.mark.parametrize("page_size", [0, 16])
def test_tensors_that_agree_are_taken(page_size, called):
    case = _case(pages=page_size)
    _append(case)
    _append(case, q_rope=None, q_out=None, c_norm=None, rope_cos=None, rope_sin=None)
    assert _append(case, q_out=None).shape == (5, 4, 64)
    assert _append(case, c=_f16(1, 256), k_rope=_f16(1, 64), q_rope=_f16(1, 1, 64), q_out=None).shape == (1, 1, 64)
    attn.latent_read(case, _i32(3), 6, first=_i32(2))
    attn.latent_attend(case, _f16(5, 4, 320), _i32(3), 3, lse_out=torch.zeros(5, 4))
    x = _f16(7, 4, 256)
    attn.latent_prefill(_f16(5, 4, 192), x[..., :128], x[..., 128:], _f16(7, 64), _i32(3), _i32(3), 3, 0.1)
    assert [c[0] for c in called] == ["attn_latent_append"] * 4 + ["attn_latent_read", "attn_latent_attend", "attn_latent_prefill"]


def test_calls_without_a_token_are_not_made(called):
    case = _case()
    _append(case, c=_f16(0, 256), k_rope=_f16(0, 64), q_rope=_f16(0, 4, 64), q_out=None)
    attn.latent_read(case, _i32(3), 0)
    attn.latent_attend(case, _f16(0, 4, 320), _i32(3), 0)
    attn.latent_prefill(_f16(0, 4, 192), _f16(7, 4, 128), _f16(7, 4, 128), _f16(7, 64), _i32(3), _i32(3), 0, 0.1)
    assert not called


@pytest.mark.parametrize("kw", [
    dict(c=_f16(5, 320)), dict(c=_f16(4, 256)), dict(k_rope=_f16(5, 32)), dict(k_rope=torch.zeros(5, 64)),
    dict(c=_f16(256, 5).T), dict(q_rope=_f16(4, 4, 64)), dict(q_rope=_f16(5, 4, 128)), dict(q_rope=torch.zeros(5, 4, 64)),
    dict(q_out=_f16(5, 3, 64)), dict(q_out=torch.zeros(5, 4, 64)), dict(q_out=_f16(5, 64, 4).transpose(1, 2)),
    dict(c_norm=torch.ones(320)), dict(c_norm=_f16(256)), dict(rope_sin=None), dict(rope_sin=torch.ones(19, 32)),
    dict(rope_cos=torch.ones(20, 64), rope_sin=torch.ones(20, 64)), dict(q_start=_i32(2)), dict(kv_len=_i32(1)),
    dict(q_start=torch.zeros(3, dtype=torch.int64)), dict(c=torch.zeros(5, 256, dtype=torch.float16, device="meta")),
], ids="-".join)
def test_append_refuses_tensors_that_do_not_agree(kw, called):
    _refuses(lambda: _append(_case(), **kw), called)


@pytest.mark.parametrize("kw", [
    dict(cache=torch.zeros(2, 20, 320)), dict(cache=_f16(2, 20, 640)[..., ::2]), dict(cache=_f16(1, 20, 320)),
    dict(cache=_f16(40, 320)), dict(page_table=_i32(4).view(2, 2), page_size=16, max_pages=2),
    dict(page_table=_i32(2).view(2, 1), page_size=20, max_pages=2), dict(page_table=_i32(4).view(2, 2).long(), page_size=20, max_pages=2),
], ids="-".join)
def test_caches_that_do_not_agree_are_refused(kw, called):
    _refuses(lambda: _append(_case(**kw)), called)
    _refuses(lambda: attn.latent_read(_case(**kw), _i32(3), 4), called)
    _refuses(lambda: attn.latent_attend(_case(**kw), _f16(5, 4, 320), _i32(3), 3), called)


@pytest.mark.parametrize("kw", [
    dict(q=_f16(5, 4, 256)), dict(q=torch.zeros(5, 4, 320)), dict(q=_f16(5, 8, 320)[:, ::2]), dict(q_start=_i32(2)),
    dict(kv_len=_i32(1)), dict(out=_f16(5, 4, 320)), dict(out=torch.zeros(5, 4, 256)), dict(lse_out=torch.zeros(5)),
    dict(lse_out=_f16(5, 4)),
], ids="-".join)
def test_attend_refuses_tensors_that_do_not_agree(kw, called):
    args = dict(q=_f16(5, 4, 320), q_start=_i32(3), max_q=3)
    args.update(kw)
    _refuses(lambda: attn.latent_attend(_case(), **args), called)


@pytest.mark.parametrize("kw", [
    dict(q=_f16(5, 4, 128)), dict(q=torch.zeros(5, 4, 192)), dict(q=_f16(5, 4, 256)[..., :192]), dict(k=_f16(7, 3, 128)),
    dict(k=_f16(7, 4, 64), v=_f16(7, 4, 64)), dict(v=_f16(6, 4, 128)), dict(v=torch.zeros(7, 4, 128)), dict(k_rope=_f16(6, 64)),
    dict(k_rope=_f16(7, 32)), dict(kv_start=_i32(4)), dict(q_start=_i32(1), kv_start=_i32(1)), dict(out=_f16(5, 4, 192)),
    dict(lse_out=torch.zeros(4, 4)), dict(k=_f16(7, 128, 4).transpose(1, 2)),
], ids="-".join)
def test_prefill_refuses_tensors_that_do_not_agree(kw, called):
    args = dict(q=_f16(5, 4, 192), k=_f16(7, 4, 128), v=_f16(7, 4, 128), k_rope=_f16(7, 64), q_start=_i32(3), kv_start=_i32(3),
                max_q=3, scale=0.1)
    args.update(kw)
    _refuses(lambda: attn.latent_prefill(**args), called)


# ------------------------------------------------------------------ argument structs
def _fields(name):
    """The header's struct of a call, as (name, ctypes type) in order."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "attn.h")).read()
    body = re.search(r"typedef struct %s_args \{(.*?)\}" % name, text, re.S).group(1)
    kinds = {"int": ctypes.c_int, "attn_dtype": ctypes.c_int, "float": ctypes.c_float, "long long": ctypes.c_longlong,
             "size_t": ctypes.c_size_t}
    out = []
    for line in body.split(";")[:-1]:
        line = " ".join(line.split()).replace("*", " * ")
        first, *more = line.split(",")
        kind = first.replace("*", " ").replace("const ", "").split()
        for at, item in enumerate([first] + more):
            out.append((item.split()[-1], ctypes.c_void_p if "*" in item else kinds[" ".join(kind[:-1])]))
    return out


@pytest.mark.parametrize("name", sorted(GOOD))
def test_argument_structs_lie_as_the_header_says(name, monkeypatch):
    fields = _fields(name)
    assert [f for f, _ in fields] == ORDER[name].split()
    Args = type("Args", (ctypes.Structure,), {"_fields_": fields})
    values = {f: (0.5 + i if t is ctypes.c_float else 64 * (i + 1)) for i, (f, t) in enumerate(fields)}
    values.update((f, 1) for f in ("rope_interleaved", "causal") if f in values)   # flags
    seen = []

    class Lib:
        def __getattr__(self, what):
            return lambda data: seen.append((what, data)) or attn.ATTN_OK
    monkeypatch.setattr(attn, "load", Lib)
    getattr(attn, name)(*[values[f] for f, _ in fields])
    (what, data), = seen
    assert what == name + "_from"
    got = Args.from_buffer_copy(data.ljust(ctypes.sizeof(Args), b"\0"))
    assert {f: getattr(got, f) for f, _ in fields} == values


@pytest.mark.parametrize("name,kw,status", [
    ("append", dict(c=None), EINVAL), ("append", dict(q_out_stride=576), EINVAL), ("append", dict(latent_dim=128), EUNSUPPORTED),
    ("append", dict(total_q=1 << 40), EINVAL), ("append", dict(norm_eps=1e300), EINVAL), ("append", dict(n_heads=2.5), EINVAL),
    ("read", dict(k_rope_out=FAKE + 8), EINVAL), ("read", dict(rope_dim=32), EUNSUPPORTED), ("read", dict(total=-1), EINVAL),
    ("attend", dict(workspace=FAKE + 128), EINVAL), ("attend", dict(workspace_bytes=-1), EINVAL),
    ("attend", dict(scale=float("nan")), EINVAL), ("attend", dict(max_q=-1), EINVAL),
    ("prefill", dict(k_stride=1 << 64), EINVAL), ("prefill", dict(kv_start=None), EINVAL), ("prefill", dict(head_dim=64), EUNSUPPORTED),
], ids=str)
def test_the_binding_refuses_what_the_calls_refuse(name, kw, status):
    name = "attn_latent_" + name
    args = dict(GOOD[name], stream=0)
    getattr(attn, name)(*[args[k] for k in ORDER[name].split()])
    args.update(kw)
    with pytest.raises(attn.AttnError) as e:
        getattr(attn, name)(*[args[k] for k in ORDER[name].split()])
    assert e.value.status == status


@pytest.mark.parametrize("name", sorted(GOOD))
def test_a_missing_struct_is_refused(name):
    assert getattr(attn.load(), name + "_from")(None) == EINVAL
