"""The binding's own allocations when a call is given another stream than torch's
current one: scratch and outputs are that stream's memory, so calls on different
streams never share a workspace and a block that the current stream has freed is
not written while its work there may still run."""
import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from cache_util import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _chunks(seed=1):
    return si.make_chunked_case(2, 8, 2, 128, [3, 70], [9000, 100], seed=seed, page_size=16, int8=True)


def _decode(seed=1):
    return si.make_decode_case(4, 8, 2, 128, [3000, 100, 7, 4000], seed=seed)


CALLS = {"prefill_paged": (_chunks, attn.prefill_paged, "attn_prefill_paged_ex"),
         "decode": (_decode, attn.decode, "attn_decode")}


def _handles(s):
    return (s, s.cuda_stream)   # a stream, or its handle


@pytest.mark.parametrize("name", sorted(CALLS))
def test_calls_on_two_streams_have_their_own_workspace(name, monkeypatch):
    # no kernel is launched: the entry point is replaced by one that notes its workspace
    make, call, entry = CALLS[name]
    g = make().to("cuda")
    seen = []

    def note(*args):
        seen.append(next(x.data_ptr() for x in args if isinstance(x, torch.Tensor) and x.dtype == torch.uint8))

    monkeypatch.setattr(attn, entry, note)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for sa, sb in zip(_handles(a), _handles(b)):
        del seen[:]
        for s in (None, sa, sb, sa):
            call(g, stream=s)
        assert len(set(seen[:3])) == 3
        assert seen[1] == seen[3]     # in the order of its own stream a block is used again


@pytest.mark.parametrize("what", ["prefill_paged", "decode", "append", "kv_read"])
def test_outputs_do_not_take_blocks_that_the_current_stream_freed(what, monkeypatch):
    for entry in ("attn_prefill_paged_ex", "attn_decode", "attn_append", "attn_kv_read"):
        monkeypatch.setattr(attn, entry, lambda *args: None)
    start, n = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 20], [20]))
    cache = Cache("plain", 1, 2, 64, 32).to("cuda")
    x = si.f16_normal((20, 2, 64), 3).cuda()
    chunks, dec = _chunks().to("cuda"), _decode().to("cuda")
    call = {"prefill_paged": lambda s: attn.prefill_paged(chunks, stream=s),
            "decode": lambda s: attn.decode(dec, stream=s),
            "append": lambda s: attn.append(cache, x, x, x, start, n, stream=s),
            "kv_read": lambda s: attn.kv_read(cache, start, 20, kv_len=n, stream=s)[0]}[what]
    freed = call(None).data_ptr()
    assert call(None).data_ptr() == freed
    s = torch.cuda.Stream()
    for h in _handles(s):
        assert call(h).data_ptr() != freed


def test_calls_on_two_streams_without_their_contexts():
    cases = [_chunks(s) for s in (1, 2)]
    decs = [_decode(s) for s in (3, 4)]
    g = [c.to("cuda") for c in cases + decs]
    calls = [attn.prefill_paged, attn.prefill_paged, attn.decode, attn.decode]
    alone = [f(x) for f, x in zip(calls, g)]
    streams = [torch.cuda.Stream() for _ in g]
    torch.cuda.synchronize()
    outs = [[f(x, stream=s) for f, x, s in zip(calls, g, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for got in outs:
        for a, b in zip(got, alone):
            assert torch.equal(a, b)


def test_steps_on_another_stream_drop_what_they_return():
    # outputs that nothing holds any more while the stream still works on them
    cache = Cache("paged", 2, 2, 128, 512, int8=True, fill=True, seed=5).to("cuda")
    kv = torch.tensor([512, 300], dtype=torch.int32).cuda()
    start = torch.tensor([0, 512, 812], dtype=torch.int32).cuda()
    want = attn.kv_read(cache, start, 812, kv_len=kv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        attn.kv_read(cache, start, 812, kv_len=kv, stream=s)
        torch.zeros((812, 2, 128), dtype=torch.float16, device="cuda")
    got = attn.kv_read(cache, start, 812, kv_len=kv, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_capture_with_a_forked_stream():
    g = _chunks().to("cuda")
    want = attn.prefill_paged(g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = attn.prefill_paged(g, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
