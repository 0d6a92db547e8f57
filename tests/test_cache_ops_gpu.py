"""GPU parity of attn_append and attn_kv_read, and runs of the cache operators
together, against plain 64-bit forms."""
import math

import pytest
import torch

import attention_split_kv_gb300 as attn
import oracle
import seeded_inputs as si
from cache_util import F16_HALF, F16_TINY, F32_CHAIN, Cache, chunk_reference, norm_rotate, tables
from parity_util import INT8_MAX_ABS, INT8_REL_L2, assert_close, errors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _starts(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)


def _check_append(layout, lens, kv, *, Hq=4, Hkv=2, D=64, int8=False, f32=False, q_f32=False, norm=True, offset=0.0,
                  R=None, interleaved=False, page_size=16, ring=32, extra=0, scale_up=1.0, seed=1):
    """Append ragged chunks of slices of one [T, (Hq + 2 Hkv) D] projection and check
    every value of q_out and of the whole cache."""
    R = D if R is None else R
    B, T = len(lens), sum(lens)
    cache = Cache(layout, B, Hkv, D, max(kv), int8=int8, page_size=page_size, ring=ring, seed=seed)
    dt = torch.float32 if f32 else torch.float16
    qkv = (si.f32_normal((T + extra, (Hq + 2 * Hkv) * D), seed + 50) * scale_up).to(dt)
    qw, kw = (1.0 - offset + 0.2 * si.f32_normal((D,), seed + i) for i in (60, 61)) if norm else (None, None)
    cos, sin = tables(max(kv), R) if R else (None, None)
    q_start, kv_len = _starts(lens), torch.tensor(kv, dtype=torch.int32)

    g = cache.to("cuda")
    gx = qkv.cuda().view(T + extra, Hq + 2 * Hkv, D)
    up = lambda x: None if x is None else x.cuda()  # noqa: E731
    q_out = torch.full((T + extra, Hq, D), 55.0, dtype=torch.float32 if q_f32 else torch.float16, device="cuda")
    attn.append(g, gx[:, :Hq], gx[:, Hq:Hq + Hkv], gx[:, Hq + Hkv:], q_start.cuda(), kv_len.cuda(), up(qw), up(kw),
                1e-6, offset, up(cos), up(sin), interleaved, q_out)
    torch.cuda.synchronize()
    q_out, got = q_out.cpu(), g.to("cpu")
    x = qkv.view(T + extra, Hq + 2 * Hkv, D)

    def near(a, z, mag, half, tiny, what):
        tol = half * z.abs() + tiny + F32_CHAIN * mag * (1 + half)
        bad = (a.double() - z).abs() - tol
        assert float(bad.max()) <= 0, "%s: off by %.3g over its tolerance" % (what, float(bad.max()))

    written = set()
    for b in range(B):
        for i in range(lens[b]):
            t, p = int(q_start[b]) + i, kv[b] - lens[b] + i
            for h in range(Hq):
                z, mag = norm_rotate(x[t, h], qw, 1e-6, offset, cos, sin, p, interleaved)
                near(q_out[t, h], z, mag, 0.0 if q_f32 else F16_HALF, 0.0 if q_f32 else F16_TINY,
                     "q seq %d token %d head %d" % (b, i, h))
            if ring and layout == "ring" and p < kv[b] - ring:
                continue
            slot = cache.where(b, p)
            written.add(slot)
            for h in range(Hkv):
                for name, z, mag in (("k",) + norm_rotate(x[t, Hq + h], kw, 1e-6, offset, cos, sin, p, interleaved),
                                     ("v", x[t, Hq + Hkv + h].double(), torch.zeros(D, dtype=torch.float64))):
                    a = got.head(name, b, p, h)
                    what = "%s seq %d position %d head %d" % (name, b, p, h)
                    if int8:
                        s = float(getattr(got, name + "_scales")[slot[0], h, slot[1]])
                        top = float(z.abs().max())
                        assert abs(s - top / 127) <= (F16_HALF + F32_CHAIN * 2) * top / 127 + F16_TINY, what
                        # half a code, and what the f16 scale's own rounding clamps off the largest value
                        clamp = (z.abs() - 127 * s).clamp_min(0)
                        near(a, z, mag, 0.0, 0.5 * s + clamp, what)
                    else:
                        near(a, z, mag, F16_HALF, F16_TINY, what)
                    if name == "v" and int8 and not f32:
                        c, sc = si.quantize_int8_rows(x[t, Hq + Hkv + h][None].half())
                        assert torch.equal(got.v[slot[0], slot[1], h], c[0]) and s == float(sc[0]), what
    # nothing else was touched
    q_rest = q_out[T:]
    assert q_rest.numel() == 0 or bool((q_rest == 55).all())
    for name in ("k", "v"):
        full, was = getattr(got, name), getattr(cache, name)
        mask = torch.ones(full.shape[:2], dtype=torch.bool)
        for s, r in written:
            mask[s, r] = False
        assert torch.equal(full[mask], was[mask])
        if int8:
            a, c = (getattr(y, name + "_scales").transpose(1, 2) for y in (got, cache))
            assert torch.equal(a[mask], c[mask])


@pytest.mark.parametrize("layout", ["plain", "paged", "ring"])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_layouts(layout, int8, D):
    # ragged chunks with an empty one, one whole prompt, one token at the end of a cache
    _check_append(layout, [3, 0, 9, 1], [20, 5, 9, 40], D=D, int8=int8, extra=2, seed=D)


@pytest.mark.parametrize("f32,q_f32", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("int8", [False, True])
def test_append_types(f32, q_f32, int8):
    _check_append("paged", [4, 2], [10, 30], f32=f32, q_f32=q_f32, int8=int8, D=128, seed=3)


@pytest.mark.parametrize("R,interleaved", [(0, False), (16, False), (32, True), (48, False), (64, True), (128, True),
                                           (112, False)])
def test_append_rotations(R, interleaved):
    _check_append("plain", [5, 3], [70, 3], D=128, R=R, interleaved=interleaved, seed=R + 1)


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (7, 7, 64), (15, 3, 128), (5, 1, 256), (40, 8, 128), (3, 3, 256)])
def test_append_head_counts(Hq, Hkv, D):
    _check_append("paged", [2, 5], [33, 5], Hq=Hq, Hkv=Hkv, D=D, int8=True, page_size=8, offset=1.0, seed=Hq)


@pytest.mark.parametrize("layout", ["plain", "paged"])
def test_append_without_norm(layout):
    _check_append(layout, [6], [6], norm=False, int8=True, D=64, seed=8)


@pytest.mark.parametrize("page_size", [1, 2, 256, 1024])
def test_append_page_sizes(page_size):
    _check_append("paged", [5, 9], [9, 300], page_size=page_size, seed=page_size)


def test_append_chunk_longer_than_its_ring():
    # 70 tokens into 32 slots: the newest 32 are kept, each slot written once
    _check_append("ring", [70, 1, 33], [100, 64, 33], ring=32, seed=4)
    _check_append("ring", [70], [100], ring=48, int8=True, seed=4)


@pytest.mark.parametrize("f32,scale_up", [(False, 1e-6), (False, 2000.0), (True, 1e-12), (True, 1e5)])
def test_append_small_and_large_values(f32, scale_up):
    # norms bring q and k back to one; v codes keep their own scale, down to f16 subnormals and 0
    _check_append("plain", [4], [4], f32=f32, int8=True, scale_up=scale_up, seed=6)


@pytest.mark.parametrize("B", [33, 1000, 1500])
def test_append_many_sequences(B):
    # the sequence search takes one, two and three steps of 32
    lens = [(b * 7) % 3 for b in range(B)]
    lens[-1] = 2
    _check_append("plain", lens, [n + (b % 5) if n + b % 5 else 1 for b, n in enumerate(lens)], Hq=1, Hkv=1, seed=B)


def test_append_heads_that_are_not_finite_or_zero():
    D, x = 64, torch.zeros(5, 1, 64)
    x[1, 0, 3] = math.inf
    x[2, 0, 9] = math.nan
    x[3, 0, 60], x[3, 0, 0] = -math.inf, math.nan
    x[4, 0, :] = -2.0
    g = Cache("plain", 1, 1, D, 8, int8=True).to("cuda")
    v = x.half().cuda()
    attn.append(g, None, v, v, torch.tensor([0, 5], dtype=torch.int32, device="cuda"),
                torch.tensor([5], dtype=torch.int32, device="cuda"))
    k, _ = attn.kv_read(g, torch.tensor([0, 5], dtype=torch.int32, device="cuda"), 5,
                        kv_len=torch.tensor([5], dtype=torch.int32, device="cuda"), out_f32=True)
    k = k.cpu()
    assert bool((k[0] == 0).all()) and bool(k[1:4].isnan().all())
    s = torch.tensor(2.0 / 127).half().float()
    assert torch.equal(k[4, 0], -127 * s.expand(D))
    assert bool((g.k[0, 5:] == 77).all())


def test_append_leaves_out_positions_outside():
    # sequence 0 starts below position 0, sequence 1 ends above the capacity of 16,
    # and the tables hold 12 rows: all three are reported, the rest is written
    D, lens, kv = 64, [4, 4, 3], [2, 18, 14]
    cache = Cache("plain", 3, 1, D, 16, seed=2)
    g = cache.to("cuda")
    x = si.f16_normal((11, 1, D), 9).cuda()
    cos, sin = tables(18, D)
    start, kv_len = _starts(lens).cuda(), torch.tensor(kv, dtype=torch.int32).cuda()
    q = torch.full((11, 1, D), 55.0, dtype=torch.float16, device="cuda")
    attn.append(g, x, x, x, start, kv_len, q_out=q)
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    assert "position" in attn.attn_last_error()
    assert attn.attn_device_status() == attn.ATTN_OK
    kept = [2, 3, 4, 5, 8, 9, 10]      # rows of positions 0, 1 of sequence 0; 14, 15 of 1; 11, 12, 13 of 2
    out = [0, 1, 6, 7]
    assert torch.equal(q[kept], x[kept]) and bool((q[out] == 55).all())
    want = cache.v.clone()
    for b, p, t in [(0, 0, 2), (0, 1, 3), (1, 14, 4), (1, 15, 5), (2, 11, 8), (2, 12, 9), (2, 13, 10)]:
        want[b, p] = x[t].cpu()
    assert torch.equal(g.v.cpu(), want)
    g = cache.to("cuda")
    attn.append(g, x, x, x, start, kv_len, rope_cos=cos[:12].contiguous().cuda(), rope_sin=sin[:12].contiguous().cuda())
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    want = cache.v.clone()
    for b, p, t in [(0, 0, 2), (0, 1, 3), (2, 11, 8)]:
        want[b, p] = x[t].cpu()
    assert torch.equal(g.v.cpu(), want)


def test_padded_batches_are_no_error():
    # decode steps of 5 slots, two of them without a sequence (kv_len 0), and a padded chunk
    D, kv = 64, [3, 0, 16, 0, 1]
    cache = Cache("paged", 5, 1, D, 16, int8=True, page_size=8, seed=7)
    cache.page_table[1], cache.page_table[3] = -1, -1
    g = cache.to("cuda")
    x = si.f16_normal((5, 1, D), 9).cuda()
    cos, sin = (t.cuda() for t in tables(16, D))
    n = torch.tensor(kv, dtype=torch.int32).cuda()
    start = torch.arange(6, dtype=torch.int32).cuda()
    q = torch.full((5, 1, D), 55.0, dtype=torch.float16, device="cuda")
    attn.append(g, x, x, x, start, n, rope_cos=cos, rope_sin=sin, q_out=q)
    k, _ = attn.kv_read(g, start, 5, first=n - 1, kv_len=n)
    assert attn.attn_device_status() == attn.ATTN_OK
    assert bool((q[[1, 3]] == 55).all()) and bool((k[[1, 3]] == 0).all())
    assert bool((q[[0, 2, 4]] != 55).any()) and bool((k[[0, 2, 4]] != 0).any(2).all())
    start = torch.tensor([0, 4, 5, 5, 5, 5], dtype=torch.int32).cuda()    # 4 rows for the 3 tokens of sequence 0
    attn.append(g, x, x, x, start, n, rope_cos=cos, rope_sin=sin, q_out=q)
    assert attn.attn_device_status() == attn.ATTN_OK


def test_the_binding_refuses_other_types_and_strides():
    g = Cache("plain", 1, 1, 64, 8).to("cuda")
    x = si.f16_normal((2, 1, 64), 9).cuda()
    start, n = torch.tensor([0, 2], dtype=torch.int32).cuda(), torch.tensor([2], dtype=torch.int32).cuda()
    cos, sin = (t.cuda() for t in tables(8, 64))
    for kw in (dict(q_norm=torch.ones(64, device="cuda").half()), dict(kv_len=n.long()),
               dict(rope_cos=cos.half(), rope_sin=sin), dict(rope_cos=cos.t().contiguous().t(), rope_sin=sin)):
        with pytest.raises(attn.AttnError):
            attn.append(g, x, x, x, start, **{**dict(kv_len=n), **kw})
    with pytest.raises(attn.AttnError):
        attn.append(g, x.float(), x, x, start, n)
    with pytest.raises(attn.AttnError):
        attn.append(g, x, x.transpose(0, 2), x, start, n)
    with pytest.raises(attn.AttnError):
        attn.kv_read(g, start.long(), 2, kv_len=n)


@pytest.mark.parametrize("bad", [-1, 10_000_000])
def test_append_and_read_of_page_ids_outside_the_pool(bad):
    cache = Cache("paged", 1, 2, 64, 32, int8=True, page_size=8, seed=5)
    cache.page_table[0, 1] = bad
    g = cache.to("cuda")
    x = si.f16_normal((20, 2, 64), 3).cuda()
    start, n = torch.tensor([0, 20], dtype=torch.int32).cuda(), torch.tensor([20], dtype=torch.int32).cuda()
    q = attn.append(g, x, x, x, start, n)
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    assert "page" in attn.attn_last_error()
    assert torch.equal(q, x)           # q does not depend on the pages
    k, v = attn.kv_read(g, start, 20, kv_len=n)
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    assert bool((v[8:16] == 0).all()) and bool((v[:8] != 0).any()) and bool((v[16:] != 0).any())
    touched = set(cache.page_table[0, [0, 2]].tolist())
    for page in range(cache.k.shape[0]):
        assert torch.equal(g.k[page].cpu(), cache.k[page]) == (page not in touched)


def test_append_in_place_and_q_less():
    cache = Cache("plain", 1, 1, 128, 16, seed=6)
    x = si.f16_normal((9, 3, 128), 4).cuda()
    kv = si.f16_normal((9, 1, 128), 5).cuda()
    cos, sin = (t.cuda() for t in tables(16, 128))
    start, n = torch.tensor([0, 9], dtype=torch.int32).cuda(), torch.tensor([12], dtype=torch.int32).cuda()
    a, b, c = (cache.to("cuda") for _ in range(3))
    q = attn.append(a, x, kv, kv, start, n, rope_cos=cos, rope_sin=sin)
    y = x.clone()
    assert attn.append(b, y, kv, kv, start, n, rope_cos=cos, rope_sin=sin, q_out=y) is y
    assert attn.append(c, None, kv, kv, start, n, rope_cos=cos, rope_sin=sin) is None
    assert torch.equal(q, y) and torch.equal(a.k, b.k) and torch.equal(a.k, c.k) and torch.equal(a.v, c.v)


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("layout", ["plain", "paged", "ring"])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 8), (256, 1)])
def test_read(layout, int8, out_f32, D, Hkv):
    # ragged ranges: an empty one, the head, the middle, past the end, below 0
    kv, first, lens = [40, 17, 70, 9, 30], [0, 3, 33, 5, -3], [40, 0, 20, 9, 7]
    cache = Cache(layout, 5, Hkv, D, 70, int8=int8, page_size=8, ring=48, fill=True, seed=D + Hkv)
    g = cache.to("cuda")
    T = sum(lens)
    start = _starts(lens)
    k = torch.full((T + 3, Hkv, D), 5.0, dtype=torch.float32 if out_f32 else torch.float16, device="cuda")
    v = k.clone()
    P, mp, np_, cap, ring = (cache.page_size, cache.max_pages, cache.k.shape[0], cache.cap, cache.ring)
    attn.attn_kv_read(g.k, g.v, torch.tensor(kv, dtype=torch.int32).cuda(), torch.tensor(first, dtype=torch.int32).cuda(),
                      start.cuda(), g.page_table, P, mp, np_, cap, ring, g.k_scales, g.v_scales, int(int8), 5, T + 3,
                      Hkv, D, k, v, int(out_f32))
    torch.cuda.synchronize()
    for name, x in (("k", k.cpu()), ("v", v.cpu())):
        assert bool((x[T:] == 5).all())
        for b in range(5):
            for i in range(lens[b]):
                p = first[b] + i
                held = 0 <= p < kv[b] and p >= (kv[b] - 48 if layout == "ring" else 0)
                for h in range(Hkv):
                    z = cache.head(name, b, p, h) if held else torch.zeros(D, dtype=torch.float64)
                    z = z.float() if out_f32 else z.float().half()   # a product of 7 and 11 bits is exact in f32
                    assert torch.equal(x[int(start[b]) + i, h], z), (name, b, i, h)


def test_read_from_the_start_by_default():
    cache = Cache("plain", 2, 1, 64, 16, int8=True, fill=True, seed=3)
    g = cache.to("cuda")
    k, _ = attn.kv_read(g, torch.tensor([0, 4, 7], dtype=torch.int32).cuda(), 7,
                        kv_len=torch.tensor([16, 2], dtype=torch.int32).cuda(), out_f32=True)
    assert torch.equal(k[:4, 0].cpu().double(), torch.stack([cache.head("k", 0, p, 0) for p in range(4)]))
    assert torch.equal(k[4:6, 0].cpu().double(), torch.stack([cache.head("k", 1, p, 0) for p in range(2)]))
    assert bool((k[6] == 0).all())


@pytest.mark.parametrize("n", [5, 3400])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (5, 128), (7, 256)])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("out_f32", [False, True])
def test_read_of_few_and_of_many_rows(n, Hkv, D, int8, out_f32):
    # rows of one and of several passes, shared by warps or not
    cache = Cache("plain", 3, Hkv, D, 3500, int8=int8, fill=True, seed=Hkv)
    g = cache.to("cuda")
    start = torch.arange(0, 3 * n + 1, n, dtype=torch.int32).cuda()
    first = torch.tensor([0, 1, 99], dtype=torch.int32).cuda()
    k, v = attn.kv_read(g, start, 3 * n, first=first, kv_len=torch.full((3,), 3500, dtype=torch.int32).cuda(),
                        out_f32=out_f32)
    for x, name in ((k, "k"), (v, "v")):
        want = getattr(g, name).float()
        if int8:
            want = want * getattr(g, name + "_scales").float().transpose(1, 2)[..., None]
        want = torch.cat([want[b, f:f + n] for b, f in enumerate((0, 1, 99))])
        assert torch.equal(x, want if out_f32 else want.half()), name


def test_read_offsets_past_32_bits():
    # 5.4e9 codes of one sequence: the last tokens' offsets need more than 32 bits
    Hkv, D, cap = 8, 256, 1 << 20
    n = 2 * cap * Hkv * D
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("needs 16 GB free")
    g = Cache("plain", 1, Hkv, D, 8, int8=True)
    g.cap = 3 * cap // 2 // 8 * 8
    g.k = torch.zeros((1, g.cap, Hkv, D), dtype=torch.int8, device="cuda")
    g.v = torch.zeros_like(g.k)
    g.k_scales = torch.zeros((1, Hkv, g.cap), dtype=torch.float16, device="cuda")
    g.v_scales = torch.zeros_like(g.k_scales)
    x = si.f16_normal((3, Hkv, D), 8).cuda()
    start, kv = torch.tensor([0, 3], dtype=torch.int32).cuda(), torch.tensor([g.cap], dtype=torch.int32).cuda()
    assert g.cap * Hkv * D > 1 << 31
    attn.append(g, None, x, x, start, kv)
    k, v = attn.kv_read(g, start, 3, first=kv - 3, kv_len=kv)
    c, s = si.quantize_int8_rows(x.cpu())
    want = (c.float() * s.float()[..., None]).half()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    assert torch.equal(g.k[0, -3:].cpu(), c) and int(g.k[0, :-3].abs().max()) == 0


@pytest.mark.parametrize("layout", ["plain", "paged"])
def test_append_and_read_past_unsigned_32_bits(layout):
    # 4.3e9 codes of one sequence: the last tokens' offsets have more than 32 bits, signed or not
    Hkv, D, cap, P = 8, 256, (1 << 21) + 64, 64
    n = cap * Hkv * D
    assert (cap - 3) * Hkv * D > 1 << 32
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("needs 17 GB free")
    g = Cache("plain", 1, Hkv, D, 8, int8=True)
    shape = (1, cap, Hkv, D)
    if layout == "paged":
        shape = (cap // P, P, Hkv, D)
        g.page_size, g.max_pages = P, cap // P
        g.page_table = torch.arange(cap // P, dtype=torch.int32, device="cuda").view(1, -1)
    g.k, g.v = (torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2))
    g.k_scales, g.v_scales = (torch.zeros((shape[0], Hkv, shape[1]), dtype=torch.float16, device="cuda") for _ in range(2))
    x, y = (si.f16_normal((3, Hkv, D), s).cuda() for s in (8, 9))
    start, kv = torch.tensor([0, 3], dtype=torch.int32).cuda(), torch.tensor([cap], dtype=torch.int32).cuda()
    attn.append(g, None, x, y, start, kv)
    k, v = attn.kv_read(g, start, 3, first=kv - 3, kv_len=kv)
    for got, cache, z in ((k, g.k, x), (v, g.v, y)):
        c, s = si.quantize_int8_rows(z.cpu())
        assert torch.equal(got.cpu(), (c.float() * s.float()[..., None]).half())
        flat = cache.view(cap, Hkv, D)
        assert torch.equal(flat[-3:].cpu(), c) and not bool(flat[:-3].any())


# ------------------------------------------------------------------ together
def _serve(stream_of=lambda: None):
    """A prompt chunk, then three decode tokens, appended to int8 pages and attended;
    the plain form quantises the same rows (no norm, no rotation: the codes agree bit
    for bit)."""
    B, Hq, Hkv, D, P = 3, 8, 2, 128, 16
    lens, kv = [37, 5, 64], [37, 70, 64]
    cache = Cache("paged", B, Hkv, D, 96, int8=True, page_size=P, fill=True, seed=12)
    g = cache.to("cuda")
    results = []
    for step in range(4):
        T = sum(lens)
        x = si.f16_normal((T, Hq + 2 * Hkv, D), 100 + step)
        start, n = _starts(lens), torch.tensor(kv, dtype=torch.int32)
        gx, gs, gn = x.cuda(), start.cuda(), n.cuda()
        q = attn.append(g, gx[:, :Hq], gx[:, Hq:Hq + Hkv], gx[:, Hq + Hkv:], gs, gn, stream=stream_of())
        case = si.ChunkCase(q=q, k=g.k, v=g.v, q_start=gs, kv_len=gn, page_table=g.page_table, batch=B, n_heads=Hq,
                            n_kv_heads=Hkv, head_dim=D, page_size=P, max_pages=g.max_pages, max_q=max(lens),
                            scale=D ** -0.5, q_lens=list(lens), kv_lens=list(kv), k_scales=g.k_scales,
                            v_scales=g.v_scales)
        out = attn.prefill_paged(case, stream=stream_of())
        dec = None
        if step:
            dc = si.DecodeCase(q=q, k=g.k, v=g.v, kv_len=gn, batch=B, n_heads=Hq, n_kv_heads=Hkv, head_dim=D,
                               cap=g.max_pages * P, int8=True, k_scales=g.k_scales, v_scales=g.v_scales,
                               page_table=g.page_table, page_size=P, max_pages=g.max_pages, scale=D ** -0.5)
            dec = attn.decode(dc, stream=stream_of())
        torch.cuda.synchronize()
        # the plain cache
        c, s = si.quantize_int8_rows(x[:, Hq:])
        for b in range(B):
            for i in range(lens[b]):
                t, (slot, row) = int(start[b]) + i, cache.where(b, kv[b] - lens[b] + i)
                cache.k[slot, row], cache.v[slot, row] = c[t, :Hkv], c[t, Hkv:]
                cache.k_scales[slot, :, row], cache.v_scales[slot, :, row] = s[t, :Hkv], s[t, Hkv:]
        for name in ("k", "v", "k_scales", "v_scales"):
            assert torch.equal(getattr(g, name).cpu(), getattr(cache, name)), (step, name)
        cpu = si.ChunkCase(**{**case.__dict__, **dict(q=x[:, :Hq], k=cache.k, v=cache.v, q_start=start, kv_len=n,
                                                      page_table=cache.page_table, k_scales=cache.k_scales,
                                                      v_scales=cache.v_scales)})
        ref, _ = chunk_reference(cpu)
        results.append((out.float().cpu(), None if dec is None else dec.float().cpu(), ref))
        lens, kv = [1] * B, [L + 1 for L in kv]
    return results


def _close(got, ref, what):
    mx, rel = errors(got.double().numpy(), ref.numpy())
    assert mx <= INT8_MAX_ABS and rel <= INT8_REL_L2, "%s: max-abs %.3g rel-L2 %.3g" % (what, mx, rel)


def test_append_then_chunk_then_decode_steps():
    for step, (out, dec, ref) in enumerate(_serve()):
        _close(out, ref, "step %d chunk" % step)
        if dec is not None:
            _close(dec, ref, "step %d decode" % step)


def test_append_then_chunk_on_another_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for step, (out, _, ref) in enumerate(_serve(lambda: s)):
            _close(out, ref, "step %d" % step)


def test_migration_between_caches_keeps_the_values():
    # int8 pages -> rows -> an f16 ring; reading both gives the same f16 values
    src = Cache("paged", 2, 2, 128, 64, int8=True, page_size=16, fill=True, seed=21).to("cuda")
    dst = Cache("ring", 2, 2, 128, 64, ring=64, seed=22).to("cuda")
    kv = torch.tensor([64, 31], dtype=torch.int32).cuda()
    start = torch.tensor([0, 64, 95], dtype=torch.int32).cuda()
    k, v = attn.kv_read(src, start, 95, kv_len=kv)
    attn.append(dst, None, k, v, start, kv)
    k2, v2 = attn.kv_read(dst, start, 95, kv_len=kv)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_a_prompt_longer_than_its_ring_is_attended_first():
    # a sliding-window model: the prompt goes to a contiguous cache, whose rows attn_prefill takes, and
    # to the ring, whose window the next tokens decode over
    S, Hq, Hkv, D, W = 200, 4, 2, 128, 64
    x = si.f16_normal((S + 3, Hq + 2 * Hkv, D), 41).cuda()
    cos, sin = (t.cuda() for t in tables(S + 3, D))
    flat = Cache("plain", 1, Hkv, D, S, seed=1).to("cuda")
    ring = Cache("ring", 1, Hkv, D, S, ring=W, seed=2).to("cuda")

    def rows(a, b):
        return x[a:b, :Hq], x[a:b, Hq:Hq + Hkv], x[a:b, Hq + Hkv:]

    start, n = torch.tensor([0, S], dtype=torch.int32).cuda(), torch.tensor([S], dtype=torch.int32).cuda()
    q, k, v = rows(0, S)
    q = attn.append(flat, q, k, v, start, n, rope_cos=cos, rope_sin=sin)
    attn.append(ring, None, k, v, start, n, rope_cos=cos, rope_sin=sin)
    pc = si.PrefillCase(q=q, k=flat.k[0], v=flat.v[0], seq_len=S, n_heads=Hq, n_kv_heads=Hkv, head_dim=D, causal=True,
                        window=W, scale=D ** -0.5)
    out = attn.prefill(pc)
    ref, _ = oracle.prefill(pc.to("cpu"))
    assert_close(out.float().cpu().numpy().reshape(ref.shape), ref, what="prompt")
    for i in range(W):   # the ring holds what the contiguous cache does
        assert torch.equal(ring.k[0, (S - W + i) % W], flat.k[0, S - W + i])
    start = torch.tensor([0, 1], dtype=torch.int32).cuda()
    for p in range(S, S + 3):
        n = torch.tensor([p + 1], dtype=torch.int32).cuda()
        q = attn.append(ring, *rows(p, p + 1), start, n, rope_cos=cos, rope_sin=sin)
        dc = si.DecodeCase(q=q, k=ring.k, v=ring.v, kv_len=n, batch=1, n_heads=Hq, n_kv_heads=Hkv, head_dim=D, cap=W,
                           ring=W, window=W, scale=D ** -0.5)
        out = attn.decode(dc)
        ref, _ = oracle.decode(dc.to("cpu"))
        assert_close(out.float().cpu().numpy().reshape(ref.shape), ref, what="token at %d" % p)


def test_ragged_prompts_move_from_pages_to_a_ring():
    # chunks attended over int8 pages; their newest tokens then move to an f16 ring
    B, Hq, Hkv, D, P, W = 2, 4, 2, 64, 16, 48
    lens = [150, 20]
    pages = Cache("paged", B, Hkv, D, 160, int8=True, page_size=P, seed=3).to("cuda")
    ring = Cache("ring", B, Hkv, D, 160, ring=W, seed=4).to("cuda")
    x = si.f16_normal((sum(lens), Hq + 2 * Hkv, D), 42).cuda()
    start, n = _starts(lens).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    q = attn.append(pages, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], start, n)
    case = si.ChunkCase(q=q, k=pages.k, v=pages.v, q_start=start, kv_len=n, page_table=pages.page_table, batch=B,
                        n_heads=Hq, n_kv_heads=Hkv, head_dim=D, page_size=P, max_pages=pages.max_pages, max_q=150,
                        window=W, scale=0.125, q_lens=lens, kv_lens=lens, k_scales=pages.k_scales, v_scales=pages.v_scales)
    _close(attn.prefill_paged(case).float().cpu(), chunk_reference(case.to("cpu"))[0], "chunks")
    keep = [min(L, W) for L in lens]
    start = _starts(keep).cuda()
    k, v = attn.kv_read(pages, start, sum(keep), first=n - torch.tensor(keep, dtype=torch.int32).cuda(), kv_len=n)
    attn.append(ring, None, k, v, start, n)
    k2, v2 = attn.kv_read(ring, start, sum(keep), first=n - torch.tensor(keep, dtype=torch.int32).cuda(), kv_len=n)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    q = si.f16_normal((B, Hq, D), 43).cuda()
    dc = si.DecodeCase(q=q, k=ring.k, v=ring.v, kv_len=n, batch=B, n_heads=Hq, n_kv_heads=Hkv, head_dim=D, cap=W, ring=W,
                       window=W, scale=0.125)
    out = attn.decode(dc)
    ref, _ = oracle.decode(dc.to("cpu"))
    assert_close(out.float().cpu().numpy().reshape(ref.shape), ref, what="decode over the ring")


def test_append_of_f32_values_that_no_f16_scale_holds():
    D = 64
    x = torch.ones(3, 1, D)
    x[0, 0, 5], x[1, 0, 5], x[2, 0, 5] = 127 * 65504.0, -8.4e6, 1e30
    g = Cache("plain", 1, 1, D, 8, int8=True).to("cuda")
    start, n = torch.tensor([0, 3], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    attn.append(g, None, x.cuda(), x.cuda(), start, n)
    k, v = attn.kv_read(g, start, 3, kv_len=n, out_f32=True)
    want = torch.zeros(D)
    want[5] = 127 * 65504.0
    for y in (k.cpu(), v.cpu()):
        assert torch.equal(y[0, 0], want) and bool(y[1:].isnan().all())


def test_captured_step_replays_on_new_inputs():
    # append + chunk + read in one graph: new rows, lengths and pages go into the same buffers
    B, Hq, Hkv, D, P = 2, 4, 2, 64, 16
    cache = Cache("paged", B, Hkv, D, 64, int8=True, page_size=P, fill=True, seed=31)
    g = cache.to("cuda")
    x = si.f16_normal((6, Hq + 2 * Hkv, D), 1).cuda()
    start, n = torch.tensor([0, 3, 6], dtype=torch.int32).cuda(), torch.tensor([20, 9], dtype=torch.int32).cuda()
    q = torch.empty((6, Hq, D), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(attn.attn_prefill_paged_workspace_size(B, 6, Hq, Hkv, D, attn.ATTN_KV_INT8), dtype=torch.uint8,
                     device="cuda")
    case = si.ChunkCase(q=q, k=g.k, v=g.v, q_start=start, kv_len=n, page_table=g.page_table, batch=B, n_heads=Hq,
                        n_kv_heads=Hkv, head_dim=D, page_size=P, max_pages=g.max_pages, max_q=6, scale=0.125,
                        q_lens=[6], kv_lens=[], k_scales=g.k_scales, v_scales=g.v_scales)

    def step():
        attn.append(g, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], start, n, q_out=q)
        attn.prefill_paged(case, out=out, workspace=ws)
        return attn.kv_read(g, start, 6, first=n - 3, kv_len=n)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k, v = step()
    for seed, s, L in [(2, [0, 3, 6], [20, 9]), (3, [0, 1, 6], [33, 40]), (4, [0, 6, 6], [64, 1])]:
        x.copy_(si.f16_normal((6, Hq + 2 * Hkv, D), seed))
        start.copy_(torch.tensor(s, dtype=torch.int32))
        n.copy_(torch.tensor(L, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), k.clone(), v.clone()
        k2, v2 = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], k2) and torch.equal(got[2], v2)
        now = g.to("cpu")
        cpu = si.ChunkCase(**{**case.__dict__, **dict(q=q.cpu(), k=now.k, v=now.v, q_start=start.cpu(), kv_len=n.cpu(),
                                                      page_table=now.page_table, k_scales=now.k_scales,
                                                      v_scales=now.v_scales)})
        _close(out.float().cpu(), chunk_reference(cpu)[0], "replay %d" % seed)
