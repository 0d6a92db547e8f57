"""GPU parity of attn_prefill_paged_ex over int8 pages against the plain 64-bit
form on code * scale: one token to several tiles, ragged and empty chunks, splits
over long caches, head groups of every size, masks that leave rows or tiles empty."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_split_kv_gb300 as attn
import seeded_inputs as si
from cache_util import chunk_reference
from parity_util import INT8_MAX_ABS, INT8_REL_L2, LSE_MAX_ABS, errors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    attn.build()
    attn.load()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    yield
    assert attn.attn_device_status() == attn.ATTN_OK


def _run(case, extra=0):
    """out, lse with `extra` rows behind the last sequence that the call must leave alone."""
    g = case.to("cuda")
    T = case.q.shape[0]
    g.q = torch.cat((g.q, torch.zeros((extra,) + tuple(g.q.shape[1:]), dtype=torch.float16, device="cuda")))
    g.q_lens = [T + extra]
    lse = torch.full((T + extra, case.n_heads), 7.0, dtype=torch.float32, device="cuda")
    out = torch.full((T + extra, case.n_heads, case.head_dim), 7.0, dtype=torch.float16, device="cuda")
    attn.prefill_paged(g, out=out, lse_out=lse)
    torch.cuda.synchronize()
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())
    return out[:T].float().cpu(), lse[:T].cpu()


def _check(case, what, extra=0):
    ref, ref_lse = chunk_reference(case)
    T = int(case.q_start[-1])
    out, lse = _run(case, extra)
    out, lse, ref, ref_lse = out[:T], lse[:T], ref[:T], ref_lse[:T]
    assert bool(torch.isfinite(out).all()), what
    mx, rel = errors(out.numpy(), ref.numpy())
    assert mx <= INT8_MAX_ABS and rel <= INT8_REL_L2, "%s: max-abs %.3g rel-L2 %.3g" % (what, mx, rel)
    empty = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), empty), what
    assert bool((out[empty] == 0).all()), what
    if not bool(empty.all()):
        assert float((lse.double() - ref_lse)[~empty].abs().max()) <= LSE_MAX_ABS, what


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page_size", [8, 16, 64, 256, 1024])
def test_chunks(D, page_size):
    case = si.make_chunked_case(4, 4, 2, D, [130, 0, 1, 37], [300, 50, 777, 0], seed=D + page_size,
                                page_size=page_size, int8=True)
    _check(case, "D=%d P=%d" % (D, page_size), extra=3)


@pytest.mark.parametrize("G,Hkv", [(1, 1), (1, 8), (2, 3), (3, 2), (4, 8), (5, 1), (7, 2), (8, 2), (12, 1), (16, 1),
                                   (33, 1), (71, 1), (128, 1), (150, 1)])
def test_head_groups(G, Hkv):
    case = si.make_chunked_case(3, G * Hkv, Hkv, 64, [3, 40, 1], [200, 11, 0], seed=G * 10 + Hkv, page_size=16,
                                int8=True)
    _check(case, "G=%d Hkv=%d" % (G, Hkv))


@pytest.mark.parametrize("D,G", [(128, 3), (128, 20), (256, 4), (256, 7), (256, 130)])
def test_head_groups_of_wide_heads(D, G):
    case = si.make_chunked_case(2, G, 1, D, [50, 9], [90, 300], seed=G, page_size=16, int8=True)
    _check(case, "D=%d G=%d" % (D, G))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_few_rows_over_a_long_cache(D, n):
    # one sequence, few rows: the keys are split over every CTA
    case = si.make_chunked_case(1, 8, 2, D, [n], [20011], seed=D + n, page_size=32, int8=True)
    _check(case, "D=%d n=%d" % (D, n))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_steps_of_ragged_lengths(D):
    ctx = [0, 1, 126, 127, 128, 129, 255, 256, 1000, 4095, 33, 7]
    case = si.make_chunked_case(12, 8, 2, D, [1] * 12, ctx, seed=D, page_size=8, int8=True)
    _check(case, "D=%d" % D)


def test_mixed_steps():
    # prompts, chunks and single tokens in one call
    case = si.make_chunked_case(6, 8, 2, 128, [300, 1, 1, 65, 1, 129], [0, 3000, 17, 500, 127, 1], seed=9,
                                page_size=16, int8=True)
    _check(case, "mixed")


def test_many_sequences():
    rng = np.random.default_rng(3)
    q = [int(x) for x in rng.integers(0, 9, 700)]
    ctx = [int(x) for x in rng.integers(0, 60, 700)]
    case = si.make_chunked_case(700, 2, 1, 64, q, ctx, seed=7, page_size=8, int8=True)
    _check(case, "700 sequences")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,softcap,scale", [(1, 0.0, 0.1), (50, 0.0, 0.1), (300, 5.0, 0.1), (0, 30.0, 0.3),
                                                  (0, 0.0, -0.1), (0, 0.0, 0.0), (129, 0.0, 0.1)])
def test_masks_and_caps(D, window, softcap, scale):
    case = si.make_chunked_case(3, 8, 2, D, [90, 1, 260], [400, 99, 1000], seed=window + D, page_size=32,
                                window=window, softcap=softcap, scale=scale, int8=True)
    _check(case, "D=%d window %d softcap %g scale %g" % (D, window, softcap, scale))


def test_saturated_cap_and_large_logits():
    case = si.make_chunked_case(2, 4, 2, 64, [20, 3], [100, 300], seed=3, page_size=16, softcap=1.0, scale=8.0,
                                int8=True)
    _check(case, "saturated")
    case = si.make_chunked_case(2, 4, 2, 128, [20, 3], [100, 300], seed=4, page_size=16, scale=3.0, int8=True)
    _check(case, "peaked softmax")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_growing_logits_rescale(D):
    # key j's scale grows along the cache, so every tile moves the running maximum
    case = si.make_chunked_case(1, 4, 2, D, [70], [1200], seed=D, page_size=16, int8=True)
    n = case.max_pages * 16
    grow = torch.linspace(0.2, 40.0, n)
    for i in range(case.max_pages):
        case.k_scales[int(case.page_table[0, i])] *= grow[i * 16:(i + 1) * 16].half()[None]
    _check(case, "D=%d" % D)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 30, 100])
def test_logits_that_step_up_every_64_keys(D, n):
    # the running maximum moves in the second half of a tile too, by more than any threshold
    case = si.make_chunked_case(2, 4, 2, D, [n, 1], [900, 411], seed=D + n, page_size=16, scale=3.2 / math.sqrt(D),
                                int8=True)
    for b in range(2):
        for i in range(-(-int(case.kv_len[b]) // 16)):   # (table entries behind them are -1)
            case.k_scales[int(case.page_table[b, i])] *= 1 + i // 4
    _check(case, "D=%d n=%d" % (D, n))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 16), (1, 17), (1, 64), (1, 65), (2, 9), (3, 5), (3, 6), (3, 20), (3, 21), (4, 5),
                                 (4, 8), (4, 16), (4, 17), (5, 4), (5, 13), (7, 8), (7, 9), (8, 2), (8, 3), (8, 9),
                                 (11, 2), (11, 4), (11, 5), (16, 1), (16, 2), (16, 4), (16, 5), (17, 2)])
def test_few_queries_by_quarters(D, G, n):
    # row counts around those that the quarters of a tile take; shorter chunks beside the longest
    case = si.make_chunked_case(4, 2 * G, 2, D, [n, 1, max(n // 2, 1), 0], [500, 130, 0, 9], seed=16 * G + n,
                                page_size=16, int8=True)
    _check(case, "D=%d G=%d n=%d" % (D, G, n), extra=2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_that_keep_no_key(D):
    # chunks longer than their caches: rows at negative positions; a sequence without tokens
    case = si.make_chunked_case(3, 4, 2, D, [40, 10, 200], [0, 5, 0], seed=29, page_size=16, int8=True)
    case.kv_len = torch.tensor([25, 0, 7], dtype=torch.int32)
    _check(case, "negative positions")
    out, lse = _run(case)
    assert bool((out[:15] == 0).all()) and bool(torch.isneginf(lse[:15]).all())


def test_lengths_past_the_table_are_clamped():
    case = si.make_chunked_case(2, 4, 2, 64, [8, 4], [56, 20], seed=30, page_size=16, int8=True)
    case.kv_len = torch.tensor([70, 24], dtype=torch.int32)   # the table holds 64: rows at 62 .. 69 keep keys below 64
    _check(case, "clamped")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", ["inf", "nan"])
def test_scales_behind_the_mask_are_not_used(D, what):
    # everything no row keeps is poisoned: pages' ends, tokens before the window, unused pages
    case = si.make_chunked_case(3, 4, 2, D, [20, 1, 3], [300, 40, 0], seed=D, page_size=32, window=64, int8=True)
    clean = chunk_reference(case)
    poison = math.inf if what == "inf" else math.nan
    used = torch.zeros(case.k.shape[0], 32, dtype=torch.bool)
    for b in range(3):
        L, n = case.kv_lens[b], case.q_lens[b]
        for p in range(max(0, L - n - 63), L):
            used[int(case.page_table[b, p // 32]), p % 32] = True
    for s in (case.k_scales, case.v_scales):
        s.copy_(torch.where(used[:, None, :], s, torch.tensor(poison).half()))
    case.k[~used], case.v[~used] = 127, -127
    out, lse = _run(case)
    mx, rel = errors(out.numpy(), clean[0].numpy())
    assert mx <= INT8_MAX_ABS and rel <= INT8_REL_L2
    assert float((lse.double() - clean[1]).abs().max()) <= LSE_MAX_ABS


@pytest.mark.parametrize("name", ["k_scales", "v_scales"])
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_a_key_that_is_not_finite_spoils_its_own_rows_only(name, what):
    # position 110 of 130, chunk 90 .. 129: rows from 110 on keep it
    case = si.make_chunked_case(1, 4, 2, 128, [40], [90], seed=6, page_size=16, int8=True)
    ref, _ = chunk_reference(case)
    getattr(case, name)[int(case.page_table[0, 110 // 16]), 0, 110 % 16] = what
    out, _ = _run(case)
    assert bool(out[20:, :2].isnan().all())
    clean = torch.ones(40, 4, dtype=torch.bool)
    clean[20:, :2] = False
    mx, rel = errors(out[clean].numpy(), ref[clean].numpy())
    assert mx <= INT8_MAX_ABS and rel <= INT8_REL_L2


def test_one_key_gives_its_value():
    case = si.make_chunked_case(1, 4, 2, 128, [1], [0], seed=5, page_size=8, int8=True)
    out, _ = _run(case)
    page = int(case.page_table[0, 0])
    v = (case.v[page, 0].double() * case.v_scales[page, :, 0].double()[:, None]).repeat_interleave(2, 0)
    # the weight is p / p: a few f32 roundings, then the output's own
    assert bool(((out[0].double() - v).abs() <= (2.0 ** -11 + 8 * 2.0 ** -24) * v.abs() + 2.0 ** -25).all())


def _two_keys(D, n, ctx, ia, ib, gap, vs_a, vs_b, seed):
    """Every key but ia and ib has a logit of -200 or less (log2 units), ia 0 and ib `gap` times a
    query's own factor of 0.75 to 1."""
    case = si.make_chunked_case(1, 16, 2, D, [n], [ctx], seed=seed, page_size=16, int8=True)
    f = 0.75 + 0.25 * torch.rand(n, 16, generator=torch.Generator().manual_seed(seed))
    case.q.zero_()
    case.q[:, :, 0] = f.half()
    case.scale = 1.0 / (127 * 1.4426950408889634)
    case.k.zero_()
    case.k[..., 0] = 127
    case.k_scales.fill_(-300.0)
    for i, logit, vs in ((ia, 0.0, vs_a), (ib, gap, vs_b)):
        page = int(case.page_table[0, i // 16])
        case.k_scales[page, :, i % 16] = logit
        case.v_scales[page, :, i % 16] = vs
    return case


def _check_two_keys(case, ia, ib, what):
    """The weight of each key is rounded to f16 (2^-11 of itself) and their sum is taken over the
    rounded weights, so an output is off by at most w_a w_b 2^-10 |v_a - v_b|, a few f32 roundings
    and its own rounding."""
    ref, ref_lse = chunk_reference(case)
    out, lse = _run(case)
    L, r = case.kv_lens[0], 127 * case.scale
    w = torch.empty(case.q.shape[0], 16, 2, dtype=torch.float64)
    v = []
    for e, i in enumerate((ia, ib)):
        page = int(case.page_table[0, i // 16])
        w[..., e] = r * case.q[:, :, 0].double() * case.k_scales[page, :, i % 16].double().repeat_interleave(8)
        v.append((case.v[page, i % 16].double() * case.v_scales[page, :, i % 16].double()[:, None]).repeat_interleave(8, 0))
    w = torch.softmax(w, -1)
    f32 = 2.0 ** -20   # the exponents' (6.5 log2 units in f32, ex2) and the quotient's roundings
    tol = (2.0 ** -11 + f32) * ref.abs() + 2.0 ** -25 + \
        ((2.0 ** -10 + f32) * w.prod(-1))[..., None] * (v[0] - v[1]).abs()[None]
    worst = ((out.double() - ref).abs() / tol).max()
    assert L > max(ia, ib) and float(worst) <= 1, "%s: %.3f of its tolerance" % (what, float(worst))
    # the sum's weights are off by 2^-11 each, and log2 by a few f32 roundings
    assert float((lse.double() - ref_lse).abs().max()) <= 2.0 ** -11 + 2.0 ** -18, what


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 300])
@pytest.mark.parametrize("ib", [70, 130, 300, 391])
def test_a_dominant_key_gives_its_value(D, n, ib):
    # key 5 sets the running maximum, and ib lies less than 2^8 above it, so its weight is no power of two
    case = _two_keys(D, n, 400, 5, ib, 6.5, 0.03, 0.03, seed=D + n + ib)
    _check_two_keys(case, 5, ib, "D=%d n=%d key %d" % (D, n, ib))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 300])
@pytest.mark.parametrize("vs", [0.0, 2.0 ** -24, -2.0 ** -24, 7 * 2.0 ** -24, 2.0 ** -18, 2.0 ** -13])
def test_a_key_of_a_tiny_value_keeps_its_mass(D, n, vs):
    # its weight for the values is far below the other key's, its share of the sum is not
    for ia, ib in ((5, 6), (5, 300), (300, 5)):
        case = _two_keys(D, n, 400, ia, ib, 0.0, vs, 0.03, seed=D + n)
        _check_two_keys(case, ia, ib, "D=%d n=%d keys %d, %d" % (D, n, ia, ib))


@pytest.mark.parametrize("Hkv", [7, 9, 12, 13, 16, 20])
def test_heads_in_several_batches(Hkv):
    # head counts that 152 CTAs take in 2 to 13 batches; runs that end inside items of any of them
    case = si.make_chunked_case(3, 2 * Hkv, Hkv, 64, [3, 70, 1], [2500, 300, 0], seed=Hkv, page_size=16, int8=True)
    _check(case, "Hkv=%d" % Hkv)
    case = si.make_chunked_case(2, Hkv, Hkv, 128, [300, 1], [1500, 6000], seed=Hkv, page_size=32, window=900, int8=True)
    _check(case, "Hkv=%d, two row tiles" % Hkv)


@pytest.mark.parametrize("Hkv,G,D", [(153, 1, 64), (160, 1, 64), (305, 2, 64), (20, 130, 64), (13, 1, 256),
                                     (153, 1, 256)])
def test_more_heads_than_ctas_and_a_partial_last_batch(Hkv, G, D):
    case = si.make_chunked_case(2, G * Hkv, Hkv, D, [5, 1], [200, 700], seed=Hkv, page_size=16, int8=True)
    _check(case, "Hkv=%d G=%d D=%d" % (Hkv, G, D))


def test_invalid_page_id_reads_as_zeros_and_is_reported():
    case = si.make_chunked_case(2, 4, 2, 64, [20, 20], [100, 100], seed=31, page_size=16, int8=True)
    ref, _ = chunk_reference(case)
    case.page_table[0, 2] = 10_000_000
    out, _ = _run(case)
    assert bool(torch.isfinite(out).all())
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    assert attn.attn_device_status() == attn.ATTN_OK
    mx, rel = errors(out[20:].numpy(), ref[20:].numpy())
    assert mx <= INT8_MAX_ABS and rel <= INT8_REL_L2
    zero = case.to("cpu")
    zero.page_table = zero.page_table.clone()
    zero.k, zero.v = torch.cat((zero.k, torch.zeros_like(zero.k[:1]))), torch.cat((zero.v, torch.zeros_like(zero.v[:1])))
    zero.k_scales = torch.cat((zero.k_scales, torch.zeros_like(zero.k_scales[:1])))
    zero.v_scales = torch.cat((zero.v_scales, torch.zeros_like(zero.v_scales[:1])))
    zero.page_table[0, 2] = zero.k.shape[0] - 1
    ref, _ = chunk_reference(zero)
    mx, rel = errors(out[:20].numpy(), ref[:20].numpy())
    assert mx <= INT8_MAX_ABS and rel <= INT8_REL_L2


def test_pages_past_unsigned_32_bits():
    # the last pages of a pool of 4.3e9 codes give what the same pages give in a small pool
    Hkv, D, P = 8, 256, 64
    case = si.make_chunked_case(2, 16, Hkv, D, [5, 70], [300, 100], seed=3, page_size=P, int8=True)
    small, n = case.to("cuda"), case.k.shape[0]
    want = attn.prefill_paged(small)
    pages = (1 << 32) // (P * Hkv * D) + n
    if torch.cuda.mem_get_info()[0] < 2 * pages * P * Hkv * D + (8 << 30):
        pytest.skip("needs 17 GB free")
    big = case.to("cuda")
    for name in ("k", "v", "k_scales", "v_scales"):
        x = getattr(small, name)
        pool = torch.zeros((pages,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
        pool[pages - n:] = x
        setattr(big, name, pool)
    big.page_table = torch.where(small.page_table >= 0, small.page_table + (pages - n), small.page_table)
    assert torch.equal(attn.prefill_paged(big), want)


@pytest.mark.parametrize("int8", [False, True])
def test_an_invalid_page_is_reported_as_the_chunk_call_s(int8):
    case = si.make_chunked_case(1, 4, 2, 64, [20], [100], seed=31, page_size=16, int8=int8)
    case.page_table[0, 2] = -5
    attn.prefill_paged(case.to("cuda"))
    assert attn.attn_device_status() == attn.ATTN_EBOUNDS
    message = attn.attn_last_error()
    assert "attn_prefill_paged" in message and "zeros" in message and "attn_decode" not in message


@pytest.mark.parametrize("D", [64, 256])
def test_f16_caches_are_attn_prefill_paged_bit_for_bit(D):
    case = si.make_chunked_case(2, 4, 2, D, [64, 130], [200, 3], seed=D, page_size=16).to("cuda")
    a = attn.prefill_paged(case)
    b = torch.empty_like(a)
    attn.attn_prefill_paged_ex(case.q, case.k, case.v, case.q_start, case.kv_len, case.page_table, 16, case.max_pages,
                               int(case.k.shape[0]), None, None, attn.ATTN_KV_F16, 2, case.total_q, case.max_q, 4, 2, D,
                               0, 0.0, case.scale, b, None, None, 0)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_repeated_calls_give_the_same_bits():
    case = si.make_chunked_case(5, 8, 2, 128, [3, 140, 1, 0, 260], [5000, 20, 777, 4, 300], seed=41, page_size=16,
                                int8=True)
    a, la = _run(case)
    for _ in range(3):
        b, lb = _run(case)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_two_streams_with_their_own_workspaces():
    cases = [si.make_chunked_case(2, 8, 2, 128, [3, 70], [9000, 100], seed=s, page_size=16, int8=True) for s in (1, 2)]
    alone = [_run(c)[0] for c in cases]
    g = [c.to("cuda") for c in cases]
    streams = [torch.cuda.Stream() for _ in g]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for c, s in zip(g, streams):
            with torch.cuda.stream(s):
                outs.append(attn.prefill_paged(c, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o.float().cpu(), alone[i % 2])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [3, 300])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(D, n):
    # the testing hook holds back the first S tile's signal for 20 ms waits: every role leaves
    # its loop, copies and MMAs in flight land, and the tensor memory is free again
    case = si.make_chunked_case(2, 8, 2, D, [n, 5], [700, 2000], seed=n + D, page_size=16, int8=True)
    g = case.to("cuda")
    assert attn.attn_testing_set_waits(20_000_000, 1) == attn.ATTN_OK
    try:
        attn.prefill_paged(g)
        status = attn.attn_device_status()
    finally:
        assert attn.attn_testing_set_waits(0, 0) == attn.ATTN_OK
    assert status == attn.ATTN_ETIMEOUT
    assert attn.attn_device_status() == attn.ATTN_OK
    _check(case, "after a timeout, D=%d n=%d" % (D, n))


@pytest.mark.parametrize("limit_ns", [20_000, 300_000, 5_000_000])
def test_waits_that_run_out_anywhere_end_every_role(limit_ns):
    # with limits this short any role's wait may be the first to run out, in any segment; every warp
    # still leaves its loops as a whole, and the next call is right
    cases = [si.make_chunked_case(3, 2 * Hkv, Hkv, D, [n, 1, 40], [900, 3000, 70], seed=n + D, page_size=16, int8=True)
             for D, Hkv, n in ((64, 3, 200), (128, 2, 5), (128, 8, 300), (256, 2, 90))]
    g = [c.to("cuda") for c in cases]
    for _ in range(3):
        assert attn.attn_testing_set_waits(limit_ns, 1) == attn.ATTN_OK
        try:
            for x in g:
                attn.prefill_paged(x)
            status = attn.attn_device_status()
        finally:
            assert attn.attn_testing_set_waits(0, 0) == attn.ATTN_OK
        assert status == attn.ATTN_ETIMEOUT
    for c in cases:
        _check(c, "after short limits, D=%d" % c.head_dim)


TRACED = """
import torch
import attention_split_kv_gb300 as attn
import seeded_inputs as si
import sys
sys.path.insert(0, "tests")
from cache_util import Cache
attn.load()
attn.prefill_paged(si.make_chunked_case(2, 8, 2, 128, [3, 2], [70, 20], seed=1, page_size=16, int8=True).to("cuda"))
attn.prefill_paged(si.make_chunked_case(2, 8, 2, 128, [300, 2], [70, 20], seed=1, page_size=16, int8=True).to("cuda"))
g = Cache("paged", 1, 2, 64, 32, int8=True).to("cuda")
x = si.f16_normal((20, 2, 64), 3).cuda()
start, n = torch.tensor([0, 20], dtype=torch.int32).cuda(), torch.tensor([20], dtype=torch.int32).cuda()
attn.append(g, x, x, x, start, n)
attn.kv_read(g, start, 20, kv_len=n)
torch.cuda.synchronize()
"""


def test_launches_are_traced():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", TRACED], cwd=root, env=dict(os.environ, ATTN_TRACE="1"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [ln for ln in r.stderr.splitlines() if ln.startswith("[libattn]")]
    assert len(lines) == 4, r.stderr
    assert "prefill8_kernel<D=128,row_tiles=1,cap=0>" in lines[0]      # 3 queries: a row tile holds 32
    assert "prefill8_kernel<D=128,row_tiles=2,cap=0>" in lines[1]
    assert "append_kernel<D=64,in=f16,q_out=f16,int8=1>" in lines[2]
    assert "kv_read_kernel<out=f16,int8=1>" in lines[3]
