"""Expansion of a shared prefix and attention over it against the fp64 oracle
(GPU required).

Expansion: bf16 products summed in fp32 (any order of 512) and rounded once:
2^-8 of the value (keys, bf16) or 2^-11 of it and half of fp16's smallest step
(values) plus 512 * 2^-23 sum |a b|.  Attention: oracle.attend_error_bound
derives its bound, and the result's own rounding (2^-8, bf16) comes on top.
"""

import math

import numpy as np
import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle
import workloads as wl

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _build():
    from mla_latent_kv_09_gb300 import build
    build.build()
    m.load()
    assert torch.cuda.is_available()


def rand(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- expansion

def assert_expanded(k_nope, k_pe, v, lat, pe, w_uk, w_uv, rows=None):
    """Against the oracle, on the listed rows only if given."""
    if rows is not None:
        k_nope, v, k_pe, lat, pe = k_nope[:, rows], v[:, rows], k_pe[rows], lat[rows], pe[rows]
    assert np.array_equal(f64(k_pe), pe)
    for got, w, eps, least in ((k_nope, w_uk, 2.0 ** -8, 0.0), (v, w_uv, 2.0 ** -11, 2.0 ** -25)):
        ref = oracle.prefix_expand(lat, f64(w))
        mass = oracle.prefix_expand(np.abs(lat), np.abs(f64(w)))
        assert (np.abs(f64(got) - ref) <= eps * np.abs(ref) + least + 512 * 2.0 ** -23 * mass).all()


def cache_and_rows(P, fp8, seed):
    """A pool with a shuffled prefix of P rows: (cache, table, latent, pe in fp64)."""
    w = wl.make_workload("p", [P], seed=seed, device="cuda", kv_fp8=fp8)
    bt = w.block_table[0].cpu().numpy()
    rows = np.array([bt[p // 64] * 64 + p % 64 for p in range(P)])
    if fp8:
        flat = oracle.fp8_rows_to_f64(w.kv.cpu().numpy().reshape(-1, 656))[rows]
    else:
        flat = f64(w.kv.view(-1, 576))[rows]
    return w.kv, w.block_table[0].contiguous(), flat[:, :512], flat[:, 512:]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("P,H", [(1, 1), (63, 3), (64, 128), (65, 2), (127, 5), (128, 1), (257, 16), (700, 7)])
def test_expansion_matches_the_oracle(P, H, fp8):
    kv, bt, lat, pe = cache_and_rows(P, fp8, P)
    w_uk, w_uv = rand((H, 512, 128), 1) * 512 ** -0.5, rand((H, 512, 128), 2) * 512 ** -0.5
    status = status_word()
    out = m.prefix_expand(kv, bt, P, w_uk, w_uv, status=status)
    assert int(status) == 0
    assert_expanded(*out, lat, pe, w_uk, w_uv)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_long_prefix_all_heads(fp8):
    P, H = 5000, 128
    kv, bt, lat, pe = cache_and_rows(P, fp8, 7)
    w_uk, w_uv = rand((H, 512, 128), 1) * 512 ** -0.5, rand((H, 512, 128), 2) * 512 ** -0.5
    out = m.prefix_expand(kv, bt, P, w_uk, w_uv)
    rows = np.array([0, 1, 255, 256, 2559, 2560, 4095, 4096, 4991, 4992, 4999])
    assert_expanded(*out, lat, pe, w_uk, w_uv, rows)
    # every row against a batched product in 32 bits (a row in a wrong place would be far off)
    rows32 = torch.tensor(lat, device="cuda", dtype=torch.float32)
    for got, w in ((out[0], w_uk), (out[2], w_uv)):
        ref = torch.matmul(rows32, w.float())
        assert float((got.float() - ref).abs().max()) <= 2.0 ** -8 * float(ref.abs().max()) + 1e-3


@pytest.mark.parametrize("fp8", [False, True])
def test_expansion_leaves_the_rows_behind_the_prefix_alone(fp8):
    P, H, R = 130, 4, 200
    kv, bt, lat, pe = cache_and_rows(P, fp8, 3)
    w_uk, w_uv = rand((H, 512, 128), 1), rand((H, 512, 128), 2)
    out = (rand((H, R, 128), 5), rand((R, 64), 6), rand((H, R, 128), 7, torch.float16))
    was = [t.clone() for t in out]
    got = m.prefix_expand(kv, bt, P, w_uk, w_uv, out=out)
    assert all(a is b for a, b in zip(got, out))
    assert torch.equal(out[0][:, P:], was[0][:, P:]) and torch.equal(out[2][:, P:], was[2][:, P:])
    assert torch.equal(out[1][P:], was[1][P:])
    assert_expanded(out[0][:, :P], out[1][:P], out[2][:, :P], lat, pe, w_uk, w_uv)


@pytest.mark.parametrize("fp8", [False, True])
def test_what_lies_behind_the_prefix_in_its_last_page_does_not_matter(fp8):
    P, H = 70, 2
    kv, bt, lat, pe = cache_and_rows(P, fp8, 3)
    w_uk, w_uv = rand((H, 512, 128), 1), rand((H, 512, 128), 2)
    tail = kv[int(bt[1]), 6:]
    tail.fill_(0x7f if fp8 else float("nan"))
    status = status_word()
    out = m.prefix_expand(kv, bt, P, w_uk, w_uv, status=status)
    assert int(status) == 0
    assert_expanded(*out, lat, pe, w_uk, w_uv)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool_and_values_outside_fp16_are_reported(fp8):
    P, H = 200, 3
    kv, bt, lat, pe = cache_and_rows(P, fp8, 4)
    w_uk, w_uv = rand((H, 512, 128), 1) * 512 ** -0.5, rand((H, 512, 128), 2) * 512 ** -0.5
    for bad in (-1, kv.shape[0], 2 ** 31 - 1):
        t, status = bt.clone(), status_word()
        t[1] = bad
        out = m.prefix_expand(kv, t, P, w_uk, w_uv, status=status)
        assert int(status) == m.MLA_ERR_BAD_TABLE
        rows = np.r_[0:64, 128:200]
        assert_expanded(*out, lat, pe, w_uk, w_uv, rows)
    big, status = w_uv.clone(), status_word()
    big[2, :, 77] = 3e4
    out = m.prefix_expand(kv, bt, P, w_uk, big, status=status)
    assert int(status) == m.MLA_ERR_VALUE_RANGE
    big[2, :, 77] = float("nan")
    status = status_word()
    out = m.prefix_expand(kv, bt, P, w_uk, big, status=status)
    assert int(status) == m.MLA_ERR_VALUE_RANGE
    assert_expanded(out[0][:2], out[1], out[2][:2], lat, pe, w_uk[:2], w_uv[:2])


def test_fp8_scales_of_every_size_and_codes_that_are_no_numbers():
    """Scales from 2^-27 to 2^23 (and 2^-127: next to nothing); a NaN code or a
    NaN scale makes its row's keys and values NaN, and no other's."""
    P, H = 300, 2
    kv, bt, lat, _ = cache_and_rows(P, True, seed=12)
    table = bt.cpu().numpy()
    place = lambda p: (int(table[p // 64]), p % 64)  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(13)
    kv[..., 512:516] = torch.randint(100, 151, kv[..., 512:516].shape, generator=g, device="cuda").to(torch.uint8)
    kv[place(70)][512:516] = 0
    kv[place(5)][300] = 0x7f
    kv[place(64)][17] = 0xff
    kv[place(299)][514] = 255
    bad, tiny = [5, 64, 299], 70
    rows = [p for p in range(P) if p not in bad and p != tiny]
    w_uk, w_uv = rand((H, 512, 128), 14) * 2.0 ** -30, rand((H, 512, 128), 15) * 2.0 ** -24
    status = status_word()
    k_nope, k_pe, v = m.prefix_expand(kv, bt, P, w_uk, w_uv, status=status)
    assert int(status) == m.MLA_ERR_VALUE_RANGE
    assert bool(k_nope[:, bad].isnan().all()) and bool(v[:, bad].isnan().all())
    assert float(k_nope[:, tiny].abs().max()) < 1e-30 and not v[:, tiny].any()
    flat = oracle.fp8_rows_to_f64(kv.cpu().numpy().reshape(-1, 656))
    held = flat[[table[p // 64] * 64 + p % 64 for p in range(P)]]
    assert_expanded(k_nope, k_pe, v, held[:, :512], held[:, 512:], w_uk, w_uv, rows)


@pytest.mark.parametrize("P,H", [(100, 3), (1000, 16), (3000, 40), (8192, 128)])
def test_fp8_rows_expand_as_the_bf16_rows_of_their_values(P, H):
    """Codes times power-of-two scales are bf16 numbers, and both caches take the
    same products in the same order: bit for bit the same keys and values, however
    often and whatever runs beside.  (Rows handed to the other SM's products
    before they are all there would differ.)"""
    kv, bt, _, _ = cache_and_rows(P, True, 31)
    scales = torch.exp2(kv[..., 512:516].float() - 127)
    lat = (kv[..., :512].view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128)) * scales[..., None]).flatten(-2)
    same = torch.cat([lat.bfloat16(), kv[..., 528:].contiguous().view(torch.bfloat16)], -1)
    assert torch.equal(same[..., :512].float(), lat)
    w_uk, w_uv = rand((H, 512, 128), 1) * 512 ** -0.5, rand((H, 512, 128), 2) * 512 ** -0.5
    want = m.prefix_expand(same, bt, P, w_uk, w_uv)
    side, noise = torch.cuda.Stream(), torch.empty(1 << 26, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        if i % 2:
            with torch.cuda.stream(side):
                noise.add_(1)
        status = status_word()
        got = m.prefix_expand(kv, bt, P, w_uk, w_uv, status=status)
        assert int(status) == 0 and all(torch.equal(x, y) for x, y in zip(got, want))
    torch.cuda.synchronize()


@pytest.mark.parametrize("fp8", [False, True])
def test_expansion_repeats_bit_for_bit(fp8):
    """Products are summed in one order, whatever the timing."""
    P, H = 1394, 128
    kv, bt, _, _ = cache_and_rows(P, fp8, 33)
    w_uk, w_uv = rand((H, 512, 128), 1) * 512 ** -0.5, rand((H, 512, 128), 2) * 512 ** -0.5
    want = m.prefix_expand(kv, bt, P, w_uk, w_uv)
    out = tuple(torch.empty_like(t) for t in want)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(2000):
        m.prefix_expand(kv, bt, P, w_uk, w_uv, out=out)
        for x, y in zip(out, want):
            differ += (x.view(torch.int16) != y.view(torch.int16)).any()
    assert int(differ) == 0


def test_keys_that_are_not_finite_are_reported():
    kv, bt, lat, pe = cache_and_rows(200, False, 4)
    w_uk, w_uv = rand((2, 512, 128), 1), rand((2, 512, 128), 2)
    for bad, expected in ((1e38, m.MLA_ERR_VALUE_RANGE), (float("inf"), m.MLA_ERR_VALUE_RANGE), (1e30, 0)):
        w, status = w_uk.clone(), status_word()
        w[1, :, 5] = bad
        m.prefix_expand(kv, bt, 200, w, w_uv, status=status)
        assert int(status) == expected


def test_rows_and_pages_beyond_32_bit_offsets():
    """More than 2^31 elements between the first and the last head's rows, and
    between the first and the last page."""
    H, R, P = 128, 140000, 300
    k_nope = torch.empty((H, R, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((H, R, 128), dtype=torch.float16, device="cuda")
    k_pe = torch.empty((R, 64), dtype=torch.bfloat16, device="cuda")
    for fp8 in (False, True):
        small, bt, lat, pe = cache_and_rows(P, fp8, 8)
        pages = 120000
        kv = torch.empty((pages, *small.shape[1:]), dtype=small.dtype, device="cuda")
        kv[pages - small.shape[0]:] = small
        w_uk, w_uv = rand((H, 512, 128), 1) * 512 ** -0.5, rand((H, 512, 128), 2) * 512 ** -0.5
        status = status_word()
        m.prefix_expand(kv, bt + (pages - small.shape[0]), P, w_uk, w_uv, out=(k_nope, k_pe, v), status=status)
        assert int(status) == 0
        last = slice(H - 1, H)
        assert_expanded(k_nope[last, :P], k_pe[:P], v[last, :P], lat, pe, w_uk[last], w_uv[last])
        del kv
    for T in (3, 140):
        q = rand((T, H, 192), 9)
        out, lse = m.prefix_attend(q[..., :128], q[..., 128:], k_nope, k_pe, v, SCALE, prefix_len=P, out_fp32=True)
        assert_attended(out, lse, q[..., :128], q[..., 128:], k_nope[:, :P], k_pe[:P], v[:, :P], tokens=np.array([0, T - 1]),
                        heads=np.array([0, H - 1]))


@pytest.mark.parametrize("P", [130, 0])
def test_more_query_rows_than_32_bit_offsets_reach(P):
    """More than 2^31 elements between the first and the last token's rows."""
    T, H = 140000, 128
    q = torch.empty((T, H, 192), dtype=torch.bfloat16, device="cuda").fill_(0.5)
    q[:2], q[-3:] = rand((2, H, 192), 1), rand((3, H, 192), 2)
    k, pe, v = rand((H, P, 128), 3), rand((P, 64), 4), rand((H, P, 128), 5, torch.float16)
    so, sl = torch.zeros((T, H, 128), dtype=torch.bfloat16, device="cuda"), torch.full((T, H), -math.inf, device="cuda")
    so[-3:], sl[-3:] = rand((3, H, 128), 6), rand((3, H), 7, torch.float32)
    ends = lambda t: torch.cat([t[:2], t[-3:]])  # noqa: E731
    suffix = ends(so), ends(sl)
    status = status_word()
    out, lse = m.prefix_attend(q[..., :128], q[..., 128:], k, pe, v, SCALE, suffix_out=so, suffix_lse=sl, out=so, lse=sl,
                               status=status)
    assert int(status) == 0
    some = ends(q)
    assert_attended(ends(out), ends(lse), some[..., :128], some[..., 128:], k, pe, v, suffix=suffix, heads=np.array([0, 64, 127]))
    # the tokens between have one query: each within the bound of its result (heads
    # are cut at other places from row block to row block, so not bit for bit)
    a = [f64(t) for t in (q[2:3, :, :128], q[2:3, :, 128:], k, pe, v)]
    ref, ref_lse = oracle.prefix_attend(*a, SCALE)
    bo, bl = oracle.attend_error_bound(*a, SCALE, ref)
    ref, bo, bl = [torch.tensor(t, device="cuda") for t in (ref, bo + 2.0 ** -8 * np.abs(ref) * 1.01, bl + 2.0 ** -21)]
    ref_lse = torch.tensor(ref_lse, device="cuda")
    for t in range(2, T - 3, 10000):
        part = slice(t, min(t + 10000, T - 3))
        assert bool(((out[part].double() - ref).abs() <= bo).all())
        assert bool(((lse[part].double() - ref_lse).abs() <= bl).all()) if P else bool((lse[part] == -math.inf).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_expansion_captured_replayed_and_beside_another(fp8):
    """A replay reads the cache as it is then; two calls at once on two streams
    do not disturb each other."""
    P, H = 500, 8
    kv, bt, _, _ = cache_and_rows(P, fp8, 21)
    kv2, bt2, _, _ = cache_and_rows(P, fp8, 22)
    w_uk, w_uv = rand((H, 512, 128), 5) / 16, rand((H, 512, 128), 6) / 16
    first, second = m.prefix_expand(kv, bt, P, w_uk, w_uv), m.prefix_expand(kv2, bt2, P, w_uk, w_uv)
    status = status_word()
    out = tuple(torch.empty_like(t) for t in first)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        m.prefix_expand(kv, bt, P, w_uk, w_uv, out=out, status=status)
    side = torch.cuda.Stream()
    for _ in range(10):
        beside = m.prefix_expand(kv2, bt2, P, w_uk, w_uv, stream=side)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, first)) and all(torch.equal(x, y) for x, y in zip(beside, second))
    kv.copy_(kv2)
    bt.copy_(bt2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, second)) and int(status) == 0


def test_expansion_refusals():
    kv, bt, _, _ = cache_and_rows(70, False, 1)
    w = rand((2, 512, 128), 1)
    k, pe, v = m.prefix_expand(kv, bt, 70, w, w)
    for bad in [lambda: m.prefix_expand(kv, bt, 129, w, w), lambda: m.prefix_expand(kv, bt, -1, w, w),
                lambda: m.prefix_expand(kv, bt[None], 70, w, w), lambda: m.prefix_expand(kv, bt, 70, w, w[:1]),
                lambda: m.prefix_expand(kv, bt, 70, w.float(), w), lambda: m.prefix_expand(kv[..., :512], bt, 70, w, w),
                lambda: m.prefix_expand(kv, bt, 70, w, w, out=(k[:, :60], pe, v)),
                lambda: m.prefix_expand(kv, bt, 70, w, w, out=(k, pe, v.bfloat16()))]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MlaError):
        m.prefix_expand(kv, bt, 70, rand((129, 512, 128), 1), rand((129, 512, 128), 1))
    assert m.prefix_expand(kv, bt, 0, w, w)[0].shape == (2, 0, 128)


# ---------------------------------------------------------------- attention

def inputs(T, H, P, seed=0, spiked=False):
    q = rand((T, H, 192), seed + 1)
    k, pe, v = rand((H, P, 128), seed + 2), rand((P, 64), seed + 3), rand((H, P, 128), seed + 4, torch.float16)
    if spiked:
        k[:, ::17] *= 8
    return q[..., :128], q[..., 128:], k, pe, v


def assert_attended(out, lse, q_nope, q_pe, k, pe, v, visible=None, suffix=(None, None), tokens=None, heads=None,
                    scale=SCALE):
    """Against the oracle, on the listed tokens and heads only if given."""
    ti = slice(None) if tokens is None else tokens
    hi = slice(None) if heads is None else heads
    a = [f64(x)[ti][:, hi] for x in (q_nope, q_pe)] + [f64(k[hi]), f64(pe), f64(v[hi])]
    vis = None if visible is None else visible.cpu().numpy()[ti]
    ref, ref_lse = oracle.prefix_attend(*a, scale, vis)
    bo, bl = oracle.attend_error_bound(*a, scale, ref, vis)
    if suffix[0] is not None:
        so, sl = f64(suffix[0])[ti][:, hi], f64(suffix[1])[ti][:, hi]
        both, total = oracle.join(ref, ref_lse, so, sl)
        # the prefix's share of the result moves with its LSE: by at most a quarter of bl
        with np.errstate(invalid="ignore"):
            share = np.where(np.isfinite(total), np.exp(np.where(np.isfinite(total), ref_lse - total, 0)), 0.0)
        share = np.where(np.isfinite(ref_lse), share, 0.0)
        seen = np.isfinite(sl) & np.isfinite(ref_lse)
        gap = np.abs(ref - np.where(np.isfinite(so), so, 0.0))
        bo = bo * share[..., None] + np.where(seen, bl / 4 + 2.0 ** -20, 2.0 ** -21)[..., None] * gap + 2.0 ** -21 * np.abs(both)
        bl = bl * share + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(total), total, 0)))
        ref, ref_lse = both, total
    got, got_lse = f64(out)[ti][:, hi], f64(lse)[ti][:, hi]
    last = 2.0 ** -8 * np.abs(ref) * 1.01 if out.dtype == torch.bfloat16 else 0.0
    nan = np.isnan(ref)  # a suffix row that counts and is not a number
    assert np.array_equal(nan, np.isnan(got))
    err = np.abs(got - ref)[~nan]
    assert (err <= (bo + last + 1e-30)[~nan]).all(), (err - (bo + last)[~nan]).max()
    fin = np.isfinite(ref_lse)
    assert np.array_equal(fin, np.isfinite(got_lse)) and (got_lse[~fin] == -np.inf).all()
    assert (np.abs(got_lse[fin] - ref_lse[fin]) <= bl[fin]).all()
    assert not got[~fin].any()


@pytest.mark.parametrize("out_fp32", [False, True])
@pytest.mark.parametrize("T,H,P", [(1, 1, 1), (1, 128, 1), (1, 3, 127), (2, 5, 128), (3, 2, 129), (64, 4, 300),
                                   (127, 2, 64), (128, 1, 256), (129, 3, 385), (255, 1, 200), (256, 2, 130),
                                   (257, 1, 513), (300, 2, 65), (600, 1, 128), (5, 16, 1000)])
def test_attention_matches_the_oracle(T, H, P, out_fp32):
    x = inputs(T, H, P, seed=T + P)
    status = status_word()
    out, lse = m.prefix_attend(*x, SCALE, out_fp32=out_fp32, status=status)
    assert int(status) == 0
    assert out.dtype == (torch.float32 if out_fp32 else torch.bfloat16)
    assert_attended(out, lse, *x)


@pytest.mark.parametrize("T,H,P", [(1, 1, 20000), (7, 1, 4097), (64, 128, 2048), (200, 128, 900), (1000, 6, 700),
                                   (2500, 2, 300), (33, 128, 8192)])
def test_long_and_large_sizes(T, H, P):
    x = inputs(T, H, P, seed=P)
    out, lse = m.prefix_attend(*x, SCALE, out_fp32=True)
    rng = np.random.default_rng(P)
    tokens = np.unique(np.r_[0, T - 1, rng.integers(0, T, 4)])
    heads = np.unique(np.r_[0, H - 1, rng.integers(0, H, 3)])
    assert_attended(out, lse, *x, tokens=tokens, heads=heads)
    # every element against the plain form in 32 bits
    q = torch.cat([x[0], x[1]], -1).float().transpose(0, 1)
    key = torch.cat([x[2].float(), x[3].float().expand(H, P, 64)], -1)
    s = torch.matmul(q, key.transpose(1, 2)) * SCALE
    ref = torch.matmul(torch.softmax(s, -1), x[4].float()).transpose(0, 1)
    assert float((out - ref).abs().max()) <= 4e-3 and float((lse - torch.logsumexp(s, -1).t()).abs().max()) <= 1e-3


@pytest.mark.parametrize("T,H,P", [(5, 2, 400), (70, 3, 1000), (300, 2, 700)])
def test_peaked_softmax(T, H, P):
    x = inputs(T, H, P, seed=2, spiked=True)
    out, lse = m.prefix_attend(*x, 1.0, out_fp32=True)  # scores of hundreds
    assert_attended(out, lse, *x, scale=1.0)


@pytest.mark.parametrize("T,H,P", [(6, 2, 300), (40, 3, 513), (290, 1, 400)])
def test_scores_that_rise_along_the_prefix(T, H, P):
    """Every tile raises the maximum: the accumulators are rescaled each time."""
    x = inputs(T, H, P, seed=3)
    ramp = torch.linspace(0, 60, P, device="cuda")[:, None]
    x[3][:] = (ramp * torch.ones(64, device="cuda")).to(torch.bfloat16)
    qp = x[1]
    qp.fill_(0.25)
    for k_pe in (x[3], x[3].flip(0).contiguous()):
        out, lse = m.prefix_attend(x[0], qp, x[2], k_pe, x[4], 1.0, out_fp32=True)
        assert_attended(out, lse, x[0], qp, x[2], k_pe, x[4], scale=1.0)


@pytest.mark.parametrize("suffix", [False, True])
@pytest.mark.parametrize("T,H,P", [(1, 4, 200), (9, 2, 300), (130, 3, 260), (300, 2, 520)])
def test_partly_shared_prefixes_and_empty_rows(T, H, P, suffix):
    x = inputs(T, H, P, seed=5)
    vis = torch.randint(0, P + 1, (T,), device="cuda", dtype=torch.int32)
    edges = torch.tensor([0, P, -5, P + 100, 1, 127, 128, 129, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=torch.int32)
    n = min(T, len(edges))
    vis[:n] = edges[:n]
    so = sl = None
    if suffix:
        so, sl = rand((T, H, 128), 6), 3 * rand((T, H), 7, torch.float32)
        sl[::3] = -math.inf
        so[::3] = float("nan")  # not read as a number where its LSE says that there is nothing
        sl[1::5] = 80.0
    out, lse = m.prefix_attend(*x, SCALE, visible=vis, suffix_out=so, suffix_lse=sl, out_fp32=True)
    assert_attended(out, lse, *x, visible=vis, suffix=(so, sl))


@pytest.mark.parametrize("T", [3, 140])
def test_tokens_that_see_nothing_at_all(T):
    H, P = 2, 300
    x = inputs(T, H, P)
    vis = torch.zeros(T, dtype=torch.int32, device="cuda")
    out, lse = m.prefix_attend(*x, SCALE, visible=vis)
    assert not out.any() and bool((lse == -math.inf).all())
    so, sl = rand((T, H, 128), 6), rand((T, H), 7, torch.float32)
    out, lse = m.prefix_attend(*x, SCALE, visible=vis, suffix_out=so, suffix_lse=sl)
    assert torch.equal(out, so) and float((lse - sl).abs().max()) <= 1e-6
    out, lse = m.prefix_attend(x[0], x[1], x[2][:, :0], x[3][:0], x[4][:, :0], SCALE, suffix_out=so, suffix_lse=sl)
    assert torch.equal(out, so) and float((lse - sl).abs().max()) <= 1e-6
    out, lse = m.prefix_attend(*x, SCALE, prefix_len=0)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("P", [100, 1000])
@pytest.mark.parametrize("T", [6, 150, 300])
def test_queries_of_padded_tokens_may_hold_anything(T, P):
    """A token that sees nothing gets the suffix's result or zeros, whatever its
    query holds, and the other tokens theirs."""
    H = 3
    x = inputs(T, H, P)
    pad = torch.arange(T, device="cuda") % 3 == 1
    vis = torch.where(pad, 0, P).to(torch.int32)
    so, sl = rand((T, H, 128), 6), math.log(P) + rand((T, H), 7, torch.float32)
    sl[::2] = -math.inf
    want = [m.prefix_attend(*x, SCALE, visible=vis), m.prefix_attend(*x, SCALE, visible=vis, suffix_out=so, suffix_lse=sl)]
    assert not want[0][0][pad].any() and bool((want[0][1][pad] == -math.inf).all())
    for bad in (float("nan"), float("inf"), 3e38):
        x[0][pad], x[1][pad] = bad, bad
        for (out, lse), kw in zip(want, ({}, dict(suffix_out=so, suffix_lse=sl))):
            got, got_lse = m.prefix_attend(*x, SCALE, visible=vis, **kw)
            assert torch.equal(got, out) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("big", [3e38, -3e38, "both"])
@pytest.mark.parametrize("T,H,P", [(6, 2, 700), (128, 1, 600), (150, 3, 1000), (300, 2, 4000)])
def test_hidden_keys_whose_scores_overflow(T, H, P, big):
    """Keys that no token sees may be any finite numbers: their scores, infinite
    or no numbers in fp32, reach no result."""
    x = inputs(T, H, P, seed=11)
    vis = torch.randint(0, 301, (T,), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(3))
    vis[:4] = torch.tensor([300, 0, 1, 256], device="cuda", dtype=torch.int32)
    want, want_lse = m.prefix_attend(*x, SCALE, visible=vis, out_fp32=True)
    assert_attended(want, want_lse, *x, visible=vis, tokens=np.arange(6))
    x[2][:, 300:] = 3e38 * torch.sign(x[2][:, 300:]) if big == "both" else big
    x[3][300:] = 3e38 if big == "both" else big
    assert bool(x[2].isfinite().all())
    out, lse = m.prefix_attend(*x, SCALE, visible=vis, out_fp32=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_suffix_joined_in_place():
    T, H, P = 20, 3, 333
    x = inputs(T, H, P)
    so, sl = rand((T, H, 128), 6), math.log(P) + rand((T, H), 7, torch.float32)
    want, want_lse = m.prefix_attend(*x, SCALE, suffix_out=so, suffix_lse=sl)
    assert_attended(want, want_lse, *x, suffix=(so, sl))
    out, lse = m.prefix_attend(*x, SCALE, suffix_out=so, suffix_lse=sl, out=so, lse=sl)
    assert out is so and lse is sl and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("how", ["plain", "fp32", "in place"])
@pytest.mark.parametrize("T,H,P", [(1, 1, 20000), (7, 1, 4097), (3, 5, 1400), (70, 16, 3001), (100, 5, 900), (256, 3, 30000),
                                   (700, 1, 5000), (300, 3, 1000), (2500, 2, 3000), (129, 100, 3000)])
def test_heads_cut_in_pieces_with_a_suffix_and_partly_visible(T, H, P, how):
    """Calls whose heads are split over SMs (few and many pieces, rows of both
    kernels, ranges that end one head and begin another): pieces that a token
    sees nothing of, the suffix's share, and its rows written over."""
    assert m.mla_prefix_attend_workspace_size(T, H, P) > 0  # split
    x = inputs(T, H, P, seed=T + H)
    vis = torch.randint(0, P + 1, (T,), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(P))
    edges = torch.tensor([P - 1, 1, 0, P, 129, 128, -1, P // 2], device="cuda", dtype=torch.int32)
    n = min(T, len(edges))
    vis[T - n:] = edges[:n]
    so, sl = rand((T, H, 128), 6), math.log(P) - 2 + 3 * rand((T, H), 7, torch.float32)
    if T > 1:
        sl[::3] = -math.inf
        so[::3] = float("nan")
    sl[T // 2, H - 1] = 90.0
    kw = dict(out=so.clone(), lse=sl.clone()) if how == "in place" else dict(out_fp32=how == "fp32")
    suffix = (kw["out"], kw["lse"]) if how == "in place" else (so, sl)
    status = status_word()
    out, lse = m.prefix_attend(*x, SCALE, visible=vis, suffix_out=suffix[0], suffix_lse=suffix[1], status=status, **kw)
    assert int(status) == 0
    rng = np.random.default_rng(P)
    tokens = np.unique(np.r_[0, T // 2, T - n + rng.permutation(n)[:5], rng.integers(0, T, 3)])
    heads = np.unique(np.r_[0, H - 1, rng.integers(0, H, 2)])
    assert_attended(out, lse, *x, visible=vis, suffix=(so, sl), tokens=tokens, heads=heads)
    # every element against the plain form in 32 bits, a head at a time
    for h in range(H):
        s = (x[0][:, h].float() @ x[2][h].float().t() + x[1][:, h].float() @ x[3].float().t()) * SCALE
        s.masked_fill_(torch.arange(P, device="cuda")[None] >= vis[:, None], -math.inf)
        own = torch.logsumexp(s, -1)
        total = torch.logaddexp(own, sl[:, h])
        base = total.masked_fill(total == -math.inf, 0)
        ref = torch.exp(s - base[:, None]) @ x[4][h].float()
        share = torch.exp(sl[:, h] - base)[:, None]
        ref += torch.where(share > 0, share * so[:, h].float(), 0)  # a row that counts and is not a number stays so
        fin = torch.isfinite(total)
        assert torch.equal(fin, torch.isfinite(lse[:, h])) and not out[~fin, h].any()
        assert float((lse[fin, h] - total[fin]).abs().max()) <= 1e-3
        nan, got = ref.isnan(), out[:, h].float()
        tol = 4e-3 + (2.0 ** -8 * ref.abs() if how != "fp32" else 0)
        assert torch.equal(nan, got.isnan()) and bool((((got - ref).abs() <= tol) | nan).all())


@pytest.mark.parametrize("T,H", [(1, 1), (20, 3), (333, 7)])
def test_no_prefix_in_place(T, H):
    """The suffix's result, written over itself."""
    x = inputs(T, H, 5)
    so, sl = rand((T, H, 128), 6), rand((T, H), 7, torch.float32)
    sl[::2] = -math.inf
    so[::2] = float("nan")
    want, want_lse = torch.where(torch.isfinite(sl)[..., None], so, 0), sl.clone()
    for _ in range(3):
        out, lse = m.prefix_attend(*x, SCALE, prefix_len=0, suffix_out=so, suffix_lse=sl, out=so, lse=sl)
        assert out is so and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("T", [4, 200])
def test_fewer_rows_than_held_and_what_lies_behind_them(T):
    """Rows behind prefix_len may hold anything."""
    H, R, P = 2, 400, 259
    x = inputs(T, H, R)
    want, want_lse = m.prefix_attend(x[0], x[1], x[2][:, :P].contiguous(), x[3][:P].contiguous(),
                                     x[4][:, :P].contiguous(), SCALE)
    for bad in (float("nan"), float("inf")):
        x[2][:, P:], x[3][P:], x[4][:, P:] = bad, bad, bad
        out, lse = m.prefix_attend(*x, SCALE, prefix_len=P)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_strided_queries():
    T, H, P = 10, 4, 150
    x = inputs(T, H, P)
    wide = rand((T, H, 576), 9)
    wide[..., 64:192], wide[..., 512:] = x[0], x[1]
    out, lse = m.prefix_attend(wide[..., 64:192], wide[..., 512:], *x[2:], SCALE)
    want, want_lse = m.prefix_attend(*x, SCALE)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("T,H", [(1, 5), (5, 1), (1, 1)])
def test_queries_whose_strides_of_a_dim_of_one_say_nothing(T, H):
    P = 150
    x = inputs(T, H, P)
    want, want_lse = m.prefix_attend(*x, SCALE)
    q = torch.cat((x[0], x[1]), -1)
    odd = torch.empty_strided(q.shape, (7 if T == 1 else 192, 7 if H == 1 else 192, 1), dtype=q.dtype, device="cuda")
    odd.copy_(q)
    assert torch.equal(odd, q)
    out, lse = m.prefix_attend(odd[..., :128], odd[..., 128:], *x[2:], SCALE)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # one head of several, one token of several
    many = rand((T + 3, H + 3, 192), 9)
    many[2:2 + T, 1:1 + H] = q
    if T == 1 or H == 1:
        part = many[2:2 + T, 1:1 + H]
        out, lse = m.prefix_attend(part[..., :128], part[..., 128:], *x[2:], SCALE)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_results_repeat_bit_for_bit():
    x = inputs(70, 16, 3001)
    a = m.prefix_attend(*x, SCALE)
    for _ in range(5):
        b = m.prefix_attend(*x, SCALE)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_replayed_on_two_streams_with_their_own_workspaces():
    T, H, P = 40, 32, 1500
    x = inputs(T, H, P)
    so, sl = rand((T, H, 128), 6), math.log(P) + rand((T, H), 7, torch.float32)
    want = m.prefix_attend(*x, SCALE, suffix_out=so, suffix_lse=sl)
    need = m.mla_prefix_attend_workspace_size(T, H, P)
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out, lse, status = torch.empty_like(so), torch.empty_like(sl), status_word()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.prefix_attend(*x, SCALE, suffix_out=so, suffix_lse=sl, workspace=ws, out=out, lse=lse, status=status)
        graphs.append((g, out, lse, status, ws))
    torch.cuda.synchronize()
    for _ in range(4):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out, lse, status, _ in graphs:
        assert int(status) == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    got = m.prefix_attend(*x, SCALE, suffix_out=so, suffix_lse=sl, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_refusals():
    x = inputs(4, 2, 50)
    so, sl = rand((4, 2, 128), 6), rand((4, 2), 7, torch.float32)
    for bad in [lambda: m.prefix_attend(x[0].float(), *x[1:], SCALE), lambda: m.prefix_attend(x[0][:3], *x[1:], SCALE),
                lambda: m.prefix_attend(*x[:2], x[2][:1], *x[3:], SCALE), lambda: m.prefix_attend(*x[:4], x[4].bfloat16(), SCALE),
                lambda: m.prefix_attend(*x[:3], x[3][:49], x[4], SCALE), lambda: m.prefix_attend(*x, SCALE, prefix_len=51),
                lambda: m.prefix_attend(*x, SCALE, prefix_len=-1), lambda: m.prefix_attend(*x, SCALE, suffix_out=so),
                lambda: m.prefix_attend(*x, SCALE, suffix_lse=sl), lambda: m.prefix_attend(*x, SCALE, suffix_out=so.float(), suffix_lse=sl),
                lambda: m.prefix_attend(*x, SCALE, visible=torch.zeros(4, device="cuda")),
                lambda: m.prefix_attend(x[0].contiguous(), *x[1:], SCALE), lambda: m.prefix_attend(*x, SCALE, out=so.float()),
                lambda: m.prefix_attend(*x[:2], x[2].transpose(1, 2).contiguous().transpose(1, 2), *x[3:], SCALE)]:
        with pytest.raises(ValueError):
            bad()
    y = inputs(4, 2, 5000)  # two heads, split over many SMs
    need = m.mla_prefix_attend_workspace_size(4, 2, 5000)
    assert need > 0
    for bad in [lambda: m.prefix_attend(*x, 0.0), lambda: m.prefix_attend(*x, float("nan")),
                lambda: m.prefix_attend(*y, SCALE, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")),
                lambda: m.prefix_attend(*y, SCALE, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises(m.MlaError):
            bad()
    assert m.prefix_attend(x[0][:0], x[1][:0], *x[2:], SCALE)[0].shape == (0, 2, 128)


# ---------------------------------------------------------------- all of them together

def test_a_context_stretched_by_yarn():
    """Queries and keys turned with YaRN's frequencies, its factor in the softmax
    scale: the scores of queries and keys multiplied by it as a whole, in fp64 on
    the rows as they are held."""
    T, H, P = 4, 3, 200
    inv, factor = m.rope_frequencies(64, yarn=40.0)
    ints = lambda a: torch.tensor(a, device="cuda", dtype=torch.int32)  # noqa: E731
    cache, table = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device="cuda"), ints([2, 0, 3, 1])
    x, q = rand((P, 576), 1), rand((T, H, 192), 2)
    m.cache_append(x[:, :512], x[:, 512:], cache, table[None], ints(np.arange(P)), inv_freq=inv)
    m.rope(q, ints(np.arange(P, P + T)), inv, offset=128, out=q)
    w_uk, w_uv = rand((H, 512, 128), 3) * 512 ** -0.5, rand((H, 512, 128), 4) * 512 ** -0.5
    k_nope, k_pe, v = m.prefix_expand(cache, table, P, w_uk, w_uv)
    out, lse = m.prefix_attend(q[..., :128], q[..., 128:], k_nope, k_pe, v, m.softmax_scale(192, factor), out_fp32=True)
    a = [f64(t) for t in (q[..., :128], q[..., 128:], k_nope, k_pe, v)]
    whole = [factor * t for t in a[:4]] + a[4:]
    ref, ref_lse = oracle.prefix_attend(*whole, 192 ** -0.5)
    bo, bl = oracle.attend_error_bound(*whole, 192 ** -0.5, ref)
    assert (np.abs(f64(out) - ref) <= bo).all() and (np.abs(f64(lse) - ref_lse) <= bl).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_step_over_a_shared_prefix(fp8):
    """Prefix tokens appended to the cache and expanded once; then a step of B
    requests: their new tokens appended, the query turned, the suffix attended
    to in the absorbed form and joined with the prefix.  Against attention over
    prefix and suffix at once, in fp64, on the cache's own rows.  The absorbed
    side rounds its query and output to bf16 (2^-8 each of values of order 1):
    the two forms may differ by a few of those, 3e-2."""
    B, H, P = 5, 128, 333
    own = [1, 70, 5, 64, 130]  # each request's tokens behind the prefix, the new one among them
    inv, _ = m.rope_frequencies(64)
    ints = lambda a: torch.tensor(a, device="cuda", dtype=torch.int32)  # noqa: E731
    pages = [(n + 63) // 64 for n in own]
    first = (P + 63) // 64
    total = first + sum(pages)
    cache = torch.zeros((total, 64, 656), dtype=torch.uint8, device="cuda") if fp8 else rand((total, 64, 576), 1)
    perm = np.random.default_rng(0).permutation(total)
    table = perm[:first]
    bt = np.zeros((B, max(pages)), np.int32)
    at = first
    for b, n in enumerate(pages):
        bt[b, :n] = perm[at:at + n]
        at += n
    weight = (1 + 0.1 * rand((512,), 2).float()).to(torch.bfloat16)
    # the prefix: positions 0 .. P - 1; its pages are a table of their own
    x = rand((P, 576), 3)
    kw = dict(norm_weight=weight, inv_freq=inv)
    m.cache_append(x[:, :512], x[:, 512:], cache, ints(table[None]), ints(np.arange(P)), **kw)
    # the suffixes: places 0 .. own - 1 of their own pages, angles P on: turned before the append
    req = np.repeat(np.arange(B), own)
    pos = np.concatenate([np.arange(n) for n in own])
    y = rand((len(req), 576), 4)
    pe = m.rope(y[:, None, 512:], ints(pos + P), inv)[:, 0]
    m.cache_append(y[:, :512], pe, cache, ints(bt), ints(pos), request_ids=ints(req), norm_weight=weight)
    w_uk, w_uv = rand((H, 512, 128), 5) * 512 ** -0.5, rand((H, 512, 128), 6) * 512 ** -0.5
    k_nope, k_pe, v = m.prefix_expand(cache, ints(table), P, w_uk, w_uv)
    # the step
    q = rand((B, H, 192), 7)
    m.rope(q, ints([P + n - 1 for n in own]), inv, offset=128, out=q)
    lens = ints(own)
    query = m.absorb_q(q[..., :128], w_uk, q[..., 128:])
    o, lse = m.decode_step(query.view(B, 1, H, 576), cache, ints(bt), lens, SCALE)
    so = m.absorb_o(o.view(B, H, 512), w_uv)
    out, total_lse = m.prefix_attend(q[..., :128], q[..., 128:], k_nope, k_pe, v, SCALE, suffix_out=so,
                                     suffix_lse=lse.view(B, H), out_fp32=True)
    rows = oracle.fp8_rows_to_f64(cache.cpu().numpy().reshape(-1, 656)) if fp8 else f64(cache.view(-1, 576))
    at = lambda t, n: np.array([t[p // 64] * 64 + p % 64 for p in range(n)])  # noqa: E731
    for b in range(B):
        r = np.concatenate([rows[at(table, P)], rows[at(bt[b], own[b])]])
        for h in (0, 77, 127):
            wk, wv = f64(w_uk[h])[None], f64(w_uv[h])[None]
            ref, ref_lse = oracle.prefix_attend(f64(q[b:b + 1, h:h + 1, :128]), f64(q[b:b + 1, h:h + 1, 128:]),
                                                oracle.prefix_expand(r[:, :512], wk), r[:, 512:],
                                                oracle.prefix_expand(r[:, :512], wv), SCALE)
            assert np.abs(f64(out[b, h]) - ref[0, 0]).max() <= 3e-2
            assert abs(float(total_lse[b, h]) - ref_lse[0, 0]) <= 2e-2
