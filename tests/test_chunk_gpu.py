"""Attention of chunks of new tokens over the paged cache against the fp64
oracle (GPU required).  oracle.chunk_error_bound derives the bound; a bf16
result's own rounding (2^-8) comes on top."""

import numpy as np
import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle

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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts_of(counts):
    return [0] + np.cumsum(counts).tolist()


def paged(lens, fp8, seed, spread=1.0, extra=2):
    """A pool with shuffled pages: (cache, block table, each request's rows in fp64)."""
    held = [(n + 63) // 64 for n in lens]
    pages = sum(held) + extra
    if fp8:
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache = torch.zeros((pages, 64, 656), dtype=torch.uint8, device="cuda")
        codes = torch.randn((pages, 64, 512), generator=g, device="cuda") * 40
        cache[..., :512] = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[..., 512:516] = torch.randint(118, 124, (pages, 64, 4), generator=g, device="cuda").to(torch.uint8)
        cache[..., 528:] = rand((pages, 64, 64), seed + 1).view(torch.uint8)
        flat = oracle.fp8_rows_to_f64(cache.cpu().numpy().reshape(-1, 656))
    else:
        cache = (rand((pages, 64, 576), seed).float() * spread).bfloat16()
        flat = f64(cache).reshape(-1, 576)
    order = np.random.default_rng(seed).permutation(pages)
    table = np.full((len(lens), max(max(held), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    rows = [flat.reshape(pages, 64, 576)[table[b, :h]].reshape(-1, 576)[:n] for b, (h, n) in enumerate(zip(held, lens))]
    return cache, ints(table.tolist()), rows


def attend(*args, **kw):
    """chunk_attend, with its results' memory poisoned before and its status checked after."""
    q, status = args[0], ints([0])
    kw.setdefault("out", torch.full((q.shape[0], 128, 512), 77.0, device="cuda",
                                    dtype=torch.float32 if kw.get("out_fp32") else torch.bfloat16))
    kw.setdefault("lse", torch.full((q.shape[0], 128), 77.0, device="cuda"))
    got = m.chunk_attend(*args, status=status, **kw)
    assert int(status) == 0
    return got


def assert_chunk(out, lse, q, rows, starts, causal=True, tokens=None):
    """Against the oracle (on the listed tokens only if given)."""
    q, got, got_lse = f64(q), f64(out), f64(lse)
    if tokens is not None:  # each as a chunk of its own, with the rows that it sees
        parts, order = [], []
        for b in range(len(rows)):
            n = starts[b + 1] - starts[b]
            for t in tokens:
                if starts[b] <= t < starts[b + 1]:
                    parts.append(rows[b][:oracle.chunk_visible(n, len(rows[b]), t - starts[b], causal)])
                    order.append(t)
        q, got, got_lse, rows, starts = q[order], got[order], got_lse[order], parts, list(range(len(order) + 1))
    ref, ref_lse = oracle.chunk_attend(q, rows, starts, SCALE, causal)
    bo, bl = oracle.chunk_error_bound(q, rows, starts, SCALE, np.nan_to_num(ref), causal)
    mine = ~np.isnan(ref_lse)
    eps = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    some = np.isfinite(ref_lse) & mine
    assert np.array_equal(np.isneginf(got_lse[mine]), np.isneginf(ref_lse[mine]))
    assert (np.abs(got - ref)[some] <= bo[some] + eps * (np.abs(ref[some]) + bo[some])).all()
    assert (np.abs(got_lse[some] - ref_lse[some]) <= bl[some]).all()
    assert not got[mine & ~some].any()


CASES = [([1], [1]), ([1], [300]), ([2], [64]), ([3], [65]), ([9], [9]), ([16], [777]), ([5, 0, 8, 1], [130, 70, 8, 1]),
         ([17, 2], [129, 4000]), ([33, 1, 1, 1, 12], [1000, 63, 64, 65, 128])]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("counts,lens", CASES)
def test_chunks_match_the_oracle(counts, lens, causal, fp8):
    cache, table, rows = paged(lens, fp8, sum(lens))
    starts = starts_of(counts)
    q = rand((starts[-1], 128, 576), 3)
    out, lse = attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts), causal=causal,
                      out_fp32=len(lens) == 1)
    assert_chunk(out, lse, q, rows, starts, causal)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_tokens_of_a_long_request(fp8):
    """More pairs than units, and units that end inside a pair's tiles."""
    lens, counts = [3333, 5001], [150, 61]
    cache, table, rows = paged(lens, fp8, 5)
    q = rand((211, 128, 576), 6)
    out, lse = attend(q, cache, table, ints(lens), SCALE, token_starts=ints([0, 150, 211]), out_fp32=True)
    assert_chunk(out, lse, q, rows, [0, 150, 211], tokens=[0, 1, 2, 77, 78, 148, 149, 150, 180, 209, 210])


def test_more_pairs_than_the_plan_keeps_in_shared_memory():
    """8,400 tokens of 3 requests, one of them most."""
    lens, counts = [70, 300, 200], [8301, 1, 98]
    cache, table, rows = paged(lens, False, 31)
    starts = starts_of(counts)
    q = rand((starts[-1], 128, 576), 32)
    out, lse = attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts), causal=False)
    assert_chunk(out, lse, q, rows, starts, False, tokens=[0, 1, 4095, 4096, 8191, 8192, 8193, 8299, 8300, 8301, 8302, 8398, 8399])
    # equal queries, equal results, wherever in the line they are
    q[:8301] = q[5]
    out, lse = attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts), causal=False, out_fp32=True)
    bo, bl = oracle.chunk_error_bound(f64(q[5:6]), rows[:1], [0, 1], SCALE,
                                      oracle.chunk_attend(f64(q[5:6]), rows[:1], [0, 1], SCALE, False)[0], False)
    assert (f64((out[:8301] - out[5]).abs().amax(0)) <= 2 * bo[0]).all() and (f64((lse[:8301] - lse[5]).abs().amax(0)) <= 2 * bl[0]).all()


@pytest.mark.parametrize("out_fp32", [False, True])
def test_many_short_requests_one_after_the_other(out_fp32):
    """Segments of one tile and two, several to a unit, pairs and single tokens in turn."""
    counts = [1 + (i * 7) % 3 for i in range(300)]
    lens = [max(n, 1 + (i * 37) % 200) for i, n in enumerate(counts)]
    starts = starts_of(counts)
    cache, table, rows = paged(lens, False, 61)
    q = rand((starts[-1], 128, 576), 62)
    for _ in range(3):
        out, lse = attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts), out_fp32=out_fp32)
        assert_chunk(out, lse, q, rows, starts)


def test_a_peaked_softmax():
    lens, counts = [900, 333], [7, 20]
    cache, table, rows = paged(lens, False, 8, spread=8.0)
    q = rand((27, 128, 576), 9)
    out, lse = attend(q, cache, table, ints(lens), SCALE, token_starts=ints([0, 7, 27]), out_fp32=True)
    assert_chunk(out, lse, q, rows, [0, 7, 27])


@pytest.mark.parametrize("growth", [1.5, 4.0])
def test_scores_that_grow_along_the_cache(growth):
    """Every tile's largest score beats the last one's, up to what fp16 weights would not hold unscaled."""
    lens = [1500]
    cache, table, rows = paged(lens, False, 33)
    q = rand((5, 128, 576), 34)
    j = torch.arange(1500, device="cuda")
    place = table[0].long()[j // 64] * 64 + j % 64
    flat = cache.view(-1, 576)
    flat[place] = (flat[place].float() * (1 + growth * j[:, None] / 128)).bfloat16()
    rows = [f64(flat[place])]
    out, lse = attend(q, cache, table, ints(lens), SCALE, out_fp32=True)
    assert_chunk(out, lse, q, rows, [0, 5])


def test_equal_runs_are_the_decode_step():
    """Two tokens a request: the decode step's kernel, and (where no score beats
    the first tile's largest by 2^8, as here) its very bits."""
    lens = [130, 64, 700]
    cache, table, rows = paged(lens, False, 10)
    q = rand((6, 128, 576), 11)
    out, lse = attend(q, cache, table, ints(lens), SCALE)
    o2, l2 = m.decode_step(q.view(3, 2, 128, 576), cache, table, ints(lens), SCALE, causal=True)
    assert torch.equal(out, o2.view_as(out)) and torch.equal(lse, l2.view_as(lse))


def test_more_tokens_than_rows_see_nothing_at_first():
    cache, table, rows = paged([3, 0], False, 12)
    q = rand((9, 128, 576), 13)
    out, lse = attend(q, cache, table, ints([3, 0]), SCALE, token_starts=ints([0, 6, 9]))
    assert torch.isneginf(lse[:3]).all() and torch.isneginf(lse[6:]).all() and not out[:3].any() and not out[6:].any()
    assert_chunk(out, lse, q, rows, [0, 6, 9])


@pytest.mark.parametrize("fp8", [False, True])
def test_hidden_rows_may_hold_anything(fp8):
    """Rows behind the end, other requests' pages, and, for each token, the rows of the tokens after it."""
    lens, starts = [70, 200], [0, 5, 12]
    cache, table, rows = paged(lens, fp8, 14, extra=4)
    bad = cache.clone().view(-1, cache.shape[-1])
    keep = torch.zeros(bad.shape[0], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        keep[table[b].long()[j // 64] * 64 + j % 64] = True
    last = table[1].long()[199 // 64] * 64 + 199 % 64  # the last token's own row: nobody else sees it
    keep[last] = False
    bad[~keep] = 0x7f if fp8 else float("nan")
    q = rand((12, 128, 576), 15)
    want, wl = attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts))
    got, gl = attend(q, bad.view_as(cache), table, ints(lens), SCALE, token_starts=ints(starts))
    assert torch.equal(got[:11], want[:11]) and torch.equal(gl[:11], wl[:11])
    assert torch.isnan(got[11]).all() and torch.isnan(gl[11]).all()
    if not fp8:
        for v in (float("inf"), -float("inf")):
            bad[~keep] = v
            got, gl = attend(q, bad.view_as(cache), table, ints(lens), SCALE, token_starts=ints(starts))
            assert torch.equal(got[:11], want[:11]) and torch.equal(gl[:11], wl[:11])


def test_a_query_that_is_no_number_stays_with_its_token():
    lens, starts = [500, 4000], [0, 5, 8]
    cache, table, rows = paged(lens, False, 16)
    q = rand((8, 128, 576), 17)
    want, wl = attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts))
    q[2, 7, 5] = float("nan")
    q[6] = float("nan")
    got, gl = attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts))
    assert torch.isnan(got[2, 7]).all() and torch.isnan(gl[2, 7]) and torch.isnan(got[6]).all() and torch.isnan(gl[6]).all()
    got[2, 7], gl[2, 7], got[6], gl[6] = want[2, 7], wl[2, 7], want[6], wl[6]
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_tokens_of_no_request_are_left_alone():
    lens, starts = [100, 333], [2, 5, 12]
    cache, table, rows = paged(lens, False, 18)
    q, out, lse = rand((15, 128, 576), 19), rand((15, 128, 512), 20), rand((15, 128), 21, torch.float32)
    was = out.clone(), lse.clone()
    attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts), out=out, lse=lse)
    for a, b in zip((out, lse), was):
        assert torch.equal(a[:2], b[:2]) and torch.equal(a[12:], b[12:])
    assert_chunk(out, lse, q, rows, starts)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_tables_are_reported_and_read_as_zeros(fp8):
    lens, starts = [130, 70], [0, 4, 7]
    cache, table, rows = paged(lens, fp8, 22)
    q = rand((7, 128, 576), 23)
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad
        status = ints([0])
        out, lse = m.chunk_attend(q, cache, t, ints(lens), SCALE, token_starts=ints(starts), status=status)
        assert int(status) == m.MLA_ERR_BAD_TABLE
        zeroed = [rows[0].copy(), rows[1]]
        zeroed[0][64:128] = 0
        assert_chunk(out, lse, q, zeroed, starts)
    for bad_lens, bad_starts in (([200, 70], starts), ([-1, 70], starts), (lens, [0, 8, 7]), (lens, [0, 4, 9])):
        status = ints([0])
        m.chunk_attend(q, cache, table, ints(bad_lens), SCALE, token_starts=ints(bad_starts), max_len=130, status=status)
        assert int(status) == m.MLA_ERR_BAD_TABLE


def test_tables_in_slices_and_a_bound_of_the_lengths():
    lens, starts = [130, 70], [0, 4, 7]
    cache, table, rows = paged(lens, False, 24)
    wide = torch.full((2, 11), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + table.shape[1]] = table
    q = rand((7, 128, 576), 25)
    status = ints([0])
    out, lse = m.chunk_attend(q, cache, wide[:, 4:], ints(lens), SCALE, token_starts=ints(starts), max_len=130,
                              status=status)
    assert int(status) == 0
    assert_chunk(out, lse, q, rows, starts)


@pytest.mark.parametrize("fp8", [False, True])
def test_capture_streams_and_two_calls_at_once(fp8):
    lens, starts = [400, 999], [0, 10, 31]
    cache, table, rows = paged(lens, fp8, 26)
    q = [rand((31, 128, 576), s) for s in (27, 28)]
    want = [m.chunk_attend(x, cache, table, ints(lens), SCALE, token_starts=ints(starts)) for x in q]
    args = (cache, table, ints(lens), SCALE)
    held = q[0].clone()
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    s = ints(starts)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.chunk_attend(held, *args, token_starts=s, out=out, lse=lse)
    for i in (0, 1, 0):
        held.copy_(q[i])
        out.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[m.chunk_attend(q[i], *args, token_starts=s, stream=streams[i]) for i in (0, 1)] for _ in range(4)]
    torch.cuda.synchronize()
    for pair in got:
        for i in (0, 1):
            assert torch.equal(pair[i][0], want[i][0]) and torch.equal(pair[i][1], want[i][1])


def test_refusals():
    cache, table, _ = paged([130, 70], False, 29)
    q, lens = rand((7, 128, 576), 30), ints([130, 70])
    good = dict(token_starts=ints([0, 4, 7]))
    for kw in (dict(), dict(token_starts=ints([0, 7])), dict(good, max_len=0), dict(good, max_len=193),
               dict(good, out=torch.empty((7, 128, 512), device="cuda")), dict(good, lse=torch.empty((7, 127), device="cuda"))):
        with pytest.raises(ValueError):
            m.chunk_attend(q, cache, table, lens, SCALE, **kw)
    for args in ((q[:, :64], cache, table, lens), (q.half(), cache, table, lens), (q, cache.half(), table, lens),
                 (q, cache, table.long(), lens), (q, cache, table, lens.long()), (q, cache, table, lens[:1])):
        with pytest.raises(ValueError):
            m.chunk_attend(*args, SCALE, **good)
    with pytest.raises(m.MlaError):
        m.chunk_attend(q, cache, table, lens, SCALE, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), **good)
    with pytest.raises(m.MlaError):
        m.chunk_attend(q, cache, table, lens, 0.0, **good)
    out, lse = m.chunk_attend(q[:0], cache, table, lens, SCALE)
    assert out.shape == (0, 128, 512) and lse.shape == (0, 128)
