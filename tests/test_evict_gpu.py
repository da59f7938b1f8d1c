"""The attention weight of cached rows, the choice of the rows to keep and their
move, against the fp64 oracle (GPU required).  oracle.attention_weights derives
the bound of the first; the others are exact."""

import numpy as np
import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle
from test_chunk_gpu import SCALE, f64, ints, paged, rand, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from mla_latent_kv_09_gb300 import build
    build.build()
    m.load()
    assert torch.cuda.is_available()


# ---------------------------------------------------------------- weights

def assert_weights(got, was, decay, q, lse, rows, starts, causal=True):
    ref, bound = oracle.attention_weights(f64(q), f64(lse), rows, starts, SCALE, causal)
    got, was = f64(got), f64(was)
    for b, (w, e) in enumerate(zip(ref, bound)):
        L = len(w)
        if starts[b + 1] == starts[b]:
            assert np.array_equal(got[b], was[b])
            continue
        old = decay * was[b, :L]
        assert (np.abs(got[b, :L] - (old + w)) <= e + 2.0 ** -23 * (np.abs(old) + w)).all()
        assert np.array_equal(got[b, L:], was[b, L:])


CASES = [([1], [1]), ([1], [300]), ([2], [64]), ([3], [65]), ([9], [9]), ([16], [777]), ([5, 0, 8, 1], [130, 70, 8, 1]),
         ([17, 2], [129, 4000]), ([33, 1, 1, 1, 12], [1000, 255, 256, 257, 128]), ([1] * 40, list(range(100, 900, 20)))]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("counts,lens", CASES)
def test_weights_match_the_oracle(counts, lens, causal, fp8):
    cache, table, rows = paged(lens, fp8, sum(lens))
    starts = starts_of(counts)
    q = rand((starts[-1], 128, 576), 3)
    _, lse = m.chunk_attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts), causal=causal)
    was = rand((len(lens), table.shape[1] * 64), 4, torch.float32)
    status = ints([0])
    out = m.attention_weights(q, lse, cache, table, ints(lens), SCALE, was.clone(), token_starts=ints(starts), causal=causal,
                              decay=0.75, status=status)
    assert int(status) == 0
    assert_weights(out, was, 0.75, q, lse, rows, starts, causal)


def test_weights_in_place_elsewhere_and_none_before():
    lens, starts = [200, 77], [0, 2, 4]
    cache, table, rows = paged(lens, False, 5)
    q = rand((4, 128, 576), 6)
    _, lse = m.decode_step(q.view(2, 2, 128, 576), cache, table, ints(lens), SCALE, causal=True)
    lse = lse.view(4, 128)
    args = (q, lse, cache, table, ints(lens), SCALE)
    none = m.attention_weights(*args)
    assert none.shape == (2, 256) and not none[0, 200:].any() and not none[1, 77:].any()
    assert_weights(none, torch.zeros_like(none), 1.0, q, lse, rows, starts)
    was = rand((2, 300), 7, torch.float32)[:, 20:]  # rows wider than the lengths, strided
    mine = was.clone()
    there = torch.full((2, 333), 5.0, device="cuda")
    assert m.attention_weights(*args, was, out=there) is there
    assert torch.equal(was, mine)
    assert (there[0, 200:] == 5).all() and (there[1, 77:] == 5).all()
    assert m.attention_weights(*args, was) is was
    assert torch.equal(was[0, :200], there[0, :200]) and torch.equal(was[1, :77], there[1, :77])
    assert torch.equal(was[:, 200:], mine[:, 200:])
    assert_weights(was, mine, 1.0, q, lse, rows, starts)
    # no older weights count with a decay of 0, whatever they hold
    nan = torch.full((2, 256), float("nan"), device="cuda")
    got = m.attention_weights(*args, nan, decay=0.0, out=torch.zeros((2, 256), device="cuda"))
    assert torch.equal(got, none)


def test_heads_that_attended_to_nothing_and_wider_sums():
    lens, starts = [130], [0, 3]
    cache, table, rows = paged(lens, False, 8)
    q = rand((3, 128, 576), 9)
    _, lse = m.chunk_attend(q, cache, table, ints(lens), SCALE)
    lse[0] = -float("inf")
    lse[1, 5] = -float("inf")
    lse[2] += 1.5  # attention that saw a prefix elsewhere too
    out = m.attention_weights(q, lse, cache, table, ints(lens), SCALE)
    assert_weights(out, torch.zeros_like(out), 1.0, q, lse, rows, starts)


@pytest.mark.parametrize("fp8", [False, True])
def test_heads_without_a_result_add_nothing_whatever_their_query(fp8):
    """Padded tokens (all heads) and single heads: lse = -inf, queries NaN or
    infinite.  The others' weights are those of zeros in their place, bit for bit."""
    lens, starts = [700, 300], [0, 3, 5]
    cache, table, _ = paged(lens, fp8, 77)
    q = rand((5, 128, 576), 78)
    args = (cache, table, ints(lens), SCALE)
    _, lse = m.chunk_attend(q, *args, token_starts=ints(starts))
    none = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    none[1] = True
    none[3, ::7] = True
    none[4, 64:] = True
    lse[none] = -float("inf")
    q[none] = 0.0
    want = m.attention_weights(q, lse, *args, token_starts=ints(starts))
    q[1] = float("nan")
    q[3, ::7] = float("inf")
    q[4, 64:, 5] = -float("inf")
    got = m.attention_weights(q, lse, *args, token_starts=ints(starts))
    assert torch.equal(got, want) and bool((got[0, :697] > 0).all())


def test_weights_over_fp8_rows_of_every_scale():
    """Scales from 2^-27 to 2^33, NaN codes and scales among rows that are seen: only theirs are no numbers."""
    lens = [300]
    cache, table, _ = paged(lens, True, 33)
    g = torch.Generator(device="cuda").manual_seed(34)
    scale = torch.randint(100, 161, (4,), generator=g, device="cuda")
    scale[0], scale[1] = 100, 160
    cache[..., 512:516] = scale.to(torch.uint8)
    flat = cache.view(-1, 656)
    j = torch.arange(300, device="cuda")
    place = table[0].long()[j // 64] * 64 + j % 64
    flat[place[7], 100] = 0x7f
    flat[place[200], 511] = 0xff
    flat[place[290], 513] = 255
    rows = [oracle.fp8_rows_to_f64(flat[place].cpu().numpy())]
    # queries that undo the scales, so that all four groups count
    q = rand((3, 128, 576), 35).float()
    q[..., :512] *= torch.exp2(121.0 - scale).repeat_interleave(128)
    q = q.bfloat16()
    seen = [np.nan_to_num(rows[0], nan=0.0)]
    lse = torch.tensor(oracle.chunk_attend(f64(q), seen, [0, 3], SCALE)[1], device="cuda").float()
    got = m.attention_weights(q, lse, cache, table, ints(lens), SCALE)
    bad = np.isnan(rows[0]).any(1)
    assert bad.sum() == 3 and np.array_equal(np.isnan(f64(got)[0, :300]), bad)
    ref, bound = oracle.attention_weights(f64(q), f64(lse), seen, [0, 3], SCALE)
    assert (np.abs(f64(got)[0, :300] - ref[0])[~bad] <= bound[0][~bad]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_hidden_rows_reach_no_weight(fp8):
    lens, starts = [70, 200], [0, 5, 12]
    cache, table, rows = paged(lens, fp8, 14, extra=4)
    q = rand((12, 128, 576), 15)
    _, lse = m.chunk_attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts))
    want = m.attention_weights(q, lse, cache, table, ints(lens), SCALE, token_starts=ints(starts))
    bad = cache.clone().view(-1, cache.shape[-1])
    keep = torch.zeros(bad.shape[0], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        keep[table[b].long()[j // 64] * 64 + j % 64] = True
    bad[~keep] = 0x7f if fp8 else float("nan")
    # a row that is no number has no number as its weight, and no other row has
    j = 130
    bad[table[1].long()[j // 64] * 64 + j % 64] = 0x7f if fp8 else float("nan")
    got = m.attention_weights(q, lse, bad.view_as(cache), table, ints(lens), SCALE, token_starts=ints(starts))
    assert torch.isnan(got[1, j])
    got[1, j] = want[1, j]
    assert torch.equal(got, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_tables_of_weights_are_reported(fp8):
    lens, starts = [130, 70], [0, 4, 7]
    cache, table, rows = paged(lens, fp8, 22)
    q = rand((7, 128, 576), 23)
    _, lse = m.chunk_attend(q, cache, table, ints(lens), SCALE, token_starts=ints(starts))
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad
        status = ints([0])
        out = m.attention_weights(q, lse, cache, t, ints(lens), SCALE, token_starts=ints(starts), status=status)
        assert int(status) == m.MLA_ERR_BAD_TABLE
        zeroed = [rows[0].copy(), rows[1]]
        zeroed[0][64:128] = 0
        assert_weights(out, torch.zeros_like(out), 1.0, q, lse, zeroed, starts)
    for bad_lens, bad_starts in (([200, 70], starts), ([-1, 70], starts), (lens, [0, 8, 7]), (lens, [0, 4, 9])):
        status = ints([0])
        m.attention_weights(q, lse, cache, table, ints(bad_lens), SCALE, token_starts=ints(bad_starts), max_len=130,
                            status=status)
        assert int(status) == m.MLA_ERR_BAD_TABLE


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_are_the_same_bits_every_time(fp8):
    """Captured, on another stream, beside another call."""
    lens, starts = [700, 2222, 90], [0, 9, 40, 41]
    cache, table, _ = paged(lens, fp8, 30)
    q = rand((41, 128, 576), 31)
    s, n = ints(starts), ints(lens)
    _, lse = m.chunk_attend(q, cache, table, n, SCALE, token_starts=s)
    was = rand((3, table.shape[1] * 64), 32, torch.float32).abs()
    args = (q, lse, cache, table, n, SCALE, was)
    want = m.attention_weights(*args, token_starts=s, out=torch.zeros_like(was))
    out = torch.zeros_like(was)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.attention_weights(*args, token_starts=s, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(was) for _ in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        m.attention_weights(*args, token_starts=s, out=o, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


# ---------------------------------------------------------------- select

def assert_choice(kept, new_lens, new, weights, lens, keep, sinks, recent):
    kept, new_lens = kept.cpu().numpy(), new_lens.cpu().numpy()
    w = weights.cpu().numpy()
    for b, L in enumerate(lens):
        ref = oracle.evict_select(w[b], L, keep, sinks, recent)
        assert new_lens[b] == len(ref)
        assert np.array_equal(kept[b, :len(ref)], ref) and (kept[b, len(ref):] == -1).all()
        if new is not None:
            n = new[b].cpu().numpy()
            assert np.array_equal(n[:len(ref)], w[b, ref], equal_nan=True) and not n[len(ref):].any()


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "signs"])
@pytest.mark.parametrize("lens,keep,sinks,recent", [
    ([1], 1, 0, 0), ([2, 1, 0], 1, 0, 1), ([33, 32, 31], 17, 3, 4), ([1000, 17, 513, 1024], 200, 4, 32),
    ([1000, 999], 999, 0, 0), ([4097, 4096, 300], 1500, 0, 0), ([5000], 64, 32, 32), ([20000, 9000, 12], 7777, 5, 333)])
def test_the_choice_matches_the_oracle(lens, keep, sinks, recent, kind):
    w = rand((len(lens), max(lens)), sum(lens) + keep, torch.float32)
    if kind == "ties":
        w = (w * 2).round()
    elif kind == "equal":
        w = torch.full_like(w, 0.125)
    elif kind == "spread":
        w = torch.exp(3 * w)
    status = ints([0])
    out = m.evict_select(w, ints(lens), keep, sinks=sinks, recent=recent, status=status)
    assert int(status) == 0
    assert_choice(*out, w, lens, keep, sinks, recent)


def test_a_choice_among_special_values():
    inf = float("inf")
    w = torch.tensor([[1.0, float("nan"), inf, -0.0, 0.0, -inf, 3e-45, -3e-45, inf, float("nan"), -inf, 3e38]], device="cuda")
    for keep in range(1, 13):
        assert_choice(*m.evict_select(w, ints([12]), keep), w, [12], keep, 0, 0)


@pytest.mark.parametrize("L", [131072, 500000])
def test_a_long_choice(L):
    """Slices that shared memory does not hold among them."""
    w = torch.exp(rand((2, L), 3, torch.float32)).bfloat16().float()  # many equal ones
    lens, keep = [L, L - 12345], L // 3
    kept, new_lens, new = m.evict_select(w, ints(lens), keep, sinks=4, recent=1000)
    for b, n in enumerate(lens):
        x = w[b, :n].cpu().numpy()
        inner = np.arange(4, n - 1000)
        order = inner[np.argsort(-x[inner], kind="stable")]
        ref = np.sort(np.concatenate((np.arange(4), order[:keep - 1004], np.arange(n - 1000, n))))
        assert int(new_lens[b]) == keep and np.array_equal(kept[b].cpu().numpy(), ref)
        assert np.array_equal(new[b, :keep].cpu().numpy(), x[ref]) and not new[b, keep:].any()


def test_a_choice_among_more_rows_than_shared_memory_holds():
    L, keep = 1_000_003, 123_456
    w = torch.exp(rand((1, L), 4, torch.float32)).bfloat16().float()
    kept, new_lens, new = m.evict_select(w, ints([L]), keep, sinks=3, recent=70)
    x = w[0].cpu().numpy()
    inner = np.arange(3, L - 70)
    order = inner[np.argsort(-x[inner], kind="stable")]
    ref = np.sort(np.concatenate((np.arange(3), order[:keep - 73], np.arange(L - 70, L))))
    assert int(new_lens) == keep and np.array_equal(kept[0].cpu().numpy(), ref)
    assert np.array_equal(new[0, :keep].cpu().numpy(), x[ref]) and not new[0, keep:].any()


def test_choice_and_move_captured_and_on_another_stream():
    lens, keep = [300, 64, 700], 90
    cache, table, rows = paged(lens, False, 50)
    tables = table.shape[1]
    pages = cache.shape[0]
    both = torch.cat((cache, torch.zeros((6, 64, 576), dtype=cache.dtype, device="cuda")))
    w = [rand((3, 64 * tables), s, torch.float32) for s in (51, 52)]
    new_table = ints([[pages + 2 * b, pages + 2 * b + 1] for b in range(3)])
    n = ints(lens)

    def run(weights, to, **kw):
        kept, new_lens, _ = m.evict_select(weights, n, keep, sinks=2, recent=5, **kw)
        m.cache_compact(to, table, kept, new_lens, new_table, **kw)
        return kept, new_lens

    def check(weights, to, kept, new_lens):
        for b, L in enumerate(lens):
            ref = oracle.evict_select(weights[b].cpu().numpy(), L, keep, 2, 5)
            assert int(new_lens[b]) == len(ref) and np.array_equal(kept[b, :len(ref)].cpu().numpy(), ref)
            got = to[new_table[b].long()].reshape(-1, 576)[:len(ref)]
            assert np.array_equal(f64(got), rows[b][ref])

    held = w[0].clone()
    run(held, both)  # (memory of the graph's outputs aside)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept, new_lens = run(held, both)
    for i in (1, 0, 1):
        held.copy_(w[i])
        both[pages:].zero_()
        g.replay()
        torch.cuda.synchronize()
        check(w[i], both, kept, new_lens)
    side = torch.cuda.Stream()
    both[pages:].zero_()
    torch.cuda.synchronize()
    kept, new_lens = run(w[0], both, stream=side)
    torch.cuda.synchronize()
    check(w[0], both, kept, new_lens)


def test_choices_in_slices_and_without_weights():
    lens, keep = [300, 40], 100
    big = rand((2, 512), 40, torch.float32)
    w = big[:, 100:400]
    kept, new_lens = torch.full((2, keep), 9, dtype=torch.int32, device="cuda"), ints([9, 9])
    m.evict_select(w, ints(lens), keep, recent=10, out=(kept, new_lens, None))
    assert_choice(kept, new_lens, None, w, lens, keep, 0, 10)
    room = torch.full((2, 200), 7.0, device="cuda")
    m.evict_select(w, ints(lens), keep, recent=10, out=(kept, new_lens, room[:, :150]))
    assert_choice(kept, new_lens, room[:, :150], w, lens, keep, 0, 10)
    assert (room[:, 150:] == 7).all()
    status = ints([0])
    kept, new_lens, _ = m.evict_select(w, ints([301, -1]), keep, status=status)
    assert int(status) == m.MLA_ERR_BAD_TABLE and new_lens.tolist() == [100, 0] and (kept[1] == -1).all()
    kept, new_lens, new = m.evict_select(w[:0], ints([]), keep)
    assert kept.shape == (0, keep)
    kept, new_lens, new = m.evict_select(w[:, :0], ints([0, 0]), 3)
    assert new_lens.tolist() == [0, 0] and (kept == -1).all()


# ---------------------------------------------------------------- compact

def move_tables(lens, kept_lens, seed, extra=3):
    held, new = [(n + 63) // 64 for n in lens], [(n + 63) // 64 for n in kept_lens]
    pages = sum(held) + sum(new) + extra
    order = np.random.default_rng(seed).permutation(pages)
    tables, at = [], 0
    for counts in (held, new):
        t = np.full((len(lens), max(max(counts), 1)), -1, np.int32)
        for b, n in enumerate(counts):
            t[b, :n] = order[at:at + n]
            at += n
        tables.append(ints(t.tolist()))
    return tables[0], tables[1], pages


def rows_pool(kind, pages, seed):
    if kind == "fp8":
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randint(0, 256, (pages, 64, 656), generator=g, device="cuda", dtype=torch.uint8)
    return rand((pages, 64, 128 if kind == "index" else 576), seed)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "index"])
@pytest.mark.parametrize("lens,keep", [([1], 1), ([64, 65, 0], 64), ([300, 77, 129], 100), ([3000], 2999), ([5000, 20], 33)])
def test_rows_move_to_their_places(lens, keep, kind):
    kept_lens = [min(n, keep) for n in lens]
    table, out_table, pages = move_tables(lens, kept_lens, keep)
    cache = rows_pool(kind, pages, 50)
    rng = np.random.default_rng(keep)
    kept = np.full((len(lens), keep), -1, np.int32)
    for b, (n, k) in enumerate(zip(lens, kept_lens)):
        kept[b, :k] = np.sort(rng.permutation(n)[:k])
    was = cache.view(torch.uint8).cpu().numpy().reshape(pages * 64, -1).copy()
    want, t, o = was.copy(), table.cpu().numpy(), out_table.cpu().numpy()
    for b, k in enumerate(kept_lens):
        for i in range(k):
            j = kept[b, i]
            want[o[b, i // 64] * 64 + i % 64] = was[t[b, j // 64] * 64 + j % 64]
    status = ints([0])
    assert m.cache_compact(cache, table, ints(kept.tolist()), ints(kept_lens), out_table, status=status) is cache
    assert int(status) == 0
    assert np.array_equal(cache.view(torch.uint8).cpu().numpy().reshape(pages * 64, -1), want)


def test_rows_without_a_place_are_skipped_and_reported():
    table, out_table, pages = move_tables([200], [70], 1)
    cache = rows_pool("bf16", pages, 2)
    kept = torch.arange(70, dtype=torch.int32, device="cuda")[None] * 2
    for change, word in (("row", m.MLA_ERR_BAD_INDEX), ("far", m.MLA_ERR_BAD_INDEX), ("page", m.MLA_ERR_BAD_TABLE),
                         ("out", m.MLA_ERR_BAD_TABLE), ("len", m.MLA_ERR_BAD_TABLE)):
        c, k, t, o, n = cache.clone(), kept.clone(), table.clone(), out_table.clone(), 70
        gone = torch.zeros(70, dtype=torch.bool, device="cuda")
        if change in ("row", "far"):
            k[0, 5] = -1 if change == "row" else 64 * table.shape[1]
            gone[5] = True
        elif change == "page":
            t[0, 1] = pages
            gone[(k[0] // 64) == 1] = True
        elif change == "out":
            o[0, 0] = -7
            gone[:64] = True
        else:
            n = 71
        status = ints([0])
        m.cache_compact(c, t, k, ints([n]), o, status=status)
        assert int(status) == word, change
        want = cache.clone().view(-1, 576)
        i = torch.arange(70, device="cuda")[~gone]
        j = kept[0].long()[i]
        want[out_table[0].long()[i // 64] * 64 + i % 64] = cache.view(-1, 576)[table[0].long()[j // 64] * 64 + j % 64]
        assert torch.equal(c.view(-1, 576), want), change


def test_refusals():
    cache, table, _ = paged([130, 70], False, 29)
    q, lens, lse = rand((4, 128, 576), 30), ints([130, 70]), torch.zeros((4, 128), device="cuda")
    w, w3 = torch.zeros((2, 192), device="cuda"), torch.zeros((3, 192), device="cuda")
    for kw in (dict(out=w[:, :100]), dict(max_len=193), dict(out=w.double()), dict(token_starts=ints([0, 4]))):
        with pytest.raises(ValueError):
            m.attention_weights(q, lse, cache, table, lens, SCALE, w[:, :100] if "out" not in kw and "max_len" in kw else w,
                                **dict(kw, max_len=kw.get("max_len", 192)))
    with pytest.raises(ValueError):
        m.attention_weights(q, lse[:, :64], cache, table, lens, SCALE, w)
    with pytest.raises(m.MlaError):
        m.attention_weights(q, lse, cache, table, lens, SCALE, w, decay=float("nan"))
    for kw in (dict(keep=0), dict(keep=5, sinks=3, recent=3), dict(keep=5, sinks=-1), dict(keep=5, recent=-1)):
        with pytest.raises(ValueError):
            m.evict_select(w, lens, **kw)
    with pytest.raises(m.MlaError):  # over the weights, a row further on
        m.attention_weights(q, lse, cache, table, lens, SCALE, w3[:2], out=w3[1:])
    with pytest.raises(m.MlaError):  # into the weights themselves
        m.evict_select(w, lens, 8, out=(torch.empty((2, 8), dtype=torch.int32, device="cuda"), ints([0, 0]), w))
    kept = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        m.cache_compact(cache, table, kept, lens, table)
    with pytest.raises(ValueError):
        m.cache_compact(cache.float(), table, kept, lens, table.clone())
    with pytest.raises(ValueError):
        m.cache_compact(cache, table, kept.long(), lens, table.clone())


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fp8", [False, True])
def test_pages_beyond_32_bit_offsets(fp8):
    """A pool of more than 2^32 bytes, its last pages in use."""
    lens, starts = [300, 129], [0, 2, 5]
    cache, table, rows = paged(lens, fp8, 90)
    pages = 2 ** 32 // (64 * cache.shape[2] * cache.element_size()) + 100
    pool = torch.empty((pages,) + cache.shape[1:], dtype=cache.dtype, device="cuda")
    pool[pages - cache.shape[0]:] = cache
    far = torch.where(table >= 0, table + (pages - cache.shape[0]), table)
    q, s, n = rand((5, 128, 576), 91), ints(starts), ints(lens)
    want = m.chunk_attend(q, cache, table, n, SCALE, token_starts=s)
    got = m.chunk_attend(q, pool, far, n, SCALE, token_starts=s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w = m.attention_weights(q, got[1], pool, far, n, SCALE, token_starts=s)
    assert torch.equal(w, m.attention_weights(q, got[1], cache, table, n, SCALE, token_starts=s))
    kept, new_lens, _ = m.evict_select(w, n, 100)
    m.cache_compact(pool, far, kept, new_lens, ints([[5, 6], [7, 8]]))
    for b in range(2):
        old = pool[far[b, kept[b].long() // 64].long(), kept[b].long() % 64]
        assert torch.equal(pool[5 + 2 * b:7 + 2 * b].reshape(128, -1)[:100].view(torch.uint8), old.view(torch.uint8))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_prompt_in_chunks_whose_cache_shrinks(fp8):
    """Append, chunk attention, weights, choice and move, index keys too; then a
    decode step over the shrunk cache is one over the kept rows."""
    N, keep, B = 300, 128, 2
    inv, _ = m.rope_frequencies(64)
    pool = 2 * B * 5 + 2
    cache = torch.zeros((pool, 64, 656), dtype=torch.uint8, device="cuda") if fp8 else torch.zeros(
        (pool, 64, 576), dtype=torch.bfloat16, device="cuda")
    index = rand((pool, 64, 128), 60)
    table = torch.randperm(pool, device="cuda").to(torch.int32)[:2 * B * 5].view(2, B, 5)
    table, out_table = table[0].contiguous(), table[1].contiguous()
    latent, k_pe, q = rand((B, N, 512), 61), rand((B, N, 64), 62), rand((B, N, 128, 576), 63)
    weights, done = torch.zeros((B, 320), device="cuda"), 0
    for n in (150, 149, 1):
        pos = torch.arange(done, done + n, dtype=torch.int32, device="cuda").repeat(B)
        part = slice(done, done + n)
        m.cache_append(latent[:, part].reshape(-1, 512), k_pe[:, part].reshape(-1, 64), cache, table, pos, inv_freq=inv)
        done += n
        lens = ints([done] * B)
        x = q[:, part].reshape(-1, 128, 576).contiguous()
        out, lse = m.chunk_attend(x, cache, table, lens, SCALE)
        m.attention_weights(x, lse, cache, table, lens, SCALE, weights)
    flat = oracle.fp8_rows_to_f64(cache.cpu().numpy().reshape(-1, 656)) if fp8 else f64(cache).reshape(-1, 576)
    t = table.cpu().numpy()
    rows = [flat.reshape(pool, 64, 576)[t[b]].reshape(-1, 576)[:N] for b in range(B)]
    # every token and head has handed out a weight of one
    assert np.allclose(f64(weights.sum(1)), 128 * N, rtol=1e-4)
    kept, new_lens, new_weights = m.evict_select(weights, ints([N] * B), keep, sinks=4, recent=16)
    assert_choice(kept, new_lens, new_weights, weights, [N] * B, keep, 4, 16)
    for c in (cache, index):
        before = c.clone()
        m.cache_compact(c, table, kept, new_lens, out_table)
        k = kept[1].long()
        assert torch.equal(c[out_table[1].long()].flatten(0, 1)[:keep], before[table[1].long()].flatten(0, 1)[k])
    step = rand((B, 1, 128, 576), 64)
    o, l = m.decode_step(step, cache, out_table, new_lens, SCALE, out_fp32=True)
    chosen = [rows[b][kept[b].cpu().numpy()] for b in range(B)]
    ref, ref_lse = oracle.chunk_attend(f64(step[:, 0]), chosen, [0, 1, 2], SCALE)
    bo, bl = oracle.chunk_error_bound(f64(step[:, 0]), chosen, [0, 1, 2], SCALE, ref)
    assert (np.abs(f64(o[:, 0]) - ref) <= bo + 2.0 ** -11 * np.abs(ref)).all()
    assert (np.abs(f64(l[:, 0]) - ref_lse) <= bl).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_calls_in_a_row_are_those_that_wait(fp8):
    """The four calls, each on what the one before it leaves, launched one behind
    the other without a wait: the bits of the same calls with a wait after each."""
    lens, starts, keep = [500, 77, 1300], [0, 7, 8, 20], 200
    cache, table, _ = paged(lens, fp8, 120)
    pages, per = cache.shape[0], (keep + 63) // 64
    pool = torch.cat((cache, torch.zeros((3 * per,) + cache.shape[1:], dtype=cache.dtype, device="cuda")))
    free = ints([[pages + per * b + i for i in range(per)] for b in range(3)])
    q, s, n = rand((20, 128, 576), 121), ints(starts), ints(lens)

    def chain(wait):
        got = list(m.chunk_attend(q, pool, table, n, SCALE, token_starts=s))
        wait()
        got.append(m.attention_weights(q, got[1], pool, table, n, SCALE, token_starts=s))
        wait()
        got += m.evict_select(got[2], n, keep, sinks=2, recent=9)
        wait()
        m.cache_compact(pool, table, got[3], got[4], free)
        wait()
        got += m.chunk_attend(q, pool, free, got[4], SCALE, token_starts=s, causal=False)
        wait()
        return got

    want = chain(torch.cuda.synchronize)
    for _ in range(20):
        pool[pages:].zero_()
        got = chain(lambda: None)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
