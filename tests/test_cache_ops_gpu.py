"""Rotary positions and the append to the paged latent cache against the fp64
oracle (GPU required).

Bounds.  A turned dim is a cos - b sin in fp32: cosine and sine are off by 2
ulp of sincospif and by the rounding of the angle's fraction of a turn to 24
bits (pi 2^-24), the factor and the three operations by 2^-24 each: within
2^-20 factor (|a| + |b|) in all; then one rounding to bf16, 2^-8 of the value.
The normed latent is three products after a sum of 512 squares (positive: off
by 2^-15 at most in any order) under a square root: 2^-14 of the value covers
it, before the rounding to bf16 (2^-8) or E4M3 (2^-4, or half of the smallest
step, 2^-10, in units of the group's scale).
"""

from fractions import Fraction

import numpy as np
import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle
import workloads as wl

pytestmark = pytest.mark.gpu


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


def assert_rope(got, x, pos, inv, offset, half, inverse, scale):
    x, inv, pos, R = f64(x), inv.cpu().numpy(), pos.cpu().numpy(), 2 * len(inv)
    ref = oracle.rope(x, pos, inv, offset, half, inverse, scale)
    got = f64(got)
    r = slice(offset, offset + R)
    part = np.abs(x[..., r])
    pair = part[..., :R // 2] + part[..., R // 2:] if half else part[..., 0::2] + part[..., 1::2]
    mass = np.concatenate([pair, pair], -1) if half else np.repeat(pair, 2, -1)
    err = np.abs(got - ref)
    assert (err[..., r] <= 2.0 ** -8 * np.abs(ref[..., r]) + 2.0 ** -20 * scale * mass).all()
    keep = np.ones(x.shape[-1], bool)
    keep[r] = False
    assert np.array_equal(got[..., keep], x[..., keep])


# ---------------------------------------------------------------- rotation

@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H,D,offset,R", [(1, 1, 64, 0, 64), (1, 128, 192, 128, 64), (3, 5, 64, 0, 64),
                                            (37, 3, 128, 0, 64), (2, 128, 128, 0, 128), (5, 7, 264, 8, 256),
                                            (130, 2, 128, 64, 32), (4, 9, 32, 8, 16), (300, 128, 64, 0, 64)])
def test_rope_matches_the_oracle(T, H, D, offset, R, half):
    x = rand((T, H, D), T * 7 + D)
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", dtype=torch.int32)
    pos[0] = 0
    inv, scale = m.rope_frequencies(R, yarn=40.0 if half else 1.0)
    assert_rope(m.rope(x, pos, inv, offset=offset, half=half, scale=scale), x, pos, inv, offset, half, False, scale)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H,D,offset,R", [(1217, 1, 64, 0, 64), (4099, 1, 16, 0, 16), (2000, 3, 192, 128, 64),
                                            (1300, 5, 264, 8, 256), (6000, 2, 64, 32, 32), (700, 17, 32, 0, 32)])
def test_many_tokens_of_few_heads(T, H, D, offset, R, half):
    """Several tokens share a CTA; in place too."""
    x = rand((T, H, D), T + D)
    pos = torch.randint(-1000, 1 << 20, (T,), device="cuda", dtype=torch.int32)
    inv, scale = m.rope_frequencies(R, yarn=4.0)
    out = m.rope(x, pos, inv, offset=offset, half=half, scale=scale)
    assert_rope(out, x, pos, inv, offset, half, False, scale)
    y = x.clone()
    assert torch.equal(m.rope(y, pos, inv, offset=offset, half=half, scale=scale, out=y), out)


@pytest.mark.parametrize("half", [False, True])
def test_far_and_negative_positions_keep_their_angle(half):
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 1 << 30, 12345678, 0], device="cuda", dtype=torch.int32)
    x = rand((6, 2, 64), 3)
    inv, _ = m.rope_frequencies(64)
    got = m.rope(x, pos, inv, half=half)
    # the oracle's own angle, p f in fp64, is off by 2^-53 of up to 2^31 radians: 2^-22, under the bound's 2^-20
    assert_rope(got, x, pos, inv, 0, half, False, 1.0)


def test_frequencies_of_whole_turns_and_above():
    inv = torch.tensor([2 * np.pi, 7.0, 0.0, 1e-9, -0.5, 3.5, 100.0, 0.25], dtype=torch.float64, device="cuda")
    x, pos = rand((9, 3, 16), 4), torch.arange(9, device="cuda", dtype=torch.int32)
    assert_rope(m.rope(x, pos, inv), x, pos, inv, 0, False, False, 1.0)


def angles(inv, pos):
    """pos * inv modulo one turn in radians, from 400 bits of pi (Machin's formula)."""
    one = 1 << 432

    def atan_inverse(x):
        total = term = one // x
        n = 1
        while term:
            term //= x * x
            n += 2
            total += term // n * (-1 if n % 4 == 3 else 1)
        return total

    pi = Fraction(4 * (4 * atan_inverse(5) - atan_inverse(239)), one)
    assert float(pi) == np.pi
    turn = lambda f, p: (Fraction(f) * int(p) / (2 * pi)) % 1  # noqa: E731
    return np.array([[2 * np.pi * float(turn(float(f), p)) for f in inv] for p in pos])


@pytest.mark.parametrize("half", [False, True])
def test_every_frequency_keeps_its_angle_at_far_positions(half):
    """Frequencies of more than a radian at far positions: p f in fp64 would be
    off by 2^-53 of it, up to a whole turn here, so the angles come from whole
    numbers; the bound is the other tests'."""
    inv = np.array([1.0, 7.0, 100.0, 2 * np.pi, -7.0, 1e-9, 12345.678, 2.0 ** 40 + 0.5, -(2.0 ** 51), 0.0, -1e-300, 5e-324,
                    3.5, -0.001, 4.0e15, 0.5])
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 1, 123456789, 1 << 30, 0, -987654321])
    x = rand((len(pos), 2, 32), 41)
    got = f64(m.rope(x, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(inv, device="cuda"), half=half))

    def check(got, x, a):
        n = a.shape[-1]
        part = lambda t: (t[..., :n], t[..., n:]) if half else (t[..., 0::2], t[..., 1::2])  # noqa: E731
        u, v = part(x)
        mass = np.abs(u) + np.abs(v)
        for y, ref in zip(part(got), (u * np.cos(a) - v * np.sin(a), u * np.sin(a) + v * np.cos(a))):
            assert (np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * mass).all()

    check(got, f64(x), angles(inv, pos)[:, None])
    # the append's rows too
    pe, inv32, at = rand((4, 64), 42), np.r_[inv, inv], np.array([5, 100000, 12345678, 64 * 300000 - 1])
    bt, cache = torch.arange(300000, device="cuda", dtype=torch.int32)[None] % 4, pool(4, False, 43)
    m.cache_append(rand((4, 512), 44), pe, cache, bt, torch.tensor(at, dtype=torch.int32, device="cuda"),
                   request_ids=torch.zeros(4, dtype=torch.int32, device="cuda"), inv_freq=torch.tensor(inv32, device="cuda"),
                   half=half)
    check(f64(cache)[at // 64 % 4, at % 64, 512:], f64(pe), angles(inv32, at))


@pytest.mark.parametrize("half", [False, True])
def test_strided_rows_in_and_out_and_what_lies_between_is_left_alone(half):
    T, H = 9, 6
    proj = rand((T, H, 192), 5)
    query = rand((T, H, 576), 6)
    before = query.clone()
    pos = torch.arange(100, 100 + T, device="cuda", dtype=torch.int32)
    inv, _ = m.rope_frequencies(64)
    out = m.rope(proj[..., 128:], pos, inv, half=half, out=query[..., 512:])
    assert out.data_ptr() == query[..., 512:].data_ptr()
    assert_rope(out, proj[..., 128:], pos, inv, 0, half, False, 1.0)
    assert torch.equal(query[..., :512], before[..., :512])
    # heads outside tokens
    other = torch.zeros((H, T, 64), dtype=torch.bfloat16, device="cuda")
    m.rope(proj[..., 128:], pos, inv, half=half, out=other.transpose(0, 1))
    assert torch.equal(other.transpose(0, 1), out)
    # one row for all heads
    assert torch.equal(m.rope(proj[:, :1, 128:].expand(T, H, 64), pos, inv, half=half)[:, 3], out[:, 0])


@pytest.mark.parametrize("T,H", [(1, 5), (5, 1), (1, 1)])
def test_strides_of_a_dim_of_one_say_nothing(T, H):
    x = rand((T, H, 64), 7)
    pos = torch.arange(9, 9 + T, device="cuda", dtype=torch.int32)
    inv, _ = m.rope_frequencies(64)
    want = m.rope(x, pos, inv)
    odd = torch.empty_strided(x.shape, (7 if T == 1 else 64, 7 if H == 1 else 64, 1), dtype=x.dtype, device="cuda")
    odd.copy_(x)
    assert torch.equal(m.rope(odd, pos, inv), want)
    assert torch.equal(m.rope(x, pos, inv, out=torch.empty_like(odd)), want)
    assert torch.equal(m.rope(odd, pos, inv, out=odd), want)


@pytest.mark.parametrize("half", [False, True])
def test_in_place_equals_out_of_place_and_leaves_the_rest(half):
    x = rand((33, 4, 192), 8)
    pos = torch.randint(0, 5000, (33,), device="cuda", dtype=torch.int32)
    inv, _ = m.rope_frequencies(64)
    want = m.rope(x, pos, inv, offset=128, half=half)
    y = x.clone()
    assert m.rope(y, pos, inv, offset=128, half=half, out=y) is y
    assert torch.equal(y, want)


@pytest.mark.parametrize("half", [False, True])
def test_inverse_is_the_gradient(half):
    """The rotation is linear: its gradient for g is the transposed map of g,
    against the oracle's formula and against differences of the oracle."""
    T, H, R = 5, 3, 64
    g = rand((T, H, R), 9)
    pos = torch.randint(0, 100000, (T,), device="cuda", dtype=torch.int32)
    inv, scale = m.rope_frequencies(R, yarn=8.0)
    got = m.rope(g, pos, inv, half=half, inverse=True, scale=scale)
    assert_rope(got, g, pos, inv, 0, half, True, scale)
    rng = np.random.default_rng(1)
    x, step = rng.standard_normal((T, H, R)), rng.standard_normal((T, H, R))
    f = lambda z: float((oracle.rope(z, pos.cpu().numpy(), inv.cpu().numpy(), 0, half, False, scale) * f64(g)).sum())  # noqa: E731
    ref = oracle.rope(f64(g), pos.cpu().numpy(), inv.cpu().numpy(), 0, half, True, scale)
    assert (f(x + 1e-3 * step) - f(x - 1e-3 * step)) / 2e-3 == pytest.approx(float((ref * step).sum()), rel=1e-8)


def test_rope_refusals():
    x, pos = rand((4, 2, 64), 1), torch.zeros(4, dtype=torch.int32, device="cuda")
    inv, _ = m.rope_frequencies(64)
    for bad in [lambda: m.rope(x.float(), pos, inv), lambda: m.rope(x, pos.long(), inv), lambda: m.rope(x, pos[:3], inv),
                lambda: m.rope(x, pos, inv.float()), lambda: m.rope(x, pos, inv.cpu()),
                lambda: m.rope(x.transpose(1, 2), pos, inv), lambda: m.rope(x, pos, inv, out=x[:, :1])]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: m.rope(x, pos, inv, offset=8), lambda: m.rope(x, pos, inv[:4]),
                lambda: m.rope(x[..., 4:60], pos, inv[:16]), lambda: m.rope(x, pos, inv, scale=float("nan"))]:
        with pytest.raises(m.MlaError):
            bad()
    assert m.rope(x[:0], pos[:0], inv).shape == (0, 2, 64)


# ---------------------------------------------------------------- append

def fp8_split(rows):
    return (rows[..., :512].view(torch.float8_e4m3fn).double().cpu().numpy(), rows[..., 512:516].cpu().numpy().astype(int) - 127,
            rows[..., 528:].contiguous().view(torch.bfloat16).double().cpu().numpy(), rows[..., 516:528].cpu().numpy())


def assert_rows(got, lat, pe, k_pe, turned, fp8, skip_nan=False):
    """got: the written rows; lat, pe: the oracle's values before rounding."""
    if fp8:
        codes, e, gpe, unused = fp8_split(got)
        ref_e = oracle.group_scales(lat)
        m_ = np.where(np.isfinite(lat), np.abs(lat), 0).reshape(-1, 4, 128).max(-1)
        edge = np.abs(m_ / (448.0 * 2.0 ** ref_e) - 1) < 2.0 ** -13     # just below the largest code: either scale is right
        edge |= np.abs(m_ / (448.0 * 2.0 ** (ref_e - 1.0)) - 1) < 2.0 ** -13
        assert ((e == ref_e) | (edge & (np.abs(e - ref_e) == 1))).all()
        x = lat.reshape(-1, 4, 128) / 2.0 ** e[..., None]
        c = codes.reshape(-1, 4, 128)
        fin = np.isfinite(x)
        assert np.isnan(c[~fin]).all()
        bound = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + 2.0 ** -13 * np.abs(x)
        assert (np.abs(c - np.where(fin, x, 0))[fin] <= bound[fin]).all()
        assert not unused.any()
    else:
        g = f64(got)
        gpe = g[..., 512:]
        assert (np.abs(g[..., :512] - lat) <= (2.0 ** -8 + 2.0 ** -13) * np.abs(lat)).all()
    if not turned:
        assert np.array_equal(gpe, f64(k_pe))
    else:
        mass = np.abs(f64(k_pe)).max(-1, keepdims=True) * 2
        assert (np.abs(gpe - pe) <= 2.0 ** -8 * np.abs(pe) + 2.0 ** -20 * mass).all()


def pool(pages, fp8, seed):
    if fp8:
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randint(0, 256, (pages, 64, 656), generator=g, device="cuda", dtype=torch.uint8)
    return rand((pages, 64, 576), seed)


def append_case(lens_old, counts, fp8, norm, turned, half, seed=0, shuffle=True):
    """Requests with lens_old cached tokens get counts new ones, in a random
    order, over randomly placed pages; the whole pool is checked."""
    rng = np.random.default_rng(seed)
    B = len(counts)
    req = np.repeat(np.arange(B), counts)
    pos = np.concatenate([np.arange(o, o + c) for o, c in zip(lens_old, counts)])
    if shuffle:
        p = rng.permutation(len(req))
        req, pos = req[p], pos[p]
    need = [(o + c + 63) // 64 for o, c in zip(lens_old, counts)]
    perm = rng.permutation(sum(need) + 2)
    bt = np.full((B, max(need) + 1), -1, np.int32)
    k = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[k:k + n]
        k += n
    T = len(req)
    x = rand((T, 576), seed + 1)
    w = (1 + 0.2 * rand((512,), seed + 2).float()).to(torch.bfloat16) if norm else None
    inv, scale = m.rope_frequencies(64, yarn=4.0)
    cache = pool(len(perm), fp8, seed + 3)
    before = cache.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = m.cache_append(x[:, :512], x[:, 512:], cache, dev(bt), dev(pos), request_ids=dev(req), norm_weight=w,
                         eps=1e-5, inv_freq=inv if turned else None, half=half, rope_scale=scale, status=status)
    assert out is cache and int(status) == 0
    lat, pe = oracle.appended_rows(f64(x[:, :512]), f64(x[:, 512:]), pos, None if w is None else f64(w), 1e-5,
                                   inv.cpu().numpy() if turned else None, half, scale)
    rows = torch.tensor(oracle.append_places(pos, req, bt), device="cuda")
    flat = cache.flatten(0, 1)
    assert_rows(flat[rows], lat, pe, x[:, 512:], turned, fp8)
    rest = torch.ones(flat.shape[0], dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.equal(flat[rest], before.flatten(0, 1)[rest])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm,turned,half", [(True, True, False), (True, True, True), (False, False, False),
                                              (False, True, False), (True, False, True)])
def test_append_matches_the_oracle(fp8, norm, turned, half):
    append_case([0, 63, 64, 127, 5], [1, 2, 64, 130, 3], fp8, norm, turned, half)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("old,counts", [([0], [1]), ([4000], [1]), ([10] * 64, [1] * 64), ([0, 1, 2], [333, 1, 64])])
def test_append_sizes(fp8, old, counts):
    append_case(old, counts, fp8, True, True, False, seed=11)


@pytest.mark.parametrize("fp8", [False, True])
def test_equal_runs_need_no_request_ids(fp8):
    B, n = 5, 2
    x = rand((B * n, 576), 1)
    inv, _ = m.rope_frequencies(64)
    bt = torch.arange(B * 2, device="cuda", dtype=torch.int32).view(B, 2)
    pos = torch.tensor([62, 63, 63, 64, 0, 1, 5, 6, 126, 127], device="cuda", dtype=torch.int32)
    req = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(n)
    a, b = pool(B * 2, fp8, 2), pool(B * 2, fp8, 2)
    m.cache_append(x[:, :512], x[:, 512:], a, bt, pos, inv_freq=inv)
    m.cache_append(x[:, :512].contiguous(), x[:, 512:].contiguous(), b, bt, pos, request_ids=req, inv_freq=inv)
    assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_is_skipped_and_bad_places_are_reported(fp8):
    x = rand((6, 576), 1)
    bt = torch.tensor([[0, 99], [3, -1]], device="cuda", dtype=torch.int32)
    ints = lambda *a: torch.tensor(a, device="cuda", dtype=torch.int32)  # noqa: E731
    for pos, req, bad in [((-1,) * 6, (0, 1, -7, 99, 0, 1), False), ((5, -1, 6, -2 ** 31, 7, -1), (0, 9, 1, 9, 1, 0), False),
                          ((5, 64, 6, 7, 8, 9), (0, 0, 0, 0, 0, 0), True),      # page 99
                          ((5, 64, 6, 7, 8, 9), (1, 1, 1, 1, 1, 1), True),      # page -1
                          ((5, 128, 6, 7, 8, 9), (1, 1, 1, 1, 1, 1), True),     # past the table
                          ((5, 2 ** 31 - 1, 6, 7, 8, 9), (1, 1, 1, 1, 1, 1), True),
                          ((5, 3, 6, 7, 8, 9), (1, 2, 1, 1, 1, 1), True),       # no such request
                          ((5, 3, 6, 7, 8, 9), (1, -1, 1, 1, 1, 1), True)]:
        cache = pool(4, fp8, 5)
        before = cache.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        m.cache_append(x[:, :512], x[:, 512:], cache, bt, ints(*pos), request_ids=ints(*req), status=status)
        assert int(status) == (m.MLA_ERR_BAD_TABLE if bad else 0)
        good = [t for t in range(6) if 0 <= pos[t] < 64 and req[t] in (0, 1)]
        rows = torch.tensor([(0 if req[t] == 0 else 3) * 64 + pos[t] for t in good], dtype=torch.long, device="cuda")
        lat, pe = oracle.appended_rows(f64(x[good, :512]), f64(x[good, 512:]), [pos[t] for t in good])
        if good:
            assert_rows(cache.flatten(0, 1)[rows], lat, pe, x[good, 512:], False, fp8)
        rest = torch.ones(4 * 64, dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert torch.equal(cache.flatten(0, 1)[rest], before.flatten(0, 1)[rest])


def test_a_slice_of_a_wider_block_table():
    """Entries outside the slice are neither used nor taken for the row's next ones."""
    x = rand((4, 576), 1)
    wide = torch.arange(12, device="cuda", dtype=torch.int32).view(3, 4)
    ints = lambda *a: torch.tensor(a, device="cuda", dtype=torch.int32)  # noqa: E731
    for lo, hi in ((0, 2), (1, 3), (2, 4)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(positions=ints(3, 64, 127, 5), request_ids=ints(0, 1, 2, 2), status=status)
        a, b = pool(12, False, 5), pool(12, False, 5)
        m.cache_append(latent=x[:, :512], k_pe=x[:, 512:], kv_cache=a, block_table=wide[:, lo:hi], **kw)
        m.cache_append(x[:, :512], x[:, 512:], b, wide[:, lo:hi].contiguous(), **kw)
        assert torch.equal(a, b) and int(status) == 0
        before = a.clone()
        m.cache_append(x[:, :512], x[:, 512:], a, wide[:, lo:hi], ints(128, 128, 128, 200), request_ids=ints(0, 1, 2, 2),
                       status=status)
        assert int(status) == m.MLA_ERR_BAD_TABLE and torch.equal(a, before)


def test_a_block_table_of_one_column_may_have_any_stride():
    """The stride of a dim of one says nothing: a row turned into a column."""
    x = rand((3, 576), 1)
    ints = lambda *a: torch.tensor(a, device="cuda", dtype=torch.int32)  # noqa: E731
    column = ints([3, 1, 2]).t()
    assert column.shape == (3, 1) and column.stride() == (1, 3)
    spaced = ints([3, 0, 0], [1, 0, 0], [2, 0, 0])[:, :1]
    want = pool(4, False, 5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_append(x[:, :512], x[:, 512:], want, ints([3], [1], [2]), ints(0, 5, 63), status=status)
    for bt in (column, spaced):
        got = pool(4, False, 5)
        m.cache_append(x[:, :512], x[:, 512:], got, bt, ints(0, 5, 63), status=status)
        assert torch.equal(got, want) and int(status) == 0


def test_fp8_groups_of_zeros_tiny_huge_and_not_finite_values():
    x = rand((8, 576), 3).float()
    x[0, :128] = 0
    x[1, :128] *= 2.0 ** -126
    x[2, 128:256] *= 2.0 ** 120
    x[3, 5], x[3, 200], x[3, 300] = float("inf"), float("-inf"), float("nan")
    x[4, :] = 0
    x[5, :512] = 0
    x[5, 3] = 448.0
    x[6, :512] = 0
    x[6, 3] = 450.0
    x[7, :128] = float("inf")
    x = x.to(torch.bfloat16)
    cache = pool(1, True, 4)
    pos = torch.arange(8, device="cuda", dtype=torch.int32)
    m.cache_append(x[:, :512], x[:, 512:], cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), pos)
    lat, pe = oracle.appended_rows(f64(x[:, :512]), f64(x[:, 512:]), pos.cpu().numpy())
    assert_rows(cache[0, :8], lat, pe, x[:, 512:], False, True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_latents_whose_squares_leave_the_range_of_fp32(fp8, eps):
    """Normed, they are numbers of order one all the same (or, below sqrt(eps),
    small ones)."""
    x = rand((8, 576), 51).float()
    x[:, :512] *= torch.tensor([1e18, 3e19, 1e30, 1e37, 1e-17, 1e-25, 1e-38, 1.0], device="cuda")[:, None]
    x = x.to(torch.bfloat16)
    w = (1 + 0.2 * rand((512,), 52).float()).to(torch.bfloat16)
    cache, pos = pool(1, fp8, 4), torch.arange(8, device="cuda", dtype=torch.int32)
    m.cache_append(x[:, :512], x[:, 512:], cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), pos, norm_weight=w,
                   eps=eps)
    lat, pe = oracle.appended_rows(f64(x[:, :512]), f64(x[:, 512:]), pos.cpu().numpy(), f64(w), eps)
    rows = slice(None) if eps == 0 else [0, 1, 2, 3, 4, 5, 7]  # 1e-38 / sqrt(eps): below bf16's normal numbers' precision
    assert_rows(cache[0, :8][rows], lat[rows], pe[rows], x[rows, 512:], False, fp8)


def test_appended_rows_are_what_the_decode_reads():
    """Append a request's tokens, then decode over them: bf16 and FP8 rows."""
    L = 150
    for fp8 in (False, True):
        x = rand((L, 576), 21)
        q = rand((1, 1, 128, 576), 22)
        cache = pool(4, fp8, 23) if not fp8 else torch.zeros((4, 64, 656), dtype=torch.uint8, device="cuda")
        bt = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
        inv, _ = m.rope_frequencies(64)
        m.cache_append(x[:, :512], x[:, 512:], cache, bt, torch.arange(L, device="cuda", dtype=torch.int32), inv_freq=inv)
        lens = torch.tensor([L], dtype=torch.int32, device="cuda")
        o, lse = m.decode_step(q, cache, bt, lens, 192 ** -0.5, out_fp32=True)
        if fp8:
            ro, rl = oracle.mla_decode_fp8(wl.bf16_bits(q), cache.cpu().numpy(), bt.cpu().numpy(), lens.cpu().numpy(), 192 ** -0.5)
        else:
            ro, rl = oracle.mla_decode(wl.bf16_bits(q), wl.bf16_bits(cache), bt.cpu().numpy(), lens.cpu().numpy(), 192 ** -0.5)
        assert np.abs(f64(o) - ro).max() <= 2e-2 and np.abs(f64(lse) - rl).max() <= 1e-3


def test_calls_captured_replayed_and_on_another_stream():
    x = rand((64, 576), 31)
    pos = torch.arange(64, device="cuda", dtype=torch.int32)
    bt = torch.zeros((64, 2), dtype=torch.int32, device="cuda")
    bt[:] = torch.arange(128, device="cuda", dtype=torch.int32).view(64, 2)
    inv, _ = m.rope_frequencies(64)
    q = rand((64, 128, 64), 32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want_cache, cache = pool(128, False, 33), pool(128, False, 33)
    out = torch.empty_like(q)
    m.cache_append(x[:, :512], x[:, 512:], want_cache, bt, pos, inv_freq=inv, status=status)
    want = m.rope(q, pos, inv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.cache_append(x[:, :512], x[:, 512:], cache, bt, pos, inv_freq=inv, stream=side)
    got = m.rope(q, pos, inv, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(cache, want_cache) and torch.equal(got, want)
    cache.copy_(pool(128, False, 33))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        m.cache_append(x[:, :512], x[:, 512:], cache, bt, pos, inv_freq=inv, status=status)
        m.rope(q, pos, inv, out=out)
    for step in range(2):  # the graph takes what its inputs hold when it runs
        pos += step
        g.replay()
        torch.cuda.synchronize()
        m.cache_append(x[:, :512], x[:, 512:], want_cache, bt, pos, inv_freq=inv, status=status)
        assert torch.equal(cache, want_cache) and torch.equal(out, m.rope(q, pos, inv))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_pool_and_rows_beyond_32_bit_offsets(fp8):
    pages, width = 120000, 656 if fp8 else 576
    cache = torch.zeros((pages, 64, width), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    x = rand((3, 576), 1)
    bt = torch.tensor([[0, pages - 1, pages // 2]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 127, 128], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.cache_append(x[:, :512], x[:, 512:], cache, bt, pos, request_ids=torch.zeros(3, dtype=torch.int32, device="cuda"),
                   status=status)
    assert int(status) == 0
    lat, pe = oracle.appended_rows(f64(x[:, :512]), f64(x[:, 512:]), [0, 127, 128])
    got = torch.stack([cache[0, 0], cache[pages - 1, 63], cache[pages // 2, 0]])
    assert_rows(got, lat, pe, x[:, 512:], False, fp8)
    assert int((cache.view(torch.int16) != 0).any(-1).sum()) == 3  # three rows written


def test_rope_beyond_32_bit_offsets():
    T, H, D = 120000, 128, 192
    x = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    x[-1] = rand((H, D), 1)
    pos = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    inv, _ = m.rope_frequencies(64)
    y = m.rope(x, pos, inv, offset=128)
    assert_rope(y[-1:], x[-1:], pos[-1:], inv, 128, False, False, 1.0)
    assert not y[:-1].any()


def test_append_refusals():
    x, pos = rand((4, 576), 1), torch.zeros(4, dtype=torch.int32, device="cuda")
    bt, cache = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), pool(4, False, 2)
    lat, pe = x[:, :512], x[:, 512:]
    for bad in [lambda: m.cache_append(lat.float(), pe, cache, bt, pos), lambda: m.cache_append(lat, pe[:3], cache, bt, pos),
                lambda: m.cache_append(lat, pe, cache[:, :32], bt, pos), lambda: m.cache_append(lat, pe, cache.half(), bt, pos),
                lambda: m.cache_append(lat, pe, cache, bt.long(), pos), lambda: m.cache_append(lat, pe, cache, bt, pos[:2]),
                lambda: m.cache_append(lat, pe, cache, bt[:1].expand(4, 1), pos),
                lambda: m.cache_append(lat, pe, cache, bt, pos, norm_weight=torch.ones(512, device="cuda")),
                lambda: m.cache_append(lat, pe, cache, bt, pos, inv_freq=torch.ones(16, dtype=torch.float64, device="cuda")),
                lambda: m.cache_append(lat, pe, cache, bt, pos, request_ids=pos.long())]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: m.cache_append(lat, pe, cache, bt[:3], pos),  # 4 tokens are not 3 equal runs
                lambda: m.cache_append(lat, pe, cache, bt, pos, norm_weight=x[0, :512].contiguous(), eps=-1.0)]:
        with pytest.raises(m.MlaError):
            bad()
    assert m.cache_append(lat[:0], pe[:0], cache, bt, pos[:0]) is cache
