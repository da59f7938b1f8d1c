"""Host logic and oracle pins of the cache-filling and shared-prefix calls (no
GPU): argument checks, the frequencies, and the fp64 oracles on cases that
can be worked out by hand."""

import math

import numpy as np
import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle
from mla_latent_kv_09_gb300 import build as mbuild

OK = 1 << 20  # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load()


# ---------------------------------------------------------------- argument checks

def check(f, good, bad, status):
    for i, v in bad:
        a = list(good)
        a[i] = v
        assert f(*a) == status, (f.__name__, i, v)


#       x   ts    hs  pos  T  H   D   off  R  freq scale flags out ots  ohs stream
ROPE = [OK, 1024, 128, OK, 4, 8, 128, 64, 64, OK, 1.0, 0, 2 * OK, 1024, 128, None]


def test_rope_checks_its_arguments(lib):
    check(lib.mla_rope, ROPE, [(0, None), (3, None), (9, None), (12, None), (0, OK + 8), (12, OK + 8), (3, OK + 2),
                               (9, OK + 4), (4, -1), (5, 0), (1, 1025), (2, 132), (13, 4), (7, -8), (7, 72),
                               (10, math.inf), (10, math.nan), (11, 1), (14, 64), (13, 128), (1, -128),
                               (1, 1 << 40)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_rope, ROPE, [(6, 132), (7, 4), (8, 24), (8, 264)], m.MLA_ERR_UNSUPPORTED)
    # in place with other strides than the input's
    a = list(ROPE)
    a[12], a[13] = a[0], 2048
    assert lib.mla_rope(*a) == m.MLA_ERR_INVALID_ARG


#         lat  ls   kpe  ks  wt  eps   freq sc  pos req T  bt  s  w  B  cache pages flags status stream
APPEND = [OK, 576, OK, 576, OK, 1e-6, OK, 1.0, OK, OK, 4, OK, 3, 3, 2, OK, 10, 0, OK, None]


def test_append_checks_its_arguments(lib):
    check(lib.mla_cache_append, APPEND,
          [(0, None), (2, None), (8, None), (11, None), (15, None), (18, None), (0, OK + 8), (2, OK + 2), (4, OK + 8),
           (6, OK + 4), (8, OK + 2), (9, OK + 1), (11, OK + 2), (15, OK + 8), (18, OK + 2), (1, 504), (1, 577), (3, 56),
           (10, -1), (12, 2), (13, 0), (13, 4), (14, 0), (16, 0), (17, 1), (17, 64), (5, -1.0), (5, math.nan),
           (7, math.inf)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_cache_append, APPEND, [(16, 1 << 40), (10, 2 ** 31 - 1)], m.MLA_ERR_UNSUPPORTED)
    a = list(APPEND)  # equal runs that are not
    a[9], a[10] = None, 5
    assert lib.mla_cache_append(*a) == m.MLA_ERR_INVALID_ARG


#         cache pages bt  P   wk  wv  H  fl k   v   rows kpe ws bytes status stream
EXPAND = [OK, 10, OK, 100, OK, OK, 16, 0, OK, OK, 100, OK, OK, None]


def test_expand_checks_its_arguments(lib):
    check(lib.mla_prefix_expand, EXPAND,
          [(0, None), (2, None), (4, None), (5, None), (8, None), (9, None), (11, None), (12, None), (0, OK + 8),
           (4, OK + 8), (5, OK + 2), (8, OK + 8), (9, OK + 8), (11, OK + 8), (12, OK + 1), (1, 0),
           (3, -1), (3, 101), (7, 1), (7, 32)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_prefix_expand, EXPAND, [(6, 0), (6, 129), (1, 1 << 40)], m.MLA_ERR_UNSUPPORTED)


#         qn  qp        qs  k   v  rows kpe  P  vis  T   H  scale so    sl   fl ws  bytes  out lse status stream
ATTEND = [OK, OK + 256, 192, OK, OK, 64, OK, 64, None, 4, 16, 0.07, None, None, 0, OK, 1 << 40, OK, OK, OK, None]


def test_attend_checks_its_arguments(lib):
    check(lib.mla_prefix_attend, ATTEND,
          [(0, None), (1, None), (3, None), (4, None), (6, None), (17, None), (18, None), (19, None),
           (0, OK + 8), (1, OK + 8), (3, OK + 8), (4, OK + 8), (6, OK + 8), (8, OK + 2), (12, OK), (13, OK),
           (15, OK + 128), (17, OK + 8), (18, OK + 2), (19, OK + 1), (2, 120), (2, 196), (2, 1 << 40), (5, 63),
           (7, -1), (9, -1), (11, 0.0), (11, -1.0), (11, math.nan), (11, math.inf), (14, 1)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_prefix_attend, ATTEND, [(10, 0), (10, 129), (9, 1 << 30), (5, 1 << 32)], m.MLA_ERR_UNSUPPORTED)
    a = list(ATTEND)  # an fp32 result over the bf16 suffix
    a[12], a[13], a[14], a[17] = OK, OK, m.MLA_FLAG_OUT_FP32, OK
    assert lib.mla_prefix_attend(*a) == m.MLA_ERR_INVALID_ARG


def test_python_calls_refuse_tensors_off_the_gpu():
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.rope(x, torch.zeros(2, dtype=torch.int32), torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        m.cache_append(x[:, 0], x[:, 0], x, x, x)
    with pytest.raises(ValueError):
        m.prefix_expand(x, x, 1, x, x)
    with pytest.raises(ValueError):
        m.prefix_attend(x, x, x, x, x, 1.0)
    with pytest.raises(ValueError):  # by name
        m.rope(x=x, positions=torch.zeros(2, dtype=torch.int32), inv_freq=torch.ones(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        m.rope(positions=torch.zeros(2, dtype=torch.int32))


# ---------------------------------------------------------------- frequencies

def test_plain_and_interpolated_frequencies():
    f, scale = m.rope_frequencies(64, 10000.0, device="cpu")
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert scale == 1.0 and f.dtype == torch.float64
    assert np.allclose(f.numpy(), want, rtol=1e-14, atol=0)
    g, _ = m.rope_frequencies(64, 10000.0, linear=8.0, device="cpu")
    assert np.allclose(g.numpy(), np.array(want) / 8, rtol=1e-14, atol=0)


def test_yarn_keeps_fast_pairs_and_slows_slow_ones():
    f, _ = m.rope_frequencies(64, device="cpu")
    y, scale = m.rope_frequencies(64, yarn=40.0, original_len=4096, device="cpu")
    assert scale == pytest.approx(0.1 * math.log(40) + 1, rel=1e-15)
    ratio = (y / f).numpy()
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert (ratio[turns > 64] == 1).all()                                    # well above beta_fast: kept
    assert np.allclose(ratio[turns < 0.5], 1 / 40, rtol=1e-14)               # well below beta_slow: stretched
    assert (np.diff(ratio) <= 1e-15).all() and (ratio >= 1 / 40 - 1e-15).all()


def test_yarn_factor_of_heads_that_turn_in_part():
    """YaRN multiplies whole queries and keys by its factor.  Of 192 dims 64 turn:
    the scale on the softmax gives these scores, one on the turned dims others."""
    rng = np.random.default_rng(3)
    f, factor = m.rope_frequencies(64, yarn=40.0, device="cpu")
    q, k = rng.standard_normal((2, 5, 192))
    pos_q, pos_k = rng.integers(0, 100000, (2, 5))
    turn = lambda x, p, scale=1.0: oracle.rope(x[:, None], p, f.numpy(), offset=128, scale=scale)[:, 0]  # noqa: E731
    want = (factor * turn(q, pos_q)) @ (factor * turn(k, pos_k)).T / math.sqrt(192)
    got = m.softmax_scale(192, factor) * turn(q, pos_q) @ turn(k, pos_k).T
    assert np.allclose(got, want, rtol=1e-12, atol=0)
    assert not np.allclose(m.softmax_scale() * turn(q, pos_q, factor) @ turn(k, pos_k, factor).T, want, rtol=1e-2)
    assert m.softmax_scale() == 192 ** -0.5 and m.softmax_scale(128) == 128 ** -0.5


@pytest.mark.parametrize("a", [(0,), (-1,), (192, 0.0), (192, math.nan), (192, math.inf)])
def test_softmax_scale_refuses(a):
    with pytest.raises(ValueError):
        m.softmax_scale(*a)


@pytest.mark.parametrize("kw", [dict(rope_dim=63), dict(rope_dim=0), dict(base=1.0), dict(linear=0.5), dict(yarn=0.0),
                                dict(original_len=0), dict(beta_fast=1.0, beta_slow=2.0), dict(beta_slow=0.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        m.rope_frequencies(**{"rope_dim": 64, **kw}, device="cpu")


# ---------------------------------------------------------------- oracle pins

def test_a_quarter_turn():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]])
    inv = [math.pi / 2, math.pi]
    assert np.allclose(oracle.rope(x, [1], inv, offset=2), [[[1, 2, -4, 3, -5, -6]]])
    assert np.allclose(oracle.rope(x, [1], inv, offset=2, half=True), [[[1, 2, -5, -4, 3, -6]]])
    assert np.allclose(oracle.rope(x, [1], inv, offset=2, scale=2.0), [[[1, 2, -8, 6, -10, -12]]])
    back = oracle.rope(oracle.rope(x, [7], inv, half=True), [7], inv, half=True, inverse=True)
    assert np.allclose(back, x)


def test_rotation_keeps_relative_positions():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 64))
    inv = 10000.0 ** (-np.arange(32) / 32)
    dot = lambda a, b: float((oracle.rotate(q, [a], inv) * oracle.rotate(k, [b], inv)).sum())  # noqa: E731
    assert dot(5, 3) == pytest.approx(dot(1005, 1003), abs=1e-9)


def test_fp8_scales_are_the_smallest_that_hold():
    lat = np.zeros((1, 512))
    lat[0, 0], lat[0, 130], lat[0, 257] = 448.0, 448.0001, 2.0 ** -200
    assert oracle.group_scales(lat).tolist() == [[0, 1, -127, 0]]
    lat[0, 0], lat[0, 1] = np.inf, 3.5
    assert oracle.group_scales(lat)[0, 0] == -7  # 3.5 = 448 / 2^7


def test_one_visible_row_returns_its_value_and_none_the_suffix():
    rng = np.random.default_rng(1)
    q, pe = rng.standard_normal((3, 2, 128)), rng.standard_normal((3, 2, 64))
    k, kp, v = rng.standard_normal((2, 5, 128)), rng.standard_normal((5, 64)), rng.standard_normal((2, 5, 128))
    so, sl = rng.standard_normal((3, 2, 128)), rng.standard_normal((3, 2))
    out, lse = oracle.prefix_attend(q, pe, k, kp, v, 0.1, [1, 0, 5])
    assert np.allclose(out[0], v[:, 0]) and not out[1].any() and (lse[1] == -np.inf).all()
    out, lse = oracle.prefix_attend(q, pe, k, kp, v, 0.1, [1, 0, 5], so, sl)
    assert np.allclose(out[1], so[1]) and np.allclose(lse[1], sl[1])
    # rows split in two and joined are rows attended to at once
    a = oracle.prefix_attend(q, pe, k[:, :2], kp[:2], v[:, :2], 0.1)
    b = oracle.prefix_attend(q, pe, k[:, 2:], kp[2:], v[:, 2:], 0.1)
    whole = oracle.prefix_attend(q, pe, k, kp, v, 0.1)
    for x, y in zip(oracle.join(*a, *b), whole):
        assert np.allclose(x, y)


def test_expanded_attention_is_absorbed_attention():
    """q . (W latent) = (W^T q) . latent, and W (sum p latent) = sum p (W latent)."""
    rng = np.random.default_rng(2)
    lat, kp = rng.standard_normal((9, 512)), rng.standard_normal((9, 64))
    wk, wv = rng.standard_normal((2, 2, 512, 128)) / 20
    q, pe = rng.standard_normal((1, 2, 128)), rng.standard_normal((1, 2, 64))
    out, lse = oracle.prefix_attend(q, pe, oracle.prefix_expand(lat, wk), kp, oracle.prefix_expand(lat, wv), 0.07)
    q_lat = np.einsum("hcd,thd->thc", wk, q)
    s = 0.07 * (np.einsum("thc,pc->thp", q_lat, lat) + pe @ kp.T)
    p = np.exp(s - s.max(-1, keepdims=True))
    z = p.sum(-1, keepdims=True)
    assert np.allclose(lse, (s.max(-1) + np.log(z[..., 0])))
    assert np.allclose(out, np.einsum("thc,hcd->thd", p / z @ lat, wv))
