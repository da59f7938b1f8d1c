"""Host logic and oracle pins of chunk attention and of the cache's eviction (no
GPU): argument checks, and the fp64 oracle on cases that can be worked out by
hand."""

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


def check(f, good, bad, status):
    for i, v in bad:
        a = list(good)
        a[i] = v
        assert f(*a) == status, (f.__name__, i, v)


#        q   kv  pages bt  st lens max starts B  N  H    scale fl ws  bytes    out lse status stream
CHUNK = [OK, OK, 10, OK, 4, OK, 200, OK, 3, 12, 128, 0.07, 0, OK, 1 << 40, OK, OK, OK, None]


def test_chunk_checks_its_arguments(lib):
    check(lib.mla_chunk_attend, CHUNK,
          [(0, None), (1, None), (3, None), (5, None), (13, None), (15, None), (16, None), (17, None), (0, OK + 8),
           (1, OK + 8), (3, OK + 2), (5, OK + 2), (7, OK + 1), (13, OK + 128), (15, OK + 8), (16, OK + 2), (17, OK + 2),
           (2, 0), (4, 0), (4, 3), (6, 0), (6, -5), (8, 0), (9, -1), (11, 0.0), (11, -1.0), (11, math.nan),
           (11, math.inf), (12, 4), (12, 8), (12, 32)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_chunk_attend, CHUNK, [(10, 64), (10, 0), (2, 1 << 40)], m.MLA_ERR_UNSUPPORTED)
    a = list(CHUNK)  # equal runs that are not
    a[7], a[9] = None, 13
    assert lib.mla_chunk_attend(*a) == m.MLA_ERR_INVALID_ARG


def test_chunk_workspace_refuses_sizes(lib):
    import ctypes
    err = ctypes.c_int(0)
    for args, status in [((-1, 1, 64, 0), m.MLA_ERR_INVALID_ARG), ((1, 0, 64, 0), m.MLA_ERR_INVALID_ARG),
                         ((1, 1, 0, 0), m.MLA_ERR_INVALID_ARG), ((1, 1, 64, 8), m.MLA_ERR_INVALID_ARG),
                         ((1 << 24, 1, 64, 0), m.MLA_ERR_UNSUPPORTED), ((1 << 20, 1, 1 << 30, 0), m.MLA_ERR_UNSUPPORTED)]:
        assert lib.mla_chunk_attend_workspace_size(*args, ctypes.byref(err)) == 0 and err.value == status, args


#          q   lse kv  pages bt  st lens max starts B  N  H   scale dec  w   wst  fl ws  bytes   out ost status stream
WEIGHTS = [OK, OK, OK, 10, OK, 4, OK, 200, OK, 3, 12, 128, 0.07, 1.0, OK, 200, 0, OK, 1 << 40, OK, 200, OK, None]


def test_weights_check_their_arguments(lib):
    check(lib.mla_attention_weights, WEIGHTS,
          [(0, None), (1, None), (2, None), (4, None), (6, None), (14, None), (17, None), (19, None), (21, None),
           (0, OK + 8), (1, OK + 2), (2, OK + 8), (4, OK + 2), (6, OK + 2), (8, OK + 2), (14, OK + 2), (17, OK + 128),
           (19, OK + 1), (21, OK + 2), (3, 0), (5, 0), (5, 3), (7, 0), (9, 0), (10, -1), (12, 0.0), (12, math.nan),
           (13, math.nan), (13, math.inf), (15, 199), (16, 2), (16, 4), (20, 199), (20, 256)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_attention_weights, WEIGHTS, [(11, 16), (3, 1 << 40), (10, 1 << 24)], m.MLA_ERR_UNSUPPORTED)
    check(lib.mla_attention_weights, WEIGHTS, [(18, 0)], m.MLA_ERR_WORKSPACE)
    for w, wst, out, ost, fits in [(OK, 200, OK + 400, 200, False), (OK, 200, OK, 256, False), (OK, 200, OK + 2396, 200, False),
                                   (OK, 400, OK + 800, 400, True), (OK, 400, OK + 796, 400, False), (OK, 200, OK, 200, True),
                                   (OK + 2400, 200, OK, 200, True), (OK + 2396, 200, OK, 200, False)]:
        a = list(WEIGHTS)
        a[14], a[15], a[19], a[20] = w, wst, out, ost
        a[18] = 0  # (what passes the other checks fails for its workspace)
        assert lib.mla_attention_weights(*a) == (m.MLA_ERR_WORKSPACE if fits else m.MLA_ERR_INVALID_ARG), (w, wst, out, ost)


#         w   st   lens B  L    keep si re kept lens new     nst  nw   status stream
SELECT = [OK, 100, OK, 3, 100, 40, 4, 8, OK, OK, 2 * OK, 100, 100, OK, None]


def test_select_checks_its_arguments(lib):
    check(lib.mla_evict_select, SELECT,
          [(0, None), (2, None), (8, None), (9, None), (13, None), (0, OK + 2), (2, OK + 2), (8, OK + 2), (9, OK + 2),
           (10, OK + 2), (13, OK + 2), (10, OK), (1, 99), (3, -1), (4, 0), (5, 0), (5, 11), (6, -1), (6, 41), (7, -1),
           (7, 37), (7, 2 ** 31 - 1), (11, 99), (12, 39)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_evict_select, SELECT, [(3, 1 << 29)], m.MLA_ERR_UNSUPPORTED)
    for new, nst in [(OK + 4, 100), (OK + 1196, 100), (OK - 1196, 100), (OK + 200, 250)]:  # into the weights
        a = list(SELECT)
        a[10], a[11] = new, nst
        assert lib.mla_evict_select(*a) == m.MLA_ERR_INVALID_ARG


#          cache pages row  bt  st w kept kst kw lens B  out_table ost ow status stream
COMPACT = [OK, 10, 1152, OK, 4, 4, OK, 40, 40, OK, 3, 2 * OK, 2, 2, OK, None]


def test_compact_checks_its_arguments(lib):
    check(lib.mla_cache_compact, COMPACT,
          [(0, None), (3, None), (6, None), (9, None), (11, None), (14, None), (0, OK + 8), (3, OK + 2), (6, OK + 2),
           (9, OK + 2), (11, OK), (11, OK + 2), (14, OK + 2), (1, 0), (5, 0), (4, 3), (7, 39), (8, -1), (10, -1),
           (12, 1), (13, 0)], m.MLA_ERR_INVALID_ARG)
    check(lib.mla_cache_compact, COMPACT, [(2, 1024), (2, 0), (1, 1 << 40)], m.MLA_ERR_UNSUPPORTED)


def test_python_calls_refuse_tensors_off_the_gpu():
    x = torch.zeros((2, 128, 576), dtype=torch.bfloat16)
    i = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        m.chunk_attend(x, x, i, i[:, 0], 1.0)
    with pytest.raises(ValueError):
        m.attention_weights(x, x, x, i, i[:, 0], 1.0)
    with pytest.raises(ValueError):
        m.evict_select(torch.zeros(2, 5), i[:, 0], 3)
    with pytest.raises(ValueError):
        m.cache_compact(x, i, i, i[:, 0], i)


# ---------------------------------------------------------------- the oracle

def test_a_chunk_of_one_token_is_the_decode_steps_oracle():
    rng = np.random.default_rng(0)
    q, rows = rng.standard_normal((3, 4, 576)), [rng.standard_normal((n, 576)) for n in (5, 70)]
    out, lse = oracle.chunk_attend(q, rows, [0, 1, 3], 0.07)
    for t, (b, seen) in enumerate([(0, 5), (1, 69), (1, 70)]):
        o, l = oracle.attend(q[t], rows[b][:seen], 0.07)
        assert np.allclose(out[t], o, rtol=1e-12, atol=1e-13) and np.allclose(lse[t], l, rtol=1e-12)


def test_tokens_that_see_nothing_and_tokens_of_no_request():
    rows = [np.ones((2, 576))]
    out, lse = oracle.chunk_attend(np.ones((5, 1, 576)), rows, [0, 4], 1.0)
    assert np.array_equal(lse[:2, 0], [-np.inf, -np.inf]) and not out[:2].any()
    assert np.allclose(lse[2:4, 0], [576, 576 + math.log(2)]) and np.allclose(out[2:4], 1)
    assert np.isnan(out[4]).all()
    out, lse = oracle.chunk_attend(np.ones((5, 1, 576)), rows, [0, 4], 1.0, causal=False)
    assert np.allclose(lse[:4, 0], 576 + math.log(2))


def test_weights_of_an_attention_sum_to_its_tokens_and_heads():
    rng = np.random.default_rng(1)
    q, rows, starts = rng.standard_normal((5, 6, 576)), [rng.standard_normal((9, 576)), rng.standard_normal((80, 576))], [0, 2, 5]
    lse = oracle.chunk_attend(q, rows, starts, 0.05)[1]
    got, bound = oracle.attention_weights(q, lse, rows, starts, 0.05)
    assert [round(float(w.sum()), 9) for w in got] == [12.0, 18.0]
    assert all((e > 0).all() for e in bound)
    # a token without a result weighs nothing
    lse[:2] = -np.inf
    assert not oracle.attention_weights(q, lse, rows, starts, 0.05)[0][0].any()


def test_the_choice_of_rows_by_hand():
    w = [0.5, 3.0, 2.0, 2.0, math.nan, 2.0, 9.0, 0.0]
    pick = lambda *a, **k: oracle.evict_select(w, *a, **k).tolist()  # noqa: E731
    assert pick(8, 8) == list(range(8)) and pick(3, 5) == [0, 1, 2]
    assert pick(8, 3) == [1, 2, 6]                # the first of the equal ones
    assert pick(8, 4) == [1, 2, 3, 6]
    assert pick(8, 3, 1, 1) == [0, 6, 7]
    assert pick(8, 2, 1, 1) == [0, 7]
    assert pick(8, 7) == [0, 1, 2, 3, 5, 6, 7]    # NaN goes first
    assert pick(0, 2) == []
