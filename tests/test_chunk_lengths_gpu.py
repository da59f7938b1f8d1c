"""Lengths out of range are reported wherever they stand, those of requests
without new tokens among them (GPU required)."""

import pytest
import torch

import mla_latent_kv_09_gb300 as m
from test_chunk_gpu import SCALE, ints, paged, rand, starts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from mla_latent_kv_09_gb300 import build
    build.build()
    m.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("counts", [[3, 0, 1], [0, 0, 1, 0, 0, 0, 0, 0, 0], [5, 0], [0, 5], [1] * 7, [0] * 130 + [2] + [0] * 130])
def test_a_bad_length_of_any_request_is_reported(counts, fp8):
    lens = [64 + n for n in counts]
    cache, table, _ = paged(lens, fp8, 3)
    starts = starts_of(counts)
    q = rand((starts[-1], 128, 576), 4)
    args = dict(token_starts=ints(starts), max_len=table.shape[1] * 64)
    status = ints([0])
    want = m.chunk_attend(q, cache, table, ints(lens), SCALE, status=status, **args)
    _, lse = want
    assert int(status) == 0
    at = [0, len(counts) - 1, len(counts) // 2] + [b for b, n in enumerate(counts) if not n][:2]
    for b in sorted(set(at)):
        for bad in (-1, table.shape[1] * 64 + 1, 2 ** 31 - 1):
            wrong = list(lens)
            wrong[b] = bad
            status, other = ints([0]), ints([0])
            # (a length beyond the table's rows reads pages that are not there, which is reported too)
            got = m.chunk_attend(q, cache, table.clamp_min(0), ints(wrong), SCALE, status=status, **args)
            m.attention_weights(q, lse, cache, table.clamp_min(0), ints(wrong), SCALE, status=other, **args)
            assert int(status) == m.MLA_ERR_BAD_TABLE and int(other) == m.MLA_ERR_BAD_TABLE, (b, bad)
            for c in range(len(counts)):  # the other requests' results are what they are
                if c != b and counts[c]:
                    part = slice(starts[c], starts[c + 1])
                    # (cut into other pieces, perhaps)
                    assert torch.allclose(got[0][part].float(), want[0][part].float(), rtol=2.0 ** -6, atol=2.0 ** -6)


def test_a_bad_length_in_equal_runs_is_reported():
    cache, table, _ = paged([70, 70, 70], False, 5)
    q = rand((6, 128, 576), 6)
    for b in range(3):
        for bad in (-1, 129):
            lens = [70, 70, 70]
            lens[b] = bad
            status = ints([0])
            m.chunk_attend(q, cache, table, ints(lens), SCALE, status=status)
            assert int(status) == m.MLA_ERR_BAD_TABLE
