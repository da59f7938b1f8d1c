"""evict_select with the new lengths in the memory of the old ones: a loop that
keeps one tensor of lengths."""

import numpy as np
import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle
from mla_latent_kv_09_gb300 import build as mbuild

OK = 1 << 20  # an aligned address that is never followed


def test_lengths_of_another_request_are_refused():
    mbuild.build()
    f = m.load().mla_evict_select
    #       w   st   lens B  L    keep si re kept lens new     nst  nw   status stream
    good = [OK, 100, OK, 3, 100, 40, 4, 8, OK, OK, 2 * OK, 100, 100, OK, None]
    for there, fits in ((OK, True), (OK + 4, False), (OK + 8, False), (OK + 12, True), (OK - 4, False), (OK - 12, True)):
        a = list(good)
        a[9] = there
        if not fits:
            assert f(*a) == m.MLA_ERR_INVALID_ARG, there
        else:  # (passes the lengths' check; the next one refuses: new weights over the weights)
            a[10] = OK
            assert f(*a) == m.MLA_ERR_INVALID_ARG
            a[10], a[3] = 2 * OK, 0  # (nothing to launch: without a GPU the device is what is missing)
            assert f(*a) in (m.MLA_OK, m.MLA_ERR_DEVICE), there


@pytest.mark.gpu
@pytest.mark.parametrize("lens,keep", [([1], 1), ([900, 3, 0, 64], 64), ([4096, 1200, 1025], 1024), ([30000, 12, 29999], 5000),
                                       ([131072], 777), ([70000, 131072, 500], 40000)])
def test_new_lengths_in_place_of_the_old(lens, keep):
    """One CTA a request and clusters of up to sixteen, requests that are cut and
    requests that are not, over and over."""
    g = torch.Generator(device="cuda").manual_seed(sum(lens))
    w = torch.randn((len(lens), max(lens)), generator=g, device="cuda")
    old = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = m.evict_select(w, old, keep, sinks=min(4, keep), recent=keep // 3 if keep > 4 else 0)
    held, status = old.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, new = torch.empty_like(want[0]), torch.empty_like(want[2])
    for _ in range(20):
        held.copy_(old)
        kept.fill_(9)
        new.fill_(9.0)
        m.evict_select(w, held, keep, sinks=min(4, keep), recent=keep // 3 if keep > 4 else 0, out=(kept, held, new),
                       status=status)
        assert torch.equal(kept, want[0]) and torch.equal(held, want[1]) and torch.equal(new, want[2])
    assert int(status) == 0
    b = int(np.argmax(lens))
    ref = oracle.evict_select(w[b].cpu().numpy(), lens[b], keep, min(4, keep), keep // 3 if keep > 4 else 0)
    assert np.array_equal(kept[b, :len(ref)].cpu().numpy(), ref) and int(held[b]) == len(ref)


@pytest.mark.gpu
def test_lengths_out_of_range_in_place():
    w = torch.randn((4, 9000), device="cuda")
    held, status = torch.tensor([9001, -3, 9000, 20], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32,
                                                                                                      device="cuda")
    want = m.evict_select(w, held.clone(), 100)
    kept, new = torch.empty_like(want[0]), torch.empty_like(want[2])
    m.evict_select(w, held, 100, out=(kept, held, new), status=status)
    assert int(status) == m.MLA_ERR_BAD_TABLE and held.tolist() == [100, 0, 100, 20]
    assert torch.equal(kept, want[0]) and torch.equal(new, want[2])


@pytest.mark.gpu
def test_lengths_of_weights_without_columns():
    """Nothing to choose from: lengths other than 0 are out of range there too."""
    w = torch.zeros((3, 0), device="cuda")
    for lens, before, after in (([0, 0, 0], 0, m.MLA_OK), ([0, 5, 0], 0, m.MLA_ERR_BAD_TABLE), ([0, 0, -1], 0, m.MLA_ERR_BAD_TABLE),
                                ([0, 5, 0], m.MLA_ERR_BAD_INDEX, m.MLA_ERR_BAD_INDEX)):
        status = torch.full((1,), before, dtype=torch.int32, device="cuda")
        kept, new_lens, _ = m.evict_select(w, torch.tensor(lens, dtype=torch.int32, device="cuda"), 4, status=status)
        assert int(status) == after and new_lens.tolist() == [0, 0, 0] and bool((kept == -1).all())
    held = torch.tensor([0, 5, 0], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.evict_select(w, held, 4, out=(torch.empty((3, 4), dtype=torch.int32, device="cuda"), held, None), status=status)
    assert int(status) == m.MLA_ERR_BAD_TABLE and held.tolist() == [0, 0, 0]
