"""How exact attention weights are on the whole, beside the worst case that
oracle.attention_weights bounds (GPU required).

A tensor core truncates as it accumulates: for N(0, 1) queries and rows, fp32
accumulation towards zero over K = 576 in steps of 16 puts the weight of a row
1.62e-6 too low on average (deviation from that: 0.35e-6) if one accumulator takes
all 36 additions, and 0.75e-6 (0.15e-6) if two of 20 and 16 are added after it
(worked out in 64 bits with every addition truncated).  The exponential's 2^-22
may add 0.24e-6.  So means within 1.1e-6 and root mean squares within 1.2e-6 say
that the products run in two accumulators and that nothing behind them loses
more."""

import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle
from test_chunk_gpu import ints, rand

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _build():
    from mla_latent_kv_09_gb300 import build
    build.build()
    m.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("requests,tokens", [(1, 32), (8, 4)])
def test_weights_on_the_whole(requests, tokens, fp8):
    L = 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    pages = requests * L // 64
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(requests, -1)
    if fp8:
        cache = torch.zeros((pages, 64, 656), dtype=torch.uint8, device="cuda")
        codes = torch.randn((pages, 64, 512), generator=g, device="cuda") * 64
        cache[..., :512] = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[..., 512:516] = 121  # 2^-6
        cache[..., 528:] = rand((pages, 64, 64), 2).view(torch.uint8)
        flat = torch.tensor(oracle.fp8_rows_to_f64(cache.cpu().numpy().reshape(-1, 656)), device="cuda")
    else:
        cache = rand((pages, 64, 576), 3)
        flat = cache.double().view(-1, 576)
    q = rand((requests * tokens, 128, 576), 4)
    scale = float(torch.tensor(SCALE, dtype=torch.float32))
    rows = [flat.view(pages, 64, 576)[t.long()].reshape(L, 576) for t in table]
    scores = [scale * (x.double().reshape(-1, 576) @ r.t()) for x, r in zip(q.view(requests, tokens, 128, 576), rows)]
    lse = torch.cat([s.logsumexp(1) for s in scores]).view(-1, 128).float()
    got = m.attention_weights(q, lse, cache, table, ints([L] * requests), SCALE, causal=False)
    ref = torch.stack([(s - l.double().reshape(-1, 1)).exp().sum(0) for s, l in zip(scores, lse.view(requests, -1))])
    off = got.double() / ref - 1
    assert abs(float(off.mean())) <= 1.1e-6
    assert float(off.square().mean().sqrt()) <= 1.2e-6


@pytest.mark.parametrize("L,tokens", [(200, 600), (700, 300), (256, 76), (1000, 1)])
def test_older_weights_are_rounded_three_times_at_most(L, tokens):
    """Large older weights, whose tile's tokens are cut into many ranges: times the
    decay, plus the first range's sum, plus that of the others, a rounding each."""
    cache, table = rand(((L + 63) // 64, 64, 576), 5), torch.arange((L + 63) // 64, dtype=torch.int32, device="cuda")[None]
    q = rand((tokens, 128, 576), 6)
    rows = cache.double().view(-1, 576)[:L]
    scale = float(torch.tensor(SCALE, dtype=torch.float32))
    s = scale * (q.double().view(-1, 576) @ rows.t())
    lse = s.logsumexp(1).view(tokens, 128).float()
    new = (s - lse.double().view(-1, 1)).exp().sum(0)
    was = 1e5 * (1 + torch.rand((1, L), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda"))
    got = m.attention_weights(q, lse, cache, table, ints([L]), SCALE, was.clone(), causal=False, decay=0.75)
    old = 0.75 * was[0].double()
    # the new sum's own error: 2e-5 of it at most (the test above: 1e-6), next to nothing beside a rounding of the whole
    allowed = 3 * 2.0 ** -24 * (old + new) * 1.001 + 2e-5 * new
    assert float(((got[0].double() - (old + new)).abs() / allowed).max()) <= 1
