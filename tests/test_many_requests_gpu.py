"""More requests than a CTA has threads, or a grid's second axis blocks (GPU
required)."""

import pytest
import torch

import mla_latent_kv_09_gb300 as m
from test_chunk_gpu import SCALE, ints, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from mla_latent_kv_09_gb300 import build
    build.build()
    m.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B", [384, 385, 1500, 5000])
def test_chunks_and_weights_of_many_requests(B, fp8):
    """Requests of no token, one, and two over at most a page: results do not
    depend on the batch that they stand in, so those of a few requests at a time
    are the reference."""
    g = torch.Generator(device="cuda").manual_seed(B)
    if fp8:
        cache = torch.zeros((B, 64, 656), dtype=torch.uint8, device="cuda")
        cache[..., :512] = (torch.randn((B, 64, 512), generator=g, device="cuda") * 40).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
        cache[..., 512:516], cache[..., 528:] = 121, rand((B, 64, 64), 1).view(torch.uint8)
    else:
        cache = rand((B, 64, 576), 1)
    table = torch.randperm(B, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    counts = torch.randint(0, 3, (B,), generator=g, device="cuda")
    lens = torch.randint(2, 65, (B,), generator=g, device="cuda").to(torch.int32)
    starts = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0))).to(torch.int32)
    T = int(starts[-1])
    q, status = rand((T, 128, 576), 2), ints([0])
    out, lse = m.chunk_attend(q, cache, table, lens, SCALE, token_starts=starts, status=status)
    was = torch.rand((B, 64), generator=g, device="cuda")
    got = m.attention_weights(q, lse, cache, table, lens, SCALE, was.clone(), token_starts=starts, decay=0.5, status=status)
    assert int(status) == 0
    # each row's weights hold every token's 128 heads once, behind the end they are as they were
    inside = torch.arange(64, device="cuda")[None] < lens[:, None]
    new = torch.where(inside & (counts > 0)[:, None], got - 0.5 * was, torch.zeros_like(got))
    assert torch.allclose(new.sum(1), 128.0 * counts, rtol=1e-4, atol=1e-2)
    assert torch.equal(torch.where(inside & (counts > 0)[:, None], was, got), was)
    for b0 in (0, 1, B // 2 - 20, B - 41):
        part = slice(b0, b0 + 40)
        s = starts[b0:b0 + 41]
        t = slice(int(s[0]), int(s[-1]))
        o, l = m.chunk_attend(q[t], cache, table[part], lens[part], SCALE, token_starts=s - s[0])
        # two bf16 roundings of 2^-8, behind weights and partial results in fp16; an fp32 LSE below 16, a few steps of
        # 2^-20; weights in fp32, their parts added in another order
        assert torch.allclose(out[t].float(), o.float(), rtol=2.0 ** -7, atol=2.0 ** -9) and torch.allclose(lse[t], l, rtol=0, atol=1e-5)
        w = m.attention_weights(q[t], lse[t], cache, table[part], lens[part], SCALE, was[part].clone(), token_starts=s - s[0],
                                decay=0.5)
        assert torch.allclose(got[part], w, rtol=1e-6, atol=0)


def test_choice_and_move_of_many_requests():
    """66,000 requests of up to 20 rows, 3 of which stay."""
    B, L, keep = 66000, 20, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.rand((B, L), generator=g, device="cuda")
    lens = torch.randint(0, L + 1, (B,), generator=g, device="cuda").to(torch.int32)
    status = ints([0])
    kept, new_lens, new = m.evict_select(w, lens, keep, status=status)
    masked = torch.where(torch.arange(L, device="cuda")[None] < lens[:, None], w, torch.full_like(w, -1.0))
    best = masked.topk(keep, 1)
    want = torch.where(best.values >= 0, best.indices, torch.full_like(best.indices, L)).sort(1).values
    want = torch.where(want < L, want, torch.full_like(want, -1)).to(torch.int32)
    assert torch.equal(kept, want) and torch.equal(new_lens, lens.clamp_max(keep))
    assert torch.equal(new[:, :keep], torch.where(want >= 0, w.gather(1, want.clamp_min(0).long()), torch.zeros_like(new[:, :keep])))
    cache = rand((2 * B, 64, 128), 4)
    order = torch.randperm(2 * B, generator=g, device="cuda").to(torch.int32)
    table, free = order[:B, None].contiguous(), order[B:, None].contiguous()
    m.cache_compact(cache, table, kept, new_lens, free, status=status)
    assert int(status) == 0
    some = want >= 0
    old = cache[table.long().expand(B, keep)[some], want.long()[some]]
    place = torch.arange(keep, device="cuda").expand(B, keep)[some]
    assert torch.equal(cache[free.long().expand(B, keep)[some], place], old)
