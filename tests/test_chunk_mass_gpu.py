"""Chunk attention where many rows of small weight carry mass together: one row
far above a long, light remainder (GPU required).

Values have a mean of 1, so that mass which 16-bit weights lose shows in every
dim instead of averaging out.  The bound is oracle.chunk_error_bound's, whose
term for weights below fp16's normal range is 2^-25 of a head's largest weight
for every row that it sees."""

import numpy as np
import pytest
import torch

import mla_latent_kv_09_gb300 as m
import oracle
from test_chunk_gpu import attend, f64, ints, rand

pytestmark = pytest.mark.gpu

JUMPERS = torch.arange(5, 128, 32)  # one head of each 32


@pytest.fixture(scope="module", autouse=True)
def _build():
    from mla_latent_kv_09_gb300 import build
    build.build()
    m.load()
    assert torch.cuda.is_available()


def remainder(N, noise, at, fp8, seed):
    """A request of N rows and one token's query [128, 576].  Scores come from
    three position dims alone: row 0 is 12 to 14 above the others for most
    heads; row `at` 18 above them for the jumpers, and 13 for their neighbours on
    one side, which do not see row 0 so; the others' deviation is `noise`."""
    pages = N // 64 + 2
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:N // 64].to(torch.int32).cuda()[None]
    g = torch.Generator(device="cuda").manual_seed(seed)
    values = torch.rand((N, 512), generator=g, device="cuda") + 0.5
    values[0] = values[at] = 0.0
    pe = torch.zeros((N, 64), device="cuda")
    pe[0, 0] = pe[at, 1] = 16.0
    pe[:, 2] = noise * torch.randn(N, generator=g, device="cuda")
    pe[0, 2] = pe[at, 2] = 0.0
    if fp8:
        rows = torch.zeros((N, 656), dtype=torch.uint8, device="cuda")
        rows[:, :512] = values.to(torch.float8_e4m3fn).view(torch.uint8)
        rows[:, 512:516] = 127
        rows[:, 528:] = pe.bfloat16().view(torch.uint8)
        flat = oracle.fp8_rows_to_f64(rows.cpu().numpy())
    else:
        rows = torch.cat((values, pe), 1).bfloat16()
        flat = f64(rows)
    cache = torch.zeros((pages, 64, rows.shape[1]), dtype=rows.dtype, device="cuda")
    cache[table[0].long()] = rows.view(-1, 64, rows.shape[1])
    q = torch.zeros((128, 576), device="cuda")
    q[:, 512] = (12.0 + 0.5 * (torch.arange(128) % 5)) / 16
    q[:, 514] = 1.0
    q[JUMPERS, 512], q[JUMPERS, 513] = 0.0, 18.0 / 16
    q[JUMPERS + 1, 512], q[JUMPERS + 1, 513] = 0.0, 13.0 / 16
    return cache, table, flat, q.bfloat16()


def of_allowed(got, ref, allowed):
    """The largest error, of what is allowed (NaN: a result that is no number)."""
    ref, allowed = (torch.tensor(x, device="cuda") for x in (ref, allowed))
    return float(((got.double() - ref).abs() / allowed).max())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("noise", [1.0, 0.0])
@pytest.mark.parametrize("N", [8192, 65536])
def test_a_light_remainder_keeps_its_mass(N, noise, fp8):
    """Heads with nothing new beside one that jumps, the one that jumps, and ones
    that jump less: 128 tokens with the same query see the same rows, some of
    their pairs in one piece and some cut."""
    cache, table, flat, q = remainder(N, noise, N // 8, fp8, 7)
    x = q.expand(128, 128, 576).contiguous()
    out, lse = attend(x, cache, table, ints([N]), 1.0, causal=False, out_fp32=True)
    ref, ref_lse = oracle.chunk_attend(f64(q)[None], [flat], [0, 1], 1.0, False)
    bo, bl = oracle.chunk_error_bound(f64(q)[None], [flat], [0, 1], 1.0, ref, False)
    allowed = bo + 2.0 ** -24 * (np.abs(ref) + bo)
    assert of_allowed(out, ref, allowed) <= 1 and of_allowed(lse, ref_lse, bl) <= 1
    # and so does a decode step's
    o2, _ = m.decode_step(x[:2][None], cache, table, ints([N]), 1.0, out_fp32=True)
    assert of_allowed(o2[0], ref, allowed) <= 1


@pytest.mark.parametrize("N", [8192, 65536])
def test_a_heads_result_does_not_depend_on_its_neighbours(N):
    """The same heads with and without jumping ones among them: where the
    reference moves differently weights are rounded differently, each time
    within the bound around the same result."""
    cache, table, flat, q = remainder(N, 1.0, N // 8, False, 8)
    calm = q.clone()
    calm[JUMPERS] = q[JUMPERS - 1]
    outs = [attend(y.expand(128, 128, 576).contiguous(), cache, table, ints([N]), 1.0, causal=False, out_fp32=True)
            for y in (q, calm)]
    same = torch.ones(128, dtype=torch.bool)
    same[JUMPERS] = False
    ref = oracle.chunk_attend(f64(q)[None], [flat], [0, 1], 1.0, False)[0]
    bo, _ = oracle.chunk_error_bound(f64(q)[None], [flat], [0, 1], 1.0, ref, False)
    allowed = 2 * (bo + 2.0 ** -24 * (np.abs(ref) + bo))
    assert of_allowed(outs[0][0][:, same], f64(outs[1][0])[:, same], allowed[:, same]) <= 1


def test_a_prompts_chunk_with_sinks():
    """A causal chunk of 256 different tokens over 8192 rows, most of the softmax on
    row 0 and values of mean 1: single tokens against their definition."""
    N, T = 8192, 256
    cache, table, flat, q = remainder(N, 1.0, 1000, False, 9)
    x = q.expand(T, 128, 576).clone()
    x[..., 515:] = rand((T, 128, 61), 10) * 0.25
    flat_rows = cache.view(-1, 576)
    j = torch.arange(N, device="cuda")
    place = table[0].long()[j // 64] * 64 + j % 64
    flat_rows[place, 515:] = rand((N, 61), 11) * 0.25
    rows = f64(flat_rows[place])
    out, lse = attend(x, cache, table, ints([N]), 1.0, out_fp32=True)
    for t in (0, 1, 100, 254, 255):
        seen = [rows[:N - T + t + 1]]
        ref, ref_lse = oracle.chunk_attend(f64(x[t:t + 1]), seen, [0, 1], 1.0)
        bo, bl = oracle.chunk_error_bound(f64(x[t:t + 1]), seen, [0, 1], 1.0, ref)
        assert of_allowed(out[t:t + 1], ref, bo + 2.0 ** -24 * (np.abs(ref) + bo)) <= 1
        assert of_allowed(lse[t:t + 1], ref_lse, bl) <= 1
