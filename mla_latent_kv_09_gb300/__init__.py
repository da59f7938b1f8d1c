"""GB300 (sm_103a) weight-absorbed MLA decode over a paged latent KV cache.

The computation lives in libmla_decode.so (CUDA, hand-written tcgen05/TMA
kernels); this package is its Python face:

  * the C-ABI entry points under their C names (mla_decode_plan, mla_decode,
    mla_combine, ...) taking raw pointers or torch tensors;
  * `decode_step`, which allocates the outputs and runs plan -> decode ->
    combine on the current stream;
  * `decode_step_host`, the same call for host-resident inputs (copies in,
    runs, copies the outputs back);
  * `absorb_q` / `absorb_o`, the weight-absorption BMMs on either side of
    the attention (query through W_UK, output through W_UV);
  * `indexer_scores` / `topk_indices`, the sparse-attention indexer that
    produces the top-k lists the sparse decode consumes;
  * `rope` / `rope_frequencies` / `softmax_scale` and `cache_append`, which
    turn the RoPE dims and put tokens into the paged latent cache;
  * `prefix_expand` / `prefix_attend`, attention for a batch that shares a
    long prefix: its keys and values expanded once, attended to by all.

PyTorch is used only to allocate device memory and to name streams.
"""

from __future__ import annotations

from ._binding import (  # noqa: F401
    MLA_ERR_BAD_INDEX,
    MLA_ERR_BAD_TABLE,
    MLA_ERR_CUDA,
    MLA_ERR_DEVICE,
    MLA_ERR_INVALID_ARG,
    MLA_ERR_TIMEOUT,
    MLA_ERR_UNSUPPORTED,
    MLA_ERR_VALUE_RANGE,
    MLA_ERR_WORKSPACE,
    MLA_FLAG_CAUSAL,
    MLA_FLAG_BF16_PV,
    MLA_FLAG_KV_FP8,
    MLA_FLAG_OUT_FP32,
    MLA_FLAG_ROPE_HALF,
    MLA_FLAG_ROPE_INVERSE,
    MLA_FLAG_VALIDATE,
    MLA_OK,
    SIGNATURES,
    MlaError,
    load,
    mla_absorb_o,
    mla_absorb_q,
    mla_cache_append,
    mla_indexer_scores,
    mla_prefix_attend,
    mla_prefix_attend_workspace_size,
    mla_prefix_expand,
    mla_rope,
    mla_topk,
    mla_combine,
    mla_decode,
    mla_decode_noalloc,
    mla_noalloc_status,
    mla_noalloc_workspace,
    mla_decode_plan,
    mla_decode_plan_host,
    mla_decode_workspace_size,
    mla_default_num_units,
    mla_status_string,
    mla_workspace_status,
    mla_selftest_wait_timeout,
)

NUM_HEADS = 128
D_QK = 576
D_V = 512
PAGE = 64


class Workspace:
    """A device workspace sized for (batch, s_q, num_units)."""

    def __init__(self, batch: int, s_q: int, num_units: int = 0, device=None):
        import torch
        self.batch, self.s_q = batch, s_q
        self.num_units = num_units or mla_default_num_units(s_q)
        self.nbytes = mla_decode_workspace_size(batch, s_q, NUM_HEADS, self.num_units)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")


def decode_step(q, kv_cache, block_table, cache_lens, softmax_scale: float, *, causal: bool = False,
                topk_idx=None, out_fp32: bool = False, validate: bool = False, bf16_pv: bool = False,
                num_units: int = 0, workspace: Workspace | None = None, out=None, lse=None, stream=None):
    """One MLA decode step on device tensors: plan, attention, combine.

    q [B, s_q, 128, 576] bf16; kv_cache [num_pages, 64, 576] bf16, or
    uint8 [num_pages, 64, 656] FP8 rows (MLA_FLAG_KV_FP8 is then set);
    block_table [B, W] int32; cache_lens [B] int32; topk_idx [B, s_q, k]
    int32 or None.  bf16_pv selects MLA_FLAG_BF16_PV (two-token dense path:
    faster, less precise value product).  With validate=True the inputs are
    checked on the device first and the step's status is read back (a host
    synchronisation) and raised as MlaError if it is not MLA_OK.
    Returns (O [B, s_q, 128, 512] bf16 or fp32, LSE fp32).
    """
    import torch
    B, s_q = q.shape[0], q.shape[1]
    if workspace is None:
        workspace = Workspace(B, s_q, num_units, q.device)
    U = workspace.num_units
    if out is None:
        out = torch.empty((B, s_q, NUM_HEADS, D_V), dtype=torch.float32 if out_fp32 else torch.bfloat16,
                          device=q.device)
    if lse is None:
        lse = torch.empty((B, s_q, NUM_HEADS), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    topk = 0 if topk_idx is None else topk_idx.shape[-1]
    flags = (MLA_FLAG_CAUSAL if causal else 0) | (MLA_FLAG_OUT_FP32 if out_fp32 else 0) | (
        MLA_FLAG_VALIDATE if validate else 0) | (MLA_FLAG_BF16_PV if bf16_pv else 0)
    if kv_cache.dtype == torch.uint8:
        flags |= MLA_FLAG_KV_FP8
    mla_decode_plan(cache_lens, B, s_q, topk, U, workspace.buf, workspace.nbytes, stream)
    mla_decode(q, kv_cache, kv_cache.shape[0], block_table, block_table.stride(0), cache_lens, B, s_q,
               NUM_HEADS, softmax_scale, topk_idx, topk, flags, U, workspace.buf, workspace.nbytes, out,
               lse, stream)
    mla_combine(workspace.buf, workspace.nbytes, B, s_q, NUM_HEADS, flags, U, out, lse, stream)
    if validate:
        # the check runs on the device; its outcome is read back here (the
        # C calls themselves never synchronise for it)
        status = mla_workspace_status(workspace.buf, stream)
        if status != MLA_OK:
            raise MlaError("mla_decode (validate)", status)
    return out, lse


def decode_step_host(q, kv_cache, block_table, cache_lens, softmax_scale: float, *, device="cuda",
                     causal: bool = False, topk_idx=None, out_fp32: bool = False, bf16_pv: bool = False,
                     num_units: int = 0,
                     workspace: Workspace | None = None, dev_buffers=None, out_host=None, lse_host=None):
    """decode_step for HOST tensors (pinned for speed): H2D copies, the step,
    D2H copies of O and LSE.  `dev_buffers` may hold preallocated device
    tensors with the same keys as the inputs to avoid allocation per call."""
    import torch
    d = dev_buffers or {}

    def up(name, t):
        if t is None:
            return None
        dst = d.get(name)
        if dst is None:
            dst = torch.empty(t.shape, dtype=t.dtype, device=device)
        dst.copy_(t, non_blocking=True)
        return dst

    o, l = decode_step(up("q", q), up("kv_cache", kv_cache), up("block_table", block_table),
                       up("cache_lens", cache_lens), softmax_scale, causal=causal,
                       topk_idx=up("topk_idx", topk_idx), out_fp32=out_fp32, bf16_pv=bf16_pv,
                       num_units=num_units,
                       workspace=workspace, out=d.get("out"), lse=d.get("lse"))
    if out_host is None:
        out_host = torch.empty(o.shape, dtype=o.dtype, pin_memory=True)
    if lse_host is None:
        lse_host = torch.empty(l.shape, dtype=l.dtype, pin_memory=True)
    out_host.copy_(o, non_blocking=True)
    lse_host.copy_(l, non_blocking=True)
    torch.cuda.current_stream(device).synchronize()
    return out_host, lse_host


def _rows(t, dims: int, name: str) -> int:
    """Row stride of a token-major [T, H, dims] activation whose rows may be
    spaced wider than `dims` (e.g. a slice of a [T, H, 192] tensor)."""
    if t.dim() != 3 or t.shape[2] != dims or t.stride(2) != 1 or t.stride(0) != t.shape[1] * t.stride(1):
        raise ValueError(f"{name}: expected [T, H, {dims}] with unit stride in the last dim and rows "
                         "evenly spaced over (token, head)")
    return t.stride(1)


def absorb_q(q_nope, w_uk, q_pe=None, *, out=None, status=None, stream=None):
    """Query-side absorption: q_latent[t, h] = W_UK[h] @ q_nope[t, h].

    q_nope [T, H, 128] bf16 (rows may be strided, e.g. [..., :128] of a
    [T, H, 192] projection output), w_uk [H, 512, 128] bf16, q_pe [T, H, 64]
    bf16 with the same row stride, or None.  Returns `out`, by default a new
    [T, H, 576] tensor (the decode attention's query) with the RoPE dims in
    512..575, or [T, H, 512] without q_pe.  `status` (int32 device tensor,
    one element) receives MLA_ERR_TIMEOUT if a device wait runs out.
    """
    import torch
    T, H = q_nope.shape[0], q_nope.shape[1]
    q_stride = _rows(q_nope, 128, "q_nope")
    if q_pe is not None and _rows(q_pe, 64, "q_pe") != q_stride:
        raise ValueError("q_pe must have the row stride of q_nope")
    if out is None:
        out = torch.empty((T, H, D_QK if q_pe is not None else D_V), dtype=torch.bfloat16, device=q_nope.device)
    out_stride = _rows(out, out.shape[2], "out")
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=q_nope.device)
    if stream is None:
        stream = torch.cuda.current_stream(q_nope.device)
    mla_absorb_q(q_nope, q_pe, q_stride, w_uk, T, H, out, out_stride, status, stream)
    return out


def absorb_o(o, w_uv, *, out=None, status=None, stream=None):
    """Output-side absorption: out[t, h] = O[t, h] @ W_UV[h].

    o [T, H, 512] bf16 (the decode attention's output), w_uv [H, 512, 128]
    bf16.  Returns `out`, by default a new [T, H, 128] bf16 tensor.
    """
    import torch
    T, H = o.shape[0], o.shape[1]
    o_stride = _rows(o, 512, "o")
    if out is None:
        out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=o.device)
    out_stride = _rows(out, 128, "out")
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=o.device)
    if stream is None:
        stream = torch.cuda.current_stream(o.device)
    mla_absorb_o(o, o_stride, w_uv, T, H, out, out_stride, status, stream)
    return out


def indexer_scores(q_idx, w_idx, k_idx_cache, block_table, cache_lens, *, causal: bool = False,
                   max_len: int | None = None, scores=None, status=None, stream=None):
    """Index scores of every visible position.

    q_idx [B, s_q, 64, 128] bf16, w_idx [B, s_q, 64] fp32, k_idx_cache
    [num_pages, 64, 128] bf16 (paged like the latent cache, same block
    table).  Returns `scores` (default a new fp32 [B, s_q, max_len] tensor;
    positions past a token's visible count are left unwritten).
    """
    import torch
    B, s_q = q_idx.shape[0], q_idx.shape[1]
    if max_len is None:
        max_len = block_table.shape[1] * PAGE
    if scores is None:
        stride = (max_len + 3) // 4 * 4
        scores = torch.empty((B, s_q, stride), dtype=torch.float32, device=q_idx.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=q_idx.device)
    if stream is None:
        stream = torch.cuda.current_stream(q_idx.device)
    mla_indexer_scores(q_idx, w_idx, k_idx_cache, k_idx_cache.shape[0], block_table, block_table.stride(0),
                       cache_lens, B, s_q, MLA_FLAG_CAUSAL if causal else 0, max_len, scores, scores.stride(1),
                       status, stream)
    return scores


def topk_indices(scores, cache_lens, topk: int, *, causal: bool = False, max_len: int | None = None, out=None,
                 status=None, stream=None):
    """Top-k lists [B, s_q, topk] int32 (increasing positions, -1 padded)
    from index scores [B, s_q, stride] (as `indexer_scores` returns them)."""
    import torch
    B, s_q = scores.shape[0], scores.shape[1]
    if max_len is None:
        max_len = scores.shape[2]
    if out is None:
        out = torch.empty((B, s_q, topk), dtype=torch.int32, device=scores.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=scores.device)
    if stream is None:
        stream = torch.cuda.current_stream(scores.device)
    mla_topk(scores, scores.stride(1), cache_lens, B, s_q, MLA_FLAG_CAUSAL if causal else 0, max_len, topk, out,
             status, stream)
    return out


def _tensor(t, name: str, dtype, shape, device, contiguous: bool = True):
    """Checks a tensor argument: its type, shape and device, and that it is
    contiguous, or with contiguous=False that its last dim is (whose stride says
    nothing if it is one).  (Called for every tensor of a call that may be
    shorter than ten of these checks: it does little, and words are found only
    for a failure.)"""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not (
            t.is_contiguous() if contiguous else t.stride(-1) == 1 or t.shape[-1] == 1):
        raise ValueError(f"{name}: expected {dtype} {list(shape)} on GPU {device}, "
                         f"{'contiguous' if contiguous else 'unit stride in the last dim'}; got {t.dtype} "
                         f"{list(t.shape)} on {t.device}, strides {list(t.stride())}")


def _elsewhere(first, stream, name: str):
    """What has to be entered for a call on first's device and on `stream` (a
    torch stream, or its raw handle): with that stream current the kernels are
    launched there, and what the call allocates belongs to it."""
    import torch
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"{name}: expected tensors on a GPU, got {dev}")
    if stream is None:
        return torch.cuda.device(dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    if stream.device != dev:
        raise ValueError(f"{name}: a stream of {stream.device} for tensors of {dev}")
    return torch.cuda.stream(stream)


def rope_frequencies(rope_dim: int, base: float = 10000.0, *, linear: float = 1.0, yarn: float = 1.0,
                     original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Frequencies of a rotation of `rope_dim` dims, for `rope` and
    `cache_append`: (fp64 [rope_dim / 2] radians per position, YaRN's factor).

    Pair i turns by base^(-2i / rope_dim) a position.  For contexts longer
    than the `original_len` a model was trained on: `linear` divides every
    frequency (position interpolation); `yarn` is YaRN's stretch: pairs of
    fewer than beta_slow turns over original_len are slowed down by it, pairs
    of more than beta_fast turns are kept, those between are blended linearly
    over the pair's index, and the factor is 0.1 ln(yarn) + 1 (else 1).

    The factor belongs on the whole query and the whole key, squared on their
    score.  Heads of which every dim turns may have it as `rope`'s and
    `cache_append`'s scale.  Heads of which only a part turns (MLA: 64 of 192)
    must not, or it would weigh the turned part of a score against the rest:
    there the rotations keep their scale of 1, and the attention takes
    `softmax_scale(head_dim, factor)`.
    """
    import math

    import torch
    if rope_dim < 2 or rope_dim % 2 or not base > 1 or not linear >= 1 or not yarn >= 1 or not original_len > 0:
        raise ValueError("rope_frequencies: rope_dim must be even, base > 1, linear and yarn >= 1, original_len > 0")
    if not beta_fast > beta_slow > 0:
        raise ValueError("rope_frequencies: beta_fast > beta_slow > 0")
    index = torch.arange(rope_dim // 2, dtype=torch.float64)
    inv = base ** (-2 * index / rope_dim) / linear
    factor = 1.0
    if yarn > 1:
        # the (fractional) index whose pair makes `beta` turns over original_len
        def at(beta):
            return rope_dim * math.log(original_len / (2 * math.pi * beta)) / (2 * math.log(base))
        low, high = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rope_dim - 1)
        slow = ((index - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        inv = inv / yarn * slow + inv * (1 - slow)
        factor = 0.1 * math.log(yarn) + 1.0
    return inv.to(device), factor


def softmax_scale(head_dim: int = 192, factor: float = 1.0) -> float:
    """The attention's softmax scale, factor^2 / sqrt(head_dim): `head_dim` dims
    of a query and a key before absorption (MLA: 128 + 64), `factor` as
    `rope_frequencies` returns it."""
    if head_dim < 1 or not 0 < factor < float("inf"):
        raise ValueError("softmax_scale: head_dim >= 1, factor > 0 and finite")
    return factor * factor * head_dim ** -0.5


def rope(x, positions, inv_freq, *, offset: int = 0, half: bool = False, inverse: bool = False, scale: float = 1.0,
         out=None, stream=None):
    """Rotary positions over part of each head.

    x [T, H, D] bf16 (tokens and heads may be strided), positions [T] int32,
    inv_freq [R / 2] fp64 (see `rope_frequencies`; below 2^52): dims [offset, offset + R)
    of row (t, h) are turned by positions[t] * inv_freq and multiplied by
    `scale`, the others copied.  Pairs are (2i, 2i + 1), or (i, i + R / 2)
    with half=True; inverse=True turns back (the gradient of the rotation, and
    with scale 1 its inverse).  Returns `out`, by default a new [T, H, D]
    tensor; out=x turns in place (and leaves the other dims alone); `out` and
    x must not overlap otherwise.
    """
    import torch
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != torch._C._cuda_getDevice():
        with _elsewhere(x, stream, "rope"):
            return rope(x, positions, inv_freq, offset=offset, half=half, inverse=inverse, scale=scale, out=out)
    T, H, D = x.shape
    _tensor(x, "x", torch.bfloat16, (T, H, D), dev, contiguous=False)
    _tensor(positions, "positions", torch.int32, (T,), dev)
    R2, = inv_freq.shape
    _tensor(inv_freq, "inv_freq", torch.float64, (R2,), dev)
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
    else:
        _tensor(out, "out", torch.bfloat16, (T, H, D), dev, contiguous=False)
    if T == 0 or H == 0:
        return out
    # (torch.cuda.current_stream builds a stream object, twenty times as long)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    # (the stride of a dim of one says nothing)
    mla_rope(x, x.stride(0) if T > 1 else 0, x.stride(1) if H > 1 else 0, positions, T, H, D, offset, 2 * R2, inv_freq,
             scale, (MLA_FLAG_ROPE_HALF if half else 0) | (MLA_FLAG_ROPE_INVERSE if inverse else 0), out,
             out.stride(0) if T > 1 else 0, out.stride(1) if H > 1 else 0, stream)
    return out


def _cache_flags(kv_cache, device) -> int:
    import torch
    if kv_cache.dtype == torch.uint8:
        _tensor(kv_cache, "kv_cache", torch.uint8, (kv_cache.shape[0], PAGE, 656), device)
        return MLA_FLAG_KV_FP8
    _tensor(kv_cache, "kv_cache", torch.bfloat16, (kv_cache.shape[0], PAGE, D_QK), device)
    return 0


def cache_append(latent, k_pe, kv_cache, block_table, positions, *, request_ids=None, norm_weight=None,
                 eps: float = 1e-6, inv_freq=None, half: bool = False, rope_scale: float = 1.0, status=None,
                 stream=None):
    """Append tokens to the paged latent cache.

    latent [T, 512] and k_pe [T, 64] bf16 (rows may be strided: the two parts
    of a [T, 576] projection output); kv_cache [num_pages, 64, 576] bf16 or
    uint8 [num_pages, 64, 656] FP8 rows; block_table [B, W] int32 (rows may be
    strided), positions
    [T] int32, token t's position in its request (negative: padding, nothing
    is written); request_ids [T] int32, or None when the tokens are B equal
    runs in order.  With norm_weight [512] bf16 the latent is RMS-normed with
    `eps` first; with inv_freq [32] fp64 k_pe is turned by its position (as
    `rope` does, with `half` and `rope_scale`).  No two tokens may name the
    same row.  `status` (int32 device tensor, one element) receives
    MLA_ERR_BAD_TABLE if a token's request, position or page is out of range;
    that token is skipped (without a `status` nobody learns of it).  Returns
    kv_cache.
    """
    import torch
    dev = latent.get_device()
    if stream is not None or dev < 0 or dev != torch._C._cuda_getDevice():
        with _elsewhere(latent, stream, "cache_append"):
            return cache_append(latent, k_pe, kv_cache, block_table, positions, request_ids=request_ids,
                                norm_weight=norm_weight, eps=eps, inv_freq=inv_freq, half=half, rope_scale=rope_scale,
                                status=status)
    T = latent.shape[0]
    _tensor(latent, "latent", torch.bfloat16, (T, D_V), dev, contiguous=False)
    _tensor(k_pe, "k_pe", torch.bfloat16, (T, D_QK - D_V), dev, contiguous=False)
    flags = _cache_flags(kv_cache, dev)
    B, width = block_table.shape
    _tensor(block_table, "block_table", torch.int32, (B, width), dev, contiguous=False)
    _tensor(positions, "positions", torch.int32, (T,), dev)
    if request_ids is not None:
        _tensor(request_ids, "request_ids", torch.int32, (T,), dev)
    if norm_weight is not None:
        _tensor(norm_weight, "norm_weight", torch.bfloat16, (D_V,), dev)
    if inv_freq is not None:
        _tensor(inv_freq, "inv_freq", torch.float64, ((D_QK - D_V) // 2,), dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    else:
        _tensor(status, "status", torch.int32, status.shape, dev)
    if T == 0:
        return kv_cache
    # (the stride of a dim of one says nothing)
    bt_stride = block_table.stride(0) if B > 1 else width
    if bt_stride < width:
        raise ValueError("block_table: its rows overlap")
    stream = torch._C._cuda_getCurrentRawStream(dev)
    mla_cache_append(latent, latent.stride(0) if T > 1 else D_V, k_pe, k_pe.stride(0) if T > 1 else D_QK - D_V,
                     norm_weight, eps, inv_freq, rope_scale, positions, request_ids, T, block_table, bt_stride, width,
                     B, kv_cache, kv_cache.shape[0], flags | (MLA_FLAG_ROPE_HALF if half else 0), status, stream)
    return kv_cache


def prefix_expand(kv_cache, block_table, prefix_len: int, w_uk, w_uv, *, out=None, status=None, stream=None):
    """Per-head keys and values of a shared prefix, from its cached latents.

    kv_cache [num_pages, 64, 576] bf16 or uint8 [num_pages, 64, 656] FP8
    rows; block_table [W] int32, the prefix's pages in order; w_uk, w_uv
    [H, 512, 128] bf16 (as for `absorb_q` / `absorb_o`).  Returns (k_nope
    [H, R, 128] bf16, k_pe [R, 64] bf16, v [H, R, 128] fp16), by default new
    with R = prefix_len; `out` may hold them with any R >= prefix_len, whose
    further rows are left as they are.  `status` (int32 device tensor, one
    element; without it nobody learns of these) receives MLA_ERR_BAD_TABLE for a
    page outside the pool and MLA_ERR_VALUE_RANGE for a key or value that is not
    finite once rounded.
    """
    import torch
    dev = kv_cache.get_device()
    if stream is not None or dev < 0 or dev != torch._C._cuda_getDevice():
        with _elsewhere(kv_cache, stream, "prefix_expand"):
            return prefix_expand(kv_cache, block_table, prefix_len, w_uk, w_uv, out=out, status=status)
    flags = _cache_flags(kv_cache, dev)
    pages, = block_table.shape
    _tensor(block_table, "block_table", torch.int32, (pages,), dev)
    if prefix_len < 0 or prefix_len > pages * PAGE:
        raise ValueError("prefix_len: outside the block table")
    H = w_uk.shape[0]
    _tensor(w_uk, "w_uk", torch.bfloat16, (H, D_V, 128), dev)
    _tensor(w_uv, "w_uv", torch.bfloat16, (H, D_V, 128), dev)
    if out is None:
        out = (torch.empty((H, prefix_len, 128), dtype=torch.bfloat16, device=dev),
               torch.empty((prefix_len, D_QK - D_V), dtype=torch.bfloat16, device=dev),
               torch.empty((H, prefix_len, 128), dtype=torch.float16, device=dev))
    k_nope, k_pe, v = out
    R = k_nope.shape[1]
    _tensor(k_nope, "k_nope", torch.bfloat16, (H, R, 128), dev)
    _tensor(k_pe, "k_pe", torch.bfloat16, (R, D_QK - D_V), dev)
    _tensor(v, "v", torch.float16, (H, R, 128), dev)
    if R < prefix_len:
        raise ValueError("out: fewer rows than prefix_len")
    if prefix_len == 0:
        return out
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    else:
        _tensor(status, "status", torch.int32, status.shape, dev)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    mla_prefix_expand(kv_cache, kv_cache.shape[0], block_table, prefix_len, w_uk, w_uv, H, flags, k_nope, v, R, k_pe,
                      status, stream)
    return out


def prefix_attend(q_nope, q_pe, k_nope, k_pe, v, softmax_scale: float, *, prefix_len: int | None = None, visible=None,
                  suffix_out=None, suffix_lse=None, out_fp32: bool = False, out=None, lse=None, workspace=None,
                  status=None, stream=None):
    """Attention of T query tokens over one shared, expanded prefix.

    q_nope [T, H, 128], q_pe [T, H, 64] bf16 with one row stride (slices of a
    [T, H, 192] projection output q, turned by rope(q, ..., offset=128, out=q));
    k_nope [H, R, 128], k_pe [R, 64], v [H, R, 128] as `prefix_expand` returns
    them, of which the first prefix_len (default R) rows count; every value of
    them finite.
    visible [T] int32: token t sees the first visible[t] rows only (padded
    tokens: 0).  suffix_out [T, H, 128] bf16 and suffix_lse [T, H] fp32: what
    each (token, head) attended to elsewhere (`decode_step`'s output through
    `absorb_o`, and its LSE); the result is then the attention over both.
    Returns (out [T, H, 128] bf16 or fp32, lse [T, H] fp32); out and lse may
    be suffix_out and suffix_lse themselves.  `workspace` (uint8,
    mla_prefix_attend_workspace_size bytes) is allocated if not given; `status`
    receives MLA_ERR_TIMEOUT if a device wait runs out.
    """
    import torch
    dev = q_nope.get_device()
    if stream is not None or dev < 0 or dev != torch._C._cuda_getDevice():
        with _elsewhere(q_nope, stream, "prefix_attend"):
            return prefix_attend(q_nope, q_pe, k_nope, k_pe, v, softmax_scale, prefix_len=prefix_len, visible=visible,
                                 suffix_out=suffix_out, suffix_lse=suffix_lse, out_fp32=out_fp32, out=out, lse=lse,
                                 workspace=workspace, status=status)
    T, H, _ = q_nope.shape
    _tensor(q_nope, "q_nope", torch.bfloat16, (T, H, 128), dev, contiguous=False)
    _tensor(q_pe, "q_pe", torch.bfloat16, (T, H, 64), dev, contiguous=False)
    R = k_nope.shape[1]
    _tensor(k_nope, "k_nope", torch.bfloat16, (H, R, 128), dev)
    _tensor(k_pe, "k_pe", torch.bfloat16, (R, 64), dev)
    _tensor(v, "v", torch.float16, (H, R, 128), dev)
    if prefix_len is None:
        prefix_len = R
    elif prefix_len < 0 or prefix_len > R:
        raise ValueError("prefix_len: outside the expanded rows")
    if visible is not None:
        _tensor(visible, "visible", torch.int32, (T,), dev)
    if (suffix_out is None) != (suffix_lse is None):
        raise ValueError("suffix_out and suffix_lse come together")
    if suffix_out is not None:
        _tensor(suffix_out, "suffix_out", torch.bfloat16, (T, H, 128), dev)
        _tensor(suffix_lse, "suffix_lse", torch.float32, (T, H), dev)
    if out is None:
        out = torch.empty((T, H, 128), dtype=torch.float32 if out_fp32 else torch.bfloat16, device=dev)
    else:
        _tensor(out, "out", torch.float32 if out_fp32 else torch.bfloat16, (T, H, 128), dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _tensor(lse, "lse", torch.float32, (T, H), dev)
    if T == 0 or H == 0:
        return out, lse
    # the distance between rows (the stride of a dim of one says nothing about it)
    q_stride = q_nope.stride(1) if H > 1 else q_nope.stride(0) if T > 1 else D_QK
    if (T > 1 and not q_nope.stride(0) == q_pe.stride(0) == H * q_stride) or (
            H > 1 and not q_nope.stride(1) == q_pe.stride(1) == q_stride):
        raise ValueError("q_nope, q_pe: expected rows evenly spaced over (token, head), with one stride")
    if workspace is None:
        need = mla_prefix_attend_workspace_size(T, H, prefix_len)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        _tensor(workspace, "workspace", torch.uint8, workspace.shape, dev)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    else:
        _tensor(status, "status", torch.int32, status.shape, dev)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    mla_prefix_attend(q_nope, q_pe, q_stride, k_nope, v, R, k_pe, prefix_len, visible, T, H, softmax_scale,
                      suffix_out, suffix_lse, MLA_FLAG_OUT_FP32 if out_fp32 else 0, workspace,
                      0 if workspace is None else workspace.numel(), out, lse, status, stream)
    return out, lse
