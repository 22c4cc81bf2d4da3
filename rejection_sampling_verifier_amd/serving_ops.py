"""Binding of the operators around a verification step (spec_verify.h, "Operators
around a verification step"): torch tensors in, device pointers out.

As in ``binding``, every step runs in the library's HIP kernels, a call is
enqueued on the current (or given) stream and nothing is synchronised.
Outputs and workspaces that a call allocates belong to the stream it runs on.
"""

from __future__ import annotations

import ctypes
import operator

import torch

from .binding import (SV_BF16, SV_E4M3, SV_INT8, SV_MAX_BLOCKS, SV_MAX_K, SvCache, SvControls, SvPrefix, SvRotary,
                      _cached_workspace, _check, _dtype_code, _OnStream, _stream_handle, load_library)

_KINDS = {"e4m3": SV_E4M3, "int8": SV_INT8}


class _Elsewhere:
    """Makes the device current and puts allocations on the stream, for a call
    that runs on another device or stream than the current ones."""

    def __init__(self, dev, handle):
        self.device, self.stream = torch.cuda.device(dev), _OnStream(dev, handle)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


class _Here:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_HERE = _Here()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _scope(dev, stream):
    """(stream handle, context to allocate and launch in)."""
    if stream is None and _raw_stream is not None and dev.index == torch.cuda.current_device():
        return _raw_stream(dev.index), _HERE
    handle = _stream_handle(dev, stream)
    return handle, _Elsewhere(dev, handle)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on a GPU device")
    return t.device


def _need(name, t, shape, dtype, dev):
    """A contiguous tensor of this shape (None: any size there), type and device."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape == shape and t.dtype is dtype and t.device == dev and t.is_contiguous():
        return
    if (t.dtype != dtype or t.device != dev or t.dim() != len(shape)
            or any(w is not None and n != w for n, w in zip(t.shape, shape)) or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                         f"({', '.join('any' if w is None else str(w) for w in shape)}) on {dev}")


def _maybe(name, t, shape, dtype, dev):
    if t is not None:
        _need(name, t, shape, dtype, dev)


def _rows(name, t, B, dtype, dev):
    """A [B, n] tensor whose rows are contiguous; its row pitch in elements."""
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev or t.dim() != 2 or t.shape[0] != B
            or (t.shape[1] > 1 and t.stride(1) != 1) or (B > 1 and t.stride(0) < t.shape[1])):
        raise ValueError(f"{name} must be a {dtype} tensor of shape ({B}, any) on {dev} with contiguous rows")
    return t.stride(0) if B > 1 else t.shape[1]


def _p(t):
    return None if t is None else t.data_ptr()


def _count(n, most):
    """A whole number for a C int: those past `most` count as `most`, and negative ones, which are refused, as -1."""
    return max(-1, min(operator.index(n), most))


def _logit_strides(name, t):
    """(row, position) strides of a [B, P, V] tensor with contiguous logits."""
    B, P, V = t.shape
    row, pos, one = t.stride()
    if P == 1:
        pos = V
    if B == 1:
        row = P * pos
    if (V > 1 and one != 1) or pos < V or row < (P - 1) * pos + V:
        raise ValueError(f"{name} must have contiguous, non-overlapping rows of logits")
    return row, pos


def adjust_logits(logits, tokens=None, *, parents=None, history=None, history_lens=None, prompt_lens=None,
                  repetition=None, presence=None, frequency=None, bias_ids=None, bias_values=None, bias_lens=None,
                  mask=None, mask_rows=None, out=None, stream=None):
    """spec_verify_adjust_logits: penalties, biases and grammar masks on the
    logits of a step (see the header for the formulas).

    logits [B, P, V] bf16 or fp32 with contiguous rows (a slice of a padded
    vocabulary will do); tokens [B, >= P - 1] int32 of a chain, or [B, P] node
    tokens with parents [B, P] of a tree; history [B, any] int32 with
    history_lens [B] and prompt_lens [B] int32; repetition, presence,
    frequency [B] fp32; bias_ids int32 and bias_values fp32 [B, any], bias_lens
    [B] int32; mask [R, ceil(V / 32)] int32 words, mask_rows [B, P] int32 (-1:
    no mask; without mask_rows position (b, i) goes by mask row b P + i).

    Returns ``out`` (a new contiguous [B, P, V] tensor if None; ``out=logits``
    works in place).
    """
    dev = _gpu(logits, "logits")
    if logits.dim() != 3 or 0 in logits.shape:
        raise ValueError("logits must be [B, P, V]")
    B, P, V = logits.shape
    if V > 2 ** 31 - 1 or B > 2 ** 31 - 1:
        raise ValueError(f"logits are too large: {tuple(logits.shape)}")
    dt = _dtype_code(logits)
    in_row, in_pos = _logit_strides("logits", logits)
    i32, f32 = torch.int32, torch.float32
    c = SvControls()
    tok_stride = 0
    for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
        if t is not None:
            _need(name, t, (B,), f32, dev)
            setattr(c, name, t.data_ptr())
    penalties = repetition is not None or presence is not None or frequency is not None
    if tokens is not None:
        tok_stride = _rows("tokens", tokens, B, i32, dev)
    need = P if parents is not None else P - 1
    if penalties and P > 1 and (tokens is None or tokens.shape[1] < need):
        raise ValueError(f"tokens must hold at least {need} drafted tokens per row")
    _maybe("parents", parents, (B, P), i32, dev)
    if history is not None:
        c.history_stride, c.history_width = _rows("history", history, B, i32, dev), history.shape[1]
        if history_lens is None:
            raise ValueError("history needs history_lens")
        _need("history_lens", history_lens, (B,), i32, dev)
        _maybe("prompt_lens", prompt_lens, (B,), i32, dev)
        # an empty one is none: a width of 0 would mean the pitch
        c.history = history.data_ptr() if history.shape[1] else None
        c.history_lens, c.prompt_lens = history_lens.data_ptr(), _p(prompt_lens)
    if bias_ids is not None:
        _need("bias_ids", bias_ids, (B, None), i32, dev)
        _need("bias_values", bias_values, tuple(bias_ids.shape), f32, dev)
        _maybe("bias_lens", bias_lens, (B,), i32, dev)
        c.bias_ids, c.bias_values, c.bias_lens = bias_ids.data_ptr(), bias_values.data_ptr(), _p(bias_lens)
        c.bias_stride = bias_ids.shape[1]
    if mask is not None:
        _need("mask", mask, (None, (V + 31) // 32), i32, dev)
        _maybe("mask_rows", mask_rows, (B, P), i32, dev)
        if mask_rows is None and mask.shape[0] < B * P:
            raise ValueError(f"mask must hold {B * P} rows without mask_rows")
        c.mask, c.mask_rows, c.num_masks = mask.data_ptr(), _p(mask_rows), mask.shape[0]
    handle, scope = _scope(dev, stream)
    if out is None:
        with scope:
            out = torch.empty((B, P, V), dtype=logits.dtype, device=dev)
        out_row, out_pos = P * V, V
    elif (not isinstance(out, torch.Tensor) or tuple(out.shape) != (B, P, V) or out.dtype != logits.dtype
          or out.device != dev):
        raise ValueError(f"out must be a {logits.dtype} tensor of shape {(B, P, V)} on {dev}")
    else:
        out_row, out_pos = _logit_strides("out", out)
    with scope:
        _check(load_library().spec_verify_adjust_logits(
            logits.data_ptr(), in_row, in_pos, _p(tokens), tok_stride, _p(parents), ctypes.byref(c), B, P, V, dt,
            out.data_ptr(), out_row, out_pos, handle))
    return out


class KVCache:
    """The tensors of a paged 8-bit cache (sv_cache in the header), checked once.

    k_pages [num_pages, Hkv, page, D] and v_pages [num_pages, Hkv, D, page]
    uint8 codes, k_scale and v_scale [num_pages, Hkv] fp32, k_tail and v_tail
    [B, tail, Hkv, D] bf16, block_table [B, max_blocks] int32; kind "e4m3" or
    "int8".  A row's counters (positions, blocks) are passed to each call.
    The handle keeps the tensors: copy into them, their storage must not be
    replaced (another tensor in an attribute's place is refused).
    """

    def __init__(self, k_pages, v_pages, k_scale, v_scale, k_tail, v_tail, block_table, *, kind="e4m3"):
        if kind not in _KINDS:
            raise ValueError(f"kind must be one of {sorted(_KINDS)}, got {kind!r}")
        dev = _gpu(k_pages, "k_pages")
        if k_pages.dim() != 4 or not isinstance(k_tail, torch.Tensor) or k_tail.dim() != 4:
            raise ValueError("k_pages must be [num_pages, Hkv, page, D] and k_tail [B, tail, Hkv, D]")
        pages, Hkv, page, D = k_pages.shape
        B, tail = k_tail.shape[:2]
        _need("k_pages", k_pages, (pages, Hkv, page, D), torch.uint8, dev)
        _need("v_pages", v_pages, (pages, Hkv, D, page), torch.uint8, dev)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _need(name, t, (pages, Hkv), torch.float32, dev)
        for name, t in (("k_tail", k_tail), ("v_tail", v_tail)):
            _need(name, t, (B, tail, Hkv, D), torch.bfloat16, dev)
        _need("block_table", block_table, (B, None), torch.int32, dev)
        if 0 in (pages, Hkv, page, D, B, tail, block_table.shape[1]):
            raise ValueError("a cache's sizes must be at least 1")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.k_tail, self.v_tail, self.block_table, self.kind, self.device = k_tail, v_tail, block_table, kind, dev
        self.B, self.num_pages, self.Hkv, self.D, self.page = B, pages, Hkv, D, page
        self.max_blocks, self.tail = block_table.shape[1], tail
        self._c = SvCache(k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                          k_tail.data_ptr(), v_tail.data_ptr(), block_table.data_ptr(), B, pages, Hkv, D, page,
                          self.max_blocks, tail, _KINDS[kind])
        self._ref = ctypes.byref(self._c)
        self._sizes = {}  # workspace sizes by (T, H, parents, weights, prefix)
        self._made = True

    def __setattr__(self, name, value):
        if "_made" in self.__dict__:
            raise AttributeError(f"a KVCache keeps the tensors it was made of: copy into {name}, or make another")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        raise AttributeError(f"a KVCache keeps the tensors it was made of: {name} cannot be deleted")


def new_cache(B, num_pages, Hkv, D, page=64, max_blocks=None, max_new=SV_MAX_K + 1, kind="e4m3", device="cuda"):
    """An empty cache: no pages are assigned (block_table is -1), and the tails
    hold what a commit of up to max_new tokens needs."""
    dev = torch.device(device)
    if min(B, num_pages, Hkv, D, page, max_new) < 1 or (max_blocks is not None and max_blocks < 1):
        raise ValueError("a cache's sizes must be at least 1")
    tail = -(-(page - 1 + max_new) // page) * page
    z = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device=dev)  # noqa: E731
    table = torch.full((B, max_blocks if max_blocks is not None else max(1, num_pages // B)), -1, dtype=torch.int32,
                       device=dev)
    return KVCache(z((num_pages, Hkv, page, D), torch.uint8), z((num_pages, Hkv, D, page), torch.uint8),
                   torch.ones((num_pages, Hkv), device=dev), torch.ones((num_pages, Hkv), device=dev),
                   z((B, tail, Hkv, D), torch.bfloat16), z((B, tail, Hkv, D), torch.bfloat16), table, kind=kind)


def _token_strides(name, t, shape, dev):
    """(row, token) strides of a bf16 [B, T, heads, D] view whose heads lie side by side."""
    B, T, n, D = shape
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype is not torch.bfloat16 or t.device != dev:
        raise ValueError(f"{name} must be a bfloat16 tensor of shape {shape} on {dev}")
    row, tok, head, one = t.stride()
    if one != 1 or (n > 1 and head != D):
        raise ValueError(f"the heads of {name} must lie side by side")
    if T == 1:
        tok = n * D
    if B == 1:
        row = T * tok
    if tok % 8 or row % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned in every token")
    return row, tok


def _attention_bytes(cache, T, H, tree, weights, prefix=None):
    """prefix: None or (count, max_blocks)."""
    key = (T, H, tree, weights, prefix)
    n = cache._sizes.get(key)
    if n is None:
        size = ctypes.c_size_t(0)
        some = ctypes.c_void_p(256)  # tells the query which arguments the call will have
        shared = None if prefix is None else ctypes.byref(SvPrefix(256, 256, 256, *prefix))
        _check(load_library().spec_verify_attention_prefix(
            None, 0, 0, None, None, 0, 0, cache._ref, shared, None, None, some if tree else None, None, T, H, 1.0, None,
            some if weights else None, None, ctypes.byref(size), None))
        if len(cache._sizes) >= 1024:
            cache._sizes.clear()
        n = cache._sizes[key] = size.value
    return n


def attention_workspace_bytes(cache, T, H, *, tree=False, weights=False, prefix=None):
    """Bytes of workspace that cache_attention needs for T new tokens and H
    heads; prefix: the shape of prefix_table, if any (that of (1, 65536)
    serves every table)."""
    return _attention_bytes(cache, T, H, tree, weights, None if prefix is None else tuple(prefix))


def new_attention_workspace(cache, T, H, *, tree=False, weights=False, prefix=None):
    """A zero-filled workspace for cache_attention at this shape."""
    return torch.zeros(attention_workspace_bytes(cache, T, H, tree=tree, weights=weights, prefix=prefix),
                       dtype=torch.uint8, device=cache.device)


def _prefix(table, blocks, starts, dev):
    """sv_prefix of the arguments, or None."""
    if table is None:
        if blocks is not None or starts is not None:
            raise ValueError("prefix_blocks and prefix_starts need prefix_table")
        return None
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or 0 in table.shape:
        raise ValueError("prefix_table must be [count, max_blocks]")
    n, most = table.shape
    _need("prefix_table", table, (n, most), torch.int32, dev)
    _need("prefix_blocks", blocks, (n,), torch.int32, dev)
    _need("prefix_starts", starts, (n + 1,), torch.int32, dev)
    return SvPrefix(table.data_ptr(), blocks.data_ptr(), starts.data_ptr(), n, most)


def cache_attention(q, k_new, v_new, cache, positions, blocks, *, parents=None, query_lens=None, scale=None,
                    prefix_table=None, prefix_blocks=None, prefix_starts=None, weights=None, out=None, workspace=None,
                    stream=None):
    """spec_verify_attention: attention of a step's new tokens over the cache
    and over each other; with a prefix, spec_verify_attention_prefix: over the
    pages that rows share too (see the header).

    q [B, T, H, D], k_new and v_new [B, T, Hkv, D] bf16, views with D-sized
    heads side by side (slices of a fused projection will do); positions and
    blocks [B] int32; parents [B, T] int32 for trees; query_lens [B] int32;
    scale None: D ** -0.5.  weights: True or a [B, T, max_blocks] fp32 tensor to
    get every block's attention mass.  prefix_table [n, any], prefix_blocks [n]
    and prefix_starts [n + 1] int32: rows prefix_starts[i] to prefix_starts[i +
    1] - 1 see the first prefix_blocks[i] pages of prefix_table[i] before their
    own, each read once for all of them.

    Returns out [B, T, H, D], or (out, weights).  Tensors made here hold zeros
    behind query_lens.  A call given no workspace uses one cached for its
    shape, device and stream; under graph capture it makes one that belongs to
    the graph, and clears its counters in it.
    """
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    dev, B, D = cache.device, cache.B, cache.D
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or 0 in q.shape:
        raise ValueError("q must be [B, T, H, D]")
    T, H = q.shape[1], q.shape[2]
    q_row, q_tok = _token_strides("q", q, (B, T, H, D), dev)
    kv = _token_strides("k_new", k_new, (B, T, cache.Hkv, D), dev)
    if _token_strides("v_new", v_new, (B, T, cache.Hkv, D), dev) != kv:
        raise ValueError("k_new and v_new must have the same strides")
    _need("positions", positions, (B,), torch.int32, dev)
    _need("blocks", blocks, (B,), torch.int32, dev)
    _maybe("parents", parents, (B, T), torch.int32, dev)
    _maybe("query_lens", query_lens, (B,), torch.int32, dev)
    prefix = _prefix(prefix_table, prefix_blocks, prefix_starts, dev)
    # the size that serves every prefix: a table that grows must not mean another workspace
    shared = None if prefix is None else (1, SV_MAX_BLOCKS)
    handle, scope = _scope(dev, stream)
    need = _attention_bytes(cache, T, H, parents is not None, weights is not None and weights is not False, shared)
    with scope:
        make = torch.empty if query_lens is None else torch.zeros
        if weights is True:
            weights = make((B, T, cache.max_blocks), dtype=torch.float32, device=dev)
        elif weights is False:
            weights = None
        elif weights is not None:
            _need("weights", weights, (B, T, cache.max_blocks), torch.float32, dev)
        if out is None:
            out = make((B, T, H, D), dtype=torch.bfloat16, device=dev)
        else:
            _need("out", out, (B, T, H, D), torch.bfloat16, dev)
        if workspace is None:
            if torch.cuda.is_current_stream_capturing():
                # a workspace of the graph's own: graphs replayed at once must not share one.  Its counters,
                # all that has to be zero, are cleared in the graph.
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
                workspace[:4 * B * cache.Hkv * -(-(T * (H // cache.Hkv)) // 16)].zero_()
            else:
                key = (B, T, H, cache.Hkv, D, cache.page, cache.max_blocks, parents is not None, weights is not None,
                       shared)
                workspace = _cached_workspace("attention", key, need, dev, handle)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        n = ctypes.c_size_t(workspace.numel() * workspace.element_size())
        _check(load_library().spec_verify_attention_prefix(
            q.data_ptr(), q_row, q_tok, k_new.data_ptr(), v_new.data_ptr(), kv[0], kv[1], cache._ref,
            None if prefix is None else ctypes.byref(prefix), positions.data_ptr(), blocks.data_ptr(), _p(parents),
            _p(query_lens), T, H, D ** -0.5 if scale is None else scale, out.data_ptr(), _p(weights),
            workspace.data_ptr(), ctypes.byref(n), handle))
    return out if weights is None else (out, weights)


def cache_commit(cache, k_new, v_new, num_accepted, positions, blocks, *, nodes=None, weights=None, totals=None,
                 positions_out=None, blocks_out=None, totals_out=None, stream=None):
    """spec_verify_commit: the accepted path's keys and values enter the cache
    (see the header).

    k_new, v_new as cache_attention's; num_accepted [B] int32 and, for trees,
    nodes [B, >= T - 1] int32 as verify and verify_tree return them; weights
    [B, T, max_blocks] fp32 as cache_attention returns them, totals [B,
    max_blocks] fp32.

    Writes the cache's pages, scales and tails, and returns (positions,
    blocks), or (positions, blocks, totals) where totals is given: new tensors,
    or the given outs, which may be the inputs themselves.
    """
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    dev, B, i32 = cache.device, cache.B, torch.int32
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 4 or 0 in k_new.shape:
        raise ValueError("k_new must be [B, T, Hkv, D]")
    T = k_new.shape[1]
    kv = _token_strides("k_new", k_new, (B, T, cache.Hkv, cache.D), dev)
    if _token_strides("v_new", v_new, (B, T, cache.Hkv, cache.D), dev) != kv:
        raise ValueError("k_new and v_new must have the same strides")
    for name, t in (("num_accepted", num_accepted), ("positions", positions), ("blocks", blocks)):
        _need(name, t, (B,), i32, dev)
    stride = 0
    if nodes is not None:
        stride = _rows("nodes", nodes, B, i32, dev)
        if nodes.shape[1] < T - 1:
            raise ValueError(f"nodes must hold at least {T - 1} nodes per row")
    _maybe("weights", weights, (B, T, cache.max_blocks), torch.float32, dev)
    _maybe("totals", totals, (B, cache.max_blocks), torch.float32, dev)
    if totals is None and (weights is not None or totals_out is not None):
        raise ValueError("weights and totals_out need totals")
    handle, scope = _scope(dev, stream)
    with scope:
        outs = []
        for name, t, like in (("positions_out", positions_out, positions), ("blocks_out", blocks_out, blocks),
                              ("totals_out", totals_out, totals)):
            if t is None and like is not None:
                t = torch.empty_like(like)
            elif t is not None:
                _need(name, t, tuple(like.shape), like.dtype, dev)
            outs.append(t)
        # an empty node list (T == 1) has no address, and is not read
        _check(load_library().spec_verify_commit(
            k_new.data_ptr(), v_new.data_ptr(), kv[0], kv[1], T, num_accepted.data_ptr(), _p(nodes) or None, stride,
            cache._ref, positions.data_ptr(), blocks.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(), _p(weights),
            _p(totals), _p(outs[2]), handle))
    return tuple(outs) if totals is not None else tuple(outs[:2])


def cache_evict(block_table, totals, blocks, budget, *, keep_first=0, keep_last=0, table_out=None, totals_out=None,
                blocks_out=None, evicted=None, stream=None):
    """spec_verify_evict: where a row has more than ``budget`` blocks, those of
    least totals leave it (see the header).

    block_table [B, max_blocks] int32 (a KVCache's, which table_out may be
    too), totals [B, max_blocks] fp32, blocks [B] int32.

    Returns (table, totals, blocks, evicted): new tensors, or the given outs;
    table_out, totals_out and blocks_out may be the inputs themselves.
    """
    dev = _gpu(block_table, "block_table")
    if block_table.dim() != 2 or 0 in block_table.shape:
        raise ValueError("block_table must be [B, max_blocks]")
    B, most = block_table.shape
    _need("block_table", block_table, (B, most), torch.int32, dev)
    _need("totals", totals, (B, most), torch.float32, dev)
    _need("blocks", blocks, (B,), torch.int32, dev)
    budget, keep_first, keep_last = (_count(n, most) for n in (budget, keep_first, keep_last))
    handle, scope = _scope(dev, stream)
    with scope:
        outs = []
        for name, t, like in (("table_out", table_out, block_table), ("totals_out", totals_out, totals),
                              ("blocks_out", blocks_out, blocks), ("evicted", evicted, blocks)):
            if t is None:
                t = torch.empty_like(like)
            else:
                _need(name, t, tuple(like.shape), like.dtype, dev)
            outs.append(t)
        _check(load_library().spec_verify_evict(
            totals.data_ptr(), block_table.data_ptr(), blocks.data_ptr(), B, most, budget, keep_first, keep_last,
            outs[1].data_ptr(), outs[0].data_ptr(), outs[2].data_ptr(), outs[3].data_ptr(), handle))
    return tuple(outs)


def _rotary(freqs, interleaved, axes, ids, B, T, D, dev):
    """sv_rotary, checked against tokens [B, T] of D channels."""
    _need("freqs", freqs, (None,), torch.float32, dev)
    dims = 2 * freqs.shape[0]
    if dims < 1 or dims > D:
        raise ValueError(f"freqs must hold 1 to {D // 2} frequencies")
    if ids is not None:
        _need("ids", ids, (None, B, T), torch.int32, dev)
        if ids.shape[0] < 1:
            raise ValueError("ids must have at least one axis")
    elif axes is not None:
        raise ValueError("axes needs ids")
    _maybe("axes", axes, (dims // 2,), torch.int32, dev)
    return SvRotary(freqs.data_ptr(), _p(ids), _p(axes), 0 if ids is None else ids.shape[0], dims, int(bool(interleaved)))


def _bf16_tokens(name, t):
    """Sizes of a [B, T, heads, D] bf16 tensor on a GPU."""
    _gpu(t, name)
    if t.dim() != 4 or 0 in t.shape:
        raise ValueError(f"{name} must be [B, T, heads, D]")
    return tuple(t.shape)


def rotate_tokens(q, k, freqs, positions=None, *, interleaved=False, axes=None, ids=None, parents=None,
                  query_lens=None, q_out=None, k_out=None, stream=None):
    """spec_verify_rotate: a step's queries and keys rotated by their positions
    (see sv_rotary in the header).

    q [B, T, H, D], k [B, T, Hkv, D] bf16, views with D-sized heads side by
    side; freqs [dims / 2] fp32; positions [B] int32 (a cache's), needed
    without ids; ids [axes, B, T] int32 with axes [dims / 2] int32: positions
    of several axes; parents [B, T] int32 for trees; query_lens [B] int32.

    Returns (q_out, k_out): new contiguous tensors (zeros behind query_lens),
    or the given ones, which may be q and k themselves.
    """
    B, T, H, D = shape = _bf16_tokens("q", q)
    dev = q.device
    if _bf16_tokens("k", k)[:2] != (B, T) or k.shape[3] != D:
        raise ValueError("k must be [B, T, Hkv, D] with q's B, T and D")
    kv = tuple(k.shape)
    strides = [_token_strides("q", q, shape, dev), _token_strides("k", k, kv, dev)]
    rot = _rotary(freqs, interleaved, axes, ids, B, T, D, dev)
    if positions is None and ids is None:
        raise ValueError("positions are needed without ids")
    _maybe("positions", positions, (B,), torch.int32, dev)
    _maybe("parents", parents, (B, T), torch.int32, dev)
    _maybe("query_lens", query_lens, (B,), torch.int32, dev)
    handle, scope = _scope(dev, stream)
    with scope:
        make = torch.empty if query_lens is None else torch.zeros
        outs = []
        for name, t, s in (("q_out", q_out, shape), ("k_out", k_out, kv)):
            if t is None:
                t = make(s, dtype=torch.bfloat16, device=dev)
            strides.append(_token_strides(name, t, s, dev))
            outs.append(t)
        _check(load_library().spec_verify_rotate(
            q.data_ptr(), *strides[0], k.data_ptr(), *strides[1], ctypes.byref(rot), _p(positions), _p(parents),
            _p(query_lens), B, T, H, kv[2], D, outs[0].data_ptr(), *strides[2], outs[1].data_ptr(), *strides[3],
            handle))
    return tuple(outs)


def cache_append(cache, k, v, positions, blocks, *, lens=None, freqs=None, interleaved=False, axes=None, ids=None,
                 k_out=None, positions_out=None, blocks_out=None, stream=None):
    """spec_verify_append: a prompt's keys and values enter the cache, the keys
    rotated on the way (see the header).

    k, v [B, T, Hkv, D] bf16 as cache_attention's k_new and v_new, T of any
    length; lens [B] int32: each row's tokens; freqs, interleaved, axes, ids as
    rotate_tokens' (no freqs: the keys are taken as they are); k_out [B, T,
    Hkv, D]: gets the rotated keys (k itself will do).

    Writes the cache's pages, scales and tails, and returns (positions,
    blocks): new tensors, or the given outs, which may be the inputs.
    """
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    dev, B, i32 = cache.device, cache.B, torch.int32
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or 0 in k.shape:
        raise ValueError("k must be [B, T, Hkv, D]")
    T = k.shape[1]
    shape = (B, T, cache.Hkv, cache.D)
    kv = _token_strides("k", k, shape, dev)
    if _token_strides("v", v, shape, dev) != kv:
        raise ValueError("k and v must have the same strides")
    out = (0, 0) if k_out is None else _token_strides("k_out", k_out, shape, dev)
    _need("positions", positions, (B,), i32, dev)
    _need("blocks", blocks, (B,), i32, dev)
    _maybe("lens", lens, (B,), i32, dev)
    rot = None
    if freqs is not None:
        rot = ctypes.byref(_rotary(freqs, interleaved, axes, ids, B, T, cache.D, dev))
    elif axes is not None or ids is not None:
        raise ValueError("axes and ids need freqs")
    handle, scope = _scope(dev, stream)
    with scope:
        outs = []
        for name, t in (("positions_out", positions_out), ("blocks_out", blocks_out)):
            if t is None:
                t = torch.empty_like(positions)
            else:
                _need(name, t, (B,), i32, dev)
            outs.append(t)
        _check(load_library().spec_verify_append(
            k.data_ptr(), v.data_ptr(), *kv, T, _p(lens), rot, cache._ref, positions.data_ptr(), blocks.data_ptr(),
            outs[0].data_ptr(), outs[1].data_ptr(), _p(k_out), *out, handle))
    return tuple(outs)


def _rules(logits, temperature, top_k, top_p, min_p):
    """Checks of a step's logits and its rows' rules; (B, P, V, dtype code, strides)."""
    dev = _gpu(logits, "logits")
    if logits.dim() != 3 or 0 in logits.shape:
        raise ValueError("logits must be [B, P, V]")
    B, P, V = logits.shape
    if max(B, P, V) > 2 ** 31 - 1:
        raise ValueError(f"logits are too large: {tuple(logits.shape)}")
    dt = _dtype_code(logits)
    _need("temperature", temperature, (B,), torch.float32, dev)
    _maybe("top_k", top_k, (B,), torch.int32, dev)
    _maybe("top_p", top_p, (B,), torch.float32, dev)
    _maybe("min_p", min_p, (B,), torch.float32, dev)
    return B, P, V, dt, _logit_strides("logits", logits)


_rule_sizes = {}  # workspace sizes by (kind, B, P, V, dtype, rules)


def _rule_workspace(kind, B, P, V, dt, cut, dev, handle, workspace):
    """The given workspace or one of the call's own, and its size; it need not be zero."""
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        return workspace, ctypes.c_size_t(workspace.numel() * workspace.element_size())
    key = (B, P, V, dt, cut)
    n = _rule_sizes.get((kind,) + key)
    if n is None:
        if len(_rule_sizes) >= 1024:
            _rule_sizes.clear()
        n = _rule_sizes[(kind,) + key] = _rule_bytes(kind, *key)
    if torch.cuda.is_current_stream_capturing():
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)  # the graph's own
    else:
        workspace = _cached_workspace(kind, key, n, dev, handle)
    return workspace, ctypes.c_size_t(n)


def _rule_bytes(kind, B, P, V, dt, cut):
    size, some = ctypes.c_size_t(0), ctypes.c_void_p(256 if cut else None)
    lib = load_library()
    if kind == "sample":
        _check(lib.spec_verify_sample(None, 0, 0, None, None, some, None, None, B, P, V, 1, dt, None, None, None,
                                      ctypes.byref(size), None))
    else:
        _check(lib.spec_verify_truncate(None, 0, 0, None, some, None, None, B, P, V, dt, None, 0, 0, None,
                                        ctypes.byref(size), None))
    return size.value


def sample_workspace_bytes(B, P, V, dtype=SV_BF16, *, cut=True):
    """Bytes of workspace that sample_tokens needs; cut: any of top_k, top_p and min_p is given."""
    return _rule_bytes("sample", B, P, V, dtype, cut)


def truncate_workspace_bytes(B, P, V, dtype=SV_BF16, *, cut=True):
    """Bytes of workspace that truncate_logits needs; cut: any of top_k, top_p and min_p is given."""
    return _rule_bytes("truncate", B, P, V, dtype, cut)


def sample_tokens(logits, uniforms, temperature, *, top_k=None, top_p=None, min_p=None, logprobs=None, tokens=None,
                  workspace=None, stream=None):
    """spec_verify_sample: tokens drawn from what top-k, top-p and min-p leave
    of the logits (see the header for the rules).

    logits [B, P, V] bf16 or fp32 with contiguous rows (a slice of a padded
    vocabulary will do); uniforms [B, P, n] fp32: n draws per position;
    temperature [B] fp32 (0: the largest logit); top_k [B] int32, top_p and
    min_p [B] fp32.  logprobs: True or a [B, P, n] fp32 tensor to get each
    token's log-probability among those left.

    Returns tokens [B, P, n] int32, or (tokens, logprobs).
    """
    B, P, V, dt, (row, pos) = _rules(logits, temperature, top_k, top_p, min_p)
    dev = logits.device
    _need("uniforms", uniforms, (B, P, None), torch.float32, dev)
    n = uniforms.shape[2]
    shape = (B, P, n)
    handle, scope = _scope(dev, stream)
    with scope:
        if tokens is None:
            tokens = torch.empty(shape, dtype=torch.int32, device=dev)
        else:
            _need("tokens", tokens, shape, torch.int32, dev)
        if logprobs is True:
            logprobs = torch.empty(shape, dtype=torch.float32, device=dev)
        elif logprobs is False:
            logprobs = None
        else:
            _maybe("logprobs", logprobs, shape, torch.float32, dev)
        cut = top_k is not None or top_p is not None or min_p is not None
        workspace, size = _rule_workspace("sample", B, P, V, dt, cut, dev, handle, workspace)
        _check(load_library().spec_verify_sample(
            logits.data_ptr(), row, pos, uniforms.data_ptr(), temperature.data_ptr(), _p(top_k), _p(top_p), _p(min_p),
            B, P, V, n, dt, tokens.data_ptr(), _p(logprobs), workspace.data_ptr(), ctypes.byref(size), handle))
    return tokens if logprobs is None else (tokens, logprobs)


def truncate_logits(logits, temperature, *, top_k=None, top_p=None, min_p=None, out=None, workspace=None, stream=None):
    """spec_verify_truncate: the logits that top-k, top-p and min-p leave out
    become -inf (see spec_verify_sample in the header for the rules).

    logits, temperature, top_k, top_p, min_p as sample_tokens'.  Returns
    ``out`` (a new contiguous [B, P, V] tensor if None; ``out=logits`` works in
    place).
    """
    B, P, V, dt, (row, pos) = _rules(logits, temperature, top_k, top_p, min_p)
    dev = logits.device
    handle, scope = _scope(dev, stream)
    with scope:
        if out is None:
            out = torch.empty((B, P, V), dtype=logits.dtype, device=dev)
        elif (not isinstance(out, torch.Tensor) or tuple(out.shape) != (B, P, V) or out.dtype != logits.dtype
              or out.device != dev):
            raise ValueError(f"out must be a {logits.dtype} tensor of shape {(B, P, V)} on {dev}")
        out_row, out_pos = _logit_strides("out", out)
        cut = top_k is not None or top_p is not None or min_p is not None
        workspace, size = _rule_workspace("truncate", B, P, V, dt, cut, dev, handle, workspace)
        _check(load_library().spec_verify_truncate(
            logits.data_ptr(), row, pos, temperature.data_ptr(), _p(top_k), _p(top_p), _p(min_p), B, P, V, dt,
            out.data_ptr(), out_row, out_pos, workspace.data_ptr(), ctypes.byref(size), handle))
    return out
