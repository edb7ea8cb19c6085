"""Layer operators around the routed block (Python binding of include/moe.h).

One decoder layer over t rows of a residual stream runs

    moe_add_rms_norm -> moe_qmv (q, k, v) -> moe_kv_append -> moe_kv_attention
    -> moe_qmv -> moe_add_rms_norm -> moe.moe_forward

with moe_kv_plan before a step's layers and moe_logprobs behind them.

Argument checks and marshalling only, as in :mod:`.moe`: every step runs in the
library's CUDA kernels, and there is no fallback.

* ``moe_add_rms_norm(x, gamma, residual)`` -> ``NormOut(sum, y, codes, scales)``
* ``moe_qmv(x, (codes, scales, biases))`` -> ``y``
* ``KvCache`` (the paged 8-bit cache), ``moe_kv_append(k, v, starts, cache)``,
  ``moe_kv_attention(q, starts, cache)`` -> ``out``
* ``moe_gated_rms_norm(x, gamma, residual, post_gamma, gate)`` -> ``NormOut``:
  the norms behind and before a block, with its gate and residual scale
* ``KvPages`` (a cache's free pages), ``moe_kv_plan(fresh, cache, pages, t)`` ->
  ``KvPlan(starts, seq, pos, slot)``
* ``LinearState`` (a pool of states), ``moe_linear_attention(q, k, v, log_decay,
  starts, state)`` -> ``out``
* ``moe_logprobs(logits, ids, top)`` -> ``Logprobs(logprob, entropy, lse,
  top_ids, top_logprobs)``

Every call takes ``stream`` (default: the current stream); what it allocates is
allocated for that stream.
"""

from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from .moe import (_BF16, _F16, MoeError, MoeGate, MoeKvCache, MoeKvPages, MoeQWeights, _check, _need,
                  _on_current_device, load_library, read_device_status)

__all__ = ["NormOut", "moe_add_rms_norm", "moe_gated_rms_norm", "moe_qmv", "KvCache", "moe_kv_append",
           "moe_kv_attention", "KvPages", "KvPlan", "moe_kv_plan", "LinearState", "moe_linear_attention", "Logprobs",
           "moe_logprobs"]

GROUP = 64  # weights per scale, and channels per scale of an 8-bit row


_BF = torch.bfloat16
_current_raw_stream = torch._C._cuda_getCurrentRawStream  # the handle alone: no Stream object is made


def _empty(shape, dtype, like, stream):
    """A tensor beside `like` that belongs to `stream`, so that its memory is
    not handed out again before that stream's work is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _raw(stream, dev: int) -> int:
    return _current_raw_stream(dev) if stream is None else stream.cuda_stream


def _need_rows(t, name: str, inner: tuple):
    """A bf16 tensor [rows, *inner] whose rows are dense and `stride(0)` apart (a multiple of 8)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in _BF16:
        raise TypeError(f"{name} must have dtype {' or '.join(str(d) for d in _BF16)}, got {t.dtype}")
    if tuple(t.shape[1:]) != inner:
        raise ValueError(f"{name} must have shape (rows, {', '.join(map(str, inner))}), got {tuple(t.shape)}")
    dense = 1
    for n, s in zip(reversed(inner), reversed(t.stride()[1:])):
        if s != dense and n > 1:
            raise ValueError(f"{name}: the values of a row must be contiguous, got strides {t.stride()}")
        dense *= n
    if t.stride(0) % 8 and t.shape[0] > 1:
        raise ValueError(f"{name}: rows must be a multiple of 8 elements apart, got {t.stride(0)}")
    return t


# Each call first asks in one expression whether its tensors are the ordinary
# ones (their own types and shapes, contiguous, on one device, no tensor given
# for the result); only when that is false do the checks that name what is wrong
# run, and pass the other valid forms (16-bit patterns, strided rows such as
# slices of a fused projection's, sum_out, out).  A decoded token's call is host
# time: the checks by name cost 10 us of it, the expression 1 us.

def _row_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else 0


class NormOut(NamedTuple):
    """Outputs of moe_add_rms_norm; what was not asked for is None."""

    sum: torch.Tensor | None
    y: torch.Tensor | None
    codes: torch.Tensor | None
    scales: torch.Tensor | None


def moe_add_rms_norm(x: torch.Tensor, gamma: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                     quantize: bool = False, want_y: bool | None = None, sum_out: torch.Tensor | None = None,
                     stream=None) -> NormOut:
    """a = x + residual; y = a / sqrt(mean(a^2) + eps) * gamma, per row.

    x, residual bf16 [t, h] (rows may be strided), gamma bf16 [h].  ``sum``
    (bf16 a, when a residual is given or ``sum_out`` names its tensor, which
    may be x or residual itself), ``y`` (bf16; by default unless ``quantize``)
    and, with ``quantize``, y in 8 bits: ``codes`` int8 [t, h] and ``scales``
    fp32 [t, h / 64].
    """
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be [t, h]")
    t, h = shape = x.shape
    dev = x.get_device()
    if not (dev >= 0 and dev == torch.cuda.current_device() == gamma.get_device()
            and x.dtype is _BF and x.is_contiguous() and gamma.dtype is _BF and gamma.shape == (h,) and gamma.is_contiguous()
            and (residual is None or (residual.dtype is _BF and residual.shape == shape and residual.is_contiguous()
                                      and residual.get_device() == dev))
            and sum_out is None and not (quantize and h % GROUP)):
        _need_rows(x, "x", (h,))
        _need(gamma, "gamma", _BF16, shape=(h,))
        if residual is not None:
            _need_rows(residual, "residual", (h,))
            if residual.shape[0] != t:
                raise ValueError(f"residual must have {t} rows, got {residual.shape[0]}")
        if sum_out is not None:
            _need(sum_out, "sum_out", _BF16, shape=(t, h))
        if quantize and h % GROUP:
            raise ValueError(f"h={h} must be a multiple of {GROUP} for 8-bit rows")
        _on_current_device(x=x, gamma=gamma, residual=residual, sum_out=sum_out)
    if want_y is None:
        want_y = not quantize
    y = codes = scales = None
    if sum_out is None and residual is not None:
        sum_out = _empty(shape, _BF, x, stream)
    if want_y:
        y = _empty(shape, _BF, x, stream)
    if quantize:
        codes = _empty(shape, torch.int8, x, stream)
        scales = _empty((t, h // GROUP), torch.float32, x, stream)
    status = lib.moe_add_rms_norm(
        x.data_ptr(), x.stride(0) if t > 1 else 0, None if residual is None else residual.data_ptr(),
        0 if residual is None or t == 1 else residual.stride(0), gamma.data_ptr(), eps, t, h,
        None if sum_out is None else sum_out.data_ptr(), None if y is None else y.data_ptr(),
        None if codes is None else codes.data_ptr(), None if scales is None else scales.data_ptr(), _raw(stream, dev))
    if status:
        _check(status)
    return NormOut(sum_out, y, codes, scales)


def _gate_of(gate, sigmoid: bool, t: int, h: int):
    """The gate as the C ABI takes it: values for each channel ([h] or [t, h]), or one a row ([t, 1])."""
    if not isinstance(gate, torch.Tensor):
        raise TypeError(f"gate must be a torch.Tensor, got {type(gate).__name__}")
    if gate.dtype not in _BF16:
        raise TypeError(f"gate must have dtype {' or '.join(str(d) for d in _BF16)}, got {gate.dtype}")
    if gate.shape == (h,):
        _need(gate, "gate", _BF16)
        return MoeGate(gate.data_ptr(), 0, 1, sigmoid)
    if gate.shape == (t, h) and h > 1:
        _need_rows(gate, "gate", (h,))
        return MoeGate(gate.data_ptr(), _row_stride(gate), 1, sigmoid)
    if gate.shape == (t, 1):
        return MoeGate(gate.data_ptr(), _row_stride(gate), 0, sigmoid)
    raise ValueError(f"gate must have shape ({h},), ({t}, {h}) or ({t}, 1), got {tuple(gate.shape)}")


def moe_gated_rms_norm(x: torch.Tensor, gamma: torch.Tensor, residual: torch.Tensor | None = None,
                       post_gamma: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                       gate_sigmoid: bool = False, residual_scale: float = 1.0, eps: float = 1e-6,
                       quantize: bool = False, want_y: bool | None = None, sum_out: torch.Tensor | None = None,
                       stream=None) -> NormOut:
    """b = norm(x) * post_gamma; a = residual_scale * residual + gate * b; y = norm(a) * gamma, per row.

    x bf16 [t, h] is a block's output (rows may be strided); without
    ``post_gamma`` (bf16 [h]) b = x.  gate bf16: [h] (one value a channel),
    [t, 1] (one a row) or [t, h]; with ``gate_sigmoid`` 1 / (1 + exp(-gate))
    takes its place.  residual, gamma, ``sum`` (a), ``y``, ``codes`` and
    ``scales`` as in moe_add_rms_norm; ``sum`` is given unless there is neither a
    residual nor a ``sum_out``.
    """
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be [t, h]")
    t, h = shape = x.shape
    dev = x.get_device()
    if not (dev >= 0 and dev == torch.cuda.current_device() == gamma.get_device()
            and x.dtype is _BF and x.is_contiguous() and gamma.dtype is _BF and gamma.shape == (h,) and gamma.is_contiguous()
            and (residual is None or (residual.dtype is _BF and residual.shape == shape and residual.is_contiguous()
                                      and residual.get_device() == dev))
            and (post_gamma is None or (post_gamma.dtype is _BF and post_gamma.shape == (h,) and post_gamma.is_contiguous()
                                        and post_gamma.get_device() == dev))
            and (gate is None or gate.get_device() == dev)
            and sum_out is None and not (quantize and h % GROUP)):
        _need_rows(x, "x", (h,))
        _need(gamma, "gamma", _BF16, shape=(h,))
        if post_gamma is not None:
            _need(post_gamma, "post_gamma", _BF16, shape=(h,))
        if residual is not None:
            _need_rows(residual, "residual", (h,))
            if residual.shape[0] != t:
                raise ValueError(f"residual must have {t} rows, got {residual.shape[0]}")
        if sum_out is not None:
            _need(sum_out, "sum_out", _BF16, shape=(t, h))
        if gate is not None:
            _gate_of(gate, gate_sigmoid, t, h)
        if quantize and h % GROUP:
            raise ValueError(f"h={h} must be a multiple of {GROUP} for 8-bit rows")
        _on_current_device(x=x, gamma=gamma, residual=residual, post_gamma=post_gamma, gate=gate, sum_out=sum_out)
    g = None if gate is None else ctypes.byref(_gate_of(gate, gate_sigmoid, t, h))
    if want_y is None:
        want_y = not quantize
    y = codes = scales = None
    if sum_out is None and residual is not None:
        sum_out = _empty(shape, _BF, x, stream)
    if want_y:
        y = _empty(shape, _BF, x, stream)
    if quantize:
        codes = _empty(shape, torch.int8, x, stream)
        scales = _empty((t, h // GROUP), torch.float32, x, stream)
    status = lib.moe_gated_rms_norm(
        x.data_ptr(), x.stride(0) if t > 1 else 0, None if post_gamma is None else post_gamma.data_ptr(), g,
        None if residual is None else residual.data_ptr(), 0 if residual is None or t == 1 else residual.stride(0),
        residual_scale, gamma.data_ptr(), eps, t, h, None if sum_out is None else sum_out.data_ptr(),
        None if y is None else y.data_ptr(), None if codes is None else codes.data_ptr(),
        None if scales is None else scales.data_ptr(), _raw(stream, dev))
    if status:
        _check(status)
    return NormOut(sum_out, y, codes, scales)


def moe_qmv(x, weights: tuple, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
            stream=None) -> torch.Tensor:
    """y = x W^T with 4-bit weights W = q * scale + bias in groups of 64.

    x: bf16 [t, k] (rows may be strided), or 8-bit rows (codes int8 [t, k],
    scales fp32 [t, k / 64]) as moe_add_rms_norm gives them.  weights: (codes
    uint8 [n, k / 2], scales fp16 [n, k / 64], biases fp16 [n, k / 64]).
    out: bf16 or fp32 [t, n] (``out_dtype`` when it is made here).
    """
    lib = load_library()
    codes, scales, biases = weights
    if codes.dim() != 2:
        raise ValueError("weight codes must be [n, k / 2]")
    n, kh = codes.shape
    k = 2 * kh
    dev = codes.get_device()
    rows = xc = xs = None
    if isinstance(x, torch.Tensor):
        rows = x
        t = x.shape[0]
        plain = x.dtype is _BF and x.shape == (t, k) and x.is_contiguous() and x.get_device() == dev
    else:
        xc, xs = x
        t = xc.shape[0]
        plain = (xc.dtype is torch.int8 and xc.shape == (t, k) and xc.is_contiguous() and xc.get_device() == dev
                 and xs.dtype is torch.float32 and xs.shape == (t, k // GROUP) and xs.is_contiguous()
                 and xs.get_device() == dev)
    groups = (n, k // GROUP)
    if not (plain and dev >= 0 and dev == torch.cuda.current_device() == scales.get_device() == biases.get_device()
            and codes.dtype is torch.uint8 and codes.is_contiguous()
            and scales.dtype is torch.float16 and scales.shape == groups and scales.is_contiguous()
            and biases.dtype is torch.float16 and biases.shape == groups and biases.is_contiguous()
            and out is None and (out_dtype is _BF or out_dtype is torch.float32)):
        _need(codes, "weight codes", (torch.uint8,))
        _need(scales, "weight scales", _F16, shape=groups)
        _need(biases, "weight biases", _F16, shape=groups)
        if rows is not None:
            _need_rows(rows, "x", (k,))
        else:
            _need(xc, "x codes", (torch.int8,), shape=(t, k))
            _need(xs, "x scales", (torch.float32,), shape=(t, k // GROUP))
        if out is not None:
            _need(out, "out", (torch.bfloat16, torch.float32), shape=(t, n))
        elif out_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
        _on_current_device(x=rows, x_codes=xc, x_scales=xs, codes=codes, scales=scales, biases=biases, out=out)
    if out is None:
        out = _empty((t, n), out_dtype, codes, stream)
    w = MoeQWeights(codes.data_ptr(), scales.data_ptr(), biases.data_ptr())
    status = lib.moe_qmv(
        None if rows is None else rows.data_ptr(), 0 if rows is None else _row_stride(rows),
        None if xc is None else xc.data_ptr(), None if xs is None else xs.data_ptr(), ctypes.byref(w), t, n, k,
        out.data_ptr(), out.dtype is torch.float32, _raw(stream, dev))
    if status:
        _check(status)
    return out


class KvCache:
    """A paged key/value cache in 8 bits (moe_kv_cache), with its workspace.

    codes int8 [2, n_pages, hkv, block, d] and scales fp32 [2, n_pages, hkv]
    hold keys, then values; tail bf16 [n_seq, 2, hkv, 2 * block, d] the last
    tokens as given; table int32 [n_seq, max_blocks] each sequence's pages;
    lens int32 [n_seq] its tokens.  The caller assigns pages in ``table`` and
    sets ``lens`` (the new tokens included) before moe_kv_append, in place
    (``cache.lens.copy_(...)``, ``cache.table[s, b] = page``), or has
    moe_kv_plan do both; they are read on the device.  The tensors are kept, not
    copied, and cannot be replaced by others: calls that use one cache are
    ordered on one stream.

    held int32 [n_seq, 2], made here, says up to which token each half of a
    sequence's tail is filled (0: not known); moe_kv_append keeps it, and
    reports a sequence that was cut back to where its tail does not reach.
    Copy it along with a sequence's tail, or set it to 0 where a tail is
    filled by hand.
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, tail: torch.Tensor, table: torch.Tensor,
                 lens: torch.Tensor):
        if codes.dim() != 5 or codes.shape[0] != 2:
            raise ValueError("codes must be [2, n_pages, hkv, block, d]")
        _, n_pages, hkv, block, d = codes.shape
        if table.dim() != 2:
            raise ValueError("table must be [n_seq, max_blocks]")
        n_seq, max_blocks = table.shape
        _need(codes, "codes", (torch.int8,))
        _need(scales, "scales", (torch.float32,), shape=(2, n_pages, hkv))
        _need(tail, "tail", _BF16, shape=(n_seq, 2, hkv, 2 * block, d))
        _need(table, "table", (torch.int32,))
        _need(lens, "lens", (torch.int32,), shape=(n_seq,))
        _on_current_device(codes=codes, scales=scales, tail=tail, table=table, lens=lens)
        n = load_library().moe_kv_workspace_bytes(d)
        if n == 0:
            raise MoeError(-2, f"d={d} must be 64 or 128")
        self._codes, self._scales, self._tail, self._table, self._lens = codes, scales, tail, table, lens
        self.n_seq, self.hkv, self.block, self.d = n_seq, hkv, block, d
        self._workspace = torch.zeros(n, dtype=torch.uint8, device=codes.device)
        self._filled = torch.zeros(n_seq, 2, dtype=torch.int32, device=codes.device)
        self._dev = codes.get_device()
        self._starts, self._kv, self._softmax_scale = (n_seq + 1,), (hkv, d), 1 / math.sqrt(d)
        self._ws = self.ws.data_ptr(), n
        self._held = self.held.data_ptr()
        self._c = MoeKvCache(codes.data_ptr(), scales.data_ptr(), tail.data_ptr(), table.data_ptr(), lens.data_ptr(),
                             n_seq, n_pages, max_blocks, block, hkv, d)
        self._ref = ctypes.byref(self._c)

    # Kernels read these by address, so that a tensor put in the place of one
    # would not be seen, and the one it replaced could be handed out again
    # while kernels still read it: assigning raises AttributeError.
    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    tail = property(lambda self: self._tail)
    table = property(lambda self: self._table)
    lens = property(lambda self: self._lens)
    held = property(lambda self: self._filled)
    ws = property(lambda self: self._workspace)

    @classmethod
    def new(cls, n_seq: int, n_pages: int, max_blocks: int, hkv: int, d: int, block: int = 64, device="cuda"):
        """An empty cache: all lengths and pages 0."""
        e = lambda *shape, dtype: torch.zeros(shape, dtype=dtype, device=device)  # noqa: E731
        return cls(e(2, n_pages, hkv, block, d, dtype=torch.int8), e(2, n_pages, hkv, dtype=torch.float32),
                   e(n_seq, 2, hkv, 2 * block, d, dtype=torch.bfloat16), e(n_seq, max_blocks, dtype=torch.int32),
                   e(n_seq, dtype=torch.int32))

    def read_device_status(self, stream=None) -> int:
        """Synchronise and return the device-side status (0 = clean); clears it."""
        return read_device_status(self.ws, stream)


def _need_starts(starts, cache: KvCache):
    if not isinstance(cache, KvCache):
        raise TypeError(f"cache must be a KvCache, got {type(cache).__name__}")
    return _need(starts, "starts", (torch.int32,), shape=(cache.n_seq + 1,))


def moe_kv_append(k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor, cache: KvCache, stream=None) -> None:
    """Write the new rows' keys and values (bf16 [t, hkv, d], rows may be
    strided) into the cache; sequence s owns rows starts[s] .. starts[s+1]-1
    (int32 [n_seq + 1], on the device), its last tokens."""
    lib = load_library()
    t = k.shape[0]
    dev = k.get_device()
    if not (type(cache) is KvCache and dev >= 0 and dev == torch.cuda.current_device() == cache._dev
            and v.get_device() == dev == starts.get_device()
            and k.dtype is _BF and k.shape[1:] == cache._kv and k.is_contiguous()
            and v.dtype is _BF and v.shape == k.shape and v.is_contiguous()
            and starts.dtype is torch.int32 and starts.shape == cache._starts and starts.is_contiguous()):
        _need_starts(starts, cache)
        _need_rows(k, "k", cache._kv)
        _need_rows(v, "v", cache._kv)
        if v.shape[0] != t:
            raise ValueError(f"v must have {t} rows, got {v.shape[0]}")
        _on_current_device(k=k, v=v, starts=starts, codes=cache.codes)
    status = lib.moe_kv_append_held(k.data_ptr(), _row_stride(k), v.data_ptr(), _row_stride(v), starts.data_ptr(), t,
                                    cache._ref, cache._held, *cache._ws, _raw(stream, dev))
    if status:
        _check(status)


def moe_kv_attention(q: torch.Tensor, starts: torch.Tensor, cache: KvCache, scale: float | None = None,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of the new rows q (bf16 [t, hq, d], rows may be
    strided) over the cache; ``scale`` defaults to 1 / sqrt(d).  Returns bf16
    [t, hq, d]."""
    lib = load_library()
    if q.dim() != 3:
        raise ValueError("q must be [t, hq, d]")
    t, hq, d = shape = q.shape
    dev = q.get_device()
    if not (type(cache) is KvCache and dev >= 0 and dev == torch.cuda.current_device() == cache._dev
            and starts.get_device() == dev and q.dtype is _BF and d == cache.d and q.is_contiguous() and out is None
            and starts.dtype is torch.int32 and starts.shape == cache._starts and starts.is_contiguous()):
        _need_starts(starts, cache)
        _need_rows(q, "q", (hq, cache.d))
        if out is not None:
            _need(out, "out", _BF16, shape=(t, hq, d))
        _on_current_device(q=q, starts=starts, out=out, codes=cache.codes)
    if out is None:
        out = _empty(shape, _BF, q, stream)
    status = lib.moe_kv_attention(q.data_ptr(), _row_stride(q), starts.data_ptr(), t, hq,
                                  cache._softmax_scale if scale is None else scale, cache._ref, out.data_ptr(), *cache._ws,
                                  _raw(stream, dev))
    if status:
        _check(status)
    return out


class KvPages:
    """The pages of a KvCache that are free (moe_kv_pages), with the plan's workspace.

    free int32 [n_pages], whose first ``count`` entries are the free pages,
    taken from the end; account int32 [n_seq + 1]: the blocks that each
    sequence holds pages for in the cache's table, then ``count``.  Both are
    kept, not copied, read and written on the device; a copy of both brings the
    pages back to where they stood.  Without them every page is free, the
    lowest one taken first.
    """

    def __init__(self, cache: KvCache, free: torch.Tensor | None = None, account: torch.Tensor | None = None):
        if not isinstance(cache, KvCache):
            raise TypeError(f"cache must be a KvCache, got {type(cache).__name__}")
        n_seq, n_pages = cache.n_seq, cache.codes.shape[1]
        if (free is None) != (account is None):
            raise ValueError("free and account come together")
        if free is None:
            free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=cache.codes.device)
            account = torch.zeros(n_seq + 1, dtype=torch.int32, device=cache.codes.device)
            account[n_seq] = n_pages
        _need(free, "free", (torch.int32,), shape=(n_pages,))
        _need(account, "account", (torch.int32,), shape=(n_seq + 1,))
        _on_current_device(free=free, account=account, codes=cache.codes)
        self._cache, self._free, self._account = cache, free, account
        n = load_library().moe_kv_plan_workspace_bytes(n_seq)
        if n == 0:
            raise MoeError(-2, f"n_seq={n_seq} outside [1, 65536]")
        self._workspace = torch.zeros(n, dtype=torch.uint8, device=free.device)
        self._ws = self._workspace.data_ptr(), n
        self._c = MoeKvPages(free.data_ptr(), account.data_ptr(), account.data_ptr() + 4 * n_seq)
        self._ref = ctypes.byref(self._c)
        c = cache._c
        self._table, self._sizes = cache.table.data_ptr(), (c.n_seq, c.n_pages, c.max_blocks, c.block)

    # read by address, as the cache's tensors
    cache = property(lambda self: self._cache)
    free = property(lambda self: self._free)
    account = property(lambda self: self._account)
    held = property(lambda self: self._account[:-1])
    count = property(lambda self: self._account[-1:])
    ws = property(lambda self: self._workspace)

    def read_device_status(self, stream=None) -> int:
        """Synchronise and return the device-side status (0 = clean); clears it."""
        return read_device_status(self.ws, stream)


class KvPlan(NamedTuple):
    """Outputs of moe_kv_plan: starts int32 [n_seq + 1]; of each row its sequence and position (int32 [t]) and its
    slot page * block + place (int64 [t]), -1 behind the last sequence."""

    starts: torch.Tensor
    seq: torch.Tensor
    pos: torch.Tensor
    slot: torch.Tensor


def moe_kv_plan(fresh: torch.Tensor, cache: KvCache, pages: KvPages, t: int, lens: torch.Tensor | None = None,
                stream=None) -> KvPlan:
    """Starts, lengths, page table and row maps of a batch of t rows.

    fresh int32 [n_seq]: the new tokens of each sequence (0: idle; below 0: it
    ends and its pages become free).  ``cache.lens`` becomes the lengths with
    the new tokens, from those before the call: its own, or ``lens`` (int32
    [n_seq]), to which sequences are cut back.  ``cache.table`` gets pages for
    the blocks that have none.  A batch that does not fit changes nothing, and
    is reported by ``pages.read_device_status()``.
    """
    lib = load_library()
    if not isinstance(pages, KvPages):
        raise TypeError(f"pages must be a KvPages, got {type(pages).__name__}")
    if pages._cache is not cache:
        raise ValueError("pages belong to another cache")
    before = cache._lens if lens is None else lens
    dev = fresh.get_device()
    shape = (cache.n_seq,)
    if not (dev >= 0 and dev == torch.cuda.current_device() == cache._dev == before.get_device()
            and fresh.dtype is torch.int32 and fresh.shape == shape and fresh.is_contiguous()
            and before.dtype is torch.int32 and before.shape == shape and before.is_contiguous()):
        _need(fresh, "fresh", (torch.int32,), shape=shape)
        _need(before, "lens", (torch.int32,), shape=shape)
        _on_current_device(fresh=fresh, lens=before, codes=cache.codes)
    if not 1 <= t <= 65536:  # before memory is asked for
        raise MoeError(-2, f"t={t} outside [1, 65536]")
    n_seq, n_pages, max_blocks, block = pages._sizes
    starts = _empty((n_seq + 1,), torch.int32, fresh, stream)
    seq, pos = _empty((t,), torch.int32, fresh, stream), _empty((t,), torch.int32, fresh, stream)
    slot = _empty((t,), torch.int64, fresh, stream)
    status = lib.moe_kv_plan(fresh.data_ptr(), before.data_ptr(), cache._c.lens, pages._table, pages._ref, n_seq, n_pages,
                             max_blocks, block, t, starts.data_ptr(), seq.data_ptr(), pos.data_ptr(), slot.data_ptr(),
                             *pages._ws, _raw(stream, dev))
    if status:
        _check(status)
    return KvPlan(starts, seq, pos, slot)


class LinearState:
    """A pool of states of linear attention, fp32 [n_slots, heads, d, d] (key channel, value channel), with its
    workspace.  The tensor is kept, not copied: calls that use one pool are ordered on one stream."""

    def __init__(self, states: torch.Tensor):
        if states.dim() != 4 or states.shape[2] != states.shape[3]:
            raise ValueError("states must be [n_slots, heads, d, d]")
        _need(states, "states", (torch.float32,))
        _on_current_device(states=states)
        self.n_slots, self.heads, self.d, _ = states.shape
        n = load_library().moe_linear_workspace_bytes(self.d)
        if n == 0:
            raise MoeError(-2, f"d={self.d} must be 64 or 128")
        self._states, self._dev = states, states.get_device()
        self._workspace = torch.zeros(n, dtype=torch.uint8, device=states.device)
        self._ws = self._workspace.data_ptr(), n
        self._scale = 1 / math.sqrt(self.d)

    # read by address, as a cache's tensors
    states = property(lambda self: self._states)
    ws = property(lambda self: self._workspace)

    @classmethod
    def new(cls, n_slots: int, heads: int, d: int, device="cuda"):
        """A pool of zero states."""
        return cls(torch.zeros(n_slots, heads, d, d, device=device))

    def read_device_status(self, stream=None) -> int:
        """Synchronise and return the device-side status (0 = clean); clears it."""
        return read_device_status(self.ws, stream)


def moe_linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, starts: torch.Tensor,
                         state: LinearState, slots: torch.Tensor | None = None, slots_out: torch.Tensor | None = None,
                         scale: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """S_r = exp(log_decay_r) S_(r-1) + k_r v_r^T, out_r = scale * S_r^T q_r over packed sequences.

    q, k bf16 [t, hk, d], v bf16 [t, hv, d] (rows may be strided), log_decay
    fp32 [hv] or [t, hv] (rows may be strided), starts int32 [n_seq + 1].
    Sequence s begins from the state in slot ``slots[s]`` (int32 [n_seq]; -1:
    zero; default: slot s) and leaves its last one in ``slots_out[s]`` (-1:
    nowhere; default: the same slots).  ``scale`` defaults to 1 / sqrt(d).
    Long prompts beside many sequences of a row or two cost far less in a call
    of their own: t / n_seq chooses one kernel for all (moe.h).
    Returns bf16 [t, hv, d] (``out``, which does not overlap the inputs).
    """
    lib = load_library()
    if not isinstance(state, LinearState):
        raise TypeError(f"state must be a LinearState, got {type(state).__name__}")
    if q.dim() != 3 or v.dim() != 3 or starts.dim() != 1 or log_decay.dim() not in (1, 2):
        raise ValueError("q, k and v must be [t, heads, d], log_decay [heads] or [t, heads], starts [n_seq + 1]")
    t, hk, d = q.shape
    hv, n_seq = v.shape[1], starts.shape[0] - 1
    shape = (t, hv, d)
    dev = q.get_device()
    decays = log_decay.shape
    if not (dev >= 0 and dev == torch.cuda.current_device() == state._dev and d == state.d and hv == state.heads
            and k.get_device() == dev == v.get_device() and starts.get_device() == dev == log_decay.get_device()
            and q.dtype is _BF and q.is_contiguous() and k.dtype is _BF and k.shape == q.shape and k.is_contiguous()
            and v.dtype is _BF and v.shape == shape and v.is_contiguous()
            and log_decay.dtype is torch.float32 and log_decay.is_contiguous() and (decays == (hv,) or decays == (t, hv))
            and starts.dtype is torch.int32 and starts.is_contiguous() and n_seq > 0 and out is None
            and (slots is None or (slots.dtype is torch.int32 and slots.shape == (n_seq,) and slots.is_contiguous()
                                   and slots.get_device() == dev))
            and (slots_out is None or (slots_out.dtype is torch.int32 and slots_out.shape == (n_seq,)
                                       and slots_out.is_contiguous() and slots_out.get_device() == dev))):
        if n_seq < 1:
            raise ValueError("starts must hold at least one sequence")
        _need_rows(q, "q", (hk, state.d))
        _need_rows(k, "k", (hk, d))
        _need_rows(v, "v", (state.heads, d))
        for name, r in (("k", k), ("v", v)):
            if r.shape[0] != t:
                raise ValueError(f"{name} must have {t} rows, got {r.shape[0]}")
        if log_decay.dtype is not torch.float32:
            raise TypeError(f"log_decay must have dtype torch.float32, got {log_decay.dtype}")
        if decays != (hv,) and decays != (t, hv):
            raise ValueError(f"log_decay must have shape ({hv},) or ({t}, {hv}), got {tuple(decays)}")
        if log_decay.stride(-1) != 1 and hv > 1:
            raise ValueError(f"log_decay: the values of a row must be contiguous, got strides {log_decay.stride()}")
        _need(starts, "starts", (torch.int32,))
        for name, r in (("slots", slots), ("slots_out", slots_out)):
            if r is not None:
                _need(r, name, (torch.int32,), shape=(n_seq,))
        if out is not None:
            _need(out, "out", _BF16, shape=shape)
        _on_current_device(q=q, k=k, v=v, log_decay=log_decay, starts=starts, slots=slots, slots_out=slots_out, out=out,
                           states=state.states)
    if out is None:
        out = _empty(shape, _BF, q, stream)
    status = lib.moe_linear_attention(
        q.data_ptr(), _row_stride(q), k.data_ptr(), _row_stride(k), v.data_ptr(), _row_stride(v), log_decay.data_ptr(),
        _row_stride(log_decay) if len(decays) == 2 else 0, starts.data_ptr(), t, n_seq, hk, hv, d,
        state._scale if scale is None else scale, state._states.data_ptr(), state.n_slots,
        None if slots is None else slots.data_ptr(), None if slots_out is None else slots_out.data_ptr(), out.data_ptr(),
        *state._ws, _raw(stream, dev))
    if status:
        _check(status)
    return out


class Logprobs(NamedTuple):
    """Outputs of moe_logprobs, fp32 but for the ids (int32); what was not asked for is None."""

    logprob: torch.Tensor | None
    entropy: torch.Tensor
    lse: torch.Tensor
    top_ids: torch.Tensor | None
    top_logprobs: torch.Tensor | None


def moe_logprobs(logits: torch.Tensor, ids: torch.Tensor | None = None, top: int = 0, stream=None) -> Logprobs:
    """Log probabilities of given tokens under rows of logits, their entropy and top alternatives.

    logits fp32 or bf16 [t, n] (rows may be strided); ids int32 or int64 [t] or
    [t, m], m <= 256: ``logprob`` fp32 of ids' shape.  ``entropy`` and ``lse``
    (log of the sum of exponentials) fp32 [t]; ``top_ids`` int32 and
    ``top_logprobs`` fp32 [t, top], top <= 32, the largest logits in order, the
    lower index first among equals.
    """
    lib = load_library()
    if logits.dim() != 2:
        raise ValueError("logits must be [t, n]")
    t, n = logits.shape
    dev = logits.get_device()
    f32 = logits.dtype is torch.float32
    if not (dev >= 0 and dev == torch.cuda.current_device() and (f32 or logits.dtype is _BF) and logits.is_contiguous()
            and (ids is None or (ids.get_device() == dev and ids.shape == (t,) and ids.is_contiguous()
                                 and (ids.dtype is torch.int64 or ids.dtype is torch.int32)))):
        if logits.dtype not in (torch.float32,) + _BF16:
            raise TypeError(f"logits must have dtype torch.float32 or torch.bfloat16, got {logits.dtype}")
        if logits.stride(1) != 1 and n > 1:
            raise ValueError(f"logits: the values of a row must be contiguous, got strides {logits.stride()}")
        if ids is not None:
            if ids.dim() not in (1, 2) or ids.shape[0] != t:
                raise ValueError(f"ids must have shape ({t},) or ({t}, m), got {tuple(ids.shape)}")
            _need(ids, "ids", (torch.int64, torch.int32))
        _on_current_device(logits=logits, ids=ids)
    if not 0 <= top <= 32:
        raise MoeError(-2, f"top={top} outside [0, 32]")
    logprob = top_ids = top_logprobs = None
    m = 0 if ids is None else 1 if ids.dim() == 1 else ids.shape[1]
    # tensors of their own: a view of a new tensor costs more than another tensor
    entropy, lse = _empty((t,), torch.float32, logits, stream), _empty((t,), torch.float32, logits, stream)
    if ids is not None:
        logprob = _empty(ids.shape, torch.float32, logits, stream)
    if top:
        top_ids = _empty((t, top), torch.int32, logits, stream)
        top_logprobs = _empty((t, top), torch.float32, logits, stream)
    status = lib.moe_logprobs(
        logits.data_ptr(), _row_stride(logits), f32, t, n, ids.data_ptr() if m else None,
        ids is not None and ids.dtype is torch.int64, m, top, logprob.data_ptr() if m else None, entropy.data_ptr(),
        lse.data_ptr(), top_ids.data_ptr() if top else None, top_logprobs.data_ptr() if top else None, _raw(stream, dev))
    if status:
        _check(status)
    return Logprobs(logprob, entropy, lse, top_ids, top_logprobs)
