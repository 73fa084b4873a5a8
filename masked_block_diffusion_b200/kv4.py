"""Rotary positions and the paged 4-bit KV cache on torch tensors.

``Rope`` is a rotation plan, ``rope`` rotates a tensor, ``KVCache4`` holds one layer's pages
and appends to them, reads them back and attends to them. Each call checks its tensors,
queues one or two kernels of libdllm.so on the current stream of the tensors' device
(whichever device is current) and returns; it can be captured in a CUDA graph. The C ABI
behind it (include/dllm.h) says what each call computes and how it treats padding, bad page
ids and bad lengths.

Tensors are those of the call's stream: as with any torch operation, the caller orders other
streams' work on them. A write to a tensor that the caller gave counts as one in place: a
backward pass that had saved the old values raises.
"""

from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import binding

_TYPES = {torch.float32: binding.DLLM_F32, torch.bfloat16: binding.DLLM_BF16}
_LAYOUTS = {"half": binding.DLLM_ROPE_HALF, "interleaved": binding.DLLM_ROPE_INTERLEAVED}
_SCALINGS = {"none": binding.DLLM_ROPE_NONE, "linear": binding.DLLM_ROPE_LINEAR, "ntk": binding.DLLM_ROPE_NTK,
             "yarn": binding.DLLM_ROPE_YARN}


class Rope:
    """A rotation plan: which dims of a head turn, and how fast (dllm_rope_init).

    layout: "half" pairs dims (i, i + rotary_dim / 2), "interleaved" pairs (2 i, 2 i + 1).
    scaling for contexts beyond the trained one: "none", "linear", "ntk" or "yarn" with
    `factor`; original_ctx, beta_fast and beta_slow are for "yarn".
    """

    def __init__(self, rotary_dim: int, layout: str = "half", theta: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, original_ctx: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout {layout!r}: one of {sorted(_LAYOUTS)}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling {scaling!r}: one of {sorted(_SCALINGS)}")
        self.c = binding.dllm_rope_init(int(rotary_dim), _LAYOUTS[layout], float(theta), _SCALINGS[scaling],
                                        float(factor), float(original_ctx), float(beta_fast), float(beta_slow))
        self.rotary_dim, self.layout, self.magnitude = int(rotary_dim), layout, self.c.magnitude


try:   # the current device and its current stream as integers, without the objects around them
    from torch._C import _cuda_getCurrentRawStream as _stream_of
    from torch._C import _cuda_getDevice as _current_device
except ImportError:   # pragma: no cover
    _current_device = torch.cuda.current_device

    def _stream_of(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _bad(name: str, why: str):
    raise ValueError(f"{name}: {why}")


# The checks below run on every call, so each takes what it looks at from the tensor once.

def _heads(name: str, t: torch.Tensor, dev: int, T: int, H: int, d: int, types) -> tuple:
    """A [T][H][d] tensor on device `dev` whose last dimension is contiguous: its (token stride, head stride), 0
    where a dimension has one element and no stride that matters."""
    if t.get_device() != dev:
        _bad(name, f"on {t.device}, expected cuda:{dev}")
    if t.dtype not in types:
        _bad(name, f"{t.dtype}, expected one of {[str(x) for x in types]}")
    if t.shape != (T, H, d):
        _bad(name, f"shape {tuple(t.shape)}, expected {(T, H, d)}")
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        _bad(name, "the last dimension has to be contiguous")
    return st if T > 1 else 0, sh if H > 1 else 0


def _ints(name: str, t: torch.Tensor, dev: int, n: int) -> int:
    if t.dtype is not torch.int32 or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        _bad(name, f"expected a contiguous int32 tensor of {n} on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _table(t: torch.Tensor, dev: int, n: int) -> tuple:
    """(address, rows, columns) of the table of n requests or tokens; it may be empty if there are none."""
    if t.dtype is not torch.int32 or t.dim() != 2 or t.get_device() != dev:
        _bad("table", f"expected int32 [requests][pages] on cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    rows, cols = t.shape
    if (n > 0 and (rows < 1 or cols < 1)) or not t.is_contiguous():   # (a slice's row stride would be taken for its width)
        _bad("table", f"expected a contiguous tensor of at least one row and page, got {tuple(t.shape)}")
    return t.data_ptr(), rows, cols


def _refuse_grad() -> None:
    if torch.is_grad_enabled():
        raise RuntimeError("these operations record no gradient: call them on detached tensors "
                           "(rope(..., transposed=True) is the gradient of rope)")


def _refuse_tangent(*tensors: torch.Tensor) -> None:
    """Inside a forward_ad level: none of the tensors may be a dual one. (Such a tensor does not say so by requires_grad.)"""
    if any(forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise RuntimeError("these operations carry no tangent: call them on primals (rope is linear: rope of the "
                           "tangent is the result's tangent)")


_HERE = contextlib.nullcontext()


def _on(dev: int):
    """Makes device `dev` current for a launch, where it is not."""
    return _HERE if _current_device() == dev else torch.cuda.device(dev)


def _device_of(name: str, t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        _bad(name, f"on {t.device}: a CUDA device is needed")
    return dev


def rope(x: torch.Tensor, pos: torch.Tensor, plan: Rope, out: Optional[torch.Tensor] = None,
         out_dtype: Optional[torch.dtype] = None, transposed: bool = False) -> torch.Tensor:
    """x [T][heads][head_dim] (fp32 or bf16, strided) rotated to positions pos (int32 [T]).

    out: where the result goes (x itself rotates in place); without it a new contiguous tensor
    of out_dtype (x's type by default). transposed: the transposed map, i.e. the gradient."""
    if x.dim() != 3:
        _bad("x", f"expected [T][heads][head_dim], got {tuple(x.shape)}")
    dev = _device_of("x", x)
    T, H, hd = x.shape
    xt, xh = _heads("x", x, dev, T, H, hd, _TYPES)
    at = _ints("pos", pos, dev, T)
    given = out is not None
    if not given:
        dtype = out_dtype or x.dtype
        if dtype not in _TYPES:
            _bad("out_dtype", f"{dtype}, expected one of {[str(d) for d in _TYPES]}")
        out = torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)
        yt, yh = H * hd, hd
    else:
        if out_dtype is not None and out_dtype != out.dtype:
            _bad("out", f"{out.dtype}, but out_dtype is {out_dtype}")
        if out.requires_grad:
            _refuse_grad()
        yt, yh = _heads("out", out, dev, T, H, hd, _TYPES)
    if x.requires_grad:
        _refuse_grad()
    if forward_ad._current_level >= 0:   # (a look at a number, where asking each tensor costs 0.3 us)
        _refuse_tangent(x, out)
    with _on(dev):
        binding.dllm_op_rope(plan.c, x.data_ptr(), _TYPES[x.dtype], xt, xh, at, T, H, hd, out.data_ptr(),
                             _TYPES[out.dtype], yt, yh, 1 if transposed else 0, _stream_of(dev))
    if given:
        increment_version(out)
    return out


class KVCache4:
    """One layer's pages of 4-bit keys and values, 0.5625 bytes per value.

    codes uint8 [n_pages][2][n_kv_heads][page][head_dim / 2] and scales uint8
    [n_pages][2][n_kv_heads][page][head_dim / 16], as include/dllm.h lays them out. Page tables
    belong to the caller: int32 [requests][pages per request].
    """

    def __init__(self, n_pages: int, page: int, n_kv_heads: int, head_dim: int, device="cuda"):
        if page not in (16, 32, 64, 128, 256):
            _bad("page", f"{page}: 16, 32, 64, 128 or 256 positions")
        if head_dim not in (64, 128, 176):
            _bad("head_dim", f"{head_dim}: 64, 128 or 176")
        if n_pages < 1 or n_kv_heads < 1:
            _bad("n_pages, n_kv_heads", "at least 1 each")
        shape = (n_pages, 2, n_kv_heads, page)
        self._init(torch.zeros((*shape, head_dim // 2), dtype=torch.uint8, device=device),
                   torch.zeros((*shape, head_dim // 16), dtype=torch.uint8, device=device))

    @classmethod
    def from_tensors(cls, codes: torch.Tensor, scales: torch.Tensor) -> "KVCache4":
        """A cache over the caller's own arrays."""
        self = cls.__new__(cls)
        self._init(codes, scales)
        return self

    def _init(self, codes, scales):
        for name, t in (("codes", codes), ("scales", scales)):
            if t.dtype != torch.uint8 or t.dim() != 5 or not t.is_contiguous():
                _bad(name, "expected a contiguous uint8 tensor of 5 dimensions")
            if t.data_ptr() % 16:
                _bad(name, "has to lie on a 16-byte boundary")
        if codes.device != scales.device or codes.shape[:4] != scales.shape[:4] or codes.shape[1] != 2 \
                or codes.shape[4] != 8 * scales.shape[4]:
            _bad("codes, scales", f"{tuple(codes.shape)} and {tuple(scales.shape)} do not belong together")
        self.codes, self.scales, self.device = codes, scales, codes.device
        self.n_pages, _, self.n_kv_heads, self.page = codes.shape[:4]
        self.head_dim = 2 * codes.shape[4]
        self._sizes = {}
        self.c = binding.dllm_kv4(codes.data_ptr(), scales.data_ptr(), self.n_pages, self.page, self.n_kv_heads,
                                  self.head_dim)
        self._dev = _device_of("codes, scales", codes)
        # the library's own check of the sizes
        binding.dllm_op_attn_kv4_workspace(self.c, 0, 0, 0, 0, self.n_kv_heads)

    def append(self, k: torch.Tensor, v: torch.Tensor, req: torch.Tensor, pos: torch.Tensor, table: torch.Tensor,
               rope: Optional[Rope] = None, rope_pos: Optional[torch.Tensor] = None) -> None:
        """Writes k, v [T][n_kv_heads][head_dim] (one type, fp32 or bf16, strided) to positions pos of
        table rows req (int32 [T]; req < 0: padding), k rotated by `rope` to rope_pos (pos by default)."""
        T, H, d, dev = k.shape[0], self.n_kv_heads, self.head_dim, self._dev
        kt, kh = _heads("k", k, dev, T, H, d, _TYPES)
        vt, vh = _heads("v", v, dev, T, H, d, (k.dtype,))
        if k.requires_grad or v.requires_grad:
            _refuse_grad()
        if forward_ad._current_level >= 0:
            _refuse_tangent(k, v)
        req_ptr, pos_ptr = _ints("req", req, dev, T), _ints("pos", pos, dev, T)
        rope_ptr = None if rope_pos is None else _ints("rope_pos", rope_pos, dev, T)
        tab, rows, stride = _table(table, dev, T)
        with _on(dev):
            binding.dllm_op_append_kv4(self.c, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, _TYPES[k.dtype], req_ptr,
                                       pos_ptr, rope_ptr, T, tab, rows, stride, None if rope is None else rope.c,
                                       _stream_of(dev))

    def read(self, req: torch.Tensor, pos: torch.Tensor, table: torch.Tensor, k_out: Optional[torch.Tensor] = None,
             v_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Positions pos of table rows req as bf16 (k, v), each [T][n_kv_heads][head_dim]. Rows of padding
        (req < 0) are left as they were in k_out and v_out, and are zero in outputs made here."""
        T, H, d, dev = req.shape[0], self.n_kv_heads, self.head_dim, self._dev
        outs, made = [], k_out is None or v_out is None
        if made and not (k_out is None and v_out is None):
            _bad("k_out, v_out", "give both or neither")
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is None:
                t = self.codes.new_empty((T, H, d), dtype=torch.bfloat16)
            else:
                _heads(name, t, dev, T, H, d, (torch.bfloat16,))
                if not t.is_contiguous():
                    _bad(name, "has to be contiguous")
                if t.requires_grad:
                    _refuse_grad()
            outs.append(t)
        if forward_ad._current_level >= 0:
            _refuse_tangent(*outs)
        req_ptr, pos_ptr = _ints("req", req, dev, T), _ints("pos", pos, dev, T)
        tab, rows, stride = _table(table, dev, T)
        with _on(dev):
            binding.dllm_op_read_kv4(self.c, req_ptr, pos_ptr, T, tab, rows, stride, outs[0].data_ptr(),
                                     outs[1].data_ptr(), 1 if made else 0, _stream_of(dev))
        if not made:
            increment_version(outs)
        return outs[0], outs[1]

    def attend(self, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, table: torch.Tensor, max_q: int,
               max_kv: int, causal: bool = False, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               return_lse: bool = False, workspace: Optional[torch.Tensor] = None):
        """Attention of a batch's queries over the cache (dllm_op_attn_kv4).

        q bf16 [T][heads][head_dim]; request b's queries are rows q_start[b] .. q_start[b + 1] - 1 and
        it sees positions below kv_len[b] of table row b; causal: its queries are the last of
        those. max_q, max_kv: bounds on a request's queries and keys. scale: 1 / sqrt(head_dim)
        by default. workspace: a uint8 tensor of workspace_bytes(...) for callers that allocate
        nothing here. Returns out (bf16, q's shape), with return_lse (out, lse fp32 [T][heads]); rows
        that no request covers are left as they were, so they hold anything in tensors made here."""
        if q.dim() != 3:
            _bad("q", f"expected [T][heads][head_dim], got {tuple(q.shape)}")
        T, H, hd = q.shape
        dev, B = self._dev, kv_len.shape[0]
        qt, qh = _heads("q", q, dev, T, H, self.head_dim, (torch.bfloat16,))
        if q.requires_grad:
            _refuse_grad()
        tab, rows, stride = _table(table, dev, B)
        if rows < B:
            _bad("table", f"{rows} rows for {B} requests")
        given = out is not None
        if not given:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            ot, oh = H * hd, hd
        else:
            ot, oh = _heads("out", out, dev, T, H, hd, (torch.bfloat16,))
            if out.requires_grad:
                _refuse_grad()
        if forward_ad._current_level >= 0:
            _refuse_tangent(q, out)
        lse = q.new_empty((T, H), dtype=torch.float32) if return_lse else None
        if workspace is None:
            size = self.workspace_bytes(B, T, max_q, max_kv, H)
            if size:
                workspace = self.codes.new_empty(size)
        else:
            if workspace.get_device() != dev or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
                _bad("workspace", "expected a contiguous uint8 tensor on the cache's device")
            size = workspace.numel()
        start_ptr, len_ptr = _ints("q_start", q_start, dev, B + 1), _ints("kv_len", kv_len, dev, B)
        with _on(dev):
            binding.dllm_op_attn_kv4(self.c, q.data_ptr(), qt, qh, out.data_ptr(), ot, oh,
                                     lse.data_ptr() if return_lse else None, start_ptr, len_ptr, B, T, max_q, max_kv, H,
                                     tab, stride, 1 if causal else 0, hd ** -0.5 if scale is None else scale,
                                     None if workspace is None else workspace.data_ptr(), size, _stream_of(dev))
        if given:
            increment_version(out)
        return (out, lse) if return_lse else out

    def workspace_bytes(self, B: int, T: int, max_q: int, max_kv: int, heads: int) -> int:
        """Bytes of workspace that attend() needs for these sizes."""
        sizes = (B, T, max_q, max_kv, heads)
        n = self._sizes.get(sizes)
        if n is None:
            n = binding.dllm_op_attn_kv4_workspace(self.c, *sizes)
            if len(self._sizes) >= 1024:
                self._sizes.clear()
            self._sizes[sizes] = n
        return n
