"""Attention over exact KV rows in the caller's tensors: window with sinks, decode with accumulated
attention weights and the eviction that goes by them, decode over a shared prefix. Thin owner of the
C structs and of the workspace; all arithmetic runs in ``libiskv.so``."""
from __future__ import annotations

import ctypes

import torch

from .binding import (ISKV_BF16, ISKV_F32, check, iskv_evict_workspace, iskv_exact_prefix,
                      iskv_exact_queries, iskv_exact_rows, iskv_exact_status,
                      iskv_mass_decode_workspace, iskv_prefix_decode_workspace,
                      iskv_window_attn_workspace, lib)

D = 128
_TYPES = {torch.bfloat16: ISKV_BF16, torch.float32: ISKV_F32}


def _strides(x: torch.Tensor, n: int):
    """Strides of the first ``n`` dimensions; 0 for an extent of 1, whose stride is not read."""
    return [s if e > 1 else 0 for s, e in zip(x.stride()[:n], x.shape[:n])]


class ExactKVCache:
    """Exact rows of ``batch`` sequences: ``k`` and ``v`` are ``[batch][n_kv][rows][128]`` CUDA
    tensors (bf16 or float32, the same strides, last dimension contiguous; any order of the others,
    so a view of ``[batch][rows][n_kv][128]`` is fine), attended as they are (keys already
    rotated). ``lens``: int32 ``[batch]`` on the device, the rows that each sequence holds;
    ``None``: all. The tensors are read at each call: rows written and lengths advanced between
    calls count.

    Calls run on the current stream of the tensors' device, or on ``stream``, and synchronise
    nothing. They share the object's workspace: calls that may overlap (other streams, graphs
    replayed at the same time) need objects of their own, which may hold the same tensors. A
    captured call uses addresses of this object's workspace, so the object has to outlive the
    graph. An object is not thread-safe.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, lens: torch.Tensor | None = None):
        if k.dim() != 4 or k.shape[-1] != D or k.shape != v.shape:
            raise ValueError(f"k and v must both be [batch][n_kv][rows][{D}]")
        if not k.is_cuda or k.device != v.device:
            raise ValueError("k and v must be on one CUDA device")
        if k.dtype not in _TYPES or v.dtype != k.dtype:
            raise ValueError("k and v must both be bfloat16 or float32")
        if k.stride(-1) != 1 or v.stride(-1) != 1 or _strides(k, 3) != _strides(v, 3):
            raise ValueError("k and v must have the same strides and contiguous rows")
        self.k, self.v, self.lens = k, v, lens
        self.device = k.device
        self.batch, self.n_kv_heads, self.rows = k.shape[:3]
        if lens is not None:
            self._check(lens, "lens", torch.int32, (self.batch,))
        self._rows = iskv_exact_rows(k.data_ptr(), v.data_ptr(), *_strides(k, 3), *k.shape[:3],
                                     _TYPES[k.dtype], lens.data_ptr() if lens is not None else None)
        self._rows_at = ctypes.addressof(self._rows)
        self._queries: dict = {}        # per form of the queries: (struct, its address)
        self._need: dict = {}           # per call form: workspace bytes
        self._prefix = self._prefix_form = None
        self._ws: torch.Tensor | None = None
        self._old_ws: list = []         # captured graphs may hold their addresses

    # -- plumbing --------------------------------------------------------------------------------
    def _check(self, x: torch.Tensor, what: str, dtype, shape) -> None:
        if x.device != self.device or x.dtype != dtype or tuple(x.shape) != tuple(shape):
            raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)} on {self.device}")
        if not x.is_contiguous():
            raise ValueError(f"{what} must be contiguous")

    def _stream(self, stream, *owned) -> int:
        current = torch.cuda.current_stream(self.device)
        if stream is None:
            return current.cuda_stream
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        if stream != current:
            # what this call allocated must not be reused before `stream` is done with it
            for x in owned:
                x.record_stream(stream)
        return stream.cuda_stream

    def _workspace(self, bytes_: int) -> torch.Tensor:
        if self._ws is None or self._ws.numel() < bytes_:
            if self._ws is not None:
                self._old_ws.append(self._ws)
            self._ws = torch.empty((bytes_,), dtype=torch.uint8, device=self.device)
        return self._ws

    def _form(self, q: torch.Tensor, out: torch.Tensor | None, q_lens, tokens: bool):
        """The C struct of a call's queries and outputs (kept per form) and the outputs."""
        made = out is None
        if made:
            out = torch.empty_like(q)
        key = (q.shape, q.stride(), out.stride(), q.dtype, tokens)
        known = self._queries.get(key)
        if known is None or out.shape != q.shape or out.dtype != q.dtype:
            dims = 4 if tokens else 3
            if q.dim() != dims or q.shape[0] != self.batch or q.shape[-1] != D:
                raise ValueError("q must be [batch][n_q][m][128]" if tokens else
                                 "q must be [batch][n_q][128]")
            if q.dtype not in _TYPES or out.dtype != q.dtype or out.shape != q.shape:
                raise ValueError("q and out must be of one shape, bfloat16 or float32")
            if q.stride(-1) != 1 or out.stride(-1) != 1:
                raise ValueError("q and out must have contiguous rows of 128")
            m = q.shape[2] if tokens else 1
            x = iskv_exact_queries(None, None, *(_strides(q, dims - 1) + [0] * (4 - dims)),
                                   *(_strides(out, dims - 1) + [0] * (4 - dims)), q.shape[1], m,
                                   _TYPES[q.dtype], None)
            if len(self._queries) >= 256:           # forms come and go with the chunks' lengths
                self._queries.clear()
                self._need.clear()
            known = self._queries[key] = (x, ctypes.addressof(x))
        if q.device != self.device or out.device != self.device:
            raise ValueError(f"q and out must be on {self.device}")
        if q_lens is not None:
            self._check(q_lens, "q_lens", torch.int32, (self.batch,))
        x = known[0]
        x.q, x.out = q.data_ptr(), out.data_ptr()
        x.q_lens = q_lens.data_ptr() if q_lens is not None else None
        return known, out, made, key

    def _bytes(self, key, ask) -> int:
        n = self._need.get(key)
        if n is None:
            with torch.cuda.device(self.device):
                code, n = ask()
            check(code, key[0])
            self._need[key] = n
        return n

    def _call(self, name: str, stream: int, *args) -> None:
        if torch.cuda.current_device() == self.device.index:
            check(getattr(lib, name)(*args, stream), name)
        else:
            with torch.cuda.device(self.device):
                check(getattr(lib, name)(*args, stream), name)

    # -- calls ------------------------------------------------------------------------------------
    def window_attn(self, q: torch.Tensor, *, window: int, sinks: int = 0,
                    q_lens: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
        """Attention of each sequence's last ``q_lens[b]`` rows' tokens (``None``: all ``m``), ``q``
        ``[batch][n_q][m][128]``: token i sits at position ``p = lens[b] - q_lens[b] + i`` and sees
        the rows ``j <= p`` with ``j < sinks`` or ``j > p - window``. A token that sees nothing gets
        zeros; outputs of tokens ``i >= q_lens[b]`` are not written."""
        (x, at), out, made, form = self._form(q, out, q_lens, True)
        need = self._bytes(("iskv_window_attn", form, window, sinks),
                           lambda: iskv_window_attn_workspace(self._rows, x, window, sinks))
        ws = self._workspace(need)
        s = self._stream(stream, ws, *([out] if made else []))
        self._call("iskv_window_attn", s, self._rows_at, at, window, sinks, ws.data_ptr(), need)
        return out

    def mass_decode(self, q: torch.Tensor, mass: torch.Tensor, *,
                    mass_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None):
        """Decode attention of one token per sequence (``q`` ``[batch][n_q][128]``) over all its
        rows. Adds each row's attention weight, summed over the q-heads of its kv-head, to ``mass``
        (float32 ``[batch][n_kv][rows]``), in place or into ``mass_out``. Returns
        ``(out, mass_out)``."""
        shape = (self.batch, self.n_kv_heads, self.rows)
        self._check(mass, "mass", torch.float32, shape)
        if mass_out is None:
            mass_out = mass
        else:
            self._check(mass_out, "mass_out", torch.float32, shape)
        (x, at), out, made, form = self._form(q, out, None, False)
        need = self._bytes(("iskv_mass_decode", form),
                           lambda: iskv_mass_decode_workspace(self._rows, x))
        ws = self._workspace(need)
        s = self._stream(stream, ws, *([out] if made else []))
        self._call("iskv_mass_decode", s, self._rows_at, at, mass.data_ptr(), mass_out.data_ptr(),
                   ws.data_ptr(), need)
        return out, mass_out

    def evict(self, mass: torch.Tensor, pos: torch.Tensor, *, budget: int, recent: int,
              sinks: int = 0, mass_out: torch.Tensor | None = None,
              pos_out: torch.Tensor | None = None, lens_out: torch.Tensor | None = None,
              stream=None) -> None:
        """Keeps ``budget`` rows of every (sequence, kv-head) that holds more, in its first slots:
        positions ``< sinks``, the ``recent`` latest positions, and the heaviest of the rest (ties:
        the lowest slot). Rows move in place; ``mass`` (float32), ``pos`` (int32, both
        ``[batch][n_kv][rows]``) and the lengths are updated in place or into the ``*_out``
        tensors. Without ``lens_out`` the cache needs its own ``lens``."""
        shape = (self.batch, self.n_kv_heads, self.rows)
        mass_out = mass if mass_out is None else mass_out
        pos_out = pos if pos_out is None else pos_out
        lens_out = self.lens if lens_out is None else lens_out
        if lens_out is None:
            raise ValueError("a cache without lens needs lens_out")
        self._check(mass, "mass", torch.float32, shape)
        self._check(mass_out, "mass_out", torch.float32, shape)
        self._check(pos, "pos", torch.int32, shape)
        self._check(pos_out, "pos_out", torch.int32, shape)
        self._check(lens_out, "lens_out", torch.int32, (self.batch,))
        need = self._bytes(("iskv_evict", budget), lambda: iskv_evict_workspace(self._rows, budget))
        ws = self._workspace(need)
        s = self._stream(stream, ws)
        self._call("iskv_evict", s, self._rows_at, mass.data_ptr(), mass_out.data_ptr(),
                   pos.data_ptr(), pos_out.data_ptr(), lens_out.data_ptr(), budget, recent, sinks,
                   ws.data_ptr(), need)

    def prefix_decode(self, q: torch.Tensor, prefix_k: torch.Tensor, prefix_v: torch.Tensor, *,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Decode attention of one token per sequence (``q`` ``[batch][n_q][128]``) over the rows
        ``prefix_k``, ``prefix_v`` (``[n_kv][P][128]``) that all sequences share, and its own."""
        key = (prefix_k.shape, prefix_k.stride(), prefix_v.shape, prefix_v.stride(),
               prefix_k.dtype, prefix_v.dtype, prefix_k.device, prefix_v.device)
        if self._prefix_form != key:
            for x in (prefix_k, prefix_v):
                if (x.dim() != 3 or x.shape[0] != self.n_kv_heads or x.shape[-1] != D or
                        x.dtype != self.k.dtype or x.device != self.device or x.stride(-1) != 1):
                    raise ValueError("prefix_k and prefix_v must be [n_kv][P][128], in the rows' "
                                     "dtype and on their device, with contiguous rows")
            if prefix_k.shape != prefix_v.shape or _strides(prefix_k, 2) != _strides(prefix_v, 2):
                raise ValueError("prefix_k and prefix_v must have the same shape and strides")
            self._prefix = iskv_exact_prefix(None, None, *_strides(prefix_k, 2), prefix_k.shape[1])
            self._prefix_form = key
        p = self._prefix
        p.k, p.v = prefix_k.data_ptr(), prefix_v.data_ptr()
        p_at = ctypes.addressof(p)
        (x, at), out, made, form = self._form(q, out, None, False)
        need = self._bytes(("iskv_prefix_decode", form, prefix_k.shape),
                           lambda: iskv_prefix_decode_workspace(self._rows, x, p))
        ws = self._workspace(need)
        s = self._stream(stream, ws, *([out] if made else []))
        self._call("iskv_prefix_decode", s, self._rows_at, at, p_at, ws.data_ptr(), need)
        return out

    def status(self, stream=None) -> int:
        """Status of the calls on exact caches on this device (synchronises): 0, or the code of a
        device-side wait that gave up."""
        with torch.cuda.device(self.device):
            return iskv_exact_status(stream)
