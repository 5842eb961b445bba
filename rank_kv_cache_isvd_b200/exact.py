"""Attention over exact KV rows in the caller's tensors: window with sinks, decode with accumulated
attention weights and the eviction that goes by them, decode over a shared prefix. Thin owner of the
C structs and of the workspace; all arithmetic runs in ``libiskv.so``."""
from __future__ import annotations

import ctypes

import torch

from .binding import (ISKV_BF16, ISKV_F32, _int32, check, iskv_evict_workspace, iskv_exact_prefix,
                      iskv_exact_queries, iskv_exact_rows, iskv_exact_status,
                      iskv_mass_decode_workspace, iskv_prefix_decode_workspace,
                      iskv_window_attn_workspace, lib)

D = 128
_TYPES = {torch.bfloat16: ISKV_BF16, torch.float32: ISKV_F32}


def _strides(x: torch.Tensor, n: int):
    """Strides of the first ``n`` dimensions; 0 for an extent of 1, whose stride is not read."""
    return [s if e > 1 else 0 for s, e in zip(x.stride()[:n], x.shape[:n])]


def _span(x: torch.Tensor) -> int:
    """Bytes from the first element of ``x`` to behind its last one."""
    return x.element_size() * (1 + sum((e - 1) * s for s, e in zip(x.stride(), x.shape))) if x.numel() else 0


def _overlap(delta: int, a, b, row: int) -> bool:
    """Whether two tensors of rows of ``row`` bytes share a byte: the second begins ``delta`` bytes behind the
    first; ``a``, ``b``: their rows' ``(stride in bytes, extent)``. Looks for places i, j with
    ``|delta + j . b - i . a| < row``, the longest stride first. A search that grows long (tensors whose
    dimensions do not nest) counts as an overlap."""
    reach: dict = {}                                 # stride: range of its factor
    for strides, low, high in ((a, 0, 1), (b, -1, 0)):
        for s, e in strides:
            if s > 0 and e > 1:
                x = reach.get(s, (0, 0))
                reach[s] = (x[0] + low * (e - 1), x[1] + high * (e - 1))
    dims = sorted(((s, lo, hi) for s, (lo, hi) in reach.items()), reverse=True)
    low, high = [0], [0]                             # sums of the dimensions behind
    for s, lo, hi in reversed(dims):
        low.append(low[-1] + s * lo)
        high.append(high[-1] + s * hi)
    low.reverse()
    high.reverse()
    left, steps = [(0, delta)], 0
    while left:
        i, d = left.pop()
        if i == len(dims):
            if abs(d) < row:
                return True
            continue
        s, lo, hi = dims[i]
        first = max(lo, -((row - 1 + high[i + 1] - d) // s))         # d - x s <= high + row - 1
        last = min(hi, (d - low[i + 1] + row - 1) // s)              # d - x s >= low - row + 1
        steps += max(0, last - first + 1)
        if steps > 10000:
            return True
        left.extend((i + 1, d - x * s) for x in range(first, last + 1))
    return False


def _rows_of(x: torch.Tensor):
    return [(s * x.element_size(), e) for s, e in zip(x.stride()[:-1], x.shape[:-1])]


class _Plan:
    """What a form of a call keeps: its C structs, their addresses, the spans of queries and outputs, and
    its workspace's size."""
    __slots__ = ("x", "x_at", "p", "p_at", "need", "q_span", "out_span")


class ExactKVCache:
    """Exact rows of ``batch`` sequences: ``k`` and ``v`` are ``[batch][n_kv][rows][128]`` CUDA
    tensors (bf16 or float32, the same strides, last dimension contiguous; any order of the others,
    so a view of ``[batch][rows][n_kv][128]`` is fine), attended as they are (keys already
    rotated). ``lens``: int32 ``[batch]`` on the device, the rows that each sequence holds;
    ``None``: all. The tensors are read at each call: rows written and lengths advanced in place
    between calls count; other tensors need another object.

    Calls run on the current stream of the tensors' device, or as if ``stream`` were that one, and
    synchronise nothing. They share the object's workspace: calls that may overlap (other streams, graphs
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
        self._k, self._v, self._lens = k, v, lens
        self.device = k.device
        self._index = k.get_device()
        self.batch, self.n_kv_heads, self.rows = k.shape[:3]
        self._batch_shape = torch.Size((self.batch,))
        self._mass_shape = torch.Size((self.batch, self.n_kv_heads, self.rows))
        self._mass_bytes = 4 * self._mass_shape.numel()
        if lens is not None:
            self._check(lens, "lens", torch.int32, self._batch_shape)
        self._rows = iskv_exact_rows(k.data_ptr(), v.data_ptr(), *_strides(k, 3), *k.shape[:3],
                                     _TYPES[k.dtype], lens.data_ptr() if lens is not None else None)
        self._rows_at = ctypes.addressof(self._rows)
        self._plans: dict = {}          # per form of a call: its structs and workspace size
        self._ws: torch.Tensor | None = None
        self._ws_stream = 0             # whose memory it is
        self._ws_captured = False       # a graph may hold its address
        self._old_ws: list = []         # earlier ones of which that is true

    # The C structs hold their addresses: they cannot be replaced.
    @property
    def k(self) -> torch.Tensor:
        return self._k

    @property
    def v(self) -> torch.Tensor:
        return self._v

    @property
    def lens(self) -> torch.Tensor | None:
        return self._lens

    # -- plumbing --------------------------------------------------------------------------------
    def _check(self, x: torch.Tensor, what: str, dtype, shape) -> None:
        if (x.dtype is not dtype or x.shape != shape or x.get_device() != self._index or
                not x.is_contiguous()):
            raise ValueError(f"{what} must be contiguous, {dtype} of shape {tuple(shape)} on "
                             f"{self.device}")

    def _under(self, stream):
        """Makes ``stream`` (a torch stream of the device, or a raw handle) the current one: what a
        call allocates then comes from that stream's memory."""
        if isinstance(stream, int):
            stream = (torch.cuda.ExternalStream(stream, device=self.device) if stream else
                      torch.cuda.default_stream(self.device))
        elif stream.device != self.device:
            raise ValueError(f"stream must be of {self.device}")
        return torch.cuda.stream(stream)

    def _stream(self) -> int:
        """The current stream; the workspace is not handed out before its work on it is done, nor while
        a graph that is captured now may use it."""
        raw = torch._C._cuda_getCurrentRawStream(self._index)
        if not self._ws_captured and raw:            # (the default stream cannot be captured)
            if torch._C._cuda_getDevice() == self._index:
                self._ws_captured = torch._C._cuda_isCurrentStreamCapturing()
            else:
                with torch.cuda.device(self._index):
                    self._ws_captured = torch._C._cuda_isCurrentStreamCapturing()
        if raw != self._ws_stream:
            self._ws.record_stream(torch.cuda.current_stream(self.device))
        return raw

    def _plan(self, key, make):
        """The plan of a call's form; ``make(plan)`` fills a new one and asks for its workspace."""
        plan = self._plans.get(key)
        if plan is None:
            plan = _Plan()
            with torch.cuda.device(self._index):
                code, plan.need = make(plan)
            check(code, key[0])
            if len(self._plans) >= 512:             # forms come and go with the chunks' lengths
                self._plans.clear()
            self._plans[key] = plan
        if self._ws is None or self._ws.numel() < plan.need:
            size = plan.need
            if self._ws is not None:
                # half as large again at least: forms that grow call by call ask for few, and those that
                # graphs keep add up to three times the largest
                size = max(size, self._ws.numel() * 3 // 2)
                if self._ws_captured:
                    self._old_ws.append(self._ws)
            self._ws = torch.empty((size,), dtype=torch.uint8, device=self.device)
            self._ws_stream = torch._C._cuda_getCurrentRawStream(self._index)
            self._ws_captured = False
        return plan

    def _queries(self, plan, q: torch.Tensor, out: torch.Tensor, tokens: bool):
        """Fills a plan's struct of queries and outputs, all but the pointers."""
        dims = 4 if tokens else 3
        if q.dim() != dims or q.shape[0] != self.batch or q.shape[-1] != D:
            raise ValueError("q must be [batch][n_q][m][128]" if tokens else
                             "q must be [batch][n_q][128]")
        if q.dtype not in _TYPES or out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("q and out must be of one shape, bfloat16 or float32")
        if q.stride(-1) != 1 or out.stride(-1) != 1:
            raise ValueError("q and out must have contiguous rows of 128")
        self._on_device(q, out)
        rest = [0] * (4 - dims)
        plan.x = iskv_exact_queries(q.data_ptr(), out.data_ptr(), *(_strides(q, dims - 1) + rest),
                                    *(_strides(out, dims - 1) + rest), q.shape[1],
                                    q.shape[2] if tokens else 1, _TYPES[q.dtype], None)
        plan.x_at = ctypes.addressof(plan.x)
        plan.q_span, plan.out_span = _span(q), _span(out)

    @staticmethod
    def _apart(plan, q: torch.Tensor, out: torch.Tensor):
        """Addresses of queries and outputs. Blocks that share queries read them at different times,
        so outputs cannot take the place of any."""
        at, to = q.data_ptr(), out.data_ptr()
        if at < to + plan.out_span and to < at + plan.q_span and _overlap(
                to - at, _rows_of(q), _rows_of(out), D * q.element_size()):
            raise ValueError("out must not overlap q")
        return at, to

    @staticmethod
    def _in_place(at: int, to: int, size: int, what: str) -> None:
        """Of contiguous arrays of ``size`` bytes: the one at ``to`` is the one at ``at``, or apart."""
        if at != to and -size < to - at < size:
            raise ValueError(f"{what} must be the input or not overlap it")

    def _on_device(self, *tensors) -> None:
        for x in tensors:
            if x.get_device() != self._index:
                raise ValueError(f"tensors must be on {self.device}")

    def _call(self, name: str, fn, *args) -> None:
        if torch._C._cuda_getDevice() == self._index:
            code = fn(*args)
        else:
            with torch.cuda.device(self._index):
                code = fn(*args)
        if code:
            check(code, name)

    # -- calls ------------------------------------------------------------------------------------
    def window_attn(self, q: torch.Tensor, *, window: int, sinks: int = 0,
                    q_lens: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
        """Attention of each sequence's last ``q_lens[b]`` rows' tokens (``None``: all ``m``), ``q``
        ``[batch][n_q][m][128]``: token i sits at position ``p = lens[b] - q_lens[b] + i`` and sees
        the rows ``j <= p`` with ``j < sinks`` or ``j > p - window``. A token that sees nothing gets
        zeros; outputs of tokens ``i >= q_lens[b]`` are not written."""
        if stream is not None:
            with self._under(stream):
                return self.window_attn(q, window=window, sinks=sinks, q_lens=q_lens, out=out)
        if out is None:
            out = torch.empty_like(q)

        def make(plan):
            self._queries(plan, q, out, True)
            return iskv_window_attn_workspace(self._rows, plan.x, window, sinks)

        plan = self._plan(("iskv_window_attn", q.shape, q.stride(), out.shape, out.stride(), q.dtype,
                           out.dtype, window, sinks), make)
        self._on_device(q, out)
        x, ws = plan.x, self._ws
        x.q, x.out = self._apart(plan, q, out)
        x.q_lens = None
        if q_lens is not None:
            self._check(q_lens, "q_lens", torch.int32, self._batch_shape)
            x.q_lens = q_lens.data_ptr()
        s = self._stream()
        self._call("iskv_window_attn", lib.iskv_window_attn, self._rows_at, plan.x_at, window, sinks,
                   ws.data_ptr(), plan.need, s)
        return out

    def mass_decode(self, q: torch.Tensor, mass: torch.Tensor, *,
                    mass_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None):
        """Decode attention of one token per sequence (``q`` ``[batch][n_q][128]``) over all its
        rows. Adds each row's attention weight, summed over the q-heads of its kv-head, to ``mass``
        (float32 ``[batch][n_kv][rows]``), in place or into ``mass_out``. Returns
        ``(out, mass_out)``."""
        if stream is not None:
            with self._under(stream):
                return self.mass_decode(q, mass, mass_out=mass_out, out=out)
        self._check(mass, "mass", torch.float32, self._mass_shape)
        if mass_out is None:
            mass_out = mass
        else:
            self._check(mass_out, "mass_out", torch.float32, self._mass_shape)
            self._in_place(mass.data_ptr(), mass_out.data_ptr(), self._mass_bytes, "mass_out")
        if out is None:
            out = torch.empty_like(q)

        def make(plan):
            self._queries(plan, q, out, False)
            return iskv_mass_decode_workspace(self._rows, plan.x)

        plan = self._plan(("iskv_mass_decode", q.shape, q.stride(), out.shape, out.stride(), q.dtype,
                           out.dtype), make)
        self._on_device(q, out)
        x, ws = plan.x, self._ws
        x.q, x.out = self._apart(plan, q, out)
        s = self._stream()
        self._call("iskv_mass_decode", lib.iskv_mass_decode, self._rows_at, plan.x_at,
                   mass.data_ptr(), mass_out.data_ptr(), ws.data_ptr(), plan.need, s)
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
        if stream is not None:
            with self._under(stream):
                return self.evict(mass, pos, budget=budget, recent=recent, sinks=sinks,
                                  mass_out=mass_out, pos_out=pos_out, lens_out=lens_out)
        mass_out = mass if mass_out is None else mass_out
        pos_out = pos if pos_out is None else pos_out
        lens_out = self._lens if lens_out is None else lens_out
        if lens_out is None:
            raise ValueError("a cache without lens needs lens_out")
        shape = self._mass_shape
        self._check(mass, "mass", torch.float32, shape)
        self._check(pos, "pos", torch.int32, shape)
        if mass_out is not mass:
            self._check(mass_out, "mass_out", torch.float32, shape)
        if pos_out is not pos:
            self._check(pos_out, "pos_out", torch.int32, shape)
        self._check(lens_out, "lens_out", torch.int32, self._batch_shape)
        m, m_to, p, p_to = mass.data_ptr(), mass_out.data_ptr(), pos.data_ptr(), pos_out.data_ptr()
        l_to = lens_out.data_ptr()
        self._in_place(m, m_to, self._mass_bytes, "mass_out")
        self._in_place(p, p_to, self._mass_bytes, "pos_out")
        if self._rows.lens:
            self._in_place(self._rows.lens, l_to, 4 * self.batch, "lens_out")
        def make(plan):
            _int32(recent=recent, sinks=sinks)
            return iskv_evict_workspace(self._rows, budget)

        plan = self._plan(("iskv_evict", budget, recent, sinks), make)
        ws = self._ws
        self._call("iskv_evict", lib.iskv_evict, self._rows_at, m, m_to, p, p_to, l_to, budget, recent,
                   sinks, ws.data_ptr(), plan.need, self._stream())

    def prefix_decode(self, q: torch.Tensor, prefix_k: torch.Tensor, prefix_v: torch.Tensor, *,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Decode attention of one token per sequence (``q`` ``[batch][n_q][128]``) over the rows
        ``prefix_k``, ``prefix_v`` (``[n_kv][P][128]``) that all sequences share, and its own."""
        if stream is not None:
            with self._under(stream):
                return self.prefix_decode(q, prefix_k, prefix_v, out=out)
        if out is None:
            out = torch.empty_like(q)

        def make(plan):
            for x in (prefix_k, prefix_v):
                if (x.dim() != 3 or x.shape[0] != self.n_kv_heads or x.shape[-1] != D or
                        x.dtype != self._k.dtype or x.device != self.device or x.stride(-1) != 1):
                    raise ValueError("prefix_k and prefix_v must be [n_kv][P][128], in the rows' "
                                     "dtype and on their device, with contiguous rows")
            if prefix_k.shape != prefix_v.shape or _strides(prefix_k, 2) != _strides(prefix_v, 2):
                raise ValueError("prefix_k and prefix_v must have the same shape and strides")
            self._queries(plan, q, out, False)
            plan.p = iskv_exact_prefix(prefix_k.data_ptr(), prefix_v.data_ptr(),
                                       *_strides(prefix_k, 2), prefix_k.shape[1])
            plan.p_at = ctypes.addressof(plan.p)
            return iskv_prefix_decode_workspace(self._rows, plan.x, plan.p)

        plan = self._plan(("iskv_prefix_decode", q.shape, q.stride(), out.shape, out.stride(),
                           q.dtype, out.dtype, prefix_k.shape, prefix_k.stride(), prefix_v.shape,
                           prefix_v.stride(), prefix_k.dtype, prefix_v.dtype), make)
        self._on_device(q, out, prefix_k, prefix_v)
        x, p, ws = plan.x, plan.p, self._ws
        x.q, x.out = self._apart(plan, q, out)
        p.k, p.v = prefix_k.data_ptr(), prefix_v.data_ptr()
        s = self._stream()
        self._call("iskv_prefix_decode", lib.iskv_prefix_decode, self._rows_at, plan.x_at, plan.p_at,
                   ws.data_ptr(), plan.need, s)
        return out

    def status(self, stream=None) -> int:
        """Status of the calls on exact caches on this device (synchronises): 0, or the code of a
        device-side wait that gave up."""
        with torch.cuda.device(self.device):
            return iskv_exact_status(stream)
