"""GB300 (sm_103a) linear-recurrence state update behind a C ABI.

``scan_runtime_gb300`` is the Python face of ``libsn.so``:

* ``scan_runtime_gb300._abi`` -- the C functions under their C names
  (``sn_scan_fma``, ``sn_recur_rwkv7``, ...), argument marshalling only;
* ``Context`` -- a small convenience wrapper that owns an ``SnCtx``,
  allocates output tensors with PyTorch and raises ``SnError`` on a non-zero
  status.

PyTorch supplies device memory and streams; every step of the recurrences
runs in libsn's kernels.  Nothing here computes a result on the CPU.
"""
from __future__ import annotations

from . import _abi
from ._abi import *  # noqa: F401,F403  (C names and constants)


def build(force: bool = False) -> str:
    """Compile libsn.so for sm_103a (in-tree)."""
    from ._build import build as _b
    return _b(force=force)


class SnError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status} ({_abi.sn_status_str(status)})")


def _check(status: int, what: str) -> None:
    if status != _abi.SN_OK:
        raise SnError(status, what)


class Context:
    """Owns an ``SnCtx`` bound to one CUDA device."""

    def __init__(self, device: int = 0):
        import torch
        self.device = device
        self._torch = torch
        s, h = _abi.sn_ctx_create(device)
        _check(s, "sn_ctx_create")
        self.handle = h
        self._ws = None
        self._kept = []
        self._lib = _abi.load()
        self._dev, self._empty, self._f32 = torch.device("cuda", device), torch.empty, torch.float32
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._kinds = {torch.float32: _abi.SN_DTYPE_F32, torch.bfloat16: _abi.SN_DTYPE_BF16,
                       torch.float8_e4m3fn: _abi.SN_DTYPE_E4M3}
        self._ids_kinds = {torch.int32: _abi.SN_INDEX_I32, torch.int64: _abi.SN_INDEX_I64}

    def close(self) -> None:
        if getattr(self, "handle", None):
            _abi.sn_ctx_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---------------------------------------------------------------- ctx
    def set_option(self, key: int, value: int) -> None:
        _check(_abi.sn_ctx_set_option(self.handle, key, value), "sn_ctx_set_option")

    def get_option(self, key: int) -> int:
        s, v = _abi.sn_ctx_get_option(self.handle, key)
        _check(s, "sn_ctx_get_option")
        return v

    def last_error(self) -> int:
        return _abi.sn_ctx_last_error(self.handle)

    def ensure_workspace(self, B: int, T: int, N: int) -> None:
        """Give the context enough workspace for the look-back scan of (B, T, N)."""
        self.ensure_workspace_bytes(_abi.sn_workspace_bytes(_abi.SN_OP_SCAN_FMA, B, T, N))

    def ensure_workspace_bytes(self, need: int) -> None:
        """Give the context a workspace of at least `need` bytes.  One that a
        captured call uses is kept beside the new one as long as the context
        lives, because the graph writes to it at every replay; ask for the
        most that will be needed before a capture to have a single one."""
        if self._ws is not None and self._ws.numel() >= need:
            return
        if self._ws is not None and self.get_option(_abi.SN_OPT_WORKSPACE_CAPTURED):
            self._kept.append(self._ws)
        self._ws = self._torch.empty(max(need, 256), dtype=self._torch.uint8, device=f"cuda:{self.device}")
        _check(_abi.sn_ctx_set_workspace(self.handle, self._ws, self._ws.numel()), "sn_ctx_set_workspace")

    def _out(self, shape, want):
        if want is None or want is False:
            return None
        if want is True:
            return self._torch.empty(shape, dtype=self._torch.float32, device=f"cuda:{self.device}")
        return want

    # ---------------------------------------------------------------- tier 1
    def scan_fma(self, a, b, s0=None, *, s_out=True, s_final=True, stream=None):
        B, T, N = a.shape
        so, sf = self._out((B, T, N), s_out), self._out((B, N), s_final)
        _check(_abi.sn_scan_fma(self.handle, B, T, N, a, b, s0, sf, so, stream), "sn_scan_fma")
        return so, sf

    def scan_gated(self, a, u, s0=None, *, s_out=True, s_final=True, stream=None):
        B, T, N = a.shape
        so, sf = self._out((B, T, N), s_out), self._out((B, N), s_final)
        _check(_abi.sn_scan_gated(self.handle, B, T, N, a, u, s0, sf, so, stream), "sn_scan_gated")
        return so, sf

    def scan_host(self, a, b=None, u=None, s0=None, *, out=None, rows_per_chunk=1):
        """Scan host (CPU, ideally pinned) tensors through the GPU with
        ``sn_scan_host``: the FMA form when ``b`` is given, the gated form when
        ``u`` is given, sharing the upload of ``a``; batch rows stream through
        the device in chunks of ``rows_per_chunk`` on the context's three
        pipeline streams.  Returns ``{"fma": (s_out, s_final), "gated": (...)}``
        as CPU tensors, filled once the call returns; pass ``out`` (the same
        dict shape, pinned tensors) to reuse buffers across calls."""
        torch = self._torch
        B, T, N = a.shape
        forms = [f for f, x in (("fma", b), ("gated", u)) if x is not None]
        if not forms:
            raise ValueError("give b (FMA form), u (gated form) or both")
        outs = dict(out or {})
        for f in forms:
            if f not in outs:
                outs[f] = (torch.empty((B, T, N), pin_memory=True), torch.empty((B, N), pin_memory=True))
        mask = (1 if b is not None else 0) | (2 if u is not None else 0)
        need = _abi.sn_scan_host_staging_bytes(B, T, N, mask, rows_per_chunk)
        if need < 0:
            raise ValueError("invalid dimensions for sn_scan_host")
        if getattr(self, "_staging", None) is None or self._staging.numel() < need:
            self._staging = torch.empty(max(need, 256), dtype=torch.uint8, device=f"cuda:{self.device}")
        fo, go = outs.get("fma", (None, None)), outs.get("gated", (None, None))
        stream = torch.cuda.current_stream(torch.device(f"cuda:{self.device}"))
        _check(_abi.sn_scan_host(self.handle, B, T, N, rows_per_chunk, a, b, u, s0, fo[0], fo[1], go[0], go[1],
                                 self._staging, self._staging.numel(), stream), "sn_scan_host")
        stream.synchronize()
        return outs

    def scan_backward(self, form, a, s, grad_s, *, s0=None, grad_final=None, u=None, stream=None):
        """Reverse scan of `form` ("fma" or "gated"); returns (grad_a, grad_b|grad_u, grad_s0)."""
        B, T, N = a.shape
        ga, gb, g0 = self._out((B, T, N), True), self._out((B, T, N), True), self._out((B, N), True)
        if form == "fma":
            st = _abi.sn_scan_fma_backward(self.handle, B, T, N, a, s0, s, grad_s, grad_final, ga, gb, g0, stream)
        else:
            st = _abi.sn_scan_gated_backward(self.handle, B, T, N, a, u, s0, s, grad_s, grad_final, ga, gb, g0,
                                             stream)
        _check(st, f"sn_scan_{form}_backward")
        return ga, gb, g0

    # ---------------------------------------------------------------- tier 2
    def recur_diag(self, q, k, v, d, S_in=None, *, H, G, decay_kind, scale, S_out=True, o=True, stream=None):
        B, T, _, dk = k.shape
        dv = v.shape[3]
        So, oo = self._out((B, H, dk, dv), S_out), self._out((B, T, H, dv), o)
        _check(_abi.sn_recur_diag(self.handle, B, T, H, G, dk, dv, decay_kind, scale, q, k, v, d, S_in, So, oo,
                                  stream), "sn_recur_diag")
        return oo, So

    def recur_diag_chunked(self, q, k, v, d, S_in=None, *, H, G, decay_kind, scale, S_out=True, o=True,
                           stream=None):
        """Chunked tensor-core form of recur_diag (tf32 operands); sizes the
        context workspace on first use."""
        B, T, _, dk = k.shape
        dv = v.shape[3]
        need = _abi.sn_recur_chunked_workspace_bytes(B, T, H, dk, dv)
        if need < 0:
            raise SnError(_abi.SN_E_INVAL, "sn_recur_chunked_workspace_bytes")
        self.ensure_workspace_bytes(need)
        So, oo = self._out((B, H, dk, dv), S_out), self._out((B, T, H, dv), o)
        _check(_abi.sn_recur_diag_chunked(self.handle, B, T, H, G, dk, dv, decay_kind, scale, q, k, v, d, S_in, So,
                                          oo, stream), "sn_recur_diag_chunked")
        return oo, So

    def readout_norm_gate(self, o, g, w=None, *, eps, y=True, stream=None):
        """GLA readout epilogue y = RMSNorm(o) * w * silu(g); o, g (B, T, H, dv).
        Pass y=o to write in place."""
        B, T, H, dv = o.shape
        yy = self._out((B, T, H, dv), y)
        _check(_abi.sn_readout_norm_gate(self.handle, B, T, H, dv, o, g, w, eps, yy, stream), "sn_readout_norm_gate")
        return yy

    def readout_dskip(self, o, x, D, *, y=True, stream=None):
        """Mamba-2 skip connection y = o + D_h x; o, x (B, T, H, dv), D (H,)."""
        B, T, H, dv = o.shape
        yy = self._out((B, T, H, dv), y)
        _check(_abi.sn_readout_dskip(self.handle, B, T, H, dv, o, x, D, yy, stream), "sn_readout_dskip")
        return yy

    def recur_delta_chunked(self, q, k, v, beta, S_in=None, *, scale, S_out=True, o=True, stream=None):
        """Chunked tensor-core form of recur_delta (tf32 operands); sizes the
        context workspace on first use."""
        B, T, H, dk = k.shape
        dv = v.shape[3]
        need = _abi.sn_recur_delta_chunked_workspace_bytes(B, T, H, dk, dv)
        if need < 0:
            raise SnError(_abi.SN_E_INVAL, "sn_recur_delta_chunked_workspace_bytes")
        self.ensure_workspace_bytes(need)
        So, oo = self._out((B, H, dk, dv), S_out), self._out((B, T, H, dv), o)
        _check(_abi.sn_recur_delta_chunked(self.handle, B, T, H, dk, dv, scale, q, k, v, beta, S_in, So, oo, stream),
               "sn_recur_delta_chunked")
        return oo, So

    def recur_delta(self, q, k, v, beta, S_in=None, *, scale, S_out=True, o=True, stream=None):
        B, T, H, dk = k.shape
        dv = v.shape[3]
        So, oo = self._out((B, H, dk, dv), S_out), self._out((B, T, H, dv), o)
        _check(_abi.sn_recur_delta(self.handle, B, T, H, dk, dv, scale, q, k, v, beta, S_in, So, oo, stream),
               "sn_recur_delta")
        return oo, So

    def recur_rwkv7(self, q, k, v, w, S_in=None, *, S_out=True, o=True, stream=None):
        B, T, H, dk = k.shape
        dv = v.shape[3]
        So, oo = self._out((B, H, dv, dk), S_out), self._out((B, T, H, dv), o)
        _check(_abi.sn_recur_rwkv7(self.handle, B, T, H, dk, dv, q, k, v, w, S_in, So, oo, stream),
               "sn_recur_rwkv7")
        return oo, So

    # ---------------------------------------------------------------- around the recurrent layer
    # A decoding loop makes these calls for single tokens, where the host's
    # share is most of the time: the checks below cost well under a
    # microsecond a tensor.
    def _kind(self, dtype, what):
        """SN_DTYPE_* of a torch dtype."""
        k = self._kinds.get(dtype)
        if k is None:
            raise ValueError(f"{what}: {dtype} is not supported")
        return k

    def _row_kind(self, dtype, what):
        """SN_DTYPE_* of a torch dtype that may not be 8 bits."""
        k = self._kinds.get(dtype)
        if k is None or k == _abi.SN_DTYPE_E4M3:
            raise ValueError(f"{what}: {dtype} is not supported")
        return k

    def _ids_kind(self, dtype, what):
        k = self._ids_kinds.get(dtype)
        if k is None:
            raise ValueError(f"{what}: {dtype} is not supported (int32 or int64)")
        return k

    def _in(self, what, t, shape=None, dtype=None):
        """Address of an operand, checked: on this device, contiguous, and of
        the shape and type expected.  None stays NULL."""
        if t is None:
            return None
        if t.get_device() != self.device:
            raise ValueError(f"{what} is on {t.device}, the context on cuda:{self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{what} is {t.dtype}, expected {dtype}")
        return t.data_ptr()

    def _output(self, what, given, shape, dtype):
        """(tensor, address) of an output: a new tensor for True, none for
        False or None, else the one given, checked."""
        if given is True:
            t = self._empty(shape, dtype=dtype, device=self._dev)
            return t, t.data_ptr()
        if given is None or given is False:
            return None, None
        return given, self._in(what, given, shape, dtype)

    def _on(self, stream, *tensors):
        """The handle of a stream given as such or as a torch stream (default:
        the current one of this device).  On another stream than the current
        one, tells the allocator of the tensors' use there, so that it does not
        hand their memory out early."""
        if stream is None:
            return self._raw_stream(self.device)
        if isinstance(stream, int):
            if stream == self._raw_stream(self.device):
                return stream
            # (1 is another name of the default stream, whose handle is 0)
            stream = self._torch.cuda.ExternalStream(0 if stream == 1 else stream, self._dev)
        if stream.cuda_stream != self._raw_stream(self.device):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        return stream.cuda_stream

    def _workspace(self, need, what):
        if need < 0:
            raise SnError(_abi.SN_E_INVAL, what)
        if self._ws is None or self._ws.numel() < need:
            self.ensure_workspace_bytes(need)

    def embed(self, ids, table, *, scale=1.0, dtype=None, out=True, stream=None):
        """scale * table[ids]: ids of any shape (int32 or int64), table (V, D);
        rows of ids outside [0, V) are zeros.  The output's type is `dtype`
        (default: the table's) or that of the `out` given."""
        V, D = table.shape
        if out is None or out is False:
            out = True
        dtype = (dtype or table.dtype) if out is True else out.dtype
        out, op = self._output("out", out, (*ids.shape, D), dtype)
        _check(self._lib.sn_embed(
            self.handle, ids.numel(), V, D, self._row_kind(table.dtype, "table"), self._row_kind(dtype, "out"),
            self._ids_kind(ids.dtype, "ids"), self._in("ids", ids), self._in("table", table), scale, op,
            self._on(stream, ids, table, out)), "sn_embed")
        return out

    def embed_backward(self, ids, grad_out, V, *, scale=1.0, dtype=None, grad_table=True, accumulate=False,
                       stream=None):
        """Gradient of ``embed`` with respect to the (V, D) table, in `dtype`
        (default: grad_out's); with ``accumulate`` it is added to the
        `grad_table` given.  Sizes the context workspace on first use."""
        D = grad_out.shape[-1]
        if grad_table is None or grad_table is False:
            grad_table = True
        if accumulate and grad_table is True:
            raise ValueError("accumulate needs a grad_table to add to")
        n = ids.numel()
        self._workspace(self._lib.sn_embed_backward_workspace_bytes(n, V, D), "sn_embed_backward_workspace_bytes")
        dtype = (dtype or grad_out.dtype) if grad_table is True else grad_table.dtype
        gt, gp = self._output("grad_table", grad_table, (V, D), dtype)
        _check(self._lib.sn_embed_backward(
            self.handle, n, V, D, self._row_kind(grad_out.dtype, "grad_out"), self._row_kind(dtype, "grad_table"),
            self._ids_kind(ids.dtype, "ids"), self._in("ids", ids), self._in("grad_out", grad_out, (*ids.shape, D)),
            scale, 1 if accumulate else 0, gp, self._on(stream, ids, grad_out, gt, self._ws)), "sn_embed_backward")
        return gt

    def add_rmsnorm(self, x, r=None, w=None, *, eps, dtype=None, group=0, h=True, y=True, rstd=False, stream=None):
        """h = x + r and y = RMSNorm(h) * w over the last dimension; returns
        (y, scales, h, rstd).  `dtype` is y's type (default x's); for
        ``torch.float8_e4m3fn`` scales (..., groups) holds one fp32 scale a row
        (group=0) or for every 128 columns (group=128), else it is None.
        h=False leaves the sum unwritten; rstd=True returns what
        ``add_rmsnorm_backward`` takes."""
        shape, xt, f32 = x.shape, x.dtype, self._f32
        lead, D = shape[:-1], shape[-1]
        R = x.numel() // D if D else 0
        if y is None or y is False:
            y = True
        yt = (dtype or xt) if y is True else y.dtype
        kind, scales, sp = self._kind(yt, "y"), None, None
        y, yp = self._output("y", y, shape, yt)
        h, hp = self._output("h", h, shape, xt)
        rstd, rp = self._output("rstd", rstd, lead, f32)
        if kind == _abi.SN_DTYPE_E4M3:
            scales, sp = self._output("scales", True, (*lead, 1 if group == 0 else -(-D // 128)), f32)
        _check(self._lib.sn_add_rmsnorm(
            self.handle, R, D, self._row_kind(xt, "x"), kind, group, self._in("x", x), self._in("r", r, shape, xt),
            self._in("w", w, (D,), f32), eps, hp, yp, sp, rp, self._on(stream, x, r, w, h, y, scales, rstd)),
            "sn_add_rmsnorm")
        return y, scales, h, rstd

    def add_rmsnorm_backward(self, dy, h, w, rstd, dh=None, *, dx=True, dw=True, stream=None):
        """Gradient of ``add_rmsnorm`` from the h and rstd it returned: (dx, dw),
        dx being the gradient of x and of r alike; dh is the gradient that
        reaches h from elsewhere.  dw=False skips the weight's.  Sizes the
        context workspace on first use."""
        shape, ht, f32 = h.shape, h.dtype, self._f32
        D = shape[-1]
        R = h.numel() // D if D else 0
        dx, xp = self._output("dx", True if dx is None or dx is False else dx, shape, ht)
        dw, wp = self._output("dw", dw, (D,), f32)
        ws = None
        if dw is not None:
            need = self._lib.sn_add_rmsnorm_backward_workspace_bytes(R, D)
            if need < 0 < R * D:
                raise SnError(_abi.SN_E_UNSUPPORTED, "sn_add_rmsnorm_backward_workspace_bytes")
            self._workspace(need, "sn_add_rmsnorm_backward_workspace_bytes")
            ws = self._ws
        _check(self._lib.sn_add_rmsnorm_backward(
            self.handle, R, D, self._row_kind(ht, "h"), self._row_kind(dy.dtype, "dy"), self._in("dy", dy, shape),
            self._in("h", h), self._in("w", w, (D,), f32), self._in("rstd", rstd, shape[:-1], f32),
            self._in("dh", dh, shape, ht), xp, wp, self._on(stream, dy, h, w, rstd, dh, dx, dw, ws)),
            "sn_add_rmsnorm_backward")
        return dx, dw

    def linear_ce(self, h, w, targets, *, logit_scale=1.0, loss=True, lse=True, stream=None):
        """Cross entropy of the logits logit_scale * h w^T, h (..., D) and w
        (V, D) in one type, without forming them all: (loss, lse), fp32 of
        targets' shape, 0 where a target is outside [0, V).  Sizes the context
        workspace on first use."""
        V, D = w.shape
        shape, N, kind = targets.shape, targets.numel(), self._row_kind(h.dtype, "h")
        self._workspace(self._lib.sn_linear_ce_workspace_bytes(N, V, D, kind, 0), "sn_linear_ce_workspace_bytes")
        loss, lop = self._output("loss", loss, shape, self._f32)
        lse, lsp = self._output("lse", True if lse is None or lse is False else lse, shape, self._f32)
        _check(self._lib.sn_linear_ce(
            self.handle, N, V, D, kind, self._ids_kind(targets.dtype, "targets"), self._in("h", h, (*shape, D)),
            self._in("w", w, None, h.dtype), self._in("targets", targets), logit_scale, lop, lsp,
            self._on(stream, h, w, targets, loss, lse, self._ws)), "sn_linear_ce")
        return loss, lse

    def linear_ce_backward(self, h, w, targets, lse, grad_loss=None, *, logit_scale=1.0, dh=True, dw=True,
                           stream=None):
        """Gradient of ``linear_ce`` from the lse it returned: (dh, dw) in h's
        type; grad_loss (default ones) has targets' shape.  Either gradient may
        be left out with False.  Sizes the context workspace on first use."""
        V, D = w.shape
        shape, N, ht = targets.shape, targets.numel(), h.dtype
        kind = self._row_kind(ht, "h")
        self._workspace(self._lib.sn_linear_ce_workspace_bytes(N, V, D, kind, 1), "sn_linear_ce_workspace_bytes")
        dh, hp = self._output("dh", dh, h.shape, ht)
        dw, wp = self._output("dw", dw, w.shape, ht)
        _check(self._lib.sn_linear_ce_backward(
            self.handle, N, V, D, kind, self._ids_kind(targets.dtype, "targets"), self._in("h", h, (*shape, D)),
            self._in("w", w, None, ht), self._in("targets", targets), logit_scale,
            self._in("lse", lse, shape, self._f32), self._in("grad_loss", grad_loss, shape, self._f32), hp, wp,
            self._on(stream, h, w, targets, lse, grad_loss, dh, dw, self._ws)), "sn_linear_ce_backward")
        return dh, dw
