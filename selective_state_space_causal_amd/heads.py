"""The head scan (linear attention with one decay per head) and the norms around a mixer block: the
binding of the ``mamba_mixer_heads_*``, ``mamba_mixer_gate_norm*`` and ``mamba_mixer_residual_norm*``
calls.  Like the rest of the binding it checks shapes and types, allocates outputs and workspace and
passes pointers; the computation is in the library's kernels.

Token tensors may be column ranges of a wider one (a projection's output): their rows may be strided,
the elements of a row are contiguous.

With ``stream`` given the kernels run on that stream, and what a call allocates belongs to it: the workspace
goes back to that stream's memory, and outputs may be used and dropped on the stream that was current at the call,
once it has waited for the given one.  Ordering the inputs before the call, and keeping them until the stream has
read them, is the caller's part, as with any work on a second stream.
"""
from __future__ import annotations

from . import MM_OK, MambaMixError, _check, _io_code, check_cu_seqlens, load, _new_on

torch = _BF16 = _F32 = _raw_stream = None  # (the package can be imported without torch)


def _lib():
    """The library; torch and its types are at hand from then on: calls of a few microseconds have no time for more."""
    global torch, _BF16, _F32, _raw_stream
    if torch is None:
        import torch as t

        torch, _BF16, _F32 = t, t.bfloat16, t.float32
        _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None)
    return load()


def _need(t, shape, dtype, name):
    """``_check`` with the answer yes found quickly."""
    if not (t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        _check(t, shape, dtype, name)


def _code(t) -> int:
    return 1 if t.dtype is _BF16 else 0 if t.dtype is _F32 else _io_code(t)


_MAX_STRIDE = 4194304  # MM_HEADS_MAX_STRIDE


def _plan_code(code, *strides) -> int:
    """The io type whose workspace a head scan of these row strides needs: wider rows take float32's path."""
    return code if max(strides) <= _MAX_STRIDE else 0


def _opt(t):
    return t.data_ptr() if t is not None else None


def _on(stream, t):
    """The raw stream a call goes to: the given one, or the current one of the tensor's device."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(t.device.index)
    return torch.cuda.current_stream(t.device).cuda_stream


def _rows(t, shape, dtype, name) -> int:
    """Check a token tensor [T, ...] whose rows may be strided; returns the row stride in elements."""
    if t.shape == shape and t.dtype is dtype and t.is_cuda:
        stride, width = t.stride(), 1
        for n, s in zip(shape[:0:-1], stride[:0:-1]):
            if n != 1 and s != width:
                break
            width *= n
        else:
            if width > 0 and (shape[0] <= 1 or stride[0] >= width):
                return stride[0] if shape[0] > 1 else width
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    width = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != width and t.numel() > 0:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        width *= n
    if t.shape[0] <= 1 or t.numel() == 0:
        return max(width, 1)
    raise ValueError(f"{name}: rows must not overlap (stride {t.stride(0)}, row length {width})")


def _head_inputs(x, dt, B, C, A_log, D, dt_bias):
    """Checks of the inputs all three head-scan calls share; returns (T, H, P, G, N, strides)."""
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [T, H, P] and B [T, G, N]")
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    io = x.dtype
    _lib()
    _code(x)
    strides = [_rows(x, (T, H, P), io, "x"), 0, _rows(B, (T, G, N), io, "B"), _rows(C, (T, G, N), io, "C")]
    _need(A_log, (H,), _F32, "A_log")
    if dt is not None:
        strides[1] = _rows(dt, (T, H), io, "dt")
        if dt_bias is None:
            raise ValueError("dt_bias: required with dt")
        _need(dt_bias, (H,), _F32, "dt_bias")
    if D is not None:
        _need(D, (H,), _F32, "D")
    return T, H, P, G, N, strides


def _new(shape, dtype, device, stream):
    return torch.empty(shape, dtype=dtype, device=device) if stream is None else _new_on(stream, shape, dtype, device)


def _workspace(given, need, device, stream):
    if given is None and need > 0:
        if stream is None:
            given = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            given = _new_on(stream, need, torch.uint8, device, returned=False)
    return given, _opt(given), 0 if given is None else given.numel() * given.element_size()


def _out(t, shape, dtype, device, name, stream):
    """An output tensor: the caller's (rows may be strided) or a new one; returns it and its row stride."""
    if t is None:
        t = _new(shape, dtype, device, stream)
    return t, _rows(t, shape, dtype, name)


def _raise(rc, where):
    if rc != MM_OK:
        raise MambaMixError(rc, where)


def heads_prefill(x, dt, B, C, A_log, D, dt_bias, cu_seqlens, state_in=None, state_out=None, y=None, workspace=None,
                  stream=None):
    """The head scan over packed sequences (see ``mamba_mixer_heads_prefill``).

    x [T, H, P], dt [T, H] (None: a fixed decay for each head), B, C [T, G, N] share one io dtype
    (float32 or bfloat16); A_log, D, dt_bias [H] float32 (D may be None); cu_seqlens [S+1] int32;
    state_in [S, H, P, N] float32 (None: zeros).  Returns (y [T, H, P], state_out [S, H, P, N]);
    pass state_out=state_in to update a state in place.
    """
    from . import CHECK_CU

    T, H, P, G, N, strides = _head_inputs(x, dt, B, C, A_log, D, dt_bias)
    S = cu_seqlens.shape[0] - 1
    _need(cu_seqlens, (S + 1,), torch.int32, "cu_seqlens")
    if CHECK_CU:
        check_cu_seqlens(cu_seqlens, T)
    if state_in is not None:
        _need(state_in, (S, H, P, N), _F32, "state_in")
    if state_out is None:
        state_out = _new((S, H, P, N), _F32, x.device, stream)
    else:
        _need(state_out, (S, H, P, N), _F32, "state_out")
    if y is None:
        y = _new((T, H, P), x.dtype, x.device, stream)
    else:
        _need(y, (T, H, P), x.dtype, "y")
    io = _code(x)
    need = 0
    if workspace is None:
        need = _lib().mamba_mixer_heads_prefill_workspace_bytes(S, T, H, P, G, N, _plan_code(io, *strides))
    workspace, wptr, wbytes = _workspace(workspace, need, x.device, stream)
    rc = _lib().mamba_mixer_heads_prefill(
        x.data_ptr(), _opt(dt), B.data_ptr(), C.data_ptr(), A_log.data_ptr(), _opt(D), _opt(dt_bias),
        cu_seqlens.data_ptr(), _opt(state_in), state_out.data_ptr(), y.data_ptr(), S, T, H, P, G, N, io, *strides,
        wptr, wbytes, _on(stream, x))
    _raise(rc, "mamba_mixer_heads_prefill")
    return y, state_out


def heads_decode(x, dt, B, C, A_log, D, dt_bias, state_in=None, state_out=None, y=None, stream=None):
    """One token of the head scan for each of Bs rows (see ``mamba_mixer_heads_decode``): x [Bs, H, P],
    dt [Bs, H] or None, B, C [Bs, G, N], state_in [Bs, H, P, N] float32 (None: zeros).  Returns
    (y [Bs, H, P], state_out); pass state_out=state_in to update the states in place."""
    Bs, H, P, G, N, strides = _head_inputs(x, dt, B, C, A_log, D, dt_bias)
    if state_in is not None:
        _need(state_in, (Bs, H, P, N), _F32, "state_in")
    if state_out is None:
        state_out = _new((Bs, H, P, N), _F32, x.device, stream)
    else:
        _need(state_out, (Bs, H, P, N), _F32, "state_out")
    if y is None:
        y = _new((Bs, H, P), x.dtype, x.device, stream)
    else:
        _need(y, (Bs, H, P), x.dtype, "y")
    rc = _lib().mamba_mixer_heads_decode(
        x.data_ptr(), _opt(dt), B.data_ptr(), C.data_ptr(), A_log.data_ptr(), _opt(D), _opt(dt_bias),
        _opt(state_in), state_out.data_ptr(), y.data_ptr(), Bs, H, P, G, N, _code(x), *strides, _on(stream, x))
    _raise(rc, "mamba_mixer_heads_decode")
    return y, state_out


def heads_backward(x, dt, B, C, A_log, D, dt_bias, cu_seqlens, state_in, dy, dstate_out=None, dx=None, ddt=None,
                   dB=None, dC=None, need_dstate=True, workspace=None, stream=None) -> dict:
    """The gradients of ``heads_prefill`` (see ``mamba_mixer_heads_backward``) from dy [T, H, P] and
    dstate_out [S, H, P, N] (None: the loss does not depend on the final states).  dx, ddt, dB and dC may be
    given (column ranges of one gradient, for instance).  Returns a dict of dx, ddt, dB, dC (io), dA_log, dD,
    ddt_bias and dstate_in (float32); ddt and ddt_bias are None without dt, dD without D, dstate_in with
    need_dstate=False."""
    from . import CHECK_CU

    T, H, P, G, N, strides = _head_inputs(x, dt, B, C, A_log, D, dt_bias)
    S = cu_seqlens.shape[0] - 1
    io, dev = x.dtype, x.device
    _need(cu_seqlens, (S + 1,), torch.int32, "cu_seqlens")
    if CHECK_CU:
        check_cu_seqlens(cu_seqlens, T)
    for t, n in ((state_in, "state_in"), (dstate_out, "dstate_out")):
        if t is not None:
            _need(t, (S, H, P, N), _F32, n)
    _need(dy, (T, H, P), io, "dy")
    dx, sx = _out(dx, (T, H, P), io, dev, "dx", stream)
    ddt, sd = _out(ddt, (T, H), io, dev, "ddt", stream) if dt is not None else (None, 0)
    dB, sb = _out(dB, (T, G, N), io, dev, "dB", stream)
    dC, sc = _out(dC, (T, G, N), io, dev, "dC", stream)
    new = lambda *s: _new(s, _F32, dev, stream)  # noqa: E731
    dA_log, dD, dbias = new(H), new(H) if D is not None else None, new(H) if dt is not None else None
    dstate_in = new(S, H, P, N) if need_dstate else None
    code = _code(x)
    need = 0
    if workspace is None:
        need = _lib().mamba_mixer_heads_backward_workspace_bytes(S, T, H, P, G, N, _plan_code(code, *strides, sx))
    workspace, wptr, wbytes = _workspace(workspace, need, dev, stream)
    rc = _lib().mamba_mixer_heads_backward(
        x.data_ptr(), _opt(dt), B.data_ptr(), C.data_ptr(), A_log.data_ptr(), _opt(D), _opt(dt_bias),
        cu_seqlens.data_ptr(), _opt(state_in), dy.data_ptr(), _opt(dstate_out), dx.data_ptr(), _opt(ddt),
        dB.data_ptr(), dC.data_ptr(), dA_log.data_ptr(), _opt(dD), _opt(dbias), _opt(dstate_in), S, T, H, P, G, N,
        code, *strides, sx, sd, sb, sc, wptr, wbytes, _on(stream, x))
    _raise(rc, "mamba_mixer_heads_backward")
    return dict(dx=dx, ddt=ddt, dB=dB, dC=dC, dA_log=dA_log, dD=dD, ddt_bias=dbias, dstate_in=dstate_in)


def _gate_inputs(y, z, weight, groups):
    if y.dim() != 2:
        raise ValueError("y must be [rows, d]")
    rows, d = y.shape
    _lib()
    _code(y)
    _need(weight, (d,), _F32, "weight")
    return rows, d, _rows(y, (rows, d), y.dtype, "y"), _rows(z, (rows, d), y.dtype, "z")


def gate_norm(y, z, weight, groups: int = 1, eps: float = 1e-5, gate_first: bool = True, out=None, stream=None):
    """The norm after a mixer block, fused with its gate (see ``mamba_mixer_gate_norm``): with s = SiLU(z),
    weight n(y s) (gate_first) or weight n(y) s, n the root-mean-square norm of each of `groups` column
    ranges.  y, z [rows, d] io, weight [d] float32.  Returns out [rows, d]."""
    rows, d, ys, zs = _gate_inputs(y, z, weight, groups)
    if out is None:
        out = _new((rows, d), y.dtype, y.device, stream)
    else:
        _need(out, (rows, d), y.dtype, "out")
    rc = _lib().mamba_mixer_gate_norm(
        y.data_ptr(), z.data_ptr(), weight.data_ptr(), out.data_ptr(), rows, d, int(groups), float(eps),
        1 if gate_first else 0, _code(y), ys, zs, _on(stream, y))
    _raise(rc, "mamba_mixer_gate_norm")
    return out


def gate_norm_backward(dout, y, z, weight, groups: int = 1, eps: float = 1e-5, gate_first: bool = True, dy=None,
                       dz=None, workspace=None, stream=None):
    """The gradients of ``gate_norm`` from dout [rows, d]: (dy, dz, dweight); dy and dz may be given (with
    strided rows)."""
    rows, d, ys, zs = _gate_inputs(y, z, weight, groups)
    _need(dout, (rows, d), y.dtype, "dout")
    dy, dys = _out(dy, (rows, d), y.dtype, y.device, "dy", stream)
    dz, dzs = _out(dz, (rows, d), y.dtype, y.device, "dz", stream)
    dweight = _new((d,), _F32, y.device, stream)
    need = _lib().mamba_mixer_gate_norm_backward_workspace_bytes(rows, d, int(groups)) if workspace is None else 0
    workspace, wptr, wbytes = _workspace(workspace, need, y.device, stream)
    rc = _lib().mamba_mixer_gate_norm_backward(
        dout.data_ptr(), y.data_ptr(), z.data_ptr(), weight.data_ptr(), dy.data_ptr(), dz.data_ptr(),
        dweight.data_ptr(), rows, d, int(groups), float(eps), 1 if gate_first else 0, _code(y), ys, zs, dys, dzs,
        wptr, wbytes, _on(stream, y))
    _raise(rc, "mamba_mixer_gate_norm_backward")
    return dy, dz, dweight


def _residual_inputs(h, residual, weight, post_weight, scale_vec):
    if h.dim() != 2:
        raise ValueError("h must be [rows, d]")
    rows, d = h.shape
    _lib()
    _need(h, (rows, d), h.dtype, "h")
    _code(h)
    for t, n in ((weight, "weight"), (post_weight, "post_weight"), (scale_vec, "scale_vec")):
        if t is not None:
            _need(t, (d,), _F32, n)
    res = residual.dtype if residual is not None else h.dtype
    if residual is not None:
        if res is not _F32 and res is not h.dtype:
            raise TypeError(f"residual: expected float32 or {h.dtype}, got {res}")
        _need(residual, (rows, d), res, "residual")
    return rows, d, res


def residual_norm(h, residual, weight, post_weight=None, scale: float = 1.0, scale_vec=None, eps: float = 1e-5,
                  residual_out=None, out=None, stream=None):
    """The boundary between two blocks (see ``mamba_mixer_residual_norm``): p = h, or post_weight n(h);
    r' = residual + scale scale_vec p; out = weight n(r').  h [rows, d] io; residual [rows, d] float32 or h's
    type (None: zeros, of h's type); weight, post_weight, scale_vec [d] float32.  Returns (out, residual_out);
    pass residual_out=residual to update the residual in place."""
    rows, d, res = _residual_inputs(h, residual, weight, post_weight, scale_vec)
    if residual_out is None:
        residual_out = _new((rows, d), res, h.device, stream)
    else:
        if residual is None:
            res = residual_out.dtype
        _need(residual_out, (rows, d), res, "residual_out")
    if out is None:
        out = _new((rows, d), h.dtype, h.device, stream)
    else:
        _need(out, (rows, d), h.dtype, "out")
    rc = _lib().mamba_mixer_residual_norm(
        h.data_ptr(), _opt(residual), weight.data_ptr(), _opt(post_weight), _opt(scale_vec), float(scale),
        residual_out.data_ptr(), out.data_ptr(), rows, d, float(eps), _code(h), _code(residual_out), _on(stream, h))
    _raise(rc, "mamba_mixer_residual_norm")
    return out, residual_out


def residual_norm_backward(dout, dresidual_out, h, residual_out, weight, post_weight=None, scale: float = 1.0,
                           scale_vec=None, eps: float = 1e-5, dresidual=None, dh=None, workspace=None,
                           stream=None) -> dict:
    """The gradients of ``residual_norm`` from dout [rows, d] and dresidual_out [rows, d] (None: zeros);
    residual_out is the new residual that the forward call returned.  Returns a dict of dresidual, dh, dweight
    and, with post_weight and scale_vec, dpost_weight and dscale_vec."""
    rows, d, res = _residual_inputs(h, residual_out, weight, post_weight, scale_vec)
    _need(dout, (rows, d), h.dtype, "dout")
    if dresidual_out is not None:
        _need(dresidual_out, (rows, d), res, "dresidual_out")
    if dresidual is None:
        dresidual = _new((rows, d), res, h.device, stream)
    else:
        _need(dresidual, (rows, d), res, "dresidual")
    if dh is None:
        dh = _new((rows, d), h.dtype, h.device, stream)
    else:
        _need(dh, (rows, d), h.dtype, "dh")
    new = lambda: _new((d,), _F32, h.device, stream)  # noqa: E731
    got = dict(dresidual=dresidual, dh=dh, dweight=new())
    if post_weight is not None:
        got["dpost_weight"] = new()
    if scale_vec is not None:
        got["dscale_vec"] = new()
    need = _lib().mamba_mixer_residual_norm_backward_workspace_bytes(rows, d) if workspace is None else 0
    workspace, wptr, wbytes = _workspace(workspace, need, h.device, stream)
    rc = _lib().mamba_mixer_residual_norm_backward(
        dout.data_ptr(), _opt(dresidual_out), h.data_ptr(), residual_out.data_ptr(), weight.data_ptr(),
        _opt(post_weight), _opt(scale_vec), float(scale), dresidual.data_ptr(), dh.data_ptr(), got["dweight"].data_ptr(),
        _opt(got.get("dpost_weight")),
        _opt(got.get("dscale_vec")), rows, d, float(eps), _code(h), _code(residual_out), wptr, wbytes,
        _on(stream, h))
    _raise(rc, "mamba_mixer_residual_norm_backward")
    return got
