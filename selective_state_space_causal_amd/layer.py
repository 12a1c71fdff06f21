"""The causal depthwise convolution by itself, the gated recurrence (one decay and one state per channel) and the
norms of queries and keys with their rotation: the binding of the ``mamba_mixer_conv_*``, ``mamba_mixer_gated_*`` and
``mamba_mixer_qk_norm*`` calls.  It checks shapes, types and devices, allocates outputs and workspace and passes
pointers, as the binding of the head scan does; rows and streams are as there.
"""
from __future__ import annotations

from . import heads as _h
from . import check_cu_seqlens
from .heads import _code, _need, _new, _on, _opt, _out, _raise, _rows, _workspace

GATES = {"silu": 0, "gelu": 1}
GATED_BLOCK = 64  # MM_GATED_BLOCK: tokens between two checkpoints

_current_device = None


def _lib():
    global _current_device
    lib = _h._lib()
    if _current_device is None:
        _current_device = getattr(_h.torch._C, "_cuda_getDevice", None) or _h.torch.cuda.current_device
    return lib


def _run(name, x, tensors, *args):
    """The library's call, on x's device, which all its tensors have to be on."""
    index = x.get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name}: tensors on {x.device} and {t.device}")
    call = getattr(_lib(), name)
    if index < 0 or index == _current_device():
        rc = call(*args)
    else:
        with _h.torch.cuda.device(index):
            rc = call(*args)
    if rc:
        _raise(rc, name)


def _sequences(cu_seqlens, T):
    from . import CHECK_CU

    S = cu_seqlens.shape[0] - 1
    _need(cu_seqlens, (S + 1,), _h.torch.int32, "cu_seqlens")
    if CHECK_CU:
        check_cu_seqlens(cu_seqlens, T)
    return S


def _given(t, shape, dtype, name, device, stream):
    """A contiguous output: the caller's or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    _need(t, shape, dtype, name)
    return t


def _rows_out(t, shape, dtype, name, device, stream, width):
    """An output whose rows (of `width` elements) may be strided, and their stride: the caller's or a new one."""
    return (_new(shape, dtype, device, stream), width) if t is None else _out(t, shape, dtype, device, name, stream)


def _conv_inputs(x, weight, bias):
    lib = _lib()
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [T, d] and weight [d, W]")
    T, d = x.shape
    W = weight.shape[1]
    io = _code(x)
    _need(weight, (d, W), _h._F32, "weight")
    if bias is not None:
        _need(bias, (d,), _h._F32, "bias")
    return lib, T, d, W, io, _rows(x, (T, d), x.dtype, "x")


def conv_prefill(x, weight, bias, cu_seqlens, state_in=None, state_out=None, silu: bool = True, y=None, stream=None):
    """The causal depthwise convolution over packed sequences (see ``mamba_mixer_conv_prefill``): x [T, d] io (rows may
    be strided), weight [d, W] and bias [d] (or None) float32, cu_seqlens [S+1] int32, state_in [S, d, W-1] float32
    (None: zeros), the raw inputs before each sequence, oldest first.  Returns (y [T, d], state_out); pass
    state_out=state_in to update the states in place."""
    _, T, d, W, io, xs = _conv_inputs(x, weight, bias)
    S = _sequences(cu_seqlens, T)
    shape = (S, d, W - 1)
    if state_in is not None:
        _need(state_in, shape, _h._F32, "state_in")
    state_out = _given(state_out, shape, _h._F32, "state_out", x.device, stream)
    y = _given(y, (T, d), x.dtype, "y", x.device, stream)
    _run("mamba_mixer_conv_prefill", x, (weight, bias, cu_seqlens, state_in, state_out, y), x.data_ptr(), weight.data_ptr(),
         _opt(bias), cu_seqlens.data_ptr(), _opt(state_in), state_out.data_ptr(), y.data_ptr(), S, T, d, W,
         1 if silu else 0, io, xs, _on(stream, x))
    return y, state_out


def conv_decode(x, weight, bias, state_in=None, state_out=None, silu: bool = True, y=None, stream=None):
    """One token of the convolution for each of Bs rows (see ``mamba_mixer_conv_decode``): x [Bs, d], state_in
    [Bs, d, W-1] float32 (None: zeros).  Returns (y [Bs, d], state_out)."""
    _, Bs, d, W, io, xs = _conv_inputs(x, weight, bias)
    shape = (Bs, d, W - 1)
    if state_in is not None:
        _need(state_in, shape, _h._F32, "state_in")
    state_out = _given(state_out, shape, _h._F32, "state_out", x.device, stream)
    y = _given(y, (Bs, d), x.dtype, "y", x.device, stream)
    _run("mamba_mixer_conv_decode", x, (weight, bias, state_in, state_out, y), x.data_ptr(), weight.data_ptr(), _opt(bias),
         _opt(state_in), state_out.data_ptr(), y.data_ptr(), Bs, d, W, 1 if silu else 0, io, xs, _on(stream, x))
    return y, state_out


def conv_backward(x, weight, bias, cu_seqlens, state_in, dy, dstate_out=None, silu: bool = True, dx=None,
                  need_dstate: bool = True, workspace=None, stream=None) -> dict:
    """The gradients of ``conv_prefill`` (see ``mamba_mixer_conv_backward``) from dy [T, d] and dstate_out [S, d, W-1]
    (None: the loss does not depend on the final states); dx may be given (with strided rows).  Returns a dict of dx
    (io), dweight, dbias (None without bias) and dstate_in (None with need_dstate=False), float32."""
    lib, T, d, W, io, xs = _conv_inputs(x, weight, bias)
    S, dev = _sequences(cu_seqlens, T), x.device
    shape = (S, d, W - 1)
    for t, n in ((state_in, "state_in"), (dstate_out, "dstate_out")):
        if t is not None:
            _need(t, shape, _h._F32, n)
    _need(dy, (T, d), x.dtype, "dy")
    dx, dxs = _rows_out(dx, (T, d), x.dtype, "dx", dev, stream, d)
    dweight = _new((d, W), _h._F32, dev, stream)
    dbias = _new((d,), _h._F32, dev, stream) if bias is not None else None
    dstate_in = _new(shape, _h._F32, dev, stream) if need_dstate else None
    need = lib.mamba_mixer_conv_backward_workspace_bytes(T, d, W) if workspace is None else 0
    workspace, wptr, wbytes = _workspace(workspace, need, dev, stream)
    _run("mamba_mixer_conv_backward", x, (weight, bias, cu_seqlens, state_in, dy, dstate_out, dx, workspace), x.data_ptr(),
         weight.data_ptr(), _opt(bias), cu_seqlens.data_ptr(), _opt(state_in), dy.data_ptr(), _opt(dstate_out),
         dx.data_ptr(), dweight.data_ptr(), _opt(dbias), _opt(dstate_in), S, T, d, W, 1 if silu else 0, io, xs, dxs, wptr,
         wbytes, _on(stream, x))
    return dict(dx=dx, dweight=dweight, dbias=dbias, dstate_in=dstate_in)


def _gated_inputs(x, r, g, z, lam, gate):
    lib = _lib()
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    shape, dtype = x.shape, x.dtype
    if gate not in GATES:
        raise ValueError(f"gate: expected one of {sorted(GATES)}, got {gate!r}")
    io = _code(x)
    if lam is not None:
        _need(lam, (shape[1],), _h._F32, "lam")
    return lib, shape[0], shape[1], io, (
        _rows(x, shape, dtype, "x"), _rows(r, shape, dtype, "r"), _rows(g, shape, dtype, "g") if g is not None else 0,
        _rows(z, shape, dtype, "z") if z is not None else 0)


def gated_prefill(x, r, g, z, lam, cu_seqlens, state_in=None, state_out=None, c: float = 8.0, gate: str = "silu", y=None,
                  ckpt=None, workspace=None, stream=None):
    """The gated recurrence over packed sequences (see ``mamba_mixer_gated_prefill``): with rho = sigmoid(r) and
    iota = sigmoid(g) (g None: 1),

        lam given:  a = exp(-c softplus(lam) rho), m = sqrt(1 - a^2);   lam None:  a = rho, m = 1 - rho
        h = a h + m iota x;   y = h act(z), act the SiLU or the tanh form of GELU by `gate` (z None: y = h)

    x, r, g, z [T, d] io (rows may be strided), lam [d] float32, cu_seqlens [S+1] int32, state_in [S, d] float32 (None:
    zeros).  Returns (y [T, d], state_out [S, d]); pass state_out=state_in to update the states in place.  ckpt
    [ceil(T / GATED_BLOCK), d] float32, if given, takes the states that ``gated_backward`` can start from."""
    lib, T, d, io, strides = _gated_inputs(x, r, g, z, lam, gate)
    S = _sequences(cu_seqlens, T)
    if state_in is not None:
        _need(state_in, (S, d), _h._F32, "state_in")
    state_out = _given(state_out, (S, d), _h._F32, "state_out", x.device, stream)
    y = _given(y, (T, d), x.dtype, "y", x.device, stream)
    if ckpt is not None:
        _need(ckpt, (-(-T // GATED_BLOCK), d), _h._F32, "ckpt")
    need = lib.mamba_mixer_gated_prefill_workspace_bytes(T, d) if workspace is None else 0
    workspace, wptr, wbytes = _workspace(workspace, need, x.device, stream)
    _run("mamba_mixer_gated_prefill", x, (r, g, z, lam, cu_seqlens, state_in, state_out, y, ckpt, workspace), x.data_ptr(),
         r.data_ptr(), _opt(g), _opt(z), _opt(lam), cu_seqlens.data_ptr(), _opt(state_in), state_out.data_ptr(),
         y.data_ptr(), _opt(ckpt), S, T, d, c, GATES[gate], io, *strides, wptr, wbytes, _on(stream, x))
    return y, state_out


def gated_prefill_train(x, r, g, z, lam, cu_seqlens, state_in=None, state_out=None, c: float = 8.0, gate: str = "silu",
                        y=None, ckpt=None, workspace=None, stream=None):
    """``gated_prefill`` as the forward of a training step: returns (y, state_out, ckpt), ckpt for
    ``gated_backward``, which then need not make the states again."""
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    _lib()
    ckpt = _given(ckpt, (-(-x.shape[0] // GATED_BLOCK), x.shape[1]), _h._F32, "ckpt", x.device, stream)
    y, state_out = gated_prefill(x, r, g, z, lam, cu_seqlens, state_in, state_out, c, gate, y, ckpt, workspace, stream)
    return y, state_out, ckpt


def gated_decode(x, r, g, z, lam, state_in=None, state_out=None, c: float = 8.0, gate: str = "silu", y=None, stream=None):
    """One token of the gated recurrence for each of Bs rows (see ``mamba_mixer_gated_decode``): x, r, g, z [Bs, d],
    state_in [Bs, d] float32 (None: zeros).  Returns (y [Bs, d], state_out)."""
    _, Bs, d, io, strides = _gated_inputs(x, r, g, z, lam, gate)
    if state_in is not None:
        _need(state_in, (Bs, d), _h._F32, "state_in")
    state_out = _given(state_out, (Bs, d), _h._F32, "state_out", x.device, stream)
    y = _given(y, (Bs, d), x.dtype, "y", x.device, stream)
    _run("mamba_mixer_gated_decode", x, (r, g, z, lam, state_in, state_out, y), x.data_ptr(), r.data_ptr(), _opt(g), _opt(z),
         _opt(lam), _opt(state_in), state_out.data_ptr(), y.data_ptr(), Bs, d, c, GATES[gate], io, *strides, _on(stream, x))
    return y, state_out


def gated_backward(x, r, g, z, lam, cu_seqlens, state_in, dy, dstate_out=None, ckpt=None, c: float = 8.0,
                   gate: str = "silu", dx=None, dr=None, dg=None, dz=None, need_dstate: bool = True, workspace=None,
                   stream=None) -> dict:
    """The gradients of ``gated_prefill`` (see ``mamba_mixer_gated_backward``) from dy [T, d] and dstate_out [S, d] (None:
    the loss does not depend on the final states); ckpt is what ``gated_prefill_train`` returned for these inputs (None:
    the states are made again).  dx, dr, dg and dz may be given (column ranges of one gradient, for instance).  Returns a
    dict of dx, dr, dg, dz (io), dlam and dstate_in (float32); dg is None without g, dz without z, dlam without lam,
    dstate_in with need_dstate=False."""
    lib, T, d, io, strides = _gated_inputs(x, r, g, z, lam, gate)
    S, dev = _sequences(cu_seqlens, T), x.device
    for t, n in ((state_in, "state_in"), (dstate_out, "dstate_out")):
        if t is not None:
            _need(t, (S, d), _h._F32, n)
    if ckpt is not None:
        _need(ckpt, (-(-T // GATED_BLOCK), d), _h._F32, "ckpt")
    _need(dy, (T, d), x.dtype, "dy")
    one = lambda t, n: _rows_out(t, (T, d), x.dtype, n, dev, stream, d)  # noqa: E731
    (dx, xs), (dr, rs) = one(dx, "dx"), one(dr, "dr")
    dg, gs = one(dg, "dg") if g is not None else (None, 0)
    dz, zs = one(dz, "dz") if z is not None else (None, 0)
    dlam = _new((d,), _h._F32, dev, stream) if lam is not None else None
    dstate_in = _new((S, d), _h._F32, dev, stream) if need_dstate else None
    need = lib.mamba_mixer_gated_backward_workspace_bytes(T, d, 0 if ckpt is None else 1) if workspace is None else 0
    workspace, wptr, wbytes = _workspace(workspace, need, dev, stream)
    _run("mamba_mixer_gated_backward", x, (r, g, z, lam, cu_seqlens, state_in, dy, dstate_out, ckpt, dx, dr, dg, dz, workspace),
         x.data_ptr(), r.data_ptr(), _opt(g), _opt(z), _opt(lam), cu_seqlens.data_ptr(), _opt(state_in), dy.data_ptr(),
         _opt(dstate_out), _opt(ckpt), dx.data_ptr(), dr.data_ptr(), _opt(dg), _opt(dz), _opt(dlam), _opt(dstate_in), S, T, d,
         c, GATES[gate], io, *strides, xs, rs, gs, zs, wptr, wbytes, _on(stream, x))
    return dict(dx=dx, dr=dr, dg=dg, dz=dz, dlam=dlam, dstate_in=dstate_in)


def _qk_inputs(q, k, q_weight, k_weight, positions, inv_freq):
    lib = _lib()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, Hq, D] and k [T, Hk, D]")
    T, Hq, D = q.shape
    Hk = k.shape[1]
    io = _code(q)
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq: both or neither")
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        _need(t, (D,), _h._F32, n)
    R = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [R / 2]")
        R = 2 * inv_freq.shape[0]
        _need(inv_freq, (R // 2,), _h._F32, "inv_freq")
        _need(positions, (T,), _h.torch.int32, "positions")
    return lib, T, Hq, Hk, D, R, io, _rows(q, (T, Hq, D), q.dtype, "q"), _rows(k, (T, Hk, D), q.dtype, "k")


def qk_norm(q, k, q_weight, k_weight, positions=None, inv_freq=None, eps: float = 1e-5, interleaved: bool = False,
            q_out=None, k_out=None, stream=None):
    """The norms of queries and keys, head by head, and their rotation by position (see ``mamba_mixer_qk_norm``): q
    [T, Hq, D], k [T, Hk, D] io (rows may be strided), q_weight, k_weight [D] float32, positions [T] int32, inv_freq
    [R / 2] float32: the first R columns turn, in pairs (k, k + R / 2), or (2 k, 2 k + 1) when interleaved; neither given:
    the norms alone.  Returns (q_out, k_out), which may be given (with strided rows) and may be q and k themselves."""
    _, T, Hq, Hk, D, R, io, qs, ks = _qk_inputs(q, k, q_weight, k_weight, positions, inv_freq)
    dev = q.device
    q_out, qos = _rows_out(q_out, (T, Hq, D), q.dtype, "q_out", dev, stream, Hq * D)
    k_out, kos = _rows_out(k_out, (T, Hk, D), q.dtype, "k_out", dev, stream, Hk * D)
    _run("mamba_mixer_qk_norm", q, (k, q_weight, k_weight, positions, inv_freq, q_out, k_out), q.data_ptr(), k.data_ptr(),
         q_weight.data_ptr(), k_weight.data_ptr(), _opt(positions), _opt(inv_freq), q_out.data_ptr(), k_out.data_ptr(), T,
         Hq, Hk, D, R, eps, 1 if interleaved else 0, io, qs, ks, qos, kos, _on(stream, q))
    return q_out, k_out


def qk_norm_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions=None, inv_freq=None, eps: float = 1e-5,
                     interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """The gradients of ``qk_norm`` from dq_out [T, Hq, D] and dk_out [T, Hk, D]: (dq, dk, dq_weight, dk_weight); dq and dk
    may be given (with strided rows)."""
    lib, T, Hq, Hk, D, R, io, qs, ks = _qk_inputs(q, k, q_weight, k_weight, positions, inv_freq)
    _need(dq_out, (T, Hq, D), q.dtype, "dq_out")
    _need(dk_out, (T, Hk, D), q.dtype, "dk_out")
    dev = q.device
    dq, dqs = _rows_out(dq, (T, Hq, D), q.dtype, "dq", dev, stream, Hq * D)
    dk, dks = _rows_out(dk, (T, Hk, D), q.dtype, "dk", dev, stream, Hk * D)
    dwq, dwk = (_new((D,), _h._F32, dev, stream) for _ in range(2))
    need = lib.mamba_mixer_qk_norm_backward_workspace_bytes(T, Hq, Hk, D) if workspace is None else 0
    workspace, wptr, wbytes = _workspace(workspace, need, dev, stream)
    _run("mamba_mixer_qk_norm_backward", q, (dq_out, dk_out, k, q_weight, k_weight, positions, inv_freq, dq, dk, workspace),
         dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(),
         _opt(positions), _opt(inv_freq), dq.data_ptr(), dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr(), T, Hq, Hk, D, R, eps,
         1 if interleaved else 0, io, qs, ks, dqs, dks, wptr, wbytes, _on(stream, q))
    return dq, dk, dwq, dwk
