"""What the binding allocates for a call on a given stream belongs to that stream: the allocator hands memory on in the
order of the stream it was allocated on, so a workspace of the current stream could be given to its next user while
the call still runs on the other one.  Without a GPU: device tensors, streams and the library's launches are
stand-ins that record what is allocated where."""
from __future__ import annotations

import contextlib
import ctypes

import pytest
import torch

import selective_state_space_causal_amd as mm

F32, BF16 = torch.float32, torch.bfloat16


class OnDevice(torch.Tensor):
    is_cuda = True

    def record_stream(self, stream):
        LOG.used.append((self.data_ptr(), stream))


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Log:
    def __init__(self):
        self.now, self.made, self.used, self.launched = None, [], [], []


LOG = Log()
CURRENT, SIDE = Stream(0x123456789), Stream(0x987654321)


class Library:
    """The library's size queries, and launches that do nothing."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if "workspace" in name or "plan" in name or "name" in name or "bytes" in name:
            return getattr(self.real, name)
        return lambda *a: LOG.launched.append({getattr(v, "value", v) for v in a if not isinstance(v, ctypes.Array)}) or 0


def dev(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture(autouse=True)
def recorded(monkeypatch):
    global LOG
    LOG = Log()
    library = Library(mm.load())
    real = torch.empty

    def empty(*a, **kw):
        t = real(*a, **kw).as_subclass(OnDevice)
        LOG.made.append((t, LOG.now))
        return t

    @contextlib.contextmanager
    def on(stream):
        before, LOG.now = LOG.now, stream
        yield
        LOG.now = before

    monkeypatch.setattr(mm, "_lib", library)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t, dtype=None: empty(t.shape, dtype=dtype or t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: CURRENT)


def cu(T, S=2):
    return torch.tensor([0] + [T] * S, dtype=torch.int32).as_subclass(OnDevice)


def heads(T, H=4, P=64, G=2, N=128):
    return [dev(T, H, P), dev(T, H), dev(T, G, N), dev(T, G, N), dev(H, dtype=F32), dev(H, dtype=F32), dev(H, dtype=F32)]


def heads_prefill(**kw):
    return mm.heads_prefill(*heads(700), cu(700), **kw)


def heads_decode(**kw):
    return mm.heads_decode(*heads(3), **kw)


def heads_backward(**kw):
    return list(mm.heads_backward(*heads(700), cu(700), None, dev(700, 4, 64), **kw).values())


def gate_norm(**kw):
    return [mm.gate_norm(dev(3, 64), dev(3, 64), dev(64, dtype=F32), **kw)]


def gate_norm_backward(**kw):
    return mm.gate_norm_backward(dev(3, 64), dev(3, 64), dev(3, 64), dev(64, dtype=F32), **kw)


def residual_norm(**kw):
    return mm.residual_norm(dev(3, 64), None, dev(64, dtype=F32), **kw)


def residual_norm_backward(**kw):
    w = dev(64, dtype=F32)
    return list(mm.residual_norm_backward(dev(3, 64), None, dev(3, 64), dev(3, 64), w, w, scale_vec=w, **kw).values())


def mixer(T=600, S=2, d=64, N=16, states=True):
    """x, z, dt, B, C, the parameters, cu_seqlens and the states of the selective scan's calls."""
    return [dev(T, d), dev(T, d), dev(T, d), dev(T, N), dev(T, N), dev(d, N, dtype=F32), dev(d, dtype=F32), dev(d, dtype=F32),
            dev(d, 4, dtype=F32), dev(d, dtype=F32), cu(T, S), dev(S, d, 3, dtype=F32), dev(S, d, N, dtype=F32)]


def ring(W, Bs, d=64, N=16):
    p = mixer(Bs, Bs)
    return [dev(W, Bs, d), dev(W, Bs, d), dev(W, Bs, N)], [dev(Bs, d), dev(Bs, N)], p[5:10], p[11:]


def prefill(**kw):
    return [mm.prefill(*mixer(), chunk_len=64, **kw)]


def prefill_noalloc(**kw):
    return [mm.prefill_noalloc(*mixer(), **kw)]


def prefill_train(**kw):
    return mm.prefill_train(*mixer(), chunk_len=64, **kw)


def prefill_backward(**kw):
    return list(mm.prefill_backward(*mixer(), dev(600, 64), **kw).values())


def project(**kw):
    p = mixer()
    return mm.project(p[0], p[8], p[9], p[10], p[11], dev(64, 8 + 32), dev(8, 64), **kw)


def decode(**kw):
    p = mixer(3, 3)
    return [mm.decode(*p[:10], *p[11:], **kw)]


def decode_replay(**kw):
    rings, now, params, states = ring(4, 3)
    return [mm.decode_replay(*rings, *now, *params, *states, 1, **kw)]


def replay_checkpoint_lo(**kw):
    return mm.replay_checkpoint_lo(*ring(4, 3)[3], **kw)


def decode_replay_dual(**kw):
    rings, now, params, states = ring(4, 3)
    return [mm.decode_replay_dual(*rings, *now, *params, *states, dev(3, 64, 4), dev(3, 64, 16), 1, **kw)]


def decode_replay_multi(**kw):
    rings, _, params, states = ring(4, 3)
    return [mm.decode_replay_multi(*rings, dev(4, 3, 64), dev(4, 3, 16), *params, *states, 0, 1, **kw)]


CALLS = [heads_prefill, heads_decode, heads_backward, gate_norm, gate_norm_backward, residual_norm, residual_norm_backward,
         prefill, prefill_noalloc, prefill_train, prefill_backward, project, decode, decode_replay, replay_checkpoint_lo,
         decode_replay_dual, decode_replay_multi]
WITH_WORKSPACE = (heads_prefill, heads_backward, gate_norm_backward, residual_norm_backward, prefill, prefill_train,
                  prefill_backward, project)


@pytest.mark.parametrize("call", CALLS, ids=[c.__name__ for c in CALLS])
def test_allocations_belong_to_the_given_stream(call):
    outputs = [t for t in call(stream=SIDE) if t is not None]
    assert len(LOG.launched) == 1 and SIDE.cuda_stream in LOG.launched[0]
    assert LOG.made and all(stream is SIDE for _, stream in LOG.made)
    assert len(LOG.made) == len(outputs) + (call in WITH_WORKSPACE)
    used = {p for p, stream in LOG.used if stream is CURRENT}
    assert used == {t.data_ptr() for t in outputs}, "the current stream will use the outputs, and they alone"


@pytest.mark.parametrize("call", CALLS, ids=[c.__name__ for c in CALLS])
def test_allocations_of_a_call_on_the_current_stream(call, monkeypatch):
    import selective_state_space_causal_amd.heads as binding

    monkeypatch.setattr(binding, "_raw_stream", lambda index: CURRENT.cuda_stream)
    call()
    assert LOG.made and all(stream is None for _, stream in LOG.made) and not LOG.used
