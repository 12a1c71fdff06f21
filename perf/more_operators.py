"""The measured cases of the causal convolution, the gated recurrence and the head norm with its rotation: their inputs,
their plain forms in torch, and the calls a user makes of the library.

Symbols: T tokens in S packed sequences, d channels, a convolution of W taps; Hq query and Hk key heads of D columns,
rotated in their first R.  Where a user has column ranges of a projection's output in hand, so do these: their rows are
strided."""
import math

import torch

own = False

EPS = 1e-5
C = 8.0  # the recurrence's log decay is -C softplus(lam) sigmoid(r)


# ------------------------------------------------------------------------------------------------ cases
def listed():
    packed = "425,3261,647,3703,4011,2536,1801"  # lengths U[128, 4096] to 16384 tokens
    train = ",".join(["2048"] * 8)
    return [
        # a packed prompt batch through a 1.4B-shaped layer: x | B | C of d_inner 4096, one group of 128
        dict(name="conv prefill 16384x4352", op="conv", lens=packed, d=4352, W=4, silu=True, bias=True, io="bf16"),
        # one token of one chat: latency
        dict(name="conv decode 1x4096", op="conv_decode", rows=1, d=4096, W=4, silu=True, bias=True, io="bf16"),
        # a training step's backward of a 130m-shaped layer (d_inner 1536 and B, C of 128)
        dict(name="conv backward 8x2048x1792", op="conv_backward", lens=train, d=1792, W=4, silu=True, bias=True,
             io="bf16"),
        # a packed prompt batch through a recurrent layer of d_inner 4096
        dict(name="gated prefill 16384x4096", op="gated", lens=packed, d=4096, lam=True, g=True, gate="gelu", io="bf16"),
        # one long prompt through a layer as wide as a 2.8B-shaped model: one sequence, a long axis
        dict(name="gated prefill 32768x2560", op="gated", lens="32768", d=2560, lam=True, g=True, gate="gelu",
             io="bf16"),
        # short ragged float32 sequences (empty and one-token ones among them), odd sizes, gates that add up to one
        dict(name="gated prefill ragged f32", op="gated", lens="1,0,63,200,5,129,0,379", d=250, lam=False, g=False,
             gate="silu", io="f32"),
        # a full serving batch, one token each, d_inner 8192
        dict(name="gated decode 256x8192", op="gated_decode", rows=256, d=8192, lam=True, g=True, gate="gelu", io="bf16"),
        # a training step of a 130m-shaped layer: forward, then backward
        dict(name="gated train 8x2048x1536", op="gated_train", lens=train, d=1536, lam=True, g=True, gate="gelu",
             io="bf16"),
        # gradients of short ragged float32 sequences with nothing kept from the forward, odd sizes
        dict(name="gated backward ragged f32", op="gated_backward", lens="1,65,0,190,133", d=250, lam=True, g=True,
             gate="none", io="f32"),
        # queries and keys of a packed prompt batch: C and B of a head scan, eight groups of 128
        dict(name="qk_norm 16384 8+8x128", op="qk", lens=packed, Hq=8, Hk=8, D=128, R=128, inter=False, io="bf16"),
        # one token of one chat: latency
        dict(name="qk_norm 1 8+8x128", op="qk", lens="1", Hq=8, Hk=8, D=128, R=128, inter=False, io="bf16"),
        # a training step's backward, 24 heads of 64 with as many keys, half of the columns rotated in neighbouring pairs
        dict(name="qk_norm backward 8x2048 24x64", op="qk_backward", lens=train, Hq=24, Hk=24, D=64, R=32, inter=True,
             io="bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm, not a multiple of three (so odd ones are common)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    v = max(lo, min(hi, v))
    return v if v % 3 else v + 1 if v < hi else v - 1


def _draw_lens(rng, T):
    S = min(T, rng.choice([1, 2, 3, 5, 8, 16, 40]))
    cuts = sorted(rng.randint(0, T) for _ in range(S - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["conv", "conv_decode", "conv_backward", "gated", "gated_decode", "gated_train", "gated_backward",
                     "qk", "qk_backward"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("qk"):
        D = rng.choice([16, 32, 40, 64, 64, 80, 96, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 1, 2, 3, 4])
        T = _log_int(rng, 1, min(16384, 16384 * 48 * 64 // ((Hq + Hk) * D * (1 if io == "bf16" else 2))))
        return dict(op=op, lens=_draw_lens(rng, T), Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D, D // 2 & ~1, 0]),
                    inter=rng.random() < 0.5, io=io)
    d = _log_int(rng, 16, 5120)
    if op.startswith("conv"):
        c = dict(op=op, d=d, W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, bias=rng.random() < 0.7, io=io)
    else:
        lam = rng.random() < 0.7
        c = dict(op=op, d=d, lam=lam, g=rng.random() < (0.8 if lam else 0.3), gate=rng.choice(["none", "silu", "gelu"]),
                 io=io)
    if op.endswith("decode"):
        return dict(c, rows=_log_int(rng, 1, 256))
    most = dict(conv=16384 * 4352, gated=32768 * 2560).get(op, 8 * 2048 * 1536)
    T = _log_int(rng, 1, min(32768, most // d // (1 if io == "bf16" else 2)))
    return dict(c, lens=_draw_lens(rng, T))


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def work(case):
    """Bytes: every input read once, every output written once.  Operations: per element, the exponential-class ones
    counted as one."""
    e, op = (2 if case["io"] == "bf16" else 4), case["op"]
    T = case["rows"] if op.endswith("decode") else sum(_lens(case))
    S = case["rows"] if op.endswith("decode") else len(_lens(case))
    if op.startswith("qk"):
        n = T * (case["Hq"] + case["Hk"]) * case["D"]
        back = op == "qk_backward"
        return dict(bytes=n * e * (3 if back else 2) + T * 4 + (4 if back else 2) * case["D"] * 4, flops=n * (16 if back else 8))
    d = case["d"]
    n = T * d
    if op.startswith("conv"):
        W = case["W"]
        back = op == "conv_backward"
        return dict(bytes=n * e * (3 if back else 2) + (3 if back else 2) * S * d * (W - 1) * 4 + (2 if back else 1) * d * (W + 1) * 4,
                    flops=n * (2 * W + 6) * (3 if back else 1))
    ins = 2 + case["g"] + (case["gate"] != "none")  # x, r, g, z
    forward = dict(bytes=n * e * (ins + 1) + 2 * S * d * 4 + 4 * d, flops=n * 20)
    back = dict(bytes=n * e * (2 * ins + 1) + 3 * S * d * 4 + 8 * d, flops=n * 60)
    if op == "gated_train":
        return {k: forward[k] + back[k] for k in forward}
    return back if op == "gated_backward" else forward


# ----------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    io, op = (torch.bfloat16 if case["io"] == "bf16" else torch.float32), case["op"]
    lens = [1] * case["rows"] if op.endswith("decode") else _lens(case)
    T, S = sum(lens), len(lens)
    st = dict(case=case, lens=lens)
    st["cu"] = torch.tensor([sum(lens[:i]) for i in range(S + 1)], dtype=torch.int32, device="cuda")
    if op.startswith("qk"):
        Hq, Hk, D, R = (case[k] for k in ("Hq", "Hk", "D", "R"))
        proj = randn(T, (Hq + 2 * Hk) * D).to(io)  # queries | keys | values
        st["q"] = proj[:, :Hq * D].unflatten(1, (Hq, D))
        st["k"] = proj[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        st["wq"], st["wk"] = 1.0 + 0.1 * randn(D), 1.0 + 0.1 * randn(D)
        # each sequence continues at a place of its own, up to a million tokens in
        at = (rand(S) * (1 << 20)).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(lens, device="cuda"), output_size=T)
        st["pos"] = at[seq] + torch.arange(T, dtype=torch.int32, device="cuda") - st["cu"][seq]
        st["freq"] = 10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=torch.float32) * 2 / max(R, 1))
        if R == 0:
            st["pos"] = st["freq"] = None
        if op == "qk_backward":
            st["dq"], st["dk"] = randn(T, Hq, D).to(io), randn(T, Hk, D).to(io)
        return st
    d = case["d"]
    if op.startswith("conv"):
        W = case["W"]
        st["x"] = randn(T, 2 * d).to(io)[:, d:]  # beside the gate in a projection's output
        st["weight"] = (rand(d, W) - 0.5) * 2 * W ** -0.5
        st["bias"] = (rand(d) - 0.5) if case["bias"] else None
        st["state"] = randn(S, d, W - 1)
        if op == "conv_backward":
            st["dy"], st["dstate"] = randn(T, d).to(io), randn(S, d, W - 1)
        return st
    # x out of a convolution; r and g out of one product of gates; z beside x in the input projection
    st["x"] = randn(T, d).to(io)
    gates = randn(T, 2 * d)
    if not case["lam"]:
        gates[:, :d] += 2.0  # decays around 0.9: sigmoid(r) is the decay itself
    gates = gates.to(io)
    st["r"], st["g"] = gates[:, :d], gates[:, d:] if case["g"] else None
    st["z"] = randn(T, 2 * d).to(io)[:, :d] if case["gate"] != "none" else None
    far = 0.9 + 0.099 * rand(d)  # the decay of a fully open gate
    st["lam"] = torch.log(torch.expm1(-torch.log(far) / C)) if case["lam"] else None
    st["state"] = randn(S, d)
    if op in ("gated_train", "gated_backward"):
        st["dy"], st["dstate"] = randn(T, d).to(io), randn(S, d)
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _f(v):
    return v.float() if v is not None else None


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _places(st):
    """For each token the sequence it is in and its place there."""
    cu, T = st["cu"].long(), sum(st["lens"])
    seq = torch.repeat_interleave(torch.arange(len(st["lens"]), device=cu.device), cu[1:] - cu[:-1], output_size=T)
    return seq, torch.arange(T, device=cu.device) - cu[seq]


def _windows(st, W):
    """The W raw inputs under each token's taps, oldest first: [W][T, d]; and where they are in [x; state's rows]."""
    seq, place = _places(st)
    T, d = st["x"].shape
    # all raw inputs: the tokens', then each sequence's W - 1 older ones
    raw = torch.cat([st["x"].float(), st["state"].transpose(1, 2).reshape(-1, d)])
    token = torch.arange(T, device=raw.device)
    at = [torch.where(place >= back, token - back, T + seq * (W - 1) + (W - 1) + place - back) for back in range(W - 1, -1, -1)]
    return raw, at


def _last(st, W):
    """Where each sequence's newest W - 1 raw inputs are in [x; state's rows], oldest first: [S, W - 1]."""
    cu, T, S = st["cu"].long(), st["x"].shape[0], len(st["lens"])
    back = torch.arange(W - 1, 0, -1, device=cu.device)
    n = (cu[1:] - cu[:-1])[:, None]
    s = torch.arange(S, device=cu.device)[:, None]
    return torch.where(n >= back, cu[1:, None] - back, T + s * (W - 1) + (W - 1) + n - back)


def _plain_conv(st):
    W, w = st["case"]["W"], st["weight"]
    raw, at = _windows(st, W)
    u = sum(raw[a] * w[:, k] for k, a in enumerate(at)) + (st["bias"] if st["bias"] is not None else 0.0)
    y = u * _sigmoid(u) if st["case"]["silu"] else u
    return y.to(st["x"].dtype), raw[_last(st, W)].transpose(1, 2).contiguous()


def _plain_conv_backward(st):
    W, w, (T, d) = st["case"]["W"], st["weight"], st["x"].shape
    raw, at = _windows(st, W)
    g = st["dy"].float()
    if st["case"]["silu"]:
        u = sum(raw[a] * w[:, k] for k, a in enumerate(at)) + (st["bias"] if st["bias"] is not None else 0.0)
        s = _sigmoid(u)
        g = g * s * (1.0 + u * (1.0 - s))
    draw_ = torch.zeros_like(raw)
    for k, a in enumerate(at):  # no place is twice in one `a`
        draw_[a] += g * w[:, k]
    for k in range(W - 1):
        draw_[_last(st, W)[:, k]] += st["dstate"][:, :, k]
    dw = torch.stack([(g * raw[a]).sum(0) for a in at], 1)
    out = dict(dx=draw_[:T].to(st["x"].dtype), dweight=dw, dstate=draw_[T:].unflatten(0, (-1, W - 1)).transpose(1, 2))
    if st["bias"] is not None:
        out["dbias"] = g.sum(0)
    return out


def _decay(st):
    """rho, iota, log a, a, m and their factors for the gated recurrence."""
    rho = _sigmoid(_f(st["r"]))
    iota = _sigmoid(_f(st["g"])) if st["g"] is not None else torch.ones((), device=rho.device)
    if st["lam"] is None:
        return rho, iota, None, rho, _sigmoid(-_f(st["r"]))
    L = -C * _softplus(st["lam"]) * rho
    return rho, iota, L, torch.exp(L), torch.sqrt(-torch.expm1(2.0 * L))


def _act(z, kind):
    """The output gate and its derivative: z sigmoid(k), k = z or GELU's tanh form."""
    c0, c1 = (1.0, 0.0) if kind == "silu" else (2.0 * math.sqrt(2.0 / math.pi), 2.0 * math.sqrt(2.0 / math.pi) * 0.044715)
    s = _sigmoid(z * (c0 + c1 * z * z))
    return z * s, s + z * s * (1.0 - s) * (c0 + 3.0 * c1 * z * z)


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the rows, in log2(longest) steps (a is 0 where a sequence starts)."""
    a, h, k = a.clone(), b.clone(), 1
    while k < longest:
        h[k:] = h[k:] + a[k:] * h[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return h


def _states(st, a, b):
    """h of every token, h before it, and the sequences' final states."""
    cu = st["cu"].long()
    there = cu[1:] > cu[:-1]
    first, last = cu[:-1][there], cu[1:][there] - 1
    a2, b2 = a.clone(), b.clone()
    b2[first] += a2[first] * st["state"][there]
    a2[first] = 0.0
    h = _scan(a2, b2, max(st["lens"]))
    before = torch.cat([h[:1], h[:-1]]) if len(h) else h.clone()
    before[first] = st["state"][there]
    final = st["state"].clone()
    final[there] = h[last]
    return h, before, final


def _plain_gated(st):
    c = st["case"]
    _, iota, _, a, m = _decay(st)
    h, _, final = _states(st, a, m * iota * st["x"].float())
    y = h if st["z"] is None else h * _act(st["z"].float(), c["gate"])[0]
    return y.to(st["x"].dtype), final


def _plain_gated_backward(st):
    c, cu = st["case"], st["cu"].long()
    rho, iota, L, a, m = _decay(st)
    x = st["x"].float()
    u = iota * x
    h, before, _ = _states(st, a, m * u)
    dh, out = st["dy"].float(), {}
    if st["z"] is not None:
        act, dact = _act(st["z"].float(), c["gate"])
        out["dz"] = (dh * h * dact).to(st["z"].dtype)
        dh = dh * act
    there = cu[1:] > cu[:-1]
    first, last = cu[:-1][there], cu[1:][there] - 1
    dh = dh.clone()
    dh[last] += st["dstate"][there]
    after = torch.cat([a[1:], a[:1]]) if len(a) else a.clone()  # the decay of the next token
    after[last] = 0.0
    G = _scan(after.flip(0), dh.flip(0), max(st["lens"])).flip(0)
    dstate = st["dstate"].clone()
    dstate[there] = a[first] * G[first]
    out["dstate"] = dstate
    out["dx"] = (G * m * iota).to(st["x"].dtype)
    if st["g"] is not None:
        out["dg"] = (G * m * x * iota * (1.0 - iota)).to(st["g"].dtype)
    if L is None:
        out["dr"] = (G * (before - u) * rho * (1.0 - rho)).to(st["r"].dtype)
    else:
        # the gradient of log a, times log a; dm / d(log a) = -a^2 / m, and log a / m -> 0 with log a
        dL = G * (a * before * L - u * a * a * torch.where(L < 0, L / m, 0.0))
        out["dr"] = (dL * (1.0 - rho)).to(st["r"].dtype)
        out["dlam"] = dL.sum(0) * _sigmoid(st["lam"]) / _softplus(st["lam"])
    return out


def _plain_gated_train(st):
    y, final = _plain_gated(st)
    return dict(_plain_gated_backward(st), y=y, final=final)


def _angles(st):
    """cos and sin, [T, 1, R / 2]: the angles in 64 bits."""
    ang = st["pos"].double()[:, None, None] * st["freq"].double()
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(v, cos, sin, R, inter):
    a, b = (v[..., :R:2], v[..., 1:R:2]) if inter else (v[..., :R // 2], v[..., R // 2:R])
    p, q = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([p, q], -1).flatten(-2) if inter else torch.cat([p, q], -1), v[..., R:]], -1)


def _plain_qk(st):
    c = st["case"]
    out = []
    for v, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        f = v.float()
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
        out.append((_rotate(f, *_angles(st), c["R"], c["inter"]) if c["R"] else f).to(v.dtype))
    return out


def _plain_qk_backward(st):
    c = st["case"]
    got = []
    for v, w, do in ((st["q"], st["wq"], st["dq"]), (st["k"], st["wk"], st["dk"])):
        f, g = v.float(), do.float()
        if c["R"]:
            cos, sin = _angles(st)
            g = _rotate(g, cos, -sin, c["R"], c["inter"])
        r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        n = f * r
        dn = g * w
        got.append(((r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(v.dtype), (g * n).sum((0, 1))))
    return [got[0][0], got[1][0], got[0][1], got[1][1]]


PLAIN = dict(conv=_plain_conv, conv_decode=_plain_conv, conv_backward=_plain_conv_backward, gated=_plain_gated,
             gated_decode=_plain_gated, gated_train=_plain_gated_train, gated_backward=_plain_gated_backward,
             qk=_plain_qk, qk_backward=_plain_qk_backward)


# ------------------------------------------------------------------------------------- the library's calls
def _own(st):
    import selective_state_space_causal_amd as mm

    c = st["case"]
    op = c["op"]
    if op.startswith("qk"):
        rest = dict(positions=st["pos"], inv_freq=st["freq"], eps=EPS, interleaved=c["inter"])
        if op == "qk":
            return mm.qk_norm(st["q"], st["k"], st["wq"], st["wk"], **rest)
        return mm.qk_norm_backward(st["dq"], st["dk"], st["q"], st["k"], st["wq"], st["wk"], **rest)
    if op.startswith("conv"):
        ins = (st["x"], st["weight"], st["bias"])
        if op == "conv":
            return mm.conv_prefill(*ins, st["cu"], st["state"], silu=c["silu"])
        if op == "conv_decode":
            return mm.conv_decode(*ins, st["state"], silu=c["silu"])
        g = mm.conv_backward(*ins, st["cu"], st["state"], st["dy"], st["dstate"], silu=c["silu"])
        out = dict(dx=g["dx"], dweight=g["dweight"], dstate=g["dstate_in"])
        return dict(out, dbias=g["dbias"]) if c["bias"] else out
    ins = (st["x"], st["r"], st["g"], st["z"], st["lam"])
    rest = dict(c=C, gate="silu" if c["gate"] == "none" else c["gate"])
    if op == "gated":
        return mm.gated_prefill(*ins, st["cu"], st["state"], **rest)
    if op == "gated_decode":
        return mm.gated_decode(*ins, st["state"], **rest)
    out, kept = {}, None
    if op == "gated_train":
        out["y"], out["final"], kept = mm.gated_prefill_train(*ins, st["cu"], st["state"], **rest)
    g = mm.gated_backward(*ins, st["cu"], st["state"], st["dy"], st["dstate"], ckpt=kept, **rest)
    out.update({k: v for k, v in g.items() if k != "dstate_in" and v is not None}, dstate=g["dstate_in"])
    return out


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------- 64-bit references
def _padded(v, lens, before=0):
    out = v.new_zeros((len(lens), before + max(lens)) + v.shape[1:], dtype=torch.float64)
    at = 0
    for s, n in enumerate(lens):
        out[s, before:before + n] = v[at:at + n]
        at += n
    return out


def _packed(v, lens):
    return torch.cat([v[s, :n] for s, n in enumerate(lens)])


def _exact_conv(st, lens):
    """The definition, sequence by sequence; the gradients through torch's differentiation of it."""
    W, back = st["case"]["W"], st["case"]["op"] == "conv_backward"
    leaves = [v.double().requires_grad_(back) for v in (st["x"], st["state"], st["weight"])]
    x, state, w = leaves
    b = (st["bias"] if st["bias"] is not None else torch.zeros_like(w[:, 0])).double().requires_grad_(back)
    ys, last, at = [], [], 0
    for s, n in enumerate(lens):
        X = torch.cat([state[s].T, x[at:at + n]])
        at += n
        u = b + sum(X[k:k + n] * w[:, k] for k in range(W))
        ys.append(u * torch.sigmoid(u) if st["case"]["silu"] else u)
        last.append(X[n:].T)
    y, last = torch.cat(ys), torch.stack(last)
    if not back:
        return y, last
    dx, ds, dw, db = torch.autograd.grad((y, last), (x, state, w, b), (st["dy"].double(), st["dstate"].double()))
    out = dict(dx=dx, dstate=ds, dweight=dw)
    return dict(out, dbias=db) if st["bias"] is not None else out


def _exact_gated(st, lens, back):
    """The recurrence token after token and its adjoint from the end."""
    leaf = lambda k: _padded(st[k].double(), lens).requires_grad_(back) if st[k] is not None else None  # noqa: E731
    kind = st["case"]["gate"]
    x, r, g, z = (leaf(k) for k in "xrgz")
    lam = st["lam"].double().requires_grad_(back) if st["lam"] is not None else None
    there = (torch.arange(max(lens), device=x.device) < torch.tensor(lens, device=x.device)[:, None])[..., None]
    rho = torch.sigmoid(r)
    if lam is None:
        a, m = rho, torch.sigmoid(-r)
    else:
        L = -C * torch.logaddexp(lam, torch.zeros_like(lam)) * rho
        a, m = torch.exp(L), torch.sqrt(-torch.expm1(2 * L))
    b = m * x * (torch.sigmoid(g) if g is not None else 1.0)
    A, Bv = torch.where(there, a, 1.0).detach(), torch.where(there, b, 0.0).detach()
    h, hs = st["state"].double(), []
    for t in range(max(lens)):
        h = A[:, t] * h + Bv[:, t]
        hs.append(h)
    hs = torch.stack(hs, 1)
    act = 1.0
    if z is not None:
        act = torch.nn.functional.silu(z) if kind == "silu" else torch.nn.functional.gelu(z, approximate="tanh")
    got = dict(y=_packed((hs * act).detach(), lens), final=h)
    if not back:
        return got
    dy = _padded(st["dy"].double(), lens)
    dh = (dy * act).detach() if z is not None else dy
    G, Gs = st["dstate"].double(), []
    for t in reversed(range(max(lens))):
        G = G + dh[:, t]
        Gs.append(G)
        G = A[:, t] * G
    Gs = torch.where(there, torch.stack(Gs[::-1], 1), 0.0)
    before = torch.cat([st["state"].double()[:, None], hs[:, :-1]], 1)
    leaves = {k: v for k, v in dict(dx=x, dr=r, dg=g, dlam=lam).items() if v is not None}
    grads = dict(zip(leaves, torch.autograd.grad((a, b), list(leaves.values()), (Gs * before, Gs))))
    if z is not None:
        grads["dz"] = torch.autograd.grad(act, z, dy * hs)[0]
    got.update({k: v if k == "dlam" else _packed(v, lens) for k, v in grads.items()}, dstate=G)
    return got


def _exact_qk(st, back):
    """The norm by its definition and the rotation as a product of complex numbers; gradients by torch."""
    c = st["case"]
    R, outs = c["R"], []
    for v, w, do in ((st["q"], st["wq"], st.get("dq")), (st["k"], st["wk"], st.get("dk"))):
        v, w = v.double().requires_grad_(back), w.double().requires_grad_(back)
        n = v / torch.sqrt((v ** 2).mean(-1, keepdim=True) + EPS) * w
        if R:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=v.device), st["pos"].double()[:, None] * st["freq"].double())
            pairs = n[..., :R].unflatten(-1, (R // 2, 2)) if c["inter"] else n[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
            n = torch.cat([(pairs if c["inter"] else pairs.transpose(-1, -2)).flatten(-2), n[..., R:]], -1)
        outs.append(torch.autograd.grad(n, (v, w), do.double()) if back else n)
    return [outs[0][0], outs[1][0], outs[0][1], outs[1][1]] if back else outs


def exact(case, seed):
    st = prepare(case, seed)
    lens, op = st["lens"], case["op"]
    if op.startswith("qk"):
        return _exact_qk(st, op == "qk_backward")
    if op.startswith("conv"):
        return _exact_conv(st, lens)
    got = _exact_gated(st, lens, op in ("gated_train", "gated_backward"))
    if op in ("gated", "gated_decode"):
        return got["y"], got["final"]
    if op == "gated_backward":
        del got["y"], got["final"]
    return got
