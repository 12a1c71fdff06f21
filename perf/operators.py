"""The measured cases of the head scan (linear attention with a decay for each head), the gated norm and the
residual norm: their inputs, their plain forms in torch, and the calls a user makes of the library.

Symbols: T tokens in S packed sequences, H heads of P channels, G groups of N-wide B and C vectors (H / G heads
share one), d = H P.  x, z, B, C and dt are column ranges of one projection output [T, z | x | B | C | dt], as an
input projection leaves them, so their rows are strided."""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 128  # tokens per chunk of the plain chunked scan


# ------------------------------------------------------------------------------------------------ cases
def listed():
    packed = "425,3261,647,3703,4011,2536,1801"  # lengths U[128, 4096] to 16384 tokens
    return [
        # a packed prompt batch through a 1.4B-shaped layer (d_inner 4096), one B/C group
        dict(name="prefill packed 16384 d4096", op="prefill", lens=packed, H=64, P=64, G=1, N=128, io="bf16"),
        # one long prompt through a 2.8B-shaped layer (d_inner 5120), eight groups: few sequences, long axis
        dict(name="prefill long 32768 d5120", op="prefill", lens="32768", H=80, P=64, G=8, N=128, io="bf16"),
        # short ragged float32 sequences (empty and one-token ones among them), odd sizes
        dict(name="prefill ragged f32", op="prefill", lens="1,0,63,200,5,129,0,379", H=6, P=40, G=3, N=24, io="f32"),
        # one sequence, one token: the latency of a chat's decode step
        dict(name="decode 1 d4096", op="decode", rows=1, H=64, P=64, G=1, N=128, io="bf16"),
        # a full serving batch through a 7B-shaped layer (d_inner 8192): streaming the states
        dict(name="decode 256 d8192", op="decode", rows=256, H=128, P=64, G=8, N=128, io="bf16"),
        # a training step of a 130m-shaped layer (d_inner 1536)
        dict(name="backward 8x2048 d1536", op="backward", lens=",".join(["2048"] * 8), H=24, P=64, G=1, N=128,
             io="bf16"),
        # gradients of short ragged float32 sequences, odd sizes
        dict(name="backward ragged f32", op="backward", lens="1,65,0,190,133", H=6, P=40, G=3, N=24, io="f32"),
        # the gate and norm after the scan of a packed prompt batch
        dict(name="gate_norm 16384x4096", op="gate_norm", rows=16384, d=4096, groups=1, gate_first=True, io="bf16"),
        # its training backward with eight groups, the gate after the norm
        dict(name="gate_norm backward 8192x5120", op="gate_norm_backward", rows=8192, d=5120, groups=8,
             gate_first=False, io="bf16"),
        # one token between two blocks: latency
        dict(name="residual_norm 1x2048", op="residual_norm", rows=1, d=2048, post=True, vec=True, io="bf16",
             res="f32"),
        # a prompt batch between two blocks, float32 residual stream, norms before and after the block
        dict(name="residual_norm 16384x2048", op="residual_norm", rows=16384, d=2048, post=True, vec=True, io="bf16",
             res="f32"),
        # its training backward at a 2.8B-shaped model width
        dict(name="residual_norm backward 8191x2560", op="residual_norm_backward", rows=8191, d=2560, post=True,
             vec=True, io="bf16", res="f32"),
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm, not a multiple of three (so odd ones are common)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    v = max(lo, min(hi, v))
    return v if v % 3 else v + 1 if v < hi else v - 1


def _draw_heads(rng):
    G = rng.choice([1, 1, 2, 4, 8])
    H = G * rng.choice([1, 2, 4, 5, 7, 8, 10])
    return dict(H=H, P=rng.choice([16, 20, 32, 40, 64, 64, 80, 128]), G=G, N=rng.choice([16, 20, 32, 50, 64, 100, 128, 128]),
                io=rng.choice(["bf16", "bf16", "bf16", "f32"]))


def _draw_lens(rng, T):
    S = min(T, rng.choice([1, 2, 3, 5, 8, 16]))
    cuts = sorted(rng.randint(0, T) for _ in range(S - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))


def draw(rng):
    op = rng.choice(["prefill", "decode", "backward", "gate_norm", "gate_norm_backward", "residual_norm",
                     "residual_norm_backward"])
    if op == "prefill":
        return dict(op=op, lens=_draw_lens(rng, _log_int(rng, 1, 16384)), **_draw_heads(rng))
    if op == "backward":
        c = _draw_heads(rng)
        most = min(16384, 16384 * 24 * 64 * 128 // (c["H"] * c["P"] * c["N"]))
        return dict(op=op, lens=_draw_lens(rng, _log_int(rng, 1, most)), **c)
    if op == "decode":
        return dict(op=op, rows=_log_int(rng, 1, 256), **_draw_heads(rng))
    io = rng.choice(["bf16", "bf16", "f32"])
    rows = _log_int(rng, 1, 8192)
    if op.startswith("gate_norm"):
        groups = rng.choice([1, 1, 2, 4, 8])
        return dict(op=op, rows=rows, d=groups * _log_int(rng, 16, 8192 // groups), groups=groups,
                    gate_first=rng.random() < 0.5, io=io)
    return dict(op=op, rows=rows, d=_log_int(rng, 64, 8192), post=rng.random() < 0.5, vec=rng.random() < 0.5, io=io,
                res=rng.choice(["f32", io]))


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def work(case):
    """Bytes: every input read once, every output written once.  Operations: those of the recurrence (the state's
    update and its readout, 2 P N each per token and head), three times that for the gradients; about ten per
    element for the norms."""
    e = 2 if case["io"] == "bf16" else 4
    if case["op"] in ("prefill", "decode", "backward"):
        H, P, G, N = (case[k] for k in "HPGN")
        T = case["rows"] if case["op"] == "decode" else sum(_lens(case))
        S = case["rows"] if case["op"] == "decode" else len(_lens(case))
        state, token = S * H * P * N * 4, H * P + H + 2 * G * N
        if case["op"] == "backward":
            return dict(bytes=T * e * (2 * token + H * P) + 3 * state + 24 * H, flops=12.0 * T * H * P * N)
        return dict(bytes=T * e * (token + H * P) + 2 * state + 12 * H, flops=4.0 * T * H * P * N)
    n, d = case["rows"] * case["d"], case["d"]
    if case["op"] == "gate_norm":
        return dict(bytes=3 * n * e + 4 * d, flops=10 * n)
    if case["op"] == "gate_norm_backward":
        return dict(bytes=5 * n * e + 8 * d, flops=25 * n)
    f = 4 if case["res"] == "f32" else 2
    if case["op"] == "residual_norm":
        return dict(bytes=n * (2 * e + 2 * f) + 12 * d, flops=12 * n)
    return dict(bytes=n * (3 * e + 3 * f) + 24 * d, flops=30 * n)


# ----------------------------------------------------------------------------------------------- inputs
def _dtype(io):
    return torch.bfloat16 if io == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    io = _dtype(case["io"])
    st = dict(case=case)
    if case["op"] in ("prefill", "decode", "backward"):
        H, P, G, N = (case[k] for k in "HPGN")
        lens = [1] * case["rows"] if case["op"] == "decode" else _lens(case)
        T, S, d = sum(lens), len(lens), H * P
        proj = randn(T, 2 * d + 2 * G * N + H)
        proj[:, 2 * d:2 * d + 2 * G * N] *= N ** -0.25  # so that C . B is about N(0, 1)
        proj = proj.to(io)
        st["lens"] = lens
        st["cu"] = torch.tensor([sum(lens[:i]) for i in range(S + 1)], dtype=torch.int32, device="cuda")
        st["x"] = proj[:, d:2 * d].unflatten(1, (H, P))
        st["B"] = proj[:, 2 * d:2 * d + G * N].unflatten(1, (G, N))
        st["C"] = proj[:, 2 * d + G * N:2 * d + 2 * G * N].unflatten(1, (G, N))
        st["dt"] = proj[:, 2 * d + 2 * G * N:]
        st["A_log"] = torch.log(1.0 + 15.0 * rand(H))
        dt0 = torch.exp(math.log(1e-3) + (math.log(0.1) - math.log(1e-3)) * rand(H))
        st["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))  # the inverse of softplus at dt0
        st["D"] = 1.0 + 0.1 * randn(H)
        st["state"] = 0.5 * randn(S, H, P, N)
        if case["op"] == "backward":
            st["dy"] = randn(T, H, P).to(io)
            st["dstate"] = 0.5 * randn(S, H, P, N)  # of the final state: a later part of the sequence asks for it
        return st
    rows, d = case["rows"], case["d"]
    st["weight"] = 1.0 + 0.1 * randn(d)
    if case["op"].startswith("gate_norm"):
        st["y"] = randn(rows, d).to(io)
        st["z"] = randn(rows, 2 * d).to(io)[:, :d]
        st["dout"] = randn(rows, d).to(io) if case["op"] == "gate_norm_backward" else None
        return st
    res = _dtype(case["res"])
    st["h"] = randn(rows, d).to(io)
    st["residual"] = (3.0 * randn(rows, d)).to(res)
    st["post_weight"] = 1.0 + 0.1 * randn(d) if case["post"] else None
    st["scale"], st["scale_vec"] = 0.5, 1.0 + 0.1 * randn(d) if case["vec"] else None
    if case["op"] == "residual_norm_backward":
        st["dout"], st["dresidual"] = randn(rows, d).to(io), randn(rows, d).to(res)
    return st


# ------------------------------------------------------------------------------------------ plain forms
def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan(x, dt, B, C, A_log, D, dt_bias, state, cu, lens):
    """The chunked scan in 32 bits, every chunk and sequence at once: products within the chunks, and one product
    over the chunks that brings each the state it starts from."""
    T, H, P = x.shape
    G, N = B.shape[1:]
    S, L = len(lens), CHUNK
    length = (cu[1:] - cu[:-1]).long()
    count = (length + L - 1) // L
    nc = sum(-(-n // L) for n in lens)
    seq = torch.repeat_interleave(torch.arange(S, device=x.device), count, output_size=nc)
    first = count.cumsum(0) - count
    number = torch.arange(nc, device=x.device) - first[seq]
    tok = cu[seq].long()[:, None] + number[:, None] * L + torch.arange(L, device=x.device)
    there = tok < cu[seq + 1].long()[:, None]
    tok = tok.clamp(max=max(T - 1, 0))
    delta = _softplus(dt + dt_bias)
    log_a = -torch.exp(A_log) * delta
    xc = x[tok] * there[:, :, None, None]                                   # [nc, L, H, P]
    Bc, Cc = B[tok] * there[:, :, None, None], C[tok] * there[:, :, None, None]
    dc = (delta[tok] * there[:, :, None]).permute(0, 2, 1)                  # [nc, H, L]
    lc = (log_a[tok] * there[:, :, None]).permute(0, 2, 1)
    # sums over the tokens between j and i, not differences of running sums, which would cancel
    below = torch.ones(L, L, dtype=torch.bool, device=x.device).tril(-1)
    between = (lc[..., None] * below).cumsum(2)                             # [nc, H, i, j]: tokens j < k <= i
    decay = torch.exp(between.masked_fill(below.T, -math.inf))
    cum, total = lc.cumsum(2), lc.sum(2)                                    # [nc, H, L], [nc, H]
    scores = Cc.permute(0, 2, 1, 3) @ Bc.permute(0, 2, 3, 1)                # [nc, G, L, L]
    M = (scores[:, :, None] * decay.unflatten(1, (G, H // G))).flatten(1, 2) * dc[:, :, None, :]
    xh = xc.permute(0, 2, 1, 3)                                             # [nc, H, L, P]
    Bh = Bc.permute(0, 2, 1, 3).repeat_interleave(H // G, 1)                # [nc, H, L, N]
    Ch = Cc.permute(0, 2, 1, 3).repeat_interleave(H // G, 1)
    weight = torch.exp(between[:, :, -1]) * dc
    local = (xh * weight[..., None]).transpose(2, 3) @ Bh                   # what each chunk adds: [nc, H, P, N]
    # carried[c] = sum over earlier chunks c' of the sequence of the decays between them times local[c'], and
    # the initial state's share; since[h, c, j] = sum of the totals of chunks j .. c - 1
    chunk = torch.arange(nc, device=x.device)
    since = (total.T[:, :, None] * (chunk[:, None] >= chunk)).cumsum(1)
    since = torch.cat([since.new_zeros(H, 1, nc), since[:, :-1]], 1)
    earlier = (seq[:, None] == seq) & (chunk < chunk[:, None])
    R = torch.exp(torch.cat([since[:, :, 1:], since[:, :, :1]], 2).masked_fill(~earlier, -math.inf))
    carried = (R @ local.permute(1, 0, 2, 3).flatten(2)).unflatten(2, (P, N)).permute(1, 0, 2, 3)
    carried = carried + torch.exp(since[:, chunk, first[seq]]).T[:, :, None, None] * state[seq]
    y = M @ xh + torch.exp(cum)[..., None] * (Ch @ carried.transpose(2, 3))
    y = y + D[:, None, None] * xh
    out = x.new_zeros(T, H, P).index_put((tok[there],), y.permute(0, 2, 1, 3)[there])
    final = torch.exp(total)[:, :, None, None] * carried + local
    final = torch.where((count > 0)[:, None, None, None], final[(first + count - 1).clamp(min=0)], state)
    return out, final


def _plain_prefill(st):
    f = [st[k].float() for k in ("x", "dt", "B", "C", "A_log", "D", "dt_bias", "state")]
    y, final = _plain_scan(*f, st["cu"], st["lens"])
    return y.to(st["x"].dtype), final


def _plain_backward(st):
    names = ("x", "dt", "B", "C", "A_log", "D", "dt_bias", "state")
    f = [st[k].float().detach().requires_grad_(True) for k in names]
    y, final = _plain_scan(*f, st["cu"], st["lens"])
    grads = torch.autograd.grad((y, final), f, (st["dy"].float(), st["dstate"]))
    return [g.to(st[k].dtype) for g, k in zip(grads, names)]


def _plain_decode(st):
    x, dt, B, C = (st[k].float() for k in ("x", "dt", "B", "C"))
    H, G = x.shape[1], B.shape[1]
    delta = _softplus(dt + st["dt_bias"])
    a = torch.exp(-torch.exp(st["A_log"]) * delta)
    Bh, Ch = B.repeat_interleave(H // G, 1), C.repeat_interleave(H // G, 1)
    new = a[..., None, None] * st["state"] + (delta[..., None] * x)[..., None] * Bh[:, :, None, :]
    y = (new * Ch[:, :, None, :]).sum(3) + st["D"][:, None] * x
    return y.to(st["x"].dtype), new


def _grouped(v, groups):
    return v.float().unflatten(1, (groups, -1))


def _plain_gate_norm(st):
    c = st["case"]
    y, z = _grouped(st["y"], c["groups"]), _grouped(st["z"], c["groups"])
    s = z / (1.0 + torch.exp(-z))
    u = y * s if c["gate_first"] else y
    out = u * torch.rsqrt((u * u).mean(2, keepdim=True) + EPS) * st["weight"].unflatten(0, (c["groups"], -1))
    return (out if c["gate_first"] else out * s).flatten(1).to(st["y"].dtype)


def _plain_gate_norm_backward(st):
    c = st["case"]
    y, z, do = (_grouped(st[k], c["groups"]) for k in ("y", "z", "dout"))
    w = st["weight"].unflatten(0, (c["groups"], -1))
    sig = 1.0 / (1.0 + torch.exp(-z))
    s = z * sig
    ds = sig * (1.0 + z * (1.0 - sig))
    u = y * s if c["gate_first"] else y
    r = torch.rsqrt((u * u).mean(2, keepdim=True) + EPS)
    n = u * r
    if c["gate_first"]:
        dn = do * w
        du = r * (dn - n * (dn * n).mean(2, keepdim=True))
        dy, dz, dw = du * s, du * y * ds, (do * n).sum(0)
    else:
        dn = do * w * s
        dy, dz, dw = r * (dn - n * (dn * n).mean(2, keepdim=True)), do * w * n * ds, (do * n * s).sum(0)
    return dy.flatten(1).to(st["y"].dtype), dz.flatten(1).to(st["z"].dtype), dw.flatten()


def _plain_residual_norm(st):
    h = st["h"].float()
    if st["post_weight"] is not None:
        h = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["post_weight"]
    scale = st["scale"] if st["scale_vec"] is None else st["scale"] * st["scale_vec"]
    r = st["residual"].float() + scale * h
    out = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * st["weight"]
    return out.to(st["h"].dtype), r.to(st["residual"].dtype)


def _plain_residual_norm_backward(st):
    """Gradients for a block boundary whose new residual is st["residual"]."""
    do, dr, h, r = (st[k].float() for k in ("dout", "dresidual", "h", "residual"))
    k = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    n = r * k
    dn = do * st["weight"]
    dr = dr + k * (dn - n * (dn * n).mean(1, keepdim=True))
    dw = (do * n).sum(0)
    scale = st["scale"] if st["scale_vec"] is None else st["scale"] * st["scale_vec"]
    dp = dr * scale
    got = dict(dresidual=dr.to(st["residual"].dtype), dweight=dw)
    if st["post_weight"] is None:
        p, dh = h, dp
    else:
        k = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        n = h * k
        p = n * st["post_weight"]
        got["dpost_weight"] = (dp * n).sum(0)
        dn = dp * st["post_weight"]
        dh = k * (dn - n * (dn * n).mean(1, keepdim=True))
    if st["scale_vec"] is not None:
        got["dscale_vec"] = (st["scale"] * dr * p).sum(0)
    got["dh"] = dh.to(st["h"].dtype)
    return got


PLAIN = dict(prefill=_plain_prefill, backward=_plain_backward, decode=_plain_decode, gate_norm=_plain_gate_norm,
             gate_norm_backward=_plain_gate_norm_backward, residual_norm=_plain_residual_norm,
             residual_norm_backward=_plain_residual_norm_backward)


# ------------------------------------------------------------------------------------- the library's calls
def _own(st):
    import selective_state_space_causal_amd as mm

    c = st["case"]
    if c["op"] in ("prefill", "decode", "backward"):
        tokens = [st[k] for k in ("x", "dt", "B", "C", "A_log", "D", "dt_bias")]
    if c["op"] == "prefill":
        return mm.heads_prefill(*tokens, st["cu"], st["state"])
    if c["op"] == "decode":
        return mm.heads_decode(*tokens, st["state"])
    if c["op"] == "backward":
        g = mm.heads_backward(*tokens, st["cu"], st["state"], st["dy"], st["dstate"])
        return [g[k] for k in ("dx", "ddt", "dB", "dC", "dA_log", "dD", "ddt_bias", "dstate_in")]
    if c["op"] == "gate_norm":
        return mm.gate_norm(st["y"], st["z"], st["weight"], groups=c["groups"], eps=EPS, gate_first=c["gate_first"])
    if c["op"] == "gate_norm_backward":
        return mm.gate_norm_backward(st["dout"], st["y"], st["z"], st["weight"], groups=c["groups"], eps=EPS,
                                     gate_first=c["gate_first"])
    rest = dict(post_weight=st["post_weight"], scale=st["scale"], scale_vec=st["scale_vec"], eps=EPS)
    if c["op"] == "residual_norm":
        return mm.residual_norm(st["h"], st["residual"], st["weight"], **rest)
    return mm.residual_norm_backward(st["dout"], st["dresidual"], st["h"], st["residual"], st["weight"], **rest)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------------- 64-bit references
def _padded(v, lens, fill=0.0):
    out = v.new_full((len(lens), max(lens)) + v.shape[1:], fill, dtype=torch.float64)
    at = 0
    for s, n in enumerate(lens):
        out[s, :n] = v[at:at + n]
        at += n
    return out


def _packed(v, lens):
    return torch.cat([v[s, :n] for s, n in enumerate(lens)])


def _exact_tokens(st, lens):
    H, G = st["x"].shape[1], st["B"].shape[1]
    x, dt, B, C = (st[k].double() for k in ("x", "dt", "B", "C"))
    v = dt + st["dt_bias"].double()
    delta = torch.logaddexp(v, torch.zeros_like(v))
    a = torch.exp(-torch.exp(st["A_log"].double()) * delta)
    head = torch.arange(H, device=x.device) // (H // G)
    return (_padded(x, lens), _padded(delta, lens), _padded(a, lens, 1.0), _padded(B[:, head], lens),
            _padded(C[:, head], lens), torch.sigmoid(v))


def _exact_forward(st, lens):
    """The recurrence itself, token after token."""
    x, delta, a, B, C, _ = _exact_tokens(st, lens)
    h, y = st["state"].double(), torch.empty_like(x)
    for t in range(x.shape[1]):
        h = h * a[:, t, :, None, None] + (delta[:, t, :, None] * x[:, t])[..., None] * B[:, t, :, None, :]
        y[:, t] = (h @ C[:, t, :, :, None])[..., 0]
    return _packed(y + st["D"].double()[:, None] * x, lens), h


def _exact_backward(st, lens):
    """The recurrence's adjoint, token after token from the end; the states of 64 tokens at a time are made again
    from those kept at every 64th."""
    x, delta, a, B, C, sig = _exact_tokens(st, lens)
    dy = _padded(st["dy"].double(), lens)
    S, L, H, P = x.shape
    G, every = st["B"].shape[1], 64
    A, D = -torch.exp(st["A_log"].double()), st["D"].double()
    step = lambda h, t: h * a[:, t, :, None, None] + (delta[:, t, :, None] * x[:, t])[..., None] * B[:, t, :, None, :]  # noqa: E731
    kept, h = [], st["state"].double()
    for t in range(L):
        if t % every == 0:
            kept.append(h)
        h = step(h, t)
    g = st["dstate"].double()
    dx, dB, dC = torch.empty_like(x), torch.empty_like(B), torch.empty_like(C)
    ddelta, dl = torch.empty_like(delta), torch.empty_like(delta)
    for b in reversed(range(len(kept))):
        states = [kept[b]]
        for t in range(b * every, min(L, (b + 1) * every)):
            states.append(step(states[-1], t))
        for t in reversed(range(b * every, min(L, (b + 1) * every))):
            old, new = states[t - b * every], states[t - b * every + 1]
            g = g + dy[:, t, :, :, None] * C[:, t, :, None, :]
            dC[:, t] = (dy[:, t, :, None, :] @ new)[..., 0, :]
            gB = (g @ B[:, t, :, :, None])[..., 0]
            dB[:, t] = delta[:, t, :, None] * (x[:, t, :, None, :] @ g)[..., 0, :]
            dx[:, t] = delta[:, t, :, None] * gB + D[:, None] * dy[:, t]
            g = g * a[:, t, :, None, None]
            dl[:, t] = (g * old).sum((2, 3))
            ddelta[:, t] = (x[:, t] * gB).sum(2) + A * dl[:, t]
    share = lambda v: _packed(v, lens).unflatten(1, (G, H // G)).sum(2)  # noqa: E731
    ddt = _packed(ddelta, lens) * sig
    dA = (_packed(delta * dl, lens) * A).sum(0)
    dD = (st["x"].double() * st["dy"].double()).sum((0, 2))
    return [_packed(dx, lens), ddt, share(dB), share(dC), dA, dD, ddt.sum(0), g]


def _exact_norms(st, case):
    """The definitions in 64 bits; the gradients through torch's differentiation of them."""
    leaf = lambda k: st[k].double().requires_grad_(True)  # noqa: E731
    norm = lambda v: v / torch.sqrt((v ** 2).mean(-1, keepdim=True) + EPS)  # noqa: E731
    w = leaf("weight")
    if case["op"].startswith("gate_norm"):
        y, z = leaf("y"), leaf("z")
        shape = (case["rows"], case["groups"], case["d"] // case["groups"])
        s = z * torch.sigmoid(z)
        out = norm((y * s if case["gate_first"] else y).reshape(shape)).reshape(y.shape) * w
        out = out if case["gate_first"] else out * s
        if case["op"] == "gate_norm":
            return out.detach()
        return torch.autograd.grad(out, (y, z, w), st["dout"].double())
    h, r = leaf("h"), leaf("residual")
    p = norm(h) * (wp := leaf("post_weight")) if case["post"] else h
    change = st["scale"] * p * ((vec := leaf("scale_vec")) if case["vec"] else 1.0)
    if case["op"] == "residual_norm":
        return (norm(r + change) * w).detach(), (r + change).detach()
    dr, dw = torch.autograd.grad(norm(r) * w, (r, w), st["dout"].double())
    dr = dr + st["dresidual"].double()
    names = ["dh"] + ["dpost_weight"] * case["post"] + ["dscale_vec"] * case["vec"]
    leaves = [h] + ([wp] if case["post"] else []) + ([vec] if case["vec"] else [])
    return dict(zip(names, torch.autograd.grad(change, leaves, dr)), dresidual=dr, dweight=dw)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("prefill", "decode", "backward"):
        lens = st.get("lens")
        return _exact_backward(st, lens) if case["op"] == "backward" else _exact_forward(st, lens)
    return _exact_norms(st, case)
