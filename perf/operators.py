"""Workloads of the sequence-block operators: gated linear recurrence, gated
feed-forward and 4-bit matrix-vector product.

Each case names one operator in one direction and type.  ``run`` computes it
either in plain torch operations (``own = False``: 32-bit arithmetic, rounded
once at the end) or through the library (``own = True``).  ``exact`` is the
definition in 64 bits.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGEST_SCAN = 512 * 128 * 1024          # elements of the largest recurrence
LARGEST_GLU = 65536 * 1024 * 4096        # M * K * F of the largest feed-forward
LARGEST_W4 = 32768 * 4096                # weights of the largest 4-bit matrix


def listed():
    return [
        # one generated token for each of 128 sequences: a launch's latency
        dict(name="scan_step", op="scan", form="step", dtype="bf16", T=1, N=128, H=1024, D=1, G=3, varlen=False),
        # one long document, one sequence: time has to be split to fill the card
        dict(name="scan_long", op="scan", form="forward", dtype="bf16", T=65536, N=1, H=1024, D=1, G=3, varlen=False),
        # speech-sized padded batch of both directions, 32-bit training
        dict(name="scan_bidir_lengths", op="scan", form="train", dtype="f32", T=300, N=20, H=800, D=2, G=2, varlen=True),
        # the large stack's batch, 16-bit training with an output gate
        dict(name="scan_train", op="scan", form="train", dtype="bf16", T=512, N=128, H=1024, D=1, G=3, varlen=False),
        # one token: the bytes of the weights
        dict(name="glu_token", op="glu", form="forward", dtype="bf16", M=1, K=1024, F=4096, act="silu"),
        # one step of a batch of 20 in 32 bits
        dict(name="glu_batch20_f32", op="glu", form="forward", dtype="f32", M=20, K=800, F=2160, act="gelu"),
        # sizes that no tile divides
        dict(name="glu_odd", op="glu", form="forward", dtype="bf16", M=777, K=1003, F=2731, act="gelu"),
        # a speech-sized batch in 32-bit training
        dict(name="glu_train_f32", op="glu", form="train", dtype="f32", M=6000, K=800, F=2160, act="sigmoid"),
        # the large stack's batch in 16-bit training
        dict(name="glu_train", op="glu", form="train", dtype="bf16", M=65536, K=1024, F=4096, act="silu"),
        # a small projection for one token: latency
        dict(name="w4_small", op="w4", form="forward", dtype="bf16", M=1, R=1024, K=1024, group=64, zeros=False),
        # the projection to a vocabulary for one token
        dict(name="w4_vocab", op="w4", form="forward", dtype="bf16", M=1, R=32768, K=4096, group=128, zeros=False),
        # eight tokens, small groups with zero points, a ragged K, 32 bits
        dict(name="w4_batch8_f32", op="w4", form="forward", dtype="f32", M=8, R=16384, K=6007, group=32, zeros=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A width: mostly a multiple of 8, sometimes any number."""
    v = _log(rng, lo, hi)
    if rng.random() < 0.65:
        v = max(lo, v // 8 * 8)
    return v + 8 if v in (1536, 3072) else v


def draw(rng):
    op = rng.choice(("scan", "glu", "w4"))
    dtype = rng.choice(("bf16", "f32"))
    if op == "scan":
        form = rng.choice(("forward", "train", "train", "step"))
        D = rng.choice((1, 2)) if form != "step" else 1
        H = _size(rng, 16, 2048)
        N = _log(rng, 1, 128)
        T = 1 if form == "step" else _log(rng, 1, max(1, min(65536, LARGEST_SCAN // (N * H * D))))
        return dict(op=op, form=form, dtype=dtype, T=T, N=N, H=H, D=D, G=rng.choice((2, 3)),
                    varlen=form != "step" and rng.random() < 0.5)
    if op == "glu":
        form = rng.choice(("forward", "forward", "train"))
        K, F = _size(rng, 64, 2048), _size(rng, 64, 8192)
        M = _log(rng, 1, max(1, min(16384, LARGEST_GLU // (4 * K * F))))
        if form == "train":
            M = max(M, 16)
        return dict(op=op, form=form, dtype=dtype, M=M, K=K, F=F, act=rng.choice(("silu", "gelu", "sigmoid")))
    K = _size(rng, 64, 16384)
    R = _log(rng, 64, max(64, min(65536, LARGEST_W4 // K)))
    return dict(op=op, form="forward", dtype=dtype, M=_log(rng, 1, 16), R=R if R != 3072 else 3073, K=K,
                group=rng.choice((32, 64, 128)), zeros=rng.random() < 0.5)


def _lengths(c):
    """Valid lengths of a padded batch: spread evenly over 0 .. T, in a mixed
    order (they depend on the sizes alone, so that the work is known)."""
    T, N = c["T"], c["N"]
    return [T if N == 1 else ((i * 7 + N - 1) % N) * T // (N - 1) for i in range(N)]


def work(case):
    c = case
    b = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "scan":
        steps = sum(_lengths(c)) if c["varlen"] else c["T"] * c["N"]
        width, states = c["D"] * c["H"], 4 * c["N"] * c["D"] * c["H"]
        forward = b * width * (steps * c["G"] + c["T"] * c["N"]) + 2 * states
        flops = (10 + 5 * (c["G"] - 2)) * steps * width
        if c["form"] != "train":
            return {"bytes": forward, "flops": flops}
        # the backward pass: gx and dy read, dgx written (zeros past a length too)
        back = b * width * (steps * (c["G"] + 1) + c["T"] * c["N"] * c["G"]) + 3 * states
        return {"bytes": forward + back, "flops": 3 * flops}
    if c["op"] == "glu":
        M, K, F = c["M"], c["K"], c["F"]
        if c["form"] == "forward":
            return {"bytes": b * (M * K + 2 * F * K + M * F), "flops": 4 * M * K * F}
        return {"bytes": b * (2 * M * K + 4 * F * K + 2 * M * F), "flops": 12 * M * K * F}
    M, R, K = c["M"], c["R"], c["K"]
    groups = R * (-(-K // c["group"]))
    return {"bytes": R * K // 2 + groups * (b + (1 if c["zeros"] else 0)) + b * M * (K + R), "flops": 2 * M * R * K}


def _inputs(case, seed):
    """The inputs alone, made on the GPU from the seed."""
    c, dt = case, TYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    if c["op"] == "scan":
        T, N, H, D, G = (c[k] for k in "TNHDG")
        gx = normal(T, N, D, G, H)
        gx[:, :, :, 0] += 2.0           # forget gates mostly open, as trained ones are
        s = dict(gx=gx.reshape(T, N, D * G * H).to(dt), h0=normal(D, N, H))
        if c["form"] == "train":
            s.update(dy=normal(T, N, D * H).to(dt), dhy=normal(D, N, H))
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda") if c["varlen"] else None
        return s
    if c["op"] == "glu":
        M, K, F = c["M"], c["K"], c["F"]
        s = dict(x=normal(M, K).to(dt), W=(normal(2 * F, K) / math.sqrt(K)).to(dt))
        if c["form"] == "train":
            s["dy"] = normal(M, F).to(dt)
        return s
    M, R, K = c["M"], c["R"], c["K"]
    pitch, groups = -(-(-(-K // 2)) // 16) * 16, -(-K // c["group"])
    s = dict(x=normal(M, K).to(dt))
    s["q"] = torch.randint(0, 256, (R, pitch), generator=gen, device="cuda", dtype=torch.uint8)
    s["scales"] = ((0.5 + torch.rand((R, groups), generator=gen, device="cuda")) / (8 * math.sqrt(K))).to(dt)
    s["zeros"] = torch.randint(0, 16, (R, groups), generator=gen, device="cuda", dtype=torch.uint8) if c["zeros"] else None
    return s


def prepare(case, seed):
    c, dt = dict(case), TYPES[case["dtype"]]
    s = _inputs(case, seed)
    s["case"] = c
    if not own:
        return s
    # what a user's program keeps beside its data: a handle, the results'
    # buffers and the workspace
    from layer_rnn_gb300 import binding
    ops = s["ops"] = binding.Ops(c["dtype"])
    new = lambda *shape, t=dt: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    if c["op"] == "scan":
        T, N, H, D = (c[k] for k in "TNHD")
        s.update(y=new(T, N, D * H), hy=new(D, N, H, t=torch.float32))
        if c["form"] == "train":
            s.update(dgx=torch.empty_like(s["gx"]), dh0=torch.empty_like(s["h0"]),
                     ws=new(ops.scan_workspace_bytes(T, N, H, D), t=torch.uint8))
    elif c["op"] == "glu":
        M, K, F = c["M"], c["K"], c["F"]
        train = c["form"] == "train"
        s.update(y=new(M, F), ws=new(ops.glu_workspace_bytes(M, K, F, backward=train), t=torch.uint8))
        if train:
            s.update(dx=new(M, K), dW=new(2 * F, K))
    else:
        s["y"] = new(c["M"], c["R"])
    return s


def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    return {"scan": _plain_scan, "glu": _plain_glu, "w4": _plain_w4}[c["op"]](s, c)


def _own(s, c):
    ops = s["ops"]
    if c["op"] == "scan":
        gate = c["G"] == 3
        if c["form"] == "step":
            ops.scan_step(s["gx"][0], s["h0"][0], s["hy"][0], s["y"][0], out_gate=gate)
            return {"y": s["y"], "hy": s["hy"]}
        ws = s.get("ws")
        ops.scan_forward(s["gx"], s["h0"], s["y"], s["hy"], lengths=s["lengths"], ws=ws, out_gate=gate)
        if c["form"] == "forward":
            return {"y": s["y"], "hy": s["hy"]}
        ops.scan_backward(s["gx"], s["dy"], s["dhy"], s["dgx"], s["dh0"], ws, lengths=s["lengths"], out_gate=gate)
        return {"y": s["y"], "hy": s["hy"], "dgx": s["dgx"], "dh0": s["dh0"]}
    if c["op"] == "glu":
        ops.glu_forward(s["x"], s["W"], s["y"], s["ws"], act=c["act"])
        if c["form"] == "forward":
            return {"y": s["y"]}
        ops.glu_backward(s["x"], s["W"], s["dy"], s["dx"], s["dW"], s["ws"], act=c["act"])
        return {"y": s["y"], "dx": s["dx"], "dW": s["dW"]}
    ops.w4_matvec(s["x"], s["q"], s["scales"], s["y"], group=c["group"], zeros=s["zeros"])
    return {"y": s["y"]}


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------

def _scan(a, b):
    """Inclusive scan of h -> a h + b along dimension 0: the product of the a
    and the value from a zero start (doubling: log2 T passes)."""
    s = 1
    while s < a.shape[0]:
        b = torch.cat([b[:s], b[s:] + a[s:] * b[:-s]])
        a = torch.cat([a[:s], a[s:] * a[:-s]])
        s *= 2
    return a, b


def _plain_scan(s, c):
    T, N, H, D, G = (c[k] for k in "TNHDG")
    dt = TYPES[c["dtype"]]
    gx = s["gx"].float().view(T, N, D, G, H)
    p, z = gx[:, :, :, 0], gx[:, :, :, 1]
    f, i = torch.sigmoid(p), torch.sigmoid(-p)
    valid = None
    a, b = f, i * z
    if s["lengths"] is not None:
        valid = (torch.arange(T, device="cuda")[:, None] < s["lengths"][None, :])[:, :, None, None]
        a, b = torch.where(valid, a, 1.0), torch.where(valid, b, 0.0)
    h0 = s["h0"].transpose(0, 1)                              # [N, D, H]
    turn = lambda v: v if D == 1 else torch.stack([v[:, :, 0], v[:, :, 1].flip(0)], 2)  # noqa: E731
    A, B = _scan(turn(a), turn(b))
    hw = B + A * h0                                           # in the order each direction walks
    before = turn(torch.cat([h0[None], hw[:-1]]))             # h_{t-1}, in time order
    hy = hw[-1].transpose(0, 1).contiguous()
    h = turn(hw)
    o = torch.sigmoid(gx[:, :, :, 2]) if G == 3 else None
    y = h if o is None else o * h
    y = y if valid is None else torch.where(valid, y, 0.0)
    out = {"y": y.reshape(T, N, D * H).to(dt), "hy": hy}
    if c["form"] != "train":
        return out
    dy = s["dy"].float().view(T, N, D, H)
    direct = dy if o is None else dy * o
    direct = direct if valid is None else torch.where(valid, direct, 0.0)
    # against the walk: e_t = a_t (direct_t + e_{t+1}), e_T = dhy
    aw, bw = turn(a).flip(0), turn(a * direct).flip(0)
    A, B = _scan(aw, bw)
    dhy = s["dhy"].transpose(0, 1)
    e = B + A * dhy
    out["dh0"] = e[-1].transpose(0, 1).contiguous()
    into = turn(torch.cat([dhy[None], e[:-1]]).flip(0))
    dh = direct + into
    parts = [dh * (before - z) * f * i, dh * i]
    if o is not None:
        parts.append(dy * h * o * (1 - o))
    dgx = torch.stack(parts, 3)
    dgx = dgx if valid is None else torch.where(valid[..., None], dgx, 0.0)
    out["dgx"] = dgx.reshape(T, N, D * G * H).to(dt)
    return out


C0, C1 = math.sqrt(2 / math.pi), 0.044715


def _plain_act(g, act):
    """act(g) and its derivative."""
    if act == "gelu":
        th = torch.tanh(C0 * (g + C1 * g * g * g))
        return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * C0 * (1 + 3 * C1 * g * g)
    sg = torch.sigmoid(g)
    if act == "silu":
        return g * sg, sg * (1 + g * (1 - sg))
    return sg, sg * (1 - sg)


def _plain_glu(s, c):
    F, dt = c["F"], TYPES[c["dtype"]]
    x, W = s["x"].float(), s["W"].float()
    gu = x @ W.t()
    g, u = gu[:, :F], gu[:, F:]
    v, d = _plain_act(g, c["act"])
    out = {"y": (v * u).to(dt)}
    if c["form"] != "train":
        return out
    dy = s["dy"].float()
    dgu = torch.cat([dy * u * d, dy * v], 1)
    out["dx"] = (dgu @ W).to(dt)
    out["dW"] = (dgu.t() @ x).to(dt)
    return out


def _plain_w4(s, c):
    K, group = c["K"], c["group"]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], 2).view(c["R"], -1)[:, :K].float()
    of = torch.arange(K, device="cuda") // group
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, of]
    w = (q - zero) * s["scales"].float()[:, of]
    return {"y": (s["x"].float() @ w.t()).to(TYPES[c["dtype"]])}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    return {"scan": _exact_scan, "glu": _exact_glu, "w4": _exact_w4}[case["op"]](s, case)


def _logistic(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _exact_scan(s, c):
    """Step by step, as the recurrence is written."""
    T, N, H, D, G = (c[k] for k in "TNHDG")
    train = c["form"] == "train"
    gx = s["gx"].view(T, N, D, G, H)
    y = torch.zeros((T, N, D, H), dtype=torch.float64, device="cuda")
    dgx = torch.zeros((T, N, D, G, H), dtype=torch.float64, device="cuda") if train else None
    hy, dh0 = (torch.empty((D, N, H), dtype=torch.float64, device="cuda") for _ in range(2))
    lens = s["lengths"]
    for d in range(D):
        order = range(T) if d == 0 else range(T - 1, -1, -1)
        g = gx[:, :, d].double()
        f = _logistic(g[:, :, 0])
        if lens is not None:
            live = (torch.arange(T, device="cuda")[:, None] < lens[None, :])[:, :, None].double()
            keep = f * live + (1 - live)
            new = (1 - f) * g[:, :, 1] * live
        else:
            live, keep, new = None, f, (1 - f) * g[:, :, 1]
        o = _logistic(g[:, :, 2]) if G == 3 else torch.ones_like(f)
        o = o if live is None else o * live
        h = s["h0"][d].double()
        before = torch.empty((T, N, H), dtype=torch.float64, device="cuda") if train else None
        hs = torch.empty((T, N, H), dtype=torch.float64, device="cuda")
        for t in order:
            if train:
                before[t] = h
            h = torch.addcmul(new[t], keep[t], h)
            hs[t] = h
        hy[d] = h
        y[:, :, d] = o * hs
        if not train:
            continue
        dy = s["dy"].view(T, N, D, H)[:, :, d].double()
        direct = dy * o
        dh = torch.empty((T, N, H), dtype=torch.float64, device="cuda")
        e = s["dhy"][d].double()
        for t in reversed(order):
            dh[t] = direct[t] + e
            e = keep[t] * dh[t]
        dh0[d] = e
        mask = 1.0 if live is None else live
        dgx[:, :, d, 0] = dh * (before - g[:, :, 1]) * f * (1 - f) * mask
        dgx[:, :, d, 1] = dh * (1 - f) * mask
        if G == 3:
            dgx[:, :, d, 2] = dy * hs * o * (1 - _logistic(g[:, :, 2]))
    out = {"y": y.view(T, N, D * H), "hy": hy}
    if train:
        out.update(dgx=dgx.view(T, N, D * G * H), dh0=dh0)
    return out


def _exact_glu(s, c):
    """In blocks of rows: the pre-activations of all rows in 64 bits are large."""
    F, act = c["F"], c["act"]
    W = s["W"].double()
    ys, dxs, dW = [], [], torch.zeros_like(W)
    for r in range(0, c["M"], 8192):
        x = s["x"][r:r + 8192].double()
        g, u = x @ W[:F].t(), x @ W[F:].t()
        if act == "gelu":
            th = torch.tanh(C0 * (g + C1 * g ** 3))
            v = g * (1 + th) / 2
            d = (1 + th) / 2 + g / 2 * (1 - th ** 2) * C0 * (1 + 3 * C1 * g ** 2)
        else:
            sg = _logistic(g)
            v, d = (g * sg, sg + g * sg * (1 - sg)) if act == "silu" else (sg, sg * (1 - sg))
        ys.append(v * u)
        if c["form"] == "train":
            dy = s["dy"][r:r + 8192].double()
            dg, du = dy * u * d, dy * v
            dxs.append(dg @ W[:F] + du @ W[F:])
            dW[:F] += dg.t() @ x
            dW[F:] += du.t() @ x
    out = {"y": torch.cat(ys)}
    if c["form"] == "train":
        out.update(dx=torch.cat(dxs), dW=dW)
    return out


def _exact_w4(s, c):
    K, group, R = c["K"], c["group"], c["R"]
    k = torch.arange(K, device="cuda")
    x = s["x"].double()
    y = torch.empty((c["M"], R), dtype=torch.float64, device="cuda")
    for r in range(0, R, 4096):
        byte = s["q"][r:r + 4096][:, k // 2].long()
        q = torch.where(k % 2 == 0, byte % 16, byte // 16).double()
        zero = 8.0 if s["zeros"] is None else s["zeros"][r:r + 4096].double()[:, k // group]
        w = (q - zero) * s["scales"][r:r + 4096].double()[:, k // group]
        y[:, r:r + 4096] = x @ w.t()
    return {"y": y}
