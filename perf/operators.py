"""Cases and plain forms of the operators around the TTT layer: rotary positions with the
head layout change, the norms / gate / residual of a block (forward and backward), and the
gated linear recurrence (forward, backward, single-token step).

With ``own`` false, ``run`` computes each operator from elementary torch operations in
32 bits; with ``own`` true it calls the framework's entry points.  ``exact`` is the
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}

# The largest number of elements of one token tensor (2 x 32768 tokens of width 2048).
MAX_ELEMS = 2 * 32768 * 2048


def listed():
    return [
        # one decoding step of 64 sequences at the 125M layer's heads, each sequence at a
        # position of its own
        dict(name="rope_decode", op="rope", B=64, T=1, H=12, d=64, rot=64, interleaved=False, inverse=False,
             period=0, rows=32768, given=True, scaling="none", dtype="bf16"),
        # the 125M layer's batch, positions counted inside each 16-token mini-batch, token-major
        # projections turned into the layer's head-major layout
        dict(name="rope_125m", op="rope", B=8, T=2048, H=12, d=64, rot=64, interleaved=False, inverse=False,
             period=16, rows=16, given=False, scaling="none", dtype="bf16"),
        # the gradient's way back at the long-context layer: interleaved pairs on half of each head,
        # frequencies stretched for a long context
        dict(name="rope_long_inverse", op="rope", B=2, T=32768, H=32, d=64, rot=32, interleaved=True, inverse=True,
             period=0, rows=32768, given=False, scaling="yarn", dtype="bf16"),
        # one decoding step of 64 sequences through the sandwich: post norm, gate, residual, pre norm
        dict(name="norm_decode", op="norm", B=64, T=1, D=768, heads=12, post="rms", act="silu", res=True,
             scale=True, pre="rms", train=False, dtype="bf16"),
        # behind a 125M TTT layer in prefill: layer norm of the head-major output times GELU(gate),
        # the input of the output projection
        dict(name="norm_gate_125m", op="norm", B=8, T=2048, D=768, heads=12, post="layer", act="gelu", res=False,
             scale=False, pre="none", train=False, dtype="bf16"),
        # a training step of the sandwich at the 125M shape, token-major
        dict(name="norm_train_125m", op="norm", B=8, T=2048, D=768, heads=1, post="rms", act="silu", res=True,
             scale=True, pre="rms", train=True, dtype="bf16"),
        # odd width and token count in 32 bits, layer norms on both sides
        dict(name="norm_train_odd_f32", op="norm", B=3, T=701, D=1001, heads=1, post="layer", act="sigmoid", res=True,
             scale=True, pre="layer", train=True, dtype="f32"),
        # a training step at the long-context layer
        dict(name="norm_train_long", op="norm", B=2, T=32768, D=2048, heads=32, post="layer", act="gelu", res=True,
             scale=True, pre="rms", train=True, dtype="bf16"),
        # one decoding step of 64 sequences
        dict(name="recurrence_decode", op="recurrence", B=64, T=1, C=768, mode="mix", reset=False, train=False,
             dtype="bf16"),
        # prefill at the 125M layer's width
        dict(name="recurrence_125m", op="recurrence", B=8, T=2048, C=768, mode="mix", reset=False, train=False,
             dtype="bf16"),
        # packed sequences (resets) of odd sizes in 32 bits, training
        dict(name="recurrence_train_odd_f32", op="recurrence", B=3, T=1999, C=333, mode="sigmoid", reset=True,
             train=True, dtype="f32"),
        # training on a long context
        dict(name="recurrence_train_long", op="recurrence", B=2, T=32768, C=2048, mode="mix", reset=False, train=True,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + (n % 1024 == 0 and lo < n < hi)  # whole multiples are what the listed cases have


def draw(rng):
    op = rng.choice(["rope", "norm", "recurrence"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    cap = MAX_ELEMS // 4 if dtype == "f32" else MAX_ELEMS // 2
    if op == "rope":
        # heads and widths of the framework's layers and some that no vector width divides
        d = rng.choice([16, 20, 32, 48, 64, 64, 80, 96, 128])
        H = rng.choice([1, 2, 3, 5, 6, 12, 24, 32])
        if H * d % 1024 == 0 and H * d < 4096:
            H -= 1
        T = min(_log_int(rng, 1, 32768), cap // (H * d))
        B = max(1, min(_log_int(rng, 1, 64), cap // (T * H * d)))
        rot = rng.choice([d, d, d // 2, d // 4])
        rot = max(2, rot - rot % 2)
        period = rng.choice([0, 0, 16])
        return dict(op=op, B=B, T=T, H=H, d=d, rot=rot, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4,
                    period=period, rows=period if period else _log_int(rng, T, T + 4097), given=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "yarn"]), dtype=dtype)
    if op == "norm":
        heads = rng.choice([1, 1, 3, 6, 12, 32])
        D = _log_int(rng, 16, 8192)
        if heads > 1:
            d = rng.choice([16, 20, 32, 64, 64, 128])
            D = heads * d
        T = _log_int(rng, 1, 32768)
        B = max(1, min(_log_int(rng, 1, 64), cap // (T * D)))
        T = max(1, min(T, cap // (B * D)))
        post = rng.choice(["none", "rms", "layer"])
        pre = rng.choice(["none", "rms", "layer"])
        return dict(op=op, B=B, T=T, D=D, heads=heads, post=post, act=rng.choice(["none", "sigmoid", "silu", "gelu"]),
                    res=rng.random() < 0.7, scale=rng.random() < 0.6, pre=pre, train=rng.random() < 0.6, dtype=dtype)
    C = _log_int(rng, 8, 4096)
    T = _log_int(rng, 1, 32768)
    B = max(1, min(_log_int(rng, 1, 64), cap // (T * C)))
    T = max(1, min(T, cap // (B * C)))
    return dict(op=op, B=B, T=T, C=C, mode=rng.choice(["decay", "sigmoid", "mix"]), reset=rng.random() < 0.4,
                train=rng.random() < 0.6, dtype=dtype)


# ------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype, mean=0.0, std=1.0):
    """Normal draws of a token tensor, made in pieces so that no 32-bit copy of it is held."""
    out = torch.empty(shape, device="cuda", dtype=dtype)
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(std).add_(mean)
    return out


def _frequencies(rot, scaling):
    """Inverse frequencies of the rotated pairs in 64 bits and the factor on cos and sin.
    linear: positions divided by 4.  yarn: by wavelength, from unscaled (short waves, 32 turns
    and more over 8192 positions) to divided by 4 (one turn and less), factor 0.1 ln 4 + 1."""
    i = np.arange(rot // 2, dtype=np.float64)
    inv = 10000.0 ** (-2.0 * i / rot)
    if scaling == "linear":
        return inv / 4.0, 1.0
    if scaling == "yarn":
        turns = 8192.0 * inv / (2.0 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return inv * keep + inv / 4.0 * (1.0 - keep), 0.1 * math.log(4.0) + 1.0
    return inv, 1.0


def _table(rows, rot, scaling):
    """[rows, rot / 2, 2] cos and sin of every position's angles, rounded to 32 bits."""
    inv, m = _frequencies(rot, scaling)
    inv = torch.from_numpy(inv).cuda()
    ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
    return (m * torch.stack([ang.cos(), ang.sin()], -1)).float()


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    dt = DT[c["dtype"]]
    s = {"case": c}
    if c["op"] == "rope":
        B, T, H, d = c["B"], c["T"], c["H"], c["d"]
        if c["inverse"]:
            # gradients in the layer's head-major layout, going to one token-major buffer
            s["q"], s["k"], s["v"] = (_randn(g, (B, H, T, d), dt) for _ in range(3))
        else:
            # one token-major projection of the three
            qkv = _randn(g, (B, T, 3, H, d), dt)
            s["q"], s["k"], s["v"] = qkv.permute(2, 0, 3, 1, 4).unbind(0)
        s["table"] = _table(c["rows"], c["rot"], c["scaling"])
        s["positions"] = None
        if c["given"]:
            hi = c["rows"] if not c["period"] else 1 << 20
            start = torch.randint(0, max(1, hi - T + 1), (B, 1), generator=g, device="cuda")
            s["positions"] = start + torch.arange(T, device="cuda")
        return s
    if c["op"] == "norm":
        B, T, D, Hh = c["B"], c["T"], c["D"], c["heads"]
        s["y"] = _randn(g, (B, Hh, T, D // Hh) if Hh > 1 else (B, T, D), dt, 0.1, 0.7)
        s["x"] = _randn(g, (B, T, D), dt, 0.0, 1.5) if c["res"] else None
        s["gate"] = _randn(g, (B, T, D), dt) if c["act"] != "none" else None

        def vec(on, mean, std):
            return torch.randn(D, generator=g, device="cuda").mul_(std).add_(mean) if on else None
        s["post_weight"] = vec(c["post"] != "none", 1.0, 0.1)
        s["post_bias"] = vec(c["post"] == "layer", 0.0, 0.1)
        s["scale"] = vec(c["scale"], 0.5, 0.1)
        s["pre_weight"] = vec(c["pre"] != "none", 1.0, 0.1)
        s["pre_bias"] = vec(c["pre"] == "layer", 0.0, 0.1)
        if c["train"]:
            s["dh"] = _randn(g, (B, T, D), dt)
            s["du"] = _randn(g, (B, T, D), dt) if c["pre"] != "none" else None
        return s
    B, T, C = c["B"], c["T"], c["C"]
    s["x"] = _randn(g, (B, T, C), dt)
    if c["mode"] == "decay":  # the decay itself, in (0.6, 1)
        f = _randn(g, (B, T, C), dt, 2.0, 1.0)
        for b in range(B):
            f[b] = 0.6 + 0.4 * torch.sigmoid(f[b].float())
        s["f"] = f
    else:  # logits: decays mostly between 0.5 and 0.99
        s["f"] = _randn(g, (B, T, C), dt, 2.0, 1.5)
    s["h0"] = torch.randn((B, C), generator=g, device="cuda")
    s["reset"] = None
    if c["reset"]:  # a new sequence about every 200 tokens
        s["reset"] = torch.rand((B, T), generator=g, device="cuda") < 0.005
    if c["train"]:
        s["dh"] = _randn(g, (B, T, C), dt)
        s["dh_last"] = torch.randn((B, C), generator=g, device="cuda")
    return s


# -------------------------------------------------------------------- plain forms


def _rope_positions(s):
    c = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["T"], device="cuda")[None].expand(c["B"], -1)
    if c["period"]:
        pos = pos % c["period"]
    return pos


def _plain_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    cs = s["table"][_rope_positions(s)][:, None]  # [B, 1, T, rot / 2, 2]
    cos, sin = cs[..., 0], cs[..., 1]
    if c["inverse"]:
        sin = -sin
    out = []
    for t in (s["q"], s["k"]):
        x = t[..., :rot].float()
        if c["interleaved"]:
            x0, x1 = x[..., 0::2], x[..., 1::2]
        else:
            x0, x1 = x[..., :half], x[..., half:]
        y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
        y = torch.stack([y0, y1], -1).flatten(-2) if c["interleaved"] else torch.cat([y0, y1], -1)
        out.append(torch.cat([y.to(t.dtype), t[..., rot:]], -1))
    out.append(s["v"])
    if c["inverse"]:
        return torch.stack([o.transpose(1, 2) for o in out], 2)  # [B, T, 3, H, d]
    return [o.contiguous() for o in out]


def _merge(y):
    return y.transpose(1, 2).flatten(2) if y.dim() == 4 else y


def _norm_parts(kind, v, eps):
    """Normalised rows and the reciprocal spread."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * r, r


def _act(kind, g):
    """The gate's value and its derivative."""
    if kind == "sigmoid":
        a = torch.sigmoid(g)
        return a, a * (1 - a)
    if kind == "silu":
        a = torch.sigmoid(g)
        return g * a, a * (1 + g * (1 - a))
    cdf = 0.5 * (1 + torch.erf(g * 0.7071067811865476))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * 0.3989422804014327


EPS = 1e-6


def _norm_backward(kind, dn, n, r):
    """Gradient of the row from the gradient dn of its normalised form n."""
    t = dn - n * (dn * n).mean(-1, keepdim=True)
    if kind == "layer":
        t = t - dn.mean(-1, keepdim=True)
    return t * r


def _plain_norm(s):
    c = s["case"]
    dt = DT[c["dtype"]]
    y = _merge(s["y"]).float()
    p, ny = y, None
    if c["post"] != "none":
        ny, ry = _norm_parts(c["post"], y, EPS)
        p = ny * s["post_weight"]
        if s["post_bias"] is not None:
            p = p + s["post_bias"]
    A = dA = None
    m = p
    if c["act"] != "none":
        A, dA = _act(c["act"], s["gate"].float())
        m = m * A
    if c["scale"]:
        m = m * s["scale"]
    h = m if s["x"] is None else s["x"].float() + m
    out = [h.to(dt)]
    nh = None
    if c["pre"] != "none":
        nh, rh = _norm_parts(c["pre"], h, EPS)
        u = nh * s["pre_weight"]
        if s["pre_bias"] is not None:
            u = u + s["pre_bias"]
        out.append(u.to(dt))
    if not c["train"]:
        return out
    # gradients, in the order dy, dx, dgate, post weight, post bias, scale, pre weight, pre bias
    G = s["dh"].float()
    pw = pb = scg = prw = prb = dg = dx = None
    if c["pre"] != "none":
        du = s["du"].float()
        prw = (du * nh).sum((0, 1))
        if s["pre_bias"] is not None:
            prb = du.sum((0, 1))
        G = G + _norm_backward(c["pre"], du * s["pre_weight"], nh, rh)
    if s["x"] is not None:
        dx = G.to(dt)
    if c["scale"]:
        scg = (G * (p if A is None else p * A)).sum((0, 1))
    Gs = G * s["scale"] if c["scale"] else G
    dp = Gs
    if A is not None:
        dg = (Gs * p * dA).to(dt)
        dp = Gs * A
    dy = dp
    if c["post"] != "none":
        pw = (dp * ny).sum((0, 1))
        if s["post_bias"] is not None:
            pb = dp.sum((0, 1))
        dy = _norm_backward(c["post"], dp * s["post_weight"], ny, ry)
    if c["heads"] > 1:
        dy = dy.unflatten(-1, (c["heads"], -1)).transpose(1, 2).contiguous()
    return out + [t for t in (dy.to(dt), dx, dg, pw, pb, scg, prw, prb) if t is not None]


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from a zero state, by doubling strides."""
    T, n = a.shape[1], 1
    while n < T:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _plain_recurrence(s):
    c = s["case"]
    dt = DT[c["dtype"]]
    x, f = s["x"].float(), s["f"].float()
    a = f if c["mode"] == "decay" else torch.sigmoid(f)
    na = torch.sigmoid(-f) if c["mode"] == "mix" else None  # 1 - a
    keep = a
    if s["reset"] is not None:
        keep = a.masked_fill(s["reset"][..., None], 0.0)
    b = x if na is None else na * x
    b = torch.cat([b[:, :1] + keep[:, :1] * s["h0"][:, None], b[:, 1:]], 1)
    h = _scan(keep, b)
    out = [h.to(dt), h[:, -1].clone()]
    if not c["train"]:
        return out
    dh = s["dh"].float()
    dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh_last"][:, None]], 1)
    nxt = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)  # a_{t+1} on the way back
    S = _scan(nxt.flip(1), dh.flip(1)).flip(1)
    prev = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    if s["reset"] is not None:
        prev = prev.masked_fill(s["reset"][..., None], 0.0)
    if c["mode"] == "decay":
        df, dx = S * prev, S
    elif c["mode"] == "sigmoid":
        df, dx = S * prev * a * (1 - a), S
    else:
        df, dx = S * (prev - x) * a * na, S * na
    return out + [dx.to(dt), df.to(dt), keep[:, 0] * S[:, 0]]


# ------------------------------------------------------------------------- a pass


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "norm": _plain_norm, "recurrence": _plain_recurrence}[c["op"]](s)
    from test_sequence_layers_gb300 import abi
    if c["op"] == "rope":
        kw = dict(positions=s["positions"], period=c["period"], interleaved=c["interleaved"], inverse=c["inverse"])
        if not c["inverse"]:
            return list(abi.ttt_rope(s["q"], s["k"], s["v"], s["table"], **kw))
        B, H, T, d = s["q"].shape
        dqkv = torch.empty((B, T, 3, H, d), device="cuda", dtype=s["q"].dtype)
        dq, dk, dv = dqkv.permute(2, 0, 3, 1, 4).unbind(0)
        abi.ttt_rope(s["q"], s["k"], s["v"], s["table"], q_out=dq, k_out=dk, v_out=dv, **kw)
        return dqkv
    if c["op"] == "norm":
        kw = dict(x=s["x"], gate=s["gate"], act=c["act"], post=c["post"], post_weight=s["post_weight"],
                  post_bias=s["post_bias"], scale=s["scale"], pre=c["pre"], pre_weight=s["pre_weight"],
                  pre_bias=s["pre_bias"], post_eps=EPS, pre_eps=EPS)
        h, u, stats = abi.ttt_block_norm_fwd(s["y"], want_stats=c["train"], **kw)
        out = [h] if u is None else [h, u]
        if c["train"]:
            grads = abi.ttt_block_norm_bwd(s["dh"], s["du"], s["y"], stats, **kw)
            out += [t for t in grads if t is not None]
        return out
    h, h_last, states = abi.ttt_recurrence_fwd(s["x"], s["f"], s["h0"], mode=c["mode"], reset=s["reset"],
                                               want_states=c["train"])
    if not c["train"]:
        return [h, h_last]
    return [h, h_last] + list(abi.ttt_recurrence_bwd(s["dh"], s["x"], s["f"], states, mode=c["mode"],
                                                     reset=s["reset"], dh_last=s["dh_last"]))


def work(case):
    c, es = case, ES[case["dtype"]]
    if c["op"] == "rope":
        n = c["B"] * c["T"] * c["H"] * c["d"]
        rows = c["period"] or min(c["rows"], c["B"] * c["T"] if c["given"] else c["T"])
        nbytes = 6 * n * es + min(rows, c["rows"]) * c["rot"] * 4 + (8 * c["B"] * c["T"] if c["given"] else 0)
        return {"bytes": nbytes, "flops": 6 * c["B"] * c["T"] * c["H"] * c["rot"]}
    if c["op"] == "norm":
        n = c["B"] * c["T"] * c["D"]
        post, pre, act = c["post"] != "none", c["pre"] != "none", c["act"] != "none"
        ins = 1 + c["res"] + act
        outs = 1 + pre
        vecs = post + (c["post"] == "layer") + c["scale"] + pre + (c["pre"] == "layer")
        flops = 6 * post + 6 * pre + 6 * act + c["scale"] + c["res"]
        if c["train"]:
            outs += 1 + c["res"] + act
            ins += 1 + pre
            vecs *= 2
            flops *= 3
        return {"bytes": (ins + outs) * n * es + vecs * c["D"] * 4, "flops": max(1, flops) * n}
    n = c["B"] * c["T"] * c["C"]
    tensors, states, flops = 3, 2, {"decay": 2, "sigmoid": 5, "mix": 7}[c["mode"]]
    if c["train"]:
        tensors, states, flops = 6, 4, flops + 8
    return {"bytes": tensors * n * es + states * c["B"] * c["C"] * 4 + (c["B"] * c["T"] if c["reset"] else 0),
            "flops": flops * n}


# ------------------------------------------------------------ the definition, 64 bits


def _exact_rope(s):
    c = s["case"]
    B, T, H, d, rot = c["B"], c["T"], c["H"], c["d"], c["rot"]
    tab = s["table"].double()
    z = torch.complex(tab[..., 0], tab[..., 1])  # a rotation is a complex factor
    if c["inverse"]:
        z = z.conj()
    where = torch.arange(T, device="cuda").repeat(B, 1) if s["positions"] is None else s["positions"]
    if c["period"]:
        where = torch.remainder(where, c["period"])
    out = []
    for src in (s["q"], s["k"], s["v"]):
        o = src.double().clone()
        out.append(o)
        if src is s["v"]:
            break
        first = torch.arange(0, rot, 2, device="cuda") if c["interleaved"] else torch.arange(rot // 2, device="cuda")
        second = first + (1 if c["interleaved"] else rot // 2)
        for b in range(B):
            r = torch.complex(o[b][..., first], o[b][..., second]) * z[where[b]]
            o[b][..., first], o[b][..., second] = r.real, r.imag
    if c["inverse"]:
        return torch.stack(out).permute(1, 3, 0, 2, 4).contiguous()
    return [o.contiguous() for o in out]


def _exact_norm(s):
    """The definition in 64 bits over batch entries, gradients by differentiation."""
    c = s["case"]
    names = ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")
    par = {n: (None if s[n] is None else s[n].double().requires_grad_(c["train"])) for n in names}
    hs, us, gy, gx, gg = [], [], [], [], []

    def norm(kind, v, w, b):
        if kind == "none":
            return v
        if kind == "rms":
            return w * v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
        var, mu = torch.var_mean(v, -1, correction=0, keepdim=True)
        return b + w * (v - mu) / torch.sqrt(var + EPS)

    for b in range(c["B"]):
        leaf = {n: (None if s[n] is None else s[n][b].double().requires_grad_(c["train"])) for n in ("y", "x", "gate")}
        y = leaf["y"]
        if y.dim() == 3:
            y = y.permute(1, 0, 2).reshape(c["T"], c["D"])
        t = norm(c["post"], y, par["post_weight"], par["post_bias"])
        if c["act"] == "sigmoid":
            t = t / (1 + torch.exp(-leaf["gate"]))
        elif c["act"] == "silu":
            t = t * leaf["gate"] / (1 + torch.exp(-leaf["gate"]))
        elif c["act"] == "gelu":
            t = t * leaf["gate"] * torch.special.erfc(-leaf["gate"] / math.sqrt(2.0)) / 2
        if c["scale"]:
            t = par["scale"] * t
        h = t if leaf["x"] is None else leaf["x"] + t
        u = norm(c["pre"], h, par["pre_weight"], par["pre_bias"])
        hs.append(h.detach())
        us.append(u.detach())
        if c["train"]:
            obj = (h * s["dh"][b].double()).sum()
            if c["pre"] != "none":
                obj = obj + (u * s["du"][b].double()).sum()
            obj.backward()
            for lst, n in ((gy, "y"), (gx, "x"), (gg, "gate")):
                lst.append(None if leaf[n] is None else leaf[n].grad)
    out = [torch.stack(hs)] + ([torch.stack(us)] if c["pre"] != "none" else [])
    if c["train"]:
        out += [torch.stack(l) for l in (gy, gx, gg) if l[0] is not None]
        out += [par[n].grad for n in names if par[n] is not None]
    return out


def _exact_recurrence(s):
    """Token by token in 64 bits, and token by token back."""
    c = s["case"]
    B, T, C = s["x"].shape
    one = torch.ones((), device="cuda", dtype=torch.float64)
    live = None if s["reset"] is None else (~s["reset"]).double()[..., None]
    h = s["h0"].double()
    H = torch.empty((B, T, C), device="cuda", dtype=torch.float64)
    x, f = s["x"].double(), s["f"].double()
    if c["mode"] != "decay":
        f = one / (one + torch.exp(-f))
    k = f if live is None else f * live
    w = x * (1 - f) if c["mode"] == "mix" else x
    for t in range(T):
        h = torch.addcmul(w[:, t], k[:, t], h)
        H[:, t] = h
    out = [H, H[:, -1].clone()]
    if not c["train"]:
        return out
    r = s["dh_last"].double()
    S = torch.empty_like(H)
    d = s["dh"].double()
    for t in range(T - 1, -1, -1):
        S[:, t] = d[:, t] + r
        r = k[:, t] * S[:, t]
    before = torch.cat([s["h0"].double()[:, None], H[:, :-1]], 1)
    if live is not None:
        before = before * live
    if c["mode"] == "mix":
        return out + [S * (1 - f), S * (before - x) * f * (1 - f), r]
    df = S * before
    if c["mode"] == "sigmoid":
        df = df * f * (1 - f)
    return out + [S, df, r]


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "norm": _exact_norm, "recurrence": _exact_recurrence}[case["op"]](s)
