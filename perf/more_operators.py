"""Cases and plain forms of the operators of the backbone around the TTT layer: the short
causal convolution (forward, backward, single tokens), the selective state space scan
behind it (forward, backward, single tokens), and rotary positions with several axes for
the token grids of images and video.

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

# The largest drawn convolution or rotation: elements of one token tensor (half of the long
# training case's), and the largest drawn scan: elements of the states over all tokens.
MAX_ELEMS = 32768 * 2048
MAX_STATES = 8 * 2048 * 768 * 16


def listed():
    return [
        # one decoding step of 64 sequences, inner width twice the 125M layer's, the last inputs of
        # each sequence kept as its state
        dict(name="conv_decode", op="conv", B=64, T=1, C=1536, K=4, act="silu", bias=True, state=True, reset=False,
             train=False, dtype="bf16"),
        # prefill at the 125M layer's batch and width, states handed to the decoder
        dict(name="conv_125m", op="conv", B=8, T=2048, C=768, K=4, act="silu", bias=True, state=True, reset=False,
             train=False, dtype="bf16"),
        # packed sequences of odd sizes in 32 bits, training, the gradients of the states too
        dict(name="conv_train_odd_f32", op="conv", B=3, T=701, C=1001, K=3, act="none", bias=False, state=True,
             reset=True, train=True, dtype="f32"),
        # training on a long context
        dict(name="conv_train_long", op="conv", B=2, T=32768, C=2048, K=4, act="silu", bias=True, state=False,
             reset=False, train=True, dtype="bf16"),
        # one decoding step of 64 sequences
        dict(name="scan_decode", op="scan", B=64, T=1, C=1536, N=16, G=1, rank=48, softplus=True, gate=True, skip=True,
             reset=False, state=True, train=False, dtype="bf16"),
        # prefill at the 125M layer's batch and length
        dict(name="scan_125m", op="scan", B=8, T=2048, C=1536, N=16, G=1, rank=48, softplus=True, gate=True, skip=True,
             reset=False, state=True, train=False, dtype="bf16"),
        # one long prompt: few channels, many tokens
        dict(name="scan_prompt_long", op="scan", B=1, T=32768, C=2048, N=16, G=1, rank=128, softplus=True, gate=True,
             skip=True, reset=False, state=False, train=False, dtype="bf16"),
        # packed sequences of odd sizes in 32 bits, three groups, training
        dict(name="scan_train_odd_f32", op="scan", B=3, T=701, C=333, N=12, G=3, rank=21, softplus=True, gate=False,
             skip=True, reset=True, state=True, train=True, dtype="f32"),
        # a training step at the 125M layer's batch and length
        dict(name="scan_train_125m", op="scan", B=8, T=2048, C=1536, N=16, G=1, rank=48, softplus=True, gate=True,
             skip=True, reset=False, state=False, train=True, dtype="bf16"),
        # one decoding step of 64 sequences with text and video in their past: time, height and width
        # of each sequence's token are given
        dict(name="axes_decode", op="axes", B=64, T=1, H=12, d=64, sections="16 8 8", layout="blocks",
             interleaved=False, inverse=False, grid="", rows=32768, dtype="bf16"),
        # the vision layer: 14 x 14 tokens an image, height and width each on half of the pairs
        dict(name="axes_vision", op="axes", B=256, T=196, H=6, d=64, sections="16 16", layout="blocks",
             interleaved=False, inverse=False, grid="14 14", rows=14, dtype="bf16"),
        # the gradients' way back at a video of 16 frames of 28 x 28 tokens, the axes in turn over
        # neighbouring pairs
        dict(name="axes_video_inverse", op="axes", B=4, T=16 * 28 * 28, H=12, d=64, sections="12 10 10",
             layout="cyclic", interleaved=True, inverse=True, grid="16 28 28", rows=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + (n % 1024 == 0 and lo < n < hi)  # whole multiples are what the listed cases have


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "axes"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    cap = MAX_ELEMS // 2 if dtype == "f32" else MAX_ELEMS
    if op == "conv":
        C = _log_int(rng, 8, 4096)
        if rng.random() < 0.5:
            C = max(8, C - C % 8)
        T = min(_log_int(rng, 1, 32768), cap // C)
        B = max(1, min(_log_int(rng, 1, 64), cap // (T * C)))
        return dict(op=op, B=B, T=T, C=C, K=rng.choice([2, 3, 4, 4]), act=rng.choice(["none", "silu", "silu"]),
                    bias=rng.random() < 0.7, state=rng.random() < 0.5, reset=rng.random() < 0.4,
                    train=rng.random() < 0.5, dtype=dtype)
    if op == "scan":
        N = rng.choice([1, 4, 8, 12, 16, 16, 16, 24, 32, 64])
        G = rng.choice([1, 1, 1, 2, 3, 4])
        C = G * _log_int(rng, 8, 1024)
        if rng.random() < 0.5:
            C = max(8 * G, C - C % (8 * G))
        cap = MAX_STATES // 2 if dtype == "f32" else MAX_STATES
        T = max(1, min(_log_int(rng, 1, 32768), cap // (C * N)))
        B = max(1, min(_log_int(rng, 1, 64), cap // (T * C * N)))
        return dict(op=op, B=B, T=T, C=C, N=N, G=G, rank=rng.choice([0, 5, 16, 48]), softplus=rng.random() < 0.8,
                    gate=rng.random() < 0.6, skip=rng.random() < 0.7, reset=rng.random() < 0.4,
                    state=rng.random() < 0.5, train=rng.random() < 0.5, dtype=dtype)
    d = rng.choice([16, 20, 32, 48, 64, 64, 80, 96, 128])
    H = rng.choice([1, 2, 3, 5, 6, 12, 24, 31])
    axes = rng.choice([2, 3, 3])
    rot = rng.choice([d, d, d // 2])
    rot = max(2 * axes, rot - rot % 2)
    least = rot // 2 // axes
    sections = [rot // 2 - least * (axes - 1)] + [least] * (axes - 1)
    grid = None
    if rng.random() < 0.6:
        side = [_log_int(rng, 1, 64) for _ in range(2)]
        frames = max(1, min(_log_int(rng, 1, 32), cap // (side[0] * side[1] * H * d)))
        grid = side if axes == 2 else [frames] + side
        T = math.prod(grid)
    else:
        T = min(_log_int(rng, 1, 32768), cap // (H * d))
    B = max(1, min(_log_int(rng, 1, 256), cap // (T * H * d)))
    return dict(op=op, B=B, T=T, H=H, d=d, sections=" ".join(map(str, sections)), layout=rng.choice(["blocks", "cyclic"]),
                interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4,
                grid=" ".join(map(str, grid or [])), rows=max(grid) + _log_int(rng, 1, 4096) if grid else _log_int(rng, 64, 32768), dtype=dtype)


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


def _vec(g, n, mean, std):
    return torch.randn(n, generator=g, device="cuda").mul_(std).add_(mean)


def _ints(text):
    return [int(v) for v in text.split()]


def _pair_axis(sections, layout):
    """The axis of every pair: one block of pairs after the other, or the axes in turn for as
    long as each has pairs left."""
    if layout == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    dt = DT[c["dtype"]]
    s = {"case": c}
    B, T = c["B"], c["T"]
    if c["op"] == "axes":
        H, d, sec = c["H"], c["d"], _ints(c["sections"])
        s["grid"] = _ints(c["grid"]) or None
        if c["inverse"]:
            # gradients in the layer's head-major layout, going to one token-major buffer
            s["q"], s["k"], s["v"] = (_randn(g, (B, H, T, d), dt) for _ in range(3))
        else:
            # one token-major projection of the three
            qkv = _randn(g, (B, T, 3, H, d), dt)
            s["q"], s["k"], s["v"] = qkv.permute(2, 0, 3, 1, 4).unbind(0)
        s["axis"] = _pair_axis(sec, c["layout"])
        # every axis has frequencies of its own, 10000^(-j / pairs) for its j-th pair
        inv, seen = [], [0] * len(sec)
        for a in s["axis"]:
            inv.append(10000.0 ** (-seen[a] / sec[a]))
            seen[a] += 1
        ang = (torch.arange(c["rows"], device="cuda", dtype=torch.float64)[:, None]
               * torch.tensor(inv, device="cuda", dtype=torch.float64))
        s["table"] = torch.stack([ang.cos(), ang.sin()], -1).float()
        s["positions"] = None
        if s["grid"] is None:
            # text and pictures mixed: time never runs back, height and width anywhere
            top = torch.randint(0, c["rows"], (B, T), generator=g, device="cuda").sort(1).values
            rest = [torch.randint(0, min(64, c["rows"]), (B, T), generator=g, device="cuda") for _ in sec[1:]]
            s["positions"] = torch.stack([top, *rest])
        return s
    C = c["C"]
    s["reset"] = None
    if c["reset"]:  # a new sequence about every 200 tokens
        s["reset"] = torch.rand((B, T), generator=g, device="cuda") < 0.005
    if c["op"] == "conv":
        K = c["K"]
        s["x"] = _randn(g, (B, T, C), dt)
        s["weight"] = _vec(g, C * K, 0.0, K ** -0.5).view(C, K)
        s["bias"] = _vec(g, C, 0.0, 0.1) if c["bias"] else None
        s["state"] = _randn(g, (B, K - 1, C), dt) if c["state"] else None
        if c["train"]:
            s["dy"] = _randn(g, (B, T, C), dt)
            s["dstate_out"] = _randn(g, (B, K - 1, C), torch.float32) if c["state"] else None
        return s
    N, G, R = c["N"], c["G"], c["rank"]
    # x and the gate are halves of one projection, B and C lie in another behind the rate's part
    both = _randn(g, (B, T, 2 * C), dt)
    s["x"] = both[..., :C]
    s["z"] = both[..., C:] if c["gate"] else None
    proj = _randn(g, (B, T, R + 2 * G * N), dt)
    s["Bm"] = proj[..., R:R + G * N].unflatten(-1, (G, N))
    s["Cm"] = proj[..., R + G * N:].unflatten(-1, (G, N))
    # rates around 0.001 .. 0.1, decays of the states 1 .. N times as fast
    rate = torch.exp(torch.rand(C, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    s["A"] = -(torch.arange(1, N + 1, device="cuda") * torch.exp(_vec(g, C * N, 0.0, 0.1).view(C, N))).contiguous()
    if c["softplus"]:
        s["delta"] = _randn(g, (B, T, C), dt, 0.0, 0.5)
        s["delta_bias"] = torch.log(torch.expm1(rate))
    else:
        d = torch.empty((B, T, C), device="cuda", dtype=dt)
        for b in range(B):
            d[b] = torch.exp(torch.randn((T, C), generator=g, device="cuda") * 0.5) * rate
        s["delta"], s["delta_bias"] = d, None
    s["D"] = _vec(g, C, 1.0, 0.1) if c["skip"] else None
    s["h0"] = _randn(g, (B, C, N), torch.float32, 0.0, 0.3) if c["state"] else None
    if c["train"]:
        s["dy"] = _randn(g, (B, T, C), dt)
        s["dh_last"] = _randn(g, (B, C, N), torch.float32, 0.0, 0.1) if c["state"] else None
    return s


# -------------------------------------------------------------------- plain forms


def _plain_conv(s):
    c = s["case"]
    B, T, C, K = c["B"], c["T"], c["C"], c["K"]
    dt = DT[c["dtype"]]
    past = torch.zeros((B, K - 1, C), device="cuda", dtype=dt) if s["state"] is None else s["state"]
    rows = torch.cat([past, s["x"]], 1)  # row t + K - 1 is token t
    seq = None
    if s["reset"] is not None:  # which packed sequence a row belongs to
        seq = torch.cat([torch.zeros((B, K - 1), device="cuda", dtype=torch.int64), s["reset"].cumsum(1)], 1)
    pre = torch.zeros((B, T, C), device="cuda") if s["bias"] is None else s["bias"].expand(B, T, C).clone()
    taps = []
    for j in range(K):
        v = rows[:, j:j + T].float()
        if seq is not None:
            v = torch.where((seq[:, j:j + T] == seq[:, K - 1:])[..., None], v, 0.0)
        taps.append(v if c["train"] else None)
        pre += v * s["weight"][:, j]
    sg = torch.sigmoid(pre) if c["act"] == "silu" else None
    last = rows[:, T:]
    if seq is not None:
        last = torch.where((seq[:, T:] == seq[:, -1:])[..., None], last, torch.zeros_like(last))
    out = [(pre if sg is None else pre * sg).to(dt)]
    if c["state"]:
        out.append(last.clone())
    if not c["train"]:
        return out
    dpre = s["dy"].float()
    if sg is not None:
        dpre = dpre * sg * (1 + pre * (1 - sg))
    drows = torch.zeros((B, T + K - 1, C), device="cuda")
    for j in range(K):
        v = dpre * s["weight"][:, j]
        if seq is not None:
            v = torch.where((seq[:, j:j + T] == seq[:, K - 1:])[..., None], v, 0.0)
        drows[:, j:j + T] += v
    if s["dstate_out"] is not None:
        v = s["dstate_out"]
        if seq is not None:
            v = torch.where((seq[:, T:] == seq[:, -1:])[..., None], v, 0.0)
        drows[:, T:] += v
    out += [drows[:, K - 1:].to(dt), torch.stack([(dpre * t).sum((0, 1)) for t in taps], -1)]
    if s["bias"] is not None:
        out.append(dpre.sum((0, 1)))
    if c["state"]:
        out.append(drows[:, :K - 1].clone())
    return out


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from a zero state, by doubling strides."""
    T, n = a.shape[1], 1
    while n < T:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _plain_scan(s):
    c = s["case"]
    B, T, C, N, G = c["B"], c["T"], c["C"], c["N"], c["G"]
    dt = DT[c["dtype"]]
    x, raw = s["x"].float(), s["delta"].float()
    if s["delta_bias"] is not None:
        raw = raw + s["delta_bias"]
    # softplus
    rate = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())) if c["softplus"] else raw
    u = rate * x
    zero = None if s["reset"] is None else s["reset"][..., None]

    def per_channel(m, n):  # [B,T,G,N] -> [B,T,C] of state n
        return m[..., n].float().repeat_interleave(C // G, -1)

    def decays(n):
        a = torch.exp(rate * s["A"][:, n])
        return a, (a if zero is None else a.masked_fill(zero, 0.0))

    def states(n, keep):
        b = u * per_channel(s["Bm"], n)
        if s["h0"] is not None:
            b = torch.cat([b[:, :1] + keep[:, :1] * s["h0"][:, None, :, n], b[:, 1:]], 1)
        return _scan(keep, b)

    pre = torch.zeros((B, T, C), device="cuda") if s["D"] is None else x * s["D"]
    last = torch.empty((B, C, N), device="cuda")
    for n in range(N):
        h = states(n, decays(n)[1])
        last[..., n] = h[:, -1]
        pre += per_channel(s["Cm"], n) * h
    sg = None
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
    out = [(pre if sg is None else pre * (z * sg)).to(dt), last]
    if not c["train"]:
        return out
    dy = s["dy"].float()
    dz = None
    if sg is not None:
        dz = (dy * pre * sg * (1 + z * (1 - sg))).to(dt)
        dy = dy * (z * sg)
    du, drate = torch.zeros_like(u), torch.zeros_like(u)
    dA = torch.empty((C, N), device="cuda")
    dB, dC = (torch.empty((B, T, G, N), device="cuda") for _ in range(2))
    dh0 = torch.empty((B, C, N), device="cuda")
    for n in range(N):
        a, keep = decays(n)
        h = states(n, keep)
        d = dy * per_channel(s["Cm"], n)
        if s["dh_last"] is not None:
            d = torch.cat([d[:, :-1], d[:, -1:] + s["dh_last"][:, None, :, n]], 1)
        nxt = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)  # a_{t+1} on the way back
        S = _scan(nxt.flip(1), d.flip(1)).flip(1)
        dC[..., n] = (dy * h).unflatten(-1, (G, -1)).sum(-1)
        dB[..., n] = (S * u).unflatten(-1, (G, -1)).sum(-1)
        du += S * per_channel(s["Bm"], n)
        first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None, :, n]
        q = S * keep * torch.cat([first, h[:, :-1]], 1)
        drate += q * s["A"][:, n]
        dA[:, n] = (q * rate).sum((0, 1))
        dh0[..., n] = keep[:, 0] * S[:, 0]
    drate += du * x
    dx = du * rate
    if s["D"] is not None:
        dx = dx + dy * s["D"]
    if c["softplus"]:
        drate = drate * torch.sigmoid(raw)
    out += [dx.to(dt), drate.to(dt), dA, dB.to(dt), dC.to(dt)]
    if s["D"] is not None:
        out.append((dy * x).sum((0, 1)))
    if dz is not None:
        out.append(dz)
    if s["delta_bias"] is not None:
        out.append(drate.sum((0, 1)))
    return out + [dh0]


def _grid_positions(s):
    """[axes, B, T]: row-major coordinates of the token grid."""
    t, out = torch.arange(s["case"]["T"], device="cuda"), []
    for n in reversed(s["grid"]):
        out.insert(0, t % n)
        t = t // n
    return torch.stack(out)[:, None].expand(-1, s["case"]["B"], -1)


def _plain_axes(s):
    c = s["case"]
    half = s["table"].shape[1]
    rot = 2 * half
    pos = _grid_positions(s) if s["positions"] is None else s["positions"]
    axis = torch.tensor(s["axis"], device="cuda")
    where = pos[axis].permute(1, 2, 0)  # [B, T, rot / 2]
    cs = s["table"][where, torch.arange(half, device="cuda")][:, None]
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


# ------------------------------------------------------------------------- a pass


def run(s):
    c = s["case"]
    if not own:
        return {"conv": _plain_conv, "scan": _plain_scan, "axes": _plain_axes}[c["op"]](s)
    from test_sequence_layers_gb300 import abi
    if c["op"] == "axes":
        kw = dict(positions=s["positions"], grid=s["grid"], interleaved=c["interleaved"], inverse=c["inverse"])
        if not c["inverse"]:
            return list(abi.ttt_rope_axes(s["q"], s["k"], s["v"], s["table"], s["axis"], **kw))
        B, H, T, d = s["q"].shape
        dqkv = torch.empty((B, T, 3, H, d), device="cuda", dtype=s["q"].dtype)
        dq, dk, dv = dqkv.permute(2, 0, 3, 1, 4).unbind(0)
        abi.ttt_rope_axes(s["q"], s["k"], s["v"], s["table"], s["axis"], q_out=dq, k_out=dk, v_out=dv, **kw)
        return dqkv
    if c["op"] == "conv":
        kw = dict(bias=s["bias"], act=c["act"], reset=s["reset"], state=s["state"])
        y, last = abi.ttt_short_conv_fwd(s["x"], s["weight"], want_state=c["state"], **kw)
        out = [y] if last is None else [y, last]
        if c["train"]:
            g = abi.ttt_short_conv_bwd(s["dy"], s["x"], s["weight"], dstate_out=s["dstate_out"], **kw)
            out += [t for t in g if t is not None]
        return out
    kw = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=c["softplus"], reset=s["reset"])
    y, last, states = abi.ttt_selective_scan_fwd(s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], h0=s["h0"],
                                                 want_states=c["train"], **kw)
    if not c["train"]:
        return [y, last]
    g = abi.ttt_selective_scan_bwd(s["dy"], s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], states,
                                   dh_last=s["dh_last"], **kw)
    return [y, last] + [t for t in g if t is not None]


def work(case):
    c, es = case, ES[case["dtype"]]
    B, T = c["B"], c["T"]
    if c["op"] == "axes":
        n, rot = B * T * c["H"] * c["d"], 2 * sum(_ints(c["sections"]))
        rows = max(_ints(c["grid"])) if c["grid"] else min(c["rows"], B * T)
        return {"bytes": 6 * n * es + rows * rot * 4 + (0 if c["grid"] else 8 * len(_ints(c["sections"])) * B * T),
                "flops": 6 * B * T * c["H"] * rot}
    n = B * T * c["C"]
    marks = B * T if c["reset"] else 0
    if c["op"] == "conv":
        K, C = c["K"], c["C"]
        state = B * (K - 1) * C if c["state"] else 0
        par = C * K * 4 + (C * 4 if c["bias"] else 0)
        act = 5 if c["act"] == "silu" else 0
        if not c["train"]:
            return {"bytes": 2 * n * es + 2 * state * es + par + marks, "flops": (2 * K + act) * n}
        # x and dy read, y and dx written
        return {"bytes": 4 * n * es + 2 * state * es + 8 * state + 2 * par + marks, "flops": (6 * K + 2 * act) * n}
    N, C = c["N"], c["C"]
    bc = 2 * B * T * c["G"] * N
    state = B * C * N * 4
    par = C * N * 4 + C * 4 * (c["softplus"] + c["skip"])
    tensors = 3 + c["gate"]  # x, delta, y and the gate
    # a state: the decay's argument and exponential, its step, its part of the output
    flops = n * (N * 7 + 4 * c["softplus"] + 6 * c["gate"] + 2 * c["skip"])
    if not c["train"]:
        return {"bytes": tensors * n * es + bc * es + state * (1 + c["state"]) + par + marks, "flops": flops}
    # dy read, the gradients of x, delta and the gate written
    tensors += 3 + c["gate"]
    return {"bytes": tensors * n * es + 2 * bc * es + state * (2 + 2 * c["state"]) + 2 * par + marks,
            "flops": flops + n * (N * 16 + 12)}


# ------------------------------------------------------------ the definition, 64 bits


def _silu64(v):
    return v / (1 + torch.exp(-v))


def _exact_conv(s):
    """The definition in 64 bits, one batch entry at a time, gradients by differentiation."""
    c = s["case"]
    B, T, C, K, train = c["B"], c["T"], c["C"], c["K"], c["train"]
    w = s["weight"].double().requires_grad_(train)
    bias = None if s["bias"] is None else s["bias"].double().requires_grad_(train)
    ys, lasts, gx, gs = [], [], [], []
    for b in range(B):
        x = s["x"][b].double().requires_grad_(train)
        past = (torch.zeros((K - 1, C), device="cuda", dtype=torch.float64) if s["state"] is None
                else s["state"][b].double()).requires_grad_(train)
        pos = torch.arange(T, device="cuda")
        # the first row a token may look at: -(K - 1) .. -1 are the state's
        first = torch.full((T,), -(K - 1), device="cuda", dtype=torch.int64)
        if s["reset"] is not None:
            first = torch.where(s["reset"][b], pos, first).cummax(0).values
        y = torch.zeros((T, C), device="cuda", dtype=torch.float64) if bias is None else bias.expand(T, C)
        for back in range(K):
            idx = pos - back
            part = torch.zeros((T, C), device="cuda", dtype=torch.float64)
            inx = (idx >= 0) & (idx >= first)
            part = part.index_put((pos[inx],), x[idx[inx]])
            ins = (idx < 0) & (idx >= first)
            part = part.index_put((pos[ins],), past[idx[ins] + K - 1])
            y = y + w[:, K - 1 - back] * part
        if c["act"] == "silu":
            y = _silu64(y)
        rows = []
        for r in range(T - K + 1, T):  # the last K - 1 rows of the running sequence
            if r < int(first[-1]):
                rows.append(torch.zeros(C, device="cuda", dtype=torch.float64))
            else:
                rows.append(x[r] if r >= 0 else past[r + K - 1])
        last = torch.stack(rows)
        ys.append(y.detach())
        lasts.append(last.detach())
        if train:
            obj = (y * s["dy"][b].double()).sum()
            if s["dstate_out"] is not None:
                obj = obj + (last * s["dstate_out"][b].double()).sum()
            obj.backward()
            gx.append(x.grad)
            gs.append(past.grad)
    out = [torch.stack(ys)] + ([torch.stack(lasts)] if c["state"] else [])
    if train:
        out += [torch.stack(gx), w.grad] + ([] if bias is None else [bias.grad])
        if c["state"]:
            out.append(torch.stack(gs))
    return out


def _exact_scan(s):
    """Token by token in 64 bits, and token by token back."""
    c = s["case"]
    B, T, C, N, G = c["B"], c["T"], c["C"], c["N"], c["G"]
    f64 = dict(device="cuda", dtype=torch.float64)
    A = s["A"].double()
    v = s["delta"].double()
    if s["delta_bias"] is not None:
        v = v + s["delta_bias"].double()
    if c["softplus"]:
        slope = 1 / (1 + torch.exp(-v))
        rate = torch.logaddexp(v, torch.zeros((), **f64))
    else:
        slope, rate = torch.ones((), **f64), v
    x = s["x"].double()
    grp = torch.arange(C, device="cuda") // (C // G)
    live = torch.ones((B, T), **f64) if s["reset"] is None else (~s["reset"]).double()
    gate = dgate = None
    if s["z"] is not None:
        z = s["z"].double()
        e = 1 / (1 + torch.exp(-z))
        gate, dgate = z * e, e + z * e * (1 - e)
    h = torch.zeros((B, C, N), **f64) if s["h0"] is None else s["h0"].double()
    start = h
    raw = torch.empty((B, T, C), **f64)
    H = torch.empty((T, B, C, N), **f64) if c["train"] else None
    for t in range(T):
        a = torch.exp(rate[:, t, :, None] * A) * live[:, t, None, None]
        h = a * h + (rate[:, t] * x[:, t])[..., None] * s["Bm"][:, t].double()[:, grp]
        raw[:, t] = torch.einsum("bcn,bcn->bc", h, s["Cm"][:, t].double()[:, grp])
        if H is not None:
            H[t] = h
    if s["D"] is not None:
        raw += x * s["D"].double()
    out = [raw if gate is None else raw * gate, h]
    if not c["train"]:
        return out
    dy = s["dy"].double()
    dz = None
    if gate is not None:
        dz = dy * raw * dgate
        dy = dy * gate
    r = torch.zeros((B, C, N), **f64) if s["dh_last"] is None else s["dh_last"].double()
    dx, dr = torch.empty((B, T, C), **f64), torch.empty((B, T, C), **f64)
    dA = torch.zeros((C, N), **f64)
    dBm, dCm = torch.empty((B, T, G, N), **f64), torch.empty((B, T, G, N), **f64)
    for t in range(T - 1, -1, -1):
        Bt, Ct = s["Bm"][:, t].double()[:, grp], s["Cm"][:, t].double()[:, grp]
        dCm[:, t] = (dy[:, t, :, None] * H[t]).view(B, G, C // G, N).sum(2)
        r = r + dy[:, t, :, None] * Ct
        dBm[:, t] = (r * (rate[:, t] * x[:, t])[..., None]).view(B, G, C // G, N).sum(2)
        into = (r * Bt).sum(-1)
        r = r * torch.exp(rate[:, t, :, None] * A) * live[:, t, None, None]
        q = r * (H[t - 1] if t else start)
        dr[:, t] = (q * A).sum(-1) + into * x[:, t]
        dA += (q * rate[:, t, :, None]).sum(0)
        dx[:, t] = into * rate[:, t]
    dr = dr * slope
    if s["D"] is not None:
        dx = dx + dy * s["D"].double()
    out += [dx, dr, dA, dBm, dCm]
    if s["D"] is not None:
        out.append((dy * x).sum((0, 1)))
    if dz is not None:
        out.append(dz)
    if s["delta_bias"] is not None:
        out.append(dr.sum((0, 1)))
    return out + [r]


def _exact_axes(s):
    c = s["case"]
    B, T = c["B"], c["T"]
    tab = s["table"].double()
    rot = 2 * tab.shape[1]
    z = torch.complex(tab[..., 0], tab[..., 1])  # a rotation is a complex factor
    if c["inverse"]:
        z = z.conj()
    first = torch.arange(0, rot, 2, device="cuda") if c["interleaved"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if c["interleaved"] else rot // 2)
    out = [t.double().clone() for t in (s["q"], s["k"], s["v"])]
    for p, a in enumerate(s["axis"]):
        if s["positions"] is not None:
            where = s["positions"][a]
        else:
            coord = np.unravel_index(np.arange(T), s["grid"])[a]
            where = torch.from_numpy(coord).cuda().expand(B, T)
        f = z[where, p][:, None]
        i, j = int(first[p]), int(second[p])
        for o in out[:2]:
            r = torch.complex(o[..., i], o[..., j]) * f
            o[..., i], o[..., j] = r.real, r.imag
    if c["inverse"]:
        return torch.stack(out).permute(1, 3, 0, 2, 4).contiguous()
    return [o.contiguous() for o in out]


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "axes": _exact_axes}[case["op"]](s)
