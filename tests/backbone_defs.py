"""The short convolution and the selective scan token by token in 64 bits, on any device, with
bounds on how far the arithmetic of the kernels may be from them.

E is 2^-20: 32-bit products, sums, exponentials and quotients in the short chains that make
one rate, gate or tap (each within 2^-22, fewer than four in a row; an exponential's argument
carries its own rounding into the result, E times its size).  A sum of n terms adds n 2^-24 of
the sum of their sizes.  What an output rounds to its own type is added by `bound`."""
import torch

E = 2.0 ** -20


def bound(ref, dtype, slack):
    """|got - ref| allowed: half a step of the output's type and the arithmetic's part."""
    return torch.finfo(dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -6) + slack


def check(name, got, ref, slack):
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    got = got.double().to(ref.device)
    assert bool(torch.isfinite(got).all()), name
    # (a result below the type's normal range is held to its smallest step)
    over = (got - ref).abs() - slack - 1e-36
    worst = float((over / (ref.abs() + slack + 1e-30)).max()) if ref.numel() else 0.0
    assert bool((over <= 0).all()), (name, worst)


def close(name, got, ref, slack):
    check(name, got, ref, bound(ref, got.dtype, slack))


def conv(i):
    """{output: (value, slack)} of inputs x, weight, bias, act, reset, state, dy, dstate_out."""
    d = lambda t: None if t is None else t.double()
    x, w, b, st, dy, dso = (d(i.get(n)) for n in ("x", "weight", "bias", "state", "dy", "dstate_out"))
    B, T, C = x.shape
    K = w.shape[1]
    rows = torch.cat([x.new_zeros(B, K - 1, C) if st is None else st, x], 1)
    first = torch.full((B, T), -(K - 1), dtype=torch.int64, device=x.device)  # the earliest row a token sees
    if i.get("reset") is not None:
        for t in range(T):
            if t:
                first[:, t] = first[:, t - 1]
            first[:, t] = torch.where(i["reset"][:, t].bool(), torch.full_like(first[:, t], t), first[:, t])
    pre = torch.zeros_like(x) + (0 if b is None else b)
    mag = pre.abs()
    t_ = torch.arange(T, device=x.device)
    see = [((t_ + j - (K - 1))[None] >= first)[..., None] for j in range(K)]  # tap j of every token
    for j in range(K):
        v = torch.where(see[j], rows[:, j:j + T], torch.zeros_like(x))
        pre = pre + w[:, j] * v
        mag = mag + (w[:, j] * v).abs()
    s = torch.sigmoid(pre)
    silu = i["act"] == "silu"
    y = pre * s if silu else pre
    out = {"y": (y, E * mag)}
    last = rows[:, T:].clone()
    keep = (torch.arange(T - K + 1, T, device=x.device)[None] >= first[:, -1:])[..., None] if T else None
    if T:
        last = torch.where(keep, last, torch.zeros_like(last))
    out["state_out"] = (last, torch.zeros_like(last))
    if dy is None:
        return out
    g = dy * s * (1 + pre * (1 - s)) if silu else dy
    gm = dy.abs() * (1 + mag)
    drows, dmag = torch.zeros_like(rows), torch.zeros_like(rows)
    dw, dwm = [], []
    for j in range(K):
        z = torch.zeros_like(x)
        drows[:, j:j + T] += torch.where(see[j], w[:, j] * g, z)
        dmag[:, j:j + T] += torch.where(see[j], w[:, j].abs() * gm, z)
        v = torch.where(see[j], rows[:, j:j + T], z)
        dw.append((g * v).sum((0, 1)))
        dwm.append((gm * v.abs()).sum((0, 1)))
    if dso is not None:
        drows[:, T:] += torch.where(keep, dso, torch.zeros_like(dso))
        dmag[:, T:] += dso.abs()
    many = (256 + B * T / 256) * 2.0 ** -24  # terms summed one after the other
    out["dx"] = (drows[:, K - 1:], 2 * E * dmag[:, K - 1:])
    out["dweight"] = (torch.stack(dw, -1), (2 * E + many) * torch.stack(dwm, -1))
    out["dbias"] = (g.sum((0, 1)), (2 * E + many) * gm.sum((0, 1)))
    out["dstate"] = (drows[:, :K - 1], 2 * E * dmag[:, :K - 1])
    return out


def scan(i):
    """{output: (value, slack)} of inputs x, delta, A, B, C ([B,T,G,N]), D, z, delta_bias,
    softplus, reset, h0, dy, dh_last."""
    d = lambda t: None if t is None else t.double()
    x, dl, A, Bm, Cm, D, z, bias, h0, dy, dhl = (d(i.get(n)) for n in ("x", "delta", "A", "B", "C", "D", "z", "delta_bias",
                                                                      "h0", "dy", "dh_last"))
    nb, T, C = x.shape
    N, G = A.shape[1], Bm.shape[2]
    rep = lambda m: m.repeat_interleave(C // G, 2)  # [B,T,C,N]
    Bc, Cc = rep(Bm), rep(Cm)
    v = dl + (0 if bias is None else bias)
    rate = torch.nn.functional.softplus(v, threshold=1e9) if i["softplus"] else v
    slope = torch.sigmoid(v) if i["softplus"] else torch.ones_like(v)
    # a softplus' argument is rounded once: its part of the rate
    err_rate = E * rate.abs() + 2.0 ** -23 * v.abs() * slope
    u = rate * x
    err_u = E * u.abs() + err_rate * x.abs()
    live = torch.ones(nb, T, 1, 1, dtype=x.dtype, device=x.device)
    if i.get("reset") is not None:
        live = 1.0 - i["reset"].double()[:, :, None, None]
    # decays, and the size of their relative error
    def decay(t):
        arg = rate[:, t, :, None] * A
        return torch.exp(arg) * live[:, t], E * (1 + arg.abs()) + (err_rate[:, t, :, None] * A.abs())
    h = x.new_zeros(nb, C, N) if h0 is None else h0
    hm, he = h.abs(), torch.zeros_like(h)
    H, HM, HE, Y, YM = [], [], [], [], []
    for t in range(T):
        H.append(h), HM.append(hm), HE.append(he)  # before the token
        a, ra = decay(t)
        b = u[:, t, :, None] * Bc[:, t]
        he = a * he + a * hm * ra + err_u[:, t, :, None] * Bc[:, t].abs() + E * b.abs()
        h = a * h + b
        hm = a * hm + b.abs()
        Y.append((Cc[:, t] * h).sum(-1))
        YM.append((Cc[:, t].abs() * (he + (E + N * 2.0 ** -24) * hm)).sum(-1))
    H.append(h), HM.append(hm), HE.append(he)
    zero = x.new_zeros(nb, 0, C)
    pre = torch.stack(Y, 1) if T else zero
    pm = torch.stack(YM, 1) if T else zero
    if D is not None:
        pre, pm = pre + D * x, pm + E * (D * x).abs()
    pm = pm + E * pre.abs()
    gate = dgate = None
    if z is not None:
        s = torch.sigmoid(z)
        gate, dgate = z * s, s * (1 + z * (1 - s))
    out = {"y": (pre, pm) if gate is None else (pre * gate, pm * gate.abs() + E * (1 + z.abs()) * (pre * gate).abs()),
           "h_last": (h, he + E * hm)}
    if dy is None:
        return out
    g, gm = dy, dy.abs()
    if gate is not None:
        out["dz"] = (dy * pre * dgate, dy.abs() * (pm * dgate.abs() + 4 * E * (1 + z.abs()) * (pre.abs() + pm)))
        g, gm = dy * gate, (dy * gate).abs()
    eg = E * (1 + (0 if z is None else z.abs())) * gm
    r = x.new_zeros(nb, C, N) if dhl is None else dhl
    rm, re = r.abs(), torch.zeros_like(r)
    groups = lambda m: m.view(nb, G, C // G, N).sum(2)
    names = ("dx", "ddelta", "dB", "dC")
    val, tol = {n: [None] * T for n in names}, {n: [None] * T for n in names}
    dA, tA = torch.zeros_like(A), torch.zeros_like(A)
    chans = C // G * 2.0 ** -24
    many = (256 + nb * T / 32) * 2.0 ** -24
    for t in range(T - 1, -1, -1):
        gt, Ct, Bt = g[:, t, :, None], Cc[:, t], Bc[:, t]
        a, ra = decay(t)
        s = r + gt * Ct
        sm = rm + gm[:, t, :, None] * Ct.abs()
        se = re + eg[:, t, :, None] * Ct.abs() + E * sm
        val["dC"][t] = groups(gt * H[t + 1])
        tol["dC"][t] = groups(gm[:, t, :, None] * (HE[t + 1] + (E + chans) * HM[t + 1]) + eg[:, t, :, None] * HM[t + 1])
        ut = u[:, t, :, None]
        val["dB"][t] = groups(s * ut)
        tol["dB"][t] = groups(se * ut.abs() + sm * ((E + chans) * ut.abs() + err_u[:, t, :, None]))
        e, em = (s * Bt).sum(-1), ((se + (E + N * 2.0 ** -24) * sm) * Bt.abs()).sum(-1)
        eabs = (sm * Bt.abs()).sum(-1)
        p = H[t] * live[:, t]
        q = a * s * p
        qm = a * sm * HM[t]
        qe = a * (sm * HE[t] + se * HM[t]) + qm * (ra + E)
        dd = e * x[:, t] + (q * A).sum(-1)
        dde = em * x[:, t].abs() + ((qe + (E + N * 2.0 ** -24) * qm) * A.abs()).sum(-1) + E * (eabs * x[:, t].abs())
        val["dx"][t] = e * rate[:, t] + (0 if D is None else g[:, t] * D)
        tol["dx"][t] = (em * rate[:, t].abs() + eabs * err_rate[:, t] + E * (eabs * rate[:, t].abs())
                        + (0 if D is None else (eg[:, t] + E * gm[:, t]) * D.abs()))
        val["ddelta"][t] = dd * slope[:, t]
        big = eabs * x[:, t].abs() + (qm * A.abs()).sum(-1)
        tol["ddelta"][t] = (dde + (E + 2.0 ** -23 * v[:, t].abs()) * big) * slope[:, t]
        dA = dA + (q * rate[:, t, :, None]).sum(0)
        tA = tA + (qe * rate[:, t, :, None].abs() + qm * (err_rate[:, t, :, None] + (E + many) * rate[:, t, :, None].abs())).sum(0)
        r, rm, re = a * s, a * sm, a * (se + sm * ra)
    for n in names:
        shape = (nb, 0, C) if n in ("dx", "ddelta") else (nb, 0, G, N)
        out[n] = (torch.stack(val[n], 1), torch.stack(tol[n], 1)) if T else (x.new_zeros(shape),) * 2
    out["dA"] = (dA, tA)
    if D is not None:
        out["dD"] = ((g * x).sum((0, 1)), (eg * x.abs()).sum((0, 1)) + (E + many) * (gm * x.abs()).sum((0, 1)))
    if bias is not None:
        out["ddelta_bias"] = (out["ddelta"][0].sum((0, 1)),
                              out["ddelta"][1].sum((0, 1)) + many * out["ddelta"][0].abs().sum((0, 1)))
    out["dh0"] = (r, re + E * rm)
    return out


def conv_inputs(B, T, C, K, dtype=torch.bfloat16, act="silu", bias=True, state=True, resets=0.0, train=True, seed=0,
                device="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    i = {"x": r(B, T, C).to(dtype), "weight": r(C, K) / K ** 0.5, "bias": 0.1 * r(C) if bias else None, "act": act,
         "state": r(B, K - 1, C).to(dtype) if state else None,
         "reset": torch.rand(B, T, generator=g) < resets if resets else None,
         "dy": r(B, T, C).to(dtype) if train else None, "dstate_out": r(B, K - 1, C) if train and state else None}
    return {k: t.to(device) if isinstance(t, torch.Tensor) else t for k, t in i.items()}


def scan_inputs(B, T, C, N, G=1, dtype=torch.bfloat16, softplus=True, gate=True, skip=True, resets=0.0, state=True,
                train=True, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    rate = torch.exp(torch.rand(C, generator=g) * 4.6 - 6.9)
    i = {"x": r(B, T, C), "z": r(B, T, C) if gate else None, "B": r(B, T, G, N), "C": r(B, T, G, N),
         "dy": r(B, T, C) if train else None,
         "delta": 0.5 * r(B, T, C) if softplus else torch.exp(0.5 * r(B, T, C)) * rate}
    i = {k: None if t is None else t.to(dtype) for k, t in i.items()}
    i.update(A=-torch.arange(1, N + 1) * torch.exp(0.1 * r(C, N)), D=1 + 0.1 * r(C) if skip else None,
             delta_bias=torch.log(torch.expm1(rate)) if softplus else None, softplus=softplus,
             h0=0.3 * r(B, C, N) if state else None, dh_last=0.1 * r(B, C, N) if train and state else None,
             reset=torch.rand(B, T, generator=g) < resets if resets else None)
    return {k: t.to(device) if isinstance(t, torch.Tensor) else t for k, t in i.items()}
