"""The layer for a few tokens stated plainly in 64 bits, its inputs, and the bound that the
arithmetic of its kernels gives."""
import torch

FP8 = torch.float8_e4m3fn


def route(z, bias, K, router):
    """(experts [T][K], weights, the least gap between neighbouring keys at and above the cut)"""
    b = 0 if bias is None else bias.double()
    a = torch.sigmoid(z) if router == "sigmoid" else z + b
    key = a + b if router == "sigmoid" else a
    s = torch.sort(key, dim=1, descending=True, stable=True)
    idx = s.indices[:, :K]
    gap = float("inf")
    if z.shape[1] > K:
        gap = (s.values[:, K - 1] - s.values[:, K]).min().item()
    v = a.gather(1, idx)
    w = v / (v.sum(1, keepdim=True) + 1e-6) if router == "sigmoid" else torch.softmax(v, 1)
    return idx, w, gap


def inputs(T, d, E, K, I, Is, router, fmt, seed, bias=True, residual=True, same=False):  # noqa: E741
    """A layer whose choice of experts is clear at fp32 precision (tokens are drawn again until
    it is).  same: every token is the same row."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    c = dict(T=T, d=d, E=E, K=K, I=I, Is=Is, router=router, fmt=fmt)
    c["w_g"] = (rnd(E, d) / d ** 0.5).bfloat16()
    c["bias"] = 0.1 * rnd(E) if bias else None
    x = torch.empty(T, d, dtype=torch.bfloat16)
    for t in range(T):
        for _ in range(1000):
            x[t] = x[0] if same and t else rnd(d).bfloat16()
            z = x[t:t + 1].double() @ c["w_g"].double().T
            if route(z, c["bias"], K, router)[2] > 1e-4:
                break
    c["x"] = x
    c["residual"] = rnd(T, d).bfloat16() if residual else None
    for n, rows, cols, lead in (("w_gate", I, d, [E]), ("w_up", I, d, [E]), ("w_down", d, I, [E]),
                                ("ws_gate", Is, d, []), ("ws_up", Is, d, []), ("ws_down", d, Is, [])):
        if not rows or not cols:
            continue
        v = rnd(*lead, rows, cols) / cols ** 0.5
        if fmt == "bf16":
            c[n] = v.bfloat16()
            continue
        if fmt == "fp8":
            s = v.abs().amax(-1, keepdim=True) / 448
            c[n], c["s" + n[1:]] = (v / s).to(FP8).view(torch.uint8), s[..., 0].contiguous()
        else:
            b = v.view(*lead, rows // 128, 128, cols // 128, 128)
            s = b.abs().amax((-3, -1), keepdim=True) / 448
            c[n] = (b / s).reshape(v.shape).to(FP8).view(torch.uint8)
            c["s" + n[1:]] = s[..., 0, :, 0].contiguous()
    return c


def matrix(c, n, e=None):
    w = c[n] if e is None else c[n][e]
    if c["fmt"] == "bf16":
        return w.double()
    s = c["s" + n[1:]] if e is None else c["s" + n[1:]][e]
    w, s = w.view(FP8).double(), s.double()
    if c["fmt"] == "fp8":
        return w * s[:, None]
    return w * s.repeat_interleave(128, 0).repeat_interleave(128, 1)


def layer(c):
    """(y, bound of its error): with M the magnitudes that a sum adds, a sum on the tensor
    cores is off by (n / 16 + 32) 2^-23 M (an add a product of 16 terms, the parts and planes
    after it, each losing at most a last place); x 2^-21 of the row's largest value under 8-bit
    weights (half a step of the second plane, 2^-10 / 16, of a scale below 1 / 224 of it); SiLU 2^-20 of it; h 2^-16 (bf16) or 2^-12 of its value and, with 8-bit weights,
    2^-21 of the largest of its 128 (448 steps of a scale, the third plane's half step 2^-10
    finer by 16^2); a routing weight 2^-18; y rounded once, 2^-8."""
    x, T = c["x"].double(), c["T"]
    idx, w, gap = route(x @ c["w_g"].double().T, c["bias"], c["K"], c["router"])
    assert gap > 1e-4
    y = torch.zeros_like(x) if c["residual"] is None else c["residual"].double().clone()
    tol = 2.0 ** -22 * y.abs()
    eight = c["fmt"] != "bf16"
    for e in ([None] if c["Is"] else []) + sorted(set(idx.flatten().tolist())):
        t = list(range(T)) if e is None else [i for i in range(T) if e in idx[i].tolist()]
        pre = "ws_" if e is None else "w_"
        wt = torch.ones(T, 1, dtype=torch.float64) if e is None else \
            torch.stack([w[i, idx[i].tolist().index(e)] for i in t])[:, None]
        gate, up, down = (matrix(c, pre + n, e) for n in ("gate", "up", "down"))
        xr = x[t]
        g, u = xr @ gate.T, xr @ up.T
        act = torch.nn.functional.silu(g)
        h = act * u
        cx = (c["d"] / 16 + 32) * 2.0 ** -23
        off_x = xr.abs() * cx
        if eight:
            off_x = off_x + xr.abs().amax(1, keepdim=True) * 2.0 ** -21
        dg, du = off_x @ gate.abs().T, off_x @ up.abs().T
        n = h.shape[1]
        dh = 1.1 * u.abs() * dg + act.abs() * du + h.abs() * 2.0 ** -20
        dh = dh + h.abs() * ((n / 16 + 32) * 2.0 ** -23 + (2.0 ** -12 if eight else 2.0 ** -16))
        if eight:
            top = h.abs().view(len(t), n // 128, 128).amax(2, keepdim=True)
            dh = dh + (top * 2.0 ** -21).expand(-1, -1, 128).reshape(h.shape)
        o = h @ down.T
        y[t] += wt * o
        tol[t] += wt * (dh @ down.abs().T + 2.0 ** -18 * (h.abs() @ down.abs().T))
    return y, tol + 2.0 ** -8 * (y.abs() + tol)
