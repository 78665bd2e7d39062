"""What a router is trained with, as measurable cases: the balance loss with its
per-expert counts, its gradient joined with that of the routing weights, dropout
from a counter-based generator (alone and in the combine), and the combine's
backward pass.

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()`
makes the inputs, `run()` makes one pass: in elementary torch operations, or
through the framework's entry points where `own` is true.  `exact()` is the
operators' definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

# A case's fields:
#   op      balance | route_grad | dropout | combine | combine_grad
#   T, E, K, d    tokens, experts, experts per token, width
#   router  softmax | sigmoid      dtype   bf16 | f32 (rows; scores are fp32)
#   seqs    sequences packed in the batch (0: the batch is one sequence)
#   pad     share of the tokens that are padding (masked)
#   gate, balance   which gradients route_grad joins
#   shared, residual, rows   optional operands; rows: combine_grad also gives d_y_perm
#   p       dropout probability


def listed():
    return [
        # one small fp32 layer's step: a launch or two, latency alone
        dict(name="balance_tiny", op="balance", T=64, E=8, K=2, router="softmax", seqs=0, pad=0.0),
        # a packed prefill-sized batch of sequences, the loss per sequence, with padding
        dict(name="balance_packed", op="balance", T=16384, E=256, K=8, router="sigmoid", seqs=16,
             pad=0.05),
        # a long-context training batch: the largest scores matrix
        dict(name="balance_long", op="balance", T=131072, E=256, K=8, router="sigmoid", seqs=64,
             pad=0.0),
        # few experts, the whole batch as one sequence, both gradients
        dict(name="route_grad_few", op="route_grad", T=4096, E=8, K=2, router="softmax", seqs=0,
             pad=0.0, gate=True, balance=True),
        # many experts, packed sequences with padding, both gradients
        dict(name="route_grad_packed", op="route_grad", T=16384, E=256, K=8, router="sigmoid",
             seqs=16, pad=0.05, gate=True, balance=True),
        # an odd token count and an expert count that is no power of two; the loss alone
        dict(name="route_grad_odd", op="route_grad", T=40009, E=60, K=6, router="softmax", seqs=7,
             pad=0.0, gate=False, balance=True),
        # hidden rows of one small step, with the residual stream
        dict(name="dropout_step", op="dropout", T=8, d=7168, dtype="bf16", residual=True, p=0.1),
        # hidden rows of a prefill-sized batch
        dict(name="dropout_batch", op="dropout", T=16384, d=7168, dtype="bf16", residual=True,
             p=0.1),
        # the small fp32 layer's combine
        dict(name="combine_tiny", op="combine", T=64, E=8, K=2, d=256, dtype="f32", shared=False,
             residual=True, p=0.1),
        # a prefill-sized batch over many experts, shared expert and residual
        dict(name="combine_batch", op="combine", T=16384, E=256, K=8, d=7168, dtype="bf16",
             shared=True, residual=True, p=0.1),
        # few experts: two rows a token
        dict(name="combine_grad_few", op="combine_grad", T=4096, E=8, K=2, d=4096, dtype="bf16",
             shared=False, rows=True, p=0.1),
        # the prefill-sized batch's backward: every expert row read and its gradient written
        dict(name="combine_grad_batch", op="combine_grad", T=16384, E=256, K=8, d=7168,
             dtype="bf16", shared=True, rows=True, p=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "route_grad", "dropout", "combine", "combine_grad"])
    if op in ("balance", "route_grad"):
        E = rng.choice([8, 64, 256, _log_int(rng, 2, 1024)])
        K = rng.randint(1, min(E, 12))
        T = _log_int(rng, 1, max(1, min(131072, 131072 * 256 // E)))
        c = dict(op=op, T=T, E=E, K=K, router=rng.choice(["softmax", "sigmoid"]),
                 seqs=rng.choice([0, 1, _log_int(rng, 2, 512)]), pad=rng.choice([0.0, 0.0, 0.1]))
        if op == "route_grad":
            c["gate"], c["balance"] = rng.choice([(True, True), (True, True), (True, False),
                                                  (False, True)])
        return c
    dtype = rng.choice(["bf16", "bf16", "f32"])
    p = rng.choice([0.0, 0.1, 0.2, rng.uniform(0.01, 0.6)])
    if op == "dropout":
        d = _log_int(rng, 1, 16384)
        T = _log_int(rng, 1, max(1, min(131072, 16384 * 7168 // (d * (2 if dtype == "f32" else 1)))))
        return dict(op=op, T=T, d=d, dtype=dtype, residual=rng.random() < 0.5, p=p)
    E = rng.choice([8, 64, 256])
    K = rng.randint(1, 8)
    d = 64 * _log_int(rng, 1, 256)
    most = 16384 * 7168 * 8 // (d * K * (2 if dtype == "f32" else 1))
    T = _log_int(rng, 1, max(1, min(32768, most)))
    c = dict(op=op, T=T, E=E, K=K, d=d, dtype=dtype, shared=rng.random() < 0.5, p=p)
    if op == "combine":
        c["residual"] = rng.random() < 0.7
    else:
        c["rows"] = rng.random() < 0.7
    return c


ALPHA = 0.01    # weight of the balance loss
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
MASK = 0xFFFFFFFF


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _cuts(T, n, seed):
    """n sequences over T tokens, ragged, some of them empty."""
    r = np.random.RandomState(seed % (2 ** 31))
    at = np.sort(r.randint(0, T + 1, n - 1)) if n > 1 else np.zeros(0, np.int64)
    return np.concatenate([[0], at, [T]]).astype(np.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    if op in ("balance", "route_grad"):
        T, E, K = case["T"], case["E"], case["K"]
        # scores with a popularity that falls off over the experts, as an untrained
        # or drifting router gives
        pop = torch.arange(1, E + 1, device="cuda").float().log().mul_(-0.4)
        pop = pop[torch.randperm(E, generator=g, device="cuda")]
        z = rnd(T, E).add_(pop)
        s["logits"] = z
        s["topk_idx"] = z.topk(K, dim=1).indices.to(torch.int32)
        s["mask"] = None
        if case["pad"] > 0:
            s["mask"] = (torch.rand(T, generator=g, device="cuda") >= case["pad"]).to(torch.uint8)
        s["seq"] = None
        if case["seqs"] > 0:
            s["seq"] = torch.from_numpy(_cuts(T, case["seqs"], seed)).cuda()
        if op == "route_grad":
            # gradients of a loss that is a mean over the tokens
            s["d_topk_w"] = rnd(T, K).mul_(0.05 / T) if case["gate"] else None
            s["d_loss"] = torch.ones(1, device="cuda")
            s["counts"] = _counts(s) if case["balance"] else None
        return s
    dt = TORCH[case["dtype"]]
    T, d = case["T"], case["d"]
    s["rng"] = torch.tensor([0x1234567 * (seed + 1) % (1 << 62), (40 * seed + 3) % (1 << 62)],
                            device="cuda")
    if op == "dropout":
        s["x"] = rnd(T, d).to(dt)
        s["residual"] = rnd(T, d).to(dt) if case["residual"] else None
        return s
    E, K = case["E"], case["K"]
    z = rnd(T, E)
    top = z.topk(K, dim=1)
    s["topk_w"] = torch.softmax(top.values, dim=1)
    order = torch.argsort(top.indices.reshape(-1), stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * K, device="cuda")
    s["inv_perm"] = inv.to(torch.int32)
    y_perm = torch.empty(T * K, d, dtype=dt, device="cuda")
    for r in range(0, T * K, 16384):  # no fp32 copy of the whole
        y_perm[r:r + 16384] = rnd(min(16384, T * K - r), d)
    s["y_perm"] = y_perm
    if op == "combine":
        s["y_shared"] = rnd(T, d).to(dt) if case["shared"] else None
        s["residual"] = rnd(T, d).to(dt) if case["residual"] else None
    else:
        s["d_y"] = rnd(T, d).to(dt)
    return s


# ---- the plain forms --------------------------------------------------------

def _seq_of(s):
    """(sequence of each token, number of sequences)."""
    T = s["T"]
    if s["seq"] is None:
        return torch.zeros(T, dtype=torch.int64, device="cuda"), 1
    cu = s["seq"].long()
    t = torch.arange(T, device="cuda")
    return torch.searchsorted(cu, t, right=True) - 1, cu.numel() - 1


def _counts(s):
    seq, n = _seq_of(s)
    one = torch.ones_like(s["topk_idx"])
    if s["mask"] is not None:
        one = one * (s["mask"] != 0).int()[:, None]
    at = seq[:, None] * s["E"] + s["topk_idx"].long()
    out = torch.zeros(n * s["E"], dtype=torch.int32, device="cuda")
    return out.scatter_add_(0, at.reshape(-1), one.reshape(-1)).view(n, s["E"])


def _probs(s):
    z = s["logits"]
    if s["router"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    a = 1 / (1 + torch.exp(-z))
    return a / a.sum(1, keepdim=True)


def _balance(s):
    E, K = s["E"], s["K"]
    seq, n = _seq_of(s)
    counts = _counts(s)
    p = _probs(s)
    if s["mask"] is not None:
        p = p * (s["mask"] != 0)[:, None]
    member = (seq == torch.arange(n, device="cuda")[:, None]).float()
    tokens = (counts.sum(1, keepdim=True) // K).clamp(min=1)
    mean = member @ p / tokens
    freq = counts.double() * E / (K * tokens)
    loss = ALPHA / n * (freq * mean).sum()
    return counts, mean, loss.float().reshape(1)


def _route_grad(s):
    z, E, K = s["logits"], s["E"], s["K"]
    idx = s["topk_idx"].long()
    seq, n = _seq_of(s)
    out = torch.zeros_like(z)
    if s["counts"] is not None:
        c = s["counts"].double()
        tokens = (c.sum(1, keepdim=True) / K).clamp(min=1)
        coef = (s["d_loss"].double() * ALPHA / n * E * c / (K * tokens * tokens)).float()
        g = coef[seq]
        p = _probs(s)
        out = p * (g - (p * g).sum(1, keepdim=True))
        if s["router"] == "sigmoid":
            out = out / (1 + torch.exp(z))
    if s["d_topk_w"] is not None:
        dw = s["d_topk_w"]
        zk = z.gather(1, idx)
        if s["router"] == "softmax":
            e = torch.exp(zk - zk.amax(1, keepdim=True))
            w = e / e.sum(1, keepdim=True)
            dz = w * (dw - (w * dw).sum(1, keepdim=True))
        else:
            a = 1 / (1 + torch.exp(-zk))
            tot = a.sum(1, keepdim=True) + 1e-6
            dz = a / (1 + torch.exp(zk)) * (dw - (a / tot * dw).sum(1, keepdim=True)) / tot
        out = out.scatter_add(1, idx, dz)
    if s["mask"] is not None:
        out = out * (s["mask"] != 0)[:, None]
    return out


def _drop_threshold(p):
    return int(p * 65536 + 0.5)


def _mulhilo(m, x):
    """High and low 32 bits of m * x for 32-bit values held in 64-bit signed ones."""
    top = m * (x >> 16)
    low = m * (x & 0xFFFF)
    return (top + (low >> 16)) >> 16, ((top << 16) + low) & MASK


def _keep(n, p, rng):
    """The elements that stay: 16 bits an element from Philox4x32-10 (Salmon, Moraes,
    Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), the counter
    (element / 8, offset), the key the seed."""
    g = torch.arange((n + 7) // 8, device="cuda")
    c0, c1, c2, c3 = g & MASK, g >> 32, rng[1] & MASK, (rng[1] >> 32) & MASK
    k0, k1 = rng[0] & MASK, (rng[0] >> 32) & MASK
    for _ in range(10):
        h0, l0 = _mulhilo(0xD2511F53, c0)
        h1, l1 = _mulhilo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    w = torch.stack([c0, c1, c2, c3], 1)
    u = torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]
    return u >= _drop_threshold(p)


def _dropped(v, s):
    """v after dropout, in fp32."""
    thr = _drop_threshold(s["p"])
    if thr == 0:
        return v
    keep = _keep(v.numel(), s["p"], s["rng"]).view(v.shape)
    return torch.where(keep, v * (65536 / max(65536 - thr, 1)), torch.zeros_like(v))


def _dropout(s):
    y = _dropped(s["x"].float(), s)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _combine(s):
    T, K, d = s["T"], s["K"], s["d"]
    rows = s["y_perm"][s["inv_perm"].long()].view(T, K, d).float()
    y = (rows * s["topk_w"][:, :, None]).sum(1)
    if s["y_shared"] is not None:
        y = y + s["y_shared"].float()
    y = _dropped(y, s)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["y_perm"].dtype)


def _combine_grad(s):
    T, K, d = s["T"], s["K"], s["d"]
    dt, inv = s["y_perm"].dtype, s["inv_perm"].long()
    dz = _dropped(s["d_y"].float(), s)
    rows = s["y_perm"][inv].view(T, K, d).float()
    out = {"d_topk_w": (rows * dz[:, None]).sum(2)}
    if s["rows"]:
        out["d_y_perm"] = torch.empty_like(s["y_perm"])
        out["d_y_perm"][inv] = (s["topk_w"][:, :, None] * dz[:, None]).to(dt).view(T * K, d)
    if s["shared"]:
        out["d_shared"] = dz.to(dt)
    return out


# ---- through the framework --------------------------------------------------

def _shape(s):
    import sparse_expert_ffn_moe_gb300 as moe
    if "shape" not in s:
        s["shape"] = moe.make_shape(s["T"], s.get("d", 64), s.get("E", 1), s.get("K", 1), 64, 0,
                                    s.get("dtype", "f32"), s.get("router", "softmax"))
    return moe, s["shape"]


def _own_balance(s):
    moe, shape = _shape(s)
    n = max(1, s["seqs"])
    if "workspace" not in s:
        s["workspace"] = moe.alloc_balance_workspace(shape, n)
    counts = torch.empty(n, s["E"], dtype=torch.int32, device="cuda")
    mean = torch.empty(n, s["E"], device="cuda")
    loss = torch.empty(1, device="cuda")
    moe.moe_balance_loss(shape, s["logits"], s["topk_idx"], s["mask"], s["seq"], ALPHA, counts,
                         mean, loss, s["workspace"])
    return counts, mean, loss


def _own_route_grad(s):
    moe, shape = _shape(s)
    out = torch.empty_like(s["logits"])
    moe.moe_route_backward(shape, s["logits"], s["topk_idx"], s["d_topk_w"], s["mask"], s["seq"],
                           ALPHA, s["counts"], s["d_loss"], out)
    return out


def _own_dropout(s):
    import sparse_expert_ffn_moe_gb300 as moe
    y = torch.empty_like(s["x"])
    moe.moe_dropout(s["x"], s["residual"], s["p"], s["rng"], y)
    return y


def _own_combine(s):
    moe, shape = _shape(s)
    y = torch.empty(s["T"], s["d"], dtype=s["y_perm"].dtype, device="cuda")
    moe.moe_combine_dropout(shape, s["y_perm"], s["inv_perm"], s["topk_w"], s["y_shared"],
                            s["residual"], s["p"], s["rng"], y)
    return y


def _own_combine_grad(s):
    moe, shape = _shape(s)
    out = {"d_topk_w": torch.empty(s["T"], s["K"], device="cuda")}
    if s["rows"]:
        out["d_y_perm"] = torch.empty_like(s["y_perm"])
    if s["shared"]:
        out["d_shared"] = torch.empty_like(s["d_y"])
    moe.moe_combine_backward(shape, s["d_y"], s["y_perm"], s["inv_perm"], s["topk_w"], s["p"],
                             s["rng"], out.get("d_y_perm"), out["d_topk_w"], out.get("d_shared"))
    return out


PLAIN = dict(balance=_balance, route_grad=_route_grad, dropout=_dropout, combine=_combine,
             combine_grad=_combine_grad)
OWN = dict(balance=_own_balance, route_grad=_own_route_grad, dropout=_own_dropout,
           combine=_own_combine, combine_grad=_own_combine_grad)


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def work(case):
    op = case["op"]
    T = case["T"]
    if op in ("balance", "route_grad"):
        E, K, n = case["E"], case["K"], max(1, case["seqs"])
        b = 4 * (n + 1) * (case["seqs"] > 0) + T * (case["pad"] > 0)
        if op == "balance":
            return {"bytes": b + 4 * T * (E + K) + 8 * n * E + 4, "flops": 6 * T * E}
        if not case["balance"]:  # the scores of the chosen experts alone
            return {"bytes": b + 12 * T * K + 4 * T * E, "flops": 10 * T * K}
        return {"bytes": b + 8 * T * E + 4 * n * E + (8 * T * K if case["gate"] else 0),
                "flops": 10 * T * E + (10 * T * K if case["gate"] else 0)}
    size = 2 if case["dtype"] == "bf16" else 4
    row = T * case["d"]
    if op == "dropout":
        return {"bytes": size * row * (2 + case["residual"]), "flops": 2 * row}
    K = case["K"]
    if op == "combine":
        return {"bytes": size * row * (K + 1 + case["shared"] + case["residual"]) + 8 * T * K,
                "flops": 2 * row * K}
    return {"bytes": size * row * (1 + K * (1 + case["rows"]) + case["shared"]) + 12 * T * K,
            "flops": row * K * (2 + case["rows"])}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_keep(n, p, rng):
    """Philox4x32-10 on the host, in unsigned 64-bit products."""
    u = np.uint64
    seed, offset = (int(v) & (1 << 64) - 1 for v in rng)
    out = np.empty(((n + 7) // 8, 8), np.uint16)
    low, sh = u(MASK), u(32)
    for at in range(0, len(out), 1 << 20):
        g = np.arange(at, min(at + (1 << 20), len(out)), dtype=u)
        c = [g & low, g >> sh, np.full_like(g, offset & MASK), np.full_like(g, offset >> 32)]
        key = [seed & MASK, seed >> 32]
        for r in range(10):
            a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
            c = [(b >> sh) ^ c[1] ^ u((key[0] + r * 0x9E3779B9) & MASK), b & low,
                 (a >> sh) ^ c[3] ^ u((key[1] + r * 0xBB67AE85) & MASK), a & low]
        for j in range(4):
            out[at:at + len(g), 2 * j] = c[j] & u(0xFFFF)
            out[at:at + len(g), 2 * j + 1] = c[j] >> u(16)
    return torch.from_numpy(out.reshape(-1)[:n] >= np.uint32(int(p * 65536 + 0.5))).cuda()


def _exact_scale(s, shape):
    """What each element is multiplied by: 0, or 1 over the share that stays."""
    thr = int(s["p"] * 65536 + 0.5)
    if thr == 0:
        return torch.ones(shape, dtype=torch.float64, device="cuda")
    keep = _exact_keep(shape[0] * shape[1], s["p"], s["rng"].tolist()).view(shape)
    return keep.double() / (1 - thr / 65536)


def _spans(s):
    cu = [0, s["T"]] if s["seq"] is None else s["seq"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _live(s, a, b):
    """The tokens of [a, b) that are no padding."""
    t = torch.arange(a, b, device="cuda")
    return t if s["mask"] is None else t[s["mask"][a:b].bool()]


def _exact_probs(s, z):
    return torch.softmax(z, 1) if s["router"] == "softmax" else \
        torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "balance":
        spans, E, K = _spans(s), s["E"], s["K"]
        mean = torch.zeros(len(spans), E, dtype=torch.float64, device="cuda")
        loss = 0.0
        for i, (a, b) in enumerate(spans):
            t = _live(s, a, b)
            if len(t):
                mean[i] = _exact_probs(s, s["logits"][t].double()).mean(0)
                picks = torch.bincount(s["topk_idx"][t].reshape(-1), minlength=E).double()
                loss = loss + ALPHA / len(spans) * (picks * E / (K * len(t)) * mean[i]).sum().item()
        return None, mean, torch.full((1,), loss, dtype=torch.float64)
    if op == "route_grad":
        out = torch.zeros_like(s["logits"], dtype=torch.float64)
        spans = _spans(s)
        for i, (a, b) in enumerate(spans):
            t = _live(s, a, b)
            if not len(t):
                continue
            z = s["logits"][t].double().requires_grad_()
            idx = s["topk_idx"][t].long()
            total = 0.0
            if s["counts"] is not None:  # the loss itself, differentiated
                freq = s["counts"][i].double() * s["E"] / (s["K"] * len(t))
                total = total + ALPHA / len(spans) * (freq * _exact_probs(s, z).mean(0)).sum()
            if s["d_topk_w"] is not None:
                zk = z.gather(1, idx)
                if s["router"] == "softmax":
                    w = torch.softmax(zk, 1)
                else:
                    w = torch.sigmoid(zk)
                    w = w / (w.sum(1, keepdim=True) + 1e-6)
                total = total + (w * s["d_topk_w"][t].double()).sum()
            out[t] = torch.autograd.grad(total, z)[0]
        return out
    if op == "dropout":
        y = s["x"].double() * _exact_scale(s, s["x"].shape)
        return y if s["residual"] is None else y + s["residual"].double()
    T, K, d = s["T"], s["K"], s["d"]
    scale = _exact_scale(s, (T, d))
    inv = s["inv_perm"].long().view(T, K)
    w = s["topk_w"].double()
    step = max(1, (1 << 27) // (K * d))
    if op == "combine":
        y = torch.empty(T, d, dtype=torch.float64, device="cuda")
        for a in range(0, T, step):
            b = min(T, a + step)
            v = torch.einsum("tk,tkd->td", w[a:b], s["y_perm"][inv[a:b]].double())
            if s["y_shared"] is not None:
                v = v + s["y_shared"][a:b].double()
            v = v * scale[a:b]
            y[a:b] = v if s["residual"] is None else v + s["residual"][a:b].double()
        return y
    dz = s["d_y"].double() * scale
    out = {"d_topk_w": torch.empty(T, K, dtype=torch.float64, device="cuda")}
    if s["rows"]:
        out["d_y_perm"] = torch.empty(T * K, d, dtype=torch.float64, device="cuda")
    if s["shared"]:
        out["d_shared"] = dz
    for a in range(0, T, step):
        b = min(T, a + step)
        out["d_topk_w"][a:b] = torch.einsum("td,tkd->tk", dz[a:b], s["y_perm"][inv[a:b]].double())
        if s["rows"]:
            out["d_y_perm"][inv[a:b].reshape(-1)] = \
                (w[a:b, :, None] * dz[a:b, None]).view(-1, d)
    return out
