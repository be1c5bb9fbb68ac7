"""The operators around a trainable router, as their users call them: sizes, inputs, plain forms, exact values.

Four operators, measured one pass at a time:

  adapters       router logits of a batch of many requests, each with a low-rank adapter of its own beside the
                 shared projection: h_i = x_i W_r + s_a B_a (A_a x_i), a = adapter_idx[i] (-1: none)
  adapters_grad  its backward: dx, dA, dB and, when the shared projection is trained too, dW_r
  loss           the balance loss over ragged sequences with masked tokens, its sequence-wise form and the
                 z-loss, per-expert counts, and the gradient of the logits (the gates' own gradient joined in)
  combine_grad   the backward of the gated combine: the gradient of every expert row and of every gate

`own` picks what `run` does: the framework's entry points, or the plain form in elementary torch operations.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each of 32 requests over 24 adapters: what a serving step of the layer asks for
        dict(name="adapters, a step of 32 requests", op="adapters", m=32, d=2048, n=64, r=16, na=24, dtype="bf16",
             order="token", bare=0.1),
        # prompts of ragged lengths beside one another, odd token count, the 128-expert router
        dict(name="adapters, ragged prompts", op="adapters", m=8191, d=768, n=128, r=8, na=12, dtype="bf16",
             order="request", bare=0.2),
        # a tuning batch of the widest router
        dict(name="adapters, tuning batch", op="adapters", m=65536, d=4096, n=64, r=16, na=16, dtype="bf16",
             order="request", bare=0.1),
        # the small fp32 layer
        dict(name="adapters, small fp32", op="adapters", m=1024, d=64, n=8, r=4, na=3, dtype="fp32",
             order="request", bare=0.0),
        # adapters tuned with the shared projection frozen
        dict(name="gradient, tuning batch", op="adapters_grad", m=65536, d=4096, n=64, r=16, na=16, dtype="bf16",
             order="request", bare=0.1, train_w=False),
        # adapters and shared projection trained together
        dict(name="gradient, all weights", op="adapters_grad", m=16384, d=2048, n=64, r=32, na=5, dtype="bf16",
             order="request", bare=0.0, train_w=True),
        dict(name="gradient, small fp32", op="adapters_grad", m=1001, d=64, n=8, r=4, na=3, dtype="fp32",
             order="request", bare=0.2, train_w=True),
        # a short batch of a small layer
        dict(name="loss, short batch", op="loss", m=777, n=8, k=1, score="softmax", renorm=False, seqs=5, dead=0,
             masked=0.1, alpha_seq=0.0, z=1e-3),
        # sigmoid scores, six picks
        dict(name="loss, sigmoid, six picks", op="loss", m=16384, n=64, k=6, score="sigmoid", renorm=False, seqs=37,
             dead=0, masked=0.05, alpha_seq=1e-3, z=0.0),
        # the widest router, eight renormalised picks, some experts switched off
        dict(name="loss, 256 experts", op="loss", m=65536, n=256, k=8, score="softmax", renorm=True, seqs=48, dead=5,
             masked=0.05, alpha_seq=1e-3, z=1e-3),
        # one pick per token with dropped tokens
        dict(name="combine gradient, one pick", op="combine_grad", m=8192, d=768, n=128, k=1, capacity=80,
             dtype="bf16"),
        # the global batch: two picks per token
        dict(name="combine gradient, two picks", op="combine_grad", m=65536, d=4096, n=64, k=2, capacity=4096,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adapters", "adapters_grad", "loss", "combine_grad"])
    if op in ("adapters", "adapters_grad"):
        fp32 = rng.random() < 0.25
        d = (4 if fp32 else 8) * _log_int(rng, 8, 256 if fp32 else 512)
        n = _log_int(rng, 4, 256)
        most = min(65536, (1 << 34) // (d * n), 8192 if fp32 else 65536)
        m = _log_int(rng, 1, most)
        r = _log_int(rng, 1, 64)
        na = _log_int(rng, 1, max(1, min(64, (1 << 26) // (m * r))))
        case = dict(op=op, m=m, d=d, n=n, r=r, na=na, dtype="fp32" if fp32 else "bf16",
                    order=rng.choice(["request", "request", "token"]), bare=rng.choice([0.0, 0.1, 0.5]))
        if op == "adapters_grad":
            case["train_w"] = rng.random() < 0.4
        return case
    if op == "loss":
        n = _log_int(rng, 4, 256)
        k = rng.randint(1, min(8, n - 2))
        m = _log_int(rng, 1, 65536)
        return dict(op=op, m=m, n=n, k=k, score=rng.choice(["softmax", "softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, seqs=_log_int(rng, 1, max(1, min(64, m))),
                    dead=rng.choice([0, 0, 1]), masked=rng.choice([0.0, 0.1]), alpha_seq=rng.choice([0.0, 1e-3]),
                    z=rng.choice([0.0, 1e-3]))
    fp32 = rng.random() < 0.25
    d = 8 * _log_int(rng, 8, 512)
    n = _log_int(rng, 4, 256)
    k = rng.randint(1, min(8, n))
    m = _log_int(rng, 1, min(65536, (1 << (28 if fp32 else 29)) // (d * k)))
    return dict(op=op, m=m, d=d, n=n, k=k, capacity=max(1, int(m * k / n * rng.choice([1.0, 1.25, 2.0]))),
                dtype="fp32" if fp32 else "bf16")


# ---------------------------------------------------------------- inputs
def _lengths(g, parts, total):
    """`parts` ragged lengths (some may be zero) that add up to at most `total`."""
    w = torch.rand(parts, generator=g, device="cuda").add_(0.05)
    return (w / w.sum() * total).floor().to(torch.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] in ("adapters", "adapters_grad"):
        m, d, n, r, na = (case[key] for key in ("m", "d", "n", "r", "na"))
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = randn(m, d).to(dt)
        s["w_r"] = randn(d, n) / math.sqrt(d)
        s["a"] = (randn(na, r, d) / math.sqrt(d)).to(dt)
        s["b"] = (randn(na, n, r) * 0.1).to(dt)
        s["scale"] = 0.5 + torch.rand(na, generator=g, device="cuda")
        requests = m if case["order"] == "token" else min(m, 2 * na + 3)
        which = torch.randint(0, na, (requests,), generator=g, device="cuda")
        which[torch.rand(requests, generator=g, device="cuda") < case["bare"]] = -1
        if case["order"] == "request":
            ends = torch.cumsum(_lengths(g, requests, m), 0)
            which = which[torch.searchsorted(ends, torch.arange(m, device="cuda"), right=True).clamp(max=requests - 1)]
        s["adapter_idx"] = which.to(torch.int32).contiguous()
        s["logits"] = torch.empty(m, n, device="cuda")
        s["hidden"] = torch.empty(m, r, device="cuda")
        if case["op"] == "adapters_grad":
            s["dlogits"] = randn(m, n) / m
            # what the forward pass left for the backward: each row's A_a x_i
            at = torch.arange(na * r, device="cuda").view(na, r)[s["adapter_idx"].long().clamp(min=0)]
            every = torch.mm(s["x"].float(), s["a"].float().view(na * r, d).t())
            s["hidden"] = every.gather(1, at) * (s["adapter_idx"] >= 0)[:, None]
            s["dx"] = torch.empty_like(s["x"])
            s["da"] = torch.empty(na, r, d, device="cuda")
            s["db"] = torch.empty(na, n, r, device="cuda")
            s["dw_r"] = torch.empty(d, n, device="cuda") if case["train_w"] else None
    elif case["op"] == "loss":
        m, n, k, seqs = (case[key] for key in ("m", "n", "k", "seqs"))
        logits = randn(m, n) + randn(n) * 0.5
        logits[:, :case["dead"]] = -math.inf  # experts switched off
        s["logits"] = logits
        s["topk_idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        ends = torch.cumsum(_lengths(g, seqs, m), 0)  # the rows behind the last sequence are padding
        s["seq_offsets"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
        s["token_mask"] = (torch.rand(m, generator=g, device="cuda") >= case["masked"]).to(torch.uint8) \
            if case["masked"] else None
        s["dgate"] = randn(m, k) * (1e-2 / m)
        s["dloss"] = torch.ones(1, device="cuda")
        s["dlogits"] = torch.empty(m, n, device="cuda")
    else:
        m, d, n, k, cap = (case[key] for key in ("m", "d", "n", "k", "capacity"))
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        picks = torch.topk(torch.rand(m, n, generator=g, device="cuda") + torch.linspace(0, 0.2, n, device="cuda"), k,
                           dim=1).indices
        experts, order = torch.sort(picks.reshape(-1), stable=True)  # expert-major, token order inside
        start = torch.searchsorted(experts, torch.arange(n, device="cuda"))
        kept = torch.arange(m * k, device="cuda") - start[experts] < cap
        row = torch.where(kept, torch.cumsum(kept, 0) - 1, -1)
        s["dest_row"] = torch.empty(m * k, dtype=torch.int32, device="cuda")
        s["dest_row"][order] = row.to(torch.int32)
        s["dest_row"] = s["dest_row"].view(m, k)
        s["topk_gate"] = torch.softmax(randn(m, k), 1) if k > 1 else torch.rand(m, 1, generator=g, device="cuda")
        s["dy"] = randn(m, d).to(dt)
        s["ybuf"] = randn(m * k, d).to(dt)
        s["dybuf"] = torch.zeros(m * k, d, dtype=dt, device="cuda")  # rows behind the kept ones stay zero
        s["dgate"] = torch.empty(m, k, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _slots(adapter_idx, na):
    """[m, na] ones where a row's adapter is."""
    return (adapter_idx[:, None] == torch.arange(na, device=adapter_idx.device)).float()


def _plain_adapters(s):
    na, r, d = s["a"].shape
    n = s["w_r"].shape[1]
    x = s["x"].float()
    slots = _slots(s["adapter_idx"], na)
    every = (x @ s["a"].float().reshape(na * r, d).t()).view(-1, na, r)
    own_u = every * slots[:, :, None]
    scaled = own_u * s["scale"][None, :, None]
    logits = x @ s["w_r"] + scaled.reshape(-1, na * r) @ s["b"].float().transpose(1, 2).reshape(na * r, n)
    return dict(logits=logits, hidden=own_u.sum(1))


def _plain_adapters_grad(s):
    na, r, d = s["a"].shape
    n = s["w_r"].shape[1]
    x, dh = s["x"].float(), s["dlogits"]
    at = _slots(s["adapter_idx"], na) * s["scale"]
    du = (dh @ s["b"].float().permute(1, 0, 2).reshape(n, na * r)).view(-1, na, r) * at[:, :, None]
    du = du.reshape(-1, na * r)
    dx = dh @ s["w_r"].t() + du @ s["a"].float().reshape(na * r, d)
    u = (s["hidden"][:, None, :] * at[:, :, None]).reshape(-1, na * r)
    out = dict(dx=dx.to(s["x"].dtype), da=(du.t() @ x).view(na, r, d),
               db=(u.t() @ dh).view(na, r, n).transpose(1, 2).contiguous())
    if s["dw_r"] is not None:
        out["dw_r"] = x.t() @ dh
    return out


def _plain_loss(s):
    case = s["case"]
    alpha, alpha_seq, z = 1e-2, case["alpha_seq"], case["z"]
    h, idx = s["logits"], s["topk_idx"].long()
    m, n = h.shape
    k = idx.shape[1]
    offsets = s["seq_offsets"].long()
    seqs = offsets.numel() - 1
    rows = torch.arange(m, device=h.device)
    seq = torch.searchsorted(offsets, rows, right=True) - 1
    valid = (seq >= 0) & (seq < seqs)
    if s["token_mask"] is not None:
        valid = valid & (s["token_mask"] != 0)
    # `seqs` stands for the whole batch in the tables below; padding goes to a row behind it that is cut off
    seq = torch.where(valid, seq, seqs + 1)
    top = h.amax(1, keepdim=True)
    e = (h - top).exp()
    lse = top[:, 0] + e.sum(1).log()
    soft = e / e.sum(1, keepdim=True)
    p = soft if case["score"] == "softmax" else 1 / (1 + (-h).exp())
    hits = torch.zeros(m, n, dtype=torch.float64, device=h.device).scatter_(1, idx, 1.0)
    ones = torch.ones(m, dtype=torch.float64, device=h.device)
    tokens = torch.zeros(seqs + 2, dtype=torch.float64, device=h.device).index_add_(0, seq, ones)
    counts = torch.zeros(seqs + 2, n, dtype=torch.float64, device=h.device).index_add_(0, seq, hits)
    psum = torch.zeros(seqs + 2, n, dtype=torch.float64, device=h.device).index_add_(0, seq, p.double())
    tokens[seqs], counts[seqs], psum[seqs] = tokens[:seqs].sum(), counts[:seqs].sum(0), psum[:seqs].sum(0)
    tokens, counts, psum = tokens[:seqs + 1], counts[:seqs + 1], psum[:seqs + 1]
    per = tokens.clamp(min=1)[:, None]
    f, mean_p = counts / (k * per), psum / per
    each = n * (f * mean_p).sum(1)
    full = (tokens[:seqs] > 0).sum().clamp(min=1)
    batch, by_seq = alpha * each[seqs], alpha_seq * each[:seqs].sum() / full
    z_loss = z * (lse.double().square() * valid).sum() / per[seqs, 0]
    # gradient: f is held fixed, P and the gates follow the scores
    shift = 1.0 / n if case["score"] == "softmax" else 0.0  # a constant in g drops out of the softmax
    table = alpha * n * (f[seqs] - shift) / per[seqs]
    table = table + alpha_seq * n / full * (f[:seqs] - shift) / per[:seqs]
    up = s["dloss"].double()
    # the row behind the tables stands for the rows that count for nothing
    gp = torch.cat([table * up, torch.zeros(2, n, dtype=torch.float64, device=h.device)])[seq].float()
    dgate = s["dgate"]
    chosen = h.gather(1, idx)
    extra = torch.zeros_like(h)
    if case["score"] == "sigmoid" or not (case["renorm"] and k > 1):
        gp = gp.scatter_add(1, idx, dgate)
    else:
        q = (chosen - chosen.amax(1, keepdim=True)).exp()
        q = q / q.sum(1, keepdim=True)
        extra = extra.scatter_add(1, idx, q * (dgate - (q * dgate).sum(1, keepdim=True)))
    if case["score"] == "softmax":
        dh = p * (gp - (p * gp).sum(1, keepdim=True)) + extra
    else:
        dh = gp * p / (1 + h.exp())
    dh = dh + (2 * z * up / per[seqs, 0]).float() * lse[:, None] * soft
    dh = torch.where(valid[:, None], dh, torch.zeros_like(dh))
    return dict(loss=torch.stack([batch + by_seq + z_loss, batch, by_seq, z_loss]).float(),
                counts=counts.to(torch.int32), tokens=tokens.to(torch.int32), f=f.float(), P=mean_p.float(),
                dlogits=dh)


def _plain_combine_grad(s):
    dy, dest, gate = s["dy"].float(), s["dest_row"].long(), s["topk_gate"]
    kept = dest >= 0
    if s["dy"].dtype == torch.bfloat16:
        gate = gate.to(torch.bfloat16).float()  # the combine rounds the gate to the layer's type
    rows = s["ybuf"][dest.clamp(min=0)].float()
    dgate = (rows * dy[:, None, :]).sum(-1) * kept
    dybuf = torch.zeros_like(s["dybuf"])
    dybuf[dest[kept]] = (gate[:, :, None] * dy[:, None, :])[kept].to(dybuf.dtype)
    return dict(dybuf=dybuf, dgate=dgate)


# ---------------------------------------------------------------- one pass
def _own_run(s):
    import load_balanced_dispatch_b200 as lb

    case, op = s["case"], s["case"]["op"]

    def workspace(name, size, *args):  # a program allocates it once and keeps it
        if name not in s:
            s[name] = torch.empty(max(size(*args), 1), dtype=torch.uint8, device="cuda")
        return s[name]

    if op == "adapters":
        m, d, n, r, na = (case[key] for key in ("m", "d", "n", "r", "na"))
        ws = workspace("ws", lb.moe_router_adapters_workspace_size, m, d, n, r, na, s["x"].dtype)
        logits, hidden = lb.moe_router_adapters(s["x"], s["w_r"], s["a"], s["b"], s["adapter_idx"], s["scale"],
                                                logits=s["logits"], hidden=s["hidden"], workspace=ws)
        return dict(logits=logits, hidden=hidden)
    if op == "adapters_grad":
        m, d, n, r, na = (case[key] for key in ("m", "d", "n", "r", "na"))
        ws = workspace("ws", lb.moe_router_adapters_grad_workspace_size, m, d, n, r, na, s["x"].dtype)
        dx, da, db, dw_r = lb.moe_router_adapters_grad(
            s["dlogits"], s["x"], s["w_r"], s["a"], s["b"], s["adapter_idx"], s["scale"], s["hidden"], dx=s["dx"],
            da=s["da"], db=s["db"], dw_r=s["dw_r"], want_dw_r=case["train_w"], workspace=ws)
        out = dict(dx=dx, da=da, db=db)
        return dict(out, dw_r=dw_r) if case["train_w"] else out
    if op == "loss":
        fn = lb.MOE_SOFTMAX if case["score"] == "softmax" else lb.MOE_SIGMOID
        coef = dict(alpha=1e-2, alpha_seq=case["alpha_seq"], z_coef=case["z"])
        ws = workspace("ws", lb.moe_router_loss_workspace_size, case["m"], case["n"], case["seqs"])
        out = lb.moe_router_loss(s["logits"], s["topk_idx"], s["seq_offsets"], token_mask=s["token_mask"],
                                 score_fn=fn, out=s.get("out"), workspace=ws, **coef)
        s["out"] = out
        dh = lb.moe_router_loss_grad(s["logits"], s["topk_idx"], s["seq_offsets"], out["counts"], out["tokens"],
                                     token_mask=s["token_mask"], score_fn=fn, dloss=s["dloss"], dgate=s["dgate"],
                                     renorm_topk=int(case["renorm"]), dlogits=s["dlogits"], **coef)
        return dict(out, dlogits=dh)
    dybuf, dgate = lb.moe_combine_grad(s["dy"], s["ybuf"], s["dest_row"], s["topk_gate"], dybuf=s["dybuf"],
                                       dgate=s["dgate"])
    return dict(dybuf=dybuf, dgate=dgate)


def run(state):
    if own:
        return _own_run(state)
    return {"adapters": _plain_adapters, "adapters_grad": _plain_adapters_grad, "loss": _plain_loss,
            "combine_grad": _plain_combine_grad}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    m, n = case["m"], case["n"]
    if case["op"] == "loss":
        k, seqs = case["k"], case["seqs"]
        tables = (seqs + 1) * (3 * 4 * n + 4)
        return dict(bytes=2 * 4 * m * n + m * k * (4 + 4) + m + 4 * (seqs + 1) + tables, flops=20 * m * n)
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "combine_grad":
        k = case["k"]
        rows = min(m * k, n * case["capacity"])
        return dict(bytes=e * d * (m + 2 * rows) + m * k * 12, flops=3 * rows * d)
    r = case["r"]
    used = min(case["na"], m)  # adapters that a batch can name
    weights = 4 * d * n + e * used * r * (d + n)
    small = m * (4 + 4 * n + 4 * r)  # adapter ids, the logits or their gradient, the hidden rows
    if case["op"] == "adapters":
        return dict(bytes=e * m * d + weights + small, flops=2 * m * d * (n + r) + 2 * m * r * n)
    grads = 4 * case["na"] * r * (d + n) + (4 * d * n if case["train_w"] else 0)
    flops = 2 * m * d * (n + r) + 2 * m * d * r + 4 * m * r * n + (2 * m * d * n if case["train_w"] else 0)
    return dict(bytes=2 * e * m * d + weights + small + grads, flops=flops)


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_adapters(s, grad):
    x, w = s["x"].double(), s["w_r"].double()
    a, b, scale = s["a"].double(), s["b"].double(), s["scale"].double()
    if not grad:
        logits = torch.mm(x, w)
        hidden = torch.zeros(x.shape[0], a.shape[1], dtype=torch.float64, device=x.device)
        for q in range(a.shape[0]):
            rows = torch.nonzero(s["adapter_idx"] == q)[:, 0]
            u = torch.mm(x[rows], a[q].t())
            hidden[rows] = u
            logits[rows] += scale[q] * torch.mm(u, b[q].t())
        return dict(logits=logits, hidden=hidden)
    dh, u = s["dlogits"].double(), s["hidden"].double()
    out = dict(dx=torch.mm(dh, w.t()), da=torch.zeros_like(a), db=torch.zeros_like(b))
    for q in range(a.shape[0]):
        rows = torch.nonzero(s["adapter_idx"] == q)[:, 0]
        du = scale[q] * torch.mm(dh[rows], b[q])
        out["dx"][rows] += torch.mm(du, a[q])
        out["da"][q] = torch.mm(du.t(), x[rows])
        out["db"][q] = scale[q] * torch.mm(dh[rows].t(), u[rows])
    if s["dw_r"] is not None:
        out["dw_r"] = torch.mm(x.t(), dh)
    return out


def _exact_loss(s):
    case = s["case"]
    alpha, alpha_seq, z = 1e-2, case["alpha_seq"], case["z"]
    h = s["logits"].double()
    m, n = h.shape
    idx = s["topk_idx"].long()
    k = idx.shape[1]
    ends = s["seq_offsets"].tolist()
    seqs = len(ends) - 1
    keep = torch.ones(m, dtype=torch.bool, device=h.device) if s["token_mask"] is None else s["token_mask"].bool()
    members = [torch.nonzero(keep[ends[q]:ends[q + 1]])[:, 0] + ends[q] for q in range(seqs)]
    members.append(torch.cat(members))
    everyone = members[-1]
    lse = torch.logsumexp(h, 1)
    p = torch.softmax(h, 1) if case["score"] == "softmax" else torch.sigmoid(h)
    dp = torch.zeros_like(h)
    f = torch.zeros(seqs + 1, n, dtype=torch.float64, device=h.device)
    mean_p, counts = torch.zeros_like(f), torch.zeros(seqs + 1, n, dtype=torch.int64, device=h.device)
    full = max(1, sum(len(v) > 0 for v in members[:-1]))
    loss = [0.0, 0.0]
    for q, rows in enumerate(members):
        if len(rows) == 0:
            continue
        counts[q] = torch.bincount(idx[rows].reshape(-1), minlength=n)
        f[q] = counts[q] / (k * len(rows))
        mean_p[q] = p[rows].mean(0)
        weight = alpha if q == seqs else alpha_seq / full
        loss[0 if q == seqs else 1] += float(weight * n * (f[q] * mean_p[q]).sum())
        dp[rows] += weight * n * f[q] / len(rows)
    z_loss = float(z * lse[everyone].square().mean()) if len(everyone) else 0.0
    up = s["dloss"].double()
    dp = dp * up
    dgate = s["dgate"].double()
    dh = torch.zeros_like(h)
    if case["score"] == "softmax" and case["renorm"] and k > 1:
        q = torch.softmax(h.gather(1, idx), 1)
        dh.scatter_add_(1, idx, q * (dgate - (q * dgate).sum(1, keepdim=True)))
    else:
        dp.scatter_add_(1, idx, dgate)
    if case["score"] == "softmax":
        dh += p * (dp - (p * dp).sum(1, keepdim=True))
    else:
        dh += dp * p * torch.sigmoid(-h)
    dh += 2 * z * up / max(1, len(everyone)) * lse[:, None] * torch.softmax(h, 1)
    dlogits = torch.zeros_like(h)
    dlogits[everyone] = dh[everyone]
    total = torch.tensor([loss[0] + loss[1] + z_loss, loss[0], loss[1], z_loss], dtype=torch.float64)
    return dict(loss=total, counts=counts, tokens=torch.tensor([len(v) for v in members]), f=f, P=mean_p,
                dlogits=dlogits)


def _exact_combine_grad(s):
    dest = s["dest_row"].long()
    gate = s["topk_gate"].to(s["dy"].dtype).double()
    dybuf = torch.zeros(s["ybuf"].shape, dtype=torch.float64, device="cuda")
    dgate = torch.zeros(dest.shape, dtype=torch.float64, device="cuda")
    for pick in range(dest.shape[1]):
        tokens = torch.nonzero(dest[:, pick] >= 0)[:, 0]
        for part in torch.split(tokens, 8192):
            rows, dy = dest[part, pick], s["dy"][part].double()
            dybuf[rows] = gate[part, pick, None] * dy
            dgate[part, pick] = torch.einsum("td,td->t", dy, s["ybuf"][rows].double())
    return dict(dybuf=dybuf, dgate=dgate)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "loss":
        return _exact_loss(s)
    if case["op"] == "combine_grad":
        return _exact_combine_grad(s)
    return _exact_adapters(s, case["op"] == "adapters_grad")
