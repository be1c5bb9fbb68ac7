"""The trainable router's operators (adapters beside the router projection, losses over a ragged batch,
combine gradient) against their formulas in 64 bits.

Tolerances are elementwise bounds from the arithmetic, with eps = 2^-23 for one truncated or two rounded fp32
steps. A sum of K products in blocks (32 columns or 16 rows by FMA; up to 256 columns in three parts on the tensor
cores, 48 truncated steps) and then over blocks is off by at most (64 + K / 16) eps times the sum of the products'
magnitudes. A bf16 result is off by half a step more, 2^-8 of its value; its operands enter as two bf16 parts, whose
remainder and dropped product stay below 2^-14 of the magnitudes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

lb = pytest.importorskip("load_balanced_dispatch_b200")
EPS = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    from load_balanced_dispatch_b200 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    lb.sync_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound.clamp(min=1e-300)).max()):.3g} of the bound"


def poisoned(nbytes):
    """A workspace whose old contents are NaN bit patterns."""
    return torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- adapters
def adapter_inputs(m, d, n, r, na, dtype, order, seed):
    g = gen(seed)
    x = torch.randn(m, d, generator=g, device="cuda").to(dtype)
    w = torch.randn(d, n, generator=g, device="cuda") / d ** 0.5
    a = (torch.randn(na, r, d, generator=g, device="cuda") / d ** 0.5).to(dtype)
    b = (torch.randn(na, n, r, generator=g, device="cuda") * 0.3).to(dtype)
    scale = torch.rand(na, generator=g, device="cuda") + 0.5
    idx = torch.randint(-1, na, (m,), generator=g, device="cuda", dtype=torch.int32)
    if order == "none":
        idx.fill_(-1)
    elif order == "one":
        idx.fill_(na - 1)
    elif order == "runs":
        idx = idx.sort().values.roll(m // 3)
    dh = torch.randn(m, n, generator=g, device="cuda")
    return dict(x=x, w_r=w, a=a, b=b, adapter_idx=idx.contiguous(), scale=scale), dh


def adapters_ref(i):
    """(logits, hidden) and the sums of magnitudes they are made of."""
    x, w, a, b, s = (i[k].double() for k in ("x", "w_r", "a", "b", "scale"))
    idx = i["adapter_idx"].long()
    m, r = x.shape[0], a.shape[1]
    u, au = x.new_zeros(m, r), x.new_zeros(m, r)
    h, ah = x @ w, x.abs() @ w.abs()
    for q in range(a.shape[0]):
        rows = (idx == q).nonzero()[:, 0]
        if len(rows):
            u[rows], au[rows] = x[rows] @ a[q].T, x[rows].abs() @ a[q].abs().T
            h[rows] += s[q] * u[rows] @ b[q].T
            ah[rows] += s[q] * au[rows] @ b[q].abs().T
    return h, ah, u, au


SHAPES = [  # m, d, n, r, na, dtype, order
    (1, 64, 8, 4, 1, "bf16", "mixed"), (5, 2048, 64, 16, 3, "bf16", "mixed"), (130, 256, 64, 16, 5, "bf16", "runs"),
    (1000, 72, 5, 3, 7, "bf16", "mixed"), (700, 768, 128, 8, 4, "bf16", "runs"), (513, 520, 33, 17, 2, "bf16", "runs"),
    (300, 200, 256, 64, 3, "bf16", "mixed"), (640, 4096, 64, 64, 2, "bf16", "one"), (257, 136, 200, 33, 40, "bf16", "mixed"),
    (256, 128, 64, 16, 4, "bf16", "none"), (2000, 128, 96, 32, 1, "bf16", "mixed"), (37, 8, 1, 1, 2, "bf16", "mixed"),
    (3000, 64, 16, 8, 1024, "bf16", "mixed"), (20000, 64, 128, 8, 4, "bf16", "runs"),
    (19500, 72, 90, 32, 3, "bf16", "mixed"), (2600, 512, 64, 16, 6, "bf16", "runs"), (2100, 200, 128, 32, 5, "bf16", "mixed"),
    (2500, 128, 256, 16, 5, "bf16", "runs"), (20000, 64, 200, 16, 3, "bf16", "runs"), (20500, 40, 256, 33, 2, "bf16", "mixed"),
    (2200, 264, 40, 64, 9, "bf16", "runs"), (2300, 128, 20, 40, 2, "bf16", "one"),
    (1, 4, 1, 1, 1, "fp32", "mixed"), (1024, 64, 8, 4, 3, "fp32", "runs"), (333, 1000, 64, 16, 5, "fp32", "mixed"),
    (517, 36, 256, 64, 9, "fp32", "runs"), (129, 260, 17, 5, 33, "fp32", "mixed"), (600, 132, 100, 20, 2, "fp32", "one"),
]


@pytest.mark.parametrize("m,d,n,r,na,dtype,order", SHAPES)
def test_adapters_forward(m, d, n, r, na, dtype, order):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    i, _ = adapter_inputs(m, d, n, r, na, dt, order, m + d)
    ws = poisoned(lb.moe_router_adapters_workspace_size(m, d, n, r, na, dt))
    logits, hidden = lb.moe_router_adapters(**i, workspace=ws)
    lb.sync_status()
    h, ah, u, au = adapters_ref(i)
    within(hidden, u, (64 + d / 16) * EPS * au, "hidden")
    within(logits, h, (64 + d / 16 + r) * EPS * ah, "logits")
    again, none = lb.moe_router_adapters(**i, want_hidden=False)
    assert none is None and torch.equal(again, logits)


@pytest.mark.parametrize("m,d,n,r,na,dtype,order", SHAPES)
def test_adapters_backward(m, d, n, r, na, dtype, order):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    i, dh = adapter_inputs(m, d, n, r, na, dt, order, m + d + 1)
    _, _, u, _ = adapters_ref(i)
    hidden = u.float()
    ws = poisoned(lb.moe_router_adapters_grad_workspace_size(m, d, n, r, na, dt))
    dx, da, db, dw = lb.moe_router_adapters_grad(dh, hidden=hidden, want_dw_r=True, workspace=ws, **i)
    lb.sync_status()
    x, w, a, b, s = (i[k].double() for k in ("x", "w_r", "a", "b", "scale"))
    dh64, u64, idx = dh.double(), hidden.double(), i["adapter_idx"].long()
    ref, mag = dh64 @ w.T, dh64.abs() @ w.abs().T
    for q in range(na):
        rows = (idx == q).nonzero()[:, 0]
        c = len(rows)
        if c == 0:
            assert not bool(da[q].any()) and not bool(db[q].any())
            continue
        du, adu = s[q] * dh64[rows] @ b[q], s[q] * dh64[rows].abs() @ b[q].abs()
        ref[rows] += du @ a[q]
        mag[rows] += adu @ a[q].abs()
        within(da[q], du.T @ x[rows], (128 + n + c / 16) * EPS * (adu.T @ x[rows].abs()), f"da[{q}]")
        within(db[q], s[q] * dh64[rows].T @ u64[rows], (66 + c / 16) * EPS * s[q] * dh64[rows].abs().T @ u64[rows].abs(),
               f"db[{q}]")
    if dt == torch.bfloat16:
        within(dx, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag, "dx")
    else:
        within(dx, ref, (64 + n + r) * EPS * mag, "dx")
    within(dw, x.T @ dh64, (64 + m / 16) * EPS * (x.abs().T @ dh64.abs()), "dw_r")
    # the same call gives the same bits; nothing optional changes what the rest gives
    again = lb.moe_router_adapters_grad(dh, hidden=hidden, want_dw_r=True, **i)
    for p, q in zip(again, (dx, da, db, dw)):
        assert torch.equal(p, q)
    none, da2, db2, no_w = lb.moe_router_adapters_grad(dh, hidden=hidden, want_dx=False, **i)
    assert none is None and no_w is None and torch.equal(da2, da) and torch.equal(db2, db)


def test_adapters_gradient_by_differences():
    # the logits are linear in x, A, B and W_r each: a central difference is exact but for rounding
    i, dh = adapter_inputs(200, 96, 24, 6, 4, torch.float32, "mixed", 5)
    _, hidden = lb.moe_router_adapters(**i)
    dx, da, db, dw = lb.moe_router_adapters_grad(dh, hidden=hidden, want_dw_r=True, **i)
    g = gen(6)
    for key, grad in (("x", dx), ("a", da), ("b", db), ("w_r", dw)):
        step = torch.randn(i[key].shape, generator=g, device="cuda") * i[key].abs().mean()
        up, _ = lb.moe_router_adapters(**dict(i, **{key: i[key] + step}))
        down, _ = lb.moe_router_adapters(**dict(i, **{key: i[key] - step}))
        diff = ((up.double() - down.double()) / 2 * dh).sum()
        dot = (grad.double() * step).sum()
        # each logit is off by at most (64 + 96 / 16 + 6) eps of its magnitudes; so is each gradient entry
        mag = (up.abs().double() * dh.abs()).sum() + (grad.abs().double() * step.abs()).sum()
        assert abs(float(diff - dot)) <= 256 * EPS * float(mag) * 8, key


def test_adapters_no_rows():
    for dt in (torch.bfloat16, torch.float32):
        i, dh = adapter_inputs(0, 64, 8, 4, 3, dt, "mixed", 1)
        logits, hidden = lb.moe_router_adapters(**i)
        assert logits.shape == (0, 8) and hidden.shape == (0, 4)
        dx, da, db, dw = lb.moe_router_adapters_grad(dh, hidden=hidden, want_dw_r=True, **i)
        lb.sync_status()
        assert dx.shape == (0, 64) and not bool(da.any()) and not bool(db.any()) and not bool(dw.any())


@pytest.mark.parametrize("m,dtype", [(40, "bf16"), (2500, "bf16"), (300, "fp32")])
def test_adapter_index_out_of_range_is_reported_and_counts_as_none(m, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    i, dh = adapter_inputs(m, 128, 16, 8, 3, dt, "mixed", 2)
    good = i["adapter_idx"].clone()
    good[::3] = -1
    bad = good.clone()
    bad[::3] = 3
    bad[0] = -7
    want = lb.moe_router_adapters(**dict(i, adapter_idx=good))
    got = lb.moe_router_adapters(**dict(i, adapter_idx=bad))
    with pytest.raises(lb.MoEError, match="adapter index"):
        lb.sync_status()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    wg = lb.moe_router_adapters_grad(dh, hidden=want[1], **dict(i, adapter_idx=good))
    gg = lb.moe_router_adapters_grad(dh, hidden=want[1], **dict(i, adapter_idx=bad))
    with pytest.raises(lb.MoEError, match="adapter index"):
        lb.sync_status()
    for p, q in zip(gg[:3], wg[:3]):
        assert torch.equal(p, q)


def test_adapters_do_not_mix_rows():
    # a NaN token stays in its own row of the logits, and in its own adapter's gradients
    i, dh = adapter_inputs(400, 256, 32, 8, 4, torch.bfloat16, "mixed", 3)
    i["adapter_idx"][17] = 2
    clean, hidden = lb.moe_router_adapters(**i)
    i["x"][17, 5] = float("nan")
    logits, hidden2 = lb.moe_router_adapters(**i)
    rest = torch.arange(400, device="cuda") != 17
    assert torch.equal(logits[rest], clean[rest]) and bool(logits[17].isnan().all())
    dx, da, db, _ = lb.moe_router_adapters_grad(dh, hidden=hidden2, **i)
    lb.sync_status()
    assert bool(da[2, :, 5].isnan().all()) and not bool(da[[0, 1, 3]].isnan().any())
    assert not bool(dx.isnan().any()) and bool(db[2].isnan().all()) and not bool(db[[0, 1, 3]].isnan().any())


# ---------------------------------------------------------------- router losses
def loss_inputs(m, n, k, nseq, mask, seed, dead=0):
    g = gen(seed)
    h = torch.randn(m, n, generator=g, device="cuda") * 2
    h[:, :dead] = -float("inf")
    idx = torch.topk(h + torch.rand(m, n, generator=g, device="cuda"), k, dim=1).indices.to(torch.int32)
    cuts = torch.randint(0, max(1, m - m // 8) + 1, (nseq + 1,), generator=g, device="cuda").sort().values
    tm = (torch.rand(m, generator=g, device="cuda") > 0.2).to(torch.uint8) if mask else None
    dgate = torch.randn(m, k, generator=g, device="cuda") / m
    return h, idx.contiguous(), cuts.to(torch.int32), tm, dgate


def loss_ref(h, idx, cuts, tm, fn, alpha, alpha_seq, z, dgate=None, renorm=False, up=1.0):
    """Everything in 64 bits, sequence by sequence; also the magnitudes that dlogits is made of."""
    h, idx, cuts = h.double(), idx.long(), cuts.tolist()
    m, n = h.shape
    k = idx.shape[1]
    ok = torch.ones(m, dtype=torch.bool, device=h.device) if tm is None else tm.bool()
    rows = [torch.arange(cuts[q], cuts[q + 1], device=h.device) for q in range(len(cuts) - 1)]
    rows = [v[ok[v]] for v in rows]
    every = torch.cat(rows)
    rows.append(every)
    alive = ~(h == -float("inf")).all(1)
    safe = torch.where(alive[:, None], h, torch.zeros_like(h))
    soft = torch.softmax(safe, 1) * alive[:, None]
    lse = torch.logsumexp(safe, 1) * alive
    p = soft if fn == lb.MOE_SOFTMAX else torch.sigmoid(h)
    S = len(rows) - 1
    f, P = h.new_zeros(S + 1, n), h.new_zeros(S + 1, n)
    counts, tokens = torch.zeros(S + 1, n, dtype=torch.int32, device=h.device), [len(v) for v in rows]
    nonempty = max(1, sum(t > 0 for t in tokens[:-1]))
    gp, mag = torch.zeros_like(h), torch.zeros_like(h)
    L = [0.0, 0.0]
    for q, v in enumerate(rows):
        if len(v) == 0:
            continue
        counts[q] = torch.bincount(idx[v].reshape(-1), minlength=n)
        f[q], P[q] = counts[q].double() / (k * len(v)), p[v].mean(0)
        c = alpha if q == S else alpha_seq / nonempty
        L[int(q < S)] += c * n * float((f[q] * P[q]).sum())
        gp[v] += up * c * n / len(v) * f[q]
        mag[v] += abs(up) * c * n / len(v) * (f[q] - (1 / n if fn == lb.MOE_SOFTMAX else 0)).abs()
    T = max(1, len(every))
    Lz = z * float(lse[every].square().sum()) / T
    dh = torch.zeros_like(h)
    extra = torch.zeros_like(h)
    if dgate is not None:
        d64 = dgate.double()
        if fn == lb.MOE_SOFTMAX and renorm and k > 1:
            q = torch.softmax(safe.gather(1, idx), 1)
            dh.scatter_add_(1, idx, q * (d64 - (q * d64).sum(1, keepdim=True)))
            extra.scatter_add_(1, idx, q * (d64.abs() + (q * d64.abs()).sum(1, keepdim=True)))
        else:
            gp.scatter_add_(1, idx, d64)
            mag.scatter_add_(1, idx, d64.abs())
    if fn == lb.MOE_SOFTMAX:
        dh += p * (gp - (p * gp).sum(1, keepdim=True))
        mag = p * (mag + (p * mag).sum(1, keepdim=True)) + extra
    else:
        dh += gp * p * torch.sigmoid(-h)
        mag = mag * p * torch.sigmoid(-h)
    dh += 2 * z * up / T * lse[:, None] * soft
    mag += 2 * z * abs(up) / T * lse.abs()[:, None] * soft
    keep = torch.zeros(m, 1, dtype=torch.bool, device=h.device)
    keep[every] = True
    return dict(loss=[L[0] + L[1] + Lz, L[0], L[1], Lz], counts=counts, tokens=tokens, f=f, P=P,
                dlogits=torch.where(keep, dh, torch.zeros_like(dh)), mag=torch.where(keep, mag, torch.zeros_like(mag)))


# a score's relative error: h - top is off by 2^-24 of at most 16, the exponential by 2 + 1.2 * 16 ulp, the sum of at
# most 256 terms by eight rounded steps, the quotient by one: 2^-24 * (16 + 2 * 21 + 8 + 2) = 2^-17.9
REL = 2.0 ** -17.9


@pytest.mark.parametrize("m,n,k,nseq,mask,fn,renorm,dead", [
    (1, 1, 1, 1, False, 0, 0, 0), (7, 4, 2, 3, True, 0, 1, 1), (777, 8, 1, 5, True, 0, 0, 0),
    (1000, 64, 6, 17, True, 1, 0, 0), (513, 64, 2, 1, False, 0, 1, 3), (2000, 256, 8, 40, True, 0, 1, 5),
    (300, 200, 20, 9, False, 0, 0, 0), (129, 17, 16, 4, True, 0, 1, 0), (640, 128, 4, 640, True, 0, 0, 0),
    (333, 33, 3, 8, True, 1, 0, 2), (5000, 6, 3, 2, False, 1, 0, 0), (90, 256, 40, 3, False, 0, 1, 0)])
def test_router_loss_and_gradient(m, n, k, nseq, mask, fn, renorm, dead):
    h, idx, cuts, tm, dgate = loss_inputs(m, n, k, nseq, mask, m + n, dead)
    coef = dict(alpha=1e-2, alpha_seq=3e-3, z_coef=1e-3)
    up = torch.full((1,), 0.7, device="cuda")
    # padding and masked rows: NaN logits and nonsense picks are not looked at
    ref = loss_ref(h, idx, cuts, tm, fn, 1e-2, 3e-3, 1e-3, dgate, bool(renorm), float(up))
    counted = torch.zeros(m, dtype=torch.bool, device="cuda")
    counted[int(cuts[0]):int(cuts[-1])] = True
    if tm is not None:
        counted &= tm.bool()
    h[~counted] = float("nan")
    idx[~counted] = 10 ** 6
    ws = poisoned(lb.moe_router_loss_workspace_size(m, n, nseq))
    out = lb.moe_router_loss(h, idx, cuts, tm, fn, workspace=ws, **coef)
    lb.sync_status()
    assert torch.equal(out["counts"], ref["counts"]) and out["tokens"].tolist() == ref["tokens"]
    assert np.allclose(out["loss"].tolist(), ref["loss"], rtol=REL, atol=1e-12)
    within(out["f"], ref["f"], 2 * EPS * ref["f"], "f")
    within(out["P"], ref["P"], REL * ref["P"] + 1e-12, "P")
    dh = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], tm, fn, dloss=up, dgate=dgate,
                                 renorm_topk=renorm, **coef)
    lb.sync_status()
    within(dh, ref["dlogits"], 2 * REL * ref["mag"] + 1e-14, "dlogits")
    assert not bool(dh[~counted].any())
    # without the gates, and the same bits again
    ref0 = loss_ref(torch.nan_to_num(h, nan=0.0, neginf=-float("inf")), idx.clamp(max=n - 1), cuts, tm, fn, 1e-2, 3e-3, 1e-3)
    dh0 = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], tm, fn, **coef)
    within(dh0, ref0["dlogits"], 2 * REL * ref0["mag"] + 1e-14, "dlogits without gates")
    out2 = lb.moe_router_loss(h, idx, cuts, tm, fn, **coef)
    for key in out:
        assert torch.equal(out[key], out2[key]), key


def test_router_loss_equal_segments_match_balance_stats():
    # no mask, equal sequences, no z-loss: the numbers of moe_balance_stats and moe_balance_loss_grad
    m, n, k, seg = 1024, 64, 2, 128
    h = torch.randn(m, n, generator=gen(3), device="cuda")
    idx, _, probs = lb.moe_router_topk(None, None, n, k, logits_in=h)
    old = lb.moe_balance_stats(probs, idx, n, seg)
    cuts = torch.arange(0, m + 1, seg, dtype=torch.int32, device="cuda")
    out = lb.moe_router_loss(h, idx, cuts, alpha=1e-2, alpha_seq=1e-2)
    assert torch.equal(out["f"], old["f"])
    assert torch.allclose(out["P"], old["P"], rtol=1e-6)
    assert torch.allclose(out["loss"][1], old["aux"][m // seg + 1], rtol=1e-6)
    assert torch.allclose(out["loss"][2], old["aux"][m // seg], rtol=1e-6)
    g_old = lb.moe_balance_loss_grad(probs, old["f"], seg, w_micro=1.0, w_global=1.0)
    g_new = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], alpha=1e-2, alpha_seq=1e-2)
    # the older form subtracts g's mean in fp32: off by 2^-22 of p times alpha n (f^G / m + f^s / m)
    assert float((g_old - g_new).abs().max()) <= 2.0 ** -20 * 1e-2 * n * 2 / m * float(old["f"].max()) * 2


@pytest.mark.parametrize("fn,renorm", [(0, 0), (0, 1), (1, 0)])
def test_router_loss_gradient_by_differences(fn, renorm):
    m, n, k = 64, 16, 3
    h, idx, cuts, tm, _ = loss_inputs(m, n, k, 4, True, 11)
    coef = dict(alpha=0.3, alpha_seq=0.2, z_coef=0.05)
    out = lb.moe_router_loss(h, idx, cuts, tm, fn, **coef)
    dh = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], tm, fn, **coef)
    v = torch.randn(m, n, generator=gen(12), device="cuda")
    step = 1e-2
    up = lb.moe_router_loss(h + step * v, idx, cuts, tm, fn, **coef)["loss"][0]
    down = lb.moe_router_loss(h - step * v, idx, cuts, tm, fn, **coef)["loss"][0]
    diff = float(up.double() - down.double()) / (2 * step)
    # the losses are rounded to fp32 (2^-24 each side, over 2 step); the third derivative of a softmax or
    # log-sum-exp along v is at most 8 |v|_inf^3 times the terms' weight, step^2 / 6 of it remains
    slack = 2.0 ** -23 * float(up.abs()) / (2 * step) + 8 * float(v.abs().max()) ** 3 * step ** 2 / 6 * float(up.abs())
    assert abs(diff - float((dh.double() * v).sum())) <= slack


def test_router_loss_nothing_counts():
    h, idx, cuts, _, dgate = loss_inputs(100, 12, 2, 3, False, 4)
    for kw in (dict(token_mask=torch.zeros(100, dtype=torch.uint8, device="cuda")), dict()):
        c = cuts if kw else torch.full_like(cuts, 50)
        out = lb.moe_router_loss(h, idx, c, alpha_seq=1e-2, z_coef=1e-2, **kw)
        dh = lb.moe_router_loss_grad(h, idx, c, out["counts"], out["tokens"], alpha_seq=1e-2, z_coef=1e-2, dgate=dgate, **kw)
        lb.sync_status()
        assert not any(bool(out[key].any()) for key in out) and not bool(dh.any())
    # no rows at all
    e = torch.empty(0, 12, device="cuda")
    ei = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    c = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = lb.moe_router_loss(e, ei, c)
    assert not any(bool(out[key].any()) for key in out)
    assert lb.moe_router_loss_grad(e, ei, c, out["counts"], out["tokens"]).shape == (0, 12)
    lb.sync_status()


@pytest.mark.parametrize("low", [-float("inf"), torch.finfo(torch.float32).min])
def test_router_loss_rows_without_scores(low):
    # rows that are -inf throughout have no scores; rows of the type's lowest value are an even softmax
    h, idx, _, _, dgate = loss_inputs(260, 20, 2, 1, False, 8)
    h[3] = low
    h[200:210] = low
    cuts = torch.tensor([0, 100, 260], dtype=torch.int32, device="cuda")
    z = 0.0 if low != -float("inf") else 1e-2
    for fn in (0, 1):
        ref = loss_ref(h, idx, cuts, None, fn, 1e-2, 1e-2, z, None)
        out = lb.moe_router_loss(h, idx, cuts, None, fn, alpha_seq=1e-2, z_coef=z)
        assert torch.equal(out["counts"], ref["counts"])
        assert np.allclose(out["loss"].tolist(), ref["loss"], rtol=REL, atol=1e-12)
        dh = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], None, fn, alpha_seq=1e-2, z_coef=z)
        within(dh, ref["dlogits"], 2 * REL * ref["mag"] + 1e-14, "dlogits")
        gated = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], None, fn, dgate=dgate, renorm_topk=1)
        assert bool(gated.isfinite().all())
    lb.sync_status()


def test_router_loss_reports_bad_picks_and_offsets():
    h, idx, cuts, _, _ = loss_inputs(300, 16, 2, 3, False, 9)
    cuts = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    good = lb.moe_router_loss(h, idx, cuts)
    idx2 = idx.clone()
    idx2[5, 0] = 16
    out = lb.moe_router_loss(h, idx2, cuts)
    with pytest.raises(lb.MoEError, match="expert index"):
        lb.sync_status()
    want = good["counts"].clone()
    want[[0, 3], int(idx[5, 0])] -= 1
    assert torch.equal(out["counts"], want)
    for bad in ([0, 200, 100, 300], [0, 100, 200, 301], [-4, 100, 200, 300]):
        lb.moe_router_loss(h, idx, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        with pytest.raises(lb.MoEError, match="sequence offsets"):
            lb.sync_status()


# ---------------------------------------------------------------- combine gradient
def combine_inputs(m, d, k, dtype, keep, seed, spare=5):
    g = gen(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    dy = torch.randn(m, d, generator=g, device="cuda").to(dt)
    dest = torch.randperm(m * k, generator=g, device="cuda")
    dest[torch.rand(m * k, generator=g, device="cuda") > keep] = -1
    ybuf = torch.randn(m * k + spare, d, generator=g, device="cuda").to(dt)
    gate = torch.rand(m, k, generator=g, device="cuda")
    return dy, ybuf, dest.view(m, k).to(torch.int32).contiguous(), gate


@pytest.mark.parametrize("m,d,k,dtype,keep", [
    (1, 8, 1, "bf16", 1.0), (3, 4096, 2, "bf16", 0.8), (1000, 768, 1, "bf16", 0.7), (513, 264, 2, "bf16", 0.9),
    (200, 128, 8, "bf16", 0.5), (64, 72, 5, "bf16", 0.9), (40, 2048, 33, "bf16", 0.9), (300, 4, 1, "fp32", 0.8),
    (777, 100, 3, "fp32", 0.8), (128, 1028, 6, "fp32", 1.0), (50, 64, 2, "bf16", 0.0), (1, 16384, 4, "bf16", 1.0),
    (33, 8200, 2, "fp32", 0.9)])
def test_combine_gradient(m, d, k, dtype, keep):
    dy, ybuf, dest, gate = combine_inputs(m, d, k, dtype, keep, m + d)
    dybuf = torch.full_like(ybuf, 3.0)
    got, dgate = lb.moe_combine_grad(dy, ybuf, dest, gate, dybuf=dybuf)
    lb.sync_status()
    kept = dest >= 0
    rows = dest.long().clamp(min=0)
    g = gate.to(dy.dtype).double()
    # one product of two values, rounded once
    want = torch.full_like(ybuf, 3.0)
    want[dest.long()[kept]] = (g[:, :, None] * dy.double()[:, None])[kept].to(dy.dtype)
    assert torch.equal(got, want)
    prod = ybuf[rows].double() * dy.double()[:, None] * kept[:, :, None]
    # a lane adds d / 32 products in order (fewer in a wider reduction), the lanes' sums in five more steps
    within(dgate, prod.sum(-1), (d / 32 + 16) * EPS * prod.abs().sum(-1) + 1e-30, "dgate")
    none, again = lb.moe_combine_grad(dy, ybuf, dest, gate, want_dybuf=False)
    assert none is None and torch.equal(again, dgate)
    fresh, _ = lb.moe_combine_grad(dy, ybuf, dest, gate)
    unnamed = torch.ones(ybuf.shape[0], dtype=torch.bool, device="cuda")
    unnamed[dest.long()[kept]] = False
    assert torch.equal(fresh[~unnamed], want[~unnamed]) and not bool(fresh[unnamed].any())


def test_combine_gradient_by_differences():
    # y is linear in the rows and in the gates
    dy, ybuf, dest, gate = combine_inputs(120, 64, 3, "fp32", 0.8, 21)
    dybuf, dgate = lb.moe_combine_grad(dy, ybuf, dest, gate)
    g = gen(22)
    vy, vg = torch.randn(ybuf.shape, generator=g, device="cuda"), torch.randn(gate.shape, generator=g, device="cuda")
    for key, v, grad in (("ybuf", vy, dybuf), ("gate", vg, dgate)):
        at = dict(ybuf=ybuf, gate=gate)
        up = lb.moe_combine(**{**{"ybuf": at["ybuf"], "dest_row": dest, "topk_gate": at["gate"]},
                               **({"ybuf": ybuf + v} if key == "ybuf" else {"topk_gate": gate + v})})
        down = lb.moe_combine(**{**{"ybuf": at["ybuf"], "dest_row": dest, "topk_gate": at["gate"]},
                                 **({"ybuf": ybuf - v} if key == "ybuf" else {"topk_gate": gate - v})})
        diff = ((up.double() - down.double()) / 2 * dy).sum()
        mag = (up.abs().double() * dy.abs()).sum() + (grad.abs().double() * v.abs()).sum()
        assert abs(float(diff - (grad.double() * v).sum())) <= 64 * EPS * float(mag), key


def test_combine_gradient_reports_rows_past_the_buffer():
    dy, ybuf, dest, gate = combine_inputs(20, 64, 2, "bf16", 1.0, 23, spare=0)
    bad = dest.clone()
    bad[4, 1] = 40
    dybuf, dgate = lb.moe_combine_grad(dy, ybuf, bad, gate)
    with pytest.raises(lb.MoEError, match="max_rows"):
        lb.sync_status()
    bad[4, 1] = -1
    want, wgate = lb.moe_combine_grad(dy, ybuf, bad, gate)
    assert torch.equal(dybuf, want) and torch.equal(dgate, wgate)


# ---------------------------------------------------------------- together, in graphs, on streams
def train_step(i, dy, ybuf_of, cuts, tm, k, stream=None):
    """One router training step on these inputs: logits, picks, combine gradient, losses, gradients."""
    kw = dict(stream=stream)
    n = i["w_r"].shape[1]
    logits, hidden = lb.moe_router_adapters(**i, **kw)
    idx, gate, _ = lb.moe_router_topk(None, None, n, k, renorm_topk=1, logits_in=logits, **kw)
    slots = lb.moe_capacity_slots(idx, n, 1 << 20, **kw)
    dybuf, dgate = lb.moe_combine_grad(dy, ybuf_of, slots["dest_row"], gate, **kw)
    out = lb.moe_router_loss(logits, idx, cuts, tm, alpha_seq=1e-2, z_coef=1e-3, **kw)
    dh = lb.moe_router_loss_grad(logits, idx, cuts, out["counts"], out["tokens"], tm, alpha_seq=1e-2, z_coef=1e-3,
                                 dgate=dgate, renorm_topk=1, **kw)
    dx, da, db, dw = lb.moe_router_adapters_grad(dh, hidden=hidden, want_dw_r=True, **i, **kw)
    return dict(out, logits=logits, dybuf=dybuf, dgate=dgate, dh=dh, dx=dx, da=da, db=db, dw=dw)


def step_inputs(seed, m=600, d=256, n=32, k=2):
    i, _ = adapter_inputs(m, d, n, 8, 5, torch.bfloat16, "runs", seed)
    g = gen(seed + 1)
    dy = torch.randn(m, d, generator=g, device="cuda").to(torch.bfloat16)
    ybuf = torch.randn(m * k, d, generator=g, device="cuda").to(torch.bfloat16)
    cuts = torch.tensor([0, 10, 10, 300, m - 50], dtype=torch.int32, device="cuda")
    tm = (torch.rand(m, generator=g, device="cuda") > 0.1).to(torch.uint8)
    return i, dy, ybuf, cuts, tm, k


def test_step_on_a_side_stream_and_in_a_graph():
    args = step_inputs(31)
    want = train_step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = train_step(*args, stream=side)
    side.synchronize()
    lb.sync_status(side)
    for key in want:
        assert torch.equal(got[key], want[key]), key
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = train_step(*args, stream=torch.cuda.current_stream())
    # new contents of the same buffers, replayed twice
    new = step_inputs(77)
    for key in args[0]:
        args[0][key].copy_(new[0][key])
    for old, fresh in zip(args[1:5], new[1:5]):
        old.copy_(fresh)
    want2 = train_step(*args)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for key in want2:
            assert torch.equal(cap[key], want2[key]), key
    lb.sync_status()


def test_two_steps_at_once_on_two_streams():
    a, b = step_inputs(41, m=900), step_inputs(42, m=5000, d=512, n=64)
    wa, wb = train_step(*a), train_step(*b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for _ in range(4):
        runs.append((train_step(*a, stream=s1), train_step(*b, stream=s2)))
    torch.cuda.synchronize()
    for ga, gb in runs:
        for key in wa:
            assert torch.equal(ga[key], wa[key]) and torch.equal(gb[key], wb[key]), key
    lb.sync_status()


def test_refusals_of_the_binding():
    i, dh = adapter_inputs(64, 128, 16, 8, 3, torch.bfloat16, "mixed", 1)
    _, hidden = lb.moe_router_adapters(**i)
    for key, bad in (("x", i["x"].t().contiguous().t()), ("a", i["a"].float()), ("b", i["b"][:, :, :4].contiguous()),
                     ("adapter_idx", i["adapter_idx"].long()), ("scale", i["scale"].cpu()), ("w_r", i["w_r"].t())):
        with pytest.raises((ValueError, TypeError)):
            lb.moe_router_adapters(**dict(i, **{key: bad}))
    with pytest.raises(ValueError):
        lb.moe_router_adapters_grad(dh[:, :8].contiguous(), hidden=hidden, **i)
    with pytest.raises(ValueError):
        lb.moe_router_adapters_grad(dh, hidden=None, **i)
    with pytest.raises(lb.MoEError):  # a rank above 64
        lb.moe_router_adapters(i["x"], i["w_r"], i["a"].repeat(1, 9, 1), i["b"].repeat(1, 1, 9), i["adapter_idx"], i["scale"])
    with pytest.raises(lb.MoEError):  # rows that do not start on 16 bytes
        flat = torch.zeros(64 * 128 + 8, dtype=torch.bfloat16, device="cuda")
        lb.moe_router_adapters(**dict(i, x=flat[1:64 * 128 + 1].view(64, 128)))
    with pytest.raises(lb.MoEError):  # a short workspace
        lb.moe_router_adapters_grad(dh, hidden=hidden, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **i)
    h, idx, cuts, tm, dgate = loss_inputs(50, 8, 2, 3, True, 1)
    with pytest.raises(ValueError):
        lb.moe_router_loss(h, idx, cuts.long())
    with pytest.raises(ValueError):
        lb.moe_router_loss(h, idx, cuts, tm.bool())
    with pytest.raises(lb.MoEError):
        lb.moe_router_loss(h, idx, cuts, alpha=float("nan"))
    dy, ybuf, dest, gate = combine_inputs(20, 64, 2, "bf16", 1.0, 1)
    with pytest.raises(lb.MoEError):
        lb.moe_combine_grad(dy, ybuf, dest, gate, dybuf=ybuf)
    with pytest.raises(ValueError):
        lb.moe_combine_grad(dy, ybuf.float(), dest, gate)


@pytest.mark.parametrize("m,d,n,r,na,order", [(20000, 512, 64, 16, 7, "runs"), (9000, 640, 128, 40, 30, "mixed"),
                                              (30, 2048, 64, 16, 24, "mixed"), (12000, 256, 32, 8, 3, "patches")])
def test_calls_that_follow_one_another(m, d, n, r, na, order):
    # nothing waits between the calls: a kernel's prologue overlaps the one before it, and slabs of rows that follow
    # one another take turns with gathered ones
    i, dh = adapter_inputs(m, d, n, r, na, torch.bfloat16, "runs" if order == "patches" else order, 51)
    if order == "patches":
        g = gen(52)
        at = torch.randint(0, m, (60,), generator=g, device="cuda")
        i["adapter_idx"][at] = torch.randint(-1, na, (60,), generator=g, device="cuda", dtype=torch.int32)
    first = lb.moe_router_adapters(**i)
    grads = lb.moe_router_adapters_grad(dh, hidden=first[1], want_dw_r=True, **i)
    lb.sync_status()
    outs = []
    for _ in range(40):
        f = lb.moe_router_adapters(**i)
        outs.append((f, lb.moe_router_adapters_grad(dh, hidden=f[1], want_dw_r=True, **i)))
        outs = outs[-3:]
    lb.sync_status()
    for f, b in outs:
        for p, q in zip(f + b, first + grads):
            assert torch.equal(p, q)


@pytest.mark.parametrize("m,d,n,r,na", [(700, 520, 64, 16, 3), (300, 264, 40, 50, 2), (260, 512, 128, 8, 2),
                                        (300, 200, 100, 64, 3), (515, 392, 256, 16, 4), (140, 128, 200, 40, 2)])
def test_adapters_backward_dx_keeps_fp32_sums(m, d, n, r, na):
    # the gradient of a softmax adds up to zero over the experts, so what the columns of W_r have in common cancels in
    # dx: what is left has to be right to fp32 sums of the products, not to a multiple of the common part
    i, dh = adapter_inputs(m, d, n, r, na, torch.bfloat16, "mixed", 71)
    g = gen(72)
    p = torch.softmax(dh, 1)
    dh = p * (dh - (p * dh).sum(1, keepdim=True))
    i["w_r"] = 8 * torch.randn(d, 1, generator=g, device="cuda") + i["w_r"] / 8
    i["b"] = (i["b"].float() + 1).to(torch.bfloat16)  # B_a's columns have a common part as well
    dx, _, _, _ = lb.moe_router_adapters_grad(dh, hidden=torch.zeros(m, r, device="cuda"), **i)
    lb.sync_status()
    w, a, b, s = (i[k].double() for k in ("w_r", "a", "b", "scale"))
    dh64 = dh.double()
    ref, mag = dh64 @ w.T, dh64.abs() @ w.abs().T
    for q in range(na):
        rows = (i["adapter_idx"] == q).nonzero()[:, 0]
        ref[rows] += s[q] * dh64[rows] @ b[q] @ a[q]
        mag[rows] += s[q] * dh64[rows].abs() @ b[q].abs() @ a[q].abs()
    assert float((mag / ref.abs().clamp(min=1e-30)).median()) > 50
    # three products of the parts for each 16 experts and each 16 ranks, an eps each (12 ceil(n / 64) + 12 steps); du is
    # a sum of n products; what two fp16 parts a side leave out is below 3 * 2^-22, six eps
    within(dx, ref, 2.0 ** -8 * ref.abs() + (12 * -(-n // 64) + 12 + n + 6) * EPS * mag, "dx")


@pytest.mark.parametrize("m,d,n,r,na", [(300, 264, 64, 16, 3), (200, 136, 200, 40, 2)])
def test_adapters_backward_dx_at_any_scale(m, d, n, r, na):
    # rows of dlogits and of W_r (which the kernels scale to fit fp16 parts) of very different sizes, some all zero, next
    # to adapters that are not as large or small as their row of W_r; elements of a row that differ by up to 2^12
    i, dh = adapter_inputs(m, d, n, r, na, torch.bfloat16, "mixed", 73)
    g = gen(74)

    def powers(low, high, *shape):
        return 2.0 ** torch.randint(low, high + 1, shape, generator=g, device="cuda").float()
    dh = dh * powers(-110, 30, m, 1) * powers(-12, 0, m, n)
    i["w_r"] = i["w_r"] * powers(-30, 30, d, 1) * powers(-12, 0, d, n)
    i["a"] = (i["a"].float() * powers(-20, 10, na, r, d)).to(torch.bfloat16)
    dh[5], dh[17, 1:], i["w_r"][3] = 0, 0, 0
    dx, _, _, _ = lb.moe_router_adapters_grad(dh, hidden=torch.zeros(m, r, device="cuda"), **i)
    lb.sync_status()
    w, a, b, s = (i[k].double() for k in ("w_r", "a", "b", "scale"))
    dh64 = dh.double()
    ref, mag = dh64 @ w.T, dh64.abs() @ w.abs().T
    for q in range(na):
        rows = (i["adapter_idx"] == q).nonzero()[:, 0]
        ref[rows] += s[q] * dh64[rows] @ b[q] @ a[q]
        mag[rows] += s[q] * dh64[rows].abs() @ b[q].abs() @ a[q].abs()
    # as above, 2^-38 of the largest product of the row's and the column's values for each of n terms, and half a step of
    # bf16's subnormal values
    top = 2.0 ** -134 + n * 2.0 ** -38 * dh64.abs().amax(1)[:, None] * w.abs().amax(1)
    within(dx, ref, 2.0 ** -8 * ref.abs() + (12 * -(-n // 64) + 12 + n + 6) * EPS * mag + top, "dx")
    assert not bool(dx[5].any())


@pytest.mark.parametrize("n,r", [(64, 16), (40, 33), (128, 8), (100, 64), (256, 16), (200, 40)])
@pytest.mark.parametrize("side", ["dlogits", "w_r", "du"])
def test_adapters_backward_dx_is_exact_where_fp32_is(n, r, side):
    # pairs of 21-bit integers (times 2^-20) that add up to at most 16: fp32 sums of four pairs are exact, and so is
    # their bf16 value; parts that keep fewer than 21 bits of dlogits, W_r or du are off by about a unit of the sum
    m, d = 300, 264
    g = gen(75 + n)
    i, dh = adapter_inputs(m, d, n, r, 3, torch.bfloat16, "mixed", 76)
    i["scale"].fill_(1.0)
    wide = d if side == "w_r" else m
    q = torch.randint(2 ** 20, 2 ** 21, (wide, n // 2), generator=g, device="cuda")
    small = torch.randint(-16, 17, (wide, n // 2), generator=g, device="cuda")
    pairs = torch.stack([q, small - q], 2).view(wide, -1)  # columns 2 p and 2 p + 1 belong together
    pick = torch.randint(0, min(n, r) // 2 if side == "du" else n // 2, (m,), generator=g, device="cuda")
    both = (torch.arange(n // 2, device="cuda") == pick[:, None]).repeat_interleave(2, 1)
    if side == "w_r":  # a row of dlogits names one pair of each row of W_r
        dh = both.float()
        i["w_r"] = pairs.float() * 2.0 ** -20
        i["adapter_idx"].fill_(-1)
        want = small[:, pick].T.float() * 2.0 ** -20
    else:
        dh = (pairs * both).float() * 2.0 ** -20
        total = small.gather(1, pick[:, None]).float() * 2.0 ** -20
        if side == "dlogits":
            i["w_r"] = torch.ones_like(i["w_r"])
            i["adapter_idx"].fill_(-1)
        else:  # du takes the values over one by one, and A_a adds them up
            i["w_r"] = torch.zeros_like(i["w_r"])
            i["a"] = torch.ones_like(i["a"])
            i["b"] = torch.eye(n, r, device="cuda").to(torch.bfloat16).repeat(3, 1, 1)
            total = total * (i["adapter_idx"] >= 0)[:, None]
        want = total.expand(m, d)
    dx, _, _, _ = lb.moe_router_adapters_grad(dh, hidden=torch.zeros(m, r, device="cuda"), **i)
    lb.sync_status()
    assert torch.equal(dx.float(), want)


# ---------------------------------------------------------------- the gates that the router gives and their gradient
@pytest.mark.parametrize("m,d,n,dtype,probs", [
    (300, 0, 64, None, True), (200, 0, 256, None, False), (517, 768, 128, "bf16", True), (20000, 64, 64, "bf16", True),
    (400, 128, 100, "bf16", False), (259, 128, 256, "bf16", True), (100, 64, 8, "fp32", True)])
def test_one_pick_keeps_its_score_when_renormalising(m, d, n, dtype, probs):
    # renorm_topk is for two picks and more: one pick's gate is its softmax score, on every path of the router
    g = gen(m + n)
    if dtype is None:
        x = w = None
        kw = dict(logits_in=torch.randn(m, n, generator=g, device="cuda"))
    else:
        x = torch.randn(m, d, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        w = torch.randn(d, n, generator=g, device="cuda") / d ** 0.5
        kw = {}
    idx, gate, p = lb.moe_router_topk(x, w, n, 1, renorm_topk=1, want_probs=probs, **kw)
    idx0, gate0, _ = lb.moe_router_topk(x, w, n, 1, renorm_topk=0, want_probs=probs, **kw)
    lb.sync_status()
    assert torch.equal(idx, idx0) and torch.equal(gate, gate0)
    if probs:
        assert torch.equal(gate, p.gather(1, idx.long()))


@pytest.mark.parametrize("fn,renorm,k", [(0, 0, 1), (0, 1, 1), (0, 0, 3), (0, 1, 3), (1, 0, 2), (1, 1, 1)])
def test_gate_gradient_by_differences_of_the_router(fn, renorm, k):
    # sum_r dgate_r gate_r with the gates that moe_router_topk itself gives; the bias keeps the picks fixed
    m, n, step = 200, 16, 2.0 ** -7
    g = gen(91)
    h = torch.randn(m, n, generator=g, device="cuda")
    v = torch.randn(m, n, generator=g, device="cuda").clamp(-2, 2)
    dgate = torch.randn(m, k, generator=g, device="cuda")
    bias = torch.zeros(n, device="cuda")
    bias[:k] = torch.arange(k, 0, -1, device="cuda") * 4.0
    cuts = torch.tensor([0, m], dtype=torch.int32, device="cuda")

    def gates(logits):
        idx, gate, _ = lb.moe_router_topk(None, None, n, k, fn, renorm, rank_bias=bias, logits_in=logits)
        assert torch.equal(idx, torch.arange(k, device="cuda", dtype=torch.int32).expand(m, k))
        return idx.contiguous(), gate
    idx, gate = gates(h)
    out = lb.moe_router_loss(h, idx, cuts, None, fn, alpha=0.0)
    dh = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], None, fn, alpha=0.0, dgate=dgate,
                                 renorm_topk=renorm)
    diff = ((gates(h + step * v)[1].double() - gates(h - step * v)[1].double()) / (2 * step) * dgate).sum(1)
    lb.sync_status()
    # a gate is off by 16 eps of itself on each side; a score's third derivative along v is at most 8 |v|_inf^3 of its
    # weight (a softmax's is p times a cubic in the centred steps, |v_j - mean| <= 2 |v|_inf, with coefficients 1, 3, 2:
    # at most 48 |v|^3 p), step^2 / 6 of it remains
    mag = (gate.double() * dgate.abs()).sum(1)
    bound = 16 * EPS * mag / step + 48 * 8 * step ** 2 / 6 * mag + 64 * EPS * (dh.abs() * v.abs()).sum(1) + 1e-9
    assert bool(((diff - (dh.double() * v).sum(1)).abs() <= bound).all())
    assert fn == 1 or renorm == 0 or k > 1 or bool((dh.abs().sum(1) > 0).any())


@pytest.mark.parametrize("fn", [0, 1])
def test_router_loss_gradient_with_pooled_counts(fn):
    # two ranks that put the sums of both into the last rows get the gradient of the loss of both batches
    h, idx, _, tm, _ = loss_inputs(700, 48, 2, 3, True, 33)
    cut, coef = 300, dict(alpha=1e-2, z_coef=1e-3)
    whole = torch.tensor([0, 700], dtype=torch.int32, device="cuda")
    both = lb.moe_router_loss(h, idx, whole, tm, fn, **coef)
    want = lb.moe_router_loss_grad(h, idx, whole, both["counts"], both["tokens"], tm, fn, **coef)
    parts = []
    for rows in (slice(0, cut), slice(cut, 700)):
        part = [t[rows].contiguous() for t in (h, idx, tm)]
        ends = torch.tensor([0, len(part[0])], dtype=torch.int32, device="cuda")
        parts.append((part, ends, lb.moe_router_loss(part[0], part[1], ends, part[2], fn, **coef)))
    counts = sum(out["counts"][-1] for _, _, out in parts)
    tokens = sum(out["tokens"][-1] for _, _, out in parts)
    assert torch.equal(counts, both["counts"][-1]) and int(tokens) == int(both["tokens"][-1])
    got = []
    for (ph, pi, pm), ends, out in parts:
        out["counts"][-1], out["tokens"][-1] = counts, tokens
        got.append(lb.moe_router_loss_grad(ph, pi, ends, out["counts"], out["tokens"], pm, fn, **coef))
    lb.sync_status()
    assert torch.equal(torch.cat(got), want)


@pytest.mark.parametrize("fn", [0, 1])
@pytest.mark.parametrize("n", [8, 16, 32, 64, 100, 200])
def test_router_loss_scores_are_right_to_a_few_roundings(fn, n):
    # logits that are multiples of 2^-5 down to -84: differences from the row's best are exact, so a score is off by the
    # exponential (2 ulp, four times 2^-24), the sum (that and 16 additions), the quotient and the product alone,
    # 2^-24 * (4 + 4 + 16 + 2); the mean is taken in 64 bits and rounded once. A logistic: 4 and two roundings
    m, k = 300, 2
    g = gen(81)
    step = torch.floor(torch.tensor(84.0 * 32 / (n - 1))) / 32
    h = (-step * torch.arange(n)).float().cuda()[torch.stack([torch.randperm(n, generator=g, device="cuda") for _ in range(m)])]
    h[:100] = h[0]
    h = h.contiguous()
    idx = torch.topk(h, k, dim=1).indices.to(torch.int32).contiguous()
    cuts = torch.tensor([0, 100, m], dtype=torch.int32, device="cuda")
    ref = loss_ref(h, idx, cuts, None, fn, 1e-2, 0.0, 0.0)
    out = lb.moe_router_loss(h, idx, cuts, None, fn)
    dh = lb.moe_router_loss_grad(h, idx, cuts, out["counts"], out["tokens"], None, fn)
    lb.sync_status()
    within(out["P"], ref["P"], (27 if fn == 0 else 8) * 2.0 ** -24 * ref["P"], "P")
    # softmax, p (g - sum p g): g 3 roundings, p 26, the sum 26 and 3 and 16; logistic, g t w w: 3, 4, 6, 6 and 3
    within(dh, ref["dlogits"], (80 if fn == 0 else 24) * 2.0 ** -24 * ref["mag"] + 1e-37, "dlogits")


@pytest.mark.parametrize("order", ["runs", "mixed"])
@pytest.mark.parametrize("m,d,n,r,na", [
    (2600, 512, 64, 16, 6),    # W_r's parts and A_a in one operand
    (2600, 200, 128, 40, 3),   # two column tiles, rank above 32
    (20000, 64, 128, 8, 5),    # operands apart: 128 and 96 columns
    (19500, 72, 90, 32, 3), (2300, 136, 200, 64, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_adapters_do_not_mix_rows_on_the_tensor_cores(m, d, n, r, na, order, bad):
    # the rows before and behind a group's end: a box of 32 rows takes in rows of the next group, stages keep old rows
    i, dh = adapter_inputs(m, d, n, r, na, torch.bfloat16, order, m + n)
    assert lb.moe_router_adapters_workspace_size(m, d, n, r, na) > 0  # not the kernel of few rows
    idx = i["adapter_idx"]
    ends = (idx[1:] != idx[:-1]).nonzero()[:, 0]
    ends = ends[torch.randperm(len(ends), generator=gen(5), device="cuda")[:7]]
    clean = lb.moe_router_adapters(**i)
    want = lb.moe_router_adapters_grad(dh, hidden=clean[1], want_dw_r=True, **i)
    for rows in (ends, ends + 1, torch.tensor([0, m - 1], device="cuda")):
        rest = torch.ones(m, dtype=torch.bool, device="cuda")
        rest[rows] = False
        x = i["x"].clone()
        x[rows, 3] = bad
        logits, hidden = lb.moe_router_adapters(**dict(i, x=x))
        assert torch.equal(logits[rest], clean[0][rest]) and torch.equal(hidden[rest], clean[1][rest])
        assert not bool(logits[rows].isfinite().any())
        assert not bool(hidden[rows][idx[rows] >= 0].isfinite().any()) and not bool(hidden[rows][idx[rows] < 0].any())
        hit = torch.zeros(na, dtype=torch.bool, device="cuda")
        hit[idx[rows][idx[rows] >= 0].long()] = True
        cols = torch.arange(d, device="cuda") != 3
        # x: column 3 of its adapters' dA and of dW_r, nothing else
        dx, da, db, dw = lb.moe_router_adapters_grad(dh, hidden=clean[1], want_dw_r=True, **dict(i, x=x))
        assert torch.equal(dx, want[0]) and torch.equal(db, want[2])
        assert torch.equal(da[~hit], want[1][~hit]) and torch.equal(da[:, :, cols], want[1][:, :, cols])
        assert not bool(da[hit][:, :, 3].isfinite().any())
        assert torch.equal(dw[cols], want[3][cols]) and not bool(dw[3].isfinite().any())
        # dlogits: its own row of dx, its adapters' dA and dB, a column of dW_r
        dh2 = dh.clone()
        dh2[rows, 1] = bad
        dx, da, db, dw = lb.moe_router_adapters_grad(dh2, hidden=clean[1], want_dw_r=True, **i)
        assert torch.equal(dx[rest], want[0][rest]) and not bool(dx[rows].isfinite().any())
        assert torch.equal(da[~hit], want[1][~hit]) and torch.equal(db[~hit], want[2][~hit])
        assert not bool(da[hit].isfinite().any()) and not bool(db[hit][:, 1].isfinite().any())
        other = torch.arange(n, device="cuda") != 1
        assert torch.equal(dw[:, other], want[3][:, other]) and not bool(dw[:, 1].isfinite().any())
    lb.sync_status()
