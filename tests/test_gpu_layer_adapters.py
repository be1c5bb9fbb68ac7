"""The layer with low-rank adapters beside its router: forward as composed by hand, backward by differences, graphs."""
import pytest
import torch

import workloads as W
from load_balanced_dispatch_b200.layer import LayerShape, MoELayer, weights_to_device

pytestmark = pytest.mark.gpu

lb = pytest.importorskip("load_balanced_dispatch_b200")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from load_balanced_dispatch_b200 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    lb.sync_status()


def make(name, seed=3, na=3, r=4, **kw):
    cfg = W.scaled_config(name, **kw)
    inp = W.make_layer_inputs(cfg, seed=seed)
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    layer = MoELayer(LayerShape(m=cfg.m, d=cfg.d, n=cfg.n, k=cfg.k, d_ff=cfg.d_ff, score_fn=cfg.score_fn, dtype=dt,
                                capacity=cfg.capacity, seg_len=cfg.seg_len, renorm_topk=cfg.renorm_topk),
                     weights_to_device(inp, dt))
    x = torch.from_numpy(inp["x"]).to("cuda", dt)
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = (torch.randn(na, r, cfg.d, generator=g, device="cuda") / cfg.d ** 0.5).to(dt)
    b = (torch.randn(na, cfg.n, r, generator=g, device="cuda") * 0.3).to(dt)
    scale = torch.rand(na, generator=g, device="cuda") + 0.5
    idx = torch.randint(-1, na, (cfg.m,), generator=g, device="cuda", dtype=torch.int32)
    dy = torch.randn(cfg.m, cfg.d, generator=g, device="cuda").to(dt)
    return layer, x, dict(a=a, b=b, scale=scale, adapter_idx=idx), dy


TINY = dict(m=192, d=64, d_ff=64, n=8, k=2, capacity=192, seg_len=192)
GLOBAL = dict(m=2304, d=512, d_ff=128, seg_len=768, capacity=200)
SWITCH = dict(m=512, d=256, d_ff=128, seg_len=512, capacity=6)


@pytest.mark.parametrize("name,kw,r", [("tiny", TINY, 4), ("global", GLOBAL, 16), ("switch", SWITCH, 8)])
def test_forward_with_adapters(name, kw, r):
    layer, x, ad, _ = make(name, r=r, **kw)
    s = layer.shape
    plain = layer.forward(x).clone()
    layer.enable_adapters(**ad)
    y = layer.forward(x).clone()
    lb.sync_status()
    assert not torch.equal(plain, y)
    # by hand, from the adapters' logits on
    logits, _ = lb.moe_router_adapters(x, layer.w["w_r"], **ad)
    idx, gate, _ = lb.moe_router_topk(None, None, s.n, s.k, renorm_topk=s.renorm_topk, logits_in=logits)
    slots = lb.moe_capacity_slots(idx, s.n, s.capacity, s.seg_len or s.m)
    xbuf = lb.moe_dispatch_tokens(x, slots["dest_row"], s.m * s.k)
    ybuf = lb.moe_expert_ffn(xbuf, layer.w["w1"], layer.w["b1"], layer.w["w2"], layer.w["b2"], slots["expert_offsets"])
    assert torch.equal(layer.buf["topk_idx"], idx) and torch.equal(layer.buf["dest_row"], slots["dest_row"])
    assert torch.equal(y, lb.moe_combine(ybuf, slots["dest_row"], gate))
    # no adapter anywhere: the logits of the shared projection alone
    ad["adapter_idx"].fill_(-1)
    layer.forward(x)
    want = x.double() @ layer.w["w_r"].double()
    mag = x.double().abs() @ layer.w["w_r"].double().abs()
    assert bool(((layer.buf["logits"].double() - want).abs() <= (64 + s.d / 16) * 2.0 ** -23 * mag).all())
    # captured: follows what adapter_idx holds at the replay
    layer.capture(x)
    ad["adapter_idx"].copy_(torch.randint(-1, 3, (s.m,), device="cuda", dtype=torch.int32))
    got = layer.replay().clone()
    assert torch.equal(got, layer.forward(x))
    lb.sync_status()


def test_router_backward_by_differences():
    # J = <y, dy> + the router's losses, with the picks fixed; the layer in fp32
    layer, x, ad, dy = make("tiny", seed=8, **TINY)
    layer.shape.renorm_topk = 1
    layer.shape.alpha = 0.5
    layer.enable_adapters(**ad)
    cuts = torch.tensor([0, 50, 50, 180], dtype=torch.int32, device="cuda")
    kw = dict(alpha_seq=0.2, z_coef=0.05)
    dy[180:] = 0  # padding: neither in y's objective nor in the losses
    layer.forward(x)
    out = layer.router_backward(x, dy, cuts, want_dw_r=True, **kw)
    lb.sync_status()
    picks = layer.buf["topk_idx"].clone()  # held fixed: another logit may overtake one at a step

    def objective():
        logits, _ = lb.moe_router_adapters(x, layer.w["w_r"], **ad)
        gate = torch.softmax(logits.double().gather(1, picks.long()), 1).float()
        terms = lb.moe_combine(layer.buf["ybuf"], layer.buf["dest_row"], gate).double() * dy.double()
        loss = lb.moe_router_loss(logits, picks, cuts, alpha=0.5, **kw)["loss"][0]
        return float(terms.sum() + loss.double()), float(terms.abs().sum(1).square().sum().sqrt())

    g = torch.Generator(device="cuda").manual_seed(1)
    for key, grad in (("a", out["da"]), ("b", out["db"]), ("w_r", out["dw_r"])):
        p = layer.w["w_r"] if key == "w_r" else ad[key]
        v = torch.randn(p.shape, generator=g, device="cuda") * p.abs().mean()
        old, found, rows = p.clone(), [], 0.0
        for h in (2.0 ** -6, 2.0 ** -7):
            p.copy_(old + h * v)
            up, rows = objective()
            p.copy_(old - h * v)
            found.append((up - objective()[0]) / (2 * h))
        p.copy_(old)
        # a row's terms share the errors of its logits and gates, below 2^-21 of their magnitude, and the rows' errors
        # are independent: six deviations of their sum, over the smaller step; a central difference's curvature part
        # falls by four with the step, so the two differences show three times what the second one has
        slack = 6 * 2.0 ** -21 * rows / 2.0 ** -7 + abs(found[0] - found[1])
        assert abs(found[1] - float((grad.double() * v).sum())) <= slack, key


def test_router_backward_shapes_and_pieces():
    layer, x, ad, dy = make("global", r=16, **GLOBAL)
    layer.enable_adapters(**ad)
    cuts = torch.tensor([0, 700, 1500, 2304], dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError):
        MoELayer(layer.shape, layer.w).router_backward(x, dy, cuts)
    layer.forward(x)
    out = layer.router_backward(x, dy, cuts, alpha_seq=1e-3, z_coef=1e-3)
    lb.sync_status()
    b = layer.buf
    dybuf, dgate = lb.moe_combine_grad(dy, b["ybuf"], b["dest_row"], b["topk_gate"])
    assert torch.equal(out["dybuf"], dybuf) and torch.equal(out["dgate"], dgate) and out["dw_r"] is None
    logits, hidden = lb.moe_router_adapters(x, layer.w["w_r"], **ad)
    dx, da, db, _ = lb.moe_router_adapters_grad(out["dlogits"], x, layer.w["w_r"], hidden=hidden, **ad)
    for key, want in (("dx", dx), ("da", da), ("db", db)):
        assert torch.equal(out[key], want), key


def test_router_backward_on_a_side_stream_with_growing_batches():
    # the sequences grow from call to call, other work allocates and writes on the main stream, nothing waits in between
    layer, x, ad, dy = make("global", r=16, **GLOBAL)
    layer.enable_adapters(**ad)
    layer.forward(x)
    cuts = [torch.linspace(0, 2304, nseq + 1, device="cuda").to(torch.int32) for nseq in (1, 7, 300, 2000)]
    want = [layer.router_backward(x, dy, c, alpha_seq=1e-3, want_dw_r=True) for c in cuts]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(3):
        for c in cuts:
            got.append(layer.router_backward(x, dy, c, alpha_seq=1e-3, want_dw_r=True, stream=side))
            for size in (1 << 16, 1 << 20, 1 << 23):
                torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    lb.sync_status()
    for j, out in enumerate(got):
        for key in out:
            assert torch.equal(out[key], want[j % len(cuts)][key]), (key, j)


def test_router_backward_captured_before_a_larger_batch():
    # a captured backward keeps its memory when a later call has more sequences
    layer, x, ad, dy = make("tiny", **TINY)
    layer.enable_adapters(**ad)
    layer.forward(x)
    few = torch.tensor([0, 60, 192], dtype=torch.int32, device="cuda")
    many = torch.arange(0, 193, dtype=torch.int32, device="cuda")
    want = layer.router_backward(x, dy, few, alpha_seq=1e-2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.router_backward(x, dy, few, alpha_seq=1e-2)
    eager = layer.router_backward(x, dy, many, alpha_seq=1e-2)
    keep = {key: t.clone() for key, t in eager.items() if t is not None}
    graph.replay()
    torch.cuda.synchronize()
    for key, t in want.items():
        assert t is None or torch.equal(got[key], t), key
    for key, t in keep.items():
        assert torch.equal(eager[key], t), key


def test_capture_then_enable_then_enable_again():
    layer, x, ad, dy = make("switch", r=8, **SWITCH)
    _, _, other, _ = make("switch", seed=9, na=2, r=16, **SWITCH)
    cuts = torch.tensor([0, 100, 512], dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError):
        layer.replay()
    layer.capture(x)
    plain = layer.replay().clone()
    for adapters in (ad, other, ad):
        layer.enable_adapters(**adapters)
        with pytest.raises(RuntimeError):
            layer.replay()
        layer.capture(x)
        for t in layer.buf.values():  # what the replay does not write would show
            if t.dtype.is_floating_point:
                t.fill_(float("nan"))
        got = layer.replay().clone()
        out = layer.router_backward(x, dy, cuts)
        lb.sync_status()
        logits, hidden = lb.moe_router_adapters(x, layer.w["w_r"], **adapters)
        assert torch.equal(layer.buf["logits"], logits) and torch.equal(layer.buf["hidden"], hidden)
        assert not torch.equal(got, plain) and torch.equal(got, layer.forward(x))
        assert all(bool(out[key].isfinite().all()) for key in ("da", "db", "dx", "dlogits"))


@pytest.mark.parametrize("name,kw,r", [("tiny", TINY, 4), ("global", GLOBAL, 16), ("switch", SWITCH, 8)])
def test_serving_forward_and_back_to_the_plain_layer(name, kw, r):
    layer, x, ad, _ = make(name, r=r, **kw)
    fused, launches = layer.ffn_combine, layer.launches_per_forward()
    plain = layer.forward(x).clone()
    layer.enable_adapters(**ad)
    want = layer.forward(x).clone()
    layer.enable_adapters(**ad, backward=False)
    assert layer.ffn_combine == fused == (layer.buf["ybuf"].shape[0] == 0)
    assert torch.equal(layer.forward(x), want)
    layer.capture(x)
    assert torch.equal(layer.replay(), want)
    layer.disable_adapters()
    with pytest.raises(RuntimeError):
        layer.replay()
    assert torch.equal(layer.forward(x), plain) and layer.launches_per_forward() == launches
    layer.capture(x)
    assert torch.equal(layer.replay(), plain)
    lb.sync_status()
