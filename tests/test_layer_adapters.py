"""The layer with adapters beside its router: what it asks of the entry points, and its refusals (host only: the entry
points are stood in for)."""
import pytest
import torch

from load_balanced_dispatch_b200 import layer as L


@pytest.fixture(scope="module", autouse=True)
def _built():
    from load_balanced_dispatch_b200 import build
    build.build()


@pytest.fixture
def calls(monkeypatch):
    """Stands in for the entry points that router_backward calls; the list of (name, keyword arguments)."""
    seen = []
    t = torch.zeros(1)
    gives = dict(moe_combine_grad=(t, t), moe_router_loss=dict(loss=t, counts=t, tokens=t, f=t, P=t),
                 moe_router_loss_grad=t, moe_router_adapters_grad=(t, t, t, None))
    for name, out in gives.items():
        monkeypatch.setattr(L, name, lambda *a, _n=name, _o=out, **kw: (seen.append((_n, kw)), _o)[1])
    return seen


def bare_layer(m=64, d=32, n=8, k=2, dtype=torch.bfloat16):
    """A layer after a forward with adapters, without its device buffers."""
    layer = object.__new__(L.MoELayer)
    layer.shape = L.LayerShape(m=m, d=d, n=n, k=k, d_ff=16, dtype=dtype)
    layer.device = torch.device("cpu")
    layer.w = dict(w_r=torch.zeros(d, n))
    layer.buf = {key: torch.zeros(1) for key in ("ybuf", "dest_row", "topk_gate", "logits", "topk_idx", "hidden", "probs")}
    layer.ws, layer.global_stats, layer.ffn_combine = {}, None, False
    layer.graphs = layer.graph_all = None
    layer.adapters = dict(a=torch.zeros(3, 4, d), b=torch.zeros(3, n, 4), scale=torch.zeros(3),
                          adapter_idx=torch.zeros(m, dtype=torch.int32), backward=True, ran=True,
                          split_combine=False)
    return layer


def test_router_backward_leaves_workspaces_to_the_stream_of_each_call(calls):
    # a workspace that the layer keeps would be made on the current stream and replaced when a batch has more sequences,
    # while `stream` may still use it
    layer, side = bare_layer(), object()
    for nseq in (1, 5, 500):
        layer.router_backward(torch.zeros(64, 32), torch.zeros(64, 32), torch.zeros(nseq + 1, dtype=torch.int32), stream=side)
    assert [name for name, _ in calls] == ["moe_combine_grad", "moe_router_loss", "moe_router_loss_grad",
                                           "moe_router_adapters_grad"] * 3
    assert all(kw["stream"] is side and kw.get("workspace") is None for _, kw in calls)
    assert not layer.ws


def some_adapters(layer, na=3, r=4):
    s = layer.shape
    return dict(a=torch.zeros(na, r, s.d, dtype=s.dtype), b=torch.zeros(na, s.n, r, dtype=s.dtype), scale=torch.zeros(na),
                adapter_idx=torch.zeros(s.m, dtype=torch.int32))


def test_enable_adapters_drops_a_captured_forward(monkeypatch):
    # a forward captured before is another one, and one captured with other adapters would write to buffers that are gone
    waited = []
    monkeypatch.setattr(torch.cuda, "synchronize", waited.append)
    layer = bare_layer()

    class Graph:
        def replay(self):
            raise AssertionError("a stale graph ran")
    for _ in range(2):
        layer.graphs, layer.graph_all = [Graph()] * 6, Graph()
        layer.enable_adapters(**some_adapters(layer))
        assert waited.pop() == layer.device
        with pytest.raises(RuntimeError, match="capture"):
            layer.replay()


@pytest.mark.parametrize("key,bad", [
    ("a", torch.zeros(3, 4, 24, dtype=torch.bfloat16)), ("a", torch.zeros(3, 4, 32)), ("a", torch.zeros(4, 32, dtype=torch.bfloat16)),
    ("b", torch.zeros(3, 4, 8, dtype=torch.bfloat16)), ("b", torch.zeros(2, 8, 4, dtype=torch.bfloat16)), ("scale", torch.zeros(2)),
    ("adapter_idx", torch.zeros(63, dtype=torch.int32)), ("adapter_idx", torch.zeros(64, dtype=torch.int64))])
def test_enable_adapters_refuses_and_changes_nothing(monkeypatch, key, bad):
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev: None)
    layer = bare_layer()
    before, buf = layer.adapters, dict(layer.buf)
    layer.graphs = layer.graph_all = "captured"
    with pytest.raises(ValueError, match=key):
        layer.enable_adapters(**dict(some_adapters(layer), **{key: bad}))
    assert layer.adapters is before and layer.buf == buf and layer.graph_all == "captured"


def test_enable_adapters_without_memory_leaves_the_plain_layer(monkeypatch):
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev: None)
    layer = bare_layer(k=1)
    layer.disable_adapters()
    layer.ffn_combine, layer.rows_max = True, 64
    empty = torch.empty

    def short(shape, **kw):
        if tuple(shape) == (64, 32):  # the expert rows
            raise torch.cuda.OutOfMemoryError("out of memory")
        return empty(shape, **kw)
    monkeypatch.setattr(torch, "empty", short)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        layer.enable_adapters(**some_adapters(layer))
    assert layer.adapters is None and layer.ffn_combine and "logits" not in layer.buf


def test_router_backward_needs_a_forward_with_these_adapters(monkeypatch, calls):
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev: None)
    layer = bare_layer()
    args = torch.zeros(64, 32), torch.zeros(64, 32), torch.zeros(2, dtype=torch.int32)
    layer.router_backward(*args)
    layer.enable_adapters(**some_adapters(layer))
    del calls[:]
    with pytest.raises(RuntimeError, match="forward"):  # logits and hidden are not there yet
        layer.router_backward(*args)
    assert not calls
    monkeypatch.setattr(L, "moe_router_adapters", lambda *a, **kw: None)
    monkeypatch.setattr(L, "moe_router_topk", lambda *a, **kw: None)
    layer._stage(0, args[0], None)
    layer.router_backward(*args)
    assert len(calls) == 4


def test_router_backward_refuses_pooled_statistics(calls):
    # the layer's balance loss is then the pooled one, whose gradient does not follow from this rank's counts
    layer = bare_layer()
    layer.global_stats = dict(m_total=128)
    with pytest.raises(RuntimeError, match="pooled"):
        layer.router_backward(torch.zeros(64, 32), torch.zeros(64, 32), torch.zeros(2, dtype=torch.int32))
    assert not calls


def test_serving_keeps_the_fused_combine_and_refuses_the_backward(monkeypatch, calls):
    monkeypatch.setattr(torch.cuda, "synchronize", lambda dev: None)
    layer = bare_layer(k=1)
    layer.disable_adapters()
    layer.ffn_combine, layer.rows_max = True, 64
    layer.buf["ybuf"] = torch.zeros(0, 32, dtype=torch.bfloat16)
    args = torch.zeros(64, 32), torch.zeros(64, 32), torch.zeros(2, dtype=torch.int32)
    for backward in (False, True, True, False):
        layer.enable_adapters(**some_adapters(layer), backward=backward)
        assert layer.ffn_combine is not backward
        assert layer.buf["ybuf"].shape == ((64 if backward else 0), 32) and ("hidden" in layer.buf) == backward
        layer.adapters["ran"] = True
        if backward:
            layer.router_backward(*args)
        else:
            with pytest.raises(RuntimeError, match="backward"):
                layer.router_backward(*args)
    layer.enable_adapters(**some_adapters(layer))
    layer.disable_adapters()
    assert layer.adapters is None and layer.ffn_combine and layer.buf["ybuf"].shape == (0, 32)
    assert not {"logits", "hidden"} & set(layer.buf) and "adapters" not in layer.ws
    with pytest.raises(RuntimeError):
        layer.router_backward(*args)
