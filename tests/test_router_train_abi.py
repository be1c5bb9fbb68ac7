"""Argument checks and workspace queries of the trainable router's entry points (host only: nothing is launched)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def L():
    from load_balanced_dispatch_b200 import build
    build.build()
    import load_balanced_dispatch_b200 as lb
    return lb.lib()


def _err(L):
    buf = C.create_string_buffer(256)
    L.moe_last_error(buf, 256)
    return buf.value.decode()


F = C.c_void_p(256)  # never dereferenced: validation fails first
ODD = C.c_void_p(264)  # not 16-byte aligned
BIG = 1 << 40


@pytest.mark.parametrize("change,word", [
    (dict(dt=2), "dtype"), (dict(m=-1), "m must be"), (dict(m=(1 << 24) + 1), "m must be"), (dict(n=0), "n must be"),
    (dict(n=257), "n must be"), (dict(r=0), "r must be"), (dict(r=65), "r must be"), (dict(na=0), "n_adapters"),
    (dict(na=1025), "n_adapters"), (dict(d=0), "d must be"), (dict(d=12), "d must be"), (dict(d=1 << 21), "d must be"),
    (dict(x=None), "x and adapter_idx"), (dict(x=ODD), "aligned"), (dict(w=None), "required"), (dict(a=None), "required"),
    (dict(scale=None), "required"), (dict(idx=None), "adapter_idx"), (dict(a=ODD), "aligned"), (dict(out=ODD), "aligned"),
    (dict(out=None), "required")])
def test_adapters_refusals(L, change, word):
    v = dict(dict(dt=1, m=64, d=128, n=16, r=8, na=3, x=F, w=F, a=F, b=F, idx=F, scale=F, out=F), **change)
    rc = L.moe_router_adapters(v["x"], v["dt"], v["w"], v["a"], v["b"], v["idx"], v["scale"], v["m"], v["d"], v["n"],
                               v["r"], v["na"], v["out"], None, F, BIG, None)
    assert rc == 1 and word in _err(L)
    rc = L.moe_router_adapters_grad(F, v["x"], v["dt"], v["w"], v["a"], v["b"], v["idx"], v["scale"], F, v["m"],
                                    v["d"], v["n"], v["r"], v["na"], None, v["out"], F, None, F, BIG, None)
    assert rc == 1 and word in _err(L)


def test_adapters_backward_refusals(L):
    def call(dh=F, hidden=F, dx=None, x=F, ws=F, size=BIG):
        return L.moe_router_adapters_grad(dh, x, 1, F, F, F, F, F, hidden, 64, 128, 16, 8, 3, dx, F, F, None, ws, size, None)
    assert call(dh=None) == 1 and "dlogits" in _err(L)
    assert call(hidden=None) == 1 and "hidden" in _err(L)
    assert call(dx=F) == 1 and "alias" in _err(L)
    assert call(ws=None) == 3 and "workspace" in _err(L)
    assert call(size=16) == 3 and "workspace" in _err(L)
    assert call(ws=ODD) == 3


def test_router_loss_refusals(L):
    f = C.c_float

    def call(logits=F, idx=F, m=64, n=16, k=2, off=F, nseq=3, fn=0, alpha=0.01, loss=F, ws=F, size=BIG):
        return L.moe_router_loss(logits, idx, m, n, k, off, nseq, None, fn, f(alpha), f(0), f(0), loss, F, F, F, F, ws, size, None)
    for kw, word in ((dict(m=-1), "m must"), (dict(n=300), "n must"), (dict(k=17), "k must"), (dict(off=None), "seq_offsets"),
                     (dict(nseq=0), "nseq"), (dict(nseq=1 << 22), "nseq"), (dict(fn=3), "score"), (dict(alpha=float("inf")), "finite"),
                     (dict(logits=None), "logits"), (dict(logits=ODD), "aligned"), (dict(loss=None), "loss"),
                     (dict(m=1 << 31), "m * k")):
        assert call(**kw) == 1 and word in _err(L), kw
    assert call(ws=None) == 3 and call(size=8) == 3

    def grad(counts=F, dlogits=C.c_void_p(512), logits=F, k=2):
        return L.moe_router_loss_grad(logits, F, 64, 16, k, F, 3, None, 0, f(0.01), f(0), f(0), counts, F, None, None, 0, dlogits, None)
    assert grad(counts=None) == 1 and "counts" in _err(L)
    assert grad(dlogits=None) == 1 and "dlogits" in _err(L)
    assert grad(dlogits=F) == 1 and "alias" in _err(L)
    assert grad(k=0) == 1


def test_combine_grad_refusals(L):
    def call(dy=F, ybuf=C.c_void_p(512), dt=1, dest=F, gate=F, m=4, k=1, d=64, rows=4, dybuf=C.c_void_p(1024), dgate=F):
        return L.moe_combine_grad(dy, ybuf, dt, dest, gate, m, k, d, rows, dybuf, dgate, None)
    for kw, word in ((dict(dt=5), "dtype"), (dict(d=12), "d must"), (dict(k=0), "bad k"), (dict(rows=-1), "max_rows"),
                     (dict(dy=None), "required"), (dict(ybuf=None), "ybuf"), (dict(dgate=None), "required"),
                     (dict(dy=ODD), "aligned"), (dict(dybuf=C.c_void_p(512)), "alias"), (dict(dybuf=F), "alias")):
        assert call(**kw) == 1 and word in _err(L), kw


def test_workspace_queries(L):
    assert L.moe_router_loss_workspace_size(65536, 256, 48) >= 512 * 256 * 8
    assert L.moe_router_loss_workspace_size(0, 8, 1) > 0
    assert L.moe_router_adapters_grad_workspace_size(1024, 64, 8, 4, 3, 0) > 0
    assert L.moe_router_adapters_grad_workspace_size(-1, 64, 8, 4, 3, 0) == 0
