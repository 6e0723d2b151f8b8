"""CPU checks of the entry points around the layers: size queries and the refusal
of invalid arguments on the host."""
import ctypes
import os

import pytest

P = 4096   # any aligned, never-dereferenced address: validation fails first
R = ctypes.byref
BIG = 1 << 50


@pytest.fixture(scope="module")
def sl():
    import contextual_sparsity_lora_svd_amd as m
    if not os.path.exists(m.LIB_PATH):
        from contextual_sparsity_lora_svd_amd import build
        build.build(verbose=False)
    m.lib()
    return m


def test_embedding_refusals(sl):
    L, lay = sl.lib(), sl.Layout([0, 0], 4)
    nan, inf = float("nan"), float("inf")

    def fwd(dt=1, layout=lay, V=100, D=64, scale=1.0, E=P, ids=P, Y=P):
        return L.sl_embed_fwd(dt, layout.ref, V, D, scale, E, ids, Y, None)

    def bwd(dt=1, layout=lay, V=100, D=64, scale=1.0, ids=P, dY=P, gdt=0, dE=P, ws=P, n=BIG):
        return L.sl_embed_bwd(dt, layout.ref, V, D, scale, ids, dY, gdt, dE, ws, n, None)

    for f in (fwd, bwd):
        assert f() in (7, 8) and f(dt=0) in (7, 8) and f(D=8) in (7, 8) and f(D=65536, V=1 << 30) in (7, 8)
        assert f(dt=2) == 4
        assert f(ids=None) == 1 and f(ids=P + 4) == 2
        assert f(D=12) == 3 and f(D=0) == 3 and f(D=65544) == 3
        assert f(V=0) == 5 and f(V=(1 << 30) + 1) == 5
        assert f(scale=nan) == 5 and f(scale=inf) == 5
        assert f(layout=sl.Layout([0] * 65, 4)) == 5 and f(layout=sl.Layout([0], 0)) == 5
        assert f(layout=sl.Layout([0], (1 << 26) + 1)) == 5
    assert fwd(E=None) == 1 and fwd(Y=None) == 1 and fwd(E=P + 2) == 2 and fwd(Y=P + 8) == 2
    assert bwd(dY=None) == 1 and bwd(dE=None) == 1 and bwd(dY=P + 2) == 2 and bwd(dE=P + 8) == 2 and bwd(ws=P + 8) == 2
    assert bwd(gdt=1) in (7, 8) and bwd(gdt=2) == 4
    need = L.sl_embed_workspace_bytes(lay.ref, 64)
    assert need >= 2 * 8 * 4 + 2 * 64 * 4
    assert bwd(n=need) in (7, 8) and bwd(n=need - 1) == 6 and bwd(ws=None) == 6
    assert L.sl_embed_workspace_bytes(lay.ref, 60) == 0 and L.sl_embed_workspace_bytes(None, 64) == 0


def _norm(sl, D=64, centered=1, eps=1e-5, w=P, b=P):
    return sl.api.SlLayerNorm(D, centered, eps, w, b)


def test_layer_norm_refusals(sl):
    L, lay = sl.lib(), sl.Layout([0, 0], 4)

    def fwd(dt=1, layout=lay, p=None, x=P, r=P, h=P, y=P, stats=P):
        return L.sl_layer_norm_fwd(dt, layout.ref, R(p or _norm(sl)), x, r, h, y, stats, None)

    def bwd(dt=1, layout=lay, p=None, h=P, stats=P, dy=P, dh=P, dx=P, dw=P, db=P, ws=P, n=BIG):
        return L.sl_layer_norm_bwd(dt, layout.ref, R(p or _norm(sl)), h, stats, dy, dh, dx, dw, db, ws, n, None)

    for f in (fwd, bwd):
        assert f() in (7, 8) and f(dt=0) in (7, 8)
        assert f(p=_norm(sl, b=None)) in (7, 8) and f(p=_norm(sl, D=16384)) in (7, 8)
        assert f(dt=9) == 4
        assert f(p=_norm(sl, w=None)) == 1 and f(p=_norm(sl, w=P + 4)) == 2 and f(p=_norm(sl, b=P + 4)) == 2
        for D in (0, 4, 12, 16392, -8):
            assert f(p=_norm(sl, D=D)) == 3, D
        assert f(p=_norm(sl, centered=0)) == 3                  # a bias, not centred
        for eps in (-1.0, float("nan"), float("inf")):
            assert f(p=_norm(sl, eps=eps)) == 5
        assert f(layout=sl.Layout([0] * 65, 4)) == 5 and f(layout=sl.Layout([0], 0)) == 5
    rms = _norm(sl, centered=0, b=None)
    assert fwd(p=rms) in (7, 8) and fwd(r=None, h=None, stats=None) in (7, 8)
    assert fwd(x=None) == 1 and fwd(y=None) == 1 and fwd(r=None) == 1 and fwd(h=None) == 1
    assert fwd(x=P + 2) == 2 and fwd(r=P + 8) == 2 and fwd(stats=P + 4) == 2
    assert bwd(p=rms) == 3 and bwd(p=rms, db=None) in (7, 8) and bwd(dh=None, db=None) in (7, 8)
    assert bwd(h=None) == 1 and bwd(stats=None) == 1 and bwd(dy=None) == 1 and bwd(dx=None) == 1 and bwd(dw=None) == 1
    assert bwd(dh=P + 2) == 2 and bwd(dx=P + 8) == 2 and bwd(db=P + 4) == 2 and bwd(ws=P + 8) == 2
    need = L.sl_layer_norm_workspace_bytes(lay.ref, 64)
    assert need > 0 and need % (2 * 64 * 4) == 0
    for dt in (0, 1):
        assert bwd(dt=dt, n=need) in (7, 8)
    assert bwd(n=2 * 64 * 4 - 1) == 6 and bwd(ws=None) == 6
    assert L.sl_layer_norm_workspace_bytes(lay.ref, 60) == 0


def _targets(sl, V=100, top=5, tau=1.0, hard=0.5, ids=P, tl=P, labels=P):
    return sl.api.SlDistill(V, top, tau, hard, ids, tl, labels)


def test_distillation_refusals(sl):
    L, lay = sl.lib(), sl.Layout([4, 0], 4)

    def fwd(dt=1, layout=lay, p=None, z=P, ld=100, loss=P, stats=P):
        return L.sl_distill_fwd(dt, layout.ref, R(p or _targets(sl)), z, ld, loss, stats, None)

    def bwd(dt=1, layout=lay, p=None, z=P, ld=100, stats=P, g=P, dz=P, ldo=100):
        return L.sl_distill_bwd(dt, layout.ref, R(p or _targets(sl)), z, ld, stats, g, dz, ldo, None)

    def step(dt=1, layout=lay, p=None, z=P, ld=100, g=P, loss=P, dz=P, ldo=100):
        return L.sl_distill_step(dt, layout.ref, R(p or _targets(sl)), z, ld, g, loss, dz, ldo, None)

    for f in (fwd, bwd, step):
        assert f() in (7, 8) and f(dt=0) in (7, 8) and f(ld=101) in (7, 8)
        assert f(p=_targets(sl, hard=0.0, labels=None)) in (7, 8)
        assert f(p=_targets(sl, hard=1.0, top=0, ids=None, tl=None)) in (7, 8)
        assert f(p=_targets(sl, top=256)) in (7, 8) and f(p=_targets(sl, V=1)) in (7, 8)
        assert f(dt=3) == 4
        assert f(z=None) == 1 and f(z=P + 1) == 2 and f(z=P + 2) in (7, 8) and f(dt=0, z=P + 2) == 2 and f(ld=99) == 3
        assert f(p=_targets(sl, ids=None)) == 1 and f(p=_targets(sl, tl=None)) == 1 and f(p=_targets(sl, labels=None)) == 1
        assert f(p=_targets(sl, ids=P + 4)) == 2 and f(p=_targets(sl, labels=P + 4)) == 2
        for top in (0, -1, 257):
            assert f(p=_targets(sl, top=top)) == 5, top
        for V in (0, (1 << 30) + 1):
            assert f(p=_targets(sl, V=V)) == 5, V
        for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-45, 1e-7, 2e6):
            assert f(p=_targets(sl, tau=tau)) == 5, tau
        for hard in (-0.1, 1.1, float("nan")):
            assert f(p=_targets(sl, hard=hard)) == 5, hard
        for ctx in ([5, 0], [-1, 0]):
            assert f(layout=sl.Layout(ctx, 4)) == 5
        assert f(layout=sl.Layout([0] * 65, 4)) == 5 and f(layout=sl.Layout([0], 0)) == 5
    assert fwd(loss=None) == 1 and fwd(stats=None) == 1 and fwd(stats=P + 4) == 2
    assert bwd(stats=None) == 1 and bwd(dz=None) == 1 and bwd(dz=P + 1) == 2 and bwd(ldo=99) == 3 and bwd(g=None) in (7, 8) and bwd(g=P + 4) == 2
    assert step(loss=None) == 1 and step(dz=None) == 1 and step(ldo=99) == 3 and step(g=None) in (7, 8)


def test_binding_refusals(sl):
    """Shapes, types, strides, devices and overlaps that the binding turns away."""
    torch = pytest.importorskip("torch")
    E, lay = sl.SparseLoraError, sl.Layout([0, 0], 4)
    x, ids, w = torch.zeros(8, 16), torch.zeros(8, dtype=torch.int32), torch.ones(16)
    for bad in (dict(ids=ids.long()), dict(ids=ids[:7]), dict(E=x.half()), dict(E=x[:, ::2]), dict(E=x[0]), dict()):   # the last: no GPU
        with pytest.raises(E):
            sl.embed_fwd(**{"E": x, "ids": ids, **bad}, layout=lay)
    with pytest.raises(E):
        sl.embed_bwd(ids, x, lay, 10, grad_dtype=torch.float16)
    with pytest.raises(E):
        sl.embed_bwd(ids, x[:, ::2], lay, 10)
    for bad in (dict(x=x[:7]), dict(w=w[:8]), dict(w=w.bfloat16()), dict(b=w[:8]), dict(residual=x.bfloat16()), dict()):
        with pytest.raises(E):
            sl.layer_norm_fwd(**{"x": x, "w": w, "b": None, **bad}, layout=lay)
    with pytest.raises(E, match="nothing is added"):
        sl.layer_norm_fwd(x, w, None, lay, out=(None, torch.zeros(8, 16)))
    with pytest.raises(E):
        sl.layer_norm_bwd(x, w, torch.zeros(8, 2), lay, x)
    p = sl.DistillTargets(torch.zeros(8, 3, dtype=torch.int32), torch.zeros(8, 3))
    for z in (x[:7], x.half(), x[:, ::2], x[:1].expand(8, 16), x.t(), torch.zeros(8, 2, 8), x):
        with pytest.raises(E):
            sl.distill_fwd(p, z, lay)
    dev = None
    for bad in (sl.DistillTargets(None, None), sl.DistillTargets(p.top_ids, None), sl.DistillTargets(p.top_ids, p.top_logits, hard=0.5),
                sl.DistillTargets(p.top_ids.long(), p.top_logits), sl.DistillTargets(p.top_ids, p.top_logits.bfloat16()),
                sl.DistillTargets(p.top_ids[:7], p.top_logits[:7])):
        with pytest.raises(E):
            bad._c(8, 16, dev)


def test_rows_apart_that_share_memory_are_refused(sl):
    torch = pytest.importorskip("torch")
    buf = torch.zeros(8, 40)
    a, b = buf[:, :16], buf[:, 16:32]            # rows between each other: refused, their spans overlap
    with pytest.raises(sl.SparseLoraError, match="may not share memory"):
        sl.api._refuse_spans(("dlogits", a), (("logits", b),))
    sl.api._refuse_spans(("dlogits", buf[:4, :16]), (("logits", buf[4:, :16]), ("none", None)))
