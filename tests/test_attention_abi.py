"""CPU checks of the entry points around attention: the rotary table against
its formula, size queries, and the refusal of invalid arguments on the host."""
import ctypes
import os

import numpy as np
import pytest

import oracle as O

P = 4096   # any aligned, never-dereferenced address: validation fails first


@pytest.fixture(scope="module")
def sl():
    import contextual_sparsity_lora_svd_amd as m
    if not os.path.exists(m.LIB_PATH):
        from contextual_sparsity_lora_svd_amd import build
        build.build(verbose=False)
    m.lib()
    return m


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("base", 8.0), ("wavelength", 8.0),
                                            ("yarn", 16.0)])
@pytest.mark.parametrize("rot", [2, 40, 128, 256])
def test_rotary_table_is_the_formula(sl, scaling, factor, rot):
    r = sl.Rotary(rot, scaling=scaling, factor=factor, original_len=2048, device="cpu")
    f, amp = O.rotary_frequencies(rot, scaling=scaling, factor=factor, original_len=2048)
    turns = r.turns.numpy().view(np.uint64).astype(np.float64)
    # both sides compute f in at least 53 bits over a handful of operations;
    # an entry is a whole number of 2^-64 turns, so at most one such step off
    # (2 pi 2^-64 = 3.4e-19 radians, whatever the frequency)
    np.testing.assert_allclose(turns * 2 * np.pi / 2.0 ** 64, f, rtol=64 * 2.0 ** -53, atol=2 * np.pi * 2.0 ** -64)
    assert r.amplitude == np.float32(amp)


@pytest.mark.parametrize("bad", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=258), dict(rot_dim=8, base=1.0),
                                 dict(rot_dim=8, base=float("nan")), dict(rot_dim=8, scaling="other"),
                                 dict(rot_dim=8, scaling="linear", factor=0.5),
                                 dict(rot_dim=8, scaling="wavelength", factor=2.0, low_turns=4.0, high_turns=4.0),
                                 dict(rot_dim=8, scaling="yarn", factor=2.0, original_len=0),
                                 dict(rot_dim=8, scaling="yarn", factor=float("inf"))])
def test_rotary_table_refusals(sl, bad):
    with pytest.raises(sl.SparseLoraError):
        sl.Rotary(**bad, device="cpu")


def _rot(sl, rot_dim=8, turns=P, pos=None, amp=1.0):
    return sl.api.SlRotary(rot_dim, 0, amp, turns, pos)


def test_rotary_and_norm_refusals(sl):
    L = sl.lib()
    lay, R = sl.Layout([4, 4], 4), ctypes.byref

    def rot(dt=1, heads=(4, 2, 16), r=None, q=P, k=P, qo=P, ko=P, layout=lay):
        return L.sl_rotary_apply(dt, layout.ref, R(sl.api.SlHeads(*heads)), R(r or _rot(sl)), q, k, qo, ko, 0, None)

    assert rot() in (7, 8)                          # valid: stops at the device check
    assert rot(k=None, ko=None) in (7, 8)
    assert rot(dt=5) == 4
    assert rot(q=None) == 1 and rot(k=None) == 1 and rot(ko=None) == 1
    assert rot(q=P + 2) == 2 and rot(ko=P + 8) == 2
    assert rot(r=_rot(sl, turns=None)) == 1
    assert rot(r=_rot(sl, turns=P + 8)) == 2
    assert rot(r=_rot(sl, rot_dim=7)) == 3 and rot(r=_rot(sl, rot_dim=18)) == 3
    assert rot(r=_rot(sl, rot_dim=0, turns=None)) in (7, 8)
    assert rot(r=_rot(sl, amp=float("nan"))) == 5
    assert rot(heads=(4, 2, 15)) == 3 and rot(heads=(4, 2, 258)) == 3 and rot(heads=(0, 2, 16)) == 3
    assert rot(layout=sl.Layout([1] * 65, 4)) == 5 and rot(layout=sl.Layout([0], 0)) == 5

    def fwd(eps=1e-6, q=P, k=P, wq=P, wk=P, qo=P, ko=P, r=None):
        return L.sl_head_norm_fwd(1, lay.ref, R(sl.api.SlHeads(4, 2, 16)), r, eps, q, k, wq, wk, qo, ko, None)

    assert fwd() in (7, 8) and fwd(r=R(_rot(sl))) in (7, 8) and fwd(k=None, wk=None, ko=None) in (7, 8)
    assert fwd(wq=None) == 1 and fwd(wk=None) == 1 and fwd(ko=None) == 1
    assert fwd(eps=-1.0) == 5 and fwd(eps=float("nan")) == 5
    assert fwd(wq=P + 4) == 2

    h = sl.api.SlHeads(4, 2, 16)
    need = L.sl_head_norm_workspace_bytes(lay.ref, R(h))
    assert need == 8 * 2 * 16 * 4                   # one partial sum per row of eight, q and k
    assert L.sl_head_norm_workspace_bytes(lay.ref, R(sl.api.SlHeads(4, 2, 15))) == 0

    def bwd(k=P, wk=P, dko=P, dk=P, dwk=P, dq=P, ws=P, n=need):
        return L.sl_head_norm_bwd(1, lay.ref, R(h), None, 1e-6, P, k, P, wk, P, dko, dq, dk, P, dwk, ws, n, None)

    assert bwd() in (7, 8)
    assert bwd(k=None, wk=None, dko=None, dk=None, dwk=None) in (7, 8)
    assert bwd(k=None) == 1 and bwd(dwk=None) == 1 and bwd(dq=None) == 1
    assert bwd(n=need - 1) == 6 and bwd(ws=None) == 6 and bwd(dk=P + 1) == 2


def _diff(sl, heads=(4, 2, 16), lam=0.8, scale=0.25, lens=None, lq1=P):
    return sl.api.SlDiffAttn(sl.api.SlHeads(*heads), lam, scale, 1, lens, lq1, P, P, P)


def test_diff_attention_refusals(sl):
    L = sl.lib()
    lay, R = sl.Layout([4, 4], 4), ctypes.byref
    big = 1 << 40

    def fwd(p=None, dt=1, layout=lay, q=P, v=P, a=P, saved=P, ns=big, ws=P, nw=big):
        return L.sl_diff_attn_fwd(dt, layout.ref, R(p or _diff(sl)), q, P, v, a, saved, ns, ws, nw, None)

    assert fwd() in (7, 8) and fwd(dt=0) in (7, 8)
    assert fwd(dt=3) == 4
    assert fwd(q=None) == 1 and fwd(v=None) == 1 and fwd(a=None) == 1 and fwd(_diff(sl, lq1=None)) == 1
    assert fwd(q=P + 2) == 2 and fwd(ws=P + 4) == 2 and fwd(_diff(sl, lq1=P + 4)) == 2
    for heads in ((3, 1, 16), (4, 3, 16), (6, 4, 16), (2, 4, 16), (0, 0, 16), (4, 2, 12), (4, 2, 136), (4, 2, 0)):
        assert fwd(_diff(sl, heads=heads)) == 3, heads
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert fwd(_diff(sl, scale=scale)) == 5
    assert fwd(_diff(sl, lam=float("nan"))) == 5
    for lens in ((5, 1), (-1, 4)):
        assert fwd(_diff(sl, lens=(ctypes.c_int32 * 2)(*lens))) == 5
    assert fwd(_diff(sl, lens=(ctypes.c_int32 * 2)(0, 4))) in (7, 8)
    assert fwd(layout=sl.Layout([1] * 65, 4)) == 5
    # 65536 rows of 32768 values: 2^31 elements
    assert fwd(_diff(sl, heads=(256, 2, 128)), layout=sl.Layout([4096] * 16, 4096)) == 5
    h = sl.api.SlHeads(4, 2, 16)
    ns, nw = (f(1, lay.ref, R(h)) for f in (L.sl_diff_attn_saved_bytes, L.sl_diff_attn_workspace_bytes))
    assert ns >= 8 * 4 * 4 + 8 * 64 * 2 and nw > 0
    assert L.sl_diff_attn_saved_bytes(1, lay.ref, R(sl.api.SlHeads(4, 3, 16))) == 0
    assert fwd(ns=ns, nw=nw) in (7, 8)
    assert fwd(ns=ns - 1) == 6 and fwd(nw=nw - 1) == 6 and fwd(saved=None) == 6 and fwd(ws=None) == 6
    g = sl.api.SlDiffAttnGrads(P, P, P, P)

    def bwd(p=None, da=P, dv=P, g=g, ns=big, nw=big):
        return L.sl_diff_attn_bwd(1, lay.ref, R(p or _diff(sl)), P, P, P, P, P, ns, da, P, P, dv, R(g), P, nw, None)

    assert bwd() in (7, 8)
    assert bwd(da=None) == 1 and bwd(dv=None) == 1 and bwd(g=sl.api.SlDiffAttnGrads(P, P, None, P)) == 1
    assert bwd(dv=P + 2) == 2 and bwd(ns=ns - 1) == 6 and bwd(nw=nw - 1) == 6


def test_binding_refusals(sl):
    """Shapes, types, strides and devices that the binding turns away."""
    torch = pytest.importorskip("torch")
    lay, heads = sl.Layout([4, 4], 4), (4, 2, 16)
    q, k = torch.zeros(8, 64), torch.zeros(8, 32)
    r = sl.Rotary(16, device="cpu")
    E = sl.SparseLoraError
    for bad in (dict(q=q[:7]), dict(q=q[:, :32]), dict(k=k.bfloat16()), dict(q=q.half()),
                dict(q=torch.zeros(64, 8).t()), dict(q=q)):        # the last: not on the GPU
        with pytest.raises(E):
            sl.rotary(**{"q": q, "k": k, **bad}, layout=lay, heads=heads, rot=r)
    w = torch.ones(16)
    with pytest.raises(E):
        sl.head_norm_fwd(q, k, w[:8], w, lay, heads)
    t = {n: w for n in sl.DiffAttnParams.NAMES}
    p = sl.DiffAttnParams(t, heads)
    with pytest.raises(E):
        sl.DiffAttnWorkspace(p, lay, torch.float16, "cpu")
    with pytest.raises(E):
        sl.DiffAttnWorkspace(p, lay, torch.float32, "cpu", lens=[4])
    with pytest.raises(E):
        sl.diff_attn_fwd(p, q, None, None, lay)
    with pytest.raises(E):
        sl.diff_attn_fwd(p, q, k, k, lay)


def test_diff_attention_buffers_of_another_call_are_refused(sl):
    torch = pytest.importorskip("torch")
    heads, t = (4, 2, 16), {n: torch.ones(16) for n in sl.DiffAttnParams.NAMES}
    lay, p = sl.Layout([4, 4], 4), sl.DiffAttnParams(t, heads)
    q, kv = torch.zeros(8, 64), torch.zeros(8, 32)
    like = sl.api._diff_buffers
    buf = sl.DiffAttnWorkspace(p, lay, torch.float32, "cpu", lens=[4, 3])
    assert like(buf, p, lay, q)[1] == buf.saved.numel()
    for other in (sl.DiffAttnWorkspace(p, sl.Layout([8], 8), torch.float32, "cpu", lens=[8]),
                  sl.DiffAttnWorkspace(p, sl.Layout([2] * 4, 2), torch.float32, "cpu"),
                  sl.DiffAttnWorkspace(p, lay, torch.bfloat16, "cpu"),
                  sl.DiffAttnWorkspace(sl.DiffAttnParams(t, (4, 4, 16)), lay, torch.float32, "cpu")):
        with pytest.raises(sl.SparseLoraError, match="buffers made for"):
            like(other, p, lay, q)


def test_diff_attention_forward_without_a_workspace(sl):
    """The forward uses none: it takes NULL with 0 bytes, and buffers made without
    scratch; the backward still needs its own."""
    torch = pytest.importorskip("torch")
    L, lay, R, big = sl.lib(), sl.Layout([4, 4], 4), ctypes.byref, 1 << 40
    assert L.sl_diff_attn_fwd(1, lay.ref, R(_diff(sl)), P, P, P, P, P, big, None, 0, None) in (7, 8)
    g = sl.api.SlDiffAttnGrads(P, P, P, P)
    assert L.sl_diff_attn_bwd(1, lay.ref, R(_diff(sl)), P, P, P, P, P, big, P, P, P, P, R(g), None, 0, None) == 6
    p = sl.DiffAttnParams({n: torch.ones(16) for n in sl.DiffAttnParams.NAMES}, (4, 2, 16))
    q = torch.zeros(8, 64)
    buf = sl.DiffAttnWorkspace(p, lay, torch.float32, "cpu", scratch=False)
    assert sl.api._diff_buffers(buf, p, lay, q)[2:] == (None, 0)
    n = L.sl_diff_attn_workspace_bytes(0, lay.ref, R(sl.api.SlHeads(4, 2, 16)))
    assert buf.ws.numel() == n and buf.ws is buf.ws
    assert sl.api._diff_buffers(buf, p, lay, q)[2:] == (buf.ws.data_ptr(), n)
    assert sl.DiffAttnWorkspace(p, lay, torch.float32, "cpu")._ws.numel() == n


def test_head_norm_workspace_of_calls_without_k(sl):
    """The norms take q alone whatever the kv head count, none included: the size
    query answers for all of them alike."""
    L, lay, R = sl.lib(), sl.Layout([4, 4], 4), ctypes.byref
    need = L.sl_head_norm_workspace_bytes(lay.ref, R(sl.api.SlHeads(4, 2, 16)))
    assert need == L.sl_head_norm_workspace_bytes(lay.ref, R(sl.api.SlHeads(4, 0, 16))) > 0
    assert L.sl_head_norm_workspace_bytes(lay.ref, R(sl.api.SlHeads(4, -1, 16))) == 0
    assert L.sl_head_norm_workspace_bytes(lay.ref, None) == 0
    h = sl.api.SlHeads(4, 0, 16)
    assert L.sl_head_norm_fwd(1, lay.ref, R(h), None, 1e-6, P, None, P, None, P, None, None) in (7, 8)
    bwd = lambda n: L.sl_head_norm_bwd(1, lay.ref, R(h), None, 1e-6, P, None, P, None, P, None, P, None, P, None, P, n,
                                       None)
    assert bwd(need) in (7, 8) and bwd(need - 1) == 6
    assert sl.HeadNormWorkspace(lay, (4, 0, 16), "cpu").ws.numel() == need


def test_outputs_over_other_tensors_are_refused(sl):
    """Outputs that share memory with an input (but where a call works in place),
    with another output or with the buffers."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(64)
    a, b, c, mid = x[:16], x[16:32], x[32:48], x[8:24]
    no = sl.api._refuse_overlap
    no((("a", a), ("b", b)), (("c", c), ("none", None)))
    no((("a", a),), (("q", a), ("k", b)), in_place=(("a", "q"),))
    for outs, ins, same in (((("a", a), ("b", a)), (), ()), ((("a", a), ("b", mid)), (), ()),
                            ((("a", a),), (("q", a),), ()), ((("a", mid),), (("q", a),), (("a", "q"),)),
                            ((("a", a), ("b", b)), (("q", b), ("k", a)), (("a", "q"), ("b", "k")))):
        with pytest.raises(sl.SparseLoraError, match="may not share memory"):
            no(outs, ins, in_place=same)
