"""CPU checks of what the modules and the binding hand to the library where their inputs
are views that start at no 16-byte border; stand-ins for the kernels ask for one."""
import pytest

torch = pytest.importorskip("torch")


def _start(t):
    return t.data_ptr() % 16


@pytest.fixture
def mods(monkeypatch):
    import contextual_sparsity_lora_svd_amd as sl
    from contextual_sparsity_lora_svd_amd import layer
    seen = []

    def rows(*ts):
        for t in ts:
            if t is not None:
                assert t.is_contiguous() and _start(t) == 0
                seen.append(t)

    def norm_fwd(x, w, b, layout, eps, centered, r):
        rows(x, r)
        h = x.clone() if r is None else x + r
        return 2 * h, h, torch.zeros(len(x), 3)

    def norm_bwd(h, w, stats, layout, dy, dh, centered, bias):
        rows(h, dy, dh)
        g = {"dx": dy if dh is None else dy + dh, "dw": torch.ones_like(w)}
        return {**g, "db": torch.ones_like(w)} if bias else g

    def embed_bwd(ids, dY, layout, vocab, scale, dtype):
        rows(dY)
        return torch.zeros(vocab, dY.shape[1], dtype=dtype)

    def pair(q, k, *_, **__):
        rows(q, k)
        return 1 * q, 1 * k

    def attn_fwd(p, q, k, v, layout, buf=None):
        rows(q, k, v)
        return q[:, :q.shape[1]] * 1, buf

    def attn_bwd(p, q, k, v, a, layout, buf, da):
        rows(q, k, v, da)
        return {"dq": 1 * q, "dk": 1 * k, "dv": 1 * v, **{"d" + n: torch.zeros(4) for n in sl.DiffAttnParams.NAMES}}

    class Buf:
        def __init__(self, *a, **k):
            self.saved = torch.zeros(1)

    for n, f in (("layer_norm_fwd", norm_fwd), ("layer_norm_bwd", norm_bwd), ("embed_bwd", embed_bwd), ("rotary", pair),
                 ("embed_fwd", lambda E, ids, layout, scale: E[ids.long()] * scale), ("diff_attn_fwd", attn_fwd),
                 ("diff_attn_bwd", attn_bwd), ("DiffAttnWorkspace", Buf)):
        monkeypatch.setattr(layer.sl, n, f)
    return sl, layer, seen


def _beside(odd, *ys):
    """The sum of a cat of an odd vector and of rows: the rows' gradients are views behind it."""
    return torch.cat([odd, *(y.reshape(-1) for y in ys)]).pow(2).sum()


def test_gradients_that_are_parts_of_a_larger_one(mods):
    sl, layer, seen = mods
    lay, odd = sl.Layout([0], 3), torch.ones(5, requires_grad=True)
    g = torch.ones(11)[5:]
    assert g.is_contiguous() and _start(g) == 4                        # what a cat's part is
    x, r = (torch.randn(3, 16, requires_grad=True) for _ in range(2))
    norm = sl.LayerNorm(16, device="cpu")
    _beside(odd, *norm(x, lay, r)).backward()
    assert torch.isfinite(x.grad).all() and len(seen) == 5
    emb = sl.TokenEmbedding(torch.randn(7, 8))
    _beside(odd, emb(torch.tensor([1, 2, 1], dtype=torch.int32), lay)).backward()
    assert len(seen) == 6
    q, k, v = (torch.randn(3, 8, requires_grad=True) for _ in range(3))
    _beside(odd, *layer._RotaryStep.apply(q, k, lay, (2, 2, 4), None, None)).backward()
    assert len(seen) == 10
    core = sl.DiffAttention((2, 2, 4), device="cpu")
    _beside(odd, core(q, k, v, lay)).backward()
    assert len(seen) == 17
    assert len({t.data_ptr() for t in seen}) > 1


def test_inputs_that_are_parts_of_a_larger_one(mods):
    sl, _, seen = mods
    flat = torch.randn(3 + 48)
    x = flat[3:].view(3, 16)
    assert x.is_contiguous() and _start(x) == 12
    sl.LayerNorm(16, device="cpu")(x, sl.Layout([0], 3))
    assert torch.equal(seen[0], x)


def test_projections_take_gradients_that_are_parts_of_a_larger_one(monkeypatch):
    import contextual_sparsity_lora_svd_amd as sl
    from contextual_sparsity_lora_svd_amd import layer
    from types import SimpleNamespace as NS
    monkeypatch.setattr(layer.sl, "FFNWeights", lambda t, s: NS(t=t))
    monkeypatch.setattr(layer.sl, "FFNWorkspace", lambda *a: None)
    monkeypatch.setattr(layer.sl, "ffn_fwd", lambda w, X, layout, k, idx, buf: (2 * X, buf))

    def ffn_bwd(w, X, layout, k, idx, buf, dY):
        assert _start(dY) == 0 and dY.is_contiguous()
        return {"dX": 2 * dY, **{"d" + n: torch.zeros(4) for n in ("Ag", "Bg", "Au", "Bu", "Ad", "Bd")}}

    monkeypatch.setattr(layer.sl, "ffn_bwd", ffn_bwd)
    X, lora = torch.randn(3, 16, requires_grad=True), [torch.zeros(4) for _ in range(6)]
    Y = layer._FFNStep.apply(X, *lora, NS(dtype=torch.float32, frozen={}, lora_scale=1.0), None, 4, None)
    _beside(torch.ones(5, requires_grad=True), Y).backward()
    assert X.grad is not None

    def qkvo_bwd(w, Xc, ac, layout, k_qk, iqk, k_vo, ivo, buf, **g):
        assert all(_start(t) == 0 and t.is_contiguous() for t in g.values())
        return {n: torch.zeros(3, 16) for n in ("dX", "da")} | {"d" + m + n: torch.zeros(4) for m in "AB" for n in "qkvo"}

    monkeypatch.setattr(layer.sl, "qkvo_fwd", lambda w, X, a, *_: ({"q": 1 * X, "k": 2 * X, "v": 3 * X} if a is None else {"o": 1 * a}, None))
    monkeypatch.setattr(layer.sl, "qkvo_bwd", qkvo_bwd)
    st = layer._QKVOState(NS(heads=(2, 2, 8)), None, 16, None, 16, None, None)
    q, k, v = layer._QKVStep.apply(X, *lora, st)
    o = layer._OStep.apply(q, lora[0], lora[1], st)
    _beside(torch.ones(5, requires_grad=True), o, k, v).backward()


def test_values_read_one_at_a_time_may_start_anywhere(monkeypatch):
    import contextual_sparsity_lora_svd_amd as sl
    from contextual_sparsity_lora_svd_amd import api
    monkeypatch.setattr(api, "_check_rows", lambda name, t, shape, dtype, dev=None: t.data_ptr())
    ids = torch.arange(9, dtype=torch.int32)
    assert _start(ids) == 0
    p, held = api._check_values("ids", ids[:8], (8,), torch.int32)
    assert p == ids.data_ptr() and held.data_ptr() == p                # in place where it can be
    p, held = api._check_values("ids", ids[1:], (8,), torch.int32)
    assert p % 16 == 0 and held.data_ptr() == p and torch.equal(held, ids[1:])
    tops, logits = torch.arange(30, dtype=torch.int32).view(10, 3)[1:9], torch.randn(10, 3)[1:9]
    c = sl.DistillTargets(tops, logits, ids[1:], 2.0, 0.5)._c(8, 100, None)
    assert c.top_ids % 16 == c.top_logits % 16 == c.labels % 16 == 0
    assert [t.data_ptr() for t in c.held] == [c.top_ids, c.top_logits, c.labels]
    assert all(torch.equal(a, b) for a, b in zip(c.held, (tops, logits, ids[1:])))
    rot = sl.Rotary(8, device="cpu")
    c = rot._c(ids[1:], 8, None)
    assert c.pos % 16 == 0 and torch.equal(c.held, ids[1:])
    assert rot._c(None, 8, None).pos is None
