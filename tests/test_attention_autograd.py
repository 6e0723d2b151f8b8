"""CPU checks of the autograd steps around the attention operators, with stand-ins
for the kernels."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def core(monkeypatch):
    """DiffAttention whose operators are replaced: (module maker, record of the
    parameters that each call got)."""
    import contextual_sparsity_lora_svd_amd as sl
    from contextual_sparsity_lora_svd_amd import layer
    calls = []

    def norm_bwd(q, k, wq, wk, layout, heads, dq, dk, rot=None, pos=None, eps=0.0):
        return {"dq": 2 * dq, "dk": 2 * dk, "dwq": torch.ones_like(wq), "dwk": torch.ones_like(wk)}

    def attn_fwd(p, q, k, v, layout, lens=None, buf=None, out=None):
        calls.append(("fwd", p))
        return q * 2, buf

    def attn_bwd(p, q, k, v, a, layout, buf, da, out=None):
        calls.append(("bwd", p))
        g = {"dq": 2 * da, "dk": torch.ones_like(k), "dv": torch.ones_like(v)}
        g.update({"d" + n: torch.ones_like(p.t[n]) for n in p.NAMES})
        return g

    monkeypatch.setattr(layer.sl, "rotary", lambda q, k, *a, **kw: (q.clone(), k.clone()))
    monkeypatch.setattr(layer.sl, "head_norm_fwd", lambda q, k, *a, **kw: (2 * q, 2 * k))
    monkeypatch.setattr(layer.sl, "head_norm_bwd", norm_bwd)
    monkeypatch.setattr(layer.sl, "diff_attn_fwd", attn_fwd)
    monkeypatch.setattr(layer.sl, "diff_attn_bwd", attn_bwd)

    def make(qk_norm):
        return sl.DiffAttention((2, 2, 8), rot=sl.Rotary(8, device="cpu"), qk_norm=qk_norm, device="cpu")
    return make, calls, sl.Layout([3], 3)


@pytest.mark.parametrize("step", ["rotary", "norm", "attention"])
def test_a_second_derivative_is_refused(core, step):
    """The steps' gradients come from kernels that autograd cannot look into: asked
    for a second derivative it has to say so, not to take them as constants."""
    from contextual_sparsity_lora_svd_amd import layer
    make, _, lay = core
    m = make(step == "norm")
    x = [torch.randn(3, 16, requires_grad=True) for _ in range(3)]
    if step == "rotary":
        y = sum(t.sum() for t in layer._RotaryStep.apply(x[0], x[1], lay, m.heads, m.rot, None))
    elif step == "norm":
        y = sum(t.sum() for t in layer._HeadNormStep.apply(x[0], x[1], m.wq, m.wk, lay, m.heads, m.rot, None, 1e-6))
    else:
        y = layer._DiffAttnStep.apply(*x, m.lq1, m.lk1, m.lq2, m.lk2, m, lay, None).sum()
    # the gradient depends on x[0] for autograd, through the weight it is multiplied by
    (g,) = torch.autograd.grad((x[0].sum() * y), x[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_the_backward_takes_the_settings_of_its_forward(core):
    """Settings of the module that change between a forward and its backward (a
    schedule, an evaluation in between) are the next forward's."""
    make, calls, lay = core
    m = make(False)
    x = [torch.randn(3, 16, requires_grad=True) for _ in range(3)]
    y = m(*x, lay)
    m.causal, m.scale, m.lambda_init, m.heads = False, 3.0, 0.1, (4, 4, 4)
    y.sum().backward()
    (_, f), (_, b) = calls
    for n in ("causal", "scale", "lambda_init", "heads"):
        assert getattr(f, n) == getattr(b, n), n
    assert (f.causal, f.scale, f.heads) == (True, 8 ** -0.5, (2, 2, 8))
    for n in f.NAMES:
        assert torch.equal(b.t[n], getattr(m, n))
