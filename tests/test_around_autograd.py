"""CPU checks of the autograd steps around the layers, with stand-ins for the kernels."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def mods(monkeypatch):
    import contextual_sparsity_lora_svd_amd as sl
    from contextual_sparsity_lora_svd_amd import layer
    calls = []

    def norm_fwd(x, w, b, layout, eps, centered, r):
        calls.append(("fwd", eps, centered))
        h = x if r is None else x + r
        return 2 * h, h, torch.zeros(len(x), 3)

    def norm_bwd(h, w, stats, layout, dy, dh, centered, bias):
        calls.append(("bwd", dh is None, centered, bias))
        g = {"dx": 2 * dy if dh is None else 2 * dy + dh, "dw": torch.ones_like(w)}
        if bias:
            g["db"] = torch.ones_like(w)
        return g

    def embed_bwd(ids, dY, layout, vocab, scale, dtype):
        assert dY.is_contiguous()
        return torch.ones(vocab, dY.shape[1], dtype=dtype)

    def distill_fwd(p, z, layout):
        return z.float().sum(1), torch.zeros(len(z), 4)

    def distill_bwd(p, z, stats, layout, dloss):
        assert dloss.is_contiguous()
        calls.append(("distill", p.temperature, p.hard))
        return dloss[:, None].expand_as(z).to(z.dtype).contiguous()

    monkeypatch.setattr(layer.sl, "layer_norm_fwd", norm_fwd)
    monkeypatch.setattr(layer.sl, "layer_norm_bwd", norm_bwd)
    monkeypatch.setattr(layer.sl, "embed_fwd", lambda E, ids, layout, scale: E[ids.long()] * scale)
    monkeypatch.setattr(layer.sl, "embed_bwd", embed_bwd)
    monkeypatch.setattr(layer.sl, "distill_fwd", distill_fwd)
    monkeypatch.setattr(layer.sl, "distill_bwd", distill_bwd)
    return sl, calls, sl.Layout([0], 3)


def test_gradients_go_where_they_belong(mods):
    sl, calls, lay = mods
    norm = sl.LayerNorm(16, device="cpu")
    x, r = (torch.randn(3, 16, requires_grad=True) for _ in range(2))
    y, h = norm(x, lay, r)
    (y.sum() + 5 * h.sum()).backward()
    assert torch.equal(x.grad, torch.full_like(x, 7.0)) and torch.equal(r.grad, x.grad)
    assert x.grad.data_ptr() != r.grad.data_ptr()
    assert norm.weight.grad is not None and norm.bias.grad is not None
    x.grad = None
    norm(x, lay, r)[0].sum().backward()                   # h unused: no gradient of its own
    assert calls[-1][1] is True and torch.equal(x.grad, torch.full_like(x, 2.0))
    x.grad = None
    norm(x, lay, r)[1].sum().backward()                   # y unused
    assert calls[-1][1] is False and torch.equal(x.grad, torch.ones_like(x))
    rms = sl.LayerNorm(16, centered=False, device="cpu")
    assert rms.bias is None
    rms(x, lay).sum().backward()
    assert calls[-1] == ("bwd", True, False, False)


def test_the_table_has_its_own_type_of_gradient(mods):
    sl, _, lay = mods
    emb = sl.TokenEmbedding(torch.randn(7, 8).bfloat16(), scale=2.0)
    emb(torch.tensor([1, 2, 1], dtype=torch.int32), lay).sum().backward()
    assert emb.weight.grad.dtype == torch.bfloat16 and emb.weight.grad.shape == (7, 8)


def test_the_backward_takes_the_settings_of_its_forward(mods):
    sl, calls, lay = mods
    crit, z = sl.DistillLoss(2.0, 0.0), torch.randn(3, 9, requires_grad=True)
    loss = crit(z, lay, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))
    crit.temperature, crit.hard = 9.0, 1.0
    loss.mean().backward()                                # dloss arrives expanded from one value
    assert calls[-1] == ("distill", 2.0, 0.0) and torch.allclose(z.grad, torch.full_like(z, 1 / 3))
    norm, x = sl.LayerNorm(16, eps=0.5, device="cpu"), torch.randn(3, 16, requires_grad=True)
    y = norm(x, lay)
    norm.centered = False
    y.sum().backward()
    assert calls[-2] == ("fwd", 0.5, True) and calls[-1][2] is True


@pytest.mark.parametrize("step", ["embed", "norm", "distill"])
def test_a_second_derivative_is_refused(mods, step):
    sl, _, lay = mods
    if step == "embed":
        emb = sl.TokenEmbedding(torch.randn(7, 8))
        x, y = emb.weight, emb(torch.tensor([1, 2, 1], dtype=torch.int32), lay)
    elif step == "norm":
        x = torch.randn(3, 16, requires_grad=True)
        y = sl.LayerNorm(16, device="cpu")(x, lay)
    else:
        x = torch.randn(3, 9, requires_grad=True)
        y = sl.DistillLoss()(x, lay, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2))
    (g,) = torch.autograd.grad(x.sum() * y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_a_gradient_over_saved_logits_is_noticed(mods, monkeypatch):
    """step() may write the gradient over the logits; a backward pass that needs them raises."""
    sl, _, lay = mods
    from contextual_sparsity_lora_svd_amd import layer

    def distill_step(p, z, layout, w, out):
        out.data.fill_(0.5)
        return torch.zeros(len(z)), out

    monkeypatch.setattr(layer.sl, "distill_step", distill_step)
    ids, top = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    x = torch.randn(3, 9, requires_grad=True)
    z = torch.tanh(x)                                     # its backward reads its result
    _, dz = sl.DistillLoss().step(z, lay, ids, top, out=z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward(dz)
    z = 2 * x
    loss = sl.DistillLoss()(z, lay, ids, top)
    _, dz = sl.DistillLoss().step(z, lay, ids, top, out=z)
    z.backward(dz, retain_graph=True)                     # nothing of this product's backward is z
    assert torch.equal(x.grad, torch.ones_like(x))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    with torch.inference_mode():
        z = torch.randn(3, 9)
        assert sl.DistillLoss().step(z, lay, ids, top, out=z)[1] is z
