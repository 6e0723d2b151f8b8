"""A training step from tokens to a distilled loss through the modules: embedding, norms
with the residual sum and sparse LoRA FFN, an output head and the loss, against the same
step in fp64 with torch's autograd."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class _Model:
    """Two pre-norm FFN layers on a token embedding, tied to the output head."""

    def __init__(self, sl, dt, centered, V=261, D=64, F=160, seed=0):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)
        self.sl, self.dt, self.V, self.D = sl, dt, V, D
        cuda = lambda x: x.to(dt).cuda()
        self.emb = sl.TokenEmbedding(cuda(0.5 * rn(V, D)), scale=2.0)
        self.ffn = [sl.SparseLoRAFFN(cuda(rn(F, D) / 8), cuda(rn(F, D) / 8), cuda(rn(D, F) / 12), 4, lora_scale=0.5,
                                     init_std=0.2, generator=g) for _ in range(2)]
        self.norm = [sl.LayerNorm(D, centered=centered) for _ in range(3)]
        for n in self.norm:
            n.weight.data += 0.2 * rn(D).cuda()
            if n.bias is not None:
                n.bias.data += 0.2 * rn(D).cuda()
        self.crit = sl.DistillLoss(temperature=2.0, hard=0.25)

    def parameters(self):
        return [*self.emb.parameters(), *(p for m in self.ffn + self.norm for p in m.parameters())]

    def logits(self, ids, lay, k):
        h = self.emb(ids, lay)
        y = self.norm[0](h, lay)
        for i, f in enumerate(self.ffn):
            y, h = self.norm[i + 1](f(y, lay, k=k), lay, residual=h)
        return y @ self.emb.weight.t()


def _batch(V, T, K=5, seed=1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, V, (T,), generator=g).int()
    top = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]).int()
    labels = torch.randint(-1, V, (T,), generator=g).int()
    return ids, top, torch.randn(T, K, generator=g), labels


def _reference(m, ids, top, tl, labels, ctx, L, k, weights):
    """The same step in fp64 on the CPU; the channel sets are the modules' own."""
    P = {id(p): p.detach().cpu().double().requires_grad_(True) for p in m.parameters()}
    at = lambda p: P[id(p)]
    T = len(ids)
    row = torch.arange(T)
    context = (row % L) < torch.tensor(ctx)[row // L]
    is_token = ((ids >= 0) & (ids < m.V))[:, None]
    h = torch.where(is_token, at(m.emb.weight)[ids.long().clamp(min=0)] * 2.0, 0.0)

    def norm(n, x):
        d = x - x.mean(-1, keepdim=True) if n.centered else x
        y = d * torch.rsqrt((d * d).mean(-1, keepdim=True) + n.eps) * at(n.weight)
        return y if n.bias is None else y + at(n.bias)

    y = norm(m.norm[0], h)
    for i, f in enumerate(m.ffn):
        Wg, Wu, WdT = (f.frozen[n].cpu().double() for n in ("Wg", "Wu", "WdT"))
        keep = torch.ones(T, f.d_ff, dtype=torch.float64)
        for b, idx in enumerate(f.last_idx.cpu().long()):
            rows = context & (row // L == b)
            on = torch.zeros(f.d_ff, dtype=torch.float64)
            on[idx] = 1.0
            keep[rows] = on
        low = lambda x, A, B: 0.5 * (x @ at(A).t()) @ at(B).t()
        u = torch.nn.functional.silu(y @ Wg.t() + low(y, f.Ag, f.Bg)) * (y @ Wu.t() + low(y, f.Au, f.Bu)) * keep
        h = h + u @ WdT + low(u, f.Ad, f.Bd)
        y = norm(m.norm[i + 1], h)
    z = y @ at(m.emb.weight).t()
    p = torch.softmax(tl.double() / 2.0, 1)
    logq = torch.log_softmax(z / 2.0, 1).gather(1, top.long())
    loss = 0.75 * 4.0 * (p * (p.log() - logq)).sum(1)
    ok = labels >= 0
    ce = -torch.log_softmax(z, 1).gather(1, labels.long().clamp(min=0)[:, None]).squeeze(1)
    loss = torch.where(context, 0.0, loss + 0.25 * torch.where(ok, ce, 0.0))
    (loss * weights.double()).sum().backward()
    return z.detach(), loss.detach(), [P[id(p)].grad for p in m.parameters()]


@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("k", [160, 60])
def test_a_training_step_matches_fp64(centered, k):
    import contextual_sparsity_lora_svd_amd as sl
    ctx, L = [9, 0, 16], 16
    lay, T = sl.Layout(ctx, L), 48
    m = _Model(sl, torch.float32, centered)
    ids, top, tl, labels = _batch(m.V, T)
    weights = torch.linspace(0.2, 1.0, T) / T
    dev = [t.cuda() for t in (ids, top, tl, labels)]
    z = m.logits(dev[0], lay, k)
    loss = m.crit(z, lay, *dev[1:])
    grads = torch.autograd.grad((loss * weights.cuda()).sum(), m.parameters())
    rz, rl, rg = _reference(m, ids, top, tl, labels, ctx, L, k, weights)
    # fp32 throughout, some dozen operations over sums of at most 261 terms each: 1e-5 of the largest value
    close = lambda a, b: float((a.detach().cpu().double() - b).abs().max()) <= 1e-5 * float(b.abs().max())
    assert close(z, rz) and close(loss, rl)
    for p, a, b in zip(m.parameters(), grads, rg):
        assert close(a, b), tuple(p.shape)
    # losses and gradient in one call
    z2 = m.logits(dev[0], lay, k)
    l2, dz = m.crit.step(z2, lay, *dev[1:], weights=weights.cuda())
    assert torch.equal(l2, loss)
    for a, b in zip(torch.autograd.grad(z2, m.parameters(), dz), grads):
        assert float((a - b).abs().max()) <= 2.0 ** -20 * float(b.abs().max())


def test_a_training_step_captured_and_replayed():
    """Forward and backward through every module in one graph, on inputs that change,
    with eager steps in between."""
    import contextual_sparsity_lora_svd_amd as sl
    lay, T = sl.Layout([100, 37], 150), 300
    m = _Model(sl, torch.bfloat16, True)
    ids, top, tl, labels = (t.cuda() for t in _batch(m.V, T))

    def step():
        z = m.logits(ids, lay, 160)
        loss = m.crit(z, lay, top, tl, labels)
        return [loss.detach(), *torch.autograd.grad(loss.sum(), m.parameters())]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        with torch.no_grad():
            ids.copy_(torch.roll(ids, 7))
            tl.mul_(-1.0)
            m.emb.weight.mul_(0.5 if i % 2 else 2.0)
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        for u, v in zip(got, step()):
            assert torch.equal(u, v)


def test_modules_hold_little_between_the_passes():
    """Between forward and backward a norm holds its input and three numbers a row."""
    import contextual_sparsity_lora_svd_amd as sl
    T, D, lay = 2048, 1024, sl.Layout([0], 2048)
    norm, x = sl.LayerNorm(D), torch.randn(T, D, device="cuda").bfloat16().requires_grad_(True)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = norm(x, lay)
    assert torch.cuda.memory_allocated() - before <= T * D * 2 + T * 12 + 4096
    first = torch.autograd.grad(y.sum(), [x, *norm.parameters()], retain_graph=True)
    for u, v in zip(first, torch.autograd.grad(y.sum(), [x, *norm.parameters()])):
        assert torch.equal(u, v)
