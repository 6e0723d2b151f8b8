"""q/k/v projections, head norms with the rotation, differential attention and
the o projection run together through the modules, outputs and every gradient
against the oracle on the same channel sets.

Each stage is compared on the values that reached it.  A chain of oracles from
X on would not do: without the norm this layer's scores reach into the tens,
and the projections' own rounding of q and k (half a step, 2^-8) moves a score
s by up to 2^-7 |s| and its weight by the factor e^(2^-7 |s|), 1.27 at |s| = 30."""
import numpy as np
import pytest

import oracle as O
import workloads as W
from tests.gpu_helpers import assert_close, to_np

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _bf(x):
    return W.round_to_bf16(np.asarray(x, dtype=np.float32))


@pytest.mark.parametrize("qk_norm,step", [(True, 0), (True, 5), (False, 5)])
def test_sparse_layer_with_differential_attention(qk_norm, step):
    import contextual_sparsity_lora_svd_amd as sl
    D, hq, hkv, hd, r, L = 128, 4, 2, 32, 8, 48
    heads, ctx = (hq, hkv, hd), [32, 40]
    nq, nkv, T = hq * hd, hkv * hd, 2 * 48
    rng = np.random.default_rng(31)
    Wq, Wk, Wv = (_bf(rng.standard_normal(s) * 0.05) for s in ((nq, D), (nkv, D), (nkv, D)))
    Wo = _bf(rng.standard_normal((D, nq)) * 0.05)
    X = W.make_activations(12, T, D, 16, "bf16")
    dO = _bf(rng.standard_normal((T, D)))
    sched = sl.SparsitySchedule([sl.LayerRatios(qk=50, vo=50)], total_steps=20)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.bfloat16)
    gen = torch.Generator().manual_seed(4)
    proj = sl.SparseLoRAQKVO(dev(Wq), dev(Wk), dev(Wv), dev(Wo), heads, r, est_rank=4, lora_scale=0.5,
                             schedule=sched, generator=gen)
    core = sl.DiffAttention(heads, lambda_init=0.4, rot=sl.Rotary(hd), qk_norm=qk_norm, eps=1e-2, generator=gen)
    lay = sl.Layout(ctx, L)
    seen = {}

    def attention(q, k, v):
        a = core(q, k, v, lay)
        for n, t in (("q", q), ("k", k), ("v", v), ("a", a)):
            t.retain_grad()
            seen[n] = t
        return a

    Xd = dev(X).requires_grad_(True)
    out = proj(Xd, lay, attention if step else core.bind(lay), step=step)
    if not step:                                     # the bound core is the same call
        again = proj(Xd, lay, attention, step=step)
        assert torch.equal(out, again)
        out = again
    out.backward(dev(dO))
    torch.cuda.synchronize()
    iqk, ivo = (t.cpu().numpy() for t in proj.last_idx)
    val = {n: to_np(t) for n, t in seen.items()}
    grad = {n: to_np(t.grad) for n, t in seen.items()}

    # the projections, on the core's output and gradients
    names = ("Aq", "Bq", "Ak", "Bk", "Av", "Bv", "Ao", "Bo")
    p = {"X": X, "Wq": Wq, "Wk": Wk, "Wv": Wv, "Wo": Wo, "a": val["a"]}
    p.update({n: _bf(getattr(proj, n).detach().cpu().numpy()) for n in names})
    ref, cache = O.qkvo_forward(p, ctx, L, list(iqk), list(ivo), heads, 0.5)
    gr = O.qkvo_backward(p, cache, {"dq": grad["q"], "dk": grad["k"], "dv": grad["v"], "d_out": dO}, 0.5)
    for n in "qkv":
        assert_close(val[n], ref[n], "bf16", n)
    assert_close(to_np(out), ref["o"], "bf16", "o")
    assert_close(to_np(Xd.grad), gr["dX"], "bf16", "dX")
    assert_close(grad["a"], gr["da"], "bf16", "da")
    for n in names:
        assert_close(to_np(getattr(proj, n).grad), gr["d" + n], "bf16", "d" + n)

    # the core, on the projections' q, k, v and the gradient that came back.
    # Its rotated rows are rounded once (half a step, 2^-8) before the scores:
    # the oracle takes them rounded too
    pos, (f, amp) = np.arange(T) % L, O.rotary_frequencies(hd)
    lv = [getattr(core, n).detach().cpu().double().numpy() for n in sl.DiffAttnParams.NAMES]
    one = np.ones(hd)
    y = {n: _bf(O.rotate(O.head_norm(val[n], one, hd, 1e-2) if qk_norm else val[n], pos, f, amp, hd, False))
         for n in "qk"}
    g = O.diff_attention(y["q"], y["k"], val["v"], lv, 0.4, 2, heads, hd ** -0.5, True, da=grad["a"])
    assert_close(val["a"], g["a"], "bf16", "a")
    assert_close(grad["v"], g["dv"], "bf16", "dv")
    for n in "qk":
        t = O.rotate(g["d" + n], pos, f, amp, hd, False, inverse=True)
        if qk_norm:
            t, dw, _, _ = O.head_norm_backward(val[n], one, t, hd, 1e-2)
            assert_close(to_np(getattr(core, "w" + n).grad), dw, "bf16", "dw" + n)
        assert_close(grad[n], t, "bf16", "d" + n)
    for n in sl.DiffAttnParams.NAMES:
        assert_close(to_np(getattr(core, n).grad), g["d" + n], "bf16", "d" + n)


def test_module_backward_twice_is_refused_and_padding_has_no_gradient():
    import contextual_sparsity_lora_svd_amd as sl
    heads, lay = (4, 2, 16), sl.Layout([20, 20], 20)
    core = sl.DiffAttention(heads, rot=sl.Rotary(8, interleaved=True), generator=torch.Generator().manual_seed(1))
    x = [torch.randn(40, h * 16, device="cuda", requires_grad=True) for h in (4, 2, 2)]
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    a = core(*x, lay, lens=[20, 7], pos=pos)
    a.sum().backward()
    for t in x:
        assert not t.grad[27:].any() and t.grad[:27].any()
    with pytest.raises(RuntimeError):
        a.sum().backward()


def test_module_holds_no_scratch_between_forward_and_backward():
    """Between the passes: a, q, k, v and what the backward reads, not its scratch
    (here 2.5 times as much); after the backward, or without gradients, nothing but
    the results.  A second backward of a retained graph gives the same."""
    import contextual_sparsity_lora_svd_amd as sl
    heads, L = (16, 4, 64), 2048
    lay = sl.Layout([L], L)
    core = sl.DiffAttention(heads, generator=torch.Generator().manual_seed(1))
    x = [torch.randn(L, h * 64, device="cuda").to(torch.bfloat16).requires_grad_(True) for h in (16, 4, 4)]
    p = core._params(core.lq1, core.lk1, core.lq2, core.lk2)
    buf = sl.DiffAttnWorkspace(p, lay, torch.bfloat16, "cuda")
    saved, ws = buf.saved.numel(), buf.ws.numel()
    assert ws > 2 << 20
    del buf, p
    out_bytes, slack = L * 16 * 64 * 2, 1 << 20
    with torch.no_grad():
        core(*x, lay)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        a = core(*x, lay)
        assert torch.cuda.memory_allocated() - before <= out_bytes + slack
        assert torch.cuda.max_memory_allocated() - before <= out_bytes + saved + slack
        del a
    a = core(*x, lay)
    assert torch.cuda.memory_allocated() - before <= out_bytes + saved + slack
    da = torch.randn_like(a)
    first = torch.autograd.grad(a, x, da, retain_graph=True)
    again = torch.autograd.grad(a, x, da)
    for u, v in zip(first, again):
        assert torch.equal(u, v)
    del first, again, u, v
    held = torch.cuda.memory_allocated() - before - da.numel() * 2
    assert held <= out_bytes + slack, held                  # a itself is still here


def test_module_step_captured_and_replayed():
    """Forward and backward of the module in one graph (no eager result of the same
    leaves alive while it is captured), replayed on inputs that change, with eager
    steps in between."""
    import contextual_sparsity_lora_svd_amd as sl
    heads, lay = (8, 4, 32), sl.Layout([300, 300], 300)
    core = sl.DiffAttention(heads, rot=sl.Rotary(32), qk_norm=True, generator=torch.Generator().manual_seed(1))
    x = [torch.randn(600, h * 32, device="cuda").to(torch.bfloat16).requires_grad_(True) for h in (8, 4, 4)]
    da = torch.randn(600, 256, device="cuda").to(torch.bfloat16)

    def step():
        a = core(*x, lay, lens=[300, 211])
        return [a.detach(), *torch.autograd.grad(a, [*x, *core.parameters()], da)]

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
            x[0].copy_(torch.roll(x[0], 1, 0))
            core.lq1.mul_(0.5 if i % 2 else 2.0)
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        for u, v in zip(got, step()):
            assert torch.equal(u, v)
