"""GPU parity of token embedding, row norms and distillation where their kernels change
their way: borders of number ranges, of pieces of work and of memory."""
import numpy as np
import pytest

import oracle as O
from tests.test_gpu_rows import DT, HALF, TINY, U32, _dev, _ints, _sl, _within

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---- distillation ------------------------------------------------------------------
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("tau,hard,border_of", [(1.0, 0.0, 1.0), (1.0, 1.0, 1.0), (2.0, 0.5, 1.0), (0.5, 0.4, 0.5), (1e-6, 0.0, 1e-6)])
def test_maxima_on_both_sides_of_2_to_the_20th(tau, hard, border_of, sign):
    """Exponents of either side of 2^20 are formed in two ways.  Rows whose running maxima
    stand on both: within a thread, between the lanes of a wave and between waves."""
    sl = _sl()
    rng, T, V, K = np.random.default_rng(17), 12, 4096, 6
    tau32, hard32 = float(np.float32(tau)), float(np.float32(hard))
    at = np.float32(2.0 ** 20 * np.log(2.0) * (border_of if border_of == 1.0 else float(np.float32(border_of))))
    step = np.spacing(at)
    k = rng.integers(-40, 11, (T, V))
    vec = np.arange(V) // 4                                # 256 threads, a vector of 4 at a time
    low = np.stack([vec % 2 == 0, vec % 64 < 40, vec % 256 < 128, np.zeros(V, bool)])[np.arange(T) % 4]
    k = np.where(low, np.minimum(k, -4), k)
    z = (sign * np.float64(at) + k * np.float64(step)).astype(np.float32)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    tl, labels = rng.standard_normal((T, K)).astype(np.float32), rng.integers(0, V, T)
    p = sl.DistillTargets(_ints(ids), _dev(tl * np.float32(tau)), _ints(labels), tau, hard)
    lay, zt = sl.Layout([0], T), _dev(z)
    rl, rz, bl, bz = O.distill(z, ids, tl * np.float32(tau), labels, tau32, hard32)
    n = V / 256 + 80                                       # a thread's values, a wave's lanes, the waves, the entries
    loss, stats = sl.distill_fwd(p, zt, lay)
    _within(loss, rl, U32 * (bl(n) + np.abs(rl)), "loss")
    dz = sl.distill_bwd(p, zt, stats, lay)
    _within(dz, rz, HALF["f32"] * np.abs(rz) + U32 * bz(n) + TINY, "dz")
    l2, d2 = sl.distill_step(p, zt, lay)
    assert torch.equal(l2, loss) and torch.equal(d2, dz)


@pytest.mark.parametrize("tau", [2.54, 5.54, 5.69])
def test_the_scale_of_exponents_is_rounded_once(tau):
    """Logits far below the maximum: their exponents y = z log2(e) / tau have the scale's rounding, half a step
    relative to y, and their own, half a step of numbers from 64 on.  (At these temperatures log2(e) times a rounded
    1 / tau is off by 1.7 half steps.)"""
    sl = _sl()
    V, lay, tau32 = 4096, sl.Layout([0], 2), float(np.float32(tau))
    z = -np.random.default_rng(1).uniform(60.0 * tau32, 80.0 * tau32, (2, V)).astype(np.float32)
    z[:, 0] = 0.0
    p = sl.DistillTargets(_ints([[0], [0]]), torch.zeros(2, 1, device="cuda"), None, tau, 0.0)
    below = z[:, 1:].astype(np.float64) / tau32
    want = tau32 * np.exp(below)                           # the sum over the row is 1 to less than half a step
    y = -below / np.log(2.0)
    assert (y > 64).all() and (y < 128).all()
    # the exponential's step and two products behind it
    bound = want * (np.log(2.0) * (y * U32 + 2.0 ** -18) + 4 * U32)
    z_ = _dev(z)
    _, dz = sl.distill_step(p, z_, lay)
    _within(dz[:, 1:], want, bound, "dz")
    _, stats = sl.distill_fwd(p, z_, lay)
    assert torch.equal(sl.distill_bwd(p, z_, stats, lay), dz)


# ---- views that start at no 16-byte border -------------------------------------------
def _apart(t):
    """The same values one element behind a 16-byte border."""
    v = torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    assert v.is_contiguous() and v.data_ptr() % 16 == t.element_size()
    return v


def _row_values(T, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = lambda *s: torch.randint(-1, V, s, generator=g, device="cuda").int()
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return ids, rn


def test_values_of_rows_may_start_anywhere():
    """Ids, labels, entries, positions, weights and statistics as views of longer arrays:
    bit for bit what arrays of their own give."""
    sl = _sl()
    T, V, D, lay = 9, 103, 64, sl.Layout([2], 9)
    ids_, rn = _row_values(T, V)
    ids, tops, labels = ids_(T), ids_(T, 5), ids_(T)
    E, dY, z, tl, w = rn(V, D), rn(T, D), rn(T, V), rn(T, 5), rn(T)
    assert torch.equal(sl.embed_fwd(E, _apart(ids), lay), sl.embed_fwd(E, ids, lay))
    assert torch.equal(sl.embed_bwd(_apart(ids), dY, lay, V), sl.embed_bwd(ids, dY, lay, V))
    nw = torch.ones(D, device="cuda")
    _, h, stats = sl.layer_norm_fwd(dY, nw, None, lay)
    a, b = (sl.layer_norm_bwd(h, nw, s, lay, dY) for s in (stats, _apart(stats)))
    assert all(torch.equal(a[n], b[n]) for n in a)
    p = sl.DistillTargets(tops, tl, labels, 2.0, 0.5)
    q = sl.DistillTargets(_apart(tops), _apart(tl), _apart(labels), 2.0, 0.5)
    for u, v in zip(sl.distill_step(p, z, lay, w), sl.distill_step(q, z, lay, _apart(w))):
        assert torch.equal(u, v)
    (l1, s1), (l2, s2) = sl.distill_fwd(p, z, lay), sl.distill_fwd(q, z, lay)
    assert torch.equal(l1, l2) and torch.equal(s1, s2)
    assert torch.equal(sl.distill_bwd(p, z, s1, lay, w), sl.distill_bwd(q, z, _apart(s2), lay, _apart(w)))
    rot, heads, pos = sl.Rotary(16), (2, 2, 32), ids_(T).abs() * 50
    for u, v in zip(sl.rotary(dY, dY, lay, heads, rot, pos), sl.rotary(dY, dY, lay, heads, rot, _apart(pos))):
        assert torch.equal(u, v)
    hw = torch.ones(32, device="cuda")
    for f in (lambda pos: sl.head_norm_fwd(dY, dY, hw, hw, lay, heads, rot, pos),
              lambda pos: sl.head_norm_bwd(dY, dY, hw, hw, lay, heads, dY, dY, rot, pos).values()):
        for u, v in zip(f(pos), f(_apart(pos))):
            assert torch.equal(u, v)


def test_values_that_start_anywhere_in_a_graph():
    """The copy of such a view is part of the graph: replays see what the view holds then."""
    sl = _sl()
    T, V, D, lay = 33, 103, 64, sl.Layout([0], 33)
    ids_, rn = _row_values(T, V, 1)
    E, dY, z, tl, w, ids, tops = rn(V, D), rn(T, D), rn(T, V), _apart(rn(T, 5)), _apart(rn(T)), _apart(ids_(T)), _apart(ids_(T, 5))

    def call():
        return [sl.embed_fwd(E, ids, lay), sl.embed_bwd(ids, dY, lay, V), *sl.distill_step(sl.DistillTargets(tops, tl), z, lay, w)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        for t in (ids, tops, tl, w):
            t.copy_(torch.roll(t, i + 1, 0))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        for u, v in zip(got, call()):
            assert torch.equal(u, v)


def test_two_losses_in_one_vector():
    """The gradient of the second of two losses in a cat starts where the first one ends."""
    sl = _sl()
    V, crit = 211, sl.DistillLoss(2.0, 0.25)
    ids_, rn = _row_values(13, V, 2)
    z, tops, tl, labels = rn(13, V), ids_(13, 3), rn(13, 3), ids_(13)
    w, got, want = rn(13), [], []
    parts = [(slice(0, 5), sl.Layout([1], 5)), (slice(5, 13), sl.Layout([2], 8))]
    zs = [z[s].clone().requires_grad_(True) for s, _ in parts]
    loss = torch.cat([crit(x, lay, tops[s], tl[s], labels[s]) for x, (s, lay) in zip(zs, parts)])
    got = torch.autograd.grad((loss * w).sum(), zs)
    for x, (s, lay), g in zip(zs, parts, got):
        p = sl.DistillTargets(tops[s].clone(), tl[s].clone(), labels[s].clone(), 2.0, 0.25)
        assert torch.equal(g, sl.distill_step(p, x.detach(), lay, w[s].clone())[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_modules_take_gradients_that_start_anywhere(dt):
    """Rows whose gradient is a part of a larger one, behind an odd number of values."""
    sl = _sl()
    lay, T, D, V = sl.Layout([5], 21), 21, 64, 50
    ids_, rn = _row_values(T, V, 3)
    odd = rn(3).to(DT[dt]).requires_grad_(True)
    emb, norm, ids = sl.TokenEmbedding(rn(V, D).to(DT[dt])), sl.LayerNorm(D), _apart(ids_(T))
    core = sl.DiffAttention((2, 2, 32), rot=sl.Rotary(32), qk_norm=True, generator=torch.Generator().manual_seed(0))

    def grads(join):
        h = emb(ids, lay)
        y, h = norm(h, lay, h)
        a = core(y, h, y, lay)
        ps = [emb.weight, *norm.parameters(), *core.parameters()]
        return torch.autograd.grad(join(a, h), ps)

    weight = rn(2 * T * D).to(DT[dt])
    behind = grads(lambda a, h: (torch.cat([odd, a.reshape(-1), h.reshape(-1)])[3:] * weight).sum())
    alone = grads(lambda a, h: (a.reshape(-1) * weight[:T * D]).sum() + (h.reshape(-1) * weight[T * D:]).sum())
    for u, v in zip(behind, alone):
        assert torch.equal(u, v)
