"""GPU parity of token embedding, row norms and distillation where their kernels change
their way: borders of number ranges, of pieces of work and of memory."""
import numpy as np
import pytest

import oracle as O
from tests.test_gpu_rows import DT, HALF, TINY, U32, _dev, _draw, _ints, _sl, _within
from workloads import round_to_bf16

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---- token embedding -----------------------------------------------------------------
# Sorted tokens are summed in pieces of 64, 512 columns of the joined sums to a block.
PIECES = [  # rows of each id, one id behind the other, and the width
    ([64], 520), ([65], 520), ([128], 4096), ([129], 4096),      # a run that ends at a border and one row behind it
    ([1, 63, 64, 65], 520), ([30, 34, 1], 4096), ([63, 2, 63], 1032),
    ([64 * 64], 1032), ([64 * 65 + 1], 1032),                    # as many pieces as a wave looks at once, and more
    ([5, 64 * 131 + 7, 50], 1544),
]


@pytest.mark.parametrize("dt,gdt", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("counts,D", PIECES, ids=str)
def test_embedding_gradient_of_runs_over_pieces(counts, D, dt, gdt):
    sl = _sl()
    rng, T, V = np.random.default_rng(sum(counts)), sum(counts), len(counts) + 2
    ids = rng.permutation(np.repeat(np.arange(1, len(counts) + 1), counts))
    dY = _draw(rng, (T, D), dt)
    got = sl.embed_bwd(_ints(ids), _dev(dY, dt), sl.Layout([0], T), V, scale=1.5, grad_dtype=DT[gdt])
    ref, mag, n = np.zeros((V, D)), np.zeros((V, D)), np.bincount(ids, minlength=V)
    for v in range(V):
        rows = dY[ids == v].astype(np.float64) * 1.5
        ref[v], mag[v] = rows.sum(0), np.abs(rows).sum(0)
    _within(got, ref, HALF[gdt] * np.abs(ref) + (n[:, None] + 8) * U32 * mag + TINY, "dE")
    assert not got[0].any() and not got[V - 1].any()


@pytest.mark.parametrize("dt,T,D", [("bf16", 16387, 4096), ("f32", 16387, 1000), ("bf16", 8201, 4096), ("bf16", 600001, 64)])
def test_lookup_of_many_rows(dt, T, D):
    """Enough blocks that a thread holds four rows in flight, the last round of rows not full."""
    sl = _sl()
    g, V, s = torch.Generator(device="cuda").manual_seed(T), 777, 1.7
    E = torch.randn(V, D, generator=g, device="cuda").to(DT[dt])
    ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda").int()
    ok = ((ids >= 0) & (ids < V))[:, None]
    for scale in (1.0, s):
        want = torch.where(ok, E[ids.long().clamp(0, V - 1)].float() * torch.tensor(scale, device="cuda"), 0.0).to(DT[dt])
        assert torch.equal(sl.embed_fwd(E, ids, sl.Layout([0], T), scale=scale), want)


# ---- norm of whole rows ------------------------------------------------------------------
# More rows than one round of the forward's blocks (768, 512 of them where a row takes over 512
# lanes), the last round with rows for some of a block's groups only.
WALKS = [  # rows, width
    (1100, 16384),       # two and four vectors a lane
    (1031, 8192),
    (1601, 4104),        # 576 lanes a row in bf16
    (3001, 1032),        # 192 lanes, two rows to a block
    (3101, 1000),        # 128 lanes, four rows to a block
    (7001, 520),
    (25003, 72),         # 16 and 32 lanes of a wave
    (50021, 8),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("T,D", WALKS)
def test_norm_forward_over_several_rounds_of_rows(T, D, centered, dt):
    sl = _sl()
    rng, lay = np.random.default_rng(T), sl.Layout([0], T)
    x, r = _draw(rng, (T, D), dt), _draw(rng, (T, D), dt)
    x += np.arange(T, dtype=np.float32)[:, None] % 5      # rows that tell each other apart
    x = round_to_bf16(x) if dt == "bf16" else x
    w, b = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32), rng.standard_normal(D).astype(np.float32)
    bt, bn = (_dev(b), b) if centered else (None, None)
    xt, rt, wt = _dev(x, dt), _dev(r, dt), _dev(w)
    y, h, stats = sl.layer_norm_fwd(xt, wt, bt, lay, 1e-5, centered, rt)
    hn = (x + r).astype(np.float32)
    hn = round_to_bf16(hn) if dt == "bf16" else hn
    assert np.array_equal(h.float().cpu().numpy(), hn)
    ref, u, s = O.layer_norm(hn, w, bn, 1e-5, centered)
    # a lane's 16 values, 6 steps over a wave, 16 waves, the squares' halved by the root
    own = (np.abs(u) + 1) * np.abs(w) + (0 if bn is None else np.abs(bn))
    _within(y, ref, HALF[dt] * np.abs(ref) + 96 * U32 * own, "y")
    _within(stats[:, 2], s[:, 0], 96 * U32 * s[:, 0], "s")
    for swap in (False, True):                            # in place, over several rounds too
        c = xt.clone(), rt.clone()
        y2, h2, s2 = sl.layer_norm_fwd(c[0], wt, bt, lay, 1e-5, centered, c[1], out=c[::-1] if swap else c)
        assert torch.equal(y2, y) and torch.equal(h2, h) and torch.equal(s2, stats)
    y3, _, s3 = sl.layer_norm_fwd(h, wt, bt, lay, 1e-5, centered)          # no residual
    assert torch.equal(y3, y) and torch.equal(s3, stats)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("centered", [True, False])
@pytest.mark.parametrize("T,D", WALKS)
def test_norm_backward_over_several_rounds_of_rows(T, D, centered, dt):
    sl = _sl()
    rng, lay = np.random.default_rng(T + 1), sl.Layout([0], T)
    h, dy, dh = (_draw(rng, (T, D), dt) for _ in range(3))
    w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32)
    t = {n: _dev(v, dt) for n, v in (("h", h), ("dy", dy), ("dh", dh))}
    _, _, stats = sl.layer_norm_fwd(t["h"], _dev(w), None, lay, 1e-5, centered)
    g = sl.layer_norm_bwd(t["h"], _dev(w), stats, lay, t["dy"], t["dh"], centered)
    dx, dw, db, mx, mw, mb = O.layer_norm_backward(h, w, dy, dh, 1e-5, centered)
    _within(g["dx"], dx, HALF[dt] * np.abs(dx) + 128 * U32 * mx, "dx")
    # rows of a group one after the other, the block's groups, the blocks by 64 and those
    chain = T / 8 + 64 + 16 + 96
    _within(g["dw"], dw, chain * U32 * mw, "dw")
    if centered:
        _within(g["db"], db, chain * U32 * mb, "db")
    again = sl.layer_norm_bwd(t["h"], _dev(w), stats, lay, t["dy"], t["dh"], centered, out={"dx": t["dy"]})
    for n in g:
        assert torch.equal(again[n], g[n]), n


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


@pytest.mark.parametrize("dt,T,V,ctx", [("bf16", 4000, 32000, 0), ("bf16", 4000, 32000, 3000), ("bf16", 2100, 32000, 500),
                                        ("f32", 1000, 32000, 900), ("f32", 1900, 32000, 0)])
def test_large_logits_of_few_rows_with_a_loss(dt, T, V, ctx):
    """What goes past the caches depends on all rows and on those with a loss: bit for bit
    what calls of a hundred rows give, zeros at context rows."""
    sl = _sl()
    g = torch.Generator(device="cuda").manual_seed(3)
    z = (3 * torch.randn(T, V, generator=g, device="cuda")).to(DT[dt])
    tops, labels = (torch.randint(0, V, s, generator=g, device="cuda").int() for s in ((T, 8), (T,)))
    tl, w = torch.randn(T, 8, generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")
    lay, p = sl.Layout([ctx], T), sl.DistillTargets(tops, tl, labels, 1.5, 0.25)
    loss, stats = sl.distill_fwd(p, z, lay)
    dz = sl.distill_bwd(p, z, stats, lay, w)
    l2, d2 = sl.distill_step(p, z, lay, w)
    assert torch.equal(l2, loss) and torch.equal(d2, dz)
    assert not loss[:ctx].any() and not dz[:ctx].any()
    for a in {ctx, ctx + (T - ctx) // 2 // 100 * 100, T - 100}:
        s = slice(a, a + 100)
        q = sl.DistillTargets(tops[s], tl[s], labels[s], 1.5, 0.25)
        l3, s3 = sl.distill_fwd(q, z[s], sl.Layout([0], 100))
        assert torch.equal(l3, loss[s]) and torch.equal(s3, stats[s])
        assert torch.equal(sl.distill_bwd(q, z[s], s3, sl.Layout([0], 100), w[s]), dz[s])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_more_rows_than_blocks(dt):
    """Past 2^20 rows a block takes several, rows with a loss and context rows."""
    sl = _sl()
    T, V, ctx = (1 << 20) + 70003, 5, 40000
    g = torch.Generator(device="cuda").manual_seed(9)
    z = (2 * torch.randn(T, V, generator=g, device="cuda")).to(DT[dt])
    tops, labels = (torch.randint(-1, V, s, generator=g, device="cuda").int() for s in ((T, 2), (T,)))
    tl, w = torch.randn(T, 2, generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")
    lay, p = sl.Layout([ctx], T), sl.DistillTargets(tops, tl, labels, 2.0, 0.5)
    loss, stats = sl.distill_fwd(p, z, lay)
    dz = sl.distill_bwd(p, z, stats, lay, w)
    l2, d2 = sl.distill_step(p, z, lay, w)
    assert torch.equal(l2, loss) and torch.equal(d2, dz) and not loss[:ctx].any() and not dz[:ctx].any()
    # a row's result is its own: the same rows in calls of fewer (V odd: at the same place to a 16-byte border)
    for a in (ctx, ctx + 123456, 1 << 20, T - 5000):
        a -= a % 8
        a = max(a, ctx)
        s = slice(a, min(a + 5000, T))
        n = s.stop - s.start
        q = sl.DistillTargets(tops[s], tl[s], labels[s], 2.0, 0.5)
        l3, d3 = sl.distill_step(q, z[s], sl.Layout([0], n), w[s])
        assert torch.equal(l3, loss[s]) and torch.equal(d3, dz[s]), a
