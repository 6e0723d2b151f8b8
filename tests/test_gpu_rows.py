"""GPU parity of token embedding, row norms and distillation with the fp64 oracle:
element by element, within bounds derived from the number formats (half a step of
the output's type, fp32 sums at the length of their longest run of additions)."""
import numpy as np
import pytest

import oracle as O
from workloads import round_to_bf16

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}          # half a step, relative
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -125                                     # results below the normal numbers may be 0


def _sl():
    import contextual_sparsity_lora_svd_amd as sl
    return sl


def _draw(rng, shape, dt, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return round_to_bf16(x) if dt == "bf16" else x


def _dev(x, dt="f32"):
    return torch.from_numpy(np.array(x, dtype=np.float32)).cuda().to(DT[dt])


def _ints(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def _np(t):
    return t.detach().cpu().double().numpy()


def _within(got, ref, bound, what):
    got = _np(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    assert over.max() <= 0, (f"{what}: off by {np.abs(got - ref).ravel()[over.argmax()]:.3e}, "
                             f"bound {np.broadcast_to(bound, over.shape).ravel()[over.argmax()]:.3e}")


# ---- token embedding -----------------------------------------------------------
EMBED = [  # batch, seq, vocab, width, kind of tokens
    (1, 1, 1, 8, "any"),
    (1, 1, 7, 64, "absent"),
    (3, 5, 11, 24, "any"),
    (2, 64, 1000, 520, "any"),
    (1, 33, 40, 4096, "one"),            # one id: its run crosses every border of the pieces
    (1, 32, 5, 520, "one"),              # a run that ends at a border
    (1, 2048, 33, 16, "any"),
    (1, 2049, 100, 64, "any"),           # two sorted chunks, the second of one token
    (4, 1500, 17, 136, "few"),           # long runs in several chunks
    (1, 9000, 3000, 40, "any"),          # pieces of the longer kind
    (1, 8192, 2, 8, "sorted"),
    (3, 11000, 50, 8, "falling"),        # more chunks than one merge takes
    (2, 40000, 70001, 8, "any"),
]


def _tokens(rng, T, V, kind):
    if kind == "one":
        return np.full(T, V // 2)
    ids = rng.integers(-1, V + 1, T) if kind == "any" else rng.integers(0, min(V, 3), T)
    if kind == "absent":
        ids = rng.choice([-1, -2 ** 31, V, 2 ** 31 - 1], T)
    if kind == "sorted":
        ids = np.sort(ids)
    if kind == "falling":
        ids = np.arange(T)[::-1] % V
    return ids


@pytest.mark.parametrize("dt,gdt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("case", EMBED, ids=lambda c: "x".join(map(str, c)))
def test_embedding(case, dt, gdt):
    sl = _sl()
    B, L, V, D, kind = case
    rng, T = np.random.default_rng(L + V), B * L
    lay = sl.Layout([0] * B, L)
    E, dY, ids = _draw(rng, (V, D), dt), _draw(rng, (T, D), dt), _tokens(rng, T, V, kind)
    dE_, dY_, ids_ = _dev(E, dt), _dev(dY, dt), _ints(ids)
    # the lookup alone is exact, a product with the scale rounded in fp32 and then to the type
    assert np.array_equal(_np(sl.embed_fwd(dE_, ids_, lay)), O.embed(E, ids))
    s = float(np.float32(D ** 0.5))
    ref = O.embed(E, ids, s)
    _within(sl.embed_fwd(dE_, ids_, lay, scale=s), ref, (HALF[dt] + U32) * np.abs(ref) + TINY, "Y")
    ref, mag, n = O.embed_backward(ids, dY, V, s)
    got = sl.embed_bwd(ids_, dY_, lay, V, scale=s, grad_dtype=DT[gdt])
    # a run's rows one after the other, and the pieces' sums: fewer than its rows and 8 additions
    _within(got, ref, HALF[gdt] * np.abs(ref) + (n[:, None] + 8) * U32 * mag + TINY, "dE")
    assert not _np(got)[n == 0].any()


def test_embedding_ignores_rows_without_a_token():
    sl = _sl()
    lay, ids = sl.Layout([0], 6), _ints([2, -1, 0, 9, 2, -7])
    dY = torch.ones(6, 8, device="cuda")
    dY[[1, 3, 5]] = float("nan")
    dE = sl.embed_bwd(ids, dY, lay, 4)
    assert torch.equal(dE.cpu(), torch.tensor([1.0, 0, 2, 0])[:, None].expand(4, 8))
    E = torch.full((4, 8), float("inf"), device="cuda")
    E[2] = 3.0
    assert not sl.embed_fwd(E, ids, lay)[[1, 3, 5]].any()


def test_embedding_gradient_is_the_same_every_time():
    """Bit for bit, whatever the workspace and the output held, and whatever the order
    in which blocks run."""
    sl = _sl()
    rng, lay, V, D = np.random.default_rng(5), sl.Layout([0], 20000), 300, 264
    ids, dY = _ints((rng.random(20000) ** 4 * V).astype(int)), _dev(_draw(rng, (20000, D), "f32"))
    first = sl.embed_bwd(ids, dY, lay, V)
    for fill in (0, 255, 127):
        buf = sl.EmbedWorkspace(lay, D, "cuda")
        buf.ws.fill_(fill)
        out = torch.full((V, D), float("nan"), device="cuda")
        assert torch.equal(sl.embed_bwd(ids, dY, lay, V, buf=buf, out=out), first)


def test_embedding_of_large_gradients():
    """Past 64 MiB of rows: against sums in 64 bits, of exact terms."""
    sl = _sl()
    T, D, V, lay = 9000, 4096, 700, sl.Layout([0], 9000)
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = (torch.rand(T, generator=g, device="cuda") ** 6 * V).int()
    dY = torch.randint(-8, 9, (T, D), generator=g, device="cuda").bfloat16()
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dY.double())
    assert torch.equal(sl.embed_bwd(ids, dY, lay, V).double(), want)            # whole numbers below 2^24
    assert torch.equal(sl.embed_bwd(ids, dY.float(), lay, V).double(), want)


def test_embedding_offsets_past_32_bits():
    """A table of more than 2^31 elements: its last rows."""
    sl = _sl()
    V, D, lay = (1 << 31) // 4096 + 9, 4096, sl.Layout([0], 5)
    E = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    E[-3:] = torch.arange(3, device="cuda", dtype=torch.bfloat16)[:, None] + 1
    ids = _ints([V - 1, V - 3, V, V - 2, V - 1])
    assert sl.embed_fwd(E, ids, lay)[:, ::4095].tolist() == [[3, 3], [1, 1], [0, 0], [2, 2], [3, 3]]
    dY = torch.ones(5, D, dtype=torch.bfloat16, device="cuda")
    dE = sl.embed_bwd(ids, dY, lay, V, grad_dtype=torch.bfloat16, out=E.fill_(7.0))
    assert dE[-3:, ::4095].tolist() == [[1, 1], [1, 1], [2, 2]]
    assert not dE[:-3].any()


# ---- norm of whole rows ----------------------------------------------------------
NORM = [  # batch, seq, width
    (1, 1, 8), (3, 5, 24), (1, 7, 64), (2, 9, 136), (1, 33, 512), (1, 5, 520), (2, 17, 1000), (1, 9, 1032),
    (1, 2, 2048), (2, 3, 4096), (1, 5, 5120), (1, 3, 8200), (1, 3, 16384), (1, 2100, 72), (1, 1300, 640), (5, 300, 2056),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", NORM, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("centered", [True, False])
def test_layer_norm(case, dt, centered):
    sl = _sl()
    B, L, D = case
    rng, T, lay = np.random.default_rng(D), B * L, sl.Layout([0] * B, L)
    x = _draw(rng, (T, D), dt) * 1.0 + np.float32(0.5)
    x = round_to_bf16(x) if dt == "bf16" else x
    r, dy, dh = (_draw(rng, (T, D), dt) for _ in range(3))
    w, b = (1 + 0.3 * rng.standard_normal(D)).astype(np.float32), rng.standard_normal(D).astype(np.float32)
    t = {"x": _dev(x, dt), "r": _dev(r, dt), "dy": _dev(dy, dt), "dh": _dev(dh, dt), "w": _dev(w), "b": _dev(b)}
    for add, bias in ((True, centered), (False, False)):
        bt, bn = (t["b"], b) if bias else (None, None)
        y, h, stats = sl.layer_norm_fwd(t["x"], t["w"], bt, lay, 1e-5, centered, t["r"] if add else None)
        hn = x
        if add:
            hn = (x + r).astype(np.float32)
            hn = round_to_bf16(hn) if dt == "bf16" else hn
            assert np.array_equal(_np(h), hn.astype(np.float64))
        else:
            assert h is t["x"]
        ref, u, s = O.layer_norm(hn, w, bn, 1e-5, centered)
        # a row's sums: 16 values of a lane, 6 steps over a wave, 16 waves, and the squares' halved by
        # the root; u is off by that relative to itself and, through the mean, to the row's size
        own = (np.abs(u) + 1) * np.abs(w) + (0 if bn is None else np.abs(bn))
        _within(y, ref, HALF[dt] * np.abs(ref) + 96 * U32 * own, "y")
        g = sl.layer_norm_bwd(h, t["w"], stats, lay, t["dy"], t["dh"] if add else None, centered, bias)
        dx, dw, db, mx, mw, mb = O.layer_norm_backward(hn, w, dy, dh if add else None, 1e-5, centered)
        _within(g["dx"], dx, HALF[dt] * np.abs(dx) + 128 * U32 * mx, "dx")
        # rows of a group one after the other, the block's groups, the blocks by 64 and those
        chain = T / 8 + 64 + 16 + 96
        _within(g["dw"], dw, chain * U32 * mw, "dw")
        if bias:
            _within(g["db"], db, chain * U32 * mb, "db")
        else:
            assert "db" not in g


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_layer_norm_in_place(dt):
    sl = _sl()
    rng, lay, D = np.random.default_rng(3), sl.Layout([0] * 3, 40), 1032
    x, r, dy, dh = (_dev(_draw(rng, (120, D), dt), dt) for _ in range(4))
    w, b = _dev(rng.standard_normal(D)), _dev(rng.standard_normal(D))
    y, h, stats = sl.layer_norm_fwd(x, w, b, lay, residual=r)
    for swap in (False, True):
        c = x.clone(), r.clone()
        out = (c[1], c[0]) if swap else c
        y2, h2, s2 = sl.layer_norm_fwd(*c[:1], w, b, lay, residual=c[1], out=out)
        assert torch.equal(y2, y) and torch.equal(h2, h) and torch.equal(s2, stats) and h2 is out[1]
    g = sl.layer_norm_bwd(h, w, stats, lay, dy, dh)
    for n in range(3):
        c = [h.clone(), dy.clone(), dh.clone()]
        got = sl.layer_norm_bwd(c[0], w, stats, lay, c[1], c[2], out={"dx": c[n]})
        for k in g:
            assert torch.equal(got[k], g[k]), (n, k)
    c = x.clone()                                         # without a residual: where no backward follows
    y2, h2, s2 = sl.layer_norm_fwd(c, w, b, lay, want_stats=False, out=(c, None))
    assert y2 is c and h2 is c and s2 is None and torch.equal(c, sl.layer_norm_fwd(x, w, b, lay)[0])
    E = sl.SparseLoraError
    with pytest.raises(E, match="may not share"):
        sl.layer_norm_fwd(x, w, b, lay, out=(x, None))
    with pytest.raises(E, match="may not share"):
        sl.layer_norm_fwd(x, w, b, lay, residual=r, out=(x, x))
    with pytest.raises(E, match="may not share"):
        sl.layer_norm_bwd(h, w, stats, lay, dy, dh, out={"dx": dy, "dw": w})


def test_layer_norm_rows_far_from_zero():
    """A spread of 1 at an offset of 1e4: the rounding of the mean (up to 5e-4) is
    taken out, where it would be an error of that size in every value."""
    sl = _sl()
    rng, lay, D = np.random.default_rng(4), sl.Layout([0], 6), 4096
    h = (rng.standard_normal((6, D)) + 1e4).astype(np.float32)
    w, dy = np.ones(D, np.float32), _draw(rng, (6, D), "f32")
    y, _, stats = sl.layer_norm_fwd(_dev(h), _dev(w), None, lay)
    ref, u, _ = O.layer_norm(h, w)
    _within(y, ref, 96 * U32 * (np.abs(u) + 1), "y")
    g = sl.layer_norm_bwd(_dev(h), _dev(w), stats, lay, _dev(dy), bias=False)
    dx, dw, _, mx, mw, _ = O.layer_norm_backward(h, w, dy)
    _within(g["dx"], dx, 128 * U32 * mx, "dx")
    _within(g["dw"], dw, 200 * U32 * mw, "dw")


def test_layer_norm_of_constant_rows_and_of_rows_that_are_not_finite():
    sl = _sl()
    lay = sl.Layout([0], 5)
    x = torch.zeros(5, 72, device="cuda")
    x[1] = 1234.5678
    x[2, 3], x[3, 3], x[4, 3] = float("nan"), float("inf"), float("-inf")
    w, b = torch.full((72,), 2.0, device="cuda"), torch.full((72,), 0.5, device="cuda")
    y, _, stats = sl.layer_norm_fwd(x, w, b, lay, eps=0.25)
    assert torch.equal(y[:2], torch.full_like(y[:2], 0.5)) and y[2:].isnan().all()
    y, _, _ = sl.layer_norm_fwd(x, w, None, lay, eps=0.25, centered=False)
    assert not y[0].any() and y[2].isnan().all()
    dy = torch.zeros_like(x)
    dy[0] = torch.arange(72.0, device="cuda")
    g = sl.layer_norm_bwd(x[:1], w, stats[:1], sl.Layout([0], 1), dy[:1])
    # the gradient of a constant row is g = dy w less its mean 71, times 1 / sqrt(eps) = 2; the mean is a
    # product with 1/72, which is no fp32 number: two roundings of 71, and one each of the difference and
    # of the product with 2
    want = (np.arange(72) - 35.5) * 4.0
    _within(g["dx"][0], want, U32 * (2 * 2 * 71 + 2 * np.abs(want)), "dx")
    assert not g["dw"].any() and torch.equal(g["db"], dy[0])
    assert sl.layer_norm_fwd(x, w, None, lay, eps=0.0)[0][0].isnan().all()


def test_layer_norm_gradient_against_differences():
    """The loss sum(y c) along a direction, in fp64 from the oracle's forward."""
    sl = _sl()
    rng, lay, D = np.random.default_rng(8), sl.Layout([0], 4), 264
    h, w, c, e = rng.standard_normal((4, D)), rng.standard_normal(D), rng.standard_normal((4, D)), rng.standard_normal((4, D))
    h, w, c = (v.astype(np.float32) for v in (h, w, c))
    for centered in (True, False):
        _, _, stats = sl.layer_norm_fwd(_dev(h), _dev(w), None, lay, centered=centered)
        g = sl.layer_norm_bwd(_dev(h), _dev(w), stats, lay, _dev(c), centered=centered, bias=False)
        f = lambda s: (O.layer_norm(h + s * e, w, None, 1e-5, centered)[0] * c).sum()
        d = 1e-4
        want = (f(d) - f(-d)) / (2 * d)
        size = np.abs(_np(g["dx"]) * e).sum()
        assert abs((_np(g["dx"]) * e).sum() - want) <= 1e-5 * size + 1e-6 * abs(want)


# ---- distillation ------------------------------------------------------------------
DISTILL = [  # batch, seq, ctx, vocab, top
    (1, 1, [0], 1, 1),
    (1, 3, [0], 7, 7),
    (2, 4, [1, 4], 8, 3),
    (3, 5, [0, 5, 2], 1003, 20),
    (1, 6, [2], 4096, 64),
    (2, 3, [0, 1], 16385, 256),
    (1, 4, [0], 32000, 64),
    (1, 3, [1], 50021, 5),
    (1, 2, [0], 128256, 128),
    (3, 2, [0, 1, 0], 300, 256),         # more entries than threads
    (2, 40, [3, 0], 513, 65),
]


def _distill_case(rng, case, dt, spread=3.0):
    B, L, ctx, V, K = case
    T = B * L
    z = _draw(rng, (T, V), dt, spread)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    if T > 1:
        ids[-1, K // 2:] = -1                                  # fewer entries
        ids[0, -1] = ids[0, 0]                                 # the same id twice
    if T > 3:
        ids[-3] = V                                            # none at all
    tl = (2 * rng.standard_normal((T, K))).astype(np.float32)
    if K > 2:
        tl[0, 1] = -np.inf
    labels = rng.integers(-1, V, T)
    labels[0] = ids[0, 0]
    rows = (np.arange(L)[None, :] >= np.array(ctx)[:, None]).reshape(-1)
    g = rng.standard_normal(T).astype(np.float32)
    return z, ids, tl, labels, rows, g


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", DISTILL, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
@pytest.mark.parametrize("tau,hard", [(1.0, 0.0), (2.0, 0.0), (0.5, 0.4), (1.0, 0.3), (1.0, 1.0)])
def test_distillation(case, dt, tau, hard):
    sl = _sl()
    B, L, ctx, V, K = case
    rng = np.random.default_rng(V + K)
    z, ids, tl, labels, rows, g = _distill_case(rng, case, dt)
    lay = sl.Layout(ctx, L)
    p = sl.DistillTargets(_ints(ids), _dev(tl), _ints(labels), tau, hard)
    zt, gt = _dev(z, dt), _dev(g)
    tau32, hard32 = float(np.float32(tau)), float(np.float32(hard))
    rl, rz, bl, bz = O.distill(z, ids, tl, labels, tau32, hard32, rows, g)
    n = V / 512 + 80                        # a thread's values, a wave's lanes, 8 waves; the K entries of a lane
    loss, stats = sl.distill_fwd(p, zt, lay)
    _within(loss, rl, U32 * (bl(n) + np.abs(rl)), "loss")
    dz = sl.distill_bwd(p, zt, stats, lay, gt)
    _within(dz, rz, HALF[dt] * np.abs(rz) + U32 * bz(n) + TINY, "dz")
    assert not dz[_ints(np.nonzero(~rows)[0]).long()].any()
    l2, dz2 = sl.distill_step(p, zt, lay, gt)
    assert torch.equal(l2, loss) and torch.equal(dz2, dz)
    one = sl.distill_step(p, zt, lay)[1]    # no weights: ones
    assert torch.equal(one, sl.distill_bwd(p, zt, stats, lay)) and torch.equal(one, sl.distill_bwd(p, zt, stats, lay, torch.ones_like(gt)))
    # in place, and rows that stand apart: what is behind them stays
    c = zt.clone()
    assert sl.distill_bwd(p, c, stats, lay, gt, out=c) is c and torch.equal(c, dz)
    c = zt.clone()
    l3, _ = sl.distill_step(p, c, lay, gt, out=c)
    assert torch.equal(c, dz) and torch.equal(l3, loss)
    # (a row's vectors start at its first 16-byte border, so rows elsewhere are summed in another
    # order: the bounds above hold for every order of additions of that length)
    for pad in (1, 13, 16):
        wide, out = (torch.full((B * L, V + pad), float("nan"), dtype=DT[dt], device="cuda") for _ in range(2))
        wide[:, :V] = zt
        l4, s4 = sl.distill_fwd(p, wide[:, :V], lay)
        _within(l4, rl, U32 * (bl(n) + np.abs(rl)), "loss of rows apart")
        sl.distill_bwd(p, wide[:, :V], s4, lay, gt, out=out[:, :V])
        _within(out[:, :V], rz, HALF[dt] * np.abs(rz) + U32 * bz(n) + TINY, "dz of rows apart")
        assert out[:, V:].isnan().all()
        d4 = out[:, :V].clone()
        l5, d5 = sl.distill_step(p, wide[:, :V], lay, gt)          # rows of logits and gradient that stand differently
        assert torch.equal(l5, l4) and torch.equal(d5, d4)
        assert torch.equal(sl.distill_step(p, wide[:, :V], lay, gt, out=wide[:, :V])[1], d4) and wide[:, V:].isnan().all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tau,hard", [(1.0, 0.0), (0.25, 0.5), (4.0, 0.5)])
def test_distillation_of_masked_and_extreme_logits(dt, tau, hard):
    """Logits of -inf and of the type's lowest value among ordinary ones, rows that
    hold nothing but the lowest value, sizes past 1e30, and rows without a distribution."""
    sl = _sl()
    rng, V, T = np.random.default_rng(11), 999, 8
    low = float(torch.finfo(DT[dt]).min)
    z = _draw(rng, (T, V), dt, 3.0)
    z[0, 100:] = -np.inf
    z[1, 100:] = low
    z[2] = low
    z[3] = low
    z[3, 50] = -low                                       # one value that is everything
    z[4] *= np.float32(2.0 ** 100)
    z[5] = -np.inf
    z[6, 7] = np.inf
    z[7, 7] = np.nan
    ids = np.stack([rng.permutation(100)[:9] for _ in range(T)])
    ids[3, 0], ids[4, :] = 50, np.argmax(z[4])
    ids[3, 1:] = -1
    labels = ids[:, 0]
    tl = rng.standard_normal((T, 9)).astype(np.float32)
    p = sl.DistillTargets(_ints(ids), _dev(tl), _ints(labels), tau, hard)
    lay = sl.Layout([0], T)
    loss, dz = sl.distill_step(p, _dev(z, dt), lay)
    assert loss[5:].isnan().all() and dz[5:].isnan().all()
    rl, rz, bl, bz = O.distill(z[:5], ids[:5], tl[:5], labels[:5], tau, hard)
    _within(loss[:5], rl, U32 * (bl(100) + np.abs(rl)), "loss")
    _within(dz[:5], rz, HALF[dt] * np.abs(rz) + U32 * bz(100) + TINY, "dz")
    l2, stats = sl.distill_fwd(p, _dev(z, dt), lay)
    assert torch.equal(l2.nan_to_num(-1.0), loss.nan_to_num(-1.0))
    assert torch.equal(sl.distill_bwd(p, _dev(z, dt), stats, lay).nan_to_num(-1.0), dz.nan_to_num(-1.0))


def test_distillation_where_the_student_has_no_probability():
    """An entry whose logit is -inf costs infinitely much and has a finite gradient;
    one without weight costs nothing.  Teacher's entries that are no numbers."""
    sl = _sl()
    z = torch.zeros(4, 24, device="cuda")
    z[:, 3] = float("-inf")
    ids = _ints([[3, 5], [3, 5], [4, 5], [4, 5]])
    tl = _dev([[0.0, 0.0], [-np.inf, 0.0], [np.nan, 0.0], [np.inf, 0.0]])
    p = sl.DistillTargets(ids, tl)
    loss, dz = sl.distill_step(p, z, sl.Layout([0], 4))
    assert loss[0] == float("inf") and abs(float(dz[0, 3]) + 0.5) < 1e-6 and abs(float(dz[0, 5]) + 0.5 - 1 / 23) < 1e-6
    assert abs(float(loss[1]) - np.log(23.0)) < 1e-5 and float(dz[1, 3]) == 0.0
    assert loss[2:].isnan().all()


def test_rows_without_a_loss_are_not_read():
    """Context rows, rows of weight 0 in the backward, rows without entries and label."""
    sl = _sl()
    V, lay = 1003, sl.Layout([2, 0], 3)
    rng = np.random.default_rng(0)
    z = _dev(_draw(rng, (6, V), "f32"))
    z[[0, 1, 4]] = float("nan")
    ids = _ints(np.full((6, 2), 5))
    ids[4] = -1
    labels = _ints([1, 2, 3, 4, -1, 6])
    p = sl.DistillTargets(ids, torch.zeros(6, 2, device="cuda"), labels, 2.0, 0.5)
    loss, stats = sl.distill_fwd(p, z, lay)
    assert not loss[[0, 1, 4]].any() and loss[[2, 3, 5]].isfinite().all()
    g = torch.ones(6, device="cuda")
    dz = sl.distill_bwd(p, z, stats, lay, g)
    assert not dz[[0, 1, 4]].any() and dz[[2, 3, 5]].any(1).all()
    l2, d2 = sl.distill_step(p, z, lay, g)
    assert torch.equal(l2, loss) and torch.equal(d2, dz)
    z[3], g[3] = float("nan"), 0.0
    assert not sl.distill_bwd(p, z, stats, lay, g)[3].any()
    l3, d3 = sl.distill_step(p, z, lay, g)
    assert l3[3].isnan() and not d3[3].any() and torch.equal(d3[[2, 5]], dz[[2, 5]])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [32000, 32001])
def test_large_logits_take_the_same_steps(dt, V):
    """Past 112 MiB whole rows go past the caches: bit for bit what fewer rows give."""
    sl = _sl()
    T = 2400
    g = torch.Generator(device="cuda").manual_seed(3)
    z = (3 * torch.randn(T, V, generator=g, device="cuda")).to(DT[dt])
    ids, labels = (torch.randint(0, V, s, generator=g, device="cuda").int() for s in ((T, 7), (T,)))
    tl, w = torch.randn(T, 7, generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")
    lay = sl.Layout([600, 0], T // 2)
    p = sl.DistillTargets(ids, tl, labels, 1.5, 0.25)
    loss, stats = sl.distill_fwd(p, z, lay)
    dz = sl.distill_bwd(p, z, stats, lay, w)
    l2, d2 = sl.distill_step(p, z, lay, w)
    assert torch.equal(l2, loss) and torch.equal(d2, dz) and not loss[:600].any() and not dz[:600].any()
    for a in (600, 1100, 1200, 2300):
        s = slice(a, a + 100)
        q = sl.DistillTargets(ids[s].clone(), tl[s].clone(), labels[s].clone(), 1.5, 0.25)
        l3, d3 = sl.distill_step(q, z[s], sl.Layout([0], 100), w[s].clone())     # (z at any alignment of its rows)
        assert torch.equal(l3, loss[s]) and torch.equal(d3, dz[s]), a


def test_distillation_offsets_past_32_bits():
    sl = _sl()
    V, T = 131071, 16400
    lay = sl.Layout([T - 2], T)
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    assert z.numel() > 2 ** 31
    z[-1, -1] = 4.0
    ids = torch.full((T, 2), V - 1, dtype=torch.int32, device="cuda")
    p = sl.DistillTargets(ids, torch.zeros(T, 2, device="cuda"))
    loss, dz = sl.distill_step(p, z, lay, out=z)
    S = np.exp(4.0) + V - 1
    # two entries of probability 1/2, each 1/2 (log 1/2 - log q)
    assert abs(float(loss[-1]) - (np.log(S) - 4.0 - np.log(2))) < 1e-4
    assert abs(float(loss[-2]) - (np.log(V) - np.log(2))) < 1e-4
    assert not loss[:-2].any() and not dz[:-2].any()
    want = np.array([1 / S, np.exp(4.0) / S - 1.0])
    np.testing.assert_allclose(_np(dz[-1, [0, V - 1]]), want, rtol=2.0 ** -7)


def test_distillation_gradient_against_differences():
    sl = _sl()
    rng, case = np.random.default_rng(21), (2, 4, [1, 0], 211, 6)
    z, ids, tl, labels, rows, g = _distill_case(rng, case, "f32")
    e = rng.standard_normal(z.shape)
    p = sl.DistillTargets(_ints(ids), _dev(tl), _ints(labels), 1.5, 0.25)
    _, dz = sl.distill_step(p, _dev(z), sl.Layout(case[2], case[1]), _dev(g))
    f = lambda s: (O.distill(z + s * e, ids, tl, labels, 1.5, 0.25, rows)[0] * g).sum()
    d = 1e-5
    size = np.abs(_np(dz) * e).sum()
    assert abs((_np(dz) * e).sum() - (f(d) - f(-d)) / (2 * d)) <= 1e-5 * size


# ---- all of them ---------------------------------------------------------------------
def _everything(sl, D=520, V=1003, T=70, dt="bf16", seed=0):
    """Inputs of every operator and a function that runs them all."""
    rng, lay = np.random.default_rng(seed), sl.Layout([5, 0], T // 2)
    t = {"E": _dev(_draw(rng, (V, D), dt), dt), "ids": _ints(rng.integers(0, V, T)), "r": _dev(_draw(rng, (T, D), dt), dt),
         "dy": _dev(_draw(rng, (T, D), dt), dt), "w": _dev(rng.standard_normal(D)), "b": _dev(rng.standard_normal(D)),
         "z": _dev(_draw(rng, (T, V), dt), dt), "top": _ints(rng.integers(0, V, (T, 9))), "tl": _dev(rng.standard_normal((T, 9))),
         "labels": _ints(rng.integers(0, V, T)), "g": _dev(rng.standard_normal(T))}
    ew, nw = sl.EmbedWorkspace(lay, D, "cuda"), sl.LayerNormWorkspace(lay, D, "cuda")

    def call():
        x = sl.embed_fwd(t["E"], t["ids"], lay, scale=3.0)
        y, h, stats = sl.layer_norm_fwd(x, t["w"], t["b"], lay, residual=t["r"])
        gr = sl.layer_norm_bwd(h, t["w"], stats, lay, t["dy"], dh=t["dy"], buf=nw)
        dE = sl.embed_bwd(t["ids"], gr["dx"], lay, V, scale=3.0, buf=ew)
        p = sl.DistillTargets(t["top"], t["tl"], t["labels"], 2.0, 0.5)
        loss, st = sl.distill_fwd(p, t["z"], lay)
        dz = sl.distill_bwd(p, t["z"], st, lay, t["g"])
        return [x, y, h, gr["dx"], gr["dw"], gr["db"], dE, loss, dz, *sl.distill_step(p, t["z"], lay, t["g"])]
    return t, call


def test_two_graphs_replayed_with_eager_work_between():
    sl = _sl()
    runs = []
    for seed in (0, 1):
        t, call = _everything(sl, T=5000 if seed else 70, seed=seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        runs.append((t, call, graph, out))
    for i in range(3):
        for t, call, graph, out in runs:
            t["r"].copy_(torch.roll(t["r"], 1, 0))
            t["ids"].copy_(torch.roll(t["ids"], 3, 0))
            t["z"].mul_(-1.0)
        for _, _, graph, _ in runs:
            graph.replay()
        got = [[x.clone() for x in out] for *_, out in runs]
        torch.cuda.synchronize()
        for (t, call, _, _), have in zip(runs, got):
            for u, v in zip(have, call()):
                assert torch.equal(u, v)


def test_calls_on_two_streams_at_once():
    sl = _sl()
    (_, a), (_, b) = (_everything(sl, T=3000, seed=s) for s in (2, 3))
    want = [[x.clone() for x in f()] for f in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, f in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for u, v in zip(g, w):
                assert torch.equal(u, v)


def test_outputs_over_other_tensors_are_refused():
    sl = _sl()
    E_, lay = sl.SparseLoraError, sl.Layout([0], 8)
    x, ids = torch.zeros(8, 16, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(E_, match="may not share"):
        sl.embed_fwd(x, ids, lay, out=x)
    with pytest.raises(E_, match="may not share"):
        sl.embed_bwd(ids, x, lay, 8, out=x)
    p = sl.DistillTargets(torch.zeros(8, 4, dtype=torch.int32, device="cuda"), torch.zeros(8, 4, device="cuda"))
    buf = torch.zeros(9, 16, device="cuda")
    with pytest.raises(E_, match="may not share"):
        sl.distill_step(p, buf[:8], lay, out=buf[1:])
    z = torch.zeros(8, 4, device="cuda")
    _, stats = sl.distill_fwd(p, z, lay)
    with pytest.raises(E_, match="may not share"):
        sl.distill_bwd(p, z, stats, lay, out=stats)
    with pytest.raises(E_, match="may not share"):
        sl.distill_step(p, z, lay, out=p.top_logits)
