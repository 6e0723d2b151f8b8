"""Sparse projections around differential attention with grouped kv heads: query
head 2 h + m meets kv head 2 (h / G) + m, and the channels that the projections
keep have to follow it."""
import warnings

import numpy as np
import pytest

import oracle as O
import workloads as W

torch = pytest.importorskip("torch")

HEADS = [(4, 2, 32), (8, 2, 16), (16, 4, 16), (4, 4, 16)]


def _pairs(heads):
    return heads[0] // 2, heads[1] // 2, 2 * heads[2]


def _layout(L=24, ctx=(24, 17)):
    rows = [b * L + t for b, n in enumerate(ctx) for t in range(n)]
    return L, list(ctx), rows


@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_kept_channels_meet_where_the_projections_see_pairs(heads):
    """In the oracle: a is 0 at context rows outside the columns that o keeps, and
    every kept channel of q meets a kept one of k, with the pairs as heads.  With
    the heads themselves neither holds once G > 1."""
    L, ctx, rows = _layout()
    hq, hkv, hd = heads
    rng = np.random.default_rng(3)
    idx = [[np.sort(rng.choice(hkv * hd, hkv * hd // 2, replace=False)) for _ in ctx] for _ in range(2)]
    x = {n: rng.standard_normal((2 * L, h * hd)) for n, h in (("q", hq), ("k", hkv), ("v", hkv))}
    for seen, holds in ((_pairs(heads), True), (heads, hq == hkv)):
        mq, mk, mv, mo = O.attn_masks(ctx, L, idx[0], idx[1], *seen)
        a = O.diff_attention(x["q"] * mq, x["k"] * mk, x["v"] * mv, [np.zeros(hd)] * 4, 0.4, 2, heads, hd ** -0.5,
                             True)["a"]
        assert (not a[rows][mo[rows] == 0].any()) == holds
        kq = mq[0].reshape(hq // 2, 2, hd)
        meets = mk[0].reshape(hkv // 2, 2, hd).repeat(hq // hkv, axis=0)
        assert np.array_equal(kq, meets) == holds


def test_pair_heads():
    import contextual_sparsity_lora_svd_amd as sl
    assert sl.pair_heads((32, 8, 128)) == (16, 4, 256)
    for bad in ((3, 1, 16), (4, 1, 16)):
        with pytest.raises(sl.SparseLoraError):
            sl.pair_heads(bad)
    core = sl.DiffAttention((8, 4, 16), device="cpu")
    lay = sl.Layout([4], 4)
    assert core.projection_heads == core.bind(lay).projection_heads == (4, 2, 32)


def _bf(x):
    return W.round_to_bf16(np.asarray(x, dtype=np.float32))


def _layer(sl, heads, D=128, r=8, seed=31):
    hq, hkv, hd = heads
    rng = np.random.default_rng(seed)
    w = {n: _bf(rng.standard_normal(s) * 0.05) for n, s in
         (("Wq", (hq * hd, D)), ("Wk", (hkv * hd, D)), ("Wv", (hkv * hd, D)), ("Wo", (D, hq * hd)))}
    dev = {n: torch.from_numpy(t).cuda().to(torch.bfloat16) for n, t in w.items()}
    gen = torch.Generator().manual_seed(4)
    sched = sl.SparsitySchedule([sl.LayerRatios(qk=50, vo=50)], total_steps=20)
    proj = sl.SparseLoRAQKVO(dev["Wq"], dev["Wk"], dev["Wv"], dev["Wo"], heads, r, est_rank=4, lora_scale=0.5,
                             schedule=sched, generator=gen)
    return w, proj, gen


@pytest.mark.gpu
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_bound_core_between_sparse_projections(heads):
    """Through the modules: a and its gradient are 0 at context rows outside o's
    columns, o loses nothing of a, the kept q/k channels are the best by the norms
    of the heads that meet, and the projections' outputs and gradients are the
    oracle's with the pairs as heads."""
    import contextual_sparsity_lora_svd_amd as sl
    from tests.gpu_helpers import assert_close, check_selection, to_np
    L, ctx, rows = _layout()
    hq, hkv, hd = heads
    w, proj, gen = _layer(sl, heads)
    core = sl.DiffAttention(heads, lambda_init=0.4, generator=gen)
    lay = sl.Layout(ctx, L)
    X = W.make_activations(12, 2 * L, 128, 16, "bf16")
    dO = _bf(np.random.default_rng(5).standard_normal((2 * L, 128)))
    seen, bound = {}, core.bind(lay)

    def attention(q, k, v):
        a = bound(q, k, v)
        for n, t in (("q", q), ("k", k), ("v", v), ("a", a)):
            t.retain_grad()
            seen[n] = t
        return a
    attention.projection_heads = bound.projection_heads

    Xd = torch.from_numpy(X).cuda().to(torch.bfloat16).requires_grad_(True)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        out = proj(Xd, lay, attention, step=5)
    assert torch.equal(out, proj(Xd, lay, bound, step=5))
    out.backward(torch.from_numpy(dO).cuda().to(torch.bfloat16))
    iqk, ivo = (t.cpu().numpy() for t in proj.last_idx)
    pairs = _pairs(heads)
    mo = O.attn_masks(ctx, L, iqk, ivo, *pairs)[3]
    val = {n: to_np(t) for n, t in seen.items()}
    grad = {n: to_np(t.grad) for n, t in seen.items()}
    assert val["a"][rows].any() and not val["a"][rows][mo[rows] == 0].any()
    assert grad["a"][rows].any() and not grad["a"][rows][mo[rows] == 0].any()

    names = ("Aq", "Bq", "Ak", "Bk", "Av", "Bv", "Ao", "Bo")
    p = {"X": X, "a": val["a"], **w}
    p.update({n: _bf(getattr(proj, n).detach().cpu().numpy()) for n in names})
    ref, cache = O.qkvo_forward(p, ctx, L, list(iqk), list(ivo), pairs, 0.5)
    gr = O.qkvo_backward(p, cache, {"dq": grad["q"], "dk": grad["k"], "dv": grad["v"], "d_out": dO}, 0.5)
    for n in "qkv":
        assert_close(val[n], ref[n], "bf16", n)
    assert_close(to_np(out), ref["o"], "bf16", "o")
    assert_close(to_np(Xd.grad), gr["dX"], "bf16", "dX")
    assert_close(grad["a"], gr["da"], "bf16", "da")
    for n in names:
        assert_close(to_np(getattr(proj, n).grad), gr["d" + n], "bf16", "d" + n)

    f = {n: [t.float().cpu().numpy() for t in proj.est[n]] for n in ("Wq", "Wk")}
    sc = np.stack([O.scores_qk_norm(X[b * L:b * L + n], f["Wq"][0].T, f["Wq"][1], f["Wk"][0].T, f["Wk"][1], *pairs,
                                    dtype=np.float64) for b, n in enumerate(ctx)])
    check_selection(iqk, sc, proj.last_k[0])


@pytest.mark.gpu
def test_a_core_without_its_heads_warns_and_wrong_ones_are_refused():
    import contextual_sparsity_lora_svd_amd as sl
    L, ctx, _ = _layout()
    heads, lay = (4, 2, 32), sl.Layout(ctx, L)
    _, proj, gen = _layer(sl, heads)
    core = sl.DiffAttention(heads, generator=gen)
    X = torch.randn(2 * L, 128, device="cuda").to(torch.bfloat16)
    with pytest.warns(UserWarning, match="do not meet"):
        proj(X, lay, lambda q, k, v: core(q, k, v, lay), step=5)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        proj(X, lay, lambda q, k, v: core(q, k, v, lay), step=0)       # dense: every channel is kept
        core(*(torch.randn(2 * L, n, device="cuda") for n in (128, 64, 64)), lay)
    other = sl.DiffAttention((8, 4, 32), generator=gen)
    with pytest.raises(sl.SparseLoraError, match="projection_heads"):
        proj(X, lay, other.bind(lay), step=5)
