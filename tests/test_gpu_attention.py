"""GPU parity of rotary positions, head norms and differential attention with
the fp64 oracle: element by element, within bounds derived from the number
formats (half a step of the output's type, half a step of each matrix operand
that is rounded, fp32 sums at their worst case)."""
import numpy as np
import pytest

import oracle as O
from workloads import round_to_bf16

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}          # half a step, relative
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _sl():
    import contextual_sparsity_lora_svd_amd as sl
    return sl


def _draw(rng, shape, dt, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    return round_to_bf16(x) if dt == "bf16" else x


def _dev(x, dt):
    return torch.from_numpy(np.array(x, dtype=np.float32)).cuda().to(DT[dt])


def _np(t):
    return t.detach().cpu().double().numpy()


def _within(got, ref, bound, what):
    got = _np(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    assert over.max() <= 0, (f"{what}: off by {np.abs(got - ref).ravel()[over.argmax()]:.3e}, "
                             f"bound {np.broadcast_to(bound, over.shape).ravel()[over.argmax()]:.3e}")


# ---- rotary and head norms --------------------------------------------------
ROT = [  # batch, seq, hq, hkv, hd, rot, interleaved, scaling, factor
    (1, 1, 1, 1, 2, 2, False, "none", 1.0),
    (2, 3, 4, 2, 16, 16, True, "linear", 4.0),
    (1, 37, 32, 8, 128, 128, False, "wavelength", 8.0),
    (3, 5, 5, 1, 80, 40, True, "none", 1.0),
    (1, 9, 3, 3, 80, 80, False, "yarn", 16.0),
    (2, 7, 2, 1, 256, 64, False, "base", 4.0),
    (1, 4, 2, 2, 6, 4, True, "none", 1.0),
    (1, 5, 2, 1, 250, 250, False, "none", 1.0),       # single pairs, two units to a lane
    (1, 3, 7, 2, 96, 24, False, "none", 1.0),
    (1, 2500, 2, 1, 64, 64, False, "none", 1.0),      # more tokens than blocks
]


def _positions(rng, T, kind):
    if kind == "row":
        return None, None
    p = rng.integers(-5 if kind == "near" else 0, 50 if kind == "near" else 2 ** 31 - 1, T)
    return p, torch.from_numpy(p.astype(np.int32)).cuda()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", ROT, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("where", ["row", "near", "far"])
def test_rotary_and_head_norm(case, dt, where):
    sl = _sl()
    B, Ls, hq, hkv, hd, rot, inter, scaling, factor = case
    rng = np.random.default_rng(hash((B, Ls, hd)) % 1000)
    T, heads = B * Ls, (hq, hkv, hd)
    lay = sl.Layout([Ls] * B, Ls)
    pos_np, pos = _positions(rng, T, where)
    pos_np = np.arange(T) % Ls if pos_np is None else pos_np
    r = sl.Rotary(rot, interleaved=inter, scaling=scaling, factor=factor, original_len=2048)
    f, amp = O.rotary_frequencies(rot, scaling=scaling, factor=factor, original_len=2048)
    # the oracle's angles at far positions are off by p f 2^-53, the table's by p 2^-64 turns
    ang = 2.0 ** 31 * 2.0 ** -50 if where == "far" else 0.0
    x = {n: _draw(rng, (T, h * hd), dt) for n, h in (("q", hq), ("k", hkv))}
    g = {n: _draw(rng, (T, h * hd), dt) for n, h in (("q", hq), ("k", hkv))}
    w = {n: (1 + 0.3 * rng.standard_normal(hd)).astype(np.float32) for n in "qk"}
    d = {n: _dev(t, dt) for n, t in x.items()}
    dg = {n: _dev(t, dt) for n, t in g.items()}
    dw = {n: torch.from_numpy(t).cuda() for n, t in w.items()}

    def check(got, xin, inverse, what):
        ref = O.rotate(xin, pos_np, f, amp, hd, inter, inverse)
        mag = O.rotate(xin, pos_np, f, amp, hd, inter, absolute=True)
        # cosine, amplitude, two products and their sum: below 8 half steps of fp32
        _within(got, ref, HALF[dt] * np.abs(ref) + (8 * U32 + ang) * mag, what)

    for inverse in (False, True):
        q, k = sl.rotary(d["q"], d["k"], lay, heads, r, pos, inverse=inverse)
        check(q, x["q"], inverse, "q")
        check(k, x["k"], inverse, "k")
    q1, none = sl.rotary(d["q"], None, lay, heads, r, pos)
    assert none is None
    check(q1, x["q"], False, "q alone")
    c = d["q"].clone(), d["k"].clone()
    sl.rotary(*c, lay, heads, r, pos, out=c)                 # in place
    check(c[0], x["q"], False, "q in place")
    check(c[1], x["k"], False, "k in place")

    for use_rot in (True, False):
        rr, ff = (r, f) if use_rot else (None, np.zeros(0))
        y = dict(zip("qk", sl.head_norm_fwd(d["q"], d["k"], dw["q"], dw["k"], lay, heads, rr, pos, 1e-5)))
        gr = sl.head_norm_bwd(d["q"], d["k"], dw["q"], dw["k"], lay, heads, dg["q"], dg["k"], rr, pos, 1e-5)
        for n in "qk":
            u = O.head_norm(x[n], w[n], hd, 1e-5)
            ref = O.rotate(u, pos_np, ff, amp, hd, inter)
            mag = O.rotate(u, pos_np, ff, amp, hd, inter, absolute=True)
            # mean square: hd terms in fp32, halved by the root; then the rotation
            _within(y[n], ref, HALF[dt] * np.abs(ref) + ((hd / 2 + 16) * U32 + ang) * mag, "norm " + n)
            gb = O.rotate(g[n], pos_np, ff, amp, hd, inter, inverse=True)
            gm = O.rotate(g[n], pos_np, ff, amp, hd, inter, absolute=True)
            dx, dwn, _, _ = O.head_norm_backward(x[n], w[n], gb, hd, 1e-5)
            _, _, mx, mw = O.head_norm_backward(x[n], w[n], gm, hd, 1e-5)
            _within(gr["d" + n], dx, HALF[dt] * np.abs(dx) + ((2 * hd + 32) * U32 + 2 * ang) * mx, "d" + n)
            chain = hd / 2 + 64 + T * max(hq, hkv) / 256        # longest run of additions in one sum
            _within(gr["dw" + n], dwn, (chain * U32 + 2 * ang) * mw, "dw" + n)


def test_norm_of_zero_rows_and_alone():
    """Zero rows stay zero, their gradient is g w / sqrt(eps); k left out."""
    sl = _sl()
    lay, heads = sl.Layout([3], 3), (2, 1, 32)
    x = torch.zeros(3, 64, device="cuda")
    w = torch.full((32,), 2.0, device="cuda")
    y, k = sl.head_norm_fwd(x, None, w, None, lay, heads, eps=0.25)
    assert k is None and not y.any()
    g = sl.head_norm_bwd(x, None, w, None, lay, heads, torch.ones_like(x), None, eps=0.25)
    assert torch.equal(g["dq"], torch.full_like(x, 4.0)) and not g["dwq"].any() and "dk" not in g


# ---- differential attention --------------------------------------------------
DIFF = [  # batch, seq, hq, hkv, hd, causal, lens
    (1, 1, 2, 2, 8, True, None),
    (1, 2, 4, 2, 16, False, None),
    (2, 33, 4, 2, 16, False, [33, 0]),
    (1, 64, 4, 4, 32, True, None),
    (3, 65, 8, 2, 64, True, [65, 1, 31]),
    (2, 130, 4, 2, 80, True, [130, 77]),
    (2, 96, 6, 2, 96, False, None),
    (1, 257, 4, 4, 128, True, None),
    (2, 200, 8, 2, 128, False, [200, 129]),
    (3, 32, 2, 2, 40, True, [0, 32, 16]),
    (1, 515, 2, 2, 64, True, None),
    (1, 140, 2, 2, 128, True, [128]),
]


def _diff_inputs(case, dt, seed=0, spread=1.0):
    B, Ls, hq, hkv, hd, causal, lens = case
    rng = np.random.default_rng(seed + Ls)
    T = B * Ls
    x = {"q": _draw(rng, (T, hq * hd), dt, spread), "k": _draw(rng, (T, hkv * hd), dt, spread),
         "v": _draw(rng, (T, hkv * hd), dt), "da": _draw(rng, (T, hq * hd), dt)}
    lv = [(0.3 * rng.standard_normal(hd) / np.sqrt(hd / 8)).astype(np.float32) for _ in range(4)]
    return x, lv


def _run_diff(sl, case, dt, x, lv, lam0=0.6, pad=float("nan")):
    B, Ls, hq, hkv, hd, causal, lens = case
    lay = sl.Layout([Ls] * B, Ls)
    d = {n: _dev(t, dt) for n, t in x.items()}
    if lens is not None:
        for b, n in enumerate(lens):                        # padding may hold anything
            for t in d.values():
                t[b * Ls + n:(b + 1) * Ls] = pad
    p = sl.DiffAttnParams(dict(zip(sl.DiffAttnParams.NAMES, (torch.from_numpy(t).cuda() for t in lv))), (hq, hkv, hd),
                          lambda_init=lam0, causal=causal)
    a, buf = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], lay, lens=lens)
    g = sl.diff_attn_bwd(p, d["q"], d["k"], d["v"], a, lay, buf, d["da"])
    return p, d, lay, a, g, buf


def _check_diff(case, dt, x, lv, a, g, lam0=0.6):
    B, Ls, hq, hkv, hd, causal, lens = case
    ref = O.diff_attention(x["q"], x["k"], x["v"], lv, lam0, B, (hq, hkv, hd), float(np.float32(hd ** -0.5)), causal,
                           lens, x["da"], rnd=HALF["bf16"] if dt == "bf16" else 0.0)
    for n, got in [("a", a)] + sorted(g.items()):
        half = U32 if n.startswith("dl") else HALF[dt]
        _within(got, ref[n], half * np.abs(ref[n]) + ref["bound"][n] * (1 + half) + 1e-30, n)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", DIFF, ids=lambda c: "x".join(map(str, c)).replace(" ", ""))
def test_diff_attention(case, dt):
    sl = _sl()
    x, lv = _diff_inputs(case, dt)
    _, _, _, a, g, _ = _run_diff(sl, case, dt, x, lv)
    _check_diff(case, dt, x, lv, a, g)
    B, Ls, lens = case[0], case[1], case[6]
    if lens is not None:                                     # padding: outputs and gradients are 0
        for b, n in enumerate(lens):
            for t in (a, g["dq"], g["dk"], g["dv"]):
                assert not t[b * Ls + n:(b + 1) * Ls].any()


# The bf16 kernels' other halves: workgroups of 128 rows (many head pairs and
# sequences), a kv group's heads cut into three parts, the most sequences of a
# layout; head widths that fill no tile.
MANY = [  # batch, seq, hq, hkv, hd, causal, lens
    (6, 140, 32, 32, 24, False, None),
    (6, 140, 32, 32, 64, False, [140, 0, 129, 1, 64, 97]),
    (6, 140, 32, 32, 72, False, None),
    (6, 140, 32, 32, 128, False, [140, 139, 128, 127, 33, 32]),
    (16, 140, 32, 16, 64, True, [140, 1, 32, 33, 64, 65, 96, 97, 127, 128, 129, 0, 139, 31, 63, 95]),
    (16, 140, 32, 32, 120, True, None),
    (16, 140, 32, 32, 8, True, None),
    (16, 140, 32, 32, 96, True, None),
    (6, 300, 24, 8, 32, False, [300, 256, 257, 0, 1, 290]),
    (8, 300, 24, 8, 128, True, [300, 256, 257, 0, 1, 290, 128, 129]),
    (1, 300, 20, 4, 56, True, None),
    (64, 9, 4, 2, 16, True, list(range(10)) * 6 + [9, 0, 9, 1]),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "x".join(map(str, c[:6])))
def test_diff_attention_many_heads(case):
    test_diff_attention(case, "bf16")


@pytest.mark.parametrize("hd,causal,L", [(64, True, 150), (128, False, 150), (32, True, 77), (96, True, 200)])
def test_diff_attention_scores_that_outgrow_the_first_tile(hd, causal, L):
    """Every 40 keys the scores rise by about 2^92 in the weights: relative to the
    first tile's maximum the rows' sums overflow fp32 from the second step on.  One
    sequence's rows do, the other's stay small."""
    sl = _sl()
    case = (2, L, 4, 2, hd, causal, None)
    x, lv = _diff_inputs(case, "bf16", seed=12)
    rise = (64.0 / np.sqrt(hd)) * (np.arange(L)[:, None] // 40) * 0.5
    x["q"][:L] = 2.0
    x["k"][:L] = round_to_bf16((rise + 0.125 * x["k"][:L]).astype(np.float32))
    _, _, _, a, g, _ = _run_diff(sl, case, "bf16", x, lv)
    _check_diff(case, "bf16", x, lv, a, g)

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["peaked", "flat", "late", "negative"])
def test_diff_attention_distributions(dt, kind):
    """One key takes all the weight; all weights equal; the maximum arrives with
    the last keys, far above the rest; lambda below zero."""
    sl = _sl()
    case = (1, 150, 4, 2, 64, kind != "flat", None)
    x, lv = _diff_inputs(case, dt, seed=5)
    if kind == "peaked":
        x["q"] = _draw(np.random.default_rng(1), x["q"].shape, dt, 3.0)
        x["k"] = _draw(np.random.default_rng(2), x["k"].shape, dt, 3.0)
    if kind == "flat":
        x["k"][:] = 0
    if kind == "late":
        x["q"][:] = 0.5
        x["k"][:] = 0.25 * (np.arange(150)[:, None] // 40) ** 2
    lam0 = -0.9 if kind == "negative" else 0.6
    _, _, _, a, g, _ = _run_diff(sl, case, dt, x, lv, lam0)
    _check_diff(case, dt, x, lv, a, g, lam0)


def test_diff_attention_gradient_against_differences():
    """Central differences of the fp32 kernel's own forward along random
    directions.  With step e the difference is off by O(e^2) times the third
    derivative and by the forward's rounding over e: at e = 2^-6 both stay
    below a hundredth of the gradient's size here."""
    sl = _sl()
    case = (1, 40, 4, 2, 16, True, None)
    x, lv = _diff_inputs(case, "f32", seed=9)
    p, d, lay, a, g, _ = _run_diff(sl, case, "f32", x, lv)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(q, k, v, t):
        pp = sl.DiffAttnParams(t, p.heads, p.lambda_init, causal=True)
        return (sl.diff_attn_fwd(pp, q, k, v, lay)[0].double() * d["da"].double()).sum().item()

    base = {"q": d["q"], "k": d["k"], "v": d["v"], **p.t}
    e = 2.0 ** -6
    for n in base:
        v = torch.randn(base[n].shape, generator=gen, device="cuda")
        v /= v.norm()
        f = []
        for s in (e, -e):
            y = dict(base)
            y[n] = (base[n] + s * v).contiguous()
            f.append(loss(y["q"], y["k"], y["v"], {m: y[m] for m in p.NAMES}))
        num = (f[0] - f[1]) / (2 * e)
        size = g["d" + n].double().norm().item()
        assert abs(num - (g["d" + n].double() * v).sum().item()) <= 0.01 * size, n


def test_calls_are_repeatable_and_independent():
    """The same call gives the same bits; two calls on two streams with their
    own buffers give what each gives alone; the inputs are left as they were."""
    sl = _sl()
    cases = [(2, 130, 8, 2, 64, True, [130, 100]), (1, 200, 4, 4, 128, False, None)]
    runs = []
    for c in cases:
        x, lv = _diff_inputs(c, "bf16", seed=3)
        runs.append((c, x, lv, _run_diff(sl, c, "bf16", x, lv, pad=0.0)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for s, (c, x, lv, (p, d, lay, a, g, _)) in zip(streams, runs):
        before = {n: t.clone() for n, t in d.items()}
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            a2, buf = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], lay, lens=c[6])
            g2 = sl.diff_attn_bwd(p, d["q"], d["k"], d["v"], a2, lay, buf, d["da"])
        outs.append((a, g, a2, g2, d, before))
    torch.cuda.synchronize()
    for a, g, a2, g2, d, before in outs:
        assert torch.equal(a, a2)
        for n in g:
            assert torch.equal(g[n], g2[n]), n
        for n in d:
            assert torch.equal(d[n], before[n]), n


def test_results_do_not_depend_on_what_the_buffers_held():
    sl = _sl()
    case = (2, 97, 4, 2, 64, True, [97, 40])
    x, lv = _diff_inputs(case, "bf16", seed=4)
    p, d, lay, a, g, buf = _run_diff(sl, case, "bf16", x, lv, pad=0.0)
    buf2 = sl.DiffAttnWorkspace(p, lay, torch.bfloat16, "cuda", lens=case[6])
    out = {n: torch.full_like(t, float("nan")) for n, t in g.items()}
    for t in (buf2.saved, buf2.ws):
        t.fill_(0xFF)
    a2, _ = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], lay, buf=buf2, out=torch.full_like(a, float("nan")))
    buf2.ws.fill_(0xFF)
    g2 = sl.diff_attn_bwd(p, d["q"], d["k"], d["v"], a2, lay, buf2, d["da"], out=out)
    assert torch.equal(a, a2)
    for n in g:
        assert torch.equal(g[n], g2[n]), n
    nbuf = sl.HeadNormWorkspace(lay, p.heads, "cuda")
    w = torch.ones(64, device="cuda")
    ref = sl.head_norm_bwd(d["q"], d["k"], w, w, lay, p.heads, d["da"], d["v"], buf=nbuf)
    nbuf.ws.fill_(0xFF)
    again = sl.head_norm_bwd(d["q"], d["k"], w, w, lay, p.heads, d["da"], d["v"], buf=nbuf)
    for n in ref:
        assert torch.equal(ref[n], again[n]), n


def test_graph_replays_match_eager():
    """The three operators, forward and backward, captured once and replayed
    on changing inputs, with the program's own eager work in between."""
    sl = _sl()
    case = (2, 70, 4, 2, 64, True, [70, 50])
    x, lv = _diff_inputs(case, "bf16", seed=6)
    lay, heads = sl.Layout([70, 70], 70), (4, 2, 64)
    rot, w = sl.Rotary(64), torch.ones(64, device="cuda")
    d = {n: _dev(t, "bf16") for n, t in x.items()}
    p = sl.DiffAttnParams(dict(zip(sl.DiffAttnParams.NAMES, (torch.from_numpy(t).cuda() for t in lv))), heads)
    buf, nbuf = sl.DiffAttnWorkspace(p, lay, torch.bfloat16, "cuda", lens=case[6]), sl.HeadNormWorkspace(lay, heads, "cuda")

    def step():
        q, k = sl.head_norm_fwd(d["q"], d["k"], w, w, lay, heads, rot)
        a, _ = sl.diff_attn_fwd(p, q, k, d["v"], lay, buf=buf)
        g = sl.diff_attn_bwd(p, q, k, d["v"], a, lay, buf, d["da"])
        n = sl.head_norm_bwd(d["q"], d["k"], w, w, lay, heads, g["dq"], g["dk"], rot, buf=nbuf)
        r = sl.rotary(n["dq"], n["dk"], lay, heads, rot, inverse=True)
        return [a, g["dv"], g["dlq1"], n["dq"], n["dk"], n["dwq"], n["dwk"], *r]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        d["q"].copy_(torch.roll(d["q"], 1, 0))
        d["da"].mul_(0.5 if i % 2 else 2.0)
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        for u, v in zip(got, step()):
            assert torch.equal(u, v)


def test_long_sequence_last_rows():
    """Past one tile and one workgroup: a 2100-row causal sequence, its last
    rows against the oracle's formula."""
    sl = _sl()
    L, heads = 2100, (2, 2, 128)
    rng = np.random.default_rng(8)
    x = {n: _draw(rng, (L, 256), "bf16") for n in ("q", "k", "v")}
    lv = [(0.05 * rng.standard_normal(128)).astype(np.float32) for _ in range(4)]
    p = sl.DiffAttnParams(dict(zip(sl.DiffAttnParams.NAMES, (torch.from_numpy(t).cuda() for t in lv))), heads, 0.5)
    d = {n: _dev(t, "bf16") for n, t in x.items()}
    a, _ = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], sl.Layout([L], L))
    lam = O.diff_lambda(lv, 0.5)[0]
    rows = np.array([0, 1, 127, 128, 1023, 2047, 2048, L - 1])
    k, v = x["k"].astype(np.float64), x["v"].astype(np.float64)
    for r in rows:
        maps = []
        for m in (0, 1):
            s = x["q"][r, 128 * m:128 * (m + 1)].astype(np.float64) @ k[:r + 1, 128 * m:128 * (m + 1)].T * 128 ** -0.5
            w = np.exp(s - s.max())
            maps.append(w / w.sum())
        ref = (maps[0] - lam * maps[1]) @ v[:r + 1]
        mag = (maps[0] + abs(lam) * maps[1]) @ np.abs(v[:r + 1])
        _within(a[r], ref, HALF["bf16"] * np.abs(ref) + (HALF["bf16"] + U32 * (r + 2000)) * mag, f"row {r}")


def test_outputs_that_are_inputs_are_refused():
    sl = _sl()
    case = (1, 20, 2, 2, 16, True, None)
    x, lv = _diff_inputs(case, "bf16")
    p, d, lay, a, g, buf = _run_diff(sl, case, "bf16", x, lv)
    for out in (d["q"], d["k"], d["v"]):
        with pytest.raises(sl.SparseLoraError):
            sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], lay, buf=buf, out=out)
    for out in ({"dq": d["da"]}, {"dk": d["k"]}, {"dq": g["dk"], "dk": g["dk"]}):
        with pytest.raises(sl.SparseLoraError):
            sl.diff_attn_bwd(p, d["q"], d["k"], d["v"], a, lay, buf, d["da"], out=out)


@pytest.mark.parametrize("case", [(2, 97, 4, 2, 64, True, None), (1, 70, 8, 2, 24, False, [65]), (1, 600, 8, 2, 32, True, None)],
                         ids=lambda c: "x".join(map(str, c[:6])))
def test_fp32_results_do_not_depend_on_what_the_buffers_held(case):
    sl = _sl()
    x, lv = _diff_inputs(case, "f32", seed=4)
    p, d, lay, a, g, _ = _run_diff(sl, case, "f32", x, lv, pad=0.0)
    buf = sl.DiffAttnWorkspace(p, lay, torch.float32, "cuda", lens=case[6])
    for t in (buf.saved, buf.ws):
        t.fill_(0xFF)
    a2, _ = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], lay, buf=buf)
    buf.ws.fill_(0xFF)
    g2 = sl.diff_attn_bwd(p, d["q"], d["k"], d["v"], a2, lay, buf, d["da"])
    assert torch.equal(a, a2)
    for n in g:
        assert torch.equal(g[n], g2[n]), n
    _check_diff(case, "f32", x, lv, a, g)


@pytest.mark.parametrize("case", MANY[3:5] + MANY[8:11], ids=lambda c: "x".join(map(str, c[:6])))
def test_diff_attention_many_heads_fp32(case):
    test_diff_attention(case, "f32")


def test_fp32_scores_that_outgrow_the_first_tile():
    sl = _sl()
    case = (1, 150, 4, 2, 64, True, None)
    x, lv = _diff_inputs(case, "f32", seed=12)
    x["q"][:] = 2.0
    x["k"][:] = (np.arange(150)[:, None] // 40) * 4.0 + 0.125 * x["k"]
    _, _, _, a, g, _ = _run_diff(sl, case, "f32", x, lv)
    _check_diff(case, "f32", x, lv, a, g)


def test_two_graphs_with_their_own_buffers():
    """Two captured steps with buffers of their own, replayed in turn and at once
    on two streams, give what the eager calls give."""
    sl = _sl()
    cases = [(2, 70, 4, 2, 64, True, [70, 50]), (1, 190, 4, 4, 32, False, None)]
    made, alive = [], []                # a graph reads the tensors it was captured with
    for c in cases:
        x, lv = _diff_inputs(c, "bf16", seed=6)
        p, d, lay, a, g, _ = _run_diff(sl, c, "bf16", x, lv, pad=0.0)
        buf = sl.DiffAttnWorkspace(p, lay, torch.bfloat16, "cuda", lens=c[6])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a2, _ = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], lay, buf=buf)
            g2 = sl.diff_attn_bwd(p, d["q"], d["k"], d["v"], a2, lay, buf, d["da"])
        made.append((graph, a, g, a2, g2))
        alive.append((p, d, buf))
    streams = [torch.cuda.Stream() for _ in made]
    for together in (False, True, True):
        for s, (graph, a, g, a2, g2) in zip(streams, made):
            a2.fill_(float("nan"))
            torch.cuda.synchronize()
            if not together:
                graph.replay()
        if together:
            for s, m in zip(streams, made):
                with torch.cuda.stream(s):
                    m[0].replay()
        torch.cuda.synchronize()
        for _, a, g, a2, g2 in made:
            assert torch.equal(a, a2)
            for n in g:
                assert torch.equal(g[n], g2[n]), n


def test_fp32_weights_do_not_drift_with_the_tiles():
    """Scores near 31000 that are exact in fp32 and differ by at most 2, the maximum
    in the first keys, values of opposite sign in the two halves.  A rescaling by the
    rounding of maximum * scale (here 3e-4 in the exponent) at each of a wave's 33
    tiles would move the result by 1e-3.  What remains: the exponential, within 2
    half steps; a product over 33 tiles of 32 keys per wave, n / 4 additions; the
    row sums and the join, fewer than 128 more."""
    sl = _sl()
    L, hd, lam, top = 4133, 16, -0.5, 31000.0
    sc = np.float32(np.float32(hd ** -0.5) * np.float32(1.44269504088896341))
    assert abs(top * float(sc) - float(np.float32(np.float32(top) * sc))) > 2.0 ** -12
    raw = np.full(L, top - 1)                                # q . k
    raw[5::7], raw[:32] = top - 2, top
    d = {"q": torch.full((L, 2 * hd), 64.0, device="cuda"),
         "k": _dev((raw / (64 * hd))[:, None].repeat(2 * hd, 1), "f32")}
    assert np.array_equal(_np(d["k"])[:, 0] * 64 * hd, raw)
    v = np.where(np.arange(L) < L // 2, 1.0, -1.0)[:, None] * (1 + np.arange(2 * hd) / 32)
    d["v"] = _dev(v, "f32")
    p = sl.DiffAttnParams({n: torch.zeros(hd, device="cuda") for n in sl.DiffAttnParams.NAMES}, (2, 2, hd), lam,
                          causal=False)
    a, _ = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], sl.Layout([L], L))
    w = np.exp((raw - top) * hd ** -0.5)
    w /= w.sum()
    _within(a, np.broadcast_to((1 - lam) * (w @ v), a.shape),
            (L / 4 + 128) * U32 * (1 - lam) * (w @ np.abs(v)), "a")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_norm_of_q_without_kv_heads(dt):
    """q alone, in a layout of heads that has no kv heads: forward and backward as
    with any kv head count."""
    sl = _sl()
    lay, rng = sl.Layout([5], 5), np.random.default_rng(2)
    x, g = (_dev(_draw(rng, (5, 96), dt), dt) for _ in range(2))
    w = torch.rand(32, device="cuda") + 0.5
    res = []
    for hkv in (0, 1):
        y, _ = sl.head_norm_fwd(x, None, w, None, lay, (3, hkv, 32))
        gr = sl.head_norm_bwd(x, None, w, None, lay, (3, hkv, 32), g, None)
        res.append((y, gr["dq"], gr["dwq"]))
    for u, v in zip(*res):
        assert torch.equal(u, v) and u.any()


# Sequences of many tiles, so that every ring of tiles wraps several times, in enough
# workgroups for the launch rules to take the 128-row kernels of every width (the first
# ten, with a kv group's heads cut into parts), and sequences past 1024 rows in both the
# 128-row and the 64-row kernels.
LONG = [  # batch, seq, hq, hkv, hd, causal, lens
    (8, 330, 48, 16, 24, True, [330, 330, 329, 330, 257, 300, 290, 330]),
    (2, 330, 48, 16, 32, False, None),
    (8, 330, 48, 16, 64, True, None),
    (2, 330, 48, 16, 56, False, [330, 321]),
    (8, 330, 48, 16, 88, True, None),
    (2, 330, 48, 16, 96, False, None),
    (8, 330, 48, 16, 128, True, [330, 330, 329, 330, 257, 300, 290, 330]),
    (2, 330, 48, 16, 128, False, [330, 322]),
    (3, 600, 32, 8, 64, False, [600, 333, 64]),
    (4, 520, 32, 8, 128, True, [520, 519, 385, 400]),
    (4, 1100, 32, 8, 32, True, None),
    (4, 1030, 32, 8, 128, True, [1030, 1029, 1030, 1025]),
    (1, 2060, 32, 8, 72, True, None),
    (1, 2060, 28, 4, 32, True, None),
    (1, 1100, 8, 4, 64, True, None),
    (1, 1100, 4, 4, 128, False, None),
    (1, 700, 4, 2, 88, True, None),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "x".join(map(str, c[:6])))
def test_diff_attention_long(case):
    test_diff_attention(case, "bf16")


@pytest.mark.parametrize("case", [LONG[9], LONG[13]], ids=lambda c: "x".join(map(str, c[:6])))
def test_diff_attention_long_fp32(case):
    test_diff_attention(case, "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.03, 0.7])
@pytest.mark.parametrize("causal", [True, False])
def test_diff_attention_scale(dt, scale, causal):
    """A scale other than head_dim ** -0.5, in the forward and every gradient."""
    sl = _sl()
    B, Ls, hq, hkv, hd = 2, 150, 8, 4, 40
    case = (B, Ls, hq, hkv, hd, causal, None)
    x, lv = _diff_inputs(case, dt, seed=21)
    d = {n: _dev(t, dt) for n, t in x.items()}
    p = sl.DiffAttnParams(dict(zip(sl.DiffAttnParams.NAMES, (torch.from_numpy(t).cuda() for t in lv))), (hq, hkv, hd),
                          lambda_init=0.6, scale=scale, causal=causal)
    lay = sl.Layout([Ls] * B, Ls)
    a, buf = sl.diff_attn_fwd(p, d["q"], d["k"], d["v"], lay)
    g = sl.diff_attn_bwd(p, d["q"], d["k"], d["v"], a, lay, buf, d["da"])
    ref = O.diff_attention(x["q"], x["k"], x["v"], lv, 0.6, B, (hq, hkv, hd), float(np.float32(scale)), causal, None,
                           x["da"], rnd=HALF["bf16"] if dt == "bf16" else 0.0)
    for n, got in [("a", a)] + sorted(g.items()):
        half = U32 if n.startswith("dl") else HALF[dt]
        _within(got, ref[n], half * np.abs(ref[n]) + ref["bound"][n] * (1 + half) + 1e-30, n)


# more than 4096 tokens, in groups of four that the norm's backward walks twice and three
# times over its blocks, the last group not whole
WALK = [  # as ROT
    (1, 4099, 2, 1, 32, 32, False, "none", 1.0),
    (3, 2731, 3, 1, 16, 8, True, "linear", 4.0),
    (1, 4101, 1, 1, 250, 250, False, "none", 1.0),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", WALK, ids=lambda c: "x".join(map(str, c)))
def test_rotary_and_head_norm_over_many_tokens(case, dt):
    test_rotary_and_head_norm(case, dt, "near")


def test_outputs_over_other_tensors_are_refused_by_every_call():
    """q and k swapped as outputs, one output given twice, views that overlap in part,
    vector gradients over parameters: refused before anything is launched."""
    sl = _sl()
    lay, heads, E = sl.Layout([6], 6), (2, 2, 16), sl.SparseLoraError
    flat = torch.randn(8 * 6 * 32, device="cuda")
    n = 6 * 32
    q, k, v, da, y, z = (flat[i * n:(i + 1) * n].view(6, 32) for i in range(6))
    part = flat[n // 2:n // 2 + n].view(6, 32)
    w, rot = torch.ones(16, device="cuda"), sl.Rotary(16)
    before = flat.clone()
    for out in ((k, q), (y, y), (part, y), (y, q)):
        with pytest.raises(E, match="may not share memory"):
            sl.rotary(q, k, lay, heads, rot, out=out)
        with pytest.raises(E, match="may not share memory"):
            sl.head_norm_fwd(q, k, w, w, lay, heads, rot, out=out)
    dw = torch.ones(16, device="cuda")
    for out in ({"dq": k}, {"dq": da}, {"dk": y}, {"dq": z, "dk": z}, {"dwq": dw, "dwk": dw}, {"dwq": w}):
        with pytest.raises(E, match="may not share memory"):
            sl.head_norm_bwd(q, k, w, w, lay, heads, y, da, rot, out=out)
    p = sl.DiffAttnParams({m: torch.ones(16, device="cuda") for m in sl.DiffAttnParams.NAMES}, heads)
    buf = sl.DiffAttnWorkspace(p, lay, torch.float32, "cuda")
    with pytest.raises(E, match="may not share memory"):
        sl.diff_attn_fwd(p, q, k, v, lay, buf=buf, out=part)
    for out in ({"dq": part}, {"dv": y}, {"dlq1": dw, "dlk2": dw}, {"dlq1": p.t["lk1"]},
                {"dk": buf.saved[:n * 4].view(torch.float32).view(6, 32)}):
        with pytest.raises(E, match="may not share memory"):
            sl.diff_attn_bwd(p, q, k, v, y, lay, buf, da, out=out)
    torch.cuda.synchronize()
    assert torch.equal(flat, before)
    # in place, and results beside each other, are as before
    ref = sl.head_norm_bwd(q, k, w, w, lay, heads, y, da, rot)
    for over in (("dq_out", "dk_out"), ("q", "k")):
        t = {"q": q.clone(), "k": k.clone(), "dq_out": y.clone(), "dk_out": da.clone()}
        g = sl.head_norm_bwd(t["q"], t["k"], w, w, lay, heads, t["dq_out"], t["dk_out"], rot,
                             out={"dq": t[over[0]], "dk": t[over[1]]})
        for m in ref:
            assert torch.equal(ref[m], g[m]), m


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(3, 1, 8, 4, 64, True, None), (2, 1, 6, 2, 128, False, None), (4, 9, 4, 2, 40, False, [1, 9, 0, 1]),
                                  (3, 70, 8, 2, 96, True, [70, 1, 33]), (6, 140, 32, 32, 128, True, None)],
                         ids=lambda c: "x".join(map(str, c[:6])))
def test_rows_with_a_single_key(case, dt):
    """The weight of a single key is 1 whatever its score: the first row of a causal
    sequence, and a sequence of one row, have no gradient to their scores at all."""
    sl = _sl()
    B, Ls, hq, hkv, hd, causal, lens = case
    x, lv = _diff_inputs(case, dt, seed=14)
    _, d, _, a, g, _ = _run_diff(sl, case, dt, x, lv)
    _check_diff(case, dt, x, lv, a, g)
    for b, n in enumerate(lens or [Ls] * B):
        if n and (causal or n == 1):
            assert not g["dq"][b * Ls].any()
        if n == 1:
            assert not g["dk"][b * Ls].any() and g["dv"][b * Ls].any()


SHORT = [  # batch, seq, hq, hkv, hd, causal, lens: at most 256 rows, every width, 64- and 128-row kernels
    (2, 1, 48, 16, 128, False, None),
    (4, 2, 8, 4, 32, True, [2, 1, 2, 2]),
    (1, 3, 2, 2, 80, True, None),
    (8, 8, 32, 8, 128, True, None),
    (7, 5, 4, 4, 128, False, [5, 4, 3, 2, 1, 0, 5]),
    (1, 33, 6, 2, 16, False, None),
    (1, 89, 8, 4, 96, True, None),
    (6, 140, 32, 32, 64, False, [140, 0, 129, 1, 64, 97]),
    (6, 140, 32, 32, 128, True, None),
    (5, 256, 24, 8, 32, True, None),
    (3, 256, 24, 8, 96, False, [256, 255, 97]),
    (2, 255, 6, 2, 128, False, None),
]


@pytest.mark.parametrize("case", SHORT, ids=lambda c: "x".join(map(str, c[:6])))
def test_bf16_products_of_short_sequences_keep_16_bits(case):
    """Up to 256 rows the weights and the score gradients enter their products as the
    sum of two bf16 values, half a step of a half step off (2^-16), O_2 is stored as
    16-bit integers of its row's largest value and O's rounding as 8-bit ones of the
    largest rounding (2^-8 of O): both within 2^-15.  The results' own rounding comes
    on top."""
    sl = _sl()
    B, Ls, hq, hkv, hd, causal, lens = case
    x, lv = _diff_inputs(case, "bf16", seed=17)
    _, _, _, a, g, _ = _run_diff(sl, case, "bf16", x, lv)
    ref = O.diff_attention(x["q"], x["k"], x["v"], lv, 0.6, B, (hq, hkv, hd), float(np.float32(hd ** -0.5)), causal,
                           lens, x["da"], rnd=2.0 ** -16, stored=2.0 ** -15)
    for n, got in [("a", a)] + sorted(g.items()):
        half = U32 if n.startswith("dl") else HALF["bf16"]
        _within(got, ref[n], half * np.abs(ref[n]) + ref["bound"][n] * (1 + half) + 1e-30, n)


@pytest.mark.parametrize("hd,causal,L", [(64, True, 300), (128, False, 270), (24, True, 290), (96, False, 300)])
def test_diff_attention_longer_scores_that_outgrow_the_first_tile(hd, causal, L):
    test_diff_attention_scores_that_outgrow_the_first_tile(hd, causal, L)
