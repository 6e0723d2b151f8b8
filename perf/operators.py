"""Cases of the operators that run between the q/k/v projections and the
attention output projection: rotary positions, per-head norms with the rotation,
and differential attention, forward and backward.

Each case is a dict of plain values.  ``prepare`` makes its inputs from a seed,
``run`` makes one pass through the operator: in its plain form (elementary torch
operations in 32 bits, angles in 64), or, where ``own`` is true, through the
package's entry points.  ``exact`` is the operator's definition in 64 bits.

Tokens are packed as batch * seq_len rows; q is [T, Hq * hd], k and v are
[T, Hkv * hd], as the q/k/v projections write them.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# the cases
def listed():
    return [
        # ---- rotary positions -------------------------------------------------
        # one new token in each of eight conversations, far into a long context
        dict(name="rotary_tokens", op="rotary", type="bf16", batch=8, seq=1, hq=32, hkv=8, hd=128, rot=128,
             interleaved=False, scaling="wavelength", factor=8.0, original=8192, positions="far", train=False),
        # LLaMA2-7B attention layer, a training step's forward and backward
        dict(name="rotary_train", op="rotary", type="bf16", batch=2, seq=1024, hq=32, hkv=32, hd=128, rot=128,
             interleaved=False, scaling="none", factor=1.0, original=4096, positions="row", train=True),
        # a ragged batch of short sequences, interleaved pairs on half of an 80-wide head
        dict(name="rotary_odd", op="rotary", type="bf16", batch=3, seq=333, hq=10, hkv=5, hd=80, rot=40,
             interleaved=True, scaling="linear", factor=4.0, original=2048, positions="packed", train=True),
        # LLaMA3-8B long-context layer in fp32, stretched eightfold
        dict(name="rotary_long_f32", op="rotary", type="f32", batch=1, seq=4096, hq=32, hkv=8, hd=128, rot=128,
             interleaved=False, scaling="yarn", factor=8.0, original=4096, positions="row", train=True),
        # ---- head norms with the rotation -------------------------------------
        # one token in each of four sequences
        dict(name="norm_tokens", op="norm", type="bf16", batch=4, seq=1, hq=32, hkv=8, hd=128, rot=128,
             interleaved=False, scaling="none", factor=1.0, original=4096, positions="far", train=False),
        # the LLaMA2-7B attention layer's forward and backward with the weight gradients
        dict(name="norm_train", op="norm", type="bf16", batch=2, seq=1024, hq=32, hkv=32, hd=128, rot=128,
             interleaved=False, scaling="none", factor=1.0, original=4096, positions="row", train=True),
        # odd lengths, a quarter of the head rotated in interleaved pairs, fp32
        dict(name="norm_odd_f32", op="norm", type="f32", batch=3, seq=211, hq=12, hkv=3, hd=96, rot=24,
             interleaved=True, scaling="base", factor=4.0, original=2048, positions="packed", train=True),
        # the LLaMA3-8B layer over two long sequences
        dict(name="norm_long", op="norm", type="bf16", batch=2, seq=8192, hq=32, hkv=8, hd=128, rot=128,
             interleaved=False, scaling="wavelength", factor=8.0, original=8192, positions="row", train=True),
        # ---- differential attention -------------------------------------------
        # a small fp32 layer
        dict(name="diff_small_f32", op="diff", type="f32", batch=2, seq=64, hq=8, hkv=4, hd=32, causal=True,
             ragged=False, train=True),
        # the LLaMA2-7B attention layer's forward and backward
        dict(name="diff_train", op="diff", type="bf16", batch=2, seq=1024, hq=32, hkv=32, hd=128, causal=True,
             ragged=False, train=True),
        # a padded batch of odd lengths that attend both ways, one sequence empty
        dict(name="diff_ragged", op="diff", type="bf16", batch=4, seq=777, hq=12, hkv=4, hd=64, causal=False,
             ragged=True, train=True),
        # the LLaMA3-8B long-context layer, one 4096-token sequence, eight shared kv heads
        dict(name="diff_long", op="diff", type="bf16", batch=1, seq=4096, hq=32, hkv=8, hd=128, causal=True,
             ragged=False, train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = max(work(c)["bytes"] for c in listed() if c["op"] != "diff")
    top_flops = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["rotary", "norm", "diff"])
        c = dict(op=op, type=rng.choice(["bf16", "bf16", "f32"]), batch=_log_int(rng, 1, 16),
                 seq=_log_int(rng, 1, 8192), train=rng.random() < 0.75)
        groups = rng.choice([1, 1, 2, 3, 4])
        if op == "diff":
            c["hd"] = rng.choice([16, 32, 64, 64, 80, 96, 128, 128])
            c["hkv"] = 2 * rng.choice([1, 2, 3, 4, 8])
            c["hq"] = c["hkv"] * groups
            c["causal"] = rng.random() < 0.7
            c["ragged"] = rng.random() < 0.4
        else:
            c["hd"] = rng.choice([32, 64, 80, 96, 128, 128, 256])
            c["rot"] = rng.choice([c["hd"], c["hd"], c["hd"] // 2, c["hd"] // 4])
            c["hkv"] = rng.choice([1, 2, 3, 5, 8, 16])
            c["hq"] = c["hkv"] * groups
            c["interleaved"] = rng.random() < 0.4
            c["scaling"] = rng.choice(["none", "linear", "base", "wavelength", "yarn"])
            c["factor"] = 1.0 if c["scaling"] == "none" else float(rng.choice([2, 4, 8, 16]))
            c["original"] = rng.choice([2048, 4096, 8192])
            c["positions"] = rng.choice(["row", "packed", "far"])
        w = work(c)
        if op == "diff":
            # the fp32 products run at a sixteenth of the bf16 rate
            if w["flops"] * (16 if c["type"] == "f32" else 1) <= top_flops and c["batch"] * c["seq"] <= 16384:
                return c
        elif w["bytes"] <= top:
            return c


# ---------------------------------------------------------------------------
# what a pass cannot do without
def _lens(case):
    """Valid rows of each sequence (the rest is padding); the last but one of
    a ragged batch of three or more is empty."""
    B, L = case["batch"], case["seq"]
    if not case.get("ragged"):
        return [L] * B
    lens = [max(1, L - (L * b) // (B + 1)) for b in range(B)]
    if B >= 3:
        lens[-2] = 0
    return lens


def work(case):
    T, es = case["batch"] * case["seq"], 2 if case["type"] == "bf16" else 4
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    nq, nkv = T * hq * hd, T * hkv * hd
    if case["op"] == "rotary":
        passes = 2 if case["train"] else 1
        pos = 4 * T if case["positions"] != "row" else 0
        return {"bytes": passes * 2 * (nq + nkv) * es + pos,
                "flops": passes * 3 * T * (hq + hkv) * case["rot"]}
    if case["op"] == "norm":
        rows = 5 if case["train"] else 2          # x, y, then x's second reading, dy, dx
        pos = 4 * T if case["positions"] != "row" else 0
        return {"bytes": rows * (nq + nkv) * es + 2 * 4 * hd * (2 if case["train"] else 1) + pos,
                "flops": (nq + nkv) * (16 if case["train"] else 5)}
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _lens(case))
    valid = sum(_lens(case))
    # per (query, key) and head pair: two score products over hd, two value
    # products over 2 hd; backward: the gradient of the weights (2 hd), of the
    # values (2 hd), and two each of the queries and the keys (hd)
    flops = pairs * (hq // 2) * (28 if case["train"] else 12) * hd
    nb = valid * hd * es * ((2 * hq + 2 * hkv) + ((2 * hq + 2 * hkv) if case["train"] else 0))
    return {"bytes": max(nb, 1), "flops": max(flops, 1)}


# ---------------------------------------------------------------------------
# inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1009 + salt)
    return g


def _rows(g, T, heads, hd, dt, shared=0.3):
    """Head rows with a component that every token shares and one feature in
    sixteen larger than the rest, as projections write them."""
    x = torch.randn(T, heads, hd, generator=g, device=DEV)
    x += shared * torch.randn(1, heads, hd, generator=g, device=DEV)
    s = torch.ones(hd, device=DEV)
    s[::16] = 2.0
    return (x * s).reshape(T, heads * hd).to(dt)


def _positions(case, g):
    T = case["batch"] * case["seq"]
    if case["positions"] == "row":
        return None
    if case["positions"] == "far":
        start = torch.randint(0, 1 << 20, (case["batch"], 1), generator=g, device=DEV)
        return (start + torch.arange(case["seq"], device=DEV)).reshape(T).to(torch.int32)
    # documents packed one behind the other: the position starts over inside a row
    cut = torch.randint(1, max(2, case["seq"]), (case["batch"], 1), generator=g, device=DEV)
    r = torch.arange(case["seq"], device=DEV)[None, :]
    return torch.where(r < cut, r, r - cut).reshape(T).to(torch.int32).contiguous()


def _inputs(case, seed):
    g = _gen(seed, 7)
    dt = TYPES[case["type"]]
    T, hq, hkv, hd = case["batch"] * case["seq"], case["hq"], case["hkv"], case["hd"]
    t = {"q": _rows(g, T, hq, hd, dt), "k": _rows(g, T, hkv, hd, dt)}
    if case["op"] == "diff":
        # the scores' spread is about one, as after a norm of the heads
        t["q"], t["k"] = (t["q"].float() * 0.9).to(dt), (t["k"].float() * 0.9).to(dt)
        t["v"] = _rows(g, T, hkv, hd, dt)
        for n in ("lq1", "lk1", "lq2", "lk2"):
            t[n] = 0.1 * torch.randn(hd, generator=g, device=DEV)
        if case["train"]:
            t["da"] = torch.randn(T, hq * hd, generator=g, device=DEV).to(dt)
        return t
    t["pos"] = _positions(case, g)
    if case["train"]:
        t["dq"] = torch.randn(T, hq * hd, generator=g, device=DEV).to(dt)
        t["dk"] = torch.randn(T, hkv * hd, generator=g, device=DEV).to(dt)
    if case["op"] == "norm":
        t["wq"] = 1.0 + 0.2 * torch.randn(hd, generator=g, device=DEV)
        t["wk"] = 1.0 + 0.2 * torch.randn(hd, generator=g, device=DEV)
    return t


BASE, EPS, LAMBDA_INIT = 10000.0, 1e-6, 0.55


def prepare(case, seed):
    st = {"case": case, "t": _inputs(case, seed)}
    if not own:
        return st
    import contextual_sparsity_lora_svd_amd as sl
    st["sl"] = sl
    st["layout"] = sl.Layout([case["seq"]] * case["batch"], case["seq"])
    st["heads"] = (case["hq"], case["hkv"], case["hd"])
    t = st["t"]
    if case["op"] == "diff":
        st["p"] = sl.DiffAttnParams({n: t[n] for n in ("lq1", "lk1", "lq2", "lk2")}, st["heads"],
                                    lambda_init=LAMBDA_INIT, causal=case["causal"])
        st["buf"] = sl.DiffAttnWorkspace(st["p"], st["layout"], t["q"].dtype, t["q"].device,
                                         lens=_lens(case) if case["ragged"] else None)
    else:
        st["rot"] = sl.Rotary(case["rot"], base=BASE, interleaved=case["interleaved"], scaling=case["scaling"],
                              factor=case["factor"], original_len=case["original"], device=t["q"].device)
        if case["op"] == "norm" and case["train"]:
            st["buf"] = sl.HeadNormWorkspace(st["layout"], st["heads"], t["q"].device)
    return st


# ---------------------------------------------------------------------------
# angles: position * frequency, frequencies as the scaling asks
def _frequencies(case):
    rot, kind, s = case["rot"], case["scaling"], case["factor"]
    base = BASE * (s ** (rot / (rot - 2)) if kind == "base" and rot > 2 else 1.0)
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    amp = 1.0
    if kind == "linear":
        f = [x / s for x in f]
    elif kind == "wavelength":
        # turns within the original length: few -> stretched, many -> kept
        out = []
        for x in f:
            turns = case["original"] * x / (2 * math.pi)
            keep = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            out.append(x * keep + x / s * (1.0 - keep))
        f = out
    elif kind == "yarn":
        # a ramp over the pair index between 32 turns and one turn
        def index(turns):
            return rot * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
        span = max(hi - lo, 0.001)
        out = []
        for i, x in enumerate(f):
            stretch = min(max((i - lo) / span, 0.0), 1.0)
            out.append(x / s * stretch + x * (1.0 - stretch))
        f = out
        amp = 0.1 * math.log(s) + 1.0
    return torch.tensor(f, dtype=torch.float64, device=DEV), amp


def _cos_sin(case, pos, dt):
    T = case["batch"] * case["seq"]
    f, amp = _frequencies(case)
    if pos is None:
        pos = torch.arange(T, device=DEV) % case["seq"]
    ang = pos.double()[:, None] * f[None, :]
    return (torch.cos(ang) * amp).to(dt)[:, None, :], (torch.sin(ang) * amp).to(dt)[:, None, :]


def _rotate(x, cos, sin, case, sign):
    """x [T, H, hd]: its first rot values turned by the angles."""
    rot = case["rot"]
    h = x[..., :rot]
    if case["interleaved"]:
        a, b = h[..., 0::2], h[..., 1::2]
    else:
        a, b = h[..., :rot // 2], h[..., rot // 2:]
    ra, rb = a * cos - b * sin * sign, b * cos + a * sin * sign
    y = x.clone()
    if case["interleaved"]:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    return y


def _plain_positions(case, t, wide):
    dt = TYPES[case["type"]]
    cos, sin = _cos_sin(case, t["pos"], wide)
    hd, out = case["hd"], []

    def heads(x):
        return x.to(wide).view(x.shape[0], -1, hd)

    def flat(x, ref):
        y = x.reshape(ref.shape)
        return y if wide == torch.float64 else y.to(dt)

    if case["op"] == "rotary":
        for n in ("q", "k"):
            out.append(flat(_rotate(heads(t[n]), cos, sin, case, 1.0), t[n]))
        if case["train"]:
            for n, ref in (("dq", "q"), ("dk", "k")):
                out.append(flat(_rotate(heads(t[n]), cos, sin, case, -1.0), t[ref]))
        return out
    grads, wgrads = [], []
    for n in ("q", "k"):
        x, w = heads(t[n]), t["w" + n].to(wide)
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        out.append(flat(_rotate(x * r * w, cos, sin, case, 1.0), t[n]))
        if case["train"]:
            g = _rotate(heads(t["d" + n]), cos, sin, case, -1.0)
            h = g * w
            dx = r * (h - x * (r * r * (h * x).mean(-1, keepdim=True)))
            grads.append(flat(dx, t[n]))
            wgrads.append((g * x * r).sum((0, 1)))
    return out + grads + wgrads


# ---------------------------------------------------------------------------
# differential attention, one head pair at a time:
#   A = softmax(s q1 k1') - lambda softmax(s q2 k2'),  out = A v
# with lambda = exp(lq1.lk1) - exp(lq2.lk2) + lambda_init; the query heads 2h and
# 2h + 1 are a pair, so are the kv heads, and v's pair is one 2 hd wide value.
def _plain_diff(case, t, wide):
    B, L, hq, hkv, hd = case["batch"], case["seq"], case["hq"], case["hkv"], case["hd"]
    T, dt, dev = B * L, TYPES[case["type"]], t["q"].device
    e1 = torch.exp((t["lq1"].to(wide) * t["lk1"].to(wide)).sum())
    e2 = torch.exp((t["lq2"].to(wide) * t["lk2"].to(wide)).sum())
    lam = e1 - e2 + LAMBDA_INIT
    sc = 1.0 / math.sqrt(hd)
    groups = hq // hkv
    q, k, v = t["q"].view(B, L, hq, hd), t["k"].view(B, L, hkv, hd), t["v"].view(B, L, hkv // 2, 2 * hd)
    od = wide if wide == torch.float64 else dt
    a = torch.zeros(B, L, hq // 2, 2 * hd, dtype=od, device=dev)
    if case["train"]:
        da = t["da"].view(B, L, hq // 2, 2 * hd)
        dq = torch.zeros(B, L, hq, hd, dtype=od, device=dev)
        dk = torch.zeros(B, L, hkv, hd, dtype=wide, device=dev)
        dv = torch.zeros(B, L, hkv // 2, 2 * hd, dtype=wide, device=dev)
        dlam = torch.zeros((), dtype=torch.float64, device=dev)
    for b, n in enumerate(_lens(case)):
        if n == 0:
            continue
        hidden = None
        if case["causal"]:
            i = torch.arange(n, device=dev)
            hidden = i[None, :] > i[:, None]
        for h in range(hq // 2):
            g = h // groups
            vv = v[b, :n, g].to(wide)
            qs = [q[b, :n, 2 * h + m].to(wide) for m in (0, 1)]
            ks = [k[b, :n, 2 * g + m].to(wide) for m in (0, 1)]
            P = []
            for m in (0, 1):
                s = (qs[m] @ ks[m].t()) * sc
                if hidden is not None:
                    s.masked_fill_(hidden, float("-inf"))
                s = torch.exp_(s - s.amax(-1, keepdim=True))
                P.append(s / s.sum(-1, keepdim=True))
            A = P[0] - lam * P[1]
            a[b, :n, h] = (A @ vv).to(od)
            if not case["train"]:
                continue
            do = da[b, :n, h].to(wide)
            dv[b, :n, g] += A.t() @ do
            del A
            dP = do @ vv.t()
            for m, c in ((0, 1.0), (1, -lam)):
                row = (P[m] * dP).sum(-1, keepdim=True)
                if m == 1:
                    dlam -= row.sum(dtype=torch.float64)
                dS = P[m] * (dP - row) * (c * sc)
                dq[b, :n, 2 * h + m] = (dS @ ks[m]).to(od)
                dk[b, :n, 2 * g + m] += dS.t() @ qs[m]
    if not case["train"]:
        return [a.view(T, hq * hd)]
    dlam = dlam.to(wide)
    vec = [dlam * e1 * t["lk1"], dlam * e1 * t["lq1"], -dlam * e2 * t["lk2"], -dlam * e2 * t["lq2"]]
    return [a.view(T, hq * hd), dq.view(T, hq * hd), dk.to(od).view(T, hkv * hd),
            dv.to(od).view(T, hkv * hd)] + [x.to(wide) for x in vec]


# ---------------------------------------------------------------------------
def run(state):
    case, t = state["case"], state["t"]
    if not own:
        if case["op"] == "diff":
            return _plain_diff(case, t, torch.float32)
        return _plain_positions(case, t, torch.float32)
    sl, lay, heads = state["sl"], state["layout"], state["heads"]
    if case["op"] == "rotary":
        out = list(sl.rotary(t["q"], t["k"], lay, heads, state["rot"], pos=t["pos"]))
        if case["train"]:
            out += sl.rotary(t["dq"], t["dk"], lay, heads, state["rot"], pos=t["pos"], inverse=True)
        return out
    if case["op"] == "norm":
        out = list(sl.head_norm_fwd(t["q"], t["k"], t["wq"], t["wk"], lay, heads, rot=state["rot"], pos=t["pos"],
                                    eps=EPS))
        if case["train"]:
            g = sl.head_norm_bwd(t["q"], t["k"], t["wq"], t["wk"], lay, heads, t["dq"], t["dk"], rot=state["rot"],
                                 pos=t["pos"], eps=EPS, buf=state["buf"])
            out += [g["dq"], g["dk"], g["dwq"], g["dwk"]]
        return out
    a, buf = sl.diff_attn_fwd(state["p"], t["q"], t["k"], t["v"], lay, buf=state["buf"])
    if not case["train"]:
        return [a]
    g = sl.diff_attn_bwd(state["p"], t["q"], t["k"], t["v"], a, lay, buf, t["da"])
    return [a, g["dq"], g["dk"], g["dv"], g["dlq1"], g["dlk1"], g["dlq2"], g["dlk2"]]


def exact(case, seed):
    t = _inputs(case, seed)
    if case["op"] == "diff":
        return _exact_diff(case, t)
    return _exact_positions(case, t)


def _exact_positions(case, t):
    """Pairs as complex numbers: the rotation is a product with amp e^(i angle)."""
    B, L, hd, rot = case["batch"], case["seq"], case["hd"], case["rot"]
    f, amp = _frequencies(case)
    pos = torch.arange(L, device=DEV).repeat(B) if t["pos"] is None else t["pos"]
    turn = torch.polar(torch.full((B * L, rot // 2), amp, dtype=torch.float64, device=DEV),
                       torch.outer(pos.double(), f)).unsqueeze(1)

    def pairs(x):
        x = x.reshape(B * L, -1, hd)[..., :rot]
        if case["interleaved"]:
            return torch.view_as_complex(x.reshape(B * L, -1, rot // 2, 2).contiguous())
        return torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:].contiguous())

    def turned(x, conj):
        z = pairs(x) * (turn.conj() if conj else turn)
        z = torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat((z.real, z.imag), -1)
        return torch.cat((z, x.reshape(B * L, -1, hd)[..., rot:]), -1)

    if case["op"] == "rotary":
        names = [("q", False), ("k", False)] + ([("dq", True), ("dk", True)] if case["train"] else [])
        return [turned(t[n].double(), c).reshape(t[n].shape) for n, c in names]
    ys, dxs, dws = [], [], []
    for n in ("q", "k"):
        x = t[n].double().reshape(B * L, -1, hd)
        w = t["w" + n].double()
        rms = (x.square().sum(-1, keepdim=True) / hd + EPS).sqrt()
        u = x / rms
        ys.append(turned(u * w, False).reshape(t[n].shape))
        if case["train"]:
            g = turned(t["d" + n].double(), True)
            dws.append((g * u).flatten(0, 1).sum(0))
            gw = g * w
            # u has norm sqrt(hd) (up to eps): its derivative drops the part along u
            dxs.append(((gw - u * (gw * u).sum(-1, keepdim=True) / hd) / rms).reshape(t[n].shape))
    return ys + dxs + dws


def _exact_diff(case, t):
    """The scores' log-sum-exp first, then the weights; the gradient of a
    score is its weight times the gradient of the output along (value - mean
    value of its map)."""
    B, L, hq, hkv, hd = case["batch"], case["seq"], case["hq"], case["hkv"], case["hd"]
    D = {n: x.double() for n, x in t.items()}
    lam1, lam2 = torch.dot(D["lq1"], D["lk1"]).exp(), torch.dot(D["lq2"], D["lk2"]).exp()
    lam = lam1 - lam2 + LAMBDA_INIT
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=DEV)
    out, dq, dk, dv, dlam = z(B * L, hq * hd), z(B * L, hq * hd), z(B * L, hkv * hd), z(B * L, hkv * hd), z(())
    for b, n in enumerate(_lens(case)):
        rows = slice(b * L, b * L + n)
        if n == 0:
            continue
        future = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1) if case["causal"] else None
        for h in range(hq // 2):
            g = h * hkv // hq
            V = D["v"][rows, 2 * g * hd:2 * (g + 1) * hd]
            span = slice(2 * h * hd, 2 * (h + 1) * hd)
            maps, means = [], []
            for m in (0, 1):
                Q = D["q"][rows, (2 * h + m) * hd:(2 * h + m + 1) * hd]
                K = D["k"][rows, (2 * g + m) * hd:(2 * g + m + 1) * hd]
                S = torch.mm(Q, K.t()).div_(math.sqrt(hd))
                if future is not None:
                    S.masked_fill_(future, -math.inf)
                W = torch.exp_(S.sub_(torch.logsumexp(S, 1, keepdim=True)))
                maps.append((Q, K, W))
                means.append(torch.mm(W, V))
            out[rows, span] = means[0] - lam * means[1]
            if not case["train"]:
                continue
            G = D["da"][rows, span]
            dlam -= (G * means[1]).sum()
            along = torch.mm(G, V.t())
            for m, coef in ((0, 1.0), (1, -lam)):
                Q, K, W = maps[m]
                dv[rows, 2 * g * hd:2 * (g + 1) * hd] += coef * torch.mm(W.t(), G)
                E = W.mul_(along - (G * means[m]).sum(1, keepdim=True)).mul_(coef / math.sqrt(hd))
                dq[rows, (2 * h + m) * hd:(2 * h + m + 1) * hd] = torch.mm(E, K)
                dk[rows, (2 * g + m) * hd:(2 * g + m + 1) * hd] += torch.mm(E.t(), Q)
    if not case["train"]:
        return [out]
    return [out, dq, dk, dv, dlam * lam1 * D["lk1"], dlam * lam1 * D["lq1"], -dlam * lam2 * D["lk2"],
            -dlam * lam2 * D["lq2"]]
