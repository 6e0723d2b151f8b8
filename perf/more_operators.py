"""Cases of the operators around a model's sparse layers: the token embedding,
the norm of whole rows with the residual sum, and distillation from a teacher's
top logits, forward and backward.

Each case is a dict of plain values.  ``prepare`` makes its inputs from a seed,
``run`` makes one pass through the operator: in its plain form (elementary torch
operations in 32 bits), or, where ``own`` is true, through the package's entry
points.  ``exact`` is the operator's definition in 64 bits.

Tokens are packed as batch * seq rows.
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
        # ---- token embedding ---------------------------------------------------
        # one new token in each of eight conversations
        dict(name="embed_tokens", op="embed", type="bf16", grad="f32", batch=8, seq=1, vocab=32000, width=4096,
             scale=1.0, pad="none", train=False),
        # LLaMA2-7B: a training step's lookup and the table's fp32 gradient
        dict(name="embed_train", op="embed", type="bf16", grad="f32", batch=2, seq=1024, vocab=32000, width=4096,
             scale=1.0, pad="none", train=True),
        # an odd vocabulary and width in fp32, rows scaled by the root of the width, rows without a token
        dict(name="embed_odd_f32", op="embed", type="f32", grad="f32", batch=3, seq=333, vocab=50021, width=1000,
             scale=math.sqrt(1000.0), pad="absent", train=True),
        # LLaMA3-8B: eight long sequences, a quarter of the rows one padding token, bf16 gradient
        dict(name="embed_long", op="embed", type="bf16", grad="bf16", batch=8, seq=4096, vocab=128256, width=4096,
             scale=1.0, pad="token", train=True),
        # ---- norm of whole rows ------------------------------------------------
        # one token in each of four sequences
        dict(name="norm_tokens", op="norm", type="bf16", batch=4, seq=1, width=4096, centered=True, bias=True,
             residual=True, train=False),
        # a training step of a layer of LLaMA2-7B's width: residual sum and layer norm, forward and backward
        dict(name="norm_train", op="norm", type="bf16", batch=2, seq=1024, width=4096, centered=True, bias=True,
             residual=True, train=True),
        # odd lengths and width, no residual, fp32
        dict(name="norm_odd_f32", op="norm", type="f32", batch=3, seq=211, width=1000, centered=True, bias=True,
             residual=False, train=True),
        # the LLaMA layers' own norm (uncentred) over two long sequences
        dict(name="norm_long", op="norm", type="bf16", batch=2, seq=8192, width=5120, centered=False, bias=False,
             residual=True, train=True),
        # ---- distillation ------------------------------------------------------
        # a small fp32 head, loss then gradient
        dict(name="distill_small_f32", op="distill", type="f32", batch=2, seq=16, ctx=0, vocab=1003, top=8,
             temperature=1.0, hard=0.0, ragged=False, fused=False),
        # the LLaMA2-7B step of 4 x 512 tokens, 128 output tokens a sequence, mixed with hard labels
        dict(name="distill_train", op="distill", type="bf16", batch=4, seq=512, ctx=384, vocab=32000, top=64,
             temperature=2.0, hard=0.5, ragged=False, fused=True),
        # an odd vocabulary, teacher sets and prompts of differing length, loss then gradient
        dict(name="distill_odd", op="distill", type="bf16", batch=3, seq=333, ctx=100, vocab=50021, top=20,
             temperature=1.5, hard=0.0, ragged=True, fused=False),
        # LLaMA3-8B: one long sequence, every token an output
        dict(name="distill_long", op="distill", type="bf16", batch=1, seq=4096, ctx=0, vocab=128256, top=128,
             temperature=1.0, hard=0.1, ragged=False, fused=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {op: max(work(c)["bytes"] for c in listed() if c["op"] == op) for op in ("embed", "norm", "distill")}
    while True:
        c = dict(op=rng.choice(["embed", "norm", "distill"]), type=rng.choice(["bf16", "bf16", "f32"]),
                 batch=_log_int(rng, 1, 16), seq=_log_int(rng, 1, 8192))
        if c["op"] == "distill":
            c["ctx"] = rng.choice([0, c["seq"] // 2, c["seq"] * 3 // 4])
            c["vocab"] = _log_int(rng, 1000, 131072)
            c["top"] = _log_int(rng, 1, 128)
            c["temperature"] = rng.choice([0.5, 1.0, 1.5, 2.0, 4.0])
            c["hard"] = rng.choice([0.0, 0.0, 0.1, 0.5, 1.0])
            c["ragged"], c["fused"] = rng.random() < 0.4, rng.random() < 0.5
        elif c["op"] == "embed":
            c["grad"] = rng.choice(["f32", "bf16"]) if c["type"] == "bf16" else "f32"
            c["vocab"], c["width"] = _log_int(rng, 1000, 131072), 8 * _log_int(rng, 8, 1024)
            c["scale"] = rng.choice([1.0, math.sqrt(c["width"])])
            c["pad"], c["train"] = rng.choice(["none", "token", "absent"]), rng.random() < 0.75
        else:
            c["width"] = 8 * _log_int(rng, 8, 2048)
            c["centered"] = rng.random() < 0.6
            c["bias"] = c["centered"] and rng.random() < 0.7
            c["residual"], c["train"] = rng.random() < 0.6, rng.random() < 0.75
        if work(c)["bytes"] <= top[c["op"]]:
            return c


# ---------------------------------------------------------------------------
# what a pass cannot do without
def _ctx(case):
    """Context rows of each sequence: no loss there.  Prompts of a ragged batch differ."""
    ctx, L = case["ctx"], case["seq"]
    return [max(0, ctx - (ctx * b) // (2 * case["batch"])) if case["ragged"] else ctx for b in range(case["batch"])]


def work(case):
    T, es = case["batch"] * case["seq"], 2 if case["type"] == "bf16" else 4
    if case["op"] == "embed":
        n, gs = T * case["width"], 2 if case["grad"] == "bf16" else 4
        # lookup: rows read and written; gradient: rows read, the table written
        back = n * es + case["vocab"] * case["width"] * gs if case["train"] else 0
        return {"bytes": 2 * n * es + 4 * T + back, "flops": n * (2 if case["train"] else 1)}
    if case["op"] == "norm":
        n = T * case["width"]
        rows = 4 if case["residual"] else 2                     # x, y; the other summand and the sum
        if case["train"]:
            rows += 4 if case["residual"] else 3                # the sum, dy, dx; the sum's other gradient
        vec = case["width"] * 4 * (1 + case["bias"]) * (2 if case["train"] else 1)
        return {"bytes": rows * n * es + vec, "flops": n * (18 if case["train"] else 7)}
    out = T - sum(_ctx(case))
    # the output rows' logits read once, every row's gradient written once
    return {"bytes": (out + T) * case["vocab"] * es + T * (8 * case["top"] + 12),
            "flops": out * case["vocab"] * (12 if 0.0 < case["hard"] < 1.0 and case["temperature"] != 1.0 else 7)}


# ---------------------------------------------------------------------------
# inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1009 + salt)
    return g


def _token_ids(case, g):
    """Tokens as text has them: the n-th most frequent about 1 / n as often as
    the first, scattered over the vocabulary; the end of a padded batch's later
    sequences is one padding token, or no token at all."""
    B, L, V = case["batch"], case["seq"], case["vocab"]
    u = torch.rand(B * L, generator=g, device=DEV, dtype=torch.float64)
    rank = ((V + 1.0) ** u - 1.0).floor().to(torch.int64).clamp_(0, V - 1)
    ids = (rank * 7919 + 13) % V
    if case["pad"] != "none":
        b = torch.arange(B, device=DEV)[:, None]
        short = torch.arange(L, device=DEV)[None, :] >= L - (L * b) // (2 * B)
        ids = torch.where(short.reshape(-1), 2 if case["pad"] == "token" else -1, ids)
    return ids.to(torch.int32)


def _inputs(case, seed):
    g = _gen(seed, 11)
    dt, T = TYPES[case["type"]], case["batch"] * case["seq"]
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    if case["op"] == "embed":
        V, D = case["vocab"], case["width"]
        t = {"E": (0.02 * rn(V, D)).to(dt), "ids": _token_ids(case, g)}
        if case["train"]:
            t["dY"] = rn(T, D).to(dt)
        return t
    if case["op"] == "norm":
        D = case["width"]
        # a residual stream: every row its own size and offset, some features far larger than the rest
        big = torch.ones(D, device=DEV)
        big[::97] = 12.0
        t = {"x": ((rn(T, D) * big + 0.3) * torch.exp(0.5 * rn(T, 1))).to(dt)}
        t["r"] = (0.5 * rn(T, D)).to(dt) if case["residual"] else None
        t["w"] = 1.0 + 0.2 * rn(D)
        t["b"] = 0.1 * rn(D) if case["bias"] else None
        if case["train"]:
            t["dy"] = rn(T, D).to(dt)
            t["dh"] = rn(T, D).to(dt) if case["residual"] else None
        return t
    V, K = case["vocab"], min(case["top"], case["vocab"])
    z = 2.0 * rn(T, V)
    # the teacher's entries: distinct places, falling values, the student near them
    k = torch.arange(K, device=DEV)
    ids = (torch.randint(0, V, (T, 1), generator=g, device=DEV) + k * (97 if V % 97 else 89)) % V
    tl = 12.0 - 1.5 * torch.log1p(k.float()) + 0.3 * rn(T, K)
    z.scatter_(1, ids, tl + 1.5 * rn(T, K))
    if case["ragged"]:
        ids = torch.where(k < torch.randint(0, K + 1, (T, 1), generator=g, device=DEV), ids, -1)
    label = torch.where(torch.rand(T, generator=g, device=DEV) < 0.7, ids[:, 0],
                        torch.randint(-V // 20, V, (T,), generator=g, device=DEV))
    w = (0.5 + torch.rand(T, generator=g, device=DEV)) / T
    return {"z": z.to(dt), "ids": ids.to(torch.int32), "tl": tl, "label": label.clamp(min=-1).to(torch.int32), "w": w}


EPS = 1e-5


def prepare(case, seed):
    st = {"case": case, "t": _inputs(case, seed)}
    if not own:
        return st
    import contextual_sparsity_lora_svd_amd as sl
    t, B, L = st["t"], case["batch"], case["seq"]
    st["sl"] = sl
    st["layout"] = sl.Layout(_ctx(case) if case["op"] == "distill" else [0] * B, L)
    if case["op"] == "distill":
        st["p"] = sl.DistillTargets(t["ids"], t["tl"], t["label"], temperature=case["temperature"], hard=case["hard"])
    elif case["train"] and case["op"] == "embed":
        st["buf"] = sl.EmbedWorkspace(st["layout"], case["width"], t["E"].device)
    elif case["train"]:
        st["buf"] = sl.LayerNormWorkspace(st["layout"], case["width"], t["x"].device)
    return st


# ---------------------------------------------------------------------------
# plain forms, 32 bits
def _plain_embed(case, t):
    V, dt, s = case["vocab"], TYPES[case["type"]], case["scale"]
    is_token = ((t["ids"] >= 0) & (t["ids"] < V))[:, None]
    ids = t["ids"].long().clamp(0, V - 1)
    Y = torch.where(is_token, t["E"][ids].float() * s, 0.0).to(dt)
    if not case["train"]:
        return [Y]
    dE = torch.zeros(V, case["width"], device=DEV)
    dE.index_add_(0, ids, torch.where(is_token, t["dY"].float() * s, 0.0))
    return [Y, dE.to(TYPES[case["grad"]])]


def _plain_norm(case, t):
    dt = TYPES[case["type"]]
    h = t["x"] if t["r"] is None else (t["x"].float() + t["r"].float()).to(dt)
    d = h.float()
    if case["centered"]:
        d = d - d.mean(-1, keepdim=True)
    s = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    u = d * s
    y = u * t["w"]
    if t["b"] is not None:
        y = y + t["b"]
    out = [y.to(dt)] + ([h] if t["r"] is not None else [])
    if not case["train"]:
        return out
    dy = t["dy"].float()
    g = dy * t["w"]
    dx = g - u * (g * u).mean(-1, keepdim=True)
    if case["centered"]:
        dx = dx - g.mean(-1, keepdim=True)
    dx = dx * s
    if t["dh"] is not None:
        dx = dx + t["dh"].float()
    return out + [dx.to(dt), (dy * u).sum(0)] + ([dy.sum(0)] if t["b"] is not None else [])


def _rows_with_loss(case):
    ctx = torch.tensor(_ctx(case), device=DEV)[:, None]
    return (torch.arange(case["seq"], device=DEV)[None, :] >= ctx).reshape(-1)


def _plain_distill(case, t):
    V, dt, tau, hard = case["vocab"], TYPES[case["type"]], case["temperature"], case["hard"]
    keep = torch.nonzero(_rows_with_loss(case)).squeeze(1)
    loss, dz = torch.zeros(t["z"].shape[0], device=DEV), torch.zeros_like(t["z"])
    z, w = t["z"][keep].float(), t["w"][keep, None]
    z = z - z.amax(-1, keepdim=True)
    grad = torch.zeros_like(z)
    rows = torch.zeros(z.shape[0], device=DEV)
    if hard < 1.0:
        given = (t["ids"][keep] >= 0) & (t["ids"][keep] < V)
        ids = t["ids"][keep].long().clamp(0, V - 1)
        tl = torch.where(given, t["tl"][keep] / tau, float("-inf"))
        some = given.any(-1, keepdim=True)
        top = torch.where(some, tl.amax(-1, keepdim=True), 0.0)
        e = torch.exp(tl - top)
        es = torch.where(some, e.sum(-1, keepdim=True), 1.0)
        p = e / es
        q = torch.exp(z / tau)
        S = q.sum(-1, keepdim=True)
        logq = z.gather(1, ids) / tau - torch.log(S)
        logp = tl - top - torch.log(es)
        rows += (1.0 - hard) * tau * tau * torch.where(p > 0, p * (logp - logq), 0.0).sum(-1)
        q = q / S * some
        q.scatter_add_(1, ids, -p)
        grad += (1.0 - hard) * tau * q
    if hard > 0.0:
        label = t["label"][keep].long()[:, None]
        some = (label >= 0) & (label < V)
        q = torch.exp(z)
        S = q.sum(-1, keepdim=True)
        label = label.clamp(0, V - 1)
        rows += hard * torch.where(some, torch.log(S) - z.gather(1, label), 0.0).squeeze(1)
        q = q / S * some
        q.scatter_add_(1, label, -some.float())
        grad += hard * q
    loss[keep] = rows
    dz[keep] = (grad * w).to(dt)
    return [loss, dz]


# ---------------------------------------------------------------------------
def run(state):
    case, t = state["case"], state["t"]
    if not own:
        return {"embed": _plain_embed, "norm": _plain_norm, "distill": _plain_distill}[case["op"]](case, t)
    sl, lay = state["sl"], state["layout"]
    if case["op"] == "embed":
        out = [sl.embed_fwd(t["E"], t["ids"], lay, scale=case["scale"])]
        if case["train"]:
            out.append(sl.embed_bwd(t["ids"], t["dY"], lay, case["vocab"], scale=case["scale"],
                                    grad_dtype=TYPES[case["grad"]], buf=state["buf"]))
        return out
    if case["op"] == "norm":
        y, h, stats = sl.layer_norm_fwd(t["x"], t["w"], t["b"], lay, eps=EPS, centered=case["centered"],
                                        residual=t["r"], want_stats=case["train"])
        out = [y] + ([h] if t["r"] is not None else [])
        if case["train"]:
            g = sl.layer_norm_bwd(h, t["w"], stats, lay, t["dy"], dh=t["dh"], centered=case["centered"],
                                  bias=case["bias"], buf=state["buf"])
            out += [g["dx"], g["dw"]] + ([g["db"]] if case["bias"] else [])
        return out
    if case["fused"]:
        return list(sl.distill_step(state["p"], t["z"], lay, dloss=t["w"]))
    loss, stats = sl.distill_fwd(state["p"], t["z"], lay)
    return [loss, sl.distill_bwd(state["p"], t["z"], stats, lay, dloss=t["w"])]


# ---------------------------------------------------------------------------
# definitions in 64 bits
def exact(case, seed):
    t = _inputs(case, seed)
    return {"embed": _exact_embed, "norm": _exact_norm, "distill": _exact_distill}[case["op"]](case, t)


def _exact_embed(case, t):
    """Lookup row by row; the gradient as sums over runs of the sorted tokens."""
    V = case["vocab"]
    good = torch.nonzero((t["ids"] >= 0) & (t["ids"] < V)).squeeze(1)
    tok = t["ids"][good].long()
    Y = torch.zeros(t["ids"].shape[0], case["width"], dtype=torch.float64, device=DEV)
    Y[good] = t["E"][tok].double() * case["scale"]
    if not case["train"]:
        return [Y]
    order = torch.argsort(tok, stable=True)
    ahead = torch.cat((torch.zeros(1, case["width"], dtype=torch.float64, device=DEV),
                       torch.cumsum(t["dY"][good[order]].double(), 0)))
    count = torch.bincount(tok, minlength=V)
    end = torch.cumsum(count, 0)
    return [Y, (ahead[end] - ahead[end - count]) * case["scale"]]


def _exact_norm(case, t):
    """Rows as vectors: a layer norm takes the part along (1, ..., 1) out of a
    row and divides by its length; so does its derivative."""
    dt, D = TYPES[case["type"]], case["width"]
    x = t["x"].double()
    full = x if t["r"] is None else x + t["r"].double()
    h = full.to(dt).double()                          # the sum as it is kept
    c = h - h.sum(-1, keepdim=True) / D if case["centered"] else h
    size = ((c.norm(dim=-1, keepdim=True) ** 2) / D + EPS).sqrt()
    w = t["w"].double()
    y = c / size * w
    if t["b"] is not None:
        y += t["b"].double()
    out = [y] + ([full] if t["r"] is not None else [])
    if not case["train"]:
        return out
    dy = t["dy"].double()
    gw = dy * w
    if case["centered"]:
        gw = gw - gw.sum(-1, keepdim=True) / D
    dx = gw / size - c * ((gw * c).sum(-1, keepdim=True) / (D * size ** 3))
    if t["dh"] is not None:
        dx += t["dh"].double()
    return out + [dx, (dy * (c / size)).sum(0)] + ([dy.sum(0)] if t["b"] is not None else [])


def _exact_distill(case, t):
    """The teacher's and the label's distributions spread over the vocabulary;
    cross entropies less the teacher's entropy; gradients softmax - target."""
    V, tau, hard = case["vocab"], case["temperature"], case["hard"]
    T = t["z"].shape[0]
    keep = torch.nonzero(_rows_with_loss(case)).squeeze(1)
    loss, dz = (torch.zeros(*s, dtype=torch.float64, device=DEV) for s in ((T,), (T, V)))
    z, ids, tl = t["z"][keep].double(), t["ids"][keep].long(), t["tl"][keep].double()
    rows, grad = torch.zeros(len(keep), dtype=torch.float64, device=DEV), torch.zeros_like(z)
    if hard < 1.0:
        weight = torch.where((ids >= 0) & (ids < V), torch.exp((tl - tl.max()) / tau), 0.0)
        mass = weight.sum(1, keepdim=True)
        p = weight / torch.where(mass > 0, mass, 1.0)
        target = torch.zeros_like(z).scatter_add_(1, ids.clamp(0, V - 1), p)
        logq = torch.log_softmax(z / tau, 1)
        entropy = -torch.special.xlogy(p, p).sum(1)
        rows += (1 - hard) * tau ** 2 * (-(target * logq).sum(1) - entropy)
        grad += (1 - hard) * tau * (logq.exp_() * (mass > 0) - target)
        del logq, target
    if hard > 0.0:
        label = t["label"][keep].long()
        has = torch.nonzero((label >= 0) & (label < V)).squeeze(1)
        logq = torch.log_softmax(z[has], 1)
        rows[has] -= hard * logq[torch.arange(len(has), device=DEV), label[has]]
        q = logq.exp_()
        q[torch.arange(len(has), device=DEV), label[has]] -= 1.0
        grad[has] += hard * q
    loss[keep] = rows
    dz[keep] = grad * t["w"][keep, None].double()
    return [loss, dz]
