"""The oracle of the operators around the layers against torch's own operations
in 64 bits and their autograd, and against differences."""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")


def test_embedding_and_its_gradient():
    rng = np.random.default_rng(0)
    E, ids = rng.standard_normal((11, 8)), np.array([3, 3, 0, -1, 10, 11, 3, 0])
    Y = O.embed(E, ids, 1.5)
    assert not Y[[3, 5]].any()
    w = torch.tensor(E, requires_grad=True)
    ok = [i for i in range(8) if 0 <= ids[i] < 11]
    y = torch.nn.functional.embedding(torch.tensor(ids[ok]), w) * 1.5
    np.testing.assert_allclose(Y[ok], y.detach().numpy(), rtol=1e-15)
    dY = rng.standard_normal((8, 8))
    (y * torch.tensor(dY[ok])).sum().backward()
    dE, mag, n = O.embed_backward(ids, dY, 11, 1.5)
    np.testing.assert_allclose(dE, w.grad.numpy(), rtol=1e-13, atol=1e-15)
    assert (mag >= np.abs(dE) - 1e-15).all() and n.tolist() == [2, 0, 0, 3, 0, 0, 0, 0, 0, 0, 1]


@pytest.mark.parametrize("centered", [True, False])
def test_layer_norm_and_its_gradient(centered):
    rng = np.random.default_rng(1)
    h, w, b = rng.standard_normal((5, 24)) + 3.0, rng.standard_normal(24), rng.standard_normal(24)
    dy, dh = rng.standard_normal((5, 24)), rng.standard_normal((5, 24))
    th, tw, tb = (torch.tensor(v, requires_grad=True) for v in (h, w, b))
    if centered:
        y = torch.nn.functional.layer_norm(th, (24,), tw, tb, 1e-3)
    else:
        y = torch.nn.functional.rms_norm(th, (24,), tw, 1e-3)
    ((y * torch.tensor(dy)).sum() + (th * torch.tensor(dh)).sum()).backward()
    np.testing.assert_allclose(O.layer_norm(h, w, b if centered else None, 1e-3, centered)[0], y.detach().numpy(),
                               rtol=1e-12, atol=1e-13)
    dx, dw, db, mx, mw, _ = O.layer_norm_backward(h, w, dy, dh, 1e-3, centered)
    np.testing.assert_allclose(dx, th.grad.numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-11, atol=1e-13)
    if centered:
        np.testing.assert_allclose(db, tb.grad.numpy(), rtol=1e-12)
    assert (mx >= np.abs(dx)).all() and (mw >= np.abs(dw)).all()


@pytest.mark.parametrize("temperature,hard", [(1.0, 0.0), (2.5, 0.0), (0.5, 0.3), (1.0, 1.0)])
def test_distillation_and_its_gradient(temperature, hard):
    rng = np.random.default_rng(2)
    T, V, K = 6, 40, 5
    z = 2 * rng.standard_normal((T, V))
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    ids[1, 3:], ids[2], ids[3, 4] = -1, V, ids[3, 0]        # few entries, none, the same id twice
    tl = rng.standard_normal((T, K))
    labels = np.array([3, -1, 7, V, 0, ids[5, 1]])
    rows, g = np.array([1, 1, 1, 1, 0, 1], bool), rng.standard_normal(T)
    loss, dz, bl, bz = O.distill(z, ids, tl, labels, temperature, hard, rows, g)
    x = torch.tensor(z, requires_grad=True)
    total = []
    for t in range(T):
        v = torch.zeros((), dtype=torch.float64)
        ok = (ids[t] >= 0) & (ids[t] < V)
        if rows[t] and hard < 1 and ok.any():
            p = torch.softmax(torch.tensor(tl[t][ok]) / temperature, 0)
            q = torch.log_softmax(x[t] / temperature, 0)[torch.tensor(ids[t][ok])]
            v = v + (1 - hard) * temperature ** 2 * (p * (p.log() - q)).sum()
        if rows[t] and hard > 0 and 0 <= labels[t] < V:
            v = v + hard * torch.nn.functional.cross_entropy(x[t:t + 1], torch.tensor([labels[t]]))
        total.append(v)
    total = torch.stack(total)
    (total * torch.tensor(g)).sum().backward()
    np.testing.assert_allclose(loss, total.detach().numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(dz, x.grad.numpy(), rtol=1e-11, atol=1e-14)
    assert (bz(1) >= np.abs(dz)).all()
    # differences
    e = rng.standard_normal((T, V)) * 1e-5
    up, down = (O.distill(z + s * e, ids, tl, labels, temperature, hard, rows)[0] for s in (1, -1))
    np.testing.assert_allclose(((up - down) / 2 * g).sum(), (dz * e).sum(), rtol=1e-7)
