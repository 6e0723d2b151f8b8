"""CPU pins of the oracle of the operators around attention: rotations against
complex products and their own inverse, the head norm and differential
attention against central differences and against a torch composition."""
import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    hd, rot, T, H = 12, 8, 5, 3
    f, amp = O.rotary_frequencies(rot)
    pos = np.array([0, 1, 7, 100, 99999])
    x = rng.standard_normal((T, H * hd))
    y = O.rotate(x, pos, f, 1.5, hd, interleaved).reshape(T, H, hd)
    xh = x.reshape(T, H, hd)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        z = (xh[..., a] + 1j * xh[..., b]) * 1.5 * np.exp(1j * pos * f[i])[:, None]
        np.testing.assert_allclose(y[..., a], z.real, atol=1e-12)
        np.testing.assert_allclose(y[..., b], z.imag, atol=1e-12)
    assert np.array_equal(y[..., rot:], xh[..., rot:])
    back = O.rotate(O.rotate(x, pos, f, 1.0, hd, interleaved), pos, f, 1.0, hd, interleaved, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-12)


def test_scaled_frequencies_at_their_ends():
    f, _ = O.rotary_frequencies(64)
    lin, _ = O.rotary_frequencies(64, scaling="linear", factor=4)
    np.testing.assert_allclose(lin, f / 4)
    base, _ = O.rotary_frequencies(64, scaling="base", factor=4)
    assert base[0] == 1.0
    np.testing.assert_allclose(base[-1], f[-1] / 4)       # the slowest pair is stretched by the factor
    for kind in ("wavelength", "yarn"):
        s, amp = O.rotary_frequencies(64, scaling=kind, factor=4, original_len=2048)
        np.testing.assert_allclose(s[0], f[0])            # the fastest pair is kept
        np.testing.assert_allclose(s[-1], f[-1] / 4)
        assert np.all(s <= f * (1 + 1e-15)) and np.all(s >= f / 4 * (1 - 1e-15))
        assert amp == (1.0 if kind == "wavelength" else pytest.approx(1 + 0.1 * np.log(4)))


def _difference(f, x, d, e=1e-6):
    return (f(x + e * d) - f(x - e * d)) / (2 * e)


def test_head_norm_backward_against_differences():
    rng = np.random.default_rng(1)
    hd, T, H = 6, 4, 3
    x, w, g = rng.standard_normal((T, H * hd)), rng.standard_normal(hd), rng.standard_normal((T, H * hd))
    dx, dw, _, _ = O.head_norm_backward(x, w, g, hd, 1e-3)
    for _ in range(4):
        d = rng.standard_normal(x.shape)
        assert (dx * d).sum() == pytest.approx(_difference(lambda t: (O.head_norm(t, w, hd, 1e-3) * g).sum(), x, d), rel=1e-6)
        d = rng.standard_normal(hd)
        assert (dw * d).sum() == pytest.approx(_difference(lambda t: (O.head_norm(x, t, hd, 1e-3) * g).sum(), w, d), rel=1e-6)


@pytest.mark.parametrize("causal,lens", [(True, None), (False, [5, 0]), (True, [3, 7])])
def test_diff_attention_backward_against_differences(causal, lens):
    rng = np.random.default_rng(2)
    B, L, heads = 2, 7, (8, 4, 4)
    hq, hkv, hd = heads
    x = {"q": rng.standard_normal((B * L, hq * hd)), "k": rng.standard_normal((B * L, hkv * hd)),
         "v": rng.standard_normal((B * L, hkv * hd))}
    x.update({n: 0.5 * rng.standard_normal(hd) for n in ("lq1", "lk1", "lq2", "lk2")})
    da = rng.standard_normal((B * L, hq * hd))

    def out(t, **kw):
        return O.diff_attention(t["q"], t["k"], t["v"], [t[n] for n in ("lq1", "lk1", "lq2", "lk2")], 0.6, B, heads,
                                0.7, causal, lens, **kw)

    g = out(x, da=da)
    for n in x:
        for _ in range(3):
            d = rng.standard_normal(x[n].shape)
            num = _difference(lambda t: (out({**x, n: t})["a"] * da).sum(), x[n], d)
            assert (g["d" + n] * d).sum() == pytest.approx(num, rel=2e-6, abs=1e-8), n


def test_diff_attention_against_two_softmaxes():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    L, heads = 9, (4, 2, 8)
    q, k, v = (rng.standard_normal((L, h * 8)) for h in (4, 2, 2))
    lv = [0.3 * rng.standard_normal(8) for _ in range(4)]
    a = O.diff_attention(q, k, v, lv, 0.5, 1, heads, 8 ** -0.5, True)["a"]
    lam = O.diff_lambda(lv, 0.5)[0]
    tq, tk, tv = (torch.from_numpy(x) for x in (q, k, v))
    mask = torch.ones(L, L, dtype=torch.bool).tril()
    for h in range(2):
        maps = [torch.softmax((tq[:, (2 * h + m) * 8:(2 * h + m + 1) * 8] @ tk[:, m * 8:(m + 1) * 8].T * 8 ** -0.5)
                              .masked_fill(~mask, float("-inf")), -1) for m in (0, 1)]
        np.testing.assert_allclose(a[:, 16 * h:16 * (h + 1)], ((maps[0] - lam * maps[1]) @ tv).numpy(), atol=1e-12)
