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
