"""The balance loss's gradient does not depend on what a token's logits have in
common; the z loss of logits whose squares leave fp32's range."""
import numpy as np
import pytest

from oracle import router_train_oracle as R
from tests.test_gpu_router_train import U, close, f64, run_balance

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()


@pytest.mark.parametrize("T,E,k", [(5, 3, 1), (70, 64, 8), (513, 130, 4), (300, 248, 20)])
@pytest.mark.parametrize("offset", [0.0, 1e2, 1e4, 1e7])
def test_balance_gradient_of_an_offset(T, E, k, offset):
    """Logits are fp32 numbers around the offset, spaced so that fp64 sees the same ones.
    p: exp off by 2 ulp, its argument by u |s - lse| (lse's own rounding is common to the
    row), a sum of 256 at most in 8 + 5 additions, a quotient: 128 u as at offset 0."""
    rng = np.random.default_rng(T + E)
    s = (rng.standard_normal((T, E)) * 3 + offset).astype(np.float32)
    idx = np.argsort(-s, axis=1, kind="stable")[:, :k].astype(np.int32)
    a, dl = np.float32(0.3), np.array([1.7], np.float32)
    live = np.ones(T, bool)
    d = run_balance(s, idx, None, a, 0.0, dl)[-1]
    s64 = s.astype(np.float64)
    want = R.balance_loss_grad(s64, idx, k, a, 0.0, live, dloss=float(dl[0]))
    f, p = R.expert_counts(idx, E, live) / (T * k), R.softmax(s64)
    size = dl[0] / T * p * a * E * (f + (p @ f)[:, None])
    close(f64(d), want, 256 * U * size + 1e-38, "dlogits")
    # a row's gradients add up to nothing, but for roundings
    total = np.abs(f64(d).sum(1))
    assert (total <= 256 * U * size.sum(1) + 1e-38).all()


@pytest.mark.parametrize("T", [40, 600])
def test_z_loss_beyond_fp32s_range(T):
    """lse = 1e20 in half of the rows: z is 5e39, an infinity in fp32; the loss holds the
    balance term alone where its coefficient is 0, and 1e-30 z where it is that."""
    E, k = 33, 2
    rng = np.random.default_rng(T)
    s = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-s, axis=1)[:, :k].astype(np.int32)
    s[::2] = -1e20
    s[::2, 7] = 1e20
    live = np.ones(T, bool)
    for b in (0.0, 1e-30):
        (loss, bal, z, n), *_ = R.balance_loss(s.astype(np.float64), idx, k, 1.0, float(np.float32(b)), live)
        stats, *_, d = run_balance(s, idx, None, 1.0, b)
        got = f64(stats)
        assert np.isposinf(got[2]) and z > 1e39
        close(got[:2], np.array([loss, bal]), 256 * U * np.array([abs(loss), bal]), "loss, balance")
        assert np.isfinite(f64(d)).all()
