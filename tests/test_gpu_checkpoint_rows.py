"""Checkpointed rows at the type's ends through the backward calls: where the sum of
squares is infinite rstd is 0, and the row counts as zeros, whether it holds an
infinity (whose codes stand for 1.75 2^128) or finite values above 1.8e19."""
import numpy as np
import pytest

from oracle import router_train_oracle as R
from tests.test_gpu_router_train import (BF16, U, bits, chain, checkpoint_of, close, f64, router_tol,
                                         run_router, up, val)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()


INF, HUGE = 3, 8


def rows_of(T, d, rng):
    """Token 3 holds infinities, token 8 values of 1e30; the rows as kept, their rstd."""
    h = rng.standard_normal((T, d))
    h[INF, 1], h[INF, d - 1] = np.inf, -np.inf
    h[HUGE] = 1e30 * np.sign(h[HUGE])
    q, sc, rstd = checkpoint_of(bits(h), 1e-5)
    assert f64(rstd)[[INF, HUGE]].tolist() == [0, 0] and bool((rstd[:3] > 0).all())
    v = R.checkpoint_rows(q.cpu().numpy(), sc.cpu().numpy())
    assert v[INF, 1] == 1.75 * 2.0 ** 128 and np.isfinite(v).all()
    return q, sc, rstd, v


@pytest.mark.parametrize("T,E,d", [(20, 5, 96), (60, 70, 64), (200, 20, 320), (700, 130, 96)])
def test_router_gradients_of_such_rows(T, E, d):
    """Both paths, both stage widths. An infinite gradient of such a token still shows."""
    rng = np.random.default_rng(T)
    q, sc, rstd, v = rows_of(T, d, rng)
    g = rng.uniform(0.5, 1.5, d).astype(np.float32)
    dl, Wr = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal((E, d)).astype(np.float32)
    src = {"q": q, "scales": sc, "rstd": rstd, "g": up(g)}
    x = v * f64(rstd)[:, None] * g
    a = dl.astype(np.float64), Wr.astype(np.float64), x, np.ones(T, bool)
    want = R.router_grad(*a)
    tol = router_tol(*a, want)
    o = run_router(dl, Wr, src, None)
    for n, w, t in zip(("dW", "db"), want, tol):
        close(f64(o[n]), w, t, n)
    dl[INF, 1] = np.inf
    bad = f64(run_router(dl, Wr, src, None, want=("dW",))["dW"])
    assert np.isnan(bad[1]).all() and np.isfinite(np.delete(bad, 1, 0)).all()


@pytest.mark.parametrize("T,d", [(20, 64), (150, 2880), (12, 8192), (12, 16384)])
def test_norm_backward_of_such_rows(T, d):
    """dh is dh_in there and dg gets nothing; a NaN in such a token's dx still shows."""
    from sparse_moe_layer_05_b200 import binding as B
    rng = np.random.default_rng(d)
    q, sc, rstd, v = rows_of(T, d, rng)
    g = rng.uniform(0.5, 1.5, d).astype(np.float32)
    dx, dh_in = bits(rng.standard_normal((T, d))), bits(rng.standard_normal((T, d)))
    ws = torch.empty(B.moe_rms_norm_backward_workspace_size(T, d), dtype=torch.uint8, device="cuda")

    def run(dx):
        dh, dg = torch.empty((T, d), dtype=torch.uint16, device="cuda"), torch.empty(d, device="cuda")
        B.moe_rms_norm_backward(up(dx), up(g), rstd, T, d, dh, dg, ws, q=q, scales=sc, dh_in=up(dh_in))
        torch.cuda.synchronize()
        return dh.cpu().numpy(), f64(dg)

    r, live = f64(rstd), np.ones(T, bool)
    want_dh, want_dg = R.rms_norm_grad(val(dx), v, r, g.astype(np.float64), live, val(dh_in))
    dh, dg = run(dx)
    n, un = np.abs(v * r[:, None]), np.abs(val(dx)) * g
    close(dg, want_dg, chain(T) * U * (np.abs(val(dx)) * n).sum(0) + 1e-38, "dg")
    size = r[:, None] * (un + n * (un * n).mean(1, keepdims=True)) + np.abs(val(dh_in))
    close(val(dh), want_dh, BF16 * np.abs(want_dh) + 72 * U * size + 1e-38, "dh")
    assert np.array_equal(dh[[INF, HUGE]], dh_in[[INF, HUGE]])
    dx[INF, 0] = 0x7FC0
    dh, dg = run(dx)
    assert np.isnan(val(dh[INF])[0]) and np.isnan(dg[0])
