"""The fp64 formulas of the router's training step against central differences
of the functions they differentiate, and against hand-made values."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import router_train_oracle as R


def numeric(f, a, step=1e-5):
    """Central differences of a scalar function at every element of a."""
    out = np.zeros_like(a)
    for i in np.ndindex(*a.shape):
        hi, lo = a.copy(), a.copy()
        hi[i] += step
        lo[i] -= step
        out[i] = (f(hi) - f(lo)) / (2 * step)
    return out


# central differences of step h: h^2/6 f''' (about 1e-10 for these smooth functions of size
# one) plus 2^-52/h (about 2e-11) times the function's size
TOL = 1e-8


def case(T=7, E=6, k=3, d=8, seed=0):
    rng = np.random.default_rng(seed)
    live = rng.random(T) < 0.7
    live[0], live[1] = True, False
    s = rng.standard_normal((T, E)) * 2
    idx = np.argsort(-s, axis=1)[:, :k]
    return rng, live, s, idx


def test_balance_gradient_is_the_difference_quotient():
    rng, live, s, idx = case()
    k = idx.shape[1]
    got = R.balance_loss_grad(s, idx, k, 0.3, 0.2, live, dloss=1.7)
    want = numeric(lambda a: 1.7 * R.balance_loss(a, idx, k, 0.3, 0.2, live)[0][0], s)
    assert np.abs(got - want).max() < TOL
    assert not got[~live].any()


def test_balance_of_even_routing_is_one():
    """Equal probabilities and equal counts: E * sum (1/E)(1/E) = 1; z = log(E)^2."""
    E, k, T = 4, 2, 6
    idx = np.array([[t % 2 * 2, t % 2 * 2 + 1] for t in range(T)])
    (loss, bal, z, n), counts, mean, lse = R.balance_loss(np.zeros((T, E)), idx, k, 1.0, 0.5,
                                                          np.ones(T, bool))
    assert counts.tolist() == [3, 3, 3, 3] and n == T
    assert abs(bal - 1) < 1e-15 and abs(z - np.log(E) ** 2) < 1e-15
    assert abs(loss - (1 + 0.5 * np.log(E) ** 2)) < 1e-15


def test_empty_rows_dropped_pairs_and_no_tokens():
    s = np.array([[0.0, -np.inf, 1.0], [-np.inf] * 3])
    idx = np.array([[2, -1], [0, 3]])
    live = np.ones(2, bool)
    (loss, bal, z, n), counts, mean, lse = R.balance_loss(s, idx, 2, 1.0, 1.0, live)
    assert counts.tolist() == [1, 0, 1] and n == 2
    assert np.isneginf(lse[1]) and abs(z - np.log(1 + np.e) ** 2 / 2) < 1e-14
    assert mean[1] == 0 and abs(mean.sum() - 0.5) < 1e-15
    g = R.balance_loss_grad(s, idx, 2, 1.0, 1.0, live)
    assert not g[1].any() and np.isfinite(g).all()
    none = R.balance_loss(s, idx, 2, 1.0, 1.0, np.zeros(2, bool))
    assert none[0] == (0.0, 0.0, 0.0, 0) and not none[1].any()


def test_gate_gradient_is_the_difference_quotient():
    rng, live, s, idx = case(seed=1)
    (T, E), k, d = s.shape, idx.shape[1], 8
    y, dout = rng.standard_normal((T, k, d)), rng.standard_normal((T, d))

    def out(a):
        return (R.softmax(np.take_along_axis(a, idx, 1))[:, :, None] * y).sum(1)

    w = R.softmax(np.take_along_axis(s, idx, 1))
    got = R.gate_grad(dout, (w[:, :, None] * y).reshape(T * k, d), idx, w, E, live)
    want = numeric(lambda a: (out(a) * dout)[live].sum(), s)
    assert np.abs(got - want).max() < TOL


def test_router_and_norm_gradients_are_difference_quotients():
    rng, live, s, idx = case(seed=2)
    (T, E), d = s.shape, 8
    h, W, b, g = (rng.standard_normal(n) for n in ((T, d), (E, d), (E,), (d,)))
    ds, eps = rng.standard_normal((T, E)), 1e-3

    def loss(h_, W_, b_, g_):
        return ((R.rms_norm(h_, g_, eps) @ W_.T + b_) * ds)[live].sum()

    dW, db, dx = R.router_grad(ds, W, R.rms_norm(h, g, eps), live)
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    dh, dg = R.rms_norm_grad(dx, h, rstd, g, live)
    for got, at, f in ((dW, W, lambda a: loss(h, a, b, g)), (db, b, lambda a: loss(h, W, a, g)),
                       (dh, h, lambda a: loss(a, W, b, g)), (dg, g, lambda a: loss(h, W, b, a))):
        assert np.abs(got - numeric(f, at)).max() < TOL * max(1.0, np.abs(got).max())
    assert np.array_equal(R.rms_norm_grad(dx, h, rstd, g, live, dh_in=h)[0], dh + h)


def test_checkpoint_rows_invert_the_mx_conversion():
    """Codes and scales as the MX conversion of the oracle gives them."""
    codes = np.arange(256)
    grid = R.e4m3_value(codes)
    assert np.isnan(grid[127]) and np.isnan(grid[255])
    assert grid[0x7E] == 448 and grid[1] == 2.0 ** -9 and grid[8] == 2.0 ** -6 and grid[0x38] == 1
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 64)) * 100
    got = O.mx_quantize(x, "e4m3")
    vals, sb = (got if isinstance(got, tuple) else (got, None))[:2]
    pos = grid[:127]
    scale = np.exp2(np.floor(np.log2(np.abs(x.reshape(3, 2, 32)).max(2))) - 8)
    q = np.searchsorted(pos, np.abs(vals).reshape(3, 2, 32) / scale[:, :, None])
    code = (q + np.where(vals.reshape(q.shape) < 0, 128, 0)).reshape(3, 64).astype(np.uint8)
    s = (np.log2(scale) + 127).astype(np.uint8)
    assert np.array_equal(R.checkpoint_rows(code, s), vals)


@pytest.mark.parametrize("plant", ["f", "mean", "n", "z"])
def test_planted_mistakes_are_seen(plant, monkeypatch):
    """A dropped term of the balance gradient does not pass the difference test."""
    rng, live, s, idx = case(seed=4)
    k = idx.shape[1]
    p, lse = R.softmax(s), R.log_sum_exp(s)[:, None]
    n, E = live.sum(), s.shape[1]
    f = R.expert_counts(idx, E, live) / (n * k)
    fp = (p @ f)[:, None]
    wrong = {"f": 0 * f - fp, "mean": f - 0 * fp, "n": (f - fp), "z": (f - fp)}[plant]
    got = (1 / n if plant != "n" else 1 / len(s)) * p * (0.3 * E * wrong + (0.0 if plant == "z" else 0.4) * lse)
    want = numeric(lambda a: R.balance_loss(a, idx, k, 0.3, 0.2, live)[0][0], s)
    assert np.abs(np.where(live[:, None], got, 0) - want).max() > 1e-4
