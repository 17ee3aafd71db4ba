"""dx of the router's gradients on the tensor cores holds the bounds that the header
states: an fp32 product's error, whatever the sizes of gradients and weights."""
import numpy as np
import pytest

from oracle import router_train_oracle as R
from tests.test_gpu_router_train import BF16, U, bits, close, run_router, up, val

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()


def dx_tol(dl, Wr, want, dx_in=None):
    """The header's bound, then one rounding to bf16 (2^-134: half its smallest step)."""
    a, w, E = np.abs(dl), np.abs(Wr), dl.shape[1]
    size = a @ w + (0 if dx_in is None else np.abs(dx_in))
    far = (2.0 ** -39 * a.max(1, keepdims=True) + 2.0 ** -151) * w.sum(0)
    far = far + (2.0 ** -39 * w.max() + 2.0 ** -151) * a.sum(1, keepdims=True)
    err = (2.0 ** -20 + 3 * E * 2.0 ** -27) * size + far
    return BF16 * np.abs(want) + (1 + BF16) * err + 2.0 ** -134


def dx_of(dl, Wr, mask=None, dx_in=None):
    """dx beside the other outputs and by itself: the same bits."""
    T, d = len(dl), Wr.shape[1]
    one = run_router(dl, Wr, {}, mask, dx_in, want=("dx",))["dx"].cpu().numpy()
    x = up(bits(np.ones((T, d))))
    every = run_router(dl, Wr, {"x": x}, mask, dx_in)["dx"].cpu().numpy()
    assert np.array_equal(one, every)
    return one


@pytest.mark.parametrize("T,E,d", [(4096, 16, 256), (3000, 32, 320), (2000, 128, 512), (1000, 248, 640),
                                   (150, 130, 2880)])
def test_dx_rounds_as_an_fp32_products(T, E, d):
    """Against the rounded fp64 product. Dropped terms: 3 2^-22 of a product at most, each
    evenly spread, so sqrt(E) of them with random signs make about 2^-22 of dx's norm. An
    addition in TMEM that truncates is off by half a step (2^-24) of the running sum on
    average, half of that again as the sum grows; after the small products there are
    E / 8 of them. A value that is off by r |dx| rounds to the other neighbour, 2^-8 |dx|
    to 2^-7 |dx| away, with a chance of r over that distance: the rounded outputs are
    apart by sqrt(r 2^-7) of dx's norm, times sqrt(2) for what is near zero and off by
    more than r of itself. (Two bf16 terms: r = 4.4e-6 and 1.3e-4 apart.)"""
    rng = np.random.default_rng(T + E)
    p = rng.standard_normal((T, E))
    p = np.exp(p) / np.exp(p).sum(1, keepdims=True)
    dl = ((rng.standard_normal((T, E)) + 0.01) * p / T).astype(np.float32)
    Wr = (rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32)
    want = dl.astype(np.float64) @ Wr.astype(np.float64)
    got = val(dx_of(dl, Wr))
    close(got, want, dx_tol(dl.astype(np.float64), Wr.astype(np.float64), want), "dx")
    r = 2.0 ** -22 + E / 8 * 2.0 ** -25
    apart = np.linalg.norm(got - val(bits(want))) / np.linalg.norm(want)
    print(f"apart {apart:.2e}, allowed {np.sqrt(2 * r * 2.0 ** -7):.2e}")
    assert apart <= np.sqrt(2 * r * 2.0 ** -7), apart


@pytest.mark.parametrize("with_in", [False, True])
@pytest.mark.parametrize("T,E,d", [(1000, 1, 64), (150, 2, 32), (150, 3, 64), (700, 20, 96), (400, 100, 320),
                                   (300, 200, 64)])
def test_dx_of_sizes_far_apart(T, E, d, with_in):
    """Tokens whose gradients lie between fp32's smallest subnormal and 2^100, each
    token's over 60 powers of two; weights over 40; whole rows of zeros."""
    rng = np.random.default_rng(E)
    e = rng.integers(-140, 100, (T, 1)) - np.where(rng.random((T, E)) < 0.5, 0, rng.integers(0, 60, (T, E)))
    dl = (rng.standard_normal((T, E)) * np.exp2(e.astype(np.float64))).astype(np.float32)
    dl[::17] = 0
    Wr = (rng.standard_normal((E, d)) * np.exp2(-rng.integers(0, 40, (E, d)).astype(np.float64))).astype(np.float32)
    dx_in = bits(rng.standard_normal((T, d)) * np.exp2(e[:, :1] - 3.0)) if with_in else None
    mask = (rng.random(T) < 0.9).astype(np.uint8)
    live = mask != 0
    a, w = np.where(live[:, None], dl, 0).astype(np.float64), Wr.astype(np.float64)
    di = None if dx_in is None else val(dx_in)
    want = R.router_grad(a, w, np.zeros((T, d)), live, di)[2]
    dl[~live] = np.nan
    close(val(dx_of(dl, Wr, mask, dx_in)), want, dx_tol(a, w, want, di), "dx")


@pytest.mark.parametrize("wexp", [-149, -126, -60, 60, 120])
def test_dx_of_weights_at_fp32s_ends(wexp):
    rng = np.random.default_rng(5)
    T, E, d = 200, 40, 128
    Wr = np.clip(rng.standard_normal((E, d)), -3, 3) * 2.0 ** wexp
    dl = np.clip(rng.standard_normal((T, E)), -3, 3) * 2.0 ** np.clip(-20 - wexp, -100, 110)
    Wr, dl = Wr.astype(np.float32), dl.astype(np.float32)
    a, w = dl.astype(np.float64), Wr.astype(np.float64)
    close(val(dx_of(dl, Wr)), a @ w, dx_tol(a, w, a @ w), "dx")


@pytest.mark.parametrize("T,E,d", [(200, 6, 64), (1000, 70, 320), (300, 200, 64)])
def test_infinities_and_nans_stay_in_their_tokens_and_columns(T, E, d):
    """An infinite or NaN gradient reaches its token's row, a weight its column; what is
    left is as exact as without them (no scale comes from an infinity)."""
    rng = np.random.default_rng(E)
    dl = (rng.standard_normal((T, E)) / T).astype(np.float32)
    Wr = rng.standard_normal((E, d)).astype(np.float32)
    a, w = dl.astype(np.float64), Wr.astype(np.float64)
    dl[3, 1], dl[7, 0], dl[T - 1, E - 1] = np.inf, np.nan, -np.inf
    Wr[0, 5], Wr[E - 1, d - 1] = -np.inf, np.nan
    got = val(dx_of(dl, Wr))
    rows, cols = [3, 7, T - 1], [5, d - 1]
    assert not np.isfinite(got[rows]).any() and not np.isfinite(got[:, cols]).any()
    keep = np.ix_(np.delete(np.arange(T), rows), np.delete(np.arange(d), cols))
    close(got[keep], (a @ w)[keep], dx_tol(a, w, a @ w)[keep], "dx")
    few = val(run_router(dl[:20], Wr, {}, None, want=("dx",))["dx"].cpu().numpy())   # the CUDA cores' path
    assert np.array_equal(np.isfinite(few[[0, 3, 7, 9]]), np.isfinite(got[[0, 3, 7, 9]]))
