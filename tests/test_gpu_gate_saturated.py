"""The gate's gradient of tokens that one expert has almost for itself: as exact, in
each pair of slots, as for even weights."""
import numpy as np
import pytest

from tests.test_gpu_router_train import U, bits, close, f64, up, val

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()


@pytest.mark.parametrize("T,k,d", [(3, 2, 64), (61, 4, 2880), (300, 8, 352), (3000, 3, 96), (40, 32, 128)])
@pytest.mark.parametrize("gap", [3.0, 12.0, 20.0, 60.0])
def test_gate_gradient_of_a_dominant_weight(T, k, d, gap):
    """sum over l of p_l A_j - p_j A_l with the unrounded softmax p. A: chains of at most
    d / 32 + 16 additions; a weight's rounding, the product's and k + 1 additions. The
    smallest weights (2^-87 at gap 60) are normal numbers."""
    from sparse_moe_layer_05_b200 import binding as B
    rng = np.random.default_rng(int(T + gap))
    E = k + 3
    s = rng.standard_normal((T, k))
    s[np.arange(T), rng.integers(0, k, T)] += gap
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = p.astype(np.float32)
    dout = bits(rng.standard_normal((T, d)))
    yw = (w[:, :, None] * rng.standard_normal((T, k, d))).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    out = torch.empty((T, E), device="cuda")
    B.moe_gate_backward(up(dout), up(yw.reshape(T * k, d)), up(idx), up(w), E, k, T, d, out)
    torch.cuda.synchronize()
    x, y = val(dout), yw.astype(np.float64)
    A, S = np.einsum("td,tkd->tk", x, y), np.einsum("td,tkd->tk", np.abs(x), np.abs(y))
    pair = p[:, None, :] * A[:, :, None] - p[:, :, None] * A[:, None, :]         # [t, j, l]
    size = p[:, None, :] * S[:, :, None] + p[:, :, None] * S[:, None, :]
    size[:, np.arange(k), np.arange(k)] = 0
    want, tol = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, idx, pair.sum(2), 1)
    np.put_along_axis(tol, idx, (d / 32 + k + 20) * U * size.sum(2) + 1e-38, 1)
    close(f64(out), want, tol, "dlogits")


def test_one_slot_has_no_gradient():
    """p is 1 whatever the logit: exactly zero."""
    from sparse_moe_layer_05_b200 import binding as B
    rng = np.random.default_rng(0)
    T, d, E = 50, 320, 6
    out = torch.full((T, E), 7.0, device="cuda")
    B.moe_gate_backward(up(bits(rng.standard_normal((T, d)))), up(rng.standard_normal((T, d)).astype(np.float32)),
                        up(rng.integers(0, E, (T, 1)).astype(np.int32)), up(np.ones((T, 1), np.float32)), E, 1, T, d,
                        out)
    torch.cuda.synchronize()
    assert not out.any()
