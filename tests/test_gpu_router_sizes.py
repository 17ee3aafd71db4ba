"""The training calls at sizes that only their largest plans reach: grids of more blocks
than the chip holds at a time, batches that are split by the length of a running sum,
arrays of more than 2^31 elements. The long ones against fp64 products on the GPU."""
import pytest

from tests import test_gpu_router_train as train
from tests.test_gpu_router_train import BF16, U, chain, ws_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


# (T + E) % 4 picks the mask: the first half of the tokens at 150 + 256 and 130 + 200, some at
# 133 + 200, none otherwise
@pytest.mark.parametrize("rows", ["bf16", "8bit"])
@pytest.mark.parametrize("T,E,d", [(150, 256, 16384), (152, 256, 16384), (130, 200, 16352), (133, 200, 16352),
                                   (300, 20, 16352)])
def test_more_blocks_than_the_chip_holds(T, E, d, rows):
    """256 blocks of dW and of dx (d / 64 tiles, the last one half a unit at 16352)."""
    train.test_router_gradients(T, E, d, rows)


def chunks(T, n=10000):
    return [slice(t, min(t + n, T)) for t in range(0, T, n)]


def random_bf16(T, d, gen):
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    for c in chunks(T):
        x[c] = torch.randn(x[c].shape, device="cuda", generator=gen).bfloat16()
    return x


def within(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    assert bool((off <= 0).all()), (what, float(off.max()))       # NaN fails too


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows", ["bf16", "8bit"])
@pytest.mark.parametrize("T,E,d", [(140000, 2, 6400), (139999, 130, 3232)])
def test_batches_split_by_the_length_of_a_running_sum(T, E, d, rows, masked):
    """50 tiles (or 26 of two groups) leave room for two splits on the chip; running sums
    of 65536 tokens at most ask for three. chain(T) as for short batches."""
    from sparse_moe_layer_05_b200 import binding as B
    gen = torch.Generator(device="cuda").manual_seed(T)
    dl = torch.randn((T, E), device="cuda", generator=gen) / T
    live = torch.rand(T, device="cuda", generator=gen) < 0.9 if masked else torch.ones(T, dtype=torch.bool, device="cuda")
    g = torch.rand(d, device="cuda", generator=gen) + 0.5
    if rows == "bf16":
        x = random_bf16(T, d, gen)
        src, rows_of = {"x": x}, lambda c: x[c].double()
    else:
        q = torch.randint(0, 127, (T, d), dtype=torch.uint8, device="cuda", generator=gen)
        sc = torch.randint(110, 125, (T, d // 32), dtype=torch.uint8, device="cuda", generator=gen)
        r = torch.rand(T, device="cuda", generator=gen) + 0.5
        src = {"q": q, "scales": sc, "rstd": r, "g": g}

        def rows_of(c):
            v = q[c].view(torch.float8_e4m3fn).double().view(-1, d // 32, 32)
            s = torch.exp2(sc[c].double() - 127)
            return (v * s[:, :, None]).view(-1, d) * r[c].double()[:, None] * g.double()

    dW, db = torch.empty((E, d), device="cuda"), torch.empty(E, device="cuda")
    B.moe_router_backward(dl, None, E, T, d, dW, db, None, ws_of(B.moe_router_backward_workspace_size(E, T, d)),
                          token_mask=live if masked else None, **src)
    want, size = torch.zeros((E, d), dtype=torch.float64, device="cuda"), torch.zeros((E, d), dtype=torch.float64,
                                                                                     device="cuda")
    a = torch.where(live[:, None], dl.double(), 0)
    for c in chunks(T):
        v = rows_of(c)
        want += a[c].t() @ v
        size += a[c].abs().t() @ v.abs()
    tol = chain(T) * 2 * U
    within(dW, want, tol * size, "dW")
    within(db, a.sum(0), tol * a.abs().sum(0), "db")


def ends(T):
    """Rows on both sides of element 2^31 and at the ends."""
    return [0, 1, T // 3, T - 2, T - 1]


def test_arrays_of_more_than_2_31_elements():
    """T d = 2.3e9: the norm with its checkpoint and its backward pass, dx of the router;
    rows from both ends against the formulas, dg against all."""
    from sparse_moe_layer_05_b200 import binding as B
    T, d, E = 140000, 16384, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    h = random_bf16(T, d, gen)
    g = torch.rand(d, device="cuda", generator=gen) + 0.5
    x = torch.empty_like(h)
    q = torch.empty((T, d), dtype=torch.uint8, device="cuda")
    sc, rstd = torch.empty((T, d // 32), dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    B.moe_rms_norm_checkpoint(h, g, 1e-5, T, d, x, q, sc, rstd)
    x2, q2, sc2 = torch.empty_like(x), torch.empty_like(q), torch.empty_like(sc)
    B.moe_rms_norm(h, g, 1e-5, T, d, x2)
    B.moe_mx_quantize(h, T, d, B.ACT_MXFP8, q2, sc2)
    assert torch.equal(x.view(torch.int16), x2.view(torch.int16)) and torch.equal(q, q2) and torch.equal(sc, sc2)
    del x2, q2, sc2
    at = ends(T)
    r = 1 / (h[at].double().square().mean(1) + 1e-5).sqrt()
    within(rstd[at], r, (d / 64 + 8) * U * r, "rstd")

    # dx = dlogits W + dx_in of the router, x as dx_in
    dl, W = torch.randn((T, E), device="cuda", generator=gen), torch.randn((E, d), device="cuda", generator=gen)
    dx = torch.empty_like(x)
    B.moe_router_backward(dl, W, E, T, d, None, None, dx, ws_of(B.moe_router_backward_workspace_size(E, T, d)), dx_in=x)
    want = dl[at].double() @ W.double() + x[at].double()
    size = dl[at].double().abs() @ W.double().abs() + x[at].double().abs()
    within(dx[at], want, BF16 * want.abs() + (2.0 ** -16 + 4 * E * U) * size, "dx")

    ws = ws_of(B.moe_rms_norm_backward_workspace_size(T, d))
    for src in ({"h": h}, {"q": q, "scales": sc}):
        dh, dg = torch.empty_like(h), torch.empty(d, device="cuda")
        B.moe_rms_norm_backward(dx, g, rstd, T, d, dh, dg, ws, dh_in=x, **src)

        def n_of(c):
            if "h" in src:
                v = h[c].double()
            else:
                v = q[c].view(torch.float8_e4m3fn).double().view(-1, d // 32, 32)
                v = (v * torch.exp2(sc[c].double() - 127)[:, :, None]).view(-1, d)
            return v * rstd[c].double()[:, None]

        n, u, rr = n_of(at), dx[at].double() * g.double(), rstd[at].double()[:, None]
        want = rr * (u - n * (u * n).mean(1, keepdim=True)) + x[at].double()
        size = rr * (u.abs() + n.abs() * (u * n).abs().mean(1, keepdim=True)) + x[at].double().abs()
        within(dh[at], want, BF16 * want.abs() + 72 * U * size, "dh")
        total, sizes = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
        for c in chunks(T, 5000):
            v = dx[c].double() * n_of(c)
            total += v.sum(0)
            sizes += v.abs().sum(0)
        within(dg, total, chain(T) * U * sizes, "dg")


def test_gate_gradient_of_more_than_2_31_elements():
    from sparse_moe_layer_05_b200 import binding as B
    T, k, d, E = 40000, 4, 16384, 6
    gen = torch.Generator(device="cuda").manual_seed(4)
    yw = torch.empty((T * k, d), device="cuda")
    for c in chunks(T * k):
        yw[c] = torch.randn(yw[c].shape, device="cuda", generator=gen)
    dout = random_bf16(T, d, gen)
    idx = torch.argsort(torch.rand((T, E), device="cuda", generator=gen), dim=1)[:, :k].int().contiguous()
    w = torch.softmax(torch.randn((T, k), device="cuda", generator=gen), 1)
    out = torch.empty((T, E), device="cuda")
    B.moe_gate_backward(dout, yw, idx, w, E, k, T, d, out)
    at = ends(T)
    y, x, p = yw.view(T, k, d)[at].double(), dout[at].double()[:, None, :], w[at].double()
    A, S = (y * x).sum(2), (y * x).abs().sum(2)
    want = torch.zeros((len(at), E), dtype=torch.float64, device="cuda").scatter_(1, idx[at].long(), A - p * A.sum(1, keepdim=True))
    tol = torch.zeros_like(want).scatter_(1, idx[at].long(), (d / 32 + k + 18) * U * (S + p * S.sum(1, keepdim=True)))
    within(out[at], want, tol, "dlogits")
