"""The router's training step on the GPU against the fp64 formulas of
oracle/router_train_oracle.py, on the same fp32, bf16 and 8-bit inputs.

Tolerances count roundings: u = 2^-24 is half an fp32 step relative to the
value, 2^-8 bounds half a bf16 step. A sum of n terms in fp32 is off by at most
(length of its longest chain of additions) u times the sum of the terms' sizes;
the chains are stated at each test."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import router_train_oracle as R
from sparse_moe_layer_05_b200 import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()


def up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bits(a):
    return W.f32_to_bf16_bits(np.asarray(a, dtype=np.float32))


def val(u16):
    return O.bf16_to_f64(u16)


def f64(t):
    return t.cpu().numpy().astype(np.float64)


def empty(*shape, dtype=torch.float32):
    """An output with 64 guard elements behind it; `guarded` checks them."""
    n = int(np.prod(shape))
    byte = dtype in (torch.uint8,)
    raw = torch.full((n + 64,), 77 if byte else -7, dtype=torch.int16 if dtype == torch.uint16 else dtype,
                     device="cuda")
    t = raw[:n].view(dtype).view(*shape)
    empty.made.append((raw, n, 77 if byte else -7))
    return t


empty.made = []


def guarded():
    for raw, n, v in empty.made:
        assert bool((raw[n:] == v).all()), "written past the output's end"
    empty.made.clear()


def ws_of(nbytes):
    assert nbytes > 0
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def close(got, want, tol, what):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        t = np.broadcast_to(tol, want.shape)[i]
        raise AssertionError(f"{what}{i}: {got[i]!r}, want {want[i]!r}, off by {abs(got[i] - want[i]):.3e}, "
                             f"allowed {t:.3e} ({int(bad.sum())} of {bad.size})")


def chain(T):
    """Longest chain of fp32 additions over T tokens: the kernels sum at most
    512 tokens (T / 64 for very long batches) one after another."""
    return min(T, 512 + T // 64) + 16


MASKS = ["none", "some", "first", "all"]


def live_of(mask, T, rng):
    if mask == "none":
        return None, np.ones(T, bool)
    live = {"some": rng.random(T) < 0.8, "first": np.arange(T) < (T + 1) // 2,
            "all": np.zeros(T, bool)}[mask]
    # any byte but 0 counts as live
    return (live * rng.integers(1, 256, T)).astype(np.uint8), live


# ------------------------------------------------------------ balance loss --

BALANCE = [(1, 1, 1, "none"), (1, 256, 32, "none"), (7, 2, 1, "some"), (61, 5, 3, "first"),
           (64, 64, 8, "none"), (1000, 33, 4, "some"), (4093, 248, 20, "none"), (300, 32, 4, "all"),
           (9001, 128, 4, "some")]


def run_balance(logits, idx, mask, a, b, dloss=None, E=None, accumulate=None):
    from sparse_moe_layer_05_b200 import binding as B
    T, E = logits.shape
    k = idx.shape[1]
    lt, it, mt = up(logits), up(idx), up(mask)
    stats, counts = empty(4), empty(E, dtype=torch.int32)
    mean, lse = empty(E), empty(T)
    B.moe_balance_loss(lt, it, E, k, T, a, b, stats, counts, mean, lse,
                       ws_of(B.moe_balance_loss_workspace_size(E, k, T)), token_mask=mt)
    d = empty(T, E)
    if accumulate is not None:
        d.copy_(up(accumulate))
    B.moe_balance_loss_backward(lt, lse, counts, stats, E, k, T, a, b, d, dloss=up(dloss), token_mask=mt,
                                accumulate=accumulate is not None)
    torch.cuda.synchronize()
    guarded()
    return stats, counts, mean, lse, d


@pytest.mark.parametrize("T,E,k,mask", BALANCE)
def test_balance_loss_and_gradient(T, E, k, mask):
    """lse: exp off by 2 ulp, arguments off by u |s - max| (their p-weighted sum at
    most log E + 1 < 8), 14 additions, log and the last addition: 32 u + 4 u |lse|.
    p adds its own argument's rounding (|s - lse| < 40): 128 u in all."""
    rng = np.random.default_rng(T + E)
    m, live = live_of(mask, T, rng)
    s = (rng.standard_normal((T, E)) * 3 + rng.standard_normal(E)).astype(np.float32)
    idx = np.argsort(-s, axis=1)[:, :k].astype(np.int32)
    s[~live] = np.nan                                # padded rows may hold anything
    a, b, dl = 0.3, 0.02, np.array([1.7], np.float32)
    base = rng.standard_normal((T, E)).astype(np.float32)
    stats, counts, mean, lse, d = run_balance(s, idx, m, a, b, dl)
    s64 = np.where(live[:, None], s.astype(np.float64), 0.0)
    (loss, bal, z, n), cnt, mp, l64 = R.balance_loss(s64, idx, k, np.float32(a), np.float32(b), live)
    assert counts.cpu().numpy().tolist() == cnt.tolist()
    ltol = 32 * U + 4 * U * np.abs(l64)
    close(f64(lse), l64, np.where(live, ltol, 0.0), "lse")
    ptol = (128 + chain(T)) * U
    close(f64(mean), mp, ptol * mp + 1e-38, "mean_probs")
    ztol = (2 * np.abs(l64) * ltol)[live].sum() / max(n, 1) + 4 * U * z
    close(f64(stats), np.array([loss, bal, z, n]),
          np.array([a * ptol * bal + b * ztol + 4 * U * abs(loss), ptol * bal + 2 * U * bal, ztol, 0.0]), "stats")
    want = R.balance_loss_grad(s64, idx, k, np.float32(a), np.float32(b), live, dloss=float(dl[0]))
    f = cnt / max(n * k, 1)
    p = np.where(live[:, None], R.softmax(s64), 0.0)
    size = dl[0] / max(n, 1) * p * (a * E * (f + (p @ f)[:, None]) + 2 * b * np.abs(l64)[:, None])
    close(f64(d), want, 256 * U * size + 1e-38, "dlogits")
    *_, d2 = run_balance(s, idx, m, a, b, dl, accumulate=base)
    close(f64(d2), want + base, 256 * U * size + U * np.abs(want + base) + 1e-38, "accumulated dlogits")
    assert np.array_equal(d2.cpu().numpy()[~live], base[~live])


def test_balance_edge_rows():
    """-inf logits, a row of nothing but -inf, a row with one +inf and one with a NaN,
    dropped pairs; NaN appears only where the definition has it."""
    E, k = 40, 2
    rng = np.random.default_rng(3)
    s = rng.standard_normal((9, E)).astype(np.float32)
    idx = np.argsort(-s, axis=1)[:, :k].astype(np.int32)
    s[0, 5:] = -np.inf
    s[1] = -np.inf
    idx[2, 1], idx[3, 0] = -1, E
    s[4] = 80 * np.sign(s[4])                        # exp(80) overflows without the max
    s[5] -= 1e4
    stats, counts, mean, lse, d = run_balance(s, idx, None, 1.0, 0.0)
    live = np.ones(9, bool)
    (loss, bal, z, n), cnt, mp, l64 = R.balance_loss(s.astype(np.float64), idx, k, 1.0, 0.0, live)
    assert counts.cpu().numpy().tolist() == cnt.tolist()
    got = f64(lse)
    assert np.isneginf(got[1])
    rest = np.arange(9) != 1
    close(got[rest], l64[rest], 32 * U + 4 * U * np.abs(l64[rest]), "lse")
    # arguments up to 1e4 are rounded to u 1e4 before exp
    close(f64(mean), mp, 2e4 * U * mp + 1e-38, "mean")
    want = R.balance_loss_grad(s.astype(np.float64), idx, k, 1.0, 0.0, live)
    size = 1 / 9 * E * np.where(np.isneginf(l64)[:, None], 0, R.softmax(s.astype(np.float64)))
    close(f64(d), want, 3e4 * U * size + 1e-38, "dlogits")
    assert not f64(d)[1].any()
    s[6, 3], s[7, 8] = np.inf, np.nan
    stats, counts, mean, lse, d = run_balance(s, idx, None, 1.0, 0.1)
    dn = f64(d)
    assert np.isnan(f64(stats)[0]) and np.isnan(dn[6]).any() and np.isnan(dn[7]).all()
    assert np.isfinite(dn[[0, 1, 2, 3, 4, 5, 8]]).all()
    m = np.ones(9, np.uint8)
    m[[6, 7]] = 0
    stats, counts, mean, lse, d = run_balance(s, idx, m, 1.0, 0.1)
    assert np.isfinite(f64(stats)).all() and np.isfinite(f64(d)).all() and not f64(d)[[6, 7]].any()


# ----------------------------------------------------------- gate gradient --

GATE = [(1, 1, 1, 32, "none"), (3, 2, 2, 64, "none"), (61, 64, 8, 2880, "some"), (130, 256, 32, 96, "first"),
        (257, 248, 20, 352, "none"), (5, 7, 3, 16384, "none"), (40, 32, 4, 2880, "all"),
        (1500, 32, 4, 1024, "some")]


@pytest.mark.parametrize("T,E,k,d,mask", GATE)
def test_gate_gradient(T, E, k, d, mask):
    """Each dot product: chains of at most d / 32 + 16 additions; then A_j - p_j sum A
    with k + 2 more roundings."""
    from sparse_moe_layer_05_b200 import binding as B
    rng = np.random.default_rng(T * 7 + k)
    m, live = live_of(mask, T, rng)
    dout = bits(rng.standard_normal((T, d)))
    yw = rng.standard_normal((T * k, d)).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    w /= w.sum(1, keepdims=True)
    if T > 2:
        idx[1, 0] = -1                                # a dropped pair
        idx[2, -1] = idx[2, 0]                        # the same expert twice
        w[2, :] = 0
        w[2, 0] = 1                                   # weights that underflowed
    dout[~live] = 0x7FC0
    yw.reshape(T, k * d)[~live] = np.nan
    out = empty(T, E)
    args = (up(dout), up(yw), up(idx), up(w), E, k, T, d)
    B.moe_gate_backward(*args, out, token_mask=up(m))
    torch.cuda.synchronize()
    x = np.where(live[:, None], val(dout), 0.0)
    y = np.where(live[:, None], yw.reshape(T, k * d).astype(np.float64), 0.0).reshape(T * k, d)
    w64 = w.astype(np.float64)
    want = R.gate_grad(x, y, idx, w64, E, live)
    S = np.einsum("td,tkd->tk", np.abs(x), np.abs(y.reshape(T, k, d)))
    tol = (d / 32 + k + 18) * U * (S + w64 * S.sum(1, keepdims=True))
    full = np.zeros((T, E))
    for t in range(T):
        for j in range(k):
            if 0 <= idx[t, j] < E:
                full[t, idx[t, j]] += tol[t, j]
    close(f64(out), want, full, "dlogits")
    base = rng.standard_normal((T, E)).astype(np.float32)
    acc = empty(T, E)
    acc.copy_(up(base))
    B.moe_gate_backward(*args, acc, token_mask=up(m), accumulate=True)
    torch.cuda.synchronize()
    close(f64(acc), want + base, full + U * np.abs(want + base), "accumulated")
    guarded()


# --------------------------------------------------------- router gradient --

def checkpoint_of(h, eps):
    """(q, scales, rstd) by the GPU's own norm, and the values they stand for."""
    from sparse_moe_layer_05_b200 import binding as B
    T, d = h.shape
    q, sc = empty(T, d, dtype=torch.uint8), empty(T, d // 32, dtype=torch.uint8)
    rstd = empty(T)
    B.moe_rms_norm_checkpoint(up(h), None, eps, T, d, None, q, sc, rstd)
    torch.cuda.synchronize()
    guarded()
    return q, sc, rstd


ROUTER = [(1, 1, 32), (1, 256, 64), (7, 2, 96), (61, 64, 2880), (128, 16, 128), (300, 248, 352),
          (515, 33, 64), (1000, 128, 320), (2049, 32, 2880), (4097, 130, 192), (6007, 8, 160),
          (777, 256, 1024), (20, 5, 16384)]


def run_router(dl, Wr, rows, mask, dx_in=None, accumulate=None, want=("dW", "db", "dx"), alias=False):
    from sparse_moe_layer_05_b200 import binding as B
    T, E = dl.shape
    d = Wr.shape[1]
    o = {"dW": empty(E, d), "db": empty(E), "dx": empty(T, d, dtype=torch.uint16)}
    if accumulate is not None:
        o["dW"].copy_(up(accumulate[0]))
        o["db"].copy_(up(accumulate[1]))
    di = up(dx_in)
    if alias:
        o["dx"].copy_(di)
        di = o["dx"]
    o = {n: (t if n in want else None) for n, t in o.items()}
    B.moe_router_backward(up(dl), up(Wr), E, T, d, o["dW"], o["db"], o["dx"],
                          ws_of(B.moe_router_backward_workspace_size(E, T, d)), dx_in=di, token_mask=up(mask),
                          accumulate=accumulate is not None, **rows)
    torch.cuda.synchronize()
    guarded()
    return o


def router_tol(dl, Wr, x, live, want, dx_in=None):
    """dW and db: chain(T) additions, each off by at most 2 u (the tensor cores may
    truncate), and the parts' splits and products (16 more). dx: operands in two
    bf16 terms (3 2^-18 of each product), E additions, then one bf16 rounding."""
    T, E = dl.shape
    dW, db, dx = want
    size = R.router_grad(np.abs(dl), np.abs(Wr), np.abs(x), live,
                         None if dx_in is None else np.abs(dx_in))
    c = chain(T) * 2 * U
    return c * size[0] + 1e-38, c * size[1] + 1e-38, BF16 * np.abs(dx) + (2.0 ** -16 + 4 * E * U) * size[2] + 1e-38


@pytest.mark.parametrize("rows", ["bf16", "8bit"])
@pytest.mark.parametrize("T,E,d", ROUTER)
def test_router_gradients(T, E, d, rows):
    rng = np.random.default_rng(T + E + d)
    mask = MASKS[(T + E) % 4] if T > 1 else "none"
    m, live = live_of(mask, T, rng)
    # sizes over several powers of two, as small as a mean loss over the batch gives
    dl = (rng.standard_normal((T, E)) * np.exp2(rng.integers(-6, 3, (T, 1))) / T).astype(np.float32)
    Wr = (rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32)
    dx_in = bits(rng.standard_normal((T, d)) / T) if E % 2 == 0 else None
    if rows == "bf16":
        xb = bits(rng.standard_normal((T, d)) * np.exp2(rng.integers(-3, 4, (T, 1))))
        x = val(xb)
        xb[~live] = 0x7FC0
        src = {"x": up(xb)}
    else:
        h = bits(rng.standard_normal((T, d)) * np.exp2(rng.integers(-8, 9, (T, 1))))
        q, sc, rstd = checkpoint_of(h, 1e-5)
        g = rng.uniform(0.5, 1.5, d).astype(np.float32)
        x = R.checkpoint_rows(q.cpu().numpy(), sc.cpu().numpy()) * f64(rstd)[:, None] * g.astype(np.float64)
        dead = up((~live).astype(np.uint8)).bool()
        q[dead], rstd[dead], sc[dead] = 127, float("nan"), 255
        src = {"q": q, "scales": sc, "rstd": rstd, "g": up(g)}
    dl64 = np.where(live[:, None], dl.astype(np.float64), 0)
    dl[~live] = np.inf
    W64 = Wr.astype(np.float64)
    di64 = None if dx_in is None else val(dx_in)
    want = R.router_grad(dl64, W64, x, live, di64)
    tol = router_tol(dl64, W64, x, live, want, di64)
    o = run_router(dl, Wr, src, m, dx_in)
    for n, w, t in zip(("dW", "db"), want, tol):
        close(f64(o[n]), w, t, n)
    close(val(o["dx"].cpu().numpy()), want[2], tol[2], "dx")
    if (~live).any():
        dead = o["dx"].cpu().numpy()[~live]
        assert np.array_equal(dead, dx_in[~live] if dx_in is not None else np.zeros_like(dead))
    # accumulated, with dx_in in dx's place; the same bits from the same call
    a = rng.standard_normal((E, d)).astype(np.float32), rng.standard_normal(E).astype(np.float32)
    o2 = run_router(dl, Wr, src, m, dx_in, accumulate=a, alias=dx_in is not None)
    close(f64(o2["dW"]), want[0] + a[0], tol[0] + U * np.abs(want[0] + a[0]), "accumulated dW")
    close(f64(o2["db"]), want[1] + a[1], tol[1] + U * np.abs(want[1] + a[1]), "accumulated db")
    assert torch.equal(o2["dx"].view(torch.int16), o["dx"].view(torch.int16))
    o3 = run_router(dl, Wr, src, m, dx_in)
    assert all(torch.equal(o3[n].view(torch.int16), o[n].view(torch.int16)) for n in o)


# every layout of the terms (experts rounded up to 16: 16 .. 128 in one group, two
# groups above), each side of the paths' borders, one 64-column tile and part tiles
LAYOUTS = [(1000, 3, 32), (144, 60, 64), (145, 60, 64), (96, 200, 2880), (97, 200, 2880), (145, 256, 64),
           (1500, 100, 320), (700, 90, 448), (2600, 80, 96), (900, 161, 128), (5000, 200, 64), (1100, 112, 2080),
           (1030, 17, 8256)]


@pytest.mark.parametrize("rows", ["bf16", "8bit"])
@pytest.mark.parametrize("T,E,d", LAYOUTS)
def test_router_gradients_of_every_layout(T, E, d, rows):
    test_router_gradients(T, E, d, rows)


@pytest.mark.parametrize("want", [("dW",), ("db",), ("dx",), ("dW", "db"), ("db", "dx")])
@pytest.mark.parametrize("T,E,d", [(33, 16, 96), (3000, 40, 256)])
def test_router_gradients_by_themselves(T, E, d, want):
    """Each output alone has the bits it has beside the others; without dW the rows
    need not be given."""
    rng = np.random.default_rng(1)
    dl, Wr = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal((E, d)).astype(np.float32)
    x = up(bits(rng.standard_normal((T, d))))
    every = run_router(dl, Wr, {"x": x}, None)
    some = run_router(dl, Wr, {"x": x} if "dW" in want else {}, None, want=want)
    for n in want:
        assert torch.equal(some[n].view(torch.int16), every[n].view(torch.int16)), n


@pytest.mark.parametrize("T,E,d", [(1, 3, 32), (60, 20, 96), (700, 20, 96), (2700, 40, 320), (1500, 200, 64)])
@pytest.mark.parametrize("with_in", [False, True])
def test_a_padded_tokens_dx_stays_under_weights_that_are_no_numbers(T, E, d, with_in):
    """dx of a padded token is its dx_in row, bit for bit, or 0, whatever the weights
    hold; a live token's shows the infinity."""
    rng = np.random.default_rng(T)
    dl, Wr = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal((E, d)).astype(np.float32)
    Wr[0, 5], Wr[E - 1, 9] = np.inf, np.nan
    live = rng.random(T) < 0.7
    live[-1] = T > 1 and T % 2 == 0
    dx_in = bits(np.where(rng.random((T, d)) < 0.2, -0.0, rng.standard_normal((T, d)))) if with_in else None
    o = run_router(dl, Wr, {}, live.astype(np.uint8), dx_in, want=("dx",))["dx"].cpu().numpy()
    assert np.array_equal(o[~live], dx_in[~live] if with_in else 0 * o[~live])
    v = val(o[live])
    assert not np.isfinite(v[:, [5, 9]]).any() and np.isfinite(np.delete(v, [5, 9], 1)).all()


def test_router_gradients_of_values_at_the_types_ends():
    """Gradients near fp32's smallest normal numbers, weights and rows near bf16's
    largest; a zero batch. Terms below 2^-126 are lost: at most 2^-126 each."""
    T, E, d = 200, 24, 64
    rng = np.random.default_rng(9)
    dl = (rng.standard_normal((T, E)) * 2.0 ** -100).astype(np.float32)
    Wr = (rng.standard_normal((E, d)) * 2.0 ** 90).astype(np.float32)
    xb = bits(rng.standard_normal((T, d)) * 2.0 ** 110)
    live = np.ones(T, bool)
    o = run_router(dl, Wr, {"x": up(xb)}, None)
    a = dl.astype(np.float64), Wr.astype(np.float64), val(xb)
    want = R.router_grad(*a, live)
    tol = router_tol(*a, live, want)
    for n, w, t in zip(("dW", "db"), want, tol):
        close(f64(o[n]), w, t, n)
    close(val(o["dx"].cpu().numpy()), want[2], tol[2], "dx")
    o = run_router(0 * dl, Wr, {"x": up(xb)}, None)
    assert not any(f64(t.view(torch.int16)).any() for t in o.values())


# ------------------------------------------------------------------- norms --

NORM = [(1, 32), (3, 64), (61, 2880), (1021, 352), (4099, 96), (33, 4096), (5, 16384), (19, 8224), (700, 2880)]


def hidden(T, d, rng):
    h = rng.standard_normal((T, d)) * np.exp2(rng.integers(-6, 7, (T, 1)))
    h[:, ::97] *= 12
    b = bits(h)
    if T > 2:
        b[1] = 0                                      # a row of zeros
        b[2, : 32] = 0                                # a group of zeros
    return b


@pytest.mark.parametrize("T,d", NORM)
def test_norm_checkpoint(T, d):
    """x is moe_rms_norm's and q, scales moe_mx_quantize's, byte for byte; rstd: a sum
    of squares with chains of d / 32 + 5, its division, root and inverse."""
    from sparse_moe_layer_05_b200 import binding as B
    rng = np.random.default_rng(T + d)
    h, g = hidden(T, d, rng), rng.uniform(0.5, 1.5, d).astype(np.float32)
    ht, gt = up(h), up(g)
    x, q = empty(T, d, dtype=torch.uint16), empty(T, d, dtype=torch.uint8)
    sc, rstd = empty(T, d // 32, dtype=torch.uint8), empty(T)
    B.moe_rms_norm_checkpoint(ht, gt, 1e-5, T, d, x, q, sc, rstd)
    x2, q2, sc2 = torch.empty_like(x), torch.empty_like(q), torch.empty_like(sc)
    B.moe_rms_norm(ht, gt, 1e-5, T, d, x2)
    B.moe_mx_quantize(ht, T, d, B.ACT_MXFP8, q2, sc2)
    torch.cuda.synchronize()
    assert torch.equal(x.view(torch.int16), x2.view(torch.int16))
    assert torch.equal(q, q2) and torch.equal(sc, sc2)
    v = val(h)
    want = 1 / np.sqrt((v * v).mean(1) + np.float32(1e-5))
    close(f64(rstd), want, (d / 64 + 8) * U * want, "rstd")
    q3, sc3, r3 = torch.empty_like(q), torch.empty_like(sc), torch.empty_like(rstd)
    B.moe_rms_norm_checkpoint(ht, None, 1e-5, T, d, None, q3, sc3, r3)
    torch.cuda.synchronize()
    assert torch.equal(q, q3) and torch.equal(sc, sc3) and torch.equal(rstd, r3)
    guarded()


def test_norm_checkpoint_of_values_at_bf16s_ends():
    """Subnormal, largest, infinite and NaN inputs: the same bytes as moe_mx_quantize."""
    from sparse_moe_layer_05_b200 import binding as B
    T, d = 70, 320
    rng = np.random.default_rng(8)
    h = rng.integers(0, 1 << 16, (T, d)).astype(np.uint16)
    h[:30] &= 0x80FF                                  # subnormals and the smallest normals
    h[30:40, ::3] = 0x7F7F
    q, sc, rstd = empty(T, d, dtype=torch.uint8), empty(T, d // 32, dtype=torch.uint8), empty(T)
    q2, sc2 = torch.empty_like(q), torch.empty_like(sc)
    B.moe_rms_norm_checkpoint(up(h), None, 1e-5, T, d, None, q, sc, rstd)
    B.moe_mx_quantize(up(h), T, d, B.ACT_MXFP8, q2, sc2)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(sc, sc2)
    guarded()


@pytest.mark.parametrize("rows", ["bf16", "8bit"])
@pytest.mark.parametrize("T,d", NORM)
def test_norm_backward(T, d, rows):
    """dg: chain(T) additions. dh: the row's mean with chains of at most 64, products
    (8 more), then one bf16 rounding."""
    from sparse_moe_layer_05_b200 import binding as B
    rng = np.random.default_rng(T * 3 + d)
    m, live = live_of(MASKS[(T + d // 32) % 3], T, rng)
    h, g = hidden(T, d, rng), rng.uniform(0.5, 1.5, d).astype(np.float32)
    q, sc, rstd = checkpoint_of(h, 1e-5)
    dx = bits(rng.standard_normal((T, d)) / T)
    dh_in = bits(rng.standard_normal((T, d)) / T) if d % 64 == 0 else None
    v = val(h) if rows == "bf16" else R.checkpoint_rows(q.cpu().numpy(), sc.cpu().numpy())
    r = f64(rstd)
    dxv, g64 = val(dx), g.astype(np.float64)
    want_dh, want_dg = R.rms_norm_grad(dxv, v, r, g64, live, None if dh_in is None else val(dh_in))
    dead = up((~live).astype(np.uint8)).bool()
    dx[~live] = 0x7FC0
    if rows == "bf16":
        h = h.copy()
        h[~live] = 0xFF80
        src = {"h": up(h)}
    else:
        q[dead], sc[dead] = 127, 255
        src = {"q": q, "scales": sc}
    rstd[dead] = float("inf")
    ws = ws_of(B.moe_rms_norm_backward_workspace_size(T, d))

    def run(acc=None, alias=None):
        dh, dg = empty(T, d, dtype=torch.uint16), empty(d)
        a, b = up(dx), up(dh_in)
        if acc is not None:
            dg.copy_(up(acc))
        if alias == "dx":
            dh.copy_(a)
            a = dh
        if alias == "dh_in" and b is not None:
            dh.copy_(b)
            b = dh
        B.moe_rms_norm_backward(a, up(g), rstd, T, d, dh, dg, ws, dh_in=b, token_mask=up(m),
                                accumulate=acc is not None, **src)
        torch.cuda.synchronize()
        guarded()
        return dh, dg

    dh, dg = run()
    n = np.where(live[:, None], v * r[:, None], 0)
    un = np.where(live[:, None], np.abs(dxv) * g64, 0)
    dgtol = chain(T) * U * (np.where(live[:, None], np.abs(dxv), 0) * np.abs(n)).sum(0) + 1e-38
    close(f64(dg), want_dg, dgtol, "dg")
    size = r[:, None] * (un + np.abs(n) * (un * np.abs(n)).mean(1, keepdims=True))
    if dh_in is not None:
        size = size + np.abs(val(dh_in))
    close(val(dh.cpu().numpy()), want_dh, BF16 * np.abs(want_dh) + 72 * U * size + 1e-38, "dh")
    if (~live).any():
        got = dh.cpu().numpy()[~live]
        assert np.array_equal(got, dh_in[~live] if dh_in is not None else np.zeros_like(got))
    acc = rng.standard_normal(d).astype(np.float32)
    dh2, dg2 = run(acc, "dx")
    assert torch.equal(dh2.view(torch.int16), dh.view(torch.int16))
    close(f64(dg2), want_dg + acc, dgtol + U * np.abs(want_dg + acc), "accumulated dg")
    dh3, dg3 = run(None, "dh_in")
    assert torch.equal(dh3.view(torch.int16), dh.view(torch.int16)) and torch.equal(dg3, dg)


# ----------------------------------------------------- no tokens, refusals --

def test_no_tokens():
    from sparse_moe_layer_05_b200 import binding as B
    E, k, d = 6, 2, 64
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")
    stats, counts, mean = empty(4), empty(E, dtype=torch.int32), empty(E)
    B.moe_balance_loss(z(0, E), z(0, k, dtype=torch.int32), E, k, 0, 1.0, 1.0, stats, counts, mean, z(0),
                       ws_of(B.moe_balance_loss_workspace_size(E, k, 0)))
    B.moe_balance_loss_backward(z(0, E), z(0), counts, stats, E, k, 0, 1.0, 1.0, z(0, E))
    B.moe_gate_backward(z(0, d, dtype=torch.bfloat16), z(0, d), z(0, k, dtype=torch.int32), z(0, k), E, k, 0, d,
                        z(0, E))
    dW, db, dg = empty(E, d), empty(E), empty(d)
    B.moe_router_backward(z(0, E), z(E, d), E, 0, d, dW, db, z(0, d, dtype=torch.bfloat16),
                          ws_of(B.moe_router_backward_workspace_size(E, 0, d)), x=z(0, d, dtype=torch.bfloat16))
    B.moe_rms_norm_backward(z(0, d, dtype=torch.bfloat16), z(d), z(0), 0, d, z(0, d, dtype=torch.bfloat16), dg,
                            ws_of(B.moe_rms_norm_backward_workspace_size(0, d)), h=z(0, d, dtype=torch.bfloat16))
    torch.cuda.synchronize()
    for t in (stats, counts, mean, dW, db, dg):
        assert not t.any()
    kept = torch.ones(d, device="cuda")
    B.moe_rms_norm_backward(z(0, d, dtype=torch.bfloat16), z(d), z(0), 0, d, z(0, d, dtype=torch.bfloat16), kept,
                            ws_of(B.moe_rms_norm_backward_workspace_size(0, d)), h=z(0, d, dtype=torch.bfloat16),
                            accumulate=True)
    torch.cuda.synchronize()
    assert bool((kept == 1).all())
    guarded()


def test_no_tokens_leave_a_status():
    from sparse_moe_layer_05_b200 import binding as B
    E, d = 6, 64
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")
    ws = ws_of(B.moe_router_backward_workspace_size(E, 0, d)).fill_(9)
    B.moe_router_backward(z(0, E), z(E, d), E, 0, d, None, None, z(0, d, dtype=torch.bfloat16), ws)
    torch.cuda.synchronize()
    assert not ws[:4].any()


def test_tensors_of_another_size_type_or_place_are_refused():
    from sparse_moe_layer_05_b200 import binding as B
    T, E, k, d = 8, 4, 2, 64
    f = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")
    good = dict(dout=f(T, d, dtype=torch.bfloat16), yw=f(T * k, d), topk_idx=f(T, k, dtype=torch.int32),
                topk_w=f(T, k))
    out = f(T, E)
    for name, bad in [("dout", f(T, d)), ("dout", f(T - 1, d, dtype=torch.bfloat16)), ("yw", f(T * k, 2 * d)[:, ::2]),
                      ("topk_idx", f(T, k, dtype=torch.int64)), ("topk_w", torch.zeros(T, k)),
                      ("yw", None), ("topk_w", f(T * k + 4)[:T * k + 1][1:])]:
        with pytest.raises((ValueError, B.MoEError)):
            B.moe_gate_backward(**{**good, name: bad}, E=E, k=k, T=T, d=d, dlogits=out)
    with pytest.raises(ValueError):
        B.moe_gate_backward(**good, E=E, k=k, T=T, d=d, dlogits=out, token_mask=f(T))
    with pytest.raises(B.MoEError):                   # workspace too small
        B.moe_rms_norm_backward(good["dout"], f(d), f(T), T, d, f(T, d, dtype=torch.bfloat16), f(d),
                                f(16, dtype=torch.uint8), h=good["dout"])
