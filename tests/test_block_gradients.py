"""The gradients of the whole sublayer out = h + MoE(RMSNorm(h)) in h and g: what the
backward calls compute with the experts' share of the gradient as dx_in, and that it
takes that share. In fp64 against difference quotients, then backward_block on the GPU
against the formulas."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import router_train_oracle as R

EPS = 1e-3


def experts_share(dout, x, idx, p, weights):
    """Gradient to the rows x of sum <dout, sum_j p_j y_j(x)>, the p_j held: through
    y = (silu(x Wg^T) * (x Wu^T)) Wd^T of the chosen experts. weights[e] = (Wgu, Wd)."""
    out = np.zeros_like(x)
    for e, (Wgu, Wd) in enumerate(weights):
        I = Wd.shape[1]
        t, j = np.nonzero(idx == e)
        z, u = x[t] @ Wgu[:I].T, x[t] @ Wgu[I:].T
        s = 1 / (1 + np.exp(-z))
        dh = (p[t, j][:, None] * dout[t]) @ Wd
        np.add.at(out, t, (dh * u * s * (1 + z * (1 - s))) @ Wgu[:I] + (dh * z * s) @ Wgu[I:])
    return out


def test_with_the_experts_share_they_are_the_sublayers():
    rng = np.random.default_rng(5)
    T, d, I, E, k = 4, 6, 5, 4, 2
    h, g, dout = rng.standard_normal((T, d)), rng.uniform(0.5, 1.5, d), rng.standard_normal((T, d))
    W, b = rng.standard_normal((E, d)), rng.standard_normal(E)
    weights = [(rng.standard_normal((2 * I, d)) / 2, rng.standard_normal((d, I)) / 2) for _ in range(E)]
    idx = O.topk_select(R.rms_norm(h, g, EPS) @ W.T + b, k)

    def rows(x):
        y = np.empty((T, k, d))
        for t in range(T):
            for j in range(k):
                Wgu, Wd = weights[idx[t, j]]
                y[t, j] = O.expert_out(O.expert_hidden(x[t:t + 1], Wgu, I), Wd)[0]
        return y

    def probs(x):
        return R.softmax(np.take_along_axis(x @ W.T + b, idx, 1))

    def loss(h_, g_):
        x = R.rms_norm(h_, g_, EPS)
        return (dout * (h_ + (probs(x)[:, :, None] * rows(x)).sum(1))).sum()

    def numeric(f, a, step=1e-5):
        out = np.zeros_like(a)
        for i in np.ndindex(*a.shape):
            hi, lo = a.copy(), a.copy()
            hi[i] += step
            lo[i] -= step
            out[i] = (f(hi) - f(lo)) / (2 * step)
        return out

    x, live = R.rms_norm(h, g, EPS), np.ones(T, bool)
    p = probs(x)
    ds = R.gate_grad(dout, (p[:, :, None] * rows(x)).reshape(T * k, d), idx, p, E, live)
    share = experts_share(dout, x, idx, p, weights)
    rstd = 1 / np.sqrt((h * h).mean(1) + EPS)
    whole = R.rms_norm_grad(R.router_grad(ds, W, x, live, share)[2], h, rstd, g, live, dout)
    alone = R.rms_norm_grad(R.router_grad(ds, W, x, live)[2], h, rstd, g, live, dout)
    want = numeric(lambda a: loss(a, g), h), numeric(lambda a: loss(h, a), g)
    for got, without, w in zip(whole, alone, want):
        # step 1e-5: h^2 / 6 f''' and 2^-52 / h of a function of size ten
        assert np.abs(got - w).max() < 1e-8 * max(1.0, np.abs(w).max())
        assert np.abs(without - w).max() > 1e-2 * np.abs(w).max()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [24, 300])
def test_backward_block_takes_the_experts_share(T):
    """dh and dg with dx_in as the formulas have them, bounds as in the step's test (dx:
    its rounding, and what the logits' gradient carries); dW_r, db_r keep their bits."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()
    from tests.test_gpu_router_train import BF16, U, bits, chain, close, f64, up, val
    from tests.test_gpu_router_train_step import make_step
    d, I, E, k = 256, 128, 8, 3
    s = make_step(d, I, E, k, T, seed=61, mask=False)
    layer, inp, gr, ck, t = s["layer"], s["inp"], s["gr"], s["ck"], s["t"]
    layer.forward_block(t["h"], t["g"], EPS, checkpoint=ck)
    layer.backward_block(t["dout"], t["g"], ck, gr)
    torch.cuda.synchronize()
    first = gr.dW_r.clone(), gr.db_r.clone()
    rows = R.checkpoint_rows(ck.q.cpu().numpy(), ck.scales.cpu().numpy())
    rstd, g, dout = f64(ck.rstd), s["g"].astype(np.float64), val(s["dout"])
    x, live, W_r = rows * rstd[:, None] * g, np.ones(T, bool), inp.W_r.astype(np.float64)
    w, idx = f64(layer.intermediate("topk_w", T)), layer.intermediate("topk_idx", T).cpu().numpy()
    weights = [(O.mxfp4_decode(inp.Wgu_codes[e], inp.Wgu_scales[e]),
                O.mxfp4_decode(inp.Wd_codes[e], inp.Wd_scales[e])) for e in range(E)]
    dx_in = bits(experts_share(dout, x, idx, w, weights))
    dh = layer.backward_block(t["dout"], t["g"], ck, gr, dx_in=up(dx_in))
    torch.cuda.synchronize()
    assert torch.equal(gr.dW_r, first[0]) and torch.equal(gr.db_r, first[1])
    yw = f64(layer.intermediate("yw", T))
    ds = R.gate_grad(dout, yw, idx, w, E, live)
    dx = R.router_grad(ds, W_r, x, live, val(dx_in))[2]
    dh64, dg64 = R.rms_norm_grad(dx, rows, rstd, g, live, dout)
    S = np.einsum("td,tkd->tk", np.abs(dout), np.abs(yw.reshape(T, k, d)))
    tds = np.zeros((T, E))
    np.add.at(tds, (np.arange(T)[:, None], idx), (d / 32 + k + 18) * U * (S + w * S.sum(1, keepdims=True)))
    size = np.abs(ds) @ np.abs(W_r) + np.abs(val(dx_in))
    tdx = BF16 * np.abs(dx) + (1 + BF16) * ((2.0 ** -16 + 4 * E * U) * size + tds @ np.abs(W_r)) + 1e-38
    nn, tu = np.abs(rows) * rstd[:, None], tdx * np.abs(g)
    u = np.abs(dx) * np.abs(g) + tu
    move = rstd[:, None] * (tu + nn * (tu * nn).mean(1, keepdims=True))
    full = rstd[:, None] * (u + nn * (u * nn).mean(1, keepdims=True)) + np.abs(dout)
    close(val(dh.cpu().numpy()), dh64, (1 + BF16) * move + BF16 * np.abs(dh64) + 72 * U * full, "dh")
    close(f64(gr.dg), dg64, (tdx * nn).sum(0) + chain(T) * U * (u / np.abs(g) * nn).sum(0), "dg")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [24, 700])
def test_backward_blocks_loss_is_the_operators(T):
    """The step's loss, counts and shares have the bits of moe_balance_loss on the logits
    and choices that the forward pass left."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import binding as B
    from sparse_moe_layer_05_b200 import build
    build.build()
    from tests.test_gpu_router_train_step import A, B_Z, make_step, run_step
    E, k = 8, 2
    s = make_step(352, 224, E, k, T, seed=62)
    run_step(s)
    layer, gr = s["layer"], s["gr"]
    other = B.RouterGrads(E, k, T, 352)
    B.moe_balance_loss(layer.intermediate("logits", T), layer.intermediate("topk_idx", T), E, k, T, A, B_Z,
                       other.stats, other.counts, other.mean_probs, other.lse, other.workspace,
                       token_mask=s["t"]["mask"])
    torch.cuda.synchronize()
    for name in ("stats", "counts", "mean_probs", "lse"):
        assert torch.equal(getattr(gr, name), getattr(other, name)), name
