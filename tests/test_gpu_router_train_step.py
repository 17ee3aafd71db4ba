"""The training step of the sublayer out = h + MoE(RMSNorm(h)) with frozen experts,
as a user runs it: the forward pass that leaves the checkpoint, then the backward
calls one after another; on other streams, in graphs, two at once."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import router_train_oracle as R
from sparse_moe_layer_05_b200 import workloads as W
from tests.test_gpu_router_train import BF16, U, bits, chain, close, f64, up, val

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()


EPS, A, B_Z = 1e-5, 0.02, 0.003


def make_step(d, I, E, k, T, seed, mask=True):
    from sparse_moe_layer_05_b200 import binding as B
    inp = W.make_custom(d, I, E, k, T, seed=seed)
    rng = np.random.default_rng(seed + 1)
    s = dict(inp=inp, layer=B.MoELayer(inp, block=True), ck=B.NormCheckpoint(T, d),
             gr=B.RouterGrads(E, k, T, d))
    s["h"] = bits(val(inp.x) * 3.0 + 0.25)
    s["g"] = rng.uniform(0.5, 1.5, d).astype(np.float32)
    s["dout"] = bits(rng.standard_normal((T, d)) / T)
    s["live"] = rng.random(T) < 0.85 if mask else np.ones(T, bool)
    s["t"] = {n: up(s[n]) for n in ("h", "g", "dout")}
    s["t"]["mask"] = up(s["live"].astype(np.uint8)) if mask else None
    return s


def run_step(s, stream=None, accumulate=False):
    t = s["t"]
    out = s["layer"].forward_block(t["h"], t["g"], EPS, checkpoint=s["ck"], stream=stream)
    dh = s["layer"].backward_block(t["dout"], t["g"], s["ck"], s["gr"], A, B_Z, token_mask=t["mask"],
                                   accumulate=accumulate, stream=stream)
    return out, dh


@pytest.mark.parametrize("d,I,E,k,T", [(2880, 2880, 16, 4, 64), (352, 224, 8, 2, 700), (448, 320, 6, 2, 1300)],
                         ids=["decode_tiles", "bf16_tiles", "pair_tiles"])
def test_step_against_the_formulas(d, I, E, k, T):
    """Every gradient against the fp64 formulas, chained, on the logits, choices,
    weights and rows that the forward pass left. Bounds: dlogits as its own
    operators' tests have them; dx carries dlogits' error through |W_r| and its own
    rounding; dh and dg carry dx's."""
    from sparse_moe_layer_05_b200 import binding as B
    s = make_step(d, I, E, k, T, seed=71)
    layer, inp, live = s["layer"], s["inp"], s["live"]
    out, dh = run_step(s)
    assert B.moe_sync_status(layer.workspace) == 0 and B.moe_sync_status(s["gr"].workspace) == 0
    # the same output bits as without the checkpoint, whose rows are the conversion's
    plain = B.MoELayer(inp, block=True).forward_block(s["t"]["h"], s["t"]["g"], EPS)
    assert torch.equal(out.view(torch.int16), plain.view(torch.int16))
    q2, sc2 = torch.empty_like(s["ck"].q), torch.empty_like(s["ck"].scales)
    B.moe_mx_quantize(s["t"]["h"], T, d, B.ACT_MXFP8, q2, sc2)
    torch.cuda.synchronize()
    assert torch.equal(q2, s["ck"].q) and torch.equal(sc2, s["ck"].scales)

    logits, w, yw = (f64(layer.intermediate(n, T)) for n in ("logits", "topk_w", "yw"))
    idx = layer.intermediate("topk_idx", T).cpu().numpy()
    rows = R.checkpoint_rows(s["ck"].q.cpu().numpy(), s["ck"].scales.cpu().numpy())
    rstd, g, dout, W_r = f64(s["ck"].rstd), s["g"].astype(np.float64), val(s["dout"]), inp.W_r.astype(np.float64)
    a, b = float(np.float32(A)), float(np.float32(B_Z))
    ds = R.gate_grad(dout, yw, idx, w, E, live) + R.balance_loss_grad(logits, idx, k, a, b, live)
    x = rows * rstd[:, None] * g
    dW, db, dx = R.router_grad(ds, W_r, x, live)
    dh64, dg = R.rms_norm_grad(dx, rows, rstd, g, live, dout)

    S = np.einsum("td,tkd->tk", np.abs(dout), np.abs(yw.reshape(T, k, d))) * live[:, None]
    gate = np.zeros((T, E))
    np.add.at(gate, (np.arange(T)[:, None], idx), (d / 32 + k + 18) * U * (S + w * S.sum(1, keepdims=True)))
    p, n = R.softmax(logits), live.sum()
    f = R.expert_counts(idx, E, live) / (n * k)
    bal = 256 * U / n * p * (a * E * (f + (p @ f)[:, None]) + 2 * b * np.abs(R.log_sum_exp(logits))[:, None])
    tds = np.where(live[:, None], gate + bal + U * np.abs(ds), 0)
    close(f64(s["gr"].dlogits), ds, tds + 1e-38, "dlogits")
    size = R.router_grad(np.abs(ds), np.abs(W_r), np.abs(x), live)
    carried = R.router_grad(tds, np.abs(W_r), np.abs(x), live)
    c = chain(T) * 2 * U
    close(f64(s["gr"].dW_r), dW, c * size[0] + carried[0], "dW_r")
    close(f64(s["gr"].db_r), db, c * size[1] + carried[1], "db_r")
    tdx = BF16 * np.abs(dx) + (2.0 ** -16 + 4 * E * U) * size[2] + (1 + BF16) * carried[2] + 1e-38
    nn = np.where(live[:, None], np.abs(rows) * rstd[:, None], 0)
    # a padded token's dx row is zero: nothing reaches dh or dg from it
    tu = np.where(live[:, None], tdx, 0) * np.abs(g)
    u = np.where(live[:, None], np.abs(dx), 0) * np.abs(g) + tu
    move = rstd[:, None] * (tu + nn * (tu * nn).mean(1, keepdims=True))
    full = rstd[:, None] * (u + nn * (u * nn).mean(1, keepdims=True)) + np.abs(dout)
    close(val(dh.cpu().numpy()), dh64, (1 + BF16) * move + BF16 * np.abs(dh64) + 72 * U * full, "dh")
    close(f64(s["gr"].dg), dg, ((np.where(live[:, None], tdx, 0) * nn).sum(0)
                                + chain(T) * U * (u / np.abs(g) * nn).sum(0)), "dg")
    (loss, bl, z, nl), counts, mean, lse = R.balance_loss(logits, idx, k, a, b, live)
    assert s["gr"].counts.cpu().numpy().tolist() == counts.tolist()
    close(f64(s["gr"].stats), np.array([loss, bl, z, nl]), 1e-4 * np.array([loss, bl, z, 0]), "stats")
    # accumulated over a second pass of the same batch: twice the gradients
    first = [t.clone() for t in (s["gr"].dW_r, s["gr"].db_r, s["gr"].dg)]
    run_step(s, accumulate=True)
    torch.cuda.synchronize()
    for one, two in zip(first, (s["gr"].dW_r, s["gr"].db_r, s["gr"].dg)):
        assert torch.equal(one + one, two)


def test_router_gradient_is_the_difference_quotient_of_the_layer():
    """The loss <dout, MoE(x)> of the fp64 layer along the gradient's own direction,
    the choice of experts unchanged: the difference quotient (error below 1e-6 of the
    slope here) is |grad|^2 once the rows that the kernel read (the layer's, whose
    experts run in bf16) are replaced by the fp64 layer's: sum (ds64 - ds) slope, ds
    by the formula on either rows. What is left are the kernels' fp32 roundings."""
    from sparse_moe_layer_05_b200 import binding as B
    d, I, E, k, T = 256, 128, 8, 3, 24
    inp = W.make_custom(d, I, E, k, T, seed=77)
    layer = B.MoELayer(inp)
    rng = np.random.default_rng(78)
    dout = bits(rng.standard_normal((T, d)) / T)
    layer.forward(up(inp.x))
    ds = torch.empty((T, E), device="cuda")
    B.moe_gate_backward(up(dout), layer.intermediate("yw", T), layer.intermediate("topk_idx", T),
                        layer.intermediate("topk_w", T), E, k, T, d, ds)
    dW, db = torch.empty((E, d), device="cuda"), torch.empty(E, device="cuda")
    B.moe_router_backward(ds, layer.W_r, E, T, d, dW, db, None,
                          torch.empty(B.moe_router_backward_workspace_size(E, T, d), dtype=torch.uint8,
                                      device="cuda"), x=up(inp.x))
    torch.cuda.synchronize()
    gW, gb = f64(dW), f64(db)
    size = np.sqrt((gW ** 2).sum() + (gb ** 2).sum())
    step = 1e-4 / size

    def loss(sign):
        W_r, b_r = inp.W_r + sign * step * gW, inp.b_r + sign * step * gb
        out = O.moe_forward(inp.x, W_r, b_r, inp.Wgu_codes, inp.Wgu_scales, inp.Wd_codes, inp.Wd_scales, k=k)
        return (out * val(dout)).sum(), np.sort(np.argsort(-(val(inp.x) @ W_r.T + b_r), axis=1)[:, :k], axis=1)

    (hi, ih), (lo, il) = loss(1), loss(-1)
    assert np.array_equal(ih, il)                      # no expert changed on the way
    want = (hi - lo) / (2 * step)
    yw = f64(layer.intermediate("yw", T))
    w, idx = f64(layer.intermediate("topk_w", T)), layer.intermediate("topk_idx", T).cpu().numpy()
    x, live = val(inp.x), np.ones(T, bool)
    r = O.route(inp.x, inp.W_r, inp.b_r, k)
    assert np.array_equal(r.idx, idx)
    exact = np.zeros((T, k, d))
    for e in range(E):
        t, j = np.nonzero(idx == e)
        rows = O.expert_out(O.expert_hidden(x[t], O.mxfp4_decode(inp.Wgu_codes[e], inp.Wgu_scales[e]), I),
                            O.mxfp4_decode(inp.Wd_codes[e], inp.Wd_scales[e]))
        exact[t, j] = r.p[t, j][:, None] * rows
    ds_read = R.gate_grad(val(dout), yw, idx, w, E, live)
    ds_exact = R.gate_grad(val(dout), exact.reshape(T * k, d), idx, r.p, E, live)
    slope = x @ gW.T + gb                              # change of each logit along the gradient
    moved = ((ds_exact - ds_read) * slope).sum()
    S = np.einsum("td,tkd->tk", np.abs(val(dout)), np.abs(yw.reshape(T, k, d)))
    tol = ((d / 32 + k + 18) * U * (S + w * S.sum(1, keepdims=True)) * np.abs(np.take_along_axis(slope, idx, 1))).sum()
    tol += chain(T) * 2 * U * (np.abs(ds_read).T @ np.abs(x) * np.abs(gW)).sum()
    assert tol < 1e-3 * size ** 2 and abs(moved) < 0.05 * size ** 2
    assert abs(want - size ** 2 - moved) <= tol + 1e-6 * size ** 2, (want, size ** 2, moved, tol)


def outputs(s, dh):
    g = s["gr"]
    return [t.clone() for t in (g.dW_r, g.db_r, g.dg, g.dlogits, g.stats, g.mean_probs, g.counts,
                                dh.view(torch.int16))]


@pytest.mark.parametrize("T", [64, 900])
def test_step_on_a_side_stream_and_in_a_graph(T):
    """The same bits on another stream than the current one, and from a captured
    graph replayed on inputs that came after the capture; a second graph shares the
    workspaces."""
    s = make_step(352, 224, 8, 2, T, seed=81)
    _, dh = run_step(s)
    torch.cuda.synchronize()
    want = outputs(s, dh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, dh = run_step(s, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outputs(s, dh), want))
    graphs, dhs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _, dh = run_step(s)
        graphs.append(g)
        dhs.append(dh)
    h, dout = s["t"]["h"].clone(), s["t"]["dout"].clone()
    s["t"]["h"].copy_(torch.flip(h, [0]))
    s["t"]["dout"].copy_(torch.flip(dout, [0]))
    graphs[0].replay()
    torch.cuda.synchronize()
    other = outputs(s, dhs[0])
    assert not torch.equal(other[0], want[0])
    s["t"]["h"].copy_(h)
    s["t"]["dout"].copy_(dout)
    for g, d in ((graphs[1], dhs[1]), (graphs[0], dhs[0]), (graphs[1], dhs[1])):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs(s, d), want))


def test_two_steps_at_once():
    """Two layers' steps on two streams, interleaved call by call."""
    steps = [make_step(352, 224, 8, 2, 900, seed=91 + i) for i in range(2)]
    want = []
    for s in steps:
        _, dh = run_step(s)
        torch.cuda.synchronize()
        want.append(outputs(s, dh))
    streams = [torch.cuda.Stream() for _ in steps]
    for x in streams:
        x.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        dhs = [run_step(s, stream=x)[1] for s, x in zip(steps, streams)]
    torch.cuda.synchronize()
    for s, dh, w in zip(steps, dhs, want):
        assert all(torch.equal(a, b) for a, b in zip(outputs(s, dh), w))


def test_shorter_batches_leave_the_rows_behind_them():
    """A batch of fewer tokens than the buffers hold: rows behind the last token stay."""
    s = make_step(352, 224, 8, 2, 300, seed=95, mask=False)
    gr, ck, T = s["gr"], s["ck"], 77
    gr.dlogits.fill_(5)
    gr.lse.fill_(5)
    ck.q.fill_(9)
    ck.scales.fill_(9)
    ck.rstd.fill_(9)
    gr.dx.view(torch.int16).fill_(9)
    h, dout = s["t"]["h"][:T], s["t"]["dout"][:T]
    s["layer"].forward_block(h, s["t"]["g"], EPS, checkpoint=ck)
    s["layer"].backward_block(dout, s["t"]["g"], ck, gr, A, B_Z)
    torch.cuda.synchronize()
    assert bool((gr.dlogits[T:] == 5).all()) and bool((gr.lse[T:] == 5).all())
    assert bool((ck.q[T:] == 9).all()) and bool((ck.scales[T:] == 9).all()) and bool((ck.rstd[T:] == 9).all())
    assert bool((gr.dx.view(torch.int16)[T:] == 9).all())
    with pytest.raises(ValueError):
        s["layer"].backward_block(torch.empty((301, 352), dtype=torch.uint16, device="cuda"), s["t"]["g"], ck, gr)
