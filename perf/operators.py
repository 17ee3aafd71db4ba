"""The operators that train the layer's router, each as one measurable pass.

Four kinds of case, which one training step of the MoE sublayer with frozen
experts runs one after another:

  balance   the load-balance and z loss of a batch's router logits, the
            per-expert counts, and the loss's gradient to the logits
  gate      the gradient that reaches the logits through the selected-set
            softmax, from the layer's output gradient and the weighted expert
            rows that the forward pass left behind
  router    the gradients of the router's weights, bias and input rows, the
            rows either as bf16 or rebuilt from an 8-bit checkpoint
  norm      the RMSNorm in front of the router: forward with the 8-bit
            checkpoint of its input ("fwd"), and backward ("bwd") from that
            checkpoint or from bf16 rows

``run`` computes a case in plain torch operations, or with ``own`` set through
the package's entry points. Inputs come from the seed alone.
"""
import math

import torch

own = False

BALANCE_COEF, Z_COEF = 1e-2, 1e-3
EPS = 1e-5
_binding = None


def listed():
    return [
        # a 64-token micro batch on the 64-expert top-8 layer: launches and latency
        {"name": "balance_64a8_T64", "op": "balance", "T": 64, "E": 64, "k": 8, "mask": False},
        # the largest logits array of the workloads, with padded tokens
        {"name": "balance_128a4_T16384", "op": "balance", "T": 16384, "E": 128, "k": 4, "mask": True},
        # many experts, an odd token count
        {"name": "balance_248a20_T4093", "op": "balance", "T": 4093, "E": 248, "k": 20, "mask": False},
        # micro batch: few tokens, the row dot products split over the SMs
        {"name": "gate_64a8_T64", "op": "gate", "T": 64, "E": 64, "k": 8, "d": 2880, "mask": False},
        # the 20b layer's training batch
        {"name": "gate_20b_T8192", "op": "gate", "T": 8192, "E": 32, "k": 4, "d": 2880, "mask": False},
        # twenty expert rows per token, with padding: the largest read of all
        {"name": "gate_248a20_T4096", "op": "gate", "T": 4096, "E": 248, "k": 20, "d": 2880, "mask": True},
        # ragged micro batch
        {"name": "router_64a8_T61", "op": "router", "T": 61, "E": 64, "d": 2880, "rows": "bf16",
         "dx_in": False, "mask": False},
        # the 20b layer, the experts' share of dx added in the same pass
        {"name": "router_20b_T8192", "op": "router", "T": 8192, "E": 32, "d": 2880, "rows": "bf16",
         "dx_in": True, "mask": False},
        # 128 experts, input rows rebuilt from the 8-bit checkpoint, padded tokens
        {"name": "router_128a4_T16384", "op": "router", "T": 16384, "E": 128, "d": 2880, "rows": "8bit",
         "dx_in": False, "mask": True},
        # the sublayer's norm at the 20b batch: forward with the checkpoint
        {"name": "norm_fwd_T8192", "op": "norm", "way": "fwd", "T": 8192, "d": 2880, "rows": "8bit",
         "mask": False},
        # its backward from the 8-bit rows, with the residual's gradient
        {"name": "norm_bwd_8bit_T8192", "op": "norm", "way": "bwd", "T": 8192, "d": 2880, "rows": "8bit",
         "mask": False},
        # odd rows of a narrow layer, bf16 rows, padded tokens
        {"name": "norm_bwd_bf16_T1021", "op": "norm", "way": "bwd", "T": 1021, "d": 352, "rows": "bf16",
         "mask": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["balance", "gate", "router", "norm"])
    T = _spread(rng, 1, 16384)
    E = _spread(rng, 2, 248)
    k = _spread(rng, 1, min(E, 20))
    d = 32 * rng.randint(2, 90)
    mask = rng.random() < 0.5
    if op == "balance":
        return {"op": op, "T": min(T, 16384 * 128 // E), "E": E, "k": k, "mask": mask}
    if op == "gate":      # one expert alone has weight 1 and no gradient
        k = max(k, 2)
        return {"op": op, "T": min(T, 4096 * 20 * 2880 // (k * d)), "E": E, "k": k, "d": d, "mask": mask}
    if op == "router":
        return {"op": op, "T": min(T, 16384 * 128 // E), "E": E, "d": d, "rows": rng.choice(["bf16", "8bit"]),
                "dx_in": rng.random() < 0.5, "mask": mask}
    return {"op": op, "way": rng.choice(["fwd", "bwd"]), "T": T, "d": d, "rows": rng.choice(["bf16", "8bit"]),
            "mask": mask}


# ------------------------------------------------------------------ inputs ----

def _to_mx8(h):
    """[T, d] bf16 -> E4M3 values of groups of 32 and their power-of-two scales."""
    v = h.float().view(h.shape[0], -1, 32)
    amax = v.abs().amax(2, keepdim=True)
    e = torch.frexp(amax)[1].float() - 1.0                      # floor(log2 amax)
    x = torch.where(amax > 0, (e - 8.0).clamp(min=-127.0), torch.zeros_like(e))
    q = (v * torch.exp2(-x)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(h.shape), torch.exp2(x).view(h.shape[0], -1).to(torch.float8_e8m0fnu)


def _hidden(T, d, gen):
    """Rows of a residual stream: N(0, 1) times a size of each row, a few strong channels."""
    size = torch.exp(0.5 * torch.randn(T, 1, device="cuda", generator=gen))
    chan = torch.ones(d, device="cuda")
    chan[::97] = 12.0
    return (torch.randn(T, d, device="cuda", generator=gen) * size * chan).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = case["T"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = dict(case)
    s["live"] = None
    if case["mask"]:      # padded tokens, at least one token left
        s["live"] = (torch.rand(T, device="cuda", generator=gen) < 0.9).to(torch.uint8)
        s["live"][0] = 1
    if case["op"] in ("balance", "gate"):
        E, k = case["E"], case["k"]
        s["logits"] = randn(T, E) + 0.3 * randn(E)
        top = s["logits"].topk(k, dim=1)
        s["idx"] = top.indices.int()
        s["w"] = torch.softmax(top.values, 1)
    if case["op"] == "balance":
        s["dloss"] = torch.rand(1, device="cuda", generator=gen) + 0.5
    if case["op"] == "gate":
        # dout of a mean loss over the batch; expert rows already times their weight
        s["dout"] = (randn(T, case["d"]) / T).bfloat16()
        s["yw"] = torch.randn(T * k, case["d"], device="cuda", generator=gen)
        s["yw"] *= s["w"].reshape(-1, 1)
    if case["op"] == "router":
        E, d = case["E"], case["d"]
        p = torch.softmax(randn(T, E), 1)
        s["dlogits"] = (randn(T, E) * p + 1e-2 * p) / T
        s["W_r"] = randn(E, d) / math.sqrt(d)
        s["dx_in"] = (randn(T, d) / T).bfloat16() if case["dx_in"] else None
    if case["op"] in ("router", "norm"):
        d = case["d"]
        s["g"] = 1.0 + 0.1 * randn(d)
        s["h"] = _hidden(T, d, gen)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["q"], s["scale"] = _to_mx8(s["h"])
        if case["op"] == "router":
            s["x"] = (s["h"].float() * s["rstd"][:, None] * s["g"]).bfloat16()
    if case["op"] == "norm":
        s["dx"] = (randn(T, case["d"]) / T).bfloat16()
        s["dh_in"] = (randn(T, case["d"]) / T).bfloat16()
    return s


# --------------------------------------------------------------- plain form ----

def _live_rows(s, a):
    """`a` with the rows of padded tokens as zeros."""
    return a if s["live"] is None else torch.where(s["live"].bool()[:, None], a, torch.zeros_like(a))


def _rows(s):
    """[T, d] fp32 rows of the norm's input as the checkpoint holds them."""
    if s["rows"] == "bf16":
        return s["h"].float()
    return (s["q"].float().view(s["T"], -1, 32) * s["scale"].float()[:, :, None]).view(s["T"], -1)


def _balance(s):
    T, E, k = s["T"], s["E"], s["k"]
    live = torch.ones(T, device="cuda") if s["live"] is None else s["live"].float()
    n = live.sum()
    top = s["logits"].amax(1, keepdim=True)
    ex = (s["logits"] - top).exp()
    total = ex.sum(1, keepdim=True)
    p = ex / total
    lse = (top + total.log()).squeeze(1) * live
    chosen = (s["idx"].long()[:, :, None] == torch.arange(E, device="cuda")).sum(1)
    counts = (chosen * live[:, None].long()).sum(0)
    share = counts.float() / (n * k)
    mean = (p * live[:, None]).double().sum(0) / n
    balance = E * (share * mean).sum()
    z = lse.square().double().sum() / n
    loss = BALANCE_COEF * balance + Z_COEF * z
    c = s["dloss"] * live[:, None] / n
    d = p * (BALANCE_COEF * E * (share - (p * share).sum(1, keepdim=True)) + Z_COEF * 2.0 * lse[:, None]) * c
    return {"stats": torch.stack([loss, balance, z, n.double()]).float(), "counts": counts.int(),
            "mean_probs": mean.float(), "lse": lse, "dlogits": d}


def _gate(s):
    T, E, k, d = s["T"], s["E"], s["k"], s["d"]
    a = (s["dout"].float()[:, None, :] * s["yw"].view(T, k, d)).sum(2)
    da = _live_rows(s, a - s["w"] * a.sum(1, keepdim=True))
    out = torch.zeros(T, E, device="cuda")
    out.scatter_(1, s["idx"].long(), da)
    return {"dlogits": out}


def _router(s):
    dl = _live_rows(s, s["dlogits"])
    x = s["x"].float() if s["rows"] == "bf16" else _rows(s) * s["rstd"][:, None] * s["g"]
    dx = dl @ s["W_r"]
    if s["dx_in"] is not None:
        dx = dx + s["dx_in"].float()
    return {"dW": dl.t() @ _live_rows(s, x), "db": dl.sum(0), "dx": dx.bfloat16()}


def _norm_fwd(s):
    h = s["h"].float()
    rstd = 1.0 / (h.square().mean(1) + EPS).sqrt()
    q, scale = _to_mx8(s["h"])
    return {"x": (h * rstd[:, None] * s["g"]).bfloat16(), "q": q, "scale": scale, "rstd": rstd}


def _norm_bwd(s):
    n = _rows(s) * s["rstd"][:, None]
    dx = s["dx"].float()
    dn = dx * s["g"]
    dh = _live_rows(s, s["rstd"][:, None] * (dn - n * (dn * n).mean(1, keepdim=True)))
    return {"dh": (dh + s["dh_in"].float()).bfloat16(), "dg": _live_rows(s, dx * n).sum(0)}


# -------------------------------------------------------------- the package ----

def _buffers(B, s):
    """What a training program allocates once for a shape: outputs and workspaces."""
    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    T, op = s["T"], s["op"]
    if op in ("balance", "gate"):
        s["o_dlogits"] = empty(T, s["E"])
    if op == "balance":
        s["o_stats"], s["o_mean"], s["o_lse"] = empty(4), empty(s["E"]), empty(T)
        s["o_counts"] = empty(s["E"], dtype=torch.int32)
        s["ws"] = empty(B.moe_balance_loss_workspace_size(s["E"], s["k"], T), dtype=torch.uint8)
    if op == "router":
        s["o_dW"], s["o_db"] = empty(s["E"], s["d"]), empty(s["E"])
        s["o_dx"] = empty(T, s["d"], dtype=torch.bfloat16)
        s["ws"] = empty(B.moe_router_backward_workspace_size(s["E"], T, s["d"]), dtype=torch.uint8)
    if op == "norm":
        s["o_x"] = empty(T, s["d"], dtype=torch.bfloat16)
        s["o_q"] = empty(T, s["d"], dtype=torch.uint8)
        s["o_scale"] = empty(T, s["d"] // 32, dtype=torch.uint8)
        s["o_rstd"], s["o_dg"] = empty(T), empty(s["d"])
        s["o_dh"] = empty(T, s["d"], dtype=torch.bfloat16)
        s["ws"] = empty(B.moe_rms_norm_backward_workspace_size(T, s["d"]), dtype=torch.uint8)
    s["ready"] = True


def _own(s):
    global _binding
    if _binding is None:
        from sparse_moe_layer_05_b200 import binding
        _binding = binding
    B = _binding
    if "ready" not in s:
        _buffers(B, s)
    T, op = s["T"], s["op"]
    if op == "balance":
        B.moe_balance_loss(s["logits"], s["idx"], s["E"], s["k"], T, BALANCE_COEF, Z_COEF, s["o_stats"],
                           s["o_counts"], s["o_mean"], s["o_lse"], s["ws"], token_mask=s["live"])
        B.moe_balance_loss_backward(s["logits"], s["o_lse"], s["o_counts"], s["o_stats"], s["E"], s["k"], T,
                                    BALANCE_COEF, Z_COEF, s["o_dlogits"], dloss=s["dloss"],
                                    token_mask=s["live"])
        return {"stats": s["o_stats"], "counts": s["o_counts"], "mean_probs": s["o_mean"], "lse": s["o_lse"],
                "dlogits": s["o_dlogits"]}
    if op == "gate":
        B.moe_gate_backward(s["dout"], s["yw"], s["idx"], s["w"], s["E"], s["k"], T, s["d"], s["o_dlogits"],
                            token_mask=s["live"])
        return {"dlogits": s["o_dlogits"]}
    if op == "router":
        if s["rows"] == "bf16":
            B.moe_router_backward(s["dlogits"], s["W_r"], s["E"], T, s["d"], s["o_dW"], s["o_db"], s["o_dx"],
                                  s["ws"], x=s["x"], dx_in=s["dx_in"], token_mask=s["live"])
        else:
            B.moe_router_backward(s["dlogits"], s["W_r"], s["E"], T, s["d"], s["o_dW"], s["o_db"], s["o_dx"],
                                  s["ws"], q=s["q"], scales=s["scale"], rstd=s["rstd"], g=s["g"],
                                  dx_in=s["dx_in"], token_mask=s["live"])
        return {"dW": s["o_dW"], "db": s["o_db"], "dx": s["o_dx"]}
    if s["way"] == "fwd":
        B.moe_rms_norm_checkpoint(s["h"], s["g"], EPS, T, s["d"], s["o_x"], s["o_q"], s["o_scale"], s["o_rstd"])
        return {"x": s["o_x"], "q": s["o_q"].view(torch.float8_e4m3fn),
                "scale": s["o_scale"].view(torch.float8_e8m0fnu), "rstd": s["o_rstd"]}
    if s["rows"] == "bf16":
        B.moe_rms_norm_backward(s["dx"], s["g"], s["rstd"], T, s["d"], s["o_dh"], s["o_dg"], s["ws"], h=s["h"],
                                dh_in=s["dh_in"], token_mask=s["live"])
    else:
        B.moe_rms_norm_backward(s["dx"], s["g"], s["rstd"], T, s["d"], s["o_dh"], s["o_dg"], s["ws"], q=s["q"],
                                scales=s["scale"], dh_in=s["dh_in"], token_mask=s["live"])
    return {"dh": s["o_dh"], "dg": s["o_dg"]}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _norm_fwd(state) if state["way"] == "fwd" else _norm_bwd(state)
    return {"balance": _balance, "gate": _gate, "router": _router}[state["op"]](state)


# --------------------------------------------------------------------- work ----

def work(case):
    T = case["T"]
    live = T if case["mask"] else 0
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        return {"bytes": T * (8 * E + 4 * k + 4) + live + 8 * E, "flops": 14 * T * E}
    if case["op"] == "gate":
        E, k, d = case["E"], case["k"], case["d"]
        return {"bytes": T * (4 * k * d + 2 * d + 8 * k + 4 * E) + live, "flops": 2 * T * k * d}
    d = case["d"]
    if case["op"] == "router":
        E = case["E"]
        rows = 2 * d if case["rows"] == "bf16" else d + d // 32 + 4
        return {"bytes": T * (rows + 2 * d + (2 * d if case["dx_in"] else 0) + 4 * E) + live + 8 * E * d,
                "flops": 4 * T * E * d}
    if case["way"] == "fwd":
        return {"bytes": T * (2 * d + 2 * d + d + d // 32 + 4) + 4 * d, "flops": 6 * T * d}
    rows = 2 * d if case["rows"] == "bf16" else d + d // 32
    return {"bytes": T * (rows + 6 * d + 4) + live + 8 * d, "flops": 9 * T * d}


# -------------------------------------------------------------------- exact ----

def exact(case, seed):
    """From the definitions in 64 bits; gradients by differentiating the forward formula."""
    s = prepare(case, seed)
    T = s["T"]
    keep = torch.arange(T, device="cuda") if s["live"] is None else s["live"].nonzero().squeeze(1)

    def whole(part, width):
        out = torch.zeros(T, width, dtype=torch.float64, device="cuda")
        out[keep] = part
        return out

    if s["op"] == "balance":
        E, k = s["E"], s["k"]
        logits = s["logits"][keep].double().requires_grad_()
        lse = torch.logsumexp(logits, 1)
        mean = torch.softmax(logits, 1).mean(0)
        counts = torch.bincount(s["idx"][keep].reshape(-1).long(), minlength=E)
        balance = E * (mean * counts.double() / (len(keep) * k)).sum()
        z = (lse ** 2).mean()
        loss = BALANCE_COEF * balance + Z_COEF * z
        (loss * s["dloss"].double().sum()).backward()
        stats = torch.stack([loss, balance, z, torch.tensor(float(len(keep)), device="cuda").double()])
        return {"stats": stats.detach(), "counts": counts, "mean_probs": mean.detach(),
                "lse": whole(lse.detach()[:, None], 1).squeeze(1), "dlogits": whole(logits.grad, E)}
    if s["op"] == "gate":
        E, k, d = s["E"], s["k"], s["d"]
        # out = sum_j p_j y_j with y_j = yw_j / w_j, p the softmax of the chosen logits
        chosen = s["logits"].gather(1, s["idx"].long()).double().requires_grad_()
        p = torch.softmax(chosen, 1)
        dots = torch.einsum("td,tkd->tk", s["dout"].double(), s["yw"].view(T, k, d).double())
        ((p / s["w"].double()) * dots)[keep].sum().backward()
        out = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        return {"dlogits": out.scatter(1, s["idx"].long(), chosen.grad)}
    d = s["d"]
    h = s["h"].double()
    if s["rows"] == "8bit" and not (s["op"] == "norm" and s["way"] == "fwd"):
        h = s["q"].to(torch.float64) * s["scale"].to(torch.float64).repeat_interleave(32, 1)
    if s["op"] == "router":
        x = s["x"].double() if s["rows"] == "bf16" else h * s["rstd"].double()[:, None] * s["g"].double()
        x = x[keep].requires_grad_()
        W = s["W_r"].double().requires_grad_()
        b = torch.zeros(s["E"], dtype=torch.float64, device="cuda", requires_grad=True)
        ((x @ W.t() + b) * s["dlogits"][keep].double()).sum().backward()
        dx = whole(x.grad, d)
        if s["dx_in"] is not None:
            dx = dx + s["dx_in"].double()
        return {"dW": W.grad, "db": b.grad, "dx": dx}
    if s["way"] == "fwd":
        rstd = (h.square().mean(1) + EPS).rsqrt()
        groups = h.view(T, -1, 32)
        amax = groups.abs().amax(2, keepdim=True)
        # amax = m 2^e with m in [0.5, 1): its binade starts at 2^(e - 1)
        one = torch.ones_like(amax)
        scale = torch.where(amax > 0, torch.ldexp(one, torch.frexp(amax)[1] - 9), one)
        v = groups / scale
        step = torch.ldexp(torch.ones_like(v), torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 4)   # E4M3's spacing at v
        q = ((v / step).round() * step).clamp(-448, 448)
        return {"x": h * rstd[:, None] * s["g"].double(), "q": q.view(T, d), "scale": scale.view(T, -1), "rstd": rstd}
    # x = g n with n = h rstd(h): its Jacobian, with the kept rstd
    r = s["rstd"].double()[:, None]
    n = h * r
    u = s["dx"].double() * s["g"].double()
    dh = r * (u - n * ((u * n).sum(1, keepdim=True) / d))
    return {"dh": whole(dh[keep], d) + s["dh_in"].double(), "dg": (s["dx"].double() * n)[keep].sum(0)}
