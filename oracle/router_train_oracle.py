"""fp64 oracle of the router's training step (test infrastructure; shares no
code with the CUDA path). Rows of a padded batch are left out by `live`, a
boolean array over the tokens. Every gradient here is the formula; the tests
compare each against central differences of the function it belongs to."""
import numpy as np


def log_sum_exp(s):
    """Row-wise log sum exp; -inf for a row of nothing but -inf."""
    m = s.max(axis=1)
    base = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        return base + np.log(np.exp(s - base[:, None]).sum(axis=1))


def softmax(s):
    """Row-wise softmax over all experts; a row of nothing but -inf gives zeros."""
    lse = log_sum_exp(s)
    empty = np.isneginf(lse)
    return np.where(empty[:, None], 0.0, np.exp(s - np.where(empty, 0.0, lse)[:, None]))


def expert_counts(idx, E, live):
    """Live pairs per expert; indices outside 0..E-1 are not counted."""
    chosen = idx[live].reshape(-1)
    return np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)


def balance_loss(s, idx, k, balance_coef, z_coef, live):
    """(loss, balance, z, n), counts, mean probabilities, lse per token."""
    T, E = s.shape
    n = int(live.sum())
    counts = expert_counts(idx, E, live)
    lse = np.zeros(T)
    lse[live] = log_sum_exp(s[live])
    if n == 0:
        return (0.0, 0.0, 0.0, 0), counts, np.zeros(E), lse
    mean = softmax(s[live]).sum(axis=0) / n
    balance = E * float((counts / (n * k) * mean).sum())
    z = float(np.where(np.isneginf(lse[live]), 0.0, lse[live]) ** 2 @ np.ones(n)) / n
    return (balance_coef * balance + z_coef * z, balance, z, n), counts, mean, lse


def balance_loss_grad(s, idx, k, balance_coef, z_coef, live, dloss=1.0):
    T, E = s.shape
    n = int(live.sum())
    out = np.zeros((T, E))
    if n == 0:
        return out
    f = expert_counts(idx, E, live) / (n * k)
    p = softmax(s[live])
    lse = log_sum_exp(s[live])
    lse = np.where(np.isneginf(lse), 0.0, lse)[:, None]
    out[live] = dloss / n * p * (balance_coef * E * (f - (p @ f)[:, None]) + 2.0 * z_coef * lse)
    return out


def gate_dots(dout, yw, k):
    """A[t, j] = <dout_t, yw_{t k + j}>."""
    T, d = dout.shape
    return np.einsum("td,tkd->tk", dout, yw.reshape(T, k, d))


def gate_grad(dout, yw, idx, w, E, live):
    T, k = idx.shape
    A = gate_dots(np.where(live[:, None], dout, 0.0),
                  np.where(np.repeat(live, k)[:, None], yw, 0.0), k)
    g = A - w * A.sum(axis=1, keepdims=True)
    out = np.zeros((T, E))
    for t in np.nonzero(live)[0]:
        for j in range(k):
            if 0 <= idx[t, j] < E:
                out[t, idx[t, j]] += g[t, j]
    return out


def router_grad(ds, W, x, live, dx_in=None):
    """dW, db, dx of sum(ds * (x W^T + b)) over the live tokens."""
    ds = np.where(live[:, None], ds, 0.0)
    x = np.where(live[:, None], x, 0.0)
    dx = ds @ W
    return ds.T @ x, ds.sum(axis=0), dx if dx_in is None else dx + dx_in


def rms_norm(h, g, eps):
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * g


def rms_norm_grad(dx, h, rstd, g, live, dh_in=None):
    """dh, dg of sum(dx * rms_norm(h)), rstd = 1/sqrt(mean(h^2) + eps) given."""
    n = np.where(live[:, None], h * np.where(live, rstd, 0.0)[:, None], 0.0)
    v = np.where(live[:, None], dx, 0.0)
    u = v * g
    dh = np.where(live, rstd, 0.0)[:, None] * (u - n * (u * n).mean(axis=1, keepdims=True))
    return dh if dh_in is None else dh + dh_in, (v * n).sum(axis=0)


def e4m3_value(code):
    """Values of E4M3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F is NaN."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def checkpoint_rows(q, scales):
    """[T, d] values of an 8-bit checkpoint (E8M0 scale 2^(s - 127) per 32 elements)."""
    return e4m3_value(q) * np.exp2(scales.astype(np.float64) - 127.0).repeat(32, axis=1)
