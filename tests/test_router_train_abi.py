"""The router-training entry points refuse bad arguments before any launch, and
need no GPU to do so (the addresses here are never dereferenced)."""
import ctypes

import pytest

from sparse_moe_layer_05_b200 import binding as B
from sparse_moe_layer_05_b200 import build as BUILD

G = 0x10000      # a 16-byte aligned address
BIG = 1 << 40    # a workspace that is large enough
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.load()


def f(x):
    return ctypes.c_float(x)


CALLS = {
    "moe_balance_loss": dict(logits=G, idx=G, mask=None, E=8, k=2, T=4, a=f(1), b=f(1), stats=G, counts=G,
                             mean=G, lse=G, ws=G, bytes=BIG, stream=None),
    "moe_balance_loss_backward": dict(logits=G, lse=G, counts=G, stats=G, mask=None, E=8, k=2, T=4, a=f(1),
                                      b=f(1), dloss=None, accumulate=0, dlogits=G, stream=None),
    "moe_gate_backward": dict(dout=G, yw=G, idx=G, w=G, mask=None, E=8, k=2, T=4, d=64, accumulate=0,
                              dlogits=G, stream=None),
    "moe_router_backward": dict(dlogits=G, W=G, x=G, q=None, scales=None, rstd=None, g=None, mask=None, E=8,
                                T=4, d=64, dx_in=None, accumulate=0, dW=G, db=G, dx=G, ws=G, bytes=BIG,
                                stream=None),
    "moe_rms_norm_checkpoint": dict(h=G, g=G, eps=f(1e-5), T=4, d=64, x=G, q=G, scales=G, rstd=G, stream=None),
    "moe_rms_norm_backward": dict(dx=G, h=G, q=None, scales=None, rstd=G, g=G, mask=None, T=4, d=64,
                                  dh_in=None, accumulate=0, dh=G, dg=G, ws=G, bytes=BIG, stream=None),
}
POINTERS = {name: [a for a, v in args.items() if v == G] for name, args in CALLS.items()}


def call(lib, name, **changes):
    assert set(changes) <= set(CALLS[name])
    return getattr(lib, name)(*{**CALLS[name], **changes}.values())


@pytest.mark.parametrize("name", list(CALLS))
def test_null_and_misaligned_pointers(lib, name):
    for a in POINTERS[name]:
        assert call(lib, name, **{a: G + 4}) == INVALID, a
        optional = {"moe_router_backward": ("dW", "db", "dx"), "moe_rms_norm_checkpoint": ("x",)}.get(name, ())
        if a not in optional:
            assert call(lib, name, **{a: None}) == INVALID, a


@pytest.mark.parametrize("name", list(CALLS))
def test_shapes(lib, name):
    for a, bad, code in [("E", 0, INVALID), ("E", 257, UNSUPPORTED), ("k", 0, INVALID), ("k", 9, UNSUPPORTED),
                         ("T", -1, INVALID), ("d", 0, INVALID), ("d", 48, UNSUPPORTED), ("d", 16416, UNSUPPORTED),
                         ("accumulate", 2, INVALID)]:
        if a in CALLS[name]:
            assert call(lib, name, **{a: bad}) == code, (a, bad)
    if "k" in CALLS[name]:
        assert call(lib, name, E=64, k=33) == UNSUPPORTED
        assert call(lib, name, E=64, k=32, T=1 << 26) == UNSUPPORTED      # T k = 2^31
    if "bytes" in CALLS[name]:
        assert call(lib, name, bytes=15) == WORKSPACE


def test_rows_come_as_one_of_two_forms(lib):
    r = "moe_router_backward"
    q = dict(q=G, scales=G, rstd=G, g=G)
    assert call(lib, r, **q) == INVALID                                    # x and a checkpoint
    for missing in q:
        assert call(lib, r, x=None, **{**q, missing: None}) == INVALID
    assert call(lib, r, x=None) == INVALID                                 # no rows for dW
    assert call(lib, r, W=None, dW=None, db=None) == INVALID               # dx needs W
    assert call(lib, r, dW=None, db=None, dx=None) == INVALID              # nothing to compute
    assert call(lib, r, dx=None, dx_in=G) == INVALID
    n = "moe_rms_norm_backward"
    assert call(lib, n, q=G, scales=G) == INVALID
    assert call(lib, n, h=None, q=G) == INVALID
    assert call(lib, n, h=None, scales=G) == INVALID
    assert call(lib, "moe_rms_norm_checkpoint", eps=f(-1)) == INVALID
    assert call(lib, "moe_rms_norm_checkpoint", eps=f(float("nan"))) == INVALID
    assert call(lib, "moe_rms_norm_checkpoint", g=None) == INVALID         # x needs the gain


def test_calls_on_no_tokens_launch_nothing(lib):
    """Those whose outputs are all per token; sums over tokens are written as zero."""
    assert call(lib, "moe_balance_loss_backward", T=0) == OK
    assert call(lib, "moe_gate_backward", T=0, dout=None, yw=None, idx=None, w=None, dlogits=None) == OK
    assert call(lib, "moe_rms_norm_checkpoint", T=0, h=None, x=None, q=None, scales=None, rstd=None) == OK


def test_block_checkpoint_arguments(lib):
    b = [G, G, f(1e-5)] + [G] * 8 + [4, 2, 8, 64, 128, G, G, G, G, G, 1 << 30, None]
    fn = lib.moe_forward_block_checkpoint
    for i in (17, 18, 19):
        for bad in (None, G + 8):
            a = list(b)
            a[i] = bad
            assert fn(*a) == INVALID
    a = list(b)
    a[21] = 16
    assert fn(*a) == WORKSPACE
    a = list(b)
    a[13] = 0
    assert fn(*a) == OK


def test_workspace_sizes():
    for T in (0, 1, 61, 4096, 16384):
        for E, d in ((1, 32), (64, 2880), (256, 16384)):
            assert B.moe_balance_loss_workspace_size(E, 1, T) > 0
            assert B.moe_router_backward_workspace_size(E, T, d) > 0
            assert B.moe_rms_norm_backward_workspace_size(T, d) > 0
    assert B.moe_balance_loss_workspace_size(4, 5, 8) == 0
    assert B.moe_router_backward_workspace_size(257, 8, 64) == 0
    assert B.moe_router_backward_workspace_size(4, 8, 40) == 0
    assert B.moe_rms_norm_backward_workspace_size(8, 16416) == 0
    assert B.moe_rms_norm_backward_workspace_size(-1, 64) == 0


def test_a_workspace_for_more_tokens_serves_fewer(lib):
    """Sizes never fall as T grows: a caller sizes a workspace for its largest batch."""
    Ts = [*range(0, 700), *range(700, 40000, 131)]
    sizes = {f"balance {E}": [lib.moe_balance_loss_workspace_size(E, 1, T) for T in Ts] for E in (1, 32, 256)}
    sizes |= {f"router {E} {d}": [lib.moe_router_backward_workspace_size(E, T, d) for T in Ts]
              for E, d in ((4, 512), (32, 2880), (161, 64), (248, 2880))}
    sizes |= {f"norm {d}": [lib.moe_rms_norm_backward_workspace_size(T, d) for T in Ts] for d in (32, 2880, 16384)}
    for name, s in sizes.items():
        falls = [Ts[i] for i in range(1, len(s)) if s[i] < s[i - 1]]
        assert not falls, (name, falls[:3])
