"""MoELayer's methods on another stream than the current one: a result that they
allocate belongs to the stream whose kernels write it, so its memory is not handed
out again while they run. On the CPU with the launches replaced; on the GPU by where
the allocator puts the next tensor."""
import contextlib
import types

import numpy as np
import pytest

from sparse_moe_layer_05_b200 import binding as B
from sparse_moe_layer_05_b200 import workloads as W

torch = pytest.importorskip("torch")

T, D = 5, 32


class Stream:
    """As far as the binding looks at one."""

    def __init__(self, number):
        self.cuda_stream = number


class Allocated:
    def __init__(self, stream, shape):
        self.stream, self.shape, self.recorded = stream, shape, []

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def streams(monkeypatch):
    main, side = Stream(1), Stream(2)
    now = [main]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[-1])
    monkeypatch.setattr(torch, "empty", lambda shape, **kw: Allocated(now[-1], shape))
    for name in ("moe_forward", "moe_forward_block", "moe_forward_block_checkpoint", "moe_gate_backward",
                 "moe_balance_loss", "moe_balance_loss_backward", "moe_router_backward", "moe_rms_norm_backward"):
        monkeypatch.setattr(B, name, lambda *a, **kw: None)
    return main, side


def calls():
    layer = B.MoELayer.__new__(B.MoELayer)
    layer.d, layer.I, layer.E, layer.k, layer.T_max = D, 64, 4, 2, T
    for n in ("W_r", "b_r", "Wgu_codes", "Wgu_scales", "Wd_codes", "Wd_scales", "workspace"):
        setattr(layer, n, None)
    layer.intermediate = lambda name, n: None
    rows = torch.zeros((T, D))
    ck = types.SimpleNamespace(rows=lambda n: (None, None, None))
    gr = types.SimpleNamespace(T=T, dlogits=rows, dx=rows, lse=rows, workspace=None, dW_r=None, db_r=None, dg=None,
                               stats=None, counts=None, mean_probs=None)
    return {"forward": lambda **kw: layer.forward(rows, **kw),
            "forward_block": lambda **kw: layer.forward_block(rows, None, 1e-5, **kw),
            "training form": lambda **kw: layer.forward_block(rows, None, 1e-5, checkpoint=ck, **kw),
            "backward_block": lambda **kw: layer.backward_block(rows, None, ck, gr, 0.1, 0.1, **kw)}


@pytest.mark.parametrize("name", ["forward", "forward_block", "training form", "backward_block"])
def test_a_result_is_allocated_on_the_stream_that_writes_it(streams, name):
    main, side = streams
    call = calls()[name]
    out = call(stream=side)
    assert out.stream is side and out.recorded == [main] and out.shape == (T, D)
    for kw in ({}, {"stream": main}):
        out = call(**kw)
        assert out.stream is main and out.recorded == []


@pytest.mark.gpu
def test_memory_of_a_dropped_result_stays_its_streams():
    """A result of 2.2 MB dropped while its stream may still write it: the current
    stream's next tensors of that size lie elsewhere."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_moe_layer_05_b200 import build
    build.build()
    n, d = 1100, 1024
    inp = W.make_custom(d, 256, 4, 2, n, seed=5)
    layer, ck, gr = B.MoELayer(inp, block=True), B.NormCheckpoint(n, d), B.RouterGrads(4, 2, n, d)
    x = torch.from_numpy(inp.x).cuda()
    g = torch.from_numpy(np.ones(d, np.float32)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in (lambda: layer.forward(x, stream=side),
                 lambda: layer.forward_block(x, g, 1e-5, checkpoint=ck, stream=side),
                 lambda: layer.backward_block(x, g, ck, gr, 0.1, 0.1, stream=side)):
        out = call()
        at = out.data_ptr()
        del out
        kept = [torch.empty((n, d), dtype=torch.uint16, device="cuda") for _ in range(4)]
        assert at not in [t.data_ptr() for t in kept]
        torch.cuda.synchronize()
