"""What the tensor forms hand to the library: memory of which stream, of which device.  A stand-in takes the place of
the library and of the device, so these run without a GPU."""
import contextlib

import pytest
import torch

import moe_expert_forward_gb300 as M
from moe_expert_forward_gb300 import ops

CURRENT, SIDE = 0, 7


class Stand:
    """Streams are numbers, the CPU is the current device; every tensor made is noted with the stream current then."""

    def __init__(self):
        self.current, self.made, self.shared, self.calls = CURRENT, [], [], []

    @contextlib.contextmanager
    def on(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before

    def maker(self, make):
        def made(*args, **kw):
            t = make(*args, **kw)
            self.made.append((t.data_ptr(), self.current))
            return t
        return made

    def __getattr__(self, name):           # the library: every entry point notes its arguments
        def call(*args):
            self.calls.append((name, args))
            return M.MM_MOE_OK
        return call

    def args(self, name):
        return [a for n, a in self.calls if n == name][-1]

    def stream_of(self, address):
        return [s for p, s in self.made if p == address][-1]


@pytest.fixture
def stand(monkeypatch):
    s = Stand()
    monkeypatch.setattr(ops, "lib", lambda: s)
    monkeypatch.setattr(ops, "_device", lambda: -1)               # what a CPU tensor says of its device
    monkeypatch.setattr(ops, "_raw_stream", lambda device: s.current)
    monkeypatch.setattr(torch.cuda, "stream", s.on)
    monkeypatch.setattr(torch.cuda, "set_stream", lambda stream: setattr(s, "current", stream))
    monkeypatch.setattr(ops, "_streams", {})
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: s.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: p)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, on: s.shared.append((t.data_ptr(), on)))
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, s.maker(getattr(torch, name)))
    return s


def weights(E, N, C):
    return ops.MxWeights(torch.ones(E, N, C // 2, dtype=torch.uint8),
                         torch.ones(E * ops._scale_bytes(N, C), dtype=torch.uint8), E, N, C)


def test_the_workspace_of_a_linear_is_the_launch_streams(stand):
    """The caller never sees it: on the current stream's pool it would be handed out again while `stream` runs."""
    x, w = torch.ones(64, 64), weights(1, 32, 64)
    for stream, owner in ((None, CURRENT), (SIDE, SIDE), (CURRENT, CURRENT)):
        ops.mx_linear(x, w, stream=stream)
        a = stand.args("mm_moe_mx_linear")
        assert a[17] > 0 and stand.stream_of(a[16]) == owner and a[19] == owner
    with stand.on(SIDE):                       # and the default stream's, where another is current
        ops.mx_linear(x, w, stream=0)
        assert stand.stream_of(stand.args("mm_moe_mx_linear")[16]) == 0
    assert stand.current == CURRENT


def test_the_status_word_of_a_product_is_the_launch_streams(stand):
    """Its zeroing too: queued on another stream it would be in no order with the kernel."""
    w = weights(1, 32, 64)
    codes, sf = torch.ones(8, 32, dtype=torch.uint8), torch.ones(ops._scale_bytes(8, 64), dtype=torch.uint8)
    for stream, owner in ((None, CURRENT), (SIDE, SIDE)):
        ops.mx_product(codes, sf, w, stream=stream)
        assert stand.stream_of(stand.args("mm_moe_mx_product")[13]) == owner


def results(stream):
    """One call of every form that allocates a result, and what it returned."""
    x, idx, w = torch.ones(6, 64), torch.ones(6, 2, dtype=torch.int32), weights(1, 32, 64)
    routing = ops.sort_tokens(idx, 4, 128, stream=stream)
    rows = ops.permute(x, routing, stream=stream)
    topk_w = torch.ones(6, 2)
    codes, sf = ops.mx_quantize(x, stream=stream)
    chunked = ops.mx_quantize(x, chunks=True, stream=stream)
    made = [routing._buf, rows, codes, sf, *chunked, ops.unpermute(rows, routing, topk_w, stream=stream),
            ops.permute_backward(rows, routing, stream=stream),
            *ops.unpermute_backward(x, rows, routing, topk_w, stream=stream), *ops.route(x, 2, stream=stream),
            ops.route_backward(x, idx, topk_w, stream=stream), ops.mx_dequantize(codes, sf, 64, stream=stream),
            ops.mx_weights(codes, sf, stream=stream).sfp, ops.mx_product(*chunked, w, stream=stream),
            ops.mx_linear(x, w, stream=stream)]
    return [t.data_ptr() for t in made], made        # made: kept, so that no address is used twice


def test_results_are_the_launch_streams_and_marked_for_the_current_one(stand):
    """The current stream's free memory may still be written by work queued there, which `stream` does not wait for."""
    for stream, owner in ((None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE)):
        stand.shared.clear()
        pointers, kept = results(stream)
        assert len(pointers) == 17 and [stand.stream_of(p) for p in pointers] == [owner] * 17
        marked = [p for p, on in stand.shared if on == CURRENT]
        assert set(pointers) <= set(marked) if owner == SIDE else not marked


class Elsewhere(torch.Tensor):
    """A tensor of another device than the current one."""

    def get_device(self):
        return 1


def test_routings_and_weights_of_another_device_are_refused(stand):
    """Their addresses go to the library as they are: another device's would be read, or fault, there."""
    x, idx, topk_w = torch.ones(6, 64), torch.ones(6, 2, dtype=torch.int32), torch.ones(6, 2)
    here, there = ops.sort_tokens(idx, 4, 128), ops.sort_tokens(idx, 4, 128)
    there._buf = there._buf.as_subclass(Elsewhere)
    w, rows = weights(4, 32, 64), ops.permute(x, here)
    codes, sf = ops.mx_quantize(x, routing=here, chunks=True)
    one = weights(1, 32, 64)
    dense = ops.mx_quantize(x, chunks=True)
    before = len(stand.calls)
    for call in (lambda r: ops.permute(x, r), lambda r: ops.unpermute(rows, r, topk_w),
                 lambda r: ops.permute_backward(rows, r), lambda r: ops.unpermute_backward(x, rows, r, topk_w),
                 lambda r: ops.mx_quantize(x, routing=r), lambda r: ops.mx_product(codes, sf, w, routing=r),
                 lambda r: ops.mx_linear(x, w, routing=r)):
        with pytest.raises(M.MMError):
            call(there)
        assert len(stand.calls) == before
        call(here)
        before = len(stand.calls)
    for field in ("codes", "sfp"):
        far = one._replace(**{field: getattr(one, field).as_subclass(Elsewhere)})
        for call in (lambda: ops.mx_linear(x, far), lambda: ops.mx_product(*dense, far)):
            with pytest.raises(M.MMError):
                call()
    assert len(stand.calls) == before


def test_sync_status_asks_the_library(monkeypatch):
    monkeypatch.setattr(ops, "mm_moe_ops_status", lambda stream: (M.MM_MOE_ERR_TIMEOUT, stream))
    assert ops.sync_status(SIDE) == (M.MM_MOE_ERR_TIMEOUT, SIDE)
    if not torch.cuda.is_available():
        from moe_expert_forward_gb300 import build
        build.build()
        assert M.mm_moe_ops_status(None) == (M.MM_MOE_ERR_CUDA, 0)


def test_tensors_that_require_grad_are_refused_where_a_gradient_would_be_lost(stand):
    x, idx, topk_w = torch.ones(6, 64), torch.ones(6, 2, dtype=torch.int32), torch.ones(6, 2)
    r, w = ops.sort_tokens(idx, 4, 128), weights(1, 32, 64)
    rows = ops.permute(x, r)
    need = [t.clone().requires_grad_() for t in (x, rows, topk_w)]
    need_x, need_rows, need_w = need
    calls = [lambda: ops.route(need_x, 2), lambda: ops.route(x, 2, bias=need_x[0], score="sigmoid"),
             lambda: ops.permute(need_x, r), lambda: ops.unpermute(need_rows, r, topk_w),
             lambda: ops.unpermute(rows, r, need_w), lambda: ops.mx_linear(need_x, w)]
    for call in calls:
        before = len(stand.calls)
        with pytest.raises(M.MMError, match="requires grad"):
            call()
        assert len(stand.calls) == before
        with torch.no_grad():
            call()
        assert len(stand.calls) == before + 1
    for call in (lambda: ops.unpermute(rows, r, [1.0]), lambda: ops.route(x, 2, bias=[1.0], score="sigmoid")):
        with pytest.raises(M.MMError, match="must be a tensor"):
            call()
    # no gradient passes through these: rounding to 4 bits, and gradients themselves
    ops.mx_quantize(need_x)
    ops.route_backward(need_x, idx, topk_w)
    ops.unpermute_backward(x, need_rows, r, need_w)
    ops.permute_backward(need_rows, r)
