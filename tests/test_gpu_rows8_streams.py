"""The operators on rows in 8 bits on streams that are not the current one, in graphs, and on memory of other devices."""
import pytest
import torch

from rows8_util import randn, routing

pytestmark = pytest.mark.gpu

BUSY = 20_000_000        # clock cycles a stream is kept busy: about 10 ms


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    ops.sync_status()
    return ops


class Step:
    """Inputs, and everything that the operators make of them, in the order of a training step."""

    def __init__(self, ops, seed, T=400, H=1024, I=320, N=200, E=6, K=2):
        self.ops, self.E = ops, E
        self.x, self.res, self.d = (randn(seed + i, T, H, dt="bf16").cuda() for i in range(3))
        self.w = (1 + 0.1 * randn(seed, H)).cuda()
        self.idx = routing(T, E, K, 0.1, seed).cuda()
        self.tw = torch.rand(T, K, generator=torch.Generator().manual_seed(seed)).cuda()
        self.r = ops.sort_tokens(self.idx, E)
        self.h = randn(seed + 4, self.r.rows, 2 * I, dt="bf16").cuda()
        self.da = randn(seed + 5, self.r.rows, I, dt="bf16").cuda()
        self.dy = randn(seed + 6, self.r.rows, N, dt="bf16").cuda()
        self.dz = randn(seed + 7, T, 64, dt="bf16").cuda()

    def run(self, stream=None):
        o, s = self.ops, {} if stream is None else {"stream": stream}
        n = o.rms_norm(self.x, self.w, self.res, quant="mx", **s)
        m = o.rms_norm(self.x, self.w, quant="f8", **s)
        f = o.swiglu(self.h, self.r, self.tw, quant=True, keep=True, **s)
        q = o.quantize8(self.x, **s)
        out = [*n, m.y, m.codes, m.sf, *f, *q, o.dequantize8(*q, self.x.shape[1], **s)]
        out += o.rms_norm_backward(self.d, n.h, self.w, n.rstd, self.d, **s)
        out += o.swiglu_backward(self.da, f.kept, f.kept_sf, self.r, self.tw, **s)
        H = self.x.shape[1]
        out += [o.weight_grad(self.dy, n.codes, n.sf, H, self.r, True, **s),               # gathered, many tiles
                o.weight_grad(self.dz, n.codes, n.sf, H, dtype=torch.float32, **s),        # few tiles, in parts or not
                o.weight_grad(self.h[:, 1:101], f.codes, f.sf, self.da.shape[1], self.r, **s)]   # rows on no boundary
        return out


def same(a, b):
    return len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


def scribble(tensors):
    """Takes and overwrites memory of these sizes on the current stream, and waits for it."""
    kept = [torch.full((t.numel() * t.element_size(),), 255, dtype=torch.uint8, device="cuda") for t in tensors for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    return kept


def test_a_busy_stream_keeps_what_its_calls_made(ops):
    step = Step(ops, 1)
    want = step.run()
    for as_number in (False, True):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        got = step.run(s.cuda_stream if as_number else s)
        kept = scribble(want)
        s.synchronize()
        assert same(got, want) and all((k == 255).all() for k in kept)


def test_two_streams_at_once(ops):
    steps = [Step(ops, 11), Step(ops, 22)]
    want = [s.run() for s in steps]
    for _ in range(5):
        streams = [torch.cuda.Stream() for _ in steps]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                torch.cuda._sleep(BUSY // 10)
        got = [step.run(s) for step, s in zip(steps, streams)]
        for s in streams:
            s.synchronize()
        assert all(same(g, w) for g, w in zip(got, want))
    assert ops.sync_status() == (0, 0)


def test_the_stream_of_a_context(ops):
    step = Step(ops, 3)
    want = step.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
        got = step.run()
    s.synchronize()
    assert same(got, want)


def test_captured_and_replayed_with_new_inputs(ops):
    """Two graphs of the same calls, replayed in turn and after eager calls; new inputs, and a new routing, reach them."""
    steps = [Step(ops, 5), Step(ops, 6)]
    other = [Step(ops, 7), Step(ops, 8)]
    want = [s.run() for s in steps]
    graphs = []
    for s in steps:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s.run()
        graphs.append((g, out))
    for _ in range(2):
        for (g, out), w in zip(graphs, want):
            for t in out:
                t.view(torch.uint8).fill_(77)
            g.replay()
            torch.cuda.synchronize()
            assert same(out, w)
    for (g, out), s, o in zip(graphs, steps, other):
        new = o.run()
        for name in ("x", "res", "d", "w", "tw", "dz"):
            getattr(s, name).copy_(getattr(o, name))
        s.r._buf.copy_(o.r._buf)
        for name in ("h", "da", "dy"):
            getattr(s, name).copy_(getattr(o, name))
        g.replay()
        torch.cuda.synchronize()
        assert same(out, new)
    assert ops.sync_status() == (0, 0)


def test_host_memory_is_refused(ops):
    from moe_expert_forward_gb300 import MMError
    step = Step(ops, 9, T=40)
    n = ops.rms_norm(step.x, step.w, quant="mx")
    f = ops.swiglu(step.h, step.r, step.tw, keep=True)
    r = ops.Routing(40, 2, 6, 16, step.r.rows, "cpu", 0)
    for call in (lambda: ops.quantize8(step.x.cpu()), lambda: ops.dequantize8(n.codes.cpu(), n.sf, 1024),
                 lambda: ops.dequantize8(n.codes, n.sf.cpu(), 1024), lambda: ops.rms_norm(step.x, step.w.cpu()),
                 lambda: ops.rms_norm(step.x, step.w, step.res.cpu()), lambda: ops.swiglu(step.h.cpu()),
                 lambda: ops.rms_norm_backward(step.d, n.h, step.w, n.rstd.cpu()),
                 lambda: ops.swiglu(step.h, r, step.tw), lambda: ops.swiglu(step.h, step.r, step.tw.cpu()),
                 lambda: ops.swiglu_backward(step.da, f.kept.cpu(), f.kept_sf), lambda: ops.weight_grad(step.dy, n.codes, n.sf, 1024, r, True),
                 lambda: ops.weight_grad(step.dy.cpu(), n.codes, n.sf, 1024, step.r, True)):
        with pytest.raises(MMError):
            call()
    torch.cuda.synchronize()
