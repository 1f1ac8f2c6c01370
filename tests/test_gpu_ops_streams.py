"""Calls on a stream that is not the current one, while the current one takes and writes memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BUSY = 20_000_000        # clock cycles a stream is kept busy: about 10 ms


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


@pytest.fixture
def linear(ops):
    g = torch.Generator(device="cuda").manual_seed(1)
    w = ops.mx_weights(torch.randint(0, 256, (512, 512), generator=g, device="cuda", dtype=torch.uint8),
                       torch.randint(119, 123, (512, 32), generator=g, device="cuda", dtype=torch.uint8))
    xs = [torch.randn(300, 1024, generator=g, device="cuda") for _ in range(2)]
    return w, xs, [ops.mx_linear(x, w) for x in xs]


def side_streams(n):
    streams = [torch.cuda.Stream() for _ in range(n)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    return streams


def scribble(sizes, times=4):
    """Takes and overwrites blocks of these sizes on the current stream, and waits for it."""
    kept = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(times)]
    torch.cuda.current_stream().synchronize()
    return kept


def test_a_linear_on_a_busy_stream_keeps_its_workspace(ops, linear):
    w, xs, want = linear
    out = torch.empty(300, 512, device="cuda")
    for as_number in (False, True):
        s, = side_streams(1)
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        ops.mx_linear(xs[0], w, out=out, stream=s.cuda_stream if as_number else s)
        kept = scribble([ops._linear_bytes(300, 1024)])
        s.synchronize()
        assert torch.equal(out, want[0])
        assert all((k == 255).all() for k in kept)


def test_linears_on_two_streams_have_a_workspace_each(ops, linear):
    w, xs, want = linear
    for _ in range(10):
        streams = side_streams(2)
        outs = [torch.empty(300, 512, device="cuda") for _ in range(2)]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                torch.cuda._sleep(BUSY // 10)
        for s, x, o in zip(streams, xs, outs):
            ops.mx_linear(x, w, out=o, stream=s)
        for s in streams:
            s.synchronize()
        assert all(torch.equal(o, y) for o, y in zip(outs, want))


def test_a_product_on_a_busy_stream_keeps_its_status_word(ops, linear):
    w, xs, want = linear
    codes, sf = ops.mx_quantize(xs[0], chunks=True)
    out = torch.empty(300, 512, device="cuda")
    s, = side_streams(1)
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    ops.mx_product(codes, sf, w, out=out, dtype=torch.float32, stream=s)
    kept = scribble([16])
    s.synchronize()
    assert torch.equal(out, want[0]) and all((k == 255).all() for k in kept)


def test_results_on_an_idle_stream_are_not_what_the_current_one_still_writes(ops):
    """The current stream is busy with a queued write to a block that it has already freed on the host's side."""
    x = torch.randn(300, 1024, device="cuda")
    idx = torch.arange(300, device="cuda", dtype=torch.int32).remainder(4).view(300, 1).contiguous()
    r = ops.sort_tokens(idx, 4)
    rows = ops.permute(x, r)
    back = ops.unpermute(rows, r)
    s, = side_streams(1)
    torch.cuda.synchronize()
    for call, want in ((lambda: ops.permute(x, r, stream=s), rows), (lambda: ops.unpermute(rows, r, stream=s), back)):
        for _ in range(3):
            torch.cuda._sleep(BUSY)
            late = [torch.empty(want.numel() * 4, dtype=torch.uint8, device="cuda").fill_(255) for _ in range(4)]
            del late
            got = call()
            s.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_results_outlive_their_last_use_on_the_current_stream(ops):
    """Freed while the current stream still reads it, a result's memory does not go to the side stream's next call."""
    x, y = torch.ones(300, 1024, device="cuda"), torch.zeros(300, 1024, device="cuda")
    r = ops.sort_tokens(torch.zeros(300, 1, dtype=torch.int32, device="cuda"), 1)
    s, = side_streams(1)
    for _ in range(3):
        rows = ops.permute(x, r, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(BUSY)
        copy = rows.clone()
        del rows
        other = [ops.permute(y, r, stream=s) for _ in range(3)]
        torch.cuda.synchronize()
        assert (copy[r.slot[:, 0].long()] == 1).all() and not any(o.any() for o in other)
