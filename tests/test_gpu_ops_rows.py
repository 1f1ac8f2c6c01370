"""Tokens sorted by expert and back, with their gradients, against a plain
implementation in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # significands of 24, 8 and 11 bits


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def routing(T, E, K, masked, seed):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.choice(E, K, replace=False) for _ in range(T)]) if T else np.zeros((0, K))
    idx = idx.astype(np.int32)
    idx[rng.random(idx.shape) < masked] = -1
    return idx


def check(ops, T, H, E, K, block=16, dt="f32", masked=0.0, seed=0, idx=None):
    idx = routing(T, E, K, masked, seed) if idx is None else idx
    r = ops.sort_tokens(torch.from_numpy(idx).cuda(), E, block)
    ref = O.route(idx, E, block)
    slot = ref["slot"]
    assert np.array_equal(r.cnt.cpu().numpy(), ref["cnt"]) and np.array_equal(r.slot.cpu().numpy(), slot)
    assert np.array_equal(r.blk_off.cpu().numpy(), ref["blk_off"]) and int(r.status[0]) == 0
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(DT[dt])
    rows = torch.randn(r.rows, H, generator=g).to(DT[dt])
    w = torch.randn(T, K, generator=g)
    x64, rows64, w64 = x.double().numpy(), rows.double().numpy(), w.double().numpy()
    ulp = HALF_ULP[dt]

    got = ops.permute(x.cuda(), r).double().cpu().numpy()
    want = np.zeros((r.rows, H))
    for t, k in zip(*np.nonzero(slot >= 0)):
        want[slot[t, k]] = x64[t]
    assert np.array_equal(got, want)                      # copies, and zeros everywhere else

    live = (slot >= 0)[:, :, None]
    at = np.where(slot >= 0, slot, 0)
    picked = np.where(live, rows64[at] if r.rows else np.zeros((T, K, H)), 0.0)
    # K fp32 roundings of a sum, one of the product, one to the type
    for weights, wd in ((w64, w.cuda()), (None, None)):
        terms = picked * (1.0 if weights is None else weights[:, :, None])
        y = (ops.unpermute(rows.cuda(), r, wd) if weights is not None else
             ops.permute_backward(rows.cuda(), r)).double().cpu().numpy()
        want = terms.sum(1)
        tol = (K + 1) * 2.0 ** -24 * np.abs(terms).sum(1) + ulp * np.abs(want) * 1.01 + 1e-30
        if dt == "f16":
            tol = tol + 2.0 ** -25                        # results below the type's normal range
        assert (np.abs(y - want) <= tol).all(), np.abs(y - want).max()

    d_rows, d_w = ops.unpermute_backward(x.cuda(), rows.cuda(), r, w.cuda())
    want = np.zeros((r.rows, H))
    for t, k in zip(*np.nonzero(slot >= 0)):
        want[slot[t, k]] = w64[t, k] * x64[t]
    got = d_rows.double().cpu().numpy()
    assert (np.abs(got - want) <= (2.0 ** -24 + ulp) * 1.01 * np.abs(want) + (2.0 ** -25 if dt == "f16" else 1e-30)).all()
    prod = picked * x64[:, None, :]
    err = np.abs(d_w.double().cpu().numpy() - prod.sum(2))
    assert (err <= H * 2.0 ** -24 * np.abs(prod).sum(2) + 1e-30).all()
    assert (d_w.cpu().numpy()[slot < 0] == 0).all()
    plain_rows, none = ops.unpermute_backward(x.cuda(), None, r)
    assert none is None and torch.equal(plain_rows, ops.permute(x.cuda(), r))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H", [1, 2, 3, 5, 8, 12, 31, 64, 100, 257, 1000, 1001, 2048, 5000])
def test_widths(ops, H, dt):
    check(ops, 23, H, 9, 3, dt=dt, masked=0.1, seed=H)


@pytest.mark.parametrize("T", [0, 1, 2, 7, 128, 300])
@pytest.mark.parametrize("K,E", [(1, 1), (2, 5), (8, 64), (16, 40), (5, 1024)])
def test_tokens_and_experts(ops, T, K, E):
    check(ops, T, 72, E, K, block=32, dt="bf16", seed=T + K)


@pytest.mark.parametrize("block", [16, 48, 128, 256])
def test_blocks(ops, block):
    check(ops, 200, 40, 7, 2, block=block, seed=block)


@pytest.mark.parametrize("T,K,E,block", [(512, 4, 9, 16), (513, 4, 300, 32), (3000, 3, 384, 16), (8192, 6, 384, 16),
                                         (12288, 16, 1024, 64), (12289, 16, 1024, 64), (50000, 8, 256, 128)])
def test_sorts_of_every_size(ops, T, K, E, block):
    """Clusters of 4 to 16 CTAs, and (past 196608 pairs) the two launches."""
    rng = np.random.default_rng(T)
    idx = rng.integers(0, E, (T, K)).astype(np.int32)
    idx[rng.random(idx.shape) < 0.05] = -1
    r = ops.sort_tokens(torch.from_numpy(idx).cuda(), E, block)
    ref = O.route(idx, E, block)
    assert int(r.status[0]) == 0
    assert np.array_equal(r.cnt.cpu().numpy(), ref["cnt"]) and np.array_equal(r.blk_off.cpu().numpy(), ref["blk_off"])
    assert np.array_equal(r.slot.cpu().numpy(), ref["slot"])
    assert np.array_equal(r.src.cpu().numpy()[:len(ref["src"])], ref["src"])
    bad = idx.copy()
    bad[T // 2, 0] = E
    assert int(ops.sort_tokens(torch.from_numpy(bad).cuda(), E, block).status[0]) == 5


def test_every_slot_masked(ops):
    check(ops, 33, 64, 4, 2, idx=np.full((33, 2), -1, np.int32))


def test_one_expert_takes_everything(ops):
    idx = np.full((130, 1), 3, np.int32)
    check(ops, 130, 48, 6, 1, block=128, idx=idx)


def test_ids_out_of_range_are_masked_and_flagged(ops):
    from moe_expert_forward_gb300 import MM_MOE_ERR_BAD_ROUTING
    idx = torch.tensor([[0, 9], [1, -3]], dtype=torch.int32, device="cuda")
    r = ops.sort_tokens(idx, 4)
    assert int(r.status[0]) == MM_MOE_ERR_BAD_ROUTING
    y = ops.unpermute(torch.ones(r.rows, 8, device="cuda"), r)
    assert (y == 1).all()


def test_masked_rows_are_not_read(ops):
    """NaN in rows that no slot names, and weights of masked slots, reach nothing."""
    idx = np.array([[0, -1], [-1, -1], [1, 0]], np.int32)
    r = ops.sort_tokens(torch.from_numpy(idx).cuda(), 2)
    rows = torch.full((r.rows, 24), float("nan"), device="cuda")
    slot = r.slot.cpu().numpy()
    for s in slot[slot >= 0]:
        rows[int(s)] = 1.0
    w = torch.where(r.slot < 0, float("nan"), 0.5)
    y = ops.unpermute(rows, r, w)
    assert y[:, 0].cpu().tolist() == [0.5, 0.0, 1.0]
    d_rows, d_w = ops.unpermute_backward(torch.ones(3, 24, device="cuda"), rows, r, w)
    assert torch.isfinite(d_rows).all() and torch.isfinite(d_w).all()


def test_strided_and_unaligned_inputs(ops):
    idx = torch.from_numpy(routing(40, 6, 2, 0.0, 4)).cuda()
    r = ops.sort_tokens(idx, 6)
    wide = torch.randn(40, 200, device="cuda", dtype=torch.bfloat16)
    for lo, hi in ((0, 64), (1, 65), (4, 68), (8, 200)):
        x = wide[:, lo:hi]
        assert torch.equal(ops.permute(x, r), ops.permute(x.contiguous(), r))
        rows = torch.randn(r.rows, hi - lo, device="cuda").to(torch.bfloat16)
        w = torch.rand(40, 2, device="cuda")
        a, b = ops.unpermute_backward(x, rows, r, w), ops.unpermute_backward(x.contiguous(), rows, r, w)
        assert torch.equal(a[0], b[0])
        assert torch.allclose(a[1], b[1], rtol=1e-4, atol=1e-4)   # another access width adds in another order


def test_gradients_against_differences(ops):
    """<d_rows, v> + <d_w, u> against the change of <dy, unpermute> along (v, u), in 64 bits:
    unpermute is bilinear, so the central difference is exact but for rounding."""
    idx = routing(12, 5, 3, 0.2, 8)
    r = ops.sort_tokens(torch.from_numpy(idx).cuda(), 5)
    g = torch.Generator().manual_seed(1)
    rows, v = torch.randn(r.rows, 20, generator=g), torch.randn(r.rows, 20, generator=g)
    w, u, dy = torch.randn(12, 3, generator=g), torch.randn(12, 3, generator=g), torch.randn(12, 20, generator=g)
    slot = r.slot.cpu()

    def forward(a, b):
        got = a[slot.clamp_min(0).long()] * (slot >= 0)[:, :, None]
        return float(((got * b[:, :, None]).sum(1) * dy.double()).sum())

    h = 0.5
    step = (forward(rows.double() + h * v, w.double() + h * u) - forward(rows.double() - h * v, w.double() - h * u)) / (2 * h)
    d_rows, d_w = ops.unpermute_backward(dy.cuda(), rows.cuda(), r, w.cuda())
    used = (slot >= 0).double()
    along = float((d_rows.double().cpu() * v.double()).sum() + (d_w.double().cpu() * u.double() * used).sum())
    assert abs(along - step) <= 1e-4 * max(1.0, abs(step))


def test_refusals(ops):
    from moe_expert_forward_gb300 import MMError
    idx = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    r = ops.sort_tokens(idx, 2)
    x = torch.zeros(4, 8, device="cuda")
    rows = torch.zeros(r.rows, 8, device="cuda")
    w = torch.zeros(4, 1, device="cuda")
    for call in (lambda: ops.sort_tokens(idx.long(), 2), lambda: ops.sort_tokens(idx, 2, 8),
                 lambda: ops.sort_tokens(idx, 2, 24), lambda: ops.sort_tokens(idx[:, 0], 2),
                 lambda: ops.sort_tokens(torch.zeros(4, 3, dtype=torch.int32, device="cuda"), 2),
                 lambda: ops.permute(x[:3], r), lambda: ops.permute(x.cpu(), r), lambda: ops.permute(x.int(), r),
                 lambda: ops.permute(torch.zeros(4, 0, device="cuda"), r),
                 lambda: ops.unpermute(rows[:-1], r), lambda: ops.unpermute(rows, r, w[:, 0]),
                 lambda: ops.unpermute(rows, r, w.double()),
                 lambda: ops.unpermute_backward(x, rows.bfloat16(), r, w),
                 lambda: ops.unpermute_backward(x[:2], rows, r, w)):
        with pytest.raises(MMError):
            call()
