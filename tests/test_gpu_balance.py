"""Per-expert counts, balance and z loss and their gradient (redmoe_balance_*) against the
definition in 64 bits.

Tolerances: counts and rows are exact. A probability is a few units off (the exponent
v - max rounded: |v - max| units, at most 20 for logits of two standard deviations; ex2 and one
reciprocal; a sum of at most 32 values of a lane and 5 shuffles): under 64 U; its mean adds the rows of a warp,
16 warps and the blocks, each one U: T / 16 + 64 + 160 more. The gradient is one such row.
"""

import pytest
import torch

import sparse_moe_gemv_b200 as smg
from plain_ops import U, balance_backward, balance_forward, store_tol

pytestmark = pytest.mark.gpu


def make(T, E, k, dtype="f32", masked=0.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(77 + seed)
    logits = (2.0 * torch.randn(T, E, generator=g, device="cuda")).to(smg.TORCH_DTYPES[dtype])
    ids = logits.float().topk(k, dim=1).indices.to(torch.int32) if T else torch.empty(0, k, device="cuda", dtype=torch.int32)
    mask = None
    if masked:
        mask = (torch.rand(T, generator=g, device="cuda") >= masked).to(torch.uint8)
        pad = mask == 0
        logits[pad] = float("nan")
        ids[pad] = 5 % E
    return logits, ids, mask


def run(logits, ids, mask, grad=(0.5, 0.25), ws=None):
    T, E = logits.shape
    loss, prob = torch.full((2,), 9.0, device="cuda"), torch.full((E,), 9.0, device="cuda")
    counts, n = torch.full((E,), -7, device="cuda", dtype=torch.int32), torch.full((1,), -7, device="cuda", dtype=torch.int32)
    ws = smg.new_balance_workspace(T, E) if ws is None else ws
    smg.redmoe_balance_forward(logits, ids, loss, counts, prob, n, ws, mask=mask)
    dl = torch.full_like(logits, 9.0)
    smg.redmoe_balance_backward(logits, counts, n, torch.tensor(grad, device="cuda"), dl, ids.shape[1], mask=mask)
    torch.cuda.synchronize()
    assert int(ws[:256].count_nonzero()) == 0  # the control block is left zero
    return loss, counts, prob, n, dl


def check(logits, ids, mask, got, grad=(0.5, 0.25)):
    loss, counts, prob, n, dl = (v.cpu() for v in got)
    T, k = ids.shape
    rl, rc, rp, rn, mag = balance_forward(logits, ids, mask)
    assert int(n) == rn and torch.equal(counts, rc)
    deep = (64 + T / 16 + 224) * U
    assert bool(((prob.double() - rp).abs() <= store_tol(rp, deep * rp, torch.float32)).all())
    assert bool(((loss.double() - rl).abs() <= store_tol(rl, deep * mag, torch.float32)).all())
    rd, md = balance_backward(logits, counts, rn, k, grad, mask)
    bad = (dl.double() - rd).abs() - store_tol(rd, 128 * U * md, dl.dtype)
    assert not dl.isnan().any() and (bad.numel() == 0 or float(bad.max()) <= 0)


@pytest.mark.parametrize("T,E,k,dtype,masked", [
    (1, 1, 1, "f32", 0.0), (1, 512, 10, "f32", 0.0), (2, 2, 2, "bf16", 0.0), (33, 61, 4, "f32", 0.1),
    (33, 61, 4, "bf16", 0.3), (100, 128, 8, "f32", 0.5), (257, 129, 3, "bf16", 0.0), (64, 256, 8, "bf16", 0.2),
    (999, 512, 10, "f32", 0.2), (500, 512, 10, "bf16", 0.0), (300, 513, 32, "f32", 0.0), (70, 1000, 10, "bf16", 0.1),
    (41, 1023, 7, "bf16", 0.0), (130, 1024, 16, "f32", 0.2), (41, 1024, 16, "bf16", 0.0), (3001, 20, 2, "f32", 0.0),
    (40, 132, 6, "f32", 0.0), (40, 264, 6, "bf16", 0.0),
])
def test_forward_and_gradient(gpu_lib, T, E, k, dtype, masked):
    logits, ids, mask = make(T, E, k, dtype, masked)
    got = run(logits, ids, mask)
    check(logits, ids, mask, got)
    again = run(logits, ids, mask)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_no_rows_and_no_live_rows(gpu_lib):
    for T, mask in ((0, None), (5, torch.zeros(5, device="cuda", dtype=torch.uint8)),
                    (5, torch.zeros(5, device="cuda", dtype=torch.bool))):
        logits, ids, _ = make(T, 40, 3)
        loss, counts, prob, n, dl = run(logits, ids, mask)
        assert float(loss.abs().max()) == 0 and int(counts.abs().max()) == 0 and float(prob.abs().max()) == 0
        assert int(n) == 0 and (T == 0 or float(dl.abs().max()) == 0)


@pytest.mark.parametrize("dtype,E", [("f32", 64), ("bf16", 64), ("f32", 61), ("bf16", 61)])
def test_infinities_lowest_values_and_stray_ids(gpu_lib, dtype, E):
    """Experts switched off by -infinity, a row of the type's lowest value, a row that allows no
    expert, ids that name none, the same id twice."""
    logits, ids, _ = make(40, E, 4, dtype)
    logits[:, 3::5] = -float("inf")
    logits[7] = -float("inf")
    logits[9, :] = -200.0
    logits[9, 2] = torch.finfo(logits.dtype).min
    ids[11] = torch.tensor([-1, E, 2 ** 30, -2 ** 31], dtype=torch.int32)
    ids[12] = ids[12, 0]
    got = run(logits, ids, None)
    assert int(got[3]) == 39 and float(got[4][7].abs().max()) == 0
    check(logits, ids, None, got)
    # a whole row of the lowest value is an even row; its z loss overflows by definition
    logits[9] = torch.finfo(logits.dtype).min
    loss, _, prob, n, dl = run(logits, ids, None, grad=(0.5, 0.0))
    assert int(n) == 39 and bool(prob.isfinite().all()) and bool(dl.isfinite().all())
    assert float(loss[1]) == float("inf") and bool(loss[0].isfinite())


def test_nan_in_a_live_row_shows(gpu_lib):
    logits, ids, _ = make(20, 64, 4)
    logits[3, 5] = float("nan")
    loss, counts, prob, n, dl = run(logits, ids, None)
    assert bool(loss.isnan().all()) and bool(prob.isnan().all()) and int(n) == 20
    assert bool(dl[3].isnan().all()) and not bool(dl[:3].isnan().any()) and not bool(dl[4:].isnan().any())


def test_even_counts_leave_no_balance_gradient(gpu_lib):
    logits, _, _ = make(64, 16, 16)
    ids = torch.arange(16, device="cuda", dtype=torch.int32).repeat(64, 1)
    loss, counts, _, _, dl = run(logits, ids, None, grad=(1.0, 0.0))
    assert bool((counts == 64).all()) and float(dl.abs().max()) == 0.0
    assert abs(float(loss[0]) - 1.0) <= 300 * U


def test_gradient_in_place_streams_and_graph(gpu_lib):
    logits, ids, mask = make(700, 512, 10, masked=0.2)
    want = run(logits, ids, mask)
    E = 512
    ws = smg.new_balance_workspace(700, E)
    loss, prob = torch.empty(2, device="cuda"), torch.empty(E, device="cuda")
    counts, n = torch.empty(E, device="cuda", dtype=torch.int32), torch.empty(1, device="cuda", dtype=torch.int32)
    grad = torch.tensor([0.5, 0.25], device="cuda")
    buf = logits.clone()

    def both():
        smg.redmoe_balance_forward(buf, ids, loss, counts, prob, n, ws, mask=mask)
        smg.redmoe_balance_backward(buf, counts, n, grad, buf, 10, mask=mask)  # over the logits

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    for a, b in zip((loss, counts, prob, n, buf), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for scale in (1.0, 0.5):
        l2 = torch.where(mask.bool()[:, None], logits * scale, logits)
        buf.copy_(l2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((loss, counts, prob, n, buf), run(l2, ids, mask)):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits(gpu_lib):
    """More than 2^31 logits: only the last rows count, and they equal a small call's."""
    T, E, k = 2 ** 21 + 3, 1024, 2
    logits = torch.zeros(T, E, device="cuda", dtype=torch.bfloat16)
    small, ids_small, _ = make(3, E, k, "bf16")
    logits[-3:] = small
    ids = torch.zeros(T, k, device="cuda", dtype=torch.int32)
    ids[-3:] = ids_small
    mask = torch.zeros(T, device="cuda", dtype=torch.bool)
    mask[-3:] = True
    loss, counts, prob, n, dl = run(logits, ids, mask)
    check(small, ids_small, None, (loss, counts, prob, n, dl[-3:]))
    assert int(dl[:-3].count_nonzero()) == 0


def test_router_statistics_agree_with_the_layer(gpu_lib):
    """redmoe_router's logits and ids in, the counts of redmoe_route_build out."""
    import moe_inputs as mi
    shape = mi.LayerShape(H=256, E=48, k=4, I=128, Is=128, sigma=0.05)
    L = mi.make_layer(shape, 5, "cuda")
    x = mi.make_x(shape, 90, 5, "cuda")
    lay = smg.Layer.from_shape(L, shape)
    ids = torch.empty(90, 4, device="cuda", dtype=torch.int32)
    w, sg, lg = torch.empty(90, 4, device="cuda"), torch.empty(90, device="cuda"), torch.empty(90, 48, device="cuda")
    smg.redmoe_router(lay, x, ids, w, sg, smg.new_workspace(lay, 90), logits=lg)
    got = run(lg, ids, None)
    check(lg, ids, None, got)
    counts, off = torch.empty(48, device="cuda", dtype=torch.int32), torch.empty(49, device="cuda", dtype=torch.int32)
    smg.redmoe_route_build(ids, 48, counts, off, torch.empty(360, device="cuda", dtype=torch.int32))
    assert torch.equal(counts, got[1])


def test_binding_refusals_on_the_device(gpu_lib):
    logits, ids, _ = make(8, 16, 2)
    good = dict(logits=logits, topk_ids=ids, loss=torch.empty(2, device="cuda"),
                counts=torch.empty(16, device="cuda", dtype=torch.int32), prob=torch.empty(16, device="cuda"),
                n_rows=torch.empty(1, device="cuda", dtype=torch.int32), workspace=smg.new_balance_workspace(8, 16))
    for bad in (dict(logits=logits.half()), dict(logits=logits[:, :8]), dict(topk_ids=ids.long()), dict(topk_ids=ids[:4]),
                dict(loss=torch.empty(1, device="cuda")), dict(mask=torch.ones(7, device="cuda", dtype=torch.uint8)),
                dict(mask=torch.ones(8, device="cuda")), dict(prob=torch.empty(16))):
        with pytest.raises(ValueError):
            smg.redmoe_balance_forward(**{**good, **bad})
    with pytest.raises(smg.RedmoeError, match="WORKSPACE"):
        smg.redmoe_balance_forward(**{**good, "workspace": good["workspace"][:256]})
