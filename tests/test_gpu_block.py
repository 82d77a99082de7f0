"""The residual block around the layer, and the operators run together as a decoder step and a
router-training step would."""

import pytest
import torch

import moe_inputs as mi
import sparse_moe_gemv_b200 as smg
from parity import assert_layer_parity, tolerances
from plain_ops import NormCase, U, balance_backward, d, gemv_err, gemv_rows, store_tol

pytestmark = pytest.mark.gpu

QWEN = mi.LayerShape(H=2048, E=512, k=10, I=512, Is=512)
SMALL = mi.LayerShape(H=256, E=16, k=2, I=128, Is=128, sigma=0.05)
TINY = mi.WORKLOADS["tiny_f32"]["shape"]


def close(name, got, value, err):
    bad = (got.cpu().double() - value).abs() - store_tol(value, err, got.dtype)
    assert float(bad.max()) <= 0, f"{name}: {float(bad.max()):.3e} beyond its bound"


def setup(shape, T, seed, post, gate):
    L = mi.make_layer(shape, seed, "cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = shape.x_dtype

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda").to(smg.TORCH_DTYPES[dt])

    w = [1.0 + 0.1 * rnd(shape.H) for _ in range(3)]
    before = smg.Norm(shape.H, h_dtype=dt, x_dtype=dt, pre_w=w[0])
    after = smg.Norm(shape.H, h_dtype=dt, x_dtype=dt, pre_w=w[1], post_w=w[2] if post else None, gate=gate, gate_dtype=dt)
    gt = {"none": None, "token": (T,), "channel": (shape.H,)}[gate]
    return L, before, after, rnd(T, shape.H), None if gt is None else rnd(*gt)


@pytest.mark.parametrize("shape,T,post,gate", [(QWEN, 1, False, "none"), (QWEN, 2, True, "channel"),
                                               (QWEN, 3, False, "token"), (TINY, 4, True, "none"),
                                               (SMALL, 37, True, "channel"), (QWEN, 65, False, "none")])
def test_block_is_its_three_steps(gpu_lib, shape, T, post, gate):
    """Norm and residual step against their definitions on the layer's own input and output, the layer
    between them against the oracle."""
    L, before, after, h, gt = setup(shape, T, 400 + T, post, gate)
    lay = smg.Layer.from_shape(L, shape)
    ws = smg.new_workspace_block(lay, T)
    ho, xn = torch.empty_like(h), torch.empty_like(h)
    ids, w = torch.empty(T, shape.k, device="cuda", dtype=torch.int32), torch.empty(T, shape.k, device="cuda")
    smg.redmoe_forward_block(lay, before, after, h, ho, ids, w, ws, x_next=xn, gate=gt)
    smg.redmoe_check_timeout(ws)

    x, out = torch.empty_like(h), torch.empty(T, shape.H, device="cuda")
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    smg.redmoe_norm_forward(before, h, x=x)
    smg.redmoe_forward(lay, x, out, ids2, w2, smg.new_workspace(lay, T))
    _, vx, _, mx = NormCase(h, pre_w=before.pre_w).forward()
    close("x", x, vx, 64 * U * mx)
    out_tol, w_tol = tolerances(shape)
    r = assert_layer_parity(shape, L, x, out, ids2, w2, out_tol, w_tol, "layer in the block")
    assert torch.equal(ids, ids2)
    # the batched layer adds expert outputs in any order: within out_tol of its RMS, not to the bit
    case = NormCase(h, out, gt, after.pre_w, after.post_w, post=post, kind=gate)
    vh, vx, mh, mx = case.forward()
    g, rr, w1 = case.act_gate()[0].abs(), case.r(case.y) if post else 1.0, case.w(case.post_w).abs() if post else 1.0
    loose = (1e-6 if T > 4 else 0.0) * 64 * r["rms"]
    slack = g * rr * w1 * loose
    close("h_out", ho, vh, 64 * U * mh + slack)
    close("x_next", xn, vx, 64 * U * mx + 4 * slack.max() * case.r(vh) * case.w(case.pre_w).abs())


def test_block_in_place_without_next_norm_and_in_a_graph(gpu_lib):
    shape, T = QWEN, 1
    L, before, after, h, _ = setup(shape, T, 9, False, "none")
    lay = smg.Layer.from_shape(L, shape)
    ws = smg.new_workspace_block(lay, T)
    ids, w = torch.empty(T, shape.k, device="cuda", dtype=torch.int32), torch.empty(T, shape.k, device="cuda")
    want, start = torch.empty_like(h), h.clone()
    smg.redmoe_forward_block(lay, before, after, h, want, ids, w, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smg.redmoe_forward_block(lay, before, after, h, h, ids, w, ws)
    h.copy_(start)
    graph.replay()
    smg.redmoe_check_timeout(ws)
    assert torch.equal(h, want)


def test_decode_step_of_two_blocks_and_a_head(gpu_lib):
    """Two blocks, each handing the next one its normalised input, then an int4 head on the last."""
    shape, T = QWEN, 1
    hs, xs = [], []
    h = None
    for i in range(2):
        L, before, after, h0, _ = setup(shape, T, 600 + i, i == 1, "none")
        h = h0 if h is None else hs[-1]
        lay = smg.Layer.from_shape(L, shape)
        ws = smg.new_workspace_block(lay, T)
        ids, w = torch.empty(T, shape.k, device="cuda", dtype=torch.int32), torch.empty(T, shape.k, device="cuda")
        ho, xn = torch.empty_like(h), torch.empty_like(h)
        smg.redmoe_forward_block(lay, before, after, h, ho, ids, w, ws, x_next=xn)
        smg.redmoe_check_timeout(ws)
        hs.append(ho)
        xs.append(xn)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    hw, hsc = mi.quantize_int4g32(0.02 * torch.randn(1000, shape.H, generator=g, device="cuda"))
    y = torch.empty(T, 1000, device="cuda")
    smg.redmoe_gemv(smg.Matrix(hw, hsc, 1000, shape.H), xs[-1], y)
    v, m, ms = gemv_rows(hw, hsc, xs[-1])
    assert bool(((y.cpu().double() - v).abs() <= store_tol(v, gemv_err(m, ms, shape.H), torch.float32)).all())
    assert bool(xs[-1].isfinite().all())


def test_router_training_step(gpu_lib):
    """Losses of a router behind a norm and their way back to the residual stream: the gradient of the
    logits, of the router's input and weight (plain products) and of the norm, against 64 bits."""
    shape, T = SMALL, 24
    L, before, _, h, _ = setup(shape, T, 71, False, "none")
    lay = smg.Layer.from_shape(L, shape)
    x = torch.empty_like(h)
    ids, w = torch.empty(T, shape.k, device="cuda", dtype=torch.int32), torch.empty(T, shape.k, device="cuda")
    sg, lg = torch.empty(T, device="cuda"), torch.empty(T, shape.E, device="cuda")
    smg.redmoe_norm_forward(before, h, x=x)
    smg.redmoe_router(lay, x, ids, w, sg, smg.new_workspace(lay, T), logits=lg)
    loss, prob = torch.empty(2, device="cuda"), torch.empty(shape.E, device="cuda")
    counts, n = torch.empty(shape.E, device="cuda", dtype=torch.int32), torch.empty(1, device="cuda", dtype=torch.int32)
    smg.redmoe_balance_forward(lg, ids, loss, counts, prob, n, smg.new_balance_workspace(T, shape.E))
    coef = torch.tensor([1.0, 0.1], device="cuda")
    dl = torch.empty_like(lg)
    smg.redmoe_balance_backward(lg, counts, n, coef, dl, shape.k)
    dx = (dl @ L["router_w"].float()).to(x.dtype)
    dh, dw = torch.empty_like(h), torch.empty(shape.H, device="cuda")
    smg.redmoe_norm_backward(before, h, dh, smg.new_norm_workspace(before, T), dx=dx, dpre_w=dw)
    rd, md = balance_backward(lg, counts, int(n), shape.k, coef.tolist())
    assert bool(((dl.cpu().double() - rd).abs() <= store_tol(rd, 128 * U * md, torch.float32)).all())
    ref = NormCase(h, pre_w=before.pre_w).backward(None, dx)
    close("dh", dh, ref["dh"][0], 256 * U * ref["dh"][1])
    close("dw", dw, ref["dpre_w"][0], 256 * U * ref["dpre_w"][1])
    # the whole way: the router's losses as a function of h, by 64-bit autograd through the same selection.
    # h_out, x and dx are stored in bf16: a few half steps (2^-8 each) of the largest gradient
    hh = d(h).requires_grad_()
    xx = hh * torch.rsqrt(hh.pow(2).mean(1, keepdim=True) + 1e-6) * d(before.pre_w)
    ll = xx @ d(L["router_w"]).T
    p = torch.softmax(ll, 1)
    f = counts.cpu().double() / (T * shape.k)
    (shape.E * (f * p.mean(0)).sum() + 0.1 * torch.logsumexp(ll, 1).pow(2).mean()).backward()
    assert float((dh.cpu().double() - hh.grad).abs().max()) <= 8 * 2.0 ** -8 * float(hh.grad.abs().max())


@pytest.mark.parametrize("T,H", [(1, 264), (37, 264), (300, 2048)])
def test_calls_that_follow_one_another_closely(gpu_lib, T, H):
    """A call's kernel may be placed while the one before it ends. A chain in which each call reads or
    overwrites what the ones before it read or wrote (rows that end inside a sector, in place, with copies
    and fills between, over two streams) equals the same calls one at a time, eager and captured."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)

    def rnd(*s, dt=torch.bfloat16):
        return torch.randn(*s, generator=g, device="cuda").to(dt)

    step = smg.Norm(H, y_dtype="bf16", pre_w=rnd(H), post_w=rnd(H), gate="element", gate_act="sigmoid", res_scale=0.5)
    wide = smg.Norm(H, pre_w=rnd(H))
    n = -(-H // 32) * 32
    mats = [smg.Matrix(*mi.quantize_int4g32(torch.randn(H, n, generator=g, device="cuda")), H, n) for _ in range(2)]
    E, k, rows = 61, 3, min(T, 32)
    first = {"h": rnd(T, H), "y": rnd(T, H), "x": rnd(T, H), "gate": rnd(T, H), "in": rnd(rows, n), "lg": rnd(T, E, dt=torch.float32)}
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ws, wb = smg.new_norm_workspace(step, T), smg.new_balance_workspace(T, E)
    side = torch.cuda.Stream()

    def chain(s, wait):
        out = {"dh": torch.empty_like(s["h"]), "dy": torch.empty_like(s["y"]), "dg": torch.empty_like(s["gate"]),
               "dpre": torch.empty(H, device="cuda"), "dpost": torch.empty(H, device="cuda")}
        loss, prob = torch.empty(2, device="cuda"), torch.empty(E, device="cuda")
        counts, nr = torch.empty(E, device="cuda", dtype=torch.int32), torch.empty(1, device="cuda", dtype=torch.int32)
        coef = torch.ones(2, device="cuda")
        for i in range(6):
            for j in range(3):
                smg.redmoe_norm_forward(step, s["h"], h_out=s["h"], x=s["x"], y=s["y"], gate=s["gate"])
                wait()
            s["in"].zero_()
            s["in"][:, :H].copy_(s["x"][:rows])
            wait()
            smg.redmoe_gemv(mats[i % 2], s["in"], s["y"][:rows])   # the next step's y
            wait()
            smg.redmoe_norm_backward(step, s["h"], out["dh"], ws, dh_out=s["x"], dx=s["gate"], y=s["y"], gate=s["gate"],
                                     dy=out["dy"], dgate=out["dg"], dpost_w=out["dpost"], dpre_w=out["dpre"])
            wait()
            side.wait_stream(torch.cuda.current_stream())
            smg.redmoe_balance_forward(s["lg"], ids, loss, counts, prob, nr, wb, stream=side)
            smg.redmoe_balance_backward(s["lg"], counts, nr, coef, s["lg"], k, stream=side)   # in place
            wait()
            smg.redmoe_norm_forward(wide, out["dh"], x=s["gate"])   # the next step's gate
            torch.cuda.current_stream().wait_stream(side)
            wait()
            smg.redmoe_balance_backward(s["lg"], counts, nr, coef, s["lg"], k)
            wait()
        return {**s, **out, "loss": loss, "counts": counts, "prob": prob}

    want = chain({k_: v.clone() for k_, v in first.items()}, torch.cuda.synchronize)
    torch.cuda.synchronize()
    got = chain({k_: v.clone() for k_, v in first.items()}, lambda: None)
    torch.cuda.synchronize()
    assert all(bool(v.isfinite().all()) for v in want.values())
    assert all(torch.equal(got[n_], want[n_]) for n_ in want), [n_ for n_ in want if not torch.equal(got[n_], want[n_])]
    held = {k_: v.clone() for k_, v in first.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(held, lambda: None)
    for _ in range(3):
        for n_, v in first.items():
            held[n_].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n_], want[n_]) for n_ in want), [n_ for n_ in want if not torch.equal(got[n_], want[n_])]
