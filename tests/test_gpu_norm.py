"""The step between blocks (redmoe_norm_forward, redmoe_norm_backward) against its definition
in 64 bits.

Tolerances: every result is a fixed expression of fp32 operations on exact inputs. A sum over a
row is at most 16 products of a thread, 5 shuffle steps and 16 warps deep, rsqrtf adds a few units,
each of the few further products one, and the logistic function of a gate a up to |a| + 6 (the exponent's
rounding, ex2 and the reciprocal), a dozen for normal gates: under 64 U of the result's magnitude
forward. Backward chains two such reductions, and a column sum adds the rows of a
thread, up to 8 groups and up to 37 + 8 blocks: under 256 U for the sizes here. A stored value
adds half a step of its type.
"""

import pytest
import torch

import sparse_moe_gemv_b200 as smg
from plain_ops import NormCase, U, store_tol

pytestmark = pytest.mark.gpu

DT = smg.TORCH_DTYPES


def make(T, H, h="bf16", y="f32", x="bf16", w="bf16", post=False, kind="none", act="linear", gdt="bf16", offset=0.0,
         res=1.0, block=1.0, branch=True, seed=0, weights=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 + seed)

    def rnd(*s, dt="f32"):
        return torch.randn(*s, generator=g, device="cuda").to(DT[dt])

    t = {"h": rnd(T, H, dt=h), "y": rnd(T, H, dt=y) if branch else None,
         "pre_w": rnd(H, dt=w) if weights else None, "post_w": rnd(H, dt=w) if post and weights else None}
    shape = {"none": None, "token": (T,), "channel": (H,), "element": (T, H)}[kind]
    t["gate"] = rnd(*shape, dt=gdt) if shape and branch else None
    norm = smg.Norm(H, h_dtype=h, y_dtype=y, x_dtype=x, pre_w=t["pre_w"], post_w=t["post_w"], post_norm=post, gate=kind,
                    gate_act=act, gate_dtype=gdt, w_offset=offset, res_scale=res, block_scale=block)
    kw = dict(post=post, kind=kind if branch else "none", act=act, offset=offset, res=res, block=block)
    t.update(dh_out=rnd(T, H, dt=h), dx=rnd(T, H, dt=x))
    return norm, t, kw


def plain(t, kw):
    return NormCase(t["h"], t["y"], t["gate"], t["pre_w"], t["post_w"], **kw)


def close(name, got, value, err):
    got = got.cpu()
    bad = (got.double() - value).abs() - store_tol(value, err, got.dtype)
    assert not torch.isnan(got).any(), f"{name}: NaN"
    assert bad.numel() == 0 or float(bad.max()) <= 0, f"{name}: {float(bad.max()):.3e} beyond its bound"


def forward(norm, t, pad=3):
    """h_out and x in buffers with rows behind the last one, which must stay as they were."""
    T, H = t["h"].shape
    ho = torch.full((T + pad, H), 7.0, device="cuda", dtype=norm.h_torch)
    x = torch.full((T + pad, H), 7.0, device="cuda", dtype=norm.x_torch)
    branch = t["y"] is not None
    smg.redmoe_norm_forward(norm, t["h"], h_out=ho[:T] if branch else None, x=x[:T], y=t["y"], gate=t["gate"])
    torch.cuda.synchronize()
    assert bool((ho[T if branch else 0:] == 7.0).all()) and bool((x[T:] == 7.0).all())
    return ho[:T], x[:T]


def backward(norm, t, T, H, dx=True, dh_out=True):
    full = lambda *s, dt=torch.float32: torch.full(s, float("nan"), device="cuda", dtype=dt)  # noqa: E731
    branch = t["y"] is not None
    o = {"dh": full(T, H, dt=norm.h_torch), "dy": full(T, H, dt=norm.y_torch) if branch else None,
         "dpre_w": full(H) if dx and t["pre_w"] is not None else None,
         "dpost_w": full(H) if t["post_w"] is not None else None, "dgate": None}
    if t["gate"] is not None:
        o["dgate"] = full(*t["gate"].shape, dt=norm.gate_torch if norm.gate == "element" else torch.float32)
    ws = smg.new_norm_workspace(norm, T)
    smg.redmoe_norm_backward(norm, t["h"], o["dh"], ws, dh_out=t["dh_out"] if dh_out else None,
                             dx=t["dx"] if dx else None, y=t["y"], gate=t["gate"], dy=o["dy"], dgate=o["dgate"],
                             dpost_w=o["dpost_w"], dpre_w=o["dpre_w"])
    torch.cuda.synchronize()
    return {n: v for n, v in o.items() if v is not None}


CASES = [
    dict(T=1, H=2048), dict(T=1, H=8, h="f32", x="f32"), dict(T=2, H=2048, y="bf16", post=True),
    dict(T=5, H=264, h="f32", y="f32", x="f32", w="f32", post=True, kind="token", act="sigmoid", gdt="f32", block=0.25),
    dict(T=33, H=256, post=True, kind="channel", offset=1.0, res=0.9),
    dict(T=19, H=1000, h="f32", y="bf16", post=True, kind="element", act="sigmoid", offset=1.0),
    dict(T=300, H=520, kind="element", gdt="f32", block=0.5), dict(T=7, H=4096, y="bf16", kind="token"),
    dict(T=3, H=4104, h="f32", x="f32", post=True, kind="channel", act="sigmoid", gdt="f32"),
    dict(T=4, H=8192, h="bf16", y="bf16", post=True, kind="element"), dict(T=601, H=64, post=True, kind="channel"),
    dict(T=9, H=2048, post=True, weights=False), dict(T=6, H=136, branch=False), dict(T=2, H=8192, branch=False, x="f32"),
    dict(T=1, H=1024, branch=False, h="f32"), dict(T=70, H=5120, y="bf16", post=True, kind="channel", act="sigmoid"),
    # y of fp32 under every pair of the other types, and bf16 under the rest
    dict(T=3, H=320, h="f32", y="f32", x="bf16"), dict(T=3, H=320, h="bf16", y="f32", x="f32"),
    dict(T=3, H=320, h="f32", y="bf16", x="f32", w="f32"), dict(T=3, H=320, h="bf16", y="bf16", x="f32"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_forward(gpu_lib, case):
    norm, t, kw = make(**case)
    ho, x = forward(norm, t)
    vh, vx, mh, mx = plain(t, kw).forward()
    if t["y"] is not None:
        close("h_out", ho, vh, 64 * U * mh)
    close("x", x, vx, 64 * U * mx)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_backward(gpu_lib, case):
    norm, t, kw = make(**case)
    o = backward(norm, t, case["T"], case["H"])
    ref = plain(t, kw).backward(t["dh_out"], t["dx"])
    assert set(ref) - ({"dpre_w", "dpost_w"} if not case.get("weights", True) else set()) == set(o)
    for n in o:
        close(n, o[n], ref[n][0], 256 * U * ref[n][1])


@pytest.mark.parametrize("dx,dh_out", [(True, False), (False, True)])
@pytest.mark.parametrize("branch", [True, False])
def test_backward_with_one_arriving_gradient(gpu_lib, dx, dh_out, branch):
    norm, t, kw = make(11, 512, post=branch, kind="channel" if branch else "none", branch=branch)
    o = backward(norm, t, 11, 512, dx=dx, dh_out=dh_out)
    ref = plain(t, kw).backward(t["dh_out"] if dh_out else None, t["dx"] if dx else None)
    for n in o:
        close(n, o[n], ref[n][0], 256 * U * ref[n][1])


def test_backward_matches_differences_of_the_kernel(gpu_lib):
    """dh, dy and the weights' gradients against central differences of the forward kernel itself
    (fp32 storage; step 1/64: truncation step^2 / 6 times a third derivative of order 1 on a
    cotangent of norm sqrt(T H), rounding 64 U T H / step)."""
    T, H = 2, 16
    norm, t, kw = make(T, H, h="f32", x="f32", w="f32", post=True, kind="token", act="sigmoid", gdt="f32")
    vh = plain(t, kw).forward()[0].float().cuda()

    def value(**over):
        u = {**t, **over}
        n = smg.Norm(H, h_dtype="f32", y_dtype="f32", x_dtype="f32", pre_w=u["pre_w"], post_w=u["post_w"], gate="token",
                     gate_act="sigmoid", gate_dtype="f32")
        ho, x = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
        smg.redmoe_norm_forward(n, u["h"], h_out=ho, x=x, y=u["y"], gate=u["gate"])
        return float((ho.double() * t["dh_out"].double()).sum() + (x.double() * t["dx"].double()).sum())

    t["dh_out"] = t["dh_out"].float()
    o = backward(norm, {**t, "h": vh}, T, H)
    step = 2.0 ** -6
    for name, key in (("dh", "h"), ("dy", "y"), ("dpre_w", "pre_w"), ("dpost_w", "post_w"), ("dgate", "gate")):
        for i in range(t[key].numel()):
            e = torch.zeros(t[key].numel(), device="cuda")
            e[i] = step
            e = e.reshape(t[key].shape)
            diff = (value(**{key: t[key] + e}) - value(**{key: t[key] - e})) / (2 * step)
            assert abs(diff - float(o[name].reshape(-1)[i])) < 0.02, (name, i)


def test_rows_are_independent_and_extremes_stay_in_their_row(gpu_lib):
    T, H = 8, 512
    norm, t, kw = make(T, H, h="f32", x="f32", post=True)
    want, want_x = (v.clone() for v in forward(norm, t))
    t["y"][2] = float("nan")
    t["h"][4, 7] = float("inf")
    t["y"][6] = 0.0
    t["h"][6] = 0.0
    ho, x = forward(norm, t)
    keep = [0, 1, 3, 5, 7]
    assert torch.equal(ho[keep], want[keep]) and torch.equal(x[keep], want_x[keep])
    assert bool(ho[2].isnan().all()) and bool(x[2].isnan().all())
    assert float(ho[4, 7]) == float("inf") and bool(x[4, 7].isnan())
    assert float(ho[6].abs().max()) == 0.0 and float(x[6].abs().max()) == 0.0  # eps keeps a zero row finite


def test_in_place(gpu_lib):
    norm, t, _ = make(17, 1024, post=True)
    want, want_x = (v.clone() for v in forward(norm, t))
    x = torch.empty_like(want_x)
    h = t["h"].clone()
    smg.redmoe_norm_forward(norm, h, h_out=h, x=x, y=t["y"])
    assert torch.equal(h, want) and torch.equal(x, want_x)
    o = backward(norm, t, 17, 1024)
    dh, dy = t["dh_out"].clone(), torch.empty_like(o["dy"])
    smg.redmoe_norm_backward(norm, t["h"], dh, None, dh_out=dh, dx=t["dx"], y=t["y"], dy=dy)  # no weight gradients
    assert torch.equal(dh, o["dh"]) and torch.equal(dy, o["dy"])


def test_no_rows(gpu_lib):
    norm, t, _ = make(0, 256, post=True, kind="channel")
    forward(norm, t)
    o = backward(norm, t, 0, 256)
    for n in ("dpre_w", "dpost_w", "dgate"):
        assert float(o[n].abs().max()) == 0.0


def test_same_bits_twice_on_another_stream_and_in_a_graph(gpu_lib):
    T, H = 777, 512
    norm, t, kw = make(T, H, post=True, kind="channel")
    first, first_x = (v.clone() for v in forward(norm, t))
    grads = backward(norm, t, T, H)
    again = backward(norm, t, T, H)
    assert all(torch.equal(grads[n], again[n]) for n in grads)
    s = torch.cuda.Stream()
    ho, x = torch.empty_like(first), torch.empty_like(first_x)
    o = {n: torch.empty_like(v) for n, v in grads.items()}
    ws = smg.new_norm_workspace(norm, T)

    def both():
        smg.redmoe_norm_forward(norm, t["h"], h_out=ho, x=x, y=t["y"], gate=t["gate"])
        smg.redmoe_norm_backward(norm, t["h"], o["dh"], ws, dh_out=t["dh_out"], dx=t["dx"], y=t["y"], gate=t["gate"],
                                 dy=o["dy"], dgate=o["dgate"], dpost_w=o["dpost_w"], dpre_w=o["dpre_w"])

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    assert torch.equal(ho, first) and torch.equal(x, first_x) and all(torch.equal(o[n], grads[n]) for n in grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    t["y"].mul_(2.0)  # new inputs in the captured buffers
    for v in (ho, x, *o.values()):
        v.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    want, want_x = forward(norm, t)
    grads = backward(norm, t, T, H)
    assert torch.equal(ho, want) and torch.equal(x, want_x) and all(torch.equal(o[n], grads[n]) for n in grads)


@pytest.mark.parametrize("T,H", [(5, 264), (37, 64), (300, 16), (64, 2048)])
def test_repeated_calls_with_one_workspace(gpu_lib, T, H):
    """A few blocks' sums are added within a cluster, more by a second kernel: both leave the control block
    zero and the same workspace serves the next call, other sizes, gradients left out and replays included."""
    norm, t, kw = make(T, H, post=True, kind="channel")
    first = backward(norm, t, T, H)
    ws = smg.new_norm_workspace(norm, T)
    o = {n: torch.empty_like(v) for n, v in first.items()}

    def call(rows=T, **drop):
        kw = dict(dgate=o["dgate"], dpost_w=o["dpost_w"], dpre_w=o["dpre_w"])
        kw.update(drop)
        smg.redmoe_norm_backward(norm, t["h"][:rows], o["dh"][:rows], ws, dh_out=t["dh_out"][:rows], dx=t["dx"][:rows],
                                 y=t["y"][:rows], gate=t["gate"], dy=o["dy"][:rows], **kw)

    for drop in ({}, dict(dgate=None), dict(dpost_w=None), dict(dpre_w=None), dict(rows=1), dict(dgate=None, dpre_w=None)):
        call(**drop)
        torch.cuda.synchronize()
        assert int(ws[:256].count_nonzero()) == 0
        for v in o.values():
            v.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(o[n], first[n]) for n in first) and int(ws[:256].count_nonzero()) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(3):
        for v in o.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[n], first[n]) for n in first) and int(ws[:256].count_nonzero()) == 0


def test_calls_at_once_with_workspaces_of_their_own(gpu_lib):
    cases = [make(T, H, post=True, kind="channel", seed=i) for i, (T, H) in enumerate([(37, 64), (700, 512), (5, 264), (64, 2048)])]
    want = [backward(n, t, *t["h"].shape) for n, t, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    works = [smg.new_norm_workspace(n, t["h"].shape[0]) for n, t, _ in cases]
    got = [{k: torch.empty_like(v) for k, v in w.items()} for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (n, t, _), o, ws, s in zip(cases, got, works, streams):
            smg.redmoe_norm_backward(n, t["h"], o["dh"], ws, dh_out=t["dh_out"], dx=t["dx"], y=t["y"], gate=t["gate"],
                                     dy=o["dy"], dgate=o["dgate"], dpost_w=o["dpost_w"], dpre_w=o["dpre_w"], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        assert all(torch.equal(o[k], w[k]) for k in w)


def test_offsets_beyond_32_bits(gpu_lib):
    """More than 2^31 elements: the last rows, forward and backward, equal those of a small call."""
    T, H = 2 ** 18 + 5, 8192
    w = torch.randn(H, device="cuda").to(torch.bfloat16)
    norm = smg.Norm(H, pre_w=w)
    h = torch.empty(T, H, device="cuda", dtype=torch.bfloat16).normal_()
    x = torch.empty_like(h)
    smg.redmoe_norm_forward(norm, h, x=x)
    tail = torch.empty(8, H, device="cuda", dtype=torch.bfloat16)
    smg.redmoe_norm_forward(norm, h[-8:], x=tail)
    assert torch.equal(x[-8:], tail)
    smg.redmoe_norm_backward(norm, h, x, None, dx=h.clone())
    smg.redmoe_norm_backward(norm, h[-8:], tail, None, dx=h[-8:].clone())
    assert torch.equal(x[-8:], tail)


def test_binding_refusals_on_the_device(gpu_lib):
    norm, t, _ = make(4, 256, post=True)
    ok = torch.empty_like(t["h"])
    for bad in (dict(h=t["h"].float()), dict(h=t["h"][:, :128]), dict(h=t["h"].t().contiguous().t()),
                dict(y=t["y"][:2]), dict(h_out=t["h"].float()), dict(x=torch.empty(4, 256)), dict(gate=t["y"])):
        a = {**dict(h=t["h"], h_out=ok, x=torch.empty_like(ok), y=t["y"], gate=None), **bad}
        with pytest.raises(ValueError):
            smg.redmoe_norm_forward(norm, **a)
    with pytest.raises(smg.RedmoeError, match="INVALID_ARG"):
        smg.redmoe_norm_forward(norm, t["h"], h_out=ok, x=ok, y=t["y"])
    with pytest.raises(smg.RedmoeError, match="WORKSPACE"):
        smg.redmoe_norm_backward(norm, t["h"], ok, None, dh_out=t["dh_out"], dx=t["dx"], y=t["y"],
                                 dy=torch.empty_like(t["y"]), dpre_w=torch.empty(256, device="cuda"))
