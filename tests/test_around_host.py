"""Host-side checks of the operators around the layer (no GPU): argument refusals of the C ABI
and of the binding, and the plain 64-bit gradients against central differences."""

import ctypes as C
import os

import pytest
import torch

import sparse_moe_gemv_b200 as smg
from plain_ops import NormCase, balance_backward, balance_forward

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x7f0000000000     # 256-byte aligned addresses that these calls never dereference,
STEP = 0x100000000     # 4 GiB apart: no range meets another


def at(i):
    return A + STEP * i


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(smg.LIB_PATH):
        from sparse_moe_gemv_b200 import build
        build.build()
    return smg.load()


def norm_struct(**over):
    s = smg._Norm(hidden=2048, h_dtype=1, y_dtype=0, x_dtype=1, w_dtype=1, post_norm=1, gate_kind=2, gate_act=1,
                  gate_dtype=1, eps=1e-6, w_offset=1.0, res_scale=1.0, block_scale=1.0, post_w=at(1), pre_w=at(2))
    for k, v in over.items():
        setattr(s, k, v)
    return s


def fwd(lib, N, h=at(3), y=at(4), gate=at(5), T=0, h_out=at(6), x=at(7)):
    return lib.redmoe_norm_forward(C.byref(N), h, y, gate, T, h_out, x, None)


@pytest.mark.parametrize("over,expect", [
    (dict(hidden=0), INVALID), (dict(hidden=2050), INVALID), (dict(hidden=-8), INVALID), (dict(hidden=8200), UNSUPPORTED),
    (dict(h_dtype=7), INVALID), (dict(h_dtype=2), UNSUPPORTED), (dict(gate_dtype=3), UNSUPPORTED),
    (dict(gate_kind=4), INVALID), (dict(gate_act=2), INVALID), (dict(post_norm=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(res_scale=float("inf")), INVALID), (dict(pre_w=at(2) + 8), INVALID),
    (dict(post_norm=0), INVALID), (dict(), OK),
])
def test_norm_descriptor_refusals(lib, over, expect):
    N = norm_struct(**over)
    assert fwd(lib, N) == expect
    assert (lib.redmoe_norm_workspace_bytes(C.byref(N), 4) > 0) == (expect == OK)


def test_norm_forward_refusals(lib):
    N = norm_struct()
    H2, H4 = 2048 * 2, 2048 * 4
    assert lib.redmoe_norm_forward(None, at(3), at(4), at(5), 1, at(6), at(7), None) == INVALID
    assert fwd(lib, N, T=-1) == INVALID
    for bad in (dict(h=None), dict(h=at(3) + 8), dict(y=at(4) + 4), dict(gate=None), dict(gate=at(5) + 2),
                dict(h_out=None), dict(x=at(7) + 2),
                dict(y=None), dict(y=None, gate=None), dict(y=None, gate=None, h_out=None, x=None)):
        assert fwd(lib, N, T=4, **bad) == INVALID, bad
    # overlaps: outputs with inputs (h_out == h alone is allowed), with one another, with a weight
    for bad in (dict(h_out=at(3) + H2), dict(x=at(3)), dict(x=at(6) + 3 * H2), dict(x=at(4) + 3 * H4), dict(h_out=at(5)),
                dict(h_out=at(2)), dict(x=at(1) + H2 - 16)):
        assert fwd(lib, N, T=4, **bad) == INVALID, bad


def bwd(lib, N, T=4, ws=at(20), ws_bytes=1 << 31, **over):
    a = dict(h_out=at(3), y=at(4), gate=at(5), dh_out=at(6), dx=at(7), dh=at(8), dy=at(9), dgate=at(10), dpost_w=at(11),
             dpre_w=at(12))
    a.update(over)
    return lib.redmoe_norm_backward(C.byref(N), a["h_out"], a["y"], a["gate"], a["dh_out"], a["dx"], T, a["dh"], a["dy"],
                                    a["dgate"], a["dpost_w"], a["dpre_w"], ws, ws_bytes, None)


def test_norm_backward_refusals(lib):
    N = norm_struct()
    need = lib.redmoe_norm_workspace_bytes(C.byref(N), 4)
    assert need % 256 == 0 and need >= 4 * 2 * 2048 * 4  # two column sums a block
    for bad in (dict(T=-1), dict(h_out=None), dict(dh=None), dict(dy=None), dict(gate=None), dict(dh_out=None, dx=None),
                dict(dx=None), dict(dh=at(8) + 4), dict(dpost_w=at(11) + 4), dict(y=None), dict(dh=at(3)), dict(dy=at(4)),
                dict(dh=at(6) + 16), dict(dgate=at(8)), dict(dpre_w=at(11) + 16), dict(dpre_w=at(20)), dict(dy=at(2))):
        assert bwd(lib, N, **bad) == INVALID, bad
    assert bwd(lib, norm_struct(pre_w=None)) == INVALID           # a gradient of a weight that is not there
    assert bwd(lib, norm_struct(post_w=None)) == INVALID
    assert bwd(lib, norm_struct(gate_kind=0), gate=None) == INVALID
    for bad in (dict(ws=None), dict(ws=at(20) + 128), dict(ws_bytes=need - 256)):
        assert bwd(lib, N, **bad) == WORKSPACE, bad


def bal(lib, T=8, E=16, k=2, dt=0, logits=at(1), ids=at(2), mask=at(3), loss=at(4), counts=at(5), prob=at(6), n=at(7),
        ws=at(8), ws_bytes=1 << 30):
    return lib.redmoe_balance_forward(logits, dt, ids, mask, T, E, k, loss, counts, prob, n, ws, ws_bytes, None)


def test_balance_refusals(lib):
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(E=64, k=33), dict(dt=9),
                dict(T=1 << 30, k=2), dict(logits=None), dict(logits=at(1) + 4), dict(ids=None), dict(ids=at(2) + 1),
                dict(loss=None), dict(counts=at(5) + 2), dict(prob=None), dict(n=None), dict(loss=at(1) + 16),
                dict(counts=at(6)), dict(n=at(3) + 4), dict(prob=at(8) + 512)):
        assert bal(lib, **bad) == INVALID, bad
    assert bal(lib, dt=2) == UNSUPPORTED
    need = lib.redmoe_balance_workspace_bytes(8, 16)
    assert need % 256 == 0 and need > 256
    for bad in (dict(ws=None), dict(ws=at(8) + 64), dict(ws_bytes=need - 1)):
        assert bal(lib, **bad) == WORKSPACE, bad
    assert lib.redmoe_balance_workspace_bytes(-1, 16) == 0 and lib.redmoe_balance_workspace_bytes(8, 2000) == 0

    def back(T=8, E=16, k=2, dt=0, logits=at(1), mask=at(3), counts=at(5), n=at(7), grad=at(9), dl=at(10)):
        return lib.redmoe_balance_backward(logits, dt, mask, T, E, k, counts, n, grad, dl, None)

    for bad in (dict(T=-1), dict(E=0), dict(k=99), dict(logits=None), dict(counts=None), dict(n=None), dict(grad=None),
                dict(dl=None), dict(dl=at(10) + 8), dict(dl=at(1) + 16), dict(dl=at(5) - 16), dict(dl=at(3))):
        assert back(**bad) == INVALID, bad
    assert back(dt=3) == UNSUPPORTED
    assert back(T=0) == OK


def test_gemv_refusals(lib):
    def gv(rows=64, cols=128, dt=2, w=at(1), s=at(2), x=at(3), xdt=1, T=1, y=at(4), ydt=0):
        M = smg._Matrix(rows=rows, cols=cols, dtype=dt, w=w, s=s)
        return lib.redmoe_gemv(C.byref(M), x, xdt, T, y, ydt, None)

    assert lib.redmoe_gemv(None, at(3), 1, 1, at(4), 0, None) == INVALID
    for bad in (dict(rows=0), dict(cols=0), dict(cols=100), dict(dt=9), dict(xdt=-1), dict(T=-1), dict(w=None),
                dict(w=at(1) + 8), dict(s=None), dict(s=at(2) + 2), dict(x=None), dict(x=at(3) + 2), dict(y=None),
                dict(y=at(4) + 2), dict(y=at(3)), dict(y=at(1) + 64 * 64 - 4), dict(y=at(2))):
        assert gv(**bad) == INVALID, bad
    for bad in (dict(dt=1), dict(dt=3), dict(xdt=0), dict(ydt=2), dict(T=33), dict(cols=65568)):
        assert gv(**bad) == UNSUPPORTED, bad
    assert gv(T=0) == OK


def layer_struct(**over):
    s = smg._Layer()
    s.hidden, s.n_experts, s.top_k, s.inter, s.shared_inter = 2048, 512, 10, 512, 512
    s.x_dtype = s.router_dtype = s.expert_dtype = 1
    for i, (name, _) in enumerate(smg._Layer._fields_[8:]):
        setattr(s, name, at(40 + i))
    s.router_bias = None
    for k, v in over.items():
        setattr(s, k, v)
    return s


def test_block_refusals(lib):
    L = layer_struct()
    before, after = norm_struct(), norm_struct(gate_kind=0)

    def blk(L=L, before=before, after=after, h=at(3), gate=None, T=1, h_out=at(4), x_next=at(5), ids=at(6), w=at(7),
            ws=at(8), ws_bytes=1 << 31):
        return lib.redmoe_forward_block(C.byref(L), C.byref(before), C.byref(after), h, gate, T, h_out, x_next, ids, w, ws,
                                        ws_bytes, None)

    assert blk(T=0) == OK
    assert blk(T=-1) == INVALID and blk(L=layer_struct(top_k=0)) == INVALID
    for bad in (dict(before=norm_struct(hidden=1024)), dict(after=norm_struct(hidden=1024)),
                dict(before=norm_struct(x_dtype=0)), dict(after=norm_struct(gate_kind=0, y_dtype=1)),
                dict(after=norm_struct(gate_kind=0, h_dtype=0)), dict(h=None), dict(h_out=None), dict(ids=None),
                dict(w=at(7) + 2), dict(gate=at(9)), dict(h=at(3) + 8), dict(h_out=at(3) + 16), dict(x_next=at(4)),
                dict(ids=at(4)), dict(x_next=at(8) + 256)):
        assert blk(**bad) == INVALID, bad
    need = lib.redmoe_workspace_bytes_block(C.byref(L), 1)
    assert need >= lib.redmoe_workspace_bytes(C.byref(L), 1) + 2048 * 6
    assert blk(ws=None) == WORKSPACE and blk(ws_bytes=need - 256) == WORKSPACE
    assert blk(L=layer_struct(inter=192), T=5) == UNSUPPORTED      # rows the batched path does not take
    assert blk(L=layer_struct(expert_dtype=3), T=2) == UNSUPPORTED  # int2 experts: one row only


def test_binding_refuses_tensors_it_would_misread():
    """Wrong device, type, shape and layout raise ValueError before the library is called."""
    n = smg.Norm(64, h_dtype="f32", x_dtype="f32")
    with pytest.raises(ValueError, match="CUDA"):
        smg.redmoe_norm_forward(n, torch.zeros(2, 64), x=torch.zeros(2, 64))
    with pytest.raises(ValueError, match="one dtype"):
        smg.Norm(64, pre_w=torch.zeros(64), post_w=torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        smg.Norm(64, pre_w=torch.zeros(64, dtype=torch.float16))
    with pytest.raises(ValueError):
        smg.redmoe_balance_forward(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(2),
                                   torch.zeros(8, dtype=torch.int32), torch.zeros(8), torch.zeros(1, dtype=torch.int32),
                                   torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError):
        smg.Matrix(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.bfloat16), 4, 32)


def test_binding_refuses_sizes_that_int32_would_cut():
    """ctypes drops the upper bits of a long integer: 2^32 + 8 would arrive as 8."""
    for n in (2 ** 31, 2 ** 32 + 8):
        with pytest.raises(ValueError, match="int32"):
            smg.Norm(n)
        with pytest.raises(ValueError, match="int32"):
            smg.redmoe_balance_workspace_bytes(n, 8)
        with pytest.raises(ValueError, match="int32"):
            smg.redmoe_norm_workspace_bytes(smg.Norm(64), n)


@pytest.mark.parametrize("kind", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("post", [False, True])
def test_plain_norm_gradients_match_differences(kind, post):
    g = torch.Generator().manual_seed(3 + post)
    T, H, act = 3, 8, "sigmoid" if post else "linear"

    def rnd(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    gate = {"none": None, "token": rnd(T), "channel": rnd(H), "element": rnd(T, H)}[kind]
    v = {"h": rnd(T, H), "y": rnd(T, H), "pre_w": rnd(H), "post_w": rnd(H) if post else None, "gate": gate}
    ct, cx = rnd(T, H), rnd(T, H)
    kw = dict(post=post, kind=kind, act=act, offset=1.0, res=0.9, block=0.5)

    def f(**over):
        h_out, x, _, _ = NormCase(**{**v, **over}, **kw).forward()
        return float((h_out * ct).sum() + (x * cx).sum())

    h_out = NormCase(**v, **kw).forward()[0]
    got = NormCase(**{**v, "h": h_out}, **kw).backward(ct, cx)
    # central differences: step 1e-5 leaves about 1e-10 of truncation and 1e-11 of rounding
    for name, key in (("dh", "h"), ("dy", "y"), ("dpre_w", "pre_w"), ("dpost_w", "post_w"), ("dgate", "gate")):
        if v[key] is None:
            assert name not in got
            continue
        for i in range(v[key].numel()):
            e = torch.zeros_like(v[key]).reshape(-1)
            e[i] = 1e-5
            e = e.reshape(v[key].shape)
            diff = (f(**{key: v[key] + e}) - f(**{key: v[key] - e})) / 2e-5
            assert abs(diff - float(got[name][0].reshape(-1)[i])) < 1e-7, (name, i)


def test_plain_balance_gradients_match_differences():
    g = torch.Generator().manual_seed(9)
    T, E, k = 5, 6, 2
    l = torch.randn(T, E, generator=g, dtype=torch.float64)
    ids = l.topk(k, dim=1).indices.to(torch.int32)
    mask = torch.tensor([1, 0, 1, 1, 1], dtype=torch.uint8)
    _, counts, _, n, _ = balance_forward(l, ids, mask)
    grad = (0.7, -0.3)
    got, _ = balance_backward(l, counts, n, k, grad, mask)
    assert n == 4 and float(got[1].abs().max()) == 0.0
    for t in range(T):
        for e in range(E):
            s = torch.zeros_like(l)
            s[t, e] = 1e-5
            (a, *_), (b, *_) = balance_forward(l + s, ids, mask), balance_forward(l - s, ids, mask)
            diff = float((a - b) @ torch.tensor(grad, dtype=torch.float64)) / 2e-5
            assert abs(diff - float(got[t, e])) < 1e-7
