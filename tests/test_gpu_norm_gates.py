"""Gradients of sigmoid gates far from zero, and of rows beyond the fp32 range of their squares.

Tolerance: as in test_gpu_norm.py, 256 U of a gradient's magnitude for gates of order one. The slope
of the logistic function at a, s(a) s(-a), adds what rounding the exponent |a| log2(e) costs: the
constant is off by 0.7 U and the product by U, so e^-|a| by less than 2 |a| U; a closed gate's own value
likewise. Below the smallest normal fp32 number a result is held to that number.
"""

import pytest
import torch

from plain_ops import NormCase, U
from test_gpu_norm import backward, make

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -126
GATES = (-80.0, -20.0, -12.0, -6.0, 6.0, 10.0, 12.0, 15.0, 17.0, 20.0, 80.0)


class Slope(NormCase):
    """The slope without the difference 1 - s, which 64 bits cannot hold either from 37 on."""

    def act_gate(self):
        a = self.gate[:, None] if self.kind == "token" else self.gate
        return torch.sigmoid(a), torch.sigmoid(a) * torch.sigmoid(-a)


def plain(t, kw):
    return Slope(t["h"], t["y"], t["gate"], t["pre_w"], t["post_w"], **kw)


def close(name, got, value, err):
    got = got.cpu().double()
    bad = (got - value).abs() - (err * (1 + U) + U * value.abs() + TINY)
    assert not got.isnan().any() and float(bad.max()) <= 0, f"{name}: {float(bad.max()):.3e} beyond its bound"


@pytest.mark.parametrize("kind", ["token", "channel", "element"])
@pytest.mark.parametrize("T,H", [(11, 264), (2, 4104), (700, 512)])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
def test_open_and_closed_sigmoid_gates(gpu_lib, kind, T, H, gdt):
    norm, t, kw = make(T, H, h="f32", x="f32", w="f32", y="f32", post=True, kind=kind, act="sigmoid", gdt=gdt)
    gate = t["gate"]
    gate.copy_(torch.tensor(GATES, device="cuda").repeat(gate.numel() // len(GATES) + 1)[:gate.numel()].reshape(gate.shape))
    o = backward(norm, t, T, H)
    ref = plain(t, kw).backward(t["dh_out"], t["dx"])
    a = gate.double().abs().cpu()
    if gdt == "bf16" and kind == "element":  # a stored bf16 gradient: half a step more
        got, (value, mag) = o["dgate"].cpu().double(), ref["dgate"]
        half = 2.0 ** -8
        bad = (got - value).abs() - ((256 + 2 * a) * U * mag * (1 + half) + half * value.abs() + TINY)
        assert float(bad.max()) <= 0
    else:
        close("dgate", o["dgate"], ref["dgate"][0], (256 + 2 * a) * U * ref["dgate"][1])
    for n in set(o) - {"dgate"}:
        close(n, o[n], ref[n][0], (256 + 2 * 80) * U * ref[n][1])


def test_an_infinite_gate_has_no_slope(gpu_lib):
    norm, t, kw = make(3, 256, h="f32", x="f32", w="f32", post=True, kind="element", act="sigmoid", gdt="f32")
    t["gate"][0, 3], t["gate"][1, 5], t["gate"][2, 7] = float("inf"), -float("inf"), float("nan")
    o = backward(norm, t, 3, 256)
    assert float(o["dgate"][0, 3]) == 0.0 and float(o["dgate"][1, 5]) == 0.0 and bool(o["dgate"][2, 7].isnan())


@pytest.mark.parametrize("T,H,kind", [(6, 512, "none"), (6, 512, "token"), (6, 512, "element"), (6, 4104, "channel"),
                                      (700, 2048, "channel")])
@pytest.mark.parametrize("size", [1e25, 3e38])
def test_rows_beyond_the_range_of_their_squares(gpu_lib, T, H, kind, size):
    """Forward normalises such a row to zero, whatever it holds: a norm that is constant there sends
    nothing back, and the rows beside it keep their gradients."""
    norm, t, kw = make(T, H, h="f32", x="f32", w="f32", y="f32", post=True, kind=kind)
    t["h"][1] = size
    t["y"][3] = size
    t["dx"][1] = t["dx"][1].abs() + 1.0  # sums of one sign, which overflow too
    t["dh_out"][3] = t["dh_out"][3].abs() + 1.0
    t["h"][4] = size
    t["y"][4] = -size
    o = backward(norm, t, T, H)
    assert all(not v.isnan().any() for v in o.values())
    assert torch.equal(o["dh"][1], t["dh_out"][1]) and torch.equal(o["dh"][4], t["dh_out"][4])
    assert float(o["dy"][3].abs().max()) == 0.0 and float(o["dy"][4].abs().max()) == 0.0
    keep = [i for i in range(T) if i not in (1, 3, 4)]
    rest = {n: v if v is None or v.shape[:1] != (T,) else v[keep].contiguous() for n, v in t.items()}
    ref = NormCase(rest["h"], rest["y"], rest["gate"], rest["pre_w"], rest["post_w"], **kw).backward(rest["dh_out"], rest["dx"])
    for n in ("dh", "dy"):
        close(n, o[n][keep], ref[n][0], 256 * U * ref[n][1])
    # row 1 reaches the sums over rows through y, row 3 through h, row 4 not at all
    zero_h, zero_y = t["h"].double().cpu(), t["y"].double().cpu()
    zero_h[[1, 4]] = 0.0
    zero_y[[3, 4]] = 0.0
    dxs = t["dx"].clone()
    dxs[[1, 4]] = 0.0
    ref = NormCase(zero_h, zero_y, t["gate"], t["pre_w"], t["post_w"], **kw).backward(t["dh_out"], dxs)
    for n in ("dpre_w", "dpost_w") + (("dgate",) if kind == "channel" else ()):
        close(n, o[n], ref[n][0], 256 * U * ref[n][1])
