"""The residual block refuses outputs that lie over its gate or its norms' weights (no GPU)."""

import ctypes as C

import pytest

import sparse_moe_gemv_b200 as smg
from test_around_host import INVALID, at, layer_struct, lib, norm_struct  # noqa: F401

PRE, POST, NEXT, GATE = at(60), at(61), at(62), at(63)
H2 = 2048 * 2


@pytest.mark.parametrize("kind,gate_bytes", [(1, 3 * 2), (2, H2), (3, 3 * H2)])
def test_outputs_over_the_gate_or_the_weights(lib, kind, gate_bytes):  # noqa: F811
    L = layer_struct()
    before = norm_struct(gate_kind=0, post_norm=0, post_w=None, pre_w=PRE)
    after = norm_struct(gate_kind=kind, pre_w=NEXT, post_w=POST)
    need = smg.load().redmoe_workspace_bytes_block(C.byref(L), 3)

    def blk(T=3, h_out=at(4), x_next=at(5), ids=at(6), w=at(7), ws=at(8)):
        return lib.redmoe_forward_block(C.byref(L), C.byref(before), C.byref(after), at(3), GATE, T, h_out, x_next, ids, w,
                                        ws, need, None)

    for start, size in ((PRE, H2), (POST, H2), (NEXT, H2), (GATE, gate_bytes)):
        first, last = start, (start + size - 1) // 4 * 4  # 4-byte outputs at both ends of the range
        for bad in (dict(ids=first), dict(ids=last), dict(w=first), dict(w=last), dict(ws=start),
                    dict(ws=start - (need - 256)),   # the workspace's last bytes
                    dict(ws=start - need // 512 * 256), dict(h_out=start), dict(x_next=start)):
            assert blk(**bad) == INVALID, (hex(start), bad)
