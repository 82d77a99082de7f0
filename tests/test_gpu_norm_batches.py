"""The forms of the step between blocks that long batches run: two chunks of a row a thread with several
rows a block, and gradients whose groups walk rows while the column sums build up.

On 148 multiprocessors a row of more than 32 chunks of eight columns takes two chunks a thread from
T ceil(chunks / 32) > 4736 on, and the gradients' grid holds 296 blocks of 256 threads (148 of more): the
sizes below have four rows or more for every group.

Tolerances: as in test_gpu_norm.py up to the column sums, 180 U of a gradient's magnitude at most: a row
sum is 16 products of a thread, 5 shuffle steps and 16 warps deep (30 U), r2 and r2^2 s1 / H follow
(70 U), the terms of G and their product with y r1 (40 more) and 40 for the sums of the branch. A column
sum adds up to 5 rows of a group, 8 groups, then 10 blocks of a slice and 32 slices: 55 U. Under 256 U.
"""

import pytest
import torch

import sparse_moe_gemv_b200 as smg
from plain_ops import U
from test_gpu_norm import backward, close, forward, make, plain

pytestmark = pytest.mark.gpu

CASES = [
    dict(T=2500, H=2048, y="bf16", post=True, kind="channel", act="sigmoid"),       # 256 chunks: all of both in use
    dict(T=2500, H=2048, h="f32", y="f32", x="f32", w="f32", post=True, kind="token", gdt="f32"),
    dict(T=2499, H=2056, post=True, kind="element", res=0.9, block=0.5),            # 257 chunks: the second partial
    dict(T=5001, H=520, y="bf16", post=True, kind="channel", offset=1.0),           # 65 chunks, four rows a block
    dict(T=10007, H=264, h="f32", x="f32", post=True, kind="token", act="sigmoid"),  # 33 chunks, eight rows a block
    dict(T=3001, H=1000, kind="element", gdt="f32"),
    dict(T=1301, H=4096, post=True, kind="channel"),                                # the layer's fp32 y: no row ahead
    dict(T=1301, H=4096, h="f32", y="f32", x="f32", w="f32", post=True, kind="element", gdt="f32"),
    dict(T=1300, H=3592, h="f32", y="f32", x="f32", w="f32", post=True, kind="element", gdt="f32", act="sigmoid"),
    dict(T=700, H=8192, y="bf16", post=True, kind="channel"),                       # one block of 512 threads
    dict(T=20011, H=256, post=True, kind="channel"),                                # one chunk a thread, eight rows
    dict(T=2503, H=2048, branch=False, h="f32", x="f32", w="f32"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_forward_of_long_batches(gpu_lib, case):
    norm, t, kw = make(**case)
    ho, x = forward(norm, t)
    vh, vx, mh, mx = plain(t, kw).forward()
    if t["y"] is not None:
        close("h_out", ho, vh, 64 * U * mh)
    close("x", x, vx, 64 * U * mx)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_gradients_of_long_batches(gpu_lib, case):
    norm, t, kw = make(**case)
    o = backward(norm, t, case["T"], case["H"])
    ref = plain(t, kw).backward(t["dh_out"], t["dx"])
    for n in o:
        close(n, o[n], ref[n][0], 256 * U * ref[n][1])


@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[7]], ids=lambda c: "-".join(str(v) for v in c.values()))
def test_gradients_of_long_batches_in_place(gpu_lib, case):
    norm, t, _ = make(**case)
    T, H = case["T"], case["H"]
    want = backward(norm, t, T, H)
    o = {n: torch.empty_like(v) for n, v in want.items()}
    dh = t["dh_out"].clone()
    smg.redmoe_norm_backward(norm, t["h"], dh, smg.new_norm_workspace(norm, T), dh_out=dh, dx=t["dx"], y=t["y"],
                             gate=t["gate"], dy=o["dy"], dgate=o["dgate"], dpost_w=o["dpost_w"], dpre_w=o["dpre_w"])
    o["dh"] = dh
    torch.cuda.synchronize()
    assert all(torch.equal(o[n], want[n]) for n in want)


def test_a_row_of_a_long_batch_is_that_row_alone_up_to_rounding(gpu_lib):
    """Another number of rows may mean another order of a row's sums: equal within both calls' bounds."""
    norm, t, kw = make(2500, 2048, post=True, kind="channel")
    ho, x = forward(norm, t)
    few = {n: v if v is None or v.shape[0] != 2500 else v[:3].contiguous() for n, v in t.items()}
    ho3, x3 = forward(norm, few)
    vh, vx, mh, mx = plain(few, kw).forward()
    for got in (ho[:3], ho3):
        close("h_out", got, vh, 64 * U * mh)
    for got in (x[:3], x3):
        close("x", got, vx, 64 * U * mx)
