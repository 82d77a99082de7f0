"""int4 products in steps of two row tiles (2 to 8 tokens, matrices of many rows) whose columns are no
multiple of 256 or whose outputs are bf16, and matrices of few and many rows in between. Bounds as in
test_gpu_gemv.py."""

import pytest
import torch

from test_gpu_gemv import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2, 3, 5, 8])
@pytest.mark.parametrize("N,K", [(9001, 288), (9001, 1056), (9472, 32), (9003, 512), (14209, 480), (9001, 992)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_two_tiles_a_step(gpu_lib, N, K, T, out):
    w, s, x = make(N, K, T)
    y = run(w, s, x, out)
    check(w, s, x, y)
    assert torch.equal(y, run(w, s, x, out))


@pytest.mark.parametrize("T", [1, 13, 32])
@pytest.mark.parametrize("N,K", [(9001, 288), (9001, 992), (2500, 1056)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_one_tile_a_step_of_many_rows(gpu_lib, N, K, T, out):
    w, s, x = make(N, K, T)
    check(w, s, x, run(w, s, x, out))


@pytest.mark.parametrize("T", [1, 5, 13])
@pytest.mark.parametrize("power", [-100, 113])
def test_scales_at_both_ends(gpu_lib, T, power):
    """A group's sum is at most 4 in units of its row's largest x, so 2^114 over all of 2048 groups still
    fits, and the roundings of subnormal partial sums stay under the bound from 2^-100 on."""
    w, s, x = make(40, 512, T)
    s = torch.full_like(s, 2.0 ** power)
    s[::3, 1] = 0.0
    check(w, s, x, run(w, s, x))
    tiny = (x.float() * 2.0 ** -100).to(torch.bfloat16) if power > 0 else (x.float() * 2.0 ** 60).to(torch.bfloat16)
    check(w, s, tiny, run(w, s, tiny))
