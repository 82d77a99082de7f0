"""Balance statistics and gradients of long batches: several live rows for every warp, so that ring slots,
mask words and column sums are used again, and blocks of 24 warps (more than 2368 rows of 129 to 512
columns on 148 multiprocessors). A step of the grid is 9472 rows up to 128 columns, 3552 rows with 24
warps and 2368 with 16; a warp looks its mask bytes up for 32 steps at a time (8, up to 128 columns).

Tolerances: counts and rows are exact. A probability is under 64 U off (test_gpu_balance.py); its mean
adds the R = ceil(T / step) rows of a lane, two shuffles, up to 24 warps and up to 160 blocks in a
fixed order: R + 192 more. The z loss adds the same way, from lse^2. The gradient is one row: 128 U.
"""

import pytest
import torch

import sparse_moe_gemv_b200 as smg
from plain_ops import U, balance_backward, balance_forward, store_tol
from test_gpu_balance import make, run

pytestmark = pytest.mark.gpu

GRAD = (0.5, 0.25)
SIZES = [
    (20011, 512, 10, "f32", 0.2), (30001, 512, 10, "bf16", 0.2), (20003, 501, 4, "f32", 0.1), (20003, 501, 4, "bf16", 0.0),
    (20000, 256, 8, "bf16", 0.0), (20000, 256, 8, "f32", 0.3), (130003, 129, 3, "bf16", 0.1), (130003, 132, 3, "f32", 0.0),
    (12007, 1023, 7, "f32", 0.2), (12007, 1023, 7, "bf16", 0.1), (12000, 1024, 16, "bf16", 0.0), (2369, 512, 10, "f32", 0.0),
    (160003, 61, 4, "f32", 0.2), (160003, 61, 4, "bf16", 0.0), (170000, 64, 6, "bf16", 0.3), (80000, 128, 8, "f32", 0.1),
    (160001, 20, 2, "f32", 0.1), (100001, 1, 1, "bf16", 0.5),
]


def step(T, E):
    return 9472 if E <= 128 else 3552 if E <= 512 and T > 2368 else 2368


@pytest.mark.parametrize("T,E,k,dtype,masked", SIZES)
def test_long_batches(gpu_lib, T, E, k, dtype, masked):
    logits, ids, mask = make(T, E, k, dtype, masked)
    got = run(logits, ids, mask, GRAD)
    loss, counts, prob, n, dl = (v.cpu() for v in got)
    rl, rc, rp, rn, mag = balance_forward(logits, ids, mask)
    assert int(n) == rn and torch.equal(counts, rc)
    deep = (64 + -(-T // step(T, E)) + 192) * U
    assert bool(((prob.double() - rp).abs() <= store_tol(rp, deep * rp, torch.float32)).all())
    assert bool(((loss.double() - rl).abs() <= store_tol(rl, deep * mag, torch.float32)).all())
    rd, md = balance_backward(logits, counts, rn, k, GRAD, mask)
    bad = (dl.double() - rd).abs() - store_tol(rd, 128 * U * md, dl.dtype)
    assert not dl.isnan().any() and float(bad.max()) <= 0
    # over the logits themselves, and once more
    buf = logits.clone()
    smg.redmoe_balance_backward(buf, got[1], got[3], torch.tensor(GRAD, device="cuda"), buf, k, mask=mask)
    assert torch.equal(buf, got[4])
    again = run(logits, ids, mask, GRAD)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("E,dtype", [(512, "f32"), (501, "bf16"), (61, "f32"), (64, "bf16")])
def test_runs_of_masked_rows_between_live_ones(gpu_lib, E, dtype):
    """Whole steps of a warp are skipped, and the rows that count come back at any place of its mask words."""
    T, k = 4 * step(10 ** 6, E) * 5 + 37, 3
    logits, ids, _ = make(T, E, k, dtype, seed=2)
    s = step(T, E)
    mask = ((torch.arange(T, device="cuda") // s) % 3 == 1) | (torch.arange(T, device="cuda") % 41 == 5)
    logits[~mask] = float("nan")
    loss, counts, prob, n, dl = (v.cpu() for v in run(logits, ids, mask, GRAD))
    rl, rc, rp, rn, mag = balance_forward(logits, ids, mask)
    deep = (64 + -(-T // s) + 192) * U
    assert int(n) == rn and torch.equal(counts, rc)
    assert bool(((prob.double() - rp).abs() <= store_tol(rp, deep * rp, torch.float32)).all())
    assert bool(((loss.double() - rl).abs() <= store_tol(rl, deep * mag, torch.float32)).all())
    rd, md = balance_backward(logits, counts, rn, k, GRAD, mask)
    bad = (dl.double() - rd).abs() - store_tol(rd, 128 * U * md, dl.dtype)
    assert not dl.isnan().any() and float(bad.max()) <= 0


@pytest.mark.parametrize("T,E,dtype", [(2000003, 20, "f32"), (700001, 130, "bf16")])
def test_sums_over_many_equal_rows(gpu_lib, T, E, dtype):
    """Equal rows round their sums in one direction: the bound of (256 + T / R) U still holds."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    row = torch.randn(1, E, generator=g, device="cuda").to(smg.TORCH_DTYPES[dtype])
    logits, ids = row.expand(T, E).contiguous(), torch.full((T, 1), 3, device="cuda", dtype=torch.int32)
    loss, counts, prob, n, _ = (v.cpu() for v in run(logits, ids, None, GRAD))
    rl, _, rp, _, mag = balance_forward(row, ids[:1])
    bound = (256 + T / (9472 if E <= 128 else 2368)) * U
    assert int(n) == T and int(counts[3]) == T and int(counts.sum()) == T
    assert bool(((prob.double() - rp).abs() <= store_tol(rp, bound * rp, torch.float32)).all())
    assert bool(((loss.double() - rl).abs() <= store_tol(rl, bound * mag, torch.float32)).all())
