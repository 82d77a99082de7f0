"""The binding refuses tensors of another rank than its calls take with a ValueError, scalars included."""

import pytest
import torch

import sparse_moe_gemv_b200 as smg
from test_gpu_block import QWEN, setup
from test_gpu_gemv import make as gemv_make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(), (256,), (1, 4, 256)])
def test_norms(gpu_lib, shape):
    norm = smg.Norm(256, h_dtype="f32", x_dtype="f32")
    t = torch.zeros(shape, device="cuda")
    with pytest.raises(ValueError):
        smg.redmoe_norm_forward(norm, t, x=torch.empty_like(t))
    with pytest.raises(ValueError):
        smg.redmoe_norm_backward(norm, t, torch.empty_like(t), None, dx=torch.empty_like(t))


@pytest.mark.parametrize("shape", [(), (128,), (1, 2, 128)])
def test_products(gpu_lib, shape):
    w, s, _ = gemv_make(64, 128, 1)
    x = torch.zeros(shape, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        smg.redmoe_gemv(smg.Matrix(w, s, 64, 128), x, torch.empty(1, 64, device="cuda"))


@pytest.mark.parametrize("shape", [(), (16,), (1, 4, 16)])
def test_balance(gpu_lib, shape):
    t = torch.zeros(shape, device="cuda")
    f, i = torch.empty(16, device="cuda"), torch.empty(16, device="cuda", dtype=torch.int32)
    n = torch.empty(1, device="cuda", dtype=torch.int32)
    ws = smg.new_balance_workspace(4, 16)
    ids = torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError):
        smg.redmoe_balance_forward(t, ids, f[:2], i, f, n, ws)
    with pytest.raises(ValueError):
        smg.redmoe_balance_forward(torch.zeros(4, 16, device="cuda"), torch.zeros(shape, device="cuda", dtype=torch.int32),
                                   f[:2].clone(), i, f, n, ws)
    with pytest.raises(ValueError):
        smg.redmoe_balance_backward(t, i, n, f[:2], torch.empty_like(t), 2)


@pytest.mark.parametrize("shape", [(), (2048,), (1, 1, 2048)])
def test_block(gpu_lib, shape):
    L, before, after, h, _ = setup(QWEN, 1, 3, False, "none")
    lay = smg.Layer.from_shape(L, QWEN)
    ids, w = torch.empty(1, QWEN.k, device="cuda", dtype=torch.int32), torch.empty(1, QWEN.k, device="cuda")
    bad = torch.zeros(shape, device="cuda", dtype=h.dtype)
    with pytest.raises(ValueError):
        smg.redmoe_forward_block(lay, before, after, bad, torch.empty_like(bad), ids, w, smg.new_workspace_block(lay, 1))
