"""The norm and the 8-bit rows at the widths of a model's hidden state and at prompts' numbers of rows, from which on a
thread holds two pieces of 16-bit rows; every code and sum."""
import numpy as np
import pytest

import prompt_reference as ref
from test_gpu_norm import check, near, numbers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


@pytest.mark.parametrize("K", [4104, 5119, 5120, 8191, 8192])
@pytest.mark.parametrize("rows", [255, 256, 257, 300])
@pytest.mark.parametrize("type_,wtype,residual", [("bfloat16", "bfloat16", True), ("bfloat16", "float32", False),
                                                  ("float16", "float16", False), ("float16", "float32", True)])
def test_norm(env, type_, wtype, residual, rows, K):
    check(env, rows, K, type_, wtype, residual, K % 2 == 1 or rows == 256, True, rows + K)


@pytest.mark.parametrize("K", [4104, 5119, 5120, 8191, 8192, 8200, 17408])
@pytest.mark.parametrize("rows", [256, 300])
@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
def test_quantize_rows(env, type_, rows, K):
    pn, torch, dev = env
    x = numbers(torch, np.random.default_rng(rows + K), (rows, K), getattr(torch, type_))
    x[1, K // 3] = float("nan")
    x[rows - 1, K - 1] = float("inf")
    codes = torch.full((rows, K), 55, dtype=torch.int8, device=dev)
    scales = torch.full((rows,), 55.0, device=dev)
    pn.int8_quantize_rows(x.to(dev), codes, scales)
    torch.cuda.synchronize()
    want, want_scales = ref.int8_rows(x.double().numpy())
    assert (codes.cpu().numpy() == want).all()
    near(scales, want_scales, "float32")
