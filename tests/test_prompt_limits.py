"""Limits of the prompt's entry points that are decided before anything runs: scales, sizes of launches, tensors that the
binding is given."""
import ctypes as C

import pytest
import torch  # first: the library takes its HIP runtime

import block_quantized_weight_pn3t_amd as pn
from test_prompt_reference import gemm, logp


@pytest.mark.parametrize("V,scale,refused", [
    (1, 2.0 ** -121, False), (1, 2.0 ** -122, True), (5000, 1.881e-33, False), (5000, 1.880e-33, True), (5000, 1e-37, True),
    ((1 << 30) - 1, 4.1e-28, False), ((1 << 30) - 1, 4.0e-28, True)])
def test_logprobs_scales(V, scale, refused):
    """From V * 2^-121 on no sum of a row's differences passes fp32."""
    assert (logp(V=V, stride=V, scale=scale, logits=0x1000, R=1, tokens=0x1002) == -2) == refused


@pytest.mark.parametrize("M,N,refused", [
    (64 * ((1 << 25) - 1), 1, True), (256 * ((1 << 23) - 1), 1, False), (1, 256 * ((1 << 23) - 1), False),
    (64 << 12, 64 << 13, True), (64 << 12, 64 * ((1 << 13) - 1), False)])
def test_gemm_int8_tiles(M, N, refused):
    """Outputs of which one launch has tiles of 256 for all."""
    assert (gemm(M=M, N=N, K=16, a=C.c_void_p(0x1008)) == -2) == refused
