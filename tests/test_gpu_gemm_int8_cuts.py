"""Every kernel of the 8-bit products and every way of cutting them at the depths of a model's matrices, all outputs in all
types; each case says which it is for, so that a change of the rule that chooses shows."""
import ctypes as C

import pytest

from test_gpu_gemm_int8 import call, exact, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    yield pn, torch, torch.device("cuda:0")
    torch.cuda.empty_cache()


def cut(pn, M, N, K):
    parts = C.c_int()
    return pn.lib().pn_gemm_int8_cut(M, N, K, C.addressof(parts)), parts.value


def check(env, M, N, K, type_, seed):
    pn, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    a = torch.randint(-128, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=dev, dtype=torch.int8)
    sa = torch.exp(torch.randn(M, generator=g, device=dev)) / 128
    sw = torch.exp(torch.randn(N, generator=g, device=dev)) / 128 / K ** 0.5
    wide = torch.full((M, N + 3), 7.0, dtype=getattr(torch, type_), device=dev)
    out = wide[:, :N]
    call(pn, torch, a, sa, w, sw, out)
    torch.cuda.synchronize()
    for at in range(0, N, 4096):
        part = slice(at, at + 4096)
        within(torch, out[:, part], exact(torch, a, w[part]), sa, sw[part], type_)
    assert bool((wide[:, N:] == 7).all())


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,N,K,size,parts", [
    (64, 1024, 5120, 64, 4), (300, 1024, 17408, 64, 6), (200, 3000, 8016, 64, 2),    # parts in tiles of 64
    (777, 1024, 5120, 64, 1), (1000, 1300, 2064, 64, 1), (40, 34816, 5120, 64, 1),   # whole, one and two a CU
    (256, 5120, 5120, 128, 3), (250, 5100, 17408, 128, 3), (700, 1500, 5136, 128, 3),  # parts in tiles of 128
    (512, 5120, 5120, 128, 1), (1024, 5100, 5136, 128, 1), (96, 34816, 5120, 128, 1),  # whole
    (2048, 6144, 5120, 256, 1), (1500, 5123, 6144, 256, 1), (2049, 6145, 5136, 256, 1), (130, 34816, 5120, 256, 1)])
def test_tiles(env, type_, M, N, K, size, parts):
    assert cut(env[0], M, N, K) == (size, parts)
    check(env, M, N, K, type_, M)


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M", [1, 4, 8, 9, 13, 16, 17, 20, 32])
@pytest.mark.parametrize("N,K", [(34816, 5120), (26500, 5136), (5120, 17408)])
def test_streams(env, type_, M, N, K):
    """Weights of more than 128 MB, which pass the caches by, and fewer."""
    assert cut(env[0], M, N, K) == (0, 1)
    check(env, M, N, K, type_, M)


def test_cuts_that_are_refused(env):
    pn = env[0]
    assert pn.lib().pn_gemm_int8_cut(1, 1, 24, None) == -2 and pn.lib().pn_gemm_int8_cut(0, 1, 16, None) == -2
    assert pn.lib().pn_gemm_int8_cut(1, 1, 16, None) == 0
