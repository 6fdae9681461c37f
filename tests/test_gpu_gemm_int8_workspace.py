"""One workspace for products of a weight matrix with any number of rows up to the one that it was made for."""
import pytest

from test_gpu_gemm_int8 import exact, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,most", [(1024, 5120, 700), (1024, 5120, 2000), (5120, 4096, 600), (70, 17408, 40000)])
def test_fewer_rows_of_one_workspace(N, K, most):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(N)
    a = torch.randint(-128, 128, (most, K), generator=g, device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=dev, dtype=torch.int8)
    sa, sw = torch.rand(most, generator=g, device=dev), torch.rand(N, generator=g, device=dev)
    need = pn.gemm_int8_workspace_bytes(most, N, K)
    work = torch.full((need + 16,), 0xA5, dtype=torch.uint8, device=dev)
    for M in (most, 1, 33, 64, 100, 200, 256, 300, 498, 512, 640):
        if M > most:
            continue
        out = torch.zeros(M, N, device=dev)
        pn.gemm_int8(a[:M], sa[:M], w, sw, out, work[:need])
        torch.cuda.synchronize()
        for at in range(0, M, 4096):
            part = slice(at, min(M, at + 4096))
            within(torch, out[part], exact(torch, a[part], w), sa[part], sw, "float32")
        assert bool((work[need:] == 0xA5).all())
