"""Validation and decoding of more rows than one launch takes (2^32 threads)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    torch.cuda.empty_cache()
    yield pn, torch, torch.device("cuda:0")
    torch.cuda.empty_cache()


def test_fp8row_decode(env):
    """A head of 248,320 x 17,408, every number."""
    pn, torch, dev = env
    N, K = 248320, 17408
    codes = torch.randint(0, 256, (N, K), dtype=torch.uint8, device=dev)
    codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.rand(N, device=dev).bfloat16()
    out = torch.full((N, K), 3.0, device=dev)
    pn.fp8row_dequantize_rows(codes, scales.view(torch.int16), N, K, out)
    torch.cuda.synchronize()
    for at in range(0, N, 20000):
        part = slice(at, at + 20000)
        assert torch.equal(out[part], codes[part].view(torch.float8_e4m3fn).float() * scales[part, None].float())


def test_nvfp4_decode(env):
    """The rows behind the first launch's against a call of their own."""
    pn, torch, dev = env
    N, K = (1 << 33) // 16384 + 100, 16384
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.randint(0, 0x7F, (N, K // 16), dtype=torch.uint8, device=dev)
    out, again = torch.full((N, K), 3.0, device=dev), torch.zeros(200, K, device=dev)
    pn.nvfp4_dequantize_rows(codes, scales, 0.5, N, K, out)
    for at in (0, N // 2, N - 300, N - 200):
        pn.nvfp4_dequantize_rows(codes[at:at + 200], scales[at:at + 200], 0.5, 200, K, again)
        torch.cuda.synchronize()
        assert torch.equal(out[at:at + 200], again)


def test_pn_decode(env):
    pn, torch, dev = env
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 155 GB")
    nb = 256
    N, K = (1 << 32) // (8 * nb) + 100, 64 * nb
    W = torch.zeros(N, 34 * nb, dtype=torch.uint8, device=dev)  # 18 GB
    tail = torch.randint(0, 256, (300, 34 * nb), dtype=torch.uint8, device=dev)
    tail.view(300, nb, 34)[:, :, 1] &= 0x3F  # scales that are finite
    W[-300:], W[:300] = tail, tail
    out, again = torch.empty(N, K, device=dev), torch.zeros(300, K, device=dev)  # 137 GB
    out[-300:] = 3.0
    pn.dequantize_rows(pn.PN4T, W, N, K, out)
    pn.dequantize_rows(pn.PN4T, tail, 300, K, again)
    torch.cuda.synchronize()
    assert torch.equal(out[:300], again) and torch.equal(out[-300:], again)


def test_validation(env):
    pn, torch, dev = env
    N = (1 << 26) + 5
    wrong = torch.tensor([0, 1, 77, (1 << 26) - 4, (1 << 26) - 3, 1 << 26, N - 1], device=dev)
    want = torch.ones(N, dtype=torch.int32, device=dev)
    want[wrong] = 0
    verdict = torch.full_like(want, 7)
    for type_, K in ((pn.PN4T, 64), (pn.PN3T, 80)):
        W = torch.zeros(N, 34, dtype=torch.uint8, device=dev)
        W[wrong, 1] = 0x7C  # an infinite scale
        verdict.fill_(7)
        pn.validate_rows(type_, W, N, K, verdict)
        torch.cuda.synchronize()
        assert torch.equal(verdict, want)
    del W
    scales = torch.full((N, 1), 0x38, dtype=torch.uint8, device=dev)
    scales[wrong] = 0x7F
    verdict.fill_(7)
    pn.nvfp4_validate_rows(scales, 1.0, N, 16, verdict)
    torch.cuda.synchronize()
    assert torch.equal(verdict, want)
    codes, multipliers = torch.zeros(N, 16, dtype=torch.uint8, device=dev), torch.ones(N, dtype=torch.bfloat16, device=dev)
    codes[wrong, 15] = 0xFF
    verdict.fill_(7)
    pn.fp8row_validate_rows(codes, multipliers.view(torch.int16), N, 16, verdict)
    torch.cuda.synchronize()
    assert torch.equal(verdict, want)
