"""More rows than one launch takes (2^32 threads)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    yield pn, torch, torch.device("cuda:0")
    torch.cuda.empty_cache()


def codes_of(torch, t):
    """Codes and T of the 8-bit rows of t (64 bits)."""
    top = t.abs().amax(-1, keepdim=True)
    return torch.round(127.0 * t / torch.where(top > 0, top, 1.0)).to(torch.int8), top[:, 0]


def test_norm_of_narrow_rows(env):
    """A wave a row: every output of every row."""
    pn, torch, dev = env
    rows, K = (1 << 26) + 5, 8
    x = torch.randn(rows, K, dtype=torch.bfloat16, device=dev)
    residual = torch.randn(rows, K, dtype=torch.bfloat16, device=dev)
    weight = torch.randn(K, device=dev).bfloat16()
    total, out = torch.zeros_like(x), torch.zeros_like(x)
    codes, scales = torch.zeros(rows, K, dtype=torch.int8, device=dev), torch.zeros(rows, device=dev)
    pn.add_norm(x, weight, 1e-6, out=out, codes=codes, scales=scales, residual=residual, sum=total)
    torch.cuda.synchronize()
    for at in range(0, rows, 1 << 23):
        part = slice(at, at + (1 << 23))
        h = x[part] + residual[part]
        assert torch.equal(total[part], h)
        t = h.double() * weight.double()
        r = 1.0 / torch.sqrt(h.double().square().mean(-1) + float(torch.tensor(1e-6)))
        want, top = codes_of(torch, t)
        assert torch.equal(codes[part], want)
        # one rounding of what 64 bits give to fp32, and to bf16
        s, y = top * r / 127.0, t * r[:, None]
        assert bool(((scales[part].double() - s).abs() <= 2.0 ** -24 * 1.000001 * s).all())
        assert bool(((out[part].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -23) * y.abs()).all())


def test_rows_of_a_workgroup_each(env):
    """Rows that overlap in memory, each of 192 threads."""
    pn, torch, dev = env
    rows, K = (1 << 32) // 192 + 7, 1032
    base = torch.randn(rows + K - 1, device=dev).bfloat16()
    x = base.as_strided((rows, K), (1, 1))
    codes, scales = torch.zeros(rows, K, dtype=torch.int8, device=dev), torch.zeros(rows, device=dev)  # 23 GB
    pn.int8_quantize_rows(x, codes, scales)
    torch.cuda.synchronize()
    top = torch.nn.functional.max_pool1d(base.float().abs()[None, None], K, 1)[0, 0]
    assert torch.equal(scales, (top.double() / 127.0).float())
    for at in (0, rows // 2, (1 << 32) // 192 - 2000, rows - 4000):
        assert torch.equal(codes[at:at + 4000], codes_of(torch, x[at:at + 4000].double())[0])


def test_logprobs_of_many_rows(env):
    pn, torch, dev = env
    R, V, top = (1 << 24) + 5, 3, 2
    x = torch.randn(R, V, device=dev)
    tokens = torch.randint(0, V, (R,), dtype=torch.int32, device=dev)
    got = dict(logprob=torch.zeros(R, device=dev), rank=torch.full((R,), 9, dtype=torch.int32, device=dev),
               entropy=torch.zeros(R, device=dev), lse=torch.zeros(R, device=dev),
               top_ids=torch.full((R, top), 9, dtype=torch.int32, device=dev), top_logprobs=torch.zeros(R, top, device=dev))
    work = torch.empty(pn.logprobs_workspace_bytes(R, V, top), dtype=torch.uint8, device=dev)
    pn.logprobs(x, tokens, workspace=work, **got)
    torch.cuda.synchronize()
    at = tokens.long()[:, None]
    assert torch.equal(got["rank"], (x > x.gather(1, at)).sum(-1).int())
    order = torch.sort(x, stable=True, dim=-1, descending=True)[1][:, :top]
    assert torch.equal(got["top_ids"].long(), order)
    p = torch.log_softmax(x.double(), -1)
    # each of a few roundings of numbers of up to some 15
    for name, want in (("logprob", p.gather(1, at)[:, 0]), ("entropy", -(p.exp() * p).sum(-1)),
                       ("lse", torch.logsumexp(x.double(), -1)), ("top_logprobs", p.gather(1, order))):
        assert float((got[name].double() - want).abs().max()) <= 2.0 ** -24 * 400, name


def test_product_of_many_rows(env):
    """More tiles of 64 than one launch takes."""
    pn, torch, dev = env
    M, N, K = (1 << 30) + 3, 2, 16
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device=dev)  # 17 GB
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=dev)
    sa, sw = torch.rand(M, device=dev), torch.rand(N, device=dev)
    out = torch.full((M, N), 7.0, device=dev)
    work = torch.empty(pn.gemm_int8_workspace_bytes(M, N, K), dtype=torch.uint8, device=dev)
    pn.gemm_int8(a, sa, w, sw, out, work)
    torch.cuda.synchronize()
    for at in range(0, M, 1 << 26):
        part = slice(at, at + (1 << 26))
        sums = torch.matmul(a[part].float(), w.float().t())  # whole numbers below 2^24
        assert torch.equal(out[part], sums * sa[part, None] * sw)


def test_nvfp4_rows_that_no_launch_takes(env):
    """One token that is not 16-byte aligned: a workgroup for eight rows, 2^24 of them."""
    pn, torch, dev = env
    N, K = 1 << 27, 16
    codes, scales = torch.zeros(N, K // 2, dtype=torch.uint8, device=dev), torch.zeros(N, 1, dtype=torch.uint8, device=dev)
    x, y = torch.zeros(K + 1, dtype=torch.bfloat16, device=dev)[1:], torch.zeros(1, N, device=dev)
    call = pn.lib().pn_gemv_nvfp4
    args = lambda n: (codes.data_ptr(), scales.data_ptr(), 1.0, n, K, x.data_ptr(), 1, y.data_ptr(), None)  # noqa: E731
    torch.cuda.synchronize()
    assert call(*args(N)) == -2 and call(*args(N - 8)) == 0
    torch.cuda.synchronize()
