"""The prompt's operators in calls that overlap, on another device than the current one, and at cuts of their work that
other tests do not reach."""
import numpy as np
import pytest

import prompt_reference as ref
from test_gpu_gemm_int8 import exact, within
from test_gpu_logprobs import call as logprobs_call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


@pytest.mark.parametrize("M,N,K", [(2, 262145, 32), (20, 300001, 16), (9, 257, 144)])
def test_stream_of_many_rows(env, M, N, K):
    """More rows than a workgroup a CU holds scales of, and shares of one row or two."""
    pn, torch, dev = env
    a = torch.randint(-128, 128, (M, K), device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), device=dev, dtype=torch.int8)
    sa, sw = torch.rand(M, device=dev), torch.rand(N, device=dev)
    out = torch.zeros(M, N, device=dev)
    pn.gemm_int8(a, sa, w, sw, out)
    torch.cuda.synchronize()
    within(torch, out, exact(torch, a, w), sa, sw, "float32")


@pytest.mark.parametrize("M", [33, 64, 65, 128, 200, 257])
@pytest.mark.parametrize("K", [1552, 4112, 17424, 20000])
def test_parts_that_end_inside_a_line(env, M, K):
    pn, torch, dev = env
    N = 100
    a = torch.randint(-128, 128, (M, K), device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), device=dev, dtype=torch.int8)
    sa, sw = torch.rand(M, device=dev), torch.rand(N, device=dev)
    for fill in (0, 255):
        out = torch.zeros(M, N, device=dev)
        work = torch.full((pn.gemm_int8_workspace_bytes(M, N, K) + 16,), fill, dtype=torch.uint8, device=dev)
        pn.gemm_int8(a, sa, w, sw, out, work)
        torch.cuda.synchronize()
        within(torch, out, exact(torch, a, w), sa, sw, "float32")


def test_the_same_product_however_cut(env):
    """A token's outputs are the same bits among any number of tokens."""
    pn, torch, dev = env
    N, K = 515, 5136
    a = torch.randint(-128, 128, (1500, K), device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), device=dev, dtype=torch.int8)
    sa, sw = torch.rand(1500, device=dev), torch.rand(N, device=dev)

    def product(M):
        out = torch.zeros(M, N, device=dev)
        work = torch.zeros(pn.gemm_int8_workspace_bytes(M, N, K) + 16, dtype=torch.uint8, device=dev)
        pn.gemm_int8(a[:M], sa[:M], w, sw, out, work)
        torch.cuda.synchronize()
        return out
    full = product(1500)
    for M in (1, 8, 9, 16, 17, 32, 33, 64, 130, 300, 900):
        assert torch.equal(product(M), full[:M]), M


def test_two_streams_at_once(env):
    """Each operator on two streams without a wait between, each call with a workspace of its own."""
    pn, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    sizes = [(64, 1024, 5120), (3, 5000, 4096), (300, 600, 2048)]
    products = []
    for M, N, K in sizes:
        for _ in range(2):
            a = torch.randint(-128, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
            w = torch.randint(-128, 128, (N, K), generator=g, device=dev, dtype=torch.int8)
            work = torch.zeros(pn.gemm_int8_workspace_bytes(M, N, K) + 16, dtype=torch.uint8, device=dev)
            products.append((a, torch.rand(M, device=dev), w, torch.rand(N, device=dev), torch.zeros(M, N, device=dev), work))
    rows = [3 * torch.randn(5, 100003, generator=g, device=dev) for _ in range(2)]
    tokens = torch.zeros(5, dtype=torch.int32, device=dev)
    want = [logprobs_call(pn, torch, x, tokens, 1.0, 20) for x in rows]
    x = torch.randn(100, 2048, generator=g, device=dev).bfloat16()
    norm = torch.ones(2048, device=dev)
    normed = torch.empty_like(x)
    pn.add_norm(x, norm, 1e-6, out=normed)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        got, outs = [], []
        for p in products:
            p[4].zero_()
        torch.cuda.synchronize()
        for i in range(len(sizes)):
            for n, s in enumerate(streams):
                with torch.cuda.stream(s):
                    pn.gemm_int8(*products[2 * i + n])
                    got.append((n, logprobs_call(pn, torch, rows[n], tokens, 1.0, 20, fill=rep)))
                    outs.append(torch.empty_like(x))
                    pn.add_norm(x, norm, 1e-6, out=outs[-1])
        torch.cuda.synchronize()
        for a, sa, w, sw, out, _ in products:
            within(torch, out, exact(torch, a, w), sa, sw, "float32")
        for n, each in got:
            for name in each:
                assert torch.equal(each[name], want[n][name]), name
        for out in outs:
            assert torch.equal(out, normed)


def test_tensors_of_another_device(env, monkeypatch):
    """With another device current, the call is refused and nothing runs."""
    pn, torch, dev = env
    x, w = torch.zeros(4, 64, device=dev), torch.ones(64, device=dev)
    codes, scales = torch.zeros(4, 64, dtype=torch.int8, device=dev), torch.ones(4, device=dev)
    cache = pn.Cache(pn.MXFP8, 1, 64, 32, torch.zeros(pn.cache_page_bytes(pn.MXFP8, 1, 64, 32), dtype=torch.uint8, device=dev))
    k, slots = torch.zeros(4, 1, 64, device=dev), torch.arange(4, device=dev)
    calls = (lambda: pn.add_norm(x, w, 1e-6, out=x), lambda: pn.int8_quantize_rows(x, codes, scales),
             lambda: pn.gemm_int8(codes, scales, codes, scales, torch.zeros(4, 4, device=dev)),
             lambda: pn.cache_append(cache, k, k, slots, torch.zeros(4, 64, device=dev)),
             lambda: pn.logprobs(x, entropy=scales, workspace=torch.zeros(4096, dtype=torch.uint8, device=dev)))
    for call in calls:
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(pn._Torch, "device", staticmethod(lambda: 1))
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_norms_that_pass_fp32(env):
    """Rows whose products leave fp32's range or fall below it, from 16-bit numbers, beside ordinary ones."""
    pn, torch, dev = env
    K = 1600
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(size=(6, K)).astype(np.float32)).bfloat16()
    w = torch.from_numpy(rng.normal(size=K).astype(np.float32)).bfloat16()
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3, ::2] *= 1e38
    for scale in (1.0, 1e30, 1e-30):
        weight = (w.float() * scale).bfloat16()
        codes, scales = torch.full((6, K), 9, dtype=torch.int8, device=dev), torch.empty(6, device=dev)
        pn.add_norm(x.to(dev), weight.to(dev), 0.0, codes=codes, scales=scales)
        torch.cuda.synchronize()
        _, t, r = ref.norm(x.double().numpy(), weight.double().numpy(), 0.0)
        want, want_scales = ref.int8_rows(t, r)
        assert (codes.cpu().numpy() == want).all()
        got = scales.double().cpu().numpy()
        bad = np.isnan(want_scales)  # a row with an infinity
        assert (np.isnan(got) == bad).all()
        err = np.abs(got - want_scales)
        assert (err <= 2.0 ** -24 * want_scales * (1 + 1e-6) + 2.0 ** -150)[~bad].all()


@pytest.mark.parametrize("V", [40003, 248320])
@pytest.mark.parametrize("R", [1, 2, 255, 256])
def test_rows_beside_the_change_of_workgroups(env, R, V):
    """The same bits of a row in calls of few rows and of many need not be; the same tokens must."""
    pn, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(R)
    x = (3 * torch.randn(R, V, generator=g, device=dev)).bfloat16()  # many ties
    tokens = torch.randint(0, V, (R,), generator=g, device=dev, dtype=torch.int32)
    got = logprobs_call(pn, torch, x, tokens, 1.0, 64)
    f = x.float()
    assert torch.equal(got["rank"].long(), (f > f.gather(1, tokens.long()[:, None])).sum(1))
    bits = f.view(torch.int32)
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits).long() << 32
    key -= torch.arange(V, device=dev)
    assert torch.equal(got["top_ids"].long(), torch.topk(key, 64, -1)[1])
    lse = torch.logsumexp(f.double(), 1)
    assert bool(((got["lse"].double() - lse).abs() <= 1e-5).all())
