"""Products of 8-bit integers on the GPU against exact sums: three fp32 roundings and the type's."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 2.0 ** -150, "bfloat16": 2.0 ** -134, "float16": 2.0 ** -25}


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


def exact(torch, a, w):
    """The sums in 64 bits: a product in double precision is exact below 2^53."""
    return torch.matmul(a.double(), w.double().t())


def call(pn, torch, a, sa, w, sw, out, fill=0xA5):
    need = pn.gemm_int8_workspace_bytes(a.shape[0], w.shape[0], a.shape[1])
    work = torch.full((need + 16,), fill, dtype=torch.uint8, device=a.device)
    pn.gemm_int8(a, sa, w, sw, out, work)
    return work


def within(torch, out, sums, sa, sw, type_):
    want = sums * sa.double()[:, None] * sw.double()
    most = want.abs() * ((1 + 3 * 2.0 ** -24) * (1 + HALF[type_]) - 1 + 2.0 ** -46) + TINY[type_] + 2.0 ** -148
    err = (out.double() - want).abs()
    assert bool((err <= most).all()), float((err - most).max())


def check(env, M, N, K, type_, seed, full=False, stride=None):
    pn, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    a = torch.randint(-128, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=dev, dtype=torch.int8)
    if full:  # the largest sums, of either sign
        a[:], w[:] = -128, -128
        w[::2] = 127
    sa = torch.exp(torch.randn(M, generator=g, device=dev)) / 128
    sw = torch.exp(torch.randn(N, generator=g, device=dev)) / 128 / K ** 0.5
    wide = torch.full((M, stride or N), 7.0, dtype=getattr(torch, type_), device=dev)
    out = wide[:, :N]
    call(pn, torch, a, sa, w, sw, out)
    torch.cuda.synchronize()
    within(torch, out, exact(torch, a, w), sa, sw, type_)
    assert bool((wide[:, N:] == 7).all())


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 13, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 600])
@pytest.mark.parametrize("N,K", [(1, 16), (17, 48), (64, 64), (100, 272), (259, 1040)])
def test_sizes(env, M, N, K):
    check(env, M, N, K, "float32", M * 1000 + N)


@pytest.mark.parametrize("K", [16, 32, 112, 128, 144, 240, 256, 272, 496, 512, 528, 1008, 1024, 1040, 2064, 4096, 5120, 17408])
@pytest.mark.parametrize("M,N", [(1, 70), (16, 33), (70, 130), (300, 530)])
def test_depths(env, M, N, K):
    check(env, M, N, K, "float32", K)


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,N,K", [(1, 1024, 5120), (4, 5120, 6144), (13, 5120, 17408), (40, 1024, 5120), (777, 1024, 5120),
                                   (515, 2050, 1296), (1000, 6144, 640)])
def test_types(env, type_, M, N, K):
    check(env, M, N, K, type_, 3)


@pytest.mark.parametrize("K", [16, 96, 128, 144, 256, 272, 400, 528])
@pytest.mark.parametrize("M,N,type_", [(1030, 10245, "bfloat16"), (600, 17410, "float32"), (3001, 5123, "float16")])
def test_many_outputs_of_few_products(env, M, N, K, type_):
    check(env, M, N, K, type_, K)


@pytest.mark.parametrize("M", [1, 16, 40, 130, 400])
@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
def test_rows_of_a_wider_output(env, M, type_):
    check(env, M, 70, 320, type_, 4, stride=103)
    check(env, M, 256, 320, type_, 5, stride=512)


@pytest.mark.parametrize("M", [1, 5, 16, 33, 128, 300])
@pytest.mark.parametrize("K", [17408, 131056])
def test_largest_sums(env, M, K):
    check(env, M, 40, K, "float32", 6, full=True)


def test_sums_are_exact(env):
    """Scales of one and sums below 2^24: whole numbers, equal; one row of each side differs per output."""
    pn, torch, dev = env
    for M, N, K in ((1, 300, 1040), (16, 300, 1040), (50, 300, 1040), (300, 520, 1040)):
        g = torch.Generator(device=dev)
        g.manual_seed(M)
        a = torch.randint(-127, 128, (M, K), generator=g, device=dev, dtype=torch.int8)
        w = torch.randint(-127, 128, (N, K), generator=g, device=dev, dtype=torch.int8)
        out = torch.empty(M, N, device=dev)
        call(pn, torch, a, torch.ones(M, device=dev), w, torch.ones(N, device=dev), out)
        torch.cuda.synchronize()
        assert torch.equal(out.double(), exact(torch, a, w))


def test_scales_that_are_not_finite(env):
    """A NaN scale makes its row NaN and no other; so quantised rows that are not finite stay marked."""
    pn, torch, dev = env
    for M in (3, 40, 300):
        a = torch.ones(M, 64, dtype=torch.int8, device=dev)
        w = torch.ones(90, 64, dtype=torch.int8, device=dev)
        sa, sw = torch.ones(M, device=dev), torch.ones(90, device=dev)
        sa[1], sw[5] = float("nan"), float("inf")
        out = torch.empty(M, 90, device=dev)
        call(pn, torch, a, sa, w, sw, out)
        torch.cuda.synchronize()
        assert out[1].isnan().all() and (out[0, :5] == 64).all() and (out[2:, 5] == float("inf")).all()
        assert (out[2:, 6:] == 64).all()


def test_large_offsets(env):
    """Operands and outputs past 2^31 bytes: the last rows against the first ones' copy."""
    pn, torch, dev = env
    M, N, K = 40000, 27000, 32
    a = torch.randint(-128, 128, (M, K), device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), device=dev, dtype=torch.int8)
    sa, sw = torch.ones(M, device=dev), torch.ones(N, device=dev)
    out = torch.zeros(M, N, device=dev)  # 4.3 GB
    call(pn, torch, a, sa, w, sw, out)
    torch.cuda.synchronize()
    for at in (0, 20000, M - 700):
        assert torch.equal(out[at:at + 700].double(), exact(torch, a[at:at + 700], w))
    del out
    M, N, K = 20, 17000, 131056  # 2.2 GB of weights
    w = torch.randint(-128, 128, (N, K), device=dev, dtype=torch.int8)
    for M in (2, 40, 300):
        a = torch.randint(-128, 128, (M, K), device=dev, dtype=torch.int8)
        out = torch.zeros(M, N, device=dev)
        sa, sw = torch.ones(M, device=dev), torch.ones(N, device=dev)
        call(pn, torch, a, sa, w, sw, out)
        torch.cuda.synchronize()
        within(torch, out[:, -200:], exact(torch, a, w[-200:]), sa, sw[-200:], "float32")


def test_graphs_that_share_a_workspace(env):
    """Two captured products of different sizes over one workspace, replayed in turn with eager calls between."""
    pn, torch, dev = env
    sizes = [(3, 100, 4096), (40, 64, 17408), (70, 130, 8192)]
    need = max(pn.gemm_int8_workspace_bytes(*s) for s in sizes)
    work = torch.randint(0, 256, (need + 16,), dtype=torch.uint8, device=dev)
    made = []
    for M, N, K in sizes:
        a = torch.randint(-128, 128, (M, K), device=dev, dtype=torch.int8)
        w = torch.randint(-128, 128, (N, K), device=dev, dtype=torch.int8)
        sa, sw = torch.rand(M, device=dev), torch.rand(N, device=dev)
        out = torch.empty(M, N, device=dev)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pn.gemm_int8(a, sa, w, sw, out, work)
        made.append((graph, a, sa, w, sw, out))
    for n in range(4):
        for graph, a, sa, w, sw, out in made:
            a.copy_(torch.randint(-128, 128, a.shape, device=dev, dtype=torch.int8))
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            again = torch.empty_like(out)
            call(pn, torch, a, sa, w, sw, again, fill=n)
            torch.cuda.synchronize()
            assert torch.equal(out, again)
            within(torch, out, exact(torch, a, w), sa, sw, "float32")


def test_side_stream(env):
    pn, torch, dev = env
    a = torch.randint(-128, 128, (20, 2048), device=dev, dtype=torch.int8)
    w = torch.randint(-128, 128, (333, 2048), device=dev, dtype=torch.int8)
    sa, sw = torch.rand(20, device=dev), torch.rand(333, device=dev)
    one, two = torch.empty(20, 333, device=dev), torch.empty(20, 333, device=dev)
    call(pn, torch, a, sa, w, sw, one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    work = torch.empty(pn.gemm_int8_workspace_bytes(20, 333, 2048) + 16, dtype=torch.uint8, device=dev)
    pn.gemm_int8(a, sa, w, sw, two, work, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(one, two)


def test_empty_and_refusals(env):
    pn, torch, dev = env
    a, w = torch.zeros(4, 64, dtype=torch.int8, device=dev), torch.zeros(8, 64, dtype=torch.int8, device=dev)
    sa, sw, out = torch.ones(4, device=dev), torch.ones(8, device=dev), torch.zeros(4, 8, device=dev)
    pn.gemm_int8(a[:0], sa[:0], w, sw, out[:0])
    pn.gemm_int8(a, sa, w[:0], sw[:0], out[:, :0].contiguous())
    for args in ((a.cpu(), sa, w, sw, out), (a, sa[:3], w, sw, out), (a, sa, w[:, :32], sw, out), (a, sa, w, sw[:7], out),
                 (a, sa, w, sw, out.double()), (a, sa, w, sw, out.t().contiguous()), (a.int(), sa, w, sw, out),
                 (a, sa, w.float(), sw, out), (a, sa, w, sw, out[:, :7]), (a[0], sa, w, sw, out),
                 (a, sa, w, sw, out[:1].expand(4, 8)), (a, sa, w, sw, torch.zeros(8, 4, device=dev).t())):
        with pytest.raises(ValueError):
            pn.gemm_int8(*args)
    with pytest.raises(pn.PNError):  # K is not a multiple of 16
        pn.gemm_int8(a[:, :24].contiguous(), sa, w[:, :24].contiguous(), sw, out)
    for M, N, K in ((40, 64, 17408), (3, 64, 17408)):
        need = pn.gemm_int8_workspace_bytes(M, N, K)
        if need:
            a, w = torch.zeros(M, K, dtype=torch.int8, device=dev), torch.zeros(N, K, dtype=torch.int8, device=dev)
            sa, sw, out = torch.ones(M, device=dev), torch.ones(N, device=dev), torch.zeros(M, N, device=dev)
            for work in (None, torch.zeros(need - 1, dtype=torch.uint8, device=dev),
                         torch.zeros(need + 16, dtype=torch.uint8, device=dev)[8:8 + need]):
                with pytest.raises(pn.PNError):
                    pn.gemm_int8(a, sa, w, sw, out, work)
