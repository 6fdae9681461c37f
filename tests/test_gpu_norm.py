"""The residual norm and the 8-bit rows on the GPU against their definitions in 64 bits: sums and codes bit
for bit, plain outputs and scales within their roundings."""
import numpy as np
import pytest

import prompt_reference as ref

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 2.0 ** -150, "bfloat16": 2.0 ** -134, "float16": 2.0 ** -25}  # half the smallest subnormal


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


def numbers(torch, rng, shape, dtype, spread=3.0):
    x = rng.normal(size=shape) * np.exp2(spread * rng.normal(size=shape[:-1] + (1,)))
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(dtype)


def near(got, want, type_):
    """What 64 bits computed (its own error: under 2^-45 of it) rounded to fp32 and to the type."""
    got, want = got.double().cpu().numpy(), np.asarray(want)
    fine = np.isfinite(want)
    with np.errstate(over="ignore"):
        most = np.abs(want) * (HALF[type_] * (1 + 1e-6) + (type_ != "float32") * 2.0 ** -24) + TINY[type_]
        assert (np.isnan(got) == np.isnan(want)).all()
        # what rounds past the type's largest number is infinite
        err = np.abs(np.where(fine, got, 0.0) - np.where(fine, want, 0.0))
    assert (got[~fine & ~np.isnan(want)] == want[~fine & ~np.isnan(want)]).all()
    over = fine & np.isinf(got) & (np.abs(want) >= {"float32": 3.4028235e38, "bfloat16": 3.38e38, "float16": 65504.0}[type_])
    assert (over | (err <= most))[fine].all(), (err - most)[fine & ~over].max()


def check(env, rows, K, type_, wtype, residual, plain, codes, seed, x=None, res=None, weight=None, eps=1e-6, place=None):
    """place: turns a host tensor into the device tensor that the call is given."""
    pn, torch, dev = env
    rng = np.random.default_rng(seed)
    dt = getattr(torch, type_)
    x = numbers(torch, rng, (rows, K), dt) if x is None else x
    weight = (1 + 0.3 * torch.from_numpy(rng.normal(size=K).astype(np.float32))).to(getattr(torch, wtype)) if weight is None else weight
    if residual and res is None:
        res = numbers(torch, rng, (rows, K), dt)
    place = place or (lambda t: t.to(dev))
    h = (x.float() + res.float()).to(dt) if residual else x
    y, t, r = ref.norm(h.double().numpy(), weight.double().numpy(), eps)
    a = dict(residual=place(res), sum=place(torch.zeros(rows, K, dtype=dt))) if residual else {}
    if plain:
        a["out"] = place(torch.zeros(rows, K, dtype=dt))
    if codes:
        a["codes"] = torch.full((rows, K), 77, dtype=torch.int8, device=dev)
        a["scales"] = torch.full((rows,), 77.0, device=dev)
    pn.add_norm(place(x), weight.to(dev), eps, **a)
    torch.cuda.synchronize()
    if residual:
        got = a["sum"].cpu()
        assert torch.equal(got.isnan(), h.isnan()) and torch.equal(got[~h.isnan()], h[~h.isnan()])
    if plain:
        near(a["out"], y, type_)
    if codes:
        want, scales = ref.int8_rows(t, r)
        bad = np.nonzero(a["codes"].cpu().numpy() != want)
        assert bad[0].size == 0, (bad[0][:5], bad[1][:5])
        near(a["scales"], scales, "float32")


WIDTHS = [1, 7, 8, 64, 200, 512, 520, 1000, 1024, 1032, 4096, 4104, 5120, 8192, 8200, 17408]


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("K", WIDTHS)
def test_widths(env, K, type_):
    rows = 9 if K < 4096 else 3
    check(env, rows, K, type_, type_, True, True, True, K)


@pytest.mark.parametrize("K", [8191, 8193, 32768, 65528, 65535, 65536])
@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
def test_widest(env, K, type_):
    check(env, 2, K, type_, "float32", False, True, True, K)


@pytest.mark.parametrize("residual,plain,codes", [(False, True, False), (False, False, True), (True, True, False),
                                                  (True, False, True)])
@pytest.mark.parametrize("type_,wtype", [("float32", "bfloat16"), ("bfloat16", "float32"), ("float16", "bfloat16"),
                                         ("bfloat16", "float16")])
def test_outputs_and_types(env, residual, plain, codes, type_, wtype):
    check(env, 5, 640, type_, wtype, residual, plain, codes, 5)
    check(env, 5, 77, type_, wtype, residual, plain, codes, 6)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 257, 1030])
@pytest.mark.parametrize("K", [96, 1536])
def test_rows(env, rows, K):
    check(env, rows, K, "bfloat16", "bfloat16", True, True, True, rows)


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("K", [48, 640])
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (0, 1), (16, 5)])
def test_strided_and_unaligned(env, type_, K, pad, off):
    """Rows as slices of a wider matrix, at strides and offsets that no vector load takes."""
    pn, torch, dev = env

    def place(t):
        wide = torch.full((t.shape[0] * (K + pad) + off + 16,), 3.0, dtype=t.dtype, device=dev)
        view = wide[off:off + t.shape[0] * (K + pad)].view(t.shape[0], K + pad)[:, :K]
        view.copy_(t)
        return view
    check(env, 6, K, type_, type_, True, True, True, 8, place=place)


def test_strides_leave_what_lies_between(env):
    pn, torch, dev = env
    x = torch.randn(4, 64, device=dev)
    wide = torch.full((4, 100), 9.0, device=dev)
    pn.add_norm(x, torch.ones(64, device=dev), 1e-6, out=wide[:, 8:72])
    torch.cuda.synchronize()
    assert (wide[:, :8] == 9).all() and (wide[:, 72:] == 9).all() and (wide[:, 8:72] != 9).all()


@pytest.mark.parametrize("K", [72, 1032, 5120])
def test_in_place(env, K):
    """sum over the residual, out over x, and sum over x: the same bits."""
    pn, torch, dev = env
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x, res = (torch.randn(7, K, generator=g, device=dev).bfloat16() for _ in range(2))
    w = torch.randn(K, generator=g, device=dev)
    out, s = torch.empty_like(x), torch.empty_like(x)
    pn.add_norm(x, w, 1e-5, out=out, residual=res, sum=s)
    x1, res1 = x.clone(), res.clone()
    pn.add_norm(x1, w, 1e-5, out=x1, residual=res1, sum=res1)
    x2, out2 = x.clone(), torch.empty_like(x)
    pn.add_norm(x2, w, 1e-5, out=out2, residual=res, sum=x2)
    torch.cuda.synchronize()
    assert torch.equal(x1, out) and torch.equal(res1, s) and torch.equal(out2, out) and torch.equal(x2, s)


@pytest.mark.parametrize("K", [40, 77, 2056])
@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
def test_rows_that_are_not_finite(env, K, type_):
    """NaN and infinities, in x and made by the addition; rows of zeros; the largest and smallest numbers."""
    pn, torch, dev = env
    dt = getattr(torch, type_)
    rng = np.random.default_rng(K)
    x = numbers(torch, rng, (12, K), dt, 0.5)
    big, small = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    x[0, 3] = float("nan")
    x[1, K - 1] = float("inf")
    x[2, 0] = -float("inf")
    x[3] = 0.0
    x[4] = -0.0
    x[5] = big
    x[6] = -big * 0.5
    x[6, 0] = big
    x[7] = torch.from_numpy(rng.normal(size=K)).to(dt) * small * 4
    x[8] = 0.0
    x[8, 2] = small / 4
    x[9] = small / 8
    res = torch.zeros_like(x)
    res[10], x[10] = big, big  # the sum is infinite
    check(env, 12, K, type_, type_, True, True, True, 1, x=x, res=res)
    check(env, 12, K, type_, "float32", False, True, True, 1, x=x, eps=0.0)
    huge = torch.full((K,), 3e38)
    huge[::2] = 1e-38
    check(env, 12, K, type_, "float32", False, True, True, 1, x=x, weight=huge)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weight_that_is_not_finite(env, value):
    pn, torch, dev = env
    w = torch.ones(600)
    w[599] = value
    x = torch.randn(3, 600)
    x[1, 599] = 0.0
    check(env, 3, 600, "float32", "float32", False, True, True, 1, x=x, weight=w)


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("K", [1, 8, 63, 511, 520, 5120, 17408])
def test_quantize_rows(env, type_, K):
    """Ties, their neighbours, and ordinary numbers; rows of zeros, NaN and infinities."""
    pn, torch, dev = env
    rng = np.random.default_rng(K)
    dt = getattr(torch, type_)
    x = numbers(torch, rng, (8, K), dt, 2.0)
    steps = torch.from_numpy(rng.integers(-254, 255, size=K) / 2.0).to(dt)  # halves of a step
    steps[0] = 127.0
    x[1], x[2] = steps, steps * 3 if type_ != "float16" else steps
    if type_ == "float32":
        x[3] = torch.nextafter(steps, torch.full_like(steps, 1e9))
        x[3, 0] = 127.0
    x[4] = 0.0
    x[5, K // 2] = float("nan")
    x[6, K - 1] = -float("inf")
    codes = torch.full((8, K), 55, dtype=torch.int8, device=dev)
    scales = torch.full((8,), 55.0, device=dev)
    pn.int8_quantize_rows(x.to(dev), codes, scales)
    torch.cuda.synchronize()
    want, want_scales = ref.int8_rows(x.double().numpy())
    assert (codes.cpu().numpy() == want).all()
    near(scales, want_scales, "float32")
    wide = torch.zeros(8, K + 5, dtype=dt, device=dev)
    wide[:, 2:2 + K] = x.to(dev)
    again = torch.full_like(codes, 55)
    pn.int8_quantize_rows(wide[:, 2:2 + K], again, scales)
    torch.cuda.synchronize()
    assert torch.equal(codes, again)


def test_many_ties_after_a_norm(env):
    """Products that land on borders between codes: exact in 64 bits, not in 32."""
    pn, torch, dev = env
    K = 1024
    w = torch.full((K,), 3.0)
    x = torch.arange(K).float()[None] * 0.5 - 128.0
    x = x.clamp(-127, 127)
    check(env, 1, K, "float32", "float32", False, False, True, 1, x=x, weight=w)
    w = torch.full((K,), 1.0 + 2.0 ** -23)
    check(env, 1, K, "float32", "float32", False, False, True, 1, x=x, weight=w)


def test_streams_and_graph(env):
    pn, torch, dev = env
    x = torch.randn(33, 1280, device=dev).bfloat16()
    w = torch.randn(1280, device=dev).bfloat16()
    codes, scales = torch.empty(33, 1280, dtype=torch.int8, device=dev), torch.empty(33, device=dev)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pn.add_norm(x, w, 1e-6, out=out, codes=codes, scales=scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pn.add_norm(x, w, 1e-6, out=out, codes=codes, scales=scales)
        pn.int8_quantize_rows(out, codes, scales)
    for n in range(4):
        x.copy_(torch.randn(33, 1280, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        again, c2, s2 = torch.empty_like(out), torch.empty_like(codes), torch.empty_like(scales)
        pn.add_norm(x, w, 1e-6, out=again, stream=side)
        side.synchronize()
        pn.int8_quantize_rows(again, c2, s2)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(codes, c2) and torch.equal(scales, s2)


def test_empty_and_refusals(env):
    pn, torch, dev = env
    w = torch.ones(64, device=dev)
    x = torch.zeros(0, 64, device=dev)
    pn.add_norm(x, w, 1e-6, out=x)
    pn.int8_quantize_rows(x, torch.zeros(0, 64, dtype=torch.int8, device=dev), torch.zeros(0, device=dev))
    x = torch.zeros(4, 64, device=dev)
    codes, scales = torch.zeros(4, 64, dtype=torch.int8, device=dev), torch.zeros(4, device=dev)
    for bad in (dict(), dict(codes=codes), dict(scales=scales), dict(out=x.bfloat16()), dict(out=x[:3]),
                dict(out=x, residual=x.half()), dict(out=x, sum=torch.zeros(64, 4, device=dev).t()),
                dict(out=x, codes=codes.int(), scales=scales), dict(out=x, codes=codes, scales=scales[:3]),
                dict(out=x[:1].expand(4, 64))):
        with pytest.raises(ValueError):
            pn.add_norm(x, w, 1e-6, **bad)
    for bad in (w[:63], w.double(), w.cpu(), torch.ones(128, device=dev)[::2]):
        with pytest.raises(ValueError):
            pn.add_norm(x, bad, 1e-6, out=x)
    with pytest.raises(ValueError):
        pn.add_norm(x.double(), w, 1e-6, out=x)
    with pytest.raises(pn.PNError):
        pn.add_norm(x, w, -1.0, out=x)
    with pytest.raises(pn.PNError):
        pn.add_norm(torch.zeros(1, 65537, device=dev), torch.ones(65537, device=dev), 1e-6,
                    out=torch.zeros(1, 65537, device=dev))
    with pytest.raises(ValueError):
        pn.int8_quantize_rows(x[0], codes, scales)
