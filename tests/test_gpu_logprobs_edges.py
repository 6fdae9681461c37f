"""Log probabilities where their arithmetic or their launch ends: signalling NaN."""
import numpy as np
import pytest

from test_gpu_logprobs import call, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


@pytest.mark.parametrize("type_,whole,bits", [("float32", "int32", 0x7F800001), ("float32", "int32", -0x7FFFFF),
                                              ("bfloat16", "int16", 0x7F81), ("float16", "int16", 0x7C01)])
@pytest.mark.parametrize("V", [70, 5000, 70000])
@pytest.mark.parametrize("top", [0, 1, 20, 64])
def test_signalling_nan(env, type_, whole, bits, V, top):
    """Bits of a signalling NaN beside the largest logits: rank and the likeliest go by comparisons alone, as beside a
    quiet one."""
    pn, torch, dev = env
    rng = np.random.default_rng(V)
    away = [-513, -512, -256, -3, -2, -1, 1, 2, 3, 4, 8, 16, 255, 256, 257, 511, 512, 1024]
    x = torch.from_numpy((3 * rng.normal(size=(len(away) + 3, V))).astype(np.float32)).to(getattr(torch, type_))
    raw = x.view(getattr(torch, whole))
    for r, d in enumerate(away):
        for at in rng.choice(V, size=min(V // 2, 40), replace=False):
            x[r, at] = 20.0 + float(rng.integers(0, 64)) / 8
            raw[r, (at + d) % V] = bits
    raw[-3, torch.from_numpy(rng.random(V) < 0.3)] = bits
    raw[-2, torch.from_numpy(rng.random(V) < 0.99)] = bits
    raw[-1] = bits
    values = x.double().numpy()
    assert np.isnan(values).any(1).all()
    tokens = np.array([rng.choice(np.append(np.nonzero(~np.isnan(v))[0], 0)) for v in values], np.int32)
    tokens[0] = int(np.nanargmax(values[0]))
    got = call(pn, torch, x.to(dev), torch.from_numpy(tokens).to(dev), 1.0, top)
    torch.cuda.synchronize()
    same(got, values, tokens, 1.0, top)


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("scale", [0.25, 1e-3, 1.0])
def test_differences_past_fp32(env, type_, scale):
    """The largest and the smallest numbers in one row, of which a scale below one makes log probabilities within fp32."""
    pn, torch, dev = env
    low = {"float32": -3.4028234663852886e38, "bfloat16": -3.3895313892515355e38}[type_]
    x = np.zeros((3, 50))
    x[0, 3], x[0, 7] = -low, low
    x[1], x[1, 40] = low, -low / 2
    x[2, 5], x[2, 6], x[2, 7] = -low, -np.inf, low
    tokens = np.array([7, 0, 6], np.int32)
    t = torch.from_numpy(x.astype(np.float32)).to(getattr(torch, type_))
    got = call(pn, torch, t.to(dev), torch.from_numpy(tokens).to(dev), scale, 50)
    torch.cuda.synchronize()
    if scale < 1.0:  # in full; at one the definition passes fp32 too
        assert got["logprob"].isfinite().tolist() == [True, True, False]
        same(got, t.double().numpy(), tokens, scale, 50)
    else:
        assert bool((got["logprob"][[0, 2]] == -float("inf")).all()) and bool((got["top_ids"][0, :2].cpu() == torch.tensor([3, 0])).all())


@pytest.mark.parametrize("V,scale", [(1, 2.0 ** -121), (7001, 2.7e-33), (70001, 2.7e-32)])
def test_smallest_scales(env, V, scale):
    """Logits as large as such a scale makes ordinary."""
    pn, torch, dev = env
    rng = np.random.default_rng(V)
    x = torch.from_numpy((3 / scale * rng.normal(size=(4, V))).clip(-3e38, 3e38).astype(np.float32))
    tokens = rng.integers(0, V, size=4).astype(np.int32)
    got = call(pn, torch, x.to(dev), torch.from_numpy(tokens).to(dev), scale, min(V, 9))
    torch.cuda.synchronize()
    same(got, x.double().numpy(), tokens, scale, min(V, 9))
