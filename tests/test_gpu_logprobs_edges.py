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
