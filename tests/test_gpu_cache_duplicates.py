"""Slots that repeat in one read of the cache, next to each other and far apart: the same numbers each
time."""
import numpy as np
import pytest

from step_reference import MXFP4, MXFP8
from test_gpu_cache import env, pair  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 32), (3, 128, 64), (2, 256, 32)])
def test_duplicate_reads(env, type_, fmt, heads, dim, page):
    pn, torch, dev = env
    rng = np.random.default_rng(dim)
    host, cache = pair(pn, torch, dev, fmt, heads, dim, page, 3)
    n = 3 * page
    k, v = rng.normal(size=(2, n, heads, dim))
    host.write(k, v, np.arange(n))
    cache.data.copy_(torch.from_numpy(host.data))
    slots = np.concatenate([[5, 5, 5, 5, 5], rng.integers(0, n, 40), np.repeat(rng.integers(0, n, 9), 3), [5, -1, -1, n]])
    dt = getattr(torch, type_)
    got = [torch.full((len(slots), heads, dim), 7.0, dtype=dt, device=dev) for _ in range(2)]
    pn.cache_read(cache, torch.from_numpy(slots).to(dev), *got)
    torch.cuda.synchronize()
    for x, want in zip(got, host.read(slots)):
        assert torch.equal(x.cpu(), torch.from_numpy(want).float().to(dt))
        assert torch.equal(x[0], x[4]) and torch.equal(x[0], x[-4]) and not x[-3:].any()
