"""The microscaled cache on the GPU against its definition in 64 bits: every byte that writing leaves,
every number that reading gives."""
import numpy as np
import pytest

import step_reference as ref
from step_reference import MXFP4, MXFP8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


def pair(pn, torch, dev, fmt, heads, dim, page, pages, fill=0):
    """The same cache on the host and on the device."""
    c = ref.Cache(fmt, heads, dim, page, pages, fill)
    return c, pn.Cache(fmt, heads, dim, page, torch.from_numpy(c.data.copy()).to(dev))


def numbers(torch, rng, shape, dtype, special):
    """Numbers of the type (as a float64 array too): normal ones over many binades and, where
    `special`, blocks of ties, subnormals, signed zeros, huge numbers, NaN and infinities."""
    x = rng.normal(size=shape) * np.exp2(rng.integers(-20, 6, size=shape[:-1] + (1,)))
    if special:
        flat = x.reshape(-1, 32)
        n = len(flat)
        half = np.float64([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -0.0, 0.0])
        flat[0 % n, :12] = half
        flat[1 % n] = 0.0
        flat[2 % n, 3] = np.nan
        flat[3 % n, 31] = np.inf
        flat[4 % n, 0] = -np.inf
        flat[5 % n] = 448.0 * (1 + np.arange(32) / 16)   # both sides of the exponent's border
        flat[6 % n] = np.exp2(-np.arange(32.0))          # down to the element type's zero
        flat[7 % n] = -np.exp2(-np.arange(32.0)) * 1.5
        flat[8 % n] = (16 + np.arange(32)) * 2.0 ** -9   # ties of E4M3
        flat[8 % n, 0] = 448.0
        if dtype != torch.float16:
            flat[9 % n] = 1e-38 * np.arange(32)          # subnormal, and the smallest exponent
            flat[10 % n] = 2.0 ** 126 * np.linspace(0.5, 1.99, 32)
            flat[11 % n, 7] = 2.0 ** 127
            flat[12 % n] = 2.0 ** -118 * np.arange(32)
    with np.errstate(over="ignore"):
        t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return t, t.double().numpy()


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("heads,dim,page,T", [(1, 64, 32, 1), (3, 64, 64, 37), (2, 128, 32, 66), (4, 256, 128, 35),
                                              (5, 128, 1024, 3)])
def test_write_every_byte(env, type_, fmt, heads, dim, page, T):
    pn, torch, dev = env
    rng = np.random.default_rng(dim + T + fmt)
    pages = (T + 7) // page + 2
    host, cache = pair(pn, torch, dev, fmt, heads, dim, page, pages, fill=0xA5)
    dt = getattr(torch, type_)
    k, k64 = numbers(torch, rng, (T, heads, dim), dt, True)
    v, v64 = numbers(torch, rng, (T, heads, dim), dt, True)
    slots = 7 + np.arange(T)
    if T > 3:
        order = rng.permutation(pages)
        slots = order[slots // page] * page + slots % page
        slots[[1, 2]] = [-1, pages * page]  # padding, and past the end
        slots[3] = -(1 << 40)
    host.write(k64, v64, slots)
    pn.cache_write(cache, k.to(dev), v.to(dev), torch.from_numpy(slots).to(dev))
    torch.cuda.synchronize()
    got = cache.data.cpu().numpy()
    bad = np.nonzero(got != host.data)[0]
    assert bad.size == 0, (bad[:5], got[bad[:5]], host.data[bad[:5]])


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
def test_write_strided_and_unaligned(env, type_, fmt):
    """k and v as slices of one fused projection, at strides that no vector load takes."""
    pn, torch, dev = env
    rng = np.random.default_rng(11)
    T, heads, dim = 21, 3, 64
    host, cache = pair(pn, torch, dev, fmt, heads, dim, 32, 2)
    dt = getattr(torch, type_)
    k, k64 = numbers(torch, rng, (T, heads, dim), dt, True)
    v, v64 = numbers(torch, rng, (T, heads, dim), dt, True)
    buf = torch.zeros(T, 2 * heads * (dim + 1) + 3, dtype=dt, device=dev)
    kd = buf[:, 1:1 + heads * (dim + 1)].unflatten(1, (heads, dim + 1))[..., :dim]
    vd = buf[:, 1 + heads * (dim + 1):1 + 2 * heads * (dim + 1)].unflatten(1, (heads, dim + 1))[..., 1:]
    kd.copy_(k)
    vd.copy_(v)
    # and with heads outermost
    ke = k.transpose(0, 1).contiguous().to(dev).transpose(0, 1)
    ve = v.transpose(0, 1).contiguous().to(dev).transpose(0, 1)
    slots = rng.permutation(64)[:T]
    host.write(k64, v64, slots)
    for a, b in ((kd, vd), (ke, ve)):
        cache.data.zero_()
        pn.cache_write(cache, a, b, torch.from_numpy(slots).to(dev))
        torch.cuda.synchronize()
        assert np.array_equal(cache.data.cpu().numpy(), host.data)


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("heads,dim,page,T", [(1, 64, 32, 1), (3, 64, 64, 50), (2, 128, 32, 67), (2, 256, 128, 33)])
def test_read_every_number(env, type_, fmt, heads, dim, page, T):
    """Random bytes are a cache too: every code, every exponent from 16 up, NaN blocks."""
    pn, torch, dev = env
    rng = np.random.default_rng(dim + T)
    host, cache = pair(pn, torch, dev, fmt, heads, dim, page, 3)
    rec = host.data.reshape(-1, ref.record_bytes(fmt, dim))
    exps = rec.shape[1] - 2 * dim
    rec[:, :exps] = rng.integers(0, 256, rec[:, :exps].shape)
    rec[:, exps:] = rng.integers(16, 248 if fmt == MXFP8 else 253, rec[:, exps:].shape)
    rec[:, exps + 3::17] = 255
    cache.data.copy_(torch.from_numpy(host.data))
    slots = rng.integers(0, 3 * page, T)
    if T > 3:
        slots[[0, 2]] = [-5, 3 * page]
        slots[3] = slots[4]
    dt = getattr(torch, type_)
    k = torch.full((T, heads, dim), 7.0, dtype=dt, device=dev)
    v = torch.full_like(k, 7.0)
    pn.cache_read(cache, torch.from_numpy(slots).to(dev), k, v)
    torch.cuda.synchronize()
    for got, want in zip((k, v), host.read(slots)):
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want).to(torch.float32).to(dt)  # exact, then one rounding
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=0.0), torch.nan_to_num(want, nan=0.0))


def test_no_tokens_and_duplicate_reads(env):
    pn, torch, dev = env
    _, cache = pair(pn, torch, dev, MXFP8, 2, 64, 32, 1)
    none = torch.zeros(0, dtype=torch.int64, device=dev)
    kv = torch.zeros(0, 2, 64, device=dev)
    pn.cache_write(cache, kv, kv, none)
    pn.cache_read(cache, none, kv, kv)
    torch.cuda.synchronize()


def test_binding_refusals(env):
    pn, torch, dev = env
    _, cache = pair(pn, torch, dev, MXFP8, 2, 64, 32, 1)
    kv = torch.zeros(3, 2, 64, device=dev)
    slots = torch.arange(3, device=dev)
    for k, v, s in ((kv[:2], kv, slots), (kv, kv.half(), slots), (kv.double(), kv.double(), slots),
                    (kv, kv, slots.int()), (kv, kv, slots[:2]), (kv.cpu(), kv, slots), (kv, kv, slots.cpu()),
                    (torch.zeros(3, 64, 2, device=dev).transpose(1, 2), kv, slots)):
        with pytest.raises(ValueError):
            pn.cache_write(cache, k, v, s)
        with pytest.raises(ValueError):
            pn.cache_read(cache, s, k, v)
    with pytest.raises(ValueError):
        pn.Cache(MXFP8, 2, 64, 32, cache.data[:-1])
    with pytest.raises(pn.PNError):  # 4-byte offset of an 8-byte-per-4 store
        odd = torch.zeros(3 * 2 * 64 + 1, device=dev)[1:].view(3, 2, 64)
        pn.cache_read(cache, slots, odd, kv)
