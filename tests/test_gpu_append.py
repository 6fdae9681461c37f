"""Rotated keys into the cache on the GPU against the definition in 64 bits: every byte of the cache and every
bit of the turned queries."""
import numpy as np
import pytest

import prompt_reference as ref
import step_reference as step
from step_reference import MXFP4, MXFP8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


def numbers(torch, rng, shape, dtype):
    x = rng.normal(size=shape) * np.exp2(rng.integers(-12, 6, size=shape[:-1] + (1,)))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def check(env, fmt, heads, dim, page, T, Hq, rot, type_, interleaved, seed=0, slots=None, positions=None, rows=None,
          place=None, in_place=False, k=None, q=None):
    pn, torch, dev = env
    rng = np.random.default_rng(seed + dim + T + rot)
    dt = getattr(torch, type_)
    pages = (T + 7) // page + 2
    host = step.Cache(fmt, heads, dim, page, pages, 0xA5)
    cache = pn.Cache(fmt, heads, dim, page, torch.from_numpy(host.data.copy()).to(dev))
    k = numbers(torch, rng, (T, heads, dim), dt) if k is None else k
    v = numbers(torch, rng, (T, heads, dim), dt)
    if q is None:
        q = numbers(torch, rng, (T, Hq, dim), dt) if Hq else None
    if slots is None:
        slots = 7 + np.arange(T)
        order = rng.permutation(pages)
        slots = order[slots // page] * page + slots % page
    rows = rows or T + 40
    table = ref.table(rows, rot)
    given = positions
    if positions is None:
        given = rng.integers(0, rows, size=T)
    row = table[np.clip(given, 0, rows - 1)]
    host.write(ref.turn(k.double().numpy(), row, interleaved).astype(np.float64), v.double().numpy(), slots)
    place = place or (lambda t: t.to(dev))
    a = {}
    if Hq:
        a["q"] = place(q)
        a["q_out"] = a["q"] if in_place else place(torch.zeros_like(q))
    pn.cache_append(cache, place(k), place(v), torch.from_numpy(np.asarray(slots)).to(dev), torch.from_numpy(table).to(dev),
                    positions=torch.from_numpy(given).to(dev), interleaved=interleaved, **a)
    torch.cuda.synchronize()
    got = cache.data.cpu().numpy()
    bad = np.nonzero(got != host.data)[0]
    assert bad.size == 0, (bad.size, bad[:5], got[bad[:5]], host.data[bad[:5]])
    if Hq:
        want = torch.from_numpy(ref.turn(q.double().numpy(), row, interleaved)).to(dt)
        have = a["q_out"].cpu()
        assert torch.equal(have.isnan(), want.isnan()) and torch.equal(have[~want.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,page,T,Hq,rot", [
    (1, 64, 32, 1, 1, 64), (3, 64, 64, 37, 5, 32), (2, 128, 32, 66, 12, 128), (4, 256, 128, 35, 24, 256),
    (2, 256, 64, 5, 3, 64), (5, 128, 1024, 3, 7, 8)])
def test_every_byte(env, type_, fmt, interleaved, heads, dim, page, T, Hq, rot):
    check(env, fmt, heads, dim, page, T, Hq, rot, type_, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_width_of_rotation(env, dim, interleaved):
    for rot in range(8, dim + 1, 8):
        check(env, MXFP8, 2, dim, 32, 5, 3, rot, "bfloat16", interleaved)


@pytest.mark.parametrize("T", [2, 4, 16, 31, 32, 33, 64, 129, 300])
def test_lengths(env, T):
    check(env, MXFP8, 2, 64, 32, T, 4, 64, "bfloat16", False)
    check(env, MXFP4, 1, 128, 64, T, 9, 96, "float32", False)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [24, 64])
def test_queries_in_place(env, rot, interleaved):
    check(env, MXFP8, 2, 64, 32, 21, 6, rot, "float16", interleaved, in_place=True)


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_and_unaligned(env, type_, interleaved):
    """q, k and v as slices of one fused projection, at strides and offsets that no vector load takes."""
    pn, torch, dev = env

    def place(t, token=3, off=1):
        n = t.shape[1] * t.shape[2]
        wide = torch.zeros(t.shape[0] * (n + token) + 8, dtype=t.dtype, device=dev)
        view = wide[off:off + t.shape[0] * (n + token)].view(-1, n + token)[:, :n].view(t.shape)
        view.copy_(t)
        return view
    check(env, MXFP8, 3, 64, 32, 21, 5, 48, type_, interleaved, place=place)
    check(env, MXFP4, 2, 128, 32, 9, 4, 128, type_, interleaved, place=lambda t: place(t, 4, 4))
    # heads before tokens
    check(env, MXFP8, 3, 64, 32, 21, 5, 64, type_, interleaved,
          place=lambda t: t.transpose(0, 1).contiguous().to(dev).transpose(0, 1))


def test_slots_outside_and_positions_outside(env):
    T, page = 40, 32
    slots = 7 + np.arange(T)
    slots[[1, 2, 39]] = [-1, 1 << 40, -(1 << 40)]
    slots[5] = ((T + 7) // page + 2) * page  # one past the last
    positions = np.arange(T)
    positions[[0, 3, 4]] = [-5, 1 << 40, 10 ** 6]
    check(env, MXFP8, 2, 64, page, T, 4, 64, "float32", False, slots=slots, positions=positions)


def test_positions_left_out(env):
    """A row of the table for each token, as rotations of several axes come."""
    pn, torch, dev = env
    T, table = 17, ref.table(20, 64)
    k = torch.randn(T, 2, 64, device=dev)
    slots = torch.arange(T, device=dev)
    data = [torch.zeros(2 * pn.cache_page_bytes(MXFP8, 2, 64, 32), dtype=torch.uint8, device=dev) for _ in range(2)]
    for d, positions in zip(data, (None, torch.arange(T, device=dev))):
        pn.cache_append(pn.Cache(MXFP8, 2, 64, 32, d), k, k, slots, torch.from_numpy(table).to(dev), positions=positions)
    torch.cuda.synchronize()
    assert torch.equal(*data)
    with pytest.raises(pn.PNError):
        pn.cache_append(pn.Cache(MXFP8, 2, 64, 32, data[0]), k, k, slots, torch.from_numpy(table[:16]).to(dev))


def test_numbers_that_are_not_finite(env):
    pn, torch, dev = env
    rng = np.random.default_rng(2)
    k = numbers(torch, rng, (9, 2, 128), torch.float32)
    k[0, 0, 3], k[1, 1, 100], k[2, 0, 64] = float("nan"), float("inf"), -float("inf")
    k[3] = 3e38   # a turn may pass the largest number
    k[4] = 1e-45
    k[5] = 0.0
    k[6] = -0.0
    q = numbers(torch, rng, (9, 4, 128), torch.float32)
    q[0, 0, 3], q[1, 1, 100] = float("nan"), float("inf")
    for interleaved in (False, True):
        for fmt in (MXFP8, MXFP4):
            check(env, fmt, 2, 128, 32, 9, 4, 96, "float32", interleaved, k=k, q=q)


def test_as_cache_write_without_a_turn(env):
    """Angles of zero: the bytes of cache_write."""
    pn, torch, dev = env
    table = torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], 1).to(dev)
    for fmt in (MXFP8, MXFP4):
        k, v = torch.randn(50, 3, 128, device=dev).half(), torch.randn(50, 3, 128, device=dev).half()
        slots = torch.randperm(64, device=dev)[:50]
        data = [torch.zeros(2 * pn.cache_page_bytes(fmt, 3, 128, 32), dtype=torch.uint8, device=dev) for _ in range(2)]
        pn.cache_write(pn.Cache(fmt, 3, 128, 32, data[0]), k, v, slots)
        pn.cache_append(pn.Cache(fmt, 3, 128, 32, data[1]), k, v, slots, table, positions=torch.zeros_like(slots))
        torch.cuda.synchronize()
        assert torch.equal(*data)


def test_cache_past_4_gib(env):
    pn, torch, dev = env
    heads, dim, page = 4, 256, 1024
    each = pn.cache_page_bytes(MXFP8, heads, dim, page)
    pages = (5 << 30) // each
    cache = pn.Cache(MXFP8, heads, dim, page, torch.empty(pages * each, dtype=torch.uint8, device=dev))
    slots = torch.tensor([0, pages * page - 1, pages * page - 700], device=dev)
    k = torch.randn(3, heads, dim, device=dev).bfloat16()
    table = torch.cat([torch.ones(1, 128), torch.zeros(1, 128)], 1).to(dev)
    pn.cache_append(cache, k, k, slots, table, positions=torch.zeros_like(slots))
    back, v = torch.empty_like(k), torch.empty_like(k)
    pn.cache_read(cache, slots, back, v)
    torch.cuda.synchronize()
    assert torch.equal(back, v) and bool(((back - k).abs() <= k.abs().amax(-1, keepdim=True) / 16).all())


def test_streams_and_graph(env):
    pn, torch, dev = env
    q, k, v = (torch.randn(6, n, 128, device=dev) for n in (8, 2, 2))
    q_out, slots, positions = torch.empty_like(q), torch.arange(6, device=dev), torch.arange(6, device=dev)
    table = torch.from_numpy(ref.table(100, 128)).to(dev)
    data = [torch.zeros(pn.cache_page_bytes(MXFP8, 2, 128, 64), dtype=torch.uint8, device=dev) for _ in range(2)]
    cache, other = (pn.Cache(MXFP8, 2, 128, 64, d) for d in data)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pn.cache_append(cache, k, v, slots, table, positions=positions, q=q, q_out=q_out)
    side = torch.cuda.Stream()
    for n in range(4):
        k.copy_(torch.randn_like(k))
        positions += 3
        slots += 4
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        again = torch.empty_like(q)
        pn.cache_append(other, k, v, slots, table, positions=positions, q=q, q_out=again, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(*data) and torch.equal(q_out, again)


def test_empty_and_refusals(env):
    pn, torch, dev = env
    cache = pn.Cache(MXFP8, 2, 64, 32, torch.zeros(pn.cache_page_bytes(MXFP8, 2, 64, 32), dtype=torch.uint8, device=dev))
    table = torch.zeros(10, 64, device=dev)
    k, slots = torch.zeros(3, 2, 64, device=dev), torch.arange(3, device=dev)
    pn.cache_append(cache, k[:0], k[:0], slots[:0], table)
    for a, b in (((cache, k[:, :1], k, slots, table), {}), ((cache, k, k.half(), slots, table), {}),
                 ((cache, k, k, slots.int(), table), {}), ((cache, k, k, slots[:2], table), {}),
                 ((cache, k, k, slots, table.double()), {}), ((cache, k, k, slots, table[:, ::2]), {}),
                 ((cache, k, k, slots, table), dict(positions=slots.int())), ((cache, k, k, slots, table), dict(q=k)),
                 ((cache, k, k, slots, table), dict(q=k, q_out=k[:2])), ((cache, k, k, slots, table), dict(q=k.half(), q_out=k)),
                 ((cache, k.cpu(), k, slots, table), {}), ((cache, k, k, slots, table[0]), {})):
        with pytest.raises(ValueError):
            pn.cache_append(*a, **b)
    for t in (torch.zeros(10, 12, device=dev), torch.zeros(10, 72, device=dev), torch.zeros(0, 64, device=dev),
              torch.zeros(641, device=dev)[1:].view(10, 64)):
        with pytest.raises(pn.PNError):
            pn.cache_append(cache, k, k, slots, t)
