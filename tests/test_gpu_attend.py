"""Attention over the microscaled cache on the GPU against the 64-bit formula.

The bound of a row, from the roundings on its way (u = 2^-24, the fp32 one; u16 = 2^-8, the bf16 one):
  a score     q in two bf16 parts (fp32 q) is off by 2^-16 relative, exact otherwise; the sum of dim
              products of exact factors by (dim + 1) u, each relative to sum |scale q k|; scaling,
              subtracting the maximum and the exponential by 4 u (|s| + |m|) + 4 u
  a weight    that, and its rounding to bf16 (u16), to two bf16 parts (2^-16) for fp32 and fp16 q
  the sums    one addition a record of a wave, then the joins: (tokens / 32 + 64) u
Weights enter the numerator and the sum, so the relative errors count twice, against
sum w |v| / sum w; the output is rounded to its type at the end."""
import numpy as np
import pytest

import step_reference as ref
from step_reference import MXFP4, MXFP8
from test_gpu_cache import pair

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


class Case:
    def __init__(self, env, seed, fmt, heads, group, dim, page, prefix, lens, Q, type_, q_lens=None, scale=None,
                 poison=0x7F, amp=1.5, prefill=None):
        self.pn, self.torch, self.dev = pn, torch, dev = env
        rng = np.random.default_rng(seed)
        self.dtype = getattr(torch, type_)
        B = len(lens)
        width = max(1, -(-max(lens) // page))
        npp = -(-prefix // page)
        pages = npp + B * width + 1
        # unwritten places hold NaN codes and NaN exponents
        self.host, self.cache = pair(pn, torch, dev, fmt, heads, dim, page, pages, fill=poison)
        self.host.data.reshape(-1, ref.record_bytes(fmt, dim))[:, -2 * dim:] = 255
        order = rng.permutation(pages)
        self.prefix_table, self.prefix = order[:npp].astype(np.int32), prefix
        self.table = order[npp:npp + B * width].reshape(B, width).astype(np.int32)
        self.lens = np.array(lens, np.int32)
        slots = ref.slots_of(self.prefix_table, prefix, page)
        for b in range(B):
            slots += ref.slots_of(self.table[b], lens[b], page)
        self.slots = np.array(slots, np.int64).reshape(-1)
        T = len(slots)
        k = rng.normal(size=(T, heads, dim)).astype(np.float32)
        v = rng.normal(size=(T, heads, dim)).astype(np.float32)
        if prefill is not None:
            prefill(self, k, v)
        self.host.write(k.astype(np.float64), v.astype(np.float64), self.slots)
        self.cache.data.copy_(torch.from_numpy(self.host.data))
        for b in range(B):  # pages that no token of the sequence needs are not pages at all
            self.table[b, -(-lens[b] // page):] = -7 if b % 2 else 1 << 30
        q = torch.from_numpy((amp * rng.normal(size=(B, Q, heads * group, dim))).astype(np.float32)).to(self.dtype)
        self.q64, self.q = q.double().numpy(), q.to(dev)
        self.q_lens = None if q_lens is None else np.array(q_lens, np.int32)
        self.scale = dim ** -0.5 if scale is None else scale

    def up(self, a):
        return None if a is None else self.torch.from_numpy(a).to(self.dev)

    def args(self, q=None):
        torch = self.torch
        q = self.q if q is None else q
        table = self.up(self.table)
        need = self.pn.attend_workspace_bytes(self.cache, q, table, self.prefix)
        work = torch.full((need,), 0xFF, dtype=torch.uint8, device=self.dev)  # NaN to begin with
        out = torch.full(q.shape, float("nan"), dtype=self.dtype, device=self.dev)
        lse = torch.full(q.shape[:3], float("nan"), device=self.dev)
        return (self.cache, q, table, self.up(self.lens), out, lse, work), dict(
            prefix_table=self.up(self.prefix_table), prefix_len=self.prefix, q_lens=self.up(self.q_lens),
            scale=self.scale)

    def run(self, q=None):
        a, kw = self.args(q)
        self.pn.attend(*a, **kw)
        self.torch.cuda.synchronize()
        return a[4].cpu(), a[5].cpu()

    def check(self, got=None):
        out, lse = self.run() if got is None else got
        want, lse_want, mix, size, count = ref.attend(
            self.host, self.q64, self.table, self.lens, self.prefix_table, self.prefix, self.scale, self.q_lens)
        two = self.dtype != self.torch.bfloat16
        dim = self.q.shape[3]
        nan = np.isnan(want)
        with np.errstate(invalid="ignore"):
            tokens = count[:, :, None]
            score = size * ((2.0 ** -16 if self.dtype == self.torch.float32 else 0.0) + (dim + 1) * U + 8 * U) + 4 * U
            sums = (tokens / 32 + 64) * U
            weight = (2.0 ** -16 if two else 2.0 ** -8) + score
            tol = (weight + score + 2 * sums)[..., None] * mix
            last = {self.torch.float32: U, self.torch.bfloat16: 2.0 ** -8, self.torch.float16: 2.0 ** -11}[self.dtype]
            tol = tol * (1 + last) + last * np.abs(want) + (2.0 ** -25 if self.dtype == self.torch.float16 else 1e-37)
            got = out.double().numpy()
            assert np.array_equal(np.isnan(got), nan), "NaN in other places"
            worst = np.max(np.where(nan, 0.0, np.abs(got - want) / tol), initial=0.0)
            assert worst <= 1.0, f"out: {worst} of the bound"
            seen = np.isfinite(lse_want)
            l = lse.double().numpy()
            off = np.where(seen, np.abs(l - lse_want), 0.0)
            ltol = score + sums + 2 * U * (2 + np.abs(np.where(seen, lse_want, 0.0)))
            assert np.array_equal(np.isneginf(l), np.isneginf(lse_want)), "rows that see nothing"
            assert np.array_equal(np.isnan(l), np.isnan(lse_want))
            assert np.all(off <= np.where(seen, ltol, 1.0)), f"lse: {np.max(off / ltol)} of the bound"
        return out, lse


TYPES = ["float32", "bfloat16", "float16"]


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("heads,group,dim,page", [(1, 1, 64, 32), (2, 6, 64, 64), (1, 5, 128, 32), (2, 6, 128, 128),
                                                  (1, 6, 256, 64)])
def test_own_tokens(env, type_, fmt, heads, group, dim, page):
    """No prefix: lengths around a record and a page, none at all, one query token or three."""
    lens = [0, 1, 31, 32, 33, 95, 200]
    for Q in (1, 3):
        Case(env, 100 + dim + Q, fmt, heads, group, dim, page, 0, lens, Q, type_).check()


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("dim,prefix,Q,B", [(64, 1, 1, 2), (64, 97, 4, 3), (128, 33, 1, 2), (128, 257, 5, 4),
                                            (256, 64, 1, 3), (256, 161, 3, 4)])
def test_shared_prefix(env, type_, fmt, dim, prefix, Q, B):
    lens = [(17 * b + 1) % 70 for b in range(B)]
    lens[-1] = 0
    Case(env, 200 + dim + prefix, fmt, 2, 6, dim, 32, prefix, lens, Q, type_).check()


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_ranges_and_row_blocks(env, type_, fmt, dim):
    """Long enough for many token ranges, rows enough for several row blocks of either part."""
    Case(env, 300 + dim, fmt, 1, 12, dim, 64, 1500, [700, 65, 3], 6, type_).check()
    Case(env, 301 + dim, fmt, 1, 8, dim, 64, 0, [2500], 1, type_).check()


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("prefix", [0, 40])
def test_ragged_drafts(env, type_, prefix):
    """Sequences with fewer query tokens than the call, none among them; lengths below the drafts."""
    c = Case(env, 401, MXFP8, 2, 4, 128, 32, prefix, [50, 2, 33, 0, 130], 4, type_, q_lens=[4, 3, 0, 2, 1])
    out, lse = c.check()
    assert not out[2].any() and np.isneginf(lse[2].numpy()).all()
    assert not out[0, 3:].any() or c.q_lens[0] == 4


@pytest.mark.parametrize("type_", TYPES)
def test_strided_queries(env, type_):
    """q as part of a fused projection with heads padded, at an odd offset, and with heads outermost."""
    c = Case(env, 500, MXFP8, 2, 3, 64, 32, 45, [40, 70], 2, type_)
    plain = c.check()
    torch, q = c.torch, c.q
    B, Q, H, D = q.shape
    padded = torch.zeros(B, Q, H + 2, D + 3, dtype=q.dtype, device=c.dev)[:, :, 1:1 + H, 1:1 + D]
    padded.copy_(q)
    outer = q.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    for other in (padded, outer):
        assert other.stride() != q.stride()
        got = c.run(other)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 2.5])
def test_scales(env, scale):
    Case(env, 600, MXFP8, 1, 4, 64, 32, 33, [70, 5], 2, "float32", scale=scale).check()


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
def test_scores_that_grow_along_the_tokens(env, type_):
    """Every record raises the maximum: the running sums are rescaled each time; and one key far above
    all others."""
    def grow(c, k, v):
        k *= np.linspace(0.01, 4.0, len(k))[:, None, None].astype(np.float32)
    Case(env, 700, MXFP8, 1, 4, 64, 32, 500, [600, 40], 2, type_, prefill=grow, amp=3.0).check()

    def spike(c, k, v):
        k[5] *= 30
        k[-3] *= 30
    Case(env, 701, MXFP8, 1, 4, 64, 32, 200, [300, 40], 2, type_, prefill=spike).check()


@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
def test_nan_only_where_it_is_seen(env, fmt, type_):
    """A NaN block in v or k of a drafted token reaches that token's row and later ones, not the rows
    before it, nor the other sequence; one in the prefix reaches all."""
    def bad_v(c, k, v):
        v[-2, 0, 40] = np.nan   # the last sequence's last token but one: channels 32..63 of head 0

    def bad_k(c, k, v):
        k[-2, 1, 3] = np.inf    # all of head 1's output

    def bad_prefix(c, k, v):
        v[3, 1, 0] = np.nan
    for prefill, heads in ((bad_v, 2), (bad_k, 2), (bad_prefix, 2)):
        c = Case(env, 800, fmt, heads, 3, 64, 32, 40, [20, 45], 3, type_, prefill=prefill)
        out, _ = c.check()
        if prefill is not bad_prefix:
            nan = c.torch.isnan(out)
            assert not nan[0].any() and not nan[1, 0].any() and nan[1, 1:].any()


def test_nan_and_infinite_queries(env):
    c = Case(env, 810, MXFP8, 1, 4, 64, 32, 40, [40], 2, "float32")
    c.q[0, 0, 1, 5] = float("nan")
    c.q64[0, 0, 1, 5] = np.nan
    out, lse = c.run()
    assert c.torch.isnan(out[0, 0, 1]).all() and c.torch.isnan(lse[0, 0, 1])
    rest = np.ones((2, 4), bool)
    rest[0, 1] = False
    assert np.isfinite(out[0].numpy()[rest]).all()


def test_pages_outside_the_cache_stay_in_bounds(env):
    """A page number that is none gives some value; the other sequences' are not touched by it."""
    c = Case(env, 820, MXFP8, 1, 4, 64, 32, 0, [70, 70], 1, "float32")
    good = c.check()
    c.table[1, 0] = -(1 << 31)
    c.table[1, 1] = (1 << 31) - 1
    out, _ = c.run()
    assert c.torch.equal(out[0], good[0][0])


def test_lengths_outside_the_table(env):
    """A negative length is none, one past the table's pages is all of them."""
    c = Case(env, 830, MXFP8, 1, 4, 64, 32, 20, [64, 64], 1, "float32")
    plain = c.check()
    c.lens = np.array([1 << 30, 64], np.int32)
    out, lse = c.run()
    assert c.torch.equal(out, plain[0])
    c.lens = np.array([-5, 64], np.int32)
    out, lse = c.run()
    c.lens = np.array([0, 64], np.int32)
    c.check((out, lse))


def test_no_sequence_no_query_no_lse(env):
    c = Case(env, 840, MXFP8, 1, 4, 64, 32, 20, [64, 10], 2, "float32")
    pn, torch = c.pn, c.torch
    a, kw = c.args()
    full = c.check()
    a = a[:5] + (None,) + a[6:]
    pn.attend(*a, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a[4].cpu(), full[0])
    for shape in ((0, 2, 4, 64), (2, 0, 4, 64)):
        q = torch.zeros(shape, device=c.dev)
        table = torch.zeros(shape[0], 2, dtype=torch.int32, device=c.dev)
        lens = torch.zeros(shape[0], dtype=torch.int32, device=c.dev)
        assert pn.attend_workspace_bytes(c.cache, q, table) == 0
        pn.attend(c.cache, q, table, lens, torch.empty_like(q))


def test_sequences_without_own_pages(env):
    """A table of no columns: the prefix alone; and no prefix either."""
    c = Case(env, 850, MXFP4, 1, 4, 64, 32, 50, [0, 0], 2, "float32")
    c.table = np.zeros((2, 0), np.int32)
    c.check()
    c.prefix = 0
    out, lse = c.run()
    assert not out.any() and np.isneginf(lse.numpy()).all()


@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
def test_cache_past_four_gigabytes(env, fmt):
    """Pages at both ends of a cache whose byte offsets pass 32 bits, written, read and attended to."""
    pn, torch, dev = env
    heads, dim, page = 2, 256, 1024
    each = pn.cache_page_bytes(fmt, heads, dim, page)
    pages = (9 << 29) // each + 2  # a little over 4.5 GiB
    cache = pn.Cache(fmt, heads, dim, page, torch.zeros(pages * each, dtype=torch.uint8, device=dev))
    rng = np.random.default_rng(9)
    T = 70
    k, v = (torch.from_numpy(rng.normal(size=(T, heads, dim)).astype(np.float32)).to(dev) for _ in range(2))
    small = pn.Cache(fmt, heads, dim, page, torch.zeros(2 * each, dtype=torch.uint8, device=dev))
    at = torch.arange(T, device=dev)
    q = torch.from_numpy(rng.normal(size=(1, 2, 8, dim)).astype(np.float32)).to(dev)
    got = []
    for c, first, second in ((cache, pages - 1, pages - 2), (small, 1, 0)):
        pn.cache_write(c, k, v, first * page + at)
        pn.cache_write(c, v, k, second * page + at)
        rk, rv = torch.empty_like(k), torch.empty_like(v)
        pn.cache_read(c, first * page + at, rk, rv)
        table = torch.tensor([[first]], dtype=torch.int32, device=dev)
        prefix = torch.tensor([second], dtype=torch.int32, device=dev)
        lens = torch.tensor([T], dtype=torch.int32, device=dev)
        out, lse = torch.empty_like(q), torch.empty(1, 2, 8, device=dev)
        work = torch.empty(pn.attend_workspace_bytes(c, q, table, T), dtype=torch.uint8, device=dev)
        pn.attend(c, q, table, lens, out, lse, work, prefix_table=prefix, prefix_len=T)
        got.append((rk, rv, out, lse))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0].abs().max() > 1


def test_streams_and_graph_replays(env):
    """A step (write, attend) on a side stream and in a captured graph: the eager bits each time."""
    c = Case(env, 900, MXFP8, 2, 6, 128, 32, 300, [100, 33], 2, "float32")
    pn, torch, dev = env
    eager = c.run()
    a, kw = c.args()
    slots = torch.from_numpy(c.slots[-2:].copy()).to(dev)
    k, v = torch.empty(2, 2, 128, device=dev), torch.empty(2, 2, 128, device=dev)
    pn.cache_read(c.cache, slots, k, v)  # what stands there: writing it again changes nothing
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        pn.cache_write(c.cache, k, v, slots, stream=s)
        pn.attend(*a, stream=s, **kw)
    step()
    s.synchronize()
    assert torch.equal(a[4].cpu(), eager[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for rep in range(4):
        a[4].fill_(float("nan"))
        a[5].fill_(float("nan"))
        a[6].fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[4].cpu(), eager[0]) and torch.equal(a[5].cpu(), eager[1]), f"replay {rep}"


def test_binding_refusals(env):
    c = Case(env, 910, MXFP8, 1, 4, 64, 32, 20, [64, 10], 2, "float32")
    pn, torch = c.pn, c.torch
    a, kw = c.args()

    def bad(i, x, **more):
        b = list(a)
        b[i] = x
        with pytest.raises((ValueError, pn.PNError)):
            pn.attend(*b, **{**kw, **more})
    q = a[1]
    bad(1, q.double())
    bad(1, q[0])
    bad(1, q[..., :32])
    bad(1, q.cpu())
    bad(1, torch.zeros(2, 2, 64, 4, device=c.dev).transpose(2, 3))
    bad(2, a[2].long())
    bad(2, a[2][:1])
    bad(3, a[3].long())
    bad(3, a[3][:1])
    bad(4, a[4].half())
    bad(4, a[4][:1])
    bad(5, a[5].double())
    bad(6, None)
    bad(6, a[6][:-1])
    bad(0, c.cache, prefix_len=33)
    bad(0, c.cache, prefix_len=-1)
    bad(0, c.cache, prefix_table=kw["prefix_table"].long())
    bad(0, c.cache, q_lens=torch.zeros(3, dtype=torch.int32, device=c.dev))
    bad(0, c.cache, scale=float("nan"))


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("fmt,dim,prefix,B", [(MXFP8, 64, 700, 2), (MXFP4, 128, 700, 12), (MXFP8, 256, 0, 3)])
def test_other_rows_do_not_change_a_row(env, type_, fmt, dim, prefix, B):
    """A row's bits stay as they are whatever the rows beside it hold: others whose scores grow along the
    tokens move their references, not this row's. Stream and shared workgroups of the prefix, own tokens."""
    def grow(c, k, v):
        k *= np.linspace(0.05, 3.0, len(k))[:, None, None].astype(np.float32)
    c = Case(env, 920 + dim, fmt, 1, 6, dim, 64, prefix, [600 if not prefix else 50] * B, 2, type_, prefill=grow)
    plain = c.check()
    other = c.q.clone()
    other[0, 1] *= 9
    other[1:] *= -7
    other[0, 0, 1:] *= 5
    got = c.run(other)
    assert not c.torch.equal(got[0][0, 1], plain[0][0, 1])
    for new, old in zip(got, plain):
        assert c.torch.equal(new[0, 0, 0], old[0, 0, 0])
