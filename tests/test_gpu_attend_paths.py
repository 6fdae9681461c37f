"""Every way that a call's rows are dealt to the attention kernels: a prefix's row tiles in stream and in
shared workgroups, several row blocks of them, the joining of few and of many rows, tables wider than the
lengths, with ragged drafts and sequences without tokens in each.

The bound of a row, against sum w |v| / sum w, from the roundings on its way (u = 2^-24):
  a score     q and k are exact; parts * dim products summed, each sum within u of sum |scale q k|; scaling
              and the subtraction 5 u of it, the references of two joins 4 u, and 8 u of exponentials
  a weight    its parts: 2^-24 for fp32 q, 2^-16 for fp16 and bf16, 2^-8 for bf16 in shared workgroups
  the sums    an addition a token and part, and 64 of the joins, the inverse and the product
Errors of the weights count in the numerator and in the sum. The output is rounded to its type once."""
import numpy as np
import pytest

import step_reference as ref
from step_reference import MXFP4, MXFP8
from test_gpu_attend import Case, env  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float32": U, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
PARTS = {"float32": 3, "bfloat16": 1, "float16": 2}
TYPES = ["float32", "bfloat16", "float16"]


def close(c, type_):
    out, lse = (x.double().numpy() for x in c.run())
    want, lse_want, mix, size, count = ref.attend(c.host, c.q64, c.table, c.lens, c.prefix_table, c.prefix, c.scale,
                                                  c.q_lens)
    B, Q, Hq, dim = want.shape
    shared = c.prefix > 0 and B * Q * Hq // c.cache.heads > 64
    tokens = count[:, :, None]
    score = ((PARTS[type_] * dim + 16) * size + 8) * U
    sums = (max(PARTS[type_], 2) * tokens + 64) * U
    weight = {"float32": U, "float16": 2.0 ** -16, "bfloat16": 2.0 ** -8 if shared else 2.0 ** -16}[type_]
    tol = (weight + 2 * score + 2 * sums)[..., None] * mix
    tol = tol + HALF[type_] * (np.abs(want) + tol) + (2.0 ** -25 if type_ == "float16" else 1e-37)
    assert np.isfinite(out).all()
    assert (np.abs(out - want) <= tol).all(), np.max(np.abs(out - want) / tol)
    seen = np.isfinite(lse_want)
    assert np.array_equal(np.isneginf(lse), ~seen)
    ltol = score + sums + 8 * U * (1 + np.abs(np.where(seen, lse_want, 0.0)))
    off = np.abs(np.where(seen, lse, 0.0) - np.where(seen, lse_want, 0.0))
    assert (off <= ltol).all(), np.max(off / ltol)
    nq = np.full(B, Q) if c.q_lens is None else c.q_lens
    none = np.arange(Q) >= nq[:, None]  # places without a query token
    assert not out[none].any() and np.isneginf(lse[none]).all()
    return out, lse


# sequences, query tokens, query heads a KV head, KV heads: rows of a KV head and in all
ROWS = [(2, 3, 8, 2),   # 48: four tiles of a stream workgroup
        (1, 4, 8, 2),   # 32: two
        (3, 4, 8, 2),   # 96: shared, 16 rows a wave
        (6, 4, 8, 2),   # 192: 32 rows a wave where registers allow, else two blocks
        (9, 6, 8, 3)]   # 432, 1296 in all: the most a wave holds, blocks, a join of many rows


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("fmt", [MXFP8, MXFP4])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("B,Q,G,heads", ROWS)
def test_rows_of_a_prefix(env, type_, fmt, dim, B, Q, G, heads):
    """Own lengths from none to three records, query tokens from none to all."""
    lens = [(37 * b + 5) % 75 if b % 4 != 3 else 0 for b in range(B)]
    q_lens = [Q - b % (Q + 1) for b in range(B)]
    close(Case(env, 1000 + dim + B, fmt, heads, G, dim, 32, 300, lens, Q, type_, q_lens=q_lens), type_)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_rows_without_a_prefix(env, type_, dim):
    """Rows enough for the join of many, cut into several ranges each."""
    B, Q, G, heads = 5, 7, 10, 3
    lens = [0, 1, 700, 33, 6]
    close(Case(env, 1100 + dim, MXFP8, heads, G, dim, 64, 0, lens, Q, type_, q_lens=[7, 7, 3, 6, 0]), type_)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("fmt,dim", [(MXFP8, 64), (MXFP4, 128), (MXFP8, 256)])
@pytest.mark.parametrize("wide", [5, 200])
def test_tables_wider_than_the_lengths(env, type_, fmt, dim, wide):
    """The cut goes by the table; what its columns past a sequence's tokens hold is no page."""
    c = Case(env, 1200 + dim, fmt, 2, 4, dim, 32, 0, [100, 33, 0, 257], 2, type_)
    rest = np.full((4, wide), 1 << 30, np.int32)
    rest[:, ::2] = -9
    c.table = np.ascontiguousarray(np.concatenate([c.table, rest], 1))
    close(c, type_)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("prefix", [0, 64])
def test_rows_without_a_query_beside_long_ones(env, type_, prefix):
    """Fewer query tokens than the call over many records: their rows see none of them."""
    c = Case(env, 1300, MXFP8, 1, 6, 128, 64, prefix, [900, 400, 64, 1], 4, type_, q_lens=[1, 2, 4, 3])
    close(c, type_)


@pytest.mark.parametrize("type_", TYPES)
def test_the_same_bits_each_time(env, type_):
    """Own tokens in several ranges, stream and shared prefixes: a call repeats its bits, in another
    workspace and after another call."""
    for B, Q, G, heads in (ROWS[0], ROWS[3]):
        c = Case(env, 1400, MXFP8, heads, G, 128, 32, 300, [60] * B, Q, type_)
        first = c.run()
        Case(env, 1401, MXFP4, 1, 3, 64, 32, 40, [30] * 7, 2, type_).run()
        again = c.run()
        assert c.torch.equal(first[0], again[0]) and c.torch.equal(first[1], again[1])
