"""What attention makes of single numbers: infinite, huge and NaN queries, and the bits that a query and a
softmax weight keep on their way through the bf16 products.

Three ways through the kernels: own tokens, a prefix under few rows, a prefix under more than 64 rows."""
import numpy as np
import pytest

from step_reference import MXFP4, MXFP8
from test_gpu_attend import Case, env  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float32": U, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}  # half a step, relative to a binade's start
TYPES = ["float32", "bfloat16", "float16"]
WAYS = {  # prefix given the tokens, own lengths, B, Q, query heads of the one KV head
    "own": (False, 2, 3, 8),
    "prefix": (True, 2, 3, 8),
    "shared": (True, 5, 4, 4),
    "shared, more rows": (True, 15, 4, 8),
}


def case(env, seed, way, tokens, type_, fmt, dim, prefill, **more):
    """Every query token sees all `tokens` tokens: with a prefix no own ones, else own ones and nq = 1 or
    what is asked for."""
    prefix, B, Q, G = WAYS[way]
    if prefix:
        return Case(env, seed, fmt, 1, G, dim, 32, tokens, [0] * B, Q, type_, prefill=prefill, **more)
    return Case(env, seed, fmt, 1, Q * G, dim, 32, 0, [tokens] * B, 1, type_, prefill=prefill, **more)


def put(c, q):
    """q [B][Q][Hq][dim], as the case's queries."""
    q = c.torch.from_numpy(q.astype(np.float32)).to(c.dtype)
    c.q64, c.q = q.double().numpy(), q.to(c.dev)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinite_queries(env, type_, way, dim):
    """By the channel's keys: all positive, of both signs, zero in one token. A score of +infinity leaves
    the mean undefined (NaN, log of the sum +infinity), NaN too; a row whose every score is -infinity has
    no weight anywhere, as one that sees nothing. The other rows keep their bits."""
    def keys(c, k, v):
        k[:, 0, 1] = np.abs(k[:, 0, 1]) + 1.0
        k[0, 0, 2], k[1, 0, 2] = 2.0, -2.0
        k[:, 0, 3] = np.abs(k[:, 0, 3]) + 1.0
        k[2, 0, 3] = 0.0
    c = case(env, 60 + dim, way, 40, type_, MXFP8, dim, keys)
    plain = c.run()
    q, inf, nan = c.q64.copy(), np.inf, np.nan
    rows = q.reshape(-1, dim)
    want = {0: (1, inf, nan, inf), 3: (1, -inf, 0.0, -inf), 4: (2, inf, nan, inf), 9: (2, -inf, nan, inf),
            13: (3, inf, nan, nan), 14: (3, -inf, nan, nan), 20: (5, nan, nan, nan), len(rows) - 1: (1, -inf, 0.0, -inf)}
    for r, (channel, x, _, _) in want.items():
        rows[r, channel] = x
    put(c, q)
    out, lse = c.run()
    out, lse = out.double().numpy().reshape(-1, dim), lse.double().numpy().ravel()
    for r, (_, _, o, l) in want.items():
        assert np.array_equal(out[r], np.full(dim, o), equal_nan=True), (r, out[r][:8], o)
        assert np.array_equal(lse[r], l, equal_nan=True), (r, lse[r], l)
    others = np.setdiff1d(np.arange(len(rows)), list(want))
    assert np.array_equal(out[others], plain[0].double().numpy().reshape(-1, dim)[others])
    assert np.array_equal(lse[others], plain[1].double().numpy().ravel()[others])


def one_key(c, k, v):
    """Token 0 of a sequence (or of the prefix) has a key of zeros and a value of zeros, token 1 a key of one
    in channel 0 and a value of ones."""
    k[:], v[:] = 0.0, 0.0
    k[1::2, :, 0] = 1.0
    v[1::2] = 1.0


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("fmt,dim", [(MXFP8, 64), (MXFP4, 128), (MXFP8, 256)])
def test_a_query_keeps_its_bits(env, type_, way, fmt, dim):
    """One token with a key of one in one channel: the log of the sum is the score, scale * q, itself. q
    enters in parts that make it up, and products with 1 and 0 and their sums are exact. Then the score
    times scale * log2(e) (two constants and a product: 3 u), the same less itself to the exponential and
    back (u of it, 4 u from 2^x and log2), one sum and ln 2 (3 u): within 8 u of |scale q| + 1."""
    def keys(c, k, v):
        k[:], v[:] = 0.0, 1.0
        k[:, :, 0] = 1.0
    c = case(env, 70, way, 1, type_, fmt, dim, keys, scale=0.125)
    rng = np.random.default_rng(71)
    q = np.zeros(c.q64.shape)
    q[..., 0] = rng.normal(size=q.shape[:-1]) * np.exp2(rng.integers(-6, 8, size=q.shape[:-1]))
    put(c, q)
    out, lse = c.run()
    want = 0.125 * c.q64[..., 0]
    off = np.abs(lse.double().numpy() - want) / (8 * U * (np.abs(want) + 1))
    assert off.max() <= 1, off.max()
    assert (out.double().numpy() == 1.0).all()


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_the_largest_queries(env, way, dim):
    """q up to the largest fp32 number, which no bf16 part can hold alone, over keys that small: finite
    scores, within the bound of the test before."""
    def keys(c, k, v):
        k[:], v[:] = 0.0, 1.0
        k[:, :, 1] = 2.0 ** -117
    c = case(env, 72, way, 1, "float32", MXFP8, dim, keys, scale=2.0 ** -4)
    top = np.float64(np.finfo(np.float32).max)
    q = np.zeros(c.q64.shape)
    n = q[..., 0].size
    q[..., 1] = (top * np.linspace(0.99, 1.0, n) * np.where(np.arange(n) % 2, 1, -1)).reshape(q.shape[:-1])
    put(c, q)
    out, lse = c.run()
    want = 2.0 ** -121 * c.q64[..., 1]
    off = np.abs(lse.double().numpy() - want) / (8 * U * (np.abs(want) + 1))
    assert off.max() <= 1, off.max()
    assert (out.numpy() == 1.0).all()


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("fmt,dim", [(MXFP8, 64), (MXFP4, 128), (MXFP8, 256)])
def test_a_weight_keeps_its_bits(env, type_, way, fmt, dim):
    """Two tokens, scores 0 and s = scale * q, values 0 and 1: the output is e^s / (1 + e^s). s is exact as
    above; its scaling and the subtraction are off by 4 u |s| (|s| <= 6), two exponentials by 2 u each, the
    sum, its inverse and the product by u each: 32 u together. The weights enter the product with the
    values as three bf16 parts, which make them up, for fp32; as two (2^-16 at most) for fp16 and bf16; the
    shared way takes bf16 queries' weights as one (2^-8). The output is rounded once."""
    c = case(env, 73, way, 2, type_, fmt, dim, one_key, scale=0.25)
    rng = np.random.default_rng(74)
    q = np.zeros(c.q64.shape)
    q[..., 0] = rng.uniform(-24, 24, size=q.shape[:-1])
    put(c, q)
    out, _ = c.run()
    want = 1 / (1 + np.exp(-0.25 * c.q64[..., 0]))
    parts = {"float32": 0.0, "float16": 2.0 ** -16, "bfloat16": 2.0 ** -8 if way.startswith("shared") else 2.0 ** -16}
    tol = (32 * U + parts[type_]) * want
    tol = tol + HALF[type_] * np.exp2(np.floor(np.log2(want + tol)))
    off = np.abs(out.double().numpy() - want[..., None]) / tol[..., None]
    assert off.max() <= 1, off.max()


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("way", WAYS)
def test_a_scale_of_zero_and_the_largest(env, type_, way):
    """Scores of q.k up to 1e38 under a scale of zero weigh alike, whatever q; and a scale up to the largest
    fp32 number gives finite scores of queries that small. One bound as above: 0 and s are exact."""
    def keys(c, k, v):
        one_key(c, k, v)
        k[:, :, 0] *= 2.0 ** 60
    c = case(env, 75, way, 2, type_, MXFP8, 64, keys, scale=0.0)
    q = np.zeros(c.q64.shape)
    q[..., 0] = np.linspace(-1, 1, q[..., 0].size).reshape(q.shape[:-1]) * 2.0 ** 66
    put(c, q)
    out, lse = c.run()
    assert (out.double().numpy() == 0.5).all()
    assert np.abs(lse.double().numpy() - np.log(2)).max() <= 8 * U

    def zeros(c, k, v):
        k[:] = 0.0
    for scale in (2.0 ** 127, float(np.finfo(np.float32).max), -2.0 ** 127.5):
        c = case(env, 76, way, 1, type_, MXFP8, 64, zeros, scale=float(np.float32(scale)))
        _, lse = c.run()
        assert (lse.double().numpy() == 0.0).all()

        def small(c, k, v):
            k[:], v[:] = 0.0, 1.0
            k[:, :, 0] = 2.0 ** -60
        c = case(env, 77, way, 1, type_, MXFP8, 64, small, scale=float(np.float32(scale)))
        q = np.zeros(c.q64.shape)
        q[..., 0] = np.linspace(-1, 1, q[..., 0].size).reshape(q.shape[:-1]) * 2.0 ** -65
        put(c, q)
        out, lse = c.run()
        want = np.float64(np.float32(scale)) * 2.0 ** -60 * c.q64[..., 0]
        assert np.abs(want).max() >= 4
        off = np.abs(lse.double().numpy() - want) / (8 * U * (np.abs(want) + 1))
        assert off.max() <= 1, off.max()
        assert (out.double().numpy() == 1.0).all()


@pytest.mark.parametrize("type_", ["float32", "float16"])
@pytest.mark.parametrize("way", ["own", "prefix"])
@pytest.mark.parametrize("fmt,dim", [(MXFP8, 128), (MXFP4, 256)])
def test_small_parts_of_a_score_add_up(env, type_, way, fmt, dim):
    """A score of one large product and of pairs 1 + d, -1 whose second parts d each 32 channels' product
    adds: less than half a step of the large one each time, one or two whole steps together. Against a
    key without the pairs the weights differ by e^(scale * their sum). Every sum is exact if the small
    parts meet each other first; then the exponents are off by their own rounding alone, below 32 u."""
    big, k0, d, scale = (2.0 ** 9, 1.0, 2.0 ** -19, 2.0 ** 13) if type_ == "float32" else (
        2.0 ** 15, 4.0, 2.0 ** -10, 2.0 ** 5)
    pairs = 1024 // dim if type_ == "float32" else 4  # of the 16 that 32 channels of one product hold

    def keys(c, k, v):
        k[:], v[:] = 0.0, 0.0
        k[0::2] = 1.0
        v[0::2] = 1.0
        k[:, :, 0] = k0
        k[:, :, 1] = 0.0
    c = case(env, 78, way, 2, type_, fmt, dim, keys, scale=scale)
    q = np.zeros(c.q64.shape)
    for p in range(dim // 64):
        for j in range(2):  # channels 64p + 16g + 8j + 0..7 are one product's
            for n in range(pairs):
                at = 64 * p + 16 * (n % 4) + 8 * j + 2 + 2 * (n // 4)
                q[..., at], q[..., at + 1] = 1.0 + d, -1.0
    q[..., 0] = big
    put(c, q)
    assert np.array_equal(c.q64, q)
    total = dim // 32 * pairs * d
    step = 2.0 ** -23 * big * k0
    assert pairs * d < step / 2 and total % step == 0 and total >= step
    out, _ = c.run()
    want = 1 / (1 + np.exp(-scale * total))
    tol = 32 * U * want + HALF[type_] * np.exp2(np.floor(np.log2(want)))
    assert 0.55 < want < 0.95
    off = np.abs(out.double().numpy() - want) / tol
    assert off.max() <= 1, off.max()
