"""Log probabilities, ranks, entropies and likeliest tokens on the GPU against the definition in 64 bits.

Whole numbers are equal. With u = 2^-24 and d the scaled distance of a logit to its row's largest, an
exponential is off by at most (3 |d| + 4) u of itself (the difference, the scale's product and the constant's
rounding, the instruction), so their sum by (3 sum p |d| + 4 + n) u, n the longest chain of additions and
rescalings, and sum p |d| by (3 sum p d^2 + (7 + n) sum p |d|) u. A logarithm of 1 to 2^30 adds 3 u of itself
and the results' own roundings a few u of the numbers they are made of."""
import numpy as np
import pytest

import prompt_reference as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


def call(pn, torch, logits, tokens, scale, top, fill=0xA5, stream=None):
    R, V = logits.shape
    dev = logits.device
    got = dict(logprob=torch.full((R,), 5.0, device=dev), rank=torch.full((R,), 5, dtype=torch.int32, device=dev),
               entropy=torch.full((R,), 5.0, device=dev), lse=torch.full((R,), 5.0, device=dev))
    if top:
        got.update(top_ids=torch.full((R, top), 5, dtype=torch.int32, device=dev),
                   top_logprobs=torch.full((R, top), 5.0, device=dev))
    work = torch.full((pn.logprobs_workspace_bytes(R, V, top) + 16,), fill, dtype=torch.uint8, device=dev)
    pn.logprobs(logits, tokens, workspace=work, scale=scale, stream=stream, **got)
    return got


def same(got, x, tokens, scale, top):
    """got's tensors against x's rows in 64 bits."""
    scale = float(np.float32(scale))
    want = ref.logprobs(x, tokens, scale, top)
    R, V = x.shape
    chain = V / 64 + 60  # at least 64 lanes share a row; joins
    sum_err = U * (3 * want["away"] + 4 + chain)
    tail = U * 30
    with np.errstate(all="ignore"):
        size = np.abs(np.where(np.isfinite(want["logprob"]), want["logprob"], 0.0))
        bounds = {"logprob": sum_err + tail + 6 * U * (size + 25),
                  "entropy": sum_err + tail + U * (3 * want["away2"] + (chain + 12) * want["away"] + 80),
                  "lse": sum_err + tail + 4 * U * (np.abs(np.nan_to_num(want["lse"], posinf=0, neginf=0))
                                                   + np.abs(scale * np.nanmax(np.where(np.isfinite(x), x, 0), 1)) + 25)}
        for name, bound in bounds.items():
            g, w = got[name].double().cpu().numpy(), want[name]
            fine = np.isfinite(w)
            assert (np.isnan(g) == np.isnan(w)).all(), name
            assert (g[~fine & ~np.isnan(w)] == w[~fine & ~np.isnan(w)]).all(), name
            err = np.abs(g - w)[fine]
            assert (err <= bound[fine]).all(), (name, (err / bound[fine]).max())
    assert (got["rank"].cpu().numpy() == want["rank"]).all()
    if top:
        assert (got["top_ids"].cpu().numpy() == want["top_ids"]).all()
        g, w = got["top_logprobs"].double().cpu().numpy(), want["top_logprobs"]
        assert (np.isnan(g) == np.isnan(w)).all()
        fine = np.isfinite(w)
        assert (g[~fine & ~np.isnan(w)] == w[~fine & ~np.isnan(w)]).all()
        bound = (sum_err + tail)[:, None] + 6 * U * (np.abs(np.where(fine, w, 0.0)) + 25)
        assert (np.abs(np.where(fine, g - w, 0.0)) <= bound).all()


def check(env, x, type_, scale=1.0, top=5, tokens=None, seed=0, place=None):
    pn, torch, dev = env
    rng = np.random.default_rng(seed)
    t = torch.from_numpy(np.asarray(x, np.float32)).to(getattr(torch, type_))
    R, V = t.shape
    if tokens is None:
        tokens = rng.integers(0, V, size=R)
    tokens = np.asarray(tokens, np.int32)
    logits = place(t) if place else t.to(dev)
    got = call(pn, torch, logits, torch.from_numpy(tokens).to(dev), scale, top)
    torch.cuda.synchronize()
    same(got, t.double().numpy(), tokens, scale, top)


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 255, 1000, 1023, 1024, 1025, 2048, 2049, 4096, 4097, 9000, 32003])
def test_vocabularies(env, type_, V):
    rng = np.random.default_rng(V)
    check(env, 3 * rng.normal(size=(5, V)), type_, top=min(V, 20))


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,V", [(1, 248320), (2, 248321), (70, 20011), (600, 4099), (1100, 2100), (2100, 1500)])
def test_rows(env, type_, R, V):
    rng = np.random.default_rng(V)
    check(env, 3 * rng.normal(size=(R, V)), type_, top=20)


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,V", [(1, 1200007), (2, 8193), (3, 16385), (3, 32769), (128, 20001), (129, 20001), (256, 16384),
                                 (256, 16385), (257, 9001), (257, 131073), (341, 65537), (342, 65537), (512, 8193), (513, 8193)])
def test_rows_at_the_cuts(env, type_, R, V):
    """Rows shared by many, two and no workgroups, of four, eight and 16 waves."""
    rng = np.random.default_rng(R)
    check(env, 3 * rng.normal(size=(R, V)), type_, top=5)
    check(env, 3 * rng.normal(size=(R, V)), type_, top=0)


@pytest.mark.parametrize("top", [0, 1, 2, 7, 8, 9, 32, 63, 64])
@pytest.mark.parametrize("V", [5, 64, 3000, 50001])
def test_top(env, top, V):
    rng = np.random.default_rng(top)
    check(env, 3 * rng.normal(size=(3, V)), "float32", top=top)


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [900, 30000, 140001])
def test_order(env, type_, V):
    """Rows that rise, fall, are constant, have few values, and have their largest at the ends."""
    rng = np.random.default_rng(1)
    x = np.zeros((8, V))
    x[0] = np.linspace(-20, 20, V)
    x[1] = x[0, ::-1]
    x[2] = 1.5
    x[3] = rng.integers(0, 3, size=V)
    x[4, 0], x[5, V - 1] = 9.0, 9.0
    x[6] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    x[7] = np.repeat(np.arange(-(-V // 64)), 64)[:V] % 100 * 0.25  # lanes' neighbours are equal
    check(env, x, type_, top=64)
    check(env, x, type_, top=3)


@pytest.mark.parametrize("type_", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("V", [70, 5000, 70000])
def test_masks_and_numbers_that_are_not_finite(env, type_, V):
    rng = np.random.default_rng(4)
    x = 3 * rng.normal(size=(12, V))
    low = {"float32": -3.4028234663852886e38, "bfloat16": -3.3895313892515355e38, "float16": -65504.0}[type_]
    x[0, rng.random(V) < 0.95] = -np.inf
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, V // 3] = 2.0                 # one token alone
    x[3, rng.random(V) < 0.9] = low    # masks of the type's lowest number
    x[4] = low
    x[5, V // 2] = np.nan
    x[6, V - 1] = np.inf
    x[7, [3, V // 2]] = np.inf
    x[8] = np.nan
    x[9, :V // 2] = -np.inf            # whole batches without a token
    x[10, V // 2:] = -np.inf
    x[11, 0] = -low                    # the largest number
    tokens = rng.integers(0, V, size=12)
    tokens[0] = int(np.nonzero(x[0] > -np.inf)[0][0])
    tokens[2] = V // 3
    tokens[9] = 0                      # one that is masked
    tokens[11] = 0
    check(env, x, type_, top=20, tokens=tokens)
    check(env, x, type_, top=20, tokens=np.where(np.arange(12) % 2, -1, V))
    check(env, x, type_, top=0, tokens=np.full(12, -(1 << 31)))


@pytest.mark.parametrize("scale", [1e-30, 0.1, 0.7, 3.0, 1e4, 1e30])
def test_scales(env, scale):
    rng = np.random.default_rng(5)
    check(env, 2 * rng.normal(size=(4, 7001)), "float32", scale=scale, top=5)


def test_far_logits(env):
    """Rows whose logits lie far from zero, and far apart."""
    rng = np.random.default_rng(6)
    x = np.float64(np.float32(rng.normal(size=(4, 9001))))
    x[0] += 1000.0
    x[1] -= 30000.0
    x[2] *= 1e4
    x[3] *= 1e30
    check(env, x, "float32", top=10)


@pytest.mark.parametrize("type_", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (3, 2), (64, 0)])
def test_strided_and_unaligned(env, type_, pad, off):
    """Rows as slices of a padded vocabulary: what lies past their end is not looked at."""
    pn, torch, dev = env
    rng = np.random.default_rng(7)

    def place(t):
        R, V = t.shape
        wide = torch.full((R * (V + pad) + off + 8,), 1e30, dtype=t.dtype, device=dev)
        view = wide[off:off + R * (V + pad)].view(R, V + pad)[:, :V]
        view.copy_(t)
        return view
    check(env, 3 * rng.normal(size=(3, 5003)), type_, place=place)
    check(env, 3 * rng.normal(size=(3, 30001)), type_, place=place)


def test_outputs_left_out(env):
    pn, torch, dev = env
    x = torch.randn(3, 9000, device=dev)
    tokens = torch.tensor([4, 5, 6], dtype=torch.int32, device=dev)
    full = call(pn, torch, x, tokens, 1.0, 4)
    work = torch.empty(pn.logprobs_workspace_bytes(3, 9000, 4), dtype=torch.uint8, device=dev)
    for name in ("logprob", "rank", "entropy", "lse"):
        one = {name: torch.empty_like(full[name])}
        pn.logprobs(x, tokens if name in ("logprob", "rank") else None, workspace=work, **one)
        torch.cuda.synchronize()
        assert torch.equal(one[name], full[name])
    ids, lp = torch.empty_like(full["top_ids"]), torch.empty_like(full["top_logprobs"])
    pn.logprobs(x, workspace=work, top_ids=ids, top_logprobs=lp)
    torch.cuda.synchronize()
    assert torch.equal(ids, full["top_ids"]) and torch.equal(lp, full["top_logprobs"])


def test_large_offsets(env):
    """Rows past 2^31 elements."""
    pn, torch, dev = env
    R, V = 9000, 248320
    x = torch.empty(R, V, dtype=torch.bfloat16, device=dev)  # 4.5 GB
    x.copy_(torch.randn(V, device=dev))
    x[R - 1, 77] = 50.0
    tokens = torch.full((R,), 77, dtype=torch.int32, device=dev)
    got = call(pn, torch, x, tokens, 1.0, 3)
    torch.cuda.synchronize()
    rows = [0, 1, R - 2, R - 1]
    same({k: v[rows] for k, v in got.items()}, x[rows].double().cpu().numpy(), np.full(4, 77), 1.0, 3)
    assert bool((got["top_ids"][:-1] == got["top_ids"][0]).all()) and bool((got["entropy"][:-1] == got["entropy"][0]).all())


def test_the_same_bits_each_time(env):
    pn, torch, dev = env
    x = torch.randn(3, 200003, device=dev)
    tokens = torch.zeros(3, dtype=torch.int32, device=dev)
    first = call(pn, torch, x, tokens, 1.0, 20)
    for n in range(5):
        again = call(pn, torch, x, tokens, 1.0, 20, fill=n)
        torch.cuda.synchronize()
        for name in first:
            assert torch.equal(first[name], again[name]), name


def test_graphs_that_share_a_workspace(env):
    pn, torch, dev = env
    sizes = [(1, 60000, 20), (5, 9001, 3), (2, 248320, 64)]
    need = max(pn.logprobs_workspace_bytes(*s) for s in sizes)
    work = torch.randint(0, 256, (need,), dtype=torch.uint8, device=dev)
    made = []
    for R, V, top in sizes:
        x, tokens = torch.randn(R, V, device=dev), torch.zeros(R, dtype=torch.int32, device=dev)
        out = dict(logprob=torch.empty(R, device=dev), entropy=torch.empty(R, device=dev),
                   rank=torch.empty(R, dtype=torch.int32, device=dev), lse=torch.empty(R, device=dev),
                   top_ids=torch.empty(R, top, dtype=torch.int32, device=dev), top_logprobs=torch.empty(R, top, device=dev))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pn.logprobs(x, tokens, workspace=work, **out)
        made.append((graph, x, tokens, out, top))
    side = torch.cuda.Stream()
    for n in range(4):
        for graph, x, tokens, out, top in made:
            x.copy_(torch.randn_like(x) * 3)
            tokens += 11
            graph.replay()
            side.wait_stream(torch.cuda.current_stream())
            again = call(pn, torch, x, tokens, 1.0, top, fill=n, stream=side)
            torch.cuda.synchronize()
            for name in out:
                assert torch.equal(out[name], again[name]), name
            same(out, x.double().cpu().numpy(), tokens.cpu().numpy(), 1.0, top)


def test_empty_and_refusals(env):
    pn, torch, dev = env
    x, tokens = torch.zeros(3, 9000, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    s, ids = torch.zeros(3, device=dev), torch.zeros(3, 4, dtype=torch.int32, device=dev)
    work = torch.zeros(pn.logprobs_workspace_bytes(3, 9000, 4), dtype=torch.uint8, device=dev)
    pn.logprobs(x[:0], tokens[:0], s[:0])
    for a in (dict(logprob=s), dict(rank=tokens), dict(tokens=tokens.long(), logprob=s), dict(entropy=s[:2]),
              dict(top_ids=ids), dict(top_ids=ids, top_logprobs=ids), dict(top_ids=ids[0], top_logprobs=s),
              dict(lse=s.double()), dict(entropy=s.cpu())):
        with pytest.raises(ValueError):
            pn.logprobs(x, workspace=work, **a)
    for bad in (x[0], x.double(), x.t(), x.cpu()):
        with pytest.raises(ValueError):
            pn.logprobs(bad, entropy=s, workspace=work)
    wide = torch.zeros(3, 65, dtype=torch.int32, device=dev)
    for a in (dict(entropy=s, scale=0.0, workspace=work), dict(entropy=s, scale=-1.0, workspace=work), dict(entropy=s),
              dict(top_ids=wide, top_logprobs=wide.float(), workspace=work), dict(entropy=s, workspace=work[:64])):
        with pytest.raises(pn.PNError):
            pn.logprobs(x, **a)
