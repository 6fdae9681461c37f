"""Verification of drafted tokens on the GPU against the definition in 64 bits: the same tokens."""
import numpy as np
import pytest

import step_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_quantized_weight_pn3t_amd as pn
    return pn, torch, torch.device("cuda:0")


def run(env, p, q, draft, ua, us, n_draft=None):
    pn, torch, dev = env

    def up(a):
        return a if a is None or torch.is_tensor(a) else torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    B, K = draft.shape
    tokens = torch.full((B, K + 1), -99, dtype=torch.int32, device=dev)
    accepted = torch.full((B,), -99, dtype=torch.int32, device=dev)
    p = up(p)
    work = torch.full((pn.verify_workspace_bytes(B, p.shape[2]),), 0xFF, dtype=torch.uint8, device=dev)
    pn.verify(p, up(q), up(draft), up(ua), up(us), tokens, accepted, work, n_draft=up(n_draft))
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), accepted.cpu().numpy()


def check(env, p, q, draft, ua, us, n_draft=None):
    pn, torch, dev = env
    host = [x.float().cpu().numpy() if torch.is_tensor(x) else x for x in (p, q)]
    want = ref.verify(host[0], host[1], draft, ua, us, n_draft)
    got = run(env, p, q, draft, ua, us, n_draft)
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[0], want[0]), (got[0], want[0])
    return got


def inputs(torch, dev, seed, B, K, V, dtype, certain=False, near=0.5):
    rng = np.random.default_rng(seed)
    x = 2.5 * rng.normal(size=(B, K + 1, V))
    y = x[:, :K] + near * rng.normal(size=(B, K, V))

    def soft(z):
        e = np.exp(z - z.max(-1, keepdims=True)) if z.size else z
        return torch.from_numpy((e / e.sum(-1, keepdims=True) if z.size else e).astype(np.float32)).to(dtype)
    p, q = soft(x), soft(y)
    draft = np.zeros((B, K), np.int32)
    for b in range(B):
        for i in range(K):
            w = q[b, i].double().numpy()
            draft[b, i] = rng.choice(V, p=w / w.sum()) if not certain or rng.random() < 0.3 else int(p[b, i].argmax())
    return (p.to(dev), None if certain else q.to(dev), draft, rng.random((B, K)).astype(np.float32),
            rng.random(B).astype(np.float32))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("B,K,V", [(1, 0, 5), (1, 1, 1), (2, 3, 2), (5, 4, 255), (3, 8, 2047), (4, 2, 2048),
                                   (4, 3, 2049), (2, 5, 32003), (17, 1, 4096), (1, 63, 300)])
def test_tokens(env, dtype, certain, B, K, V):
    pn, torch, dev = env
    for near in (0.1, 1.5):
        args = inputs(torch, dev, B * 1000 + K + V, B, K, V, getattr(torch, dtype), certain, near)
        check(env, *args)


def test_large_vocabulary(env):
    pn, torch, dev = env
    check(env, *inputs(torch, dev, 5, 3, 2, 248320, torch.float32))


def test_fewer_drafts_than_places(env):
    pn, torch, dev = env
    p, q, draft, ua, us = inputs(torch, dev, 7, 6, 4, 3001, torch.float32, near=0.05)
    for certain in (False, True):
        n = np.array([0, 1, 2, 3, 4, 4], np.int32)
        check(env, p, None if certain else q, draft, ua, us, n)
    a = run(env, p, q, draft, ua, us, np.array([-3, 9, 4, 4, 4, 4], np.int32))
    b = run(env, p, q, draft, ua, us, np.array([0, 4, 4, 4, 4, 4], np.int32))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_edges_of_the_random_numbers(env):
    """u = 0 accepts wherever p is positive and draws the first token with any weight; u near 1 the last."""
    pn, torch, dev = env
    p, q, draft, ua, us = inputs(torch, dev, 8, 4, 2, 5000, torch.float32)
    p[:, :, :7] = 0.0
    p[:, :, -9:] = 0.0
    below = np.float32(np.nextafter(np.float32(1), np.float32(0)))
    for u in (0.0, below):
        for w in (0.0, below):
            check(env, p, q, draft, np.full_like(ua, u), np.full_like(us, w))
    # a draw past the sum takes the last token with weight
    tokens, accepted = run(env, p, None, draft, np.zeros_like(ua) - 1, np.ones_like(us) + 1)
    assert (accepted == 2).all() and (tokens[:, 2] == 4990).all()


def test_rows_that_hold_nothing(env):
    """q = p leaves no residual: the draw is from p; p of zeros: no token; NaN and negative numbers count
    as zero."""
    pn, torch, dev = env
    p, _, draft, ua, us = inputs(torch, dev, 9, 3, 2, 2500, torch.float32)
    one = np.full_like(ua, 1.0)
    check(env, p, p[:, :2].clone(), draft, one, us)
    zero = torch.zeros_like(p)
    tokens, accepted = check(env, zero, p[:, :2].clone(), draft, ua, us)
    assert (accepted == 0).all() and (tokens == -1).all()
    odd = p.clone()
    odd[:, :, 100:1300] = float("nan")
    odd[:, :, 1300:1400] = -1.0
    draft[0, 0] = 200
    check(env, odd, p[:, :2].clone(), draft, ua, us)
    check(env, odd, None, draft, ua, us)
    q = p[:, :2].clone()
    q[:, :, 5:900] = float("nan")
    check(env, p, q, draft, ua, us)


def test_drafts_that_are_no_tokens(env):
    pn, torch, dev = env
    p, q, draft, ua, us = inputs(torch, dev, 10, 4, 3, 700, torch.float32, near=0.01)
    draft[:, 1] = [-1, 700, 1 << 30, -(1 << 31)]
    got = check(env, p, q, draft, ua * 0, us)
    assert (got[1] == 1).all()
    check(env, p, None, draft, ua * 0, us)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_padded_rows(env, dtype, pad):
    """Rows spaced wider than the vocabulary, by odd amounts too; what lies between is not read as
    probability."""
    pn, torch, dev = env
    p, q, draft, ua, us = inputs(torch, dev, 11, 3, 2, 4097, getattr(torch, dtype))

    def wide(x):
        w = torch.full((*x.shape[:2], x.shape[2] + pad), float("inf"), dtype=x.dtype, device=dev)
        w[..., :x.shape[2]] = x
        return w[..., :x.shape[2]]
    check(env, wide(p), wide(q), draft, ua, us)


def test_repeated_calls_and_graph(env):
    pn, torch, dev = env
    p, q, draft, ua, us = inputs(torch, dev, 12, 4, 3, 9001, torch.float32)
    want = ref.verify(p.cpu().numpy(), q.cpu().numpy(), draft, ua, us)
    tokens = torch.zeros(4, 4, dtype=torch.int32, device=dev)
    accepted = torch.zeros(4, dtype=torch.int32, device=dev)
    work = torch.empty(pn.verify_workspace_bytes(4, 9001), dtype=torch.uint8, device=dev)
    d, a, s = (torch.from_numpy(x).to(dev) for x in (draft, ua, us))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pn.verify(p, q, d, a, s, tokens, accepted, work, stream=st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pn.verify(p, q, d, a, s, tokens, accepted, work, stream=st)
    for rep in range(4):
        tokens.fill_(-5)
        accepted.fill_(-5)
        work.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])


def test_binding_refusals(env):
    pn, torch, dev = env
    p, q, draft, ua, us = inputs(torch, dev, 13, 2, 3, 100, torch.float32)
    tokens = torch.zeros(2, 4, dtype=torch.int32, device=dev)
    accepted = torch.zeros(2, dtype=torch.int32, device=dev)
    work = torch.empty(pn.verify_workspace_bytes(2, 100), dtype=torch.uint8, device=dev)
    good = [p, q, *(torch.from_numpy(x).to(dev) for x in (draft, ua, us)), tokens, accepted, work]
    pn.verify(*good)
    for i, x in ((0, p.double()), (0, p[:, :3]), (0, p.transpose(1, 2)), (0, p.cpu()), (1, q.half()), (1, q[:, :2]),
                 (2, good[2].long()), (3, good[3][:, :2].contiguous()), (4, good[4].double()), (5, tokens[:, :3]),
                 (6, accepted[:1]), (7, work[:-1])):
        bad = list(good)
        bad[i] = x
        with pytest.raises((ValueError, pn.PNError)):
            pn.verify(*bad)
    torch.cuda.synchronize()
